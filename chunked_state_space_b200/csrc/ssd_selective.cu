// The selective scan with a step per channel, for prompts and single tokens:
//   s = softplus(dt + bias);  h[n] = e^{s A[c,n]} h[n] + s B[n] x
//   y = (sum_n C[n] h[n] + D x) silu(z)
//
// With a decay per state entry and a step per channel there is no matrix
// product in it: N exponentials and 4 N fp32 operations per token and channel.
// At N = 16 that is 20 special-function operations (two each for softplus and
// silu) at 16 per clock and SM against 8 bytes of bf16, so a prompt is bound by
// the exponentials, at about four times its HBM time.  One token is bound by
// its f32 state, read and written once.
//
// Prompt: a channel's entries lie on LPC lanes of a warp, NS to a lane, in
// registers over the whole sequence; a block takes 128 / LPC channels of one
// group.  Its inputs come tile by tile: the next tile's rows are loaded into
// registers while this one is computed; step and scaled input are formed once
// per (token, channel) and put in shared memory; B and C are widened to f32 once per tile.
#include <limits.h>

#include "ssd_rows.cuh"

namespace ssd {
namespace selective {

// of a block: lanes of the recurrence, and two teams of helpers (operands in, outputs out)
constexpr int LANES = 128, HELPERS = 64, THREADS = LANES + 2 * HELPERS;
constexpr int64_t SCHEDULERS = 4 * 148;  // warp schedulers of the GPU

template <typename T>
struct Args {
  Rows<const T> x, dt, z, bm, cm;
  Rows<T> y;
  const float *A, *D, *dt_bias;
  const float* init;
  float* final_state;
  const int32_t* lengths;
  int64_t L;
  int C, N, G, per_group;
  uint32_t blocks_per_group, total;
  bool softplus, vec, bvec;
};

// max(v, 0) + log1p(e^-|v|).  The exponent's rounding is put back to first
// order, so that small steps keep f32 accuracy; log1p(e) = e P(e) with P the
// minimax polynomial of degree 8 of log1p(e) / e on [0, 1] (Remez exchange,
// P(0) = 1; at most 1.8e-7 off, relative, evaluated in f32).
__device__ __forceinline__ F2 softplus2(F2 v) {
  const F2 m{-fabsf(v.x), -fabsf(v.y)}, t = mul2(m, both(LOG2E));
  const F2 p{ex2(t.x), ex2(t.y)};
  const F2 lost = mul2(fma2(m, both(LOG2E), F2{-t.x, -t.y}), both(0.69314718f));
  const F2 e = fma2(p, lost, p);
  F2 q = both(0.0053648264f);
  q = fma2(q, e, both(-0.030065801f));
  q = fma2(q, e, both(0.07920455f));
  q = fma2(q, e, both(-0.13753803f));
  q = fma2(q, e, both(0.19153656f));
  q = fma2(q, e, both(-0.24857163f));
  q = fma2(q, e, both(0.33321324f));
  q = fma2(q, e, both(-0.49999648f));
  q = fma2(q, e, both(1.0f));
  return fma2(q, e, F2{v.x < 0.f ? 0.f : v.x, v.y < 0.f ? 0.f : v.y});  // v, not max(v, 0): NaN stays
}
__device__ __forceinline__ float softplus(float v) { return softplus2(both(v)).x; }

template <typename T, int NS, int LPC, bool VEC, bool BVEC>
struct Shape {
  static constexpr int CB = LANES / LPC;                       // channels of a block
  static constexpr int NP = NS * LPC;                      // state entries, the last ones empty where N is less
  static constexpr int V = VEC ? 16 / (int)sizeof(T) : 1;   // elements per load of x, dt, z and per store of y
  static constexpr int VB = BVEC ? 16 / (int)sizeof(T) : 1;  // ... per load of B, C
  // tokens of a tile: eight elements of x per helper thread, fewer where B and C would not leave room (in shared
  // memory, or in registers as single elements)
  static constexpr int TT = NP <= 16 ? 8 * HELPERS / CB : NP == 32 ? (BVEC ? 32 : 16) : NP == 64 ? (BVEC ? 16 : 8) : 8;
  static constexpr int XP = TT * CB / V, BP = TT * NP / VB;        // pieces of a tile of x (dt, z), of B (C)
  static constexpr int APART = HELPERS / (CB / V);                 // tokens between the pieces of a thread
  // B and C of an entry lie side by side: two bf16 in a word (half the shared-memory traffic, which would bound the
  // kernel, for two instructions more per entry), or two f32
  static constexpr int WORDS = sizeof(T) == 2 ? 1 : 2;
  static constexpr int NX = (XP + HELPERS - 1) / HELPERS;          // of them, per helper thread
  static constexpr int NB = (BP + HELPERS - 1) / HELPERS;
  // y's sums over the states are left in PW parts per (token, channel), which the output pass adds up; more lanes than
  // that exchange theirs first, RED tokens together, each exchange halving what a lane still holds.
  static constexpr int PW = LPC < 4 ? LPC : 4, RED = LPC / PW;
  static constexpr int U = RED < 2 ? 2 : RED;  // tokens that a lane works on together
  static constexpr int ROWS = TT + 2 * U;      // rows of operands: a tile, and what the loop reads behind it for nothing
  static_assert(TT % (2 * U) == 0, "a tile is a whole number of turns of its loop");
  static_assert(NP % VB == 0 && CB % V == 0 && HELPERS % (CB / V) == 0, "rows of a tile are whole pieces");
  // Where (token, channel) lies in a tile of 8-byte entries: a thread writes V neighbouring channels, two per
  // instruction, so its pairs are turned by the piece's number to fall on different banks; the channels that a warp
  // reads together share the turn or lie in different pieces.
  __device__ static __forceinline__ int at(int t, int ch) {
    const int i = t * (CB / V) + ch / V;
    const int turn = V == 8 ? (i >> 1) & 3 : V == 4 ? (i >> 2) & 1 : 0;
    return t * CB + (ch ^ (turn << 1));
  }
  // The same for entries of PW f32 (up to 16 bytes), which a thread reads one per instruction.
  __device__ static __forceinline__ int sum_at(int t, int ch) {
    const int i = t * (CB / V) + ch / V;
    return (t * CB + (ch ^ (V == 8 ? i & 7 : V == 4 ? (i >> 1) & 3 : 0))) * PW;
  }
};

// The block's barriers beside __syncthreads(): FULL + k, the operands of
// buffer k are written and its sums have been taken; DONE + k, its operands
// have been used and its sums are written.  Every thread of the block takes
// part in each of them once per tile, waiting or only arriving.
enum { FULL = 1, DONE = 3 };
__device__ __forceinline__ void wait_for(int bar) { asm volatile("bar.sync %0, %1;" ::"r"(bar), "n"(THREADS) : "memory"); }
__device__ __forceinline__ void arrive_at(int bar) {
  asm volatile("bar.arrive %0, %1;" ::"r"(bar), "n"(THREADS) : "memory");
}

template <typename T, int NS, int LPC, bool VEC, bool BVEC>
__global__ void __launch_bounds__(THREADS, NS * LPC <= 16 && VEC && BVEC ? 3 : 2) k_selective(const Args<T> a) {
  using S = Shape<T, NS, LPC, VEC, BVEC>;
  constexpr int CB = S::CB, NP = S::NP, V = S::V, VB = S::VB, TT = S::TT, XP = S::XP, BP = S::BP, NX = S::NX, NB = S::NB,
                PW = S::PW, RED = S::RED, U = S::U, ROWS = S::ROWS, WORDS = S::WORDS, APART = S::APART;
  __shared__ __align__(16) float2 s_step[2][ROWS * CB];    // (s, s x)
  __shared__ __align__(16) uint32_t s_bc[2][ROWS * NP * WORDS];  // (B, C)
  __shared__ __align__(16) float s_y[2][TT * CB * PW];
  __shared__ __align__(16) float s_D[CB], s_bias[CB];
  const uint32_t r = blockIdx.x / a.blocks_per_group, cb = blockIdx.x - r * a.blocks_per_group;
  const uint32_t b = r / a.G, g = r - b * a.G;
  const int c0 = (int)g * a.per_group + (int)cb * CB;  // first channel of the block
  const int nc = min(CB, ((int)g + 1) * a.per_group - c0);
  const int tid = threadIdx.x;
  const int64_t len = row_length(a.lengths, b, a.L);
  const int tiles = (int)((len + TT - 1) / TT);
  for (int i = tid; i < CB; i += THREADS) {
    s_D[i] = a.D && i < nc ? a.D[c0 + i] : 0.f;
    s_bias[i] = a.dt_bias && i < nc ? a.dt_bias[c0 + i] : 0.f;
  }
  __syncthreads();

  if (tid >= LANES + HELPERS) {
    // ---- output: add up the sums, skip and gate, store
    const int me = tid - LANES - HELPERS;
    const bool gate = a.z.p != nullptr;
    for (int k = 0; k < 2 && k < tiles; ++k) arrive_at(FULL + k);
    // piece k of a thread: token t0 + k * APART of the tile, channels c ..
    const int t0 = me / (CB / V), c = me % (CB / V) * V;
    const T* px = a.x.row(b, t0) + c0 + c;
    const T* pz = gate ? a.z.row(b, t0) + c0 + c : px;
    T* py = a.y.row(b, t0) + c0 + c;
    Pack<T, V> nx[NX], nz[NX];
    auto fetch = [&](int left) {  // tokens of the sequence from this tile on
#pragma unroll
      for (int k = 0; k < NX; ++k) {
        if (me + k * HELPERS < XP && t0 + k * APART < left && c < nc) {
          nx[k] = load_pack<T, V>(px + k * APART * a.x.ts);
          if (gate) nz[k] = load_pack<T, V>(pz + k * APART * a.z.ts);
        }
      }
      px += TT * a.x.ts;
      pz += TT * a.z.ts;
    };
    int left = (int)min(len, (int64_t)INT_MAX);
    fetch(left);
#pragma unroll 1
    for (int tile = 0; tile < tiles; ++tile) {
      const int k2 = tile & 1;
      Pack<T, V> x[NX], z[NX];
#pragma unroll
      for (int k = 0; k < NX; ++k) x[k] = nx[k], z[k] = nz[k];
      if (tile + 1 < tiles) fetch(left - TT);
      wait_for(DONE + k2);
      // sums of channels c + e and, where two are asked for, c + e + 1
      auto sums = [&](int t, int e) {
        const float* p = &s_y[k2][S::sum_at(t, c + e)];
        const float* r = &s_y[k2][S::sum_at(t, V > 1 ? c + e + 1 : c + e)];
        if constexpr (PW == 4) {
          const float4 v = *reinterpret_cast<const float4*>(p), w = *reinterpret_cast<const float4*>(r);
          const F2 f = add2(F2{v.x, v.y}, F2{v.z, v.w}), g = add2(F2{w.x, w.y}, F2{w.z, w.w});
          return F2{f.x + f.y, g.x + g.y};
        } else {
          const float2 v = *reinterpret_cast<const float2*>(p), w = *reinterpret_cast<const float2*>(r);
          return F2{v.x + v.y, w.x + w.y};
        }
      };
#pragma unroll
      for (int k = 0; k < NX; ++k) {
        const int t = t0 + k * APART;
        if (me + k * HELPERS < XP && t < left && c < nc) {
          float out[V];
          if constexpr (V == 1) {
            out[0] = fmaf(s_D[c], x[k].get(0), sums(t, 0).x);
            if (gate) out[0] *= silu(z[k].get(0));
          } else {
#pragma unroll
            for (int e = 0; e < V; e += 2) {
              F2 y = fma2(F2{s_D[c + e], s_D[c + e + 1]}, F2{x[k].get(e), x[k].get(e + 1)}, sums(t, e));
              if (gate) y = mul2(y, silu2(F2{z[k].get(e), z[k].get(e + 1)}));
              out[e] = y.x, out[e + 1] = y.y;
            }
          }
          store_pack<T, V>(py + k * APART * a.y.ts, to_pack<T, V>(out));
        }
      }
      py += TT * a.y.ts;
      left -= TT;
      if (tile + 2 < tiles) arrive_at(FULL + k2);
    }
    return;
  }

  if (tid >= LANES) {
    // ---- operands: the step and the scaled input of every (token, channel), B and C
    const int me = tid - LANES;
    const int t0 = me / (CB / V), c = me % (CB / V) * V;
    const T* px = a.x.row(b, t0) + c0 + c;
    const T* pd = a.dt.row(b, t0) + c0 + c;
    const T* pb = a.bm.row(b, 0) + (int64_t)g * a.N;
    const T* pc = a.cm.row(b, 0) + (int64_t)g * a.N;
    Pack<T, V> nx[NX], nd[NX];
    Pack<T, VB> nb[NB], nc2[NB];
    auto fetch = [&](int left) {
#pragma unroll
      for (int k = 0; k < NX; ++k) {
        if (me + k * HELPERS < XP && t0 + k * APART < left && c < nc) {
          nx[k] = load_pack<T, V>(px + k * APART * a.x.ts);
          nd[k] = load_pack<T, V>(pd + k * APART * a.dt.ts);
        }
      }
#pragma unroll
      for (int k = 0; k < NB; ++k) {
        const int i = me + k * HELPERS, t = i / (NP / VB), n = i % (NP / VB) * VB;
        if (i < BP && t < left && n < a.N) {
          nb[k] = load_pack<T, VB>(pb + t * a.bm.ts + n);
          nc2[k] = load_pack<T, VB>(pc + t * a.cm.ts + n);
        }
      }
      px += TT * a.x.ts;
      pd += TT * a.dt.ts;
      pb += TT * a.bm.ts;
      pc += TT * a.cm.ts;
    };
    int left = (int)min(len, (int64_t)INT_MAX);
    fetch(left);
#pragma unroll 1
    for (int tile = 0; tile < tiles; ++tile) {
      const int k2 = tile & 1;
      if (tile >= 2) wait_for(DONE + k2);
      // behind the sequence's end the step is 0, which leaves the state as it is
#pragma unroll
      for (int k = 0; k < NX; ++k) {
        const int t = t0 + k * APART;
        if (me + k * HELPERS < XP) {
          const bool in = t < left && c < nc;
          if constexpr (V == 1) {
            float s = 0.f, sx = 0.f;
            if (in) {
              s = nd[k].get(0) + s_bias[c];
              if (a.softplus) s = softplus(s);
              sx = s * nx[k].get(0);
            }
            s_step[k2][S::at(t, c)] = make_float2(s, sx);
          } else {
            F2 s[V / 2], sx[V / 2];
            if (in) {
#pragma unroll
              for (int e = 0; e < V; e += 2)
                s[e / 2] = add2(F2{nd[k].get(e), nd[k].get(e + 1)}, F2{s_bias[c + e], s_bias[c + e + 1]});
              if (a.softplus) {
#pragma unroll
                for (int e = 0; e < V; e += 2) s[e / 2] = softplus2(s[e / 2]);
              }
#pragma unroll
              for (int e = 0; e < V; e += 2) sx[e / 2] = mul2(s[e / 2], F2{nx[k].get(e), nx[k].get(e + 1)});
            } else {
#pragma unroll
              for (int e = 0; e < V; e += 2) s[e / 2] = sx[e / 2] = both(0.f);
            }
#pragma unroll
            for (int e = 0; e < V; e += 2)
              *reinterpret_cast<float4*>(&s_step[k2][S::at(t, c + e)]) =
                  make_float4(s[e / 2].x, sx[e / 2].x, s[e / 2].y, sx[e / 2].y);
          }
        }
      }
#pragma unroll
      for (int k = 0; k < NB; ++k) {
        const int i = me + k * HELPERS, t = i / (NP / VB), n = i % (NP / VB) * VB;
        if (i < BP) {
          const bool in = t < left && n < a.N;
          uint32_t w[VB * WORDS];
#pragma unroll
          for (int e = 0; e < VB; ++e) {
            const uint32_t bw = in ? __float_as_uint(nb[k].get(e)) : 0u, cw = in ? __float_as_uint(nc2[k].get(e)) : 0u;
            if constexpr (WORDS == 1)
              w[e] = __byte_perm(bw, cw, 0x7632);
            else
              w[2 * e] = bw, w[2 * e + 1] = cw;
          }
          uint32_t* to = &s_bc[k2][i * VB * WORDS];
          if constexpr (VB * WORDS % 4 == 0) {
#pragma unroll
            for (int e = 0; e < VB * WORDS; e += 4)
              *reinterpret_cast<uint4*>(to + e) = make_uint4(w[e], w[e + 1], w[e + 2], w[e + 3]);
          } else {
#pragma unroll
            for (int e = 0; e < VB * WORDS; ++e) to[e] = w[e];
          }
        }
      }
      left -= TT;
      arrive_at(FULL + k2);
      if (tile + 1 < tiles) fetch(left);
    }
    for (int tile = tiles > 2 ? tiles - 2 : 0; tile < tiles; ++tile) arrive_at(DONE + (tile & 1));
    return;
  }

  // ---- the recurrence
  const int q = tid % LPC, ch = tid / LPC;
  float A2[NS], h[NS];
#pragma unroll
  for (int k = 0; k < NS; ++k) {
    const int n = q * NS + k;
    const bool in = ch < nc && n < a.N;
    A2[k] = in ? a.A[(int64_t)(c0 + ch) * a.N + n] * LOG2E : 0.f;
    h[k] = in && a.init ? a.init[((int64_t)b * a.C + c0 + ch) * a.N + n] : 0.f;
  }
  struct Operands {  // of U tokens
    float2 st[U];
    uint32_t bc[U][NS * WORDS];
    __device__ __forceinline__ float b(int j, int k) const {
      return __uint_as_float(WORDS == 1 ? bc[j][k] << 16 : bc[j][2 * k]);
    }
    __device__ __forceinline__ float c(int j, int k) const {
      return __uint_as_float(WORDS == 1 ? bc[j][k] & 0xffff0000u : bc[j][(2 * k + 1) % (NS * WORDS)]);
    }
  };
  auto read = [&](int k2, int tg, Operands& o) {
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const int t = tg + j;
      o.st[j] = s_step[k2][S::at(t, ch)];
      const uint32_t* from = &s_bc[k2][(t * NP + q * NS) * WORDS];
      if constexpr (NS * WORDS % 4 == 0) {
#pragma unroll
        for (int k = 0; k < NS * WORDS; k += 4)
          *reinterpret_cast<uint4*>(&o.bc[j][k]) = *reinterpret_cast<const uint4*>(from + k);
      } else if constexpr (NS * WORDS == 2) {
        *reinterpret_cast<uint2*>(o.bc[j]) = *reinterpret_cast<const uint2*>(from);
      } else {
        o.bc[j][0] = from[0];
      }
    }
  };
  auto rates = [&](const Operands& o, float (&e)[U][NS]) {
#pragma unroll
    for (int j = 0; j < U; ++j) {
      if constexpr (NS == 1) {
        e[j][0] = ex2(o.st[j].x * A2[0]);
      } else {
#pragma unroll
        for (int k = 0; k < NS; k += 2) {
          const F2 v = mul2(both(o.st[j].x), F2{A2[k], A2[k + 1]});
          e[j][k] = ex2(v.x);
          e[j][k + 1] = ex2(v.y);
        }
      }
    }
  };
  // Where a group's sums take two exchanges they are stored with the next group's: by then the last has come back.
  constexpr bool DEFER = RED > 2;
  float mine[U / RED], last = 0.f;
  auto store = [&](int k2, int tg) {
#pragma unroll
    for (int j = 0; j < U / RED; ++j) s_y[k2][S::sum_at(tg + j + q / PW, ch) + q % PW] = DEFER ? mine[j] + last : mine[j];
  };
  auto finish = [&](int k2, int tg, const Operands& o, const float (&e)[U][NS]) {
    float part[U];
#pragma unroll
    for (int j = 0; j < U; ++j) {
      if constexpr (NS == 1) {
        h[0] = fmaf(e[j][0], h[0], o.st[j].y * o.b(j, 0));
        part[j] = o.c(j, 0) * h[0];
      } else {
        F2 y{0.f, 0.f};
#pragma unroll
        for (int k = 0; k < NS; k += 2) {
          const F2 bx = mul2(both(o.st[j].y), F2{o.b(j, k), o.b(j, k + 1)});
          const F2 hn = fma2(F2{e[j][k], e[j][k + 1]}, F2{h[k], h[k + 1]}, bx);
          h[k] = hn.x;
          h[k + 1] = hn.y;
          const F2 cv{o.c(j, k), o.c(j, k + 1)};
          y = k == 0 ? mul2(cv, hn) : fma2(cv, hn, y);
        }
        part[j] = y.x + y.y;
      }
    }
    if (DEFER && tg > 0) store(k2, tg - U);
#pragma unroll
    for (int half = RED / 2; half > 0; half /= 2) {
      const bool up = (q & (half * PW)) != 0;
#pragma unroll
      for (int j = 0; j < half; ++j) {
        const float give = up ? part[j] : part[j + half], keep = up ? part[j + half] : part[j];
        const float got = __shfl_xor_sync(0xffffffffu, give, half * PW);
        if (DEFER && half == 1)
          part[0] = keep, last = got;
        else
          part[j] = keep + got;
      }
    }
#pragma unroll
    for (int j = 0; j < U / RED; ++j) mine[j] = part[j];
    if (!DEFER) store(k2, tg);
  };
#pragma unroll 1
  for (int tile = 0; tile < tiles; ++tile) {
    const int k2 = tile & 1;
    wait_for(FULL + k2);
    // Software pipeline over groups of U tokens: while group g is finished, the exponentials of g + 1 are under way
    // and the operands of g + 2 are loaded.
    Operands o[2];
    float e[2][U][NS];
    read(k2, 0, o[0]);
    read(k2, U, o[1]);
    rates(o[0], e[0]);
#pragma unroll 1
    for (int tg = 0; tg < TT; tg += 2 * U) {
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        rates(o[1 - w], e[1 - w]);
        finish(k2, tg + w * U, o[w], e[w]);
        read(k2, tg + (w + 2) * U, o[w]);
      }
    }
    if (DEFER) store(k2, TT - U);
    arrive_at(DONE + k2);
  }
  if (a.final_state && ch < nc) {
#pragma unroll
    for (int k = 0; k < NS; ++k)
      if (q * NS + k < a.N) a.final_state[((int64_t)b * a.C + c0 + ch) * a.N + q * NS + k] = h[k];
  }
}

template <typename T, int NS, int LPC>
cudaError_t launch_as(Args<T> a, int64_t B, cudaStream_t st) {
  a.blocks_per_group = (uint32_t)ceil_div(a.per_group, LANES / LPC);
  const unsigned blocks = (unsigned)(B * a.G * a.blocks_per_group);
  if constexpr (NS * LPC % (16 / (int)sizeof(T)) == 0) {
    if (a.vec && a.bvec) {
      k_selective<T, NS, LPC, true, true><<<blocks, THREADS, 0, st>>>(a);
      return cudaGetLastError();
    }
  }
  if constexpr (NS > 1) {
    if (a.vec)
      k_selective<T, NS, LPC, true, false><<<blocks, THREADS, 0, st>>>(a);
    else
      k_selective<T, NS, LPC, false, false><<<blocks, THREADS, 0, st>>>(a);
  }
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_prompt(Args<T> a, int64_t B, cudaStream_t st) {
  // rows on 16 bytes (vec, bvec as given) are moved in 16-byte pieces where groups of channels, and of states, are
  // whole pieces too
  constexpr int V = 16 / (int)sizeof(T);
  a.vec = a.vec && a.per_group % V == 0;
  a.bvec = a.bvec && a.N % V == 0;
  if (a.N <= 4) return launch_as<T, 2, 2>(a, B, st);
  if (a.N <= 8) return launch_as<T, 4, 2>(a, B, st);
  if (a.N <= 16) {
    // More lanes per channel make more warps of a small problem, at more work per channel (each lane reads the step,
    // sums are exchanged): 16 lanes while that is at most two warps per scheduler (768 channels of 2048 tokens 43 us,
    // against 72 with 8 lanes and 98 with 4), 8 up to four (5120 channels 143 us against 163 with 4 lanes), 4 beyond
    // (10240 channels 228 us against 238 with 8).  Not 16 where inputs come element by element, which its helpers
    // cannot keep up with (128 channels, 512 tokens: 21 us with 8 lanes, 25 with 16).
    const int64_t channels = B * a.C, warp = 32;
    if (a.vec && a.bvec && channels * 16 <= 2 * SCHEDULERS * warp) return launch_as<T, 1, 16>(a, B, st);
    if (channels * 8 <= 4 * SCHEDULERS * warp) return launch_as<T, 2, 8>(a, B, st);
    return launch_as<T, 4, 4>(a, B, st);
  }
  if (a.N <= 32) return launch_as<T, 4, 8>(a, B, st);
  if (a.N <= 64) return launch_as<T, 4, 16>(a, B, st);
  return launch_as<T, 8, 16>(a, B, st);
}

// One token: four state entries to a lane, a channel on ceil(N / 4) lanes
// (rounded up to a power of two), y summed by shuffles.  A lane takes its
// channel of up to ROWS sequences, whose states it loads before the first is
// used, with A, D and the bias loaded once.
template <typename T, bool VEC, int ROWS>
__global__ void __launch_bounds__(LANES) k_selective_step(const Args<T> a, float* state, int64_t B, int lpc) {
  const uint32_t i = (blockIdx.x * LANES + threadIdx.x) / lpc;
  const int q = threadIdx.x % lpc;
  const bool on = i < a.total;
  const uint32_t j = on ? i : a.total - 1;  // lanes behind the end take part in the shuffles
  const uint32_t r = j / a.C;
  const int64_t b0 = (int64_t)r * ROWS;
  const int c = (int)(j - r * a.C), n0 = q * 4, some = min(4, a.N - n0);
  const int64_t gn = (int64_t)(c / a.per_group) * a.N + n0;
  const int n1 = some > 0 ? n0 : 0;  // lanes behind the last entry read the first, for nothing
  const int64_t gn1 = gn - n0 + n1;
  // every load of the lane, none of them conditional and none of them looked at before the last is issued
  Pack<float, VEC ? 4 : 1> hp[ROWS][VEC ? 1 : 4], ap[VEC ? 1 : 4];
  Pack<T, VEC ? 4 : 1> bp[ROWS][VEC ? 1 : 4], cp[ROWS][VEC ? 1 : 4];
  Pack<T, 1> x[ROWS], dt[ROWS], z[ROWS];
  const bool gate = a.z.p != nullptr;
#pragma unroll
  for (int m = 0; m < ROWS; ++m) {
    const int64_t b = b0 + m < B ? b0 + m : B - 1;
#pragma unroll
    for (int k = 0; k < (VEC ? 1 : 4); ++k) {
      const int e = k < some ? k : 0;
      hp[m][k] = load_pack<float, VEC ? 4 : 1>(state + (b * a.C + c) * a.N + n1 + e);
      bp[m][k] = load_pack<T, VEC ? 4 : 1>(a.bm.row(b, 0) + gn1 + e);
      cp[m][k] = load_pack<T, VEC ? 4 : 1>(a.cm.row(b, 0) + gn1 + e);
    }
    x[m] = load_pack<T, 1>(a.x.row(b, 0) + c);
    dt[m] = load_pack<T, 1>(a.dt.row(b, 0) + c);
    z[m] = load_pack<T, 1>((gate ? a.z : a.x).row(b, 0) + c);
  }
#pragma unroll
  for (int k = 0; k < (VEC ? 1 : 4); ++k)
    ap[k] = load_pack<float, VEC ? 4 : 1>(a.A + (int64_t)c * a.N + n1 + (k < some ? k : 0));
  const float D = a.D ? a.D[c] : 0.f, bias = a.dt_bias ? a.dt_bias[c] : 0.f;
#pragma unroll
  for (int m = 0; m < ROWS; ++m) {
    float step = dt[m].get(0) + bias;
    if (a.softplus) step = softplus(step);
    const float xv = x[m].get(0), sx = step * xv;
    float h[4], y = 0.f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int i = VEC ? 0 : k, e = VEC ? k : 0;
      h[k] = fmaf(ex2(step * (ap[i].get(e) * LOG2E)), hp[m][i].get(e), sx * bp[m][i].get(e));
      if (k < some) y = fmaf(cp[m][i].get(e), h[k], y);
    }
    for (int off = 1; off < lpc; off <<= 1) y += __shfl_xor_sync(0xffffffffu, y, off);
    if (on && b0 + m < B) {
      float* st = state + ((b0 + m) * a.C + c) * a.N + n0;
      if (VEC) {
        if (some > 0) store_pack<float, 4>(st, to_pack<float, 4>(h));
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (k < some) st[k] = h[k];
      }
      if (q == 0) {
        y = fmaf(D, xv, y);
        if (gate) y *= silu(z[m].get(0));
        a.y.row(b0 + m, 0)[c] = from_f32<T>(y);
      }
    }
  }
}

template <typename T, bool VEC>
cudaError_t launch_token_as(Args<T> a, float* state, int64_t B, int lpc, cudaStream_t st) {
  // four sequences a lane where that still makes eight blocks for every SM
  if (ceil_div(B, 4) * a.C * lpc >= int64_t(148) * 8 * LANES) {
    a.total = (uint32_t)(ceil_div(B, 4) * a.C);
    k_selective_step<T, VEC, 4><<<(unsigned)ceil_div((int64_t)a.total * lpc, LANES), LANES, 0, st>>>(a, state, B, lpc);
  } else {
    a.total = (uint32_t)(B * a.C);
    k_selective_step<T, VEC, 1><<<(unsigned)ceil_div((int64_t)a.total * lpc, LANES), LANES, 0, st>>>(a, state, B, lpc);
  }
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_token(const Args<T>& a, float* state, int64_t B, cudaStream_t st) {
  int lpc = 1;
  while (lpc * 4 < a.N) lpc *= 2;
  const uintptr_t t = reinterpret_cast<uintptr_t>(a.bm.p) | reinterpret_cast<uintptr_t>(a.cm.p) |
                      (uintptr_t)(B > 1 ? a.bm.bs * sizeof(T) : 0);
  // four entries by one access: whole fours of states, on 16 bytes (B and C: on four elements)
  if (a.N % 4 == 0 && on_16(state) && on_16(a.A) && (t & (4 * sizeof(T) - 1)) == 0)
    return launch_token_as<T, true>(a, state, B, lpc, st);
  return launch_token_as<T, false>(a, state, B, lpc, st);
}

ssd_status validate(const ssd_selective_dims* d, int64_t seqlen) {
  if (!d) return SSD_ERR_INVALID_ARG;
  if (d->flags & ~SSD_SELECTIVE_SOFTPLUS) return SSD_ERR_INVALID_ARG;
  if (d->io_dtype != SSD_F32 && d->io_dtype != SSD_BF16) return SSD_ERR_DTYPE;
  if (d->batch < 1 || seqlen < 1 || d->channels < 1 || d->dstate < 1 || d->ngroups < 1 ||
      d->channels % d->ngroups != 0)
    return SSD_ERR_SHAPE;
  // one index per (sequence, channel, lane) stays below 2^31
  if (d->dstate > 128 || d->channels > (int64_t(1) << 24) || d->batch > (int64_t(1) << 24) ||
      d->batch * d->channels > (int64_t(1) << 25) || seqlen > (int64_t(1) << 31))
    return SSD_ERR_UNSUPPORTED;
  return SSD_OK;
}

// The tensors of a call: a prompt's, or a single token's (L = 1) with the state that it updates.
struct Call {
  RowArg x, dt, z, bm, cm, y;
  const float *A, *D, *dt_bias, *init;
  float* final_state;
  const int32_t* lengths;
  float* state;
};

ssd_status run(const ssd_selective_dims* d, int64_t L, const Call& k, cudaStream_t st) {
  ssd_status s;
  if (!k.x.p || !k.dt.p || !k.A || !k.bm.p || !k.cm.p || !k.y.p) return SSD_ERR_INVALID_ARG;
  const int64_t B = d->batch, C = d->channels, N = d->dstate;
  const size_t es = io_bytes(d->io_dtype);
  for (const RowArg* r : {&k.x, &k.dt, &k.z, &k.bm, &k.cm})
    if (r->p && (s = check_rows(*r, B, L, es, false)) != SSD_OK) return s;
  if ((s = check_rows(k.y, B, L, es, true)) != SSD_OK) return s;
  for (const void* p : {(const void*)k.A, (const void*)k.D, (const void*)k.dt_bias, (const void*)k.init,
                        (const void*)k.final_state, (const void*)k.lengths})
    if (!f32_aligned(p)) return SSD_ERR_ALIGN;
  const size_t state = sizeof(float) * B * C * N;
  const Span sy{k.y.p, row_extent(k.y, B, L, es)}, sf{k.final_state, state}, si{k.init, state};
  for (const RowArg* r : {&k.x, &k.dt, &k.z, &k.bm, &k.cm}) {
    const Span in{r->p, r->p ? row_extent(*r, B, L, es) : 0};
    if (spans_meet(sy, in) || spans_meet(sf, in)) return SSD_ERR_INVALID_ARG;
  }
  for (const Span& in : {Span{k.A, sizeof(float) * C * N}, Span{k.D, sizeof(float) * C},
                         Span{k.dt_bias, sizeof(float) * C}, Span{k.lengths, sizeof(int32_t) * B}})
    if (spans_meet(sy, in) || spans_meet(sf, in)) return SSD_ERR_INVALID_ARG;
  if (spans_meet(sy, si) || spans_meet(sy, sf) || (k.init != k.final_state && spans_meet(sf, si)))
    return SSD_ERR_INVALID_ARG;
  auto go = [&](auto t) {
    using T = decltype(t);
    auto rows = [](const RowArg& r) { return Rows<const T>{(const T*)r.p, r.bs, r.ts}; };
    Args<T> a{};
    a.x = rows(k.x);
    a.dt = rows(k.dt);
    a.z = rows(k.z);
    a.bm = rows(k.bm);
    a.cm = rows(k.cm);
    a.y = Rows<T>{(T*)k.y.p, k.y.bs, k.y.ts};
    a.A = k.A;
    a.D = k.D;
    a.dt_bias = k.dt_bias;
    a.init = k.init;
    a.final_state = k.final_state;
    a.lengths = k.lengths;
    a.L = L;
    a.C = (int)C;
    a.N = (int)N;
    a.G = (int)d->ngroups;
    a.per_group = (int)(C / d->ngroups);
    a.softplus = (d->flags & SSD_SELECTIVE_SOFTPLUS) != 0;
    if (k.state) return launch_token<T>(a, k.state, B, st);
    a.vec = true;
    for (const RowArg* r : {&k.x, &k.dt, &k.z, &k.y})
      if (r->p && !rows_on_16(*r, B, L, es)) a.vec = false;
    a.bvec = rows_on_16(k.bm, B, L, es) && rows_on_16(k.cm, B, L, es);
    return launch_prompt<T>(a, B, st);
  };
  return cuda_status(d->io_dtype == SSD_BF16 ? go(__nv_bfloat16()) : go(float()));
}

}  // namespace selective
}  // namespace ssd

extern "C" ssd_status ssd_selective_fwd(const ssd_selective_dims* d, const void* x, int64_t x_bstride,
                                        int64_t x_tstride, const void* dt, int64_t dt_bstride, int64_t dt_tstride,
                                        const float* A, const void* Bm, const void* Cm, int64_t bc_bstride,
                                        int64_t bc_tstride, const float* D, const void* z, int64_t z_bstride,
                                        int64_t z_tstride, const float* dt_bias, const float* init_state,
                                        const int32_t* lengths, void* y, int64_t y_bstride, int64_t y_tstride,
                                        float* final_state, void* stream) {
  using namespace ssd;
  const ssd_status s = selective::validate(d, d ? d->seqlen : 1);
  if (s != SSD_OK) return s;
  const int64_t C = d->channels, gn = d->ngroups * d->dstate;
  const selective::Call k{{x, x_bstride, x_tstride, C},   {dt, dt_bstride, dt_tstride, C}, {z, z_bstride, z_tstride, C},
                          {Bm, bc_bstride, bc_tstride, gn}, {Cm, bc_bstride, bc_tstride, gn}, {y, y_bstride, y_tstride, C},
                          A, D, dt_bias, init_state, final_state, lengths, nullptr};
  return selective::run(d, d->seqlen, k, static_cast<cudaStream_t>(stream));
}

extern "C" ssd_status ssd_selective_step(const ssd_selective_dims* d, const void* x, int64_t x_bstride,
                                         const void* dt, int64_t dt_bstride, const float* A, const void* Bm,
                                         const void* Cm, int64_t bc_bstride, const float* D, const void* z,
                                         int64_t z_bstride, const float* dt_bias, float* state, void* y,
                                         int64_t y_bstride, void* stream) {
  using namespace ssd;
  const ssd_status s = selective::validate(d, 1);
  if (s != SSD_OK) return s;
  if (!state) return SSD_ERR_INVALID_ARG;
  const int64_t C = d->channels, gn = d->ngroups * d->dstate;
  const selective::Call k{{x, x_bstride, 0, C},   {dt, dt_bstride, 0, C}, {z, z_bstride, 0, C},
                          {Bm, bc_bstride, 0, gn}, {Cm, bc_bstride, 0, gn}, {y, y_bstride, 0, C},
                          A, D, dt_bias, state, state, nullptr, state};
  return selective::run(d, 1, k, static_cast<cudaStream_t>(stream));
}
