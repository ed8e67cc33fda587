// The selective scan of a prompt:
//   s = softplus(dt + bias);  h[n] = e^{s A[c,n]} h[n] + s B[n] x
//   y = (sum_n C[n] h[n] + D x) silu(z)
//
// With a decay per state entry and a step per channel there is no matrix
// product in it: N exponentials and 4 N fp32 operations per token and channel,
// and four special-function operations more for softplus and silu.  At N = 16
// these 20 take 1.25 clocks of an SM (16 per clock), four times what the
// token's 8 bytes of bf16 take of HBM: a prompt is bound by the exponentials,
// and in practice by the instructions around them.
//
// A channel's entries lie on LPC lanes of a warp, NS to a lane, in registers
// over the whole sequence; a block takes 128 / LPC channels of one group.  Its
// inputs come tile by tile, the next tile's rows loaded into registers while
// this one is computed: the step and the scaled input of each (token, channel)
// are formed once and put in shared memory, and so are B and C, which all
// channels of the block read.  The partial sums of y go back through shared
// memory to be gated and stored by whole rows.  Two kernels do this:
//   k_selective_teams  four warps run the recurrence, fed by two warps that
//       prepare operands and drained by two that finish outputs, over double
//       buffers: no warp waits for a phase of its own, which counts where a
//       scheduler has few warps;
//   k_selective_many   every warp does everything, phase by phase: fewer
//       registers and no idle warps, which counts where blocks fill the SMs.
// Long sequences of few channels are cut into segments that run at once
// (segments, below).
#pragma once

#include <algorithm>

#include "ssd_rows.cuh"

namespace ssd {
namespace selective {

constexpr int LANES = 128;  // lanes of a block that carry the recurrence
constexpr int HELPERS = 64, TEAM_THREADS = LANES + 2 * HELPERS;
constexpr int64_t SCHEDULERS = 4 * 148;  // warp schedulers of the GPU
constexpr int MAX_SEGMENTS = 64;

template <typename T>
struct Args {
  Rows<const T> x, dt, z, bm, cm;
  Rows<T> y;
  const float *A, *D, *dt_bias;
  const float* init;
  float* final_state;
  const int32_t* lengths;
  int64_t B, L;
  int C, N, G, per_group;
  uint32_t blocks_per_group, total;
  bool softplus, vec, bvec;
  // Segments of seg_len tokens of every sequence (1: the whole sequences).  With more than one, starts [nseg,B,C,N]
  // holds the state that each begins with, sums [nseg - 1,B,C] the steps that it takes in all.
  int nseg;
  int64_t seg_len;
  float *starts, *sums;
};

// max(v, 0) + log1p(e^-|v|); |v| beyond 128, infinite or the type's lowest, counts
// as 128, whose e^-|v| is 0.  The exponent's rounding is put back to first
// order, so that small steps keep f32 accuracy; log1p(e) = e P(e) with P the
// minimax polynomial of degree 8 of log1p(e) / e on [0, 1] (Remez exchange,
// P(0) = 1; at most 1.8e-7 off, relative, evaluated in f32).
__device__ __forceinline__ F2 softplus2(F2 v) {
  const F2 m{fmaxf(-fabsf(v.x), -128.f), fmaxf(-fabsf(v.y), -128.f)}, t = mul2(m, both(LOG2E));
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

// Where (token, channel) lies in a tile of 8-byte entries: a thread writes V
// neighbouring channels, two per instruction, so its pairs are turned by the
// piece's number to fall on different banks; the channels that a warp reads
// together share the turn or lie in different pieces.
template <int CB, int V>
__device__ __forceinline__ int step_at(int t, int ch) {
  const int i = t * (CB / V) + ch / V;
  const int turn = V == 8 ? (i >> 1) & 3 : V == 4 ? (i >> 2) & 1 : 0;
  return t * CB + (ch ^ (turn << 1));
}

// Step and scaled input of the piece (t, c .. c + V - 1).  Where there is no
// such token or channel the step is 0, which leaves the state as it is.
template <typename T, int CB, int V>
__device__ __forceinline__ void put_steps(float2* s_step, int t, int c, bool in, const Pack<T, V>& x,
                                          const Pack<T, V>& dt, const float* s_bias, bool with_softplus) {
  if constexpr (V == 1) {
    float s = 0.f, sx = 0.f;
    if (in) {
      s = dt.get(0) + s_bias[c];
      if (with_softplus) s = softplus(s);
      sx = s * x.get(0);
    }
    s_step[step_at<CB, V>(t, c)] = make_float2(s, sx);
  } else {
    F2 s[V / 2], sx[V / 2];
    if (in) {
#pragma unroll
      for (int e = 0; e < V; e += 2) s[e / 2] = add2(F2{dt.get(e), dt.get(e + 1)}, F2{s_bias[c + e], s_bias[c + e + 1]});
      if (with_softplus) {
#pragma unroll
        for (int e = 0; e < V; e += 2) s[e / 2] = softplus2(s[e / 2]);
      }
#pragma unroll
      for (int e = 0; e < V; e += 2) sx[e / 2] = mul2(s[e / 2], F2{x.get(e), x.get(e + 1)});
    } else {
#pragma unroll
      for (int e = 0; e < V; e += 2) s[e / 2] = sx[e / 2] = both(0.f);
    }
#pragma unroll
    for (int e = 0; e < V; e += 2)
      *reinterpret_cast<float4*>(&s_step[step_at<CB, V>(t, c + e)]) =
          make_float4(s[e / 2].x, sx[e / 2].x, s[e / 2].y, sx[e / 2].y);
  }
}

// B and C of an entry lie side by side: two bf16 in a word (which halves the
// shared-memory traffic that would bound the kernels, for two instructions per
// entry), or two f32.
template <typename T>
constexpr int WORDS = sizeof(T) == 2 ? 1 : 2;

template <typename T, int VB>
__device__ __forceinline__ void put_bc(uint32_t* to, bool in, const Pack<T, VB>& b, const Pack<T, VB>& c) {
  uint32_t w[VB * WORDS<T>];
#pragma unroll
  for (int e = 0; e < VB; ++e) {
    const uint32_t bw = in ? __float_as_uint(b.get(e)) : 0u, cw = in ? __float_as_uint(c.get(e)) : 0u;
    if constexpr (WORDS<T> == 1)
      w[e] = __byte_perm(bw, cw, 0x7632);  // the upper halves: the bf16 themselves
    else
      w[2 * e] = bw, w[2 * e + 1] = cw;
  }
  if constexpr (VB * WORDS<T> % 4 == 0) {
#pragma unroll
    for (int e = 0; e < VB * WORDS<T>; e += 4)
      *reinterpret_cast<uint4*>(to + e) = make_uint4(w[e], w[e + 1], w[e + 2], w[e + 3]);
  } else {
#pragma unroll
    for (int e = 0; e < VB * WORDS<T>; ++e) to[e] = w[e];
  }
}

template <typename T, int NS>
struct Entries {  // B and C of a lane's NS entries of one token
  uint32_t w[NS * WORDS<T>];
  __device__ __forceinline__ void read(const uint32_t* from) {
    constexpr int N = NS * WORDS<T>;
    if constexpr (N % 4 == 0) {
#pragma unroll
      for (int k = 0; k < N; k += 4) *reinterpret_cast<uint4*>(&w[k]) = *reinterpret_cast<const uint4*>(from + k);
    } else if constexpr (N == 2) {
      *reinterpret_cast<uint2*>(w) = *reinterpret_cast<const uint2*>(from);
    } else {
      w[0] = from[0];
    }
  }
  __device__ __forceinline__ float b(int k) const { return __uint_as_float(WORDS<T> == 1 ? w[k] << 16 : w[2 * k]); }
  __device__ __forceinline__ float c(int k) const {
    return __uint_as_float(WORDS<T> == 1 ? w[k] & 0xffff0000u : w[(2 * k + 1) % (NS * WORDS<T>)]);
  }
};

// h = e h + sx B for a lane's entries of one token; returns its part of sum_n C h.
template <typename T, int NS>
__device__ __forceinline__ float advance(float (&h)[NS], const float (&e)[NS], float sx, const Entries<T, NS>& bc) {
  if constexpr (NS == 1) {
    h[0] = fmaf(e[0], h[0], sx * bc.b(0));
    return bc.c(0) * h[0];
  } else {
    F2 y{0.f, 0.f};
#pragma unroll
    for (int k = 0; k < NS; k += 2) {
      const F2 hn = fma2(F2{e[k], e[k + 1]}, F2{h[k], h[k + 1]}, mul2(both(sx), F2{bc.b(k), bc.b(k + 1)}));
      h[k] = hn.x;
      h[k + 1] = hn.y;
      const F2 c{bc.c(k), bc.c(k + 1)};
      y = k == 0 ? mul2(c, hn) : fma2(c, hn, y);
    }
    return y.x + y.y;
  }
}

// e^{s A} of a lane's entries (A2 = A log2 e)
template <int NS>
__device__ __forceinline__ void decays(float s, const float (&A2)[NS], float (&e)[NS]) {
  if constexpr (NS == 1) {
    e[0] = ex2(s * A2[0]);
  } else {
#pragma unroll
    for (int k = 0; k < NS; k += 2) {
      const F2 v = mul2(both(s), F2{A2[k], A2[k + 1]});
      e[k] = ex2(v.x);
      e[k + 1] = ex2(v.y);
    }
  }
}

// y of a piece: sums(e) gives the sums of channels e and e + 1 of it.
template <typename T, int V, typename F>
__device__ __forceinline__ Pack<T, V> outputs(const Pack<T, V>& x, const Pack<T, V>& z, bool gate, const float* D,
                                              F&& sums) {
  float out[V];
  if constexpr (V == 1) {
    out[0] = fmaf(D[0], x.get(0), sums(0).x);
    if (gate) out[0] *= silu(z.get(0));
  } else {
#pragma unroll
    for (int e = 0; e < V; e += 2) {
      F2 y = fma2(F2{D[e], D[e + 1]}, F2{x.get(e), x.get(e + 1)}, sums(e));
      if (gate) y = mul2(y, silu2(F2{z.get(e), z.get(e + 1)}));
      out[e] = y.x, out[e + 1] = y.y;
    }
  }
  return to_pack<T, V>(out);
}

// The block's segment of a sequence and its channels, and a lane's rates and
// states.
template <int CB>
struct Place {
  uint32_t b, g, seg;
  int c0, nc;  // first channel, how many
  int64_t t0;  // first token
  int len;     // tokens
};
template <int CB, typename T>
__device__ __forceinline__ Place<CB> place(const Args<T>& a) {
  Place<CB> p;
  uint32_t r = blockIdx.x / a.blocks_per_group;
  const uint32_t cb = blockIdx.x - r * a.blocks_per_group;
  p.g = r % (uint32_t)a.G;
  r /= (uint32_t)a.G;
  p.b = a.nseg == 1 ? r : r % (uint32_t)a.B;
  p.seg = a.nseg == 1 ? 0 : r / (uint32_t)a.B;
  p.c0 = (int)p.g * a.per_group + (int)cb * CB;
  p.nc = min(CB, ((int)p.g + 1) * a.per_group - p.c0);
  p.t0 = p.seg * a.seg_len;
  const int64_t rest = row_length(a.lengths, p.b, a.L) - p.t0;
  p.len = (int)(rest < 0 ? 0 : rest < a.seg_len ? rest : a.seg_len);
  return p;
}
template <int NS, int CB, typename T>
__device__ __forceinline__ void begin(const Args<T>& a, const Place<CB>& p, int ch, int q, float (&A2)[NS], float (&h)[NS],
                                      bool from_zero = false) {
  const float* from = from_zero ? nullptr : a.nseg == 1 ? a.init : a.starts + (int64_t)p.seg * a.B * a.C * a.N;
#pragma unroll
  for (int k = 0; k < NS; ++k) {
    const int n = q * NS + k;
    const bool in = ch < p.nc && n < a.N;
    A2[k] = in ? a.A[(int64_t)(p.c0 + ch) * a.N + n] * LOG2E : 0.f;
    h[k] = in && from ? from[((int64_t)p.b * a.C + p.c0 + ch) * a.N + n] : 0.f;
  }
}
template <int NS, int CB, typename T>
__device__ __forceinline__ void put_state(const Args<T>& a, const Place<CB>& p, int ch, int q, const float (&h)[NS],
                                          float* to) {
  if (!to || ch >= p.nc) return;
#pragma unroll
  for (int k = 0; k < NS; ++k)
    if (q * NS + k < a.N) to[((int64_t)p.b * a.C + p.c0 + ch) * a.N + q * NS + k] = h[k];
}

// ---------------------------------------------------------------- teams

template <typename T, int NS, int LPC, bool VEC, bool BVEC>
struct Teams {
  static constexpr int CB = LANES / LPC;                     // channels of a block
  static constexpr int NP = NS * LPC;                        // state entries, the last ones empty where N is less
  static constexpr int V = VEC ? 16 / (int)sizeof(T) : 1;    // elements per load of x, dt, z and per store of y
  static constexpr int VB = BVEC ? 16 / (int)sizeof(T) : 1;  // ... per load of B, C
  // tokens of a tile: eight elements of x per helper thread, fewer where B and C would not leave room (in shared
  // memory, or in registers as single elements)
  static constexpr int TT = NP <= 16 ? 8 * HELPERS / CB : NP == 32 ? (BVEC ? 32 : 16) : NP == 64 ? (BVEC ? 16 : 8) : 8;
  static constexpr int XP = TT * CB / V, BP = TT * NP / VB;  // pieces of a tile of x (dt, z), of B (C)
  static constexpr int NX = (XP + HELPERS - 1) / HELPERS, NB = (BP + HELPERS - 1) / HELPERS;  // ... per thread
  static constexpr int APART = HELPERS / (CB / V);           // tokens between the pieces of a thread
  // y's sums over the states are left in PW parts per (token, channel), which the output team adds up; more than four
  // lanes exchange theirs first, RED tokens together, each exchange halving what a lane still holds.
  static constexpr int PW = 4, RED = LPC / PW;
  static constexpr int U = RED < 2 ? 2 : RED;  // tokens that a lane works on together
  static constexpr int ROWS = TT + 2 * U;      // rows of operands: a tile, and what the loop reads behind it for nothing
  static_assert(TT % (2 * U) == 0, "a tile is a whole number of turns of its loop");
  static_assert(NP % VB == 0 && CB % V == 0 && HELPERS % (CB / V) == 0, "rows of a tile are whole pieces");
  // Where the parts of (token, channel) lie: a thread reads them channel by channel, 16 bytes at a time.
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
template <int THREADS>
__device__ __forceinline__ void wait_for(int bar) {
  asm volatile("bar.sync %0, %1;" ::"r"(bar), "n"(THREADS) : "memory");
}
template <int THREADS>
__device__ __forceinline__ void arrive_at(int bar) {
  asm volatile("bar.arrive %0, %1;" ::"r"(bar), "n"(THREADS) : "memory");
}

// END: no outputs (and no output team), but what a segment adds to the state:
// its end state from a zero start, and the sum of its steps, whose e^{A sum} is
// what the segment leaves of the state that it begins with.
template <typename T, int NS, int LPC, bool VEC, bool BVEC, bool END>
__global__ void __launch_bounds__(TEAM_THREADS, NS * LPC <= 16 && VEC && BVEC ? 3 : 2) k_selective_teams(const Args<T> a) {
  constexpr int THREADS = END ? LANES + HELPERS : TEAM_THREADS;
  using S = Teams<T, NS, LPC, VEC, BVEC>;
  constexpr int CB = S::CB, NP = S::NP, V = S::V, VB = S::VB, TT = S::TT, XP = S::XP, BP = S::BP, NX = S::NX, NB = S::NB,
                PW = S::PW, RED = S::RED, U = S::U, ROWS = S::ROWS, APART = S::APART, W = WORDS<T>;
  __shared__ __align__(16) float2 s_step[2][ROWS * CB];   // (s, s x)
  __shared__ __align__(16) uint32_t s_bc[2][ROWS * NP * W];  // (B, C)
  __shared__ __align__(16) float s_y[2][END ? 4 : TT * CB * PW];
  __shared__ __align__(16) float s_D[CB], s_bias[CB];
  const Place<CB> p = place<CB>(a);
  const int tid = threadIdx.x, tiles = (int)(((int64_t)p.len + TT - 1) / TT);
  for (int i = tid; i < CB; i += THREADS) {
    s_D[i] = a.D && i < p.nc ? a.D[p.c0 + i] : 0.f;
    s_bias[i] = a.dt_bias && i < p.nc ? a.dt_bias[p.c0 + i] : 0.f;
  }
  __syncthreads();

  if (!END && tid >= LANES + HELPERS) {
    // ---- output: add up the sums, skip and gate, store
    const int me = tid - LANES - HELPERS;
    const bool gate = a.z.p != nullptr;
    for (int k = 0; k < 2 && k < tiles; ++k) arrive_at<THREADS>(FULL + k);
    // piece k of a thread: token t0 + k * APART of the tile, channels c ..
    const int t0 = me / (CB / V), c = me % (CB / V) * V;
    const T* px = a.x.row(p.b, p.t0 + t0) + p.c0 + c;
    const T* pz = gate ? a.z.row(p.b, p.t0 + t0) + p.c0 + c : px;
    T* py = a.y.row(p.b, p.t0 + t0) + p.c0 + c;
    Pack<T, V> nx[NX], nz[NX];
    auto fetch = [&](int left) {  // left: tokens of the sequence from this tile on
#pragma unroll
      for (int k = 0; k < NX; ++k) {
        if (me + k * HELPERS < XP && t0 + k * APART < left && c < p.nc) {
          nx[k] = load_pack<T, V>(px + k * APART * a.x.ts);
          if (gate) nz[k] = load_pack<T, V>(pz + k * APART * a.z.ts);
        }
      }
      px += TT * a.x.ts;
      pz += TT * a.z.ts;
    };
    int left = p.len;
    fetch(left);
#pragma unroll 1
    for (int tile = 0; tile < tiles; ++tile) {
      const int k2 = tile & 1;
      Pack<T, V> x[NX], z[NX];
#pragma unroll
      for (int k = 0; k < NX; ++k) x[k] = nx[k], z[k] = nz[k];
      if (tile + 1 < tiles) fetch(left - TT);
      wait_for<THREADS>(DONE + k2);
#pragma unroll
      for (int k = 0; k < NX; ++k) {
        const int t = t0 + k * APART;
        if (me + k * HELPERS < XP && t < left && c < p.nc) {
          auto sums = [&](int e) {
            const float* u = &s_y[k2][S::sum_at(t, c + e)];
            const float* v = &s_y[k2][S::sum_at(t, V > 1 ? c + e + 1 : c + e)];
            const float4 f = *reinterpret_cast<const float4*>(u), g = *reinterpret_cast<const float4*>(v);
            const F2 f2 = add2(F2{f.x, f.y}, F2{f.z, f.w}), g2 = add2(F2{g.x, g.y}, F2{g.z, g.w});
            return F2{f2.x + f2.y, g2.x + g2.y};
          };
          store_pack<T, V>(py + k * APART * a.y.ts, outputs<T, V>(x[k], z[k], gate, &s_D[c], sums));
        }
      }
      py += TT * a.y.ts;
      left -= TT;
      if (tile + 2 < tiles) arrive_at<THREADS>(FULL + k2);
    }
    return;
  }

  if (tid >= LANES) {
    // ---- operands: the step and the scaled input of every (token, channel), B and C
    const int me = tid - LANES;
    const int t0 = me / (CB / V), c = me % (CB / V) * V;
    const T* px = a.x.row(p.b, p.t0 + t0) + p.c0 + c;
    const T* pd = a.dt.row(p.b, p.t0 + t0) + p.c0 + c;
    const T* pb = a.bm.row(p.b, p.t0) + (int64_t)p.g * a.N;
    const T* pc = a.cm.row(p.b, p.t0) + (int64_t)p.g * a.N;
    Pack<T, V> nx[NX], nd[NX];
    Pack<T, VB> nb[NB], nc[NB];
    auto fetch = [&](int left) {
#pragma unroll
      for (int k = 0; k < NX; ++k) {
        if (me + k * HELPERS < XP && t0 + k * APART < left && c < p.nc) {
          nx[k] = load_pack<T, V>(px + k * APART * a.x.ts);
          nd[k] = load_pack<T, V>(pd + k * APART * a.dt.ts);
        }
      }
#pragma unroll
      for (int k = 0; k < NB; ++k) {
        const int i = me + k * HELPERS, t = i / (NP / VB), n = i % (NP / VB) * VB;
        if (i < BP && t < left && n < a.N) {
          nb[k] = load_pack<T, VB>(pb + t * a.bm.ts + n);
          nc[k] = load_pack<T, VB>(pc + t * a.cm.ts + n);
        }
      }
      px += TT * a.x.ts;
      pd += TT * a.dt.ts;
      pb += TT * a.bm.ts;
      pc += TT * a.cm.ts;
    };
    int left = p.len;
    fetch(left);
#pragma unroll 1
    for (int tile = 0; tile < tiles; ++tile) {
      const int k2 = tile & 1;
      if (tile >= 2) wait_for<THREADS>(DONE + k2);
#pragma unroll
      for (int k = 0; k < NX; ++k) {
        const int t = t0 + k * APART;
        if (me + k * HELPERS < XP)
          put_steps<T, CB, V>(s_step[k2], t, c, t < left && c < p.nc, nx[k], nd[k], s_bias, a.softplus);
      }
#pragma unroll
      for (int k = 0; k < NB; ++k) {
        const int i = me + k * HELPERS, t = i / (NP / VB), n = i % (NP / VB) * VB;
        if (i < BP) put_bc<T, VB>(&s_bc[k2][i * VB * W], t < left && n < a.N, nb[k], nc[k]);
      }
      left -= TT;
      arrive_at<THREADS>(FULL + k2);
      if (tile + 1 < tiles) fetch(left);
    }
    for (int tile = tiles > 2 ? tiles - 2 : 0; tile < tiles; ++tile) arrive_at<THREADS>(DONE + (tile & 1));
    return;
  }

  // ---- the recurrence
  const int q = tid % LPC, ch = tid / LPC;
  float A2[NS], h[NS];
  begin(a, p, ch, q, A2, h, END);
  float steps = 0.f;  // END: the sum of the steps
  struct Operands {  // of U tokens
    float2 st[U];
    Entries<T, NS> bc[U];
  };
  auto read = [&](int k2, int tg, Operands& o) {
#pragma unroll
    for (int j = 0; j < U; ++j) {
      o.st[j] = s_step[k2][step_at<CB, V>(tg + j, ch)];
      o.bc[j].read(&s_bc[k2][((tg + j) * NP + q * NS) * W]);
    }
  };
  auto rates = [&](const Operands& o, float (&e)[U][NS]) {
#pragma unroll
    for (int j = 0; j < U; ++j) decays<NS>(o.st[j].x, A2, e[j]);
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
    for (int j = 0; j < U; ++j) part[j] = advance<T, NS>(h, e[j], o.st[j].y, o.bc[j]);
    if constexpr (END) {
#pragma unroll
      for (int j = 0; j < U; ++j) steps += o.st[j].x;
      return;
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
    wait_for<THREADS>(FULL + k2);
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
    if (DEFER && !END) store(k2, TT - U);
    arrive_at<THREADS>(DONE + k2);
  }
  if (END) {
    const int64_t channels = a.B * a.C;
    put_state(a, p, ch, q, h, a.starts + (p.seg + 1) * channels * a.N);
    if (q == 0 && ch < p.nc) a.sums[p.seg * channels + (int64_t)p.b * a.C + p.c0 + ch] = steps;
  } else if (p.seg + 1 == a.nseg) {
    put_state(a, p, ch, q, h, a.final_state);
  }
}

// ---------------------------------------------------------------- many

template <typename T, int NS, int LPC, bool VEC, bool BVEC>
__global__ void __launch_bounds__(LANES, VEC && BVEC ? 5 : 4) k_selective_many(const Args<T> a) {
  constexpr int CB = LANES / LPC, NP = NS * LPC, TT = 8 * LPC;  // eight elements of x per thread and tile
  constexpr int V = VEC ? 16 / (int)sizeof(T) : 1, VB = BVEC ? 16 / (int)sizeof(T) : 1, W = WORDS<T>;
  constexpr int NX = 8 / V, BP = TT * NP / VB, NB = (BP + LANES - 1) / LANES, APART = LANES / (CB / V);
  constexpr int U = 8;           // tokens whose sums are exchanged together: a lane ends up with U / LPC of them
  constexpr int KEEP = U / LPC;
  constexpr int YS = CB + (LPC == 4 ? 8 : 4);  // a row of sums: a warp writes 32 / LPC channels of LPC tokens
  static_assert(NP % VB == 0 && CB % V == 0 && U % LPC == 0 && TT % U == 0, "rows and tiles are whole pieces");
  __shared__ __align__(16) float2 s_step[TT * CB];     // (s, s x)
  __shared__ __align__(16) uint32_t s_bc[TT * NP * W];  // (B, C)
  __shared__ __align__(16) float s_y[TT * YS];
  __shared__ __align__(16) float s_D[CB], s_bias[CB];
  const Place<CB> p = place<CB>(a);
  const int tid = threadIdx.x, q = tid % LPC, ch = tid / LPC;
  float A2[NS], h[NS];
  begin(a, p, ch, q, A2, h);
  for (int i = tid; i < CB; i += LANES) {
    s_D[i] = a.D && i < p.nc ? a.D[p.c0 + i] : 0.f;
    s_bias[i] = a.dt_bias && i < p.nc ? a.dt_bias[p.c0 + i] : 0.f;
  }
  const bool gate = a.z.p != nullptr;
  // piece k of a thread: token t0 + k * APART of the tile, channels c ..
  const int t0 = tid / (CB / V), c = tid % (CB / V) * V;
  const T* px = a.x.row(p.b, t0) + p.c0 + c;
  const T* pd = a.dt.row(p.b, t0) + p.c0 + c;
  const T* pz = gate ? a.z.row(p.b, t0) + p.c0 + c : px;
  T* py = a.y.row(p.b, t0) + p.c0 + c;
  const T* pb = a.bm.row(p.b, 0) + (int64_t)p.g * a.N;
  const T* pc = a.cm.row(p.b, 0) + (int64_t)p.g * a.N;
  Pack<T, V> nx[NX], nd[NX], nz[NX];
  Pack<T, VB> nb[NB], nc[NB];
  auto fetch = [&](int left) {
#pragma unroll
    for (int k = 0; k < NX; ++k) {
      if (t0 + k * APART < left && c < p.nc) {
        nx[k] = load_pack<T, V>(px + k * APART * a.x.ts);
        nd[k] = load_pack<T, V>(pd + k * APART * a.dt.ts);
        if (gate) nz[k] = load_pack<T, V>(pz + k * APART * a.z.ts);
      }
    }
#pragma unroll
    for (int k = 0; k < NB; ++k) {
      const int i = tid + k * LANES, t = i / (NP / VB), n = i % (NP / VB) * VB;
      if (i < BP && t < left && n < a.N) {
        nb[k] = load_pack<T, VB>(pb + t * a.bm.ts + n);
        nc[k] = load_pack<T, VB>(pc + t * a.cm.ts + n);
      }
    }
    px += TT * a.x.ts;
    pd += TT * a.dt.ts;
    pz += TT * a.z.ts;
    pb += TT * a.bm.ts;
    pc += TT * a.cm.ts;
  };
  fetch(p.len);
  __syncthreads();  // s_D, s_bias
#pragma unroll 1
  for (int left = p.len; left > 0; left -= TT) {
    Pack<T, V> x[NX], z[NX];
#pragma unroll
    for (int k = 0; k < NX; ++k) {
      x[k] = nx[k];
      z[k] = nz[k];
      const int t = t0 + k * APART;
      put_steps<T, CB, V>(s_step, t, c, t < left && c < p.nc, x[k], nd[k], s_bias, a.softplus);
    }
#pragma unroll
    for (int k = 0; k < NB; ++k) {
      const int i = tid + k * LANES, t = i / (NP / VB), n = i % (NP / VB) * VB;
      if (i < BP) put_bc<T, VB>(&s_bc[i * VB * W], t < left && n < a.N, nb[k], nc[k]);
    }
    __syncthreads();
    if (left > TT) fetch(left - TT);
#pragma unroll 1
    for (int tg = 0; tg < TT; tg += U) {
      float part[U];
#pragma unroll
      for (int j = 0; j < U; ++j) {
        const float2 st = s_step[step_at<CB, V>(tg + j, ch)];
        Entries<T, NS> bc;
        bc.read(&s_bc[((tg + j) * NP + q * NS) * W]);
        float e[NS];
        decays<NS>(st.x, A2, e);
        part[j] = advance<T, NS>(h, e, st.y, bc);
      }
      // the LPC parts of every sum: each exchange halves the tokens that a lane still holds
#pragma unroll
      for (int half = LPC / 2; half > 0; half /= 2) {
        const bool up = (q & half) != 0;
#pragma unroll
        for (int j = 0; j < half * KEEP; ++j) {
          const float give = up ? part[j] : part[j + half * KEEP], keep = up ? part[j + half * KEEP] : part[j];
          part[j] = keep + __shfl_xor_sync(0xffffffffu, give, half);
        }
      }
#pragma unroll
      for (int j = 0; j < KEEP; ++j) s_y[(tg + q * KEEP + j) * YS + ch] = part[j];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < NX; ++k) {
      const int t = t0 + k * APART;
      if (t < left && c < p.nc) {
        auto sums = [&](int e) {
          const float* u = &s_y[t * YS + c + e];
          return F2{u[0], u[V > 1 ? 1 : 0]};
        };
        store_pack<T, V>(py + k * APART * a.y.ts, outputs<T, V>(x[k], z[k], gate, &s_D[c], sums));
      }
    }
    py += TT * a.y.ts;
  }
  put_state(a, p, ch, q, h, a.final_state);
}

// ---------------------------------------------------------------- segments
//
// The state that each segment begins with, in order: starts[k] arrives as the
// end state of segment k - 1 from a zero start and leaves as
//   starts[0] = init,  starts[k] += e^{A sums[k-1]} starts[k-1].
// A state of 0 stays out of it: rates above 0 can make the factor infinite.
template <typename T>
__global__ void __launch_bounds__(256) k_selective_starts(const Args<T> a) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, states = a.B * a.C * a.N;
  if (i >= states) return;
  const int64_t channel = i / a.N;
  const float A2 = a.A[channel % a.C * a.N + i % a.N] * LOG2E;
  float h = a.init ? a.init[i] : 0.f;
  a.starts[i] = h;
  // eight segments' loads under way together
  constexpr int AT = 8;
  for (int k = 1; k < a.nseg; k += AT) {
    float sum[AT], end[AT];
#pragma unroll
    for (int j = 0; j < AT; ++j) {
      const bool in = k + j < a.nseg;
      sum[j] = in ? a.sums[(k + j - 1) * a.B * a.C + channel] : 0.f;
      end[j] = in ? a.starts[(k + j) * states + i] : 0.f;
    }
#pragma unroll
    for (int j = 0; j < AT; ++j) {
      h = h == 0.f ? end[j] : fmaf(ex2(sum[j] * A2), h, end[j]);
      if (k + j < a.nseg) a.starts[(k + j) * states + i] = h;
    }
  }
}

// ---------------------------------------------------------------- choice

template <typename T, int NS, int LPC, bool END = false>
cudaError_t launch_teams(Args<T> a, int64_t B, cudaStream_t st) {
  a.blocks_per_group = (uint32_t)ceil_div(a.per_group, LANES / LPC);
  const unsigned blocks = (unsigned)(B * a.G * a.blocks_per_group * (END ? a.nseg - 1 : a.nseg));
  constexpr int threads = END ? LANES + HELPERS : TEAM_THREADS;
  if constexpr (NS * LPC % (16 / (int)sizeof(T)) == 0) {
    if (a.vec && a.bvec) {
      k_selective_teams<T, NS, LPC, true, true, END><<<blocks, threads, 0, st>>>(a);
      return cudaGetLastError();
    }
  }
  if (a.vec)
    k_selective_teams<T, NS, LPC, true, false, END><<<blocks, threads, 0, st>>>(a);
  else
    k_selective_teams<T, NS, LPC, false, false, END><<<blocks, threads, 0, st>>>(a);
  return cudaGetLastError();
}

// A few channels leave most SMs idle, and a token takes the 16-lane kernel the
// same time however few they are: a long sequence is cut into segments that run
// at once, first for their end states, then, from the states that these give,
// for the outputs.  That doubles the work, so it pays up to two thirds of the
// SMs.  The count is the one of least estimated time among those that make one,
// two or three blocks per SM, if that is at most 0.9 of the whole's; ns per token
// as measured (bf16, rows on 16 bytes, all or but for B and C, or not; 4096 and
// 16384 tokens).  Whole and cut:
// 64 channels of 1024 tokens 23 and 11 us, of 16384 tokens 323 and 34, of 65536
// tokens 1282 and 100; 384 of 4096 83 and 44, of 1024 23 and 18; 760 of 16384
// 332 and 250; 1024 of 16384 346 and 356 (not taken).
struct Rates {
  double whole, per_sm[3];
};
inline int segments(const ssd_selective_dims* d, bool vec, bool bvec) {
  if (d->dstate > 16 || d->seqlen <= 256) return 1;  // 256 tokens take 6 us: as long as the two launches more
  static constexpr Rates ON_16{20, {19, 28, 32.5}}, X_ON_16{21.4, {27, 31.5, 1e9}}, APART{29, {35, 36, 1e9}};
  const Rates& r = !vec ? APART : bvec ? ON_16 : X_ON_16;
  const int64_t blocks = d->batch * d->ngroups * ceil_div(d->channels / d->ngroups, LANES / 16);
  int best = 1;
  double least = 0.9 * r.whole * d->seqlen;
  for (int k = 0; k < 3; ++k) {
    const int64_t n = std::min<int64_t>((k + 1) * 148 / blocks, MAX_SEGMENTS);
    const double cut = 2 * r.per_sm[k] * ceil_div(d->seqlen, n < 1 ? 1 : n) + 5000 + 200 * n;
    if (n >= 2 && cut <= least) least = cut, best = (int)n;
  }
  return best;
}
// starts (a multiple of 256 bytes) and sums of n segments, or 0
inline size_t starts_bytes(const ssd_selective_dims* d, int n) {
  return (size_t)ceil_div(n * d->batch * d->channels * d->dstate * 4, 256) * 256;
}
inline size_t segment_bytes(const ssd_selective_dims* d, int n) {
  return n > 1 ? starts_bytes(d, n) + (size_t)(n - 1) * d->batch * d->channels * 4 : 0;
}
// for rows of any alignment
inline size_t segment_bytes(const ssd_selective_dims* d) {
  return segment_bytes(d, std::max({segments(d, true, true), segments(d, true, false), segments(d, false, false)}));
}

template <typename T>
cudaError_t launch_segments(const Args<T>& a, int64_t B, cudaStream_t st) {
  cudaError_t e = launch_teams<T, 1, 16, true>(a, B, st);
  if (e != cudaSuccess) return e;
  k_selective_starts<T><<<(unsigned)ceil_div(B * a.C * a.N, 256), 256, 0, st>>>(a);
  e = cudaGetLastError();
  return e == cudaSuccess ? launch_teams<T, 1, 16>(a, B, st) : e;
}

template <typename T, int NS, int LPC>
cudaError_t launch_many(Args<T> a, int64_t B, cudaStream_t st) {
  a.blocks_per_group = (uint32_t)ceil_div(a.per_group, LANES / LPC);
  const unsigned blocks = (unsigned)(B * a.G * a.blocks_per_group);
  if (a.vec && a.bvec)
    k_selective_many<T, NS, LPC, true, true><<<blocks, LANES, 0, st>>>(a);
  else if (a.vec)
    k_selective_many<T, NS, LPC, true, false><<<blocks, LANES, 0, st>>>(a);
  else
    k_selective_many<T, NS, LPC, false, false><<<blocks, LANES, 0, st>>>(a);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_prompt(Args<T> a, int64_t B, const ssd_selective_dims* d, void* workspace, cudaStream_t st) {
  // rows on 16 bytes (vec, bvec as given) are moved in 16-byte pieces where groups of channels, and of states, are
  // whole pieces too
  constexpr int V = 16 / (int)sizeof(T);
  a.vec = a.vec && a.per_group % V == 0;
  a.bvec = a.bvec && a.N % V == 0;
  if (workspace) {
    a.nseg = segments(d, a.vec, a.bvec);
    a.seg_len = ceil_div(a.L, a.nseg);
    a.starts = static_cast<float*>(workspace);
    a.sums = a.starts + starts_bytes(d, a.nseg) / sizeof(float);
    if (a.nseg > 1) return launch_segments(a, B, st);
  }
  // More lanes per channel make more warps of a small problem, at more instructions per channel, and teams help where
  // a scheduler has few warps.  The rule counts the recurrence's warps; the times are of 16 states, bf16, unless said
  // otherwise.  In a padded batch (lengths) sequences end early and it counts half of them (five sequences, three of
  // them with tokens, 1530 channels: 42 us with teams, 52 with many).
  const int64_t channels = a.lengths ? ceil_div(B * a.C, 2) : B * a.C;
  auto warps = [&](int lpc) { return channels * lpc / 32; };
  // 16 lanes, one entry to each: 768 channels of 2048 tokens 44 us, with 8 lanes 67 (4096 channels of 1024: 65 and
  // 50); also for fewer entries than lanes (4 states, 770 channels of 14400 tokens: 461 us, with 4 lanes 1129)
  if (a.N <= 16 && warps(16) <= 2 * SCHEDULERS) return launch_teams<T, 1, 16>(a, B, st);
  // 8 states, 10240 channels of 1024 tokens: 81 us, with many as much (768 channels 41 and 58)
  if (a.N <= 8) return launch_teams<T, 2, 4>(a, B, st);
  if (a.N <= 16) {
    // 4096 channels of 1024 tokens 50 us, with many 53 (7680 channels: 96 and 83)
    if (warps(8) <= 2 * SCHEDULERS) return launch_teams<T, 2, 8>(a, B, st);
    // 10240 channels of 2048 tokens 195 us, with 4 lanes 215 (40960 channels: 667 and 559)
    if (warps(8) <= 6 * SCHEDULERS) return launch_many<T, 2, 8>(a, B, st);
    return launch_many<T, 4, 4>(a, B, st);
  }
  if (a.N <= 32) {
    // 32 states, 1024 tokens: 768 channels 51 us, with many 60 (10240 channels: 191 and 148)
    if (warps(8) <= 2 * SCHEDULERS) return launch_teams<T, 4, 8>(a, B, st);
    return launch_many<T, 4, 8>(a, B, st);
  }
  if (a.N <= 64) return launch_teams<T, 4, 16>(a, B, st);
  return launch_teams<T, 8, 16>(a, B, st);
}

}  // namespace selective
}  // namespace ssd
