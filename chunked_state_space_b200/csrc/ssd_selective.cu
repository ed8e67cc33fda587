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
// per (token, channel) and put in shared memory twice each, as the operands of
// packed f32x2 instructions; B and C are widened to f32 once per tile.  The LPC
// partial sums of y of LPC tokens are reduced together, each exchange halving
// what a lane still holds, so that lane q ends up with token q's sum.
#include "ssd_rows.cuh"

namespace ssd {
namespace selective {

constexpr int THREADS = 128;
constexpr float LOG2E = 1.4426950408889634f;

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
  bool softplus, vec;
};

__device__ __forceinline__ float ex2(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

// Two f32 lanes per instruction, each rounded like the scalar operation.
struct F2 {
  float x, y;
};
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  const float2 r = vdecay::mul2(make_float2(a.x, a.y), make_float2(b.x, b.y));
  return {r.x, r.y};
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  const float2 r = vdecay::fma2(make_float2(a.x, a.y), make_float2(b.x, b.y), make_float2(c.x, c.y));
  return {r.x, r.y};
}

// max(v, 0) + log1p(e^-|v|).  The exponent's rounding is put back to first
// order, so that small steps keep f32 accuracy; log1p(e) = e P(e) with P the
// minimax polynomial of degree 8 of log1p(e) / e on [0, 1] (Remez exchange,
// P(0) = 1; at most 1.8e-7 off, relative, evaluated in f32).
__device__ __forceinline__ float softplus(float v) {
  const float m = -fabsf(v), t = m * LOG2E;
  const float p = ex2(t), e = fmaf(p, fmaf(m, LOG2E, -t) * 0.69314718f, p);
  float q = 0.0053648264f;
  q = fmaf(q, e, -0.030065801f);
  q = fmaf(q, e, 0.07920455f);
  q = fmaf(q, e, -0.13753803f);
  q = fmaf(q, e, 0.19153656f);
  q = fmaf(q, e, -0.24857163f);
  q = fmaf(q, e, 0.33321324f);
  q = fmaf(q, e, -0.49999648f);
  q = fmaf(q, e, 1.0f);
  return fmaf(q, e, v < 0.f ? 0.f : v);  // v, not max(v, 0): NaN stays
}

template <typename T, int NS, int LPC, bool VEC>
struct Shape {
  static constexpr int CB = THREADS / LPC;                 // channels of a block
  static constexpr int NP = NS * LPC;                      // state entries, the last ones empty where N is less
  static constexpr int V = VEC ? 16 / (int)sizeof(T) : 1;  // elements per load
  // tokens of a tile: E elements of x per thread, fewer where B and C would not leave room
  static constexpr int E = NP <= 32 ? 8 : NP == 64 ? 4 : 2;
  static constexpr int TT = LPC == 1 ? 16 : E * LPC;
  static constexpr int NX = (TT * CB / V + THREADS - 1) / THREADS;  // loads of x (dt, z) per thread
  static constexpr int NB = (TT * NP / V + THREADS - 1) / THREADS;  // loads of B (C) per thread
  // a row of y sums: lanes of a warp hold 32 / LPC channels of LPC tokens, which should fall on different banks
  static constexpr int YS = LPC == 1 ? CB : LPC == 2 ? CB + 16 : LPC == 4 ? CB + 8 : CB + 4;
  static_assert(TT % LPC == 0, "a tile is a whole number of reductions");
  static_assert(NP % V == 0 && CB % V == 0, "rows of a tile are whole pieces");
  // Where (token, channel) lies in a tile of 16-byte entries: a thread writes V neighbouring channels, one per
  // instruction, so they are turned by the piece's number to fall on different banks; the channels that a warp reads
  // together share the turn.
  __device__ static __forceinline__ int at(int t, int ch) {
    if (V == 8) return t * CB + (ch ^ ((t * (CB / 8) + (ch >> 3)) & 7));
    if (V == 4) return t * CB + (ch ^ (((t * (CB / 4) + (ch >> 2)) >> 1) & 3));
    return t * CB + ch;
  }
};

template <typename T, int NS, int LPC, bool VEC>
__global__ void __launch_bounds__(THREADS) k_selective(const Args<T> a) {
  using S = Shape<T, NS, LPC, VEC>;
  constexpr int CB = S::CB, NP = S::NP, V = S::V, TT = S::TT, NX = S::NX, NB = S::NB, YS = S::YS;
  __shared__ float4 s_step[TT * CB];  // (s, s, s x, s x)
  __shared__ __align__(16) float s_b[TT * NP], s_c[TT * NP];
  __shared__ __align__(16) float s_y[TT * YS];
  __shared__ float s_D[CB], s_bias[CB];
  const uint32_t r = blockIdx.x / a.blocks_per_group, cb = blockIdx.x - r * a.blocks_per_group;
  const uint32_t b = r / a.G, g = r - b * a.G;
  const int c0 = (int)g * a.per_group + (int)cb * CB;  // first channel of the block
  const int nc = min(CB, ((int)g + 1) * a.per_group - c0);
  const int tid = threadIdx.x, q = tid % LPC, ch = tid / LPC;
  const int64_t len = row_length(a.lengths, b, a.L);
  const int64_t at = ((int64_t)b * a.C + c0 + ch) * a.N;
  float A2[NS], h[NS];
#pragma unroll
  for (int k = 0; k < NS; ++k) {
    const int n = q * NS + k;
    const bool in = ch < nc && n < a.N;
    A2[k] = in ? a.A[(int64_t)(c0 + ch) * a.N + n] * LOG2E : 0.f;
    h[k] = in && a.init ? a.init[at + n] : 0.f;
  }
  if (tid < CB) {
    s_D[tid] = a.D && tid < nc ? a.D[c0 + tid] : 0.f;
    s_bias[tid] = a.dt_bias && tid < nc ? a.dt_bias[c0 + tid] : 0.f;
  }
  const bool gate = a.z.p != nullptr;
  Pack<T, V> nx[NX], nd[NX], nz[NX], nb[NB], ncm[NB];  // the next tile's rows
  auto fetch = [&](int64_t t0) {
#pragma unroll
    for (int k = 0; k < NX; ++k) {
      const int i = tid + k * THREADS, t = i / (CB / V), c = i % (CB / V) * V;
      if (i < TT * CB / V && t0 + t < len && c < nc) {
        nx[k] = load_pack<T, V>(a.x.row(b, t0 + t) + c0 + c);
        nd[k] = load_pack<T, V>(a.dt.row(b, t0 + t) + c0 + c);
        if (gate) nz[k] = load_pack<T, V>(a.z.row(b, t0 + t) + c0 + c);
      }
    }
#pragma unroll
    for (int k = 0; k < NB; ++k) {
      const int i = tid + k * THREADS, t = i / (NP / V), n = i % (NP / V) * V;
      if (i < TT * NP / V && t0 + t < len && n < a.N) {
        nb[k] = load_pack<T, V>(a.bm.row(b, t0 + t) + (int64_t)g * a.N + n);
        ncm[k] = load_pack<T, V>(a.cm.row(b, t0 + t) + (int64_t)g * a.N + n);
      }
    }
  };
  fetch(0);
  __syncthreads();  // s_D, s_bias
  for (int64_t t0 = 0; t0 < len; t0 += TT) {
    // stage this tile; behind the sequence's end the step is 0, which leaves the state as it is
    Pack<T, V> x[NX], z[NX];
#pragma unroll
    for (int k = 0; k < NX; ++k) {
      x[k] = nx[k];
      z[k] = nz[k];
      const int i = tid + k * THREADS, t = i / (CB / V), c = i % (CB / V) * V;
      if (i < TT * CB / V) {
        const bool in = t0 + t < len && c < nc;
#pragma unroll
        for (int e = 0; e < V; ++e) {
          float s = 0.f, sx = 0.f;
          if (in) {
            s = to_f32(nd[k].v[e]) + s_bias[c + e];
            if (a.softplus) s = softplus(s);
            sx = s * to_f32(x[k].v[e]);
          }
          s_step[S::at(t, c + e)] = make_float4(s, s, sx, sx);
        }
      }
    }
#pragma unroll
    for (int k = 0; k < NB; ++k) {
      const int i = tid + k * THREADS, t = i / (NP / V), n = i % (NP / V) * V;
      if (i < TT * NP / V) {
        const bool in = t0 + t < len && n < a.N;
#pragma unroll
        for (int e = 0; e < V; ++e) {
          s_b[i * V + e] = in ? to_f32(nb[k].v[e]) : 0.f;
          s_c[i * V + e] = in ? to_f32(ncm[k].v[e]) : 0.f;
        }
      }
    }
    __syncthreads();
    if (t0 + TT < len) fetch(t0 + TT);
#pragma unroll 1
    for (int tg = 0; tg < TT; tg += LPC) {
      float part[LPC];
#pragma unroll
      for (int j = 0; j < LPC; ++j) {
        const int t = tg + j;
        const float4 st = s_step[S::at(t, ch)];
        const float* bt = &s_b[t * NP + q * NS];
        const float* ct = &s_c[t * NP + q * NS];
        float bv[NS], cv[NS];
        if constexpr (NS % 4 == 0) {
#pragma unroll
          for (int k = 0; k < NS; k += 4) {
            *reinterpret_cast<float4*>(&bv[k]) = *reinterpret_cast<const float4*>(bt + k);
            *reinterpret_cast<float4*>(&cv[k]) = *reinterpret_cast<const float4*>(ct + k);
          }
        } else if constexpr (NS == 2) {
          *reinterpret_cast<float2*>(bv) = *reinterpret_cast<const float2*>(bt);
          *reinterpret_cast<float2*>(cv) = *reinterpret_cast<const float2*>(ct);
        } else {
#pragma unroll
          for (int k = 0; k < NS; ++k) bv[k] = bt[k], cv[k] = ct[k];
        }
        if constexpr (NS == 1) {
          h[0] = fmaf(ex2(st.x * A2[0]), h[0], st.z * bv[0]);
          part[j] = cv[0] * h[0];
        } else {
          F2 y{0.f, 0.f};
#pragma unroll
          for (int k = 0; k < NS; k += 2) {
            const F2 e = mul2(F2{st.x, st.y}, F2{A2[k], A2[k + 1]});
            const F2 bx = mul2(F2{st.z, st.w}, F2{bv[k], bv[k + 1]});
            const F2 hn = fma2(F2{ex2(e.x), ex2(e.y)}, F2{h[k], h[k + 1]}, bx);
            h[k] = hn.x;
            h[k + 1] = hn.y;
            y = k == 0 ? mul2(F2{cv[0], cv[1]}, hn) : fma2(F2{cv[k], cv[k + 1]}, hn, y);
          }
          part[j] = y.x + y.y;
        }
      }
#pragma unroll
      for (int half = LPC / 2; half > 0; half /= 2) {
        const bool up = (q & half) != 0;
#pragma unroll
        for (int j = 0; j < half; ++j) {
          const float give = up ? part[j] : part[j + half], keep = up ? part[j + half] : part[j];
          part[j] = keep + __shfl_xor_sync(0xffffffffu, give, half);
        }
      }
      s_y[(tg + q) * YS + ch] = part[0];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < NX; ++k) {
      const int i = tid + k * THREADS, t = i / (CB / V), c = i % (CB / V) * V;
      if (i < TT * CB / V && t0 + t < len && c < nc) {
        Pack<T, V> out;
#pragma unroll
        for (int e = 0; e < V; ++e) {
          float y = fmaf(s_D[c + e], to_f32(x[k].v[e]), s_y[t * YS + c + e]);
          if (gate) y *= silu(to_f32(z[k].v[e]));
          out.v[e] = from_f32<T>(y);
        }
        store_pack<T, V>(a.y.row(b, t0 + t) + c0 + c, out);
      }
    }
  }
  if (a.final_state && ch < nc) {
#pragma unroll
    for (int k = 0; k < NS; ++k)
      if (q * NS + k < a.N) a.final_state[at + q * NS + k] = h[k];
  }
}

template <typename T, int NS, int LPC>
cudaError_t launch_as(Args<T> a, int64_t B, cudaStream_t st) {
  a.blocks_per_group = (uint32_t)ceil_div(a.per_group, THREADS / LPC);
  const unsigned blocks = (unsigned)(B * a.G * a.blocks_per_group);
  // 16-byte pieces: rows on 16 bytes, groups of channels and of states that are whole pieces
  constexpr int V = 16 / (int)sizeof(T);
  if constexpr (NS * LPC % V == 0) {
    if (a.vec && a.per_group % V == 0 && a.N % V == 0) {
      k_selective<T, NS, LPC, true><<<blocks, THREADS, 0, st>>>(a);
      return cudaGetLastError();
    }
  }
  k_selective<T, NS, LPC, false><<<blocks, THREADS, 0, st>>>(a);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_prompt(const Args<T>& a, int64_t B, cudaStream_t st) {
  if (a.N <= 4) return launch_as<T, 4, 1>(a, B, st);
  if (a.N <= 8) return launch_as<T, 4, 2>(a, B, st);
  if (a.N <= 16) return launch_as<T, 4, 4>(a, B, st);
  if (a.N <= 32) return launch_as<T, 4, 8>(a, B, st);
  if (a.N <= 64) return launch_as<T, 4, 16>(a, B, st);
  return launch_as<T, 8, 16>(a, B, st);
}

// One token: four state entries to a lane, a channel on ceil(N / 4) lanes
// (rounded up to a power of two), y summed by shuffles.
template <typename T, bool VEC>
__global__ void __launch_bounds__(THREADS) k_selective_step(const Args<T> a, float* state, int lpc) {
  const uint32_t i = (blockIdx.x * THREADS + threadIdx.x) / lpc;
  const int q = threadIdx.x % lpc;
  const bool on = i < a.total;
  const uint32_t j = on ? i : a.total - 1;  // lanes behind the end take part in the shuffles
  const uint32_t b = j / a.C;
  const int c = (int)(j - b * a.C), n0 = q * 4, some = min(4, a.N - n0);
  const int64_t gn = (int64_t)(c / a.per_group) * a.N + n0;
  float h[4] = {}, A[4] = {}, bv[4] = {}, cv[4] = {};
  float* st = state + (int64_t)j * a.N + n0;
  const float* ap = a.A + (int64_t)c * a.N + n0;
  const T* bp = a.bm.row(b, 0) + gn;
  const T* cp = a.cm.row(b, 0) + gn;
  if (VEC) {
    if (some > 0) {
      const Pack<float, 4> hp = load_pack<float, 4>(st), rp = load_pack<float, 4>(ap);
      const Pack<T, 4> b4 = load_pack<T, 4>(bp), c4 = load_pack<T, 4>(cp);
#pragma unroll
      for (int k = 0; k < 4; ++k) h[k] = hp.v[k], A[k] = rp.v[k], bv[k] = to_f32(b4.v[k]), cv[k] = to_f32(c4.v[k]);
    }
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (k < some) h[k] = st[k], A[k] = ap[k], bv[k] = to_f32(bp[k]), cv[k] = to_f32(cp[k]);
  }
  const float x = to_f32(a.x.row(b, 0)[c]);
  float s = to_f32(a.dt.row(b, 0)[c]) + (a.dt_bias ? a.dt_bias[c] : 0.f);
  const float z = a.z.p ? to_f32(a.z.row(b, 0)[c]) : 0.f;
  if (a.softplus) s = softplus(s);
  const float sx = s * x;
  float y = 0.f;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    h[k] = fmaf(ex2(s * (A[k] * LOG2E)), h[k], sx * bv[k]);
    y = fmaf(cv[k], h[k], y);
  }
  for (int off = 1; off < lpc; off <<= 1) y += __shfl_xor_sync(0xffffffffu, y, off);
  if (!on) return;
  if (VEC) {
    if (some > 0) store_pack<float, 4>(st, Pack<float, 4>{{h[0], h[1], h[2], h[3]}});
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (k < some) st[k] = h[k];
  }
  if (q == 0) {
    y = fmaf(a.D ? a.D[c] : 0.f, x, y);
    if (a.z.p) y *= silu(z);
    a.y.row(b, 0)[c] = from_f32<T>(y);
  }
}

template <typename T>
cudaError_t launch_token(Args<T> a, float* state, int64_t B, cudaStream_t st) {
  int lpc = 1;
  while (lpc * 4 < a.N) lpc *= 2;
  a.total = (uint32_t)(B * a.C);
  const unsigned blocks = (unsigned)ceil_div((int64_t)a.total * lpc, THREADS);
  const uintptr_t f = reinterpret_cast<uintptr_t>(state) | reinterpret_cast<uintptr_t>(a.A);
  const uintptr_t t = reinterpret_cast<uintptr_t>(a.bm.p) | reinterpret_cast<uintptr_t>(a.cm.p) | a.bm.bs * sizeof(T);
  // four entries by one access: whole fours of states, on 16 bytes (B and C: on four elements)
  if (a.N % 4 == 0 && (f & 15) == 0 && (t & (4 * sizeof(T) - 1)) == 0)
    k_selective_step<T, true><<<blocks, THREADS, 0, st>>>(a, state, lpc);
  else
    k_selective_step<T, false><<<blocks, THREADS, 0, st>>>(a, state, lpc);
  return cudaGetLastError();
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
    for (const RowArg* r : {&k.x, &k.dt, &k.z, &k.bm, &k.cm, &k.y})
      if (r->p && !rows_on_16(*r, B, L, es)) a.vec = false;
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
