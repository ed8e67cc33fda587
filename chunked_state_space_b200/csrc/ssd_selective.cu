// The selective scan with a step per channel, for prompts and single tokens:
//   s = softplus(dt + bias);  h[n] = e^{s A[c,n]} h[n] + s B[n] x
//   y = (sum_n C[n] h[n] + D x) silu(z)
// A channel's N state entries lie on LPC = ceil(N / 4) lanes of a warp (rounded
// up to a power of two), four to a lane in registers; y is summed over the
// lanes by shuffles.
#include "ssd_rows.cuh"

namespace ssd {
namespace selective {

constexpr int THREADS = 128;
constexpr int PER = 4;  // state entries per lane
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
  int C, N, per_group, lpc;
  uint32_t blocks_per_row;
  bool softplus;
};

__device__ __forceinline__ float ex2(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

__device__ __forceinline__ float softplus(float v) { return fmaxf(v, 0.f) + log1pf(expf(-fabsf(v))); }

template <typename T>
__global__ void __launch_bounds__(THREADS) k_selective(const Args<T> a) {
  const uint32_t b = blockIdx.x / a.blocks_per_row, cb = blockIdx.x - b * a.blocks_per_row;
  const int lane = threadIdx.x % a.lpc;
  const int c = (int)cb * (THREADS / a.lpc) + threadIdx.x / a.lpc;
  const bool on = c < a.C;
  const int cc = on ? c : a.C - 1, g = cc / a.per_group;
  const int64_t len = row_length(a.lengths, b, a.L);
  const int64_t at = ((int64_t)b * a.C + cc) * a.N;
  float A2[PER], h[PER];
#pragma unroll
  for (int k = 0; k < PER; ++k) {
    const int n = lane * PER + k;
    A2[k] = n < a.N ? a.A[(int64_t)cc * a.N + n] * LOG2E : 0.f;
    h[k] = n < a.N && a.init ? a.init[at + n] : 0.f;
  }
  const float D = a.D ? a.D[cc] : 0.f, bias = a.dt_bias ? a.dt_bias[cc] : 0.f;
  for (int64_t t = 0; t < len; ++t) {
    const float x = to_f32(a.x.row(b, t)[cc]);
    float s = to_f32(a.dt.row(b, t)[cc]) + bias;
    if (a.softplus) s = softplus(s);
    const float sx = s * x;
    const T* bt = a.bm.row(b, t) + (int64_t)g * a.N;
    const T* ct = a.cm.row(b, t) + (int64_t)g * a.N;
    float y = 0.f;
#pragma unroll
    for (int k = 0; k < PER; ++k) {
      const int n = lane * PER + k;
      if (n < a.N) {
        h[k] = fmaf(ex2(s * A2[k]), h[k], sx * to_f32(bt[n]));
        y = fmaf(to_f32(ct[n]), h[k], y);
      }
    }
    for (int off = 1; off < a.lpc; off <<= 1) y += __shfl_xor_sync(0xffffffffu, y, off);
    if (lane == 0 && on) {
      y = fmaf(D, x, y);
      if (a.z.p) y *= silu(to_f32(a.z.row(b, t)[cc]));
      a.y.row(b, t)[cc] = from_f32<T>(y);
    }
  }
  if (a.final_state && on) {
#pragma unroll
    for (int k = 0; k < PER; ++k)
      if (lane * PER + k < a.N) a.final_state[at + lane * PER + k] = h[k];
  }
}

template <typename T>
cudaError_t launch(Args<T> a, int64_t B, cudaStream_t st) {
  a.lpc = 1;
  while (a.lpc * PER < a.N) a.lpc *= 2;
  a.blocks_per_row = (uint32_t)ceil_div(a.C, THREADS / a.lpc);
  k_selective<T><<<(unsigned)(B * a.blocks_per_row), THREADS, 0, st>>>(a);
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

// The tensors of a call, of which a single token's has L = 1.
struct Call {
  RowArg x, dt, z, bm, cm, y;
  const float *A, *D, *dt_bias, *init;
  float* final_state;
  const int32_t* lengths;
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
    a.per_group = (int)(C / d->ngroups);
    a.softplus = (d->flags & SSD_SELECTIVE_SOFTPLUS) != 0;
    return launch<T>(a, B, st);
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
                          A, D, dt_bias, init_state, final_state, lengths};
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
                          A, D, dt_bias, state, state, nullptr};
  return selective::run(d, 1, k, static_cast<cudaStream_t>(stream));
}
