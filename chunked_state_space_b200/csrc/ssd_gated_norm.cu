// The gated RMS norm behind a scan:
//   u = x silu(z);  out = weight u / sqrt(mean over the feature's group of u^2 + eps)
// Bound by HBM: x and z are read once and out is written once.  A run of
// features (one group of one row) is held in registers as u between the sum
// and the scaling, PER 16-byte pieces per thread, all loaded before the first
// is used; the sum of squares is f32 and reduced in a fixed order.
#include "ssd_rows.cuh"

namespace ssd {
namespace gnorm {

constexpr int PER = 4;  // pieces of a row per thread
constexpr int MOST = 512;  // threads of a block

template <typename T>
struct Args {
  Rows<const T> x, z;
  Rows<T> out;
  const float* weight;
  float eps;
  int64_t runs;      // rows * groups
  uint32_t groups, L;
  int64_t n;         // features of a group
};

template <typename T, int VEC>
__device__ __forceinline__ void gated(const Pack<T, VEC>& x, const Pack<T, VEC>& z, bool gate, float (&u)[VEC]) {
#pragma unroll
  for (int i = 0; i < VEC; ++i) u[i] = gate ? x.get(i) * silu(z.get(i)) : x.get(i);
}

// One run per warp (BLOCK false, four warps of a block on four runs) or per block.
template <typename T, int VEC, bool BLOCK>
__global__ void __launch_bounds__(BLOCK ? MOST : 128) k_gated_norm(const Args<T> a) {
  __shared__ float part[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t run = BLOCK ? (int64_t)blockIdx.x : (int64_t)blockIdx.x * (blockDim.x >> 5) + warp;
  if (run >= a.runs) return;
  const int me = BLOCK ? (int)threadIdx.x : lane, all = BLOCK ? (int)blockDim.x : 32;
  const int64_t r = run / a.groups, g = run - r * a.groups;
  const int64_t b = r / a.L, t = r - b * a.L;
  const T* x = a.x.row(b, t) + g * a.n;
  const bool gate = a.z.p != nullptr;
  const T* z = gate ? a.z.row(b, t) + g * a.n : x;
  T* out = a.out.row(b, t) + g * a.n;
  const int64_t pieces = a.n / VEC;
  float u[PER][VEC];
  float ss = 0.f;
  for (int64_t p0 = 0; p0 < pieces; p0 += (int64_t)PER * all) {
    Pack<T, VEC> px[PER], pz[PER];
#pragma unroll
    for (int k = 0; k < PER; ++k) {
      const int64_t p = p0 + me + k * all;
      if (p < pieces) {
        px[k] = load_pack<T, VEC>(x + p * VEC);
        pz[k] = load_pack<T, VEC>(z + p * VEC);
      }
    }
#pragma unroll
    for (int k = 0; k < PER; ++k) {
      if (p0 + me + k * all < pieces) {
        gated(px[k], pz[k], gate, u[k]);
#pragma unroll
        for (int i = 0; i < VEC; ++i) ss = fmaf(u[k][i], u[k][i], ss);
      }
    }
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
  if (BLOCK) {
    if (lane == 0) part[warp] = ss;
    __syncthreads();
    ss = 0.f;
    for (int w = 0; w < all / 32; ++w) ss += part[w];
  }
  const float inv = 1.0f / sqrtf(ss / (float)a.n + a.eps);
  for (int64_t p0 = 0; p0 < pieces; p0 += (int64_t)PER * all) {
#pragma unroll
    for (int k = 0; k < PER; ++k) {
      const int64_t p = p0 + me + k * all;
      if (p < pieces) {
        // a run longer than the registers hold is read again
        if (pieces > (int64_t)PER * all) gated(load_pack<T, VEC>(x + p * VEC), load_pack<T, VEC>(z + p * VEC), gate, u[k]);
        float o[VEC];
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          const float w = a.weight ? a.weight[g * a.n + p * VEC + i] : 1.f;
          o[i] = u[k][i] * inv * w;
        }
        store_pack<T, VEC>(out + p * VEC, to_pack<T, VEC>(o));
      }
    }
  }
}

// A run of up to 32 * PER pieces takes a warp, a longer one a block of as many
// warps as hold it (at most MOST threads; a run beyond them is read twice).
template <typename T, int VEC>
cudaError_t launch(const Args<T>& a, cudaStream_t st) {
  const int64_t pieces = a.n / VEC;
  if (pieces <= 32 * PER) {
    k_gated_norm<T, VEC, false><<<(unsigned)ceil_div(a.runs, 4), 128, 0, st>>>(a);
  } else {
    int64_t threads = ceil_div(ceil_div(pieces, PER), 32) * 32;
    if (threads > MOST) threads = MOST;
    k_gated_norm<T, VEC, true><<<(unsigned)a.runs, (unsigned)threads, 0, st>>>(a);
  }
  return cudaGetLastError();
}

}  // namespace gnorm
}  // namespace ssd

extern "C" ssd_status ssd_rmsnorm_gated(const ssd_norm_dims* d, const void* x, int64_t x_bstride, int64_t x_tstride,
                                        const void* z, int64_t z_bstride, int64_t z_tstride, const float* weight,
                                        float eps, void* out, int64_t out_bstride, int64_t out_tstride, void* stream) {
  using namespace ssd;
  if (!d || d->flags != 0) return SSD_ERR_INVALID_ARG;
  if (d->io_dtype != SSD_F32 && d->io_dtype != SSD_BF16) return SSD_ERR_DTYPE;
  const int64_t B = d->batch, L = d->seqlen, F = d->features, G = d->ngroups;
  if (B < 1 || L < 1 || F < 1 || G < 1 || F % G != 0) return SSD_ERR_SHAPE;
  if (B > 0x7fffffff || L > 0x7fffffff || F > 0x7fffffff || B * L > 0x7fffffff / G) return SSD_ERR_UNSUPPORTED;
  if (!x || !out || !(eps >= 0.0f)) return SSD_ERR_INVALID_ARG;
  const size_t es = io_bytes(d->io_dtype);
  const RowArg rx{x, x_bstride, x_tstride, F}, rz{z, z_bstride, z_tstride, F}, ro{out, out_bstride, out_tstride, F};
  ssd_status s;
  if ((s = check_rows(rx, B, L, es, false)) != SSD_OK || (s = check_rows(ro, B, L, es, true)) != SSD_OK) return s;
  if (z && (s = check_rows(rz, B, L, es, false)) != SSD_OK) return s;
  if (!f32_aligned(weight)) return SSD_ERR_ALIGN;
  const Span so{out, row_extent(ro, B, L, es)}, sx{x, row_extent(rx, B, L, es)},
      sz{z, z ? row_extent(rz, B, L, es) : 0}, sw{weight, sizeof(float) * F};
  const bool in_place = x == out && (B == 1 || x_bstride == out_bstride) && (L == 1 || x_tstride == out_tstride);
  if ((!in_place && spans_meet(so, sx)) || spans_meet(so, sz) || spans_meet(so, sw)) return SSD_ERR_INVALID_ARG;
  bool vec = rows_on_16(rx, B, L, es) && rows_on_16(ro, B, L, es) && (!z || rows_on_16(rz, B, L, es));
  vec = vec && (F / G * es) % 16 == 0;
  auto go = [&](auto t, auto v) {
    using T = decltype(t);
    gnorm::Args<T> a{};
    a.x = Rows<const T>{(const T*)x, x_bstride, x_tstride};
    a.z = Rows<const T>{(const T*)z, z_bstride, z_tstride};
    a.out = Rows<T>{(T*)out, out_bstride, out_tstride};
    a.weight = weight;
    a.eps = eps;
    a.groups = (uint32_t)G;
    a.L = (uint32_t)L;
    a.runs = B * L * G;
    a.n = F / G;
    return gnorm::launch<T, v.value>(a, static_cast<cudaStream_t>(stream));
  };
  if (d->io_dtype == SSD_BF16)
    return cuda_status(vec ? go(__nv_bfloat16(), std::integral_constant<int, 8>())
                           : go(__nv_bfloat16(), std::integral_constant<int, 1>()));
  return cuda_status(vec ? go(float(), std::integral_constant<int, 4>())
                         : go(float(), std::integral_constant<int, 1>()));
}
