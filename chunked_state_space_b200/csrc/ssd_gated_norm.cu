// The gated RMS norm behind a scan:
//   u = x silu(z);  out = weight u / sqrt(mean over the feature's group of u^2 + eps)
// Bound by HBM: x and z are read once and out is written once.  A run of
// features (one group of one row) is held in registers as u between the sum
// and the scaling, up to five 16-byte pieces per thread; blocks stay for many
// rows, with the next row's loads under way while this one's sum is reduced.
// The sum of squares is f32, in a fixed order.
#include "ssd_rows.cuh"

namespace ssd {
namespace gnorm {

constexpr int FIVE = 5;    // pieces of a row per thread of a block
constexpr int MOST = 640;  // threads of a block (which leaves a thread 96 registers)

template <typename T>
struct Args {
  Rows<const T> x, z;
  Rows<T> out;
  const float* weight;
  float eps;
  int64_t rows;
  uint32_t L;
  int64_t n;  // features of a group
};

// u of a piece, and the sum of its squares
template <typename T, int VEC>
__device__ __forceinline__ float gated(const Pack<T, VEC>& x, const Pack<T, VEC>& z, bool gate, float (&u)[VEC]) {
  if constexpr (VEC == 1) {
    u[0] = gate ? x.get(0) * silu(z.get(0)) : x.get(0);
    return u[0] * u[0];
  } else {
    F2 ss = both(0.f);
#pragma unroll
    for (int i = 0; i < VEC; i += 2) {
      F2 v{x.get(i), x.get(i + 1)};
      if (gate) v = mul2(v, silu2(F2{z.get(i), z.get(i + 1)}));
      ss = fma2(v, v, ss);
      u[i] = v.x, u[i + 1] = v.y;
    }
    return ss.x + ss.y;
  }
}

// u times inv and the weights
template <int VEC>
__device__ __forceinline__ void scaled(float (&u)[VEC], float inv, const float (&w)[VEC]) {
  if constexpr (VEC == 1) {
    u[0] *= inv * w[0];
  } else {
#pragma unroll
    for (int i = 0; i < VEC; i += 2) {
      const F2 v = mul2(mul2(F2{u[i], u[i + 1]}, both(inv)), F2{w[i], w[i + 1]});
      u[i] = v.x, u[i + 1] = v.y;
    }
  }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}

// A run of at most 16 pieces: a piece to a thread, `lanes` threads (a power of
// two) to a run, neighbouring groups side by side.
template <typename T, int VEC>
__global__ void __launch_bounds__(256) k_gated_norm_short(const Args<T> a, uint32_t groups, uint32_t runs, int lanes) {
  const uint32_t run = blockIdx.x * (256u / lanes) + threadIdx.x / lanes;
  const int p = threadIdx.x & (lanes - 1);
  const bool on = run < runs && p * VEC < a.n;  // the others take part in the shuffles
  const uint32_t row = run / groups, g = run - row * groups, b = row / a.L, t = row - b * a.L;
  const int64_t f = (int64_t)g * a.n + p * VEC;  // the piece's first feature
  float u[VEC] = {}, w[VEC], ss = 0.f;
  if (on) {
    const bool gate = a.z.p != nullptr;
    const Pack<T, VEC> x = load_pack<T, VEC>(a.x.row(b, t) + f), z = load_pack<T, VEC>((gate ? a.z : a.x).row(b, t) + f);
#pragma unroll
    for (int i = 0; i < VEC; ++i) w[i] = 1.f;
    if (a.weight) load_params<VEC, (VEC >= 4)>(a.weight + f, w);
    ss = gated(x, z, gate, u);
  }
  for (int off = lanes / 2; off > 0; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
  if (on) {
    scaled(u, 1.0f / sqrtf(ss / (float)a.n + a.eps), w);
    store_pack<T, VEC>(a.out.row(b, t) + f, to_pack<T, VEC>(u));
  }
}

// Runs of group blockIdx.y, one at a time per warp (BLOCK false) or block.
template <typename T, int VEC, bool BLOCK, int PER>
__global__ void __launch_bounds__(BLOCK ? MOST : 128) k_gated_norm(const Args<T> a) {
  __shared__ float part[2][MOST / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int me = BLOCK ? (int)threadIdx.x : lane, all = BLOCK ? (int)blockDim.x : 32;
  const int64_t g0 = (int64_t)blockIdx.y * a.n;  // the group's first feature
  const int pieces = (int)(a.n / VEC);
  const bool gate = a.z.p != nullptr;
  int64_t row = BLOCK ? (int64_t)blockIdx.x : (int64_t)blockIdx.x * (blockDim.x >> 5) + warp;
  const int64_t step = BLOCK ? (int64_t)gridDim.x : (int64_t)gridDim.x * (blockDim.x >> 5);
  // A warp with a run of its own holds the weights; a block reads them again for each row (from L1): their registers
  // would cost it a quarter of its warps (16384 rows of 5120 features bf16: 97 us, against 82).
  auto weights = [&](int k, float (&w)[VEC]) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) w[i] = 1.f;
    if (a.weight && me + k * all < pieces) load_params<VEC, (VEC >= 4)>(a.weight + g0 + (int64_t)(me + k * all) * VEC, w);
  };
  float held[BLOCK ? 1 : PER][VEC];
  if constexpr (!BLOCK) {
#pragma unroll
    for (int k = 0; k < PER; ++k) weights(k, held[k]);
  }
  Pack<T, VEC> x[PER], z[PER];
  auto fetch = [&](int64_t r) {
    const int64_t b = r / a.L, t = r - b * a.L;
#pragma unroll
    for (int k = 0; k < PER; ++k) {
      const int p = me + k * all;
      if (p < pieces) {
        x[k] = load_pack<T, VEC>(a.x.row(b, t) + g0 + (int64_t)p * VEC);
        if (gate) z[k] = load_pack<T, VEC>(a.z.row(b, t) + g0 + (int64_t)p * VEC);
      }
    }
  };
  if (row < a.rows) fetch(row);
  for (int turn = 0; row < a.rows; row += step, turn ^= 1) {
    float u[PER][VEC];
    float ss = 0.f;
#pragma unroll
    for (int k = 0; k < PER; ++k) {
      if (me + k * all < pieces) ss += gated(x[k], z[k], gate, u[k]);
    }
    if (row + step < a.rows) fetch(row + step);
    ss = warp_sum(ss);
    if (BLOCK) {
      // two sets of sums in turn: a warp that is a row ahead does not write over what another still reads
      if (lane == 0) part[turn][warp] = ss;
      __syncthreads();
      ss = 0.f;
      for (int k = 0; k < all / 32; ++k) ss += part[turn][k];
    }
    const float inv = 1.0f / sqrtf(ss / (float)a.n + a.eps);
    const int64_t b = row / a.L, t = row - b * a.L;
    T* out = a.out.row(b, t) + g0;
#pragma unroll
    for (int k = 0; k < PER; ++k) {
      const int p = me + k * all;
      if (p < pieces) {
        if constexpr (BLOCK) weights(k, held[0]);
        scaled(u[k], inv, held[BLOCK ? 0 : k]);
        store_pack<T, VEC>(out + (int64_t)p * VEC, to_pack<T, VEC>(u[k]));
      }
    }
  }
}

// A run longer than the registers of a block hold: read twice.
template <typename T, int VEC>
__global__ void __launch_bounds__(MOST) k_gated_norm_long(const Args<T> a) {
  __shared__ float part[MOST / 32];
  const int64_t row = blockIdx.x, b = row / a.L, t = row - b * a.L, g0 = (int64_t)blockIdx.y * a.n;
  const bool gate = a.z.p != nullptr;
  const T* x = a.x.row(b, t) + g0;
  const T* z = gate ? a.z.row(b, t) + g0 : x;
  T* out = a.out.row(b, t) + g0;
  const int64_t pieces = a.n / VEC;
  float u[VEC], ss = 0.f;
  for (int64_t p = threadIdx.x; p < pieces; p += MOST) {
    ss += gated(load_pack<T, VEC>(x + p * VEC), load_pack<T, VEC>(z + p * VEC), gate, u);
  }
  ss = warp_sum(ss);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = ss;
  __syncthreads();
  ss = 0.f;
  for (int k = 0; k < MOST / 32; ++k) ss += part[k];
  const float inv = 1.0f / sqrtf(ss / (float)a.n + a.eps);
  for (int64_t p = threadIdx.x; p < pieces; p += MOST) {
    gated(load_pack<T, VEC>(x + p * VEC), load_pack<T, VEC>(z + p * VEC), gate, u);
    float w[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) w[i] = 1.f;
    if (a.weight) load_params<VEC, (VEC >= 4)>(a.weight + g0 + p * VEC, w);
    scaled(u, inv, w);
    store_pack<T, VEC>(out + p * VEC, to_pack<T, VEC>(u));
  }
}

// A run of up to 16 pieces takes part of a warp (16384 rows of eight runs of
// eight features bf16 4 us, 34 with a warp each), one of up to 160 a warp with
// as few pieces per thread as hold it (registers for more would cost it warps:
// 9280 rows of eight runs of 560 features bf16 66 us, 85 with five pieces for
// all), a longer one a block of as many warps as hold it; the grid is what the
// SMs hold.
template <typename T, int VEC>
cudaError_t launch(const Args<T>& a, unsigned groups, cudaStream_t st) {
  const int64_t pieces = a.n / VEC;
  auto blocks = [](int64_t want, int64_t most) { return (unsigned)(want < most ? want : most); };
  auto warp = [&](auto per, int64_t resident) {
    k_gated_norm<T, VEC, false, per.value><<<dim3(blocks(ceil_div(a.rows, 4), 148 * resident), groups), 128, 0, st>>>(a);
  };
  if (pieces <= 16 && a.rows * groups <= 0x7fffffff) {
    int lanes = 1;
    while (lanes < pieces) lanes *= 2;
    const int64_t runs = a.rows * groups;
    k_gated_norm_short<T, VEC><<<(unsigned)ceil_div(runs, 256 / lanes), 256, 0, st>>>(a, groups, (uint32_t)runs, lanes);
  } else if (pieces <= 32) {
    warp(std::integral_constant<int, 1>(), 8);
  } else if (pieces <= 64) {
    warp(std::integral_constant<int, 2>(), 6);
  } else if (pieces <= 96) {
    warp(std::integral_constant<int, 3>(), 5);
  } else if (pieces <= 160) {
    warp(std::integral_constant<int, 5>(), 4);
  } else if (pieces <= MOST * FIVE) {
    const int64_t threads = ceil_div(ceil_div(pieces, FIVE), 32) * 32;
    k_gated_norm<T, VEC, true, FIVE>
        <<<dim3(blocks(a.rows, 148 * (MOST / threads)), groups), (unsigned)threads, 0, st>>>(a);
  } else {
    k_gated_norm_long<T, VEC><<<dim3((unsigned)a.rows, groups), MOST, 0, st>>>(a);
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
  if (B > 0x7fffffff || L > 0x7fffffff || F > 0x7fffffff || B * L > 0x7fffffff || G > 65535) return SSD_ERR_UNSUPPORTED;
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
  auto on = [&](size_t bytes) {
    return rows_on(rx, B, L, es, bytes) && rows_on(ro, B, L, es, bytes) && (!z || rows_on(rz, B, L, es, bytes)) &&
           (F / G * es) % bytes == 0;
  };
  auto go = [&](auto t, auto v) {
    using T = decltype(t);
    gnorm::Args<T> a{};
    a.x = Rows<const T>{(const T*)x, x_bstride, x_tstride};
    a.z = Rows<const T>{(const T*)z, z_bstride, z_tstride};
    a.out = Rows<T>{(T*)out, out_bstride, out_tstride};
    a.weight = weight;
    a.eps = eps;
    a.L = (uint32_t)L;
    a.rows = B * L;
    a.n = F / G;
    return gnorm::launch<T, v.value>(a, (unsigned)G, static_cast<cudaStream_t>(stream));
  };
  auto pieces = [&](auto t, auto whole) {
    if (on(16) && on_16(weight)) return go(t, whole);
    if (on(2 * es)) return go(t, std::integral_constant<int, 2>());
    return go(t, std::integral_constant<int, 1>());
  };
  return cuda_status(d->io_dtype == SSD_BF16 ? pieces(__nv_bfloat16(), std::integral_constant<int, 8>())
                                             : pieces(float(), std::integral_constant<int, 4>()));
}
