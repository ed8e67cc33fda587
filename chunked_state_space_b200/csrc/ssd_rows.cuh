// Shared by the layer operators around the scan (convolution, selective scan,
// gated norm): strided rows of dense channels, vector access to them, the
// checks of their entry points, and the scalar functions they apply.
#pragma once

#include "ssd_common.cuh"

namespace ssd {

// Element (b, t, c) at p + b*bs + t*ts + c.
template <typename T>
struct Rows {
  T* p;
  int64_t bs, ts;
  __device__ __forceinline__ T* row(int64_t b, int64_t t) const { return p + b * bs + t * ts; }
};

// VEC consecutive elements moved by one access (16 bytes, or one element where
// the rows do not start on 16 bytes).
template <typename T, int VEC>
struct alignas(sizeof(T) * VEC) Pack {
  T v[VEC];
};

template <typename T, int VEC>
__device__ __forceinline__ Pack<T, VEC> load_pack(const T* p) {
  return *reinterpret_cast<const Pack<T, VEC>*>(p);
}
template <typename T, int VEC>
__device__ __forceinline__ void store_pack(T* p, const Pack<T, VEC>& v) {
  *reinterpret_cast<Pack<T, VEC>*>(p) = v;
}

// v / (1 + e^-v); e^-v = inf for v < -88 gives -0, as the limit does.
__device__ __forceinline__ float silu(float v) { return __fdividef(v, 1.0f + __expf(-v)); }

__device__ __forceinline__ int64_t row_length(const int32_t* lengths, int64_t b, int64_t L) {
  if (!lengths) return L;
  const int64_t n = lengths[b];
  return n < 0 ? 0 : n > L ? L : n;
}

// Host side: what an entry point knows of one tensor of rows.
struct RowArg {
  const void* p;
  int64_t bs, ts;
  int64_t width;  // dense elements per row
};

inline size_t io_bytes(int io) { return io == SSD_BF16 ? 2 : 4; }

// Bytes from the first to behind the last element.
inline size_t row_extent(const RowArg& r, int64_t B, int64_t L, size_t es) {
  return es * (size_t)((B > 1 ? (B - 1) * r.bs : 0) + (L > 1 ? (L - 1) * r.ts : 0) + r.width);
}

// Inputs: strides >= 0.  Outputs: rows apart from one another, the tokens of a
// sequence inside the stride between sequences or the other way round.
inline ssd_status check_rows(const RowArg& r, int64_t B, int64_t L, size_t es, bool output) {
  if ((B > 1 && r.bs < 0) || (L > 1 && r.ts < 0)) return SSD_ERR_SHAPE;
  if (output) {
    const bool tokens_inside = (L == 1 || r.ts >= r.width) && (B == 1 || r.bs >= (L > 1 ? (L - 1) * r.ts : 0) + r.width);
    const bool batch_inside = (B == 1 || r.bs >= r.width) && (L == 1 || r.ts >= (B > 1 ? (B - 1) * r.bs : 0) + r.width);
    if (!tokens_inside && !batch_inside) return SSD_ERR_SHAPE;
  }
  return (reinterpret_cast<uintptr_t>(r.p) & (es - 1)) ? SSD_ERR_ALIGN : SSD_OK;
}

// Whether every row can be read in 16-byte pieces.
inline bool rows_on_16(const RowArg& r, int64_t B, int64_t L, size_t es) {
  return (reinterpret_cast<uintptr_t>(r.p) & 15u) == 0 && (B == 1 || (r.bs * es) % 16 == 0) &&
         (L == 1 || (r.ts * es) % 16 == 0) && (r.width * es) % 16 == 0;
}

struct Span {
  const void* p;
  size_t bytes;
};
inline bool spans_meet(const Span& a, const Span& b) {
  if (!a.p || !b.p) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return x < y + b.bytes && y < x + a.bytes;
}

inline bool f32_aligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

}  // namespace ssd
