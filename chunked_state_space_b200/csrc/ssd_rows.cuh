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

// VEC consecutive elements as one access moves them: 16 bytes, or two elements
// or one where rows do not start on 16 bytes (four bf16 beside four f32).  Kept as
// whole words until an element is asked for: unpacked where they are loaded,
// each load would be waited for on the spot.
template <typename T, int VEC>
struct Pack;
template <>
struct alignas(16) Pack<__nv_bfloat16, 8> {
  uint32_t w[4];
  __device__ __forceinline__ float get(int i) const {
    return __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
  }
  __device__ __forceinline__ void set2(int i, float lo, float hi) {  // elements i (even) and i + 1
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    w[i / 2] = *reinterpret_cast<const uint32_t*>(&v);
  }
};
template <>
struct alignas(8) Pack<__nv_bfloat16, 4> {
  uint32_t w[2];
  __device__ __forceinline__ float get(int i) const {
    return __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
  }
};
template <>
struct alignas(4) Pack<__nv_bfloat16, 2> {
  uint32_t w;
  __device__ __forceinline__ float get(int i) const { return __uint_as_float(i & 1 ? w & 0xffff0000u : w << 16); }
  __device__ __forceinline__ void set2(int, float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    w = *reinterpret_cast<const uint32_t*>(&v);
  }
};
template <>
struct alignas(8) Pack<float, 2> {
  float w[2];
  __device__ __forceinline__ float get(int i) const { return w[i]; }
  __device__ __forceinline__ void set2(int, float lo, float hi) { w[0] = lo, w[1] = hi; }
};
template <>
struct alignas(16) Pack<float, 4> {
  float w[4];
  __device__ __forceinline__ float get(int i) const { return w[i]; }
  __device__ __forceinline__ void set2(int i, float lo, float hi) { w[i] = lo, w[i + 1] = hi; }
};
template <>
struct Pack<__nv_bfloat16, 1> {
  uint16_t w;
  __device__ __forceinline__ float get(int) const { return __uint_as_float((uint32_t)w << 16); }
  __device__ __forceinline__ void set(float v) { w = __bfloat16_as_ushort(__float2bfloat16_rn(v)); }
};
template <>
struct Pack<float, 1> {
  float w;
  __device__ __forceinline__ float get(int) const { return w; }
  __device__ __forceinline__ void set(float v) { w = v; }
};

template <typename T, int VEC>
__device__ __forceinline__ Pack<T, VEC> load_pack(const T* p) {
  return *reinterpret_cast<const Pack<T, VEC>*>(p);
}
template <typename T, int VEC>
__device__ __forceinline__ void store_pack(T* p, const Pack<T, VEC>& v) {
  *reinterpret_cast<Pack<T, VEC>*>(p) = v;
}
template <typename T, int VEC>
__device__ __forceinline__ Pack<T, VEC> to_pack(const float (&v)[VEC]) {
  Pack<T, VEC> r;
  if constexpr (VEC == 1) {
    r.set(v[0]);
  } else {
#pragma unroll
    for (int i = 0; i < VEC; i += 2) r.set2(i, v[i], v[i + 1]);
  }
  return r;
}

// Two f32 values per instruction (packed f32x2), each rounded like the scalar
// operation.
struct F2 {
  float x, y;
};
__device__ __forceinline__ F2 both(float v) { return {v, v}; }
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 d;
  asm("{\n\t.reg .b64 ra, rb, rd;\n\t"
      "mov.b64 ra, {%2, %3};\n\t"
      "mov.b64 rb, {%4, %5};\n\t"
      "mul.rn.f32x2 rd, ra, rb;\n\t"
      "mov.b64 {%0, %1}, rd;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  F2 d;
  asm("{\n\t.reg .b64 ra, rb, rd;\n\t"
      "mov.b64 ra, {%2, %3};\n\t"
      "mov.b64 rb, {%4, %5};\n\t"
      "add.rn.f32x2 rd, ra, rb;\n\t"
      "mov.b64 {%0, %1}, rd;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 d;
  asm("{\n\t.reg .b64 ra, rb, rc, rd;\n\t"
      "mov.b64 ra, {%2, %3};\n\t"
      "mov.b64 rb, {%4, %5};\n\t"
      "mov.b64 rc, {%6, %7};\n\t"
      "fma.rn.f32x2 rd, ra, rb, rc;\n\t"
      "mov.b64 {%0, %1}, rd;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}

__device__ __forceinline__ float ex2(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float rcp(float v) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

constexpr float LOG2E = 1.4426950408889634f;

// v / (1 + e^-v); e^-v = inf for v < -88 gives -0, as the limit does.
__device__ __forceinline__ float silu(float v) { return v * rcp(1.0f + ex2(v * -LOG2E)); }
__device__ __forceinline__ F2 silu2(F2 v) {
  const F2 t = mul2(v, both(-LOG2E)), d = add2(F2{ex2(t.x), ex2(t.y)}, both(1.0f));
  return mul2(v, F2{rcp(d.x), rcp(d.y)});
}

__device__ __forceinline__ int64_t row_length(const int32_t* lengths, int64_t b, int64_t L) {
  if (!lengths) return L;
  const int64_t n = lengths[b];
  return n < 0 ? 0 : n > L ? L : n;
}

// N consecutive f32 parameters; ALIGNED: N is a multiple of 4 and p on 16 bytes.
template <int N, bool ALIGNED>
__device__ __forceinline__ void load_params(const float* p, float (&v)[N]) {
  if constexpr (ALIGNED) {
#pragma unroll
    for (int i = 0; i < N; i += 4) *reinterpret_cast<float4*>(&v[i]) = *reinterpret_cast<const float4*>(p + i);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = p[i];
  }
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

// Whether every row can be read in pieces of `bytes`.
inline bool rows_on(const RowArg& r, int64_t B, int64_t L, size_t es, size_t bytes) {
  return reinterpret_cast<uintptr_t>(r.p) % bytes == 0 && (B == 1 || (r.bs * es) % bytes == 0) &&
         (L == 1 || (r.ts * es) % bytes == 0) && (r.width * es) % bytes == 0;
}
inline bool rows_on_16(const RowArg& r, int64_t B, int64_t L, size_t es) { return rows_on(r, B, L, es, 16); }

struct Span {
  const void* p;
  size_t bytes;
};
inline bool spans_meet(const Span& a, const Span& b) {
  if (!a.p || !b.p) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return x < y + b.bytes && y < x + a.bytes;
}

inline bool on_16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool f32_aligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

}  // namespace ssd
