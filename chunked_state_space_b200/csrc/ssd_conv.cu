// Short causal depthwise convolution with bias and SiLU, for prompts and for
// single tokens:
//   y[b,t,c] = act(bias[c] + sum_{k<W} w[c,k] x[b, t-(W-1)+k, c])
// with the inputs before the first token taken from a cached state (or 0).
//
// Bound by HBM: each element is read once and written once, against about a
// dozen fp32 operations and two special-function ones (e^-v and a reciprocal).
// A thread owns 16 bytes of channels (two elements or one where rows are not
// 16-byte aligned) and a run of consecutive tokens, and keeps the last W-1
// inputs in registers, so a tap costs no further load; only the W-1 rows before
// a run are read twice.
#include "ssd_rows.cuh"

namespace ssd {
namespace conv {

constexpr int THREADS = 128;

template <typename T>
struct Args {
  Rows<const T> x;
  Rows<T> y;
  const float* weight;
  const float* bias;
  const T* init;
  T* final_state;
  const int32_t* lengths;
  int64_t B, L, C;
  uint32_t nvec, ntiles, total;
  int64_t tile;  // tokens per thread, at least W - 1
};

template <int W, int VEC, bool SILU>
struct Taps {
  float w[W][VEC], b[VEC];
  __device__ __forceinline__ void load(const float* weight, const float* bias, int64_t c) {
    float rows[VEC * W];
    load_params<VEC * W, (VEC >= 4)>(weight + c * W, rows);
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
#pragma unroll
      for (int k = 0; k < W; ++k) w[k][i] = rows[i * W + k];
      b[i] = 0.f;
    }
    if (bias) load_params<VEC, (VEC >= 4)>(bias + c, b);
  }
  // old[0] is the oldest of the W-1 inputs before `in`
  template <typename T>
  __device__ __forceinline__ Pack<T, VEC> apply(const float (&old)[W - 1][VEC], const float (&in)[VEC]) const {
    float out[VEC];
    if constexpr (VEC == 1) {
      float acc = b[0];
#pragma unroll
      for (int k = 0; k < W - 1; ++k) acc = fmaf(w[k][0], old[k][0], acc);
      acc = fmaf(w[W - 1][0], in[0], acc);
      out[0] = SILU ? silu(acc) : acc;
    } else {
#pragma unroll
      for (int i = 0; i < VEC; i += 2) {
        F2 acc{b[i], b[i + 1]};
#pragma unroll
        for (int k = 0; k < W - 1; ++k) acc = fma2(F2{w[k][i], w[k][i + 1]}, F2{old[k][i], old[k][i + 1]}, acc);
        acc = fma2(F2{w[W - 1][i], w[W - 1][i + 1]}, F2{in[i], in[i + 1]}, acc);
        if (SILU) acc = silu2(acc);
        out[i] = acc.x, out[i + 1] = acc.y;
      }
    }
    return to_pack<T, VEC>(out);
  }
};

// AHEAD: rows that a thread loads before it computes the AHEAD rows before them
template <typename T, int W, int VEC, bool SILU, int AHEAD>
__global__ void __launch_bounds__(THREADS, AHEAD == 8 ? 3 : 4) k_conv_fwd(const Args<T> a) {
  const uint32_t idx = blockIdx.x * THREADS + threadIdx.x;
  if (idx >= a.total) return;
  const uint32_t r = idx / a.nvec;
  const int64_t c = (int64_t)(idx - r * a.nvec) * VEC;
  const uint32_t b32 = r / a.ntiles, tile = r - b32 * a.ntiles;
  const int64_t b = b32;
  const int64_t len = row_length(a.lengths, b, a.L);
  const int64_t t0 = (int64_t)tile * a.tile;
  if (t0 >= len && tile != 0) return;
  const int64_t t1 = t0 + a.tile < len ? t0 + a.tile : len;
  float old[W - 1][VEC];  // the W-1 inputs before the next token, oldest first
#pragma unroll
  for (int k = 0; k < W - 1; ++k) {
    Pack<T, VEC> v{};
    if (tile != 0) {
      v = load_pack<T, VEC>(a.x.row(b, t0 - (W - 1) + k) + c);
    } else if (a.init) {
      v = load_pack<T, VEC>(a.init + (b * (W - 1) + k) * a.C + c);
    }
#pragma unroll
    for (int i = 0; i < VEC; ++i) old[k][i] = v.get(i);
  }
  if (tile == 0 && a.final_state) {
    // The thread that read these channels of init_state writes their final
    // state, so that both may be one buffer.
    Pack<T, VEC> last[W - 1];
#pragma unroll
    for (int k = 0; k < W - 1; ++k) {
      const int64_t t = len - (W - 1) + k;
      last[k] = Pack<T, VEC>{};
      if (t >= 0)
        last[k] = load_pack<T, VEC>(a.x.row(b, t) + c);
      else if (a.init)
        last[k] = load_pack<T, VEC>(a.init + (b * (W - 1) + (t + W - 1)) * a.C + c);
    }
#pragma unroll
    for (int k = 0; k < W - 1; ++k) store_pack<T, VEC>(a.final_state + (b * (W - 1) + k) * a.C + c, last[k]);
  }
  Taps<W, VEC, SILU> taps;
  taps.load(a.weight, a.bias, c);
  const T* x = a.x.row(b, t0) + c;
  T* y = a.y.row(b, t0) + c;
  auto token = [&](const Pack<T, VEC>& in) {
    float cur[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) cur[i] = in.get(i);
    store_pack<T, VEC>(y, taps.template apply<T>(old, cur));
    y += a.y.ts;
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
#pragma unroll
      for (int k = 0; k + 1 < W - 1; ++k) old[k][i] = old[k + 1][i];
      old[W - 2][i] = cur[i];
    }
  };
  int64_t t = t0;
  if (t + AHEAD <= t1) {
    Pack<T, VEC> in[AHEAD], next[AHEAD];
#pragma unroll
    for (int j = 0; j < AHEAD; ++j, x += a.x.ts) in[j] = load_pack<T, VEC>(x);
#pragma unroll 1
    for (; t + AHEAD <= t1; t += AHEAD) {
      if (t + 2 * AHEAD <= t1) {
#pragma unroll
        for (int j = 0; j < AHEAD; ++j, x += a.x.ts) next[j] = load_pack<T, VEC>(x);
      }
#pragma unroll
      for (int j = 0; j < AHEAD; ++j) token(in[j]);
#pragma unroll
      for (int j = 0; j < AHEAD; ++j) in[j] = next[j];
    }
  }
#pragma unroll 1
  for (; t < t1; ++t, x += a.x.ts) token(load_pack<T, VEC>(x));
}

// One token: a thread takes as many channels of up to ROWS sequences, with
// their weights loaded once.
template <typename T, int W, int VEC, bool SILU, int ROWS>
__global__ void __launch_bounds__(THREADS) k_conv_step(const T* __restrict__ x, int64_t xbs, const float* weight,
                                                       const float* bias, T* state, T* __restrict__ y, int64_t ybs,
                                                       int64_t B, int64_t C, uint32_t nvec, uint32_t total) {
  const uint32_t idx = blockIdx.x * THREADS + threadIdx.x;
  if (idx >= total) return;
  const uint32_t r = idx / nvec;
  const int64_t b0 = (int64_t)r * ROWS, c = (int64_t)(idx - r * nvec) * VEC;
  Pack<T, VEC> seen[ROWS][W];
#pragma unroll
  for (int j = 0; j < ROWS; ++j) {
    if (b0 + j < B) {
#pragma unroll
      for (int k = 0; k < W - 1; ++k) seen[j][k] = load_pack<T, VEC>(state + ((b0 + j) * (W - 1) + k) * C + c);
      seen[j][W - 1] = load_pack<T, VEC>(x + (b0 + j) * xbs + c);
    }
  }
  Taps<W, VEC, SILU> taps;
  taps.load(weight, bias, c);
#pragma unroll
  for (int j = 0; j < ROWS; ++j) {
    if (b0 + j < B) {
      float old[W - 1][VEC], cur[VEC];
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
#pragma unroll
        for (int k = 0; k < W - 1; ++k) old[k][i] = seen[j][k].get(i);
        cur[i] = seen[j][W - 1].get(i);
      }
      store_pack<T, VEC>(y + (b0 + j) * ybs + c, taps.template apply<T>(old, cur));
#pragma unroll
      for (int k = 0; k < W - 1; ++k) store_pack<T, VEC>(state + ((b0 + j) * (W - 1) + k) * C + c, seen[j][k + 1]);
    }
  }
}

// Tokens per thread: as many as leave every SM 4096 channels at a time (the
// rows before a run are read twice, so longer runs read less), at most 64.
// 4 x 4096 tokens x 1792 channels bf16 29.5 us, 33 with 8192 channels; 5 x 1111
// x 1792 f32 6.3 us, 8.3 with 2048.
inline int tile_tokens(int64_t B, int64_t L, int64_t C) {
  int tile = 64;
  while (tile > 8 && B * C * ceil_div(L, tile) < 148 * 4096) tile /= 2;
  return tile;
}

template <typename T, int W, int VEC>
cudaError_t launch(const Args<T>& a0, bool use_silu, cudaStream_t st) {
  Args<T> a = a0;
  const int64_t nvec = a.C / VEC;
  int64_t tile = tile_tokens(a.B, a.L, a.C);
  while (a.B * nvec * ceil_div(a.L, tile) > 0x7fff0000) tile *= 2;  // thread indices stay below 2^31
  a.tile = tile;
  a.nvec = (uint32_t)nvec;
  a.ntiles = (uint32_t)ceil_div(a.L, tile);
  a.total = (uint32_t)(a.B * nvec * a.ntiles);
  const unsigned blocks = (a.total + THREADS - 1) / THREADS;
  // Eight rows ahead keep HBM busy at three blocks per SM (131072 tokens x 5376 channels bf16 481 us, 520 with four
  // rows and four blocks); short runs are over before that pays (5 x 1111 tokens x 1792 channels f32 6.3 us with four
  // rows, 7.3 with eight).
  auto go = [&](auto silu) {
    if (tile >= 32)
      k_conv_fwd<T, W, VEC, silu.value, 8><<<blocks, THREADS, 0, st>>>(a);
    else
      k_conv_fwd<T, W, VEC, silu.value, 4><<<blocks, THREADS, 0, st>>>(a);
  };
  if (use_silu)
    go(std::true_type());
  else
    go(std::false_type());
  return cudaGetLastError();
}

template <typename T, int W, int VEC>
cudaError_t launch_step(const ssd_conv_dims* d, const void* x, int64_t xbs, const float* weight, const float* bias,
                        void* state, void* y, int64_t ybs, cudaStream_t st) {
  const int64_t nvec = d->channels / VEC;
  auto go = [&](auto silu, auto rows) {
    const uint32_t total = (uint32_t)(ceil_div(d->batch, rows.value) * nvec);
    k_conv_step<T, W, VEC, silu.value, rows.value><<<(total + THREADS - 1) / THREADS, THREADS, 0, st>>>(
        (const T*)x, xbs, weight, bias, (T*)state, (T*)y, ybs, d->batch, d->channels, (uint32_t)nvec, total);
  };
  // Four sequences a thread where that still makes a block for every other SM: 64 sequences of 5376 channels bf16
  // 2.8 us, 3.4 with one each, 256 5.1 and 8.2 (64 of 1792 channels: 2.7 and 2.1).
  const bool many = ceil_div(d->batch, 4) * nvec >= 74 * THREADS;
  auto pick = [&](auto silu) {
    if (many)
      go(silu, std::integral_constant<int, 4>());
    else
      go(silu, std::integral_constant<int, 1>());
  };
  if (d->flags & SSD_CONV_SILU)
    pick(std::true_type());
  else
    pick(std::false_type());
  return cudaGetLastError();
}

// f(T, W, VEC) for the call's type, width and alignment: 16-byte pieces (vec
// 2), pairs of elements (1) or single ones (0).
template <typename F>
cudaError_t dispatch(int io, int64_t width, int vec, F&& f) {
  auto with_width = [&](auto t, auto v) {
    switch (width) {
      case 2: return f(t, std::integral_constant<int, 2>(), v);
      case 3: return f(t, std::integral_constant<int, 3>(), v);
      default: return f(t, std::integral_constant<int, 4>(), v);
    }
  };
  auto with_type = [&](auto t, auto whole) {
    if (vec == 2) return with_width(t, whole);
    if (vec == 1) return with_width(t, std::integral_constant<int, 2>());
    return with_width(t, std::integral_constant<int, 1>());
  };
  return io == SSD_BF16 ? with_type(__nv_bfloat16(), std::integral_constant<int, 8>())
                        : with_type(float(), std::integral_constant<int, 4>());
}

ssd_status validate(const ssd_conv_dims* d, int64_t seqlen) {
  if (!d) return SSD_ERR_INVALID_ARG;
  if (d->flags & ~SSD_CONV_SILU) return SSD_ERR_INVALID_ARG;
  if (d->io_dtype != SSD_F32 && d->io_dtype != SSD_BF16) return SSD_ERR_DTYPE;
  if (d->batch < 1 || seqlen < 1 || d->channels < 1 || d->width < 1) return SSD_ERR_SHAPE;
  if (d->width < 2 || d->width > 4) return SSD_ERR_UNSUPPORTED;
  // thread indices stay below 2^31 (a run of tokens per thread can grow, a row cannot)
  if (d->channels > (int64_t(1) << 24) || d->batch > (int64_t(1) << 24) || d->batch * d->channels > 0x7fff0000 ||
      seqlen > 0x7fffffff)
    return SSD_ERR_UNSUPPORTED;
  return SSD_OK;
}

}  // namespace conv
}  // namespace ssd

extern "C" ssd_status ssd_conv_fwd(const ssd_conv_dims* d, const void* x, int64_t x_bstride, int64_t x_tstride,
                                   const float* weight, const float* bias, const void* init_state,
                                   const int32_t* lengths, void* y, int64_t y_bstride, int64_t y_tstride,
                                   void* final_state, void* stream) {
  using namespace ssd;
  ssd_status s = conv::validate(d, d ? d->seqlen : 1);
  if (s != SSD_OK) return s;
  if (!x || !weight || !y) return SSD_ERR_INVALID_ARG;
  const int64_t B = d->batch, L = d->seqlen, C = d->channels, W = d->width;
  const size_t es = io_bytes(d->io_dtype);
  const RowArg rx{x, x_bstride, x_tstride, C}, ry{y, y_bstride, y_tstride, C};
  const RowArg ri{init_state, (W - 1) * C, C, C}, rf{final_state, (W - 1) * C, C, C};
  if ((s = check_rows(rx, B, L, es, false)) != SSD_OK || (s = check_rows(ry, B, L, es, true)) != SSD_OK) return s;
  if (check_rows(ri, B, W - 1, es, false) != SSD_OK || check_rows(rf, B, W - 1, es, false) != SSD_OK ||
      !f32_aligned(weight) || !f32_aligned(bias) || !f32_aligned(lengths))
    return SSD_ERR_ALIGN;
  const Span sx{x, row_extent(rx, B, L, es)}, sy{y, row_extent(ry, B, L, es)}, sw{weight, sizeof(float) * C * W},
      sb{bias, sizeof(float) * C}, si{init_state, es * B * (W - 1) * C}, sl{lengths, sizeof(int32_t) * B},
      sf{final_state, es * B * (W - 1) * C};
  for (const Span& in : {sx, sw, sb, sl})
    if (spans_meet(sy, in) || spans_meet(sf, in)) return SSD_ERR_INVALID_ARG;
  if (spans_meet(sy, si) || spans_meet(sy, sf) || (final_state != init_state && spans_meet(sf, si)))
    return SSD_ERR_INVALID_ARG;
  auto on = [&](size_t bytes) {
    return rows_on(rx, B, L, es, bytes) && rows_on(ry, B, L, es, bytes) && rows_on(ri, B, W - 1, es, bytes) &&
           rows_on(rf, B, W - 1, es, bytes);
  };
  const int vec = on(16) && on_16(weight) && on_16(bias) ? 2 : on(2 * es) ? 1 : 0;
  return cuda_status(conv::dispatch(d->io_dtype, W, vec, [&](auto t, auto w, auto v) {
    using T = decltype(t);
    conv::Args<T> a{};
    a.x = Rows<const T>{(const T*)x, x_bstride, x_tstride};
    a.y = Rows<T>{(T*)y, y_bstride, y_tstride};
    a.weight = weight;
    a.bias = bias;
    a.init = (const T*)init_state;
    a.final_state = (T*)final_state;
    a.lengths = lengths;
    a.B = B;
    a.L = L;
    a.C = C;
    return conv::launch<T, w.value, v.value>(a, (d->flags & SSD_CONV_SILU) != 0, static_cast<cudaStream_t>(stream));
  }));
}

extern "C" ssd_status ssd_conv_step(const ssd_conv_dims* d, const void* x, int64_t x_bstride, const float* weight,
                                    const float* bias, void* state, void* y, int64_t y_bstride, void* stream) {
  using namespace ssd;
  ssd_status s = conv::validate(d, 1);
  if (s != SSD_OK) return s;
  if (!x || !weight || !state || !y) return SSD_ERR_INVALID_ARG;
  const int64_t B = d->batch, C = d->channels, W = d->width;
  const size_t es = io_bytes(d->io_dtype);
  const RowArg rx{x, x_bstride, 0, C}, ry{y, y_bstride, 0, C}, rs{state, (W - 1) * C, C, C};
  if ((s = check_rows(rx, B, 1, es, false)) != SSD_OK || (s = check_rows(ry, B, 1, es, true)) != SSD_OK) return s;
  if (check_rows(rs, B, W - 1, es, false) != SSD_OK || !f32_aligned(weight) || !f32_aligned(bias)) return SSD_ERR_ALIGN;
  const Span sx{x, row_extent(rx, B, 1, es)}, sy{y, row_extent(ry, B, 1, es)}, sw{weight, sizeof(float) * C * W},
      sb{bias, sizeof(float) * C}, ss{state, es * B * (W - 1) * C};
  for (const Span& in : {sx, sw, sb})
    if (spans_meet(sy, in) || spans_meet(ss, in)) return SSD_ERR_INVALID_ARG;
  if (spans_meet(sy, ss)) return SSD_ERR_INVALID_ARG;
  auto on = [&](size_t bytes) {
    return rows_on(rx, B, 1, es, bytes) && rows_on(ry, B, 1, es, bytes) && rows_on(rs, B, W - 1, es, bytes);
  };
  const int vec = on(16) && on_16(weight) && on_16(bias) ? 2 : on(2 * es) ? 1 : 0;
  return cuda_status(conv::dispatch(d->io_dtype, W, vec, [&](auto t, auto w, auto v) {
    return conv::launch_step<decltype(t), w.value, v.value>(d, x, x_bstride, weight, bias, state, y, y_bstride,
                                                            static_cast<cudaStream_t>(stream));
  }));
}
