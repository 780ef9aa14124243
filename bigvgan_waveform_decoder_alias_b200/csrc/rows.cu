// Operators on the rows of a token stream [rows, cols]: the root-mean-square
// norm with the residual's addition, in the stream's type or in 8 bits with a
// scale for each row, and the 8-bit quantisation of rows as they are.
//
//   h = x + residual (32 bits), rstd = 1 / sqrt(mean(h^2) + eps), t = h gain,
//   y = t rstd;   8 bits: a = max |t|, q = rint(t (127 / a)),
//                 scale = a rstd / 127
// q is written from t and a alone: rstd scales a row and its maximum alike, so
// it belongs into the scale.  max is exact in any order, hence q does not
// depend on how a row's sum is split over threads, nor on the batch.
//
// Bound by memory: each value is read once and written once.  A row lives in
// the registers of one warp or one block between its only read and its write;
// the sum of squares and the maximum go through one reduction together.  Rows
// past the registers of a block are read twice.
#include "token_types.cuh"

namespace bv {
namespace {

constexpr unsigned kInfBits = 0x7f800000u;

template <typename T, int N>
struct alignas(sizeof(T) * N) Pack {
  T v[N];
};

// N values at p, `valid` of them in range (the others 0).  Plain loads: the
// rows may be overwritten by this kernel (sum may be x or the residual).
template <typename T, int N>
__device__ __forceinline__ Pack<T, N> load_pack(const T *p, int valid) {
  Pack<T, N> r;
  if (valid >= N) {
    r = *reinterpret_cast<const Pack<T, N> *>(p);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) r.v[i] = i < valid ? p[i] : from_f32<T>(0.0f);
  }
  return r;
}
template <typename T, int N>
__device__ __forceinline__ void store_pack(T *p, const Pack<T, N> &r, int valid) {
  if (valid >= N) {
    *reinterpret_cast<Pack<T, N> *>(p) = r;
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (i < valid) p[i] = r.v[i];
  }
}

__device__ __forceinline__ unsigned abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// Sum of `s` and maximum of `m` over the row's threads (a warp, or the block),
// in every thread.  `buf` alternates between calls, so one barrier is enough.
struct Red {
  float s[2][32];
  unsigned m[2][32];
};
template <bool BLOCK>
__device__ __forceinline__ void reduce_row(float &s, unsigned &m, Red &red, int &buf) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  m = __reduce_max_sync(0xffffffffu, m);
  if constexpr (BLOCK) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
    if (lane == 0) {
      red.s[buf][warp] = s;
      red.m[buf][warp] = m;
    }
    __syncthreads();
    s = lane < nw ? red.s[buf][lane] : 0.0f;
    m = lane < nw ? red.m[buf][lane] : 0u;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    m = __reduce_max_sync(0xffffffffu, m);
    buf ^= 1;
  }
}

// 2^k for -126 <= k <= 127.
__device__ __forceinline__ float pow2(int k) { return __int_as_float((k + 127) << 23); }

// How a row's t becomes 8-bit values: q = rint((t pre) inv).
// A row with a value that is not finite has q = 0 and scale NaN.  Rows below
// 2^-100 are lifted by 2^64 first: 127 / a would overflow.
struct Quant {
  float pre, inv, scale;
};
__device__ __forceinline__ Quant make_quant(unsigned abits, float rstd) {
  Quant r{1.0f, 0.0f, 0.0f};
  if (abits >= kInfBits) {
    r.scale = __int_as_float(0x7fc00000);
  } else if (abits != 0) {
    float a = __uint_as_float(abits);
    float back = 1.0f;
    if (a < pow2(-100)) {
      r.pre = pow2(64);
      back = pow2(-64);
      a *= r.pre;
    }
    r.inv = __fdiv_rn(127.0f, a);
    r.scale = __fdiv_rn(__fmul_rn(a, rstd), 127.0f) * back;
  }
  return r;
}
__device__ __forceinline__ int8_t quantise(float t, const Quant &z) {
  // rint(t inv) is within [-127, 127]: |t| <= a, and a (127 / a) is off by at
  // most two roundings.  inv = 0 marks a row of zeros or of no finite scale.
  return z.inv == 0.0f ? (int8_t)0 : (int8_t)__float2int_rn(__fmul_rn(t * z.pre, z.inv));
}

// 1 / sqrt(mean + eps) of a row whose sum of squares is `s`.
__device__ __forceinline__ float row_rstd(float s, int cols, float eps) {
  return __frsqrt_rn(__fadd_rn(__fdiv_rn(s, (float)cols), eps));
}

// A thread holds NV groups of VEC values, group i at VEC (tid + i threads).
// BLOCK: a block a row; else a warp a row.
template <typename T, typename G, int VEC, int NV, bool BLOCK, bool NORM>
__global__ void __launch_bounds__(BLOCK ? 1024 : 128) rows_kernel(NormArgs a) {
  __shared__ Red red;
  const int tpr = BLOCK ? blockDim.x : 32;
  const int tid = BLOCK ? threadIdx.x : (threadIdx.x & 31);
  const int64_t row0 =
      BLOCK ? blockIdx.x : blockIdx.x * (int64_t)(blockDim.x >> 5) + (threadIdx.x >> 5);
  const int64_t step = BLOCK ? gridDim.x : gridDim.x * (int64_t)(blockDim.x >> 5);
  int buf = 0;
  Pack<G, VEC> g[NV];
  if (NORM && a.gain) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = VEC * (tid + i * tpr);
      if (c < a.cols) g[i] = load_pack<G, VEC>(static_cast<const G *>(a.gain) + c, a.cols - c);
    }
  }
  for (int64_t row = row0; row < a.rows; row += step) {
    float h[NV][VEC];
    {
      const T *x = static_cast<const T *>(a.x) + row * a.xs;
      const T *r = static_cast<const T *>(a.residual) + row * a.rs;
      Pack<T, VEC> px[NV], pr[NV];
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = VEC * (tid + i * tpr);
        if (c < a.cols) px[i] = load_pack<T, VEC>(x + c, a.cols - c);
        if (NORM && a.residual && c < a.cols) pr[i] = load_pack<T, VEC>(r + c, a.cols - c);
      }
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const bool in = VEC * (tid + i * tpr) < a.cols;
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          h[i][e] = in ? to_f32(px[i].v[e]) : 0.0f;
          if (NORM && a.residual && in) h[i][e] += to_f32(pr[i].v[e]);
        }
      }
    }
    auto t_of = [&](int i, int e) {
      return NORM && a.gain ? __fmul_rn(h[i][e], to_f32(g[i].v[e])) : h[i][e];
    };
    float s = 0.0f;
    unsigned m = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = VEC * (tid + i * tpr);
      if (c < a.cols) {
        if (NORM && a.sum) {
          Pack<T, VEC> o;
#pragma unroll
          for (int e = 0; e < VEC; ++e) o.v[e] = from_f32<T>(h[i][e]);
          store_pack<T, VEC>(static_cast<T *>(a.sum) + row * a.ss + c, o, a.cols - c);
        }
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          if (NORM) s = fmaf(h[i][e], h[i][e], s);
          if (a.q && c + e < a.cols) m = max(m, abs_bits(t_of(i, e)));
        }
      }
    }
    reduce_row<BLOCK>(s, m, red, buf);
    float rstd = 1.0f;
    if (NORM) {
      rstd = row_rstd(s, a.cols, a.eps);
      if (!(s < __uint_as_float(kInfBits))) {
        // The squares overflowed: if every h is finite, scale the row by a
        // power of two and sum again (hm is past 2^48 then, so that down is
        // a normal number).
        float s2 = 0.0f;
        unsigned hm = 0;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
          for (int e = 0; e < VEC; ++e) hm = max(hm, abs_bits(h[i][e]));
        reduce_row<BLOCK>(s2, hm, red, buf);
        if (hm < kInfBits) {
          const float down = pow2(167 - (int)(hm >> 23));  // the maximum to 2^40 .. 2^41
          s2 = 0.0f;
#pragma unroll
          for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int e = 0; e < VEC; ++e) s2 = fmaf(h[i][e] * down, h[i][e] * down, s2);
          unsigned none = 0;
          reduce_row<BLOCK>(s2, none, red, buf);
          rstd = row_rstd(s2, a.cols, a.eps * down * down) * down;
        }
      }
    }
    const Quant z = a.q ? make_quant(m, rstd) : Quant{1.0f, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = VEC * (tid + i * tpr);
      if (c < a.cols) {
        if (NORM && a.y) {
          Pack<T, VEC> o;
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            // (h rstd) gain: h rstd is at most sqrt(cols), so it cannot overflow
            float v = h[i][e] * rstd;
            if (a.gain) v *= to_f32(g[i].v[e]);
            o.v[e] = from_f32<T>(v);
          }
          store_pack<T, VEC>(static_cast<T *>(a.y) + row * a.ys + c, o, a.cols - c);
        }
        if (a.q) {
          Pack<int8_t, VEC> o;
#pragma unroll
          for (int e = 0; e < VEC; ++e) o.v[e] = quantise(t_of(i, e), z);
          store_pack<int8_t, VEC>(a.q + row * a.qs + c, o, a.cols - c);
        }
      }
    }
    if (a.q && tid == 0) a.scale[row] = z.scale;
  }
}

// Rows longer than a block's registers: one block a row, read twice (the
// second time mostly from L2).  The sum is written on the second read, by the
// thread that read its operands, so it may be x or the residual.
template <typename T, typename G, bool NORM>
__global__ void __launch_bounds__(1024) long_rows_kernel(NormArgs a) {
  __shared__ Red red;
  int buf = 0;
  const G *gain = static_cast<const G *>(a.gain);
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const T *x = static_cast<const T *>(a.x) + row * a.xs;
    const T *r = static_cast<const T *>(a.residual) + row * a.rs;
    auto h_of = [&](int c) {
      float h = to_f32(x[c]);
      if (NORM && a.residual) h += to_f32(r[c]);
      return h;
    };
    auto t_of = [&](float h, int c) {
      return NORM && gain ? __fmul_rn(h, to_f32(gain[c])) : h;
    };
    float s = 0.0f;
    unsigned m = 0, hm = 0;
    for (int c = threadIdx.x; c < a.cols; c += blockDim.x) {
      const float h = h_of(c);
      s = fmaf(h, h, s);
      hm = max(hm, abs_bits(h));
      m = max(m, abs_bits(t_of(h, c)));
    }
    reduce_row<true>(s, m, red, buf);
    float rstd = 1.0f;
    if (NORM) {
      rstd = row_rstd(s, a.cols, a.eps);
      if (!(s < __uint_as_float(kInfBits))) {  // as in rows_kernel
        float s2 = 0.0f;
        reduce_row<true>(s2, hm, red, buf);
        if (hm < kInfBits) {
          const float down = pow2(167 - (int)(hm >> 23));
          s2 = 0.0f;
          for (int c = threadIdx.x; c < a.cols; c += blockDim.x) {
            const float h = h_of(c) * down;
            s2 = fmaf(h, h, s2);
          }
          unsigned none = 0;
          reduce_row<true>(s2, none, red, buf);
          rstd = row_rstd(s2, a.cols, a.eps * down * down) * down;
        }
      }
    }
    const Quant z = a.q ? make_quant(m, rstd) : Quant{1.0f, 0.0f, 0.0f};
    for (int c = threadIdx.x; c < a.cols; c += blockDim.x) {
      const float h = h_of(c);
      if (NORM && a.sum) static_cast<T *>(a.sum)[row * a.ss + c] = from_f32<T>(h);
      if (NORM && a.y) {
        float v = h * rstd;
        if (gain) v *= to_f32(gain[c]);
        static_cast<T *>(a.y)[row * a.ys + c] = from_f32<T>(v);
      }
      if (a.q) a.q[row * a.qs + c] = quantise(t_of(h, c), z);
    }
    if (a.q && threadIdx.x == 0) a.scale[row] = z.scale;
  }
}

template <typename T, typename G, int VEC, int NV, bool NORM>
void launch_nv(const NormArgs &a, int groups, cudaStream_t st) {
  constexpr int64_t kMaxGrid = 0x7fffffff;
  if (groups <= 32 * NV) {
    const int64_t blocks = (a.rows + 3) / 4;
    rows_kernel<T, G, VEC, NV, false, NORM>
        <<<(unsigned)(blocks < kMaxGrid ? blocks : kMaxGrid), 128, 0, st>>>(a);
  } else {
    const int threads = ((groups + NV - 1) / NV + 31) / 32 * 32;
    rows_kernel<T, G, VEC, NV, true, NORM>
        <<<(unsigned)(a.rows < kMaxGrid ? a.rows : kMaxGrid), threads, 0, st>>>(a);
  }
}

template <typename T, typename G, bool NORM>
void launch_typed(const NormArgs &a, cudaStream_t st) {
  constexpr int VEC = 16 / (int)sizeof(T);
  auto vec_rows = [&](const void *p, int64_t stride, int esize) {
    return !p || (aligned_to(p, VEC * esize) && (stride % VEC == 0 || a.rows <= 1));
  };
  const bool vec = vec_rows(a.x, a.xs, sizeof(T)) && vec_rows(a.residual, a.rs, sizeof(T)) &&
                   vec_rows(a.sum, a.ss, sizeof(T)) && vec_rows(a.y, a.ys, sizeof(T)) &&
                   vec_rows(a.q, a.qs, 1) && vec_rows(a.gain, 0, sizeof(G) < 4 ? 2 : 4);
  if (vec) {
    const int groups = (a.cols + VEC - 1) / VEC;
    if (groups <= 256) launch_nv<T, G, VEC, 1, NORM>(a, groups, st);
    else if (groups <= 512) launch_nv<T, G, VEC, 2, NORM>(a, groups, st);
    else if (groups <= 4096) launch_nv<T, G, VEC, 4, NORM>(a, groups, st);
  } else {
    if (a.cols <= 1024) launch_nv<T, G, 1, 4, NORM>(a, a.cols, st);
    else if (a.cols <= 16384) launch_nv<T, G, 1, 16, NORM>(a, a.cols, st);
  }
  if (vec ? (a.cols + VEC - 1) / VEC > 4096 : a.cols > 16384) {
    const int64_t grid = a.rows < 0x7fffffff ? a.rows : 0x7fffffff;
    long_rows_kernel<T, G, NORM><<<(unsigned)grid, 1024, 0, st>>>(a);
  }
}

// Row offsets of a tensor stay far inside 64 bits.
bool extent_ok(int64_t rows, int64_t stride, int64_t cols) {
  return ((double)rows * (double)stride + (double)cols) * 4.0 < 0x1p60;
}

// Views of a call's rows, for the overlap checks.
RowView view(const void *p, int64_t rows, int cols, int64_t stride, int esize) {
  return RowView{p, rows, stride * esize, (int64_t)cols * esize};
}

bv_status check_rows(const char *what, const void *x, int64_t xs, int64_t rows, int cols,
                     int dtype) {
  if (!dtype_ok(dtype)) return fail(BV_ERR_ARG, "%s: dtype %d", what, dtype);
  if (rows < 0 || cols < 1 || xs < 0 || !extent_ok(rows, xs, cols))
    return fail(BV_ERR_SHAPE, "%s: rows=%lld cols=%d stride=%lld", what, (long long)rows, cols,
                (long long)xs);
  if (rows > 0 && !x) return fail(BV_ERR_ARG, "%s: null input", what);
  if (!aligned_to(x, dtype_size(dtype))) return fail(BV_ERR_ARG, "%s: misaligned input", what);
  return BV_OK;
}

bv_status check_out(const char *what, const char *name, const RowView &o, int64_t cols_bytes,
                    int align) {
  if (!o.p) return BV_OK;
  if (o.rows > 1 && o.stride < cols_bytes)
    return fail(BV_ERR_SHAPE, "%s: the rows of %s overlap one another", what, name);
  if (!aligned_to(o.p, align)) return fail(BV_ERR_ARG, "%s: misaligned %s", what, name);
  return BV_OK;
}

}  // namespace

bv_status launch_rows(const NormArgs &a, int dtype, int gain_dtype, cudaStream_t st) {
  if (a.rows == 0) return BV_OK;
  const double n = (double)a.rows * a.cols;
  const int es = dtype_size(dtype);
  const double bytes = n * es * (1 + (a.residual ? 1 : 0) + (a.sum ? 1 : 0) + (a.y ? 1 : 0)) +
                       (a.q ? n + 4.0 * a.rows : 0.0);
  {
    LaunchTimer tm(st, a.norm ? "rms_norm" : "quantize_rows", (a.norm ? 6.0 : 3.0) * n, bytes);
    if (a.norm) {
      const bool f32g = gain_dtype == BV_F32;
      if (dtype == BV_F32) launch_typed<float, float, true>(a, st);
      else if (dtype == BV_BF16 && f32g) launch_typed<__nv_bfloat16, float, true>(a, st);
      else if (dtype == BV_BF16) launch_typed<__nv_bfloat16, __nv_bfloat16, true>(a, st);
      else if (f32g) launch_typed<__half, float, true>(a, st);
      else launch_typed<__half, __half, true>(a, st);
    } else {
      if (dtype == BV_F32) launch_typed<float, float, false>(a, st);
      else if (dtype == BV_BF16) launch_typed<__nv_bfloat16, __nv_bfloat16, false>(a, st);
      else launch_typed<__half, __half, false>(a, st);
    }
  }
  count_launch();
  return check_launch(a.norm ? "rms_norm" : "quantize_rows");
}

namespace {

bv_status norm_entry(const char *what, const void *x, int64_t xs, const void *residual, int64_t rs,
                     void *sum, int64_t ss, const void *gain, int gain_dtype, float eps,
                     int64_t rows, int cols, int dtype, void *y, int64_t ys, int8_t *q, int64_t qs,
                     float *scale, bool int8, void *stream) {
  clear_error();
  BV_TRY(check_rows(what, x, xs, rows, cols, dtype));
  const int es = dtype_size(dtype);
  if (rows > 0 && (int8 ? (!q || !scale) : !y)) return fail(BV_ERR_ARG, "%s: null output", what);
  if (!(eps > 0.0f) || !(eps < 1e30f)) return fail(BV_ERR_ARG, "%s: eps %g", what, (double)eps);
  if (gain && gain_dtype != BV_F32 && gain_dtype != dtype)
    return fail(BV_ERR_ARG, "%s: gain of type %d for rows of type %d", what, gain_dtype, dtype);
  if ((residual && (rs < 0 || !extent_ok(rows, rs, cols))) ||
      (sum && (ss < 0 || !extent_ok(rows, ss, cols))) ||
      (int8 ? qs < 0 || !extent_ok(rows, qs, cols) : ys < 0 || !extent_ok(rows, ys, cols)))
    return fail(BV_ERR_SHAPE, "%s: row stride", what);
  if (!aligned_to(residual, es) ||
      !aligned_to(gain, gain && gain_dtype == BV_F32 ? 4 : 2) || !aligned_to(scale, 4))
    return fail(BV_ERR_ARG, "%s: misaligned pointer", what);
  const RowView vx = view(x, rows, cols, xs, es), vr = view(residual, rows, cols, rs, es);
  const RowView vs = view(sum, rows, cols, ss, es);
  const RowView vo = int8 ? view(q, rows, cols, qs, 1) : view(y, rows, cols, ys, es);
  const RowView vg = RowView{gain, 1, 0, (int64_t)cols * (gain_dtype == BV_F32 ? 4 : 2)};
  const RowView vsc = RowView{int8 ? scale : nullptr, 1, 0, rows * 4};
  BV_TRY(check_out(what, "sum", vs, (int64_t)cols * es, es));
  BV_TRY(check_out(what, int8 ? "q" : "y", vo, (int64_t)cols * (int8 ? 1 : es), int8 ? 1 : es));
  // the sum may be written over x or the residual, each row in its place
  if ((rows_overlap(vs, vx) && !same_rows(vs, vx)) || (rows_overlap(vs, vr) && !same_rows(vs, vr)))
    return fail(BV_ERR_ARG, "%s: sum partially overlaps its operands", what);
  if (rows_overlap(vo, vx) || rows_overlap(vo, vr) || rows_overlap(vo, vs) ||
      rows_overlap(vo, vg) || rows_overlap(vs, vg) || rows_overlap(vsc, vx) ||
      rows_overlap(vsc, vr) || rows_overlap(vsc, vs) || rows_overlap(vsc, vg) ||
      rows_overlap(vsc, vo))
    return fail(BV_ERR_ARG, "%s: an output overlaps another tensor", what);
  BV_TRY(require_device());
  const NormArgs a{x,  residual, gain, sum, int8 ? nullptr : y, int8 ? q : nullptr, scale, xs, rs,
                   ss, ys,       qs,   rows, cols, eps, 1};
  return launch_rows(a, dtype, gain_dtype, as_stream(stream));
}

}  // namespace
}  // namespace bv

using namespace bv;

extern "C" {

bv_status bv_rms_norm(const void *x, int64_t x_stride, const void *residual,
                      int64_t residual_stride, void *sum, int64_t sum_stride, const void *gain,
                      int gain_dtype, float eps, int64_t rows, int cols, int dtype, void *y,
                      int64_t y_stride, void *stream) {
  return norm_entry("bv_rms_norm", x, x_stride, residual, residual_stride, sum, sum_stride, gain,
                    gain_dtype, eps, rows, cols, dtype, y, y_stride, nullptr, 0, nullptr, false,
                    stream);
}

bv_status bv_rms_norm_int8(const void *x, int64_t x_stride, const void *residual,
                           int64_t residual_stride, void *sum, int64_t sum_stride,
                           const void *gain, int gain_dtype, float eps, int64_t rows, int cols,
                           int dtype, int8_t *q, int64_t q_stride, float *scale, void *stream) {
  return norm_entry("bv_rms_norm_int8", x, x_stride, residual, residual_stride, sum, sum_stride,
                    gain, gain_dtype, eps, rows, cols, dtype, nullptr, 0, q, q_stride, scale, true,
                    stream);
}

bv_status bv_quantize_rows(const void *x, int64_t x_stride, int64_t rows, int cols, int dtype,
                           int8_t *q, int64_t q_stride, float *scale, void *stream) {
  const char *what = "bv_quantize_rows";
  clear_error();
  BV_TRY(check_rows(what, x, x_stride, rows, cols, dtype));
  if (q_stride < 0 || !extent_ok(rows, q_stride, cols))
    return fail(BV_ERR_SHAPE, "%s: row stride", what);
  if (rows > 0 && (!q || !scale)) return fail(BV_ERR_ARG, "%s: null output", what);
  if (!aligned_to(scale, 4)) return fail(BV_ERR_ARG, "%s: misaligned scale", what);
  const RowView vx = view(x, rows, cols, x_stride, dtype_size(dtype));
  const RowView vq = view(q, rows, cols, q_stride, 1);
  const RowView vsc = RowView{scale, 1, 0, rows * 4};
  BV_TRY(check_out(what, "q", vq, cols, 1));
  if (rows_overlap(vq, vx) || rows_overlap(vsc, vx) || rows_overlap(vsc, vq))
    return fail(BV_ERR_ARG, "%s: an output overlaps another tensor", what);
  BV_TRY(require_device());
  const NormArgs a{x, nullptr, nullptr, nullptr, nullptr, q,   scale, x_stride, 0,
                   0, 0,       q_stride, rows,    cols,    1.0f, 0};
  return launch_rows(a, dtype, dtype, as_stream(stream));
}

}  // extern "C"
