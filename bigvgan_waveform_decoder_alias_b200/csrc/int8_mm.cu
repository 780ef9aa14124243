// Matrix product of 8-bit integers with a scale for each token and channel:
//   y[m, n] = a_scale[m] w_scale[n] sum_k a[m, k] w[n, k] + bias[n] + residual[m, n]
// The sum is exact in 32-bit integers (|a w| <= 2^14 and K < 2^17), so it does
// not depend on how K is split; the scales, the bias and the residual join in
// 32-bit floats and the result is rounded once.
#include "token_types.cuh"

namespace bv {
namespace {

constexpr int TILE = 64, KC = 32;

// 64 x 64 outputs a block, 4 x 4 a thread, four products an instruction; the
// operands are read byte by byte, so rows may start anywhere.
template <typename T>
__global__ void __launch_bounds__(256) int8_tile_kernel(Int8Args p, int tiles_m) {
  __shared__ int as[KC / 4][TILE + 1], ws[KC / 4][TILE + 1];
  const int m0 = (int)(blockIdx.x % tiles_m) * TILE, n0 = (int)(blockIdx.x / tiles_m) * TILE;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  int acc[4][4] = {};
  for (int k0 = 0; k0 < p.K; k0 += KC) {
    for (int i = threadIdx.x; i < TILE * (KC / 4); i += 256) {
      const int k4 = i % (KC / 4), r = i / (KC / 4);
      unsigned va = 0, vw = 0;
      for (int b = 0; b < 4; ++b) {
        const int k = k0 + 4 * k4 + b;
        if (k < p.K) {
          if (m0 + r < p.M) va |= (unsigned)(uint8_t)p.a[(int64_t)(m0 + r) * p.as + k] << (8 * b);
          if (n0 + r < p.N) vw |= (unsigned)(uint8_t)p.w[(int64_t)(n0 + r) * p.ws + k] << (8 * b);
        }
      }
      as[k4][r] = (int)va;
      ws[k4][r] = (int)vw;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < KC / 4; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          acc[i][j] = __dp4a(as[k][ty + 16 * i], ws[k][tx + 16 * j], acc[i][j]);
    __syncthreads();
  }
  const T *res = static_cast<const T *>(p.residual);
  T *y = static_cast<T *>(p.y);
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 4; ++j) {
      const int m = m0 + ty + 16 * i, n = n0 + tx + 16 * j;
      if (m >= p.M || n >= p.N) continue;
      float v = (float)acc[i][j] * (p.a_scale[m] * p.w_scale[n]);
      if (p.bias) v += p.bias[n];
      const int64_t ri = p.channels_first ? n * p.rs + m : m * p.rs + n;
      const int64_t yi = p.channels_first ? n * p.ys + m : m * p.ys + n;
      if (res) v += to_f32(res[ri]);
      y[yi] = from_f32<T>(v);
    }
}

}  // namespace

bv_status launch_int8_matmul(const Int8Args &p, int dtype, cudaStream_t st) {
  if (p.M == 0 || p.N == 0) return BV_OK;
  const int64_t tm = (p.M + TILE - 1) / TILE, tn = (p.N + TILE - 1) / TILE;
  if (tm * tn > 0x7fffffff) return fail(BV_ERR_SHAPE, "bv_int8_matmul: grid");
  const double out = (double)p.M * p.N;
  {
    LaunchTimer t(st, "int8_matmul", 2.0 * out * p.K,
                  ((double)p.M + p.N) * p.K + out * dtype_size(dtype) * (p.residual ? 2 : 1));
    const unsigned grid = (unsigned)(tm * tn);
    if (dtype == BV_F32) int8_tile_kernel<float><<<grid, 256, 0, st>>>(p, (int)tm);
    else if (dtype == BV_BF16) int8_tile_kernel<__nv_bfloat16><<<grid, 256, 0, st>>>(p, (int)tm);
    else int8_tile_kernel<__half><<<grid, 256, 0, st>>>(p, (int)tm);
  }
  count_launch();
  return check_launch("int8_matmul");
}

}  // namespace bv

using namespace bv;

extern "C" {

bv_status bv_int8_matmul(const int8_t *a, int64_t a_stride, const float *a_scale, const int8_t *w,
                         int64_t w_stride, const float *w_scale, const float *bias, int M, int N,
                         int K, const void *residual, int64_t residual_stride, void *y,
                         int64_t y_stride, int dtype, int channels_first, void *stream) {
  const char *what = "bv_int8_matmul";
  clear_error();
  if (!dtype_ok(dtype)) return fail(BV_ERR_ARG, "%s: dtype %d", what, dtype);
  if (M < 0 || N < 1 || K < 1 || K > BV_INT8_MAX_DEPTH)
    return fail(BV_ERR_SHAPE, "%s: M=%d N=%d K=%d", what, M, N, K);
  const int64_t max_stride = (int64_t)1 << 28;  // rows (below 2^31) x stride x 4 bytes < 2^62
  if (a_stride < 0 || a_stride > max_stride || w_stride < 0 || w_stride > max_stride ||
      (residual && (residual_stride < 0 || residual_stride > (int64_t)1 << 31)) || y_stride < 0 ||
      y_stride > (int64_t)1 << 31)
    return fail(BV_ERR_SHAPE, "%s: row stride", what);
  if (M == 0) return BV_OK;
  if (!a || !a_scale || !w || !w_scale || !y) return fail(BV_ERR_ARG, "%s: null pointer", what);
  const int es = dtype_size(dtype);
  if (!aligned_to(a_scale, 4) || !aligned_to(w_scale, 4) || !aligned_to(bias, 4) ||
      !aligned_to(residual, es) || !aligned_to(y, es))
    return fail(BV_ERR_ARG, "%s: misaligned pointer", what);
  const int64_t yr = channels_first ? N : M, yc = channels_first ? M : N;
  if (yr > 1 && y_stride < yc) return fail(BV_ERR_SHAPE, "%s: the rows of y overlap", what);
  const RowView vy{y, yr, y_stride * es, yc * es};
  const RowView vr{residual, yr, residual_stride * es, yc * es};
  const RowView va{a, M, a_stride, K}, vw{w, N, w_stride, K};
  const RowView vas{a_scale, 1, 0, (int64_t)M * 4}, vws{w_scale, 1, 0, (int64_t)N * 4};
  const RowView vb{bias, 1, 0, (int64_t)N * 4};
  if (rows_overlap(vy, vr) && !same_rows(vy, vr))
    return fail(BV_ERR_ARG, "%s: residual partially overlaps y", what);
  if (rows_overlap(vy, va) || rows_overlap(vy, vw) || rows_overlap(vy, vas) ||
      rows_overlap(vy, vws) || rows_overlap(vy, vb))
    return fail(BV_ERR_ARG, "%s: y overlaps an operand", what);
  BV_TRY(require_device());
  const Int8Args p{a,  w,  a_scale, w_scale, bias, residual,       y, a_stride, w_stride,
                   residual_stride, y_stride, M, N, K, channels_first ? 1 : 0};
  return launch_int8_matmul(p, dtype, as_stream(stream));
}

}  // extern "C"
