// The token front end: the norm and the projection that end a generative
// model, giving the latents a decoder reads.  Two launches (one norm, one
// product; a product a side where the latents are laid out by side), the
// 8-bit rows between them in the caller's workspace.
#include "token_types.cuh"

namespace bv {
namespace {

int64_t padded(int cols) { return ((int64_t)cols + 15) / 16 * 16; }
size_t rows_bytes(int64_t tokens, int cols) {
  return ((size_t)tokens * padded(cols) + 255) / 256 * 256;
}

}  // namespace
}  // namespace bv

using namespace bv;

extern "C" {

size_t bv_token_front_end_workspace_size(int S, int T, int cols) {
  clear_error();
  if (S < 1 || T < 1 || cols < 1 || cols > BV_INT8_MAX_DEPTH || (int64_t)S * T > 0x7fffffff) {
    fail(BV_ERR_SHAPE, "bv_token_front_end: S=%d T=%d cols=%d", S, T, cols);
    return 0;
  }
  return rows_bytes((int64_t)S * T, cols) + (size_t)S * T * sizeof(float);
}

bv_status bv_token_front_end(const void *x, int64_t x_stride, const void *residual,
                             int64_t residual_stride, const void *gain, int gain_dtype, float eps,
                             int S, int T, int cols, int dtype, const int8_t *w, int64_t w_stride,
                             const float *w_scale, const float *bias, int Cout, int by_side,
                             float *z, void *workspace, size_t ws_bytes, void *stream) {
  const char *what = "bv_token_front_end";
  const size_t need = bv_token_front_end_workspace_size(S, T, cols);
  if (need == 0) return BV_ERR_SHAPE;
  if (Cout < 1) return fail(BV_ERR_SHAPE, "%s: Cout=%d", what, Cout);
  if (!x || !w || !w_scale || !z) return fail(BV_ERR_ARG, "%s: null pointer", what);
  if (!workspace || ws_bytes < need)
    return fail(BV_ERR_WORKSPACE, "%s: %zu bytes, need %zu", what, ws_bytes, need);
  if (!aligned_to(workspace, 256)) return fail(BV_ERR_ARG, "%s: workspace alignment", what);
  const int64_t max_stride = (int64_t)1 << 28;
  if (x_stride < 0 || x_stride > max_stride || (residual && (residual_stride < 0 ||
      residual_stride > max_stride)) || w_stride < 0 || w_stride > max_stride)
    return fail(BV_ERR_SHAPE, "%s: row stride", what);
  const int64_t tokens = (int64_t)S * T;
  // (what only the product would refuse is refused before the norm is launched)
  if (Cout > kMaxMmRows || (by_side ? T : tokens) > kMaxMmRows || !extent_ok(tokens, Cout, 0))
    return fail(BV_ERR_SHAPE, "%s: S=%d T=%d Cout=%d", what, S, T, Cout);
  if (!aligned_to(w_scale, 4) || !aligned_to(bias, 4) || !aligned_to(z, 4))
    return fail(BV_ERR_ARG, "%s: misaligned pointer", what);
  const int64_t xe = x_stride * (tokens - 1) + cols, re = residual_stride * (tokens - 1) + cols;
  const int es = dtype_ok(dtype) ? dtype_size(dtype) : 1;
  const RowView vws{workspace, 1, 0, (int64_t)need};
  const RowView vz{z, 1, 0, tokens * Cout * 4};
  const RowView others[] = {{x, 1, 0, xe * es},
                            {residual, 1, 0, re * es},
                            {gain, 1, 0, (int64_t)cols * (gain_dtype == BV_F32 ? 4 : 2)},
                            {w, 1, 0, w_stride * (Cout - 1) + cols},
                            {w_scale, 1, 0, (int64_t)Cout * 4},
                            {bias, 1, 0, (int64_t)Cout * 4},
                            vz};
  for (const RowView &o : others) {
    if (rows_overlap(vws, o)) return fail(BV_ERR_ARG, "%s: workspace overlaps a tensor", what);
    if (&o != &others[6] && rows_overlap(vz, o)) return fail(BV_ERR_ARG, "%s: z overlaps a tensor", what);
  }
  int8_t *q = static_cast<int8_t *>(workspace);
  float *scale = reinterpret_cast<float *>(q + rows_bytes(tokens, cols));
  const int64_t qs = padded(cols);
  BV_TRY(bv_rms_norm_int8(x, x_stride, residual, residual_stride, nullptr, 0, gain, gain_dtype, eps,
                          tokens, cols, dtype, q, qs, scale, stream));
  if (!by_side)
    return bv_int8_matmul(q, qs, scale, w, w_stride, w_scale, bias, (int)tokens, Cout, cols,
                          nullptr, 0, z, tokens, BV_F32, 1, stream);
  for (int s = 0; s < S; ++s)
    BV_TRY(bv_int8_matmul(q + (int64_t)s * T * qs, qs, scale + (int64_t)s * T, w, w_stride, w_scale,
                          bias, T, Cout, cols, nullptr, 0, z + (int64_t)s * Cout * T, T, BV_F32, 1,
                          stream));
  return BV_OK;
}

}  // extern "C"
