// Element types, row views and argument checks shared by the token operators.
#pragma once

#include <cuda_bf16.h>

#include <utility>

#include "common.cuh"

namespace bv {

inline bool dtype_ok(int dt) { return dt == BV_F32 || dt == BV_BF16 || dt == BV_F16; }
inline int dtype_size(int dt) { return dt == BV_F32 ? 4 : 2; }

// Row offsets of a tensor stay far inside 64 bits.
inline bool extent_ok(int64_t rows, int64_t stride, int64_t cols) {
  return ((double)rows * (double)stride + (double)cols) * 4.0 < 0x1p60;
}

// `rows` rows of `row_bytes` bytes, `stride` bytes apart.
struct RowView {
  const void *p;
  int64_t rows, stride, row_bytes;
};

// Do two views share a byte?  Views of one stride are compared within the
// stride (column slices of one matrix are disjoint); others by their spans.
inline bool rows_overlap(const RowView &a, const RowView &b) {
  if (!a.p || !b.p || a.rows < 1 || b.rows < 1) return false;
  const int64_t pa = (int64_t)reinterpret_cast<uintptr_t>(a.p);
  const int64_t pb = (int64_t)reinterpret_cast<uintptr_t>(b.p);
  const int64_t ea = pa + (a.rows - 1) * a.stride + a.row_bytes;
  const int64_t eb = pb + (b.rows - 1) * b.stride + b.row_bytes;
  if (ea <= pb || eb <= pa) return false;
  if (a.stride == b.stride && a.rows > 1 && b.rows > 1 && a.row_bytes <= a.stride &&
      b.row_bytes <= b.stride) {
    const int64_t d = ((pb - pa) % a.stride + a.stride) % a.stride;  // b's rows start d into a's
    return !(d >= a.row_bytes && d + b.row_bytes <= a.stride);
  }
  return true;
}
inline bool same_rows(const RowView &a, const RowView &b) {
  return a.p == b.p && (a.stride == b.stride || a.rows <= 1);
}

inline bool aligned_to(const void *p, int bytes) {
  return (reinterpret_cast<uintptr_t>(p) & (uintptr_t)(bytes - 1)) == 0;
}

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) {
  return v;
}
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) {
  return __float2half_rn(v);
}

// Two 32-bit floats an instruction.  (A packed sum of a packed product is
// contracted to one fma; where two roundings are meant the sum is scalar.)
__device__ __forceinline__ uint64_t bits(float2 v) {
  return (uint64_t)__float_as_uint(v.x) | ((uint64_t)__float_as_uint(v.y) << 32);
}
__device__ __forceinline__ float2 pair(uint64_t b) {
  return make_float2(__uint_as_float((unsigned)b), __uint_as_float((unsigned)(b >> 32)));
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;\n" : "=l"(r) : "l"(bits(a)), "l"(bits(b)));
  return pair(r);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;\n" : "=l"(r) : "l"(bits(a)), "l"(bits(b)));
  return pair(r);
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;\n" : "=l"(r) : "l"(bits(a)), "l"(bits(b)), "l"(bits(c)));
  return pair(r);
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// The 16 bytes from byte `off` (0 to 15) on of a's and b's 32.
__device__ __forceinline__ uint4 bytes_from(const uint4 &a, const uint4 &b, int off) {
  unsigned w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  if (off & 8) {
#pragma unroll
    for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
  }
  if (off & 4) {
#pragma unroll
    for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
  }
  const int s = 8 * (off & 3);
  return make_uint4(__funnelshift_r(w[0], w[1], s), __funnelshift_r(w[1], w[2], s),
                    __funnelshift_r(w[2], w[3], s), __funnelshift_r(w[3], w[4], s));
}

// The token operators follow one another in short launches, so each may be
// scheduled before the kernel ahead of it has ended (launch_next): its blocks
// set up and then wait (after_previous) until that kernel has completed and its
// writes are visible.  Nothing in memory is touched before, and what is read
// after is read by plain loads or copies: the read-only path (__ldg) is for data
// that nobody writes while the kernel runs, and the kernel ahead may still write
// these operands when this one has begun.  A kernel lets the
// next one in (admit_next) when all its blocks hold what they need of an SM,
// TMEM too: the next one's blocks, which wait for it, can then take nothing that
// it still asks for.  (Launches back to back: the norm of one row of 4096 bf16
// values 2.5 -> 2.05 us, a product of 24 x 2048 x 8192 11.1 -> 9.3 us.  The
// figures beside the rules that choose kernels and tiles were taken before,
// on both sides alike.)
__device__ __forceinline__ void admit_next() {
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
}
__device__ __forceinline__ void after_previous() {
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
}
template <typename... P, typename... A>
cudaError_t launch_next(void (*kernel)(P...), int64_t grid, int threads, size_t smem, int cluster,
                        cudaStream_t st, A &&...args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cluster > 1) {
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim = {(unsigned)cluster, 1, 1};
    cfg.numAttrs = 2;
  }
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<A>(args)...);
}

// ---- launchers (arguments checked by the ABI entries) ------------------------

struct NormArgs {
  const void *x, *residual, *gain;  // residual, gain may be null
  void *sum, *y;                    // may be null
  int8_t *q;                        // may be null
  float *scale;
  int64_t xs, rs, ss, ys, qs;  // strides in elements
  int64_t rows;
  int cols;
  float eps;
  int norm;  // 0: rows are quantised as they are (no norm, residual or gain)
};
bv_status launch_rows(const NormArgs &a, int dtype, int gain_dtype, cudaStream_t st);

struct Int8Args {
  const int8_t *a, *w;
  const float *a_scale, *w_scale, *bias;  // bias may be null
  const void *residual;                   // may be null; may be y
  void *y;
  int64_t as, ws, rs, ys;  // strides: bytes, bytes, elements, elements
  int M, N, K;
  int channels_first;
};
constexpr int kMaxMmRows = 0x7fffff00;  // M and N: tile indexes stay inside 32 bits
bv_status launch_int8_matmul(const Int8Args &a, int dtype, cudaStream_t st);

}  // namespace bv
