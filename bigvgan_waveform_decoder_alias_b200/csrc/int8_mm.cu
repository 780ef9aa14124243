// Matrix product of 8-bit integers with a scale for each token and channel:
//   y[m, n] = a_scale[m] w_scale[n] sum_k a[m, k] w[n, k] + bias[n] + residual[m, n]
// The sum is exact in 32-bit integers (|a w| <= 2^14 and K < 2^17), so it does
// not depend on how K is split; the scales, the bias and the residual join in
// 32-bit floats and the result is rounded once.
//
// Three kernels see the product as rows x columns, the rows being the
// dimension that y keeps consecutive: channels, or tokens where y is channels
// first.
//   int8_dot_kernel   one to four columns, on the CUDA cores;
//   int8_tile_kernel  few tiles: tcgen05.mma kind::i8, K shared by a cluster;
//   int8_pair_kernel  many tiles: the same on persistent CTA pairs.
// On the tensor cores rows are the M side, so a TMEM lane is one row and a warp
// writes 32 consecutive outputs of a column.  Operand tiles are K-major, 128
// bytes (128 values) a row, 128-byte swizzle.
#include <algorithm>

#include "tc_ptx.cuh"
#include "token_types.cuh"

namespace bv {
namespace {

constexpr int BR = 128;       // rows of a CTA's tile
constexpr int BK = 128;       // values of K in a stage: one swizzled row
constexpr int MAX_SPLIT = 8;  // CTAs of a cluster that share a tile's K

// The product as rows x columns; element (row, col) of y at col ys + row.
struct Mm {
  const int8_t *r, *c;  // [rows, K], [cols, K]
  int64_t rstride, cstride;
  int rows, cols, K;
  const float *r_scale, *c_scale;
  const float *r_bias, *c_bias;  // one of them, or none
  const void *residual;          // may be y
  void *y;
  int64_t rs, ys;
  bool pairs;  // 16-bit outputs: y takes two rows in one aligned store
};

// Instruction descriptor of kind::i8: D s32, A and B s8, both K-major.
__host__ __device__ constexpr uint32_t i8_idesc(int m, int n) {
  return (2u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(n >> 3) << 17) |
         ((uint32_t)(m >> 4) << 24);
}
template <int CTAS>
__device__ __forceinline__ void mma_i8(unsigned tmem_d, uint64_t a, uint64_t b, uint32_t idesc,
                                       unsigned acc) {
  if constexpr (CTAS == 1)
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n}\n" ::"r"(tmem_d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
  else
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p;\n}\n" ::"r"(tmem_d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}
__device__ __forceinline__ void tma_load_2d(unsigned dst, const CUtensorMap *map, int c0, int c1,
                                            unsigned bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3}], [%4];\n" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(bar)
      : "memory");
}
// 16 accumulator columns of this thread's lane.
__device__ __forceinline__ void tmem_ld16(unsigned addr, int *v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,"
      "%12,%13,%14,%15}, [%16];\n"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
        "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]),
        "=r"(v[14]), "=r"(v[15])
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_wait_ld() {
  asm volatile("tcgen05.wait::ld.sync.aligned;\n" ::: "memory");
}

__device__ __forceinline__ unsigned bits16(__nv_bfloat16 v) { return __bfloat16_as_ushort(v); }
__device__ __forceinline__ unsigned bits16(__half v) { return __half_as_ushort(v); }
[[maybe_unused]] __device__ __forceinline__ unsigned bits16(float) { return 0; }

// The residual of a warp's 32 rows (row0 + lane) x N columns from col0 on.
template <typename T, int N>
__device__ __forceinline__ void load_residual(const Mm &p, int row0, int lane, int col0, T (&r)[N]) {
  if (!p.residual || row0 + lane >= p.rows) return;
  const T *res = static_cast<const T *>(p.residual) + (int64_t)col0 * p.rs + row0 + lane;
  if (col0 + N <= p.cols) {
#pragma unroll
    for (int e = 0; e < N; ++e) r[e] = res[e * p.rs];
  } else {
#pragma unroll
    for (int e = 0; e < N; ++e)
      if (col0 + e < p.cols) r[e] = res[e * p.rs];
  }
}

// Those columns of the accumulator go out: `rscale`, `rbias` are this lane's
// row's, cs and cb (shared memory, 8-byte aligned) the columns' scales and biases,
// cb zeros where the bias belongs to the rows.  The residual (`r`) was loaded
// before; it may be y: an element is read by the lane that writes it or, of the
// 16-bit pairs below, by its neighbour, whose half of the word reaches the writer
// through a shuffle after it was read.
// A 16-bit column is half a word a lane, so lanes swap halves in pairs: the
// even one writes two rows of the even column, the odd one two rows of the odd
// column.
// WHOLE: 32 rows and N columns in range (and, of 16-bit outputs, `pairs`); this
// form has no branch, so that the columns' steps overlap (with branches between
// them a warp took some 250 cycles a pair, and the epilogue of 4800 x 4096 x
// 1024 four times the products' time).
template <typename T, int N, bool WHOLE, bool RESIDUAL>
__device__ __forceinline__ void write_columns(const Mm &p, const int (&acc)[N], int row, int lane,
                                              int col0, int nc, float rscale, float rbias,
                                              const float *cs, const float *cb, const T (&r)[N]) {
  constexpr bool PAIRS = WHOLE && sizeof(T) == 2;
  const int odd = PAIRS ? lane & 1 : 0;
  const bool in = row < p.rows;
  T *y = static_cast<T *>(p.y) + (int64_t)(col0 + odd) * p.ys + (row - odd);
#pragma unroll
  for (int e = 0; e < N; e += 2) {
    const float2 s = mul2(*reinterpret_cast<const float2 *>(cs + e), both(rscale));
    const float2 b = add2(*reinterpret_cast<const float2 *>(cb + e), both(rbias));
    float2 f = fma2(make_float2((float)acc[e], (float)acc[e + 1]), s, b);
    if constexpr (RESIDUAL) f = add2(f, make_float2(to_f32(r[e]), to_f32(r[e + 1])));
    if constexpr (PAIRS) {
      const unsigned v0 = bits16(from_f32<T>(f.x)), v1 = bits16(from_f32<T>(f.y));
      const unsigned got = __shfl_xor_sync(0xffffffffu, odd ? v0 : v1, 1);
      *reinterpret_cast<unsigned *>(y + e * p.ys) = odd ? __byte_perm(got, v1, 0x5410)
                                                        : __byte_perm(v0, got, 0x5410);
    } else {
      if (WHOLE || (in && e < nc)) y[e * p.ys] = from_f32<T>(f.x);
      if (WHOLE || (in && e + 1 < nc)) y[(e + 1) * p.ys] = from_f32<T>(f.y);
    }
  }
}
template <typename T, int N>
__device__ __forceinline__ void store_columns(const Mm &p, const int (&acc)[N], int row0, int lane,
                                              int col0, float rscale, float rbias, const float *cs,
                                              const float *cb, const T (&r)[N]) {
  static_assert(N % 2 == 0, "columns go out in pairs");
  const int nc = min(N, p.cols - col0);  // warp-uniform
  if (row0 >= p.rows || nc <= 0) return;
  const bool whole = nc == N && row0 + 32 <= p.rows && (sizeof(T) == 4 || p.pairs);
  if (p.residual) {
    if (whole) write_columns<T, N, true, true>(p, acc, row0 + lane, lane, col0, nc, rscale, rbias, cs, cb, r);
    else write_columns<T, N, false, true>(p, acc, row0 + lane, lane, col0, nc, rscale, rbias, cs, cb, r);
  } else {
    if (whole) write_columns<T, N, true, false>(p, acc, row0 + lane, lane, col0, nc, rscale, rbias, cs, cb, r);
    else write_columns<T, N, false, false>(p, acc, row0 + lane, lane, col0, nc, rscale, rbias, cs, cb, r);
  }
}

__device__ __forceinline__ void prefetch_map(const CUtensorMap *map) {
  asm volatile("prefetch.tensormap [%0];\n" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}

__host__ __device__ constexpr int tmem_cols(int n) {
  return n <= 32 ? 32 : n <= 64 ? 64 : n <= 128 ? 128 : n <= 256 ? 256 : 512;
}

// 16 bytes of K from byte k on of a row that starts anywhere, zero past K: the
// one or two aligned 16-byte words that hold them are read (fetch), then
// shifted into place (bytes).  Near the ends of the operand [lo, hi), where a
// word would reach outside, single bytes are read.
struct Piece {
  uint4 a, b;
  int off, n;  // where the bytes begin in a; how many are inside K

  __device__ __forceinline__ void fetch(const int8_t *row, int k, int K, const int8_t *lo,
                                        const int8_t *hi) {
    a = b = make_uint4(0, 0, 0, 0);
    off = 0;
    n = min(16, K - k);
    if (n <= 0) return;
    const int8_t *p = row + k;
    const int at = (int)(reinterpret_cast<uintptr_t>(p) & 15);
    const int8_t *w = p - at;
    const bool two = at + n > 16;
    if (w >= lo && w + (two ? 32 : 16) <= hi) {
      off = at;
      a = *reinterpret_cast<const uint4 *>(w);
      if (two) b = reinterpret_cast<const uint4 *>(w)[1];
    } else {
      unsigned v[4] = {0, 0, 0, 0};
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (i < n) v[i / 4] |= (unsigned)(uint8_t)p[i] << (8 * (i % 4));
      a = make_uint4(v[0], v[1], v[2], v[3]);
    }
  }
  __device__ __forceinline__ uint4 bytes() const {
    const uint4 w = bytes_from(a, b, off);
    unsigned v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int left = n - 4 * i;  // bytes of this word inside K
      if (left < 4) v[i] = left <= 0 ? 0u : v[i] & (0xffffffffu >> (32 - 8 * left));
    }
    return make_uint4(v[0], v[1], v[2], v[3]);
  }
};

// ------------------------------------------------------------- few columns
//
// One to four columns (single tokens): bound by the rows' bytes, each read
// once, so the dot products stay on the CUDA cores (four products an
// instruction) and nothing is staged.  A block takes R rows and all of K: a
// thread reads 16 bytes of each row and column at a time, 128 threads apart.
// One token x 8192 x 8192: 14.3 us = 4.7 TB/s; x 4096 x 4096 4.8 us = 3.5 TB/s,
// where the first bytes' latency counts.

constexpr int DOT_THREADS = 128;

template <typename T, int R, int C, bool ALIGNED>
__global__ void __launch_bounds__(DOT_THREADS) int8_dot_kernel(const Mm p) {
  __shared__ int part[DOT_THREADS / 32][R * C];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row0 = (int)blockIdx.x * R;
  const int8_t *rhi = p.r + (int64_t)(p.rows - 1) * p.rstride + p.K;
  const int8_t *chi = p.c + (int64_t)(p.cols - 1) * p.cstride + p.K;
  int acc[R][C] = {};
  admit_next();
  after_previous();
  for (int k = 16 * threadIdx.x; k < p.K; k += 16 * DOT_THREADS) {
    uint4 r[R], c[C];
    if (ALIGNED && k + 16 <= p.K) {
#pragma unroll
      for (int i = 0; i < R; ++i)
        r[i] = *reinterpret_cast<const uint4 *>(
            p.r + (int64_t)min(row0 + i, p.rows - 1) * p.rstride + k);
#pragma unroll
      for (int j = 0; j < C; ++j)
        c[j] = *reinterpret_cast<const uint4 *>(
            p.c + (int64_t)min(j, p.cols - 1) * p.cstride + k);
    } else {
      Piece pr[R], pc[C];
#pragma unroll
      for (int i = 0; i < R; ++i)
        pr[i].fetch(p.r + (int64_t)min(row0 + i, p.rows - 1) * p.rstride, k, p.K, p.r, rhi);
#pragma unroll
      for (int j = 0; j < C; ++j)
        pc[j].fetch(p.c + (int64_t)min(j, p.cols - 1) * p.cstride, k, p.K, p.c, chi);
#pragma unroll
      for (int i = 0; i < R; ++i) r[i] = pr[i].bytes();
#pragma unroll
      for (int j = 0; j < C; ++j) c[j] = pc[j].bytes();
    }
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int j = 0; j < C; ++j) {
        int s = acc[i][j];
        s = __dp4a((int)r[i].x, (int)c[j].x, s);
        s = __dp4a((int)r[i].y, (int)c[j].y, s);
        s = __dp4a((int)r[i].z, (int)c[j].z, s);
        acc[i][j] = __dp4a((int)r[i].w, (int)c[j].w, s);
      }
  }
#pragma unroll
  for (int i = 0; i < R; ++i)
#pragma unroll
    for (int j = 0; j < C; ++j) {
      const int s = __reduce_add_sync(0xffffffffu, acc[i][j]);
      if (lane == 0) part[warp][i * C + j] = s;
    }
  // what the epilogue reads, on its way to the barrier
  const int i = threadIdx.x / C, j = threadIdx.x % C, row = row0 + i;
  const bool mine = threadIdx.x < R * C && row < p.rows && j < p.cols;
  float s = 0.0f, b = 0.0f, res = 0.0f;
  if (mine) {
    s = __fmul_rn(p.c_scale[j], p.r_scale[row]);
    b = p.r_bias ? p.r_bias[row] : p.c_bias ? p.c_bias[j] : 0.0f;
    if (p.residual) res = to_f32(static_cast<const T *>(p.residual)[j * p.rs + row]);
  }
  __syncthreads();
  if (mine) {
    int sum = 0;
#pragma unroll
    for (int w = 0; w < DOT_THREADS / 32; ++w) sum += part[w][i * C + j];
    float f = fmaf((float)sum, s, b);
    if (p.residual) f += res;
    static_cast<T *>(p.y)[j * p.ys + row] = from_f32<T>(f);
  }
}

// ------------------------------------------------------------- few tiles
//
// One CTA a tile of 128 rows x NT columns, or a cluster of up to eight CTAs
// that take a share of K each: with few tokens the weight's bytes bound the
// product, and only a split over K gives every SM some of them.  The shares
// are joined through distributed shared memory: each CTA leaves its partial
// sums in its own, then sums and writes NT / split of the columns.  Integers, so
// the join's order does not show.  24 x 2048 x 8192: 9.3 us, 64 x 4096 x 4096 10.4 us =
// 1.6 TB/s: set-up, the first bytes' latency and the join take most of it.  (Adding to the owner's shared memory from
// afar instead took longer: 16 x 8192 x 2048 11.2 us, 10.0 us so.)
//
// Thread 0 loads the stages by TMA.  Where an operand's rows do not start on 16
// bytes (COPY_R, COPY_C) eight more warps copy that operand instead: aligned
// words, shifted into place.

constexpr int TILE_MAX_STAGES = 12;

template <int NT>
constexpr int tile_stage_bytes() {
  return (BR + NT) * BK;
}

constexpr int COPY_WARPS = 8;

template <typename T, int NT, bool COPY_R, bool COPY_C>
__global__ void __launch_bounds__(COPY_R || COPY_C ? 128 + 32 * COPY_WARPS : 128)
int8_tile_kernel(const __grid_constant__ CUtensorMap map_r, const __grid_constant__ CUtensorMap map_c,
                 const Mm p, int tiles_r, int split, int stages, int *status,
                 long long wait_limit) {
  constexpr int STAGE = tile_stage_bytes<NT>();
  constexpr bool COPY = COPY_R || COPY_C, TMA = !COPY_R || !COPY_C;
  constexpr unsigned TMEM = tmem_cols(NT);
  extern __shared__ unsigned char smem_raw[];
  unsigned char *smem = reinterpret_cast<unsigned char *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  __shared__ uint64_t bars[3 * TILE_MAX_STAGES + 1];
  __shared__ Ctl ctl;
  __shared__ __align__(16) float cs[NT], cb[NT];  // the tile's columns' scales and biases
  const unsigned bar_full = smem_u32(&bars[0]);
  const unsigned bar_empty = smem_u32(&bars[TILE_MAX_STAGES]);
  const unsigned bar_copied = smem_u32(&bars[2 * TILE_MAX_STAGES]);
  const unsigned bar_done = smem_u32(&bars[3 * TILE_MAX_STAGES]);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)(blockIdx.x % (unsigned)split), tile = (int)(blockIdx.x / (unsigned)split);
  const int row0 = tile % tiles_r * BR, col0 = tile / tiles_r * NT;
  const int chunks = (p.K + BK - 1) / BK;
  const int c0 = (int)((int64_t)chunks * rank / split);
  const int n = (int)((int64_t)chunks * (rank + 1) / split) - c0;
  const WaitCtx wc{&ctl, 0u, status, wait_limit};

  if (threadIdx.x == 0) {
    if (!COPY_R) prefetch_map(&map_r);
    if (!COPY_C) prefetch_map(&map_c);
    ctl.abort = 0;
    for (int s = 0; s < stages; ++s) {
      mbar_init(bar_full + 8 * s, 1);
      mbar_init(bar_copied + 8 * s, COPY_WARPS);
      mbar_init(bar_empty + 8 * s, 1);
    }
    mbar_init(bar_done, 1);
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(
                     smem_u32(&ctl.tmem)),
                 "n"(TMEM)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n" ::: "memory");
  }
  asm volatile("tcgen05.fence::before_thread_sync;\n" ::: "memory");
  __syncthreads();
  asm volatile("tcgen05.fence::after_thread_sync;\n" ::: "memory");
  const unsigned tmem = ctl.tmem;
  admit_next();
  after_previous();
  // what the epilogue needs of the scales, on its way during the products
  const int row = row0 + 32 * warp + lane;  // of warps 0..3
  const bool in = warp < 4 && row < p.rows;
  const float rscale = in ? p.r_scale[row] : 0.0f;
  const float rbias = in && p.r_bias ? p.r_bias[row] : 0.0f;
  if (warp == 2 || warp == 3)
    for (int c = threadIdx.x - 64; c < NT; c += 64) {
      const bool have = col0 + c < p.cols;
      cs[c] = have ? p.c_scale[col0 + c] : 0.0f;
      cb[c] = have && p.c_bias ? p.c_bias[col0 + c] : 0.0f;
    }

  if (TMA && warp == 0 && lane == 0) {
    int c = 0;
    for (; c < n; ++c) {
      const int s = c % stages, u = c / stages;
      if (u > 0 && !mbar_wait(bar_empty + 8 * s, (u - 1) & 1, wc, 301)) break;
      const unsigned dst = smem_u32(smem + s * STAGE), fb = bar_full + 8 * s;
      mbar_arrive_tx(fb, (COPY_R ? 0 : BR * BK) + (COPY_C ? 0 : NT * BK));
      if (!COPY_R) tma_load_2d(dst, &map_r, (c0 + c) * BK, row0, fb);
      if (!COPY_C) tma_load_2d(dst + BR * BK, &map_c, (c0 + c) * BK, col0, fb);
    }
    // the last load into each slot has landed before the CTA can exit
    for (int d = c - stages; d < c; ++d)
      if (d >= 0) mbar_drain(bar_full + 8 * (d % stages), (d / stages) & 1);
  } else if (warp == 1 && lane == 0) {
    for (int c = 0; c < n; ++c) {
      const int s = c % stages;
      const unsigned phase = (unsigned)(c / stages) & 1u;
      if (TMA && !mbar_wait(bar_full + 8 * s, phase, wc, 302)) break;
      if (COPY && !mbar_wait(bar_copied + 8 * s, phase, wc, 305)) break;
      asm volatile("tcgen05.fence::after_thread_sync;\n" ::: "memory");
      const unsigned at = smem_u32(smem + s * STAGE);
      const uint64_t da = sw128_desc(at), db = sw128_desc(at + BR * BK);
#pragma unroll
      for (int k = 0; k < BK / 32; ++k)  // 32 values = 32 bytes an MMA
        mma_i8<1>(tmem, da + 2 * k, db + 2 * k, i8_idesc(BR, NT), c > 0 || k > 0 ? 1u : 0u);
      mma_commit(bar_empty + 8 * s);
    }
    mma_commit(bar_done);
    mbar_drain(bar_done, 0);  // after an abort too, no MMA outlives the tile
  } else if (COPY && warp >= 4) {
    // a warp's lanes take 4 rows x 8 pieces of 16 bytes at a time
    const int8_t *rhi = p.r + (int64_t)(p.rows - 1) * p.rstride + p.K;
    const int8_t *chi = p.c + (int64_t)(p.cols - 1) * p.cstride + p.K;
    const int piece = lane & 7, sub = (warp - 4) * 4 + (lane >> 3);
    constexpr int PASS = 4 * COPY_WARPS;  // rows a pass over the warps
    // rows [first, last) of a stage: BR rows, then NT columns
    constexpr int FIRST = COPY_R ? 0 : BR, LAST = COPY_C ? BR + NT : BR;
    constexpr int PASSES = COPY ? (LAST - FIRST + PASS - 1) / PASS : 1;
    // this lane's rows (past the last row of an operand: the last, whose
    // products no one stores)
    const int8_t *from[PASSES];
#pragma unroll
    for (int i = 0; i < PASSES; ++i) {
      const int r = FIRST + i * PASS + sub;
      from[i] = r < BR ? p.r + (int64_t)min(row0 + r, p.rows - 1) * p.rstride
                       : p.c + (int64_t)min(col0 + r - BR, p.cols - 1) * p.cstride;
    }
    for (int c = 0; c < n; ++c) {
      const int s = c % stages, u = c / stages;
      if (u > 0 && !warp_wait(bar_empty + 8 * s, (u - 1) & 1, wc, 303)) break;
      unsigned char *at = smem + s * STAGE;
      const int k0 = (c0 + c) * BK, k = k0 + 16 * piece;
      auto put = [&](int i, const uint4 &v) {
        const int r = FIRST + i * PASS + sub;
        if (LAST - FIRST == PASSES * PASS || r < LAST)
          *reinterpret_cast<uint4 *>(at + r * BK + ((piece ^ (r & 7)) << 4)) = v;
      };
      if (k0 >= 16 && k0 + BK + 16 <= p.K) {
        // every word that holds some of the chunk lies inside its row (also
        // taking chunks that reach into the neighbouring rows here, with their
        // bytes past K masked, made all of them dearer: 3633 x 3706 x 1228 62 -> 71 us)
#pragma unroll
        for (int g = 0; g < PASSES; g += 4) {
          uint4 lo[4], hi[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (g + i >= PASSES) continue;
            const int8_t *w = from[g + i] + k;
            w -= reinterpret_cast<uintptr_t>(w) & 15;
            lo[i] = *reinterpret_cast<const uint4 *>(w);
            hi[i] = reinterpret_cast<const uint4 *>(w)[1];
          }
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (g + i < PASSES)
              put(g + i, bytes_from(lo[i], hi[i],
                                    (int)(reinterpret_cast<uintptr_t>(from[g + i]) & 15)));
        }
      } else {
#pragma unroll
        for (int g = 0; g < PASSES; g += 4) {
          Piece v[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (g + i >= PASSES) continue;
            const bool is_r = FIRST + (g + i) * PASS + sub < BR;
            v[i].fetch(from[g + i], k, p.K, is_r ? p.r : p.c, is_r ? rhi : chi);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (g + i < PASSES) put(g + i, v[i].bytes());
        }
      }
      asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_copied + 8 * s);
    }
  }
  __syncwarp();

  if (warp < 4) {
    asm volatile("bar.sync 1, 128;\n" ::: "memory");  // cs, cb
    warp_wait(bar_done, 0, wc, 304);
    asm volatile("tcgen05.fence::after_thread_sync;\n" ::: "memory");
  }
  const unsigned lanes = (unsigned)(32 * warp) << 16;  // of warps 0..3
  if (split == 1) {
    if (warp < 4) {
#pragma unroll
      for (int c = 0; c < NT; c += 16) {
        int v[16];
        T r[16];
        tmem_ld16(tmem + lanes + c, v);
        load_residual(p, row0 + 32 * warp, lane, col0 + c, r);
        tmem_wait_ld();
        if (!ctl.abort)
          store_columns(p, v, row0 + 32 * warp, lane, col0 + c, rscale, rbias, cs + c, cb + c, r);
      }
    }
  } else {
    // partial sums [NT][128] over the stages, which no copy or MMA uses now
    int *part = reinterpret_cast<int *>(smem);
    if (warp < 4) {
#pragma unroll
      for (int c = 0; c < NT; c += 16) {
        int v[16];
        tmem_ld16(tmem + lanes + c, v);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 16; ++e) part[(c + e) * BR + 32 * warp + lane] = v[e];
      }
    }
    cluster_sync();
    if (warp < 4) {
      const unsigned mine = smem_u32(part + 32 * warp + lane);
      unsigned from[MAX_SPLIT];
#pragma unroll
      for (int s = 0; s < MAX_SPLIT; ++s) from[s] = s < split ? map_to_rank(mine, s) : 0u;
      // NT / split columns a CTA (NT >= 16, split a power of two up to 8)
      const int nc = NT / split;
      for (int c = rank * nc; c < (rank + 1) * nc; c += 2) {
        int v[2] = {0, 0}, got[2][MAX_SPLIT];
        T r[2];
        load_residual(p, row0 + 32 * warp, lane, col0 + c, r);
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int s = 0; s < MAX_SPLIT; ++s) {
            got[j][s] = 0;
            if (s < split)
              asm volatile("ld.shared::cluster.s32 %0, [%1];\n"
                           : "=r"(got[j][s])
                           : "r"(from[s] + (unsigned)((c + j) * BR * 4))
                           : "memory");
          }
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int s = 0; s < MAX_SPLIT; ++s) v[j] += got[j][s];
        if (!ctl.abort)
          store_columns(p, v, row0 + 32 * warp, lane, col0 + c, rscale, rbias, cs + c, cb + c, r);
      }
    }
    cluster_sync();  // every peer has read this CTA's sums
  }
  asm volatile("tcgen05.fence::before_thread_sync;\n" ::: "memory");
  __syncthreads();
  if (warp == 1) {
    asm volatile("tcgen05.fence::after_thread_sync;\n" ::: "memory");
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;\n" ::"r"(tmem), "n"(TMEM)
                 : "memory");
  }
}

// ------------------------------------------------------------- many tiles
//
// Persistent CTA pairs: a pair's tile is 256 rows x NT columns (cta_group::2:
// each CTA holds half of the rows and loads half of the columns), TMA fills a
// ring of stages, and two accumulators of NT columns in TMEM let sixteen warps a
// CTA write one tile out while the tensor cores work on the next.  Tiles are
// walked in bands of BAND row tiles, so that the pairs at work at one time share
// operand tiles in L2.  8192 x 8192 x 8192: 357 us = 3.08 POP/s, the tensor pipe 84 %
// busy at the 1.58 GHz that the power cap leaves it.  With a short K the operands'
// way from L2 and the epilogue bound it: 4800 x 4096 x 1024 24.9 us (with eight
// epilogue warps, before launches overlapped, 31.7 us, its products alone 21 us).

constexpr int PAIR_EPI_WARPS = 16;  // of a CTA: four for each 32 rows
constexpr int PAIR_THREADS = 128 + 32 * PAIR_EPI_WARPS;
constexpr int BAND = 8;

template <int NT>
constexpr int pair_stage_bytes() {
  return (BR + NT / 2) * BK;
}
template <int NT>
constexpr int pair_stages() {
  return 200 * 1024 / pair_stage_bytes<NT>();
}
// Arrive at the even CTA's barrier: this warp's TMEM reads are complete.
__device__ __forceinline__ void arrive_remote(unsigned cluster_addr) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];\n" ::"r"(cluster_addr)
               : "memory");
}

template <typename T, int NT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(PAIR_THREADS, 1)
int8_pair_kernel(const __grid_constant__ CUtensorMap map_r, const __grid_constant__ CUtensorMap map_c,
                 const Mm p, int tiles_r, int tiles_c, int *status, long long wait_limit) {
  constexpr int STAGE = pair_stage_bytes<NT>(), STAGES = pair_stages<NT>();
  constexpr unsigned TMEM = tmem_cols(2 * NT);
  extern __shared__ unsigned char smem_raw[];
  unsigned char *smem = reinterpret_cast<unsigned char *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  __shared__ uint64_t bars[2 * STAGES + 5];
  __shared__ Ctl ctl;
  __shared__ __align__(16) float cs[2][NT], cb[2][NT];  // columns' scales and biases, two tiles
  // the even CTA's full and free barriers serve the pair
  const unsigned bar_full = smem_u32(&bars[0]), bar_empty = smem_u32(&bars[STAGES]);
  const unsigned bar_acc = smem_u32(&bars[2 * STAGES]), bar_free = smem_u32(&bars[2 * STAGES + 2]);
  const unsigned bar_done = smem_u32(&bars[2 * STAGES + 4]);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const unsigned rank = cluster_rank();
  const bool leader = rank == 0;
  const int pairs = (int)(gridDim.x >> 1), pid = (int)(blockIdx.x >> 1);
  const int n_tiles = tiles_r * tiles_c;
  const int chunks = (p.K + BK - 1) / BK;
  const WaitCtx wc{&ctl, map_to_rank(smem_u32(&ctl.abort), rank ^ 1u), status, wait_limit};
  auto tile_at = [&](int tau, int &row0, int &col0) {
    const int band = tau / (BAND * tiles_c), in = tau - band * BAND * tiles_c;
    const int high = min(BAND, tiles_r - band * BAND);
    row0 = (band * BAND + in % high) * 2 * BR + (int)rank * BR;  // this CTA's rows
    col0 = in / high * NT;
  };

  if (threadIdx.x == 0) {
    prefetch_map(&map_r);
    prefetch_map(&map_c);
    ctl.abort = 0;
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(bar_full + 8 * s, 1);
      mbar_init(bar_empty + 8 * s, 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(bar_acc + 8 * s, 1);
      mbar_init(bar_free + 8 * s, 2 * PAIR_EPI_WARPS);
    }
    mbar_init(bar_done, 1);
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(
                     smem_u32(&ctl.tmem)),
                 "n"(TMEM)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;\n" ::: "memory");
  }
  asm volatile("tcgen05.fence::before_thread_sync;\n" ::: "memory");
  cluster_sync();  // both CTAs' barriers exist before anyone signals them
  asm volatile("tcgen05.fence::after_thread_sync;\n" ::: "memory");
  const unsigned tmem = ctl.tmem;
  admit_next();
  after_previous();

  if (warp == 0) {
    if (lane == 0) {
      int s = 0, issued = 0;
      unsigned pass = 0;  // over the ring
      bool ok = true;
      for (int tau = pid; tau < n_tiles && ok; tau += pairs) {
        int row0, col0;
        tile_at(tau, row0, col0);
        for (int c = 0; c < chunks; ++c) {
          if (pass > 0 && !mbar_wait(bar_empty + 8 * s, (pass - 1) & 1, wc, 311)) {
            ok = false;
            break;
          }
          const unsigned dst = smem_u32(smem + s * STAGE), fb = bar_full + 8 * s;
          if (leader) mbar_arrive_tx(fb, 2 * STAGE);
          tma_load_2d_pair(dst, &map_r, c * BK, row0, fb);
          tma_load_2d_pair(dst + BR * BK, &map_c, c * BK, col0 + (int)rank * (NT / 2), fb);
          ++issued;
          if (++s == STAGES) {
            s = 0;
            ++pass;
          }
        }
      }
      // the pair's last load into each slot has landed before the CTA can
      // exit (the even CTA's barriers count both CTAs' bytes, and the final
      // cluster barrier holds the odd CTA until then)
      if (leader)
        for (int d = issued - STAGES; d < issued; ++d)
          if (d >= 0) mbar_drain(bar_full + 8 * (d % STAGES), (d / STAGES) & 1);
    }
  } else if (warp == 1) {
    if (leader && lane == 0) {
      int s = 0, it = 0;  // ring slot, tiles begun
      unsigned phase = 0;
      bool ok = true;
      for (int tau = pid; tau < n_tiles && ok; tau += pairs, ++it) {
        const int buf = it & 1;
        if (it >= 2 && !mbar_wait(bar_free + 8 * buf, (it / 2 - 1) & 1, wc, 312)) break;
        asm volatile("tcgen05.fence::after_thread_sync;\n" ::: "memory");
        const unsigned acc = tmem + (unsigned)(buf * NT);
        for (int c = 0; c < chunks; ++c) {
          if (!mbar_wait(bar_full + 8 * s, phase, wc, 313)) {
            ok = false;
            break;
          }
          asm volatile("tcgen05.fence::after_thread_sync;\n" ::: "memory");
          const unsigned at = smem_u32(smem + s * STAGE);
          const uint64_t da = sw128_desc(at), db = sw128_desc(at + BR * BK);
#pragma unroll
          for (int k = 0; k < BK / 32; ++k)
            mma_i8<2>(acc, da + 2 * k, db + 2 * k, i8_idesc(2 * BR, NT), c > 0 || k > 0 ? 1u : 0u);
          mma_commit_pair(bar_empty + 8 * s);
          if (++s == STAGES) {
            s = 0;
            phase ^= 1u;
          }
        }
        if (ok) mma_commit_pair(bar_acc + 8 * buf);
      }
      // every MMA issued above has completed before TMEM can be freed
      mma_commit_pair(bar_done);
      mbar_drain(bar_done, 0);
    }
  } else if (warp >= 4) {
    const int q = warp & 3, part = (warp - 4) >> 2;  // TMEM lanes 32 q .., a quarter of the columns
    const int ct = threadIdx.x - 128;                // column whose scale this thread fetches
    const unsigned free_leader = map_to_rank(bar_free, 0);
    // a tile's scales and biases are fetched while the tile before it goes out
    float n_cs = 0.0f, n_cb = 0.0f, n_rs = 0.0f, n_rb = 0.0f;
    auto fetch = [&](int tau) {
      if (tau >= n_tiles) return;
      int row0, col0;
      tile_at(tau, row0, col0);
      const int row = row0 + 32 * q + lane, col = col0 + ct;
      n_rs = row < p.rows ? p.r_scale[row] : 0.0f;
      n_rb = row < p.rows && p.r_bias ? p.r_bias[row] : 0.0f;
      const bool have = ct < NT && col < p.cols;
      n_cs = have ? p.c_scale[col] : 0.0f;
      n_cb = have && p.c_bias ? p.c_bias[col] : 0.0f;
    };
    fetch(pid);
    int it = 0;
    for (int tau = pid; tau < n_tiles; tau += pairs, ++it) {
      int row0, col0;
      tile_at(tau, row0, col0);
      row0 += 32 * q;
      const int buf = it & 1;
      const float rscale = n_rs, rbias = n_rb;
      if (ct < NT) {
        cs[buf][ct] = n_cs;
        cb[buf][ct] = n_cb;
      }
      fetch(tau + pairs);
      const int c0 = part * (NT / 4);
      T r[16];
      load_residual(p, row0, lane, col0 + c0, r);
      // one warp waits for the sums; the barrier hands that on, and cs and cb
      if (warp == 4) warp_wait(bar_acc + 8 * buf, (it >> 1) & 1, wc, 314);
      asm volatile("bar.sync 1, %0;\n" ::"n"(32 * PAIR_EPI_WARPS) : "memory");
      asm volatile("tcgen05.fence::after_thread_sync;\n" ::: "memory");
      const unsigned acc = tmem + ((unsigned)(32 * q) << 16) + (unsigned)(buf * NT + c0);
#pragma unroll
      for (int c = 0; c < NT / 4; c += 16) {
        int v[16];
        tmem_ld16(acc + c, v);
        tmem_wait_ld();
        if (c + 16 == NT / 4) {
          asm volatile("tcgen05.fence::before_thread_sync;\n" ::: "memory");
          __syncwarp();
          if (lane == 0) arrive_remote(free_leader + 8 * buf);
        }
        if (!ctl.abort)  // after a wait that gave up nothing more is written
          store_columns(p, v, row0, lane, col0 + c0 + c, rscale, rbias, cs[buf] + c0 + c,
                        cb[buf] + c0 + c, r);
        if (c + 16 < NT / 4) load_residual(p, row0, lane, col0 + c0 + c + 16, r);
      }
    }
  }
  __syncwarp();
  asm volatile("tcgen05.fence::before_thread_sync;\n" ::: "memory");
  __syncthreads();
  // after an abort the odd CTA may have loads in flight that the even CTA's
  // barriers did not count; they land in a few microseconds
  if (!leader && threadIdx.x == 0 && ctl.abort)
    for (int i = 0; i < 64; ++i) __nanosleep(1000);
  cluster_sync();  // no MMA, remote arrive or copy of the pair is in flight
  if (warp == 1) {
    asm volatile("tcgen05.fence::after_thread_sync;\n" ::: "memory");
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;\n" ::"r"(tmem), "n"(TMEM)
                 : "memory");
  }
}

// ------------------------------------------------------------------ launching

bool tma_rows(const int8_t *p, int64_t stride, int rows, int K) {
  return aligned_to(p, 16) && (rows == 1 || (stride % 16 == 0 && stride >= K));
}

// [rows, K] bytes, box 128 bytes x box_rows, 128-byte swizzle; bytes past K
// and rows past the last read as zero.
bv_status encode_rows(CUtensorMap *map, const int8_t *p, int64_t stride, int rows, int K,
                      int box_rows) {
  if (!encode_fn()) return fail(BV_ERR_UNSUPPORTED, "bv_int8_matmul: no cuTensorMapEncodeTiled");
  const cuuint64_t dims[2] = {(cuuint64_t)K, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)(rows == 1 ? (K + 15) / 16 * 16 : stride)};
  const cuuint32_t box[2] = {(cuuint32_t)BK, (cuuint32_t)box_rows};
  const cuuint32_t estr[2] = {1, 1};
  const CUresult r =
      encode_fn()(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<int8_t *>(p), dims, strides,
                  box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(BV_ERR_CUDA, "bv_int8_matmul: tensor map (%d)", (int)r);
  return BV_OK;
}

template <typename T, int NT, bool COPY_R, bool COPY_C>
bv_status run_tile(const Mm &p, int split, cudaStream_t st) {
  const int64_t tiles_r = ((int64_t)p.rows + BR - 1) / BR, tiles_c = ((int64_t)p.cols + NT - 1) / NT;
  const int64_t tiles = tiles_r * tiles_c;
  const int chunks = (p.K + BK - 1) / BK;
  if (tiles * split > 0x7fffffff) return fail(BV_ERR_SHAPE, "bv_int8_matmul: grid");
  constexpr int STAGE = tile_stage_bytes<NT>();
  const int per = (chunks + split - 1) / split;
  // Two CTAs an SM; room for the partial sums of a split tile.  A CTA of a split
  // tile has two stages at least (per >= 2), so that the TMEM of such CTAs fits an
  // SM whose shared memory they fit: one that waited for TMEM would hold up its
  // cluster.
  int stages = std::min(std::min(per, TILE_MAX_STAGES), (112 * 1024 - 1024) / STAGE);
  const int least = split > 1 ? (NT * BR * 4 + STAGE - 1) / STAGE : 1;
  stages = std::max(stages, least);
  const size_t smem = (size_t)stages * STAGE + 1024;
  auto kernel = int8_tile_kernel<T, NT, COPY_R, COPY_C>;
  // (room beside the kernel's static shared memory too)
  BV_TRY(ensure_dynamic_smem((const void *)kernel, smem + 2048, "bv_int8_matmul smem"));
  CUtensorMap mr{}, mc{};
  if (!COPY_R) BV_TRY(encode_rows(&mr, p.r, p.rstride, p.rows, p.K, BR));
  if (!COPY_C) BV_TRY(encode_rows(&mc, p.c, p.cstride, p.cols, p.K, NT));
  int *status = device_status_ptr();
  if (!status) return fail(BV_ERR_CUDA, "bv_int8_matmul: status word");
  CUDA_TRY(launch_next(kernel, tiles * split, COPY_R || COPY_C ? 128 + 32 * COPY_WARPS : 128, smem,
                       split, st, mr, mc, p, (int)tiles_r, split, stages, status, wait_limit()));
  return BV_OK;
}

template <typename T, int NT>
bv_status run_pair(const Mm &p, cudaStream_t st) {
  const int64_t tiles_r = ((int64_t)p.rows + 2 * BR - 1) / (2 * BR);
  const int64_t tiles_c = ((int64_t)p.cols + NT - 1) / NT;
  // (tile indexes run past the last by at most a grid)
  if (tiles_r * tiles_c > 0x7fff0000 || tiles_c > 0x7fff0000 / BAND)
    return fail(BV_ERR_SHAPE, "bv_int8_matmul: grid");
  constexpr size_t smem = (size_t)pair_stages<NT>() * pair_stage_bytes<NT>() + 1024;
  auto kernel = int8_pair_kernel<T, NT>;
  BV_TRY(ensure_dynamic_smem((const void *)kernel, smem, "bv_int8_matmul smem"));
  CUtensorMap mr, mc;
  BV_TRY(encode_rows(&mr, p.r, p.rstride, p.rows, p.K, BR));
  BV_TRY(encode_rows(&mc, p.c, p.cstride, p.cols, p.K, NT / 2));
  int *status = device_status_ptr();
  if (!status) return fail(BV_ERR_CUDA, "bv_int8_matmul: status word");
  const int grid = 2 * (int)std::min<int64_t>(tiles_r * tiles_c, 74);
  CUDA_TRY(launch_next(kernel, grid, PAIR_THREADS, smem, 1, st, mr, mc, p, (int)tiles_r, (int)tiles_c,
                       status, wait_limit()));
  return BV_OK;
}

template <typename T, int R, int C, bool ALIGNED>
bv_status run_dot(const Mm &p, cudaStream_t st) {
  CUDA_TRY(launch_next(int8_dot_kernel<T, R, C, ALIGNED>, (p.rows + (int64_t)R - 1) / R, DOT_THREADS, 0,
                       1, st, p));
  return BV_OK;
}
template <typename T, int C, bool ALIGNED>
bv_status run_dot_rows(const Mm &p, cudaStream_t st) {
  // the most rows a block that leave three blocks an SM
  const int blocks = 3 * 148;
  if (p.rows >= 8 * blocks) return run_dot<T, 8, C, ALIGNED>(p, st);
  if (p.rows >= 4 * blocks) return run_dot<T, 4, C, ALIGNED>(p, st);
  if (p.rows >= 2 * blocks) return run_dot<T, 2, C, ALIGNED>(p, st);
  return run_dot<T, 1, C, ALIGNED>(p, st);
}
template <typename T, bool ALIGNED>
bv_status run_dots(const Mm &p, cudaStream_t st) {
  if (p.cols == 1) return run_dot_rows<T, 1, ALIGNED>(p, st);
  if (p.cols == 2) return run_dot_rows<T, 2, ALIGNED>(p, st);
  return run_dot_rows<T, 4, ALIGNED>(p, st);
}

int64_t tile_count(const Mm &p, int rows, int cols) {
  return (((int64_t)p.rows + rows - 1) / rows) * (((int64_t)p.cols + cols - 1) / cols);
}

// Columns of a pair's tile, or 0 where there are too few tiles to go round.  A
// wave of tiles takes about as long as its operands take from L2, which is as
// 256 + NT; e.g. 512 x 4096 x 4096: 17.7 us with 128 columns (one wave), 28.1 us with
// 64 (two), 19.2 us with 256 (one).  From 60 tiles of 64 columns on the pairs win
// (256 x 4096 x 4096 16.7 us, 16.9 us in few tiles; 128 x 4096 x 4096 16.4 and 13.5 us).
int pick_pair(const Mm &p) {
  if (tile_count(p, 2 * BR, 64) < 60) return 0;
  int best = 0;
  int64_t least = INT64_MAX;
  for (int nt : {256, 192, 128, 64}) {
    const int64_t cost = (tile_count(p, 2 * BR, nt) + 73) / 74 * (2 * BR + nt);
    if (cost < least) {
      least = cost;
      best = nt;
    }
  }
  return best;
}

// Few tiles: columns of a tile, and CTAs that share its K.  With a short K as
// many CTAs as there are to go round, none split (333 x 777 x 1120: 7.2 us in 16
// columns, 9.8 us in 64).  With a long one at most one tile to two SMs, each
// split as far as two CTAs an SM and two stages a CTA allow (64 x 4096 x 4096: 11.4 us
// in 32 columns over 4 CTAs, 15 us in 16 over 2).
void pick_tile(const Mm &p, int *nt, int *split) {
  const int chunks = (p.K + BK - 1) / BK;
  const bool whole = chunks < 16;
  *nt = 16;
  while (*nt < 128 && tile_count(p, BR, *nt) > (whole ? 296 : 74)) *nt *= 2;
  const int64_t tiles = tile_count(p, BR, *nt);
  *split = 1;
  while (!whole && *split < MAX_SPLIT && 2 * *split * tiles <= 296 && chunks >= 4 * *split) *split *= 2;
}

template <typename T, bool COPY_R, bool COPY_C>
bv_status run_tiles(const Mm &p, cudaStream_t st) {
  int nt, split;
  pick_tile(p, &nt, &split);
  if (nt == 16) return run_tile<T, 16, COPY_R, COPY_C>(p, split, st);
  if (nt == 32) return run_tile<T, 32, COPY_R, COPY_C>(p, split, st);
  if (nt == 64) return run_tile<T, 64, COPY_R, COPY_C>(p, split, st);
  return run_tile<T, 128, COPY_R, COPY_C>(p, split, st);
}

template <typename T>
bv_status run_typed(const Mm &p, cudaStream_t st) {
  const bool tma_r = tma_rows(p.r, p.rstride, p.rows, p.K);
  const bool tma_c = tma_rows(p.c, p.cstride, p.cols, p.K);
  // (four columns: 4096 x 4096 9.2 us by dot products, 9.4 us in tiles; eight 11.2 us)
  if (p.cols <= 4) return tma_r && tma_c ? run_dots<T, true>(p, st) : run_dots<T, false>(p, st);
  if (!tma_r && !tma_c) return run_tiles<T, true, true>(p, st);
  if (!tma_r) return run_tiles<T, true, false>(p, st);
  if (!tma_c) return run_tiles<T, false, true>(p, st);
  const int nt = pick_pair(p);
  if (nt == 256) return run_pair<T, 256>(p, st);
  if (nt == 192) return run_pair<T, 192>(p, st);
  if (nt == 128) return run_pair<T, 128>(p, st);
  if (nt == 64) return run_pair<T, 64>(p, st);
  return run_tiles<T, false, false>(p, st);
}

}  // namespace

bv_status launch_int8_matmul(const Int8Args &a, int dtype, cudaStream_t st) {
  if (a.M == 0 || a.N == 0) return BV_OK;
  Mm p{};
  const bool cf = a.channels_first != 0;
  p.r = cf ? a.a : a.w;
  p.c = cf ? a.w : a.a;
  p.rstride = cf ? a.as : a.ws;
  p.cstride = cf ? a.ws : a.as;
  p.rows = cf ? a.M : a.N;
  p.cols = cf ? a.N : a.M;
  p.K = a.K;
  p.r_scale = cf ? a.a_scale : a.w_scale;
  p.c_scale = cf ? a.w_scale : a.a_scale;
  p.r_bias = cf ? nullptr : a.bias;
  p.c_bias = cf ? a.bias : nullptr;
  p.residual = a.residual;
  p.y = a.y;
  p.rs = a.rs;
  p.ys = a.ys;
  p.pairs = aligned_to(a.y, 4) && (a.ys % 2 == 0 || p.cols == 1);
  const double out = (double)a.M * a.N;
  {
    LaunchTimer t(st, "int8_matmul", 2.0 * out * a.K,
                  ((double)a.M + a.N) * a.K + out * dtype_size(dtype) * (a.residual ? 2 : 1));
    if (dtype == BV_F32) BV_TRY(run_typed<float>(p, st));
    else if (dtype == BV_BF16) BV_TRY(run_typed<__nv_bfloat16>(p, st));
    else BV_TRY(run_typed<__half>(p, st));
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
  if (M < 0 || M > kMaxMmRows || N < 1 || N > kMaxMmRows || K < 1 || K > BV_INT8_MAX_DEPTH)
    return fail(BV_ERR_SHAPE, "%s: M=%d N=%d K=%d", what, M, N, K);
  const int64_t max_stride = (int64_t)1 << 28, max_out = (int64_t)1 << 31;
  const int64_t yr = channels_first ? N : M, yc = channels_first ? M : N;
  if (a_stride < 0 || a_stride > max_stride || w_stride < 0 || w_stride > max_stride ||
      (residual && (residual_stride < 0 || residual_stride > max_out ||
                    !extent_ok(yr, residual_stride, yc))) ||
      y_stride < 0 || y_stride > max_out || !extent_ok(yr, y_stride, yc))
    return fail(BV_ERR_SHAPE, "%s: row stride", what);
  if (M == 0) return BV_OK;
  if (!a || !a_scale || !w || !w_scale || !y) return fail(BV_ERR_ARG, "%s: null pointer", what);
  const int es = dtype_size(dtype);
  if (!aligned_to(a_scale, 4) || !aligned_to(w_scale, 4) || !aligned_to(bias, 4) ||
      !aligned_to(residual, es) || !aligned_to(y, es))
    return fail(BV_ERR_ARG, "%s: misaligned pointer", what);
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
