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
// past the registers of a block are read twice.  (Of 16-bit rows of 2048 groups
// and more, some of the block forms' values are spilled, up to 650 bytes a
// thread: a block of 1024 has 64 registers a thread.  40 rows of 16384 f16 values to
// 8 bits with f32 gains 10.6 us, of bf16, which spills 20 bytes, 4.8 us.)
#include <algorithm>

#include "tc_ptx.cuh"
#include "token_types.cuh"

namespace bv {
namespace {

constexpr unsigned kInfBits = 0x7f800000u;

// What a kernel writes: the norm in the rows' type, the norm in 8 bits, or the
// rows themselves in 8 bits.
enum Mode { kNorm, kNorm8, kQuant };

template <typename T, int N>
struct alignas(sizeof(T) * N) Pack {
  T v[N];
};

// The larger of m, |a| and |b|; NaN if one is.
__device__ __forceinline__ float max_abs(float m, float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;\n" : "=f"(r) : "f"(m), "f"(fabsf(a)), "f"(fabsf(b)));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;\n" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Elements 2 p and 2 p + 1 of a pack, and back (rounded).
template <int N>
__device__ __forceinline__ float2 get2(const Pack<float, N> &v, int p) {
  return make_float2(v.v[2 * p], v.v[2 * p + 1]);
}
template <int N>
__device__ __forceinline__ float2 get2(const Pack<__nv_bfloat16, N> &v, int p) {
  const unsigned w = reinterpret_cast<const unsigned *>(&v)[p];
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
template <int N>
__device__ __forceinline__ float2 get2(const Pack<__half, N> &v, int p) {
  return __half22float2(reinterpret_cast<const __half2 *>(&v)[p]);
}
template <int N>
__device__ __forceinline__ void set2(Pack<float, N> &v, int p, float2 f) {
  v.v[2 * p] = f.x;
  v.v[2 * p + 1] = f.y;
}
template <int N>
__device__ __forceinline__ void set2(Pack<__nv_bfloat16, N> &v, int p, float2 f) {
  reinterpret_cast<__nv_bfloat162 *>(&v)[p] = __floats2bfloat162_rn(f.x, f.y);
}
template <int N>
__device__ __forceinline__ void set2(Pack<__half, N> &v, int p, float2 f) {
  reinterpret_cast<__half2 *>(&v)[p] = __floats2half2_rn(f.x, f.y);
}

// Sum of `s` and maximum of `m` (not negative, or NaN) over the row's threads,
// in every thread: the block, or `tpr` lanes of a warp.  `buf` alternates
// between calls, so one barrier is enough.
struct Red {
  float s[2][32], m[2][32];
};
template <bool BLOCK>
__device__ __forceinline__ void reduce_row(float &s, float &m, Red &red, int &buf, int tpr) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    if (BLOCK || o < tpr) {
      s += __shfl_xor_sync(0xffffffffu, s, o);
      m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
    }
  if constexpr (BLOCK) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
    if (nw == 1) return;
    if (lane == 0) {
      red.s[buf][warp] = s;
      red.m[buf][warp] = m;
    }
    __syncthreads();
    s = lane < nw ? red.s[buf][lane] : 0.0f;
    m = lane < nw ? red.m[buf][lane] : 0.0f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      s += __shfl_xor_sync(0xffffffffu, s, o);
      m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
    }
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
__device__ __forceinline__ Quant make_quant(float a, float rstd) {
  Quant r{1.0f, 0.0f, 0.0f};
  if (!(a < __uint_as_float(kInfBits))) {
    r.scale = __int_as_float(0x7fc00000);
  } else if (a != 0.0f) {
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

// rint(v) in the lowest byte, for |v| <= 128: adding 1.5 2^23 rounds to the
// nearest whole number, ties to even, and leaves it in the sum's low bits.
// (t inv is within [-127, 127] but for two roundings.)
constexpr float kRound = 12582912.0f;
// N values as bytes; none where the row has no scale (inv = 0).
template <int P>
__device__ __forceinline__ uint64_t quantise(const float2 (&t)[P], const Quant &z) {
  if (z.inv == 0.0f) return 0;
  unsigned w[2] = {0, 0};
#pragma unroll
  for (int p = 0; p < P; p += 2) {
    float2 a = t[p], b = t[p + 1];
    if (z.pre != 1.0f) {
      a = mul2(a, both(z.pre));
      b = mul2(b, both(z.pre));
    }
    // (the packed product and sum would become one fma, with one rounding)
    a = mul2(a, both(z.inv));
    b = mul2(b, both(z.inv));
    auto bits_of = [](float v) { return __float_as_uint(__fadd_rn(v, kRound)); };
    const unsigned lo = __byte_perm(bits_of(a.x), bits_of(a.y), 0x0040);
    const unsigned hi = __byte_perm(bits_of(b.x), bits_of(b.y), 0x0040);
    w[p / 2] = __byte_perm(lo, hi, 0x5410);
  }
  return (uint64_t)w[0] | ((uint64_t)w[1] << 32);
}

// 1 / sqrt(mean + eps) of a row whose sum of squares is `s`.
__device__ __forceinline__ float row_rstd(float s, int cols, float eps) {
  return __frsqrt_rn(__fadd_rn(__fdiv_rn(s, (float)cols), eps));
}

// How a row lies on its `tpr` threads: NV groups of VEC values each, group i at
// VEC (tid + i tpr) - m.  RAGGED: cols is no multiple of VEC, or the rows of x,
// residual, sum and y start m values past a 16-byte boundary (the same m in
// one row, another in the next); groups follow the boundaries, so that all but
// a row's two ends move 16 bytes at a time.
template <int VEC, bool RAGGED>
struct Lay {
  int tid, tpr, m, cols;
  __device__ __forceinline__ int first(int i) const {
    return VEC * (tid + i * tpr) - (RAGGED ? m : 0);
  }
  __device__ __forceinline__ bool some(int i) const { return first(i) < cols; }
  __device__ __forceinline__ bool whole(int i) const {
    return RAGGED ? first(i) + VEC <= cols && first(i) >= 0 : first(i) < cols;
  }
  __device__ __forceinline__ bool has(int i, int e) const {
    return (!RAGGED || first(i) + e >= 0) && first(i) + e < cols;
  }
};

// Group i of a row straight from memory (zero outside the row); [lo, hi) is the
// whole tensor, so a row's ends are read with their neighbours' values unless
// those lie outside it.  Plain loads: the row may be overwritten by this kernel.
template <typename T, int VEC, bool RAGGED>
__device__ __forceinline__ Pack<T, VEC> load_group(const T *row, const Lay<VEC, RAGGED> &l, int i,
                                                   const T *lo, const T *hi) {
  Pack<T, VEC> p;
  const int first = l.first(i);
  const T *at = row + first;
  if (RAGGED ? l.some(i) && at >= lo && at + VEC <= hi : l.whole(i)) {
    p = *reinterpret_cast<const Pack<T, VEC> *>(at);
    if (RAGGED && !l.whole(i)) {
#pragma unroll
      for (int e = 0; e < VEC; ++e)
        if (e < -first || e >= l.cols - first) p.v[e] = from_f32<T>(0.0f);
    }
  } else {
#pragma unroll
    for (int e = 0; e < VEC; ++e)
      p.v[e] = RAGGED && l.has(i, e) ? at[e] : from_f32<T>(0.0f);
  }
  return p;
}

// Bytes [lo, hi) of w to the 16-byte aligned `to`, in pieces of 8, 4, 2 and 1
// bytes where one end is 0 or 16 (of a row's two ends in one group, value by value).
template <int SIZE>
__device__ __forceinline__ void store_part(char *to, const uint4 &w, int lo, int hi) {
  if (lo == 0) {
    int at = 0;
    if (hi & 8) {
      *reinterpret_cast<uint2 *>(to) = make_uint2(w.x, w.y);
      at = 8;
    }
    if (hi & 4) {
      *reinterpret_cast<unsigned *>(to + at) = at ? w.z : w.x;
      at += 4;
    }
    if (SIZE == 2 && (hi & 2)) {
      const unsigned v = at & 8 ? (at & 4 ? w.w : w.z) : (at & 4 ? w.y : w.x);
      *reinterpret_cast<unsigned short *>(to + at) = (unsigned short)v;
    }
  } else if (hi == 16) {
    const int n = 16 - lo;
    int at = 16;
    if (n & 8) {
      *reinterpret_cast<uint2 *>(to + 8) = make_uint2(w.z, w.w);
      at = 8;
    }
    if (n & 4) {
      at -= 4;
      *reinterpret_cast<unsigned *>(to + at) = at == 12 ? w.w : w.y;
    }
    if (SIZE == 2 && (n & 2)) {
      at -= 2;
      const unsigned v = at & 8 ? (at & 4 ? w.w : w.z) : (at & 4 ? w.y : w.x);
      *reinterpret_cast<unsigned short *>(to + at) = (unsigned short)(v >> 16);
    }
  } else {
    const unsigned v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 16; i += SIZE)
      if (i >= lo && i < hi) {
        if (SIZE == 2) *reinterpret_cast<unsigned short *>(to + i) = (unsigned short)(v[i / 4] >> (8 * (i & 2)));
        else *reinterpret_cast<unsigned *>(to + i) = v[i / 4];
      }
  }
}
template <typename T, int VEC, bool RAGGED>
__device__ __forceinline__ void store_group(T *row, const Lay<VEC, RAGGED> &l, int i,
                                            const Pack<T, VEC> &o) {
  const int first = l.first(i);
  if (l.whole(i)) {
    *reinterpret_cast<Pack<T, VEC> *>(row + first) = o;
  } else if (RAGGED && l.some(i)) {
    constexpr int ES = (int)sizeof(T);
    store_part<ES>(reinterpret_cast<char *>(row + first), *reinterpret_cast<const uint4 *>(&o),
                   ES * max(0, -first), ES * min(VEC, l.cols - first));
  }
}
// Gain of group i.  Only its elements' alignment is known where RAGGED: there the
// two 16-byte words that hold it are read and shifted.
template <typename G, int VEC, bool RAGGED>
__device__ __forceinline__ Pack<G, VEC> load_gain(const G *gain, const Lay<VEC, RAGGED> &l, int i) {
  Pack<G, VEC> g;
  if constexpr (!RAGGED) {
    if (l.whole(i)) g = *reinterpret_cast<const Pack<G, VEC> *>(gain + l.first(i));
    return g;
  } else {
    const int first = l.first(i);
    if constexpr (sizeof(G) * VEC == 16) {
      const char *p = reinterpret_cast<const char *>(gain + first);
      const int off = (int)(reinterpret_cast<uintptr_t>(p) & 15);
      const char *w = p - off;
      if (l.whole(i) && w >= reinterpret_cast<const char *>(gain) &&
          w + 32 <= reinterpret_cast<const char *>(gain + l.cols)) {
        const uint4 a = *reinterpret_cast<const uint4 *>(w);
        const uint4 b = reinterpret_cast<const uint4 *>(w)[1];
        *reinterpret_cast<uint4 *>(&g) = bytes_from(a, b, off);
        return g;
      }
    } else if (l.whole(i)) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) g.v[e] = gain[first + e];
      return g;
    }
#pragma unroll
    for (int e = 0; e < VEC; ++e)
      g.v[e] = l.has(i, e) ? gain[first + e] : from_f32<G>(0.0f);
    return g;
  }
}

// Writes a group's VEC 8-bit values, the bytes of `word`.  q's rows start on
// VEC bytes, so where RAGGED the group that q stores whole, [c0, c0 + VEC), is
// the upper part of this thread's word and the lower part of the next one's;
// where a warp or a row ends the parts go out in smaller pieces.  Every lane of
// the warp calls this.
template <int VEC, bool RAGGED>
__device__ __forceinline__ void store_q(int8_t *q, uint64_t word, const Lay<VEC, RAGGED> &l, int i) {
  const int c0 = VEC * (l.tid + i * l.tpr);
  auto whole_store = [&](uint64_t w) {
    if constexpr (VEC == 8) *reinterpret_cast<uint64_t *>(q + c0) = w;
    else *reinterpret_cast<unsigned *>(q + c0) = (unsigned)w;
  };
  if constexpr (!RAGGED) {
    if (l.whole(i)) whole_store(word);
  } else {
    const int lane = threadIdx.x & 31, m = l.m;
    const uint64_t next = __shfl_down_sync(0xffffffffu, word, 1);
    const bool high = lane == 31 || l.tid == l.tpr - 1;
    if (m > 0 && (lane == 0 || l.tid == 0) && c0 > 0) {
      // the lower part, [c0 - m, c0): the lane that stores it whole is not here
      if (c0 <= l.cols) {
        int at = c0;
        uint64_t w = word << (8 * (8 - m));  // its last byte on top
        if (m & 4) {
          at -= 4;
          *reinterpret_cast<unsigned *>(q + at) = (unsigned)(w >> 32);
          w <<= 32;
        }
        if (m & 2) {
          at -= 2;
          *reinterpret_cast<unsigned short *>(q + at) = (unsigned short)(w >> 48);
          w <<= 16;
        }
        if (m & 1) q[at - 1] = (int8_t)(w >> 56);
      } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e)
          if (e < m && c0 - m + e < l.cols) q[c0 - m + e] = (int8_t)(word >> (8 * e));
      }
    }
    uint64_t all = m == 0 ? word : (word >> (8 * m)) | (high ? 0 : next << (8 * (VEC - m)));
    const int n = min(l.cols - c0, high ? VEC - m : VEC);  // values of [c0, c0 + VEC) in hand
    if (n >= VEC) {
      whole_store(all);
    } else if (n > 0) {
      int8_t *to = q + c0;
      if (n & 4) {
        *reinterpret_cast<unsigned *>(to) = (unsigned)all;
        to += 4;
        all >>= 32;
      }
      if (n & 2) {
        *reinterpret_cast<unsigned short *>(to) = (unsigned short)all;
        to += 2;
        all >>= 16;
      }
      if (n & 1) *to = (int8_t)all;
    }
  }
}

// The row once its values h and gains g are in registers: sum, norm, outputs.
// `freed()` runs after the row's first reduction, when every thread of the row
// holds its values.
template <typename T, typename G, int NV, bool BLOCK, Mode MODE, bool RAGGED, typename F>
__device__ __forceinline__ void finish_row(const NormArgs &a, int64_t row,
                                           const Lay<16 / (int)sizeof(T), RAGGED> &l,
                                           const float2 (&h)[NV][8 / sizeof(T)],
                                           const Pack<G, 16 / sizeof(T)> (&g)[NV], Red &red,
                                           int &buf, F freed) {
  constexpr int VEC = 16 / (int)sizeof(T), P = VEC / 2;
  const bool gained = MODE != kQuant && a.gain;
  float2 s2 = both(0.0f);
  float top = 0.0f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    if (!l.some(i)) continue;
#pragma unroll
    for (int p = 0; p < P; ++p) {
      if (MODE != kQuant) s2 = fma2(h[i][p], h[i][p], s2);
      if (MODE != kNorm) {
        const float2 t = gained ? mul2(h[i][p], get2(g[i], p)) : h[i][p];
        top = max_abs(top, t.x, t.y);
      }
    }
    if (MODE != kQuant && a.sum) {
      Pack<T, VEC> o;
#pragma unroll
      for (int p = 0; p < P; ++p) set2(o, p, h[i][p]);
      store_group(static_cast<T *>(a.sum) + row * a.ss, l, i, o);
    }
  }
  float s = s2.x + s2.y;
  reduce_row<BLOCK>(s, top, red, buf, l.tpr);
  freed();
  float rstd = 1.0f;
  if (MODE != kQuant) {
    rstd = row_rstd(s, a.cols, a.eps);
    const bool over = !(s < __uint_as_float(kInfBits));
    // (a block takes the branch as one; of a warp with several rows, all lanes
    // take part for any of them)
    if (BLOCK ? over : __any_sync(0xffffffffu, over)) {
      // The squares overflowed: if every h is finite, scale the row by a
      // power of two and sum again (hm is past 2^48 then, so that down is
      // a normal number).
      float hm = 0.0f, none = 0.0f, zero = 0.0f;
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int p = 0; p < P; ++p) hm = max_abs(hm, h[i][p].x, h[i][p].y);
      reduce_row<BLOCK>(zero, hm, red, buf, l.tpr);
      const bool finite = hm < __uint_as_float(kInfBits);
      const float down =
          over && finite ? pow2(167 - (int)(__float_as_uint(hm) >> 23)) : 1.0f;  // to 2^40 .. 2^41
      float2 d2 = both(0.0f);
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int p = 0; p < P; ++p) {
          const float2 v = mul2(h[i][p], both(down));
          d2 = fma2(v, v, d2);
        }
      float d = d2.x + d2.y;
      reduce_row<BLOCK>(d, none, red, buf, l.tpr);
      if (over && finite) rstd = row_rstd(d, a.cols, a.eps * down * down) * down;
    }
  }
  if constexpr (MODE == kNorm) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (!l.some(i)) continue;
      Pack<T, VEC> o;
#pragma unroll
      for (int p = 0; p < P; ++p) {
        // (h rstd) gain: h rstd is at most sqrt(cols), it cannot overflow
        float2 v = mul2(h[i][p], both(rstd));
        if (gained) v = mul2(v, get2(g[i], p));
        set2(o, p, v);
      }
      store_group(static_cast<T *>(a.y) + row * a.ys, l, i, o);
    }
  } else {
    const Quant z = make_quant(top, rstd);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float2 t[P];
#pragma unroll
      for (int p = 0; p < P; ++p) t[p] = gained ? mul2(h[i][p], get2(g[i], p)) : h[i][p];
      store_q(a.q + row * a.qs, quantise(t, z), l, i);
    }
    if (l.tid == 0 && l.cols > 0) a.scale[row] = z.scale;
  }
}

template <typename T, int VEC>
__device__ __forceinline__ int shift_of(const T *row) {
  return (int)((reinterpret_cast<uintptr_t>(row) / sizeof(T)) & (uintptr_t)(VEC - 1));
}

// Few rows, or short ones: each goes from memory into the registers of a block
// (BLOCK) or of `tpr` lanes.
template <typename T, typename G, int NV, bool BLOCK, Mode MODE, bool RAGGED>
__global__ void __launch_bounds__(BLOCK ? 1024 : 128) rows_kernel(NormArgs a, int tpr) {
  constexpr int VEC = 16 / (int)sizeof(T), P = VEC / 2;
  __shared__ Red red;
  Lay<VEC, RAGGED> l;
  l.tpr = BLOCK ? blockDim.x : tpr;
  l.tid = BLOCK ? threadIdx.x : (threadIdx.x & (tpr - 1));
  l.cols = a.cols;
  const int per = BLOCK ? 1 : 128 / tpr;  // rows a block
  const T *x0 = static_cast<const T *>(a.x), *x1 = x0 + (a.rows - 1) * a.xs + a.cols;
  const T *r0 = static_cast<const T *>(a.residual), *r1 = r0 + (a.rows - 1) * a.rs + a.cols;
  int buf = 0;
  admit_next();
  after_previous();
  for (int64_t first = blockIdx.x * (int64_t)per; first < a.rows; first += gridDim.x * (int64_t)per) {
    int64_t row = first + (BLOCK ? 0 : threadIdx.x / tpr);
    // lanes past the last row take part in the warp's steps with no columns
    l.cols = row < a.rows ? a.cols : 0;
    if (!BLOCK && row >= a.rows) row = a.rows - 1;
    const T *x = static_cast<const T *>(a.x) + row * a.xs;
    const T *r = static_cast<const T *>(a.residual) + row * a.rs;
    l.m = RAGGED ? shift_of<T, VEC>(x) : 0;
    float2 h[NV][P];
    Pack<G, VEC> g[NV];
    {
      Pack<T, VEC> px[NV], pr[NV];
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        px[i] = load_group(x, l, i, x0, x1);
        if (MODE != kQuant && a.residual) pr[i] = load_group(r, l, i, r0, r1);
        if (MODE != kQuant && a.gain) g[i] = load_gain(static_cast<const G *>(a.gain), l, i);
      }
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int p = 0; p < P; ++p) {
          h[i][p] = get2(px[i], p);
          if (MODE != kQuant && a.residual) h[i][p] = add2(h[i][p], get2(pr[i], p));
        }
    }
    finish_row<T, G, NV, BLOCK, MODE, RAGGED>(a, row, l, h, g, red, buf, [] {});
  }
}

// Many rows: persistent blocks, a row a block, each with a ring of row slots
// in shared memory that bulk copies fill ahead of the row in work, so the reads
// of the next rows are in flight while a row is reduced and written; the gains
// stay in registers.  (Straight loads wait out each row's latency: 16384 rows of
// 8192 bf16 values with a residual took 259 us from rows_kernel, 171 us = 6.3
// TB/s from here; 8192 x 4096 to 8 bits 71 and 47 us.)  A slot holds the 16-byte
// pieces that cover x's row, then the residual's; RAGGED rows share pieces with
// their neighbours, so those at the ends of the tensor's first and last row are
// left out and read from memory.
struct Ring {
  int slots;
  int row_bytes;   // one operand
  int slot_bytes;  // both
};
constexpr int kMaxSlots = 3;

template <typename T, typename G, int NV, Mode MODE, bool RAGGED>
__global__ void __launch_bounds__(512)
stream_rows_kernel(NormArgs a, Ring ring, int *status, long long wait_limit) {
  constexpr int VEC = 16 / (int)sizeof(T), P = VEC / 2;
  extern __shared__ __align__(128) unsigned char ring_smem[];
  __shared__ Red red;
  __shared__ uint64_t bars[kMaxSlots];
  Lay<VEC, RAGGED> l;
  l.tpr = blockDim.x;
  l.tid = threadIdx.x;
  l.m = 0;
  l.cols = a.cols;
  const int64_t step = gridDim.x;
  const unsigned full = smem_u32(&bars[0]);
  const bool residual = MODE != kQuant && a.residual;
  const T *x0 = static_cast<const T *>(a.x), *r0 = static_cast<const T *>(a.residual);
  // a row whose partial pieces may reach outside its tensor
  auto at_end = [&](int64_t row, int64_t stride) {
    return row == 0 || row == a.rows - 1 || stride < VEC;
  };
  auto fetch_row = [&](const T *p, bool end, unsigned dst, unsigned bar, bool issue) {
    uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    uintptr_t hi = lo + (uintptr_t)a.cols * sizeof(T);
    if constexpr (RAGGED) {
      const uintptr_t at = lo & ~(uintptr_t)15;  // the slot's first piece
      lo = end ? (lo + 15) & ~(uintptr_t)15 : at;
      hi = end ? hi & ~(uintptr_t)15 : (hi + 15) & ~(uintptr_t)15;
      if (hi <= lo) return 0u;
      dst += (unsigned)(lo - at);
    }
    if (issue) bulk_load(dst, lo, (unsigned)(hi - lo), bar);
    return (unsigned)(hi - lo);
  };
  auto fetch = [&](int64_t row, int slot) {  // one thread
    const unsigned dst = smem_u32(ring_smem + slot * ring.slot_bytes), bar = full + 8 * slot;
    const T *x = x0 + row * a.xs, *r = r0 + row * a.rs;
    const bool xe = at_end(row, a.xs), re = at_end(row, a.rs);
    unsigned bytes = fetch_row(x, xe, dst, bar, false);
    if (residual) bytes += fetch_row(r, re, dst + ring.row_bytes, bar, false);
    mbar_arrive_tx(bar, bytes);
    fetch_row(x, xe, dst, bar, true);
    if (residual) fetch_row(r, re, dst + ring.row_bytes, bar, true);
  };
  admit_next();
  if (threadIdx.x == 0) {
    for (int s = 0; s < ring.slots; ++s) mbar_init(full + 8 * s, 1);
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
  }
  after_previous();
  if (threadIdx.x == 0) {
    for (int s = 0; s < ring.slots; ++s)
      if (blockIdx.x + s * step < a.rows) fetch(blockIdx.x + s * step, s);
  }
  // the gains stay in registers (where rows are shifted, as long as m does)
  Pack<G, VEC> g[NV];
  int gm = -1;
  __syncthreads();
  int buf = 0, slot = 0;
  unsigned parity = 0;
  long long limit = wait_limit;
  for (int64_t row = blockIdx.x; row < a.rows; row += step) {
    if (RAGGED) l.m = shift_of<T, VEC>(x0 + row * a.xs);
    if (MODE != kQuant && a.gain && gm != l.m) {
      gm = l.m;
#pragma unroll
      for (int i = 0; i < NV; ++i) g[i] = load_gain(static_cast<const G *>(a.gain), l, i);
    }
    // A wait that runs out is reported and the copy drained (with its own
    // bound); later waits then only look once.
    bool ok = false;
    for (long long it = 0; it < limit && !ok; ++it) ok = mbar_try_wait(full + 8 * slot, parity);
    if (!ok) {
      if (status) atomicExch(status, 401);
      mbar_drain(full + 8 * slot, parity);
      limit = 1;
    }
    const unsigned char *at = ring_smem + slot * ring.slot_bytes;
    auto take = [&](const T *tensor, int64_t stride, int off, int i) {
      Pack<T, VEC> p;
      const bool whole = l.whole(i);
      if (whole || (RAGGED && l.some(i) && !at_end(row, stride))) {
        p = *reinterpret_cast<const Pack<T, VEC> *>(at + off + 16 * (l.tid + i * l.tpr));
        if (!whole) {
          const int first = l.first(i);
#pragma unroll
          for (int e = 0; e < VEC; ++e)
            if (e < -first || e >= l.cols - first) p.v[e] = from_f32<T>(0.0f);
        }
      } else {
        const T *p_row = tensor + row * stride;
#pragma unroll
        for (int e = 0; e < VEC; ++e)
          p.v[e] = RAGGED && l.has(i, e) ? p_row[l.first(i) + e] : from_f32<T>(0.0f);
      }
      return p;
    };
    float2 h[NV][P];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const Pack<T, VEC> px = take(x0, a.xs, 0, i);
#pragma unroll
      for (int p = 0; p < P; ++p) h[i][p] = get2(px, p);
      if (residual) {
        const Pack<T, VEC> pr = take(r0, a.rs, ring.row_bytes, i);
#pragma unroll
        for (int p = 0; p < P; ++p) h[i][p] = add2(h[i][p], get2(pr, p));
      }
    }
    const int64_t next = row + ring.slots * step;
    finish_row<T, G, NV, true, MODE, RAGGED>(a, row, l, h, g, red, buf, [&] {
      if (threadIdx.x == 0 && next < a.rows) fetch(next, slot);
    });
    if (++slot == ring.slots) {
      slot = 0;
      parity ^= 1u;
    }
  }
}

// Rows longer than a block's registers, and tensors whose rows do not start
// alike: one block a row, value by value, read twice (the second time mostly
// from L2).  The sum is written on the second read, by the thread that read its
// operands, so it may be x or the residual.  A row is walked in parts of
// kPart values a thread, so that offsets within a part fit an int (with the
// simple addresses that gives) however long the row is; a part's sum of squares
// joins the thread's in 64 bits (of 2^26 equal values, 2^16 a thread, sums in 32
// bits alone put y off by 1e-4 to 4e-4).  300 x 100000 bf16 values
// 113 us, 40 x 40000 with a residual to 8 bits 24.5 us.
constexpr int kPart = 64;
template <typename T, typename G, Mode MODE>
__global__ void __launch_bounds__(1024) long_rows_kernel(NormArgs a) {
  __shared__ Red red;
  int buf = 0;
  const int n = blockDim.x;
  const int64_t step = (int64_t)kPart * n;
  admit_next();
  after_previous();
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const T *x = static_cast<const T *>(a.x) + row * a.xs;
    const T *r = static_cast<const T *>(a.residual) + row * a.rs;
    const G *g = static_cast<const G *>(a.gain);
    // (c counts from where the part begins)
    auto h_of = [&](const T *x, const T *r, int c) {
      float h = to_f32(x[c]);
      if (MODE != kQuant && a.residual) h += to_f32(r[c]);
      return h;
    };
    auto t_of = [&](float h, const G *g, int c) {
      return MODE != kQuant && a.gain ? __fmul_rn(h, to_f32(g[c])) : h;
    };
    double total = 0.0;
    float top = 0.0f, hm = 0.0f;
    for (int64_t at = threadIdx.x; at < a.cols; at += step) {
      const int end = (int)min(step, a.cols - at);
      float part = 0.0f;
#pragma unroll 4
      for (int c = 0; c < end; c += n) {
        const float h = h_of(x + at, r + at, c);
        part = fmaf(h, h, part);
        hm = max_abs(hm, h, 0.0f);
        top = max_abs(top, t_of(h, g + at, c), 0.0f);
      }
      total += part;
    }
    float s = (float)total;
    reduce_row<true>(s, top, red, buf, n);
    float rstd = 1.0f;
    if (MODE != kQuant) {
      rstd = row_rstd(s, a.cols, a.eps);
      if (!(s < __uint_as_float(kInfBits))) {  // as in finish_row
        float zero = 0.0f, none = 0.0f;
        reduce_row<true>(zero, hm, red, buf, n);
        if (hm < __uint_as_float(kInfBits)) {
          const float down = pow2(167 - (int)(__float_as_uint(hm) >> 23));
          total = 0.0;
          for (int64_t at = threadIdx.x; at < a.cols; at += step) {
            const int end = (int)min(step, a.cols - at);
            float part = 0.0f;
            for (int c = 0; c < end; c += n) {
              const float h = h_of(x + at, r + at, c) * down;
              part = fmaf(h, h, part);
            }
            total += part;
          }
          float d = (float)total;
          reduce_row<true>(d, none, red, buf, n);
          rstd = row_rstd(d, a.cols, a.eps * down * down) * down;
        }
      }
    }
    const Quant z = MODE != kNorm ? make_quant(top, rstd) : Quant{1.0f, 0.0f, 0.0f};
    for (int64_t at = threadIdx.x; at < a.cols; at += step) {
      const int end = (int)min(step, a.cols - at);
      T *sum = static_cast<T *>(a.sum) + row * a.ss + at;
      T *y = static_cast<T *>(a.y) + row * a.ys + at;
      int8_t *q = a.q + row * a.qs + at;
#pragma unroll 4
      for (int c = 0; c < end; c += n) {
        const float h = h_of(x + at, r + at, c);
        if (MODE != kQuant && a.sum) sum[c] = from_f32<T>(h);
        if constexpr (MODE == kNorm) {
          float v = h * rstd;
          if (a.gain) v *= to_f32((g + at)[c]);
          y[c] = from_f32<T>(v);
        } else {
          const float2 t[2] = {make_float2(t_of(h, g + at, c), 0.0f), both(0.0f)};
          q[c] = (int8_t)quantise(t, z);
        }
      }
    }
    if (MODE != kNorm && threadIdx.x == 0) a.scale[row] = z.scale;
  }
}

int up32(int v) { return (v + 31) / 32 * 32; }

constexpr int kSms = 148;
constexpr int kMaxGroups = 4096;  // 16-byte groups a row that a block's registers hold

template <typename T, typename G, int NV, Mode MODE, bool RAGGED>
bv_status launch_stream(const NormArgs &a, int threads, cudaStream_t st) {
  // Blocks an SM: 1024 threads' worth (8192 x 2048 bf16 to 8 bits: 27.3 us so,
  // 28.0 us with half of them).  Past 256 threads one block with a residual
  // (16384 x 8192 bf16 173 us, two blocks 194 us), else two (8192 x 8192 f32 to
  // 8 bits 53 us, one block 61 us).
  Ring ring;
  ring.row_bytes = (a.cols * (int)sizeof(T) + (RAGGED ? 30 : 0)) / 16 * 16;
  ring.slot_bytes = ring.row_bytes * (a.residual ? 2 : 1);
  int per_sm = threads <= 256 ? 1024 / threads : a.residual ? 1 : 2;
  per_sm = std::max(1, std::min(per_sm, 200 * 1024 / (2 * ring.slot_bytes)));
  ring.slots = std::min(per_sm == 1 ? 3 : 2, 216 * 1024 / ring.slot_bytes);  // 1 past 108 KB
  int *status = device_status_ptr();
  if (!status) return fail(BV_ERR_CUDA, "rms_norm: status word");
  const size_t smem = (size_t)ring.slots * ring.slot_bytes;
  auto k = stream_rows_kernel<T, G, NV, MODE, RAGGED>;
  // (room beside the kernel's static shared memory too)
  BV_TRY(ensure_dynamic_smem((const void *)k, smem + 2048, "rms_norm smem"));
  // (RAGGED: in eights, so that a block's rows all have the same m)
  const int64_t blocks = std::min<int64_t>(a.rows, RAGGED ? kSms * per_sm / 8 * 8 : kSms * per_sm);
  CUDA_TRY(launch_next(k, blocks, threads, smem, 1, st, a, ring, status, wait_limit()));
  return BV_OK;
}

template <typename T, typename G, int NV, bool BLOCK, Mode MODE, bool RAGGED>
bv_status launch_direct(const NormArgs &a, int threads, cudaStream_t st) {
  const int per = BLOCK ? 1 : 128 / threads;
  const int64_t blocks = std::min<int64_t>((a.rows + per - 1) / per, 0x7fffffff);
  CUDA_TRY(launch_next(rows_kernel<T, G, NV, BLOCK, MODE, RAGGED>, blocks, BLOCK ? threads : 128, 0,
                       1, st, a, threads));
  return BV_OK;
}

// Which kernel, and how many of a row's groups a thread takes.
template <typename T, typename G, Mode MODE, bool RAGGED>
bv_status launch_vec(const NormArgs &a, cudaStream_t st) {
  constexpr int VEC = 16 / (int)sizeof(T);
  const int groups = (a.cols + (RAGGED ? VEC - 1 : 0) + VEC - 1) / VEC;
  // Short rows: the fewest lanes with two groups each (65536 rows of 64 f32
  // values: 8.7 us with 8 lanes of two groups, 10.2 us with 16 of one).
  if (groups <= 64) {
    int lanes = 4;
    while (2 * lanes < groups) lanes *= 2;
    return launch_direct<T, G, 2, false, MODE, RAGGED>(a, lanes, st);
  }
  // Two blocks an SM and more go through the ring (300 x 4096 bf16 to 8 bits:
  // 5.3 us, 5.7 us without it; 1200 x 4096: 9.7 and 13.8 us; ragged 8192 x 4097
  // f32 107 and 128 us).  Ragged rows spend their time on the rows' ends, so
  // there fewer threads take more groups and more rows are in work at a time
  // (8192 x 8191 bf16 157 us with 160 threads, 172 us with 288).
  const bool many = a.rows >= 2 * kSms;
  if (many) {
    const int nv = RAGGED ? (groups <= 256 ? 2 : groups <= 1024 ? 4 : 8)
                          : (groups <= 1024 ? 2 : groups <= 2048 ? 4 : 8);
    const int threads = up32((groups + nv - 1) / nv);
    if (nv == 2) return launch_stream<T, G, 2, MODE, RAGGED>(a, threads, st);
    if (nv == 4) return launch_stream<T, G, 4, MODE, RAGGED>(a, threads, st);
    return launch_stream<T, G, 8, MODE, RAGGED>(a, threads, st);
  }
  // Few rows: one group a thread, as long as a block has threads (one row of
  // 4096 bf16 values: 2.6 us with 512 threads, 3.0 us with 256).
  if (groups <= 1024) return launch_direct<T, G, 1, true, MODE, RAGGED>(a, up32(groups), st);
  if (groups <= 2048)
    return launch_direct<T, G, 2, true, MODE, RAGGED>(a, up32((groups + 1) / 2), st);
  return launch_direct<T, G, 4, true, MODE, RAGGED>(a, up32((groups + 3) / 4), st);
}

template <typename T, typename G, Mode MODE>
bv_status launch_typed(const NormArgs &a, cudaStream_t st) {
  constexpr int VEC = 16 / (int)sizeof(T);
  // a tensor's rows start on whole groups (its elements' alignment is given)
  auto starts = [&](const void *p, int64_t stride, int esize) {
    return !p || (aligned_to(p, VEC * esize) && (stride % VEC == 0 || a.rows <= 1));
  };
  // rows as far past a group's start as x's, each of them
  auto follows = [&](const void *p, int64_t stride) {
    return !p || (((reinterpret_cast<uintptr_t>(p) - reinterpret_cast<uintptr_t>(a.x)) % 16 == 0) &&
                  ((stride - a.xs) % VEC == 0 || a.rows <= 1));
  };
  constexpr int es = (int)sizeof(T);
  const bool fits =
      ((int64_t)a.cols + 2 * VEC - 2) / VEC <= kMaxGroups && starts(a.q, a.qs, 1);
  if (fits && a.cols % VEC == 0 && starts(a.x, a.xs, es) && starts(a.residual, a.rs, es) &&
      starts(a.sum, a.ss, es) && starts(a.y, a.ys, es) && starts(a.gain, 0, (int)sizeof(G)))
    return launch_vec<T, G, MODE, false>(a, st);
  if (fits && follows(a.residual, a.rs) && follows(a.sum, a.ss) && follows(a.y, a.ys))
    return launch_vec<T, G, MODE, true>(a, st);
  const int64_t grid = std::min<int64_t>(a.rows, 0x7fffffff);
  const int threads = a.cols >= 4096 ? 1024 : up32((a.cols + 3) / 4);
  CUDA_TRY(launch_next(long_rows_kernel<T, G, MODE>, grid, threads, 0, 1, st, a));
  return BV_OK;
}

template <typename T, typename G>
bv_status launch_norm(const NormArgs &a, cudaStream_t st) {
  return a.q ? launch_typed<T, G, kNorm8>(a, st) : launch_typed<T, G, kNorm>(a, st);
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
      if (dtype == BV_F32) BV_TRY((launch_norm<float, float>(a, st)));
      else if (dtype == BV_BF16 && f32g) BV_TRY((launch_norm<__nv_bfloat16, float>(a, st)));
      else if (dtype == BV_BF16) BV_TRY((launch_norm<__nv_bfloat16, __nv_bfloat16>(a, st)));
      else if (f32g) BV_TRY((launch_norm<__half, float>(a, st)));
      else BV_TRY((launch_norm<__half, __half>(a, st)));
    } else {
      if (dtype == BV_F32) BV_TRY((launch_typed<float, float, kQuant>(a, st)));
      else if (dtype == BV_BF16) BV_TRY((launch_typed<__nv_bfloat16, __nv_bfloat16, kQuant>(a, st)));
      else BV_TRY((launch_typed<__half, __half, kQuant>(a, st)));
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
