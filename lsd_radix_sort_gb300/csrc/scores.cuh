// Device helpers shared by the losses: score types, base-2 exponentials,
// warp sums and maxima.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"

namespace lsdrs {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLog2eLow = static_cast<float>(1.4426950408889634 - static_cast<double>(kLog2e));

// One score type: its raw word in memory and its conversions.
template <int TYPE>
struct Score;
template <>
struct Score<RS_SCORE_F16> {
  using Raw = uint16_t;
  static __device__ __forceinline__ float load(Raw r) { return __half2float(__ushort_as_half(r)); }
  static __device__ __forceinline__ Raw store(float v) {
    return __half_as_ushort(__float2half_rn(v));
  }
};
template <>
struct Score<RS_SCORE_BF16> {
  using Raw = uint16_t;
  static __device__ __forceinline__ float load(Raw r) {
    return __uint_as_float(static_cast<uint32_t>(r) << 16);
  }
  static __device__ __forceinline__ Raw store(float v) {
    return __bfloat16_as_ushort(__float2bfloat16_rn(v));
  }
};
template <>
struct Score<RS_SCORE_F32> {
  using Raw = uint32_t;
  static __device__ __forceinline__ float load(Raw r) { return __uint_as_float(r); }
  static __device__ __forceinline__ Raw store(float v) { return __float_as_uint(v); }
};

template <int TYPE>
struct ScoreTag {
  static constexpr int value = TYPE;
};

__device__ __forceinline__ int64_t load_index(const void* p, int bytes, int64_t i) {
  return bytes == 8 ? static_cast<const int64_t*>(p)[i] : static_cast<const int32_t*>(p)[i];
}

// 2^x; 0 for -inf, NaN for NaN.
__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, o));
  return v;
}

// A softmax in progress: the largest score m and sum = sum exp((x - m) / t).
// Scores of -inf leave it as it is, so m = -inf and sum = 0 until the first
// other one; a NaN or +inf score makes the sum NaN for good.
struct Softmax {
  float m, sum;
};

// The point that exponents are taken from: m, or 0 while there is no score
// (so that -inf - m stays -inf).
__device__ __forceinline__ float origin(float m) { return m == -INFINITY ? 0.0f : m; }

// (a - b) scale, where the difference of two finite scores may be more than a
// float holds (half of it is not; the factors of 2 are exact).
__device__ __forceinline__ float apart2(float a, float b, float scale) {
  return __fmaf_rn(0.5f, a, -0.5f * b) * scale * 2.0f;
}

// Both halves of a row: scale2 = log2(e) / temperature.
__device__ __forceinline__ Softmax join(Softmax a, Softmax b, float scale2) {
  const float m = fmaxf(a.m, b.m), o = origin(m);
  return {m, a.sum * exp2_approx(apart2(a.m, o, scale2)) +
                 b.sum * exp2_approx(apart2(b.m, o, scale2))};
}

__device__ __forceinline__ Softmax warp_join(Softmax v, float scale2) {
  const float m = warp_max(v.m);
  return {m, warp_sum(v.sum * exp2_approx(apart2(v.m, origin(m), scale2)))};
}

// ---- 16-byte vectors of scores --------------------------------------------
// Pairs of floats in one 64-bit register: one instruction for both (8,192 x
// 65,536 bf16 policy gradients took 361 us with them, 375 with scalar ones).
__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t exp2_2(uint64_t v) {
  float a, b;
  unpack2(v, a, b);
  return pack2(exp2_approx(a), exp2_approx(b));
}

// One 32-bit word of two 16-bit scores, or two words of one 32-bit score
// each, as a pair of floats; and the largest of four words (NaN ignored).
template <int TYPE>
struct ScoreVec;

template <>
struct ScoreVec<RS_SCORE_F16> {
  static constexpr int kCount = 8;
  static constexpr uint32_t kMinusInf = 0xFC00FC00u;
  static __device__ __forceinline__ uint64_t pair(uint32_t w) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
    return pack2(f.x, f.y);
  }
  static __device__ __forceinline__ uint32_t word(uint64_t v) {
    float a, b;
    unpack2(v, a, b);
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  static __device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) {
    const __half2 h =
        __hmax2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
    return *reinterpret_cast<const uint32_t*>(&h);
  }
};

template <>
struct ScoreVec<RS_SCORE_BF16> {
  static constexpr int kCount = 8;
  static constexpr uint32_t kMinusInf = 0xFF80FF80u;
  static __device__ __forceinline__ uint64_t pair(uint32_t w) {
    return pack2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
  }
  static __device__ __forceinline__ uint32_t word(uint64_t v) {
    float a, b;
    unpack2(v, a, b);
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  static __device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) {
    const __nv_bfloat162 h = __hmax2(*reinterpret_cast<const __nv_bfloat162*>(&a),
                                     *reinterpret_cast<const __nv_bfloat162*>(&b));
    return *reinterpret_cast<const uint32_t*>(&h);
  }
};

template <>
struct ScoreVec<RS_SCORE_F32> {
  static constexpr int kCount = 4;
  static constexpr uint32_t kMinusInf = 0xFF800000u;
};

// The largest score of VECS vectors; NaN is ignored.
template <int TYPE, int VECS>
__device__ __forceinline__ float vec_max(const uint4 (&v)[VECS]) {
  if constexpr (TYPE == RS_SCORE_F32) {
    float m = -INFINITY;
#pragma unroll
    for (int u = 0; u < VECS; ++u)
      m = fmaxf(m, fmaxf(fmaxf(__uint_as_float(v[u].x), __uint_as_float(v[u].y)),
                         fmaxf(__uint_as_float(v[u].z), __uint_as_float(v[u].w))));
    return m;
  } else {
    using V = ScoreVec<TYPE>;
    uint32_t m = V::kMinusInf;
#pragma unroll
    for (int u = 0; u < VECS; ++u)
      m = V::larger(m, V::larger(V::larger(v[u].x, v[u].y), V::larger(v[u].z, v[u].w)));
    float a, b;
    unpack2(V::pair(m), a, b);
    return fmaxf(a, b);
  }
}

// A vector as kCount / 2 pairs of floats.
template <int TYPE>
__device__ __forceinline__ void vec_pairs(const uint4& v,
                                          uint64_t (&p)[ScoreVec<TYPE>::kCount / 2]) {
  if constexpr (TYPE == RS_SCORE_F32) {
    p[0] = pack2(__uint_as_float(v.x), __uint_as_float(v.y));
    p[1] = pack2(__uint_as_float(v.z), __uint_as_float(v.w));
  } else {
    using V = ScoreVec<TYPE>;
    p[0] = V::pair(v.x);
    p[1] = V::pair(v.y);
    p[2] = V::pair(v.z);
    p[3] = V::pair(v.w);
  }
}

template <int TYPE>
__device__ __forceinline__ uint4 vec_of(const uint64_t (&p)[ScoreVec<TYPE>::kCount / 2]) {
  uint4 v;
  if constexpr (TYPE == RS_SCORE_F32) {
    float a, b;
    unpack2(p[0], a, b);
    v.x = __float_as_uint(a);
    v.y = __float_as_uint(b);
    unpack2(p[1], a, b);
    v.z = __float_as_uint(a);
    v.w = __float_as_uint(b);
  } else {
    using V = ScoreVec<TYPE>;
    v = make_uint4(V::word(p[0]), V::word(p[1]), V::word(p[2]), V::word(p[3]));
  }
  return v;
}

// For an origin whose product with the scale is 2^30 or more (scores of -1e30
// that mask, or a very small temperature): neighbouring scores are then at
// least 2^6 apart in the exponent, so that only those equal to the origin
// count, and the product is rounded by 2^6 and more, soon too far to be put
// right by a factor.  Any scale gives the same 1 or 0 that keeps neighbours apart;
// the power of two that takes the origin to [2^33, 2^34) does (2^9 at least
// between neighbours), and its product with the origin is exact.
__device__ __forceinline__ bool far_origin(float o, float os2) {
  return !(fabsf(os2) < 1073741824.0f) && !isinf(o);
}
__device__ __forceinline__ float far_scale(float o) {
  return __uint_as_float(((127u + 127u + 33u) << 23) - (__float_as_uint(o) & 0x7F800000u));
}

// exp2((x - o) scale) of pairs of scores.  One multiply-add per score takes
// x * scale - os2 with os2 = o * scale rounded: the product is exact inside,
// so the result is that of a slightly other origin, and `mend` = the factor
// 2^(os2 - o scale) puts it right, once per sum.
struct Exponent {
  float scale, os2, mend;

  __device__ __forceinline__ Exponent(float o, float scale_) : scale(scale_), os2(o * scale_) {
    if (far_origin(o, os2)) {
      scale = far_scale(o);
      os2 = o * scale;
    }
    mend = exp2_approx(__fmaf_rn(-o, scale, os2));
  }
  // the exponential of one score, put right
  __device__ __forceinline__ float one(float x) const {
    return exp2_approx(__fmaf_rn(x, scale, -os2)) * mend;
  }
  __device__ __forceinline__ uint64_t of(uint64_t x) const {
    return exp2_2(fma2(x, pack2(scale, scale), pack2(-os2, -os2)));
  }
};

// From here on (and for an lse that is none, or that a float does not hold) a
// saved lse carries too little of its row: it is rounded by up to 2^-15 at
// 1024, which a probability then is off by; at 2^24 the sum of a row is lost
// altogether.  The backward call takes the statistics of such a row again.
constexpr float kFarLse = 1024.0f;
__device__ __forceinline__ bool far_lse(float lse) { return fabsf(lse) >= kFarLse; }

// exp2(x scale - lse log2 e) for a saved lse, which came from the temperature
// itself: the rounding of scale would not cancel against it as it does against
// a sum taken with the same scale, and is off by |x| scale 2^-24 in the
// exponent.  So scale = hi + lo, and both products are added for 32-bit
// scores (LOW; 16-bit results are rounded far above that).
template <bool LOW>
struct ExponentOfLse {
  float hi, lo, least, os2, mend;

  __device__ __forceinline__ ExponentOfLse(float lse, float hi_, float lo_)
      : hi(hi_),
        lo(lo_),
        least(fmaxf((lse * kLog2e - 300.0f) / hi_, -3.0e38f)),
        os2(lse * kLog2e) {
    mend = exp2_approx(__fmaf_rn(-lse, kLog2e, os2) - lse * kLog2eLow);
  }
  // -os2, with the low product; that of a score whose exponential is 0 anyway
  // must not be infinite (for lo < 0 it would be +inf)
  __device__ __forceinline__ float rest(float x) const {
    return LOW ? __fmaf_rn(fmaxf(x, least), lo, -os2) : -os2;
  }
  __device__ __forceinline__ float one(float x) const {
    return exp2_approx(__fmaf_rn(x, hi, rest(x))) * mend;
  }
  __device__ __forceinline__ uint64_t of(uint64_t x) const {
    float a, b;
    unpack2(x, a, b);
    return exp2_2(fma2(x, pack2(hi, hi), pack2(rest(a), rest(b))));
  }
};

// Adds the exponentials of a vector to two pairs of partial sums.
template <int TYPE>
__device__ __forceinline__ void vec_exp_sum(const uint4& v, const Exponent& e,
                                            uint64_t (&acc)[2]) {
  uint64_t p[ScoreVec<TYPE>::kCount / 2];
  vec_pairs<TYPE>(v, p);
#pragma unroll
  for (int i = 0; i < ScoreVec<TYPE>::kCount / 2; ++i)
    acc[i & 1] = add2(acc[i & 1], e.of(p[i]));
}

// f times the exponentials of a vector, rounded to the scores' type.
template <int TYPE, class E>
__device__ __forceinline__ uint4 vec_grad(const uint4& v, const E& e, uint64_t f) {
  uint64_t p[ScoreVec<TYPE>::kCount / 2];
  vec_pairs<TYPE>(v, p);
#pragma unroll
  for (int i = 0; i < ScoreVec<TYPE>::kCount / 2; ++i) p[i] = mul2(e.of(p[i]), f);
  return vec_of<TYPE>(p);
}

// A thread's softmax in progress over many vectors.  The origin is the
// largest score of some vectors past; it moves only when a score exceeds it
// by more than 2^8 would (so no sum overflows), which keeps the maximum off
// the path of the exponentials.  (Exponents up to 8 are rounded by 2^-22 at
// most, as exponentials are anyway; and 8 is less than half of what
// neighbouring scores of a far origin are apart, so that the limit is then
// the origin itself.)  The result is taken from the largest score of all: the
// logarithm of the sum is then small where one score outweighs the others, and
// a loss near 0 no difference of two large numbers.
template <int TYPE>
struct RunningSoftmax {
  float scale, slack, o, limit, top;
  Exponent e;
  uint64_t acc[2];

  __device__ __forceinline__ explicit RunningSoftmax(float scale2)
      : scale(scale2),
        slack(8.0f / scale2),
        o(-INFINITY),
        limit(-INFINITY),
        top(-INFINITY),
        e(0.0f, scale2) {
    acc[0] = acc[1] = 0;
  }
  __device__ __forceinline__ float total() const {
    float a, b;
    unpack2(add2(acc[0], acc[1]), a, b);
    return (a + b) * e.mend;
  }
  __device__ __forceinline__ void move(float m) {
    const float sum = total() * exp2_approx(apart2(o, m, scale));
    o = m;
    limit = m + slack;
    e = Exponent(m, scale);
    acc[0] = pack2(__fdividef(sum, e.mend), 0.0f);
    acc[1] = 0;
  }
  template <int VECS>
  __device__ __forceinline__ void add(const uint4 (&v)[VECS]) {
    const float m = vec_max<TYPE>(v);
    top = fmaxf(top, m);
    if (m > limit) move(m);
#pragma unroll
    for (int u = 0; u < VECS; ++u) vec_exp_sum<TYPE>(v[u], e, acc);
  }
  __device__ __forceinline__ Softmax result() const {
    const float sum = total();
    return {top, top > o ? sum * exp2_approx(apart2(o, top, scale)) : sum};
  }
};

// The softmax of vectors that a thread holds all at once.
template <int TYPE, int VECS>
__device__ __forceinline__ Softmax softmax_of(const uint4 (&v)[VECS], float scale2) {
  const float m = vec_max<TYPE>(v);
  const Exponent e(origin(m), scale2);
  uint64_t acc[2] = {0, 0};
#pragma unroll
  for (int u = 0; u < VECS; ++u) vec_exp_sum<TYPE>(v[u], e, acc);
  float a, b;
  unpack2(add2(acc[0], acc[1]), a, b);
  return {m, (a + b) * e.mend};
}

// A row of scores as 16-byte vectors of memory: vector 0 begins at the row's
// address rounded down to 16 bytes, so its first `lead` scores, and the last
// vector's scores past the row, belong to others and are never touched.
template <int TYPE>
struct RowVecs {
  using Raw = typename Score<TYPE>::Raw;
  static constexpr int kN = ScoreVec<TYPE>::kCount;
  int lead, cols, count;

  __device__ __forceinline__ RowVecs(const void* row, int cols_)
      : lead(static_cast<int>(reinterpret_cast<uintptr_t>(row) % 16 / sizeof(Raw))),
        cols(cols_),
        count((lead + cols_ + kN - 1) / kN) {}

  // Vectors [whole_begin, whole_end) lie inside the row entirely.
  __device__ __forceinline__ int whole_begin() const { return lead != 0; }
  __device__ __forceinline__ int whole_end() const { return (lead + cols) / kN; }
  __device__ __forceinline__ bool whole(int v) const {
    return v >= whole_begin() && v < whole_end();
  }

  // A vector that is not whole, the foreign places filled with -inf.
  __device__ __forceinline__ uint4 load_edge(const Raw* row, int v) const {
    uint32_t w[4] = {ScoreVec<TYPE>::kMinusInf, ScoreVec<TYPE>::kMinusInf,
                     ScoreVec<TYPE>::kMinusInf, ScoreVec<TYPE>::kMinusInf};
    const int64_t first = static_cast<int64_t>(v) * kN - lead;
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const int64_t j = first + i;
      if (j >= 0 && j < cols) {
        if constexpr (sizeof(Raw) == 4) {
          w[i] = row[j];
        } else {
          const int sh = 16 * (i & 1);
          w[i >> 1] = (w[i >> 1] & ~(0xFFFFu << sh)) | (static_cast<uint32_t>(row[j]) << sh);
        }
      }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }

  // Any vector, -inf past the row; vec0: the 16 bytes that vector 0 begins in.
  __device__ __forceinline__ uint4 load(const uint4* vec0, const Raw* row, int v) const {
    if (whole(v)) return vec0[v];
    constexpr uint32_t kNone = ScoreVec<TYPE>::kMinusInf;
    return v < count ? load_edge(row, v) : make_uint4(kNone, kNone, kNone, kNone);
  }

  // The same of an edge to 16 bytes of shared memory, one lane per score.
  __device__ __forceinline__ void copy_edge(const Raw* row, int v, void* to, int lane) const {
    if (lane < kN) {
      const int64_t j = static_cast<int64_t>(v) * kN - lead + lane;
      static_cast<Raw*>(to)[lane] = j >= 0 && j < cols
                                        ? row[j]
                                        : static_cast<Raw>(ScoreVec<TYPE>::kMinusInf);
    }
  }

  // Any vector, score by score.
  __device__ __forceinline__ void store_scores(Raw* row, int v, const uint4& x) const {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    const int64_t first = static_cast<int64_t>(v) * kN - lead;
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const int64_t j = first + i;
      if (j >= 0 && j < cols) {
        if constexpr (sizeof(Raw) == 4)
          row[j] = w[i];
        else
          row[j] = static_cast<Raw>(w[i >> 1] >> (16 * (i & 1)));
      }
    }
  }
};

// Where a row of results goes that is computed as the vectors of a RowVecs:
// the same vectors of memory if both rows begin at the same place in their 16
// bytes, else `shift` scores later.
template <int TYPE>
struct RowOut {
  using Raw = typename Score<TYPE>::Raw;
  static constexpr int kN = ScoreVec<TYPE>::kCount;
  Raw* row;
  uint4* vec0;  // the 16 bytes that vector 0 begins in
  int shift;

  __device__ __forceinline__ RowOut(Raw* row_, const RowVecs<TYPE>& vecs)
      : row(row_),
        vec0(reinterpret_cast<uint4*>(reinterpret_cast<uintptr_t>(row_ - vecs.lead) &
                                      ~static_cast<uintptr_t>(15))),
        shift(static_cast<int>(reinterpret_cast<uintptr_t>(row_ - vecs.lead) % 16 / sizeof(Raw))) {}

  // Consecutive lanes store consecutive vectors v, all of them whole, shift
  // != 0: 16 bytes of memory hold the end of one lane's vector and the
  // beginning of the next one's.  (Score by score, a misaligned f32 gradient
  // of 1,021 x 50,001 took 83 us instead of 71.)
  __device__ __forceinline__ void store_shifted(int v, const uint4& x) const {
    const uint32_t lane = lane_id();
    uint32_t c[8] = {x.x, x.y, x.z, x.w, x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = __shfl_up_sync(kFull, c[i], 1);
    const int bytes = shift * static_cast<int>(sizeof(Raw));
    const bool two = bytes & 8, one = bytes & 4, half = bytes & 2;
    uint32_t a[6], b[5];  // words -2 .. 3 and -1 .. 3 of the result
#pragma unroll
    for (int k = 0; k < 6; ++k) a[k] = two ? c[k] : c[k + 2];
#pragma unroll
    for (int k = 0; k < 5; ++k) b[k] = one ? a[k] : a[k + 1];
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) w[k] = half ? __funnelshift_l(b[k], b[k + 1], 16) : b[k + 1];
    if (lane != 0) __stcs(vec0 + v, make_uint4(w[0], w[1], w[2], w[3]));
    Raw* first = reinterpret_cast<Raw*>(vec0 + v) + shift;  // of this lane's own vector
    const uint32_t own[4] = {x.x, x.y, x.z, x.w};
    if (lane == 0 || lane == kWarp - 1) {
#pragma unroll
      for (int i = 0; i < kN; ++i) {
        const uint32_t word = own[i * sizeof(Raw) / 4];
        const Raw r = static_cast<Raw>(sizeof(Raw) == 4 ? word : word >> (16 * (i & 1)));
        if (lane == 0 ? i < kN - shift : i >= kN - shift) first[i] = r;
      }
    }
  }

  // Any vector of the row, whole or not.
  __device__ __forceinline__ void store(const RowVecs<TYPE>& vecs, int v, const uint4& x) const {
    if (shift == 0 && vecs.whole(v))
      vec0[v] = x;
    else
      vecs.store_scores(row, v, x);
  }
};

}  // namespace lsdrs
