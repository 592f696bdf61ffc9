// Building blocks of the router kernels: lane exchanges within a row's lanes,
// sortable keys that carry their expert's index, sorted top lists and their
// merging, and the exponentials.
#pragma once

#include "common.h"

namespace moe {

__device__ __forceinline__ float rt_neg_inf() { return -__builtin_huge_valf(); }
// The hardware's one-instruction exponential and logarithm (base 2, 1 ulp); the
// argument's rounding adds |x| 2^-24 of the result, as a - m itself has.
__device__ __forceinline__ float rt_exp(float x) { return __builtin_amdgcn_exp2f(x * 1.44269504f); }  // x <= 0
__device__ __forceinline__ float rt_log(float x) { return __builtin_amdgcn_logf(x) * 0.69314718f; }  // log2 -> log

// Two registers whose corresponding elements belong to two partner halves of
// 2D lanes: {x, partner's x} for D <= 8 (a DPP permutation: quads, then
// mirrored halves and rows), {lower half's, upper half's} for D = 16, 32 (a
// lane swap). Every use is symmetric in the two.
struct RtPair {
  uint32_t a, b;
};
template <int D>
__device__ __forceinline__ RtPair rt_pair(uint32_t x) {
  if constexpr (D == 16) {
    auto r = __builtin_amdgcn_permlane16_swap(x, x, false, false);
    return {r[0], r[1]};
  } else if constexpr (D == 32) {
    auto r = __builtin_amdgcn_permlane32_swap(x, x, false, false);
    return {r[0], r[1]};
  } else {
    constexpr int ctrl = D == 1 ? 0xB1 : D == 2 ? 0x4E : D == 4 ? 0x141 : 0x140;
    return {x, (uint32_t)__builtin_amdgcn_mov_dpp((int)x, ctrl, 0xF, 0xF, true)};
  }
}

// Sum over the 2D-lane blocks [FROM, LPR): every lane gets its block's sum.
// (Mirrored exchanges pair unequal lanes, so each step needs the steps below
// it done; FROM = 1 sums over a row's LPR lanes.)
template <int LPR, int D = 1>
__device__ __forceinline__ float rt_sum(float x) {
  if constexpr (D < LPR) {
    const RtPair p = rt_pair<D>(__float_as_uint(x));
    return rt_sum<LPR, 2 * D>(__uint_as_float(p.a) + __uint_as_float(p.b));
  } else {
    return x;
  }
}
template <int LPR, int D = 1>
__device__ __forceinline__ float rt_max(float x) {
  if constexpr (D < LPR) {
    const RtPair p = rt_pair<D>(__float_as_uint(x));
    return rt_max<LPR, 2 * D>(fmaxf(__uint_as_float(p.a), __uint_as_float(p.b)));
  } else {
    return x;
  }
}
// Sum of lane l's values over the wave's 64 / LPR rows (lanes l, l + LPR, ..).
template <int LPR, int D = LPR>
__device__ __forceinline__ float rt_sum_rows(float x) {
  if constexpr (D == 8) {  // rotate the 16-lane row by 8: l and l ^ 8
    const int y = __builtin_amdgcn_mov_dpp((int)__float_as_uint(x), 0x128, 0xF, 0xF, true);
    return rt_sum_rows<LPR, 16>(x + __uint_as_float((uint32_t)y));
  } else if constexpr (D < 64) {
    const RtPair p = rt_pair<D>(__float_as_uint(x));
    return rt_sum_rows<LPR, 2 * D>(__uint_as_float(p.a) + __uint_as_float(p.b));
  } else {
    return x;
  }
}

// Keys: a total order by logit (largest first), equal logits by expert
// (lowest first), with the expert recoverable. NaN ranks as -inf; -0 as 0.
//
// The bits of z with NaN as -inf and -0 as 0 (the sum is never -0 and quiet,
// and the maximum takes its other operand for a NaN).
__device__ __forceinline__ uint32_t rt_rankable(float z) { return __float_as_uint(fmaxf(z + 0.0f, rt_neg_inf())); }

// bf16 logits: the ordered 16 bits above the inverted index, as a uint32.
struct RtKey16 {
  using type = uint32_t;
  __device__ static type lowest() { return 0x007F0000u; }  // -inf, no expert
  __device__ static type make(float z, int e) {
    const uint32_t u = rt_rankable(z);
    const uint32_t o = u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
    return (o & 0xFFFF0000u) | (0xFFFFu - (uint32_t)e);
  }
  __device__ static type mx(type a, type b) { return a > b ? a : b; }
  __device__ static type mn(type a, type b) { return a < b ? a : b; }
  __device__ static float value(type k) {
    const uint32_t o = k & 0xFFFF0000u;
    return __uint_as_float((o & 0x80000000u ? o ^ 0x80000000u : ~o) & 0xFFFF0000u);
  }
  __device__ static int expert(type k) { return (int)(0xFFFFu - (k & 0xFFFFu)); }
  template <int D>
  __device__ static void pair(type k, type& a, type& b) {
    const RtPair p = rt_pair<D>(k);
    a = p.a;
    b = p.b;
  }
};
// fp32 logits: the logit's bits above the index as a double. The bits of a
// non-NaN fp32 are never a NaN's as the high half of a double, doubles order
// like their bits, and v_max_f64 / v_min_f64 run at full rate, so ordering a
// pair of 64-bit keys takes two instructions (five on integers).
struct RtKey32 {
  using type = double;
  __device__ static type bits(uint32_t hi, uint32_t lo) {
    return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
  }
  __device__ static type lowest() { return bits(0xFF800000u, 0xFFFFFFFFu); }
  __device__ static type make(float z, int e) {
    const uint32_t u = rt_rankable(z);
    // a larger low half is a larger magnitude: the inverted index for
    // positive logits, the index itself for negative ones
    return bits(u, ~(uint32_t)e ^ (uint32_t)((int32_t)u >> 31));
  }
  __device__ static type mx(type a, type b) { return __builtin_fmax(a, b); }
  __device__ static type mn(type a, type b) { return __builtin_fmin(a, b); }
  __device__ static uint32_t hi(type k) { return (uint32_t)(__builtin_bit_cast(uint64_t, k) >> 32); }
  __device__ static float value(type k) { return __uint_as_float(hi(k)); }
  __device__ static int expert(type k) {
    const uint32_t lo = (uint32_t)__builtin_bit_cast(uint64_t, k);
    return (int)(~lo ^ (uint32_t)((int32_t)hi(k) >> 31));
  }
  template <int D>
  __device__ static void pair(type k, type& a, type& b) {
    const uint64_t u = __builtin_bit_cast(uint64_t, k);
    const RtPair l = rt_pair<D>((uint32_t)u), h = rt_pair<D>((uint32_t)(u >> 32));
    a = bits(h.a, l.a);
    b = bits(h.b, l.b);
  }
};

template <class K>
__device__ __forceinline__ void rt_order(typename K::type& a, typename K::type& b) {
  const typename K::type x = K::mx(a, b), y = K::mn(a, b);
  a = x;
  b = y;
}
// Sorts v[0..N), largest first (Batcher's odd-even merge sort).
template <class K, int N>
__device__ __forceinline__ void rt_sort(typename K::type (&v)[N]) {
#pragma unroll
  for (int p = 1; p < N; p *= 2)
#pragma unroll
    for (int k = p; k >= 1; k /= 2)
#pragma unroll
      for (int j = k % p; j + k < N; j += 2 * k)
#pragma unroll
        for (int i = 0; i < k; ++i)
          if (i + j + k < N && (i + j) / (2 * p) == (i + j + k) / (2 * p)) rt_order<K>(v[i + j], v[i + j + k]);
}
// The L largest of two sorted lists, sorted: the larger of each opposite pair
// is a bitonic list of them.
template <class K, int L>
__device__ __forceinline__ void rt_merge(typename K::type (&v)[L], const typename K::type (&w)[L]) {
#pragma unroll
  for (int i = 0; i < L; ++i) v[i] = K::mx(v[i], w[L - 1 - i]);
#pragma unroll
  for (int d = L / 2; d >= 1; d /= 2)
#pragma unroll
    for (int i = 0; i < L; ++i)
      if ((i & d) == 0) rt_order<K>(v[i], v[i + d]);
}
// The L largest of a row: every lane's list becomes the row's.
template <class K, int L, int LPR, int D = 1>
__device__ __forceinline__ void rt_merge_lanes(typename K::type (&v)[L]) {
  if constexpr (D < LPR) {
    typename K::type a[L], b[L];
#pragma unroll
    for (int i = 0; i < L; ++i) K::template pair<D>(v[i], a[i], b[i]);
    rt_merge<K, L>(a, b);
#pragma unroll
    for (int i = 0; i < L; ++i) v[i] = a[i];
    rt_merge_lanes<K, L, LPR, 2 * D>(v);
  }
}

// Elements of a row in 16-byte pieces: piece c of lane l of the row holds the
// experts (c LPR + l) VEC .. + VEC - 1, so the lanes of a row read whole
// cache lines. Rows need no alignment beyond their elements'.
template <class T>
struct RtVec;
template <>
struct RtVec<float> {
  static constexpr int N = 4;
  using key = RtKey32;
  typedef float vec __attribute__((ext_vector_type(4), aligned(4)));
  __device__ static float get(vec v, int i) { return v[i]; }
  __device__ static float one(const float* p) { return *p; }
  __device__ static void put(vec& v, int i, float x) { v[i] = x; }
  __device__ static void put(float* p, float x) { *p = x; }
};
template <>
struct RtVec<uint16_t> {
  static constexpr int N = 8;
  using key = RtKey16;
  typedef uint16_t vec __attribute__((ext_vector_type(8), aligned(2)));
  __device__ static float get(vec v, int i) { return bf16_bits_to_f32(v[i]); }
  __device__ static float one(const uint16_t* p) { return bf16_bits_to_f32(*p); }
  __device__ static uint16_t bits(float x) { return __builtin_bit_cast(uint16_t, (__bf16)x); }  // nearest even
  __device__ static void put(vec& v, int i, float x) { v[i] = bits(x); }
  __device__ static void put(uint16_t* p, float x) { *p = bits(x); }
};

// A row's logits, VPL per lane; -inf past E and where !on.
template <class T, int LPR, int VPL>
__device__ __forceinline__ void rt_load_row(const T* row, int E, int l, bool on, float (&z)[VPL]) {
  using V = RtVec<T>;
  if (E == LPR * VPL && __all(on)) {  // the usual case, without a choice per lane
#pragma unroll
    for (int c = 0; c < VPL / V::N; ++c) {
      const typename V::vec v = *reinterpret_cast<const typename V::vec*>(row + (c * LPR + l) * V::N);
#pragma unroll
      for (int i = 0; i < V::N; ++i) z[c * V::N + i] = V::get(v, i);
    }
    return;
  }
  // No branch per piece: a load behind a branch waits for the one before it.
  // A lane whose piece lies past E, or is partial, reads the row's first
  // instead (none if E < N, where all are partial).
#pragma unroll
  for (int i = 0; i < VPL; ++i) z[i] = rt_neg_inf();
  if (!on) return;
  if (E >= V::N) {
    typename V::vec v[VPL / V::N];
#pragma unroll
    for (int c = 0; c < VPL / V::N; ++c) {
      const int e = (c * LPR + l) * V::N;
      v[c] = *reinterpret_cast<const typename V::vec*>(row + (e + V::N <= E ? e : 0));
    }
#pragma unroll
    for (int c = 0; c < VPL / V::N; ++c)
#pragma unroll
      for (int i = 0; i < V::N; ++i)
        z[c * V::N + i] = (c * LPR + l) * V::N + V::N <= E ? V::get(v[c], i) : rt_neg_inf();
  }
  if (E % V::N != 0) {  // the last, partial piece: of lane (E / N) % LPR
    if (E / V::N % LPR != l) return;
    const int last = E / V::N * V::N;
    float x[V::N - 1];
#pragma unroll
    for (int i = 0; i < V::N - 1; ++i) x[i] = V::one(row + min(last + i, E - 1));
#pragma unroll
    for (int c = 0; c < VPL / V::N; ++c)
#pragma unroll
      for (int i = 0; i < V::N - 1; ++i)
        if (last == (c * LPR + l) * V::N && last + i < E) z[c * V::N + i] = x[i];
  }
}

// The unnormalised probability of logit z in a row whose largest is m (at
// most 1, and not below about 1/2 for the largest itself):
//   softmax: exp(z - m)
//   sigmoid: sigmoid(z) = exp(z) / (1 + exp(z)), relative to exp(m) where m is
//     below 0, so that small shares underflow with the share, not with the
//     score (the exponential's results below 2^-126 are 0)
// rt_base(m) is the part of m that the row's scores are relative to.
template <bool SIGMOID>
__device__ __forceinline__ float rt_base(float m) {
  return m == rt_neg_inf() ? 0.0f : SIGMOID ? fminf(m, 0.0f) : m;
}
template <bool SIGMOID>
__device__ __forceinline__ float rt_score(float z, float base) {
  if (!SIGMOID) return rt_exp(z - base);
  // (a NaN z must stay NaN: z > 0 is false for it)
  return rt_exp((z > 0.0f ? 0.0f : z) - base) * __builtin_amdgcn_rcpf(1.0f + rt_exp(-fabsf(z)));
}

}  // namespace moe
