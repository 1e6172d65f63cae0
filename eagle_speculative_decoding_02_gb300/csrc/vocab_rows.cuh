// Shared parts of the operators on vocabulary rows (vocab_rows.cu: long rows,
// vocab_short.cu: short ones): elements, two-float arithmetic, sums of
// exponentials, the order of alternatives, the teacher, a row's last steps.
#pragma once

#include <cfloat>
#include <type_traits>

#include "../../include/eagle.h"
#include "common.cuh"
#include "vocab_rows.h"

namespace eg {
namespace vocab {

constexpr unsigned kFull = 0xffffffffu;
constexpr float kNoTail = -1e30f;  // unlisted logits this far below the largest, in temperatures: masked

// ---- elements --------------------------------------------------------------------------------------

// A 16-byte vector of kVec logits as 4 words.
template <typename T> struct El { static constexpr int kVec = 16 / sizeof(T); };

__device__ __forceinline__ float up(float v) { return v; }
__device__ __forceinline__ float up(bf16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float up(__half v) { return __half2float(v); }
template <typename T> __device__ __forceinline__ T down(float v);
template <> __device__ __forceinline__ float down<float>(float v) { return v; }
template <> __device__ __forceinline__ bf16 down<bf16>(float v) { return __float2bfloat16_rn(v); }
template <> __device__ __forceinline__ __half down<__half>(float v) { return __float2half_rn(v); }

// Two neighbouring entries: words 2w, 2w + 1 of a float vector, the halves of word w of the others.
__device__ __forceinline__ uint32_t word_of(const uint4& q, int w) {
  return w == 0 ? q.x : w == 1 ? q.y : w == 2 ? q.z : q.w;
}
template <typename T> __device__ __forceinline__ float2 pair_of(const uint4& q, int w);
template <> __device__ __forceinline__ float2 pair_of<float>(const uint4& q, int w) {
  return make_float2(__uint_as_float(word_of(q, 2 * w)), __uint_as_float(word_of(q, 2 * w + 1)));
}
template <> __device__ __forceinline__ float2 pair_of<bf16>(const uint4& q, int w) {
  const uint32_t u = word_of(q, w);
  return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}
template <> __device__ __forceinline__ float2 pair_of<__half>(const uint4& q, int w) {
  const uint32_t u = word_of(q, w);
  return __half22float2(*reinterpret_cast<const __half2*>(&u));
}

// Largest entry of a vector (NaNs are passed over).
template <typename T> __device__ __forceinline__ float vec_max(const uint4& q);
template <> __device__ __forceinline__ float vec_max<float>(const uint4& q) {
  return fmaxf(fmaxf(__uint_as_float(q.x), __uint_as_float(q.y)), fmaxf(__uint_as_float(q.z), __uint_as_float(q.w)));
}
template <> __device__ __forceinline__ float vec_max<bf16>(const uint4& q) {
  auto h = [](const uint32_t& u) { return *reinterpret_cast<const __nv_bfloat162*>(&u); };
  const __nv_bfloat162 m = __hmax2(__hmax2(h(q.x), h(q.y)), __hmax2(h(q.z), h(q.w)));
  return fmaxf(__low2float(m), __high2float(m));
}
template <> __device__ __forceinline__ float vec_max<__half>(const uint4& q) {
  auto h = [](const uint32_t& u) { return *reinterpret_cast<const __half2*>(&u); };
  const __half2 m = __hmax2(__hmax2(h(q.x), h(q.y)), __hmax2(h(q.z), h(q.w)));
  return fmaxf(__low2float(m), __high2float(m));
}

// Largest entry of kN vectors.
template <typename T, int kN> __device__ __forceinline__ float vecs_max(const uint4 (&q)[kN]) {
  if constexpr (sizeof(T) == 4) {
    float m = vec_max<T>(q[0]);
#pragma unroll
    for (int i = 1; i < kN; ++i) m = fmaxf(m, vec_max<T>(q[i]));
    return m;
  } else {
    using T2 = std::conditional_t<std::is_same_v<T, bf16>, __nv_bfloat162, __half2>;
    auto h = [](const uint32_t& u) { return *reinterpret_cast<const T2*>(&u); };
    T2 m = h(q[0].x);
#pragma unroll
    for (int i = 0; i < kN; ++i) m = __hmax2(__hmax2(__hmax2(m, h(q[i].x)), h(q[i].y)), __hmax2(h(q[i].z), h(q[i].w)));
    return fmaxf(-INFINITY, fmaxf(up(m.x), up(m.y)));
  }
}

template <typename T> __device__ __forceinline__ uint32_t pack(float2 v);
template <> __device__ __forceinline__ uint32_t pack<bf16>(float2 v) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(v.x, v.y);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <> __device__ __forceinline__ uint32_t pack<__half>(float2 v) {
  const __half2 h = __floats2half2_rn(v.x, v.y);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// ---- arithmetic ------------------------------------------------------------------------------------

__device__ __forceinline__ float ex2(float x) {  // relative error below 2^-22; below 2^-126: 0
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Two float operations in one instruction.
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 r;
  asm("{\n.reg .b64 p, q, s;\nmov.b64 p, {%2, %3};\nmov.b64 q, {%4, %5};\nadd.rn.f32x2 s, p, q;\nmov.b64 {%0, %1}, s;\n}"
      : "=f"(r.x), "=f"(r.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 r;
  asm("{\n.reg .b64 p, q, s;\nmov.b64 p, {%2, %3};\nmov.b64 q, {%4, %5};\nmul.rn.f32x2 s, p, q;\nmov.b64 {%0, %1}, s;\n}"
      : "=f"(r.x), "=f"(r.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 r;
  asm("{\n.reg .b64 p, q, s, t;\nmov.b64 p, {%2, %3};\nmov.b64 q, {%4, %5};\nmov.b64 s, {%6, %7};\n"
      "fma.rn.f32x2 t, p, q, s;\nmov.b64 {%0, %1}, t;\n}"
      : "=f"(r.x), "=f"(r.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return r;
}

// The scale of exponents: 2^(c x) = exp(x / temperature), c = hi + lo; inv + inv_lo = 1 / temperature.
struct Scale {
  float hi, lo, inv, inv_lo;
};

// 2^(d c) with the rounding of d c made good (d c of 20 bits alone would cost 2^-20).
__device__ __forceinline__ float exp_scaled(float d, const Scale& c) {
  const float x = d * c.hi;
  const float rest = fmaf(d, c.hi, -x) + d * c.lo;
  const float y = ex2(x);
  return y > 0.f ? fmaf(y, rest * 0.6931472f, y) : y;  // y = 0: d may be infinite, and the rest NaN
}

// A number as the sum of two floats, for the last steps of a row, where differences
// of logarithms of some 10 in size have to be good to 2^-24 of a result near 0. Sums by
// Knuth's two-sum, products by a fused multiply-add's rest.
// (float64 would do, at a 64th of float32's rate on this GPU.) Where h is infinite l
// may be NaN: value() takes h alone then.
struct Two {
  float h, l;
  __device__ float value() const { return fabsf(h) <= FLT_MAX ? h + l : h; }
};
__device__ __forceinline__ Two sum_of(float a, float b) {  // exact
  const float s = a + b, t = s - a;
  return Two{s, (a - (s - t)) + (b - t)};
}
__device__ __forceinline__ Two operator+(Two a, Two b) {
  Two s = sum_of(a.h, b.h);
  s.l += a.l + b.l;
  return s;
}
__device__ __forceinline__ Two operator-(Two a, Two b) { return a + Two{-b.h, -b.l}; }
__device__ __forceinline__ Two operator*(Two a, float f) {
  const float p = a.h * f;
  return Two{p, fmaf(a.h, f, -p) + a.l * f};
}
__device__ __forceinline__ Two in_temperatures(Two d, const Scale& c) {  // d / temperature
  Two x = d * c.inv;
  x.l += d.h * c.inv_lo;
  return x;
}
// (z - top) / temperature where the difference is beyond float32's range, which the division may bring back.
inline __device__ __noinline__ double far_in_temperatures(float z, float top, const Scale& c) {
  return ((double)z - top) * ((double)c.inv + c.inv_lo);
}
__device__ __forceinline__ Two warp_sum_two(Two v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = v + Two{__shfl_xor_sync(kFull, v.h, o), __shfl_xor_sync(kFull, v.l, o)};
  return v;
}
// Logarithm of a sum (a normal number, 0 or not finite): of its exponent, e ln 2 with ln 2
// in two parts (Cody and Waite: the first with 16 bits, so that the product is exact),
// and of the rest, in [0.71, 1.42). Out of line, like all that runs once a row: the code
// of the row's ends would otherwise push the loops out of the instruction cache.
inline __device__ __noinline__ Two log_of(float s) {
  if (!(s > 0.f) || !(s <= FLT_MAX)) return Two{s == 0.f ? -INFINITY : s, 0.f};
  const int bits = __float_as_int(s), e = (bits - 0x3f3504f3) >> 23;
  constexpr float kHi = 0.693145751953125f, kLo = 1.4286068203094173e-06f;
  return sum_of(e * kHi, logf(__int_as_float(bits - (e << 23)))) + Two{0.f, e * kLo};
}
// exp of a two-float number.
__device__ __forceinline__ float exp_of(Two x) {
  const float y = expf(x.h);
  return y > 0.f && y <= FLT_MAX ? fmaf(y, x.l, y) : y;
}

// ---- sums of exponentials --------------------------------------------------------------------------

// Sums over some entries relative to m, which is near the largest of them, top:
// s = sum 2^x, u = sum 2^x x, x = (z - m) c. No entry: m = top = -inf, s = u = 0. A NaN
// or +inf among the entries makes s NaN.
struct Sums {
  float m, s, u, top;
};
__device__ __forceinline__ Sums no_sums() { return Sums{-INFINITY, 0.f, 0.f, -INFINITY}; }

// Joined over each kLanes neighbouring lanes of a warp; every one of them gets the result.
template <int kLanes, bool kEntropy> __device__ __forceinline__ Sums join_lanes(Sums a, float c) {
  float m = a.m;
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) {
    m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
    a.top = fmaxf(a.top, __shfl_xor_sync(kFull, a.top, o));
  }
  // without an entry s is 0 (or NaN, which stays); capped, since 0 times -inf is NaN
  const float d = a.m == m ? 0.f : fmaxf((a.m - m) * c, -1e4f);
  const float f = ex2(d);
  if (kEntropy) a.u = (a.u + d * a.s) * f;
  a.s *= f;
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) {
    a.s += __shfl_xor_sync(kFull, a.s, o);
    if (kEntropy) a.u += __shfl_xor_sync(kFull, a.u, o);
  }
  a.m = m;
  return a;
}

// Exponents relative to a value m, the same for a warp. As one fused multiply-add,
// z c - R with R = m c rounded, while |R| is below 2^16; the factor 2^(R - m c) by which
// the results are then off is given back at the end (rest). Beyond that (z - m) c: z c
// may overflow, or R be off by whole exponents.
struct Ref {
  float m, R;
  bool slow;
  __device__ void set(float ref, float c) {
    m = ref;
    R = ref * c;
    slow = !(fabsf(R) < 65536.f);
  }
  __device__ float rest(float c) const { return slow ? 0.f : fmaf(m, c, -R); }  // m c - R
  __device__ float2 operator()(float2 z, float c) const {
    const float2 cc = make_float2(c, c);
    return slow ? mul2(add2(z, make_float2(-m, -m)), cc) : fma2(z, cc, make_float2(-R, -R));
  }
};

// A warp's running sums.
template <typename T, bool kEntropy, int kN, int kStride> struct Acc {
  Ref ref;
  float limit, s, u, top;  // limit: a larger entry moves the reference; s, u, top are the lane's
  bool set, masked;
  __device__ void clear() {
    ref.m = ref.R = 0.f;
    ref.slow = set = masked = false;
    limit = -INFINITY;
    s = u = 0.f;
    top = -INFINITY;
  }
  template <bool kAll, bool kMasked>
  __device__ __forceinline__ void terms(const uint4 (&q)[kN], int at, int n, float c, float& s_out, float& u_out) const {
    float2 s2 = make_float2(0.f, 0.f), u2 = s2;
    const float2 cc = make_float2(c, c), nR = make_float2(-ref.R, -ref.R);
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      if (!kAll && i * kStride + at >= n) break;
#pragma unroll
      for (int w = 0; w < El<T>::kVec / 2; ++w) {
        const float2 x = fma2(pair_of<T>(q[i], w), cc, nR);
        const float2 e = make_float2(ex2(x.x), ex2(x.y));
        s2 = add2(s2, e);
        // an exponent of -inf counts as -10^4: the product is 0, not NaN
        if (kEntropy) u2 = fma2(e, kMasked ? make_float2(fmaxf(x.x, -1e4f), fmaxf(x.y, -1e4f)) : x, u2);
      }
    }
    s_out = s2.x + s2.y;
    u_out = u2.x + u2.y;
  }
  // The vectors again, in shared memory, for references beyond the fast form.
  static __device__ __noinline__ float2 slow_terms(const uint4* v, int at, int n, float m, float c) {
    float s = 0.f, u = 0.f;
    const T* e = reinterpret_cast<const T*>(v);
    for (int i = at; i < n; i += kStride)
      for (int h = 0; h < El<T>::kVec; ++h) {
        const float x = (up(e[i * El<T>::kVec + h]) - m) * c, t = ex2(x);
        s += t;
        u = fmaf(t, fmaxf(x, -1e4f), u);
      }
    return make_float2(s, u);
  }
  // Vectors v[at], v[at + kStride], ... below n, kN at most, in shared memory.
  __device__ __forceinline__ void add(const uint4* v, int at, int n, float c) {
    if (!kEntropy && n == kN * kStride) add_some<true>(v, at, n, c);  // without a branch per vector
    else add_some<false>(v, at, n, c);
  }
  template <bool kAll> __device__ __forceinline__ void add_some(const uint4* v, int at, int n, float c) {
    uint4 q[kN];
    float t = -INFINITY;
#pragma unroll
    for (int i = 0; i < kN; ++i)
      if (kAll || i * kStride + at < n) {
        q[i] = v[i * kStride + at];
        if (!kAll) t = fmaxf(t, vec_max<T>(q[i]));
      }
    if (kAll) t = vecs_max<T>(q);
    if (__any_sync(kFull, t > limit)) move(t, c);
    top = fmaxf(top, t);
    float sc, uc;
    if (ref.slow) {
      const float2 r = slow_terms(v, at, n, ref.m, c);
      sc = r.x;
      uc = r.y;
    } else if (!kEntropy || !masked) {
      terms<kAll, false>(q, at, n, c, sc, uc);
      if (kEntropy && __any_sync(kFull, uc != uc)) {  // an entry of -inf: masked from here on
        masked = true;
        terms<kAll, true>(q, at, n, c, sc, uc);
      }
    } else {
      terms<kAll, true>(q, at, n, c, sc, uc);
    }
    s += sc;
    u += uc;
  }
  // The reference becomes the largest of the lanes' t. In the fast form the sums are relative to R, which is off
  // from m c by rest(), up to 2^-9; in the slow one to m c itself.
  __device__ __forceinline__ void move(float t, float c) {
    const float m = warp_max(t);
    const Ref old = ref;
    ref.set(m, c);
    if (set) {
      const float d = old.slow || ref.slow ? fmaxf((old.m - m) * c - old.rest(c) + ref.rest(c), -1e4f) : old.R - ref.R;
      const float f = ex2(d);
      u = (u + d * s) * f;
      s *= f;
    }
    set = true;
    limit = m + 4.f / c;  // sums relative to a value at most 4 bits below the largest
  }
  __device__ Sums total(float c) const {
    const float rest = ref.rest(c), f = ex2(-rest);
    Sums a;
    a.s = warp_sum(s);
    a.u = kEntropy ? (warp_sum(u) - rest * a.s) * f : 0.f;
    a.s *= f;
    a.m = set ? ref.m : -INFINITY;
    a.top = warp_max(top);
    return a;
  }
};

// Sums over single entries, one a lane where `on`.
template <bool kEntropy> __device__ __forceinline__ Sums lane_sums(float z, bool on, float c) {
  Sums a;
  a.m = a.top = warp_max(on ? z : -INFINITY);
  const float x = on ? (z - (a.m == -INFINITY ? 0.f : a.m)) * c : -INFINITY, e = ex2(x);
  a.s = warp_sum(e);
  a.u = kEntropy ? warp_sum(e * fmaxf(x, -1e4f)) : 0.f;
  return a;
}

// ---- the order of alternatives ---------------------------------------------------------------------

// Larger value first, then lower index; -0 and +0 are equal. The key of a valid entry is never 0.
__device__ __forceinline__ uint32_t order_bits(float v) {
  const uint32_t b = __float_as_uint(v + 0.f);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float bits_value(uint32_t o) {
  return __uint_as_float((o & 0x80000000u) ? (o & 0x7fffffffu) : ~o);
}
__device__ __forceinline__ unsigned long long order_key(float v, int j) {
  return ((unsigned long long)order_bits(v) << 32) | (uint32_t)~j;
}
__device__ __forceinline__ float key_value(unsigned long long key) { return bits_value((uint32_t)(key >> 32)); }
__device__ __forceinline__ int key_index(unsigned long long key) { return (int)~(uint32_t)key; }

// A value of the order that at least k of a warp's 32 * kN numbers reach, near the k-th
// largest. (Of maxima of disjoint entries it is a lower bound of the k-th largest entry.)
// o: order_bits; absent numbers are 0. For small k the k-th of the lanes' maxima, a
// third of the way further down, but found at once (400 cycles against 4,000); else by
// bisection until no more than 1.25 k are above.
template <int kN> __device__ __forceinline__ uint32_t kth_bits(const uint32_t (&o)[kN], int k) {
  uint32_t hi = 0;
#pragma unroll
  for (int i = 0; i < kN; ++i) hi = max(hi, o[i]);
  if (k <= 24) {
    const int lane = threadIdx.x & 31;
    int at = 0;  // lanes before this one: a larger number, or as large at a lower lane
#pragma unroll 8
    for (int l = 0; l < 32; ++l) {
      const uint32_t v = __shfl_sync(kFull, hi, l);
      at += v > hi || (v == hi && l < lane);
    }
    return __shfl_sync(kFull, hi, __ffs(__ballot_sync(kFull, at == k - 1)) - 1);
  }
  uint32_t lo = 0;
  hi = __reduce_max_sync(kFull, hi);
  while (lo < hi) {
    const uint32_t mid = lo + (hi - lo) / 2 + 1;
    int n = 0;
#pragma unroll
    for (int i = 0; i < kN; ++i) n += o[i] >= mid;
    n = __reduce_add_sync(kFull, n);
    if (n < k) hi = mid - 1;
    else lo = mid;
    if (n >= k && n <= k + k / 4) break;
  }
  return lo;
}

// ---- candidates for the best alternatives ----------------------------------------------------------

constexpr int kCand = 96;  // of a warp

// What the warps that look for a row's candidates share.
struct Cut {
  unsigned long long key;  // one that at least k entries reach
  unsigned begun, ended;   // compactions so far: while one is under way a candidate may be seen in two places
};

// Leaves the warp's k best candidates and raises the cut to the least of them. For rows
// whose candidates do not fit: many entries are equal, or each chunk is above the last;
// no entry is lost, as the cut is a key (value and index).
inline __device__ __noinline__ int compact(unsigned long long* cand, Cut* cut, int k) {
  const int lane = threadIdx.x & 31;
  unsigned long long key[kCand / 32];
  __syncwarp();
#pragma unroll
  for (int i = 0; i < kCand / 32; ++i) key[i] = cand[i * 32 + lane];
  unsigned long long lo = 1, hi = ~0ull;  // at least k keys (or all) reach lo
  while (lo < hi) {
    const unsigned long long mid = lo + (hi - lo) / 2 + 1;
    int n = 0;
#pragma unroll
    for (int i = 0; i < kCand / 32; ++i) n += key[i] >= mid;
    n = __reduce_add_sync(kFull, n);
    if (n >= k) lo = mid;
    else hi = mid - 1;
    if (n == k) break;
  }
  if (lane == 0) {
    atomicMax(&cut->key, lo);
    atomicAdd(&cut->begun, 1u);
  }
  __threadfence_block();
  int n = 0;
  __syncwarp();
#pragma unroll
  for (int i = 0; i < kCand / 32; ++i) cand[i * 32 + lane] = 0;
  __syncwarp();
#pragma unroll
  for (int i = 0; i < kCand / 32; ++i) {
    const bool on = key[i] >= lo;
    const uint32_t ons = __ballot_sync(kFull, on);
    if (on) cand[n + __popc(ons & ((1u << lane) - 1))] = key[i];
    n += __popc(ons);
  }
  __threadfence_block();
  __syncwarp();
  if (lane == 0) atomicAdd(&cut->ended, 1u);
  return n;
}

// Raises the cut to nearly the k-th of kN candidates' values. One warp; others may add candidates
// meanwhile (one not yet written is 0). Where one moved its candidates meanwhile, which may have been
// seen twice and made the k-th too high, the cut stays.
template <int kN> __device__ __noinline__ void raise_cut(const unsigned long long* cand, Cut* cut, int k) {
  const int lane = threadIdx.x & 31;
  uint32_t o[kN / 32];
  const unsigned ended = __shfl_sync(kFull, *(volatile unsigned*)&cut->ended, 0);
  __threadfence_block();
  __syncwarp();
#pragma unroll
  for (int i = 0; i < kN / 32; ++i) o[i] = (uint32_t)(((const volatile unsigned long long*)cand)[i * 32 + lane] >> 32);
  __threadfence_block();
  __syncwarp();
  const unsigned begun = __shfl_sync(kFull, *(volatile unsigned*)&cut->begun, 0);
  if (begun != ended) return;
  const uint32_t bits = kth_bits(o, k);
  if (lane == 0) atomicMax(&cut->key, (unsigned long long)bits << 32);
}

// Whether a vector has an entry that reaches `value`, any float: rounded to the type, up or down, it passes over no
// entry that does (rounded up, it is the least of the type's numbers above it), and scan_hits compares keys exactly.
template <typename T> __device__ __forceinline__ bool reaches(const uint4& q, float value);
template <> __device__ __forceinline__ bool reaches<float>(const uint4& q, float value) { return vec_max<float>(q) >= value; }
template <> __device__ __forceinline__ bool reaches<bf16>(const uint4& q, float value) {
  auto h = [](const uint32_t& u) { return *reinterpret_cast<const __nv_bfloat162*>(&u); };
  const __nv_bfloat162 m = __hmax2(__hmax2(h(q.x), h(q.y)), __hmax2(h(q.z), h(q.w)));
  return __hge2_mask(m, __float2bfloat162_rn(value)) != 0;
}
template <> __device__ __forceinline__ bool reaches<__half>(const uint4& q, float value) {
  auto h = [](const uint32_t& u) { return *reinterpret_cast<const __half2*>(&u); };
  const __half2 m = __hmax2(__hmax2(h(q.x), h(q.y)), __hmax2(h(q.z), h(q.w)));
  return __hge2_mask(m, __float2half2_rn(value)) != 0;
}
// The least value to look for: the cut's, or the least finite one.
template <typename T> __device__ __forceinline__ float cut_value(unsigned long long cut) {
  const float low = sizeof(T) == 4 ? -FLT_MAX : std::is_same_v<T, bf16> ? -3.38953139e38f : -65504.f;
  return cut ? fmaxf(key_value(cut), low) : low;
}

// One warp: the entries of some vectors that reach the cut become candidates; returns
// how many there are then. Bit i of the lane's hits: vector i * stride + first + lane of
// `chunk` has one; entry: the index of the chunk's first.
template <typename T>
__device__ __forceinline__ int scan_hits(const T* chunk, uint32_t hits, int stride, int first, int64_t entry,
                                         unsigned long long* cand, int n_cand, Cut* shared_cut, int k) {
  constexpr int kVec = El<T>::kVec;
  const int lane = threadIdx.x & 31;
  unsigned long long cut = *(volatile unsigned long long*)&shared_cut->key;
#pragma unroll 1
  for (uint32_t all; (all = __ballot_sync(kFull, hits != 0)) != 0;) {
    // one vector of each of the first 4 or 8 lanes that have some, one entry a lane
    uint32_t left = all;
    int src = -1;
#pragma unroll
    for (int q = 0; q < 32 / kVec; ++q) {
      if (lane / kVec == q) src = __ffs(left) - 1;
      left &= left - 1;
    }
    const int i = __shfl_sync(kFull, __ffs(hits) - 1, max(src, 0));
    const int at = (i * stride + first + src) * kVec + lane % kVec;
    const float val = src >= 0 ? up(chunk[at]) : -INFINITY;
    const unsigned long long key = order_key(val, (int)entry + at);
    const bool on = val > -INFINITY && key >= cut;
    const uint32_t ons = __ballot_sync(kFull, on);
    if (n_cand + __popc(ons) > kCand) {  // no room: again after making some (k + 32 <= kCand)
      n_cand = compact(cand, shared_cut, k);
      cut = *(volatile unsigned long long*)&shared_cut->key;
      continue;
    }
    if (on) cand[n_cand + __popc(ons & ((1u << lane) - 1))] = key;
    n_cand += __popc(ons);
    if ((all & ~left) >> lane & 1) hits &= hits - 1;
  }
  return n_cand;
}

// One warp: of kN candidates (0: none) those that can be among the k best to the front of the array: the ones that
// reach `cut` and nearly the k-th of them. Returns how many.
template <int kN> __device__ __forceinline__ int keep_best(unsigned long long* cand, unsigned long long cut, int k) {
  const int lane = threadIdx.x & 31;
  unsigned long long key[kN / 32];
  uint32_t o[kN / 32];
#pragma unroll
  for (int i = 0; i < kN / 32; ++i) {
    key[i] = cand[i * 32 + lane];
    o[i] = (uint32_t)(key[i] >> 32);
  }
  cut = max(max((unsigned long long)kth_bits(o, k) << 32, cut), 1ull);
  __syncwarp();
  int n = 0;
#pragma unroll
  for (int i = 0; i < kN / 32; ++i) {
    const uint32_t ons = __ballot_sync(kFull, key[i] >= cut);
    if (key[i] >= cut) cand[n + __popc(ons & ((1u << lane) - 1))] = key[i];
    n += __popc(ons);
  }
  __syncwarp();
  return n;
}

// One warp: f(place, key) for the k best of n candidates; an entry's place is the number of entries before it
// (keys are distinct).
template <typename F> __device__ __forceinline__ void rank_best(const unsigned long long* cand, int n, int k, F f) {
#pragma unroll 1
  for (int i = threadIdx.x & 31; i < n; i += 32) {
    const unsigned long long key = cand[i];
    int at = 0;
#pragma unroll 4
    for (int o = 0; o < n; ++o) at += cand[o] > key;
    if (at < k) f(at, key);
  }
}

// ---- token log probabilities: a row's last steps ---------------------------------------------------

// From a row's sums: log probabilities are (z - top) / temperature - log_s.
struct Answer {
  float top, all;
  Two log_s;
  bool good;  // false for all -inf, a NaN or a +inf
  __device__ Answer(const Sums& p, const Scale& c) {
    top = p.top;
    all = p.s * exp_scaled(p.m - p.top, c);
    good = all > 0.f && all <= FLT_MAX;
    log_s = log_of(all);
  }
  __device__ float logprob(float z, const Scale& c) const {
    const Two away = sum_of(z, -top);
    if (away.h == -INFINITY && z != -INFINITY) return far_in_temperatures(z, top, c);  // log_s is below its last bit
    return (in_temperatures(away, c) - log_s).value();
  }
};

__device__ __forceinline__ void store_answer(const TokenLogprobs& t, int64_t row, const Answer& a, const Sums& p, int tok,
                                             float zt, int vocab, const Scale& c) {
  if (t.logprob)
    t.logprob[row] = tok == -1 ? 0.f : a.good && tok >= 0 && tok < vocab ? a.logprob(zt, c) : NAN;
  // -sum q log q = log_s - sum q x ln 2 with x relative to the largest entry: u / s, moved by (m - top) c
  if (t.entropy)
    t.entropy[row] = a.good ? (a.log_s - Two{(p.u / p.s + (p.m - p.top) * c.hi) * 0.6931472f, 0.f}).value() : NAN;
  if (t.lse) t.lse[row] = a.good ? (in_temperatures(Two{a.top, 0.f}, c) + a.log_s).value() : NAN;
}

// ---- distillation ----------------------------------------------------------------------------------

// A row's teacher: entries 0..k-1 that count (an index twice counts the first
// time), their probabilities and log probabilities, what they leave to the other
// tokens (pt), and the student's logits of them.
struct Teacher {
  int idx[kMaxTeacher];  // -1: absent
  float lp[kMaxTeacher];
  float p[kMaxTeacher];
  float z[kMaxTeacher];
  float e[kMaxTeacher];  // 2^((z - zmax) c)
  float zmax, esum;      // over the entries that count
  float sum, pt;
  int any, broken;
};

// Marks of tokens (by 14 bits of a hash), all clear between uses: two entries that share
// one may be the same token. Looking each of 64 entries up among all others instead
// costs some 4,000 cycles, most of a row's time; one row in eight still does it.
struct Marks {
  static constexpr int kWords = 512;
  uint32_t w[kWords];
  static __device__ int of(int idx) { return (int)((uint32_t)idx * 2654435769u >> 18); }
};

// One warp; lane l brings entries l and l + 32 (idx -1 where there is none) and the
// student's logits of them. Entries of -1 are absent; any other index outside the vocabulary, and a log probability that is NaN
// or whose exponential is not finite, break the row.
inline __device__ __noinline__ void load_teacher(Teacher& t, Marks& marks, const Distill& d, const int (&idx)[2], const float (&raw)[2], const float (&zv)[2],
                             int vocab, const Scale& c) {
  const int lane = threadIdx.x & 31;
  bool on[2], bad = false;
  float lp[2], e[2], mx = -INFINITY;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    bad |= idx[h] < -1 || idx[h] >= vocab;
    on[h] = idx[h] >= 0 && idx[h] < vocab;
    t.idx[lane + 32 * h] = idx[h];
  }
  __syncwarp();
  bool again[2] = {false, false}, shared = false;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int m = Marks::of(idx[h]);
    if (on[h]) shared |= atomicOr(&marks.w[m / 32], 1u << m % 32) >> m % 32 & 1;
  }
  shared = __any_sync(kFull, shared);
#pragma unroll
  for (int h = 0; h < 2; ++h)
    if (on[h]) marks.w[Marks::of(idx[h]) / 32] = 0;
  if (shared) {
#pragma unroll 1
    for (int q = 0; q < d.k; ++q) {
      const int j = t.idx[q];
      again[0] |= j == idx[0] && q < lane;
      again[1] |= j == idx[1] && q < lane + 32;
    }
  }
  __syncwarp();
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    on[h] = on[h] && !again[h];
    lp[h] = on[h] ? raw[h] : -INFINITY;
    bad |= !(lp[h] < INFINITY);
    mx = fmaxf(mx, lp[h]);
  }
  mx = warp_max(mx);
  const float zmax = warp_max(fmaxf(on[0] ? zv[0] : -INFINITY, on[1] ? zv[1] : -INFINITY));
  const float base = d.tail || mx == -INFINITY ? 0.f : mx;
  const float p[2] = {expf(lp[0] - base), expf(lp[1] - base)};
  const Two two = warp_sum_two(sum_of(p[0], p[1]));
  const float sum = two.value();
  bad |= !(sum <= FLT_MAX);
#pragma unroll
  for (int h = 0; h < 2; ++h)  // zmax = -inf: every entry is -inf or NaN
    e[h] = !on[h] ? 0.f : zmax == -INFINITY ? (zv[h] == zv[h] ? 0.f : zv[h]) : exp_scaled(zv[h] - zmax, c);
  const float esum = warp_sum(e[0] + e[1]);
  const bool any = __any_sync(kFull, on[0] || on[1]);
  bad = __any_sync(kFull, bad);
  const bool scaled = !d.tail && sum > 0.f;
  const Two log_norm = scaled ? log_of(sum) + Two{0.f, two.l / sum} : Two{0.f, 0.f};
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int i = lane + 32 * h;
    t.idx[i] = on[h] ? idx[h] : -1;
    t.lp[i] = scaled ? (sum_of(lp[h], -base) - log_norm).value() : lp[h];
    t.p[i] = scaled ? p[h] / sum : p[h];
    t.z[i] = zv[h];
    t.e[i] = e[h];
  }
  if (lane == 0) {
    t.zmax = zmax;
    t.esum = esum;
    t.pt = d.tail ? fmaxf(0.f, (1.f - two.h) - two.l) : 0.f;
    t.sum = d.tail ? sum : sum > 0.f ? 1.f : 0.f;
    t.any = any;
    t.broken = bad;
  }
  __syncwarp();
}

// What a row's gradient is made of: of an unlisted entry coef 2^((z - ref) c), of the listed ones g[]. Unlisted
// entries are (w q's share - p_t / q_t's) relative to their own maximum, one exponential each, so that a row whose
// unlisted tokens are all far down keeps their share.
struct Coef {
  Ref ref;
  float coef;
  int zero;  // the row gets zeros whatever it holds
  float g[kMaxTeacher];
  __device__ void put(float r, float k, bool z, float c) {
    ref.set(r, c);
    coef = k * ex2(-ref.rest(c));
    zero = z;
  }
  __device__ __forceinline__ float at(float z, float c) const { return ex2(ref(make_float2(z, z), c).x) * coef; }
};

// A row's student from the sums over its unlisted entries and its teacher.
struct Student {
  float mu, su;    // largest unlisted entry, sum relative to it
  float top, all;  // of all entries
  float far_u, far_l;  // 2^((mu - top) c), 2^((zmax - top) c)
  bool good, others;
  __device__ Student(const Sums& p, const Teacher& t, const Distill& d, const Scale& c) {
    mu = p.top;
    su = p.s * (mu == -INFINITY ? 1.f : exp_scaled(p.m - mu, c));  // a NaN stays
    top = fmaxf(mu, t.zmax);
    far_u = mu == -INFINITY ? 0.f : exp_scaled(mu - top, c);
    far_l = t.zmax == -INFINITY ? 0.f : exp_scaled(t.zmax - top, c);
    all = su * (mu == -INFINITY ? 1.f : far_u) + t.esum * (t.zmax == -INFINITY ? 1.f : far_l);
    good = all > 0.f && all <= FLT_MAX && !t.broken;
    others = d.tail && (mu - top) * c.inv >= kNoTail;  // false where both are -inf
  }
};

// One warp: the gradient's coefficients (whoever reads them waits).
__device__ __forceinline__ void store_coef(Coef& x, const Student& s, const Teacher& t, float gr, const Scale& c) {
  const int lane = threadIdx.x & 31;
  const float pt = s.others ? t.pt : 0.f, w = (t.sum + pt) / s.all, gt = gr * c.inv;
  const float bad = s.good ? 0.f : NAN;
  if (lane == 0)
    x.put(s.mu == -INFINITY ? 0.f : s.mu, gt * (w * s.far_u - (pt > 0.f ? pt / s.su : 0.f)) + bad,
          gr == 0.f || (!t.any && !t.broken), c.hi);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int i = lane + 32 * h;
    x.g[i] = gt * (w * s.far_l * t.e[i] - t.p[i]) + bad;
  }
}

// One warp: the coefficients from the sums that the loss left.
__device__ __forceinline__ void store_coef(Coef& x, const float* stats, const Teacher& t, const Distill& d, float gr,
                                           const Scale& c) {
  const int lane = threadIdx.x & 31;
  const float top = stats[0], log_s = stats[1], mu = stats[2], log_u = stats[3];
  const bool others = d.tail && mu != -INFINITY;
  const float pt = others ? t.pt : 0.f, w = t.sum + pt, gt = gr * c.inv, bad = t.broken ? NAN : 0.f;
  auto q = [&](float z) { return exp_of(in_temperatures(sum_of(z, -top), c) - Two{log_s, 0.f}); };
  if (lane == 0)
    x.put(others ? mu : top, gt * (w * (others ? q(mu) : expf(-log_s)) - (pt > 0.f ? pt * expf(-log_u) : 0.f)) + bad,
          gr == 0.f || (!t.any && !t.broken), c.hi);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int i = lane + 32 * h;
    x.g[i] = gt * (w * q(t.z[i]) - t.p[i]) + bad;
  }
}

// One warp: the row's loss and the sums for the gradient.
__device__ __forceinline__ void store_loss(const Distill& d, int64_t row, const Student& s, const Teacher& t, const Scale& c) {
  const int lane = threadIdx.x & 31;
  const Two log_s = log_of(s.all), log_u = log_of(s.su);
  Two loss{0.f, 0.f};
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int i = lane + 32 * h;
    if (t.p[i] > 0.f && t.idx[i] >= 0) {
      const Two away = in_temperatures(sum_of(t.z[i], -s.top), c);
      if (away.h == -INFINITY && t.z[i] != -INFINITY)  // beyond float's range, but a small p may bring it back
        loss = loss + Two{(float)(-far_in_temperatures(t.z[i], s.top, c) * t.p[i]), 0.f};
      else
        loss = loss + (Two{t.lp[i], 0.f} - (away - log_s)) * t.p[i];
    }
  }
  loss = warp_sum_two(loss);
  if (t.pt > 0.f && s.others)
    loss = loss + (log_of(t.pt) - (in_temperatures(sum_of(s.mu, -s.top), c) + log_u - log_s)) * t.pt;
  if (lane == 0) {
    d.loss[row] = t.broken ? NAN : !t.any ? 0.f : s.good ? loss.value() : NAN;
    float* out = d.stats + 4 * row;
    if (!d.stats) return;
    out[0] = s.good ? s.top : NAN;
    out[1] = s.good ? log_s.value() : NAN;
    out[2] = !s.good ? NAN : s.others ? s.mu : d.tail ? -INFINITY : 0.f;
    out[3] = !s.good ? NAN : s.others ? log_u.value() : 0.f;
  }
}

// Gradient entries of one vector of logits, as words to store.
template <typename T> __device__ __forceinline__ uint4 grad_vec(const uint4& q, const Ref& ref, float coef, bool zero, float c) {
  const float2 kk = make_float2(coef, coef);
  uint32_t out[4];
#pragma unroll
  for (int w = 0; w < El<T>::kVec / 2; ++w) {
    const float2 x = ref(pair_of<T>(q, w), c);
    float2 g = mul2(make_float2(ex2(x.x), ex2(x.y)), kk);
    if (zero) g = make_float2(0.f, 0.f);
    if constexpr (sizeof(T) == 4) {
      out[2 * w] = __float_as_uint(g.x);
      out[2 * w + 1] = __float_as_uint(g.y);
    } else {
      out[w] = pack<T>(g);
    }
  }
  return make_uint4(out[0], out[1], out[2], out[3]);
}
// Entry by entry, for gradients that start at another offset from a 16-byte boundary than the logits.
template <typename T> __device__ __forceinline__ void store_unaligned(T* p, const uint4& q) {
#pragma unroll
  for (int h = 0; h < El<T>::kVec; ++h) {
    if constexpr (sizeof(T) == 4) *reinterpret_cast<uint32_t*>(p + h) = word_of(q, h);
    else *reinterpret_cast<uint16_t*>(p + h) = (uint16_t)(word_of(q, h / 2) >> (h % 2 * 16));
  }
}

// ---- rows ------------------------------------------------------------------------------------------

constexpr int kEdges = 16;

// A row: `head` entries before the first 16-byte boundary, nb whole vectors, the rest
// after them; both ends, the edges, are read entry by entry.
template <typename T> struct Row {
  const T* row;
  int head, nb, n;
  __device__ Row(const void* z, int64_t ld, int64_t r, int vocab) {
    row = reinterpret_cast<const T*>(z) + r * ld;
    n = vocab;
    head = min(n, (int)((16 - reinterpret_cast<uintptr_t>(row) % 16) % 16 / sizeof(T)));
    nb = (n - head) / El<T>::kVec;
  }
  __device__ int64_t entry(int vec) const { return head + (int64_t)vec * El<T>::kVec; }
  // The entry of edge place 0..15 (8 before, 8 after the whole vectors), -1: none.
  __device__ int edge(int place) const {
    const int64_t j = place < 8 ? place : entry(nb) + place - 8;
    return place < 8 ? (place < head ? place : -1) : j < n ? (int)j : -1;
  }
};

template <typename F> cudaError_t by_type(int dtype, F f) {
  if (dtype == EAGLE_DTYPE_BF16) return f(bf16{});
  if (dtype == EAGLE_DTYPE_F16) return f(__half{});
  return f(float{});
}

inline Scale scale_of(float temperature) {
  const double inv = 1.0 / temperature, c = 1.4426950408889634074 / temperature;
  Scale s;
  s.inv = (float)inv;
  s.inv_lo = (float)(inv - s.inv);
  s.hi = (float)c;
  s.lo = (float)(c - s.hi);
  return s;
}

enum Mode { kLogprobs, kLoss, kStep, kGrad };

struct Args {
  VocabRows r;
  TokenLogprobs t;
  Distill d;
  Scale c;
  // long rows: blocks a row; units, whose sums are joined, of a row and of a block; vectors of a unit
  int C, units, mine, unit;
  unsigned long long wait_ns;  // limit of a wait
};

// The results of a row of a call whose kernel gave up a wait: NaN (index -1), by `threads` threads.
template <typename T, int kMode> __device__ __noinline__ void no_results(const Args& a, int64_t row, int thread, int threads) {
  if constexpr (kMode == kLogprobs) {
    if (thread == 0) {
      if (a.t.logprob) a.t.logprob[row] = NAN;
      if (a.t.entropy) a.t.entropy[row] = NAN;
      if (a.t.lse) a.t.lse[row] = NAN;
    }
#pragma unroll 1
    for (int i = thread; i < a.t.k; i += threads) {
      a.t.idx[row * a.t.k + i] = -1;
      a.t.val[row * a.t.k + i] = NAN;
    }
  } else {
    if (kMode != kGrad && thread == 0) {
      a.d.loss[row] = NAN;
      for (int i = 0; a.d.stats && i < 4; ++i) a.d.stats[4 * row + i] = NAN;
    }
    if constexpr (kMode != kLoss)
#pragma unroll 1
      for (int64_t j = thread; j < a.r.vocab; j += threads) (reinterpret_cast<T*>(a.d.dz) + row * a.d.ld_dz)[j] = down<T>(NAN);
  }
}

constexpr int kShortRow = 16 << 10;  // bytes of a row that one warp does by itself
cudaError_t short_rows(const Args& a, int mode, cudaStream_t s);

}  // namespace vocab
}  // namespace eg
