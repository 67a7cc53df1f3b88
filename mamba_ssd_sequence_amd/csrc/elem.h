// Device helpers of the per-channel kernels (gated_scan.hip, norms.hip): the
// logistic function, and pieces of rows as they are stored.
#pragma once

#include "common.h"

#include <type_traits>

namespace ssd {

// e^x to (|x| + 3) roundings: 2^(x log2 e) on the hardware exponential (1 ulp),
// whose argument is rounded once.  Infinities and NaN come out as e^x has them.
// (Putting that rounding back to first order costs 4 more instructions; the
// error it leaves is that of terms which e^{-|x|} has made small.)
__device__ __forceinline__ float exp_fast(float x) { return exp2_fast(x * LOG2E); }

// sigmoid(x) and 1 - sigmoid(x) = sigmoid(-x).  The smaller of the two is
// e / (1 + e) with e = e^{-|x|} and has its own relative accuracy; the larger
// is one minus it, a single rounding: a decay near 1 is then right to half an
// ulp, without the bias of a reciprocal that a thousand tokens would add up.
__device__ __forceinline__ void sigmoid_pair(float x, float& s, float& rest) {
  const float e = exp_fast(-fabsf(x));
  const float small = e * __builtin_amdgcn_rcpf(1.f + e);
  const float large = 1.f - small;
  s = x > 0.f ? large : small;
  rest = x > 0.f ? small : large;
}

// sigmoid(x) alone: 1 / (1 + e^{-x}), to a few roundings at either end (below
// x = -88, where the result is under 1e-38, it is 0).
__device__ __forceinline__ float sigmoid_v(float x) {
  return __builtin_amdgcn_rcpf(1.f + exp_fast(-x));
}

// Nontemporal accesses (NT), for arrays that pass through once: they leave the
// caches to what is used again.
template <bool NT, typename P>
__device__ __forceinline__ P load_as(const void* p) {
  const P* q = static_cast<const P*>(p);
  if constexpr (NT) return __builtin_nontemporal_load(q);
  return *q;
}

template <bool NT, typename P>
__device__ __forceinline__ void store_as(void* p, P v) {
  P* q = static_cast<P*>(p);
  if constexpr (NT) {
    __builtin_nontemporal_store(v, q);
  } else {
    *q = v;
  }
}

// f(true_type) or f(false_type): two copies of a group of accesses, kept from
// being merged (which would drop the nontemporal ones' mark) by the empty asm
template <typename F>
__device__ __forceinline__ void either(bool c, F&& f) {
  if (c) {
    asm volatile("");
    f(std::true_type{});
    asm volatile("");
  } else {
    f(std::false_type{});
  }
}

// Element e of an array, by a 32-bit byte offset from a uniform address (less
// than 2^32 bytes): the offset then needs one register and no 64-bit sum.
template <typename T>
__device__ __forceinline__ T* element(T* p, unsigned e) {
  typedef typename std::conditional<std::is_const<T>::value, const char, char>::type byte;
  return reinterpret_cast<T*>(reinterpret_cast<byte*>(p) + e * (unsigned)sizeof(T));
}

// Pieces of 4 elements, at the alignment of one: rows of any width are read and
// written in whole pieces (the hardware takes them at any element's address).
typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
typedef u32x2 u32x2_any __attribute__((aligned(2)));
typedef bf16x4 bf16x4_any __attribute__((aligned(2)));
typedef f32x4 f32x4_any __attribute__((aligned(4)));

// V consecutive elements of a row as they are stored.  or_else(): the elements,
// or one bit pattern for all of them (fp32's upper half) where `in` is false;
// forget(): what was computed from them is not kept for later use.
template <typename T, int V> struct Raw;
template <> struct Raw<uint16_t, 4> {
  u32x2 r;
  __device__ __forceinline__ void or_else(bool in, unsigned other) {
    other = other << 16 | other;
    r.x = in ? r.x : other;
    r.y = in ? r.y : other;
  }
  __device__ __forceinline__ void forget() { asm volatile("" : "+v"(r.x), "+v"(r.y)); }
  template <bool NT = false> __device__ __forceinline__ void load(const uint16_t* p) { r = load_as<NT, u32x2_any>(p); }
  __device__ __forceinline__ float get(int v) const {
    const unsigned w = v < 2 ? r.x : r.y;
    return __uint_as_float(v % 2 ? w & 0xffff0000u : w << 16);
  }
};
template <> struct Raw<float, 4> {
  f32x4 r;
  __device__ __forceinline__ void or_else(bool in, unsigned other) {
#pragma unroll
    for (int v = 0; v < 4; ++v) r[v] = in ? r[v] : __uint_as_float(other << 16);
  }
  __device__ __forceinline__ void forget() { asm volatile("" : "+v"(r)); }
  template <bool NT = false> __device__ __forceinline__ void load(const float* p) { r = load_as<NT, f32x4_any>(p); }
  __device__ __forceinline__ float get(int v) const { return r[v]; }
};
template <> struct Raw<uint16_t, 1> {
  uint16_t r;
  __device__ __forceinline__ void or_else(bool in, unsigned other) { r = in ? r : (uint16_t)other; }
  __device__ __forceinline__ void forget() { asm volatile("" : "+v"(r)); }
  template <bool NT = false> __device__ __forceinline__ void load(const uint16_t* p) { r = load_as<NT, uint16_t>(p); }
  __device__ __forceinline__ float get(int) const { return bf16_to_f32(r); }
};
template <> struct Raw<float, 1> {
  float r;
  __device__ __forceinline__ void or_else(bool in, unsigned other) { r = in ? r : __uint_as_float(other << 16); }
  __device__ __forceinline__ void forget() { asm volatile("" : "+v"(r)); }
  template <bool NT = false> __device__ __forceinline__ void load(const float* p) { r = load_as<NT, float>(p); }
  __device__ __forceinline__ float get(int) const { return r; }
};

template <int V, bool NT = false>
__device__ __forceinline__ void store_row(float* p, const float (&v)[V]) {
  if constexpr (V == 4)
    store_as<NT, f32x4_any>(p, f32x4{v[0], v[1], v[2], v[3]});
  else
    store_as<NT, float>(p, v[0]);
}

template <int V, bool NT = false>
__device__ __forceinline__ void store_row(uint16_t* p, const float (&v)[V]) {
  if constexpr (V == 4)
    store_as<NT, bf16x4_any>(
        p, bf16x4{f32_to_bf16(v[0]), f32_to_bf16(v[1]), f32_to_bf16(v[2]), f32_to_bf16(v[3])});
  else
    store_as<NT, __bf16>(p, f32_to_bf16(v[0]));
}

}  // namespace ssd
