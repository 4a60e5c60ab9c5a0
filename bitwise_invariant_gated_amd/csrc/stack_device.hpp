// Device helpers of the kernels around a stack's layers (gdn_stack.h): eight
// elements at a time, and reductions over a wave.
#pragma once

#include "attn_device.hpp"

namespace stack {

using attn::dpp;
using attn::f32x4;
using attn::pack2;
using attn::sum_over_lanes;
using attn::u32x2;
using attn::u32x4;

// Sixteen bytes at an address that is a multiple of that, or of an element only
// (the memory unit splits what crosses a line).
template <bool ANY>
struct Pick {
  typedef u32x4 U;
  typedef f32x4 F;
};
template <>
struct Pick<true> {
  typedef u32x4 U __attribute__((aligned(2)));
  typedef f32x4 F __attribute__((aligned(4)));
};

// Eight consecutive elements of one lane.
struct F8 {
  f32x4 a, b;
  __device__ __forceinline__ float& operator[](int i) { return i < 4 ? ((float*)&a)[i] : ((float*)&b)[i - 4]; }
};

// Element access: T the stored type, RAW eight of them as loaded.  ANY: at any
// element's address; ONCE: not to be kept in the caches.
struct B16 {
  typedef uint16_t T;
  typedef u32x4 RAW;
  template <bool ANY, bool ONCE = false>
  static __device__ __forceinline__ RAW load(const T* p) {
    if constexpr (ONCE) return __builtin_nontemporal_load((const typename Pick<ANY>::U*)p);
    return *(const typename Pick<ANY>::U*)p;
  }
  static __device__ __forceinline__ float one(T x) { return __uint_as_float((uint32_t)x << 16); }
  static __device__ __forceinline__ T round(float x) { return __builtin_bit_cast(uint16_t, (__bf16)x); }
  static __device__ __forceinline__ F8 wide(RAW r) {
    F8 f;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      f.a[2 * i] = __uint_as_float(r[i] << 16);
      f.a[2 * i + 1] = __uint_as_float(r[i] & 0xffff0000u);
      f.b[2 * i] = __uint_as_float(r[2 + i] << 16);
      f.b[2 * i + 1] = __uint_as_float(r[2 + i] & 0xffff0000u);
    }
    return f;
  }
  // a vector of eight from and to runs of 16 bytes
  static __device__ __forceinline__ void widen(F8& f, const u32x4* r) { f = wide(r[0]); }
  static __device__ __forceinline__ void narrow_to(const F8& f, u32x4* r) { r[0] = narrow(f); }
  static __device__ __forceinline__ RAW narrow(F8 f) {
    return RAW{pack2(f.a[0], f.a[1]), pack2(f.a[2], f.a[3]), pack2(f.b[0], f.b[1]), pack2(f.b[2], f.b[3])};
  }
  static __device__ __forceinline__ void store(T* p, RAW r) { *(u32x4*)p = r; }
};

struct F32 {
  typedef float T;
  typedef F8 RAW;
  template <bool ANY, bool ONCE = false>
  static __device__ __forceinline__ RAW load(const T* p) {
    typedef typename Pick<ANY>::F V;
    if constexpr (ONCE) return F8{__builtin_nontemporal_load((const V*)p), __builtin_nontemporal_load((const V*)(p + 4))};
    return F8{*(const V*)p, *(const V*)(p + 4)};
  }
  static __device__ __forceinline__ float one(T x) { return x; }
  static __device__ __forceinline__ T round(float x) { return x; }
  static __device__ __forceinline__ F8 wide(RAW r) { return r; }
  static __device__ __forceinline__ RAW narrow(F8 f) { return f; }
  static __device__ __forceinline__ void widen(F8& f, const u32x4* r) {
    f = F8{__builtin_bit_cast(f32x4, r[0]), __builtin_bit_cast(f32x4, r[1])};
  }
  static __device__ __forceinline__ void narrow_to(const F8& f, u32x4* r) {
    r[0] = __builtin_bit_cast(u32x4, f.a);
    r[1] = __builtin_bit_cast(u32x4, f.b);
  }
  static __device__ __forceinline__ void store(T* p, RAW r) {
    *(f32x4*)p = r.a;
    *(f32x4*)(p + 4) = r.b;
  }
};

// Sum over aligned groups of L lanes (16 .. 64), the same bits in every lane.
template <int L>
__device__ __forceinline__ float sum_lanes(float x) {
  x = sum_over_lanes<(L > 32 ? 32 : L)>(x);
  if constexpr (L == 64) {
    const auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = __uint_as_float(a[0]) + __uint_as_float(a[1]);
  }
  return x;
}

// The largest of three; a quiet NaN counts for nothing.  (The instruction itself:
// fmaxf would first quiet each of its operands.)
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("v_max3_f32 %0, %1, %2, %3" : "=v"(r) : "v"(a), "v"(b), "v"(c));
  return r;
}

// Maximum over aligned groups of 16 lanes, and over the four groups of a wave.
// (Canonicalising x first puts an instruction of the compiler's own before the
// lane exchange, whose wait states it then counts.)
__device__ __forceinline__ float max_16(float x) {
  x = __builtin_canonicalizef(x);
  x = fmaxf(x, dpp<0xB1>(x));
  x = fmaxf(x, dpp<0x4E>(x));
  x = fmaxf(x, dpp<0x141>(x));
  return fmaxf(x, dpp<0x140>(x));
}

__device__ __forceinline__ float max_groups(float x) { return attn::max_over_groups(x); }

}  // namespace stack
