// Device helpers of the attention layer's kernels (gdn_attn.h): element
// access, wave reductions, and the cache's formats.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace attn {

constexpr int kBlock = 64;  // tokens of a cache block

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef int32_t i32x2 __attribute__((ext_vector_type(2)));

// two floats to bf16, nearest even, packed
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const bf16x2 p = {(__bf16)lo, (__bf16)hi};
  return __builtin_bit_cast(uint32_t, p);
}

// STREAM: not to be kept in the caches
template <bool STREAM, class V>
__device__ __forceinline__ void store(V* p, V x) {
  if constexpr (STREAM)
    __builtin_nontemporal_store(x, p);
  else
    *p = x;
}

template <bool STREAM, class V>
__device__ __forceinline__ V load(const V* p) {
  if constexpr (STREAM)
    return __builtin_nontemporal_load(p);
  else
    return *p;
}

// four consecutive elements of the input type as floats, and back
struct ElemBf16 {
  typedef uint16_t T;
  static __device__ __forceinline__ f32x4 load4(const T* p) {
    const u32x2 r = *(const u32x2*)p;
    return f32x4{__uint_as_float(r[0] << 16), __uint_as_float(r[0] & 0xffff0000u), __uint_as_float(r[1] << 16),
                 __uint_as_float(r[1] & 0xffff0000u)};
  }
  template <bool STREAM>
  static __device__ __forceinline__ void store4(T* p, f32x4 x) {
    store<STREAM>((u32x2*)p, u32x2{pack2(x[0], x[1]), pack2(x[2], x[3])});
  }
};

struct ElemF32 {
  typedef float T;
  static __device__ __forceinline__ f32x4 load4(const T* p) { return *(const f32x4*)p; }
  template <bool STREAM>
  static __device__ __forceinline__ void store4(T* p, f32x4 x) { store<STREAM>((f32x4*)p, x); }
};

template <int CTRL>
__device__ __forceinline__ float dpp(float x) {
  return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(x), CTRL, 0xf, 0xf, true));
}

// max over lanes l, l ^ 16, l ^ 32, l ^ 48 (the four lanes that hold one row
// of an accumulator tile)
__device__ __forceinline__ float max_over_groups(float x) {
  auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  x = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
  auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}

// Sum over aligned groups of L lanes (8, 16 or 32); every lane gets it, the
// same bits in each (a butterfly of commutative adds).
template <int L>
__device__ __forceinline__ float sum_over_lanes(float x) {
  x += dpp<0xB1>(x);   // quad_perm [1,0,3,2]
  x += dpp<0x4E>(x);   // quad_perm [2,3,0,1]
  x += dpp<0x141>(x);  // row_half_mirror: the other quad of 8
  if (L >= 16) x += dpp<0x140>(x);  // row_mirror: the other 8 of 16
  if (L >= 32) {
    auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = __uint_as_float(a[0]) + __uint_as_float(a[1]);
  }
  return x;
}

// the batch entry whose cu range holds token t: the last i with cu[i] <= t
__device__ __forceinline__ int seq_of(const int32_t* cu, int N, int t) {
  int lo = 0, hi = N - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (cu[mid] <= t)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

// cache row of batch entry i, or -1
__device__ __forceinline__ int row_of(const int32_t* slot, int i, int num_slots) {
  const int r = slot ? slot[i] : i;
  return r >= 0 && r < num_slots ? r : -1;
}

}  // namespace attn
