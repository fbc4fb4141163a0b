// Element types of the float matrices, vector types, and loads and stores of several
// values at any element's address.
#pragma once

#include <hip/hip_runtime.h>

namespace gemm {
namespace mx {

constexpr int kF32 = 0, kBf16 = 1, kF16 = 2;   // GEMM_TYPE_*

typedef int intx4 __attribute__((ext_vector_type(4)));
typedef int intx8 __attribute__((ext_vector_type(8)));
typedef unsigned uintx2 __attribute__((ext_vector_type(2)));
typedef unsigned uintx4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef unsigned short u16;

// ---------------------------------------------------------------------------
// Element types.
template <int TYPE>
struct Elem;
template <>
struct Elem<kF32> {
  typedef float store;
  static __device__ inline float get(float v) { return v; }
  static __device__ inline float put(float v) { return v; }
};
template <>
struct Elem<kBf16> {
  typedef u16 store;
  static __device__ inline float get(u16 v) {
    return __builtin_bit_cast(float, static_cast<unsigned>(v) << 16);
  }
  static __device__ inline u16 put(float v) {
    return __builtin_bit_cast(u16, static_cast<__bf16>(v));   // nearest, ties to even
  }
};
template <>
struct Elem<kF16> {
  typedef u16 store;
  static __device__ inline float get(u16 v) {
    return static_cast<float>(__builtin_bit_cast(_Float16, v));
  }
  static __device__ inline u16 put(float v) {
    return __builtin_bit_cast(u16, static_cast<_Float16>(v));
  }
};

// 16 bytes at any element's address: the memory system takes loads and stores that
// are not aligned to their size.
typedef uintx4 uintx4_any __attribute__((aligned(2)));

// 8 consecutive values from p, the first `n` of them, zeros for the rest.
template <int TYPE>
__device__ inline void load8(const typename Elem<TYPE>::store *p, int n, float (&v)[8]) {
  if (n >= 8) {
    if constexpr (TYPE == kF32) {
      const uintx4 a = reinterpret_cast<const uintx4_any *>(p)[0];
      const uintx4 b = reinterpret_cast<const uintx4_any *>(p)[1];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const unsigned x = a[i], y = b[i];   // (the cast of a vector's element itself takes the first)
        v[i] = __builtin_bit_cast(float, x);
        v[4 + i] = __builtin_bit_cast(float, y);
      }
    } else {
      const uintx4 a = *reinterpret_cast<const uintx4_any *>(p);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = Elem<TYPE>::get(static_cast<u16>(a[i]));
        v[2 * i + 1] = Elem<TYPE>::get(static_cast<u16>(a[i] >> 16));
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < n ? Elem<TYPE>::get(p[i]) : 0.0f;
  }
}

template <int TYPE>
__device__ inline void store8(typename Elem<TYPE>::store *p, int n, const float (&v)[8]) {
  if (n >= 8) {
    if constexpr (TYPE == kF32) {
      uintx4 a, b;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        a[i] = __builtin_bit_cast(unsigned, v[i]);
        b[i] = __builtin_bit_cast(unsigned, v[4 + i]);
      }
      reinterpret_cast<uintx4_any *>(p)[0] = a;
      reinterpret_cast<uintx4_any *>(p)[1] = b;
    } else {
      uintx4 a;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        a[i] = Elem<TYPE>::put(v[2 * i]) | (static_cast<unsigned>(Elem<TYPE>::put(v[2 * i + 1])) << 16);
      *reinterpret_cast<uintx4_any *>(p) = a;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = Elem<TYPE>::put(v[i]);
  }
}

// Order between the LDS accesses of a wave's lanes: LDS serves them in order, so only
// the compiler has to keep them.
__device__ inline void wave_order() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

}  // namespace mx
}  // namespace gemm
