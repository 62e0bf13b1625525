// Element types of the operators that take fp32 or bfloat16 arrays: loads
// and stores of a few neighbouring elements as fp32 values.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace fc {

// bfloat16 is converted with the compiler's __bf16 (rounds to nearest even).
using bf16 = __bf16;

template <class T, int V>
struct alignas(sizeof(T) * V) Pack {
  T e[V];
};

// V elements at p (aligned to V * sizeof(T)) as fp32
template <class T, int V>
__device__ __forceinline__ void load_f32(const T* p, float* x) {
  const Pack<T, V> t = *reinterpret_cast<const Pack<T, V>*>(p);
#pragma unroll
  for (int i = 0; i < V; ++i) x[i] = static_cast<float>(t.e[i]);
}

template <class T, int V>
__device__ __forceinline__ void store_f32(T* p, const float* x) {
  Pack<T, V> t;
#pragma unroll
  for (int i = 0; i < V; ++i) t.e[i] = static_cast<T>(x[i]);
  *reinterpret_cast<Pack<T, V>*>(p) = t;
}

}  // namespace fc
