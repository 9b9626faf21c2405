// Element types and row access shared by the row-moving kernels: W consecutive
// elements of bf16, fp16 or fp32 as one load or store, converted to fp32.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"

namespace moe {

__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f32(float v) { return v; }
template <typename T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ __nv_bfloat16 from_f32(float v) { return __float2bfloat16_rn(v); }
template <> __device__ __forceinline__ __half from_f32(float v) { return __float2half_rn(v); }
template <> __device__ __forceinline__ float from_f32(float v) { return v; }

// W elements of T as raw bits: one memory access of 2, 4, 8, 16 or 32 bytes, aligned
// to its size.
struct alignas(32) Raw32 {
  uint4 a, b;
};
__device__ __forceinline__ Raw32 load32(const void* p) {
  Raw32 r;
  asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r.a.x), "=r"(r.a.y), "=r"(r.a.z), "=r"(r.a.w), "=r"(r.b.x), "=r"(r.b.y),
                 "=r"(r.b.z), "=r"(r.b.w)
               : "l"(p) : "memory");
  return r;
}
__device__ __forceinline__ void store32(void* p, const Raw32& r) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(r.a.x),
               "r"(r.a.y), "r"(r.a.z), "r"(r.a.w), "r"(r.b.x), "r"(r.b.y), "r"(r.b.z), "r"(r.b.w)
               : "memory");
}
template <int BYTES> struct RawOf;
template <> struct RawOf<32> { using type = Raw32; };
template <> struct RawOf<16> { using type = uint4; };
template <> struct RawOf<8> { using type = uint2; };
template <> struct RawOf<4> { using type = uint32_t; };
template <> struct RawOf<2> { using type = uint16_t; };

template <typename T, int W> struct Vec {
  using Raw = typename RawOf<sizeof(T) * W>::type;
  static __device__ __forceinline__ Raw load(const T* p) {   // read-only data
    if constexpr (sizeof(Raw) == 32) return load32(p);
    else return __ldg(reinterpret_cast<const Raw*>(p));
  }
  static __device__ __forceinline__ Raw load_rw(const T* p) {   // data this kernel also writes
    if constexpr (sizeof(Raw) == 32) return load32(p);
    else return *reinterpret_cast<const Raw*>(p);
  }
  static __device__ __forceinline__ Raw zero() {
    Raw r;
    memset(&r, 0, sizeof(r));
    return r;
  }
  static __device__ __forceinline__ void store(T* p, const Raw& r) {
    if constexpr (sizeof(Raw) == 32) store32(p, r);
    else *reinterpret_cast<Raw*>(p) = r;
  }
  static __device__ __forceinline__ void unpack(const Raw& r, float* f) {
    T e[W];
    memcpy(e, &r, sizeof(r));
#pragma unroll
    for (int i = 0; i < W; ++i) f[i] = to_f32(e[i]);
  }
  static __device__ __forceinline__ Raw pack(const float* f) {   // round to nearest even
    T e[W];
#pragma unroll
    for (int i = 0; i < W; ++i) e[i] = from_f32<T>(f[i]);
    Raw r;
    memcpy(&r, e, sizeof(r));
    return r;
  }
};

// Zeros n elements from p on, by G threads (this one is t): 16 bytes a store whatever
// the row's alignment, its ragged ends element by element.
template <typename T, int G>
__device__ __forceinline__ void zero_span(T* p, int n, int t) {
  const int head = min(n, (int)((16 - (reinterpret_cast<uintptr_t>(p) & 15)) % 16 / sizeof(T)));
  constexpr int E = 16 / sizeof(T);
  const int body = (n - head) / E;
  for (int i = t; i < body; i += G)
    reinterpret_cast<uint4*>(p + head)[i] = make_uint4(0, 0, 0, 0);
  const int tail = head + body * E;
  for (int i = t; i < head + n - tail; i += G) {
    const int at = i < head ? i : tail + i - head;
    Vec<T, 1>::store(p + at, Vec<T, 1>::zero());
  }
}

inline int dtype_bytes(int dtype) {
  return dtype == MOE_F32 ? 4 : (dtype == MOE_BF16 || dtype == MOE_F16) ? 2 : 0;
}

// A matrix of rows: base pointer and row stride in elements.
struct RowsIn {
  const void* p;
  long long ld;
};
struct RowsOut {
  void* p;
  long long ld;
};

// The widest access (bytes: 16, 4 or the element) that divides the row length,
// every row stride and every base address.
inline int access_bytes(int dtype, int d, const RowsIn* in, int n_in, const RowsOut* out,
                        int n_out) {
  const int es = dtype_bytes(dtype);
  for (int b = 16; b > es; b = b == 16 ? 4 : es) {
    bool ok = (long long)d * es % b == 0;
    for (int i = 0; i < n_in; ++i)
      ok = ok && (!in[i].p || ((uintptr_t)in[i].p % b == 0 && in[i].ld * es % b == 0));
    for (int i = 0; i < n_out; ++i)
      ok = ok && (!out[i].p || ((uintptr_t)out[i].p % b == 0 && out[i].ld * es % b == 0));
    if (ok) return b;
  }
  return es;
}

}  // namespace moe
