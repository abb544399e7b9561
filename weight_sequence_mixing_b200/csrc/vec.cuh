// Vectors of 2 to 16 bytes of fp32 or bf16 channels: loaded and stored as one word of
// memory, computed on as floats, one at a time or two at a time in the packed fp32
// arithmetic of sm_100 (one instruction for both).
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace ttt {

struct One {
  static constexpr int N = 1;
  float v;
  __device__ __forceinline__ float operator[](int) const { return v; }
  static __device__ __forceinline__ One of(const float* f) { return {f[0]}; }
  static __device__ __forceinline__ One all(float f) { return {f}; }
};
struct Two {
  static constexpr int N = 2;
  uint64_t w;
  __device__ __forceinline__ float operator[](int i) const { return __uint_as_float(uint32_t(i ? w >> 32 : w)); }
  static __device__ __forceinline__ Two of(const float* f);
  static __device__ __forceinline__ Two all(float f);
};
__device__ __forceinline__ Two two(float a, float b) {
  Two r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.w) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ Two Two::of(const float* f) { return two(f[0], f[1]); }
__device__ __forceinline__ Two Two::all(float f) { return two(f, f); }
__device__ __forceinline__ One fma_(One a, One b, One c) { return {fmaf(a.v, b.v, c.v)}; }
__device__ __forceinline__ One mul_(One a, One b) { return {a.v * b.v}; }
__device__ __forceinline__ One add_(One a, One b) { return {a.v + b.v}; }
__device__ __forceinline__ One sub_(One a, One b) { return {a.v - b.v}; }
__device__ __forceinline__ Two fma_(Two a, Two b, Two c) {
  Two r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.w) : "l"(a.w), "l"(b.w), "l"(c.w));
  return r;
}
__device__ __forceinline__ Two mul_(Two a, Two b) {
  Two r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.w) : "l"(a.w), "l"(b.w));
  return r;
}
__device__ __forceinline__ Two add_(Two a, Two b) {
  Two r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.w) : "l"(a.w), "l"(b.w));
  return r;
}
__device__ __forceinline__ Two sub_(Two a, Two b) { return fma_(b, two(-1.f, -1.f), a); }

// The hardware's 2^v (2^-22 off) and 1 / v (2^-23 off), subnormal results as zero
__device__ __forceinline__ float exp2_fast(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float rcp_fast(float v) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
template <class F>
__device__ __forceinline__ One each(One a, F f) { return {f(a.v)}; }
template <class F>
__device__ __forceinline__ Two each(Two a, F f) { return two(f(a[0]), f(a[1])); }

template <int N>
struct PackOf {
  using type = Two;
};
template <>
struct PackOf<1> {
  using type = One;
};

template <class T, int BYTES>
struct Vec {
  static constexpr int N = BYTES / int(sizeof(T));
  static constexpr int kWords = (BYTES + 3) / 4;
  uint32_t w[kWords];

  __device__ __forceinline__ void load(const T* p) {
    if constexpr (BYTES == 16) {
      const uint4 q = *reinterpret_cast<const uint4*>(p);
      w[0] = q.x, w[1] = q.y, w[2] = q.z, w[3] = q.w;
    } else if constexpr (BYTES == 8) {
      const uint2 q = *reinterpret_cast<const uint2*>(p);
      w[0] = q.x, w[1] = q.y;
    } else if constexpr (BYTES == 4) {
      w[0] = *reinterpret_cast<const uint32_t*>(p);
    } else {
      w[0] = *reinterpret_cast<const uint16_t*>(p);
    }
  }
  __device__ __forceinline__ void store(T* p) const {
    if constexpr (BYTES == 16)
      *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    else if constexpr (BYTES == 8)
      *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    else if constexpr (BYTES == 4)
      *reinterpret_cast<uint32_t*>(p) = w[0];
    else
      *reinterpret_cast<uint16_t*>(p) = uint16_t(w[0]);
  }
  __device__ __forceinline__ void open(float (&v)[N]) const {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if constexpr (sizeof(T) == 4)
        v[i] = __uint_as_float(w[i]);
      else
        v[i] = __uint_as_float(i % 2 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
    }
  }
  using P = typename PackOf<N == 1 ? 1 : 2>::type;  // one or two of the values
  static constexpr int kPacks = N / P::N;
  __device__ __forceinline__ void open(P (&p)[kPacks]) const {
    float v[N];
    open(v);
#pragma unroll
    for (int i = 0; i < kPacks; ++i) p[i] = P::of(v + i * P::N);
  }
  __device__ __forceinline__ void close(const P (&p)[kPacks]) {
    float v[N];
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = p[i / P::N][i % P::N];
    close(v);
  }
  // rounded to nearest where T is bf16
  __device__ __forceinline__ void close(const float (&v)[N]) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < N; ++i) w[i] = __float_as_uint(v[i]);
    } else if constexpr (N == 1) {
      w[0] = __bfloat16_as_ushort(__float2bfloat16_rn(v[0]));
    } else {
#pragma unroll
      for (int i = 0; i < N; i += 2) {
        const __nv_bfloat162 p = __floats2bfloat162_rn(v[i], v[i + 1]);
        w[i / 2] = *reinterpret_cast<const uint32_t*>(&p);
      }
    }
  }
};

}  // namespace ttt
