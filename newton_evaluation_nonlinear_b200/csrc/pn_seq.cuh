// pn_seq.cuh -- what the sequence-layer operators share: element types, rows of
// heads, the rotary plan and the checks of their entry points.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "../../include/pn.h"

constexpr int kMaxRotPairs = 128;   // rot_dim <= 256

// The plan of one rotation: host memory only, so that it serves every device
// and stream and travels to the kernels by value.  Frequencies are turns per
// position in 64-bit fixed point, f / (2 pi) mod 1 = turn / 2^64: position *
// turn mod 2^64 is then the angle's fraction of a turn, exact but for the
// rounding of turn itself (|position| 2^-65 turns), however far the position
// lies.  A 32-bit float angle would be off by half a radian at position 2^23.
struct pn_rotary_plan {
  int pairs;      // rot_dim / 2
  int interleaved;
  float factor;   // m, on both components
  unsigned long long turn[kMaxRotPairs];
};

namespace pn {

void set_thread_error(const char* msg);   // pn_api.cu: the text of pn_last_error(NULL)
pn_status seq_fail(pn_status st, const char* fmt, ...);
// Device of a device (or managed) pointer; *dev < 0 takes that device, else it must match.
pn_status seq_device(const void* p, const char* name, int* dev);
// Refuses an output [B][T][H] of rows of dim elements that overlap each other.
pn_status seq_output(const pn_heads* y, const char* name, long long B, long long T, int H, int dim);
// Refuses an output that is the memory of another array of the call (arrays that overlap in part are the caller's care).
pn_status seq_apart(const void* y, const char* name, const void* x, const char* other);
inline size_t dtype_size(int dtype) { return dtype == PN_F32 ? 4 : 2; }

// Restores the caller's current device on scope exit.
struct SeqDeviceGuard {
  int prev = -1;
  explicit SeqDeviceGuard(int dev) {
    if (cudaGetDevice(&prev) == cudaSuccess && prev != dev) cudaSetDevice(dev);
    else prev = -1;
  }
  ~SeqDeviceGuard() {
    if (prev >= 0) cudaSetDevice(prev);
  }
};

template <typename T> __device__ __forceinline__ float to_f(T v);
template <> __device__ __forceinline__ float to_f(float v) { return v; }
template <> __device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
template <> __device__ __forceinline__ float to_f(__half v) { return __half2float(v); }
template <typename T> __device__ __forceinline__ T from_f(float v);
template <> __device__ __forceinline__ float from_f(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f(float v) { return __float2bfloat16_rn(v); }
template <> __device__ __forceinline__ __half from_f(float v) { return __float2half_rn(v); }

// V consecutive elements as one load or store (V * sizeof(T) <= 16, aligned to that)
template <int BYTES> struct RawVec;
template <> struct RawVec<2> { using type = unsigned short; };
template <> struct RawVec<4> { using type = unsigned; };
template <> struct RawVec<8> { using type = uint2; };
template <> struct RawVec<16> { using type = uint4; };

// two float32 products or sums to an instruction
__device__ __forceinline__ unsigned long long pack2(float a, float b) {
  unsigned long long r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack2(unsigned long long v, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
__device__ __forceinline__ unsigned long long mul2(unsigned long long a, unsigned long long b) {
  unsigned long long r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ unsigned long long fma2(unsigned long long a, unsigned long long b, unsigned long long c) {
  unsigned long long r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// V consecutive elements in registers, widened and rounded two at a time where they are 16 bits wide (element by
// element the compiler takes three instructions for what one does).
template <typename T, int V> union VecOf {
  typename RawVec<V * (int)sizeof(T)>::type raw;
  T e[V];
  uint32_t two[V * (int)sizeof(T) / 4 > 0 ? V * (int)sizeof(T) / 4 : 1];
  __device__ VecOf() {}
  __device__ __forceinline__ void widen(float (&v)[V]) const {
    if constexpr (sizeof(T) == 2 && V >= 2) {
#pragma unroll
      for (int i = 0; i < V; i += 2) {
        if constexpr (std::is_same_v<T, __nv_bfloat16>) {
          v[i] = __uint_as_float(two[i / 2] << 16);
          v[i + 1] = __uint_as_float(two[i / 2] & 0xffff0000u);
        } else {
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&two[i / 2]));
          v[i] = f.x;
          v[i + 1] = f.y;
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] = to_f<T>(e[i]);
    }
  }
  __device__ __forceinline__ void round(const float (&v)[V]) {
    if constexpr (sizeof(T) == 2 && V >= 2) {
#pragma unroll
      for (int i = 0; i < V; i += 2) {
        if constexpr (std::is_same_v<T, __nv_bfloat16>) {
          const __nv_bfloat162 p = __floats2bfloat162_rn(v[i], v[i + 1]);
          two[i / 2] = *reinterpret_cast<const uint32_t*>(&p);
        } else {
          const __half2 p = __floats2half2_rn(v[i], v[i + 1]);
          two[i / 2] = *reinterpret_cast<const uint32_t*>(&p);
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) e[i] = from_f<T>(v[i]);
    }
  }
};

template <typename T, int V> __device__ __forceinline__ void ld_vec(const T* p, float (&v)[V]) {
  VecOf<T, V> u;
  u.raw = *reinterpret_cast<const typename RawVec<V * (int)sizeof(T)>::type*>(p);
  u.widen(v);
}
template <typename T, int V> __device__ __forceinline__ void st_vec(T* p, const float (&v)[V]) {
  VecOf<T, V> u;
  u.round(v);
  *reinterpret_cast<typename RawVec<V * (int)sizeof(T)>::type*>(p) = u.raw;
}
// elementwise, two to an instruction: y = a b, y += a b, y = y s
template <int V> __device__ __forceinline__ void mul_vec(const float (&a)[V], const float (&b)[V], float (&y)[V]) {
  if constexpr (V % 2 == 0) {
#pragma unroll
    for (int i = 0; i < V; i += 2) unpack2(mul2(pack2(a[i], a[i + 1]), pack2(b[i], b[i + 1])), y[i], y[i + 1]);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) y[i] = a[i] * b[i];
  }
}
template <int V> __device__ __forceinline__ void fma_vec(const float (&a)[V], const float (&b)[V], const float (&c)[V], float (&y)[V]) {
  if constexpr (V % 2 == 0) {
#pragma unroll
    for (int i = 0; i < V; i += 2)
      unpack2(fma2(pack2(a[i], a[i + 1]), pack2(b[i], b[i + 1]), pack2(c[i], c[i + 1])), y[i], y[i + 1]);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) y[i] = fmaf(a[i], b[i], c[i]);
  }
}
template <int V> __device__ __forceinline__ void scale_vec(float s, float (&y)[V]) {
  if constexpr (V % 2 == 0) {
    const unsigned long long ss = pack2(s, s);
#pragma unroll
    for (int i = 0; i < V; i += 2) unpack2(mul2(ss, pack2(y[i], y[i + 1])), y[i], y[i + 1]);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) y[i] *= s;
  }
}
// sum of products, with one running sum for even and one for odd elements
template <int V> __device__ __forceinline__ void dot_vec(const float (&a)[V], const float (&b)[V], unsigned long long& s) {
  if constexpr (V % 2 == 0) {
#pragma unroll
    for (int i = 0; i < V; i += 2) s = fma2(pack2(a[i], a[i + 1]), pack2(b[i], b[i + 1]), s);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) s = fma2(pack2(a[i], 0.0f), pack2(b[i], 0.0f), s);
  }
}

// cos and sin (times m) of position * turn: the top 32 bits of the fraction are
// the angle in units of 2^-32 turns.  FAST is for results that are all rounded to
// 16 bits: the special-function unit's sine and cosine, within 2^-21.4 for angles up
// to pi (their documented bound), with the angle's own rounding 2^-20.8.
template <bool FAST>
__device__ __forceinline__ void turn_cos_sin(unsigned long long turn, long long pos, float m, float& c, float& s) {
  const int hi = (int)(unsigned)((turn * (unsigned long long)pos) >> 32);
  if constexpr (FAST) __sincosf((float)hi * 1.4629180792671596e-9f, &s, &c);   // 2 pi 2^-32
  else sincospif((float)hi * 0x1p-31f, &s, &c);
  c *= m;
  s *= m;
}

}  // namespace pn
