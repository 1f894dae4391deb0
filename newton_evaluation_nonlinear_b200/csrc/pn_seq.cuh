// pn_seq.cuh -- what the sequence-layer operators share: element types, rows of
// heads, the rotary plan and the checks of their entry points.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

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

template <typename T, int V> union VecOf {
  typename RawVec<V * (int)sizeof(T)>::type raw;
  T e[V];
  __device__ VecOf() {}
};

template <typename T, int V> __device__ __forceinline__ void ld_vec(const T* p, float (&v)[V]) {
  VecOf<T, V> u;
  u.raw = *reinterpret_cast<const typename RawVec<V * (int)sizeof(T)>::type*>(p);
#pragma unroll
  for (int i = 0; i < V; ++i) v[i] = to_f<T>(u.e[i]);
}
template <typename T, int V> __device__ __forceinline__ void st_vec(T* p, const float (&v)[V]) {
  VecOf<T, V> u;
#pragma unroll
  for (int i = 0; i < V; ++i) u.e[i] = from_f<T>(v[i]);
  *reinterpret_cast<typename RawVec<V * (int)sizeof(T)>::type*>(p) = u.raw;
}

// cos and sin (times m) of position * turn: the top 32 bits of the fraction are
// the angle in units of 2^-31 half turns.
__device__ __forceinline__ void turn_cos_sin(unsigned long long turn, long long pos, float m, float& c, float& s) {
  const int hi = (int)(unsigned)((turn * (unsigned long long)pos) >> 32);
  sincospif((float)hi * 0x1p-31f, &s, &c);
  c *= m;
  s *= m;
}

}  // namespace pn
