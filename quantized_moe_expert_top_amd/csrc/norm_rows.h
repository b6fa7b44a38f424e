// Rows of norms in registers: chunks of 8 values per thread, loads and stores in their
// types, sums over the waves that hold a row.
#pragma once
#include "mm.h"

namespace moe {

template <class T>
__device__ __forceinline__ void unpack8(const uint4& p, float (&v)[8]) {
  unpack2<T>(p.x, v[0], v[1]);
  unpack2<T>(p.y, v[2], v[3]);
  unpack2<T>(p.z, v[4], v[5]);
  unpack2<T>(p.w, v[6], v[7]);
}
// Eight values of a row as they are stored: 16 bytes of T, or 32 of float32.
template <class T, bool F32>
struct Row8 {
  uint4 lo, hi;   // hi: float32 only
  __device__ __forceinline__ void load(const void* x, size_t at) {
    if constexpr (F32) {
      lo = ld16(static_cast<const float*>(x) + at);
      hi = ld16(static_cast<const float*>(x) + at + 4);
    } else {
      lo = ld16(static_cast<const uint16_t*>(x) + at);
    }
  }
  __device__ __forceinline__ void zero() {
    lo = make_uint4(0, 0, 0, 0);
    hi = make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ void values(float (&v)[8]) const {
    if constexpr (F32) {
      const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(w[i]);
    } else {
      unpack8<T>(lo, v);
    }
  }
};
template <class T>
__device__ __forceinline__ void row_load8(const void* p, size_t at, bool f32, float (&v)[8]) {
  if (f32) {
    const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(p) + at);
    const float4 a = q[0], b = q[1];
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  } else {
    const uint4 w = ld16(static_cast<const uint16_t*>(p) + at);
    unpack2<T>(w.x, v[0], v[1]);
    unpack2<T>(w.y, v[2], v[3]);
    unpack2<T>(w.z, v[4], v[5]);
    unpack2<T>(w.w, v[6], v[7]);
  }
}
template <class T>
__device__ __forceinline__ void row_store8(void* p, size_t at, bool f32, const float (&v)[8]) {
  if (f32) {
    float4* q = reinterpret_cast<float4*>(static_cast<float*>(p) + at);
    q[0] = make_float4(v[0], v[1], v[2], v[3]);
    q[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + at) =
        make_uint4(pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3]), pack2<T>(v[4], v[5]),
                   pack2<T>(v[6], v[7]));
  }
}
// Rows of results; STREAM: past the caches (see mm_put16), where a call writes more
// than the L2s' 32 MB (forward of 16384 x 2048: 49 us against 62).
template <class T, bool STREAM>
__device__ __forceinline__ void row_put8(void* p, size_t at, bool f32, const float (&v)[8]) {
  if constexpr (STREAM) {
    if (f32) {
      f32x4_t* q = reinterpret_cast<f32x4_t*>(static_cast<float*>(p) + at);
      __builtin_nontemporal_store(f32x4_t{v[0], v[1], v[2], v[3]}, q);
      __builtin_nontemporal_store(f32x4_t{v[4], v[5], v[6], v[7]}, q + 1);
    } else {
      __builtin_nontemporal_store(mm_pack8<T>(v),
                                  reinterpret_cast<i32x4_t*>(static_cast<uint16_t*>(p) + at));
    }
  } else {
    row_store8<T>(p, at, f32, v);
  }
}
template <class T>
__device__ __forceinline__ float load1(const void* p, size_t at) {
  float lo, hi;
  unpack2<T>(static_cast<const uint16_t*>(p)[at], lo, hi);
  return lo;
}

// Sum over a row held by WPR waves; every thread gets it. `red` holds WPR
// floats and is free again after the next call's barrier (two slots alternate).
template <int WPR>
__device__ __forceinline__ float row_sum(float v, float* red) {
  v = wave_sum_f32(v);
  if constexpr (WPR == 1) return v;
  const int lane = threadIdx.x & (kWave - 1), w = threadIdx.x >> 6;
  if (lane == 0) red[w] = v;
  __syncthreads();
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < WPR; ++i) s += red[i];
  return s;
}

}  // namespace moe
