// norm_device.h -- rows of a norm in registers, 8 channels a thread and piece: loads, stores, sums over the threads that
// share a row, weights.
#pragma once

#include "ssm_device.h"

namespace cssm {

struct F8 {
  float f[8];
};
__device__ __forceinline__ F8 zero8() {
  F8 v;
#pragma unroll
  for (int e = 0; e < 8; ++e) v.f[e] = 0.f;
  return v;
}
__device__ __forceinline__ F8 unpack8(u32x4 u) {
  F8 v;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    v.f[2 * e] = bf_lo(u[e]);
    v.f[2 * e + 1] = bf_hi(u[e]);
  }
  return v;
}
// 8 values as they are in memory
struct Raw16 {
  u32x4 v;
  // forget what was computed from v: a second pass unpacks again instead of keeping the first one's FP32
  // values (twice the registers, and the gates beside them)
  __device__ __forceinline__ void again() { asm("" : "+v"(v)); }
  __device__ __forceinline__ F8 get() const { return unpack8(v); }
};
struct Raw32 {
  f32x4 a, b;
  __device__ __forceinline__ void again() {}
  __device__ __forceinline__ F8 get() const { return F8{{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]}}; }
};
__device__ __forceinline__ Raw16 raw8(const uint16_t* p, int64_t n) {
  Raw16 r;
  if (n >= 8) {
    r.v = __builtin_nontemporal_load(reinterpret_cast<const u32x4_a2*>(p));
    return r;
  }
  r.v = u32x4{0u, 0u, 0u, 0u};
#pragma unroll
  for (int e = 0; e < 7; ++e)
    if (e < n) r.v[e >> 1] |= (uint32_t)p[e] << (16 * (e & 1));
  return r;
}
__device__ __forceinline__ Raw32 raw8(const float* p, int64_t n) {
  Raw32 r;
  if (n >= 8) {
    r.a = __builtin_nontemporal_load(reinterpret_cast<const f32x4_a4*>(p));
    r.b = __builtin_nontemporal_load(reinterpret_cast<const f32x4_a4*>(p + 4));
    return r;
  }
  r.a = r.b = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int e = 0; e < 7; ++e)
    if (e < n) (e < 4 ? r.a : r.b)[e & 3] = p[e];
  return r;
}
__device__ __forceinline__ Raw16 zero_raw(const uint16_t*) { return Raw16{u32x4{0u, 0u, 0u, 0u}}; }
__device__ __forceinline__ Raw32 zero_raw(const float*) { return Raw32{f32x4{0.f, 0.f, 0.f, 0.f}, f32x4{0.f, 0.f, 0.f, 0.f}}; }
template <typename R>
using RawOf = decltype(raw8((const R*)nullptr, 0));
__device__ __forceinline__ F8 load8(const uint16_t* p, int64_t n) {  // the first n (>= 8: all) of 8 values
  if (n >= 8) return unpack8(__builtin_nontemporal_load(reinterpret_cast<const u32x4_a2*>(p)));
  F8 v = zero8();
  for (int e = 0; e < 7; ++e)
    if (e < n) v.f[e] = bf_f32(p[e]);
  return v;
}
__device__ __forceinline__ F8 load8(const float* p, int64_t n) {
  F8 v = zero8();
  if (n >= 8) {
    const f32x4 a = __builtin_nontemporal_load(reinterpret_cast<const f32x4_a4*>(p));
    const f32x4 b = __builtin_nontemporal_load(reinterpret_cast<const f32x4_a4*>(p + 4));
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v.f[e] = a[e];
      v.f[4 + e] = b[e];
    }
    return v;
  }
  for (int e = 0; e < 7; ++e)
    if (e < n) v.f[e] = p[e];
  return v;
}
__device__ __forceinline__ void store8(uint16_t* p, const F8& v, int64_t n) {
  u32x4 u;
#pragma unroll
  for (int e = 0; e < 4; ++e) u[e] = pk_bf16(v.f[2 * e], v.f[2 * e + 1]);
  if (n >= 8) {
    __builtin_nontemporal_store(u, reinterpret_cast<u32x4_a2*>(p));
    return;
  }
#pragma unroll
  for (int e = 0; e < 7; ++e)
    if (e < n) p[e] = (uint16_t)(u[e >> 1] >> (16 * (e & 1)));
}
__device__ __forceinline__ void store8(float* p, const F8& v, int64_t n) {
  if (n >= 8) {
    __builtin_nontemporal_store(f32x4{v.f[0], v.f[1], v.f[2], v.f[3]}, reinterpret_cast<f32x4_a4*>(p));
    __builtin_nontemporal_store(f32x4{v.f[4], v.f[5], v.f[6], v.f[7]}, reinterpret_cast<f32x4_a4*>(p + 4));
    return;
  }
#pragma unroll
  for (int e = 0; e < 7; ++e)
    if (e < n) p[e] = v.f[e];
}
__device__ __forceinline__ F8 load_w(const NormArgs& a, int64_t c, int64_t n) {
  return a.w_f32 ? load8(static_cast<const float*>(a.w) + c, n) : load8(static_cast<const uint16_t*>(a.w) + c, n);
}
// the value as it is stored (the norm of a bf16 residual reads the rounded sum)
__device__ __forceinline__ float as_stored(float v, uint16_t*) { return bf_lo(pk_bf16(v, 0.f)); }
__device__ __forceinline__ float as_stored(float v, float*) { return v; }

// sum over the T threads of a unit, in every one of them
template <int T>
__device__ __forceinline__ float unit_sum(float v, float* lds) {
  v = wave_sum(v);
  if constexpr (T > 64) {
    __syncthreads();  // lds may still be read from the sum before
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0.f;
#pragma unroll
    for (int k = 0; k < T / 64; ++k) v += lds[k];
  }
  return v;
}

// This thread's place: unit = (row split, group), first row, lane in the unit.
template <int T>
struct Place {
  int64_t split, col0;
  int t;
  bool ok;
  __device__ __forceinline__ Place(const NormArgs& a) {
    const int64_t unit = T == 64 ? (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6) : blockIdx.x;
    t = T == 64 ? threadIdx.x & 63 : threadIdx.x;
    ok = unit < a.parts * a.groups;
    split = unit / a.groups;
    col0 = unit % a.groups * a.group;
  }
};

// Weights of a thread's channels: kept in registers, or, where 1024 threads leave too few, read for each row.
template <int T, int V>
struct Weights {
  static constexpr bool kKept = T < 1024;
  F8 w[kKept ? V : 1];
  __device__ __forceinline__ Weights(const NormArgs& a, int64_t col0, int t) {
    if constexpr (kKept) {
#pragma unroll
      for (int v = 0; v < V; ++v) w[v] = load_w(a, col0 + (v * T + t) * 8, a.group - (v * T + t) * 8);
    }
  }
  __device__ __forceinline__ F8 get(const NormArgs& a, int64_t col0, int t, int v) const {
    if constexpr (kKept) return w[v];
    else return load_w(a, col0 + (v * T + t) * 8, a.group - (v * T + t) * 8);
  }
};

}  // namespace cssm
