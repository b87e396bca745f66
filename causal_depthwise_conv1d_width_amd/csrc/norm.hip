// norm.hip -- RMS norms around a mixer block, forward and backward.
//
//   gated, gate first:  u = x silu(z),  y = w u / rms(u)          by groups of channels
//   gated, norm first:  u = x,          y = w u / rms(u) silu(z)
//   residual:           r' = r + scale x (stored),  y = w r' / rms(r')
// with rms(u)^2 = mean(u^2) + eps.  With n = u / rms(u) and d the gradient of n:
//   du = (d - n mean(d n)) / rms(u),   dw = sum over rows of (gradient of w n) n.
//
// These are streams: one pass over the rows, each value read and written once, all arithmetic FP32.
// T threads share a row's group (64: one wave, up to 2048 channels; 256 or 1024 threads: a block)
// and keep it in registers, four pieces of 8 channels a thread.  A thread keeps its channels' weights
// (and, backward, its dw sums) in registers over all the rows it visits; the sums go to one partial row
// per row split, and a second kernel adds those in ascending order (no atomics: the same bits every run).
#include "ssm_device.h"

namespace cssm {

constexpr int kVec = 4;  // pieces of 8 channels a thread holds

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

template <int T, bool NORM_FIRST>
__global__ __launch_bounds__(T == 64 ? 256 : T) void gated_norm_fwd_kernel(NormArgs a) {
  __shared__ float lds[16];
  const Place<T> u(a);
  if (!u.ok) return;  // whole waves (T == 64); never with T > 64
  F8 w[kVec];
#pragma unroll
  for (int v = 0; v < kVec; ++v) {
    const int64_t c = (v * T + u.t) * 8;
    w[v] = load_w(a, u.col0 + c, a.group - c);
  }
  for (int64_t row = u.split; row < a.rows; row += a.parts) {
    F8 x[kVec], z[kVec];
    float s = 0.f;
#pragma unroll
    for (int v = 0; v < kVec; ++v) {
      const int64_t c = (v * T + u.t) * 8;
      if (v * T * 8 >= a.group) break;
      x[v] = load8(a.x + row * a.x_ld + u.col0 + c, a.group - c);
      z[v] = load8(a.z + row * a.z_ld + u.col0 + c, a.group - c);
    }
#pragma unroll
    for (int v = 0; v < kVec; ++v) {
      if (v * T * 8 >= a.group) break;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        z[v].f[e] *= sigmoid(z[v].f[e]);
        if (!NORM_FIRST) x[v].f[e] *= z[v].f[e];
        s = __builtin_fmaf(x[v].f[e], x[v].f[e], s);
      }
    }
    const float inv = rsqrtf(unit_sum<T>(s, lds) / (float)a.group + a.eps);
#pragma unroll
    for (int v = 0; v < kVec; ++v) {
      const int64_t c = (v * T + u.t) * 8;
      if (v * T * 8 >= a.group) break;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        x[v].f[e] *= inv * w[v].f[e];
        if (NORM_FIRST) x[v].f[e] *= z[v].f[e];
      }
      store8(a.y + row * a.y_ld + u.col0 + c, x[v], a.group - c);
    }
  }
}

template <int T, bool NORM_FIRST>
__global__ __launch_bounds__(T == 64 ? 256 : T) void gated_norm_bwd_kernel(NormArgs a) {
  __shared__ float lds[16];
  const Place<T> u(a);
  if (!u.ok) return;
  F8 w[kVec], dw[kVec];
#pragma unroll
  for (int v = 0; v < kVec; ++v) {
    const int64_t c = (v * T + u.t) * 8;
    w[v] = load_w(a, u.col0 + c, a.group - c);
    dw[v] = zero8();
  }
  for (int64_t row = u.split; row < a.rows; row += a.parts) {
    F8 x[kVec], z[kVec], d[kVec];
    float s = 0.f, sd = 0.f;
#pragma unroll
    for (int v = 0; v < kVec; ++v) {
      const int64_t c = (v * T + u.t) * 8;
      if (v * T * 8 >= a.group) break;
      x[v] = load8(a.x + row * a.x_ld + u.col0 + c, a.group - c);
      z[v] = load8(a.z + row * a.z_ld + u.col0 + c, a.group - c);
      d[v] = load8(a.dy + row * a.dy_ld + u.col0 + c, a.group - c);
    }
    // s = sum u^2, sd = sum u d w (both before the division by the rms)
#pragma unroll
    for (int v = 0; v < kVec; ++v) {
      if (v * T * 8 >= a.group) break;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float gate = z[v].f[e] * sigmoid(z[v].f[e]);
        const float uu = NORM_FIRST ? x[v].f[e] : x[v].f[e] * gate;
        const float dn = (NORM_FIRST ? d[v].f[e] * gate : d[v].f[e]) * w[v].f[e];
        s = __builtin_fmaf(uu, uu, s);
        sd = __builtin_fmaf(uu, dn, sd);
      }
    }
    const float n = (float)a.group;
    const float inv = rsqrtf(unit_sum<T>(s, lds) / n + a.eps);
    const float m = unit_sum<T>(sd, lds) * inv / n;  // mean of d n
#pragma unroll
    for (int v = 0; v < kVec; ++v) {
      const int64_t c = (v * T + u.t) * 8;
      if (v * T * 8 >= a.group) break;
      F8 dz;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float zz = z[v].f[e], sg = sigmoid(zz), gate = zz * sg;
        const float slope = sg * (1.f + zz * (1.f - sg));
        const float uu = NORM_FIRST ? x[v].f[e] : x[v].f[e] * gate;
        const float nn = uu * inv, dy = d[v].f[e];
        const float dn = NORM_FIRST ? dy * gate : dy;
        dw[v].f[e] = __builtin_fmaf(dn, nn, dw[v].f[e]);
        const float du = inv * (dn * w[v].f[e] - nn * m);
        dz.f[e] = (NORM_FIRST ? dy * nn * w[v].f[e] : du * x[v].f[e]) * slope;
        x[v].f[e] = NORM_FIRST ? du : du * gate;
      }
      store8(a.dx + row * a.dx_ld + u.col0 + c, x[v], a.group - c);
      store8(a.dz + row * a.dz_ld + u.col0 + c, dz, a.group - c);
    }
  }
  float* part = a.part + u.split * a.groups * a.group + u.col0;
#pragma unroll
  for (int v = 0; v < kVec; ++v) {
    const int64_t c = (v * T + u.t) * 8;
    if (c < a.group) store8(part + c, dw[v], a.group - c);
  }
}

template <int T, typename R>
__global__ __launch_bounds__(T == 64 ? 256 : T) void residual_norm_fwd_kernel(NormArgs a) {
  __shared__ float lds[16];
  const Place<T> u(a);
  if (!u.ok) return;
  F8 w[kVec];
#pragma unroll
  for (int v = 0; v < kVec; ++v) {
    const int64_t c = (v * T + u.t) * 8;
    w[v] = load_w(a, c, a.group - c);
  }
  const R* r_in = static_cast<const R*>(a.r);
  R* r_out = static_cast<R*>(a.r_out);
  for (int64_t row = u.split; row < a.rows; row += a.parts) {
    F8 h[kVec];
    float s = 0.f;
#pragma unroll
    for (int v = 0; v < kVec; ++v) {
      const int64_t c = (v * T + u.t) * 8;
      if (v * T * 8 >= a.group) break;
      const F8 x = load8(a.x + row * a.x_ld + c, a.group - c);
      h[v] = load8(r_in + row * a.r_ld + c, a.group - c);
#pragma unroll
      for (int e = 0; e < 8; ++e) h[v].f[e] = __builtin_fmaf(a.scale, x.f[e], h[v].f[e]);
    }
#pragma unroll
    for (int v = 0; v < kVec; ++v) {
      const int64_t c = (v * T + u.t) * 8;
      if (v * T * 8 >= a.group) break;
      store8(r_out + row * a.ro_ld + c, h[v], a.group - c);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        h[v].f[e] = as_stored(h[v].f[e], r_out);
        s = __builtin_fmaf(h[v].f[e], h[v].f[e], s);
      }
    }
    const float inv = rsqrtf(unit_sum<T>(s, lds) / (float)a.group + a.eps);
#pragma unroll
    for (int v = 0; v < kVec; ++v) {
      const int64_t c = (v * T + u.t) * 8;
      if (v * T * 8 >= a.group) break;
#pragma unroll
      for (int e = 0; e < 8; ++e) h[v].f[e] *= inv * w[v].f[e];
      store8(a.y + row * a.y_ld + c, h[v], a.group - c);
    }
  }
}

template <int T, typename R>
__global__ __launch_bounds__(T == 64 ? 256 : T) void residual_norm_bwd_kernel(NormArgs a) {
  __shared__ float lds[16];
  const Place<T> u(a);
  if (!u.ok) return;
  F8 w[kVec], dw[kVec];
#pragma unroll
  for (int v = 0; v < kVec; ++v) {
    const int64_t c = (v * T + u.t) * 8;
    w[v] = load_w(a, c, a.group - c);
    dw[v] = zero8();
  }
  const R* r = static_cast<const R*>(a.r);
  const R* dri = static_cast<const R*>(a.dr_in);
  R* dro = static_cast<R*>(a.r_out);
  for (int64_t row = u.split; row < a.rows; row += a.parts) {
    F8 h[kVec], d[kVec], o[kVec];
    float s = 0.f, sd = 0.f;
#pragma unroll
    for (int v = 0; v < kVec; ++v) {
      const int64_t c = (v * T + u.t) * 8;
      if (v * T * 8 >= a.group) break;
      h[v] = load8(r + row * a.r_ld + c, a.group - c);
      d[v] = load8(a.dy + row * a.dy_ld + c, a.group - c);
      o[v] = dri ? load8(dri + row * a.dri_ld + c, a.group - c) : zero8();
    }
#pragma unroll
    for (int v = 0; v < kVec; ++v) {
      if (v * T * 8 >= a.group) break;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        s = __builtin_fmaf(h[v].f[e], h[v].f[e], s);
        sd = __builtin_fmaf(h[v].f[e], d[v].f[e] * w[v].f[e], sd);
      }
    }
    const float n = (float)a.group;
    const float inv = rsqrtf(unit_sum<T>(s, lds) / n + a.eps);
    const float m = unit_sum<T>(sd, lds) * inv / n;
#pragma unroll
    for (int v = 0; v < kVec; ++v) {
      const int64_t c = (v * T + u.t) * 8;
      if (v * T * 8 >= a.group) break;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float nn = h[v].f[e] * inv;
        dw[v].f[e] = __builtin_fmaf(d[v].f[e], nn, dw[v].f[e]);
        o[v].f[e] += inv * (d[v].f[e] * w[v].f[e] - nn * m);
        h[v].f[e] = a.scale * o[v].f[e];
      }
      store8(dro + row * a.ro_ld + c, o[v], a.group - c);
      store8(a.dx + row * a.dx_ld + c, h[v], a.group - c);
    }
  }
  float* part = a.part + u.split * a.group;
#pragma unroll
  for (int v = 0; v < kVec; ++v) {
    const int64_t c = (v * T + u.t) * 8;
    if (c < a.group) store8(part + c, dw[v], a.group - c);
  }
}

// dw[c] = the partial rows' sum: 16 threads a channel take the rows k, k + 16, ... in ascending order,
// and their sums are added in ascending order of k.
__global__ __launch_bounds__(1024) void norm_dw_kernel(const float* __restrict__ part, int64_t parts, int64_t d,
                                                       float* __restrict__ dw) {
  __shared__ float lds[16][64];
  const int t = threadIdx.x & 63, k = threadIdx.x >> 6;
  const int64_t c = (int64_t)blockIdx.x * 64 + t;
  float s = 0.f;
  if (c < d) {
#pragma unroll 8
    for (int64_t r = k; r < parts; r += 16) s += part[r * d + c];
  }
  lds[k][t] = s;
  __syncthreads();
  if (k == 0 && c < d) {
#pragma unroll
    for (int j = 1; j < 16; ++j) s += lds[j][t];
    dw[c] = s;
  }
}

static uint32_t blocks(const NormArgs& a, int T) {
  const int64_t units = a.parts * a.groups;
  return (uint32_t)(T == 64 ? (units + 3) / 4 : units);
}
static hipError_t reduce_dw(const NormArgs& a, hipStream_t s) {
  const int64_t d = a.groups * a.group;
  norm_dw_kernel<<<dim3((uint32_t)((d + 63) / 64)), 1024, 0, s>>>(a.part, a.parts, d, a.dw);
  return hipGetLastError();
}

template <int T>
static void gated(const NormArgs& a, bool bwd, hipStream_t s) {
  const dim3 grid(blocks(a, T)), block(T == 64 ? 256 : T);
  if (bwd) {
    if (a.norm_first) gated_norm_bwd_kernel<T, true><<<grid, block, 0, s>>>(a);
    else gated_norm_bwd_kernel<T, false><<<grid, block, 0, s>>>(a);
  } else {
    if (a.norm_first) gated_norm_fwd_kernel<T, true><<<grid, block, 0, s>>>(a);
    else gated_norm_fwd_kernel<T, false><<<grid, block, 0, s>>>(a);
  }
}
template <int T>
static void residual(const NormArgs& a, bool bwd, hipStream_t s) {
  const dim3 grid(blocks(a, T)), block(T == 64 ? 256 : T);
  if (bwd) {
    if (a.r_f32) residual_norm_bwd_kernel<T, float><<<grid, block, 0, s>>>(a);
    else residual_norm_bwd_kernel<T, uint16_t><<<grid, block, 0, s>>>(a);
  } else {
    if (a.r_f32) residual_norm_fwd_kernel<T, float><<<grid, block, 0, s>>>(a);
    else residual_norm_fwd_kernel<T, uint16_t><<<grid, block, 0, s>>>(a);
  }
}

#define CSSM_BY_THREADS(fn, bwd)                          \
  switch (norm_threads(a.group)) {                        \
    case 64: fn<64>(a, bwd, s); break;                    \
    case 256: fn<256>(a, bwd, s); break;                  \
    default: fn<1024>(a, bwd, s); break;                  \
  }

hipError_t launch_gated_fwd(const NormArgs& a, hipStream_t s) {
  CSSM_BY_THREADS(gated, false)
  return hipGetLastError();
}
hipError_t launch_gated_bwd(const NormArgs& a, hipStream_t s) {
  if (a.rows > 0) CSSM_BY_THREADS(gated, true)
  return reduce_dw(a, s);
}
hipError_t launch_residual_fwd(const NormArgs& a, hipStream_t s) {
  CSSM_BY_THREADS(residual, false)
  return hipGetLastError();
}
hipError_t launch_residual_bwd(const NormArgs& a, hipStream_t s) {
  if (a.rows > 0) CSSM_BY_THREADS(residual, true)
  return reduce_dw(a, s);
}

}  // namespace cssm
