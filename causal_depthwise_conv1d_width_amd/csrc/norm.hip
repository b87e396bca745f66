// norm.hip -- RMS norms around a mixer block, forward and backward.
//
//   gated, gate first:  u = x silu(z),  y = w u / rms(u)          by groups of channels
//   gated, norm first:  u = x,          y = w u / rms(u) silu(z)
//   residual:           r' = r + scale x (stored),  y = w r' / rms(r')
// with rms(u)^2 = mean(u^2) + eps.  With n = u / rms(u) and d the gradient of n:
//   du = (d - n mean(d n)) / rms(u),   dw = sum over rows of (gradient of w n) n.
//
// These are streams: one pass over the rows, each value read and written once, all arithmetic FP32.
// T threads share a row's group and keep it in registers, V pieces of 8 channels a thread (64 up to
// 512 channels, 1024 from 8192), the bf16 inputs packed as they are in memory: with FP32 copies of x, z and dy
// the gated backward had 262 registers and 2 waves a SIMD, too few to cover its loads (302 us at
// 16384 x 4096 in groups of 1024, against 128 us).  A thread keeps its channels' weights (and, backward, its dw sums) in
// registers over all the rows it visits; the sums go to one partial row per row split, and a second kernel adds
// those in ascending order (no atomics: the same bits every run).
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

template <int T, int V, bool NORM_FIRST>
__global__ __launch_bounds__(T == 64 ? 256 : T) void gated_norm_fwd_kernel(NormArgs a) {
  __shared__ float lds[16];
  const Place<T> u(a);
  if (!u.ok) return;  // whole waves (T == 64); never with T > 64
  const Weights<T, V> ww(a, u.col0, u.t);
  for (int64_t row = u.split; row < a.rows; row += a.parts) {
    Raw16 x[V], z[V];
    float s = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int64_t c = (v * T + u.t) * 8;
      x[v] = raw8(a.x + row * a.x_ld + u.col0 + c, a.group - c);
      z[v] = raw8(a.z + row * a.z_ld + u.col0 + c, a.group - c);
    }
    F8 f[V], gate[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      f[v] = x[v].get();
      gate[v] = z[v].get();
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        gate[v].f[e] *= sigmoid(gate[v].f[e]);
        if (!NORM_FIRST) f[v].f[e] *= gate[v].f[e];
        s = __builtin_fmaf(f[v].f[e], f[v].f[e], s);
      }
    }
    const float inv = rsqrtf(unit_sum<T>(s, lds) / (float)a.group + a.eps);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int64_t c = (v * T + u.t) * 8;
      const F8 w = ww.get(a, u.col0, u.t, v);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        f[v].f[e] *= inv * w.f[e];
        if (NORM_FIRST) f[v].f[e] *= gate[v].f[e];
      }
      store8(a.y + row * a.y_ld + u.col0 + c, f[v], a.group - c);
    }
  }
}

template <int T, int V, bool NORM_FIRST>
__global__ __launch_bounds__(T == 64 ? 256 : T) void gated_norm_bwd_kernel(NormArgs a) {
  __shared__ float lds[16];
  const Place<T> u(a);
  if (!u.ok) return;
  const Weights<T, V> ww(a, u.col0, u.t);
  F8 dw[V];
#pragma unroll
  for (int v = 0; v < V; ++v) dw[v] = zero8();
  for (int64_t row = u.split; row < a.rows; row += a.parts) {
    Raw16 x[V], z[V], d[V];
    float s = 0.f, sd = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int64_t c = (v * T + u.t) * 8;
      x[v] = raw8(a.x + row * a.x_ld + u.col0 + c, a.group - c);
      z[v] = raw8(a.z + row * a.z_ld + u.col0 + c, a.group - c);
      d[v] = raw8(a.dy + row * a.dy_ld + u.col0 + c, a.group - c);
    }
    // s = sum u^2, sd = sum u d w (both before the division by the rms)
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const F8 fx = x[v].get(), fz = z[v].get(), fd = d[v].get(), w = ww.get(a, u.col0, u.t, v);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float gate = fz.f[e] * sigmoid(fz.f[e]);
        const float uu = NORM_FIRST ? fx.f[e] : fx.f[e] * gate;
        const float dn = (NORM_FIRST ? fd.f[e] * gate : fd.f[e]) * w.f[e];
        s = __builtin_fmaf(uu, uu, s);
        sd = __builtin_fmaf(uu, dn, sd);
      }
    }
    const float n = (float)a.group;
    const float inv = rsqrtf(unit_sum<T>(s, lds) / n + a.eps);
    const float m = unit_sum<T>(sd, lds) * inv / n;  // mean of d n
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int64_t c = (v * T + u.t) * 8;
      x[v].again(), z[v].again(), d[v].again();
      const F8 fx = x[v].get(), fz = z[v].get(), fd = d[v].get(), w = ww.get(a, u.col0, u.t, v);
      F8 dx, dz;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float zz = fz.f[e], sg = sigmoid(zz), gate = zz * sg;
        const float slope = sg * (1.f + zz * (1.f - sg));
        const float uu = NORM_FIRST ? fx.f[e] : fx.f[e] * gate;
        const float nn = uu * inv, dy = fd.f[e];
        const float dn = NORM_FIRST ? dy * gate : dy;
        dw[v].f[e] = __builtin_fmaf(dn, nn, dw[v].f[e]);
        const float du = inv * (dn * w.f[e] - nn * m);
        dz.f[e] = (NORM_FIRST ? dy * nn * w.f[e] : du * fx.f[e]) * slope;
        dx.f[e] = NORM_FIRST ? du : du * gate;
      }
      store8(a.dx + row * a.dx_ld + u.col0 + c, dx, a.group - c);
      store8(a.dz + row * a.dz_ld + u.col0 + c, dz, a.group - c);
    }
  }
  float* part = a.part + u.split * a.groups * a.group + u.col0;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int64_t c = (v * T + u.t) * 8;
    if (c < a.group) store8(part + c, dw[v], a.group - c);
  }
}

template <int T, int V, typename R>
__global__ __launch_bounds__(T == 64 ? 256 : T) void residual_norm_fwd_kernel(NormArgs a) {
  __shared__ float lds[16];
  const Place<T> u(a);
  if (!u.ok) return;
  const Weights<T, V> ww(a, 0, u.t);
  const R* r_in = static_cast<const R*>(a.r);
  R* r_out = static_cast<R*>(a.r_out);
  for (int64_t row = u.split; row < a.rows; row += a.parts) {
    Raw16 x[V];
    RawOf<R> r[V];
    F8 h[V];
    float s = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int64_t c = (v * T + u.t) * 8;
      x[v] = raw8(a.x + row * a.x_ld + c, a.group - c);
      r[v] = raw8(r_in + row * a.r_ld + c, a.group - c);
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int64_t c = (v * T + u.t) * 8;
      const F8 fx = x[v].get();
      h[v] = r[v].get();
#pragma unroll
      for (int e = 0; e < 8; ++e) h[v].f[e] = __builtin_fmaf(a.scale, fx.f[e], h[v].f[e]);
      store8(r_out + row * a.ro_ld + c, h[v], a.group - c);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        h[v].f[e] = as_stored(h[v].f[e], r_out);
        s = __builtin_fmaf(h[v].f[e], h[v].f[e], s);
      }
    }
    const float inv = rsqrtf(unit_sum<T>(s, lds) / (float)a.group + a.eps);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int64_t c = (v * T + u.t) * 8;
      const F8 w = ww.get(a, 0, u.t, v);
#pragma unroll
      for (int e = 0; e < 8; ++e) h[v].f[e] *= inv * w.f[e];
      store8(a.y + row * a.y_ld + c, h[v], a.group - c);
    }
  }
}

template <int T, int V, typename R>
__global__ __launch_bounds__(T == 64 ? 256 : T) void residual_norm_bwd_kernel(NormArgs a) {
  __shared__ float lds[16];
  const Place<T> u(a);
  if (!u.ok) return;
  const Weights<T, V> ww(a, 0, u.t);
  F8 dw[V];
#pragma unroll
  for (int v = 0; v < V; ++v) dw[v] = zero8();
  const R* r = static_cast<const R*>(a.r);
  const R* dri = static_cast<const R*>(a.dr_in);
  R* dro = static_cast<R*>(a.r_out);
  for (int64_t row = u.split; row < a.rows; row += a.parts) {
    RawOf<R> h[V], o[V];
    Raw16 d[V];
    float s = 0.f, sd = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int64_t c = (v * T + u.t) * 8;
      h[v] = raw8(r + row * a.r_ld + c, a.group - c);
      d[v] = raw8(a.dy + row * a.dy_ld + c, a.group - c);
      o[v] = dri ? raw8(dri + row * a.dri_ld + c, a.group - c) : zero_raw(dri);
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const F8 fh = h[v].get(), fd = d[v].get(), w = ww.get(a, 0, u.t, v);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        s = __builtin_fmaf(fh.f[e], fh.f[e], s);
        sd = __builtin_fmaf(fh.f[e], fd.f[e] * w.f[e], sd);
      }
    }
    const float n = (float)a.group;
    const float inv = rsqrtf(unit_sum<T>(s, lds) / n + a.eps);
    const float m = unit_sum<T>(sd, lds) * inv / n;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int64_t c = (v * T + u.t) * 8;
      h[v].again(), d[v].again();
      const F8 fh = h[v].get(), fd = d[v].get(), w = ww.get(a, 0, u.t, v);
      F8 g = o[v].get(), dx;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float nn = fh.f[e] * inv;
        dw[v].f[e] = __builtin_fmaf(fd.f[e], nn, dw[v].f[e]);
        g.f[e] += inv * (fd.f[e] * w.f[e] - nn * m);
        dx.f[e] = a.scale * g.f[e];
      }
      store8(dro + row * a.ro_ld + c, g, a.group - c);
      store8(a.dx + row * a.dx_ld + c, dx, a.group - c);
    }
  }
  float* part = a.part + u.split * a.group;
#pragma unroll
  for (int v = 0; v < V; ++v) {
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

template <int T, int V>
static void gated(const NormArgs& a, bool bwd, hipStream_t s) {
  const dim3 grid(blocks(a, T)), block(T == 64 ? 256 : T);
  if (bwd) {
    if (a.norm_first) gated_norm_bwd_kernel<T, V, true><<<grid, block, 0, s>>>(a);
    else gated_norm_bwd_kernel<T, V, false><<<grid, block, 0, s>>>(a);
  } else {
    if (a.norm_first) gated_norm_fwd_kernel<T, V, true><<<grid, block, 0, s>>>(a);
    else gated_norm_fwd_kernel<T, V, false><<<grid, block, 0, s>>>(a);
  }
}
template <int T, int V>
static void residual(const NormArgs& a, bool bwd, hipStream_t s) {
  const dim3 grid(blocks(a, T)), block(T == 64 ? 256 : T);
  if (bwd) {
    if (a.r_f32) residual_norm_bwd_kernel<T, V, float><<<grid, block, 0, s>>>(a);
    else residual_norm_bwd_kernel<T, V, uint16_t><<<grid, block, 0, s>>>(a);
  } else {
    if (a.r_f32) residual_norm_fwd_kernel<T, V, float><<<grid, block, 0, s>>>(a);
    else residual_norm_fwd_kernel<T, V, uint16_t><<<grid, block, 0, s>>>(a);
  }
}

// threads and pieces a thread by the group's channels (norm_threads gives the same threads)
#define CSSM_BY_GROUP(fn, bwd)                              \
  do {                                                      \
    switch (norm_threads(a.group)) {                        \
      case 64: fn<64, 1>(a, bwd, s); break;                 \
      case 128: fn<128, 1>(a, bwd, s); break;               \
      case 256: fn<256, 1>(a, bwd, s); break;               \
      case 512: fn<512, 1>(a, bwd, s); break;               \
      default:                                              \
        if (a.group <= 8192) fn<1024, 1>(a, bwd, s);        \
        else if (a.group <= 16384) fn<1024, 2>(a, bwd, s);  \
        else fn<1024, 4>(a, bwd, s);                        \
    }                                                       \
  } while (0)

hipError_t launch_gated_fwd(const NormArgs& a, hipStream_t s) {
  CSSM_BY_GROUP(gated, false);
  return hipGetLastError();
}
hipError_t launch_gated_bwd(const NormArgs& a, hipStream_t s) {
  if (a.rows > 0) CSSM_BY_GROUP(gated, true);
  return reduce_dw(a, s);
}
hipError_t launch_residual_fwd(const NormArgs& a, hipStream_t s) {
  CSSM_BY_GROUP(residual, false);
  return hipGetLastError();
}
hipError_t launch_residual_bwd(const NormArgs& a, hipStream_t s) {
  if (a.rows > 0) CSSM_BY_GROUP(residual, true);
  return reduce_dw(a, s);
}

}  // namespace cssm
