// layer_norm.hip -- layer norm before a block, alone or of the residual's sum, forward and backward.
//
//   h = x, or r' = r + scale x (stored);  n = (h - mean(h)) / sd,  y = w n + bias,  sd^2 = var(h) + eps
// With d = w dy:  dh = (d - mean(d) - n mean(d n)) / sd + dr',  dr = dh,  dx = scale dh,
//   dw = sum over rows of dy n,  dbias = sum over rows of dy.
// Rows are held in registers as in the RMS norms (norm.hip): one pass over memory, FP32.  The variance is that of the
// centred values, a second sum over the registers.  Backward, the first sum takes h and d, the second their centred
// products, so that there are two sums, not four.  Bound by memory: 16384 rows of 2048, with an FP32 residual, forward and
// backward in 185 us, 5.1 TB/s (a large copy: 4.9).  dw and dbias: one partial row of each a row split, added in
// ascending order by a second kernel.
#include "delta_launch.h"
#include "norm_device.h"

namespace cssm {

struct Pair {
  float a, b;
};
// both sums over the T threads of a unit, in every one of them
template <int T>
__device__ __forceinline__ Pair unit_sum2(Pair v, Pair* lds) {
  v.a = wave_sum(v.a), v.b = wave_sum(v.b);
  if constexpr (T > 64) {
    __syncthreads();  // lds may still be read from the sum before
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
    __syncthreads();
    v = Pair{0.f, 0.f};
#pragma unroll
    for (int k = 0; k < T / 64; ++k) {
      v.a += lds[k].a;
      v.b += lds[k].b;
    }
  }
  return v;
}

template <int T, int V, typename R, bool RES>
__global__ __launch_bounds__(T == 64 ? 256 : T) void layer_norm_fwd_kernel(LayerArgs l) {
  __shared__ float lds[16];
  const NormArgs& a = l.n;
  const Place<T> u(a);
  if (!u.ok) return;  // whole waves (T == 64); never with T > 64
  const Weights<T, V> ww(a, 0, u.t);
  NormArgs ab = a;
  ab.w = l.bias;
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
      if constexpr (RES) r[v] = raw8(r_in + row * a.r_ld + c, a.group - c);
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int64_t c = (v * T + u.t) * 8;
      h[v] = x[v].get();
      if constexpr (RES) {
        const F8 fr = r[v].get();
#pragma unroll
        for (int e = 0; e < 8; ++e) h[v].f[e] = __builtin_fmaf(a.scale, h[v].f[e], fr.f[e]);
        store8(r_out + row * a.ro_ld + c, h[v], a.group - c);
#pragma unroll
        for (int e = 0; e < 8; ++e) h[v].f[e] = as_stored(h[v].f[e], r_out);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) s += h[v].f[e];
    }
    const float mean = unit_sum<T>(s, lds) / (float)a.group;
    s = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int64_t n = a.group - (v * T + u.t) * 8;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        h[v].f[e] = e < n ? h[v].f[e] - mean : 0.f;
        s = __builtin_fmaf(h[v].f[e], h[v].f[e], s);
      }
    }
    const float inv = rsqrtf(unit_sum<T>(s, lds) / (float)a.group + a.eps);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int64_t c = (v * T + u.t) * 8;
      const F8 w = ww.get(a, 0, u.t, v);
      const F8 b = l.bias ? load_w(ab, c, a.group - c) : zero8();
#pragma unroll
      for (int e = 0; e < 8; ++e) h[v].f[e] = __builtin_fmaf(h[v].f[e] * inv, w.f[e], b.f[e]);
      store8(a.y + row * a.y_ld + c, h[v], a.group - c);
    }
  }
}

template <int T, int V, typename R>
__global__ __launch_bounds__(T == 64 ? 256 : T) void layer_norm_bwd_kernel(LayerArgs l) {
  __shared__ Pair lds[16];
  const NormArgs& a = l.n;
  const Place<T> u(a);
  if (!u.ok) return;
  const Weights<T, V> ww(a, 0, u.t);
  F8 dw[V], db[V];
#pragma unroll
  for (int v = 0; v < V; ++v) dw[v] = db[v] = zero8();
  const R* r = static_cast<const R*>(a.r);
  const R* dri = static_cast<const R*>(a.dr_in);
  R* dro = static_cast<R*>(a.r_out);
  const float n = (float)a.group;
  for (int64_t row = u.split; row < a.rows; row += a.parts) {
    RawOf<R> h[V], o[V];
    Raw16 d[V];
    Pair s = {0.f, 0.f};
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
        s.a += fh.f[e];
        s.b = __builtin_fmaf(fd.f[e], w.f[e], s.b);
      }
    }
    s = unit_sum2<T>(s, lds);
    const float mean = s.a / n, mean_d = s.b / n;
    s = Pair{0.f, 0.f};
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int64_t in = a.group - (v * T + u.t) * 8;
      h[v].again(), d[v].again();
      const F8 fh = h[v].get(), fd = d[v].get(), w = ww.get(a, 0, u.t, v);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float c = e < in ? fh.f[e] - mean : 0.f;
        s.a = __builtin_fmaf(c, c, s.a);
        s.b = __builtin_fmaf(c, fd.f[e] * w.f[e], s.b);
      }
    }
    s = unit_sum2<T>(s, lds);
    const float inv = rsqrtf(s.a / n + a.eps), m = s.b * inv / n;  // mean of d n
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int64_t c = (v * T + u.t) * 8;
      h[v].again(), d[v].again();
      const F8 fh = h[v].get(), fd = d[v].get(), w = ww.get(a, 0, u.t, v);
      F8 g = o[v].get(), dx;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float nn = (fh.f[e] - mean) * inv;  // past the channels dy is zero
        dw[v].f[e] = __builtin_fmaf(fd.f[e], nn, dw[v].f[e]);
        db[v].f[e] += fd.f[e];
        g.f[e] += inv * (fd.f[e] * w.f[e] - mean_d - nn * m);
        dx.f[e] = a.scale * g.f[e];
      }
      if (dro) store8(dro + row * a.ro_ld + c, g, a.group - c);
      store8(a.dx + row * a.dx_ld + c, dx, a.group - c);
    }
  }
  float* part = a.part + u.split * 2 * a.group;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int64_t c = (v * T + u.t) * 8;
    if (c >= a.group) continue;
    store8(part + c, dw[v], a.group - c);
    store8(part + a.group + c, db[v], a.group - c);
  }
}

// dw[c] and dbias[c]: the partial rows' sums, 16 threads a channel taking the rows k, k + 16, ... in ascending order
__global__ __launch_bounds__(1024) void layer_norm_sum_kernel(const float* __restrict__ part, int64_t parts, int64_t d,
                                                              float* __restrict__ dw, float* __restrict__ db) {
  __shared__ float lds[16][64];
  const int t = threadIdx.x & 63, k = threadIdx.x >> 6;
  const int64_t c = (int64_t)blockIdx.x * 64 + t;
  float s = 0.f;
  if (c < 2 * d) {
#pragma unroll 8
    for (int64_t r = k; r < parts; r += 16) s += part[r * 2 * d + c];
  }
  lds[k][t] = s;
  __syncthreads();
  if (k == 0 && c < 2 * d) {
#pragma unroll
    for (int j = 1; j < 16; ++j) s += lds[j][t];
    if (c < d) dw[c] = s;
    else if (db) db[c - d] = s;
  }
}

template <int T, int V>
static void layer(const LayerArgs& l, bool bwd, hipStream_t s) {
  const NormArgs& a = l.n;
  const dim3 grid((uint32_t)(T == 64 ? (a.parts + 3) / 4 : a.parts)), block(T == 64 ? 256 : T);
  if (bwd) {
    if (a.r_f32) layer_norm_bwd_kernel<T, V, float><<<grid, block, 0, s>>>(l);
    else layer_norm_bwd_kernel<T, V, uint16_t><<<grid, block, 0, s>>>(l);
  } else if (!a.r) {
    layer_norm_fwd_kernel<T, V, uint16_t, false><<<grid, block, 0, s>>>(l);
  } else {
    if (a.r_f32) layer_norm_fwd_kernel<T, V, float, true><<<grid, block, 0, s>>>(l);
    else layer_norm_fwd_kernel<T, V, uint16_t, true><<<grid, block, 0, s>>>(l);
  }
}

// threads and pieces a thread by the channels, as for the RMS norms
static void by_channels(const LayerArgs& l, bool bwd, hipStream_t s) {
  const int64_t d = l.n.group;
  switch (norm_threads(d)) {
    case 64: return layer<64, 1>(l, bwd, s);
    case 128: return layer<128, 1>(l, bwd, s);
    case 256: return layer<256, 1>(l, bwd, s);
    case 512: return layer<512, 1>(l, bwd, s);
    default:
      if (d <= 8192) return layer<1024, 1>(l, bwd, s);
      if (d <= 16384) return layer<1024, 2>(l, bwd, s);
      return layer<1024, 4>(l, bwd, s);
  }
}

hipError_t launch_layer_fwd(const LayerArgs& l, hipStream_t s) {
  by_channels(l, false, s);
  return hipGetLastError();
}
hipError_t launch_layer_bwd(const LayerArgs& l, hipStream_t s) {
  if (l.n.rows > 0) by_channels(l, true, s);
  layer_norm_sum_kernel<<<dim3((uint32_t)((2 * l.n.group + 63) / 64)), 1024, 0, s>>>(l.n.part, l.n.rows > 0 ? l.n.parts : 0,
                                                                                    l.n.group, l.n.dw, l.db);
  return hipGetLastError();
}

}  // namespace cssm
