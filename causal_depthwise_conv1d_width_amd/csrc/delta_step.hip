// delta_step.hip -- the gated delta rule for one token a sequence against the slot pool of FP32 states.
//
//   u = r (v - a S k),   S' = a S + u k^T,   y = scale S' q = scale (a S q + u (k q))
// A stream over the states (read and written once): 8 bytes for 7 operations, bound by memory: 64 sequences of 32 heads of
// 128 x 128 in 52 us, 5.2 TB/s (a large copy: 4.9).  One sequence takes 14 us, which is its launch.  A lane holds four
// columns n of a row p; LN lanes (a power of two, up to 64) share a row, and a wave keeps kRowsHeld rows a lane in flight.
// Both of a row's products come from the state as it was read, so that their sums over the lanes run side by side.
#include "delta_launch.h"
#include "ssm_device.h"

namespace cssm {

constexpr int kRowsHeld = 4;

// sum over the LN lanes of a row, in every one of them
template <int LN>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
  for (int m = LN / 2; m > 0; m >>= 1) v += __shfl_xor(v, m);
  return v;
}

template <int LN, bool VEC>
__global__ __launch_bounds__(256) void delta_step_kernel(DeltaStepArgs a) {
  constexpr int kRows = 64 / LN * kRowsHeld;  // rows a wave covers
  const int lane = threadIdx.x & 63;
  const int per_head = (a.P + kRows - 1) / kRows;
  const int64_t job = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  const int64_t seq = job / ((int64_t)a.H * per_head);
  if (seq >= a.nseq) return;
  const int rest = (int)(job % ((int64_t)a.H * per_head)), h = rest / per_head;
  const int p0 = rest % per_head * kRows + lane / LN, n = lane % LN * 4;
  const int64_t slot = a.ci[seq];
  uint16_t* y = a.y + seq * a.y_ld + (int64_t)h * a.P;
  if (slot < 0 || slot >= a.slots) {
    if (lane % LN == 0)
      for (int k = 0; k < kRowsHeld; ++k)
        if (p0 + k * (64 / LN) < a.P) y[p0 + k * (64 / LN)] = 0;
    return;
  }
  float* S = a.pool + slot * a.s_slot + (int64_t)h * a.P * a.N;
  const bool n_in = n < a.N;
  f32x4 st[kRowsHeld];
#pragma unroll
  for (int k = 0; k < kRowsHeld; ++k) {
    const int p = p0 + k * (64 / LN);
    const float* src = S + (int64_t)(p < a.P ? p : 0) * a.N + (n_in ? n : 0);
    if constexpr (VEC) {
      st[k] = __builtin_nontemporal_load(reinterpret_cast<const f32x4_a4*>(src));
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) st[k][e] = src[n + e < a.N ? e : 0];
    }
  }
  const float step = step_size(load_num(a.dt, seq * a.dt_ld + h, a.f32) + (a.bias ? a.bias[h] : 0.f), a.softplus);
  const float decay = ex2(step * (a.A[h] * kLog2e));
  const float rate = a.beta_max / (1.f + ex2(-kLog2e * load_num(a.b, seq * a.b_ld + h, a.f32)));
  const int64_t gn = (int64_t)(h / (a.H / a.G)) * a.N;
  f32x4 kv, qv;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const bool in = n + e < a.N;
    const int64_t o = gn + (in ? n + e : 0);
    const float x = bf_f32(a.k[seq * a.k_ld + o]), z = bf_f32(a.q[seq * a.q_ld + o]);
    kv[e] = in ? x : 0.f;
    qv[e] = in ? z : 0.f;
  }
  float kk = 0.f, qq = 0.f, kq = 0.f;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    kk = __builtin_fmaf(kv[e], kv[e], kk);
    qq = __builtin_fmaf(qv[e], qv[e], qq);
    kq = __builtin_fmaf(kv[e], qv[e], kq);
  }
  kk = lanes_sum<LN>(kk), qq = lanes_sum<LN>(qq), kq = lanes_sum<LN>(kq);
  // kk - kk: a NaN where the sum is not finite
  const float kn = a.qk_norm ? rsqrtf(kk + a.norm_eps) + (kk - kk) : 1.f;
  const float qn = (a.qk_norm ? rsqrtf(qq + a.norm_eps) + (qq - qq) : 1.f) * a.scale;
  float sk[kRowsHeld], sq[kRowsHeld];
#pragma unroll
  for (int k = 0; k < kRowsHeld; ++k) {
    sk[k] = sq[k] = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float s = n + e < a.N ? st[k][e] : 0.f;  // places past the columns hold other values
      sk[k] = __builtin_fmaf(s, kv[e], sk[k]);
      sq[k] = __builtin_fmaf(s, qv[e], sq[k]);
    }
  }
#pragma unroll
  for (int k = 0; k < kRowsHeld; ++k) sk[k] = lanes_sum<LN>(sk[k]), sq[k] = lanes_sum<LN>(sq[k]);
#pragma unroll
  for (int k = 0; k < kRowsHeld; ++k) {
    const int p = p0 + k * (64 / LN);
    const float v = bf_f32(a.v[seq * a.v_ld + (int64_t)h * a.P + (p < a.P ? p : 0)]);
    const float u = rate * (v - decay * (kn * sk[k])) * kn;  // times the key's factor
#pragma unroll
    for (int e = 0; e < 4; ++e) st[k][e] = __builtin_fmaf(u, kv[e], decay * st[k][e]);
    if (p < a.P && n_in) {
      float* dst = S + (int64_t)p * a.N + n;
      if constexpr (VEC) {
        __builtin_nontemporal_store(st[k], reinterpret_cast<f32x4_a4*>(dst));
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (n + e < a.N) dst[e] = st[k][e];
      }
    }
    if (lane % LN == 0 && p < a.P) y[p] = to_bf16(qn * (decay * sq[k] + u * kq));
  }
}

template <int LN>
static void launch(const DeltaStepArgs& a, hipStream_t s) {
  constexpr int kRows = 64 / LN * kRowsHeld;
  const int64_t jobs = a.nseq * a.H * ((a.P + kRows - 1) / kRows);
  const dim3 grid((uint32_t)((jobs + 3) / 4));
  if (a.N % 4 == 0) delta_step_kernel<LN, true><<<grid, 256, 0, s>>>(a);
  else delta_step_kernel<LN, false><<<grid, 256, 0, s>>>(a);
}

hipError_t launch_delta_step(const DeltaStepArgs& a, hipStream_t s) {
  if (a.N <= 16) launch<4>(a, s);
  else if (a.N <= 32) launch<8>(a, s);
  else if (a.N <= 64) launch<16>(a, s);
  else if (a.N <= 128) launch<32>(a, s);
  else launch<64>(a, s);
  return hipGetLastError();
}

}  // namespace cssm
