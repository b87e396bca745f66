// ssm_step.hip -- one token a sequence against the slot pool of FP32 states.
//
//   S = e^{dt A} S + dt x B^T,   y = S C + D x
// A stream over the states (read and written once): 8 bytes for 5 operations, bound by memory.  A lane
// holds four columns n of a row p; LN lanes (a power of two, up to 64) share a row, and a wave keeps kStepRows
// rows a lane in flight, so the whole of a small call is one memory round trip after the slot's.
#include "ssm_device.h"

namespace cssm {

// rows a lane holds: 64 sequences of 64 heads of 64 rows, N = 128, 50.3 us with 4 (5.4 TB/s), 52.3 with 8, 58 with 2,
// 56 with 16
constexpr int kStepRows = 4;

template <int LN, bool VEC>
__global__ __launch_bounds__(256) void ssm_step_kernel(StepArgs a) {
  constexpr int kRows = 64 / LN * kStepRows;  // rows a wave covers
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
      for (int k = 0; k < kStepRows; ++k)
        if (p0 + k * (64 / LN) < a.P) y[p0 + k * (64 / LN)] = 0;
    return;
  }
  float* S = a.pool + slot * a.s_slot + (int64_t)h * a.P * a.N;
  const bool n_in = n < a.N;
  f32x4 st[kStepRows];
#pragma unroll
  for (int k = 0; k < kStepRows; ++k) {
    const int p = p0 + k * (64 / LN);
    const float* src = S + (int64_t)(p < a.P ? p : 0) * a.N + (n_in ? n : 0);
    if constexpr (VEC) {
      st[k] = __builtin_nontemporal_load(reinterpret_cast<const f32x4_a4*>(src));
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) st[k][e] = src[n + e < a.N ? e : 0];
    }
  }
  const float d = step_size(load_num(a.dt, seq * a.dt_ld + h, a.dt_f32) + (a.bias ? a.bias[h] : 0.f), a.softplus);
  const float decay = ex2(d * (a.A[h] * kLog2e)), Dh = a.D ? a.D[h] : 0.f;
  const int64_t gn = (int64_t)(h / (a.H / a.G)) * a.N;
  f32x4 b, c;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const bool in = n + e < a.N;
    const int64_t o = gn + (in ? n + e : 0);
    const float bv = bf_f32(a.B[seq * a.B_ld + o]), cv = bf_f32(a.C[seq * a.C_ld + o]);
    b[e] = in ? bv : 0.f;
    c[e] = in ? cv : 0.f;
  }
#pragma unroll
  for (int k = 0; k < kStepRows; ++k) {
    const int p = p0 + k * (64 / LN);
    const float x = bf_f32(a.x[seq * a.x_ld + (int64_t)h * a.P + (p < a.P ? p : 0)]);
    const float dx = d * x;
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      st[k][e] = __builtin_fmaf(dx, b[e], decay * st[k][e]);
      s = __builtin_fmaf(st[k][e], n + e < a.N ? c[e] : 0.f, s);
    }
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
    s = n_in ? s : 0.f;  // lanes past the columns hold other rows' values
#pragma unroll
    for (int m = LN / 2; m > 0; m >>= 1) s += __shfl_xor(s, m);
    if (lane % LN == 0 && p < a.P) y[p] = to_bf16(s + Dh * x);
  }
}

template <int LN>
static void launch(const StepArgs& a, hipStream_t s) {
  constexpr int kRows = 64 / LN * kStepRows;
  const int64_t jobs = a.nseq * a.H * ((a.P + kRows - 1) / kRows);
  const dim3 grid((uint32_t)((jobs + 3) / 4));
  if (a.N % 4 == 0) ssm_step_kernel<LN, true><<<grid, 256, 0, s>>>(a);
  else ssm_step_kernel<LN, false><<<grid, 256, 0, s>>>(a);
}

hipError_t launch_step(const StepArgs& a, hipStream_t s) {
  if (a.N <= 16) launch<4>(a, s);
  else if (a.N <= 32) launch<8>(a, s);
  else if (a.N <= 64) launch<16>(a, s);
  else if (a.N <= 128) launch<32>(a, s);
  else launch<64>(a, s);
  return hipGetLastError();
}

}  // namespace cssm
