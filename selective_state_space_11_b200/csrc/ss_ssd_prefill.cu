// ss_ssd_prefill.cu -- the Mamba-2 SSD scan of ragged prompts on a cache of
// states, for sm_100a.
//
// "Mamba" (stanleyjacob.dev), Part V: per sequence and head h of group g,
//   Delta_t = softplus(dt_t + dt_bias_h)
//   H_t     = exp(Delta_t A_h) H_{t-1} + Delta_t x_t B_t^T          (64 x dstate)
//   y_t     = (H_t C_t + D_h x_t) * SiLU(z_t)                       (no gate: z null)
// H starts from the sequence's cache slot (or zero) and ends there.
//
// The plain recurrence: a block per (sequence, head), four threads per state
// row with a quarter of its columns in registers.
#include "ss_device.cuh"
#include "ss_internal.h"
#include "ss_ragged.cuh"

namespace ss {

static __device__ unsigned int g_fault_prefill = 0;

namespace {

constexpr int kP = 64, kStage = 16;

template <typename T, int N>
__global__ void __launch_bounds__(256) prefill_walk_kernel(const SsdPrefillParams p) {
  __shared__ float sB[kStage][N], sC[kStage][N], sx[kStage][kP], sdl[kStage], sdec[kStage];
  const int h = blockIdx.x, i = blockIdx.y, tid = threadIdx.x;
  const int begin = seq_begin(p.seq, i), end = seq_end(p.seq, i, begin);
  if (h == 0 && i == 0) check_offsets(p.seq, &g_fault_prefill);
  int slot = -1;
  if (p.state) {
    slot = claim_slot(p.slots, i, &g_fault_prefill);
    if (slot < 0) return;
  }
  const int g = h / (p.nheads / p.ngroups);
  const int row = tid >> 2, q = tid & 3;  // columns 4 (q + 4 j) .. +3
  float* st = p.state ? p.state + (((size_t)slot * p.nheads + h) * kP + row) * N : nullptr;
  float hv[N / 16][4];
#pragma unroll
  for (int j = 0; j < N / 16; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e)
      hv[j][e] = st && !(p.slots.fresh && p.slots.fresh[i]) ? st[4 * (q + 4 * j) + e] : 0.f;
  const float A2 = p.A[h] * kLog2e, Dh = p.D ? p.D[h] : 0.f, bias = p.dt_bias ? p.dt_bias[h] : 0.f;
  for (int t0 = begin; t0 < end; t0 += kStage) {
    const int nt = min(kStage, end - t0);
    __syncthreads();
    for (int k = tid; k < nt * N; k += 256) {
      const int t = k / N, n = k - t * N;
      sB[t][n] = ldf(static_cast<const T*>(p.B) + (int64_t)(t0 + t) * p.ldb + g * N + n);
      sC[t][n] = ldf(static_cast<const T*>(p.C) + (int64_t)(t0 + t) * p.ldc + g * N + n);
    }
    for (int k = tid; k < nt * kP; k += 256)
      sx[k / kP][k % kP] = ldf(static_cast<const T*>(p.x) + (int64_t)(t0 + k / kP) * p.ldx + h * kP + k % kP);
    if (tid < nt) {
      const float v = ldf(static_cast<const T*>(p.dt) + (int64_t)(t0 + tid) * p.lddt + h) + bias;
      sdl[tid] = p.softplus ? softplus_f(v) : v;
      sdec[tid] = ex2(sdl[tid] * A2);
    }
    __syncthreads();
    for (int t = 0; t < nt; ++t) {
      const float xv = sx[t][row], u = sdl[t] * xv, dec = sdec[t];
      float a = 0.f;
#pragma unroll
      for (int j = 0; j < N / 16; ++j) {
        const float4 b = *reinterpret_cast<const float4*>(&sB[t][4 * (q + 4 * j)]);
        const float4 c = *reinterpret_cast<const float4*>(&sC[t][4 * (q + 4 * j)]);
        hv[j][0] = fmaf(dec, hv[j][0], u * b.x);
        hv[j][1] = fmaf(dec, hv[j][1], u * b.y);
        hv[j][2] = fmaf(dec, hv[j][2], u * b.z);
        hv[j][3] = fmaf(dec, hv[j][3], u * b.w);
        a = fmaf(hv[j][0], c.x, fmaf(hv[j][1], c.y, fmaf(hv[j][2], c.z, fmaf(hv[j][3], c.w, a))));
      }
      a += __shfl_xor_sync(0xffffffffu, a, 1);
      a += __shfl_xor_sync(0xffffffffu, a, 2);
      if (q == 0) {
        float o = fmaf(Dh, xv, a);
        if (p.z) {
          const float zv = ldf(static_cast<const T*>(p.z) + (int64_t)(t0 + t) * p.ldz + h * kP + row);
          o *= zv * sigmoid_f(zv);
        }
        stf(static_cast<T*>(p.y) + ((int64_t)(t0 + t) * p.nheads + h) * kP + row, o);
      }
    }
  }
  if (st)
#pragma unroll
    for (int j = 0; j < N / 16; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) st[4 * (q + 4 * j) + e] = hv[j][e];
}

template <typename T>
cudaError_t run_t(const SsdPrefillParams& p, cudaStream_t s) {
  const dim3 grid(p.nheads, p.seq.nseq);
  if (p.dstate == 128) prefill_walk_kernel<T, 128><<<grid, 256, 0, s>>>(p);
  else prefill_walk_kernel<T, 64><<<grid, 256, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_ssd_prefill(const SsdPrefillParams& p, DType dt, cudaStream_t s) {
  switch (dt) {
    case DType::BF16: return run_t<__nv_bfloat16>(p, s);
    case DType::F16: return run_t<__half>(p, s);
    default: return cudaErrorInvalidValue;
  }
}

cudaError_t read_fault_prefill(unsigned* bits, bool clear) {
  cudaError_t e = cudaMemcpyFromSymbol(bits, g_fault_prefill, sizeof(unsigned));
  if (e != cudaSuccess || !clear) return e;
  const unsigned zero = 0;
  return cudaMemcpyToSymbol(g_fault_prefill, &zero, sizeof(unsigned));
}

}  // namespace ss
