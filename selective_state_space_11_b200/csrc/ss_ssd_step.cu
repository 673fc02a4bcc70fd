// ss_ssd_step.cu -- one decode token of a Mamba-2 layer between its two
// projections, for sm_100a: the causal convolution's window advance, then the
// state update and read-out, on cached states picked by slot.
//
// "Mamba" (stanleyjacob.dev), Part IV Stage 7 (one token in, a fixed-size
// state updated in place, one token out) on the Part V recurrence.  Per
// request and head h of group g:
//   x|B|C  = SiLU(conv_bias + w . [window, xbc]);  the window drops its oldest input
//   Delta  = softplus(dt_h + dt_bias_h)
//   H      <- exp(Delta A_h) H + Delta x_h B_g^T
//   y_h    = (H C_g + D_h x_h) * SiLU(z_h)                       (no gate: z null)
//
// Bound by the state's bytes: 64 x dstate fp32 read and written per head.
// Every head of a group needs the group's convolved B and C, and only one
// reader may overwrite their window, so the convolution is a launch of its
// own; its fp32 outputs stay in L2.  The state kernel is launched with
// programmatic stream serialisation: its blocks start while the convolution
// runs and have their whole 64 x dstate state in registers (16-byte loads,
// all in flight) before they wait for it.  Those early loads are safe: the
// convolution's launch itself waited for everything before it, and it writes no state.
// Measured: 64 requests x 80 heads x 128, 345 MB, 64 us (5.4 TB/s, 84% of a
// copy's rate); 243 requests x 24 heads x 64, fp16, 203 MB, 38 us (5.3
// TB/s); one request of 24 heads 8.4 us, the time of two launches.
#include "ss_device.cuh"
#include "ss_internal.h"
#include "ss_ragged.cuh"

namespace ss {

static __device__ unsigned int g_fault_step = 0;

namespace {

constexpr int kP = 64;

template <typename T, int W>
__global__ void __launch_bounds__(128) step_conv_kernel(const SsdStepParams p) {
  pdl_trigger();
  const int b = blockIdx.x;
  const int slot = claim_slot(p.slots, b, &g_fault_step);
  const int c = blockIdx.y * 128 + threadIdx.x;
  const int dim = p.nheads * kP + 2 * p.ngroups * p.dstate;
  if (slot < 0 || c >= dim) return;
  const float xv = ldf(static_cast<const T*>(p.xbc) + (int64_t)b * p.ldx + c);
  float* st = p.conv_state + ((size_t)slot * dim + c) * (W - 1);
  float in[W];
#pragma unroll
  for (int k = 0; k < W - 1; ++k) in[k] = st[k];
  in[W - 1] = xv;
  float pre = p.bias ? p.bias[c] : 0.f;
#pragma unroll
  for (int k = 0; k < W; ++k) pre = fmaf(p.w[(size_t)c * W + k], in[k], pre);
#pragma unroll
  for (int k = 0; k < W - 1; ++k) st[k] = in[k + 1];
  p.xconv[(size_t)b * dim + c] = p.silu ? pre * sigmoid_f(pre) : pre;
}

// 128 threads per (request, head): N / 4 lanes hold a state row (one 16-byte
// vector each), so a warp covers 32 / (N / 4) rows at once and 16 in all.
template <typename T, int N>
__global__ void __launch_bounds__(128) step_state_kernel(const SsdStepParams p) {
  constexpr int kLanes = N / 4, kRows = 32 / kLanes, kIter = 16 / kRows;
  const int h = blockIdx.x, b = blockIdx.y;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int slot = claim_slot(p.slots, b, &g_fault_step);
  if (slot < 0) {
    pdl_wait();  // this launch ends behind the convolution's also when every request is skipped
    return;
  }
  const int n0 = (lane % kLanes) * 4;
  const int r0 = 16 * warp + lane / kLanes;  // rows r0 + i * kRows
  float4* st = reinterpret_cast<float4*>(p.state + ((size_t)slot * p.nheads + h) * kP * N + (size_t)r0 * N + n0);
  float4 hv[kIter];
#pragma unroll
  for (int i = 0; i < kIter; ++i) hv[i] = __ldcs(st + i * kRows * N / 4);
  const float dtv = ldf(static_cast<const T*>(p.dt) + (int64_t)b * p.lddt + h) + (p.dt_bias ? p.dt_bias[h] : 0.f);
  const float dl = p.softplus ? softplus_f(dtv) : dtv;
  const float dec = ex2(dl * p.A[h] * kLog2e);
  const float Dh = p.D ? p.D[h] : 0.f;
  pdl_wait();
  const int d = p.nheads * kP, g = h / (p.nheads / p.ngroups);
  const float* xc = p.xconv + (size_t)b * (d + 2 * p.ngroups * N);
  const float4 Bv = *reinterpret_cast<const float4*>(xc + d + g * N + n0);
  const float4 Cv = *reinterpret_cast<const float4*>(xc + d + (p.ngroups + g) * N + n0);
  const float* xh = xc + h * kP + r0;
  float acc[kIter];
#pragma unroll
  for (int i = 0; i < kIter; ++i) {
    const float u = dl * xh[i * kRows];
    hv[i].x = fmaf(dec, hv[i].x, u * Bv.x);
    hv[i].y = fmaf(dec, hv[i].y, u * Bv.y);
    hv[i].z = fmaf(dec, hv[i].z, u * Bv.z);
    hv[i].w = fmaf(dec, hv[i].w, u * Bv.w);
    __stcs(st + i * kRows * N / 4, hv[i]);
    acc[i] = fmaf(hv[i].x, Cv.x, fmaf(hv[i].y, Cv.y, fmaf(hv[i].z, Cv.z, hv[i].w * Cv.w)));
  }
#pragma unroll
  for (int i = 0; i < kIter; ++i)
#pragma unroll
    for (int o = kLanes / 2; o; o >>= 1) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], o);
#pragma unroll
  for (int i = 0; i < kIter; ++i) {
    if (lane % kLanes != i) continue;  // one lane of the row's finishes it
    const int r = r0 + i * kRows;
    float o = fmaf(Dh, xh[i * kRows], acc[i]);
    if (p.z) {
      const float zv = ldf(static_cast<const T*>(p.z) + (int64_t)b * p.ldz + h * kP + r);
      o *= zv * sigmoid_f(zv);
    }
    stf(static_cast<T*>(p.y) + ((size_t)b * p.nheads + h) * kP + r, o);
  }
}

template <typename T, int W>
cudaError_t run_conv(const SsdStepParams& p, cudaStream_t s) {
  const int dim = p.nheads * kP + 2 * p.ngroups * p.dstate;
  step_conv_kernel<T, W><<<dim3(p.batch, (dim + 127) / 128), 128, 0, s>>>(p);
  return cudaGetLastError();
}

template <typename T>
cudaError_t run_t(const SsdStepParams& p, cudaStream_t s) {
  cudaError_t e = cudaErrorInvalidValue;
  switch (p.width) {
    case 1: e = run_conv<T, 1>(p, s); break;
    case 2: e = run_conv<T, 2>(p, s); break;
    case 3: e = run_conv<T, 3>(p, s); break;
    case 4: e = run_conv<T, 4>(p, s); break;
  }
  if (e != cudaSuccess) return e;
  const dim3 grid(p.nheads, p.batch);
  return p.dstate == 128 ? launch_behind(step_state_kernel<T, 128>, grid, 128, 0, s, p)
                         : launch_behind(step_state_kernel<T, 64>, grid, 128, 0, s, p);
}

}  // namespace

cudaError_t launch_ssd_step(const SsdStepParams& p, DType dt, cudaStream_t s) {
  switch (dt) {
    case DType::F32: return run_t<float>(p, s);
    case DType::BF16: return run_t<__nv_bfloat16>(p, s);
    case DType::F16: return run_t<__half>(p, s);
  }
  return cudaErrorInvalidValue;
}

cudaError_t read_fault_step(unsigned* bits, bool clear) {
  cudaError_t e = cudaMemcpyFromSymbol(bits, g_fault_step, sizeof(unsigned));
  if (e != cudaSuccess || !clear) return e;
  const unsigned zero = 0;
  return cudaMemcpyToSymbol(g_fault_step, &zero, sizeof(unsigned));
}

}  // namespace ss
