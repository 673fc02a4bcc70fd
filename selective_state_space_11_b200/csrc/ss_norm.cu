// ss_norm.cu -- gated RMS norm over groups of columns, forward and backward,
// for sm_100a: the last operation of a Mamba-2 mixer before its output
// projection.
//
// Per row and group of G columns, s(z) = z sigmoid(z):
//   gate first (default):  v = x s(z),  n = v rstd,  y = n w
//   gate last:             v = x,       n = v rstd,  y = n w s(z)
//   rstd = 1 / sqrt(mean(v^2) + eps)        (no z: no gate, s = 1)
// Backward for <dy, y>, q = dy (gate last: dy s(z)), dn = q w,
// c = mean over the group of dn n:
//   dv = rstd (dn - n c),  dw = sum over rows of q n
//   gate first: dx = dv s(z),  dz = dv x s'(z)
//   gate last:  dx = dv,       dz = dy n w s'(z)
// with s'(z) = sigmoid(z) (1 + z (1 - sigmoid(z))).
//
// Bound by HBM: forward 3 arrays, backward 5.  A row's group lives in
// registers between the sum and the output, so each array moves once.  WPR
// warps share a group (several groups per 256-thread block when it is
// small); their sums meet in shared memory in a fixed order.  The backward
// walks rows with dw in registers, writes one partial row per walker, and a
// second kernel sums those in order: no atomics.  All sums are fp32.
#include "ss_device.cuh"
#include "ss_internal.h"

namespace ss {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;

// K vectors of V elements per thread of a group's WPR warps: vector i of the
// thread is vector t + i * WPR * 32 of the group.
template <typename T, int V>
struct Vec {
  float f[V];
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (V == 8) load8(p, f);
    else f[0] = ldf(p);
  }
  __device__ __forceinline__ void store(T* p) const {
    if constexpr (V == 8) store8(p, f);
    else stf(p, f[0]);
  }
};

// Sum over the WPR warps of a group; every thread gets it.  `sh` holds one
// float per warp; the caller alternates two of them between calls.
template <int WPR>
__device__ __forceinline__ float group_sum(float v, float* sh) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (WPR == 1) return v;
  const int warp = threadIdx.x >> 5;
  if ((threadIdx.x & 31) == 0) sh[warp] = v;
  __syncthreads();
  float a = 0.f;
#pragma unroll
  for (int i = 0; i < WPR; ++i) a += sh[warp / WPR * WPR + i];
  return a;
}

template <typename T, int V, int K, int WPR>
__global__ void __launch_bounds__(kThreads) norm_fwd_kernel(const NormParams p) {
  __shared__ float sh[kWarps];
  constexpr int kSlots = kWarps / WPR;
  const int ngroups = p.dim / p.group;
  const int64_t item = (int64_t)blockIdx.x * kSlots + threadIdx.x / (32 * WPR);
  const bool live = item < p.rows * ngroups;
  const int64_t row = live ? item / ngroups : 0;
  const int g = live ? (int)(item - row * ngroups) : 0;
  const int t = threadIdx.x % (32 * WPR);
  const int nvec = p.group / V;
  const int c0 = g * p.group;
  const T* x = static_cast<const T*>(p.x) + row * p.ldx + c0;
  const T* z = p.z ? static_cast<const T*>(p.z) + row * p.ldz + c0 : nullptr;
  Vec<T, V> v[K], gt[K];
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < K; ++i) {
    const int j = t + i * WPR * 32;
    if (live && j < nvec) {
      v[i].load(x + j * V);
      if (z) gt[i].load(z + j * V);
    } else {
#pragma unroll
      for (int e = 0; e < V; ++e) v[i].f[e] = gt[i].f[e] = 0.f;
    }
  }
#pragma unroll
  for (int i = 0; i < K; ++i)
#pragma unroll
    for (int e = 0; e < V; ++e) {
      if (z) {
        gt[i].f[e] *= sigmoid_f(gt[i].f[e]);
        if (!p.gate_last) v[i].f[e] *= gt[i].f[e];
      }
      ss = fmaf(v[i].f[e], v[i].f[e], ss);
    }
  ss = group_sum<WPR>(ss, sh);
  if (!live) return;
  const float rstd = rsqrtf(ss / p.group + p.eps);
  T* y = static_cast<T*>(p.y) + row * p.dim + c0;
#pragma unroll
  for (int i = 0; i < K; ++i) {
    const int j = t + i * WPR * 32;
    if (j >= nvec) break;
    Vec<float, V> w;
    w.load(p.w + c0 + j * V);
#pragma unroll
    for (int e = 0; e < V; ++e) {
      float o = v[i].f[e] * rstd * w.f[e];
      if (z && p.gate_last) o *= gt[i].f[e];
      v[i].f[e] = o;
    }
    v[i].store(y + j * V);
  }
  if (p.rstd && t == 0) p.rstd[item] = rstd;
}

template <typename T, int V, int K, int WPR>
__global__ void __launch_bounds__(kThreads) norm_bwd_kernel(const NormParams p) {
  __shared__ float sh[2][kWarps];
  constexpr int kSlots = kWarps / WPR;
  const int ngroups = p.dim / p.group;
  const int g = blockIdx.y;
  const int walker = blockIdx.x * kSlots + threadIdx.x / (32 * WPR);
  const int t = threadIdx.x % (32 * WPR);
  const int nvec = p.group / V;
  const int c0 = g * p.group;
  const int64_t step = (int64_t)p.nblk * kSlots;
  Vec<float, V> w[K], dw[K];
#pragma unroll
  for (int i = 0; i < K; ++i) {
    const int j = t + i * WPR * 32;
#pragma unroll
    for (int e = 0; e < V; ++e) w[i].f[e] = dw[i].f[e] = 0.f;
    if (j < nvec) w[i].load(p.w + c0 + j * V);
  }
  int flip = 0;
  // every slot of the block makes the same number of turns (the sum holds a block barrier)
  for (int64_t r0 = (int64_t)blockIdx.x * kSlots; r0 < p.rows; r0 += step, flip ^= 1) {
    const int64_t row = r0 + threadIdx.x / (32 * WPR);
    const bool live = row < p.rows;
    const T* x = static_cast<const T*>(p.x) + row * p.ldx + c0;
    const T* z = p.z ? static_cast<const T*>(p.z) + row * p.ldz + c0 : nullptr;
    const T* dy = static_cast<const T*>(p.dy) + row * p.dim + c0;
    Vec<T, V> vx[K], vz[K], vd[K];
#pragma unroll
    for (int i = 0; i < K; ++i) {
      const int j = t + i * WPR * 32;
#pragma unroll
      for (int e = 0; e < V; ++e) vx[i].f[e] = vz[i].f[e] = vd[i].f[e] = 0.f;
      if (live && j < nvec) {
        vx[i].load(x + j * V);
        vd[i].load(dy + j * V);
        if (z) vz[i].load(z + j * V);
      }
    }
    const float rstd = live ? p.rstd[row * ngroups + g] : 0.f;
    float c = 0.f;
#pragma unroll
    for (int i = 0; i < K; ++i)
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float zv = vz[i].f[e], sg = sigmoid_f(zv);
        const float gate = z ? zv * sg : 1.f;
        const float n = (p.gate_last ? vx[i].f[e] : vx[i].f[e] * gate) * rstd;
        const float q = p.gate_last ? vd[i].f[e] * gate : vd[i].f[e];
        dw[i].f[e] = fmaf(q, n, dw[i].f[e]);
        c = fmaf(q * w[i].f[e], n, c);
      }
    c = group_sum<WPR>(c, sh[flip]) / p.group;
    if (live) {
      T* dx = static_cast<T*>(p.dx) + row * p.lddx + c0;
      T* dz = z ? static_cast<T*>(p.dz) + row * p.lddz + c0 : nullptr;
#pragma unroll
      for (int i = 0; i < K; ++i) {
        const int j = t + i * WPR * 32;
        if (j >= nvec) break;
        Vec<T, V> ox, oz;
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const float zv = vz[i].f[e], sg = sigmoid_f(zv);
          const float gate = z ? zv * sg : 1.f, dgate = sg * fmaf(zv, 1.f - sg, 1.f);
          const float n = (p.gate_last ? vx[i].f[e] : vx[i].f[e] * gate) * rstd;
          const float dn = (p.gate_last ? vd[i].f[e] * gate : vd[i].f[e]) * w[i].f[e];
          const float dv = rstd * fmaf(-n, c, dn);
          ox.f[e] = p.gate_last ? dv : dv * gate;
          oz.f[e] = (p.gate_last ? vd[i].f[e] * n * w[i].f[e] : dv * vx[i].f[e]) * dgate;
        }
        ox.store(dx + j * V);
        if (z) oz.store(dz + j * V);
      }
    }
  }
  float* part = p.part + (size_t)walker * p.dim + c0;
#pragma unroll
  for (int i = 0; i < K; ++i) {
    const int j = t + i * WPR * 32;
    if (j < nvec) dw[i].store(part + j * V);
  }
}

__global__ void __launch_bounds__(256) norm_reduce_kernel(const NormParams p, int parts) {
  __shared__ float sh[8][32];
  const int lane = threadIdx.x & 31, row = threadIdx.x >> 5;
  const int j = blockIdx.x * 32 + lane;
  float a = 0.f;
  if (j < p.dim)
    for (int s = row; s < parts; s += 8) a += p.part[(size_t)s * p.dim + j];
  sh[row][lane] = a;
  __syncthreads();
  if (row != 0 || j >= p.dim) return;
#pragma unroll
  for (int r = 1; r < 8; ++r) a += sh[r][lane];
  p.dw[j] = a;
}

template <typename T, int V, int K, int WPR>
cudaError_t run(const NormParams& p, bool backward, cudaStream_t s) {
  constexpr int kSlots = kWarps / WPR;
  const int ngroups = p.dim / p.group;
  if (!backward) {
    const int64_t blocks = (p.rows * ngroups + kSlots - 1) / kSlots;
    norm_fwd_kernel<T, V, K, WPR><<<(unsigned)blocks, kThreads, 0, s>>>(p);
    return cudaGetLastError();
  }
  if (p.nblk > 0) {
    norm_bwd_kernel<T, V, K, WPR><<<dim3(p.nblk, ngroups), kThreads, 0, s>>>(p);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  norm_reduce_kernel<<<(p.dim + 31) / 32, 256, 0, s>>>(p, p.nblk * kSlots);
  return cudaGetLastError();
}

// Warps per group and vectors per thread: the fewest warps whose threads hold
// at most two vectors each, all eight (and more vectors) for wide groups.
template <typename T, int V>
cudaError_t run_shape(const NormParams& p, bool backward, cudaStream_t s) {
  const int nvec = p.group / V;
  if (nvec <= 32) return run<T, V, 1, 1>(p, backward, s);
  if (nvec <= 64) return run<T, V, 2, 1>(p, backward, s);
  if (nvec <= 128) return run<T, V, 2, 2>(p, backward, s);
  if (nvec <= 256) return run<T, V, 2, 4>(p, backward, s);
  if (nvec <= 512) return run<T, V, 2, 8>(p, backward, s);
  if (nvec <= 768) return run<T, V, 3, 8>(p, backward, s);
  if (nvec <= 1024) return run<T, V, 4, 8>(p, backward, s);
  if (V == 1 && nvec <= 8192) return run<T, V, V == 1 ? 32 : 1, 8>(p, backward, s);
  return cudaErrorInvalidValue;
}

template <typename T>
cudaError_t run_t(const NormParams& p, bool backward, bool vec, cudaStream_t s) {
  return vec ? run_shape<T, 8>(p, backward, s) : run_shape<T, 1>(p, backward, s);
}

}  // namespace

// Groups a block holds at once (as run_shape picks them).
int norm_slots(int group, bool vec) {
  const int nvec = vec ? group / 8 : group;
  return nvec <= 64 ? 8 : nvec <= 128 ? 4 : nvec <= 256 ? 2 : 1;
}

cudaError_t launch_gated_norm(const NormParams& p, bool backward, DType dt, bool vec, cudaStream_t s) {
  switch (dt) {
    case DType::F32: return run_t<float>(p, backward, vec, s);
    case DType::BF16: return run_t<__nv_bfloat16>(p, backward, vec, s);
    case DType::F16: return run_t<__half>(p, backward, vec, s);
  }
  return cudaErrorInvalidValue;
}

}  // namespace ss
