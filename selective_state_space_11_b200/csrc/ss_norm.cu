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
// Bound by HBM: forward 3 arrays, backward 5.  A thread holds 8 columns of a
// group, so a group of G columns takes ceil(G / 256) warps and a block as many
// groups as fill 20 warps; the group's sum meets in shared memory, in a fixed
// order.  Blocks walk their rows, and a row's loads are under way while the row
// before is summed and written: each array moves once, and HBM does not wait
// for the block's barrier.  The backward keeps w and dw in registers over its
// rows, writes one partial row per walker, and a second kernel sums those in
// order: no atomics, bitwise reproducible.  All sums are fp32.
// Measured at 16384 x 5120 bf16, one group: forward 108 us (4.7 TB/s of 503 MB),
// backward 163 us (5.1 TB/s of 839 MB); with 4 columns per thread, one product
// at a time and the next row not on its way, 151 and 429 us.  A ring of rows in
// shared memory instead of registers took 146 and 230 us.
#include <type_traits>

#include "ss_device.cuh"
#include "ss_internal.h"

namespace ss {
namespace {

constexpr int kE = 8;  // columns per thread

// A thread's columns of one row, as loaded.  Vector rows: 8 adjacent ones (16
// or 32 bytes); others: single ones, a group's threads apart.
template <typename T, bool VEC>
struct Cols {
  static constexpr int kWords = kE * (int)sizeof(T) / 4;
  uint32_t w[kWords];
  __device__ __forceinline__ void load(const T* row, int t, int nt, int n) {
    if constexpr (VEC) {
      if (t * kE < n) {
#pragma unroll
        for (int i = 0; i < kWords / 4; ++i) {
          const uint4 v = __ldg(reinterpret_cast<const uint4*>(row + t * kE) + i);
          w[4 * i] = v.x; w[4 * i + 1] = v.y; w[4 * i + 2] = v.z; w[4 * i + 3] = v.w;
        }
        return;
      }
      zero();
    } else if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < kE; ++i)
        w[i] = t + i * nt < n ? __ldg(reinterpret_cast<const uint32_t*>(row) + t + i * nt) : 0u;
    } else {
      const unsigned short* r = reinterpret_cast<const unsigned short*>(row);
#pragma unroll
      for (int i = 0; i < kWords; ++i) {
        const uint32_t a = t + 2 * i * nt < n ? __ldg(r + t + 2 * i * nt) : 0u;
        const uint32_t b = t + (2 * i + 1) * nt < n ? __ldg(r + t + (2 * i + 1) * nt) : 0u;
        w[i] = a | (b << 16);
      }
    }
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = 0u;
  }
  __device__ __forceinline__ f2_t pair(int i) const {
    if constexpr (std::is_same<T, __half>::value) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      return pk2(f.x, f.y);
    } else {
      return pk2(at(2 * i), at(2 * i + 1));
    }
  }
  __device__ __forceinline__ float at(int i) const {
    if constexpr (sizeof(T) == 4) return __uint_as_float(w[i]);
    else if constexpr (std::is_same<T, __nv_bfloat16>::value)
      return __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
    else
      return __half2float(__ushort_as_half(static_cast<unsigned short>(i & 1 ? w[i / 2] >> 16 : w[i / 2] & 0xffffu)));
  }
};
template <typename T, bool VEC>
__device__ __forceinline__ void store_cols(T* row, int t, int nt, int n, const float (&f)[kE]) {
  if constexpr (VEC) {
    if (t * kE < n) store8(row + t * kE, f);
  } else {
#pragma unroll
    for (int i = 0; i < kE; ++i)
      if (t + i * nt < n) stf(row + t + i * nt, f[i]);
  }
}

__device__ __forceinline__ f2_t sigmoid_2(f2_t x) {
  const f2_t d = add2(pk2(1.f, 1.f), ex2_2(mul2(x, pk2(-kLog2e, -kLog2e))));
  return pk2(rcp(lo2(d)), rcp(hi2(d)));
}
template <typename T, bool VEC>
__device__ __forceinline__ void store_pairs(T* row, int t, int nt, int n, const f2_t (&f)[kE / 2]) {
  float o[kE];
#pragma unroll
  for (int i = 0; i < kE; ++i) o[i] = i & 1 ? hi2(f[i / 2]) : lo2(f[i / 2]);
  store_cols<T, VEC>(row, t, nt, n, o);
}

// Sum over the `warps` warps of a group; every thread gets it.  `sh` holds a
// float per warp; the caller alternates two of them between calls.
__device__ __forceinline__ float group_sum(float v, float* sh, int warps) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (warps == 1) return v;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (lane == 0) sh[warp] = v;
  __syncthreads();
  v = lane < warps ? sh[warp / warps * warps + lane] : 0.f;
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// GATE: there is a z; LAST: its gate multiplies the normalised row.
template <typename T, bool VEC, int THREADS, bool GATE, bool LAST>
__global__ void __launch_bounds__(THREADS, THREADS == 640 ? 2 : 1) norm_fwd_kernel(const NormParams p) {
  __shared__ float sh[2][32];
  const int nt = p.warps * 32, slot = threadIdx.x / nt, t = threadIdx.x - slot * nt, n = p.group;
  const int ngroups = p.dim / n;
  const int64_t items = p.rows * ngroups, step = (int64_t)gridDim.x * p.slots;
  Cols<T, VEC> x, z, ax, az;  // this row's, and the next one's on their way
  auto fetch = [&](int64_t item) {
    ax.zero();
    az.zero();
    if (item >= items) return;
    const int64_t row = ngroups == 1 ? item : item / ngroups;
    const int c0 = (int)(item - row * ngroups) * n;
    ax.load(static_cast<const T*>(p.x) + row * p.ldx + c0, t, nt, n);
    if (GATE) az.load(static_cast<const T*>(p.z) + row * p.ldz + c0, t, nt, n);
  };
  fetch((int64_t)blockIdx.x * p.slots + slot);
  int flip = 0;
  // every slot of a block makes the same number of turns (the sum holds a block barrier)
  for (int64_t base = (int64_t)blockIdx.x * p.slots; base < items; base += step, flip ^= 1) {
    const int64_t item = base + slot;
    x = ax;
    z = az;
    fetch(item + step);
    f2_t v[kE / 2], gate[kE / 2], sq = pk2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < kE / 2; ++i) {
      v[i] = x.pair(i);
      if (GATE) {
        gate[i] = mul2(z.pair(i), sigmoid_2(z.pair(i)));
        if (!LAST) v[i] = mul2(v[i], gate[i]);
      }
      sq = fma2(v[i], v[i], sq);
    }
    const float ss = group_sum(lo2(sq) + hi2(sq), sh[flip], p.warps);
    if (item >= items) continue;
    const float rstd = rsqrtf(ss / n + p.eps);
    const int64_t row = ngroups == 1 ? item : item / ngroups;
    const int c0 = (int)(item - row * ngroups) * n;
    Cols<float, VEC> w;
    w.load(p.w + c0, t, nt, n);
    const f2_t rstd2 = pk2(rstd, rstd);
#pragma unroll
    for (int i = 0; i < kE / 2; ++i) {
      v[i] = mul2(mul2(v[i], rstd2), w.pair(i));
      if (GATE && LAST) v[i] = mul2(v[i], gate[i]);
    }
    store_pairs<T, VEC>(static_cast<T*>(p.y) + row * p.dim + c0, t, nt, n, v);
    if (p.rstd && t == 0) p.rstd[item] = rstd;
  }
}

// GATE: there is a z; LAST: its gate multiplies the normalised row.
template <typename T, bool VEC, int THREADS, bool GATE, bool LAST>
__global__ void __launch_bounds__(THREADS) norm_bwd_kernel(const NormParams p) {
  __shared__ float sh[2][32];
  const int nt = p.warps * 32, slot = threadIdx.x / nt, t = threadIdx.x - slot * nt, n = p.group;
  const int g = blockIdx.y, ngroups = gridDim.y, c0 = g * n;
  const int64_t step = (int64_t)p.nblk * p.slots;
  Cols<float, VEC> w;
  w.load(p.w + c0, t, nt, n);
  f2_t dw[kE / 2];
#pragma unroll
  for (int i = 0; i < kE / 2; ++i) dw[i] = pk2(0.f, 0.f);
  Cols<T, VEC> x, z, d, ax, az, ad;
  float rstd = 0.f, arstd = 0.f;
  auto fetch = [&](int64_t row) {
    ax.zero();
    az.zero();
    ad.zero();
    arstd = 0.f;
    if (row >= p.rows) return;
    ax.load(static_cast<const T*>(p.x) + row * p.ldx + c0, t, nt, n);
    if (GATE) az.load(static_cast<const T*>(p.z) + row * p.ldz + c0, t, nt, n);
    ad.load(static_cast<const T*>(p.dy) + row * p.dim + c0, t, nt, n);
    arstd = p.rstd[row * ngroups + g];
  };
  fetch((int64_t)blockIdx.x * p.slots + slot);
  int flip = 0;
  for (int64_t base = (int64_t)blockIdx.x * p.slots; base < p.rows; base += step, flip ^= 1) {
    const int64_t row = base + slot;
    x = ax;
    z = az;
    d = ad;
    rstd = arstd;
    fetch(row + step);
    const f2_t rstd2 = pk2(rstd, rstd), one = pk2(1.f, 1.f), minus = pk2(-1.f, -1.f);
    f2_t sg[kE / 2], nv[kE / 2], dn[kE / 2], sum = pk2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < kE / 2; ++i) {
      f2_t q = d.pair(i);
      nv[i] = mul2(x.pair(i), rstd2);
      if (GATE) {
        sg[i] = sigmoid_2(z.pair(i));
        const f2_t gate = mul2(z.pair(i), sg[i]);
        if (LAST) q = mul2(q, gate);
        else nv[i] = mul2(nv[i], gate);
      }
      dw[i] = fma2(q, nv[i], dw[i]);
      dn[i] = mul2(q, w.pair(i));
      sum = fma2(dn[i], nv[i], sum);
    }
    const float c = group_sum(lo2(sum) + hi2(sum), sh[flip], p.warps) / n;
    if (row >= p.rows) continue;
    const f2_t c2 = pk2(-c, -c);
    f2_t ox[kE / 2], oz[kE / 2];
#pragma unroll
    for (int i = 0; i < kE / 2; ++i) {
      ox[i] = mul2(rstd2, fma2(nv[i], c2, dn[i]));  // dv
      if (GATE) {
        const f2_t zv = z.pair(i), dgate = mul2(sg[i], fma2(zv, fma2(sg[i], minus, one), one));
        if (LAST) {
          oz[i] = mul2(mul2(d.pair(i), w.pair(i)), mul2(nv[i], dgate));
        } else {
          oz[i] = mul2(mul2(ox[i], x.pair(i)), dgate);
          ox[i] = mul2(ox[i], mul2(zv, sg[i]));
        }
      }
    }
    store_pairs<T, VEC>(static_cast<T*>(p.dx) + row * p.lddx + c0, t, nt, n, ox);
    if (GATE) store_pairs<T, VEC>(static_cast<T*>(p.dz) + row * p.lddz + c0, t, nt, n, oz);
  }
  float* part = p.part + (size_t)(blockIdx.x * p.slots + slot) * p.dim + c0;
  store_pairs<float, VEC>(part, t, nt, n, dw);
}

__global__ void __launch_bounds__(256) norm_reduce_kernel(const NormParams p, int parts) {
  __shared__ float sh[8][32];
  const int lane = threadIdx.x & 31, row = threadIdx.x >> 5;
  const int j = blockIdx.x * 32 + lane;
  float a = 0.f;
  if (j < p.dim)
#pragma unroll 8
    for (int s = row; s < parts; s += 8) a += p.part[(size_t)s * p.dim + j];
  sh[row][lane] = a;
  __syncthreads();
  if (row != 0 || j >= p.dim) return;
#pragma unroll
  for (int r = 1; r < 8; ++r) a += sh[r][lane];
  p.dw[j] = a;
}

template <typename T, bool VEC, int THREADS, bool GATE, bool LAST>
cudaError_t run(const NormParams& p, bool backward, int sms, cudaStream_t s) {
  const int ngroups = p.dim / p.group;
  if (!backward) {
    NormParams q = p;
    const int64_t items = p.rows * ngroups;
    while (q.slots > 1 && items < (int64_t)sms * q.slots) --q.slots;  // few rows: spread them over the SMs
    const int threads = q.slots * q.warps * 32;
    const int64_t need = (items + q.slots - 1) / q.slots;
    const int64_t most = (int64_t)sms * (1280 / threads > 0 ? 1280 / threads : 1);
    norm_fwd_kernel<T, VEC, THREADS, GATE, LAST><<<(unsigned)(need < most ? need : most), threads, 0, s>>>(q);
    return cudaGetLastError();
  }
  const int threads = p.slots * p.warps * 32;
  if (p.nblk > 0) {
    norm_bwd_kernel<T, VEC, THREADS, GATE, LAST><<<dim3(p.nblk, ngroups), threads, 0, s>>>(p);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  norm_reduce_kernel<<<(p.dim + 31) / 32, 256, 0, s>>>(p, p.nblk * p.slots);
  return cudaGetLastError();
}

template <typename T, bool VEC, int THREADS>
cudaError_t run_g(const NormParams& p, bool backward, int sms, cudaStream_t s) {
  if (!p.z) return run<T, VEC, THREADS, false, false>(p, backward, sms, s);
  return p.gate_last ? run<T, VEC, THREADS, true, true>(p, backward, sms, s)
                     : run<T, VEC, THREADS, true, false>(p, backward, sms, s);
}
template <typename T, bool VEC>
cudaError_t run_v(const NormParams& p, bool backward, int sms, cudaStream_t s) {
  // wide groups need the threads of a whole block and have half the registers each
  return p.slots * p.warps <= 20 ? run_g<T, VEC, 640>(p, backward, sms, s) : run_g<T, VEC, 1024>(p, backward, sms, s);
}
template <typename T>
cudaError_t run_t(const NormParams& p, bool backward, bool vec, int sms, cudaStream_t s) {
  return vec ? run_v<T, true>(p, backward, sms, s) : run_v<T, false>(p, backward, sms, s);
}

}  // namespace

void norm_shape(int group, int* warps, int* slots) {
  *warps = (group + 32 * kE - 1) / (32 * kE);
  *slots = *warps >= 20 ? 1 : 20 / *warps;
}

cudaError_t launch_gated_norm(const NormParams& p, bool backward, DType dt, bool vec, int sms, cudaStream_t s) {
  switch (dt) {
    case DType::F32: return run_t<float>(p, backward, vec, sms, s);
    case DType::BF16: return run_t<__nv_bfloat16>(p, backward, vec, sms, s);
    case DType::F16: return run_t<__half>(p, backward, vec, sms, s);
  }
  return cudaErrorInvalidValue;
}

}  // namespace ss
