// ss_conv_tm.cu -- time-major causal depthwise conv1d + SiLU over the packed
// x|B|C projection of a Mamba-2 layer, for sm_100a.
//
// "Mamba" (stanleyjacob.dev), Part IV Stage 2, in the layout the Mamba-2 scan
// reads (time-major, channels contiguous):
//   pre[t,c] = bias[c] + sum_{k<W} w[c,k] xin[t-(W-1)+k, c],  y = SiLU(pre)
// xin is x inside the token's own sequence and, before its start, the window
// kept in the sequence's cache slot (or zero).  The output columns are cut
// into up to three contiguous arrays (x, B, C), which is what the scan takes.
//
// Both passes are bound by HBM: forward 2 + 2 bytes per element in bf16
// against W FMAs and two SFU operations.  A thread owns V adjacent channels
// (one 16-byte load a token) and walks a tile of tokens with the W-1 previous
// inputs in registers, four tokens' loads in flight.
//
// Forward: tiles never straddle two sequences (ss_ragged.cuh), so only a
// sequence's first tile needs the incoming window, and the threads that read
// it are the ones that write the new window over it: no second launch and no
// race between reader and writer.
//
// Backward (no window: training starts every sequence from zero): strips of
// the token axis whatever the sequences.  dx[t] needs dpre[t .. t+W-1], so a
// strip recomputes dpre for W-1 tokens behind it.  dw and dbias stay in
// registers over the strip, go to one partial per strip, and a second kernel
// sums the strips in order: no atomics, bitwise reproducible.
#include "ss_device.cuh"
#include "ss_internal.h"
#include "ss_ragged.cuh"

namespace ss {

static __device__ unsigned int g_fault_conv_tm = 0;

namespace {

// V elements of a row as loaded: 16 bytes (V > 1) or one element.
template <typename T, int V>
struct Raw {
  static constexpr int kWords = V * (int)sizeof(T) / 4;
  uint32_t w[kWords];
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (kWords == 4) {
      const uint4 v = __ldg(reinterpret_cast<const uint4*>(p));
      w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
    } else if constexpr (kWords == 2) {
      const uint2 v = __ldg(reinterpret_cast<const uint2*>(p));
      w[0] = v.x; w[1] = v.y;
    }
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = 0u;
  }
  __device__ __forceinline__ float at(int i) const { return Elt<T>::to_f(reinterpret_cast<const T*>(w)[i]); }
};
template <typename T>
struct Raw<T, 1> {
  T v;
  __device__ __forceinline__ void load(const T* p) { v = *p; }
  __device__ __forceinline__ void zero() { v = Elt<T>::from_f(0.f); }
  __device__ __forceinline__ float at(int) const { return Elt<T>::to_f(v); }
};
template <typename T, int V>
__device__ __forceinline__ void store_v(T* p, const float (&f)[V]) {
  if constexpr (V == 1) {
    *p = Elt<T>::from_f(f[0]);
  } else {
    uint32_t w[V * sizeof(T) / 4];
    T* e = reinterpret_cast<T*>(w);
#pragma unroll
    for (int i = 0; i < V; ++i) e[i] = Elt<T>::from_f(f[i]);
    if constexpr (sizeof(w) == 16) *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    else *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
  }
}

__device__ __forceinline__ float silu_f(float x) { return x * sigmoid_f(x); }

// The piece that holds channel c, and c's place in it.
struct PieceAt {
  void* p;
  int width, col;
};
__device__ __forceinline__ PieceAt piece_at(const Pieces& y, int c) {
  int i = 0;
  if (c >= y.width[0]) { c -= y.width[0]; i = 1; }
  if (i == 1 && c >= y.width[1]) { c -= y.width[1]; i = 2; }
  return {i == 0 ? y.p[0] : i == 1 ? y.p[1] : y.p[2], i == 0 ? y.width[0] : i == 1 ? y.width[1] : y.width[2], c};
}

template <typename T, int V, int W>
__global__ void __launch_bounds__(128) conv_tm_fwd_kernel(const ConvTmParams p, int tile) {
  if (blockIdx.x == 0 && blockIdx.y == 0) check_offsets(p.seq, &g_fault_conv_tm);
  const RaggedTile rt = ragged_tile(p.seq, blockIdx.x, tile);
  const int s = rt.begin + rt.k * tile;
  if (rt.k > 0 && s >= rt.end) return;
  int slot = -1;
  if (p.slots.count > 0) {
    slot = claim_slot(p.slots, rt.seq, &g_fault_conv_tm);
    if (slot < 0) return;
  }
  const int c = (blockIdx.y * blockDim.x + threadIdx.x) * V;
  if (c >= p.dim) return;

  constexpr int H = W > 1 ? W - 1 : 1;
  const T* __restrict__ x = static_cast<const T*>(p.x) + c;
  float wk[W][V], bv[V], win[H][V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    bv[i] = p.bias ? p.bias[c + i] : 0.f;
#pragma unroll
    for (int k = 0; k < W; ++k) wk[k][i] = p.w[(size_t)(c + i) * W + k];
#pragma unroll
    for (int k = 0; k < H; ++k) win[k][i] = 0.f;
  }
  const bool first = rt.k == 0;
  float* st = p.slots.count > 0 ? p.state + ((size_t)slot * p.dim + c) * (W - 1) : nullptr;
  if (W > 1) {
    if (first) {
      if (st && !(p.slots.fresh && p.slots.fresh[rt.seq])) {
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
          for (int k = 0; k < W - 1; ++k) win[k][i] = st[i * (W - 1) + k];
      }
    } else {
#pragma unroll
      for (int k = 0; k < W - 1; ++k) {  // a tile holds at least W - 1 tokens: these are the sequence's own
        Raw<T, V> r;
        r.load(x + (int64_t)(s - (W - 1) + k) * p.ldx);
#pragma unroll
        for (int i = 0; i < V; ++i) win[k][i] = r.at(i);
      }
    }
  }
  if (W > 1 && first && st) {  // the window after the sequence: its last W-1 inputs, old entries where it is shorter
    const int len = rt.end - rt.begin;
#pragma unroll
    for (int k = 0; k < W - 1; ++k) {
      const int pos = len - (W - 1) + k;
      Raw<T, V> r;
      r.zero();
      if (pos >= 0) r.load(x + (int64_t)(rt.begin + pos) * p.ldx);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        float v = r.at(i);
#pragma unroll
        for (int j = 0; j < W - 1; ++j)
          if (pos < 0 && j == W - 1 + pos) v = win[j][i];
        st[i * (W - 1) + k] = v;
      }
    }
  }
  const PieceAt at = piece_at(p.y, c);
  T* __restrict__ y = static_cast<T*>(at.p) + at.col;
  const int e = min(rt.end, s + tile);
  constexpr int U = 4;
  for (int t = s; t < e; t += U) {
    Raw<T, V> r[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (t + u < e) r[u].load(x + (int64_t)(t + u) * p.ldx);
      else r[u].zero();
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (t + u >= e) break;
      float o[V];
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float xv = r[u].at(i);
        float pre = fmaf(wk[W - 1][i], xv, bv[i]);
#pragma unroll
        for (int k = 0; k < W - 1; ++k) pre = fmaf(wk[k][i], win[k][i], pre);
        o[i] = p.silu ? silu_f(pre) : pre;
#pragma unroll
        for (int k = 0; k + 1 < W - 1; ++k) win[k][i] = win[k + 1][i];
        if (W > 1) win[H - 1][i] = xv;
      }
      store_v<T, V>(y + (int64_t)(t + u) * at.width, o);
    }
  }
}

// The sequence walk of a strip: the position of each token in its sequence
// (-1 outside every sequence), advanced one token at a time.
struct Walk {
  int seq, begin, end;
  __device__ __forceinline__ void start(const Ragged& r, int t) {
    seq = begin = end = 0;
    if (r.nseq == 0) return;
    int lo = 0, hi = r.nseq - 1;
    while (lo < hi) {  // the last sequence that begins at or before t
      const int mid = (lo + hi + 1) >> 1;
      if (seq_begin(r, mid) <= t) lo = mid;
      else hi = mid - 1;
    }
    seq = lo;
    begin = seq_begin(r, seq);
    end = seq_end(r, seq, begin);
  }
  __device__ __forceinline__ int pos(const Ragged& r, int t) {
    while (t >= end && seq + 1 < r.nseq) {
      ++seq;
      begin = seq_begin(r, seq);
      end = seq_end(r, seq, begin);
    }
    return t >= begin && t < end ? t - begin : -1;
  }
};

template <typename T, int V, int W>
__global__ void __launch_bounds__(128) conv_tm_bwd_kernel(const ConvTmParams p) {
  if (blockIdx.x == 0 && blockIdx.y == 0) check_offsets(p.seq, &g_fault_conv_tm);
  const int c = (blockIdx.y * blockDim.x + threadIdx.x) * V;
  if (c >= p.dim) return;
  const int s = blockIdx.x * p.strip, e = min(p.seq.tokens, s + p.strip);
  constexpr int H = W > 1 ? W - 1 : 1;
  const T* __restrict__ x = static_cast<const T*>(p.x) + c;
  const PieceAt at = piece_at(p.y, c);
  const T* __restrict__ dy = static_cast<const T*>(at.p) + at.col;
  T* __restrict__ dx = static_cast<T*>(p.dx) + c;
  float wk[W][V], bv[V], win[H][V], dp[W][V], dwk[W][V], dbv[V];
  int ps[W];  // positions of tokens t-(W-1) .. t, or -1
#pragma unroll
  for (int i = 0; i < V; ++i) {
    bv[i] = p.bias ? p.bias[c + i] : 0.f;
    dbv[i] = 0.f;
#pragma unroll
    for (int k = 0; k < W; ++k) {
      wk[k][i] = p.w[(size_t)(c + i) * W + k];
      dwk[k][i] = 0.f;
      dp[k][i] = 0.f;
    }
  }
#pragma unroll
  for (int k = 0; k < W; ++k) ps[k] = -1;
#pragma unroll
  for (int k = 0; k < H; ++k) {  // the inputs before the strip; masked by position below
    Raw<T, V> r;
    r.zero();
    const int t = s - H + k;
    if (W > 1 && t >= 0) r.load(x + (int64_t)t * p.ldx);
#pragma unroll
    for (int i = 0; i < V; ++i) win[k][i] = r.at(i);
  }
  Walk walk;
  walk.start(p.seq, s);
  const int last = min(p.seq.tokens, e + W - 1);  // tokens whose dpre the strip needs
  constexpr int U = 2;
  for (int t = s; t < e + W - 1; t += U) {
    Raw<T, V> rx[U], rg[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      rx[u].zero();
      rg[u].zero();
      if (t + u < last) {
        rx[u].load(x + (int64_t)(t + u) * p.ldx);
        rg[u].load(dy + (int64_t)(t + u) * at.width);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int tt = t + u;
      if (tt >= e + W - 1) break;
      const int pos = tt < last ? walk.pos(p.seq, tt) : -1;
#pragma unroll
      for (int k = 0; k + 1 < W; ++k) ps[k] = ps[k + 1];
      ps[W - 1] = pos;
      const bool own = tt < e;  // else only dx of earlier tokens needs this dpre
      float dxv[V];
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float xv = rx[u].at(i);
        float tap[W];
#pragma unroll
        for (int k = 0; k < W - 1; ++k) tap[k] = pos >= W - 1 - k ? win[k][i] : 0.f;
        tap[W - 1] = xv;
        float pre = bv[i];
#pragma unroll
        for (int k = 0; k < W; ++k) pre = fmaf(wk[k][i], tap[k], pre);
        float d = rg[u].at(i);
        if (p.silu) {
          const float sg = sigmoid_f(pre);
          d *= sg * fmaf(pre, 1.f - sg, 1.f);
        }
        if (pos < 0) d = 0.f;  // a token of no sequence
        if (own && pos >= 0) {
          dbv[i] += d;
#pragma unroll
          for (int k = 0; k < W; ++k) dwk[k][i] = fmaf(d, tap[k], dwk[k][i]);
        }
#pragma unroll
        for (int k = 0; k + 1 < W; ++k) dp[k][i] = dp[k + 1][i];
        dp[W - 1][i] = d;
        // dx of token tt-(W-1): the dpre of the m-th token after it, where that is of the same sequence
        float a = 0.f;
#pragma unroll
        for (int m = 0; m < W; ++m)
          if (ps[0] >= 0 && ps[m] >= m) a = fmaf(wk[W - 1 - m][i], dp[m][i], a);
        dxv[i] = a;
#pragma unroll
        for (int k = 0; k + 1 < W - 1; ++k) win[k][i] = win[k + 1][i];
        if (W > 1) win[H - 1][i] = xv;
      }
      const int td = tt - (W - 1);
      if (td >= s) store_v<T, V>(dx + (int64_t)td * p.lddx, dxv);
    }
  }
  float* part = p.part + ((size_t)blockIdx.x * p.dim + c) * (W + 1);
#pragma unroll
  for (int i = 0; i < V; ++i) {
#pragma unroll
    for (int k = 0; k < W; ++k) part[i * (W + 1) + k] = dwk[k][i];
    part[i * (W + 1) + W] = dbv[i];
  }
}

// Sum of the strips' partials, in order within each of a block's 8 rows of
// threads and then over the 8.
__global__ void __launch_bounds__(256) conv_tm_reduce_kernel(const ConvTmParams p) {
  __shared__ float sh[8][32];
  const int lane = threadIdx.x & 31, row = threadIdx.x >> 5;
  const int n = p.dim * (p.width + 1);
  const int j = blockIdx.x * 32 + lane;
  float a = 0.f;
  if (j < n)
    for (int s = row; s < p.nstrip; s += 8) a += p.part[(size_t)s * n + j];
  sh[row][lane] = a;
  __syncthreads();
  if (row != 0 || j >= n) return;
#pragma unroll
  for (int r = 1; r < 8; ++r) a += sh[r][lane];
  const int c = j / (p.width + 1), k = j - c * (p.width + 1);
  if (k < p.width) p.dw[(size_t)c * p.width + k] = a;
  else if (p.dbias) p.dbias[c] = a;
}

// Blocks of at most 128 threads over `nvec` channel vectors: the width that
// leaves the fewest threads idle.
int block_threads(int nvec) {
  const int n0 = (nvec + 127) / 128;
  int best = 128, idle = INT32_MAX;
  for (int nb = n0; nb <= n0 + 2; ++nb) {
    const int nt = ((nvec + nb - 1) / nb + 31) / 32 * 32;
    if (nt >= 64 || nt >= nvec || nb == n0) {
      const int waste = nb * nt - nvec;
      if (nt <= 128 && waste < idle) { idle = waste; best = nt; }
    }
  }
  return best;
}

template <typename T, int V, int W>
cudaError_t run(const ConvTmParams& p, bool backward, int sms, cudaStream_t s) {
  const int nvec = (p.dim + V - 1) / V;
  const int nt = block_threads(nvec);
  const unsigned ny = (nvec + nt - 1) / nt;
  if (!backward) {
    // longer tiles re-read less (W-1 rows each); shorter ones keep every SM busy on few tokens
    int tile = 64;
    while (tile > 8 && (long long)(p.seq.tokens / tile) * ny * nt < (long long)sms * 1024) tile /= 2;
    const long long tiles = ragged_tiles(p.seq, tile);
    conv_tm_fwd_kernel<T, V, W><<<dim3((unsigned)tiles, ny), nt, 0, s>>>(p, tile);
    return cudaGetLastError();
  }
  if (p.nstrip > 0) {
    conv_tm_bwd_kernel<T, V, W><<<dim3((unsigned)p.nstrip, ny), nt, 0, s>>>(p);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  conv_tm_reduce_kernel<<<(unsigned)(((long long)p.dim * (W + 1) + 31) / 32), 256, 0, s>>>(p);
  return cudaGetLastError();
}

template <typename T, int V>
cudaError_t run_w(const ConvTmParams& p, bool backward, int sms, cudaStream_t s) {
  switch (p.width) {
    case 1: return run<T, V, 1>(p, backward, sms, s);
    case 2: return run<T, V, 2>(p, backward, sms, s);
    case 3: return run<T, V, 3>(p, backward, sms, s);
    case 4: return run<T, V, 4>(p, backward, sms, s);
  }
  return cudaErrorInvalidValue;
}

// Channels per thread: a 16-byte vector forward; backward, whose windows and
// sums need W times the registers, an 8-byte one for 16-bit types.
template <typename T>
cudaError_t run_t(const ConvTmParams& p, bool backward, bool vec, int sms, cudaStream_t s) {
  if (!vec) return run_w<T, 1>(p, backward, sms, s);
  return backward ? run_w<T, 4>(p, true, sms, s) : run_w<T, 16 / sizeof(T)>(p, false, sms, s);
}

cudaError_t dispatch(const ConvTmParams& p, bool backward, DType dt, bool vec, int sms, cudaStream_t s) {
  switch (dt) {
    case DType::F32: return run_t<float>(p, backward, vec, sms, s);
    case DType::BF16: return run_t<__nv_bfloat16>(p, backward, vec, sms, s);
    case DType::F16: return run_t<__half>(p, backward, vec, sms, s);
  }
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_conv_tm_fwd(const ConvTmParams& p, DType dt, bool vec, int sms, cudaStream_t s) {
  return dispatch(p, false, dt, vec, sms, s);
}
cudaError_t launch_conv_tm_bwd(const ConvTmParams& p, DType dt, bool vec, cudaStream_t s) {
  return dispatch(p, true, dt, vec, 0, s);
}

cudaError_t read_fault_conv_tm(unsigned* bits, bool clear) {
  cudaError_t e = cudaMemcpyFromSymbol(bits, g_fault_conv_tm, sizeof(unsigned));
  if (e != cudaSuccess || !clear) return e;
  const unsigned zero = 0;
  return cudaMemcpyToSymbol(g_fault_conv_tm, &zero, sizeof(unsigned));
}

}  // namespace ss
