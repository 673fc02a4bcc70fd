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
// against W FMAs and two SFU operations.  A thread owns 4 adjacent channels
// and walks a tile of tokens, four at a time, with the W-1 previous inputs in
// registers and the next rows on their way to its own shared-memory slots; two
// channels go through an instruction as an fp32 pair.  At 16384 x 5376 bf16 (352
// MB) the forward takes 69 us (5.1 TB/s): plain loads held it at 128, one token
// at a time at 77.
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
// sums the strips in order: no atomics, bitwise reproducible.  131 us at the
// same size (529 MB, 4.0 TB/s; the second kernel starts under the first).  W + 1
// products and the SiLU' of every token are formed, then 2 W more for dw and
// dx, 30 instructions an element.  Neither pipe is full (issue slots 58%, HBM
// 62%): latency bounds it, with the 16 warps that 128 registers leave an SM.  One
// token at a time, masked wherever it is, it took 191 us and 45 instructions; 5
// blocks per SM, in 96 registers, 170.
#include <type_traits>

#include "ss_device.cuh"
#include "ss_internal.h"
#include "ss_ragged.cuh"

namespace ss {

static __device__ unsigned int g_fault_conv_tm = 0;

namespace {

// One of the two 16-bit elements of a word, and two elements as a word.
template <typename T>
__device__ __forceinline__ float word_f(uint32_t w, int hi) {
  if constexpr (std::is_same<T, __nv_bfloat16>::value)
    return __uint_as_float(hi ? w & 0xffff0000u : w << 16);
  else
    return __half2float(__ushort_as_half(static_cast<unsigned short>(hi ? w >> 16 : w & 0xffffu)));
}
template <typename T>
__device__ __forceinline__ uint32_t word_of(float lo, float hi) {
  if constexpr (std::is_same<T, __nv_bfloat16>::value) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
  } else {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
}

// V elements of a row as loaded: 4 (8 bytes of a 16-bit type, 16 of fp32) or one.
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
  __device__ __forceinline__ float at(int i) const {
    if constexpr (sizeof(T) == 4) return __uint_as_float(w[i]);
    else return word_f<T>(w[i >> 1], i & 1);
  }
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
#pragma unroll
    for (int i = 0; i < V * (int)sizeof(T) / 4; ++i) {
      if constexpr (sizeof(T) == 4) w[i] = __float_as_uint(f[i]);
      else w[i] = word_of<T>(f[2 * i], f[2 * i + 1]);
    }
    if constexpr (sizeof(w) == 16) *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    else *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
  }
}

// A thread's own rows on their way from global to shared memory: D rows of one
// V-element vector per thread, copied asynchronously (cp.async) by the thread
// that reads them, so that no barrier is needed and loads in flight cost no
// registers.  Rows go in groups of kG.  Single elements (V == 1) are loaded
// when they are read.
constexpr int kG = 4;
template <typename T, int V>
struct Ring {
  static constexpr int kBytes = V * (int)sizeof(T);
  static constexpr int D = 32 / (int)sizeof(T);  // 16 rows of 16-bit types, 8 of fp32
  static constexpr int kPitch = 128 * kBytes;    // from row to row; a block has at most 128 threads
  static constexpr int kSize = V > 1 ? D * kPitch : 0;
  unsigned char* slot;  // this thread's, in row 0
  __device__ __forceinline__ void start(unsigned char* base) { slot = base + threadIdx.x * kBytes; }
  // Row k of the group that starts at row g (a multiple of kG).
  __device__ __forceinline__ unsigned char* at(int g, int k) const {
    return slot + (g & (D - 1)) * kPitch + k * kPitch;
  }
  __device__ __forceinline__ void put(int g, int k, const T* p) const {
    if constexpr (V > 1) {
      const unsigned to = static_cast<unsigned>(__cvta_generic_to_shared(at(g, k)));
      if constexpr (kBytes == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(to), "l"(p) : "memory");
      else
        asm volatile("cp.async.ca.shared.global [%0], [%1], 8;\n" ::"r"(to), "l"(p) : "memory");
    }
  }
  // The group at row g: rows p, p + ld, ..., the first n of them.
  __device__ __forceinline__ void put_group(int g, const T* p, int64_t ld, int n) const {
    if constexpr (V > 1) {
      if (n >= kG) {
#pragma unroll
        for (int k = 0; k < kG; ++k, p += ld) put(g, k, p);
      } else {
#pragma unroll
        for (int k = 0; k < kG - 1; ++k, p += ld)
          if (k < n) put(g, k, p);
      }
    }
  }
  __device__ __forceinline__ void get(int g, int k, const T* p, Raw<T, V>& r) const {
    if constexpr (V == 1) {
      r.load(p);
    } else if constexpr (kBytes == 16) {
      const uint4 v = *reinterpret_cast<const uint4*>(at(g, k));
      r.w[0] = v.x; r.w[1] = v.y; r.w[2] = v.z; r.w[3] = v.w;
    } else {
      const uint2 v = *reinterpret_cast<const uint2*>(at(g, k));
      r.w[0] = v.x; r.w[1] = v.y;
    }
  }
};

// Channels go through the arithmetic two at a time (packed fp32 pairs); of a
// single channel the high half is idle.
template <int V>
constexpr int pairs() { return (V + 1) / 2; }
template <typename T, int V>
__device__ __forceinline__ f2_t pair_at(const Raw<T, V>& r, int i) {
  if constexpr (V == 1) return pk2(r.at(0), 0.f);
  else return pk2(r.at(2 * i), r.at(2 * i + 1));
}
template <typename T, int V>
__device__ __forceinline__ void store_pairs(T* p, const f2_t (&f)[pairs<V>()]) {
  float o[V];
#pragma unroll
  for (int i = 0; i < V; ++i) o[i] = i & 1 ? hi2(f[i / 2]) : lo2(f[i / 2]);
  store_v<T, V>(p, o);
}
__device__ __forceinline__ f2_t silu_2(f2_t x) {
  const f2_t d = add2(pk2(1.f, 1.f), ex2_2(mul2(x, pk2(-kLog2e, -kLog2e))));
  return mul2(x, pk2(rcp(lo2(d)), rcp(hi2(d))));
}
// The taps of V adjacent channels, w (dim, W): contiguous, 16 bytes at a time
// where there is more than one channel (they are aligned then); and their biases.
template <int V, int W>
__device__ __forceinline__ void load_taps(const ConvTmParams& p, int c, f2_t (&wk)[W][pairs<V>()],
                                          f2_t (&bv)[pairs<V>()]) {
  const float* w = p.w + (size_t)c * W;
  float f[V * W];
  if constexpr (V * W % 4 == 0 && V > 1) {
#pragma unroll
    for (int i = 0; i < V * W; i += 4) {
      const float4 v = __ldg(reinterpret_cast<const float4*>(w + i));
      f[i] = v.x; f[i + 1] = v.y; f[i + 2] = v.z; f[i + 3] = v.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < V * W; ++i) f[i] = __ldg(w + i);
  }
#pragma unroll
  for (int i = 0; i < pairs<V>(); ++i) {
#pragma unroll
    for (int k = 0; k < W; ++k) wk[k][i] = pk2(f[2 * i * W + k], V > 1 ? f[(2 * i + 1) % V * W + k] : 0.f);
    bv[i] = p.bias ? pk2(p.bias[c + 2 * i], V > 1 ? p.bias[c + (2 * i + 1) % V] : 0.f) : pk2(0.f, 0.f);
  }
}

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
  // no tile of a sequence: ahead of the first one's first, or behind a sequence's last
  if (rt.k < 0 || (rt.k > 0 && (long long)rt.k * tile >= rt.end - rt.begin)) return;
  const int s = rt.begin + rt.k * tile;
  int slot = -1;
  if (p.slots.count > 0) {
    slot = claim_slot(p.slots, rt.seq, &g_fault_conv_tm);
    if (slot < 0) return;
  }
  const int c = (blockIdx.y * blockDim.x + threadIdx.x) * V;
  if (c >= p.dim) return;

  constexpr int H = W > 1 ? W - 1 : 1;
  const T* __restrict__ x = static_cast<const T*>(p.x) + c;
  const int e = min(rt.end, s + tile);
  extern __shared__ __align__(16) unsigned char smem[];
  Ring<T, V> ring;
  ring.start(smem);
#pragma unroll
  for (int g = 0; g < ring.D - kG; g += kG) {
    ring.put_group(g, x + (int64_t)(s + g) * p.ldx, p.ldx, e - s - g);
    cp_async_commit();
  }
  constexpr int NP = pairs<V>();
  f2_t wk[W][NP], bv[NP], win[H][NP];
  load_taps<V, W>(p, c, wk, bv);
#pragma unroll
  for (int i = 0; i < NP; ++i)
#pragma unroll
    for (int k = 0; k < H; ++k) win[k][i] = pk2(0.f, 0.f);
  const bool first = rt.k == 0;
  float* st = p.slots.count > 0 ? p.state + ((size_t)slot * p.dim + c) * (W - 1) : nullptr;
  if (W > 1) {
    if (first) {
      if (st && !(p.slots.fresh && p.slots.fresh[rt.seq])) {
#pragma unroll
        for (int i = 0; i < NP; ++i)
#pragma unroll
          for (int k = 0; k < W - 1; ++k)
            win[k][i] = pk2(st[2 * i * (W - 1) + k], V > 1 ? st[(2 * i + 1) % V * (W - 1) + k] : 0.f);
      }
    } else {
#pragma unroll
      for (int k = 0; k < W - 1; ++k) {  // a tile holds at least W - 1 tokens: these are the sequence's own
        Raw<T, V> r;
        r.load(x + (int64_t)(s - (W - 1) + k) * p.ldx);
#pragma unroll
        for (int i = 0; i < NP; ++i) win[k][i] = pair_at(r, i);
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
      for (int i = 0; i < NP; ++i) {
        f2_t v = pair_at(r, i);
#pragma unroll
        for (int j = k; j < W - 1; ++j)
          if (pos < 0 && j == W - 1 + pos) v = win[j][i];
        st[2 * i * (W - 1) + k] = lo2(v);
        if (V > 1) st[(2 * i + 1) % V * (W - 1) + k] = hi2(v);
      }
    }
  }
  const PieceAt at = piece_at(p.y, c);
  T* __restrict__ y = static_cast<T*>(at.p) + at.col;
  const int64_t ldx = p.ldx, ldy = at.width;
#pragma unroll 1
  for (int t = s; t < e; t += kG) {
    const int ahead = t + ring.D - kG;
    ring.put_group(ahead - s, x + (int64_t)ahead * ldx, ldx, e - ahead);
    cp_async_commit();
    cp_async_wait_group<ring.D / kG - 1>();
    const T* xt = x + (int64_t)t * ldx;
    T* yt = y + (int64_t)t * ldy;
    auto group = [&](auto whole) {
      Raw<T, V> r[kG];
#pragma unroll
      for (int k = 0; k < kG; ++k, xt += ldx) {
        r[k].zero();
        if (decltype(whole)::value || t + k < e) ring.get(t - s, k, xt, r[k]);
      }
#pragma unroll
      for (int k = 0; k < kG; ++k, yt += ldy) {
        f2_t o[NP];
#pragma unroll
        for (int i = 0; i < NP; ++i) {
          const f2_t xv = pair_at(r[k], i);
          o[i] = fma2(wk[W - 1][i], xv, bv[i]);
#pragma unroll
          for (int j = 0; j < W - 1; ++j) o[i] = fma2(wk[j][i], win[j][i], o[i]);
          if (p.silu) o[i] = silu_2(o[i]);
#pragma unroll
          for (int j = 0; j + 1 < W - 1; ++j) win[j][i] = win[j + 1][i];
          if (W > 1) win[H - 1][i] = xv;
        }
        if (decltype(whole)::value || t + k < e) store_pairs<T, V>(yt, o);
      }
    };
    if (t + kG <= e) group(std::true_type{});
    else group(std::false_type{});
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

template <typename T, int V, int W, bool SILU>
__global__ void __launch_bounds__(128) conv_tm_bwd_kernel(const ConvTmParams p) {
  pdl_trigger();
  if (blockIdx.x == 0 && blockIdx.y == 0) check_offsets(p.seq, &g_fault_conv_tm);
  const int c = (blockIdx.y * blockDim.x + threadIdx.x) * V;
  if (c >= p.dim) return;
  const int s = blockIdx.x * p.strip, e = min(p.seq.tokens, s + p.strip);
  constexpr int H = W > 1 ? W - 1 : 1;
  const T* __restrict__ x = static_cast<const T*>(p.x) + c;
  const PieceAt at = piece_at(p.y, c);
  const T* __restrict__ dy = static_cast<const T*>(at.p) + at.col;
  T* __restrict__ dx = static_cast<T*>(p.dx) + c;
  const int last = min(p.seq.tokens, e + W - 1);  // tokens whose dpre the strip needs
  extern __shared__ __align__(16) unsigned char smem[];
  const int64_t ldx = p.ldx, ldg = at.width, lddx = p.lddx;
  Ring<T, V> ringx, ringg;
  ringx.start(smem);
  ringg.start(smem + ringx.kSize);
#pragma unroll
  for (int g = 0; g < ringx.D - kG; g += kG) {
    ringx.put_group(g, x + (int64_t)(s + g) * ldx, ldx, last - s - g);
    ringg.put_group(g, dy + (int64_t)(s + g) * ldg, ldg, last - s - g);
    cp_async_commit();
  }
  constexpr int NP = pairs<V>();
  // win, dp: the inputs and dpre of the W-1 tokens before the one that comes next
  f2_t wk[W][NP], bv[NP], win[H][NP], dp[H][NP], dwk[W][NP], dbv[NP];
  load_taps<V, W>(p, c, wk, bv);
  int ps[W];  // positions of the last W tokens in their sequences, or -1
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    dbv[i] = pk2(0.f, 0.f);
#pragma unroll
    for (int k = 0; k < W; ++k) dwk[k][i] = pk2(0.f, 0.f);
#pragma unroll
    for (int k = 0; k < H; ++k) dp[k][i] = pk2(0.f, 0.f);
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
    for (int i = 0; i < NP; ++i) win[k][i] = pair_at(r, i);
  }
  Walk walk;
  walk.start(p.seq, s);
  const f2_t zero = pk2(0.f, 0.f), one = pk2(1.f, 1.f);
  // dL/dpre of a token from its dL/dy
  auto dpre = [&](f2_t pre, f2_t g) {
    if (!SILU) return g;
    const f2_t den = add2(one, ex2_2(mul2(pre, pk2(-kLog2e, -kLog2e))));
    const f2_t sg = pk2(rcp(lo2(den)), rcp(hi2(den)));
    return mul2(g, mul2(sg, fma2(pre, fma2(sg, pk2(-1.f, -1.f), one), one)));
  };
#pragma unroll 1
  for (int tt = s; tt < e + W - 1; tt += kG) {
    const int ahead = tt + ringx.D - kG;
    ringx.put_group(ahead - s, x + (int64_t)ahead * ldx, ldx, last - ahead);
    ringg.put_group(ahead - s, dy + (int64_t)ahead * ldg, ldg, last - ahead);
    cp_async_commit();
    cp_async_wait_group<ringx.D / kG - 1>();
    const T* xt = x + (int64_t)tt * ldx;
    const T* gt = dy + (int64_t)tt * ldg;
    T* dxt = dx + (int64_t)(tt - (W - 1)) * lddx;
    const int pos0 = tt < last ? walk.pos(p.seq, tt) : -1;
    // A group of the strip's own tokens, or the W-1 behind it, all in one sequence from its W-th token on: all
    // taps of each, and all tokens that dx of the tokens W-1 before takes, are of that sequence.  Nothing to mask.
    auto group = [&](auto own) {
      constexpr bool kOwn = decltype(own)::value;
      constexpr int kN = kOwn ? kG : W - 1;
      Raw<T, V> rx[kN], rg[kN];
#pragma unroll
      for (int k = 0; k < kN; ++k, xt += ldx, gt += ldg) {
        ringx.get(tt - s, k, xt, rx[k]);
        ringg.get(tt - s, k, gt, rg[k]);
      }
      f2_t dxv[kN][NP];
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        f2_t in[W - 1 + kN], d[W - 1 + kN];
#pragma unroll
        for (int k = 0; k < W - 1; ++k) {
          in[k] = win[k][i];
          d[k] = dp[k][i];
        }
#pragma unroll
        for (int k = 0; k < kN; ++k) {
          in[W - 1 + k] = pair_at(rx[k], i);
          f2_t pre = bv[i];
#pragma unroll
          for (int j = 0; j < W; ++j) pre = fma2(wk[j][i], in[k + j], pre);
          const f2_t dv = dpre(pre, pair_at(rg[k], i));
          d[W - 1 + k] = dv;
          if (kOwn) {
            dbv[i] = add2(dbv[i], dv);
#pragma unroll
            for (int j = 0; j < W; ++j) dwk[j][i] = fma2(dv, in[k + j], dwk[j][i]);
          }
        }
#pragma unroll
        for (int k = 0; k < kN; ++k) {
          f2_t a = zero;
#pragma unroll
          for (int m = 0; m < W; ++m) a = fma2(wk[W - 1 - m][i], d[k + m], a);
          dxv[k][i] = a;
        }
#pragma unroll
        for (int k = 0; k < W - 1; ++k) {
          win[k][i] = in[kN + k];
          dp[k][i] = d[kN + k];
        }
      }
#pragma unroll
      for (int k = 0; k < kN; ++k, dxt += lddx)
        if (k >= W - 1 || tt > s) store_pairs<T, V>(dxt, dxv[k]);  // (dx before the strip is another's)
#pragma unroll
      for (int k = 0; k < W; ++k) ps[k] = pos0 + kN - W + k;
    };
    if (pos0 >= W - 1 && tt + kG <= min(e, walk.end)) {
      group(std::true_type{});
      continue;
    }
    if constexpr (W > 1 && W - 1 <= kG) {
      if (pos0 >= W - 1 && tt == e && tt + W - 1 <= walk.end) {
        group(std::false_type{});
        break;
      }
    }
#pragma unroll 1
    for (int k = 0; k < kG && tt + k < e + W - 1; ++k, xt += ldx, gt += ldg, dxt += lddx) {
      const int t = tt + k;
      Raw<T, V> rx, rg;
      rx.zero();
      rg.zero();
      if (t < last) {
        ringx.get(tt - s, k, xt, rx);
        ringg.get(tt - s, k, gt, rg);
      }
      const int pos = t < last ? walk.pos(p.seq, t) : -1;
#pragma unroll
      for (int j = 0; j + 1 < W; ++j) ps[j] = ps[j + 1];
      ps[W - 1] = pos;
      f2_t dxv[NP];
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        f2_t in[W], d[W];
#pragma unroll
        for (int j = 0; j < W - 1; ++j) {
          in[j] = pos < W - 1 - j ? zero : win[j][i];
          d[j] = dp[j][i];
        }
        in[W - 1] = pair_at(rx, i);
        f2_t pre = bv[i];
#pragma unroll
        for (int j = 0; j < W; ++j) pre = fma2(wk[j][i], in[j], pre);
        const f2_t dv = pos < 0 ? zero : dpre(pre, pair_at(rg, i));  // (a token of no sequence)
        d[W - 1] = dv;
        if (t < e && pos >= 0) {  // else only dx of earlier tokens needs this dpre
          dbv[i] = add2(dbv[i], dv);
#pragma unroll
          for (int j = 0; j < W; ++j) dwk[j][i] = fma2(dv, in[j], dwk[j][i]);
        }
        // dx of token t-(W-1): the dpre of the m-th token after it, where that is of the same sequence
        f2_t a = zero;
#pragma unroll
        for (int m = 0; m < W; ++m)
          if (ps[0] >= 0 && ps[m] >= m) a = fma2(wk[W - 1 - m][i], d[m], a);
        dxv[i] = a;
#pragma unroll
        for (int j = 0; j + 1 < W - 1; ++j) win[j][i] = win[j + 1][i];
        if (W > 1) win[H - 1][i] = in[W - 1];
#pragma unroll
        for (int j = 0; j + 1 < W; ++j) dp[j][i] = d[j + 1];
      }
      if (t - (W - 1) >= s) store_pairs<T, V>(dxt, dxv);
    }
  }
  float* part = p.part + ((size_t)blockIdx.x * p.dim + c) * (W + 1);
#pragma unroll
  for (int i = 0; i < V; ++i) {
#pragma unroll
    for (int k = 0; k < W; ++k) part[i * (W + 1) + k] = i & 1 ? hi2(dwk[k][i / 2]) : lo2(dwk[k][i / 2]);
    part[i * (W + 1) + W] = i & 1 ? hi2(dbv[i / 2]) : lo2(dbv[i / 2]);
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
  pdl_wait();
  if (j < n)
#pragma unroll 8
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
    int tile = 32;
    while (tile > 8 && (long long)(p.seq.tokens / tile) * ny * nt < (long long)sms * 1024) tile /= 2;
    const long long tiles = ragged_tiles(p.seq, tile);
    conv_tm_fwd_kernel<T, V, W><<<dim3((unsigned)tiles, ny), nt, Ring<T, V>::kSize, s>>>(p, tile);
    return cudaGetLastError();
  }
  if (p.nstrip > 0) {
    const size_t smem = 2 * Ring<T, V>::kSize;
    if (p.silu) conv_tm_bwd_kernel<T, V, W, true><<<dim3((unsigned)p.nstrip, ny), nt, smem, s>>>(p);
    else conv_tm_bwd_kernel<T, V, W, false><<<dim3((unsigned)p.nstrip, ny), nt, smem, s>>>(p);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  return launch_behind(conv_tm_reduce_kernel, (unsigned)(((long long)p.dim * (W + 1) + 31) / 32), 256, 0, s,
                       p);
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

// Channels per thread: 4 where rows are aligned, whatever the type: the windows,
// taps and sums of more would not fit the registers of the backward.
template <typename T>
cudaError_t run_t(const ConvTmParams& p, bool backward, bool vec, int sms, cudaStream_t s) {
  if (!vec) return run_w<T, 1>(p, backward, sms, s);
  return run_w<T, 4>(p, backward, sms, s);
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
