// ss_ssd_prefill.cu -- the Mamba-2 SSD scan of ragged prompts on a cache of
// states, on the sm_100a tensor cores.
//
// "Mamba" (stanleyjacob.dev), Part V ("Mamba-2 and state-space duality"): per
// sequence and head h of group g,
//   Delta_t = softplus(dt_t + dt_bias_h)
//   H_t     = exp(Delta_t A_h) H_{t-1} + Delta_t x_t B_t^T          (64 x N, N = dstate)
//   y_t     = (H_t C_t + D_h x_t) * SiLU(z_t)                       (no gate: z null)
// H starts from the sequence's cache slot (or zero) and ends there.  With
// cs_t = A_h sum of Delta up to t inside a chunk of Q = 128 tokens, a chunk is
//   G  = C B^T                                              (Q x Q, shared by the group's heads)
//   M  = G o [exp(cs_i - cs_j) Delta_j]_{j <= i}
//   Y  = diag(exp cs) C H^T + M X                           H: the state entering the chunk
//   H <- exp(cs_last) H + Xw^T B,   Xw_t = exp(cs_last - cs_t) Delta_t x_t
//   y  = (Y + D x) SiLU(z)
//
// One block of 256 threads per SM takes two heads of a group at a time, so that
// G, B and C are formed and loaded once for both, every product has 128 rows,
// and the state update's accumulator [2 x 64 head rows][N] fills all TMEM lanes:
//   G   C (K-major)     x B (K-major)         128 x 128, K = N
//   Yc  C (K-major)     x H copy (K-major)    128 x 128, K = N
//   Ym  M_h (in TMEM)   x X_h (MN-major)      128 x 64 per head, K = 128
//   S   Xw^T (MN-major) x B (MN-major)        128 x N, K = 128, three times
// TMEM: G, then Ym | Yc | M_0, M_1 (16-bit, two per column) | S: all 512 columns.
//
// Roundings to 16 bits: M and the H copy, once each (the operands of y, which
// is itself rounded to 16 bits).  The state is not: Xw, a product of an fp32
// weight and a 16-bit input, goes through the tensor core as three 16-bit
// pieces whose sum is Xw to 24 bits, against the exact B, and H lives in fp32
// registers.  For fp16 the pieces are formed of Xw times a power of two that
// puts the chunk's largest product below 2^15 (undone exactly on S), so that
// small values do not fall out of fp16's range.
//
// Decays.  Exponents are formed from sums inside blocks of 32 tokens and the
// blocks' totals, never as differences of long prefix sums, so a strong decay
// loses no bits: exp(cs_i - cs_j) for j in an earlier block is
// exp(from the end of j's block to i) x exp(from j to the end of its block),
// both at most 1 for A < 0, and only the diagonal blocks take an exponential per
// element.
//
// Work split.  The chunks of all (sequence, head pair) units, in order, are
// cut into equal contiguous ranges, one per block; a planning kernel finds the
// cuts from the lengths in device memory.  A unit that a cut falls into is
// handed over: the block that has its first part runs that part first and
// publishes the state; the block with its last part runs that part last.  A
// block whose whole range lies inside one unit first runs its state products
// alone from zero, then adds the published state of the block before, decayed,
// publishes the sum and runs its range in full.  Blocks take their number from
// a counter, so a block only ever waits for one that has started; the wait is
// bounded all the same.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstring>
#include <type_traits>

#include "ss_device.cuh"
#include "ss_internal.h"
#include "ss_ragged.cuh"
#include "ss_tc.cuh"

namespace ss {

static __device__ unsigned int g_fault_prefill = 0;

namespace {

constexpr int kP = 64;         // head dimension
constexpr int kQ = 128;        // chunk length
constexpr int kThreads = 256;
constexpr uint32_t kWaitLimit = 1u << 22;
constexpr uint32_t kFlagLimit = 1u << 22;  // polls of a predecessor's flag
constexpr uint32_t kG = 0, kYc = 128, kM = 256, kS = 384;  // TMEM columns (Ym over G)

// Workspace: the plan, then the published states.
struct Cut {
  int seq, pair, chunk, nchunk;  // position of a range's first chunk; chunks of that sequence
};
__host__ __device__ inline size_t align256(size_t x) { return (x + 255) / 256 * 256; }
struct PlanLayout {
  size_t prefix, cuts, flags, carry, total;
};
__host__ __device__ inline PlanLayout plan_layout(int64_t nseq, int blocks, int dstate) {
  PlanLayout l;
  l.prefix = 0;                                              // long long [nseq + 1]: chunks before sequence i
  l.cuts = align256((nseq + 1) * sizeof(long long));         // Cut [blocks + 1]
  l.flags = l.cuts + align256((blocks + 1) * sizeof(Cut));   // unsigned [blocks], then the counter
  l.carry = l.flags + align256((blocks + 1) * sizeof(unsigned));
  l.total = l.carry + (size_t)blocks * 2 * kP * dstate * sizeof(float);
  return l;
}

// Fewest chunks worth a block of its own.
constexpr int kMinRange = 4;

__global__ void __launch_bounds__(1024) prefill_plan_kernel(const SsdPrefillParams p, int npairs, int blocks) {
  pdl_trigger();
  __shared__ long long s_warp[32];
  __shared__ long long s_base;
  const PlanLayout lay = plan_layout(p.seq.nseq, blocks, p.dstate);
  long long* prefix = reinterpret_cast<long long*>(static_cast<char*>(p.ws) + lay.prefix);
  Cut* cuts = reinterpret_cast<Cut*>(static_cast<char*>(p.ws) + lay.cuts);
  unsigned* flags = reinterpret_cast<unsigned*>(static_cast<char*>(p.ws) + lay.flags);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nseq = p.seq.nseq;
  check_offsets(p.seq, &g_fault_prefill);
  for (int i = tid; i <= blocks; i += 1024) flags[i] = 0;
  if (tid == 0) s_base = 0;
  __syncthreads();
  for (int i0 = 0; i0 < nseq; i0 += 1024) {
    const int i = i0 + tid;
    long long n = 0;
    if (i < nseq) {
      const int b = seq_begin(p.seq, i), e = seq_end(p.seq, i, b);
      n = e > b ? (e - b + kQ - 1) / kQ : 1;  // an empty sequence is a unit too: its state may have to be zeroed
    }
    long long run = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long v = __shfl_up_sync(0xffffffffu, run, o);
      if (lane >= o) run += v;
    }
    if (lane == 31) s_warp[warp] = run;
    __syncthreads();
    long long before = s_base;
    for (int w = 0; w < warp; ++w) before += s_warp[w];
    if (i < nseq) prefix[i] = before + run - n;
    if (i == nseq - 1) prefix[nseq] = before + run;
    __syncthreads();
    if (tid == 1023) s_base = before + run;
    __syncthreads();
  }
  const long long units = prefix[nseq] * npairs;
  const long long least = (units + kMinRange - 1) / kMinRange;
  const long long used = least < blocks ? least : blocks;
  for (int j = tid; j <= blocks; j += 1024) {
    Cut c{nseq, 0, 0, 0};
    if (j < used) {
      const long long lin = j * units / used;
      int lo = 0, hi = nseq - 1;
      while (lo < hi) {  // the last sequence whose chunks start at or before lin
        const int mid = (lo + hi + 1) >> 1;
        if (prefix[mid] * npairs <= lin) lo = mid;
        else hi = mid - 1;
      }
      c.seq = lo;
      c.nchunk = (int)(prefix[lo + 1] - prefix[lo]);
      const long long in = lin - prefix[lo] * npairs;
      c.pair = (int)(in / c.nchunk);
      c.chunk = (int)(in - (long long)c.pair * c.nchunk);
    }
    cuts[j] = c;
  }
}

// Byte offsets in the (1024-aligned) shared-memory block.
template <int N>
struct Lay {
  static constexpr int kTile = N * 256;               // 128 rows x N 16-bit
  static constexpr int kB = 0;                        // two of them
  static constexpr int kC = 2 * kTile;
  static constexpr int kX = kC + kTile;               // 2 heads x 128 rows x 128 B
  static constexpr int kW = kX + 32768;               // 3 pieces x 2 heads x 64 rows x 128 B
  static constexpr int kH = kW + 49152;               // 128 rows x N 16-bit
  static constexpr int kF = kH + kTile;               // float [2 heads][128]: 2^(to the end of the block) Delta
  static constexpr int kPre = kF + 1024;              // float [2][128]: log2 decay from the block's start
  static constexpr int kDl = kPre + 1024;             // float [2][128]: Delta
  static constexpr int kTot = kDl + 1024;             // float [2][4]: log2 decay of each block of 32
  static constexpr int kMax = kTot + 32;              // unsigned [2]: largest |x| of the chunk (fp16)
  static constexpr int kBars = kMax + 16;             // mbarriers
  static constexpr int kSlot = kBars + 80;
  static constexpr int kBytes = kSlot + 16;
  static constexpr int kAlloc = kBytes + 1024;
};
enum : int { kBarB0 = 0, kBarB1 = 1, kBarC = 2, kBarX = 3, kBarG = 4, kBarYc = 5, kBarS0 = 6, kBarYm = 7, kBarS1 = 8,
             kNumBars = 9 };

__device__ __forceinline__ uint32_t swz(int r, int c) {
  return static_cast<uint32_t>(r * 128 + ((c ^ (r & 7)) << 4));
}

template <typename T> struct Pk;
template <> struct Pk<__nv_bfloat16> {
  __device__ __forceinline__ static uint32_t pack(float lo, float hi) {
    __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&v);
  }
  __device__ __forceinline__ static float2 unpack(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  }
};
template <> struct Pk<__half> {
  __device__ __forceinline__ static uint32_t pack(float lo, float hi) {
    __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&v);
  }
  __device__ __forceinline__ static float2 unpack(uint32_t w) {
    return __half22float2(*reinterpret_cast<__half2*>(&w));
  }
};

template <typename T, int N>
__global__ void __launch_bounds__(kThreads, 1)
    prefill_tc_kernel(const SsdPrefillParams p, int npairs, int blocks, const __grid_constant__ CUtensorMap map_x,
                      const __grid_constant__ CUtensorMap map_b, const __grid_constant__ CUtensorMap map_c) {
  using L = Lay<N>;
  constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
  constexpr uint32_t kId = tc::idesc_f16(kBf16, 128, 128, false, false);  // G, Yc
  constexpr uint32_t kIdS = tc::idesc_f16(kBf16, 128, N, true, true);
  constexpr uint32_t kIdYm = tc::idesc_f16(kBf16, 128, 64, false, true);
  constexpr int HN = N / 2;          // state columns per thread
  constexpr int kMma = 0, kTma = 128;

  extern __shared__ unsigned char smem_raw[];
  const uint32_t raw = tc::saddr(smem_raw);
  const uint32_t pad = (1024u - (raw & 1023u)) & 1023u;
  unsigned char* const sm = smem_raw + pad;
  const uint32_t sb = raw + pad;
  float* const sF = reinterpret_cast<float*>(sm + L::kF);
  float* const sPre = reinterpret_cast<float*>(sm + L::kPre);
  float* const sDl = reinterpret_cast<float*>(sm + L::kDl);
  float* const sTot = reinterpret_cast<float*>(sm + L::kTot);
  unsigned* const sMax = reinterpret_cast<unsigned*>(sm + L::kMax);
  uint32_t* const sslot = reinterpret_cast<uint32_t*>(sm + L::kSlot);
  __shared__ unsigned s_block;
  auto bar = [&](int i) { return sb + L::kBars + 8u * static_cast<uint32_t>(i); };

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int wg = tid >> 7, row = tid & 127, blk = row >> 5;  // TMEM lane = row
  const uint32_t lane_base = static_cast<uint32_t>(32 * (warp & 3)) << 16;
  const int hrow = row >> 6;       // the head (of the two) of state row `row`

  if (tid == kMma) {
#pragma unroll
    for (int i = 0; i < kNumBars; ++i) tc::mbar_init(bar(i), 1);
    tc::fence_mbar_init();
  }
  if (tid == kTma) {
    tc::prefetch_map(&map_x);
    tc::prefetch_map(&map_b);
    tc::prefetch_map(&map_c);
  }
  if (warp == 0) tc::tmem_alloc(tc::saddr(sslot), 512);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = *sslot;
  {  // the blocks of M above the diagonal stay zero
    const uint32_t zero[16] = {};
    for (int j = blk + 1; j < 4; ++j) tc::st32x32b_x16(tmem + lane_base + kM + 64 * wg + 16 * j, zero);
    tc::st_wait();
  }
  pdl_wait();  // the plan is written

  char* const ws = static_cast<char*>(p.ws);
  const PlanLayout play = plan_layout(p.seq.nseq, blocks, N);
  const Cut* const cuts = reinterpret_cast<const Cut*>(ws + play.cuts);
  unsigned* const flags = reinterpret_cast<unsigned*>(ws + play.flags);
  float4* const carry = reinterpret_cast<float4*>(ws + play.carry);
  if (tid == 0) s_block = atomicAdd(flags + blocks, 1u);
  __syncthreads();
  const int me = (int)s_block;
  const Cut A = cuts[me], E = cuts[me + 1];

  // bookkeeping of armed barriers for the drain (copy thread: loads, MMA thread: products)
  uint32_t armed = 0, last_par = 0, next_par = 0;
  auto arm = [&](int i) {
    const uint32_t m = 1u << i;
    armed |= m;
    last_par = (last_par & ~m) | (next_par & m);
    next_par ^= m;
  };
  bool ok = true;
  auto fault = [&](unsigned bit) {
    atomicOr(&g_fault_prefill, bit);
    ok = false;
  };
  // parity of the next wait on each barrier, kept by every thread
  uint32_t phase = 0;
  auto wait = [&](int i, unsigned bit) {  // the same sequence of waits in every thread that waits
    if (!tc::wait(bar(i), (phase >> i) & 1u, kWaitLimit)) fault(bit);
  };
  auto flip = [&](int i) { phase ^= 1u << i; };

  float hs[HN];
  const int per = p.nheads / p.ngroups, ppg = (per + 1) / 2;  // heads and pairs per group
  const bool same = A.seq == E.seq && A.pair == E.pair;
  const bool middle = same && A.chunk > 0 && E.chunk > 0;
  int stage = middle ? 0 : E.chunk > 0 ? 2 : 3;
  if (A.seq >= p.seq.nseq) stage = 6;
  int useq = A.seq, upair = A.pair;  // cursor of the whole units
  if (!middle && A.chunk > 0) {
    if (++upair == npairs) { upair = 0; ++useq; }
  }
  uint32_t it = 0;  // chunks so far: which B buffer is next

  while (stage < 6) {
    // ---- the next run: a unit, its chunks [c0, c1), where its state comes from and goes to
    int seq, pair, c0, c1 = -1;
    bool full = true, from_slot = true, from_carry = false, publish = false, to_slot = false;
    if (stage == 0) {         // middle: the range's own state, from zero
      seq = A.seq; pair = A.pair; c0 = A.chunk; c1 = E.chunk;
      full = from_slot = false;
      stage = 1;
    } else if (stage == 1) {  // middle: in full
      seq = A.seq; pair = A.pair; c0 = A.chunk; c1 = E.chunk;
      from_slot = false;
      from_carry = true;
      stage = 6;
    } else if (stage == 2) {  // the first part of the unit at the range's end
      seq = E.seq; pair = E.pair; c0 = 0; c1 = E.chunk;
      publish = true;
      stage = same ? 6 : 3;
    } else if (stage == 3) {  // whole units
      if (useq == E.seq && upair == E.pair) {
        stage = 4;
        continue;
      }
      seq = useq; pair = upair; c0 = 0;
      to_slot = true;
      if (++upair == npairs) { upair = 0; ++useq; }
    } else {                  // the last part of the unit at the range's start
      if (stage == 4 && A.chunk == 0) break;
      seq = A.seq; pair = A.pair; c0 = A.chunk;
      from_slot = false;
      from_carry = true;
      to_slot = true;
      stage = 6;
    }
    const int begin = seq_begin(p.seq, seq), end = seq_end(p.seq, seq, begin);
    if (c1 < 0) c1 = max(1, (end - begin + kQ - 1) / kQ);
    int slot = -1;
    if (p.state) {
      slot = claim_slot(p.slots, seq, &g_fault_prefill);
      if (slot < 0) {
        if (stage == 1) stage = 6;  // the middle of a skipped sequence
        continue;
      }
    }
    const int g = pair / ppg, h0 = g * per + 2 * (pair - g * ppg);
    const int nh2 = min(2, g * per + per - h0);  // an odd group's last pair holds one head
    const int h = h0 + min(wg, nh2 - 1);         // this thread's head for y
    const bool mine = wg < nh2, owns = hrow < nh2;
    const float A2 = p.A[h] * kLog2e, Dh = p.D ? p.D[h] : 0.f, bias = p.dt_bias ? p.dt_bias[h] : 0.f;
    const T* dtg = static_cast<const T*>(p.dt) + h;

    auto load = [&](int i, uint32_t off, const CUtensorMap* map, int col, int t, int nblocks) {
      tc::expect_tx(bar(i), 16384u * nblocks);
      for (int b = 0; b < nblocks; ++b) tc::tma_load_2d(sb + off + 16384u * b, map, col + 64 * b, t, bar(i));
      arm(i);
    };
    auto load_b = [&](int c, uint32_t k) { load(kBarB0 + (k & 1), L::kB + (k & 1) * L::kTile, &map_b, g * N, begin + c * kQ, N / 64); };
    auto load_c = [&](int c) { load(kBarC, L::kC, &map_c, g * N, begin + c * kQ, N / 64); };
    auto load_x = [&](int c) { load(kBarX, L::kX, &map_x, h0 * kP, begin + c * kQ, nh2); };
    const bool any = end > begin;
    if (tid == kTma && any) {
      load_b(c0, it);
      if (full) load_c(c0);
      load_x(c0);
    }
    T dtn = Elt<T>::from_f(0.f);
    if (begin + c0 * kQ + row < end) dtn = dtg[(int64_t)(begin + c0 * kQ + row) * p.lddt];

    // ---- the state entering the run
    float* st = p.state && owns ? p.state + (((size_t)slot * p.nheads + h0) * kP + row) * N + wg * HN : nullptr;
    if (from_carry) {
      if (tid == 0 && !middle) {  // the middle's first pass has waited already
        uint32_t polls = 0, v = 0;
        do {
          asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(flags + me - 1) : "memory");
        } while (!v && ++polls < kFlagLimit);
        if (!v) fault(2u);
      }
      if (__syncthreads_or(!ok)) break;
      const float4* src = carry + (size_t)(me - 1) * (2 * kP * N / 4);
#pragma unroll
      for (int i = 0; i < HN / 4; ++i) {
        const float4 v = __ldcg(src + i * kThreads + tid);
        hs[4 * i] = v.x; hs[4 * i + 1] = v.y; hs[4 * i + 2] = v.z; hs[4 * i + 3] = v.w;
      }
    } else if (from_slot && st && !(p.slots.fresh && p.slots.fresh[seq])) {
#pragma unroll
      for (int i = 0; i < HN / 4; ++i) {
        const float4 v = __ldcs(reinterpret_cast<const float4*>(st) + i);
        hs[4 * i] = v.x; hs[4 * i + 1] = v.y; hs[4 * i + 2] = v.z; hs[4 * i + 3] = v.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < HN; ++i) hs[i] = 0.f;
    }
    // its 16-bit copy, K-major rows of n
    auto write_copy = [&]() {
      unsigned char* base = sm + L::kH + (N == 128 ? wg * 16384 : 0);
      const int cb = N == 128 ? 0 : 4 * wg;
#pragma unroll
      for (int c = 0; c < HN / 8; ++c)
        *reinterpret_cast<uint4*>(base + swz(row, cb + c)) =
            make_uint4(Pk<T>::pack(hs[8 * c], hs[8 * c + 1]), Pk<T>::pack(hs[8 * c + 2], hs[8 * c + 3]),
                       Pk<T>::pack(hs[8 * c + 4], hs[8 * c + 5]), Pk<T>::pack(hs[8 * c + 6], hs[8 * c + 7]));
    };
    if (full) write_copy();
    if (nh2 == 1)  // the missing head's x is zero
      for (int i = tid; i < 1024; i += kThreads) *reinterpret_cast<uint4*>(sm + L::kX + 16384 + 16 * i) = make_uint4(0, 0, 0, 0);
    tc::fence_proxy_async();
    tc::fence_before();
    if (__syncthreads_or(!ok)) break;
    float psum = 0.f;  // log2 decay of the run so far (head hrow)

    bool stop = false;
    for (int c = c0; c < c1 && any; ++c, ++it) {
      const int t0 = begin + c * kQ, nval = min(kQ, end - t0);
      const bool more = c + 1 < c1;
      const int bb = kBarB0 + (it & 1);
      const uint32_t offB = L::kB + (it & 1) * L::kTile;
      // ---- G and Yc need only B, C and the state copy
      if (tid == kMma && full) {
        tc::fence_after();
        wait(bb, 1u);
        wait(kBarC, 1u);
        tc::fence_after();
        const uint64_t dc = tc::desc_sw128(sb + L::kC, 16, 1024), db = tc::desc_sw128(sb + offB, 16, 1024),
                       dh = tc::desc_sw128(sb + L::kH, 16, 1024);
#pragma unroll
        for (int kk = 0; kk < N / 16; ++kk) {
          const uint32_t ko = ((kk >> 2) * 16384 + (kk & 3) * 32) >> 4;
          tc::mma(tmem + kG, dc + ko, db + ko, kId, kk > 0);
        }
        tc::commit(bar(kBarG));
        arm(kBarG);
#pragma unroll
        for (int kk = 0; kk < N / 16; ++kk) {
          const uint32_t ko = ((kk >> 2) * 16384 + (kk & 3) * 32) >> 4;
          tc::mma(tmem + kYc, dc + ko, dh + ko, kId, kk > 0);
        }
        tc::commit(bar(kBarYc));
        arm(kBarYc);
      }
      __syncwarp();
      if (tid == kTma && more) load_b(c + 1, it + 1);  // its buffer's last reader, S of the chunk before, is done
      __syncwarp();
      // ---- Delta and the decays (thread: head wg, token row)
      float pre, suf;
      {
        float d = 0.f;
        if (row < nval && mine) {
          const float v = Elt<T>::to_f(dtn) + bias;
          d = p.softplus ? softplus_f(v) : v;
        }
        const float a = d * A2;
        pre = a;
        suf = a;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const float u = __shfl_up_sync(0xffffffffu, pre, o), v = __shfl_down_sync(0xffffffffu, suf, o);
          if (lane >= o) pre += u;
          if (lane + o < 32) suf += v;
        }
        if (lane == 31) sTot[4 * wg + blk] = pre;
        suf = __shfl_down_sync(0xffffffffu, suf, 1);  // the tokens after this one
        if (lane == 31) suf = 0.f;
        sF[tid] = ex2(suf) * d;
        sPre[tid] = pre;
        sDl[tid] = d;
        if (!kBf16 && tid < 2) sMax[tid] = 0u;
      }
      if (more && t0 + kQ + row < end) dtn = dtg[(int64_t)(t0 + kQ + row) * p.lddt];
      wait(kBarX, 1u);
      if (nval < kQ) {  // rows behind the sequence belong to others: no NaN of theirs may meet a zero weight
        wait(bb, 1u);
        if (full) wait(kBarG, 2u);
        const uint4 zero = make_uint4(0, 0, 0, 0);
        for (int i = tid; i < (kQ - nval) * 8; i += kThreads) {
          const uint32_t o = (nval + i / 8) * 128 + (i & 7) * 16;
#pragma unroll
          for (int b = 0; b < N / 64; ++b) *reinterpret_cast<uint4*>(sm + offB + 16384 * b + o) = zero;
          *reinterpret_cast<uint4*>(sm + L::kX + o) = zero;
          *reinterpret_cast<uint4*>(sm + L::kX + 16384 + o) = zero;
        }
        tc::fence_proxy_async();
      }
      if (__syncthreads_or(!ok)) { stop = true; break; }
      float unscale = 1.f;
      // ---- Xw of 64 tokens as three 16-bit pieces (thread: token tid % 64, 32 columns)
      const int xr = tid & 63, xh = tid >> 7, xc = ((tid >> 6) & 1) * 4;
      float scale = 1.f;
      if constexpr (!kBf16) {  // fp16: the power of two that puts max |x| max Delta below 2^15
        unsigned m = 0;
        const int xhead = tid >> 7;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const uint4 v = *reinterpret_cast<const uint4*>(sm + L::kX + xhead * 16384 + swz(row, k));
          m = __vmaxu2(m, __vmaxu2(__vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu), __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu)));
        }
        m = max(m & 0xffffu, m >> 16);
        float wmax = __half2float(__ushort_as_half((unsigned short)m)) * fabsf(sDl[tid]);
        wmax = wmax < 3.0e38f ? wmax : 1.f;
#pragma unroll
        for (int o = 16; o; o >>= 1) wmax = fmaxf(wmax, __shfl_xor_sync(0xffffffffu, wmax, o));
        if (lane == 0) atomicMax(sMax + xhead, __float_as_uint(wmax));
        if (__syncthreads_or(!ok)) { stop = true; break; }
        auto power = [](unsigned m) {  // 2^(14 - exponent of m), within fp32's range
          const int e = (int)(m >> 23) - 127;
          return m == 0 ? 0 : min(100, max(-100, 14 - e));
        };
        scale = __uint_as_float((unsigned)(127 + power(sMax[xhead])) << 23);
        unscale = __uint_as_float((unsigned)(127 - power(sMax[hrow])) << 23);
      }
      auto write_xw = [&](int half) {
        const int r = 64 * half + xr;
        float later = 0.f;
#pragma unroll
        for (int b = 1; b < 4; ++b)
          if (b > (r >> 5)) later += sTot[4 * xh + b];
        const float w = sF[128 * xh + r] * ex2(later) * scale;
        const unsigned char* xs = sm + L::kX + xh * 16384;
        unsigned char* wd = sm + L::kW + xh * 8192;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint4 xv = *reinterpret_cast<const uint4*>(xs + swz(r, xc + k));
          const uint32_t in[4] = {xv.x, xv.y, xv.z, xv.w};
          uint32_t a[4], b[4], d[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 f = Pk<T>::unpack(in[e]);
            const float v0 = f.x * w, v1 = f.y * w;
            a[e] = Pk<T>::pack(v0, v1);
            const float2 fa = Pk<T>::unpack(a[e]);
            const float r0 = v0 - fa.x, r1 = v1 - fa.y;
            b[e] = Pk<T>::pack(r0, r1);
            const float2 fb = Pk<T>::unpack(b[e]);
            d[e] = Pk<T>::pack(r0 - fb.x, r1 - fb.y);
          }
          const uint32_t o = swz(xr, xc + k);
          *reinterpret_cast<uint4*>(wd + o) = make_uint4(a[0], a[1], a[2], a[3]);
          *reinterpret_cast<uint4*>(wd + 16384 + o) = make_uint4(b[0], b[1], b[2], b[3]);
          *reinterpret_cast<uint4*>(wd + 32768 + o) = make_uint4(d[0], d[1], d[2], d[3]);
        }
        tc::fence_proxy_async();
      };
      auto issue_s = [&](int half, int b) {
        const uint64_t dbm = tc::desc_sw128(sb + offB + half * 8192, 16384, 1024);
#pragma unroll
        for (int q = 0; q < 3; ++q) {
          const uint64_t dw = tc::desc_sw128(sb + L::kW + 16384 * q, 8192, 1024);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            tc::mma(tmem + kS, dw + kk * (2048 >> 4), dbm + kk * (2048 >> 4), kIdS, (half | q | kk) != 0);
        }
        tc::commit(bar(b));
        arm(b);
      };
      write_xw(0);
      if (__syncthreads_or(!ok)) { stop = true; break; }
      if (tid == kMma) {
        if (!full) wait(bb, 1u);
        tc::fence_after();
        issue_s(0, kBarS0);
      }
      __syncwarp();
      // ---- M_h, row `row`, head wg
      if (full) {
        wait(kBarG, 2u);
        tc::fence_after();
        float between = 0.f;  // log2 decay of the blocks between j's and i's
        for (int j = blk; j >= 0; --j) {
          float gv[32];
          tc::ld32x32b_x32(tmem + lane_base + kG + 32 * j, gv);
          uint32_t mp[16];
          if (j == blk) {
            const float4* pr = reinterpret_cast<const float4*>(sPre + 128 * wg + 32 * j);
            const float4* dl = reinterpret_cast<const float4*>(sDl + 128 * wg + 32 * j);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const float4 pv = pr[k], dv = dl[k];
              float m[4] = {gv[4 * k] * ex2(pre - pv.x) * dv.x, gv[4 * k + 1] * ex2(pre - pv.y) * dv.y,
                            gv[4 * k + 2] * ex2(pre - pv.z) * dv.z, gv[4 * k + 3] * ex2(pre - pv.w) * dv.w};
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if (4 * k + e > lane) m[e] = 0.f;
              mp[2 * k] = Pk<T>::pack(m[0], m[1]);
              mp[2 * k + 1] = Pk<T>::pack(m[2], m[3]);
            }
          } else {
            const float ei = ex2(pre + between);
            between += sTot[4 * wg + j];
            const float4* fj = reinterpret_cast<const float4*>(sF + 128 * wg + 32 * j);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const float4 fv = fj[k];
              mp[2 * k] = Pk<T>::pack(gv[4 * k] * (ei * fv.x), gv[4 * k + 1] * (ei * fv.y));
              mp[2 * k + 1] = Pk<T>::pack(gv[4 * k + 2] * (ei * fv.z), gv[4 * k + 3] * (ei * fv.w));
            }
          }
          tc::st32x32b_x16(tmem + lane_base + kM + 64 * wg + 16 * j, mp);
        }
        tc::st_wait();
      }
      wait(kBarS0, 2u);
      write_xw(1);
      tc::fence_before();
      if (__syncthreads_or(!ok)) { stop = true; break; }
      if (tid == kMma) {
        tc::fence_after();
        if (full) {
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const uint64_t dx = tc::desc_sw128(sb + L::kX + 16384 * q, 16384, 1024);
#pragma unroll
            for (int kk = 0; kk < kQ / 16; ++kk)
              tc::mma_ta(tmem + kG + 64 * q, tmem + kM + 64 * q + 8 * kk, dx + kk * (2048 >> 4), kIdYm, kk > 0);
          }
          tc::commit(bar(kBarYm));
          arm(kBarYm);
        }
        issue_s(1, kBarS1);
      }
      __syncwarp();
      // ---- y = (2^cs Yc + Ym + D x) SiLU(z)
      if (full) {
        wait(kBarYc, 2u);
        if (tid == kTma && more) load_c(c + 1);
        wait(kBarYm, 2u);
        if (tid == kTma && more) load_x(c + 1);
        __syncwarp();
        tc::fence_after();
        float cs = pre;
        for (int b = 0; b < blk; ++b) cs += sTot[4 * wg + b];
        const float e = ex2(cs);
        const bool out = row < nval && mine;
        const int64_t t = t0 + row;
        const T* xg = static_cast<const T*>(p.x) + t * p.ldx + h * kP;
        const T* zg = p.z ? static_cast<const T*>(p.z) + t * p.ldz + h * kP : nullptr;
        T* yg = static_cast<T*>(p.y) + (t * p.nheads + h) * kP;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          float yc[16], ym[16];
          tc::ld32x32b_x16(tmem + lane_base + kYc + 64 * wg + 16 * k, yc);
          tc::ld32x32b_x16(tmem + lane_base + kG + 64 * wg + 16 * k, ym);
          if (out) {
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              float xv[8], o[8];
              load8(xg + 16 * k + 8 * u, xv);
#pragma unroll
              for (int v = 0; v < 8; ++v) o[v] = fmaf(Dh, xv[v], fmaf(e, yc[8 * u + v], ym[8 * u + v]));
              if (zg) {
#pragma unroll
                for (int v = 0; v < 8; ++v) {
                  const float zv = ldf(zg + 16 * k + 8 * u + v);
                  o[v] *= zv * sigmoid_f(zv);
                }
              }
              store8(yg + 16 * k + 8 * u, o);
            }
          }
        }
      }
      // ---- H <- 2^cs_last H + S
      wait(kBarS1, 2u);
      if (!full && tid == kTma && more) load_x(c + 1);
      __syncwarp();
      tc::fence_after();
      {
        const float tot = (sTot[4 * hrow] + sTot[4 * hrow + 1]) + (sTot[4 * hrow + 2] + sTot[4 * hrow + 3]);
        psum += tot;
        const float dec = ex2(tot);
#pragma unroll
        for (int k = 0; k < HN; k += 16) {
          float sv[16];
          tc::ld32x32b_x16(tmem + lane_base + kS + wg * HN + k, sv);
#pragma unroll
          for (int i = 0; i < 16; ++i) hs[k + i] = fmaf(dec, hs[k + i], kBf16 ? sv[i] : sv[i] * unscale);
        }
        if (full && more) write_copy();  // C H^T of this chunk is done with the old copy
      }
      flip(bb);
      flip(kBarX);
      flip(kBarS0);
      flip(kBarS1);
      if (full) {
        flip(kBarC);
        flip(kBarG);
        flip(kBarYc);
        flip(kBarYm);
      }
      tc::fence_proxy_async();
      tc::fence_before();
      if (__syncthreads_or(!ok)) { stop = true; break; }
      tc::fence_after();
    }
    if (stop) break;

    // ---- the state leaving the run
    if (!full) {  // the middle of a unit: add what enters it, decayed
      if (tid == 0) {
        uint32_t polls = 0, v = 0;
        do {
          asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(flags + me - 1) : "memory");
        } while (!v && ++polls < kFlagLimit);
        if (!v) fault(2u);
      }
      if (__syncthreads_or(!ok)) break;
      const float dec = ex2(psum);
      const float4* src = carry + (size_t)(me - 1) * (2 * kP * N / 4);
#pragma unroll
      for (int i = 0; i < HN / 4; ++i) {
        const float4 v = __ldcg(src + i * kThreads + tid);
        hs[4 * i] = fmaf(dec, v.x, hs[4 * i]);
        hs[4 * i + 1] = fmaf(dec, v.y, hs[4 * i + 1]);
        hs[4 * i + 2] = fmaf(dec, v.z, hs[4 * i + 2]);
        hs[4 * i + 3] = fmaf(dec, v.w, hs[4 * i + 3]);
      }
      publish = true;
    }
    if (publish) {
      float4* dst = carry + (size_t)me * (2 * kP * N / 4);
#pragma unroll
      for (int i = 0; i < HN / 4; ++i)
        dst[i * kThreads + tid] = make_float4(hs[4 * i], hs[4 * i + 1], hs[4 * i + 2], hs[4 * i + 3]);
      __threadfence();
      __syncthreads();
      if (tid == 0) asm volatile("st.release.gpu.global.u32 [%0], 1;" ::"l"(flags + me) : "memory");
    } else if (to_slot && st) {
#pragma unroll
      for (int i = 0; i < HN / 4; ++i)
        __stcs(reinterpret_cast<float4*>(st) + i, make_float4(hs[4 * i], hs[4 * i + 1], hs[4 * i + 2], hs[4 * i + 3]));
    }
  }

  // Drain: copies and products in flight must be done before shared memory and
  // TMEM are given back (a no-op on the normal path).
  if (tid == kMma || tid == kTma) {
#pragma unroll
    for (int i = 0; i < kNumBars; ++i)
      if ((armed >> i) & 1u)
        if (!tc::wait(bar(i), (last_par >> i) & 1u, kWaitLimit)) atomicOr(&g_fault_prefill, 4u);
  }
  tc::fence_before();
  __syncthreads();
  if (warp == 0) {
    tc::fence_after();
    tc::tmem_dealloc(tmem, 512);
  }
}

int pairs(const SsdPrefillParams& p) { return p.ngroups * ((p.nheads / p.ngroups + 1) / 2); }

template <typename T, int N>
cudaError_t run(const SsdPrefillParams& p, cudaStream_t s) {
  CUtensorMap mx, mb, mc;
  std::memset(&mx, 0, sizeof(mx));
  std::memset(&mb, 0, sizeof(mb));
  std::memset(&mc, 0, sizeof(mc));
  constexpr bool bf = std::is_same<T, __nv_bfloat16>::value;
  if (p.seq.tokens > 0 &&  // without tokens the maps are never used
      (!tc::encode_2d(&mx, bf, p.x, (int64_t)p.nheads * kP, p.seq.tokens, p.ldx, kQ) ||
       !tc::encode_2d(&mb, bf, p.B, (int64_t)p.ngroups * N, p.seq.tokens, p.ldb, kQ) ||
       !tc::encode_2d(&mc, bf, p.C, (int64_t)p.ngroups * N, p.seq.tokens, p.ldc, kQ)))
    return cudaErrorInvalidValue;
  const int npairs = pairs(p), blocks = prefill_blocks(p.seq.tokens, p.seq.nseq, npairs, p.sms);
  prefill_plan_kernel<<<1, 1024, 0, s>>>(p, npairs, blocks);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int smem = Lay<N>::kAlloc;
  e = cudaFuncSetAttribute(prefill_tc_kernel<T, N>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, prefill_tc_kernel<T, N>, p, npairs, blocks, mx, mb, mc);
}

template <typename T>
cudaError_t run_t(const SsdPrefillParams& p, cudaStream_t s) {
  return p.dstate == 128 ? run<T, 128>(p, s) : run<T, 64>(p, s);
}

}  // namespace

int prefill_blocks(int64_t tokens, int64_t nseq, int npairs, int sms) {
  const int64_t units = (tokens / kQ + nseq) * npairs;  // at most this many chunks
  const int64_t least = (units + kMinRange - 1) / kMinRange;
  return (int)(least < sms ? (least < 1 ? 1 : least) : sms);
}

size_t prefill_workspace(int64_t tokens, int64_t nseq, int64_t nheads, int64_t ngroups, int64_t dstate, int sms) {
  const int npairs = (int)(ngroups * ((nheads / ngroups + 1) / 2));
  return plan_layout(nseq, prefill_blocks(tokens, nseq, npairs, sms), (int)dstate).total;
}

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
