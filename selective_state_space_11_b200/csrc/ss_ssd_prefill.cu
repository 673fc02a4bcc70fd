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
// A block takes two heads of a group at a time, so that G, B and C are formed
// and loaded once for both, every product has 128 rows, and the state update's
// accumulator [2 x 64 head rows][N] fills all TMEM lanes:
//   G   C (K-major)     x B (K-major)         128 x 128, K = N
//   Yc  C (K-major)     x H copy (K-major)    128 x 128, K = N
//   Ym  M_h (in TMEM)   x X_h (MN-major)      128 x 64 per head, K = 128
//   S   Xw^T (MN-major) x B (MN-major)        128 x N, K = 128, once per piece
// TMEM: G, then Ym | Yc | M_0, M_1 (16-bit, two per column) | S: all 512 columns.
//
// One block of 640 threads per SM, its warps in roles that meet in mbarriers
// and flow from run to run of the block's work without meeting otherwise: 0-7
// form M and y (a warpgroup per head, a thread per token), 8-11 hold the state
// (a thread per row), 12-15 form Xw a quarter of the chunk at a time, and one
// warp each issues the products of y, those of the state, issues the copies and
// finds the next run, and forms the decays.  The state's products of a chunk run
// beside its y, and the state copy for the next chunk is written while the state
// is updated, so the chain from chunk to chunk is Xw -> S -> H -> copy -> Yc.
//
// Roundings to 16 bits: M and the H copy, once each (the operands of y, which
// is itself rounded to 16 bits).  Against 64 bits y is then 2.05e-3 off in bf16
// and 2.5e-4 in fp16 where its own rounding alone leaves 1.66e-3 and 2.1e-4;
// nearly all of the difference is M's.  M in two pieces (the second in G's columns,
// M X added to the scaled Yc) brings it to 1.67e-3 and 2.1e-4, but takes 213 us
// for 169 (4 x 4096 x 80), 177 for 147 (ragged) and 218 for 178 (32768 x 24): the
// y warps' issue slots, which Xw's warps need.  So one rounding each, as in
// ss_ssd_fwd.  The state is not rounded: Xw, a product of an fp32
// weight and a 16-bit input, goes through the tensor core as 16-bit pieces,
// against the exact B, and H lives in fp32 registers.  Three pieces of bf16 hold
// 24 bits.  Two of fp16 hold 22, and are formed of Xw times a power of two that
// puts the largest of the chunk and head into [2^14, 2^15) (undone exactly on S),
// so that a growing state does not leave fp16's range and small values do not
// fall out of it: each is within 2^-22 of itself or 2^-39 of the largest.  The
// largest is taken of the weighted products, decay to the chunk's end included:
// of |x| Delta alone, growth by more than 2 in a chunk made the state NaN, and a
// token that a later one makes the state forget set the scale for all.
//
// Decays.  Exponents are formed from sums inside blocks of 32 tokens and the
// blocks' totals, never as differences of long prefix sums, so a strong decay
// loses no bits: exp(cs_i - cs_j) for j in an earlier block is
// exp(from the end of j's block to i) x exp(from j to the end of its block),
// both at most 1 for A < 0, and only the diagonal blocks take an exponential per
// element, of a difference of sums inside the block.  There a token's log2 decay
// counts down to kForget, whose power of two is 0 in fp32 as that of any below
// is: else the sums of the tokens behind one that resets the state lose the bits
// that set them apart (a decay of e^-40000 left y 11 half steps of fp16 off).
//
// Work split.  The chunks of all (sequence, head pair) units, in order, are
// cut into contiguous ranges of equal cost, one per block; a planning kernel
// finds the cuts from the lengths in device memory.  A unit that a cut falls
// into is handed over: the block that has its first part runs that part first
// and publishes the state; a block whose whole range lies inside the unit first
// runs its state products alone, from zero, and publishes that state and its
// decay.  Neither waits for anyone.  Then such a block, and the one with the
// last part (as its last run), sums the published states before its own, each
// decayed over the ranges between, and runs its range in full.  (Handing one sum
// on from block to block took 215 us for 32768 tokens x 24 heads, 25 of them in
// the chain; summing took 185.)  Blocks take their number from a counter, so a
// block only ever waits for one that has started; the wait is bounded all the
// same, as every wait here is: one that runs out sets a bit of the fault word
// and the block drains its copies and products and leaves.
//
// What bounds it: the matrix instructions it needs (26 MFLOP per chunk and
// pair at N = 128, half of them for the exact state) are 75 us at the rate of a
// large bf16 product for 4 x 4096 tokens x 80 heads, its bytes 57 us.  Measured
// on B200, in a graph replayed on one state, part of which stays in L2: 169 us
// (0.76 PFLOP/s), 177 us for one sequence of 32768 tokens x 24 heads in fp16, 148
// us for 8192 tokens of ragged prompts x 80 heads with their states, 16.5 us for
// one prompt of 37 tokens.  On three states in turn 4 x 4096 x 80 takes 174 to 181
// us, in a loop of seconds, at the power limit, 188.  With a gate z it is 306, and
// 236 ragged: a thread reads a token's row of z by itself.  The rest is the chain
// above, and the issue slots of Xw: its warps work 7 of a chunk's 9 thousand
// cycles.  What made the difference on the way: at 4 x 4096 x 80, one group of 8
// warps that does everything in turn 338 us, copies and products in warps of
// their own 242, the state's warps apart from y's 234, two operand buffers for S
// and the copy written on the way 212, rolled loops and short waits, which keep
// what the roles run most inside the instruction cache, 179 (a look at a stop flag
// in every wait's loop: 218 for 169), the gate compiled apart and accumulators
// given back early 166; ragged, a block barrier behind every run 237, flowing from
// run to run 204, ranges of equal cost 146.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
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
// Warps: 0-7 the y group, 8-11 the state's, 12-15 Xw's, then the helpers.
constexpr int kGroupY = 256, kGroupS = 128;  // threads of the y group, of the state's and Xw's
constexpr int kMmaY = 16, kMmaS = 17, kTmaWarp = 18;  // and 19, the decays
constexpr int kThreads = 640;
// The registers of a block, 96 per thread at launch, are split unevenly: a
// thread of the state's warps holds a whole state row.  What a row of 64 leaves
// goes to Xw's warps and the helpers: 176 us for 32768 tokens x 24 heads, where
// the split of 128 took 185.  Sums: 2 x 96 + S + X + Help <= 5 x 96.
template <int N>
struct Regs {
  static constexpr int kS = N == 64 ? 112 : 168, kX = N == 64 ? 88 : 64, kHelp = N == 64 ? 88 : 56;
  static_assert(2 * 96 + kS + kX + kHelp <= 5 * 96, "a split above the launch's registers would wait forever");
};
// Polls of a wait.  One that fails has blocked for 4 us (measured, of a lane and
// of 1 to 20 warps alike), so a wait gives up after a second; what it is for
// takes microseconds, and a predecessor's state 2 us for each chunk of its range.
constexpr uint32_t kWaitLimit = 1u << 18;
constexpr uint32_t kFlagLimit = 1u << 22;  // polls of a predecessor's flag
constexpr float kForget = -160.f;
constexpr uint32_t kG = 0, kYc = 128, kM = 256, kS = 384;  // TMEM columns (Ym over G)

// Workspace: the plan, then the published states.
struct Cut {
  int seq, pair, chunk;  // position of a range's first chunk
};
__host__ __device__ inline size_t align256(size_t x) { return (x + 255) / 256 * 256; }
struct PlanLayout {
  size_t prefix, cuts, flags, decay, carry, total;
};
__host__ __device__ inline PlanLayout plan_layout(int64_t nseq, int blocks, int dstate) {
  PlanLayout l;
  l.prefix = 0;                                              // long long [nseq + 1]: cost before sequence i
  l.cuts = align256((nseq + 1) * sizeof(long long));         // Cut [blocks + 1]
  l.flags = l.cuts + align256((blocks + 1) * sizeof(Cut));   // unsigned [blocks], then the counter
  // float [blocks][2]: log2 decay over the published run
  l.decay = l.flags + align256((blocks + 1) * sizeof(unsigned));
  l.carry = l.decay + align256(blocks * 2 * sizeof(float));
  l.total = l.carry + (size_t)blocks * 2 * kP * dstate * sizeof(float);
  return l;
}

// A block for every unit or for every kMinRange chunks, whichever is more: a
// cut inside a unit costs a handover of its state.
constexpr int kMinRange = 4;
// What a unit costs in time: its chunks, and as much as another one for the
// state's way in and out.  Without the latter, a block of many one-chunk
// prompts has up to twice the work of the others: 204 against 146 us for 24
// prompts of 8192 tokens in all, 80 heads.
constexpr int kChunkCost = 1, kUnitCost = 1;

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
      // an empty sequence is a unit too: its state may have to be zeroed
      n = kUnitCost + kChunkCost * (e > b ? (e - b + kQ - 1) / kQ : 1);
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
  const long long cost = prefix[nseq] * npairs, units = (long long)nseq * npairs;
  const long long most = max(units, ((cost - units * kUnitCost) / kChunkCost + kMinRange - 1) / kMinRange);
  const long long used = most < blocks ? most : blocks;
  for (int j = tid; j <= blocks; j += 1024) {
    Cut c{nseq, 0, 0};
    if (j < used) {
      const long long lin = j * cost / used;
      int lo = 0, hi = nseq - 1;
      while (lo < hi) {  // the last sequence whose cost starts at or before lin
        const int mid = (lo + hi + 1) >> 1;
        if (prefix[mid] * npairs <= lin) lo = mid;
        else hi = mid - 1;
      }
      c.seq = lo;
      const long long unit = prefix[lo + 1] - prefix[lo], in = lin - prefix[lo] * npairs;
      c.pair = (int)(in / unit);
      c.chunk = (int)(max(in - c.pair * unit - kUnitCost, 0ll) / kChunkCost);
    }
    cuts[j] = c;
  }
}

// Byte offsets in the (1024-aligned) shared-memory block.
template <int N>
struct Lay {
  static constexpr int kTile = N * 256;               // 128 rows x N 16-bit
  static constexpr int kB = 0;
  static constexpr int kC = kTile;
  static constexpr int kX = kC + kTile;               // two of 2 heads x 128 rows x 128 B: x, then y in its place
  static constexpr int kW = kX + 65536;               // two of 3 pieces x 2 heads x 32 rows x 128 B
  static constexpr int kH = kW + 2 * 24576;           // 128 rows x N 16-bit
  static constexpr int kArr = kH + kTile;             // two of Arrays
  static constexpr int kMax = kArr + 2 * 3104;        // unsigned [2]: largest |x| Delta of the chunk (fp16)
  static constexpr int kUn = kMax + 16;               // float [2][2]: 1 / Xw's power of two (fp16), by chunk and head
  static constexpr int kBars = kUn + 16;              // mbarriers
  static constexpr int kSlot = kBars + 256;           // TMEM base address
  static constexpr int kBytes = kSlot + 16;
  static constexpr int kAlloc = kBytes + 1024;
};
struct Arrays {      // per head of the pair and token of the chunk
  float f[2][kQ];    // 2^(log2 decay from the token to the end of its block of 32) Delta
  float pre[2][kQ];  // log2 decay from the start of the block up to the token
  float dl[2][kQ];   // Delta
  float tot[2][4];   // log2 decay of each block
};
static_assert(sizeof(Arrays) == 3104, "Lay::kMax");

// mbarriers: copies landed; products done; arrivals of the warps of a group.
// A parity names a phase only to a thread that can be neither a phase behind
// nor one ahead.  The pairs [2] alternate between chunks (or chunks in full,
// for those of y), because their waiters and the next chunk's signallers are
// not ordered more tightly; kBarS and kBarW alternate between the quarters of
// a chunk, two phases each; the others have one phase per chunk (in full).
enum : int {
  kBarX = 0,      // [2]
  kBarSall = 2,   // [2] all of S (for the copies)
  kBarS = 4,      // [2] a quarter of S is done, and with its Xw
  kBarB = 6,
  kBarC = 7,
  kBarG = 8,      // G
  kBarYc = 9,     // C H^T
  kBarYm = 10,    // M X
  kNumTx = 11,    // those above are armed by the copy and product threads
  kBarA = 11,     // [2] the decays are written
  kBarW = 13,     // [2] a quarter of Xw is written
  kBarM = 15,     // M is written
  kBarR = 16,     // [2] Xw's warps are done with x
  kBarH = 18,     // [2] the state copy is written
  kBarY = 20,     // [2] y is in place of x
  kBarT = 22,     // y's accumulators are read
  kBarE = 23,     // S is read: the next chunk's products may start
  kBarN = 24,     // [kRuns] a run is found
  kBarD = 28,     // [kRuns] a run is done in all warps
  kNumBars = 32
};
constexpr int kRuns = 4;  // runs known at a time
__host__ __device__ constexpr unsigned arrivals(int i) {
  return i < kBarW || (i >= kBarN && i < kBarD)     ? 1  // the thread in charge
         : i >= kBarD                               ? kThreads / 32
         : i == kBarM || (i >= kBarY && i <= kBarT) ? 8   // the warps of the y group
                                                    : 4;  // those of the state's or Xw's
}

__device__ __forceinline__ uint32_t swz(int r, int c) {
  return static_cast<uint32_t>(r * 128 + ((c ^ (r & 7)) << 4));
}
__device__ __forceinline__ void arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];\n" ::"r"(bar) : "memory");
}
// Barriers of the y group, of Xw's warps and of the state's; true everywhere
// if any thread's flag is set.
template <int ID, int THREADS>
__device__ __forceinline__ bool sync_or(bool v) {
  int r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.b32 p, %1, 0;\n barrier.cta.red.or.pred q, %2, %3, p;\n"
      " selp.b32 %0, 1, 0, q;\n}\n"
      : "=r"(r)
      : "r"((int)v), "n"(ID), "n"(THREADS)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ bool sync_y(bool v) { return sync_or<1, kGroupY>(v); }
__device__ __forceinline__ bool sync_x(bool v) { return sync_or<2, kGroupS>(v); }
__device__ __forceinline__ bool sync_s(bool v) { return sync_or<3, kGroupS>(v); }
// 32 bytes of one thread, 32-byte aligned.
__device__ __forceinline__ void ld_v8(const float* p, float* v) {
  asm volatile("ld.global.v8.f32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n"
               : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7])
               : "l"(p)
               : "memory");
}
__device__ __forceinline__ void st_v8(float* p, const float* v) {
  asm volatile("st.global.v8.f32 [%8], {%0,%1,%2,%3,%4,%5,%6,%7};\n" ::"f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]),
               "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]), "l"(p)
               : "memory");
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
template <typename T>
__device__ __forceinline__ uint4 pack8(const float* f) {
  return make_uint4(Pk<T>::pack(f[0], f[1]), Pk<T>::pack(f[2], f[3]), Pk<T>::pack(f[4], f[5]), Pk<T>::pack(f[6], f[7]));
}

// A run of a block: a unit, its chunks [c0, c0 + n), where its state comes from
// and goes to.  n < 0: there are no more.
struct Run {
  int seq, pair, c0, n, begin, end, slot, g, h0, nh2;
  bool full, from_slot, from_carry, publish, to_slot;
  __device__ __forceinline__ int t0(int j) const { return begin + (c0 + j) * kQ; }
};

// Finds the runs of a block one after the other (in shared memory; all lanes of a warp call next).
struct Runs {
  Cut A, E;
  int stage, useq, upair, npairs, per, ppg;
  int seen, slot;  // the last sequence asked for and its slot: a sequence has a unit per pair
  bool same;

  __device__ __forceinline__ void start(const SsdPrefillParams& p, const Cut* cuts, int npairs_) {
    A = cuts[0];
    E = cuts[1];
    npairs = npairs_;
    per = p.nheads / p.ngroups;
    ppg = (per + 1) / 2;  // heads and pairs per group
    seen = -1;
    same = A.seq == E.seq && A.pair == E.pair;
    stage = same && A.chunk > 0 && E.chunk > 0 ? 0 : E.chunk > 0 ? 2 : 3;
    if (A.seq >= p.seq.nseq) stage = 6;
    useq = A.seq;  // cursor of the whole units
    upair = A.pair;
    if (stage > 0 && A.chunk > 0 && ++upair == npairs) {
      upair = 0;
      ++useq;
    }
  }
  __device__ __forceinline__ void next(const SsdPrefillParams& p, Run* out) {
    Run run;
    run.n = -1;
    int stage = this->stage, useq = this->useq, upair = this->upair, seen = this->seen, slot = this->slot;
    __syncwarp();
    while (stage < 6) {
      int c1 = -1;
      run.full = run.from_slot = true;
      run.from_carry = run.publish = run.to_slot = false;
      if (stage <= 1) {         // inside one unit: the range's own state, from zero; then in full
        run.seq = A.seq; run.pair = A.pair; run.c0 = A.chunk; c1 = E.chunk;
        run.from_slot = false;
        run.full = run.from_carry = stage == 1;
        run.publish = stage == 0;
        stage = stage == 0 ? 1 : 6;
      } else if (stage == 2) {  // the first part of the unit at the range's end
        run.seq = E.seq; run.pair = E.pair; run.c0 = 0; c1 = E.chunk;
        run.publish = true;
        stage = same ? 6 : 3;
      } else if (stage == 3) {  // whole units
        if (useq == E.seq && upair == E.pair) {
          stage = A.chunk > 0 ? 4 : 6;
          continue;
        }
        run.seq = useq; run.pair = upair; run.c0 = 0;
        run.to_slot = true;
        if (++upair == npairs) { upair = 0; ++useq; }
      } else {                  // the last part of the unit at the range's start
        run.seq = A.seq; run.pair = A.pair; run.c0 = A.chunk;
        run.from_slot = false;
        run.from_carry = run.to_slot = true;
        stage = 6;
      }
      run.slot = -1;
      if (p.state) {
        if (run.seq != seen) slot = claim_slot_warp(p.slots, run.seq, &g_fault_prefill);
        seen = run.seq;
        run.slot = slot;
        if (run.slot < 0) {
          if (stage == 1) stage = 6;  // the middle of a skipped sequence
          continue;
        }
      }
      run.begin = seq_begin(p.seq, run.seq);
      run.end = seq_end(p.seq, run.seq, run.begin);
      if (c1 < 0) c1 = (run.end - run.begin + kQ - 1) / kQ;
      run.n = c1 - run.c0;  // 0 for an empty sequence: the state passes through
      run.g = run.pair / ppg;
      run.h0 = run.g * per + 2 * (run.pair - run.g * ppg);
      run.nh2 = min(2, run.g * per + per - run.h0);  // an odd group's last pair holds one head
      break;
    }
    if ((threadIdx.x & 31) == 0) {
      *out = run;
      this->stage = stage;
      this->useq = useq;
      this->upair = upair;
      this->seen = seen;
      this->slot = slot;
    }
    __syncwarp();
  }
};

template <typename T, int N, bool GATE>
__global__ void __launch_bounds__(kThreads, 1)
    prefill_tc_kernel(const SsdPrefillParams p, int npairs, int blocks, const __grid_constant__ CUtensorMap map_x,
                      const __grid_constant__ CUtensorMap map_b, const __grid_constant__ CUtensorMap map_c,
                      const __grid_constant__ CUtensorMap map_y) {
  using L = Lay<N>;
  constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
  constexpr int kPieces = kBf16 ? 3 : 2;
  constexpr uint32_t kId = tc::idesc_f16(kBf16, 128, 128, false, false);  // G, Yc
  constexpr uint32_t kIdS = tc::idesc_f16(kBf16, 128, N, true, true);
  constexpr uint32_t kIdYm = tc::idesc_f16(kBf16, 128, 64, false, true);

  extern __shared__ unsigned char smem_raw[];
  const uint32_t raw = tc::saddr(smem_raw);
  const uint32_t pad = (1024u - (raw & 1023u)) & 1023u;
  unsigned char* const sm = smem_raw + pad;
  const uint32_t sb = raw + pad;
  Arrays* const arr = reinterpret_cast<Arrays*>(sm + L::kArr);
  unsigned* const sMax = reinterpret_cast<unsigned*>(sm + L::kMax);
  float* const sUn = reinterpret_cast<float*>(sm + L::kUn);
  uint32_t* const sslot = reinterpret_cast<uint32_t*>(sm + L::kSlot);
  __shared__ unsigned s_block;
  __shared__ Run s_run[kRuns];
  __shared__ Runs s_runs;
  auto bar = [&](int i) { return sb + L::kBars + 8u * static_cast<uint32_t>(i); };

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // the groups: TMEM lane = row; a warpgroup of the y group per head of the pair
  const int hd = (warp >> 2) & 1, blk = warp & 3, row = 32 * blk + lane;
  const uint32_t lane_base = static_cast<uint32_t>(32 * blk) << 16;
  const int hrow = row >> 6;         // the head of state row `row`

  if (tid < kNumBars) {
    tc::mbar_init(bar(tid), arrivals(tid));
    tc::fence_mbar_init();
  }
  if (tid == 32 * kTmaWarp && p.seq.tokens > 0) {
    tc::prefetch_map(&map_x);
    tc::prefetch_map(&map_b);
    tc::prefetch_map(&map_c);
    tc::prefetch_map(&map_y);
  }
  if (warp == 0) tc::tmem_alloc(tc::saddr(sslot), 512);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = *sslot;
  if (warp < 8) {  // the blocks of M above the diagonal stay zero
    const uint32_t zero[16] = {};
    for (int j = blk + 1; j < 4; ++j) tc::st32x32b_x16(tmem + lane_base + kM + 64 * hd + 16 * j, zero);
    tc::st_wait();
  }
  pdl_wait();  // the plan is written

  char* const ws = static_cast<char*>(p.ws);
  const PlanLayout play = plan_layout(p.seq.nseq, blocks, N);
  unsigned* const flags = reinterpret_cast<unsigned*>(ws + play.flags);
  const Cut* const cuts = reinterpret_cast<const Cut*>(ws + play.cuts);
  float* const decay = reinterpret_cast<float*>(ws + play.decay);
  float4* const carry = reinterpret_cast<float4*>(ws + play.carry);
  if (warp == kTmaWarp) {
    unsigned b = 0;
    if (lane == 0) b = atomicAdd(flags + blocks, 1u);
    b = __shfl_sync(0xffffffffu, b, 0);
    if (lane == 0) s_block = b;
    if (lane == 0) s_runs.start(p, cuts + b, npairs);
  }
  __syncthreads();
  const int me = (int)s_block;

  // A wait that runs out makes the warp's `ok` false: it waits for nothing any
  // more, and its role leaves its loop where all of the role's warps can.  `ok`
  // is the same in all lanes where a whole warp waits; wait_lane is for one lane.
  bool ok = true;
  auto wait = [&](int i, uint32_t parity) {
    if (ok) ok = tc::wait_warp(bar(i), parity & 1u, kWaitLimit);
  };
  auto wait_lane = [&](int i, uint32_t parity) {
    if (ok) ok = tc::wait(bar(i), parity & 1u, kWaitLimit);
  };
  // the pairs that alternate between chunks
  auto wait2 = [&](int i, uint32_t k) { wait(i + (int)(k & 1), k >> 1); };
  auto wait2_lane = [&](int i, uint32_t k) { wait_lane(i + (int)(k & 1), k >> 1); };
  // barriers that the copy and the product thread have armed, and the parity
  // of the last phase, for the drain
  uint32_t armed = 0, last_par = 0, next_par = 0;
  auto arm = [&](int i) {
    const uint32_t m = 1u << i;
    armed |= m;
    last_par = (last_par & ~m) | (next_par & m);
    next_par ^= m;
  };

  auto signal = [&](int i) {  // the warp's shared-memory and TMEM accesses, then one arrival
    tc::fence_proxy_async();
    tc::fence_before();
    __syncwarp();
    if (lane == 0) arrive(bar(i));
  };
  uint32_t it = 0, itf = 0;  // chunks, and chunks in full, so far

  // Run r of the block, found by the copying warp ahead of time; false behind
  // the last, or when a wait of the role has run out (`any`: of any of its threads).
  const Run* run = nullptr;
  auto next = [&](uint32_t r, auto any) -> bool {
    wait(kBarN + (int)(r % kRuns), r / kRuns);
    run = &s_run[r % kRuns];
    return !any(!ok) && run->n >= 0;
  };
  auto any_warp = [&](bool v) { return __any_sync(0xffffffffu, v) != 0; };
  // The run is done in this warp.  The roles flow from run to run, each as far
  // as its barriers let it; only behind a run of the state alone they meet, so
  // that the roles which have no part in it find the barriers in phase.
  auto done = [&](uint32_t r) {
    const int n = run->n;
    const bool full = run->full;
    it += n;
    if (full) itf += n;
    __syncwarp();
    if (lane == 0) arrive(bar(kBarD + (int)(r % kRuns)));
    if (!full) wait(kBarD + (int)(r % kRuns), r / kRuns);
  };

  if (warp < 8) {
    for (uint32_t r = 0; next(r, sync_y); ++r) {
      const int n = run->n, end = run->end, h0 = run->h0, nh2 = run->nh2;
      const bool full = run->full;
      // ----------------------------------------------------------- M and y
      const int h = h0 + min(hd, nh2 - 1);
      const bool mine = hd < nh2;
      const float Dh = p.D ? p.D[h] : 0.f;
#pragma unroll 1
      for (int j = 0; full && j < n; ++j) {
        const uint32_t k = it + j, kf = itf + j;
        const int t0 = run->t0(j), nval = min(kQ, end - t0);
        const Arrays& a = arr[k & 1];
        unsigned char* const xs = sm + L::kX + (k & 1) * 32768 + hd * 16384;
        wait2(kBarA, k);
        const float pre = a.pre[hd][row];
        wait(kBarG, kf);
        tc::fence_after();
        // ---- M, row `row`: 32 columns at a time, from the diagonal block to the left
        float between = pre;  // log2 decay from the end of block i to this row
#pragma unroll 1
        for (int i = blk; i >= 0; --i) {
          float gv[32];
          tc::ld32x32b_x32(tmem + lane_base + kG + 32 * i, gv);
          uint32_t mp[16];
          if (i == blk) {
            const float4* pr = reinterpret_cast<const float4*>(a.pre[hd] + 32 * i);
            const float4* dl = reinterpret_cast<const float4*>(a.dl[hd] + 32 * i);
            const f2_t pre2 = pk2(pre, pre), minus = pk2(-1.f, -1.f);
#pragma unroll
            for (int u = 0; u < 8; ++u) {
              const float4 pv = pr[u], dv = dl[u];
              const f2_t e01 = ex2_2(fma2(pk2(pv.x, pv.y), minus, pre2));
              const f2_t e23 = ex2_2(fma2(pk2(pv.z, pv.w), minus, pre2));
              const f2_t m01 = mul2(mul2(pk2(gv[4 * u], gv[4 * u + 1]), e01), pk2(dv.x, dv.y));
              const f2_t m23 = mul2(mul2(pk2(gv[4 * u + 2], gv[4 * u + 3]), e23), pk2(dv.z, dv.w));
              float m[4] = {lo2(m01), hi2(m01), lo2(m23), hi2(m23)};
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if (4 * u + e > lane) m[e] = 0.f;
              mp[2 * u] = Pk<T>::pack(m[0], m[1]);
              mp[2 * u + 1] = Pk<T>::pack(m[2], m[3]);
            }
          } else {
            const float ei = ex2(between);
            between += a.tot[hd][i];
            const f2_t ei2 = pk2(ei, ei);
            const float4* fj = reinterpret_cast<const float4*>(a.f[hd] + 32 * i);
#pragma unroll
            for (int u = 0; u < 8; ++u) {
              const float4 fv = fj[u];
              const f2_t m01 = mul2(pk2(gv[4 * u], gv[4 * u + 1]), mul2(ei2, pk2(fv.x, fv.y)));
              const f2_t m23 = mul2(pk2(gv[4 * u + 2], gv[4 * u + 3]), mul2(ei2, pk2(fv.z, fv.w)));
              mp[2 * u] = Pk<T>::pack(lo2(m01), hi2(m01));
              mp[2 * u + 1] = Pk<T>::pack(lo2(m23), hi2(m23));
            }
          }
          tc::st32x32b_x16(tmem + lane_base + kM + 64 * hd + 16 * i, mp);
        }
        tc::st_wait();
        signal(kBarM);
        // ---- y = (2^cs Yc + Ym + D x) SiLU(z), in place of x
        const float e = ex2(between);  // from the start of the chunk to this row
        const f2_t e2 = pk2(e, e), D2 = pk2(Dh, Dh);
        const int64_t t = t0 + row;
        const T* zg = GATE && mine && row < nval ? static_cast<const T*>(p.z) + t * p.ldz + h * kP : nullptr;
        wait2(kBarR, k);   // x has landed, and Xw's warps are done with it
        wait(kBarYm, kf);  // and so is Yc, issued before
        tc::fence_after();
#pragma unroll 1
        for (int i = 0; i < 4; ++i) {
          float yc[16], ym[16];
          const uint32_t col = tmem + lane_base + 64 * hd + 16 * i;
          tc::ld32x32b_x16_pair(col + kYc, col + kG, yc, ym);
          if (i == 3) signal(kBarT);  // the next chunk's products may start
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            uint4* at = reinterpret_cast<uint4*>(xs + swz(row, 2 * i + u));
            const uint4 xv = *at;
            const uint32_t in[4] = {xv.x, xv.y, xv.z, xv.w};
            float o[8];
#pragma unroll
            for (int v = 0; v < 4; ++v) {
              const float2 f = Pk<T>::unpack(in[v]);
              const int at8 = 8 * u + 2 * v;
              const f2_t r =
                  fma2(D2, pk2(f.x, f.y), fma2(e2, pk2(yc[at8], yc[at8 + 1]), pk2(ym[at8], ym[at8 + 1])));
              o[2 * v] = lo2(r);
              o[2 * v + 1] = hi2(r);
            }
            if (GATE && zg) {
              float zv[8];
              if (p.zvec) load8(zg + 16 * i + 8 * u, zv);
              else
#pragma unroll
                for (int v = 0; v < 8; ++v) zv[v] = ldf(zg + 16 * i + 8 * u + v);
#pragma unroll
              for (int v = 0; v < 8; ++v) o[v] *= zv[v] * sigmoid_f(zv[v]);
            }
            if (mine) *at = pack8<T>(o);
          }
        }
        if (nval < kQ) {  // the rows of a ragged chunk, one by one
          sync_y(false);
#pragma unroll 1
          for (int i = tid; i < nval * 8 * nh2; i += kGroupY) {
            const int hh = i / (nval * 8), r = (i >> 3) - hh * nval, cc = i & 7;
            const uint4 v = *reinterpret_cast<const uint4*>(sm + L::kX + (k & 1) * 32768 + hh * 16384 + swz(r, cc));
            T* const to = static_cast<T*>(p.y) + ((int64_t)(t0 + r) * p.nheads + h0 + hh) * kP;
            *reinterpret_cast<uint4*>(to + 8 * cc) = v;
          }
        }
        signal(kBarY + (kf & 1));
      }
      done(r);
    }
  } else if (warp < 12) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(Regs<N>::kS));
    for (uint32_t r = 0; next(r, sync_s); ++r) {
      const int n = run->n, h0 = run->h0, nh2 = run->nh2;
      const bool full = run->full;
      // ----------------------------------------------------- the state -------
      const bool owns = hrow < nh2;
      const int stid = tid - kGroupY;
      auto wait_flag = [&](int b) {  // the state that block b publishes
        if (stid == 0) {
          uint32_t polls = 0, v = 0;
          do {
            asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(flags + b) : "memory");
          } while (!v && ++polls < kFlagLimit);
          if (!v) ok = false;
        }
        ok = !sync_s(!ok);
        return ok;
      };
      // ---- the state entering the run
      float hs[N];
      float* st = p.state && owns ? p.state + (((size_t)run->slot * p.nheads + h0) * kP + row) * N : nullptr;
#pragma unroll
      for (int i = 0; i < N; ++i) hs[i] = 0.f;
      if (run->from_carry) {  // the unit's runs before this one, each decayed over those between, back to its first
        float between = 0.f;
#pragma unroll 1
        for (int b = me - 1; b >= 0 && wait_flag(b); --b) {
          const float4* const src = carry + (size_t)b * (2 * kP * N / 4);
          const float dec = ex2(between);
#pragma unroll
          for (int i = 0; i < N / 4; ++i) {
            const float4 v = __ldcg(src + i * kGroupS + stid);
            hs[4 * i] = fmaf(dec, v.x, hs[4 * i]);
            hs[4 * i + 1] = fmaf(dec, v.y, hs[4 * i + 1]);
            hs[4 * i + 2] = fmaf(dec, v.z, hs[4 * i + 2]);
            hs[4 * i + 3] = fmaf(dec, v.w, hs[4 * i + 3]);
          }
          const Cut c = cuts[b];
          if (c.seq != run->seq || c.pair != run->pair || c.chunk == 0) break;
          between += __ldcg(decay + 2 * b + hrow);
        }
      } else if (run->from_slot && st && !(p.slots.fresh && p.slots.fresh[run->seq])) {
#pragma unroll
        for (int i = 0; i < N; i += 8) ld_v8(st + i, hs + i);
      }
      // its 16-bit copy: K-major, row = state row
      auto write_copy = [&]() {
#pragma unroll
        for (int q = 0; q < N / 8; ++q)
          *reinterpret_cast<uint4*>(sm + L::kH + (q / 8) * 16384 + swz(row, q % 8)) = pack8<T>(hs + 8 * q);
      };
      if (n > 0) {
        if (full) write_copy();
        signal(kBarH + (it & 1));
      }
      float psum = 0.f;  // log2 decay of the run so far (head hrow)

#pragma unroll 1
      for (int j = 0; j < n; ++j) {
        const uint32_t k = it + j, kf = itf + j;
        const Arrays& a = arr[k & 1];
        wait2(kBarA, k);
        // ---- H <- 2^cs_last H + S
        const float tot = (a.tot[hrow][0] + a.tot[hrow][1]) + (a.tot[hrow][2] + a.tot[hrow][3]);
        psum += tot;
        const float dec = ex2(tot);
        if (full) wait(kBarYc, kf);  // C H^T is done with the state copy
        wait2(kBarSall, k);
        if (!kBf16) wait2(kBarR, k);  // (Xw's scale)
        tc::fence_after();
        const f2_t dec2 = pk2(dec, dec), un2 = kBf16 ? 0 : pk2(sUn[2 * (k & 1) + hrow], sUn[2 * (k & 1) + hrow]);
        const bool more = j + 1 < n;
#pragma unroll
        for (int q = 0; q < N; q += 16) {  // with the next chunk's 16-bit copy
          float sv[16];
          tc::ld32x32b_x16(tmem + lane_base + kS + q, sv);
#pragma unroll
          for (int i = 0; i < 16; i += 2) {
            f2_t v = pk2(sv[i], sv[i + 1]);
            if (!kBf16) v = mul2(v, un2);
            v = fma2(dec2, pk2(hs[q + i], hs[q + i + 1]), v);
            hs[q + i] = lo2(v);
            hs[q + i + 1] = hi2(v);
          }
          if (more && full)
#pragma unroll
            for (int i = q / 8; i < q / 8 + 2; ++i)
              *reinterpret_cast<uint4*>(sm + L::kH + (i / 8) * 16384 + swz(row, i % 8)) = pack8<T>(hs + 8 * i);
        }
        signal(kBarE);
        if (more) signal(kBarH + ((k + 1) & 1));
      }
      // ---- the state leaving the run
      if (run->publish) {
        float4* dst = carry + (size_t)me * (2 * kP * N / 4);
#pragma unroll
        for (int i = 0; i < N / 4; ++i)
          dst[i * kGroupS + stid] = make_float4(hs[4 * i], hs[4 * i + 1], hs[4 * i + 2], hs[4 * i + 3]);
        if ((stid & 63) == 0) decay[2 * me + hrow] = psum;
        __threadfence();
        sync_s(false);
        if (stid == 0) asm volatile("st.release.gpu.global.u32 [%0], 1;" ::"l"(flags + me) : "memory");
      } else if (run->to_slot && st) {
#pragma unroll
        for (int i = 0; i < N; i += 8) st_v8(st + i, hs + i);
      }
      done(r);
    }
  } else if (warp < 16) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(Regs<N>::kX));
    // ----------------------------------------------------------------- Xw
    // a warp: 32 columns of head xh, lanes over tokens
    const int stid = tid - kGroupY - kGroupS, xh = blk >> 1, xc = 4 * (blk & 1);
    for (uint32_t r = 0; next(r, sync_x); ++r) {
      const int n = run->n, end = run->end, nh2 = run->nh2;
#pragma unroll 1
      for (int j = 0; j < n; ++j) {
        const uint32_t k = it + j;
        const int nval = min(kQ, end - run->t0(j));
        const Arrays& a = arr[k & 1];
        unsigned char* const xs = sm + L::kX + (k & 1) * 32768;
        wait2(kBarX, k);
        wait2(kBarA, k);
        float scale = 1.f;
        if constexpr (!kBf16) {  // fp16: the power of two that puts max |Xw| into [2^14, 2^15)
          if (stid < 2) sMax[stid] = 0u;
          sync_x(false);
#pragma unroll 1
          for (int e = 0; e < 2; ++e) {
            unsigned m = 0;
#pragma unroll
            for (int q = 0; q < 8; ++q) {
              const uint4 v = *reinterpret_cast<const uint4*>(xs + e * 16384 + swz(row, q));
              const unsigned m0 = __vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu);
              m = __vmaxu2(m, __vmaxu2(m0, __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu)));
            }
            m = min(max(m & 0xffffu, m >> 16), 0x7bffu);  // (an infinity or a NaN counts as the largest number)
            // the weight as below: the decay up to the chunk's end takes part
            const float4 tot = *reinterpret_cast<const float4*>(a.tot[e]);
            const float later = (blk < 1 ? tot.y : 0.f) + (blk < 2 ? tot.z : 0.f) + (blk < 3 ? tot.w : 0.f);
            float top = __half2float(__ushort_as_half((unsigned short)m)) * fabsf(a.f[e][row] * ex2(later));
            top = row < nval && e < nh2 ? fminf(top, 3.0e38f) : 0.f;
#pragma unroll
            for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            if (lane == 0) atomicMax(sMax + e, __float_as_uint(top));
          }
          sync_x(false);
          auto power = [](unsigned v) {  // 2^(14 - exponent of v), so that it and its inverse are fp32 numbers
            const int e = (int)(v >> 23) - 127;
            return v == 0 ? 0 : min(126, 14 - e);
          };
          scale = __uint_as_float((unsigned)(127 + power(sMax[xh])) << 23);
          if (stid < 2) sUn[2 * (k & 1) + stid] = __uint_as_float((unsigned)(127 - power(sMax[stid])) << 23);
        }
        // ---- Xw, 32 tokens at a time, as 16-bit pieces.  Rows behind the
        // sequence belong to others, and a missing head has none: no NaN of
        // theirs may meet a zero weight, so x, and with its last rows B, become zero there.
        const int xval = xh < nh2 ? nval : 0;
        constexpr int kAhead = N == 64 ? 4 : 2;  // vectors of x at a time, as far as the registers go
#pragma unroll 1
        for (int q = 0; q < 4; ++q) {
          float later = 0.f;  // log2 decay of the blocks behind
          for (int b = q + 1; b < 4; ++b) later += a.tot[xh][b];
          float w = a.f[xh][32 * q + lane] * ex2(later);
          if constexpr (!kBf16) {  // finite weights stay finite: a token of zeros has no part in the scale
            const float ws = w * scale;
            w = fabsf(w) <= 3.0e38f ? fminf(fmaxf(ws, -3.0e38f), 3.0e38f) : ws;
          }
          const f2_t w2 = pk2(w, w), minus = pk2(-1.f, -1.f);
          unsigned char* const from = xs + xh * 16384;
          const bool live = 32 * q + lane < xval;
          unsigned char* const to = sm + L::kW + (q & 1) * 24576 + xh * 4096;
          // the products of the quarter before the last have read the buffer
          if (q > 1 || k > 0) wait(kBarS + (q & 1), q > 1 ? 0 : 1);
#pragma unroll 1
          for (int k0 = xc; k0 < xc + 4; k0 += kAhead) {
            uint4 xv[kAhead];
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
              uint4* const xp = reinterpret_cast<uint4*>(from + swz(32 * q + lane, k0 + i));
              if (!live) *xp = make_uint4(0, 0, 0, 0);
              xv[i] = *xp;
            }
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
              const int k4 = k0 + i;
              const uint32_t in[4] = {xv[i].x, xv[i].y, xv[i].z, xv[i].w};
              uint32_t u[4], v[4], z[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float2 f = Pk<T>::unpack(in[e]);
                const f2_t x0 = mul2(pk2(f.x, f.y), w2);
                u[e] = Pk<T>::pack(lo2(x0), hi2(x0));
                const float2 f0 = Pk<T>::unpack(u[e]);
                const f2_t x1 = fma2(pk2(f0.x, f0.y), minus, x0);
                v[e] = Pk<T>::pack(lo2(x1), hi2(x1));
                if (kPieces == 3) {
                  const float2 f1 = Pk<T>::unpack(v[e]);
                  const f2_t x2 = fma2(pk2(f1.x, f1.y), minus, x1);
                  z[e] = Pk<T>::pack(lo2(x2), hi2(x2));
                }
              }
              const uint32_t o = swz(lane, k4);
              *reinterpret_cast<uint4*>(to + o) = make_uint4(u[0], u[1], u[2], u[3]);
              *reinterpret_cast<uint4*>(to + 8192 + o) = make_uint4(v[0], v[1], v[2], v[3]);
              if (kPieces == 3) *reinterpret_cast<uint4*>(to + 16384 + o) = make_uint4(z[0], z[1], z[2], z[3]);
            }
          }
          if (32 * q + 32 > nval) {
            wait(kBarB, k);
            const int first = max(nval - 32 * q, 0);
#pragma unroll 1
            for (int i = 8 * first + stid; i < 256; i += kGroupS)
#pragma unroll
              for (int b = 0; b < N / 64; ++b)
                *reinterpret_cast<uint4*>(sm + L::kB + 16384 * b + 4096 * q + 16 * i) = make_uint4(0, 0, 0, 0);
          }
          signal(kBarW + (q & 1));
        }
        if (lane == 0) arrive(bar(kBarR + (k & 1)));  // (the signal above ordered the warp's accesses)
      }
      done(r);
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(Regs<N>::kHelp));
    if (warp == kTmaWarp) {
      // y of the last two chunks in full, to be stored when its buffer is needed
      // or at the end (t < 0: a ragged chunk, whose y the y group writes)
      int t_a = -1, h_a = 0, t_b = -1, h_b = 0;  // h: first head, and the number of heads above bit 16
      auto store_y = [&](int t, int h, uint32_t k) {
        if (t < 0) return;
#pragma unroll 1
        for (int b = 0; b < h >> 16; ++b)
          tc::tma_store_2d(&map_y, ((h & 0xffff) + b) * kP, t, sb + L::kX + (k & 1) * 32768 + 16384u * b);
        tc::bulk_commit();
      };
      auto publish = [&](uint32_t r) {  // run r
        if (r >= kRuns) wait(kBarD + (int)(r % kRuns), r / kRuns - 1);
        if (any_warp(!ok)) return;
        Run* const then = &s_run[r % kRuns];
        s_runs.next(p, then);
        if (lane == 0) {
          arrive(bar(kBarN + (int)(r % kRuns)));
          if (then->n > 0) {  // bring what its first chunk waits for into L2
            tc::tma_prefetch_2d(&map_x, then->h0 * kP, then->t0(0));
            if (then->nh2 > 1) tc::tma_prefetch_2d(&map_x, then->h0 * kP + kP, then->t0(0));
            if (then->from_slot && p.state && !(p.slots.fresh && p.slots.fresh[then->seq]))
              tc::bulk_prefetch(p.state + ((size_t)then->slot * p.nheads + then->h0) * kP * N,
                                then->nh2 * kP * N * 4);
          }
        }
        __syncwarp();
      };
      publish(0);
      for (uint32_t r = 0; next(r, any_warp); ++r) {
        const int n = run->n, end = run->end, h0 = run->h0, nh2 = run->nh2;
        const bool full = run->full;
        // ------------------------------------------------ copies; the next run
        auto load = [&](int i, uint32_t off, const CUtensorMap* map, int col, int t, int nb) {
          tc::expect_tx(bar(i), 16384u * nb);
#pragma unroll 1
          for (int b = 0; b < nb; ++b) tc::tma_load_2d(sb + off + 16384u * b, map, col + 64 * b, t, bar(i));
          arm(i);
        };
#pragma unroll 1
        for (int j = 0; j <= n; ++j) {
          if (j == (n > 0)) publish(r + 1);  // behind the first chunk's copies
          if (j == n) break;
          const uint32_t k = it + j, kf = itf + j;
          const int t = run->t0(j);
          if (lane == 0 && ok) {  // each buffer as its last reader is done
            if (full) {
              if (kf > 1) wait2_lane(kBarY, kf - 2);
              if (ok) store_y(t_a, h_a, k);
              t_a = t_b;
              h_a = h_b;
              t_b = t + kQ <= end ? t : -1;
              h_b = h0 | nh2 << 16;
              tc::bulk_wait_read_all();
            }
            if (ok) load(kBarX + (k & 1), L::kX + (k & 1) * 32768, &map_x, h0 * kP, t, nh2);
            if (full) {
              if (kf > 0) wait_lane(kBarYc, kf - 1);
              if (ok) load(kBarC, L::kC, &map_c, run->g * N, t, N / 64);
            }
            if (k > 0) wait2_lane(kBarSall, k - 1);
            if (ok) load(kBarB, L::kB, &map_b, run->g * N, t, N / 64);
          }
          ok = __all_sync(0xffffffffu, ok);
        }
        done(r);
      }
      if (lane == 0) {
        if (itf > 1) wait2_lane(kBarY, itf - 2);
        if (ok) store_y(t_a, h_a, it);
        if (itf > 0) wait2_lane(kBarY, itf - 1);
        if (ok) store_y(t_b, h_b, it + 1);
      }
    } else if (warp == kMmaY) {
      // Products.  The issuing lane is picked by elect.sync: in a branch on the
      // thread number the compiler cannot take descriptors for uniform, and a
      // product of 128 x 128 x 16 takes 170-220 cycles to issue instead of the
      // 66 it takes to execute.
      // ----------------------------------------------------- products of y
      const uint64_t dc = tc::desc_sw128(sb + L::kC, 16, 1024), db0 = tc::desc_sw128(sb + L::kB, 16, 1024),
                     dh = tc::desc_sw128(sb + L::kH, 16, 1024), dx0 = tc::desc_sw128(sb + L::kX, 16384, 1024);
      for (uint32_t r = 0; next(r, any_warp); ++r) {
        const int n = run->full ? run->n : 0;
#pragma unroll 1
        for (int j = 0; j < n && ok; ++j) {
          const uint32_t k = it + j, kf = itf + j;
          wait(kBarB, k);
          wait(kBarC, kf);
          if (kf > 0) wait(kBarT, kf - 1);  // the accumulators are read
#pragma unroll 1
          for (int e = 0; e < 2; ++e) {  // G = C B^T, then Yc = C H^T
            if (e == 1) wait2(kBarH, k);
            if (!ok) break;
            tc::fence_after();
            if (tc::elect()) {
              const uint64_t db = e ? dh : db0;
              const uint32_t to = tmem + kG + (kYc - kG) * e;
#pragma unroll 1
              for (int kk = 0; kk < N / 16; ++kk) {
                const uint32_t ko = ((kk >> 2) * 16384 + (kk & 3) * 32) >> 4;
                tc::mma(to, dc + ko, db + ko, kId, kk > 0);
              }
              tc::commit(bar(kBarG + e));
            }
            __syncwarp();
            arm(kBarG + e);
          }
          // test hook (SS_INJECT_WAIT_TIMEOUT): y's accumulators, which hold nothing yet, are not read
          if (p.inject_timeout && kf == 0) ok = ok && tc::wait_warp(bar(kBarT), 0, 1u << 12);
          wait2(kBarX, k);
          wait(kBarM, kf);
          if (run->t0(j + 1) > run->end) wait2(kBarR, k);  // a ragged chunk's x is cleared behind its end
          if (!ok) break;
          tc::fence_after();
          if (tc::elect()) {
            const uint64_t dx = dx0 + (k & 1) * (32768 >> 4);
#pragma unroll 1
            for (int i = 0; i < 16; ++i)  // two heads, 8 steps of 16 tokens; the second head's x is 16 KB on
              tc::mma_ta(tmem + kG + 64 * (i >> 3), tmem + kM + 8 * i, dx + i * (2048 >> 4), kIdYm, (i & 7) != 0);
            tc::commit(bar(kBarYm));
          }
          __syncwarp();
          arm(kBarYm);
        }
        done(r);
      }
    } else if (warp == kMmaS) {
      // --------------------------------------------- products of the state
      const uint64_t db = tc::desc_sw128(sb + L::kB, 16384, 1024), dw0 = tc::desc_sw128(sb + L::kW, 4096, 1024);
      for (uint32_t r = 0; next(r, any_warp); ++r) {
        const int n = run->n;
#pragma unroll 1
        for (int j = 0; j < n && ok; ++j) {
          const uint32_t k = it + j;
          wait(kBarB, k);
          if (k > 0) wait(kBarE, k - 1);
#pragma unroll 1
          for (int q = 0; q < 4; ++q) {
            wait(kBarW + (q & 1), q >> 1);
            if (!ok) break;
            tc::fence_after();
            if (tc::elect()) {
              const uint64_t dw = dw0 + (q & 1) * (24576 >> 4), dbq = db + q * (4096 >> 4);
#pragma unroll 1
              for (int i = 0; i < 2 * kPieces; ++i)  // the pieces, two steps of 16 tokens
                tc::mma(tmem + kS, dw + ((i >> 1) * 8192 + (i & 1) * 2048) / 16, dbq + (i & 1) * (2048 >> 4), kIdS,
                        (q | i) != 0);
              tc::commit(bar(kBarS + (q & 1)));
              if (q == 3) tc::commit(bar(kBarSall + (k & 1)));
            }
            __syncwarp();
            arm(kBarS + (q & 1));
          }
          if (!ok) break;
          arm(kBarSall + (k & 1));
        }
        done(r);
      }
    } else {
      // ------------- Delta and the decays of both heads, as pairs (lo: the first)
      // lane: tokens 4 lane .. + 3 of the chunk, so a block of 32 is 8 lanes
      const int seg = lane & 7;
      const f2_t zero = pk2(0.f, 0.f);
      for (uint32_t r = 0; next(r, any_warp); ++r) {
        const int n = run->n, h = run->h0, h1 = run->nh2 - 1;  // (a missing head's are computed and dropped)
        const f2_t A2 = pk2(p.A[h] * kLog2e, p.A[h + h1] * kLog2e);
        const f2_t bias = p.dt_bias ? pk2(p.dt_bias[h], p.dt_bias[h + h1]) : zero;
#pragma unroll 1
        for (int j = 0; j < n; ++j) {
          const uint32_t k = it + j;
          Arrays& a = arr[k & 1];
          const int t = run->t0(j) + 4 * lane, left = run->end - t;
          const T* const dtg = static_cast<const T*>(p.dt) + h;
          f2_t d[4], ld[4], in[4];  // ld: a token's log2 decay
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const T* const at = dtg + (int64_t)min(t + i, run->end - 1) * p.lddt;
            d[i] = pk2(Elt<T>::to_f(at[0]), Elt<T>::to_f(at[h1]));
          }
          // the readers of this buffer, two chunks before
          if (k > 1) wait2(kBarH, k - 1);
          if (run->full && itf + j > 1) wait2(kBarY, itf + j - 2);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            d[i] = add2(d[i], bias);
            if (p.softplus) d[i] = pk2(softplus_f(lo2(d[i])), softplus_f(hi2(d[i])));
            if (i >= left) d[i] = zero;
            if (h1 == 0) d[i] = pk2(lo2(d[i]), 0.f);
            const f2_t e = mul2(d[i], A2);
            ld[i] = pk2(lo2(e) < kForget ? kForget : lo2(e), hi2(e) < kForget ? kForget : hi2(e));
            in[i] = i ? add2(in[i - 1], ld[i]) : ld[i];
          }
          f2_t before = in[3], after = in[3];
#pragma unroll
          for (int o = 1; o < 8; o <<= 1) {
            const f2_t u = __shfl_up_sync(0xffffffffu, before, o), v = __shfl_down_sync(0xffffffffu, after, o);
            if (seg >= o) before = add2(before, u);
            if (seg + o < 8) after = add2(after, v);
          }
          if (seg == 7) {
            a.tot[0][lane >> 3] = lo2(before);
            a.tot[1][lane >> 3] = hi2(before);
          }
          f2_t u = __shfl_up_sync(0xffffffffu, before, 1), v = __shfl_down_sync(0xffffffffu, after, 1);
          if (seg == 0) u = zero;
          if (seg == 7) v = zero;
          f2_t f[4];  // from the token to the end of its block
          f[3] = v;
          f[2] = ld[3];
          f[1] = add2(ld[2], f[2]);
          f[0] = add2(add2(ld[1], f[1]), v);
          f[1] = add2(f[1], v);
          f[2] = add2(f[2], v);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            in[i] = add2(u, in[i]);
            f[i] = mul2(ex2_2(f[i]), d[i]);
          }
          auto put = [&](float (&to)[2][kQ], const f2_t (&x)[4]) {
            *reinterpret_cast<float4*>(to[0] + 4 * lane) = make_float4(lo2(x[0]), lo2(x[1]), lo2(x[2]), lo2(x[3]));
            *reinterpret_cast<float4*>(to[1] + 4 * lane) = make_float4(hi2(x[0]), hi2(x[1]), hi2(x[2]), hi2(x[3]));
          };
          put(a.pre, in);
          put(a.dl, d);
          put(a.f, f);
          __syncwarp();
          if (lane == 0) arrive(bar(kBarA + (k & 1)));
        }
        done(r);
      }
    }
  }

  // Drain: copies and products in flight must be done before shared memory and
  // TMEM are given back (a no-op on the normal path, but for the last y).
  if (lane == 0 && warp >= 16) {
    bool drained = true;
#pragma unroll 1
    for (int i = 0; i < kNumTx; ++i) {
      if (!((armed >> i) & 1u)) continue;
      uint32_t polls = 0;
#pragma unroll 1
      while (!tc::wait(bar(i), (last_par >> i) & 1u, 1) && ++polls < kWaitLimit) {}
      drained &= polls < kWaitLimit;
    }
    if (!drained) atomicOr(&g_fault_prefill, 4u);
    tc::bulk_wait_all();
  }
  tc::fence_before();
  __syncthreads();
  if (!ok) atomicOr(&g_fault_prefill, 2u);
  if (warp == 0) {
    tc::fence_after();
    tc::tmem_dealloc(tmem, 512);
  }
}

int pairs(const SsdPrefillParams& p) { return p.ngroups * ((p.nheads / p.ngroups + 1) / 2); }

template <typename T, int N, bool GATE>
cudaError_t run(const SsdPrefillParams& p, cudaStream_t s) {
  CUtensorMap mx, mb, mc, my;
  std::memset(&my, 0, sizeof(my));
  std::memset(&mx, 0, sizeof(mx));
  std::memset(&mb, 0, sizeof(mb));
  std::memset(&mc, 0, sizeof(mc));
  constexpr bool bf = std::is_same<T, __nv_bfloat16>::value;
  if (p.seq.tokens > 0 &&  // without tokens the maps are never used
      (!tc::encode_2d(&mx, bf, p.x, (int64_t)p.nheads * kP, p.seq.tokens, p.ldx, kQ) ||
       !tc::encode_2d(&mb, bf, p.B, (int64_t)p.ngroups * N, p.seq.tokens, p.ldb, kQ) ||
       !tc::encode_2d(&mc, bf, p.C, (int64_t)p.ngroups * N, p.seq.tokens, p.ldc, kQ) ||
       !tc::encode_2d(&my, bf, p.y, (int64_t)p.nheads * kP, p.seq.tokens, (int64_t)p.nheads * kP, kQ)))
    return cudaErrorInvalidValue;
  const int npairs = pairs(p), blocks = prefill_blocks(p.seq.tokens, p.seq.nseq, npairs, p.sms);
  prefill_plan_kernel<<<1, 1024, 0, s>>>(p, npairs, blocks);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int smem = Lay<N>::kAlloc;
  e = cudaFuncSetAttribute(prefill_tc_kernel<T, N, GATE>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  return launch_behind(prefill_tc_kernel<T, N, GATE>, blocks, kThreads, smem, s, p, npairs, blocks, mx, mb, mc, my);
}

template <typename T>
cudaError_t run_t(const SsdPrefillParams& p, cudaStream_t s) {
  if (p.z) return p.dstate == 128 ? run<T, 128, true>(p, s) : run<T, 64, true>(p, s);
  return p.dstate == 128 ? run<T, 128, false>(p, s) : run<T, 64, false>(p, s);
}

}  // namespace

int prefill_blocks(int64_t tokens, int64_t nseq, int npairs, int sms) {
  const int64_t units = (tokens / kQ + nseq) * npairs;  // at most this many chunks
  const int64_t most = std::max(nseq * npairs, (units + kMinRange - 1) / kMinRange);
  return (int)std::max<int64_t>(1, std::min<int64_t>(most, sms));
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
