// ssv_verify_attn_fp8: verification attention over cached keys in e4m3 pages
// (head_dim 128, bf16 queries and fresh rows, fp32 accumulation).
//
// SimSD summary, section 2 "Temporal Attention Mask" and section 4
// "Verification": O = softmax(scale q K^T | allowed) V, the mask evaluated per
// (row, key) from tau on the fly.
//
// Work unit = (sequence, kv head g, UR consecutive query rows) x the G query
// heads of the group: MT tiles of 128 packed rows, R = 128 / G query rows each
// (row m of a tile is query row m / G, head m % G; rows behind R * G are
// empty).  Its keys are cut into blocks of 128: the cached ones (visible to
// every row), then the fresh ones up to the last a row needs.
//
// Arithmetic of a cached block, on the codes themselves:
//   scores  q = 2^e (hi + lo), hi and lo e4m3, e per row (an element down to
//           2^-10 of the row's largest is exact, the rest off by 2^-18 of it).
//           S = hi K^T + lo K^T on the fp8 tensor path, at the cost of one bf16
//           product and without converting K; the scale of a page enters with
//           2^e as a factor of the column group.  A small kernel before this one
//           writes hi, lo and 2^e of every query row to the workspace.
//   values  converted to fp16, with the page's scale: code * vs / 2^u, u one
//           exponent per unit that follows the largest scale met, from -64 up
//           (a scale that is a power of two is exact down to 2^-20 of the
//           largest).  P = 2^7 exp2(x - m) in fp16: at most 2^15 where the
//           running maximum lags by 2^8, and 11 bits down to weights of 2^-21.
//           O gathers in units of 2^u.
// Fresh blocks: bf16 S; V as it is, P = 2^(7-u) exp2(x - m) in bf16.
//
// Scheduling: persistent, one CTA per SM; per kv head the units' blocks are
// cut into contiguous ranges of equal estimated cost, one per CTA; a unit cut
// across CTAs leaves fp32 partials (O, m, l) in the workspace, merged in CTA
// order by the CTA that holds its first block (bounded wait on per-row-group
// counters).  The plan is derived on the device from seqs.
//
// Roles of a CTA (16 warps, 128 registers each):
//   warp 0        page lookups (32 pages ahead, one per lane), TMA of K pages
//                 (swizzled, the operand itself) and V pages (raw) into rings,
//                 fresh rows into two ring stages at once
//   warp 1        MMA issue for two S / P / O sets in turn: PV(n), S(n + 2), so
//                 that a set's softmax runs under the other set's products.  The
//                 whole warp waits, and one elected lane issues a round's
//                 products and commits in one branch; a predicate on every MMA
//                 took twice the instructions (mixed batch 268 us, 249 us so),
//                 and a loop run by a single lane 1640-2400 cycles for the 1025
//                 of a PV and an S beside busy softmax warps
//   warp 2        query tiles, in the form of the cached and of the fresh blocks
//   warp 3        the scales of the pages, and with them the unit u
//   warps 4..11   softmax, four per set, one TMEM lane quadrant each.  A unit of
//                 two tiles gives each its set (job n: block n / 2); a unit of
//                 one tile gives the sets its blocks in turn (job n: block n),
//                 and the first set joins both at the end
//   warps 12..15  V codes to fp16, fresh V copied (rows behind the last token
//                 become 0, so nothing there is ever multiplied)
// Bounds.  A block of two tiles takes about 3700 cycles of an SM: its products
// alone 2050 (the tensor pipe is 42-50% busy), its two softmaxes alone 1650, and
// each set's S - softmax - P - PV chain leaves gaps that the other does not fill,
// as S, P and O of two sets fill the 512 TMEM columns and no S can be ahead.
// Among the sixteen warps the instruction cache is the other bound: 57 misses per
// product pair with 130 KB of code, and softmax loops at half their speed alone.
// Rolled cold loops and waits beyond the first try out of line brought 20, and the
// mixed batch from 308 to 242 us; with 100 KB the softmax could be unrolled again
// (chunks of 32 columns instead of 16): 232 us.  Rows that do not fill a tile
// cost whole ones: 1.57 (mixed) and 1.94 (long) times the products needed below.
// Measured:
//   8 x 1024 cached keys, 16 / 8 heads             19 us   (bytes: 2.7 us)
//   64 sequences of 256..8192, 32 / 8 heads       232 us   2.6 TB/s, 636 TFLOP/s
//   3 sequences of 90001..110007, pages of 16     267 us   2.4 TB/s, 637 TFLOP/s
//   4 prompts of 2048 over 4096..6200 cached      723 us   1193 TFLOP/s
// Every wait is bounded; an expired one raises the CTA's abort flag, copies and
// MMAs in flight are drained, TMEM is freed and SSV_ERR_TIMEOUT reported.
#include "ssv_internal.cuh"
#include "paged.cuh"
#include "tc_ptx.cuh"

#include <cuda.h>
#include <cudaTypedefs.h>
#include <math.h>

#include <algorithm>
#include <atomic>
#include <mutex>
#include <type_traits>

namespace ssv {
namespace {

using namespace ptx;

constexpr int D = 128;
constexpr int BN = 128;                     // keys per block
constexpr int NK = 4;                       // K ring stages
constexpr int NSC = 8;                      // blocks of page scales in flight
constexpr uint32_t STAGE = 128 * 128;       // one e4m3 tile, or half a 16-bit one
constexpr uint32_t TMEM_COLS = 512;
constexpr int kSoft = 8, kConv = 4, kThreads = 512;
constexpr uint32_t TM_O = 256;              // O of set t at columns 256 + 128 t; S / P at 128 t
constexpr float kLazy = 8.f;                // the running maximum may lag by 2^8
constexpr float kWeight = 7.f;              // P holds weights times 2^7
constexpr float kUnitTop = 7.f;             // vs / 2^u <= 2^7: |code| vs / 2^u < 2^16 in fp16
constexpr float kUnitRoom = 2.f;            // u leaves that much for larger scales to come
// u goes no lower, however small the cached values are (2^-100 is the scale of zero pages): weights of fresh keys are
// then at most 2^(7 + 8 + 64), and O in units of 2^u holds sums of weights times fresh values up to 2^48.
constexpr float kUnitMin = -64.f;
constexpr int SC = 20;                      // words of a block's scales: K factor of every 16 keys x 8, vs / 2^u of
                                            // every 16 keys as an fp16 pair x 8, u
// Estimated costs of the plan, in units of 0.1 us: a block of one / two tiles
// and a segment's fixed work.  (Blocks of one tile take 0.5 of two when alone; 7 : 12 and 40 measured best of 4..10 : 12
// and 20..160 over ragged batches.)
constexpr int kBlock1 = 7, kBlock2 = 12, kSegCost = 40;
// Units cut across CTAs, where there are CTAs to spare: a merge costs about kMergeFixed blocks, and kMergePart for each
// part (they are read one after the other), so parts of sqrt(kMergePart n) blocks end a unit of n soonest.  One head
// of K, one sequence of 16384 keys: 169 us over all CTAs, 38 us so; kMergePart of 0.8 or 2 gives 39 us.
constexpr float kMergeFixed = 4.f, kMergePart = 1.2f;

enum : uint32_t {
  B_K_FULL = 0,
  B_K_EMPTY = B_K_FULL + NK,
  B_R_FULL = B_K_EMPTY + NK,     // raw V ring (at most NK stages)
  B_R_EMPTY = B_R_FULL + NK,
  B_V_FULL = B_R_EMPTY + NK,     // 16-bit V, two stages
  B_V_EMPTY = B_V_FULL + 2,
  B_C_FULL = B_V_EMPTY + 2,      // scales
  B_C_EMPTY = B_C_FULL + NSC,
  B_Q_FULL = B_C_EMPTY + NSC,    // query operand here / its last S complete
  B_Q_EMPTY = B_Q_FULL + 1,
  B_S_FULL = B_Q_EMPTY + 1,      // + set
  B_P_FULL = B_S_FULL + 2,       // + set
  B_SEG_DONE = B_P_FULL + 2,     // every PV of the segment complete
  B_O_FREE = B_SEG_DONE + 1,     // both sets' O read
  B_ML_FULL = B_O_FREE + 1,      // the second set's maxima and sums (one tile)
  B_FINAL = B_ML_FULL + 1,
  B_COUNT = B_FINAL + 1
};

struct AttnFp8Params {
  const float* q_scale;  // [total_rows][Hq]: 2^e of the split queries
  const float *k_scale, *v_scale;
  const int32_t* pages;
  __nv_bfloat16* o;
  int Hq, Hkv, ps_log2, n_pages, table_len;
  float scale;
  const ssv_seq* seqs;
  int batch;
  const int32_t* tau;
  int total_rows, total_slots, max_cache, max_new, max_block;
  int32_t* dev_status;
  long long wait_budget;
  int fault_skip;
  int early;  // the kernel before this one is the query split, which writes nothing but what warps 2 and 4..11 wait for
  int ordered;  // the plan's sums are known to fit 32 bits only for sequences that share no rows: see fp8_layout
};

struct Fp8Maps {
  CUtensorMap kc, vc, kn, vn, q, qhi, qlo;
};

// The counters lie at the front of the workspace, in an area whose size no argument of a call changes, and nothing else
// is ever written there: zero again after a call of any sizes, they are zero before a call of any other.
struct Fp8Work {
  int32_t* cnt;    // [grid][2][4] arrival counters of the unit that a CTA merges (zero between calls)
  int32_t* plan;   // [grid][4][batch + 1] planning tables that do not fit shared memory
  float* part_ml;  // [grid][MT][128][2]
  float* part_o;   // [grid][MT][D / 4][128][4]
};

// Per head: units of total cost Wc dealt to Pe CTAs; this CTA's head g and
// its blocks [begin, end), which start at block k0 of unit u0.  (Wc last: 233 us for the mixed batch of 64, first 237.)
struct PlanHdr {
  int Pe, g, begin, end, u0, k0, Wc;
};

template <int MT>
struct Cfg {
  static constexpr int NR = MT == 1 ? 4 : 2;                // raw V stages
  static constexpr uint32_t SM_Q = 0;                       // per tile: hi, lo; or the bf16 tile
  static constexpr uint32_t SM_K = SM_Q + MT * 2 * STAGE;
  static constexpr uint32_t SM_R = SM_K + NK * STAGE;
  static constexpr uint32_t SM_V = SM_R + NR * STAGE;       // 2 x 32 KB
  static constexpr uint32_t SM_SC = SM_V + 4 * STAGE;       // [NSC][SC]
  static constexpr uint32_t SM_ML = SM_SC + NSC * SC * 4;   // [128] (m, l) of the second set; then its u
  static constexpr uint32_t SM_BAR = SM_ML + 128 * 8 + 8;
  static constexpr uint32_t SM_PLAN = SM_BAR + 8 * B_COUNT + 16;
  static constexpr uint32_t SM_TOTAL = (SM_PLAN + sizeof(PlanHdr) + 15) / 16 * 16;  // planning tables follow
};
constexpr size_t kMaxSmem = 227 * 1024;
static_assert(Cfg<2>::SM_TOTAL <= kMaxSmem && Cfg<1>::SM_TOTAL <= kMaxSmem, "shared memory");
static_assert(Cfg<2>::SM_PLAN % 8 == 0 && Cfg<1>::SM_PLAN % 8 == 0 && Cfg<1>::SM_BAR % 8 == 0, "alignment");

struct Unit {
  int b, C, N, B, rows, q_off, kv_off, tau_off;
  int row0, nvalid, mc, cache_blocks, nblocks, full_new;
};

__device__ __forceinline__ int cdiv(int a, int b) { return (a + b - 1) / b; }

// Bounded wait of a warp that has tried once: out of line, for the sake of the instruction cache (see above).
__device__ __noinline__ bool warp_wait_more(uint32_t bar, uint32_t parity, volatile int* abort, long long budget) {
  const long long t0 = clock64();
  while (true) {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    if (__any_sync(0xffffffffu, *abort != 0)) return false;
    if (__any_sync(0xffffffffu, clock64() - t0 > budget)) {
      *abort = 1;
      return false;
    }
  }
}
// floor(r c / n) of the 32-bit costs c of a head, 0 <= r <= n: rank r's range starts there
__device__ __forceinline__ int cost_start(int r, int c, int n) { return r * (c / n) + r * (c % n) / n; }
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ void mbar_arrive_n(uint32_t bar, uint32_t n) {
  asm volatile("{\n\t.reg .b64 st;\n\tmbarrier.arrive.shared::cta.b64 st, [%0], %1;\n\t}" ::"r"(bar), "r"(n) : "memory");
}

__device__ __forceinline__ void red_release_add(int32_t* p, int v) {
  asm volatile("red.release.gpu.global.add.s32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}
__device__ __forceinline__ int ld_acquire(const int32_t* p) {
  int v;
  asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ bool wait_count(const int32_t* p, int target, volatile int* abort, long long budget) {
  const long long t0 = clock64();
  while (ld_acquire(p) < target) {
    if (*abort) return false;
    if (clock64() - t0 > budget) {
      *abort = 1;
      return false;
    }
  }
  return true;
}

// Float4 group c4 of partial row `slot_row` (= slot * 128 + row): the 32 lanes of a warp
// (consecutive rows) touch 512 contiguous bytes per access.
__device__ __forceinline__ float4* part_at(float* part_o, size_t slot_row, int c4) {
  return reinterpret_cast<float4*>(part_o + (slot_row >> 7) * (128 * D)) + (size_t)c4 * 128 + (slot_row & 127);
}

// bits [0, n) set, n clamped to [0, 32]
__device__ __forceinline__ uint32_t prefix32(int n) {
  return n >= 32 ? 0xffffffffu : (n <= 0 ? 0u : ((1u << n) - 1u));
}

// 32-bit window [t0, t0 + 32) of the 128-bit mask m[1..4], zero outside [0, 128); m[0] = m[5] = 0
__device__ __forceinline__ uint32_t window32(const uint32_t* m, int t0) {
  if (t0 <= -32 || t0 >= 128) return 0u;
  const int w = t0 >> 5;  // floor division
  return __funnelshift_r(m[w + 1], m[w + 2], t0 & 31);
}

// Instruction descriptors: fp32 accumulator, shape 128 x 128, B K-major or MN-major.
constexpr uint32_t kIdShape = (1u << 4) | ((128u >> 3) << 17) | ((128u >> 4) << 24);
constexpr uint32_t kIdE4m3 = kIdShape;                     // kind::f8f6f4, e4m3 x e4m3
constexpr uint32_t kIdBf16 = kIdShape | (1u << 7) | (1u << 10);
constexpr uint32_t kIdPvF16 = kIdShape | (1u << 16);       // kind::f16, f16 x f16, B MN-major
constexpr uint32_t kIdPvBf16 = kIdBf16 | (1u << 16);

__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

// Tensor operations issued by one elected lane of a converged warp: 128 x 128 x 128 products as eight MMAs,
// the first of which accumulates iff acc.
//   gemm_q8: (hi + lo) K^T of e4m3 operands, hi at a, lo 1024 descriptor units behind it, both K-major SW128 like b
//   gemm_qk: bf16 Q K^T, two 64-column halves of either operand 1024 units apart
//   gemm_pv: P V, P in TMEM (two elements per column), V MN-major
__device__ __forceinline__ bool elect_one() {
  uint32_t e;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
  return e != 0;
}
__device__ __forceinline__ void mma_f8(uint32_t d, uint64_t a, uint64_t b, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(kIdE4m3), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void mma_bf16(uint32_t d, uint64_t a, uint64_t b, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(kIdBf16), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void mma_pv(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void gemm_q8(uint32_t d, uint64_t a, uint64_t b) {
#pragma unroll
  for (uint32_t s = 0; s < 8; ++s) mma_f8(d, a + (s >> 2) * 1024 + (s & 3) * 2, b + (s & 3) * 2, s);
}
__device__ __forceinline__ void gemm_qk(uint32_t d, uint64_t a, uint64_t b) {
#pragma unroll 4
  for (uint32_t s = 0; s < 8; ++s) mma_bf16(d, a + (s >> 2) * 1024 + (s & 3) * 2, b + (s >> 2) * 1024 + (s & 3) * 2, s);
}
__device__ __forceinline__ void gemm_pv(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
#pragma unroll
  for (uint32_t s = 0; s < 8; ++s) mma_pv(d, a + s * 8, b + s * 128, idesc, s | acc);
}
__device__ __forceinline__ void commit_elect(uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar)
      : "memory");
}
// 32 lanes x 16 columns and the largest of each lane's 16 values
__device__ __forceinline__ float tmem_max16(uint32_t taddr) {
  [[maybe_unused]] uint32_t r[16];
  float mx;
  asm volatile(
      "tcgen05.ld.red.sync.aligned.32x32b.x16.max.f32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15}, %16, [%17];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=f"(mx)
      : "r"(taddr)
      : "memory");
  return mx;
}

template <int MT>
__global__ void __launch_bounds__(kThreads, 1)
attn_fp8_kernel(const __grid_constant__ Fp8Maps maps, const AttnFp8Params p, const Fp8Work work, int G,
                int plan_smem) {
  using C_ = Cfg<MT>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = smem_u32(smem);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C_::SM_BAR + 8 * B_COUNT);
  volatile int* abort = reinterpret_cast<volatile int*>(smem + C_::SM_BAR + 8 * B_COUNT + 4);
  PlanHdr* plan = reinterpret_cast<PlanHdr*>(smem + C_::SM_PLAN);
  int* s_prefU = plan_smem ? reinterpret_cast<int*>(smem + C_::SM_TOTAL)
                           : work.plan + (size_t)blockIdx.x * 4 * (p.batch + 1);
  int* s_prefB = s_prefU + (p.batch + 1);
  int* s_prefC = s_prefB + (p.batch + 1);
  int* s_ntile = s_prefC + (p.batch + 1);
  auto bar = [&](uint32_t i) -> uint32_t { return sbase + C_::SM_BAR + 8u * i; };

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long wb = p.wait_budget;
  const int R = 128 / G, UR = MT * R, ps = 1 << p.ps_log2, ppb = BN >> p.ps_log2;  // pages per block
  const int cta = blockIdx.x;
  if (sbase & 1023u) {  // the swizzled tiles need it; dynamic shared memory starts there
    if (threadIdx.x == 0) report(p.dev_status, SSV_ERR_CUDA);
    return;
  }

  auto mc_of = [&](int rows, int row0) -> int { return MT == 2 && min(UR, rows - row0) > R ? 2 : 1; };
  auto cost_of = [&](int rows, int row0) -> int { return mc_of(rows, row0) == 2 ? kBlock2 : kBlock1; };
  // key blocks of the unit at row0: the cached ones, then the fresh ones up to its last prompt
  // row (causal), or all where it holds tail rows
  auto blocks_of = [&](int C, int N, int rows, int row0) -> int {
    return cdiv(C, BN) + cdiv(row0 + UR <= N ? row0 + UR : rows, BN);
  };

  // ------------------------------------------------------------------ plan
  if (warp == 0) {
    if (!p.early) pdl_wait();
    int carryU = 0, carryB = 0, carryC = 0, top = 0;  // top: blocks of the longest unit
    int carryE = 0;                                   // end of the rows so far
    for (int b0 = 0; b0 < p.batch; b0 += 32) {
      const int b = b0 + lane;
      int units = 0, blocks = 0, cost = 0;
      ssv_seq s{};
      if (b < p.batch) s = p.seqs[b];
      const bool idle = seq_idle(s);
      const int rows = s.new_len + 2 * s.block;
      const long long np = ((long long)s.cache_len + ps - 1) >> p.ps_log2;
      bool ok = s.cache_len >= 0 && s.new_len >= 0 && s.block >= 1 && s.block <= 64 && s.q_off >= 0 &&
                (long long)s.q_off + s.new_len + 2LL * s.block <= p.total_rows && s.kv_off >= 0 &&
                s.kv_off + np <= p.table_len && s.tau_off >= 0 && (long long)s.tau_off + s.block <= p.total_slots &&
                s.cache_len <= p.max_cache && s.new_len <= p.max_new && s.block <= p.max_block;
      if (p.ordered) {  // (behind a sequence whose rows it shares: refused)
        int e = ok ? s.q_off + rows : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, e, o);
          if (lane >= o) e = max(e, y);
        }
        const int before = __shfl_up_sync(0xffffffffu, e, 1);
        ok = ok && s.q_off >= (lane ? max(before, carryE) : carryE);
        carryE = max(carryE, __shfl_sync(0xffffffffu, e, 31));
      }
      if (!ok && !idle && cta == 0) report(p.dev_status, SSV_ERR_INVALID);
      if (ok) {
        units = cdiv(rows, UR);
#pragma unroll 1
        for (int t = 0; t < units; ++t) {
          const int nb = blocks_of(s.cache_len, s.new_len, rows, t * UR);
          blocks += nb;
          top = max(top, nb);
          cost += kSegCost + cost_of(rows, t * UR) * nb;
        }
      }
      if (b < p.batch) s_ntile[b] = units;
      int iu = units, ib = blocks, ic = cost;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int yu = __shfl_up_sync(0xffffffffu, iu, o), yb = __shfl_up_sync(0xffffffffu, ib, o);
        const int yc = __shfl_up_sync(0xffffffffu, ic, o);
        if (lane >= o) { iu += yu; ib += yb; ic += yc; }
      }
      if (b < p.batch) { s_prefU[b + 1] = carryU + iu; s_prefB[b + 1] = carryB + ib; s_prefC[b + 1] = carryC + ic; }
      carryU += __shfl_sync(0xffffffffu, iu, 31);
      carryB += __shfl_sync(0xffffffffu, ib, 31);
      carryC += __shfl_sync(0xffffffffu, ic, 31);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    __syncwarp();
    if (lane == 0) {
      s_prefU[0] = s_prefB[0] = s_prefC[0] = 0;
      PlanHdr h;
      // CTAs per head: all, unless there are no more units than CTAs and one CTA per unit ends
      // sooner than spreading the blocks and merging
      const int cap = max((int)gridDim.x / p.Hkv, 1);
      int ph = cap;
      if (carryU > 0 && carryU <= cap) {
        const float B = (float)carryB, longest = (float)top;
        const float w = sqrtf(kMergePart * longest);  // blocks per CTA that part and merge a unit soonest
        ph = min(max((int)(B / w + 0.5f), carryU), cap);
        const float each = B / (float)ph;
        if (longest <= each + kMergeFixed + kMergePart * longest / each) ph = carryU;
      }
      // every range at least one block wide, so the CTAs holding a unit's blocks are consecutive
      ph = min(min(ph, max(carryB, 1)), max(carryC / kBlock2, 1));
      h.Pe = ph;
      h.g = cta % p.Hkv;
      h.Wc = carryC;
      // Ranks run against the CTAs' order.  A merge waits on higher ranks, so on CTAs that were dispatched before
      // the waiting one: where other kernels hold some of the SMs it still ends.
      // unit u occupies the costs [c_u, c_u + kSegCost + w n_u), its i-th block sits at
      // c_u + kSegCost + w i; rank r owns the blocks in [r Wc / Pe, (r + 1) Wc / Pe).
      // First block at or after cost c, as (block, unit, offset in the unit):
      auto locate = [&](int c, int& u_out, int& k_out) -> int {
        int lo = 0, hi = p.batch - 1, b = 0;
        while (lo <= hi) {
          const int mid = (lo + hi) >> 1;
          if (s_prefC[mid] <= c) { b = mid; lo = mid + 1; } else { hi = mid - 1; }
        }
        const ssv_seq s = p.seqs[b];
        const int rows = s.new_len + 2 * s.block;
        int xs = s_prefB[b], uu = s_prefU[b];
        int cu = s_prefC[b];
        for (int t = 0;; ++t, ++uu) {
          const int nb = blocks_of(s.cache_len, s.new_len, rows, t * UR), w = cost_of(rows, t * UR);
          if (t >= s_ntile[b] - 1 || cu + kSegCost + w * nb > c) {
            const int dd = c - cu - kSegCost;
            const int i = dd <= 0 ? 0 : min(w == kBlock2 ? cdiv(dd, kBlock2) : cdiv(dd, kBlock1), nb);
            u_out = (i == nb) ? uu + 1 : uu;
            k_out = (i == nb) ? 0 : i;
            return xs + i;
          }
          xs += nb;
          cu += kSegCost + w * nb;
        }
      };
      const int r = ph - 1 - cta / p.Hkv;
      h.begin = h.end = h.u0 = h.k0 = 0;
      if (cta < ph * p.Hkv && carryB > 0) {
        int u1, k1;
        h.begin = locate(cost_start(r, carryC, ph), h.u0, h.k0);
        h.end = (r + 1 == ph) ? carryB : locate(cost_start(r + 1, carryC, ph), u1, k1);
      }
      *plan = h;
    }
  } else if (warp == 1) {
    for (uint32_t i = lane; i < B_COUNT; i += 32) {
      uint32_t n = 1;
      if (i >= B_R_EMPTY && i < B_V_EMPTY) n = kConv;
      if (i >= B_C_EMPTY && i < B_Q_FULL) n = kSoft + kConv;
      if (i == B_O_FREE) n = kSoft;
      if (i == B_P_FULL || i == B_P_FULL + 1 || i == B_ML_FULL) n = 4;
      mbar_init(bar(i), n);
    }
    fence_mbar_init();
    if (lane == 0) *abort = 0;
  } else if (warp == 2) {
    tmem_alloc(smem_u32(tmem_slot), TMEM_COLS);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_trigger();
  const uint32_t tmem = *tmem_slot;
  const int begin = plan->begin, end = plan->end, Ph = plan->Pe, gh = plan->g;
  const int Wc = plan->Wc;
  const int rank = Ph - 1 - cta / p.Hkv;

  auto seq_of = [&](int u) -> int {
    int lo = 0, hi = p.batch - 1, b = 0;
    while (lo <= hi) {
      const int mid = (lo + hi) >> 1;
      if (s_prefU[mid] <= u) { b = mid; lo = mid + 1; } else { hi = mid - 1; }
    }
    return b;
  };
  auto decode = [&](int u) -> Unit {
    Unit x;
    x.b = seq_of(u);
    const ssv_seq s = p.seqs[x.b];
    x.C = s.cache_len; x.N = s.new_len; x.B = s.block;
    x.q_off = s.q_off; x.kv_off = s.kv_off; x.tau_off = s.tau_off;
    x.rows = x.N + 2 * x.B;
    x.row0 = (u - s_prefU[x.b]) * UR;
    x.nvalid = min(UR, x.rows - x.row0);
    x.mc = mc_of(x.rows, x.row0);
    x.cache_blocks = cdiv(x.C, BN);
    x.nblocks = blocks_of(x.C, x.N, x.rows, x.row0);
    x.full_new = (x.row0 < x.N) ? (x.row0 + 1) : x.N;  // fresh keys that every row sees
    return x;
  };
  auto owner_at = [&](int c) -> int {  // rank owning the block at cost c
    int r = (int)((float)c / (float)max(Wc, 1) * (float)Ph);
    r = min(max(r, 0), Ph - 1);
    while (r + 1 < Ph && cost_start(r + 1, Wc, Ph) <= c) ++r;
    while (r > 0 && cost_start(r, Wc, Ph) > c) --r;
    return r;
  };
  auto unit_cost = [&](int u) -> int {  // cost at which unit u starts
    const int b = seq_of(u);
    const ssv_seq s = p.seqs[b];
    const int rows = s.new_len + 2 * s.block;
    int c = s_prefC[b];
#pragma unroll 1
    for (int t = 0; t < u - s_prefU[b]; ++t)
      c += kSegCost + cost_of(rows, t * UR) * blocks_of(s.cache_len, s.new_len, rows, t * UR);
    return c;
  };
  auto warp_wait = [&](uint32_t b, uint32_t parity) -> bool {
    return __all_sync(0xffffffffu, mbar_try_wait(b, parity)) || __all_sync(0xffffffffu, warp_wait_more(b, parity, abort, wb));
  };
  // page of lane `lane` of window w (32 pages) of a segment that starts at block k and holds np pages:
  // -1 behind the last one, -2 where the table names none (reported; read as zeros)
  auto page_at = [&](const Unit& x, int k, int np, int w) -> int {
    const int t = 32 * w + lane;
    if (t >= np) return -1;
    const int pg = p.pages[x.kv_off + (size_t)k * ppb + t];
    if (pg >= 0 && pg < p.n_pages) return pg;
    report(p.dev_status, SSV_ERR_INVALID);
    return -2;
  };
  // ring index n of a ring of S stages: FULL parity of the use, EMPTY parity of the use before
  auto full_par = [](int n, int S) -> uint32_t { return (uint32_t)(n / S) & 1u; };
  auto empty_par = [](int n, int S) -> uint32_t { return (uint32_t)(n / S - 1) & 1u; };

  if (warp == 0) {
    // ============================================================ producer
    if (begin < end) {
      if (lane == 0) { tma_prefetch(&maps.kc); tma_prefetch(&maps.vc); tma_prefetch(&maps.kn); tma_prefetch(&maps.vn); }
      int u = plan->u0, k = plan->k0, remaining = end - begin;
      int n = 0;                 // ring index of K and raw V
      int k_end = 0, v_end = 0;  // behind the last filled stage of either ring
      bool run = true;
      auto take = [&](uint32_t empty, int S) -> bool {  // stage n % S is free
        return n < S || warp_wait(bar(empty + n % S), empty_par(n, S));
      };
      const int row_oob = (int)min((long long)p.n_pages * p.Hkv * ps, 0x7fffffffLL);
      while (run && remaining > 0) {
        const Unit x = decode(u);
        const int len = min(x.nblocks - k, remaining), cached = min(max(x.cache_blocks - k, 0), len);
        // pages of the segment: t = 0 .. np, 32 of them per window, one per lane
        const int np = min(cdiv(x.C, ps), (k + cached) * ppb) - k * ppb;
        int pg0 = page_at(x, k, np, 0), pg1 = page_at(x, k, np, 1);
#pragma unroll 1
        for (int i = 0; run && i < cached; ++i) {
          const int t0 = i * ppb, nb = min(ppb, np - t0);
          if (i > 0 && (t0 & 31) == 0) {
            pg0 = pg1;
            pg1 = page_at(x, k, np, (t0 >> 5) + 1);
          }
          const int pg = __shfl_sync(0xffffffffu, pg0, (t0 + lane) & 31);
          const int row = pg >= 0 ? (pg * p.Hkv + gh) * ps : row_oob;
#pragma unroll 1
          for (int v = 0; run && v < 2; ++v) {  // K, then V
            const int S = v ? C_::NR : NK, st = n & (S - 1);
            if (!take(v ? B_R_EMPTY : B_K_EMPTY, S)) { run = false; break; }
            if (v || cta != 0 || n != p.fault_skip) {  // (test support: this key block's copy is left out)
              const uint32_t full = bar((v ? B_R_FULL : B_K_FULL) + st);
              if (lane == 0) mbar_expect_tx(full, nb * ps * 128);
              __syncwarp();
              if (lane < nb)
                tma_load_2d(sbase + (v ? C_::SM_R : C_::SM_K) + st * STAGE + lane * ps * 128, v ? &maps.vc : &maps.kc, 0, row,
                            full);
            }
            (v ? v_end : k_end) = n + 1;
          }
          if (!run) break;
          ++n;
        }
        // fresh rows: a 16-bit block takes two stages, from an even one on
#pragma unroll 1
        for (int i = cached; run && i < len; ++i) {
          if (n & 1) {
            if (!take(B_K_EMPTY, NK) || !take(B_R_EMPTY, C_::NR)) { run = false; break; }
            if (lane == 0) { mbar_arrive(bar(B_K_FULL + n % NK)); mbar_arrive(bar(B_R_FULL + n % C_::NR)); }
            ++n;
          }
          const int z = x.q_off + (k + i - x.cache_blocks) * BN;
          auto pair = [&](const CUtensorMap* map, uint32_t ring, uint32_t full, uint32_t empty, int S) -> bool {
            if (n >= S && !(warp_wait(bar(empty + n % S), empty_par(n, S)) &&
                            warp_wait(bar(empty + (n + 1) % S), empty_par(n + 1, S))))
              return false;
            if (lane == 0) {
              const uint32_t f = bar(full + n % S), dst = sbase + ring + (n % S) * STAGE;
              mbar_expect_tx(f, 2 * STAGE);
              tma_load_3d(dst, map, 0, gh, z, f);
              tma_load_3d(dst + STAGE, map, 64, gh, z, f);
              mbar_arrive(bar(full + (n + 1) % S));
            }
            __syncwarp();
            return true;
          };
          if (!pair(&maps.kn, C_::SM_K, B_K_FULL, B_K_EMPTY, NK)) { run = false; break; }
          k_end = n + 2;
          if (!pair(&maps.vn, C_::SM_R, B_R_FULL, B_R_EMPTY, C_::NR)) { run = false; break; }
          v_end = n + 2;
          n += 2;
        }
        remaining -= len;
        ++u;
        k = 0;
      }
      // drain (bounded, regardless of abort): the copies that may still be in flight
      auto drain = [&](uint32_t full, int S, int last) {
#pragma unroll 1
        for (int i = max(last - S, 0); i < last; ++i) {
          const long long t0 = clock64();
          while (!mbar_try_wait(bar(full + i % S), full_par(i, S)) && clock64() - t0 < wb) {
          }
        }
      };
      drain(B_K_FULL, NK, k_end);
      drain(B_R_FULL, C_::NR, v_end);
    }
  } else if (warp == 1) {
    // ============================================================ MMA issuer (converged; see above)
    auto uni = [](int v) -> int { return __shfl_sync(0xffffffffu, v, 0); };
    const uint32_t tm = (uint32_t)uni((int)tmem);
    int u = uni(plan->u0), k = uni(plan->k0), remaining = uni(end - begin), nseg = 0;
    int n = 0, nv = 0, nq = 0;       // K ring index, V blocks, query phases
    uint32_t pph0 = 0u, pph1 = 0u;   // parity of the next P of either set
    bool run = true;
    const uint64_t dq0 = smem_desc_sw128(sbase + C_::SM_Q, 16, 1024);
    const uint64_t dk0 = smem_desc_sw128(sbase + C_::SM_K, 16, 1024);
    const uint64_t dv0 = smem_desc_sw128(sbase + C_::SM_V, STAGE, 1024);
    auto wait = [&](uint32_t b, uint32_t parity) -> bool { return warp_wait(bar(b), parity); };
    while (run && remaining > 0) {
      const Unit x = decode(u);
      const int len = uni(min(x.nblocks - k, remaining)), cached = uni(min(max(x.cache_blocks - k, 0), len));
      const bool two = uni(x.mc) == 2;
      const int jobs = two ? 2 * len : len;
      // Round j: PV of job j and S of job j + 2, of the same set.  What does not hang on the weights is waited
      // for first, so that between the weights' arrival and the products there is only their issue.
#pragma unroll 1
      for (int j = -2; run && j < jobs; ++j) {
        const int t = j & 1, js = j + 2, i = two ? js >> 1 : js;  // S: block i
        const bool has_s = js < jobs, q8 = i < cached, last = !two || t == 1;
        if (has_s && (!two || t == 0)) {  // the first job of block i
          if ((i == 0 || i == cached) && !wait(B_Q_FULL, (uint32_t)(nq++) & 1u)) { run = false; break; }
          if (!q8 && (n & 1)) {  // the stage left out
            if (!wait(B_K_FULL + n % NK, full_par(n, NK))) { run = false; break; }
            commit_elect(bar(B_K_EMPTY + n % NK));
            ++n;
          }
          if (!wait(B_K_FULL + n % NK, full_par(n, NK)) || (!q8 && !wait(B_K_FULL + (n + 1) % NK, full_par(n + 1, NK)))) {
            run = false;
            break;
          }
        }
        const uint64_t dq = dq0 + (two ? t : 0) * (2 * STAGE >> 4), dk = dk0 + (n % NK) * (STAGE >> 4);
        const uint64_t dv = dv0 + (nv & 1) * (2 * STAGE >> 4);
        const uint32_t tS = tm + t * 128;
        const bool q_last = i == cached - 1 || i == len - 1;
        const uint32_t id_pv = (two ? j >> 1 : j) < cached ? kIdPvF16 : kIdPvBf16;
        if (j >= 0) {
          if (((!two || t == 0) && !wait(B_V_FULL + (nv & 1), (uint32_t)(nv >> 1) & 1u)) ||
              (j == 0 && nseg > 0 && !wait(B_O_FREE, (nseg - 1) & 1)) || !wait(B_P_FULL + t, t ? pph1 : pph0)) {
            run = false;
            break;
          }
          if (t) pph1 ^= 1u; else pph0 ^= 1u;
        }
        tc_fence_after();
        if (elect_one()) {
          if (j >= 0) gemm_pv(tS + TM_O, tS, dv, id_pv, j > 1 ? 1u : 0u);
          if (has_s) {
            if (q8) gemm_q8(tS, dq, dk);
            else gemm_qk(tS, dq, dk);
            mma_commit(bar(B_S_FULL + t));
            if (last) {
              mma_commit(bar(B_K_EMPTY + n % NK));
              if (!q8) mma_commit(bar(B_K_EMPTY + (n + 1) % NK));
              if (q_last) mma_commit(bar(B_Q_EMPTY));
            }
          }
          if (j >= 0 && last) mma_commit(bar(B_V_EMPTY + (nv & 1)));
        }
        __syncwarp();
        if (has_s && last) n += q8 ? 1 : 2;
        if (j >= 0 && last) ++nv;
      }
      if (!run) break;
      commit_elect(bar(B_SEG_DONE));
      ++nseg;
      remaining -= len;
      ++u;
      k = 0;
    }
    // every MMA issued completes before TMEM is released
    commit_elect(bar(B_FINAL));
    const long long t0 = clock64();
    while (!mbar_try_wait(bar(B_FINAL), 0) && clock64() - t0 < wb) {
    }
  } else if (warp == 2) {
    // ============================================================ query tiles
    if (lane == 0 && begin < end) {
      tma_prefetch(&maps.q); tma_prefetch(&maps.qhi); tma_prefetch(&maps.qlo);
      int u = plan->u0, k = plan->k0, remaining = end - begin, nq = 0;
      bool run = true;
      pdl_wait();  // the split queries come from the kernel before this one
      const uint32_t tile_bytes = R * G * 256;
      while (run && remaining > 0) {
        const Unit x = decode(u);
        const int len = min(x.nblocks - k, remaining), cached = min(max(x.cache_blocks - k, 0), len);
        for (int form = cached > 0 ? 0 : 1; form < (len > cached ? 2 : 1); ++form, ++nq) {
          // the tile is free once the last S of the form before is complete
          if (nq > 0 && !mbar_wait(bar(B_Q_EMPTY), (uint32_t)(nq - 1) & 1u, abort, wb)) { run = false; break; }
          mbar_expect_tx(bar(B_Q_FULL), x.mc * tile_bytes);
#pragma unroll 1
          for (int t = 0; t < x.mc; ++t) {
            const uint32_t dst = sbase + C_::SM_Q + t * 2 * STAGE;
            const int z = x.q_off + x.row0 + t * R;
            tma_load_3d(dst, form ? &maps.q : &maps.qhi, 0, gh * G, z, bar(B_Q_FULL));
            tma_load_3d(dst + STAGE, form ? &maps.q : &maps.qlo, form ? 64 : 0, gh * G, z, bar(B_Q_FULL));
          }
        }
        remaining -= len;
        ++u;
        k = 0;
      }
      if (nq > 0) {  // drain (bounded): the last tiles may still be in flight
        const long long t0 = clock64();
        while (!mbar_try_wait(bar(B_Q_FULL), (uint32_t)(nq - 1) & 1u) && clock64() - t0 < wb) {
        }
      }
    }
  } else if (warp == 3) {
    // ============================================================ scales
    int u = plan->u0, k = plan->k0, remaining = end - begin, nc = 0;
    bool run = true;
    while (run && remaining > 0) {
      const Unit x = decode(u);
      const int len = min(x.nblocks - k, remaining), cached = min(max(x.cache_blocks - k, 0), len);
      const int np = min(cdiv(x.C, ps), (k + cached) * ppb) - k * ppb;
      float unit = 0.f, kf = 0.f, lv = -126.f, ks1, vs1;
      auto fetch = [&](int w) {
        const int pg = page_at(x, k, np, w);
        ks1 = vs1 = 0.f;
        if (pg >= 0) {
          ks1 = __ldg(p.k_scale + (size_t)pg * p.Hkv + gh);
          vs1 = __ldg(p.v_scale + (size_t)pg * p.Hkv + gh);
        }
      };
      if (cached > 0) fetch(0);
#pragma unroll 1
      for (int i = 0; i < cached; ++i) {
        const int t0 = i * ppb, nb = min(ppb, np - t0);
        if ((t0 & 31) == 0) {  // the window's pages, and the loads of the next
          kf = ks1 * (p.scale * 1.4426950408889634f);
          lv = fmaxf(log2f(vs1), -126.f);
          fetch((t0 >> 5) + 1);
        }
        // lane < 8: its 16 keys' page (the last one again behind it)
        const int src = t0 + min((lane & 7) >> (p.ps_log2 - 4), nb - 1);
        const float kf16 = __shfl_sync(0xffffffffu, kf, src & 31), lv16 = __shfl_sync(0xffffffffu, lv, src & 31);
        float top = lv16;
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        if (i == 0 || top > unit + kUnitTop) unit = fmaxf(ceilf(top) + kUnitRoom - kUnitTop, kUnitMin);
        if (nc >= NSC && !warp_wait(bar(B_C_EMPTY + nc % NSC), empty_par(nc, NSC))) { run = false; break; }
        float* sc = reinterpret_cast<float*>(smem + C_::SM_SC) + (nc % NSC) * SC;
        if (lane < 8) {
          const __half2 f = __float2half2_rn(ex2(lv16 - unit));
          sc[lane] = kf16;
          reinterpret_cast<uint32_t*>(sc)[8 + lane] = *reinterpret_cast<const uint32_t*>(&f);
        }
        if (lane == 0) sc[16] = unit;
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(B_C_FULL + nc % NSC));
        ++nc;
      }
      remaining -= len;
      ++u;
      k = 0;
    }
  } else if (warp >= 12) {
    // ============================================================ converters
    const int ct = threadIdx.x - 32 * 12;
    constexpr int NT = 32 * kConv;
    int u = plan->u0, k = plan->k0, remaining = end - begin;
    int n = 0, nv = 0, nc = 0;
    bool run = true;
    while (run && remaining > 0) {
      const Unit x = decode(u);
      const int len = min(x.nblocks - k, remaining), cached = min(max(x.cache_blocks - k, 0), len);
      auto v_ready = [&]() -> bool {  // the 16-bit stage of V block nv is free
        return nv < 2 || warp_wait(bar(B_V_EMPTY + (nv & 1)), (uint32_t)((nv >> 1) - 1) & 1u);
      };
      auto v_done = [&](int stages) {
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(bar(B_V_FULL + (nv & 1)));
          for (int e = 0; e < stages; ++e) mbar_arrive(bar(B_R_EMPTY + (n + e) % C_::NR));
        }
        n += stages;
        ++nv;
      };
      if (cached > 0) {
#pragma unroll 1
        for (int i = 0; i < cached; ++i) {
          if (!warp_wait(bar(B_C_FULL + nc % NSC), full_par(nc, NSC)) ||
              !warp_wait(bar(B_R_FULL + n % C_::NR), full_par(n, C_::NR)) || !v_ready()) {
            run = false;
            break;
          }
          const float* sc = reinterpret_cast<const float*>(smem + C_::SM_SC) + (nc % NSC) * SC;
          const int keys = x.C - (k + i) * BN;  // rows behind it become zeros
          static_assert(NT == 128, "sixteen keys per round");
          // this thread: 16 codes (chunk c) of a key in sixteen, which become 16-byte chunks 2 c, 2 c + 1 of the key's
          // 256 bytes in two 64-element columns.  Eight lanes read chunks 0..3 of one key and 4..7 of its
          // neighbour, so that both their reads and their writes (swizzled by the key) meet all banks.
          const int c = ct & 7, key0 = (ct >> 3) ^ (c >> 2), c0 = (c & 3) * 2, sw = key0 & 7;
          const uint8_t* raw = smem + C_::SM_R + (n % C_::NR) * STAGE + key0 * 128 + c * 16;
          uint8_t* dst = smem + C_::SM_V + (nv & 1) * 2 * STAGE + (c >> 2) * STAGE + key0 * 128;
          uint8_t *dst0 = dst + ((c0 ^ sw) << 4), *dst1 = dst + (((c0 + 1) ^ sw) << 4);
#pragma unroll 1
          for (int g = 0; g < 8; g += 4) {
            uint4 s[4];
#pragma unroll
            for (int it = 0; it < 4; ++it) s[it] = *reinterpret_cast<const uint4*>(raw + (g + it) * 16 * 128);
            if (keys < BN) {
#pragma unroll
              for (int it = 0; it < 4; ++it)
                if ((g + it) * 16 + key0 >= keys) s[it] = make_uint4(0, 0, 0, 0);
            }
            const uint4 f4 = reinterpret_cast<const uint4*>(sc)[2 + (g >> 2)];
            const uint32_t f[4] = {f4.x, f4.y, f4.z, f4.w};
#pragma unroll
            for (int it = 0; it < 4; ++it) {
              const uint32_t w[4] = {s[it].x, s[it].y, s[it].z, s[it].w};
              uint32_t h[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const uint32_t v = e4m3x2_to_f16x2((uint16_t)(w[e >> 1] >> (16 * (e & 1))));
                const __half2 y = __hmul2(*reinterpret_cast<const __half2*>(&v), *reinterpret_cast<const __half2*>(&f[it]));
                h[e] = *reinterpret_cast<const uint32_t*>(&y);
              }
              *reinterpret_cast<uint4*>(dst0 + (g + it) * 16 * 128) = make_uint4(h[0], h[1], h[2], h[3]);
              *reinterpret_cast<uint4*>(dst1 + (g + it) * 16 * 128) = make_uint4(h[4], h[5], h[6], h[7]);
            }
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(B_C_EMPTY + nc % NSC));
          ++nc;
          v_done(1);
        }
      }
      if (run && len > cached) {
#pragma unroll 1
        for (int i = cached; i < len; ++i) {
          if (n & 1) {  // the stage left out
            if (!warp_wait(bar(B_R_FULL + n % C_::NR), full_par(n, C_::NR))) { run = false; break; }
            if (lane == 0) mbar_arrive(bar(B_R_EMPTY + n % C_::NR));
            ++n;
          }
          if (!warp_wait(bar(B_R_FULL + n % C_::NR), full_par(n, C_::NR)) ||
              !warp_wait(bar(B_R_FULL + (n + 1) % C_::NR), full_par(n + 1, C_::NR)) || !v_ready()) {
            run = false;
            break;
          }
          const uint4* raw = reinterpret_cast<const uint4*>(smem + C_::SM_R + (n % C_::NR) * STAGE);
          uint4* dst = reinterpret_cast<uint4*>(smem + C_::SM_V + (nv & 1) * 2 * STAGE);
          const int keys = x.rows - (k + i - x.cache_blocks) * BN;
#pragma unroll 4
          for (int idx = ct; idx < 2048; idx += NT)
            dst[idx] = ((idx & 1023) >> 3) < keys ? raw[idx] : make_uint4(0, 0, 0, 0);
          v_done(2);
        }
      }
      remaining -= len;
      ++u;
      k = 0;
    }
  } else if (warp >= 4) {
    // ============================================================ softmax
    const int set = (warp - 4) >> 2, q4 = warp & 3, m = q4 * 32 + lane;
    const uint32_t lane_base = static_cast<uint32_t>(q4 * 32) << 16;
    const uint32_t tS = tmem + lane_base + set * 128, tO = tmem + lane_base + TM_O + set * 128;
    const float cexp = p.scale * 1.4426950408889634f;
    int u = plan->u0, k = plan->k0, remaining = end - begin, seg = 0;
    int nc = 0, nml = 0;  // cached blocks, joins so far
    uint32_t sph = 0u;            // parity of this set's next S
    bool run = true;
    pdl_wait();  // the row factors come from the kernel before this one
    while (run && remaining > 0) {
      const Unit x = decode(u);
      const int len = min(x.nblocks - k, remaining), cached = min(max(x.cache_blocks - k, 0), len);
      const bool complete = (k == 0 && len == x.nblocks);
      const bool two = x.mc == 2;
      const int mt = two ? set : 0, jobs = two ? 2 * len : len;
      {
        const int r_local = mt * R + m / G, hj = m % G;
        const int i = x.row0 + r_local;  // local query row
        const bool valid = m < R * G && r_local < x.nvalid;
        const bool warp_active = q4 * 32 < R * G && (mt * R + (q4 * 32) / G) < x.nvalid;
        // (the kernel that writes the factors may have run beside this one's start: not read as constant data)
        const float rowf = cached > 0 && valid ? __ldcg(p.q_scale + (size_t)(x.q_off + i) * p.Hq + gh * G + hj) : 1.f;
        const bool prompt = i < x.N;
        const int r = i - x.N;
        uint32_t tm[6] = {0u, 0u, 0u, 0u, 0u, 0u};  // allowed tail keys of this row (in local memory: seldom read)
        if (warp_active && len > cached && x.row0 + x.nvalid > x.N) {  // warp-uniform: fresh blocks and tail rows
          const int32_t* tau = p.tau + x.tau_off;
          const int ta = lane < x.B ? tau[lane] : 0, tb = lane + 32 < x.B ? tau[lane + 32] : 0;
          const bool tail_row = valid && !prompt;
          const int slot_r = tail_row ? (r % x.B) : 0;
          const int tra = __shfl_sync(0xffffffffu, ta, slot_r & 31), trb = __shfl_sync(0xffffffffu, tb, slot_r & 31);
          const int tr = slot_r < 32 ? tra : trb;
          // le / lt: the slots whose stage is <= tr / < tr, one ballot pair per stage
          unsigned long long acc = 0ull, le = 0ull, lt = 0ull;
          bool bad = false;  // (a bad stage map cannot index out of range: report only)
#pragma unroll 1
          for (int v = 1; v <= x.B; ++v) {
            const uint32_t lo = __ballot_sync(0xffffffffu, ta == v), hi = __ballot_sync(0xffffffffu, tb == v);
            acc |= ((unsigned long long)hi << 32) | lo;
            bad |= __popc(lo) + __popc(hi) != 1;
            if (v == tr - 1) lt = acc;
            if (v == tr) le = acc;
          }
          if (bad && lane == 0) report(p.dev_status, SSV_ERR_BAD_TAU);
          // a data row sees the data slots of stages <= its own; a mask row the data slots of
          // earlier stages and the mask slots of its own stage and later ones
          const unsigned long long bmask = (x.B >= 64) ? ~0ull : ((1ull << x.B) - 1ull);
          const bool data_row = r < x.B;
          const unsigned long long lo_part = !tail_row ? 0ull : (data_row ? le : lt);
          const unsigned long long hi_part = (!tail_row || data_row) ? 0ull : (~lt & bmask);
          const unsigned long long w01 = lo_part | (x.B < 64 ? (hi_part << x.B) : 0ull);
          const unsigned long long w23 = x.B < 64 ? (hi_part >> (64 - x.B)) : hi_part;
          tm[1] = (uint32_t)w01; tm[2] = (uint32_t)(w01 >> 32);
          tm[3] = (uint32_t)w23; tm[4] = (uint32_t)(w23 >> 32);
        }
        // rows without a query follow along unmasked, whatever their tile rows hold, and are dropped at the end
        float m_used = valid ? -INFINITY : 0.f, l_sum = 0.f, unit = 0.f;
#pragma unroll 1
        for (int job = set; job < jobs; job += 2) {
          const int jj = two ? job >> 1 : job, j = k + jj;
          const bool is_cache = jj < cached, first = job == set;
          const int e = nc + jj;  // scales of the block
          // ---- the block's scales: factors of the scores of every 16 columns, the unit of O
          float unit_new = first ? 0.f : unit;
          const float* sc = reinterpret_cast<const float*>(smem + C_::SM_SC) + (e % NSC) * SC;
          if (is_cache) {
            if (!warp_wait(bar(B_C_FULL + e % NSC), full_par(e, NSC))) { run = false; break; }
            unit_new = sc[16];
          }
          auto factor = [&](int q) -> float {  // of columns [16 q, 16 q + 16)
            return is_cache ? fmaxf(rowf * sc[q], 1.17549435e-38f) : cexp;
          };
          // (a block that one set alone works on is given back by it for both)
          auto give_back = [&]() {
            __syncwarp();
            if (lane == 0) {
              if (is_cache) mbar_arrive_n(bar(B_C_EMPTY + e % NSC), two ? 1 : 2);
              mbar_arrive(bar(B_P_FULL + set));
            }
          };
          if (!warp_wait(bar(B_S_FULL + set), sph)) { run = false; break; }
          sph ^= 1u;
          if (!warp_active) {
            give_back();
            continue;
          }
          tc_fence_after();
          // ---- which of the 128 keys this row sees
          const int kbase = is_cache ? j * BN : (j - x.cache_blocks) * BN;
          const bool full = is_cache ? (kbase + BN <= x.C) : (kbase + BN <= x.full_new);
          int lim = BN, lim_rows = 0, toff = 0;  // a prefix, and tail bits for columns < lim_rows
          if (!full) {
            if (is_cache) {
              lim = x.C - kbase;
            } else if (prompt) {
              lim = min(i + 1, x.rows) - kbase;
            } else {
              lim = x.N - kbase;
              lim_rows = x.rows - kbase;
              toff = kbase - x.N;
            }
          }
          auto vis32 = [&](int q) -> uint32_t {
            uint32_t v = prefix32(lim - 32 * q);
            if (lim_rows > 32 * q) v |= window32(tm, toff + 32 * q) & prefix32(lim_rows - 32 * q);
            return v;
          };
          const float shift = is_cache ? kWeight : kWeight - unit_new;  // P = exp2(x - m + shift)
          float lsum = 0.f;  // of P
          // ---- the row's maximum over the block
          float mx = -INFINITY;
          if (full) {
#pragma unroll
            for (int g = 0; g < 2; ++g) {
              float a[4], f[4];
#pragma unroll
              for (int h = 0; h < 4; ++h) f[h] = factor(4 * g + h);
#pragma unroll
              for (int h = 0; h < 4; ++h) a[h] = tmem_max16(tS + g * 64 + h * 16);
              tmem_wait_ld();
#pragma unroll
              for (int h = 0; h < 4; ++h) mx = fmaxf(mx, a[h] * f[h]);
            }
          } else {
#pragma unroll 1
            for (int q = 0; q < BN / 16; ++q) {
              uint32_t sr[16];
              tmem_ld16(tS + q * 16, sr);
              tmem_wait_ld();
              const uint32_t vw = vis32(q >> 1) >> ((q & 1) * 16);
              float a = -INFINITY;
#pragma unroll
              for (int v = 0; v < 16; ++v) a = fmaxf(a, ((vw >> v) & 1u) ? __uint_as_float(sr[v]) : -INFINITY);
              mx = fmaxf(mx, a * factor(q));
            }
          }
          // ---- the reference may lag behind it; O is brought to a new one, or to a new unit
          const bool need = mx > -INFINITY && (m_used == -INFINITY || mx > m_used + kLazy);
          if (!first && __any_sync(0xffffffffu, need || unit_new != unit)) {
            // O of this set holds its earlier PVs; they are complete, as S of this job was issued behind them
            const float fm = need ? ex2(m_used - mx) : 1.f;
            const float f = fm * ex2(unit - unit_new);
            uint32_t raw[32];
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
              tmem_ld32(tO + c * 32, raw);
              tmem_wait_ld();
#pragma unroll
              for (int v = 0; v < 32; ++v) raw[v] = __float_as_uint(__uint_as_float(raw[v]) * f);
              tmem_st32(tO + c * 32, raw);
            }
            tmem_wait_st();
            l_sum *= fm;
          }
          if (need) m_used = mx;
          const float off = shift - ((m_used == -INFINITY) ? 0.f : m_used);
          // ---- P = exp2(x - m + shift) over S: chunk q reads S columns [32 q, 32 q + 32) and writes P columns
          // [16 q, 16 q + 16), which lie in S columns already read
          auto exps = [&](auto cache_tag) {
            constexpr bool kCache = decltype(cache_tag)::value;
            const uint64_t of2 = pack2(off, off);
            uint64_t lp0 = 0ull, lp1 = 0ull;
            uint32_t b0[32], b1[32];
            tmem_ld32(tS, b0);
            tmem_wait_ld();
            auto chunk = [&](int q, const uint32_t* cur, float ca, float cb) {
              uint32_t pw[16];
#pragma unroll
              for (int v = 0; v < 16; ++v) {
                const float c = v < 8 ? ca : cb;
                const uint64_t cc2 = pack2(c, c);
                float x0, x1;
                unpack2(ffma2(pack2(__uint_as_float(cur[2 * v]), __uint_as_float(cur[2 * v + 1])), cc2, of2), x0, x1);
                const float p0 = ex2(x0), p1 = ex2(x1);
                if constexpr (kCache) {
                  const __half2 w = __floats2half2_rn(p0, p1);
                  pw[v] = *reinterpret_cast<const uint32_t*>(&w);
                } else {
                  const __nv_bfloat162 w = __floats2bfloat162_rn(p0, p1);
                  pw[v] = *reinterpret_cast<const uint32_t*>(&w);
                }
                if (v & 1) lp1 = fadd2(lp1, pack2(p0, p1)); else lp0 = fadd2(lp0, pack2(p0, p1));
              }
              tmem_wait_ld();  // the next chunk is here, so this one's P may go over it
              tmem_st16(tS + q * 16, pw);
            };
#pragma unroll 1
            for (int q = 0; q < 4; q += 2) {
              const float f[4] = {factor(2 * q), factor(2 * q + 1), factor(2 * q + 2), factor(2 * q + 3)};
              tmem_ld32(tS + (q + 1) * 32, b1);
              chunk(q, b0, f[0], f[1]);
              if (q < 2) tmem_ld32(tS + (q + 2) * 32, b0);
              chunk(q + 1, b1, f[2], f[3]);
            }
            float y0, y1;
            unpack2(fadd2(lp0, lp1), y0, y1);
            lsum = y0 + y1;
          };
          if (full) {
            if (is_cache) exps(std::true_type{});
            else exps(std::false_type{});
          } else {
#pragma unroll 1
            for (int q = 0; q < BN / 16; ++q) {
              uint32_t sr[16], pw[8];
              tmem_ld16(tS + q * 16, sr);
              tmem_wait_ld();
              const uint32_t vw = vis32(q >> 1) >> ((q & 1) * 16);
              const float c = factor(q);
#pragma unroll
              for (int v = 0; v < 8; ++v) {
                const float p0 = ((vw >> (2 * v)) & 1u) ? ex2(fmaf(__uint_as_float(sr[2 * v]), c, off)) : 0.f;
                const float p1 = ((vw >> (2 * v + 1)) & 1u) ? ex2(fmaf(__uint_as_float(sr[2 * v + 1]), c, off)) : 0.f;
                if (is_cache) {
                  const __half2 w = __floats2half2_rn(p0, p1);
                  pw[v] = *reinterpret_cast<const uint32_t*>(&w);
                } else {
                  const __nv_bfloat162 w = __floats2bfloat162_rn(p0, p1);
                  pw[v] = *reinterpret_cast<const uint32_t*>(&w);
                }
                lsum += p0 + p1;
              }
              tmem_st8(tS + q * 8, pw);
            }
          }
          unit = unit_new;
          if (!is_cache) lsum *= ex2(unit_new);  // the row sum counts 2^7 exp2(x - m)
          tmem_wait_st();
          l_sum += lsum;
          tc_fence_before();
          give_back();
        }
        nc += cached;
        if (!run) break;
        // ---- epilogue: every PV of the segment is complete; O stays in TMEM until O_FREE
        if (!warp_wait(bar(B_SEG_DONE), seg & 1)) {
          run = false;
          break;
        }
        float f0 = exp2f(unit), f1 = 0.f;  // factors of this set's O and, where they are joined, the other's
        bool join = false;
        if (!two) {
          float2* ml = reinterpret_cast<float2*>(smem + C_::SM_ML);
          float* ml_unit = reinterpret_cast<float*>(smem + C_::SM_ML + 128 * 8);
          if (set == 1) {
            // the first set joins both; what it needs besides O:
            ml[m] = make_float2(m_used, l_sum);
            if (m == 0) *ml_unit = unit;
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
              mbar_arrive(bar(B_ML_FULL));
              mbar_arrive(bar(B_O_FREE));
            }
          } else {
            if (!warp_wait(bar(B_ML_FULL), (uint32_t)(nml++) & 1u)) { run = false; break; }
            join = jobs > 1;  // else the second set has had no block, and its O holds nothing
            if (join) {
              const float2 o = ml[m];
              const float M = fmaxf(m_used, o.x);
              const float g0 = M == -INFINITY ? 0.f : ex2(m_used - M), g1 = M == -INFINITY ? 0.f : ex2(o.x - M);
              l_sum = l_sum * g0 + o.y * g1;
              f0 *= g0;
              f1 = exp2f(*ml_unit) * g1;
              m_used = M;
            }
          }
        }
        if (two || set == 0) {
        if (warp_active) {
          tc_fence_after();
          // 32 columns of O, joined, in true units
          auto load_o = [&](int q, float* v, float f) {
            uint32_t raw[32];
            tmem_ld32(tO + q * 32, raw);
            tmem_wait_ld();
#pragma unroll
            for (int c = 0; c < 32; ++c) v[c] = __uint_as_float(raw[c]) * (f0 * f);
            if (join) {
              tmem_ld32(tO + 128 + q * 32, raw);
              tmem_wait_ld();
#pragma unroll
              for (int c = 0; c < 32; ++c) v[c] = fmaf(__uint_as_float(raw[c]), f1 * f, v[c]);
            }
          };
          __nv_bfloat16* orow = p.o + ((size_t)(x.q_off + i) * p.Hq + gh * G + hj) * D;
          auto store_chunk = [&](int q, const float* v, float inv) {
            if (!valid) return;
#pragma unroll
            for (int c = 0; c < 32; c += 8) {
              uint32_t w[4];
#pragma unroll
              for (int h = 0; h < 4; ++h) {
                const __nv_bfloat162 bv = __floats2bfloat162_rn(v[c + 2 * h] * inv, v[c + 2 * h + 1] * inv);
                w[h] = *reinterpret_cast<const uint32_t*>(&bv);
              }
              *reinterpret_cast<uint4*>(orow + q * 32 + c) = make_uint4(w[0], w[1], w[2], w[3]);
            }
          };
          if (complete) {
            const float inv = (l_sum > 0.f) ? 1.f / l_sum : NAN;  // (every row sees its own key)
#pragma unroll 1
            for (int q = 0; q < D / 32; ++q) {
              float v[32];
              load_o(q, v, 1.f);
              store_chunk(q, v, inv);
            }
          } else {
            // ---- a unit cut across ranks c_a .. c_b of the head: c_a holds its first block, at the end of
            // its own range, and merges; the others publish their partials and move on
            const int cu = unit_cost(u) + kSegCost;
            const int c_a = owner_at(cu);
            const int c_b = owner_at(cu + cost_of(x.rows, x.row0) * (x.nblocks - 1));
            // (a cut unit ends c_a's range, so a CTA merges one unit at most, and its counters serve that one)
            int32_t* counter = work.cnt + ((c_a * p.Hkv + gh) * 2 + mt) * 4 + q4;
            auto slot_of = [&](int rr) -> size_t { return ((size_t)(rr * p.Hkv + gh) * MT + mt) * 128 + m; };
            if (rank != c_a) {
              const size_t mine = slot_of(rank);
              __stcg(reinterpret_cast<float2*>(work.part_ml + mine * 2), make_float2(m_used, l_sum));
#pragma unroll 1
              for (int q = 0; q < D / 32; ++q) {
                float v[32];
                load_o(q, v, 1.f);
#pragma unroll
                for (int c = 0; c < 32; c += 4)
                  __stcg(part_at(work.part_o, mine, q * 8 + c / 4), make_float4(v[c], v[c + 1], v[c + 2], v[c + 3]));
              }
              __syncwarp();
              if (lane == 0) red_release_add(counter, 1);
            } else {
              int ok = 1;
              if (lane == 0) ok = wait_count(counter, c_b - c_a, abort, wb) ? 1 : 0;
              ok = __shfl_sync(0xffffffffu, ok, 0);
              __syncwarp();
              if (!ok) run = false;
            }
            if (rank == c_a && run) {
              // in CTA order, so that equal inputs give equal bits
              float M = m_used;
#pragma unroll 1
              for (int cc = c_a + 1; cc <= c_b; ++cc) M = fmaxf(M, __ldcg(work.part_ml + slot_of(cc) * 2));
              const float g = M == -INFINITY ? 0.f : ex2(m_used - M);
              float L = l_sum * g;
#pragma unroll 1
              for (int cc = c_a + 1; cc <= c_b; ++cc) {
                const float2 ml = __ldcg(reinterpret_cast<const float2*>(work.part_ml + slot_of(cc) * 2));
                if (M > -INFINITY) L += ml.y * ex2(ml.x - M);
              }
              const float inv = (L > 0.f) ? 1.f / L : NAN;
#pragma unroll 1
              for (int q = 0; q < D / 32; ++q) {
                float v[32];
                load_o(q, v, g);
#pragma unroll 1
                for (int cc = c_a + 1; cc <= c_b; ++cc) {
                  const size_t sl = slot_of(cc);
                  const float f = (M == -INFINITY) ? 0.f : ex2(__ldcg(work.part_ml + sl * 2) - M);
                  float4 w4[8];
#pragma unroll
                  for (int c = 0; c < 8; ++c) w4[c] = __ldcg(part_at(work.part_o, sl, q * 8 + c));
#pragma unroll
                  for (int c = 0; c < 8; ++c) {
                    v[4 * c] += w4[c].x * f; v[4 * c + 1] += w4[c].y * f;
                    v[4 * c + 2] += w4[c].z * f; v[4 * c + 3] += w4[c].w * f;
                  }
                }
                store_chunk(q, v, inv);
              }
              if (lane == 0) *counter = 0;  // ready for the next call
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(B_O_FREE));
        }
      }
      remaining -= len;
      ++seg;
      ++u;
      k = 0;
    }
  }
  // ------------------------------------------------------------------ teardown
  __syncwarp();
  pdl_wait();  // this grid never completes before the one it follows
  tc_fence_before();
  __syncthreads();
  if (*abort && threadIdx.x == 0) report(p.dev_status, SSV_ERR_TIMEOUT);
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc(tmem, TMEM_COLS);
  }
}

// ---------------------------------------------------------------------------
// The queries of a pass as 2^e (hi + lo): sixteen lanes per (row, head), eight elements each; one read of Q
// and one write of the same bytes.
// ---------------------------------------------------------------------------
constexpr int kSplitThreads = 256;

__global__ void __launch_bounds__(kSplitThreads) query_split_kernel(const uint4* q, uint2* hi, uint2* lo, float* scale,
                                                                    long long heads) {
  pdl_wait();
  pdl_trigger();  // every kernel before this one is complete: the next may read what they wrote
  const long long h = ((long long)blockIdx.x * kSplitThreads + threadIdx.x) >> 4;
  const int c = threadIdx.x & 15;
  uint4 v = make_uint4(0, 0, 0, 0);
  if (h < heads) v = __ldcg(q + h * 16 + c);  // (nor here: the kernel before may write q while this one starts)
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  float x[8], amax = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (fabsf(x[i]) < INFINITY) amax = fmaxf(amax, fabsf(x[i]));
    else x[i] = NAN;  // an infinity would be clamped
  }
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  // smallest e >= -100 with amax <= 448 2^e = 1.75 2^(e + 8)
  const uint32_t bits = __float_as_uint(amax);
  const int ex = max((int)(bits >> 23) - 127 - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0), -100);
  const float f = __uint_as_float((uint32_t)(127 - ex) << 23);
  uint16_t hh[4], ll[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float a = x[2 * i] * f, b = x[2 * i + 1] * f;
    hh[i] = f32_to_e4m3x2(a, b);
    const uint32_t back = e4m3x2_to_f16x2(hh[i]);
    const float2 r = __half22float2(*reinterpret_cast<const __half2*>(&back));
    ll[i] = f32_to_e4m3x2(a - r.x, b - r.y);
  }
  if (h >= heads) return;
  hi[h * 16 + c] = make_uint2(hh[0] | (uint32_t)hh[1] << 16, hh[2] | (uint32_t)hh[3] << 16);
  lo[h * 16 + c] = make_uint2(ll[0] | (uint32_t)ll[1] << 16, ll[2] | (uint32_t)ll[3] << 16);
  if (c == 0) scale[h] = __uint_as_float((uint32_t)(127 + ex) << 23);
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
PFN_cuTensorMapEncodeTiled_v12000 fp8_encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  });
  return fn;
}

// [rows, 128] codes, one page of one head per box
bool encode_pages(CUtensorMap* m, const void* base, long long rows, int page, CUtensorMapSwizzle sw) {
  const cuuint64_t dims[2] = {128, (cuuint64_t)rows}, strides[1] = {128};
  const cuuint32_t box[2] = {128, (cuuint32_t)page}, es[2] = {1, 1};
  return fp8_encode_fn()(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, es,
                         CU_TENSOR_MAP_INTERLEAVE_NONE, sw, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// [rows, heads, 128] elements of `es` bytes (bf16 or e4m3), rows `stride` elements apart; a box is 128 bytes of
// box_heads heads of box_rows rows
bool encode_rows(CUtensorMap* m, const void* base, int es, int heads, long long rows, long long stride, int box_heads,
                 int box_rows) {
  const cuuint64_t dims[3] = {128, (cuuint64_t)heads, (cuuint64_t)rows};
  const cuuint64_t strides[2] = {(cuuint64_t)(128 * es), (cuuint64_t)(stride * es)};
  const cuuint32_t box[3] = {(cuuint32_t)(128 / es), (cuuint32_t)box_heads, (cuuint32_t)box_rows}, steps[3] = {1, 1, 1};
  return fp8_encode_fn()(m, es == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8, 3,
                         const_cast<void*>(base), dims, strides, box, steps, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct Fp8Layout {
  size_t cnt, plan, ml, o, q, qs, total;
  int grid, mt, ordered;
};

// Two tiles share a unit's keys where some sequence fills more than one.
bool fp8_layout(const ssv_attn_fp8_args* a, Fp8Layout* L) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&L->grid, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    L->grid = 152;  // no device: the size of a GB300
  const int G = a->Hq / a->Hkv, R = 128 / G;
  const long long max_rows = (long long)a->max_new + 2LL * a->max_block;
  L->mt = max_rows > R ? 2 : 1;
  const long long tiles = (max_rows + (long long)L->mt * R - 1) / (L->mt * R);
  // The plan's sums are 32-bit.  They hold for any records where every sequence may be as long as the longest; where
  // not, sequences that share no rows have total_rows between them, which the kernel then checks of them.
  const long long most = (1LL << 30) / kBlock2, per = a->max_cache / BN + max_rows / BN + 2 + kSegCost / kBlock1 + 1;
  const long long units = std::min(a->batch * tiles, a->total_rows / ((long long)L->mt * R) + a->batch);
  if (units > most / per || a->Hkv > L->grid) return false;
  L->ordered = a->batch * tiles > most / per ? 1 : 0;
  size_t off = 0;
  L->cnt = off;  // first, and of one size: see Fp8Work
  off = align_up(off + sizeof(int32_t) * (size_t)L->grid * 2 * 4, 256);
  L->plan = off;
  off = align_up(off + sizeof(int32_t) * (size_t)L->grid * 4 * (a->batch + 1), 256);
  L->ml = off;
  off = align_up(off + sizeof(float) * 2 * (size_t)L->grid * L->mt * 128, 256);
  L->o = off;
  off = align_up(off + sizeof(float) * (size_t)L->grid * L->mt * 128 * D, 256);
  // the split queries, where keys may be cached
  const size_t heads = a->max_cache > 0 ? (size_t)a->total_rows * a->Hq : 0;
  L->q = off;
  off = align_up(off + heads * 2 * D, 256);
  L->qs = off;
  off = align_up(off + heads * sizeof(float), 256);
  L->total = off;
  return true;
}

ssv_status fp8_check(const ssv_attn_fp8_args* a) {
  if (!a) return SSV_ERR_INVALID;
  if (a->batch < 0 || a->total_rows < 0 || a->total_slots < 0 || a->table_len < 0 || a->n_pages < 0)
    return SSV_ERR_INVALID;
  if (a->Hq <= 0 || a->Hkv <= 0 || a->Hq % a->Hkv != 0 || !page_size_ok(a->page_size)) return SSV_ERR_INVALID;
  if (a->d != 128 || a->Hq / a->Hkv > 128) return SSV_ERR_UNSUPPORTED;
  if (a->max_block < 1 || a->max_block > 64 || a->max_cache < 0 || a->max_new < 0) return SSV_ERR_INVALID;
  if (!isfinite(a->scale) || a->scale < 0.f) return SSV_ERR_INVALID;
  if ((long long)a->n_pages * a->page_size > 0x7fffffffLL / a->Hkv) return SSV_ERR_INVALID;
  const int64_t width = (int64_t)a->Hkv * a->d;
  if ((a->k_stride && a->k_stride < width) || (a->v_stride && a->v_stride < width) || ((a->k_stride | a->v_stride) & 7))
    return SSV_ERR_INVALID;
  if (a->batch == 0 || a->total_rows == 0) return SSV_OK;
  if (!a->q || !a->k_new || !a->v_new || !a->o || !a->seqs || !a->tau) return SSV_ERR_INVALID;
  if (a->n_pages > 0 && (!a->k_cache || !a->v_cache || !a->k_scale || !a->v_scale)) return SSV_ERR_INVALID;
  if (a->table_len > 0 && !a->pages) return SSV_ERR_INVALID;
  const uintptr_t al = (uintptr_t)a->q | (uintptr_t)a->k_cache | (uintptr_t)a->v_cache | (uintptr_t)a->k_new |
                       (uintptr_t)a->v_new | (uintptr_t)a->o;
  return (al & 15u) ? SSV_ERR_INVALID : SSV_OK;
}

template <int MT>
cudaError_t launch_fp8(const AttnFp8Params& p, const Fp8Maps& maps, const Fp8Work& w, int G, int grid, cudaStream_t st) {
  // a merge waits (bounded) on other CTAs' partials: all must be resident at once, one per SM (asked once per device)
  static std::atomic<unsigned long long> ready{0};
  int dev = 0, per_sm = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !(ready.load() >> dev & 1)) {
    e = cudaFuncSetAttribute(attn_fp8_kernel<MT>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kMaxSmem);
    if (e == cudaSuccess)
      e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, attn_fp8_kernel<MT>, kThreads, kMaxSmem);
    if (e == cudaSuccess && per_sm < 1) e = cudaErrorCooperativeLaunchTooLarge;
    if (e != cudaSuccess) return e;
    if (dev < 64) ready |= 1ull << dev;
  }
  const size_t tables = sizeof(int32_t) * 4 * (size_t)(p.batch + 1);
  const int in_smem = Cfg<MT>::SM_TOTAL + tables <= kMaxSmem ? 1 : 0;
  const size_t smem = Cfg<MT>::SM_TOTAL + (in_smem ? tables : 0);
  return launch_pdl(attn_fp8_kernel<MT>, dim3(grid), dim3(kThreads), smem, st, maps, p, w, G, in_smem);
}

}  // namespace
}  // namespace ssv

extern "C" ssv_status ssv_verify_attn_fp8_workspace(const ssv_attn_fp8_args* a, size_t* bytes) {
  using namespace ssv;
  if (!bytes) return SSV_ERR_INVALID;
  const ssv_status st = fp8_check(a);
  if (st != SSV_OK) return st;
  Fp8Layout L;
  if (!fp8_layout(a, &L)) return SSV_ERR_UNSUPPORTED;
  *bytes = (a->batch == 0 || a->total_rows == 0) ? 0 : L.total;
  return SSV_OK;
}

extern "C" ssv_status ssv_verify_attn_fp8(const ssv_attn_fp8_args* a, void* ws, size_t ws_bytes, void* stream) {
  using namespace ssv;
  const ssv_status st = fp8_check(a);
  if (st != SSV_OK) return st;
  Fp8Layout L;
  if (!fp8_layout(a, &L)) return SSV_ERR_UNSUPPORTED;
  if (a->batch == 0 || a->total_rows == 0) return SSV_OK;
  if (!ws || ((uintptr_t)ws & 255u) || ws_bytes < L.total) return SSV_ERR_WORKSPACE;
  const int64_t width = (int64_t)a->Hkv * a->d;
  // other CTAs still read the rows while the first ones write o
  auto meets_o = [&](const void* x, int64_t stride, int64_t cols) {
    const uintptr_t o = (uintptr_t)a->o, y = (uintptr_t)x;
    return o < y + 2 * ((a->total_rows - 1) * stride + cols) && y < o + 2 * (int64_t)a->total_rows * a->Hq * D;
  };
  if (meets_o(a->q, (int64_t)a->Hq * D, (int64_t)a->Hq * D) || meets_o(a->k_new, a->k_stride ? a->k_stride : width, width) ||
      meets_o(a->v_new, a->v_stride ? a->v_stride : width, width))
    return SSV_ERR_INVALID;
  const FaultSetting f = fault_for(SSV_FAULT_ATTN);
  char* w = static_cast<char*>(ws);
  const int G = a->Hq / a->Hkv, max_cache = a->n_pages > 0 ? a->max_cache : 0;
  AttnFp8Params p{reinterpret_cast<const float*>(w + L.qs), a->k_scale, a->v_scale, a->pages,
                  static_cast<__nv_bfloat16*>(a->o), a->Hq, a->Hkv, ilog2(a->page_size), a->n_pages, a->table_len,
                  a->scale > 0.f ? a->scale : (float)(1.0 / sqrt((double)a->d)), a->seqs, a->batch, a->tau,
                  a->total_rows, a->total_slots, max_cache, a->max_new, a->max_block, a->dev_status, f.budget, f.skip,
                  max_cache > 0 ? 1 : 0, L.ordered};
  Fp8Maps maps;
  if (!fp8_encode_fn()) return SSV_ERR_CUDA;
  if (!encode_rows(&maps.kn, a->k_new, 2, a->Hkv, a->total_rows, a->k_stride ? a->k_stride : width, 1, BN) ||
      !encode_rows(&maps.vn, a->v_new, 2, a->Hkv, a->total_rows, a->v_stride ? a->v_stride : width, 1, BN) ||
      !encode_rows(&maps.q, a->q, 2, a->Hq, a->total_rows, (int64_t)a->Hq * D, G, 128 / G))
    return SSV_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (max_cache > 0) {
    const long long rows = (long long)a->n_pages * a->Hkv * a->page_size;
    if (!encode_pages(&maps.kc, a->k_cache, rows, a->page_size, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !encode_pages(&maps.vc, a->v_cache, rows, a->page_size, CU_TENSOR_MAP_SWIZZLE_NONE))
      return SSV_ERR_CUDA;
    const long long heads = (long long)a->total_rows * a->Hq, blocks = (heads * 16 + kSplitThreads - 1) / kSplitThreads;
    char *hi = w + L.q, *lo = hi + heads * D;
    if (!encode_rows(&maps.qhi, hi, 1, a->Hq, a->total_rows, (int64_t)a->Hq * D, G, 128 / G) ||
        !encode_rows(&maps.qlo, lo, 1, a->Hq, a->total_rows, (int64_t)a->Hq * D, G, 128 / G))
      return SSV_ERR_CUDA;
    if (blocks > 0x7fffffffLL) return SSV_ERR_INVALID;
    if (launch_pdl(query_split_kernel, dim3((unsigned)blocks), dim3(kSplitThreads), 0, s,
                   static_cast<const uint4*>(a->q), reinterpret_cast<uint2*>(hi), reinterpret_cast<uint2*>(lo),
                   reinterpret_cast<float*>(w + L.qs), heads) != cudaSuccess)
      return SSV_ERR_CUDA;
  } else {
    maps.kc = maps.qhi = maps.qlo = maps.q;  // never read: no sequence may have cached keys
    maps.vc = maps.vn;
  }
  const Fp8Work work{reinterpret_cast<int32_t*>(w + L.cnt), reinterpret_cast<int32_t*>(w + L.plan),
                     reinterpret_cast<float*>(w + L.ml), reinterpret_cast<float*>(w + L.o)};
  const cudaError_t e = L.mt == 2 ? launch_fp8<2>(p, maps, work, G, L.grid, s) : launch_fp8<1>(p, maps, work, G, L.grid, s);
  return e == cudaSuccess ? SSV_OK : SSV_ERR_CUDA;
}
