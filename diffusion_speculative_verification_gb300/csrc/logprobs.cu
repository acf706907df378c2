// ssv_logprobs: log-probabilities of given tokens, their ranks, the entropy of
// each row and its top alternatives.
//
//   x_v = l_v / T, m = max_v l_v, S = sum_v exp((l_v - m) / T)
//   lse = m / T + ln S,  logprob = (l_t - m) / T - ln S,
//   entropy = ln S - (1 / S) sum_v exp((l_v - m) / T) (l_v - m) / T
//   rank of t: 1 + entries before it by (logit descending, index ascending)
//
// One pass over a row.  Every thread keeps the running maximum of its elements
// and, relative to it, S and W = sum e (l - m) sc in fp32 (sc = log2(e) / T; both
// rescaled when the maximum grows), and counts the elements before the given
// token, two at a time where their batch's maximum does not rule them out.  The
// warps of a cluster send their sums to each other, and every warp that needs them
// joins them in the same order, in 48 bits.  Where one token has nearly all the
// probability, S is 1 and a little, and entropy and log-probability are made of the
// little: a thread keeps the sum of the step that holds its maximum apart from the
// others', and a warp whose sum is nearly 1 forms that step's again without the
// maximum.
//
// Top alternatives.  The K-th largest of any K or more elements bounds the row's
// K-th from below.  Each warp gives the j largest of its lanes' maxima, j so that
// the cluster's warps give about 2 K (where lanes are fewer, the maxima of their
// even and odd elements); with the K-th of these as threshold, batches
// whose maximum (kept in shared memory, rounded up to bf16) passes it are listed,
// read again from L2, one per thread, and their elements that pass it, hardly
// more than K, go to the cluster's first CTA as keys (order of the value above
// the complemented index: equal values in the order of their indices).  It ranks
// them by counting.  Where more pass than its list holds (long runs of equal
// values, and rows masked with a number instead of -inf that leave fewer than K
// tokens, whose threshold is the mask), it finds the K-th key by bisection over the
// row: some fifty readings by one CTA.
//
// Bound by HBM in the long cases, though 9 instructions per element (the
// exponential, the sum for the entropy, two maxima, the rank) are close behind.  The
// short ones are bound by latency, more than half of it behind the pass (stamps of
// an earlier, alike form: of 19200 cycles for one row the pass is 5700, the first
// exchange of the cluster 3400, results and threshold 1900, reading again and
// listing 2000, the second exchange 2100; of 21900 for a short masked row the pass
// is 5600, results and threshold 3700, batches 1400, reading again and listing 4900,
// ranking 1800).  With alternatives a cluster meets three times, without them twice.
// CTAs are small, so that six on an SM keep copies in flight while some rank.
// Measured: 8192 rows of 151936 bf16 without alternatives 371 us, the copy rate
// (registers for seven CTAs per SM 430 us, loads into registers 403 us, 256 threads
// 417 us, each beside 383 .. 391); with tokens at random, whose ranks are long counts,
// 389 us, with 20 alternatives 434, with 128 588; 960 fp32 rows, 30% of them idle,
// with 32 alternatives 73 us, 85% (256 threads 86 us, rows in halves 92 us, beside
// 77); 64 rows with 20 alternatives 13.3 us; one row 9.5 us; 300 rows of 9001 fp32,
// nine tenths masked, with 64 alternatives 12.8 us.
// By bisection, all but 3 of 151936 bf16 tokens masked with the type's lowest number
// and 20 asked for: one row 3.6 ms, 64 rows 3.9 ms, 960 rows 10.7 ms (with -inf 10.8,
// 13.2 and 59.7 us); rows that are all equal 1.4, 1.5 and 4.2 ms.
#include "logits.cuh"

#include <algorithm>
#include <type_traits>
#include <utility>

namespace ssv {
namespace {

constexpr int kStages = 2;                                  // steps in flight
constexpr int kList = 512;                                  // keys that a list holds
constexpr int kThreads = 128;                               // most threads of a CTA
constexpr int kPool = 2 * kLogitsMaxTop + 4 * kMaxCluster + 4;  // values of the pool: 2 K, one of each warp, and a rest
constexpr int kParts = 4 * kMaxCluster;                     // warps of a cluster: one lane each joins them

struct LogprobsParams {
  const void* logits;
  int64_t stride;
  int V, total_rows, K;
  const int32_t* rows;
  const int32_t* tokens;
  Scale T;
  float* logprob;
  int32_t* rank;
  float* entropy;
  float* lse;
  float* top_logprob;
  int32_t* top_token;
  int32_t* dev_status;
  int log_c, log_nt;
  int give;  // maxima that a warp gives to the pool; 32: of all lanes, 64: of all lanes' even and odd elements
};

// bytes of the ring, in which the lists have room
__host__ __device__ constexpr size_t ring_bytes(int threads) {
  const size_t ring = (size_t)kStages * kBatch * 16 * threads + kSlotSlack, lists = (2 * 8 + 4) * kList;
  return ring > lists ? ring : lists;
}

struct Shared {
  uint32_t part[kParts][8];   // of every warp: maximum, S (a pair), W, elements before the token
  int groups, count, total;   // batches and keys listed here, keys sent to the cluster's first CTA
  int at;
  uint32_t least[kThreads / 32];
  int sum[kThreads / 32];
  alignas(16) uint32_t pool[kPool];  // order of the largest lane maxima of every warp of the cluster, 0: none
};

// What the ring's memory holds after the pass.
struct Lists {
  unsigned long long merged[kList], list[kList];
  int group[kList];
};

__device__ __forceinline__ uint32_t order_bits(float x) {
  const uint32_t b = __float_as_uint(x == 0.f ? 0.f : x);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float from_order(uint32_t b) {
  return __uint_as_float((b & 0x80000000u) ? (b & 0x7FFFFFFFu) : ~b);
}
__device__ __forceinline__ unsigned long long element_key(float x, int v) {
  return ((unsigned long long)order_bits(x) << 32) | (0xFFFFFFFFu - (uint32_t)v);
}

// The given token and how elements compare with it: in vectors in front of its own an element is before it when no
// smaller, that is, greater than the next number below; in those behind when greater.
template <typename T>
struct Given {
  int t, own, below;  // own: the token's vector; below: lt's next lower number as bits of T
  float lt;

  __device__ __forceinline__ void set(const RowView<T>& row, int token, bool there) {
    t = token;
    own = (row.lead + token) / kVec<T>;
    lt = there ? load_element(row.row + token) : NAN;  // without a token nothing compares
    uint32_t b = __float_as_uint(lt) >> (sizeof(T) == 2 ? 16 : 0);
    const uint32_t sign = sizeof(T) == 2 ? 0x8000u : 0x80000000u;
    below = (int)((b & ~sign) == 0 ? sign | 1u : (b & sign) ? b + 1 : b - 1);
  }

  // Elements of a step's vectors, i and every NT-th behind it up to `end`, that are before the token; vectors from
  // there on are -inf.
  __device__ __forceinline__ int before(const uint4 (&x)[kBatch], int i, int NT, int end, const RowView<T>& row) const {
    if (lt == -INFINITY || (i <= own && own <= i + NT * (kBatch - 1))) {
      int n = 0;
#pragma unroll
      for (int u = 0; u < kBatch; ++u)
        if (i + NT * u < end) n += among(x[u], row.first(i + NT * u));
      return n;
    }
    if constexpr (sizeof(T) == 2) {
      const uint32_t b = i < own ? (uint32_t)below : __float_as_uint(lt) >> 16, both = b << 16 | b;
      const __nv_bfloat162 than = *reinterpret_cast<const __nv_bfloat162*>(&both);
      __nv_bfloat162 c = __floats2bfloat162_rn(0.f, 0.f);  // counts up to 16 are exact
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const uint32_t w[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) c = __hadd2(c, __hgt2(*reinterpret_cast<const __nv_bfloat162*>(&w[k]), than));
      }
      return (int)(__low2float(c) + __high2float(c));
    } else {
      const float than = i < own ? __uint_as_float((uint32_t)below) : lt;
      int n = 0;
#pragma unroll
      for (int u = 0; u < kBatch; ++u)
        n += (__uint_as_float(x[u].x) > than ? 1 : 0) + (__uint_as_float(x[u].y) > than ? 1 : 0) +
             (__uint_as_float(x[u].z) > than ? 1 : 0) + (__uint_as_float(x[u].w) > than ? 1 : 0);
      return n;
    }
  }

  // The same, element by element, for the token's own vector and for tokens at -inf.
  __device__ __noinline__ int among(const uint4 r, int v0) const {
    int n = 0;
#pragma unroll
    for (int i = 0; i < kVec<T> / 2; ++i) {
      const float2 x = pair_of<T>(r, i);
      const int v = v0 + 2 * i;  // below 0: in front of the row
      n += (x.x > lt || (x.x == lt && v >= 0 && v < t)) ? 1 : 0;
      n += (x.y > lt || (x.y == lt && v + 1 >= 0 && v + 1 < t)) ? 1 : 0;
    }
    return n;
  }
};

// Sum of a step's vectors, i and every NT-th behind it up to `end`, without their maximum m, once.
template <typename T>
__device__ __noinline__ float step_without(const RowView<T>& row, int i, int NT, int end, float m, float sc) {
  uint4 x[kBatch];
#pragma unroll
  for (int u = 0; u < kBatch; ++u) {
    x[u].x = x[u].y = x[u].z = x[u].w = none_bits<T>();
    if (i + NT * u < end) x[u] = row.load(i + NT * u);
  }
  float s = 0.f;
  bool found = false;
#pragma unroll
  for (int u = 0; u < kBatch; ++u) {
#pragma unroll
    for (int e = 0; e < kVec<T>; ++e) {
      const float2 y = pair_of<T>(x[u], e / 2);
      const float z = (e & 1) ? y.y : y.x;
      if (!found && z == m) found = true; else s += ex2((z - m) * sc);
    }
  }
  return s;
}

// Whole CTA: keys of the row that are >= key.
template <typename T>
__device__ int count_keys(const RowView<T>& row, unsigned long long key, Shared& sm) {
  int n = 0;
  for (int i = threadIdx.x; i < row.n; i += blockDim.x) {
    const uint4 r = row.load(i);
    const int v0 = row.first(i);
#pragma unroll
    for (int k = 0; k < kVec<T> / 2; ++k) {
      const float2 x = pair_of<T>(r, k);
      n += (x.x > -INFINITY && element_key(x.x, v0 + 2 * k) >= key) ? 1 : 0;
      n += (x.y > -INFINITY && element_key(x.y, v0 + 2 * k + 1) >= key) ? 1 : 0;
    }
  }
  n = warp_sum(n);
  if ((threadIdx.x & 31) == 0) sm.sum[threadIdx.x >> 5] = n;
  __syncthreads();
  int sum = 0;
  for (int w = 0; w < (int)blockDim.x / 32; ++w) sum += sm.sum[w];
  __syncthreads();
  return sum;
}

// Keys of a vector's elements that are >= `key` and not -inf: to keys[0, kList), counted in `count`.
template <typename T>
__device__ __forceinline__ void list_keys(const uint4& r, int v0, unsigned long long key, unsigned long long* keys,
                                          int* count) {
#pragma unroll
  for (int e = 0; e < kVec<T>; ++e) {
    const float2 y = pair_of<T>(r, e / 2);
    const float z = (e & 1) ? y.y : y.x;
    if (z > -INFINITY && element_key(z, v0 + e) >= key) {
      const int at = atomicAdd(count, 1);
      if (at < kList) keys[at] = element_key(z, v0 + e);
    }
  }
}

// Whole CTA: the row's K greatest keys into `merged` (more than K elements are above -inf).
template <typename T>
__device__ __noinline__ void bisect_top(const RowView<T>& row, int K, float least, float most, Shared& sm,
                                        unsigned long long* merged) {
  // the largest key that at least K keys reach: first the value, then the index
  uint32_t lo = order_bits(least), hi = order_bits(most);
  while (lo < hi) {  // count(lo) >= K throughout
    const uint32_t mid = lo + (hi - lo + 1) / 2;
    if (count_keys<T>(row, (unsigned long long)mid << 32, sm) >= K) lo = mid; else hi = mid - 1;
  }
  uint32_t ilo = 0xFFFFFFFFu - (uint32_t)row.V, ihi = 0xFFFFFFFFu;
  while (ilo < ihi) {
    const uint32_t mid = ilo + (ihi - ilo + 1) / 2;
    if (count_keys<T>(row, ((unsigned long long)lo << 32) | mid, sm) >= K) ilo = mid; else ihi = mid - 1;
  }
  const unsigned long long key = ((unsigned long long)lo << 32) | ilo;
  if (threadIdx.x == 0) sm.count = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < row.n; i += blockDim.x) list_keys<T>(row.load(i), row.first(i), key, merged, &sm.count);
  __syncthreads();
}

// LOG_NT: 2^LOG_NT threads in a CTA, so that a step's addresses are constants apart (when it was taken: 8192 rows 379 us,
// known at the launch alone 391); 0: as many as the launch says, for short rows.
template <typename T, bool TOP, int LOG_NT>
__global__ void __launch_bounds__(kThreads, 6) logprobs_kernel(const LogprobsParams p) {
  extern __shared__ __align__(128) unsigned char dynamic[];  // the ring, then the lists; behind them each batch's maximum
  __shared__ Shared sm;
  const int log_nt = LOG_NT ? LOG_NT : p.log_nt;
  const int tid = threadIdx.x, NT = 1 << log_nt, lane = tid & 31, warp = tid >> 5, nw = NT >> 5;
  const int c = 1 << p.log_c;
  const int rank = (int)blockIdx.x & (c - 1), entry = (int)blockIdx.x >> p.log_c;
  Lists& lists = *reinterpret_cast<Lists*>(dynamic);
  __nv_bfloat16* tops = reinterpret_cast<__nv_bfloat16*>(dynamic + ring_bytes(NT));
  if (TOP && tid < 4) sm.pool[(nw * p.give << p.log_c & ~3) + tid] = 0u;  // behind the last; the pool may write over it
  if (tid == 0) {
    sm.groups = 0;
    sm.count = 0;
    sm.total = 0;
  }
  __syncthreads();
  if (c > 1) cluster_arrive();  // waited for before the first access to another CTA's shared memory
  pdl_wait();                   // tokens, rows and logits may come from the kernels before this one
  pdl_trigger();

  // the entry's row and token
  const int r = p.rows ? p.rows[entry] : entry;
  const int t = p.tokens ? p.tokens[entry] : 0;
  const bool bad = r < -1 || r >= p.total_rows || t < -1 || t >= p.V;
  const bool idle = bad || r == -1 || t == -1;
  if (idle) {
    if (rank == 0) {
      if (tid == 0) {
        if (bad) report(p.dev_status, SSV_ERR_INVALID);
        if (p.logprob) p.logprob[entry] = 0.f;
        if (p.rank) p.rank[entry] = 0;
        if (p.entropy) p.entropy[entry] = 0.f;
        if (p.lse) p.lse[entry] = 0.f;
      }
      for (int k = tid; k < p.K; k += NT) {
        p.top_logprob[(size_t)entry * p.K + k] = -INFINITY;
        p.top_token[(size_t)entry * p.K + k] = -1;
      }
    }
    if (c > 1) cluster_wait();
    return;
  }
  const RowView<T> row(static_cast<const T*>(p.logits) + (int64_t)r * p.stride, p.V);
  const PartView<T> part(row, rank, p.log_c, log_nt);
  const int i0 = part.i0, i1 = part.i1, steps = part.steps;
  uint4* ring = part.slots_in(dynamic, row);
  auto slots = [&](int k) { return ring + kBatch * (k % kStages) * NT + tid; };
  for (int k = 0; k < kStages; ++k) part.fetch(row, k, slots(k));
  Given<T> given;
  given.set(row, t, p.tokens != nullptr);
  const float lt = given.lt;

  // ------------------------------------------------------------ the pass
  float m = -INFINITY, S_top = 0.f, S = 0.f, W = 0.f;  // S_top: of step k_top, which holds the maximum; S: of the others
  int k_top = 0;
  float even = -INFINITY, odd = -INFINITY;  // m by elements
  int before = 0;
  const float2 sc2 = make_float2(p.T.sc, p.T.sc);
  auto step = [&](auto is_full, int k) {
    constexpr bool FULL = decltype(is_full)::value;
    uint4 x[kBatch];
    part.template take<FULL>(k, slots(k), x);
    const float2 mx2 = step_max<T>(x);
    const float mx = fmaxf(mx2.x, mx2.y);
    if (TOP) {
      even = fmaxf(even, mx2.x);
      odd = fmaxf(odd, mx2.y);
    }
    part.fetch(row, k + kStages, slots(k));  // into the slots that have just been read
    if (TOP) tops[k * NT + tid] = __float2bfloat16_ru(mx);
    const int ib = i0 + tid + NT * kBatch * k;
    if (mx >= lt) before += given.before(x, ib, NT, i1, row);
    if (mx > m) {  // sums so far on the new scale
      const float d = shift_of(m, mx, p.T.sc), f = ex2(d);
      S += S_top;
      W = f * (W + d * S);
      S = f * S;
      m = mx;
      k_top = k;
    }
    // Nothing but -inf and NaN so far: relative to 0, so that -inf counts nothing and NaN stays.
    const float mm = m == -INFINITY ? 0.f : m;
    const float2 nm = make_float2(-mm, -mm);
    float2 S2 = make_float2(0.f, 0.f), W2 = make_float2(0.f, 0.f);
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      if (!FULL && ib + NT * u >= i1) break;
#pragma unroll
      for (int i = 0; i < kVec<T> / 2; ++i) {
        float2 y = mul2(add2(pair_of<T>(x[u], i), nm), sc2);
        y.x = max_nan(y.x, -200.f);  // 2^-200 is 0 and 0 * -200 too; -inf would make it NaN
        y.y = max_nan(y.y, -200.f);
        const float2 e = make_float2(ex2(y.x), ex2(y.y));
        S2 = add2(S2, e);
        W2 = fma2(e, y, W2);
      }
    }
    if (k == k_top) S_top = S2.x + S2.y; else S += S2.x + S2.y;
    W += W2.x + W2.y;
  };
  for (int k = 0; k < steps; ++k) {
    copy_wait<kStages - 1>();
    if (part.full(k)) step(std::true_type{}, k); else step(std::false_type{}, k);
  }
  copy_wait<0>();

  // ------------------------------------------------------------ every warp's part, to every CTA that joins them
  {
    const float M = warp_max(m);
    const float d = shift_of(m, M, p.T.sc), f = ex2(d);
    const float Ww = warp_sum(f * (W + d * (S + S_top)));
    Pair Sw = warp_sum(Pair{f * S_top, f * S});
    if (M > -INFINITY && value_of(Sw) < 1.f + 0x1p-7f) {  // 1 for the maximum, and the rest again
      Pair rest = {f * S_top, f * S};
      if (lane == __ffs(__ballot_sync(0xffffffffu, m == M)) - 1)
        rest = Pair{S, step_without<T>(row, i0 + tid + NT * kBatch * k_top, NT, i1, M, p.T.sc)};
      Sw = Pair{1.f, value_of(warp_sum(rest))};
    }
    const int nb = warp_sum(before);
    const int me = rank * nw + warp;
    if (c > 1) cluster_wait();
    for (int i = lane; i < 8 * (TOP ? c : 1); i += 32) {  // without alternatives the first CTA joins them alone
      const int w = i & 7;
      if (w > 4) continue;
      const uint32_t word = __float_as_uint(w == 0 ? M : w == 1 ? Sw.hi : w == 2 ? Sw.lo : Ww);
      if (c == 1)
        sm.part[me][w] = w == 4 ? (uint32_t)nb : word;
      else
        cluster_store(cluster_addr(&sm.part[me][w], i >> 3), w == 4 ? (uint32_t)nb : word);
    }
    if (TOP) {
      auto give = [&](int i, uint32_t v) {  // by every lane
        uint32_t* to = &sm.pool[me * p.give + i];
        if (c == 1) {
          if (lane == 0) *to = v;
        } else if (lane < c) {
          cluster_store(cluster_addr(to, lane), v);
        }
      };
      uint32_t b = order_bits(m);
      if (p.give < 32) {  // the largest
        for (int i = 0; i < p.give; ++i) {
          const uint32_t most = __reduce_max_sync(0xffffffffu, b);
          if (lane == __ffs(__ballot_sync(0xffffffffu, b == most)) - 1) b = 0u;
          give(i, most);
        }
      } else {
        const uint32_t e = order_bits(even), o = order_bits(odd);
        if (c == 1) {
          sm.pool[me * p.give + lane] = p.give == 32 ? b : e;
          if (p.give == 64) sm.pool[me * p.give + 32 + lane] = o;
        }
        for (int i = 0; c > 1 && i < p.give; ++i) give(i, __shfl_sync(0xffffffffu, p.give == 32 ? b : i < 32 ? e : o, i & 31));
      }
    }
  }
  if (c > 1) {
    cluster_arrive();
    if (!TOP && rank != 0) return;
    cluster_wait();
  } else {
    __syncthreads();
  }
  float Mr, St, Wt;
  Pair S_row;
  int nb;
  {
    const bool there = lane < c * nw;
    const float ml = there ? __uint_as_float(sm.part[lane][0]) : -INFINITY;
    Mr = warp_max(ml);
    Pair s = {0.f, 0.f};
    float w = 0.f;
    nb = 0;
    if (there) {
      const float d = shift_of(ml, Mr, p.T.sc), f = ex2(d);
      const Pair Sl = {__uint_as_float(sm.part[lane][1]), __uint_as_float(sm.part[lane][2])};
      s = Pair{f * Sl.hi, f * Sl.lo};
      w = f * (__uint_as_float(sm.part[lane][3]) + d * value_of(Sl));
      nb = (int)sm.part[lane][4];
    }
    S_row = warp_sum(s);
    St = value_of(S_row);
    Wt = warp_sum(w);
    nb = warp_sum(nb);
  }

  // ------------------------------------------------------------ results (the cluster's first CTA)
  const bool empty = Mr == -INFINITY && St == 0.f;  // nothing above -inf
  const Pair lnS = log_sum(S_row);
  if (rank == 0 && tid == NT - 1) {
    const Pair inv = {p.T.hi, p.T.lo};
    if (p.lse) p.lse[entry] = empty ? -INFINITY : value_of(Pair{Mr, 0.f} * inv + lnS);
    if (p.entropy) p.entropy[entry] = empty ? 0.f : value_of(lnS + Pair{-(Wt / St) * kLn2, 0.f});
    if (p.logprob) p.logprob[entry] = empty ? -INFINITY : value_of(two_sum(lt, -Mr) * inv + -lnS);
    if (p.rank) p.rank[entry] = lt == lt ? nb + 1 : 0;
  }

  // ------------------------------------------------------------ alternatives
  if (TOP) {
    // the K-th of the pool: the least value that fewer than K exceed
    const int pooled = c * nw * p.give;
    uint32_t mine_least = 0xFFFFFFFFu;
    for (int i = tid; i < pooled; i += NT) {
      const uint32_t v = sm.pool[i];
      int above = 0;
      for (int j = 0; j < pooled; j += 4) {  // a multiple of four, or 0 behind the last
        const uint4 o = *reinterpret_cast<const uint4*>(&sm.pool[j]);
        above += (o.x > v ? 1 : 0) + (o.y > v ? 1 : 0) + (o.z > v ? 1 : 0) + (o.w > v ? 1 : 0);
      }
      if (above < p.K) mine_least = min(mine_least, v);
    }
    mine_least = __reduce_min_sync(0xffffffffu, mine_least);
    if (lane == 0) sm.least[warp] = mine_least;
    __syncthreads();
    for (int w = 0; w < nw; ++w) mine_least = min(mine_least, sm.least[w]);
    // fewer values than K bound nothing (0: a lane without elements)
    const float least = pooled < p.K || mine_least == 0u ? -INFINITY : from_order(mine_least);
    // batches that reach it
    if (m >= least && m > -INFINITY)
      for (int k = 0; k < steps; ++k) {
        const float top = __bfloat162float(tops[k * NT + tid]);
        if (top >= least && top > -INFINITY) {
          const int at = atomicAdd(&sm.groups, 1);
          if (at < kList) lists.group[at] = k * NT + tid;
        }
      }
    __syncthreads();
    // their elements that do
    const int ng = sm.groups;
    const unsigned long long key = (unsigned long long)order_bits(least) << 32;
    if (ng <= kList) {
      for (int q = tid; q < ng * kBatch; q += NT) {
        const int b = lists.group[q / kBatch];
        const int i = i0 + (b & (NT - 1)) + NT * (kBatch * (b >> log_nt) + q % kBatch);
        if (i < i1) list_keys<T>(row.load(i), row.first(i), key, lists.list, &sm.count);
      }
    } else if (tid == 0) {
      sm.count = kList + 1;  // hardly fewer: every batch has one but for the rounding of its maximum
    }
    __syncthreads();
    const int mine = sm.count;
    if (c > 1) {
      if (tid == 0) sm.at = cluster_add(cluster_addr(&sm.total, 0), mine);
      __syncthreads();
      const int at = sm.at;
      if (at + mine <= kList)
        for (int i = tid; i < mine; i += NT) cluster_store64(cluster_addr(&lists.merged[at + i], 0), lists.list[i]);
      cluster_arrive();
      if (rank != 0) return;
      cluster_wait();
    } else {
      for (int i = tid; i < min(mine, kList); i += NT) lists.merged[i] = lists.list[i];
      if (tid == 0) sm.total = mine;
      __syncthreads();
    }
    int n = sm.total;
    if (n > kList) {
      bisect_top<T>(row, p.K, least, Mr, sm, lists.merged);
      n = sm.count;
    }
    const float ln = value_of(lnS);
    float* lp = p.top_logprob + (size_t)entry * p.K;
    int32_t* tk = p.top_token + (size_t)entry * p.K;
    for (int i = tid; i < n; i += NT) {
      const unsigned long long mine_key = lists.merged[i];
      int place = 0;
#pragma unroll 8
      for (int j = 0; j < n; ++j) place += lists.merged[j] > mine_key ? 1 : 0;
      if (place < p.K) {
        const float x = from_order((uint32_t)(mine_key >> 32));
        lp[place] = (x - Mr) * p.T.hi - ln;
        tk[place] = (int32_t)(0xFFFFFFFFu - (uint32_t)mine_key);
      }
    }
    for (int i = n + tid; i < p.K; i += NT) {
      lp[i] = -INFINITY;
      tk[i] = -1;
    }
  }
}

template <typename T, bool TOP, int LOG_NT>
cudaError_t logprobs_launch_as(const LogprobsParams& p, int n, const RowSplit& sp, cudaStream_t st) {
  static uint64_t done = 0;
  const size_t smem = ring_bytes(sp.threads) + (TOP ? (size_t)sp.batches() * sp.threads * sizeof(__nv_bfloat16) : 0);
  const cudaError_t e = allow_shared(logprobs_kernel<T, TOP, LOG_NT>, smem, &done);
  return e != cudaSuccess ? e : launch_rows(logprobs_kernel<T, TOP, LOG_NT>, n, sp, sp.threads, smem, st, p);
}

template <typename T, bool TOP>
cudaError_t logprobs_launch(const LogprobsParams& p, int n, const RowSplit& sp, cudaStream_t st) {
  return TOP || sp.log_nt == 7 ? logprobs_launch_as<T, TOP, 7>(p, n, sp, st) : logprobs_launch_as<T, TOP, 0>(p, n, sp, st);
}

// CTAs per row: more of them while they stay below three per SM (of the 152 that the part has) and a CTA has more than two
// steps (64 rows of 151936 bf16, four CTAs each: 13.4 us; two 17.2 us; eight 15.2 us.  300 rows of 9001 fp32, one each:
// 12.9 us when measured beside two, 14.2 us).
RowSplit logprobs_split(int rows, int V, int element_size, int top_k) {
  // alternatives are ranked by every thread: none of them less for a short row
  const int vectors = std::max(row_vectors(V, element_size), top_k > 0 ? kThreads : 1);
  int c = 1;
  while (c < kMaxCluster && (long long)rows * c * 2 <= 456 && vectors > 2 * c * kThreads * kBatch) c *= 2;
  return split_of(vectors, c, kThreads);
}

}  // namespace
}  // namespace ssv

extern "C" ssv_status ssv_logprobs(const ssv_logprobs_args* a, void* stream) {
  using namespace ssv;
  if (!a) return SSV_ERR_INVALID;
  if (!logits_shape_ok(a->logits, a->logits_stride, a->dtype, a->V, a->total_rows) || a->n < 0 || a->top_k < 0)
    return SSV_ERR_INVALID;
  LogprobsParams p;
  if (!logits_scale(a->T, &p.T)) return SSV_ERR_NOT_FINITE;
  if (a->V > kLogitsMaxVocab || a->top_k > kLogitsMaxTop) return SSV_ERR_UNSUPPORTED;
  if (!a->rows && a->n > a->total_rows) return SSV_ERR_INVALID;
  if (a->n == 0) return SSV_OK;
  if ((!a->logits && a->total_rows > 0) || (a->tokens ? !a->logprob : (a->logprob || a->rank)) ||
      (a->top_k > 0 && (!a->top_logprob || !a->top_token)))
    return SSV_ERR_INVALID;
  if (!a->logprob && !a->entropy && !a->lse && a->top_k == 0) return SSV_ERR_INVALID;
  if (((uintptr_t)a->rows | (uintptr_t)a->tokens | (uintptr_t)a->logprob | (uintptr_t)a->rank | (uintptr_t)a->entropy |
       (uintptr_t)a->lse | (uintptr_t)a->top_logprob | (uintptr_t)a->top_token | (uintptr_t)a->dev_status) & 3u)
    return SSV_ERR_INVALID;
  p.logits = a->logits;
  p.stride = a->logits_stride ? a->logits_stride : a->V;
  const size_t n4 = 4 * (size_t)a->n, k4 = n4 * a->top_k;
  const int es = a->dtype == SSV_BF16 ? 2 : 4;
  for (const auto& o : {std::make_pair((const void*)a->logprob, n4), std::make_pair((const void*)a->rank, n4),
                        std::make_pair((const void*)a->entropy, n4), std::make_pair((const void*)a->lse, n4),
                        std::make_pair((const void*)a->top_logprob, k4), std::make_pair((const void*)a->top_token, k4)})
    if (meets_rows(o.first, o.second, a->logits, p.stride, a->V, a->total_rows, es)) return SSV_ERR_INVALID;
  p.V = a->V;
  p.total_rows = a->total_rows;
  p.K = a->top_k;
  p.rows = a->rows;
  p.tokens = a->tokens;
  p.logprob = a->logprob;
  p.rank = a->rank;
  p.entropy = a->entropy;
  p.lse = a->lse;
  p.top_logprob = a->top_logprob;
  p.top_token = a->top_token;
  p.dev_status = a->dev_status;
  const RowSplit sp = logprobs_split(a->n, a->V, es, a->top_k);
  p.log_c = sp.log_c;
  p.log_nt = sp.log_nt;
  const int warps = sp.ctas * (sp.threads / 32);
  p.give = (2 * a->top_k + warps - 1) / warps;
  // fewer lanes with elements than that: even and odd elements apart (four warps at most, so that the pool holds them)
  if (p.give > 32 || (warps <= 4 && row_vectors(a->V, es) < 2 * a->top_k)) p.give = 64;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  using bf16 = __nv_bfloat16;
  cudaError_t e;
  if (a->top_k > 0)
    e = a->dtype == SSV_BF16 ? logprobs_launch<bf16, true>(p, a->n, sp, st) : logprobs_launch<float, true>(p, a->n, sp, st);
  else
    e = a->dtype == SSV_BF16 ? logprobs_launch<bf16, false>(p, a->n, sp, st) : logprobs_launch<float, false>(p, a->n, sp, st);
  return e == cudaSuccess ? SSV_OK : SSV_ERR_CUDA;
}
