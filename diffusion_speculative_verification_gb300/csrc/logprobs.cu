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
// token, which its group's maximum lets it skip mostly.
//
// Top alternatives.  The K-th largest of any K or more elements bounds the row's
// K-th from below.  Each warp gives the j largest of its lanes' maxima, j so that
// the cluster's warps give about 2 K; with the K-th of these as threshold, groups
// whose maximum (kept in shared memory, one word per 32 bytes of the row) passes
// it are listed, read again from L2, one per thread, and their elements that pass
// it, hardly more than K, go to the cluster's first CTA as keys (order of the value above the complemented
// index: equal values in the order of their indices).  It ranks them by counting.
// Where more pass than its list holds (long runs of equal values), it finds the
// K-th key by bisection over the row.
#include "logits.cuh"

#include <algorithm>

namespace ssv {
namespace {

constexpr int kList = 512;        // keys that a list holds
constexpr int kMaxCluster = 8;
constexpr int kPool = 2 * kLogitsMaxTop + 8 * kMaxCluster;  // values of the pool at most: 2 K, and one of each warp

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
  int ctas;
  int give;  // lane maxima that a warp gives to the pool
};

struct Part {  // what a CTA knows of its part of the row
  float m, S, W;
  int before;
};
constexpr int kPartWords = sizeof(Part) / 4;

struct Shared {
  Part part[kMaxCluster];
  float red[kLogitsThreads / 32];
  float redS[kLogitsThreads / 32], redW[kLogitsThreads / 32];
  int redN[kLogitsThreads / 32];
  int groups, count, total;  // groups and keys listed here, keys sent to the cluster's first CTA
  int at;
  float least;
  alignas(16) uint32_t pool[kPool];  // order of the largest lane maxima of every warp of the cluster, 0: none
  int group[kList];
  unsigned long long merged[kList];
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

// The given token and how elements compare with it: of groups in front of its own an element is before it when no
// smaller, that is, greater than the next number below; of those behind when greater.
template <typename T>
struct Given {
  int t, group, below;  // below: lt's next lower number as bits of T
  float lt;

  __device__ __forceinline__ void set(const RowView<T>& row, int token, bool there) {
    t = token;
    group = (row.lead + token) / kGroup<T>;
    lt = there ? load_element(row.row + token) : NAN;  // without a token nothing compares
    uint32_t b = __float_as_uint(lt) >> (sizeof(T) == 2 ? 16 : 0);
    const uint32_t sign = sizeof(T) == 2 ? 0x8000u : 0x80000000u;
    below = (int)((b & ~sign) == 0 ? sign | 1u : (b & sign) ? b + 1 : b - 1);
  }

  // Elements of group g that are before the token.  lt is above -inf.
  __device__ __forceinline__ int before(const Raw& r, int g, const RowView<T>& row) const {
    if (g == group) return among(r, row.first(g));
    int n = 0;
    if (sizeof(T) == 2) {
      const uint32_t b = g < group ? (uint32_t)below : __float_as_uint(lt) >> 16, both = b << 16 | b;
      const __nv_bfloat162 than = *reinterpret_cast<const __nv_bfloat162*>(&both);
      __nv_bfloat162 c = __floats2bfloat162_rn(0.f, 0.f);
#pragma unroll
      for (int i = 0; i < 8; ++i) c = __hadd2(c, __hgt2(*reinterpret_cast<const __nv_bfloat162*>(&r.w[i]), than));
      n = (int)(__low2float(c) + __high2float(c));
    } else {
      const float than = g < group ? __uint_as_float((uint32_t)below) : lt;
#pragma unroll
      for (int i = 0; i < 8; ++i) n += __uint_as_float(r.w[i]) > than ? 1 : 0;
    }
    return n;
  }

  // The same, element by element, for the token's own group and for tokens at -inf.
  __device__ __noinline__ int among(const Raw r, int v0) const {
    int n = 0;
#pragma unroll
    for (int i = 0; i < kGroup<T> / 2; ++i) {
      const float2 x = pair_of<T>(r, i);
      const int v = v0 + 2 * i;  // below 0: in front of the row
      n += (x.x > lt || (x.x == lt && v >= 0 && v < t)) ? 1 : 0;
      n += (x.y > lt || (x.y == lt && v + 1 >= 0 && v + 1 < t)) ? 1 : 0;
    }
    return n;
  }
};

// Whole CTA: keys of the row that are >= key.
template <typename T>
__device__ int count_keys(const RowView<T>& row, unsigned long long key, Shared& sm) {
  int n = 0;
  for (int g = threadIdx.x; g < row.n; g += blockDim.x) {
    const Raw r = row.load(g);
    const int v0 = row.first(g);
#pragma unroll
    for (int i = 0; i < kGroup<T> / 2; ++i) {
      const float2 x = pair_of<T>(r, i);
      n += (x.x > -INFINITY && element_key(x.x, v0 + 2 * i) >= key) ? 1 : 0;
      n += (x.y > -INFINITY && element_key(x.y, v0 + 2 * i + 1) >= key) ? 1 : 0;
    }
  }
  n = warp_sum(n);
  if ((threadIdx.x & 31) == 0) sm.redN[threadIdx.x >> 5] = n;
  __syncthreads();
  int sum = 0;
  for (int w = 0; w < (int)blockDim.x / 32; ++w) sum += sm.redN[w];
  __syncthreads();
  return sum;
}

// Whole CTA: the row's K greatest keys into sm.merged (more than K elements are above -inf).
template <typename T>
__device__ __noinline__ void bisect_top(const RowView<T>& row, int K, float least, float most, Shared& sm) {
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
  for (int g = threadIdx.x; g < row.n; g += blockDim.x) {
    const Raw r = row.load(g);
    const int v0 = row.first(g);
    for (int e = 0; e < kGroup<T>; ++e) {
      float2 x = make_float2(0.f, 0.f);
#pragma unroll
      for (int i = 0; i < kGroup<T> / 2; ++i)
        if (i == e / 2) x = pair_of<T>(r, i);
      const float y = (e & 1) ? x.y : x.x;
      if (y > -INFINITY && element_key(y, v0 + e) >= key) {
        const int at = atomicAdd(&sm.count, 1);
        if (at < kList) sm.merged[at] = element_key(y, v0 + e);
      }
    }
  }
  __syncthreads();
}

template <typename T, bool TOP>
__global__ void __launch_bounds__(kLogitsThreads, 4) logprobs_kernel(const LogprobsParams p) {
  // TOP: largest number of every group of this CTA; then the keys listed here
  extern __shared__ __align__(16) unsigned char dynamic[];
  float* group_top = reinterpret_cast<float*>(dynamic);
  unsigned long long* list = reinterpret_cast<unsigned long long*>(dynamic);
  __shared__ Shared sm;
  const int tid = threadIdx.x, NT = blockDim.x, lane = tid & 31, warp = tid >> 5, nw = NT >> 5;
  const int c = p.ctas;
  const int rank = (int)blockIdx.x % c, entry = (int)blockIdx.x / c;
  if (tid == 0) {
    sm.groups = 0;
    sm.count = 0;
    sm.total = 0;
    sm.least = -INFINITY;
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
  const int g0 = (int)((long long)row.n * rank / c), g1 = (int)((long long)row.n * (rank + 1) / c);
  Given<T> given;
  given.set(row, t, p.tokens != nullptr);
  const float lt = given.lt;

  // ------------------------------------------------------------ the pass
  float m = -INFINITY, S = 0.f, W = 0.f;
  int before = 0;
  const float2 sc2 = make_float2(p.T.sc, p.T.sc);
  for (int gb = g0 + tid; gb < g1; gb += NT * kBatch) {
    Raw x[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int g = gb + u * NT;
      if (g < g1) x[u] = row.load(g); else set_none<T>(x[u]);
    }
    float top[kBatch], mx = -INFINITY;
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      top[u] = group_max<T>(x[u]);
      mx = fmaxf(mx, top[u]);
      const int g = gb + u * NT;
      if (TOP && g < g1) group_top[g - g0] = top[u];
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u)
      if (top[u] >= lt && gb + u * NT < g1)
        before += lt == -INFINITY ? given.among(x[u], row.first(gb + u * NT)) : given.before(x[u], gb + u * NT, row);
    if (mx > m) {  // sums so far on the new scale
      const float d = shift_of(m, mx, p.T.sc), f = ex2(d);
      W = f * (W + d * S);
      S = f * S;
      m = mx;
    }
    // A group of nothing but -inf and NaN: relative to 0, so that -inf counts nothing and NaN stays.
    const float mm = m == -INFINITY ? 0.f : m;
    const float2 nm = make_float2(-mm, -mm);
    float2 S2 = make_float2(0.f, 0.f), W2 = make_float2(0.f, 0.f);
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      if (u && gb + u * NT >= g1) break;
#pragma unroll
      for (int i = 0; i < kGroup<T> / 2; ++i) {
        float2 y = mul2(add2(pair_of<T>(x[u], i), nm), sc2);
        y.x = max_nan(y.x, -200.f);  // 2^-200 is 0 and 0 * -200 too; -inf would make it NaN
        y.y = max_nan(y.y, -200.f);
        const float2 e = make_float2(ex2(y.x), ex2(y.y));
        S2 = add2(S2, e);
        W2 = fma2(e, y, W2);
      }
    }
    S += S2.x + S2.y;
    W += W2.x + W2.y;
  }

  // ------------------------------------------------------------ this CTA's part
  const int given_n = nw * p.give;  // values that a CTA gives to the pool
  if (TOP) {
    uint32_t* mine = sm.pool + rank * given_n + warp * p.give;
    uint32_t b = order_bits(m);
    if (p.give == 32) {
      mine[lane] = b;
    } else {
      for (int i = 0; i < p.give; ++i) {
        const uint32_t most = __reduce_max_sync(0xffffffffu, b);
        const int who = __ffs(__ballot_sync(0xffffffffu, b == most)) - 1;
        if (lane == who) {
          mine[i] = b;
          b = 0u;
        }
      }
    }
  }
  const float M = cta_max(m, sm.red);
  {
    const float d = shift_of(m, M, p.T.sc), f = ex2(d);
    const float Sw = warp_sum(f * S), Ww = warp_sum(f * (W + d * S));
    const int nb = warp_sum(before);
    if (lane == 0) {
      sm.redS[warp] = Sw;
      sm.redW[warp] = Ww;
      sm.redN[warp] = nb;
    }
  }
  __syncthreads();
  if (tid == 0) {
    Part& me = sm.part[rank];
    me.m = M;
    me.S = me.W = 0.f;
    me.before = 0;
    for (int w = 0; w < nw; ++w) {
      me.S += sm.redS[w];
      me.W += sm.redW[w];
      me.before += sm.redN[w];
    }
  }
  __syncthreads();
  if (c > 1) {
    // every CTA of the cluster (the first alone, without alternatives) gets every part
    cluster_wait();
    const uint32_t* mine = reinterpret_cast<const uint32_t*>(&sm.part[rank]);
    const int to = TOP ? c : 1;
    for (int i = tid; i < to * kPartWords; i += NT) {
      const int dst = i / kPartWords, w = i % kPartWords;
      if (dst != rank) cluster_store(cluster_addr(&sm.part[rank], dst) + 4 * w, mine[w]);
    }
    if (TOP)
      for (int i = tid; i < c * given_n; i += NT) {
        const int dst = i / given_n, w = rank * given_n + i % given_n;
        if (dst != rank) cluster_store(cluster_addr(&sm.pool[w], dst), sm.pool[w]);
      }
    cluster_arrive();
    if (!TOP && rank != 0) return;
    cluster_wait();
  }
  float Mr = -INFINITY;
  for (int i = 0; i < c; ++i) Mr = fmaxf(Mr, sm.part[i].m);

  // ------------------------------------------------------------ alternatives
  float least = -INFINITY;
  if (TOP) {
    // the K-th of the pool: every value's place in it
    const int n = c * given_n;
    for (int i = tid; i < n; i += NT) {
      const uint32_t v = sm.pool[i];
      int place = 0;
#pragma unroll 4
      for (int j = 0; j < n; ++j) {
        const uint32_t o = sm.pool[j];
        place += (o > v || (o == v && j < i)) ? 1 : 0;
      }
      if (place == p.K - 1 && v) sm.least = from_order(v);
    }
    __syncthreads();
    least = sm.least;
    // groups that reach it
    if (m >= least && m > -INFINITY)
      for (int g = g0 + tid; g < g1; g += NT) {
        const float gt = group_top[g - g0];
        if (gt >= least && gt > -INFINITY) {
          const int at = atomicAdd(&sm.groups, 1);
          if (at < kList) sm.group[at] = g;
        }
      }
    __syncthreads();
    // their elements that do; more groups than the list holds are more elements, too
    const int ng = sm.groups;
    if (ng > kList && tid == 0) sm.count = ng;
    for (int i = tid; i < ng && ng <= kList; i += NT) {
      const int g = sm.group[i];
      const Raw x = row.load(g);
      const int v0 = row.first(g);
#pragma unroll
      for (int e = 0; e < kGroup<T>; ++e) {
        const float2 y = pair_of<T>(x, e / 2);
        const float z = (e & 1) ? y.y : y.x;
        if (z >= least && z > -INFINITY) {
          const int at = atomicAdd(&sm.count, 1);
          if (at < kList) list[at] = element_key(z, v0 + e);
        }
      }
    }
    __syncthreads();
    const int mine = sm.count;
    if (c > 1) {
      if (tid == 0) sm.at = cluster_add(cluster_addr(&sm.total, 0), mine);
      __syncthreads();
      const int at = sm.at;
      if (at + mine <= kList)
        for (int i = tid; i < mine; i += NT) cluster_store64(cluster_addr(&sm.merged[at + i], 0), list[i]);
      cluster_arrive();
      if (rank != 0) return;
      cluster_wait();
    } else {
      for (int i = tid; i < min(mine, kList); i += NT) sm.merged[i] = list[i];
      if (tid == 0) sm.total = mine;
      __syncthreads();
    }
  }

  // ------------------------------------------------------------ results (the cluster's first CTA)
  float St = 0.f, Wt = 0.f;
  int nb = 0;
  for (int i = 0; i < c; ++i) {
    const Part& q = sm.part[i];
    const float d = shift_of(q.m, Mr, p.T.sc), f = ex2(d);
    St += f * q.S;
    Wt += f * (q.W + d * q.S);
    nb += q.before;
  }
  const bool empty = Mr == -INFINITY && St == 0.f;  // nothing above -inf
  const Pair lnS = log_sum(St);
  if (tid == NT - 1) {
    const Pair inv = {p.T.hi, p.T.lo};
    if (p.lse) p.lse[entry] = empty ? -INFINITY : value_of(Pair{Mr, 0.f} * inv + lnS);
    if (p.entropy) p.entropy[entry] = empty ? 0.f : value_of(lnS + Pair{-(Wt / St) * kLn2, 0.f});
    if (p.logprob) p.logprob[entry] = empty ? -INFINITY : value_of(two_sum(lt, -Mr) * inv + -lnS);
    if (p.rank) p.rank[entry] = lt == lt ? nb + 1 : 0;
  }
  if (TOP) {
    const int total = sm.total;
    int n = total;
    if (total > kList) {
      bisect_top<T>(row, p.K, least, Mr, sm);
      n = p.K;
    }
    float* lp = p.top_logprob + (size_t)entry * p.K;
    int32_t* tk = p.top_token + (size_t)entry * p.K;
    const float ln = value_of(lnS);
    for (int i = tid; i < n; i += NT) {
      const unsigned long long key = sm.merged[i];
      int place = 0;
#pragma unroll 4
      for (int j = 0; j < n; ++j) place += sm.merged[j] > key ? 1 : 0;
      if (place < p.K) {
        const float x = from_order((uint32_t)(key >> 32));
        lp[place] = (x - Mr) * p.T.hi - ln;
        tk[place] = (int32_t)(0xFFFFFFFFu - (uint32_t)key);
      }
    }
    for (int i = n + tid; i < p.K; i += NT) {
      lp[i] = -INFINITY;
      tk[i] = -1;
    }
  }
}

template <typename T>
cudaError_t logprobs_launch(const LogprobsParams& p, int n, const RowSplit& sp, cudaStream_t st) {
  if (p.K == 0) return launch_rows(logprobs_kernel<T, false>, n, sp, 0, st, p);
  return launch_rows(logprobs_kernel<T, true>, n, sp, std::max(sizeof(float) * sp.groups, sizeof(unsigned long long) * kList), st, p);
}

}  // namespace

// CTAs per row: while that leaves SMs without work and a CTA more groups than one
// batch of its threads.
RowSplit split_rows(int rows, int V, int element_size) {
  const int groups = most_groups(V, element_size);
  int c = 1;
  while (c < 8 && (long long)rows * c * 2 <= 608 && groups > 2 * c * kLogitsThreads) c *= 2;
  while (c < 8 && groups > c * 9600) c *= 2;  // shared memory: a word per group
  RowSplit sp;
  sp.ctas = c;
  sp.groups = (groups + c - 1) / c;
  sp.threads = sp.groups >= kLogitsThreads ? kLogitsThreads : (sp.groups + 31) / 32 * 32;
  return sp;
}

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
  p.logits = a->logits;
  p.stride = a->logits_stride ? a->logits_stride : a->V;
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
  const RowSplit sp = split_rows(a->n, a->V, a->dtype == SSV_BF16 ? 2 : 4);
  p.ctas = sp.ctas;
  const int warps = sp.ctas * (sp.threads / 32);
  p.give = std::min(32, (2 * a->top_k + warps - 1) / warps);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = a->dtype == SSV_BF16 ? logprobs_launch<__nv_bfloat16>(p, a->n, sp, st)
                                             : logprobs_launch<float>(p, a->n, sp, st);
  return e == cudaSuccess ? SSV_OK : SSV_ERR_CUDA;
}
