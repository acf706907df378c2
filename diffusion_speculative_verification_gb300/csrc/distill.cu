// ssv_distill, ssv_distill_backward: a drafter's logits against the target's top
// alternatives, and the gradient.
//
// The target of a row: probabilities p_j of K listed tokens (softmax of the given
// values, or their exponentials with r = 1 - sum p left to the other tokens);
// x_v = z_v / T, q = softmax(x), u = share of q that is not listed, P = sum p + r:
//   loss = w [ sum_j p_j (ln p_j - ln q_j) + r (ln r - ln u) ]
//   d loss / d z_v = (w / T) (P q_v - p_v)                       listed v
//                    (w / T) (q_v / u) (P u - r)                 other v
// (q_v / u: the softmax among the other tokens, from their own maximum.)  u is
// summed from the other tokens alone, never as 1 - (listed): a drafter that has
// learnt its target leaves little there.  For that the listed tokens of a CTA's
// part are bits of a map in shared memory, by which a thread drops its listed
// elements.
//
// ssv_distill.  One pass over a row for the maximum and sum of the other tokens,
// its vectors coming through a ring; one or two other warps bring the target meanwhile
// (K gathers, the softmax of the given values, tokens listed twice met in a small
// table).  The CTAs of a cluster send each other their sums; with the gradient,
// each then takes its steps again from the last one on -- the last three are still
// in the ring, the others come from L2 -- and the listed tokens' entries are
// written over what the others' formula left there.
// Bound by HBM and by instructions alike: each logit is fetched from HBM once and
// each gradient written once (4096 rows of 151936 bf16, K = 128: DRAM traffic at the
// 2.49 GB that there are), 18 instructions per element at 2.5 per cycle.
// Measured: that case 424 .. 427 us, 87% of the copy rate (at earlier steps: 475 us
// with whole rows per CTA, which outgrow L2: 1.2 times the traffic; 677 us in
// quarters, whose ring and target are too much for a part; first steps again first, a
// row per CTA: 534 us beside 492); 1024 rows, K = 64, 109 us (81%); 700 fp32
// rows of 32003 34.3 us; the loss of 32 rows 6.6 us, latency, of 4096 rows, K = 128,
// 194 us (96%), of 1024 rows 55 us (84%).
//
// ssv_distill_backward.  The same second part from the statistics, in parts of 48 KB
// that a CTA holds in shared memory: 1500 rows of 151936 fp32 248 us, 7.0 TB/s, a
// little above a copy (parts of 96 KB 276 us); 2000 rows of 9001 bf16, padded, 12.0
// us; 32 rows of 151936 bf16 5.4 us.
#include "logits.cuh"

#include <algorithm>
#include <type_traits>

namespace ssv {
namespace {

constexpr int kThreads = 512;                  // most threads that share a row's part
constexpr int kHash = 2 * kLogitsMaxTop;       // places of the table in which repeated tokens meet
constexpr int kTeam = 2;                       // most warps that bring a target beside those that stream the row

struct DistillParams {
  const void* logits;
  int64_t stride, grad_stride;
  int V, K, mode;
  const int32_t* token;
  const float* logp;
  Scale T;
  const float* weight;
  float* loss;
  float* stats;             // [n, 4]: Sums of each row (written by the forward, read by the backward)
  const float* stats_in;
  const float* grad_loss;
  void* grad;
  int32_t* dev_status;
  int log_c, log_nt;
  int slot_bytes;  // of the ring
  int vec;  // rows of the gradient lie as those of the logits do to 16-byte boundaries
};

struct Mass {
  float sum, rest;  // sum p, r
};

// The target of a row: listed tokens (-1: absent), each once, their probabilities and (for a loss) the logarithms of these,
// as pairs, and the drafter's logits of them.
struct Target {
  int token[kLogitsMaxTop];
  float p[kLogitsMaxTop], z[kLogitsMaxTop];
  Pair t[kLogitsMaxTop];
  int hash[kHash];
  Mass mass;
  float top;        // largest of z
  Pair sum[kTeam];  // sum of exp((z - top) / T), of each warp of the team
  float team_mx[kTeam], team_top[kTeam];
  int team_twice[kTeam];
  Pair team_all[kTeam];
};

// TEAM warps bring a row's target while the others are busy with the row: entry 32 (member + TEAM k) + lane is a lane's
// k-th.
template <int TEAM>
struct Listed {
  static constexpr int kEach = kLogitsMaxTop / (32 * TEAM);
  int v[kEach];
  float t[kEach];
  int member;

  __device__ __forceinline__ int at(int k) const { return 32 * (member + TEAM * k) + (threadIdx.x & 31); }
  __device__ __forceinline__ bool none(int k, int K) const { return 32 * (member + TEAM * k) >= K; }  // of any lane
  __device__ __forceinline__ void load(const DistillParams& p, int row, int member_) {
    member = member_;
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
      const int j = at(k);
      v[k] = j < p.K ? p.token[(size_t)row * p.K + j] : -1;
      t[k] = j < p.K ? p.logp[(size_t)row * p.K + j] : -INFINITY;
    }
  }
  __device__ __forceinline__ void check(const DistillParams& p, bool tell) {
#pragma unroll
    for (int k = 0; k < kEach; ++k)
      if (v[k] < 0 || v[k] >= p.V) {
        if (v[k] != -1 && tell) report(p.dev_status, SSV_ERR_INVALID);
        v[k] = -1;
        t[k] = -INFINITY;
      }
  }
};

template <int TEAM>
__device__ __forceinline__ void team_sync() {
  if (TEAM == 1) __syncwarp(); else asm volatile("barrier.sync 1, %0;" ::"n"(32 * TEAM) : "memory");
}

// The team's entries to shared memory: `row` their logits, those of [lo, hi) alone (the others are not asked for).
// LOSS: with what a loss needs, the sum over the listed tokens.
template <bool LOSS, typename T, int TEAM>
__device__ __forceinline__ void weigh_listed(const DistillParams& p, Listed<TEAM>& l, const T* row, int lo, int hi,
                                             Target& tg) {
  constexpr int kEach = Listed<TEAM>::kEach;
  const int lane = threadIdx.x & 31;
  float z[kEach];
#pragma unroll
  for (int k = 0; k < kEach; ++k) z[k] = l.v[k] >= lo && l.v[k] < hi ? load_element(row + l.v[k]) : -INFINITY;
  // tokens listed twice meet in a table
  for (int h = lane + 32 * l.member; h < kHash; h += 32 * TEAM) tg.hash[h] = -1;
  team_sync<TEAM>();
  bool twice = false;
#pragma unroll
  for (int k = 0; k < kEach; ++k) {
    if (l.none(k, p.K)) break;
    if (l.v[k] < 0) continue;
    // at most K of 2 K places are taken, so that a free one is met within K steps
    uint32_t h = ((uint32_t)l.v[k] * 2654435761u) >> 24;
    for (int s = 0; s < kHash; ++s, h = (h + 1) % kHash) {
      const int was = atomicCAS(&tg.hash[h], -1, l.v[k]);
      twice |= was == l.v[k];
      if (was == -1 || was == l.v[k]) break;
    }
  }
  twice = __any_sync(0xffffffffu, twice);
  // probabilities: relative to the largest for a softmax; as they are where they are log-probabilities
  const bool as_is = p.mode == SSV_DISTILL_REST;
  // What an exponential rounded to 32 bits is off by, from its logarithm: the rest is what the sum leaves of 1, and the other
  // tokens' gradient is what r leaves of u, so that bf16 shows it too (r of 1e-6 would be off by up to 7%; 32 rows bf16 5.2
  // us without, 5.4 with it).  Without a rest it is no more than what the drafter's own exponentials are off by (2000 rows
  // of 9001 bf16: 12.0 us without; with it, when it was taken, 13.0).
  const bool exact = LOSS || sizeof(T) == 4 || as_is;
  float mx = -INFINITY, top = -INFINITY, e[kEach], off[kEach];
  Pair all = {0.f, 0.f};
#pragma unroll
  for (int k = 0; k < kEach; ++k) {
    mx = fmaxf(mx, l.t[k]);
    top = fmaxf(top, z[k]);
  }
  mx = warp_max(mx);
  top = warp_max(top);
  if (TEAM > 1) {
    if (lane == 0) {
      tg.team_mx[l.member] = mx;
      tg.team_top[l.member] = top;
      tg.team_twice[l.member] = twice;
    }
    team_sync<TEAM>();
#pragma unroll
    for (int o = 0; o < TEAM; ++o) {
      mx = fmaxf(mx, tg.team_mx[o]);
      top = fmaxf(top, tg.team_top[o]);
      twice |= tg.team_twice[o] != 0;
    }
  }
  const float ref = as_is || mx == -INFINITY ? 0.f : mx;
#pragma unroll
  for (int k = 0; k < kEach; ++k) {
    e[k] = off[k] = 0.f;
    if (l.none(k, p.K)) continue;
    e[k] = expf(l.t[k] - ref);
    if (exact && e[k] > 0.f) off[k] = e[k] * value_of(two_sum(l.t[k], -ref) + -log_sum(e[k]));
    all = all + Pair{e[k], off[k]};
  }
  all = warp_sum(all);
  if (TEAM > 1) {
    if (lane == 0) tg.team_all[l.member] = all;
    team_sync<TEAM>();
    all = tg.team_all[0];
#pragma unroll
    for (int o = 1; o < TEAM; ++o) all = all + tg.team_all[o];
  }
  const float s = value_of(all);
  const float norm = as_is || s == 0.f ? 1.f : s;
  const Pair ln = as_is || s == 0.f ? Pair{0.f, 0.f} : log_sum(all);
#pragma unroll
  for (int k = 0; k < kEach; ++k) {
    if (l.none(k, p.K)) break;
    const float q = e[k] / norm;
    e[k] = as_is || !(s < INFINITY) ? e[k] + off[k] : q + (fmaf(-q, all.hi, e[k]) + (off[k] - q * all.lo)) / norm;
    if (LOSS) tg.t[l.at(k)] = two_sum(l.t[k], -ref) + -ln;
  }
  if (twice) {  // the first of equal tokens takes the others' probabilities
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
      tg.token[l.at(k)] = l.v[k];
      tg.p[l.at(k)] = e[k];
    }
    team_sync<TEAM>();
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
      const int j = l.at(k), v = l.v[k];
      if (v < 0) continue;
      for (int o = 0; o < p.K; ++o) {
        if (o == j || tg.token[o] != v) continue;
        if (o < j) {
          l.v[k] = -1;
          break;
        }
        e[k] += tg.p[o];
        if (LOSS) tg.t[j] = log_sum(e[k]);
      }
      if (l.v[k] < 0) {
        e[k] = 0.f;
        z[k] = -INFINITY;
      }
    }
    team_sync<TEAM>();
  }
  Pair sum = {0.f, 0.f};
#pragma unroll
  for (int k = 0; k < kEach; ++k) {
    const int j = l.at(k);
    tg.token[j] = l.v[k];
    tg.p[j] = e[k];
    tg.z[j] = z[k];
  }
  if (LOSS) {
    const float zero = top == -INFINITY ? 0.f : top;  // -inf counts nothing, NaN stays
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
      if (l.none(k, p.K)) break;
      const Pair x = two_sum(z[k], -zero) * Pair{p.T.hi, p.T.lo};
      const float e1 = expf(x.hi);
      sum = sum + Pair{e1, e1 > 0.f ? e1 * x.lo : 0.f};  // -inf has no low part; NaN stays
    }
    sum = warp_sum(sum);
    if (lane == 0) tg.sum[l.member] = sum;
  }
  if (lane == 0 && l.member == 0) {
    tg.mass.sum = as_is || s == 0.f || s != s ? s : 1.f;
    const float left = as_is ? value_of(Pair{1.f, 0.f} + -all) : 0.f;
    tg.mass.rest = left < 0.f ? 0.f : left;  // NaN stays
    tg.top = top;
  }
}

// What a row's softmax needs: maximum and sum, relative to it, over the row and over the tokens that are not listed.
struct Sums {
  float m, S, mr, Sr;

  __device__ __forceinline__ bool none() const { return mr == -INFINITY && Sr == 0.f; }  // nothing is left to the others
  __device__ __forceinline__ bool empty() const { return none() && S == 0.f; }           // the row is all -inf
  // r.  Where the drafter leaves the other tokens nothing (every one is listed or masked, with -inf or with a number more
  // than 100 T below the row's largest: u is below 2^19 e^-100), what the roundings of fp32 log-probabilities leave of 1 is
  // no probability of theirs: its loss would be the mask's own size.
  __device__ __forceinline__ float rest_of(const Mass& t, const Scale& T) const {
    return t.rest < 0x1p-20f && !((mr - m) * T.hi >= -100.f) ? 0.f : t.rest;  // (NaN where the row has nothing, or a NaN)
  }
};

// e^x: -inf has no low part; NaN stays
__device__ __forceinline__ float exp_of(Pair x) {
  const float e = expf(x.hi);
  return e > 0.f ? fmaf(e, x.lo, e) : e;
}

// The gradient's coefficients.
struct Slope {
  float ref, coef;   // other tokens: coef 2^((z - ref) sc)
  float top, share;  // listed ones: wT (share 2^((z - top) sc) - p)
  float wT;
  bool empty;
};

__device__ __forceinline__ Slope slope_of(const Sums& s, const Mass& t, const Scale& T, float w) {
  const float rest = s.rest_of(t, T), P = t.sum + rest;
  Slope k;
  k.wT = w * T.hi;
  k.ref = s.none() ? 0.f : s.mr;
  // P u - r is a small difference where the drafter has come near its target: u's exponent to more than 32 bits
  const float u = exp_of(two_sum(s.mr, -s.m) * Pair{T.hi, T.lo}) * (s.Sr / s.S);
  k.coef = s.none() ? 0.f : k.wT * fmaf(P, u, -rest) / s.Sr;
  k.top = s.m;
  k.share = P / s.S;
  k.empty = s.empty();
  return k;
}

__device__ __forceinline__ void store_vector(void* p, const uint4& r) {
  asm volatile("st.global.cs.v4.b32 [%0], {%1, %2, %3, %4};" ::"l"(p), "r"(r.x), "r"(r.y), "r"(r.z), "r"(r.w) : "memory");
}

template <typename T>
__device__ __forceinline__ uint32_t two_of(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// a vector of eight or four values f(e)
template <typename T, typename F>
__device__ __forceinline__ uint4 pack_vector(F f) {
  uint4 y;
  if constexpr (sizeof(T) == 2) {
    y.x = two_of<T>(f(0), f(1));
    y.y = two_of<T>(f(2), f(3));
    y.z = two_of<T>(f(4), f(5));
    y.w = two_of<T>(f(6), f(7));
  } else {
    y.x = __float_as_uint(f(0));
    y.y = __float_as_uint(f(1));
    y.z = __float_as_uint(f(2));
    y.w = __float_as_uint(f(3));
  }
  return y;
}

// Vectors of the output, with f(v) for element v, at any offset from a vector of the input.
template <typename T, typename F>
__device__ __forceinline__ void write_elements(T* out, int lo, int hi, F f) {
  const int lead = (int)((reinterpret_cast<uintptr_t>(out) & 15) / sizeof(T));
  char* base = reinterpret_cast<char*>(reinterpret_cast<uintptr_t>(out) & ~uintptr_t(15));
  const int first = (lo + lead) / kVec<T>, end = (hi + lead + kVec<T> - 1) / kVec<T>;
  for (int i = first + threadIdx.x; i < end; i += blockDim.x) {
    const int v0 = i * kVec<T> - lead;
    if (v0 >= lo && v0 + kVec<T> <= hi) {
      store_vector(base + (size_t)i * 16, pack_vector<T>([&](int e) { return f(v0 + e); }));
    } else {
      for (int v = max(v0, lo); v < min(v0 + kVec<T>, hi); ++v) out[v] = Elem<T>::from_f32(f(v));
    }
  }
}

// The gradient of the other tokens, of one vector.
template <typename T>
struct Gradient {
  float2 ref2, sc2, lo2, c2;

  __device__ __forceinline__ Gradient(const Slope& k, const Scale& T_)
      : ref2(make_float2(-k.ref, -k.ref)), sc2(make_float2(T_.down, T_.down)), lo2(make_float2(T_.rest, T_.rest)),
        c2(make_float2(k.coef, k.coef)) {}
  __device__ __forceinline__ uint4 operator()(const uint4& x) const {
    float2 y[kVec<T> / 2];
#pragma unroll
    for (int e = 0; e < kVec<T> / 2; ++e) {
      const float2 d = add2(pair_of<T>(x, e), ref2);
      float2 a = mul2(d, sc2);
      if (sizeof(T) == 4) a = fma2(d, lo2, a);  // the scale to 48 bits, as in the sums; bf16 would not show it
      y[e] = mul2(make_float2(ex2(a.x), ex2(a.y)), c2);
    }
    return pack_vector<T>([&](int e) { return e & 1 ? y[e / 2].y : y[e / 2].x; });
  }
};

// The elements of a vector that is not whole.
template <typename T>
__device__ __noinline__ void write_edge(const RowView<T>& row, int i, const uint4 y, T* out) {
  const int v0 = row.first(i);
  for (int e = 0; e < kVec<T>; ++e) {
    const uint32_t w = e * (int)sizeof(T) < 4 ? y.x : e * (int)sizeof(T) < 8 ? y.y : e * (int)sizeof(T) < 12 ? y.z : y.w;
    if (v0 + e < 0 || v0 + e >= row.V) continue;
    if (sizeof(T) == 2)
      reinterpret_cast<uint16_t*>(out)[v0 + e] = (uint16_t)(e & 1 ? w >> 16 : w);
    else
      reinterpret_cast<uint32_t*>(out)[v0 + e] = w;
  }
}

// Step k of the thread's vectors, from its slots to an output whose vectors are those of the input; the row's first and
// last vectors by element.
template <typename T>
__device__ __forceinline__ void write_step(const RowView<T>& row, const PartView<T>& part, int k, const uint4* slots, T* out,
                                           const Gradient<T>& gradient) {
  const int NT = part.NT, i = part.i0 + (int)threadIdx.x + NT * kBatch * k;
  char* to = reinterpret_cast<char*>(reinterpret_cast<uintptr_t>(out) & ~uintptr_t(15)) + (size_t)i * 16;
  if (part.full(k)) {
#pragma unroll
    for (int u = 0; u < kBatch; ++u) store_vector(to + (size_t)(NT * 16) * u, gradient(slots[NT * u]));
  } else {
    const int end = min(part.i1, row.hi);
#pragma unroll
    for (int u = 0; u < kBatch; ++u)
      if (i + NT * u >= row.lo && i + NT * u < end) store_vector(to + (size_t)(NT * 16) * u, gradient(slots[NT * u]));
    part.edges(row, k, [&](int d, int edge) { write_edge<T>(row, edge, gradient(slots[d]), out); });
  }
}

// Of an output at any offset from the input, with elements from `in`.
template <typename T>
__device__ __forceinline__ void write_apart(const PartView<T>& part, const T* in, T* out, const Slope& k, const Scale& T_) {
  write_elements<T>(out, part.lo, part.hi, [&](int v) {
    const float d = Elem<T>::to_f32(in[v]) - k.ref;
    return ex2(fmaf(d, T_.rest, d * T_.down)) * k.coef;
  });
}

// The listed tokens' entries, over what is there (after a barrier).
template <typename T>
__device__ __forceinline__ void write_listed(const DistillParams& p, const PartView<T>& part, T* out, const Slope& k,
                                             const Target& tg) {
  for (int j = threadIdx.x; j < p.K; j += blockDim.x) {
    const int v = tg.token[j];
    if (v < part.lo || v >= part.hi) continue;
    const float q = k.share * exp_of(two_sum(tg.z[j], -k.top) * Pair{p.T.hi, p.T.lo});
    out[v] = Elem<T>::from_f32(k.wT * (q - tg.p[j]));
  }
}

template <typename T>
__device__ __forceinline__ void write_zeros(const PartView<T>& part, T* out) {
  write_elements<T>(out, part.lo, part.hi, [](int) { return 0.f; });
}

template <int THREADS>
struct Shared {
  Target tg;
  Slope slope;
  uint32_t part[THREADS / 32 * kMaxCluster][4];  // of every warp: maximum and sum (a pair) of its other tokens
};

// Steps in flight: three with the gradient, which find the last three fifths of a part of 152 KB there (4096 rows, when it was
// taken: 428 us; two 433).  With 256 threads a ring of two would let a fourth CTA onto an SM for parts above 48 KB (700 fp32
// rows of 32003: 35.3 us with three, 31.2 with two; other sizes 18.9 -> 14.8, 112 -> 96, but also 47 -> 51 and 125 -> 135).
template <bool GRAD> constexpr int kStages = GRAD ? 3 : 2;

// Most threads that share a row, and how many CTAs of them the registers are to leave room for on an SM (one more would
// spill by tens of bytes; distill_kernel<bf16, true, 0, 1> spills 4 as it is).  Shared memory may hold fewer: of 256 threads
// with the gradient four only where a part has at most three steps (48 KB), three above.
constexpr int most_threads(bool grad, int log_nt) { return grad && log_nt == 9 ? kThreads : kThreads / 2; }
constexpr int ctas_per_sm(bool grad, int log_nt, int team) { return !grad ? 4 : log_nt == 9 ? 2 : team == 1 ? 4 : 3; }

// LOG_NT: 2^LOG_NT threads share a row, so that a step's addresses are constants apart (when it was taken: 4096 rows 444 us,
// known at the launch alone 451); 0: as many as the launch says, for rows that are too short for them.  TEAM warps bring the
// target.
template <typename T, bool GRAD, int LOG_NT, int TEAM>
__global__ void __launch_bounds__(most_threads(GRAD, LOG_NT) + 32 * TEAM, ctas_per_sm(GRAD, LOG_NT, TEAM))
    distill_kernel(const DistillParams p) {
  // a ring of slots; behind it a word per thread and step, whose bit (vector of the step, element) says that the
  // element is a listed token
  extern __shared__ __align__(128) unsigned char dynamic[];
  __shared__ Shared<most_threads(GRAD, LOG_NT)> sm;
  // NT threads share the row, and the team behind them brings its target; the team's first warp joins the sums
  const int log_nt = LOG_NT ? LOG_NT : p.log_nt;
  const int tid = threadIdx.x, NT = 1 << log_nt, lane = tid & 31, warp = tid >> 5, nw = NT >> 5;
  const bool streams = warp < nw, joins = warp == nw;
  const int c = 1 << p.log_c;
  const int rank = (int)blockIdx.x & (c - 1), entry = (int)blockIdx.x >> p.log_c;
  uint32_t* listed = reinterpret_cast<uint32_t*>(dynamic + p.slot_bytes);
  if (c > 1) cluster_arrive();  // waited for before the first access to another CTA's shared memory
  pdl_wait();
  pdl_trigger();
  const float w = p.weight ? p.weight[entry] : 1.f;
  const RowView<T> row(static_cast<const T*>(p.logits) + (int64_t)entry * p.stride, p.V);
  const PartView<T> part(row, rank, p.log_c, log_nt);
  T* out = GRAD ? static_cast<T*>(p.grad) + (int64_t)entry * p.grad_stride : nullptr;
  if (w == 0.f) {  // not read at all
    if (rank == 0 && tid == 0) {
      p.loss[entry] = 0.f;
      if (p.stats)
        for (int i = 0; i < 4; ++i) p.stats[4 * (size_t)entry + i] = 0.f;
    }
    if (GRAD) write_zeros<T>(part, out);
    if (c > 1) cluster_wait();
    return;
  }
  uint4* slots = part.slots_in(dynamic, row);
  auto step_slots = [&](int k) { return slots + kBatch * (k % kStages<GRAD>) * NT + tid; };
  if (streams)
    for (int k = 0; k < kStages<GRAD>; ++k) part.fetch(row, k, step_slots(k));

  // ------------------------------------------------------------ the target
  Target& tg = sm.tg;
  Listed<TEAM> mine;
  if (!streams) mine.load(p, entry, warp - nw);
  for (int i = tid; i < part.steps * NT; i += blockDim.x) listed[i] = 0u;
  __syncthreads();
  if (!streams) {
    mine.check(p, rank == 0);
#pragma unroll
    for (int k = 0; k < mine.kEach; ++k) {
      const int v = mine.v[k];
      if (v < part.lo || v >= part.hi) continue;
      const int i = (v - part.at) / kVec<T>, e = (v - part.at) % kVec<T>, s = i >> log_nt;
      atomicOr(&listed[s / kBatch * NT + (i & (NT - 1))], 1u << (s % kBatch * kVec<T> + e));
    }
  }
  __syncthreads();

  // ------------------------------------------------------------ the other tokens
  float m = -INFINITY, S = 0.f;
  const float2 sc2 = make_float2(p.T.down, p.T.down), lo2 = make_float2(p.T.rest, p.T.rest);
  auto step = [&](auto is_full, int k) {
    constexpr bool FULL = decltype(is_full)::value;
    uint4* at = step_slots(k);
    // a listed element counts as -inf from here on (its gradient is written over)
    for (uint32_t bits = listed[k * NT + tid]; bits; bits &= bits - 1) {
      const int b = __ffs(bits) - 1;
      reinterpret_cast<T*>(at + NT * (b / kVec<T>))[b % kVec<T>] = Elem<T>::from_f32(-INFINITY);
    }
    uint4 x[kBatch];
    part.template take<FULL>(k, at, x);
    const float2 mx2 = step_max<T>(x);
    const float mx = fmaxf(mx2.x, mx2.y);
    part.fetch(row, k + kStages<GRAD>, at);  // into the slots that have just been read
    if (mx > m) {
      S *= ex2(shift_of(m, mx, p.T.sc));
      m = mx;
    }
    const float mm = m == -INFINITY ? 0.f : m;  // nothing but -inf and NaN so far
    const float2 nm = make_float2(-mm, -mm);
    float2 S2 = make_float2(0.f, 0.f);
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      if (!FULL && part.i0 + tid + NT * (kBatch * k + u) >= part.i1) break;
#pragma unroll
      for (int i = 0; i < kVec<T> / 2; ++i) {
        // the scale to 48 bits: rounded to 24 it would move every term the same way, by up to 2^-25 of its exponent
        const float2 d = add2(pair_of<T>(x[u], i), nm), y = fma2(d, lo2, mul2(d, sc2));
        S2 = add2(S2, make_float2(ex2(y.x), ex2(y.y)));
      }
    }
    S += S2.x + S2.y;
  };
  if (streams) {
    for (int k = 0; k < part.steps; ++k) {
      copy_wait<kStages<GRAD> - 1>();
      if (part.full(k)) step(std::true_type{}, k); else step(std::false_type{}, k);
    }
    copy_wait<0>();
  } else {
    weigh_listed<true>(p, mine, row.row, 0, p.V, tg);
  }
  if (c > 1) cluster_wait();
  if (streams) {
    const float M = warp_max(m);
    const Pair Sw = warp_sum(Pair{ex2(shift_of(m, M, p.T.sc)) * S, 0.f});
    const int me = rank * nw + warp;
    const uint32_t word = (lane & 3) == 0 ? __float_as_uint(M) : __float_as_uint((lane & 3) == 1 ? Sw.hi : Sw.lo);
    if (c == 1) {
      if (lane < 3) sm.part[me][lane] = word;
    } else if (lane < 4 * (GRAD ? c : 1)) {  // the loss alone is the first CTA's
      cluster_store(cluster_addr(&sm.part[me][lane & 3], lane >> 2), word);
    }
  }
  if (c > 1) {
    cluster_arrive();
    if (!GRAD && rank != 0) return;
    cluster_wait();
  } else {
    __syncthreads();
  }
  if (!GRAD && !joins) return;

  // ------------------------------------------------------------ the row's sums, by one warp of each CTA in the same order
  // (The sums are of 32 bits, joined in 48: the last few additions would cost a loss, which is a small difference of
  // their logarithms, as much as all before.)
  Sums sums;
  Pair S_all, S_rest;
  float listed_share = 0.f;  // 1 - u
  if (joins) {
    const int n = c * nw;
    float mx = -INFINITY;
    for (int q = lane; q < n; q += 32) mx = fmaxf(mx, __uint_as_float(sm.part[q][0]));
    mx = warp_max(mx);
    S_rest = Pair{0.f, 0.f};
    for (int q = lane; q < n; q += 32) {
      const float f = ex2(shift_of(__uint_as_float(sm.part[q][0]), mx, p.T.sc));
      S_rest = S_rest + Pair{f * __uint_as_float(sm.part[q][1]), f * __uint_as_float(sm.part[q][2])};
    }
    S_rest = warp_sum(S_rest);
    const float m_all = fmaxf(mx, tg.top);
    const float fr = ex2(shift_of(mx, m_all, p.T.sc)), ft = ex2(shift_of(tg.top, m_all, p.T.sc));
    Pair st = tg.sum[0];
#pragma unroll
    for (int o = 1; o < TEAM; ++o) st = st + tg.sum[o];
    st = Pair{ft * st.hi, ft * st.lo};
    S_all = Pair{fr * S_rest.hi, fr * S_rest.lo} + st;
    sums = {m_all, value_of(S_all), mx, value_of(S_rest)};
    listed_share = value_of(st) / sums.S;
    if (GRAD) {
      if (lane == 0) sm.slope = slope_of(sums, tg.mass, p.T, w);
    }
  }
  if (GRAD) __syncthreads();
  if (rank == 0 && joins) {
    const Pair inv = {p.T.hi, p.T.lo}, lnS = log_sum(S_all);
    Pair loss = {0.f, 0.f};
#pragma unroll
    for (int k = 0; k < kLogitsMaxTop / 32; ++k) {
      const int j = lane + 32 * k;
      const float pj = j < p.K ? tg.p[j] : 0.f;
      if (pj > 0.f || pj != pj) {
        // ln p - ln q, a small difference of large numbers: rounded once
        const Pair q = two_sum(tg.z[j], -sums.m) * inv + -lnS;
        loss = loss + Pair{pj, 0.f} * Pair{value_of(tg.t[j] + -q), 0.f};
      }
    }
    loss = warp_sum(loss);
    if (lane == 0) {
      const float rest = sums.rest_of(tg.mass, p.T), P = tg.mass.sum + rest;
      // a share of more than half from what is listed: the difference of two logarithms would be off by their rounding
      const Pair ln_u = listed_share < 0.5f ? Pair{log1pf(-listed_share), 0.f}
                        : sums.none()       ? Pair{-INFINITY, 0.f}
                                            : two_sum(sums.mr, -sums.m) * inv + (log_sum(S_rest) + -lnS);
      if (rest > 0.f) loss = loss + Pair{rest, 0.f} * Pair{value_of(log_sum(rest) + -ln_u), 0.f};
      float l = w * value_of(loss);
      if (sums.S != sums.S) l = sums.S;
      if (sums.empty()) l = P == 0.f ? 0.f : w * (INFINITY * P);  // no token of the target has a chance; NaN stays
      p.loss[entry] = l;
      if (p.stats) {
        float* to = p.stats + 4 * (size_t)entry;
        to[0] = sums.m;
        to[1] = sums.S;
        to[2] = sums.mr;
        to[3] = sums.Sr;
      }
    }
  }
  if (GRAD) {
    const Slope k = sm.slope;
    if (k.empty) {
      write_zeros<T>(part, out);
      return;
    }
    if (p.vec) {
      // from the last step on: the last ones are still in the ring, and what was read late is the likeliest to be in L2
      const Gradient<T> gradient(k, p.T);
      for (int q = streams ? part.steps - 1 : -1; q >= 0; --q) {
        copy_wait<kStages<GRAD> - 1>();
        write_step<T>(row, part, q, step_slots(q), out, gradient);
        part.fetch(row, q - kStages<GRAD>, step_slots(q));
      }
    } else {
      write_apart<T>(part, row.row, out, k, p.T);
    }
    __syncthreads();
    write_listed<T>(p, part, out, k, tg);
  }
}

template <typename T>
__global__ void __launch_bounds__(128, 8) distill_backward_kernel(const DistillParams p) {
  extern __shared__ __align__(128) unsigned char dynamic[];
  __shared__ Target tg;
  __shared__ Slope slope;
  const int tid = threadIdx.x, NT = blockDim.x;
  const int c = 1 << p.log_c;
  const int rank = (int)blockIdx.x & (c - 1), entry = (int)blockIdx.x >> p.log_c;
  pdl_wait();
  pdl_trigger();
  const float w = p.weight ? p.weight[entry] : 1.f;
  const RowView<T> row(static_cast<const T*>(p.logits) + (int64_t)entry * p.stride, p.V);
  const PartView<T> part(row, rank, p.log_c, p.log_nt);
  T* out = static_cast<T*>(p.grad) + (int64_t)entry * p.grad_stride;
  if (w == 0.f) {
    write_zeros<T>(part, out);
    return;
  }
  uint4* slots = part.slots_in(dynamic, row);
  for (int k = 0; k < part.steps; ++k) part.fetch(row, k, slots + kBatch * k * NT + tid);
  if (tid < 32) {
    Listed<1> mine;
    mine.load(p, entry, 0);
    const float* from = p.stats_in + 4 * (size_t)entry;
    const Sums sums = {from[0], from[1], from[2], from[3]};
    const float up = p.grad_loss ? p.grad_loss[entry] : 1.f;
    mine.check(p, rank == 0);
    weigh_listed<false>(p, mine, row.row, part.lo, part.hi, tg);
    __syncwarp();
    if (tid == 0) slope = slope_of(sums, tg.mass, p.T, w * up);
  }
  __syncthreads();
  copy_wait<0>();
  if (slope.empty) {
    write_zeros<T>(part, out);
    return;
  }
  if (p.vec) {
    const Gradient<T> gradient(slope, p.T);
    for (int k = 0; k < part.steps; ++k) write_step<T>(row, part, k, slots + kBatch * k * NT + tid, out, gradient);
  } else {
    __syncthreads();  // every thread's vectors are there
    write_apart<T>(part, reinterpret_cast<const T*>(slots) - part.at, out, slope, p.T);
  }
  __syncthreads();
  write_listed<T>(p, part, out, slope, tg);
}

// The gradient's rows apart from the logits', or on them exactly.
bool rows_apart(const void* x, const void* y, int64_t xs, int64_t ys, int V, int n, int es) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(x), b = reinterpret_cast<uintptr_t>(y);
  if (a == b && (xs == ys || n == 1)) return true;
  const uintptr_t ae = a + ((uintptr_t)(n - 1) * xs + V) * es, be = b + ((uintptr_t)(n - 1) * ys + V) * es;
  if (a >= be || b >= ae) return true;
  if (xs != ys) return false;
  // parts of the same wider rows
  const uintptr_t d = (a < b ? b - a : a - b) % ((uintptr_t)xs * es);
  return d >= (uintptr_t)V * es && d + (uintptr_t)V * es <= (uintptr_t)xs * es;
}

ssv_status distill_check(const ssv_distill_args* a, DistillParams& p) {
  if (!a) return SSV_ERR_INVALID;
  if (!logits_shape_ok(a->logits, a->logits_stride, a->dtype, a->V, a->n) || a->K < 1 ||
      (a->mode != SSV_DISTILL_RENORM && a->mode != SSV_DISTILL_REST))
    return SSV_ERR_INVALID;
  if (!logits_scale(a->T, &p.T)) return SSV_ERR_NOT_FINITE;
  if (a->V > kLogitsMaxVocab || a->K > kLogitsMaxTop) return SSV_ERR_UNSUPPORTED;
  if (a->n == 0) return SSV_OK;
  if (!a->logits || !a->teacher_token || !a->teacher_logprob) return SSV_ERR_INVALID;
  if (((uintptr_t)a->teacher_token | (uintptr_t)a->teacher_logprob | (uintptr_t)a->weight | (uintptr_t)a->loss |
       (uintptr_t)a->stats | (uintptr_t)a->grad_loss | (uintptr_t)a->dev_status) & 3u)
    return SSV_ERR_INVALID;
  p.logits = a->logits;
  p.stride = a->logits_stride ? a->logits_stride : a->V;
  p.V = a->V;
  p.K = a->K;
  p.mode = a->mode;
  p.token = a->teacher_token;
  p.logp = a->teacher_logprob;
  p.weight = a->weight;
  p.loss = a->loss;
  p.stats = a->stats;
  p.stats_in = a->stats;
  p.grad_loss = a->grad_loss;
  p.grad = a->grad;
  p.dev_status = a->dev_status;
  p.grad_stride = a->grad_stride ? a->grad_stride : a->V;
  p.vec = 0;
  if (a->grad) {
    const int es = a->dtype == SSV_BF16 ? 2 : 4;
    if (!logits_shape_ok(a->grad, a->grad_stride, a->dtype, a->V, a->n) ||
        !rows_apart(a->logits, a->grad, p.stride, p.grad_stride, a->V, a->n, es))
      return SSV_ERR_INVALID;
    p.vec = (((uintptr_t)a->logits ^ (uintptr_t)a->grad) & 15u) == 0 &&
            (a->n == 1 || ((uint64_t)(p.stride - p.grad_stride) * es) % 16 == 0);
  }
  return SSV_OK;
}

// A row in parts of at most `bytes`, as far as `most` CTAs go; more of them while all rows' are no more than `room` and a
// part has more than one step.  (Loss of 32 rows: 6.6 us with room for four per SM, for two and for eight.)
RowSplit distill_split(int rows, int V, int element_size, int bytes, int most, int threads, int room) {
  const int vectors = row_vectors(V, element_size);
  int c = 1;
  while (c < most && (vectors + c - 1) / c > bytes / 16) c *= 2;
  while (c < most && (long long)rows * c * 2 <= room && vectors > 4 * c * threads) c *= 2;
  return split_of(vectors, c, threads);
}

template <typename T, bool GRAD, int LOG_NT, int TEAM>
cudaError_t distill_launch_as(const DistillParams& p, int n, const RowSplit& sp, size_t smem, cudaStream_t st) {
  static uint64_t done = 0;
  const cudaError_t e = allow_shared(distill_kernel<T, GRAD, LOG_NT, TEAM>, smem, &done);
  return e != cudaSuccess ? e : launch_rows(distill_kernel<T, GRAD, LOG_NT, TEAM>, n, sp, sp.threads + 32 * TEAM, smem, st, p);
}

template <typename T, bool GRAD, int TEAM>
cudaError_t distill_launch_team(const DistillParams& p, int n, const RowSplit& sp, size_t smem, cudaStream_t st) {
  if constexpr (GRAD)
    if (sp.log_nt == 9) return distill_launch_as<T, GRAD, 9, TEAM>(p, n, sp, smem, st);
  return sp.log_nt == 8 ? distill_launch_as<T, GRAD, 8, TEAM>(p, n, sp, smem, st)
                        : distill_launch_as<T, GRAD, 0, TEAM>(p, n, sp, smem, st);
}

template <typename T, bool GRAD>
cudaError_t distill_launch(DistillParams& p, int n, cudaStream_t st) {
  // With the gradient parts of 160 KB: two CTAs per SM then have 46 MB of rows on their way, which L2 holds, and 512
  // threads make the most of a part's fixed cost (4096 rows: 424 us; 256 threads 465 us).  Parts of up to 128 KB go to 256
  // threads, in which steps are shorter and one CTA's barriers are other CTAs' time (rows of 100277 bf16: 147 us with 512
  // threads, 124 with 256; of 9001 fp32: 27 and 20 us).  The loss alone reads a row once: no limit, and 256 threads (32
  // rows: 6.6 us; 512 threads 8.3 us).
  // Rows are cut further while all parts are no more than an SM holds of short ones at a time, on 152 SMs (64 rows of 151936
  // bf16, K = 64: 12.2 us, 18.9 where one fewer fits; 150, K = 128: 17.9 us, 24.0 with one more).
  const int per_sm = GRAD && p.K > 64 ? 3 : 4;
  RowSplit sp = distill_split(n, p.V, sizeof(T), GRAD ? 160 * 1024 : 1 << 20, kMaxCluster, 256, 152 * per_sm);
  if (GRAD && sp.vectors > 128 * 1024 / 16) sp = split_of(row_vectors(p.V, sizeof(T)), sp.ctas, 512);
  p.log_c = sp.log_c;
  p.log_nt = sp.log_nt;
  p.slot_bytes = 16 * kStages<GRAD> * kBatch * sp.threads + kSlotSlack;
  const size_t smem = p.slot_bytes + sizeof(uint32_t) * (size_t)sp.batches() * sp.threads;
  // The target is as long on its way as the row's first reading where a warp has four tokens per lane: two warps for more
  // than 64 tokens (when it was taken, 4096 rows, K = 128: 428 us; one warp 444, four 435, whose registers do not suffice),
  // one for fewer (1024 rows, K = 64: 109 us; two 111) and for the loss, of whose 256 threads two take more room (32 rows,
  // K = 32: 6.6 us; two 7.8).
  if constexpr (GRAD)
    if (p.K > 64) return distill_launch_team<T, GRAD, 2>(p, n, sp, smem, st);
  return distill_launch_team<T, GRAD, 1>(p, n, sp, smem, st);
}

template <typename T>
cudaError_t backward_launch(DistillParams& p, int n, cudaStream_t st) {
  static uint64_t done = 0;
  // (1500 fp32 rows: 248 us in parts of 48 KB and of 24, 276 us in parts of 96; 265 us with 256 threads, for whom a
  // part's fixed cost is too much)
  const RowSplit sp = distill_split(n, p.V, sizeof(T), 48 * 1024, 64, 128, 608);
  p.log_c = sp.log_c;
  p.log_nt = sp.log_nt;
  const size_t smem = 16 * (size_t)sp.vectors + kSlotSlack;
  const cudaError_t e = allow_shared(distill_backward_kernel<T>, smem, &done);
  return e != cudaSuccess ? e : launch_rows(distill_backward_kernel<T>, n, sp, sp.threads, smem, st, p);
}

}  // namespace
}  // namespace ssv

extern "C" ssv_status ssv_distill(const ssv_distill_args* a, void* stream) {
  using namespace ssv;
  DistillParams p;
  const ssv_status s = distill_check(a, p);
  if (s != SSV_OK) return s;
  if (a->n == 0) return SSV_OK;
  if (!a->loss || a->grad_loss) return SSV_ERR_INVALID;
  const int es = a->dtype == SSV_BF16 ? 2 : 4;
  if (meets_rows(a->loss, 4 * (size_t)a->n, a->logits, p.stride, a->V, a->n, es) ||
      meets_rows(a->stats, 16 * (size_t)a->n, a->logits, p.stride, a->V, a->n, es) ||
      (a->grad && (meets_rows(a->loss, 4 * (size_t)a->n, a->grad, p.grad_stride, a->V, a->n, es) ||
                   meets_rows(a->stats, 16 * (size_t)a->n, a->grad, p.grad_stride, a->V, a->n, es))))
    return SSV_ERR_INVALID;
  using bf16 = __nv_bfloat16;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (a->grad)
    e = a->dtype == SSV_BF16 ? distill_launch<bf16, true>(p, a->n, st) : distill_launch<float, true>(p, a->n, st);
  else
    e = a->dtype == SSV_BF16 ? distill_launch<bf16, false>(p, a->n, st) : distill_launch<float, false>(p, a->n, st);
  return e == cudaSuccess ? SSV_OK : SSV_ERR_CUDA;
}

extern "C" ssv_status ssv_distill_backward(const ssv_distill_args* a, void* stream) {
  using namespace ssv;
  DistillParams p;
  const ssv_status s = distill_check(a, p);
  if (s != SSV_OK) return s;
  if (a->n == 0) return SSV_OK;
  if (!a->stats || !a->grad) return SSV_ERR_INVALID;
  if (meets_rows(a->stats, 16 * (size_t)a->n, a->grad, p.grad_stride, a->V, a->n, a->dtype == SSV_BF16 ? 2 : 4))
    return SSV_ERR_INVALID;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e =
      a->dtype == SSV_BF16 ? backward_launch<__nv_bfloat16>(p, a->n, st) : backward_launch<float>(p, a->n, st);
  return e == cudaSuccess ? SSV_OK : SSV_ERR_CUDA;
}
