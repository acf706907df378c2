// ssv_distill, ssv_distill_backward: a drafter's logits against the target's top
// alternatives, and the gradient.
//
// The target of a row: probabilities p_j of K listed tokens (softmax of the given
// values, or their exponentials with r = 1 - sum p left to the other tokens);
// x_v = z_v / T, q = softmax(x), u = share of q that is not listed, P = sum p + r:
//   loss = w [ sum_j p_j (ln p_j - ln q_j) + r (ln r - ln u) ]
//   d loss / d z_v = (w / T) (P q_v - p_v)                       listed v
//                    (w / T) (q_v / u) (P u - r)                 other v
// (q_v / u: the softmax among the other tokens, from their own maximum.)  u is summed from
// the other tokens alone, never as 1 - (listed): a drafter that has learnt its
// target leaves little there.  For that the listed tokens of a CTA's part are
// bits of a map in shared memory, by which a group drops its listed elements.
//
// Forward: one pass over a row for the maximum and sum of the other tokens; the
// listed ones, K gathers, join at the end.  With the gradient, the cluster's CTAs
// exchange their sums, and each reads its part of the row again, from L2, and
// writes the gradient; the listed tokens' entries are then written over.  Backward:
// the same second pass from the forward's statistics.
#include "logits.cuh"

namespace ssv {
namespace {

constexpr int kMaxCluster = 8;

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
  int ctas;
  int vec;  // rows of the gradient lie as those of the logits do to 32-byte boundaries
};

// The target of a row: listed tokens (-1: absent), each once, their probabilities and the logarithms of these.
struct Target {
  int token[kLogitsMaxTop];
  float p[kLogitsMaxTop], t[kLogitsMaxTop];
  float z[kLogitsMaxTop];  // the drafter's logits of them
  float sum, rest;         // sum p, r
};

// Whole CTA: the target of row i.  A token listed more than once counts with the sum of its probabilities.
__device__ __forceinline__ void load_target(const DistillParams& p, int i, bool tell, Target& tg) {
  const int tid = threadIdx.x, NT = blockDim.x;
  for (int j = tid; j < p.K; j += NT) {
    int v = p.token[(size_t)i * p.K + j];
    float t = p.logp[(size_t)i * p.K + j];
    if (v < 0 || v >= p.V) {
      if (v != -1 && tell) report(p.dev_status, SSV_ERR_INVALID);
      v = -1;
      t = -INFINITY;
    }
    tg.token[j] = v;
    tg.t[j] = t;
  }
  __syncthreads();
  if (tid < 32) {
    // probabilities, by one warp: four entries per lane, the sums in a fixed order
    float x[kLogitsMaxTop / 32], mx = -INFINITY;
#pragma unroll
    for (int k = 0; k < kLogitsMaxTop / 32; ++k) {
      const int j = tid + 32 * k;
      x[k] = j < p.K ? tg.t[j] : -INFINITY;
      mx = fmaxf(mx, x[k]);
    }
    mx = warp_max(mx);
    // relative to the largest for a softmax; as they are where they are log-probabilities
    const float ref = p.mode == SSV_DISTILL_REST || mx == -INFINITY ? 0.f : mx;
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < kLogitsMaxTop / 32; ++k) {
      x[k] -= ref;
      s += expf(x[k]);
    }
    s = warp_sum(s);
    const float norm = p.mode == SSV_DISTILL_REST || s == 0.f ? 1.f : s;
    const float ln = logf(norm);
#pragma unroll
    for (int k = 0; k < kLogitsMaxTop / 32; ++k) {
      const int j = tid + 32 * k;
      if (j < p.K) {
        tg.p[j] = expf(x[k]) / norm;
        tg.t[j] = x[k] - ln;
      }
    }
    if (tid == 0) {
      tg.sum = p.mode == SSV_DISTILL_REST ? s : (s == 0.f ? 0.f : 1.f);
      if (s != s) tg.sum = s;
      tg.rest = p.mode == SSV_DISTILL_REST ? (s > 1.f ? 0.f : 1.f - s) : 0.f;  // NaN stays
    }
  }
  __syncthreads();
  // duplicates: the first of them takes the others' probabilities
  float p_all[(kLogitsMaxTop + 31) / 32];
  unsigned twice = 0, later = 0;
  int n = 0;
  for (int j = tid; j < p.K; j += NT, ++n) {
    const int v = tg.token[j];
    float s = tg.p[j];
    bool first = true;
    for (int i2 = 0; i2 < p.K; ++i2) {
      if (i2 == j || v < 0 || tg.token[i2] != v) continue;
      if (i2 < j) first = false; else { s += tg.p[i2]; twice |= 1u << n; }
    }
    if (!first) later |= 1u << n;
    if (n < (kLogitsMaxTop + 31) / 32) p_all[n] = s;
  }
  __syncthreads();
  n = 0;
  for (int j = tid; j < p.K; j += NT, ++n) {
    if (later >> n & 1) {
      tg.token[j] = -1;
      tg.p[j] = 0.f;
      tg.t[j] = -INFINITY;
    } else if (twice >> n & 1) {
      tg.p[j] = p_all[n];
      tg.t[j] = logf(p_all[n]);
    }
  }
}

// r, where the drafter leaves the other tokens nothing (every one is listed or masked): there, what the roundings of
// fp32 log-probabilities leave of 1 is no probability of other tokens.
__device__ __forceinline__ float rest_of(const Target& tg, bool none) {
  return none && tg.rest < 0x1p-20f ? 0.f : tg.rest;
}

// What a row's softmax needs: maximum and sum, relative to it, over the row and over the tokens that are not listed.
struct Sums {
  float m, S, mr, Sr;

  __device__ __forceinline__ bool none() const { return mr == -INFINITY && Sr == 0.f; }  // nothing is left to the others
  __device__ __forceinline__ bool empty() const { return none() && S == 0.f; }           // the row is all -inf
  // ln of the others' share
  __device__ __forceinline__ Pair ln_u(const Scale& T) const {
    if (none()) return {-INFINITY, 0.f};
    return two_sum(mr, -m) * Pair{T.hi, T.lo} + (log_sum(Sr) + -log_sum(S));
  }
};

struct Slope {
  float ref, coef;   // other tokens: coef 2^((z - ref) sc)
  float top, share;  // listed ones: wT (share 2^((z - top) sc) - p)
  float wT;
};

__device__ __forceinline__ Slope slope_of(const Sums& s, const Target& tg, const Scale& T, float w) {
  const float rest = rest_of(tg, s.none()), P = tg.sum + rest;
  Slope k;
  k.wT = w * T.hi;
  k.ref = s.none() ? 0.f : s.mr;
  k.coef = s.none() ? 0.f : k.wT * (P * expf(value_of(s.ln_u(T))) - rest) / s.Sr;
  k.top = s.m;
  k.share = P / s.S;
  return k;
}

// Gradient over the groups [g0, g1) of a row: of the other tokens, then that of the listed ones over it.
template <typename T>
__device__ __forceinline__ void write_gradient(const DistillParams& p, const RowView<T>& row, T* out, int g0, int g1,
                                               const Slope& k, const Target& tg) {
  const int tid = threadIdx.x, NT = blockDim.x;
  const int v_lo = max(0, row.first(g0)), v_hi = min(row.V, row.first(g1));
  if (p.vec) {
    char* to = reinterpret_cast<char*>(reinterpret_cast<uintptr_t>(out) & ~uintptr_t(31));
    const float2 sc2 = make_float2(p.T.sc, p.T.sc), ref2 = make_float2(-k.ref, -k.ref), c2 = make_float2(k.coef, k.coef);
    for (int gb = g0 + tid; gb < g1; gb += NT * kBatch) {
      Raw x[kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int g = gb + u * NT;
        if (g < g1 && row.whole(g)) x[u] = load_raw(row.base + (size_t)g * 32);
      }
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int g = gb + u * NT;
        if (g >= g1) continue;
        if (row.whole(g)) {
          Raw y;
#pragma unroll
          for (int i = 0; i < kGroup<T> / 2; ++i) {
            const float2 a = mul2(add2(pair_of<T>(x[u], i), ref2), sc2);
            put_pair<T>(y, i, mul2(make_float2(ex2(a.x), ex2(a.y)), c2));
          }
          store_raw(to + (size_t)g * 32, y);
        } else {
          for (int e = 0; e < kGroup<T>; ++e) {
            const int v = row.first(g) + e;
            if (v >= 0 && v < row.V)
              out[v] = Elem<T>::from_f32(ex2((load_element(row.row + v) - k.ref) * p.T.sc) * k.coef);
          }
        }
      }
    }
  } else {
    for (int v = v_lo + tid; v < v_hi; v += NT)
      out[v] = Elem<T>::from_f32(ex2((load_element(row.row + v) - k.ref) * p.T.sc) * k.coef);
  }
  __syncthreads();
  for (int j = tid; j < p.K; j += NT) {
    const int v = tg.token[j];
    if (v >= v_lo && v < v_hi) out[v] = Elem<T>::from_f32(k.wT * (k.share * ex2((tg.z[j] - k.top) * p.T.sc) - tg.p[j]));
  }
}

template <typename T>
__device__ __forceinline__ void write_zeros(const DistillParams& p, const RowView<T>& row, T* out, int g0, int g1) {
  const int tid = threadIdx.x, NT = blockDim.x;
  const int v_lo = max(0, row.first(g0)), v_hi = min(row.V, row.first(g1));
  if (p.vec) {
    char* to = reinterpret_cast<char*>(reinterpret_cast<uintptr_t>(out) & ~uintptr_t(31));
    Raw zero;
#pragma unroll
    for (int i = 0; i < 8; ++i) zero.w[i] = 0u;
    for (int g = g0 + tid; g < g1; g += NT) {
      if (row.whole(g)) {
        store_raw(to + (size_t)g * 32, zero);
      } else {
        for (int e = 0; e < kGroup<T>; ++e) {
          const int v = row.first(g) + e;
          if (v >= 0 && v < row.V) out[v] = Elem<T>::from_f32(0.f);
        }
      }
    }
  } else {
    for (int v = v_lo + tid; v < v_hi; v += NT) out[v] = Elem<T>::from_f32(0.f);
  }
}

struct Part {
  float m, S;  // maximum and sum of the other tokens of a CTA's part
};

struct Shared {
  Target tg;
  Part part[kMaxCluster];
  float red[kLogitsThreads / 32], redS[kLogitsThreads / 32];
  Pair redL[kLogitsMaxTop / 32];
};

template <typename T, bool GRAD>
__global__ void __launch_bounds__(kLogitsThreads, 4) distill_kernel(const DistillParams p) {
  extern __shared__ uint32_t listed[];  // a bit per element of this CTA's groups: it is a listed token
  __shared__ Shared sm;
  const int tid = threadIdx.x, NT = blockDim.x, lane = tid & 31, warp = tid >> 5, nw = NT >> 5;
  const int c = p.ctas;
  const int rank = (int)blockIdx.x % c, entry = (int)blockIdx.x / c;
  if (c > 1) cluster_arrive();  // waited for before the first access to another CTA's shared memory
  pdl_wait();
  pdl_trigger();
  const float w = p.weight ? p.weight[entry] : 1.f;
  const RowView<T> row(static_cast<const T*>(p.logits) + (int64_t)entry * p.stride, p.V);
  T* out = GRAD ? static_cast<T*>(p.grad) + (int64_t)entry * p.grad_stride : nullptr;
  const int g0 = (int)((long long)row.n * rank / c), g1 = (int)((long long)row.n * (rank + 1) / c);
  if (w == 0.f) {  // not read at all
    if (rank == 0 && tid == 0) {
      p.loss[entry] = 0.f;
      if (p.stats)
        for (int i = 0; i < 4; ++i) p.stats[4 * (size_t)entry + i] = 0.f;
    }
    if (GRAD) write_zeros<T>(p, row, out, g0, g1);
    if (c > 1) cluster_wait();
    return;
  }

  // ------------------------------------------------------------ the target
  Target& tg = sm.tg;
  const int words = ((g1 - g0) * kGroup<T> + 31) / 32;
  for (int i = tid; i < words; i += NT) listed[i] = 0u;
  load_target(p, entry, rank == 0, tg);
  __syncthreads();
  const int at0 = row.first(g0);
  for (int j = tid; j < p.K; j += NT) {
    const int v = tg.token[j];
    if (v < 0) continue;
    tg.z[j] = load_element(row.row + v);
    const int b = v - at0;
    if (b >= 0 && b < (g1 - g0) * kGroup<T>) atomicOr(&listed[b >> 5], 1u << (b & 31));
  }
  __syncthreads();

  // ------------------------------------------------------------ the other tokens
  float m = -INFINITY, S = 0.f;
  const float2 sc2 = make_float2(p.T.sc, p.T.sc);
  for (int gb = g0 + tid; gb < g1; gb += NT * kBatch) {
    Raw x[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int g = gb + u * NT;
      if (g < g1) x[u] = row.load(g); else set_none<T>(x[u]);
    }
    float mx = -INFINITY;
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int g = gb + u * NT;
      if (g < g1) {
        const int b = (g - g0) * kGroup<T>;
        unsigned bits = listed[b >> 5] >> (b & 31) & ((1u << kGroup<T>) - 1u);
        while (bits) {
          drop_element<T>(x[u], __ffs(bits) - 1);
          bits &= bits - 1;
        }
      }
      mx = fmaxf(mx, group_max<T>(x[u]));
    }
    if (mx > m) {
      S *= ex2(shift_of(m, mx, p.T.sc));
      m = mx;
    }
    const float mm = m == -INFINITY ? 0.f : m;  // nothing but -inf and NaN so far
    const float2 nm = make_float2(-mm, -mm);
    float2 S2 = make_float2(0.f, 0.f);
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
#pragma unroll
      for (int i = 0; i < kGroup<T> / 2; ++i) {
        const float2 y = mul2(add2(pair_of<T>(x[u], i), nm), sc2);
        S2 = add2(S2, make_float2(ex2(y.x), ex2(y.y)));
      }
    }
    S += S2.x + S2.y;
  }
  const float M = cta_max(m, sm.red);
  {
    const float Sw = warp_sum(ex2(shift_of(m, M, p.T.sc)) * S);
    if (lane == 0) sm.redS[warp] = Sw;
  }
  __syncthreads();
  if (tid == 0) {
    float s = 0.f;
    for (int i = 0; i < nw; ++i) s += sm.redS[i];
    sm.part[rank].m = M;
    sm.part[rank].S = s;
  }
  __syncthreads();
  if (c > 1) {
    cluster_wait();
    const int to = GRAD ? c : 1;  // the loss alone is the first CTA's
    if (tid < 2 * to && tid / 2 != rank)
      cluster_store(cluster_addr(&sm.part[rank], tid / 2) + 4 * (tid & 1),
                    reinterpret_cast<const uint32_t*>(&sm.part[rank])[tid & 1]);
    cluster_arrive();
    if (!GRAD && rank != 0) return;
    cluster_wait();
  }

  // ------------------------------------------------------------ the row's statistics
  float mr = -INFINITY;
  for (int i = 0; i < c; ++i) mr = fmaxf(mr, sm.part[i].m);
  float Sr = 0.f;
  for (int i = 0; i < c; ++i) Sr += ex2(shift_of(sm.part[i].m, mr, p.T.sc)) * sm.part[i].S;
  float mt = -INFINITY;
  for (int j = tid; j < p.K; j += NT)
    if (tg.token[j] >= 0) mt = fmaxf(mt, tg.z[j]);
  const float m_all = fmaxf(mr, cta_max(mt, sm.red));
  float st = 0.f;
  for (int j = tid; j < p.K; j += NT)
    if (tg.token[j] >= 0) st += ex2((tg.z[j] - (m_all == -INFINITY ? 0.f : m_all)) * p.T.sc);
  st = warp_sum(st);
  if (lane == 0) sm.redS[warp] = st;
  __syncthreads();
  const float shift = shift_of(mr, m_all, p.T.sc);
  float S_all = ex2(shift) * Sr;
  for (int i = 0; i < nw; ++i) S_all += sm.redS[i];
  const Sums sums = {m_all, S_all, mr, Sr};
  if (rank == 0) {
    const Pair lnS = log_sum(S_all), inv = {p.T.hi, p.T.lo};
    Pair part = {0.f, 0.f};
    for (int j = tid; j < p.K; j += NT) {
      const float pj = tg.p[j];
      if (pj > 0.f || pj != pj) {
        // ln p - ln q, a small difference of large numbers: rounded once
        const Pair q = two_sum(tg.z[j], -m_all) * inv + -lnS;
        const float d = value_of(Pair{tg.t[j], 0.f} + -q);
        part = part + Pair{pj, 0.f} * Pair{d, 0.f};
      }
    }
    if (warp < kLogitsMaxTop / 32) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1)
        part = part + Pair{__shfl_xor_sync(0xffffffffu, part.hi, o), __shfl_xor_sync(0xffffffffu, part.lo, o)};
      if (lane == 0) sm.redL[warp] = part;
    }
    __syncthreads();
    if (tid == 0) {
      const float rest = rest_of(tg, sums.none()), P = tg.sum + rest;
      Pair loss = {0.f, 0.f};
      for (int i = 0; i < min(nw, kLogitsMaxTop / 32); ++i) loss = loss + sm.redL[i];
      if (rest > 0.f) loss = loss + Pair{rest, 0.f} * Pair{value_of(Pair{logf(rest), 0.f} + -sums.ln_u(p.T)), 0.f};
      float l = w * value_of(loss);
      if (S_all != S_all) l = S_all;
      if (sums.empty()) l = P == 0.f ? 0.f : w * INFINITY;  // no token of the target has a chance
      p.loss[entry] = l;
      if (p.stats) {
        float* to = p.stats + 4 * (size_t)entry;
        to[0] = m_all;
        to[1] = S_all;
        to[2] = mr;
        to[3] = Sr;
      }
    }
  }
  if (GRAD) {
    if (sums.empty())
      write_zeros<T>(p, row, out, g0, g1);
    else
      write_gradient<T>(p, row, out, g0, g1, slope_of(sums, tg, p.T, w), tg);
  }
}

template <typename T>
__global__ void __launch_bounds__(kLogitsThreads, 4) distill_backward_kernel(const DistillParams p) {
  __shared__ Target tg;
  const int tid = threadIdx.x, NT = blockDim.x;
  const int c = p.ctas;
  const int rank = (int)blockIdx.x % c, entry = (int)blockIdx.x / c;
  pdl_wait();
  pdl_trigger();
  const float w = p.weight ? p.weight[entry] : 1.f;
  const RowView<T> row(static_cast<const T*>(p.logits) + (int64_t)entry * p.stride, p.V);
  T* out = static_cast<T*>(p.grad) + (int64_t)entry * p.grad_stride;
  const int g0 = (int)((long long)row.n * rank / c), g1 = (int)((long long)row.n * (rank + 1) / c);
  if (w == 0.f) {
    write_zeros<T>(p, row, out, g0, g1);
    return;
  }
  load_target(p, entry, rank == 0, tg);
  __syncthreads();
  const int v_lo = max(0, row.first(g0)), v_hi = min(row.V, row.first(g1));
  for (int j = tid; j < p.K; j += NT) {
    const int v = tg.token[j];
    tg.z[j] = v >= v_lo && v < v_hi ? load_element(row.row + v) : 0.f;  // others belong to other CTAs
  }
  __syncthreads();
  const float* from = p.stats_in + 4 * (size_t)entry;
  const Sums sums = {from[0], from[1], from[2], from[3]};
  const float up = p.grad_loss ? p.grad_loss[entry] : 1.f;
  if (sums.empty())
    write_zeros<T>(p, row, out, g0, g1);
  else
    write_gradient<T>(p, row, out, g0, g1, slope_of(sums, tg, p.T, w * up), tg);
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
    p.vec = (((uintptr_t)a->logits ^ (uintptr_t)a->grad) & 31u) == 0 &&
            (a->n == 1 || ((uint64_t)(p.stride - p.grad_stride) * es) % 32 == 0);
  }
  return SSV_OK;
}

template <typename T>
cudaError_t distill_launch(const DistillParams& p, int n, const RowSplit& sp, cudaStream_t st) {
  const size_t smem = ((size_t)sp.groups * kGroup<T> + 31) / 32 * 4;
  return p.grad ? launch_rows(distill_kernel<T, true>, n, sp, smem, st, p)
                : launch_rows(distill_kernel<T, false>, n, sp, smem, st, p);
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
  const RowSplit sp = split_rows(a->n, a->V, a->dtype == SSV_BF16 ? 2 : 4);
  p.ctas = sp.ctas;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = a->dtype == SSV_BF16 ? distill_launch<__nv_bfloat16>(p, a->n, sp, st)
                                             : distill_launch<float>(p, a->n, sp, st);
  return e == cudaSuccess ? SSV_OK : SSV_ERR_CUDA;
}

extern "C" ssv_status ssv_distill_backward(const ssv_distill_args* a, void* stream) {
  using namespace ssv;
  DistillParams p;
  const ssv_status s = distill_check(a, p);
  if (s != SSV_OK) return s;
  if (a->n == 0) return SSV_OK;
  if (!a->stats || !a->grad) return SSV_ERR_INVALID;
  const RowSplit sp = split_rows(a->n, a->V, a->dtype == SSV_BF16 ? 2 : 4);
  p.ctas = sp.ctas;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = a->dtype == SSV_BF16 ? launch_rows(distill_backward_kernel<__nv_bfloat16>, a->n, sp, 0, st, p)
                                             : launch_rows(distill_backward_kernel<float>, a->n, sp, 0, st, p);
  return e == cudaSuccess ? SSV_OK : SSV_ERR_CUDA;
}
