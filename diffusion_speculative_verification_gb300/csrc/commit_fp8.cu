// ssv_commit_fp8: commit of a verification pass into an e4m3 paged cache.
//
// Which rows are appended and where is ssv_commit's rule (SimSD summary,
// section 4 "Speculative decoding pipeline").  Per touched (page, head), K and
// V apart, with X the rows appended to the page:
//   s = 2^e, e smallest with max |X| <= 448 2^e;  s = max(s_old, s) if the page
//   already holds rows of the sequence;  codes = rn_e4m3(X / s), and the rows
//   already there become rn_e4m3(code * s_old / s) when s grew.
//
// Work: one CTA per (chunk of packed rows, groups of heads of K or V).  A page is
// led by the first token appended to it; the tokens' append indices i < N + n_acc
// are counted along the packed rows from q_off, so a chunk holds one leader per
// page boundary or sequence start in it, and the number of CTAs follows from
// total_rows alone, however ragged the batch.
// Per leader, page_size / 16 warps take one (page, head): sixteen rows each, in
// registers between the maximum and the rounding, so that each element is read
// once and each code written once.  Groups of one chunk are neighbours in the
// grid: together they read whole packed rows.
//
// Bound: for prompts, HBM and the instructions around it.  4 x 8192 rows of 8
// heads of 128, bf16: 38.5 us, 5.2 TB/s of the 6.8 TB/s that a copy reaches;
// maxima taken on the integer bits two at a time, the addresses of whole prompt
// pages stepped, and the look-ups shared by two groups took it there from 61 us.
// For a decode pass, latency (sequences; table and stage map; rows: three
// dependent rounds): 5 us for 16 sequences, which is why a CTA's warps serve
// different heads of the same page.
#include "ssv_internal.cuh"
#include "paged.cuh"

#include <math.h>

namespace ssv {
namespace {

constexpr int kC8Threads = 256;
// A CTA takes several groups of heads of its chunk, one after the other, while that many CTAs remain: three rounds of
// four per SM.  A prompt of 4 x 8192 rows, 8 heads: 38.5 us with two groups per CTA, 43 us with one or four.
// A chunk is a page's rows, or fewer (16 at least) while the CTAs stay within one per SM: pages are written one after the
// other in a CTA.  11 sequences of one head, pages of 128: 15.8 us with chunks of a page, 7.1 us so.
constexpr int kC8Few = 152;
constexpr int kC8Ctas = 3 * 4 * 152;
constexpr int kScaleMin = -100;  // exponent of an all-zero page's scale

struct Commit8Params {
  const uint8_t *k_new, *v_new;
  uint8_t *k_cache, *v_cache;
  float *k_scale, *v_scale;
  const int32_t* pages;
  const ssv_seq* seqs;
  const int32_t *tau, *n_acc, *cache_len;
  int32_t *new_len, *dev_status;
  int64_t k_stride, v_stride;  // bytes
  int Hkv, ps_log2, n_pages, table_len, batch, total_rows, total_slots, max_new, max_block, chunk_rows, chunks, groups, ctas_y;
};

// The checks of sequence s that need no loop, na its accepted stages.
__device__ __forceinline__ bool commit8_sizes(const Commit8Params& p, const ssv_seq& s, int na) {
  const int B = s.block, N = s.new_len, C = s.cache_len;
  if (B < 1 || B > 64 || B > p.max_block || N < 0 || N > p.max_new || C < 0 || na < 0 || na > B) return false;
  if (s.tau_off < 0 || (long long)s.tau_off + B > p.total_slots) return false;
  if (s.q_off < 0 || (long long)s.q_off + N + 2LL * B > p.total_rows) return false;
  const long long len = (long long)C + N + na, pages = (len + (1 << p.ps_log2) - 1) >> p.ps_log2;
  return len <= 0x7fffffffLL && s.kv_off >= 0 && s.kv_off + pages <= p.table_len;
}

// Whether lane `first` of `step` sees a bad page among the touched ones.
__device__ __forceinline__ bool commit8_bad_page(const Commit8Params& p, const ssv_seq& s, int na, int first, int step) {
  const int app = s.new_len + na;
  if (app == 0) return false;
  const int j1 = (s.cache_len + app - 1) >> p.ps_log2;
  bool bad = false;
  for (int j = (s.cache_len >> p.ps_log2) + first; j <= j1; j += step) {
    const int page = p.pages[s.kv_off + j];
    bad |= page < 0 || page >= p.n_pages;
  }
  return bad;
}

// bits of 2^e with e the smallest integer >= kScaleMin such that amax <= 448 * 2^e
__device__ __forceinline__ float scale_for(float amax) {
  if (!(amax > 0.f)) return exp2f((float)kScaleMin);
  int x;
  const float f = frexpf(amax, &x);  // amax = f 2^x, 448 = 0.875 * 2^9
  return ldexpf(1.f, max(x - (f <= 0.875f ? 9 : 8), kScaleMin));
}

// sixteen bytes of fresh elements, as the integers of their bits
template <typename T> struct Bits;
template <> struct Bits<float> {
  static constexpr uint32_t kInf = 0x7f800000u;
  static __device__ __forceinline__ uint32_t max4(uint32_t top, const uint4& x) {
    return max(max(max(top, x.x & 0x7fffffffu), x.y & 0x7fffffffu), max(x.z & 0x7fffffffu, x.w & 0x7fffffffu));
  }
  static __device__ __forceinline__ uint32_t max4_finite(uint32_t top, uint4& x) {
    uint32_t* w = &x.x;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if ((w[e] & 0x7fffffffu) >= kInf) w[e] = 0x7fc00000u;
      else top = max(top, w[e] & 0x7fffffffu);
    }
    return top;
  }
  static __device__ __forceinline__ uint32_t largest(uint32_t top) { return top; }
  static __device__ __forceinline__ float value(uint32_t bits) { return __uint_as_float(bits); }
  static __device__ __forceinline__ void pair(const uint32_t* w, int e, float& lo, float& hi) {
    lo = __uint_as_float(w[2 * e]);
    hi = __uint_as_float(w[2 * e + 1]);
  }
};
template <> struct Bits<__nv_bfloat16> {  // two to a word
  static constexpr uint32_t kInf = 0x7f80u;
  static __device__ __forceinline__ uint32_t max4(uint32_t top, const uint4& x) {
    return __vmaxu2(__vmaxu2(__vmaxu2(top, x.x & 0x7fff7fffu), x.y & 0x7fff7fffu),
                    __vmaxu2(x.z & 0x7fff7fffu, x.w & 0x7fff7fffu));
  }
  static __device__ __forceinline__ uint32_t max4_finite(uint32_t top, uint4& x) {
    uint32_t* w = &x.x;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if ((w[e] & 0x7fffu) >= kInf) w[e] = (w[e] & 0xffff0000u) | 0x7fc0u;
      else top = __vmaxu2(top, w[e] & 0x7fffu);
      if ((w[e] >> 16 & 0x7fffu) >= kInf) w[e] = (w[e] & 0xffffu) | 0x7fc00000u;
      else top = __vmaxu2(top, w[e] & 0x7fff0000u);
    }
    return top;
  }
  static __device__ __forceinline__ uint32_t largest(uint32_t top) { return max(top & 0xffffu, top >> 16); }
  static __device__ __forceinline__ float value(uint32_t bits) { return __uint_as_float(bits << 16); }
  static __device__ __forceinline__ void pair(const uint32_t* w, int e, float& lo, float& hi) {
    lo = __uint_as_float(w[e] << 16);
    hi = __uint_as_float(w[e] & 0xffff0000u);
  }
};

template <typename T, int D>
__global__ void __launch_bounds__(kC8Threads, sizeof(T) == 2 ? 4 : 2) commit_fp8_kernel(const Commit8Params p) {
  constexpr int VEC = 16 / (int)sizeof(T), LANES = D / VEC;  // lanes per row
  using E = Bits<T>;
  constexpr int RPP = 32 / LANES, PASSES = 16 / RPP;         // rows per pass of a warp, passes over its sixteen
  __shared__ int2 s_lead[128];  // first row, sequence
  __shared__ int s_inv[64], s_nlead, s_na[kC8Threads];
  __shared__ float s_max[2][kC8Threads / 32];
  __shared__ ssv_seq s_seq[kC8Threads];
  pdl_wait();  // n_acc and the fresh rows may come from the kernels before this one
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, ps = 1 << p.ps_log2;
  const int chunk = blockIdx.x / p.ctas_y, group = blockIdx.x - chunk * p.ctas_y;
  if (chunk >= p.chunks) {
    // new lengths and statuses: one warp per sequence
    const int b = ((int)blockIdx.x - p.chunks * p.ctas_y) * (kC8Threads / 32) + warp;
    if (b >= p.batch) return;
    const ssv_seq s = p.seqs[b];
    const int na = p.n_acc[b];
    int bad = 0;
    if (!seq_idle(s)) {
      if (!commit8_sizes(p, s, na)) bad = SSV_ERR_INVALID;
      else if (!warp_tau_is_permutation(p.tau + s.tau_off, s.block)) bad = SSV_ERR_BAD_TAU;
      else if (__any_sync(0xffffffffu, commit8_bad_page(p, s, na, lane, 32))) bad = SSV_ERR_INVALID;
    }
    if (lane == 0) {
      if (bad) report(p.dev_status, bad);
      if (!bad && !seq_idle(s)) p.new_len[b] = s.cache_len + s.new_len + na;
      else if (p.cache_len) p.new_len[b] = p.cache_len[b];  // (which may be new_len itself)
      else p.new_len[b] = bad ? -1 : s.cache_len;
    }
    return;
  }
  // ---- leaders of this chunk's rows
  const bool table = p.batch <= kC8Threads;
  if (table && (int)threadIdx.x < p.batch) {
    s_seq[threadIdx.x] = p.seqs[threadIdx.x];
    s_na[threadIdx.x] = p.n_acc[threadIdx.x];
  }
  if (threadIdx.x == 0) s_nlead = 0;
  __syncthreads();
  if ((int)threadIdx.x < p.chunk_rows) {
    const int row = chunk * p.chunk_rows + threadIdx.x;
    const int b = row < p.total_rows ? find_seq_by_row(table ? s_seq : p.seqs, p.batch, row) : -1;
    if (b >= 0) {
      const ssv_seq s = table ? s_seq[b] : p.seqs[b];
      const int i = row - s.q_off;
      const int na = table ? s_na[b] : p.n_acc[b];
      if (!seq_idle(s) && commit8_sizes(p, s, na) && i < s.new_len + na &&
          (i == 0 || ((s.cache_len + i) & (ps - 1)) == 0))
        s_lead[atomicAdd(&s_nlead, 1)] = make_int2(row, b);
    }
  }
  __syncthreads();
  const int nlead = s_nlead;
  // this warp: rows [16 part, 16 part + 16) of head `head` of K or V
  const int parts = ps >> 4, per_cta = (kC8Threads / 32) / parts, part = warp & (parts - 1);
  const int r0 = part * 16 + lane / LANES, c = lane % LANES;  // of the appended rows
  int turn = 0;
  for (int l = 0; l < nlead; ++l) {
    const int row = s_lead[l].x, b = s_lead[l].y;
    const ssv_seq s = table ? s_seq[b] : p.seqs[b];
    const int N = s.new_len, B = s.block, na = table ? s_na[b] : p.n_acc[b], i0 = row - s.q_off;
    const int t0 = s.cache_len + i0, o0 = t0 & (ps - 1);            // first appended row of the page
    const int n = min(ps - o0, N + na - i0);                        // rows appended to it
    const int page = p.pages[s.kv_off + (t0 >> p.ps_log2)];
    // the whole sequence is good, or nothing of it is written
    int bad = commit8_bad_page(p, s, na, threadIdx.x, kC8Threads);
    if (warp == 0) bad |= !warp_tau_is_permutation(p.tau + s.tau_off, B);
    int stage = 0;
    if ((int)threadIdx.x < B) stage = p.tau[s.tau_off + threadIdx.x];
    if (__syncthreads_or(bad)) continue;
    if ((int)threadIdx.x < B) s_inv[stage - 1] = threadIdx.x;  // slot of each stage
    __syncthreads();
    // sixteen rows in order, as in all of a prompt but its ends: the addresses step
    const bool prompt = part * 16 + 16 <= min(n, N - i0);
    for (int y = group; y < p.groups; y += p.ctas_y, turn ^= 1) {
      const int unit = y * per_cta + warp / parts;
      const bool mine = unit < 2 * p.Hkv, is_v = unit >= p.Hkv;
      const int head = is_v ? unit - p.Hkv : unit;
      const int64_t at = (int64_t)page * p.Hkv + head;
      uint8_t* cache = (is_v ? p.v_cache : p.k_cache) + at * ps * D;
      float* scale = (is_v ? p.v_scale : p.k_scale) + at;
      uint4 x[PASSES];
      float s_old = 0.f, amax = 0.f;
      if (mine) {
        const int64_t stride = is_v ? p.v_stride : p.k_stride;
        const uint8_t* fresh = (is_v ? p.v_new : p.k_new) + (int64_t)head * D * sizeof(T) + c * 16 + s.q_off * stride;
        if (o0 > 0) s_old = *scale;
        if (prompt) {
          fresh += (i0 + r0) * stride;
#pragma unroll
          for (int k = 0; k < PASSES; ++k) {
            x[k] = __ldcs(reinterpret_cast<const uint4*>(fresh));
            fresh += RPP * stride;
          }
        } else {
#pragma unroll
          for (int k = 0; k < PASSES; ++k) {
            const int r = r0 + k * RPP;
            if (r >= n) continue;
            const int i = i0 + r;
            x[k] = *reinterpret_cast<const uint4*>(fresh + (i < N ? i : N + s_inv[i - N]) * stride);
          }
        }
        // magnitudes as integers, which order alike; what is not finite lies above kInf
        uint32_t top = 0;
#pragma unroll
        for (int k = 0; k < PASSES; ++k) {
          if (r0 + k * RPP < n) top = E::max4(top, x[k]);
        }
        if (E::largest(top) >= E::kInf) {  // rare: such elements become NaN and do not count
          top = 0;
#pragma unroll
          for (int k = 0; k < PASSES; ++k) {
            if (r0 + k * RPP < n) top = E::max4_finite(top, x[k]);
          }
        }
        amax = E::value(E::largest(top));
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        if (lane == 0) s_max[turn][warp] = amax;
      }
      __syncthreads();  // (every warp of the page has read its old scale, too)
      if (mine) {
        for (int w = 0; w < parts; ++w) amax = fmaxf(amax, s_max[turn][warp - part + w]);
        const float sc = fmaxf(scale_for(amax), s_old);
        const float inv = 1.f / sc;  // a power of two, exact
#pragma unroll
        for (int k = 0; k < PASSES; ++k) {
          const int r = r0 + k * RPP;
          if (r >= n) continue;
          const uint32_t w[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
          uint16_t q[VEC / 2];
#pragma unroll
          for (int e = 0; e < VEC / 2; ++e) {
            float lo, hi;
            E::pair(w, e, lo, hi);
            q[e] = f32_to_e4m3x2(lo * inv, hi * inv);
          }
          uint8_t* dst = cache + (o0 + r) * D + c * VEC;
          if constexpr (VEC == 8) {
            *reinterpret_cast<uint2*>(dst) = make_uint2(q[0] | (uint32_t)q[1] << 16, q[2] | (uint32_t)q[3] << 16);
          } else {
            *reinterpret_cast<uint32_t*>(dst) = q[0] | (uint32_t)q[1] << 16;
          }
        }
        if (o0 > 0 && sc > s_old) {
          // the rows already there, 16 codes at a time
          const float ratio = s_old * inv;
          for (int v = part * 32 + lane; v < o0 * D / 16; v += parts * 32) {
            const uint4 raw = reinterpret_cast<const uint4*>(cache)[v];
            uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              uint32_t out = 0;
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const uint32_t f2 = e4m3x2_to_f16x2((uint16_t)(w[e] >> (16 * h)));
                const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&f2));
                out |= (uint32_t)f32_to_e4m3x2(f.x * ratio, f.y * ratio) << (16 * h);
              }
              w[e] = out;
            }
            reinterpret_cast<uint4*>(cache)[v] = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
        if (part == 0 && lane == 0) *scale = sc;
      }
    }
    __syncthreads();  // s_inv is reused
  }
}

}  // namespace
}  // namespace ssv

extern "C" ssv_status ssv_commit_fp8(const ssv_commit_fp8_args* a, void* stream) {
  using namespace ssv;
  if (!a) return SSV_ERR_INVALID;
  if (a->batch < 0 || a->total_rows < 0 || a->total_slots < 0 || a->table_len < 0 || a->n_pages < 0 || a->Hkv <= 0 ||
      a->max_new < 0 || a->max_block < 1 || a->max_block > 64 || !page_size_ok(a->page_size))
    return SSV_ERR_INVALID;
  if (a->dtype != SSV_F32 && a->dtype != SSV_BF16) return SSV_ERR_INVALID;
  if (a->d != 64 && a->d != 128) return SSV_ERR_UNSUPPORTED;
  if (a->batch == 0) return SSV_OK;
  if (!a->seqs || !a->n_acc || !a->new_len) return SSV_ERR_INVALID;
  if (a->total_rows > 0 && (!a->k_new || !a->v_new || !a->tau)) return SSV_ERR_INVALID;
  if ((a->n_pages > 0 && (!a->k_cache || !a->v_cache || !a->k_scale || !a->v_scale)) || (a->table_len > 0 && !a->pages))
    return SSV_ERR_INVALID;
  if (a->Hkv > 32767 || (long long)a->n_pages * a->page_size > 0x7fffffffLL) return SSV_ERR_INVALID;
  const int64_t es = a->dtype == SSV_BF16 ? 2 : 4, width = (int64_t)a->Hkv * a->d;
  const int64_t ks = a->k_stride ? a->k_stride : width, vs = a->v_stride ? a->v_stride : width;
  if (ks < width || vs < width) return SSV_ERR_INVALID;
  const uintptr_t al = (uintptr_t)a->k_new | (uintptr_t)a->v_new | (uintptr_t)a->k_cache | (uintptr_t)a->v_cache |
                       (uintptr_t)(ks * es) | (uintptr_t)(vs * es);
  if (al & 15u) return SSV_ERR_INVALID;
  const int per_cta = (kC8Threads / 32) / (a->page_size / 16);  // heads of K or V per CTA
  Commit8Params p{static_cast<const uint8_t*>(a->k_new), static_cast<const uint8_t*>(a->v_new),
                  static_cast<uint8_t*>(a->k_cache), static_cast<uint8_t*>(a->v_cache), a->k_scale, a->v_scale,
                  a->pages, a->seqs, a->tau, a->n_acc, a->cache_len, a->new_len, a->dev_status, ks * es, vs * es, a->Hkv,
                  ilog2(a->page_size), a->n_pages, a->table_len, a->batch, a->total_rows, a->total_slots, a->max_new,
                  a->max_block, 16, 0, (2 * a->Hkv + per_cta - 1) / per_cta, 0};
  for (;; p.chunk_rows *= 2) {
    p.chunks = (int)(((long long)a->total_rows + p.chunk_rows - 1) / p.chunk_rows);
    if (p.chunk_rows == a->page_size || (long long)p.chunks * p.groups <= kC8Few) break;
  }
  const long long turns = (long long)p.chunks * p.groups / kC8Ctas;
  p.ctas_y = p.groups / (turns < 1 ? 1 : turns > p.groups ? p.groups : (int)turns);
  const long long ctas = (long long)p.chunks * p.ctas_y + (a->batch + 7) / 8;
  if (ctas > 0x7fffffffLL) return SSV_ERR_INVALID;
  const dim3 grid((unsigned)ctas);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (a->dtype == SSV_BF16)
    e = a->d == 128 ? launch_pdl(commit_fp8_kernel<__nv_bfloat16, 128>, grid, dim3(kC8Threads), 0, st, p)
                    : launch_pdl(commit_fp8_kernel<__nv_bfloat16, 64>, grid, dim3(kC8Threads), 0, st, p);
  else
    e = a->d == 128 ? launch_pdl(commit_fp8_kernel<float, 128>, grid, dim3(kC8Threads), 0, st, p)
                    : launch_pdl(commit_fp8_kernel<float, 64>, grid, dim3(kC8Threads), 0, st, p);
  return e == cudaSuccess ? SSV_OK : SSV_ERR_CUDA;
}
