// ssv_verify_attn_fp8: verification attention over cached keys in e4m3 pages.
//
// One warp per (query row, query head), fp32 throughout, online softmax in
// the log2 domain.  SimSD summary, section 2: the temporal mask is evaluated
// from tau for the 2B tail keys.
#include "ssv_internal.cuh"
#include "paged.cuh"

#include <math.h>

namespace ssv {
namespace {

struct AttnFp8Params {
  const __nv_bfloat16* q;
  const uint8_t *k_cache, *v_cache;
  const float *k_scale, *v_scale;
  const int32_t* pages;
  const __nv_bfloat16 *k_new, *v_new;
  __nv_bfloat16* o;
  int64_t k_stride, v_stride;  // elements
  int Hq, Hkv, ps_log2, n_pages, table_len;
  float scale;
  const ssv_seq* seqs;
  int batch;
  const int32_t* tau;
  int total_rows, total_slots, max_cache, max_new, max_block;
  int32_t* dev_status;
};

// Extents of sequence s within the call's buffers and stated maxima.
__device__ __forceinline__ bool fp8_seq_ok(const AttnFp8Params& p, const ssv_seq& s) {
  const long long pages = ((long long)s.cache_len + (1 << p.ps_log2) - 1) >> p.ps_log2;
  return s.cache_len >= 0 && s.new_len >= 0 && s.block >= 1 && s.block <= 64 && s.q_off >= 0 &&
         (long long)s.q_off + s.new_len + 2LL * s.block <= p.total_rows && s.kv_off >= 0 &&
         s.kv_off + pages <= p.table_len && s.tau_off >= 0 && (long long)s.tau_off + s.block <= p.total_slots &&
         s.cache_len <= p.max_cache && s.new_len <= p.max_new && s.block <= p.max_block;
}

constexpr int kRowWarps = 4;

__global__ void __launch_bounds__(kRowWarps * 32) attn_fp8_row_kernel(const AttnFp8Params p) {
  constexpr int D = 128, E = 4, U = 4;
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const long long w = (long long)blockIdx.x * kRowWarps + (threadIdx.x >> 5);
  if (w >= (long long)p.total_rows * p.Hq) return;
  const int row = (int)(w / p.Hq), h = (int)(w % p.Hq);
  const int b = find_seq_by_row(p.seqs, p.batch, row);
  if (b < 0) return;
  const ssv_seq s = p.seqs[b];
  if (seq_idle(s)) return;
  const int i = row - s.q_off, B = s.block, N = s.new_len, C = s.cache_len;
  if (!fp8_seq_ok(p, s)) {
    if (lane == 0) report(p.dev_status, SSV_ERR_INVALID);
    return;
  }
  if (i >= N + 2 * B) return;
  const int32_t* tau = p.tau + s.tau_off;
  if (!warp_tau_is_permutation(tau, B)) {
    if (lane == 0) report(p.dev_status, SSV_ERR_BAD_TAU);
    return;
  }
  const int ps = 1 << p.ps_log2;
  bool bad = false;
  for (int j = lane; j < (C + ps - 1) >> p.ps_log2; j += 32) {
    const int page = p.pages[s.kv_off + j];
    bad |= page < 0 || page >= p.n_pages;
  }
  if (__any_sync(0xffffffffu, bad)) {
    if (lane == 0) report(p.dev_status, SSV_ERR_INVALID);
    return;
  }
  const int kvh = h / (p.Hq / p.Hkv);
  auto wide = [&](const __nv_bfloat16* x, float* out) {
    const uint2 v = *reinterpret_cast<const uint2*>(x + lane * E);
    out[0] = __uint_as_float(v.x << 16); out[1] = __uint_as_float(v.x & 0xffff0000u);
    out[2] = __uint_as_float(v.y << 16); out[3] = __uint_as_float(v.y & 0xffff0000u);
  };
  auto codes = [&](const uint8_t* x, float sc, float* out) {
    const uint32_t v = *reinterpret_cast<const uint32_t*>(x + lane * E);
    const uint32_t f01 = e4m3x2_to_f16x2((uint16_t)v), f23 = e4m3x2_to_f16x2((uint16_t)(v >> 16));
    const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&f01));
    const float2 c = __half22float2(*reinterpret_cast<const __half2*>(&f23));
    out[0] = a.x * sc; out[1] = a.y * sc; out[2] = c.x * sc; out[3] = c.y * sc;
  };
  float q[E];
  wide(p.q + ((size_t)row * p.Hq + h) * D, q);
  const float qs = p.scale * 1.4426950408889634f;
#pragma unroll
  for (int e = 0; e < E; ++e) q[e] *= qs;
  float m = -INFINITY, l = 0.f, acc[E] = {0.f, 0.f, 0.f, 0.f};
  const bool tail_row = i >= N;
  const int r = i - N, tau_r = tail_row ? tau[r % B] : 0;
  const int total = C + (tail_row ? N + 2 * B : i + 1);
  for (int j0 = 0; j0 < total; j0 += U) {
    float sc[U], vv[U][E];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int j = j0 + u;
      bool ok = j < total;
      float kk[E] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int e = 0; e < E; ++e) vv[u][e] = 0.f;
      if (ok && j < C) {
        const size_t at = (size_t)p.pages[s.kv_off + (j >> p.ps_log2)] * p.Hkv + kvh;
        const size_t off = (at * ps + (j & (ps - 1))) * D;
        codes(p.k_cache + off, p.k_scale[at], kk);
        codes(p.v_cache + off, p.v_scale[at], vv[u]);
      } else if (ok) {
        const int jn = j - C, t = jn - N;
        if (tail_row && t >= 0) ok = tail_allowed(r, t, B, tau_r, tau[t % B]);
        if (ok) {
          wide(p.k_new + (int64_t)(s.q_off + jn) * p.k_stride + kvh * D, kk);
          wide(p.v_new + (int64_t)(s.q_off + jn) * p.v_stride + kvh * D, vv[u]);
        }
      }
      float part = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) part = fmaf(q[e], kk[e], part);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) part += __shfl_xor_sync(0xffffffffu, part, o);
      sc[u] = ok ? part : -INFINITY;
    }
    float mx = m;
#pragma unroll
    for (int u = 0; u < U; ++u) mx = fmaxf(mx, sc[u]);
    if (mx == -INFINITY) continue;
    const float corr = exp2f(m - mx);
    l *= corr;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] *= corr;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const float pk = exp2f(sc[u] - mx);
      l += pk;
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] = fmaf(pk, vv[u][e], acc[e]);
    }
    m = mx;
  }
  const float inv = 1.f / l;
  const __nv_bfloat162 o01 = __floats2bfloat162_rn(acc[0] * inv, acc[1] * inv);
  const __nv_bfloat162 o23 = __floats2bfloat162_rn(acc[2] * inv, acc[3] * inv);
  *reinterpret_cast<uint2*>(p.o + ((size_t)row * p.Hq + h) * D + lane * E) =
      make_uint2(*reinterpret_cast<const uint32_t*>(&o01), *reinterpret_cast<const uint32_t*>(&o23));
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

}  // namespace
}  // namespace ssv

extern "C" ssv_status ssv_verify_attn_fp8_workspace(const ssv_attn_fp8_args* a, size_t* bytes) {
  if (!bytes) return SSV_ERR_INVALID;
  const ssv_status st = ssv::fp8_check(a);
  if (st == SSV_OK) *bytes = 256;
  return st;
}

extern "C" ssv_status ssv_verify_attn_fp8(const ssv_attn_fp8_args* a, void* ws, size_t ws_bytes, void* stream) {
  using namespace ssv;
  size_t need = 0;
  const ssv_status st = ssv_verify_attn_fp8_workspace(a, &need);
  if (st != SSV_OK) return st;
  if (a->batch == 0 || a->total_rows == 0) return SSV_OK;
  if (!ws || ((uintptr_t)ws & 255u) || ws_bytes < need) return SSV_ERR_WORKSPACE;
  const int64_t width = (int64_t)a->Hkv * a->d;
  AttnFp8Params p{static_cast<const __nv_bfloat16*>(a->q), static_cast<const uint8_t*>(a->k_cache),
                  static_cast<const uint8_t*>(a->v_cache), a->k_scale, a->v_scale, a->pages,
                  static_cast<const __nv_bfloat16*>(a->k_new), static_cast<const __nv_bfloat16*>(a->v_new),
                  static_cast<__nv_bfloat16*>(a->o), a->k_stride ? a->k_stride : width,
                  a->v_stride ? a->v_stride : width, a->Hq, a->Hkv, ilog2(a->page_size), a->n_pages, a->table_len,
                  a->scale > 0.f ? a->scale : (float)(1.0 / sqrt((double)a->d)), a->seqs, a->batch, a->tau,
                  a->total_rows, a->total_slots, a->max_cache, a->max_new, a->max_block, a->dev_status};
  const long long grid = ((long long)a->total_rows * a->Hq + kRowWarps - 1) / kRowWarps;
  if (grid > 0x7fffffffLL) return SSV_ERR_INVALID;
  const cudaError_t e = launch_pdl(attn_fp8_row_kernel, dim3((unsigned)grid), dim3(kRowWarps * 32), 0,
                                   static_cast<cudaStream_t>(stream), p);
  return e == cudaSuccess ? SSV_OK : SSV_ERR_CUDA;
}
