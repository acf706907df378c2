// ssv_norm_rope_copy: RMS norm of each query / key head and the RoPE-copy
// rotation in one pass.
//
//   y = x / sqrt(mean(x^2) + eps) * w;  (y_i, y_{i+d/2}) turned by pos * theta_i
//
// The CHUNKS = (d/2) / VEC lanes that hold a head (16 bytes of either half
// each) sum its squares with shuffles; nothing else couples the elements, so
// each is read and written once.  Positions as ssv_rope_copy (SimSD summary,
// section 3 "Position Encoding Alignment").
//
// Angles: theta_i / (2 pi) is given as a 64-bit fixed-point fraction F_i of a
// turn; pos * F_i mod 2^64 is the angle mod one turn exactly, in one integer
// multiplication (the fp64 pipe of this part is far slower).  Error: that of F_i,
// at most 3 * 2^-53, times pos -- 6e-9 turns at position 2^24 -- and the
// rounding of the fraction to fp32.
//
// Bound by HBM.  A lane holds one 16-byte chunk of either half; the lanes of a
// warp are 32 / CHUNKS rows of one head, so that a lane's cosines, sines and
// weights serve all heads of its row, and a CTA's eight warps take every eighth
// head.  In a small batch (fewer rows than fill the SMs) a CTA has one row, and a
// warp 32 / CHUNKS heads of it.  The first loads are issued before the positions
// are known.
//
// Measured: 4 x 8192 rows of 32 + 8 heads of 128, bf16, out of a fused projection:
// 120 us, 5.6 TB/s of the 6.8 TB/s that a copy reaches (158 us with one head per
// warp); 37 ragged sequences, fp32, heads of 64: 13.1 us, 4.7 TB/s of little more
// than one wave of CTAs; 8 sequences of 16 rows: 3.5 us, latency.
#include "ssv_internal.cuh"
#include "paged.cuh"

#include <math.h>

namespace ssv {
namespace {

constexpr int kNormThreads = 256, kNormWarps = kNormThreads / 32;
// heads per thread in flight (fp32: 2 with four CTAs per SM 13.1 us in the ragged case above, 5 with three 16.2 us)
template <typename T>
constexpr int kNormPre = sizeof(T) == 2 ? 5 : 2;

struct NormTheta {
  uint64_t turn[64];  // theta_i / (2 pi) in units of 2^-64 turns
};

struct NormParams {
  const void *q_in, *k_in, *q_w, *k_w;
  void *q_out, *k_out;
  int64_t qis, kis, qos, kos;  // row strides, elements
  int Hq, Hkv, batch, total_rows;
  float eps;
  const ssv_seq* seqs;
  const int32_t* positions;
  int32_t* dev_status;
};

template <typename T> constexpr int kVec = 16 / (int)sizeof(T);

template <typename T>
__device__ __forceinline__ void widen(const uint4 raw, float* out) {
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < 4; ++i) out[i] = __uint_as_float(w[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      out[2 * i] = __uint_as_float(w[i] << 16);
      out[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
}

template <typename T>
__device__ __forceinline__ uint4 narrow(const float* v) {
  uint32_t w[4];
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = __float_as_uint(v[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Position of `row` under sequence record s: -1 if the row is to be left alone
// (reporting what is wrong with it, if anything).
__device__ __forceinline__ int row_position(const NormParams& p, const ssv_seq& s, int row) {
  const int i = row - s.q_off;
  if (seq_idle(s)) return -1;
  if (s.cache_len < 0 || s.new_len < 0 || s.block < 1 || s.block > 64 || s.q_off < 0 ||
      (long long)s.q_off + s.new_len + 2LL * s.block > p.total_rows ||
      (long long)s.cache_len + s.new_len + s.block > 0x7fffffffLL) {
    report(p.dev_status, SSV_ERR_INVALID);
    return -1;
  }
  if (i >= s.new_len + 2 * s.block) return -1;
  // a tail row takes its data row's position
  const int j = i < s.new_len ? i : s.new_len + (i - s.new_len) % s.block;
  if (!p.positions) return s.cache_len + j;
  const int pos = p.positions[s.q_off + j];
  if (pos < 0) {
    report(p.dev_status, SSV_ERR_INVALID);
    return -1;
  }
  return pos;
}

template <typename T, int D, bool kOneRow>
__global__ void __launch_bounds__(kNormThreads, sizeof(T) == 2 ? 2 : 4)
norm_rope_kernel(const NormParams p, const __grid_constant__ NormTheta th) {
  constexpr int HALF = D / 2, VEC = kVec<T>, CHUNKS = HALF / VEC, GROUPS = 32 / CHUNKS;
  constexpr int ROWS = kOneRow ? 1 : GROUPS;
  constexpr int STEP = kOneRow ? kNormWarps * GROUPS : kNormWarps;  // heads between two of a lane's
  __shared__ __align__(16) float s_cos[ROWS][HALF], s_sin[ROWS][HALF];
  __shared__ int s_pos[ROWS];
  __shared__ ssv_seq s_seq[kNormThreads];
  pdl_wait();  // the rows come from the kernel before this one
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, ch = lane % CHUNKS, g = lane / CHUNKS;
  const int row0 = blockIdx.x * ROWS, lr = kOneRow ? 0 : g, heads = p.Hq + p.Hkv;
  const int64_t row = row0 + lr;
  const bool here = row < p.total_rows;
  const int head0 = kOneRow ? warp * GROUPS + g : warp;
  auto in_at = [&](int hh) -> const T* {
    return (hh < p.Hq ? static_cast<const T*>(p.q_in) + row * p.qis + hh * D
                      : static_cast<const T*>(p.k_in) + row * p.kis + (hh - p.Hq) * D) + ch * VEC;
  };
  auto out_at = [&](int hh) -> T* {
    return (hh < p.Hq ? static_cast<T*>(p.q_out) + row * p.qos + hh * D
                      : static_cast<T*>(p.k_out) + row * p.kos + (hh - p.Hq) * D) + ch * VEC;
  };
  uint4 ra[kNormPre<T>], rb[kNormPre<T>];
  auto fetch = [&](int h0) {
#pragma unroll
    for (int k = 0; k < kNormPre<T>; ++k) {
      const int hh = h0 + k * STEP;
      if (here && hh < heads) {
        const T* x = in_at(hh);
        ra[k] = *reinterpret_cast<const uint4*>(x);
        rb[k] = *reinterpret_cast<const uint4*>(x + HALF);
      } else {
        ra[k] = rb[k] = make_uint4(0, 0, 0, 0);
      }
    }
  };
  fetch(head0);
  const T *wq = static_cast<const T*>(p.q_w) + ch * VEC, *wk = static_cast<const T*>(p.k_w) + ch * VEC;
  // plain loads, which stay behind the wait above: the kernel before may write the weights, too
  const uint4 wq1 = *reinterpret_cast<const uint4*>(wq), wq2 = *reinterpret_cast<const uint4*>(wq + HALF);
  const uint4 wk1 = *reinterpret_cast<const uint4*>(wk), wk2 = *reinterpret_cast<const uint4*>(wk + HALF);
  const bool table = p.batch <= kNormThreads;
  if (table && threadIdx.x < p.batch) s_seq[threadIdx.x] = p.seqs[threadIdx.x];
  __syncthreads();
  if (threadIdx.x < ROWS) {
    const int r = row0 + threadIdx.x;
    int pos = -1;
    if (r < p.total_rows) {
      const int b = find_seq_by_row(table ? s_seq : p.seqs, p.batch, r);
      if (b >= 0) pos = row_position(p, table ? s_seq[b] : p.seqs[b], r);
    }
    s_pos[threadIdx.x] = pos;
  }
  __syncthreads();
  for (int t = threadIdx.x; t < ROWS * HALF; t += kNormThreads) {
    const int r = t / HALF, i = t % HALF;
    // the angle mod one turn, as a signed fraction of half a turn
    const uint64_t a = (uint64_t)(uint32_t)max(s_pos[r], 0) * th.turn[i];
    sincospif((float)(int32_t)(a >> 32) * 0x1p-31f, &s_sin[r][i], &s_cos[r][i]);
  }
  __syncthreads();
  const bool live = here && s_pos[lr] >= 0;
  float c[VEC], s[VEC];
#pragma unroll
  for (int v = 0; v < VEC; v += 4) {
    *reinterpret_cast<float4*>(c + v) = *reinterpret_cast<const float4*>(&s_cos[lr][ch * VEC + v]);
    *reinterpret_cast<float4*>(s + v) = *reinterpret_cast<const float4*>(&s_sin[lr][ch * VEC + v]);
  }
#pragma unroll 1
  for (int h0 = head0; h0 - head0 < heads; h0 += kNormPre<T> * STEP) {
    if (h0 != head0) fetch(h0);
#pragma unroll
    for (int k = 0; k < kNormPre<T>; ++k) {
      const int hh = h0 + k * STEP;
      float x1[VEC], x2[VEC], w1[VEC], w2[VEC], ss = 0.f;
      widen<T>(ra[k], x1);
      widen<T>(rb[k], x2);
#pragma unroll
      for (int v = 0; v < VEC; ++v) ss = fmaf(x1[v], x1[v], fmaf(x2[v], x2[v], ss));
#pragma unroll
      for (int o = CHUNKS / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      if (!live || hh >= heads) continue;
      const float r = 1.f / sqrtf(ss * (1.f / D) + p.eps);
      widen<T>(hh < p.Hq ? wq1 : wk1, w1);
      widen<T>(hh < p.Hq ? wq2 : wk2, w2);
#pragma unroll
      for (int v = 0; v < VEC; ++v) {
        const float y1 = x1[v] * r * w1[v], y2 = x2[v] * r * w2[v];
        x1[v] = y1 * c[v] - y2 * s[v];
        x2[v] = y2 * c[v] + y1 * s[v];
      }
      T* o = out_at(hh);
      *reinterpret_cast<uint4*>(o) = narrow<T>(x1);
      *reinterpret_cast<uint4*>(o + HALF) = narrow<T>(x2);
    }
  }
}

template <typename T, int D>
cudaError_t launch_norm(const NormParams& p, const NormTheta& th, cudaStream_t st) {
  constexpr int ROWS = 32 / (D / 2 / kVec<T>);
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  if ((long long)p.total_rows < (long long)ROWS * sms)
    return launch_pdl(norm_rope_kernel<T, D, true>, dim3(p.total_rows), dim3(kNormThreads), 0, st, p, th);
  return launch_pdl(norm_rope_kernel<T, D, false>, dim3((p.total_rows + ROWS - 1) / ROWS), dim3(kNormThreads), 0, st, p,
                    th);
}

}  // namespace
}  // namespace ssv

extern "C" ssv_status ssv_norm_rope_copy(const ssv_norm_rope_args* a, void* stream) {
  using namespace ssv;
  if (!a) return SSV_ERR_INVALID;
  if (a->total_rows < 0 || a->batch < 0 || a->Hq <= 0 || a->Hkv <= 0) return SSV_ERR_INVALID;
  if (a->total_rows == 0 || a->batch == 0) return SSV_OK;
  if (!a->q_in || !a->k_in || !a->q_out || !a->k_out || !a->q_weight || !a->k_weight || !a->seqs)
    return SSV_ERR_INVALID;
  if (a->d != 64 && a->d != 128) return SSV_ERR_UNSUPPORTED;
  if (a->dtype != SSV_F32 && a->dtype != SSV_BF16) return SSV_ERR_INVALID;
  if (!(a->base > 1.0) || !isfinite(a->base) || !(a->eps >= 0.f) || !isfinite(a->eps)) return SSV_ERR_INVALID;
  if (((long long)a->Hq + a->Hkv) * a->d > 0x3fffffffLL) return SSV_ERR_INVALID;
  const int64_t es = a->dtype == SSV_BF16 ? 2 : 4, qw = (int64_t)a->Hq * a->d, kw = (int64_t)a->Hkv * a->d;
  NormParams p{a->q_in, a->k_in, a->q_weight, a->k_weight, a->q_out, a->k_out,
               a->q_in_stride ? a->q_in_stride : qw, a->k_in_stride ? a->k_in_stride : kw,
               a->q_out_stride ? a->q_out_stride : qw, a->k_out_stride ? a->k_out_stride : kw,
               a->Hq, a->Hkv, a->batch, a->total_rows, a->eps, a->seqs, a->positions, a->dev_status};
  if (p.qis < qw || p.qos < qw || p.kis < kw || p.kos < kw) return SSV_ERR_INVALID;
  const uintptr_t al = (uintptr_t)a->q_in | (uintptr_t)a->k_in | (uintptr_t)a->q_out | (uintptr_t)a->k_out |
                       (uintptr_t)a->q_weight | (uintptr_t)a->k_weight | (uintptr_t)(p.qis * es) |
                       (uintptr_t)(p.kis * es) | (uintptr_t)(p.qos * es) | (uintptr_t)(p.kos * es);
  if (al & 15u) return SSV_ERR_INVALID;
  NormTheta th;
  // theta_i / (2 pi) by repeated products: i roundings on a theta_i that falls, at most 3 * 2^-53 turns per position
  const double ratio = pow(a->base, -2.0 / a->d);
  double turns = 0.15915494309189535;
  for (int i = 0; i < 64; ++i, turns *= ratio) th.turn[i] = i < a->d / 2 ? (uint64_t)(turns * 18446744073709551616.0) : 0;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (a->dtype == SSV_BF16)
    e = a->d == 128 ? launch_norm<__nv_bfloat16, 128>(p, th, st) : launch_norm<__nv_bfloat16, 64>(p, th, st);
  else
    e = a->d == 128 ? launch_norm<float, 128>(p, th, st) : launch_norm<float, 64>(p, th, st);
  return e == cudaSuccess ? SSV_OK : SSV_ERR_CUDA;
}
