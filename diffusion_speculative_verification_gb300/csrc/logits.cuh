// Rows of logits, as the kernels on a pass's logits read and write them
// (ssv_logprobs, ssv_distill, ssv_distill_backward).
//
// A row of V elements at any element-aligned address is cut at the 32-byte
// boundaries of memory into groups: group g holds the elements
// [g E - lead, (g + 1) E - lead), E = 32 / element size, lead the elements
// between the boundary at or below the row's start and that start.  All but the
// first and the last group lie inside the row and move as one 32-byte access;
// the edges are read element by element, and what they lack counts as -inf.
//
// A row is shared out over the CTAs of a cluster by contiguous ranges of groups;
// a CTA's threads take every NT-th group, kBatch of them in flight.
#pragma once

#include "ssv_internal.cuh"

#include <float.h>
#include <math.h>

namespace ssv {

constexpr int kLogitsThreads = 256;       // most threads of a CTA
constexpr int kLogitsMaxVocab = 1 << 19;  // largest V
constexpr int kLogitsMaxTop = 128;        // most alternatives of a row
constexpr int kBatch = 4;                 // groups in flight per thread
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.693147180559945309f;

struct Raw {  // one group
  uint32_t w[8];
};

template <typename T> constexpr int kGroup = 32 / (int)sizeof(T);

__device__ __forceinline__ Raw load_raw(const void* p) {
  Raw r;
  asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r.w[0]), "=r"(r.w[1]), "=r"(r.w[2]), "=r"(r.w[3]), "=r"(r.w[4]), "=r"(r.w[5]), "=r"(r.w[6]),
                 "=r"(r.w[7])
               : "l"(p));
  return r;
}

__device__ __forceinline__ void store_raw(void* p, const Raw& r) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(r.w[0]), "r"(r.w[1]),
               "r"(r.w[2]), "r"(r.w[3]), "r"(r.w[4]), "r"(r.w[5]), "r"(r.w[6]), "r"(r.w[7])
               : "memory");
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// the larger; NaN if either is
__device__ __forceinline__ float max_nan(float a, float b) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}

// two fp32 in one operation
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 y;
  asm("{ .reg .b64 a, b, y; mov.b64 a, {%2, %3}; mov.b64 b, {%4, %5}; add.rn.f32x2 y, a, b; mov.b64 {%0, %1}, y; }"
      : "=f"(y.x), "=f"(y.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return y;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 y;
  asm("{ .reg .b64 a, b, y; mov.b64 a, {%2, %3}; mov.b64 b, {%4, %5}; mul.rn.f32x2 y, a, b; mov.b64 {%0, %1}, y; }"
      : "=f"(y.x), "=f"(y.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return y;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 y;
  asm("{ .reg .b64 a, b, c, y; mov.b64 a, {%2, %3}; mov.b64 b, {%4, %5}; mov.b64 c, {%6, %7}; "
      "fma.rn.f32x2 y, a, b, c; mov.b64 {%0, %1}, y; }"
      : "=f"(y.x), "=f"(y.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return y;
}

// element pair i of a group
template <typename T>
__device__ __forceinline__ float2 pair_of(const Raw& r, int i) {
  if (sizeof(T) == 2) return make_float2(__uint_as_float(r.w[i] << 16), __uint_as_float(r.w[i] & 0xFFFF0000u));
  return make_float2(__uint_as_float(r.w[(2 * i) & 7]), __uint_as_float(r.w[(2 * i + 1) & 7]));
}

template <typename T>
__device__ __forceinline__ void put_pair(Raw& r, int i, float2 v) {
  if (sizeof(T) == 2) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(v.x, v.y);
    r.w[i] = *reinterpret_cast<const uint32_t*>(&h);
  } else {
    r.w[(2 * i) & 7] = __float_as_uint(v.x);
    r.w[(2 * i + 1) & 7] = __float_as_uint(v.y);
  }
}

template <typename T>
__device__ __forceinline__ void set_none(Raw& r) {
#pragma unroll
  for (int i = 0; i < 8; ++i) r.w[i] = sizeof(T) == 2 ? 0xFF80FF80u : 0xFF800000u;  // -inf
}

// element e of a group becomes -inf
template <typename T>
__device__ __forceinline__ void drop_element(Raw& r, int e) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (sizeof(T) == 2) {
      if (e == 2 * i) r.w[i] = (r.w[i] & 0xFFFF0000u) | 0xFF80u;
      if (e == 2 * i + 1) r.w[i] = (r.w[i] & 0xFFFFu) | 0xFF800000u;
    } else if (e == i) {
      r.w[i] = 0xFF800000u;
    }
  }
}

// largest number of a group, -inf where there is none (NaN are passed over)
template <typename T>
__device__ __forceinline__ float group_max(const Raw& r) {
  if (sizeof(T) == 2) {
    __nv_bfloat162 h[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] = *reinterpret_cast<const __nv_bfloat162*>(&r.w[i]);
#pragma unroll
    for (int s = 4; s > 0; s >>= 1)
#pragma unroll
      for (int i = 0; i < s; ++i) h[i] = __hmax2(h[i], h[i + s]);
    return fmaxf(-INFINITY, fmaxf(__low2float(h[0]), __high2float(h[0])));
  }
  float m = -INFINITY;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = fmaxf(m, __uint_as_float(r.w[i]));
  return m;
}

// A row, cut into groups.
template <typename T>
struct RowView {
  const char* base;  // address of group 0 (32-byte boundary at or below the row)
  const T* row;
  int lead, V, n;    // n groups, those of [lo, hi) whole
  int lo, hi;

  __device__ __forceinline__ RowView(const T* p, int V_) : row(p), V(V_) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    base = reinterpret_cast<const char*>(a & ~uintptr_t(31));
    lead = (int)((a & 31) / sizeof(T));
    n = (lead + V + kGroup<T> - 1) / kGroup<T>;
    lo = lead ? 1 : 0;
    hi = (lead + V) / kGroup<T>;
  }
  __device__ __forceinline__ bool whole(int g) const { return g >= lo && g < hi; }
  __device__ __forceinline__ int first(int g) const { return g * kGroup<T> - lead; }  // element at the group's start
  __device__ __forceinline__ Raw load(int g) const {
    if (whole(g)) return load_raw(base + (size_t)g * 32);
    Raw r;
    set_none<T>(r);
    const int v0 = first(g);
#pragma unroll
    for (int e = 0; e < kGroup<T>; ++e) {
      const int v = v0 + e;
      if (v < 0 || v >= V) continue;
      if (sizeof(T) == 2) {
        const uint32_t x = *(reinterpret_cast<const volatile uint16_t*>(row) + v);
        r.w[(e / 2) & 7] = (e & 1) ? (r.w[(e / 2) & 7] & 0xFFFFu) | (x << 16) : (r.w[(e / 2) & 7] & 0xFFFF0000u) | x;
      } else {
        r.w[e & 7] = *(reinterpret_cast<const volatile uint32_t*>(row) + v);
      }
    }
    return r;
  }
};

template <typename T>
__device__ __forceinline__ float load_element(const T* p) {
  if (sizeof(T) == 2) return __uint_as_float((uint32_t)*reinterpret_cast<const volatile uint16_t*>(p) << 16);
  return __uint_as_float(*reinterpret_cast<const volatile uint32_t*>(p));
}

// ---------------------------------------------------------------------------
// clusters
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }

// shared-memory address of `p` in CTA `rank` of the cluster
__device__ __forceinline__ uint32_t cluster_addr(const void* p, uint32_t rank) {
  uint32_t a = (uint32_t)__cvta_generic_to_shared(p), y;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(y) : "r"(a), "r"(rank));
  return y;
}
__device__ __forceinline__ void cluster_store(uint32_t addr, uint32_t v) {
  asm volatile("st.shared::cluster.b32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ void cluster_store64(uint32_t addr, unsigned long long v) {
  asm volatile("st.shared::cluster.b64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}
__device__ __forceinline__ int cluster_add(uint32_t addr, int v) {
  int old;
  asm volatile("atom.relaxed.cluster.shared::cluster.add.s32 %0, [%1], %2;" : "=r"(old) : "r"(addr), "r"(v) : "memory");
  return old;
}

// ---------------------------------------------------------------------------
// sums over a CTA, in a fixed order
// ---------------------------------------------------------------------------
__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}
template <typename N>
__device__ __forceinline__ N warp_sum(N x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// largest of every thread's x; `red` holds a value per warp.  Ends with a barrier before `red` is read alone.
__device__ __forceinline__ float cta_max(float x, float* red) {
  x = warp_max(x);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = x;
  __syncthreads();
  float m = red[0];
  for (int w = 1; w < (int)blockDim.x / 32; ++w) m = fmaxf(m, red[w]);
  return m;
}

// A value hi + lo of about 48 bits: the logarithms and products that results are differences of.  (The fp64 pipe
// of this part would take a microsecond for them.)
struct Pair {
  float hi, lo;
};

__device__ __forceinline__ Pair two_sum(float a, float b) {  // exact
  const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
  return {s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t))};
}
__device__ __forceinline__ Pair operator+(Pair a, Pair b) {
  const Pair s = two_sum(a.hi, b.hi);
  return {s.hi, s.lo + (a.lo + b.lo)};
}
__device__ __forceinline__ Pair operator-(Pair a) { return {-a.hi, -a.lo}; }
__device__ __forceinline__ Pair operator*(Pair a, Pair b) {
  const float p = __fmul_rn(a.hi, b.hi);
  return {p, fmaf(a.hi, b.hi, -p) + (a.hi * b.lo + a.lo * b.hi)};
}
// rounded once; infinities and NaN as the leading part has them
__device__ __forceinline__ float value_of(Pair a) { return fabsf(a.hi) < INFINITY ? a.hi + a.lo : a.hi; }

// ln S of a sum: the exponent apart, so that only the mantissa's logarithm is rounded to 32 bits
__device__ __forceinline__ Pair log_sum(float s) {
  if (!(s > 0.f) || isinf(s)) return {logf(s), 0.f};
  int e;
  const float f = frexpf(s, &e);
  // ln 2 = 355 / 512 - 2.1219444005469058e-4; e * 355 / 512 is exact
  const Pair y = two_sum((float)e * 0.693359375f, logf(f));
  return {y.hi, y.lo + (float)e * -2.1219444005469058e-4f};
}

// 2^y on the scale of exp2 for partial sums: f = 2^((from - to) sc); 0 where `from` is -inf
__device__ __forceinline__ float shift_of(float from, float to, float sc) {
  return from == -INFINITY ? -200.f : fmaxf((from - to) * sc, -200.f);
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
// CTAs per row and threads per CTA.
struct RowSplit {
  int ctas, threads, groups;  // groups: most groups of one CTA
};

template <typename... KArgs, typename... Args>
inline cudaError_t launch_rows(void (*kernel)(KArgs...), int rows, const RowSplit& sp, size_t smem, cudaStream_t st,
                               Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)rows * (unsigned)sp.ctas);
  cfg.blockDim = dim3(sp.threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = sp.ctas;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<KArgs>(args)...);
}

inline int most_groups(int V, int element_size) { return (V * element_size + 31) / 32 + 1; }

RowSplit split_rows(int rows, int V, int element_size);

// T as the kernels take it
struct Scale {
  float sc;          // log2(e) / T, of exponents
  float hi, lo;      // 1 / T
};

// false where T is not positive or the scale leaves the normal numbers
inline bool logits_scale(float T, Scale* s) {
  if (!isfinite(T) || !(T > 0.f)) return false;
  const double inv = 1.0 / (double)T;
  s->sc = (float)(1.4426950408889634 * inv);
  s->hi = (float)inv;
  s->lo = (float)(inv - (double)s->hi);
  return isfinite(s->sc) && s->sc >= FLT_MIN && s->hi >= FLT_MIN;
}

// [rows, V] with `stride` elements between rows
inline bool logits_shape_ok(const void* p, int64_t stride, int dtype, int32_t V, int32_t rows) {
  if (dtype != SSV_F32 && dtype != SSV_BF16) return false;
  const uintptr_t es = dtype == SSV_BF16 ? 2 : 4;
  return V >= 1 && rows >= 0 && stride >= 0 && (stride == 0 || stride >= V) && stride < (int64_t)1 << 40 &&
         ((uintptr_t)p & (es - 1)) == 0;
}

}  // namespace ssv
