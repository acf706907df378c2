// Rows of logits, as the kernels on a pass's logits read and write them
// (ssv_logprobs, ssv_distill, ssv_distill_backward).
//
// A row of V elements at any element-aligned address is cut at the 16-byte
// boundaries of memory into vectors: vector i holds the elements
// [i E - lead, (i + 1) E - lead), E = 16 / element size, lead the elements
// between the boundary at or below the row's start and that start.  All but the
// first and the last lie inside the row and move as one access; the edges are read
// element by element, and what they lack counts as -inf.
//
// A CTA has a part of a row's vectors.  Its threads take every NT-th, kBatch of
// them in a step, and copy them to shared memory ahead of their use (cp.async,
// each thread to slots that it reads itself, so that no barrier is needed),
// through a ring of a few steps or, a short part, all at once.
#pragma once

#include "ssv_internal.cuh"

#include <float.h>
#include <math.h>

namespace ssv {

constexpr int kLogitsMaxVocab = 1 << 19;  // largest V
constexpr int kLogitsMaxTop = 128;        // most alternatives of a row
constexpr int kMaxCluster = 8;
constexpr int kLogBatch = 2, kBatch = 1 << kLogBatch;  // vectors of a thread in one step
constexpr float kLn2 = 0.693147180559945309f;

template <typename T> constexpr int kVec = 16 / (int)sizeof(T);

__device__ __forceinline__ void copy_async(void* shared, const void* global) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(shared)), "l"(global)
               : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// all but the last N groups have landed
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
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

// element pair i of a vector
template <typename T>
__device__ __forceinline__ float2 pair_of(const uint4& r, int i) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
  if (sizeof(T) == 2) return make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
  return make_float2(__uint_as_float(w[(2 * i) & 3]), __uint_as_float(w[(2 * i + 1) & 3]));
}

template <typename T>
__device__ __forceinline__ uint32_t none_bits() { return sizeof(T) == 2 ? 0xFF80FF80u : 0xFF800000u; }  // -inf

// largest of the even and of the odd elements of kBatch vectors, -inf where there is none (NaN are passed over)
template <typename T>
__device__ __forceinline__ float2 step_max(const uint4 (&x)[kBatch]) {
  if constexpr (sizeof(T) == 2) {
    __nv_bfloat162 h[4 * kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const uint32_t w[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) h[4 * u + i] = *reinterpret_cast<const __nv_bfloat162*>(&w[i]);
    }
#pragma unroll
    for (int s = 2 * kBatch; s > 0; s >>= 1)
#pragma unroll
      for (int i = 0; i < s; ++i) h[i] = __hmax2(h[i], h[i + s]);
    return make_float2(fmaxf(-INFINITY, __low2float(h[0])), fmaxf(-INFINITY, __high2float(h[0])));
  } else {
    float2 m = make_float2(-INFINITY, -INFINITY);
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      m.x = fmaxf(m.x, fmaxf(__uint_as_float(x[u].x), __uint_as_float(x[u].z)));
      m.y = fmaxf(m.y, fmaxf(__uint_as_float(x[u].y), __uint_as_float(x[u].w)));
    }
    return m;
  }
}

// A row, cut into vectors.
template <typename T>
struct RowView {
  const char* base;  // address of vector 0 (16-byte boundary at or below the row)
  const T* row;
  int lead, V, n;    // n vectors, those of [lo, hi) whole
  int lo, hi;

  __device__ __forceinline__ RowView(const T* p, int V_) : row(p), V(V_) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    base = reinterpret_cast<const char*>(a & ~uintptr_t(15));
    lead = (int)((a & 15) / sizeof(T));
    n = (lead + V + kVec<T> - 1) / kVec<T>;
    lo = lead ? 1 : 0;
    hi = (lead + V) / kVec<T>;
  }
  __device__ __forceinline__ bool whole(int i) const { return i >= lo && i < hi; }
  __device__ __forceinline__ int first(int i) const { return i * kVec<T> - lead; }  // element at the vector's start

  // An edge, element by element.  Its loads depend on nothing, so that they take one way to memory and not one each.
  __device__ __noinline__ uint4 edge(int i) const {
    const int v0 = first(i);
    uint32_t x[kVec<T>], w[4];
#pragma unroll
    for (int e = 0; e < kVec<T>; ++e) {
      const int v = min(max(v0 + e, 0), V - 1);
      x[e] = sizeof(T) == 2 ? *(reinterpret_cast<const volatile uint16_t*>(row) + v)
                            : *(reinterpret_cast<const volatile uint32_t*>(row) + v);
    }
#pragma unroll
    for (int e = 0; e < kVec<T>; ++e)
      if (v0 + e < 0 || v0 + e >= V) x[e] = sizeof(T) == 2 ? none_bits<T>() & 0xFFFFu : none_bits<T>();
#pragma unroll
    for (int k = 0; k < 4; ++k) w[k] = sizeof(T) == 2 ? x[(2 * k) % kVec<T>] | x[(2 * k + 1) % kVec<T>] << 16 : x[k];
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  __device__ __forceinline__ uint4 load(int i) const {
    if (!whole(i)) return edge(i);
    uint4 r;
    asm volatile("ld.global.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
                 : "l"(base + (size_t)i * 16));
    return r;
  }
};

// A CTA's part of a row: vectors [i0, i1), elements [lo, hi), the first one's start at element `at`; a step is kBatch
// vectors of every thread.
template <typename T>
struct PartView {
  int i0, i1, lo, hi, at, steps;
  int NT;            // threads that share it
  int full0, full1;  // steps [full0, full1) are full: every thread has kBatch whole vectors

  // CTA `rank` of 2^log_c, of 2^log_nt threads (no division: eight warps of every CTA would spend more on it than on
  // some rows)
  __device__ __forceinline__ PartView(const RowView<T>& row, int rank, int log_c, int log_nt) {
    i0 = (int)(((long long)row.n * rank) >> log_c);
    i1 = (int)(((long long)row.n * (rank + 1)) >> log_c);
    at = row.first(i0);
    lo = max(0, at);
    hi = min(row.V, row.first(i1));
    NT = 1 << log_nt;
    const int log_per = log_nt + kLogBatch;
    steps = (i1 - i0 + (1 << log_per) - 1) >> log_per;
    full0 = i0 < row.lo ? 1 : 0;
    full1 = max(0, min(i1, row.hi) - i0) >> log_per;
  }
  // Slots for the part in `memory` (128-byte aligned): placed to the 128-byte lines of shared memory as the vectors are
  // to those of global memory (with slots 48 bytes off the lines the gradient of 4096 rows took 553 us, on them 492).
  __device__ __forceinline__ uint4* slots_in(unsigned char* memory, const RowView<T>& row) const {
    return reinterpret_cast<uint4*>(memory) + (((uint32_t)(reinterpret_cast<uintptr_t>(row.base) >> 4) + (uint32_t)i0) & 7u);
  }
  __device__ __forceinline__ bool full(int k) const { return k >= full0 && k < full1; }
  // f(d, i) for the row's first and last vectors that are not whole, where vector i is the thread's in step k, d slots
  // behind its first (a row of one vector may have it twice)
  template <typename F>
  __device__ __forceinline__ void edges(const RowView<T>& row, int k, F f) const {
    const int j = (int)threadIdx.x + NT * kBatch * k;
    const int head = i0 < row.lo && i0 < i1 ? 0 : -1, tail = i1 > row.hi ? row.hi - i0 : -1;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int d = (e ? tail : head) - j;
      if (d >= 0 && d < NT * kBatch && (d & (NT - 1)) == 0) f(d, i0 + j + d);
    }
  }
  // the thread's vectors of step k, from `slots` on, NT apart
  __device__ __forceinline__ void fetch(const RowView<T>& row, int k, uint4* slots) const {
    if (k < 0) {  // none, but a group of copies all the same
      copy_commit();
      return;
    }
    const int i = i0 + (int)threadIdx.x + NT * kBatch * k;
    const char* from = row.base + (size_t)i * 16;
    if (full(k)) {
#pragma unroll
      for (int u = 0; u < kBatch; ++u) copy_async(slots + NT * u, from + (size_t)(NT * 16) * u);
    } else if (k < steps) {
      const int lowest = row.lo, end = min(i1, row.hi);
#pragma unroll
      for (int u = 0; u < kBatch; ++u)
        if (i + NT * u >= lowest && i + NT * u < end) copy_async(slots + NT * u, from + (size_t)(NT * 16) * u);
      edges(row, k, [&](int d, int e) { slots[d] = row.edge(e); });
    }
    copy_commit();
  }
  // the same from the slots, -inf where there is none
  template <bool FULL>
  __device__ __forceinline__ void take(int k, const uint4* slots, uint4 (&x)[kBatch]) const {
    const int i = i0 + (int)threadIdx.x + NT * kBatch * k;
#pragma unroll
    for (int u = 0; u < kBatch; ++u)
      if (FULL || i + NT * u < i1)
        x[u] = slots[NT * u];
      else
        x[u].x = x[u].y = x[u].z = x[u].w = none_bits<T>();
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
// sums over a warp, in a fixed order
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

__device__ __forceinline__ Pair warp_sum(Pair x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    x = x + Pair{__shfl_xor_sync(0xffffffffu, x.hi, o), __shfl_xor_sync(0xffffffffu, x.lo, o)};
  return x;
}

// ln s of a positive number to about 2^-30: s = 2^e f with f in [sqrt(1/2), sqrt(2)), and ln f = 2 atanh((f - 1) / (f + 1))
// by its series, whose first term alone needs more than 32 bits
__device__ __forceinline__ Pair log_sum(float s) {
  if (!(s > 0.f) || isinf(s)) return {logf(s), 0.f};
  int e;
  float f = frexpf(s, &e);
  if (f < 0.70710678f) {
    f *= 2.f;
    --e;
  }
  const float a = f - 1.f;  // exact
  const Pair b = two_sum(f, 1.f);
  // q to 2 or 3 units and what it lacks; the series takes it in by its slope, 1 + z.  (A quotient rounded to the last bit
  // would cost a call two divisions: 7 rows of bf16, backward, 4.6 us with them, 4.4 without.)
  const float inv = __fdividef(1.f, b.hi), q = a * inv, low = (fmaf(-q, b.hi, a) - q * b.lo) * inv, z = q * q;
  const float series = z * (1.f / 3 + z * (1.f / 5 + z * (1.f / 7 + z * (1.f / 9 + z * (1.f / 11)))));
  // ln 2 = 355 / 512 - 2.1219444005469058e-4; e * 355 / 512 is exact
  const Pair y = two_sum((float)e * 0.693359375f, 2.f * q);
  return {y.hi, y.lo + (2.f * (fmaf(low, z, low) + q * series) + (float)e * -2.1219444005469058e-4f)};
}

__device__ __forceinline__ Pair log_sum(Pair s) {
  const float v = value_of(s);
  const Pair y = log_sum(v);
  return v > 0.f && v < INFINITY ? Pair{y.hi, y.lo + ((s.hi - v) + s.lo) / v} : y;
}

// 2^y on the scale of exp2 for partial sums: f = 2^((from - to) sc); 0 where `from` is -inf
__device__ __forceinline__ float shift_of(float from, float to, float sc) {
  return from == -INFINITY ? -200.f : fmaxf((from - to) * sc, -200.f);
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
// CTAs per row and threads per CTA, powers of two; most vectors of a CTA.
struct RowSplit {
  int ctas, threads, vectors, log_c, log_nt;
  int batches() const { return (vectors + threads * kBatch - 1) / (threads * kBatch); }
};

// Dynamic shared memory above the default needs the kernel's leave, once per device.
template <typename K>
inline cudaError_t allow_shared(K kernel, size_t bytes, uint64_t* done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || bytes <= 40 * 1024) return e;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0ull;
  if (__atomic_load_n(done, __ATOMIC_ACQUIRE) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 216 * 1024);
  if (e == cudaSuccess) __atomic_fetch_or(done, bit, __ATOMIC_RELEASE);
  return e;
}

// CTAs of a row are a cluster, up to kMaxCluster of them; more are independent.
template <typename... KArgs, typename... Args>
inline cudaError_t launch_rows(void (*kernel)(KArgs...), int rows, const RowSplit& sp, int threads, size_t smem,
                               cudaStream_t st, Args&&... args) {
  if ((long long)rows * sp.ctas > 0x7FFFFFFFLL) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)rows * (unsigned)sp.ctas);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = sp.ctas <= kMaxCluster ? sp.ctas : 1;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<KArgs>(args)...);
}

constexpr int kSlotSlack = 128;  // bytes that slots_in may leave in front, up to a line

// vectors of a row at most
inline int row_vectors(int V, int element_size) { return (V * element_size + 15) / 16 + 1; }

// `vectors` of a row over c CTAs
inline RowSplit split_of(int vectors, int c, int most_threads) {
  RowSplit sp;
  sp.ctas = c;
  sp.vectors = (vectors + c - 1) / c;
  for (sp.log_c = 0; 1 << sp.log_c < c;) ++sp.log_c;
  for (sp.log_nt = 5; 1 << sp.log_nt < most_threads && 1 << sp.log_nt < sp.vectors;) ++sp.log_nt;
  sp.threads = 1 << sp.log_nt;
  return sp;
}

// T as the kernels take it
struct Scale {
  float sc;      // log2(e) / T, of exponents
  float down;    // the same rounded down, and
  float rest;    // what that leaves, above 0 (so that -inf times either is -inf)
  float hi, lo;  // 1 / T to 48 bits
};

// false where T is not positive or the scale leaves the normal numbers
inline bool logits_scale(float T, Scale* s) {
  if (!isfinite(T) || !(T > 0.f)) return false;
  const double inv = 1.0 / (double)T;
  s->sc = (float)(1.4426950408889634 * inv);
  const double exact = 1.4426950408889634 * inv;
  s->down = (double)s->sc > exact ? nextafterf(s->sc, 0.f) : s->sc;
  s->rest = fmaxf((float)(exact - (double)s->down), FLT_TRUE_MIN);
  s->hi = (float)inv;
  s->lo = (float)(inv - (double)s->hi);
  return isfinite(s->sc) && s->sc >= FLT_MIN && s->hi >= FLT_MIN;
}

// whether `bytes` at p meet a [rows, V] matrix with `stride` elements between rows, gaps included
inline bool meets_rows(const void* p, size_t bytes, const void* rows_at, int64_t stride, int V, int rows, int es) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(rows_at);
  return p && bytes && rows > 0 && a < b + ((uintptr_t)(rows - 1) * stride + V) * es && b < a + bytes;
}

// [rows, V] with `stride` elements between rows
inline bool logits_shape_ok(const void* p, int64_t stride, int dtype, int32_t V, int32_t rows) {
  if (dtype != SSV_F32 && dtype != SSV_BF16) return false;
  const uintptr_t es = dtype == SSV_BF16 ? 2 : 4;
  return V >= 1 && rows >= 0 && stride >= 0 && (stride == 0 || stride >= V) && stride < (int64_t)1 << 40 &&
         ((uintptr_t)p & (es - 1)) == 0;
}

}  // namespace ssv
