// Shared pieces of the attention-side kernels (dq4_attn.h): typed groups of values, the
// rotation of a lane's two groups, the search of a sequence by its first unit of work,
// and the launch with programmatic stream serialization.
#pragma once

#include <type_traits>

#include "common.cuh"
#include "dq4_attn.h"

namespace dq4d {
namespace {

constexpr unsigned kAllLanes = 0xFFFFFFFFu;

// Wait for the kernel before this one in the stream (launched with programmatic stream
// serialization, see launch_ordered); nothing is read or written before it.
__device__ __forceinline__ void wait_for_stream() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// A plain load.  What a kernel before may have written is read with these only: a read-only
// (non-coherent) load has no place in the order of memory accesses, so that it could be moved
// ahead of wait_for_stream.
template <typename T>
__device__ __forceinline__ T load_global(const T* p) {
  return *p;
}

// Loads from L2 of what other CTAs of the same kernel have written, in order after the atomic
// that says so.
__device__ __forceinline__ float load_l2(const float* p) {
  float f;
  asm volatile("ld.global.cg.f32 %0, [%1];" : "=f"(f) : "l"(p) : "memory");
  return f;
}
__device__ __forceinline__ float2 load_l2(const float2* p) {
  float2 f;
  asm volatile("ld.global.cg.v2.f32 {%0, %1}, [%2];" : "=f"(f.x), "=f"(f.y) : "l"(p) : "memory");
  return f;
}
__device__ __forceinline__ float4 load_l2(const float4* p) {
  float4 f;
  asm volatile("ld.global.cg.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(f.x), "=f"(f.y), "=f"(f.z), "=f"(f.w) : "l"(p) : "memory");
  return f;
}

// ------------------------------------------------------------------ element types
template <int DT>
struct Elem;
template <>
struct Elem<DQ4_OUT_F16> {
  using T = __half;
  static __device__ __forceinline__ float load(const T* p) { return __half2float(*p); }
  static __device__ __forceinline__ T make(float f) { return __float2half_rn(f); }
};
template <>
struct Elem<DQ4_OUT_BF16> {
  using T = __nv_bfloat16;
  static __device__ __forceinline__ float load(const T* p) { return __bfloat162float(*p); }
  static __device__ __forceinline__ T make(float f) { return __float2bfloat16_rn(f); }
};
template <>
struct Elem<DQ4_OUT_F32> {
  using T = float;
  static __device__ __forceinline__ float load(const T* p) { return *p; }
  static __device__ __forceinline__ T make(float f) { return f; }
};

// ----------------------------------------------------------------- groups of values
// Raw bits of a group of V consecutive values: 8 or 16 bytes.
template <int DT, int V>
struct Raw {
  static constexpr int kBytes = V * int(sizeof(typename Elem<DT>::T));
  static_assert(kBytes == 8 || kBytes == 16, "one load");
  std::conditional_t<kBytes == 8, uint2, uint4> u;
};

template <int DT, int V>
__device__ __forceinline__ Raw<DT, V> load_group(const typename Elem<DT>::T* p) {
  return {load_global(reinterpret_cast<const decltype(Raw<DT, V>::u)*>(p))};
}

// The same for what is read, or written, once: it leaves the caches first.  (Volatile and with
// a memory clobber: this load, too, keeps its place after wait_for_stream.)
template <int DT, int V>
__device__ __forceinline__ Raw<DT, V> load_group_once(const typename Elem<DT>::T* p) {
  Raw<DT, V> r;
  if constexpr (sizeof(r.u) == 8) {
    asm volatile("ld.global.cs.v2.b32 {%0, %1}, [%2];"
                 : "=r"(r.u.x), "=r"(r.u.y) : "l"(p) : "memory");
  } else {
    asm volatile("ld.global.cs.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r.u.x), "=r"(r.u.y), "=r"(r.u.z), "=r"(r.u.w) : "l"(p) : "memory");
  }
  return r;
}

// A lane's two groups in FP32: values 0 .. V - 1 are group a of lane_place, the others b.
template <int V>
struct Vals {
  float v[2 * V];
};

template <int DT, int V>
__device__ __forceinline__ Vals<V> widen(const Raw<DT, V>& ra, const Raw<DT, V>& rb) {
  Vals<V> f;
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    uint32_t w[Raw<DT, V>::kBytes / 4];
    memcpy(w, half ? &rb.u : &ra.u, sizeof(w));
    float* to = f.v + half * V;
#pragma unroll
    for (int i = 0; i < V; i += 2) {
      if constexpr (DT == DQ4_OUT_F32) {
        to[i] = __uint_as_float(w[i]);
        to[i + 1] = __uint_as_float(w[i + 1]);
      } else if constexpr (DT == DQ4_OUT_BF16) {
        to[i] = __uint_as_float(w[i / 2] << 16);
        to[i + 1] = __uint_as_float(w[i / 2] & 0xFFFF0000u);
      } else {
        __half2 h;
        memcpy(&h, &w[i / 2], 4);
        to[i] = __low2float(h);
        to[i + 1] = __high2float(h);
      }
    }
  }
  return f;
}

// Group a (half 0) or b of a lane's values, in the element type.
template <int DT, int V>
__device__ __forceinline__ Raw<DT, V> narrow(const Vals<V>& x, int half) {
  uint32_t w[Raw<DT, V>::kBytes / 4];
  const float* from = x.v + half * V;
#pragma unroll
  for (int i = 0; i < V; i += 2) {
    if constexpr (DT == DQ4_OUT_F32) {
      w[i] = __float_as_uint(from[i]);
      w[i + 1] = __float_as_uint(from[i + 1]);
    } else {
      w[i / 2] = pack2<DT>(from[i], from[i + 1]);
    }
  }
  Raw<DT, V> r;
  memcpy(&r.u, w, sizeof(w));
  return r;
}

template <int DT, int V>
__device__ __forceinline__ void store_group(typename Elem<DT>::T* p, const Raw<DT, V>& r) {
  *reinterpret_cast<decltype(Raw<DT, V>::u)*>(p) = r.u;
}
template <int DT, int V>
__device__ __forceinline__ void store_group_once(typename Elem<DT>::T* p, const Raw<DT, V>& r) {
  __stcs(reinterpret_cast<decltype(Raw<DT, V>::u)*>(p), r.u);
}

// ------------------------------------------------------------------- the rotation
// A head of kDim values is held by kDim / 2 V lanes, two groups of V values each, so chosen
// that both values of every rotated pair sit in one lane and no lane needs another's.
// Half-split pairs (i, i + rotary / 2): lane l < rotary / 2 V takes groups l and
// l + rotary / 2 V, the others two neighbouring groups past rotary.  Neighbours paired: groups
// 2 l and 2 l + 1.  Either way lane l turns with the table entries V l .. V l + V - 1 of its
// position's row.  rotary is a multiple of 2 V.
struct LanePlace {
  int a, b;     // first values of the two groups
  bool turned;  // whether the lane's values are rotated
};

template <int V>
__device__ __forceinline__ LanePlace lane_place(int l, int rotary, bool interleaved) {
  LanePlace p;
  p.turned = 2 * V * l < rotary;
  if (interleaved || !p.turned) {
    p.a = 2 * V * l;
    p.b = 2 * V * l + V;
  } else {
    p.a = V * l;
    p.b = V * l + rotary / 2;
  }
  return p;
}

// A lane's V entries of a row of a table.
template <int V>
__device__ __forceinline__ void load_entries(const float* p, float (&x)[V]) {
#pragma unroll
  for (int i = 0; i < V; i += 4) {
    const float4 f = load_global(reinterpret_cast<const float4*>(p + i));
    x[i] = f.x;
    x[i + 1] = f.y;
    x[i + 2] = f.z;
    x[i + 3] = f.w;
  }
}

// Value i of a lane turns with its partner y by entry turn_entry of the lane's cosines and sines:
// x c - y s, or x c + y s if turn_adds (the second of a pair).
template <bool kInterleaved, int V>
__device__ __forceinline__ constexpr int partner(int i) { return kInterleaved ? i ^ 1 : i ^ V; }
template <bool kInterleaved, int V>
__device__ __forceinline__ constexpr int turn_entry(int i) { return kInterleaved ? i / 2 : i % V; }
template <bool kInterleaved, int V>
__device__ __forceinline__ constexpr bool turn_adds(int i) { return kInterleaved ? i & 1 : i >= V; }

// A lane's values turned (kBack: turned back), every product and sum rounded on its own.
template <bool kInterleaved, bool kBack, int V>
__device__ __forceinline__ Vals<V> turned(const Vals<V>& x, const float (&c)[V],
                                          const float (&s)[V]) {
  Vals<V> r;
#pragma unroll
  for (int i = 0; i < 2 * V; ++i) {
    const int e = turn_entry<kInterleaved, V>(i);
    const float xc = __fmul_rn(x.v[i], c[e]);
    const float ys = __fmul_rn(x.v[partner<kInterleaved, V>(i)], s[e]);
    r.v[i] = turn_adds<kInterleaved, V>(i) != kBack ? __fadd_rn(xc, ys) : __fsub_rn(xc, ys);
  }
  return r;
}

// --------------------------------------------------------------- ragged sequences
// The last b in [0, n) with first(b) <= u, for a non-decreasing first with first(0) <= u:
// 32 probes a step, one per lane; every lane gets the answer.
template <typename First>
__device__ __forceinline__ int64_t find_last(int64_t n, int64_t u, First first) {
  const int lane = threadIdx.x & 31;
  int64_t lo = 0;
  while (n > 1) {
    const int64_t step = (n + 31) / 32;
    const int64_t at = lane * step;
    const bool in = at < n && first(lo + at) <= u;
    const int hits = __popc(__ballot_sync(kAllLanes, in));
    const int64_t skip = (hits - 1) * step;
    lo += skip;
    n = n - skip < step ? n - skip : step;
  }
  return lo;
}

// ------------------------------------------------------------------------ host side
inline bool aligned(const void* p, uintptr_t to) { return reinterpret_cast<uintptr_t>(p) % to == 0; }

// Launch on `stream` with programmatic stream serialization: the grid may be scheduled
// while the kernel before it drains, and waits for it (wait_for_stream) before it touches
// memory.
template <typename... KArgs, typename... Actual>
int launch_ordered(void (*kernel)(KArgs...), dim3 grid, int threads, size_t smem,
                   cudaStream_t stream, Actual&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, std::forward<Actual>(args)...);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return fail_cuda(DQ4_ERR_LAUNCH, e);
  }
  return DQ4_OK;
}

// Let `kernel` have `bytes` of dynamic shared memory, once for each device (bit dev of
// *allowed; devices past 63 every time).
template <typename Kernel>
int allow_smem(Kernel kernel, int bytes, int dev, std::atomic<uint64_t>* allowed) {
  const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
  if (allowed->load(std::memory_order_relaxed) & bit) return DQ4_OK;
  const cudaError_t e =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return fail_cuda(DQ4_ERR_LAUNCH, e);
  allowed->fetch_or(bit, std::memory_order_relaxed);
  return DQ4_OK;
}

inline bool valid_dtype(int32_t dtype, bool with_f32) {
  return dtype == DQ4_OUT_F16 || dtype == DQ4_OUT_BF16 || (with_f32 && dtype == DQ4_OUT_F32);
}

}  // namespace
}  // namespace dq4d
