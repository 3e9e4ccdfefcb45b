// Shared pieces of the attention-side kernels (dq4_attn.h): typed 4-value groups, the
// rotation of a lane's eight values, the search of a sequence by its first unit of work,
// and the launch with programmatic stream serialization.
#pragma once

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

// ------------------------------------------------------------ groups of four values
struct F4 {
  float v[4];
};

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

// Raw bits of four consecutive values: 8 bytes (16-bit types) or 16 (FP32).
template <int DT>
struct Raw4 {
  uint2 u;
};
template <>
struct Raw4<DQ4_OUT_F32> {
  uint4 u;
};

template <int DT>
__device__ __forceinline__ Raw4<DT> load4(const typename Elem<DT>::T* p) {
  Raw4<DT> r;
  if constexpr (DT == DQ4_OUT_F32) {
    r.u = load_global(reinterpret_cast<const uint4*>(p));
  } else {
    r.u = load_global(reinterpret_cast<const uint2*>(p));
  }
  return r;
}

// The same for what is read, or written, once: it leaves the caches first.
template <int DT>
__device__ __forceinline__ Raw4<DT> load4_once(const typename Elem<DT>::T* p) {
  Raw4<DT> r;
  if constexpr (DT == DQ4_OUT_F32) {
    r.u = __ldcs(reinterpret_cast<const uint4*>(p));
  } else {
    r.u = __ldcs(reinterpret_cast<const uint2*>(p));
  }
  return r;
}

template <int DT>
__device__ __forceinline__ F4 widen(const Raw4<DT>& r) {
  F4 f;
  if constexpr (DT == DQ4_OUT_F32) {
    f.v[0] = __uint_as_float(r.u.x);
    f.v[1] = __uint_as_float(r.u.y);
    f.v[2] = __uint_as_float(r.u.z);
    f.v[3] = __uint_as_float(r.u.w);
  } else if constexpr (DT == DQ4_OUT_BF16) {
    f.v[0] = __uint_as_float(r.u.x << 16);
    f.v[1] = __uint_as_float(r.u.x & 0xFFFF0000u);
    f.v[2] = __uint_as_float(r.u.y << 16);
    f.v[3] = __uint_as_float(r.u.y & 0xFFFF0000u);
  } else {
    __half2 a, b;
    memcpy(&a, &r.u.x, 4);
    memcpy(&b, &r.u.y, 4);
    f.v[0] = __low2float(a);
    f.v[1] = __high2float(a);
    f.v[2] = __low2float(b);
    f.v[3] = __high2float(b);
  }
  return f;
}

template <int DT>
__device__ __forceinline__ void store4(typename Elem<DT>::T* p, const F4& f) {
  if constexpr (DT == DQ4_OUT_F32) {
    *reinterpret_cast<float4*>(p) = make_float4(f.v[0], f.v[1], f.v[2], f.v[3]);
  } else {
    *reinterpret_cast<uint2*>(p) =
        make_uint2(pack2<DT>(f.v[0], f.v[1]), pack2<DT>(f.v[2], f.v[3]));
  }
}

template <int DT>
__device__ __forceinline__ void store4_once(typename Elem<DT>::T* p, const F4& f) {
  if constexpr (DT == DQ4_OUT_F32) {
    __stcs(reinterpret_cast<float4*>(p), make_float4(f.v[0], f.v[1], f.v[2], f.v[3]));
  } else {
    __stcs(reinterpret_cast<uint2*>(p),
           make_uint2(pack2<DT>(f.v[0], f.v[1]), pack2<DT>(f.v[2], f.v[3])));
  }
}

// ------------------------------------------------------------------- the rotation
// A head of kDim values is held by kDim / 8 lanes, eight values each: two groups of four,
// at values 4 a and 4 b, so chosen that both values of every rotated pair sit in one lane
// and no lane needs another's.  Half-split pairs (i, i + rotary / 2): lane l < rotary / 8
// takes groups l and l + rotary / 8, the others two neighbouring groups past rotary.
// Neighbours paired: groups 2 l and 2 l + 1.  Either way lane l turns with the table
// entries 4 l .. 4 l + 3 of its position's row.
struct LanePlace {
  int a, b;     // first values of the two groups
  bool turned;  // whether the lane's values are rotated
};

__device__ __forceinline__ LanePlace lane_place(int l, int rotary, bool interleaved) {
  LanePlace p;
  p.turned = 8 * l < rotary;
  if (interleaved || !p.turned) {
    p.a = 8 * l;
    p.b = 8 * l + 4;
  } else {
    p.a = 4 * l;
    p.b = 4 * l + rotary / 2;
  }
  return p;
}

// (x, y) -> (x c - y s, y c + x s), every product and sum rounded on its own
__device__ __forceinline__ void turn_pair(float& x, float& y, float c, float s) {
  const float xc = __fmul_rn(x, c), ys = __fmul_rn(y, s);
  const float yc = __fmul_rn(y, c), xs = __fmul_rn(x, s);
  x = __fsub_rn(xc, ys);
  y = __fadd_rn(yc, xs);
}

__device__ __forceinline__ void turn(F4& a, F4& b, const float4& c, const float4& s,
                                     bool interleaved) {
  if (interleaved) {
    turn_pair(a.v[0], a.v[1], c.x, s.x);
    turn_pair(a.v[2], a.v[3], c.y, s.y);
    turn_pair(b.v[0], b.v[1], c.z, s.z);
    turn_pair(b.v[2], b.v[3], c.w, s.w);
  } else {
    turn_pair(a.v[0], b.v[0], c.x, s.x);
    turn_pair(a.v[1], b.v[1], c.y, s.y);
    turn_pair(a.v[2], b.v[2], c.z, s.z);
    turn_pair(a.v[3], b.v[3], c.w, s.w);
  }
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
