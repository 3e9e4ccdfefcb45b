// What the kernels of the layers with 8-bit weights share (dq4_int8.h): codes as FP16, the FP16
// tensor-core product of a warp, tensor maps.
//
// The integer tensor-core rate of this GPU is far below its FP16 rate, and codes are exact in
// FP16, so products of codes are FP16 products with FP32 sums: exact while sums are below 2^24.
#pragma once

#include "attn.cuh"
#include "dq4_int8.h"
#include "tcgen05.cuh"
#include "tmap.cuh"

namespace dq4d {
namespace {

constexpr float kRecip127 = 0.007874015718698502f;  // RN32(1 / 127)
constexpr int kMaxOutliers = 128;
constexpr int64_t kInt8Counters = 4096;  // bytes of counters at the head of a workspace

// Four codes as FP16 pairs: 1152 is taken from 1024 + 128 + code, both exact.
__device__ __forceinline__ void codes_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  const uint32_t u = w ^ 0x80808080u;
  const __half2 off = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));
  uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
  __half2 x, y;
  memcpy(&x, &a, 4);
  memcpy(&y, &b, 4);
  x = __hsub2(x, off);
  y = __hsub2(y, off);
  memcpy(&lo, &x, 4);
  memcpy(&hi, &y, 4);
}

// D += A B, 16 x 16 by 16 x 8, FP16 with FP32 sums.
__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                          uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// A load whose place among the others is kept: ahead of its use.
__device__ __forceinline__ float load_ahead(const float* p) {
  float v;
  asm volatile("ld.global.f32 %0, [%1];" : "=f"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ uint4 load_ahead(const uint4* p) {
  uint4 v;
  asm volatile("ld.global.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p) : "memory");
  return v;
}

// Of the kernels that stream a weight past few tokens: warps of a CTA, and the values of K of a
// copy.
constexpr int kStreamWarps = 8, kStreamThreads = 32 * kStreamWarps;
constexpr int kChunk = 128;

__device__ __forceinline__ uint8_t* aligned_1024(uint8_t* p) {
  return reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(p) + 1023) & ~uintptr_t(1023));
}

// A matrix's map for TMA: boxes of box_w x box_h values, swizzled.
inline int encode_2d(CUtensorMap* map, CUtensorMapDataType type, const void* base, int64_t width,
                     int64_t height, int64_t stride_bytes, int box_w, int box_h,
                     CUtensorMapSwizzle swizzle) {
  const EncodeTiled encode = tensor_map_encoder();
  if (!encode) return fail_cuda(DQ4_ERR_LAUNCH, cudaErrorNotSupported);
  const cuuint64_t size[2] = {cuuint64_t(width), cuuint64_t(height)};
  const cuuint64_t stride[1] = {cuuint64_t(stride_bytes)};
  const cuuint32_t box[2] = {cuuint32_t(box_w), cuuint32_t(box_h)};
  const cuuint32_t step[2] = {1, 1};
  const CUresult r = encode(map, type, 2, const_cast<void*>(base), size, stride, box, step,
                            CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
                            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? DQ4_OK : fail_cuda(DQ4_ERR_LAUNCH, cudaErrorInvalidValue);
}

template <typename T>
__device__ __forceinline__ float load_half(const void* p, int64_t i) {
  return float(static_cast<const T*>(p)[i]);
}
__device__ __forceinline__ float load_16(const void* p, int64_t i, bool bf16) {
  return bf16 ? load_half<__nv_bfloat16>(p, i) : load_half<__half>(p, i);
}
__device__ __forceinline__ float load_any(const void* p, int64_t i, int dtype) {
  return dtype == DQ4_OUT_F32 ? static_cast<const float*>(p)[i]
                              : load_16(p, i, dtype == DQ4_OUT_BF16);
}
__device__ __forceinline__ void store_any(void* p, int64_t i, float f, int dtype) {
  if (dtype == DQ4_OUT_F32) store_one<DQ4_OUT_F32>(p, i, f);
  else if (dtype == DQ4_OUT_BF16) store_one<DQ4_OUT_BF16>(p, i, f);
  else store_one<DQ4_OUT_F16>(p, i, f);
}

}  // namespace

// The arguments of the two product kernels.
struct Int8Linear {
  const int8_t* codes;  // [M][K]
  const float* scales;
  const int8_t* CB;  // [N][K]
  const float* SCB;
  int64_t M, N, K;
  const int64_t* cols;  // [L]
  const void* outliers;  // [M][L]
  int L;
  bool outliers_bf16;
  const void* bias;
  int out_dtype;
  void* Y;
  int* bad;
};

}  // namespace dq4d
