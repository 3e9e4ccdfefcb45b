// What the kernels of the layers with 8-bit weights share (dq4_int8.h): codes as FP16, the FP16
// tensor-core product of a warp, sums over the warps of a CTA.
//
// The integer tensor-core rate of this GPU is far below its FP16 rate, and codes are exact in
// FP16, so products of codes are FP16 products with FP32 sums: exact while sums are below 2^24.
#pragma once

#include "attn.cuh"
#include "dq4_int8.h"

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

// 16 bytes of a weight, read once.
__device__ __forceinline__ uint4 load_weight(const int8_t* p) {
  uint4 v;
  asm volatile("ld.global.cs.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p) : "memory");
  return v;
}


// ------------------------------------------------- a warp's product of weight rows and tokens
// acc += W X^T for 16 RT weight rows and 8 NT tokens over chunks of 64 of K, first, first + step ..
// below end.  The order of K inside a product is free: lane (g, c) = (lane / 4, lane % 4) reads 16
// consecutive codes of rows g and g + 8 of each 16, and the same places of token g of each 8, so
// that nothing passes through shared memory; four products take them four at a time.
//   row[rt][h]  this lane's rows, advanced to its 16 c; null: a row of zeros
//   Src         the tokens' values: raw words of a place, and of those the two operand words
template <int RT, int NT, int U, typename Src>
__device__ __forceinline__ void warp_product(float (&acc)[RT][NT][4], const int8_t* const (&row)[RT][2],
                                             const Src& src, int64_t K, int first, int step,
                                             int end) {
  const int c = threadIdx.x & 3;
  for (int j0 = first; j0 < end; j0 += step * U) {
    uint4 w[U][RT][2];
    typename Src::Raw x[U][NT];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t k = int64_t(j0 + u * step) * 64;
      const bool in = j0 + u * step < end && k + 16 * c < K;
#pragma unroll
      for (int rt = 0; rt < RT; ++rt)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          w[u][rt][h] = make_uint4(0, 0, 0, 0);
          if (in && row[rt][h]) w[u][rt][h] = load_weight(row[rt][h] + k);
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t k = int64_t(j0 + u * step) * 64;
      const bool in = j0 + u * step < end && k + 16 * c < K;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) src.load(x[u][nt], nt, k, in);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        uint32_t b[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) src.words(x[u][nt], nt, s, b[nt][0], b[nt][1]);
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
          uint32_t a[4];
          codes_f16(reinterpret_cast<const uint32_t*>(&w[u][rt][0])[s], a[0], a[2]);
          codes_f16(reinterpret_cast<const uint32_t*>(&w[u][rt][1])[s], a[1], a[3]);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            mma_16816(acc[rt][nt], a[0], a[1], a[2], a[3], b[nt][0], b[nt][1]);
        }
      }
    }
  }
}

// Tokens in 8 bits: lane's token of each 8, advanced to its 16 c, or null.
template <int NT>
struct CodeTokens {
  using Raw = uint4;
  const int8_t* at[NT];
  __device__ __forceinline__ void load(uint4& x, int nt, int64_t k, bool in) const {
    x = make_uint4(0, 0, 0, 0);
    if (in && at[nt]) x = load_global(reinterpret_cast<const uint4*>(at[nt] + k));
  }
  __device__ __forceinline__ void words(const uint4& x, int, int s, uint32_t& b0,
                                        uint32_t& b1) const {
    codes_f16(reinterpret_cast<const uint32_t*>(&x)[s], b0, b1);
  }
};

// The warps' sums of a CTA: part[warp][token][row], then row r of token t of all of them.
template <int RT, int NT>
__device__ __forceinline__ void put_part(float* part, const float (&acc)[RT][NT][4]) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  float* to = part + warp * (RT * 16 * NT * 8);
#pragma unroll
  for (int rt = 0; rt < RT; ++rt)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        to[(8 * nt + 2 * c + (i & 1)) * (16 * RT) + 16 * rt + 8 * (i >> 1) + g] = acc[rt][nt][i];
}
template <int RT, int NT>
__device__ __forceinline__ float sum_parts(const float* part, int warps, int token, int row) {
  float v = 0.f;
  for (int w = 0; w < warps; ++w)
    v += part[w * (RT * 16 * NT * 8) + token * (16 * RT) + row];
  return v;
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
