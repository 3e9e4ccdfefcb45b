// What the two attention kernels over the 8-bit cache share: their arguments, a sequence's
// keys in sight, the scaling of query rows to FP16, and the softmax in base 2.
#pragma once

#include "kv8.cuh"
#include "tcgen05.cuh"
#include "tmap.cuh"

namespace dq4d {

struct AttendArgs {
  Kv8 c;
  Batch s;
  const void* q;
  int64_t token_stride, head_stride;
  int heads, group;  // query heads, and of them per kv head
  bool bf16;         // q and out: BF16 or FP16
  float scale_log2;  // softmax scale times log2(e)
  int causal, window;
  void* out;
  float* lse;
  int* bad;
  int* count;        // few rows: arrivals at a shared item
  float* part;       // few rows: unnormalized rows of parts of items,
  float2* stats;     // and their {m, l}
};

namespace {

// The head of the workspace: arrival counters, of either kernel, zero between calls.
constexpr int64_t kCounterBytes = 2048;

constexpr float kMinScale = 7.888609052210118e-31f;  // 2^-100, the least scale append writes
constexpr float kLn2 = 0.6931471805599453f;

// Weights are 2^(s - m + kLift): the largest sits near the top of FP16's range (V's codes are
// summed in FP32), so that a weight 2^-28 of the largest still has all its bits and one down
// to 2^-38 is not lost.
constexpr float kLift = 14.f;

// The sum l of the weights over the pages' V scales is held in units of 2^16.  A weight is below
// 2^16 and a scale 2^-100 to 2^120, so that 2^27 keys at the least scale stay below 2^128 (they
// are log n in lse), and the largest weight of a row alone, 2^14 (few rows) or 2^10 at least
// (many), is 2^-126 or more at the largest scale.
constexpr float kSumUnit = 1.f / 65536;
constexpr float kLogSumUnit = 16 * kLn2;

// The factor of O that makes a row's result, and its log-sum: of sum l, with weights 2^(x - ref).
__device__ __forceinline__ float inverse_sum(float l) { return l == 0.f ? 0.f : kSumUnit / l; }
__device__ __forceinline__ float log_sum(float ref, float l) {
  return l == 0.f ? -INFINITY : fmaf(ref, kLn2, logf(l) + kLogSumUnit);
}

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// A scale as it is used: not below the least (a page of zeros), NaN kept.
__device__ __forceinline__ float used_scale(float s) { return s < kMinScale ? kMinScale : s; }

// The keys of a sequence that are there: its length, or the table's width in tokens.
__device__ __forceinline__ int held_keys(const AttendArgs& p, int len) {
  const int64_t most = int64_t(p.s.table_width) << p.c.log2_page;
  return len < most ? max(len, 0) : int(most);
}

// The keys [lo, hi) that a query at position pos sees.
__device__ __forceinline__ int first_key(const AttendArgs& p, int pos) {
  return p.window > 0 && pos >= p.window ? pos - p.window + 1 : 0;
}
__device__ __forceinline__ int last_key(const AttendArgs& p, int pos, int held) {
  return p.causal ? min(held, pos + 1) : held;
}

// Two 16-bit values of q as floats.
__device__ __forceinline__ void widen2(uint32_t u, bool bf16, float& a, float& b) {
  if (bf16) {
    a = __uint_as_float(u << 16);
    b = __uint_as_float(u & 0xFFFF0000u);
  } else {
    __half2 h;
    memcpy(&h, &u, 4);
    a = __low2float(h);
    b = __high2float(h);
  }
}

// Codes that are no numbers among four e4m3 codes: 0x80 in the byte of each.
__device__ __forceinline__ uint32_t nan_codes(uint32_t w) {
  return ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
}
__device__ __forceinline__ uint32_t nan_codes(uint4 v) {
  return nan_codes(v.x) | nan_codes(v.y) | nan_codes(v.z) | nan_codes(v.w);
}
// The same codes with zeros in their place.
__device__ __forceinline__ uint4 without_nan(uint4 v) {
  auto clean = [](uint32_t w) { return w & ~((nan_codes(w) >> 7) * 0xFFu); };
  return make_uint4(clean(v.x), clean(v.y), clean(v.z), clean(v.w));
}

// The same of two FP16 values, 0x8000 in the place of each; and their larger values, or NaN.
__device__ __forceinline__ uint32_t nan_halves(uint32_t w) {
  return ((w & 0x7FFF7FFFu) + 0x03FF03FFu) & 0x80008000u;
}
__device__ __forceinline__ uint32_t larger_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// The keys lo <= key + i < hi of 64, one bit each.
__device__ __forceinline__ uint64_t seen_keys(int key, int lo, int hi) {
  const int a = max(lo - key, 0), b = min(hi - key, 64);
  return a < b ? ~uint64_t(0) >> (64 - (b - a)) << a : 0;
}

constexpr uint32_t kNaN = 0x7FC00000u;

// The power of two that brings a row's largest magnitude into [2^14, 2^15), and its inverse.
// FP16 then holds a BF16 row as it is down to 2^-31 of its largest, an FP16 row down to 2^-28;
// smaller values are rounded to 2^-38 of it, below what the FP32 sum of the products holds.
// A row with an infinity or a NaN gets a NaN inverse.
__device__ __forceinline__ void row_scaling(float top, float& up, float& down) {
  const int e = int(__float_as_uint(top) >> 23);  // biased; 0 also for subnormal rows
  // 2^k and 2^-k both normal: only rows whose largest is below 2^-112 miss the range
  const int k = min(max(14 - (e - 127), -126), 126);
  up = __uint_as_float(uint32_t(k + 127) << 23);
  down = __uint_as_float(uint32_t(127 - k) << 23);
  if (!(top < INFINITY)) down = __uint_as_float(0x7FC00000u);
}

__device__ __forceinline__ uint32_t pack_f16(float a, float b) { return pack2<DQ4_OUT_F16>(a, b); }

__device__ __forceinline__ uint32_t pack_out(float a, float b, bool bf16) {
  return bf16 ? pack2<DQ4_OUT_BF16>(a, b) : pack2<DQ4_OUT_F16>(a, b);
}

// Two e4m3 codes (the low 16 bits of w) as FP16.
__device__ __forceinline__ uint32_t f16_of_e4m3(uint32_t w) {
  uint32_t r;
  asm("{\n.reg .b16 lo, hi;\nmov.b32 {lo, hi}, %1;\ncvt.rn.f16x2.e4m3x2 %0, lo;\n}"
      : "=r"(r) : "r"(w));
  return r;
}
__device__ __forceinline__ uint32_t f16_of_e4m3_high(uint32_t w) {
  uint32_t r;
  asm("{\n.reg .b16 lo, hi;\nmov.b32 {lo, hi}, %1;\ncvt.rn.f16x2.e4m3x2 %0, hi;\n}"
      : "=r"(r) : "r"(w));
  return r;
}

__device__ __forceinline__ void sts_v4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c,
                                       uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};"
               :: "r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
__device__ __forceinline__ void sts_b32(uint32_t addr, uint32_t v) {
  asm volatile("st.shared.b32 [%0], %1;" :: "r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ uint32_t lds_b32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}
__device__ __forceinline__ void sts_v4(uint32_t addr, const uint4& v) {
  sts_v4(addr, v.x, v.y, v.z, v.w);
}

}  // namespace

// The two kernels (kv8_decode.cu, kv8_prefill.cu).
// rows: query rows a kv head; keys: the most that a sequence holds or sees (estimates, both)
int launch_decode(const AttendArgs& p, int head_dim, int64_t rows, int64_t keys, int dev, int sms,
                  void* workspace, cudaStream_t stream);
int64_t decode_workspace_bytes();
int launch_prefill(const AttendArgs& p, int head_dim, int dev, int sms, void* workspace,
                   cudaStream_t stream);
int64_t prefill_workspace_bytes(int64_t tokens, int64_t seqs, int64_t group, int head_dim);

}  // namespace dq4d
