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
// summed in FP32), so that a weight 2^-24 of the largest still has all its bits and one down
// to 2^-38 is not lost.
constexpr float kLift = 14.f;

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
  return p.window > 0 ? max(0, pos - p.window + 1) : 0;
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

// The power of two that brings a row's largest magnitude into [2^14, 2^15), and its inverse.
// FP16 then holds a BF16 or FP16 row as it is, but for values below 2^-38 of its largest.
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
