// The gradient of the 8-bit product's input: dq4_int8_linear_backward (dq4_int8.h).
#include "int8.cuh"

namespace dq4d {
namespace {

constexpr int kThreadsBack = 128, kRowsBack = 8;

struct BackArgs {
  const void* dY;
  bool bf16;
  const int8_t* CB;
  const float* SCB;
  int64_t M, N, K;
  void* dX;
};

// A thread a column of dX, 8 rows of it.
__global__ void __launch_bounds__(kThreadsBack) dq4_int8_backward_kernel(const BackArgs p) {
  wait_for_stream();
  const int64_t k = int64_t(blockIdx.x) * kThreadsBack + threadIdx.x;
  if (k >= p.K) return;
  for (int64_t m0 = int64_t(blockIdx.y) * kRowsBack; m0 < p.M; m0 += int64_t(gridDim.y) * kRowsBack) {
    float sum[kRowsBack] = {};
    for (int64_t n = 0; n < p.N; ++n) {
      float w = __fmul_rn(__fmul_rn(float(p.CB[n * p.K + k]), p.SCB[n]), kRecip127);
      w = p.bf16 ? __bfloat162float(__float2bfloat16_rn(w)) : __half2float(__float2half_rn(w));
#pragma unroll
      for (int i = 0; i < kRowsBack; ++i)
        if (m0 + i < p.M) sum[i] = fmaf(load_16(p.dY, (m0 + i) * p.N + n, p.bf16), w, sum[i]);
    }
#pragma unroll
    for (int i = 0; i < kRowsBack; ++i)
      if (m0 + i < p.M)
        store_any(p.dX, (m0 + i) * p.K + k, sum[i], p.bf16 ? DQ4_OUT_BF16 : DQ4_OUT_F16);
  }
}

}  // namespace
}  // namespace dq4d

using namespace dq4d;

extern "C" {

int64_t dq4_int8_linear_backward_workspace_bytes(int64_t M, int64_t N, int64_t K) { return 0; }

int dq4_int8_linear_backward(const void* dY, int32_t dtype, const int8_t* CB, const float* SCB,
                             int64_t M, int64_t N, int64_t K, void* dX, void* workspace,
                             int64_t workspace_bytes, int* bad, void* stream) {
  if (M < 0 || N < 0 || K < 0 || M > INT32_MAX || N > INT32_MAX || K > INT32_MAX || K % 16 != 0 ||
      N % 8 != 0 || M * N >= int64_t(1) << 47 || N * K >= int64_t(1) << 47 ||
      M * K >= int64_t(1) << 47)
    return DQ4_ERR_N;
  if (!valid_dtype(dtype, false)) return DQ4_ERR_DTYPE;
  if (M == 0 || K == 0) return DQ4_OK;
  if (!dX || (N > 0 && (!dY || !CB || !SCB))) return DQ4_ERR_NULL;
  if (misaligned(dY, 16) || misaligned(CB, 16) || misaligned(SCB, 4) || misaligned(dX, 2) ||
      misaligned(bad, 4))
    return DQ4_ERR_ALIGN;
  int dev, sms;
  if (const int st = current_device(&dev, &sms)) return st;
  const BackArgs p = {dY, dtype == DQ4_OUT_BF16, CB, SCB, M, N, K, dX};
  const int64_t y = (M + kRowsBack - 1) / kRowsBack;
  const dim3 grid(unsigned((K + kThreadsBack - 1) / kThreadsBack), unsigned(y < 65535 ? y : 65535));
  return launch_ordered(dq4_int8_backward_kernel, grid, kThreadsBack, 0,
                        static_cast<cudaStream_t>(stream), p);
}

}  // extern "C"
