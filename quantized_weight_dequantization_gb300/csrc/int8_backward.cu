// The gradient of the 8-bit product's input, dq4_int8_linear_backward (dq4_int8.h): the entry
// point.  The kernel is the product's (int8_gemm.cu, with what it measured), the weight's columns
// its rows: the sum runs over the weight's rows, whose scales go into its 16-bit values.
#include "int8_gemm.cuh"

using namespace dq4d;

extern "C" {

int64_t dq4_int8_linear_backward_workspace_bytes(int64_t M, int64_t N, int64_t K) {
  if (M <= 0 || N <= 0 || K <= 0 || M > INT32_MAX || N > INT32_MAX || K > INT32_MAX) return 0;
  int dev, sms;
  if (current_device(&dev, &sms) != DQ4_OK) return -DQ4_ERR_DEVICE;
  return int8_backward_workspace(M, N, K, sms);
}

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
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (N == 0) {
    const cudaError_t e = cudaMemsetAsync(dX, 0, size_t(M) * size_t(K) * 2, s);
    return e == cudaSuccess ? DQ4_OK : fail_cuda(DQ4_ERR_LAUNCH, e);
  }
  if (!workspace || workspace_bytes < int8_backward_workspace(M, N, K, sms))
    return DQ4_ERR_WORKSPACE;
  if (misaligned(workspace, 256)) return DQ4_ERR_ALIGN;
  const Int8Backward p = {dY, dtype == DQ4_OUT_BF16, CB, SCB, M, N, K, dX, bad};
  return launch_int8_backward(p, dev, sms, workspace, s);
}

}  // extern "C"
