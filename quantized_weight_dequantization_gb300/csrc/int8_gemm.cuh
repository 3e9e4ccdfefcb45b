// The tcgen05 products of the layers with 8-bit weights (int8_gemm.cu), as the entry points call
// them.
#pragma once

#include "int8.cuh"

namespace dq4d {

struct Int8Backward {
  const void* dY;  // [M][N]
  bool bf16;
  const int8_t* CB;  // [N][K]
  const float* SCB;
  int64_t M, N, K;
  void* dX;  // [M][K]
  int* bad;
};

int64_t int8_gemm_workspace(int64_t M, int64_t N, int64_t K, int L, int sms);
int launch_int8_gemm(const Int8Linear& a, int dev, int sms, void* workspace, cudaStream_t stream);
int64_t int8_backward_workspace(int64_t M, int64_t N, int64_t K, int sms);
int launch_int8_backward(const Int8Backward& a, int dev, int sms, void* workspace,
                         cudaStream_t stream);

}  // namespace dq4d
