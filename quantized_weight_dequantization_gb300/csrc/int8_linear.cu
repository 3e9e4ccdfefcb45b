// The product of rows in 8 bits with a weight in 8 bits, dq4_int8_linear (dq4_int8.h): the entry
// point, and the kernel for few rows.
//
// Few rows are bound by the weight's bytes, each read once: a CTA takes 16 RT weight rows, its
// warps take turns at chunks of 64 of K, and all operands go from global memory to registers
// (the rows' codes come from L2, and all CTAs read the same).  Outlier columns are added in FP32.
#include "int8_gemm.cuh"

namespace dq4d {
namespace {

constexpr int kWarps = 8;

// Whether entry l of the columns is used: in range and above all before it.
struct Columns {
  int64_t top = -1;
  int bad = 0;
  __device__ __forceinline__ bool next(int64_t c, int64_t K) {
    if (c > top && c < K) {
      top = c;
      return true;
    }
    bad += c != -1;
    return false;
  }
};

template <int RT, int NT, int U>
__global__ void __launch_bounds__(32 * kWarps, 2) dq4_int8_few_kernel(const Int8Linear p) {
  constexpr int kRows = 16 * RT, kTokens = 8 * NT;
  __shared__ float s_part[kWarps * kRows * kTokens];
  wait_for_stream();
  asm volatile("griddepcontrol.launch_dependents;");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const int64_t n0 = int64_t(blockIdx.x) * kRows, m0 = int64_t(blockIdx.y) * kTokens;
  const int8_t* row[RT][2];
#pragma unroll
  for (int rt = 0; rt < RT; ++rt)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int64_t n = n0 + 16 * rt + 8 * h + g;
      row[rt][h] = n < p.N ? p.CB + n * p.K + 16 * c : nullptr;
    }
  CodeTokens<NT> src;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int64_t m = m0 + 8 * nt + g;
    src.at[nt] = m < p.M ? p.codes + m * p.K + 16 * c : nullptr;
  }
  float acc[RT][NT][4] = {};
  warp_product<RT, NT, U>(acc, row, src, p.K, warp, kWarps, int((p.K + 63) / 64));
  put_part<RT, NT>(s_part, acc);
  __syncthreads();
  for (int i = threadIdx.x; i < kRows * kTokens; i += 32 * kWarps) {
    const int64_t n = n0 + i % kRows, m = m0 + i / kRows;
    if (n >= p.N || m >= p.M) continue;
    float sum = sum_parts<RT, NT>(s_part, kWarps, i / kRows, i % kRows);
    const float sn = load_global(p.SCB + n) * kRecip127;
    const float sm = load_global(p.scales + m) * kRecip127;
    float y = 0.f;
    if (p.L > 0) {
      Columns used;
      float more = 0.f;
      for (int l = 0; l < p.L; ++l) {
        const int64_t k = load_global(p.cols + l);
        if (!used.next(k, p.K)) continue;
        const float w = p.CB[n * p.K + k], x = load_16(p.outliers, m * p.L + l, p.outliers_bf16);
        sum -= w * float(p.codes[m * p.K + k]);
        more += x * w + (x - x);  // (not finite: NaN)
      }
      y = more * sn;
      if (i == 0 && blockIdx.x == 0 && blockIdx.y == 0 && used.bad && p.bad)
        atomicAdd(p.bad, used.bad);
    }
    y += sum * sm * sn;
    if (p.bias) y += load_any(p.bias, n, p.out_dtype);
    store_any(p.Y, m * p.N + n, y, p.out_dtype);
  }
}

// Whether a product goes to the kernel for few rows.
bool few_rows(int64_t M, int64_t K) { return M <= 32 || K == 0; }

template <int RT, int NT, int U>
int launch_few(const Int8Linear& p, cudaStream_t stream) {
  const dim3 grid(unsigned((p.N + 16 * RT - 1) / (16 * RT)), unsigned((p.M + 8 * NT - 1) / (8 * NT)));
  return launch_ordered(dq4_int8_few_kernel<RT, NT, U>, grid, 32 * kWarps, 0, stream, p);
}

}  // namespace
}  // namespace dq4d

using namespace dq4d;

extern "C" {

int64_t dq4_int8_linear_workspace_bytes(int64_t M, int64_t N, int64_t K, int32_t L) {
  if (M <= 0 || N <= 0 || K < 0 || L < 0 || L > kMaxOutliers || M > INT32_MAX || N > INT32_MAX ||
      K > INT32_MAX || few_rows(M, K))
    return 0;
  int dev, sms;
  if (current_device(&dev, &sms) != DQ4_OK) return -DQ4_ERR_DEVICE;
  return int8_gemm_workspace(M, N, K, L, sms);
}

int dq4_int8_linear(const int8_t* codes, const float* scales, const int8_t* CB, const float* SCB,
                    int64_t M, int64_t N, int64_t K, const int64_t* cols, int32_t L,
                    const void* outliers, int32_t outlier_dtype, const void* bias,
                    int32_t out_dtype, void* Y, void* workspace, int64_t workspace_bytes,
                    int* bad, void* stream) {
  if (M < 0 || N < 0 || K < 0 || M > INT32_MAX || N > INT32_MAX || K > INT32_MAX || K % 16 != 0 ||
      L < 0 || L > kMaxOutliers || M * K >= int64_t(1) << 47 || N * K >= int64_t(1) << 47)
    return DQ4_ERR_N;
  if (!valid_dtype(out_dtype, true) || (L > 0 && !valid_dtype(outlier_dtype, false)))
    return DQ4_ERR_DTYPE;
  if (M == 0 || N == 0) return DQ4_OK;
  if (!scales || !SCB || !Y || (K > 0 && (!codes || !CB)) || (L > 0 && (!cols || !outliers)))
    return DQ4_ERR_NULL;
  if (misaligned(codes, 16) || misaligned(CB, 16) || misaligned(scales, 4) ||
      misaligned(SCB, 4) || misaligned(cols, 8) || misaligned(outliers, 2) ||
      misaligned(bias, out_itemsize(out_dtype)) || misaligned(Y, out_itemsize(out_dtype)) ||
      misaligned(bad, 4))
    return DQ4_ERR_ALIGN;
  int dev, sms;
  if (const int st = current_device(&dev, &sms)) return st;
  const Int8Linear p = {codes, scales, CB, SCB, M, N, K, cols, outliers, L,
                        L > 0 && outlier_dtype == DQ4_OUT_BF16, bias, out_dtype, Y, bad};
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (!few_rows(M, K)) {
    if (!workspace || workspace_bytes < int8_gemm_workspace(M, N, K, L, sms))
      return DQ4_ERR_WORKSPACE;
    if (misaligned(workspace, 256)) return DQ4_ERR_ALIGN;
    return launch_int8_gemm(p, dev, sms, workspace, s);
  }
  if (M <= 8) return launch_few<1, 1, 4>(p, s);
  if (M <= 16) return launch_few<1, 2, 4>(p, s);
  return launch_few<2, 4, 2>(p, s);
}

}  // extern "C"
