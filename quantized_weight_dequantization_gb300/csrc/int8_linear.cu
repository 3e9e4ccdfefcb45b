// The product of rows in 8 bits with a weight in 8 bits, dq4_int8_linear (dq4_int8.h): the entry
// point, and the kernel for few rows.
//
// Few rows are bound by the weight's bytes, each read once (Streamed in int8.cuh; the rows' codes
// come from L2, and all CTAs read the same).  Outlier columns are added in FP32.
#include "int8_gemm.cuh"

namespace dq4d {
namespace {

// The outlier columns of a call, in shared memory.
struct FewColumns {
  int count;
  int entry[kMaxOutliers], col[kMaxOutliers];
};

// The columns among cols[0 .. L) that are used: in range and above all before them.  One warp.
__device__ __forceinline__ void list_columns(const Int8Linear& p, FewColumns* s) {
  const int lane = threadIdx.x & 31;
  int64_t top = -1;
  int n = 0, wrong = 0;
  for (int l0 = 0; l0 < p.L; l0 += 32) {
    const int64_t c = l0 + lane < p.L ? load_global(p.cols + l0 + lane) : -1;
    int64_t run = c < p.K ? c : -1;  // the largest so far, this one's included
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t up = __shfl_up_sync(kAllLanes, run, o);
      if (lane >= o && up > run) run = up;
    }
    int64_t before = __shfl_up_sync(kAllLanes, run, 1);
    before = lane == 0 || before < top ? top : before;
    const bool use = c > before && c < p.K && c >= 0;
    const unsigned hits = __ballot_sync(kAllLanes, use);
    if (use) {
      const int at = n + __popc(hits & ((1u << lane) - 1));
      s->entry[at] = l0 + lane;
      s->col[at] = int(c);
    }
    n += __popc(hits);
    wrong += __popc(__ballot_sync(kAllLanes, !use && c != -1));
    const int64_t last = __shfl_sync(kAllLanes, run, 31);
    if (last > top) top = last;
  }
  if (lane == 0) {
    s->count = n;
    if (wrong && p.bad && blockIdx.x == 0) atomicAdd(p.bad, wrong);
  }
}

template <int RT, int NT, int kDepth>
struct FewJobs {
  using S = Streamed<RT, NT, 1, 2, false, kDepth>;
  static constexpr int kRows = 16 * RT, kTokens = 8 * NT;
  static constexpr int kAhead = 4;  // outlier codes of a row loaded ahead
  const Int8Linear& p;
  FewColumns* s;
  float* coef;  // [used columns][M]: what a column's codes have to be multiplied by
  int64_t tiles_m;  // (more than one only without codes, K = 0)
  float sn, bias;   // of this thread's row
  uint32_t ahead[kAhead];

  __device__ __forceinline__ int64_t row_of(int64_t job, int t, int64_t& m0) const {
    const int64_t tn = tiles_m == 1 ? job : job / tiles_m;
    m0 = (job - tn * tiles_m) * kTokens;
    return tn * kRows + t % kRows;
  }
  __device__ __forceinline__ void places(int64_t job, int (&y)[1]) const { y[0] = int(job * kRows); }
  __device__ __forceinline__ void tokens(int64_t, const uint8_t* (&tok)[NT]) const {
    const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
      tok[nt] = reinterpret_cast<const uint8_t*>(p.codes + min(int64_t(8 * nt + g), p.M - 1) * p.K +
                                                 32 * c);
  }
  __device__ __forceinline__ void start() {
    if (p.L == 0) return;
    if (threadIdx.x < 32) list_columns(p, s);
    __syncthreads();
    const int n = s->count * int(p.M);
    for (int i = threadIdx.x; i < n; i += kStreamThreads) {
      const int u = i / int(p.M), m = i - u * int(p.M);
      const float x = load_16(p.outliers, int64_t(m) * p.L + s->entry[u], p.outliers_bf16);
      const float code = p.codes[m * p.K + s->col[u]];
      // in the place of its code's value; not finite: NaN
      coef[i] = x + (x - x) - code * (load_global(p.scales + m) * kRecip127);
    }
    __syncthreads();
  }
  __device__ __forceinline__ void begin(int64_t job, int t) {
    int64_t m0;
    const int64_t n = min(row_of(job, t, m0), p.N - 1);
    sn = load_ahead(p.SCB + n);
    bias = p.bias ? load_any(p.bias, n, p.out_dtype) : 0.f;
    if (p.L > 0) {
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        ahead[u] = 0;
        if (u < s->count)
          asm volatile("ld.global.s8 %0, [%1];"
                       : "=r"(ahead[u]) : "l"(p.CB + n * p.K + s->col[u]) : "memory");
      }
    }
  }
  __device__ __forceinline__ void finish(int64_t job, const float* part, int warps, int t,
                                         int threads) const {
    int64_t m0;
    const int64_t n = row_of(job, t, m0);  // (a thread's outputs are all of one row)
    if (n >= p.N) return;
    const float s_n = sn * kRecip127;
#pragma unroll 2
    for (int j = t / kRows; j < kTokens && m0 + j < p.M; j += threads / kRows) {
      const float s_m = load_global(p.scales + m0 + j) * kRecip127;
      float y = S::sum(part, warps, j, t % kRows) * s_m * s_n;
      if (p.L > 0) {
        float more = 0.f;
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
          if (u < s->count) more += float(int(ahead[u])) * coef[u * int(p.M) + j];
        for (int u = kAhead; u < s->count; ++u)
          more += float(load_global(p.CB + n * p.K + s->col[u])) * coef[u * int(p.M) + j];
        y += more * s_n;
      }
      store_any(p.Y, (m0 + j) * p.N + n, y + bias, p.out_dtype);
    }
  }
};

template <int RT, int NT, int kDepth, int kCtas>
__global__ void __launch_bounds__(kStreamThreads, kCtas)
    dq4_int8_few_kernel(const __grid_constant__ CUtensorMap map_w, const Int8Linear p) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ FewColumns s_cols;
  using Jobs = FewJobs<RT, NT, kDepth>;
  uint8_t* smem = aligned_1024(smem_raw);
  Jobs::S::setup(smem);
  wait_for_stream();
  asm volatile("griddepcontrol.launch_dependents;");
  Jobs jobs = {p, &s_cols, reinterpret_cast<float*>(smem + Jobs::S::kBytes),
               (p.M + 8 * NT - 1) / (8 * NT)};
  Jobs::S::run(jobs, smem, (p.N + 16 * RT - 1) / (16 * RT) * jobs.tiles_m, p.K, map_w, p.bad);
}

// Whether a product goes to the kernel for few rows.
bool few_rows(int64_t M, int64_t K) { return M <= 32 || K == 0; }

template <int RT, int NT, int kDepth, int kCtas>
int launch_few(const Int8Linear& p, int dev, int sms, cudaStream_t stream) {
  auto kernel = dq4_int8_few_kernel<RT, NT, kDepth, kCtas>;
  constexpr int kRings = FewJobs<RT, NT, kDepth>::S::kBytes + 1024;
  constexpr int kMost = kRings + 8 * NT * kMaxOutliers * 4;
  static_assert(kMost + int(sizeof(FewColumns)) + 1024 <= 227 * 1024, "shared memory");
  CUtensorMap w = {};  // (without codes, K = 0, nothing is copied)
  if (p.K > 0)
    if (const int st = encode_2d(&w, CU_TENSOR_MAP_DATA_TYPE_UINT8, p.CB, p.K, p.N, p.K, kChunk,
                                 16 * RT, CU_TENSOR_MAP_SWIZZLE_128B))
      return st;
  static std::atomic<uint64_t> allowed{0};
  if (const int st = allow_smem(kernel, kMost, dev, &allowed)) return st;
  const int bytes = kRings + (p.M <= 8 * NT ? int(p.M) * p.L * 4 : 0);
  const int64_t jobs = (p.N + 16 * RT - 1) / (16 * RT) * ((p.M + 8 * NT - 1) / (8 * NT));
  // (a CTA takes a job at least)
  const int64_t grid = jobs < kCtas * sms ? jobs : kCtas * sms;
  return launch_ordered(kernel, dim3(unsigned(grid)), kStreamThreads, bytes, stream, w, p);
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
  if (M <= 8) return launch_few<1, 1, 4, 3>(p, dev, sms, s);
  if (M <= 16) return launch_few<1, 2, 4, 3>(p, dev, sms, s);
  return launch_few<2, 4, 2, 2>(p, dev, sms, s);
}

}  // extern "C"
