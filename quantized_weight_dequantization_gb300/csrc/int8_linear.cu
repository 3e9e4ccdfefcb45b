// The product of rows in 8 bits with a weight in 8 bits, dq4_int8_linear (dq4_int8.h): the entry
// point, and the kernel for few rows.
//
// Few rows are bound by the weight's bytes, each read once, by TMA, and multiplied on the tensor
// cores in FP16 (the integer products of four, dp4a, run at 16 lanes a clock here: 1 row took 41
// us at 28672 x 8192, 4 rows 91).  Outlier columns are added in FP32.
// One row through 4096 x 4096: 5.5 us, of which the bytes take 2.5 and a launch with its first
// copies 2.5; 8 rows with 5 outlier columns and bias through 4096 x 11008: 13.1 of 6.7; 8 rows
// through 8192 x 28672: 0.68 of the copy rate (a cold run under a profiler).
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

constexpr int kFewRows = 16;  // weight rows of a job
constexpr int kAhead = 4;     // outlier columns whose codes are loaded ahead

// A job is 16 weight rows and 8 NT tokens (all there are), shared by `group` warps of a CTA, which
// take turns at chunks of 128 of K; one job a group, so that there is little code to fetch (with
// jobs in turn, as in int8_moe.cu, a call took 4 to 5 us more).  The order of K in a product is
// free: lane (g, c) takes 32 consecutive codes of rows g and g + 8, and of token g of each 8.
template <int NT, int kFewDepth>
__global__ void __launch_bounds__(kStreamThreads, kFewDepth == 2 && NT < 4 ? 3 : 2)
    dq4_int8_few_kernel(const __grid_constant__ CUtensorMap map_w, const Int8Linear p,
                        const int group) {
  constexpr int kTokens = 8 * NT, kStage = kFewRows * kChunk;
  extern __shared__ uint8_t smem_raw[];
  __shared__ FewColumns s_cols;
  __shared__ uint64_t s_bars[kStreamWarps][kFewDepth];
  __shared__ float s_part[kStreamWarps][kFewRows * kTokens];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const int in_cta = warp / group, member = warp - in_cta * group;
  const int64_t n0 = (int64_t(blockIdx.x) * (kStreamWarps / group) + in_cta) * kFewRows;
  uint8_t* rings = aligned_1024(smem_raw);
  // (the outliers, with the codes in whose place they are, go where the rings were: with a place of
  // their own an SM held two CTAs in place of three, 16 rows with 5 outlier columns through 4096 x
  // 11008 took 20.6 us)
  float2* coef = reinterpret_cast<float2*>(rings);
  static_assert(kTokens * kMaxOutliers * 8 <= kStreamWarps * kFewDepth * kStage, "factors fit");
  const uint32_t ring = smem_u32(rings) + warp * kFewDepth * kStage, bars = smem_u32(s_bars[warp]);
  const uint64_t map = reinterpret_cast<uint64_t>(&map_w);
  // this warp's chunks, member + i * group for i < mine, in turn from `i0` on: warps that went
  // through the tokens side by side would queue at single lines of L2
  const int chunks = n0 < p.N ? int((p.K + kChunk - 1) / kChunk) : 0;
  const int mine = chunks > member ? (chunks - member + group - 1) / group : 0;
  const int i0 = mine > 0 ? int((uint32_t(n0) / kFewRows) % uint32_t(mine)) : 0;
  auto chunk = [&](int i) { return member + (i0 + i < mine ? i0 + i : i0 + i - mine) * group; };
  if (lane == 0) {
    for (int i = 0; i < kFewDepth; ++i) mbar_init(bars + 8 * i, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    // the first chunks to L2, while the kernel before this one ends (nothing is read of them yet)
#pragma unroll 1
    for (int i = 0; i < kFewDepth && i < mine; ++i)
      asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global [%0, {%1, %2}];"
                   :: "l"(map), "r"(chunk(i) * kChunk), "r"(int(n0)) : "memory");
  }
  wait_for_stream();
  asm volatile("griddepcontrol.launch_dependents;");
  auto copy = [&](int i, int slot) {
    mbar_expect(bars + 8 * slot, kStage);
    tma_load_2d(ring + slot * kStage, map, chunk(i) * kChunk, int(n0), bars + 8 * slot);
  };
  if (lane == 0)
#pragma unroll 1
    for (int i = 0; i < kFewDepth && i < mine; ++i) copy(i, i);
  __syncwarp();
  // the outputs that this thread finishes are all of one row
  const int t = 32 * member + lane, threads = 32 * group;
  const int64_t n = n0 + t % kFewRows, n_in = min(n, p.N - 1);
  const float sn = load_ahead(p.SCB + n_in);
  uint32_t ahead[kAhead];
  int used = 0;
  const int8_t* tok[NT];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
    tok[nt] = p.codes + min(int64_t(8 * nt + g), p.M - 1) * p.K + 32 * c;
  float acc[NT][4] = {};
  bool ok = true;
  int slot = 0, i = 0;
  uint32_t phase = 0;
  // the tokens' codes, from L2, a chunk ahead
  uint4 next[NT][2];
  auto fetch = [&](int i) {
    const int64_t k = int64_t(chunk(i)) * kChunk;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        next[nt][h] = make_uint4(0, 0, 0, 0);
        if (i < mine && k + 32 * c + 16 * h < p.K)
          next[nt][h] = load_ahead(reinterpret_cast<const uint4*>(tok[nt] + k) + h);
      }
  };
  fetch(0);
  if (p.L > 0 && warp == 0) list_columns(p, &s_cols);  // (while the first codes are on their way)
#pragma unroll 1
  for (; i < mine; ++i) {
    uint4 x[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      x[nt][0] = next[nt][0];
      x[nt][1] = next[nt][1];
    }
    fetch(i + 1);
    ok = __all_sync(kAllLanes, mbar_wait(bars + 8 * slot, phase));
    if (!ok) break;
    const uint32_t at = ring + slot * kStage + g * kChunk;
#pragma unroll
    for (int h = 0; h < 2; ++h) {  // 128-byte rows, their 16-byte pieces in place i ^ row % 8
      const uint4 w0 = lds_v4(at + (((2 * c + h) ^ g) << 4));
      const uint4 w1 = lds_v4(at + 8 * kChunk + (((2 * c + h) ^ g) << 4));
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        uint32_t a0, a1, a2, a3;
        codes_f16(reinterpret_cast<const uint32_t*>(&w0)[s], a0, a2);
        codes_f16(reinterpret_cast<const uint32_t*>(&w1)[s], a1, a3);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          uint32_t b0, b1;
          codes_f16(reinterpret_cast<const uint32_t*>(&x[nt][h])[s], b0, b1);
          mma_16816(acc[nt], a0, a1, a2, a3, b0, b1);
        }
      }
    }
    __syncwarp();  // every lane has read the chunk
    if (lane == 0 && i + kFewDepth < mine) copy(i + kFewDepth, slot);
    if (++slot == kFewDepth) {
      slot = 0;
      phase ^= 1u;
    }
  }
  if (!ok) {  // copies in flight land before the CTA leaves
    if (lane == 0 && p.bad) atomicAdd(p.bad, 1);
    for (int k = 0; k < kFewDepth && i < mine; ++k, ++i) {
      mbar_wait(bars + 8 * slot, phase);
      if (++slot == kFewDepth) {
        slot = 0;
        phase ^= 1u;
      }
    }
  }
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      s_part[warp][(8 * nt + 2 * c + (i & 1)) * kFewRows + 8 * (i >> 1) + g] = acc[nt][i];
  if (p.L > 0) {
    __syncthreads();
    used = s_cols.count;
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      ahead[u] = 0;
      if (u < used)
        asm volatile("ld.global.s8 %0, [%1];"
                     : "=r"(ahead[u]) : "l"(p.CB + n_in * p.K + s_cols.col[u]) : "memory");
    }
    for (int i = threadIdx.x; i < used * int(p.M); i += kStreamThreads) {
      const int u = i / int(p.M), m = i - u * int(p.M);
      const float x = load_16(p.outliers, int64_t(m) * p.L + s_cols.entry[u], p.outliers_bf16);
      // (not finite: NaN)
      coef[i] = make_float2(x + (x - x), float(load_global(p.codes + m * p.K + s_cols.col[u])));
    }
    __syncthreads();
  } else if (group == 1) {
    __syncwarp();
  } else {
    asm volatile("bar.sync %0, %1;" :: "r"(1 + in_cta), "r"(threads) : "memory");
  }
  if (n >= p.N) return;
  const float s_n = sn * kRecip127;
  const float bias = p.bias ? load_any(p.bias, n, p.out_dtype) : 0.f;
#pragma unroll 1
  for (int m = t / kFewRows; m < p.M; m += threads / kFewRows) {
    float sum = 0.f;
    if (m < kTokens)  // (more rows only without codes, K = 0)
      for (int w = 0; w < group; ++w)
        sum += s_part[in_cta * group + w][m * kFewRows + t % kFewRows];
    // (the weight's scale first: rows may be near FP32's largest number, their results not)
    const float s_m = load_global(p.scales + m) * kRecip127;
    float y;
    if (used > 0) {
      float more = 0.f, instead = 0.f;  // the outliers' sum, and that of the codes where they are
      auto add = [&](int u, float w) {
        const float2 x = coef[u * int(p.M) + m];
        more += w * s_n * x.x;
        instead += w * x.y;
      };
#pragma unroll
      for (int u = 0; u < kAhead; ++u)
        if (u < used) add(u, float(int(ahead[u])));
      for (int u = kAhead; u < used; ++u)
        add(u, float(load_global(p.CB + n * p.K + s_cols.col[u])));
      // (whole numbers, sum and instead: their difference is as exact as the sum)
      y = (sum - instead) * s_n * s_m + more;
    } else {
      y = sum * s_n * s_m;
    }
    store_any(p.Y, m * p.N + n, y + bias, p.out_dtype);
  }
}

// Whether a product goes to the kernel for few rows: up to 16, and up to 32 where the weight is
// small; with outlier columns, whose sums are N M for each that is used, where N is, too.
// Few / many, in us, for 16 rows, K to N:
//   1024 to 1024   2048 to 2048   4096 to 4096   4096 to 11008   8192 to 28672   65536 to 256
//    3.2 / 8.6      3.9 / 10.4     6.6 / 11.7     14.4 / 20.2     49 / 55         35.2 / 36.3
// and for 17 to 32 rows, without, with 5 and with 30 outlier columns:
//   1024 to 4096    4.5 to 4.9 / 8.5     6.6 to 7.3 / 9.9    11.4 to 15.7 / 10.1
//   4096 to 256     5.6 to 6.0 / 10.1    7.4 to 7.9 / 11.3   10.3 to 12.7 / 11.5
//   4096 to 2048    5.9 to 6.4 / 11.3    7.7 to 8.1 / 12.6   10.6 to 13.0 / 12.8
//   8192 to 2048    9.5 to 9.6 / 14.8   11.2 to 11.3 / 16.2  14.3 to 16.2 / 16.8
//  16384 to 1024   15.9 / 15.9          17.4 to 17.6 / 17.2  20.6 to 22.4 / 17.7
//  65536 to 256    54.9 / 36.7          56.4 / 38.0          (a CTA takes a sum of 65536)
//   2048 to 4096    7.9 / 10.5          11.5 to 11.9 / 11.6  17.3 to 21.2 / 11.9
//   4096 to 4096   11.4 to 12.1 / 12.1  15.0 to 15.8 / 13.5  20.7 to 25.4 / 14.4
//   1024 to 11008   9.2 to 10.3 / 8.8   14.8 to 16.8 / 11.2  26.4 to 38.5 / 12.0
bool few_rows(int64_t M, int64_t N, int64_t K, int L) {
  if (M <= 16 || K == 0) return true;
  return M <= 32 && N <= 4096 && K < 16384 && N * K <= 16 << 20 &&
         (L == 0 || N <= 2048 || N * K <= 4 << 20);
}

template <int NT, int kFewDepth>
int launch_few_depth(const CUtensorMap& w, const Int8Linear& p, int64_t grid, int group, int dev,
                     cudaStream_t stream) {
  auto kernel = dq4_int8_few_kernel<NT, kFewDepth>;
  constexpr int kRings = kStreamWarps * kFewDepth * kFewRows * kChunk + 1024;
  static std::atomic<uint64_t> allowed{0};
  if (const int st = allow_smem(kernel, kRings, dev, &allowed, kFewDepth == 2 ? 50 : 70)) return st;
  return launch_ordered(kernel, dim3(unsigned(grid)), kStreamThreads, kRings, stream, w, p, group);
}

template <int NT>
int launch_few(const Int8Linear& p, int dev, int sms, cudaStream_t stream) {
  CUtensorMap w = {};  // (without codes, K = 0, nothing is copied)
  if (p.K > 0)
    if (const int st = encode_2d(&w, CU_TENSOR_MAP_DATA_TYPE_UINT8, p.CB, p.K, p.N, p.K, kChunk,
                                 kFewRows, CU_TENSOR_MAP_SWIZZLE_128B))
      return st;
  const int64_t jobs = (p.N + kFewRows - 1) / kFewRows, chunks = (p.K + kChunk - 1) / kChunk;
  // warps of a job: enough for all that the SMs hold (three CTAs), with two chunks each at least
  int group = 1;
  while (group < kStreamWarps && jobs * group * 2 <= 3 * kStreamWarps * sms && chunks >= 4 * group)
    group *= 2;
  const int64_t grid = (jobs * group + kStreamWarps - 1) / kStreamWarps;
  // Shared memory is taken from the L1 that the tokens are read through: rings of two chunks
  // where an SM gets three CTAs (half of the 256 KB), of four where it gets two at most and its
  // warps need more each on their way (70 %; by the driver's choice 8.2 and 26 us instead of the
  // first two).  Two / four chunks, one row, in us: 4096 x 4096 5.8 / 5.5, 14336 to 4096
  // 16.6 / 12.8, 4096 to 11008 11.1 / 13.6, 8192 to 28672 37 / 44.
  if (grid <= 2 * sms) return launch_few_depth<NT, 4>(w, p, grid, group, dev, stream);
  return launch_few_depth<NT, 2>(w, p, grid, group, dev, stream);
}

}  // namespace
}  // namespace dq4d

using namespace dq4d;

extern "C" {

int64_t dq4_int8_linear_workspace_bytes(int64_t M, int64_t N, int64_t K, int32_t L) {
  if (M <= 0 || N <= 0 || K < 0 || L < 0 || L > kMaxOutliers || M > INT32_MAX || N > INT32_MAX ||
      K > INT32_MAX || few_rows(M, N, K, L))
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
  if (!few_rows(M, N, K, L)) {
    if (!workspace || workspace_bytes < int8_gemm_workspace(M, N, K, L, sms))
      return DQ4_ERR_WORKSPACE;
    if (misaligned(workspace, 256)) return DQ4_ERR_ALIGN;
    return launch_int8_gemm(p, dev, sms, workspace, s);
  }
  if (M <= 8) return launch_few<1>(p, dev, sms, s);
  return M <= 16 ? launch_few<2>(p, dev, sms, s) : launch_few<4>(p, dev, sms, s);
}

}  // extern "C"
