// Rows in 8 bits with outlier columns: dq4_int8_quantize (dq4_int8.h).
//
// Bound by memory: 2 bytes a value in, 1 out.  A row lies in the registers of a warp (up to 1024
// values) or of a CTA, is read once, and its codes are written as if there were no outlier
// columns; values past the threshold only set their column's bit in a mask.  A second, small
// launch lists the mask's columns, takes their codes out and copies their values: 2 M L
// scattered accesses instead of a second pass over X.
// The maximum is taken on the bits of |x|, two values an instruction: for values that are not
// negative the order of the bits is that of the numbers, infinity and NaN last.
#include "int8.cuh"

namespace dq4d {
namespace {

constexpr int kRowThreads = 256;  // of a CTA

struct QuantArgs {
  const uint16_t* X;
  int64_t row_stride, M, K;
  uint32_t loud;  // the least |x| that is an outlier, as 16 bits
  int8_t* codes;
  float* scales;
  uint32_t* mask;  // a bit for each column
};

template <bool kBf16>
__device__ __forceinline__ float widen(uint32_t bits) {
  if constexpr (kBf16) return __uint_as_float(bits << 16);
  else return __half2float(__ushort_as_half(uint16_t(bits)));
}

// x * inverse to the nearest integer, in the low byte: 1.5 * 2^23 leaves no bits behind the point.
__device__ __forceinline__ uint32_t code_of(float x, float inverse, bool limit) {
  float v = __fmul_rn(x, inverse);
  if (limit) v = fminf(fmaxf(v, -127.f), 127.f);
  return __float_as_uint(__fadd_rn(v, 12582912.f));
}

// kRow threads a row, kGroups groups of 8 values for each at a time.  kVec: groups are whole and
// aligned.  Rows longer than the registers hold are read twice (the second time from L2).
template <bool kBf16, bool kVec, bool kThr, int kRow, int kGroups>
__global__ void __launch_bounds__(kRowThreads) int8_quantize_kernel(const QuantArgs p) {
  constexpr uint32_t kInf = kBf16 ? 0x7F80u : 0x7C00u;
  constexpr int64_t kSpan = int64_t(kRow) * 8 * kGroups;
  __shared__ uint32_t s_top[kRowThreads / 32];
  wait_for_stream();
  asm volatile("griddepcontrol.launch_dependents;");
  const int t = threadIdx.x % kRow;
  const int64_t row = int64_t(blockIdx.x) * (kRowThreads / kRow) + threadIdx.x / kRow;
  if (row >= p.M) return;  // (whole warps: a warp's row, or the CTA's only one)
  const uint16_t* x = p.X + row * p.row_stride;
  uint4 v[kGroups];
  auto load = [&](int64_t base) {
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      const int64_t e = base + (int64_t(g) * kRow + t) * 8;
      v[g] = make_uint4(0, 0, 0, 0);
      if constexpr (kVec) {
        if (e < p.K) v[g] = load_global(reinterpret_cast<const uint4*>(x + e));
      } else {
        uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (e + i < p.K) w[i / 2] |= uint32_t(load_global(x + e + i)) << (16 * (i & 1));
        v[g] = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
  };
  auto word = [&](int g, int i) { return i == 0 ? v[g].x : i == 1 ? v[g].y : i == 2 ? v[g].z : v[g].w; };

  // ---- the largest |x|
  uint32_t top = 0;
  for (int64_t base = 0; base < p.K; base += kSpan) {
    load(base);
    uint32_t m = 0;
#pragma unroll
    for (int g = 0; g < kGroups; ++g)
#pragma unroll
      for (int i = 0; i < 4; ++i) m = __vmaxu2(m, word(g, i) & 0x7FFF7FFFu);
    uint32_t most = max(m & 0xFFFFu, m >> 16);
    if (kThr && most >= p.loud) {  // seldom: which, and the largest of the others
      most = 0;
#pragma unroll
      for (int g = 0; g < kGroups; ++g)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint32_t b = word(g, i / 2) >> (16 * (i & 1)) & 0x7FFFu;
          if (b < p.loud || b > kInf) {
            most = max(most, b);
          } else {
            const int64_t col = base + (int64_t(g) * kRow + t) * 8 + i;
            const uint32_t bit = 1u << (col & 31);
            uint32_t* at = p.mask + (col >> 5);
            if (!(*reinterpret_cast<volatile uint32_t*>(at) & bit)) atomicOr(at, bit);
          }
        }
    }
    top = max(top, most);
  }
  top = __reduce_max_sync(kAllLanes, top);
  if constexpr (kRow > 32) {
    if ((threadIdx.x & 31) == 0) s_top[threadIdx.x >> 5] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kRowThreads / 32; ++w) top = max(top, s_top[w]);
  }
  float scale = widen<kBf16>(top);
  if (top >= kInf) scale = __uint_as_float(0x7FC00000u);
  if (scale < 7.888609052210118e-31f) scale = 0.f;  // 2^-100
  if (t == 0) p.scales[row] = scale;

  // ---- the codes
  const float inverse = scale > 0.f ? __fdiv_rn(127.f, scale) : 0.f;
  int8_t* to = p.codes + row * p.K;
  for (int64_t base = 0; base < p.K; base += kSpan) {
    if (p.K > kSpan) load(base);
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      const int64_t e = base + (int64_t(g) * kRow + t) * 8;
      uint32_t c[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t w = word(g, i / 2);
        c[i] = code_of(widen<kBf16>(i & 1 ? w >> 16 : w & 0xFFFFu), inverse, kThr);
      }
      uint32_t lo = __byte_perm(__byte_perm(c[0], c[1], 0x0040), __byte_perm(c[2], c[3], 0x0040),
                                0x5410);
      uint32_t hi = __byte_perm(__byte_perm(c[4], c[5], 0x0040), __byte_perm(c[6], c[7], 0x0040),
                                0x5410);
      if (!(scale > 0.f)) lo = hi = 0;
      if constexpr (kVec) {
        if (e < p.K) __stcs(reinterpret_cast<uint2*>(to + e), make_uint2(lo, hi));
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (e + i < p.K) to[e + i] = int8_t((i < 4 ? lo : hi) >> (8 * (i & 3)));
      }
    }
  }
}

struct OutlierArgs {
  const uint16_t* X;
  int64_t row_stride, M, K;
  int8_t* codes;
  int64_t* cols;
  int max_cols;
  uint16_t* outliers;
  int32_t* count;
  uint32_t* mask;
  int* done;  // CTAs that have read the mask
  int64_t rows;  // of a CTA
};

// The mask's columns, listed by every CTA for itself (K / 32 words from L2), their values and
// codes for its rows; the last CTA to have read the mask clears it.
__global__ void __launch_bounds__(kRowThreads) int8_outliers_kernel(const OutlierArgs p) {
  __shared__ int64_t s_cols[kMaxOutliers];
  __shared__ int s_sums[kRowThreads / 32];
  __shared__ bool s_last;
  wait_for_stream();
  asm volatile("griddepcontrol.launch_dependents;");
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const int64_t words = (p.K + 31) / 32;
  int found = 0;
  for (int64_t w0 = 0; w0 < words; w0 += kRowThreads) {
    uint32_t bits = w0 + t < words ? load_global(p.mask + w0 + t) : 0;
    const int mine = __popc(bits);
    int run = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(kAllLanes, run, o);
      if (lane >= o) run += up;
    }
    if (lane == 31) s_sums[warp] = run;
    __syncthreads();
    int at = found + run - mine;
#pragma unroll
    for (int w = 0; w < kRowThreads / 32; ++w) {
      if (w < warp) at += s_sums[w];
      found += s_sums[w];
    }
    for (; bits != 0 && at < p.max_cols; bits &= bits - 1, ++at)
      s_cols[at] = (w0 + t) * 32 + __ffs(bits) - 1;
    __syncthreads();
  }
  if (t == 0) s_last = atomic_add_acq_rel(p.done, 1) == int(gridDim.x) - 1;
  const int kept = min(found, p.max_cols);
  if (blockIdx.x == 0) {
    for (int l = t; l < p.max_cols; l += kRowThreads) p.cols[l] = l < kept ? s_cols[l] : -1;
    if (t == 0) *p.count = found;
  }
  const int64_t row0 = blockIdx.x * p.rows;
  const int64_t n = min(p.rows, p.M - row0) * p.max_cols;
  for (int64_t i = t; i < n; i += kRowThreads) {
    const int64_t row = row0 + i / p.max_cols;
    const int l = int(i % p.max_cols);
    uint16_t v = 0;
    if (l < kept) {
      v = load_global(p.X + row * p.row_stride + s_cols[l]);
      p.codes[row * p.K + s_cols[l]] = 0;
    }
    p.outliers[row * p.max_cols + l] = v;
  }
  __syncthreads();
  if (s_last) {
    for (int64_t w = t; w < words; w += kRowThreads) p.mask[w] = 0;
    if (t == 0) *p.done = 0;
  }
}

constexpr int64_t kMaskAt = 256;  // bytes of the workspace before the mask

template <bool kBf16, bool kThr>
int launch_rows(const QuantArgs& p, bool vec, cudaStream_t stream) {
  auto go = [&](auto kernel, int rows) {
    return launch_ordered(kernel, dim3(unsigned((p.M + rows - 1) / rows)), kRowThreads, 0, stream,
                          p);
  };
  if (!vec) return go(int8_quantize_kernel<kBf16, false, kThr, 256, 2>, 1);
  if (p.K <= 1024) return go(int8_quantize_kernel<kBf16, true, kThr, 32, 4>, kRowThreads / 32);
  if (p.K <= 4096) return go(int8_quantize_kernel<kBf16, true, kThr, 256, 2>, 1);
  return go(int8_quantize_kernel<kBf16, true, kThr, 256, 8>, 1);
}

}  // namespace
}  // namespace dq4d

using namespace dq4d;

extern "C" {

int64_t dq4_int8_quantize_workspace_bytes(int64_t K) {
  return K < 0 ? 0 : kMaskAt + (K + 31) / 32 * 4;
}

int dq4_int8_quantize(const void* X, int64_t row_stride, int32_t dtype, int64_t M, int64_t K,
                      float threshold, int8_t* codes, float* scales, int64_t* cols,
                      int32_t max_cols, void* outliers, int32_t* count, void* workspace,
                      int64_t workspace_bytes, void* stream) {
  if (M < 0 || K < 0 || M > INT32_MAX || K > (int64_t(1) << 40) || !(threshold >= 0.f) ||
      (threshold > 0.f && (max_cols < 1 || max_cols > kMaxOutliers)))
    return DQ4_ERR_N;
  if (!valid_dtype(dtype, false)) return DQ4_ERR_DTYPE;
  const bool thr = threshold > 0.f;
  if (M == 0 && !thr) return DQ4_OK;
  if ((M > 0 && (!scales || (K > 0 && (!X || !codes)))) ||
      (thr && (!cols || !count || (M > 0 && !outliers))))
    return DQ4_ERR_NULL;
  if (misaligned(X, 2) || misaligned(scales, 4) || misaligned(cols, 8) ||
      misaligned(outliers, 2) || misaligned(count, 4))
    return DQ4_ERR_ALIGN;
  if (thr) {
    if (!workspace || workspace_bytes < kMaskAt + (K + 31) / 32 * 4) return DQ4_ERR_WORKSPACE;
    if (misaligned(workspace, 256)) return DQ4_ERR_ALIGN;
  }
  int dev, sms;
  if (const int st = current_device(&dev, &sms)) return st;
  QuantArgs p = {static_cast<const uint16_t*>(X), row_stride, M, K, 0, codes, scales, nullptr};
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (thr) {
    // the least value of the type that is not below the threshold
    if (dtype == DQ4_OUT_BF16) {
      uint32_t b;
      memcpy(&b, &threshold, 4);
      p.loud = (b >> 16) + ((b & 0xFFFFu) != 0);
      if (p.loud > 0x7F80u) p.loud = 0x7F80u;
    } else {
      p.loud = __half_as_ushort(__float2half_ru(threshold));
    }
    p.mask = reinterpret_cast<uint32_t*>(static_cast<char*>(workspace) + kMaskAt);
  }
  const bool vec = K % 8 == 0 && row_stride % 8 == 0 && !misaligned(X, 16) && !misaligned(codes, 8);
  if (M > 0) {
    const bool bf16 = dtype == DQ4_OUT_BF16;
    const int st = bf16 ? (thr ? launch_rows<true, true>(p, vec, s) : launch_rows<true, false>(p, vec, s))
                        : (thr ? launch_rows<false, true>(p, vec, s)
                               : launch_rows<false, false>(p, vec, s));
    if (st || !thr) return st;
  }
  OutlierArgs o = {p.X, row_stride, M, K, codes, cols, max_cols, static_cast<uint16_t*>(outliers),
                   count, p.mask, static_cast<int*>(workspace), 1};
  // rows of a CTA: one wave of the SMs, two CTAs each
  o.rows = (M + 2 * sms - 1) / (2 * sms);
  if (o.rows < 1) o.rows = 1;
  const int64_t grid = M > 0 ? (M + o.rows - 1) / o.rows : 1;
  return launch_ordered(int8_outliers_kernel, dim3(unsigned(grid)), kRowThreads, 0, s, o);
}

}  // extern "C"
