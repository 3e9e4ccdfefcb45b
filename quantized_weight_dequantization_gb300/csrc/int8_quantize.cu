// Rows in 8 bits with outlier columns: dq4_int8_quantize (dq4_int8.h).
//
// Bound by memory: 2 bytes a value in, 1 out.  A row lies in the registers of a warp (up to 1024
// values) or of a CTA, is read once, and its codes are written as if there were no outlier columns;
// values past the threshold only mark their column (their own codes are nothing yet).  A second,
// small launch lists the marked columns, takes their codes out and copies their values: 2 M L
// scattered accesses instead of a second pass over X.  A mark is a bit set by an atomic that
// nothing waits for, in one of 16 copies: one word takes an atomic (or a store) every 2 to 3 ns,
// and 16384 x 1024 with 5 such columns took 31 to 37 us with a single copy.
// The maximum is taken on the bits of |x|, two values an instruction: for values that are not
// negative the order of the bits is that of the numbers, infinity and NaN last.
//
// 2048 x 14336: 14 us, of which the bytes take 13.0 (0.93 of the copy rate); with 21 outlier
// columns 21.7, the second launch; 1 x 4096 1.5 us, the launch.
#include "int8.cuh"

namespace dq4d {
namespace {

constexpr int kRowThreads = 256;  // of a CTA
constexpr int kCopies = 16;       // of the marks

struct QuantArgs {
  const uint16_t* X;
  int64_t row_stride, M, K;
  uint32_t loud;  // the least |x| that is an outlier, as 16 bits
  int8_t* codes;
  float* scales;
  uint32_t* marks;  // [kCopies][K / 32 words]: a bit for each column
};

template <bool kBf16>
__device__ __forceinline__ float widen(uint32_t bits) {
  if constexpr (kBf16) return __uint_as_float(bits << 16);
  else return __half2float(__ushort_as_half(uint16_t(bits)));
}

// Two values of 16 bits as FP32.
template <bool kBf16>
__device__ __forceinline__ float2 widen2(uint32_t w) {
  if constexpr (kBf16) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
  } else {
    __half2 h;
    memcpy(&h, &w, 4);
    return __half22float2(h);
  }
}

// x * inverse to the nearest integer, in the low byte of each half: 1.5 * 2^23 leaves no bits
// behind the point.  (Two values an instruction.  The product is rounded on its own: ptxas makes
// one instruction of a packed product and sum, whatever their modifiers, so the sum is an FMA by
// 1.)
__device__ __forceinline__ uint64_t codes_of(float2 x, uint64_t inverse2) {
  const uint64_t magic2 = 0x4B4000004B400000ull, one2 = 0x3F8000003F800000ull;
  uint64_t v;
  memcpy(&v, &x, 8);
  asm("mul.rn.f32x2 %0, %0, %1;" : "+l"(v) : "l"(inverse2));
  asm("fma.rn.f32x2 %0, %0, %1, %2;" : "+l"(v) : "l"(one2), "l"(magic2));
  return v;
}

// kRow threads a row, kGroups groups of 8 values for each at a time: 8 that follow one another,
// where they are whole and aligned (kVec), else every kRow-th, so that a warp's loads follow one
// another.  (8000 x 1001: 24 us with 8 that follow one another and a CTA a row, so 7.8.)  Rows
// longer than the registers hold are read twice (the second time from L2).
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
  uint32_t* marks = p.marks + (blockIdx.x % kCopies) * ((p.K + 31) / 32);
  uint4 v[kGroups];
  auto column_of = [&](int64_t base, int g, int i) {
    return kVec ? base + (g * kRow + t) * 8 + i : base + (g * 8 + i) * kRow + t;
  };
  auto load = [&](int64_t base) {
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      const int64_t e = column_of(base, g, 0);
      v[g] = make_uint4(0, 0, 0, 0);
      if constexpr (kVec) {
        if (e < p.K) v[g] = load_global(reinterpret_cast<const uint4*>(x + e));
      } else {
        uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (e + i * kRow < p.K)
            w[i / 2] |= uint32_t(load_global(x + e + i * kRow)) << (16 * (i & 1));
        v[g] = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
  };
  auto word = [&](int g, int i) {
    return i == 0 ? v[g].x : i == 1 ? v[g].y : i == 2 ? v[g].z : v[g].w;
  };

  // ---- the largest |x|
  uint32_t top = 0;
  for (int64_t base = 0; base < p.K; base += kSpan) {
    load(base);
    uint32_t most = 0, hot = 0;  // hot: groups with outliers
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      const uint32_t m = __vmaxu2(__vmaxu2(v[g].x & 0x7FFF7FFFu, v[g].y & 0x7FFF7FFFu),
                                  __vmaxu2(v[g].z & 0x7FFF7FFFu, v[g].w & 0x7FFF7FFFu));
      const uint32_t mg = max(m & 0xFFFFu, m >> 16);
      if (kThr && mg >= p.loud)
        hot |= 1u << g;
      else
        most = max(most, mg);
    }
    if (kThr && hot) {  // seldom: which values, and the largest of the others
#pragma unroll
      for (int g = 0; g < kGroups; ++g) {
        if (!(hot >> g & 1)) continue;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint32_t b = word(g, i / 2) >> (16 * (i & 1)) & 0x7FFFu;
          if (b < p.loud || b > kInf) {
            most = max(most, b);
          } else {
            const int64_t col = column_of(base, g, i);
            atomicOr(marks + (col >> 5), 1u << (col & 31));
          }
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
  const uint64_t inverse2 = uint64_t(__float_as_uint(inverse)) << 32 | __float_as_uint(inverse);
  int8_t* to = p.codes + row * p.K;
  for (int64_t base = 0; base < p.K; base += kSpan) {
    if (p.K > kSpan) load(base);
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      const int64_t e = column_of(base, g, 0);
      uint32_t c[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint64_t a = codes_of(widen2<kBf16>(word(g, 2 * h)), inverse2);
        const uint64_t b = codes_of(widen2<kBf16>(word(g, 2 * h + 1)), inverse2);
        c[h] = __byte_perm(__byte_perm(uint32_t(a), uint32_t(a >> 32), 0x0040),
                           __byte_perm(uint32_t(b), uint32_t(b >> 32), 0x0040), 0x5410);
        if (!(scale > 0.f)) c[h] = 0;
      }
      if constexpr (kVec) {
        if (e < p.K) __stcs(reinterpret_cast<uint2*>(to + e), make_uint2(c[0], c[1]));
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (e + i * kRow < p.K) to[e + i * kRow] = int8_t(c[i / 4] >> (8 * (i & 3)));
      }
    }
  }
}

struct OutlierArgs {
  const uint16_t* X;
  int64_t row_stride, M, K;
  uint32_t loud;
  int8_t* codes;
  const float* scales;
  int64_t* cols;
  int max_cols;
  uint16_t* outliers;
  int32_t* count;
  uint32_t* marks;
  int* done;  // CTAs that have read the marks
  int64_t rows;  // of a CTA
};

// The marked columns, listed by every CTA for itself (from L2), their values and codes for
// its rows; the last CTA to have read the marks clears them.
__global__ void __launch_bounds__(kRowThreads) int8_outliers_kernel(const OutlierArgs p) {
  constexpr int kAtOnce = 8;
  __shared__ int64_t s_cols[kMaxOutliers];
  __shared__ int s_sums[kRowThreads / 32];
  __shared__ bool s_last;
  wait_for_stream();
  asm volatile("griddepcontrol.launch_dependents;");
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const int64_t words = (p.K + 31) / 32;
  auto marks_of = [&](int64_t w) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < kCopies; ++i) m |= load_global(p.marks + i * words + w);
    return m;
  };
  int found = 0;
  for (int64_t w0 = 0; w0 < words; w0 += kRowThreads) {
    uint32_t m = w0 + t < words ? marks_of(w0 + t) : 0;
    const int mine = __popc(m);
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
    for (; m != 0 && at < p.max_cols; m &= m - 1, ++at) s_cols[at] = (w0 + t) * 32 + __ffs(m) - 1;
    __syncthreads();
  }
  const int kept = min(found, p.max_cols);
  if (blockIdx.x == 0) {
    for (int l = t; l < p.max_cols; l += kRowThreads) p.cols[l] = l < kept ? s_cols[l] : -1;
    if (t == 0) *p.count = found;
  }
  const int64_t row0 = blockIdx.x * p.rows;
  const int rows = int(min(p.rows, p.M - row0));
  // (a thread keeps to one of the columns: 128 at most, a power of two of threads for each row)
  const int wide = p.max_cols <= 32 ? 32 : p.max_cols <= 64 ? 64 : 128;
  const int l = t % wide, step = kRowThreads / wide;
  if (l < p.max_cols) {
    const int64_t col = l < kept ? s_cols[l] : -1;
    for (int r0 = t / wide; r0 < rows; r0 += step * kAtOnce) {
      uint16_t v[kAtOnce];
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i) {
        const int r = r0 + i * step;
        v[i] = 0;
        if (col >= 0 && r < rows) v[i] = load_global(p.X + (row0 + r) * p.row_stride + col);
      }
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i) {
        const int64_t row = row0 + r0 + i * step;
        if (r0 + i * step >= rows) break;
        if (col >= 0) p.codes[row * p.K + col] = 0;
        p.outliers[row * p.max_cols + l] = v[i];
      }
    }
  }
  // Outlier columns past the last that is kept: their outliers' codes end at +-127 (they are above
  // the scale).  A warp looks at 32 words of marks, and takes the columns of a word side by side,
  // or, where they are few, the rows of one.
  if (found > p.max_cols) {
    const int64_t after = s_cols[p.max_cols - 1] + 1;
    auto clip = [&](int64_t row, int64_t col) {
      const uint32_t b = load_global(p.X + row * p.row_stride + col);
      if ((b & 0x7FFFu) >= p.loud && load_global(p.scales + row) > 0.f)
        p.codes[row * p.K + col] = b & 0x8000u ? -127 : 127;
    };
    for (int64_t w0 = after / 32 + warp * 32; w0 < words; w0 += kRowThreads) {
      uint32_t own = w0 + lane < words ? marks_of(w0 + lane) : 0;
      if (w0 + lane == after / 32) own &= 0xFFFFFFFFu << (after & 31);
      for (uint32_t some = __ballot_sync(kAllLanes, own != 0); some != 0; some &= some - 1) {
        const int at = __ffs(some) - 1;
        uint32_t m = __shfl_sync(kAllLanes, own, at);
        const int64_t col = (w0 + at) * 32;
        if (__popc(m) >= 8) {
          if (m >> lane & 1)
#pragma unroll 4
            for (int r = 0; r < rows; ++r) clip(row0 + r, col + lane);
        } else {
          for (; m != 0; m &= m - 1)
            for (int r = lane; r < rows; r += 32) clip(row0 + r, col + __ffs(m) - 1);
        }
      }
    }
  }
  __syncthreads();
  if (t == 0) s_last = atomic_add_acq_rel(p.done, 1) == int(gridDim.x) - 1;
  __syncthreads();
  if (s_last) {
    for (int64_t w = t; w < kCopies * words; w += kRowThreads) p.marks[w] = 0;
    if (t == 0) *p.done = 0;
  }
}

constexpr int64_t kMarksAt = 256;  // bytes of the workspace before the marks

int64_t mark_bytes(int64_t K) { return kCopies * ((K + 31) / 32) * 4; }

template <bool kBf16, bool kThr>
int launch_rows(const QuantArgs& p, bool vec, cudaStream_t stream) {
  auto go = [&](auto kernel, int rows) {
    return launch_ordered(kernel, dim3(unsigned((p.M + rows - 1) / rows)), kRowThreads, 0, stream,
                          p);
  };
  if (!vec && p.K <= 1024)
    return go(int8_quantize_kernel<kBf16, false, kThr, 32, 4>, kRowThreads / 32);
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
  return K < 0 ? 0 : kMarksAt + mark_bytes(K);
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
    if (!workspace || workspace_bytes < kMarksAt + mark_bytes(K)) return DQ4_ERR_WORKSPACE;
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
    p.marks = reinterpret_cast<uint32_t*>(static_cast<char*>(workspace) + kMarksAt);
  }
  const bool vec = K % 8 == 0 && (M <= 1 || row_stride % 8 == 0) && !misaligned(X, 16) &&
                   !misaligned(codes, 8);
  if (M > 0) {
    const bool bf16 = dtype == DQ4_OUT_BF16;
    const int st = bf16 ? (thr ? launch_rows<true, true>(p, vec, s)
                               : launch_rows<true, false>(p, vec, s))
                        : (thr ? launch_rows<false, true>(p, vec, s)
                               : launch_rows<false, false>(p, vec, s));
    if (st || !thr) return st;
  }
  OutlierArgs o = {p.X, row_stride, M, K, p.loud, codes, scales, cols, max_cols,
                   static_cast<uint16_t*>(outliers), count, p.marks, static_cast<int*>(workspace),
                   1};
  // rows of a CTA: one wave of the SMs, two CTAs each
  o.rows = (M + 2 * sms - 1) / (2 * sms);
  if (o.rows < 1) o.rows = 1;
  const int64_t grid = M > 0 ? (M + o.rows - 1) / o.rows : 1;
  return launch_ordered(int8_outliers_kernel, dim3(unsigned(grid)), kRowThreads, 0, s, o);
}

}  // extern "C"
