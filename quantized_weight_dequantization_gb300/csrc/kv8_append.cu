// Appending keys and values to the 8-bit paged cache, with the rotation of the keys on the
// way: dq4_kv8_append (dq4_attn.h).
//
// For each page and head that gets tokens, of K and of V:
//   fit = 2^e, e the least with max|x| <= 448 2^e;  scale = max(old scale, fit)
//   code = e4m3(x / scale);  earlier codes become e4m3(code * old / scale)
// Scales are powers of two, so that a page that grows its scale loses nothing but what
// falls below e4m3's smallest step: rounding does not pile up over a page's tokens.
//
// A group of page * dim / 32 threads owns one page and head of K or of V, so nothing is shared
// between groups: it reads its tokens once into registers (rotated in FP32), reduces max|x|,
// and writes codes.  A CTA has the groups of a few heads of one page, so that finding the page
// is paid for once.
// Two bytes a value in, one out: bound by HBM for prompts, by the chain of dependent loads
// (length, page id, scale; tokens) for single tokens.
#include "kv8.cuh"

namespace dq4d {
namespace {

struct AppendArgs {
  Kv8 c;
  Batch s;
  const void* x[2];
  int64_t token_stride[2], head_stride[2];
  const float* cos;
  const float* sin;
  int64_t table_rows;
  int rotary;
  bool interleaved;
  int* bad;
  int group;  // threads of a page and head
};

constexpr int kPasses = 4;  // 8-value pieces a thread handles
constexpr int kCtaThreads = 256;  // a CTA takes heads up to about as many threads

__device__ __forceinline__ uint32_t e4m3x4(const F4& f) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(f.v[1]), "f"(f.v[0]));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(f.v[3]), "f"(f.v[2]));
  return uint32_t(lo) | uint32_t(hi) << 16;
}

// Four e4m3 codes times r, as codes again.
__device__ __forceinline__ uint32_t rescale4(uint32_t codes, float r) {
  F4 f;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint16_t two = uint16_t(codes >> (16 * i));
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(two));
    __half2 v;
    memcpy(&v, &h, 4);
    f.v[2 * i] = __low2float(v) * r;
    f.v[2 * i + 1] = __high2float(v) * r;
  }
  return e4m3x4(f);
}

// The least power of two that holds amax in e4m3's +-448 = 1.75 2^8, at least 2^-100.
__device__ __forceinline__ float fitting_scale(float amax) {
  const uint32_t u = __float_as_uint(amax);
  if (u >= 0x7F800000u) return __uint_as_float(0x7FC00000u);  // infinite or NaN
  const int e = int(u >> 23) - 127 - ((u & 0x7FFFFFu) <= 0x600000u ? 8 : 7);
  return __uint_as_float(uint32_t(max(e, -100) + 127) << 23);
}

template <int DT, int kDim>
__global__ void __launch_bounds__(1024) dq4_kv8_append_kernel(const AppendArgs p) {
  using T = typename Elem<DT>::T;
  constexpr int kLanes = kDim / 8;
  __shared__ float s_max[32];
  wait_for_stream();
  const int which = blockIdx.z, lane = threadIdx.x & 31;
  const int heads = blockDim.x / p.group;  // of this CTA
  const int mine = threadIdx.x / p.group, tid = threadIdx.x - mine * p.group;
  const bool real = blockIdx.y * heads + mine < p.c.heads;
  const int head = min(blockIdx.y * heads + mine, p.c.heads - 1);
  const int l = tid % kLanes, first = tid / kLanes, step = p.group / kLanes;
  const int page = p.c.page, log2_page = p.c.log2_page;
  // The sequence and the page within it.  Sequence b's pages start at unit
  // row / page + 2 b: n tokens touch at most n / page + 2 pages, and the units of the
  // next sequence start that many further on at least.
  int64_t b = blockIdx.x, u0 = b;
  if (p.s.cu) {
    auto start = [&](int64_t i) { return (seq_row(p.s, i) >> log2_page) + 2 * i; };
    b = find_last(p.s.seqs, int64_t(blockIdx.x), start);
    u0 = start(b);
  }
  const Seq q = seq_at(p.s, b);
  const int begin = q.len - q.n;                  // position of the first new token
  const int j = (begin >> log2_page) + int(blockIdx.x - u0);  // the page within the sequence
  const int lo = max(begin, j << log2_page), hi = min(q.len, (j + 1) << log2_page);
  if (lo >= hi) return;
  // (the page id is on its way while the tokens are read)
  const int id = j >= 0 && j < p.s.table_width
                     ? load_global(p.s.table + b * p.s.table_stride + j) : -1;

  const bool turning = which == 0 && p.cos != nullptr;
  const LanePlace at = lane_place(l, turning ? p.rotary : 0, p.interleaved);
  const T* x = static_cast<const T*>(p.x[which]) + head * p.head_stride[which];
  Raw4<DT> ra[kPasses], rb[kPasses];
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    const int pos = (j << log2_page) + first + i * step;
    if (pos < lo || pos >= hi) continue;
    const T* row = x + (q.row + (pos - begin)) * p.token_stride[which];
    ra[i] = load4_once<DT>(row + at.a);
    rb[i] = load4_once<DT>(row + at.b);
  }
  if (id < 0 || id >= p.c.pages) {
    if (p.bad && threadIdx.x == 0 && blockIdx.y == 0 && which == 0) atomicAdd(p.bad, hi - lo);
    return;
  }
  const int64_t block = int64_t(id) * p.c.heads + head;
  uint8_t* codes = p.c.codes[which] + block * page * kDim;
  float* scale_at = p.c.scale[which] + block;
  const bool earlier = lo > (j << log2_page);
  const float old = earlier ? *scale_at : 0.f;

  F4 a[kPasses], c[kPasses];
  float amax = 0.f;
  bool unordered = false;
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    const int pos = (j << log2_page) + first + i * step;
    a[i] = c[i] = F4{};
    if (pos < lo || pos >= hi) continue;
    a[i] = widen<DT>(ra[i]);
    c[i] = widen<DT>(rb[i]);
    if (turning && pos >= p.table_rows) {
      a[i] = c[i] = F4{};
      if (p.bad && l == 0 && head == 0 && real) atomicAdd(p.bad, 1);
    } else if (at.turned) {
      const int64_t row0 = int64_t(pos) * (p.rotary / 2) + 4 * l;
      turn(a[i], c[i], load_global(reinterpret_cast<const float4*>(p.cos + row0)),
           load_global(reinterpret_cast<const float4*>(p.sin + row0)), p.interleaved);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      amax = fmaxf(amax, fmaxf(fabsf(a[i].v[k]), fabsf(c[i].v[k])));  // fmaxf drops NaN
      unordered |= isnan(a[i].v[k]) | isnan(c[i].v[k]);
    }
  }
  if (unordered) amax = __uint_as_float(0x7F800000u);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(kAllLanes, amax, o));
  if (lane == 0) s_max[threadIdx.x >> 5] = amax;
  __syncthreads();  // also: every thread has read the old scale
  if (!real) return;
  const int warps = p.group >> 5;
  amax = s_max[mine * warps + (lane < warps ? lane : 0)];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(kAllLanes, amax, o));

  const float fit = fitting_scale(amax);
  const float scale = isnan(old) || isnan(fit) ? __uint_as_float(0x7FC00000u) : fmaxf(old, fit);
  if (tid == 0) *scale_at = scale;
  // 1 / 2^e is exact, so that multiplying is the same as dividing; a scale that append did
  // not write may be any number
  const bool pow2 = (__float_as_uint(scale) & 0x7FFFFFu) == 0;
  const float inverse = 1.f / scale;
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    const int slot = first + i * step, pos = (j << log2_page) + slot;
    if (pos < lo || pos >= hi) continue;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      a[i].v[k] = pow2 ? a[i].v[k] * inverse : a[i].v[k] / scale;
      c[i].v[k] = pow2 ? c[i].v[k] * inverse : c[i].v[k] / scale;
    }
    *reinterpret_cast<uint32_t*>(codes + slot * kDim + at.a) = e4m3x4(a[i]);
    *reinterpret_cast<uint32_t*>(codes + slot * kDim + at.b) = e4m3x4(c[i]);
  }
  if (earlier && !(old == scale)) {
    const float ratio = old / scale;
    const int words = (lo - (j << log2_page)) * (kDim / 16);
    uint4* at16 = reinterpret_cast<uint4*>(codes);
    for (int i = tid; i < words; i += p.group) {
      uint4 w = at16[i];
      w.x = rescale4(w.x, ratio);
      w.y = rescale4(w.y, ratio);
      w.z = rescale4(w.z, ratio);
      w.w = rescale4(w.w, ratio);
      at16[i] = w;
    }
  }
}

template <int DT, int kDim>
int launch_append(AppendArgs p, int64_t units, cudaStream_t stream) {
  p.group = p.c.page * kDim / (8 * kPasses);  // 32 .. 1024
  const int most = kCtaThreads / p.group > 1 ? kCtaThreads / p.group : 1;
  const int heads = most < p.c.heads ? most : p.c.heads;
  return launch_ordered(dq4_kv8_append_kernel<DT, kDim>,
                        dim3(unsigned(units), unsigned((p.c.heads + heads - 1) / heads), 2),
                        p.group * heads, 0, stream, p);
}

}  // namespace
}  // namespace dq4d

using namespace dq4d;

extern "C" int dq4_kv8_append(const dq4_kv8_cache* cache, const void* k, int64_t k_token_stride,
                              int64_t k_head_stride, const void* v, int64_t v_token_stride,
                              int64_t v_head_stride, int32_t dtype, int64_t tokens,
                              const int32_t* block_table, int64_t table_stride,
                              int32_t table_width, const int32_t* seq_lens, const int32_t* cu,
                              int64_t seqs, const float* cos, const float* sin,
                              int64_t table_rows, int32_t rotary, int32_t interleaved, int* bad,
                              void* stream) {
  AppendArgs p = {};
  if (const int st = make_cache(cache, &p.c)) return st;
  if (!valid_dtype(dtype, false)) return DQ4_ERR_DTYPE;
  p.s = {block_table, table_stride, table_width, seq_lens, cu, seqs, tokens};
  if (const int st = check_batch(p.s)) return st;
  if ((cos == nullptr) != (sin == nullptr)) return DQ4_ERR_NULL;
  const int dim = cache->head_dim;
  if (cos && (rotary < 8 || rotary > dim || rotary % 8 != 0 || table_rows < 0))
    return DQ4_ERR_ROTARY;
  if (tokens == 0 || seqs == 0) return DQ4_OK;
  if (!k || !v) return DQ4_ERR_NULL;
  if (misaligned(k, 8) || misaligned(v, 8) || k_token_stride % 4 || k_head_stride % 4 ||
      v_token_stride % 4 || v_head_stride % 4 || misaligned(cos, 16) || misaligned(sin, 16) ||
      misaligned(bad, 4))
    return DQ4_ERR_ALIGN;
  p.x[0] = k;
  p.x[1] = v;
  p.token_stride[0] = k_token_stride;
  p.token_stride[1] = v_token_stride;
  p.head_stride[0] = k_head_stride;
  p.head_stride[1] = v_head_stride;
  p.cos = cos;
  p.sin = sin;
  p.table_rows = table_rows;
  p.rotary = rotary;
  p.interleaved = interleaved != 0;
  p.bad = bad;
  int dev, sms;
  if (const int st = current_device(&dev, &sms)) return st;
  const int64_t units = cu ? tokens / p.c.page + 2 * seqs : seqs;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (dtype == DQ4_OUT_BF16)
    return dim == 64 ? launch_append<DQ4_OUT_BF16, 64>(p, units, s)
                     : launch_append<DQ4_OUT_BF16, 128>(p, units, s);
  return dim == 64 ? launch_append<DQ4_OUT_F16, 64>(p, units, s)
                   : launch_append<DQ4_OUT_F16, 128>(p, units, s);
}
