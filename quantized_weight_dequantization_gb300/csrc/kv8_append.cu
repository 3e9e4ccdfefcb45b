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
// Two bytes a value in, one out.  Measured: 64 sequences x 1 token 5.0 us, the chain of dependent
// loads (sequence, length, page id, scale) and the launch; prompts, 13 000 tokens of 8 heads of
// 128, FP16, pages of 16, half of each key rotated: 18.5 us (80 MB, 4.3 TB/s of a copy's 6.8),
// most of it the instructions of a value (widen, turn, compare, scale, convert).
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

constexpr int kThreadValues = 32;  // values of a thread: passes of two groups each
// a CTA takes heads up to about as many threads (512: 21.3 us for 13 000 tokens, 256: 19.3,
// 128: 18.5)
constexpr int kCtaThreads = 128;

__device__ __forceinline__ uint32_t e4m3x4(float4 f) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(f.y), "f"(f.x));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(f.w), "f"(f.z));
  return uint32_t(lo) | uint32_t(hi) << 16;
}

// Four e4m3 codes times r, as codes again.
__device__ __forceinline__ uint32_t rescale4(uint32_t codes, float r) {
  float f[4];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint16_t two = uint16_t(codes >> (16 * i));
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(two));
    __half2 v;
    memcpy(&v, &h, 4);
    f[2 * i] = __low2float(v) * r;
    f[2 * i + 1] = __high2float(v) * r;
  }
  return e4m3x4(make_float4(f[0], f[1], f[2], f[3]));
}

// A lane's two groups as codes, at their places in a slot.
template <int V>
__device__ __forceinline__ void store_codes(uint8_t* to, const LanePlace& at, const Vals<V>& x) {
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    uint32_t w[V / 4];
#pragma unroll
    for (int i = 0; i < V / 4; ++i) {
      const float* f = x.v + half * V + 4 * i;
      w[i] = e4m3x4(make_float4(f[0], f[1], f[2], f[3]));
    }
    uint8_t* p = to + (half ? at.b : at.a);
    if constexpr (V == 8) {
      *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    } else {
      *reinterpret_cast<uint32_t*>(p) = w[0];
    }
  }
}

// The larger of two, or NaN if one is.
__device__ __forceinline__ float larger(float x, float y) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(y));
  return r;
}

// The least power of two that holds amax in e4m3's +-448 = 1.75 2^8, at least 2^-100.
__device__ __forceinline__ float fitting_scale(float amax) {
  const uint32_t u = __float_as_uint(amax);
  if (u >= 0x7F800000u) return __uint_as_float(0x7FC00000u);  // infinite or NaN
  const int e = int(u >> 23) - 127 - ((u & 0x7FFFFFu) <= 0x600000u ? 8 : 7);
  return __uint_as_float(uint32_t(max(e, -100) + 127) << 23);
}

template <int DT, int kDim, int V>
__global__ void __launch_bounds__(1024) dq4_kv8_append_kernel(const AppendArgs p) {
  using T = typename Elem<DT>::T;
  constexpr int kLanes = kDim / (2 * V), kPasses = kThreadValues / (2 * V);
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
  const LanePlace at = lane_place<V>(l, turning ? p.rotary : 0, p.interleaved);
  const T* x = static_cast<const T*>(p.x[which]) + head * p.head_stride[which];
  Raw<DT, V> ra[kPasses], rb[kPasses];
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    const int pos = (j << log2_page) + first + i * step;
    if (pos < lo || pos >= hi) continue;
    const T* row = x + (q.row + (pos - begin)) * p.token_stride[which];
    ra[i] = load_group_once<DT, V>(row + at.a);
    rb[i] = load_group_once<DT, V>(row + at.b);
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

  Vals<V> v[kPasses];
  float amax = 0.f;
  auto bring = [&](auto interleaved) {
    constexpr bool kInterleaved = decltype(interleaved)::value;
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      const int pos = (j << log2_page) + first + i * step;
      v[i] = Vals<V>{};
      if (pos < lo || pos >= hi) continue;
      v[i] = widen<DT, V>(ra[i], rb[i]);
      if (turning && pos >= p.table_rows) {
        v[i] = Vals<V>{};
        if (p.bad && l == 0 && head == 0 && real) atomicAdd(p.bad, 1);
      } else if (at.turned) {
        const int64_t row0 = int64_t(pos) * (p.rotary / 2) + V * l;
        float cs[V], sn[V];
        load_entries(p.cos + row0, cs);
        load_entries(p.sin + row0, sn);
        v[i] = turned<kInterleaved, false>(v[i], cs, sn);
      }
#pragma unroll
      for (int k = 0; k < 2 * V; ++k) amax = larger(amax, fabsf(v[i].v[k]));
    }
  };
  if (p.interleaved) {
    bring(std::true_type{});
  } else {
    bring(std::false_type{});
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = larger(amax, __shfl_xor_sync(kAllLanes, amax, o));
  if (lane == 0) s_max[threadIdx.x >> 5] = amax;
  __syncthreads();  // also: every thread has read the old scale
  if (!real) return;
  const int warps = p.group >> 5;
  amax = s_max[mine * warps + (lane < warps ? lane : 0)];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = larger(amax, __shfl_xor_sync(kAllLanes, amax, o));

  const float fit = fitting_scale(amax);
  const float scale = isnan(old) || isnan(fit) ? __uint_as_float(0x7FC00000u) : fmaxf(old, fit);
  if (tid == 0) *scale_at = scale;
  // 1 / 2^e is exact, so that multiplying is the same as dividing; a scale that append did
  // not write may be any number
  if ((__float_as_uint(scale) & 0x7FFFFFu) == 0) {
    const float inverse = 1.f / scale;
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
#pragma unroll
      for (int k = 0; k < 2 * V; ++k) v[i].v[k] *= inverse;
    }
  } else {
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
#pragma unroll
      for (int k = 0; k < 2 * V; ++k) v[i].v[k] /= scale;
    }
  }
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    const int slot = first + i * step, pos = (j << log2_page) + slot;
    if (pos < lo || pos >= hi) continue;
    store_codes<V>(codes + slot * kDim, at, v[i]);
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

template <int DT, int kDim, int V>
int launch_groups(AppendArgs p, int64_t units, cudaStream_t stream) {
  p.group = p.c.page * kDim / kThreadValues;  // 32 .. 1024
  const int most = kCtaThreads / p.group > 1 ? kCtaThreads / p.group : 1;
  const int heads = most < p.c.heads ? most : p.c.heads;
  return launch_ordered(dq4_kv8_append_kernel<DT, kDim, V>,
                        dim3(unsigned(units), unsigned((p.c.heads + heads - 1) / heads), 2),
                        p.group * heads, 0, stream, p);
}

// Groups of 8 values, 16 bytes, where tokens and pairs allow it, else of 4: half the memory
// instructions and steps over the lanes (19.3 us with 8, 22.4 with 4, for 13 000 tokens).
template <int DT, int kDim>
int launch_append(const AppendArgs& p, int64_t units, cudaStream_t stream) {
  bool wide = p.cos == nullptr || p.rotary % 16 == 0;
  for (int n = 0; n < 2; ++n)
    wide = wide && p.token_stride[n] % 8 == 0 && p.head_stride[n] % 8 == 0 && aligned(p.x[n], 16);
  return wide ? launch_groups<DT, kDim, 8>(p, units, stream)
              : launch_groups<DT, kDim, 4>(p, units, stream);
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
