// Attention of new tokens over the 8-bit paged cache: dq4_kv8_attention (dq4_attn.h).
//
//   out = sum_j e_j v_j / sum_j e_j,  e_j = exp(scale q . k_j) over the keys in sight
//
// One pass over the keys with the running maximum m and sum l of the softmax: a new
// maximum scales what was summed by exp(m_old - m_new).  This form takes a warp for each
// query head of each token: a lane scores one key of 32, then sums the values of dim / 32
// columns over the 32 keys.
#include "kv8_attend.cuh"

namespace dq4d {
namespace {

constexpr int kRowWarps = 4;

__device__ __forceinline__ float e4m3(uint32_t code) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(uint16_t(code & 0xFFu)));
  __half2 v;
  memcpy(&v, &h, 4);
  return __low2float(v);
}

template <int DT, int kDim>
__global__ void __launch_bounds__(32 * kRowWarps) dq4_kv8_rows_kernel(const AttendArgs p) {
  using T = typename Elem<DT>::T;
  __shared__ float s_q[kRowWarps][kDim];
  wait_for_stream();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t r = int64_t(blockIdx.x) * kRowWarps + warp;
  const int64_t t = r / p.heads;
  if (t >= p.s.tokens) return;
  const int h = int(r - t * p.heads), kvh = h / p.group;
  int64_t b = t;
  if (p.s.cu) b = find_last(p.s.seqs, t, [&](int64_t i) { return seq_row(p.s, i); });
  const Seq s = seq_at(p.s, b);
  const T* q = static_cast<const T*>(p.q) + t * p.token_stride + h * p.head_stride;
  for (int i = lane; i < kDim; i += 32) s_q[warp][i] = Elem<DT>::load(q + i);
  __syncwarp();
  const int pos = s.len - s.n + int(t - s.row);
  const int held = min(s.len, int(min(int64_t(INT32_MAX), int64_t(p.s.table_width) * p.c.page)));
  const int end = p.causal ? min(held, pos + 1) : held;
  const int begin = p.window > 0 ? max(0, pos - p.window + 1) : 0;
  constexpr int kCols = kDim / 32;
  float m = -INFINITY, l = 0.f, o[kCols] = {};
  bool met_bad = held < s.len;
  for (int j0 = begin; j0 < end; j0 += 32) {
    const int j = j0 + lane;
    int64_t block = -1;
    float score = -INFINITY, vs = 0.f;
    if (j < end) {
      const int id = __ldg(p.s.table + b * p.s.table_stride + (j >> p.c.log2_page));
      if (id >= 0 && id < p.c.pages) {
        block = int64_t(id) * p.c.heads + kvh;
        const uint8_t* k = p.c.codes[0] + (block * p.c.page + (j & (p.c.page - 1))) * kDim;
        float dot = 0.f;
        for (int i = 0; i < kDim; ++i) dot = fmaf(s_q[warp][i], e4m3(k[i]), dot);
        score = dot * p.c.scale[0][block] * p.scale_log2;
        vs = p.c.scale[1][block];
      } else {
        met_bad = true;
      }
    }
    float top = score;
    for (int w = 16; w > 0; w >>= 1) top = fmaxf(top, __shfl_xor_sync(kAllLanes, top, w));
    const float next = fmaxf(m, top);
    if (!__any_sync(kAllLanes, block >= 0)) continue;
    const float base = next == -INFINITY ? 0.f : next;
    const float e = block >= 0 ? exp2f(score - base) : 0.f;
    const float keep = exp2f(m - base);
    m = next;
    l = l * keep + e;
    for (int i = 0; i < kCols; ++i) o[i] *= keep;
    for (int jj = 0; jj < 32; ++jj) {
      const int64_t at = __shfl_sync(kAllLanes, block, jj);
      const float w = __shfl_sync(kAllLanes, e, jj), scale = __shfl_sync(kAllLanes, vs, jj);
      if (at < 0) continue;
      const uint8_t* v = p.c.codes[1] + (at * p.c.page + ((j0 + jj) & (p.c.page - 1))) * kDim;
      for (int i = 0; i < kCols; ++i) o[i] = fmaf(w, scale * e4m3(v[lane * kCols + i]), o[i]);
    }
  }
  for (int w = 16; w > 0; w >>= 1) l += __shfl_xor_sync(kAllLanes, l, w);
  if (p.bad && __any_sync(kAllLanes, met_bad) && lane == 0) atomicAdd(p.bad, 1);
  T* out = static_cast<T*>(p.out) + r * kDim + lane * kCols;
  for (int i = 0; i < kCols; ++i) out[i] = Elem<DT>::make(l != 0.f ? o[i] / l : 0.f);
  if (p.lse && lane == 0) p.lse[r] = fmaf(m, kLn2, logf(l));
}

}  // namespace
}  // namespace dq4d

using namespace dq4d;

extern "C" {

int64_t dq4_kv8_attention_workspace_bytes(int64_t tokens, int64_t seqs, int32_t heads,
                                          int32_t kv_heads, int32_t head_dim) {
  if (tokens <= 0 || seqs <= 0 || heads < 1 || kv_heads < 1 || head_dim < 1) return 0;
  return decode_workspace_bytes();
}

int dq4_kv8_attention(const dq4_kv8_cache* cache, const void* q, int64_t q_token_stride,
                      int64_t q_head_stride, int32_t dtype, int64_t tokens, int32_t heads,
                      const int32_t* block_table, int64_t table_stride, int32_t table_width,
                      const int32_t* seq_lens, const int32_t* cu, int64_t seqs,
                      int32_t max_new, float scale, int32_t causal, int32_t window, void* out,
                      float* lse, void* workspace, int64_t workspace_bytes, int* bad,
                      void* stream) {
  AttendArgs p = {};
  if (const int st = make_cache(cache, &p.c)) return st;
  if (!valid_dtype(dtype, false)) return DQ4_ERR_DTYPE;
  if (heads < 1 || heads > 65535 || heads % cache->kv_heads != 0) return DQ4_ERR_HEADS;
  p.s = {block_table, table_stride, table_width, seq_lens, cu, seqs, tokens};
  if (const int st = check_batch(p.s)) return st;
  if (window < 0 || max_new < 0 || cache->pages * cache->kv_heads > INT32_MAX) return DQ4_ERR_N;
  if (tokens == 0 || seqs == 0) return DQ4_OK;
  if (!q || !out) return DQ4_ERR_NULL;
  if (misaligned(q, 16) || misaligned(out, 16) || q_token_stride % 8 || q_head_stride % 8 ||
      misaligned(lse, 4) || misaligned(bad, 4))
    return DQ4_ERR_ALIGN;
  if (!workspace || workspace_bytes < dq4_kv8_attention_workspace_bytes(
                                          tokens, seqs, heads, cache->kv_heads, cache->head_dim))
    return DQ4_ERR_WORKSPACE;
  if (misaligned(workspace, 256)) return DQ4_ERR_ALIGN;
  p.q = q;
  p.token_stride = q_token_stride;
  p.head_stride = q_head_stride;
  p.heads = heads;
  p.group = heads / cache->kv_heads;
  p.bf16 = dtype == DQ4_OUT_BF16;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.causal = causal;
  p.window = window;
  p.out = out;
  p.lse = lse;
  p.bad = bad;
  int dev, sms;
  if (const int st = current_device(&dev, &sms)) return st;
  if (int64_t(max_new) * p.group <= 64)
    return launch_decode(p, cache->head_dim, max_new * p.group, sms, workspace,
                         static_cast<cudaStream_t>(stream));
  const int64_t grid = (tokens * heads + kRowWarps - 1) / kRowWarps;
  if (grid > kMaxGrid) return DQ4_ERR_N;
  const bool bf16 = dtype == DQ4_OUT_BF16, small = cache->head_dim == 64;
  return launch_ordered(bf16 ? (small ? dq4_kv8_rows_kernel<DQ4_OUT_BF16, 64>
                                      : dq4_kv8_rows_kernel<DQ4_OUT_BF16, 128>)
                             : (small ? dq4_kv8_rows_kernel<DQ4_OUT_F16, 64>
                                      : dq4_kv8_rows_kernel<DQ4_OUT_F16, 128>),
                        dim3(unsigned(grid)), 32 * kRowWarps, 0,
                        static_cast<cudaStream_t>(stream), p);
}

}  // extern "C"
