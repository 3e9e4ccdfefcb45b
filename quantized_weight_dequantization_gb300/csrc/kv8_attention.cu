// The entry point of the attention over the 8-bit paged cache, dq4_kv8_attention
// (dq4_attn.h): checks its arguments and chooses the kernel.
#include "kv8_attend.cuh"

namespace dq4d {
namespace {

// Whether a call goes to the kernel for many query rows a kv head.  The one for few takes
// about a third of the time for a unit of 64 keys that the other takes for its 256 rows, but
// once for each 8 or 16 rows; the other starts about 15 us later (two launches, longer units).
// With `keys` the most that a sequence can hold or see, both measured at 8 kv heads of 128, in
// us (few / many):
//   rows   1 x 1000   1 x 20000   8 x 2000   8 x 10000   32 x 1000   32 x 5000   (seqs x keys)
//     32    15 / 31     34 / 73    26 / 41     78 / 95     49 / 59    135 / 169
//     64    15 / 32     46 / 71    43 / 42    130 / 98     79 / 62    243 / 172
//    128    15 / 33     70 / 63    68 / 44    232 / 103   133 / 65    444 / 184
//    512    33 / 40    221 / 89   206 / 71    832 / 204   449 / 146  1680 / 398
bool many_rows(int64_t rows, int64_t seqs, int64_t kv_heads, int64_t keys) {
  const double units = double(seqs * kv_heads) * double((keys + 63) / 64);  // may be huge
  const double tiles = double((rows + 15) / 16);
  return tiles > 2 && (tiles - 2) * units > 6000;
}

}  // namespace
}  // namespace dq4d

using namespace dq4d;

extern "C" {

int64_t dq4_kv8_attention_workspace_bytes(int64_t tokens, int64_t seqs, int32_t heads,
                                          int32_t kv_heads, int32_t head_dim) {
  if (tokens <= 0 || seqs <= 0 || heads < 1 || kv_heads < 1 || head_dim < 1) return 0;
  const int64_t few = decode_workspace_bytes();
  const int64_t many = prefill_workspace_bytes(tokens, seqs, heads / kv_heads, head_dim);
  return few > many ? few : many;
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
  // (query rows of a kv head, and blocks of the cache, are counted in 32 bits)
  if (window < 0 || max_new < 0 || cache->pages * cache->kv_heads > INT32_MAX ||
      tokens * (heads / cache->kv_heads) > INT32_MAX)
    return DQ4_ERR_N;
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
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int64_t rows = int64_t(max_new) * p.group;
  int64_t keys = int64_t(table_width) * cache->page;
  if (window > 0 && keys > int64_t(window) + max_new) keys = int64_t(window) + max_new;
  if (many_rows(rows, seqs, cache->kv_heads, keys))
    return launch_prefill(p, cache->head_dim, dev, sms, workspace, s);
  return launch_decode(p, cache->head_dim, rows, keys, dev, sms, workspace, s);
}

}  // extern "C"
