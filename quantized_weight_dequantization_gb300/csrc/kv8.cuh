// The 8-bit paged key/value cache (dq4_attn.h) as its kernels see it.
#pragma once

#include "attn.cuh"

namespace dq4d {

struct Kv8 {
  uint8_t* codes[2];  // k, v: [pages][kv_heads][page][dim]
  float* scale[2];    // [pages][kv_heads]
  int64_t pages;
  int heads, page, log2_page;
};

// The ragged batch of a call: its new tokens, lengths and pages.
struct Batch {
  const int32_t* table;
  int64_t table_stride;
  int table_width;
  const int32_t* lens;
  const int32_t* cu;  // null: one token each
  int64_t seqs, tokens;
};

namespace {

// Sequence b's first new token, new tokens, and length with them.  Whatever cu holds, the
// rows stay inside the call's tokens.
struct Seq {
  int64_t row;
  int n, len;
};

__device__ __forceinline__ int64_t seq_row(const Batch& s, int64_t b) {
  if (s.cu == nullptr) return b;
  const int64_t r = load_global(s.cu + b);
  return r < 0 ? 0 : r > s.tokens ? s.tokens : r;
}

__device__ __forceinline__ Seq seq_at(const Batch& s, int64_t b) {
  Seq q;
  q.row = seq_row(s, b);
  const int64_t n = s.cu ? seq_row(s, b + 1) - q.row : 1;
  q.n = n < 0 ? 0 : int(n);
  q.len = load_global(s.lens + b);
  return q;
}

// ------------------------------------------------------------------------ host side
inline int make_cache(const dq4_kv8_cache* c, Kv8* k) {
  if (!c) return DQ4_ERR_NULL;
  if (c->head_dim != 64 && c->head_dim != 128) return DQ4_ERR_HEADS;
  if (c->kv_heads < 1 || c->kv_heads > 65535) return DQ4_ERR_HEADS;
  if (c->page < 16 || c->page > 256 || !is_pow2(c->page)) return DQ4_ERR_PAGE;
  if (c->pages < 0 || c->pages > INT32_MAX) return DQ4_ERR_N;
  if (c->pages > 0 && (!c->k || !c->v || !c->k_scale || !c->v_scale)) return DQ4_ERR_NULL;
  if (misaligned(c->k, 16) || misaligned(c->v, 16) || misaligned(c->k_scale, 4) ||
      misaligned(c->v_scale, 4))
    return DQ4_ERR_ALIGN;
  *k = {{static_cast<uint8_t*>(c->k), static_cast<uint8_t*>(c->v)},
        {c->k_scale, c->v_scale},
        c->pages,
        c->kv_heads,
        c->page,
        log2_exact(c->page)};
  return DQ4_OK;
}

inline int check_batch(const Batch& s) {
  if (s.tokens < 0 || s.tokens > INT32_MAX || s.seqs < 0 || s.seqs > (1 << 24) ||
      s.table_width < 0 || (!s.cu && s.tokens != s.seqs))
    return DQ4_ERR_N;
  if (s.tokens == 0 || s.seqs == 0) return DQ4_OK;
  if (!s.lens || (s.table_width > 0 && !s.table)) return DQ4_ERR_NULL;
  if (misaligned(s.table, 4) || misaligned(s.lens, 4) || misaligned(s.cu, 4)) return DQ4_ERR_ALIGN;
  return DQ4_OK;
}

}  // namespace
}  // namespace dq4d
