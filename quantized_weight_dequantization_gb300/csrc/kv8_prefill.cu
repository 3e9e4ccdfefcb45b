// Attention over the 8-bit paged cache for many query rows a kv head (prompts and chunks of
// them): bound by the tensor cores, 4 dim operations for each pair of a row and a key.
//
// A CTA owns 256 query rows of one sequence and kv head (two tiles of 128; row = new token
// x head of the group, so that grouped heads share the keys) and walks the keys that any
// of them sees, 128 at a time:
//   S = Q K^T    (128 x 128, tcgen05, FP16 operands from shared memory, FP32 in TMEM)
//   P = 2^(c S + log2 vs - m + kTileLift)  FP16, written over S in TMEM
//   O += P V     (A operand P from TMEM, B operand V from shared memory, FP32 in TMEM)
//   l += P / vs
// with c the softmax scale times the row's and the key page's scale, and vs the page's V
// scale, which enters the exponent so that V's codes are the operand as they are.
//
// Roles (four groups of four warps):
//  * warps 0..3 and 4..7: the softmax of tile 0 and 1, one thread a row, no shuffles.  They
//    first bring the query rows to FP16 in shared memory.  m is the reference of a row, not
//    always its maximum: it moves, and O and l with it, only when a score passes it by
//    2^kSlack.  So a step's weights are computed against the reference at hand in one pass
//    over S, with the maximum found on the way, and kept in registers; only if some row has
//    to move is S read again;
//  * warps 8..11: bring keys and values from the cache to FP16 in shared memory (codes are
//    exact in FP16), loaded a step ahead into registers;
//  * warps 12 and 13: issue the products of tile 0 and 1.  A product holds its issuing thread
//    longer than the tensor cores take for its 128 x 128 x 16, so one thread would not keep
//    them busy.  While a tile's softmax runs, the tensor cores work for the other tile.
// Registers move from the last two groups to the softmax, which holds 64 packed weights and
// two chunks of S.
// Q, K and V are held K-major / MN-major with 128-byte swizzle: rows of 64 values.
#include "kv8_attend.cuh"

namespace dq4d {
namespace {

constexpr int kTileRows = 128;     // query rows of a tile = TMEM lanes
constexpr int kCtaRows = 2 * kTileRows;
constexpr int kKeys = 128;         // keys of a step
constexpr int kGrans = kKeys / 16; // granules of 16 keys: never of two pages
constexpr int kLoadThreads = 128;
constexpr int kPrefillThreads = kCtaRows + kLoadThreads + 128;
constexpr int kLoadWarp = kCtaRows / 32;
constexpr int kIssueWarp = kLoadWarp + kLoadThreads / 32;
// registers a thread of the softmax, load and issue groups: 128 each at launch
constexpr int kSoftmaxRegs = 152, kLoadRegs = 128, kIssueRegs = 80;
static_assert(2 * kSoftmaxRegs + kLoadRegs + kIssueRegs == 4 * 128, "what the launch holds");
constexpr int kSteps2 = 2;         // steps of keys in shared memory
// P <= 2^(kTileLift + kSlack) = 2^15 fits FP16
constexpr float kTileLift = 7.f, kSlack = 8.f;

template <int kDim>
struct PrefillSmem {
  static constexpr int kBlocks = kDim / 64;            // 64-value column blocks
  static constexpr int kBlock = kKeys * 128;           // bytes of one: 128 rows x 128 bytes
  static constexpr int kOperand = kBlocks * kBlock;
  static constexpr int kQ = 0;
  static constexpr int kK = 2 * kOperand;
  static constexpr int kV = kK + kSteps2 * kOperand;
  static constexpr int kGran = kV + kSteps2 * kOperand;  // [step][granule]{ks, log2 vs, 1 / vs, -}
  static constexpr int kBars = kGran + kSteps2 * kGrans * 16;
  static constexpr int kBytes = kBars + 32 * 8 + 1024;   // + alignment slack
  static_assert(kBytes + 256 <= 227 * 1024, "shared memory budget");
};
static_assert(PrefillSmem<128>::kBytes > 116 * 1024, "one CTA per SM: it takes all of TMEM");

// Shared-memory matrix descriptor of a B operand with N contiguous (MN-major), 128-byte
// swizzle: blocks of 64 values `block` bytes apart, groups of 8 rows along K 1024 apart.
__device__ __forceinline__ uint64_t smem_desc_mn(uint32_t addr, uint32_t block) {
  uint64_t d = static_cast<uint64_t>((addr >> 4) & 0x3FFF);
  d |= static_cast<uint64_t>(block >> 4) << 16;
  d |= static_cast<uint64_t>(1024 >> 4) << 32;
  d |= static_cast<uint64_t>(1) << 46;
  d |= static_cast<uint64_t>(2) << 61;
  return d;
}

__device__ __forceinline__ void sts_v4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c,
                                       uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};"
               :: "r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

__device__ __forceinline__ void commit_to(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];"
               :: "r"(bar) : "memory");
}

// 32 consecutive columns of this warp's TMEM lanes.  The registers may be read only after
// tmem_loaded(), and in volatile statements only (scale_pair): the compiler keeps those in
// order, but knows of no dependence between the wait and the registers.
__device__ __forceinline__ void tmem_load(uint32_t addr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
      "%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr));
}
__device__ __forceinline__ void tmem_loaded() {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

// Two FP32 values in a register pair, for the packed fma and add.
__device__ __forceinline__ uint64_t pair_of(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void split(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
// (a c + d, b c + d) for a and b from a TMEM load, c and d the same in both halves
__device__ __forceinline__ void scale_pair(uint32_t a, uint32_t b, uint64_t c, uint64_t d, float& x,
                                           float& y) {
  asm volatile(
      "{\n.reg .b64 v;\nmov.b64 v, {%2, %3};\nfma.rn.f32x2 v, v, %4, %5;\n"
      "mov.b64 {%0, %1}, v;\n}"
      : "=f"(x), "=f"(y) : "r"(a), "r"(b), "l"(c), "l"(d));
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// One pass over a row's 128 scores in TMEM (the next 32 loaded while 32 are used): weights
// 2^x, x = c S + bias - from, packed in FP16 into w; l gets sum 2^x / vs; the largest x is
// returned.  gran: the step's {ks, log2 vs, 1 / vs} of 16 keys each.  kMasked: only keys lo <=
// key + i < hi are seen.
template <bool kMasked>
__device__ __forceinline__ float softmax_pass(uint32_t scores, uint32_t gran, float cq,
                                              float from, int key, int lo, int hi, float& l,
                                              uint32_t (&w)[kKeys / 2]) {
  float top = -INFINITY;
  uint32_t s[2][32];
  tmem_load(scores, s[0]);
#pragma unroll
  for (int c = 0; c < kKeys / 32; ++c) {
    tmem_loaded();
    if (c + 1 < kKeys / 32) tmem_load(scores + 32 * (c + 1), s[(c + 1) & 1]);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint4 gi = lds_v4(gran + (2 * c + h) * 16);
      const float ck = cq * __uint_as_float(gi.x), add = __uint_as_float(gi.y) - from;
      const uint64_t ck2 = pair_of(ck, ck), off2 = pair_of(add, add);
      uint64_t sum2 = 0;
#pragma unroll
      for (int i = 0; i < 16; i += 2) {
        float x, y;
        scale_pair(s[c & 1][16 * h + i], s[c & 1][16 * h + i + 1], ck2, off2, x, y);
        if constexpr (kMasked) {
          const int k = key + 32 * c + 16 * h + i;
          if (k < lo || k >= hi) x = -INFINITY;
          if (k + 1 < lo || k + 1 >= hi) y = -INFINITY;
        }
        top = fmaxf(fmaxf(x, y), top);
        x = exp2_fast(x);
        y = exp2_fast(y);
        sum2 = add2(sum2, pair_of(x, y));
        w[16 * c + 8 * h + i / 2] = pack_f16(x, y);
      }
      float a, b;
      split(sum2, a, b);
      const float sum = a + b;
      // an unseen granule's scale may be no number
      if (!kMasked || sum != 0.f) l = fmaf(sum, __uint_as_float(gi.z), l);
    }
  }
  return top;
}

template <int kDim>
__global__ void __launch_bounds__(kPrefillThreads, 1) dq4_kv8_prefill_kernel(const AttendArgs p) {
  using S = PrefillSmem<kDim>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint32_t s_tmem;
  __shared__ volatile int s_abort;
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(base);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t bar0 = sbase + S::kBars;
  auto k_full = [&](int s) { return bar0 + 8 * s; };
  auto k_empty = [&](int s) { return bar0 + 8 * (2 + s); };
  auto v_full = [&](int s) { return bar0 + 8 * (4 + s); };
  auto v_empty = [&](int s) { return bar0 + 8 * (6 + s); };
  auto s_full = [&](int t) { return bar0 + 8 * (8 + t); };   // scores of tile t ready
  auto p_full = [&](int t) { return bar0 + 8 * (10 + t); };  // its weights written
  auto o_done = [&](int t) { return bar0 + 8 * (12 + t); };  // its O summed so far
  const uint32_t q_full = bar0 + 8 * 14;
  auto all_done = [&](int t) { return bar0 + 8 * (15 + t); };
  if (tid == 0) {
    s_abort = 0;
    for (int i = 0; i < 2; ++i) {
      mbar_init(k_full(i), kLoadThreads);
      mbar_init(v_full(i), kLoadThreads);
      mbar_init(k_empty(i), 2);
      mbar_init(v_empty(i), 2);
      mbar_init(s_full(i), 1);
      mbar_init(p_full(i), kTileRows);
      mbar_init(o_done(i), 1);
    }
    mbar_init(q_full, kCtaRows);
    mbar_init(all_done(0), 1);
    mbar_init(all_done(1), 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  wait_for_stream();

  // ---- this CTA's rows: heads fastest, then the row tiles from the last one back (with a
  // causal mask the last rows see the most keys, and the longest work starts first).
  // Sequence b's tiles start at unit row * group / 256 + b.
  const int64_t units = gridDim.x / p.c.heads;
  const int head = blockIdx.x % p.c.heads;
  const int64_t unit = units - 1 - blockIdx.x / p.c.heads;
  auto first_unit = [&](int64_t b) { return seq_row(p.s, b) * p.group / kCtaRows + b; };
  const int64_t b = find_last(p.s.seqs, unit, first_unit);
  const Seq q = seq_at(p.s, b);
  const int rows = q.n * p.group;
  const int r0 = int(unit - first_unit(b)) * kCtaRows;
  if (r0 >= rows) return;
  const int held = held_keys(p, q.len);
  // the steps of keys that tile t's rows see: from step 0 at key0 to steps[t]
  int steps[2];
  const int key0 = first_key(p, q.len - q.n + r0 / p.group) & ~(kKeys - 1);
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int last = min(rows, r0 + (t + 1) * kTileRows) - 1;
    const int end = last_key(p, q.len - q.n + last / p.group, held);
    steps[t] = r0 + t * kTileRows < rows ? max(0, (end - key0 + kKeys - 1) / kKeys) : 0;
  }
  const int nsteps = max(steps[0], steps[1]);

  if (warp == kIssueWarp) {  // the whole TMEM: S and P of both tiles, then O of both
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;"
                 :: "r"(smem_u32(&s_tmem)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tmem = s_tmem;
  auto t_s = [&](int t) { return tmem + t * kKeys; };
  auto t_o = [&](int t) { return tmem + 2 * kKeys + t * kDim; };
  auto fail = [&] {
    s_abort = 1;
    if (p.bad) atomicAdd(p.bad, 1);
  };
  auto wait = [&](uint32_t bar, int phase) {
    if (s_abort) return false;
    if (mbar_wait(bar, uint32_t(phase) & 1u)) return true;
    fail();
    return false;
  };
  // the same for a whole warp: true once every lane has seen the phase
  auto wait_warp = [&](uint32_t bar, int phase) {
    return bool(__all_sync(kAllLanes, wait(bar, phase)));
  };

  if (warp < kLoadWarp) {
    // ------------------------------------------------------------------ softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" :: "n"(kSoftmaxRegs));
    const int t = warp >> 2;
    const int row = tid & (kTileRows - 1);  // of the tile = its TMEM lane
    const uint32_t lanes = uint32_t((warp & 3) * 32) << 16;
    const int r = r0 + t * kTileRows + row;
    const bool real = r < rows;
    const int tok = min(r, rows - 1) / p.group;
    const int pos = q.len - q.n + tok;
    const int64_t at = (q.row + tok) * p.heads + head * p.group + (min(r, rows - 1) - tok * p.group);
    float cq;
    {
      uint4 raw[kDim / 8];
#pragma unroll
      for (int i = 0; i < kDim / 8; ++i) raw[i] = make_uint4(0, 0, 0, 0);
      if (real) {
        const uint16_t* src = static_cast<const uint16_t*>(p.q) +
                              (q.row + tok) * p.token_stride +
                              (head * p.group + r - tok * p.group) * p.head_stride;
#pragma unroll
        for (int i = 0; i < kDim / 8; ++i) raw[i] = __ldg(reinterpret_cast<const uint4*>(src) + i);
      }
      const uint32_t* w = reinterpret_cast<const uint32_t*>(raw);
      float top = 0.f;
#pragma unroll
      for (int i = 0; i < kDim / 2; ++i) {
        float x, y;
        widen2(w[i], p.bf16, x, y);
        top = fmaxf(top, fmaxf(fabsf(x), fabsf(y)));
      }
      float up, down;
      row_scaling(top, up, down);
      cq = down * fabsf(p.scale_log2);  // a negative scale turns the row instead
      if (p.scale_log2 < 0.f) up = -up;
#pragma unroll
      for (int i = 0; i < kDim / 8; ++i) {
        uint32_t h[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float x, y;
          widen2(w[4 * i + j], p.bf16, x, y);
          h[j] = pack_f16(x * up, y * up);
        }
        sts_v4(sbase + S::kQ + t * S::kOperand + (i / 8) * S::kBlock + row * 128 +
                   (((i & 7) ^ (row & 7)) << 4),
               h[0], h[1], h[2], h[3]);
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      mbar_arrive(q_full);
    }
    const int lo = first_key(p, pos), hi = last_key(p, pos, held);
    // keys that every row of the tile sees
    const int last_r = min(rows, r0 + (t + 1) * kTileRows) - 1;
    const int all_lo = first_key(p, q.len - q.n + last_r / p.group);
    const int all_hi = last_key(p, q.len - q.n + (r0 + t * kTileRows) / p.group, held);
    // from: what is taken off a row's exponents (the reference m less kTileLift)
    float from = 0.f, l = 0.f;
    bool fresh = true;  // no key seen yet
    const int n = steps[t];
    bool ok = true;
    for (int j = 0; j < n; ++j) {
      const int slot = j & 1;
      // (the step's scales come with V, long before the scores do)
      ok = wait_warp(v_full(slot), j >> 1) && wait_warp(s_full(t), j);
      if (!ok) break;
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      const uint32_t gran = sbase + S::kGran + slot * kGrans * 16;
      const int key = key0 + j * kKeys;
      const bool masked = key < all_lo || key + kKeys > all_hi;
      uint32_t w[kKeys / 2];
      float more = 0.f;
      const float top =
          masked ? softmax_pass<true>(t_s(t) + lanes, gran, cq, from, key, lo, hi, more, w)
                 : softmax_pass<false>(t_s(t) + lanes, gran, cq, from, key, lo, hi, more, w);
      const bool move = fresh ? top > -INFINITY : top > kTileLift + kSlack;
      if (__any_sync(kAllLanes, move)) {
        const float to = move ? from + top - kTileLift : from;
        const float keep = fresh ? 0.f : exp2_fast(from - to);
        from = to;
        fresh = fresh && !move;
        l *= keep;
        if (j > 0) {
          ok = wait_warp(o_done(t), j - 1);
          if (!ok) break;
          asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
#pragma unroll 1
          for (int c = 0; c < kDim / 32; ++c) {
            uint32_t o[32];
            tmem_ld32(t_o(t) + lanes + 32 * c, o);
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * keep);
            tmem_st<32>(t_o(t) + lanes + 32 * c, o);
          }
        }
        more = 0.f;
        softmax_pass<true>(t_s(t) + lanes, gran, cq, from, key, lo, hi, more, w);
      }
      l += more;
#pragma unroll
      for (int c = 0; c < kKeys / 64; ++c) {
        uint32_t part[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) part[i] = w[32 * c + i];
        tmem_st<32>(t_s(t) + lanes + 32 * c, part);
      }
      asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
      asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
      mbar_arrive(p_full(t));
    }
    // ---- the rows' results
    if (n > 0 && ok) {
      ok = wait_warp(o_done(t), n - 1);
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    }
    if (ok) {
      const float inv = l == 0.f ? 0.f : 1.f / l;
      uint4* out = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + at * kDim);
#pragma unroll
      for (int c = 0; c < kDim / 32; ++c) {
        uint32_t o[32];
        if (n > 0) {
          tmem_ld32(t_o(t) + lanes + 32 * c, o);
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = 0;
        }
        if (real) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
              w[k] = pack_out(__uint_as_float(o[8 * i + 2 * k]) * inv,
                              __uint_as_float(o[8 * i + 2 * k + 1]) * inv, p.bf16);
            out[4 * c + i] = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
      }
      if (real && p.lse)
        p.lse[at] = l == 0.f ? -INFINITY : fmaf(from, kLn2, logf(l));
    }
  } else if (warp < kIssueWarp) {
    // --------------------------------------------------- keys and values to FP16
    // A thread takes 16 bytes (16 values) of a row in each pass: piece `col` of rows row0,
    // row0 + kRowsPass, ...  Eight neighbouring lanes take four pieces of one 64-value block
    // in two rows, so that their 16-byte stores meet eight different bank groups.
    constexpr int kCols = kDim / 16;                 // pieces of a row
    constexpr int kRowsPass = kLoadThreads / kCols;  // 16 or 32
    constexpr int kPasses = kKeys / kRowsPass;
    const int lw = warp - kLoadWarp;
    const int col = kDim == 128 ? (lane & 3) + ((lane >> 3) & 1) * 4 : lane & 3;
    const int row0 =
        kDim == 128 ? lw * 4 + ((lane >> 2) & 1) + ((lane >> 4) & 1) * 2 : lw * 8 + (lane >> 2);
    const uint32_t line = (col >> 2) * S::kBlock + row0 * 128;
    const uint32_t to[2] = {line + (((2 * (col & 3)) ^ (row0 & 7)) << 4),
                            line + (((2 * (col & 3) + 1) ^ (row0 & 7)) << 4)};
    bool met_bad = held < q.len;
    const int32_t* table = p.s.table + b * p.s.table_stride;
    // Lane x holds granule x % kGrans of a step: its page's block (page * kv_heads + head), or
    // -1 where there are no such keys.
    auto find_block = [&](int j) {
      const int key = key0 + j * kKeys + (lane & (kGrans - 1)) * 16;
      if (j >= nsteps || key >= held) return -1;
      const int id = __ldg(table + (key >> p.c.log2_page));
      if (id >= 0 && id < p.c.pages) return int(id * p.c.heads + head);
      met_bad = true;
      return -1;
    };
    uint4 raw[2][kPasses];
    float gk, gv;
    const int page_bytes = p.c.page * kDim;
    auto fetch = [&](int j, int block) {
#pragma unroll
      for (int i = 0; i < kPasses; ++i) {
        const int row = row0 + i * kRowsPass;
        const int key = key0 + j * kKeys + row;
        int at = __shfl_sync(kAllLanes, block, row >> 4);
        if (key >= held) at = -1;  // a slot never written: it may hold no number
        const int64_t off =
            int64_t(at) * page_bytes + ((key & (p.c.page - 1)) * kDim + col * 16);
#pragma unroll
        for (int x = 0; x < 2; ++x)
          raw[x][i] = at < 0 ? make_uint4(0, 0, 0, 0)
                             : __ldg(reinterpret_cast<const uint4*>(p.c.codes[x] + off));
      }
      gk = block < 0 ? 0.f : __ldg(p.c.scale[0] + block);
      gv = block < 0 ? -1.f : __ldg(p.c.scale[1] + block);
    };
    auto put = [&](uint32_t at, const uint4& v) {
      sts_v4(at + to[0], f16_of_e4m3(v.x), f16_of_e4m3_high(v.x), f16_of_e4m3(v.y),
             f16_of_e4m3_high(v.y));
      sts_v4(at + to[1], f16_of_e4m3(v.z), f16_of_e4m3_high(v.z), f16_of_e4m3(v.w),
             f16_of_e4m3_high(v.w));
    };
    fetch(0, find_block(0));
    int block = find_block(1);
    for (int j = 0; j < nsteps; ++j) {
      const int slot = j & 1;
      bool ok = j < kSteps2 || wait(k_empty(slot), (j >> 1) - 1);
      if (!__all_sync(kAllLanes, ok)) break;
#pragma unroll
      for (int i = 0; i < kPasses; ++i)
        put(sbase + S::kK + slot * S::kOperand + i * kRowsPass * 128, raw[0][i]);
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      mbar_arrive(k_full(slot));
      ok = j < kSteps2 || wait(v_empty(slot), (j >> 1) - 1);
      if (!__all_sync(kAllLanes, ok)) break;
#pragma unroll
      for (int i = 0; i < kPasses; ++i)
        put(sbase + S::kV + slot * S::kOperand + i * kRowsPass * 128, raw[1][i]);
      if (lw == 0 && lane < kGrans) {
        // keys that are not there: S = 0 and an exponent of -infinity
        const float vs = used_scale(gv);
        const bool none = gv == -1.f;
        sts_v4(sbase + S::kGran + (slot * kGrans + lane) * 16, __float_as_uint(gk),
               __float_as_uint(none ? -INFINITY : log2f(vs)), __float_as_uint(none ? 0.f : 1.f / vs),
               0);
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      mbar_arrive(v_full(slot));
      if (j + 1 < nsteps) {
        fetch(j + 1, block);
        block = find_block(j + 2);
      }
    }
    if (p.bad && __any_sync(kAllLanes, met_bad) && lane == 0) atomicAdd(p.bad, 1);
  } else {
    // -------------------------------------------------------------- the products
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(kIssueRegs));
    const int t = warp - kIssueWarp;
    if (t < 2 && lane == 0) {
      const uint32_t idesc_s = instr_desc_f16<kTileRows, kKeys>(false);
      const uint32_t idesc_o =
          instr_desc_f16<kTileRows, kDim>(false) | (1u << 16);  // B: N contiguous
      const int n = steps[t];
      auto scores = [&](int j) {  // S = Q K_j^T
        const uint32_t a = sbase + S::kQ + t * S::kOperand;
        const uint32_t k = sbase + S::kK + (j & 1) * S::kOperand;
#pragma unroll
        for (int i = 0; i < kDim / 16; ++i) {
          const uint32_t off = (i / 4) * S::kBlock + (i % 4) * 32;
          asm volatile(
              "{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\n"
              "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}"
              :: "r"(t_s(t)), "l"(smem_desc(a + off)), "l"(smem_desc(k + off)), "r"(idesc_s),
                 "r"(i > 0 ? 1u : 0u));
        }
        commit_to(s_full(t));
      };
      auto values = [&](int j) {  // O += P V_j
        const uint32_t v = sbase + S::kV + (j & 1) * S::kOperand;
#pragma unroll
        for (int i = 0; i < kKeys / 16; ++i) {
          asm volatile(
              "{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\n"
              "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}"
              :: "r"(t_o(t)), "r"(t_s(t) + 8 * i), "l"(smem_desc_mn(v + i * 2048, S::kBlock)),
                 "r"(idesc_o), "r"(j > 0 || i > 0 ? 1u : 0u));
        }
        commit_to(o_done(t));
      };
      // Both issuers pass every step's barriers, also those past their tile's last step, so
      // that each slot's phase ends with one arrival of each.
      // The weights are waited for last: what follows is then issued in one go.
      bool ok = nsteps > 0 && wait(q_full, 0);
      for (int j = -1; j < nsteps && ok; ++j) {
        const bool more = j + 1 < nsteps;
        if (j >= 0) ok = wait(v_full(j & 1), j >> 1);
        if (more) ok = ok && wait(k_full((j + 1) & 1), (j + 1) >> 1);
        if (j >= 0 && j < n) ok = ok && wait(p_full(t), j);
        if (!ok) break;
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        if (j >= 0 && j < n) values(j);
        if (j >= 0) commit_to(v_empty(j & 1));
        if (j + 1 < n) scores(j + 1);
        if (more) commit_to(k_empty((j + 1) & 1));
      }
      // every product issued is done before TMEM and shared memory go
      commit_to(all_done(t));
      mbar_wait(all_done(t), 0);
    }
  }
  __syncwarp();
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  if (warp == kIssueWarp) {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" :: "r"(tmem));
  }
}

template <int kDim>
int launch_one(const AttendArgs& p, cudaStream_t stream) {
  constexpr int kBytes =
      PrefillSmem<kDim>::kBytes > 117 * 1024 ? PrefillSmem<kDim>::kBytes : 117 * 1024;
  const int64_t units = p.s.tokens * p.group / kCtaRows + p.s.seqs;
  if (units * p.c.heads > kMaxGrid) return DQ4_ERR_N;
  auto kernel = dq4_kv8_prefill_kernel<kDim>;
  const cudaError_t e =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes);
  if (e != cudaSuccess) return fail_cuda(DQ4_ERR_LAUNCH, e);
  return launch_ordered(kernel, dim3(unsigned(units * p.c.heads)), kPrefillThreads, kBytes, stream,
                        p);
}

}  // namespace

int launch_prefill(const AttendArgs& p, int head_dim, cudaStream_t stream) {
  return head_dim == 64 ? launch_one<64>(p, stream) : launch_one<128>(p, stream);
}

}  // namespace dq4d
