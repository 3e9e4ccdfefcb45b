// Attention over the 8-bit paged cache for many query rows a kv head (prompts and chunks of
// them): bound by the tensor cores, 4 dim operations for each pair of a row and a key.
//
// A unit is 256 query rows of one sequence and kv head: two tiles of 128 (row = new token x
// head of the group, so that grouped heads share the keys).  It walks the keys that any of
// its rows sees, 64 at a step:
//   S = Q K^T    (128 x 64 a tile, tcgen05, FP16 operands from shared memory, FP32 in TMEM)
//   P = 2^(c S + log2 vs - m + kTileLift)  FP16, written over S in TMEM
//   O += P V     (A operand P from TMEM, B operand V from shared memory, FP32 in TMEM)
//   l += P / vs   (in units of 2^16)
// with c the softmax scale times the row's and the key page's scale, and vs the page's V
// scale, which enters the exponent so that V's codes are the operand as they are.
//
// One CTA runs per SM, on an equal run of all units' steps, whatever the lengths are: a
// planning kernel lists the units and where their steps start.  A unit that several CTAs
// share is summed from their FP32 parts, in the order of the keys, by the last of them to
// finish, tile by tile.
//
// Roles (four groups of four warps):
//  * warps 0..3 and 4..7: the softmax of tile 0 and 1, one thread a row, no shuffles.  They
//    first bring a unit's query rows to FP16 in shared memory, and at its end write the
//    result or the part.  m is the reference of a row, not always its maximum: it moves, and
//    O and l with it, only when a score passes it by 2^kSlack.  So one pass over S gives a
//    step's weights: the maximum of 32 scores is looked at before their exponentials, and if
//    some row has to move, the weights before them are scaled by a power of two;
//  * warps 8..11: bring keys and values from the cache to FP16 in shared memory (codes are
//    exact in FP16), their codes copied to shared memory some steps ahead, where each thread
//    takes back what it asked for itself;
//  * warps 12 .. 15: issue Q K^T of tile 0 and 1, and P V of tile 0 and 1.  The tensor cores
//    take a new product about when the last one ends, so that a thread that waits for one
//    kind's operands would keep them from the other kinds.
// Each tile has two S buffers: the scores of the next step are computed while the softmax
// works on this one, and P V of this one while it works on the next.
// Q, K and V are held K-major / MN-major with 128-byte swizzle: rows of 64 values.
//
// Measured: a causal prompt of 8192 tokens, 32 heads over 8 of 128, BF16, 564 to 576 us by its
// data (550 GFLOP, 0.96 PFLOP/s, 0.51 of a library GEMM's rate); 5 chunks of up to 1025 tokens
// over up to 16411 keys, 16 heads over 8 of 64, 340 us (186 GFLOP, 548 TFLOP/s; at 64 a key takes
// as many exponentials and scores for half the operations).  A step takes about 2000 cycles for 1300 of the tensor
// cores': the conversion of the codes, and roles that share the issue slots (half of them busy)
// and the instruction caches; starting and ending a unit takes about nine steps more.  Dropped
// after measuring: one thread that issues all products, the softmax tiles taking turns, codes by
// TMA (each within 5 %), the next unit's query rows prefetched to L2 (605 us for 607), issue code
// with all operands static (1954 us: it no longer fits the instruction caches).  Times of
// dropped forms are those of their day, to be compared with each other.
#include "kv8_attend.cuh"

namespace dq4d {
namespace {

constexpr int kTileRows = 128;     // query rows of a tile = TMEM lanes
constexpr int kUnitRows = 2 * kTileRows;
constexpr int kKeys = 64;          // keys of a step
constexpr int kGrans = kKeys / 16; // granules of 16 keys: never of two pages
constexpr int kSlots = 3;          // steps of keys and of values in shared memory, as FP16
constexpr int kRawSlots = 4;       // and of their codes
// steps whose scales stay in shared memory: a step's are read until its weights are done, by
// when the keys of no step past the fifth after it have been placed.  (A slot of keys is free
// again once both tiles have passed its step.  With steps of its own a tile passes none before
// the weights of the second step before it; without, none past the second after its last step
// before that one's weights: see `last`.)
constexpr int kGranSlots = 8;
constexpr int kLoadThreads = 128;
constexpr int kPrefillThreads = kUnitRows + kLoadThreads + 128;
constexpr int kLoadWarp = kUnitRows / 32;
constexpr int kIssueWarp = kLoadWarp + kLoadThreads / 32;
constexpr int kMaxCtas = 160;      // CTAs the workspace has room for
// What starting and ending a unit counts for in the division of the work, in steps: about 9 by
// the cycles of most runs.  When it was chosen, a prompt of 8192 took 536 to 560 us with 13, 528 to
// 562 with 10 and 520 to 571 with 8, by its data, one of 2048 78, 75 and 74.
constexpr int kOpening = 10;
constexpr int kMinSteps = 16;      // steps that a CTA takes at least
constexpr int kPlanThreads = 1024;
// P <= 2^(kTileLift + kSlack) < 65504 fits FP16.  A row's reference is set so that its largest
// weight so far is 2^13 to 2^14: weights down to 2^-14, 2^-27 of the largest, have all their bits, smaller
// ones a step of 2^-24.  (That shows where one key dominates that has no values.)  The slack is
// what a row's maximum may grow by before the rows of its warp move.  A prompt of 8192, by its
// data (two draws of one distribution), and chunks over 16k at dim 64: 578, 562 and 334 us.  With the moves found after the exponentials, which are then computed again, 681, 644 and
// 380, and 583, 529 and 342 with 2^2 and 2^13, where small weights lose eleven bits.
constexpr float kTileLift = 13.f, kSlack = 2.9f;

// A unit, as planned.
struct alignas(16) Unit {
  int64_t start;     // its first step among a kv head's, kOpening of them before its keys
  int b, r0, rows;   // sequence, first query row, and the sequence's rows
  int key0;          // first key, a multiple of kKeys
  int steps[2];      // of its tiles (0: no rows)
  int pos, row;      // the sequence's first new token: its position, and its row of q
  int held;          // the sequence's keys that are there
  int first;         // the first key of the pages that hold a key which some row sees
  int all_lo, all_hi;  // the keys that every row sees
};
static_assert(sizeof(Unit) == 64, "read as 16-byte words");

template <int kDim>
struct PrefillSmem {
  static constexpr int kBlocks = kDim / 64;         // 64-value column blocks
  static constexpr int kQBlock = kTileRows * 128;   // bytes of one of Q: 128 rows x 128 bytes
  static constexpr int kBlock = kKeys * 128;        // and of one of K or V
  static constexpr int kQTile = kBlocks * kQBlock;
  static constexpr int kOperand = kBlocks * kBlock;
  static constexpr int kQ = 0;
  static constexpr int kK = 2 * kQTile;
  static constexpr int kV = kK + kSlots * kOperand;
  static constexpr int kGran = kV + kSlots * kOperand;  // [slot][granule]{ks, log2 vs, kSumUnit / vs, -}
  // codes: [slot][K, V][pass][load thread], 16 bytes each; and {block, ks, vs} of granules
  static constexpr int kRawPass = kLoadThreads * 16;
  static constexpr int kRaw = kGran + kGranSlots * kGrans * 16;
  static constexpr int kNote = kRaw + kRawSlots * 2 * kKeys * kDim;
  // [tile][step % 4] keys of a mixed step with NaN codes of V; [tile] rows that see such, a bit each
  static constexpr int kNan = kNote + kRawSlots * kGrans * 16;
  static constexpr int kLost = kNan + 2 * 4 * 16;
  static constexpr int kBars = kLost + 2 * 16;
  static constexpr int kBytes = kBars + 38 * 8 + 1024;  // + alignment slack
  static_assert(kBytes + 256 <= 227 * 1024, "shared memory budget");
};

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

// The products and their commits, by the lane of the warp that leads (the other operands are
// the same for all lanes).  A from shared memory, or from TMEM.
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add,
                                       uint32_t leads) {
  asm volatile(
      "{\n.reg .pred p, q;\nsetp.ne.b32 p, %4, 0;\nsetp.ne.b32 q, %5, 0;\n"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}"
      :: "r"(d), "l"(a), "l"(b), "r"(idesc), "r"(uint32_t(add)), "r"(leads));
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add,
                                       uint32_t leads) {
  asm volatile(
      "{\n.reg .pred p, q;\nsetp.ne.b32 p, %4, 0;\nsetp.ne.b32 q, %5, 0;\n"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}"
      :: "r"(d), "r"(a), "l"(b), "r"(idesc), "r"(uint32_t(add)), "r"(leads));
}
__device__ __forceinline__ void commit_if(uint32_t bar, uint32_t leads) {
  asm volatile(
      "{\n.reg .pred q;\nsetp.ne.b32 q, %1, 0;\n"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}"
      :: "r"(bar), "r"(leads) : "memory");
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

// A row's sums: weights are 2^(s - from) of its scores s in base 2.
struct RowSum {
  float from = 0.f;
  float peak = -INFINITY;  // log2 of the largest weight so far
  float l = 0.f;
  bool fresh = true;       // no key seen yet
};

// One pass over a row's 64 scores in TMEM (the next 32 loaded while 32 are used): weights
// 2^x, x = c S + bias - from, packed in FP16 into w; l gets sum 2^x / vs.  gran: the step's {ks,
// log2 vs, kSumUnit / vs} of 16 keys each.  kMasked: only keys lo <= key + i < hi are seen.
// If some row's weights would grow past 2^(kTileLift + kSlack), all rows of the warp move their
// references to their maxima, and what has been summed by powers of two: the 32 scores at hand
// before their exponentials, the weights before them and l here, O by the caller (returns whether
// they moved, and the factor in keep).
template <bool kMasked>
__device__ __forceinline__ bool softmax_pass(uint32_t scores, uint32_t gran, float cq, int key,
                                             int lo, int hi, RowSum& r, float& keep,
                                             uint32_t (&w)[kKeys / 2]) {
  bool moved = false;
  keep = 1.f;
  uint32_t s[kKeys / 32][32];
  tmem_load(scores, s[0]);
#pragma unroll
  for (int c = 0; c < kKeys / 32; ++c) {
    tmem_loaded();
    float x[32], inverse[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint4 gi = lds_v4(gran + (2 * c + h) * 16);
      const float ck = cq * __uint_as_float(gi.x), add = __uint_as_float(gi.y) - r.from;
      const uint64_t ck2 = pair_of(ck, ck), off2 = pair_of(add, add);
      inverse[h] = __uint_as_float(gi.z);
#pragma unroll
      for (int i = 16 * h; i < 16 * h + 16; i += 2) {
        scale_pair(s[c][i], s[c][i + 1], ck2, off2, x[i], x[i + 1]);
        if constexpr (kMasked) {
          const int k = key + 32 * c + i;
          if (k < lo || k >= hi) x[i] = -INFINITY;
          if (k + 1 < lo || k + 1 >= hi) x[i + 1] = -INFINITY;
        }
        r.peak = fmaxf(fmaxf(x[i], x[i + 1]), r.peak);
      }
    }
    if (__any_sync(kAllLanes, r.peak > (r.fresh ? -INFINITY : kTileLift + kSlack))) {
      // (of a fresh row nothing has been summed, and its peak may be anything)
      const float over = r.peak - kTileLift;
      const float by = !r.fresh ? fmaxf(0.f, floorf(over)) : r.peak > -INFINITY ? over : 0.f;
      const float factor = r.fresh ? 1.f : exp2_fast(-by);
      r.from += by;
      r.peak -= by;
      r.l *= factor;
      keep *= factor;
      moved = true;
#pragma unroll
      for (int i = 0; i < 32; ++i) x[i] -= by;
      // (in two factors, as FP16 holds no power below 2^-24)
      const float most = fminf(by, 15.f);
      const __half2 f1 = __float2half2_rn(r.fresh ? 1.f : exp2_fast(-most));
      const __half2 f2 = __float2half2_rn(r.fresh ? 1.f : exp2_fast(most - by));
#pragma unroll
      for (int i = 0; i < 16 * c; ++i) {
        __half2 v;
        memcpy(&v, &w[i], 4);
        v = __hmul2(__hmul2(v, f1), f2);
        memcpy(&w[i], &v, 4);
      }
      r.fresh = r.fresh && !(r.peak > -INFINITY);
    }
    if (c + 1 < kKeys / 32) tmem_load(scores + 32 * (c + 1), s[c + 1]);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint64_t sum2 = 0;
#pragma unroll
      for (int i = 16 * h; i < 16 * h + 16; i += 2) {
        const float y = exp2_fast(x[i]), z = exp2_fast(x[i + 1]);
        sum2 = add2(sum2, pair_of(y, z));
        w[16 * c + i / 2] = pack_f16(y, z);
      }
      float y, z;
      split(sum2, y, z);
      const float sum = y + z;
      // an unseen granule's scale may be no number
      if (!kMasked || sum != 0.f) r.l = fmaf(sum, inverse[h], r.l);
    }
  }
  return moved;
}

// A step's V as FP16 at `values`: what is no number becomes zero, and the keys that had such are
// returned, a bit each.  Either tile's warp looks for itself, so what it finds it notes (`mine`:
// {keys, step}) before it goes, for the other one (`other`), which may come too late to see it.
template <int kDim>
__device__ __noinline__ uint64_t clean_values(uint32_t values, uint32_t mine, uint32_t other, int g) {
  const int lane = threadIdx.x & 31;
  constexpr int kPieces = kDim / 8;  // of 16 bytes, of a key
  auto piece_at = [&](int key, int i) {
    return values + (i / 8) * PrefillSmem<kDim>::kBlock + key * 128 + (((i ^ key) & 7) << 4);
  };
  uint64_t keys = 0;
#pragma unroll 1
  for (int key = lane; key < kKeys; key += 32) {
    uint32_t top = 0;  // the largest of each half, or NaN if one is
#pragma unroll 4
    for (int i = 0; i < kPieces; ++i) {
      const uint4 v = lds_v4(piece_at(key, i));
      top = larger_f16x2(larger_f16x2(larger_f16x2(top, v.x), larger_f16x2(v.y, v.z)), v.w);
    }
    keys |= uint64_t(__ballot_sync(kAllLanes, nan_halves(top) != 0)) << (key & 32);
  }
  if (keys != 0) {
    if (lane == 0) sts_v4(mine, uint32_t(keys), uint32_t(keys >> 32), uint32_t(g), 0);
    __threadfence_block();
    __syncwarp();
#pragma unroll 1
    for (int key = lane; key < kKeys; key += 32) {
      if (!(keys >> key & 1)) continue;
#pragma unroll 1
      for (int i = 0; i < kPieces; ++i) {
        const uint4 v = lds_v4(piece_at(key, i));
        auto clean = [](uint32_t w) { return w & ~((nan_halves(w) >> 15) * 0xFFFFu); };
        sts_v4(piece_at(key, i), clean(v.x), clean(v.y), clean(v.z), clean(v.w));
      }
    }
  }
  // (also for what the other warp wrote, and this one has seen)
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  __threadfence_block();
  __syncwarp();
  const uint4 note = lds_v4(other);
  return int(note.z) == g ? keys | note.x | uint64_t(note.y) << 32 : keys;
}

// The call, and where its workspace holds what.
struct PrefillArgs {
  AttendArgs a;
  Unit* units;
  int64_t max_units;
  int64_t* total;   // a kv head's steps, all units
  int* count;       // [CTA][tile] arrivals at a shared unit whose last part the CTA has
  float2* stats;    // [CTA][2][tile][row]{from, l}
  float4* part;     // [CTA][2][tile][dim / 4][row] unnormalized O
};

// List the units: sequence b's stand at index row / 256 + b and on, as many as its rows need;
// indexes in between are units without rows.  One CTA, as the list is short (a unit for 256 rows)
// and each unit's start needs the sum before it: 5.5 us for 4 sequences from cold caches,
// where the other kernel takes 38.
__global__ void __launch_bounds__(kPlanThreads) dq4_kv8_plan_kernel(const PrefillArgs w) {
  const AttendArgs& p = w.a;
  __shared__ int64_t s_sums[32];
  wait_for_stream();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  auto first_unit = [&](int64_t b) { return seq_row(p.s, b) * p.group / kUnitRows + b; };
  int64_t total = 0;
  for (int64_t u0 = 0; u0 < w.max_units; u0 += kPlanThreads) {
    const int64_t u = u0 + tid;
    Unit x = {};
    int64_t cost = 0;
    if (u < w.max_units) {
      int64_t lo = 0, hi = p.s.seqs;  // the last sequence whose first unit is at or before u
      while (hi - lo > 1) {
        const int64_t mid = (lo + hi) / 2;
        if (first_unit(mid) <= u) lo = mid; else hi = mid;
      }
      const Seq q = seq_at(p.s, lo);
      x.b = int(lo);
      x.rows = q.n * p.group;
      const int64_t r0 = (u - first_unit(lo)) * kUnitRows;
      if (r0 < x.rows) {
        x.r0 = int(r0);
        x.pos = q.len - q.n;
        x.row = int(q.row);
        x.held = held_keys(p, q.len);
        const int first_pos = x.pos + x.r0 / p.group;
        x.first = first_key(p, first_pos) & -p.c.page;
        x.key0 = min(first_key(p, first_pos), x.held) & ~(kKeys - 1);
        x.all_lo = first_key(p, x.pos + (min(x.rows, x.r0 + kUnitRows) - 1) / p.group);
        x.all_hi = last_key(p, first_pos, x.held);
        if (x.held < q.len && p.bad) atomicAdd(p.bad, 1);
        for (int t = 0; t < 2; ++t) {
          const int first = x.r0 + t * kTileRows;
          if (first >= x.rows) break;
          const int last = min(x.rows, first + kTileRows) - 1;
          const int end = last_key(p, x.pos + last / p.group, x.held);
          // (one at least: rows that see no key get their zeros)
          x.steps[t] = max(1, (end - x.key0 + kKeys - 1) / kKeys);
        }
        cost = max(x.steps[0], x.steps[1]) + kOpening;
      }
    }
    int64_t run = cost;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t up = __shfl_up_sync(kAllLanes, run, o);
      if (lane >= o) run += up;
    }
    __syncthreads();
    if (lane == 31) s_sums[warp] = run;
    __syncthreads();
    int64_t before = total + run - cost;
    for (int i = 0; i < kPlanThreads / 32; ++i) {
      if (i < warp) before += s_sums[i];
      total += s_sums[i];
    }
    x.start = before;
    if (u < w.max_units) w.units[u] = x;
  }
  if (tid == 0) *w.total = total;
}

// A step of a unit is mixed if some row does not see one of its keys.  A weight of 0 does not
// keep a value that is no number from its row, so in such steps V's codes that are none become
// zeros before the product, and l brings them to the rows that see their keys.  (By the warps
// that issue P V, which have the time: a prompt of 8192 takes 531 -> 544 us.  By those that bring
// the values, or by the softmax, 550 to 573.)
__device__ __forceinline__ bool mixed_step(int all_lo, int all_hi, int key) {
  return key < all_lo || key + kKeys > all_hi;
}

// The rows of a tile that see a key of `nan` (bits of the keys from `key` on) are noted at
// `lost`, after all rows have read what was noted of the unit before.  By one warp.
__device__ __noinline__ void lose_rows(const AttendArgs& p, const Unit& x, int t, int key,
                                       uint64_t nan, uint32_t lost) {
  const int lane = threadIdx.x & 31;
#pragma unroll 1
  for (int i = 0; i < kTileRows / 32; ++i) {
    const int r = min(x.r0 + t * kTileRows + i * 32 + lane, x.rows - 1), pos = x.pos + r / p.group;
    const bool sees = nan & seen_keys(key, first_key(p, pos), last_key(p, pos, x.held));
    const uint32_t rows = __ballot_sync(kAllLanes, sees);
    if (lane == 0 && rows)
      asm volatile("red.shared.or.b32 [%0], %1;" :: "r"(lost + 4 * i), "r"(rows) : "memory");
  }
  __threadfence_block();
  __syncwarp();
}

// A CTA's walk over its run of steps, the same for each of its roles: all kv heads' steps
// one after the other, each head's units in their order.
struct Walk {
  int64_t v, v1;      // next step and end of the run
  int64_t total;      // a head's steps
  int64_t u;          // unit of v, or one before it
  int head;
  int steps;          // so far
};

// The steps [a, e) of a unit that fall to this CTA.
struct Segment {
  Unit x;
  int head;
  int a, e;
  int step0;      // the CTA's steps before it
  int64_t item0;  // the unit's first step of keys among all
};

__device__ __forceinline__ Walk start_walk(const PrefillArgs& w, int64_t v0, int64_t v1,
                                           int64_t total) {
  Walk k = {v0, v1, total, 0, int(v0 / total), 0};
  const int64_t at = v0 - k.head * total;
  k.u = find_last(w.max_units, at, [&](int64_t i) { return load_global(&w.units[i].start); });
  return k;
}

// The next segment, if any (false at the end of the run).
__device__ __forceinline__ bool next_segment(const PrefillArgs& w, Walk& k, Segment& s) {
  while (k.v < k.v1) {
    if (k.u >= w.max_units) {
      k.u = 0;
      ++k.head;
    }
    const int4* src = reinterpret_cast<const int4*>(w.units + k.u);
    int4* dst = reinterpret_cast<int4*>(&s.x);
#pragma unroll
    for (int i = 0; i < int(sizeof(Unit) / 16); ++i) dst[i] = load_global(src + i);
    const int steps = max(s.x.steps[0], s.x.steps[1]);
    s.item0 = k.head * k.total + s.x.start + kOpening;
    ++k.u;
    if (steps == 0 || s.item0 + steps <= k.v) continue;
    s.a = int(max(int64_t(0), k.v - s.item0));
    k.v = min(k.v1, s.item0 + steps);
    s.e = int(k.v - s.item0);
    s.head = k.head;
    s.step0 = k.steps;
    if (s.e <= s.a) continue;
    k.steps += s.e - s.a;
    return true;
  }
  return false;
}

// mbar_wait where the phase was not complete at first sight: kept out of line, as the roles'
// loops share the instruction caches.
__device__ __noinline__ bool wait_longer(uint32_t bar, uint32_t parity) {
  return mbar_wait(bar, parity);
}

template <int kDim>
__global__ void __launch_bounds__(kPrefillThreads, 1) dq4_kv8_prefill_kernel(const PrefillArgs w) {
  using S = PrefillSmem<kDim>;
  const AttendArgs& p = w.a;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint32_t s_tmem;
  __shared__ volatile int s_abort;
  __shared__ volatile int s_last[2];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(base);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t bar0 = sbase + S::kBars;
  auto k_full = [&](int s) { return bar0 + 8 * s; };
  static_assert(kSlots <= 4, "barriers 0 .. 15");
  auto k_empty = [&](int s) { return bar0 + 8 * (4 + s); };
  auto v_full = [&](int s) { return bar0 + 8 * (8 + s); };
  auto v_empty = [&](int s) { return bar0 + 8 * (12 + s); };
  // tile t: scores ready in buffer u, its weights written there, O summed up to that step; Q
  // there.  Steps alternate between the buffers' barriers, so that a wait never lags more
  // than one phase behind its barrier, which a parity could not tell.
  auto s_full = [&](int t, int u) { return bar0 + 8 * (16 + 2 * t + u); };
  auto p_full = [&](int t, int u) { return bar0 + 8 * (20 + 2 * t + u); };
  auto o_done = [&](int t, int u) { return bar0 + 8 * (24 + 2 * t + u); };
  auto q_full = [&](int t) { return bar0 + 8 * (28 + t); };
  auto all_done = [&](int i) { return bar0 + 8 * (30 + i); };
  // tile t, where a unit is shared: its part is written; whether it was the last part is known
  auto part_full = [&](int t) { return bar0 + 8 * (34 + t); };
  auto last_full = [&](int t) { return bar0 + 8 * (36 + t); };
  if (tid < 8) sts_v4(sbase + S::kNan + 16 * tid, 0, 0, uint32_t(-1), 0);
  if (tid < 2) sts_v4(sbase + S::kLost + 16 * tid, 0, 0, 0, 0);
  if (tid == 0) {
    s_abort = 0;
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(k_full(i), kLoadThreads);
      mbar_init(v_full(i), kLoadThreads);
      mbar_init(k_empty(i), 2);
      mbar_init(v_empty(i), 2);
    }
    for (int t = 0; t < 2; ++t) {
      for (int u = 0; u < 2; ++u) {
        mbar_init(s_full(t, u), 1);
        mbar_init(p_full(t, u), kTileRows);
        mbar_init(o_done(t, u), 1);
      }
      mbar_init(q_full(t), kTileRows);
      mbar_init(all_done(t), 1);
      mbar_init(all_done(2 + t), 1);
      mbar_init(part_full(t), kTileRows);
      mbar_init(last_full(t), 1);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kIssueWarp) {  // the whole TMEM: S and P of both tiles, then O of both
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;"
                 :: "r"(smem_u32(&s_tmem)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  wait_for_stream();
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tmem = s_tmem;
  auto t_s = [&](int t, int u) { return tmem + t * 128 + u * kKeys; };
  auto t_o = [&](int t) { return tmem + 256 + t * kDim; };

  // ---- this CTA's run of the steps
  const int64_t total = load_global(w.total), all = total * p.c.heads;
  const int64_t ctas = max(int64_t(1), min(int64_t(gridDim.x), all / kMinSteps));
  const int64_t v0 = min(int64_t(blockIdx.x), ctas) * all / ctas;
  const int64_t v1 = min(int64_t(blockIdx.x) + 1, ctas) * all / ctas;
  auto begin_of = [&](int64_t cta) { return cta * all / ctas; };
  auto cta_of = [&](int64_t v) { return int(((v + 1) * ctas - 1) / all); };

  auto fail = [&] {
    s_abort = 1;
    if (p.bad) atomicAdd(p.bad, 1);
  };
  auto wait = [&](uint32_t bar, int phase) {
    if (mbar_test(bar, uint32_t(phase) & 1u)) return true;
    if (s_abort) return false;
    if (wait_longer(bar, uint32_t(phase) & 1u)) return true;
    fail();
    return false;
  };
  // the same for a whole warp: true once every lane has seen the phase
  auto wait_warp = [&](uint32_t bar, int phase) {
    return bool(__all_sync(kAllLanes, wait(bar, phase)));
  };

  Segment sg;
  Walk walk = {};
  if (v0 < v1) walk = start_walk(w, v0, v1, total);

  if (warp < kLoadWarp) {
    // ------------------------------------------------------------------ softmax
    const int t = warp >> 2;
    const int row = tid & (kTileRows - 1);  // of the tile = its TMEM lane
    const uint32_t lanes = uint32_t((warp & 3) * 32) << 16;
    int step = 0;   // the tile's steps so far: buffers and their phases
    int joins = 0;  // and its shared units
    bool ok = true;
    // A unit as this thread's row sees it.
    struct Row {
      int64_t at;   // token and head, as of q and out
      int pos;
      bool real;
    };
    auto count_of = [&](const Segment& s) { return min(s.e, s.x.steps[t]) - s.a; };
    auto next_of_tile = [&](Segment& s) {
      while (next_segment(w, walk, s))
        if (count_of(s) > 0) return true;
      return false;
    };
    auto row_at = [&](const Segment& s, int64_t& src) {
      const int first = s.x.r0 + t * kTileRows;
      const int r = min(first + row, s.x.rows - 1);
      const int tok = r / p.group, q_head = s.head * p.group + r - tok * p.group;
      src = int64_t(s.x.row + tok) * p.token_stride + q_head * p.head_stride;
      return Row{int64_t(s.x.row + tok) * p.heads + q_head, s.x.pos + tok,
                 first + row < s.x.rows};
    };
    // The query row, scaled, to shared memory; its factor for the scores.  (The unit before
    // has no more use for its own: its last scores were waited for.)
    auto load_query = [&](int64_t src) {
      // a warp copies its rows, whole lines at a time, and each thread then takes its own
      constexpr int kPieces = kDim / 8;  // of 16 bytes
      auto piece_at = [&](int row, int i) {
        return sbase + S::kQ + t * S::kQTile + (i / 8) * S::kQBlock + row * 128 +
               (((i & 7) ^ (row & 7)) << 4);
      };
#pragma unroll 1
      for (int i = 0; i < kPieces; ++i) {
        const int r = i * (32 / kPieces) + lane / kPieces, piece = lane % kPieces;
        const uint16_t* from = static_cast<const uint16_t*>(p.q) +
                               __shfl_sync(kAllLanes, src, r) + piece * 8;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;"
                     :: "r"(piece_at((warp & 3) * 32 + r, piece)), "l"(from) : "memory");
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
      __syncwarp();
      uint4 raw[kPieces];
#pragma unroll
      for (int i = 0; i < kPieces; ++i) raw[i] = lds_v4(piece_at(row, i));
      const uint32_t* h = reinterpret_cast<const uint32_t*>(raw);
      float top = 0.f;
#pragma unroll
      for (int i = 0; i < kDim / 2; ++i) {
        float y, z;
        widen2(h[i], p.bf16, y, z);
        top = fmaxf(top, fmaxf(fabsf(y), fabsf(z)));
      }
      float up, down;
      row_scaling(top, up, down);
      if (p.scale_log2 < 0.f) up = -up;  // a negative scale turns the row instead
#pragma unroll
      for (int i = 0; i < kDim / 8; ++i) {
        uint32_t f[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float y, z;
          widen2(h[4 * i + j], p.bf16, y, z);
          f[j] = pack_f16(y * up, z * up);
        }
        sts_v4(piece_at(row, i), f[0], f[1], f[2], f[3]);
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      mbar_arrive(q_full(t));
      return down * fabsf(p.scale_log2);
    };
    bool have = next_of_tile(sg);
    int64_t src = 0;
    Row me = {};
    float cq = 0.f;
    if (have) {
      me = row_at(sg, src);
      cq = load_query(src);
    }
    while (have) {
      const Unit& x = sg.x;
      const int count = count_of(sg);
      const int pos = me.pos;
      const int lo = first_key(p, pos), hi = last_key(p, pos, x.held);
      const int all_lo = x.all_lo, all_hi = x.all_hi;
      RowSum sum;
      for (int j = 0; j < count; ++j, ++step) {
        const int u = step & 1;
        ok = wait_warp(s_full(t, u), step >> 1);  // and with the scores, the step's scales
        if (!ok) break;
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        const uint32_t gran = sbase + S::kGran + (sg.step0 + j) % kGranSlots * (kGrans * 16);
        const uint32_t scores = t_s(t, u) + lanes;
        const int key = x.key0 + (sg.a + j) * kKeys;
        const bool masked = mixed_step(all_lo, all_hi, key);
        uint32_t wt[kKeys / 2];
        float keep;
        const bool moved = masked ? softmax_pass<true>(scores, gran, cq, key, lo, hi, sum, keep, wt)
                                  : softmax_pass<false>(scores, gran, cq, key, lo, hi, sum, keep, wt);
        tmem_st<32>(scores, wt);
        if (moved && j > 0) {
          ok = wait_warp(o_done(t, u ^ 1), (step - 1) >> 1);
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
        asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
        asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
        mbar_arrive(p_full(t, u));
      }
      if (!ok) break;
      // ---- the next unit's query row goes first: its scores are computed while this unit's
      // result, or the part of it that this CTA has, is written
      const Segment was = sg;
      const Row mine = me;
      const int64_t at = mine.at;
      const bool real = mine.real;
      have = next_of_tile(sg);
      if (have) {
        me = row_at(sg, src);
        cq = load_query(src);
      }
      ok = wait_warp(o_done(t, (step - 1) & 1), (step - 1) >> 1);
      if (!ok) break;
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      const uint32_t lost_at = sbase + S::kLost + 16 * t + 4 * (warp & 3);
      const uint32_t lost = lds_b32(lost_at);
      if (lost != 0) {
        if (lost >> lane & 1) sum.l = __uint_as_float(kNaN);
        __syncwarp();
        if (lane == 0) sts_b32(lost_at, 0);
      }
      uint4* out = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + at * kDim);
      auto put = [&](int c, const float (&o)[8], float inv) {  // columns 8 c .. of the row
        uint32_t f[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) f[k] = pack_out(o[2 * k] * inv, o[2 * k + 1] * inv, p.bf16);
        if (real) out[c] = make_uint4(f[0], f[1], f[2], f[3]);
      };
      auto put_lse = [&](float ref, float l) {
        if (real && p.lse) p.lse[at] = log_sum(ref, l);
      };
      const bool whole = was.a == 0 && count == was.x.steps[t];
      const int64_t slot_at = 2 * blockIdx.x + (was.item0 - kOpening <= v0 ? 0 : 1);
      auto part_of = [&](int64_t s) { return w.part + (s * 2 + t) * (kDim / 4) * kTileRows + row; };
      auto stats_of = [&](int64_t s) { return w.stats + (s * 2 + t) * kTileRows + row; };
#pragma unroll 1
      for (int c = 0; c < kDim / 32; ++c) {
        uint32_t o[32];
        tmem_ld32(t_o(t) + lanes + 32 * c, o);
        if (whole) {
          const float inv = inverse_sum(sum.l);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float f[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) f[k] = __uint_as_float(o[8 * i + k]);
            put(4 * c + i, f, inv);
          }
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            part_of(slot_at)[(8 * c + i) * kTileRows] =
                make_float4(__uint_as_float(o[4 * i]), __uint_as_float(o[4 * i + 1]),
                            __uint_as_float(o[4 * i + 2]), __uint_as_float(o[4 * i + 3]));
        }
      }
      if (whole) {
        put_lse(sum.from, sum.l);
        continue;
      }
      *stats_of(slot_at) = make_float2(sum.fresh ? -INFINITY : sum.from, sum.l);
      const int c0 = cta_of(was.item0), c1 = cta_of(was.item0 + was.x.steps[t] - 1);
      // (barriers whose waits have a limit, as any other of a thread may have run out)
      mbar_arrive(part_full(t));
      if (row == 0 && wait(part_full(t), joins)) {
        int* counter = w.count + 2 * c1 + t;
        s_last[t] = atomic_add_acq_rel(counter, 1) == c1 - c0;
        if (s_last[t]) *counter = 0;  // ready for the next call
        mbar_arrive(last_full(t));
      }
      ok = wait_warp(last_full(t), joins++);
      if (!ok) break;
      if (!s_last[t]) continue;
      const int64_t slot0 = 2 * c0 + (was.item0 - kOpening <= begin_of(c0) ? 0 : 1);
      auto slot_of = [&](int c) { return c == c0 ? slot0 : int64_t(2 * c); };
      float top = -INFINITY, l = 0.f;
      for (int c = c0; c <= c1; ++c) top = fmaxf(top, load_l2(stats_of(slot_of(c))).x);
      const float ref = top == -INFINITY ? 0.f : top;
      for (int c = c0; c <= c1; ++c) {
        const float2 st = load_l2(stats_of(slot_of(c)));
        l = fmaf(exp2_fast(st.x - ref), st.y, l);
      }
      const float inv = inverse_sum(l);
#pragma unroll 1
      for (int i = 0; i < kDim / 32; ++i) {
        float4 acc[8] = {};
        for (int c = c0; c <= c1; ++c) {
          const float f = exp2_fast(load_l2(stats_of(slot_of(c))).x - ref);
          const float4* src = part_of(slot_of(c)) + 8 * i * kTileRows;
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const float4 y = load_l2(src + k * kTileRows);
            acc[k].x = fmaf(f, y.x, acc[k].x);
            acc[k].y = fmaf(f, y.y, acc[k].y);
            acc[k].z = fmaf(f, y.z, acc[k].z);
            acc[k].w = fmaf(f, y.w, acc[k].w);
          }
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float4 y = acc[2 * k], z = acc[2 * k + 1];
          const float f[8] = {y.x, y.y, y.z, y.w, z.x, z.y, z.z, z.w};
          put(4 * i + k, f, inv);
        }
      }
      put_lse(ref, l);
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
    const int page_bytes = p.c.page * kDim;
    bool met_bad = false;
    // Where the next step to read stands: its segment, and the step within the unit.
    bool more = next_segment(w, walk, sg);
    int j = more ? sg.a : 0;
    // Lane x holds granule x % kGrans of a step: its page's block (page * kv_heads + head), or
    // -1 where there are no such keys.
    struct Step {
      int key, held, block;  // first key
    };
    auto find_step = [&] {
      Step s = {0, 0, -1};
      if (!more) return s;
      s.key = sg.x.key0 + j * kKeys;
      s.held = sg.x.held;
      const int key = s.key + (lane & (kGrans - 1)) * 16;
      // (pages before the rows' windows are not looked at)
      if (key < s.held && key >= sg.x.first) {
        const int id =
            load_global(p.s.table + sg.x.b * p.s.table_stride + (key >> p.c.log2_page));
        if (id >= 0 && id < p.c.pages) {
          s.block = id * p.c.heads + sg.head;
        } else {
          met_bad = true;
        }
      }
      if (++j == sg.e) {
        more = next_segment(w, walk, sg);
        j = sg.a;
      }
      return s;
    };
    const int lt = tid - kUnitRows;
    int brought = 0, g = 0;  // steps asked for, and placed
    auto note_at = [&](int step) {
      return sbase + S::kNote + (step % kRawSlots * kGrans + (lane & (kGrans - 1))) * 16;
    };
    // Ask for a step's codes and scales; an empty group of copies past the last step.
    auto fetch = [&](bool valid, const Step& s) {
      if (valid) {
        const uint32_t dst = sbase + S::kRaw + brought % kRawSlots * (2 * kKeys * kDim) + lt * 16;
        // One page, all of it there: the usual case, and the shortest (668 -> 651 us for a prompt
        // of 8192).  Not for dim 64, where a step is two passes only and a second way through
        // the loop costs more, by the instruction caches, than it saves (353 -> 371 us for chunks
        // over 16k).
        const int only = kDim == 128 && p.c.page >= kKeys && s.key + kKeys <= s.held
                             ? __shfl_sync(kAllLanes, s.block, 0) : -1;
        if (only >= 0) {
          const int64_t off = int64_t(only) * page_bytes +
                              (((s.key & (p.c.page - 1)) + row0) * kDim + col * 16);
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const uint8_t* src = p.c.codes[x] + off;
#pragma unroll
            for (int i = 0; i < kPasses; ++i)
              asm volatile("cp.async.cg.shared.global [%0], [%1], 16;"
                           :: "r"(dst + (x * kPasses + i) * S::kRawPass),
                              "l"(src + i * kRowsPass * kDim) : "memory");
          }
        } else {
#pragma unroll (kDim == 64 ? kPasses : 1)
          for (int i = 0; i < kPasses; ++i) {
            const int row = row0 + i * kRowsPass, key = s.key + row;
            const int at = __shfl_sync(kAllLanes, s.block, row >> 4);
            // a slot never written may hold no number: zeros
            const int size = at >= 0 && key < s.held ? 16 : 0;
            const int64_t off =
                int64_t(at) * page_bytes + ((key & (p.c.page - 1)) * kDim + col * 16);
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const void* src = size ? static_cast<const void*>(p.c.codes[x] + off) : w.units;
              asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;"
                           :: "r"(dst + (x * kPasses + i) * S::kRawPass), "l"(src), "r"(size)
                           : "memory");
            }
          }
        }
        if (lw == 0 && lane < kGrans) {
          const uint32_t note = note_at(brought);
          asm volatile("st.shared.b32 [%0], %1;" :: "r"(note), "r"(s.block) : "memory");
          if (s.block >= 0) {
#pragma unroll
            for (int x = 0; x < 2; ++x)
              asm volatile("cp.async.ca.shared.global [%0], [%1], 4;"
                           :: "r"(note + 4 + 4 * x), "l"(p.c.scale[x] + s.block) : "memory");
          }
        }
        ++brought;
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    auto put = [&](uint32_t at, const uint4& v) {
      sts_v4(at + to[0], f16_of_e4m3(v.x), f16_of_e4m3_high(v.x), f16_of_e4m3(v.y),
             f16_of_e4m3_high(v.y));
      sts_v4(at + to[1], f16_of_e4m3(v.z), f16_of_e4m3_high(v.z), f16_of_e4m3(v.w),
             f16_of_e4m3_high(v.w));
    };
    for (int i = 0; i < kRawSlots; ++i) {
      const bool valid = more;
      fetch(valid, find_step());
    }
    bool have = more;
    Step s = find_step();
    for (; g < brought; ++g) {
      const int slot = g % kSlots, phase = g / kSlots;
      asm volatile("cp.async.wait_group %0;" :: "n"(kRawSlots - 1) : "memory");
      const uint32_t from = sbase + S::kRaw + g % kRawSlots * (2 * kKeys * kDim) + lt * 16;
      uint4 codes[2][kPasses];
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int i = 0; i < kPasses; ++i)
          codes[x][i] = lds_v4(from + (x * kPasses + i) * S::kRawPass);
      if (phase > 0 && !wait_warp(k_empty(slot), phase - 1)) break;
#pragma unroll
      for (int i = 0; i < kPasses; ++i)
        put(sbase + S::kK + slot * S::kOperand + i * kRowsPass * 128, codes[0][i]);
      if (lw == 0 && lane < kGrans) {
        // keys that are not there: S = 0 and an exponent of -infinity
        const uint4 note = lds_v4(note_at(g));
        const float vs = used_scale(__uint_as_float(note.z));
        const bool none = int(note.x) < 0;
        sts_v4(sbase + S::kGran + (g % kGranSlots * kGrans + lane) * 16, none ? 0 : note.y,
               __float_as_uint(none ? -INFINITY : __log2f(vs)),
               __float_as_uint(none ? 0.f : __fdividef(kSumUnit, vs)), 0);
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      mbar_arrive(k_full(slot));
      if (phase > 0 && !wait_warp(v_empty(slot), phase - 1)) break;
#pragma unroll
      for (int i = 0; i < kPasses; ++i)
        put(sbase + S::kV + slot * S::kOperand + i * kRowsPass * 128, codes[1][i]);
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      mbar_arrive(v_full(slot));
      fetch(have, s);
      have = more;
      s = find_step();
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (p.bad && __any_sync(kAllLanes, met_bad) && lane == 0) atomicAdd(p.bad, 1);
  } else {
    // -------------------------------------------------------------- the products
    // Warps kIssueWarp + t issue tile t's scores, kIssueWarp + 2 + t its P V.  The whole warp
    // runs this, one lane issues: the operands are then the same for all lanes, which a
    // branch on the lane would hide from the compiler.
    const int role = __shfl_sync(kAllLanes, warp - kIssueWarp, 0), t = role & 1;
    const uint32_t leads = lane == 0;
    // (a descriptor's address counts 16 bytes)
    const uint64_t q_desc = smem_desc(sbase + S::kQ + t * S::kQTile);
    const uint64_t k_desc = smem_desc(sbase + S::kK);
    const uint64_t v_desc = smem_desc_mn(sbase + S::kV, S::kBlock);
    const uint32_t idesc_s = instr_desc_f16<kTileRows, kKeys>(false);
    const uint32_t idesc_o = instr_desc_f16<kTileRows, kDim>(false) | (1u << 16);  // B: N contiguous
    // Every step's barriers are passed, also past the tile's last step, so that each slot's
    // phase ends with one arrival of each tile.
    auto nan_at = [&](int t, int g) { return sbase + S::kNan + (t * 4 + (g & 3)) * 16; };
    int g = 0, step = 0, units = 0;  // steps, this tile's steps, its units so far
    int last = -kGranSlots;          // this tile's last step, among all
    bool ok = true;
    while (ok && next_segment(w, walk, sg)) {
      const int count = sg.e - sg.a;
      const int n = max(0, min(sg.e, sg.x.steps[t]) - sg.a);  // of this tile
      const int key = sg.x.key0 + sg.a * kKeys;
      const int all_lo = sg.x.all_lo, all_hi = sg.x.all_hi;
      if (role < 2 && n > 0) ok = wait_warp(q_full(t), units++);
      for (int j = 0; j < count && ok; ++j, ++g) {
        const int slot = g % kSlots, phase = g / kSlots, u = step & 1;
        if (role < 2) {  // S = Q K^T, once the weights in its buffer have been used
          ok = wait_warp(k_full(slot), phase) &&
               (j < n ? step < 2 || wait_warp(o_done(t, u), (step >> 1) - 1)
                      : g - last != 3 || wait_warp(p_full(t, u ^ 1), (step - 1) >> 1));
          if (!ok) break;
          asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
          if (j < n) {
            const uint64_t k = k_desc + slot * (S::kOperand / 16);
#pragma unroll
            for (int i = 0; i < kDim / 16; ++i)
              mma_ss(t_s(t, u), q_desc + ((i / 4) * S::kQBlock + (i % 4) * 32) / 16,
                     k + ((i / 4) * S::kBlock + (i % 4) * 32) / 16, idesc_s, i > 0, leads);
            commit_if(s_full(t, u), leads);
            last = g;
          }
          commit_if(k_empty(slot), leads);
        } else {  // O += P V
          ok = wait_warp(v_full(slot), phase);
          if (!ok) break;
          uint64_t nan = 0;
          if (j < n && mixed_step(all_lo, all_hi, key + j * kKeys))
            nan = clean_values<kDim>(sbase + S::kV + slot * S::kOperand, nan_at(t, g), nan_at(1 - t, g),
                                     g);
          ok = j >= n || wait_warp(p_full(t, u), step >> 1);
          if (!ok) break;
          if (nan != 0) lose_rows(p, sg.x, t, key + j * kKeys, nan, sbase + S::kLost + 16 * t);
          asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
          if (j < n) {
            const uint64_t v = v_desc + slot * (S::kOperand / 16);
#pragma unroll
            for (int i = 0; i < kKeys / 16; ++i)
              mma_ts(t_o(t), t_s(t, u) + 8 * i, v + i * (2048 / 16), idesc_o, j > 0 || i > 0, leads);
            commit_if(o_done(t, u), leads);
          }
          commit_if(v_empty(slot), leads);
        }
        step += j < n;
      }
    }
    // every product issued is done before TMEM and shared memory go
    commit_if(all_done(role), leads);
    if (lane == 0) mbar_wait(all_done(role), 0);
  }
  __syncwarp();
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  if (warp == kIssueWarp) {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" :: "r"(tmem));
  }
}

static_assert(kMaxCtas * 2 * 4 <= kCounterBytes, "a counter for each CTA and tile");

int64_t max_units(int64_t tokens, int64_t seqs, int64_t group) {
  return tokens * group / kUnitRows + seqs;
}

int64_t plan_bytes(int64_t units) { return 64 + (units + 1) * int64_t(sizeof(Unit)); }

template <int kDim>
int launch_one(const PrefillArgs& w, int dev, int sms, cudaStream_t stream) {
  // more than half an SM's shared memory: one CTA per SM, as it takes all of TMEM
  constexpr int kBytes =
      PrefillSmem<kDim>::kBytes > 117 * 1024 ? PrefillSmem<kDim>::kBytes : 117 * 1024;
  auto kernel = dq4_kv8_prefill_kernel<kDim>;
  static std::atomic<uint64_t> allowed{0};
  if (const int st = allow_smem(kernel, kBytes, dev, &allowed)) return st;
  if (const int st = launch_ordered(dq4_kv8_plan_kernel, dim3(1), kPlanThreads, 0, stream, w))
    return st;
  return launch_ordered(kernel, dim3(unsigned(sms < kMaxCtas ? sms : kMaxCtas)), kPrefillThreads,
                        kBytes, stream, w);
}

}  // namespace

int64_t prefill_workspace_bytes(int64_t tokens, int64_t seqs, int64_t group, int head_dim) {
  return kCounterBytes + int64_t(kMaxCtas) * 4 * kTileRows * (8 + int64_t(head_dim) * 4) +
         plan_bytes(max_units(tokens, seqs, group)) + 256;
}

int launch_prefill(const AttendArgs& p, int head_dim, int dev, int sms, void* workspace,
                   cudaStream_t stream) {
  PrefillArgs w = {};
  w.a = p;
  w.max_units = max_units(p.s.tokens, p.s.seqs, p.group);
  char* at = static_cast<char*>(workspace);
  w.count = reinterpret_cast<int*>(at);
  at += kCounterBytes;
  w.stats = reinterpret_cast<float2*>(at);
  at += int64_t(kMaxCtas) * 4 * kTileRows * 8;
  w.part = reinterpret_cast<float4*>(at);
  at += int64_t(kMaxCtas) * 4 * kTileRows * head_dim * 4;
  w.total = reinterpret_cast<int64_t*>(at);
  w.units = reinterpret_cast<Unit*>(at + 64);
  return head_dim == 64 ? launch_one<64>(w, dev, sms, stream) : launch_one<128>(w, dev, sms, stream);
}

}  // namespace dq4d
