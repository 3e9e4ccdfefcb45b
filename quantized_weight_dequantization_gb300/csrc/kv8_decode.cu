// Attention over the 8-bit paged cache for few query rows a kv head (single tokens, grouped
// heads, a few proposed tokens): bound by the cache's bytes, each read once.
//
// The call's work is cut into units of 64 keys of one item (a sequence, a kv head and up to
// 8 NT query rows of it: new tokens x heads of the group).  One CTA runs per SM, on an equal
// run of the units whatever the lengths are, and each of its 8 warps on an eighth of that
// run (for few short items, a CTA on one item).  Items that fall to one warp alone are written
// by it; for the others each warp leaves FP32 parts (at most two: of its first and of its last
// item), which the CTA joins once, at its end, and the last CTA of an item joins across CTAs.
// Parts are always summed in the order of their keys, so results do not depend on timing.
//
// A warp has a ring of shared-memory slots of its own, each 64 keys or 64 values of one
// head, filled by TMA (swizzled); lane 0 issues, all lanes consume, and a slot is refilled as
// soon as it was read.  Nothing else synchronizes warps before the end.  Page ids and
// scales are read ahead, 8 units at a time, one granule of 16 keys per lane.
//
// For a unit, with tensor-core products of FP16 operands and FP32 sums (m16n8k16):
//   S^T (keys x rows)  = K (keys x dim) Q^T      codes of K as FP16, exact
//   P   = 2^(c S + log2 vs - m + kLift)          c: softmax scale, page scale and row scale
//   O^T (dim x rows)  += V^T (dim x keys) P^T
//   l  += P / vs   (in units of 2^16)
// The page's V scale vs enters the exponent, so that P V needs no scaled V and the weights
// keep their precision whatever the scales are; l takes it out again.  Keys on the M side
// leave the N side of 8 to the few query rows.  The order of dim inside K Q^T, and of dim
// inside O^T, is free: a lane takes 16 or 32 consecutive bytes of a key for the first product
// and dim / 8 of a value for the second, so shared memory is read in 16-byte words.
//
// Measured (kv heads of 128): 64 sequences of 100 .. 8192 keys, 4 rows a head, 101 us (541 MB,
// 5.3 TB/s; the loop itself runs at 7, the rest is the start, the joins and SMs that end 20 us
// apart on equal work); 2 sequences of up to 131071 keys, 8 rows, 86 to 87 us (465 MB, 5.4 TB/s).
// Short calls are a chain of latencies: one sequence of 777 keys takes 12 us, 2 of them to find
// the work, 2 to the first keys, 4 in the loop and the rest in the joins and the launch.
#include "kv8_attend.cuh"

namespace dq4d {
namespace {

constexpr int kWarps = 8;
constexpr int kDecodeThreads = 32 * kWarps;
constexpr int kTile = 64;          // keys of a unit
constexpr int kGrans = kTile / 16; // granules of 16 keys, never of two pages
constexpr int kMaxCtas = 160;      // CTAs the workspace has room for
constexpr int kMaxRows = 16;       // query rows of an item: 8 NT
constexpr int kOpening = 1;        // what starting and ending an item costs, in units
constexpr int kItemUnits = 18;     // units of an item that a CTA takes alone (see `each`)
constexpr int kSegs = 8;           // items, or parts of them, that a warp plans at a time
constexpr int kBatch = 32 / kGrans;  // units whose pages are read ahead together
// parts: two for each warp, and two for each CTA
constexpr int kParts = kMaxCtas * (2 * kWarps + 2);

// An item, or the part of it that falls to a warp.
struct Segment {
  int64_t item0;  // where the item's first unit of keys stands among all units
  int first;      // this part's first unit, counted over the warp's
  int count;      // its units
  int tiles;      // units of the whole item
  int tile0;      // this part's first unit within the item
  int b, head;    // sequence and kv head
  int r0, rows;   // first query row of the item, and the sequence's rows
  int key0;       // the item's first key, a multiple of kTile
  int held, len, n, row;
  bool in_ring;   // a part: kept in the warp's ring, not in the workspace
};

template <int kDim>
struct DecodeSmem {
  static constexpr int kSlot = kTile * kDim;
  static constexpr int kSlots = kDim == 128 ? 3 : 6;  // 24 KB a warp
  static constexpr int kSegAt = kWarps * kSlots * kSlot;
  static constexpr int kPartAt = kSegAt + kWarps * kSegs * int(sizeof(Segment));
  static constexpr int kBars = kPartAt + kWarps * 2 * int(sizeof(Segment));
  static constexpr int kBytes = kBars + kWarps * kSlots * 8 + 1024;  // + alignment slack
  static_assert(kBytes + 256 <= 227 * 1024, "shared memory budget");
};

struct SeqWork {
  int tiles, items, key0, held;
};

// The units of a sequence: its kv heads times its row tiles, times the units of keys
// that its rows see (one at least, so that rows which see none get their zeros).  In the
// division of the work an item counts kOpening units more, placed before its keys: starting
// and ending an item takes a warp about as long as a unit does.
__device__ __forceinline__ SeqWork seq_work(const AttendArgs& p, const Seq& s, int rows_tile) {
  SeqWork w;
  w.held = held_keys(p, s.len);
  const int begin = first_key(p, s.len - s.n) & ~(kTile - 1);
  w.key0 = min(begin, w.held & ~(kTile - 1));
  w.tiles = max(1, (w.held - w.key0 + kTile - 1) / kTile);
  w.items = (s.n * p.group + rows_tile - 1) / rows_tile * p.c.heads;
  return w;
}

// a / b for 0 <= a, 0 < b: nearly always in 32 bits.
__device__ __forceinline__ int64_t divide(int64_t a, int64_t b) {
  if (((a | b) >> 32) == 0) return int64_t(uint32_t(a) / uint32_t(b));
  return a / b;
}

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                        uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The 8 x 8 matrix of 16-bit values whose row lane / 4 this lane holds two of, transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

__device__ __forceinline__ void tma_load_3d(uint32_t dst, uint64_t map, int y, int z,
                                            uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];"
      :: "r"(dst), "l"(map), "r"(0), "r"(y), "r"(z), "r"(bar) : "memory");
}

// The sum of v over the block and the sum before this thread, in thread order.
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t* s_sums, int64_t& before) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int64_t run = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t up = __shfl_up_sync(kAllLanes, run, o);
    if (lane >= o) run += up;
  }
  __syncthreads();
  if (lane == 31) s_sums[warp] = run;
  __syncthreads();
  int64_t total = 0;
  before = run - v;
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += s_sums[w];
    total += s_sums[w];
  }
  return total;
}

// A part's rows of O, unnormalized, and their {m, l}: in global or shared memory.
struct PartAt {
  const float* o;
  const float2* stats;
};

// Rows r and, if two, r2 of the n parts at(0) .. at(n - 1): columns kCols lane .. of O and m
// and l, summed in that order.  Two rows at a time keep twice the loads on the way.
template <int kCols, typename At>
__device__ __forceinline__ void join_parts(int n, int r, int r2, At at, float (&v)[2][kCols],
                                           float (&top)[2], float (&sum)[2]) {
  const int lane = threadIdx.x & 31;
  const int row[2] = {r, r2};
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    top[x] = -INFINITY;
    sum[x] = 0.f;
#pragma unroll
    for (int i = 0; i < kCols; ++i) v[x][i] = 0.f;
  }
  for (int i0 = 0; i0 < n; i0 += 32) {  // 32 parts at a time, one's m and l per lane
    float2 st[2];
    float mine[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      st[x] = make_float2(-INFINITY, 0.f);
      if (i0 + lane < n) st[x] = at(i0 + lane).stats[row[x]];
    }
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      float t = st[x].x;
#pragma unroll
      for (int w = 16; w > 0; w >>= 1) t = fmaxf(t, __shfl_xor_sync(kAllLanes, t, w));
      const float is = fmaxf(top[x], t), from = is == -INFINITY ? 0.f : is;
      const float keep = exp2_fast(top[x] - from);
      mine[x] = exp2_fast(st[x].x - from);
      sum[x] *= keep;
#pragma unroll
      for (int i = 0; i < kCols; ++i) v[x][i] *= keep;
      top[x] = is;
    }
    const int k1 = min(32, n - i0);
#pragma unroll 4
    for (int k = 0; k < k1; ++k) {
      const float* o = at(i0 + k).o + lane * kCols;
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        float u[kCols];
        if constexpr (kCols == 4) {
          const float4 y = *reinterpret_cast<const float4*>(o + row[x] * (32 * kCols));
          u[0] = y.x;
          u[1] = y.y;
          u[2] = y.z;
          u[3] = y.w;
        } else {
          const float2 y = *reinterpret_cast<const float2*>(o + row[x] * (32 * kCols));
          u[0] = y.x;
          u[1] = y.y;
        }
        const float f = __shfl_sync(kAllLanes, mine[x], k);
        sum[x] = fmaf(f, __shfl_sync(kAllLanes, st[x].y, k), sum[x]);
#pragma unroll
        for (int i = 0; i < kCols; ++i) v[x][i] = fmaf(f, u[i], v[x][i]);
      }
    }
  }
}

// A joined row to the output: this lane's columns of row r of segment s.
template <int kCols>
__device__ __forceinline__ void write_row(const AttendArgs& p, const Segment& s, int r,
                                          const float (&v)[kCols], float top, float sum) {
  const int lane = threadIdx.x & 31;
  const int tok = (s.r0 + r) / p.group;
  const int64_t at = int64_t(s.row + tok) * p.heads + s.head * p.group + s.r0 + r - tok * p.group;
  const float inv = inverse_sum(sum);
  uint32_t* out = static_cast<uint32_t*>(p.out) + (at * 32 + lane) * (kCols / 2);
#pragma unroll
  for (int i = 0; i < kCols / 2; ++i)
    out[i] = pack_out(v[2 * i] * inv, v[2 * i + 1] * inv, p.bf16);
  if (p.lse && lane == 0)
    p.lse[at] = log_sum(top - kLift, sum);
}

template <int kDim, int NT>
__global__ void __launch_bounds__(kDecodeThreads, 1)
    dq4_kv8_decode_kernel(const __grid_constant__ CUtensorMap map_k,
                          const __grid_constant__ CUtensorMap map_v, const AttendArgs p) {
  using S = DecodeSmem<kDim>;
  constexpr int kSlots = S::kSlots;
  constexpr int kRows = 8 * NT;         // query rows of an item
  constexpr int kSteps = kDim / 16;     // products along dim, and tiles of dim in O^T
  constexpr int kWordsK = kDim / 16;    // 4-byte words of a key a lane holds
  constexpr int kWordsV = kDim / 32;    // and of a value
  constexpr int kCols = kDim / 32;      // columns a lane takes where parts are joined
  extern __shared__ uint8_t smem_raw[];
  __shared__ int64_t s_sums[kWarps], s_before, s_run[2];
  __shared__ int s_b0;
  __shared__ bool s_last[2];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(base);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, c = lane & 3;
  const uint32_t ring = sbase + warp * kSlots * S::kSlot;
  const uint32_t bars = sbase + S::kBars + warp * kSlots * 8;
  Segment* seg_of = reinterpret_cast<Segment*>(base + S::kSegAt) + warp * kSegs;
  Segment* parts = reinterpret_cast<Segment*>(base + S::kPartAt);
  const uint64_t tk = reinterpret_cast<uint64_t>(&map_k), tv = reinterpret_cast<uint64_t>(&map_v);
  if (lane == 0) {
    for (int i = 0; i < kSlots; ++i) mbar_init(bars + 8 * i, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("prefetch.tensormap [%0];" :: "l"(tk));
    asm volatile("prefetch.tensormap [%0];" :: "l"(tv));
  }
  if (lane < 2) parts[2 * warp + lane].rows = 0;  // none yet
  wait_for_stream();

  // ---- the call's units, and the sequence where this CTA's run of them starts
  const int64_t seqs = p.s.seqs;
  auto units_of = [&](int64_t b) -> int64_t {
    if (b >= seqs) return 0;
    const SeqWork w = seq_work(p, seq_at(p.s, b), kRows);
    return int64_t(w.tiles + kOpening) * w.items;
  };
  int64_t units = 0, before = 0;
  const int64_t mine = units_of(tid);
  for (int64_t b = tid; b - tid < seqs; b += kDecodeThreads)
    units += block_scan(b == tid ? mine : units_of(b), s_sums, before);
  if (units == 0) return;
  // With no more items than CTAs, a CTA takes one item each, if none is longer than an equal
  // share of the units by more than kItemUnits: a unit takes a CTA 0.26 us, and a join of
  // several CTAs' parts about 5 us.  Equal shares / an item each, in us, 8 kv heads of 128:
  //   keys of a sequence   256         1024        1536        2048        3000
  //    1 sequence          12.6 / 9.8  14.4 / 13.8 15.5 / 16.0 15.6 / 18.2 15.6 / 21.3
  //    8                   13.5 / 9.7  14.7 / 14.3 16.8 / 16.5 17.3 / 18.7 19.9 / 21.6
  //   18                   14.3 / 9.9  18.4 / 14.6 19.6 / 16.8 21.5 / 19.0 28.0 / 24.1
  if (seqs <= kDecodeThreads) {
    SeqWork w = {};
    if (tid < seqs) w = seq_work(p, seq_at(p.s, tid), kRows);
    int64_t first;
    const int64_t items = block_scan(w.items, s_sums, first);
    const bool each = items <= gridDim.x;
    const bool longer = w.items > 0 && int64_t(w.tiles - kItemUnits) * gridDim.x > units;
    if (!__syncthreads_or(longer) && each) {
      if (blockIdx.x >= items) return;
      if (first <= blockIdx.x && blockIdx.x < first + w.items) {
        s_b0 = tid;
        s_before = before;
        s_run[0] = before + (blockIdx.x - first) * (w.tiles + kOpening);
        s_run[1] = s_run[0] + w.tiles + kOpening;
      }
    } else if (tid == 0) {
      s_run[1] = -1;
    }
  } else if (tid == 0) {
    s_run[1] = -1;
  }
  __syncthreads();
  const int64_t ctas = min(int64_t(gridDim.x), units);
  auto begin_of = [&](int64_t cta) { return divide(cta * units, ctas); };
  auto cta_of = [&](int64_t u) { return int(divide((u + 1) * ctas - 1, units)); };
  int64_t u0 = s_run[0], u1 = s_run[1];
  if (u1 < 0) {
    if (blockIdx.x >= ctas) return;
    u0 = begin_of(blockIdx.x);
    u1 = begin_of(blockIdx.x + 1);
    int64_t passed = 0;
    for (int64_t b = tid; b - tid < seqs; b += kDecodeThreads) {
      const int64_t v = b == tid ? mine : units_of(b);
      int64_t total = units;
      if (seqs > kDecodeThreads) total = block_scan(v, s_sums, before);
      const int64_t at = passed + before;
      if (at <= u0 && u0 < at + v) {
        s_b0 = int(b);
        s_before = at;
      }
      passed += total;
      if (passed > u0) break;  // the same for every thread
    }
    __syncthreads();
  }
  const int64_t v0 = u0 + (u1 - u0) * warp / kWarps, v1 = u0 + (u1 - u0) * (warp + 1) / kWarps;

  // ---- state of the segment a warp is in
  float o[NT][kSteps][4];
  float m[NT][2], l[NT][2], cq[NT][2];
  uint32_t qf[NT][kSteps][2];
  bool failed = false;
  int issued = 0, taken = 0;  // slots of the ring filled and consumed
  int met_bad = 0;

  // where parts are kept: warp w's two in the workspace, its last in its ring
  auto own_part = [&](int part) {
    return p.part + (int64_t(blockIdx.x) * (2 * kWarps) + part) * (kMaxRows * kDim);
  };
  auto own_stats = [&](int part) {
    return p.stats + (int64_t(blockIdx.x) * (2 * kWarps) + part) * kMaxRows;
  };
  auto ring_of = [&](int w) { return reinterpret_cast<float*>(base + w * kSlots * S::kSlot); };
  static_assert(kRows * (kDim * 4 + 8) <= kSlots * S::kSlot, "a part fits the ring");
  float* ring_part = ring_of(warp);
  float2* ring_stats = reinterpret_cast<float2*>(ring_part + kRows * kDim);

  // Rows 2 c + j of O^T (columns g kDim / 8 .. of dim): the result, or a part of it.
  // Parts go to the workspace, but for the warp's last, when its ring is free.
  auto flush = [&](const Segment& s, bool ring_free) {
    const bool whole = s.count == s.tiles;
    const int part = 2 * warp + (s.first > 0);  // of the warp's first item, or its last
    if (!whole && lane == 0) {
      parts[part] = s;
      parts[part].in_ring = ring_free;
    }
    float* part_o = ring_free ? ring_part : own_part(part);
    float2* part_stats = ring_free ? ring_stats : own_stats(part);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float sum = l[nt][j];
#pragma unroll
        for (int w = 4; w < 32; w <<= 1) sum += __shfl_xor_sync(kAllLanes, sum, w);
        const int r = nt * 8 + 2 * c + j;
        if (r >= s.rows - s.r0) continue;
        if (whole) {
          const int tok = (s.r0 + r) / p.group;
          const int64_t at =
              int64_t(s.row + tok) * p.heads + s.head * p.group + s.r0 + r - tok * p.group;
          const float inv = inverse_sum(sum);
          uint4* out = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + at * kDim +
                                                g * (kDim / 8));
#pragma unroll
          for (int i = 0; i < kSteps; i += 4)
            out[i / 4] = make_uint4(pack_out(o[nt][i][j] * inv, o[nt][i][2 + j] * inv, p.bf16),
                                    pack_out(o[nt][i + 1][j] * inv, o[nt][i + 1][2 + j] * inv, p.bf16),
                                    pack_out(o[nt][i + 2][j] * inv, o[nt][i + 2][2 + j] * inv, p.bf16),
                                    pack_out(o[nt][i + 3][j] * inv, o[nt][i + 3][2 + j] * inv, p.bf16));
          if (p.lse && g == 0)
            p.lse[at] = log_sum(m[nt][j] - kLift, sum);
        } else {
          float4* to = reinterpret_cast<float4*>(part_o + r * kDim + g * (kDim / 8));
#pragma unroll
          for (int i = 0; i < kSteps; i += 2)
            to[i / 2] = make_float4(o[nt][i][j], o[nt][i][2 + j], o[nt][i + 1][j],
                                    o[nt][i + 1][2 + j]);
          if (g == 0) part_stats[r] = make_float2(m[nt][j], sum);
        }
      }
  };

  // A new segment: its query rows as FP16 fragments, empty sums.
  auto open = [&](const Segment& s) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int r = s.r0 + nt * 8 + g;
      uint4 raw[kWordsK / 2];
#pragma unroll
      for (int i = 0; i < kWordsK / 2; ++i) raw[i] = make_uint4(0, 0, 0, 0);
      if (r < s.rows) {
        const int tok = r / p.group;
        const uint16_t* q = static_cast<const uint16_t*>(p.q) + (s.row + tok) * p.token_stride +
                            (s.head * p.group + r - tok * p.group) * p.head_stride +
                            c * (kDim / 4);
#pragma unroll
        for (int i = 0; i < kWordsK / 2; ++i)
          raw[i] = load_global(reinterpret_cast<const uint4*>(q) + i);
      }
      const uint32_t* w = reinterpret_cast<const uint32_t*>(raw);
      float top = 0.f;
#pragma unroll
      for (int i = 0; i < 2 * kWordsK; ++i) {
        float x, y;
        widen2(w[i], p.bf16, x, y);
        top = fmaxf(top, fmaxf(fabsf(x), fabsf(y)));
      }
      top = fmaxf(top, __shfl_xor_sync(kAllLanes, top, 1));
      top = fmaxf(top, __shfl_xor_sync(kAllLanes, top, 2));
      float up, down;
      row_scaling(top, up, down);
#pragma unroll
      for (int i = 0; i < 2 * kWordsK; ++i) {
        float x, y;
        widen2(w[i], p.bf16, x, y);
        qf[nt][i / 2][i & 1] = pack_f16(x * up, y * up);
      }
      // the factors of the two rows whose scores this lane gets
      cq[nt][0] = __shfl_sync(kAllLanes, down, 8 * c) * p.scale_log2;
      cq[nt][1] = __shfl_sync(kAllLanes, down, 8 * c + 4) * p.scale_log2;
      m[nt][0] = m[nt][1] = -INFINITY;
      l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
      for (int i = 0; i < kSteps; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[nt][i][j] = 0.f;
    }
  };

  // Plan up to kSegs segments from unit u on; plan_b, plan_first: a sequence at or before
  // it, and that one's first unit.  32 sequences at a time, one per lane.
  int plan_b = s_b0, nseg = 0, planned = 0;
  int64_t plan_first = s_before, plan_u = v0;
  auto plan = [&] {
    int from = -1;
    Seq s = {};
    SeqWork w = {};
    nseg = 0;
    while (plan_u < v1 && nseg < kSegs) {
      if (from < 0 || plan_b >= from + 32) {
        from = plan_b;
        w = SeqWork{1, 0, 0, 0};
        if (plan_b + lane < seqs) {
          s = seq_at(p.s, plan_b + lane);
          w = seq_work(p, s, kRows);
        }
      }
      const int src = plan_b - from;
      const int tiles = __shfl_sync(kAllLanes, w.tiles, src);
      const int items = __shfl_sync(kAllLanes, w.items, src);
      const int cost = tiles + kOpening;
      const int64_t all = int64_t(cost) * items;
      if (plan_u >= plan_first + all) {
        plan_first += all;
        ++plan_b;
        continue;
      }
      const int64_t in = plan_u - plan_first;
      const int item = int(divide(in, cost));
      const int64_t item0 = plan_first + int64_t(item) * cost + kOpening;
      const int tile = int(max(int64_t(0), plan_u - item0));
      plan_u = min(v1, item0 + tiles);
      const int count = int(plan_u - item0) - tile;
      if (count <= 0) continue;  // its keys fall to the next warp
      const int per_head = items / p.c.heads;
      const int r0 = item % per_head * kRows;
      if (lane == src)
        seg_of[nseg] = Segment{item0,  planned,         count,  tiles, tile,  plan_b, item / per_head,
                               r0,     s.n * p.group,   w.key0, w.held, s.len, s.n,    int(s.row),
                               false};
      planned += count;
      // its query rows, to L2 before they are needed: a lane for each line of 128 bytes
      constexpr int kLines = kDim / 64;
      const int r = r0 + lane / kLines;
      const int n = __shfl_sync(kAllLanes, s.n, src);
      const int row = __shfl_sync(kAllLanes, int(s.row), src);
      if (lane / kLines < kRows && r < n * p.group) {
        const int tok = r / p.group;
        const uint16_t* q = static_cast<const uint16_t*>(p.q) + (row + tok) * p.token_stride +
                            (item / per_head * p.group + r - tok * p.group) * p.head_stride;
        asm volatile("prefetch.global.L2 [%0];" :: "l"(q + lane % kLines * 64));
      }
      ++nseg;
    }
    __syncwarp();
  };

  // Pages read ahead: lane kGrans t + h holds granule h of unit kBatch batch + t of the plan.
  // Three batches are on the way, so that no load is used in the batch that issues it: the
  // page ids of batch + 2, the scales of batch + 1, and the batch that is being used.
  struct Ahead {
    int seg, key, id, head;  // id: the page, or -1 where there are no such keys, or none sees them
    int block;               // page * kv_heads + head, or -1
    float ks, vs;            // scales
  };
  int unit0 = 0, unit1 = 0;  // the plan's units, counted over the warp's
  const int rows_copy = min(p.c.page, kTile);
  auto read_pages = [&](int batch) {
    Ahead a = {0, 0, -1, 0, -1, 0.f, 1.f};
    const int i = unit0 + batch * kBatch + lane / kGrans;
    if (i >= unit1) return a;
    int sg = 0;
    while (sg + 1 < nseg && seg_of[sg + 1].first <= i) ++sg;
    const Segment& s = seg_of[sg];
    a.seg = sg;
    a.head = s.head;
    a.key = s.key0 + (s.tile0 + i - s.first) * kTile + (lane % kGrans) * 16;
    // (copies take rows_copy keys; one of which no row of the sequence sees any is left out)
    if (a.key < s.held && (a.key | (rows_copy - 1)) >= first_key(p, s.len - s.n)) {
      a.id = load_global(p.s.table + s.b * p.s.table_stride + (a.key >> p.c.log2_page));
      a.block = 0;
    }
    if (s.held < s.len) met_bad = 1;
    return a;
  };
  auto read_scales = [&](Ahead& a) {
    if (a.block < 0) return;
    if (a.id >= 0 && a.id < p.c.pages) {
      a.block = a.id * p.c.heads + a.head;
      a.ks = load_global(p.c.scale[0] + a.block);
      a.vs = load_global(p.c.scale[1] + a.block);
    } else {
      a.block = -1;
      met_bad = 1;
    }
  };
  Ahead now = {}, next = {}, later = {};
  float now_bias = 0.f, now_inv = 0.f;  // log2 and inverse (in kSumUnit) of now.vs
  auto use = [&](const Ahead& a) {
    now = a;
    const float vs = used_scale(a.vs);
    now_bias = log2f(vs);
    now_inv = kSumUnit / vs;
  };
  // The next slot of the ring: the keys (which = 0) or values of unit k of the plan, which
  // is in the batch `now` or the one after it.
  auto issue = [&](int k, int batch, int which) {
    const bool in_now = k / kBatch == batch;
    const int t = (k % kBatch) * kGrans;
    const int key = __shfl_sync(kAllLanes, in_now ? now.key : next.key, t);
    const int block = in_now ? now.block : next.block;
    int b[kGrans];
#pragma unroll
    for (int h = 0; h < kGrans; ++h) b[h] = __shfl_sync(kAllLanes, block, t + h);
    const int slot = issued % kSlots;
    ++issued;
    if (lane == 0) {
      const uint32_t dst = ring + slot * S::kSlot, bar = bars + 8 * slot;
      const uint64_t map = which ? tv : tk;
      if (rows_copy == kTile) {
        mbar_expect(bar, b[0] >= 0 ? uint32_t(kTile * kDim) : 0);
        if (b[0] >= 0) tma_load_3d(dst, map, key & (p.c.page - 1), b[0], bar);
      } else {
        const int grans = rows_copy / 16;  // granules of a copy: 1 or 2
        int copies = 0;
#pragma unroll
        for (int h = 0; h < kGrans; ++h) copies += h % grans == 0 && b[h] >= 0;
        mbar_expect(bar, uint32_t(copies * rows_copy * kDim));
#pragma unroll
        for (int h = 0; h < kGrans; ++h)
          if (h % grans == 0 && b[h] >= 0) tma_load_3d(dst + h * 16 * kDim, map, 0, b[h], bar);
      }
    }
  };
  auto arrive = [&] {  // the next slot of the ring, once its copies are in
    const int slot = taken % kSlots;
    // (for the warp as a whole: what follows a wait that ran out is collective)
    failed = !__all_sync(kAllLanes, !failed && mbar_wait(bars + 8 * slot, uint32_t(taken / kSlots) & 1u));
    ++taken;
    return ring + slot * S::kSlot;
  };

  while (plan_u < v1 && !failed) {
    unit0 = planned;
    plan();
    unit1 = planned;
    const int count = unit1 - unit0;
    if (count == 0) break;
    now = read_pages(0);
    next = read_pages(1);
    later = read_pages(2);
    read_scales(now);
    read_scales(next);
    for (int k = 0; k < kSlots; ++k)
      if (k < 2 * count) issue(k / 2, 0, k & 1);
    use(now);
    int seg = -1, all_lo = 0, all_hi = 0;
    for (int k = 0; k < count; ++k) {
      const int batch = k / kBatch, t = (k % kBatch) * kGrans;
      if (k > 0 && k % kBatch == 0) {
        use(next);
        next = later;
        read_scales(next);
        later = read_pages(batch + 2);
      }
      const int sg = __shfl_sync(kAllLanes, now.seg, t);
      if (sg != seg) {
        if (seg >= 0) flush(seg_of[seg], false);
        seg = sg;
        const Segment& s = seg_of[seg];
        open(s);
        // the keys that every row sees
        all_lo = first_key(p, s.len - s.n + min(s.rows - 1, s.r0 + kRows - 1) / p.group);
        all_hi = last_key(p, s.len - s.n + s.r0 / p.group, s.held);
      }
      const int key = __shfl_sync(kAllLanes, now.key, t);
      float ks[kGrans], bias[kGrans], inv[kGrans];
      bool there[kGrans];
      bool all = key >= all_lo && key + kTile <= all_hi;
#pragma unroll
      for (int h = 0; h < kGrans; ++h) {
        ks[h] = __shfl_sync(kAllLanes, now.ks, t + h);
        bias[h] = __shfl_sync(kAllLanes, now_bias, t + h);
        inv[h] = __shfl_sync(kAllLanes, now_inv, t + h);
        there[h] = __shfl_sync(kAllLanes, now.block, t + h) >= 0;
        all = all && there[h];
      }

      // ---- S^T: keys 16 h + g and + 8, rows 8 nt + 2 c and + 1
      const uint32_t keys = arrive();
      float st[kGrans][NT][4];
#pragma unroll
      for (int h = 0; h < kGrans; ++h) {
        uint4 raw[2][kWordsK / 4];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int row = 16 * h + 8 * j + g;
          const uint32_t at = keys + row * kDim;
#pragma unroll
          for (int i = 0; i < kWordsK / 4; ++i)
            raw[j][i] = kDim == 128 ? lds_v4(at + (((2 * c + i) ^ (row & 7)) << 4))
                                    : lds_v4(at + ((c ^ ((row >> 1) & 3)) << 4));
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int j = 0; j < 4; ++j) st[h][nt][j] = 0.f;
        const uint32_t* w0 = reinterpret_cast<const uint32_t*>(raw[0]);
        const uint32_t* w1 = reinterpret_cast<const uint32_t*>(raw[1]);
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
          const uint32_t a[4] = {f16_of_e4m3(w0[i]), f16_of_e4m3(w1[i]), f16_of_e4m3_high(w0[i]),
                                 f16_of_e4m3_high(w1[i])};
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma_f16(st[h][nt], a, qf[nt][i][0], qf[nt][i][1]);
        }
      }
      __syncwarp();  // every lane has read the keys
      // slot 2 k + kSlots of the plan's 2 count: unit k + kSlots / 2
      if (2 * k + kSlots < 2 * count && !failed)
        issue((2 * k + kSlots) / 2, batch, kSlots & 1);

      // ---- the softmax's weights, in base 2; the lanes of equal c share their rows
      uint32_t pf[kGrans][NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float x[2 * kGrans];
          float top = -INFINITY;
#pragma unroll
          for (int i = 0; i < 2 * kGrans; ++i)  // key 8 i + g
            x[i] = fmaf(st[i >> 1][nt][2 * (i & 1) + j], cq[nt][j] * ks[i >> 1], bias[i >> 1]);
          if (!all) {
            const Segment& s = seg_of[seg];
            const int r = min(s.rows - 1, s.r0 + nt * 8 + 2 * c + j);
            const int pos = s.len - s.n + r / p.group;
            const int lo = first_key(p, pos), hi = last_key(p, pos, s.held);
#pragma unroll
            for (int i = 0; i < 2 * kGrans; ++i) {
              const int at = key + 8 * i + g;
              if (at < lo || at >= hi || !there[i >> 1]) x[i] = -INFINITY;
            }
          }
#pragma unroll
          for (int i = 0; i < 2 * kGrans; ++i) top = fmaxf(top, x[i]);
#pragma unroll
          for (int w = 4; w < 32; w <<= 1) top = fmaxf(top, __shfl_xor_sync(kAllLanes, top, w));
          const float was = m[nt][j], is = fmaxf(was, top);
          const float from = is == -INFINITY ? 0.f : is - kLift;
          m[nt][j] = is;
          if (__any_sync(kAllLanes, is != was)) {
            const float keep = exp2_fast(was - (is == -INFINITY ? 0.f : is));
            l[nt][j] *= keep;
#pragma unroll
            for (int i = 0; i < kSteps; ++i) {
              o[nt][i][j] *= keep;
              o[nt][i][2 + j] *= keep;
            }
          }
#pragma unroll
          for (int h = 0; h < kGrans; ++h) {
            const float a = exp2_fast(x[2 * h] - from), b = exp2_fast(x[2 * h + 1] - from);
            st[h][nt][j] = a;
            st[h][nt][2 + j] = b;
            // an unseen granule's scale may be no number
            if (all || a + b != 0.f) l[nt][j] = fmaf(a + b, inv[h], l[nt][j]);
          }
        }
#pragma unroll
        for (int h = 0; h < kGrans; ++h) {
          pf[h][nt][0] = transpose8(pack_f16(st[h][nt][0], st[h][nt][1]));
          pf[h][nt][1] = transpose8(pack_f16(st[h][nt][2], st[h][nt][3]));
        }
      }

      // ---- O^T += V^T P^T: keys 2 c, 2 c + 1, + 8 and + 9 of each 16, dims g kDim / 8 ..
      const uint32_t values = arrive();
      // A weight of 0 does not keep a value that is no number from its row.  So where some row
      // does not see a key, such codes become zeros, and l brings them to the rows that do.
      // (24 sequences x 5 tokens under a window: 22.3 -> 23.2 us.  Looked for on the way into the
      // product instead, 22.3, but 8 x 128 tokens over 10000 keys take 1302 us for 1223.)
      if (!all && (key < all_lo || min(key + kTile, seg_of[seg].held) > all_hi)) {
        auto piece = [&](int row, int i) {
          return values + row * kDim + (i ^ (lane & (kDim / 16 - 1))) * 16;
        };
        uint32_t any = 0;
#pragma unroll
        for (int i = 0; i < kDim / 16; ++i) {
          const uint4 x = lds_v4(piece(lane, i)), y = lds_v4(piece(lane + 32, i));
          any |= nan_codes(x) | nan_codes(y);
        }
        if (__any_sync(kAllLanes, any != 0)) {
          uint64_t nan = 0;  // the keys that have such codes
#pragma unroll 1
          for (int row = lane; row < kTile; row += 32) {
            bool found = false;
#pragma unroll 1
            for (int i = 0; i < kDim / 16; ++i) {
              const uint4 v = lds_v4(piece(row, i));
              if (nan_codes(v) == 0) continue;
              found = true;
              sts_v4(piece(row, i), without_nan(v));
            }
            nan |= uint64_t(__ballot_sync(kAllLanes, found)) << (row & 32);
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // (the slot's next copy)
          __syncwarp();
#pragma unroll
          for (int h = 0; h < kGrans; ++h)
            if (!there[h]) nan &= ~(uint64_t(0xFFFF) << (16 * h));
          const Segment& s = seg_of[seg];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const int r = min(s.rows - 1, s.r0 + nt * 8 + 2 * c + j);
              const int pos = s.len - s.n + r / p.group;
              if (nan & seen_keys(key, first_key(p, pos), last_key(p, pos, s.held)))
                l[nt][j] = __uint_as_float(kNaN);
            }
        }
      }
#pragma unroll
      for (int h = 0; h < kGrans; ++h) {
        uint32_t w[4][kWordsV];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int row = 16 * h + 2 * c + (j & 1) + 8 * (j >> 1);
          const uint32_t at = values + row * kDim;
          if constexpr (kDim == 128) {
            const uint4 v = lds_v4(at + ((g ^ (row & 7)) << 4));
            w[j][0] = v.x;
            w[j][1] = v.y;
            w[j][2] = v.z;
            w[j][3] = v.w;
          } else {
            const uint2 v = lds_v2(at + (((g >> 1) ^ ((row >> 1) & 3)) << 4) + (g & 1) * 8);
            w[j][0] = v.x;
            w[j][1] = v.y;
          }
          // what was never written may be no number
          if (!all && (key + row >= seg_of[seg].held || !there[h])) {
#pragma unroll
            for (int i = 0; i < kWordsV; ++i) w[j][i] = 0;
          }
        }
#pragma unroll
        for (int i = 0; i < kWordsV; ++i) {
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const uint32_t pick = half ? 0x7362 : 0x5140;
            const uint32_t x = __byte_perm(w[0][i], w[1][i], pick);
            const uint32_t y = __byte_perm(w[2][i], w[3][i], pick);
            const uint32_t a[4] = {f16_of_e4m3(x), f16_of_e4m3_high(x), f16_of_e4m3(y),
                                   f16_of_e4m3_high(y)};
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              mma_f16(o[nt][2 * i + half], a, pf[h][nt][0], pf[h][nt][1]);
          }
        }
      }
      __syncwarp();  // every lane has read the values
      if (2 * k + 1 + kSlots < 2 * count && !failed)
        issue((2 * k + 1 + kSlots) / 2, batch, (kSlots + 1) & 1);
    }
    flush(seg_of[seg], plan_u == v1 && !failed);
  }
  // after a failure: the copies still in flight, before the ring goes away
  for (int i = failed ? max(0, issued - kSlots) : issued; i < issued; ++i)
    mbar_wait(bars + 8 * (i % kSlots), uint32_t(i / kSlots) & 1u);
  if (p.bad && (__any_sync(kAllLanes, met_bad) || failed) && lane == 0) atomicAdd(p.bad, 1);
  __syncthreads();

  // ---- join the warps' parts, item by item, and CTAs' parts of an item
  // A task is two rows of an item; the warps take them in turn.
  const int64_t cta_slots = int64_t(kMaxCtas) * (2 * kWarps);
  // An item that a CTA shares stands at its start (slot 0) or runs over its end (slot 1).
  auto cta_slot = [&](int cta, int64_t begin, const Segment& s) {
    return cta_slots + 2 * cta + (s.item0 - kOpening <= begin ? 0 : 1);
  };
  int shared[2] = {-1, -1};  // parts of the items that other CTAs have parts of, too
  float v[2][kCols], top[2], sum[2];
  for (int i = 0, task = 0; i < 2 * kWarps;) {
    if (parts[i].rows == 0) {
      ++i;
      continue;
    }
    const Segment& s = parts[i];
    const int64_t to_slot = cta_slot(blockIdx.x, u0, s);
    const bool alone = s.item0 >= u0 && s.item0 + s.tiles <= u1;
    if (!alone) shared[to_slot & 1] = i;
    // the item's parts in this CTA, in key order, four bits each
    uint64_t which = 0;
    int n = 0;
    for (; i < 2 * kWarps && (parts[i].rows == 0 || parts[i].item0 == s.item0); ++i)
      if (parts[i].rows != 0) which |= uint64_t(i) << (4 * n++);
    const int rows = min(kRows, s.rows - s.r0);
    for (int r = 0; r < rows; r += 2, ++task) {
      if (task % kWarps != warp) continue;
      const int r2 = min(r + 1, rows - 1);
      join_parts<kCols>(
          n, r, r2,
          [&](int k) {
            const int part = int((which >> (4 * k)) & 15);
            if (!parts[part].in_ring) return PartAt{own_part(part), own_stats(part)};
            const float* o = ring_of(part >> 1);
            return PartAt{o, reinterpret_cast<const float2*>(o + kRows * kDim)};
          },
          v, top, sum);
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int at = x ? r2 : r;
        if (alone) {
          write_row(p, s, at, v[x], top[x], sum[x]);
        } else {
          float* to = p.part + (to_slot * kMaxRows + at) * kDim + lane * kCols;
#pragma unroll
          for (int k = 0; k < kCols; ++k) to[k] = v[x][k];
          if (lane == 0) p.stats[to_slot * kMaxRows + at] = make_float2(top[x], sum[x]);
        }
      }
    }
  }
  if (shared[0] < 0 && shared[1] < 0) return;
  // arrivals are counted at the CTA that has the item's last part
  __syncthreads();
  if (tid < 2) {
    s_last[tid] = false;
    const int of = tid == 0 ? shared[0] : shared[1];
    if (of >= 0) {
      const Segment& s = parts[of];
      const int c0 = cta_of(s.item0), c1 = cta_of(s.item0 + s.tiles - 1);
      s_last[tid] = atomic_add_acq_rel(p.count + c1, 1) == c1 - c0;
      if (s_last[tid]) p.count[c1] = 0;  // ready for the next call
    }
  }
  __syncthreads();
  for (int k = 0, task = 0; k < 2; ++k) {
    if (!s_last[k]) continue;
    const Segment& s = parts[k == 0 ? shared[0] : shared[1]];
    const int c0 = cta_of(s.item0), c1 = cta_of(s.item0 + s.tiles - 1);
    const int64_t first = cta_slot(c0, begin_of(c0), s);
    const int rows = min(kRows, s.rows - s.r0);
    for (int r = 0; r < rows; r += 2, ++task) {
      if (task % kWarps != warp) continue;
      const int r2 = min(r + 1, rows - 1);
      join_parts<kCols>(
          c1 - c0 + 1, r, r2,
          [&](int x) {
            const int64_t slot = x == 0 ? first : cta_slots + 2 * (c0 + x);
            return PartAt{p.part + slot * (kMaxRows * kDim), p.stats + slot * kMaxRows};
          },
          v, top, sum);
      write_row(p, s, r, v[0], top[0], sum[0]);
      write_row(p, s, r2, v[1], top[1], sum[1]);
    }
  }
}

// The codes as rows of a page and head, read in boxes of a unit's keys (or of a page of 16).
// A cache without pages is never read: any address will do.
int make_map(CUtensorMap* map, const Kv8& c, int which, int dim, void* any) {
  const EncodeTiled encode = tensor_map_encoder();
  if (!encode) return fail_cuda(DQ4_ERR_DEVICE, cudaErrorNotSupported);
  const cuuint64_t size[3] = {cuuint64_t(dim), cuuint64_t(c.page),
                              cuuint64_t(c.pages ? c.pages : 1) * cuuint64_t(c.heads)};
  const cuuint64_t stride[2] = {cuuint64_t(dim), cuuint64_t(dim) * cuuint64_t(c.page)};
  const cuuint32_t box[3] = {cuuint32_t(dim), cuuint32_t(c.page < kTile ? c.page : kTile), 1};
  const cuuint32_t step[3] = {1, 1, 1};
  const CUresult r = encode(
      map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, c.pages ? c.codes[which] : any, size, stride, box, step,
      CU_TENSOR_MAP_INTERLEAVE_NONE,
      dim == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
      CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? DQ4_OK : fail_cuda(DQ4_ERR_LAUNCH, cudaErrorInvalidValue);
}

template <int kDim, int NT>
int launch_one(const AttendArgs& p, int dev, int sms, cudaStream_t stream) {
  constexpr int kBytes = DecodeSmem<kDim>::kBytes;
  CUtensorMap k, v;
  if (const int st = make_map(&k, p.c, 0, kDim, p.count)) return st;
  if (const int st = make_map(&v, p.c, 1, kDim, p.count)) return st;
  auto kernel = dq4_kv8_decode_kernel<kDim, NT>;
  static std::atomic<uint64_t> allowed{0};
  if (const int st = allow_smem(kernel, kBytes, dev, &allowed)) return st;
  return launch_ordered(kernel, dim3(unsigned(sms < kMaxCtas ? sms : kMaxCtas)), kDecodeThreads,
                        kBytes, stream, k, v, p);
}

// Query rows of an item, 8 or 16, for calls with more than 8 a kv head.  A unit takes a CTA
// 0.26 us with 8 rows and 0.47 with 16, but 8 read each key twice as often.  While the keys
// stay in L2 that is for nothing; past half of its 129 MB (other data passes through it, too)
// 16 rows are taken, and also where they make the items few enough for a CTA each.  8 / 16, in
// us, 8 kv heads of 128 (64):
//   seqs x keys   16 rows                    24 rows
//    1 x 2000     14.5 / 18.3 (13.2 / 16.5)  15.6 / 17.2 (14.3 / 15.2)
//    4 x 8000     28.6 / 31.4 (24.3 / 25.3)  36.4 / 38.6 (29.8 / 31.0)
//   64 x 1000     53.7 / 56.9 (42.3 / 38.9)  72.0 / 78.6 (55.9 / 55.6)
//   64 x 4000      186 / 114  (111 / 85)
// and with a CTA each, 16 rows, 16 x 2000 keys: 29.7 / 25.6 (25.0 / 20.2).
bool wide_items(const AttendArgs& p, int64_t rows, int64_t keys, int dim, int sms) {
  const double blocks = double(p.s.seqs * p.c.heads);  // (double: estimates may be huge)
  const double narrow = double((rows + 7) / 8), wide = double((rows + 15) / 16);
  if (rows <= 8) return false;
  if (blocks * wide <= sms && sms < blocks * narrow) return true;
  return blocks * double(keys) * (2 * dim) > 64.5e6;
}

}  // namespace

static_assert(kMaxCtas * 4 <= kCounterBytes, "a counter for each CTA");

int64_t decode_workspace_bytes() {
  return kCounterBytes + int64_t(kParts) * kMaxRows * (8 + 128 * 4);
}

int launch_decode(const AttendArgs& args, int head_dim, int64_t rows, int64_t keys, int dev,
                  int sms, void* workspace, cudaStream_t stream) {
  AttendArgs p = args;
  p.count = static_cast<int*>(workspace);
  p.stats = reinterpret_cast<float2*>(static_cast<char*>(workspace) + kCounterBytes);
  p.part = reinterpret_cast<float*>(p.stats + int64_t(kParts) * kMaxRows);
  const bool wide = wide_items(p, rows, keys, head_dim, sms);
  if (head_dim == 64)
    return wide ? launch_one<64, 2>(p, dev, sms, stream) : launch_one<64, 1>(p, dev, sms, stream);
  return wide ? launch_one<128, 2>(p, dev, sms, stream) : launch_one<128, 1>(p, dev, sms, stream);
}

}  // namespace dq4d
