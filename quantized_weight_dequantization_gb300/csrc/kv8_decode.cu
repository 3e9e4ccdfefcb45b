// Attention over the 8-bit paged cache for few query rows a kv head (single tokens, grouped
// heads, a few proposed tokens): bound by the cache's bytes, each read once.
//
// The call's work is cut into units of 32 keys of one item (a sequence, a kv head and up to
// 8 NT query rows of it: new tokens x heads of the group).  One CTA runs per SM, on an equal
// run of the units, whatever the lengths are; an item that several CTAs share is summed from
// their FP32 partial results, in CTA order, by the last of them to finish.
//
// Within a CTA the warps take its units in turn.  Each warp has a ring of shared-memory
// stages of its own, filled by TMA (32 keys and values of one head, swizzled), and no other
// synchronization until the item ends: lane 0 issues, all lanes consume.  Page ids and
// scales are read ahead, 16 units of the warp at a time, one granule of 16 keys per lane.
//
// For a unit, with tensor-core products of FP16 operands and FP32 sums (m16n8k16):
//   S^T (keys x rows)  = K (keys x dim) Q^T      codes of K as FP16, exact
//   P   = 2^(c S + log2 vs - m + kLift)          c: softmax scale, page scale and row scale
//   O^T (dim x rows)  += V^T (dim x keys) P^T
//   l  += P / vs
// The page's V scale vs enters the exponent, so that P V needs no scaled V and the weights
// keep their precision whatever the scales are; l takes it out again.  Keys on the M side
// leave the N side of 8 to the few query rows.  The order of dim inside K Q^T, and of dim
// inside O^T, is free: a lane takes 16 or 32 consecutive bytes of a key for the first product
// and dim / 8 of a value for the second, so shared memory is read in 16-byte words.
#include "kv8_attend.cuh"

namespace dq4d {
namespace {

constexpr int kWarps = 8;
constexpr int kDecodeThreads = 32 * kWarps;
constexpr int kTile = 32;       // keys of a unit
constexpr int kMaxCtas = 160;   // CTAs the workspace has room for
constexpr int kMaxRows = 16;    // query rows of an item: 8 NT
constexpr int kSegs = 16;       // items, or parts of them, that a CTA plans at a time
constexpr int kBatch = 16;      // units of a warp whose pages are read ahead together

// An item, or the part of it that falls to a CTA.
struct Segment {
  int first;      // its first unit, from the CTA's first
  int tiles;      // units of the whole item
  int tile0;      // its first unit within the item
  int b, head;    // sequence and kv head
  int r0, rows;   // first query row of the item, and the sequence's rows
  int key0;       // the item's first key, a multiple of kTile
  int held, len, n, row;
  int64_t item0;  // the item's first unit of all
};

template <int kDim>
struct DecodeSmem {
  static constexpr int kStage = 2 * kTile * kDim;
  static constexpr int kStages = kDim == 128 ? 3 : 6;  // 24 KB a warp
  static constexpr int kPad = kDim;
  static constexpr int kMerge = kWarps * kStages * kStage;
  static constexpr int kStats = kMerge + kWarps * 8 * kPad * 4;  // [warp][row]{m, l}
  static constexpr int kBars = kStats + kWarps * 8 * 8;
  static constexpr int kBytes = kBars + kWarps * kStages * 8 + 1024;  // + alignment slack
  static_assert(kBytes + 1280 <= 227 * 1024, "shared memory budget");
};

struct SeqWork {
  int tiles, items, key0, held;
};

// The units of a sequence: its kv heads times its row tiles, times the units of 32 keys
// that its rows see (one at least, so that rows which see none get their zeros).
__device__ __forceinline__ SeqWork seq_work(const AttendArgs& p, const Seq& s, int rows_tile) {
  SeqWork w;
  w.held = held_keys(p, s.len);
  const int begin = first_key(p, s.len - s.n) & ~(kTile - 1);
  w.key0 = min(begin, w.held & ~(kTile - 1));
  w.tiles = max(1, (w.held - w.key0 + kTile - 1) / kTile);
  w.items = (s.n * p.group + rows_tile - 1) / rows_tile * p.c.heads;
  return w;
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

template <int kDim, int NT>
__global__ void __launch_bounds__(kDecodeThreads, 1)
    dq4_kv8_decode_kernel(const __grid_constant__ CUtensorMap map_k,
                          const __grid_constant__ CUtensorMap map_v, const AttendArgs p) {
  using S = DecodeSmem<kDim>;
  constexpr int kStages = S::kStages;
  constexpr int kRows = 8 * NT;         // query rows of an item
  constexpr int kSteps = kDim / 16;     // products along dim, and tiles of dim in O^T
  constexpr int kWordsK = kDim / 16;    // 4-byte words of a key a lane holds
  constexpr int kWordsV = kDim / 32;    // and of a value
  constexpr int kCols = kDim / 32;      // columns of the output a lane writes
  extern __shared__ uint8_t smem_raw[];
  __shared__ int64_t s_sums[kWarps], s_before;
  __shared__ int s_b0, s_nseg, s_done;
  __shared__ bool s_last;
  __shared__ Segment s_seg[kSegs];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(base);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, c = lane & 3;
  const uint32_t ring = sbase + warp * kStages * S::kStage;
  const uint32_t bars = sbase + S::kBars + warp * kStages * 8;
  float* merge = reinterpret_cast<float*>(base + S::kMerge);
  float2* stats = reinterpret_cast<float2*>(base + S::kStats);
  const uint64_t tk = reinterpret_cast<uint64_t>(&map_k), tv = reinterpret_cast<uint64_t>(&map_v);
  if (lane == 0) {
    for (int i = 0; i < kStages; ++i) mbar_init(bars + 8 * i, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("prefetch.tensormap [%0];" :: "l"(tk));
    asm volatile("prefetch.tensormap [%0];" :: "l"(tv));
  }
  wait_for_stream();

  // ---- the call's units, and the sequence where this CTA's run of them starts
  const int64_t seqs = p.s.seqs;
  auto units_of = [&](int64_t b) -> int64_t {
    if (b >= seqs) return 0;
    const SeqWork w = seq_work(p, seq_at(p.s, b), kRows);
    return int64_t(w.tiles) * w.items;
  };
  int64_t units = 0, before;
  const int64_t mine = units_of(tid);
  for (int64_t b = tid; b - tid < seqs; b += kDecodeThreads)
    units += block_scan(b == tid ? mine : units_of(b), s_sums, before);
  if (units == 0) return;
  const int64_t ctas = min(int64_t(gridDim.x), units);
  if (blockIdx.x >= ctas) return;
  const int64_t u0 = blockIdx.x * units / ctas, u1 = (blockIdx.x + 1) * units / ctas;
  auto cta_of = [&](int64_t u) { return ((u + 1) * ctas - 1) / units; };
  int64_t passed = 0;
  for (int64_t b = tid; b - tid < seqs; b += kDecodeThreads) {
    const int64_t v = b == tid ? mine : units_of(b);
    const int64_t total = block_scan(v, s_sums, before);
    before += passed;
    if (before <= u0 && u0 < before + v) {
      s_b0 = int(b);
      s_before = before;
    }
    passed += total;
    if (passed > u0) break;  // the same for every thread
  }
  __syncthreads();

  // ---- state of the segment a warp is in
  float o[NT][kSteps][4];
  float m[NT][2], l[NT][2], cq[NT][2];
  uint32_t qf[NT][kSteps][2];
  bool failed = false;
  int issued = 0, taken = 0;  // units of this warp, over all plans: ring positions
  int met_bad = 0;

  int64_t plan_u = u0, plan_first = s_before;  // next unit to plan; first unit of plan_b
  int plan_b = s_b0;
  while (plan_u < u1) {
    // ---- plan up to kSegs segments from plan_u on (warp 0; 32 sequences at a time)
    const int i0 = int(plan_u - u0);
    if (warp == 0) {
      int nseg = 0;
      int64_t u = plan_u, first = plan_first;
      int b = plan_b, from = -1;
      Seq s = {};
      SeqWork w = {};
      while (u < u1 && nseg < kSegs) {
        if (from < 0 || b >= from + 32) {
          from = b;
          if (b + lane < seqs) {
            s = seq_at(p.s, b + lane);
            w = seq_work(p, s, kRows);
          } else {
            w = SeqWork{1, 0, 0, 0};
          }
        }
        const int src = b - from;
        const int tiles = __shfl_sync(kAllLanes, w.tiles, src);
        const int items = __shfl_sync(kAllLanes, w.items, src);
        if (u >= first + int64_t(tiles) * items) {
          first += int64_t(tiles) * items;
          ++b;
          continue;
        }
        const int64_t in = u - first;
        const int item = int(in / tiles), tile = int(in - int64_t(item) * tiles);
        const int per_head = items / p.c.heads;
        if (lane == src) {
          Segment& g0 = s_seg[nseg];
          g0.first = int(u - u0);
          g0.tiles = tiles;
          g0.tile0 = tile;
          g0.b = b;
          g0.head = item / per_head;
          g0.r0 = item % per_head * kRows;
          g0.rows = s.n * p.group;
          g0.key0 = w.key0;
          g0.held = w.held;
          g0.len = s.len;
          g0.n = s.n;
          g0.row = int(s.row);
          g0.item0 = u - tile;
        }
        u = min(u1, u - tile + tiles);
        ++nseg;
      }
      if (lane == 0) {
        s_nseg = nseg;
        s_done = int(u - u0);
        s_b0 = b;
        s_before = first;
      }
    }
    __syncthreads();
    const int nseg = s_nseg, i1 = s_done;
    plan_u = u0 + i1;
    plan_b = s_b0;
    plan_first = s_before;

    // ---- pages read ahead: lane 2 t + h holds granule h (16 keys) of this warp's unit
    // 16 batch + t of the plan
    struct Ahead {
      int seg, key, block;  // block: page * kv_heads + head, or -1
      float ks, vs;
    };
    const int my_units = i1 - i0 > warp ? (i1 - i0 - warp + kWarps - 1) / kWarps : 0;
    auto read_ahead = [&](int batch) {
      Ahead a = {0, 0, -1, 0.f, 1.f};
      const int k = batch * kBatch + (lane >> 1);
      if (k >= my_units) return a;
      const int i = i0 + warp + k * kWarps;
      int sg = 0;
      while (sg + 1 < nseg && s_seg[sg + 1].first <= i) ++sg;
      const Segment& s = s_seg[sg];
      a.seg = sg;
      a.key = s.key0 + (s.tile0 + i - s.first) * kTile + (lane & 1) * 16;
      if (a.key < s.held) {
        const int id = __ldg(p.s.table + s.b * p.s.table_stride + (a.key >> p.c.log2_page));
        if (id >= 0 && id < p.c.pages) {
          a.block = id * p.c.heads + s.head;
          a.ks = p.c.scale[0][a.block];
          a.vs = used_scale(p.c.scale[1][a.block]);
        } else {
          met_bad = 1;
        }
      }
      if (s.held < s.len) met_bad = 1;
      return a;
    };
    Ahead now = read_ahead(0), next = read_ahead(1);
    const int rows_copy = min(p.c.page, kTile);
    // copies of unit k of the plan (of this or the next batch) into the ring
    auto issue = [&](int k, int batch) {
      const Ahead& a = (k / kBatch == batch) ? now : next;
      const int t = (k % kBatch) * 2;
      const int key = __shfl_sync(kAllLanes, a.key, t);
      const int b0 = __shfl_sync(kAllLanes, a.block, t);
      const int b1 = __shfl_sync(kAllLanes, a.block, t + 1);
      const int slot = issued % kStages;
      ++issued;
      if (lane == 0) {
        const uint32_t dst = ring + slot * S::kStage, bar = bars + 8 * slot;
        const int in_page = key & (p.c.page - 1);
        const bool two = rows_copy < kTile && b1 >= 0;
        const int copies = (b0 >= 0) + two;
        mbar_expect(bar, uint32_t(copies * 2 * rows_copy * kDim));
        if (b0 >= 0) {
          tma_load_3d(dst, tk, in_page, b0, bar);
          tma_load_3d(dst + kTile * kDim, tv, in_page, b0, bar);
        }
        if (two) {
          tma_load_3d(dst + 16 * kDim, tk, 0, b1, bar);
          tma_load_3d(dst + (kTile + 16) * kDim, tv, 0, b1, bar);
        }
      }
    };

    auto clear = [&] {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        m[nt][0] = m[nt][1] = -INFINITY;
        l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
        for (int i = 0; i < kSteps; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) o[nt][i][j] = 0.f;
      }
    };
    // ---- a new segment: its query rows as FP16 fragments, empty sums
    auto open = [&](const Segment& s) {
      clear();
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const int r = s.r0 + nt * 8 + g;
        uint4 raw[kWordsK / 2];
#pragma unroll
        for (int i = 0; i < kWordsK / 2; ++i) raw[i] = make_uint4(0, 0, 0, 0);
        if (r < s.rows) {
          const int tok = r / p.group;
          const uint16_t* q = static_cast<const uint16_t*>(p.q) +
                              (s.row + tok) * p.token_stride +
                              (s.head * p.group + r - tok * p.group) * p.head_stride +
                              c * (kDim / 4);
#pragma unroll
          for (int i = 0; i < kWordsK / 2; ++i)
            raw[i] = __ldg(reinterpret_cast<const uint4*>(q) + i);
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
      }
    };

    // Row r's result: columns kCols lane .. of O, with its m and l, to the output.
    auto write_row = [&](const Segment& s, int r, const float* v, float mm, float ll) {
      const int tok = r / p.group, head = s.head * p.group + r - tok * p.group;
      const int64_t at = int64_t(s.row + tok) * p.heads + head;
      const float inv = ll == 0.f ? 0.f : 1.f / ll;
      uint32_t* out = static_cast<uint32_t*>(p.out) + (at * kDim + lane * kCols) / 2;
#pragma unroll
      for (int i = 0; i < kCols / 2; ++i)
        out[i] = pack_out(v[2 * i] * inv, v[2 * i + 1] * inv, p.bf16);
      if (p.lse && lane == 0)
        p.lse[at] = ll == 0.f ? -INFINITY : fmaf(mm - kLift, kLn2, logf(ll));
    };

    // ---- the end of segment s: the warps' sums become one (warp w takes row w of each 8),
    // and the item's result if the segment is all of it
    auto close = [&](const Segment& s) {
      const int end = min(s.first + s.tiles - s.tile0, int(u1 - u0));
      const bool whole = s.tile0 == 0 && end - s.first == s.tiles;
      const int rows = min(kRows, s.rows - s.r0);
      const int slot = 2 * blockIdx.x + (s.first == 0 ? 0 : 1);
      float* part = p.part + int64_t(slot) * kMaxRows * (kDim + 2);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        if (nt * 8 >= rows) break;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float sum = l[nt][j];
#pragma unroll
          for (int w = 4; w < 32; w <<= 1) sum += __shfl_xor_sync(kAllLanes, sum, w);
          float* row = merge + (warp * 8 + 2 * c + j) * S::kPad + g * (kDim / 8);
#pragma unroll
          for (int i = 0; i < kSteps / 2; ++i)
            *reinterpret_cast<float4*>(row + 4 * i) =
                make_float4(o[nt][2 * i][j], o[nt][2 * i][2 + j], o[nt][2 * i + 1][j],
                            o[nt][2 * i + 1][2 + j]);
          if (g == 0) stats[warp * 8 + 2 * c + j] = make_float2(m[nt][j], sum);
        }
        __syncthreads();
        const int r = nt * 8 + warp;
        if (r < rows) {
          float top = -INFINITY;
#pragma unroll
          for (int w = 0; w < kWarps; ++w) top = fmaxf(top, stats[w * 8 + warp].x);
          const float from = top == -INFINITY ? 0.f : top;
          float sum = 0.f, v[kCols] = {};
#pragma unroll
          for (int w = 0; w < kWarps; ++w) {
            const float2 st = stats[w * 8 + warp];
            const float f = exp2_fast(st.x - from);
            sum = fmaf(f, st.y, sum);
            const float* row = merge + (w * 8 + warp) * S::kPad + lane * kCols;
#pragma unroll
            for (int i = 0; i < kCols; ++i) v[i] = fmaf(f, row[i], v[i]);
          }
          if (whole) {
            write_row(s, s.r0 + r, v, top, sum);
          } else {
            float* to = part + r * (kDim + 2);
#pragma unroll
            for (int i = 0; i < kCols; ++i) to[lane * kCols + i] = v[i];
            if (lane == 0) {
              to[kDim] = top;
              to[kDim + 1] = sum;
            }
          }
        }
        __syncthreads();
      }
      if (whole) return;
      // the parts of a shared item: CTAs c0 .. c1, counted where c1's part is
      const int c0 = int(cta_of(s.item0)), c1 = int(cta_of(s.item0 + s.tiles - 1));
      if (tid == 0) {
        const int arrived = atomic_add_acq_rel(p.count + c1, 1);
        s_last = arrived == c1 - c0;
        if (s_last) p.count[c1] = 0;  // ready for the next call
      }
      __syncthreads();
      if (s_last) {
        for (int r = warp; r < rows; r += kWarps) {
          // CTA c's part is its first segment, but for c0, where the item may begin later
          auto part_of = [&](int cta) {
            const bool first = cta != c0 || cta * units / ctas == s.item0;
            return p.part + (int64_t(2 * cta + (first ? 0 : 1)) * kMaxRows + r) * (kDim + 2);
          };
          float top = -INFINITY;
          for (int cta = c0 + lane; cta <= c1; cta += 32) top = fmaxf(top, __ldcg(part_of(cta) + kDim));
#pragma unroll
          for (int w = 16; w > 0; w >>= 1) top = fmaxf(top, __shfl_xor_sync(kAllLanes, top, w));
          const float from = top == -INFINITY ? 0.f : top;
          float sum = 0.f, v[kCols] = {};
#pragma unroll 4
          for (int cta = c0; cta <= c1; ++cta) {
            const float* row = part_of(cta);
            const float f = exp2_fast(__ldcg(row + kDim) - from);
            sum = fmaf(f, __ldcg(row + kDim + 1), sum);
#pragma unroll
            for (int i = 0; i < kCols; ++i) v[i] = fmaf(f, __ldcg(row + lane * kCols + i), v[i]);
          }
          write_row(s, s.r0 + r, v, top, sum);
        }
      }
      __syncthreads();  // s_last may be set anew
    };

    // ---- the units of this plan
    int seg = -1;
    const int lead = min(kStages, my_units);
    for (int k = 0; k < lead; ++k) issue(k, 0);
    for (int k = 0; k < my_units; ++k) {
      const int batch = k / kBatch, t = (k % kBatch) * 2;
      if (k > 0 && k % kBatch == 0) {
        now = next;
        next = read_ahead(batch + 1);
      }
      const int sg = __shfl_sync(kAllLanes, now.seg, t);
      if (sg != seg) {
        for (int x = seg < 0 ? 0 : seg; x < sg; ++x) {
          if (x != seg) clear();  // no unit of it here
          close(s_seg[x]);
        }
        seg = sg;
        open(s_seg[seg]);
      }
      const Segment& s = s_seg[seg];
      const int key = __shfl_sync(kAllLanes, now.key, t);
      const int slot = taken % kStages;
      if (!failed && !mbar_wait(bars + 8 * slot, uint32_t(taken / kStages) & 1u)) failed = true;
      ++taken;
      const uint32_t kv = ring + slot * S::kStage;
      float ks[2], vs[2];
      bool there[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        ks[h] = __shfl_sync(kAllLanes, now.ks, t + h);
        vs[h] = __shfl_sync(kAllLanes, now.vs, t + h);
        there[h] = __shfl_sync(kAllLanes, now.block, t + h) >= 0;
      }
      // whether every row sees every key of the unit
      const int p0 = s.len - s.n + s.r0 / p.group;
      const int p1 = s.len - s.n + min(s.rows - 1, s.r0 + kRows - 1) / p.group;
      const bool all = there[0] && there[1] && key >= first_key(p, p1) &&
                       key + kTile <= last_key(p, p0, s.held);

      // ---- S^T: keys 16 h + g and + 8, rows 8 nt + 2 c and + 1
      float st[2][NT][4];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint4 raw[2][kWordsK / 4];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int row = 16 * h + 8 * j + g;
          const uint32_t at = kv + row * kDim;
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

      // ---- the softmax's weights, in base 2; the lanes of equal c share their rows
      float bias[2], inv[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        bias[h] = __log2f(vs[h]);
        inv[h] = 1.f / vs[h];
      }
      uint32_t pf[2][NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float x[4];
#pragma unroll
          for (int i = 0; i < 4; ++i)  // key 8 i + g
            x[i] = fmaf(st[i >> 1][nt][2 * (i & 1) + j], cq[nt][j] * ks[i >> 1], bias[i >> 1]);
          if (!all) {
            const int r = min(s.rows - 1, s.r0 + nt * 8 + 2 * c + j);
            const int pos = s.len - s.n + r / p.group;
            const int lo = first_key(p, pos), hi = last_key(p, pos, s.held);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int at = key + 8 * i + g;
              if (at < lo || at >= hi || !there[i >> 1]) x[i] = -INFINITY;
            }
          }
          float top = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
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
          for (int i = 0; i < 4; ++i) {
            x[i] = all || x[i] != -INFINITY ? exp2_fast(x[i] - from) : 0.f;
            st[i >> 1][nt][2 * (i & 1) + j] = x[i];
          }
          if (all) {
            l[nt][j] = fmaf(x[0] + x[1], inv[0], fmaf(x[2] + x[3], inv[1], l[nt][j]));
          } else {  // an unseen granule's scale may be no number
            if (x[0] + x[1] != 0.f) l[nt][j] = fmaf(x[0] + x[1], inv[0], l[nt][j]);
            if (x[2] + x[3] != 0.f) l[nt][j] = fmaf(x[2] + x[3], inv[1], l[nt][j]);
          }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          pf[h][nt][0] = transpose8(pack_f16(st[h][nt][0], st[h][nt][1]));
          pf[h][nt][1] = transpose8(pack_f16(st[h][nt][2], st[h][nt][3]));
        }
      }

      // ---- O^T += V^T P^T: keys 2 c, 2 c + 1, + 8 and + 9 of each 16, dims g kDim / 8 ..
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t w[4][kWordsV];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int row = 16 * h + 2 * c + (j & 1) + 8 * (j >> 1);
          const uint32_t at = kv + (kTile + row) * kDim;
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
          if (!all && (key + row >= s.held || !there[h])) {
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
      __syncwarp();  // every lane has read the stage
      if (k + kStages < my_units && !failed) issue(k + kStages, batch);
    }
    for (int x = seg < 0 ? 0 : seg; x < nseg; ++x) {
      if (x != seg) clear();
      close(s_seg[x]);
    }
    if (failed) {  // the copies still in flight, before the ring goes away
      for (; taken < issued; ++taken)
        mbar_wait(bars + 8 * (taken % kStages), uint32_t(taken / kStages) & 1u);
    }
    __syncthreads();  // the next plan overwrites this one
  }
  if (p.bad && (__any_sync(kAllLanes, met_bad) || failed) && lane == 0) atomicAdd(p.bad, 1);
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
int launch_one(const AttendArgs& p, int sms, cudaStream_t stream) {
  constexpr int kBytes = DecodeSmem<kDim>::kBytes;
  CUtensorMap k, v;
  if (const int st = make_map(&k, p.c, 0, kDim, p.count)) return st;
  if (const int st = make_map(&v, p.c, 1, kDim, p.count)) return st;
  auto kernel = dq4_kv8_decode_kernel<kDim, NT>;
  const cudaError_t e =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes);
  if (e != cudaSuccess) return fail_cuda(DQ4_ERR_LAUNCH, e);
  return launch_ordered(kernel, dim3(unsigned(sms < kMaxCtas ? sms : kMaxCtas)), kDecodeThreads,
                        kBytes, stream, k, v, p);
}

}  // namespace

int64_t decode_workspace_bytes() {
  return kMaxCtas * 4 + int64_t(2) * kMaxCtas * kMaxRows * (128 + 2) * 4;
}

int launch_decode(const AttendArgs& args, int head_dim, int rows, int sms, void* workspace,
                  cudaStream_t stream) {
  AttendArgs p = args;
  p.count = static_cast<int*>(workspace);
  p.part = reinterpret_cast<float*>(p.count + kMaxCtas);
  if (head_dim == 64)
    return rows <= 8 ? launch_one<64, 1>(p, sms, stream) : launch_one<64, 2>(p, sms, stream);
  return rows <= 8 ? launch_one<128, 1>(p, sms, stream) : launch_one<128, 2>(p, sms, stream);
}

}  // namespace dq4d
