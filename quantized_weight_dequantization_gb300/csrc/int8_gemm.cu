// Products of many rows with an 8-bit weight on tcgen05: Y = X W^T (dq4_int8_linear) and
// dX = dY W (dq4_int8_linear_backward).
//
// The weight is the MMA's A operand: 128 of its rows (or, for the gradient, columns) are the
// lanes of TMEM, where its 16-bit values are written a stage of 128 at a time; BX rows of the
// activations are B, read by TMA from their 16-bit form.  For the product that form is made by a
// kernel of its own (int8_rows_kernel: codes as FP16, outliers in place of their codes), which
// costs 3 bytes a value once, where converting inside would cost every weight tile the same again.
//
// A CTA takes items (a tile, or a part of a tile's sum where there are few) in turn:
//   warps 0..7    two groups that take alternate stages: codes from shared memory to 16-bit values
//                 in TMEM, a thread a lane
//   warps 8..15   read a finished tile out of TMEM, scale, store.  A part of a tile's sum is left
//                 in shared memory for the cluster, whose CTAs each add and store a share of the
//                 columns; or in the workspace, for the last part's CTA, which adds them all.  The
//                 order of the parts is that of the sum, so that the same call gives the same bits
//   then          one or two warps that issue the MMAs (alternate stages, accumulators of their
//                 own: issuing takes a thread about 120 cycles, whatever BX is), the warp that
//                 copies the weight's codes, the warp that copies the activations
// Waits are bounded; one that runs out counts into *bad, raises a flag of the CTA, and every
// role lets its copies and MMAs finish and ends.
//
// What bounds it: the MMAs, 128 x BX x 16, take about 105 cycles at BX 64 and 128 and 169 at 256,
// where 32, 64 and 128 would be the rate of the tensor cores: with A in TMEM the smaller ones are
// no faster, and the largest shares the shared memory with the copies and the producers
// (activations in and out, codes in and out: 160 cycles at 128 bytes a cycle).  8191 rows through
// 4096 x 14336: 610 to 653 us, 0.76 to 0.82 of the measured rate of the GPU; the gradient of 2047
// rows through 11008 x 4096 150 us, 0.64: its producers' instructions, three packed ones for two
// values.  (Pairs of CTAs with tiles of 256 x 256, the weight's values in TMEM or in shared
// memory: 790 to 824 us for the 8191 rows.)
#include "int8_gemm.cuh"

namespace dq4d {
namespace {

constexpr int kStep = 64;            // values of a K step: 128 bytes of 16-bit values
constexpr int kStage = 2 * kStep;    // of a stage
constexpr int kTileW = 128;          // weight rows (columns) of a tile: TMEM lanes
constexpr int kRawSlot = kTileW * kStage;  // bytes of a stage's codes
constexpr int kRawSlots = 4;
constexpr int kRing = 4;             // stages in TMEM
constexpr uint32_t kRingCol = 256;   // where they start; the accumulators lie before
constexpr uint32_t kTmemColumns = 512;
constexpr int kProducers = 8, kReaders = 8;

template <int BX, bool kBack>
struct Gemm {
  static constexpr int kIssuers = BX < 256 ? 2 : 1;
  static constexpr int kBuffers = 256 / (BX * kIssuers);  // accumulators of an issuer
  // a slot of activations is a stage for two issuers (so that stage g's slot is always taken
  // by the same one), a step for one
  static constexpr int kSlotSteps = kIssuers;
  static constexpr int kStepBytes = BX * kStep * 2;
  static constexpr int kSlot = kSlotSteps * kStepBytes;
  static constexpr int kSlots = BX == 256 ? (kBack ? 4 : 5) : BX == 128 ? 4 : 6;
  static_assert(kIssuers == 1 || kSlots % 2 == 0, "a slot belongs to one issuer");
  static constexpr int kThreads = 32 * (kProducers + kReaders + kIssuers + 2);
  static constexpr int kRawAt = kSlots * kSlot;
  static constexpr int kBarsAt = kRawAt + kRawSlots * kRawSlot;
  // where parts of a tile are joined: pieces of 32 rows (both readers' halves) in the idle rings
  static constexpr int kPiece = 2 * 32 * kTileW * 4;
  static constexpr int kPieces = kBarsAt / kPiece;
  static constexpr int kBars = 2 * kSlots + 2 * kRawSlots + 2 * kRing + 2 * kBuffers + 2 + kPieces;
  static constexpr int kBytes = kBarsAt + 8 * kBars + 1024;  // + alignment slack
  static constexpr int kStatic = kBack ? 16 * kStage + 64 : 4 * BX + 64;
  static_assert(kBytes + kStatic <= 227 * 1024, "shared memory");
  static_assert(kBytes > 116 * 1024, "one CTA per SM: the TMEM allocation never waits");
};

struct GemmArgs {
  int64_t lanes, rows;   // of the output: weight rows (columns), activation rows
  int steps, code_steps; // K steps, and of them with codes from CB (the rest: outlier columns, from
                         // their own matrix)
  int tiles_x;           // tiles along the activations
  int64_t tiles;
  int64_t units;         // tiles * stages, if CTAs take equal runs of them; 0: whole tiles in turn
  int cluster;           // CTAs that share a tile's stages, and its columns at the end; 1: none
  const float* SCB;
  int64_t N;             // weight rows
  const float* row_units;  // of the activation rows
  const void* bias;
  int out_dtype;
  void* out;             // [rows][lanes]
  float4* part;          // [CTAs][2][BX / 4][128]: a CTA's parts of its first and its last tile
  int* count;            // [CTAs] parts of the tile whose last one the CTA has
  int* bad;
};

__device__ __forceinline__ void bar_readers() {
  asm volatile("bar.sync 1, %0;" :: "n"(32 * kReaders) : "memory");
}
__device__ __forceinline__ bool all_readers(bool v) {
  uint32_t r;
  asm volatile(
      "{\n.reg .pred p, q;\nsetp.ne.u32 p, %1, 0;\nbar.red.and.pred q, 1, %2, p;\n"
      "selp.u32 %0, 1, 0, q;\n}"
      : "=r"(r) : "r"(uint32_t(v)), "n"(32 * kReaders) : "memory");
  return r != 0;
}
__device__ __forceinline__ void commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];"
               :: "r"(bar) : "memory");
}
__device__ __forceinline__ int load_acquire(const int* p) {
  int v;
  asm volatile("ld.acquire.gpu.global.b32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
// Clusters: the place in CTA r's shared memory of one in this CTA's; an arrival there, after what
// the warp wrote; what has been written before a phase that has completed; a read; all threads.
__device__ __forceinline__ uint32_t of_cta(uint32_t addr, int r) {
  uint32_t there;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(addr), "r"(r));
  return there;
}
__device__ __forceinline__ void arrive_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];"
               :: "r"(bar) : "memory");
}
__device__ __forceinline__ void see_cluster(uint32_t bar, uint32_t parity) {
  asm volatile(
      "{\n.reg .pred p;\nmbarrier.test_wait.parity.acquire.cluster.shared::cta.b64 p, [%0], %1;\n}"
      :: "r"(bar), "r"(parity) : "memory");
}
__device__ __forceinline__ void load_cluster(uint32_t addr, uint32_t* v) {
  asm volatile("ld.shared::cluster.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void sync_cluster() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;"
               ::: "memory");
}
// Four 8 x 8 matrices of 16-bit elements, transposed; a thread gives the address of a row.
__device__ __forceinline__ void load_transposed(uint32_t addr, uint32_t* m) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(m[0]), "=r"(m[1]), "=r"(m[2]), "=r"(m[3]) : "r"(addr) : "memory");
}
// 16 lanes of TMEM, 32 columns: words 4i, 4i + 1 of a thread are columns 8i + 2 (lane % 4) and
// the next of lane / 4, words 4i + 2, 4i + 3 those of lane / 4 + 8.
__device__ __forceinline__ void tmem_st_16(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x256b.x4.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15,%16};"
      :: "r"(taddr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]),
         "r"(v[7]), "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]),
         "r"(v[14]), "r"(v[15]));
}
// {a, b} + {c, c} and {a, b} * {c, d}, each rounded on its own.
__device__ __forceinline__ uint64_t pair_of(uint32_t a, uint32_t b) {
  return uint64_t(b) << 32 | a;
}
__device__ __forceinline__ uint64_t add_pair(uint64_t x, uint64_t y) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
  return r;
}
__device__ __forceinline__ uint64_t mul_pair(uint64_t x, uint64_t y) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
  return r;
}

// A ring's place and the parity of its phase, by the number of its uses.
template <int kDepth>
struct Place {
  int slot = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next() {
    if (++slot == kDepth) {
      slot = 0;
      phase ^= 1u;
    }
  }
};

// kBack: lanes are columns of the weight, the sum runs over its rows.  kBF16: 16-bit values are
// BF16 (the gradient's), else FP16.
template <int BX, bool kBack, bool kBF16>
__global__ void __launch_bounds__(Gemm<BX, kBack>::kThreads, 1)
    dq4_int8_gemm_kernel(const __grid_constant__ CUtensorMap map_w,
                         const __grid_constant__ CUtensorMap map_x,
                         const __grid_constant__ CUtensorMap map_cols, const GemmArgs p) {
  using S = Gemm<BX, kBack>;
  constexpr int kIssuers = S::kIssuers, kBuffers = S::kBuffers, kSlots = S::kSlots;
  constexpr int kOut = kBF16 ? DQ4_OUT_BF16 : DQ4_OUT_F16;
  constexpr int kMmaWarp = kProducers + kReaders;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint32_t s_tmem;
  __shared__ volatile int s_abort;
  __shared__ bool s_last;
  __shared__ __align__(16) float s_unit[kBack ? 4 : BX];  // of the item's rows
  __shared__ __align__(16) float s_scale[kBack ? 4 * kStage : 4];  // two stages of each group
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(base);
  const uint32_t bar0 = sbase + S::kBarsAt;
  auto x_full = [&](int s) { return bar0 + 8 * s; };
  auto x_empty = [&](int s) { return bar0 + 8 * (kSlots + s); };
  auto raw_full = [&](int s) { return bar0 + 8 * (2 * kSlots + s); };
  auto raw_empty = [&](int s) { return bar0 + 8 * (2 * kSlots + kRawSlots + s); };
  auto w_full = [&](int s) { return bar0 + 8 * (2 * kSlots + 2 * kRawSlots + s); };
  auto w_empty = [&](int s) { return bar0 + 8 * (2 * kSlots + 2 * kRawSlots + kRing + s); };
  auto acc_full = [&](int b) {
    return bar0 + 8 * (2 * kSlots + 2 * kRawSlots + 2 * kRing + b);
  };
  auto acc_empty = [&](int b) { return acc_full(kBuffers + b); };
  const uint32_t all_done = acc_full(2 * kBuffers);
  const uint32_t shared = acc_full(2 * kBuffers + 1);  // the cluster's accumulators can be read
  auto piece_full = [&](int s) { return acc_full(2 * kBuffers + 2 + s); };
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  volatile int* aborted = &s_abort;
  auto fail = [&] {
    *aborted = 1;
    if (p.bad) atomicAdd(p.bad, 1);
  };

  // ---- setup: touches no global memory, so it overlaps the kernel before this one
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                 :: "r"(smem_u32(&s_tmem)), "r"(kTmemColumns));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    if (lane == 0) {
      for (int s = 0; s < kSlots; ++s) {
        mbar_init(x_full(s), 1);
        mbar_init(x_empty(s), 1);
      }
      for (int s = 0; s < kRawSlots; ++s) {
        mbar_init(raw_full(s), 1);
        mbar_init(raw_empty(s), kProducers / 2);
      }
      for (int s = 0; s < kRing; ++s) {
        mbar_init(w_full(s), kProducers / 2);
        mbar_init(w_empty(s), 1);
      }
      for (int b = 0; b < kBuffers; ++b) {
        mbar_init(acc_full(b), kIssuers);
        mbar_init(acc_empty(b), kReaders);
      }
      mbar_init(all_done, kIssuers);
      mbar_init(shared, kReaders * p.cluster);
      for (int s = 0; s < S::kPieces; ++s) mbar_init(piece_full(s), 1);
      *aborted = 0;
      asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
      asm volatile("prefetch.tensormap [%0];" :: "l"(reinterpret_cast<uint64_t>(&map_w)));
      asm volatile("prefetch.tensormap [%0];" :: "l"(reinterpret_cast<uint64_t>(&map_x)));
    }
  }
  wait_for_stream();
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  if (p.cluster > 1) sync_cluster();  // (the other CTAs' barriers)
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tmem = s_tmem;

  // An item: a tile, or the part of it that falls to this CTA.  Every role walks the CTA's items;
  // stages are counted over all of them (g), and stage g is group and issuer g % 2's, in slot
  // g % depth.
  struct Item {
    int64_t tile, lane0, row0;
    int begin, end;  // stages
  };
  const int stages = (p.steps + 1) / 2;
  const int64_t ctas = gridDim.x;
  auto begin_of = [&](int64_t cta) { return cta * p.units / ctas; };
  auto cta_of = [&](int64_t u) { return ((u + 1) * ctas - 1) / p.units; };
  const int rank = int(blockIdx.x % p.cluster);  // of the cluster
  const int64_t walk0 = p.units ? begin_of(blockIdx.x) : blockIdx.x / p.cluster;
  const int64_t walk1 = p.units ? begin_of(blockIdx.x + 1) : p.cluster > 1 ? walk0 + 1 : p.tiles;
  auto next_item = [&](int64_t& at, Item& it) {
    if (at >= walk1) return false;
    it.tile = at;
    it.begin = 0;
    it.end = stages;
    if (p.units) {
      it.tile = at / stages;
      it.begin = int(at - it.tile * stages);
      it.end = int(min(int64_t(stages), it.begin + walk1 - at));
      at += it.end - it.begin;
    } else {
      it.begin = rank * stages / p.cluster;
      it.end = (rank + 1) * stages / p.cluster;
      at += ctas;
    }
    const int64_t tw = it.tile / p.tiles_x;
    it.lane0 = tw * kTileW;
    it.row0 = (it.tile - tw * p.tiles_x) * BX;
    return true;
  };
  auto steps_of = [&](int stage) { return min(2, p.steps - 2 * stage); };

  if (warp == kMmaWarp + kIssuers) {
    if (lane == 0) {
      // ---- the weight's codes: 128 rows of 128 bytes a stage
      const uint64_t map = reinterpret_cast<uint64_t>(&map_w);
      const uint64_t cols = reinterpret_cast<uint64_t>(&map_cols);
      Place<kRawSlots> at;
      int g = 0;
      bool stop = false;
      Item it;
      for (int64_t walk = walk0; !stop && next_item(walk, it);) {
        for (int s = it.begin; s < it.end; ++s, ++g, at.next()) {
          if (g >= kRawSlots && (*aborted || !mbar_wait(raw_empty(at.slot), at.phase ^ 1u))) {
            if (!*aborted) fail();
            stop = true;
            break;
          }
          const uint32_t to = sbase + S::kRawAt + at.slot * kRawSlot;
          mbar_expect(raw_full(at.slot), kRawSlot);
          if constexpr (kBack)
            tma_load_2d(to, map, int(it.lane0), s * kStage, raw_full(at.slot));
          else if (2 * s < p.code_steps)
            tma_load_2d(to, map, s * kStage, int(it.lane0), raw_full(at.slot));
          else
            tma_load_2d(to, cols, s * kStage - p.code_steps * kStep, int(it.lane0),
                        raw_full(at.slot));
        }
      }
      if (*aborted)  // copies in flight land before the CTA leaves
        for (int j = g - 1; j >= 0 && j >= g - kRawSlots; --j)
          mbar_wait(raw_full(j % kRawSlots), (j / kRawSlots) & 1);
    }
  } else if (warp == kMmaWarp + kIssuers + 1) {
    if (lane == 0) {
      // ---- the activations: BX rows of 64 values a step
      const uint64_t map = reinterpret_cast<uint64_t>(&map_x);
      Place<kSlots> at;
      int q = 0;
      bool stop = false;
      Item it;
      for (int64_t walk = walk0; !stop && next_item(walk, it);) {
        for (int s = it.begin; s < it.end && !stop; ++s) {
          const int n = steps_of(s);
          for (int sub = 0; sub < n; sub += S::kSlotSteps, ++q, at.next()) {
            if (q >= kSlots && (*aborted || !mbar_wait(x_empty(at.slot), at.phase ^ 1u))) {
              if (!*aborted) fail();
              stop = true;
              break;
            }
            const int here = min(S::kSlotSteps, n - sub);
            mbar_expect(x_full(at.slot), here * S::kStepBytes);
            for (int k = 0; k < here; ++k)
              tma_load_2d(sbase + at.slot * S::kSlot + k * S::kStepBytes, map,
                          (2 * s + sub + k) * kStep, int(it.row0), x_full(at.slot));
          }
        }
      }
      if (*aborted)
        for (int j = q - 1; j >= 0 && j >= q - kSlots; --j)
          mbar_wait(x_full(j % kSlots), (j / kSlots) & 1);
    }
  } else if (warp >= kMmaWarp) {
    if (lane == 0) {
      // ---- the MMAs: issuer `mine` takes the stages g with g % kIssuers == mine
      const int mine = warp - kMmaWarp;
      const uint32_t idesc = instr_desc_f16<kTileW, BX>(kBF16);
      Place<kRing> wp;
      Place<kSlots> xp;
      int g = 0, buffer = 0, turn = 0;
      bool stop = false;
      Item it;
      for (int64_t walk = walk0; !stop && next_item(walk, it); ++turn) {
        buffer = turn % kBuffers;
        if (turn >= kBuffers && (*aborted || !mbar_wait(acc_empty(buffer),
                                                        uint32_t(turn / kBuffers - 1) & 1u))) {
          if (!*aborted) fail();
          break;
        }
        const uint32_t acc = tmem + (mine * kBuffers + buffer) * BX;
        uint32_t more = 0;  // whether the accumulator holds something
        for (int s = it.begin; s < it.end; ++s, ++g, wp.next()) {
          const int n = steps_of(s);
          if (kIssuers > 1 && (g & 1) != mine) {
            xp.next();
            continue;
          }
          // the weight's values and the activations, looked at together first: a look costs the
          // issuing thread about 40 cycles, a wait for what is there 110, and the MMAs wait with it
          constexpr int kLooks = kIssuers == 1 ? 2 : 1;
          Place<kSlots> xn = xp;
          bool ready = mbar_test(w_full(wp.slot), wp.phase);
#pragma unroll
          for (int k = 0; k < kLooks; ++k)
            if (k < n) {
              ready &= mbar_test(x_full(xn.slot), xn.phase);
              xn.next();
            }
          if (!ready) {
            xn = xp;
            bool ok = !*aborted && mbar_wait(w_full(wp.slot), wp.phase);
            for (int k = 0; k < kLooks && k < n && ok; ++k, xn.next())
              ok = mbar_wait(x_full(xn.slot), xn.phase);
            if (!ok) {
              if (!*aborted) fail();
              stop = true;
              break;
            }
          }
          asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
#pragma unroll
          for (int sub = 0; sub < 2; ++sub) {
            if (sub >= n) break;
            const int in_slot = sub % S::kSlotSteps;
            const uint32_t a = tmem + kRingCol + (wp.slot * 2 + sub) * 32;
            const uint32_t b = sbase + xp.slot * S::kSlot + in_slot * S::kStepBytes;
#pragma unroll
            for (int k = 0; k < kStep / 16; ++k) {
              asm volatile(
                  "{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\n"
                  "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}"
                  :: "r"(acc), "r"(a + k * 8), "l"(smem_desc(b + k * 32)), "r"(idesc), "r"(more));
              more = 1;
            }
            if (in_slot == S::kSlotSteps - 1 || sub == n - 1) {
              commit(x_empty(xp.slot));
              xp.next();
            }
          }
          commit(w_empty(wp.slot));
        }
        if (stop) break;
        commit(acc_full(buffer));
      }
      // every MMA issued above has finished before the TMEM is freed
      commit(all_done);
      mbar_wait(all_done, 0);
    }
  } else if (warp < kProducers) {
    // ---- the weight's 16-bit values: thread r of a group is lane r of TMEM
    const int group = warp / 4, quad = warp & 3, r = quad * 32 + lane;
    const uint32_t to0 = tmem + (uint32_t(quad * 32) << 16) + kRingCol;
    Place<kRing> wp;
    Place<kRawSlots> rp;
    int g = 0;
    bool stop = false, given_up = false;
    // the scale of row r of this group's next stage of an item, loaded a stage of the group ahead
    float scale = 0.f;
    int loaded = -1, scale_turn = 0;  // (loaded: the stage whose scale that is)
    auto scale_of = [&](int s) {
      const int64_t n = int64_t(s) * kStage + r;
      return n < p.N ? load_global(p.SCB + n) : 0.f;
    };
    Item it;
    for (int64_t walk = walk0; !stop && next_item(walk, it);) {
      for (int s = it.begin; s < it.end; ++s, ++g, wp.next(), rp.next()) {
        if ((g & 1) != group) continue;
        if constexpr (kBack) {
          if (loaded != s) scale = scale_of(s);
          s_scale[(group * 2 + scale_turn) * kStage + r] = scale;
          // The group's scales are there; and if one of its warps gave up on its last stage, all
          // of them end here.
          uint32_t go;
          asm volatile(
              "{\n.reg .pred p, q;\nsetp.ne.u32 p, %1, 0;\nbar.red.and.pred q, %2, %3, p;\n"
              "selp.u32 %0, 1, 0, q;\n}"
              : "=r"(go) : "r"(uint32_t(!given_up)), "r"(2 + group), "n"(32 * kProducers / 2)
              : "memory");
          if (go == 0) {
            stop = true;
            break;
          }
          loaded = s + 2 < it.end ? s + 2 : -1;
          if (loaded >= 0) scale = scale_of(loaded);
        }
        const bool ok = !*aborted &&
                        (mbar_try2(raw_full(rp.slot), rp.phase, w_empty(wp.slot),
                                   g >= kRing ? wp.phase ^ 1u : 1u) ||
                         (mbar_wait(raw_full(rp.slot), rp.phase) &&
                          (g < kRing || mbar_wait(w_empty(wp.slot), wp.phase ^ 1u))));
        if (!__all_sync(kAllLanes, ok)) {
          if (lane == 0 && !*aborted) fail();
          if constexpr (kBack) {
            given_up = true;
            continue;
          }
          stop = true;
          break;
        }
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        const int n = steps_of(s);
        const uint32_t raw = sbase + S::kRawAt + rp.slot * kRawSlot;
#pragma unroll 1
        for (int sub = 0; sub < n; ++sub) {
          const uint32_t to = to0 + (wp.slot * 2 + sub) * 32;
          if constexpr (kBack) {
            // Rows are 128 bytes, their 16-byte pieces at place ^ row % 8.  A matrix of the load is
            // 8 rows of 8 pairs of columns; transposed, a thread has pair lane / 4 of two rows.
            // With rows 0, 1, 4, 5, 8, ... in one and 2, 3, 6, 7, ... in the next it has four rows
            // that follow one another, which is what it stores of a TMEM lane; columns 2c and 2c +
            // 1 become lanes c and c + 8.  (A byte at a time, a column a thread: 64 loads a step in
            // place of 4, and 2047 rows through 11008 x 4096 took 160 us; so 150.)
            const float* sc =
                s_scale + (group * 2 + scale_turn) * kStage + sub * kStep + 4 * (lane & 3);
            const int row = sub * kStep + (lane >> 4) * 16 + (lane >> 3 & 1) * 2 +
                            (lane >> 1 & 3) * 4 + (lane & 1);
            const uint32_t from = raw + row * kTileW;
            const uint64_t off = pair_of(0xCB000080u, 0xCB000080u);  // -(2^23 + 128)
            const uint64_t r127 = pair_of(__float_as_uint(kRecip127), __float_as_uint(kRecip127));
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              uint32_t o[16], m[8];
              const uint32_t piece = ((2 * quad + h) ^ (row & 7)) << 4;
              load_transposed(from + piece, m);
              load_transposed(from + 32 * kTileW + piece, m + 4);
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const float4 f = *reinterpret_cast<const float4*>(sc + 16 * i);
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                  const uint32_t x = m[2 * i + j] ^ 0x80808080u;
                  const uint64_t scale2 = j ? pair_of(__float_as_uint(f.z), __float_as_uint(f.w))
                                            : pair_of(__float_as_uint(f.x), __float_as_uint(f.y));
#pragma unroll
                  for (int c = 0; c < 2; ++c) {
                    // 2^23 + (code + 128), exactly
                    const uint64_t u = pair_of(__byte_perm(x, 0x4B000000u, c ? 0x7651 : 0x7650),
                                               __byte_perm(x, 0x4B000000u, c ? 0x7653 : 0x7652));
                    const uint64_t w = mul_pair(mul_pair(add_pair(u, off), scale2), r127);
                    o[4 * i + 2 * c + j] = pack2<kOut>(__uint_as_float(uint32_t(w)),
                                                       __uint_as_float(uint32_t(w >> 32)));
                  }
                }
              }
              tmem_st_16(to + (uint32_t(16 * h) << 16), o);
            }
          } else {
            uint32_t o[32];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const uint4 w = lds_v4(raw + r * kStage + (((4 * sub + c) ^ (r & 7)) << 4));
              codes_f16(w.x, o[8 * c], o[8 * c + 1]);
              codes_f16(w.y, o[8 * c + 2], o[8 * c + 3]);
              codes_f16(w.z, o[8 * c + 4], o[8 * c + 5]);
              codes_f16(w.w, o[8 * c + 6], o[8 * c + 7]);
            }
            tmem_st<32>(to, o);
          }
        }
        if constexpr (kBack) scale_turn ^= 1;
        asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
        asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(w_full(wp.slot));
          mbar_arrive(raw_empty(rp.slot));
        }
      }
    }
  } else {
    // ---- finished tiles: lane = weight row (column), 32 columns of activation rows at a time
    constexpr int kHalf = BX / 2, kChunks = kHalf / 32;
    const int quad = warp & 3, half = (warp - kProducers) >> 2;
    const bool f32 = p.out_dtype == DQ4_OUT_F32, bf16 = p.out_dtype == DQ4_OUT_BF16;
    // the column of this lane (see the gradient's values above)
    const int column = quad * 32 + (kBack ? (lane & 16) + (lane & 7) * 2 + (lane >> 3 & 1) : lane);
    // two lanes exchange a value, so that a store takes four bytes
    constexpr int kNext = kBack ? 8 : 1;
    const bool pairs = !f32 && p.lanes % 2 == 0 && (reinterpret_cast<uintptr_t>(p.out) & 3) == 0;
    int turn = 0, g = 0;
    Item it;
    for (int64_t walk = walk0; next_item(walk, it); ++turn) {
      const int buffer = turn % kBuffers;
      const int64_t n = it.lane0 + column, m0 = it.row0 + half * kHalf;
      const int reader = tid - 32 * kProducers;
      float scale = 1.f, bias = 0.f, unit = 0.f;
      if constexpr (!kBack) {
        if (n < p.lanes) {
          scale = load_global(p.SCB + n) * kRecip127;
          if (p.bias) bias = load_any(p.bias, n, p.out_dtype);
        }
        if (reader < BX && it.row0 + reader < p.rows)
          unit = load_global(p.row_units + it.row0 + reader);
      }
      const bool ok = !*aborted && mbar_wait(acc_full(buffer), uint32_t(turn / kBuffers) & 1u) &&
                      !*aborted;
      if (!all_readers(ok)) {
        if (!ok && lane == 0 && !*aborted) fail();
        break;
      }
      if constexpr (!kBack) {
        if (reader < BX) s_unit[reader] = unit;
        bar_readers();
      }
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      const uint32_t at = tmem + (uint32_t(quad * 32) << 16) + buffer * BX + half * kHalf;
      // the accumulators that have a stage of the item: the first stage's issuer, and with
      // two stages both
      const int first = kIssuers > 1 ? g & 1 : 0;
      const bool both = kIssuers > 1 && it.end - it.begin > 1;
      g += it.end - it.begin;
      auto read = [&](int c, uint32_t (&v)[32]) {
        tmem_ld32(at + first * kBuffers * BX + 32 * c, v);
        if (kIssuers > 1 && both) {
          uint32_t w[32];
          tmem_ld32(at + (first ^ 1) * kBuffers * BX + 32 * c, w);
#pragma unroll
          for (int j = 0; j < 32; ++j)
            v[j] = __float_as_uint(__uint_as_float(v[j]) + __uint_as_float(w[j]));
        }
      };
      auto release = [&] {
        asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
        __syncwarp();
        if (lane == 0) mbar_arrive(acc_empty(buffer));
      };
      // Columns (activation rows) from `col` on: finished, in the output's type, two in a word, and
      // stored (rows of them that are there: none for a lane past the last).
      auto finish = [&](auto& v, int col) {
        if constexpr (!kBack) {
#pragma unroll
          for (int j = 0; j < int(sizeof(v) / 4); j += 4) {
            const float4 u = *reinterpret_cast<const float4*>(s_unit + col + j);
            const float by[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int k = 0; k < 4; ++k)
              // (the weight's scale first: rows may be near FP32's largest number)
              v[j + k] = __float_as_uint(__uint_as_float(v[j + k]) * scale * by[k] + bias);
          }
        }
      };
      auto pack = [&](auto& v, int col, uint32_t* to) {
        finish(v, col);
#pragma unroll
        for (int j = 0; j < int(sizeof(v) / 4); j += 2) {
          const float a = __uint_as_float(v[j]), b = __uint_as_float(v[j + 1]);
          to[j / 2] = bf16 ? pack2<DQ4_OUT_BF16>(a, b) : pack2<DQ4_OUT_F16>(a, b);
        }
      };
      auto rows_at = [&](int col, int most) {
        return n < p.lanes ? int(min(int64_t(most), p.rows - it.row0 - col)) : 0;
      };
      auto store = [&](auto& from, int col, int at) {  // (words from `at` on: 32 columns or all)
        constexpr int kWords = int(sizeof(from) / 4) < 16 ? int(sizeof(from) / 4) : 16;
        const int rows = rows_at(col, 2 * kWords);
        if (pairs) {
          const int odd = column & 1;
          uint16_t* to = static_cast<uint16_t*>(p.out) + (it.row0 + col + odd) * p.lanes + n - odd;
#pragma unroll
          for (int j = 0; j < kWords; ++j, to += 2 * p.lanes) {
            const uint32_t other = __shfl_xor_sync(kAllLanes, from[at + j], kNext);
            const uint32_t v = odd ? __byte_perm(other, from[at + j], 0x7632)
                                   : __byte_perm(from[at + j], other, 0x5410);
            if (2 * j + odd < rows) *reinterpret_cast<uint32_t*>(to) = v;
          }
        } else {
          uint16_t* to = static_cast<uint16_t*>(p.out) + (it.row0 + col) * p.lanes + n;
#pragma unroll
          for (int j = 0; j < kWords; ++j, to += 2 * p.lanes) {
            if (2 * j < rows) to[0] = uint16_t(from[at + j]);
            if (2 * j + 1 < rows) to[p.lanes] = uint16_t(from[at + j] >> 16);
          }
        }
      };
      auto put = [&](auto& v, int col) {
        constexpr int kColumns = int(sizeof(v) / 4);
        if (f32) {
          finish(v, col);
          const int rows = rows_at(col, kColumns);
          float* to = static_cast<float*>(p.out) + (it.row0 + col) * p.lanes + n;
#pragma unroll
          for (int j = 0; j < kColumns; ++j, to += p.lanes)
            if (j < rows) *to = __uint_as_float(v[j]);
        } else {
          uint32_t keep[kColumns / 2];
          pack(v, col, keep);
          store(keep, col, 0);
        }
      };
      if (p.cluster > 1) {
        // The CTA's only item: its accumulator goes into its rings, which are idle.  Each CTA then
        // adds and stores an equal share of the columns, eight at a time.
        uint32_t to = sbase + ((half * (kHalf / 4)) * kTileW + quad * 32 + lane) * 16;
#pragma unroll 1
        for (int c = 0; c < kChunks; ++c) {
          uint32_t v[32];
          read(c, v);
#pragma unroll
          for (int j = 0; j < 8; ++j, to += kTileW * 16)
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};"
                         :: "r"(to), "r"(v[4 * j]), "r"(v[4 * j + 1]), "r"(v[4 * j + 2]),
                            "r"(v[4 * j + 3]) : "memory");
        }
        __syncwarp();
        if (lane < p.cluster) arrive_cluster(of_cta(shared, lane));
        const bool there = mbar_wait(shared, 0) && !*aborted;
        see_cluster(shared, 0);
        if (!__all_sync(kAllLanes, there)) {
          if (lane == 0 && !*aborted) fail();
          break;
        }
        const int each = BX / p.cluster;
#pragma unroll 1
        for (int col = rank * each + half * 8; col < (rank + 1) * each; col += 16) {
          const uint32_t from = sbase + (col / 4 * kTileW + quad * 32 + lane) * 16;
          uint32_t v[8];
          float sum[8] = {};
#pragma unroll 1
          for (int r = 0; r < p.cluster; ++r) {
            const uint32_t there = of_cta(from, r);
            load_cluster(there, v);
            load_cluster(there + kTileW * 16, v + 4);
#pragma unroll
            for (int j = 0; j < 8; ++j) sum[j] += __uint_as_float(v[j]);
          }
          memcpy(v, sum, sizeof(v));
          put(v, col);
        }
        break;
      }
      const bool whole = it.begin == 0 && it.end == stages;
      if (whole && !f32) {
        // all of the tile to registers, so that the next one can start, then the stores
        uint32_t keep[kHalf / 2];
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
          uint32_t v[32];
          read(c, v);
          pack(v, half * kHalf + 32 * c, keep + 16 * c);
        }
        release();
#pragma unroll
        for (int c = 0; c < kChunks; ++c) store(keep, half * kHalf + 32 * c, 16 * c);
        continue;
      }
      // (What follows runs once or twice in a CTA: loops, as code that is fetched for the first
      // time takes longer than its instructions.  Unrolled, a join of three 64 KB parts took 14
      // us.)
      // ---- a part of the sum (the CTA's first if the tile began before it, else its last); the
      // last of a tile's parts adds them, in their order
      auto part_at = [&](int64_t cta, int which) {
        return p.part + ((cta * 2 + which) * (BX / 4) + half * (kHalf / 4)) * kTileW + quad * 32 +
               lane;
      };
      const int64_t cta0 = whole ? 0 : cta_of(it.tile * stages);
      const int64_t cta1 = whole ? 0 : cta_of((it.tile + 1) * stages - 1);
      const int sharers = int(cta1 - cta0) + 1, own = int(blockIdx.x - cta0);
      // The CTA's last item: the rings are idle, and its part can stay in TMEM if the others are
      // there, as they mostly are: they are the first items of their CTAs.
      const bool over = !whole && walk >= walk1;
      bool stays = false;
      if (over) {
        if (tid == 32 * kProducers) s_last = load_acquire(p.count + cta1) == sharers - 1;
        bar_readers();
        stays = s_last;
      }
      if (!whole && !stays) {
        float4* part = part_at(blockIdx.x, it.begin == 0);
#pragma unroll 1
        for (int c = 0; c < kChunks; ++c) {
          uint32_t v[32];
          read(c, v);
#pragma unroll
          for (int j = 0; j < 8; ++j)
            part[(8 * c + j) * kTileW] =
                make_float4(__uint_as_float(v[4 * j]), __uint_as_float(v[4 * j + 1]),
                            __uint_as_float(v[4 * j + 2]), __uint_as_float(v[4 * j + 3]));
        }
        release();
        bar_readers();
        if (tid == 32 * kProducers)
          s_last = atomic_add_acq_rel(p.count + cta1, 1) == sharers - 1;
        bar_readers();
        if (!s_last) continue;
      }
      if (!whole && tid == 32 * kProducers) p.count[cta1] = 0;  // ready for the next call
      // The parts are copied into the idle rings, 32 columns of all of them at a time (which the
      // first reader warp issues), the next ones ahead.
      const int pieces = stays ? sharers - 1 : sharers;
      const bool idle = over && pieces <= S::kPieces;
      const int depth = idle ? S::kPieces / pieces : 1;
      auto copy = [&](int c) {
        const uint32_t bar = piece_full(c % depth);
        if (lane == 0) mbar_expect(bar, pieces * S::kPiece);
        __syncwarp();
        const int i = lane >> 1, h = lane & 1, q = stays && i >= own ? i + 1 : i;
        if (i < pieces)
          asm volatile(
              "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes "
              "[%0], [%1], %2, [%3];"
              :: "r"(sbase + (c % depth * pieces + i) * S::kPiece + h * (S::kPiece / 2)),
                 "l"(p.part + ((cta0 + q) * 2 + (q == 0)) * (BX / 4 * kTileW) +
                     (h * (kHalf / 4) + 8 * c) * kTileW),
                 "r"(S::kPiece / 2), "r"(bar) : "memory");
      };
      if (idle && warp == kProducers) {
        // (the parts were written by ordinary stores, and are read by the copies' own path)
        asm volatile("fence.proxy.async;" ::: "memory");
        for (int c = 0; c < kChunks && c < depth; ++c) copy(c);
      }
      bool here = true;
#pragma unroll 1
      for (int c = 0; c < kChunks; ++c) {
        uint32_t v[32];
        if (whole) {
          read(c, v);
        } else {
          if (idle) here = here && mbar_wait(piece_full(c % depth), uint32_t(c / depth) & 1u);
          uint32_t at = sbase + c % depth * pieces * S::kPiece + half * (S::kPiece / 2) +
                        (quad * 32 + lane) * 16;
          float sum[32] = {};
#pragma unroll 1
          for (int q = 0; q < sharers; ++q) {
            uint32_t more[32];
            if (stays && q == own) {
              read(c, more);
            } else if (idle) {
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                const uint4 w = lds_v4(at + j * kTileW * 16);
                memcpy(&more[4 * j], &w, 16);
              }
              at += S::kPiece;
            } else {
              const float4* from = part_at(cta0 + q, q == 0) + 8 * c * kTileW;
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                const float4 w = load_l2(from + j * kTileW);
                memcpy(&more[4 * j], &w, 16);
              }
            }
#pragma unroll
            for (int j = 0; j < 32; ++j) sum[j] += __uint_as_float(more[j]);
          }
          memcpy(v, sum, sizeof(v));
          if (idle && c + depth < kChunks) {  // their place, for later ones
            bar_readers();
            if (warp == kProducers) copy(c + depth);
          }
        }
        put(v, half * kHalf + 32 * c);
      }
      if (whole) release();
      if (!here && lane == 0) fail();
    }
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  if (p.cluster > 1) sync_cluster();  // (nothing of this CTA is read any more)
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;"
                 :: "r"(tmem), "r"(kTmemColumns));
  }
}

// ------------------------------------------------------------ rows in FP16 for the product
struct RowArgs {
  const int8_t* codes;
  const float* scales;
  int64_t M, K, width;   // width: of a row in FP16
  int64_t codes_end;     // where the outliers' second terms start in it
  int64_t row_ctas;
  const int8_t* CB;
  int64_t N;
  const int64_t* cols;
  const void* outliers;
  int L;
  bool bf16;
  uint16_t* X;     // [M][width]
  float* units;    // [M]
  int8_t* columns; // [N][width - codes_end] the weight's columns of the outliers' second terms
  int* count;      // [counts] the product's counters, to be cleared
  int counts;
  int* bad;
};

// A row's FP16 values are its codes, times the row's unit u = scale / 127.  An outlier x takes the
// place of its code as x / u, in two FP16 terms, the second in a column of its own past K, where
// the weight's column stands again: the CTAs past row_ctas gather those columns (gathered in the
// product itself, for each tile again, 4096 rows with 13 such columns through 4096 x 11008 took 293
// us; so 274).  FP16 ends at 65504 and 2^-24: where an outlier is above 2^15 u, the unit is 2^e u,
// the least that it is not above 2^15 of, and codes are 2^-e of theirs, exactly up to e = 24.
// A warp takes 512 values of a row, 16 a lane (so spread, 512 rows through 4096 x 4096 take 22.8
// us; 2048 values a warp, loaded at once, 25.4).
constexpr int kRowPart = 512;
__global__ void __launch_bounds__(256) int8_rows_kernel(const RowArgs p) {
  __shared__ int64_t s_most[8];
  __shared__ int s_col[256];  // of entry t, -1 if it is not used
  asm volatile("griddepcontrol.launch_dependents;");
  const int t = threadIdx.x, lane = t & 31;
  if (blockIdx.x == 0)
    for (int i = t; i < p.counts; i += 256) p.count[i] = 0;
  if (p.L > 0) {
    int64_t col = -1;
    // used: in range and above all before it (the largest so far, by warps and then over them)
    const int64_t c = t < p.L ? load_global(p.cols + t) : -1;
    int64_t run = c < p.K ? c : -1;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t up = __shfl_up_sync(kAllLanes, run, o);
      if ((t & 31) >= o && up > run) run = up;
    }
    if ((t & 31) == 31) s_most[t >> 5] = run;
    int64_t top = __shfl_up_sync(kAllLanes, run, 1);
    if ((t & 31) == 0) top = -1;
    __syncthreads();
    for (int w = 0; w < t >> 5; ++w) top = max(top, s_most[w]);
    if (c > top && c < p.K && c >= 0) col = c;
    const int wrong = col < 0 && c != -1;
    s_col[t] = int(col);
    if (blockIdx.x == 0 && wrong && p.bad) atomicAdd(p.bad, 1);
  }
  if (p.L > 0) __syncthreads();
  const int64_t codes_end = p.codes_end;
  if (blockIdx.x >= p.row_ctas) {
    const int64_t extra = p.width - codes_end, pieces = p.N * extra / 16;
    const int64_t step = (gridDim.x - p.row_ctas) * 256;
    for (int64_t i = (blockIdx.x - p.row_ctas) * 256 + t; i < pieces; i += step) {
      const int64_t n = i * 16 / extra;
      const int* cols = s_col + (i * 16 - n * extra);
      uint32_t code[16];
#pragma unroll
      for (int j = 0; j < 16; ++j)
        code[j] = cols[j] >= 0 ? uint8_t(load_global(p.CB + n * p.K + cols[j])) : 0;
      uint32_t o[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        o[j] = code[4 * j] | code[4 * j + 1] << 8 | code[4 * j + 2] << 16 | code[4 * j + 3] << 24;
      *reinterpret_cast<uint4*>(p.columns + i * 16) = make_uint4(o[0], o[1], o[2], o[3]);
    }
    return;
  }
  const int64_t segs = (codes_end + kRowPart - 1) / kRowPart, parts = p.M * segs;
  for (int64_t part = blockIdx.x * 8 + t / 32; part < parts; part += p.row_ctas * 8) {
    const int64_t row = part / segs, k0 = (part - row * segs) * kRowPart;
    const int8_t* from = p.codes + row * p.K;
    uint16_t* to = p.X + row * p.width;
    const int64_t k = k0 + lane * 16;
    uint4 c = make_uint4(0, 0, 0, 0);
    if (k < p.K) c = load_global(reinterpret_cast<const uint4*>(from + k));
    float unit = load_global(p.scales + row) * kRecip127, ratio = 1.f, x[kMaxOutliers / 32] = {};
    if (p.L > 0) {
      uint32_t top = 0;
#pragma unroll
      for (int j = 0; j < kMaxOutliers / 32; ++j) {
        const int l = 32 * j + lane;
        if (s_col[l] >= 0) x[j] = load_16(p.outliers, row * p.L + l, p.bf16);
        top = max(top, __float_as_uint(x[j]) & 0x7FFFFFFFu);
      }
      top = __reduce_max_sync(kAllLanes, top);
      const float most = __uint_as_float(top) * 3.0517578125e-05f;  // 2^-15 of the largest outlier
      if (top >= 0x7F800000u) {
        unit = __uint_as_float(0x7FC00000u);
      } else if (unit == 0.f) {  // (a scale of 0: codes count for nothing)
        unit = fmaxf(most, 1.17549435e-38f);
        ratio = 0.f;
      } else if (fabsf(unit) < most) {
        int e = ilogbf(most) - ilogbf(unit);
        if (fabsf(scalbnf(unit, e)) < most) ++e;
        unit = scalbnf(unit, e);
        ratio = scalbnf(1.f, -e);
      }
    }
    if (k < codes_end) {
      const uint32_t* w = reinterpret_cast<const uint32_t*>(&c);
      uint32_t o[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) codes_f16(w[j], o[2 * j], o[2 * j + 1]);
      if (ratio != 1.f) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          __half2 h;
          memcpy(&h, &o[j], 4);
          o[j] = pack2<DQ4_OUT_F16>(__low2float(h) * ratio, __high2float(h) * ratio);
        }
      }
      uint4* y = reinterpret_cast<uint4*>(to + k);
      y[0] = make_uint4(o[0], o[1], o[2], o[3]);
      y[1] = make_uint4(o[4], o[5], o[6], o[7]);
    }
    if (lane == 0 && k0 == 0) p.units[row] = unit;
    if (p.L > 0) {
      __syncwarp();  // the codes are there
#pragma unroll
      for (int j = 0; j < kMaxOutliers / 32; ++j) {
        const int l = 32 * j + lane, col = s_col[l];
        const float v = col >= 0 ? __fdiv_rn(x[j], unit) : 0.f;
        const __half high = __float2half_rn(v);
        if (col >= k0 && col < k0 + kRowPart) to[col] = __half_as_ushort(high);
        if (k0 == 0 && codes_end + l < p.width)
          to[codes_end + l] = __half_as_ushort(__float2half_rn(v - __half2float(high)));
      }
    }
  }
}

// ------------------------------------------------------------------------ host side
int64_t up256(int64_t n) { return (n + 255) / 256 * 256; }

struct Plan {
  int bx, stages;
  int64_t tiles_x, tiles;
  int ctas;
  bool split;   // equal runs of stages, else whole tiles,
  int cluster;  // by so many CTAs each
};

// The tile's width, and whether CTAs take whole tiles, a tile by clusters of 2, 4 or 8, or equal
// runs of stages over all tiles, by the estimated time in cycles, from measured ones: a stage takes
// 840, 890 and 1350 at BX 64, 128 and 256 (of 8 MMAs; the gradient's 1270, 1310 and 1600), the end
// of a tile 1500 where its accumulator is the only one.  A cluster's exchange costs 2500, 300 a CTA
// and 40 a column; runs cost 12000, the parts' writing, counting and joining, and a part's bytes by
// the CTAs that share a tile, which are more, and have no whole tile, where a run is shorter than a
// tile.  In us, whole / clusters / runs: 64 rows through 4096 x 11008 20.4 / - / 21.3, through 4096
// x 4096 19.0 / 12.1 / 15.7, 14336 to 4096 54 / 22.4 / 24.8; 512 through 4096 x 11008, 256 wide, 56
// / - / 44.5; 256 rows' gradient through 11008 x 4096, 256 wide, 76 / 29.6 / 38.5.
Plan plan_gemm(int64_t lanes, int64_t rows, int steps, bool back, int sms) {
  Plan best = {};
  double best_cost = 1e300;
  const int stages = (steps + 1) / 2;
  for (int bx = 64; bx <= 256; bx *= 2) {
    const int64_t tiles_x = (rows + bx - 1) / bx;
    const int64_t tiles = tiles_x * ((lanes + kTileW - 1) / kTileW);
    const double stage = back ? (bx == 64 ? 1270 : bx == 128 ? 1310 : 1600)
                              : (bx == 64 ? 840 : bx == 128 ? 890 : 1350);
    const double end = bx == 64 ? 200 : 1500;
    double cost = double((tiles + sms - 1) / sms) * (stages * stage + end);
    if (cost < best_cost) {
      best_cost = cost;
      best = {bx, stages, tiles_x, tiles, int(tiles < sms ? tiles : sms), false, 1};
    }
    // (76 clusters of two run at once, 32 of four, fewer than 16 of eight)
    for (int c = 2; c <= 8 && c <= stages; c *= 2) {
      if (tiles * c > (c == 2 ? sms : c == 4 ? sms * 27 / 32 : sms / 2)) continue;
      cost = (stages + c - 1) / c * stage + end + 2500 + 300 * c + 40 * bx;
      if (cost < best_cost) {
        best_cost = cost;
        best = {bx, stages, tiles_x, tiles, int(tiles) * c, false, c};
      }
    }
    const int64_t units = tiles * stages;
    const int ctas = int(units < sms ? units : sms);
    const double run = double(units) / ctas, sharers = stages / run + 1;
    cost = run * stage + (run / stages + 1) * end + 12000 +
           bx * (9 * sharers + (run < stages ? 25 : 0));
    if (cost < best_cost) {
      best_cost = cost;
      best = {bx, stages, tiles_x, tiles, ctas, true, 1};
    }
  }
  return best;
}

template <int BX, bool kBack, bool kBF16>
int launch_one(const CUtensorMap& w, const CUtensorMap& x, const CUtensorMap& cols,
               const GemmArgs& p, int dev, int ctas, cudaStream_t stream) {
  auto kernel = dq4_int8_gemm_kernel<BX, kBack, kBF16>;
  static std::atomic<uint64_t> allowed{0};
  if (const int st = allow_smem(kernel, Gemm<BX, kBack>::kBytes, dev, &allowed)) return st;
  return launch_clusters(kernel, dim3(unsigned(ctas)), Gemm<BX, kBack>::kThreads,
                         Gemm<BX, kBack>::kBytes, stream, p.cluster, w, x, cols, p);
}

template <bool kBack, bool kBF16>
int launch_plan(const Plan& pl, const CUtensorMap& w, const CUtensorMap& x,
                const CUtensorMap& cols, GemmArgs p, int dev, void* part, cudaStream_t stream) {
  p.tiles_x = int(pl.tiles_x);
  p.tiles = pl.tiles;
  p.units = pl.split ? pl.tiles * pl.stages : 0;
  p.cluster = pl.cluster;
  p.part = static_cast<float4*>(part);
  if (pl.bx == 64) return launch_one<64, kBack, kBF16>(w, x, cols, p, dev, pl.ctas, stream);
  if (pl.bx == 128) return launch_one<128, kBack, kBF16>(w, x, cols, p, dev, pl.ctas, stream);
  return launch_one<256, kBack, kBF16>(w, x, cols, p, dev, pl.ctas, stream);
}

// The steps of a row in FP16: of its codes, and of its outliers' second terms.
// (with outliers the codes end with a stage: its codes come from one matrix)
int k_steps(int64_t K) { return int((K + kStep - 1) / kStep); }
int code_steps(int64_t K, int L) { return L > 0 ? (k_steps(K) + 1) / 2 * 2 : k_steps(K); }
int all_steps(int64_t K, int L) { return code_steps(K, L) + k_steps(L); }

// The counters of parts that the product uses.  A call that completes leaves them at 0; they are
// cleared all the same, so that one whose waits ran out costs nothing but its own results.
int counters(const Plan& pl) { return pl.split ? pl.ctas : 0; }

int64_t part_bytes(const Plan& pl) {
  return pl.split ? int64_t(pl.ctas) * 2 * pl.bx * kTileW * 4 : 0;
}

}  // namespace

int64_t int8_gemm_workspace(int64_t M, int64_t N, int64_t K, int L, int sms) {
  const Plan pl = plan_gemm(N, M, all_steps(K, L), false, sms);
  return kInt8Counters + up256(N * k_steps(L) * kStep) + up256(M * 4) +
         up256(M * all_steps(K, L) * kStep * 2) + part_bytes(pl);
}

int launch_int8_gemm(const Int8Linear& a, int dev, int sms, void* workspace, cudaStream_t stream) {
  const int steps = all_steps(a.K, a.L);
  const Plan pl = plan_gemm(a.N, a.M, steps, false, sms);
  char* at = static_cast<char*>(workspace);
  int* count = reinterpret_cast<int*>(at);
  at += kInt8Counters;
  int8_t* columns = reinterpret_cast<int8_t*>(at);
  const int64_t extra = k_steps(a.L) * kStep;
  at += up256(a.N * extra);
  float* units = reinterpret_cast<float*>(at);
  at += up256(a.M * 4);
  uint16_t* X = reinterpret_cast<uint16_t*>(at);
  const int64_t width = int64_t(steps) * kStep;
  at += up256(a.M * width * 2);
  CUtensorMap w, x, cols;
  if (const int st = encode_2d(&w, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.CB, a.K, a.N, a.K, kStage,
                               kTileW, CU_TENSOR_MAP_SWIZZLE_128B))
    return st;
  cols = w;  // (not read without outliers)
  if (a.L > 0)
    if (const int st = encode_2d(&cols, CU_TENSOR_MAP_DATA_TYPE_UINT8, columns, extra, a.N, extra,
                                 kStage, kTileW, CU_TENSOR_MAP_SWIZZLE_128B))
      return st;
  if (const int st = encode_2d(&x, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, X, width, a.M, width * 2, kStep,
                               pl.bx, CU_TENSOR_MAP_SWIZZLE_128B))
    return st;
  RowArgs r = {};
  r.codes = a.codes;
  r.scales = a.scales;
  r.M = a.M;
  r.K = a.K;
  r.width = width;
  r.codes_end = int64_t(code_steps(a.K, a.L)) * kStep;
  const int64_t parts = (r.codes_end + kRowPart - 1) / kRowPart * a.M;
  r.row_ctas = (parts + 7) / 8 < 8 * sms ? (parts + 7) / 8 : 8 * sms;
  r.CB = a.CB;
  r.N = a.N;
  r.cols = a.cols;
  r.outliers = a.outliers;
  r.L = a.L;
  r.bf16 = a.outliers_bf16;
  r.X = X;
  r.units = units;
  r.columns = columns;
  r.count = count;
  r.counts = counters(pl);
  r.bad = a.bad;
  const int64_t gathers = (a.N * extra / 16 + 255) / 256;
  const int64_t row_kernel_ctas = r.row_ctas + (gathers < 4 * sms ? gathers : 4 * sms);
  // In full stream order: launched early, its CTAs gather on the SMs that the kernel before leaves
  // first (512 rows with 13 outlier columns through 4096 x 11008: 55.4 us, so 47.5).
  int8_rows_kernel<<<unsigned(row_kernel_ctas), 256, 0, stream>>>(r);
  if (const cudaError_t e = cudaGetLastError()) return fail_cuda(DQ4_ERR_LAUNCH, e);
  GemmArgs p = {};
  p.lanes = p.N = a.N;
  p.rows = a.M;
  p.steps = steps;
  p.code_steps = code_steps(a.K, a.L);
  p.SCB = a.SCB;
  p.row_units = units;
  p.bias = a.bias;
  p.out_dtype = a.out_dtype;
  p.out = a.Y;
  p.count = count;
  p.bad = a.bad;
  return launch_plan<false, false>(pl, w, x, cols, p, dev, at, stream);
}

int64_t int8_backward_workspace(int64_t M, int64_t N, int64_t K, int sms) {
  return kInt8Counters + part_bytes(plan_gemm(K, M, k_steps(N), true, sms));
}

int launch_int8_backward(const Int8Backward& a, int dev, int sms, void* workspace,
                         cudaStream_t stream) {
  const Plan pl = plan_gemm(a.K, a.M, k_steps(a.N), true, sms);
  CUtensorMap w, x;
  if (const int st = encode_2d(&w, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.CB, a.K, a.N, a.K, kTileW,
                               kStage, CU_TENSOR_MAP_SWIZZLE_128B))
    return st;
  if (const int st = encode_2d(&x, a.bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                          : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                               a.dY, a.N, a.M, a.N * 2, kStep, pl.bx, CU_TENSOR_MAP_SWIZZLE_128B))
    return st;
  GemmArgs p = {};
  p.lanes = a.K;
  p.N = a.N;
  p.rows = a.M;
  p.steps = p.code_steps = k_steps(a.N);
  p.SCB = a.SCB;
  p.out_dtype = a.bf16 ? DQ4_OUT_BF16 : DQ4_OUT_F16;
  p.out = a.dX;
  p.count = static_cast<int*>(workspace);
  p.bad = a.bad;
  char* part = static_cast<char*>(workspace) + kInt8Counters;
  if (pl.split)
    if (const cudaError_t e = cudaMemsetAsync(p.count, 0, size_t(counters(pl)) * 4, stream))
      return fail_cuda(DQ4_ERR_LAUNCH, e);
  return a.bf16 ? launch_plan<true, true>(pl, w, x, w, p, dev, part, stream)
                : launch_plan<true, false>(pl, w, x, w, p, dev, part, stream);
}

}  // namespace dq4d
