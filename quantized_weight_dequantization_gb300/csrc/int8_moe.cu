// A mixture-of-experts layer for few tokens over 8-bit weights: dq4_int8_moe (dq4_int8.h).
//
// Bound by the bytes of the chosen experts' weights, each read once.  Four launches:
//   route   a CTA a token: each chooses all tokens' experts, brings its own token's row to FP16,
//           scaled by a power of two, and puts it at the places of its choices; the first lists
//           each expert's (token, choice) pairs, by entries of up to 8
//   up      a job is 16 inner places of an entry's expert, gate and up rows together: inner =
//           silu(g) * u in FP32, and the largest of each pair's row
//   down    a job is 32 output places of an entry's expert; inner values become two terms of FP16
//           on their way in, in units of a power of two for their row.  That holds 22 bits of a
//           value, or 2^-39 of its row's largest, where FP16 ends.  (One term's 11 bits are as much
//           as FP16 results have, and move one BF16 result in ten to its neighbour.  A power of two
//           for each 16 places, brought to the row's in FP16, lost what is below 2^-25 of the row.)
//   combine each token's results by their weights
// Experts that no token chose have no jobs.  No atomic adds a value.
//
// Of 4096 x 14336: one token through 2 of 8 experts 73.5 us, where the bytes take 52, 23 tokens 255
// of 208; of 2048 x 1408, 16 tokens through 6 of 64, 96 of 65.  What is left is the ends of the
// four launches, about 4 us each, and the second product, which for one token ran at 0.68 of the
// copy rate with one term, where the first runs at 0.83.
#include "int8.cuh"

namespace dq4d {
namespace {

constexpr int kRouteThreads = 512;
constexpr int kMaxTokens = 256, kMaxExperts = 1024, kMaxTopK = 16;
constexpr int kMaxPairs = kMaxTokens * kMaxTopK;
constexpr int kEntry = 8;  // pairs of an entry at most
constexpr int kMaxEntries = kMaxExperts + kMaxPairs / kEntry;
constexpr int kUpPlaces = 16, kDownPlaces = 32;
constexpr int64_t kMaxInner = 1 << 20;
constexpr int64_t kMaxHidden = 1 << 15;

// What `route` finds out, at the head of the workspace.  Pairs (token, choice) stand in the order
// of their experts: `place` is a pair's there, and rows of xs, inner and out are by place.
struct Routed {
  int entries;                      // experts with pairs, one for each 8 of them
  uint16_t expert[kMaxEntries];     // of each
  uint16_t first[kMaxEntries + 1];  // and its first place
  uint16_t place[kMaxPairs];        // of token * top_k + choice
  uint32_t top[kMaxPairs];          // bits of the largest |inner value| of a place
  float down[kMaxPairs];            // what a place's FP16 token has to be multiplied by
};

struct MoeArgs {
  const void* X;
  int64_t row_stride;
  bool bf16;
  int T, E, top_k, renormalize;
  int64_t H, I;
  const float* logits;
  const int8_t *W1, *W2;
  const float *S1, *S2;
  int32_t* ids;
  float* weights;
  void* Y;
  Routed* r;
  uint16_t* xs;     // [pairs][H] FP16
  float* inner;     // [pairs][I in whole chunks], see inner_at
  float* out;       // [pairs][H]
  int* bad;
};

// The power of two that brings magnitudes up to `top` into FP16's upper range, and its inverse
// (NaN if top is not finite).
__device__ __forceinline__ void pow2_scaling(float top, float& up, float& down) {
  const int e = int(__float_as_uint(top) >> 23);  // biased; 0 also for subnormal rows
  const int k = min(max(14 - (e - 127), -126), 126);
  up = __uint_as_float(uint32_t(k + 127) << 23);
  down = __uint_as_float(uint32_t(127 - k) << 23);
  if (!(top < INFINITY)) down = __uint_as_float(0x7FC00000u);
}

// ------------------------------------------------------------------------- route
// Logits as integers in their order, 0 for one that was chosen (-infinity and NaN: 0x7FFFFF).
__device__ __forceinline__ uint32_t order_key(float x) {
  if (x != x) x = -INFINITY;
  const uint32_t b = __float_as_uint(x + 0.f);  // (-0 is 0)
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ float logit_of(uint32_t key) {
  return __uint_as_float(key & 0x80000000u ? key & 0x7FFFFFFFu : ~key);
}

// Every CTA finds out the whole routing for itself (the warps' tokens side by side, so that it
// takes no longer than one token's); CTA t then writes token t's row, and CTA 0 the lists.
__global__ void __launch_bounds__(kRouteThreads) dq4_moe_route_kernel(const MoeArgs p) {
  __shared__ uint16_t s_ids[kMaxPairs];
  __shared__ int s_count[kMaxExperts];
  __shared__ uint32_t s_sums[kRouteThreads / 32];
  __shared__ int s_place[kMaxTopK];
  extern __shared__ uint32_t s_keys[];  // [kRouteThreads / 32][E]
  wait_for_stream();
  asm volatile("griddepcontrol.launch_dependents;");
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  const int pairs = p.T * p.top_k, mine0 = blockIdx.x * p.top_k;
  const bool lists = blockIdx.x == 0;
  // ---- this CTA's token: its largest value, for later
  const uint16_t* x = static_cast<const uint16_t*>(p.X) + blockIdx.x * p.row_stride;
  uint32_t largest = 0;
  for (int64_t i = t * 8; i < p.H; i += kRouteThreads * 8) {
    const uint4 v = load_global(reinterpret_cast<const uint4*>(x + i));
    const uint32_t m = __vmaxu2(__vmaxu2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu),
                                __vmaxu2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu));
    largest = max(largest, max(m & 0xFFFFu, m >> 16));
  }
  // ---- the experts of each token, a warp a token
  for (int e = t; e < kMaxExperts; e += kRouteThreads) s_count[e] = 0;
  for (int token = warp; token < p.T; token += kRouteThreads / 32) {
    const float* row = p.logits + int64_t(token) * p.E;
    uint32_t* key = s_keys + warp * p.E;
    bool nan = false;
    for (int e = lane; e < p.E; e += 32) {
      const float l = load_global(row + e);
      nan |= l != l;
      key[e] = order_key(l);
    }
    nan = __any_sync(kAllLanes, nan);
    __syncwarp();
    float top = 0.f, sum = 0.f;
    if (lists && !p.renormalize) {
      uint32_t best = 0;
      for (int e = lane; e < p.E; e += 32) best = max(best, key[e]);
      top = logit_of(__reduce_max_sync(kAllLanes, best));
      for (int e = lane; e < p.E; e += 32) sum += expf(logit_of(key[e]) - top);
    }
    int mine = 0;  // lane j: the j-th choice
    float l = -INFINITY;
    for (int j = 0; j < p.top_k; ++j) {
      uint32_t best = 0;
      int at = 0;
      for (int e = lane; e < p.E; e += 32)
        if (key[e] > best) {
          best = key[e];
          at = e;
        }
      const uint32_t most = __reduce_max_sync(kAllLanes, best);
      const int e = __reduce_min_sync(kAllLanes, best == most ? unsigned(at) : 0xFFFFFFFFu);
      if (j == 0) top = logit_of(most);
      if (lane == j) {
        mine = e;
        l = logit_of(most);
      }
      if (lane == 0) key[e] = 0;
      __syncwarp();
    }
    if (lane < p.top_k) s_ids[token * p.top_k + lane] = uint16_t(mine);
    if (lists) {
      const float part = top == -INFINITY || lane >= p.top_k ? 0.f : expf(l - top);
      if (p.renormalize) sum = part;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kAllLanes, sum, o);
      float weight = top == -INFINITY ? 0.f : __fdiv_rn(part, sum);
      if (nan) weight = __uint_as_float(0x7FC00000u);
      if (lane < p.top_k) {
        p.ids[token * p.top_k + lane] = mine;
        p.weights[token * p.top_k + lane] = weight;
      }
    }
    __syncwarp();
  }
  if (lists)
    for (int i = t; i < pairs; i += kRouteThreads) p.r->top[i] = 0;
  largest = __reduce_max_sync(kAllLanes, largest);
  if (lane == 0) s_sums[warp] = largest;
  __syncthreads();
  largest = __reduce_max_sync(kAllLanes, lane < kRouteThreads / 32 ? s_sums[lane] : 0);
  // ---- each expert's pairs, in the order of the tokens
  for (int i = t; i < pairs; i += kRouteThreads) atomicAdd(s_count + s_ids[i], 1);
  __syncthreads();
  // pairs, and entries, before this thread's experts (both below 2^16)
  constexpr int kEach = kMaxExperts / kRouteThreads;
  uint32_t both = 0;
  int counts[kEach];
#pragma unroll
  for (int k = 0; k < kEach; ++k) {
    counts[k] = s_count[t * kEach + k];
    both += uint32_t(counts[k]) | uint32_t((counts[k] + kEntry - 1) / kEntry) << 16;
  }
  uint32_t run = both;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t up = __shfl_up_sync(kAllLanes, run, o);
    if (lane >= o) run += up;
  }
  if (lane == 31) s_sums[warp] = run;
  __syncthreads();
  uint32_t at = run - both, all = 0;
  for (int w = 0; w < kRouteThreads / 32; ++w) {
    if (w < warp) at += s_sums[w];
    all += s_sums[w];
  }
  int entry = at >> 16, first = at & 0xFFFF;
#pragma unroll
  for (int k = 0; k < kEach; ++k) {
    const int e = t * kEach + k;
    s_count[e] = first;  // (from here on: the expert's first place)
    if (lists)
      for (int done = 0; done < counts[k]; done += kEntry, ++entry) {
        p.r->expert[entry] = uint16_t(e);
        p.r->first[entry] = uint16_t(first + done);
      }
    first += counts[k];
  }
  if (lists && t == 0) {
    p.r->entries = int(all >> 16);
    p.r->first[all >> 16] = uint16_t(pairs);
  }
  float up, down;
  pow2_scaling(p.bf16 ? __uint_as_float(largest << 16)
                      : __half2float(__ushort_as_half(uint16_t(largest))), up, down);
  __syncthreads();
  // a choice's place: behind the pairs of its expert from tokens before (a warp a choice)
  for (int j = warp; j < p.top_k; j += kRouteThreads / 32) {
    const int e = s_ids[mine0 + j];
    int before = 0;
    for (int i = lane; i < mine0; i += 32) before += s_ids[i] == e;
    before = __reduce_add_sync(kAllLanes, before);
    if (lane == 0) {
      const int place = s_count[e] + before;
      s_place[j] = place;
      p.r->place[mine0 + j] = uint16_t(place);
      p.r->down[place] = down;
    }
  }
  __syncthreads();
  // ---- the token's row in FP16, at the places of its choices
  for (int64_t i = t * 8; i < p.H; i += kRouteThreads * 8) {
    const uint4 v = load_global(reinterpret_cast<const uint4*>(x + i));
    const uint32_t* w = reinterpret_cast<const uint32_t*>(&v);
    uint32_t o[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float a, b;
      if (p.bf16) {
        a = __uint_as_float(w[j] << 16);
        b = __uint_as_float(w[j] & 0xFFFF0000u);
      } else {
        __half2 h;
        memcpy(&h, &w[j], 4);
        a = __low2float(h);
        b = __high2float(h);
      }
      o[j] = pack2<DQ4_OUT_F16>(a * up, b * up);
    }
    for (int j = 0; j < p.top_k; ++j)
      *reinterpret_cast<uint4*>(p.xs + int64_t(s_place[j]) * p.H + i) =
          make_uint4(o[0], o[1], o[2], o[3]);
  }
}

// ------------------------------------------------ products of weight rows and an entry's tokens
// Warps take jobs (32 weight rows, up to 8 tokens) in turn: alone, or 2, 4 or 8 of a CTA together
// (a group), which then take turns at the chunks of 128 of K and add their sums at the end.  The
// order of K inside a product is free: lane (g, c) = (lane / 4, lane % 4) takes 32 consecutive
// codes of rows g and g + 8 of each 16, and the same places of token g, and eight products take
// them four at a time.  The weights come by TMA into a ring of the warp's own in shared memory, two
// chunks ahead, across the ends of jobs (lane 0 issues, all lanes consume); the tokens, which every
// job of an entry reads, from L2 into registers, while a chunk's weights are waited for (a chunk
// ahead took 1 % more).  Nothing else synchronizes warps before a job's end.  A job starts at a
// chunk of its own, so that warps do not go through the tokens side by side and queue at single
// lines of L2.
// Copies of 128-byte rows: the TMA takes about 3.5 cycles for a row whatever its width, and at 64
// bytes a row that bounds the weight's bytes (one token through 11008 x 4096, whose weight alone
// takes 10.4 us to read: 23.7 us).  Copies of 16 bytes a lane, cp.async, took 13.4 us there.
// Rings of four chunks leave the tokens less of L1: 16 tokens, 6 of 64 experts, took 5 us more.
//
// kBoxes: boxes of weight rows of a chunk.  kTwo: tokens are FP32, and become two terms (23 tokens
// through 2 of 8 experts of 4096 x 14336 254 us; 298 by going through a chunk once for each, with
// half of the registers; 259 where they become that before the weights' wait, which spills; 240
// with one term).
// Jobs:
//   places(job, y)          the first row of each box of weights
//   tokens(job)             this lane's token (for one that is not there any other, whose results
//                           are not used), advanced to its 32 c; its loads are kLoadStep apart
//   unit(job)               with kTwo: what its values are multiplied by, a power of two that
//                           brings them into FP16's upper range
//   begin(job, t)           before a job's products, thread t of its group
//   finish(job, part, ...)  the group's sums (sum(part, warps, token, row)), thread t of `threads`
//
// (Entries of 16 pairs, two products for each weight's conversion, took more: with one term, 64
// tokens through 2 of 8 experts of 4096 x 14336, 16 pairs each, 443 us, in eights, which read the
// weights twice from L2, 409, with two terms 443; 23 tokens 302 and 237.)
constexpr int kJobRows = 32;
constexpr int kDepth = 2;  // chunks of a ring
constexpr int kCtas = 2;   // of an SM

// The warps of a group: of 1, 2, 4 and 8, what takes the fewest chunks in the longest warp, where
// the end of a job costs about as much as 2.
__device__ __forceinline__ int group_warps(uint32_t jobs, uint32_t chunks, uint32_t warps) {
  int best = 1;
  uint32_t least = 0xFFFFFFFFu;
#pragma unroll
  for (int n = 1; n <= kStreamWarps; n *= 2) {
    const uint32_t rounds = (jobs + warps / n - 1) / (warps / n);
    const uint32_t cost = rounds * ((chunks + n - 1) / n + 2);
    if (cost < least) {
      least = cost;
      best = n;
    }
  }
  return best;
}

// Two values times `unit`: in FP16, and what that leaves.
__device__ __forceinline__ void two_terms(uint32_t a, uint32_t b, float unit, uint32_t& high,
                                          uint32_t& low) {
  const uint64_t minus_one = 0xBF800000BF800000ull;
  const uint32_t u = __float_as_uint(unit);
  uint64_t x = uint64_t(b) << 32 | a, left;
  asm("mul.rn.f32x2 %0, %0, %1;" : "+l"(x) : "l"(uint64_t(u) << 32 | u));
  high = pack2<DQ4_OUT_F16>(__uint_as_float(uint32_t(x)), __uint_as_float(uint32_t(x >> 32)));
  __half2 h;
  memcpy(&h, &high, 4);
  const float2 f = __half22float2(h);
  memcpy(&left, &f, 8);
  asm("fma.rn.f32x2 %0, %0, %1, %2;" : "+l"(left) : "l"(minus_one), "l"(x));
  low = pack2<DQ4_OUT_F16>(__uint_as_float(uint32_t(left)), __uint_as_float(uint32_t(left >> 32)));
}

template <int kBoxes, bool kTwo>
struct Streamed {
  using Token = std::conditional_t<kTwo, float, uint16_t>;
  static constexpr int kStage = kJobRows * kChunk;
  static constexpr int kPart = kJobRows * kEntry;  // sums of a warp
  static constexpr int kBarsAt = kStreamWarps * kDepth * kStage;
  static constexpr int kPartsAt = kBarsAt + kStreamWarps * kDepth * 8;
  static constexpr int kBytes = kPartsAt + kStreamWarps * kPart * 4;  // + 1024 to align

  template <typename Jobs>
  static __device__ __forceinline__ void run(Jobs& jobs, uint8_t* smem, int64_t all, int64_t K,
                                             const CUtensorMap& map_w, int* bad) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    const int chunks = int((K + kChunk - 1) / kChunk);
    const int group = group_warps(uint32_t(all), uint32_t(chunks), gridDim.x * kStreamWarps);
    const int in_cta = warp / group, member = warp - in_cta * group;
    const int64_t first = int64_t(blockIdx.x) * (kStreamWarps / group) + in_cta;
    const int64_t stride = int64_t(gridDim.x) * (kStreamWarps / group);
    float* part = reinterpret_cast<float*>(smem + kPartsAt) + in_cta * group * kPart;
    const uint32_t ring = smem_u32(smem) + warp * kDepth * kStage;
    const uint32_t bars = smem_u32(smem) + kBarsAt + warp * kDepth * 8;
    const int mine = chunks > member ? (chunks - member + group - 1) / group : 0;
    const uint64_t tw = reinterpret_cast<uint64_t>(&map_w);
    // ---- the weights' copies: of the next chunk of the next job
    int y[kBoxes];
    int64_t ahead = mine > 0 ? first : all;
    int ahead_chunk = 0, left = mine, slot_in = 0, in_flight = 0;
    auto start_of = [&](int64_t job) { return int(uint32_t(job) % uint32_t(mine)); };
    auto open = [&] {
      if (ahead >= all) return;
      jobs.places(ahead, y);
      ahead_chunk = start_of(ahead);
    };
    open();
    auto issue = [&] {
      if (ahead >= all) return;
      if (lane == 0) {
        const int k = (member + ahead_chunk * group) * kChunk;
        const uint32_t dst = ring + slot_in * kStage, bar = bars + 8 * slot_in;
        mbar_expect(bar, kStage);
#pragma unroll
        for (int i = 0; i < kBoxes; ++i)
          tma_load_2d(dst + i * (kStage / kBoxes), tw, k, y[i], bar);
      }
      ++in_flight;
      if (++slot_in == kDepth) slot_in = 0;
      if (++ahead_chunk == mine) ahead_chunk = 0;
      if (--left == 0) {
        left = mine;
        ahead += stride;
        open();
      }
    };
#pragma unroll 1
    for (int i = 0; i < kDepth; ++i) issue();
    // ---- the tokens, of the next chunk
    constexpr int kLoad = 16 / int(sizeof(Token)), kLoads = 32 / kLoad;  // values of a load
    const Token* tok;
    uint4 x[kLoads];
    float unit = 0.f, next_unit = 0.f;
    int64_t tok_job = mine > 0 ? first : all;
    int tok_chunk = 0, tok_left = mine;
    auto tok_open = [&] {
      if (tok_job >= all) return;
      tok = jobs.tokens(tok_job);
      if constexpr (kTwo) next_unit = jobs.unit(tok_job);
      tok_chunk = start_of(tok_job);
    };
    tok_open();
    auto fetch = [&] {
      if (tok_job >= all) return;
      const int64_t k = int64_t(member + tok_chunk * group) * kChunk;
      unit = next_unit;
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        x[i] = make_uint4(0, 0, 0, 0);  // (past the end)
        if (k + 32 * c + kLoad * i < K)
          x[i] = load_ahead(reinterpret_cast<const uint4*>(tok + k) + Jobs::kLoadStep * i);
      }
      if (++tok_chunk == mine) tok_chunk = 0;
      if (--tok_left == 0) {
        tok_left = mine;
        tok_job += stride;
        tok_open();
      }
    };
    auto join = [&] {  // the group's threads
      if (group == 1)
        __syncwarp();
      else
        asm volatile("bar.sync %0, %1;" :: "r"(1 + in_cta), "r"(32 * group) : "memory");
    };
    int slot = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int64_t job = first; job < all; job += stride) {
      jobs.begin(job, 32 * member + lane);
      constexpr int kTerms = kTwo ? 2 : 1;
      float acc[2][4] = {};
#pragma unroll 1
      for (int i = 0; i < mine && ok; ++i) {
        fetch();
        ok = __all_sync(kAllLanes, mbar_wait(bars + 8 * slot, phase));
        if (!ok) break;
        uint32_t b[kTerms][16];  // the tokens' operand words
#pragma unroll
        for (int s = 0; s < 16; ++s) {
          const uint32_t* w = reinterpret_cast<const uint32_t*>(x);
          if constexpr (kTwo)
            two_terms(w[2 * s], w[2 * s + 1], unit, b[0][s], b[1][s]);
          else
            b[0][s] = w[s];
        }
        const uint32_t at = ring + slot * kStage;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          // 128-byte rows, their 16-byte pieces in place i ^ row % 8
          uint4 w[2][2];
#pragma unroll
          for (int rt = 0; rt < 2; ++rt)
#pragma unroll
            for (int h = 0; h < 2; ++h)
              w[rt][h] = lds_v4(at + (16 * rt + 8 * h + g) * kChunk + (((2 * c + half) ^ g) << 4));
#pragma unroll
          for (int s = 0; s < 4; ++s)
#pragma unroll
            for (int rt = 0; rt < 2; ++rt) {
              uint32_t a[4];
              codes_f16(reinterpret_cast<const uint32_t*>(&w[rt][0])[s], a[0], a[2]);
              codes_f16(reinterpret_cast<const uint32_t*>(&w[rt][1])[s], a[1], a[3]);
#pragma unroll
              for (int t = 0; t < kTerms; ++t)
                mma_16816(acc[rt], a[0], a[1], a[2], a[3], b[t][8 * half + 2 * s],
                          b[t][8 * half + 2 * s + 1]);
            }
        }
        __syncwarp();  // every lane has read the chunk
        --in_flight;
        issue();
        if (++slot == kDepth) {
          slot = 0;
          phase ^= 1u;
        }
      }
      float* to = part + member * kPart;
#pragma unroll
      for (int rt = 0; rt < 2; ++rt)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          to[place(2 * c + (i & 1), 16 * rt + 8 * (i >> 1) + g)] = acc[rt][i];
      join();
      jobs.finish(job, part, group, 32 * member + lane, 32 * group);
      join();  // the sums have been read
    }
    if (!ok) {  // copies in flight land before the CTA leaves
      if (lane == 0 && bad) atomicAdd(bad, 1);
      for (; in_flight > 0; --in_flight) {
        mbar_wait(bars + 8 * slot, phase);
        if (++slot == kDepth) {
          slot = 0;
          phase ^= 1u;
        }
      }
    }
  }

  // The barriers of this warp's ring: before anything else.
  static __device__ __forceinline__ void setup(uint8_t* smem, const CUtensorMap& map_w) {
    if ((threadIdx.x & 31) == 0) {
      asm volatile("prefetch.tensormap [%0];" :: "l"(reinterpret_cast<uint64_t>(&map_w)));
      const uint32_t bars = smem_u32(smem) + kBarsAt + (threadIdx.x >> 5) * kDepth * 8;
      for (int i = 0; i < kDepth; ++i) mbar_init(bars + 8 * i, 1);
      asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncwarp();
  }

  // Where a token's and row's sum lies: the rows of a token in turn, those of every second token
  // 8 further on, so that the lanes that store or read together use different banks.
  static __device__ __forceinline__ int place(int token, int row) {
    return token * kJobRows + (row ^ (token >> 1 & 3) * 8);
  }
  static __device__ __forceinline__ float sum(const float* part, int warps, int token, int row) {
    float v = 0.f;
    for (int w = 0; w < warps; ++w) v += part[w * kPart + place(token, row)];
    return v;
  }
};

// What the other two kernels hold of it in shared memory, behind their rings.
struct Entries {
  float *up, *down;  // of a place's token: xs's `down`, or the scaling of its inner row
  uint16_t *expert, *first;
  int count;
};
int64_t entry_bytes(int64_t entries, int64_t pairs) { return pairs * 8 + entries * 4 + 2; }
int64_t most_entries(int64_t E, int64_t pairs) { return (E < pairs ? E : pairs) + pairs / kEntry; }

template <bool kInner>
__device__ __forceinline__ Entries load_entries(const MoeArgs& p, uint8_t* smem) {
  const int pairs = p.T * p.top_k;
  Entries s;
  s.count = load_global(&p.r->entries);
  s.up = reinterpret_cast<float*>(smem);
  s.down = s.up + pairs;
  for (int i = threadIdx.x; i < pairs; i += blockDim.x) {
    if constexpr (kInner)
      pow2_scaling(__uint_as_float(load_global(p.r->top + i)), s.up[i], s.down[i]);
    else
      s.down[i] = load_global(p.r->down + i);
  }
  s.expert = reinterpret_cast<uint16_t*>(s.down + pairs);
  s.first = s.expert + s.count;
  for (int i = threadIdx.x; i <= s.count; i += blockDim.x) {
    if (i < s.count) s.expert[i] = load_global(p.r->expert + i);
    s.first[i] = load_global(p.r->first + i);
  }
  __syncthreads();
  return s;
}

// Inner values lie as they are read: of a chunk lane c's i-th four, 32 c + 4 i, stand beside those
// of the other lanes, so that a load takes one line of a token.  (In their own order it took four,
// and 23 tokens through 2 of 8 experts of 4096 x 14336 took 26 us more.)
__device__ __forceinline__ int64_t inner_at(int64_t k) {
  return (k & ~int64_t(kChunk - 1)) + ((k >> 2 & 7) << 4) + ((k >> 5 & 3) << 2) + (k & 3);
}
__host__ __device__ __forceinline__ int64_t inner_width(int64_t I) {
  return (I + kChunk - 1) / kChunk * kChunk;
}

// ---------------------------------------------------------------------------- up
struct UpJobs {
  using S = Streamed<2, false>;
  static constexpr int kLoadStep = 1;
  const MoeArgs& p;
  Entries s;
  float s_gate, s_up;  // scales of this thread's place

  // (an expert's entries stand together, so that they read its weights at about the same time)
  __device__ __forceinline__ int64_t jobs() const { return p.I / kUpPlaces * s.count; }
  __device__ __forceinline__ int entry_of(int64_t job, int& tile) const {
    tile = int(uint32_t(job) / uint32_t(s.count));
    return int(job) - tile * s.count;
  }
  __device__ __forceinline__ void places(int64_t job, int (&y)[2]) const {
    int tile;
    const int entry = entry_of(job, tile);
    y[0] = int(s.expert[entry] * 2 * p.I) + tile * kUpPlaces;
    y[1] = y[0] + int(p.I);
  }
  __device__ __forceinline__ const uint16_t* tokens(int64_t job) const {
    const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    int tile;
    const int entry = entry_of(job, tile);
    return p.xs + min(s.first[entry] + g, s.first[entry + 1] - 1) * p.H + 32 * c;
  }
  __device__ __forceinline__ void begin(int64_t job, int t) {
    int tile;
    const int entry = entry_of(job, tile);
    const float* s1 = p.S1 + int64_t(s.expert[entry]) * 2 * p.I + tile * kUpPlaces + t % kUpPlaces;
    s_gate = load_ahead(s1);
    s_up = load_ahead(s1 + p.I);
  }
  __device__ __forceinline__ void finish(int64_t job, const float* part, int warps, int t,
                                         int threads) const {
    int tile;
    const int entry = entry_of(job, tile);
    const int first = s.first[entry], count = s.first[entry + 1] - first;
    const int place = t % kUpPlaces;
    // (whole warps stay together: the 16 places of a token are half of one)
    for (int j = t / kUpPlaces; j < (count + 1) / 2 * 2; j += threads / kUpPlaces) {
      float v = 0.f;
      if (j < count) {
        // (the weights' scales first: rows may be near FP32's largest number)
        const float down = s.down[first + j];
        const float gate = S::sum(part, warps, j, place) * (s_gate * kRecip127) * down;
        const float up = S::sum(part, warps, j, 16 + place) * (s_up * kRecip127) * down;
        v = __fdiv_rn(gate, 1.f + expf(-gate)) * up;
      }
      uint32_t top = __float_as_uint(v) & 0x7FFFFFFFu;
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(kAllLanes, top, o));
      if (j < count) {
        const int64_t at = first + j;
        p.inner[at * inner_width(p.I) + inner_at(tile * kUpPlaces + place)] = v;
        if (place == 0) atomicMax(p.r->top + at, top);
      }
    }
  }
};

__global__ void __launch_bounds__(kStreamThreads, kCtas)
    dq4_moe_up_kernel(const __grid_constant__ CUtensorMap map_w, const MoeArgs p) {
  extern __shared__ uint8_t smem_raw[];
  using Jobs = UpJobs;
  uint8_t* smem = aligned_1024(smem_raw);
  Jobs::S::setup(smem, map_w);
  wait_for_stream();
  asm volatile("griddepcontrol.launch_dependents;");
  Jobs jobs = {p, load_entries<false>(p, smem + Jobs::S::kBytes)};
  Jobs::S::run(jobs, smem, jobs.jobs(), p.H, map_w, p.bad);
}

// -------------------------------------------------------------------------- down
struct DownJobs {
  using S = Streamed<1, true>;
  static constexpr int kLoadStep = 4;
  const MoeArgs& p;
  Entries s;
  float s_place;  // scale of this thread's place

  __device__ __forceinline__ int64_t jobs() const {
    return (p.H + kDownPlaces - 1) / kDownPlaces * s.count;
  }
  __device__ __forceinline__ int entry_of(int64_t job, int& tile) const {
    tile = int(uint32_t(job) / uint32_t(s.count));
    return int(job) - tile * s.count;
  }
  __device__ __forceinline__ void places(int64_t job, int (&y)[1]) const {
    int tile;
    const int entry = entry_of(job, tile);
    y[0] = int(s.expert[entry] * p.H) + tile * kDownPlaces;
  }
  __device__ __forceinline__ int pair_of(int64_t job) const {
    int tile;
    const int entry = entry_of(job, tile);
    return min(s.first[entry] + (int(threadIdx.x & 31) >> 2), s.first[entry + 1] - 1);
  }
  __device__ __forceinline__ const float* tokens(int64_t job) const {
    return p.inner + pair_of(job) * inner_width(p.I) + 4 * (threadIdx.x & 3);
  }
  __device__ __forceinline__ float unit(int64_t job) const { return s.up[pair_of(job)]; }
  __device__ __forceinline__ void begin(int64_t job, int t) {
    int tile;
    const int entry = entry_of(job, tile);
    s_place = load_ahead(p.S2 + int64_t(s.expert[entry]) * p.H +
                         min(int64_t(tile) * kDownPlaces + t % kDownPlaces, p.H - 1));
  }
  __device__ __forceinline__ void finish(int64_t job, const float* part, int warps, int t,
                                         int threads) const {
    int tile;
    const int entry = entry_of(job, tile);
    const int first = s.first[entry], count = s.first[entry + 1] - first;
    const int place = t % kDownPlaces;
    const int64_t n = int64_t(tile) * kDownPlaces + place;
    if (n >= p.H) return;
    const float scale = s_place * kRecip127;
    for (int j = t / kDownPlaces; j < count; j += threads / kDownPlaces) {
      p.out[(first + j) * p.H + n] = S::sum(part, warps, j, place) * scale * s.down[first + j];
    }
  }
};

__global__ void __launch_bounds__(kStreamThreads, kCtas)
    dq4_moe_down_kernel(const __grid_constant__ CUtensorMap map_w, const MoeArgs p) {
  extern __shared__ uint8_t smem_raw[];
  using Jobs = DownJobs;
  uint8_t* smem = aligned_1024(smem_raw);
  Jobs::S::setup(smem, map_w);
  wait_for_stream();
  asm volatile("griddepcontrol.launch_dependents;");
  Jobs jobs = {p, load_entries<true>(p, smem + Jobs::S::kBytes)};
  Jobs::S::run(jobs, smem, jobs.jobs(), p.I, map_w, p.bad);
}

// ----------------------------------------------------------------------- combine
constexpr int kCombineThreads = 128;

// Each token's results by their weights, in the order of the choices: four places a thread.
__global__ void __launch_bounds__(kCombineThreads) dq4_moe_combine_kernel(const MoeArgs p) {
  wait_for_stream();
  asm volatile("griddepcontrol.launch_dependents;");
  const int64_t n = (int64_t(blockIdx.x) * kCombineThreads + threadIdx.x) * 4, token = blockIdx.y;
  if (n >= p.H) return;
  float y[4] = {};
#pragma unroll 4
  for (int j = 0; j < p.top_k; ++j) {
    const int pair = int(token) * p.top_k + j;
    const float w = load_global(p.weights + pair);
    const int64_t at = load_global(p.r->place + pair);
    const float4 v = load_global(reinterpret_cast<const float4*>(p.out + at * p.H + n));
    if (w != 0.f) {
      y[0] += w * v.x;
      y[1] += w * v.y;
      y[2] += w * v.z;
      y[3] += w * v.w;
    }
  }
  const int64_t at = token * p.H + n;
#pragma unroll
  for (int i = 0; i < 4; ++i) store_any(p.Y, at + i, y[i], p.bf16 ? DQ4_OUT_BF16 : DQ4_OUT_F16);
}

int64_t up256(int64_t n) { return (n + 255) / 256 * 256; }

int launch_moe(const MoeArgs& p, int dev, int sms, cudaStream_t s) {
  const int pairs = p.T * p.top_k;
  const int64_t entries = most_entries(p.E, pairs);
  const int more = int(entry_bytes(entries, pairs));
  constexpr int kMore = kMaxPairs * 8 + kMaxEntries * 4 + 2;
  constexpr int kUpBytes = UpJobs::S::kBytes + 1024, kDownBytes = DownJobs::S::kBytes + 1024;
  static_assert(kUpBytes + kMore <= 227 * 1024 && kDownBytes + kMore <= 227 * 1024,
                "shared memory");
  const int keys = kRouteThreads / 32 * p.E * 4;
  static std::atomic<uint64_t> allowed_route{0}, allowed_up{0}, allowed_down{0};
  if (const int st = allow_smem(dq4_moe_route_kernel, kRouteThreads / 32 * kMaxExperts * 4, dev,
                                &allowed_route))
    return st;
  if (const int st = allow_smem(dq4_moe_up_kernel, kUpBytes + kMore, dev, &allowed_up)) return st;
  if (const int st = allow_smem(dq4_moe_down_kernel, kDownBytes + kMore, dev, &allowed_down))
    return st;
  CUtensorMap w1, w2;
  if (const int st = encode_2d(&w1, CU_TENSOR_MAP_DATA_TYPE_UINT8, p.W1, p.H, 2 * p.I * p.E, p.H,
                               kChunk, kUpPlaces, CU_TENSOR_MAP_SWIZZLE_128B))
    return st;
  if (const int st = encode_2d(&w2, CU_TENSOR_MAP_DATA_TYPE_UINT8, p.W2, p.I, p.H * p.E, p.I,
                               kChunk, kDownPlaces, CU_TENSOR_MAP_SWIZZLE_128B))
    return st;
  if (const int st = launch_ordered(dq4_moe_route_kernel, dim3(unsigned(p.T)), kRouteThreads,
                                    keys, s, p))
    return st;
  // (jobs are known on the device only; no more than entries times the tiles of places)
  auto grid = [&](int64_t places, int64_t tile) {
    const int64_t jobs = (places + tile - 1) / tile * entries;
    return dim3(unsigned(jobs < kCtas * sms ? jobs : kCtas * sms));
  };
  if (const int st = launch_ordered(dq4_moe_up_kernel, grid(p.I, kUpPlaces), kStreamThreads,
                                    kUpBytes + more, s, w1, p))
    return st;
  if (const int st = launch_ordered(dq4_moe_down_kernel, grid(p.H, kDownPlaces),
                                    kStreamThreads, kDownBytes + more, s, w2, p))
    return st;
  const int64_t per = kCombineThreads * 4;
  return launch_ordered(dq4_moe_combine_kernel,
                        dim3(unsigned((p.H + per - 1) / per), unsigned(p.T)), kCombineThreads, 0, s,
                        p);
}

}  // namespace
}  // namespace dq4d

using namespace dq4d;

extern "C" {

int64_t dq4_int8_moe_workspace_bytes(int64_t T, int64_t H, int64_t I, int32_t top_k) {
  if (T <= 0 || H <= 0 || I <= 0 || top_k <= 0 || T > kMaxTokens || top_k > kMaxTopK ||
      H > kMaxHidden || I > kMaxInner)
    return 0;
  return up256(sizeof(Routed)) +
         T * top_k * (up256(H * 2) + inner_width(I) * 4 + up256(H * 4));
}

int dq4_int8_moe(const void* X, int64_t row_stride, int32_t dtype, int64_t T, int64_t H, int64_t I,
                 int64_t E, const float* logits, int32_t top_k, int32_t renormalize,
                 const int8_t* W1, const float* S1, const int8_t* W2, const float* S2,
                 int32_t* ids, float* weights, void* Y, void* workspace,
                 int64_t workspace_bytes, int* bad, void* stream) {
  if (T < 0 || T > kMaxTokens || E < 1 || E > kMaxExperts || top_k < 1 || top_k > kMaxTopK ||
      top_k > E || H < 0 || H > kMaxHidden || I < 0 || I > kMaxInner || H % 16 != 0 ||
      I % 16 != 0 || E * H * I >= int64_t(1) << 47)
    return DQ4_ERR_N;
  if (!valid_dtype(dtype, false)) return DQ4_ERR_DTYPE;
  if (T == 0) return DQ4_OK;
  if (H == 0 || I == 0) return DQ4_ERR_N;
  if (!X || !logits || !W1 || !S1 || !W2 || !S2 || !ids || !weights || !Y) return DQ4_ERR_NULL;
  if (misaligned(X, 16) || (T > 1 && row_stride % 8 != 0) || misaligned(logits, 4) ||
      misaligned(W1, 16) || misaligned(W2, 16) || misaligned(S1, 4) || misaligned(S2, 4) ||
      misaligned(ids, 4) || misaligned(weights, 4) || misaligned(Y, 2) || misaligned(bad, 4))
    return DQ4_ERR_ALIGN;
  if (!workspace || workspace_bytes < dq4_int8_moe_workspace_bytes(T, H, I, top_k))
    return DQ4_ERR_WORKSPACE;
  if (misaligned(workspace, 256)) return DQ4_ERR_ALIGN;
  int dev, sms;
  if (const int st = current_device(&dev, &sms)) return st;
  MoeArgs p = {X, row_stride, dtype == DQ4_OUT_BF16, int(T), int(E), top_k, renormalize, H, I,
               logits, W1, W2, S1, S2, ids, weights, Y, nullptr, nullptr, nullptr, nullptr, bad};
  char* at = static_cast<char*>(workspace);
  p.r = reinterpret_cast<Routed*>(at);
  at += up256(sizeof(Routed));
  p.xs = reinterpret_cast<uint16_t*>(at);
  at += T * top_k * up256(H * 2);
  p.inner = reinterpret_cast<float*>(at);
  at += T * top_k * inner_width(I) * 4;
  p.out = reinterpret_cast<float*>(at);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  return launch_moe(p, dev, sms, s);
}

}  // extern "C"
