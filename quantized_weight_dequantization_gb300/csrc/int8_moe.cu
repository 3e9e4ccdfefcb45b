// A mixture-of-experts layer for few tokens over 8-bit weights: dq4_int8_moe (dq4_int8.h).
//
// Bound by the bytes of the chosen experts' weights, each read once.  Four launches:
//   route   one CTA chooses the experts and lists each one's (token, choice) pairs, by entries of
//           up to 8 NT; one CTA a token brings its row to FP16, scaled by a power of two
//   up      a job is 16 inner places of an entry's expert, gate and up rows together: inner =
//           silu(g) * u in FP16, scaled by a power of two for each 16 places of a pair, and the
//           largest of each pair's row
//   down    a job is 32 output places of an entry's expert; inner values are brought to a scale for
//           their row on their way in, exactly (powers of two)
//   combine each token's results by their weights
// Experts that no token chose have no jobs.  No atomic adds a value.
#include "int8.cuh"

namespace dq4d {
namespace {

constexpr int kRouteThreads = 512;
constexpr int kMaxTokens = 256, kMaxExperts = 1024, kMaxTopK = 16;
constexpr int kMaxPairs = kMaxTokens * kMaxTopK;
constexpr int kMaxEntries = kMaxExperts + kMaxPairs / 8;
constexpr int kUpPlaces = 16, kDownPlaces = 32;
constexpr int64_t kMaxInner = 1 << 20;
constexpr int64_t kMaxHidden = 1 << 15;

// What `route` finds out, at the head of the workspace.  Pairs (token, choice) stand in the order
// of their experts: `place` is a pair's there, and rows of xs, inner and out are by place.
struct Routed {
  int entries;                      // experts with pairs, one for each 8 NT of them
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
  int T, E, top_k, renormalize, most;  // most: tokens of an entry
  int64_t H, I;
  const float* logits;
  const int8_t *W1, *W2;
  const float *S1, *S2;
  int32_t* ids;
  float* weights;
  void* Y;
  Routed* r;
  uint16_t* xs;     // [pairs][H] FP16
  uint16_t* inner;  // [pairs][I] FP16, scaled for each tile of 16
  float* inner_by;  // [pairs][I / 16] what a tile has to be multiplied by
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

// Every CTA finds out the whole routing for itself (the warps' tokens side by side, so that it takes
// no longer than one token's); CTA t then writes token t's row, and CTA 0 the lists.
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
    both += uint32_t(counts[k]) | uint32_t((counts[k] + p.most - 1) / p.most) << 16;
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
      for (int done = 0; done < counts[k]; done += p.most, ++entry) {
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

// What the other two kernels hold of it in shared memory, behind their rings.
struct Entries {
  float *up, *down;  // of a place's token: xs's `down`, or the scaling of its inner row
  uint16_t *expert, *first;
  int count;
};
int64_t entry_bytes(int64_t entries, int64_t pairs) { return pairs * 8 + entries * 4 + 2; }
int64_t most_entries(int64_t E, int64_t pairs, int64_t most) {
  return (E < pairs ? E : pairs) + pairs / most;
}

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

// ---------------------------------------------------------------------------- up
template <int NT, int kDepth>
struct UpJobs {
  using S = Streamed<2, NT, 2, 4, false, kDepth>;
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
  __device__ __forceinline__ void tokens(int64_t job, const uint8_t* (&tok)[NT]) const {
    const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    int tile;
    const int entry = entry_of(job, tile);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
      tok[nt] = reinterpret_cast<const uint8_t*>(
          p.xs + min(s.first[entry] + 8 * nt + g, s.first[entry + 1] - 1) * p.H + 32 * c);
  }
  __device__ __forceinline__ void start() const {}
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
        const float down = s.down[first + j] * kRecip127;
        const float gate = S::sum(part, warps, j, place) * down * s_gate;
        const float up = S::sum(part, warps, j, 16 + place) * down * s_up;
        v = __fdiv_rn(gate, 1.f + expf(-gate)) * up;
      }
      uint32_t top = __float_as_uint(v) & 0x7FFFFFFFu;
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(kAllLanes, top, o));
      if (j < count) {
        float up, down;
        pow2_scaling(__uint_as_float(top), up, down);
        const int64_t at = first + j;
        p.inner[at * p.I + tile * kUpPlaces + place] = __half_as_ushort(__float2half_rn(v * up));
        if (place == 0) {
          p.inner_by[at * (p.I / kUpPlaces) + tile] = down;
          atomicMax(p.r->top + at, top);
        }
      }
    }
  }
};

template <int NT, int kDepth, int kCtas>
__global__ void __launch_bounds__(kStreamThreads, kCtas)
    dq4_moe_up_kernel(const __grid_constant__ CUtensorMap map_w, const MoeArgs p) {
  extern __shared__ uint8_t smem_raw[];
  using Jobs = UpJobs<NT, kDepth>;
  uint8_t* smem = aligned_1024(smem_raw);
  Jobs::S::setup(smem, map_w);
  wait_for_stream();
  asm volatile("griddepcontrol.launch_dependents;");
  Jobs jobs = {p, load_entries<false>(p, smem + Jobs::S::kBytes)};
  Jobs::S::run(jobs, smem, jobs.jobs(), p.H, map_w, p.bad);
}

// -------------------------------------------------------------------------- down
template <int NT, int kDepth>
struct DownJobs {
  using S = Streamed<2, NT, 1, 4, true, kDepth>;
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
  __device__ __forceinline__ int pair_of(int entry, int nt) const {
    return min(s.first[entry] + 8 * nt + (int(threadIdx.x & 31) >> 2), s.first[entry + 1] - 1);
  }
  __device__ __forceinline__ void tokens(int64_t job, const uint8_t* (&tok)[NT]) const {
    int tile;
    const int entry = entry_of(job, tile);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
      tok[nt] = reinterpret_cast<const uint8_t*>(p.inner + pair_of(entry, nt) * p.I +
                                                 32 * (threadIdx.x & 3));
  }
  // A tile's FP16 values in the row's unit: powers of two, both.
  __device__ __forceinline__ void scales(int64_t job, int64_t k, float (&f)[2 * NT]) const {
    int tile;
    const int entry = entry_of(job, tile);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int at = pair_of(entry, nt);
#pragma unroll
      for (int h = 0; h < 2; ++h)
        f[2 * nt + h] = k + 16 * h < p.I
                            ? load_ahead(p.inner_by + at * (p.I / kUpPlaces) + k / kUpPlaces + h) *
                                  s.up[at]
                            : 0.f;
    }
  }
  __device__ __forceinline__ void start() const {}
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
      p.out[(first + j) * p.H + n] = S::sum(part, warps, j, place) * s.down[first + j] * scale;
    }
  }
};

template <int NT, int kDepth, int kCtas>
__global__ void __launch_bounds__(kStreamThreads, kCtas)
    dq4_moe_down_kernel(const __grid_constant__ CUtensorMap map_w, const MoeArgs p) {
  extern __shared__ uint8_t smem_raw[];
  using Jobs = DownJobs<NT, kDepth>;
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

// NT: tokens of an entry, by eights; depths of the rings, CTAs of an SM.
template <int NT, int kUpDepth, int kUpCtas, int kDownDepth, int kDownCtas>
int launch_moe(MoeArgs p, int dev, int sms, cudaStream_t s) {
  p.most = 8 * NT;
  auto up = dq4_moe_up_kernel<NT, kUpDepth, kUpCtas>;
  auto down = dq4_moe_down_kernel<NT, kDownDepth, kDownCtas>;
  const int pairs = p.T * p.top_k;
  const int64_t entries = most_entries(p.E, pairs, p.most);
  const int more = int(entry_bytes(entries, pairs));
  constexpr int kMore = kMaxPairs * 8 + (kMaxExperts + kMaxPairs / 8) * 4 + 2;
  constexpr int kUpBytes = UpJobs<NT, kUpDepth>::S::kBytes + 1024;
  constexpr int kDownBytes = DownJobs<NT, kDownDepth>::S::kBytes + 1024;
  static_assert(kUpBytes + kMore <= 227 * 1024 && kDownBytes + kMore <= 227 * 1024, "shared memory");
  const int keys = kRouteThreads / 32 * p.E * 4;
  static std::atomic<uint64_t> allowed_route{0}, allowed_up{0}, allowed_down{0};
  if (const int st = allow_smem(dq4_moe_route_kernel, kRouteThreads / 32 * kMaxExperts * 4, dev,
                                &allowed_route))
    return st;
  if (const int st = allow_smem(up, kUpBytes + kMore, dev, &allowed_up)) return st;
  if (const int st = allow_smem(down, kDownBytes + kMore, dev, &allowed_down)) return st;
  CUtensorMap w1, w2;
  if (const int st = encode_2d(&w1, CU_TENSOR_MAP_DATA_TYPE_UINT8, p.W1, p.H, 2 * p.I * p.E, p.H,
                               kChunk, kUpPlaces, CU_TENSOR_MAP_SWIZZLE_128B))
    return st;
  if (const int st = encode_2d(&w2, CU_TENSOR_MAP_DATA_TYPE_UINT8, p.W2, p.I, p.H * p.E, p.I, kChunk,
                               kDownPlaces, CU_TENSOR_MAP_SWIZZLE_128B))
    return st;
  if (const int st = launch_ordered(dq4_moe_route_kernel, dim3(unsigned(p.T)), kRouteThreads, keys, s,
                                    p))
    return st;
  // (jobs are known on the device only; no more than entries times the tiles of places)
  auto grid = [&](int64_t places, int64_t tile, int ctas) {
    const int64_t jobs = (places + tile - 1) / tile * entries;
    return dim3(unsigned(jobs < ctas * sms ? jobs : ctas * sms));
  };
  if (const int st = launch_ordered(up, grid(p.I, kUpPlaces, kUpCtas), kStreamThreads,
                                    kUpBytes + more, s, w1, p))
    return st;
  if (const int st = launch_ordered(down, grid(p.H, kDownPlaces, kDownCtas), kStreamThreads,
                                    kDownBytes + more, s, w2, p))
    return st;
  const int64_t per = kCombineThreads * 4;
  return launch_ordered(dq4_moe_combine_kernel, dim3(unsigned((p.H + per - 1) / per), unsigned(p.T)),
                        kCombineThreads, 0, s, p);
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
         T * top_k * (up256(H * 2) + up256(I * 2) + up256(I / 4) + up256(H * 4));
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
  if (T == 0 || H == 0) return DQ4_OK;
  if (I == 0) return DQ4_ERR_N;
  if (!X || !logits || !W1 || !S1 || !W2 || !S2 || !ids || !weights || !Y) return DQ4_ERR_NULL;
  if (misaligned(X, 16) || row_stride % 8 != 0 || misaligned(logits, 4) || misaligned(W1, 16) ||
      misaligned(W2, 16) || misaligned(S1, 4) || misaligned(S2, 4) || misaligned(ids, 4) ||
      misaligned(weights, 4) || misaligned(Y, 2) || misaligned(bad, 4))
    return DQ4_ERR_ALIGN;
  if (!workspace || workspace_bytes < dq4_int8_moe_workspace_bytes(T, H, I, top_k))
    return DQ4_ERR_WORKSPACE;
  if (misaligned(workspace, 256)) return DQ4_ERR_ALIGN;
  int dev, sms;
  if (const int st = current_device(&dev, &sms)) return st;
  MoeArgs p = {X, row_stride, dtype == DQ4_OUT_BF16, int(T), int(E), top_k, renormalize, 0, H, I, logits,
               W1, W2, S1, S2, ids, weights, Y, nullptr, nullptr, nullptr, nullptr,
               nullptr, bad};
  char* at = static_cast<char*>(workspace);
  p.r = reinterpret_cast<Routed*>(at);
  at += up256(sizeof(Routed));
  p.xs = reinterpret_cast<uint16_t*>(at);
  at += T * top_k * up256(H * 2);
  p.inner = reinterpret_cast<uint16_t*>(at);
  at += T * top_k * up256(I * 2);
  p.inner_by = reinterpret_cast<float*>(at);
  at += T * top_k * up256(I / 4);
  p.out = reinterpret_cast<float*>(at);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  // (entries of 16 pairs, two products for each weight's conversion, took more: for 64 tokens
  // through 2 of 8 experts of 4096 x 14336, 16 pairs each, 443 us, in eights, which read the weights
  // twice from L2, 409; for 23 tokens 302 and 237)
  return launch_moe<1, 2, 2, 2, 2>(p, dev, sms, s);
}

}  // extern "C"
