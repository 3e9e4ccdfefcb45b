// A mixture-of-experts layer for few tokens over 8-bit weights: dq4_int8_moe (dq4_int8.h).
//
// Bound by the bytes of the chosen experts' weights, each read once.  Three launches:
//   route   one CTA chooses the experts and lists each one's (token, choice) pairs; one CTA a token
//           brings its row to FP16, scaled by a power of two
//   up      a CTA takes 16 inner places of an expert, gate and up rows together, for all its
//           tokens: inner = silu(g) * u in FP32, and the largest of each pair's row
//   down    a CTA takes 32 output places of an expert; inner values become FP16 on their way in,
//           scaled by a power of two for each pair; the last CTA of a place sums its experts'
//           results by the weights, in the order of the choices
// Experts that no token chose have no CTA that does anything.  No atomic adds a value.
#include "int8.cuh"
#include "tcgen05.cuh"

namespace dq4d {
namespace {

constexpr int kWarps = 8;
constexpr int kMoeThreads = 32 * kWarps;
constexpr int kMaxTokens = 256, kMaxExperts = 1024, kMaxTopK = 16;
constexpr int kMaxPairs = kMaxTokens * kMaxTopK;
constexpr int kUpPlaces = 16, kDownPlaces = 32;
constexpr int64_t kMaxHidden = kInt8Counters / 4 * kDownPlaces;

// What `route` finds out, at the head of the workspace behind the counters.
struct Routed {
  int active;                     // experts with tokens
  int expert[kMaxExperts];        // of each
  int first[kMaxExperts + 1];     // and its first pair in pairs
  int pairs[kMaxPairs];           // token * top_k + choice, by expert
  uint32_t top[kMaxPairs];        // bits of the largest |inner value| of a pair
  float down[kMaxTokens];         // what a row's FP16 values have to be multiplied by
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
  int* done;     // [H / kDownPlaces] arrivals
  Routed* r;
  uint16_t* xs;  // [T][H] FP16
  float* inner;  // [pairs][I]
  float* out;    // [pairs][H]
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

__global__ void __launch_bounds__(kMoeThreads) dq4_moe_route_kernel(const MoeArgs p) {
  __shared__ uint32_t s_key[kWarps][kMaxExperts];
  __shared__ uint16_t s_ids[kMaxPairs];
  __shared__ int s_sums[kWarps];
  __shared__ uint32_t s_top[kWarps];
  wait_for_stream();
  asm volatile("griddepcontrol.launch_dependents;");
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  if (blockIdx.x > 0) {
    // ---- one token's row in FP16
    const int64_t token = blockIdx.x - 1;
    const uint16_t* x = static_cast<const uint16_t*>(p.X) + token * p.row_stride;
    uint32_t top = 0;
    for (int64_t i = t * 8; i < p.H; i += kMoeThreads * 8) {
      const uint4 v = load_global(reinterpret_cast<const uint4*>(x + i));
      const uint32_t m = __vmaxu2(__vmaxu2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu),
                                  __vmaxu2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu));
      top = max(top, max(m & 0xFFFFu, m >> 16));
    }
    top = __reduce_max_sync(kAllLanes, top);
    if (lane == 0) s_top[warp] = top;
    __syncthreads();
    for (int w = 0; w < kWarps; ++w) top = max(top, s_top[w]);
    float up, down;
    pow2_scaling(p.bf16 ? __uint_as_float(top << 16) : __half2float(__ushort_as_half(uint16_t(top))),
                 up, down);
    if (t == 0) p.r->down[token] = down;
    for (int64_t i = t * 8; i < p.H; i += kMoeThreads * 8) {
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
      *reinterpret_cast<uint4*>(p.xs + token * p.H + i) = make_uint4(o[0], o[1], o[2], o[3]);
    }
    return;
  }
  // ---- the experts of each token, a warp a token
  const int pairs = p.T * p.top_k;
  for (int token = warp; token < p.T; token += kWarps) {
    const float* row = p.logits + int64_t(token) * p.E;
    uint32_t* key = s_key[warp];
    bool nan = false;
    for (int e = lane; e < p.E; e += 32) {
      const float x = load_global(row + e);
      nan |= x != x;
      key[e] = order_key(x);
    }
    nan = __any_sync(kAllLanes, nan);
    __syncwarp();
    int mine = 0;  // lane j: the j-th choice
    for (int j = 0; j < p.top_k; ++j) {
      uint32_t best = 0;
      int at = 0;
      for (int e = lane; e < p.E; e += 32)
        if (key[e] > best) {
          best = key[e];
          at = e;
        }
      const uint32_t top = __reduce_max_sync(kAllLanes, best);
      const int e = __reduce_min_sync(kAllLanes, best == top ? unsigned(at) : 0xFFFFFFFFu);
      if (lane == j) mine = e;
      if (lane == 0) key[e] = 0;
      __syncwarp();
    }
    float l = lane < p.top_k ? load_global(row + mine) : -INFINITY;
    const float top = __shfl_sync(kAllLanes, l, 0);
    float sum = 0.f;
    const float part = top == -INFINITY ? 0.f : expf(l - top);  // of lane's choice
    if (p.renormalize) {
      if (lane < p.top_k) sum = part;
    } else {
      for (int e = lane; e < p.E; e += 32) sum += expf(load_global(row + e) - top);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kAllLanes, sum, o);
    float weight = top == -INFINITY ? 0.f : __fdiv_rn(part, sum);
    if (nan) weight = __uint_as_float(0x7FC00000u);
    if (lane < p.top_k) {
      p.ids[token * p.top_k + lane] = mine;
      p.weights[token * p.top_k + lane] = weight;
      s_ids[token * p.top_k + lane] = uint16_t(mine);
    }
    __syncwarp();
  }
  for (int i = t; i < pairs; i += kMoeThreads) p.r->top[i] = 0;
  __syncthreads();
  // ---- each expert's pairs, in their order; thread t looks after four experts
  constexpr int kEach = kMaxExperts / kMoeThreads;
  int count[kEach] = {};
  for (int i = 0; i < pairs; ++i) {
    const int e = s_ids[i] - t * kEach;
    if (e >= 0 && e < kEach) {
#pragma unroll
      for (int k = 0; k < kEach; ++k) count[k] += e == k;
    }
  }
  int both = 0;  // pairs, and experts with pairs, packed
#pragma unroll
  for (int k = 0; k < kEach; ++k) both += count[k] | (count[k] > 0) << 16;
  int run = both;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int up = __shfl_up_sync(kAllLanes, run, o);
    if (lane >= o) run += up;
  }
  if (lane == 31) s_sums[warp] = run;
  __syncthreads();
  int at = run - both, all = 0;
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) at += s_sums[w];
    all += s_sums[w];
  }
  int next[kEach], a = at >> 16, f = at & 0xFFFF;
#pragma unroll
  for (int k = 0; k < kEach; ++k) {
    next[k] = f;
    if (count[k] > 0) {
      p.r->expert[a] = t * kEach + k;
      p.r->first[a] = f;
      ++a;
      f += count[k];
    }
  }
  if (t == 0) {
    p.r->active = all >> 16;
    p.r->first[all >> 16] = pairs;
  }
  for (int i = 0; i < pairs; ++i) {
    const int e = s_ids[i] - t * kEach;
    if (e >= 0 && e < kEach) {
#pragma unroll
      for (int k = 0; k < kEach; ++k)
        if (e == k) p.r->pairs[next[k]++] = i;
    }
  }
}

// ---------------------------------------------------------------------------- up
// Tokens in FP16: lane's token of each 8, advanced to its 16 c, or null.
template <int NT>
struct HalfTokens {
  struct Raw {
    uint4 a, b;
  };
  const uint16_t* at[NT];
  __device__ __forceinline__ void load(Raw& x, int nt, int64_t k, bool in) const {
    x.a = x.b = make_uint4(0, 0, 0, 0);
    if (in && at[nt]) {
      x.a = load_global(reinterpret_cast<const uint4*>(at[nt] + k));
      x.b = load_global(reinterpret_cast<const uint4*>(at[nt] + k) + 1);
    }
  }
  __device__ __forceinline__ void words(const Raw& x, int, int s, uint32_t& b0, uint32_t& b1) const {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(s < 2 ? &x.a : &x.b);
    b0 = w[2 * (s & 1)];
    b1 = w[2 * (s & 1) + 1];
  }
};

template <int NT, int U>
__global__ void __launch_bounds__(kMoeThreads, 2) dq4_moe_up_kernel(const MoeArgs p) {
  constexpr int kTokens = 8 * NT;
  __shared__ float s_part[kWarps * 32 * kTokens];
  wait_for_stream();
  asm volatile("griddepcontrol.launch_dependents;");
  if (int(blockIdx.y) >= load_global(&p.r->active)) return;
  const int e = load_global(p.r->expert + blockIdx.y);
  const int first = load_global(p.r->first + blockIdx.y);
  const int count = load_global(p.r->first + blockIdx.y + 1) - first;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const int64_t i0 = int64_t(blockIdx.x) * kUpPlaces;
  const int8_t* row[2][2];
#pragma unroll
  for (int rt = 0; rt < 2; ++rt)
#pragma unroll
    for (int h = 0; h < 2; ++h)
      row[rt][h] = p.W1 + ((int64_t(e) * 2 + rt) * p.I + i0 + 8 * h + g) * p.H + 16 * c;
  for (int j0 = 0; j0 < count; j0 += kTokens) {
    HalfTokens<NT> src;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int j = j0 + 8 * nt + g;
      src.at[nt] = nullptr;
      if (j < count)
        src.at[nt] = p.xs + int64_t(load_global(p.r->pairs + first + j) / p.top_k) * p.H + 16 * c;
    }
    float acc[2][NT][4] = {};
    warp_product<2, NT, U>(acc, row, src, p.H, warp, kWarps, int((p.H + 63) / 64));
    __syncthreads();  // (the last tokens' sums have been read)
    put_part<2, NT>(s_part, acc);
    __syncthreads();
    for (int i = threadIdx.x; i < kUpPlaces * kTokens; i += kMoeThreads) {
      const int place = i % kUpPlaces, j = j0 + i / kUpPlaces;
      float v = 0.f;
      int pair = 0;
      if (j < count) {
        pair = load_global(p.r->pairs + first + j);
        const float down = load_global(p.r->down + pair / p.top_k) * kRecip127;
        const float* s1 = p.S1 + int64_t(e) * 2 * p.I + i0 + place;
        const float gate = sum_parts<2, NT>(s_part, kWarps, i / kUpPlaces, place) * down *
                           load_global(s1);
        const float up = sum_parts<2, NT>(s_part, kWarps, i / kUpPlaces, 16 + place) * down *
                         load_global(s1 + p.I);
        v = __fdiv_rn(gate, 1.f + expf(-gate)) * up;
        p.inner[int64_t(pair) * p.I + i0 + place] = v;
      }
      uint32_t top = __float_as_uint(v) & 0x7FFFFFFFu;
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(kAllLanes, top, o));
      if (place == 0 && j < count) atomicMax(p.r->top + pair, top);
    }
  }
}

// -------------------------------------------------------------------------- down
// Tokens in FP32, brought to FP16 by a power of two.
template <int NT>
struct ScaledTokens {
  struct Raw {
    float4 v[4];
  };
  const float* at[NT];
  float up[NT];
  __device__ __forceinline__ void load(Raw& x, int nt, int64_t k, bool in) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x.v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (in && at[nt]) x.v[i] = load_global(reinterpret_cast<const float4*>(at[nt] + k) + i);
    }
  }
  __device__ __forceinline__ void words(const Raw& x, int nt, int s, uint32_t& b0,
                                        uint32_t& b1) const {
    b0 = pack2<DQ4_OUT_F16>(x.v[s].x * up[nt], x.v[s].y * up[nt]);
    b1 = pack2<DQ4_OUT_F16>(x.v[s].z * up[nt], x.v[s].w * up[nt]);
  }
};

template <int NT, int U>
__global__ void __launch_bounds__(kMoeThreads, 2) dq4_moe_down_kernel(const MoeArgs p) {
  constexpr int kTokens = 8 * NT;
  __shared__ float s_part[kWarps * kDownPlaces * kTokens];
  __shared__ bool s_last;
  wait_for_stream();
  asm volatile("griddepcontrol.launch_dependents;");
  const int active = load_global(&p.r->active);
  if (int(blockIdx.y) >= active) return;
  const int e = load_global(p.r->expert + blockIdx.y);
  const int first = load_global(p.r->first + blockIdx.y);
  const int count = load_global(p.r->first + blockIdx.y + 1) - first;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const int64_t n0 = int64_t(blockIdx.x) * kDownPlaces;
  const int8_t* row[2][2];
#pragma unroll
  for (int rt = 0; rt < 2; ++rt)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int64_t n = n0 + 16 * rt + 8 * h + g;
      row[rt][h] = n < p.H ? p.W2 + (int64_t(e) * p.H + n) * p.I + 16 * c : nullptr;
    }
  for (int j0 = 0; j0 < count; j0 += kTokens) {
    ScaledTokens<NT> src;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int j = j0 + 8 * nt + g;
      src.at[nt] = nullptr;
      src.up[nt] = 0.f;
      if (j < count) {
        const int pair = load_global(p.r->pairs + first + j);
        float down;
        pow2_scaling(__uint_as_float(load_global(p.r->top + pair)), src.up[nt], down);
        src.at[nt] = p.inner + int64_t(pair) * p.I + 16 * c;
      }
    }
    float acc[2][NT][4] = {};
    warp_product<2, NT, U>(acc, row, src, p.I, warp, kWarps, int((p.I + 63) / 64));
    __syncthreads();
    put_part<2, NT>(s_part, acc);
    __syncthreads();
    for (int i = threadIdx.x; i < kDownPlaces * kTokens; i += kMoeThreads) {
      const int place = i % kDownPlaces, j = j0 + i / kDownPlaces;
      if (j >= count || n0 + place >= p.H) continue;
      const int pair = load_global(p.r->pairs + first + j);
      float up, down;
      pow2_scaling(__uint_as_float(load_global(p.r->top + pair)), up, down);
      p.out[int64_t(pair) * p.H + n0 + place] =
          sum_parts<2, NT>(s_part, kWarps, i / kDownPlaces, place) * down *
          (load_global(p.S2 + int64_t(e) * p.H + n0 + place) * kRecip127);
    }
  }
  // ---- the last expert of these places sums them all
  __syncthreads();
  if (threadIdx.x == 0) s_last = atomic_add_acq_rel(p.done + blockIdx.x, 1) == active - 1;
  __syncthreads();
  if (!s_last) return;
  for (int i = threadIdx.x; i < p.T * kDownPlaces; i += kMoeThreads) {
    const int64_t n = n0 + i % kDownPlaces, token = i / kDownPlaces;
    if (n >= p.H) continue;
    float y = 0.f;
    for (int j = 0; j < p.top_k; ++j) {
      const int64_t pair = token * p.top_k + j;
      const float w = load_global(p.weights + pair);
      if (w != 0.f) y += w * load_l2(p.out + pair * p.H + n);
    }
    store_any(p.Y, token * p.H + n, y, p.bf16 ? DQ4_OUT_BF16 : DQ4_OUT_F16);
  }
  if (threadIdx.x == 0) p.done[blockIdx.x] = 0;
}

int64_t up256(int64_t n) { return (n + 255) / 256 * 256; }

template <int NT, int U>
int launch_moe(const MoeArgs& p, cudaStream_t s) {
  const unsigned most = unsigned(p.E < p.T * p.top_k ? p.E : p.T * p.top_k);
  if (const int st = launch_ordered(dq4_moe_route_kernel, dim3(unsigned(p.T + 1)), kMoeThreads, 0, s, p))
    return st;
  if (const int st = launch_ordered(dq4_moe_up_kernel<NT, U>,
                                    dim3(unsigned(p.I / kUpPlaces), most), kMoeThreads, 0, s, p))
    return st;
  return launch_ordered(dq4_moe_down_kernel<NT, U>,
                        dim3(unsigned((p.H + kDownPlaces - 1) / kDownPlaces), most), kMoeThreads, 0,
                        s, p);
}

}  // namespace
}  // namespace dq4d

using namespace dq4d;

extern "C" {

int64_t dq4_int8_moe_workspace_bytes(int64_t T, int64_t H, int64_t I, int32_t top_k) {
  if (T <= 0 || H <= 0 || I <= 0 || top_k <= 0 || T > kMaxTokens || top_k > kMaxTopK ||
      H > kMaxHidden || I > INT32_MAX)
    return 0;
  return kInt8Counters + up256(sizeof(Routed)) + up256(T * H * 2) +
         T * top_k * (up256(I * 4) + up256(H * 4));
}

int dq4_int8_moe(const void* X, int64_t row_stride, int32_t dtype, int64_t T, int64_t H, int64_t I,
                 int64_t E, const float* logits, int32_t top_k, int32_t renormalize,
                 const int8_t* W1, const float* S1, const int8_t* W2, const float* S2,
                 int32_t* ids, float* weights, void* Y, void* workspace,
                 int64_t workspace_bytes, void* stream) {
  if (T < 0 || T > kMaxTokens || E < 1 || E > kMaxExperts || top_k < 1 || top_k > kMaxTopK ||
      top_k > E || H < 0 || H > kMaxHidden || I < 0 || I > INT32_MAX || H % 16 != 0 ||
      I % 16 != 0 || E * H * I >= int64_t(1) << 47)
    return DQ4_ERR_N;
  if (!valid_dtype(dtype, false)) return DQ4_ERR_DTYPE;
  if (T == 0 || H == 0) return DQ4_OK;
  if (I == 0) return DQ4_ERR_N;
  if (!X || !logits || !W1 || !S1 || !W2 || !S2 || !ids || !weights || !Y) return DQ4_ERR_NULL;
  if (misaligned(X, 16) || row_stride % 8 != 0 || misaligned(logits, 4) || misaligned(W1, 16) ||
      misaligned(W2, 16) || misaligned(S1, 4) || misaligned(S2, 4) || misaligned(ids, 4) ||
      misaligned(weights, 4) || misaligned(Y, 2))
    return DQ4_ERR_ALIGN;
  if (!workspace || workspace_bytes < dq4_int8_moe_workspace_bytes(T, H, I, top_k))
    return DQ4_ERR_WORKSPACE;
  if (misaligned(workspace, 256)) return DQ4_ERR_ALIGN;
  int dev, sms;
  if (const int st = current_device(&dev, &sms)) return st;
  MoeArgs p = {X, row_stride, dtype == DQ4_OUT_BF16, int(T), int(E), top_k, renormalize, H, I, logits,
               W1, W2, S1, S2, ids, weights, Y, nullptr, nullptr, nullptr, nullptr, nullptr};
  char* at = static_cast<char*>(workspace);
  p.done = reinterpret_cast<int*>(at);
  at += kInt8Counters;
  p.r = reinterpret_cast<Routed*>(at);
  at += up256(sizeof(Routed));
  p.xs = reinterpret_cast<uint16_t*>(at);
  at += up256(T * H * 2);
  p.inner = reinterpret_cast<float*>(at);
  at += T * top_k * up256(I * 4);
  p.out = reinterpret_cast<float*>(at);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (T <= 8) return launch_moe<1, 2>(p, s);
  return launch_moe<2, 2>(p, s);
}

}  // extern "C"
