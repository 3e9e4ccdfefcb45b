// Norm and rotation of every head of queries and keys, and its gradients:
// dq4_qk_norm_rope and dq4_qk_norm_rope_backward (dq4_attn.h).
//
// Forward, for a head x of D values at position p:
//   y = R(p) (w x r),  r = 1 / sqrt(mean(x^2) + eps)
// Backward, with g = R(-p) dy (R is orthogonal, so its transpose is R(-p)), xh = x r:
//   dx = r (g w - xh mean(g w xh)),   dw = sum over tokens and heads of g xh
// Both read every value once and write every result once.  Measured, 32 + 8 heads of 128, BF16:
// forward 8191 tokens 31 us (172 MB, 5.5 TB/s), backward 16384 tokens 103 us (512 MB, 5.0 TB/s),
// against 6.8 TB/s of a copy; 4 tokens take 1.8 us.  What holds them back from the copy is the
// instructions of 8 values a lane and the latency of a warp's chain (position, tables, rows, the
// sums over the lanes) at the occupancy that the rows in registers allow.  Tried and slower: 16
// values a lane (fewer instructions, fewer warps: 40 us and 110 us), rows through shared memory
// by asynchronous copies two units ahead (36 and 106 us), packed FP32 pairs (33 and 105 us).
#include "attn.cuh"

namespace dq4d {
namespace {

constexpr int V = 4;               // values of a lane's groups (lane_place)
// Forward: 4 warps a CTA (8191 tokens: 31.0 us; with 8 warps 32.0, with 16 33.9), and 32 warps
// per SM (24, with all the registers that a lane would take: 36 us).
constexpr int kNormThreads = 128;
constexpr int kNormCtas = 8;
constexpr int kBwdThreads = 256;   // backward: 8 warps, each with weight-gradient sums
constexpr int kBwdCtas = 2;        // and CTAs per SM
constexpr int kMaxPartials = 512;  // CTAs that may leave weight-gradient partials
constexpr int kPartGroup = 24;     // of them summed together first
constexpr int kMaxGroups = (kMaxPartials + kPartGroup - 1) / kPartGroup;
static_assert((1 + kMaxGroups) * 4 <= 256, "counters at the workspace's head");
constexpr int kMaxDim = 1024;
constexpr int kAnyWarps = 4;       // warps per CTA of the any-size kernels

struct NormArgs {
  const void* x[2];        // q, k
  const void* dy[2];       // backward: gradients of the outputs
  int64_t token_stride[2], head_stride[2];
  const void* w[2];        // weights, or null
  void* out[2];            // outputs; backward: dx
  int heads[2];
  int64_t tokens;
  float eps;
  const float* cos;
  const float* sin;
  int64_t table_rows;
  int dim, rotary;
  bool interleaved;
  const int64_t* positions;
  int* bad;
  int chunks[2];           // head chunks of a token, of q and of k
  int chunk;               // heads in a chunk
  float* dw[2];
  int* count;              // backward: CTAs that left their partials
  float* part;             // backward: [CTA][2][dim]
};

// The position's row of the tables, or -1 where it is outside them (all lanes alike).
__device__ __forceinline__ int64_t table_row(const NormArgs& p, int64_t t) {
  if (p.cos == nullptr) return 0;
  const int64_t pos = load_global(p.positions + t);
  return pos >= 0 && pos < p.table_rows ? pos : -1;
}

template <int kLanes>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) v += __shfl_xor_sync(kAllLanes, v, o);
  return v;
}

struct Turn {
  float c[V], s[V];
};

// The cosines and sines of lane l at a row of the tables.
__device__ __forceinline__ Turn load_turn(const NormArgs& p, bool turned, int64_t row, int l) {
  Turn t = {};
  if (turned && row >= 0) {
    load_entries(p.cos + row * (p.rotary / 2) + V * l, t.c);
    load_entries(p.sin + row * (p.rotary / 2) + V * l, t.s);
  }
  return t;
}

// A warp takes a unit: kRows heads of one token for each of its 32 / kLanes groups of
// kLanes = kDim / 2 V lanes, all of q or all of k.  The position's cosines and sines and the
// weights stay in registers over the unit, multiplied:
//   R(w x r) = r (x (w C) + y (w' S)),  y and w' the partners of x and w,
// and all its loads are issued before the first use.  kRows = 4 once that gives every SM 16
// warps; with fewer units one row a lane leaves more warps, and the latency of one row, to each
// SM.  kRows = 1 / 4, in us, BF16:
//   tokens            64         256        512        1024       2048        8192
//   40 heads of 128   2.0 / 2.6  2.8 / 3.0  4.1 / 3.6  6.7 / 5.1  12.2 / 8.1  52.4 / 32.1
//   20 heads of 64    1.8 / 2.4  2.0 / 2.5  2.1 / 2.5  2.8 / 3.0   4.1 / 4.2  12.2 / 11.1
template <int DT, int kDim, int kRows>
__global__ void __launch_bounds__(kNormThreads, kNormCtas) dq4_qk_norm_kernel(const NormArgs p) {
  using T = typename Elem<DT>::T;
  constexpr int kLanes = kDim / (2 * V), kGroups = 32 / kLanes;
  wait_for_stream();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int l = lane % kLanes, group = lane / kLanes;
  const int per_token = p.chunks[0] + p.chunks[1];
  const int64_t unit = int64_t(blockIdx.x) * (kNormThreads / 32) + warp;
  const int64_t t = unit >> 32 ? unit / per_token : int64_t(uint32_t(unit) / uint32_t(per_token));
  if (t >= p.tokens) return;
  int c = int(unit - t * per_token);
  const int which = c >= p.chunks[0];
  if (which) c -= p.chunks[0];
  const int h0 = c * (kRows * kGroups) + group;
  const int heads = p.heads[which];
  const LanePlace at = lane_place<V>(l, p.cos ? p.rotary : 0, p.interleaved);
  const T* x = static_cast<const T*>(p.x[which]) + t * p.token_stride[which];
  Raw<DT, V> ra[kRows], rb[kRows];
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int h = min(h0 + i * kGroups, heads - 1);
    const T* row = x + h * p.head_stride[which];
    ra[i] = load_group_once<DT, V>(row + at.a);
    rb[i] = load_group_once<DT, V>(row + at.b);
  }
  const bool normed = p.w[which] != nullptr;
  Vals<V> w = {};
  if (normed) {
    const T* from = static_cast<const T*>(p.w[which]);
    w = widen<DT, V>(load_group<DT, V>(from + at.a), load_group<DT, V>(from + at.b));
  }
  const int64_t row = table_row(p, t);
  const Turn turn = load_turn(p, at.turned, row, l);
  T* out = static_cast<T*>(p.out[which]) + (t * heads + h0) * kDim;
  auto rows = [&](auto interleaved) {
    constexpr bool kInterleaved = decltype(interleaved)::value;
    float wc[2 * V], ws[2 * V];
#pragma unroll
    for (int j = 0; j < 2 * V; ++j) {
      const int e = turn_entry<kInterleaved, V>(j);
      const float s = w.v[partner<kInterleaved, V>(j)] * turn.s[e];
      wc[j] = at.turned ? w.v[j] * turn.c[e] : w.v[j];
      ws[j] = turn_adds<kInterleaved, V>(j) ? s : -s;
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      Vals<V> v = widen<DT, V>(ra[i], rb[i]);
      if (normed) {
        float ss = 0.f;
#pragma unroll
        for (int j = 0; j < 2 * V; ++j) ss = fmaf(v.v[j], v.v[j], ss);
        const float r = rsqrtf(group_sum<kLanes>(ss) * (1.f / kDim) + p.eps);
        Vals<V> y;
#pragma unroll
        for (int j = 0; j < 2 * V; ++j) {
          y.v[j] = v.v[j] * wc[j];
          if (at.turned) y.v[j] = fmaf(v.v[partner<kInterleaved, V>(j)], ws[j], y.v[j]);
          y.v[j] *= r;
        }
        v = y;
      } else if (at.turned) {
        v = turned<kInterleaved, false>(v, turn.c, turn.s);
      }
      if (h0 + i * kGroups >= heads) continue;
      if (row < 0) {
        v = Vals<V>{};
        if (l == 0 && p.bad) atomicAdd(p.bad, 1);
      }
      store_group<DT, V>(out + i * (kGroups * kDim) + at.a, narrow<DT, V>(v, 0));
      store_group<DT, V>(out + i * (kGroups * kDim) + at.b, narrow<DT, V>(v, 1));
    }
  };
  if (p.interleaved) {
    rows(std::true_type{});
  } else {
    rows(std::false_type{});
  }
}

// Column i of the sum of the n rows of `cols` floats at src, in order, kAhead loads at a time.
__device__ __forceinline__ float sum_rows(const float* src, int n, int cols) {
  constexpr int kAhead = 16;
  float s = 0.f;
  for (int c0 = 0; c0 < n; c0 += kAhead) {
    float v[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) v[k] = c0 + k < n ? load_l2(src + int64_t(c0 + k) * cols) : 0.f;
#pragma unroll
    for (int k = 0; k < kAhead; ++k) s += v[k];
  }
  return s;
}

// Sum the CTAs' partial weight gradients (`mine`, [2][dim]): the last CTA of each kPartGroup to
// leave its own sums the group's, and the last group's the groups', always in CTA order.  (One
// CTA summing all of them took 12 us for 304 partials.)
__device__ void finish_weights(const NormArgs& p, const float* mine) {
  __shared__ bool last;
  const int cols = 2 * p.dim, group = blockIdx.x / kPartGroup;
  const int groups = (gridDim.x + kPartGroup - 1) / kPartGroup;
  const int members = min(kPartGroup, int(gridDim.x) - group * kPartGroup);
  float* part = p.part + int64_t(blockIdx.x) * cols;
  float* sums = p.part + int64_t(kMaxPartials) * cols;  // the groups'
  for (int i = threadIdx.x; i < cols; i += blockDim.x) part[i] = mine[i];
  for (int level = 0; level < 2; ++level) {
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) {
      int* count = p.count + (level == 0 ? 1 + group : 0);
      last = atomicAdd(count, 1) == (level == 0 ? members : groups) - 1;
      if (last) *count = 0;  // ready for the next call
    }
    __syncthreads();
    if (!last) return;
    __threadfence();
    for (int i = threadIdx.x; i < cols; i += blockDim.x) {
      if (level == 0) {
        sums[int64_t(group) * cols + i] =
            sum_rows(p.part + int64_t(group) * kPartGroup * cols + i, members, cols);
      } else {
        const float s = sum_rows(sums + i, groups, cols);
        float* dw = p.dw[i >= p.dim];
        if (dw) dw[i >= p.dim ? i - p.dim : i] = s;
      }
    }
  }
}

// The backward pass in the forward kernel's layout: first all of q's units, then k's.  A warp
// walks them with a fixed stride, all of a unit's loads on the way at once, and keeps, in each
// lane, the sums of its columns of the weight's gradient; lanes, warps and CTAs are then summed
// in a fixed order.  With r the row's factor and m' = mean(g w x),
//   dx = r g w - x r^3 m',   dw += r g x
// so that both sums over a row, of x^2 and of g w x, go through the lanes together.
template <int DT, int kDim, int kRows>
__global__ void __launch_bounds__(kBwdThreads, kBwdCtas)
    dq4_qk_norm_backward_kernel(const NormArgs p) {
  using T = typename Elem<DT>::T;
  constexpr int kLanes = kDim / (2 * V), kGroups = 32 / kLanes, kWarps = kBwdThreads / 32;
  __shared__ float sums[kWarps * 2 * kDim];
  wait_for_stream();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int l = lane % kLanes, group = lane / kLanes;
  const LanePlace at = lane_place<V>(l, p.cos ? p.rotary : 0, p.interleaved);
  const int64_t unit0 = int64_t(blockIdx.x) * kWarps + warp;
  const int64_t stride = int64_t(gridDim.x) * kWarps;
  const bool normed = p.w[0] != nullptr;
  struct Rows {
    Raw<DT, V> xa[kRows], xb[kRows], ga[kRows], gb[kRows];
  };
#pragma unroll 1
  for (int which = 0; which < 2; ++which) {
    const int heads = p.heads[which], chunks = p.chunks[which];
    Vals<V> dw = {};
    if (heads > 0) {
      const T* x = static_cast<const T*>(p.x[which]);
      const T* dy = static_cast<const T*>(p.dy[which]);
      T* out = static_cast<T*>(p.out[which]);
      const int64_t token_stride = p.token_stride[which], head_stride = p.head_stride[which];
      Vals<V> w = {};
      if (normed) {
        const T* from = static_cast<const T*>(p.w[which]);
        w = widen<DT, V>(load_group<DT, V>(from + at.a), load_group<DT, V>(from + at.b));
      }
      // a unit: head chunk c of token t
      const int64_t t_step = stride / chunks;
      const int c_step = int(stride - t_step * chunks);
      auto load = [&](int64_t t, int c, Rows& r) {
        if (t >= p.tokens) return;
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
          const int h = min((c * kRows + i) * kGroups + group, heads - 1);
          const T* xr = x + t * token_stride + h * head_stride;
          const T* gr = dy + (t * heads + h) * kDim;
          r.xa[i] = load_group_once<DT, V>(xr + at.a);
          r.xb[i] = load_group_once<DT, V>(xr + at.b);
          r.ga[i] = load_group_once<DT, V>(gr + at.a);
          r.gb[i] = load_group_once<DT, V>(gr + at.b);
        }
      };
      int64_t t = unit0 / chunks;
      int c = int(unit0 - t * chunks);
      Rows now;
      load(t, c, now);
      while (t < p.tokens) {
        const int64_t row = table_row(p, t);
        int64_t t2 = t + t_step;
        int c2 = c + c_step;
        if (c2 >= chunks) {
          c2 -= chunks;
          ++t2;
        }
        const Turn turn = load_turn(p, at.turned, row, l);
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
          const int h = (c * kRows + i) * kGroups + group;
          Vals<V> g = widen<DT, V>(now.ga[i], now.gb[i]);
          if (normed) {
            const Vals<V> v = widen<DT, V>(now.xa[i], now.xb[i]);
            if (at.turned)
              g = p.interleaved ? turned<true, true>(g, turn.c, turn.s)
                                : turned<false, true>(g, turn.c, turn.s);
            float ss = 0.f, gwx = 0.f;
            Vals<V> gx;
#pragma unroll
            for (int j = 0; j < 2 * V; ++j) {
              gx.v[j] = g.v[j] * v.v[j];
              ss = fmaf(v.v[j], v.v[j], ss);
              gwx = fmaf(gx.v[j], w.v[j], gwx);
            }
#pragma unroll
            for (int o = kLanes / 2; o > 0; o >>= 1) {
              ss += __shfl_xor_sync(kAllLanes, ss, o);
              gwx += __shfl_xor_sync(kAllLanes, gwx, o);
            }
            const float r = rsqrtf(ss * (1.f / kDim) + p.eps);
            const float m = -(gwx * (1.f / kDim)) * r * r * r;
#pragma unroll
            for (int j = 0; j < 2 * V; ++j) {
              if (h < heads && row >= 0) dw.v[j] = fmaf(gx.v[j], r, dw.v[j]);
              g.v[j] = fmaf(g.v[j] * w.v[j], r, v.v[j] * m);
            }
          } else if (at.turned) {
            g = p.interleaved ? turned<true, true>(g, turn.c, turn.s)
                              : turned<false, true>(g, turn.c, turn.s);
          }
          if (h >= heads) continue;
          if (row < 0) {
            g = Vals<V>{};
            if (l == 0 && p.bad) atomicAdd(p.bad, 1);
          }
          T* o = out + (t * heads + h) * kDim;
          store_group_once<DT, V>(o + at.a, narrow<DT, V>(g, 0));
          store_group_once<DT, V>(o + at.b, narrow<DT, V>(g, 1));
        }
        t = t2;
        c = c2;
        load(t, c, now);
      }
    }
    if (p.dw[0] == nullptr) continue;
#pragma unroll
    for (int j = 0; j < 2 * V; ++j) {
#pragma unroll
      for (int o = kLanes; o < 32; o <<= 1) dw.v[j] += __shfl_xor_sync(kAllLanes, dw.v[j], o);
      if (group == 0)
        sums[(warp * 2 + which) * kDim + (j < V ? at.a + j : at.b + j - V)] = dw.v[j];
    }
  }
  if (p.dw[0] == nullptr) return;
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * kDim; i += kBwdThreads) {
    float s = sums[i];
    for (int w = 1; w < kWarps; ++w) s += sums[w * 2 * kDim + i];
    sums[i] = s;
  }
  __syncthreads();
  finish_weights(p, sums);
}

// Any even head size and rotation, any alignment: a warp per head, values lane, lane + 32
// and so on, a value's partner read again from memory (L1).  For shapes that the kernels above
// could take it needs, forward and backward, 25 and 86 us for 5 and 15 (1024 tokens, 40 heads of
// 128, BF16).
template <int DT, bool kBackward>
__global__ void __launch_bounds__(32 * kAnyWarps) dq4_qk_norm_any_kernel(const NormArgs p) {
  using T = typename Elem<DT>::T;
  __shared__ float sums[kBackward ? kAnyWarps * 2 * kMaxDim : 1];
  wait_for_stream();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int all_heads = p.heads[0] + p.heads[1];
  const int64_t rows = p.tokens * all_heads;
  const int half = p.rotary / 2;
  float* mine = sums + (kBackward ? warp * 2 * p.dim : 0);
  if constexpr (kBackward) {
    for (int i = lane; i < 2 * p.dim; i += 32) mine[i] = 0.f;
  }
  for (int64_t r0 = int64_t(blockIdx.x) * kAnyWarps + warp; r0 < rows;
       r0 += int64_t(gridDim.x) * kAnyWarps) {
    const int64_t t = r0 / all_heads;
    int h = int(r0 - t * all_heads);
    const int which = h >= p.heads[0];
    if (which) h -= p.heads[0];
    const T* x = static_cast<const T*>(p.x[which]) + t * p.token_stride[which] +
                 h * p.head_stride[which];
    const int64_t o = (t * p.heads[which] + h) * p.dim;
    const T* dy = kBackward ? static_cast<const T*>(p.dy[which]) + o : nullptr;
    const T* w = static_cast<const T*>(p.w[which]);
    T* out = static_cast<T*>(p.out[which]) + o;
    const int64_t row = table_row(p, t);
    float r = 1.f;
    if (w) {
      float ss = 0.f;
      for (int i = lane; i < p.dim; i += 32) {
        const float v = Elem<DT>::load(x + i);
        ss = fmaf(v, v, ss);
      }
      r = rsqrtf(group_sum<32>(ss) / p.dim + p.eps);
    }
    // value i of the rotated (back: sign < 0) vector whose values f gives
    auto turned = [&](auto f, int i, float sign) {
      if (p.cos == nullptr || i >= p.rotary) return f(i);
      const int j = p.interleaved ? i >> 1 : i % half;
      const bool second = p.interleaved ? i & 1 : i >= half;
      const int pair = p.interleaved ? i ^ 1 : second ? i - half : i + half;
      const float c = load_global(p.cos + row * half + j), s = sign * load_global(p.sin + row * half + j);
      const float v = __fmul_rn(f(i), c), u = __fmul_rn(f(pair), s);
      return second ? __fadd_rn(v, u) : __fsub_rn(v, u);
    };
    if (row < 0) {
      for (int i = lane; i < p.dim; i += 32) out[i] = Elem<DT>::make(0.f);
      if (lane == 0 && p.bad) atomicAdd(p.bad, 1);
      continue;
    }
    if constexpr (!kBackward) {
      auto value = [&](int i) {
        const float v = Elem<DT>::load(x + i);
        return w ? v * r * Elem<DT>::load(w + i) : v;
      };
      for (int i = lane; i < p.dim; i += 32) out[i] = Elem<DT>::make(turned(value, i, 1.f));
    } else {
      auto value = [&](int i) { return Elem<DT>::load(dy + i); };
      float dot = 0.f;
      if (w) {
        for (int i = lane; i < p.dim; i += 32) {
          const float g = turned(value, i, -1.f), xh = Elem<DT>::load(x + i) * r;
          mine[which * p.dim + i] += g * xh;
          dot = fmaf(g * Elem<DT>::load(w + i), xh, dot);
        }
        dot = group_sum<32>(dot) / p.dim;
      }
      for (int i = lane; i < p.dim; i += 32) {
        float g = turned(value, i, -1.f);
        if (w) {
          const float xh = Elem<DT>::load(x + i) * r;
          g = r * fmaf(-xh, dot, g * Elem<DT>::load(w + i));
        }
        out[i] = Elem<DT>::make(g);
      }
    }
  }
  if constexpr (kBackward) {
    if (p.dw[0] == nullptr) return;
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * p.dim; i += 32 * kAnyWarps) {
      float s = sums[i];
      for (int v = 1; v < kAnyWarps; ++v) s += sums[v * 2 * p.dim + i];
      sums[i] = s;
    }
    __syncthreads();
    finish_weights(p, sums);
  }
}

// ------------------------------------------------------------------------ host side
int check_norm(const NormArgs& p, int32_t dtype) {
  if (!valid_dtype(dtype, true)) return DQ4_ERR_DTYPE;
  if (p.tokens < 0) return DQ4_ERR_N;
  if (p.heads[0] < 1 || p.heads[1] < 0 || p.heads[0] > 65536 || p.heads[1] > 65536 ||
      p.dim < 2 || p.dim > kMaxDim || p.dim % 2 != 0)
    return DQ4_ERR_HEADS;
  if ((p.cos == nullptr) != (p.sin == nullptr)) return DQ4_ERR_NULL;
  if (p.cos && (p.rotary < 2 || p.rotary > p.dim || p.rotary % 2 != 0 || p.table_rows < 0))
    return DQ4_ERR_ROTARY;
  if (p.tokens == 0) return DQ4_OK;
  if (p.cos && p.positions == nullptr) return DQ4_ERR_NULL;
  if (p.cos && (misaligned(p.cos, 4) || misaligned(p.sin, 4) || misaligned(p.positions, 8)))
    return DQ4_ERR_ALIGN;
  const uintptr_t es = dtype == DQ4_OUT_F32 ? 4 : 2;
  for (int n = 0; n < 2 && p.heads[n] > 0; ++n) {
    if (!p.x[n] || !p.out[n]) return DQ4_ERR_NULL;
    if ((p.w[0] == nullptr) != (p.w[n] == nullptr)) return DQ4_ERR_NULL;
    if (misaligned(p.x[n], es) || misaligned(p.out[n], es) || misaligned(p.w[n], es))
      return DQ4_ERR_ALIGN;
  }
  if (misaligned(p.bad, 4)) return DQ4_ERR_ALIGN;
  return DQ4_OK;
}

// Whether the kernels that hold a head in groups of V values take this call (see lane_place and
// load_group).
bool in_groups(const NormArgs& p, int32_t dtype, bool backward) {
  if (p.dim != 64 && p.dim != 128 && p.dim != 256) return false;
  if (p.cos && (p.rotary % (2 * V) != 0 || !aligned(p.cos, 16) || !aligned(p.sin, 16)))
    return false;
  const uintptr_t to = V * (dtype == DQ4_OUT_F32 ? 4 : 2);
  for (int n = 0; n < 2 && p.heads[n] > 0; ++n) {
    if (p.token_stride[n] % V != 0 || p.head_stride[n] % V != 0 || !aligned(p.x[n], to) ||
        !aligned(p.out[n], to) || !aligned(p.w[n], to) || (backward && !aligned(p.dy[n], to)))
      return false;
  }
  return true;
}

void cut_heads(NormArgs* p, int rows) {
  p->chunk = rows * 32 / (p->dim / (2 * V));
  for (int n = 0; n < 2; ++n) p->chunks[n] = (p->heads[n] + p->chunk - 1) / p->chunk;
}

template <int DT, int kDim>
int launch_forward(NormArgs p, int sms, cudaStream_t stream) {
  constexpr int kWarps = kNormThreads / 32, kRows = 32 / Raw<DT, V>::kBytes;  // 64 bytes of a lane
  cut_heads(&p, kRows);
  const bool more = p.tokens * (p.chunks[0] + p.chunks[1]) >= int64_t(sms) * 16;
  if (!more) cut_heads(&p, 1);
  const int64_t grid = (p.tokens * (p.chunks[0] + p.chunks[1]) + kWarps - 1) / kWarps;
  if (grid > kMaxGrid) return DQ4_ERR_N;
  return launch_ordered(
      more ? dq4_qk_norm_kernel<DT, kDim, kRows> : dq4_qk_norm_kernel<DT, kDim, 1>,
      dim3(unsigned(grid)), kNormThreads, 0, stream, p);
}

template <int DT, int kDim>
int launch_backward(NormArgs p, int sms, cudaStream_t stream) {
  constexpr int kWarps = kBwdThreads / 32, kRows = 32 / Raw<DT, V>::kBytes;  // 128 bytes of a lane
  cut_heads(&p, kRows);
  const int64_t units = p.tokens * (p.chunks[0] + p.chunks[1]);
  const int64_t want = (units + kWarps - 1) / kWarps;
  const int most = kBwdCtas * sms < kMaxPartials ? kBwdCtas * sms : kMaxPartials;
  return launch_ordered(dq4_qk_norm_backward_kernel<DT, kDim, kRows>,
                        dim3(unsigned(want < most ? want : most)), kBwdThreads, 0, stream, p);
}

template <int DT, int kDim>
int launch_dim(const NormArgs& p, bool backward, int sms, cudaStream_t stream) {
  return backward ? launch_backward<DT, kDim>(p, sms, stream)
                  : launch_forward<DT, kDim>(p, sms, stream);
}

template <int DT>
int launch_norm(const NormArgs& p, bool backward, int sms, cudaStream_t stream) {
  if (!in_groups(p, DT, backward)) {
    const int64_t want = (p.tokens * (p.heads[0] + p.heads[1]) + kAnyWarps - 1) / kAnyWarps;
    const int64_t most = backward ? kMaxPartials : 16 * sms;
    const dim3 grid(unsigned(want < most ? want : most));
    return backward
               ? launch_ordered(dq4_qk_norm_any_kernel<DT, true>, grid, 32 * kAnyWarps, 0, stream, p)
               : launch_ordered(dq4_qk_norm_any_kernel<DT, false>, grid, 32 * kAnyWarps, 0, stream,
                                p);
  }
  switch (p.dim) {
    case 64: return launch_dim<DT, 64>(p, backward, sms, stream);
    case 128: return launch_dim<DT, 128>(p, backward, sms, stream);
    default: return launch_dim<DT, 256>(p, backward, sms, stream);
  }
}

int run_norm(const NormArgs& p, int32_t dtype, bool backward, void* stream) {
  int dev, sms;
  if (const int st = current_device(&dev, &sms)) return st;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  switch (dtype) {
    case DQ4_OUT_F16: return launch_norm<DQ4_OUT_F16>(p, backward, sms, s);
    case DQ4_OUT_BF16: return launch_norm<DQ4_OUT_BF16>(p, backward, sms, s);
    default: return launch_norm<DQ4_OUT_F32>(p, backward, sms, s);
  }
}

}  // namespace
}  // namespace dq4d

using namespace dq4d;

extern "C" {

int dq4_qk_norm_rope(const void* q, int64_t q_token_stride, int64_t q_head_stride, const void* k,
                     int64_t k_token_stride, int64_t k_head_stride, int32_t dtype,
                     int64_t tokens, int32_t q_heads, int32_t k_heads, int32_t head_dim,
                     const void* q_weight, const void* k_weight, float eps, const float* cos,
                     const float* sin, int64_t table_rows, int32_t rotary, int32_t interleaved,
                     const int64_t* positions, void* q_out, void* k_out, int* bad,
                     void* stream) {
  NormArgs p = {{q, k}, {}, {q_token_stride, k_token_stride}, {q_head_stride, k_head_stride},
                {q_weight, k_weight}, {q_out, k_out}, {q_heads, k_heads}, tokens, eps, cos, sin,
                table_rows, head_dim, rotary, interleaved != 0, positions, bad};
  if (const int st = check_norm(p, dtype)) return st;
  if (tokens == 0) return DQ4_OK;
  return run_norm(p, dtype, false, stream);
}

int64_t dq4_qk_norm_rope_backward_workspace_bytes(int32_t head_dim) {
  if (head_dim < 2 || head_dim > kMaxDim) return 0;
  return 256 + int64_t(kMaxPartials + kMaxGroups) * 2 * head_dim * 4;
}

int dq4_qk_norm_rope_backward(const void* dq_out, const void* dk_out, const void* q,
                              int64_t q_token_stride, int64_t q_head_stride, const void* k,
                              int64_t k_token_stride, int64_t k_head_stride, int32_t dtype,
                              int64_t tokens, int32_t q_heads, int32_t k_heads,
                              int32_t head_dim, const void* q_weight, const void* k_weight,
                              float eps, const float* cos, const float* sin,
                              int64_t table_rows, int32_t rotary, int32_t interleaved,
                              const int64_t* positions, void* dq, void* dk, float* dq_weight,
                              float* dk_weight, void* workspace, int64_t workspace_bytes,
                              int* bad, void* stream) {
  NormArgs p = {{q, k}, {dq_out, dk_out}, {q_token_stride, k_token_stride},
                {q_head_stride, k_head_stride}, {q_weight, k_weight}, {dq, dk},
                {q_heads, k_heads}, tokens, eps, cos, sin, table_rows, head_dim, rotary,
                interleaved != 0, positions, bad};
  if (const int st = check_norm(p, dtype)) return st;
  const uintptr_t es = dtype == DQ4_OUT_F32 ? 4 : 2;
  for (int n = 0; n < 2 && p.heads[n] > 0; ++n) {
    if (tokens > 0 && !p.dy[n]) return DQ4_ERR_NULL;
    if (misaligned(p.dy[n], es)) return DQ4_ERR_ALIGN;
  }
  if (q_weight) {
    // k_heads == 0 leaves dk_weight's place unused; its sums are zero
    if (!dq_weight || (k_heads > 0 && !dk_weight)) return DQ4_ERR_NULL;
    if (misaligned(dq_weight, 4) || misaligned(dk_weight, 4)) return DQ4_ERR_ALIGN;
    if (!workspace || workspace_bytes < dq4_qk_norm_rope_backward_workspace_bytes(head_dim))
      return DQ4_ERR_WORKSPACE;
    if (misaligned(workspace, 256)) return DQ4_ERR_ALIGN;
    p.dw[0] = dq_weight;
    p.dw[1] = dk_weight;
    p.count = static_cast<int*>(workspace);
    p.part = reinterpret_cast<float*>(static_cast<char*>(workspace) + 256);
  }
  if (tokens == 0) {
    if (!q_weight) return DQ4_OK;
    int dev, sms;
    if (const int st = current_device(&dev, &sms)) return st;
    for (int n = 0; n < 2; ++n) {
      if (!p.dw[n]) continue;
      const cudaError_t e = cudaMemsetAsync(p.dw[n], 0, size_t(head_dim) * 4,
                                            static_cast<cudaStream_t>(stream));
      if (e != cudaSuccess) return fail_cuda(DQ4_ERR_LAUNCH, e);
    }
    return DQ4_OK;
  }
  return run_norm(p, dtype, true, stream);
}

}  // extern "C"
