// What the kernels of the layers with 8-bit weights share (dq4_int8.h): codes as FP16, the FP16
// tensor-core product of a warp, and the streaming of weights past few tokens.
//
// The integer tensor-core rate of this GPU is far below its FP16 rate, and codes are exact in
// FP16, so products of codes are FP16 products with FP32 sums: exact while sums are below 2^24.
#pragma once

#include "attn.cuh"
#include "dq4_int8.h"
#include "tcgen05.cuh"
#include "tmap.cuh"

namespace dq4d {
namespace {

constexpr float kRecip127 = 0.007874015718698502f;  // RN32(1 / 127)
constexpr int kMaxOutliers = 128;
constexpr int64_t kInt8Counters = 4096;  // bytes of counters at the head of a workspace

// Four codes as FP16 pairs: 1152 is taken from 1024 + 128 + code, both exact.
__device__ __forceinline__ void codes_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  const uint32_t u = w ^ 0x80808080u;
  const __half2 off = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));
  uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
  __half2 x, y;
  memcpy(&x, &a, 4);
  memcpy(&y, &b, 4);
  x = __hsub2(x, off);
  y = __hsub2(y, off);
  memcpy(&lo, &x, 4);
  memcpy(&hi, &y, 4);
}

// D += A B, 16 x 16 by 16 x 8, FP16 with FP32 sums.
__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                          uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}


// ------------------------------------------------- products of weight rows and few tokens
// Warps take jobs (16 RT weight rows, 8 NT tokens) in turn: alone, or 2, 4 or 8 of a CTA together
// (a group), which then take turns at the chunks of 128 of K and add their sums at the end.  The
// order of K inside a product is free: lane (g, c) = (lane / 4, lane % 4) takes 32 consecutive
// codes of rows g and g + 8 of each 16, and the same places of token g of each 8, and eight
// products take them four at a time.  The weights come by TMA into a ring of the warp's own in
// shared memory, kDepth chunks ahead, across the ends of jobs (lane 0 issues, all lanes consume);
// the tokens, which every job reads, from L2 into registers, a chunk ahead.  Nothing else
// synchronizes warps before a job's end.
// A job starts at a chunk of its own, so that warps do not go through the tokens side by side and
// queue at single lines of L2.
// (Measured for one token at 11008 x 4096, 10.4 us for reading the weight alone: rows of 128 bytes
// in a box @@ us; of 64 bytes 23.7, as the TMA takes about 3.5 cycles for a row whatever its width,
// tokens by TMA included; copies of 16 bytes a lane, cp.async, 13.4.)
//
// kBoxes: boxes of weight rows of a chunk, 16 RT / kBoxes rows each.  kWords: 16-byte words of a
// token's 32 values, 2 (codes) or 4 (FP16).
// Jobs:
//   places(job, y)          the first row of each box of weights
//   tokens(job, tok)        this lane's token of each 8 (for one that is not there any other, whose
//                           results are not used), advanced to its 32 c
//   scales(job, k, f)       for FP16 tokens that have them: the factor of values k .. k + 15
//   start()                 once, when the first copies are on their way
//   begin(job, t)           before a job's products, thread t of its group
//   finish(job, part, ...)  the group's sums (sum(part, warps, token, row)), thread t of `threads`

// A load whose place among the others is kept: ahead of its use.
__device__ __forceinline__ float load_ahead(const float* p) {
  float v;
  asm volatile("ld.global.f32 %0, [%1];" : "=f"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ uint4 load_ahead(const uint4* p) {
  uint4 v;
  asm volatile("ld.global.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p) : "memory");
  return v;
}

constexpr int kStreamWarps = 8, kStreamThreads = 32 * kStreamWarps;
constexpr int kChunk = 128;

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

// kScaled: tokens have factors (Jobs::scales), one for each 16 values.
template <int RT, int NT, int kBoxes, int kWords, bool kScaled, int kDepth>
struct Streamed {
  static constexpr int kStage = RT * 16 * kChunk;
  static constexpr int kPart = RT * 16 * NT * 8;  // sums of a warp
  static constexpr int kBarsAt = kStreamWarps * kDepth * kStage;
  static constexpr int kPartsAt = kBarsAt + kStreamWarps * kDepth * 8;
  static constexpr int kBytes = kPartsAt + kStreamWarps * kPart * 4;  // + 1024 to align
  static constexpr int kFactors = kScaled ? NT * 2 : 1;

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
    // ---- the tokens: those of the next chunk
    const uint8_t* tok[NT];
    uint4 x[NT][kWords];
    float f[kFactors];
    int64_t tok_job = mine > 0 ? first : all;
    int tok_chunk = 0, tok_left = mine;
    auto tok_open = [&] {
      if (tok_job >= all) return;
      jobs.tokens(tok_job, tok);
      tok_chunk = start_of(tok_job);
    };
    tok_open();
    auto fetch = [&] {
      if (tok_job >= all) return;
      const int64_t k = int64_t(member + tok_chunk * group) * kChunk;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < kWords; ++i) {
          x[nt][i] = make_uint4(0, 0, 0, 0);  // (past the end)
          if (k + 32 * c + i * (32 / kWords) < K)
            x[nt][i] = load_ahead(reinterpret_cast<const uint4*>(tok[nt] + k * (kWords / 2)) + i);
        }
      if constexpr (kScaled) jobs.scales(tok_job, k + 32 * c, f);
      if (++tok_chunk == mine) tok_chunk = 0;
      if (--tok_left == 0) {
        tok_left = mine;
        tok_job += stride;
        tok_open();
      }
    };
    fetch();
    jobs.start();
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
      float acc[RT][NT][4] = {};
#pragma unroll 1
      for (int i = 0; i < mine && ok; ++i) {
        // the tokens' operand words, which frees the registers for the next chunk's
        uint32_t b[NT][8][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const uint32_t* xw = reinterpret_cast<const uint32_t*>(x[nt]);
#pragma unroll
          for (int s = 0; s < 8; ++s) {
            if constexpr (kWords == 2) {
              codes_f16(xw[s], b[nt][s][0], b[nt][s][1]);
            } else {
              b[nt][s][0] = xw[2 * s];
              b[nt][s][1] = xw[2 * s + 1];
              if constexpr (kScaled) {
                const __half2 by = __float2half2_rn(f[2 * nt + (s >> 2)]);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                  __half2 v;
                  memcpy(&v, &b[nt][s][h], 4);
                  v = __hmul2(v, by);
                  memcpy(&b[nt][s][h], &v, 4);
                }
              }
            }
          }
        }
        fetch();
        ok = __all_sync(kAllLanes, mbar_wait(bars + 8 * slot, phase));
        if (!ok) break;
        const uint32_t at = ring + slot * kStage;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          // 128-byte rows, their 16-byte pieces in place i ^ row % 8
          uint4 w[RT][2];
#pragma unroll
          for (int rt = 0; rt < RT; ++rt)
#pragma unroll
            for (int h = 0; h < 2; ++h)
              w[rt][h] = lds_v4(at + (16 * rt + 8 * h + g) * kChunk + (((2 * c + half) ^ g) << 4));
#pragma unroll
          for (int s = 0; s < 4; ++s)
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
              uint32_t a[4];
              codes_f16(reinterpret_cast<const uint32_t*>(&w[rt][0])[s], a[0], a[2]);
              codes_f16(reinterpret_cast<const uint32_t*>(&w[rt][1])[s], a[1], a[3]);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
                mma_16816(acc[rt][nt], a[0], a[1], a[2], a[3], b[nt][4 * half + s][0],
                          b[nt][4 * half + s][1]);
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
      for (int rt = 0; rt < RT; ++rt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            to[place(8 * nt + 2 * c + (i & 1), 16 * rt + 8 * (i >> 1) + g)] = acc[rt][nt][i];
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
    return token * (16 * RT) + (row ^ (token >> 1 & 3) * 8 % (16 * RT));
  }
  static __device__ __forceinline__ float sum(const float* part, int warps, int token, int row) {
    float v = 0.f;
    for (int w = 0; w < warps; ++w) v += part[w * kPart + place(token, row)];
    return v;
  }
};

__device__ __forceinline__ uint8_t* aligned_1024(uint8_t* p) {
  return reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(p) + 1023) & ~uintptr_t(1023));
}

// A matrix's map for TMA: boxes of box_w x box_h values, swizzled.
inline int encode_2d(CUtensorMap* map, CUtensorMapDataType type, const void* base, int64_t width,
                     int64_t height, int64_t stride_bytes, int box_w, int box_h,
                     CUtensorMapSwizzle swizzle) {
  const EncodeTiled encode = tensor_map_encoder();
  if (!encode) return fail_cuda(DQ4_ERR_LAUNCH, cudaErrorNotSupported);
  const cuuint64_t size[2] = {cuuint64_t(width), cuuint64_t(height)};
  const cuuint64_t stride[1] = {cuuint64_t(stride_bytes)};
  const cuuint32_t box[2] = {cuuint32_t(box_w), cuuint32_t(box_h)};
  const cuuint32_t step[2] = {1, 1};
  const CUresult r = encode(map, type, 2, const_cast<void*>(base), size, stride, box, step,
                            CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
                            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? DQ4_OK : fail_cuda(DQ4_ERR_LAUNCH, cudaErrorInvalidValue);
}

template <typename T>
__device__ __forceinline__ float load_half(const void* p, int64_t i) {
  return float(static_cast<const T*>(p)[i]);
}
__device__ __forceinline__ float load_16(const void* p, int64_t i, bool bf16) {
  return bf16 ? load_half<__nv_bfloat16>(p, i) : load_half<__half>(p, i);
}
__device__ __forceinline__ float load_any(const void* p, int64_t i, int dtype) {
  return dtype == DQ4_OUT_F32 ? static_cast<const float*>(p)[i]
                              : load_16(p, i, dtype == DQ4_OUT_BF16);
}
__device__ __forceinline__ void store_any(void* p, int64_t i, float f, int dtype) {
  if (dtype == DQ4_OUT_F32) store_one<DQ4_OUT_F32>(p, i, f);
  else if (dtype == DQ4_OUT_BF16) store_one<DQ4_OUT_BF16>(p, i, f);
  else store_one<DQ4_OUT_F16>(p, i, f);
}

}  // namespace

// The arguments of the two product kernels.
struct Int8Linear {
  const int8_t* codes;  // [M][K]
  const float* scales;
  const int8_t* CB;  // [N][K]
  const float* SCB;
  int64_t M, N, K;
  const int64_t* cols;  // [L]
  const void* outliers;  // [M][L]
  int L;
  bool outliers_bf16;
  const void* bias;
  int out_dtype;
  void* Y;
  int* bad;
};

}  // namespace dq4d
