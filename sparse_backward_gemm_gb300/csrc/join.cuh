// What the forward and the backward of the residual join share: a group of
// threads owns one row at a time, the rows' tensors arrive ahead through a
// ring in shared memory (bulk copies counted on an mbarrier a stage), and row
// sums go through the group.
#pragma once

#include "internal.h"
#include "q8.cuh"
#include "tc_ptx.cuh"

namespace collider {
namespace join {

constexpr int kThreads = 256;   // of a CTA, at most
constexpr int kMaxWarps = 8;    // of a row group
constexpr int kMaxStages = 8;

// one row of a tensor, contiguous and 16-byte aligned, into this CTA's shared memory
__device__ __forceinline__ void copy_row(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}

// Two f32 values a register pair, and the Blackwell arithmetic on pairs: a
// product or sum of both halves in one instruction, each rounded to nearest.
typedef float2 f2;
__device__ __forceinline__ uint64_t bits(f2 a) { return *reinterpret_cast<uint64_t*>(&a); }
__device__ __forceinline__ f2 pair(uint64_t u) { return *reinterpret_cast<f2*>(&u); }
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(bits(a)), "l"(bits(b)), "l"(bits(c)));
  return pair(d);
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(bits(a)), "l"(bits(b)));
  return pair(d);
}
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(bits(a)), "l"(bits(b)));
  return pair(d);
}
__device__ __forceinline__ f2 both(float a) { return make_float2(a, a); }

// 8 consecutive values as four pairs, and back
struct Vec8 {
  f2 v[4];
};
__device__ __forceinline__ f2 widen(uint32_t u) {
  return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}
template <typename T>
__device__ __forceinline__ Vec8 get8(const void* p) {
  Vec8 r;
  if constexpr (sizeof(T) == 2) {
    const uint4 u = *static_cast<const uint4*>(p);
    r.v[0] = widen(u.x); r.v[1] = widen(u.y); r.v[2] = widen(u.z); r.v[3] = widen(u.w);
  } else {
    const float4 a = static_cast<const float4*>(p)[0], b = static_cast<const float4*>(p)[1];
    r.v[0] = make_float2(a.x, a.y); r.v[1] = make_float2(a.z, a.w);
    r.v[2] = make_float2(b.x, b.y); r.v[3] = make_float2(b.z, b.w);
  }
  return r;
}
template <typename T>
__device__ __forceinline__ void put8(T* p, const Vec8& a) {
  if constexpr (sizeof(T) == 2) {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(a.v[0].x, a.v[0].y), pack_bf16x2(a.v[1].x, a.v[1].y),
                                              pack_bf16x2(a.v[2].x, a.v[2].y), pack_bf16x2(a.v[3].x, a.v[3].y));
  } else {
    reinterpret_cast<float4*>(p)[0] = make_float4(a.v[0].x, a.v[0].y, a.v[1].x, a.v[1].y);
    reinterpret_cast<float4*>(p)[1] = make_float4(a.v[2].x, a.v[2].y, a.v[3].x, a.v[3].y);
  }
}
// stores a as T and returns the values as they are stored
template <typename T>
__device__ __forceinline__ Vec8 put8_stored(T* p, bool on, const Vec8& a) {
  if constexpr (sizeof(T) == 2) {
    const uint4 u = make_uint4(pack_bf16x2(a.v[0].x, a.v[0].y), pack_bf16x2(a.v[1].x, a.v[1].y),
                               pack_bf16x2(a.v[2].x, a.v[2].y), pack_bf16x2(a.v[3].x, a.v[3].y));
    if (on) *reinterpret_cast<uint4*>(p) = u;
    Vec8 r;
    r.v[0] = widen(u.x); r.v[1] = widen(u.y); r.v[2] = widen(u.z); r.v[3] = widen(u.w);
    return r;
  } else {
    if (on) put8(p, a);
    return a;
  }
}
__device__ __forceinline__ Vec8 all8(float a) {
  Vec8 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) r.v[i] = both(a);
  return r;
}
__device__ __forceinline__ void prefetch_l1(const void* p, bool there) {
  if (there) asm volatile("prefetch.global.L1 [%0];" ::"l"(p) : "memory");
}
// a parameter vector's 8 values at v: `none` where there is no such parameter,
// 0 beyond the row
template <typename T>
__device__ __forceinline__ Vec8 param8(const void* p, int v, bool on, float none) {
  if (!on) return all8(0.f);
  return p ? get8<T>(static_cast<const T*>(p) + 8 * v) : all8(none);
}

// This thread's place: warps a row group, its group in the CTA, its lane in the group.
struct Place {
  int warps, group, lane;   // lane: 0 .. 32 * warps - 1
  __device__ Place(int tpr) : warps(tpr >> 5), group(threadIdx.x / tpr), lane(threadIdx.x % tpr) {}
  __device__ void sync() const {
    if (warps == 1) __syncwarp();
    else tc::named_bar(1 + group, 32 * warps);
  }
};

// Sum of 4 values (2, 1) over a warp: lanes 0, 8, 16, 24 (0, 16; all) end with
// the sums of values 0, 1, 2, 3.  Each step halves the values a lane carries
// while there are several, so 4 values take 6 shuffles instead of 20.
template <int NV>
__device__ __forceinline__ float warp_sums(const float (&v)[NV], int lane) {
  static_assert(NV == 1 || NV == 2 || NV == 4, "");
  float a = v[0];
  if (NV == 4) {
    const bool hi = lane & 16;
    const float k0 = (hi ? v[NV == 4 ? 2 : 0] : v[0]) + __shfl_xor_sync(0xffffffffu, hi ? v[0] : v[NV == 4 ? 2 : 0], 16);
    const float k1 = (hi ? v[NV == 4 ? 3 : 0] : v[NV == 4 ? 1 : 0]) +
                     __shfl_xor_sync(0xffffffffu, hi ? v[NV == 4 ? 1 : 0] : v[NV == 4 ? 3 : 0], 16);
    const bool lo = lane & 8;
    a = (lo ? k1 : k0) + __shfl_xor_sync(0xffffffffu, lo ? k0 : k1, 8);
  } else if (NV == 2) {
    const bool hi = lane & 16;
    a = (hi ? v[NV == 2 ? 1 : 0] : v[0]) + __shfl_xor_sync(0xffffffffu, hi ? v[0] : v[NV == 2 ? 1 : 0], 16);
    a += __shfl_xor_sync(0xffffffffu, a, 8);
  } else {
    a += __shfl_xor_sync(0xffffffffu, a, 16);
    a += __shfl_xor_sync(0xffffffffu, a, 8);
  }
  a += __shfl_xor_sync(0xffffffffu, a, 4);
  a += __shfl_xor_sync(0xffffffffu, a, 2);
  a += __shfl_xor_sync(0xffffffffu, a, 1);
  return a;
}
// Sums over the group, the same bits in every thread (lanes by a fixed
// butterfly, then the warps in order).  `red` holds two halves of 4 kMaxWarps
// floats of the group, zero where there is no warp; the halves alternate, so
// one barrier a sum is enough: who writes a half again has passed the barrier
// of the sum between, which every thread reached after reading it.
template <int NV>
__device__ __forceinline__ void group_sum(const Place& pl, float* red, int& half, float (&v)[NV]) {
  constexpr int kEvery = 32 / NV;   // lanes that hold a sum
  const int lane = pl.lane & 31;
  const float a = warp_sums(v, lane);
  if (pl.warps == 1) {
    __syncwarp();
#pragma unroll
    for (int k = 0; k < NV; ++k) v[k] = __shfl_sync(0xffffffffu, a, k * kEvery);
    return;
  }
  float* r = red + half * 4 * kMaxWarps;
  half ^= 1;
  if (lane % kEvery == 0) r[(pl.lane >> 5) * NV + lane / kEvery] = a;
  pl.sync();
  // [warp][NV] floats: 4 / NV warps a vector
  float4 t = *reinterpret_cast<const float4*>(r);
#pragma unroll
  for (int w = 4 / NV; w < kMaxWarps; w += 4 / NV)
    if (w < pl.warps) {
      const float4 q = *reinterpret_cast<const float4*>(r + w * NV);
      t.x += q.x; t.y += q.y; t.z += q.z; t.w += q.w;
    }
  if (NV == 4) {
    v[0] = t.x; v[NV == 4 ? 1 : 0] = t.y; v[NV == 4 ? 2 : 0] = t.z; v[NV == 4 ? 3 : 0] = t.w;
  } else if (NV == 2) {
    v[0] = t.x + t.z; v[NV == 2 ? 1 : 0] = t.y + t.w;
  } else {
    v[0] = (t.x + t.y) + (t.z + t.w);
  }
}

// Launch shape: threads a row, row groups a CTA, ring stages.
struct Shape {
  int vpt, tpr, groups, stages;
  uint32_t stage_bytes;
  size_t smem;
};
// smem: [groups][2][4 kMaxWarps] floats | barriers | abort flag | 32 bytes of zeros | extra | rings
constexpr size_t kRedBytes = 2 * 4 * kMaxWarps * sizeof(float);
__host__ __device__ inline size_t zero_at(int groups) { return (groups * (kRedBytes + kMaxStages * 8) + 8 + 31) & ~size_t(31); }
__host__ __device__ inline size_t head_bytes(int groups) { return (zero_at(groups) + 32 + 127) & ~size_t(127); }
// A row is at most kThreads threads', of `vpt` vectors of 8 each; narrow rows
// share a CTA.  extra: bytes of shared memory beside the ring, which takes
// what is left of the budget, one stage at least.
inline Shape make_shape(int D, int vpt, uint32_t row_bytes, size_t extra, size_t budget) {
  Shape s{};
  s.vpt = vpt;
  const int warps = (D / 8 + 32 * vpt - 1) / (32 * vpt);
  s.tpr = 32 * warps;
  s.groups = kThreads / s.tpr;
  s.stage_bytes = (row_bytes + 127) & ~127u;
  const size_t head = head_bytes(s.groups) + extra;
  const size_t n = budget > head ? (budget - head) / ((size_t)s.groups * s.stage_bytes) : 1;
  s.stages = (int)(n < 1 ? 1 : n > kMaxStages ? kMaxStages : n);
  s.smem = head + (size_t)s.groups * s.stages * s.stage_bytes;
  return s;
}

// Opts kernel k in to `bytes` of dynamic shared memory on the current device,
// once for each larger amount (`granted`: the kernel's own table).
inline cudaError_t grant_smem(const void* k, size_t bytes, size_t (&granted)[64]) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || bytes <= 48 * 1024 || granted[dev & 63] >= bytes) return e;
  e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (e == cudaSuccess) granted[dev & 63] = bytes;
  return e;
}

// Lets this group's copies still in flight land (bounded) after a wait gave up.
__device__ __forceinline__ void drain(uint32_t bars, int stages, uint32_t parities) {
  for (int s = 0; s < stages; ++s) {
    const uint64_t t0 = globaltimer_ns();
    while (!tc::mbar_try(bars + 8 * s, (parities >> s) & 1u) && globaltimer_ns() - t0 < 10000000ull) {
    }
  }
}

}  // namespace join
}  // namespace collider
