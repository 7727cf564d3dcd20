// What the forward and the backward of the residual join share: a group of
// threads owns one row at a time, each thread the same columns of every row;
// the rows' tensors arrive ahead through a ring in shared memory, every thread
// copying (cp.async) and reading its own columns only, so that the ring needs
// no barrier; row sums go through the group.
//
// Streaming 8192 rows of four 4 KB tensors through such a ring took 22.9 us
// (5.9 TB/s) with one CTA an SM; bulk copies of whole rows counted on an
// mbarrier took 31 us issued by an elected lane of a converged warp, 66 us by a
// lone lane, 0.2 us for each copy.
#pragma once

#include <mutex>

#include "internal.h"
#include "q8.cuh"
#include "tc_ptx.cuh"

namespace collider {
namespace join {

constexpr int kThreads = 512;   // of a CTA, at most
constexpr int kMaxWarps = 16;   // of a row group
constexpr int kMaxStages = 6;
constexpr int kMaxSums = 16;    // of a row at a time

// asynchronous copies into this thread's own places of the ring
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy8(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// until at most n of this thread's committed groups are under way
__device__ __forceinline__ void copy_wait(int n) {
  switch (n) {
    case 0: asm volatile("cp.async.wait_group 0;" ::: "memory"); break;
    case 1: asm volatile("cp.async.wait_group 1;" ::: "memory"); break;
    case 2: asm volatile("cp.async.wait_group 2;" ::: "memory"); break;
    case 3: asm volatile("cp.async.wait_group 3;" ::: "memory"); break;
    case 4: asm volatile("cp.async.wait_group 4;" ::: "memory"); break;
    default: asm volatile("cp.async.wait_group 5;" ::: "memory"); break;
  }
}
// 8 values of T
template <typename T>
__device__ __forceinline__ void copy_vec(uint32_t dst, const T* src) {
  copy16(dst, src);
  if (sizeof(T) == 4) copy16(dst + 16, src + 4);
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
// 8 values as they are stored
template <typename T>
struct Raw8 {
  uint4 u[sizeof(T) / 2];
};
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

// Sums of NV values (a power of two) over a warp: lane l ends with the sum of
// value l / (32 / NV).  Each step halves the values a lane carries while there
// are several, so 4 values take 6 shuffles instead of 20.
template <int NV>
__device__ __forceinline__ float warp_sums(float (&v)[NV], int lane) {
  int off = 16;
#pragma unroll
  for (int n = NV; n > 1; n >>= 1, off >>= 1) {
    const bool hi = lane & off;
#pragma unroll
    for (int j = 0; j < n / 2; ++j) {
      const float send = hi ? v[j] : v[j + n / 2];
      v[j] = (hi ? v[j + n / 2] : v[j]) + __shfl_xor_sync(0xffffffffu, send, off);
    }
  }
#pragma unroll
  for (; off > 0; off >>= 1) v[0] += __shfl_xor_sync(0xffffffffu, v[0], off);
  return v[0];
}
// Sums over the group in two halves: each warp leaves its sums in `red` ([kMaxWarps][NV]
// floats of the group); after a barrier of the group every thread adds them in
// warp order, so all get the same bits.
template <int NV>
__device__ __forceinline__ void leave_sums(const Place& pl, float* red, float (&v)[NV]) {
  constexpr int kEvery = 32 / NV;   // lanes that hold a sum
  const int lane = pl.lane & 31;
  const float a = warp_sums(v, lane);
  if (lane % kEvery == 0) red[(pl.lane >> 5) * NV + lane / kEvery] = a;
}
template <int NV>
__device__ __forceinline__ void take_sums(const Place& pl, const float* red, float (&v)[NV]) {
  // (zeros where there is no warp: 8 warps are added without asking)
  constexpr int W = NV >= 4 ? 1 : 4 / NV;   // warps a vector of four floats
#pragma unroll
  for (int k = 0; k < (NV >= 4 ? NV : 4); k += 4) {
    float4 t = *reinterpret_cast<const float4*>(red + k);
    auto add = [&](int w) {
      const float4 q = *reinterpret_cast<const float4*>(red + w * NV + k);
      t.x += q.x; t.y += q.y; t.z += q.z; t.w += q.w;
    };
    if (pl.warps > 1) {
#pragma unroll
      for (int w = W; w < 8; w += W) add(w);
    }
    if (pl.warps > 8) {
#pragma unroll
      for (int w = 8; w < kMaxWarps; w += W) add(w);
    }
    if constexpr (NV >= 4) {
      v[k] = t.x; v[k + 1] = t.y; v[k + 2] = t.z; v[k + 3] = t.w;
    } else {
      v[0] = NV == 2 ? t.x + t.z : (t.x + t.y) + (t.z + t.w);
      if (NV == 2) v[NV - 1] = t.y + t.w;
    }
  }
}
// A sum at once.  The halves of `red` alternate, so one barrier a sum is enough:
// who writes a half again has passed the barrier of the sum between, which every
// thread reached after reading it.
template <int NV>
__device__ __forceinline__ void group_sum(const Place& pl, float* red, int& half, float (&v)[NV]) {
  float* r = red + half * kMaxSums * kMaxWarps;
  half ^= 1;
  leave_sums(pl, r, v);
  pl.sync();
  take_sums(pl, r, v);
}

// Launch shape: threads a row, row groups a CTA, ring stages.
struct Shape {
  int vpt, tpr, groups, stages;
  uint32_t stage_bytes;
  size_t smem;
};
// smem: [groups][2][kMaxWarps][kMaxSums] floats | 32 bytes of zeros | extra | rings
constexpr size_t kRedBytes = 2 * kMaxSums * kMaxWarps * sizeof(float);
__host__ __device__ inline size_t zero_at(int groups) { return groups * kRedBytes; }
__host__ __device__ inline size_t head_bytes(int groups) { return (zero_at(groups) + 32 + 127) & ~size_t(127); }
// A row is at most kThreads threads', of `vpt` vectors of 8 each; narrow rows
// share a CTA of 256.  extra: bytes of shared memory beside the ring, which takes
// what is left of the budget, one stage at least.
inline Shape make_shape(int D, int vpt, uint32_t row_bytes, size_t extra, size_t budget) {
  Shape s{};
  s.vpt = vpt;
  const int warps = (D / 8 + 32 * vpt - 1) / (32 * vpt);
  s.tpr = 32 * warps;
  s.groups = s.tpr >= 256 ? 1 : 256 / s.tpr;
  s.stage_bytes = (row_bytes + 127) & ~127u;
  const size_t head = head_bytes(s.groups) + extra;
  const size_t n = budget > head ? (budget - head) / ((size_t)s.groups * s.stage_bytes) : 1;
  s.stages = (int)(n < 1 ? 1 : n > kMaxStages ? kMaxStages : n);
  s.smem = head + (size_t)s.groups * s.stages * s.stage_bytes;
  return s;
}

// Opts kernel k in to `bytes` of dynamic shared memory on the current device,
// once for each larger amount (`granted`: the kernel's own table).  The lock keeps
// a second thread's smaller amount from replacing a larger one.
inline cudaError_t grant_smem(const void* k, size_t bytes, size_t (&granted)[64]) {
  static std::mutex lock;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || bytes <= 48 * 1024) return e;
  std::lock_guard<std::mutex> hold(lock);
  if (granted[dev & 63] >= bytes) return e;
  e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (e == cudaSuccess) granted[dev & 63] = bytes;
  return e;
}

}  // namespace join
}  // namespace collider
