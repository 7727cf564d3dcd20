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

constexpr int kMaxWarps = 16;   // of a row group
constexpr int kMaxStages = 8;

// one row of a tensor, contiguous and 16-byte aligned, into this CTA's shared memory
__device__ __forceinline__ void copy_row(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}

// 8 consecutive values as floats, and back
template <typename T>
__device__ __forceinline__ void get8(const void* p, float* f) {
  if constexpr (sizeof(T) == 2) {
    unpack8(*static_cast<const uint4*>(p), f);
  } else {
    const float4 a = static_cast<const float4*>(p)[0], b = static_cast<const float4*>(p)[1];
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  }
}
template <typename T>
__device__ __forceinline__ void put8(T* p, const float* f) {
  if constexpr (sizeof(T) == 2) {
    *reinterpret_cast<uint4*>(p) = pack8(f);
  } else {
    reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
  }
}
// a parameter vector's 8 values at v, or the constant where there is none
template <typename T>
__device__ __forceinline__ void param8(const T* p, int v, float none, float* f) {
  if (p) {
    get8<T>(p + 8 * v, f);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = none;
  }
}
// a value as it is stored
template <typename T>
__device__ __forceinline__ float stored(float v) {
  return sizeof(T) == 2 ? __bfloat162float(__float2bfloat16_rn(v)) : v;
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

// Sums over the group, the same bits in every thread (lanes by a fixed
// butterfly, then the warps in order).  `red` holds [2][2][kMaxWarps] floats of
// the group, zero where there is no warp; the two halves alternate, so one
// barrier a sum is enough.
template <int NV>
__device__ __forceinline__ void group_sum(const Place& pl, float* red, int& half, float (&v)[NV]) {
#pragma unroll
  for (int k = 0; k < NV; ++k) v[k] = warp_sum(v[k]);
  if (pl.warps == 1) return;
  float* r = red + half * 2 * kMaxWarps;
  half ^= 1;
  if ((pl.lane & 31) == 0) {
#pragma unroll
    for (int k = 0; k < NV; ++k) r[k * kMaxWarps + (pl.lane >> 5)] = v[k];
  }
  pl.sync();
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < kMaxWarps; w += 4) {
      if (w < pl.warps) {
        const float4 q = *reinterpret_cast<const float4*>(r + k * kMaxWarps + w);
        s += (q.x + q.y) + (q.z + q.w);
      }
    }
    v[k] = s;
  }
}

// The ring of one group: stage s at base + s * stage_bytes, its barrier at bars + 8 s.
struct Ring {
  uint32_t base, bars;
  uint32_t stage_bytes;
  int stages;
};

// Launch shape: threads a row, row groups a CTA, ring stages.
struct Shape {
  int vpt, tpr, groups, stages;
  uint32_t stage_bytes;
  size_t smem;
};
// smem: [groups][2][2][kMaxWarps] floats | barriers | abort flag | extra | rings, 128-byte aligned parts
constexpr size_t kRedBytes = 2 * 2 * kMaxWarps * sizeof(float);
__host__ __device__ inline size_t head_bytes(int groups) {
  return (groups * (kRedBytes + kMaxStages * 8) + 8 + 127) & ~size_t(127);
}
// Rows of up to 4096 values take one vector of 8 a thread; wider rows two.
// Narrow rows share a CTA of 8 warps.
inline Shape make_shape(int D, uint32_t row_bytes, size_t extra, size_t budget) {
  Shape s{};
  const int vecs = D / 8;
  s.vpt = vecs <= 32 * kMaxWarps ? 1 : 2;
  const int warps = (vecs + 32 * s.vpt - 1) / (32 * s.vpt);
  s.tpr = 32 * warps;
  s.groups = warps >= 8 ? 1 : 8 / warps;
  s.stage_bytes = (row_bytes + 127) & ~127u;
  const size_t head = head_bytes(s.groups) + extra;
  size_t n = budget > head ? (budget - head) / ((size_t)s.groups * s.stage_bytes) : 1;
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
