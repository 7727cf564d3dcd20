// 8-bit activation checkpoints: pack and unpack of rows (format: q8.cuh).
//
// Collider drops the activations of filtered tokens in the backward (arXiv
// 2502.00340, abstract), so a checkpoint needs the kept rows only, and at one
// byte a value (plus 1/32 for the exponents) it is half as large again as in
// bf16.  Both kernels are bound by HBM: a value moves 2 + 1.03 bytes once.  A
// warp takes 1024 consecutive values of one row at a time (four 16-byte vectors a
// lane in flight), so that one long row spreads over warps as many rows do; the
// maximum over a group's 32 values is two shuffles among four lanes.
#include "internal.h"
#include "q8.cuh"

namespace collider {

namespace {

constexpr int kUnroll = 4;                        // vectors of 8 values a lane
constexpr int kSegVecs = 32 * kUnroll;            // vectors of a warp's segment
constexpr int kThreads = 256;

template <typename T>
__device__ __forceinline__ void load_vec(const T* p, float* f) {
  if constexpr (sizeof(T) == 2) {
    unpack8(*reinterpret_cast<const uint4*>(p), f);
  } else {
    const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  }
}
template <typename T>
__device__ __forceinline__ void store_vec(T* p, const float* f) {
  if constexpr (sizeof(T) == 2) {
    *reinterpret_cast<uint4*>(p) = pack8(f);
  } else {
    *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
    *reinterpret_cast<float4*>(p + 4) = make_float4(f[4], f[5], f[6], f[7]);
  }
}

__device__ __forceinline__ int kept_rows(const int32_t* n_kept, int M) {
  return n_kept ? min(max(*n_kept, 0), M) : M;
}

template <typename T, int FMT>
__global__ void __launch_bounds__(kThreads) q8_pack_kernel(const T* __restrict__ src, long long src_ld, int M, int N,
                                                           const int32_t* __restrict__ idx,
                                                           const int32_t* __restrict__ n_kept, Q8View q,
                                                           DevStatus* st) {
  const int nk = kept_rows(n_kept, M);
  const int lane = threadIdx.x & 31;
  const int vecs = N >> 3, segs = (vecs + kSegVecs - 1) / kSegVecs;
  const long long units = (long long)nk * segs;
  const long long stride = (long long)gridDim.x * (kThreads / 32);
  for (long long u = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); u < units; u += stride) {
    const int r = (int)(u / segs), v0 = (int)(u % segs) * kSegVecs + lane;
    const int t = idx ? idx[r] : r;
    if ((unsigned)t >= (unsigned)M) {
      if (lane == 0) report_error(st, kErrBadIndex, 700);
      continue;
    }
    const T* s = src + (long long)t * src_ld;
    float f[kUnroll][8];
#pragma unroll
    for (int k = 0; k < kUnroll; ++k) {
      const int v = v0 + 32 * k;
      if (v < vecs) {
        load_vec(s + 8 * v, f[k]);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[k][i] = 0.f;
      }
    }
#pragma unroll
    for (int k = 0; k < kUnroll; ++k) {
      const int v = v0 + 32 * k;
      // the largest magnitude as bits: they order as the magnitudes do, with
      // infinity and the NaNs above every number
      unsigned m = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(f[k][i]) & 0x7fffffffu);
      m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
      m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
      const int byte = q8_exp_byte<FMT>(__uint_as_float(m));
      const float inv = q8_inv_scale(byte);
#pragma unroll
      for (int i = 0; i < 8; ++i) f[k][i] = byte == 255 ? 0.f : f[k][i] * inv;
      if (v < vecs) {
        *reinterpret_cast<uint2*>(q.code + (long long)r * q.code_ld + 8 * v) = q8_encode8<FMT>(f[k]);
        if ((lane & 3) == 0) q.exps[(long long)r * q.exp_ld + (v >> 2)] = (uint8_t)byte;
      }
    }
  }
}

// decodes this lane's vectors (v0 + 32 k) of row sr of q
template <typename T, int FMT>
__device__ __forceinline__ void unpack_segment(const Q8View& q, long long sr, T* d, int v0, int vecs) {
  uint2 c[kUnroll];
  unsigned e[kUnroll];
#pragma unroll
  for (int k = 0; k < kUnroll; ++k) {
    const int v = v0 + 32 * k;
    c[k] = make_uint2(0, 0);
    e[k] = 0;
    if (v < vecs) {
      c[k] = *reinterpret_cast<const uint2*>(q.code + sr * q.code_ld + 8 * v);
      e[k] = q.exps[sr * q.exp_ld + (v >> 2)];
    }
  }
#pragma unroll
  for (int k = 0; k < kUnroll; ++k) {
    const int v = v0 + 32 * k;
    float f[8];
    q8_decode8<FMT>(c[k], q8_scale(e[k]), f);
    if (v < vecs) store_vec(d + 8 * v, f);
  }
}
template <typename T>
__device__ __forceinline__ void zero_segment(T* d, int v0, int vecs) {
#pragma unroll
  for (int k = 0; k < kUnroll; ++k) {
    const float z[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (v0 + 32 * k < vecs) store_vec(d + 8 * (v0 + 32 * k), z);
  }
}

// Row slots: the kept rows first, then the rows that get zeros (the filtered
// tokens of a FULL output, the padding of a COMPACT one).
template <typename T, int FMT>
__global__ void __launch_bounds__(kThreads) q8_unpack_kernel(Q8View q, int src_full, int M, int N,
                                                             const int32_t* __restrict__ idx,
                                                             const int32_t* __restrict__ n_kept,
                                                             T* __restrict__ dst, long long dst_ld, int dst_full,
                                                             long long cap, DevStatus* st) {
  grid_dep_wait();
  const int nk = kept_rows(n_kept, M);
  const int slots = dst_full ? M : padded_rows(nk, cap);
  const int lane = threadIdx.x & 31;
  const int vecs = N >> 3, segs = (vecs + kSegVecs - 1) / kSegVecs;
  const long long units = (long long)slots * segs;
  const long long stride = (long long)gridDim.x * (kThreads / 32);
  for (long long u = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); u < units; u += stride) {
    const int r = (int)(u / segs), v0 = (int)(u % segs) * kSegVecs + lane;
    if (r >= nk) {
      const int t = dst_full ? filtered_token(idx, nk, r - nk) : r;
      zero_segment(dst + (long long)t * dst_ld, v0, vecs);
      continue;
    }
    int t = r;
    if (idx && (src_full || dst_full)) {
      t = idx[r];
      if ((unsigned)t >= (unsigned)M) {
        if (lane == 0) report_error(st, kErrBadIndex, 701);
        continue;
      }
    }
    unpack_segment<T, FMT>(q, src_full ? t : r, dst + (dst_full ? t : r) * dst_ld, v0, vecs);
  }
}

// Units of the three parts one after another: segments of xk's rows, of dyk's,
// and of dx's filtered rows.
template <int FMT>
__global__ void __launch_bounds__(kThreads) linear_prep_kernel(LinearPrep p, DevStatus* st) {
  const int nk = kept_rows(p.n_kept, p.M);
  const int lane = threadIdx.x & 31;
  const int kv = p.K >> 3, ks = (kv + kSegVecs - 1) / kSegVecs, nv = p.N >> 3, ns = (nv + kSegVecs - 1) / kSegVecs;
  const long long pad = padded_rows(nk, p.cap);
  const long long ux = p.xk ? pad * ks : 0, uy = ux + (p.dyk ? pad * ns : 0),
                  units = uy + (p.dx ? (long long)(p.M - nk) * ks : 0);
  const long long stride = (long long)gridDim.x * (kThreads / 32);
  for (long long u = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); u < units; u += stride) {
    if (u >= uy) {
      const int j = (int)((u - uy) / ks), v0 = (int)((u - uy) % ks) * kSegVecs + lane;
      zero_segment(p.dx + (long long)filtered_token(p.idx, nk, j) * p.K, v0, kv);
      continue;
    }
    const bool is_x = u < ux;
    const long long w = is_x ? u : u - ux;
    const int segs = is_x ? ks : ns, r = (int)(w / segs), v0 = (int)(w % segs) * kSegVecs + lane;
    if (r >= nk) {
      if (is_x) zero_segment(p.xk + (long long)r * p.K, v0, kv);
      else zero_segment(p.dyk + (long long)r * p.N, v0, nv);
      continue;
    }
    const int t = (is_x ? p.x_full : p.dy_full) ? p.idx[r] : r;
    if ((unsigned)t >= (unsigned)p.M) {
      if (lane == 0) report_error(st, kErrBadIndex, 702);
      continue;
    }
    if (is_x) {
      unpack_segment<__nv_bfloat16, FMT>(p.x, t, p.xk + (long long)r * p.K, v0, kv);
    } else {
      const uint4* s = reinterpret_cast<const uint4*>(p.dy + (long long)t * p.N);
      uint4* d = reinterpret_cast<uint4*>(p.dyk + (long long)r * p.N);
      uint4 c[kUnroll];
#pragma unroll
      for (int k = 0; k < kUnroll; ++k)
        if (v0 + 32 * k < nv) c[k] = s[v0 + 32 * k];
#pragma unroll
      for (int k = 0; k < kUnroll; ++k)
        if (v0 + 32 * k < nv) d[v0 + 32 * k] = c[k];
    }
  }
}

int unit_grid(const Ctx& c, long long rows, int N) {
  const long long segs = (N / 8 + kSegVecs - 1) / kSegVecs;
  const long long g = (rows * segs + kThreads / 32 - 1) / (kThreads / 32), cap = (long long)c.num_sms * 8;
  return (int)(g < 1 ? 1 : g > cap ? cap : g);
}

}  // namespace

cudaError_t launch_q8_pack(const Ctx& c, int f32, const void* src, long long src_ld, int M, int N, const int32_t* idx,
                           const int32_t* n_kept, int format, const Q8View& q) {
  prof_begin(c, "q8_pack");
  const int grid = unit_grid(c, M, N);
#define COLLIDER_PACK(T, FMT) \
  q8_pack_kernel<T, FMT><<<grid, kThreads, 0, c.stream>>>(static_cast<const T*>(src), src_ld, M, N, idx, n_kept, q, c.st)
  if (f32) {
    if (format == kQ8E4m3) COLLIDER_PACK(float, kQ8E4m3);
    else COLLIDER_PACK(float, kQ8Int8);
  } else {
    if (format == kQ8E4m3) COLLIDER_PACK(__nv_bfloat16, kQ8E4m3);
    else COLLIDER_PACK(__nv_bfloat16, kQ8Int8);
  }
#undef COLLIDER_PACK
  prof_end(c);
  count_launch();
  return cudaGetLastError();
}

cudaError_t launch_q8_unpack(const Ctx& c, int f32, int format, const Q8View& q, int src_full, int M, int N,
                             const int32_t* idx, const int32_t* n_kept, void* dst, long long dst_ld, int dst_full,
                             long long cap) {
  prof_begin(c, "q8_unpack");
  const dim3 grid(unit_grid(c, M, N));
  cudaError_t e;
#define COLLIDER_UNPACK(T, FMT)                                                                                   \
  e = launch_k(c, c.pdl, q8_unpack_kernel<T, FMT>, grid, dim3(kThreads), 0, 1, q, src_full, M, N, idx, n_kept, \
               static_cast<T*>(dst), dst_ld, dst_full, cap, c.st)
  if (f32) {
    if (format == kQ8E4m3) COLLIDER_UNPACK(float, kQ8E4m3);
    else COLLIDER_UNPACK(float, kQ8Int8);
  } else {
    if (format == kQ8E4m3) COLLIDER_UNPACK(__nv_bfloat16, kQ8E4m3);
    else COLLIDER_UNPACK(__nv_bfloat16, kQ8Int8);
  }
#undef COLLIDER_UNPACK
  prof_end(c);
  count_launch();
  return launched(e);
}

cudaError_t launch_linear_prep(const Ctx& c, const LinearPrep& p) {
  prof_begin(c, "linear_prep");
  const long long ks = (p.K / 8 + kSegVecs - 1) / kSegVecs, ns = (p.N / 8 + kSegVecs - 1) / kSegVecs;
  const long long units = p.cap * ((p.xk || p.dx ? ks : 0) + (p.dyk ? ns : 0)), fit = (long long)c.num_sms * 8;
  const long long want = (units + kThreads / 32 - 1) / (kThreads / 32);
  const int grid = (int)(want < 1 ? 1 : want < fit ? want : fit);
  if (p.format == kQ8E4m3) linear_prep_kernel<kQ8E4m3><<<grid, kThreads, 0, c.stream>>>(p, c.st);
  else linear_prep_kernel<kQ8Int8><<<grid, kThreads, 0, c.stream>>>(p, c.st);
  prof_end(c);
  count_launch();
  return cudaGetLastError();
}

}  // namespace collider
