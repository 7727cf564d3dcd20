// 8-bit activation checkpoints: pack and unpack of rows (format: q8.cuh).
//
// Collider drops the activations of filtered tokens in the backward (arXiv
// 2502.00340, abstract), so a checkpoint needs the kept rows only, and at one
// byte a value (plus 1/32 for the exponents) it is half as large as in bf16.
// Both kernels are bound by HBM: a value moves 2 + 1.03 bytes once (4916 x 11264
// values: 168 MB, 25.1 us at the measured copy rate; packing takes 26.1 us,
// unpacking 28.5).  A warp takes 1024 consecutive values of one row at a time
// (four 16-byte vectors a lane in flight), so that one long row spreads over
// warps as many rows do; the maximum over a group's 32 values is two shuffles
// among four lanes.
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

// this warp's first row, and the step to its next
__device__ __forceinline__ int first_row() { return blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); }
__device__ __forceinline__ int row_step() { return gridDim.x * (kThreads / 32); }
__device__ __forceinline__ int kept_rows(const int32_t* n_kept, int M) {
  return n_kept ? min(max(*n_kept, 0), M) : M;
}

// A lane's 8 values as loaded, and their largest magnitude as the bits of an
// f32: those order as the magnitudes do, with infinity and the NaNs above every
// number.  (bf16: two values a register are compared at a time.)
template <typename T>
struct Raw;
template <>
struct Raw<__nv_bfloat16> {
  uint4 u;
  __device__ void load(const __nv_bfloat16* p) { u = *reinterpret_cast<const uint4*>(p); }
  __device__ void clear() { u = make_uint4(0, 0, 0, 0); }
  __device__ unsigned largest() const {
    const unsigned a = __vmaxu2(u.x & 0x7fff7fffu, u.y & 0x7fff7fffu), b = __vmaxu2(u.z & 0x7fff7fffu, u.w & 0x7fff7fffu),
                   m = __vmaxu2(a, b);
    return max(m & 0xffff0000u, m << 16);
  }
  __device__ void values(float* f) const { unpack8(u, f); }
};
template <>
struct Raw<float> {
  float4 a, b;
  __device__ void load(const float* p) {
    a = *reinterpret_cast<const float4*>(p);
    b = *reinterpret_cast<const float4*>(p + 4);
  }
  __device__ void clear() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ unsigned largest() const {
    const float f[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    unsigned m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(f[i]) & 0x7fffffffu);
    return m;
  }
  __device__ void values(float* f) const {
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  }
};

template <typename T, int FMT>
__global__ void __launch_bounds__(kThreads) q8_pack_kernel(const T* __restrict__ src, long long src_ld, int M, int N,
                                                           const int32_t* __restrict__ idx,
                                                           const int32_t* __restrict__ n_kept, Q8View q,
                                                           DevStatus* st) {
  const int nk = kept_rows(n_kept, M);
  const int lane = threadIdx.x & 31, vecs = N >> 3, v0 = blockIdx.y * kSegVecs + lane;
  for (int r = first_row(); r < nk; r += row_step()) {
    const int t = idx ? idx[r] : r;
    if ((unsigned)t >= (unsigned)M) {
      if (lane == 0) report_error(st, kErrBadIndex, 700);
      continue;
    }
    const T* s = src + (long long)t * src_ld + 8 * v0;
    Raw<T> raw[kUnroll];
#pragma unroll
    for (int k = 0; k < kUnroll; ++k) {
      if (v0 + 32 * k < vecs) raw[k].load(s + 256 * k);
      else raw[k].clear();
    }
    uint8_t* code = q.code + (long long)r * q.code_ld + 8 * v0;
    uint8_t* exps = q.exps + (long long)r * q.exp_ld + (v0 >> 2);
#pragma unroll
    for (int k = 0; k < kUnroll; ++k) {
      unsigned m = raw[k].largest();
      m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
      m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
      const int byte = q8_exp_byte<FMT>(__uint_as_float(m));
      const float inv = q8_inv_scale(byte);
      float f[8];
      raw[k].values(f);
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] *= inv;
      if (byte == kQ8TopByte<FMT>) {   // values next to 2^128
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = fminf(fmaxf(f[i], -kQ8TopCode<FMT>), kQ8TopCode<FMT>);
      }
      uint2 c = q8_encode8<FMT>(f);
      if (byte == 255) c = make_uint2(0, 0);
      if (v0 + 32 * k < vecs) {
        *reinterpret_cast<uint2*>(code + 256 * k) = c;
        if ((lane & 3) == 0) exps[8 * k] = (uint8_t)byte;
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
  const int slots = dst_full == 2 ? nk : dst_full ? M : padded_rows(nk, cap);
  const int lane = threadIdx.x & 31, vecs = N >> 3, v0 = blockIdx.y * kSegVecs + lane;
  for (int r = first_row(); r < slots; r += row_step()) {
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
        if (!dst_full) zero_segment(dst + (long long)r * dst_ld, v0, vecs);   // a row of zeros to who reads it next
        continue;
      }
    }
    unpack_segment<T, FMT>(q, src_full ? t : r, dst + (dst_full ? t : r) * dst_ld, v0, vecs);
  }
}

// blockIdx.y: the segments of xk's rows, then of dyk's, then of dx's filtered rows.
template <int FMT>
__global__ void __launch_bounds__(kThreads) linear_prep_kernel(LinearPrep p, int ks, int ns, DevStatus* st) {
  const int nk = kept_rows(p.n_kept, p.M), pad = padded_rows(nk, p.cap);
  const int lane = threadIdx.x & 31, kv = p.K >> 3, nv = p.N >> 3;
  const int sx = p.xk ? ks : 0, sy = sx + (p.dyk ? ns : 0);
  const int part = (int)blockIdx.y < sx ? 0 : (int)blockIdx.y < sy ? 1 : 2;
  const int v0 = ((int)blockIdx.y - (part == 0 ? 0 : part == 1 ? sx : sy)) * kSegVecs + lane;
  if (part == 2) {
    for (int j = first_row(); j < p.M - nk; j += row_step())
      zero_segment(p.dx + (long long)filtered_token(p.idx, nk, j) * p.K, v0, kv);
    return;
  }
  for (int r = first_row(); r < pad; r += row_step()) {
    if (r >= nk) {
      if (part == 0) zero_segment(p.xk + (long long)r * p.K, v0, kv);
      else zero_segment(p.dyk + (long long)r * p.N, v0, nv);
      continue;
    }
    const int t = (part == 0 ? p.x_full : p.dy_full) ? p.idx[r] : r;
    if ((unsigned)t >= (unsigned)p.M) {   // reported, and a row of zeros to the GEMMs
      if (lane == 0) report_error(st, kErrBadIndex, 702);
      if (part == 0) zero_segment(p.xk + (long long)r * p.K, v0, kv);
      else zero_segment(p.dyk + (long long)r * p.N, v0, nv);
      continue;
    }
    if (part == 0) {
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

// blocks of x: a warp a row, up to per_sm blocks an SM in all; of y: row
// segments.  More blocks than an SM holds keep more loads in flight (packing
// 4916 x 11264 values: 26.1 us at 32 an SM, 28.2 at 8; unpacking 28.5 and 30.6);
// the copies beside a GEMM do best with fewer.
constexpr int kManyPerSm = 32, kFewPerSm = 4;
int segments(int N) { return (N / 8 + kSegVecs - 1) / kSegVecs; }
dim3 row_grid(const Ctx& c, long long rows, int segs, int per_sm) {
  const long long want = (rows + kThreads / 32 - 1) / (kThreads / 32), fit = ((long long)c.num_sms * per_sm + segs - 1) / segs;
  return dim3((unsigned)(want < 1 ? 1 : want < fit ? want : fit), (unsigned)segs);
}

}  // namespace

cudaError_t launch_q8_pack(const Ctx& c, int f32, const void* src, long long src_ld, int M, int N, const int32_t* idx,
                           const int32_t* n_kept, int format, const Q8View& q) {
  prof_begin(c, "q8_pack");
  const dim3 grid = row_grid(c, M, segments(N), kManyPerSm);
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
  const dim3 grid = row_grid(c, M, segments(N), kManyPerSm);
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
  const int ks = segments(p.K), ns = segments(p.N);
  const int segs = (p.xk ? ks : 0) + (p.dyk ? ns : 0) + (p.dx ? ks : 0);
  const dim3 grid = row_grid(c, p.cap, segs, kFewPerSm);
  if (p.format == kQ8E4m3) linear_prep_kernel<kQ8E4m3><<<grid, kThreads, 0, c.stream>>>(p, ks, ns, c.st);
  else linear_prep_kernel<kQ8Int8><<<grid, kThreads, 0, c.stream>>>(p, ks, ns, c.st);
  prof_end(c);
  count_launch();
  return cudaGetLastError();
}

}  // namespace collider
