// Gated feed-forward block: the row kernels around its products.
#include <algorithm>

#include "glu.cuh"
#include "internal.h"

namespace collider {

namespace {

__device__ __forceinline__ int rows_of(const int32_t* n_kept, int M) {
  if (!n_kept) return M;
  const int n = *n_kept;
  return n < 0 ? 0 : n < M ? n : M;
}

// whether t is among the ascending idx[0..n), by the whole warp: 32 places of
// the range left are compared at once
__device__ __forceinline__ bool warp_contains(const int32_t* __restrict__ idx, int n, int t) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = n;   // the first place >= t lies in [lo, hi]
  while (hi - lo >= 32) {
    const int step = (hi - lo + 31) / 32, at = lo + lane * step;
    const unsigned below = __ballot_sync(0xffffffffu, at < hi && idx[at < hi ? at : lo] < t);
    const int k = __popc(below);   // places 0..k-1 hold less than t
    if (k == 0) { hi = lo; break; }
    const int nlo = lo + (k - 1) * step + 1, nhi = min(lo + k * step, hi);
    lo = nlo;
    hi = nhi;
  }
  return __any_sync(0xffffffffu, lo + lane <= hi && lo + lane < n && idx[min(lo + lane, n - 1)] == t);
}

__global__ void __launch_bounds__(256) ffn_prep_kernel(FfnPrep p, DevStatus* st) {
  const int n = rows_of(p.n_kept, p.M);
  const int lane = threadIdx.x & 31, wpb = blockDim.x >> 5, vecs = p.D >> 3;
  const int w0 = blockIdx.x * wpb + (threadIdx.x >> 5), ws = gridDim.x * wpb;
  if (blockIdx.y == 2) {
    for (int t = w0; t < p.M; t += ws) {
      if (warp_contains(p.idx, n, t)) continue;
      uint4* d = reinterpret_cast<uint4*>(p.dx + (long long)t * p.dx_ld);
      for (int v = lane; v < vecs; v += 32) d[v] = make_uint4(0, 0, 0, 0);
    }
    return;
  }
  const bool is_x = blockIdx.y == 0;
  const __nv_bfloat16* src = is_x ? p.x : p.dy;
  __nv_bfloat16* dst = is_x ? p.xk : p.dyk;
  if (!dst) return;
  const long long ld = is_x ? p.x_ld : p.dy_ld;
  const bool full = (is_x ? p.x_full : p.dy_full) && p.idx;
  const int pad = padded_rows(n, p.cap);
  for (int r = w0; r < pad; r += ws) {
    uint4* d = reinterpret_cast<uint4*>(dst + (long long)r * p.D);
    int t = r;
    if (r < n && full) {
      t = p.idx[r];
      if ((unsigned)t >= (unsigned)p.M) {
        if (lane == 0) report_error(st, kErrBadIndex, 700);
        t = -1;
      }
    }
    if (r >= n || t < 0) {
      for (int v = lane; v < vecs; v += 32) d[v] = make_uint4(0, 0, 0, 0);
      continue;
    }
    const uint4* s = reinterpret_cast<const uint4*>(src + (long long)t * ld);
    int v = lane;
    for (; v + 96 < vecs; v += 128) {   // four loads in flight before their stores
      const uint4 a = s[v], b = s[v + 32], c = s[v + 64], e = s[v + 96];
      d[v] = a; d[v + 32] = b; d[v + 64] = c; d[v + 96] = e;
    }
    for (; v < vecs; v += 32) d[v] = s[v];
  }
}

__device__ __forceinline__ void load8f(const float* p, float* f) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
  f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
  f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}

template <int ACT>
__global__ void __launch_bounds__(256) glu_fwd_kernel(int M, int F, const float* __restrict__ acc, __nv_bfloat16* up,
                                                      long long up_ld, __nv_bfloat16* s) {
  const int vpr = F >> 3;
  const long long total = (long long)M * vpr;
  for (long long e = blockIdx.x * (long long)blockDim.x + threadIdx.x; e < total; e += (long long)gridDim.x * blockDim.x) {
    const long long r = e / vpr;
    const int c = (int)(e % vpr) * 8;
    float g[8], u[8], v[8];
    load8f(acc + r * 2 * F + c, g);
    load8f(acc + r * 2 * F + F + c, u);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = glu_act<ACT>(g[i]) * u[i];
    if (up) {
      *reinterpret_cast<uint4*>(up + r * up_ld + c) = pack8(g);
      *reinterpret_cast<uint4*>(up + r * up_ld + F + c) = pack8(u);
    }
    *reinterpret_cast<uint4*>(s + r * F + c) = pack8(v);
  }
}

template <int ACT>
__global__ void __launch_bounds__(256) glu_bwd_kernel(int M, int F, const float* __restrict__ ds,
                                                      const __nv_bfloat16* __restrict__ up, long long up_ld, int up_full,
                                                      __nv_bfloat16* dgu, __nv_bfloat16* s, long long cap,
                                                      const int32_t* __restrict__ idx, const int32_t* __restrict__ n_kept,
                                                      DevStatus* st) {
  const int n = rows_of(n_kept, M), pad = padded_rows(n, cap), vpr = F >> 3;
  const long long total = (long long)pad * vpr;
  for (long long e = blockIdx.x * (long long)blockDim.x + threadIdx.x; e < total; e += (long long)gridDim.x * blockDim.x) {
    const long long r = e / vpr;
    const int c = (int)(e % vpr) * 8;
    float dg[8], du[8], sv[8];
    int t = (int)r;
    if (r < n && up_full && idx) {
      t = idx[r];
      if ((unsigned)t >= (unsigned)M) {
        report_error(st, kErrBadIndex, 701);
        t = -1;
      }
    }
    if (r < n && t >= 0) {
      float d[8], g[8], u[8];
      load8f(ds + r * F + c, d);
      unpack8(*reinterpret_cast<const uint4*>(up + t * up_ld + c), g);
      unpack8(*reinterpret_cast<const uint4*>(up + t * up_ld + F + c), u);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float a, da;
        glu_both<ACT>(g[i], &a, &da);
        dg[i] = d[i] * u[i] * da;
        du[i] = d[i] * a;
        sv[i] = a * u[i];
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) dg[i] = du[i] = sv[i] = 0.f;
    }
    *reinterpret_cast<uint4*>(dgu + r * 2 * F + c) = pack8(dg);
    *reinterpret_cast<uint4*>(dgu + r * 2 * F + F + c) = pack8(du);
    *reinterpret_cast<uint4*>(s + r * F + c) = pack8(sv);
  }
}

int grid_of(const Ctx& c, long long items, int per_block) {
  const long long want = (items + per_block - 1) / per_block, most = (long long)c.num_sms * 8;
  return (int)std::max(1ll, std::min(want, most));
}

}  // namespace

cudaError_t launch_ffn_prep(const Ctx& c, const FfnPrep& p) {
  prof_begin(c, "ffn_prep");
  const int parts = p.dx ? 3 : 2;
  ffn_prep_kernel<<<dim3(grid_of(c, p.cap, 8), parts), 256, 0, c.stream>>>(p, c.st);
  prof_end(c);
  count_launch();
  return cudaGetLastError();
}

cudaError_t launch_glu_fwd(const Ctx& c, int act, int M, int F, const float* acc, __nv_bfloat16* up, long long up_ld,
                           __nv_bfloat16* s) {
  prof_begin(c, "glu_fwd");
  auto k = act == kGluSilu ? glu_fwd_kernel<kGluSilu> : glu_fwd_kernel<kGluGeluTanh>;
  k<<<grid_of(c, (long long)M * (F / 8), 256), 256, 0, c.stream>>>(M, F, acc, up, up_ld, s);
  prof_end(c);
  count_launch();
  return cudaGetLastError();
}

cudaError_t launch_glu_bwd(const Ctx& c, int act, int M, int F, const float* ds, const __nv_bfloat16* up, long long up_ld,
                           int up_full, __nv_bfloat16* dgu, __nv_bfloat16* s, long long cap, const int32_t* idx,
                           const int32_t* n_kept) {
  prof_begin(c, "glu_bwd");
  auto k = act == kGluSilu ? glu_bwd_kernel<kGluSilu> : glu_bwd_kernel<kGluGeluTanh>;
  k<<<grid_of(c, cap * (F / 8), 256), 256, 0, c.stream>>>(M, F, ds, up, up_ld, up_full, dgu, s, cap, idx, n_kept, c.st);
  prof_end(c);
  count_launch();
  return cudaGetLastError();
}

}  // namespace collider
