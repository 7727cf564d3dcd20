// Gated feed-forward block: the row copies ahead of its products.
#include <algorithm>

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

// HBM-bound, a warp a row: 4916 of 8192 rows x 2048 of x and dy (80 MB) and 13 MB
// of zeros in 16 us from memory (5.9 TB/s), 10 us between the kernels of a call.
__global__ void __launch_bounds__(256) ffn_prep_kernel(FfnPrep p, DevStatus* st) {
  // (the product behind this kernel sets itself up beside its last blocks)
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
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

}  // namespace collider
