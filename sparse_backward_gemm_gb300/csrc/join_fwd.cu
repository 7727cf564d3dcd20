// Residual join, forward: h = alpha * lambda . x + gate . post(y), a = pre(h),
// one pass over x and y.
//
// Between two blocks of a decoder stand the norm after a branch, its gate, the
// residual scale and sum, and the norm before the next branch.  Per row:
//   RMSNorm    v -> gamma v r,           r = (mean v^2 + eps)^-1/2
//   LayerNorm  v -> gamma (v - m) r + b, r = (mean (v - m)^2 + eps)^-1/2
// with the second norm taken of h as it is stored, so that a backward that
// reads h sees the very values it differentiates.  Statistics and products are
// f32; h and a are rounded once each.
//
// Bound by HBM: x and y are read and h and a written once, 8 D bytes a row in
// bf16.
#include "join.cuh"

namespace collider {

using namespace join;

namespace {

struct FwdArgs {
  int M, T, D;
  float eps, inv_d, alpha;
  int gate_rows;
  int post, pre;
  const void *x, *y;
  void *h, *a;
  long long x_ld, y_ld, h_ld, a_ld;
  const void *post_w, *post_b, *gate, *res_w, *pre_w, *pre_b;
  float *mean_y, *rstd_y, *mean_h, *rstd_h;
  int tpr, groups, stages;
  uint32_t stage_bytes;
};

template <typename T, bool LN, int VPT>
__global__ void __launch_bounds__(512) join_fwd_kernel(FwdArgs p, DevStatus* st) {
  extern __shared__ __align__(128) uint8_t smem[];
  const Place pl(p.tpr);
  float* red = reinterpret_cast<float*>(smem + pl.group * kRedBytes);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + p.groups * kRedBytes) + pl.group * kMaxStages;
  volatile int* abort_flag =
      reinterpret_cast<volatile int*>(smem + p.groups * (kRedBytes + kMaxStages * sizeof(uint64_t)));
  uint8_t* ring = smem + head_bytes(p.groups) + (size_t)pl.group * p.stages * p.stage_bytes;
  const uint32_t bar0 = tc::smem_u32(bars), ring0 = tc::smem_u32(ring);
  if (pl.lane == 0)
    for (int s = 0; s < p.stages; ++s) tc::mbar_init(bar0 + 8 * s, 1);
  for (int i = pl.lane; i < (int)(kRedBytes / 4); i += p.tpr) red[i] = 0.f;
  if (threadIdx.x == 0) *abort_flag = 0;
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  __syncthreads();

  const T *x = static_cast<const T*>(p.x), *y = static_cast<const T*>(p.y);
  T *h = static_cast<T*>(p.h), *a = static_cast<T*>(p.a);
  const int vecs = p.D / 8;
  const uint32_t row_bytes = p.D * (uint32_t)sizeof(T), total = y ? 2 * row_bytes : row_bytes;
  const int step = gridDim.x * p.groups, r0 = blockIdx.x * p.groups + pl.group;
  auto issue = [&](int r, int s) {
    const uint32_t b = bar0 + 8 * s, d = ring0 + s * p.stage_bytes;
    tc::mbar_expect_tx(b, total);
    copy_row(d, x + (long long)r * p.x_ld, row_bytes, b);
    if (y) copy_row(d + row_bytes, y + (long long)r * p.y_ld, row_bytes, b);
  };
  if (pl.lane == 0)
    for (int s = 0; s < p.stages; ++s)
      if ((long long)r0 + (long long)s * step < p.M) issue(r0 + s * step, s);

  int half = 0, s = 0;
  uint32_t parity = 0;
  for (long long r = r0; r < p.M; r += step) {
    tc::mbar_wait(bar0 + 8 * s, (parity >> s) & 1u, abort_flag, st, 710);
    const uint8_t* stage = ring + s * p.stage_bytes;
    float xv[VPT][8], yv[VPT][8];
    bool on[VPT];
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const int v = pl.lane + k * p.tpr;
      on[k] = v < vecs;
#pragma unroll
      for (int i = 0; i < 8; ++i) xv[k][i] = yv[k][i] = 0.f;
      if (on[k]) {
        get8<T>(stage + v * 8 * sizeof(T), xv[k]);
        if (y) get8<T>(stage + row_bytes + v * 8 * sizeof(T), yv[k]);
      }
    }
    parity ^= 1u << s;
    // every thread has its values: the stage is free for a row further on
    pl.sync();
    if (pl.lane == 0) {
      const long long rn = r + (long long)p.stages * step;
      if (rn < p.M) issue((int)rn, s);
    }
    if (++s == p.stages) s = 0;

    // mean and reciprocal deviation of a row held in v
    auto stats = [&](float (*v)[8], float& mean, float& rstd) {
      float q[1] = {0.f};
      mean = 0.f;
      if (LN) {
#pragma unroll
        for (int k = 0; k < VPT; ++k)
#pragma unroll
          for (int i = 0; i < 8; ++i) q[0] += v[k][i];
        group_sum(pl, red, half, q);
        mean = q[0] * p.inv_d;
        q[0] = 0.f;
      }
#pragma unroll
      for (int k = 0; k < VPT; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float d = on[k] ? v[k][i] - mean : 0.f;
          q[0] = fmaf(d, d, q[0]);
        }
      group_sum(pl, red, half, q);
      rstd = __frsqrt_rn(fmaf(q[0], p.inv_d, p.eps));
    };

    if (y) {
      float mean = 0.f, rstd = 1.f;
      if (p.post) {
        stats(yv, mean, rstd);
        if (pl.lane == 0) {
          p.rstd_y[r] = rstd;
          if (LN) p.mean_y[r] = mean;
        }
      }
      const T* gate = p.gate_rows ? static_cast<const T*>(p.gate) + (p.gate_rows > 1 ? (r / p.T) * p.D : 0) : nullptr;
#pragma unroll
      for (int k = 0; k < VPT; ++k) {
        if (!on[k]) continue;
        const int v = pl.lane + k * p.tpr;
        float w[8], b[8], g[8], l[8];
        param8(static_cast<const T*>(p.post_w), v, 1.f, w);
        param8(static_cast<const T*>(p.post_b), v, 0.f, b);
        param8(gate, v, 1.f, g);
        param8(static_cast<const T*>(p.res_w), v, 1.f, l);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float n = p.post ? norm_affine(yv[k][i], mean, rstd, w[i], b[i]) : yv[k][i];
          xv[k][i] = stored<T>(fmaf(g[i], n, p.alpha * l[i] * xv[k][i]));
        }
        put8(h + r * p.h_ld + 8 * v, xv[k]);
      }
    }
    if (p.pre) {
      float mean, rstd;
      stats(xv, mean, rstd);
      if (pl.lane == 0) {
        p.rstd_h[r] = rstd;
        if (LN) p.mean_h[r] = mean;
      }
#pragma unroll
      for (int k = 0; k < VPT; ++k) {
        if (!on[k]) continue;
        const int v = pl.lane + k * p.tpr;
        float w[8], b[8], o[8];
        param8(static_cast<const T*>(p.pre_w), v, 1.f, w);
        param8(static_cast<const T*>(p.pre_b), v, 0.f, b);
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = norm_affine(xv[k][i], mean, rstd, w[i], b[i]);
        put8(a + r * p.a_ld + 8 * v, o);
      }
    }
  }
  // (every copy issued was waited for, unless a wait gave up)
  __syncthreads();
  if (*abort_flag && pl.lane == 0) drain(bar0, p.stages, parity);
}

template <typename T, bool LN, int VPT>
cudaError_t launch(const Ctx& c, const FwdArgs& p, const Shape& s) {
  auto k = join_fwd_kernel<T, LN, VPT>;
  static size_t granted[64];   // shared memory opted in to, a device
  const cudaError_t e = grant_smem(reinterpret_cast<const void*>(k), s.smem, granted);
  if (e != cudaSuccess) return e;
  const long long want = ((long long)p.M + s.groups - 1) / s.groups, fit = (long long)c.num_sms * 2;
  k<<<(int)(want < fit ? want : fit), s.tpr * s.groups, s.smem, c.stream>>>(p, c.st);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_join_fwd(const Ctx& c, const JoinFwd& j) {
  FwdArgs p{};
  p.M = j.B * j.T; p.T = j.T; p.D = j.D;
  p.eps = j.eps; p.inv_d = 1.f / (float)j.D; p.alpha = j.alpha;
  p.gate_rows = j.gate_rows; p.post = j.post; p.pre = j.pre;
  p.x = j.x; p.y = j.y; p.h = j.h; p.a = j.a;
  p.x_ld = j.x_ld; p.y_ld = j.y_ld; p.h_ld = j.h_ld; p.a_ld = j.a_ld;
  p.post_w = j.post_w; p.post_b = j.post_b; p.gate = j.gate; p.res_w = j.res_w; p.pre_w = j.pre_w; p.pre_b = j.pre_b;
  p.mean_y = j.mean_y; p.rstd_y = j.rstd_y; p.mean_h = j.mean_h; p.rstd_h = j.rstd_h;
  const uint32_t row = (uint32_t)j.D * (j.f32 ? 4 : 2) * (j.y ? 2 : 1);
  const Shape s = make_shape(j.D, row, 0, 100 * 1024);
  p.tpr = s.tpr; p.groups = s.groups; p.stages = s.stages; p.stage_bytes = s.stage_bytes;
  prof_begin(c, "residual_norm_fwd");
  cudaError_t e;
  if (j.f32) {
    if (j.layer_norm) e = s.vpt == 1 ? launch<float, true, 1>(c, p, s) : launch<float, true, 2>(c, p, s);
    else e = s.vpt == 1 ? launch<float, false, 1>(c, p, s) : launch<float, false, 2>(c, p, s);
  } else {
    using bf = __nv_bfloat16;
    if (j.layer_norm) e = s.vpt == 1 ? launch<bf, true, 1>(c, p, s) : launch<bf, true, 2>(c, p, s);
    else e = s.vpt == 1 ? launch<bf, false, 1>(c, p, s) : launch<bf, false, 2>(c, p, s);
  }
  prof_end(c);
  count_launch();
  return e;
}

}  // namespace collider
