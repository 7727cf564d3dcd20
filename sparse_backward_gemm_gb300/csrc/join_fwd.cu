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
// Floor: x and y are read and h and a written once, 8 D bytes a row in bf16:
// 20.0 us for 8192 rows of 2048 values, which take 24.9 us (5.4 TB/s); the
// instructions of a row at 16 warps an SM are next.  On the way there 61 us
// (parameters read again for every row, scalar arithmetic), 29 (two vectors a
// thread, packed arithmetic, cp.async), 25 (the pre norm's weight in registers).
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
__global__ void __launch_bounds__(kThreads) join_fwd_kernel(FwdArgs p) {
  extern __shared__ __align__(128) uint8_t smem[];
  const Place pl(p.tpr);
  float* red = reinterpret_cast<float*>(smem + pl.group * kRedBytes);
  uint8_t* ring = smem + head_bytes(p.groups) + (size_t)pl.group * p.stages * p.stage_bytes;
  const uint32_t ring0 = tc::smem_u32(ring);
  for (int i = threadIdx.x; i < (int)(head_bytes(p.groups) / 4); i += blockDim.x) reinterpret_cast<uint32_t*>(smem)[i] = 0;
  __syncthreads();

  const T *x = static_cast<const T*>(p.x), *y = static_cast<const T*>(p.y);
  T *h = static_cast<T*>(p.h), *a = static_cast<T*>(p.a);
  const int vecs = p.D / 8;
  const uint32_t row_bytes = p.D * (uint32_t)sizeof(T);
  const uint32_t off = pl.lane * 8 * (uint32_t)sizeof(T), hop = p.tpr * 8 * (uint32_t)sizeof(T);
  const int step = gridDim.x * p.groups, r0 = blockIdx.x * p.groups + pl.group;
  auto fill = [&](long long r, int s) {   // this thread's columns of row r, if there is one, into stage s
    if (r < p.M) {
      const uint32_t d = ring0 + s * p.stage_bytes + off;
      const T *sx = x + r * p.x_ld + 8 * pl.lane, *sy = y + r * p.y_ld + 8 * pl.lane;
#pragma unroll
      for (int k = 0; k < VPT; ++k)
        if (pl.lane + k * p.tpr < vecs) {
          copy_vec(d + k * hop, sx + k * p.tpr * 8);
          if (y) copy_vec(d + row_bytes + k * hop, sy + k * p.tpr * 8);
        }
    }
    copy_commit();
  };
  for (int s = 0; s < p.stages; ++s) fill(r0 + (long long)s * step, s);

  // gate times the post norm's weight and bias, for the rows of one sequence
  // (of all sequences when there is one row of gates); 0 beyond the row
  Vec8 c1[VPT], c0[LN ? VPT : 1];
  auto set_gate = [&](int b) {
    const T* gate = p.gate_rows ? static_cast<const T*>(p.gate) + (p.gate_rows > 1 ? (long long)b * p.D : 0) : nullptr;
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const int v = pl.lane + k * p.tpr;
      const bool on = v < vecs;
      const Vec8 g = param8<T>(gate, v, on, 1.f), w = param8<T>(p.post_w, v, on, 1.f);
      const Vec8 o = param8<T>(p.post_b, v, on, 0.f);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        c1[k].v[i] = mul2(g.v[i], w.v[i]);
        if (LN) c0[LN ? k : 0].v[i] = mul2(g.v[i], o.v[i]);
      }
    }
  };
  const int seq_rows = p.gate_rows > 1 ? p.T : p.M;   // rows that share a gate
  int gate_end = 0;

  // mean and reciprocal deviation of a row held in v (0 beyond the row), and
  // the row less its mean
  int half = 0;
  auto stats = [&](Vec8 (&v)[VPT], float& mean, float& rstd) {
    float q[1];
    mean = 0.f;
    if (LN) {
      f2 t = both(0.f);
#pragma unroll
      for (int k = 0; k < VPT; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i) t = add2(t, v[k].v[i]);
      q[0] = t.x + t.y;
      group_sum(pl, red, half, q);
      mean = q[0] * p.inv_d;
#pragma unroll
      for (int k = 0; k < VPT; ++k) {
        const f2 m = both(pl.lane + k * p.tpr < vecs ? -mean : 0.f);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[k].v[i] = add2(v[k].v[i], m);
      }
    }
    f2 t = both(0.f);
#pragma unroll
    for (int k = 0; k < VPT; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i) t = fma2(v[k].v[i], v[k].v[i], t);
    q[0] = t.x + t.y;
    group_sum(pl, red, half, q);
    rstd = __frsqrt_rn(fmaf(q[0], p.inv_d, p.eps));
  };

  // threads beyond the row read zeros
  const uint8_t* zero = smem + zero_at(p.groups);
  Raw8<T> w_pre[VPT];   // this thread's part of the pre norm's weight, as stored
#pragma unroll
  for (int k = 0; k < VPT; ++k)
    w_pre[k] = *reinterpret_cast<const Raw8<T>*>(
        p.pre && pl.lane + k * p.tpr < vecs ? static_cast<const void*>(static_cast<const T*>(p.pre_w) + 8 * (pl.lane + k * p.tpr))
                                            : static_cast<const void*>(zero));
  int s = 0;
  for (int r = r0; r < p.M; r += step) {
    if (r >= gate_end) {   // the first row, and each first row of a sequence
      const int b = r / seq_rows;
      set_gate(b);
      gate_end = (int)min((long long)p.M, (b + 1ll) * seq_rows);
    }
    copy_wait(p.stages - 1);
    const uint8_t* stage = ring + s * p.stage_bytes + off;
    Vec8 xv[VPT], yv[VPT];
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const bool on = pl.lane + k * p.tpr < vecs;
      xv[k] = get8<T>(on ? stage + k * hop : zero);
      if (y) yv[k] = get8<T>(on ? stage + row_bytes + k * hop : zero);
    }
    fill(r + (long long)p.stages * step, s);
    if (++s == p.stages) s = 0;

    if (y) {
      float mean = 0.f, rstd = 1.f;
      if (p.post) {
        stats(yv, mean, rstd);
        if (pl.lane == 0) {
          p.rstd_y[r] = rstd;
          if (LN) p.mean_y[r] = mean;
        }
      }
      T* row = h + r * p.h_ld + 8 * pl.lane;
      const f2 rs = both(rstd), al = both(p.alpha);
#pragma unroll
      for (int k = 0; k < VPT; ++k) {
        const bool on = pl.lane + k * p.tpr < vecs;
        if (p.res_w) {
          const Vec8 l = param8<T>(p.res_w, pl.lane + k * p.tpr, on, 0.f);
#pragma unroll
          for (int i = 0; i < 4; ++i) xv[k].v[i] = mul2(xv[k].v[i], l.v[i]);
        }
        Vec8 o;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const f2 res = LN ? fma2(al, xv[k].v[i], c0[LN ? k : 0].v[i]) : mul2(al, xv[k].v[i]);
          o.v[i] = fma2(c1[k].v[i], mul2(yv[k].v[i], rs), res);
        }
        xv[k] = put8_stored(row + k * p.tpr * 8, on, o);
      }
    }
    if (p.pre) {
      float mean, rstd;
      stats(xv, mean, rstd);
      if (pl.lane == 0) {
        p.rstd_h[r] = rstd;
        if (LN) p.mean_h[r] = mean;
      }
      T* row = a + r * p.a_ld + 8 * pl.lane;
      const f2 rs = both(rstd);
#pragma unroll
      for (int k = 0; k < VPT; ++k) {
        const int v = pl.lane + k * p.tpr;
        if (v >= vecs) continue;
        const Vec8 w = get8<T>(&w_pre[k]);
        const Vec8 o = LN ? param8<T>(p.pre_b, v, true, 0.f) : all8(0.f);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const f2 n = mul2(xv[k].v[i], rs);
          xv[k].v[i] = LN ? fma2(n, w.v[i], o.v[i]) : mul2(n, w.v[i]);
        }
        put8(row + k * p.tpr * 8, xv[k]);
      }
    }
  }
}

template <typename T, bool LN, int VPT>
cudaError_t launch(const Ctx& c, const FwdArgs& p, const Shape& s) {
  auto k = join_fwd_kernel<T, LN, VPT>;
  static size_t granted[64];   // shared memory opted in to, a device
  const cudaError_t e = grant_smem(reinterpret_cast<const void*>(k), s.smem, granted);
  if (e != cudaSuccess) return e;
  const long long want = ((long long)p.M + s.groups - 1) / s.groups, fit = (long long)c.num_sms * 2;
  k<<<(int)(want < fit ? want : fit), s.tpr * s.groups, s.smem, c.stream>>>(p);
  return cudaGetLastError();
}

template <typename T, bool LN>
cudaError_t by_vpt(const Ctx& c, const FwdArgs& p, const Shape& s) {
  return s.vpt == 1 ? launch<T, LN, 1>(c, p, s) : launch<T, LN, 2>(c, p, s);
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
  const int vpt = j.D <= 256 ? 1 : 2;
  const Shape s = make_shape(j.D, vpt, row, 0, 60 * 1024);
  p.tpr = s.tpr; p.groups = s.groups; p.stages = s.stages; p.stage_bytes = s.stage_bytes;
  prof_begin(c, "residual_norm_fwd");
  using bf = __nv_bfloat16;
  cudaError_t e;
  if (j.f32) e = j.layer_norm ? by_vpt<float, true>(c, p, s) : by_vpt<float, false>(c, p, s);
  else e = j.layer_norm ? by_vpt<bf, true>(c, p, s) : by_vpt<bf, false>(c, p, s);
  prof_end(c);
  count_launch();
  return e;
}

}  // namespace collider
