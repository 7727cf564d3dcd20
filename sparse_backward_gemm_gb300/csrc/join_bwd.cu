// Residual join, backward on the kept rows (forward: join_fwd.cu).  With
// hh = (h - m_h) r_h and yh = (y - m_y) r_y the normalised rows, t = gamma_pre da:
//   dh = dH + r_h (t - hh mean(t hh) [- mean(t)])
//   dx = alpha lambda dh,   u = gate dh,   w = gamma_post u
//   dy = r_y (w - yh mean(w yh) [- mean(w)])
// ([ ]: LayerNorm) and, summed over the kept rows, the parameters' gradients
//   dgamma_pre = sum da hh,  dbeta_pre = sum da,  dgamma_post = sum u yh,
//   dbeta_post = sum u,  dgate_b = sum over sequence b of dh (gamma_post yh + beta_post),
//   dlambda = alpha sum dh x.
// y and h are the stored tensors or their 8-bit checkpoints, decoded as they
// are read.  Collider drops filtered rows in every layer (arXiv 2502.00340,
// abstract): only kept rows are read, and a FULL output gets zeros elsewhere.
//
// Bound by HBM: da, dH, y, h are read and dx, dy written once (12 D bytes a
// row in bf16, 10 D with 8-bit y and h).  A row's two sums depend on one
// another, so a row takes some 500 cycles however it is spread; the ring keeps
// several rows' copies in flight meanwhile.  Each thread owns the same columns
// of every row it sees and keeps their parameter sums in registers; a CTA's
// sums are parked in the workspace and added in CTA order by a second kernel,
// so the results do not change from run to run.
#include <algorithm>

#include "join.cuh"

namespace collider {

using namespace join;

namespace {

constexpr int kSrcSame = 2;   // y and h as stored (else kQ8E4m3, kQ8Int8)
// column sums
enum { kPreW, kPostW, kGate, kResW, kPreB, kPostB, kSums };

struct BwdArgs {
  int M, T, B, D;
  float inv_d, alpha;
  int gate_rows, post, pre, branch;
  const void *da, *dh, *x, *y, *h;     // y, h: T rows, or codes
  const uint8_t *y_exps, *h_exps;
  long long a_ld, h_ld, x_ld, y_ld;    // elements (strides of the gradients too)
  long long ys_ld, hs_ld;              // bytes between rows of the saved y, h
  long long ye_ld, he_ld;
  const void *post_w, *post_b, *gate, *res_w, *pre_w;
  const float *mean_y, *rstd_y, *mean_h, *rstd_h;
  const int32_t *idx, *cu, *nk;
  int saved_full, in_full, out_full;
  void *dx, *dy;
  float* sums[kSums];
  float* part;        // [kSums][grid][D]: every CTA's sums
  float* gate_part;   // [(grid + B) * groups][D]: gates of sequences, by (CTA + sequence, group)
  int grid;
  int tpr, groups, stages;
  uint32_t stage_bytes;
};

__device__ __forceinline__ int kept(const BwdArgs& p) { return p.nk ? min(max(*p.nk, 0), p.M) : p.M; }
// CTAs that have rows: each at least one
__device__ __forceinline__ int active(const BwdArgs& p, int nk) { return min(p.grid, (nk + p.groups - 1) / p.groups); }
// kept rows before sequence b
__device__ __forceinline__ int seq_begin(const BwdArgs& p, int b, int nk) {
  if (!p.cu) return min(b * (long long)p.T, (long long)nk);
  return b <= 0 ? 0 : b >= p.B ? nk : min(max(p.cu[b], 0), nk);
}
// the last sequence that begins at or before row r
__device__ int seq_of(const BwdArgs& p, int r, int nk) {
  int lo = 0, hi = p.B - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (seq_begin(p, mid, nk) <= r) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

template <typename T, int SRC>
__device__ __forceinline__ void saved8(const uint8_t* row, int v, unsigned e, float* f) {
  if constexpr (SRC == kSrcSame) get8<T>(row + v * 8 * sizeof(T), f);
  else q8_decode8<SRC>(*reinterpret_cast<const uint2*>(row + 8 * v), q8_scale(e), f);
}

template <typename T, bool LN, int SRC, int VPT>
__global__ void __launch_bounds__(512) join_bwd_kernel(BwdArgs p, DevStatus* st) {
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

  const T *da = static_cast<const T*>(p.da), *dh = static_cast<const T*>(p.dh), *x = static_cast<const T*>(p.x);
  const uint8_t *y = static_cast<const uint8_t*>(p.y), *h = static_cast<const uint8_t*>(p.h);
  T *dx = static_cast<T*>(p.dx), *dy = static_cast<T*>(p.dy);
  const int vecs = p.D / 8;
  const int nk = kept(p);
  const uint32_t row_bytes = p.D * (uint32_t)sizeof(T), src_bytes = SRC == kSrcSame ? row_bytes : (uint32_t)p.D;
  // a stage: da | dH | h | y | x, those there are
  const uint32_t o_dh = da ? row_bytes : 0, o_h = o_dh + (dh ? row_bytes : 0), o_y = o_h + (h ? src_bytes : 0),
                 o_x = o_y + (y ? src_bytes : 0), total = o_x + (x ? row_bytes : 0);
  const int A = active(p, nk);
  const bool mine = (int)blockIdx.x < A;
  const int r0 = mine ? (int)((long long)blockIdx.x * nk / A) : 0,
            r1 = mine ? (int)((long long)(blockIdx.x + 1) * nk / A) : 0;
  const int step = p.groups, first = r0 + pl.group;
  // token of kept row r (an index outside the tokens: -1, reported once)
  auto token = [&](int r) {
    if (r >= r1) return 0;
    const int t = p.idx ? p.idx[r] : r;
    return (unsigned)t < (unsigned)p.M ? t : -1;
  };
  auto issue = [&](int r, int t, int s) {
    const uint32_t b = bar0 + 8 * s, d = ring0 + s * p.stage_bytes;
    const long long tt = t < 0 ? 0 : t, sr = p.saved_full ? tt : r, ir = p.in_full ? tt : r;
    tc::mbar_expect_tx(b, total);
    if (da) copy_row(d, da + ir * p.a_ld, row_bytes, b);
    if (dh) copy_row(d + o_dh, dh + ir * p.h_ld, row_bytes, b);
    if (h) copy_row(d + o_h, h + sr * p.hs_ld, src_bytes, b);
    if (y) copy_row(d + o_y, y + sr * p.ys_ld, src_bytes, b);
    if (x) copy_row(d + o_x, x + sr * p.x_ld, row_bytes, b);
  };
  if (pl.lane == 0)
    for (int s = 0; s < p.stages; ++s)
      if (first + s * step < r1) issue(first + s * step, token(first + s * step), s);

  float acc[kSums][VPT][8];
#pragma unroll
  for (int q = 0; q < kSums; ++q)
#pragma unroll
    for (int k = 0; k < VPT; ++k)
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[q][k][i] = 0.f;

  const bool by_seq = p.gate_rows > 1;
  int b = 0, b_end = 0, b_last = 0;
  if (by_seq && mine) {
    b = seq_of(p, r0, nk);
    b_last = seq_of(p, r1 - 1, nk);
    b_end = seq_begin(p, b + 1, nk);
  }
  // parks this group's gate sum of sequence b
  auto park_gate = [&](int sb) {
    float* o = p.gate_part + (((long long)blockIdx.x + sb) * p.groups + pl.group) * p.D;
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const int v = pl.lane + k * p.tpr;
      if (v < vecs) put8(o + 8 * v, acc[kGate][k]);
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[kGate][k][i] = 0.f;
    }
  };

  // one row ahead: the next row's token, statistics and exponents
  struct Scalars {
    float mh, rh, my, ry;
    unsigned eh[VPT], ey[VPT];
  };
  auto scalars = [&](int r, int t) {
    Scalars q;
    const long long tt = t < 0 ? 0 : t;
    const bool any = r < r1;
    q.mh = (LN && p.pre && any) ? p.mean_h[tt] : 0.f;
    q.rh = (p.pre && any) ? p.rstd_h[tt] : 1.f;
    q.my = (LN && p.post && any) ? p.mean_y[tt] : 0.f;
    q.ry = (p.post && any) ? p.rstd_y[tt] : 1.f;
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      q.eh[k] = q.ey[k] = 0;
      const int v = pl.lane + k * p.tpr;
      if (SRC != kSrcSame && any && v < vecs) {
        const long long sr = p.saved_full ? tt : r;
        if (h) q.eh[k] = p.h_exps[sr * p.he_ld + (v >> 2)];
        if (y) q.ey[k] = p.y_exps[sr * p.ye_ld + (v >> 2)];
      }
    }
    return q;
  };
  int tok = token(first), tok_next = token(first + step), tok_fill = token(first + p.stages * step);
  Scalars now = scalars(first, tok);

  int half = 0, s = 0;
  uint32_t parity = 0;
  for (int r = first; r < r1; r += step) {
    const Scalars next = scalars(r + step, tok_next);
    const int tok_after = token(r + 2 * step);
    tc::mbar_wait(bar0 + 8 * s, (parity >> s) & 1u, abort_flag, st, 720);
    const uint8_t* stage = ring + s * p.stage_bytes;
    float dhv[VPT][8], tv[VPT][8], hv[VPT][8], yv[VPT][8], xv[VPT][8];
    bool on[VPT];
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const int v = pl.lane + k * p.tpr;
      on[k] = v < vecs;
#pragma unroll
      for (int i = 0; i < 8; ++i) dhv[k][i] = tv[k][i] = hv[k][i] = yv[k][i] = xv[k][i] = 0.f;
      if (on[k]) {
        if (da) get8<T>(stage + v * 8 * sizeof(T), tv[k]);
        if (dh) get8<T>(stage + o_dh + v * 8 * sizeof(T), dhv[k]);
        if (h) saved8<T, SRC>(stage + o_h, v, now.eh[k], hv[k]);
        if (y) saved8<T, SRC>(stage + o_y, v, now.ey[k], yv[k]);
        if (x) get8<T>(stage + o_x + v * 8 * sizeof(T), xv[k]);
      }
    }
    parity ^= 1u << s;
    // every thread has its values: the stage is free for a row further on
    pl.sync();
    if (pl.lane == 0) {
      const int rn = r + p.stages * step;
      if (rn < r1) issue(rn, tok_fill, s);
      tok_fill = token(rn + step);
    }
    if (++s == p.stages) s = 0;
    const int t = tok;
    tok = tok_next;
    tok_next = tok_after;
    if (t < 0) {   // (the same in every thread of the group)
      if (pl.lane == 0) report_error(st, kErrBadIndex, 721);
      now = next;
      continue;
    }
    if (by_seq)
      while (r >= b_end && b < b_last) {
        park_gate(b);
        ++b;
        b_end = seq_begin(p, b + 1, nk);
      }
    const long long orow = p.out_full ? t : r;

    if (p.pre) {
      float q[LN ? 2 : 1];
      q[0] = 0.f;
      if (LN) q[LN ? 1 : 0] = 0.f;
#pragma unroll
      for (int k = 0; k < VPT; ++k) {
        float w[8];
        if (on[k]) param8(static_cast<const T*>(p.pre_w), pl.lane + k * p.tpr, 1.f, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (!on[k]) continue;
          hv[k][i] = (hv[k][i] - now.mh) * now.rh;
          acc[kPreW][k][i] = fmaf(tv[k][i], hv[k][i], acc[kPreW][k][i]);
          if (LN) acc[kPreB][k][i] += tv[k][i];
          tv[k][i] *= w[i];
          q[0] = fmaf(tv[k][i], hv[k][i], q[0]);
          if (LN) q[LN ? 1 : 0] += tv[k][i];
        }
      }
      group_sum(pl, red, half, q);
      const float m1 = q[0] * p.inv_d, m0 = LN ? q[LN ? 1 : 0] * p.inv_d : 0.f;
#pragma unroll
      for (int k = 0; k < VPT; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float g = fmaf(-hv[k][i], m1, LN ? tv[k][i] - m0 : tv[k][i]);
          dhv[k][i] = fmaf(now.rh, g, dhv[k][i]);
        }
    }
    float q[LN ? 2 : 1];
    q[0] = 0.f;
    if (LN) q[LN ? 1 : 0] = 0.f;
    const T* gate = p.gate_rows ? static_cast<const T*>(p.gate) + (by_seq ? (long long)b * p.D : 0) : nullptr;
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      if (!on[k]) continue;
      const int v = pl.lane + k * p.tpr;
      float l[8], o[8];
      param8(static_cast<const T*>(p.res_w), v, 1.f, l);
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] = dhv[k][i] * (p.alpha * l[i]);
      put8(dx + orow * p.x_ld + 8 * v, o);
      if (x) {
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[kResW][k][i] = fmaf(dhv[k][i], xv[k][i], acc[kResW][k][i]);
      }
      if (p.branch) {
        float w[8], g[8], be[8];
        param8(static_cast<const T*>(p.post_w), v, 1.f, w);
        param8(static_cast<const T*>(p.post_b), v, 0.f, be);
        param8(gate, v, 1.f, g);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          yv[k][i] = (yv[k][i] - now.my) * now.ry;
          acc[kGate][k][i] = fmaf(dhv[k][i], fmaf(w[i], yv[k][i], be[i]), acc[kGate][k][i]);
          const float u = g[i] * dhv[k][i];
          acc[kPostW][k][i] = fmaf(u, yv[k][i], acc[kPostW][k][i]);
          if (LN) acc[kPostB][k][i] += u;
          tv[k][i] = u * w[i];
          q[0] = fmaf(tv[k][i], yv[k][i], q[0]);
          if (LN) q[LN ? 1 : 0] += tv[k][i];
        }
      }
    }
    if (p.branch) {
      float m1 = 0.f, m0 = 0.f;
      if (p.post) {
        group_sum(pl, red, half, q);
        m1 = q[0] * p.inv_d;
        if (LN) m0 = q[LN ? 1 : 0] * p.inv_d;
      }
#pragma unroll
      for (int k = 0; k < VPT; ++k) {
        if (!on[k]) continue;
        float o[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = now.ry * fmaf(-yv[k][i], m1, LN ? tv[k][i] - m0 : tv[k][i]);
        put8(dy + orow * p.y_ld + 8 * (pl.lane + k * p.tpr), o);
      }
    }
    now = next;
  }

  // park the column sums: gates of sequences by group, the others added over the CTA's groups
  if (by_seq && mine)
    for (; b <= b_last; ++b) park_gate(b);
  __syncthreads();
  if (*abort_flag && pl.lane == 0) drain(bar0, p.stages, parity);
  if (mine) {
    float* line = reinterpret_cast<float*>(smem + head_bytes(p.groups));   // the rings are done with
    if (*abort_flag == 0) {
      for (int q = 0; q < kSums; ++q) {
        if (!p.sums[q] || (q == kGate && by_seq)) continue;
        float* o = p.part + ((long long)q * p.grid + blockIdx.x) * p.D;
        if (p.groups > 1) {
#pragma unroll
          for (int k = 0; k < VPT; ++k) {
            const int v = pl.lane + k * p.tpr;
            if (v < vecs)
#pragma unroll
              for (int c = 0; c < kSums; ++c)
                if (c == q) put8(line + pl.group * p.D + 8 * v, acc[c][k]);
          }
          __syncthreads();
          for (int c = threadIdx.x; c < p.D; c += blockDim.x) {
            float sum = 0.f;
            for (int g = 0; g < p.groups; ++g) sum += line[g * p.D + c];
            o[c] = sum;
          }
          __syncthreads();
        } else {
#pragma unroll
          for (int k = 0; k < VPT; ++k) {
            const int v = pl.lane + k * p.tpr;
            if (v < vecs)
#pragma unroll
              for (int c = 0; c < kSums; ++c)
                if (c == q) put8(o + 8 * v, acc[c][k]);
          }
        }
      }
    }
  }

  // rows that get zeros: the filtered tokens of FULL outputs, the padding of COMPACT ones
  const int zeros = p.out_full ? p.M - nk : padded_rows(nk, p.M) - nk;
  const int wpb = blockDim.x >> 5, lane = threadIdx.x & 31;
  for (int j = blockIdx.x * wpb + (threadIdx.x >> 5); j < zeros; j += gridDim.x * wpb) {
    const long long row = p.out_full ? filtered_token(p.idx, nk, j) : nk + j;
    const float z[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (int v = lane; v < vecs; v += 32) {
      put8(dx + row * p.x_ld + 8 * v, z);
      if (p.branch) put8(dy + row * p.y_ld + 8 * v, z);
    }
  }
}

// sums[q][c] = the parked sums added in slot order: 32 columns a block, 32
// threads a column, each every 32nd slot, then the 32 in order.  blockIdx.y
// counts the gradients there are, a gate by sequences as B of them.
__global__ void __launch_bounds__(1024) join_sums_kernel(BwdArgs p) {
  __shared__ float red[32][33];
  grid_dep_wait();
  int q = 0, b = blockIdx.y;
  for (;; ++q) {
    const int n = !p.sums[q] ? 0 : (q == kGate && p.gate_rows > 1) ? p.B : 1;
    if (b < n) break;
    b -= n;
  }
  const int nk = kept(p), A = active(p, nk);
  const float* part = p.part + (long long)q * p.grid * p.D;
  long long s0 = 0, s1 = A;
  if (q == kGate && p.gate_rows > 1) {
    part = p.gate_part;
    const int f = seq_begin(p, b, nk), l = seq_begin(p, b + 1, nk);
    // the CTA of row r is the last whose first row, cta * nk / A, is at most r
    const auto cta = [&](int r) { return (((long long)r + 1) * A - 1) / nk; };
    s0 = l > f ? (cta(f) + b) * p.groups : 0;
    s1 = l > f ? (cta(l - 1) + b + 1) * p.groups : 0;
  }
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5, c = blockIdx.x * 32 + tx;
  float sum = 0.f;
  if (c < p.D) {
#pragma unroll 4
    for (long long s = s0 + ty; s < s1; s += 32) sum += part[s * p.D + c];
  }
  red[ty][tx] = sum;
  __syncthreads();
  if (ty == 0 && c < p.D) {
    sum = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) sum += red[i][tx];
    p.sums[q][(long long)b * p.D + c] = q == kResW ? p.alpha * sum : sum;
  }
}

constexpr int kCtasPerSm = 2, kMaxSms = 256;

template <typename T, bool LN, int SRC, int VPT>
cudaError_t launch(const Ctx& c, const BwdArgs& p, size_t smem) {
  auto k = join_bwd_kernel<T, LN, SRC, VPT>;
  static size_t granted[64];   // shared memory opted in to, a device
  const cudaError_t e = grant_smem(reinterpret_cast<const void*>(k), smem, granted);
  if (e != cudaSuccess) return e;
  k<<<p.grid, p.tpr * p.groups, smem, c.stream>>>(p, c.st);
  return cudaGetLastError();
}
template <typename T, bool LN, int SRC>
cudaError_t by_vpt(const Ctx& c, const BwdArgs& p, int vpt, size_t smem) {
  return vpt == 1 ? launch<T, LN, SRC, 1>(c, p, smem) : launch<T, LN, SRC, 2>(c, p, smem);
}
template <typename T, bool LN>
cudaError_t by_src(const Ctx& c, const BwdArgs& p, int src, int vpt, size_t smem) {
  if (src == kQ8E4m3) return by_vpt<T, LN, kQ8E4m3>(c, p, vpt, smem);
  if (src == kQ8Int8) return by_vpt<T, LN, kQ8Int8>(c, p, vpt, smem);
  return by_vpt<T, LN, kSrcSame>(c, p, vpt, smem);
}

int bwd_grid(int M, int num_sms, const Shape& s) {
  const long long want = ((long long)M + s.groups - 1) / s.groups, fit = (long long)std::min(num_sms, kMaxSms) * kCtasPerSm;
  return (int)(want < fit ? want : fit);
}
// the widest stage there is: every tensor, as stored
Shape bwd_shape(int D, uint32_t row_bytes) {
  Shape s = make_shape(D, row_bytes, 0, 100 * 1024);
  const size_t line = head_bytes(s.groups) + (s.groups > 1 ? (size_t)s.groups * D * 4 : 0);
  if (s.smem < line) s.smem = line;
  return s;
}

}  // namespace

// partial sums of the widest grid on any GPU of up to kMaxSms SMs
size_t join_bwd_part_floats(int B, int T, int D, int gate_rows) {
  const Shape s = make_shape(D, 16, 0, 0);
  const long long grid = bwd_grid(B * T, kMaxSms, s);
  return (size_t)(grid * kSums + (gate_rows > 1 ? (grid + B) * s.groups : 0)) * D;
}

cudaError_t launch_join_bwd(const Ctx& c, const JoinBwd& j) {
  BwdArgs p{};
  p.M = j.B * j.T; p.T = j.T; p.B = j.B; p.D = j.D;
  p.inv_d = 1.f / (float)j.D; p.alpha = j.alpha;
  p.gate_rows = j.gate_rows; p.post = j.post; p.pre = j.pre; p.branch = j.y != nullptr;
  p.da = j.da; p.dh = j.dh; p.x = j.x; p.y = j.y; p.h = j.pre ? j.h : nullptr;
  p.y_exps = j.y_exps; p.h_exps = j.h_exps;
  p.a_ld = j.a_ld; p.h_ld = j.h_ld; p.x_ld = j.x_ld; p.y_ld = j.y_ld;
  const bool same = j.src == kSrcSame;
  const int es = j.f32 ? 4 : 2;
  p.ys_ld = same ? j.y_ld * es : j.y_code_ld; p.hs_ld = same ? j.h_ld * es : j.h_code_ld;
  p.ye_ld = j.y_exp_ld; p.he_ld = j.h_exp_ld;
  p.post_w = j.post_w; p.post_b = j.post_b; p.gate = j.gate; p.res_w = j.res_w; p.pre_w = j.pre_w;
  p.mean_y = j.mean_y; p.rstd_y = j.rstd_y; p.mean_h = j.mean_h; p.rstd_h = j.rstd_h;
  p.idx = j.idx; p.cu = j.cu; p.nk = j.nk;
  p.saved_full = j.saved_full; p.in_full = j.in_full; p.out_full = j.out_full;
  p.dx = j.dx; p.dy = j.dy;
  p.sums[kPreW] = j.dpre_w; p.sums[kPreB] = j.dpre_b; p.sums[kPostW] = j.dpost_w; p.sums[kPostB] = j.dpost_b;
  p.sums[kGate] = j.dgate; p.sums[kResW] = j.dres_w;
  const uint32_t row = (uint32_t)j.D * es, src = same ? row : (uint32_t)j.D;
  const uint32_t total = (p.da ? row : 0) + (p.dh ? row : 0) + (p.h ? src : 0) + (p.y ? src : 0) + (p.x ? row : 0);
  const Shape s = bwd_shape(j.D, total);
  p.tpr = s.tpr; p.groups = s.groups; p.stages = s.stages; p.stage_bytes = s.stage_bytes;
  p.grid = bwd_grid(p.M, c.num_sms, s);
  p.part = j.part;
  p.gate_part = j.part + (size_t)kSums * p.grid * p.D;
  prof_begin(c, "residual_norm_bwd");
  cudaError_t e;
  if (j.f32) e = j.layer_norm ? by_src<float, true>(c, p, j.src, s.vpt, s.smem)
                              : by_src<float, false>(c, p, j.src, s.vpt, s.smem);
  else e = j.layer_norm ? by_src<__nv_bfloat16, true>(c, p, j.src, s.vpt, s.smem)
                        : by_src<__nv_bfloat16, false>(c, p, j.src, s.vpt, s.smem);
  prof_end(c);
  count_launch();
  if (e != cudaSuccess) return e;
  int tasks = 0;
  for (int q = 0; q < kSums; ++q) tasks += !p.sums[q] ? 0 : (q == kGate && j.gate_rows > 1) ? j.B : 1;
  if (tasks == 0) return cudaSuccess;
  prof_begin(c, "residual_norm_sums");
  e = launch_k(c, pdl_allowed(), join_sums_kernel, dim3((j.D + 31) / 32, tasks), dim3(1024), 0, 1, p);
  prof_end(c);
  count_launch();
  return launched(e);
}

}  // namespace collider
