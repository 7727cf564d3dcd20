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
constexpr uint32_t kHeadBytes = 32;   // of a stage

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
  uint32_t stage_bytes, ring_at;
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
__device__ __forceinline__ Vec8 saved8(const void* p, unsigned e) {
  if constexpr (SRC == kSrcSame) {
    return get8<T>(p);
  } else {
    float f[8];
    q8_decode8<SRC>(*static_cast<const uint2*>(p), q8_scale(e), f);
    Vec8 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r.v[i] = make_float2(f[2 * i], f[2 * i + 1]);
    return r;
  }
}

template <typename T, bool LN, int SRC, int VPT, bool RES, int MINB>
__global__ void __launch_bounds__(kThreads, MINB) join_bwd_kernel(BwdArgs p, DevStatus* st) {
  extern __shared__ __align__(128) uint8_t smem[];
  const Place pl(p.tpr);
  float* red = reinterpret_cast<float*>(smem + pl.group * kRedBytes);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + p.groups * kRedBytes) + pl.group * kMaxStages;
  volatile int* abort_flag =
      reinterpret_cast<volatile int*>(smem + p.groups * (kRedBytes + kMaxStages * sizeof(uint64_t)));
  uint8_t* ring = smem + p.ring_at + (size_t)pl.group * p.stages * p.stage_bytes;
  const uint32_t bar0 = tc::smem_u32(bars), ring0 = tc::smem_u32(ring);
  if (pl.lane == 0)
    for (int s = 0; s < p.stages; ++s) tc::mbar_init(bar0 + 8 * s, 2);   // the copies, and the head
  for (int i = pl.lane; i < (int)(kRedBytes / 4); i += p.tpr) red[i] = 0.f;
  if (threadIdx.x == 0) *abort_flag = 0;
  if (threadIdx.x < 8) reinterpret_cast<uint32_t*>(smem + zero_at(p.groups))[threadIdx.x] = 0;
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
  // Rows of this group: first, first + step, ... below r1.  Strided over the
  // grid, or, where gates differ by sequence, from a contiguous share of the
  // rows, so that a CTA sees few sequences.
  const bool by_seq = p.gate_rows > 1;
  const int A = active(p, nk);
  const bool mine = (int)blockIdx.x < A;
  const int r0 = by_seq && mine ? (int)((long long)blockIdx.x * nk / A) : blockIdx.x * p.groups,
            r1 = !mine ? 0 : by_seq ? (int)((long long)(blockIdx.x + 1) * nk / A) : nk;
  const int step = by_seq ? p.groups : gridDim.x * p.groups, first = r0 + pl.group;
  // A stage of the ring: the row's token and statistics, then its tensors.
  // Lane s of the group's first warp fills stage s, so that the first rows'
  // indices and statistics are fetched side by side; later it fetches the next
  // row's index when it fills the stage, and that row's statistics a row later.
  struct Head {
    int token;   // -1: an index outside the tokens
    float rh, ry, mh, my;
  };
  static_assert(sizeof(Head) <= kHeadBytes, "");
  auto token = [&](int r) {
    if (r >= r1) return -1;
    const int t = p.idx ? p.idx[r] : r;
    return (unsigned)t < (unsigned)p.M ? t : -1;
  };
  auto head = [&](int t) {
    Head q{t, 1.f, 1.f, 0.f, 0.f};
    if (t >= 0) {
      if (p.pre) q.rh = p.rstd_h[t];
      if (p.post) q.ry = p.rstd_y[t];
      if (LN && p.pre) q.mh = p.mean_h[t];
      if (LN && p.post) q.my = p.mean_y[t];
    }
    return q;
  };
  auto fill = [&](int r, int t, int s) {
    const uint32_t b = bar0 + 8 * s, d = ring0 + s * p.stage_bytes + kHeadBytes;
    const long long tt = t < 0 ? 0 : t, sr = p.saved_full ? tt : r, ir = p.in_full ? tt : r;
    tc::mbar_expect_tx(b, total);
    if (da) copy_row(d, da + ir * p.a_ld, row_bytes, b);
    if (dh) copy_row(d + o_dh, dh + ir * p.h_ld, row_bytes, b);
    if (h) copy_row(d + o_h, h + sr * p.hs_ld, src_bytes, b);
    if (y) copy_row(d + o_y, y + sr * p.ys_ld, src_bytes, b);
    if (x) copy_row(d + o_x, x + sr * p.x_ld, row_bytes, b);
  };
  auto set_head = [&](const Head& q, int s) {   // (the arrival makes it visible to who waits)
    *reinterpret_cast<Head*>(ring + s * p.stage_bytes) = q;
    tc::mbar_arrive(bar0 + 8 * s);
  };
  // the finishing kernel may be scheduled as blocks of this one exit
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  Head ahead{};          // lane s: of the row that stage s takes next
  if (pl.lane < p.stages) {
    const int r = first + pl.lane * step;
    const int t = token(r), ta = token(r + p.stages * step);
    if (r < r1) fill(r, t, pl.lane);
    const Head q = head(t);
    ahead = head(ta);
    if (r < r1) set_head(q, pl.lane);
  }

  // Column sums over this group's rows: of da hh, da (LN), and -- of one
  // sequence while gates differ by sequence -- of dh yh, dh (LN); of dh x.
  constexpr int VL = LN ? VPT : 1, VR = RES ? VPT : 1;
  Vec8 s_pre[VPT], s_da[VL], s_dhy[VPT], s_dh[VL], s_res[VR];
#pragma unroll
  for (int k = 0; k < VPT; ++k) {
    s_pre[k] = s_dhy[k] = all8(0.f);
    if (LN) s_da[LN ? k : 0] = s_dh[LN ? k : 0] = all8(0.f);
    if (RES) s_res[RES ? k : 0] = all8(0.f);
  }

  int b = 0, b_end = r1, b_last = 0;
  if (by_seq && mine) {
    b = seq_of(p, r0, nk);
    b_last = seq_of(p, r1 - 1, nk);
    b_end = seq_begin(p, b + 1, nk);
  }
  // gate times the post norm's weight, for the rows of sequence b; 0 beyond the row
  Vec8 c1[VPT];
  auto gate_at = [&](int sb) {
    return p.gate_rows ? static_cast<const T*>(p.gate) + (by_seq ? (long long)sb * p.D : 0) : nullptr;
  };
  auto set_gate = [&] {
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const int v = pl.lane + k * p.tpr;
      const Vec8 g = param8<T>(gate_at(b), v, v < vecs, 1.f), w = param8<T>(p.post_w, v, v < vecs, 1.f);
#pragma unroll
      for (int i = 0; i < 4; ++i) c1[k].v[i] = mul2(g.v[i], w.v[i]);
    }
  };
  set_gate();
#pragma unroll
  for (int k = 0; k < VPT; ++k)   // read first in the row loop
    if (pl.lane + k * p.tpr < vecs) {
      prefetch_l1(static_cast<const T*>(p.pre_w) + 8 * (pl.lane + k * p.tpr), p.pre != 0);
      prefetch_l1(static_cast<const T*>(p.res_w) + 8 * (pl.lane + k * p.tpr), RES);
    }
  // A sequence's sums become the gradient of its gate, dgate = gamma s_dhy +
  // beta s_dh, and its share of the post norm's gradients, gate s_dhy and gate
  // s_dh.  Of several sequences the shares gather in u, this thread's own line
  // of shared memory.
  Vec8* u = reinterpret_cast<Vec8*>(smem + head_bytes(p.groups)) + ((size_t)pl.group * p.tpr + pl.lane) * (LN ? 2 : 1) * VPT;
  auto end_sequence = [&](bool last) {
    float* o = p.gate_part + (((long long)blockIdx.x + b) * p.groups + pl.group) * p.D;
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const int v = pl.lane + k * p.tpr;
      const Vec8 g = param8<T>(gate_at(b), v, v < vecs, 1.f), w = param8<T>(p.post_w, v, v < vecs, 1.f),
                 be = param8<T>(p.post_b, v, v < vecs, 0.f);
      Vec8 dg;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        dg.v[i] = mul2(w.v[i], s_dhy[k].v[i]);
        if (LN) dg.v[i] = fma2(be.v[i], s_dh[LN ? k : 0].v[i], dg.v[i]);
        u[k].v[i] = fma2(g.v[i], s_dhy[k].v[i], u[k].v[i]);
        if (LN) u[VPT + k].v[i] = fma2(g.v[i], s_dh[LN ? k : 0].v[i], u[VPT + k].v[i]);
      }
      s_dhy[k] = all8(0.f);
      if (LN) s_dh[LN ? k : 0] = all8(0.f);
      if (v < vecs) put8(o + 8 * v, dg);
    }
    if (!last) {
      ++b;
      b_end = seq_begin(p, b + 1, nk);
      set_gate();
    }
  };
  if (by_seq)
#pragma unroll
    for (int i = 0; i < (LN ? 2 : 1) * VPT; ++i) u[i] = all8(0.f);

  // threads beyond the row read zeros
  const uint8_t* zero = smem + zero_at(p.groups);
  const uint32_t off = pl.lane * 8 * (uint32_t)sizeof(T), hop = p.tpr * 8 * (uint32_t)sizeof(T);
  const uint32_t s_off = SRC == kSrcSame ? off : pl.lane * 8, s_hop = SRC == kSrcSame ? hop : p.tpr * 8;
  // 8-bit y and h: this thread's exponent bytes, a row ahead
  struct Exps {
    unsigned h[VPT], y[VPT];
  };
  auto exps = [&](int r, int t) {
    Exps q;
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      q.h[k] = q.y[k] = 0;
      const int v = pl.lane + k * p.tpr;
      if (SRC != kSrcSame && t >= 0 && v < vecs) {
        const long long sr = p.saved_full ? t : r;
        if (h) q.h[k] = p.h_exps[sr * p.he_ld + (v >> 2)];
        if (y) q.y[k] = p.y_exps[sr * p.ye_ld + (v >> 2)];
      }
    }
    return q;
  };
  int tok_next = SRC == kSrcSame ? 0 : token(first + step);
  Exps now = exps(first, SRC == kSrcSame ? 0 : token(first));

  int half = 0, s = 0, prev = -1;
  uint32_t parity = 0;
  const f2 al = both(p.alpha);
  for (int r = first; r < r1; r += step) {
    Exps next;
    if (SRC != kSrcSame) {
      next = exps(r + step, tok_next);
      tok_next = token(r + 2 * step);
    }
    tc::mbar_wait(bar0 + 8 * s, (parity >> s) & 1u, abort_flag, st, 720);
    parity ^= 1u << s;
    const uint8_t* stage = ring + s * p.stage_bytes + kHeadBytes;
    const Head hd = *reinterpret_cast<const Head*>(ring + s * p.stage_bytes);
    // Once every thread has reached this row the stage before it is free for a
    // row further on: after this row's first sum over the group, or a barrier.
    // (A ring of one stage has no such stage: it is filled when the row is done.)
    auto refill = [&] {
      if (prev >= 0 && pl.lane < p.stages && p.stages > 1) {
        if (pl.lane == prev) {
          const int rn = r + (p.stages - 1) * step;
          if (rn < r1) {
            fill(rn, ahead.token, prev);
            set_head(ahead, prev);
          }
          ahead.token = token(rn + p.stages * step);
        }
        if (pl.lane == (prev == 0 ? p.stages - 1 : prev - 1)) ahead = head(ahead.token);
      }
      prev = s;
      if (++s == p.stages) s = 0;
    };
    auto row_done = [&] {
      now = next;
      if (p.stages > 1) return;
      pl.sync();
      if (pl.lane == 0) {
        if (r + step < r1) {
          fill(r + step, ahead.token, 0);
          set_head(ahead, 0);
        }
        ahead = head(token(r + 2 * step));
      }
    };
    if (hd.token < 0 || !(p.pre || p.post)) {
      pl.sync();
      refill();
    }
    if (hd.token < 0) {   // (the same in every thread of the group)
      if (pl.lane == 0) report_error(st, kErrBadIndex, 721);
      row_done();
      continue;
    }
    while (r >= b_end && b < b_last) end_sequence(false);
    const long long orow = p.out_full ? hd.token : r;
    const f2 rh = both(hd.rh), ry = both(hd.ry), mh = both(-hd.mh), my = both(-hd.my);
    // the row's vectors (read from the stage whenever they are used, which
    // keeps few registers), normalised where they have a norm
    auto on = [&](int k) { return pl.lane + k * p.tpr < vecs; };
    auto at_da = [&](int k) { return get8<T>(on(k) ? stage + off + k * hop : zero); };
    auto at_dh = [&](int k) { return get8<T>(on(k) && dh ? stage + o_dh + off + k * hop : zero); };
    auto at_h = [&](int k) {
      Vec8 v = saved8<T, SRC>(on(k) ? stage + o_h + s_off + k * s_hop : zero, now.h[k]);
#pragma unroll
      for (int i = 0; i < 4; ++i) v.v[i] = mul2(LN ? add2(v.v[i], mh) : v.v[i], rh);
      return v;
    };
    auto at_y = [&](int k) {
      Vec8 v = saved8<T, SRC>(on(k) ? stage + o_y + s_off + k * s_hop : zero, now.y[k]);
#pragma unroll
      for (int i = 0; i < 4; ++i) v.v[i] = mul2(LN ? add2(v.v[i], my) : v.v[i], ry);
      return v;
    };
    auto pre_w = [&](int k) { return param8<T>(p.pre_w, pl.lane + k * p.tpr, on(k), 0.f); };

    // Sums over the row.  RMSNorm takes them all at once: with m1 = mean(t hh),
    //   sum(w yh) = sum(c1 yh dH) + r_h (sum(c1 yh t) - m1 sum(c1 yh hh)),
    // so that the post norm's sum need not wait for dh.  LayerNorm, which would
    // need ten sums, takes the pre norm's first.
    float n1 = 0.f, n0 = 0.f, o1 = 0.f;   // -mean(t hh), -mean(t), -mean(w yh)
    if (!LN) {
      f2 q0 = both(0.f), q1 = both(0.f), q2 = both(0.f), q3 = both(0.f);
#pragma unroll
      for (int k = 0; k < VPT; ++k) {
        Vec8 t = all8(0.f), hh = all8(0.f);
        if (p.pre) {
          t = at_da(k);
          hh = at_h(k);
          const Vec8 w = pre_w(k);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            s_pre[k].v[i] = fma2(t.v[i], hh.v[i], s_pre[k].v[i]);
            t.v[i] = mul2(t.v[i], w.v[i]);
            q0 = fma2(t.v[i], hh.v[i], q0);
          }
        }
        if (p.post) {
          const Vec8 yh = at_y(k), d = at_dh(k);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const f2 cy = mul2(c1[k].v[i], yh.v[i]);
            q1 = fma2(cy, d.v[i], q1);
            q2 = fma2(cy, t.v[i], q2);
            q3 = fma2(cy, hh.v[i], q3);
          }
        }
      }
      if (p.pre || p.post) {
        float q[4] = {q0.x + q0.y, q1.x + q1.y, q2.x + q2.y, q3.x + q3.y};
        group_sum(pl, red, half, q);
        refill();
        n1 = -q[0] * p.inv_d;
        o1 = -fmaf(hd.rh, fmaf(n1, q[3], q[2]), q[1]) * p.inv_d;
      }
    } else if (p.pre) {
      f2 q1 = both(0.f), q0 = both(0.f);
#pragma unroll
      for (int k = 0; k < VPT; ++k) {
        Vec8 t = at_da(k);
        const Vec8 hh = at_h(k), w = pre_w(k);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          s_pre[k].v[i] = fma2(t.v[i], hh.v[i], s_pre[k].v[i]);
          s_da[LN ? k : 0].v[i] = add2(s_da[LN ? k : 0].v[i], t.v[i]);
          t.v[i] = mul2(t.v[i], w.v[i]);
          q1 = fma2(t.v[i], hh.v[i], q1);
          q0 = add2(q0, t.v[i]);
        }
      }
      float q[2] = {q1.x + q1.y, q0.x + q0.y};
      group_sum(pl, red, half, q);
      refill();
      n1 = -q[0] * p.inv_d;
      n0 = -q[1] * p.inv_d;
    }

    // dh, dx and the sums of dh; dy at once (RMSNorm) or after its sums
    T* rowx = dx + orow * p.x_ld + 8 * pl.lane;
    T* rowy = dy + orow * p.y_ld + 8 * pl.lane;
    const f2 n1b = both(n1), n0b = both(n0);
    f2 q1 = both(0.f), q0 = both(0.f);
    Vec8 w2[VL];   // LayerNorm: c1 dh
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      Vec8 d = at_dh(k);
      if (p.pre) {
        const Vec8 t = at_da(k), hh = at_h(k), w = pre_w(k);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const f2 g = LN ? fma2(t.v[i], w.v[i], fma2(hh.v[i], n1b, n0b)) : fma2(t.v[i], w.v[i], mul2(hh.v[i], n1b));
          d.v[i] = fma2(rh, g, d.v[i]);
        }
      }
      Vec8 o;
      if (RES) {
        const Vec8 l = param8<T>(p.res_w, pl.lane + k * p.tpr, on(k), 0.f);
        const Vec8 xv = get8<T>(on(k) && x ? stage + o_x + off + k * hop : zero);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          o.v[i] = mul2(d.v[i], mul2(al, l.v[i]));
          s_res[RES ? k : 0].v[i] = fma2(d.v[i], xv.v[i], s_res[RES ? k : 0].v[i]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) o.v[i] = mul2(d.v[i], al);
      }
      if (on(k)) put8(rowx + k * p.tpr * 8, o);
      if (!p.branch) continue;
      // (beyond the row dh and yh need not be 0 with LayerNorm; c1 is, so the
      // row's sums get nothing from there, and those columns are never stored)
      const Vec8 yh = at_y(k);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        s_dhy[k].v[i] = fma2(d.v[i], yh.v[i], s_dhy[k].v[i]);
        const f2 w = mul2(c1[k].v[i], d.v[i]);
        if (LN) {
          s_dh[LN ? k : 0].v[i] = add2(s_dh[LN ? k : 0].v[i], d.v[i]);
          q1 = fma2(w, yh.v[i], q1);
          q0 = add2(q0, w);
          w2[LN ? k : 0].v[i] = w;
        } else {
          o.v[i] = mul2(ry, fma2(yh.v[i], both(o1), w));
        }
      }
      if (!LN && on(k)) put8(rowy + k * p.tpr * 8, o);
    }
    if (LN && p.branch) {
      float m1 = 0.f, m0 = 0.f;
      if (p.post) {
        float q[2] = {q1.x + q1.y, q0.x + q0.y};
        group_sum(pl, red, half, q);
        if (!p.pre) refill();
        m1 = -q[0] * p.inv_d;
        m0 = -q[1] * p.inv_d;
      }
#pragma unroll
      for (int k = 0; k < VPT; ++k) {
        const Vec8 yh = at_y(k);
        Vec8 o;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          o.v[i] = mul2(ry, fma2(yh.v[i], both(m1), add2(w2[LN ? k : 0].v[i], both(m0))));
        if (on(k)) put8(rowy + k * p.tpr * 8, o);
      }
    }
    row_done();
  }

  // the column sums: gates of sequences by group (above), the others over the CTA's groups
  if (by_seq && mine) {
    while (b < b_last) end_sequence(false);
    end_sequence(true);
  }
  __syncthreads();
  if (*abort_flag && pl.lane == 0) drain(bar0, p.stages, parity);
  if (!mine || *abort_flag) return;
  float* line = reinterpret_cast<float*>(smem + p.ring_at);   // the rings are done with
  auto park = [&](int q, auto&& value) {
    if (!p.sums[q]) return;
    float* to = p.groups > 1 ? line + (q * p.groups + pl.group) * p.D : p.part + ((long long)q * p.grid + blockIdx.x) * p.D;
#pragma unroll
    for (int k = 0; k < VPT; ++k)
      if (pl.lane + k * p.tpr < vecs) put8(to + 8 * (pl.lane + k * p.tpr), value(k));
  };
  auto scaled = [&](const void* w, const Vec8& a, int k) {   // a times a parameter vector, where there is one
    Vec8 o = param8<T>(w, pl.lane + k * p.tpr, true, 1.f);
#pragma unroll
    for (int i = 0; i < 4; ++i) o.v[i] = mul2(o.v[i], a.v[i]);
    return o;
  };
  park(kPreW, [&](int k) { return s_pre[k]; });
  if (LN) park(kPreB, [&](int k) { return s_da[LN ? k : 0]; });
  if (RES) park(kResW, [&](int k) { return s_res[RES ? k : 0]; });
  if (by_seq) {
    park(kPostW, [&](int k) { return u[k]; });
    if (LN) park(kPostB, [&](int k) { return u[VPT + k]; });
  } else {
    park(kPostW, [&](int k) { return scaled(gate_at(0), s_dhy[k], k); });
    if (LN) park(kPostB, [&](int k) { return scaled(gate_at(0), s_dh[LN ? k : 0], k); });
    park(kGate, [&](int k) {
      Vec8 o = scaled(p.post_w, s_dhy[k], k);
      if (LN && p.post_b) {
        const Vec8 e = scaled(p.post_b, s_dh[LN ? k : 0], k);
#pragma unroll
        for (int i = 0; i < 4; ++i) o.v[i] = add2(o.v[i], e.v[i]);
      }
      return o;
    });
  }
  if (p.groups > 1) {
    __syncthreads();
    for (int q = 0; q < kSums; ++q) {
      if (!p.sums[q] || (q == kGate && by_seq)) continue;
      for (int c = threadIdx.x; c < p.D; c += blockDim.x) {
        float sum = 0.f;
        for (int g = 0; g < p.groups; ++g) sum += line[(q * p.groups + g) * p.D + c];
        p.part[((long long)q * p.grid + blockIdx.x) * p.D + c] = sum;
      }
    }
  }
}

// After the rows: zeros where there is no kept row (the first zero_ctas blocks
// of y), and sums[q][c] = the parked sums added in slot order, 32 columns a
// block, 32 threads a column, each every 32nd slot, then the 32 in order.
// blockIdx.y counts the gradients there are, a gate by sequences as B of them.
// The zero blocks touch only rows that the first kernel does not.
template <typename T>
__global__ void __launch_bounds__(1024) join_finish_kernel(BwdArgs p, int zero_ctas) {
  __shared__ float red[32][33];
  const int nk = kept(p);
  if ((int)blockIdx.y < zero_ctas) {
    T *dx = static_cast<T*>(p.dx), *dy = static_cast<T*>(p.dy);
    const int zeros = p.out_full ? p.M - nk : padded_rows(nk, p.M) - nk, vecs = p.D / 8;
    const int warps = gridDim.x * zero_ctas * 32, lane = threadIdx.x & 31;
    for (int j = (blockIdx.y * gridDim.x + blockIdx.x) * 32 + (threadIdx.x >> 5); j < zeros; j += warps) {
      const long long row = p.out_full ? filtered_token(p.idx, nk, j) : nk + j;
      for (int v = lane; v < vecs; v += 32) {
        put8(dx + row * p.x_ld + 8 * v, all8(0.f));
        if (p.branch) put8(dy + row * p.y_ld + 8 * v, all8(0.f));
      }
    }
    grid_dep_wait();
    return;
  }
  grid_dep_wait();
  int q = 0, b = blockIdx.y - zero_ctas;
  for (;; ++q) {
    const int n = !p.sums[q] ? 0 : (q == kGate && p.gate_rows > 1) ? p.B : 1;
    if (b < n) break;
    b -= n;
  }
  const int A = active(p, nk);
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

constexpr int kMaxSms = 256;

template <typename T, bool LN, int SRC, int VPT, bool RES>
cudaError_t launch(const Ctx& c, const BwdArgs& p, size_t smem) {
  constexpr int MINB = VPT <= 2 ? 2 : 1;
  auto k = join_bwd_kernel<T, LN, SRC, VPT, RES, MINB>;
  static size_t granted[64];   // shared memory opted in to, a device
  const cudaError_t e = grant_smem(reinterpret_cast<const void*>(k), smem, granted);
  if (e != cudaSuccess) return e;
  k<<<p.grid, p.tpr * p.groups, smem, c.stream>>>(p, c.st);
  return cudaGetLastError();
}
template <typename T, bool LN, int SRC, bool RES>
cudaError_t by_vpt(const Ctx& c, const BwdArgs& p, int vpt, size_t smem) {
  return vpt == 1   ? launch<T, LN, SRC, 1, RES>(c, p, smem)
         : vpt == 2 ? launch<T, LN, SRC, 2, RES>(c, p, smem)
                    : launch<T, LN, SRC, 4, RES>(c, p, smem);
}
template <typename T, bool LN, int SRC>
cudaError_t by_res(const Ctx& c, const BwdArgs& p, int vpt, size_t smem) {
  // (a learned residual scale: its sums and the reads of x and res_w)
  return p.res_w ? by_vpt<T, LN, SRC, true>(c, p, vpt, smem) : by_vpt<T, LN, SRC, false>(c, p, vpt, smem);
}
template <typename T, bool LN>
cudaError_t by_src(const Ctx& c, const BwdArgs& p, int src, int vpt, size_t smem) {
  if (src == kQ8E4m3) return by_res<T, LN, kQ8E4m3>(c, p, vpt, smem);
  if (src == kQ8Int8) return by_res<T, LN, kQ8Int8>(c, p, vpt, smem);
  return by_res<T, LN, kSrcSame>(c, p, vpt, smem);
}

// Launch shape: one vector of 8 a thread up to 2048 values, more for wider rows;
// two CTAs an SM where two stages of each fit.
struct BwdShape {
  Shape s;
  int ctas;        // an SM
  size_t own;      // bytes of the threads' own sums (gates by sequence)
};
BwdShape bwd_shape(int D, uint32_t stage, bool layer_norm, bool by_seq) {
  auto shape = [&](int vpt, int ctas) {
    BwdShape b{};
    b.ctas = ctas;
    const Shape t = make_shape(D, vpt, stage, 0, 0);
    b.own = by_seq ? (size_t)t.groups * t.tpr * vpt * 8 * 4 * (layer_norm ? 2 : 1) : 0;
    b.s = make_shape(D, vpt, stage, b.own, (ctas == 2 ? 112 : 224) * 1024);
    const size_t line = head_bytes(t.groups) + b.own + (t.groups > 1 ? (size_t)kSums * t.groups * D * 4 : 0);
    if (b.s.smem < line) b.s.smem = line;
    return b;
  };
  if (D > 4096) return shape(4, 1);
  if (D > 2048) {
    const BwdShape two = shape(2, 2);
    return two.s.stages >= 2 ? two : shape(2, 1);
  }
  return shape(1, 2);
}
int bwd_grid(int M, int num_sms, int groups, int ctas) {
  const long long want = ((long long)M + groups - 1) / groups, fit = (long long)std::min(num_sms, kMaxSms) * ctas;
  return (int)(want < fit ? want : fit);
}

}  // namespace

// partial sums of the widest grid on any GPU of up to kMaxSms SMs
size_t join_bwd_part_floats(int B, int T, int D, int gate_rows) {
  const int groups = make_shape(D, D <= 256 ? 1 : D <= 4096 ? 2 : 4, 16, 0, 0).groups;   // the most there are
  const long long grid = std::min<long long>((long long)B * T, kMaxSms * 2);
  return (size_t)(grid * kSums + (gate_rows > 1 ? (grid + B) * groups : 0)) * D;
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
  const BwdShape bs = bwd_shape(j.D, kHeadBytes + total, j.layer_norm != 0, j.gate_rows > 1);
  const Shape& s = bs.s;
  p.tpr = s.tpr; p.groups = s.groups; p.stages = s.stages; p.stage_bytes = s.stage_bytes;
  p.ring_at = (uint32_t)(head_bytes(s.groups) + bs.own);
  p.grid = bwd_grid(p.M, c.num_sms, s.groups, bs.ctas);
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
  // blocks that write zeros: a warp for each row there may be, 2 blocks an SM at most
  const int cols = (j.D + 31) / 32;
  const bool some = j.nk != nullptr;   // (dense: every row is kept)
  const long long rows = some ? (j.out_full ? p.M : std::min(p.M, 127)) : 0;
  const int zero_ctas = (int)((std::min(2LL * c.num_sms, (rows + 31) / 32) + cols - 1) / cols);
  if (tasks + zero_ctas == 0) return cudaSuccess;
  prof_begin(c, "residual_norm_finish");
  const dim3 grid(cols, tasks + zero_ctas);
  if (j.f32) e = launch_k(c, pdl_allowed(), join_finish_kernel<float>, grid, dim3(1024), 0, 1, p, zero_ctas);
  else e = launch_k(c, pdl_allowed(), join_finish_kernel<__nv_bfloat16>, grid, dim3(1024), 0, 1, p, zero_ctas);
  prof_end(c);
  count_launch();
  return launched(e);
}

}  // namespace collider
