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
// Floor: da, dH, y, h are read and dx, dy written once (12 D bytes a kept row in
// bf16, 10 D with 8-bit y and h) beside the zeros.  What bounds it is the
// instructions of a row at 16 warps an SM (0.50 issued a cycle and scheduler): at
// 4 x 2048 tokens of 2048 values, 40% filtered, the whole call takes 37.0 us,
// 4.0 TB/s of the floor's bytes (22.0 us).  On the way there: both row sums taken one after
// the other 65 us (a row waited twice for the group), all sums at once and two
// rows in flight 52, tensors kept in registers from a row's sums to its gradients
// and no question asked in the row loop 42, the pre norm's weight in registers 38.
// More CTAs an SM do not fit: above 102 registers a thread an SM's quarter holds
// four warps.
// Each thread owns the same columns of every row it sees and keeps their
// parameter sums in registers; a CTA's sums are parked in the workspace and added
// in CTA order by a second kernel, so the results do not change from run to run.
#include <algorithm>

#include "join.cuh"

namespace collider {

using namespace join;

namespace {

constexpr int kSrcSame = 2;   // y and h as stored (else kQ8E4m3, kQ8Int8)
// column sums
enum { kPreW, kPostW, kGate, kResW, kPreB, kPostB, kSums };
constexpr uint32_t kHeadBytes = 32;   // a warp's copy of a row's token and statistics

struct BwdArgs {
  int M, T, B, D;
  float inv_d, alpha;
  int gate_rows, post, pre, branch;
  const void *da, *dh, *x, *y, *h;     // y, h: T rows, or codes
  const uint8_t *y_exps, *h_exps;
  // bytes between rows (below 2^32, so that a row's offset is one multiplication)
  uint32_t a_ld, h_ld, x_ld, y_ld;     // of a, h, x, y and their gradients
  uint32_t ys_ld, hs_ld, ye_ld, he_ld; // of the saved y, h and of their exponents
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

// a stage's exponent bytes: two a vector, rounded up to whole 16s
__host__ __device__ constexpr uint32_t exps_bytes(int tpr, int vpt) { return (tpr * vpt * 2 + 15) / 16 * 16; }

template <typename T>
__device__ __forceinline__ T* row_of(T* base, uint32_t row, uint32_t ld) {
  return reinterpret_cast<T*>(reinterpret_cast<uintptr_t>(base) + (uint64_t)row * ld);
}

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

template <typename T, bool LN, int SRC, int VPT, bool RES>
__global__ void __launch_bounds__(kThreads) join_bwd_kernel(BwdArgs p, DevStatus* st) {
  extern __shared__ __align__(128) uint8_t smem[];
  const Place pl(p.tpr);
  float* red = reinterpret_cast<float*>(smem + pl.group * kRedBytes);
  uint8_t* ring = smem + p.ring_at + (size_t)pl.group * p.stages * p.stage_bytes;
  const uint32_t ring0 = tc::smem_u32(ring);
  for (int i = threadIdx.x; i < (int)(head_bytes(p.groups) / 4); i += blockDim.x) reinterpret_cast<uint32_t*>(smem)[i] = 0;
  __syncthreads();

  const T *da = static_cast<const T*>(p.da), *dh = static_cast<const T*>(p.dh), *x = static_cast<const T*>(p.x);
  const uint8_t *y = static_cast<const uint8_t*>(p.y), *h = static_cast<const uint8_t*>(p.h);
  T *dx = static_cast<T*>(p.dx), *dy = static_cast<T*>(p.dy);
  const int vecs = p.D / 8;
  const int nk = kept(p);
  // a stage: each warp's copy of the row's token and statistics, each thread's of
  // its exponent bytes of h and y, then da | dH | h | y (| x), each with a place
  // for every thread.  Places that no copy reaches (beyond the row, tensors not
  // given) hold zeros, which is what their values are, so that the row loop
  // reads and adds without asking.
  const uint32_t heads = pl.warps * kHeadBytes + (SRC == kSrcSame ? 0 : exps_bytes(p.tpr, VPT));
  const uint32_t place = p.tpr * VPT * 8 * (uint32_t)sizeof(T), s_place = SRC == kSrcSame ? place : p.tpr * VPT * 8;
  const uint32_t o_da = heads, o_dh = o_da + place, o_h = o_dh + place, o_y = o_h + s_place, o_x = o_y + s_place;
  // Rows of this group: first, first + step, ... below r1.  Strided over the
  // grid, or, where gates differ by sequence, from a contiguous share of the
  // rows, so that a CTA sees few sequences.
  const bool by_seq = p.gate_rows > 1;
  const int A = active(p, nk);
  const bool mine = (int)blockIdx.x < A;
  const int r0 = by_seq && mine ? (int)((long long)blockIdx.x * nk / A) : blockIdx.x * p.groups,
            r1 = !mine ? 0 : by_seq ? (int)((long long)(blockIdx.x + 1) * nk / A) : nk;
  const int step = by_seq ? p.groups : gridDim.x * p.groups, first = r0 + pl.group;
  struct Head {
    float rh, ry, mh, my;
    int token;   // -1: an index outside the tokens
  };
  static_assert(sizeof(Head) <= kHeadBytes, "");
  // The tokens of rows j = 32 n .. 32 n + 31 of this group, one a lane: the block
  // that is being filled, and the one after it.
  auto tokens = [&](int n) {
    const long long r = first + (32ll * n + (pl.lane & 31)) * step;
    if (r >= r1) return -1;
    const int t = p.idx ? p.idx[r] : (int)r;
    return (unsigned)t < (unsigned)p.M ? t : -1;
  };
  int block = 0, t_now = tokens(0), t_after = tokens(1);
  auto token = [&](int j) {   // of row j >= 32 block, in order
    if ((j >> 5) != block) {
      block = j >> 5;
      t_now = t_after;
      t_after = tokens(block + 1);
    }
    return __shfl_sync(0xffffffffu, t_now, j & 31);
  };
  const uint32_t off = pl.lane * 8 * (uint32_t)sizeof(T), hop = p.tpr * 8 * (uint32_t)sizeof(T);
  const uint32_t s_off = SRC == kSrcSame ? off : pl.lane * 8, s_hop = SRC == kSrcSame ? hop : p.tpr * 8;
  const uint32_t my_head = (pl.lane >> 5) * kHeadBytes;
  // Exponent bytes are loaded when their row is filled, and put where its
  // columns are a row later: e_h, e_y are on their way to stage e_stage.
  unsigned e_h[VPT] = {}, e_y[VPT] = {};
  int e_stage = -1;
  uint8_t* my_exps = ring + pl.warps * kHeadBytes + pl.lane * 2 * VPT;
  auto land_exps = [&] {
    if constexpr (SRC != kSrcSame) {
      if (e_stage < 0) return;
#pragma unroll
      for (int k = 0; k < VPT; ++k) {
        my_exps[e_stage * p.stage_bytes + 2 * k] = (uint8_t)e_h[k];
        my_exps[e_stage * p.stage_bytes + 2 * k + 1] = (uint8_t)e_y[k];
      }
      e_stage = -1;
    }
  };
  // row j of this group, if there is one, into stage s: this thread's columns,
  // and a few lanes of each warp its statistics
  auto fill = [&](int j, int s) {
    const int t = token(j), r = first + j * step;
    if (r < r1) {
      const uint32_t d = ring0 + s * p.stage_bytes;
      const int lane = pl.lane & 31;
      if (lane == 0) reinterpret_cast<Head*>(ring + s * p.stage_bytes + my_head)->token = t;
      if (t >= 0) {
        if (lane == 0 && p.pre) copy4(d + my_head, p.rstd_h + t);
        if (lane == 1 && p.post) copy4(d + my_head + 4, p.rstd_y + t);
        if (LN && lane == 2 && p.pre) copy4(d + my_head + 8, p.mean_h + t);
        if (LN && lane == 3 && p.post) copy4(d + my_head + 12, p.mean_y + t);
        const int sr = p.saved_full ? t : r, ir = p.in_full ? t : r;
        const T *s_da = row_of(da + 8 * pl.lane, ir, p.a_ld), *s_dh = row_of(dh + 8 * pl.lane, ir, p.h_ld),
                *s_x = row_of(x + 8 * pl.lane, sr, p.x_ld);
        const uint8_t *s_h = row_of(h + s_off, sr, p.hs_ld), *s_y = row_of(y + s_off, sr, p.ys_ld);
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
          const int v = pl.lane + k * p.tpr;
          if (v >= vecs) continue;
          if (da) copy_vec(d + o_da + off + k * hop, s_da + k * p.tpr * 8);
          if (dh) copy_vec(d + o_dh + off + k * hop, s_dh + k * p.tpr * 8);
          if (RES && x) copy_vec(d + o_x + off + k * hop, s_x + k * p.tpr * 8);
          if constexpr (SRC == kSrcSame) {
            if (h) copy_vec(d + o_h + off + k * hop, reinterpret_cast<const T*>(s_h) + k * p.tpr * 8);
            if (y) copy_vec(d + o_y + off + k * hop, reinterpret_cast<const T*>(s_y) + k * p.tpr * 8);
          } else {
            if (h) copy8(d + o_h + s_off + k * s_hop, s_h + k * s_hop);
            if (y) copy8(d + o_y + s_off + k * s_hop, s_y + k * s_hop);
            e_h[k] = h ? row_of(p.h_exps, sr, p.he_ld)[v >> 2] : 0;
            e_y[k] = y ? row_of(p.y_exps, sr, p.ye_ld)[v >> 2] : 0;
          }
        }
        e_stage = s;
      }
    }
    copy_commit();
  };
  // the sums' kernel may be scheduled as blocks of this one exit
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (!da || !dh || !y || (RES && !x) || vecs < p.tpr * VPT) {
    for (uint32_t i = threadIdx.x; i < p.groups * p.stages * (p.stage_bytes / 16); i += blockDim.x)
      reinterpret_cast<uint4*>(smem + p.ring_at)[i] = make_uint4(0, 0, 0, 0);
    __syncthreads();
  }
  if ((pl.lane & 31) == 0)   // statistics that are not read: 1, and 0
    for (int j = 0; j < p.stages; ++j)
      *reinterpret_cast<Head*>(ring + j * p.stage_bytes + my_head) = Head{1.f, 1.f, 0.f, 0.f, -1};
  __syncwarp();
  for (int j = 0; j < p.stages; ++j) {
    land_exps();
    fill(j, j);
  }
  // Zeros where there is no kept row -- the filtered tokens of FULL outputs, the
  // padding of COMPACT ones -- are a warp's a row, 32 vectors at a time between
  // its other work.
  const int zeros = p.out_full ? p.M - nk : padded_rows(nk, p.M) - nk, z_step = gridDim.x * (blockDim.x >> 5);
  int z = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5), z_vec = 0;
  auto zero_row = [&] { return z >= zeros ? 0 : p.out_full ? filtered_token(p.idx, nk, z) : nk + z; };
  int z_row = zero_row();
  auto zero_some = [&] {
    if (z >= zeros) return;
    const int v = z_vec + (threadIdx.x & 31);
    if (v < vecs) {
      put8(row_of(dx + 8 * v, z_row, p.x_ld), all8(0.f));
      if (p.branch) put8(row_of(dy + 8 * v, z_row, p.y_ld), all8(0.f));
    }
    z_vec += 32;
    if (z_vec >= vecs) {
      z += z_step;
      z_vec = 0;
      z_row = zero_row();
    }
  };

  // Column sums over this group's rows: of da hh, da (LN), and -- of one
  // sequence while gates differ by sequence -- of dh yh, dh (LN); of dh x.
  constexpr int VL = LN ? VPT : 1, VR = RES ? VPT : 1;
  constexpr int NS = LN ? 16 : 4;   // sums a row (10 of them used with LayerNorm)
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

  Raw8<T> w_pre[VPT];   // this thread's part of the pre norm's weight (0 where there is none), as stored
  const T* w_res[VR];   // and its places of res_w
#pragma unroll
  for (int k = 0; k < VPT; ++k) {
    const int v = pl.lane + k * p.tpr;
    const T* zero = reinterpret_cast<const T*>(smem + zero_at(p.groups));
    w_pre[k] = *reinterpret_cast<const Raw8<T>*>(p.pre && v < vecs ? static_cast<const T*>(p.pre_w) + 8 * v : zero);
    if (RES) w_res[RES ? k : 0] = v < vecs ? static_cast<const T*>(p.res_w) + 8 * v : zero;
  }

  // The rows, two at a time: while row i's sums travel through the group, row
  // i - 1's, which every thread can read by then, become its gradients; so one
  // barrier a row, which nothing waits for at once.  Of row i - 1 a thread keeps
  // t = gamma da, hh, yh and dH.
  const f2 al = both(p.alpha);
  Vec8 t[VPT], hh[VPT], yh[VPT], d[VPT];
  f2 rh = both(1.f), ry = rh;
  int s = 0, prev = 0;    // stages of rows i and i - 1
  int old_token = -1;     // of row i - 1, -1: there is none to finish
  for (int r = first, i = 0; r - step < r1; r += step, ++i) {
    if (old_token >= 0) {
      // row i - 1: its sums, dh, dx, dy and the columns' sums
      float q[NS];
      take_sums(pl, red + ((i - 1) & 1) * kMaxSums * kMaxWarps, q);
      const float n1 = -q[0] * p.inv_d;   // -mean(t hh)
      const float n0 = LN ? -q[LN ? 4 : 0] * p.inv_d : 0.f;   // -mean(t)
      // -mean(w yh) and -mean(w), w = c1 dh = c1 (dH + r_h (t + hh n1 + n0))
      float o1 = fmaf(n1, q[3], q[2]), o0 = 0.f;
      if (LN) {
        o1 = fmaf(n0, q[LN ? 5 : 0], o1);
        o0 = fmaf(n0, q[LN ? 9 : 0], fmaf(n1, q[LN ? 8 : 0], q[LN ? 7 : 0]));
        o0 = -fmaf(rh.x, o0, q[LN ? 6 : 0]) * p.inv_d;
      }
      o1 = -fmaf(rh.x, o1, q[1]) * p.inv_d;
      if (!p.post) o1 = o0 = 0.f;
      const int orow = p.out_full ? old_token : r - step;
      T *rowx = row_of(dx + 8 * pl.lane, orow, p.x_ld), *rowy = row_of(dy + 8 * pl.lane, orow, p.y_ld);
      const f2 n1b = both(n1), n0b = both(n0), o1b = both(o1), o0b = both(o0);
#pragma unroll
      for (int k = 0; k < VPT; ++k) {
        const bool on = pl.lane + k * p.tpr < vecs;
        Vec8 o;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const f2 u = LN ? add2(fma2(hh[k].v[j], n1b, n0b), t[k].v[j]) : fma2(hh[k].v[j], n1b, t[k].v[j]);
          d[k].v[j] = fma2(rh, u, d[k].v[j]);
        }
        if (RES) {
          const Vec8 l = get8<T>(w_res[RES ? k : 0]);
          const Vec8 xv = get8<T>(ring + prev * p.stage_bytes + o_x + off + k * hop);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            o.v[j] = mul2(d[k].v[j], mul2(al, l.v[j]));
            s_res[RES ? k : 0].v[j] = fma2(d[k].v[j], xv.v[j], s_res[RES ? k : 0].v[j]);
          }
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) o.v[j] = mul2(d[k].v[j], al);
        }
        if (on) put8(rowx + k * p.tpr * 8, o);
        // (beyond the row dh and yh need not be 0 with LayerNorm; those columns are never stored)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          s_dhy[k].v[j] = fma2(d[k].v[j], yh[k].v[j], s_dhy[k].v[j]);
          if (LN) s_dh[LN ? k : 0].v[j] = add2(s_dh[LN ? k : 0].v[j], d[k].v[j]);
          const f2 c = mul2(c1[k].v[j], d[k].v[j]);
          o.v[j] = mul2(ry, LN ? add2(fma2(yh[k].v[j], o1b, o0b), c) : fma2(yh[k].v[j], o1b, c));
        }
        if (on && p.branch) put8(rowy + k * p.tpr * 8, o);
      }
    }
    // row i - 1's stage takes the row `stages` further on, once the warp is done with it
    __syncwarp();
    land_exps();
    if (i > 0) {
      fill(i - 1 + p.stages, prev);
      if (p.stages == 1) land_exps();
    } else {
      copy_commit();
    }
    if (r < r1) {
      while (r >= b_end && b < b_last) end_sequence(false);
      copy_wait(p.stages - 1);
      __syncwarp();   // the head was copied by a few lanes
      const uint8_t* at = ring + s * p.stage_bytes;
      const Head hd = *reinterpret_cast<const Head*>(at + my_head);
      old_token = hd.token;
      if (old_token < 0) {   // (the same in every thread of the group)
        if (pl.lane == 0) report_error(st, kErrBadIndex, 721);
      } else {
        // Row i's sums, all at once: with m1 = mean(t hh) (and m0 = mean(t)),
        //   sum(w yh) = sum(c1 yh dH) + r_h (sum(c1 yh t) - m1 sum(c1 yh hh) - m0 sum(c1 yh)),
        // and sum(w) the same without yh, so that the post norm's sums need not wait for dh.
        rh = both(hd.rh);
        ry = both(hd.ry);
        const f2 mh = both(-hd.mh), my = both(-hd.my);
        const uint8_t* e = my_exps + s * p.stage_bytes;
        f2 q[NS];
#pragma unroll
        for (int j = 0; j < NS; ++j) q[j] = both(0.f);
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
          t[k] = get8<T>(at + o_da + off + k * hop);
          hh[k] = saved8<T, SRC>(at + o_h + s_off + k * s_hop, SRC == kSrcSame ? 0 : e[2 * k]);
          yh[k] = saved8<T, SRC>(at + o_y + s_off + k * s_hop, SRC == kSrcSame ? 0 : e[2 * k + 1]);
          d[k] = get8<T>(at + o_dh + off + k * hop);
          const Vec8 g = get8<T>(&w_pre[k]);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            hh[k].v[j] = mul2(LN ? add2(hh[k].v[j], mh) : hh[k].v[j], rh);
            yh[k].v[j] = mul2(LN ? add2(yh[k].v[j], my) : yh[k].v[j], ry);
            s_pre[k].v[j] = fma2(t[k].v[j], hh[k].v[j], s_pre[k].v[j]);
            if (LN) s_da[LN ? k : 0].v[j] = add2(s_da[LN ? k : 0].v[j], t[k].v[j]);
            t[k].v[j] = mul2(t[k].v[j], g.v[j]);
            const f2 c = c1[k].v[j], cy = mul2(c, yh[k].v[j]);
            q[0] = fma2(t[k].v[j], hh[k].v[j], q[0]);
            q[1] = fma2(cy, d[k].v[j], q[1]);
            q[2] = fma2(cy, t[k].v[j], q[2]);
            q[3] = fma2(cy, hh[k].v[j], q[3]);
            if (LN) {
              q[LN ? 4 : 0] = add2(q[LN ? 4 : 0], t[k].v[j]);
              q[LN ? 5 : 0] = add2(q[LN ? 5 : 0], cy);
              q[LN ? 6 : 0] = fma2(c, d[k].v[j], q[LN ? 6 : 0]);
              q[LN ? 7 : 0] = fma2(c, t[k].v[j], q[LN ? 7 : 0]);
              q[LN ? 8 : 0] = fma2(c, hh[k].v[j], q[LN ? 8 : 0]);
              q[LN ? 9 : 0] = add2(q[LN ? 9 : 0], c);
            }
          }
        }
        float v[NS];
#pragma unroll
        for (int j = 0; j < NS; ++j) v[j] = q[j].x + q[j].y;
        leave_sums(pl, red + (i & 1) * kMaxSums * kMaxWarps, v);
      }
    }
    zero_some();
    pl.sync();   // row i's sums are left
    prev = s;
    if (++s == p.stages) s = 0;
  }

  // the column sums: gates of sequences by group (above), the others over the CTA's groups
  if (by_seq && mine) {
    while (b < b_last) end_sequence(false);
    end_sequence(true);
  }
  while (z < zeros) zero_some();
  if (!mine) return;
  __syncthreads();
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

// sums[q][c] = the parked sums added in slot order: 32 columns a block, 32
// threads a column, each every 32nd slot, then the 32 in order.  blockIdx.x
// counts the gradients there are, a gate by sequences as B of them (which may be
// more than the 65535 blocks of y).
__global__ void __launch_bounds__(1024) join_sums_kernel(BwdArgs p) {
  __shared__ float red[32][33];
  grid_dep_wait();
  const int nk = kept(p);
  int q = 0, b = blockIdx.x;
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
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5, c = blockIdx.y * 32 + tx;
  float sum = 0.f;
  if (c < p.D) {
#pragma unroll 8
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
  auto k = join_bwd_kernel<T, LN, SRC, VPT, RES>;
  static size_t granted[64];   // shared memory opted in to, a device
  const cudaError_t e = grant_smem(reinterpret_cast<const void*>(k), smem, granted);
  if (e != cudaSuccess) return e;
  k<<<p.grid, p.tpr * p.groups, smem, c.stream>>>(p, c.st);
  return cudaGetLastError();
}
template <typename T, bool LN, int SRC, bool RES>
cudaError_t by_vpt(const Ctx& c, const BwdArgs& p, int vpt, size_t smem) {
  return vpt == 1 ? launch<T, LN, SRC, 1, RES>(c, p, smem) : launch<T, LN, SRC, 2, RES>(c, p, smem);
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

// Launch shape: one vector of 8 a thread up to 4096 values, two for wider rows;
// two CTAs an SM up to 2048 values (their registers leave no room for more).
struct BwdShape {
  Shape s;
  int ctas;        // an SM
  size_t own;      // bytes of the threads' own sums (gates by sequence)
};
// bytes: of the T tensors' values and of the saved ones' in a stage, a value
BwdShape bwd_shape(int D, uint32_t bytes, bool eight, bool layer_norm, bool by_seq) {
  BwdShape b{};
  const int vpt = D <= 4096 ? 1 : 2;
  b.ctas = D <= 2048 ? 2 : 1;
  const Shape t = make_shape(D, vpt, 16, 0, 0);
  const uint32_t stage = t.tpr * vpt * 8 * bytes + t.tpr / 32 * kHeadBytes + (eight ? exps_bytes(t.tpr, vpt) : 0);
  b.own = by_seq ? (size_t)t.groups * t.tpr * vpt * 8 * 4 * (layer_norm ? 2 : 1) : 0;
  // (64 KB of ring a CTA: more stages only lengthen the start.  4 x 2048 tokens of 2048 values: 37.0 us, 39.1 at
  // 112 KB; 2 x 4096 of 1536, y and h in 8 bits: 39.2 and 39.1)
  b.s = make_shape(D, vpt, stage, b.own, 64 * 1024 + b.own);
  if (b.s.stages < 2) b.s = make_shape(D, vpt, stage, b.own, (b.ctas == 2 ? 112 : 224) * 1024);
  const size_t line = head_bytes(t.groups) + b.own + (t.groups > 1 ? (size_t)kSums * t.groups * D * 4 : 0);
  if (b.s.smem < line) b.s.smem = line;
  return b;
}
int bwd_grid(int M, int num_sms, int groups, int ctas) {
  const long long want = ((long long)M + groups - 1) / groups, fit = (long long)std::min(num_sms, kMaxSms) * ctas;
  return (int)(want < fit ? want : fit);
}

}  // namespace

// partial sums of the widest grid on any GPU of up to kMaxSms SMs
size_t join_bwd_part_floats(int B, int T, int D, int gate_rows) {
  const int groups = make_shape(D, D <= 4096 ? 1 : 2, 16, 0, 0).groups;
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
  const bool same = j.src == kSrcSame;
  const int es = j.f32 ? 4 : 2;
  p.a_ld = (uint32_t)(j.a_ld * es); p.h_ld = (uint32_t)(j.h_ld * es);
  p.x_ld = (uint32_t)(j.x_ld * es); p.y_ld = (uint32_t)(j.y_ld * es);
  p.ys_ld = same ? p.y_ld : (uint32_t)j.y_code_ld; p.hs_ld = same ? p.h_ld : (uint32_t)j.h_code_ld;
  p.ye_ld = (uint32_t)j.y_exp_ld; p.he_ld = (uint32_t)j.h_exp_ld;
  p.post_w = j.post_w; p.post_b = j.post_b; p.gate = j.gate; p.res_w = j.res_w; p.pre_w = j.pre_w;
  p.mean_y = j.mean_y; p.rstd_y = j.rstd_y; p.mean_h = j.mean_h; p.rstd_h = j.rstd_h;
  p.idx = j.idx; p.cu = j.cu; p.nk = j.nk;
  p.saved_full = j.saved_full; p.in_full = j.in_full; p.out_full = j.out_full;
  p.dx = j.dx; p.dy = j.dy;
  p.sums[kPreW] = j.dpre_w; p.sums[kPreB] = j.dpre_b; p.sums[kPostW] = j.dpost_w; p.sums[kPostB] = j.dpost_b;
  p.sums[kGate] = j.dgate; p.sums[kResW] = j.dres_w;
  // da, dH, (x), h and y
  const uint32_t bytes = (p.res_w ? 3 : 2) * es + 2 * (same ? es : 1);
  const BwdShape bs = bwd_shape(j.D, bytes, !same, j.layer_norm != 0, j.gate_rows > 1);
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
  if (tasks == 0) return cudaSuccess;
  prof_begin(c, "residual_norm_sums");
  e = launch_k(c, pdl_allowed(), join_sums_kernel, dim3(tasks, (j.D + 31) / 32), dim3(1024), 0, 1, p);
  prof_end(c);
  count_launch();
  return launched(e);
}

}  // namespace collider
