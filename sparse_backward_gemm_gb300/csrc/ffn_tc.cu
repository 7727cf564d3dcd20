// The gated feed-forward block's matrix products on the 5th-generation tensor
// cores (sm_103a), each with what stands beside it in the formulas:
//   kUp     [g | u] = x W_up and s = act(g) u in one kernel: a tile's 256
//           accumulator columns are 128 of g and the same 128 of u, so a thread
//           of the epilogue holds both factors of the product in f32;
//   kDs     ds = dy W_down^T and [dg | du] = [ds u act'(g) | ds act(g)],
//           s = act(g) u: ds stays in tensor memory, g and u come through
//           shared memory beside the products;
//   kGroup  up to three plain products in one launch (dx, dW_up and dW_down; or
//           y alone): their tiles form one list, whose tail is cut evenly.
// All three are 2-SM kernels: a pair of CTAs works on a 256 x 256 tile, TMA
// feeds a ring of 64-deep k-slices, one thread issues the MMAs into one of two
// accumulators while the epilogue's warps empty the other.  Each CTA loads its own
// rows and its own half of the columns.  Every wait is bounded.
//   Measured at 8192 x 2048 x 5632, 40% filtered (4916 kept), from memory: kUp 202
// us (1.87 PFLOP/s of bf16, the tensor pipe 84% busy), y 110 us (1.72), kDs 100 us
// (1.14), the backward's group 315 us (1.80).  kDs's MMAs wait half of their time
// for operands: six slices in flight, beside an epilogue that moves 0.28 GB (0.35
// GB of DRAM in 100 us, 1.5 GB through L2).
#include <algorithm>
#include <mutex>

#include "glu.cuh"
#include "internal.h"
#include "tc_ptx.cuh"

namespace collider {

namespace {

using namespace tc;

constexpr int kUp = 0, kDs = 1, kGroup = 2;
// warp 0: TMA; warp 1: MMA and TMEM; the others: epilogue.  kDs's has long
// chains (copy, accumulator, activation, three stores), which twice the warps
// hide better.
constexpr int epi_warps(int epi) { return epi == kDs ? 16 : 8; }
constexpr int kBM = 128, kBK = 64;   // a CTA's rows, a k-slice; a pair's columns: NB, 256 or 128
constexpr uint32_t kABytes = kBM * kBK * 2;
constexpr int kGroupRows = 16;    // 256-row units that follow each other down a column of tiles
constexpr int kMaxWorkers = 80;   // CTA pairs of a launch, at most
constexpr int kMaxTail = 1024;    // tiles of the part that is cut
// kDs: an epilogue warp's chunk, 32 x 16 values of g and of u
constexpr int kDsCols = 16;
constexpr uint32_t kChunkBytes = 32 * kDsCols * 2;
template <int EPI, int NB>
struct Cfg {
  static constexpr uint32_t kStageBytes = kABytes + NB / 2 * kBK * 2;
  static constexpr int kWarps = epi_warps(EPI), kThreads = 64 + 32 * kWarps;
  static constexpr int kStages = EPI == kDs ? 6 : 7;
  static constexpr uint32_t kEpiBytes = EPI == kDs ? kWarps * 2 * kChunkBytes : 0;
  static constexpr size_t kSmem = 1024 + kStages * kStageBytes + kEpiBytes + 256 + (EPI == kGroup ? 4 * (kMaxWorkers + 1) + 64 : 0);
};

struct Maps {
  CUtensorMap m[6];   // A and B of each product
};
struct Params {
  int M, F, kb;       // kUp, kDs: tokens, hidden width, k-slices
  const int32_t* n_kept;   // null: every row
  const int32_t* idx;      // kDs: rows of up (null: in order); kGroup: rows of a product's output that wants them
  // kUp (up null: not kept) / kDs
  __nv_bfloat16 *up, *s, *dgu;
  long long up_ld, cap;    // cap: rows of dgu and s
  int* zero;          // counters that the launch behind this one starts from
  int n_zero;
  // kGroup
  FfnProduct p[3];
  int np;
  uint32_t by_pairs;  // 2^32 / pairs, rounded up
  float* partial;     // [2 * pairs][2][NB / 4][kBM][4] f32
  int* counters;      // [kMaxTail][2], zero on entry and left zero
  DevStatus* st;
};

// A tile list's work: whole tiles for each pair in turn, then the tail.
//   The tiles of all products stand in one list, the longest reductions first;
// pair w takes tiles w, w + W, ...  Where that would leave the last wave poorly
// filled, only the whole waves that fit the even share (all k-slices / W) are
// given out so, and the k-slices of the tiles behind them are cut into
// contiguous ranges, one a pair, that fill each pair up to its share.  A tile
// cut between pairs is finished by whichever comes last, which adds the
// parts that the others parked in memory and its own accumulator, in the order
// of the pairs: the same sum whoever that is.
//   Cutting costs a chain of memory round trips at the end: counting, parking,
// and the finisher's reading of every part.  Measured, in k-slices of 0.3 us: 14
// and 8 for every part but one (6.6 us with two pairs to a tile, 11.4 with four).
// So of ranges long enough for 2, 3, 4 or 5 pairs to a tile the best is taken,
// or none.  (Cut wherever 16 k-slices were gained: 560 x 768 x 1496 backward 44
// us, 36 so; with any number of pairs to a tile the forward of 200 x 256 x 8192
// 63 us, 29 so; never cut, the backward's group of 4916 x 2048 x 5632 20 us
// more.)
constexpr int kCutCost = 14, kPartCost = 8, kMaxParts = 4;
struct Sched {
  int np, W, wid;
  int units[3], tiles[3], kb[3];   // 256-row units, tiles, k-slices of each product
  int first[4];                    // first tile of each product
  int dp;                          // tiles given out whole
  int tail_first[3], tail_off[4];  // first tile of each product's tail, and its k-slices before
  const int* begin;                // [W + 1]: the ranges
};
// t in [a, b) with t % W == w; magic: 2^32 / W rounded up (exact below 2^32 / W)
__device__ __forceinline__ int count_mod(int a, int b, int w, uint32_t magic) {
  const int fa = a > w ? (int)__umulhi(a - w - 1, magic) + 1 : 0, fb = b > w ? (int)__umulhi(b - w - 1, magic) + 1 : 0;
  return max(0, fb - fa);
}

struct Tile {
  int p, k0, k1;
  int m0, n0;     // this CTA's first row, the tile's column of tiles
  int t;
  bool whole;
};
__device__ __forceinline__ void place(int units, int n_tiles, int t, int rank, int* m0, int* n0) {
  const int per = kGroupRows * n_tiles, g = t / per, r = t % per;
  const int gm = min(kGroupRows, units - g * kGroupRows);
  *m0 = (2 * (g * kGroupRows + r % gm) + rank) * kBM;
  *n0 = r / gm;
}

// the pair's pieces of work in order
struct Iter {
  const Sched& s;
  int tile, it, end;
  __device__ Iter(const Sched& sc) : s(sc), tile(sc.wid), it(0), end(0) {
    if (s.dp < s.first[s.np]) {
      it = s.begin[s.wid];
      end = s.begin[s.wid + 1];
    }
  }
  __device__ bool next(int rank, Tile* o) {
    if (tile < s.dp) {
      o->t = tile;
      tile += s.W;
      o->p = 0;
      while (o->p + 1 < s.np && o->t >= s.first[o->p + 1]) ++o->p;
      o->k0 = 0;
      o->k1 = s.kb[o->p];
    } else {
      if (it >= end) return false;
      o->p = 0;
      while (o->p + 1 < s.np && it >= s.tail_off[o->p + 1]) ++o->p;
      const int kb = s.kb[o->p], rel = it - s.tail_off[o->p];
      o->t = s.tail_first[o->p] + rel / kb;
      o->k0 = rel % kb;
      o->k1 = min(kb, o->k0 + end - it);
      it += o->k1 - o->k0;
    }
    o->whole = o->k0 == 0 && o->k1 == s.kb[o->p];
    place(s.units[o->p], s.tiles[o->p] / s.units[o->p], o->t - s.first[o->p], rank, &o->m0, &o->n0);
    return true;
  }
};

// Exchanges between lanes `st` apart: of each pair (a in the lower lane, b in
// the upper) the lower lane's b and the upper lane's a change places.
__device__ __forceinline__ void swap_lanes(uint4& a, uint4& b, int st) {
  const bool hi = (threadIdx.x & st) != 0;
  uint4 s = hi ? a : b;
  s.x = __shfl_xor_sync(0xffffffffu, s.x, st);
  s.y = __shfl_xor_sync(0xffffffffu, s.y, st);
  s.z = __shfl_xor_sync(0xffffffffu, s.z, st);
  s.w = __shfl_xor_sync(0xffffffffu, s.w, st);
  if (hi) a = s; else b = s;
}
// Four 16-byte pieces of each lane's row become one piece of each of four rows:
// piece (lane & 3) of rows (lane & ~3) + i, so that four lanes store 64 bytes of
// one row together (a lane that stores pieces of its own row alone touches 32
// lines with every instruction, four times the L1 cycles).
__device__ __forceinline__ void transpose4(uint4* v) {
  swap_lanes(v[0], v[1], 1);
  swap_lanes(v[2], v[3], 1);
  swap_lanes(v[0], v[2], 2);
  swap_lanes(v[1], v[3], 2);
}
// two pieces likewise: piece (lane & 1) of rows (lane & ~1) + i
__device__ __forceinline__ void transpose2(uint4* v) { swap_lanes(v[0], v[1], 1); }
// The rows that this lane stores to, as offsets (elements), -1: none; of the
// lane's own row `off`, by the whole warp.
struct Rows4 {
  long long off[4];
  __device__ __forceinline__ explicit Rows4(long long own) {
#pragma unroll
    for (int i = 0; i < 4; ++i) off[i] = __shfl_sync(0xffffffffu, own, (threadIdx.x & 28) + i);
  }
};
// 32 bf16 columns from `col` on (below cols) of the warp's 32 rows; v: this
// lane's row.  By the whole warp.
__device__ __forceinline__ void store_bf16x32(__nv_bfloat16* base, const Rows4& rows, int col, int cols, const uint4* packed) {
  uint4 v[4] = {packed[0], packed[1], packed[2], packed[3]};
  transpose4(v);
  col += 8 * (threadIdx.x & 3);
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (rows.off[i] >= 0 && col < cols) *reinterpret_cast<uint4*>(base + rows.off[i] + col) = v[i];
}
__device__ __forceinline__ void pack32(const float* v, uint4* o) {
#pragma unroll
  for (int g = 0; g < 4; ++g) o[g] = pack8(v + 8 * g);
}
// the same of a product's output, bf16 or f32
__device__ __forceinline__ void store32(const FfnProduct& p, const Rows4& rows, int col, const float* v) {
  uint4 w[4];
  if (!p.c_f32) {
    pack32(v, w);
    store_bf16x32(static_cast<__nv_bfloat16*>(p.C), rows, col, p.N, w);
    return;
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = make_uint4(__float_as_uint(v[16 * h + 4 * i]), __float_as_uint(v[16 * h + 4 * i + 1]),
                        __float_as_uint(v[16 * h + 4 * i + 2]), __float_as_uint(v[16 * h + 4 * i + 3]));
    transpose4(w);
    const int c = col + 16 * h + 4 * (threadIdx.x & 3);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (rows.off[i] >= 0 && c < p.N) *reinterpret_cast<uint4*>(static_cast<float*>(p.C) + rows.off[i] + c) = w[i];
  }
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
template <int EPI, int ACT, int NB>
__global__ void __launch_bounds__(Cfg<EPI, NB>::kThreads, 1)
    ffn_kernel(const __grid_constant__ Maps maps, const __grid_constant__ Params p) {
  using C = Cfg<EPI, NB>;
  constexpr int S = C::kStages, kEpiWarps = C::kWarps, kThreads = C::kThreads;
  constexpr uint32_t kStageBytes = C::kStageBytes;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* epi = smem + S * kStageBytes;
  uint64_t* bars = reinterpret_cast<uint64_t*>(epi + C::kEpiBytes);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * S + 4);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* last_flag = reinterpret_cast<volatile int*>(tmem_slot + 2);
  int* begin = reinterpret_cast<int*>(reinterpret_cast<uint8_t*>(bars) + 256);
  const uint32_t full0 = smem_u32(bars), empty0 = smem_u32(bars + S), tfull0 = smem_u32(bars + 2 * S),
                 tempty0 = smem_u32(bars + 2 * S + 2);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(full0 + 8 * s, 1);
      mbar_init(empty0 + 8 * s, 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(tfull0 + 8 * a, 1);
      mbar_init(tempty0 + 8 * a, 2 * 32 * kEpiWarps);
    }
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 0 && lane < (EPI == kGroup ? 2 * p.np : 2))
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&maps.m[lane])) : "memory");
  if (warp == 1) tmem_alloc_pair(smem_u32(tmem_slot), 2 * NB);
  fence_before();
  __syncthreads();
  cluster_sync();   // the peer's barriers exist before any copy or commit reaches them
  fence_after();
  const uint32_t tmem_base = *tmem_slot;
  // The kernel behind this one in the call may come as SMs fall free (all CTAs
  // of this one have started) and set itself up: the kept count is none of its
  // predecessors' in the call, the first of which was launched behind all before.
  if (EPI != kGroup) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int rank = static_cast<int>(cluster_ctarank());   // in the pair
  const int W = gridDim.x / 2, wid = blockIdx.x / 2;
  int n = p.M;
  if (p.n_kept) n = min(p.M, max(0, *p.n_kept));

  // ---------------- the tile list ----------------
  Sched sc;
  sc.W = W;
  sc.wid = wid;
  sc.begin = begin;
  if (EPI == kGroup) {
    sc.np = p.np;
    int total = 0;
    long long slices = 0;
    for (int i = 0; i < 3; ++i) {
      sc.first[i] = total;
      if (i >= p.np) { sc.units[i] = 1; sc.tiles[i] = sc.kb[i] = 0; continue; }
      const FfnProduct& q = p.p[i];
      const int m = q.dyn == 1 ? min(q.M, n) : q.M, k = q.dyn == 2 ? min(q.K, n) : q.K;
      sc.units[i] = (m + 2 * kBM - 1) / (2 * kBM);
      sc.tiles[i] = sc.units[i] * ((q.N + NB - 1) / NB);
      sc.kb[i] = (k + kBK - 1) / kBK;
      total += sc.tiles[i];
      slices += (long long)sc.tiles[i] * sc.kb[i];
      if (sc.units[i] == 0) sc.units[i] = 1;
    }
    sc.first[3] = total;
    for (int i = p.np; i < 3; ++i) sc.first[i] = total;
    sc.dp = total;
    // pair 0 has the most of every wave: its load if all tiles are whole, and
    // the whole waves that fit the even share
    const uint32_t magic = p.by_pairs;
    const int share = slices < (1ll << 30) ? (int)__umulhi((uint32_t)slices, magic) : 0;   // (within one of slices / W)
    int load0 = 0, waves = 0, fit = 0, left = 0;
    bool full = false;
    for (int i = 0; i < p.np; ++i) {
      const int c = count_mod(sc.first[i], sc.first[i] + sc.tiles[i], 0, magic);
      load0 += c * sc.kb[i];
      if (full || sc.kb[i] == 0) continue;
      const int take = min(c, max(0, (share - fit) / sc.kb[i]));
      fit += take * sc.kb[i];
      waves += take;
      left = sc.kb[i];
      full = take < c;
    }
    // (ranges shorter than a tile would cut tiles into more than two: a wave more for them)
    if (waves > 0 && share - fit < left) --waves;
    const int dp = min(total, waves * W);
    int off = 0, longest = 0;
    for (int i = 0; i < 3; ++i) {
      sc.tail_first[i] = max(sc.first[i], dp);
      sc.tail_off[i] = off;
      const int tail = i < p.np ? max(0, sc.first[i] + sc.tiles[i] - sc.tail_first[i]) : 0;
      if (total - dp <= kMaxTail) off += tail * sc.kb[i];
      if (tail) longest = max(longest, sc.kb[i]);
    }
    sc.tail_off[3] = off;
    // k-slices of a range (on average: the pairs with less work before take
    // more), and of a pair's whole work with what cutting costs
    int range = 0, best = load0;
    const int even = (int)__umulhi((uint32_t)off, magic) + 1;
    for (int parts = 2; parts <= kMaxParts + 1; ++parts) {
      const int r = max(even, (longest + parts - 2) / (parts - 1));
      const int all = share + r - even + kCutCost + kPartCost * (parts - 1);
      if (all < best) {
        best = all;
        range = r;
      }
    }
    if (p.partial && share > 0 && range > 0 && total - dp <= kMaxTail) {
      sc.dp = dp;
      if (warp == 2) {
        // a pair's range fills it up to its share; short tails go to fewer pairs
        int G = max(1, min(min(W, (off + range - 1) / range), kMaxParts * (total - dp)));
        // (few tiles of one length are cut into equal parts: no pair then has parts of two)
        if (dp == 0 && 2 * total <= G && off == total * sc.kb[0]) G -= G % total;
        int before = 0, at[kMaxWorkers / 32 + 1];
#pragma unroll
        for (int j = 0; j <= kMaxWorkers / 32; ++j) {
          const int w = lane + 32 * j;
          int load = 0;
          if (w < G)
            for (int i = 0; i < p.np; ++i) load += sc.kb[i] * count_mod(sc.first[i], min(dp, sc.first[i] + sc.tiles[i]), w, magic);
          const int room = w < G ? max(1, share + 1 - load) : 0;
          int x = room;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
          }
          at[j] = before + x - room;
          before += __shfl_sync(0xffffffffu, x, 31);
        }
        const float ratio = __fdividef((float)off, (float)before);   // (rounding moves a cut by a few k-slices at most)
#pragma unroll
        for (int j = 0; j <= kMaxWorkers / 32; ++j) {
          const int w = lane + 32 * j;
          if (w <= W) begin[w] = w >= G ? off : min(off, (int)((float)at[j] * ratio));
        }
      }
    }
    __syncthreads();
  } else {
    sc.np = 1;
    sc.units[0] = (n + 2 * kBM - 1) / (2 * kBM);
    constexpr int cols = EPI == kUp ? NB / 2 : NB;
    sc.tiles[0] = sc.units[0] * ((p.F + cols - 1) / cols);
    sc.kb[0] = p.kb;
    sc.first[0] = 0;
    for (int i = 1; i < 4; ++i) sc.first[i] = sc.tiles[0];
    sc.dp = sc.tiles[0];
    if (sc.units[0] == 0) sc.units[0] = 1;
  }
  // What the kernel ahead in the call writes is read by the producer and by
  // kGroup's epilogue alone, which wait for it (kDs: the kept rows of dy; kGroup:
  // its operands and counters).
  if (EPI != kGroup && p.zero && blockIdx.x == 0)
    for (int i = threadIdx.x; i < p.n_zero; i += kThreads) p.zero[i] = 0;

  if (EPI == kGroup && p.n_kept && n == 0) {
    // nothing kept: sums over the kept rows are 0
    grid_dep_wait();
    if (warp >= 2)
      for (int i = 0; i < p.np; ++i) {
        const FfnProduct& q = p.p[i];
        if (q.dyn != 2) continue;
        const long long bytes = (long long)q.M * q.ldc * (q.c_f32 ? 4 : 2);   // (a weight gradient's rows are contiguous)
        for (long long e = (blockIdx.x * (long long)(32 * kEpiWarps) + threadIdx.x - 64) * 16; e < bytes;
             e += (long long)gridDim.x * 32 * kEpiWarps * 16)
          *reinterpret_cast<uint4*>(static_cast<char*>(q.C) + e) = make_uint4(0, 0, 0, 0);
      }
  } else if (warp == 0) {
    // ---------------- TMA producer: the converged warp waits, one elected lane issues ----------------
    const bool leader = elect_one();
    auto wait = [&](uint32_t bar, uint32_t parity, unsigned site) {
      return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, p.st, site)) != 0;
    };
    auto aborted = [&]() { return __any_sync(0xffffffffu, *abort_flag != 0); };
    int stage = 0;
    uint32_t phase = 0, armed = 0, armed_parity = 0;   // stages with copies issued, and the phase parity armed
    Iter iter(sc);
    Tile t;
    bool more = iter.next(rank, &t);
    grid_dep_wait();
    for (; more && !aborted(); more = iter.next(rank, &t)) {
      const CUtensorMap* ma = &maps.m[EPI == kGroup ? 2 * t.p : 0];
      const CUtensorMap* mb = ma + 1;
      const bool a_mn = EPI == kGroup ? p.p[t.p].a_mn != 0 : false, b_mn = EPI == kGroup ? p.p[t.p].b_mn != 0 : EPI == kUp;
      // this CTA's half of the tile's columns: of kUp, all of g or of u
      const int nb = EPI == kUp ? t.n0 * (NB / 2) + rank * p.F : t.n0 * NB + rank * (NB / 2);
      bool ok = true;
      for (int kb = t.k0; kb < t.k1; ++kb) {
        if (!wait(empty0 + 8 * stage, phase ^ 1u, 1)) { ok = false; break; }
        const uint32_t fb = full0 + 8 * stage;
        armed |= 1u << stage;
        armed_parity = (armed_parity & ~(1u << stage)) | (phase << stage);
        if (leader) {
          const uint32_t sa = smem_u32(smem + stage * kStageBytes), sb = sa + kABytes;
          const int kx = kb * kBK;
          if (rank == 0) mbar_expect_tx(fb, 2 * kStageBytes);   // both CTAs' copies are counted on the even CTA's barrier
          const uint32_t lb = map_to_rank(fb, 0);
          if (!a_mn) {
            tma_load_2d_pair(sa, ma, lb, kx, t.m0);
          } else {
            tma_load_2d_pair(sa, ma, lb, t.m0, kx);
            tma_load_2d_pair(sa + 8192, ma, lb, t.m0 + 64, kx);
          }
          if (!b_mn) {
            tma_load_2d_pair(sb, mb, lb, kx, nb);
          } else {
            tma_load_2d_pair(sb, mb, lb, nb, kx);
            if (NB == 256) tma_load_2d_pair(sb + 8192, mb, lb, nb + 64, kx);
          }
        }
        __syncwarp();
        if (++stage == S) { stage = 0; phase ^= 1u; }
      }
      if (!ok) break;
    }
    if (!aborted()) {
      // the MMAs release every stage (their commits land in this CTA's empty
      // barriers) before this CTA may leave the cluster
      for (int i = 0; i < S; ++i) {
        if (!wait(empty0 + 8 * stage, phase ^ 1u, 5)) break;
        if (++stage == S) { stage = 0; phase ^= 1u; }
      }
    }
    if (aborted() && leader) {
      // another role gave up: let this thread's copies still in flight land
      // (bounded, 10 ms per stage) before the CTA releases its shared memory
      for (int s = 0; s < S; ++s) {
        if (!((armed >> s) & 1u)) continue;
        const uint64_t t0 = globaltimer_ns();
        while (!mbar_try(full0 + 8 * s, (armed_parity >> s) & 1u) && globaltimer_ns() - t0 < 10000000ull) {
        }
      }
    }
  } else if (warp == 1) {
    if (rank == 0) {
      // ---------------- MMA issuer (the even CTA) ----------------
      const bool leader = elect_one();
      auto wait = [&](uint32_t bar, uint32_t parity, unsigned site) {
        return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, p.st, site)) != 0;
      };
      int stage = 0;
      uint32_t phase = 0;
      int seg = 0;
      Iter iter(sc);
      Tile t;
      while (iter.next(rank, &t) && !__any_sync(0xffffffffu, *abort_flag != 0)) {
        const bool a_mn = EPI == kGroup ? p.p[t.p].a_mn != 0 : false, b_mn = EPI == kGroup ? p.p[t.p].b_mn != 0 : EPI == kUp;
        const uint32_t idesc = idesc_bf16(2 * kBM, NB, a_mn, b_mn);
        const uint32_t a_step = a_mn ? 2048 : 32, b_step = b_mn ? 2048 : 32, a_lbo = a_mn ? 8192 : 16, b_lbo = b_mn ? 8192 : 16;
        const int acc = seg & 1;
        if (!wait(tempty0 + 8 * acc, ((seg >> 1) & 1) ^ 1u, 2)) break;
        fence_after();
        const uint32_t d = tmem_base + acc * NB;
        bool ok = true;
        for (int kb = t.k0; kb < t.k1; ++kb) {
          if (!wait(full0 + 8 * stage, phase, 3)) { ok = false; break; }
          fence_after();
          if (leader) {
            const uint32_t sa = smem_u32(smem + stage * kStageBytes), sb = sa + kABytes;
#pragma unroll
            for (int kk = 0; kk < kBK / 16; ++kk)
              mma_bf16_pair(d, sdesc(sa + kk * a_step, a_lbo, 1024), sdesc(sb + kk * b_step, b_lbo, 1024), idesc,
                            (kb > t.k0) || (kk > 0));
            mma_commit_pair_mc(empty0 + 8 * stage, 3);
          }
          __syncwarp();
          if (++stage == S) { stage = 0; phase ^= 1u; }
        }
        if (!ok) break;
        if (leader) mma_commit_pair_mc(tfull0 + 8 * acc, 3);
        __syncwarp();
        ++seg;
      }
    }
  } else {
    // ---------------- epilogue (warps 2...) ----------------
    auto release_acc = [&](int acc) { mbar_arrive_cluster_relaxed(map_to_rank(tempty0 + 8 * acc, 0)); };
    volatile int no_abort = 0;   // (timeout-only waits: the threads leave together)
    const int q = warp & 3;      // TMEM lane quadrant this warp may access
    const int half = (warp - 2) >> 2;   // its share of the columns: of kUp a quarter of NB of g and of u, of kDs a quarter, else half
    const int rl = q * 32 + lane;
    int seg = 0;
    Iter iter(sc);
    Tile t;
    if constexpr (EPI == kUp) {
      while (iter.next(rank, &t)) {
        const int acc = seg & 1;
        const int row = t.m0 + rl;
        const Rows4 up_rows(row < n ? row * p.up_ld : -1), s_rows(row < n ? (long long)row * p.F : -1);
        if (!mbar_wait(tfull0 + 8 * acc, (seg >> 1) & 1, &no_abort, p.st, 4)) break;
        fence_after();
        const uint32_t tc0 = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + acc * NB + half * (NB / 4);
#pragma unroll
        for (int c = 0; c < NB / 4; c += 32) {
          float g[32], u[32];
          tmem_ld32(tc0 + c, g);
          tmem_ld32(tc0 + NB / 2 + c, u);
          if (c == NB / 4 - 32) {
            fence_before();
            release_acc(acc);
          }
          const int col = t.n0 * (NB / 2) + half * (NB / 4) + c;
          uint4 w[4];
          if (p.up) {
            pack32(g, w);
            store_bf16x32(p.up, up_rows, col, p.F, w);
            pack32(u, w);
            store_bf16x32(p.up + p.F, up_rows, col, p.F, w);
          }
#pragma unroll
          for (int i = 0; i < 32; ++i) g[i] = glu_act<ACT>(g[i]) * u[i];
          pack32(g, w);
          store_bf16x32(p.s, s_rows, col, p.F, w);
        }
        ++seg;
      }
    } else if constexpr (EPI == kDs) {
      // A chunk is 32 rows x 16 columns of this warp.  Its g and u are copied to
      // shared memory (16-byte pieces, the two of a 32-byte row swapped in every
      // other four rows, so that the lanes' reads of their own rows meet no bank
      // twice) as soon as those of the chunk before are read; a tile's first
      // before its products are done.  (A second chunk's room costs a stage of
      // the ring: 430 us instead of 425 for the backward above.)
      const uint32_t room = smem_u32(epi) + (warp - 2) * 2 * kChunkBytes;
      const uint32_t sw = ((lane >> 2) & 1) * 16;             // of this thread's row
      const int prow = lane >> 1, piece = lane & 1;           // the copies' rows: prow + 16 i
      // The copies run ahead by an iterator of their own: tile, chunk in it, and
      // the rows of `up` of the tile (row prow + 16 i of the warp's 32).
      constexpr int kNoRow = INT32_MIN, kChunks = NB / 4 / kDsCols;   // (chunks of a warp's share of a tile)
      Iter ahead(sc);
      Tile ct;
      bool copying;
      int chunk = 0;
      int src[2];
      auto next_rows = [&] {
        copying = ahead.next(rank, &ct);
        chunk = 0;
        if (!copying) return;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int r = ct.m0 + q * 32 + prow + 16 * i;
          src[i] = r < n ? p.idx ? p.idx[r] : r : kNoRow;
        }
      };
      auto copy = [&] {
        if (copying) {
          const int col = ct.n0 * NB + half * (NB / 4) + chunk * kDsCols + piece * 8;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int r = prow + 16 * i;
            const bool there = (unsigned)src[i] < (unsigned)p.M && col < p.F;
            if (chunk == 0 && !there && src[i] != kNoRow && col < p.F) report_error(p.st, kErrBadIndex, 702);
            const __nv_bfloat16* g = p.up + (there ? src[i] * p.up_ld + col : 0);
            const uint32_t at = room + r * 32 + ((piece ^ ((r >> 2) & 1)) * 16);
            cp_async16(at, g, there);
            cp_async16(at + kChunkBytes, g + (there ? p.F : 0), there);
          }
          if (++chunk == kChunks) next_rows();
        }
      };
      next_rows();
      copy();
      while (iter.next(rank, &t)) {
        const int acc = seg & 1;
        const int row = t.m0 + rl;
        // where this lane's stores go: piece (lane & 1) of rows (lane & ~1) + i
        long long out[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int r = t.m0 + q * 32 + (lane & 30) + i;
          out[i] = r < p.cap ? (long long)r * p.F : -1;
        }
        if (!mbar_wait(tfull0 + 8 * acc, (seg >> 1) & 1, &no_abort, p.st, 4)) break;
        fence_after();
        const uint32_t tc0 = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + acc * NB + half * (NB / 4);
#pragma unroll 1
        for (int c = 0; c < kChunks; ++c) {
          uint32_t d[kDsCols];
          tmem_ld16_async(tc0 + c * kDsCols, d);
          cp_async_wait_all();
          __syncwarp();
          const uint32_t buf = room + lane * 32;
          uint4 g4[2], u4[2], s4[2];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            g4[j] = lds128(buf + ((j * 16) ^ sw));
            u4[j] = lds128(buf + kChunkBytes + ((j * 16) ^ sw));
          }
          __syncwarp();     // the room is read: the next chunk may come
          copy();
          tmem_wait_ld();
          if (c == kChunks - 1) {
            fence_before();
            release_acc(acc);
          }
          if (row >= n) {   // (the rows behind the kept ones that are written are 0)
#pragma unroll
            for (int i = 0; i < kDsCols; ++i) d[i] = 0;
          }
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float g[8], u[8], s[8];
            unpack8(g4[j], g);
            unpack8(u4[j], u);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float ds = __uint_as_float(d[8 * j + i]);
              float a, da;
              glu_both<ACT>(g[i], &a, &da);
              s[i] = a * u[i];
              g[i] = ds * (u[i] * da);   // (|a'| < 1.2: ds u alone could be an infinity beside a slope of 0)
              u[i] = ds * a;
            }
            g4[j] = pack8(g);
            u4[j] = pack8(u);
            s4[j] = pack8(s);
          }
          transpose2(g4);
          transpose2(u4);
          transpose2(s4);
          const int col = t.n0 * NB + half * (NB / 4) + c * kDsCols + 8 * (lane & 1);
          if (col < p.F) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              if (out[i] < 0) continue;
              *reinterpret_cast<uint4*>(p.dgu + 2 * out[i] + col) = g4[i];
              *reinterpret_cast<uint4*>(p.dgu + 2 * out[i] + p.F + col) = u4[i];
              *reinterpret_cast<uint4*>(p.s + out[i] + col) = s4[i];
            }
          }
        }
        ++seg;
      }
      cp_async_wait_all();
    } else {
      constexpr int kHalf = NB / 2;   // columns of a warp
      grid_dep_wait();
      while (iter.next(rank, &t)) {
        const FfnProduct& pr = p.p[t.p];
        const int acc = seg & 1;
        const int M = pr.dyn == 1 ? min(pr.M, n) : pr.M;
        const int row = t.m0 + rl;
        bool row_ok = row < M;
        long long out_row = row;
        if (pr.scatter && row_ok) {
          const int o = p.idx[row];
          row_ok = o >= 0 && o < pr.c_rows;
          out_row = o;
          if (!row_ok) report_error(p.st, kErrBadIndex, 703);
        }
        // rows behind the kept ones that a COMPACT output holds zeros in
        const bool row_zero = !row_ok && pr.zero_pad && row < padded_rows(M, pr.c_rows);
        if (!mbar_wait(tfull0 + 8 * acc, (seg >> 1) & 1, &no_abort, p.st, 4)) break;
        fence_after();
        const Rows4 rows(row_ok || row_zero ? out_row * pr.ldc : -1);
        // a tile that is cut: its k-slices' places in the tail, the pairs that share it
        int x0 = 0, x1 = 0, c_first = 0, c_last = 0;
        int* ctr = nullptr;
        if (!t.whole) {
          auto owner = [&](int x) {
            int lo = 0, hi = W - 1;   // the last pair whose range begins at or before x (and is not empty)
            while (lo < hi) {
              const int mid = (lo + hi + 1) >> 1;
              if (begin[mid] <= x) lo = mid; else hi = mid - 1;
            }
            return lo;
          };
          x0 = sc.tail_off[t.p] + (t.t - sc.tail_first[t.p]) * sc.kb[t.p];
          x1 = x0 + sc.kb[t.p];
          c_first = owner(x0);
          c_last = owner(x1 - 1);
          // Low half: pairs that came, high half: parts parked.  The pair that
          // comes last finishes the tile.  Whoever came has no other tile to
          // wait for, so the last may wait for the others' parts, whichever
          // kernels hold the other SMs.
          ctr = p.counters + (t.t - sc.dp) * 2 + rank;
          if (threadIdx.x == 64) {
            int parts = 0;
            for (int w = c_first; w <= c_last; ++w) parts += begin[w] < begin[w + 1];
            const int old = atomicAdd(ctr, 1);
            last_flag[0] = (old & 0xffff) == parts - 1 ? parts : 0;
          }
        }
        const uint32_t tc0 = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + acc * NB + half * kHalf;
        const int col0 = t.n0 * NB + half * kHalf;
        if (t.whole) {
#pragma unroll 1
          for (int c = 0; c < kHalf; c += 32) {
            float v[32];
            tmem_ld32(tc0 + c, v);
            if (c == kHalf - 32) {
              fence_before();
              release_acc(acc);
            }
            if (row_zero) {
#pragma unroll
              for (int i = 0; i < 32; ++i) v[i] = 0.f;
            }
            store32(pr, rows, col0 + c, v);
          }
        } else {
          // A pair parks at most two parts: in place 0 of the tile its range
          // begins in, in place 1 of the tile it ends in.
          auto slot_of = [&](int w) {
            const int at = 2 * w + (begin[w] >= x0 && begin[w] < x1 ? 0 : 1);
            return p.partial + ((long long)at * 2 + rank) * (kBM * NB);
          };
          named_bar(1, 32 * kEpiWarps);
          const int parts = *last_flag;
          const bool live = row_ok || row_zero;   // (rows behind the last are not parked)
          if (!parts) {
            float* own = slot_of(wid);
#pragma unroll 1
            for (int c = 0; c < kHalf; c += 32) {
              float v[32];
              tmem_ld32(tc0 + c, v);
              if (!live) continue;
#pragma unroll
              for (int i = 0; i < 32; i += 4)
                __stcg(reinterpret_cast<float4*>(own + ((long long)((half * kHalf + c + i) >> 2) * kBM + rl) * 4),
                       make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]));
            }
            fence_before();
            release_acc(acc);
            __threadfence();
            named_bar(1, 32 * kEpiWarps);
            if (threadIdx.x == 64) atomicAdd(ctr, 0x10000);
          } else {
            if (threadIdx.x == 64) {
              wait_turn(ctr, ((parts - 1) << 16) + parts, p.st, 6);   // (all have come: the low half stands)
              *ctr = 0;
            }
            named_bar(1, 32 * kEpiWarps);
            __threadfence();
            // One other part (the most usual): its next 32 columns are on their
            // way while these are added.
            const int other = parts == 2 ? (c_first == wid ? c_last : c_first) : -1;
            auto load_part = [&](int w, int c, float* x) {
              if (live) {
                const float* from = slot_of(w) + ((long long)((half * kHalf + c) >> 2) * kBM + rl) * 4;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                  const float4 y = __ldcg(reinterpret_cast<const float4*>(from + i * kBM * 4));
                  x[4 * i] = y.x; x[4 * i + 1] = y.y; x[4 * i + 2] = y.z; x[4 * i + 3] = y.w;
                }
              } else {
#pragma unroll
                for (int i = 0; i < 32; ++i) x[i] = 0.f;
              }
            };
            float next[32];
            if (other >= 0) load_part(other, 0, next);
#pragma unroll 1
            for (int c = 0; c < kHalf; c += 32) {
              float v[32];
              if (other >= 0) {
                float x[32];
                tmem_ld32(tc0 + c, v);
#pragma unroll
                for (int i = 0; i < 32; ++i) x[i] = next[i];
                if (c < kHalf - 32) load_part(other, c + 32, next);
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] += x[i];   // (of two, either order is the same)
              } else {
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] = 0.f;
#pragma unroll 1
                for (int w = c_first; w <= c_last; ++w) {   // in the order of the pairs, this one's part from its accumulator
                  if (begin[w] == begin[w + 1]) continue;
                  float x[32];
                  if (w == wid) tmem_ld32(tc0 + c, x);
                  else load_part(w, c, x);
#pragma unroll
                  for (int i = 0; i < 32; ++i) v[i] += x[i];
                }
              }
              if (row_zero) {
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] = 0.f;
              }
              store32(pr, rows, col0 + c, v);
            }
            fence_before();
            release_acc(acc);
          }
          named_bar(1, 32 * kEpiWarps);   // last_flag is reused by the next piece
        }
        ++seg;
      }
    }
  }
  fence_before();
  __syncthreads();
  cluster_sync();
  if (warp == 1) {
    fence_after();
    tmem_dealloc_pair(tmem_base, 2 * NB);
  }
}

// ---------------------------------------------------------------------------
// host side
template <int EPI, int ACT, int NB>
cudaError_t launch(const Ctx& c, const char* name, const Maps& maps, Params p, long long tiles, long long m, long long n,
                   long long k, int dyn) {
  auto kern = ffn_kernel<EPI, ACT, NB>;
  constexpr size_t smem = Cfg<EPI, NB>::kSmem;
  // per device, once: the shared-memory opt-in, and how many pairs run at once
  static std::mutex mu;
  static int known[64] = {0};
  int dev = 0, fit = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  {
    std::lock_guard<std::mutex> lk(mu);
    if (dev >= 0 && dev < 64) fit = known[dev];
    if (fit == 0) {
      e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
      if (e != cudaSuccess) return e;
      cudaLaunchConfig_t cfg = {};
      cudaLaunchAttribute attr[1];
      attr[0].id = cudaLaunchAttributeClusterDimension;
      attr[0].val.clusterDim.x = 2;
      attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
      cfg.gridDim = dim3(c.num_sms / 2 * 2);
      cfg.blockDim = dim3(Cfg<EPI, NB>::kThreads);
      cfg.dynamicSmemBytes = smem;
      cfg.attrs = attr;
      cfg.numAttrs = 1;
      e = cudaOccupancyMaxActiveClusters(&fit, kern, &cfg);
      if (e != cudaSuccess) return e;
      fit = std::min({fit, c.num_sms / 2, kMaxWorkers});
      if (fit < 1) return cudaErrorNotSupported;
      if (dev >= 0 && dev < 64) known[dev] = fit;
    }
  }
  // (a group's tail may go to every pair)
  const int workers = EPI == kGroup ? fit : (int)std::max(1ll, std::min<long long>(tiles, fit));
  p.by_pairs = (uint32_t)(((1ull << 32) + workers - 1) / workers);
  if (workers < 2) p.partial = nullptr;   // (nobody to share with; 2^32 / 1 does not fit)
  prof_begin(c, name, m, n, k, dyn);
  e = launch_k(c, pdl_allowed() && c.pdl, kern, dim3(2 * workers), dim3(Cfg<EPI, NB>::kThreads), smem, 2, maps, p);
  prof_end(c);
  count_launch();
  return launched(e);
}

bool k_major(CUtensorMap* m, const void* p, long long inner, long long rows, long long ld, int box_rows) {
  return make_tensor_map(m, p, false, inner, rows, ld, 64, box_rows);
}
bool mn_major(CUtensorMap* m, const void* p, long long inner, long long rows, long long ld) {
  return make_tensor_map(m, p, false, inner, rows, ld, 64, 64);
}

}  // namespace

// The form of a list of so many 256 x 256 tiles: at most a quarter of a wave of
// SMs takes tiles of 128 columns, so that twice the SMs share the epilogues.
enum class Form { kNarrow, kPair };
static Form form_of(const Ctx& c, long long tiles) { return 4 * tiles <= c.num_sms ? Form::kNarrow : Form::kPair; }
static int cols_box(Form f) { return f == Form::kNarrow ? 64 : 128; }   // of the columns' operand, K-major
template <int EPI, int ACT, typename... A>
static cudaError_t launch_form(Form f, A... args) {
  return f == Form::kNarrow ? launch<EPI, ACT, 128>(args...) : launch<EPI, ACT, 256>(args...);
}
static long long tiles_of(Form f, long long m, long long n) {
  const int nb = f == Form::kNarrow ? 128 : 256;
  return (m + 2 * kBM - 1) / (2 * kBM) * ((n + nb - 1) / nb);
}

size_t ffn_partial_floats(long long tiles) {
  // two parts a pair, of 128 rows in each of its CTAs; at most about kMaxParts pairs work at a tile
  // (of 128-column tiles there are twice as many at most, of half the size)
  return (size_t)(2 * std::min<long long>(kMaxWorkers, kMaxParts * tiles) * 2) * kBM * 256;
}
long long ffn_tiles(long long m, long long n) { return tiles_of(Form::kPair, m, n); }
int ffn_counters() { return 2 * kMaxTail; }

cudaError_t launch_ffn_up(const Ctx& c, const FfnUp& a) {
  Maps maps{};
  const Form f = form_of(c, ffn_tiles(a.M, 2ll * a.F));
  if (!k_major(&maps.m[0], a.x, a.D, a.M, a.x_ld, kBM) || !mn_major(&maps.m[1], a.w_up, 2ll * a.F, a.D, 2ll * a.F))
    return cudaErrorInvalidValue;
  Params p{};
  p.M = a.M; p.F = a.F; p.kb = (a.D + kBK - 1) / kBK;
  p.up = a.up; p.up_ld = a.up_ld; p.s = a.s;
  p.zero = a.counters; p.n_zero = ffn_counters();
  p.st = c.st;
  const long long tiles = tiles_of(f, a.M, 2ll * a.F);
  return a.act == kGluSilu ? launch_form<kUp, kGluSilu>(f, c, "ffn_up", maps, p, tiles, a.M, 2ll * a.F, a.D, 0)
                           : launch_form<kUp, kGluGeluTanh>(f, c, "ffn_up", maps, p, tiles, a.M, 2ll * a.F, a.D, 0);
}

cudaError_t launch_ffn_ds(const Ctx& c, const FfnDs& a) {
  Maps maps{};
  const Form f = form_of(c, ffn_tiles(a.M, a.F));
  if (!k_major(&maps.m[0], a.dy, a.D, a.dy_rows, a.dy_ld, kBM) ||
      !k_major(&maps.m[1], a.w_down, a.D, a.F, a.D, cols_box(f)))
    return cudaErrorInvalidValue;
  Params p{};
  p.M = a.M; p.F = a.F; p.kb = (a.D + kBK - 1) / kBK;
  p.n_kept = a.n_kept; p.idx = a.up_full ? a.idx : nullptr;
  p.up = const_cast<__nv_bfloat16*>(a.up); p.up_ld = a.up_ld;
  p.dgu = a.dgu; p.s = a.s; p.cap = a.cap;
  p.zero = a.counters; p.n_zero = ffn_counters();
  p.st = c.st;
  const long long tiles = tiles_of(f, a.M, a.F);
  const int dyn = a.n_kept ? 1 : 0;
  return a.act == kGluSilu ? launch_form<kDs, kGluSilu>(f, c, "ffn_ds", maps, p, tiles, a.M, a.F, a.D, dyn)
                           : launch_form<kDs, kGluGeluTanh>(f, c, "ffn_ds", maps, p, tiles, a.M, a.F, a.D, dyn);
}

cudaError_t launch_ffn_group(const Ctx& c, const FfnProduct* q, int np, int M, const int32_t* idx, const int32_t* n_kept,
                             float* partial, int* counters) {
  Maps maps{};
  Params p{};
  long long tiles = 0;
  for (int i = 0; i < np; ++i) tiles += ffn_tiles(q[i].M, q[i].N);
  const Form f = form_of(c, tiles);
  for (int i = 0; i < np; ++i) {
    const bool a_ok = q[i].a_mn ? mn_major(&maps.m[2 * i], q[i].A, q[i].M, q[i].a_rows, q[i].lda)
                                : k_major(&maps.m[2 * i], q[i].A, q[i].K, q[i].a_rows, q[i].lda, kBM);
    const bool b_ok = q[i].b_mn ? mn_major(&maps.m[2 * i + 1], q[i].B, q[i].N, q[i].b_rows, q[i].ldb)
                                : k_major(&maps.m[2 * i + 1], q[i].B, q[i].K, q[i].b_rows, q[i].ldb, cols_box(f));
    if (!a_ok || !b_ok) return cudaErrorInvalidValue;
    p.p[i] = q[i];
  }
  p.np = np;
  p.M = M; p.idx = idx; p.n_kept = n_kept;
  p.partial = partial; p.counters = counters;
  p.st = c.st;
  return launch_form<kGroup, 0>(f, c, "ffn_group", maps, p, tiles, q[0].M, q[0].N, q[0].K, q[0].dyn);
}

}  // namespace collider
