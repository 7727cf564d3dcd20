// Norm of a list of gradients, and clipping: what a training step does with
// the block's and the stack's gradients before it applies them (the pages have
// no counterpart).
//   norm = scale (sum g^2)^(1/2), or scale max |g|;
//   g <- coef g, coef = scale min(1, max_norm / (norm + 1e-6)).
// HBM-bound: the norm reads every value once; clipping needs the whole norm
// before it writes the first value, so it reads a second time.
//   Measured: the norm of 1.1 G f32 values (135 tensors, 4.4 GB) 615 us, 7.2 TB/s;
// of 44 M 35 us (29 of them reading at 6 TB/s); of 492 K 8.2 us.  (A set of up to
// 4 MB in one launch, as a cluster of 16 CTAs with the partials in its shared
// memory: 8.7 us, and 12 instead of 8 for clipping 2 MB: too few SMs read.)
// Clipping them 1988 us (three passes at 6.6 TB/s) and 75 us, 89 from memory.
#include <algorithm>

#include "internal.h"

namespace collider {

namespace {

constexpr int kGradThreads = 256;
constexpr int kGradVecs = 8;             // 16-byte vectors a thread has in flight
constexpr int kGradChunk = kGradThreads * kGradVecs;   // vectors of a chunk: 32 KB
constexpr int kGradTable = 1024;         // tensors of a launch (20 KB of its 32 KB of parameters)
constexpr int kShortTable = 32;          // tensors of a short list
constexpr int kGradBlocksPerSm = 4;
constexpr size_t kGradKeep = 96 << 20;   // bytes that the norm leaves in L2 for the clipping pass (176 MB: 88 us, with none left 93)

// A launch's tensors, by value in its parameters: no copy to the device, so a
// captured call replays with the addresses it was captured with.
template <int N>
struct GradTable {
  int count;
  int chunks;            // chunks of all tensors
  long long n[N];        // values; bit 62: bf16
  const void* p[N];
  int first[N + 1];      // first chunk of each tensor
};
constexpr long long kGradBf16 = 1ll << 62;

// Tensors' chunks are numbered in list order; block b takes chunks
// [begin(b), begin(b+1)).  It leaves a partial sum for each tensor it meets at
// slot b + tensor: as b or the tensor goes up by one at every step, no two
// pairs share a slot, and every slot below blocks + count is written by
// exactly one block (with 0 where it stands for nothing).
template <typename Tab>
__device__ __forceinline__ int block_begin(const Tab& t, int b, int blocks) {
  return (int)((long long)b * t.chunks / blocks);
}
template <typename Tab>
__device__ __forceinline__ int tensor_of(const Tab& t, int chunk) {   // last tensor whose first chunk is <= chunk, with chunks
  int lo = 0, hi = t.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (t.first[mid] <= chunk) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// a tensor as 16-byte vectors of whole 16-byte places in memory: value i is
// value i + lead of the vectors; those before `lead` and behind `end` are not its
struct Span {
  const uint4* base;
  int lead;            // values before the first in its vector
  long long end;       // lead + n
  int per;             // values of a vector
};
__device__ __forceinline__ Span span_of(const void* p, long long n_flag) {
  const bool bf = (n_flag & kGradBf16) != 0;
  const long long n = n_flag & ~kGradBf16;
  const uintptr_t a = reinterpret_cast<uintptr_t>(p);
  Span s;
  s.base = reinterpret_cast<const uint4*>(a & ~uintptr_t(15));
  s.lead = (int)(a & 15) / (bf ? 2 : 4);
  s.end = s.lead + n;
  s.per = bf ? 8 : 4;
  return s;
}

template <bool BF>
__device__ __forceinline__ void unpack_vec(const uint4& u, float* f) {
  if (BF) {
    unpack8(u, f);
  } else {
    f[0] = __uint_as_float(u.x); f[1] = __uint_as_float(u.y);
    f[2] = __uint_as_float(u.z); f[3] = __uint_as_float(u.w);
  }
}
// vector v of a span whose first or last values are not all its own: those are 0
template <bool BF>
__device__ __forceinline__ uint4 load_edge(const Span& s, long long v) {
  uint32_t w[4] = {0, 0, 0, 0};
  if (BF) {
    const uint16_t* p = reinterpret_cast<const uint16_t*>(s.base + v);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const long long at = v * 8 + i;
      if (at >= s.lead && at < s.end) w[i >> 1] |= (uint32_t)p[i] << (16 * (i & 1));
    }
  } else {
    const uint32_t* p = reinterpret_cast<const uint32_t*>(s.base + v);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const long long at = v * 4 + i;
      if (at >= s.lead && at < s.end) w[i] = p[i];
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
template <bool BF>
__device__ __forceinline__ bool whole_vec(const Span& s, long long v) {
  constexpr int per = BF ? 8 : 4;
  return v * per >= s.lead && (v + 1) * per <= s.end;
}

// The vectors of a chunk that this thread takes: v0 + thread + k * kGradThreads.
// keep: what is loaded is read again soon (clipping).  Inside a tensor they are
// loaded without a question, all at once; only a tensor's first and last chunk
// ask for each vector.
template <bool BF>
__device__ __forceinline__ bool inner_chunk(const Span& s, long long v0) {
  constexpr int per = BF ? 8 : 4;
  return v0 * per >= s.lead && (v0 + kGradChunk) * per <= s.end;
}
template <bool BF>
__device__ __forceinline__ void load_chunk(const Span& s, long long v0, bool keep, uint4* u) {
  constexpr int per = BF ? 8 : 4;
  if (inner_chunk<BF>(s, v0)) {
    const uint4* p = s.base + v0 + threadIdx.x;
    if (keep) {
#pragma unroll
      for (int k = 0; k < kGradVecs; ++k) u[k] = p[k * kGradThreads];
    } else {
#pragma unroll
      for (int k = 0; k < kGradVecs; ++k) u[k] = __ldcs(p + k * kGradThreads);
    }
  } else {
    const long long vend = (s.end + per - 1) / per;
#pragma unroll
    for (int k = 0; k < kGradVecs; ++k) {
      const long long v = v0 + threadIdx.x + k * kGradThreads;
      u[k] = make_uint4(0, 0, 0, 0);
      if (v < vend) u[k] = whole_vec<BF>(s, v) ? s.base[v] : load_edge<BF>(s, v);
    }
  }
}

// Adds a thread's values of one chunk to its sum of squares (in f64), or takes
// its largest magnitude (as the bits of |v|: a NaN is above infinity).
// Squares are added in f32, at most 16 to a sum, and the sums in f64: one f64
// operation a chunk and thread (an f64 multiply-add a value would bind, at
// 1/64 of the f32 rate).  Where the largest magnitude leaves [2^-50, 2^60],
// and squares of f32 could overflow or vanish, the same values are squared in
// f64.
template <bool BF, bool MAX>
__device__ __forceinline__ void take_chunk(const uint4* u, double* sum, uint32_t* big) {
  constexpr int per = BF ? 8 : 4;
  uint32_t m = 0;
  float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int k = 0; k < kGradVecs; ++k) {
    float f[8];
    unpack_vec<BF>(u[k], f);
#pragma unroll
    for (int i = 0; i < per; ++i) {
      if (!MAX) acc[i & 3] = fmaf(f[i], f[i], acc[i & 3]);
      m = max(m, __float_as_uint(f[i]) & 0x7fffffffu);
    }
  }
  if (MAX) {
    *big = max(*big, m);
    return;
  }
  if (m != 0 && (m > __float_as_uint(1.152921504606847e18f) || m < __float_as_uint(8.881784197001252e-16f))) {
#pragma unroll
    for (int k = 0; k < kGradVecs; ++k) {
      float f[8];
      unpack_vec<BF>(u[k], f);
#pragma unroll
      for (int i = 0; i < per; ++i) *sum = fma((double)f[i], (double)f[i], *sum);
    }
  } else {
    *sum += (double)((acc[0] + acc[1]) + (acc[2] + acc[3]));
  }
}
template <bool BF, bool MAX>
__device__ __forceinline__ void take_chunks(const Span& s, int c, int cend, int keep_from, double* sum, uint32_t* big) {
  for (; c < cend; ++c) {
    uint4 u[kGradVecs];
    load_chunk<BF>(s, (long long)c * kGradChunk, c >= keep_from, u);
    take_chunk<BF, MAX>(u, sum, big);
  }
}

__device__ __forceinline__ double max_value(uint32_t bits) { return (double)__uint_as_float(bits); }
// the larger of two magnitudes, a NaN above all
__device__ __forceinline__ double max_nan(double a, double b) { return (a > b || a != a) ? a : b; }

// Sum (or maximum) over the block, in a fixed order; every thread gets it.
// One warp adds all of it: f64 runs at two operations a clock and SM, so eight
// warps that each reduced their own and then each other's values would take
// eight times as long (3 us an SM with four blocks).
__device__ __forceinline__ double block_reduce(double v, int max_kind, double* red) {
  __syncthreads();
  red[threadIdx.x] = v;
  __syncthreads();
  if (threadIdx.x < 32) {
#pragma unroll
    for (int i = 1; i < kGradThreads / 32; ++i) {
      const double w = red[threadIdx.x + 32 * i];
      v = max_kind ? max_nan(v, w) : v + w;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const double w = __shfl_xor_sync(0xffffffffu, v, o);
      v = max_kind ? max_nan(v, w) : v + w;
    }
    if (threadIdx.x == 0) red[0] = v;
  }
  __syncthreads();
  return red[0];
}

// block b's partials; the last `keep` of its chunks are left in L2
template <typename Tab>
__device__ __forceinline__ void part_block(const Tab& t, int b, int blocks, int keep, int max_kind, double* part, double* red) {
  int c = block_begin(t, b, blocks);
  const int cend = block_begin(t, b + 1, blocks);
  const int t_first = b == 0 ? 0 : tensor_of(t, c);
  const int t_last = b + 1 == blocks ? t.count : tensor_of(t, cend);   // slots b + t_first .. b + t_last are this block's
  for (int k = t_first; k <= t_last; ++k) {
    double v = 0.0;
    const int kend = k < t.count ? min(t.first[k + 1], cend) : c;
    if (c < kend) {
      const Span s = span_of(t.p[k], t.n[k]);
      double sum = 0.0;
      uint32_t big = 0;
      const int at = t.first[k], kf = cend - keep - at;
      if (s.per == 8) {
        if (max_kind) take_chunks<true, true>(s, c - at, kend - at, kf, &sum, &big);
        else take_chunks<true, false>(s, c - at, kend - at, kf, &sum, &big);
      } else {
        if (max_kind) take_chunks<false, true>(s, c - at, kend - at, kf, &sum, &big);
        else take_chunks<false, false>(s, c - at, kend - at, kf, &sum, &big);
      }
      c = kend;
      v = block_reduce(max_kind ? max_value(big) : sum, max_kind, red);
    }
    if (threadIdx.x == 0) part[b + k] = v;
  }
}

template <int N>
__global__ void __launch_bounds__(kGradThreads, kGradBlocksPerSm)
    grad_part_kernel(const __grid_constant__ GradTable<N> t, int keep, int max_kind, double* part) {
  __shared__ double red[kGradThreads];
  grid_dep_wait();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // (this call's second kernel sets itself up beside the last blocks)
  part_block(t, blockIdx.x, gridDim.x, keep, max_kind, part, red);
}

// a partial that another kernel left (no copy of L1's)
__device__ __forceinline__ double load_part(const double* p) { return *static_cast<const volatile double*>(p); }

// The root of a sum.  sqrt of an f64 costs about 1 us here; where the sum is
// well inside f32, its root r there (off by 2^-24) and one step of Newton's
// method in f64, r + (v - r^2) / (2 r), whose quotient may be an f32: off by 2^-46.
__device__ __forceinline__ double root(double v) {
  if (!(v > 1e-30 && v < 1e30)) return sqrt(v);
  const float r = __fsqrt_rn((float)v);
  return fma(fma(-(double)r, (double)r, v), (double)__fdividef(0.5f, r), (double)r);
}

// tensor k's norm (before scale) from the partials of the blocks that met it; by one warp
template <typename Tab>
__device__ __forceinline__ double tensor_norm(const Tab& t, int k, int blocks, int max_kind, const double* part) {
  double v = 0.0;
  if (t.first[k + 1] > t.first[k]) {
    // the block of a chunk c: the largest b with begin(b) <= c
    const int b0 = (int)((((long long)t.first[k] + 1) * blocks - 1) / t.chunks);
    const int b1 = (int)((((long long)t.first[k + 1]) * blocks - 1) / t.chunks);
    for (int b = b0 + (threadIdx.x & 31); b <= b1; b += 128) {   // (four loads in flight)
      double w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = b + 32 * i <= b1 ? load_part(part + b + 32 * i + k) : 0.0;
#pragma unroll
      for (int i = 0; i < 4; ++i) v = max_kind ? max_nan(v, w[i]) : v + w[i];
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const double w = __shfl_xor_sync(0xffffffffu, v, o);
      v = max_kind ? max_nan(v, w) : v + w;
    }
  }
  return max_kind ? v : root(v);
}

// the norm of everything, from all slots; every thread of the block gets it
__device__ __forceinline__ float total_norm(const double* part, int slots, int max_kind, float scale, double* red) {
  double v = 0.0;
  for (int i = threadIdx.x; i < slots; i += 4 * kGradThreads) {
    double w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = i + j * kGradThreads < slots ? load_part(part + i + j * kGradThreads) : 0.0;
#pragma unroll
    for (int j = 0; j < 4; ++j) v = max_kind ? max_nan(v, w[j]) : v + w[j];
  }
  v = block_reduce(v, max_kind, red);
  float* out = reinterpret_cast<float*>(red + 1);
  if (threadIdx.x == 0) *out = (float)((max_kind ? v : root(v)) * (double)scale);
  __syncthreads();
  return *out;
}

// the tensors' norms, by the warps of all blocks in turn
template <typename Tab>
__device__ __forceinline__ void write_norms(const Tab& t, int b, int blocks, int max_kind, float scale, int part_blocks,
                                            const double* part, float* norms) {
  constexpr int warps = kGradThreads / 32;
  for (int k = b * warps + (threadIdx.x >> 5); k < t.count; k += blocks * warps) {
    const double v = tensor_norm(t, k, part_blocks, max_kind, part);
    if ((threadIdx.x & 31) == 0) norms[k] = (float)(v * (double)scale);
  }
}

template <int N>
__global__ void __launch_bounds__(kGradThreads) grad_finish_kernel(const __grid_constant__ GradTable<N> t, int max_kind,
                                                                   float scale, int blocks, const double* part, const double* all,
                                                                   int slots, float* norm, float* norms) {
  __shared__ double red[kGradThreads];
  grid_dep_wait();
  // (the total by the last block, which has the fewest tensors' norms to do)
  if (norms) write_norms(t, blockIdx.x, gridDim.x, max_kind, scale, blocks, part, norms);
  if (blockIdx.x == gridDim.x - 1 && norm) {
    const float v = total_norm(all, slots, max_kind, scale, red);
    if (threadIdx.x == 0) *norm = v;
  }
}

template <bool BF>
__device__ __forceinline__ uint4 scaled(const uint4& u, float coef) {
  constexpr int per = BF ? 8 : 4;
  float f[8];
  unpack_vec<BF>(u, f);
#pragma unroll
  for (int i = 0; i < per; ++i) f[i] *= coef;
  return BF ? pack8(f)
            : make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
}
template <bool BF>
__device__ __forceinline__ void scale_chunk(const Span& s, long long v0, float coef) {
  constexpr int per = BF ? 8 : 4;
  uint4* out = const_cast<uint4*>(s.base);
  uint4 u[kGradVecs];
  load_chunk<BF>(s, v0, false, u);
  if (inner_chunk<BF>(s, v0)) {
    out += v0 + threadIdx.x;
#pragma unroll
    for (int k = 0; k < kGradVecs; ++k) __stcs(out + k * kGradThreads, scaled<BF>(u[k], coef));
    return;
  }
  const long long vend = (s.end + per - 1) / per;
#pragma unroll
  for (int k = 0; k < kGradVecs; ++k) {
    const long long v = v0 + threadIdx.x + k * kGradThreads;
    if (v >= vend) continue;
    const uint4 w = scaled<BF>(u[k], coef);
    if (whole_vec<BF>(s, v)) {
      out[v] = w;
      continue;
    }
    const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < per; ++i) {
      const long long at = v * per + i;
      if (at < s.lead || at >= s.end) continue;
      if (BF) reinterpret_cast<uint16_t*>(out + v)[i] = (uint16_t)(x[i >> 1] >> (16 * (i & 1)));
      else reinterpret_cast<uint32_t*>(out + v)[i] = x[i];
    }
  }
}

// Block b's gradients scaled.  Every block sums all partials for itself (6 KB
// from L2 at one launch's 608 blocks), so the coefficient needs no kernel of
// its own.
template <typename Tab>
__device__ __forceinline__ void scale_block(const Tab& t, int b, int blocks, int max_kind, float scale, float max_norm,
                                            const double* all, int slots, float* norm, float* coef_out, double* red) {
  const float nv = total_norm(all, slots, max_kind, scale, red);
  const bool fine = isfinite(nv);
  const float clip = fminf(1.f, __fdiv_rn(max_norm, __fadd_rn(nv, 1e-6f)));
  const float coef = fine ? __fmul_rn(scale, clip) : 0.f;
  if (b == 0 && threadIdx.x == 0) {
    if (norm) *norm = nv;
    if (coef_out) *coef_out = coef;
  }
  if (!fine || coef == 1.f) return;   // nothing to change
  // backwards: the last chunks that the norm read are the ones still in L2
  const int c0 = block_begin(t, b, blocks);
  int c = block_begin(t, b + 1, blocks);
  while (c > c0) {
    const int k = tensor_of(t, c - 1);
    const Span s = span_of(t.p[k], t.n[k]);
    const int base = t.first[k], stop = max(base, c0);
    if (s.per == 8)
      for (; c > stop; --c) scale_chunk<true>(s, (long long)(c - 1 - base) * kGradChunk, coef);
    else
      for (; c > stop; --c) scale_chunk<false>(s, (long long)(c - 1 - base) * kGradChunk, coef);
  }
}

template <int N>
__global__ void __launch_bounds__(kGradThreads, kGradBlocksPerSm)
    grad_scale_kernel(const __grid_constant__ GradTable<N> t, int max_kind, float scale, float max_norm, const double* part,
                      const double* all, int slots, float* norm, float* norms, float* coef_out) {
  __shared__ double red[kGradThreads];
  grid_dep_wait();
  scale_block(t, blockIdx.x, gridDim.x, max_kind, scale, max_norm, all, slots, norm, coef_out, red);
  if (norms) write_norms(t, blockIdx.x, gridDim.x, max_kind, scale, gridDim.x, part, norms);
}

int chunks_of(const GradItem& g) {
  if (g.n == 0) return 0;
  const int esz = g.bf16 ? 2 : 4, per = 16 / esz;
  const long long lead = (long long)(reinterpret_cast<uintptr_t>(g.p) & 15) / esz;
  const long long vecs = (lead + g.n + per - 1) / per;
  return (int)((vecs + kGradChunk - 1) / kGradChunk);
}

template <int N>
void fill(GradTable<N>* t, const GradItem* g, int count) {
  t->count = count;
  int c = 0;
  for (int i = 0; i < count; ++i) {
    t->p[i] = g[i].p;
    t->n[i] = g[i].n | (g[i].bf16 ? kGradBf16 : 0);
    t->first[i] = c;
    c += chunks_of(g[i]);
  }
  t->first[count] = c;
  t->chunks = c;
}

int blocks_for(const Ctx& c, int chunks) {
  const int most = c.num_sms * kGradBlocksPerSm;
  return chunks < 1 ? 1 : chunks < most ? chunks : most;
}

template <int N>
cudaError_t run_piece(const Ctx& c, const GradJob& j, int stage, const GradItem* g, int count, double* part, int* slots_used,
                      int slots, float* norms, bool first) {
  GradTable<N> t;
  fill(&t, g, count);
  const int blocks = blocks_for(c, t.chunks);
  *slots_used = blocks + count;
  Ctx cc = c;
  cudaError_t e;
  if (stage == 0) {
    prof_begin(c, "grad_part");
    const int keep = j.clip ? (int)(kGradKeep / (kGradChunk * 16) / blocks) : 0;
    e = launch_k(c, false, grad_part_kernel<N>, dim3(blocks), dim3(kGradThreads), 0, 1, t, keep, j.max_kind, part);
  } else if (j.clip) {
    prof_begin(c, "grad_scale");
    e = launch_k(cc, pdl_allowed(), grad_scale_kernel<N>, dim3(blocks), dim3(kGradThreads), 0, 1, t, j.max_kind, j.scale,
                 j.max_norm, (const double*)part, (const double*)j.part, slots, first ? j.norm : nullptr, norms,
                 first ? j.coef : nullptr);
  } else {
    prof_begin(c, "grad_finish");
    const int grid = std::max(1, std::min((count + 7) / 8, c.num_sms));
    e = launch_k(cc, pdl_allowed(), grad_finish_kernel<N>, dim3(grid), dim3(kGradThreads), 0, 1, t, j.max_kind, j.scale, blocks,
                 (const double*)part, (const double*)j.part, slots, first ? j.norm : nullptr, norms);
  }
  prof_end(c);
  count_launch();
  return launched(e);
}

}  // namespace

size_t grad_part_doubles(int count) {
  const size_t pieces = count <= 0 ? 1 : (size_t)(count + kGradTable - 1) / kGradTable;
  return pieces * kGradMaxBlocks + (size_t)(count < 0 ? 0 : count);
}

cudaError_t launch_grad(const Ctx& c, const GradJob& j) {
  const int pieces = j.count <= 0 ? 1 : (j.count + kGradTable - 1) / kGradTable;
  if (c.num_sms * kGradBlocksPerSm > kGradMaxBlocks) return cudaErrorNotSupported;
  int slots = 0;
  for (int stage = 0; stage < 2; ++stage) {
    int at = 0;
    for (int p = 0; p < pieces; ++p) {
      const int i0 = p * kGradTable, n = std::min(kGradTable, j.count - i0);
      int used = 0;
      float* norms = j.norms ? j.norms + i0 : nullptr;
      // (a short list's table is a few hundred bytes of parameters instead of 20 KB)
      const cudaError_t e = n <= kShortTable ? run_piece<kShortTable>(c, j, stage, j.items + i0, n, j.part + at, &used, slots, norms, p == 0)
                                    : run_piece<kGradTable>(c, j, stage, j.items + i0, n, j.part + at, &used, slots, norms, p == 0);
      if (e != cudaSuccess) return e;
      at += used;
    }
    slots = at;
  }
  return cudaSuccess;
}

}  // namespace collider
