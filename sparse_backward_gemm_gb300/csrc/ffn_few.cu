// The gated feed-forward block's forward of a few tokens (M <= 128, ffn_few): its time is
// the reading of the weights, so they are the wide operand.  A tile of 128
// output features (64 gates and the same 64 ups, or 128 columns of y) is the A
// of 128 x N x 16 MMAs, the tokens, padded to N = 16, 32, 64 or 128, are the B: the
// weights pass by TMA from memory to the tensor core, each once, and no thread
// touches them.  A cluster's CTAs split the reduction, so that all SMs read;
// their parts meet through distributed shared memory, in CTA order.
//   Measured at 2048 x 5632 (69 MB of weights; 10.3 us at the copy rate): 1 token
// 22 us, 64 29, 128 36; as 256-row tiles 65 (of 256 columns), 37 and 38.
#include <algorithm>
#include <mutex>

#include "glu.cuh"
#include "internal.h"
#include "tc_ptx.cuh"

namespace collider {

namespace {

using namespace tc;

constexpr int kFewThreads = 192;   // warp 0 TMA, warp 1 MMA and TMEM, warps 2-5 epilogue
constexpr uint32_t kWBytes = 128 * 64 * 2;   // a 64-deep slice of the weights' tile
constexpr int kFewRows = 128;

struct FewParams {
  int M, N, kb;        // tokens; columns of the output (kUp: F); k-slices in all
  __nv_bfloat16 *up, *out;   // up: null, or [M, 2F]; out: s or y
  long long up_ld, out_ld;
  DevStatus* st;
};

constexpr int kUp = 0, kDown = 1;   // the first product with the activation, the second

// The second product's ring fits beside one of the first's in an SM: while the
// first runs, it fills with weights.  (A deeper one, 8 slices beside 4: one of
// its clusters finds no 8 SMs with room until the others are gone, 28 us
// instead of 23 at 1 token x 2048 x 5632.)
// SPLIT (second product, M <= 64): s as the sum of two bf16 values, rows 0..M-1
// and M..2M-1 of its buffer, N / 2 columns of the MMAs each.  The products are
// free here, and y is then off by its own rounding alone (1.7e-3 of its norm; by
// that of s too 2.4e-3).
template <int NT>
struct FewCfg {
  static constexpr uint32_t kXBytes = NT * 128, kStage = kWBytes + kXBytes;
  static constexpr int kStages = NT == 128 ? 3 : NT == 64 ? 4 : 5;
  static constexpr size_t kSmem = 1024 + kStages * kStage + 128;
};

template <int NT, int PHASE, int ACT, bool SPLIT>
__global__ void __launch_bounds__(kFewThreads)
    ffn_few_kernel(const __grid_constant__ CUtensorMap mx, const __grid_constant__ CUtensorMap mw, FewParams p) {
  using C = FewCfg<NT>;
  constexpr int S = C::kStages;
  constexpr bool kTwoRows = SPLIT && PHASE == kDown;
  static_assert(S * C::kStage >= NT * kFewRows * 4, "the parts lie where the slices lay");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + S * C::kStage);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * S + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const uint32_t full0 = smem_u32(bars), empty0 = smem_u32(bars + S), done = smem_u32(bars + 2 * S);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(full0 + 8 * s, 1);
      mbar_init(empty0 + 8 * s, 1);
    }
    mbar_init(done, 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&mw)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&mx)) : "memory");
  }
  if (warp == 1) tmem_alloc(smem_u32(tmem_slot), NT < 32 ? 32 : NT);
  fence_before();
  __syncthreads();
  fence_after();
  // The second product's CTAs may come while the first's are still at work (all
  // of those have started) and fill their rings with weights.
  if (PHASE == kUp) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const uint32_t tmem = *tmem_slot;
  const int parts = gridDim.x, part = blockIdx.x, col0 = blockIdx.y * (PHASE == kUp ? 64 : 128);
  const int k0 = (int)((long long)part * p.kb / parts), k1 = (int)((long long)(part + 1) * p.kb / parts);
  if (warp == 0) {
    const bool leader = elect_one();
    auto weights = [&](int kb, int stage) {
      const uint32_t sa = smem_u32(smem + stage * C::kStage), fb = full0 + 8 * stage;
      mbar_expect_tx(fb, C::kStage);
      tma_load_2d(sa, &mw, fb, col0, kb * 64);
      tma_load_2d(sa + 8192, &mw, fb, PHASE == kUp ? p.N + col0 : col0 + 64, kb * 64);
    };
    auto tokens = [&](int kb, int stage) {
      const uint32_t sb = smem_u32(smem + stage * C::kStage) + kWBytes;
      tma_load_2d(sb, &mx, full0 + 8 * stage, kb * 64, 0);
      if (kTwoRows) tma_load_2d(sb + C::kXBytes / 2, &mx, full0 + 8 * stage, kb * 64, p.M);
    };
    const int first = min(S, k1 - k0);
    if (leader)
      for (int i = 0; i < first; ++i) weights(k0 + i, i);
    grid_dep_wait();   // (the weights are no kernel's of this call: the first product was launched behind all before it)
    if (leader)
      for (int i = 0; i < first; ++i) tokens(k0 + i, i);
    __syncwarp();
    int stage = first % S;
    uint32_t phase = first == S ? 1u : 0u;
    bool ok = true;
    for (int kb = k0 + first; kb < k1 && ok; ++kb) {
      ok = __all_sync(0xffffffffu, mbar_wait(empty0 + 8 * stage, phase ^ 1u, abort_flag, p.st, 21)) != 0;
      if (ok && leader) {
        weights(kb, stage);
        tokens(kb, stage);
      }
      __syncwarp();
      if (++stage == S) { stage = 0; phase ^= 1u; }
    }
    if (!ok && leader) {
      // let the copies in flight land (bounded) before the shared memory goes
      for (int s = 0; s < S; ++s) {
        const uint64_t t0 = globaltimer_ns();
        while (!mbar_try(full0 + 8 * s, 0) && !mbar_try(full0 + 8 * s, 1) && globaltimer_ns() - t0 < 10000000ull) {
        }
      }
    }
  } else if (warp == 1) {
    const bool leader = elect_one();
    constexpr uint32_t idesc = idesc_bf16(128, NT, true, false);
    int stage = 0;
    uint32_t phase = 0;
    for (int kb = k0; kb < k1; ++kb) {
      if (!__all_sync(0xffffffffu, mbar_wait(full0 + 8 * stage, phase, abort_flag, p.st, 22))) break;
      fence_after();
      if (leader) {
        const uint32_t sa = smem_u32(smem + stage * C::kStage), sb = sa + kWBytes;
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          mma_bf16(tmem, sdesc(sa + kk * 2048, 8192, 1024), sdesc(sb + kk * 32, 16, 1024), idesc, kb > k0 || kk > 0);
        mma_commit(empty0 + 8 * stage);
        if (kb == k1 - 1) mma_commit(done);
      }
      __syncwarp();
      if (++stage == S) { stage = 0; phase ^= 1u; }
    }
  } else {
    // the accumulators as [token][feature] f32 over the ring, which is read out
    volatile int no_abort = 0;
    const int q = warp & 3, row = q * 32 + lane;
    float* mine = reinterpret_cast<float*>(smem);
    if (k1 > k0 && mbar_wait(done, 0, &no_abort, p.st, 23)) {
      fence_after();
      const uint32_t tc0 = tmem + (static_cast<uint32_t>(q * 32) << 16);
      constexpr int T = kTwoRows ? NT / 2 : NT;   // tokens
#pragma unroll
      for (int c = 0; c < T; c += 16) {
        uint32_t r[16], lo[16];
        tmem_ld16_async(tc0 + c, r);
        if (kTwoRows && T >= 16) tmem_ld16_async(tc0 + T + c, lo);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < (T < 16 ? T : 16); ++i) {
          float v = __uint_as_float(r[i]);
          if (kTwoRows) v += __uint_as_float(T < 16 ? r[(i + T) & 15] : lo[i]);
          if (c + i < p.M) mine[(c + i) * kFewRows + row] = v;
        }
      }
      fence_before();
    }
  }
  if (parts > 1) cluster_sync(); else __syncthreads();
  if (warp >= 2) {
    // every CTA finishes its share of the tokens, a warp one at a time
    const int t0 = part * p.M / parts, t1 = (part + 1) * p.M / parts;
    const float* mine = reinterpret_cast<const float*>(smem);
    for (int t = t0 + warp - 2; t < t1; t += 4) {
      float2 a = make_float2(0.f, 0.f), b = a;
      for (int r = 0; r < parts; ++r) {
        const float* from = parts > 1 ? peer_generic(mine, r) : mine;
        const float2 x = *reinterpret_cast<const float2*>(from + t * kFewRows + 2 * lane),
                     y = *reinterpret_cast<const float2*>(from + t * kFewRows + 64 + 2 * lane);
        a.x += x.x; a.y += x.y; b.x += y.x; b.y += y.y;
      }
      const int col = col0 + 2 * lane;
      if (PHASE == kUp) {
        if (col >= p.N) continue;
        if (p.up) {
          __nv_bfloat16* o = p.up + t * p.up_ld + col;
          *reinterpret_cast<uint32_t*>(o) = pack_bf16x2(a.x, a.y);
          *reinterpret_cast<uint32_t*>(o + p.N) = pack_bf16x2(b.x, b.y);
        }
        const float sx = glu_act<ACT>(a.x) * b.x, sy = glu_act<ACT>(a.y) * b.y;
        const uint32_t hi = pack_bf16x2(sx, sy);
        *reinterpret_cast<uint32_t*>(p.out + t * p.out_ld + col) = hi;
        if (SPLIT) {   // (what an infinity leaves is 0)
          const float rx = sx - __uint_as_float(hi << 16), ry = sy - __uint_as_float(hi & 0xffff0000u);
          *reinterpret_cast<uint32_t*>(p.out + (p.M + t) * p.out_ld + col) =
              pack_bf16x2(isfinite(rx) ? rx : 0.f, isfinite(ry) ? ry : 0.f);
        }
      } else {
        __nv_bfloat16* o = p.out + t * p.out_ld + col;
        if (col < p.N) *reinterpret_cast<uint32_t*>(o) = pack_bf16x2(a.x, a.y);
        if (col + 64 < p.N) *reinterpret_cast<uint32_t*>(o + 64) = pack_bf16x2(b.x, b.y);
      }
    }
  }
  if (parts > 1) cluster_sync(); else __syncthreads();   // the parts stay until all are read
  if (warp == 1) {
    fence_after();
    tmem_dealloc(tmem, NT < 32 ? 32 : NT);
  }
}

// CTAs that split a reduction of kb slices over `blocks` tiles: the smallest
// power of two that gives every SM a CTA, a CTA at least four slices, at most 8
int few_parts(int blocks, int kb, int num_sms) {
  int parts = 1;
  while (parts < 8 && blocks * parts < num_sms * 3 / 4 && kb / (2 * parts) >= 4) parts *= 2;
  return parts;
}

template <int NT, int PHASE, int ACT, bool SPLIT>
cudaError_t launch_few(const Ctx& c, const CUtensorMap& mx, const CUtensorMap& mw, const FewParams& p) {
  auto k = ffn_few_kernel<NT, PHASE, ACT, SPLIT>;
  constexpr size_t smem = FewCfg<NT>::kSmem;
  static std::mutex mu;
  static bool known[64] = {false};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  {
    std::lock_guard<std::mutex> lk(mu);
    if (dev < 0 || dev >= 64 || !known[dev]) {
      e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
      if (e != cudaSuccess) return e;
      if (dev >= 0 && dev < 64) known[dev] = true;
    }
  }
  const int blocks = PHASE == kUp ? (p.N + 63) / 64 : (p.N + 127) / 128;
  const int parts = few_parts(blocks, p.kb, c.num_sms);
  prof_begin(c, PHASE == kUp ? "ffn_few_up" : "ffn_few_down", p.M, PHASE == kUp ? 2ll * p.N : p.N, p.kb * 64, 0);
  e = launch_k(c, PHASE == kDown && pdl_allowed(), k, dim3(parts, blocks), dim3(kFewThreads), smem, parts, mx, mw, p);
  prof_end(c);
  count_launch();
  return launched(e);
}

template <int ACT>
cudaError_t launch_up(const Ctx& c, const CUtensorMap& mx, const CUtensorMap& mw, const FewParams& p) {
  if (p.M <= 16) return launch_few<16, kUp, ACT, true>(c, mx, mw, p);
  if (p.M <= 32) return launch_few<32, kUp, ACT, true>(c, mx, mw, p);
  if (p.M <= 64) return launch_few<64, kUp, ACT, true>(c, mx, mw, p);
  return launch_few<128, kUp, ACT, false>(c, mx, mw, p);
}
cudaError_t launch_down(const Ctx& c, const CUtensorMap& mx, const CUtensorMap& mw, const FewParams& p) {
  if (p.M <= 8) return launch_few<16, kDown, 0, true>(c, mx, mw, p);
  if (p.M <= 16) return launch_few<32, kDown, 0, true>(c, mx, mw, p);
  if (p.M <= 32) return launch_few<64, kDown, 0, true>(c, mx, mw, p);
  if (p.M <= 64) return launch_few<128, kDown, 0, true>(c, mx, mw, p);
  return launch_few<128, kDown, 0, false>(c, mx, mw, p);
}

}  // namespace

cudaError_t launch_ffn_few(const Ctx& c, const FfnFew& a) {
  const int nt = a.M <= 16 ? 16 : a.M <= 32 ? 32 : a.M <= 64 ? 64 : 128;
  const bool split = a.M <= kFfnSplit;
  CUtensorMap mx, mw, ms, md;
  if (!make_tensor_map(&mx, a.x, false, a.D, a.M, a.x_ld, 64, nt) ||
      !make_tensor_map(&mw, a.w_up, false, 2ll * a.F, a.D, 2ll * a.F, 64, 64) ||
      !make_tensor_map(&ms, a.s, false, a.F, split ? 2 * a.M : a.M, a.F, 64, a.M <= 8 ? 8 : nt) ||
      !make_tensor_map(&md, a.w_down, false, a.D, a.F, a.D, 64, 64))
    return cudaErrorInvalidValue;
  FewParams p{a.M, a.F, (a.D + 63) / 64, a.up, a.s, a.up_ld, a.F, c.st};
  cudaError_t e = a.act == kGluSilu ? launch_up<kGluSilu>(c, mx, mw, p) : launch_up<kGluGeluTanh>(c, mx, mw, p);
  if (e != cudaSuccess) return e;
  p = FewParams{a.M, a.D, (a.F + 63) / 64, nullptr, a.y, 0, a.y_ld, c.st};
  return launch_down(c, ms, md, p);
}

}  // namespace collider
