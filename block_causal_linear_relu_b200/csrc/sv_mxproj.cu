// Products of microscaled operands, sm_100a: Y = X W^T with 8- or 4-bit elements and a scale per block
// of K, plain ([rows, features]) or as the Q/K/V projection (ReLU on Q and K, [B, H, N, D] outputs).
//
// The scales enter the tensor cores: tcgen05.mma with .block_scale multiplies each block's partial
// product by both operands' scales, which it reads from TMEM, and accumulates in fp32. All three
// formats use one pipeline, because a 128-byte run of codes is four K steps of 32 bytes in each:
// 128 columns of e4m3 (K = 32 a step) or 256 columns of e2m1 (K = 64 a step).
//
// A persistent kernel of CTA pairs (cta_group::2): an output tile has 256 rows and NT columns; each CTA of
// a pair holds 128 rows of A and NT / 2 of B in its shared memory, and the pair's MMA reads both, so a
// byte of shared memory feeds twice the products that it would in one CTA (with 128 x 128 tiles of one
// CTA the 4-bit kinds need the whole 128 bytes per cycle of shared memory). Few output tiles take
// 128 x 128 tiles of single CTAs, and a cluster of up to eight of them splits a tile's K: a run costs a CTA
// about 450 cycles of issue however few rows it has, so a token's latency is runs per CTA. The partial
// sums meet in distributed shared memory and are added in the order of the ranks.
// A stage holds a 128-byte run of A and B (128-byte swizzle) and their scale tiles (512 bytes per four
// blocks of K, stored in the order in which TMEM wants them). Warp 0 of each CTA issues the copies; warp 1
// (of a pair's even CTA) copies a stage's scales to TMEM and issues its four MMAs; warps 2-9 of each CTA
// drain the accumulator: the tensor scales, bf16, ReLU, a swizzled buffer, and a bulk store of 32 rows x 64
// columns (row by row where those run into another batch). A tile's rows are consecutive rows of X,
// whatever batch they belong to, because the scale tiles run over all rows.
// Measured (20240 x 2560 x 7680, plain, in bursts of 3 ms): SV_NVFP4 157 us, 5070 TFLOP/s (0.76 of four times the
// measured bf16 rate), SV_MXFP4 147, SV_MXFP8 271 us, 2940 TFLOP/s (0.89 of twice it); as the Q/K/V projection 167,
// 164 and 280 us, whose kernels of 192 and 256 columns spill 24 to 60 bytes at 168 registers. What bounds the
// 4-bit kinds is the accumulator's way out of TMEM, which stalls the MMAs (a tile's 5120 MMA cycles take 7400), and
// long runs of any kind the power limit. One row, 2560 x 2560: 4.9 us SV_NVFP4 and SV_MXFP4, 5.7 us SV_MXFP8.
// Rows past the last one and runs past K are zero-filled by the tensor maps; their scales are zero
// bytes, which both scale types read as finite numbers.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdio>
#include <mutex>

#include "../../include/svlinattn.h"
#include "sv_internal.h"
#include "sv_ptx.cuh"

namespace sv {
namespace {

constexpr int kRows = 128;          // rows of A per CTA
constexpr int kEpiWarps = 8;        // two per 32-lane quarter of TMEM, which share its column chunks
constexpr int kThreads = 64 + 32 * kEpiWarps;  // warp 0 copies, warp 1 MMAs, then the epilogue
// A tile's sum has to end before the waits for it do (2 s): 2^26 columns are half a million runs, about 0.4 s where
// every byte comes from DRAM.
constexpr int kMaxCols = 1 << 26;
constexpr int kMaxSplit = 8;        // CTAs that share a tile's K: a portable cluster
// Sixteenths of the next tile's estimated time that a tile's stores are spread over. Q/K/V of 55200 x 2560, 4 bits: 12
// takes 3 % longer and 20 up to 6 %; 16 saves 2 % of SV_MXFP4's and costs the plain products 4 %.
constexpr int kPace = 14;
constexpr int kStaging = 32 * 128;  // per epilogue warp: 32 rows x 64 bf16

template <int FMT, int CTAS, int NT>
struct Cfg {
  static constexpr int kTiles = FMT == SV_NVFP4 ? 4 : FMT == SV_MXFP4 ? 2 : 1;  // scale tiles per run and 128 rows
  static constexpr int kScaleBytes = kTiles * 512;
  static constexpr int kBBlocks = NT > 128 ? 2 : 1;  // 128-row scale blocks that a column tile touches
  static constexpr int kABytes = kRows * 128;
  static constexpr int kBBytes = NT / CTAS * 128;
  static constexpr int kStageBytes = kABytes + kBBytes + (1 + kBBlocks) * kScaleBytes;
  static constexpr int kStride = (kStageBytes + 1023) / 1024 * 1024;  // the swizzle's alignment
  static constexpr int kFit = (227 * 1024 - kEpiWarps * kStaging - 256 - 1024) / kStride;
  static constexpr int kStages = kFit < 8 ? kFit : 8;
  static constexpr int kStagingOff = kStages * kStride;
  static constexpr int kBarOff = kStagingOff + kEpiWarps * kStaging;
  static constexpr int kSmem = kBarOff + 256 + 1024;  // barriers, TMEM slot, alignment slack
  static_assert(CTAS == 2 || (NT == 128 && kStagingOff >= kRows * NT * 4), "a tile's fp32 sums fit into the stages");
  static_assert(kSmem <= 227 * 1024 && kStages >= 4, "shared memory of the microscaled product");
  // TMEM columns: the accumulators (two where they fit), then scales (A: 4 per tile, B: 4 per tile and block), a
  // buffer for every stage: a stage's buffer is written again only when its shared memory has been loaded
  // again, that is, after the MMAs that read both have retired.
  static constexpr uint32_t kScaleCols = 4 * kTiles * (1 + kBBlocks);
  static constexpr int kAccs = 2 * NT + kStages * kScaleCols <= 512 ? 2 : 1;
  static constexpr uint32_t kScaleCol = kAccs * NT;
  static_assert(kScaleCol + kStages * kScaleCols <= 512, "TMEM columns");
  // cycles that a run of K takes: 2 per column on the tensor cores, or its bytes at 60 per cycle. An estimate, for
  // ranking the widths and pacing the stores: loads alone, without MMAs, reach 90 bytes per cycle and SM.
  static constexpr int kRunCycles = 2 * NT > kStageBytes / 60 ? 2 * NT : kStageBytes / 60;
  static constexpr MxKind kKind = FMT == SV_MXFP8 ? kMx8 : FMT == SV_MXFP4 ? kMx4 : kNv4;
};

struct Geo {
  int rows;     // rows of X
  int nout;     // output features
  int runs;     // 128-byte runs of K
  int nt;       // column tiles
  int a_bytes;  // bytes of a run of A that a CTA loads (single CTAs: only the rows there are, rounded up to 8)
  int tiles;    // all tiles
  int N, H, D;  // Q/K/V only: tokens per batch, heads, head features
  int split;    // single CTAs: CTAs of a cluster that share a tile's K
};

struct Maps {
  CUtensorMap a, b;    // codes: [rows, bytes], boxes of 128 rows (A) or NT / CTAS rows (B) x 128 bytes
  CUtensorMap sa, sb;  // scale tiles: [tiles, 512 bytes], boxes of a run's tiles
  CUtensorMap o[3];    // outputs (CTA pairs): y as [rows, features], or q, k, v as [B, H, N, D]; boxes of 32 rows x 64
};

struct Ops {
  const float *ga, *gb;         // tensor scales, or NULL
  __nv_bfloat16 *o0, *o1, *o2;  // y, or q, k, v
};

// Where output feature nc goes: tensor t (0 y or q, 1 k, 2 v), its head and the feature in the head.
struct Place {
  int t, h, d;
};
template <bool kQKV>
__device__ __forceinline__ Place place(const Geo& g, int nc) {
  if (!kQKV) return {0, 0, nc};
  const int hd = g.H * g.D, t = nc / hd, f = nc - t * hd, h = f / g.D;
  return {t, h, f - h * g.D};
}
template <bool kQKV>
__device__ __forceinline__ size_t offset(const Geo& g, const Place& p, int row) {
  if (!kQKV) return static_cast<size_t>(row) * g.nout + p.d;
  const int b = row / g.N;
  return ((static_cast<size_t>(b) * g.H + p.h) * g.N + (row - b * g.N)) * g.D + p.d;
}
__device__ __forceinline__ __nv_bfloat16* output(const Ops& op, int t) {
  return t == 0 ? op.o0 : (t == 1 ? op.o1 : op.o2);
}

// The product of the tensor scales as two factors, a sum times `pre` times `post`. A product that leaves fp32's
// range (g is any positive number) can still give results inside it, and zeros. Sums are zero or between 2^-20
// and 2^54 in magnitude: with pre near 2^-60 or 2^60 the first step neither rounds to a subnormal nor overflows,
// and post is a power of two. Ordinary products, within 2^+-60, are `pre` alone, and post is 1.
struct Alpha {
  float pre, post;
};
__device__ __forceinline__ Alpha tensor_alpha(const Ops& op) {
  const double g = static_cast<double>(*op.ga) * static_cast<double>(*op.gb);  // exact
  const int e = static_cast<int>((__double_as_longlong(g) >> 52) & 0x7ff) - 1023;
  if ((e >= -60 && e <= 60) || e == -1023 || e == 1024) return {static_cast<float>(g), 1.f};  // or zero, infinite, NaN
  const int s = e > 0 ? e - 60 : e + 60, k = min(max(s, -149), 127);  // past these every sum gives zero, or infinity
  return {static_cast<float>(g * __longlong_as_double(static_cast<long long>(1023 - s) << 52)),
          __uint_as_float(k >= -126 ? static_cast<uint32_t>(k + 127) << 23 : 1u << (k + 149))};
}

__device__ __forceinline__ bool warp_all(bool ok) { return __all_sync(0xffffffffu, ok); }

// Whether a product of the tensor scales, rounded to fp32, may need two factors: outside 2^+-59, or NaN.
__device__ __forceinline__ bool far(float alpha) { return !(fabsf(alpha) >= 0x1p-59f && fabsf(alpha) <= 0x1p59f); }

// The epilogue of a warp where the tensor scales multiply to a number far from 1: the same results in the
// plainest way, each lane storing its row. Apart from the other, whose code must not grow: with the second
// factor's code in its loop the 720p Q/K/V projection took 1 to 4 % longer, although it never ran.
template <int CTAS, int NT, int kAccs, bool kQKV>
static __device__ __noinline__ void epilogue_far(Geo g, Ops op, uint32_t tmem, uint64_t* accf, uint64_t* acce,
                                                 int first, int step, int rank, uint32_t* status) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, q = warp & 3, half = (warp - 2) >> 2;
  const Alpha alpha = tensor_alpha(op);
  int tl = 0;
  for (int tile = first; tile < g.tiles; tile += step, ++tl) {
    const int a = tl % kAccs;
    if (!warp_all(mbar_wait_own(&accf[a], (tl / kAccs) & 1, status, 0x6480u | a))) return;
    tc_fence_after();
    const int m = tile / g.nt, n0 = (tile - m * g.nt) * NT;
    const int row = (m * CTAS + rank) * kRows + q * 32 + lane;
    const uint32_t ta = tmem + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(a * NT);
#pragma unroll 1
    for (int c = half; c < NT / 64; c += 2) {
      uint32_t v[64];
      tmem_ld_x64(ta + c * 64, v);
      tmem_wait_ld();
      const int nc = n0 + c * 64;
      if (nc < g.nout && row < g.rows) {
        const Place p = place<kQKV>(g, nc);
        __nv_bfloat16* const out = output(op, p.t) + offset<kQKV>(g, p, row);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if (nc + 8 * j >= g.nout) break;
          uint32_t w[4];
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const uint32_t* f = v + 8 * j + 2 * u;
            w[u] = pack_bf16x2(__uint_as_float(f[0]) * alpha.pre * alpha.post, __uint_as_float(f[1]) * alpha.pre * alpha.post);
            if (kQKV && p.t < 2) w[u] = relu_bf16x2(w[u]);
          }
          reinterpret_cast<uint4*>(out)[j] = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
      __syncwarp();  // the next read of TMEM is the whole warp's
    }
    tc_fence_before();
    __syncwarp();
    if (lane == 0) {
      if (CTAS == 1)
        mbar_arrive(&acce[a]);
      else
        mbar_arrive_pair(mapa_shared(smem_u32(&acce[a]), 0));
    }
  }
}

template <int FMT, int CTAS, int NT, bool kQKV>
__global__ void __launch_bounds__(kThreads, 1)
    mxproj_kernel(const __grid_constant__ Maps maps, const Ops op, const Geo g, uint32_t* status) {
  using C = Cfg<FMT, CTAS, NT>;
  extern __shared__ uint8_t smem_raw[];
  // the dynamic shared memory starts at the same offset in both CTAs of a pair, and so does `smem`
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kBarOff);  // [kStages] a run landed (the even CTA's counts both)
  uint64_t* empty = full + C::kStages;                              // [kStages] the run's MMAs retired
  uint64_t* accf = empty + C::kStages;                              // [2] accumulator holds a finished tile
  uint64_t* acce = accf + 2;                                        // [2] accumulator drained (the even CTA's)
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acce + 2);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int rank = CTAS == 2 ? static_cast<int>(cluster_ctarank()) : 0;
  // Tiles are numbered column tile fastest: the CTAs at work share a few row tiles of A (read from DRAM once)
  // and sweep W, which stays in L2. Blocks of 4 or 8 row tiles, which touch fewer distinct tiles at a time,
  // measured 2.5 and 5 % slower on the 720p Q/K/V projection.
  const int group = CTAS == 2 ? 2 : g.split;  // CTAs that work on one tile
  const int first = static_cast<int>(blockIdx.x) / group, step = static_cast<int>(gridDim.x) / group;
  const int krank = CTAS == 1 && g.split > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int k0 = CTAS == 2 ? 0 : krank * g.runs / g.split, k1 = CTAS == 2 ? g.runs : (krank + 1) * g.runs / g.split;
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&accf[a], 1);
      mbar_init(&acce[a], kEpiWarps * CTAS);
    }
    fence_mbar_init();
    prefetch_tmap(&maps.a);
    prefetch_tmap(&maps.b);
    prefetch_tmap(&maps.sa);
    prefetch_tmap(&maps.sb);
  }
  if (warp == 1) {
    if (CTAS == 1) {
      tmem_alloc(tmem_slot, 512);
      tmem_relinquish();
    } else {
      tmem_alloc_pair(tmem_slot, 512);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (CTAS == 2) {  // the other CTA's barriers are ready
    cluster_arrive_release();
    cluster_wait_acquire();
  }
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  griddep_wait();  // the previous kernel may still write the operands or read the outputs
  if (threadIdx.x == 0) griddep_launch_dependents();

  // Warps 0 and 1 run their loops warp-uniformly and let one lane issue: with the loops inside a one-lane
  // branch every operand of every instruction passed through a vector register, about 65 cycles each.
  if (warp == 0) {  // copies
    const uint64_t pol_a = policy_evict_first();
    const uint64_t pol_b = policy_evict_last();  // W is read by every row tile
    const bool issue = elect_one();
    int s = 0;
    uint32_t phase = 1;  // of `empty`: the first pass over the ring finds it free
    bool ok = true;
    for (int tile = first; tile < g.tiles && ok; tile += step) {
      const int m = tile / g.nt, n0 = (tile - m * g.nt) * NT;
      const int ma = m * CTAS + rank;  // this CTA's 128 rows
      int ta = (ma * g.runs + k0) * C::kTiles;
      int tb = (n0 / 128 * g.runs + k0) * C::kTiles;
      for (int kc = k0; kc < k1; ++kc, ta += C::kTiles, tb += C::kTiles) {
        if (!warp_all(mbar_wait_own(&empty[s], phase, status, 0x6100u | s))) {
          ok = false;
          break;
        }
        uint8_t* sa = smem + s * C::kStride;
        uint8_t* sb = sa + C::kABytes;
        uint8_t* sc = sb + C::kBBytes;
        if (issue) {
          if (CTAS == 1) {
            mbar_expect_tx(&full[s], C::kStageBytes - C::kABytes + g.a_bytes);
            tma_load_2d(sa, &maps.a, &full[s], kc * 128, ma * kRows, pol_a);
            tma_load_2d(sb, &maps.b, &full[s], kc * 128, n0, pol_b);
            tma_load_2d(sc, &maps.sa, &full[s], 0, ta, pol_a);
#pragma unroll
            for (int j = 0; j < C::kBBlocks; ++j)
              tma_load_2d(sc + (1 + j) * C::kScaleBytes, &maps.sb, &full[s], 0, tb + j * g.runs * C::kTiles, pol_b);
          } else {
            const uint32_t bar = mapa_shared(smem_u32(&full[s]), 0);
            if (rank == 0) mbar_expect_tx(&full[s], 2 * C::kStageBytes);
            tma_load_2d_pair(sa, &maps.a, bar, kc * 128, ma * kRows, pol_a);
            tma_load_2d_pair(sb, &maps.b, bar, kc * 128, n0 + rank * (NT / 2), pol_b);
            tma_load_2d_pair(sc, &maps.sa, bar, 0, ta, pol_a);
#pragma unroll
            for (int j = 0; j < C::kBBlocks; ++j)  // both CTAs need the scales of all NT columns
              tma_load_2d_pair(sc + (1 + j) * C::kScaleBytes, &maps.sb, bar, 0, tb + j * g.runs * C::kTiles, pol_b);
          }
        }
        __syncwarp();
        if (++s == C::kStages) s = 0, phase ^= 1;
      }
    }
    // the last runs' MMAs report to this CTA's barriers: stay until they have (a slot never used is free)
    for (int i = 0; i < C::kStages && ok; ++i) {
      ok = warp_all(mbar_wait_own(&empty[s], phase, status, 0x6180u | s));
      if (++s == C::kStages) s = 0, phase ^= 1;
    }
  } else if (warp == 1) {  // scales and MMAs
    if (rank == 0) {
      const bool issue = elect_one();
      // Per run the loop waits, builds descriptors and issues up to 17 instructions; kept short, it runs
      // ahead of the MMAs. So each run asks for the next one's data before it issues its own, and the
      // descriptors of a stage are the first one's low words plus the stage's offset.
      const uint32_t a0 = smem_u32(smem) >> 4;
      const uint64_t hi = sdesc_sw128(0, 16, 1024), hi_sc = sdesc_scales(0);
      int s = 0, tl = 0;
      uint32_t phase = 0, off = 0;
      bool ok = true, ready = mbar_test(&full[0], 0);
      for (int tile = first; tile < g.tiles && ok; tile += step, ++tl) {
        const int a = tl % C::kAccs;
        const uint32_t d = tmem + static_cast<uint32_t>(a * NT);
        const int n0 = (tile % g.nt) * NT;
        const uint32_t shift = static_cast<uint32_t>(n0 % 128) / 32;  // columns of B's first scale block before the tile
        for (int kc = k0; kc < k1; ++kc) {
          if (!warp_all(ready) && !warp_all(mbar_wait_own(&full[s], phase, status, 0x6310u | s))) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t da = hi | (a0 + off), db = hi | (a0 + off + (C::kABytes >> 4)),
                         ds = hi_sc | (a0 + off + ((C::kABytes + C::kBBytes) >> 4));
          uint64_t* const done = &empty[s];
          const uint32_t ta = tmem + C::kScaleCol + static_cast<uint32_t>(s) * C::kScaleCols;
          const uint32_t tb = ta + 4 * C::kTiles;
          off += C::kStride >> 4;
          if (++s == C::kStages) s = 0, phase ^= 1, off = 0;
          ready = mbar_test(&full[s], phase);
          if (issue) {
#pragma unroll
            for (int t = 0; t < C::kTiles; ++t) {
              tmem_copy_scales<CTAS>(ta + 4 * t, ds + 32 * t);
#pragma unroll
              for (int j = 0; j < C::kBBlocks; ++j)
                tmem_copy_scales<CTAS>(tb + 4 * (t * C::kBBlocks + j), ds + ((1 + j) * C::kScaleBytes >> 4) + 32 * t);
            }
          }
          // the accumulator's last tile is drained: asked for after the first run's scales are on their way
          if (kc == k0) {
            if (!warp_all(mbar_wait_own(&acce[a], ((tl / C::kAccs) & 1) ^ 1, status, 0x6300u | a))) {
              ok = false;
              break;
            }
            tc_fence_after();
          }
          if (issue) {
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
              // step kk (32 bytes on): scale tile t, byte id of its 32-bit cells
              const int t = FMT == SV_NVFP4 ? kk : FMT == SV_MXFP4 ? kk >> 1 : 0;
              const uint32_t id = FMT == SV_NVFP4 ? 0 : FMT == SV_MXFP4 ? (kk & 1) * 2 : kk;
              mma_mx<CTAS, C::kKind>(d, da + 2 * kk, db + 2 * kk,
                                     idesc_mx(kRows * CTAS, NT, FMT == SV_MXFP8 ? 0 : 1, FMT != SV_NVFP4, id), ta + 4 * t,
                                     tb + 4 * C::kBBlocks * t + shift, kc != k0 || kk != 0 ? 1u : 0u);
            }
            if (CTAS == 1)
              mma_commit(done);
            else
              mma_commit_pair(done);
            if (kc == k1 - 1) {
              if (CTAS == 1)
                mma_commit(&accf[a]);
              else
                mma_commit_pair(&accf[a]);
            }
          }
          __syncwarp();
        }
      }
    }
  } else if (FMT == SV_NVFP4 && (CTAS == 2 || g.split == 1) && far(*op.ga * *op.gb)) {
    epilogue_far<CTAS, NT, C::kAccs, kQKV>(g, op, tmem, accf, acce, first, step, rank, status);
  } else {  // epilogue: warp w drains TMEM lanes 32 * (w % 4) .. + 31 (rows of this CTA's half)
    const int q = warp & 3, half = (warp - 2) >> 2;
    uint8_t* stg = smem + C::kStagingOff + (warp - 2) * kStaging;
    const float alpha = FMT == SV_NVFP4 ? *op.ga * *op.gb : 1.f;
    const int sub = lane >> 3, piece = lane & 7;  // store step i: row 4 i + sub, 16-byte piece of its 128 bytes
    constexpr int kChunks = NT / 64, kRounds = (kChunks + 1) / 2;
    int tl = 0;
    for (int tile = first; tile < g.tiles; tile += step, ++tl) {
      const int a = tl % C::kAccs;
      if (!warp_all(mbar_wait_own(&accf[a], (tl / C::kAccs) & 1, status, 0x6400u | a))) break;
      tc_fence_after();
      const int m = tile / g.nt, n0 = (tile - m * g.nt) * NT;
      const int row0 = (m * CTAS + rank) * kRows + q * 32;
      const uint32_t ta = tmem + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(a * NT);
      // Stores in one burst per tile hold up the loads of the next tile's runs (a run's load took up to 3300
      // cycles instead of 1000): the warps' chunks go out one by one over the next tile's MMAs, but for the
      // last tile. Paced so, the 720p Q/K/V projection of SV_NVFP4 operands went from 532 to 493 us.
      const long long t0 = clock64();
      const long long gap = CTAS == 2 && tile + step < g.tiles
                                ? static_cast<long long>(g.runs) * C::kRunCycles / (kEpiWarps * kRounds) * kPace / 16
                                : 0;
      const int b0 = kQKV ? row0 / g.N : 0, tok0 = kQKV ? row0 - b0 * g.N : row0;
      // one bulk store takes the warp's 32 rows (clipped at the last token), unless they run into the next batch
      const bool bulk = CTAS == 2 && (!kQKV || tok0 + min(32, g.rows - row0) <= g.N);
      // Everything this warp owns goes to registers at once, and the accumulator is free: TMEM reads stall
      // the tensor cores (about 1700 cycles a tile when spread over the next tile's MMAs), and here all
      // four quarters are read at the same time, with one accumulator while the MMAs wait anyway.
      uint32_t rr[kRounds][64];
#pragma unroll
      for (int round = 0; round < kRounds; ++round)
        if (2 * round + half < kChunks) tmem_ld_x64(ta + (2 * round + half) * 64, rr[round]);
      tmem_wait_ld();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (CTAS == 1)
          mbar_arrive(&acce[a]);
        else
          mbar_arrive_pair(mapa_shared(smem_u32(&acce[a]), 0));
      }
      if (CTAS == 1 && g.split > 1) {
        // to this CTA's shared memory, whose stages are free: [128][NT] fp32, a row's 16-byte pieces swizzled by
        // the row, so that neither these writes (lanes in a column) nor the reads (lanes in a row) collide
        if (row0 + lane < g.rows) {
          float4* part = reinterpret_cast<float4*>(smem) + (q * 32 + lane) * (NT / 4);
#pragma unroll
          for (int round = 0; round < kRounds; ++round)
#pragma unroll
            for (int j = 0; j < 16; ++j)
              if (2 * round + half < kChunks)
                part[((2 * round + half) * 16 + j) ^ lane] =
                    make_float4(__uint_as_float(rr[round][4 * j]), __uint_as_float(rr[round][4 * j + 1]),
                                __uint_as_float(rr[round][4 * j + 2]), __uint_as_float(rr[round][4 * j + 3]));
        }
        continue;
      }
#pragma unroll
      for (int round = 0; round < kRounds; ++round) {
        const int c = 2 * round + half;  // the quarter's two warps take neighbouring chunks
        const int nc = n0 + c * 64;  // first output feature of the chunk
        if (c >= kChunks || nc >= g.nout) continue;
        const Place p = place<kQKV>(g, nc);
        const bool relu = kQKV && p.t < 2;
        if (CTAS == 2) {  // the last bulk store has read the buffer
          if (lane == 0) bulk_wait_read_all();
          __syncwarp();
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const uint32_t* v = rr[round] + 8 * j;
          uint32_t w[4];
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            w[u] = pack_bf16x2(__uint_as_float(v[2 * u]) * alpha, __uint_as_float(v[2 * u + 1]) * alpha);
            if (kQKV && relu) w[u] = relu_bf16x2(w[u]);
          }
          *reinterpret_cast<uint4*>(stg + lane * 128 + ((j ^ (lane & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
        }
        if (bulk) {
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0 && row0 < g.rows) {
            while (clock64() - t0 < gap * (round * kEpiWarps + warp - 2)) __nanosleep(40);
            tma_store_4d(&maps.o[p.t], stg, p.d, tok0, p.h, b0);
            bulk_commit();
          }
          __syncwarp();
        } else {
          __syncwarp();
          __nv_bfloat16* out = output(op, p.t) + piece * 8;
          const bool col_ok = nc + piece * 8 < g.nout;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int r = 4 * i + sub;
            const uint4 w = *reinterpret_cast<const uint4*>(stg + r * 128 + ((piece ^ (r & 7)) << 4));
            if (col_ok && row0 + r < g.rows) *reinterpret_cast<uint4*>(out + offset<kQKV>(g, p, row0 + r)) = w;
          }
        }
        __syncwarp();
      }
    }
    if (CTAS == 2 && lane == 0) bulk_wait_all();
  }
  tc_fence_before();
  __syncthreads();
  if (CTAS == 2 || g.split > 1) {  // neither CTA leaves while the other may still signal its barriers or read its operands
    cluster_arrive_release();
    cluster_wait_acquire();
  }
  if (CTAS == 1 && g.split > 1) {  // each CTA adds its share of the tile's (row, four columns) items
    const int m = first / g.nt, n0 = (first - m * g.nt) * NT;
    const int rows = min(kRows, g.rows - m * kRows);
    const Alpha alpha = FMT == SV_NVFP4 ? tensor_alpha(op) : Alpha{1.f, 1.f};
    constexpr int kPieces = NT / 4;
    for (int i = krank * kThreads + static_cast<int>(threadIdx.x); i < rows * kPieces; i += g.split * kThreads) {
      const int r = i / kPieces, c4 = i - r * kPieces;  // a warp reads whole rows of a rank: 512 bytes
      const uint32_t at = smem_u32(smem) + static_cast<uint32_t>(r * NT * 4 + ((c4 ^ (r & 31)) << 4));
      float4 v[kMaxSplit];
#pragma unroll
      for (int c = 0; c < kMaxSplit; ++c) {
        v[c] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (c < g.split) v[c] = ld_shared_cluster_f4(mapa_shared(at, static_cast<uint32_t>(c)));
      }
      float f[4] = {};
#pragma unroll
      for (int c = 0; c < kMaxSplit; ++c) f[0] += v[c].x, f[1] += v[c].y, f[2] += v[c].z, f[3] += v[c].w;
      const int nc = n0 + c4 * 4;
      if (nc >= g.nout) continue;
      const Place p = place<kQKV>(g, nc);
#pragma unroll
      for (int j = 0; j < 4; ++j) f[j] = f[j] * alpha.pre * alpha.post;
      uint2 w = make_uint2(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]));
      if (kQKV && p.t < 2) w = make_uint2(relu_bf16x2(w.x), relu_bf16x2(w.y));
      *reinterpret_cast<uint2*>(output(op, p.t) + offset<kQKV>(g, p, m * kRows + r)) = w;
    }
    cluster_arrive_release();  // the others may still read this CTA's sums
    cluster_wait_acquire();
  }
  if (warp == 1) {
    tc_fence_after();
    if (CTAS == 1)
      tmem_dealloc(tmem, 512);
    else
      tmem_dealloc_pair(tmem, 512);
  }
}

sv_status pfail(sv_status st, const char* fmt, long long a = 0, long long b = 0) {
  char msg[256];
  snprintf(msg, sizeof(msg), fmt, a, b);
  return set_last_error(st, msg);
}

#define MXP_TRY(x)                \
  do {                            \
    const sv_status _s = (x);     \
    if (_s != SV_OK) return _s;   \
  } while (0)

// Per device (and kernel), looked up once, thread-safe: sets the shared-memory attribute; for single CTAs
// also how many clusters of 1 .. 8 of them run at the same time (a cluster lives in one GPC).
struct DevFacts {
  bool done;
  int clusters[kMaxSplit + 1];
};
cudaLaunchConfig_t config(unsigned ctas, int cluster, int smem, cudaStream_t st, cudaLaunchAttribute (&at)[2]) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = st;
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = static_cast<unsigned>(cluster);
  at[1].val.clusterDim.y = 1;
  at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cfg;
}
template <int FMT, int CTAS, int NT, bool kQKV>
cudaError_t device_facts(int sms, DevFacts& out) {
  using C = Cfg<FMT, CTAS, NT>;
  constexpr int kMaxDev = 64;
  static std::mutex mu;
  static DevFacts facts[kMaxDev] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDev) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> lock(mu);
  DevFacts& f = facts[dev];
  if (!f.done) {
    const auto kernel = mxproj_kernel<FMT, CTAS, NT, kQKV>;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    f.clusters[1] = sms;
    for (int c = 2; CTAS == 1 && c <= kMaxSplit; ++c) {
      cudaLaunchAttribute at[2];
      const cudaLaunchConfig_t cfg = config(static_cast<unsigned>(c), c, C::kSmem, nullptr, at);
      if (cudaOccupancyMaxActiveClusters(&f.clusters[c], kernel, &cfg) != cudaSuccess) {
        cudaGetLastError();
        f.clusters[c] = 0;  // not used
      }
    }
    f.done = true;
  }
  out = f;
  return cudaSuccess;
}

template <int FMT, int CTAS, int NT, bool kQKV>
sv_status run(const sv_mx& x, const sv_mx& w, const Ops& op, Geo g, void* ws, int sms, cudaStream_t st) {
  using C = Cfg<FMT, CTAS, NT>;
  g.nt = (g.nout + NT - 1) / NT;
  const long long tiles = (x.rows + kRows * CTAS - 1) / (kRows * CTAS) * g.nt;
  // scale tiles and output tiles are counted in 32 bits
  const long long sa = mx_row_tiles(x.rows) * g.runs * C::kTiles, sb = mx_row_tiles(w.rows) * g.runs * C::kTiles;
  if (tiles > 0x3fffffffLL || sa > 0x3fffffffLL || sb > 0x3fffffffLL)
    return pfail(SV_ERR_UNSUPPORTED, "too many output tiles or scale tiles");
  g.tiles = static_cast<int>(tiles);
  const uint64_t bytes = static_cast<uint64_t>(FMT == SV_MXFP8 ? x.cols : x.cols / 2);
  g.split = 1;
  Maps maps;
  // the other rows of a short tile keep what is in shared memory: an output row depends on its own row of A
  const uint32_t a_rows = CTAS == 1 && x.rows < kRows ? static_cast<uint32_t>((x.rows + 7) / 8 * 8) : kRows;
  g.a_bytes = static_cast<int>(a_rows) * 128;
  MXP_TRY(encode_bytes_2d(&maps.a, x.codes, bytes, static_cast<uint64_t>(x.rows), a_rows));
  MXP_TRY(encode_bytes_2d(&maps.b, w.codes, bytes, static_cast<uint64_t>(w.rows), NT / CTAS));
  MXP_TRY(encode_scale_tiles(&maps.sa, x.scales, static_cast<uint64_t>(sa), C::kTiles));
  MXP_TRY(encode_scale_tiles(&maps.sb, w.scales, static_cast<uint64_t>(sb), C::kTiles));
  if (CTAS == 2) {
    const uint32_t box[4] = {64, 32, 1, 1};
    if (kQKV) {
      const uint64_t D = static_cast<uint64_t>(g.D), N = static_cast<uint64_t>(g.N), H = static_cast<uint64_t>(g.H);
      const uint64_t dims[4] = {D, N, H, static_cast<uint64_t>(x.rows) / N}, pitch[3] = {2 * D, 2 * N * D, 2 * H * N * D};
      MXP_TRY(encode_bf16_4d(&maps.o[0], op.o0, dims, pitch, box));
      MXP_TRY(encode_bf16_4d(&maps.o[1], op.o1, dims, pitch, box));
      MXP_TRY(encode_bf16_4d(&maps.o[2], op.o2, dims, pitch, box));
    } else {
      const uint64_t F = static_cast<uint64_t>(g.nout), R = static_cast<uint64_t>(x.rows);
      const uint64_t dims[4] = {F, R, 1, 1}, pitch[3] = {2 * F, 2 * R * F, 2 * R * F};
      MXP_TRY(encode_bf16_4d(&maps.o[0], op.o0, dims, pitch, box));
    }
  }
  DevFacts facts;
  cudaError_t e = device_facts<FMT, CTAS, NT, kQKV>(sms, facts);
  if (e == cudaSuccess) {
    if (CTAS == 1) {  // the split of K with the least estimated cycles: 450 a run; the sums' meeting 1800, and 32 a row
      const long long meet = 1800 + 32 * (x.rows < kRows ? x.rows : kRows);
      long long best = 0;
      for (int c = 1; c <= kMaxSplit && c <= g.runs; ++c) {
        if (facts.clusters[c] < 1 || (c > 1 && tiles > facts.clusters[c])) continue;
        const long long waves = (tiles + facts.clusters[c] - 1) / facts.clusters[c];
        const long long cycles = waves * (450ll * ((g.runs + c - 1) / c) + 1000) + (c > 1 ? meet : 0);
        if (c == 1 || cycles < best) best = cycles, g.split = c;
      }
    }
    const int group = CTAS == 2 ? 2 : g.split, groups = sms / group;
    cudaLaunchAttribute at[2];
    const cudaLaunchConfig_t cfg =
        config(static_cast<unsigned>((g.tiles < groups || g.split > 1 ? g.tiles : groups) * group), group, C::kSmem, st, at);
    e = cudaLaunchKernelEx(&cfg, mxproj_kernel<FMT, CTAS, NT, kQKV>, maps, op, g, static_cast<uint32_t*>(ws));
  }
  if (e != cudaSuccess) return pfail(SV_ERR_CUDA, "microscaled product launch failed (%lld)", static_cast<long long>(e));
  return SV_OK;
}

template <int FMT, bool kQKV>
sv_status choose(const sv_mx& x, const sv_mx& w, const Ops& op, const Geo& g, void* ws, int sms, cudaStream_t st) {
  const long long tiles = mx_row_tiles(x.rows) * ((w.rows + 127) / 128);
  if (x.rows <= kRows || tiles <= sms / 2) return run<FMT, 1, 128, kQKV>(x, w, op, g, ws, sms, st);
  // the column tile with the least estimated cycles: waves of tiles, each its runs and the draining of the
  // accumulator
  const auto cost = [&](int nt, int run_cycles) {
    const long long tiles = (x.rows + 255) / 256 * ((w.rows + nt - 1) / nt);
    return (tiles + sms / 2 - 1) / (sms / 2) * (static_cast<long long>(g.runs) * run_cycles + 700);
  };
  const long long c128 = cost(128, Cfg<FMT, 2, 128>::kRunCycles), c192 = cost(192, Cfg<FMT, 2, 192>::kRunCycles),
                  c256 = cost(256, Cfg<FMT, 2, 256>::kRunCycles);
  if (c256 <= c192 && c256 <= c128) return run<FMT, 2, 256, kQKV>(x, w, op, g, ws, sms, st);
  if (c128 < c192) return run<FMT, 2, 128, kQKV>(x, w, op, g, ws, sms, st);
  return run<FMT, 2, 192, kQKV>(x, w, op, g, ws, sms, st);
}

template <bool kQKV>
sv_status product(const sv_mx& x, const sv_mx& w, const Ops& outs, Geo g, void* ws, size_t ws_bytes, cudaStream_t st) {
  if (x.fmt != w.fmt) return pfail(SV_ERR_INVALID_ARG, "x and w have different formats (%lld and %lld)", x.fmt, w.fmt);
  if (x.cols != w.cols) return pfail(SV_ERR_INVALID_ARG, "x and w have different columns (%lld and %lld)", x.cols, w.cols);
  if (x.cols > kMaxCols) return pfail(SV_ERR_UNSUPPORTED, "cols=%lld must be at most %lld", x.cols, kMaxCols);
  if (ws == nullptr || (reinterpret_cast<uintptr_t>(ws) & 255u) != 0u || ws_bytes < static_cast<size_t>(kHeaderBytes))
    return pfail(SV_ERR_INVALID_ARG, "ws must be a 256-byte aligned workspace of at least %lld bytes", kHeaderBytes);
  const size_t n = 2 * static_cast<size_t>(x.rows) * static_cast<size_t>(kQKV ? w.rows / 3 : w.rows);
  if (overlap(outs.o0, n, outs.o1, n) || overlap(outs.o0, n, outs.o2, n) || overlap(outs.o1, n, outs.o2, n))
    return pfail(SV_ERR_INVALID_ARG, "the outputs must not overlap");
  for (const void* o : {outs.o0, outs.o1, outs.o2})
    if (overlap(x, o, n) || overlap(w, o, n)) return pfail(SV_ERR_INVALID_ARG, "an output must not overlap x or w");
  g.rows = static_cast<int>(x.rows);
  g.nout = static_cast<int>(w.rows);
  g.runs = mx_runs(x.fmt, x.cols);
  int sms = 0;
  MXP_TRY(mx_device(&sms));
  Ops op = outs;
  op.ga = x.gscale;
  op.gb = w.gscale;
  if (x.fmt == SV_MXFP8) return choose<SV_MXFP8, kQKV>(x, w, op, g, ws, sms, st);
  if (x.fmt == SV_MXFP4) return choose<SV_MXFP4, kQKV>(x, w, op, g, ws, sms, st);
  return choose<SV_NVFP4, kQKV>(x, w, op, g, ws, sms, st);
}

bool out16(const void* p) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & 15u) == 0u; }

}  // namespace
}  // namespace sv

extern "C" sv_status sv_mx_projection(const sv_mx* x, const sv_mx* w, void* y, void* ws, size_t ws_bytes,
                                      sv_stream_t stream) {
  using namespace sv;
  MXP_TRY(check_mx(x, "x"));
  MXP_TRY(check_mx(w, "w"));
  if (w->rows % 8 != 0) return pfail(SV_ERR_UNSUPPORTED, "w.rows=%lld (output features) must be a multiple of 8", w->rows);
  if (!out16(y)) return pfail(SV_ERR_INVALID_ARG, "y must be non-NULL and 16-byte aligned");
  Ops op = {};
  op.o0 = static_cast<__nv_bfloat16*>(y);
  Geo g = {};
  return product<false>(*x, *w, op, g, ws, ws_bytes, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" sv_status sv_mx_qkv_projection(const sv_mx* x, const sv_mx* w, void* q, void* k, void* v, int B, int N, int H,
                                          int D, void* ws, size_t ws_bytes, sv_stream_t stream) {
  using namespace sv;
  MXP_TRY(check_mx(x, "x"));
  MXP_TRY(check_mx(w, "w"));
  if (B < 1 || N < 1 || H < 1) return pfail(SV_ERR_INVALID_ARG, "B, N and H must be >= 1");
  if (D != 64 && D != 128) return pfail(SV_ERR_UNSUPPORTED, "the projections need D = 64 or 128, got %lld", D);
  if (static_cast<long long>(B) * N != x->rows)
    return pfail(SV_ERR_INVALID_ARG, "x must have B * N = %lld rows, got %lld", static_cast<long long>(B) * N, x->rows);
  if (3ll * H * D != w->rows)
    return pfail(SV_ERR_INVALID_ARG, "w must have 3 * H * D = %lld rows, got %lld", 3ll * H * D, w->rows);
  if (!out16(q) || !out16(k) || !out16(v)) return pfail(SV_ERR_INVALID_ARG, "q, k, v must be non-NULL and 16-byte aligned");
  Ops op = {};
  op.o0 = static_cast<__nv_bfloat16*>(q);
  op.o1 = static_cast<__nv_bfloat16*>(k);
  op.o2 = static_cast<__nv_bfloat16*>(v);
  Geo g = {};
  g.N = N;
  g.H = H;
  g.D = D;
  return product<true>(*x, *w, op, g, ws, ws_bytes, reinterpret_cast<cudaStream_t>(stream));
}
