// Products of microscaled operands, sm_100a: Y = X W^T with 8- or 4-bit elements and a scale per block
// of K, plain ([rows, features]) or as the Q/K/V projection (ReLU on Q and K, [B, H, N, D] outputs).
//
// The scales enter the tensor cores: tcgen05.mma with .block_scale multiplies each block's partial
// product by both operands' scales, which it reads from TMEM, and accumulates in fp32. All three
// formats use one pipeline, because a 128-byte run of codes is four K steps of 32 bytes in each:
// 128 columns of e4m3 (K = 32 a step) or 256 columns of e2m1 (K = 64 a step).
//
// A persistent kernel, one CTA per SM, 128 x 128 output tiles. A stage holds a run of A and of B (128
// rows x 128 bytes each, 128-byte swizzle) and their scale tiles (512 bytes per four blocks of K, stored
// in the order in which TMEM wants them, so a plain bulk copy fetches them). Warp 0 issues the copies;
// warp 1 copies a stage's scales to TMEM and issues its four MMAs into one of two fp32 accumulators;
// warps 2-5 drain the other: the tensor scales, bf16, ReLU, a swizzled buffer, and row-coalesced
// 16-byte stores. A tile's rows are consecutive rows of X, whatever batch they belong to, because the
// scale tiles run over all rows; the stores find each row's batch and token.
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

constexpr int kM = 128, kN = 128;
constexpr int kRunBytes = 128 * 128;  // one run of one operand: 128 rows x 128 bytes
constexpr int kThreads = 192;         // warp 0 copies, warp 1 MMAs, warps 2-5 epilogue
constexpr int kStaging = 32 * 128;    // per epilogue warp: 32 rows x 64 bf16

template <int FMT>
struct Cfg {
  static constexpr int kTiles = FMT == SV_NVFP4 ? 4 : FMT == SV_MXFP4 ? 2 : 1;  // scale tiles per run and 128 rows
  static constexpr int kScaleBytes = kTiles * 512;
  static constexpr int kStageBytes = 2 * kRunBytes + 2 * kScaleBytes;
  static constexpr int kStages = 5;
  static constexpr int kStagingOff = kStages * kStageBytes;
  static constexpr int kBarOff = kStagingOff + 4 * kStaging;
  static constexpr int kSmem = kBarOff + 256 + 1024;  // barriers, TMEM slot, alignment slack
  static_assert(kSmem <= 227 * 1024, "shared memory of the microscaled product");
  static_assert(kStageBytes % 1024 == 0, "stages keep the swizzle's 1024-byte alignment");
};

// TMEM columns: two accumulators, then the scales of two stages (A: 4 per tile, B: 4 per tile)
constexpr uint32_t kScaleCol = 2 * kN;
constexpr uint32_t kScaleColsPerStage = 32;

struct Geo {
  int rows;        // rows of X
  int nout;        // output features
  int runs;        // 128-byte runs of K
  int nt;          // column tiles
  int tiles;       // all tiles, column tile fastest
  int N, H, D;     // Q/K/V only: tokens per batch, heads, head features
};

struct Ops {
  const uint8_t *sa, *sb;    // scale tiles of X and W
  const float *ga, *gb;      // tensor scales, or NULL
  __nv_bfloat16 *o0, *o1, *o2;  // y, or q, k, v
};

__device__ __forceinline__ bool warp_all(bool ok) { return __all_sync(0xffffffffu, ok); }

template <int FMT, bool kQKV>
__global__ void __launch_bounds__(kThreads, 1)
    mxproj_kernel(const __grid_constant__ CUtensorMap a_map, const __grid_constant__ CUtensorMap b_map, const Ops op,
                  const Geo g, uint32_t* status) {
  using C = Cfg<FMT>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kBarOff);  // [kStages] a run of both operands landed
  uint64_t* empty = full + C::kStages;                              // [kStages] the run's MMAs retired
  uint64_t* accf = empty + C::kStages;                              // [2] accumulator holds a finished tile
  uint64_t* acce = accf + 2;                                        // [2] accumulator drained
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acce + 2);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&accf[a], 1);
      mbar_init(&acce[a], 4);
    }
    fence_mbar_init();
    prefetch_tmap(&a_map);
    prefetch_tmap(&b_map);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  griddep_wait();  // the previous kernel may still write the operands or read the outputs
  if (threadIdx.x == 0) griddep_launch_dependents();

  if (warp == 0) {
    if (lane == 0) {  // copies
      const uint64_t pol_a = policy_evict_first();
      const uint64_t pol_b = policy_evict_last();  // W is read by every row tile
      int it = 0;
      bool ok = true;
      for (int tile = blockIdx.x; tile < g.tiles && ok; tile += gridDim.x) {
        const int m = tile / g.nt, n = tile - m * g.nt;
        for (int kc = 0; kc < g.runs; ++kc, ++it) {
          const int s = it % C::kStages;
          if (!mbar_wait(&empty[s], ((it / C::kStages) & 1) ^ 1, status, 0x6100u | s)) {
            ok = false;
            break;
          }
          uint8_t* st = smem + s * C::kStageBytes;
          mbar_expect_tx(&full[s], C::kStageBytes);
          tma_load_2d(st, &a_map, &full[s], kc * 128, m * kM, pol_a);
          tma_load_2d(st + kRunBytes, &b_map, &full[s], kc * 128, n * kN, pol_b);
          uint8_t* sc = st + 2 * kRunBytes;
          bulk_load(sc, op.sa + (static_cast<size_t>(m) * g.runs + kc) * C::kScaleBytes, C::kScaleBytes, &full[s]);
          bulk_load(sc + C::kScaleBytes, op.sb + (static_cast<size_t>(n) * g.runs + kc) * C::kScaleBytes, C::kScaleBytes,
                    &full[s]);
        }
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {  // scales and MMAs
      int it = 0, tl = 0;
      bool ok = true;
      for (int tile = blockIdx.x; tile < g.tiles && ok; tile += gridDim.x, ++tl) {
        const int a = tl & 1;
        if (!mbar_wait(&acce[a], ((tl >> 1) & 1) ^ 1, status, 0x6300u | a)) break;
        tc_fence_after();
        const uint32_t d = tmem + static_cast<uint32_t>(a * kN);
        for (int kc = 0; kc < g.runs; ++kc, ++it) {
          const int s = it % C::kStages;
          if (!mbar_wait(&full[s], (it / C::kStages) & 1, status, 0x6310u | s)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t sa = smem_u32(smem + s * C::kStageBytes);
          const uint32_t sb = sa + kRunBytes;
          const uint32_t sc = sb + kRunBytes;
          const uint32_t ta = tmem + kScaleCol + static_cast<uint32_t>(it & 1) * kScaleColsPerStage;
          const uint32_t tb = ta + 4 * C::kTiles;
#pragma unroll
          for (int t = 0; t < C::kTiles; ++t) {
            tmem_copy_scales(ta + 4 * t, sc + 512 * t);
            tmem_copy_scales(tb + 4 * t, sc + C::kScaleBytes + 512 * t);
          }
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            const uint64_t da = sdesc_sw128(sa + kk * 32, 16, 1024), db = sdesc_sw128(sb + kk * 32, 16, 1024);
            const uint32_t acc = (kc | kk) != 0 ? 1u : 0u;
            if (FMT == SV_MXFP8)
              mma_mxf8(d, da, db, idesc_mx(kM, kN, 0, true, kk), ta, tb, acc);
            else if (FMT == SV_MXFP4)
              mma_mxf4(d, da, db, idesc_mx(kM, kN, 1, true, (kk & 1) * 2), ta + 4 * (kk >> 1), tb + 4 * (kk >> 1), acc);
            else
              mma_nvf4(d, da, db, idesc_mx(kM, kN, 1, false, 0), ta + 4 * kk, tb + 4 * kk, acc);
          }
          mma_commit(&empty[s]);
        }
        if (ok) mma_commit(&accf[a]);
      }
    }
  } else {  // epilogue: warp w drains TMEM lanes 32 * (w % 4) .. + 31 (rows of the tile)
    const int q = warp & 3;
    uint8_t* stg = smem + C::kStagingOff + (warp - 2) * kStaging;
    const float alpha = FMT == SV_NVFP4 ? *op.ga * *op.gb : 1.f;
    const int sub = lane >> 3, piece = lane & 7;  // store step i: row 4 i + sub, 16-byte piece of its 128 bytes
    int tl = 0;
    for (int tile = blockIdx.x; tile < g.tiles; tile += gridDim.x, ++tl) {
      const int a = tl & 1;
      if (!warp_all(mbar_wait(&accf[a], (tl >> 1) & 1, status, 0x6400u | a))) break;
      tc_fence_after();
      const int m = tile / g.nt, n = tile - m * g.nt;
      const int row0 = m * kM + q * 32;
      const uint32_t ta = tmem + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(a * kN);
      size_t at[8];  // element offsets of the rows that this lane stores
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int r = row0 + 4 * i + sub;
        if (kQKV) {
          const int b = r / g.N;
          at[i] = (static_cast<size_t>(b) * g.H * g.N + (r - b * g.N)) * g.D;
        } else {
          at[i] = static_cast<size_t>(r) * g.nout;
        }
      }
#pragma unroll 1
      for (int c = 0; c < kN / 64; ++c) {
        uint32_t rr[2][32];
        tmem_ld_x32(ta + c * 64, rr[0]);
        tmem_ld_x32(ta + c * 64 + 32, rr[1]);
        tmem_wait_ld();
        if (c == kN / 64 - 1) {  // the tile's last TMEM read: the accumulator is free
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&acce[a]);
        }
        const int nc = n * kN + c * 64;  // first output feature of the chunk
        if (nc >= g.nout) continue;
        __nv_bfloat16* out = op.o0;
        bool relu = false;
        size_t base = static_cast<size_t>(nc);
        if (kQKV) {
          const int hd = g.H * g.D, t = nc / hd, f = nc - t * hd, h = f / g.D;
          out = t == 0 ? op.o0 : (t == 1 ? op.o1 : op.o2);
          relu = t < 2;
          base = static_cast<size_t>(h) * g.N * g.D + (f - h * g.D);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const uint32_t* v = rr[j >> 2] + 8 * (j & 3);
          uint32_t w[4];
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            w[u] = pack_bf16x2(__uint_as_float(v[2 * u]) * alpha, __uint_as_float(v[2 * u + 1]) * alpha);
            if (kQKV && relu) w[u] = relu_bf16x2(w[u]);
          }
          *reinterpret_cast<uint4*>(stg + lane * 128 + ((j ^ (lane & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
        }
        __syncwarp();
        const bool col_ok = nc + piece * 8 < g.nout;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int r = 4 * i + sub;
          const uint4 w = *reinterpret_cast<const uint4*>(stg + r * 128 + ((piece ^ (r & 7)) << 4));
          if (col_ok && row0 + r < g.rows) *reinterpret_cast<uint4*>(out + at[i] + base + piece * 8) = w;
        }
        __syncwarp();
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
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

// The kernel's shared-memory attribute, set once per device (and per kernel), thread-safe.
template <int FMT, bool kQKV>
cudaError_t ensure_attr() {
  constexpr int kMaxDev = 64;
  static std::mutex mu;
  static bool done[kMaxDev] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDev) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> lock(mu);
  if (!done[dev]) {
    e = cudaFuncSetAttribute(mxproj_kernel<FMT, kQKV>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<FMT>::kSmem);
    if (e != cudaSuccess) return e;
    done[dev] = true;
  }
  return cudaSuccess;
}

template <int FMT, bool kQKV>
sv_status run(const CUtensorMap& am, const CUtensorMap& bm, const Ops& op, const Geo& g, void* ws, int sms, cudaStream_t st) {
  cudaError_t e = ensure_attr<FMT, kQKV>();
  if (e == cudaSuccess) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(g.tiles < sms ? g.tiles : sms));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = Cfg<FMT>::kSmem;
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, mxproj_kernel<FMT, kQKV>, am, bm, op, g, static_cast<uint32_t*>(ws));
  }
  if (e != cudaSuccess) return pfail(SV_ERR_CUDA, "microscaled product launch failed (%lld)", static_cast<long long>(e));
  return SV_OK;
}

template <bool kQKV>
sv_status product(const sv_mx& x, const sv_mx& w, const Ops& outs, Geo g, void* ws, size_t ws_bytes, cudaStream_t st) {
  if (x.fmt != w.fmt) return pfail(SV_ERR_INVALID_ARG, "x and w have different formats (%lld and %lld)", x.fmt, w.fmt);
  if (x.cols != w.cols) return pfail(SV_ERR_INVALID_ARG, "x and w have different columns (%lld and %lld)", x.cols, w.cols);
  if (ws == nullptr || (reinterpret_cast<uintptr_t>(ws) & 255u) != 0u || ws_bytes < static_cast<size_t>(kHeaderBytes))
    return pfail(SV_ERR_INVALID_ARG, "ws must be a 256-byte aligned workspace of at least %lld bytes", kHeaderBytes);
  g.rows = static_cast<int>(x.rows);
  g.nout = static_cast<int>(w.rows);
  g.runs = mx_runs(x.fmt, x.cols);
  g.nt = (g.nout + kN - 1) / kN;
  const long long tiles = mx_row_tiles(x.rows) * g.nt;
  if (tiles > 0x3fffffffLL) return pfail(SV_ERR_UNSUPPORTED, "too many output tiles");
  g.tiles = static_cast<int>(tiles);
  int sms = 0;
  MXP_TRY(mx_device(&sms));
  Ops op = outs;
  op.sa = static_cast<const uint8_t*>(x.scales);
  op.sb = static_cast<const uint8_t*>(w.scales);
  op.ga = x.gscale;
  op.gb = w.gscale;
  const uint64_t bytes = static_cast<uint64_t>(x.fmt == SV_MXFP8 ? x.cols : x.cols / 2);
  CUtensorMap am, bm;
  MXP_TRY(encode_bytes_2d(&am, x.codes, bytes, static_cast<uint64_t>(x.rows), kM));
  MXP_TRY(encode_bytes_2d(&bm, w.codes, bytes, static_cast<uint64_t>(w.rows), kN));
  if (x.fmt == SV_MXFP8) return run<SV_MXFP8, kQKV>(am, bm, op, g, ws, sms, st);
  if (x.fmt == SV_MXFP4) return run<SV_MXFP4, kQKV>(am, bm, op, g, ws, sms, st);
  return run<SV_NVFP4, kQKV>(am, bm, op, g, ws, sms, st);
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
