// Microscaled operands, sm_100a: quantisation to block-scaled 8- and 4-bit floating point, the way
// back, the tensor scale, and the root-mean-square norm whose output is quantised in the same pass.
//
// All of it is bound by HBM: a pass reads each input once and writes codes and scales once. A thread
// holds 16 consecutive columns in registers (one SV_NVFP4 block, half an MX block whose other half
// sits in the neighbouring lane), so a block's largest magnitude takes at most one shuffle.
//
// Rounding. An element is x / s (or x / (s g)) rounded once, to nearest even. For the MX formats s is
// a power of two and the product x * 2^-k is exact, so the conversion instruction rounds correctly.
// For SV_NVFP4 the quotient q = x * fp32(1 / fp32(s g)) is off by at most about 2^-22 relative; when
// q (1 - 2^-20) and q (1 + 2^-20) convert to the same code no border lies between them and that code is
// the answer. Otherwise (bf16 inputs and a measured g do lie on borders) |x| is compared with the
// exact borders t * s * g, products of 3 + 4 + 24 bits, in fp64. The scale's quotient a / (6 g) is
// taken in fp64 (its distance from a border of e4m3 is at least 2^-33 relative, unless it lies on it)
// and goes to fp32 towards zero with the lost bits or-ed into the lowest one, so that the second
// rounding, to e4m3, gives what a single one would.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdio>
#include <mutex>

#include "../../include/svlinattn.h"
#include "sv_internal.h"
#include "sv_ptx.cuh"

namespace sv {
namespace {

constexpr int kGroup = 16;       // columns per thread
constexpr int kMxThreads = 256;  // threads of the quantising and dequantising kernels

// ---- loads and stores of 16 columns, in two 8-column halves (16-byte aligned) ----
template <typename T>
struct Half;
template <>
struct Half<__nv_bfloat16> {
  static __device__ __forceinline__ void load(const __nv_bfloat16* p, float* f) {
    const uint4 r = *reinterpret_cast<const uint4*>(p);
    const uint32_t u[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(u[i] << 16);
      f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ void store(__nv_bfloat16* p, const float* f) {
    uint4 r;
    r.x = pack_bf16x2(f[0], f[1]);
    r.y = pack_bf16x2(f[2], f[3]);
    r.z = pack_bf16x2(f[4], f[5]);
    r.w = pack_bf16x2(f[6], f[7]);
    *reinterpret_cast<uint4*>(p) = r;
  }
  static __device__ __forceinline__ float round(float f) { return __bfloat162float(__float2bfloat16_rn(f)); }
};
template <>
struct Half<float> {
  static __device__ __forceinline__ void load(const float* p, float* f) {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
  }
  static __device__ __forceinline__ void store(float* p, const float* f) {
    reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
  }
  static __device__ __forceinline__ float round(float f) { return f; }
};

// ---- conversions ----
// eight values to eight e2m1 codes, the first in the lowest four bits
__device__ __forceinline__ uint32_t cvt_e2m1x8(const float* f) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}\n"
      : "=r"(r)
      : "f"(f[0]), "f"(f[1]), "f"(f[2]), "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7]));
  return r;
}
__device__ __forceinline__ uint32_t cvt_e4m3x4(const float* f) {
  uint32_t r;
  asm("{\n\t.reg .b16 a, b;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 b, %4, %3;\n\t"
      "mov.b32 %0, {a, b};\n\t}\n"
      : "=r"(r)
      : "f"(f[0]), "f"(f[1]), "f"(f[2]), "f"(f[3]));
  return r;
}
// four e4m3 codes to fp32 (exact)
__device__ __forceinline__ void e4m3x4_to_f32(uint32_t v, float* f) {
  uint32_t lo, hi;
  asm("{\n\t.reg .b16 a, b;\n\t"
      "mov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}\n"
      : "=r"(lo), "=r"(hi)
      : "r"(v));
  const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&lo));
  const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&hi));
  f[0] = a.x, f[1] = a.y, f[2] = b.x, f[3] = b.y;
}
// eight e2m1 codes to fp32 (exact)
__device__ __forceinline__ void e2m1x8_to_f32(uint32_t v, float* f) {
  uint32_t h[4];
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}\n"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(v));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
    f[2 * i] = a.x, f[2 * i + 1] = a.y;
  }
}
__device__ __forceinline__ float e4m3_to_f32(uint32_t b) {
  float f[4];
  e4m3x4_to_f32(b & 0xffu, f);
  return f[0];
}
// 2^k for k in [-127, 127]
__device__ __forceinline__ float pow2f_bits(int k) {
  return __uint_as_float(k > -127 ? static_cast<uint32_t>(k + 127) << 23 : 1u << 22);
}

constexpr uint32_t kInfBits = 0x7f800000u;

// the bits of max |f_i|; infinities and NaN compare above every finite value
__device__ __forceinline__ uint32_t amax_bits(const float (&f)[kGroup]) {
  uint32_t a = 0;
#pragma unroll
  for (int i = 0; i < kGroup; ++i) a = max(a, __float_as_uint(f[i]) & 0x7fffffffu);
  return a;
}

// Eight elements of SV_NVFP4 by the exact borders: code of |x| = how many borders t * d lie below it,
// a border itself going to the even code.
__device__ __forceinline__ uint32_t e2m1_exact(float x, double d) {
  const double a = fabs(static_cast<double>(x));
  uint32_t c = a > 0.25 * d;
  c += a >= 0.75 * d;
  c += a > 1.25 * d;
  c += a >= 1.75 * d;
  c += a > 2.5 * d;
  c += a >= 3.5 * d;
  c += a > 5.0 * d;
  return x < 0.f ? c | 8u : c;
}
// by value, out of line: the rare path takes no registers or local memory from the common one
static __device__ __noinline__ uint32_t e2m1x8_exact(float f0, float f1, float f2, float f3, float f4, float f5, float f6,
                                                     float f7, double d) {
  return e2m1_exact(f0, d) | e2m1_exact(f1, d) << 4 | e2m1_exact(f2, d) << 8 | e2m1_exact(f3, d) << 12 |
         e2m1_exact(f4, d) << 16 | e2m1_exact(f5, d) << 20 | e2m1_exact(f6, d) << 24 | e2m1_exact(f7, d) << 28;
}

// One thread's 16 columns to codes (SV_MXFP8: four words, else two) and the block's scale byte.
// Every lane of the warp calls it (the MX formats pair lanes 2i and 2i + 1).
template <int FMT>
__device__ __forceinline__ uint32_t quantise16(const float (&f)[kGroup], float g, uint32_t (&code)[4]) {
  uint32_t ab = amax_bits(f);
  if (FMT == SV_NVFP4) {
    if (ab >= kInfBits || !(fabsf(g) < __uint_as_float(kInfBits))) {
      code[0] = code[1] = 0u;
      return 0x7fu;  // NaN
    }
    const double gd = static_cast<double>(g);
    const double ratio = static_cast<double>(__uint_as_float(ab)) / (6.0 * gd);
    float rz = __double2float_rz(fmin(ratio, 448.0));
    if (static_cast<double>(rz) != fmin(ratio, 448.0)) rz = __uint_as_float(__float_as_uint(rz) | 1u);
    float z4[4] = {rz, 0.f, 0.f, 0.f};
    const uint32_t sb = cvt_e4m3x4(z4) & 0xffu;
    const float s = e4m3_to_f32(sb);
    const float d = s * g;
    if (!(s > 0.f) || !(gd > 0.0)) {
      code[0] = code[1] = 0u;
      return sb;
    }
    const bool fits = d > 0x1p-100f && d < 0x1p100f;  // the fp32 quotient keeps its accuracy
    const float r = fits ? 1.0f / d : 0.f;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float lo[8], hi[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float q = f[8 * h + i] * r;
        lo[i] = q * (1.0f - 0x1p-20f);
        hi[i] = q * (1.0f + 0x1p-20f);
      }
      const uint32_t c = cvt_e2m1x8(lo);
      code[h] = c;
      if (!fits || c != cvt_e2m1x8(hi)) {
        const float* v = f + 8 * h;
        code[h] = e2m1x8_exact(v[0], v[1], v[2], v[3], v[4], v[5], v[6], v[7], static_cast<double>(s) * gd);
      }
    }
    return sb;
  } else {
    ab = max(ab, __shfl_xor_sync(0xffffffffu, ab, 1));
    // a = m 2^k, 1 <= m < 2; the largest element is 1.75 * 2^8 (e4m3) or 1.5 * 2^2 (e2m1)
    const uint32_t top = FMT == SV_MXFP8 ? 0x600000u : 0x400000u;
    int k = static_cast<int>(ab >> 23) - 127 - (FMT == SV_MXFP8 ? 8 : 2) + ((ab & 0x7fffffu) > top ? 1 : 0);
    k = max(k, -127);
    const bool bad = ab >= kInfBits;
    const float r = bad ? 0.f : pow2f_bits(-k);
    float q[kGroup];
#pragma unroll
    for (int i = 0; i < kGroup; ++i) q[i] = f[i] * r;
    if (FMT == SV_MXFP8) {
#pragma unroll
      for (int i = 0; i < 4; ++i) code[i] = bad ? 0u : cvt_e4m3x4(q + 4 * i);
    } else {
      code[0] = bad ? 0u : cvt_e2m1x8(q);
      code[1] = bad ? 0u : cvt_e2m1x8(q + 8);
    }
    return bad ? 0xffu : static_cast<uint32_t>(k + 127);
  }
}

// Where a scale sits (see the layout in the header); sp: padded blocks per row.
__device__ __forceinline__ size_t scale_at(size_t row, int blk, int sp) {
  return (row >> 7) * (static_cast<size_t>(sp) << 7) + (static_cast<size_t>(blk >> 2) << 9) + (row & 31) * 16 +
         ((row >> 5) & 3) * 4 + (blk & 3);
}

// Writes one thread's codes (when `live`: it holds real columns) and, when `in` (it holds a place of the
// scale tiles), its scale byte, four blocks of a row to a 32-bit store: the padded groups of a row are a
// whole number of four-block words, so the lanes that hold a word's blocks belong to one row. Every
// lane of the warp calls it.
template <int FMT>
__device__ __forceinline__ void put16(uint8_t* codes, uint8_t* scales, size_t row, int grp, int cols, int sp, bool in,
                                      bool live, const uint32_t (&code)[4], uint32_t sb) {
  constexpr int kPer = FMT == SV_NVFP4 ? 1 : 2;  // groups per block
  const int blk = grp / kPer;
  uint32_t w = sb << (8 * (blk & 3));
  if (kPer == 1) w |= __shfl_xor_sync(0xffffffffu, w, 1);
  w |= __shfl_xor_sync(0xffffffffu, w, 2);
  if (kPer == 2) w |= __shfl_xor_sync(0xffffffffu, w, 4);
  if (in && grp % (4 * kPer) == 0) *reinterpret_cast<uint32_t*>(scales + scale_at(row, blk, sp)) = w;
  if (!live) return;
  if (FMT == SV_MXFP8)
    *reinterpret_cast<uint4*>(codes + row * cols + static_cast<size_t>(grp) * 16) =
        make_uint4(code[0], code[1], code[2], code[3]);
  else
    *reinterpret_cast<uint2*>(codes + row * (cols / 2) + static_cast<size_t>(grp) * 8) = make_uint2(code[0], code[1]);
}

// One thread per (padded row, padded group): rows rounded up to 128 and gp groups per row (a multiple
// of 8), so every warp is full and the places of the scale tiles that hold no block are written too.
template <int FMT, typename T>
__global__ void __launch_bounds__(kMxThreads) quantize_kernel(const T* __restrict__ x, int H, int N, int D, uint32_t rows,
                                                              int cols, int gp, int sp, const float* gscale,
                                                              uint8_t* codes, uint8_t* scales) {
  griddep_wait();
  if (threadIdx.x == 0) griddep_launch_dependents();
  const size_t idx = static_cast<size_t>(blockIdx.x) * kMxThreads + threadIdx.x;
  const uint32_t row = static_cast<uint32_t>(idx / static_cast<uint32_t>(gp));
  const int grp = static_cast<int>(idx - static_cast<size_t>(row) * gp);
  const bool live = row < rows && grp * kGroup < cols;
  float f[kGroup];
#pragma unroll
  for (int i = 0; i < kGroup; ++i) f[i] = 0.f;
  if (live) {
    const int c = grp * kGroup;
    if (H == 1) {
      const T* p = x + static_cast<size_t>(row) * cols + c;
      Half<T>::load(p, f);
      Half<T>::load(p + 8, f + 8);
    } else {
      const uint32_t b = row / static_cast<uint32_t>(N), n = row - b * static_cast<uint32_t>(N);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int head = (c + 8 * h) / D, d = c + 8 * h - head * D;
        Half<T>::load(x + ((static_cast<size_t>(b) * H + head) * N + n) * D + d, f + 8 * h);
      }
    }
  }
  uint32_t code[4];
  uint32_t sb = quantise16<FMT>(f, FMT == SV_NVFP4 ? *gscale : 1.f, code);
  put16<FMT>(codes, scales, row, grp, cols, sp, true, live, code, live ? sb : 0u);
}

// One thread per (row, group): value = element * scale (exact in fp32) * g, rounded once to T.
template <int FMT, typename T>
__global__ void __launch_bounds__(kMxThreads) dequantize_kernel(const uint8_t* __restrict__ codes,
                                                                const uint8_t* __restrict__ scales, const float* gscale,
                                                                int cols, int sp, T* y, size_t total) {
  griddep_wait();
  if (threadIdx.x == 0) griddep_launch_dependents();
  const size_t idx = static_cast<size_t>(blockIdx.x) * kMxThreads + threadIdx.x;
  if (idx >= total) return;
  const uint32_t gpr = static_cast<uint32_t>(cols) / kGroup;
  const uint32_t row = static_cast<uint32_t>(idx / gpr);
  const int grp = static_cast<int>(idx - static_cast<size_t>(row) * gpr);
  const uint32_t sb = scales[scale_at(row, FMT == SV_NVFP4 ? grp : grp >> 1, sp)];
  float f[kGroup];
  if (FMT == SV_MXFP8) {
    const uint4 c = *reinterpret_cast<const uint4*>(codes + idx * 16);
    e4m3x4_to_f32(c.x, f);
    e4m3x4_to_f32(c.y, f + 4);
    e4m3x4_to_f32(c.z, f + 8);
    e4m3x4_to_f32(c.w, f + 12);
  } else {
    const uint2 c = *reinterpret_cast<const uint2*>(codes + idx * 8);
    e2m1x8_to_f32(c.x, f);
    e2m1x8_to_f32(c.y, f + 8);
  }
  float s, g = 1.f;
  if (FMT == SV_NVFP4) {
    s = e4m3_to_f32(sb);
    g = *gscale;
  } else {
    s = sb == 255u ? __uint_as_float(0x7fffffffu) : pow2f_bits(static_cast<int>(sb) - 127);
  }
#pragma unroll
  for (int i = 0; i < kGroup; ++i) f[i] = f[i] * s * g;
  Half<T>::store(y + idx * kGroup, f);
  Half<T>::store(y + idx * kGroup + 8, f + 8);
}

// *g = max over the grid of max |x_i| / 2688. The quotient of non-negative values grows with |x|, so
// the maximum of the blocks' quotients (as integers: the bits of non-negative floats are ordered, NaN
// above all) is the quotient of the maximum, in any order. *g is zeroed before the launch.
template <typename T>
__global__ void __launch_bounds__(kMxThreads) global_scale_kernel(const T* __restrict__ x, size_t n, float* g) {
  uint32_t a = 0;
  const size_t step = static_cast<size_t>(gridDim.x) * kMxThreads * 8;
  for (size_t i = (static_cast<size_t>(blockIdx.x) * kMxThreads + threadIdx.x) * 8; i < n; i += step) {
    float f[8];
    if (i + 8 <= n) {
      Half<T>::load(x + i, f);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = i + j < n ? static_cast<float>(x[i + j]) : 0.f;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) a = max(a, __float_as_uint(f[j]) & 0x7fffffffu);
  }
  a = __reduce_max_sync(0xffffffffu, a);
  __shared__ uint32_t part[kMxThreads / 32];
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = a;
  __syncthreads();
  if (threadIdx.x == 0) {
#pragma unroll
    for (int w = 1; w < kMxThreads / 32; ++w) a = max(a, part[w]);
    atomicMax(reinterpret_cast<unsigned int*>(g), __float_as_uint(__uint_as_float(a) / 2688.0f) & 0x7fffffffu);
  }
}

// ---- norm ----
// A team of blockDim.x threads takes one row (blockDim.y rows per block; more than one only with
// one-warp teams). Thread t holds the groups i * blockDim.x + t, i < G, in registers from the load to
// the store, so x and the residual are read once. Squares are summed in fp64: then 1 / sqrt(mean + eps),
// rounded to fp32, does not depend on how the row is split over threads (but for one case in about 1e8),
// and quantised outputs, where a last-bit difference can move an element by a whole step, do not either.
constexpr int kPlain = -1;
constexpr int kMaxTeam = 512;

__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

template <int FMT, typename T, int G>
__global__ void __launch_bounds__(G == 1 || G == 4 ? kMaxTeam : 256) rmsnorm_kernel(const T* x, const T* res, T* h_out, const float* __restrict__ w,
                                                           size_t rows, size_t rows_padded, int cols, int gp, int sp,
                                                           float eps, T* y, const float* gscale, uint8_t* codes,
                                                           uint8_t* scales) {
  __shared__ double part[kMaxTeam / 32];
  griddep_wait();
  if (threadIdx.x == 0 && threadIdx.y == 0) griddep_launch_dependents();
  const size_t row = static_cast<size_t>(blockIdx.x) * blockDim.y + threadIdx.y;
  if (row >= rows_padded) return;  // whole warps: with blockDim.y == 1 the whole block
  const int team = blockDim.x;
  const bool real = row < rows;
  float f[G][kGroup];
  double sum = 0.0;
#pragma unroll
  for (int i = 0; i < G; ++i) {
    const int c = (i * team + static_cast<int>(threadIdx.x)) * kGroup;
#pragma unroll
    for (int j = 0; j < kGroup; ++j) f[i][j] = 0.f;
    if (!real) continue;
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      const int c8 = c + 8 * hf;
      if (c8 >= cols) continue;
      float* v = f[i] + 8 * hf;
      const size_t at = row * cols + c8;
      Half<T>::load(x + at, v);
      if (res != nullptr) {
        float r[8];
        Half<T>::load(res + at, r);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = Half<T>::round(v[j] + r[j]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < G; ++i)
#pragma unroll
    for (int j = 0; j < kGroup; ++j) {
      const double d = f[i][j];
      sum = fma(d, d, sum);
    }
  sum = warp_sum(sum);
  if (team > 32) {
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = sum;
    __syncthreads();
    sum = 0.0;
    for (int k = 0; k < team / 32; ++k) sum += part[k];
  }
  const float rstd = static_cast<float>(1.0 / sqrt(sum / cols + static_cast<double>(eps)));
  const float g = FMT == SV_NVFP4 ? *gscale : 1.f;
#pragma unroll
  for (int i = 0; i < G; ++i) {
    const int grp = i * team + static_cast<int>(threadIdx.x);
    const int c = grp * kGroup;
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      const int c8 = c + 8 * hf;
      if (!real || c8 >= cols) continue;
      float* v = f[i] + 8 * hf;
      const size_t at = row * cols + c8;
      if (h_out != nullptr) Half<T>::store(h_out + at, v);
      const float4 w0 = __ldg(reinterpret_cast<const float4*>(w + c8)), w1 = __ldg(reinterpret_cast<const float4*>(w + c8) + 1);
      const float ww[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = v[j] * rstd * ww[j];
      if (FMT == kPlain) Half<T>::store(y + at, v);
    }
    if (FMT != kPlain) {
      constexpr int F = FMT == kPlain ? 0 : FMT;
      const bool live = real && c < cols;
      uint32_t code[4];
      const uint32_t sb = quantise16<F>(f[i], g, code);
      // the team may cover more groups than the padded row has
      put16<F>(codes, scales, row, grp, cols, sp, grp < gp, live, code, live ? sb : 0u);
    }
  }
}

// ---- host side ----
sv_status mfail(sv_status st, const char* fmt, long long a = 0, long long b = 0) {
  char msg[256];
  snprintf(msg, sizeof(msg), fmt, a, b);
  return set_last_error(st, msg);
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0u; }

cudaLaunchConfig_t pdl_config(dim3 grid, dim3 block, cudaStream_t st, cudaLaunchAttribute* at) {
  at->id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at->val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.stream = st;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cfg;
}

sv_status launched(cudaError_t e, const char* what) {
  if (e == cudaSuccess) return SV_OK;
  char msg[200];
  snprintf(msg, sizeof(msg), "%s launch: %s", what, cudaGetErrorString(e));
  return set_last_error(SV_ERR_CUDA, msg);
}

sv_status check_dt(sv_dtype dt) {
  return dt == SV_BF16 || dt == SV_F32 ? SV_OK : mfail(SV_ERR_UNSUPPORTED, "dtype is not SV_BF16 or SV_F32");
}

sv_status mx_size(sv_mx_format fmt, long long rows, int cols) {
  if (fmt != SV_MXFP8 && fmt != SV_MXFP4 && fmt != SV_NVFP4)
    return mfail(SV_ERR_UNSUPPORTED, "unknown microscaled format %lld", static_cast<long long>(fmt));
  if (rows < 1 || rows > kMxMaxRows) return mfail(SV_ERR_INVALID_ARG, "rows=%lld must be in [1, %lld]", rows, kMxMaxRows);
  if (cols < 32 || cols % 32 != 0) return mfail(SV_ERR_UNSUPPORTED, "cols=%lld must be a positive multiple of 32", cols);
  return SV_OK;
}

#define MX_TRY(x)                 \
  do {                            \
    const sv_status _s = (x);     \
    if (_s != SV_OK) return _s;   \
  } while (0)

template <int FMT, typename T>
sv_status run_quantize(const void* x, int H, int N, int D, const sv_mx& m, cudaStream_t st) {
  const int sp = mx_padded_blocks(m.fmt, m.cols);
  const int gp = sp * mx_block(m.fmt) / kGroup;
  const long long blocks = mx_row_tiles(m.rows) * 128 * gp / kMxThreads;
  if (blocks > 0x7fffffffLL) return mfail(SV_ERR_UNSUPPORTED, "too many elements");
  cudaLaunchAttribute at;
  const cudaLaunchConfig_t cfg = pdl_config(dim3(static_cast<unsigned>(blocks)), dim3(kMxThreads), st, &at);
  return launched(cudaLaunchKernelEx(&cfg, quantize_kernel<FMT, T>, static_cast<const T*>(x), H, N, D,
                                     static_cast<uint32_t>(m.rows), m.cols, gp, sp, m.gscale,
                                     static_cast<uint8_t*>(m.codes), static_cast<uint8_t*>(m.scales)),
                  "quantisation");
}

template <int FMT, typename T>
sv_status run_dequantize(const sv_mx& m, void* y, cudaStream_t st) {
  const size_t total = static_cast<size_t>(m.rows) * (m.cols / kGroup);
  const size_t blocks = (total + kMxThreads - 1) / kMxThreads;
  if (blocks > 0x7fffffffull) return mfail(SV_ERR_UNSUPPORTED, "too many elements");
  cudaLaunchAttribute at;
  const cudaLaunchConfig_t cfg = pdl_config(dim3(static_cast<unsigned>(blocks)), dim3(kMxThreads), st, &at);
  return launched(cudaLaunchKernelEx(&cfg, dequantize_kernel<FMT, T>, static_cast<const uint8_t*>(m.codes),
                                     static_cast<const uint8_t*>(m.scales), m.gscale, m.cols,
                                     mx_padded_blocks(m.fmt, m.cols), static_cast<T*>(y), total),
                  "dequantisation");
}

struct NormArgs {
  const void *x, *res;
  void* h;
  const float* w;
  long long rows;
  int C;
  float eps;
  void* y;
  const sv_mx* q;
};

template <int FMT, typename T, int G>
sv_status launch_norm(const NormArgs& a, int team, int gp, int sp, cudaStream_t st) {
  const int per_block = team == 32 ? 8 : 1;
  const long long rows_padded = a.q != nullptr ? mx_row_tiles(a.rows) * 128 : a.rows;
  const long long blocks = (rows_padded + per_block - 1) / per_block;
  cudaLaunchAttribute at;
  const cudaLaunchConfig_t cfg = pdl_config(dim3(static_cast<unsigned>(blocks)), dim3(team, per_block), st, &at);
  return launched(
      cudaLaunchKernelEx(&cfg, rmsnorm_kernel<FMT, T, G>, static_cast<const T*>(a.x), static_cast<const T*>(a.res),
                         static_cast<T*>(a.h), a.w, static_cast<size_t>(a.rows), static_cast<size_t>(rows_padded), a.C,
                         gp, sp, a.eps, static_cast<T*>(a.y), a.q != nullptr ? a.q->gscale : nullptr,
                         a.q != nullptr ? static_cast<uint8_t*>(a.q->codes) : nullptr,
                         a.q != nullptr ? static_cast<uint8_t*>(a.q->scales) : nullptr),
      "norm");
}

template <int FMT, typename T>
sv_status run_norm(const NormArgs& a, cudaStream_t st) {
  const int sp = a.q != nullptr ? mx_padded_blocks(a.q->fmt, a.C) : 0;
  const int gp = a.q != nullptr ? sp * mx_block(a.q->fmt) / kGroup : (a.C + kGroup - 1) / kGroup;
  // one warp to a row while its groups fit five to a lane; a whole block beyond that
  if (gp <= 32) return launch_norm<FMT, T, 1>(a, 32, gp, sp, st);
  if (gp <= 64) return launch_norm<FMT, T, 2>(a, 32, gp, sp, st);
  if (gp <= 160) return launch_norm<FMT, T, 5>(a, 32, gp, sp, st);
  const int team = gp <= 512 ? (gp + 31) / 32 * 32 : 512;
  if (gp <= 512) return launch_norm<FMT, T, 1>(a, team, gp, sp, st);
  return launch_norm<FMT, T, 4>(a, team, gp, sp, st);
}

// Calls f<FMT, T>(args...) for a runtime format and type.
#define MX_DISPATCH(fmt, dt, f, ...)                                                             \
  do {                                                                                           \
    if ((dt) == SV_BF16) {                                                                       \
      if ((fmt) == SV_MXFP8) return f<SV_MXFP8, __nv_bfloat16>(__VA_ARGS__);                     \
      if ((fmt) == SV_MXFP4) return f<SV_MXFP4, __nv_bfloat16>(__VA_ARGS__);                     \
      return f<SV_NVFP4, __nv_bfloat16>(__VA_ARGS__);                                            \
    }                                                                                            \
    if ((fmt) == SV_MXFP8) return f<SV_MXFP8, float>(__VA_ARGS__);                               \
    if ((fmt) == SV_MXFP4) return f<SV_MXFP4, float>(__VA_ARGS__);                               \
    return f<SV_NVFP4, float>(__VA_ARGS__);                                                      \
  } while (0)

}  // namespace

sv_status check_mx(const sv_mx* m, const char* name) {
  char msg[200];
  if (m == nullptr) {
    snprintf(msg, sizeof(msg), "%s is NULL", name);
    return set_last_error(SV_ERR_INVALID_ARG, msg);
  }
  MX_TRY(mx_size(m->fmt, m->rows, m->cols));
  if (m->codes == nullptr || m->scales == nullptr || !aligned(m->codes, 16) || !aligned(m->scales, 16)) {
    snprintf(msg, sizeof(msg), "%s: codes and scales must be non-NULL and 16-byte aligned", name);
    return set_last_error(SV_ERR_INVALID_ARG, msg);
  }
  if (m->fmt == SV_NVFP4 ? m->gscale == nullptr || !aligned(m->gscale, 4) : m->gscale != nullptr) {
    snprintf(msg, sizeof(msg), "%s: gscale must be a 4-byte aligned pointer for SV_NVFP4 and NULL for the other formats", name);
    return set_last_error(SV_ERR_INVALID_ARG, msg);
  }
  return SV_OK;
}

sv_status mx_device(int* sms) {
  constexpr int kMaxDev = 64;
  static std::mutex mu;
  static int count[kMaxDev] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return mfail(SV_ERR_CUDA, "cannot query the current device");
  if (dev < 0 || dev >= kMaxDev) return mfail(SV_ERR_UNSUPPORTED, "device index %lld out of range", dev);
  std::lock_guard<std::mutex> lock(mu);
  if (count[dev] == 0) {
    int n = 0, major = 0, minor = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess)
      return mfail(SV_ERR_CUDA, "cannot query the current device");
    if (major != 10 || minor != 0)
      return mfail(SV_ERR_UNSUPPORTED, "device is sm_%lld%lld; built for sm_100a", major, minor);
    count[dev] = n;
  }
  *sms = count[dev];
  return SV_OK;
}

}  // namespace sv

extern "C" size_t sv_mx_code_bytes(sv_mx_format fmt, long long rows, int cols) {
  if (sv::mx_size(fmt, rows, cols) != SV_OK) return 0;
  return static_cast<size_t>(rows) * (fmt == SV_MXFP8 ? cols : cols / 2);
}

extern "C" size_t sv_mx_scale_bytes(sv_mx_format fmt, long long rows, int cols) {
  if (sv::mx_size(fmt, rows, cols) != SV_OK) return 0;
  return static_cast<size_t>(sv::mx_row_tiles(rows)) * 128 * sv::mx_padded_blocks(fmt, cols);
}

extern "C" sv_status sv_mx_global_scale(const void* x, long long n, sv_dtype dt, float* g, sv_stream_t stream) {
  using namespace sv;
  MX_TRY(check_dt(dt));
  if (n < 1) return mfail(SV_ERR_INVALID_ARG, "n=%lld must be >= 1", n);
  if (x == nullptr || !aligned(x, 16)) return mfail(SV_ERR_INVALID_ARG, "x must be non-NULL and 16-byte aligned");
  if (g == nullptr || !aligned(g, 4)) return mfail(SV_ERR_INVALID_ARG, "g must be non-NULL and 4-byte aligned");
  int sms = 0;
  MX_TRY(mx_device(&sms));
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = cudaMemsetAsync(g, 0, sizeof(float), st);
  if (e != cudaSuccess) return launched(e, "tensor scale");
  const long long per = static_cast<long long>(kMxThreads) * 8;
  const long long want = (n + per - 1) / per;
  const unsigned blocks = static_cast<unsigned>(want < 8ll * sms ? want : 8ll * sms);
  if (dt == SV_BF16)
    global_scale_kernel<<<blocks, kMxThreads, 0, st>>>(static_cast<const __nv_bfloat16*>(x), static_cast<size_t>(n), g);
  else
    global_scale_kernel<<<blocks, kMxThreads, 0, st>>>(static_cast<const float*>(x), static_cast<size_t>(n), g);
  return launched(cudaGetLastError(), "tensor scale");
}

extern "C" sv_status sv_mx_quantize(const void* x, int B, int H, int N, int D, sv_dtype dt, const sv_mx* out,
                                    sv_stream_t stream) {
  using namespace sv;
  MX_TRY(check_dt(dt));
  MX_TRY(check_mx(out, "out"));
  if (B < 1 || H < 1 || N < 1 || D < 1) return mfail(SV_ERR_INVALID_ARG, "B, H, N and D must be >= 1");
  if (D % 8 != 0) return mfail(SV_ERR_UNSUPPORTED, "D=%lld must be a multiple of 8", D);
  if (static_cast<long long>(B) * N != out->rows || static_cast<long long>(H) * D != out->cols)
    return mfail(SV_ERR_INVALID_ARG, "out must have B * N = %lld rows and H * D = %lld columns",
                 static_cast<long long>(B) * N, static_cast<long long>(H) * D);
  if (x == nullptr || !aligned(x, 16)) return mfail(SV_ERR_INVALID_ARG, "x must be non-NULL and 16-byte aligned");
  int sms = 0;
  MX_TRY(mx_device(&sms));
  MX_DISPATCH(out->fmt, dt, run_quantize, x, H, N, D, *out, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" sv_status sv_mx_dequantize(const sv_mx* in, void* y, sv_dtype dt, sv_stream_t stream) {
  using namespace sv;
  MX_TRY(check_dt(dt));
  MX_TRY(check_mx(in, "in"));
  if (y == nullptr || !aligned(y, 16)) return mfail(SV_ERR_INVALID_ARG, "y must be non-NULL and 16-byte aligned");
  int sms = 0;
  MX_TRY(mx_device(&sms));
  MX_DISPATCH(in->fmt, dt, run_dequantize, *in, y, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" sv_status sv_rmsnorm(const void* x, const void* residual, void* h, const float* w, long long rows, int C,
                                sv_dtype dt, float eps, void* y, const sv_mx* yq, sv_stream_t stream) {
  using namespace sv;
  MX_TRY(check_dt(dt));
  if (rows < 1 || rows > kMxMaxRows) return mfail(SV_ERR_INVALID_ARG, "rows=%lld must be in [1, %lld]", rows, kMxMaxRows);
  if (C < 8 || C > 32768 || C % 8 != 0)
    return mfail(SV_ERR_UNSUPPORTED, "C=%lld must be a multiple of 8 in [8, 32768]", C);
  if (!(eps >= 0.f) || !std::isfinite(eps)) return mfail(SV_ERR_INVALID_ARG, "eps must be finite and >= 0");
  if (x == nullptr || w == nullptr) return mfail(SV_ERR_INVALID_ARG, "x or w is NULL");
  if (residual != nullptr && h == nullptr) return mfail(SV_ERR_INVALID_ARG, "h is NULL, but there is a residual");
  if ((y == nullptr) == (yq == nullptr)) return mfail(SV_ERR_INVALID_ARG, "exactly one of y and yq must be given");
  if (y != nullptr && y == h) return mfail(SV_ERR_INVALID_ARG, "y and h must not be the same buffer");
  if (!aligned(x, 16) || !aligned(residual, 16) || !aligned(h, 16) || !aligned(w, 16) || !aligned(y, 16))
    return mfail(SV_ERR_INVALID_ARG, "x, residual, h, w and y must be 16-byte aligned");
  if (yq != nullptr) {
    MX_TRY(check_mx(yq, "yq"));
    if (yq->rows != rows || yq->cols != C)
      return mfail(SV_ERR_INVALID_ARG, "yq must have %lld rows and %lld columns", rows, C);
  }
  int sms = 0;
  MX_TRY(mx_device(&sms));
  // without a residual h is x: nothing to write where they are the same buffer
  const NormArgs a{x, residual, residual == nullptr && h == x ? nullptr : h, w, rows, C, eps, y, yq};
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (yq == nullptr)
    return dt == SV_BF16 ? run_norm<kPlain, __nv_bfloat16>(a, st) : run_norm<kPlain, float>(a, st);
  MX_DISPATCH(yq->fmt, dt, run_norm, a, st);
}
