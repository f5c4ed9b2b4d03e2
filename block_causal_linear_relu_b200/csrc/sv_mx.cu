// Microscaled operands, sm_100a: quantisation to block-scaled 8- and 4-bit floating point, the way
// back, the tensor scale, and the root-mean-square norm whose output is quantised in the same pass.
//
// A pass reads each input once and writes codes and scales once. HBM bounds all but the quantisation, where
// the issue of instructions does as much, most in SV_NVFP4. Where a thread quantises it holds 16 consecutive columns, one
// SV_NVFP4 block or half an MX block whose other half is in the neighbouring lane, so that a block's scale
// is worked out once or twice; elsewhere it holds eight (16 bytes of bf16: coalesced loads and stores).
//
// Rounding. An element is x / s (or x / (s g)) rounded once, to nearest even. For the MX formats s is
// a power of two and the product x * 2^-k is exact, so the conversion instruction rounds correctly.
// For SV_NVFP4 the fp32 quotients q (of an element, x * fp32(1 / fp32(s g)), and of the scale, a * fp32(1 /
// fp32(6 g))) are off by at most about 2^-22 relative; when q (1 - 2^-20) and q (1 + 2^-20) convert to the
// same code no border lies between them and it is the answer. Otherwise (bf16 inputs and a
// measured g do lie on borders) it is found exactly: |x| is compared with the borders t * s * g, products
// of 3 + 4 + 24 bits, in fp64; the scale's quotient a / (6 g) is taken in fp64 (its distance from a border
// of e4m3 is at least 2^-33 relative, unless it lies on it) and goes to fp32 towards zero with the lost
// bits or-ed into the lowest one, so that the second rounding, to e4m3, gives what a single one would.
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

constexpr int kOct = 8;           // columns per lane and step: 16 bytes of bf16 (norm and values)
constexpr int kGroup = 16;        // columns per lane and step where they are quantised
constexpr int kMxThreads = 256;  // threads of the quantising and dequantising kernels
// steps per thread of the second, all loaded before one is used; the first takes two or four (below)
constexpr int kValueUnroll = 4;

// two products in one instruction
__device__ __forceinline__ void mul2(float& d0, float& d1, float a0, float a1, float b0, float b1) {
  asm("{\n\t.reg .b64 a, b, d;\n\t"
      "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "mul.rn.f32x2 d, a, b;\n\t"
      "mov.b64 {%0, %1}, d;\n\t}\n"
      : "=f"(d0), "=f"(d1)
      : "f"(a0), "f"(a1), "f"(b0), "f"(b1));
}
template <int E>
__device__ __forceinline__ void scaled(float (&d)[E], const float* v, float r) {
#pragma unroll
  for (int i = 0; i < E; i += 2) mul2(d[i], d[i + 1], v[i], v[i + 1], r, r);
}

// ---- eight columns as loaded (16-byte aligned) ----
template <typename T>
struct Oct;
template <>
struct Oct<__nv_bfloat16> {
  uint4 r;
  __device__ __forceinline__ void zero() { r = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { r = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void store(__nv_bfloat16* p) const { *reinterpret_cast<uint4*>(p) = r; }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    const uint32_t u[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(u[i] << 16);
      f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
  }
  // The sum, rounded to bf16: the instruction rounds the exact sum once. (So does an addition in fp32 that
  // is rounded afterwards: where the fp32 sum is inexact, one of the two is below 2^-16 of the other.)
  __device__ __forceinline__ void add(const Oct& q) {
    r.x = add2(r.x, q.r.x), r.y = add2(r.y, q.r.y), r.z = add2(r.z, q.r.z), r.w = add2(r.w, q.r.w);
  }
  static __device__ __forceinline__ uint32_t add2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
  }
  // times a power of two
  __device__ __forceinline__ void scale(float f) {
    const uint32_t f2 = pack_bf16x2(f, f);
    r.x = mul2(r.x, f2), r.y = mul2(r.y, f2), r.z = mul2(r.z, f2), r.w = mul2(r.w, f2);
  }
  static __device__ __forceinline__ uint32_t mul2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
  }
  __device__ __forceinline__ void set(const float (&f)[8]) {  // rounded
    r = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
  }
};
template <>
struct Oct<float> {
  float4 a, b;
  __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void load(const float* p) {
    a = reinterpret_cast<const float4*>(p)[0];
    b = reinterpret_cast<const float4*>(p)[1];
  }
  __device__ __forceinline__ void store(float* p) const {
    reinterpret_cast<float4*>(p)[0] = a;
    reinterpret_cast<float4*>(p)[1] = b;
  }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
  }
  __device__ __forceinline__ void add(const Oct& q) {
    a.x += q.a.x, a.y += q.a.y, a.z += q.a.z, a.w += q.a.w;
    b.x += q.b.x, b.y += q.b.y, b.z += q.b.z, b.w += q.b.w;
  }
  __device__ __forceinline__ void scale(float f) {
    a.x *= f, a.y *= f, a.z *= f, a.w *= f;
    b.x *= f, b.y *= f, b.z *= f, b.w *= f;
  }
  __device__ __forceinline__ void set(const float (&f)[8]) {
    a = make_float4(f[0], f[1], f[2], f[3]);
    b = make_float4(f[4], f[5], f[6], f[7]);
  }
};

// E columns (8 or 16) as loaded
template <typename T, int E>
struct Cols {
  Oct<T> o[E / 8];
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < E / 8; ++i) o[i].zero();
  }
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < E / 8; ++i) o[i].load(p + 8 * i);
  }
  __device__ __forceinline__ void store(T* p) const {
#pragma unroll
    for (int i = 0; i < E / 8; ++i) o[i].store(p + 8 * i);
  }
  __device__ __forceinline__ void add(const Cols& q) {
#pragma unroll
    for (int i = 0; i < E / 8; ++i) o[i].add(q.o[i]);
  }
  __device__ __forceinline__ void scale(float f) {
#pragma unroll
    for (int i = 0; i < E / 8; ++i) o[i].scale(f);
  }
  __device__ __forceinline__ void get(float (&f)[E]) const {
#pragma unroll
    for (int i = 0; i < E / 8; ++i) o[i].get(*reinterpret_cast<float(*)[8]>(f + 8 * i));
  }
  __device__ __forceinline__ void set(const float (&f)[E]) {
#pragma unroll
    for (int i = 0; i < E / 8; ++i) o[i].set(*reinterpret_cast<const float(*)[8]>(f + 8 * i));
  }
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

// The scale of a block of SV_NVFP4 from the quotient in fp64 (see the top of the file).
static __device__ __noinline__ uint32_t e4m3_exact(float a, float g) {
  const double ratio = fmin(static_cast<double>(a) / (6.0 * static_cast<double>(g)), 448.0);
  float rz = __double2float_rz(ratio);
  if (static_cast<double>(rz) != ratio) rz = __uint_as_float(__float_as_uint(rz) | 1u);
  const float z4[4] = {rz, 0.f, 0.f, 0.f};
  return cvt_e4m3x4(z4) & 0xffu;
}

// What a thread needs to know about the tensor scale.
struct TensorScale {
  float g, inv6g;
  bool finite, fits;  // fits: the fp32 quotients keep their accuracy
};
__device__ __forceinline__ TensorScale tensor_scale(float g) {
  return {g, 1.0f / (6.0f * g), g - g == 0.0f, g > 0x1p-90f && g < 0x1p90f};
}

// The bits of max |f_i| over 16 columns, in fp32; infinities and NaN compare above every finite value.
__device__ __forceinline__ uint32_t amax16(const float (&f)[16]) {
  float a = 0.f;
#pragma unroll
  for (int i = 0; i < 16; i += 2) asm("max.NaN.f32 %0, %0, %1, %2;" : "+f"(a) : "f"(fabsf(f[i])), "f"(fabsf(f[i + 1])));
  return __float_as_uint(a);
}
// The same of 16 columns as loaded.
__device__ __forceinline__ uint32_t amax16(const Cols<__nv_bfloat16, 16>& v) {
  // pairs of 15-bit magnitudes, ordered as integers
  uint32_t a = 0;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    a = __vmaxu2(a, v.o[i].r.x & 0x7fff7fffu);
    a = __vmaxu2(a, v.o[i].r.y & 0x7fff7fffu);
    a = __vmaxu2(a, v.o[i].r.z & 0x7fff7fffu);
    a = __vmaxu2(a, v.o[i].r.w & 0x7fff7fffu);
  }
  return max(a << 16, a & 0xffff0000u);
}
__device__ __forceinline__ uint32_t amax16(const Cols<float, 16>& v) {
  float f[16];
  v.get(f);
  return amax16(f);
}

// One lane's 16 columns, whose largest magnitude has the bits amax, to codes (SV_MXFP8: four words, else
// two) and the block's scale byte: a block of SV_NVFP4, or half a block of the MX formats, whose lanes 2i
// and 2i + 1 both have it. kBf16: the values are bf16 numbers. Every lane of the warp calls it.
template <int FMT, bool kBf16>
__device__ __forceinline__ uint32_t quantise16(const float (&f)[16], uint32_t amax, const TensorScale& ts,
                                               uint32_t (&code)[4]) {
  uint32_t ab = amax;
  if (FMT == SV_NVFP4) {
    if (ab >= kInfBits || !ts.finite) {
      code[0] = code[1] = 0u;
      return 0x7fu;  // NaN
    }
    const float a = __uint_as_float(ab);
    const float t = a * ts.inv6g;
    const float two[4] = {t * (1.0f - 0x1p-20f), t * (1.0f + 0x1p-20f), 0.f, 0.f};
    const uint32_t c2 = cvt_e4m3x4(two);
    uint32_t sb = c2 & 0xffu;
    if (!ts.fits || sb != c2 >> 8) sb = e4m3_exact(a, ts.g);
    const float s = e4m3_to_f32(sb);
    if (!(s > 0.f) || !(ts.g > 0.f)) {
      code[0] = code[1] = 0u;
      return sb;
    }
    const float d = s * ts.g;
    float r;
    asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(d));  // off by 2^-23 at most
    // A bf16 value lies near a border t * d only if t * d is near a bf16 number, for t = 1, 3, 5 or 7 (the
    // borders' odd factors): four tests per block in place of a second conversion per element. Near: the
    // code of q can be wrong only within 2^-22 of a border, and d * t is off by 2^-23, which is 6 of its
    // last places at most.
    bool near = true;
    if (kBf16) {
      near = !ts.fits;
#pragma unroll
      for (int t = 1; t < 8; t += 2) near |= ((__float_as_uint(d * t) + 8u) & 0xffffu) <= 16u;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float* v = f + 8 * h;
      if (kBf16) {
        float q[8];
        scaled(q, v, r);
        code[h] = cvt_e2m1x8(q);
      }
      if (near) {
        const float rl = r * (1.0f - 0x1p-20f), rh = r * (1.0f + 0x1p-20f);
        float lo[8], hi[8];
        scaled(lo, v, rl);
        scaled(hi, v, rh);
        code[h] = cvt_e2m1x8(lo);
        if (!ts.fits || code[h] != cvt_e2m1x8(hi))
          code[h] = e2m1x8_exact(v[0], v[1], v[2], v[3], v[4], v[5], v[6], v[7],
                                 static_cast<double>(s) * static_cast<double>(ts.g));
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
    const float r = pow2f_bits(bad ? 0 : -k);
    float q[16];
    scaled(q, f, r);
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

// Writes one lane's codes (when `live`: it holds real columns) and, when `in` (it holds a place of the scale
// tiles), its block's scale byte, four blocks of a row to a 32-bit store: the padded groups of a row
// are a whole number of four-block words, so the lanes that hold a word's blocks belong to one row (a
// byte store per block instead of the two shuffles: 5000 x 16384 norm to SV_NVFP4 115 -> 153 us). Every
// lane of the warp calls it.
template <int FMT>
__device__ __forceinline__ void put16(uint8_t* codes, uint8_t* scales, size_t row, int grp, int cols, int sp, bool in,
                                      bool live, const uint32_t (&code)[4], uint32_t sb) {
  constexpr int kPer = FMT == SV_NVFP4 ? 1 : 2;  // groups per block
  const int blk = grp / kPer;
  uint32_t w = live ? sb << (8 * (blk & 3)) : 0u;
  w |= __shfl_xor_sync(0xffffffffu, w, kPer);
  w |= __shfl_xor_sync(0xffffffffu, w, 2 * kPer);
  if (in && grp % (4 * kPer) == 0) *reinterpret_cast<uint32_t*>(scales + scale_at(row, blk, sp)) = w;
  if (!live) return;
  if (FMT == SV_MXFP8)
    *reinterpret_cast<uint4*>(codes + row * cols + static_cast<size_t>(grp) * 16) =
        make_uint4(code[0], code[1], code[2], code[3]);
  else
    *reinterpret_cast<uint2*>(codes + row * (cols / 2) + static_cast<size_t>(grp) * 8) = make_uint2(code[0], code[1]);
}

// Quotients of n < 2^31 by a divisor known on the host: floor(n m / 2^(31 + s)) with 2^(s - 1) < d <= 2^s and
// m = floor(2^(31 + s) / d) + 1 (Granlund and Montgomery, 1994).
struct FastDiv {
  uint32_t d, m;
  int s;
  explicit FastDiv(uint32_t div) : d(div), m(0), s(0) {
    while ((1ull << s) < d) ++s;
    m = d > 1 ? static_cast<uint32_t>((1ull << (31 + s)) / d + 1) : 0;
  }
  __device__ __forceinline__ uint32_t operator()(uint32_t n) const { return d == 1 ? n : __umulhi(n, m) >> (s - 1); }
};

// Steps through a grid of rows of `per_row` items, kMxThreads items at a time.
struct Walk {
  FastDiv per_row;
  uint32_t step_rows;
  int step_item;  // kMxThreads in rows and items
  explicit Walk(int items) : per_row(items), step_rows(kMxThreads / items), step_item(kMxThreads % items) {}
  __device__ __forceinline__ void start(size_t idx, uint32_t& row, int& item) const {
    row = idx < 0x80000000ull ? per_row(static_cast<uint32_t>(idx)) : static_cast<uint32_t>(idx / per_row.d);
    item = static_cast<int>(idx - static_cast<size_t>(row) * per_row.d);
  }
  __device__ __forceinline__ void next(uint32_t& row, int& item) const {
    row += step_rows;
    item += step_item;
    if (item >= static_cast<int>(per_row.d)) item -= per_row.d, ++row;
  }
};

// A block's threads take kSteps groups each of the (padded row, padded group) grid, kMxThreads apart: rows
// rounded up to 128 and gp groups per row (a multiple of 8), so every warp is full and the places of the
// scale tiles that hold no block are written too. Two steps; four, in 64 registers, for bf16 to SV_NVFP4 once
// they fill the device (20240 x 2560, heads: 30 us; two steps 35.1, four in 97 registers 40.2; a block of
// 2760 rows: 6.7 and 5.7 us). Its instructions bound it there: 73 % of the issue slots and 62 % of the ALU are busy,
// with 28 warps an SM, DRAM at 42 %. The scale of every 16 columns (two conversions, a reciprocal, four border
// tests) is what it does beyond SV_MXFP4 (25 us); the conversions to e2m1, 8 cycles a pair and warp, are 5.7 us of
// either. The bounds on blocks per SM make fp32 to SV_MXFP4 and SV_MXFP8 spill 20 to 36 bytes at 40 registers, and
// the four steps of SV_NVFP4 36 at 64.
template <int FMT, typename T, bool kHeads, int kSteps>
__global__ void __launch_bounds__(kMxThreads, FMT == SV_NVFP4 ? 4 : 6)
    quantize_kernel(const T* __restrict__ x, int H, FastDiv N, FastDiv D, uint32_t rows, int cols, Walk walk, int sp,
                    uint32_t rows_padded, const float* gscale, uint8_t* codes, uint8_t* scales) {
  uint32_t row;
  int grp;
  walk.start(static_cast<size_t>(blockIdx.x) * (kMxThreads * kSteps) + threadIdx.x, row, grp);
  griddep_wait();
  if (threadIdx.x == 0) griddep_launch_dependents();
  Cols<T, 16> v[kSteps];
  {
    uint32_t r = row;
    int it = grp;
#pragma unroll
    for (int u = 0; u < kSteps; ++u) {
      const int c = it * kGroup;
      v[u].zero();
      if (r < rows && c < cols) {
        if (kHeads) {
          const uint32_t b = N(r), n = r - b * N.d;
          const T* p = x + (static_cast<size_t>(b) * H * N.d + n) * D.d;
          const size_t head_pitch = static_cast<size_t>(N.d) * D.d;
#pragma unroll
          for (int h = 0; h < 2; ++h) {  // D is a multiple of 8: an octet lies in one head
            const uint32_t ch = static_cast<uint32_t>(c) + 8 * h, head = D(ch);
            v[u].o[h].load(p + head * head_pitch + (ch - head * D.d));
          }
        } else {
          v[u].load(x + static_cast<size_t>(r) * cols + c);
        }
      }
      walk.next(r, it);
    }
  }
  const TensorScale ts = tensor_scale(FMT == SV_NVFP4 ? *gscale : 1.f);
#pragma unroll
  for (int u = 0; u < kSteps; ++u) {
    float f[16];
    v[u].get(f);
    uint32_t code[4];
    const uint32_t sb = quantise16<FMT, sizeof(T) == 2>(f, amax16(v[u]), ts, code);
    put16<FMT>(codes, scales, row, grp, cols, sp, row < rows_padded, row < rows && grp * kGroup < cols, code, sb);
    walk.next(row, grp);
  }
}

// value = element * scale (exact in fp32) * g, rounded once to T; kValueUnroll octets of the (row, octet) grid
// per thread. Bound by HBM: 20240 x 2560 SV_NVFP4 to bf16 22.2 us, 6.0 TB/s.
template <int FMT, typename T>
__global__ void __launch_bounds__(kMxThreads) dequantize_kernel(const uint8_t* __restrict__ codes,
                                                                const uint8_t* __restrict__ scales, const float* gscale,
                                                                Walk walk, int sp, T* y, size_t total) {
  const size_t idx = static_cast<size_t>(blockIdx.x) * (kMxThreads * kValueUnroll) + threadIdx.x;
  uint32_t row;
  int oct;
  walk.start(idx, row, oct);
  griddep_wait();
  if (threadIdx.x == 0) griddep_launch_dependents();
  uint2 c[kValueUnroll];
  uint32_t sb[kValueUnroll];
#pragma unroll
  for (int u = 0; u < kValueUnroll; ++u) {
    const size_t i = idx + static_cast<size_t>(u) * kMxThreads;
    c[u] = make_uint2(0, 0);
    sb[u] = 0;
    if (i < total) {
      if (FMT == SV_MXFP8)
        c[u] = *reinterpret_cast<const uint2*>(codes + i * 8);
      else
        c[u].x = *reinterpret_cast<const uint32_t*>(codes + i * 4);
      sb[u] = scales[scale_at(row, oct / (FMT == SV_NVFP4 ? 2 : 4), sp)];
    }
    walk.next(row, oct);
  }
  const float g = FMT == SV_NVFP4 ? *gscale : 1.f;
#pragma unroll
  for (int u = 0; u < kValueUnroll; ++u) {
    const size_t i = idx + static_cast<size_t>(u) * kMxThreads;
    if (i >= total) break;
    float f[8];
    if (FMT == SV_MXFP8) {
      e4m3x4_to_f32(c[u].x, f);
      e4m3x4_to_f32(c[u].y, f + 4);
    } else {
      e2m1x8_to_f32(c[u].x, f);
    }
    const float s = FMT == SV_NVFP4 ? e4m3_to_f32(sb[u])
                    : sb[u] == 255u ? __uint_as_float(0x7fffffffu)
                                    : pow2f_bits(static_cast<int>(sb[u]) - 127);
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = f[j] * s * g;
    Oct<T> o;
    o.set(f);
    o.store(y + i * kOct);
  }
}

__global__ void zero_scale_kernel(float* g) {  // instead of a memset: the next launch overlaps with it
  griddep_launch_dependents();
  griddep_wait();
  *g = 0.f;
}

// *g = max over the grid of max |x_i| / 2688. The quotient of non-negative values grows with |x|, so
// the maximum of the blocks' quotients (as integers: the bits of non-negative floats are ordered, NaN
// above all) is the quotient of the maximum, in any order. *g is zeroed before the launch, but for one block,
// which stores its result. Four vectors per thread and step, so that enough bytes are in flight: 104 MB of
// bf16 17.5 us with the zeroing, 5.9 TB/s. From the end to the start: the quantisation that follows then
// finds the first part of x in L2 (an fp32 weight to SV_NVFP4 and back 41.0 -> 39.7 us).
constexpr int kMaxBlock = 512;
template <typename T>
__global__ void __launch_bounds__(kMaxBlock) global_scale_kernel(const T* __restrict__ x, size_t n, float* g) {
  griddep_wait();
  if (threadIdx.x == 0) griddep_launch_dependents();
  uint32_t a = 0;
  const size_t vecs = n / kOct, stride = static_cast<size_t>(gridDim.x) * kMaxBlock;
  size_t i = static_cast<size_t>(blockIdx.x) * kMaxBlock + threadIdx.x;
  const auto take = [&](const Oct<T>& v) {
    float f[8];
    v.get(f);
#pragma unroll
    for (int j = 0; j < 8; ++j) a = max(a, __float_as_uint(f[j]) & 0x7fffffffu);
  };
  if (i < n % kOct) a = __float_as_uint(static_cast<float>(x[vecs * kOct + i])) & 0x7fffffffu;
  for (; i + 3 * stride < vecs; i += 4 * stride) {
    Oct<T> v[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) v[u].load(x + (vecs - 1 - i - u * stride) * kOct);
#pragma unroll
    for (int u = 0; u < 4; ++u) take(v[u]);
  }
  for (; i < vecs; i += stride) {
    Oct<T> v;
    v.load(x + (vecs - 1 - i) * kOct);
    take(v);
  }
  a = __reduce_max_sync(0xffffffffu, a);
  __shared__ uint32_t part[kMaxBlock / 32];
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = a;
  __syncthreads();
  if (threadIdx.x < 32) {
    a = __reduce_max_sync(0xffffffffu, threadIdx.x < kMaxBlock / 32 ? part[threadIdx.x] : 0u);
    const uint32_t q = __float_as_uint(__uint_as_float(a) / 2688.0f) & 0x7fffffffu;
    if (threadIdx.x == 0) {
      if (gridDim.x == 1)
        *g = __uint_as_float(q);
      else
        atomicMax(reinterpret_cast<unsigned int*>(g), q);
    }
  }
}

// ---- norm ----
// A team of blockDim.x threads takes one row (blockDim.y rows per block; more than one only with teams of at
// most a warp: 8, 16 or 32 lanes). Thread t holds the column groups i * blockDim.x + t, i < O, of E columns
// (8, or 16 where they are quantised) in registers from the load to the store, so x and the residual are read once; all
// loads are issued before the first is used (with the unpacked values in registers and loads between
// their uses the 720p prefill took 292 us, bound by their latency). Squares are summed in fp64: then
// 1 / sqrt(mean + eps), rounded to fp32, does not depend on how the row is split over threads (but for one
// case in about 1e8), and quantised outputs, where a last-bit difference can move an element by a whole
// step, do not either. 55200 x 2560 bf16 with a residual: 165 us plain (1.13 GB, 6.9 TB/s: HBM bounds it),
// 157 us to SV_MXFP8, 161 us to SV_MXFP4, 168 us to SV_NVFP4.
constexpr int kPlain = -1;
constexpr int kMaxTeam = 512;

// the sum over the lanes of a team (or of its warp)
__device__ __forceinline__ double team_sum(double v, int team) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const double w = __shfl_xor_sync(0xffffffffu, v, o);
    if (o < team) v += w;
  }
  return v;
}

template <int FMT, typename T, int O>
__global__ void __launch_bounds__(kMaxTeam)
    rmsnorm_kernel(const T* x, const T* res, T* h_out, const float* __restrict__ w, size_t rows, size_t rows_padded,
                   int cols, int gp, int sp, float eps, T* y, const float* gscale, uint8_t* codes, uint8_t* scales) {
  __shared__ double part[kMaxTeam / 32];
  griddep_wait();
  if (threadIdx.x == 0 && threadIdx.y == 0) griddep_launch_dependents();
  const size_t row = static_cast<size_t>(blockIdx.x) * blockDim.y + threadIdx.y;
  const int team = blockDim.x;
  const bool real = row < rows;
  const size_t base = row * cols;
  constexpr int E = FMT == kPlain ? kOct : kGroup;
  Cols<T, E> h[O];
#pragma unroll
  for (int i = 0; i < O; ++i) {
    const int c = (i * team + static_cast<int>(threadIdx.x)) * E;
    h[i].zero();
    if (real && c < cols) h[i].load(x + base + c);
  }
  if (res != nullptr) {
    Cols<T, E> r[O];
#pragma unroll
    for (int i = 0; i < O; ++i) {
      const int c = (i * team + static_cast<int>(threadIdx.x)) * E;
      r[i].zero();
      if (real && c < cols) r[i].load(res + base + c);
    }
#pragma unroll
    for (int i = 0; i < O; ++i) h[i].add(r[i]);
  }
  double s0 = 0.0, s1 = 0.0;
#pragma unroll
  for (int i = 0; i < O; ++i) {
    float f[E];
    h[i].get(f);
#pragma unroll
    for (int j = 0; j < E; j += 2) {
      const double a = f[j], b = f[j + 1];
      s0 = fma(a, a, s0);
      s1 = fma(b, b, s1);
    }
    const int c = (i * team + static_cast<int>(threadIdx.x)) * E;
    if (h_out != nullptr && real && c < cols) h[i].store(h_out + base + c);
  }
  double sum = team_sum(s0 + s1, team);
  if (team > 32) {
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = sum;
    __syncthreads();
    sum = 0.0;
    for (int k = 0; k < team / 32; ++k) sum += part[k];
  }
  double r = 1.0 / sqrt(sum / cols + static_cast<double>(eps));
  // 1 / rms leaves fp32's normal range (values near the largest one; subnormal values without an eps): the row is
  // scaled by a power of two first, exact where its results do not vanish. That code never runs for other rows,
  // but the registers of the loop below depend on its place: as loaded, or in the loop for the other kernels
  // (2760 x 2560: bf16 to SV_MXFP4 9.7 us instead of 10.5, fp32 to SV_MXFP8 19.8 instead of 22.2; 55200 x 2560: bf16 to
  // SV_MXFP8 as loaded 157 us instead of 166).
  constexpr bool kAsLoaded = (FMT == SV_MXFP4) != (sizeof(T) == 2);
  float shift = 1.f;
  if (r < 0x1p-126 || r > 0x1p127) {
    shift = r < 1.0 ? 0x1p-64f : 0x1p64f;
    r *= r < 1.0 ? 0x1p64 : 0x1p-64;
    if constexpr (kAsLoaded) {
#pragma unroll
      for (int i = 0; i < O; ++i) h[i].scale(shift);
    }
  }
  const float rstd = static_cast<float>(r);
  const TensorScale ts = tensor_scale(FMT == SV_NVFP4 ? *gscale : 1.f);
#pragma unroll
  for (int i = 0; i < O; ++i) {
    const int grp = i * team + static_cast<int>(threadIdx.x);
    const int c = grp * E;
    const bool live = real && c < cols;
    float f[E];
    h[i].get(f);
    if (!kAsLoaded && shift != 1.f) scaled(f, f, shift);
    if (live) {
#pragma unroll
      for (int j = 0; j < E; j += 4) {
        const float4 ww = __ldg(reinterpret_cast<const float4*>(w + c + j));
        mul2(f[j], f[j + 1], f[j], f[j + 1], rstd, rstd);
        mul2(f[j + 2], f[j + 3], f[j + 2], f[j + 3], rstd, rstd);
        mul2(f[j], f[j + 1], f[j], f[j + 1], ww.x, ww.y);
        mul2(f[j + 2], f[j + 3], f[j + 2], f[j + 3], ww.z, ww.w);
      }
    }
    if constexpr (FMT == kPlain) {
      if (live) {
        Cols<T, E> o;
        o.set(f);
        o.store(y + base + c);
      }
    } else {
      uint32_t code[4];
      const uint32_t sb = quantise16<FMT, false>(f, amax16(f), ts, code);
      // the team may cover more than gp groups
      put16<FMT>(codes, scales, row, grp, cols, sp, grp < gp && row < rows_padded, live, code, sb);
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

size_t matrix_bytes(long long rows, int cols, sv_dtype dt) {
  return static_cast<size_t>(rows) * cols * (dt == SV_F32 ? 4 : 2);
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
sv_status run_quantize(const void* x, int H, int N, int D, const sv_mx& m, int sms, cudaStream_t st) {
  const int sp = mx_padded_blocks(m.fmt, m.cols);
  const int gp = sp * (mx_block(m.fmt) / kGroup);  // padded columns may be 2^31
  const long long rows_padded = mx_row_tiles(m.rows) * 128, groups = rows_padded * gp;
  if (groups / (2 * kMxThreads) > 0x7ffffffeLL) return mfail(SV_ERR_UNSUPPORTED, "too many elements");
  const auto go = [&](auto kernel, int steps) {
    const unsigned blocks = static_cast<unsigned>((groups + kMxThreads * steps - 1) / (kMxThreads * steps));
    cudaLaunchAttribute at;
    const cudaLaunchConfig_t cfg = pdl_config(dim3(blocks), dim3(kMxThreads), st, &at);
    return launched(cudaLaunchKernelEx(&cfg, kernel, static_cast<const T*>(x), H, FastDiv(N), FastDiv(D),
                                       static_cast<uint32_t>(m.rows), m.cols, Walk(gp), sp,
                                       static_cast<uint32_t>(rows_padded), m.gscale, static_cast<uint8_t*>(m.codes),
                                       static_cast<uint8_t*>(m.scales)),
                    "quantisation");
  };
  if constexpr (FMT == SV_NVFP4 && sizeof(T) == 2) {
    if (groups >= 4ll * sms * 4 * kMxThreads)
      return H == 1 ? go(quantize_kernel<FMT, T, false, 4>, 4) : go(quantize_kernel<FMT, T, true, 4>, 4);
  }
  return H == 1 ? go(quantize_kernel<FMT, T, false, 2>, 2) : go(quantize_kernel<FMT, T, true, 2>, 2);
}

template <int FMT, typename T>
sv_status run_dequantize(const sv_mx& m, void* y, cudaStream_t st) {
  const int op = m.cols / kOct;
  const size_t total = static_cast<size_t>(m.rows) * op, per = kMxThreads * kValueUnroll;
  const size_t blocks = (total + per - 1) / per;
  if (blocks > 0x7fffffffull) return mfail(SV_ERR_UNSUPPORTED, "too many elements");
  cudaLaunchAttribute at;
  const cudaLaunchConfig_t cfg = pdl_config(dim3(static_cast<unsigned>(blocks)), dim3(kMxThreads), st, &at);
  return launched(cudaLaunchKernelEx(&cfg, dequantize_kernel<FMT, T>, static_cast<const uint8_t*>(m.codes),
                                     static_cast<const uint8_t*>(m.scales), m.gscale, Walk(op),
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

template <int FMT, typename T, int O>
sv_status launch_norm(const NormArgs& a, int team, int gp, int sp, cudaStream_t st) {
  const int per_block = team <= 32 ? 256 / team : 1;
  const long long rows_padded = a.q != nullptr ? mx_row_tiles(a.rows) * 128 : a.rows;
  const long long blocks = (rows_padded + per_block - 1) / per_block;
  cudaLaunchAttribute at;
  const cudaLaunchConfig_t cfg = pdl_config(dim3(static_cast<unsigned>(blocks)), dim3(team, per_block), st, &at);
  return launched(
      cudaLaunchKernelEx(&cfg, rmsnorm_kernel<FMT, T, O>, static_cast<const T*>(a.x), static_cast<const T*>(a.res),
                         static_cast<T*>(a.h), a.w, static_cast<size_t>(a.rows), static_cast<size_t>(rows_padded), a.C,
                         gp, sp, a.eps, static_cast<T*>(a.y), a.q != nullptr ? a.q->gscale : nullptr,
                         a.q != nullptr ? static_cast<uint8_t*>(a.q->codes) : nullptr,
                         a.q != nullptr ? static_cast<uint8_t*>(a.q->scales) : nullptr),
      "norm");
}

template <int FMT, typename T>
sv_status run_norm(const NormArgs& a, int sms, cudaStream_t st) {
  const int sp = a.q != nullptr ? mx_padded_blocks(a.q->fmt, a.C) : 0;
  const int gp = a.q != nullptr ? sp * (mx_block(a.q->fmt) / kGroup) : (a.C + kOct - 1) / kOct;
  // Narrow rows: 8, 16 or 32 lanes each. Few rows: a thread per group of columns, so that a row's latency
  // is one load's and a short sum's. Many: two groups per thread (measured on 55200 x 2560 bf16, plain:
  // 2 groups 164 us, 1 group 215, a warp per row with 10 groups 167; to SV_MXFP8: 166, 180, 348).
  constexpr int kWide = FMT == kPlain ? 8 : 4;
  if (gp <= 32) return launch_norm<FMT, T, 1>(a, gp <= 8 ? 8 : gp <= 16 ? 16 : 32, gp, sp, st);
  if (a.rows <= 4 * sms && gp <= kMaxTeam) return launch_norm<FMT, T, 1>(a, (gp + 31) / 32 * 32, gp, sp, st);
  if (gp <= 2 * kMaxTeam) return launch_norm<FMT, T, 2>(a, ((gp + 1) / 2 + 31) / 32 * 32, gp, sp, st);
  return launch_norm<FMT, T, kWide>(a, ((gp + kWide - 1) / kWide + 31) / 32 * 32, gp, sp, st);
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

bool overlap(const sv_mx& m, const void* p, size_t n) {
  return overlap(m.codes, sv_mx_code_bytes(m.fmt, m.rows, m.cols), p, n) ||
         overlap(m.scales, sv_mx_scale_bytes(m.fmt, m.rows, m.cols), p, n);
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
  // one block while its eight rounds of four vectors are about the cost of the second launch
  const long long per = static_cast<long long>(kMaxBlock) * kOct * 4;
  const long long want = n <= 8 * per ? 1 : (n + per - 1) / per;
  const unsigned blocks = static_cast<unsigned>(want < 4ll * sms ? want : 4ll * sms);
  cudaLaunchAttribute at;
  if (blocks > 1) {
    const cudaLaunchConfig_t cfg = pdl_config(dim3(1), dim3(1), st, &at);
    MX_TRY(launched(cudaLaunchKernelEx(&cfg, zero_scale_kernel, g), "tensor scale"));
  }
  const cudaLaunchConfig_t cfg = pdl_config(dim3(blocks), dim3(kMaxBlock), st, &at);
  const cudaError_t e =
      dt == SV_BF16 ? cudaLaunchKernelEx(&cfg, global_scale_kernel<__nv_bfloat16>, static_cast<const __nv_bfloat16*>(x),
                                         static_cast<size_t>(n), g)
                    : cudaLaunchKernelEx(&cfg, global_scale_kernel<float>, static_cast<const float*>(x),
                                         static_cast<size_t>(n), g);
  return launched(e, "tensor scale");
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
  if (overlap(*out, x, matrix_bytes(out->rows, out->cols, dt)))
    return mfail(SV_ERR_INVALID_ARG, "out must not overlap x");
  int sms = 0;
  MX_TRY(mx_device(&sms));
  MX_DISPATCH(out->fmt, dt, run_quantize, x, H, N, D, *out, sms, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" sv_status sv_mx_dequantize(const sv_mx* in, void* y, sv_dtype dt, sv_stream_t stream) {
  using namespace sv;
  MX_TRY(check_dt(dt));
  MX_TRY(check_mx(in, "in"));
  if (y == nullptr || !aligned(y, 16)) return mfail(SV_ERR_INVALID_ARG, "y must be non-NULL and 16-byte aligned");
  if (overlap(*in, y, matrix_bytes(in->rows, in->cols, dt))) return mfail(SV_ERR_INVALID_ARG, "y must not overlap in");
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
  // in place or apart: a row is read before it is written, but not another block's rows
  const size_t n = matrix_bytes(rows, C, dt);
  const auto apart = [&](const void* out, const void* in) { return out == in || !overlap(out, n, in, n); };
  if (!apart(h, x) || !apart(h, residual) || !apart(y, x) || !apart(y, residual) || overlap(y, n, h, n) ||
      overlap(y, n, w, 4 * static_cast<size_t>(C)) ||
      ((residual != nullptr || h != x) && overlap(h, n, w, 4 * static_cast<size_t>(C))))
    return mfail(SV_ERR_INVALID_ARG, "y and h must not overlap w, each other, or x or the residual other than in place");
  if (yq != nullptr && (overlap(*yq, x, n) || overlap(*yq, residual, n) || overlap(*yq, h, n) ||
                        overlap(*yq, w, 4 * static_cast<size_t>(C))))
    return mfail(SV_ERR_INVALID_ARG, "yq must not overlap x, residual, h or w");
  int sms = 0;
  MX_TRY(mx_device(&sms));
  // without a residual h is x: nothing to write where they are the same buffer
  const NormArgs a{x, residual, residual == nullptr && h == x ? nullptr : h, w, rows, C, eps, y, yq};
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (yq == nullptr)
    return dt == SV_BF16 ? run_norm<kPlain, __nv_bfloat16>(a, sms, st) : run_norm<kPlain, float>(a, sms, st);
  MX_DISPATCH(yq->fmt, dt, run_norm, a, sms, st);
}
