// Microscaled 4-bit floats: layout, and the quantisation of a block.
//
// A value is an e2m1 code (0, 0.5, 1, 1.5, 2, 3, 4, 6 with a sign) times its
// block's scale times its row's scale. Two formats:
//   MX  blocks of 32, scale 2^e (e8m0, code e + 127)
//   NV  blocks of 16, scale in e4m3
// Codes lie two to a byte (the even channel in the low nibble), [rows][K / 2].
// Block scales lie in atoms of 128 rows x 4 blocks, 512 bytes, as the tensor
// core takes them: row r, block b at byte (r % 32) * 16 + (r / 32 % 4) * 4 + b % 4
// of atom (r / 128) * katoms + b / 4.
//
// Rows are worked on in chunks of eight channels (16 bytes of bf16, one word of
// codes); an MX block is four chunks, an NV block two.
#pragma once
#include <cstdint>

#include "ptx.cuh"

namespace h3 {

constexpr int kFp4MX = 0, kFp4NV = 1;

__host__ __device__ constexpr int fp4_atom_channels(int fmt) { return fmt == kFp4NV ? 64 : 128; }
__host__ __device__ inline int fp4_katoms(int fmt, int K) {
  return (K + fp4_atom_channels(fmt) - 1) / fp4_atom_channels(fmt);
}
// The four bytes of row `row` in its atom `ka`.
__device__ __forceinline__ uint32_t* fp4_scale_word(uint8_t* scales, int64_t row, int katoms, int ka) {
  return reinterpret_cast<uint32_t*>(scales + ((row >> 7) * katoms + ka) * 512 + (row & 31) * 16 + ((row >> 5) & 3) * 4);
}

// max that yields NaN when either input is NaN
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ bool finite_bits(float a) { return (__float_as_uint(a) & 0x7f800000u) != 0x7f800000u; }

// e2m1 codes of eight values, v[0] in the low nibble: nearest, ties to the
// even code, beyond 6 saturates.
__device__ __forceinline__ uint32_t e2m1x8(const float* v) {
  uint32_t r;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}
// The eight values of a word of codes, as four half pairs (exact).
__device__ __forceinline__ void e2m1x8_values(uint32_t w, float (&v)[8]) {
  uint32_t h[4];
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
#pragma unroll
  for (int i = 0; i < 4; ++i)
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\tcvt.f32.f16 %0, lo;\n\tcvt.f32.f16 %1, hi;\n\t}"
        : "=f"(v[2 * i]), "=f"(v[2 * i + 1])
        : "r"(h[i]));
}

// e4m3 of a non-negative value (nearest even, saturating), and its value.
__device__ __forceinline__ uint32_t e4m3_code(float v) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.f), "f"(v));
  return r & 0xffu;
}
__device__ __forceinline__ float e4m3_value(uint32_t code) {
  uint32_t h;
  float f;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)code));
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.f32.f16 %0, lo;\n\t}" : "=f"(f) : "r"(h));
  return f;
}
__device__ __forceinline__ float e8m0_value(uint32_t code) {
  return __uint_as_float(code == 0 ? 0x00400000u : code == 255 ? 0x7fffffffu : code << 23);
}

// Unnormalised 128-point Walsh-Hadamard transforms of the eight blocks a warp
// holds, bf16 in: H128 = H16 x H8 (Kronecker) with channel = 8 i + e. The
// 16-point part, across chunks, is a product with the +-1 matrix H16 on the
// tensor cores (m16n8k16; n = block, one product for each e), exact up to the
// fp32 sum; the 8-point part then lies inside a lane. Against butterflies with
// two lane exchanges a value it takes 72 instructions a lane instead of 224.
//
// In: lane (b = lane / 4, t = lane % 4) holds chunks 2 t, 2 t + 1, 2 t + 8 and
// 2 t + 9 of block b, the pairs in the order of `swapped` blocks reversed.
// Out: lane (g = lane / 4, t): h[0..15] chunks 2 g, 2 g + 1 of block 2 t (an NV
// block), h[16..31] the same chunks of block 2 t + 1: H16's rows are taken in
// the order 0, 2, .. 14, 1, 3, .. 15.
__device__ __forceinline__ void fwht128_warp(const uint4 (&v)[4], bool swapped, int lane, float (&h)[32]) {
  const int g = lane >> 2, t = lane & 3;
  auto pm1 = [](int r, int c) { return (uint32_t)((__popc(r & c) & 1) ? 0xBF80u : 0x3F80u); };
  auto frag = [&](int r, int c) { return pm1(r, c) | (pm1(r, c + 1) << 16); };
  const uint32_t a0 = frag(2 * g, 2 * t), a1 = frag(2 * g + 1, 2 * t);
  const uint32_t a2 = frag(2 * g, 2 * t + 8), a3 = frag(2 * g + 1, 2 * t + 8);
  const uint32_t lo = swapped ? 0x1054u : 0x5410u, hi = swapped ? 0x3276u : 0x7632u;
  const uint32_t w[4][4] = {{v[0].x, v[0].y, v[0].z, v[0].w},
                            {v[1].x, v[1].y, v[1].z, v[1].w},
                            {v[2].x, v[2].y, v[2].z, v[2].w},
                            {v[3].x, v[3].y, v[3].z, v[3].w}};
  float d[8][4];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const uint32_t b0 = __byte_perm(w[0][e >> 1], w[1][e >> 1], (e & 1) ? hi : lo);
    const uint32_t b1 = __byte_perm(w[2][e >> 1], w[3][e >> 1], (e & 1) ? hi : lo);
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(d[e][0]), "=f"(d[e][1]), "=f"(d[e][2]), "=f"(d[e][3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
  }
  // 8-point transforms over e of the four (chunk, block) results
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int c = (q & 1) * 2 + (q >> 1);  // h order: chunks 2 g, 2 g + 1 of block 2 t, then of block 2 t + 1
    uint64_t p[4];
#pragma unroll
    for (int e = 0; e < 8; e += 2) {  // bit 0
      const float u = d[e][c], x = d[e + 1][c];
      p[e >> 1] = f2_pack(u + x, u - x);
    }
    const uint64_t m1 = f2_pack(-1.f, -1.f);
#pragma unroll
    for (int bit = 1; bit <= 2; bit <<= 1)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (!(e & bit)) {
          const uint64_t u = p[e], x = p[e + bit];
          p[e] = f2_add(u, x);
          p[e + bit] = f2_fma(x, m1, u);
        }
#pragma unroll
    for (int e = 0; e < 4; ++e) f2_unpack(p[e], h[8 * q + 2 * e], h[8 * q + 2 * e + 1]);
  }
}

// Largest magnitude of eight values (NaN if one is).
__device__ __forceinline__ float amax8(const float* h) {
  float a = fabsf(h[0]);
#pragma unroll
  for (int e = 1; e < 8; ++e) a = max_nan(a, fabsf(h[e]));
  return a;
}
// The same of eight bf16 values.
__device__ __forceinline__ float amax8(const uint4& v) {
  auto mx = [](uint32_t a, uint32_t b) {
    uint32_t d;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
  };
  const uint32_t m = 0x7fff7fffu;
  const uint32_t r = mx(mx(v.x & m, v.y & m), mx(v.z & m, v.w & m));
  return max_nan(__uint_as_float(r << 16), __uint_as_float(r & 0xffff0000u));
}

// MX: scale byte of a block with largest magnitude `amax`, and the factor 2^-e
// of its values. The scale is the smallest 2^e with amax <= 7 * 2^e: an amax in
// (6, 7] takes the code 6 under 2^e and under 2^(e+1) alike, so the smaller
// scale is never the worse one. Multiplying by 2^-e is exact, hence so are the
// codes. A block with a non-finite value gets the NaN scale.
__device__ __forceinline__ float mx_scale(float amax, uint32_t& scale) {
  const uint32_t bits = __float_as_uint(amax) & 0x7fffffffu;
  int code = (int)(bits >> 23) - 2 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);
  code = code < 1 ? 1 : code;
  const bool ok = bits < 0x7f800000u;
  scale = (uint32_t)(ok ? code : 255);
  return __uint_as_float((uint32_t)(ok ? 254 - code : 0) << 23);
}
__device__ __forceinline__ uint32_t quant8_mx(float* h, float inv) {
  const uint64_t inv2 = f2_pack(inv, inv);
#pragma unroll
  for (int e = 0; e < 8; e += 2) f2_unpack(f2_mul(f2_pack(h[e], h[e + 1]), inv2), h[e], h[e + 1]);
  return e2m1x8(h);
}

// Exponent E of a row's scale 2^E: the smallest with amax <= 448 * 6 * 2^E, so
// that the largest block scale lies in the upper binade of e4m3. 0 for a zero row.
__device__ __forceinline__ int nv_row_exponent(float amax) {
  const uint32_t bits = __float_as_uint(amax);
  if (bits == 0) return 0;
  const int e = (int)(bits >> 23) - 127 - 11 + ((bits & 0x7fffffu) > 0x280000u ? 1 : 0);  // 2688 = 1.3125 * 2^11
  return e < -126 ? -126 : e;
}
// a / b correctly rounded up to the last place's tie, from an approximate r of
// 1 / b: one Newton step with the exact remainder. Where the quotient is itself
// a float (as a value halfway between two codes is), it is found exactly.
__device__ __forceinline__ float quotient(float a, float b, float r) {
  const float q = a * r;
  return fmaf(fmaf(-q, b, a), r, q);
}
__device__ __forceinline__ float rcp_approx(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

__device__ __forceinline__ float pow2_float(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }
// NV: scale byte of a block with largest magnitude `amax` in a row of scale
// 2^row_exp: amax / 2^row_exp / 6 in e4m3. Returned: the scale times 2^row_exp
// and an approximate reciprocal of that. Rows of row_exp < kNvSmall, whose
// reciprocals would overflow, are multiplied by 2^kNvLift first (values, not
// amax), and `lift` is that.
constexpr int kNvSmall = -100, kNvLift = 64;
struct NvScale {
  float s, r;
};
__device__ __forceinline__ NvScale nv_scale(float amax, int row_exp, int lift, uint32_t& scale) {
  const bool ok = finite_bits(amax);
  scale = ok ? e4m3_code(quotient(amax * pow2_float(-row_exp), 6.f, 1.f / 6.f)) : 0x7fu;
  const float s = ok ? e4m3_value(scale) : 0.f;
  return {s * pow2_float(row_exp + lift), s > 0.f ? rcp_approx(s) * pow2_float(-row_exp - lift) : 0.f};
}
// Eight values h / s (see quotient()), taken as -h / s, which keeps the sign of
// a zero, and the codes' signs flipped at the end.
__device__ __forceinline__ uint32_t quant8_nv(float* h, const NvScale& sc) {
  const uint64_t nr2 = f2_pack(-sc.r, -sc.r), s2 = f2_pack(sc.s, sc.s);
#pragma unroll
  for (int e = 0; e < 8; e += 2) {
    const uint64_t u = f2_pack(h[e], h[e + 1]);
    const uint64_t nq = f2_mul(u, nr2);
    f2_unpack(f2_fma(f2_fma(nq, s2, u), nr2, nq), h[e], h[e + 1]);
  }
  return e2m1x8(h) ^ 0x88888888u;
}
__device__ __forceinline__ void nv_lift8(float* h) {
#pragma unroll
  for (int e = 0; e < 8; ++e) h[e] *= pow2_float(kNvLift);
}
__device__ __forceinline__ void unpack_bf16x8(const uint4& v, float* f) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    f[2 * q] = __uint_as_float(w[q] << 16);
    f[2 * q + 1] = __uint_as_float(w[q] & 0xffff0000u);
  }
}

}  // namespace h3
