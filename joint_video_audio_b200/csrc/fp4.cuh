// Microscaled 4-bit floats: layout, and the quantisation of a 128-channel
// block held by four lanes.
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
// A thread group of four lanes holds a block of 128 channels: lane l has the
// eight-channel chunks l, l + 4, l + 8, l + 12, so that global loads of a chunk
// take 64 contiguous bytes per group, an MX block is one chunk of each of the
// four lanes, an NV block one chunk of a lane pair, and five of the seven
// stages of the 128-point Hadamard transform stay inside a thread.
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

// Unnormalised 128-point Walsh-Hadamard transform of a group's block,
// h[8 j + e] = channel 32 j + 8 l + e of lane l.
__device__ __forceinline__ void fwht128_group(float (&h)[32], int lane) {
#pragma unroll
  for (int e = 0; e < 32; e += 2) {
    const float u = h[e], w = h[e + 1];
    h[e] = u + w;
    h[e + 1] = u - w;
  }
#pragma unroll
  for (int b = 2; b < 32; b <<= 1) {  // channel bits 1, 2 (in a chunk) and 5, 6 (across the lane's chunks)
#pragma unroll
    for (int e = 0; e < 32; e += 2) {
      if (!(e & b)) {
        const uint64_t u = f2_pack(h[e], h[e + 1]), w = f2_pack(h[e + b], h[e + b + 1]);
        f2_unpack(f2_add(u, w), h[e], h[e + 1]);
        f2_unpack(f2_fma(w, f2_pack(-1.f, -1.f), u), h[e + b], h[e + b + 1]);
      }
    }
  }
#pragma unroll
  for (int m = 1; m <= 2; m <<= 1) {  // channel bits 3, 4: the lower lane takes h + other, the upper other - h
    const float sg = (lane & m) ? -1.f : 1.f;
    const uint64_t sg2 = f2_pack(sg, sg);
#pragma unroll
    for (int e = 0; e < 32; e += 2) {
      const float o0 = __shfl_xor_sync(0xffffffffu, h[e], m), o1 = __shfl_xor_sync(0xffffffffu, h[e + 1], m);
      f2_unpack(f2_fma(sg2, f2_pack(h[e], h[e + 1]), f2_pack(o0, o1)), h[e], h[e + 1]);
    }
  }
}

// Lane l's words of four chunk columns (chunk 4 j + l in w[j]) to the words of
// its own row quarter (chunk 4 l + j): a 4 x 4 transpose inside the group.
// It is its own inverse.
__device__ __forceinline__ uint4 group_transpose(const uint32_t (&w)[4], int lane) {
  const bool o1 = lane & 1, o2 = lane & 2;
  uint32_t a0 = w[0], a1 = w[1], a2 = w[2], a3 = w[3];
  uint32_t s0 = __shfl_xor_sync(0xffffffffu, o1 ? a0 : a1, 1);
  uint32_t s1 = __shfl_xor_sync(0xffffffffu, o1 ? a2 : a3, 1);
  if (o1) {
    a0 = s0;
    a2 = s1;
  } else {
    a1 = s0;
    a3 = s1;
  }
  s0 = __shfl_xor_sync(0xffffffffu, o2 ? a0 : a2, 2);
  s1 = __shfl_xor_sync(0xffffffffu, o2 ? a1 : a3, 2);
  if (o2) {
    a0 = s0;
    a1 = s1;
  } else {
    a2 = s0;
    a3 = s1;
  }
  return make_uint4(a0, a1, a2, a3);
}

// Largest magnitude of each of a lane's four chunks.
__device__ __forceinline__ void chunk_amax(const float (&h)[32], float (&am)[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float a = fabsf(h[8 * j]);
#pragma unroll
    for (int e = 1; e < 8; ++e) a = max_nan(a, fabsf(h[8 * j + e]));
    am[j] = a;
  }
}

// Eight values of an MX block with largest magnitude `amax` -> codes and the
// block's scale byte. The scale is the smallest 2^e with amax <= 7 * 2^e: an
// amax in (6, 7] takes the code 6 under 2^e and under 2^(e+1) alike, so the
// smaller scale is never the worse one. Multiplying by 2^-e is exact, hence so
// are the codes. A block with a non-finite value gets the NaN scale.
__device__ __forceinline__ uint32_t quant8_mx(float* h, float amax, uint32_t& scale) {
  const uint32_t bits = __float_as_uint(amax) & 0x7fffffffu;
  int code = (int)(bits >> 23) - 2 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);
  code = code < 1 ? 1 : code;
  const bool ok = bits < 0x7f800000u;
  const float inv = __uint_as_float((uint32_t)(ok ? 254 - code : 0) << 23);
  scale = (uint32_t)(ok ? code : 255);
  const uint64_t inv2 = f2_pack(inv, inv);
#pragma unroll
  for (int e = 0; e < 8; e += 2) f2_unpack(f2_mul(f2_pack(h[e], h[e + 1]), inv2), h[e], h[e + 1]);
  return e2m1x8(h);
}
// MX: am[j] of the lane's chunks -> the group's codes and its four scale bytes
// (the same word in every lane).
__device__ __forceinline__ void quant_mx(float (&h)[32], float (&am)[4], uint32_t (&codes)[4], uint32_t& scale_word) {
  scale_word = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    am[j] = max_nan(am[j], __shfl_xor_sync(0xffffffffu, am[j], 1));
    am[j] = max_nan(am[j], __shfl_xor_sync(0xffffffffu, am[j], 2));
    uint32_t sc;
    codes[j] = quant8_mx(h + 8 * j, am[j], sc);
    scale_word |= sc << (8 * j);
  }
}

// NV, first half: am[j] becomes the largest magnitude of the lane pair's
// block; returns the largest finite one (0 if none).
__device__ __forceinline__ float nv_block_amax(float (&am)[4]) {
  float top = 0.f;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    am[j] = max_nan(am[j], __shfl_xor_sync(0xffffffffu, am[j], 1));
    if (finite_bits(am[j])) top = fmaxf(top, am[j]);
  }
  return top;
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

// Eight values of an NV block with largest magnitude `amax`, in a row of scale
// 1 / inv_row -> codes and the block's scale byte, amax / 6 in e4m3. The
// quotient u / s is taken as in quotient(), negated: -u / s keeps the sign of a
// zero, and the codes' signs are flipped at the end.
__device__ __forceinline__ uint32_t quant8_nv(float* h, float amax, float inv_row, uint32_t& scale) {
  const bool ok = finite_bits(amax);
  scale = ok ? e4m3_code(quotient(amax * inv_row, 6.f, 1.f / 6.f)) : 0x7fu;
  const float s = ok ? e4m3_value(scale) : 0.f;
  const float r = s > 0.f ? rcp_approx(s) : 0.f;
  const uint64_t inv2 = f2_pack(inv_row, inv_row), nr2 = f2_pack(-r, -r), s2 = f2_pack(s, s);
#pragma unroll
  for (int e = 0; e < 8; e += 2) {
    const uint64_t u = f2_mul(f2_pack(h[e], h[e + 1]), inv2);
    const uint64_t nq = f2_mul(u, nr2);
    f2_unpack(f2_fma(f2_fma(nq, s2, u), nr2, nq), h[e], h[e + 1]);
  }
  return e2m1x8(h) ^ 0x88888888u;
}
__device__ __forceinline__ float pow2_float(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }
// NV, second half: codes and the lane's four scale bytes, one per chunk (byte
// j: block 2 j + l / 2 of the 128 channels).
__device__ __forceinline__ void quant_nv(float (&h)[32], const float (&am)[4], int row_exp, uint32_t (&codes)[4],
                                         uint32_t& scale_bytes) {
  scale_bytes = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint32_t sc;
    codes[j] = quant8_nv(h + 8 * j, am[j], pow2_float(-row_exp), sc);
    scale_bytes |= sc << (8 * j);
  }
}

// Where a row's 4-bit form goes.
struct Fp4Row {
  uint8_t* codes;   // the row's first byte
  uint8_t* scales;  // the whole scale tensor
  int64_t row;
  int K, katoms;
};

// Stores a group's block `blk` (128 channels from 128 blk) where `ok` (the same
// for the four lanes). Every lane of the warp calls it. Chunks past K hold
// zeros; whole quarters past K are not stored.
template <int FMT>
__device__ __forceinline__ void store_group(bool ok, const Fp4Row& o, int blk, int lane, const uint32_t (&codes)[4],
                                            uint32_t scale) {
  const int l = lane & 3;
  const uint4 c = group_transpose(codes, lane);
  if (ok && blk * 128 + l * 32 < o.K) *reinterpret_cast<uint4*>(o.codes + blk * 64 + l * 16) = c;
  if (FMT == kFp4MX) {
    if (ok && l == 0) *fp4_scale_word(o.scales, o.row, o.katoms, blk) = scale;
  } else {
    const uint32_t other = __shfl_xor_sync(0xffffffffu, scale, 2);
    // lane 0 holds blocks 0, 2, 4, 6 of the 128 channels, lane 2 blocks 1, 3, 5, 7
    if (ok && l == 0) *fp4_scale_word(o.scales, o.row, o.katoms, 2 * blk) = __byte_perm(scale, other, 0x5140);
    if (ok && l == 2 && 2 * blk + 1 < o.katoms)
      *fp4_scale_word(o.scales, o.row, o.katoms, 2 * blk + 1) = __byte_perm(other, scale, 0x7362);
  }
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
