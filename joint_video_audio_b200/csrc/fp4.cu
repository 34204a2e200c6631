// Quantisation of bf16 rows to microscaled 4-bit floats (optionally rotated by
// the block-128 Hadamard transform, as the W8A8 path's inputs are), and back.
// Layout, formats and the arithmetic of a block: fp4.cuh.
//
// Both passes are bound by moving each value in and out once: 2 + 0.5 bytes a
// value and its block scale. A row is spread over whole warps, four lanes to a
// block of 128 channels; NV needs the row's largest magnitude before its first
// code, so a CTA holds its rows in registers across one reduction, and MX runs
// without any barrier.
#include <cuda_bf16.h>

#include "fp4.cuh"
#include "kernels.cuh"

namespace h3 {
namespace {

constexpr int kMaxRowWarps = 16;  // 1024 channels each: K <= 16384
constexpr int kSmallCta = 8;      // warps of a CTA whose rows take one warp each

// warps: warps per row; a CTA holds blockDim.x / (32 * warps) rows.
template <int FMT, bool ROT>
__global__ void __launch_bounds__(kMaxRowWarps * 32) quantize_fp4_kernel(const __nv_bfloat16* __restrict__ in, int64_t ld,
                                                                       int64_t rows, int K, int katoms, int warps,
                                                                       uint8_t* __restrict__ codes,
                                                                       uint8_t* __restrict__ scales,
                                                                       float* __restrict__ row_scale) {
  __shared__ float red[kMaxRowWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int per_cta = (blockDim.x >> 5) / warps;
  const int64_t row = (int64_t)blockIdx.x * per_cta + warp / warps;
  const int w = warp % warps;
  const int blk = w * 8 + (lane >> 2), l = lane & 3;
  const bool row_ok = row < rows;
  float h[32];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int c = blk * 128 + j * 32 + l * 8;
    uint4 v = make_uint4(0, 0, 0, 0);
    if (row_ok && c < K) v = __ldg(reinterpret_cast<const uint4*>(in + row * ld + c));
    unpack_bf16x8(v, h + 8 * j);
  }
  if (ROT) fwht128_group(h, lane);
  float am[4];
  chunk_amax(h, am);
  const Fp4Row o{codes + row * (K >> 1), scales, row, K, katoms};
  const bool store = row_ok && blk * 128 < K;
  uint32_t q[4], sc;
  constexpr float kRot = 0.08838834764831845f;  // 1 / sqrt(128)
  if (FMT == kFp4MX) {
    quant_mx(h, am, q, sc);
    store_group<FMT>(store, o, blk, lane, q, sc);
    if (row_ok && w == 0 && lane == 0) row_scale[row] = ROT ? kRot : 1.f;
  } else {
    float top = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(nv_block_amax(am))));
    if (warps > 1) {
      if (lane == 0) red[warp] = top;
      __syncthreads();
      const int first = warp - w;
      for (int i = 0; i < warps; ++i) top = fmaxf(top, red[first + i]);
    }
    const int e = nv_row_exponent(top);
    quant_nv(h, am, e, q, sc);
    store_group<FMT>(store, o, blk, lane, q, sc);
    if (row_ok && w == 0 && lane == 0) {
      const float rs = __uint_as_float((uint32_t)(127 + e) << 23);
      row_scale[row] = ROT ? rs * kRot : rs;
    }
  }
}

template <int FMT, typename T>
__global__ void __launch_bounds__(256) dequantize_fp4_kernel(const uint8_t* __restrict__ codes, uint8_t* scales,
                                                           const float* __restrict__ row_scale, int64_t rows, int K,
                                                           int katoms, int warps, T* __restrict__ out, int64_t ld) {
  const int lane = threadIdx.x & 31;
  const int64_t gw = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  const int64_t row = gw / warps;
  if (row >= rows) return;
  const int blk = (int)(gw - row * warps) * 8 + (lane >> 2), l = lane & 3;
  uint4 c = make_uint4(0, 0, 0, 0);
  if (blk * 128 + l * 32 < K) c = __ldg(reinterpret_cast<const uint4*>(codes + row * (K >> 1) + blk * 64 + l * 16));
  const uint32_t in[4] = {c.x, c.y, c.z, c.w};
  const uint4 t = group_transpose(in, lane);
  const uint32_t w[4] = {t.x, t.y, t.z, t.w};
  if (blk * 128 >= K) return;
  uint32_t s0, s1 = 0;
  if (FMT == kFp4MX) {
    s0 = *fp4_scale_word(scales, row, katoms, blk);
  } else {
    s0 = *fp4_scale_word(scales, row, katoms, 2 * blk);
    if (2 * blk + 1 < katoms) s1 = *fp4_scale_word(scales, row, katoms, 2 * blk + 1);
  }
  const float rs = __ldg(row_scale + row);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int ch = blk * 128 + j * 32 + l * 8;
    if (ch >= K) break;
    // MX: block j; NV: block 2 j + l / 2 of the 128 channels
    float s;
    if (FMT == kFp4MX) {
      s = e8m0_value((s0 >> (8 * j)) & 0xffu);
    } else {
      const uint32_t word = j < 2 ? s0 : s1;
      s = e4m3_value((word >> (16 * (j & 1) + 8 * (l >> 1))) & 0xffu);
    }
    float v[8];
    e2m1x8_values(w[j], v);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = v[e] * s * rs;  // code times block scale is exact
    if (sizeof(T) == 2) {
      uint4 o;
      o.x = pack_bf16x2(v[0], v[1]);
      o.y = pack_bf16x2(v[2], v[3]);
      o.z = pack_bf16x2(v[4], v[5]);
      o.w = pack_bf16x2(v[6], v[7]);
      *reinterpret_cast<uint4*>(out + row * ld + ch) = o;
    } else {
      float4* d = reinterpret_cast<float4*>(out + row * ld + ch);
      d[0] = make_float4(v[0], v[1], v[2], v[3]);
      d[1] = make_float4(v[4], v[5], v[6], v[7]);
    }
  }
}

template <int FMT, bool ROT>
cudaError_t launch_quant_t(const Fp4QuantArgs& a, cudaStream_t s) {
  const int warps = (a.K + 1023) / 1024;
  if (warps > kMaxRowWarps) return cudaErrorInvalidValue;
  const int per_cta = warps >= kSmallCta ? 1 : kSmallCta / warps;
  const int64_t grid = (a.rows + per_cta - 1) / per_cta;
  if (grid > 0x7fffffff) return cudaErrorInvalidValue;
  quantize_fp4_kernel<FMT, ROT><<<(unsigned)grid, 32 * warps * per_cta, 0, s>>>(
      a.in, a.ld, a.rows, a.K, fp4_katoms(FMT, a.K), warps, a.codes, a.scales, a.row_scale);
  return cudaGetLastError();
}

template <int FMT, typename T>
cudaError_t launch_dequant_t(const Fp4DequantArgs& a, cudaStream_t s) {
  const int warps = (a.K + 1023) / 1024;
  const int64_t grid = (a.rows * warps + 7) / 8;
  if (grid > 0x7fffffff) return cudaErrorInvalidValue;
  dequantize_fp4_kernel<FMT, T><<<(unsigned)grid, 256, 0, s>>>(a.codes, a.scales, a.row_scale, a.rows, a.K,
                                                               fp4_katoms(FMT, a.K), warps, static_cast<T*>(a.out), a.ld);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_quantize_fp4(const Fp4QuantArgs& a, cudaStream_t s) {
  if (a.rows <= 0) return cudaSuccess;
  if (a.nv) return a.rotate ? launch_quant_t<kFp4NV, true>(a, s) : launch_quant_t<kFp4NV, false>(a, s);
  return a.rotate ? launch_quant_t<kFp4MX, true>(a, s) : launch_quant_t<kFp4MX, false>(a, s);
}

cudaError_t launch_dequantize_fp4(const Fp4DequantArgs& a, cudaStream_t s) {
  if (a.rows <= 0) return cudaSuccess;
  if (a.f32) return a.nv ? launch_dequant_t<kFp4NV, float>(a, s) : launch_dequant_t<kFp4MX, float>(a, s);
  return a.nv ? launch_dequant_t<kFp4NV, __nv_bfloat16>(a, s) : launch_dequant_t<kFp4MX, __nv_bfloat16>(a, s);
}

}  // namespace h3
