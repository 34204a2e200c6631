// The norms after and before a block, fused with its gate and residual
// (reading of "MiniMaxH3Transformer3DModel", diffusers API page: AdaLN gates
// and pre-norms per modality tag; the norm of the block's output is this
// library's option):
//   p  = y, or rmsnorm(y, post_eps) * post_gain
//   x1 = x + branch_scale * gate * p
//   h  = rmsnorm(x1, norm_eps) * (1 + scale) + shift
// with gate / shift / scale of the row's (tag, tidx), zero for padding and for
// indices outside the table. h comes from the unrounded x1 (one rounding
// fewer than a pass over the stored x1) and leaves as bf16 or as the 4-bit
// operand of the next product, quantised from its fp32 values (fp4.cuh).
//
// Bound by moving x, y, x1 and h once: 8 bytes a value (6.5 with a 4-bit h). A
// row is spread over whole warps and lives in registers across its two or
// three reductions.
#include <cuda_bf16.h>

#include "fp4.cuh"
#include "kernels.cuh"

namespace h3 {
namespace {

constexpr int kMaxRowWarps = 16;
constexpr int kSmallCta = 8;

// Sum (IS_MAX: max of non-negative values) over the row's warps.
template <bool IS_MAX>
__device__ __forceinline__ float row_reduce(float v, float* red, int warp, int w, int warps) {
  if (IS_MAX) {
    v = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(v)));
  } else {
#pragma unroll
    for (int m = 16; m; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
  }
  if (warps == 1) return v;
  if ((threadIdx.x & 31) == 0) red[warp] = v;
  __syncthreads();
  float r = red[warp - w];
  for (int i = 1; i < warps; ++i) r = IS_MAX ? fmaxf(r, red[warp - w + i]) : r + red[warp - w + i];
  return r;
}

__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w; v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ uint4 pack8(const float* v) {
  return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
}

// HOUT: 0 no h, 1 bf16, 2 MX, 3 NV.
template <int HOUT, bool ROT>
__global__ void __launch_bounds__(kMaxRowWarps * 32) sandwich_kernel(const SandwichArgs a, int warps, int katoms) {
  __shared__ float red[3][kMaxRowWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int per_cta = (blockDim.x >> 5) / warps;
  const int64_t row = (int64_t)blockIdx.x * per_cta + warp / warps;
  const int w = warp % warps;
  const int blk = w * 8 + (lane >> 2), l = lane & 3;
  const bool ok = row < a.rows && blk * 128 < a.C;  // C is a multiple of 128: a group is all in or all out
  const float *gate = nullptr, *mod = nullptr;
  if (row < a.rows) {
    const int tg = a.tag[row], ti = a.tidx[row];
    if (tg >= 0 && tg < a.n_tags && ti >= 0 && ti < a.n_t) {
      const int64_t key = ((int64_t)tg * a.n_t + ti) * 6;
      gate = a.table + (key + a.gate_idx) * a.C;
      if (HOUT) mod = a.norm_table + (key + a.shift_idx) * a.C;  // shift, then scale
    }
  }
  const int64_t base = row * a.C + blk * 128 + l * 8;
  float x[32], y[32];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint4 xv = make_uint4(0, 0, 0, 0), yv = xv;
    if (ok) {
      xv = *reinterpret_cast<const uint4*>(a.x + base + 32 * j);
      yv = *reinterpret_cast<const uint4*>(a.y + base + 32 * j);
    }
    unpack_bf16x8(xv, x + 8 * j);
    unpack_bf16x8(yv, y + 8 * j);
  }
  float rp = a.branch_scale;
  if (a.post_norm) {
    float ss = 0.f;
#pragma unroll
    for (int e = 0; e < 32; ++e) ss = fmaf(y[e], y[e], ss);
    rp *= rsqrtf(row_reduce<false>(ss, red[0], warp, w, warps) / (float)a.C + a.post_eps);
  }
  if (ok) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int c = blk * 128 + j * 32 + l * 8;
      if (gate) {
        float g[8];
        load8(gate + c, g);
        if (a.post_gain) {
          float pg[8];
          unpack_bf16x8(__ldg(reinterpret_cast<const uint4*>(a.post_gain + c)), pg);
#pragma unroll
          for (int e = 0; e < 8; ++e) g[e] *= pg[e];
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) x[8 * j + e] = fmaf(g[e] * rp, y[8 * j + e], x[8 * j + e]);
      }
      *reinterpret_cast<uint4*>(a.x_out + base + 32 * j) = pack8(x + 8 * j);
    }
  }
  if (HOUT == 0) return;
  float ss = 0.f;
#pragma unroll
  for (int e = 0; e < 32; ++e) ss = fmaf(x[e], x[e], ss);
  const float rstd = rsqrtf(row_reduce<false>(ss, red[1], warp, w, warps) / (float)a.C + a.norm_eps);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int c = blk * 128 + j * 32 + l * 8;
    if (mod && ok) {
      float sh[8], sc[8];
      load8(mod + c, sh);
      load8(mod + a.C + c, sc);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[8 * j + e] = fmaf(x[8 * j + e] * rstd, 1.f + sc[e], sh[e]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) x[8 * j + e] *= rstd;
    }
  }
  if (HOUT == 1) {
    if (ok)
#pragma unroll
      for (int j = 0; j < 4; ++j) *reinterpret_cast<uint4*>(a.h + base + 32 * j) = pack8(x + 8 * j);
    return;
  }
  constexpr int FMT = HOUT == 3 ? kFp4NV : kFp4MX;
  constexpr float kRot = 0.08838834764831845f;  // 1 / sqrt(128)
  if (ROT) fwht128_group(x, lane);
  float am[4];
  chunk_amax(x, am);
  const Fp4Row o{a.codes + row * (a.C >> 1), a.scales, row, a.C, katoms};
  uint32_t q[4], sc;
  float rs = 1.f;
  if (FMT == kFp4MX) {
    quant_mx(x, am, q, sc);
  } else {
    const float top = row_reduce<true>(nv_block_amax(am), red[2], warp, w, warps);
    const int e = nv_row_exponent(top);
    quant_nv(x, am, e, q, sc);
    rs = __uint_as_float((uint32_t)(127 + e) << 23);
  }
  store_group<FMT>(ok, o, blk, lane, q, sc);
  if (row < a.rows && w == 0 && lane == 0) a.row_scale[row] = ROT ? rs * kRot : rs;
}

template <int HOUT, bool ROT>
cudaError_t launch_t(const SandwichArgs& a, cudaStream_t s) {
  const int warps = (a.C + 1023) / 1024;
  if (warps > kMaxRowWarps) return cudaErrorInvalidValue;
  const int per_cta = warps >= kSmallCta ? 1 : kSmallCta / warps;
  const int64_t grid = (a.rows + per_cta - 1) / per_cta;
  if (grid > 0x7fffffff) return cudaErrorInvalidValue;
  sandwich_kernel<HOUT, ROT>
      <<<(unsigned)grid, 32 * warps * per_cta, 0, s>>>(a, warps, HOUT >= 2 ? fp4_katoms(HOUT == 3 ? kFp4NV : kFp4MX, a.C) : 0);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_sandwich(const SandwichArgs& a, cudaStream_t s) {
  if (a.rows <= 0) return cudaSuccess;
  if (a.norm_table == nullptr) return launch_t<0, false>(a, s);
  if (a.h) return launch_t<1, false>(a, s);
  if (a.nv) return a.rotate ? launch_t<3, true>(a, s) : launch_t<3, false>(a, s);
  return a.rotate ? launch_t<2, true>(a, s) : launch_t<2, false>(a, s);
}

}  // namespace h3
