// Quantisation of bf16 rows to microscaled 4-bit floats (optionally rotated by
// the block-128 Hadamard transform, as the W8A8 path's inputs are), and back.
// Layout, formats and the arithmetic of a block: fp4.cuh.
//
// Both passes are bound by moving each value in and out once: 2 + 0.5 bytes a
// value and its block scale.
#include <cuda_bf16.h>

#include "fp4.cuh"
#include "kernels.cuh"

namespace h3 {
namespace {

constexpr int kMaxRowWarps = 16;  // 1024 channels each: K <= 16384
constexpr int kMaxStages = 4;

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
               ::"r"(smem_u32(dst)), "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

// Persistent CTAs of as many warps as a row of 1024 channels each takes, one
// row at a time (row = blockIdx.x + i * gridDim.x), four lanes to a block of
// 128 channels. Rows arrive by bulk copies issued `stages` rows ahead. NV needs
// the row's largest magnitude before its first code: the barrier that hands a
// slot back for refilling is also that reduction's.
//
// A lane works on four chunks, w = 0..3: unrotated chunk 4 w + l of its group's
// block (l = lane % 4; loads of a chunk take 64 contiguous bytes a group, an MX
// block is chunk w of the four lanes, an NV block that of a lane pair), rotated
// as fwht128_warp leaves them.
template <int FMT, bool ROT>
__global__ void __launch_bounds__(kMaxRowWarps * 32, 2)
    quantize_fp4_kernel(const __nv_bfloat16* __restrict__ in, int64_t ld, int64_t rows, int K, int katoms, int stages,
                        uint8_t* __restrict__ codes, uint8_t* __restrict__ scales, float* __restrict__ row_scale) {
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ uint64_t full[kMaxStages];
  __shared__ float red[2][kMaxRowWarps];
  __shared__ int fail[2];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int blk = threadIdx.x >> 2, l = threadIdx.x & 3;
  const uint32_t row_bytes = (uint32_t)K * 2u;
  if (threadIdx.x == 0) {
    for (int i = 0; i < stages; ++i) mbar_init(&full[i], 1);
    fail[0] = fail[1] = 0;
    fence_mbar_init();
  }
  __syncthreads();
  auto issue = [&](int64_t row, int slot) {
    if (row >= rows) return;
    mbar_expect_tx(&full[slot], row_bytes);
    bulk_load(ring + (uint32_t)slot * row_bytes, in + row * ld, row_bytes, &full[slot]);
  };
  if (threadIdx.x == 0)
    for (int i = 0; i < stages; ++i) issue(blockIdx.x + (int64_t)i * gridDim.x, i);
  int st = 0, phase = 0, par = 0;
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x, par ^= 1) {
    if (!mbar_wait(&full[st], phase, nullptr)) fail[par] = 1;
    // the lane's chunks; odd blocks take theirs in swapped pairs, so that the
    // two groups of a shared-memory phase take different banks
    const uint4* src = reinterpret_cast<const uint4*>(ring + (uint32_t)st * row_bytes) + blk * 16;
    const int odd = blk & 1;
    uint4 v[4];
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const int c = ROT ? (w >> 1) * 8 + 2 * l + ((w & 1) ^ odd) : 4 * (w ^ odd) + l;
      v[w] = make_uint4(0, 0, 0, 0);
      if (blk * 128 + c * 8 < K) v[w] = src[c];
    }
    float h[32], am[4], top = 0.f;
    if (ROT) fwht128_warp(v, odd, lane, h);
    // largest magnitudes of the chunks' blocks; the lanes of a block differ in
    // the lowest lane bits (rotated: in those above the two lowest)
    constexpr int kLane = ROT ? 4 : 1;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      am[w] = ROT ? amax8(h + 8 * w) : amax8(v[w]);
      am[w] = max_nan(am[w], __shfl_xor_sync(0xffffffffu, am[w], kLane));
      if (FMT == kFp4MX) am[w] = max_nan(am[w], __shfl_xor_sync(0xffffffffu, am[w], 2 * kLane));
      if (FMT == kFp4NV && finite_bits(am[w])) top = fmaxf(top, am[w]);
    }
    if (FMT == kFp4NV) {
      top = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top)));
      if (lane == 0) red[par][warp] = top;
    }
    __syncthreads();  // every thread has read the slot
    if (fail[par]) {  // a load never landed: those in flight must before the CTA's shared memory goes
      if (threadIdx.x == 0)
        for (int i = 0; i < stages && row + (int64_t)i * gridDim.x < rows; ++i) {
          mbar_wait(&full[st], phase, nullptr);
          if (++st == stages) st = 0, phase ^= 1;
        }
      return;
    }
    if (threadIdx.x == 0) {
      fail[par ^ 1] = 0;  // every thread passed the last row's check of that flag
      fence_proxy_async_smem();
      issue(row + (int64_t)stages * gridDim.x, st);
    }
    if (++st == stages) st = 0, phase ^= 1;
    int e_row = 0;
    if (FMT == kFp4NV) {
      for (int i = 0; i < warps; ++i) top = fmaxf(top, red[par][i]);
      e_row = nv_row_exponent(top);
    }
    constexpr float kRot = 0.08838834764831845f;  // 1 / sqrt(128)
    if (threadIdx.x == 0) row_scale[row] = pow2_float(e_row) * (ROT ? kRot : 1.f);
    uint32_t q[4], sc[4];
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      float u[8];
      if (!ROT) unpack_bf16x8(v[w], u);
      float* x = ROT ? h + 8 * w : u;
      q[w] = FMT == kFp4MX ? quant8_mx(x, am[w], sc[w]) : quant8_nv(x, am[w], pow2_float(-e_row), sc[w]);
    }
    uint8_t* crow = codes + row * (K >> 1);
    if (ROT) {
      // K is a multiple of 128: blocks are whole
      const int g = lane >> 2;
      const uint4 c = group_transpose<4>(q, lane);  // four chunks from 4 (g / 4) + 8 (g & 1) of block 2 l + (g / 2 & 1)
      const int b = warp * 8 + 2 * l;
      const int bs = b + ((g >> 1) & 1);
      if (bs * 128 < K) *reinterpret_cast<uint4*>(crow + bs * 64 + (g >> 2) * 16 + (g & 1) * 32) = c;
      // scale bytes of block b, then b + 1
      if (FMT == kFp4MX) {
        uint32_t s0 = sc[0] << (8 * (g >> 2)) | sc[1] << (8 * (g >> 2) + 16);
        uint32_t s1 = sc[2] << (8 * (g >> 2)) | sc[3] << (8 * (g >> 2) + 16);
        s0 |= __shfl_xor_sync(0xffffffffu, s0, 16);
        s1 |= __shfl_xor_sync(0xffffffffu, s1, 16);
        if (g < 2 && (b + g) * 128 < K) *fp4_scale_word(scales, row, katoms, b + g) = g ? s1 : s0;
      } else {
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          sc[w] <<= 8 * (g >> 1);
          sc[w] |= __shfl_xor_sync(0xffffffffu, sc[w], 8);
          sc[w] |= __shfl_xor_sync(0xffffffffu, sc[w], 16);
        }
        // lanes g = 0..3 store the words of atoms 2 b .. 2 b + 3
        const uint32_t word = g == 0 ? sc[0] : g == 1 ? sc[1] : g == 2 ? sc[2] : sc[3];
        if (g < 4 && (b + (g >> 1)) * 128 < K) *fp4_scale_word(scales, row, katoms, 2 * b + g) = word;
      }
    } else {
      const uint32_t qs[4] = {odd ? q[1] : q[0], odd ? q[0] : q[1], odd ? q[3] : q[2], odd ? q[2] : q[3]};
      const uint4 c = group_transpose(qs, lane);
      const bool ok = blk * 128 < K;
      if (ok && blk * 128 + l * 32 < K) *reinterpret_cast<uint4*>(crow + blk * 64 + l * 16) = c;
      uint32_t s = sc[0] | sc[1] << 8 | sc[2] << 16 | sc[3] << 24;
      s = __byte_perm(s, 0, odd ? 0x2301 : 0x3210);
      if (FMT == kFp4MX) {
        if (ok && l == 0) *fp4_scale_word(scales, row, katoms, blk) = s;
      } else {
        // lane 0 holds blocks 0, 2, 4, 6 of the 128 channels, lane 2 blocks 1, 3, 5, 7
        const uint32_t other = __shfl_xor_sync(0xffffffffu, s, 2);
        if (ok && l == 0) *fp4_scale_word(scales, row, katoms, 2 * blk) = __byte_perm(s, other, 0x5140);
        if (ok && l == 2 && 2 * blk + 1 < katoms)
          *fp4_scale_word(scales, row, katoms, 2 * blk + 1) = __byte_perm(other, s, 0x7362);
      }
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
  auto kern = quantize_fp4_kernel<FMT, ROT>;
  const int threads = 32 * ((a.K + 1023) / 1024);
  if (threads > 32 * kMaxRowWarps) return cudaErrorInvalidValue;
  const int stages = a.K <= 2048 ? kMaxStages : 3;
  const size_t smem = (size_t)stages * a.K * 2;
  cudaError_t e;
  if (smem > 40 * 1024 &&
      (e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem)) != cudaSuccess)
    return e;
  int dev = 0, sms = 0, per_sm = 0;
  if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
  if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
  if ((e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, threads, smem)) != cudaSuccess) return e;
  if (per_sm < 1) return cudaErrorInvalidConfiguration;
  const int64_t grid = a.rows < (int64_t)sms * per_sm ? a.rows : (int64_t)sms * per_sm;
  kern<<<(unsigned)grid, threads, smem, s>>>(a.in, a.ld, a.rows, a.K, fp4_katoms(FMT, a.K), stages, a.codes, a.scales,
                                             a.row_scale);
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
