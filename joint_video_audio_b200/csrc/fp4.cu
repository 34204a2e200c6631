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
constexpr int kGroupWarps = 4;    // of a group of narrow rows
constexpr int kMaxStages = 4;

__device__ __forceinline__ float warp_max(float v) {  // of values that are not negative
  return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(v)));
}

// Persistent CTAs, R rows at a time (rows grp R .. of grp = blockIdx.x + i *
// gridDim.x), four lanes to a block of 128 channels. Rows arrive by bulk copies
// issued `stages` groups ahead. R is 1 and a CTA as many warps as a row of 1024
// channels each takes, or, GROUPED, rows of up to 512 channels share 4 warps,
// `pitch` blocks (2 or 4) to a row. NV needs the row's largest magnitude before
// its first code: the barrier that hands a slot back for refilling is also that
// reduction's; narrow rows lie inside a warp.
//
// Measured (32768 x 14336, 2.53 / 2.56 bytes a value): MX 205 us (5.8 TB/s, 89 %
// of the copy rate), MX rotated 209 us, NV 219 us, NV rotated 285 us, the last
// two by their instructions and the latencies between them (2.6 a cycle of 4). One row per CTA at a time
// without the ring took 240, 338, 379 and 467 us. Grouped (131072 x 256): MX 22
// us, NV 27 us, one row at a time 47 and 64; groups of two rows of 5376: MX 86 us
// as without, NV 127 instead of 98.
//
// A lane works on 32 channels: unrotated the l-th 32 of its block (an MX
// block, two NV blocks; its 16-byte reads of the row in an order that gives
// each eight lanes distinct banks), rotated as fwht128_warp leaves them.
template <int FMT, bool ROT, bool GROUPED>
__global__ void __launch_bounds__(GROUPED ? kGroupWarps * 32 : kMaxRowWarps * 32, GROUPED ? 7 : 2)
    quantize_fp4_kernel(const __nv_bfloat16* __restrict__ in, int64_t ld, int64_t rows, int K, int katoms, int stages,
                        int pitch, uint8_t* __restrict__ codes, uint8_t* __restrict__ scales, float* __restrict__ row_scale,
                        int* err) {
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ uint64_t full[kMaxStages];
  __shared__ float red[2][kMaxRowWarps];
  __shared__ int fail[2];  // by parity: a thread that is ahead sets the next group's
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int l = threadIdx.x & 3, g = lane >> 2;
  const int R = GROUPED ? kGroupWarps * 8 / pitch : 1;
  const uint32_t row_bytes = (uint32_t)K * 2u;
  const int64_t groups = GROUPED ? (rows + R - 1) / R : rows;
  // row of the group and block of the row: as the lane loads them, and, rotated,
  // of the values it then holds (those of block b and the next)
  const int f_in = threadIdx.x >> 2, f = ROT ? warp * 8 + 2 * l : f_in;
  const int r_in = GROUPED ? f_in / pitch : 0, blk = GROUPED ? f_in % pitch : f_in;
  const int r = GROUPED ? f / pitch : 0, b = GROUPED ? f % pitch : f;
  pdl_launch();
  if (threadIdx.x == 0) {
    for (int i = 0; i < stages; ++i) mbar_init(&full[i], 1);
    fail[0] = fail[1] = 0;
    fence_mbar_init();
  }
  __syncthreads();
  pdl_wait();
  auto rows_of = [&](int64_t grp) { return !GROUPED || rows - grp * R > R ? R : (int)(rows - grp * R); };
  auto issue = [&](int64_t grp, int slot) {
    if (grp >= groups) return;
    const int n = rows_of(grp);
    uint8_t* dst = ring + (uint32_t)(slot * R) * row_bytes;
    const __nv_bfloat16* src = in + grp * R * ld;
    mbar_expect_tx(&full[slot], n * row_bytes);
    if (!GROUPED || ld == K)
      bulk_load(dst, src, n * row_bytes, &full[slot]);
    else
      for (int i = 0; i < n; ++i) bulk_load(dst + i * row_bytes, src + i * ld, row_bytes, &full[slot]);
  };
  if (threadIdx.x == 0)
    for (int i = 0; i < stages; ++i) issue(blockIdx.x + (int64_t)i * gridDim.x, i);
  int st = 0, phase = 0, par = 0;
  for (int64_t grp = blockIdx.x; grp < groups; grp += gridDim.x, par ^= 1) {
    if (!mbar_wait(&full[st], phase, nullptr)) fail[par] = 1;
    const int n = rows_of(grp);
    // the lane's chunks: slot w holds chunk w ^ perm of its 32 channels;
    // rotated, odd blocks take theirs in swapped pairs
    const uint4* src = reinterpret_cast<const uint4*>(ring + (uint32_t)(st * R + r_in) * row_bytes);
    const int perm = ROT ? blk & 1 : (threadIdx.x >> 1) & 3;
    uint4 v[4];
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const int c = ROT ? blk * 16 + (w >> 1) * 8 + 2 * l + ((w & 1) ^ perm) : blk * 16 + l * 4 + (w ^ perm);
      v[w] = make_uint4(0, 0, 0, 0);
      if ((!GROUPED || r_in < n) && c * 8 < K) v[w] = src[c];
    }
    // the largest magnitudes of its two groups of 16 channels; of the MX block
    // that each belongs to
    float h[32], am[2], top = 0.f;
    if (ROT) fwht128_warp(v, perm, lane, h);
#pragma unroll
    for (int i = 0; i < 2; ++i)
      am[i] = ROT ? max_nan(amax8(h + 16 * i), amax8(h + 16 * i + 8)) : max_nan(amax8(v[2 * i]), amax8(v[2 * i + 1]));
    if (FMT == kFp4MX) {
      if (ROT) {
        am[0] = max_nan(am[0], __shfl_xor_sync(0xffffffffu, am[0], 4));
        am[1] = max_nan(am[1], __shfl_xor_sync(0xffffffffu, am[1], 4));
      } else {
        am[0] = max_nan(am[0], am[1]);
      }
    } else {
      if (finite_bits(am[0])) top = am[0];
      if (finite_bits(am[1])) top = fmaxf(top, am[1]);
      if (GROUPED) {  // over the lanes of the row: rotated, all g and the l of its pairs of blocks
#pragma unroll
        for (int m = 1; m < 32; m <<= 1)
          if (ROT ? m >= 4 || 2 * m < pitch : m < 4 * pitch) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, m));
      } else {
        top = warp_max(top);
        if (lane == 0) red[par][warp] = top;
      }
    }
    __syncthreads();  // every thread has read the slot
    if (fail[par]) {  // a load never landed: those in flight must before the CTA's shared memory goes
      if (threadIdx.x == 0) {
        atomicOr(err, kErrTimeoutStream);
        for (int i = 0; i < stages && grp + (int64_t)i * gridDim.x < groups; ++i) {
          mbar_wait(&full[st], phase, nullptr);
          if (++st == stages) st = 0, phase ^= 1;
        }
      }
      return;
    }
    if (threadIdx.x == 0) {
      fence_proxy_async_smem();
      issue(grp + (int64_t)stages * gridDim.x, st);
    }
    if (++st == stages) st = 0, phase ^= 1;
    int e_row = 0;
    if (FMT == kFp4NV) {
      if (!GROUPED) top = warp_max(lane < (int)(blockDim.x >> 5) ? red[par][lane] : 0.f);
      e_row = nv_row_exponent(top);
    }
    const int64_t row = grp * R + r;
    const bool live = !GROUPED || r < n;
    constexpr float kRot = 0.08838834764831845f;  // 1 / sqrt(128)
    if (GROUPED ? live && b == 0 && (ROT ? g : l) == 0 : threadIdx.x == 0) row_scale[row] = pow2_float(e_row) * (ROT ? kRot : 1.f);
    uint32_t q[4], sc[2];
    const int lift = e_row < kNvSmall ? kNvLift : 0;
    float inv = 0.f;
    NvScale nv{};
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      if (FMT == kFp4NV && w % 2 == 0) nv = nv_scale(am[w / 2], e_row, lift, sc[w / 2]);
      if (FMT == kFp4MX && (w == 0 || (ROT && w == 2))) inv = mx_scale(am[w / 2], sc[w / 2]);
      float u[8];
      if (!ROT) unpack_bf16x8(v[w], u);
      float* x = ROT ? h + 8 * w : u;
      if (FMT == kFp4NV && lift) nv_lift8(x);
      q[w] = FMT == kFp4MX ? quant8_mx(x, inv) : quant8_nv(x, nv);
    }
    uint8_t* crow = codes + row * (K >> 1);
    if (ROT) {
      // K is a multiple of 128: blocks are whole. 16 channels each of blocks b, b + 1
      if (live && b * 128 < K) *reinterpret_cast<uint2*>(crow + b * 64 + g * 8) = make_uint2(q[0], q[1]);
      if (live && b * 128 + 128 < K) *reinterpret_cast<uint2*>(crow + b * 64 + 64 + g * 8) = make_uint2(q[2], q[3]);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if (FMT == kFp4MX) {  // byte g / 2 of the block's word
          sc[i] <<= 8 * (g >> 1);
          sc[i] |= __shfl_xor_sync(0xffffffffu, sc[i], 8);
          sc[i] |= __shfl_xor_sync(0xffffffffu, sc[i], 16);
        } else {  // byte g % 4 of the block's word g / 4
          sc[i] <<= 8 * (g & 3);
          sc[i] |= __shfl_xor_sync(0xffffffffu, sc[i], 4);
          sc[i] |= __shfl_xor_sync(0xffffffffu, sc[i], 8);
        }
      }
      const int i = g & 1;  // lanes g = 0, 1 store block b's, b + 1's (first) word, for NV g = 4, 5 the second
      if ((g & 2) == 0 && (FMT == kFp4NV || g < 4) && live && (b + i) * 128 < K)
        *fp4_scale_word(scales, row, katoms, FMT == kFp4MX ? b + i : 2 * (b + i) + (g >> 2)) = i ? sc[1] : sc[0];
    } else {
      // the words back in the channels' order
      const bool s1 = perm & 1, s2 = perm & 2;
      const uint32_t a0 = s1 ? q[1] : q[0], a1 = s1 ? q[0] : q[1], a2 = s1 ? q[3] : q[2], a3 = s1 ? q[2] : q[3];
      const bool ok = live && blk * 128 + l * 32 < K;
      if (ok)
        *reinterpret_cast<uint4*>(crow + blk * 64 + l * 16) = s2 ? make_uint4(a2, a3, a0, a1) : make_uint4(a0, a1, a2, a3);
      if (FMT == kFp4MX) {
        uint32_t s = (ok ? sc[0] : 1u) << (8 * l);  // (past K: the smallest scale)
        s |= __shfl_xor_sync(0xffffffffu, s, 1);
        s |= __shfl_xor_sync(0xffffffffu, s, 2);
        if (l == 0 && ok) *fp4_scale_word(scales, row, katoms, blk) = s;
      } else {
        uint32_t s = (s2 ? sc[1] | sc[0] << 8 : sc[0] | sc[1] << 8) << (16 * (l & 1));
        s |= __shfl_xor_sync(0xffffffffu, s, 1);
        if ((l & 1) == 0 && ok) *fp4_scale_word(scales, row, katoms, 2 * blk + (l >> 1)) = s;
      }
    }
  }
}

// A 4 x 4 transpose of words among four neighbouring lanes: lane q of them gets
// word q of each, in lane order.
__device__ __forceinline__ uint4 group_transpose(const uint32_t (&w)[4], int lane) {
  const bool o1 = lane & 1, o2 = lane & 2;
  uint32_t a0 = w[0], a1 = w[1], a2 = w[2], a3 = w[3];
  uint32_t s0 = __shfl_xor_sync(0xffffffffu, o1 ? a0 : a1, 1);
  uint32_t s1 = __shfl_xor_sync(0xffffffffu, o1 ? a2 : a3, 1);
  a0 = o1 ? s0 : a0;
  a2 = o1 ? s1 : a2;
  a1 = o1 ? a1 : s0;
  a3 = o1 ? a3 : s1;
  s0 = __shfl_xor_sync(0xffffffffu, o2 ? a0 : a2, 2);
  s1 = __shfl_xor_sync(0xffffffffu, o2 ? a1 : a3, 2);
  a0 = o2 ? s0 : a0;
  a1 = o2 ? s1 : a1;
  a2 = o2 ? a2 : s0;
  a3 = o2 ? a3 : s1;
  return make_uint4(a0, a1, a2, a3);
}

// 32 channels a lane, read as one 16-byte piece of codes and transposed among
// four lanes so that the values leave in 64-byte runs. Measured (32768 x 14336):
// to bf16 186 us MX, 190 us NV, 97 and 96 % of the copy rate, to fp32 322 us (404
// with a lane's eight values in one run). Blocks of all rows are numbered
// through: a warp per 1024 channels of a row took 82 us for 32768 x 5376, not 76,
// and 47 us for 131072 x 256, not 21.
template <int FMT, typename T>
__global__ void __launch_bounds__(256) dequantize_fp4_kernel(const uint8_t* __restrict__ codes, uint8_t* scales,
                                                           const float* __restrict__ row_scale, int64_t rows, int K,
                                                           int katoms, int blocks, T* __restrict__ out, int64_t ld) {
  const int lane = threadIdx.x & 31;
  // four lanes to a block of 128 channels
  const int64_t gb = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 2;
  const int64_t row = gb / blocks;
  pdl_launch();
  pdl_wait();
  const int blk = (int)(gb - row * blocks), l = lane & 3;
  uint4 c = make_uint4(0, 0, 0, 0);
  if (row < rows && blk * 128 + l * 32 < K)
    c = __ldg(reinterpret_cast<const uint4*>(codes + row * (K >> 1) + blk * 64 + l * 16));
  const uint32_t in[4] = {c.x, c.y, c.z, c.w};
  const uint4 t = group_transpose(in, lane);
  uint32_t w[4] = {t.x, t.y, t.z, t.w};
  // The lane's 32 values are four runs of eight, of channels 32 j + 8 l ..; in
  // fp32 eight half runs, of 32 j + 4 l .. and 16 behind, so that four lanes'
  // 16-byte stores lie side by side.
  if (sizeof(T) == 4) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int from = (lane & 28) + (l >> 1);
      const uint32_t a = __shfl_sync(0xffffffffu, w[j], from), b = __shfl_sync(0xffffffffu, w[j], from + 2);
      w[j] = __byte_perm(a, b, (l & 1) ? 0x7632 : 0x5410);
    }
  }
  if (row >= rows) return;
  uint32_t s0, s1 = 0;
  if (FMT == kFp4MX) {
    s0 = *fp4_scale_word(scales, row, katoms, blk);
  } else {
    s0 = *fp4_scale_word(scales, row, katoms, 2 * blk);
    if (2 * blk + 1 < katoms) s1 = *fp4_scale_word(scales, row, katoms, 2 * blk + 1);
  }
  float rs = __ldg(row_scale + row), eighth = 1.f;
  // MX: a code times its block's scale, up to 6 * 2^127, may pass the largest float
  // though the row's scale (1 / sqrt(128) where rotated) brings it back
  if (FMT == kFp4MX && fabsf(rs) < 1.f) rs *= 8.f, eighth = 0.125f;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (blk * 128 + j * 32 >= K) break;  // (K is a multiple of 32)
    // MX: block j; NV: blocks 2 j and 2 j + 1 of the 128 channels
    float sc[2];
    if (FMT == kFp4MX) {
      sc[0] = sc[1] = e8m0_value((s0 >> (8 * j)) & 0xffu) * eighth;
    } else {
      const uint32_t pair = (j < 2 ? s0 : s1) >> (16 * (j & 1));
      sc[0] = e4m3_value((pair >> (sizeof(T) == 2 ? 8 * (l >> 1) : 0)) & 0xffu);
      sc[1] = sizeof(T) == 2 ? sc[0] : e4m3_value((pair >> 8) & 0xffu);
    }
    float v[8];
    e2m1x8_values(w[j], v);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = v[e] * sc[e >> 2] * rs;  // code times block scale is exact
    T* o = out + row * ld + blk * 128 + j * 32;
    if (sizeof(T) == 2) {
      *reinterpret_cast<uint4*>(o + l * 8) =
          make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
    } else {
      *reinterpret_cast<float4*>(o + l * 4) = make_float4(v[0], v[1], v[2], v[3]);
      *reinterpret_cast<float4*>(o + 16 + l * 4) = make_float4(v[4], v[5], v[6], v[7]);
    }
  }
}

template <int FMT, bool ROT, bool GROUPED>
cudaError_t launch_quant_t(const Fp4QuantArgs& a, int num_sms, cudaStream_t s) {
  constexpr auto kern = quantize_fp4_kernel<FMT, ROT, GROUPED>;
  const int pitch = a.K <= 256 ? 2 : 4, R = GROUPED ? kGroupWarps * 8 / pitch : 1;
  const int threads = 32 * (GROUPED ? kGroupWarps : (a.K + 1023) / 1024);
  if (threads > 32 * kMaxRowWarps) return cudaErrorInvalidValue;
  const int stages = a.K <= 2048 ? kMaxStages : 3;
  const size_t smem = (size_t)stages * R * a.K * 2;
  const cudaError_t e = smem > 40 * 1024 ? allow_smem<kern>(smem) : cudaSuccess;
  if (e != cudaSuccess) return e;
  const int64_t most = (int64_t)num_sms * resident_ctas<kern>(threads, smem);
  const int64_t groups = (a.rows + R - 1) / R, grid = groups < most ? groups : most;
  ChainedLaunch l(dim3((unsigned)grid), threads, smem, s);
  return cudaLaunchKernelEx(&l.cfg, kern, a.in, a.ld, a.rows, a.K, fp4_katoms(FMT, a.K), stages, pitch, a.codes, a.scales,
                            a.row_scale, a.err);
}

template <int FMT, bool ROT>
cudaError_t launch_quant(const Fp4QuantArgs& a, int num_sms, cudaStream_t s) {
  return a.K <= 512 ? launch_quant_t<FMT, ROT, true>(a, num_sms, s) : launch_quant_t<FMT, ROT, false>(a, num_sms, s);
}

template <int FMT, typename T>
cudaError_t launch_dequant_t(const Fp4DequantArgs& a, cudaStream_t s) {
  const int blocks = (a.K + 127) / 128;
  const int64_t grid = (a.rows * blocks + 63) / 64;
  if (grid > 0x7fffffff) return cudaErrorInvalidValue;
  ChainedLaunch l(dim3((unsigned)grid), 256, 0, s);
  return cudaLaunchKernelEx(&l.cfg, dequantize_fp4_kernel<FMT, T>, a.codes, a.scales, a.row_scale, a.rows, a.K,
                            fp4_katoms(FMT, a.K), blocks, static_cast<T*>(a.out), a.ld);
}

}  // namespace

cudaError_t launch_quantize_fp4(const Fp4QuantArgs& a, int num_sms, cudaStream_t s) {
  if (a.rows <= 0) return cudaSuccess;
  if (a.nv) return a.rotate ? launch_quant<kFp4NV, true>(a, num_sms, s) : launch_quant<kFp4NV, false>(a, num_sms, s);
  return a.rotate ? launch_quant<kFp4MX, true>(a, num_sms, s) : launch_quant<kFp4MX, false>(a, num_sms, s);
}

cudaError_t launch_dequantize_fp4(const Fp4DequantArgs& a, cudaStream_t s) {
  if (a.rows <= 0) return cudaSuccess;
  if (a.f32) return a.nv ? launch_dequant_t<kFp4NV, float>(a, s) : launch_dequant_t<kFp4MX, float>(a, s);
  return a.nv ? launch_dequant_t<kFp4NV, __nv_bfloat16>(a, s) : launch_dequant_t<kFp4MX, __nv_bfloat16>(a, s);
}

}  // namespace h3
