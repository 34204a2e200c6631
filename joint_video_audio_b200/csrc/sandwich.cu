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
// Bound by moving x, y, x1 and h once: 8 bytes a value (6.5 with a 4-bit h),
// against 14 bytes a value of gate, gain, shift and scale if each row read
// them. So a persistent CTA takes a contiguous slice of the rows, visits them
// grouped by (tag, tidx), and a thread keeps its eight channels' vectors in
// registers while the key stays. Rows arrive by bulk copies issued several
// rows ahead; two rows of a key are worked on together, and their two or three
// reductions are one barrier each.
//
// Measured (32768 x 5376): bf16 h 229 us (6.1 TB/s, 94 % of the copy rate), MX h
// 285 us, NV h 330 us, NV rotated 422 us (330 to 420 instructions a warp and row at
// 2.2 a cycle: 21 warps, all an SM's registers hold, wait for one another's
// sums). One row at a time took 287 us, vectors read per row 557 us.
#include <cuda_bf16.h>

#include "fp4.cuh"
#include "kernels.cuh"

namespace h3 {
namespace {

constexpr int kMaxStages = 8;
constexpr int kSortRows = 256;  // rows grouped by key at a time

__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w; v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ uint4 pack8(const float* v) {
  return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
}

// Sum (IS_MAX: maximum of non-negative values) over the warp.
template <bool IS_MAX>
__device__ __forceinline__ float warp_reduce(float v) {
  if (IS_MAX) return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(v)));
#pragma unroll
  for (int m = 16; m; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
  return v;
}
// The same of R rows over the CTA; one barrier. `red` has a slot per warp, of 32,
// those past the last warp zero, and is written again after another barrier at
// least. The sums of two rows share the exchanges: after the first one a lane carries
// row lane % 2, of itself and its neighbour (bf16 h, 32768 x 5376: 242 -> 229 us).
template <bool IS_MAX, int R>
__device__ __forceinline__ void cta_reduce(float (&v)[R], float (*red)[32]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if constexpr (R == 2 && !IS_MAX) {
    const bool odd = lane & 1;
    float t = (odd ? v[1] : v[0]) + __shfl_xor_sync(0xffffffffu, odd ? v[0] : v[1], 1);
#pragma unroll
    for (int m = 2; m < 32; m <<= 1) t += __shfl_xor_sync(0xffffffffu, t, m);
    if (lane < 2) red[lane][warp] = t;
    __syncthreads();
    // 16 lanes to a row
    t = (&red[0][0])[2 * lane] + (&red[0][0])[2 * lane + 1];
#pragma unroll
    for (int m = 1; m < 16; m <<= 1) t += __shfl_xor_sync(0xffffffffu, t, m);
    v[0] = __shfl_sync(0xffffffffu, t, 0);
    v[1] = __shfl_sync(0xffffffffu, t, 16);
  } else {
#pragma unroll
    for (int r = 0; r < R; ++r) v[r] = warp_reduce<IS_MAX>(v[r]);
    if (lane == 0)
#pragma unroll
      for (int r = 0; r < R; ++r) red[r][warp] = v[r];
    __syncthreads();
#pragma unroll
    for (int r = 0; r < R; ++r) v[r] = warp_reduce<IS_MAX>(red[r][lane]);
  }
}
// Sum of the squares of eight values.
__device__ __forceinline__ float squares8(const float (&v)[8]) {
  uint64_t s2 = f2_mul(f2_pack(v[0], v[1]), f2_pack(v[0], v[1]));
#pragma unroll
  for (int e = 2; e < 8; e += 2) s2 = f2_fma(f2_pack(v[e], v[e + 1]), f2_pack(v[e], v[e + 1]), s2);
  float a, b;
  f2_unpack(s2, a, b);
  return a + b;
}
// v[e] = a[e] * s * b[e] + c[e]
__device__ __forceinline__ void scale_fma8(float (&v)[8], const float (&a)[8], float s, const float (&b)[8],
                                           const float (&c)[8]) {
#pragma unroll
  for (int e = 0; e < 8; e += 2)
    f2_unpack(f2_fma(f2_mul(f2_pack(a[e], a[e + 1]), f2_pack(s, s)), f2_pack(b[e], b[e + 1]), f2_pack(c[e], c[e + 1])),
              v[e], v[e + 1]);
}

// Unnormalised Hadamard transform of 128 channels held eight to a lane by 16
// lanes.
__device__ __forceinline__ void fwht128_lanes(float (&h)[8], int lane) {
#pragma unroll
  for (int b = 1; b < 8; b <<= 1)
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (!(e & b)) {
        const float u = h[e], w = h[e + b];
        h[e] = u + w;
        h[e + b] = u - w;
      }
#pragma unroll
  for (int m = 1; m < 16; m <<= 1) {
    const float sg = (lane & m) ? -1.f : 1.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) h[e] = fmaf(sg, h[e], __shfl_xor_sync(0xffffffffu, h[e], m));
  }
}

// A thread's eight channels of the key's vectors.
struct Vectors {
  float g[8], sh[8], sc[8];  // gate * gain, shift, 1 + scale
};

// HOUT: 0 no h, 1 bf16, 2 MX, 3 NV. R rows of a key at a time, so that their
// loads, shuffles and barriers overlap. CPT chunks of eight channels per thread
// (chunk threadIdx.x + i * blockDim.x); the vectors stay in registers for one
// chunk and are read per row for two (then R is 1).
template <int HOUT, bool ROT, int CPT, int MAXT, int R>
__global__ void __launch_bounds__(MAXT) sandwich_kernel(const SandwichArgs a, int stages, int katoms) {
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ uint64_t full[kMaxStages];
  __shared__ float red[2][3][R][32];
  __shared__ int keys[kSortRows];
  __shared__ uint16_t ord[kSortRows];
  __shared__ int fail[2];  // by parity: a thread that is ahead sets the next rows'
  const int lane = threadIdx.x & 31;
  const int nchunk = a.C >> 3;
  const uint32_t row_bytes = (uint32_t)a.C * 2u;
  const int64_t per = (a.rows + gridDim.x - 1) / gridDim.x;
  const int64_t s0 = (int64_t)blockIdx.x * per;
  const int64_t s1 = s0 + per < a.rows ? s0 + per : a.rows;
  pdl_launch();
  if (s0 >= s1) return;
  if (threadIdx.x == 0) {
    for (int i = 0; i < stages; ++i) mbar_init(&full[i], 1);
    fail[0] = fail[1] = 0;
    fence_mbar_init();
  }
  for (int i = threadIdx.x; i < 2 * 3 * R * 32; i += blockDim.x) (&red[0][0][0][0])[i] = 0.f;
  pdl_wait();
  const float inv_c = 1.f / (float)a.C;
  Vectors vec[CPT];
  int cur = -2;  // key of the vectors held
  auto load_vectors = [&](int key) {
    const float* gate = a.table + ((int64_t)key * 6 + a.gate_idx) * a.C;
    const float* mod = HOUT ? a.norm_table + ((int64_t)key * 6 + a.shift_idx) * a.C : nullptr;
#pragma unroll
    for (int i = 0; i < CPT; ++i) {
      const int c = threadIdx.x + i * blockDim.x;
#pragma unroll
      for (int e = 0; e < 8; ++e) vec[i].g[e] = vec[i].sh[e] = 0.f, vec[i].sc[e] = 1.f;
      if (key >= 0 && c < nchunk) {
        load8(gate + c * 8, vec[i].g);
        if (HOUT) {
          load8(mod + c * 8, vec[i].sh);
          load8(mod + a.C + c * 8, vec[i].sc);
#pragma unroll
          for (int e = 0; e < 8; ++e) vec[i].sc[e] += 1.f;
        }
        if (a.post_gain) {
          float pg[8];
          unpack_bf16x8(__ldg(reinterpret_cast<const uint4*>(a.post_gain) + c), pg);
#pragma unroll
          for (int e = 0; e < 8; ++e) vec[i].g[e] *= pg[e];
        }
      }
    }
  };
  int st = 0, phase = 0, par = 0;  // ring slot and its phase, row parity
  for (int64_t c0 = s0; c0 < s1; c0 += kSortRows) {
    const int n = (int)(s1 - c0 < kSortRows ? s1 - c0 : kSortRows);
    __syncthreads();  // the last group's order is no longer read; the barriers are initialised
    for (int i = threadIdx.x; i < n; i += blockDim.x) {
      const int tg = a.tag[c0 + i], ti = a.tidx[c0 + i];
      keys[i] = (tg >= 0 && tg < a.n_tags && ti >= 0 && ti < a.n_t) ? tg * a.n_t + ti : -1;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += blockDim.x) {
      const int ki = keys[i];
      int rank = 0;
      for (int j = 0; j < n; ++j) {
        const int kj = keys[j];
        rank += (kj < ki) || (kj == ki && j < i);
      }
      ord[rank] = (uint16_t)i;
    }
    __syncthreads();
    // the group's i-th row into a slot
    auto issue = [&](int i, int slot) {
      if (i >= n) return;
      const int64_t at = (c0 + ord[i]) * a.C;
      uint8_t* dst = ring + (uint32_t)slot * 2 * row_bytes;
      mbar_expect_tx(&full[slot], 2 * row_bytes);
      bulk_load(dst, a.x + at, row_bytes, &full[slot]);
      bulk_load(dst + row_bytes, a.y + at, row_bytes, &full[slot]);
    };
    if (threadIdx.x == 0) {
      fence_proxy_async_smem();  // the slots' last generic reads come before these copies
      for (int i = 0, slot = st; i < stages; ++i, slot = slot + 1 == stages ? 0 : slot + 1) issue(i, slot);
    }
    for (int k = 0; k < n;) {
      const int key = keys[ord[k]];
      // rows k .. k + cnt - 1, all of this key (a slot past them is zeros)
      int cnt = 1;
      if (R == 2 && k + 1 < n && keys[ord[k + 1]] == key) cnt = 2;
      int64_t at[R];
#pragma unroll
      for (int r = 0; r < R; ++r) at[r] = (c0 + ord[r < cnt ? k + r : k]) * a.C;
      float(&rd)[3][R][32] = red[par];
      if (key != cur) {
        if (CPT == 1) load_vectors(key);
        cur = key;
      }
      float x[R][CPT][8], y[R][CPT][8], ss[R];
#pragma unroll
      for (int r = 0; r < R; ++r) {
        int slot = st + r, ph = phase;
        if (slot >= stages) slot -= stages, ph ^= 1;
        ss[r] = 0.f;
        if (r < cnt && !mbar_wait(&full[slot], ph, nullptr)) fail[par] = 1;
#pragma unroll
        for (int i = 0; i < CPT; ++i) {
          const int c = threadIdx.x + i * blockDim.x;
          uint4 xv = make_uint4(0, 0, 0, 0), yv = xv;
          if (r < cnt && c < nchunk) {
            const uint4* src = reinterpret_cast<const uint4*>(ring + (uint32_t)slot * 2 * row_bytes);
            xv = src[c];
            yv = src[nchunk + c];
          }
          unpack_bf16x8(xv, x[r][i]);
          unpack_bf16x8(yv, y[r][i]);
          if (a.post_norm) ss[r] += squares8(y[r][i]);
        }
      }
      // a barrier: every thread has read the slots, which are refilled, or the
      // CTA stops because a load never landed
      cta_reduce<false, R>(ss, rd[0]);
      if (fail[par]) {
        if (threadIdx.x == 0) {
          atomicOr(a.err, kErrTimeoutStream);
          for (int i = k; i < k + stages && i < n; ++i) {
            mbar_wait(&full[st], phase, nullptr);
            if (++st == stages) st = 0, phase ^= 1;
          }
        }
        return;
      }
      if (threadIdx.x == 0) {
        fence_proxy_async_smem();
        issue(k + stages, st);
        if (cnt == 2) issue(k + 1 + stages, st + 1 == stages ? 0 : st + 1);
      }
      k += cnt;
      st += cnt;
      if (st >= stages) st -= stages, phase ^= 1;
      par ^= 1;
      if (CPT > 1) load_vectors(key);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        float rp = a.branch_scale;
        if (a.post_norm) rp *= rsqrtf(fmaf(ss[r], inv_c, a.post_eps));
        ss[r] = 0.f;
#pragma unroll
        for (int i = 0; i < CPT; ++i) {
          const int c = threadIdx.x + i * blockDim.x;
          if (key >= 0)  // (a zero gate times an infinite y would not leave x as it is)
            scale_fma8(x[r][i], vec[i].g, rp, y[r][i], x[r][i]);
          if (r < cnt && c < nchunk) reinterpret_cast<uint4*>(a.x_out + at[r])[c] = pack8(x[r][i]);
          ss[r] += squares8(x[r][i]);
        }
      }
      if (HOUT == 0) continue;
      cta_reduce<false, R>(ss, rd[1]);
      float am[R][CPT], top[R];
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const float rstd = rsqrtf(fmaf(ss[r], inv_c, a.norm_eps));
        top[r] = 0.f;
#pragma unroll
        for (int i = 0; i < CPT; ++i) {
          const int c = threadIdx.x + i * blockDim.x;
          scale_fma8(x[r][i], x[r][i], rstd, vec[i].sc, vec[i].sh);
          if (HOUT == 1) {
            if (r < cnt && c < nchunk) reinterpret_cast<uint4*>(a.h + at[r])[c] = pack8(x[r][i]);
            continue;
          }
          if (ROT) fwht128_lanes(x[r][i], lane);
          float& m = am[r][i];
          m = amax8(x[r][i]);
          m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, 1));
          if (HOUT == 2) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, 2));
          if (HOUT == 3 && finite_bits(m)) top[r] = fmaxf(top[r], m);
        }
      }
      if (HOUT <= 1) continue;
      if (HOUT == 3) cta_reduce<true, R>(top, rd[2]);
      constexpr float kRot = 0.08838834764831845f;  // 1 / sqrt(128)
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const int64_t row = c0 + ord[r < cnt ? k - cnt + r : k - cnt];
        const int e_row = HOUT == 3 ? nv_row_exponent(top[r]) : 0;
        const int lift = HOUT == 3 && e_row < kNvSmall ? kNvLift : 0;
        if (threadIdx.x == 0 && r < cnt) a.row_scale[row] = pow2_float(e_row) * (ROT ? kRot : 1.f);
#pragma unroll
        for (int i = 0; i < CPT; ++i) {
          const int c = threadIdx.x + i * blockDim.x;
          uint32_t sc, q;
          if (HOUT == 2) {
            q = quant8_mx(x[r][i], mx_scale(am[r][i], sc));
          } else {
            if (lift) nv_lift8(x[r][i]);
            q = quant8_nv(x[r][i], nv_scale(am[r][i], e_row, lift, sc));
          }
          if (r < cnt && c < nchunk) reinterpret_cast<uint32_t*>(a.codes + (at[r] >> 1))[c] = q;
          // the four scale bytes of an atom's row, gathered from the lanes of 4
          // blocks (MX: 16 lanes, four to a block; NV: 8 lanes, two to a block)
          constexpr int kBlk = HOUT == 2 ? 4 : 2;
          sc <<= 8 * ((lane / kBlk) & 3);
          sc |= __shfl_xor_sync(0xffffffffu, sc, kBlk);
          sc |= __shfl_xor_sync(0xffffffffu, sc, 2 * kBlk);
          if (r < cnt && c < nchunk && lane % (4 * kBlk) == 0)
            *fp4_scale_word(a.scales, row, katoms, c / (4 * kBlk)) = sc;
        }
      }
    }
  }
}

template <int HOUT, bool ROT, int CPT, int MAXT, int R>
cudaError_t launch_t(const SandwichArgs& a, int num_sms, cudaStream_t s) {
  constexpr auto kern = sandwich_kernel<HOUT, ROT, CPT, MAXT, R>;
  const int threads = ((a.C / 8 + CPT - 1) / CPT + 31) / 32 * 32;
  // up to eight rows ahead, three of the widest
  const size_t stage = (size_t)a.C * 4;
  int stages = (int)((a.C <= 2048 ? 32 * 1024 : 192 * 1024) / stage);
  stages = stages > kMaxStages ? kMaxStages : stages;
  const size_t smem = stages * stage;
  const cudaError_t e = smem > 40 * 1024 ? allow_smem<kern>(smem) : cudaSuccess;
  if (e != cudaSuccess) return e;
  const int64_t most = (int64_t)num_sms * resident_ctas<kern>(threads, smem);
  const int64_t grid = a.rows < most ? a.rows : most;
  ChainedLaunch l(dim3((unsigned)grid), threads, smem, s);
  return cudaLaunchKernelEx(&l.cfg, kern, a, stages, HOUT >= 2 ? fp4_katoms(HOUT == 3 ? kFp4NV : kFp4MX, a.C) : 0);
}

// Thread bounds by width, so that narrow rows leave registers for the vectors.
template <int HOUT, bool ROT>
cudaError_t launch_w(const SandwichArgs& a, int num_sms, cudaStream_t s) {
  if (a.C <= 2048) return launch_t<HOUT, ROT, 1, 256, 2>(a, num_sms, s);
  if (a.C <= 5632) return launch_t<HOUT, ROT, 1, 704, 2>(a, num_sms, s);
  if (a.C <= 8192) return launch_t<HOUT, ROT, 1, 1024, 1>(a, num_sms, s);
  return launch_t<HOUT, ROT, 2, 1024, 1>(a, num_sms, s);
}

}  // namespace

cudaError_t launch_sandwich(const SandwichArgs& a, int num_sms, cudaStream_t s) {
  if (a.rows <= 0) return cudaSuccess;
  if (a.C % 128 || a.C > 16384) return cudaErrorInvalidValue;
  if (a.norm_table == nullptr) return launch_w<0, false>(a, num_sms, s);
  if (a.h) return launch_w<1, false>(a, num_sms, s);
  if (a.nv) return a.rotate ? launch_w<3, true>(a, num_sms, s) : launch_w<3, false>(a, num_sms, s);
  return a.rotate ? launch_w<2, true>(a, num_sms, s) : launch_w<2, false>(a, num_sms, s);
}

}  // namespace h3
