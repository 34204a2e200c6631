// Products of microscaled 4-bit operands on the tensor cores,
// out[m, n] = ra[m] rb[n] sum_k A[m, k] B[n, k], with the block scales applied
// by the tensor core (tcgen05 block-scaled products) and the row scales, SwiGLU
// and the rounding in the epilogue.
//
// gemm_fp4_few_kernel: products of few rows, bound by reading the weight once.
// The weight rows take the product's M side (128 a CTA), the activations' rows
// its N side (16 to 128), so no tensor-core row is spent on absent rows.
//   warp 0      TMA producer: per stage 256 channels (128 bytes a row) of the
//               weight rows, of the activation rows, and their block scales
//   warp 1      TMEM allocator; copies the scale atoms to tensor memory and
//               issues the products
//   warps 2..5  epilogue (thread = weight row)
// The scales' tensor-memory columns are double-buffered per stage of 256
// channels; a buffer is rewritten once the products that read it have
// completed.
#include <cuda_bf16.h>
#include <cudaTypedefs.h>

#include "fp4.cuh"
#include "kernels.cuh"
#include "ptx.cuh"

namespace h3 {
namespace {

constexpr int kBlockK = 256;     // channels per stage: 128 bytes of codes a row
constexpr int kRowBytes = 128;
constexpr int kTile = 128 * kRowBytes;

__host__ __device__ constexpr int atoms_per_stage(int fmt) { return kBlockK / fp4_atom_channels(fmt); }

// ------------------------------------------------------------------ few rows
constexpr int kFewThreads = 192;

template <int FMT, int NT, int NW>
struct FewCfg {
  static constexpr int kAtoms = atoms_per_stage(FMT);
  static constexpr int kScaleBytes = kAtoms * 512;
  static constexpr int kStageBytes = NW * (kTile + kScaleBytes) + NT * kRowBytes + kScaleBytes;
  static constexpr int kStages = 4;
  static constexpr int kAccCols = NW * NT;
  static constexpr int kScaleCols = kAtoms * (NW + 1) * 4;  // one buffer
  static constexpr int kCols = kAccCols + 2 * kScaleCols;
  static constexpr int kTmemCols = kCols <= 64 ? 64 : kCols <= 128 ? 128 : kCols <= 256 ? 256 : 512;
  static constexpr size_t kSmem = 1024 + (size_t)kStages * kStageBytes + 256;
};

template <int FMT, int NT, int NW, typename T>
__global__ void __launch_bounds__(kFewThreads)
    gemm_fp4_few_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                        const __grid_constant__ CUtensorMap tmWS, const __grid_constant__ CUtensorMap tmXS,
                        const Fp4GemmArgs p) {
  using Cfg = FewCfg<FMT, NT, NW>;
  constexpr int kStages = Cfg::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + (((smem_u32(smem_raw) + 1023u) & ~1023u) - smem_u32(smem_raw));
  // stage: NW weight tiles, the activation tile, NW weight scale sets, the activation scales
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + (size_t)kStages * Cfg::kStageBytes);
  uint64_t* empty = full + kStages;
  uint64_t* sfree = empty + kStages;  // scale buffers
  uint64_t* tfull = sfree + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(tfull + 1);
  int* abort = reinterpret_cast<int*>(tfull + 2);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n0 = blockIdx.x * 128, m0 = blockIdx.y * NT;
  const int num_kb = (p.K + kBlockK - 1) / kBlockK;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    mbar_init(&sfree[0], 1);
    mbar_init(&sfree[1], 1);
    mbar_init(tfull, 1);
    *abort = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, Cfg::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  volatile int* vabort = abort;

  if (warp == 0) {
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      int issued = 0;
      for (int kb = 0; kb < num_kb; ++kb) {
        if (!mbar_wait(&empty[stage], phase ^ 1, vabort)) {
          *vabort = 1;
          break;
        }
        uint8_t* st = smem + (size_t)stage * Cfg::kStageBytes;
        mbar_expect_tx(&full[stage], Cfg::kStageBytes);
#pragma unroll
        for (int i = 0; i < NW; ++i) {
          const int row = n0 + i * p.N;  // SwiGLU: the up rows follow the N gate rows
          tma_load_2d(st + i * kTile, &tmW, &full[stage], kb * kRowBytes, row);
          tma_load_3d(st + NW * kTile + NT * kRowBytes + i * Cfg::kScaleBytes, &tmWS, &full[stage], 0,
                      kb * Cfg::kAtoms, row >> 7);
        }
        tma_load_2d(st + NW * kTile, &tmX, &full[stage], kb * kRowBytes, m0);
        tma_load_3d(st + NW * (kTile + Cfg::kScaleBytes) + NT * kRowBytes, &tmXS, &full[stage], 0, kb * Cfg::kAtoms,
                    m0 >> 7);
        ++issued;
        if (++stage == kStages) {
          stage = 0;
          phase ^= 1;
        }
      }
      // the last loads issued must have landed before the CTA exits
      const int outstanding = issued < kStages ? issued : kStages;
      for (int i = 0; i < outstanding; ++i) {
        if (--stage < 0) {
          stage = kStages - 1;
          phase ^= 1;
        }
        mbar_wait(&full[stage], phase, nullptr);
      }
    }
  } else if (warp == 1) {
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int kb = 0; kb < num_kb; ++kb) {
      const int buf = kb & 1;
      if (!mbar_wait_warp(&full[stage], phase, vabort) ||
          (kb >= 2 && !mbar_wait_warp(&sfree[buf], (uint32_t)((kb >> 1) - 1) & 1, vabort))) {
        if (lane == 0) *vabort = 1;
        ok = false;
        break;
      }
      tc_fence_after();
      const uint32_t st = smem_u32(smem) + (uint32_t)stage * Cfg::kStageBytes;
      const uint32_t xs = st + NW * kTile, ws0 = xs + NT * kRowBytes, xs0 = ws0 + NW * Cfg::kScaleBytes;
      const uint32_t sc = tmem + Cfg::kAccCols + buf * Cfg::kScaleCols;
      const int steps = min(4, (p.K - kb * kBlockK + 63) / 64);
#pragma unroll
      for (int a = 0; a < Cfg::kAtoms; ++a) {
        if (a * fp4_atom_channels(FMT) >= steps * 64) break;
        const uint32_t col = sc + a * (NW + 1) * 4;
#pragma unroll
        for (int i = 0; i < NW; ++i)
          tmem_cp_scales_w(col + i * 4, scale_atom_desc(ws0 + i * Cfg::kScaleBytes + a * 512));
        tmem_cp_scales_w(col + NW * 4, scale_atom_desc(xs0 + a * 512));
      }
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        if (s >= steps) break;
        const int a = FMT == kFp4NV ? s : s >> 1;
        const uint32_t id = make_idesc_fp4(128, NT, FMT == kFp4MX, FMT == kFp4MX ? (s & 1) * 2 : 0);
        const uint32_t col = sc + a * (NW + 1) * 4;
        const uint64_t xd = sw128_desc(xs + s * 32, 16);
#pragma unroll
        for (int i = 0; i < NW; ++i)
          mma_fp4_ss_w<FMT == kFp4NV>(tmem + i * NT, sw128_desc(st + i * kTile + s * 32, 16), xd, id, col + i * 4,
                                      col + NW * 4, (kb | s) != 0);
      }
      mma_commit_w(&sfree[buf]);
      mma_commit_w(&empty[stage]);
      if (++stage == kStages) {
        stage = 0;
        phase ^= 1;
      }
    }
    // the accumulators are complete (or, after a failed wait, everything
    // issued has ended) once tfull flips
    mma_commit_w(tfull);
    mbar_wait(tfull, 0, nullptr);
    if (!ok && lane == 0) *vabort = 1;
  } else {
    if (mbar_wait(tfull, 0, nullptr) && !*vabort) {
      tc_fence_after();
      const int quad = warp & 3;
      const uint32_t acc = tmem + ((uint32_t)(quad * 32) << 16);
      const int n = n0 + quad * 32 + lane;
      const bool n_ok = n < p.N;
      const float rb = n_ok ? __ldg(p.b_row + n) : 0.f;
      const float ru = NW == 2 && n_ok ? __ldg(p.b_row + p.N + n) : 0.f;
#pragma unroll 1
      for (int c = 0; c < NT; c += 16) {
        if (m0 + c >= p.M) break;
        uint32_t g[16], u[16];
        tmem_ld16(acc + c, g);
        if (NW == 2) tmem_ld16(acc + NT + c, u);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int64_t m = m0 + c + i;
          if (m < p.M && n_ok) {
            const float ra = __ldg(p.a_row + m);
            float v = __uint_as_float(g[i]) * ra * rb;
            if (NW == 2) v = v / (1.f + __expf(-v)) * (__uint_as_float(u[i]) * ra * ru);
            if (sizeof(T) == 2)
              reinterpret_cast<__nv_bfloat16*>(p.out)[m * p.ld + n] = __float2bfloat16_rn(v);
            else
              reinterpret_cast<float*>(p.out)[m * p.ld + n] = v;
          }
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, Cfg::kTmemCols);
}

// ------------------------------------------------------------------ host
bool codes_map(PFN_cuTensorMapEncodeTiled_v12000 encode, CUtensorMap* m, const void* ptr, int64_t rows, int K,
               int box_rows) {
  cuuint64_t dims[2] = {(cuuint64_t)(K / 2), (cuuint64_t)rows};
  cuuint64_t strides[1] = {(cuuint64_t)(K / 2)};
  cuuint32_t box[2] = {(cuuint32_t)kRowBytes, (cuuint32_t)box_rows};
  cuuint32_t estr[2] = {1, 1};
  return encode(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(ptr), dims, strides, box, estr,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The scale atoms as [row block][atom along K][128 words].
bool scales_map(PFN_cuTensorMapEncodeTiled_v12000 encode, CUtensorMap* m, const void* ptr, int64_t rows, int K, int fmt) {
  const cuuint64_t katoms = (cuuint64_t)fp4_katoms(fmt, K);
  cuuint64_t dims[3] = {128, katoms, (cuuint64_t)((rows + 127) / 128)};
  cuuint64_t strides[2] = {512, 512 * katoms};
  cuuint32_t box[3] = {128, (cuuint32_t)atoms_per_stage(fmt), 1};
  cuuint32_t estr[3] = {1, 1, 1};
  return encode(m, CU_TENSOR_MAP_DATA_TYPE_UINT32, 3, const_cast<void*>(ptr), dims, strides, box, estr,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct Maps {
  CUtensorMap a, b, as, bs;
};

template <int FMT, int NT, int NW, typename T>
cudaError_t launch_few_t(const Fp4GemmArgs& p, const Maps& m, cudaStream_t s) {
  using Cfg = FewCfg<FMT, NT, NW>;
  auto k = gemm_fp4_few_kernel<FMT, NT, NW, T>;
  cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Cfg::kSmem);
  if (e != cudaSuccess) return e;
  const dim3 grid((p.N + 127) / 128, (unsigned)((p.M + NT - 1) / NT));
  k<<<grid, kFewThreads, Cfg::kSmem, s>>>(m.b, m.a, m.bs, m.as, p);
  return cudaGetLastError();
}

template <int FMT, int NT>
cudaError_t launch_few(const Fp4GemmArgs& p, const Maps& m, cudaStream_t s) {
  if (p.swiglu)
    return p.f32 ? launch_few_t<FMT, NT, 2, float>(p, m, s) : launch_few_t<FMT, NT, 2, __nv_bfloat16>(p, m, s);
  return p.f32 ? launch_few_t<FMT, NT, 1, float>(p, m, s) : launch_few_t<FMT, NT, 1, __nv_bfloat16>(p, m, s);
}

template <int FMT>
cudaError_t launch_fmt(const Fp4GemmArgs& p, PFN_cuTensorMapEncodeTiled_v12000 encode, cudaStream_t s) {
  Maps m;
  const int nt = p.M <= 16 ? 16 : p.M <= 32 ? 32 : p.M <= 64 ? 64 : 128;
  const int64_t b_rows = p.swiglu ? 2 * (int64_t)p.N : p.N;
  if (!codes_map(encode, &m.a, p.a_codes, p.M, p.K, nt) || !codes_map(encode, &m.b, p.b_codes, b_rows, p.K, 128) ||
      !scales_map(encode, &m.as, p.a_scales, p.M, p.K, FMT) || !scales_map(encode, &m.bs, p.b_scales, b_rows, p.K, FMT))
    return cudaErrorInvalidValue;
  switch (nt) {
    case 16: return launch_few<FMT, 16>(p, m, s);
    case 32: return launch_few<FMT, 32>(p, m, s);
    case 64: return launch_few<FMT, 64>(p, m, s);
    default: return launch_few<FMT, 128>(p, m, s);
  }
}

}  // namespace

cudaError_t launch_gemm_fp4(const Fp4GemmArgs& p, PFN_cuTensorMapEncodeTiled_v12000 encode, int num_sms,
                            cudaStream_t s) {
  if (p.M <= 0 || p.N <= 0) return cudaSuccess;
  (void)num_sms;
  return p.nv ? launch_fmt<kFp4NV>(p, encode, s) : launch_fmt<kFp4MX>(p, encode, s);
}

}  // namespace h3
