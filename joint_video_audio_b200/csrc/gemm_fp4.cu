// Products of microscaled 4-bit operands on the tensor cores,
// out[m, n] = ra[m] rb[n] sum_k A[m, k] B[n, k], with the block scales applied
// by the tensor core (tcgen05 block-scaled products) and the row scales, SwiGLU
// and the rounding in the epilogue.
//
// gemm_fp4_few_kernel: products of few rows, bound by reading the weight once.
// The weight rows take the product's M side (128 a CTA), the activations' rows
// its N side (16 to 128), so no tensor-core row is spent on absent rows. K is
// split over a cluster of up to six CTAs when the weight rows alone do not
// occupy the SMs; the partial sums meet in distributed shared memory, added in
// the order of K.
//   warp 0      TMA producer: per stage 256 channels (128 bytes a row) of the
//               weight rows, of the activation rows, and their block scales
//   warp 1      TMEM allocator; copies the scale atoms to tensor memory and
//               issues the products
//   warps 2..5  epilogue (thread = weight row)
// The scales' tensor-memory columns are double-buffered per stage; a buffer is
// rewritten once the products that read it have completed.
//
// Measured (weights cold, launches of a graph): 1 x 5376 x 7168 NV 6.8 us, 64 x
// 21504 x 5376 MX 15.5 us (4.3 TB/s), 1 x 2 x 14336 x 5376 NV SwiGLU 16.8 us (5.2
// TB/s), 128 x 21504 x 5376 MX 17.4 us. 4 x 256 x 768 takes 2.6 us; of the first 3.7
// us are the loads (3.3 at the copy rate), 1 us the sums' meeting. Unsplit and with
// an election per instruction it took 23 us. The last with a row's scale fetched as
// the row is stored, one row at a time, 22 us; four at a time where K is split, and
// the sums lie in other SMs, 128 x 5376 x 7168 took 13.6 us, not 11.5.
//
// gemm_fp4_pair_kernel: products of many rows, see there; takes_few() chooses.
#include <cuda_bf16.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <type_traits>

#include "fp4.cuh"
#include "kernels.cuh"
#include "ptx.cuh"

namespace h3 {
namespace {

constexpr int kBlockK = 256;     // channels per stage: 128 bytes of codes a row
constexpr int kRowBytes = 128;
constexpr int kTile = 128 * kRowBytes;

__host__ __device__ constexpr int atoms_per_stage(int fmt) { return kBlockK / fp4_atom_channels(fmt); }

// silu(g) * u = g e^min(g, 0) / (1 + e^-|g|) * u: the denominator lies in [1, 2],
// where an approximate reciprocal is good to a unit of the last place (of 1 + e^-g
// it becomes 0 below g = -87.3). e^-|g| = 2^t, t = -|g| log2 e; rounding t and log2 e
// costs up to 2^-17 of it, which a bf16 output does not show, so that only an fp32
// one adds what they left out. Measured (4001 x 2 x 14336 x 5376 NV): bf16 261 us,
// fp32 319; as g / (1 + e^-g), 100 units of the last place off at -85, 258 and 298;
// with expf 275 and 320.
__device__ __forceinline__ float exp2_approx(float x) {  // (subnormal results too)
  float r;
  asm("ex2.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
template <typename T>
__device__ __forceinline__ float swiglu(float g, float u) {
  constexpr float kLog2e = 1.4426950408889634f, kLog2eRest = (float)(1.4426950408889634 - (double)kLog2e);
  const float a = fminf(fabsf(g), 128.f);  // e^-128 is 0 (and an infinity would leave a NaN below)
  const float t = -a * kLog2e;
  float e = exp2_approx(t);
  if (sizeof(T) == 4) e = fmaf(e, 0.6931471805599453f * fmaf(-a, kLog2eRest, fmaf(-a, kLog2e, -t)), e);
  return (g < 0.f ? g * e : g) * rcp_approx(1.f + e) * u;
}

// A wait ran out: the CTA's others stop, and the host can learn of it.
__device__ __forceinline__ void give_up(volatile int* abort, int* err) {
  *abort = 1;
  atomicOr(err, kErrTimeoutGemm);
}

// ------------------------------------------------------------------ few rows
constexpr int kFewThreads = 192;
constexpr int kMaxSplit = 6;  // CTAs that share a product's K

template <int FMT, int NT, int NW>
struct FewCfg {
  static constexpr int kAtoms = atoms_per_stage(FMT);
  static constexpr int kScaleBytes = kAtoms * 512;
  static constexpr int kStageBytes = NW * (kTile + kScaleBytes) + NT * kRowBytes + kScaleBytes;
  // up to four, as long as an SM has room for two CTAs (of SwiGLU, whose stages
  // are twice as large, one); a fifth gained nothing at 16 rows
  static constexpr int kFit = (228 * 1024 / (NW == 1 ? 2 : 1) - 1024 - 1280) / kStageBytes;
  static constexpr int kStages = kFit < 4 ? kFit : 4;
  static constexpr int kAccCols = NW * NT;
  static constexpr int kSlotCols = kAtoms * (NW + 1) * 4;
  static constexpr int kCols = kAccCols + 2 * kSlotCols;
  static constexpr int kTmemCols = kCols <= 64 ? 64 : kCols <= 128 ? 128 : kCols <= 256 ? 256 : 512;
  static constexpr size_t kSmem = 1024 + (size_t)kStages * kStageBytes + 256;
  static constexpr int kPerSm = 2 * (kSmem + 1024) <= 228 * 1024 ? 2 : 1;  // resident CTAs
  static_assert(NW * NT * 512 <= kStages * kStageBytes, "the partial sums take the stages' place");
};

// A whole stage's tensor work, issued by one lane (see issue_pair_stage): the
// scale copies (atoms of NW weight tiles and of the activations at sd, sd +
// kScaleBytes, ..) to the slot at column sc, the four products of 64 channels a
// weight tile into the accumulators at column d, and the commits.
#define H3_ARGS                                                                                              \
  ::"r"(d), "r"(sc), "l"(wd), "l"(xd), "l"(sd), "r"(id0), "r"(id1), "r"(accumulate), "r"(smem_u32(sfree)),   \
      "r"(smem_u32(empty)), "r"(d + NT)                                                                      \
      : "memory"
#define H3_CP(T, X) "add.u32 t, %1, " #T ";\n\tadd.s64 x, %4, " #X ";\n\t" \
                    "@e tcgen05.cp.cta_group::1.32x128b.warpx4 [t], x;\n\t"
#define H3_MM(OP, D, ID, SA, SB, WK, XK, P)                                                       \
  "add.u32 t, %1, " #SA ";\n\tadd.u32 u, %1, " #SB ";\n\t"                                      \
  "add.s64 x, %2, " #WK ";\n\tadd.s64 y, %3, " #XK ";\n\t"                                      \
  "@e tcgen05.mma.cta_group::1." OP " [" D "], x, y, " ID ", [t], [u], " P ";\n\t"
#define H3_BEGIN                                                                        \
  "{\n\t.reg .pred p, q, e;\n\t.reg .b32 t, u;\n\t.reg .b64 x, y;\n\t" H3_ELECT_PRED \
  "setp.ne.b32 p, %7, 0;\n\tsetp.eq.b32 q, 0, 0;\n\t"
#define H3_END                                                                                 \
  "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%8];\n\t"         \
  "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%9];\n\t}"
#define H3_NV "kind::mxf4nvf4.block_scale.scale_vec::4X"
#define H3_MX "kind::mxf4.block_scale.scale_vec::2X"
template <int FMT, int NT, int NW>
__device__ __forceinline__ void issue_few_stage(uint32_t d, uint32_t sc, uint64_t wd, uint64_t xd, uint64_t sd,
                                                uint32_t accumulate, uint64_t* sfree, uint64_t* empty) {
  constexpr uint32_t id0 = make_idesc_fp4(128, NT, FMT == kFp4MX, 0), id1 = make_idesc_fp4(128, NT, FMT == kFp4MX, 2);
  static_assert(kTile / 16 == 1024, "the second weight tile's offset below");
  if (FMT == kFp4NV && NW == 1) {
    asm volatile(H3_BEGIN                                                            //
                 H3_CP(0, 0) H3_CP(4, 128) H3_MM(H3_NV, "%0", "%5", 0, 4, 0, 0, "p")      //
                 H3_CP(8, 32) H3_CP(12, 160) H3_MM(H3_NV, "%0", "%5", 8, 12, 2, 2, "q")   //
                 H3_CP(16, 64) H3_CP(20, 192) H3_MM(H3_NV, "%0", "%5", 16, 20, 4, 4, "q") //
                 H3_CP(24, 96) H3_CP(28, 224) H3_MM(H3_NV, "%0", "%5", 24, 28, 6, 6, "q") H3_END H3_ARGS);
  } else if (FMT == kFp4NV) {
    asm volatile(H3_BEGIN                                                                                          //
                 H3_CP(0, 0) H3_CP(4, 128) H3_CP(8, 256) H3_MM(H3_NV, "%0", "%5", 0, 8, 0, 0, "p")                 //
                 H3_MM(H3_NV, "%10", "%5", 4, 8, 1024, 0, "p")                                                     //
                 H3_CP(12, 32) H3_CP(16, 160) H3_CP(20, 288) H3_MM(H3_NV, "%0", "%5", 12, 20, 2, 2, "q")           //
                 H3_MM(H3_NV, "%10", "%5", 16, 20, 1026, 2, "q")                                                   //
                 H3_CP(24, 64) H3_CP(28, 192) H3_CP(32, 320) H3_MM(H3_NV, "%0", "%5", 24, 32, 4, 4, "q")           //
                 H3_MM(H3_NV, "%10", "%5", 28, 32, 1028, 4, "q")                                                   //
                 H3_CP(36, 96) H3_CP(40, 224) H3_CP(44, 352) H3_MM(H3_NV, "%0", "%5", 36, 44, 6, 6, "q")           //
                 H3_MM(H3_NV, "%10", "%5", 40, 44, 1030, 6, "q") H3_END H3_ARGS);
  } else if (NW == 1) {
    asm volatile(H3_BEGIN                                                                                              //
                 H3_CP(0, 0) H3_CP(4, 64) H3_MM(H3_MX, "%0", "%5", 0, 4, 0, 0, "p")                                    //
                 H3_MM(H3_MX, "%0", "%6", 0, 4, 2, 2, "q")                                                             //
                 H3_CP(8, 32) H3_CP(12, 96) H3_MM(H3_MX, "%0", "%5", 8, 12, 4, 4, "q")                                 //
                 H3_MM(H3_MX, "%0", "%6", 8, 12, 6, 6, "q") H3_END H3_ARGS);
  } else {
    asm volatile(H3_BEGIN                                                                                              //
                 H3_CP(0, 0) H3_CP(4, 64) H3_CP(8, 128) H3_MM(H3_MX, "%0", "%5", 0, 8, 0, 0, "p")                      //
                 H3_MM(H3_MX, "%10", "%5", 4, 8, 1024, 0, "p") H3_MM(H3_MX, "%0", "%6", 0, 8, 2, 2, "q")               //
                 H3_MM(H3_MX, "%10", "%6", 4, 8, 1026, 2, "q")                                                         //
                 H3_CP(12, 32) H3_CP(16, 96) H3_CP(20, 160) H3_MM(H3_MX, "%0", "%5", 12, 20, 4, 4, "q")                //
                 H3_MM(H3_MX, "%10", "%5", 16, 20, 1028, 4, "q") H3_MM(H3_MX, "%0", "%6", 12, 20, 6, 6, "q")           //
                 H3_MM(H3_MX, "%10", "%6", 16, 20, 1030, 6, "q") H3_END H3_ARGS);
  }
}
#undef H3_ARGS
#undef H3_CP
#undef H3_MM
#undef H3_BEGIN
#undef H3_END

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
  // this CTA's share of K, in stages
  const int all_kb = (p.K + kBlockK - 1) / kBlockK;
  const int split = gridDim.z, part = blockIdx.z;
  const int kb0 = all_kb * part / split, kb1 = all_kb * (part + 1) / split;

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
  pdl_launch();  // (behind the allocation: a later kernel's CTA may wait for these columns, but cannot hold them)
  pdl_wait();

  if (warp == 0) {
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      int issued = 0;
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!mbar_wait(&empty[stage], phase ^ 1, vabort)) {
          give_up(vabort, p.err);
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
        if (!mbar_wait(&full[stage], phase, nullptr)) give_up(vabort, p.err);
      }
    }
  } else if (warp == 1) {
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int i = 0; i < kb1 - kb0; ++i) {
      const int buf = i & 1;
      const uint32_t sfree_parity = ((i >> 1) & 1) ^ 1;
      const bool r0 = mbar_try_wait(&full[stage], phase), r1 = mbar_try_wait(&sfree[buf], sfree_parity);
      if (!__all_sync(0xffffffffu, r0 && r1) &&
          !(mbar_wait_warp(&full[stage], phase, vabort) && mbar_wait_warp(&sfree[buf], sfree_parity, vabort))) {
        if (lane == 0) give_up(vabort, p.err);
        ok = false;
        break;
      }
      tc_fence_after();
      const uint32_t st = smem_u32(smem) + (uint32_t)stage * Cfg::kStageBytes;
      const uint32_t xs = st + NW * kTile, ws0 = xs + NT * kRowBytes;
      const uint32_t sc = tmem + Cfg::kAccCols + buf * Cfg::kSlotCols;
      const int left = p.K - (kb0 + i) * kBlockK;
      if (left > kBlockK - 64) {
        issue_few_stage<FMT, NT, NW>(tmem, sc, sw128_desc(st, 16), sw128_desc(xs, 16), scale_atom_desc(ws0), i != 0,
                                     &sfree[buf], &empty[stage]);
      } else {  // the last stage of a K that does not fill it
        const int steps = (left + 63) / 64;
#pragma unroll 1
        for (int s = 0; s < steps; ++s) {
          const int a = s * 64 / fp4_atom_channels(FMT);
          const uint32_t col = sc + a * (NW + 1) * 4;
          if (s * 64 % fp4_atom_channels(FMT) == 0)
            for (int j = 0; j <= NW; ++j)
              tmem_cp_scales_w(col + j * 4, scale_atom_desc(ws0 + j * Cfg::kScaleBytes + a * 512));
          const uint32_t id = make_idesc_fp4(128, NT, FMT == kFp4MX, FMT == kFp4MX ? (s & 1) * 2 : 0);
          for (int j = 0; j < NW; ++j)
            mma_fp4_ss_w<FMT == kFp4NV>(tmem + j * NT, sw128_desc(st + j * kTile + s * 32, 16), sw128_desc(xs + s * 32, 16),
                                        id, col + j * 4, col + NW * 4, (i | s) != 0);
        }
        mma_commit_w(&sfree[buf]);
        mma_commit_w(&empty[stage]);
      }
      if (++stage == kStages) {
        stage = 0;
        phase ^= 1;
      }
    }
    // the accumulators are complete (or, after a failed wait, everything
    // issued has ended) once tfull flips
    mma_commit_w(tfull);
    mbar_wait(tfull, 0, nullptr);
    if (!ok && lane == 0) give_up(vabort, p.err);
  }
  __syncwarp();
  // ------------------------------------------------------------------ epilogue
  // sums [NW * NT][128 weight rows] in the place of the stages (every load has
  // landed and been read); then each CTA of the cluster adds its share of the
  // activation rows, a warp a row, four weight rows a lane
  float* sums = reinterpret_cast<float*>(smem);
  bool good = false;
  // a warp's rows of the tile: the CTA's share, every fourth of it; lane i keeps
  // the i-th one's scale, the lane's weight rows' scales come before the products too
  const int rows = (int)(p.M - m0 < NT ? p.M - m0 : NT);
  const int first = part * 4 + warp - 2, step = 4 * split, n = n0 + 4 * lane;
  const int count = rows > first ? (rows - first + step - 1) / step : 0;
  float ra = 0.f;
  float4 rb = make_float4(0.f, 0.f, 0.f, 0.f), ru = rb;
  if (warp >= 2) {
    if (lane < count) ra = __ldg(p.a_row + m0 + first + lane * step);
    if (n < p.N) {  // N is a multiple of 8
      rb = __ldg(reinterpret_cast<const float4*>(p.b_row + n));
      if (NW == 2) ru = __ldg(reinterpret_cast<const float4*>(p.b_row + p.N + n));
    }
    good = __all_sync(0xffffffffu, mbar_wait(tfull, 0, nullptr) && !*vabort);
    if (!good && lane == 0) give_up(vabort, p.err);
    tc_fence_after();
    const int quad = warp & 3;
    const uint32_t acc = tmem + ((uint32_t)(quad * 32) << 16);
    if (good) {
#pragma unroll 1
      for (int c = 0; c < NW * NT; c += 16) {
        if ((NW == 1 || c < NT ? c : c - NT) >= rows) continue;
        uint32_t g[16];
        tmem_ld16(acc + c, g);
#pragma unroll
        for (int i = 0; i < 16; ++i) sums[(c + i) * 128 + quad * 32 + lane] = __uint_as_float(g[i]);
      }
    }
  }
  __syncwarp();
  if (split > 1)
    cluster_sync();
  else
    __syncthreads();
  if (good) {
    const uint32_t at = smem_u32(sums) + lane * 16;
    // a row's sums over the parts, in their order
    auto add_parts = [&](int row) {
      float4 v[kMaxSplit];
#pragma unroll
      for (int q = 0; q < kMaxSplit; ++q)
        if (q < split) v[q] = ld_cluster_f32x4(mapa_shared(at + row * 512, q));
#pragma unroll
      for (int q = 1; q < kMaxSplit; ++q)
        if (q < split) v[0].x += v[q].x, v[0].y += v[q].y, v[0].z += v[q].z, v[0].w += v[q].w;
      return v[0];
    };
    // R rows at a time
    auto store_rows = [&](auto at_once) {
      constexpr int R = decltype(at_once)::value;
#pragma unroll 1
      for (int i = 0; i < count; i += R) {
        float4 g[R], u[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const int c = first + (i + r < count ? i + r : i) * step;
          g[r] = add_parts(c);
          if (NW == 2) u[r] = add_parts(NT + c);
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const float rar = __shfl_sync(0xffffffffu, ra, (i + r) & 31);
          if (i + r >= count || n >= p.N) continue;
          float4 v = make_float4(g[r].x * rar * rb.x, g[r].y * rar * rb.y, g[r].z * rar * rb.z, g[r].w * rar * rb.w);
          if (NW == 2)
            v = make_float4(swiglu<T>(v.x, u[r].x * rar * ru.x), swiglu<T>(v.y, u[r].y * rar * ru.y),
                            swiglu<T>(v.z, u[r].z * rar * ru.z), swiglu<T>(v.w, u[r].w * rar * ru.w));
          const int64_t at_out = (m0 + first + (int64_t)(i + r) * step) * p.ld + n;
          if (sizeof(T) == 2)
            *reinterpret_cast<uint2*>(reinterpret_cast<__nv_bfloat16*>(p.out) + at_out) =
                make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
          else
            *reinterpret_cast<float4*>(reinterpret_cast<float*>(p.out) + at_out) = v;
        }
      }
    };
    if (split == 1)
      store_rows(std::integral_constant<int, NT >= 64 ? 4 : 1>{});
    else
      store_rows(std::integral_constant<int, 1>{});
  }
  __syncwarp();
  if (split > 1) cluster_sync_relaxed();  // no CTA leaves while another reads its sums
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, Cfg::kTmemCols);
}

// ------------------------------------------------------------------ CTA pairs
// Products of many rows: persistent clusters of two CTAs, 256 x 256 cluster
// tiles, products of M = 256, N = 256, K = 64 over both SMs' shared memory
// (each SM stages its 128 rows of A and half of the tile's weight rows, the
// scales of its A rows and those of all 256 weight rows). SwiGLU tiles hold
// 128 gate rows and the 128 up rows that go with them.
//
// Tensor memory has 512 columns. Two 256-column accumulators would leave none
// for the scales, so the second one starts inside the first, and the scales
// take the columns behind it. An epilogue warp reads its share of the
// overlapped half into registers first and then lets the next tile's products
// begin; the rest of its tile overlaps them.
//
// The scale columns are two slots, one per stage of 256 channels (NV 48
// columns, MX 24). A slot is rewritten once the products that read it, those of
// the stage before last, have completed.
//
// The tensor pipe takes 128 cycles a product, 512 a stage, and the issuing warp
// has to stay below that. Copies, products and commits of a stage are one asm
// block under one elected lane: with an election each, the issue of a stage
// took 1000-1300 cycles (NV, 8192 x 28672 x 5376: 870 us).
//
// Measured (32768 x 5376 x 14336, NV / MX): a stage takes 601 / 599 cycles and
// the product 890 / 830 us, 5.7 / 6.1 PFLOP/s, in a run of 40 launches; 1100 us,
// 4.6, in one of a quarter of a second, at the power limit. A copy that loads
// nothing (stale operands, for timing only) takes 544 / 533 cycles and reaches
// 7.3 / 7.7 PFLOP/s at a higher clock: what bounds the kernel is moving 39 / 36 KB a
// stage from L2 into each SM, in shared-memory cycles and in power. Finer scale
// slots (four of half a stage), 4 to 112 N-tiles in the raster and narrower
// tiles for a last partial wave changed it by less than 3 %.
constexpr int kPairThreads = 320;  // producer, issuer, eight epilogue warps
constexpr int kPairEpiWarps = 8;
constexpr int kGroupN = 12;  // tile raster: 12 N-tiles share each pass over M

template <int FMT>
struct PairCfg {
  static constexpr int kAtoms = atoms_per_stage(FMT);
  static constexpr int kScaleBytes = kAtoms * 512;  // of 128 rows
  static constexpr int kStageBytes = 2 * kTile + 3 * kScaleBytes;
  static constexpr int kStages = 5;
  static constexpr size_t kSlack = 768;  // to align the base to 1024 bytes
  static constexpr size_t kSmem = kSlack + (size_t)kStages * kStageBytes + kPairEpiWarps * (32 * 128 + 512) + 144;
  static_assert(kSmem <= 232448, "shared memory of a CTA");
  static constexpr int kSlotCols = 12 * kAtoms;             // scales of A, of the two halves of B; four columns an atom
  static constexpr int kScaleCol = 512 - 2 * kSlotCols;
  static constexpr int kAcc1 = kScaleCol - 256;             // the second accumulator
  static_assert(kAcc1 >= 128, "the first half of the first accumulator is not overlapped");
};

// A whole stage's tensor work for a CTA pair, issued by one lane: the scale
// copies (atoms at sd, sd + kScaleBytes, sd + 2 kScaleBytes) to the slot at
// column sc, the four products of 64 channels into the accumulator at column d,
// and the commits to `sfree` (this CTA) and `empty` (both).
#define H3_CP(T, X) "add.u32 t, %1, " #T ";\n\tadd.s64 x, %4, " #X ";\n\t" \
                    "@e tcgen05.cp.cta_group::2.32x128b.warpx4 [t], x;\n\t"
#define H3_MM(OP, ID, SA, SB, K, P)                                                      \
  "add.u32 t, %1, " #SA ";\n\tadd.u32 u, %1, " #SB ";\n\t"                             \
  "add.s64 x, %2, " #K ";\n\tadd.s64 y, %3, " #K ";\n\t"                               \
  "@e tcgen05.mma.cta_group::2." OP " [%0], x, y, " ID ", [t], [u], " P ";\n\t"
#define H3_COMMITS                                                                                                    \
  "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%8], %10;\n\t"         \
  "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%9], %11;\n\t"
#define H3_BLOCK_BEGIN                                                                 \
  "{\n\t.reg .pred p, q, e;\n\t.reg .b32 t, u;\n\t.reg .b64 x, y;\n\t" H3_ELECT_PRED \
  "setp.ne.b32 p, %7, 0;\n\tsetp.eq.b32 q, 0, 0;\n\t"
template <int FMT>
__device__ __forceinline__ void issue_pair_stage(uint32_t d, uint32_t sc, uint64_t ad, uint64_t bd, uint64_t sd,
                                                 uint32_t accumulate, uint64_t* sfree, uint64_t* empty) {
  constexpr uint32_t id0 = make_idesc_fp4(256, 256, FMT == kFp4MX, 0), id1 = make_idesc_fp4(256, 256, FMT == kFp4MX, 2);
#define H3_ARGS                                                                                             \
  ::"r"(d), "r"(sc), "l"(ad), "l"(bd), "l"(sd), "r"(id0), "r"(id1), "r"(accumulate), "r"(smem_u32(sfree)),  \
      "r"(smem_u32(empty)), "h"((uint16_t)1), "h"((uint16_t)3)                                             \
      : "memory"
  if (FMT == kFp4NV) {
    static_assert(PairCfg<kFp4NV>::kScaleBytes == 128 * 16 && PairCfg<kFp4MX>::kScaleBytes == 64 * 16, "offsets below");
    asm volatile(H3_BLOCK_BEGIN                                                      //
                 H3_CP(0, 0) H3_CP(4, 128) H3_CP(8, 256)                             //
                 H3_MM(H3_NV, "%5", 0, 4, 0, "p")                                    //
                 H3_CP(12, 32) H3_CP(16, 160) H3_CP(20, 288)                         //
                 H3_MM(H3_NV, "%5", 12, 16, 2, "q")                                  //
                 H3_CP(24, 64) H3_CP(28, 192) H3_CP(32, 320)                         //
                 H3_MM(H3_NV, "%5", 24, 28, 4, "q")                                  //
                 H3_CP(36, 96) H3_CP(40, 224) H3_CP(44, 352)                         //
                 H3_MM(H3_NV, "%5", 36, 40, 6, "q") H3_COMMITS "}" H3_ARGS);
  } else {
    asm volatile(H3_BLOCK_BEGIN                                                      //
                 H3_CP(0, 0) H3_CP(4, 64) H3_CP(8, 128)                              //
                 H3_MM(H3_MX, "%5", 0, 4, 0, "p") H3_MM(H3_MX, "%6", 0, 4, 2, "q")   //
                 H3_CP(12, 32) H3_CP(16, 96) H3_CP(20, 160)                          //
                 H3_MM(H3_MX, "%5", 12, 16, 4, "q") H3_MM(H3_MX, "%6", 12, 16, 6, "q") H3_COMMITS "}" H3_ARGS);
  }
#undef H3_ARGS
}
#undef H3_CP
#undef H3_MM
#undef H3_COMMITS
#undef H3_BLOCK_BEGIN
#undef H3_NV
#undef H3_MX

struct Tile {
  int m, n;
};
__device__ __forceinline__ Tile pair_tile(int t, int tiles_m, int tiles_n) {
  const int group = t / (kGroupN * tiles_m);
  const int first = group * kGroupN;
  const int gn = min(kGroupN, tiles_n - first);
  const int i = t - group * kGroupN * tiles_m;
  return {i / gn, first + i % gn};
}

// Output goes through shared memory, one unit of 32 rows x 128 bytes per
// epilogue warp at a time, and leaves by a TMA store that also clips it at the
// matrix's edges. Storing 16 bytes a lane from the accumulators' row-per-lane
// layout, with the scales read from global memory behind the products, an
// epilogue took 13,000 cycles a tile, more than the 11,000 of the products at
// K = 5376.
constexpr int kUnitBytes = 32 * 128;

__device__ __forceinline__ void tma_store_2d(const CUtensorMap* m, const void* src, int x, int y) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(m)),
               "r"(smem_u32(src)), "r"(x), "r"(y)
               : "memory");
}

// One epilogue warp's unit: lane's row of v, as T, to the unit with the
// 128-byte swizzle, then stored at column x, row y where that lies inside.
template <typename T>
__device__ __forceinline__ void store_unit(uint8_t* unit, const CUtensorMap* m, int lane, const float* v, int x, int64_t y,
                                           const Fp4GemmArgs& p) {
  if (lane == 0) bulk_wait_read<0>();  // the unit's last store has read it
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    uint4 o;
    if (sizeof(T) == 2)
      o = make_uint4(pack_bf16x2(v[8 * i], v[8 * i + 1]), pack_bf16x2(v[8 * i + 2], v[8 * i + 3]),
                     pack_bf16x2(v[8 * i + 4], v[8 * i + 5]), pack_bf16x2(v[8 * i + 6], v[8 * i + 7]));
    else
      o = make_uint4(__float_as_uint(v[4 * i]), __float_as_uint(v[4 * i + 1]), __float_as_uint(v[4 * i + 2]),
                     __float_as_uint(v[4 * i + 3]));
    *reinterpret_cast<uint4*>(unit + lane * 128 + ((i ^ (lane & 7)) << 4)) = o;
  }
  fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0) {
    if (x < p.N && y < p.M) tma_store_2d(m, unit, x, (int)y);
    bulk_commit();
  }
}
// 32 accumulators of a lane's row times its row scale and the 32 weight rows'.
__device__ __forceinline__ void scale_chunk(const uint32_t* r, float ra, const float* rb, float* v) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float4 b = reinterpret_cast<const float4*>(rb)[i];
    v[4 * i] = __uint_as_float(r[4 * i]) * ra * b.x;
    v[4 * i + 1] = __uint_as_float(r[4 * i + 1]) * ra * b.y;
    v[4 * i + 2] = __uint_as_float(r[4 * i + 2]) * ra * b.z;
    v[4 * i + 3] = __uint_as_float(r[4 * i + 3]) * ra * b.w;
  }
}
template <int FMT, bool SWIGLU, typename T>
__global__ void __launch_bounds__(kPairThreads, 1)
    gemm_fp4_pair_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                         const __grid_constant__ CUtensorMap tmAS, const __grid_constant__ CUtensorMap tmBS,
                         const __grid_constant__ CUtensorMap tmOut, const Fp4GemmArgs p) {
  using Cfg = PairCfg<FMT>;
  constexpr int kStages = Cfg::kStages;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  // (the declared alignment makes this 0; an early return instead of the
  // bound costs the issuing warp a fifth of its speed)
  uint8_t* smem = smem_raw + min(((smem_u32(smem_raw) + 1023u) & ~1023u) - smem_u32(smem_raw), (uint32_t)Cfg::kSlack);
  // stages (A tile, B tile, A scales, scales of the tile's first and second
  // 128 weight rows), the warps' output units, their row scales, the barriers
  uint8_t* units = smem + (size_t)kStages * Cfg::kStageBytes;
  float* rbs = reinterpret_cast<float*>(units + kPairEpiWarps * kUnitBytes);
  uint64_t* full = reinterpret_cast<uint64_t*>(rbs + kPairEpiWarps * 128);
  uint64_t* empty = full + kStages;
  uint64_t* sfree = empty + kStages;
  uint64_t* tfull = sfree + 2;
  uint64_t* tempty = tfull + 2;
  uint64_t* drain = tempty + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  int* abort_word = reinterpret_cast<int*>(drain + 2);
  volatile int* abort = abort_word;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const int cluster = blockIdx.x >> 1, n_clusters = gridDim.x >> 1;
  const int tiles_m = (int)((p.M + 255) / 256);
  const int tiles_n = SWIGLU ? p.N / 128 : (p.N + 255) / 256;
  const int num_tiles = tiles_m * tiles_n;
  const int num_kb = (p.K + kBlockK - 1) / kBlockK;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&full[i], 1);   // the first CTA's producer arrives; both CTAs' bytes complete it
      mbar_init(&empty[i], 1);  // one commit of the issuer
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sfree[i], 1);
      mbar_init(&tfull[i], 1);
    }
    mbar_init(tempty, 2 * kPairEpiWarps);
    mbar_init(drain, 1);
    *abort = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
    tma_prefetch_desc(&tmAS);
    tma_prefetch_desc(&tmBS);
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync();  // both CTAs' barriers are initialised and their tensor memory allocated
  tc_fence_after();
  // all 512 columns are this CTA's, an allocation that can only start at column
  // 0: a constant that the issue loop need not carry
  pdl_launch();  // (behind the allocation: a later kernel's CTA may wait for these columns, but cannot hold them)
  pdl_wait();

  if (warp == 0) {
    // ---------------------------------------------------------------- producer (both CTAs)
    if (lane == 0) {
      const uint32_t full0 = mapa_shared(smem_u32(full), 0);
      int stage = 0;
      uint32_t phase = 0;
      long issued = 0;
      bool ok = true;
      for (int t = cluster; t < num_tiles && ok; t += n_clusters) {
        const Tile tc = pair_tile(t, tiles_m, tiles_n);
        const int ya = tc.m * 256 + (int)rank * 128;
        const int b0 = SWIGLU ? tc.n * 128 : tc.n * 256, b1 = SWIGLU ? p.N + b0 : b0 + 128;
        for (int kb = 0; kb < num_kb; ++kb) {
          if (!mbar_wait(&empty[stage], phase ^ 1, abort)) {
            give_up(abort, p.err);
            ok = false;
            break;
          }
          uint8_t* st = smem + (size_t)stage * Cfg::kStageBytes;
          const uint32_t bar = full0 + 8u * stage;
          if (rank == 0) mbar_expect_tx(&full[stage], 2 * Cfg::kStageBytes);
          tma_load_2d_pair(st, &tmA, bar, kb * kRowBytes, ya);
          tma_load_2d_pair(st + kTile, &tmB, bar, kb * kRowBytes, rank ? b1 : b0);
          tma_load_3d_pair(st + 2 * kTile, &tmAS, bar, 0, kb * Cfg::kAtoms, ya >> 7);
          tma_load_3d_pair(st + 2 * kTile + Cfg::kScaleBytes, &tmBS, bar, 0, kb * Cfg::kAtoms, b0 >> 7);
          tma_load_3d_pair(st + 2 * kTile + 2 * Cfg::kScaleBytes, &tmBS, bar, 0, kb * Cfg::kAtoms, b1 >> 7);
          ++issued;
          if (++stage == kStages) {
            stage = 0;
            phase ^= 1;
          }
        }
      }
      // first CTA (its full barriers count both CTAs' bytes): the last loads
      // issued must have landed before either CTA exits
      if (rank == 0) {
        const long outstanding = issued < kStages ? issued : kStages;
        for (long i = 0; i < outstanding; ++i) {
          if (--stage < 0) {
            stage = kStages - 1;
            phase ^= 1;
          }
          if (!mbar_wait(&full[stage], phase, nullptr)) give_up(abort, p.err);
        }
      }
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------------- issuer (first CTA)
    if (rank == 0) {
      int stage = 0;
      uint32_t phase = 0, slot = 0;  // slot: stages issued so far
      int local = 0;
      bool ok = true;
      for (int t = cluster; t < num_tiles && ok; t += n_clusters, ++local) {
        if (local > 0 && !mbar_wait_warp(tempty, (uint32_t)(local - 1) & 1, abort)) {
          if (lane == 0) give_up(abort, p.err);
          break;
        }
        tc_fence_after();
        const uint32_t d = (local & 1) * Cfg::kAcc1;
        for (int kb = 0; kb < num_kb; ++kb) {
          // both barriers are looked at once before either is waited for; a slot's
          // first use finds its barrier's preceding phase, which counts as complete
          const uint32_t sfree_parity = ((slot >> 1) & 1) ^ 1;
          const bool r0 = mbar_try_wait(&full[stage], phase), r1 = mbar_try_wait(&sfree[slot & 1], sfree_parity);
          if (!__all_sync(0xffffffffu, r0 && r1) &&
              !(mbar_wait_warp(&full[stage], phase, abort) && mbar_wait_warp(&sfree[slot & 1], sfree_parity, abort))) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t a0 = smem_u32(smem) + (uint32_t)stage * Cfg::kStageBytes;
          const uint32_t b0 = a0 + kTile, s0 = b0 + kTile;
          const uint32_t cols = Cfg::kScaleCol + (slot & 1) * Cfg::kSlotCols;
          const int left = p.K - kb * kBlockK;
          if (left > kBlockK - 64) {
            issue_pair_stage<FMT>(d, cols, sw128_desc(a0, 16), sw128_desc(b0, 16), scale_atom_desc(s0), kb != 0,
                                  &sfree[slot & 1], &empty[stage]);
          } else {  // the last stage of a K that does not fill it
            const int steps = (left + 63) / 64;
#pragma unroll 1
            for (int s = 0; s < steps; ++s) {
              const int a = s * 64 / fp4_atom_channels(FMT);
              const uint32_t col = cols + a * 12, at = s0 + a * 512;
              if (s * 64 % fp4_atom_channels(FMT) == 0) {
                tmem_cp_scales_pair_w(col, scale_atom_desc(at));
                tmem_cp_scales_pair_w(col + 4, scale_atom_desc(at + Cfg::kScaleBytes));
                tmem_cp_scales_pair_w(col + 8, scale_atom_desc(at + 2 * Cfg::kScaleBytes));
              }
              const uint32_t id = make_idesc_fp4(256, 256, FMT == kFp4MX, FMT == kFp4MX ? (s & 1) * 2 : 0);
              mma_fp4_ss_pair_w<FMT == kFp4NV>(d, sw128_desc(a0 + s * 32, 16), sw128_desc(b0 + s * 32, 16), id, col,
                                               col + 4, (kb | s) != 0);
            }
            mma_commit_pair_w(&sfree[slot & 1], 0x1);
            mma_commit_pair_w(&empty[stage], 0x3);
          }
          ++slot;
          if (++stage == kStages) {
            stage = 0;
            phase ^= 1;
          }
        }
        if (!ok) {
          if (lane == 0) give_up(abort, p.err);
        } else {
          mma_commit_pair_w(&tfull[local & 1], 0x3);
        }
      }
      mma_commit_pair_w(drain, 0x3);
      if (!mbar_wait(drain, 0, nullptr)) give_up(abort, p.err);
    } else if (lane == 0) {
      // second CTA: its shared and tensor memory serve the pair's products
      // until the last one completes
      if (!mbar_wait(drain, 0, nullptr)) give_up(abort, p.err);
    }
  } else {
    // ---------------------------------------------------------------- epilogue (both CTAs)
    const int quad = warp & 3, half = (warp - 2) >> 2;
    const uint32_t tempty0 = mapa_shared(smem_u32(tempty), 0);
    uint8_t* unit = units + (warp - 2) * kUnitBytes;
    float* rb = rbs + (warp - 2) * 128;
    int local = 0;
    for (int t = cluster; t < num_tiles; t += n_clusters, ++local) {
      const Tile tc = pair_tile(t, tiles_m, tiles_n);
      const int buf = local & 1;
      const int64_t row0 = (int64_t)tc.m * 256 + rank * 128 + quad * 32;
      // the warp's 64 columns of each half of the tile; their weight rows' scales,
      // and the lane's own, are fetched while the products run
      const int col0 = SWIGLU ? tc.n * 128 + half * 64 : tc.n * 256 + half * 64;
      const int row_b = col0 + (lane >> 4) * (SWIGLU ? p.N : 128) + (lane & 15) * 4;
      const int rows_b = SWIGLU ? 2 * p.N : p.N;
      __syncwarp();  // the last tile's scales have been read
      reinterpret_cast<float4*>(rb)[lane] =
          row_b < rows_b ? __ldg(reinterpret_cast<const float4*>(p.b_row + row_b)) : make_float4(0.f, 0.f, 0.f, 0.f);
      const float ra = row0 + lane < p.M ? __ldg(p.a_row + row0 + lane) : 0.f;
      __syncwarp();
      if (!mbar_wait_warp(&tfull[buf], (uint32_t)(local >> 1) & 1, abort)) {  // the reads below take the whole warp
        if (lane == 0) give_up(abort, p.err);
        break;
      }
      tc_fence_after();
      const uint32_t acc = ((uint32_t)(quad * 32) << 16) + buf * Cfg::kAcc1 + half * 64;
      // this warp's columns of the tile's half that the other accumulator
      // overlaps (the first one's upper, the second one's lower), then the
      // next tile's products may begin (behind the last tile nobody waits, and an
      // arrival could come after the first CTA has left)
      uint32_t f[64];
      tmem_ld64(acc + (buf ? 0 : 128), f);
      tc_fence_before();
      __syncwarp();
      if (lane == 0 && t + n_clusters < num_tiles) mbar_arrive_cluster_relaxed(tempty0);
      constexpr int kUnitCols = 128 / (int)sizeof(T);
      float v[64];
      if (SWIGLU) {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          uint32_t r[32];
          tmem_ld32(acc + (buf ? 128 : 0) + q * 32, r);
          float g[32], u[32];
          scale_chunk(buf ? f + 32 * q : r, ra, rb + q * 32, g);
          scale_chunk(buf ? r : f + 32 * q, ra, rb + 64 + q * 32, u);
#pragma unroll
          for (int i = 0; i < 32; ++i) v[32 * q + i] = swiglu<T>(g[i], u[i]);
          if (kUnitCols == 32) store_unit<T>(unit, &tmOut, lane, v + 32 * q, col0 + 32 * q, row0, p);
        }
        if (kUnitCols == 64) store_unit<T>(unit, &tmOut, lane, v, col0, row0, p);
      } else {
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          const int h1 = hf ? buf : 1 - buf;  // which half of the tile: the overlapped one first
          if (hf) tmem_ld64(acc + (buf ? 128 : 0), f);
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            scale_chunk(f + 32 * q, ra, rb + h1 * 64 + q * 32, v + 32 * q);
            if (kUnitCols == 32) store_unit<T>(unit, &tmOut, lane, v + 32 * q, col0 + h1 * 128 + 32 * q, row0, p);
          }
          if (kUnitCols == 64) store_unit<T>(unit, &tmOut, lane, v, col0 + h1 * 128, row0, p);
        }
      }
    }
    if (lane == 0) bulk_wait_read<0>();  // the output has left shared memory (it reaches the matrix before the grid ends)
  }
  // neither CTA leaves while the other may still signal its barriers or read
  // its memory: every signal has been waited for by now, so no ordering is needed
  __syncwarp();  // (lanes of the roles above come back one by one; the cluster's barrier takes whole warps)
  tc_fence_before();
  cluster_sync_relaxed();
  tc_fence_after();
  if (warp == 1) tmem_dealloc_pair(*tmem_slot, 512);
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

// The output, stored in units of 32 rows x 128 bytes.
bool out_map(PFN_cuTensorMapEncodeTiled_v12000 encode, CUtensorMap* m, const Fp4GemmArgs& p) {
  const cuuint64_t es = p.f32 ? 4 : 2;
  cuuint64_t dims[2] = {(cuuint64_t)p.N, (cuuint64_t)p.M};
  cuuint64_t strides[1] = {(cuuint64_t)p.ld * es};
  cuuint32_t box[2] = {(cuuint32_t)(128 / es), 32};
  cuuint32_t estr[2] = {1, 1};
  return encode(m, p.f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, p.out, dims, strides,
                box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct Maps {
  CUtensorMap a, b, as, bs, out;
};

constexpr int kMinStages = 2;

// CTAs that share K in the few-rows kernel: up to six, as long as each keeps
// kMinStages stages to stream and their clusters fill no more than seven eighths
// of the SMs' places; 0 where the unsplit tiles already take more.
// Measured (NV, a row, us): 84 tiles x 21 stages split by 2 / 3 / 4 9.5 / 9.0 / 13.3;
// 56 x 21 by 3 / 4 / 5 7.0 / 7.1 / 8.1; 42 x 56 by 4 / 6 / 7 11.1 / 10.7 / 15.1.
template <int FMT, int NT, int NW>
int few_split(const Fp4GemmArgs& p, int num_sms) {
  const int64_t tiles = (p.N + 127) / 128 * ((p.M + NT - 1) / NT);
  const int64_t places = (int64_t)FewCfg<FMT, NT, NW>::kPerSm * num_sms * 7 / 8;
  const int stages = (p.K + kBlockK - 1) / kBlockK;
  int split = (int)(places / tiles < kMaxSplit ? places / tiles : kMaxSplit);
  if (split > stages / kMinStages) split = stages / kMinStages < 1 ? 1 : stages / kMinStages;
  return split;
}

template <int FMT, int NT, int NW, typename T>
cudaError_t launch_few_t(const Fp4GemmArgs& p, const Maps& m, int num_sms, cudaStream_t s) {
  using Cfg = FewCfg<FMT, NT, NW>;
  auto k = gemm_fp4_few_kernel<FMT, NT, NW, T>;
  cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Cfg::kSmem);
  if (e != cudaSuccess) return e;
  const int split = std::max(1, few_split<FMT, NT, NW>(p, num_sms));
  ChainedLaunch l(dim3((p.N + 127) / 128, (unsigned)((p.M + NT - 1) / NT), split), kFewThreads, Cfg::kSmem, s,
                  dim3(1, 1, split));
  return cudaLaunchKernelEx(&l.cfg, k, m.b, m.a, m.bs, m.as, p);
}

template <int FMT, int NT>
cudaError_t launch_few(const Fp4GemmArgs& p, const Maps& m, int num_sms, cudaStream_t s) {
  if (p.swiglu)
    return p.f32 ? launch_few_t<FMT, NT, 2, float>(p, m, num_sms, s) : launch_few_t<FMT, NT, 2, __nv_bfloat16>(p, m, num_sms, s);
  return p.f32 ? launch_few_t<FMT, NT, 1, float>(p, m, num_sms, s) : launch_few_t<FMT, NT, 1, __nv_bfloat16>(p, m, num_sms, s);
}

template <int FMT, bool SWIGLU, typename T>
cudaError_t launch_pair_t(const Fp4GemmArgs& p, const Maps& m, int num_sms, cudaStream_t s) {
  using Cfg = PairCfg<FMT>;
  auto k = gemm_fp4_pair_kernel<FMT, SWIGLU, T>;
  cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Cfg::kSmem);
  if (e != cudaSuccess) return e;
  const int64_t tiles = (p.M + 255) / 256 * (SWIGLU ? p.N / 128 : ((int64_t)p.N + 255) / 256);
  if (tiles > 0x7fffffff) return cudaErrorInvalidValue;
  const int clusters = (int)(tiles < num_sms / 2 ? tiles : num_sms / 2);
  ChainedLaunch l(dim3(2 * clusters), kPairThreads, Cfg::kSmem, s, dim3(2));
  return cudaLaunchKernelEx(&l.cfg, k, m.a, m.b, m.as, m.bs, m.out, p);
}

// Whether the few-rows kernel takes a product: always up to 64 rows, above them
// where the pair kernel's tiles would leave many SMs without work or weights
// unread. Both take a start and an end and their stages one after the other; in
// units of a pair stage (0.4 us; SwiGLU 1.2 of them) about 11 + stages x waves,
// and 15 + 1.6 (SwiGLU 2.2) x a CTA's stages. Measured (NV, us, few rows / pair):
// 128 x 21504 x 5376 17.4 / 22, 128 x 2304 x 768 5.7 / 5.2, 160 x 5376 x 7168 12.2 /
// 15.3, 160 x 7168 x 5376 13.4 / 12.8, 256 x 1024 x 7168 9.0 / 14.3, 256 x 5376 x 2048
// 8.8 / 7.5, 384 x 10752 x 5376 16.6 / 21.7, 256 x 8192 x 14336 23.4 / 26.5; at worst the
// rule's choice was 8 % slower (65 x 2 x 7168 x 7168 SwiGLU 16.2 / 17.6).
template <int FMT, int NW>
bool takes_few(const Fp4GemmArgs& p, int num_sms) {
  if (p.M <= 64) return true;
  const int split = few_split<FMT, 128, NW>(p, num_sms);
  if (split == 0) return false;
  const int64_t stages = (p.K + kBlockK - 1) / kBlockK, clusters = num_sms / 2;
  const int64_t tiles = (p.M + 255) / 256 * ((p.N + 256 / NW - 1) / (256 / NW));
  const int64_t few = 150 + (NW == 1 ? 16 : 22) * ((stages + split - 1) / split);
  return few < 110 + (NW == 1 ? 10 : 12) * stages * ((tiles + clusters - 1) / clusters);
}

template <int FMT>
cudaError_t launch_fmt(const Fp4GemmArgs& p, PFN_cuTensorMapEncodeTiled_v12000 encode, int num_sms, cudaStream_t s) {
  Maps m;
  const bool few = p.swiglu ? takes_few<FMT, 2>(p, num_sms) : takes_few<FMT, 1>(p, num_sms);
  const int nt = !few ? 128 : p.M <= 16 ? 16 : p.M <= 32 ? 32 : p.M <= 64 ? 64 : 128;
  const int64_t b_rows = p.swiglu ? 2 * (int64_t)p.N : p.N;
  if (!codes_map(encode, &m.a, p.a_codes, p.M, p.K, nt) || !codes_map(encode, &m.b, p.b_codes, b_rows, p.K, 128) ||
      !scales_map(encode, &m.as, p.a_scales, p.M, p.K, FMT) || !scales_map(encode, &m.bs, p.b_scales, b_rows, p.K, FMT))
    return cudaErrorInvalidValue;
  if (!few) {
    if (!out_map(encode, &m.out, p)) return cudaErrorInvalidValue;
    if (p.swiglu)
      return p.f32 ? launch_pair_t<FMT, true, float>(p, m, num_sms, s)
                   : launch_pair_t<FMT, true, __nv_bfloat16>(p, m, num_sms, s);
    return p.f32 ? launch_pair_t<FMT, false, float>(p, m, num_sms, s)
                 : launch_pair_t<FMT, false, __nv_bfloat16>(p, m, num_sms, s);
  }
  switch (nt) {
    case 16: return launch_few<FMT, 16>(p, m, num_sms, s);
    case 32: return launch_few<FMT, 32>(p, m, num_sms, s);
    case 64: return launch_few<FMT, 64>(p, m, num_sms, s);
    default: return launch_few<FMT, 128>(p, m, num_sms, s);
  }
}

}  // namespace

cudaError_t launch_gemm_fp4(const Fp4GemmArgs& p, PFN_cuTensorMapEncodeTiled_v12000 encode, int num_sms,
                            cudaStream_t s) {
  if (p.M <= 0 || p.N <= 0) return cudaSuccess;
  return p.nv ? launch_fmt<kFp4NV>(p, encode, num_sms, s) : launch_fmt<kFp4MX>(p, encode, num_sms, s);
}

}  // namespace h3
