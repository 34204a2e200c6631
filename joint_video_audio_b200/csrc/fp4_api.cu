// C-ABI of the 4-bit linear path and of the sandwich norm: argument checks and
// launches (see include/h3blk.h).
#include <cuda.h>
#include <cuda_runtime.h>

#include <mutex>

#include "api_internal.h"
#include "fp4.cuh"

namespace {
// What the kernels of these calls report, on each device: a bit per kind of wait
// that ran out, until h3blk_fp4_check takes it; and what it took.
__device__ int g_fp4_error, g_fp4_taken;

// (an exchange, so that no report of a kernel still running is lost)
__global__ void take_error_kernel() { g_fp4_taken = atomicExch(&g_fp4_error, 0); }

using h3api::aligned16;
using h3api::cuda_status;

constexpr int kMaxChannels = 16384;               // of a row pass, as h3blk_rotate_quantize
constexpr int kMaxGemmK = 1 << 24;
constexpr int64_t kMaxRows = (int64_t)1 << 30;
constexpr int64_t kMaxStride = (int64_t)1 << 36;  // a tensor map's strides end at 2^40 bytes

bool known_format(int f) { return f == H3BLK_FP4_MX || f == H3BLK_FP4_NV; }

size_t scale_bytes(int format, int64_t rows, int K) {
  return (size_t)((rows + 127) / 128) * (size_t)h3::fp4_katoms(format, K) * 512;
}

// A 4-bit matrix that a call reads or writes.
int check_fp4(const h3blk_fp4* q) {
  if (!q || !known_format(q->format) || q->rows < 0 || q->K < 1 || q->K % 32) return H3BLK_ERR_INVALID_ARG;
  if (!q->codes || !q->scales || !q->row_scale) return H3BLK_ERR_INVALID_ARG;
  if (!aligned16(q->codes) || !aligned16(q->scales) || !aligned16(q->row_scale)) return H3BLK_ERR_INVALID_ARG;
  if (q->rows > kMaxRows) return H3BLK_ERR_UNSUPPORTED;
  return H3BLK_OK;
}

struct Range {
  const void* p;
  size_t n;
};
bool overlap(const Range& a, const Range& b) { return h3api::overlap(a.p, a.n, b.p, b.n); }
// The three buffers of a 4-bit matrix.
struct Parts {
  Range r[3];
  explicit Parts(const h3blk_fp4* q)
      : r{{q->codes, (size_t)q->rows * (q->K / 2)},
          {q->scales, scale_bytes(q->format, q->rows, q->K)},
          {q->row_scale, (size_t)q->rows * 4}} {}
  bool overlap_one_another() const { return overlap(r[0], r[1]) || overlap(r[0], r[2]) || overlap(r[1], r[2]); }
};
bool overlaps_fp4(const Range& a, const h3blk_fp4* q) {
  const Parts b(q);
  return overlap(a, b.r[0]) || overlap(a, b.r[1]) || overlap(a, b.r[2]);
}
// The current device's error word, and what launches need besides.
struct Device {
  int sms = 0;
  PFN_cuTensorMapEncodeTiled_v12000 encode = nullptr;
  int* err = nullptr;
};
int device(Device* d) {
  constexpr int kMaxDevices = 64;
  static std::mutex mu;
  static int* words[kMaxDevices];
  const int st = h3api::device_info(&d->sms, &d->encode);
  if (st != H3BLK_OK) return st;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return H3BLK_ERR_CUDA;
  std::lock_guard<std::mutex> lock(mu);
  if (!words[dev]) {
    // (may load the module, which a capture under way on another stream would refuse)
    cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;
    if (cudaThreadExchangeStreamCaptureMode(&mode) != cudaSuccess) return H3BLK_ERR_CUDA;
    void* p = nullptr;
    const cudaError_t e = cudaGetSymbolAddress(&p, g_fp4_error);
    if (cudaThreadExchangeStreamCaptureMode(&mode) != cudaSuccess || e != cudaSuccess || !p) return H3BLK_ERR_CUDA;
    words[dev] = static_cast<int*>(p);
  }
  d->err = words[dev];
  return H3BLK_OK;
}

// A wait of the kind that these calls' kernels make, which runs out.
__global__ void late_wait_kernel(unsigned long long limit_ns, int* err) {
  __shared__ uint64_t bar;
  h3::mbar_init(&bar, 1);
  h3::fence_mbar_init();
  if (!h3::mbar_wait_for(&bar, 0, nullptr, limit_ns)) atomicOr(err, h3::kErrTimeoutStream);
}

// Bytes spanned by `rows` rows of `cols` elements, `ld` elements apart.
size_t span(int64_t rows, int64_t cols, int64_t ld, int esize) {
  return rows > 0 ? ((size_t)(rows - 1) * ld + cols) * esize : 0;
}

}  // namespace

extern "C" {

int h3blk_fp4_bytes(int format, int64_t rows, int K, size_t* codes, size_t* scales, size_t* row_scale) {
  if (!known_format(format) || rows < 0 || K < 1 || K % 32 || !codes || !scales || !row_scale)
    return H3BLK_ERR_INVALID_ARG;
  if (rows > kMaxRows) return H3BLK_ERR_UNSUPPORTED;
  *codes = (size_t)rows * (K / 2);
  *scales = scale_bytes(format, rows, K);
  *row_scale = (size_t)rows * sizeof(float);
  return H3BLK_OK;
}

int h3blk_quantize_fp4(const void* in, int64_t ld_in, int rotate, const h3blk_fp4* out, void* stream) {
  int st = check_fp4(out);
  if (st != H3BLK_OK) return st;
  if (!in || !aligned16(in) || ld_in < out->K || ld_in % 8) return H3BLK_ERR_INVALID_ARG;
  if (rotate && out->K % 128) return H3BLK_ERR_INVALID_ARG;
  if (out->K > kMaxChannels) return H3BLK_ERR_UNSUPPORTED;
  if (overlaps_fp4({in, span(out->rows, out->K, ld_in, 2)}, out) || Parts(out).overlap_one_another())
    return H3BLK_ERR_INVALID_ARG;
  Device d;
  st = device(&d);
  if (st != H3BLK_OK) return st;
  h3::Fp4QuantArgs a;
  a.in = static_cast<const __nv_bfloat16*>(in);
  a.ld = ld_in;
  a.rows = out->rows;
  a.K = out->K;
  a.nv = out->format == H3BLK_FP4_NV;
  a.rotate = rotate != 0;
  a.codes = static_cast<uint8_t*>(out->codes);
  a.scales = static_cast<uint8_t*>(out->scales);
  a.row_scale = out->row_scale;
  a.err = d.err;
  return cuda_status(h3::launch_quantize_fp4(a, d.sms, reinterpret_cast<cudaStream_t>(stream)));
}

int h3blk_dequantize_fp4(const h3blk_fp4* in, int out_type, void* out, int64_t ld_out, void* stream) {
  int st = check_fp4(in);
  if (st != H3BLK_OK) return st;
  if (out_type != H3BLK_BF16 && out_type != H3BLK_F32) return H3BLK_ERR_INVALID_ARG;
  if (!out || !aligned16(out) || ld_out < in->K || ld_out % 8) return H3BLK_ERR_INVALID_ARG;
  if (in->K > kMaxGemmK) return H3BLK_ERR_UNSUPPORTED;
  if (overlaps_fp4({out, span(in->rows, in->K, ld_out, out_type == H3BLK_F32 ? 4 : 2)}, in)) return H3BLK_ERR_INVALID_ARG;
  Device d;
  st = device(&d);
  if (st != H3BLK_OK) return st;
  h3::Fp4DequantArgs a;
  a.codes = static_cast<const uint8_t*>(in->codes);
  a.scales = static_cast<uint8_t*>(in->scales);
  a.row_scale = in->row_scale;
  a.rows = in->rows;
  a.K = in->K;
  a.nv = in->format == H3BLK_FP4_NV;
  a.f32 = out_type == H3BLK_F32;
  a.out = out;
  a.ld = ld_out;
  return cuda_status(h3::launch_dequantize_fp4(a, reinterpret_cast<cudaStream_t>(stream)));
}

int h3blk_gemm_fp4(const h3blk_fp4* A, const h3blk_fp4* B, int epilogue, int out_type, void* out, int64_t ld_out,
                   void* stream) {
  int st = check_fp4(A);
  if (st != H3BLK_OK) return st;
  st = check_fp4(B);
  if (st != H3BLK_OK) return st;
  if (A->format != B->format || A->K != B->K || B->rows < 1) return H3BLK_ERR_INVALID_ARG;
  if (epilogue != H3BLK_FP4_STORE && epilogue != H3BLK_FP4_SWIGLU) return H3BLK_ERR_INVALID_ARG;
  if (out_type != H3BLK_BF16 && out_type != H3BLK_F32) return H3BLK_ERR_INVALID_ARG;
  const bool swiglu = epilogue == H3BLK_FP4_SWIGLU;
  if (B->rows % (swiglu ? 256 : 8)) return H3BLK_ERR_UNSUPPORTED;
  if (A->K > kMaxGemmK) return H3BLK_ERR_UNSUPPORTED;
  const int64_t N = swiglu ? B->rows / 2 : B->rows;
  if (!out || !aligned16(out) || ld_out < N || ld_out % 8) return H3BLK_ERR_INVALID_ARG;
  if (ld_out > kMaxStride) return H3BLK_ERR_UNSUPPORTED;
  const Range written{out, span(A->rows, N, ld_out, out_type == H3BLK_F32 ? 4 : 2)};
  if (overlaps_fp4(written, A) || overlaps_fp4(written, B)) return H3BLK_ERR_INVALID_ARG;
  Device d;
  st = device(&d);
  if (st != H3BLK_OK) return st;
  h3::Fp4GemmArgs g;
  g.a_codes = static_cast<const uint8_t*>(A->codes);
  g.b_codes = static_cast<const uint8_t*>(B->codes);
  g.a_scales = static_cast<const uint8_t*>(A->scales);
  g.b_scales = static_cast<const uint8_t*>(B->scales);
  g.a_row = A->row_scale;
  g.b_row = B->row_scale;
  g.M = A->rows;
  g.N = (int)N;
  g.K = A->K;
  g.nv = A->format == H3BLK_FP4_NV;
  g.swiglu = swiglu;
  g.f32 = out_type == H3BLK_F32;
  g.out = out;
  g.ld = ld_out;
  g.err = d.err;
  return cuda_status(h3::launch_gemm_fp4(g, d.encode, d.sms, reinterpret_cast<cudaStream_t>(stream)));
}

int h3blk_sandwich_norm(const h3blk_sandwich* s, void* stream) {
  if (!s || s->n_rows < 0 || s->hidden < 1 || s->n_tags < 1 || s->n_t < 1) return H3BLK_ERR_INVALID_ARG;
  if (s->branch != 0 && s->branch != 1) return H3BLK_ERR_INVALID_ARG;
  if (!s->x || !s->y || !s->tag || !s->tidx || !s->mod_table || !s->x_out) return H3BLK_ERR_INVALID_ARG;
  if (s->post_gain && !s->post_norm) return H3BLK_ERR_INVALID_ARG;
  if (!(s->post_eps >= 0.f) || !(s->norm_eps >= 0.f)) return H3BLK_ERR_INVALID_ARG;
  if (s->rotate && !s->h_fp4) return H3BLK_ERR_INVALID_ARG;
  if (s->norm_table ? (!s->h == !s->h_fp4) : (s->h || s->h_fp4)) return H3BLK_ERR_INVALID_ARG;
  const void* ptrs[] = {s->x, s->y, s->post_gain, s->tag, s->tidx, s->mod_table, s->norm_table, s->x_out, s->h};
  for (const void* p : ptrs)
    if (!aligned16(p)) return H3BLK_ERR_INVALID_ARG;
  if (s->hidden % 128 || s->hidden > kMaxChannels || s->n_rows > kMaxRows) return H3BLK_ERR_UNSUPPORTED;
  // what is written shares no byte with anything else, but for x_out = x
  const size_t bytes = (size_t)s->n_rows * s->hidden * 2, channels = (size_t)s->hidden;
  const unsigned __int128 table = (unsigned __int128)s->n_tags * s->n_t * 6 * channels * 4;
  if (table >> 63) return H3BLK_ERR_INVALID_ARG;
  const Range in[] = {{s->x, bytes},
                      {s->y, bytes},
                      {s->post_gain, channels * 2},
                      {s->tag, (size_t)s->n_rows * 4},
                      {s->tidx, (size_t)s->n_rows * 4},
                      {s->mod_table, (size_t)table},
                      {s->norm_table, (size_t)table}};
  const Range x_out{s->x_out, bytes}, h{s->h, bytes};
  for (const Range& r : in) {
    const bool in_place = &r == in && s->x_out == s->x;
    if ((overlap(x_out, r) && !in_place) || overlap(h, r)) return H3BLK_ERR_INVALID_ARG;
  }
  if (overlap(h, x_out)) return H3BLK_ERR_INVALID_ARG;
  if (s->h_fp4) {
    const int st = check_fp4(s->h_fp4);
    if (st != H3BLK_OK) return st;
    if (s->h_fp4->rows != s->n_rows || s->h_fp4->K != s->hidden) return H3BLK_ERR_INVALID_ARG;
    for (const Range& r : in)
      if (overlaps_fp4(r, s->h_fp4)) return H3BLK_ERR_INVALID_ARG;
    if (overlaps_fp4(x_out, s->h_fp4) || Parts(s->h_fp4).overlap_one_another()) return H3BLK_ERR_INVALID_ARG;
  }
  Device d;
  const int st = device(&d);
  if (st != H3BLK_OK) return st;
  h3::SandwichArgs a{};
  a.x = static_cast<const __nv_bfloat16*>(s->x);
  a.y = static_cast<const __nv_bfloat16*>(s->y);
  a.post_gain = static_cast<const __nv_bfloat16*>(s->post_gain);
  a.tag = s->tag;
  a.tidx = s->tidx;
  a.table = s->mod_table;
  a.norm_table = s->norm_table;
  a.rows = s->n_rows;
  a.C = s->hidden;
  a.n_tags = s->n_tags;
  a.n_t = s->n_t;
  a.gate_idx = s->branch ? 5 : 2;
  a.shift_idx = s->branch ? 0 : 3;
  a.post_norm = s->post_norm != 0;
  a.post_eps = s->post_eps;
  a.norm_eps = s->norm_eps;
  a.branch_scale = s->branch_scale;
  a.x_out = static_cast<__nv_bfloat16*>(s->x_out);
  a.h = static_cast<__nv_bfloat16*>(s->h);
  a.err = d.err;
  if (s->h_fp4) {
    a.nv = s->h_fp4->format == H3BLK_FP4_NV;
    a.rotate = s->rotate != 0;
    a.codes = static_cast<uint8_t*>(s->h_fp4->codes);
    a.scales = static_cast<uint8_t*>(s->h_fp4->scales);
    a.row_scale = s->h_fp4->row_scale;
  }
  return cuda_status(h3::launch_sandwich(a, d.sms, reinterpret_cast<cudaStream_t>(stream)));
}

int h3blk_fp4_check(void* stream, int* status) {
  if (!status) return H3BLK_ERR_INVALID_ARG;
  Device d;
  const int st = device(&d);
  if (st != H3BLK_OK) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  int bits = 0;
  static std::mutex one;  // check at a time: they share the word that is taken to
  std::lock_guard<std::mutex> lock(one);
  take_error_kernel<<<1, 1, 0, s>>>();
  if (cudaGetLastError() != cudaSuccess ||
      cudaMemcpyFromSymbolAsync(&bits, g_fp4_taken, sizeof(int), 0, cudaMemcpyDeviceToHost, s) != cudaSuccess ||
      cudaStreamSynchronize(s) != cudaSuccess)
    return H3BLK_ERR_CUDA;
  *status = bits ? H3BLK_ERR_TIMEOUT : H3BLK_OK;
  return H3BLK_OK;
}

int h3blk_selftest_fp4_wait(int limit_ms, void* stream) {
  if (limit_ms < 1 || limit_ms > 2000) return H3BLK_ERR_INVALID_ARG;
  Device d;
  const int st = device(&d);
  if (st != H3BLK_OK) return st;
  late_wait_kernel<<<1, 1, 0, reinterpret_cast<cudaStream_t>(stream)>>>((unsigned long long)limit_ms * 1000000ull, d.err);
  return cuda_status(cudaGetLastError());
}

}  // extern "C"
