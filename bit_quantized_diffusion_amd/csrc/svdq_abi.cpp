// C ABI entry points of libsvdq.so: argument and device validation, then the
// kernel launchers.  Nothing here throws; every failure is a status code.
//
// The device check follows the "Hardware support" section of the blog
// "Nunchaku 4-bit inference in Diffusers": the capability of the GPU is
// checked when the layer is used and an unsupported GPU gets a clear error
// instead of wrong output.

#include <hip/hip_runtime.h>

#include <atomic>
#include <cmath>
#include <cstring>
#include <mutex>

#include "svdq_internal.h"

using namespace svdq;

static_assert(kNoAllocScratchBytes == SVDQ_NOALLOC_SCRATCH_BYTES, "scratch size of the header and the library agree");

namespace {

constexpr int kMaxDevices = 64;
// 0 = not probed yet, 1 = gfx950, 2 = not usable
std::atomic<int> g_dev_state[kMaxDevices];
std::mutex g_dev_mutex;

int probe_device(int device) {
  int count = 0;
  if (hipGetDeviceCount(&count) != hipSuccess || count <= 0) return SVDQ_ERR_UNSUPPORTED_DEVICE;
  if (device < 0 || device >= count || device >= kMaxDevices) return SVDQ_ERR_UNSUPPORTED_DEVICE;
  hipDeviceProp_t prop;
  if (hipGetDeviceProperties(&prop, device) != hipSuccess) return SVDQ_ERR_UNSUPPORTED_DEVICE;
  return std::strncmp(prop.gcnArchName, "gfx950", 6) == 0 ? SVDQ_OK : SVDQ_ERR_UNSUPPORTED_DEVICE;
}

int current_device_ok() {
  int dev = -1;
  if (hipGetDevice(&dev) != hipSuccess) {
    (void)hipGetLastError();
    return SVDQ_ERR_UNSUPPORTED_DEVICE;
  }
  return svdq_device_check(dev);
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int check_dtype(int dtype) { return dtype == SVDQ_BF16 || dtype == SVDQ_F16 ? SVDQ_OK : SVDQ_ERR_INVALID_ARG; }

// rows that the 16-bit operators count: a tile more still fits 31 bits
constexpr long long kMostRows = (1LL << 31) - (1LL << 16);

int check_attention_shape(int total_q, int total_k, int batch, int heads_q, int heads_k, int head_dim) {
  if (total_q < 0 || total_k < 0 || batch < 1 || heads_q < 1 || heads_k < 1 || heads_q % heads_k) return SVDQ_ERR_SHAPE;
  if (head_dim < 8 || head_dim > 128 || head_dim % 8) return SVDQ_ERR_SHAPE;
  // the rows of one key head and the keys, each rounded up to a tile, are
  // counted in 31 bits; a launch holds less than 2^32 threads: 256 for 32 rows
  const long long rows = static_cast<long long>(total_q) * (heads_q / heads_k);
  if (rows > kMostRows || total_k > kMostRows || (rows / 32 + batch) * heads_k >= 1LL << 24) return SVDQ_ERR_SHAPE;
  return SVDQ_OK;
}

bool aligned2(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 1u) == 0; }

int check_linear16_shape(int M, int N, int K) {
  if (M < 1 || N < 1 || K < 1 || M > kMostRows || N > kMostRows) return SVDQ_ERR_SHAPE;
  // a launch holds less than 2^32 threads: 256 for a tile of 64 x 64 or more,
  // for 32 channels of few rows, or for 8 channels of a row of the splits' sum
  // (of fewer than 512 tiles)
  const long long m = M, n = N;
  if (((m + 63) / 64) * ((n + 63) / 64) >= 1LL << 24 || (n + 31) / 32 >= 1LL << 24) return SVDQ_ERR_SHAPE;
  return SVDQ_OK;
}

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// codes of 8 bits: whole 16-byte chunks in a row, 256 rows of a tile in 31 bits
int check_codes(int K) { return K < 16 || K % 16 || K > 1 << 22 ? SVDQ_ERR_SHAPE : SVDQ_OK; }

int check_gemm_fp8_shape(int M, int N, int K) {
  if (M < 1 || N < 1 || M > kMostRows || N > (1 << 28) - 32) return SVDQ_ERR_SHAPE;
  // a launch holds less than 2^32 threads: at most 512 for a tile of 64 rows
  // and up to 64 channels, or for 32 channels of few rows
  if (((M + 63LL) / 64) * ((N + 63LL) / 64) >= 1LL << 23) return SVDQ_ERR_SHAPE;
  return check_codes(K);
}

int check_paged_shape(int total, int batch, int width, int heads_q, int heads_k, int head_dim) {
  if (total < 0 || batch < 1 || width < 1 || width > 1 << 24 || heads_q < 1 || heads_k < 1 || heads_q % heads_k) return SVDQ_ERR_SHAPE;
  if (head_dim < 16 || head_dim > 128 || head_dim % 16) return SVDQ_ERR_SHAPE;
  // positions, and pages of all tiles of 16 rows with 4 for each one's start,
  // are counted in 31 bits; a launch holds less
  // than 2^32 threads: 256 for such a tile, for a touched page of a head, or
  // for a token's queries
  const long long rows = static_cast<long long>(total) * (heads_q / heads_k), hk = heads_k;
  if (rows > kMostRows || rows / 16 + 2LL * batch + total >= (1LL << 24) / hk) return SVDQ_ERR_SHAPE;
  if ((rows / 16 + batch) * hk >= (1LL << 31) / (width + 4)) return SVDQ_ERR_SHAPE;
  return SVDQ_OK;
}

// strides in elements: not negative, far from overflow
bool strides_fit(const int64_t* strides, int n, int multiple) {
  for (int i = 0; i < n; ++i)
    if (strides[i] < 0 || strides[i] % multiple || strides[i] > 1LL << 40) return false;
  return true;
}

int hip_status(int e) { return e == 0 ? SVDQ_OK : SVDQ_ERR_HIP; }

}  // namespace

extern "C" {

int svdq_version(void) { return 100; }

const char* svdq_status_string(int status) {
  switch (status) {
    case SVDQ_OK: return "svdq: ok";
    case SVDQ_ERR_INVALID_ARG: return "svdq: invalid argument (NULL or misaligned pointer, or unknown precision)";
    case SVDQ_ERR_SHAPE: return "svdq: unsupported shape (check M, N >= 1, K and rank rules)";
    case SVDQ_ERR_UNSUPPORTED_DEVICE: return "svdq: no usable gfx950 (MI355X) device; the 4-bit kernels need gfx950";
    case SVDQ_ERR_HIP: return "svdq: HIP runtime error (launch failed)";
    default: return "svdq: unknown status";
  }
}

int svdq_device_check(int device) {
  if (device < 0 || device >= kMaxDevices) return SVDQ_ERR_UNSUPPORTED_DEVICE;
  int s = g_dev_state[device].load(std::memory_order_acquire);
  if (s == 0) {
    std::lock_guard<std::mutex> lock(g_dev_mutex);
    s = g_dev_state[device].load(std::memory_order_relaxed);
    if (s == 0) {
      s = probe_device(device) == SVDQ_OK ? 1 : 2;
      (void)hipGetLastError();
      g_dev_state[device].store(s, std::memory_order_release);
    }
  }
  return s == 1 ? SVDQ_OK : SVDQ_ERR_UNSUPPORTED_DEVICE;
}

int svdq_packed_sizes(int K, int N, int rank, int precision, size_t* out) {
  int st = check_precision(precision);
  if (st) return st;
  if (!out) return SVDQ_ERR_INVALID_ARG;
  if (N < 1) return SVDQ_ERR_SHAPE;
  if ((st = check_k(K, precision))) return st;
  if ((st = check_rank(rank, K, N))) return st;
  const size_t k = static_cast<size_t>(K), n = static_cast<size_t>(N), r = static_cast<size_t>(rank);
  out[0] = k * 4;
  out[1] = r * k * 2;
  out[2] = n * r * 2;
  out[3] = n * k / 2;
  out[4] = precision == SVDQ_INT4 ? (k / kInt4Group) * n * 2 : (k / kMxBlock) * n;
  return SVDQ_OK;
}

int svdq_act_sizes(int M, int K, int rank, int precision, size_t* out) {
  int st = check_precision(precision);
  if (st) return st;
  if (!out) return SVDQ_ERR_INVALID_ARG;
  if (M < 1) return SVDQ_ERR_SHAPE;
  if ((st = check_k(K, precision))) return st;
  if ((st = check_rank(rank, K, K))) return st;
  const size_t m = static_cast<size_t>(M), k = static_cast<size_t>(K), r = static_cast<size_t>(rank);
  out[0] = m * k / 2;
  out[1] = precision == SVDQ_INT4 ? (k / kInt4Group) * m * 2 : (k / kMxBlock) * m;
  out[2] = m * r * 4;
  return SVDQ_OK;
}

int svdq_quantize_act_lora_down(const void* x, int M, int K, const float* smooth_inv, const void* lora_down,
                                int rank, int precision, uint8_t* xq, void* xs, float* lora_act, void* stream) {
  int st = check_precision(precision);
  if (st) return st;
  if (!x || !smooth_inv || !xq || !xs) return SVDQ_ERR_INVALID_ARG;
  if (rank > 0 && (!lora_down || !lora_act)) return SVDQ_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(smooth_inv) || !aligned16(xq) || !aligned16(xs)) return SVDQ_ERR_INVALID_ARG;
  if (rank > 0 && (!aligned16(lora_down) || !aligned16(lora_act))) return SVDQ_ERR_INVALID_ARG;
  if (M < 1) return SVDQ_ERR_SHAPE;
  if ((st = check_k(K, precision))) return st;
  if ((st = check_rank(rank, K, K))) return st;
  if ((st = current_device_ok())) return st;
  return hip_status(svdq_launch_quantize_act_lora_down(x, M, K, smooth_inv, lora_down, rank, precision, xq, xs,
                                                       lora_act, stream));
}

int svdq_gemm_w4a4_lora_up(const uint8_t* xq, const void* xs, const uint8_t* wq, const void* ws,
                           const float* lora_act, const void* lora_up, const void* bias, void* y, int M, int N,
                           int K, int rank, int precision, void* stream) {
  int st = check_precision(precision);
  if (st) return st;
  if (!xq || !xs || !wq || !ws || !y) return SVDQ_ERR_INVALID_ARG;
  if (rank > 0 && (!lora_act || !lora_up)) return SVDQ_ERR_INVALID_ARG;
  if (!aligned16(xq) || !aligned16(xs) || !aligned16(wq) || !aligned16(ws) || !aligned16(y))
    return SVDQ_ERR_INVALID_ARG;
  if (rank > 0 && (!aligned16(lora_act) || !aligned16(lora_up))) return SVDQ_ERR_INVALID_ARG;
  if (bias && !aligned16(bias)) return SVDQ_ERR_INVALID_ARG;
  if (M < 1 || N < 1) return SVDQ_ERR_SHAPE;
  if ((st = check_k(K, precision))) return st;
  if ((st = check_rank(rank, K, N))) return st;
  if ((st = check_operand_extent(M, K, precision)) || (st = check_operand_extent(N, K, precision))) return st;
  if ((st = current_device_ok())) return st;
  return hip_status(svdq_launch_gemm_w4a4_lora_up(xq, xs, wq, ws, lora_act, lora_up, bias, y, M, N, K, rank,
                                                  precision, stream));
}

int svdq_gemm_workspace_size(int M, int N, int K, int precision, size_t* out_bytes) {
  int st = check_precision(precision);
  if (st) return st;
  if (!out_bytes) return SVDQ_ERR_INVALID_ARG;
  *out_bytes = 0;
  if (M < 1 || N < 1) return SVDQ_ERR_SHAPE;
  if ((st = check_k(K, precision))) return st;
  if ((st = check_operand_extent(M, K, precision)) || (st = check_operand_extent(N, K, precision))) return st;
  if ((st = current_device_ok())) return st;
  int splits = 1, per = 0;
  svdq_gemm_split_plan(M, N, K, precision, &splits, &per, out_bytes);
  return SVDQ_OK;
}

int svdq_gemm_w4a4_lora_up_ws(const uint8_t* xq, const void* xs, const uint8_t* wq, const void* ws,
                              const float* lora_act, const void* lora_up, const void* bias, void* y, int M, int N,
                              int K, int rank, int precision, void* workspace, size_t workspace_bytes, void* stream) {
  int st = check_precision(precision);
  if (st) return st;
  if (!xq || !xs || !wq || !ws || !y) return SVDQ_ERR_INVALID_ARG;
  if (rank > 0 && (!lora_act || !lora_up)) return SVDQ_ERR_INVALID_ARG;
  if (!aligned16(xq) || !aligned16(xs) || !aligned16(wq) || !aligned16(ws) || !aligned16(y))
    return SVDQ_ERR_INVALID_ARG;
  if (rank > 0 && (!aligned16(lora_act) || !aligned16(lora_up))) return SVDQ_ERR_INVALID_ARG;
  if (bias && !aligned16(bias)) return SVDQ_ERR_INVALID_ARG;
  if (workspace && !aligned16(workspace)) return SVDQ_ERR_INVALID_ARG;
  if (M < 1 || N < 1) return SVDQ_ERR_SHAPE;
  if ((st = check_k(K, precision))) return st;
  if ((st = check_rank(rank, K, N))) return st;
  if ((st = check_operand_extent(M, K, precision)) || (st = check_operand_extent(N, K, precision))) return st;
  if ((st = current_device_ok())) return st;
  return hip_status(svdq_launch_gemm_w4a4_lora_up_ws(xq, xs, wq, ws, lora_act, lora_up, bias, y, M, N, K, rank,
                                                     precision, workspace, workspace_bytes, stream));
}

int svdq_gemm_w4a4_lora_up_gelu(const uint8_t* xq, const void* xs, const uint8_t* wq, const void* ws,
                                const float* lora_act, const void* lora_up, const void* bias, void* y, int M, int N,
                                int K, int rank, int precision, void* stream) {
  int st = check_precision(precision);
  if (st) return st;
  if (precision != SVDQ_INT4) return SVDQ_ERR_INVALID_ARG;
  if (!xq || !xs || !wq || !ws || !y) return SVDQ_ERR_INVALID_ARG;
  if (rank > 0 && (!lora_act || !lora_up)) return SVDQ_ERR_INVALID_ARG;
  if (!aligned16(xq) || !aligned16(xs) || !aligned16(wq) || !aligned16(ws) || !aligned16(y))
    return SVDQ_ERR_INVALID_ARG;
  if (rank > 0 && (!aligned16(lora_act) || !aligned16(lora_up))) return SVDQ_ERR_INVALID_ARG;
  if (bias && !aligned16(bias)) return SVDQ_ERR_INVALID_ARG;
  if (M < 1 || N < 1) return SVDQ_ERR_SHAPE;
  if ((st = check_k(K, precision))) return st;
  if ((st = check_rank(rank, K, N))) return st;
  if ((st = check_operand_extent(M, K, precision)) || (st = check_operand_extent(N, K, precision))) return st;
  if ((st = current_device_ok())) return st;
  return hip_status(svdq_launch_gemm_int4_gelu(xq, xs, wq, ws, lora_act, lora_up, bias, y, M, N, K, rank, stream));
}

int svdq_mlp_gemm_gelu_quant(const uint8_t* xq, const void* xs, const uint8_t* wq, const void* ws,
                             const float* lora_act, const void* lora_up, const void* bias, int M, int N, int K,
                             int rank, const float* smooth_inv2, const void* lora_down2, int rank2, int precision,
                             uint8_t* xq2, void* xs2, float* lora_act2, void* stream) {
  int st = check_precision(precision);
  if (st) return st;
  if (precision != SVDQ_INT4) return SVDQ_ERR_INVALID_ARG;
  if (!xq || !xs || !wq || !ws || !smooth_inv2 || !xq2 || !xs2) return SVDQ_ERR_INVALID_ARG;
  if (rank > 0 && (!lora_act || !lora_up)) return SVDQ_ERR_INVALID_ARG;
  if (rank2 > 0 && (!lora_down2 || !lora_act2)) return SVDQ_ERR_INVALID_ARG;
  if (!aligned16(xq) || !aligned16(xs) || !aligned16(wq) || !aligned16(ws) || !aligned16(smooth_inv2) ||
      !aligned16(xq2) || !aligned16(xs2))
    return SVDQ_ERR_INVALID_ARG;
  if (rank > 0 && (!aligned16(lora_act) || !aligned16(lora_up))) return SVDQ_ERR_INVALID_ARG;
  if (rank2 > 0 && (!aligned16(lora_down2) || !aligned16(lora_act2))) return SVDQ_ERR_INVALID_ARG;
  if (bias && !aligned16(bias)) return SVDQ_ERR_INVALID_ARG;
  if (M < 1 || N < 128 || N % 128 != 0) return SVDQ_ERR_SHAPE;
  if ((st = check_k(K, precision))) return st;
  if ((st = check_rank(rank, K, N))) return st;
  if ((st = check_rank(rank2, N, N))) return st;
  if ((st = check_operand_extent(M, K, precision)) || (st = check_operand_extent(N, K, precision)) ||
      (st = check_operand_extent(M, N, precision)))
    return st;
  if ((st = current_device_ok())) return st;
  return hip_status(svdq_launch_mlp_gemm_gelu_quant(xq, xs, wq, ws, lora_act, lora_up, bias, M, N, K, rank,
                                                    smooth_inv2, lora_down2, rank2, xq2, xs2, lora_act2, stream));
}

int svdq_gemm_w4a16(const void* x, const uint8_t* wq, const void* ws, const void* bias, void* y, int M, int N,
                    int K, void* stream) {
  if (!x || !wq || !ws || !y) return SVDQ_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(wq) || !aligned16(ws) || !aligned16(y)) return SVDQ_ERR_INVALID_ARG;
  if (bias && !aligned16(bias)) return SVDQ_ERR_INVALID_ARG;
  if (M < 1 || N < 1) return SVDQ_ERR_SHAPE;
  int st;
  if ((st = check_k(K, SVDQ_INT4))) return st;
  if ((st = check_operand_extent(N, K, SVDQ_INT4))) return st;
  if ((st = current_device_ok())) return st;
  return hip_status(svdq_launch_gemm_w4a16(x, wq, ws, bias, y, M, N, K, stream));
}

int svdq_unfused_linear(const void* x, int M, int K, const float* smooth_inv, const void* lora_down, int rank,
                        const uint8_t* wq, const void* ws, const void* lora_up, const void* bias, int N,
                        int precision, uint8_t* xq, void* xs, float* lora_act, void* y, void* stream) {
  int st = check_precision(precision);
  if (st) return st;
  if (!x || !smooth_inv || !wq || !ws || !xq || !xs || !y) return SVDQ_ERR_INVALID_ARG;
  if (rank > 0 && (!lora_down || !lora_up || !lora_act)) return SVDQ_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(smooth_inv) || !aligned16(wq) || !aligned16(ws) || !aligned16(xq) ||
      !aligned16(xs) || !aligned16(y))
    return SVDQ_ERR_INVALID_ARG;
  if (rank > 0 && (!aligned16(lora_down) || !aligned16(lora_up) || !aligned16(lora_act))) return SVDQ_ERR_INVALID_ARG;
  if (bias && !aligned16(bias)) return SVDQ_ERR_INVALID_ARG;
  if (M < 1 || N < 1) return SVDQ_ERR_SHAPE;
  if ((st = check_k(K, precision))) return st;
  if ((st = check_rank(rank, K, N))) return st;
  if (precision != SVDQ_INT4) return SVDQ_ERR_INVALID_ARG;
  if ((st = check_operand_extent(M, K, precision)) || (st = check_operand_extent(N, K, precision))) return st;
  if ((st = current_device_ok())) return st;
  return hip_status(svdq_launch_unfused_linear(x, M, K, smooth_inv, lora_down, rank, wq, ws, lora_up, bias, N,
                                               precision, xq, xs, lora_act, y, stream));
}

int svdq_unfused_linear_noalloc(const void* x, int M, int K, const float* smooth_inv, const void* lora_down,
                                int rank, const uint8_t* wq, const void* ws, const void* lora_up, const void* bias,
                                int N, int precision, void* y, void* stream) {
  int st = check_precision(precision);
  if (st) return st;
  if (!x || !smooth_inv || !wq || !ws || !y) return SVDQ_ERR_INVALID_ARG;
  if (rank > 0 && (!lora_down || !lora_up)) return SVDQ_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(smooth_inv) || !aligned16(wq) || !aligned16(ws) || !aligned16(y))
    return SVDQ_ERR_INVALID_ARG;
  if (rank > 0 && (!aligned16(lora_down) || !aligned16(lora_up))) return SVDQ_ERR_INVALID_ARG;
  if (bias && !aligned16(bias)) return SVDQ_ERR_INVALID_ARG;
  if (M < 1 || N < 1) return SVDQ_ERR_SHAPE;
  if ((st = check_k(K, precision))) return st;
  if ((st = check_rank(rank, K, N))) return st;
  if (precision != SVDQ_INT4) return SVDQ_ERR_INVALID_ARG;
  if ((st = check_operand_extent(M, K, precision)) || (st = check_operand_extent(N, K, precision))) return st;
  size_t off[3];
  if (noalloc_layout(M, K, rank, off) > kNoAllocScratchBytes) return SVDQ_ERR_SHAPE;
  if ((st = current_device_ok())) return st;
  return hip_status(svdq_launch_unfused_linear_noalloc(x, M, K, smooth_inv, lora_down, rank, wq, ws, lora_up, bias, N,
                                                       precision, y, stream));
}

int svdq_attention_workspace_size(int total_q, int total_k, int batch, int heads_q, int heads_k, int head_dim,
                                  size_t* out_bytes) {
  if (!out_bytes) return SVDQ_ERR_INVALID_ARG;
  *out_bytes = 0;
  const int st = check_attention_shape(total_q, total_k, batch, heads_q, heads_k, head_dim);
  if (st) return st;
  *out_bytes = svdq_attention_plan_bytes(total_q, total_k, batch, heads_q, heads_k, head_dim);
  return SVDQ_OK;
}

int svdq_attention(const void* q, const void* k, const void* v, void* o, float* lse, const int32_t* cu_seqlens_q,
                   const int32_t* cu_seqlens_k, int batch, int total_q, int total_k, int heads_q, int heads_k,
                   int head_dim, const int64_t* strides, float scale, int causal, int dtype, void* workspace,
                   size_t workspace_bytes, void* stream) {
  int st = check_dtype(dtype);
  if (st) return st;
  if ((st = check_attention_shape(total_q, total_k, batch, heads_q, heads_k, head_dim))) return st;
  if (!strides || (total_q > 0 && (!q || !o)) || (total_q > 0 && total_k > 0 && (!k || !v))) return SVDQ_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(workspace))
    return SVDQ_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(lse) | reinterpret_cast<uintptr_t>(cu_seqlens_q) |
       reinterpret_cast<uintptr_t>(cu_seqlens_k)) & 3u)
    return SVDQ_ERR_INVALID_ARG;
  if (!cu_seqlens_q != !cu_seqlens_k || (!cu_seqlens_q && batch != 1)) return SVDQ_ERR_INVALID_ARG;
  for (int i = 0; i < 8; ++i)
    if (strides[i] < 0 || strides[i] % 8 || strides[i] > 1LL << 40) return SVDQ_ERR_INVALID_ARG;
  int64_t own[8];
  std::memcpy(own, strides, sizeof(own));
  for (int i = 2; i <= 4; i += 2) {
    // one key has no stride; rows past it must still lie outside
    if (total_k <= 1) own[i] = head_dim;
    if (own[i] < head_dim || own[i] > 1 << 23) return SVDQ_ERR_INVALID_ARG;
  }
  if (!(scale > 0.f) || std::isinf(scale * 2.f)) return SVDQ_ERR_INVALID_ARG;
  if ((st = current_device_ok())) return st;
  if (total_q == 0) return SVDQ_OK;
  return hip_status(svdq_launch_attention(q, k, v, o, lse, cu_seqlens_q, cu_seqlens_k, batch, total_q, total_k, heads_q,
                                          heads_k, head_dim, own, scale, causal != 0, dtype, workspace,
                                          workspace_bytes, stream));
}

int svdq_linear16_workspace_size(int M, int N, int K, size_t* out_bytes) {
  if (!out_bytes) return SVDQ_ERR_INVALID_ARG;
  *out_bytes = 0;
  const int st = check_linear16_shape(M, N, K);
  if (st) return st;
  *out_bytes = svdq_linear16_plan_bytes(M, N, K, 0);
  if (K % 8 == 0) {
    const size_t aligned = svdq_linear16_plan_bytes(M, N, K, 1);
    if (aligned > *out_bytes) *out_bytes = aligned;
  }
  return SVDQ_OK;
}

int svdq_linear16_workspace_size_for(const void* x, int64_t ldx, const void* w, int64_t ldw, int M, int N, int K,
                                     size_t* out_bytes) {
  if (!out_bytes) return SVDQ_ERR_INVALID_ARG;
  *out_bytes = 0;
  const int st = check_linear16_shape(M, N, K);
  if (st) return st;
  *out_bytes = svdq_linear16_plan_bytes(M, N, K, svdq_linear16_aligned(x, ldx, w, ldw, K));
  return SVDQ_OK;
}

int svdq_linear16(const void* x, int64_t ldx, const void* w, int64_t ldw, const void* bias, const void* gate,
                  int64_t ld_gate, int group_rows, const void* residual, int64_t ldr, void* y, int64_t ldy, int M, int N,
                  int K, int activation, int dtype, void* workspace, size_t workspace_bytes, void* stream) {
  int st = check_dtype(dtype);
  if (st) return st;
  if (activation != SVDQ_ACT_NONE && activation != SVDQ_ACT_GELU && activation != SVDQ_ACT_SILU)
    return SVDQ_ERR_INVALID_ARG;
  if ((st = check_linear16_shape(M, N, K))) return st;
  if (!x || !w || !y) return SVDQ_ERR_INVALID_ARG;
  if (!aligned2(x) || !aligned2(w) || !aligned2(y) || !aligned2(bias) || !aligned2(gate) || !aligned2(residual) ||
      !aligned16(workspace))
    return SVDQ_ERR_INVALID_ARG;
  if (ldx < K || ldw < K || ldy < N || (residual && ldr < N)) return SVDQ_ERR_SHAPE;
  // a tile's 256 rows are addressed with 31-bit byte offsets
  const int64_t most_ld = ldx > ldw ? ldx : ldw;
  if (most_ld > 1 << 22 || 255 * most_ld + K >= 1 << 30) return SVDQ_ERR_SHAPE;
  if (gate && (ld_gate < N || group_rows < 1)) return SVDQ_ERR_SHAPE;
  if ((st = current_device_ok())) return st;
  return hip_status(svdq_launch_linear16(x, ldx, w, ldw, bias, gate, ld_gate, group_rows, residual, ldr, y, ldy, M, N, K,
                                         activation, dtype, workspace, workspace_bytes, stream));
}

int svdq_layer_norm(const void* x, int64_t ldx, const void* weight, const void* bias, const void* scale,
                    const void* shift, int64_t ld_mod, int group_rows, void* y, int64_t ldy, int M, int K, float eps,
                    int dtype, void* stream) {
  int st = check_dtype(dtype);
  if (st) return st;
  if (!x || !y) return SVDQ_ERR_INVALID_ARG;
  if (!aligned2(x) || !aligned2(y) || !aligned2(weight) || !aligned2(bias) || !aligned2(scale) || !aligned2(shift))
    return SVDQ_ERR_INVALID_ARG;
  if (!(eps >= 0.f) || std::isinf(eps)) return SVDQ_ERR_INVALID_ARG;
  if (M < 1 || M > kMostRows || K < 1 || K > 65536 || ldx < K || ldy < K) return SVDQ_ERR_SHAPE;
  if ((scale || shift) && (ld_mod < K || group_rows < 1)) return SVDQ_ERR_SHAPE;
  if ((st = current_device_ok())) return st;
  return hip_status(svdq_launch_layer_norm(x, ldx, weight, bias, scale, shift, ld_mod, group_rows < 1 ? 1 : group_rows, y,
                                           ldy, M, K, eps, dtype, stream));
}

int svdq_rms_norm(const void* x, int64_t ldx, const void* residual, int64_t ldr, const void* weight, void* sum,
                  int64_t ld_sum, void* y, int64_t ldy, uint8_t* yq, float* ys, int M, int K, float eps, int dtype,
                  void* stream) {
  int st = check_dtype(dtype);
  if (st) return st;
  if (!x || !yq != !ys || !y == !yq) return SVDQ_ERR_INVALID_ARG;
  if (!aligned2(x) || !aligned2(residual) || !aligned2(weight) || !aligned2(sum) || !aligned2(y) || !aligned16(yq) ||
      !aligned4(ys))
    return SVDQ_ERR_INVALID_ARG;
  if (!(eps >= 0.f) || std::isinf(eps)) return SVDQ_ERR_INVALID_ARG;
  if (M < 1 || M > kMostRows || K < 1 || K > 65536 || (yq && K % 16)) return SVDQ_ERR_SHAPE;
  if (ldx < K || (residual && ldr < K) || (sum && ld_sum < K) || (y && ldy < K)) return SVDQ_ERR_SHAPE;
  if ((st = current_device_ok())) return st;
  return hip_status(svdq_launch_rms_norm(x, ldx, residual, ldr, weight, sum, ld_sum, y, ldy, yq, ys, M, K, eps, dtype, stream));
}

int svdq_quantize_fp8(const void* x, int64_t ldx, uint8_t* xq, float* xs, int M, int K, int dtype, void* stream) {
  int st = check_dtype(dtype);
  if (st) return st;
  if (!x || !xq || !xs || !aligned2(x) || !aligned16(xq) || !aligned4(xs)) return SVDQ_ERR_INVALID_ARG;
  if ((st = check_codes(K))) return st;
  if (M < 1 || M > kMostRows || ldx < K) return SVDQ_ERR_SHAPE;
  if ((st = current_device_ok())) return st;
  return hip_status(svdq_launch_quantize_fp8(x, ldx, xq, xs, M, K, dtype, stream));
}

int svdq_gemm_fp8(const uint8_t* xq, const float* xs, const uint8_t* wq, const float* ws, const void* bias, const void* gate,
                  int64_t ld_gate, int group_rows, const void* residual, int64_t ldr, void* y, int64_t ldy, int M, int N,
                  int K, int activation, int dtype, void* stream) {
  int st = check_dtype(dtype);
  if (st) return st;
  if (activation != SVDQ_ACT_NONE && activation != SVDQ_ACT_GELU && activation != SVDQ_ACT_SILU)
    return SVDQ_ERR_INVALID_ARG;
  if ((st = check_gemm_fp8_shape(M, N, K))) return st;
  if (!xq || !xs || !wq || !ws || !y) return SVDQ_ERR_INVALID_ARG;
  if (!aligned16(xq) || !aligned4(xs) || !aligned16(wq) || !aligned4(ws) || !aligned2(y) || !aligned2(bias) ||
      !aligned2(gate) || !aligned2(residual))
    return SVDQ_ERR_INVALID_ARG;
  if (ldy < N || (residual && ldr < N) || (gate && (ld_gate < N || group_rows < 1))) return SVDQ_ERR_SHAPE;
  if ((st = current_device_ok())) return st;
  return hip_status(svdq_launch_gemm_fp8(xq, xs, wq, ws, bias, gate, ld_gate, group_rows < 1 ? 1 : group_rows, residual, ldr,
                                         y, ldy, M, N, K, activation, dtype, stream));
}

int svdq_cache_append(const void* q, const void* k, const void* v, void* q_out, const int64_t* strides, uint8_t* k_cache,
                      uint8_t* v_cache, int8_t* exponents, int pages, const int32_t* block_table, int table_width,
                      const int32_t* lengths, const int32_t* cu_seqlens, int batch, int total, int heads_q, int heads_k,
                      int head_dim, const float* rope, int rope_rows, int rotary, int interleaved, int dtype, void* stream) {
  int st = check_dtype(dtype);
  if (st) return st;
  if ((st = check_paged_shape(total, batch, table_width, heads_q, heads_k, head_dim))) return st;
  if (pages < 1 || (!cu_seqlens && total != batch)) return SVDQ_ERR_SHAPE;
  if (rotary < 0 || rotary % 16 || rotary > head_dim || !rope != !rotary || (rope && rope_rows < 1)) return SVDQ_ERR_SHAPE;
  if (!strides || !k_cache || !v_cache || !exponents || !block_table || !lengths || !q != !q_out ||
      (total > 0 && (!k || !v)))
    return SVDQ_ERR_INVALID_ARG;
  if (!aligned2(q) || !aligned2(k) || !aligned2(v) || !aligned2(q_out) || !aligned16(k_cache) || !aligned16(v_cache) ||
      !aligned4(block_table) || !aligned4(lengths) || !aligned4(cu_seqlens) || !aligned4(rope))
    return SVDQ_ERR_INVALID_ARG;
  if (!strides_fit(strides, 8, 1)) return SVDQ_ERR_INVALID_ARG;
  if ((st = current_device_ok())) return st;
  if (total == 0) return SVDQ_OK;
  return hip_status(svdq_launch_cache_append(q, k, v, q_out, strides, k_cache, v_cache, exponents, pages, block_table,
                                             table_width, lengths, cu_seqlens, batch, total, heads_q, heads_k, head_dim, rope,
                                             rope_rows, rotary, interleaved != 0, dtype, stream));
}

int svdq_attention_paged_workspace_size(int total, int batch, int table_width, int heads_q, int heads_k, int head_dim,
                                        size_t* out_bytes) {
  if (!out_bytes) return SVDQ_ERR_INVALID_ARG;
  *out_bytes = 0;
  const int st = check_paged_shape(total, batch, table_width, heads_q, heads_k, head_dim);
  if (st) return st;
  *out_bytes = svdq_attention_paged_plan_bytes(total, batch, table_width, heads_q, heads_k, head_dim);
  return SVDQ_OK;
}

int svdq_attention_paged(const void* q, void* o, float* lse, const int64_t* strides, const uint8_t* k_cache,
                         const uint8_t* v_cache, const int8_t* exponents, int pages, const int32_t* block_table,
                         int table_width, const int32_t* lengths, const int32_t* cu_seqlens, int batch, int total,
                         int heads_q, int heads_k, int head_dim, float scale, int causal, int dtype, void* workspace,
                         size_t workspace_bytes, void* stream) {
  int st = check_dtype(dtype);
  if (st) return st;
  if ((st = check_paged_shape(total, batch, table_width, heads_q, heads_k, head_dim))) return st;
  if (pages < 1 || (!cu_seqlens && total != batch)) return SVDQ_ERR_SHAPE;
  if (!strides || !k_cache || !v_cache || !exponents || !block_table || !lengths || (total > 0 && (!q || !o)))
    return SVDQ_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(o) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(workspace) ||
      !aligned4(lse) || !aligned4(block_table) || !aligned4(lengths) || !aligned4(cu_seqlens))
    return SVDQ_ERR_INVALID_ARG;
  if (!strides_fit(strides, 4, 8)) return SVDQ_ERR_INVALID_ARG;
  if (!(scale >= 0x1p-80f) || !(scale < 0x1p80f)) return SVDQ_ERR_INVALID_ARG;   // a page's exponent goes with it
  if ((st = current_device_ok())) return st;
  if (total == 0) return SVDQ_OK;
  return hip_status(svdq_launch_attention_paged(q, o, lse, strides, k_cache, v_cache, exponents, pages, block_table,
                                                table_width, lengths, cu_seqlens, batch, total, heads_q, heads_k, head_dim,
                                                scale, causal != 0, dtype, workspace, workspace_bytes, stream));
}

int svdq_bench_mfma_ceiling(int precision, int blocks, int iters, float* out, void* stream) {
  if (!out || !aligned16(out)) return SVDQ_ERR_INVALID_ARG;
  if (precision != SVDQ_INT4 && precision != SVDQ_MXFP4) return SVDQ_ERR_INVALID_ARG;
  if (blocks < 1 || iters < 1) return SVDQ_ERR_SHAPE;
  int st;
  if ((st = current_device_ok())) return st;
  return hip_status(svdq_launch_mfma_ceiling(precision, blocks, iters, out, stream));
}

int svdq_debug_group_partials(const uint8_t* xq, const uint8_t* wq, int M, int N, int K, int m0, int n0, int mt,
                              int nt, int32_t* out, void* stream) {
  if (!xq || !wq || !out) return SVDQ_ERR_INVALID_ARG;
  if (!aligned16(xq) || !aligned16(wq) || !aligned16(out)) return SVDQ_ERR_INVALID_ARG;
  if (M < 1 || N < 1 || mt < 1 || nt < 1) return SVDQ_ERR_SHAPE;
  int st = check_k(K, SVDQ_INT4);
  if (st) return st;
  if (m0 < 0 || n0 < 0 || m0 + static_cast<long long>(mt) > M || n0 + static_cast<long long>(nt) > N)
    return SVDQ_ERR_SHAPE;
  if ((st = check_operand_extent(M, K, SVDQ_INT4)) || (st = check_operand_extent(N, K, SVDQ_INT4))) return st;
  if ((st = current_device_ok())) return st;
  return hip_status(svdq_launch_debug_group_partials(xq, wq, M, N, K, m0, n0, mt, nt, out, stream));
}

int svdq_debug_attention_plan(int total_q, int total_k, int batch, int heads_q, int heads_k, int head_dim, int causal,
                              int32_t* plan) {
  if (!plan) return SVDQ_ERR_INVALID_ARG;
  const int st = check_attention_shape(total_q, total_k, batch, heads_q, heads_k, head_dim);
  if (st) return st;
  svdq_attention_plan(total_q, total_k, batch, heads_q, heads_k, head_dim, causal, plan);
  return SVDQ_OK;
}

int svdq_debug_linear16_plan(int M, int N, int K, int aligned, int32_t* plan) {
  if (!plan) return SVDQ_ERR_INVALID_ARG;
  const int st = check_linear16_shape(M, N, K);
  if (st) return st;
  if (aligned && K % 8) return SVDQ_ERR_SHAPE;
  svdq_linear16_plan(M, N, K, aligned, plan);
  return SVDQ_OK;
}

int svdq_debug_attention_paged_plan(int total, int batch, int table_width, int heads_q, int heads_k, int head_dim,
                                    int32_t* plan) {
  if (!plan) return SVDQ_ERR_INVALID_ARG;
  const int st = check_paged_shape(total, batch, table_width, heads_q, heads_k, head_dim);
  if (st) return st;
  svdq_attention_paged_plan(total, batch, table_width, heads_q, heads_k, head_dim, plan);
  return SVDQ_OK;
}

int svdq_debug_gemm_fp8_plan(int M, int N, int K, int32_t* plan) {
  if (!plan) return SVDQ_ERR_INVALID_ARG;
  const int st = check_gemm_fp8_shape(M, N, K);
  if (st) return st;
  svdq_gemm_fp8_plan(M, N, K, plan);
  return SVDQ_OK;
}

}  // extern "C"
