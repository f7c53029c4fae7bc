// Adaptive layer norm for gfx950.
//
//   y = (x - mean) rstd [* w + b] [* (1 + scale_g) + shift_g],
//   mean and variance over the row's K values, rstd = 1 / sqrt(var + eps),
//   g = row / group_rows
//
// Memory-bound: x is read once and y written once, with the row held in
// registers between (16 bytes a lane and chunk).  The variance is that of
// the deviations from the mean, a second sum over the registers: rows far
// off centre lose nothing.  4608 x 3072 with scale and shift: 14.4 us, 12.2
// alone (4.6 TB/s; a copy of the same bytes 12.6).  A row belongs to LANES
// lanes of a wave (rows of up to 4096 values) or to WAVES whole waves that
// join their sums in LDS.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "svdq_device.h"
#include "svdq_internal.h"

namespace {

using namespace svdq_dev;

struct NormArgs {
  const uint16_t *x, *weight, *bias, *scale, *shift;
  uint16_t* y;
  int64_t ldx, ldy, ld_mod;
  int M, K, group_rows;
  float eps;
};

template <int LANES, int WAVES>
__device__ __forceinline__ float row_total(float v, float* lds) {
#pragma unroll
  for (int o = LANES / 2; o; o >>= 1) v += __shfl_xor(v, o);
  if constexpr (WAVES > 1) {
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0.f;
#pragma unroll
    for (int i = 0; i < WAVES; ++i) v += lds[i];
  }
  return v;
}

// Chunk of 8 values at k of a row of K: always one wide load inside the row,
// so that a lane's loads go out together.  Past the row: its last 8 values.
// TAIL (K % 8 != 0): the chunk that passes the end takes the row's last 8
// values and moves its own to the front, zeros after them.
template <bool TAIL>
__device__ __forceinline__ v4u row_chunk(const uint16_t* p, int k, int K) {
  if constexpr (!TAIL) return load8(p + min(k, K - 8));
  if (K < 8) return load8(p, K);
  v4u v = load8(p + min(k, K - 8));
  const int over = k + 8 - K;
  if (over > 0 && over < 8) {
    const int bits = 16 * over;
    uint64_t lo = v[0] | static_cast<uint64_t>(v[1]) << 32, hi = v[2] | static_cast<uint64_t>(v[3]) << 32;
    if (bits >= 64) {
      lo = hi >> (bits - 64);
      hi = 0;
    } else {
      lo = lo >> bits | hi << (64 - bits);
      hi >>= bits;
    }
    v = v4u{static_cast<uint32_t>(lo), static_cast<uint32_t>(lo >> 32), static_cast<uint32_t>(hi),
            static_cast<uint32_t>(hi >> 32)};
  }
  return v;
}

// workgroups along x, the others along y: one axis of a launch holds less
// than 2^32 threads
constexpr unsigned kGridX = 1u << 21;

// CHUNKS chunks of 8 values a lane
template <typename E, int LANES, int WAVES, int CHUNKS, bool TAIL>
__global__ __launch_bounds__(WAVES > 1 ? WAVES * 64 : 256) void k_layer_norm(NormArgs a) {
  static_assert(WAVES == 1 || LANES == 64, "several waves take whole rows");
  constexpr int kThreads = WAVES * LANES;                  // threads of a row
  constexpr int kRows = WAVES > 1 ? 1 : 256 / LANES;       // rows of a workgroup
  __shared__ float sums[2][WAVES];
  const int t = threadIdx.x % kThreads;
  const int64_t row = (static_cast<int64_t>(blockIdx.y) * kGridX + blockIdx.x) * kRows + threadIdx.x / kThreads;
  if (row >= a.M) return;   // whole rows' lanes leave together
  const uint16_t* const x = a.x + row * a.ldx;
  v4u raw[CHUNKS];
#pragma unroll
  for (int c = 0; c < CHUNKS; ++c) raw[c] = row_chunk<TAIL>(x, (c * kThreads + t) * 8, a.K);
  float f[CHUNKS][8];
  float total = 0.f;
#pragma unroll
  for (int c = 0; c < CHUNKS; ++c) {
    unpack8<E>((c * kThreads + t) * 8 < a.K ? raw[c] : v4u{0, 0, 0, 0}, f[c]);
#pragma unroll
    for (int e = 0; e < 8; ++e) total += f[c][e];
  }
  const float inv_k = 1.f / a.K;
  const float mean = row_total<LANES, WAVES>(total, sums[0]) * inv_k;
  float square = 0.f;
#pragma unroll
  for (int c = 0; c < CHUNKS; ++c) {
    const int left = a.K - (c * kThreads + t) * 8;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      f[c][e] -= mean;
      square += (TAIL ? e < left : left > 0) ? f[c][e] * f[c][e] : 0.f;
    }
  }
  const float rstd = 1.f / sqrtf(row_total<LANES, WAVES>(square, sums[1]) * inv_k + a.eps);
  const int64_t g = row / a.group_rows;
  uint16_t* const y = a.y + row * a.ldy;
#pragma unroll
  for (int c = 0; c < CHUNKS; ++c) {
    const int k = (c * kThreads + t) * 8;
    if (k >= a.K) break;
    float w[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) f[c][e] *= rstd;
    if (a.weight) {
      unpack8<E>(row_chunk<TAIL>(a.weight, k, a.K), w);
#pragma unroll
      for (int e = 0; e < 8; ++e) f[c][e] *= w[e];
    }
    if (a.bias) {
      unpack8<E>(row_chunk<TAIL>(a.bias, k, a.K), w);
#pragma unroll
      for (int e = 0; e < 8; ++e) f[c][e] += w[e];
    }
    if (a.scale) {
      unpack8<E>(row_chunk<TAIL>(a.scale + g * a.ld_mod, k, a.K), w);
#pragma unroll
      for (int e = 0; e < 8; ++e) f[c][e] *= 1.f + w[e];
    }
    if (a.shift) {
      unpack8<E>(row_chunk<TAIL>(a.shift + g * a.ld_mod, k, a.K), w);
#pragma unroll
      for (int e = 0; e < 8; ++e) f[c][e] += w[e];
    }
    // streamed: y is not read again here
    if (!TAIL || k + 8 <= a.K)
      stream8(y + k, pack8<E>(f[c]));
    else
      store8(y + k, pack8<E>(f[c]), a.K - k);
  }
}

template <typename E, int LANES, int WAVES, int CHUNKS>
void start(const NormArgs& a, hipStream_t stream) {
  constexpr int kRows = WAVES > 1 ? 1 : 256 / LANES;
  const unsigned blocks = static_cast<unsigned>((static_cast<int64_t>(a.M) + kRows - 1) / kRows);
  const dim3 grid(blocks < kGridX ? blocks : kGridX, (blocks + kGridX - 1) / kGridX);
  constexpr int kBlock = WAVES > 1 ? WAVES * 64 : 256;
  if (a.K % 8)
    k_layer_norm<E, LANES, WAVES, CHUNKS, true><<<grid, kBlock, 0, stream>>>(a);
  else
    k_layer_norm<E, LANES, WAVES, CHUNKS, false><<<grid, kBlock, 0, stream>>>(a);
}

template <typename E>
int launch(const NormArgs& a, hipStream_t stream) {
  const int chunks = (a.K + 7) / 8;
  if (chunks <= 8)
    start<E, 8, 1, 1>(a, stream);
  else if (chunks <= 16)
    start<E, 16, 1, 1>(a, stream);
  else if (chunks <= 32)
    start<E, 32, 1, 1>(a, stream);
  else if (chunks <= 64)
    start<E, 64, 1, 1>(a, stream);
  else if (chunks <= 128)
    start<E, 64, 1, 2>(a, stream);
  else if (chunks <= 256)
    start<E, 64, 1, 4>(a, stream);
  else if (chunks <= 384)
    start<E, 64, 1, 6>(a, stream);
  else if (chunks <= 512)
    start<E, 64, 1, 8>(a, stream);
  else if (chunks <= 1024)
    start<E, 64, 4, 4>(a, stream);
  else if (chunks <= 2048)
    start<E, 64, 4, 8>(a, stream);
  else
    start<E, 64, 16, 8>(a, stream);
  return static_cast<int>(hipGetLastError());
}

}  // namespace

extern "C" int svdq_launch_layer_norm(const void* x, int64_t ldx, const void* weight, const void* bias, const void* scale,
                                      const void* shift, int64_t ld_mod, int group_rows, void* y, int64_t ldy, int M,
                                      int K, float eps, int dtype, void* stream) {
  NormArgs a{};
  a.x = static_cast<const uint16_t*>(x);
  a.weight = static_cast<const uint16_t*>(weight);
  a.bias = static_cast<const uint16_t*>(bias);
  a.scale = static_cast<const uint16_t*>(scale);
  a.shift = static_cast<const uint16_t*>(shift);
  a.y = static_cast<uint16_t*>(y);
  a.ldx = ldx;
  a.ldy = ldy;
  a.ld_mod = ld_mod;
  a.M = M;
  a.K = K;
  a.group_rows = group_rows;
  a.eps = eps;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  return dtype == SVDQ_BF16 ? launch<Bf16>(a, s) : launch<F16>(a, s);
}
