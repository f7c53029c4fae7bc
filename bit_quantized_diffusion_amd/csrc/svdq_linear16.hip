// 16-bit linear with bias, activation, gate and residual in its epilogue:
//
//   y = residual + gate_g * act(x W^T + b),  g = row / group_rows
//
// for gfx950.  x [M][K], W [N][K] (nn.Linear layout), y [M][N]; products in
// the matrix core with fp32 accumulation, the epilogue in fp32, one rounding.
//
// The matrix core's A operand is W and its B operand is x, so that a lane's
// results lie along n, the dense dimension of y.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "svdq_device.h"
#include "svdq_internal.h"

namespace {

using namespace svdq_dev;

struct LinArgs {
  const uint16_t *x, *w, *bias, *gate, *residual;
  uint16_t* y;
  float* part;       // [splits][M][N] fp32, splits > 1
  int64_t ldx, ldw, ld_gate, ldr, ldy;
  int M, N, K, group_rows, act;
  int splits, stages_per_split;
};

__device__ __forceinline__ float activate(float z, int act) {
  if (act == SVDQ_ACT_NONE) return z;
  // silu: z / (1 + exp(-z)); the tanh form of gelu is z / (1 + exp(-2 u)),
  // u = sqrt(2 / pi) (z + 0.044715 z^3)
  constexpr float kLog2e = 1.4426950408889634f;
  constexpr float kG = 2.f * 0.7978845608028654f * kLog2e;
  const float t = act == SVDQ_ACT_SILU ? z * kLog2e : z * (kG + kG * 0.044715f * z * z);
  return z / (1.f + exp2_fast(-t));
}

// A lane's 8 consecutive channels of one row: the epilogue and the store.
template <typename E>
struct Columns {
  float bias[8];
  float gate[8];
  int n, count;      // first channel, channels inside N
  int64_t g;         // the group whose gate is held

  __device__ __forceinline__ void init(const LinArgs& a, int n_) {
    n = n_;
    count = min(a.N - n, 8);
    g = -1;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      bias[e] = 0.f;
      gate[e] = 1.f;
    }
    if (a.bias && count > 0) unpack8<E>(load8(a.bias + n, count), bias);
  }
  __device__ __forceinline__ void finish(const LinArgs& a, int m, float (&f)[8]) {
    if (m >= a.M || count <= 0) return;
    if (a.gate) {
      const int64_t gm = m / a.group_rows;
      if (gm != g) {
        g = gm;
        unpack8<E>(load8(a.gate + g * a.ld_gate + n, count), gate);
      }
    }
    float r[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (a.residual) unpack8<E>(load8(a.residual + m * a.ldr + n, count), r);
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = r[e] + gate[e] * activate(f[e] + bias[e], a.act);
    store8(a.y + m * a.ldy + n, pack8<E>(f), count);
  }
};

// 16-byte chunk c of row r of a tile with 64 values a row (128 bytes; two
// rows share the LDS banks) sits at chunk c ^ swz(r): the reads of one chunk
// of 16 consecutive rows fall in distinct banks.
__device__ __forceinline__ int swz(int r) { return (r >> 1) & 7; }

// ---------------------------------------------------------------------------
// Tiles of BN channels x BM rows, WN x WM waves, K in stages of 64.  DMA: both
// operands come straight to LDS, double-buffered (needs 16-byte aligned rows
// and K % 8 == 0); else through registers with unaligned loads.
// ---------------------------------------------------------------------------

template <typename E, int BN, int BM, int WN, int WM, bool DMA>
__global__ __launch_bounds__(WN * WM * 64, 2) void k_linear16(LinArgs a) {
  constexpr int kWaves = WN * WM;
  constexpr int TN = BN / WN / 32, TM = BM / WM / 32;    // 32 x 32 tiles of a wave
  constexpr int kRowB = 128;                             // bytes of a row and stage
  constexpr int kStage = (BN + BM) * kRowB;
  constexpr int kLoads = kStage / 1024 / kWaves;         // 1 KB (8 rows) each
  static_assert(kStage % (1024 * kWaves) == 0, "loads divide evenly");
  __shared__ __attribute__((aligned(1024))) uint8_t lds[2 * kStage];
  static_assert(kWaves * 32 * TN * 32 * 4 <= 2 * kStage, "the epilogue's staging fits");

  const int lane = threadIdx.x & 63, l32 = lane & 31, h = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wn = wave % WN, wm = wave / WN;

  // tile: each XCD takes a contiguous range of tiles, walked in groups of 8
  // rows of tiles, so that tiles that run together share operand panels
  const int tn = (a.N + BN - 1) / BN, tm = (a.M + BM - 1) / BM, tiles = tn * tm;
  int id = blockIdx.x;
  {
    const int per = (tiles + 7) / 8, x = id & 7, full = tiles - 8 * (per - 1);   // the first `full` XCDs take `per`
    id = (x < full ? x * per : full * per + (x - full) * (per - 1)) + (id >> 3);
  }
  const int group = id / (8 * tn), in = id - group * 8 * tn;
  const int gm = min(8, tm - group * 8);
  const int m0 = (group * 8 + in % gm) * BM, n0 = in / gm * BN;

  const int stages = (a.K + 63) / 64;
  const int s0 = blockIdx.y * a.stages_per_split, s1 = min(s0 + a.stages_per_split, stages);

  const uint32_t base = lds_addr(lds);
  // load n of a wave: rows 8 (wave kLoads + n) .. + 7 of the BN + BM rows
  int voff[kLoads];
#pragma unroll
  for (int n = 0; n < kLoads; ++n) {
    const int r = (wave * kLoads + n) * 8 + (lane >> 3);
    const bool is_x = r >= BN;
    const int rr = is_x ? r - BN : r;
    voff[n] = static_cast<int>(rr * (is_x ? a.ldx : a.ldw) * 2) + (((lane & 7) ^ swz(rr)) << 4);
  }
  auto issue = [&](int st, int buf) {
    const int k0 = st * 64;
    const uint16_t* const pw = a.w + n0 * a.ldw + k0;
    const uint16_t* const px = a.x + m0 * a.ldx + k0;
    const auto rw = buffer_of(pw, ((a.N - n0 - 1) * a.ldw + a.K - k0) * 2);
    const auto rx = buffer_of(px, ((a.M - m0 - 1) * a.ldx + a.K - k0) * 2);
    const bool tail = k0 + 64 > a.K;
#pragma unroll
    for (int n = 0; n < kLoads; ++n) {
      const int r8 = wave * kLoads + n;
      int vo = voff[n];
      if (tail && k0 + ((lane & 7) ^ swz((r8 * 8 + (lane >> 3)) % BN)) * 8 >= a.K) vo = kOutside;
      dma_b128(r8 * 8 >= BN ? rx : rw, base + buf * kStage + r8 * 1024, vo);
    }
  };
  v4u held[DMA ? 1 : kLoads];
  auto fetch = [&](int st) {
#pragma unroll
    for (int n = 0; n < kLoads; ++n) {
      const int r = (wave * kLoads + n) * 8 + (lane >> 3);
      const bool is_x = r >= BN;
      const int rr = is_x ? r - BN : r;
      const int k = st * 64 + ((lane & 7) ^ swz(rr)) * 8;
      held[DMA ? 0 : n] = v4u{0, 0, 0, 0};
      const int64_t row = is_x ? m0 + rr : n0 + rr;
      if (row < (is_x ? a.M : a.N) && k < a.K)
        held[DMA ? 0 : n] = load8((is_x ? a.x + row * a.ldx : a.w + row * a.ldw) + k, a.K - k);
    }
  };
  auto put = [&](int buf) {
#pragma unroll
    for (int n = 0; n < kLoads; ++n)
      *reinterpret_cast<v4u*>(lds + buf * kStage + (wave * kLoads + n) * 1024 + lane * 16) = held[DMA ? 0 : n];
  };

  // LDS offsets of the lane's operand reads: row, chunk 2 step + h
  uint32_t ra[4];
#pragma unroll
  for (int s = 0; s < 4; ++s) ra[s] = l32 * kRowB + (((2 * s + h) ^ swz(l32)) << 4);
  const uint32_t wbase = base + wn * TN * 32 * kRowB, xbase = base + (BN + wm * TM * 32) * kRowB;

  v16f acc[TN][TM];
#pragma unroll
  for (int i = 0; i < TN; ++i)
#pragma unroll
    for (int j = 0; j < TM; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.f;

  auto compute = [&](int buf) {
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      v4u fw[TN], fx[TM];
#pragma unroll
      for (int i = 0; i < TN; ++i) fw[i] = lds_read16(wbase + buf * kStage + ra[s] + i * 32 * kRowB);
#pragma unroll
      for (int j = 0; j < TM; ++j) fx[j] = lds_read16(xbase + buf * kStage + ra[s] + j * 32 * kRowB);
#pragma unroll
      for (int i = 0; i < TN; ++i)
#pragma unroll
        for (int j = 0; j < TM; ++j) acc[i][j] = E::mfma(fw[i], fx[j], acc[i][j]);
    }
  };

  if constexpr (DMA) {
    issue(s0, 0);
    lds_wait_barrier<0>();
    for (int st = s0; st < s1; ++st) {
      const int b = (st - s0) & 1;
      if (st + 1 < s1) issue(st + 1, b ^ 1);
      compute(b);
      lds_wait_barrier<0>();
    }
  } else {
    fetch(s0);
    put(0);
    __syncthreads();
    for (int st = s0; st < s1; ++st) {
      const int b = (st - s0) & 1;
      if (st + 1 < s1) fetch(st + 1);
      compute(b);
      if (st + 1 < s1) put(b ^ 1);
      __syncthreads();
    }
  }

  // Epilogue through the wave's own LDS: 32 rows x 32 TN channels in fp32, 16-byte
  // chunk c of row r at chunk c ^ (r % (8 TN)), then whole row segments
  constexpr int kC4 = TN * 8;              // 16-byte chunks of a staged row
  float* const stage = reinterpret_cast<float*>(lds + wave * 32 * kC4 * 16);
  constexpr int kLanesRow = TN * 4;        // lanes of a row, 8 channels each
  const int c8 = lane % kLanesRow;
  Columns<E> col;
  const int nl = n0 + wn * TN * 32 + c8 * 8;
  if (a.splits == 1) col.init(a, nl);
#pragma unroll
  for (int j = 0; j < TM; ++j) {
#pragma unroll
    for (int i = 0; i < TN; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        *reinterpret_cast<v4f*>(stage + (l32 * kC4 + ((i * 8 + 2 * q + h) ^ (l32 & (kC4 - 1)))) * 4) =
            v4f{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
#pragma unroll 2
    for (int it = 0; it < 32 * kLanesRow / 64; ++it) {
      const int r = it * (64 / kLanesRow) + lane / kLanesRow;
      const v4f lo = *reinterpret_cast<const v4f*>(stage + (r * kC4 + ((2 * c8) ^ (r & (kC4 - 1)))) * 4);
      const v4f hi = *reinterpret_cast<const v4f*>(stage + (r * kC4 + ((2 * c8 + 1) ^ (r & (kC4 - 1)))) * 4);
      float f[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
      const int m = m0 + (wm * TM + j) * 32 + r;
      if (a.splits == 1) {
        col.finish(a, m, f);
      } else if (m < a.M && nl < a.N) {
        float* p = a.part + (static_cast<int64_t>(blockIdx.y) * a.M + m) * a.N + nl;
        if (nl + 8 <= a.N && (a.N & 3) == 0) {
          *reinterpret_cast<v4f*>(p) = lo;
          *reinterpret_cast<v4f*>(p + 4) = hi;
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (nl + e < a.N) p[e] = f[e];
        }
      }
    }
  }
}

// Sum of the splits in their order, then the epilogue: 8 channels a thread.
template <typename E>
__global__ __launch_bounds__(256) void k_linear16_join(LinArgs a) {
  const int chunks = (a.N + 7) / 8;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= static_cast<int64_t>(chunks) * a.M) return;
  const int m = static_cast<int>(i / chunks);
  Columns<E> col;
  col.init(a, static_cast<int>(i - static_cast<int64_t>(m) * chunks) * 8);
  float f[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  for (int s = 0; s < a.splits; ++s) {
    const float* p = a.part + (static_cast<int64_t>(s) * a.M + m) * a.N + col.n;
    if (col.count == 8 && (a.N & 3) == 0) {
      const v4f lo = *reinterpret_cast<const v4f*>(p), hi = *reinterpret_cast<const v4f*>(p + 4);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        f[e] += lo[e];
        f[4 + e] += hi[e];
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (e < col.count) f[e] += p[e];
    }
  }
  col.finish(a, m, f);
}

// ---------------------------------------------------------------------------
// Few rows (M <= 32): bound by reading W once.  A workgroup takes 32
// channels; its 4 waves take the stages of 128 k in turn, each through LDS of
// its own (kDepth stages in flight, no barrier in the loop), and join at the
// end.  XL: 1 KB loads that bring in the rows of x (4 rows each).
// ---------------------------------------------------------------------------

template <typename E, int XL>
__global__ __launch_bounds__(256, 1) void k_linear16_few(LinArgs a) {
  constexpr int kWaves = 4, kDepth = XL > 4 ? 2 : 3;
  constexpr int kRowB = 256, kStage = (32 + 4 * XL) * kRowB;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[kWaves * kDepth * kStage];
  const int lane = threadIdx.x & 63, l32 = lane & 31, h = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n0 = blockIdx.x * 32;
  const int stages = (a.K + 127) / 128;

  // 256-byte rows; chunk c of row r at chunk c ^ (r % 16)
  int vw[8], vx[XL];
#pragma unroll
  for (int n = 0; n < 8; ++n) {
    const int r = 4 * n + (lane >> 4);
    vw[n] = static_cast<int>(r * a.ldw * 2) + (((lane & 15) ^ (r & 15)) << 4);
  }
#pragma unroll
  for (int n = 0; n < XL; ++n) {
    const int r = 4 * n + (lane >> 4);
    vx[n] = static_cast<int>(r * a.ldx * 2) + (((lane & 15) ^ (r & 15)) << 4);
  }
  const uint32_t base = lds_addr(lds) + wave * kDepth * kStage;
  auto issue = [&](int st, int slot) {
    const int k0 = st * 128;
    const auto rw = buffer_of(a.w + n0 * a.ldw + k0, ((a.N - n0 - 1) * a.ldw + a.K - k0) * 2);
    const auto rx = buffer_of(a.x + k0, ((a.M - 1) * a.ldx + a.K - k0) * 2);
    const bool tail = k0 + 128 > a.K;
    const uint32_t d = base + slot * kStage;
#pragma unroll
    for (int n = 0; n < 8; ++n) {
      const int c = (lane & 15) ^ ((4 * n + (lane >> 4)) & 15);
      dma_b128(rw, d + n * 1024, tail && k0 + c * 8 >= a.K ? kOutside : vw[n]);
    }
#pragma unroll
    for (int n = 0; n < XL; ++n) {
      const int c = (lane & 15) ^ ((4 * n + (lane >> 4)) & 15);
      dma_b128(rx, d + (8 + n) * 1024, tail && k0 + c * 8 >= a.K ? kOutside : vx[n]);
    }
  };
  uint32_t ra[8];
#pragma unroll
  for (int s = 0; s < 8; ++s) ra[s] = l32 * kRowB + (((2 * s + h) ^ (l32 & 15)) << 4);
  // rows of x past the staged ones repeat the staged ones; their results are not stored
  const int xrow = l32 % (4 * XL);
  uint32_t rx[8];
#pragma unroll
  for (int s = 0; s < 8; ++s) rx[s] = (32 + xrow) * kRowB + (((2 * s + h) ^ (xrow & 15)) << 4);

  v16f acc[2];
#pragma unroll
  for (int e = 0; e < 16; ++e) acc[0][e] = acc[1][e] = 0.f;
#pragma unroll
  for (int i = 0; i < kDepth; ++i)
    if (wave + i * kWaves < stages) issue(wave + i * kWaves, i);
  int slot = 0;
  for (int st = wave; st < stages; st += kWaves) {
    const int more = (stages - 1 - st) / kWaves;   // stages of this wave still in flight
    if (kDepth == 3 && more >= 2)
      vm_wait<2 * (8 + XL)>();
    else if (more >= 1)
      vm_wait<8 + XL>();
    else
      vm_wait<0>();
    const uint32_t b = base + slot * kStage;
#pragma unroll
    for (int s = 0; s < 8; ++s) acc[s & 1] = E::mfma(lds_read16(b + ra[s]), lds_read16(b + rx[s]), acc[s & 1]);
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // the slot is read out before it is loaded again
    if (st + kDepth * kWaves < stages) issue(st + kDepth * kWaves, slot);
    slot = slot + 1 == kDepth ? 0 : slot + 1;
  }

  // join: [wave][row m][32 channels] fp32, the rows padded by 4
  constexpr int kRow = 36;
  static_assert(kWaves * 32 * kRow * 4 <= kWaves * kDepth * kStage, "the join fits");
  __syncthreads();
  float* const out = reinterpret_cast<float*>(lds) + wave * 32 * kRow;
#pragma unroll
  for (int q = 0; q < 4; ++q)
    *reinterpret_cast<v4f*>(out + l32 * kRow + 8 * q + 4 * h) =
        v4f{acc[0][4 * q] + acc[1][4 * q], acc[0][4 * q + 1] + acc[1][4 * q + 1], acc[0][4 * q + 2] + acc[1][4 * q + 2],
            acc[0][4 * q + 3] + acc[1][4 * q + 3]};
  __syncthreads();
  const int m = threadIdx.x >> 2;
  if (m >= a.M || m >= 32) return;
  Columns<E> col;
  col.init(a, n0 + (threadIdx.x & 3) * 8);
  float f[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < kWaves; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] += reinterpret_cast<float*>(lds)[(i * 32 + m) * kRow + (threadIdx.x & 3) * 8 + e];
  col.finish(a, m, f);
}

enum { kFew, kMiddle, kLarge };
struct Plan {
  int kind, splits, per;
  size_t bytes;
};

Plan plan_for(int M, int N, int K) {
  Plan p{M <= 32 ? kFew : kMiddle, 1, 0, 0};
  const int stages = (K + 63) / 64;
  p.per = stages;
  if (p.kind == kFew) return p;
  const int64_t big = static_cast<int64_t>((M + 255) / 256) * ((N + 255) / 256);
  if (big >= 192) {
    p.kind = kLarge;
    return p;
  }
  const int64_t tiles = static_cast<int64_t>((M + 127) / 128) * ((N + 127) / 128);
  if (tiles < 256 && stages >= 16) {
    int64_t s = 512 / tiles;
    if (s > stages / 8) s = stages / 8;
    if (s > 16) s = 16;
    if (s > 1) {
      p.per = static_cast<int>((stages + s - 1) / s);
      p.splits = (stages + p.per - 1) / p.per;
      p.bytes = static_cast<size_t>(p.splits) * M * N * 4;
    }
  }
  return p;
}

template <typename E, int B, int WN, int WM, bool DMA>
void tiles(const LinArgs& a, hipStream_t stream) {
  const dim3 grid(static_cast<unsigned>((a.M + B - 1) / B) * static_cast<unsigned>((a.N + B - 1) / B), a.splits);
  k_linear16<E, B, B, WN, WM, DMA><<<grid, WN * WM * 64, 0, stream>>>(a);
}

template <typename E>
int launch(LinArgs a, Plan p, hipStream_t stream) {
  const bool aligned = a.K % 8 == 0 && a.ldx % 8 == 0 && a.ldw % 8 == 0 &&
                       ((reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.w)) & 15) == 0;
  a.splits = p.splits;
  a.stages_per_split = p.per;
  if (p.kind == kFew && aligned) {
    const unsigned blocks = (a.N + 31) / 32;
    if (a.M <= 4)
      k_linear16_few<E, 1><<<blocks, 256, 0, stream>>>(a);
    else if (a.M <= 8)
      k_linear16_few<E, 2><<<blocks, 256, 0, stream>>>(a);
    else if (a.M <= 16)
      k_linear16_few<E, 4><<<blocks, 256, 0, stream>>>(a);
    else
      k_linear16_few<E, 8><<<blocks, 256, 0, stream>>>(a);
  } else if (!aligned) {
    tiles<E, 128, 2, 2, false>(a, stream);
  } else if (p.kind == kLarge) {
    tiles<E, 256, 2, 4, true>(a, stream);
  } else {
    tiles<E, 128, 2, 2, true>(a, stream);
  }
  if (a.splits > 1) {
    const int64_t n = static_cast<int64_t>((a.N + 7) / 8) * a.M;
    k_linear16_join<E><<<dim3(static_cast<unsigned>((n + 255) / 256)), 256, 0, stream>>>(a);
  }
  return static_cast<int>(hipGetLastError());
}

}  // namespace

extern "C" {

size_t svdq_linear16_plan_bytes(int M, int N, int K) { return plan_for(M, N, K).bytes; }

int svdq_launch_linear16(const void* x, int64_t ldx, const void* w, int64_t ldw, const void* bias, const void* gate,
                         int64_t ld_gate, int group_rows, const void* residual, int64_t ldr, void* y, int64_t ldy, int M,
                         int N, int K, int activation, int dtype, void* workspace, size_t workspace_bytes, void* stream) {
  Plan p = plan_for(M, N, K);
  if (p.splits > 1 && (!workspace || workspace_bytes < p.bytes)) {
    p.splits = 1;
    p.per = (K + 63) / 64;
  }
  LinArgs a{};
  a.x = static_cast<const uint16_t*>(x);
  a.w = static_cast<const uint16_t*>(w);
  a.bias = static_cast<const uint16_t*>(bias);
  a.gate = static_cast<const uint16_t*>(gate);
  a.residual = static_cast<const uint16_t*>(residual);
  a.y = static_cast<uint16_t*>(y);
  a.part = static_cast<float*>(workspace);
  a.ldx = ldx;
  a.ldw = ldw;
  a.ld_gate = ld_gate;
  a.ldr = ldr;
  a.ldy = ldy;
  a.M = M;
  a.N = N;
  a.K = K;
  a.group_rows = group_rows;
  a.act = activation;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  return dtype == SVDQ_BF16 ? launch<Bf16>(a, p, s) : launch<F16>(a, p, s);
}

}  // extern "C"
