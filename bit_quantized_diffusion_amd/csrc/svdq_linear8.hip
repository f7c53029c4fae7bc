// 8-bit linear with a scale for each block of 128 and the 16-bit linear's
// epilogue:
//
//   z[m][n] = sum over blocks g of 128 k: sx[g][m] sw[n / 128][g] sum_k xq[m][k] wq[n][k]
//   y = residual + gate_r * act(z + b),  r = row / group_rows
//
// for gfx950.  xq [M][K] and wq [N][K] are e4m3 codes, sx and sw fp32.  One
// 16 x 16 x 128 product of the matrix core is one block's sum, from zero; its
// four results a lane are then added to the fp32 sums times the block's two
// scales, which the vector ALU does beside the next products.  A is W and B is
// x, so that a lane's results lie along n, the dense dimension of y, and its
// scale of x is that of one row.
//
// Precision: the matrix core takes the products of 8 consecutive k to the
// largest one's exponent E and cuts what lies below 2^(E - 13); groups of 8
// are added in fp32.  For random codes that is about 1e-4 of the result, a
// sixteenth of a rounding to bf16 and half of one to fp16.  Codes widened to
// bf16 would be summed exactly, at half the rate.

#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include <type_traits>

#include "svdq_device.h"
#include "svdq_internal.h"
#include "svdq_linear_tile.h"

namespace {

using namespace svdq_dev;

struct Args8 : OutArgs {
  const uint8_t *xq, *wq;
  const float *xs, *ws;   // [blocks][M], [row blocks][blocks]
};

// 16 rows x 128 k of codes: 32 bytes a lane.  Both operands take the k of a
// lane from the same places, so their order within the product is free.
struct Codes {
  v4u lo, hi;
};
__device__ __forceinline__ v4f block_sum(const Codes& a, const Codes& b) {
  const v8i x = {(int)a.lo[0], (int)a.lo[1], (int)a.lo[2], (int)a.lo[3], (int)a.hi[0], (int)a.hi[1], (int)a.hi[2], (int)a.hi[3]};
  const v8i y = {(int)b.lo[0], (int)b.lo[1], (int)b.lo[2], (int)b.lo[3], (int)b.hi[0], (int)b.hi[1], (int)b.hi[2], (int)b.hi[3]};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, y, v4f{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0, 0, 0);
}

// ---------------------------------------------------------------------------
// Tiles of BN channels x BM rows, WN x WM waves.  K runs in stages of 128:
// whole 128-byte lines of the rows of wq and xq, that loads put straight into
// LDS, both in rings of 2 + D slots, and beside them each wave's scales of its
// rows of x.  A wave goes through its TN x TM results of 16 x 16 by rows of W:
// while row i is multiplied, W of row i + 1 is read from LDS.  The one barrier
// of a stage stands before its last row: by then the stage has been read out
// and the next one has landed, so that the last row reads that one's x and
// first W.  The stage 1 + D ahead is loaded during the rows before it.
// A row of a slot is 128 bytes, two rows share the LDS banks: 16-byte chunk c
// of row r sits at chunk c ^ ((r / 2) % 8).
// ---------------------------------------------------------------------------

template <typename E, int BN, int BM, int WN, int WM, int D>
__global__ __launch_bounds__(WN * WM * 64, 2) void k_linear8(Args8 a) {
  constexpr int kWaves = WN * WM;
  constexpr int TN = BN / WN / 16, TM = BM / WM / 16;   // 16 x 16 results of a wave
  constexpr int kRowB = 128;
  constexpr int kLw = BN / 8 / kWaves, kLx = BM / 8 / kWaves, kL = kLw + kLx + 1;   // a wave's loads of a stage
  constexpr int kSlots = 2 + D, kSlotW = BN * kRowB, kSlotX = BM * kRowB;
  constexpr int kX = kSlots * kSlotW, kS = kX + kSlots * kSlotX;
  constexpr int kRing = kS + kSlots * kWaves * 256;   // a wave's scales: 64 rows, its TM * 16 first
  static_assert(BN % (16 * WN) == 0 && BM % (16 * WM) == 0 && BN % (8 * kWaves) == 0 && BM % (8 * kWaves) == 0, "even");
  static_assert(TN % 2 == 0 && TM <= 4 && 128 % (TN * 16) == 0 && kL <= (TN - 1) * TM * 3, "rows of W in turn, scales in one load");
  __shared__ __attribute__((aligned(1024))) uint8_t lds[kRing];

  const int lane = threadIdx.x & 63, l16 = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wn = wave % WN, wm = wave / WN;
  int m0, n0;
  tile_of<BN, BM>(a, blockIdx.x, m0, n0);
  const int stages = (a.K + 127) / 128;
  const int s0 = blockIdx.y * a.stages_per_split, s1 = min(s0 + a.stages_per_split, stages);

  const uint32_t base = lds_addr(lds);
  const __amdgpu_buffer_rsrc_t bw = buffer_of(a.wq + static_cast<int64_t>(n0) * a.K, static_cast<int64_t>(a.N - n0) * a.K);
  const __amdgpu_buffer_rsrc_t bx = buffer_of(a.xq + static_cast<int64_t>(m0) * a.K, static_cast<int64_t>(a.M - m0) * a.K);
  // load n of a wave: rows 8 p .. 8 p + 7 of a slot, p = wave kL + n; the
  // lane's chunk is (lane % 8) ^ (4 p + lane / 16) % 8
  auto chunk = [&](int p) { return (lane & 7) ^ (((p & 1) << 2) + (lane >> 4)); };
  const int first = wm * TM * 16 + m0;   // the wave's first row of x
  auto load = [&](int st, int slot, int n) {
    if (n < kLw) {
      const int p = wave * kLw + n, c = chunk(p) * 16;
      const int at = (p * 8 + (lane >> 3)) * a.K + st * 128 + c;
      dma_b128(bw, base + slot * kSlotW + p * 1024, st * 128 + c >= a.K ? kOutside : at);   // past K rows run on into the next
    } else if (n < kLw + kLx) {
      const int p = wave * kLx + n - kLw, c = chunk(p) * 16;
      const int at = (p * 8 + (lane >> 3)) * a.K + st * 128 + c;
      dma_b128(bx, base + kX + slot * kSlotX + p * 1024, st * 128 + c >= a.K ? kOutside : at);
    } else {
      const __amdgpu_buffer_rsrc_t bs = buffer_of(a.xs + static_cast<int64_t>(st) * a.M + first, (a.M - first) * 4LL);
      dma_b32(bs, base + kS + (slot * kWaves + wave) * 256, lane * 4);
    }
  };
  // the wave's channels lie in one block of 128: its scales of 64 stages, a lane each
  const float* const ws = a.ws + static_cast<int64_t>(min(n0 + wn * TN * 16, a.N - 1) >> 7) * stages;
  float scales = ws[min(s0 + lane, stages - 1)];

  // LDS offsets of the lane's operand reads: row, chunks q and 4 + q
  uint32_t rw[2], rx[2];
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    const uint32_t o = base + l16 * kRowB + (((4 * s + q) ^ (l16 >> 1)) << 4);
    rw[s] = o + wn * TN * 16 * kRowB;
    rx[s] = o + wm * TM * 16 * kRowB + kX;
  }
  v4f acc[TN][TM];
#pragma unroll
  for (int i = 0; i < TN; ++i)
#pragma unroll
    for (int j = 0; j < TM; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};

  Codes w[2], x[TM];
  float sx[TM], s[TM];
  auto read_w = [&](int slot, int i) {
    w[i & 1].lo = lds_read16(rw[0] + slot * kSlotW + i * 16 * kRowB);
    w[i & 1].hi = lds_read16(rw[1] + slot * kSlotW + i * 16 * kRowB);
  };
  auto read_x = [&](int slot, int j) {
    x[j].lo = lds_read16(rx[0] + slot * kSlotX + j * 16 * kRowB);
    x[j].hi = lds_read16(rx[1] + slot * kSlotX + j * 16 * kRowB);
  };
  auto read_s = [&](int slot, int j) {
    sx[j] = *reinterpret_cast<__attribute__((address_space(3))) const float*>(base + kS + (slot * kWaves + wave) * 256 +
                                                                              (j * 16 + l16) * 4);
  };
  auto scale_at = [&](int st) {
    const int i = st - s0;
    if ((i & 63) == 0 && i) scales = ws[min(st + lane, stages - 1)];
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(scales), i & 63));
  };

#pragma unroll
  for (int i = 0; i < 1 + D; ++i)
    if (s0 + i < s1)
      for (int n = 0; n < kL; ++n) load(s0 + i, i, n);
  if (s0 + D < s1)
    lds_wait_barrier<D * kL>();
  else
    lds_wait_barrier<0>();
#pragma unroll
  for (int j = 0; j < TM; ++j) {
    read_x(0, j);
    read_s(0, j);
  }
  read_w(0, 0);

  int slot = 0, ahead = 1 + D;   // slots of this stage and of the one to load
  auto stage = [&](int st, auto more) {
    constexpr bool kMore = decltype(more)::value;
    const float sw = scale_at(st);
#pragma unroll
    for (int j = 0; j < TM; ++j) s[j] = sx[j] * sw;
    const int next = slot + 1 == kSlots ? 0 : slot + 1;
    v4f p[3];
    auto add = [&](int t) {
#pragma unroll
      for (int r = 0; r < 4; ++r) acc[t / TM][t % TM][r] += p[t % 3][r] * s[t % TM];
    };
    int n = 0;
#pragma unroll
    for (int t = 0; t < TN * TM; ++t) {
      const int i = t / TM, j = t % TM;
      if (i == TN - 1 && j == 0) {
        fence();
        // read out; the next stage has landed, those after it may fly
        lds_wait_barrier<kMore ? D * kL : 0>();
      }
      p[t % 3] = block_sum(w[i & 1], x[j]);
      if (i < TN - 1) {
        if (j == 0) read_w(slot, i + 1);
        if constexpr (kMore)
          for (int e = 0; e < (kL + (TN - 1) * TM - 1) / ((TN - 1) * TM); ++e)
            if (n < kL) load(st + 1 + D, ahead, n++);
      } else {
        if (j == 0) read_w(next, 0);
        read_x(next, j);
        read_s(next, j);
      }
      if (t >= 2) add(t - 2);
      fence();
    }
    add(TN * TM - 2);
    add(TN * TM - 1);
    slot = next;
    ahead = ahead + 1 == kSlots ? 0 : ahead + 1;
  };
  int st = s0;
  for (; st + 1 + D < s1; ++st) stage(st, std::true_type{});
  // (past the last stage this reads a slot's old bytes, which are not used)
  for (; st < s1; ++st) stage(st, std::false_type{});
  lds_wait_barrier<0>();
  epilogue<E, BN, BM, WN, WM, TN, TM, staged_tiles(TM, WM * 16 * BN * 4, kRing)>(a, acc, lds, m0, n0);
}

// ---------------------------------------------------------------------------
// Few rows (M <= 16 TM): bound by reading W once.  A workgroup takes 16 NT
// channels; its waves take the stages of 128 k in turn, straight from memory
// into registers with DEPTH stages in flight, and join at the end.
// ---------------------------------------------------------------------------

template <typename E, int TM, int NT, int NW, int DEPTH>
__global__ __launch_bounds__(NW * 64, 1) void k_linear8_few(Args8 a) {
  constexpr int kRow = NT * 16 + 4;   // floats of a row of the join, padded
  __shared__ __attribute__((aligned(16))) float out[NW * TM * 16 * kRow];
  const int lane = threadIdx.x & 63, l16 = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n0 = blockIdx.x * NT * 16;
  const int stages = (a.K + 127) / 128;
  const float* const ws = a.ws + static_cast<int64_t>(n0 >> 7) * stages;
  struct Stage {
    Codes w[NT], x[TM];
    float sx[TM], sw;
  };
  // rows past the last repeat it (their results are not stored)
  const uint8_t *pw[NT], *px[TM];
#pragma unroll
  for (int i = 0; i < NT; ++i) pw[i] = a.wq + static_cast<int64_t>(min(n0 + i * 16 + l16, a.N - 1)) * a.K + 16 * q;
#pragma unroll
  for (int j = 0; j < TM; ++j) px[j] = a.xq + static_cast<int64_t>(min(j * 16 + l16, a.M - 1)) * a.K + 16 * q;
  auto get = [&](const uint8_t* p, int k) {   // past K zeros
    return k + 16 * q < a.K ? *reinterpret_cast<const v4u*>(p + k) : v4u{0, 0, 0, 0};
  };
  auto fetch = [&](int st, Stage& g) {
    const int k = st * 128;
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      g.w[i].lo = get(pw[i], k);
      g.w[i].hi = get(pw[i], k + 64);
    }
#pragma unroll
    for (int j = 0; j < TM; ++j) {
      g.x[j].lo = get(px[j], k);
      g.x[j].hi = get(px[j], k + 64);
      g.sx[j] = a.xs[static_cast<int64_t>(st) * a.M + min(j * 16 + l16, a.M - 1)];
    }
    g.sw = ws[st];
  };
  v4f acc[NT][TM];
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int j = 0; j < TM; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};
  Stage held[DEPTH];
#pragma unroll
  for (int d = 0; d < DEPTH; ++d)
    if (wave + d * NW < stages) fetch(wave + d * NW, held[d]);
  for (int st = wave; st < stages; st += DEPTH * NW) {
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) {
      if (st + d * NW >= stages) break;
      Stage& g = held[d];
#pragma unroll
      for (int j = 0; j < TM; ++j) {
        const float s = g.sx[j] * g.sw;
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          const v4f p = block_sum(g.w[i], g.x[j]);
#pragma unroll
          for (int r = 0; r < 4; ++r) acc[i][j][r] += p[r] * s;
        }
      }
      if (st + (d + DEPTH) * NW < stages) fetch(st + (d + DEPTH) * NW, g);
    }
  }
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int j = 0; j < TM; ++j)
      *reinterpret_cast<v4f*>(out + ((wave * TM + j) * 16 + l16) * kRow + i * 16 + 4 * q) = acc[i][j];
  __syncthreads();
  // a thread takes 8 channels of a row
  for (int t = threadIdx.x; t < TM * 16 * NT * 2; t += NW * 64) {
    const int m = t / (NT * 2), c = t % (NT * 2) * 8;
    if (m >= a.M) break;
    Columns<E> col;
    col.init(a, n0 + c);
    float f[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < NW; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] += out[(i * TM * 16 + m) * kRow + c + e];
    col.finish(a, m, f);
  }
}

// Schedules.  `slots`: workgroups the device holds at once; `light` and
// `full`: microseconds of a stage of 128 k with one workgroup a CU or fewer
// and with every slot taken; `fixed`: launch, first loads and epilogue.
struct Shape {
  int bn, bm, waves, slots;
  float light, full, fixed;
};
enum { k256, k128, k64, kShapes };
constexpr Shape kShape[kShapes] = {
    {256, 256, 8, 256, 1.10f, 1.45f, 8.f},
    {128, 128, 4, 512, 0.50f, 0.83f, 5.f},
    {64, 64, 4, 512, 0.20f, 0.33f, 4.f},
};
constexpr int kMaxSplits = 8;

struct Plan {
  int shape, splits, per;
  size_t bytes;
};

// The cheapest shape and number of splits: rounds of workgroups times a
// tile's stages, and for splits the join's launch and its traffic.
Plan plan_for(int M, int N, int K, int most_splits) {
  const int stages = (K + 127) / 128;
  Plan best{k64, 1, stages, 0};
  float least = INFINITY;
  for (int i = 0; i < kShapes; ++i) {
    const Shape& c = kShape[i];
    const float tiles = static_cast<float>((M + c.bm - 1) / c.bm) * ((N + c.bn - 1) / c.bn);
    for (int s = 1; s <= most_splits && s <= stages; ++s) {
      const int per = (stages + s - 1) / s;
      if ((stages + per - 1) / per != s) continue;
      const size_t bytes = s == 1 ? 0 : static_cast<size_t>(s) * M * N * 4;
      const float groups = tiles * s, load = groups / c.slots;
      const float stage = c.light + (c.full - c.light) * fminf(fmaxf(groups - 256.f * (c.slots > 256), 0.f) / 256.f, 1.f);
      const float rounds = load <= 1.f ? 1.f : 0.5f * (load + ceilf(load));
      const float us = rounds * per * stage + c.fixed + (s > 1 ? 5.5f + bytes * 2e-6f / 4.f : 0.f);
      if (us < least) {
        least = us;
        best = Plan{i, s, per, bytes};
      }
    }
  }
  return best;
}

constexpr int kFewRows = 32;   // up to these the weights are read once by k_linear8_few

template <typename E, int BN, int BM, int WN, int WM, int D>
void start(const Args8& a, hipStream_t stream) {
  const unsigned tiles = static_cast<unsigned>((a.M + BM - 1) / BM) * static_cast<unsigned>((a.N + BN - 1) / BN);
  k_linear8<E, BN, BM, WN, WM, D><<<dim3(tiles, a.splits), WN * WM * 64, 0, stream>>>(a);
}

template <typename E>
int launch(Args8 a, size_t workspace, hipStream_t stream) {
  a.splits = 1;
  if (a.M <= kFewRows) {
    if (a.M <= 16)
      k_linear8_few<E, 1, 1, 4, 6><<<(a.N + 15) / 16, 256, 0, stream>>>(a);
    else
      k_linear8_few<E, 2, 2, 4, 3><<<(a.N + 31) / 32, 256, 0, stream>>>(a);
    return static_cast<int>(hipGetLastError());
  }
  // the sum's order goes by the sizes: all of the workspace, or one piece
  Plan p = plan_for(a.M, a.N, a.K, kMaxSplits);
  if (workspace < p.bytes) p = plan_for(a.M, a.N, a.K, 1);
  a.splits = p.splits;
  a.stages_per_split = p.per;
  switch (p.shape) {
    case k256: start<E, 256, 256, 2, 4, 0>(a, stream); break;
    case k128: start<E, 128, 128, 2, 2, 0>(a, stream); break;
    default: start<E, 64, 64, 2, 2, 1>(a, stream);
  }
  if (a.splits > 1) {
    const int64_t n = static_cast<int64_t>((a.N + 7) / 8) * a.M;
    k_linear_join<E><<<dim3(static_cast<unsigned>((n + 255) / 256)), 256, 0, stream>>>(a);
  }
  return static_cast<int>(hipGetLastError());
}

}  // namespace

extern "C" {

size_t svdq_gemm_fp8_plan_bytes(int M, int N, int K) { return M <= kFewRows ? 0 : plan_for(M, N, K, kMaxSplits).bytes; }

void svdq_gemm_fp8_plan(int M, int N, int K, int32_t* plan) {
  if (M <= kFewRows) {
    plan[0] = plan[1] = M <= 16 ? 16 : 32;
    plan[2] = 4;
    plan[3] = 1;
    return;
  }
  const Plan p = plan_for(M, N, K, kMaxSplits);
  plan[0] = kShape[p.shape].bm;
  plan[1] = kShape[p.shape].bn;
  plan[2] = kShape[p.shape].waves;
  plan[3] = p.splits;
}

int svdq_launch_gemm_fp8(const uint8_t* xq, const float* xs, const uint8_t* wq, const float* ws, const void* bias,
                         const void* gate, int64_t ld_gate, int group_rows, const void* residual, int64_t ldr, void* y,
                         int64_t ldy, int M, int N, int K, int activation, int dtype, void* workspace,
                         size_t workspace_bytes, void* stream) {
  Args8 a{};
  a.xq = xq;
  a.wq = wq;
  a.xs = xs;
  a.ws = ws;
  a.bias = static_cast<const uint16_t*>(bias);
  a.gate = static_cast<const uint16_t*>(gate);
  a.residual = static_cast<const uint16_t*>(residual);
  a.y = static_cast<uint16_t*>(y);
  a.part = static_cast<float*>(workspace);
  a.ld_gate = ld_gate;
  a.ldr = ldr;
  a.ldy = ldy;
  a.M = M;
  a.N = N;
  a.K = K;
  a.group_rows = group_rows;
  a.act = activation;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const size_t bytes = workspace ? workspace_bytes : 0;
  return dtype == SVDQ_BF16 ? launch<Bf16>(a, bytes, s) : launch<F16>(a, bytes, s);
}

}  // extern "C"
