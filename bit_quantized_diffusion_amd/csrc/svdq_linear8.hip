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
//
// Measured, rows x k x channels: 8 x 4096 x 6144 7.2 us (25 MB of W, 3.5 TB/s), 333 x 4096 x 1536
// 10.2, 4608 x 4096 x 12288 with GELU 229 (2.0 PFLOP/s), 4608 x 12288 x 4096
// 212 (2.2 PFLOP/s).  Bound by the power limit, and by the scales' FMAs beside
// the products: without them the large tiles take 17 % less.  Between few rows
// and large grids it stays 1.5 to 3 times its floor (bytes at 4.9 TB/s,
// products at 2.71 PFLOP/s): k 4096 to 4096 channels 8.0 us for 64 rows, 8.4 for
// 128, 11.2 for 256, 18.8 for 512, 22.6 for 1024, 37.5 for 2048.

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
// Large tiles: 256 channels x BM = 32 TM rows, 4 x 2 waves of 64 x BM / 2 each.
// K runs in stages of 128: whole 128-byte lines of the rows of wq and xq, that
// loads put straight into LDS, both in rings of two slots, and beside them the
// rows' scales.  A wave holds its four tiles of W and goes through its TM tiles
// of x: while one is multiplied, the next is read from LDS, and the results of
// two products before are added to the sums.  The one barrier of a stage
// stands before its last tile of x: by then the stage has been read out and the
// next one has landed, so that the last tile's products lie beside the reads
// of the next one's W.  The stage after next is loaded right behind the
// barrier, during the products.
// A row of a slot is 128 bytes, two rows share the LDS banks: 16-byte chunk c
// of row r sits at chunk c ^ ((r / 2) % 8).
// ---------------------------------------------------------------------------

template <typename E, int TM>
__global__ __launch_bounds__(512, 2) void k_linear8_wide(Args8 a) {
  constexpr int BN = 256, BM = 32 * TM, WN = 4, WM = 2, TN = 4, kWaves = 8, kRowB = 128;
  // a wave's loads of a stage, 1 KB (8 rows) each; the last waves' of x may lie past the tile
  constexpr int kLw = BN / 8 / kWaves, kLx = (BM / 8 + kWaves - 1) / kWaves, kL = kLw + kLx + 1;
  constexpr int kSlotW = BN * kRowB, kSlotX = kLx * kWaves * 1024, kSlotS = kWaves * 256;
  constexpr int kX = 2 * kSlotW, kS = kX + 2 * kSlotX, kP = kS + 2 * kSlotS,
                kLds = kP + kWaves * 256;
  static_assert(BM <= 512 && kL < (TM - 1) * TN && kLds <= 160 * 1024, "a wave loads 64 rows' scales");
  __shared__ __attribute__((aligned(1024))) uint8_t lds[kLds];

  const int lane = threadIdx.x & 63, l16 = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wn = wave % WN, wm = wave / WN;
  int m0, n0;
  tile_of<BN, BM>(a, blockIdx.x, m0, n0);
  const int stages = (a.K + 127) / 128;

  const uint32_t base = lds_addr(lds);
  const __amdgpu_buffer_rsrc_t bw = buffer_of(a.wq + static_cast<int64_t>(n0) * a.K, static_cast<int64_t>(a.N - n0) * a.K);
  const __amdgpu_buffer_rsrc_t bx = buffer_of(a.xq + static_cast<int64_t>(m0) * a.K, static_cast<int64_t>(a.M - m0) * a.K);
  // load n of a wave: rows 8 p .. 8 p + 7 of a slot, p = wave kL + n; the
  // lane's chunk is (lane % 8) ^ (4 p + lane / 16) % 8
  auto chunk = [&](int p) { return (lane & 7) ^ (((p & 1) << 2) + (lane >> 4)); };
  int vw[kLw], vx[kLx];
#pragma unroll
  for (int n = 0; n < kLw; ++n) {
    const int p = wave * kLw + n;
    vw[n] = (p * 8 + (lane >> 3)) * a.K + (chunk(p) << 4);
  }
#pragma unroll
  for (int n = 0; n < kLx; ++n) {
    const int p = wave * kLx + n, r = p * 8 + (lane >> 3);
    vx[n] = r < BM ? r * a.K + (chunk(p) << 4) : kOutside;
  }
  // scales: wave wn of each half of the rows brings in 64 of them
  const int first = m0 + wm * TM * 16 + wn * 64;
  const bool rows_left = wn * 64 < TM * 16;
  auto load = [&](int st, int slot, int n) {
    if (n < kLw + kLx) {
      const bool is_x = n >= kLw;
      const int i = is_x ? n - kLw : n, p = wave * (is_x ? kLx : kLw) + i;
      const bool outside = st * 128 + (chunk(p) << 4) >= a.K;   // past K rows run on into the next
      if (is_x)
        dma_b128(bx, base + kX + slot * kSlotX + p * 1024, outside ? kOutside : vx[i], st * 128);
      else
        dma_b128(bw, base + slot * kSlotW + p * 1024, outside ? kOutside : vw[i], st * 128);
    } else {
      const __amdgpu_buffer_rsrc_t bs =
          buffer_of(a.xs + static_cast<int64_t>(st) * a.M + first, rows_left && st < stages ? (a.M - first) * 4LL : 0);
      dma_b32(bs, base + kS + slot * kSlotS + wave * 256, lane * 4);
    }
  };
  // one word of every line of a stage, of W by the first four waves, of x by
  // the others: brings the lines into L2, so that the loads proper find them
  // there (their way from memory is longer than a stage)
  const int pr = (wave & 3) * 64 + lane, pl = wave < 4 ? pr * a.K : pr < BM ? pr * a.K : kOutside;
  const __amdgpu_buffer_rsrc_t bp = wave < 4 ? bw : bx;
  auto touch = [&](int st) { dma_b32(bp, base + kP + wave * 256, st < stages ? pl + (pl == kOutside ? 0 : st * 128) : kOutside); };
  // the wave's channels lie in one block of 128: its scales of 64 stages, a lane each
  const float* const ws = a.ws + static_cast<int64_t>(min(n0 + wn * TN * 16, a.N - 1) >> 7) * stages;
  float scales = ws[min(lane, stages - 1)];

  // LDS offsets of the lane's operand reads: row, chunks q and 4 + q
  uint32_t rw[2], rx[2];
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    const uint32_t o = base + l16 * kRowB + (((4 * s + q) ^ (l16 >> 1)) << 4);
    rw[s] = o + wn * TN * 16 * kRowB;
    rx[s] = o + wm * TM * 16 * kRowB + kX;
  }
  const uint32_t rs = base + kS + wm * WN * 256 + l16 * 4;
  v4f acc[TN][TM];
#pragma unroll
  for (int i = 0; i < TN; ++i)
#pragma unroll
    for (int j = 0; j < TM; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};

  Codes w[TN], x[3];
  float sx[3];
  auto read_w = [&](int slot, int i) {
    w[i].lo = lds_read16(rw[0] + slot * kSlotW + i * 16 * kRowB);
    w[i].hi = lds_read16(rw[1] + slot * kSlotW + i * 16 * kRowB);
  };
  auto read_x = [&](int slot, int j, int to) {
    x[to].lo = lds_read16(rx[0] + slot * kSlotX + j * 16 * kRowB);
    x[to].hi = lds_read16(rx[1] + slot * kSlotX + j * 16 * kRowB);
    sx[to] = *reinterpret_cast<__attribute__((address_space(3))) const float*>(rs + slot * kSlotS + j * 64);
  };

#pragma unroll
  for (int n = 0; n < kL; ++n) load(0, 0, n);
#pragma unroll
  for (int n = 0; n < TN; ++n) load(1, 1, n);
  touch(2);
  lds_wait_barrier<TN + 1>();
#pragma unroll
  for (int i = 0; i < TN; ++i) read_w(0, i);
  read_x(0, 0, 0);

  // Tile j of x lies in x[j % 2], but the last, when that is where the next
  // stage's first one goes.  The first TN loads of the stage after next come
  // with a stage's last products, the others with the first products of the
  // next; those of stages past the last bring nothing.
  constexpr int kLast = TM & 1 ? 2 : 1;
  for (int st = 0; st < stages; ++st) {
    if ((st & 63) == 0 && st) scales = ws[min(st + lane, stages - 1)];
    const float sw = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(scales), st & 63));
    const int slot = st & 1, next = slot ^ 1;
    v4f p[3];
    float s[2];
    auto add = [&](int t) {
#pragma unroll
      for (int r = 0; r < 4; ++r) acc[t % TN][t / TN][r] += p[t % 3][r] * s[(t / TN) & 1];
    };
#pragma unroll
    for (int t = 0; t < TN * TM; ++t) {
      const int j = t / TN, i = t % TN, b = j == TM - 1 ? kLast : j & 1;
      if (i == 0) {
        s[j & 1] = sx[b] * sw;
        if (j == TM - 1) {
          fence();
          lds_wait_barrier<1>();   // read out; the next stage has landed, the touch may fly
        }
      }
      p[t % 3] = block_sum(w[i], x[b]);
      if (j < TM - 1) {
        if (i == 0) read_x(slot, j + 1, j + 1 == TM - 1 ? kLast : (j + 1) & 1);
        if (t < kL - TN) load(st + 1, next, TN + t);
        if (t == kL - TN) touch(st + 2);
      } else {
        // (past the last stage this reads zeros, which are not used)
        read_w(next, i);
        if (i == 0) read_x(next, 0, 0);
        load(st + 2, slot, i);   // the slot is free
      }
      if (t >= 2) add(t - 2);
      fence();
    }
    add(TN * TM - 2);
    add(TN * TM - 1);
  }
  lds_wait_barrier<0>();
  epilogue<E, BN, BM, WN, WM, TN, TM, staged_tiles(TM, WM * 16 * BN * 4, kLds)>(a, acc, lds, m0, n0);
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
  float scales = ws[min(lane, stages - 1)];

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
    if ((st & 63) == 0 && st) scales = ws[min(st + lane, stages - 1)];
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(scales), st & 63));
  };

#pragma unroll
  for (int i = 0; i < 1 + D; ++i)
    if (i < stages)
      for (int n = 0; n < kL; ++n) load(i, i, n);
  if (D < stages)
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
  int st = 0;
  for (; st + 1 + D < stages; ++st) stage(st, std::true_type{});
  // (past the last stage this reads a slot's old bytes, which are not used)
  for (; st < stages; ++st) stage(st, std::false_type{});
  lds_wait_barrier<0>();
  epilogue<E, BN, BM, WN, WM, TN, TM, staged_tiles(TM, WM * 16 * BN * 4, kRing)>(a, acc, lds, m0, n0);
}

// ---------------------------------------------------------------------------
// Few rows, and grids of few tiles: tiles of 16 NT channels x 16 TM rows that a
// workgroup's waves multiply together.  They take the stages of 128 KB k in
// turn, each through LDS of its own (DEPTH stages in flight, no barrier in the
// loop), and join at the end in their order.  XL: 1 KB loads that bring in the
// rows of x.
// ---------------------------------------------------------------------------

template <typename E, int NT, int XL, int NW, int DEPTH, int KB>
__global__ __launch_bounds__(NW * 64, 1) void k_linear8_few(Args8 a) {
  constexpr int kRowB = 128 * KB, kRows = 1024 / kRowB, kC = kRowB / 16;   // rows of a load, chunks of a row
  constexpr int TM = (XL * kRows + 15) / 16, kXRows = XL * kRows;
  constexpr int LW = NT * 16 / kRows, kW = LW * 1024, kX = XL * 1024, kStage = kW + kX + 256, kL = LW + XL + 1;
  constexpr int kRow = NT * 16 + 4;   // floats of a row of the join, padded
  constexpr int kLoop = NW * DEPTH * kStage, kJoin = NW * TM * 16 * kRow * 4;
  static_assert(TM * 16 * KB <= 64 && (kXRows >= 16 ? kXRows % 16 == 0 : 16 % kXRows == 0), "a stage's scales are one load");
  __shared__ __attribute__((aligned(1024))) uint8_t lds[kLoop > kJoin ? kLoop : kJoin];
  const int lane = threadIdx.x & 63, l16 = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int m0, n0;
  tile_of<NT * 16, TM * 16>(a, blockIdx.x, m0, n0);
  const int blocks = (a.K + 127) / 128, stages = (blocks + KB - 1) / KB;
  // chunk c of row r sits where rows share no LDS banks
  auto place = [](int r, int c) { return KB == 2 ? c ^ (r & 15) : c ^ ((r >> 1) & 7); };
  const int r0 = lane / kC;           // the lane's row of a load, counted from its first
  int vw[LW], vx[XL];
#pragma unroll
  for (int n = 0; n < LW; ++n) vw[n] = (n * kRows + r0) * a.K + (place(n * kRows + r0, lane % kC) << 4);
#pragma unroll
  for (int n = 0; n < XL; ++n) vx[n] = (n * kRows + r0) * a.K + (place(n * kRows + r0, lane % kC) << 4);
  const uint32_t base = lds_addr(lds) + wave * DEPTH * kStage;
  const __amdgpu_buffer_rsrc_t bw = buffer_of(a.wq + static_cast<int64_t>(n0) * a.K, static_cast<int64_t>(a.N - n0) * a.K);
  const __amdgpu_buffer_rsrc_t bx = buffer_of(a.xq + static_cast<int64_t>(m0) * a.K, static_cast<int64_t>(a.M - m0) * a.K);
  constexpr int kScaled = 64 / KB;    // rows whose scales a load brings in
  const int vs = lane % kScaled < a.M - m0 ? (lane / kScaled * a.M + lane % kScaled) * 4 : kOutside;
  auto issue = [&](int st, int slot) {
    const int k0 = st * kRowB;
    const uint32_t d = base + slot * kStage;
    auto outside = [&](int n) { return k0 + (place(n * kRows + r0, lane % kC) << 4) >= a.K; };   // past K
#pragma unroll
    for (int n = 0; n < LW; ++n) dma_b128(bw, d + n * 1024, outside(n) ? kOutside : vw[n], k0);
#pragma unroll
    for (int n = 0; n < XL; ++n) dma_b128(bx, d + kW + n * 1024, outside(n) ? kOutside : vx[n], k0);
    const int64_t at = static_cast<int64_t>(st) * KB * a.M + m0;
    dma_b32(buffer_of(a.xs + at, (static_cast<int64_t>(blocks) * a.M - at) * 4), d + kW + kX, vs);
  };
  // chunks q and 4 + q of a block's eight, of row l16 of a tile; rows of x past
  // the staged ones repeat them (their results are not stored)
  const int x16 = kXRows < 16 ? l16 % kXRows : l16;
  uint32_t rw[2 * KB], rx[2 * KB];
#pragma unroll
  for (int c = 0; c < 2 * KB; ++c) {
    rw[c] = l16 * kRowB + (place(l16, 4 * c + q) << 4);
    rx[c] = kW + x16 * kRowB + (place(x16, 4 * c + q) << 4);
  }
  const float* const ws = a.ws + static_cast<int64_t>(n0 >> 7) * blocks;
  float scales = ws[min((KB * wave & ~63) + lane, blocks - 1)];   // of 64 blocks, a lane each

  v4f acc[NT][TM];
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int j = 0; j < TM; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < DEPTH; ++i)
    if (wave + i * NW < stages) issue(wave + i * NW, i);
  int slot = 0;
#pragma unroll 1
  for (int st = wave; st < stages; st += NW) {
    const int more = (stages - 1 - st) / NW;   // stages of this wave still in flight
    if (more >= DEPTH - 1)
      vm_wait<(DEPTH - 1) * kL>();
    else
      vm_wait<0>();
    const uint32_t d = base + slot * kStage;
    if (st >= NW && (KB * st & ~63) != (KB * (st - NW) & ~63)) scales = ws[min((KB * st & ~63) + lane, blocks - 1)];
#pragma unroll
    for (int b = 0; b < KB; ++b) {
      const float sw = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(scales), (KB * st + b) & 63));
      Codes w[NT];
#pragma unroll
      for (int i = 0; i < NT; ++i)
        w[i] = {lds_read16(d + i * 16 * kRowB + rw[2 * b]), lds_read16(d + i * 16 * kRowB + rw[2 * b + 1])};
#pragma unroll
      for (int j = 0; j < TM; ++j) {
        const Codes x = {lds_read16(d + j * 16 * kRowB + rx[2 * b]), lds_read16(d + j * 16 * kRowB + rx[2 * b + 1])};
        const float s = sw * *reinterpret_cast<__attribute__((address_space(3))) const float*>(
                                 d + kW + kX + (b * kScaled + j * 16 + l16) * 4);
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          const v4f p = block_sum(w[i], x);
#pragma unroll
          for (int r = 0; r < 4; ++r) acc[i][j][r] += p[r] * s;
        }
      }
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // the slot is read out before it is loaded again
    if (st + DEPTH * NW < stages) issue(st + DEPTH * NW, slot);
    slot = slot + 1 == DEPTH ? 0 : slot + 1;
  }
  __syncthreads();
  float* const out = reinterpret_cast<float*>(lds);
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int j = 0; j < TM; ++j)
      *reinterpret_cast<v4f*>(out + ((wave * TM + j) * 16 + l16) * kRow + i * 16 + 4 * q) = acc[i][j];
  __syncthreads();
  // a thread takes 8 channels of a row
  for (int t = threadIdx.x; t < TM * 16 * NT * 2; t += NW * 64) {
    const int m = t / (NT * 2), c = t % (NT * 2) * 8;
    if (m0 + m >= a.M) break;
    Columns<E> col;
    col.init(a, n0 + c);
    float f[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < NW; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] += out[(i * TM * 16 + m) * kRow + c + e];
    col.finish(a, m0 + m, f);
  }
}

// Schedules.  `slots`: workgroups the device holds at once; `light` and
// `full`: microseconds of a stage of 128 k with one workgroup a CU or fewer
// and with every slot taken; `edge`: first loads, join and epilogue of a tile.
// Measured on random codes with K from 1024 to 12288.
struct Shape {
  int bn, bm, waves, slots;
  float light, full, edge;
};
enum { kFew16, kFew32, kFew64, k128Deep, k128, k256, kWide160, kWide192, kWide224, kWide288, kShapes };
constexpr Shape kShape[kShapes] = {
    {16, 64, 8, 256, 0.110f, 0.118f, 0.5f},    // k_linear8_few
    {32, 64, 8, 256, 0.145f, 0.150f, 0.5f},
    {64, 64, 8, 256, 0.185f, 0.200f, 1.0f},
    {128, 128, 8, 256, 0.52f, 0.58f, 2.5f},    // loads two stages further ahead
    {128, 128, 4, 512, 0.93f, 1.05f, 3.0f},    // two workgroups a CU
    {256, 256, 8, 256, 1.39f, 1.61f, 8.0f},
    {256, 160, 8, 256, 1.30f, 1.33f, 4.5f},    // k_linear8_wide
    {256, 192, 8, 256, 1.35f, 1.42f, 4.5f},
    {256, 224, 8, 256, 1.50f, 1.66f, 4.5f},
    {256, 288, 8, 256, 1.75f, 2.07f, 4.5f},
};
constexpr int kFewRows = 32;   // up to these the tiles' height goes by the rows

// The cheapest shape.  Past one round of workgroups the cost lies nearer to
// the rounded-up than to the true number of rounds: idle CUs of the last one
// leave the others a higher clock.  The many heights of large tiles are there
// for that last round: 4608 x 12288 x 4096 takes 16 x 16 tiles of 288 x 256,
// one round of 205 us, where 18 x 16 of 256 x 256 take two, 295.
int shape_for(int M, int N, int K) {
  const int stages = (K + 127) / 128;
  int best = 0;
  float least = INFINITY;
  for (int i = 0; i < kShapes; ++i) {
    const Shape& c = kShape[i];
    const float groups = static_cast<float>((M + c.bm - 1) / c.bm) * ((N + c.bn - 1) / c.bn), load = groups / c.slots;
    const float taken = c.slots > 256 ? (groups - 256.f) / (c.slots - 256) : groups / 256.f;
    const float stage = c.light + (c.full - c.light) * fminf(fmaxf(taken, 0.f), 1.f);
    const float us = (load <= 1.f ? 1.f : 0.25f * load + 0.75f * ceilf(load)) * (stages * stage + c.edge);
    if (us < least) {
      least = us;
      best = i;
    }
  }
  return best;
}

// Few rows: two waves take 32 channels where there are more tiles of 16 than
// two a CU (16 x 4096 x 18432 21 -> 13.7 us, 16 x 4096 x 6144 7.0 -> 8.4),
// eight waves 16 otherwise (16 x 12288 x 4096 with four 12.0, with eight 10.6).
// From 17 rows on eight waves, 32 channels from more than one tile of 16 a CU.
bool many_channels(int N) { return (N + 15) / 16 > 512; }
bool more_channels(int N) { return (N + 15) / 16 > 256; }

template <typename E, int BN, int BM, int WN, int WM, int D>
void start(const Args8& a, hipStream_t stream) {
  const unsigned tiles = static_cast<unsigned>((a.M + BM - 1) / BM) * static_cast<unsigned>((a.N + BN - 1) / BN);
  k_linear8<E, BN, BM, WN, WM, D><<<tiles, WN * WM * 64, 0, stream>>>(a);
}

template <typename E, int NT, int XL, int NW, int DEPTH, int KB>
void start_few(const Args8& a, hipStream_t stream) {
  constexpr int kTileM = (XL * (8 / KB) + 15) / 16 * 16;
  const unsigned tiles = static_cast<unsigned>((a.M + kTileM - 1) / kTileM) * static_cast<unsigned>((a.N + 16 * NT - 1) / (16 * NT));
  k_linear8_few<E, NT, XL, NW, DEPTH, KB><<<tiles, NW * 64, 0, stream>>>(a);
}
template <typename E, int XL>
void start_few(const Args8& a, hipStream_t stream) {
  if constexpr (XL == 8) {
    if (more_channels(a.N))
      start_few<E, 2, XL, 8, 1, 2>(a, stream);
    else
      start_few<E, 1, XL, 8, 1, 2>(a, stream);
  } else {
    if (many_channels(a.N))
      start_few<E, 2, XL, 2, 2, 2>(a, stream);
    else
      start_few<E, 1, XL, 8, 1, 2>(a, stream);
  }
}

template <typename E, int TM>
void start_wide(const Args8& a, hipStream_t stream) {
  const unsigned tiles = static_cast<unsigned>((a.M + 32 * TM - 1) / (32 * TM)) * static_cast<unsigned>((a.N + 255) / 256);
  k_linear8_wide<E, TM><<<tiles, 512, 0, stream>>>(a);
}

template <typename E>
int launch(const Args8& a, hipStream_t stream) {
  if (a.M <= 4) {
    start_few<E, 1>(a, stream);
  } else if (a.M <= 8) {
    start_few<E, 2>(a, stream);
  } else if (a.M <= 16) {
    start_few<E, 4>(a, stream);
  } else if (a.M <= kFewRows) {
    start_few<E, 8>(a, stream);
  } else {
    switch (shape_for(a.M, a.N, a.K)) {
      case kFew16: start_few<E, 1, 8, 8, 1, 1>(a, stream); break;
      case kFew32: start_few<E, 2, 8, 8, 1, 1>(a, stream); break;
      case kFew64: start_few<E, 4, 8, 8, 1, 1>(a, stream); break;
      case k128Deep: start<E, 128, 128, 2, 4, 2>(a, stream); break;
      case k128: start<E, 128, 128, 2, 2, 0>(a, stream); break;
      case k256: start<E, 256, 256, 2, 4, 0>(a, stream); break;
      case kWide160: start_wide<E, 5>(a, stream); break;
      case kWide192: start_wide<E, 6>(a, stream); break;
      case kWide224: start_wide<E, 7>(a, stream); break;
      default: start_wide<E, 9>(a, stream);
    }
  }
  return static_cast<int>(hipGetLastError());
}

}  // namespace

extern "C" {

void svdq_gemm_fp8_plan(int M, int N, int K, int32_t* plan) {
  if (M <= kFewRows) {
    const bool two = M <= 16 ? many_channels(N) : more_channels(N);
    plan[0] = M <= 16 ? 16 : 32;
    plan[1] = two ? 32 : 16;
    plan[2] = M <= 16 && two ? 2 : 8;
    return;
  }
  const Shape& c = kShape[shape_for(M, N, K)];
  plan[0] = c.bm;
  plan[1] = c.bn;
  plan[2] = c.waves;
}

int svdq_launch_gemm_fp8(const uint8_t* xq, const float* xs, const uint8_t* wq, const float* ws, const void* bias,
                         const void* gate, int64_t ld_gate, int group_rows, const void* residual, int64_t ldr, void* y,
                         int64_t ldy, int M, int N, int K, int activation, int dtype, void* stream) {
  Args8 a{};
  a.xq = xq;
  a.wq = wq;
  a.xs = xs;
  a.ws = ws;
  a.bias = static_cast<const uint16_t*>(bias);
  a.gate = static_cast<const uint16_t*>(gate);
  a.residual = static_cast<const uint16_t*>(residual);
  a.y = static_cast<uint16_t*>(y);
  a.ld_gate = ld_gate;
  a.ldr = ldr;
  a.ldy = ldy;
  a.M = M;
  a.N = N;
  a.K = K;
  a.group_rows = group_rows;
  a.act = activation;
  a.splits = 1;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  return dtype == SVDQ_BF16 ? launch<Bf16>(a, s) : launch<F16>(a, s);
}

}  // extern "C"
