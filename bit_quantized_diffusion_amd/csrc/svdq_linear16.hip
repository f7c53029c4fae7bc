// 16-bit linear with bias, activation, gate and residual in its epilogue:
//
//   y = residual + gate_g * act(x W^T + b),  g = row / group_rows
//
// for gfx950.  x [M][K], W [N][K] (nn.Linear layout), y [M][N]; products in
// the matrix core with fp32 accumulation, the epilogue in fp32, one rounding.
//
// The matrix core's A operand is W and its B operand is x, so that a lane's
// results lie along n, the dense dimension of y.
//
// Measured (passes over changing inputs, bf16): 4608 x 3072 -> 12288 with GELU
// 300 us (1160 TFLOP/s), 4608 x 3072 -> 3072 with gate and residual 75 us (1150
// TFLOP/s), both at the chip's power limit; 2 x 3072 -> 18432 22.4 us (5.1
// TB/s), bound by reading W; fp16 333 x 4096 -> 3072 20 us (415 TFLOP/s),
// bound by the operands' way from L2.

#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include <type_traits>

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
  return z * __builtin_amdgcn_rcpf(1.f + exp2_fast(-t));   // reciprocal within 1 ulp
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

// The tile of a workgroup: each XCD (consecutive ids go to consecutive XCDs)
// takes a contiguous range of tiles, walked in groups of 8 rows of tiles, so
// that tiles that run together share operand panels in its L2.
template <int BN, int BM>
__device__ __forceinline__ void tile_of(const LinArgs& a, int block, int& m0, int& n0) {
  const int tn = (a.N + BN - 1) / BN, tm = (a.M + BM - 1) / BM, tiles = tn * tm;
  const int per = (tiles + 7) / 8, x = block & 7, full = tiles - 8 * (per - 1);   // the first `full` XCDs take `per`
  const int id = (x < full ? x * per : full * per + (x - full) * (per - 1)) + (block >> 3);
  const int group = id / (8 * tn), in = id - group * 8 * tn;
  const int gm = min(8, tm - group * 8);
  m0 = (group * 8 + in % gm) * BM;
  n0 = in / gm * BN;
}

// Epilogue of a workgroup's BN x BM tile.  A wave holds TN x TM results of
// 16 x 16 (lane l, element r: channel 4 (l / 16) + r, row l % 16).  JP of its
// TM rows of tiles at a time go through LDS as [rows][BN] fp32, 16-byte chunk
// c of row r at chunk c ^ (r % 16); then a thread takes 8 channels of a row,
// always the same channels, and the threads together whole rows.  A tile that
// lies inside the result, in rows that allow 16-byte accesses and in one
// group, takes a loop without a check per row, its residual loaded
// ahead; the others go through Columns.
template <typename E, int BN, int BM, int WN, int WM, int TN, int TM, int JP>
__device__ __forceinline__ void epilogue(const LinArgs& a, const v4f (&acc)[TN][TM], uint8_t* lds, int m0, int n0) {
  constexpr int kThreads = WN * WM * 64, kC4 = BN / 4, kLanesRow = BN / 8, kPass = kThreads / kLanesRow;
  constexpr int kRowsJ = JP * WM * 16, kIter = kRowsJ / kPass;
  static_assert(kC4 % 16 == 0 && TM % JP == 0 && kThreads % kLanesRow == 0 && kRowsJ % kPass == 0,
                "the swizzle stays inside a row; whole passes");
  float* const stage = reinterpret_cast<float*>(lds);
  const int l16 = threadIdx.x & 15, q = (threadIdx.x >> 4) & 3, wave = threadIdx.x >> 6;
  const int wn = wave % WN, wm = wave / WN;
  const int c8 = threadIdx.x % kLanesRow, r0 = threadIdx.x / kLanesRow;
  const int nl = n0 + c8 * 8;
  const bool wide = a.splits == 1 && m0 + BM <= a.M && n0 + BN <= a.N && (a.ldy & 7) == 0 && (a.ldr & 7) == 0 &&
                    (!a.gate || m0 / a.group_rows == (m0 + BM - 1) / a.group_rows);
  Columns<E> col;
  if (a.splits == 1) col.init(a, nl);
  if (wide && a.gate) unpack8<E>(load8(a.gate + m0 / a.group_rows * a.ld_gate + nl), col.gate);
  // row of the tile that staged row r is, in pass jp
  auto tile_row = [&](int jp, int r) { return (((r >> 4) % WM) * TM + jp + (r >> 4) / WM) * 16 + (r & 15); };
  auto staged = [&](int r, float (&f)[8]) {
    const v4f lo = *reinterpret_cast<const v4f*>(stage + (r * kC4 + ((2 * c8) ^ (r & 15))) * 4);
    const v4f hi = *reinterpret_cast<const v4f*>(stage + (r * kC4 + ((2 * c8 + 1) ^ (r & 15))) * 4);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      f[e] = lo[e];
      f[4 + e] = hi[e];
    }
  };
#pragma unroll
  for (int jp = 0; jp < TM; jp += JP) {
    if (jp) lds_barrier();
    v4u res[kIter];
    const bool add = wide && a.residual;
    if (add) {
#pragma unroll
      for (int it = 0; it < kIter; ++it)
        res[it] = load8(a.residual + (m0 + tile_row(jp, r0 + it * kPass)) * a.ldr + nl);
    }
    // staged row (jj WM + wm) 16 + l16 is row (wm TM + jp + jj) 16 + l16 of the tile
#pragma unroll
    for (int jj = 0; jj < JP; ++jj)
#pragma unroll
      for (int i = 0; i < TN; ++i)
        *reinterpret_cast<v4f*>(stage + (((jj * WM + wm) * 16 + l16) * kC4 + ((wn * TN * 4 + i * 4 + q) ^ l16)) * 4) =
            acc[i][jp + jj];
    lds_barrier();
    if (wide) {
#pragma unroll
      for (int it = 0; it < kIter; ++it) {
        const int r = r0 + it * kPass;
        float f[8];
        staged(r, f);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] += col.bias[e];
        if (a.act != SVDQ_ACT_NONE) {
#pragma unroll
          for (int e = 0; e < 8; ++e) f[e] = activate(f[e], a.act);
        }
        if (a.gate) {
#pragma unroll
          for (int e = 0; e < 8; ++e) f[e] *= col.gate[e];
        }
        if (add) {
          float x[8];
          unpack8<E>(res[it], x);
#pragma unroll
          for (int e = 0; e < 8; ++e) f[e] += x[e];
        }
        // streamed past the caches, which keep the operands
        stream8(a.y + (m0 + tile_row(jp, r)) * a.ldy + nl, pack8<E>(f));
      }
    } else {
#pragma unroll 1
      for (int r = r0; r < kRowsJ; r += kPass) {
        float f[8];
        staged(r, f);
        const int m = m0 + tile_row(jp, r);
        if (a.splits == 1) {
          col.finish(a, m, f);
        } else if (m < a.M && nl < a.N) {
          float* p = a.part + (static_cast<int64_t>(blockIdx.y) * a.M + m) * a.N + nl;
          if (nl + 8 <= a.N && (a.N & 3) == 0) {
            *reinterpret_cast<v4f*>(p) = v4f{f[0], f[1], f[2], f[3]};
            *reinterpret_cast<v4f*>(p + 4) = v4f{f[4], f[5], f[6], f[7]};
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
              if (nl + e < a.N) p[e] = f[e];
          }
        }
      }
    }
  }
}

// rows of tiles that fit the epilogue's LDS at a time: the largest divisor of TM
constexpr int staged_tiles(int TM, int row_bytes, int bytes) {
  for (int j = TM; j > 1; --j)
    if (TM % j == 0 && j * row_bytes <= bytes) return j;
  return 1;
}

// ---------------------------------------------------------------------------
// Tiles of BN channels x BM rows, WN x WM waves; rows 16-byte aligned and
// K % 8 == 0.  K runs in stages of 64: whole 128-byte lines of the rows of W
// and of x, that loads put straight into LDS, W in a ring of 3 + D slots, x
// in one of 2 + D.  A stage's two steps of 32 k each read the next step's
// operands from LDS between their products.  The one barrier of a stage
// stands before its last step: by then the stage has been read out and the
// next one has landed, so that the last step reads that one's first
// operands.  W of stage + 2 + D is loaded in the first step, x in the last:
// loads have 1 1/2 + D stages and one + D to arrive.  They are spread evenly
// over the products: issued in one burst they block the wave (output
// projection 69 -> 75 us).  D > 0 is for small grids, whose stages are
// shorter than a load's way.
// Products of 16 x 16 x 32: the chip runs this kernel at its power limit
// (zeros 19 % faster than normal values), and they move fewer register bytes
// per product than 32 x 32 x 16 (4608 x 12288 x 3072: 318 -> 298 us).
// A row of a slot is 128 bytes, two rows share the LDS banks: 16-byte chunk c
// of row r sits at chunk c ^ ((r / 2) % 8).
// ---------------------------------------------------------------------------

template <typename E, int BN, int BM, int WN, int WM, int D>
__global__ __launch_bounds__(WN * WM * 64, 2) void k_linear16(LinArgs a) {
  constexpr int kWaves = WN * WM;
  constexpr int TN = BN / WN / 16, TM = BM / WM / 16, T = TN * TM;   // 16 x 16 tiles of a wave
  constexpr int kRowB = 128, kReads = TN + TM;
  // a wave's loads of a slot, 1 KB (8 rows) each; the last waves' may lie past the tile
  constexpr int kLw = (BN / 8 + kWaves - 1) / kWaves, kLx = (BM / 8 + kWaves - 1) / kWaves;
  constexpr int kSlotW = kLw * kWaves * 1024, kSlotX = kLx * kWaves * 1024, kX = (3 + D) * kSlotW;
  constexpr int kLds = kX + (2 + D) * kSlotX;
  static_assert(BN % (16 * WN) == 0 && BM % (16 * WM) == 0 && kReads <= T && kLw <= T && kLx <= T, "tiles divide evenly");
  __shared__ __attribute__((aligned(1024))) uint8_t lds[kLds];

  const int lane = threadIdx.x & 63, l16 = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wn = wave % WN, wm = wave / WN;
  int m0, n0;
  tile_of<BN, BM>(a, blockIdx.x, m0, n0);
  const int stages = (a.K + 63) / 64;
  const int s0 = blockIdx.y * a.stages_per_split, s1 = min(s0 + a.stages_per_split, stages);

  const uint32_t base = lds_addr(lds);
  const __amdgpu_buffer_rsrc_t bw = buffer_of(a.w + n0 * a.ldw, ((a.N - n0 - 1) * a.ldw + a.K) * 2);
  const __amdgpu_buffer_rsrc_t bx = buffer_of(a.x + m0 * a.ldx, ((a.M - m0 - 1) * a.ldx + a.K) * 2);
  // load n of a wave: rows 8 p .. 8 p + 7 of a slot, p = wave kL + n; the
  // lane's chunk is (lane % 8) ^ (4 p + lane / 16) % 8
  auto chunk = [&](int p) { return (lane & 7) ^ (((p & 1) << 2) + (lane >> 4)); };
  int vw[kLw], vx[kLx];
#pragma unroll
  for (int n = 0; n < kLw; ++n) {
    const int r = (wave * kLw + n) * 8 + (lane >> 3);
    vw[n] = r < BN ? static_cast<int>(r * a.ldw * 2) + (chunk(wave * kLw + n) << 4) : kOutside;
  }
#pragma unroll
  for (int n = 0; n < kLx; ++n) {
    const int r = (wave * kLx + n) * 8 + (lane >> 3);
    vx[n] = r < BM ? static_cast<int>(r * a.ldx * 2) + (chunk(wave * kLx + n) << 4) : kOutside;
  }
  // past K, rows would run on into the next
  auto load_w = [&](int st, uint32_t slot, int n) {
    const bool outside = st * 64 + chunk(wave * kLw + n) * 8 >= a.K;
    dma_b128(bw, base + slot + (wave * kLw + n) * 1024, outside ? kOutside : vw[n], st * 128);
  };
  auto load_x = [&](int st, uint32_t slot, int n) {
    const bool outside = st * 64 + chunk(wave * kLx + n) * 8 >= a.K;
    dma_b128(bx, base + slot + (wave * kLx + n) * 1024, outside ? kOutside : vx[n], st * 128);
  };

  // LDS offsets of the lane's operand reads: row, chunk 4 step + q
  uint32_t rw[2], rx[2];
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    const uint32_t o = base + l16 * kRowB + (((4 * s + q) ^ (l16 >> 1)) << 4);
    rw[s] = o + wn * TN * 16 * kRowB;
    rx[s] = o + wm * TM * 16 * kRowB;
  }
  v4f acc[TN][TM];
#pragma unroll
  for (int i = 0; i < TN; ++i)
#pragma unroll
    for (int j = 0; j < TM; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};

  v4u f[2][kReads];   // operands of two steps, W's tiles then x's
  // read i of a step: x's tiles first, the first products take all of them
  auto read = [&](uint32_t sw, uint32_t sx, auto step, int i) {
    constexpr int s = decltype(step)::value;
    if (i < TM)
      f[s][TN + i] = lds_read16(rx[s] + sx + i * 16 * kRowB);
    else
      f[s][i - TM] = lds_read16(rw[s] + sw + (i - TM) * 16 * kRowB);
  };
  // the products of step s, between them the reads of step s ^ 1 (slots sw,
  // sx) and the `loads` loads that `issue` makes
  auto step = [&](auto s_, uint32_t sw, uint32_t sx, auto loads, auto issue) {
    constexpr int s = decltype(s_)::value, kL = decltype(loads)::value, kGap = T / kL;
#pragma unroll
    for (int t = 0; t < T; ++t) {
      acc[t / TM][t % TM] = E::mfma16(f[s][t / TM], f[s][TN + t % TM], acc[t / TM][t % TM]);
      if (t < kReads) read(sw, sx, std::integral_constant<int, s ^ 1>{}, t);
      if (t % kGap == kGap - 1 && t / kGap < kL) issue(t / kGap);
      fence();
    }
    order();
  };
  using I0 = std::integral_constant<int, 0>;
  using I1 = std::integral_constant<int, 1>;

#pragma unroll
  for (int i = 0; i < 2 + D; ++i)
    if (s0 + i < s1) {
#pragma unroll
      for (int n = 0; n < kLw; ++n) load_w(s0 + i, i * kSlotW, n);
#pragma unroll
      for (int n = 0; n < kLx; ++n) load_x(s0 + i, kX + i * kSlotX, n);
    }
  if (s0 + 1 + D < s1)
    lds_wait_barrier<(1 + D) * (kLw + kLx)>();
  else
    lds_wait_barrier<0>();
#pragma unroll
  for (int i = 0; i < kReads; ++i) read(0, kX, I0{}, i);
  // slots of this stage; W's of the stage to load next
  uint32_t ws = 0, xs = kX, wl = (2 + D) * kSlotW;
  auto stage = [&](int st, auto more) {
    constexpr bool kMore = decltype(more)::value;
    step(I0{}, ws, xs, std::integral_constant<int, kLw>{}, [&](int n) {
      if constexpr (kMore) load_w(st + 2 + D, wl, n);
    });
    // read out; stage st + 1 has landed, W of st + 2 + D and the stages between may fly
    lds_wait_barrier<kMore ? kLw + D * (kLw + kLx) : 0>();
    wl = ws;
    ws = ws == (2 + D) * kSlotW ? 0 : ws + kSlotW;
    const uint32_t x = xs;
    xs = xs == kX + (1 + D) * kSlotX ? kX : xs + kSlotX;
    // (past the last stage this reads a slot's old bytes, which are not used)
    step(I1{}, ws, xs, std::integral_constant<int, kLx>{}, [&](int n) {
      if constexpr (kMore) load_x(st + 2 + D, x, n);
    });
  };
  int st = s0;
  for (; st + 2 + D < s1; ++st) stage(st, std::true_type{});
  for (; st < s1; ++st) stage(st, std::false_type{});
  // the reads past the last stage are done before the staging overwrites LDS
  lds_wait_barrier<0>();
  epilogue<E, BN, BM, WN, WM, TN, TM, staged_tiles(TM, WM * 16 * BN * 4, kLds)>(a, acc, lds, m0, n0);
}

// ---------------------------------------------------------------------------
// The same for rows at any 2-byte alignment and any K: tiles of B x B, 2 x 2
// waves, stages of 64 fetched with unaligned loads into registers, AHEAD
// stages before they go to LDS, and from there double-buffered.  Rows past
// the tile repeat the last one (their results are not stored); past K both
// operands are zero.  LDS rows as above.
// ---------------------------------------------------------------------------

template <typename E, int B, int AHEAD>
__global__ __launch_bounds__(256, 2) void k_linear16_any(LinArgs a) {
  constexpr int kRowB = 128, kStage = 2 * B * kRowB, kLoads = kStage / 1024 / 4, kT = B / 32;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[2 * kStage];
  const int lane = threadIdx.x & 63, l16 = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wn = wave & 1, wm = wave >> 1;
  int m0, n0;
  tile_of<B, B>(a, blockIdx.x, m0, n0);
  const int stages = (a.K + 63) / 64;
  const int s0 = blockIdx.y * a.stages_per_split, s1 = min(s0 + a.stages_per_split, stages);

  // load n of a wave: rows 8 (wave kLoads + n) .. + 7; waves 0, 1 take W, 2, 3 take x
  const bool is_x = wave >= 2;
  const uint16_t* const p = is_x ? a.x + m0 * a.ldx : a.w + n0 * a.ldw;
  const int64_t ld = is_x ? a.ldx : a.ldw;
  const int rows = is_x ? a.M - m0 : a.N - n0;
  int64_t at[kLoads];
#pragma unroll
  for (int n = 0; n < kLoads; ++n) {
    const int r = ((wave & 1) * kLoads + n) * 8 + (lane >> 3);
    at[n] = min(r, rows - 1) * ld + ((lane & 7) ^ ((r >> 1) & 7)) * 8;
  }
  v4u held[AHEAD][kLoads];
  auto fetch = [&](int st, v4u (&v)[kLoads]) {
    if (st * 64 + 64 <= a.K) {
#pragma unroll
      for (int n = 0; n < kLoads; ++n) v[n] = load8(p + at[n] + st * 64);
    } else {
#pragma unroll
      for (int n = 0; n < kLoads; ++n) {
        const int r = ((wave & 1) * kLoads + n) * 8 + (lane >> 3);
        const int left = a.K - st * 64 - ((lane & 7) ^ ((r >> 1) & 7)) * 8;
        v[n] = v4u{0, 0, 0, 0};
        if (left > 0) v[n] = load8(p + at[n] + st * 64, left);
      }
    }
  };
  v4f acc[kT][kT];
#pragma unroll
  for (int i = 0; i < kT; ++i)
#pragma unroll
    for (int j = 0; j < kT; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};
  auto stage = [&](int st, v4u (&v)[kLoads]) {
    uint8_t* const buf = lds + (st & 1) * kStage;
#pragma unroll
    for (int n = 0; n < kLoads; ++n) *reinterpret_cast<v4u*>(buf + (wave * kLoads + n) * 1024 + lane * 16) = v[n];
    // the other buffer was read out before this wave's writes of the stage
    // before; loads in flight stay in flight
    lds_barrier();
    if (st + AHEAD < s1) fetch(st + AHEAD, v);
    const uint8_t* const pw = buf + (wn * kT * 16 + l16) * kRowB;
    const uint8_t* const px = buf + (B + wm * kT * 16 + l16) * kRowB;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const int c = ((4 * s + q) ^ (l16 >> 1)) << 4;
      v4u fw[kT], fx[kT];
#pragma unroll
      for (int i = 0; i < kT; ++i) {
        fw[i] = *reinterpret_cast<const v4u*>(pw + i * 16 * kRowB + c);
        fx[i] = *reinterpret_cast<const v4u*>(px + i * 16 * kRowB + c);
      }
#pragma unroll
      for (int i = 0; i < kT; ++i)
#pragma unroll
        for (int j = 0; j < kT; ++j) acc[i][j] = E::mfma16(fw[i], fx[j], acc[i][j]);
    }
  };
#pragma unroll
  for (int i = 0; i < AHEAD; ++i)
    if (s0 + i < s1) fetch(s0 + i, held[i]);
  for (int st = s0; st < s1; st += AHEAD) {
#pragma unroll
    for (int i = 0; i < AHEAD; ++i)
      if (st + i < s1) stage(st + i, held[i]);
  }
  lds_barrier();
  epilogue<E, B, B, 2, 2, kT, kT, staged_tiles(kT, 2 * 16 * B * 4, 2 * kStage)>(a, acc, lds, m0, n0);
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
// channels; its waves take the stages of 128 k in turn, each through LDS of
// its own (two stages in flight, no barrier in the loop), and join at the
// end.  XL: 1 KB loads that bring in the rows of x (4 rows each).  Two
// workgroups share a CU's LDS, so that one reads while the other starts or
// joins (2 x 18432 x 3072: 26.7 us with three stages and one workgroup a CU,
// 23.1 with two and two: 4.9 TB/s); from 9 rows on that takes two waves, which
// pays where there are more workgroups than CUs (16 x 9216 x 3072 18.5 -> 15.9
// us, 4 x 3072 x 15360 27 -> 36).
// ---------------------------------------------------------------------------

template <typename E, int XL, int NW>
__global__ __launch_bounds__(NW * 64, 1) void k_linear16_few(LinArgs a) {
  constexpr int kWaves = NW, kDepth = 2;
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
    if (more >= 1)
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
  // a thread takes 8 channels of every 16 kWaves-th row
  for (int m = threadIdx.x >> 2; m < a.M; m += 16 * kWaves) {
    Columns<E> col;
    col.init(a, n0 + (threadIdx.x & 3) * 8);
    float f[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < kWaves; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] += reinterpret_cast<float*>(lds)[(i * 32 + m) * kRow + (threadIdx.x & 3) * 8 + e];
    col.finish(a, m, f);
  }
}

// Schedules.  `slots`: workgroups the device holds at once; `light` and
// `full`: microseconds of a stage of 64 k with one workgroup a CU or fewer
// and with every slot taken; `fixed`: launch, first loads and epilogue.
// Measured on bf16 normal values with K from 512 to 12288.
struct Shape {
  int bn, bm, waves, slots;
  float light, full, fixed;
};
enum { k256, k128, k128Deep, k64, kAny128, kAny64, kShapes };
constexpr Shape kShape[kShapes] = {
    {256, 256, 8, 256, 1.10f, 1.45f, 8.f},
    {128, 128, 4, 512, 0.50f, 0.83f, 5.f},   // two workgroups a CU
    {128, 128, 8, 256, 0.36f, 0.42f, 5.f},   // loads two stages further ahead
    {64, 64, 4, 512, 0.20f, 0.33f, 4.f},     // one stage further ahead
    {128, 128, 4, 512, 1.00f, 1.60f, 5.f},   // k_linear16_any, two stages ahead
    {64, 64, 4, 512, 0.38f, 0.65f, 4.f},     // k_linear16_any, three stages ahead
};
constexpr int kMaxSplits = 8;

struct Plan {
  int shape, splits, per;
  size_t bytes;
};

// The cheapest shape and number of splits.  Past one round of workgroups
// the cost lies between the rounded-up and the true number of rounds: idle
// CUs of the last one leave the others a higher clock.  The join of splits
// reads and writes them once more, and its launch and workspace cost the host
// as much again as the call (128 x 512 x 2048 whole 9.0 us, split 11.7; 128 x
// 512 x 4096 16.1 and 12.4; 238 x 235 x 7556 54 and 23).
Plan plan_for(int M, int N, int K, bool aligned, int most_splits) {
  const int stages = (K + 63) / 64;
  Plan best{kAny64, 1, stages, 0};
  float least = INFINITY;
  for (int i = aligned ? 0 : kAny128; i < (aligned ? kAny128 : kShapes); ++i) {
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

// up to 32 rows the weights are read once by k_linear16_few
constexpr int kFewRows = 32;
// waves of its workgroups: two from 9 rows on where there are more of them than CUs
int few_waves(int M, int N) { return M > 8 && (N + 31) / 32 > 256 ? 2 : 4; }

dim3 tiles(const LinArgs& a, int bn, int bm) {
  return dim3(static_cast<unsigned>((a.M + bm - 1) / bm) * static_cast<unsigned>((a.N + bn - 1) / bn), a.splits);
}

template <typename E, int BN, int BM, int WN, int WM, int D>
void start(const LinArgs& a, hipStream_t stream) {
  k_linear16<E, BN, BM, WN, WM, D><<<tiles(a, BN, BM), WN * WM * 64, 0, stream>>>(a);
}

template <typename E>
int launch(LinArgs a, bool aligned, size_t workspace, hipStream_t stream) {
  a.splits = 1;
  if (aligned && a.M <= kFewRows) {
    const unsigned blocks = (a.N + 31) / 32;
    const bool two = few_waves(a.M, a.N) == 2;
    if (a.M <= 4)
      k_linear16_few<E, 1, 4><<<blocks, 256, 0, stream>>>(a);
    else if (a.M <= 8)
      k_linear16_few<E, 2, 4><<<blocks, 256, 0, stream>>>(a);
    else if (a.M <= 16 && two)
      k_linear16_few<E, 4, 2><<<blocks, 128, 0, stream>>>(a);
    else if (a.M <= 16)
      k_linear16_few<E, 4, 4><<<blocks, 256, 0, stream>>>(a);
    else if (two)
      k_linear16_few<E, 8, 2><<<blocks, 128, 0, stream>>>(a);
    else
      k_linear16_few<E, 8, 4><<<blocks, 256, 0, stream>>>(a);
    return static_cast<int>(hipGetLastError());
  }
  // the sum's order goes by the sizes: all of the workspace, or one piece
  Plan p = plan_for(a.M, a.N, a.K, aligned, kMaxSplits);
  if (workspace < p.bytes) p = plan_for(a.M, a.N, a.K, aligned, 1);
  a.splits = p.splits;
  a.stages_per_split = p.per;
  switch (p.shape) {
    case k256: start<E, 256, 256, 2, 4, 0>(a, stream); break;
    case k128: start<E, 128, 128, 2, 2, 0>(a, stream); break;
    case k128Deep: start<E, 128, 128, 2, 4, 2>(a, stream); break;
    case k64: start<E, 64, 64, 2, 2, 1>(a, stream); break;
    case kAny128: k_linear16_any<E, 128, 2><<<tiles(a, 128, 128), 256, 0, stream>>>(a); break;
    default: k_linear16_any<E, 64, 3><<<tiles(a, 64, 64), 256, 0, stream>>>(a);
  }
  if (a.splits > 1) {
    const int64_t n = static_cast<int64_t>((a.N + 7) / 8) * a.M;
    k_linear16_join<E><<<dim3(static_cast<unsigned>((n + 255) / 256)), 256, 0, stream>>>(a);
  }
  return static_cast<int>(hipGetLastError());
}

}  // namespace

extern "C" {

int svdq_linear16_aligned(const void* x, int64_t ldx, const void* w, int64_t ldw, int K) {
  return K % 8 == 0 && ldx % 8 == 0 && ldw % 8 == 0 &&
         ((reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(w)) & 15) == 0;
}

size_t svdq_linear16_plan_bytes(int M, int N, int K, int aligned) {
  return aligned && M <= kFewRows ? 0 : plan_for(M, N, K, aligned, kMaxSplits).bytes;
}

void svdq_linear16_plan(int M, int N, int K, int aligned, int32_t* plan) {
  if (aligned && M <= kFewRows) {
    plan[0] = plan[1] = 32;
    plan[2] = few_waves(M, N);
    plan[3] = 1;
    return;
  }
  const Plan p = plan_for(M, N, K, aligned, kMaxSplits);
  plan[0] = kShape[p.shape].bm;
  plan[1] = kShape[p.shape].bn;
  plan[2] = kShape[p.shape].waves;
  plan[3] = p.splits;
}

int svdq_launch_linear16(const void* x, int64_t ldx, const void* w, int64_t ldw, const void* bias, const void* gate,
                         int64_t ld_gate, int group_rows, const void* residual, int64_t ldr, void* y, int64_t ldy, int M,
                         int N, int K, int activation, int dtype, void* workspace, size_t workspace_bytes, void* stream) {
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
  const bool aligned = svdq_linear16_aligned(x, ldx, w, ldw, K);
  const size_t bytes = workspace ? workspace_bytes : 0;
  return dtype == SVDQ_BF16 ? launch<Bf16>(a, aligned, bytes, s) : launch<F16>(a, aligned, bytes, s);
}

}  // extern "C"
