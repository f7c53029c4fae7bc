// What the 16-bit and the 8-bit linear share: the walk over the tiles of the
// result, and the epilogue
//
//   y = residual + gate_g * act(z + bias),  g = row / group_rows
//
// on fp32 products z, rounded once, or the fp32 parts of z that a split along
// K leaves to k_linear_join.  gfx950 only.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "svdq_device.h"
#include "svdq_internal.h"

namespace svdq_dev {
namespace {   // kernels in a header: each file has its own

struct OutArgs {
  const uint16_t *bias, *gate, *residual;
  uint16_t* y;
  float* part;       // [splits][M][N] fp32, splits > 1
  int64_t ld_gate, ldr, ldy;
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

  __device__ __forceinline__ void init(const OutArgs& a, int n_) {
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
  __device__ __forceinline__ void finish(const OutArgs& a, int m, float (&f)[8]) {
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
__device__ __forceinline__ void tile_of(const OutArgs& a, int block, int& m0, int& n0) {
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
__device__ __forceinline__ void epilogue(const OutArgs& a, const v4f (&acc)[TN][TM], uint8_t* lds, int m0, int n0) {
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

// Sum of the splits in their order, then the epilogue: 8 channels a thread.
template <typename E>
__global__ __launch_bounds__(256) void k_linear_join(OutArgs a) {
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

}  // namespace
}  // namespace svdq_dev
