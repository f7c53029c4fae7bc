// Attention over packed sequences for gfx950.
//
//   s_ij = scale q_i . k_j,  p_ij = exp(s_ij - lse_i),  o_i = sum_j p_ij v_j,
//   lse_i = log sum_j exp(s_ij)
//
// over the keys j of the query's own sequence, with causal masking counted
// from the sequences' ends: query i of len_q sees key j of len_k iff
// j <= i + len_k - len_q.  A query with no key gives o = 0, lse = -inf.
//
// Rows.  The g = heads_q / heads_k query heads that share a key head are
// packed with their tokens into one axis of len_q g rows (row R: token R / g,
// head R % g of the group), so that a tile of rows reads each key once for
// all of them and a single token still fills g rows.
//
// Products.  A wave owns 32 rows.  It computes S^T = K Q^T, so that a lane
// holds scores of one row only (column l % 32 of the result): the row's
// maximum and sum are in-lane operations plus one exchange with the lane 32
// away.  The result's registers are, rounded to 16 bits, already the B
// operand of O^T = V^T P^T if the sum over keys runs in the order in which
// they lie there: keys 16 k + 4 h + {0..3, 8..11} for lane half h.  The V^T
// operand is read in that order by two transposing LDS reads (4 keys each).
//
// Softmax.  One pass: running reference m, sum l and O are rescaled only
// when a row's maximum exceeds m by more than 2^8 in the exponent's base
// (exact for any m, since o = O / l and P <= 256 keeps its relative
// precision); O and l are held in fp32, P is rounded to 16 bits to nearest
// even for the matrix core and l sums the unrounded values.
//
// Measured (passes over changing inputs, bf16): 4608 tokens x 24 heads of 128
// 247 to 255 us from card to card (1060 to 1020 TFLOP/s), bound by power (the same
// loop on zeros runs at 1470); one token of each of 8 caches of 0 to 16384
// keys, 8 key heads, 56 us (4.3 TB/s), bound by reading K and V; 77 tokens x
// 12 heads of 64 in fp16, 5.2 us on the device, bound by its launch.  P in 16
// bits makes the error against 64 bits up to 1.41 times that of P in fp32.

#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include <type_traits>

#include "svdq_device.h"
#include "svdq_internal.h"

namespace {

using namespace svdq_dev;

struct AttnArgs {
  const uint16_t *q, *k, *v;
  uint16_t* o;
  float* lse;            // [total_q][heads_q] or null
  float* part_o;         // [splits][total_q][heads_q][D], splits > 1
  float2* part_ml;       // [splits][total_q][heads_q] {m, l}
  const int32_t *cu_q, *cu_k;   // null: one sequence
  int64_t q_t, q_h, k_t, k_h, v_t, v_h, o_t, o_h;   // strides in elements
  int total_q, total_k, batch, heads_q, heads_k, group, D;
  float scale;           // > 0
  int causal, splits, slots;
  // k_attention_spread: workgroups, results of their pieces, and the pieces
  // of the sequences before each (keys x rows in tiles of 32, and rows alone)
  int spread;
  int64_t results;       // that the workspace holds
  int64_t* before;       // [batch + 1]
  int32_t* before_q;     // [batch + 1]
};

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kSlack = 8.f;   // log2 of the largest P before a rescale

struct Tile {
  int q0, len_q, k0, len_k;   // the sequence's tokens
  int row0, rows;             // first row of the tile, rows of the sequence
  int held0, held1;           // find_tile: tokens of q that the sequences hold
  bool any;
};

// The last i in [0, n) with before(i), for a condition that holds up to some
// i (i = 0 at least): a 64-way search by the wave.
template <typename F>
__device__ __forceinline__ int last_before(int n, F before) {
  const int lane = threadIdx.x & 63;
  int at = 0;
  while (n > 1) {
    const int step = (n + 63) >> 6;
    const bool b = lane * step < n && before(at + lane * step);
    const int c = max(static_cast<int>(__popcll(__ballot(b))), 1);
    at += (c - 1) * step;
    n = min(step, n - (c - 1) * step);
  }
  return __builtin_amdgcn_readfirstlane(at);
}

// The tokens from the starts q to q1 and k to k1, inside the tensors whatever
// the starts hold.
__device__ __forceinline__ Tile between(const AttnArgs& a, int q, int q1, int k, int k1) {
  Tile t;
  t.q0 = min(max(q, 0), a.total_q);
  t.len_q = min(max(q1, t.q0), a.total_q) - t.q0;
  t.k0 = min(max(k, 0), a.total_k);
  t.len_k = min(max(k1, t.k0), a.total_k) - t.k0;
  t.rows = t.len_q * a.group;
  t.row0 = 0;
  t.any = t.rows > 0;
  return t;
}

// Sequence seq's tokens.
__device__ __forceinline__ Tile sequence(const AttnArgs& a, int seq) {
  if (!a.cu_q) return between(a, 0, a.total_q, 0, a.total_k);
  return between(a, a.cu_q[seq], a.cu_q[seq + 1], a.cu_k[seq], a.cu_k[seq + 1]);
}

// Rows are cut into tiles of BM per sequence.  Sequence i owns the slots
// from floor(cu[i] g / BM) + i up to the next sequence's first: at least as
// many as it has tiles, and known without reading lengths on the host.  The
// slots left over exit.
template <int BM>
__device__ __forceinline__ Tile find_tile(const AttnArgs& a, int slot) {
  // is sequence i's first slot, with its start, at or before this one?
  auto before = [&](int i, int start) {
    return static_cast<int64_t>(min(max(start, 0), a.total_q)) * a.group / BM + i <= slot;
  };
  int seq = 0;
  Tile t;
  if (a.batch > 1 && a.batch < 64) {
    // every start is in the wave: no second way to memory for the sequence's
    const int i = min(static_cast<int>(threadIdx.x & 63), a.batch);
    const int q = a.cu_q[i], k = a.cu_k[i];
    const uint64_t held = __ballot(i < a.batch && before(i, q));
    seq = max(static_cast<int>(__popcll(held)), 1) - 1;
    auto of = [](int v, int lane) { return __builtin_amdgcn_readlane(v, lane); };
    t = between(a, of(q, seq), of(q, seq + 1), of(k, seq), of(k, seq + 1));
    t.held0 = of(q, 0), t.held1 = of(q, a.batch);
  } else {
    if (a.batch > 1) seq = last_before(a.batch, [&](int i) { return before(i, a.cu_q[i]); });
    t = sequence(a, seq);
    t.held0 = a.cu_q ? a.cu_q[0] : 0, t.held1 = a.cu_q ? a.cu_q[a.batch] : a.total_q;
  }
  t.held0 = min(max(t.held0, 0), a.total_q);
  t.held1 = min(max(t.held1, t.held0), a.total_q);
  const int64_t first = static_cast<int64_t>(t.q0) * a.group / BM + seq;
  const int64_t row0 = (slot - first) * BM;
  t.any = slot >= first && row0 < t.rows;
  t.row0 = t.any ? static_cast<int>(row0) : 0;
  return t;
}

// Tokens of q that no sequence holds (before the first start, past the last)
// see no key: o = 0, lse = -inf, by the workgroups of a key head in turn.
template <int THREADS>
__device__ __forceinline__ void clear_outside(const AttnArgs& a, const Tile& t, int slot, int head_k) {
  const int outside = t.held0 + a.total_q - t.held1;
  if (outside == 0) return;
  const int chunks = a.D / 8, h0 = head_k * a.group;
  for (int64_t i = slot; i < outside; i += a.slots) {
    const int64_t token = i < t.held0 ? i : t.held1 + (i - t.held0);
    for (int c = threadIdx.x; c < a.group * chunks; c += THREADS) {
      const int h = c / chunks;
      *reinterpret_cast<v4u*>(a.o + token * a.o_t + (h0 + h) * a.o_h + (c - h * chunks) * 8) = v4u{0, 0, 0, 0};
    }
    if (a.lse)
      for (int h = threadIdx.x; h < a.group; h += THREADS) a.lse[token * a.heads_q + h0 + h] = -INFINITY;
  }
}

// One K or V tile of KEYS keys in LDS: rows of DP 16-bit values, unpadded.
// The 16-byte chunk c of row r sits at chunk c ^ f(r):
//   K  read 16 bytes a lane from 32 consecutive rows at one chunk: f takes
//      all values over the rows whose chunks share a 256-byte LDS line set;
//   V  read transposed, 64-byte segments of 4 consecutive rows: f moves the
//      4 rows' segments into distinct quarters of a line.
template <int DP>
__device__ __forceinline__ int swz_k(int r) { return DP == 128 ? (r & 15) : ((r >> 1) & 7); }
template <int DP>
__device__ __forceinline__ int swz_v(int r) { return DP == 128 ? (r & 3) << 2 : (r & 2) << 1; }

// byte offset in memory (from the tile's first row) of the chunk that lane
// `lane` of load `n` of a tile brings in; chunks past D lie outside
template <int DP, bool ISV>
__device__ __forceinline__ int tile_voff(int n, int lane, int64_t stride, int D) {
  constexpr int kChunks = DP / 8;
  const int r = n * (64 / kChunks) + lane / kChunks;
  const int c = (lane % kChunks) ^ (ISV ? swz_v<DP>(r) : swz_k<DP>(r));
  return c * 8 < D ? static_cast<int>(r * stride * 2) + c * 16 : kOutside;
}

template <typename E, int DP, int KEYS>
struct WaveTile {
  static constexpr int kKt = KEYS / 32;        // 32-key tiles of S^T
  static constexpr int kDt = DP / 32;          // 32-wide tiles of O^T
  static constexpr int kSteps = DP / 16;       // k steps of the first product
  static constexpr int kBytes = KEYS * DP * 2;

  v4u qf[kSteps];
  v16f acc[kDt];
  float m, l, msc, limit;   // reference, sum, m scale log2(e), m + slack
  float sc, slack;          // scale log2(e), slack in score units
  uint32_t ka[kSteps], va[kDt];   // LDS offsets of the lane's reads

  __device__ __forceinline__ void init(const AttnArgs& a, int lane) {
    const int l32 = lane & 31, h = lane >> 5, i16 = lane & 15;
#pragma unroll
    for (int s = 0; s < kSteps; ++s) ka[s] = l32 * DP * 2 + (((2 * s + h) ^ swz_k<DP>(l32)) << 4);
    const int vr = 4 * h + (i16 >> 2);           // row within 8 keys
#pragma unroll
    for (int d = 0; d < kDt; ++d) {
      const int c = d * 4 + ((lane >> 4) & 1) * 2 + ((i16 & 3) >> 1);
      va[d] = vr * DP * 2 + ((c ^ swz_v<DP>(vr)) << 4) + (i16 & 1) * 8;
    }
#pragma unroll
    for (int d = 0; d < kDt; ++d)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[d][e] = 0.f;
    sc = a.scale * kLog2e;
    slack = kSlack / sc;
    m = limit = -INFINITY;
    l = msc = 0.f;
  }

  // Q fragment: lane (row l % 32, half h), step s: d = 16 s + 8 h .. + 7
  __device__ __forceinline__ void load_q(const uint16_t* row, bool valid, int h, int D) {
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      qf[s] = v4u{0, 0, 0, 0};
      if (valid && 16 * s + 8 * h < D) qf[s] = *reinterpret_cast<const v4u*>(row + 16 * s + 8 * h);
    }
  }

  __device__ __forceinline__ void scores(uint32_t kbuf, v16f (&s)[kKt]) const {
#pragma unroll
    for (int kt = 0; kt < kKt; ++kt)
#pragma unroll
      for (int e = 0; e < 16; ++e) s[kt][e] = 0.f;
#pragma unroll
    for (int st = 0; st < kSteps; ++st)
#pragma unroll
      for (int kt = 0; kt < kKt; ++kt) s[kt] = E::mfma(read_k(kbuf, kt, st), qf[st], s[kt]);
  }

  // keys key0 + .. at or past lim are out of the row's sight
  __device__ __forceinline__ void mask(v16f (&s)[kKt], int key0, int lim, int h) const {
    const int left = lim - key0 - 4 * h;
#pragma unroll
    for (int kt = 0; kt < kKt; ++kt)
#pragma unroll
      for (int e = 0; e < 16; ++e) s[kt][e] = kt * 32 + (e >> 2) * 8 + (e & 3) < left ? s[kt][e] : -INFINITY;
  }

  __device__ __forceinline__ v4u read_k(uint32_t kbuf, int kt, int st) const { return lds_read16(kbuf + ka[st] + kt * 32 * DP * 2); }
  // 16 keys of V^T: 4 + 4 of them for each lane half
  __device__ __forceinline__ v4u read_v(uint32_t vbuf, int ks, int d) const {
    const v2u lo = lds_read_tr(vbuf + va[d] + ks * 16 * DP * 2);
    const v2u hi = lds_read_tr(vbuf + va[d] + (ks * 16 + 8) * DP * 2);
    return v4u{lo.x, lo.y, hi.x, hi.y};
  }

  // maximum over the two lanes that hold a row's keys
  static __device__ __forceinline__ float pair_max(float v) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return __builtin_elementwise_maximum(__uint_as_float(r[0]), __uint_as_float(r[1]));
  }
  __device__ __forceinline__ float top(const v16f (&s)[kKt]) const {
    float mx = s[0][0];
#pragma unroll
    for (int kt = 0; kt < kKt; ++kt)
#pragma unroll
      for (int e = 0; e < 16; ++e) mx = __builtin_elementwise_maximum(mx, s[kt][e]);
    return pair_max(mx);
  }
  // the row's maximum against the reference; O and l move to a new one if
  // any row of the wave needs it
  __device__ __forceinline__ void raise(float mx) {
    if (__ballot(mx > limit)) {
      const float m_new = mx > m ? mx : m;
      const float f = m == -INFINITY ? 0.f : exp2_fast((m - m_new) * sc);
#pragma unroll
      for (int d = 0; d < kDt; ++d) acc[d] *= f;
      l *= f;
      m = m_new;
      limit = m + slack;
      msc = m == -INFINITY ? 0.f : m * sc;
    }
  }

  // pair i of the lane's 8 kKt pairs of weights
  __device__ __forceinline__ void weigh(const v16f (&s)[kKt], v4u (&p)[2 * kKt], int i, float& sum) const {
    const int kt = i >> 3, e = (i & 7) * 2;
    const float x = exp2_fast(__builtin_fmaf(s[kt][e], sc, -msc));
    const float y = exp2_fast(__builtin_fmaf(s[kt][e + 1], sc, -msc));
    sum += x;
    sum += y;
    p[i >> 2][i & 3] = E::pack2(x, y);
  }
  __device__ __forceinline__ void weights(const v16f (&s)[kKt], v4u (&p)[2 * kKt]) {
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < 8 * kKt; ++i) weigh(s, p, i, sum);
    l += sum;
  }

  __device__ __forceinline__ void accumulate(uint32_t vbuf, const v4u (&p)[2 * kKt]) {
#pragma unroll
    for (int ks = 0; ks < 2 * kKt; ++ks)
#pragma unroll
      for (int d = 0; d < kDt; ++d) {
        acc[d] = E::mfma(read_v(vbuf, ks, d), p[ks], acc[d]);
      }
  }

  // The row's sum: its two halves hold those of different keys.  A row that
  // saw no key has no O either: a weight of zero takes a NaN or an infinity of
  // V into it.
  __device__ __forceinline__ float finish() {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(l), __float_as_uint(l), false, false);
    const float sum = __uint_as_float(r[0]) + __uint_as_float(r[1]);
    if (sum == 0.f) {
#pragma unroll
      for (int d = 0; d < kDt; ++d)
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[d][e] = 0.f;
    }
    return sum;
  }
};

__device__ __forceinline__ float lse_of(float m, float l, float scale) { return l == 0.f ? -INFINITY : m * scale + logf(l); }

// Workgroup -> (slot, key head, split).  The workgroups of one (head, split)
// read the same keys; where the units divide evenly, each of the 8 XCDs
// (consecutive ids go to consecutive XCDs) takes whole units, so that its L2
// holds them.  Causal tiles run from the last to the first: a sequence's
// longest first, the sequences of a pack in reverse order whatever their
// lengths.
struct Job {
  int slot, head, split;
};
__device__ __forceinline__ Job job_of(const AttnArgs& a, int id) {
  const int units = a.heads_k * a.splits;
  int w = id;
  if ((units & 7) == 0) w = (id & 7) * (units >> 3) * a.slots + (id >> 3);
  const int unit = w / a.slots;
  const int slot = w - unit * a.slots;
  Job j;
  j.slot = a.causal ? a.slots - 1 - slot : slot;
  j.head = unit / a.splits;
  j.split = unit - j.head * a.splits;
  return j;
}

// ---------------------------------------------------------------------------
// Many rows: NW waves of 32 rows share tiles of 64 keys.
//
// Iteration i has two phases, in each of which matrix and vector work stand
// side by side in the instruction order (a wave issues in order; two waves
// share a SIMD):
//   A  S of tile i + 1 (K), beside most weights of tile i
//   B  O += P V of tile i, beside the last weights of tile i and the maxima
//      of tile i + 1
// Operands are read from LDS kAhead products ahead, K's first ones of the
// next iteration before its barrier.  Tiles come straight to LDS, kLead
// iterations ahead: K of tile i + 2 + kLead and V of tile i + kLead, through
// rings of slots, with one barrier an iteration.  Products of 32 x 32 x 16: the
// vector work needs the issue slots that twice as many of 16 x 16 x 32 take.
//
// PARTS == 2: as many waves again take the second half of the keys, through
// rings of their own, and the first half's join the two results at the end.
// ---------------------------------------------------------------------------

template <typename E, int DP, int NW, int PARTS>
__global__ __launch_bounds__(PARTS * NW * 64, 2) void k_attention(AttnArgs a) {
  constexpr int kKeys = 64, BM = NW * 32;
  using W = WaveTile<E, DP, kKeys>;
  constexpr int kBuf = W::kBytes;
  constexpr int kLoads = kBuf / 1024 / NW;   // 1 KB loads per wave and operand tile
  // tiles ahead of the ones in use; with 4 waves two workgroups or parts share a CU's LDS
  constexpr int kLead = NW == 8 ? 2 : 1, kSlotsK = 2 + kLead, kSlotsV = 1 + kLead;
  constexpr int kPart = (kSlotsK + kSlotsV) * kBuf;   // LDS of a part
  static_assert(kLoads >= 1 && NW * 32 * DP * 2 <= kPart, "loads divide evenly; the output staging fits");
  __shared__ __attribute__((aligned(1024))) uint8_t lds[PARTS * kPart];

  const Job job = job_of(a, blockIdx.x);
  const Tile t = find_tile<BM>(a, job.slot);
  if (a.splits == 1) clear_outside<PARTS * NW * 64>(a, t, job.slot, job.head);   // else the join does
  if (!t.any) return;
  const int lane = threadIdx.x & 63, l32 = lane & 31, h = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) % NW;
  const int part = PARTS > 1 ? __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) / NW : 0;

  // this lane's row
  const int row = t.row0 + wave * 32 + l32;
  const bool valid = row < t.rows;
  const int token = row / a.group;
  const int head = job.head * a.group + (row - token * a.group);
  const int shift = t.len_k - t.len_q + 1;
  const int lim = !valid ? 0x7FFFFFFF : a.causal ? token + shift : t.len_k;

  W w;
  w.init(a, lane);
  w.load_q(a.q + (t.q0 + token) * a.q_t + head * a.q_h, valid, h, a.D);

  // key tiles: up to the last row's limit; the first `open` need no mask
  const int last_row = min(t.row0 + BM, t.rows) - 1;
  const int end = a.causal ? min(t.len_k, last_row / a.group + shift) : t.len_k;
  const int tiles = (max(end, 0) + kKeys - 1) / kKeys;
  const int first_lim = a.causal ? min(t.len_k, t.row0 / a.group + shift) : t.len_k;
  const int cuts = a.splits * PARTS, cut = job.split * PARTS;
  auto cut_at = [&](int i) { return static_cast<int>(static_cast<int64_t>(tiles) * i / cuts); };
  const int t0 = cut_at(cut + part), t1 = cut_at(cut + part + 1);
  const int open = min(max(first_lim, 0) / kKeys, t1);

  int kv[kLoads], vv[kLoads];
#pragma unroll
  for (int n = 0; n < kLoads; ++n) {
    kv[n] = tile_voff<DP, false>(wave * kLoads + n, lane, a.k_t, a.D);
    vv[n] = tile_voff<DP, true>(wave * kLoads + n, lane, a.v_t, a.D);
  }
  const uint32_t base = lds_addr(lds) + part * kPart;
  const uint32_t dst = base + wave * kLoads * 1024;
  const uint16_t* const kp = a.k + t.k0 * a.k_t + job.head * a.k_h;
  const uint16_t* const vp = a.v + t.k0 * a.v_t + job.head * a.v_h;
  // Tile i of K or V: its rows that exist, none past this split.  Loads are
  // made for every tile, those of none bring zeros without going to memory:
  // no branch parts the products from the vector work beside them.
  auto tile = [&](const uint16_t* p, int64_t stride, int i) {
    const int rows = i < t1 ? min(t.len_k - i * kKeys, kKeys) : 0;
    return buffer_of(p + i * (kKeys * stride), rows > 0 ? (rows - 1) * static_cast<int>(stride) * 2 + a.D * 2 : 0);
  };
  constexpr uint32_t kV = kSlotsK * kBuf;
  constexpr int kProducts = W::kKt * W::kSteps;         // of phase A, and of phase B
  constexpr int kAhead = 4, kWeights = 8 * W::kKt;      // pairs of weights
  constexpr int kLate = 4;                              // of which in phase B: those of the last 16 keys
  static_assert(kProducts == 2 * W::kKt * W::kDt && 4 * kLoads <= kProducts, "work divides evenly over the products");

  if (t0 < t1) {
    auto load = [&](const uint16_t* p, int64_t stride, int i, const int (&v)[kLoads], uint32_t slot) {
      const auto r = tile(p, stride, i);
#pragma unroll
      for (int n = 0; n < kLoads; ++n) dma_b128(r, dst + slot + n * 1024, v[n]);
    };
    // K0 K1 V0, then what is further ahead: K2 (V1 K3)
    load(kp, a.k_t, t0, kv, 0);
    load(kp, a.k_t, t0 + 1, kv, kBuf);
    load(vp, a.v_t, t0, vv, kV);
    load(kp, a.k_t, t0 + 2, kv, 2 * kBuf);
    if constexpr (kLead == 2) {
      load(vp, a.v_t, t0 + 1, vv, kV + kBuf);
      load(kp, a.k_t, t0 + 3, kv, 3 * kBuf);
    }
    lds_wait_barrier<2 * kLead * kLoads>();   // K of the first two tiles
    v16f s0[W::kKt], s1[W::kKt];
    w.scores(base, s0);
    if (t0 >= open) w.mask(s0, t0 * kKeys, lim, h);
    float mx = w.top(s0);
    v4u f[kAhead];   // operands read ahead
#pragma unroll
    for (int j = 0; j < kAhead; ++j) f[j] = w.read_k(base + kBuf, j % W::kKt, j / W::kKt);
    lds_wait_barrier<2 * (kLead - 1) * kLoads>();   // V of the first tile, K of the third
    // slots of K's tiles i (free), i + 1, and of V's tile i
    uint32_t k0 = 0, v0 = kV;
    auto after_k = [](uint32_t u, int n) { return u + n * kBuf < kSlotsK * kBuf ? u + n * kBuf : u + n * kBuf - kSlotsK * kBuf; };
    auto after_v = [](uint32_t u, int n) {
      return u + n * kBuf < kV + kSlotsV * kBuf ? u + n * kBuf : u + n * kBuf - kSlotsV * kBuf;
    };

    // tile i's scores in s; those of tile i + 1 go to s_next
    auto iterate = [&](int i, v16f (&s)[W::kKt], v16f (&s_next)[W::kKt], auto masked, auto next) {
      constexpr bool kNext = decltype(next)::value;
      const uint32_t k1 = after_k(k0, 1), k2 = after_k(k0, 2), v1 = after_v(v0, 1), vl = after_v(v0, kLead);
      const auto rk = tile(kp, a.k_t, i + 2 + kLead), rv = tile(vp, a.v_t, i + kLead);
      w.raise(mx);
      v4u p[2 * W::kKt];
      float sum[2] = {0.f, 0.f};
      // pairs of weights that go beside product j of n
      auto weigh = [&](int first, int count, int j, int n) {
#pragma unroll
        for (int x = first + j * count / n; x < first + (j + 1) * count / n; ++x) w.weigh(s, p, x, sum[x & 1]);
      };
#pragma unroll
      for (int j = 0; j < kProducts; ++j) {
        const int st = j / W::kKt, kt = j % W::kKt;
        if constexpr (kNext) {
          if (st == 0)
#pragma unroll
            for (int e = 0; e < 16; ++e) s_next[kt][e] = 0.f;
          s_next[kt] = E::mfma(f[j % kAhead], w.qf[st], s_next[kt]);
        }
        // the next operand: K's, then V's first ones
        if (j + kAhead < kProducts) {
          if constexpr (kNext) f[j % kAhead] = w.read_k(base + k1, (j + kAhead) % W::kKt, (j + kAhead) / W::kKt);
        } else {
          const int n = j + kAhead - kProducts;
          f[j % kAhead] = w.read_v(base + v0, n / W::kDt, n % W::kDt);
        }
        weigh(0, kWeights - kLate, j, kProducts);
        // the loads of the tiles ahead, early and apart
        if constexpr (kNext)
          if (j % 2 == 0 && j / 2 < 2 * kLoads) {
            if (j / 2 < kLoads)
              dma_b128(rv, dst + vl + j / 2 * 1024, vv[j / 2]);
            else
              dma_b128(rk, dst + k0 + (j / 2 - kLoads) * 1024, kv[j / 2 - kLoads]);
          }
        fence();
      }
      if constexpr (kNext && decltype(masked)::value) w.mask(s_next, (i + 1) * kKeys, lim, h);
      if constexpr (kNext) mx = s_next[0][0];
      order();
#pragma unroll
      for (int j = 0; j < kProducts; ++j) {
        const int ks = j / W::kDt, d = j % W::kDt;
        w.acc[d] = E::mfma(f[j % kAhead], p[ks], w.acc[d]);
        if (j + kAhead < kProducts) {
          const int n = j + kAhead;
          f[j % kAhead] = w.read_v(base + v0, n / W::kDt, n % W::kDt);
        } else if constexpr (kNext) {   // past the last tile: a slot's old bytes, not used
          const int n = j + kAhead - kProducts;
          f[j % kAhead] = w.read_k(base + k2, n % W::kKt, n / W::kKt);
        }
        // the last weights before the products that take them, then the maxima
        constexpr int kHalf = kProducts / 2;
        if (j < kHalf) weigh(kWeights - kLate, kLate, j, kHalf);
        if constexpr (kNext) {
          if (j >= kHalf) {
            constexpr int kE = 16 * W::kKt / kHalf;
#pragma unroll
            for (int x = 0; x < kE; ++x) {
              const int n = (j - kHalf) * kE + x;
              mx = __builtin_elementwise_maximum(mx, s_next[n / 16][n % 16]);
            }
          }
        }
        fence();
      }
      w.l += sum[0] + sum[1];
      if constexpr (kNext) {
        mx = W::pair_max(mx);
        // this tile is read out (all but K's operands read ahead are back);
        // K of tile i + 3 and V of tile i + 1 have landed
        order();
        lds_wait_barrier<2 * (kLead - 1) * kLoads, kAhead>();
        k0 = k1;
        v0 = v1;
      } else {
        lds_wait_barrier<0>();
      }
    };
    using Yes = std::true_type;
    using No = std::false_type;
    int i = t0;
    const int plain = min(open, t1) - 1;   // iterations whose next tile needs no mask
    for (; i + 1 < plain; i += 2) {
      iterate(i, s0, s1, No{}, Yes{});
      iterate(i + 1, s1, s0, No{}, Yes{});
    }
    for (; i < t1 - 1; ++i) {
      iterate(i, s0, s1, Yes{}, Yes{});
#pragma unroll
      for (int kt = 0; kt < W::kKt; ++kt) s0[kt] = s1[kt];
    }
    iterate(i, s0, s1, No{}, No{});
  }

  float l = w.finish();
  if constexpr (PARTS > 1) {
    // every part meets the barriers of the longest: two and one a tile
    static_assert(PARTS == 2, "the join is written for two");
    const int mine = t1 > t0 ? 2 + t1 - t0 : 0;
    const int other = cut_at(cut + 2 - part) - cut_at(cut + 1 - part);
    const int all = max(mine, other > 0 ? 2 + other : 0);
    for (int i = mine; i < all; ++i) lds_wait_barrier<0>();
    // the second part's O, m and l through its LDS, a lane's for the same lane
    constexpr int kQuads = W::kDt * 4;
    static_assert((kQuads * 16 + 8) * 64 * NW <= kPart, "the join fits");
    uint8_t* const joint = lds + kPart + wave * (kQuads * 16 + 8) * 64;
    if (part == 1) {
#pragma unroll
      for (int d = 0; d < W::kDt; ++d)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          *reinterpret_cast<v4f*>(joint + ((d * 4 + j) * 64 + lane) * 16) =
              v4f{w.acc[d][4 * j], w.acc[d][4 * j + 1], w.acc[d][4 * j + 2], w.acc[d][4 * j + 3]};
      *reinterpret_cast<v2f*>(joint + kQuads * 1024 + lane * 8) = v2f{w.m, l};
    }
    __syncthreads();
    if (part == 1) return;
    const v2f ml = *reinterpret_cast<const v2f*>(joint + kQuads * 1024 + lane * 8);
    const float m = ml[0] > w.m ? ml[0] : w.m;
    const float f0 = w.m == -INFINITY ? 0.f : exp2_fast((w.m - m) * w.sc);
    const float f1 = ml[0] == -INFINITY ? 0.f : exp2_fast((ml[0] - m) * w.sc);
    w.m = m;
    l = l * f0 + ml[1] * f1;
#pragma unroll
    for (int d = 0; d < W::kDt; ++d)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const v4f x = *reinterpret_cast<const v4f*>(joint + ((d * 4 + j) * 64 + lane) * 16);
#pragma unroll
        for (int e = 0; e < 4; ++e) w.acc[d][4 * j + e] = w.acc[d][4 * j + e] * f0 + x[e] * f1;
      }
  }
  const int64_t out_row = static_cast<int64_t>(t.q0 + token) * a.heads_q + head;
  if (a.splits > 1) {
    if (valid) {
      const int64_t part = static_cast<int64_t>(job.split) * a.total_q * a.heads_q + out_row;
      if (h == 0) a.part_ml[part] = make_float2(w.m, l);
      float* po = a.part_o + part * a.D;
#pragma unroll
      for (int d = 0; d < W::kDt; ++d)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (d * 32 + 8 * j + 4 * h < a.D)
            *reinterpret_cast<v4f*>(po + d * 32 + 8 * j + 4 * h) =
                v4f{w.acc[d][4 * j], w.acc[d][4 * j + 1], w.acc[d][4 * j + 2], w.acc[d][4 * j + 3]};
    }
    return;
  }
  if (a.lse && valid && h == 0) a.lse[out_row] = lse_of(w.m, l, a.scale);
  // O through the wave's own part of LDS, so that a store covers whole rows
  const float inv = l == 0.f ? 0.f : 1.f / l;
  constexpr int kChunks = DP / 8;
  uint8_t* const stage = lds + wave * 32 * DP * 2;
#pragma unroll
  for (int d = 0; d < W::kDt; ++d)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int c = (d * 4 + j) ^ swz_k<DP>(l32);
      *reinterpret_cast<v2u*>(stage + l32 * DP * 2 + c * 16 + h * 8) =
          v2u{E::pack2(w.acc[d][4 * j] * inv, w.acc[d][4 * j + 1] * inv),
              E::pack2(w.acc[d][4 * j + 2] * inv, w.acc[d][4 * j + 3] * inv)};
    }
#pragma unroll
  for (int it = 0; it < DP / 16; ++it) {
    const int r = it * (64 / kChunks) + lane / kChunks, c = lane % kChunks;
    const int rr = t.row0 + wave * 32 + r;
    const int tok = rr / a.group;
    const v4u x = *reinterpret_cast<const v4u*>(stage + r * DP * 2 + ((c ^ swz_k<DP>(r)) << 4));
    if (rr < t.rows && c * 8 < a.D)
      stream8(a.o + (t.q0 + tok) * a.o_t + (job.head * a.group + rr - tok * a.group) * a.o_h + c * 8, x);
  }
}

// ---------------------------------------------------------------------------
// Few rows (single tokens): tiles of 32 rows, whose 4 waves take the key
// tiles in turn, 32 keys each, through LDS of their own (no barrier in the
// loop), and join their results at the end.  Bound by reading K and V.
// ---------------------------------------------------------------------------

template <typename E, int DP>
struct Few {
  static constexpr int kKeys = 32, BM = 32, NW = 4;
  using W = WaveTile<E, DP, kKeys>;
  static constexpr int kBuf = W::kBytes;          // one operand tile
  static constexpr int kLoads = kBuf / 1024;
  static constexpr int kRow = DP + 4;             // floats of a row of O; the pad spreads rows over banks
  struct Lds {
    uint8_t kv[NW * 4 * kBuf];   // per wave: K0 V0 K1 V1, then its O
    float m[NW][32], l[NW][32];
  };

  // Key tiles [t0, t1) of a tile of rows: leaves O and l of each wave in
  // LDS, scaled to the rows' common reference.
  static __device__ __forceinline__ void run(const AttnArgs& a, const Tile& t, int head_k, int t0, int t1, Lds& lds) {
    const int lane = threadIdx.x & 63, l32 = lane & 31, h = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int row = t.row0 + l32;
    const bool valid = row < t.rows;
    const int token = row / a.group;
    const int head = head_k * a.group + (row - token * a.group);
    const int shift = t.len_k - t.len_q + 1;
    const int lim = !valid ? 0x7FFFFFFF : a.causal ? token + shift : t.len_k;

    W w;
    w.init(a, lane);
    w.load_q(a.q + (t.q0 + token) * a.q_t + head * a.q_h, valid, h, a.D);

    const int last_row = min(t.row0 + BM, t.rows) - 1;
    const int end = a.causal ? min(t.len_k, last_row / a.group + shift) : t.len_k;
    t1 = min(t1, (max(end, 0) + kKeys - 1) / kKeys);   // past it no row sees a key
    const int first_lim = a.causal ? min(t.len_k, t.row0 / a.group + shift) : t.len_k;
    int kv[kLoads], vv[kLoads];
#pragma unroll
    for (int n = 0; n < kLoads; ++n) {
      kv[n] = tile_voff<DP, false>(n, lane, a.k_t, a.D);
      vv[n] = tile_voff<DP, true>(n, lane, a.v_t, a.D);
    }
    const uint32_t base = lds_addr(lds.kv) + wave * 4 * kBuf;
    const uint16_t* const kp = a.k + t.k0 * a.k_t + head_k * a.k_h;
    const uint16_t* const vp = a.v + t.k0 * a.v_t + head_k * a.v_h;
    auto load = [&](int i, int buf) {
      const int left = t.len_k - i * kKeys;
      const auto rk = buffer_of(kp + i * kKeys * a.k_t, (left - 1) * a.k_t * 2 + a.D * 2);
      const auto rv = buffer_of(vp + i * kKeys * a.v_t, (left - 1) * a.v_t * 2 + a.D * 2);
#pragma unroll
      for (int n = 0; n < kLoads; ++n) dma_b128(rk, base + 2 * buf * kBuf + n * 1024, kv[n]);
#pragma unroll
      for (int n = 0; n < kLoads; ++n) dma_b128(rv, base + (2 * buf + 1) * kBuf + n * 1024, vv[n]);
    };
    if (t0 + wave < t1) load(t0 + wave, 0);
    if (t0 + wave + NW < t1) load(t0 + wave + NW, 1);
    int b = 0;
    for (int i = t0 + wave; i < t1; i += NW, b ^= 1) {
      if (i + NW < t1)
        vm_wait<2 * kLoads>();   // tile i is there, tile i + NW may fly
      else
        vm_wait<0>();
      v16f s[1];
      w.scores(base + 2 * b * kBuf, s);
      if ((i + 1) * kKeys > first_lim) w.mask(s, i * kKeys, lim, h);
      w.raise(w.top(s));
      v4u p[2];
      w.weights(s, p);
      w.accumulate(base + (2 * b + 1) * kBuf, p);
      // the reads of this buffer are done before it is loaded again
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      if (i + 2 * NW < t1) load(i + 2 * NW, b);
    }

    // join the waves: common reference, then O and l scaled to it
    const float l = w.finish();
    if (h == 0) lds.m[wave][l32] = w.m;
    __syncthreads();
    float m_all = lds.m[0][l32];
#pragma unroll
    for (int i = 1; i < NW; ++i) m_all = lds.m[i][l32] > m_all ? lds.m[i][l32] : m_all;
    const float f = w.m == -INFINITY ? 0.f : exp2_fast((w.m - m_all) * w.sc);
    float* const mine = reinterpret_cast<float*>(lds.kv + wave * 4 * kBuf);
    static_assert(32 * kRow * 4 <= 4 * kBuf, "a wave's O fits in its buffers");
#pragma unroll
    for (int d = 0; d < W::kDt; ++d)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        *reinterpret_cast<v4f*>(mine + l32 * kRow + d * 32 + 8 * j + 4 * h) =
            v4f{w.acc[d][4 * j] * f, w.acc[d][4 * j + 1] * f, w.acc[d][4 * j + 2] * f, w.acc[d][4 * j + 3] * f};
    if (h == 0) lds.l[wave][l32] = l * f;
    __syncthreads();
  }

  // The rows' results, kOf threads a row: ml(row, m, l) by one of them,
  // o(row, d, four unnormalized values of O, l) by all.
  template <typename ML, typename O>
  static __device__ __forceinline__ void finish(const AttnArgs& a, const Tile& t, const Lds& lds, ML ml, O o) {
    constexpr int kOf = 2 * NW;
    const int r = threadIdx.x / kOf;
    if (t.row0 + r >= t.rows) return;
    float m = lds.m[0][r], l = lds.l[0][r];
#pragma unroll
    for (int i = 1; i < NW; ++i) {
      m = lds.m[i][r] > m ? lds.m[i][r] : m;
      l += lds.l[i][r];
    }
    if (threadIdx.x % kOf == 0) ml(r, m, l);
    for (int d = threadIdx.x % kOf * 4; d < a.D; d += kOf * 4) {
      v4f x = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < NW; ++i) x += *reinterpret_cast<const v4f*>(reinterpret_cast<const float*>(lds.kv + i * 4 * kBuf) + r * kRow + d);
      o(r, d, x, l);
    }
  }
};

// One workgroup runs through all keys of a tile of rows and a key head.
template <typename E, int DP>
__global__ __launch_bounds__(256, 1) void k_attention_few(AttnArgs a) {
  using F = Few<E, DP>;
  __shared__ __attribute__((aligned(1024))) typename F::Lds lds;
  const Job job = job_of(a, blockIdx.x);
  const Tile t = find_tile<F::BM>(a, job.slot);
  clear_outside<256>(a, t, job.slot, job.head);
  if (!t.any) return;
  F::run(a, t, job.head, 0, 0x7FFFFFFF, lds);
  auto place = [&](int r, int& token, int& head) {
    token = (t.row0 + r) / a.group;
    head = job.head * a.group + t.row0 + r - token * a.group;
    token += t.q0;
  };
  F::finish(
      a, t, lds,
      [&](int r, float m, float l) {
        int token, head;
        place(r, token, head);
        if (a.lse) a.lse[static_cast<int64_t>(token) * a.heads_q + head] = lse_of(m, l, a.scale);
      },
      [&](int r, int d, v4f x, float l) {
        int token, head;
        place(r, token, head);
        const float inv = l == 0.f ? 0.f : 1.f / l;
        *reinterpret_cast<v2u*>(a.o + token * a.o_t + head * a.o_h + d) =
            v2u{E::pack2(x[0] * inv, x[1] * inv), E::pack2(x[2] * inv, x[3] * inv)};
      });
}

// Few rows and few heads: the pieces of work (a tile of 32 rows, a tile of
// 32 keys, a key head), laid in a line by head, sequence, rows and keys, are
// cut into a.spread equal parts, one a workgroup, whatever the sequences'
// lengths.  A part may run over several tiles of rows; its share of each, its
// "result" p = workgroup + (tiles of rows before this one), is written for
// k_attention_spread_join (p grows with every step along the line, so no two
// results share one).
constexpr int kSpreadBatch = 512;

// Units of a tile of rows on the line: its tiles of keys, and before them
// what starting it costs a workgroup (5 tokens of 24 heads over 1342, 124, 14,
// 4 and 1 keys: 28 us with the tiles alone, 17 with these).
constexpr int kStartUnits = 8;
__device__ __forceinline__ int line_units(int len_k) { return len_k > 0 ? ((len_k + 31) >> 5) + kStartUnits : 0; }

template <typename E, int DP>
__global__ __launch_bounds__(256, 1) void k_attention_spread(AttnArgs a) {
  using F = Few<E, DP>;
  __shared__ __attribute__((aligned(1024))) typename F::Lds lds;
  __shared__ int64_t before[kSpreadBatch + 1];
  __shared__ int32_t before_q[kSpreadBatch + 1];
  if (threadIdx.x < 64) {
    const int lane = threadIdx.x;
    int64_t sum = 0;
    int sum_q = 0;
    for (int i0 = 0; i0 < a.batch; i0 += 64) {
      int64_t n = 0;
      int nq = 0;
      if (i0 + lane < a.batch) {
        const Tile t = sequence(a, i0 + lane);
        nq = (t.rows + 31) >> 5;
        n = static_cast<int64_t>(nq) * line_units(t.len_k);
      }
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) {
        const int64_t x = __shfl_up(n, o);
        const int xq = __shfl_up(nq, o);
        if (lane >= o) {
          n += x;
          nq += xq;
        }
      }
      if (i0 + lane < a.batch) {
        before[i0 + lane + 1] = sum + n;
        before_q[i0 + lane + 1] = sum_q + nq;
      }
      sum += __shfl(n, 63);
      sum_q += __shfl(nq, 63);
    }
    if (lane == 0) {
      before[0] = 0;
      before_q[0] = 0;
    }
  }
  __syncthreads();
  if (blockIdx.x == 0)
    for (int i = threadIdx.x; i <= a.batch; i += 256) {
      a.before[i] = before[i];
      a.before_q[i] = before_q[i];
    }
  const int64_t per_head = before[a.batch], total = per_head * a.heads_k;
  const int tiles_q = before_q[a.batch];
  int64_t at = total * blockIdx.x / a.spread;
  const int64_t end = total * (blockIdx.x + 1) / a.spread;
  while (at < end) {
    const int head = static_cast<int>(at / per_head);
    const int64_t r = at - head * per_head;
    const int seq = last_before(a.batch, [&](int i) { return before[i] <= r; });
    Tile t = sequence(a, seq);
    const int units = line_units(t.len_k);
    const int64_t rest = r - before[seq];
    const int qt = static_cast<int>(rest / units), u0 = static_cast<int>(rest - static_cast<int64_t>(qt) * units);
    const int u1 = static_cast<int>(end - at < units - u0 ? u0 + (end - at) : units);
    at += u1 - u0;
    if (u1 <= kStartUnits) continue;   // its first tile of keys is the next workgroup's
    t.row0 = qt * 32;
    const int64_t p = static_cast<int64_t>(blockIdx.x) + static_cast<int64_t>(head) * tiles_q + before_q[seq] + qt;
    if (p >= a.results) return;   // only with starts that do not rise
    F::run(a, t, head, u0 > kStartUnits ? u0 - kStartUnits : 0, u1 - kStartUnits, lds);
    F::finish(
        a, t, lds, [&](int row, float m, float l) { a.part_ml[p * 32 + row] = make_float2(m, l); },
        [&](int row, int d, v4f x, float) { *reinterpret_cast<v4f*>(a.part_o + (p * 32 + row) * a.D + d) = x; });
    __syncthreads();   // LDS is read out before the next loads
  }
}

// Join of the results of one row, a workgroup's 4 waves taking them in turn,
// always in the same order.
template <typename E>
__global__ __launch_bounds__(256) void k_attention_spread_join(AttnArgs a) {
  __shared__ float top[4], sums[4], scale[256];
  __shared__ int64_t where[256];
  __shared__ v2f part[4][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int token = blockIdx.x / a.heads_q, hq = blockIdx.x - token * a.heads_q;
  int seq = 0, tiles_before, tiles_q;   // tiles of rows
  int64_t units_before, per_head;       // units of the line
  Tile t;
  if (a.batch < 64) {
    // all of it in one way to memory
    const int i = min(lane, a.batch);
    const int64_t units = a.before[i];
    const int rows = a.before_q[i];
    int q = i ? a.total_q : 0, k = i ? a.total_k : 0;
    if (a.cu_q) q = a.cu_q[i], k = a.cu_k[i];
    const uint64_t held = __ballot(i < a.batch && q <= token);
    seq = max(static_cast<int>(__popcll(held)), 1) - 1;
    auto of = [](int v, int from) { return __builtin_amdgcn_readlane(v, from); };
    auto of64 = [&](int64_t v, int from) {
      return static_cast<int64_t>(static_cast<uint64_t>(static_cast<uint32_t>(of(static_cast<int>(v >> 32), from))) << 32 |
                                  static_cast<uint32_t>(of(static_cast<int>(v), from)));
    };
    t = between(a, of(q, seq), of(q, seq + 1), of(k, seq), of(k, seq + 1));
    units_before = of64(units, seq), per_head = of64(units, a.batch);
    tiles_before = of(rows, seq), tiles_q = of(rows, a.batch);
  } else {
    seq = last_before(a.batch, [&](int i) { return a.cu_q[i] <= token; });
    t = sequence(a, seq);
    units_before = a.before[seq], per_head = a.before[a.batch];
    tiles_before = a.before_q[seq], tiles_q = a.before_q[a.batch];
  }
  const int64_t total = per_head * a.heads_k;
  const int head = hq / a.group, tiles_k = (t.len_k + 31) >> 5;
  const int row = (token - t.q0) * a.group + hq - head * a.group;
  const int qt = row >> 5;
  int n = 0;   // workgroups from the first to the last that took part
  int64_t first = 0, b0 = 0, b1 = 0, tile = 0;
  if (tiles_k > 0 && row >= 0 && row < t.rows) {
    b0 = head * per_head + units_before + static_cast<int64_t>(qt) * line_units(t.len_k) + kStartUnits;
    b1 = b0 + tiles_k;
    // workgroup w begins at floor(total w / spread)
    first = ((b0 + 1) * a.spread - 1) / total;
    n = static_cast<int>((b1 * a.spread - 1) / total - first) + 1;
    tile = static_cast<int64_t>(head) * tiles_q + tiles_before + qt;
  }
  // one result a thread (no more workgroups than threads)
  float2 ml = make_float2(-INFINITY, 0.f);
  if (static_cast<int>(threadIdx.x) < n) {
    const int64_t w = first + threadIdx.x;
    const int64_t from = total * w / a.spread, to = total * (w + 1) / a.spread;
    const int64_t at = (w + tile) * 32 + (row & 31);
    where[threadIdx.x] = at;
    // (a workgroup without a share wrote nothing)
    if ((from > b0 ? from : b0) < (to < b1 ? to : b1) && at < a.results * 32) ml = a.part_ml[at];
  }
  float m = ml.x;
#pragma unroll
  for (int o = 32; o; o >>= 1) {
    const float x = __shfl_xor(m, o);
    m = x > m ? x : m;
  }
  if (lane == 0) top[wave] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 4; ++i) m = top[i] > m ? top[i] : m;
  const float f = ml.y == 0.f ? 0.f : exp2_fast((ml.x - m) * (a.scale * kLog2e));
  float l = ml.y * f;
  scale[threadIdx.x] = f;
#pragma unroll
  for (int o = 32; o; o >>= 1) l += __shfl_xor(l, o);
  if (lane == 0) sums[wave] = l;
  __syncthreads();
  l = (sums[0] + sums[1]) + (sums[2] + sums[3]);
  v2f x = {0.f, 0.f};
  const int d = 2 * lane;
  if (d < a.D) {
#pragma unroll 4
    for (int i = wave; i < n; i += 4)
      if (scale[i] != 0.f) x += *reinterpret_cast<const v2f*>(a.part_o + where[i] * a.D + d) * scale[i];
  }
  part[wave][lane] = x;
  __syncthreads();
  if (wave) return;
  x = (part[0][lane] + part[1][lane]) + (part[2][lane] + part[3][lane]);
  const float inv = l == 0.f ? 0.f : 1.f / l;
  if (d < a.D)
    *reinterpret_cast<uint32_t*>(a.o + token * a.o_t + hq * a.o_h + d) = E::pack2(x[0] * inv, x[1] * inv);
  if (a.lse && lane == 0) a.lse[blockIdx.x] = lse_of(m, l, a.scale);
}

// Join of the splits: a wave per row, in the order of the splits.  A split
// that saw no key wrote l = 0 and is left out (its O is not read).
template <typename E>
__global__ __launch_bounds__(256) void k_attention_join(AttnArgs a) {
  const int lane = threadIdx.x & 63;
  const int64_t rows = static_cast<int64_t>(a.total_q) * a.heads_q;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 6);
  if (row >= rows) return;
  const int64_t tok = row / a.heads_q;
  // no split wrote a row that no sequence holds
  const bool held = !a.cu_q || (tok >= a.cu_q[0] && tok < a.cu_q[a.batch]);
  float2 ml = make_float2(-INFINITY, 0.f);
  if (held && lane < a.splits) ml = a.part_ml[lane * rows + row];
  float m = ml.x;
#pragma unroll
  for (int o = 32; o; o >>= 1) {
    const float x = __shfl_xor(m, o);
    m = x > m ? x : m;
  }
  const float f = ml.y == 0.f ? 0.f : exp2_fast((ml.x - m) * (a.scale * kLog2e));
  float l = ml.y * f;
#pragma unroll
  for (int o = 32; o; o >>= 1) l += __shfl_xor(l, o);
  const float inv = l == 0.f ? 0.f : 1.f / l;
  float x0 = 0.f, x1 = 0.f;
  const int d = 2 * lane;
  for (int s = 0; s < a.splits; ++s) {
    const float fs = __shfl(f, s);
    if (__shfl(ml.y, s) != 0.f && d < a.D) {
      const float2 x = *reinterpret_cast<const float2*>(a.part_o + (s * rows + row) * a.D + d);
      x0 += x.x * fs;
      x1 += x.y * fs;
    }
  }
  if (d < a.D)
    *reinterpret_cast<uint32_t*>(a.o + tok * a.o_t + (row - tok * a.heads_q) * a.o_h + d) = E::pack2(x0 * inv, x1 * inv);
  if (a.lse && lane == 0) a.lse[row] = lse_of(m, l, a.scale);
}

struct Plan {
  int waves;     // rows a workgroup takes / 32; 0: k_attention_few or k_attention_spread
  int splits;    // of a tile's keys, waves > 0
  int parts;     // of the keys within a workgroup, waves == 4
  int spread;    // workgroups of k_attention_spread, or 0
  size_t bytes;
};

// bytes of k_attention_spread's counts, before its results
size_t spread_head(int batch) { return (static_cast<size_t>(batch + 1) * 12 + 15) & ~size_t(15); }

// The schedule from the sizes the host knows.  Lengths are on the device, so
// the mean stands for them; every schedule is right for any lengths.
Plan plan_for(int total_q, int total_k, int batch, int heads_q, int heads_k, int D, bool causal) {
  const int64_t rows = static_cast<int64_t>(total_q) * (heads_q / heads_k);
  const int64_t mean_rows = rows / batch, mean_keys = total_k / batch;
  auto units = [&](int bm) { return (rows / bm > batch ? rows / bm : batch) * heads_k; };
  Plan p;
  // Rows by the 32 (k_attention_few): single tokens, and small grids of short
  // sequences that fit one round (256 tokens x 24 heads 9.2 -> 7.8 us; with
  // more workgroups than CUs 128-row tiles win, 512 tokens 31 against 14 us).
  // Tiles of 128 rows: causal (4608 x 24 heads 166 -> 147 us), grids of one
  // such tile a CU at most, and few keys, where starting up is most of it (8192
  // rows x 10 heads over 77 and 154 keys 16 -> 13 us).  Else 256 rows, which
  // read the keys half as often (4608 x 24 heads 261 -> 246 us, 2048 x 24 62 ->
  // 58, 1500 x 24 46 -> 42).
  const bool few = mean_rows <= 64 || (mean_rows <= 256 && units(32) <= 256);
  p.waves = few ? 0 : causal || units(128) <= 256 || mean_keys < 1024 ? 4 : 8;
  p.splits = 1;
  p.parts = 1;
  p.spread = 0;
  p.bytes = 0;
  const int64_t n = units(p.waves ? p.waves * 32 : 32);
  if (p.waves == 0) {
    // Where the tiles of rows are fewer than the CUs and the keys are long,
    // one workgroup a CU with equal shares of at least 12 units.
    // One token over so many keys, in one workgroup a head and spread, the
    // second kernel with it (24 heads of 128): 300 keys 8 and 14 us, 1000 keys
    // 15 and 15, 2000 keys 24 and 16, 4000 keys 54 and 22.  Of several
    // sequences the mean alone is known but the longest counts: from 256 keys
    // (4 of 300 each 8 and 14 us, 5 of 1342 .. 1 18 and 17).  From as many tiles
    // of rows as CUs on each keeps its workgroup: with equal caches that is
    // faster (64 of 2000 keys, 8 key heads of 128: 96 and 108 us in equal
    // shares, of 64: 53 and 61), with one long cache among short ones much
    // slower (16384 with 63 of 100: 183 and 34, 112 and 24).
    const int64_t tiles = (mean_keys + 31) / 32;
    if (tiles <= (batch == 1 ? 32 : 8)) return p;
    int64_t w = n / heads_k * (tiles + kStartUnits) * heads_k / 12;
    if (w > 256) w = 256;
    if (batch > kSpreadBatch || w <= n) return p;
    p.spread = static_cast<int>(w);
    const int64_t results = w + (rows / 32 + batch) * heads_k;
    p.bytes = spread_head(batch) + static_cast<size_t>(results) * 32 * (D + 2) * 4;
    return p;
  }
  // One tile of 128 rows a CU at most: its keys in two parts, so that each SIMD
  // has two waves (heads of 128, tokens x heads: 1024 x 24 23.1 -> 21.6 us, 2048
  // x 8 39 -> 32, 2048 x 16 54 -> 37, 8192 x 4 189 -> 126; with more tiles 2048
  // x 24 62 -> 74; 600 keys no difference, 512 keys 14.0 -> 14.6).
  if (p.waves == 4 && n <= 256 && mean_keys >= 768) p.parts = 2;
  // Splits, where the tiles would leave half the CUs idle: until half of them
  // have a workgroup of two parts, or all one of one (2048 x 4: 36 us whole, 30
  // in two parts, 28 in two splits of two).
  const int64_t enough = p.parts == 2 ? 128 : 256;
  int64_t s = n >= 128 ? 1 : (enough + n - 1) / n;
  if (s > mean_keys / 512) s = mean_keys / 512;
  p.splits = static_cast<int>(s < 1 ? 1 : s > 64 ? 64 : s);
  if (p.splits > 1) p.bytes = static_cast<size_t>(p.splits) * total_q * heads_q * (D + 2) * 4;
  return p;
}

template <typename E>
int launch(AttnArgs a, const Plan& p, hipStream_t stream) {
  const int bm = p.waves ? p.waves * 32 : 32;
  a.splits = p.splits;
  a.spread = p.spread;
  a.slots = static_cast<int>(static_cast<int64_t>(a.total_q) * a.group / bm) + a.batch;
  const dim3 grid(static_cast<unsigned>(a.slots) * a.heads_k * a.splits);
  const bool wide = a.D > 64;
  if (p.waves == 8) {
    if (wide)
      k_attention<E, 128, 8, 1><<<grid, 512, 0, stream>>>(a);
    else
      k_attention<E, 64, 8, 1><<<grid, 512, 0, stream>>>(a);
  } else if (p.waves == 4 && p.parts == 2) {
    if (wide)
      k_attention<E, 128, 4, 2><<<grid, 512, 0, stream>>>(a);
    else
      k_attention<E, 64, 4, 2><<<grid, 512, 0, stream>>>(a);
  } else if (p.waves == 4) {
    if (wide)
      k_attention<E, 128, 4, 1><<<grid, 256, 0, stream>>>(a);
    else
      k_attention<E, 64, 4, 1><<<grid, 256, 0, stream>>>(a);
  } else if (p.spread) {
    if (wide)
      k_attention_spread<E, 128><<<p.spread, 256, 0, stream>>>(a);
    else
      k_attention_spread<E, 64><<<p.spread, 256, 0, stream>>>(a);
    k_attention_spread_join<E><<<dim3(static_cast<unsigned>(a.total_q) * a.heads_q), 256, 0, stream>>>(a);
  } else {
    if (wide)
      k_attention_few<E, 128><<<grid, 256, 0, stream>>>(a);
    else
      k_attention_few<E, 64><<<grid, 256, 0, stream>>>(a);
  }
  if (a.splits > 1) {
    const int64_t rows = static_cast<int64_t>(a.total_q) * a.heads_q;
    k_attention_join<E><<<dim3(static_cast<unsigned>((rows + 3) / 4)), 256, 0, stream>>>(a);
  }
  return static_cast<int>(hipGetLastError());
}

}  // namespace

extern "C" {

size_t svdq_attention_plan_bytes(int total_q, int total_k, int batch, int heads_q, int heads_k, int head_dim) {
  const size_t full = plan_for(total_q, total_k, batch, heads_q, heads_k, head_dim, false).bytes;
  const size_t causal = plan_for(total_q, total_k, batch, heads_q, heads_k, head_dim, true).bytes;
  return full > causal ? full : causal;
}

void svdq_attention_plan(int total_q, int total_k, int batch, int heads_q, int heads_k, int head_dim, int causal, int32_t* plan) {
  const Plan p = plan_for(total_q, total_k, batch, heads_q, heads_k, head_dim, causal);
  plan[0] = p.waves ? p.waves * 32 : 32;
  plan[1] = p.parts;
  plan[2] = p.splits;
  plan[3] = p.spread;
}

int svdq_launch_attention(const void* q, const void* k, const void* v, void* o, float* lse, const int32_t* cu_q,
                          const int32_t* cu_k, int batch, int total_q, int total_k, int heads_q, int heads_k,
                          int head_dim, const int64_t* strides, float scale, int causal, int dtype, void* workspace,
                          size_t workspace_bytes, void* stream) {
  Plan p = plan_for(total_q, total_k, batch, heads_q, heads_k, head_dim, causal);
  if (!workspace || workspace_bytes < p.bytes) p.splits = 1, p.spread = 0;
  AttnArgs a{};
  a.q = static_cast<const uint16_t*>(q);
  a.k = static_cast<const uint16_t*>(k);
  a.v = static_cast<const uint16_t*>(v);
  a.o = static_cast<uint16_t*>(o);
  a.lse = lse;
  if (p.spread) {
    a.before = static_cast<int64_t*>(workspace);
    a.before_q = reinterpret_cast<int32_t*>(a.before + batch + 1);
    a.part_o = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + spread_head(batch));
    a.results = p.spread + (static_cast<int64_t>(total_q) * (heads_q / heads_k) / 32 + batch) * heads_k;
    a.part_ml = reinterpret_cast<float2*>(a.part_o + a.results * 32 * head_dim);
  }
  if (p.splits > 1) {
    a.part_o = static_cast<float*>(workspace);
    a.part_ml = reinterpret_cast<float2*>(a.part_o + static_cast<size_t>(p.splits) * total_q * heads_q * head_dim);
  }
  a.cu_q = cu_q;
  a.cu_k = cu_k;
  a.q_t = strides[0], a.q_h = strides[1], a.k_t = strides[2], a.k_h = strides[3];
  a.v_t = strides[4], a.v_h = strides[5], a.o_t = strides[6], a.o_h = strides[7];
  a.total_q = total_q;
  a.total_k = total_k;
  a.batch = batch;
  a.heads_q = heads_q;
  a.heads_k = heads_k;
  a.group = heads_q / heads_k;
  a.D = head_dim;
  a.scale = scale;
  a.causal = causal;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  return dtype == SVDQ_BF16 ? launch<Bf16>(a, p, s) : launch<F16>(a, p, s);
}

}  // extern "C"
