// Attention over the paged 8-bit cache:
//
//   s_ij = scale q_i . k_j,  k_j = 2^ek code,  o_i = sum_j softmax_j(s_ij) v_j,  v_j = 2^ev code
//   lse_i = log sum_j exp(s_ij);  causal: query i sees keys j <= i + length - tokens
//
// for gfx950.  Codes become 16-bit values of q's type as they are (exactly)
// and meet the matrix core there; a page's exponents go into the argument of
// the exponential:
//
//   t_ij = s_ij log2 e + ev,  p_ij = 2^(t_ij - m_i),  m_i the running maximum of t_ij
//   o_i = sum_j p_ij code_j / sum_j p_ij 2^-ev
//
// so that P, rounded to 16 bits, weighs codes of all pages alike.  With
// |ev| <= 40 the sums stay far inside fp32's range.
//
// A wave owns 16 RT rows (query heads that share a key head, packed with their
// tokens) and takes a page of 64 keys at a time, straight from memory into
// registers.  It computes S^T = K Q^T with 16 x 16 x 32 products, so that a lane
// holds scores of one row, and O^T = V^T P^T, whose operands are registers as
// they lie (svdq_cache.h).
//
// Measured, 32 / 8 heads of 128, bf16: one token of each of 8 caches (up to
// 16384 tokens, 120 MB) 31 us, of 64 caches (540 MB) 98, 5.5 TB/s: bound by
// reading the cache.  Chunks of 2048 tokens 256 us, 970 TFLOP/s: bound by the
// matrix core, the exponentials and the widening; the two kernels of most
// registers (heads past 64: many rows, and tiles of 32 few rows) also reload 68
// and 60 bytes a lane from scratch in their loops over pages.

#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include <type_traits>

#include "svdq_internal.h"
#include "svdq_cache.h"

namespace {

using namespace svdq_dev;

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// The running maximum before the first key: the least finite value, so that no
// finite score lies below it.
constexpr float kNothing = -3.402823466e38f;
constexpr int kCUs = 256;

struct PagedArgs {
  Sequences seq;
  const uint16_t* q;
  uint16_t* o;
  float* lse;
  const uint8_t *k_cache, *v_cache;
  const int8_t* exponents;
  float* part;                        // shares' parts, or null: a tile's keys are one workgroup's
  int64_t ldq, hdq, ldo, hdo;         // token and head strides
  int heads_q, heads_k, head_dim, group, causal, groups;
  float scale;                        // times log2 e
};

// Two of the 8-bit codes in a word as 16-bit values.
template <typename E>
__device__ __forceinline__ uint32_t widen(uint32_t codes, bool high);
template <>
__device__ __forceinline__ uint32_t widen<Bf16>(uint32_t codes, bool high) {
  return high ? __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes, 1.f, true))
              : __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes, 1.f, false));
}
template <>
__device__ __forceinline__ uint32_t widen<F16>(uint32_t codes, bool high) {
  return high ? __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(codes, 1.f, true))
              : __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(codes, 1.f, false));
}
template <typename E>
__device__ __forceinline__ v4u widen8(uint32_t lo, uint32_t hi) {
  return v4u{widen<E>(lo, false), widen<E>(lo, true), widen<E>(hi, false), widen<E>(hi, true)};
}

// A tile: the sequence's rows from row0 on, of one key head.
struct Tile {
  int b, h, row0;
  int tokens, length, start;   // the sequence's, its keys as far as the table holds them
  int before;                  // its keys before the first of the tokens, also those past the table; below 0 if there are more tokens
};

// Keys that row r of a tile sees.
__device__ __forceinline__ int visible(const PagedArgs& a, const Tile& t, int r) {
  const int row = t.row0 + r;
  if (row >= t.tokens * a.group) return 0;
  return a.causal ? max(0, min(t.length, t.before + row / a.group + 1)) : t.length;
}

// 16 codes that few workgroups read: past the caches' keeping (64 caches of
// 3000 to 5300 tokens 111 -> 99 us)
__device__ __forceinline__ v4u stream16(const uint8_t* p) { return __builtin_nontemporal_load(reinterpret_cast<const v4u*>(p)); }

// 16 RT rows against pages: DC chunks of 64 dimensions.
template <typename E, int DC, int RT>
struct Rows {
  v4u q[RT][DC][2];
  v4u k[4][DC], v[4 * DC];    // a page's codes as they lie
  int ek, ev;                 // its exponents
  v4f o[RT][4 * DC];
  float m[RT], l[RT];
  int sees[RT];               // keys that the lane's row sees
  int lane, l16, g;

  __device__ __forceinline__ void init(const PagedArgs& a, const Tile& t, int r0) {
    lane = threadIdx.x & 63;
    l16 = lane & 15;
    g = lane >> 4;
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      const int r = r0 + i * 16 + l16, row = t.row0 + r, token = row / a.group, head = t.h * a.group + row - token * a.group;
      sees[i] = visible(a, t, r);
      const bool in = row < t.tokens * a.group;
      const uint16_t* const p = a.q + (t.start + token) * a.ldq + head * a.hdq;
#pragma unroll
      for (int c = 0; c < DC; ++c)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int d = 64 * c + 16 * g + 8 * u;
          q[i][c][u] = in && d < a.head_dim ? load8(p + d) : v4u{0, 0, 0, 0};
        }
#pragma unroll
      for (int d = 0; d < 4 * DC; ++d) o[i][d] = v4f{0.f, 0.f, 0.f, 0.f};
      m[i] = kNothing;
      l[i] = 0.f;
    }
  }

  // The page's keys, and its exponents; and its values.
  __device__ __forceinline__ void fetch_keys(const PagedArgs& a, const Tile& t, int page) {
    const int D = a.head_dim;
    const int64_t slot = static_cast<int64_t>(max(page, 0)) * a.heads_k + t.h;
    const uint8_t* const p = a.k_cache + slot * kPage * D + l16 * D + 16 * g;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int c = 0; c < DC; ++c)
        k[i][c] = 64 * c + 16 * g < D ? stream16(p + i * 16 * D + 64 * c) : v4u{0, 0, 0, 0};
    ek = a.exponents[slot * 2];
    ev = a.exponents[slot * 2 + 1];
  }
  __device__ __forceinline__ void fetch_values(const PagedArgs& a, const Tile& t, int page) {
    const int D = a.head_dim;
    const int64_t slot = static_cast<int64_t>(max(page, 0)) * a.heads_k + t.h;
    const uint8_t* const p = a.v_cache + slot * kPage * D + (g * D + l16) * 16;
#pragma unroll
    for (int d = 0; d < 4 * DC; ++d)
      v[d] = d * 16 < D ? stream16(p + d * 256) : v4u{0, 0, 0, 0};
  }

  // Pages first, first + step, ... before last; up to key `all_see` every row
  // sees every key.  A page's keys are loaded over the last one's as soon as
  // those have been multiplied, and so are its values: one page is on its way
  // all the time.
  __device__ __forceinline__ void walk(const PagedArgs& a, const Tile& t, int first, int last, int step, int all_see) {
    if (first >= last) return;
    const int32_t* const table = a.seq.table + static_cast<int64_t>(t.b) * a.seq.width;
    // -1: a page that is not there
    auto page_at = [&](int i) {
      const int page = table[min(i, last - 1)];
      return page < a.seq.pages ? page : -1;
    };
    int id = page_at(first), next = page_at(first + step);
    fetch_keys(a, t, id);
    fetch_values(a, t, id);
    for (int at = first; at < last; at += step) {
      const float mul = a.scale * power2(clamp_exponent(ek)), add = static_cast<float>(clamp_exponent(ev));
      const float back = power2(-clamp_exponent(ev));
      v4f s[RT][4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int j = 0; j < RT; ++j) s[j][i] = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c = 0; c < DC; ++c)
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const v4u w = widen8<E>(k[i][c][2 * u], k[i][c][2 * u + 1]);
#pragma unroll
            for (int j = 0; j < RT; ++j) s[j][i] = E::mfma16(w, q[j][c][u], s[j][i]);
          }
      }
      // some keys lie past the sequence, or past what a row sees; a page that is not there has none
      const int key0 = at * kPage, length = id >= 0 ? t.length : 0;
      const bool cut = id < 0 || key0 + kPage > all_see;
      const bool more = at + step < last;
      id = next;
      if (more) {
        fetch_keys(a, t, id);
        next = page_at(at + 2 * step);
      }
      if (cut) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int at0 = key0 + 16 * i + 4 * g, left = length - at0;
#pragma unroll
          for (int j = 0; j < RT; ++j)
#pragma unroll
            for (int r = 0; r < 4; ++r)
              if (at0 + r >= min(sees[j], length)) s[j][i][r] = -INFINITY;
          // what lies past the sequence may hold anything, NaN too
          const uint32_t keep = left >= 4 ? 0xFFFFFFFFu : left <= 0 ? 0u : (1u << (8 * left)) - 1u;
#pragma unroll
          for (int d = 0; d < 4 * DC; ++d) v[d][i] &= keep;
        }
      }
      v4u w[RT][2];
#pragma unroll
      for (int j = 0; j < RT; ++j) {
        float top = kNothing;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            s[j][i][r] = s[j][i][r] * mul + add;
            top = fmaxf(top, s[j][i][r]);
          }
        top = fmaxf(top, __shfl_xor(top, 16));
        top = fmaxf(top, __shfl_xor(top, 32));
        if (__ballot(top > m[j])) {
          const float now = fmaxf(m[j], top), shrink = exp2_fast(m[j] - now);
          m[j] = now;
          l[j] *= shrink;
#pragma unroll
          for (int d = 0; d < 4 * DC; ++d) o[j][d] *= shrink;
        }
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            s[j][i][r] = exp2_fast(s[j][i][r] - m[j]);
            sum += s[j][i][r];
          }
        l[j] += sum * back;
#pragma unroll
        for (int u = 0; u < 2; ++u)
          w[j][u] = v4u{E::pack2(s[j][2 * u][0], s[j][2 * u][1]), E::pack2(s[j][2 * u][2], s[j][2 * u][3]),
                        E::pack2(s[j][2 * u + 1][0], s[j][2 * u + 1][1]), E::pack2(s[j][2 * u + 1][2], s[j][2 * u + 1][3])};
      }
#pragma unroll
      for (int d = 0; d < 4 * DC; ++d)
        if (d * 16 < a.head_dim)
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const v4u x = widen8<E>(v[d][2 * u], v[d][2 * u + 1]);
#pragma unroll
            for (int j = 0; j < RT; ++j) o[j][d] = E::mfma16(x, w[j][u], o[j][d]);
          }
      if (more) fetch_values(a, t, id);
    }
  }
};

// A row's 8 dimensions of the result, rounded.
template <typename E>
__device__ __forceinline__ void put(const PagedArgs& a, const Tile& t, int r, int d, const float (&f)[8]) {
  const int row = t.row0 + r, token = row / a.group, head = t.h * a.group + row - token * a.group;
  store8(a.o + (t.start + token) * a.ldo + head * a.hdo + d, pack8<E>(f), 8);
}
// Whether a row with the sum l saw a key.  One that saw none gets zeros, not
// its sums times zero: the values it weighed with zero may be NaN.
__device__ __forceinline__ bool saw(float l) { return l > 0.f || l != l; }
__device__ __forceinline__ float logarithm(float m, float l) { return saw(l) ? (m + log2f(l)) * kLn2 : -INFINITY; }
__device__ __forceinline__ void put_lse(const PagedArgs& a, const Tile& t, int r, float m, float l) {
  if (!a.lse) return;
  const int row = t.row0 + r, token = row / a.group, head = t.h * a.group + row - token * a.group;
  a.lse[static_cast<int64_t>(t.start + token) * a.heads_q + head] = logarithm(m, l);
}

// Queries of no sequence: zeros.
__device__ __forceinline__ void pad(const PagedArgs& a, int block, int blocks) {
  if (!a.seq.cu) return;
  const int lo = a.seq.start(0), hi = max(lo, a.seq.start(a.seq.batch));
  const int n = lo + a.seq.total - hi, chunks = a.head_dim / 8;
  for (int i = block; i < n; i += blocks) {
    const int64_t token = i < lo ? i : hi + i - lo;
    for (int e = threadIdx.x; e < a.heads_q * chunks; e += blockDim.x)
      store8(a.o + token * a.ldo + e / chunks * a.hdo + e % chunks * 8, v4u{0, 0, 0, 0}, 8);
    if (a.lse)
      for (int e = threadIdx.x; e < a.heads_q; e += blockDim.x) a.lse[token * a.heads_q + e] = -INFINITY;
  }
}

// ---------------------------------------------------------------------------
// Few rows a sequence.  All tiles of 16 RT rows lie one after the other on a
// line, each with its pages and a constant for its start; with shares every
// workgroup takes an equal part of it, whole tiles or pieces, whose parts a
// second kernel joins; without, one workgroup takes a tile.  A workgroup's
// four waves take a tile's pages in turn and join in LDS.
// ---------------------------------------------------------------------------

constexpr int kWaves = 4;
constexpr int kStart = 4;   // pages that the start of a tile costs as much as

struct Line {
  int rows, pages_too;   // rows of a tile; 0: a tile counts 1
  __device__ __forceinline__ int tiles(const PagedArgs& a, int b) const {
    return (a.seq.tokens(b) * a.group + rows - 1) / rows;
  }
  // a tile without keys still takes its place, for its zeros
  __device__ __forceinline__ int pages(const PagedArgs& a, int b) const {
    return max(1, (a.seq.length(b) + kPage - 1) / kPage);
  }
  __device__ __forceinline__ int units(const PagedArgs& a, int b) const {
    return tiles(a, b) * a.heads_k * (pages_too ? kStart + pages(a, b) : 1);
  }
  __device__ __forceinline__ int total(const PagedArgs& a) const {
    unsigned sum = 0;
    for (int b = threadIdx.x & 63; b < a.seq.batch; b += 64) sum = add_sat(sum, units(a, b));
#pragma unroll
    for (int o = 32; o; o >>= 1) sum = add_sat(sum, __shfl_xor(sum, o));
    return __builtin_amdgcn_readfirstlane(min(sum, 0x7FFFFFFFu));
  }
};

__device__ __forceinline__ Tile tile_at(const PagedArgs& a, int b, int x, int rows) {
  Tile t;
  t.b = b;
  t.h = x % a.heads_k;
  t.row0 = x / a.heads_k * rows;
  t.tokens = __builtin_amdgcn_readfirstlane(a.seq.tokens(b));
  t.length = __builtin_amdgcn_readfirstlane(a.seq.length(b));
  t.start = __builtin_amdgcn_readfirstlane(a.seq.start(b));
  t.before = __builtin_amdgcn_readfirstlane(max(a.seq.lengths[b], 0)) - t.tokens;
  return t;
}

// What the shares leave for the join: each workgroup's two parts (of a tile
// that began before its share, and of one that begins in it and goes on), O, m
// and l of a tile's rows, and a note on the latter tile.  (The 32 bytes of the
// note spare the join the search for its tile.)
struct Note {
  int parts;             // 0: none
  int rows, row0, h, start;   // the tile's rows, the first of them among its sequence's, key head, the sequence's first token
  int unused[3];
};
__host__ __device__ constexpr int part_floats(int rows, int D) { return rows * (D + 2); }
__device__ __forceinline__ Note* notes_of(const PagedArgs& a) { return reinterpret_cast<Note*>(a.part); }
__device__ __forceinline__ float* part_of(const PagedArgs& a, int group, int second, int rows) {
  return a.part + 8LL * a.groups + (2LL * group + second) * part_floats(rows, a.head_dim);
}

// LDS in which NW waves join their parts of 16 RT rows.
template <int DC, int RT, int NW>
struct Joined {
  float o[NW][16 * RT][64 * DC + 4];
  float stats[NW][16 * RT][2];   // m, l
};

// NW waves take pages first, first + 1, ... before last of a tile in turn and
// join: the result itself, or (part) a share's part of it.
template <typename E, int DC, int RT, int NW>
__device__ __forceinline__ void few_rows(const PagedArgs& a, const Tile& t, int first, int last, float* part, Joined<DC, RT, NW>& lds) {
  constexpr int kRows = 16 * RT;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), D = a.head_dim;
  const int rows = min(kRows, t.tokens * a.group - t.row0);
  Rows<E, DC, RT> r;
  r.init(a, t, 0);
  r.walk(a, t, first + wave, last, NW, visible(a, t, 0));
  // the waves' parts, joined in their order
#pragma unroll
  for (int i = 0; i < RT; ++i) {
    float l = r.l[i];
    l += __shfl_xor(l, 16);
    l += __shfl_xor(l, 32);
    const int row = i * 16 + r.l16;
    if (r.g == 0) {
      lds.stats[wave][row][0] = r.m[i];
      lds.stats[wave][row][1] = l;
    }
#pragma unroll
    for (int d = 0; d < 4 * DC; ++d) *reinterpret_cast<v4f*>(&lds.o[wave][row][d * 16 + 4 * r.g]) = r.o[i][d];
  }
  __syncthreads();
  for (int e = threadIdx.x; e < rows * (D / 8); e += NW * 64) {
    const int row = e / (D / 8), d = (e - row * (D / 8)) * 8;
    float top = lds.stats[0][row][0];
#pragma unroll
    for (int w = 1; w < NW; ++w) top = fmaxf(top, lds.stats[w][row][0]);
    float f[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f}, l = 0.f;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      const float s = exp2_fast(lds.stats[w][row][0] - top);
      l += s * lds.stats[w][row][1];
#pragma unroll
      for (int c = 0; c < 8; ++c) f[c] += s * lds.o[w][row][d + c];
    }
    if (!part) {
      const float inv = 1.f / l;
#pragma unroll
      for (int c = 0; c < 8; ++c) f[c] = saw(l) ? f[c] * inv : 0.f;
      put<E>(a, t, row, d, f);
      if (d == 0) put_lse(a, t, row, top, l);
    } else {
#pragma unroll
      for (int c = 0; c < 8; c += 4) *reinterpret_cast<v4f*>(part + row * D + d + c) = v4f{f[c], f[c + 1], f[c + 2], f[c + 3]};
      if (d == 0) {
        part[kRows * D + 2 * row] = top;
        part[kRows * D + 2 * row + 1] = l;
      }
    }
  }
  __syncthreads();
}

template <typename E, int DC, int RT>
__global__ __launch_bounds__(kWaves * 64, 2) void k_paged_few(PagedArgs a) {
  constexpr int kRows = 16 * RT;
  __shared__ __attribute__((aligned(16))) Joined<DC, RT, kWaves> lds;
  pad(a, blockIdx.x, gridDim.x);
  const bool shares = a.part != nullptr;
  const Line line{kRows, shares};
  int64_t at = blockIdx.x, end = at + 1;   // in units of the line
  int share = 1;
  if (shares) {
    const int total = line.total(a);
    share = max(2 * kStart, total / a.groups + (total % a.groups != 0));
    at *= share;
    end = min(at + share, static_cast<int64_t>(total));
    if (threadIdx.x == 0) notes_of(a)[blockIdx.x] = Note{};
    if (at >= end) return;
  }
  int b, in = static_cast<int>(at);   // the sequence, and the unit counted from its first
  if (!find(a.seq.batch, in, b, [&](int s) { return line.units(a, s); })) return;
  while (at < end) {
    const int units = line.units(a, b), pages = line.pages(a, b);
    if (in >= units) {
      in -= units;
      if (++b >= a.seq.batch) return;
      continue;
    }
    int x = in, first = 0, last = pages, step = 1;
    if (shares) {
      const int size = kStart + pages;
      x = in / size;
      const int from = in - x * size, to = static_cast<int>(min(static_cast<int64_t>(size), from + end - at));
      first = max(0, from - kStart);
      last = max(0, to - kStart);
      step = to - from;
    }
    if (first < last) {
      const Tile t = tile_at(a, b, x, kRows);
      const bool whole = first == 0 && last == pages;
      if (!whole && first == 0 && threadIdx.x == 0) {
        const int64_t after = (pages - last + static_cast<int64_t>(share) - 1) / share;   // shares that go on with it
        notes_of(a)[blockIdx.x] = Note{static_cast<int>(min<int64_t>(after, a.groups - 1 - blockIdx.x)) + 1,
                                       min(kRows, t.tokens * a.group - t.row0), t.row0, t.h, t.start};
      }
      few_rows<E, DC, RT, kWaves>(a, t, first, last, whole ? nullptr : part_of(a, blockIdx.x, first == 0, kRows), lds);
    }
    at += step;
    in += step;
  }
}

// The parts of a tile that shares cut, joined in their order: a workgroup for
// each that the note of a share names, a wave a row.  The first kAhead parts
// are loaded beside their statistics: a chain of two loads, as a part's way
// from another XCD's L2 takes 2 us.
template <typename E, int RT>
__global__ __launch_bounds__(256) void k_paged_join(PagedArgs a) {
  constexpr int kRows = 16 * RT, kAhead = 24;
  const int D = a.head_dim, lane = threadIdx.x & 63, g0 = blockIdx.x;
  const Note note = notes_of(a)[g0];
  const int parts = note.parts;
  auto part = [&](int i) { return part_of(a, g0 + i, i == 0, kRows); };
  const int d = min(2 * lane, D - 2);   // lanes past the row repeat its end
  for (int row = threadIdx.x >> 6; parts && row < note.rows; row += 4) {
    auto values = [&](int i) { return *reinterpret_cast<const v2f*>(part(i) + row * D + d); };
    v2f ahead[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) ahead[i] = values(min(i, parts - 1));
    float top = kNothing;
    for (int i = lane; i < parts; i += 64) top = fmaxf(top, part(i)[kRows * D + 2 * row]);
#pragma unroll
    for (int o = 32; o; o >>= 1) top = fmaxf(top, __shfl_xor(top, o));
    float f[2] = {0.f, 0.f}, l = 0.f;
    for (int i0 = 0; i0 < parts; i0 += 64) {
      float s = 0.f, sum = 0.f;
      if (i0 + lane < parts) {
        const float* const p = part(i0 + lane) + kRows * D + 2 * row;
        s = exp2_fast(p[0] - top);
        sum = s * p[1];
      }
      auto add = [&](int i, v2f v) {
        const float si = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(s), i));
        l += __int_as_float(__builtin_amdgcn_readlane(__float_as_int(sum), i));
        f[0] += si * v[0];
        f[1] += si * v[1];
      };
      const int n = min(64, parts - i0);
      if (i0 == 0) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
          if (i < n) add(i, ahead[i]);
      }
#pragma unroll 8
      for (int i = i0 ? 0 : kAhead; i < n; ++i) add(i, values(i0 + i));
    }
    const float inv = 1.f / l;
    const int all = note.row0 + row, token = all / a.group, head = note.h * a.group + all - token * a.group;
    if (2 * lane < D) {
      const uint32_t v = saw(l) ? E::pack2(f[0] * inv, f[1] * inv) : 0u;
      __builtin_memcpy(a.o + (note.start + token) * a.ldo + head * a.hdo + d, &v, 4);
    }
    if (lane == 0 && a.lse)
      a.lse[static_cast<int64_t>(note.start + token) * a.heads_q + head] = logarithm(top, l);
  }
}

// ---------------------------------------------------------------------------
// Many rows a sequence (chunks of prompts): NW waves of 32 rows share pages.
// Bound by the matrix core and the exponentials.  A page's codes are loaded
// into registers, widened once for all waves and put into LDS, from where they
// are the products' operands, of 32 x 32 x 16 here.
//
// Iteration i has two phases, in each of which matrix and vector work stand
// side by side in the instruction order:
//   A  S of page i + 1, beside most weights of page i
//   B  O += P V of page i, beside the last weights, the maxima of page i + 1,
//      and the widening of K of page i + 2 and V of page i + 1
// Operands are read from LDS kAhead products ahead; codes are loaded an
// iteration before they are widened.  Two buffers each for K and V, one
// barrier a page.  Past the last page the work goes on with what the buffers
// hold, and nothing of it is used: no branch parts the products from the
// vector work.  The running reference moves only when a row's maximum passes
// it by 2^8.
//
// K's rows in LDS are 128 DC bytes, 16-byte chunk c of row r at
// c ^ (r % (8 DC)); V lies as the lanes read it: 16 bytes for each of 16 keys,
// 32 dimensions and lane.  A thread widens half of such 16 bytes at a time: its
// 8-byte writes at a stride of 16 use half of the banks (17 % of the LDS
// cycles of a chunk are conflicts).
// ---------------------------------------------------------------------------

template <typename E, int DC, int NW>
__global__ __launch_bounds__(NW * 64, 2) void k_paged_many(PagedArgs a) {
  constexpr int kRows = NW * 32, kThreads = NW * 64, kDims = 64 * DC, kTile = kPage * kDims * 2;
  constexpr int kChunks = kPage * kDims / 16 / kThreads;   // of 16 codes, a thread's
  constexpr int kSteps = kDims / 16, kDt = kDims / 32, kProducts = 2 * kSteps, kAhead = 4, kWeights = 16, kLate = 4;
  constexpr float kSlack = 8.f, kFar = 0x1p20f;
  static_assert(kChunks >= 1 && kProducts == 4 * kDt, "work divides evenly");
  using Few = Joined<DC, 1, NW>;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[sizeof(Few) > 4 * kTile ? sizeof(Few) : 4 * kTile];   // K, K, V, V
  const int lane = threadIdx.x & 63, l32 = lane & 31, h = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int D = a.head_dim;
  pad(a, blockIdx.x, gridDim.x);
  const Line line{kRows, 0};
  int b, x = blockIdx.x;
  if (!find(a.seq.batch, x, b, [&](int s) { return line.units(a, s); })) return;
  // a sequence's last rows see the most keys: they come first
  x = line.tiles(a, b) * a.heads_k - 1 - x;
  const Tile t = tile_at(a, b, x, kRows);
  const int left = t.tokens * a.group - t.row0, r0 = wave * 32;
  if (left <= 32) {   // a wave's rows: the waves share its pages instead
    Tile part = t;
    for (; part.row0 < t.tokens * a.group; part.row0 += 16)
      few_rows<E, DC, 1, NW>(a, part, 0, line.pages(a, b), nullptr, *reinterpret_cast<Few*>(lds));
    return;
  }
  const int last = (visible(a, t, min(kRows, left) - 1) + kPage - 1) / kPage;   // pages that the tile's rows see
  const int every = visible(a, t, r0);                                          // keys that each of the wave's sees
  const bool idle = r0 >= left;

  // the lane's row
  const int r = r0 + l32, row = t.row0 + r, token = row / a.group, head = t.h * a.group + row - token * a.group;
  const bool valid = r < left;
  const int sees = visible(a, t, r);
  v4u q[kSteps];
#pragma unroll
  for (int st = 0; st < kSteps; ++st) {
    const int d = 16 * st + 8 * h;
    q[st] = valid && d < D ? load8(a.q + (t.start + token) * a.ldq + head * a.hdq + d) : v4u{0, 0, 0, 0};
  }
  v16f o[kDt];
#pragma unroll
  for (int d = 0; d < kDt; ++d)
#pragma unroll
    for (int e = 0; e < 16; ++e) o[d][e] = 0.f;
  float m = kNothing, l = 0.f;

  // Chunk e of a page's keys is row e / (D / 16), of its values group e / D
  // and dimension e % D.  Threads without one repeat the last and put it where
  // its own thread does.
  const uint32_t base = lds_addr(lds);
  uint32_t to_k[kChunks][2], to_v[kChunks];
  int group_v[kChunks], from[kChunks];
#pragma unroll
  for (int n = 0; n < kChunks; ++n) {
    const int e = min(static_cast<int>(threadIdx.x) + kThreads * n, 4 * D - 1), per = D / 16;
    const int kr = e / per, c = 2 * (e - kr * per), gv = e / D, d = e - gv * D;
    from[n] = e * 16;
    group_v[n] = gv;
    to_k[n][0] = base + kr * (2 * kDims) + ((c ^ (kr & (8 * DC - 1))) << 4);
    to_k[n][1] = base + kr * (2 * kDims) + (((c + 1) ^ (kr & (8 * DC - 1))) << 4);
    to_v[n] = base + 2 * kTile + (((d >> 5) * 64 + (gv & 1) * 32 + (d & 31)) << 4) + 8 * (gv >> 1);
  }
  // dimensions past D are zeros in every buffer, and stay it
  if (D < kDims) {
    for (int e = threadIdx.x; e < 4 * kTile / 16; e += kThreads) reinterpret_cast<v4u*>(lds)[e] = v4u{0, 0, 0, 0};
    __syncthreads();
  }
  const int32_t* const table = a.seq.table + static_cast<int64_t>(t.b) * a.seq.width;
  // the sequence's pages, 64 at a time, a lane each: asked for in order.  -1: a
  // page that is not there
  int ids = 0;
  auto page_at = [&](int i) {
    if ((i & 63) == 0) ids = table[min(i + lane, last - 1)];
    const int page = __builtin_amdgcn_readlane(ids, i & 63);
    return page < a.seq.pages ? page : -1;
  };
  auto slot_of = [&](int page) { return static_cast<int64_t>(max(page, 0)) * a.heads_k + t.h; };
  v4u raw_k[kChunks], raw_v[kChunks];
  auto fetch = [&](const uint8_t* cache, int page, v4u (&raw)[kChunks]) {
    const uint8_t* const p = cache + slot_of(page) * kPage * D;
#pragma unroll
    for (int n = 0; n < kChunks; ++n) raw[n] = *reinterpret_cast<const v4u*>(p + from[n]);
  };
  // what lies past the sequence may hold anything, NaN too
  auto clean = [&](int key0, int length) {
    if (key0 + kPage > length)
#pragma unroll
      for (int n = 0; n < kChunks; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int rest = length - key0 - 16 * i - 4 * group_v[n];
          raw_v[n][i] &= rest >= 4 ? 0xFFFFFFFFu : rest <= 0 ? 0u : (1u << (8 * rest)) - 1u;
        }
  };
  using Lds16 = __attribute__((address_space(3))) v4u*;
  using Lds8 = __attribute__((address_space(3))) v2u*;
  // piece i of 6 of what a thread widens of a chunk: 2 of keys, 4 of values
  constexpr int kPieces = 6 * kChunks;
  auto widen_piece = [&](int i, uint32_t off_k, uint32_t off_v) {
    const int n = i / 6, p = i % 6;
    if (p < 2) {
      *reinterpret_cast<Lds16>(to_k[n][p] + off_k) = widen8<E>(raw_k[n][2 * p], raw_k[n][2 * p + 1]);
    } else {
      const uint32_t c = raw_v[n][p - 2];
      *reinterpret_cast<Lds8>(to_v[n] + off_v + (p - 2) * kDt * 1024) = v2u{widen<E>(c, false), widen<E>(c, true)};
    }
  };
  const uint32_t rk = base + l32 * (2 * kDims), rv = base + 2 * kTile + lane * 16;
  auto read_k = [&](uint32_t off, int kt, int st) {
    return lds_read16(rk + off + kt * 32 * (2 * kDims) + (((2 * st + h) ^ (l32 & (8 * DC - 1))) << 4));
  };
  auto read_v = [&](uint32_t off, int ks, int d) { return lds_read16(rv + off + (ks * kDt + d) * 1024); };
  struct Exponents {
    int k, v;
  };
  auto exponents = [&](int page) {
    const int8_t* const e = a.exponents + slot_of(page) * 2;
    return Exponents{clamp_exponent(e[0]), clamp_exponent(e[1])};
  };
  auto mask = [&](v16f (&s)[2], int page, int at) {
    if (page >= 0 && (at + 1) * kPage <= every) return;
    const int rest = (page >= 0 ? sees : 0) - at * kPage - 4 * h;
#pragma unroll
    for (int kt = 0; kt < 2; ++kt)
#pragma unroll
      for (int e = 0; e < 16; ++e) s[kt][e] = kt * 32 + (e >> 2) * 8 + (e & 3) < rest ? s[kt][e] : -INFINITY;
  };
  auto pair_max = [](float v) {   // over the two lanes that hold a row's keys
    const auto p = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return fmaxf(__uint_as_float(p[0]), __uint_as_float(p[1]));
  };
  auto length_of = [&](int page) { return page >= 0 ? t.length : 0; };

  if (last > 0) {
    // pages at, at + 1, at + 2 of the iteration, and the exponents of the first two
    int id0 = page_at(0);
    int id1 = page_at(1);
    int id2 = page_at(2);
    Exponents x0 = exponents(id0), x1 = exponents(id1);
    fetch(a.k_cache, id0, raw_k);
    fetch(a.v_cache, id0, raw_v);
    clean(0, length_of(id0));
#pragma unroll
    for (int i = 0; i < kPieces; ++i) widen_piece(i, 0, 0);
    fetch(a.k_cache, id1, raw_k);
#pragma unroll
    for (int n = 0; n < kChunks; ++n)
#pragma unroll
      for (int p = 0; p < 2; ++p) widen_piece(6 * n + p, kTile, 0);
    fetch(a.k_cache, id2, raw_k);
    fetch(a.v_cache, id1, raw_v);
    lds_barrier();
    v16f s0[2], s1[2];
#pragma unroll
    for (int kt = 0; kt < 2; ++kt) {
#pragma unroll
      for (int e = 0; e < 16; ++e) s0[kt][e] = 0.f;
#pragma unroll
      for (int st = 0; st < kSteps; ++st) s0[kt] = E::mfma(read_k(0, kt, st), q[st], s0[kt]);
    }
    mask(s0, id0, 0);
    float top = s0[0][0];
#pragma unroll
    for (int kt = 0; kt < 2; ++kt)
#pragma unroll
      for (int e = 0; e < 16; ++e) top = fmaxf(top, s0[kt][e]);
    top = pair_max(top);
    lds_barrier();   // K of the first page is read out

    // page at's scores in s, whose maxima are in top; those of the next go to s_next
    auto iterate = [&](int at, v16f (&s)[2], v16f (&s_next)[2], auto odd) {
      constexpr uint32_t k_free = decltype(odd)::value ? kTile : 0, v_now = k_free;   // buffers of page at
      constexpr uint32_t k_next = kTile - k_free, v_free = k_next;
      float mul = a.scale * power2(x0.k);
      const float add = static_cast<float>(x0.v);
      top = __builtin_fmaf(top, mul, add);
      if (__ballot(top > m + kSlack)) {
        const float now = fmaxf(m, top), shrink = exp2_fast(m - now);
        m = now;
        l *= shrink;
#pragma unroll
        for (int d = 0; d < kDt; ++d) o[d] *= shrink;
      }
      clean((at + 1) * kPage, length_of(id1));
      // a weight is 2^(s mul + less) in one operation, whose product is not
      // rounded as the one in m was: far from 0 the two differ by more than an
      // exponential takes, and the scores are rounded like m first
      float less = add - m;
      if (__ballot(fabsf(m) > kFar)) {
#pragma unroll
        for (int kt = 0; kt < 2; ++kt)
#pragma unroll
          for (int e = 0; e < 16; ++e) s[kt][e] = __builtin_fmaf(s[kt][e], mul, add) - m;
        mul = 1.f;
        less = 0.f;
      }
      v4u p[4], f[kAhead];
      float sum[2] = {0.f, 0.f};
      // pairs of weights that go beside product j of n
      auto weigh = [&](int first, int count, int j, int n) {
#pragma unroll
        for (int i = first + j * count / n; i < first + (j + 1) * count / n; ++i) {
          const int kt = i >> 3, e = (i & 7) * 2;
          const float u = exp2_fast(__builtin_fmaf(s[kt][e], mul, less)), v = exp2_fast(__builtin_fmaf(s[kt][e + 1], mul, less));
          sum[0] += u;
          sum[1] += v;
          uint32_t pair = E::pack2(u, v);
          asm volatile("" : "+v"(pair), "+v"(sum[0]), "+v"(sum[1]));   // here, and not where it is used
          p[i >> 2][i & 3] = pair;
        }
      };
#pragma unroll
      for (int j = 0; j < kAhead; ++j) f[j] = read_k(k_next, j % 2, j / 2);
#pragma unroll
      for (int j = 0; j < kProducts; ++j) {
        if (j < 2) s_next[j] = v16f{};
        s_next[j % 2] = E::mfma(f[j % kAhead], q[j / 2], s_next[j % 2]);
        const int n = j + kAhead;
        f[j % kAhead] = n < kProducts ? read_k(k_next, n % 2, n / 2) : read_v(v_now, (n - kProducts) / kDt, (n - kProducts) % kDt);
        weigh(0, kWeights - kLate, j, kProducts);
        fence();
      }
      mask(s_next, id1, at + 1);
      float high = s_next[0][0];
      order();
#pragma unroll
      for (int j = 0; j < kProducts; ++j) {
        o[j % kDt] = E::mfma(f[j % kAhead], p[j / kDt], o[j % kDt]);
        if (j + kAhead < kProducts) f[j % kAhead] = read_v(v_now, (j + kAhead) / kDt, (j + kAhead) % kDt);
        // the last weights before the products that take them, then the maxima
        constexpr int kHalf = kProducts / 2, kE = 32 / kHalf;
        if (j < kHalf) {
          weigh(kWeights - kLate, kLate, j, kHalf);
        } else {
#pragma unroll
          for (int e = (j - kHalf) * kE; e < (j - kHalf + 1) * kE; ++e) high = fmaxf(high, s_next[e / 16][e % 16]);
        }
#pragma unroll
        for (int i = j * kPieces / kProducts; i < (j + 1) * kPieces / kProducts; ++i) widen_piece(i, k_free, v_free);
        fence();
      }
      l += (sum[0] + sum[1]) * power2(-x0.v);
      top = pair_max(high);
      id0 = id1;
      id1 = id2;
      id2 = page_at(at + 3);
      x0 = x1;
      x1 = exponents(id1);
      fetch(a.k_cache, id2, raw_k);
      fetch(a.v_cache, id1, raw_v);
      // this page's V and the next one's K are read out, what was widened is there; loads stay in flight
      lds_barrier();
    };
    if (idle) {   // rows past the sequence's: the wave widens, and waits for the others
      for (int at = 0; at < last; ++at) {
        clean((at + 1) * kPage, length_of(id1));
#pragma unroll
        for (int i = 0; i < kPieces; ++i) widen_piece(i, (at & 1) * kTile, ((at + 1) & 1) * kTile);
        id1 = id2;
        id2 = page_at(at + 3);
        fetch(a.k_cache, id2, raw_k);
        fetch(a.v_cache, id1, raw_v);
        lds_barrier();
      }
    } else {
      for (int at = 0; at < last; at += 2) {
        iterate(at, s0, s1, std::false_type{});
        if (at + 1 < last) iterate(at + 1, s1, s0, std::true_type{});
      }
    }
  }
  if (!valid) return;
  const auto both = __builtin_amdgcn_permlane32_swap(__float_as_uint(l), __float_as_uint(l), false, false);
  const float sum = __uint_as_float(both[0]) + __uint_as_float(both[1]);
  const float inv = 1.f / sum;
  const bool any = saw(sum);
  if (h == 0) put_lse(a, t, r, m, sum);
  uint16_t* const to = a.o + (t.start + token) * a.ldo + head * a.hdo + 4 * h;
#pragma unroll
  for (int d = 0; d < kDt; ++d)
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (d * 32 + 8 * j < D) {
        const v2u v = any ? v2u{E::pack2(o[d][4 * j] * inv, o[d][4 * j + 1] * inv), E::pack2(o[d][4 * j + 2] * inv, o[d][4 * j + 3] * inv)}
                          : v2u{0, 0};
        __builtin_memcpy(to + d * 32 + 8 * j, &v, 8);
      }
}

// Schedules, by sizes alone: rows of a tile, and workgroups that take equal
// shares (0: a workgroup takes a tile).
struct Plan {
  int rows, groups;
  size_t bytes;
};
// Up to 32 rows a sequence a tile has them all.  With more, tiles of many rows
// read a page once for all of them, but a tile's pages are one workgroup's:
// few such tiles leave most CUs idle, and equal shares of tiles of 32 rows are
// cheaper, though each tile reads the cache for itself.  Measured on both sides
// in us, tokens of 32 / 8 heads of 128 against 8000 keys:
//   tokens       8   64  128  256  512  768  1024  1536
//   shares      35   58   80  128  114  299   229     -
//   many rows  132  244  242  240  239  239   238   238
// The choice goes by an estimate for the table's width of keys: a page takes a
// tile of many rows 1.9 with one workgroup a CU, 2.2 with all of them at work,
// and a share of 32 rows 0.6.  The last is low: shares of whole tiles (512 and
// 1024 tokens) take 1.3 times the estimate, shares that cut the tiles up to 2.5
// times.  Of the sizes above the choice still is the faster side's but for 768
// tokens, which take shares.
Plan plan_for(int total, int batch, int width, int heads_q, int heads_k, int D) {
  const int64_t rows = static_cast<int64_t>(total) * (heads_q / heads_k);
  const int many = D > 64 ? 256 : 128;
  bool few = rows <= 32LL * batch;
  if (!few) {
    const double tiles_many = static_cast<double>(rows / many + batch) * heads_k / (many == 256 ? kCUs : 2 * kCUs);
    const double tiles_few = static_cast<double>(rows / 32 + batch) * heads_k / (2 * kCUs);
    few = tiles_few * (width + kStart) * 0.6 + 12. < (tiles_many < 1. ? 1.9 : 2.2 * tiles_many) * width;
  }
  Plan p{many, 0, 0};
  if (few) {
    p.rows = rows <= 16LL * batch ? 16 : 32;
    // up to 1024 keys a workgroup has them soon; past that every CU takes its share
    if (width > 16) {
      p.groups = 2 * kCUs;
      p.bytes = static_cast<size_t>(p.groups) * (sizeof(Note) + 2 * sizeof(float) * part_floats(p.rows, D));
    }
  }
  return p;
}

template <typename E, int DC>
void start(const PagedArgs& a, const Plan& p, hipStream_t stream) {
  const unsigned tiles = static_cast<unsigned>((static_cast<int64_t>(a.seq.total) * a.group / p.rows + a.seq.batch) * a.heads_k);
  const unsigned blocks = a.part ? a.groups : tiles;
  if (p.rows > 32)
    k_paged_many<E, DC, 4 * DC><<<tiles, 256 * DC, 0, stream>>>(a);
  else if (p.rows == 16)
    k_paged_few<E, DC, 1><<<blocks, kWaves * 64, 0, stream>>>(a);
  else
    k_paged_few<E, DC, 2><<<blocks, kWaves * 64, 0, stream>>>(a);
  if (!a.part) return;
  if (p.rows == 16)
    k_paged_join<E, 1><<<a.groups, 256, 0, stream>>>(a);
  else
    k_paged_join<E, 2><<<a.groups, 256, 0, stream>>>(a);
}

template <typename E>
void launch(const PagedArgs& a, const Plan& p, hipStream_t stream) {
  if (a.head_dim <= 64)
    start<E, 1>(a, p, stream);
  else
    start<E, 2>(a, p, stream);
}

}  // namespace

extern "C" {

size_t svdq_attention_paged_plan_bytes(int total, int batch, int width, int heads_q, int heads_k, int head_dim) {
  return plan_for(total, batch, width, heads_q, heads_k, head_dim).bytes;
}

void svdq_attention_paged_plan(int total, int batch, int width, int heads_q, int heads_k, int head_dim, int32_t* plan) {
  const Plan p = plan_for(total, batch, width, heads_q, heads_k, head_dim);
  plan[0] = p.rows;
  plan[1] = p.groups;
}

int svdq_launch_attention_paged(const void* q, void* o, float* lse, const int64_t* strides, const uint8_t* k_cache,
                                const uint8_t* v_cache, const int8_t* exponents, int pages, const int32_t* table, int width,
                                const int32_t* lengths, const int32_t* cu, int batch, int total, int heads_q, int heads_k,
                                int head_dim, float scale, int causal, int dtype, void* workspace, size_t workspace_bytes,
                                void* stream) {
  PagedArgs a{};
  a.seq = Sequences{cu, lengths, table, batch, total, width, pages};
  a.q = static_cast<const uint16_t*>(q);
  a.o = static_cast<uint16_t*>(o);
  a.lse = lse;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.exponents = exponents;
  a.ldq = strides[0];
  a.hdq = strides[1];
  a.ldo = strides[2];
  a.hdo = strides[3];
  a.heads_q = heads_q;
  a.heads_k = heads_k;
  a.head_dim = head_dim;
  a.group = heads_q / heads_k;
  a.causal = causal;
  a.scale = scale * kLog2e;
  const Plan p = plan_for(total, batch, width, heads_q, heads_k, head_dim);
  if (workspace && p.bytes && workspace_bytes >= p.bytes) {
    a.part = static_cast<float*>(workspace);
    a.groups = p.groups;
  }
  const hipStream_t s = static_cast<hipStream_t>(stream);
  if (dtype == SVDQ_BF16)
    launch<Bf16>(a, p, s);
  else
    launch<F16>(a, p, s);
  return static_cast<int>(hipGetLastError());
}

}  // extern "C"
