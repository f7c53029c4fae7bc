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

#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "svdq_internal.h"
#include "svdq_cache.h"

namespace {

using namespace svdq_dev;

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kNothing = -1e30f;    // the running maximum before the first key
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
  int tokens, length, start;   // the sequence's
};

// Keys that row r of a tile sees.
__device__ __forceinline__ int visible(const PagedArgs& a, const Tile& t, int r) {
  const int row = t.row0 + r;
  if (row >= t.tokens * a.group) return 0;
  return a.causal ? max(0, min(t.length, t.length - t.tokens + row / a.group + 1)) : t.length;
}

// 16 RT rows against pages: DC chunks of 64 dimensions.  Codes that no other
// workgroup reads bypass the caches' keeping (ONCE; 64 caches of 3000 to 5300
// tokens 111 -> 99 us).
template <bool ONCE>
__device__ __forceinline__ v4u codes16(const uint8_t* p) {
  const v4u* const v = reinterpret_cast<const v4u*>(p);
  return ONCE ? __builtin_nontemporal_load(v) : *v;
}
template <typename E, int DC, int RT, bool ONCE>
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
        k[i][c] = 64 * c + 16 * g < D ? codes16<ONCE>(p + i * 16 * D + 64 * c) : v4u{0, 0, 0, 0};
    ek = a.exponents[slot * 2];
    ev = a.exponents[slot * 2 + 1];
  }
  __device__ __forceinline__ void fetch_values(const PagedArgs& a, const Tile& t, int page) {
    const int D = a.head_dim;
    const int64_t slot = static_cast<int64_t>(max(page, 0)) * a.heads_k + t.h;
    const uint8_t* const p = a.v_cache + slot * kPage * D + (g * D + l16) * 16;
#pragma unroll
    for (int d = 0; d < 4 * DC; ++d)
      v[d] = d * 16 < D ? codes16<ONCE>(p + d * 256) : v4u{0, 0, 0, 0};
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
__device__ __forceinline__ float logarithm(float m, float l) { return l > 0.f || l != l ? (m + log2f(l)) * kLn2 : -INFINITY; }
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
  t.tokens = a.seq.tokens(b);
  t.length = a.seq.length(b);
  t.start = a.seq.start(b);
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

template <typename E, int DC, int RT>
__global__ __launch_bounds__(kWaves * 64, 2) void k_paged_few(PagedArgs a) {
  constexpr int kRows = 16 * RT, kD = 64 * DC, kLd = kD + 4;
  __shared__ __attribute__((aligned(16))) float out[kWaves][kRows][kLd];
  __shared__ float stats[kWaves][kRows][2];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int D = a.head_dim;
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
      const int rows = min(kRows, t.tokens * a.group - t.row0);
      Rows<E, DC, RT, true> r;
      r.init(a, t, 0);
      r.walk(a, t, first + wave, last, kWaves, visible(a, t, 0));
      // the waves' parts, joined in their order
#pragma unroll
      for (int i = 0; i < RT; ++i) {
        float l = r.l[i];
        l += __shfl_xor(l, 16);
        l += __shfl_xor(l, 32);
        const int row = i * 16 + r.l16;
        if (r.g == 0) {
          stats[wave][row][0] = r.m[i];
          stats[wave][row][1] = l;
        }
#pragma unroll
        for (int d = 0; d < 4 * DC; ++d) *reinterpret_cast<v4f*>(&out[wave][row][d * 16 + 4 * r.g]) = r.o[i][d];
      }
      __syncthreads();
      const bool whole = first == 0 && last == pages;
      float* const part = shares ? part_of(a, blockIdx.x, first == 0, kRows) : nullptr;
      if (!whole && first == 0 && threadIdx.x == 0) {
        const int64_t after = (pages - last + static_cast<int64_t>(share) - 1) / share;   // shares that go on with it
        notes_of(a)[blockIdx.x] = Note{static_cast<int>(min<int64_t>(after, a.groups - 1 - blockIdx.x)) + 1, rows, t.row0, t.h, t.start};
      }
      for (int e = threadIdx.x; e < rows * (D / 8); e += kWaves * 64) {
        const int row = e / (D / 8), d = (e - row * (D / 8)) * 8;
        float top = stats[0][row][0];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) top = fmaxf(top, stats[w][row][0]);
        float f[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f}, l = 0.f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
          const float s = exp2_fast(stats[w][row][0] - top);
          l += s * stats[w][row][1];
#pragma unroll
          for (int c = 0; c < 8; ++c) f[c] += s * out[w][row][d + c];
        }
        if (whole) {
          const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
#pragma unroll
          for (int c = 0; c < 8; ++c) f[c] *= inv;
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
      int i = 0;
      if (i0 == 0) {
#pragma unroll
        for (; i < kAhead; ++i)
          if (i < n) add(i, ahead[i]);
      }
#pragma unroll 8
      for (; i < n; ++i) add(i, values(i0 + i));
    }
    const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
    const int all = note.row0 + row, token = all / a.group, head = note.h * a.group + all - token * a.group;
    if (2 * lane < D) {
      const uint32_t v = E::pack2(f[0] * inv, f[1] * inv);
      __builtin_memcpy(a.o + (note.start + token) * a.ldo + head * a.hdo + d, &v, 4);
    }
    if (lane == 0 && a.lse)
      a.lse[static_cast<int64_t>(note.start + token) * a.heads_q + head] = logarithm(top, l);
  }
}

// ---------------------------------------------------------------------------
// Many rows a sequence (chunks of prompts): 32 rows a wave, 128 a workgroup,
// each wave through all pages that its rows see.
// ---------------------------------------------------------------------------

template <typename E, int DC>
__global__ __launch_bounds__(256, 2) void k_paged_many(PagedArgs a) {
  constexpr int RT = 2, kRows = 128;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  pad(a, blockIdx.x, gridDim.x);
  const Line line{kRows, 0};
  int b, x = blockIdx.x;
  if (!find(a.seq.batch, x, b, [&](int s) { return line.units(a, s); })) return;
  const Tile t = tile_at(a, b, x, kRows);
  const int left = t.tokens * a.group - t.row0, r0 = wave * 32;
  if (r0 >= left) return;
  Rows<E, DC, RT, false> r;
  r.init(a, t, r0);
  const int most = visible(a, t, min(r0 + 31, left - 1));
  r.walk(a, t, 0, (most + kPage - 1) / kPage, 1, visible(a, t, r0));
#pragma unroll
  for (int i = 0; i < RT; ++i) {
    float l = r.l[i];
    l += __shfl_xor(l, 16);
    l += __shfl_xor(l, 32);
    const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
    const int row = r0 + i * 16 + r.l16;
    if (row >= left) continue;
    if (r.g == 0) put_lse(a, t, row, r.m[i], l);
    const int all = t.row0 + row, token = all / a.group, head = t.h * a.group + all - token * a.group;
    uint16_t* const o = a.o + (t.start + token) * a.ldo + head * a.hdo + 4 * r.g;
#pragma unroll
    for (int d = 0; d < 4 * DC; ++d)
      if (d * 16 < a.head_dim) {
        const v2u v = {E::pack2(r.o[i][d][0] * inv, r.o[i][d][1] * inv), E::pack2(r.o[i][d][2] * inv, r.o[i][d][3] * inv)};
        __builtin_memcpy(o + d * 16, &v, 8);
      }
  }
}

// Schedules, by sizes alone: rows of a tile, and workgroups that take equal
// shares (0: a workgroup takes a tile).
struct Plan {
  int rows, groups;
  size_t bytes;
};
Plan plan_for(int total, int batch, int width, int heads_q, int heads_k, int D) {
  const int64_t rows = static_cast<int64_t>(total) * (heads_q / heads_k);
  Plan p{128, 0, 0};
  if (rows <= 32LL * batch) {
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
  if (p.rows == 128)
    k_paged_many<E, DC><<<tiles, 256, 0, stream>>>(a);
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
