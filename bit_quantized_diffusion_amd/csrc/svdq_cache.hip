// New tokens into the paged 8-bit cache, with the rotation by position:
//
//   (a, b) -> (a cos - b sin, b cos + a sin) for the pairs of the first
//   `rotary` values of each head of q and k, the angles' row by position
//
// and for each touched page and head of k and v
//
//   e = max(e of what the page holds, least e with amax <= 448 * 2^e),
//   code = e4m3(x 2^-e); what the page held is rescaled if e grew.
//
// for gfx950.  Bound by reading q, k and v and writing q and the codes.  One
// workgroup owns a page of one head: a thread holds four consecutive places of
// 8 dimensions, whose bytes are whole rows of 8 of the keys and whole words of
// the values, so that no byte has two writers.  Other workgroups take a
// token's query heads each.
//
// Measured: a token of each of 64 sequences, 32 / 8 heads of 128, 8.2 us a
// call, the host's time for it, and 8.6 in a HIP graph of such calls: a chain of
// loads (starts and lengths, the table, the rows, the exponents, the values'
// words) that each wait for the one before.  Loading ahead costs prompts 4 %; what
// it gives a token inside a graph was not measured.  Prompts of 141 MB in all
// 28.8 us by itself, 4.9 TB/s, the rate of a copy.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "svdq_internal.h"
#include "svdq_cache.h"

namespace {

using namespace svdq_dev;

struct AppendArgs {
  Sequences seq;
  const uint16_t *q, *k, *v;
  uint16_t* q_out;
  uint8_t *k_cache, *v_cache;
  int8_t* exponents;
  const float* rope;                    // [rope_rows][rotary]: cosines, then sines; or null
  int64_t ldq, hdq, ldk, hdk, ldv, hdv, ldo, hdo;   // token and head strides
  int heads_q, heads_k, head_dim, rope_rows, rotary, interleaved, jobs;
};

// Cosines and sines of the pairs of a chunk of 8 dimensions at d < rotary:
// half-split 8 of each, interleaved 4.
struct Angles {
  float c[8], s[8];
};
__device__ __forceinline__ void angles(const AppendArgs& a, int position, int d, Angles& t) {
  const int half = a.rotary / 2;
  const float* const row = a.rope + static_cast<int64_t>(min(max(position, 0), a.rope_rows - 1)) * a.rotary;
  const int n = a.interleaved ? 4 : 8, i = a.interleaved ? d / 2 : d < half ? d : d - half;
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (e < n) {
      t.c[e] = row[i + e];
      t.s[e] = row[half + i + e];
    }
}
__device__ __forceinline__ void rotate_pairs(const Angles& t, float (&f)[8]) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float x = f[2 * e], y = f[2 * e + 1];
    f[2 * e] = x * t.c[e] - y * t.s[e];
    f[2 * e + 1] = y * t.c[e] + x * t.s[e];
  }
}

// The query heads of one token.  A thread takes both halves of its pairs, so
// that q_out may be q.
template <typename E>
__device__ __forceinline__ void rotate_q(const AppendArgs& a, int token) {
  const int D = a.head_dim, half = a.rotary / 2;
  int position = 0;
  bool in = true;
  if (!a.seq.cu) {
    position = max(0, a.seq.lengths[token]) - 1;
  } else {
    // sequences whose end lies at or before the token
    int b = 0;
    for (int b0 = 0; b0 < a.seq.batch; b0 += 64) {
      const int i = b0 + (threadIdx.x & 63);
      b += __popcll(__ballot(i < a.seq.batch && a.seq.cu[i + 1] <= token));
    }
    in = b < a.seq.batch && token >= a.seq.cu[0];
    if (in) position = max(0, a.seq.lengths[b]) - a.seq.cu[b + 1] + token;
  }
  const int split = a.interleaved || !in ? 0 : half / 8;      // items that are two chunks each
  const int items = D / 8 - split;
  for (int i = threadIdx.x; i < a.heads_q * items; i += blockDim.x) {
    const int head = i / items, at = i - head * items;
    const uint16_t* const src = a.q + token * a.ldq + head * a.hdq;
    uint16_t* const dst = a.q_out + token * a.ldo + head * a.hdo;
    const int d = (at < split ? at : at + split) * 8;
    float f[8];
    unpack8<E>(load8(src + d), f);
    Angles t;
    if (at < split) {
      float g[8];
      unpack8<E>(load8(src + d + half), g);
      angles(a, position, d, t);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float x = f[e], y = g[e];
        f[e] = x * t.c[e] - y * t.s[e];
        g[e] = y * t.c[e] + x * t.s[e];
      }
      store8(dst + d + half, pack8<E>(g), 8);
    } else if (in && a.interleaved && d < a.rotary) {
      angles(a, position, d, t);
      rotate_pairs(t, f);
    }
    store8(dst + d, pack8<E>(f), 8);
  }
}

// finite magnitudes take part in a page's scale
__device__ __forceinline__ float finite_magnitude(float x) {
  const float a = fabsf(x);
  return a <= 3.402823466e38f ? a : 0.f;
}
// the least e with top <= 448 * 2^e = 1.75 * 2^(8 + e)
__device__ __forceinline__ int exponent_for(float top) {
  const int bits = __float_as_int(top);
  return clamp_exponent((bits >> 23) - 127 - 8 + ((bits & 0x7FFFFF) > 0x600000));
}
// what is not finite becomes NaN, what passes 448 becomes 448
__device__ __forceinline__ float to_code(float x, float shrink) {
  const float y = x * shrink;
  return fabsf(x) <= 3.402823466e38f ? fminf(fmaxf(y, -kMostF8), kMostF8) : __int_as_float(0x7FC00000);
}
__device__ __forceinline__ uint32_t rescale4(uint32_t codes, float shrink) {
  const v2f lo = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(codes), false);
  const v2f hi = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(codes), true);
  return pack4_f8(lo[0] * shrink, lo[1] * shrink, hi[0] * shrink, hi[1] * shrink);
}

template <typename E>
__global__ __launch_bounds__(256) void k_cache_append(AppendArgs a) {
  if (static_cast<int>(blockIdx.x) >= a.jobs * a.heads_k) {
    rotate_q<E>(a, blockIdx.x - a.jobs * a.heads_k);
    return;
  }
  __shared__ float tops[2][4];
  const int h = blockIdx.x % a.heads_k, D = a.head_dim, chunks = D / 8;
  int job = blockIdx.x / a.heads_k, b = job;
  auto range = [&](int s, int& from, int& to) {   // positions of the new tokens of sequence s that the table holds
    to = a.seq.length(s);
    from = max(0, max(0, a.seq.lengths[s]) - a.seq.tokens(s));
  };
  if (a.seq.cu) {
    if (!find(a.seq.batch, job, b, [&](int s) {
          int from, to;
          range(s, from, to);
          return from < to ? (to - 1) / kPage - from / kPage + 1 : 0;
        }))
      return;
  } else {
    job = 0;
  }
  int from, to;
  range(b, from, to);
  if (from >= to) return;
  const int p = from / kPage + job, first = max(from - p * kPage, 0), last = min(to - p * kPage, kPage);
  const int page = a.seq.table[static_cast<int64_t>(b) * a.seq.width + p];
  if (page < 0 || page >= a.seq.pages) return;
  // token of place 0
  const int64_t token0 = static_cast<int64_t>(a.seq.start(b)) + a.seq.tokens(b) - a.seq.lengths[b] + p * kPage;

  // four threads that stand beside each other in steps of `chunks` fill the 16 bytes of a group's values
  const int j = threadIdx.x / chunks, d = (threadIdx.x - j * chunks) * 8;
  const int g = j >> 2, t = j & 3, place = 16 * t + 4 * g;
  const bool mine = j < 16;
  float k[4][8], v[4][8];
  float top_k = 0.f, top_v = 0.f;
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const bool live = mine && place + r >= first && place + r < last;
    v4u raw_k = {0, 0, 0, 0}, raw_v = {0, 0, 0, 0};
    const uint16_t* const row = a.k + (token0 + place + r) * a.ldk + h * a.hdk;
    if (live) {
      raw_k = load8(row + d);
      raw_v = load8(a.v + (token0 + place + r) * a.ldv + h * a.hdv + d);
    }
    unpack8<E>(raw_k, k[r]);
    unpack8<E>(raw_v, v[r]);
    if (live && d < a.rotary) {
      Angles w;
      angles(a, p * kPage + place + r, d, w);
      if (a.interleaved) {
        rotate_pairs(w, k[r]);
      } else {
        const int half = a.rotary / 2;
        float other[8];
        unpack8<E>(load8(row + (d < half ? d + half : d - half)), other);
#pragma unroll
        for (int e = 0; e < 8; ++e) k[r][e] = k[r][e] * w.c[e] + (d < half ? -other[e] : other[e]) * w.s[e];
      }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      top_k = fmaxf(top_k, finite_magnitude(k[r][e]));
      top_v = fmaxf(top_v, finite_magnitude(v[r][e]));
    }
  }
#pragma unroll
  for (int o = 32; o; o >>= 1) {
    top_k = fmaxf(top_k, __shfl_xor(top_k, o));
    top_v = fmaxf(top_v, __shfl_xor(top_v, o));
  }
  if ((threadIdx.x & 63) == 0) {
    tops[0][threadIdx.x >> 6] = top_k;
    tops[1][threadIdx.x >> 6] = top_v;
  }
  __syncthreads();
  for (unsigned w = 0; w < blockDim.x / 64; ++w) {
    top_k = fmaxf(top_k, tops[0][w]);
    top_v = fmaxf(top_v, tops[1][w]);
  }
  const int64_t slot = static_cast<int64_t>(page) * a.heads_k + h;
  int8_t* const held = a.exponents + slot * 2;
  // what a page that starts here held is of no account
  const int was_k = first ? clamp_exponent(held[0]) : kLowExponent, was_v = first ? clamp_exponent(held[1]) : kLowExponent;
  const int e_k = max(was_k, exponent_for(top_k)), e_v = max(was_v, exponent_for(top_v));
  __syncthreads();   // read by all before it is written
  if (threadIdx.x == 0) {
    held[0] = static_cast<int8_t>(e_k);
    held[1] = static_cast<int8_t>(e_v);
  }
  if (!mine) return;
  const bool grew_k = first && e_k > was_k, grew_v = first && e_v > was_v;

  uint8_t* const keys = a.k_cache + (slot * kPage + place) * D + d;
  const float to_k = power2(-e_k), old_k = power2(was_k - e_k);
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    v2u* const at = reinterpret_cast<v2u*>(keys + r * D);
    if (place + r >= first && place + r < last) {
      const float(&f)[8] = k[r];
      *at = v2u{pack4_f8(to_code(f[0], to_k), to_code(f[1], to_k), to_code(f[2], to_k), to_code(f[3], to_k)),
                pack4_f8(to_code(f[4], to_k), to_code(f[5], to_k), to_code(f[6], to_k), to_code(f[7], to_k))};
    } else if (grew_k && place + r < first) {
      const v2u c = *at;
      *at = v2u{rescale4(c[0], old_k), rescale4(c[1], old_k)};
    }
  }
  // of the word of (place / 4, d): the bytes that are new, and those that are rescaled
  uint32_t fresh = 0, kept = 0;
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    if (place + r >= first && place + r < last) fresh |= 0xFFu << (8 * r);
    if (grew_v && place + r < first) kept |= 0xFFu << (8 * r);
  }
  if (!(fresh | kept)) return;
  uint32_t* const values = reinterpret_cast<uint32_t*>(a.v_cache + ((slot * 4 + g) * D + d) * 16) + t;
  uint32_t old[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  if (fresh != 0xFFFFFFFFu)
#pragma unroll
    for (int e = 0; e < 8; ++e) old[e] = values[4 * e];
  const float to_v = power2(-e_v), old_v = power2(was_v - e_v);
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const uint32_t c = pack4_f8(to_code(v[0][e], to_v), to_code(v[1][e], to_v), to_code(v[2][e], to_v), to_code(v[3][e], to_v));
    values[4 * e] = (c & fresh) | (rescale4(old[e], old_v) & kept) | (old[e] & ~(fresh | kept));
  }
}

}  // namespace

extern "C" int svdq_launch_cache_append(const void* q, const void* k, const void* v, void* q_out, const int64_t* strides,
                                        uint8_t* k_cache, uint8_t* v_cache, int8_t* exponents, int pages,
                                        const int32_t* table, int width, const int32_t* lengths, const int32_t* cu, int batch,
                                        int total, int heads_q, int heads_k, int head_dim, const float* rope, int rope_rows,
                                        int rotary, int interleaved, int dtype, void* stream) {
  AppendArgs a{};
  a.seq = Sequences{cu, lengths, table, batch, total, width, pages};
  a.q = static_cast<const uint16_t*>(q);
  a.k = static_cast<const uint16_t*>(k);
  a.v = static_cast<const uint16_t*>(v);
  a.q_out = static_cast<uint16_t*>(q_out);
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.exponents = exponents;
  a.rope = rope;
  a.ldq = strides[0];
  a.hdq = strides[1];
  a.ldk = strides[2];
  a.hdk = strides[3];
  a.ldv = strides[4];
  a.hdv = strides[5];
  a.ldo = strides[6];
  a.hdo = strides[7];
  a.heads_q = heads_q;
  a.heads_k = heads_k;
  a.head_dim = head_dim;
  a.rope_rows = rope_rows;
  a.rotary = rope ? rotary : 0;
  a.interleaved = interleaved;
  // touched pages: n tokens lie in at most (n + 62) / 64 + 1, and each page has one at least
  const int64_t most = static_cast<int64_t>(total) / kPage + 2 * static_cast<int64_t>(batch);
  a.jobs = static_cast<int>(cu && most < total ? most : total);
  const unsigned blocks = static_cast<unsigned>(a.jobs) * heads_k + (q ? total : 0);
  const unsigned threads = (2 * head_dim + 63) / 64 * 64;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  if (dtype == SVDQ_BF16)
    k_cache_append<Bf16><<<blocks, threads, 0, s>>>(a);
  else
    k_cache_append<F16><<<blocks, threads, 0, s>>>(a);
  return static_cast<int>(hipGetLastError());
}
