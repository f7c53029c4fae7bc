// The cache of keys and values in 8 bits: its layout, and where a sequence
// stands.  gfx950 only.
//
//   keys       [pages][heads][64 tokens][D] e4m3 codes
//   values     [pages][heads][4][D][16]: place p of a page is at [p / 4 % 4][d][4 (p / 16) + p % 4]
//   exponents  [pages][heads][2] int8, of keys and values: value = code * 2^exponent
//
// Values lie so that the 16 bytes of (g, d) are the keys that a lane of group
// g holds after the product K Q^T of four 16 x 16 tiles: the lane that reads
// them feeds P V without a transposition.  A page is what one wave multiplies
// at a time.  Powers of two lose nothing in e4m3 but its subnormals, and let a
// page's scale grow, as later tokens ask for it, by an exact rescaling.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "svdq_device.h"

namespace svdq_dev {

constexpr int kPage = SVDQ_PAGE;
constexpr int kLowExponent = -40, kHighExponent = 40;

// Where the sequences stand.  Whatever the arrays hold, what comes out of here
// lies inside q's tokens and the table.
struct Sequences {
  const int32_t *cu, *lengths, *table;   // cu null: one token each
  int batch, total, width, pages;

  __device__ __forceinline__ int start(int b) const { return cu ? min(max(cu[b], 0), total) : b; }
  __device__ __forceinline__ int tokens(int b) const { return cu ? max(0, min(cu[b + 1], total) - start(b)) : 1; }
  __device__ __forceinline__ int length(int b) const { return min(max(lengths[b], 0), width * kPage); }
};

__device__ __forceinline__ int clamp_exponent(int e) { return min(max(e, kLowExponent), kHighExponent); }
// 2^e for |e| <= 126
__device__ __forceinline__ float power2(int e) { return __int_as_float((e + 127) << 23); }

// a + b, at most 2^32 - 1: starts that overlap can count more than there is
__device__ __forceinline__ unsigned add_sat(unsigned a, unsigned b) { return __builtin_elementwise_add_sat(a, b); }

// The sequence of job i, where sequence b takes count(b) jobs, and i counted
// from its first (below count(b), whatever the counts); false past the last.
// Every wave searches for itself, 64 sequences at a time.
template <typename F>
__device__ __forceinline__ bool find(int batch, int& i, int& b, F count) {
  const int lane = threadIdx.x & 63;
  for (int b0 = 0; b0 < batch; b0 += 64) {
    unsigned upto = b0 + lane < batch ? count(b0 + lane) : 0;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const unsigned below = __shfl_up(upto, o);
      if (lane >= o) upto = add_sat(upto, below);
    }
    const uint64_t past = __ballot(upto > static_cast<unsigned>(i));
    if (past) {
      const int l = __builtin_ctzll(past);
      const unsigned before = l ? __shfl(upto, l - 1) : 0;
      b = __builtin_amdgcn_readfirstlane(b0 + l);
      i = __builtin_amdgcn_readfirstlane(i - static_cast<int>(before));
      return true;
    }
    i -= static_cast<int>(__shfl(upto, 63));
  }
  return false;
}

}  // namespace svdq_dev
