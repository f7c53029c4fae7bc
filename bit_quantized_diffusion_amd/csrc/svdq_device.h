// Device helpers shared by the 16-bit operators (attention, linear16, norms)
// and the 8-bit ones: element types, buffer descriptors, loads that go
// straight to LDS, waits.  gfx950 only.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace svdq_dev {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef unsigned v4u __attribute__((ext_vector_type(4)));
typedef unsigned v2u __attribute__((ext_vector_type(2)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef float v2f __attribute__((ext_vector_type(2)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef float v16f __attribute__((ext_vector_type(16)));
typedef int v8i __attribute__((ext_vector_type(8)));
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef _Float16 v2h __attribute__((ext_vector_type(2)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));

typedef __attribute__((address_space(3))) void* lds_ptr_t;

// The two 16-bit element types.  pack2 rounds two fp32 values to nearest
// even; mfma is the 32x32x16 product with fp32 accumulation,
//   A  lane l: row l % 32, k = 8 (l / 32) .. + 7
//   B  lane l: column l % 32, the same k
//   D  lane l, element 4 j + r: row 8 j + 4 (l / 32) + r, column l % 32,
// mfma16 the 16x16x32 one:
//   A  lane l: row l % 16, k = 8 (l / 16) .. + 7
//   B  lane l: column l % 16, the same k
//   D  lane l, element r: row 4 (l / 16) + r, column l % 16.
struct Bf16 {
  static __device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((v2f{lo, hi}), v2bf));
  }
  static __device__ __forceinline__ float lo(uint32_t u) { return __uint_as_float(u << 16); }
  static __device__ __forceinline__ float hi(uint32_t u) { return __uint_as_float(u & 0xFFFF0000u); }
  static __device__ __forceinline__ v16f mfma(v4u a, v4u b, v16f c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(v8bf, a), __builtin_bit_cast(v8bf, b), c, 0, 0, 0);
  }
  static __device__ __forceinline__ v4f mfma16(v4u a, v4u b, v4f c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, a), __builtin_bit_cast(v8bf, b), c, 0, 0, 0);
  }
};
struct F16 {
  static __device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((v2f{lo, hi}), v2h));
  }
  static __device__ __forceinline__ float lo(uint32_t u) {
    return static_cast<float>(__builtin_bit_cast(_Float16, static_cast<uint16_t>(u)));
  }
  static __device__ __forceinline__ float hi(uint32_t u) {
    return static_cast<float>(__builtin_bit_cast(_Float16, static_cast<uint16_t>(u >> 16)));
  }
  static __device__ __forceinline__ v16f mfma(v4u a, v4u b, v16f c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(v8h, a), __builtin_bit_cast(v8h, b), c, 0, 0, 0);
  }
  static __device__ __forceinline__ v4f mfma16(v4u a, v4u b, v4f c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, a), __builtin_bit_cast(v8h, b), c, 0, 0, 0);
  }
};

// Buffer descriptor of `bytes` bytes at base (at most 2^31 - 1): loads past
// the end return zeros, also those that go to LDS.  kOutside is an offset
// that lies past the end of every such buffer.
constexpr int kOutside = static_cast<int>(0x80000000u);
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const void* base, int64_t bytes) {
  const int n = bytes <= 0 ? 0 : bytes > 0x7FFFFFFF ? 0x7FFFFFFF : static_cast<int>(bytes);
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), static_cast<short>(0), n, 0x00020000);
}

__device__ __forceinline__ uint32_t lds_addr(const void* p) {
  return static_cast<uint32_t>(reinterpret_cast<uintptr_t>((lds_ptr_t)p));
}

// buffer_load ... lds as inline asm: 16 bytes per lane land at lds + 16 lane.
// The compiler neither counts nor waits for these loads; the kernel orders
// them itself (vm_wait, lds_wait_barrier).
__device__ __forceinline__ void dma_b128(__amdgpu_buffer_rsrc_t r, uint32_t lds, int voff) {
  asm volatile("s_nop 0\n\tbuffer_load_dwordx4 %0, %1, 0 offen lds"
               :: "v"(voff), "s"(r), "{m0}"(__builtin_amdgcn_readfirstlane(lds)) : "memory");
}

// the same with a wave-uniform offset added to voff
__device__ __forceinline__ void dma_b128(__amdgpu_buffer_rsrc_t r, uint32_t lds, int voff, int soff) {
  asm volatile("s_nop 0\n\tbuffer_load_dwordx4 %0, %1, %2 offen lds"
               :: "v"(voff), "s"(r), "s"(soff), "{m0}"(__builtin_amdgcn_readfirstlane(lds)) : "memory");
}

// 4 bytes per lane, to lds + 4 lane
__device__ __forceinline__ void dma_b32(__amdgpu_buffer_rsrc_t r, uint32_t lds, int voff) {
  asm volatile("s_nop 0\n\tbuffer_load_dword %0, %1, 0 offen lds"
               :: "v"(voff), "s"(r), "{m0}"(__builtin_amdgcn_readfirstlane(lds)) : "memory");
}

// at most N of the wave's vector-memory loads outstanding
template <int N>
__device__ __forceinline__ void vm_wait() {
  static_assert(N >= 0 && N < 64, "vmcnt field");
  asm volatile("s_waitcnt vmcnt(%0)" :: "n"(N) : "memory");
}
// the wave's LDS accesses done and at most N loads outstanding, then the
// workgroup barrier
template <int N>
__device__ __forceinline__ void lds_wait_barrier() {
  static_assert(N >= 0 && N < 64, "vmcnt field");
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" :: "n"(N) : "memory");
}

// the same with the wave's last L LDS reads still in flight
template <int N, int L>
__device__ __forceinline__ void lds_wait_barrier() {
  static_assert(N >= 0 && N < 64 && L >= 0 && L < 16, "vmcnt and lgkmcnt fields");
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(%1)\n\ts_barrier" :: "n"(N), "n"(L) : "memory");
}
// the workgroup's LDS accesses done; memory loads and stores stay in flight
__device__ __forceinline__ void lds_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }
// nothing is scheduled across this point
__device__ __forceinline__ void fence() { __builtin_amdgcn_sched_barrier(0); }
// memory operations stay on their side of this point
__device__ __forceinline__ void order() { asm volatile("" ::: "memory"); }

// 16 bytes of LDS at byte address a
__device__ __forceinline__ v4u lds_read16(uint32_t a) {
  return *reinterpret_cast<__attribute__((address_space(3))) const v4u*>(a);
}
// Transposing read: within each 16 lanes, lane i gives the address of 4
// elements (row i / 4, columns 4 (i % 4) .. + 3 of a 4 x 16 block) and
// receives column i, rows 0 .. 3.
__device__ __forceinline__ v2u lds_read_tr(uint32_t a) {
  return __builtin_bit_cast(v2u, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                     reinterpret_cast<__attribute__((address_space(3))) v4s*>(a)));
}

// 8 elements at any 2-byte aligned address (global memory takes unaligned
// 16-byte accesses); the first `count` of them, the others zero
__device__ __forceinline__ v4u load8(const uint16_t* p) {
  v4u v;
  __builtin_memcpy(&v, p, 16);
  return v;
}
__device__ __forceinline__ v4u load8(const uint16_t* p, int count) {
  if (count >= 8) return load8(p);
  v4u v = {0, 0, 0, 0};
#pragma unroll
  for (int e = 0; e < 7; ++e)
    if (e < count) v[e >> 1] |= static_cast<uint32_t>(p[e]) << (16 * (e & 1));
  return v;
}
__device__ __forceinline__ void store8(uint16_t* p, v4u v, int count) {
  if (count >= 8) {
    __builtin_memcpy(p, &v, 16);
    return;
  }
#pragma unroll
  for (int e = 0; e < 7; ++e)
    if (e < count) p[e] = static_cast<uint16_t>(v[e >> 1] >> (16 * (e & 1)));
}
// The same, not kept in the caches on its way (results that the kernel does
// not read again).  On large results, passes over changing inputs: attention
// 254 -> 246 us (4608 x 24 heads), linear 81 -> 73 (4608 x 3072 x 3072), norm
// 15.7 -> 14.4 (4608 x 3072).  In a transformer block with the quantized layers
// no difference (4608 x 3072: 1134 and 1142, 6144 x 1536: 617 and 608 us); two
// 16-bit linears in a row, 4608 x 3072 x 12288 x 3072, 578 -> 600.
__device__ __forceinline__ void stream8(uint16_t* p, v4u v) {
  typedef unsigned v4u_any __attribute__((ext_vector_type(4), aligned(2)));
  __builtin_nontemporal_store(v, reinterpret_cast<v4u_any*>(p));
}
template <typename E>
__device__ __forceinline__ void unpack8(v4u v, float (&f)[8]) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    f[2 * e] = E::lo(v[e]);
    f[2 * e + 1] = E::hi(v[e]);
  }
}
template <typename E>
__device__ __forceinline__ v4u pack8(const float (&f)[8]) {
  return v4u{E::pack2(f[0], f[1]), E::pack2(f[2], f[3]), E::pack2(f[4], f[5]), E::pack2(f[6], f[7])};
}

// 8-bit codes, e4m3: largest value 448, no infinity, NaN 0x7F.  Four fp32
// values to the bytes of a word, rounded to nearest even; past 448 and half a
// step they give NaN, so callers scale or clamp first.
constexpr float kMostF8 = 448.f;
__device__ __forceinline__ uint32_t pack4_f8(float a, float b, float c, float d) {
  const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return static_cast<uint32_t>(__builtin_amdgcn_cvt_pk_fp8_f32(c, d, lo, true));
}

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

}  // namespace svdq_dev
