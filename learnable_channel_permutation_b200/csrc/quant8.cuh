// A warp's part of quantising rows to e4m3 with a power-of-two scale for each 128 channels:
// two rows of 256 channels, eight channels a lane, permuted within blocks of at most 256.
// Used by the quantisers (quant8.cu) and by the product that quantises its own inputs (mm8.cu).
#pragma once

#include <cuda_fp8.h>

#include "lcp_internal.cuh"

namespace lcp {
namespace {

constexpr int Q8_CHUNK = 256;      // channels of a warp: two scale groups, eight channels a lane
// e8m0 byte of a block's largest magnitude.  amax = 1.f 2^(e - 127) is at most
// 448 2^k = 1.75 2^(k + 8) for k = e - 135 when f <= .75, else for k = e - 134.
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax) {
  if (amax >= 0x7f800000u) return 255u;
  if (amax == 0u) return 127u;
  const int byte = (int)(amax >> 23) - 8 + ((amax & 0x7fffffu) > 0x600000u ? 1 : 0);
  return byte < 0 ? 0u : (uint32_t)byte;
}
// 2^(127 - byte): a normal float for every byte scale_byte returns for finite
// blocks (0 .. 247); NaN for the NaN scale
__device__ __forceinline__ float scale_inverse(uint32_t byte) {
  return byte == 255u ? __uint_as_float(0x7fffffffu) : __uint_as_float((254u - byte) << 23);
}

__device__ __forceinline__ uint32_t pack4_e4m3(const float* v, float inv) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(v[0] * inv, v[1] * inv), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(v[2] * inv, v[3] * inv), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}

// Eight consecutive values of a row, 16-byte loads.
template <typename T> struct Vec8 { uint4 u[sizeof(T) / 2]; };
template <typename T> __device__ __forceinline__ Vec8<T> load8(const T* p) {
  Vec8<T> r;
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 2; ++i) r.u[i] = __ldg(reinterpret_cast<const uint4*>(p) + i);
  return r;
}
template <typename T> __device__ __forceinline__ Vec8<T> zero8() {
  Vec8<T> r;
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 2; ++i) r.u[i] = make_uint4(0u, 0u, 0u, 0u);
  return r;
}

constexpr int Q8_STAGE = Q8_CHUNK;   // words of a warp's exchange buffer

// The permutation entries of a lane's eight source channels; past the last channel, those that keep
// every place (the zeros there are moved like values, so that every slot is written).
struct __align__(16) Perm8 { uint32_t e[8]; };
__device__ __forceinline__ Perm8 load_perm(const int32_t* __restrict__ perm, int chan, int lane, int cin) {
  Perm8 r;
  if (chan < cin) {
    const uint4* at = reinterpret_cast<const uint4*>(perm + chan);
    *reinterpret_cast<uint4*>(r.e) = __ldg(at);
    *reinterpret_cast<uint4*>(r.e + 4) = __ldg(at + 1);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) r.e[j] = 8u * (uint32_t)lane + (uint32_t)j;
  }
  return r;
}
// Where those channels go in the exchange buffer (shared addresses).  An entry outside [0, B) is
// recorded in *error, and its low bits are taken, which keeps every slot in its block.
__device__ __forceinline__ void perm_slots(const Perm8& p, bool in, int lane, int bmask, const uint32_t* buf,
                                           uint32_t (&slot)[8], int* error) {
  // blocks are at least 32 wide: a lane's eight channels share the bits above the block's
  const uint32_t* e = p.e;
  const uint32_t mask = (uint32_t)bmask, block = 8u * (uint32_t)lane & ~mask;
  const uint32_t base = static_cast<uint32_t>(__cvta_generic_to_shared(buf));
  if (in && ((e[0] | e[1] | e[2] | e[3] | e[4] | e[5] | e[6] | e[7]) & ~mask)) atomicCAS(error, 0, 302);
#pragma unroll
  for (int j = 0; j < 8; ++j) slot[j] = base + 4u * (block | (e[j] & mask));
}
__device__ __forceinline__ void load_slots(const int32_t* __restrict__ perm, int chan, int lane, int cin, int bmask,
                                           const uint32_t* buf, uint32_t (&slot)[8], int* error) {
  perm_slots(load_perm(perm, chan, lane, cin), chan < cin, lane, bmask, buf, slot, error);
}
__device__ __forceinline__ void st_shared(uint32_t a, uint32_t v) {
  asm volatile("st.shared.u32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}
// Moves two rows' eight values of every lane to their slots, through `buf` (this warp's alone).
// bf16: the two rows' values of a channel share a word, so one 4-byte store moves both
// (random slots hit a bank three to four times a warp, whatever the width).  float32: one row
// after the other.
template <typename T>
__device__ __forceinline__ void permute_rows(Vec8<T>& a, Vec8<T>& b, const uint32_t (&slot)[8], const uint32_t* buf,
                                             int lane) {
  if constexpr (sizeof(T) == 2) {
    const uint32_t* x = reinterpret_cast<const uint32_t*>(&a);
    const uint32_t* y = reinterpret_cast<const uint32_t*>(&b);
    __syncwarp();
#pragma unroll
    for (int j = 0; j < 8; ++j) st_shared(slot[j], __byte_perm(x[j / 2], y[j / 2], j & 1 ? 0x7632 : 0x5410));
    __syncwarp();
    uint32_t w[8];
    *reinterpret_cast<uint4*>(w) = reinterpret_cast<const uint4*>(buf + 8 * lane)[0];
    *reinterpret_cast<uint4*>(w + 4) = reinterpret_cast<const uint4*>(buf + 8 * lane)[1];
    uint32_t* u = reinterpret_cast<uint32_t*>(&a);
    uint32_t* v = reinterpret_cast<uint32_t*>(&b);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      u[j] = __byte_perm(w[2 * j], w[2 * j + 1], 0x5410);
      v[j] = __byte_perm(w[2 * j], w[2 * j + 1], 0x7632);
    }
  } else {
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      Vec8<T>& v = r ? b : a;
      const uint32_t* e = reinterpret_cast<const uint32_t*>(&v);
      __syncwarp();
#pragma unroll
      for (int j = 0; j < 8; ++j) st_shared(slot[j], e[j]);
      __syncwarp();
      v.u[0] = reinterpret_cast<const uint4*>(buf + 8 * lane)[0];
      v.u[1] = reinterpret_cast<const uint4*>(buf + 8 * lane)[1];
    }
  }
}

// Largest magnitudes.  A fold takes eight values into a running maximum (0 to begin with); a NaN wins.
// float32: its bits, two values an instruction.  bf16: two running maxima in a word (its
// instruction that takes magnitudes itself measured slower: 8192 x 11008 permuted 49 us, 47).
__device__ __forceinline__ uint32_t max_pair(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t fold_max(uint32_t m, const Vec8<__nv_bfloat16>& v) {
  const uint32_t* w = reinterpret_cast<const uint32_t*>(&v);
#pragma unroll
  for (int j = 0; j < 4; ++j) m = max_pair(m, w[j] & 0x7fff7fffu);
  return m;
}
__device__ __forceinline__ uint32_t fold_max(uint32_t m, const Vec8<float>& v) {
  const float* f = reinterpret_cast<const float*>(&v);
  float x = __uint_as_float(m);
#pragma unroll
  for (int j = 0; j < 8; j += 2) asm("max.NaN.abs.f32 %0, %0, %1, %2;" : "+f"(x) : "f"(f[j]), "f"(f[j + 1]));
  return __float_as_uint(x);
}
// the maximum as float bits: infinities above every finite value and NaNs above those, as integers compare
template <typename T> __device__ __forceinline__ uint32_t max_bits(uint32_t m) {
  return sizeof(T) == 4 ? m : max(m << 16, m & 0xffff0000u);
}
// over the 16 lanes that share a scale group
__device__ __forceinline__ uint32_t half_max(uint32_t m) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
  return m;
}
// The group maxima of two rows (bf16: both travel in one word).
__device__ __forceinline__ void group_max(const Vec8<float> (&v)[2], uint32_t (&m)[2]) {
  m[0] = half_max(fold_max(0u, v[0]));
  m[1] = half_max(fold_max(0u, v[1]));
}
__device__ __forceinline__ void group_max(const Vec8<__nv_bfloat16> (&v)[2], uint32_t (&m)[2]) {
  const uint32_t a = fold_max(0u, v[0]), b = fold_max(0u, v[1]);
  uint32_t w = max_pair(__byte_perm(a, b, 0x5410), __byte_perm(a, b, 0x7632));
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) w = max_pair(w, __shfl_xor_sync(0xffffffffu, w, o));
  m[0] = w << 16;
  m[1] = w & 0xffff0000u;
}

// Eight values times a power of two, as e4m3.  In bf16 the product is exact too (a result below
// bf16's range is far below e4m3's).
__device__ __forceinline__ uint2 to_e4m3(const Vec8<float>& v, float inv) {
  const float* f = reinterpret_cast<const float*>(&v);
  return make_uint2(pack4_e4m3(f, inv), pack4_e4m3(f + 4, inv));
}
__device__ __forceinline__ uint32_t pair_e4m3(uint32_t w, __nv_bfloat162 inv) {
  const __nv_bfloat162 p = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&w), inv);
  const uint32_t u = *reinterpret_cast<const uint32_t*>(&p);
  return __nv_cvt_float2_to_fp8x2(make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u)), __NV_SATFINITE,
                                  __NV_E4M3);
}
__device__ __forceinline__ uint2 to_e4m3(const Vec8<__nv_bfloat16>& v, float inv) {
  const uint32_t* w = reinterpret_cast<const uint32_t*>(&v);
  const __nv_bfloat162 i2 = __float2bfloat162_rn(inv);
  return make_uint2(pair_e4m3(w[0], i2) | (pair_e4m3(w[1], i2) << 16), pair_e4m3(w[2], i2) | (pair_e4m3(w[3], i2) << 16));
}

// 4 x 4 bytes: word i byte k <-> word k byte i.
__device__ __forceinline__ void transpose_bytes(uint32_t& a, uint32_t& b, uint32_t& c, uint32_t& d) {
  const uint32_t t0 = __byte_perm(a, b, 0x5140), t1 = __byte_perm(a, b, 0x7362);
  const uint32_t t2 = __byte_perm(c, d, 0x5140), t3 = __byte_perm(c, d, 0x7362);
  a = __byte_perm(t0, t2, 0x5410);
  b = __byte_perm(t0, t2, 0x7632);
  c = __byte_perm(t1, t3, 0x5410);
  d = __byte_perm(t1, t3, 0x7632);
}
// Moves four rows' eight e4m3 values of every lane to their slots: the rows' bytes of a channel
// share a word, so one 4-byte store moves four.
__device__ __forceinline__ void permute_bytes(uint2* q, const uint32_t (&slot)[8], const uint32_t* buf, int lane) {
  transpose_bytes(q[0].x, q[1].x, q[2].x, q[3].x);
  transpose_bytes(q[0].y, q[1].y, q[2].y, q[3].y);
  __syncwarp();
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    st_shared(slot[j], q[j].x);
    st_shared(slot[4 + j], q[j].y);
  }
  __syncwarp();
  uint32_t w[8];
  *reinterpret_cast<uint4*>(w) = reinterpret_cast<const uint4*>(buf + 8 * lane)[0];
  *reinterpret_cast<uint4*>(w + 4) = reinterpret_cast<const uint4*>(buf + 8 * lane)[1];
  transpose_bytes(w[0], w[1], w[2], w[3]);
  transpose_bytes(w[4], w[5], w[6], w[7]);
#pragma unroll
  for (int j = 0; j < 4; ++j) q[j] = make_uint2(w[j], w[4 + j]);
}

}  // namespace
}  // namespace lcp
