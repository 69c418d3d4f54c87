// 8-bit operands of the deployed product: e4m3 values with one power-of-two
// scale (e8m0) for each block of 128.
//
//   activations: a block is 128 consecutive channels of one token of x_pi
//   weights:     a block is 128 rows x 128 columns of A = M.(W P_B)
//
// The scale of a block with largest magnitude amax is 2^k, k the smallest
// integer >= -127 with amax <= 448 2^k (448 is e4m3's largest value; k = 0 for a
// block of zeros), and a value becomes q = rn_e4m3(x 2^-k).  The product x 2^-k
// only moves the exponent, so the rounding to e4m3 (to nearest, ties to even) is
// the only one made.  It is at most half a step: 2^-4 of the value, or 2^-10 of
// the scale where that is more (values under 2^-6 of the scale, which e4m3 holds
// as subnormals; under 2^-10 of it they become zero).  A block that
// holds an infinity or a NaN gets the NaN scale (0xff) and NaN values, so every
// product it enters is NaN.
//
// Both kernels are bound by HBM: they read each value once and write half (bf16)
// or a quarter (float32) of the bytes.  The permutation is applied by a warp on
// its own 256 channels (whole blocks for every B <= 256), through 256 values of
// shared memory that only that warp uses: no CTA barrier.

#include <algorithm>

#include "quant8.cuh"

namespace lcp {
namespace {

__device__ int g_quant_error;   // first invalid permutation entry seen (302), 0 if none

constexpr int Q8_ROW_WARPS = 8;    // activations: warps per CTA

// Zeroes the values whose bit of `keep` (eight bits) is clear.  bf16: a product spreads four bits
// to the top bits of four bytes, whose signs a byte permutation then copies over a pair of values.
__device__ __forceinline__ void apply_mask(Vec8<float>& v, uint32_t keep) {
  uint32_t* w = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (!((keep >> j) & 1u)) w[j] = 0u;
}
// prmt's sign mode (which __byte_perm leaves out): selector nibble 8 + i is byte i's sign, eight times.
template <uint32_t SEL> __device__ __forceinline__ uint32_t byte_signs(uint32_t x) {
  uint32_t r;
  asm("prmt.b32 %0, %1, %1, %2;" : "=r"(r) : "r"(x), "n"(SEL));
  return r;
}
__device__ __forceinline__ void apply_mask(Vec8<__nv_bfloat16>& v, uint32_t keep) {
  uint32_t* w = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t tops = ((keep >> (4 * h)) & 15u) * 0x10204080u;
    w[2 * h] &= byte_signs<0x9988>(tops);
    w[2 * h + 1] &= byte_signs<0xbbaa>(tops);
  }
}

// How a kernel permutes.  Blocks of at most 128 channels keep every value in its scale group, so the
// scale does not depend on the order and the e4m3 bytes can be moved (kBytes), four rows a word: the
// exchange through shared memory, whose random accesses hit a bank three to four times a warp, is
// half of bf16's and a quarter of float32's.  Blocks of 256 move the values before the groups' maxima
// are taken (kValues).  As bytes and as values: 4096 x 13824 float32 activations 44 and 60 us,
// 8192 x 11008 bf16 47 and 50; weights of 5120 x 13824, permuted 34 and 44, masked too 41 and 48, float32
// 70 and 90.
enum class Order { kPlain, kValues, kBytes };

// The same for values that are not permuted yet.  keep[0] holds the mask bytes of rows 0 to 3, keep[1] of rows 4
// to 7, in the permuted order; g[j] becomes the bits, row r's in bit r, that source channel j meets
// at its slot.  The eight bytes are transposed as 8 x 8 bits (by exchanging 1 x 1, then 2 x 2, then 4 x 4
// squares across the diagonal), so a channel's byte is one random access, in 256 bytes that
// lie at most two words to a bank.
__device__ __forceinline__ void gather_mask(const uint32_t (&keep)[2], const uint32_t (&slot)[8], uint32_t* buf, int lane,
                                            uint32_t (&g)[8]) {
  uint32_t x = keep[1], y = keep[0], t;
  t = (x ^ (x >> 7)) & 0x00aa00aau, x ^= t ^ (t << 7);
  t = (y ^ (y >> 7)) & 0x00aa00aau, y ^= t ^ (t << 7);
  t = (x ^ (x >> 14)) & 0x0000ccccu, x ^= t ^ (t << 14);
  t = (y ^ (y >> 14)) & 0x0000ccccu, y ^= t ^ (t << 14);
  reinterpret_cast<uint2*>(buf)[lane] = make_uint2((x << 4 & 0xf0f0f0f0u) | (y & 0x0f0f0f0fu),
                                                   (x & 0xf0f0f0f0u) | (y >> 4 & 0x0f0f0f0fu));
  __syncwarp();
  const uint32_t base3 = 3u * static_cast<uint32_t>(__cvta_generic_to_shared(buf));
#pragma unroll
  for (int j = 0; j < 8; ++j)      // slot = base + 4 i, the byte is at base + i
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(g[j]) : "r"((slot[j] + base3) >> 2));
}
__device__ __forceinline__ void apply_mask_row(Vec8<float>& v, const uint32_t (&g)[8], int row) {
  uint32_t* w = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (!(g[j] >> row & 1u)) w[j] = 0u;
}
__device__ __forceinline__ void apply_mask_row(Vec8<__nv_bfloat16>& v, const uint32_t (&g)[8], int row) {
  uint32_t* w = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
  for (int j = 0; j < 4; ++j) w[j] &= byte_signs<0xaa88>((g[2 * j] | g[2 * j + 1] << 16) << (7 - row));
}

// CTAs of the activation kernel that fit an SM (bf16 of 8192 x 11008 as it is: 42 us with five, 46 with
// four; permuted: 47 with four, 50 with five, 61 with three).
template <typename T, Order ORDER> constexpr int row_ctas() {
  return (sizeof(T) == 4 ? 3 : 4) + (ORDER == Order::kPlain ? 1 : 0);
}

// Activations.  A warp keeps one 256-channel chunk and walks tokens two at a time (four where it
// moves bytes), the next two loading meanwhile, so the permutation is read once and its slots
// stay in registers.
template <typename T, Order ORDER>
__global__ void __launch_bounds__(32 * Q8_ROW_WARPS, row_ctas<T, ORDER>())
quant8_rows_kernel(const T* __restrict__ X, const int32_t* __restrict__ perm, uint8_t* __restrict__ Q,
                   uint8_t* __restrict__ S, int tokens, int cin, int bmask) {
  constexpr bool PERM = ORDER != Order::kPlain;
  constexpr int PAIRS = ORDER == Order::kBytes ? 2 : 1;      // of tokens a round
  __shared__ __align__(16) uint32_t stage[PERM ? Q8_ROW_WARPS : 1][PERM ? Q8_STAGE : 4];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int chan = blockIdx.x * Q8_CHUNK + 8 * lane;
  const int G = (cin + 127) / 128;
  const bool in = chan < cin;      // C_in is a multiple of 32: a lane's channels are inside together
  pdl_wait();
  pdl_trigger();
  const int step = gridDim.y * Q8_ROW_WARPS;
  auto load = [&](int t) { return in && t < tokens ? load8(X + (size_t)t * cin + chan) : zero8<T>(); };
  int t = blockIdx.y * Q8_ROW_WARPS + warp;
  Vec8<T> next[2] = {load(t), load(t + step)};
  uint32_t slot[8];
  if (PERM) load_slots(perm, chan, lane, cin, bmask, stage[warp], slot, &g_quant_error);
  for (; t < tokens; t += 2 * PAIRS * step) {
    uint2 q[2 * PAIRS];
    uint32_t byte[2 * PAIRS];
#pragma unroll
    for (int h = 0; h < PAIRS; ++h) {
      Vec8<T> v[2] = {next[0], next[1]};
      next[0] = load(t + (2 * h + 2) * step);
      next[1] = load(t + (2 * h + 3) * step);
      if (ORDER == Order::kValues) permute_rows(v[0], v[1], slot, stage[warp], lane);
      uint32_t m[2];
      group_max(v, m);
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        byte[2 * h + u] = scale_byte(m[u]);
        q[2 * h + u] = to_e4m3(v[u], scale_inverse(byte[2 * h + u]));
      }
    }
    if constexpr (ORDER == Order::kBytes) permute_bytes(q, slot, stage[warp], lane);
#pragma unroll
    for (int u = 0; u < 2 * PAIRS; ++u) {
      const int row = t + u * step;
      if (row >= tokens || !in) break;
      *reinterpret_cast<uint2*>(Q + (size_t)row * cin + chan) = q[u];
      if ((lane & 15) == 0) S[(size_t)row * G + chan / 128] = (uint8_t)byte[u];
    }
  }
}

// Weights.  A CTA takes 128 rows x CH channels and holds the values in registers (in their stored
// type, 32 registers a lane) while the block maxima are reduced.  CH = 256 (two blocks, a warp to a
// row) for B = 256, 128 (half a warp to a row) otherwise: smaller CTAs overlap their phases better
// (5120 x 13824 permuted and masked: 41 us, 48 at CH = 256; as it is: 32 us, 34).
template <typename T> constexpr int w_loads() { return 16 / (int)sizeof(T); }     // of a lane, each eight channels of a row
template <typename T, int CH> constexpr int w_warps() { return CH / 2 / w_loads<T>(); }
template <typename T, Order ORDER, bool MASK, int CH>
__global__ void __launch_bounds__(32 * w_warps<T, CH>(), 32 / w_warps<T, CH>())
quant8_weight_kernel(const T* __restrict__ W, const int32_t* __restrict__ perm, const uint8_t* __restrict__ mask,
                     uint8_t* __restrict__ Q, uint8_t* __restrict__ S, int cout, int cin, int bmask) {
  constexpr bool PERM = ORDER != Order::kPlain;
  constexpr int LOADS = w_loads<T>(), WARPS = w_warps<T, CH>();
  constexpr int ROWS = 256 / CH;     // of a warp's load
  __shared__ __align__(16) uint32_t stage[PERM ? WARPS : 1][PERM ? Q8_STAGE : 4];
  __shared__ uint32_t part[WARPS][2];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int chan = blockIdx.x * CH + 8 * (lane & (CH / 8 - 1));
  const int G = (cin + 127) / 128;
  const bool in = chan < cin;
  const int o0 = blockIdx.y * 128 + warp * ROWS + (CH == 128 ? lane >> 4 : 0);
  pdl_wait();
  pdl_trigger();
  Vec8<T> v[LOADS];
  uint32_t keep[2] = {0u, 0u};      // a row's eight mask bits in a byte
  // rows and channels of a whole tile are loaded and stored without bounds checks
  const bool whole = (int)(blockIdx.y + 1) * 128 <= cout && (int)(blockIdx.x + 1) * CH <= cin;
  const size_t step = (size_t)(WARPS * ROWS) * cin;
  const T* w0 = W + (size_t)o0 * cin + chan;
  const uint8_t* m0 = MASK ? mask + (size_t)o0 * (cin / 8) + chan / 8 : nullptr;
  if (whole) {
#pragma unroll
    for (int r = 0; r < LOADS; ++r) {
      v[r] = load8(w0 + r * step);
      if (MASK) keep[r / 4] |= (uint32_t)__ldg(m0 + r * (step / 8)) << (8 * (r % 4));
    }
  } else {
#pragma unroll
    for (int r = 0; r < LOADS; ++r) {
      const bool ok = in && o0 + r * WARPS * ROWS < cout;
      v[r] = ok ? load8(w0 + r * step) : zero8<T>();
      if (MASK && ok) keep[r / 4] |= (uint32_t)__ldg(m0 + r * (step / 8)) << (8 * (r % 4));
    }
  }
  uint32_t slot[8];
  if (PERM) load_slots(perm, chan, lane, cin, bmask, stage[warp], slot, &g_quant_error);
  uint32_t g[8];
  if (MASK && ORDER == Order::kBytes) gather_mask(keep, slot, stage[warp], lane, g);
  uint32_t m = 0;
#pragma unroll
  for (int r = 0; r < LOADS; ++r) {
    if (ORDER == Order::kValues && r % 2 == 0) permute_rows(v[r], v[r + 1], slot, stage[warp], lane);
    if (MASK && ORDER == Order::kBytes) apply_mask_row(v[r], g, r);
    else if (MASK) apply_mask(v[r], keep[r / 4] >> (8 * (r % 4)));
    m = fold_max(m, v[r]);
  }
  m = half_max(max_bits<T>(m));
  if ((lane & 15) == 0) part[warp][lane >> 4] = m;
  __syncthreads();
  m = 0;
#pragma unroll
  for (int w = 0; w < WARPS; ++w) m = max(m, CH == 128 ? max(part[w][0], part[w][1]) : part[w][lane >> 4]);
  const uint32_t byte = scale_byte(m);
  const float inv = scale_inverse(byte);
  uint8_t* q0 = Q + (size_t)o0 * cin + chan;
#pragma unroll
  for (int r0 = 0; r0 < LOADS; r0 += 4) {
    uint2 q[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) q[r] = to_e4m3(v[r0 + r], inv);
    if constexpr (ORDER == Order::kBytes) permute_bytes(q, slot, stage[warp], lane);
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (whole || (in && o0 + (r0 + r) * WARPS * ROWS < cout)) *reinterpret_cast<uint2*>(q0 + (r0 + r) * step) = q[r];
  }
  if (in && warp == 0 && (lane == 0 || (CH == 256 && lane == 16))) S[(size_t)blockIdx.y * G + chan / 128] = (uint8_t)byte;
}

int cdiv_host(int a, int b) { return (a + b - 1) / b; }

// As many CTAs a chunk as fit the GPU at once (one more would cost a second round of all of them).
template <typename T, Order ORDER> int row_fit(int cin) {
  return std::max(row_ctas<T, ORDER>() * device_sms() / cdiv_host(cin, Q8_CHUNK), 1);
}
template <typename T, Order ORDER>
lcp_status rows_t(const T* X, const int32_t* perm, uint8_t* Q, uint8_t* S, int tokens, int cin, int B, cudaStream_t st) {
  const int chunks = cdiv_host(cin, Q8_CHUNK);
  const int gy = std::min(cdiv_host(tokens, Q8_ROW_WARPS), row_fit<T, ORDER>(cin));
  return launch_kernel(quant8_rows_kernel<T, ORDER>, dim3((unsigned)chunks, (unsigned)gy), dim3(32 * Q8_ROW_WARPS), 0, st, 1,
                       true, "quant8", X, perm, Q, S, tokens, cin, B - 1);
}
template <typename T>
lcp_status rows_order(const T* X, const int32_t* perm, uint8_t* Q, uint8_t* S, int tokens, int cin, int B, cudaStream_t st) {
  if (!perm) return rows_t<T, Order::kPlain>(X, perm, Q, S, tokens, cin, 1, st);
  // bf16 of at most two tokens a warp: a round of the byte order is four (512 x 4096: 2.8 us, 3.5 as bytes)
  const bool few = sizeof(T) == 2 && tokens <= 2 * Q8_ROW_WARPS * row_fit<T, Order::kValues>(cin);
  if (B == 256 || few) return rows_t<T, Order::kValues>(X, perm, Q, S, tokens, cin, B, st);
  return rows_t<T, Order::kBytes>(X, perm, Q, S, tokens, cin, B, st);
}

template <typename T, Order ORDER, int CH>
lcp_status weight_ch(const T* W, const int32_t* perm, const uint32_t* mask, uint8_t* Q, uint8_t* S, int cout, int cin,
                     int B, cudaStream_t st) {
  const dim3 grid((unsigned)cdiv_host(cin, CH), (unsigned)cdiv_host(cout, 128)), block(32 * w_warps<T, CH>());
  const uint8_t* mb = reinterpret_cast<const uint8_t*>(mask);
  const auto kernel = mask ? quant8_weight_kernel<T, ORDER, true, CH> : quant8_weight_kernel<T, ORDER, false, CH>;
  return launch_kernel(kernel, grid, block, 0, st, 1, true, "quant8_weight", W, perm, mb, Q, S, cout, cin, B - 1);
}
template <typename T>
lcp_status weight_t(const T* W, const int32_t* perm, const uint32_t* mask, uint8_t* Q, uint8_t* S, int cout, int cin,
                    int B, cudaStream_t st) {
  if (!perm) return weight_ch<T, Order::kPlain, 128>(W, perm, mask, Q, S, cout, cin, 1, st);
  if (B == 256) return weight_ch<T, Order::kValues, 256>(W, perm, mask, Q, S, cout, cin, B, st);
  return weight_ch<T, Order::kBytes, 128>(W, perm, mask, Q, S, cout, cin, B, st);
}

}  // namespace

lcp_status quant_error(int* site, int reset) {
  int v = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_quant_error, sizeof(int));
  if (e == cudaSuccess && reset) {
    const int z = 0;
    e = cudaMemcpyToSymbol(g_quant_error, &z, sizeof(int));
  }
  if (e != cudaSuccess) {
    cudaGetLastError();
    return fail(LCP_ERR_CUDA, "reading the device error word: %s", cudaGetErrorString(e));
  }
  *site = v;
  return LCP_OK;
}

lcp_status launch_quant8(const void* X, const int32_t* perm, uint8_t* Q, uint8_t* S, int tokens, int cin, int B,
                         lcp_dtype dt, cudaStream_t st) {
  if (dt == LCP_F32) return rows_order(static_cast<const float*>(X), perm, Q, S, tokens, cin, B, st);
  return rows_order(static_cast<const __nv_bfloat16*>(X), perm, Q, S, tokens, cin, B, st);
}

lcp_status launch_quant8_weight(const void* W, const int32_t* perm, const uint32_t* mask, uint8_t* Q, uint8_t* S,
                                int cout, int cin, int B, lcp_dtype dt, cudaStream_t st) {
  if (dt == LCP_F32) return weight_t(static_cast<const float*>(W), perm, mask, Q, S, cout, cin, B, st);
  return weight_t(static_cast<const __nv_bfloat16*>(W), perm, mask, Q, S, cout, cin, B, st);
}

}  // namespace lcp
