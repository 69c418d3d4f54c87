// 8-bit operands of the deployed product: e4m3 values with one power-of-two
// scale (e8m0) for each block of 128.
//
//   activations: a block is 128 consecutive channels of one token of x_pi
//   weights:     a block is 128 rows x 128 columns of A = M.(W P_B)
//
// The scale of a block with largest magnitude amax is 2^k, k the smallest
// integer >= -127 with amax <= 448 2^k (448 is e4m3's largest value; k = 0 for a
// block of zeros), and a value becomes q = rn_e4m3(x 2^-k).  The product x 2^-k
// only moves the exponent, so the rounding to e4m3 (to nearest, ties to even;
// at most half a step, 2^-4 of the value) is the only one made.  A block that
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

// CTAs of the activation kernel that fit an SM.
template <typename T, bool PERM> constexpr int row_ctas() { return sizeof(T) == 4 && PERM ? 3 : 4; }

// Activations.  A warp keeps one 256-channel chunk and walks tokens two at a time, the next two
// loading meanwhile, so the permutation is read once and its slots stay in registers.
template <typename T, bool PERM>
__global__ void __launch_bounds__(32 * Q8_ROW_WARPS, row_ctas<T, PERM>())
quant8_rows_kernel(const T* __restrict__ X, const int32_t* __restrict__ perm, uint8_t* __restrict__ Q,
                   uint8_t* __restrict__ S, int tokens, int cin, int bmask) {
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
  for (; t < tokens; t += 2 * step) {
    Vec8<T> v[2] = {next[0], next[1]};
    next[0] = load(t + 2 * step);
    next[1] = load(t + 3 * step);
    if (PERM) permute_rows(v[0], v[1], slot, stage[warp], lane);
    uint32_t m[2];
    group_max(v, m);
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int row = t + u * step;
      if (row >= tokens || !in) break;
      const uint32_t byte = scale_byte(m[u]);
      *reinterpret_cast<uint2*>(Q + (size_t)row * cin + chan) = to_e4m3(v[u], scale_inverse(byte));
      if ((lane & 15) == 0) S[(size_t)row * G + chan / 128] = (uint8_t)byte;
    }
  }
}

// Weights.  A CTA takes 128 rows x CH channels and holds the values in registers (in their stored
// type, 32 registers a lane) while the block maxima are reduced.  CH = 256 (two blocks, a warp to a
// row) for B = 256 and for every permuted bf16 weight, 128 (half a warp to a row) otherwise:
// smaller CTAs overlap their phases better (5120 x 13824 as it is: 32.2 us, 33.7 at CH = 256; float32
// permuted: 90 us, 104), but bf16's exchange does not gain by it (permuted and masked: 49.7 us at
// CH = 128, 47.3 at 256).
template <typename T> constexpr int w_loads() { return 16 / (int)sizeof(T); }     // of a lane, each eight channels of a row
template <typename T, int CH> constexpr int w_warps() { return CH / 2 / w_loads<T>(); }
template <typename T, bool PERM, bool MASK, int CH>
__global__ void __launch_bounds__(32 * w_warps<T, CH>(), 32 / w_warps<T, CH>())
quant8_weight_kernel(const T* __restrict__ W, const int32_t* __restrict__ perm, const uint8_t* __restrict__ mask,
                     uint8_t* __restrict__ Q, uint8_t* __restrict__ S, int cout, int cin, int bmask) {
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
  uint32_t m = 0;
#pragma unroll
  for (int r = 0; r < LOADS; ++r) {
    if (PERM && r % 2 == 0) permute_rows(v[r], v[r + 1], slot, stage[warp], lane);
    if (MASK) apply_mask(v[r], keep[r / 4] >> (8 * (r % 4)));
    m = max(m, amax8(v[r]));
  }
  m = half_max(m);
  if ((lane & 15) == 0) part[warp][lane >> 4] = m;
  __syncthreads();
  m = 0;
#pragma unroll
  for (int w = 0; w < WARPS; ++w) m = max(m, CH == 128 ? max(part[w][0], part[w][1]) : part[w][lane >> 4]);
  const uint32_t byte = scale_byte(m);
  const float inv = scale_inverse(byte);
  if (!in) return;
  uint8_t* q0 = Q + (size_t)o0 * cin + chan;
#pragma unroll
  for (int r = 0; r < LOADS; ++r)
    if (whole || o0 + r * WARPS * ROWS < cout) *reinterpret_cast<uint2*>(q0 + r * step) = to_e4m3(v[r], inv);
  if (warp == 0 && (lane == 0 || (CH == 256 && lane == 16))) S[(size_t)blockIdx.y * G + chan / 128] = (uint8_t)byte;
}

int cdiv_host(int a, int b) { return (a + b - 1) / b; }

template <typename T>
lcp_status rows_t(const T* X, const int32_t* perm, uint8_t* Q, uint8_t* S, int tokens, int cin, int B, cudaStream_t st) {
  const int sms = device_sms(), chunks = cdiv_host(cin, Q8_CHUNK);
  // as many CTAs as fit the GPU at once (one more would cost a second round of all of them)
  const int fit = (perm ? row_ctas<T, true>() : row_ctas<T, false>()) * sms / chunks;
  const int gy = std::min(cdiv_host(tokens, Q8_ROW_WARPS), std::max(fit, 1));
  const dim3 grid((unsigned)chunks, (unsigned)gy);
  const int bmask = perm ? B - 1 : 0;
  if (perm)
    return launch_kernel(quant8_rows_kernel<T, true>, grid, dim3(32 * Q8_ROW_WARPS), 0, st, 1, true, "quant8", X, perm, Q,
                         S, tokens, cin, bmask);
  return launch_kernel(quant8_rows_kernel<T, false>, grid, dim3(32 * Q8_ROW_WARPS), 0, st, 1, true, "quant8", X, perm, Q, S,
                       tokens, cin, bmask);
}

template <typename T, bool PERM, int CH>
lcp_status weight_ch(const T* W, const int32_t* perm, const uint32_t* mask, uint8_t* Q, uint8_t* S, int cout, int cin,
                     int B, cudaStream_t st) {
  const dim3 grid((unsigned)cdiv_host(cin, CH), (unsigned)cdiv_host(cout, 128)), block(32 * w_warps<T, CH>());
  const uint8_t* mb = reinterpret_cast<const uint8_t*>(mask);
  const auto kernel = mask ? quant8_weight_kernel<T, PERM, true, CH> : quant8_weight_kernel<T, PERM, false, CH>;
  return launch_kernel(kernel, grid, block, 0, st, 1, true, "quant8_weight", W, perm, mb, Q, S, cout, cin, B - 1);
}
template <typename T>
lcp_status weight_t(const T* W, const int32_t* perm, const uint32_t* mask, uint8_t* Q, uint8_t* S, int cout, int cin,
                    int B, cudaStream_t st) {
  if (!perm) return weight_ch<T, false, 128>(W, perm, mask, Q, S, cout, cin, 1, st);
  if constexpr (sizeof(T) == 4) {
    if (B != 256) return weight_ch<T, true, 128>(W, perm, mask, Q, S, cout, cin, B, st);
  }
  return weight_ch<T, true, 256>(W, perm, mask, Q, S, cout, cin, B, st);
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
  if (dt == LCP_F32) return rows_t(static_cast<const float*>(X), perm, Q, S, tokens, cin, B, st);
  return rows_t(static_cast<const __nv_bfloat16*>(X), perm, Q, S, tokens, cin, B, st);
}

lcp_status launch_quant8_weight(const void* W, const int32_t* perm, const uint32_t* mask, uint8_t* Q, uint8_t* S,
                                int cout, int cin, int B, lcp_dtype dt, cudaStream_t st) {
  if (dt == LCP_F32) return weight_t(static_cast<const float*>(W), perm, mask, Q, S, cout, cin, B, st);
  return weight_t(static_cast<const __nv_bfloat16*>(W), perm, mask, Q, S, cout, cin, B, st);
}

}  // namespace lcp
