// Products of 8-bit operands with a power-of-two scale for each block of 128:
//
//   Y[t][o] = sum over groups g of  2^(kx[t][g] + kw[o / 128][g])
//             * sum over the 128 channels c of group g of  qx[t][c] qw[o][c]
//
// on the tensor cores (tcgen05.mma kind::mxf8f6f4, block scaled): the scales are
// e8m0 bytes, the format the instruction multiplies in by itself, so the
// accumulation over all of C_in stays in one float32 accumulator in tensor
// memory.  Output channels are the M side (128 lanes of tensor memory) and
// tokens the N side, whose width follows the token count; one lane is one
// channel, so a warp's store of one token is 32 consecutive channels of Y.

#include "tc_common.cuh"

namespace lcp {
namespace {

// D[tmem] (+)= A[smem] * B[smem]^T with the e8m0 scales of A's and B's rows in tensor
// memory: e4m3 operands, K = 32 a step, float32 accumulation.
__device__ __forceinline__ void mma_mx8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                        bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate ? 1u : 0u)
      : "memory");
}
// 32 rows of 16 bytes of shared memory to four columns of tensor memory, the same
// in every 32-lane quarter: lane r's column j is word j of row r.
__device__ __forceinline__ void copy_scales(uint32_t taddr, uint64_t sd) {
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(sd) : "memory");
}
// Shared-memory descriptor without swizzle: eight rows of 16 bytes are a unit, units 128 B apart.
__device__ __forceinline__ uint64_t sdesc_scales(uint32_t saddr) {
  return (uint64_t)((saddr >> 4) & 0x3FFFu) | ((uint64_t)(128u >> 4) << 32) | (1ull << 46);
}
// Instruction descriptor of kind::mxf8f6f4: A and B e4m3 (0), K-major, e8m0 scales (bit 23);
// `byte` selects which byte of the scale words this step uses (bits 4-5 for B, 29-30 for A).
__host__ __device__ constexpr uint32_t idesc_mx8(int M, int N) {
  return (1u << 23) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
__device__ __forceinline__ uint32_t with_byte(uint32_t idesc, int byte) {
  return idesc | ((uint32_t)byte << 4) | ((uint32_t)byte << 29);
}

constexpr int M8_BM = 128;            // output channels of a CTA: one row of weight scales
constexpr int M8_A = M8_BM * 128;     // bytes of a stage's weight tile (one scale group of channels)
constexpr int M8_SF = 4;              // ring of scale chunks (four groups each)
constexpr int M8_THREADS = 224;       // warp 0: TMA, 1: MMA, 2-5: epilogue, 6: scales
constexpr int M8_MAX_STAGES = 8;

__device__ __forceinline__ float ld_cluster_f32(uint32_t a) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
  return v;
}

// One CTA: 128 output channels x NT tokens over a range of scale groups; the S CTAs of a
// cluster share a tile and split its groups, then each adds the S partial results of its
// tokens in rank order.
//
// Scale words: a chunk is four groups, so a row's four scale bytes are one 32-bit word and
// the instruction picks the byte of the group at hand.  Warp 6 builds the words of chunk c in
// ring slot c % 4; the MMA thread copies them to tensor-memory set c % 2 and, before it does,
// waits for the products of chunk c - 2 that read that set.
template <typename OUT>
__global__ void __launch_bounds__(M8_THREADS)
mm8_split_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                 const uint8_t* __restrict__ Xs, const uint8_t* __restrict__ Ws, OUT* __restrict__ Y, int cout, int cin,
                 int tokens, int NT, int stages, int S, int w_early) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align1024(smem_raw);
  const int stage_bytes = M8_A + NT * 128;
  uint8_t* sf = smem + stages * stage_bytes;                  // M8_SF x (512 B of W, 512 B of X)
  uint64_t* bars = reinterpret_cast<uint64_t*>(sf + M8_SF * 1024);
  uint32_t* holder = reinterpret_cast<uint32_t*>(bars + 2 * M8_MAX_STAGES + 2 * M8_SF + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(holder + 1);
  auto full = [&](int s) { return smem_u32(bars + s); };
  auto empty = [&](int s) { return smem_u32(bars + M8_MAX_STAGES + s); };
  auto sffull = [&](int s) { return smem_u32(bars + 2 * M8_MAX_STAGES + s); };
  auto sfempty = [&](int s) { return smem_u32(bars + 2 * M8_MAX_STAGES + M8_SF + s); };
  const uint32_t done = smem_u32(bars + 2 * M8_MAX_STAGES + 2 * M8_SF);

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int rank = S > 1 ? (int)cluster_rank() : 0;
  const int G = cdiv(cin, 128), mtiles = cdiv(cout, M8_BM);
  const int tile = blockIdx.x / S;
  const int mt = tile % mtiles, nt = tile / mtiles;
  const int t0 = nt * NT;
  const int g0 = (int)((long long)rank * G / S), g1 = (int)((long long)(rank + 1) * G / S);   // never empty: S <= G
  const int nk = g1 - g0, nchunk = cdiv(nk, 4);

  // accumulator columns [0, NT), then two sets of (4 columns of W scales, 4 of X scales)
  uint32_t ncols = 32;
  while ((int)ncols < NT + 16) ncols *= 2;

  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 1);
    }
    for (int s = 0; s < M8_SF; ++s) {
      mbar_init(sffull(s), 32);
      mbar_init(sfempty(s), 1);
    }
    mbar_init(done, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc(smem_u32(holder), ncols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *holder;

  if (warp == 0) {
    if (lane == 0) {
      uint32_t issued = 0, issued_par = 0;
      const int ahead = w_early ? min(stages, nk) : 0;
      for (int k = 0; k < ahead; ++k) {
        mbar_expect_tx(full(k), (uint32_t)stage_bytes);
        tma_load_2d(smem_u32(smem + k * stage_bytes), &tmW, full(k), (g0 + k) * 128, mt * M8_BM);
      }
      pdl_wait();
      pdl_trigger();
      int stage = 0;
      uint32_t ph = 0;
      for (int k = 0; k < nk; ++k) {
        if (!mbar_wait(empty(stage), ph ^ 1u, abort_flag, 401)) break;
        issued |= 1u << stage;
        issued_par = (issued_par & ~(1u << stage)) | (ph << stage);
        const uint32_t dst = smem_u32(smem + stage * stage_bytes);
        if (k >= ahead) {
          mbar_expect_tx(full(stage), (uint32_t)stage_bytes);
          tma_load_2d(dst, &tmW, full(stage), (g0 + k) * 128, mt * M8_BM);
        }
        tma_load_2d(dst + M8_A, &tmX, full(stage), (g0 + k) * 128, t0);
        if (++stage == stages) { stage = 0; ph ^= 1u; }
      }
      for (int s = 0; s < stages; ++s)      // nothing of ours is in flight when the CTA ends
        if (issued & (1u << s)) mbar_wait_drain(full(s), (issued_par >> s) & 1u, 402);
    }
    __syncwarp();
  } else if (warp == 1) {
    if (lane == 0) {
      const uint32_t idesc = idesc_mx8(M8_BM, NT);
      int stage = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (int c = 0; c < nchunk && ok; ++c) {
        const int slot = c % M8_SF;
        if (!mbar_wait(sffull(slot), (uint32_t)(c / M8_SF) & 1u, abort_flag, 403)) break;
        if (c >= 2 && !mbar_wait(sfempty((c - 2) % M8_SF), (uint32_t)((c - 2) / M8_SF) & 1u, abort_flag, 404)) break;
        tc_fence_after();
        const uint32_t sfa = tmem + (uint32_t)(NT + 8 * (c & 1)), sfb = sfa + 4;
        copy_scales(sfa, sdesc_scales(smem_u32(sf + slot * 1024)));
        copy_scales(sfb, sdesc_scales(smem_u32(sf + slot * 1024 + 512)));
        for (int j = 0; j < 4 && 4 * c + j < nk; ++j) {
          if (!mbar_wait(full(stage), ph, abort_flag, 405)) { ok = false; break; }
          tc_fence_after();
          const uint32_t a0 = smem_u32(smem + stage * stage_bytes), b0 = a0 + M8_A;
          const int left = cin - (g0 + 4 * c + j) * 128;
          const int steps = left >= 128 ? 4 : left / 32;     // C_in is a multiple of 32
          const uint32_t id = with_byte(idesc, j);
          for (int k = 0; k < steps; ++k)
            mma_mx8(tmem, sdesc(a0 + k * 32, 16, 1024), sdesc(b0 + k * 32, 16, 1024), id, sfa, sfb, (c | j | k) != 0);
          mma_commit(empty(stage));
          if (++stage == stages) { stage = 0; ph ^= 1u; }
        }
        mma_commit(sfempty(slot));
      }
      mma_commit(done);
      mbar_wait_drain(done, 0, 406);
    }
    __syncwarp();
  } else if (warp == 6) {
    pdl_wait();
    bool ok = true;
    for (int c = 0; c < nchunk && ok; ++c) {
      const int slot = c % M8_SF;
      uint32_t w[4], a = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int n = j * 32 + lane, t = t0 + n;
        w[j] = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int g = g0 + 4 * c + k;
          const uint32_t byte = n < NT && t < tokens && g < g1 ? (uint32_t)__ldg(Xs + (size_t)t * G + g) : 127u;
          w[j] |= byte << (8 * k);
        }
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int g = g0 + 4 * c + k;
        a |= (g < g1 ? (uint32_t)__ldg(Ws + (size_t)mt * G + g) : 127u) << (8 * k);
      }
      ok = warp_all(mbar_wait(sfempty(slot), (uint32_t)(c / M8_SF + 1) & 1u, abort_flag, 407));
      if (ok) {
        reinterpret_cast<uint4*>(sf + slot * 1024)[lane] = make_uint4(a, a, a, a);
        reinterpret_cast<uint4*>(sf + slot * 1024 + 512)[lane] = make_uint4(w[0], w[1], w[2], w[3]);
        fence_async_smem();
        mbar_arrive(sffull(slot));
      }
    }
  } else {
    const int q = warp & 3;
    const int o = mt * M8_BM + q * 32 + lane;
    const bool ok = warp_all(mbar_wait(done, 0, abort_flag, 408));
    tc_fence_after();
    float* part = reinterpret_cast<float*>(smem);    // every stage has been read
    if (ok) {
      for (int n0 = 0; n0 < NT && t0 + n0 < tokens; n0 += 16) {
        uint32_t r[16];
        tmem_ld16(tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)n0, r);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int t = t0 + n0 + i;
          if (S > 1) part[(n0 + i) * 128 + q * 32 + lane] = __uint_as_float(r[i]);
          else if (t < tokens && o < cout) Y[(size_t)t * cout + o] = from_f32<OUT>(__uint_as_float(r[i]));
        }
      }
    }
  }
  tc_fence_before();
  if (S > 1) {
    cluster_sync_all();     // every CTA's partial result is written
    if (warp >= 2 && warp < 6) {
      const int i = (warp - 2) * 32 + lane, o = mt * M8_BM + i;
      const uint32_t mine = smem_u32(smem) + 4u * (uint32_t)i;
      for (int n = rank; n < NT && t0 + n < tokens; n += S) {
        float v[8];
#pragma unroll
        for (int r = 0; r < 8; ++r) v[r] = r < S ? ld_cluster_f32(mapa(mine + (uint32_t)n * 512u, (uint32_t)r)) : 0.f;
        float s = v[0];
#pragma unroll
        for (int r = 1; r < 8; ++r) s += v[r];
        if (o < cout) Y[(size_t)(t0 + n) * cout + o] = from_f32<OUT>(s);
      }
    }
    cluster_sync_all();     // no CTA leaves while another reads its partial result
  } else {
    __syncthreads();
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, ncols);
  }
}

// 2-D map over a row-major [rows, cin] matrix of bytes: boxes of 128 channels x `by` rows, 128-byte swizzle.
lcp_status make_map8(CUtensorMap* m, const void* base, int cin, int rows, int by, const char* what) {
  EncodeFn fn = encode_fn();
  if (!fn) return fail(LCP_ERR_CUDA, "%s: cuTensorMapEncodeTiled is unavailable from the driver", what);
  const cuuint64_t dims[2] = {(cuuint64_t)cin, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)cin};
  const cuuint32_t box[2] = {128, (cuuint32_t)by};
  const cuuint32_t es[2] = {1, 1};
  const CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, es,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(LCP_ERR_CUDA, "%s: cuTensorMapEncodeTiled failed (%d)", what, (int)r);
  return LCP_OK;
}

template <typename OUT>
lcp_status split_t(const uint8_t* Xq, const uint8_t* Xs, const uint8_t* Wq, const uint8_t* Ws, OUT* Y, int cout, int cin,
                   int tokens, bool w_early, cudaStream_t st) {
  const int NT = tokens >= 128 ? 128 : (tokens + 15) / 16 * 16;
  CUtensorMap mW, mX;
  TC_TRY(make_map8(&mW, Wq, cin, cout, M8_BM, "mm8 W"));
  TC_TRY(make_map8(&mX, Xq, cin, tokens, NT, "mm8 X"));
  const long long tiles = (long long)cdiv(cout, M8_BM) * cdiv(tokens, NT);
  const int G = cdiv(cin, 128);
  // narrow tiles: two CTAs an SM, so that one's loads cover the other's set-up and epilogue
  const int stage_bytes = M8_A + NT * 128;
  const int per_sm = NT <= 32 ? 2 : 1;
  int stages = (per_sm == 2 ? 104 * 1024 : 208 * 1024) / stage_bytes;
  if (stages > M8_MAX_STAGES) stages = M8_MAX_STAGES;
  int S = 1;
  while (S < 8 && tiles * S * 2 <= (long long)per_sm * num_sms() && G >= 4 * S) S *= 2;
  const int smem = stages * stage_bytes + M8_SF * 1024 + 1024 + 512;
  TC_TRY(set_smem(mm8_split_kernel<OUT>, smem, "mm8"));
  return launch_kernel(mm8_split_kernel<OUT>, dim3((unsigned)(tiles * S)), dim3(M8_THREADS), (size_t)smem, st, S, true,
                       "mm8", mW, mX, Xs, Ws, Y, cout, cin, tokens, NT, stages, S, w_early ? 1 : 0);
}

}  // namespace

lcp_status tc_error_mm8(int* site, int reset) { return read_tc_error(site, reset); }

lcp_status launch_mm8(const uint8_t* Xq, const uint8_t* Xs, const uint8_t* Wq, const uint8_t* Ws, void* Y, int cout,
                      int cin, int tokens, lcp_dtype ydt, bool w_early, cudaStream_t st) {
  if (ydt == LCP_F32) return split_t(Xq, Xs, Wq, Ws, static_cast<float*>(Y), cout, cin, tokens, w_early, st);
  return split_t(Xq, Xs, Wq, Ws, static_cast<__nv_bfloat16*>(Y), cout, cin, tokens, w_early, st);
}

}  // namespace lcp
