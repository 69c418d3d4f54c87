// Products of 8-bit operands with a power-of-two scale for each block of 128:
//
//   Y[t][o] = sum over groups g of  2^(kx[t][g] + kw[o / 128][g])
//             * sum over the 128 channels c of group g of  qx[t][c] qw[o][c]
//
// on the tensor cores (tcgen05.mma kind::mxf8f6f4, block scaled): the scales are
// e8m0 bytes, the format the instruction multiplies in by itself, so the
// accumulation over all of C_in stays in one float32 accumulator in tensor
// memory.  An addition there may truncate: an output is within (C_in / 32 + 40) 2^-23 of the sum of its
// terms' magnitudes (C_in = 5120: off by 7e-7 of the outputs' size, a plain float32 product by 1.5e-7).
// Output channels are the M side (128 lanes of tensor memory) and
// tokens the N side, whose width follows the token count; one lane is one
// channel, so a warp's store of one token is 32 consecutive channels of Y.

#include <algorithm>

#include "quant8.cuh"
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
// The same on a CTA pair: M = 256, each CTA's 128 rows of A, half of B's rows, A scales of its
// own rows and B scales of all N rows.
__device__ __forceinline__ void mma_mx8_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa,
                                             uint32_t sfb, bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate ? 1u : 0u)
      : "memory");
}
// Each CTA of the pair copies from its own shared memory into its own tensor memory.
__device__ __forceinline__ void copy_scales_pair(uint32_t taddr, uint64_t sd) {
  asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(sd) : "memory");
}
// Arrival on, and wait for, a barrier of the pair that announces plain shared-memory writes of
// either CTA (cluster scope).
__device__ __forceinline__ void mbar_arrive_release_cluster(uint32_t bar_cluster) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar_cluster) : "memory");
}
__device__ __forceinline__ bool mbar_try_wait_cluster(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
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

// One thread of a converged warp.  The loops that issue TMA copies and products run on it: a
// region the compiler knows to be one thread's issues a product in ~40 cycles, one under
// `lane == 0` in ~75 (its operands move to uniform registers one by one), which would bound the
// kernels (measured on four products and a commit: 157 cycles against 305).
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}

// Waits of those two threads.  Their loops have no exit on a wait that gave up: a break there makes
// the loop's values per-thread ones again (338 cycles against 206 for a wait, four products and a
// commit).  Instead, once a wait of the CTA has given up, each later one returns at once, and the
// loops run out over operands that are no longer meant to be right.  The four groups of a whole
// chunk are written out for the same reason (468 cycles a group in a loop, 200 written out).
__device__ __noinline__ void wait_slow(uint32_t bar, uint32_t parity, volatile int* abort_flag, int site) {
  if (!*abort_flag) mbar_wait_slow(bar, parity, abort_flag, site);
}
__device__ __forceinline__ void wait_through(uint32_t bar, uint32_t parity, volatile int* abort_flag, int site) {
  if (!mbar_try_wait(bar, parity)) wait_slow(bar, parity, abort_flag, site);
}
// The same on a barrier that announces plain writes of both CTAs of a pair.
__device__ __noinline__ void wait_slow_cluster(uint32_t bar, uint32_t parity, volatile int* abort_flag, int site) {
  if (!*abort_flag) mbar_wait_slow(bar, parity, abort_flag, site);
  mbar_try_wait_cluster(bar, parity);     // the acquire of the completed phase
}
__device__ __forceinline__ void wait_through_cluster(uint32_t bar, uint32_t parity, volatile int* abort_flag, int site) {
  if (!mbar_try_wait_cluster(bar, parity)) wait_slow_cluster(bar, parity, abort_flag, site);
}

constexpr int M8_BM = 128;            // output channels of a CTA: one row of weight scales
constexpr int M8_A = M8_BM * 128;     // bytes of a stage's weight tile (one scale group of channels)
constexpr int M8_SF = 4;              // ring of scale chunks (four groups each)
constexpr int M8_MAX_STAGES = 12;
constexpr int M8_RING = 210 * 1024, M8_HALF_RING = 96 * 1024;      // bytes of the operand ring: one CTA an SM, two
constexpr int M8_FUSED_TOKENS = 8;    // plain activations of up to so many tokens are quantised by the product itself
                                      // (8 tokens x 4096 x 11008: 12.3 us; 16: 17.0, 13.2 as two launches)
constexpr int M8_FUSED_WARPS = 8;     // warps that do (16 leave one CTA an SM: 16.2 us, 6.9 then, at 4096 x 4096)
// Every how many pairs of groups a quantising warp takes, where warps go round npp pairs of tokens and a ring
// of `stages` tiles.
__host__ __device__ constexpr int fused_every(int stages, int npp) {
  int every = M8_FUSED_WARPS / npp;
  while (2 * every > stages) every /= 2;
  return every;
}
constexpr bool fused_ring_ok(int bytes) {      // for one pair of tokens, where `every` is largest
  const int stages = bytes / (M8_A + 16 * 128);
  return stages <= M8_MAX_STAGES && 2 * fused_every(stages, 1) + stages <= 19;
}
static_assert(M8_FUSED_TOKENS <= 16 && fused_ring_ok(M8_RING) && fused_ring_ok(M8_HALF_RING),
              "an arrival for a missing pair of groups could fall into an older phase");
// warp 0: TMA, 1: MMA, 2-5: epilogue; 6: scales, or all from 2 on: quantisers
template <typename XT> constexpr int m8_threads() { return sizeof(XT) == 1 ? 224 : 64 + 32 * M8_FUSED_WARPS; }
constexpr int M8_SETS = 4;            // sets of scales in tensor memory

__device__ __forceinline__ float4 ld_cluster_f32x4(uint32_t a) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a));
  return v;
}
// Four consecutive outputs, `left` of them inside the row; whole rows of four are aligned.
template <typename OUT> __device__ __forceinline__ void store4(OUT* out, const float4& s, int left, bool whole) {
  if (whole) {
    if (left <= 0) return;
    if constexpr (sizeof(OUT) == 4) *reinterpret_cast<float4*>(out) = s;
    else *reinterpret_cast<uint2*>(out) = make_uint2(pack_bf16x2(s.x, s.y), pack_bf16x2(s.z, s.w));
    return;
  }
  const float v[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (i < left) out[i] = from_f32<OUT>(v[i]);
}

// One CTA: 128 output channels x NT tokens over a range of scale groups; the S CTAs of a
// cluster share a tile and split its groups, then each adds the S partial results of its
// tokens in rank order.
//
// Scale words: a chunk is four groups, so a row's four scale bytes are one 32-bit word and
// the instruction picks the byte of the group at hand.  Warp 6 builds the words of chunk c in
// ring slot c % 4 once the products of chunk c - 4 are done, and the MMA thread copies them to
// the tensor-memory set of the same number, which those products were the last to read.
//
// XT = uint8_t: X and Xs hold quantised activations; the tiles of X come by TMA, and warp 6
// builds the scale words.  XT = float or bf16 (at most 8 tokens): X holds the activations
// themselves, and eight warps quantise the CTA's channels (permuted, if PERM) straight into the
// tiles and scale words.  Every CTA of a column of tiles quantises the same tokens again, 8 at
// the most: that costs less than a launch that does it once (one token x 4096 x 4096: 6.4 us, 8.0
// as two launches).
template <typename OUT, typename XT, bool PERM>
__global__ void __launch_bounds__(m8_threads<XT>())
mm8_split_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                 const XT* __restrict__ X, const int32_t* __restrict__ perm, int bmask, const uint8_t* __restrict__ Xs,
                 const uint8_t* __restrict__ Ws, OUT* __restrict__ Y, int cout, int cin, int tokens, int NT, int stages,
                 int S, int w_early) {
  constexpr bool FUSED = sizeof(XT) != 1;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align1024(smem_raw);
  const int stage_bytes = M8_A + NT * 128;
  uint8_t* sf = smem + stages * stage_bytes;                  // M8_SF x (512 B of W, 512 B of X)
  uint32_t* exchange = reinterpret_cast<uint32_t*>(sf + M8_SF * 1024);   // PERM: a buffer for each quantising warp
  uint64_t* bars = reinterpret_cast<uint64_t*>(exchange + (PERM ? M8_FUSED_WARPS * Q8_STAGE : 0));
  uint32_t* holder = reinterpret_cast<uint32_t*>(bars + 2 * M8_MAX_STAGES + 2 * M8_SF + 1);
  static_assert(M8_SETS == M8_SF, "a ring slot and a set are both free when the same products are done");
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
  // whole pairs of groups (a permutation's blocks are at most 256 channels); never empty: 3 S <= G
  const int G2 = cdiv(G, 2);
  const int g0 = 2 * (int)((long long)rank * G2 / S), g1 = min(G, 2 * (int)((long long)(rank + 1) * G2 / S));
  const int npairs = (tokens + 1) / 2;     // FUSED: pairs of tokens, one for a warp or for several
  const int nk = g1 - g0, nchunk = cdiv(nk, 4);

  // accumulator columns [0, NT), then M8_SETS sets of (4 columns of W scales, 4 of X scales)
  uint32_t ncols = 32;
  while ((int)ncols < NT + 8 * M8_SETS) ncols *= 2;

  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) {
      mbar_init(full(s), FUSED ? 1 + npairs : 1);
      mbar_init(empty(s), 1);
    }
    for (int s = 0; s < M8_SF; ++s) {
      mbar_init(sffull(s), FUSED ? 2 * npairs : 32);
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
    if (elect_one()) {
      uint32_t issued = 0, issued_par = 0;
      const uint32_t bytes = FUSED ? M8_A : (uint32_t)stage_bytes;
      const int ahead = w_early ? min(stages, nk) : 0;
      for (int k = 0; k < ahead; ++k) {
        mbar_expect_tx(full(k), bytes);
        tma_load_2d(smem_u32(smem + k * stage_bytes), &tmW, full(k), (g0 + k) * 128, mt * M8_BM);
      }
      pdl_wait();
      pdl_trigger();
      int stage = 0;
      uint32_t ph = 0;
      for (int k = 0; k < nk; ++k) {
        wait_through(empty(stage), ph ^ 1u, abort_flag, 401);
        issued |= 1u << stage;
        issued_par = (issued_par & ~(1u << stage)) | (ph << stage);
        const uint32_t dst = smem_u32(smem + stage * stage_bytes);
        if (k >= ahead) {
          mbar_expect_tx(full(stage), bytes);
          tma_load_2d(dst, &tmW, full(stage), (g0 + k) * 128, mt * M8_BM);
        }
        if (!FUSED) tma_load_2d(dst + M8_A, &tmX, full(stage), (g0 + k) * 128, t0);
        if (++stage == stages) { stage = 0; ph ^= 1u; }
      }
      for (int s = 0; s < stages; ++s)      // nothing of ours is in flight when the CTA ends
        if (issued & (1u << s)) mbar_wait_drain(full(s), (issued_par >> s) & 1u, 402);
    }
    __syncwarp();
  } else if (warp == 1) {
    if (elect_one()) {
      const uint32_t idesc = idesc_mx8(M8_BM, NT);
      const uint64_t wd0 = sdesc(smem_u32(smem), 16, 1024), xd0 = sdesc(smem_u32(smem) + M8_A, 16, 1024);
      int stage = 0;
      uint32_t ph = 0;
      for (int c = 0; c < nchunk; ++c) {
        const int slot = c % M8_SF;
        wait_through(sffull(slot), (uint32_t)(c / M8_SF) & 1u, abort_flag, 403);
        tc_fence_after();
        const uint32_t sfa = tmem + (uint32_t)(NT + 8 * slot), sfb = sfa + 4;
        copy_scales(sfa, sdesc_scales(smem_u32(sf + slot * 1024)));
        copy_scales(sfb, sdesc_scales(smem_u32(sf + slot * 1024 + 512)));
        auto group = [&](int j, int steps) {      // the products of group j of the chunk, 32 channels a step
          wait_through(full(stage), ph, abort_flag, 405);
          tc_fence_after();
          const uint64_t wd = wd0 + (uint32_t)(stage * (stage_bytes >> 4)), xd = xd0 + (uint32_t)(stage * (stage_bytes >> 4));
          const uint32_t id = with_byte(idesc, j);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (k < steps) mma_mx8(tmem, wd + 2 * k, xd + 2 * k, id, sfa, sfb, (c | j | k) != 0);
          mma_commit(empty(stage));
          if (++stage == stages) { stage = 0; ph ^= 1u; }
        };
        const int left = min(nk * 128, cin - g0 * 128) - 512 * c;      // channels from this chunk on
        if (left >= 512) {
#pragma unroll
          for (int j = 0; j < 4; ++j) group(j, 4);
        } else {                                                       // C_in is a multiple of 32
#pragma unroll 1
          for (int j = 0; 128 * j < left; ++j) group(j, min(4, (left - 128 * j) / 32));
        }
        mma_commit(sfempty(slot));
      }
      mma_commit(done);
      mbar_wait_drain(done, 0, 406);
    }
    __syncwarp();
  } else if (!FUSED && warp == 6) {
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
    if constexpr (FUSED) {
      // Warps from 2 on: warp w takes the pair of tokens w % npp (npp: npairs rounded up to a power of two) and
      // every `every`-th pair of groups, the next one's values, permutation and scales of W loading meanwhile
      // (5 to 12 % of the kernel's time at one token; two ahead measured no better).  At most M8_FUSED_WARPS / npp warps
      // share a pair of tokens, and no more than stages / 2: a warp that waits for a tile knows from its
      // own wait before, 2 every groups back, that the tile's use before the last is over, so the parity
      // it waits for cannot be an older phase's.
      // A last chunk of one or two groups lacks its second pair, whose warp arrives on sffull without a wait.
      // That must not fall into the phase before, of chunk c - 4: the warp's own last wait, for the tile of group
      // 4 c + 3 - 2 every, says that the products of `stages` groups earlier are done, and so the words of their
      // chunk complete.  They are no earlier than chunk c - 4 where 2 every + stages <= 19 (asserted at fused_every).
      pdl_wait();
      const int w = warp - 2;
      int npp = 1;
      while (npp < npairs) npp *= 2;
      const int pair = w % npp;
      const int every = fused_every(stages, npp);
      uint32_t* buf = exchange + (PERM ? w * Q8_STAGE : 0);
      const int row0 = 2 * pair;
      auto load = [&](int p, int u) {
        const int chan = (g0 + 2 * p) * 128 + 8 * lane;
        return 2 * p < nk && chan < cin && row0 + u < tokens ? load8(X + (size_t)(row0 + u) * cin + chan) : zero8<XT>();
      };
      const auto scales = [&](int p) {      // W's two scale bytes
        const uint8_t* ws = Ws + (size_t)mt * G + g0 + 2 * p;
        return pair == 0 && 2 * p < nk ? (uint32_t)__ldg(ws) | (2 * p + 1 < nk ? (uint32_t)__ldg(ws + 1) : 127u) << 8 : 0u;
      };
      const auto entries = [&](int p) {
        return PERM ? load_perm(perm, 2 * p < nk ? (g0 + 2 * p) * 128 + 8 * lane : cin, lane, cin) : Perm8{};
      };
      int p = pair < npairs && w / npp < every ? w / npp : 2 * nchunk;
      Vec8<XT> next[2] = {load(p, 0), load(p, 1)};
      Perm8 next_perm = entries(p);
      uint32_t next_scales = scales(p);
      for (; p < 2 * nchunk; p += every) {
        Vec8<XT> v[2] = {next[0], next[1]};
        const Perm8 places = next_perm;
        const uint32_t a = next_scales;
        next[0] = load(p + every, 0);
        next[1] = load(p + every, 1);
        next_perm = entries(p + every);
        next_scales = scales(p + every);
        const int c = p / 2, slot = c % M8_SF, chan = (g0 + 2 * p) * 128 + 8 * lane;
        if (2 * p < nk) {
          if (PERM) {
            uint32_t to[8];
            perm_slots(places, chan < cin, lane, bmask, buf, to, &g_tc_error);
            permute_rows(v[0], v[1], to, buf, lane);
          }
          uint32_t m[2];
          group_max(v, m);
          // the tile and slot are free once the products that read them last are done
          const int k = 2 * p + (lane >> 4), s0 = 2 * p % stages, s1 = s0 + 1 == stages ? 0 : s0 + 1;
          bool ok = mbar_wait(empty(s0), (uint32_t)(2 * p / stages + 1) & 1u, abort_flag, 409);
          if (2 * p + 1 < nk) ok = mbar_wait(empty(s1), (uint32_t)((2 * p + 1) / stages + 1) & 1u, abort_flag, 409) && ok;
          ok = mbar_wait(sfempty(slot), (uint32_t)(c / M8_SF + 1) & 1u, abort_flag, 410) && ok;
          if (!warp_all(ok)) break;
          uint8_t* words = sf + slot * 1024;
          uint8_t* tile = smem + (lane < 16 ? s0 : s1) * stage_bytes + M8_A;
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const int row = row0 + u;
            if (k >= nk || row >= tokens) break;
            const uint32_t byte = scale_byte(m[u]);
            *reinterpret_cast<uint2*>(tile + row * 128 + ((((lane & 15) >> 1) ^ (row & 7)) << 4) + (lane & 1) * 8) =
                to_e4m3(v[u], scale_inverse(byte));
            if ((lane & 15) == 0) words[512 + row * 16 + 2 * (p & 1) + (lane >> 4)] = (uint8_t)byte;
          }
          if (pair == 0) {
#pragma unroll
            for (int j = 0; j < 4; ++j) *reinterpret_cast<uint16_t*>(words + lane * 16 + 4 * j + 2 * (p & 1)) = (uint16_t)a;
          }
          fence_async_smem();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(full(s0));
            if (2 * p + 1 < nk) mbar_arrive(full(s1));
          }
        }
        if (lane == 0) mbar_arrive(sffull(slot));     // also for the missing half of the last chunk
      }
    }
    if (warp < 6) {
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
  }
  tc_fence_before();
  if (S > 1) {
    cluster_sync_all();     // every CTA's partial result is written
    // a warp adds a token's 128 channels, four a lane; the tokens of this rank go round the warps
    const uint32_t mine = smem_u32(smem) + 16u * (uint32_t)lane;
    const int o = mt * M8_BM + 4 * lane;
    const int nmax = min(NT, tokens - t0);
#pragma unroll 2
    for (int n = rank + S * warp; n < nmax; n += S * (m8_threads<XT>() / 32)) {
      float4 v[8];
#pragma unroll
      for (int r = 0; r < 8; ++r)
        if (r < S) v[r] = ld_cluster_f32x4(mapa(mine + (uint32_t)n * 512u, (uint32_t)r));
      float4 s = v[0];
#pragma unroll
      for (int r = 1; r < 8; ++r)
        if (r < S) {
          s.x += v[r].x;
          s.y += v[r].y;
          s.z += v[r].z;
          s.w += v[r].w;
        }
      store4(Y + (size_t)(t0 + n) * cout + o, s, cout - o, (cout & 3) == 0);
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

// Four scale bytes of a row staged in shared memory, groups g .. g + 3 (unit scale past the last
// group).  The aligned words around them are read whole: up to seven bytes past the row, which
// is still shared memory of the kernel.
__device__ __forceinline__ uint32_t scale_word(const uint8_t* row, int g, int G) {
  const uint32_t a = smem_u32(row + g), b = a & ~3u;
  uint32_t lo, hi;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(lo) : "r"(b));
  if ((G & 3) == 0) return lo;                                   // rows 4-byte aligned, g a multiple of 4
  asm volatile("ld.shared.u32 %0, [%1+4];" : "=r"(hi) : "r"(b));
  const uint32_t w = __funnelshift_r(lo, hi, 8u * (a & 3u));
  const int left = G - g;
  return left >= 4 ? w : (w & ~(0xffffffffu << (8 * left))) | (0x7f7f7f7fu << (8 * left));
}
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}

// Many tokens: persistent CTA pairs (cta_group::2) on tiles of 256 output channels x N tokens.
// Each CTA stages its 128 rows of W and its half of the tile's tokens, the leader issues
// M = 256 products over both, and each CTA keeps its 128 channels x N tokens of the result in one
// of two accumulators, so the next tile's products run while the epilogue stores this one.
// Columns: two accumulators of N, then the sets of scales (4 of W, 8 of X): two at the least, so N <= 240.
constexpr int P8_THREADS = 320;       // warp 0: TMA, 1: MMA, 2-5: epilogue, 6-9: scales (128 tokens, every other slot)
constexpr int P8_SF_BYTES = 1536;     // a chunk's scale words: 512 B of W, 2 x 512 B of X
constexpr int P8_SLOT = 4;            // chunks of a ring slot: one hand-over between the CTAs for 16 groups
constexpr int P8_SLOTS = 2;
constexpr int P8_MAX_SETS = 8;        // sets of scales in tensor memory: as many as fit beside the accumulators
constexpr int P8_MAX_N = 240;
constexpr int P8_MAX_G = 256;         // C_in <= 32768: a tile's scale bytes are staged whole
constexpr int P8_RAW = 40 * 1024;     // their room at most: N G <= 40 KB
constexpr int P8_MAX_STAGES = 10;

template <typename OUT>
__global__ void __launch_bounds__(P8_THREADS, 1)
mm8_pair_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                const uint8_t* __restrict__ Xs, const uint8_t* __restrict__ Ws, OUT* __restrict__ Y, int cout, int cin,
                int tokens, int N, int stages, int raw_bytes, int tokens_fast) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align1024(smem_raw);
  const int stage_bytes = M8_A + N * 64;
  uint8_t* sf = smem + stages * stage_bytes;
  uint8_t* wraw = sf + P8_SLOTS * P8_SLOT * P8_SF_BYTES;      // the tile's W scales (one row), then its X scales (N rows)
  uint8_t* xraw = wraw + P8_MAX_G;
  uint64_t* bars = reinterpret_cast<uint64_t*>(xraw + raw_bytes);
  uint32_t* holder = reinterpret_cast<uint32_t*>(bars + 2 * P8_MAX_STAGES + 2 * P8_SLOTS + 6 + P8_MAX_SETS);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(holder + 1);
  auto full = [&](int s) { return smem_u32(bars + s); };                       // leader's counts both CTAs' halves
  auto empty = [&](int s) { return smem_u32(bars + P8_MAX_STAGES + s); };      // one per CTA
  auto sffull = [&](int s) { return smem_u32(bars + 2 * P8_MAX_STAGES + s); }; // leader's counts four warps
  auto sfempty = [&](int s) { return smem_u32(bars + 2 * P8_MAX_STAGES + P8_SLOTS + s); };
  uint64_t* rest = bars + 2 * P8_MAX_STAGES + 2 * P8_SLOTS;
  auto tfull = [&](int a) { return smem_u32(rest + a); };
  auto tempty = [&](int a) { return smem_u32(rest + 2 + a); };                 // leader: eight warps
  const uint32_t drain = smem_u32(rest + 4), rawfull = smem_u32(rest + 5);
  auto setfree = [&](int a) { return smem_u32(rest + 6 + a); };                // leader: a set of scales in tensor memory

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const uint32_t rank = cluster_rank();
  const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;
  const int G = cdiv(cin, 128), nchunk = cdiv(G, 4);
  const int mtiles = cdiv(cout, 2 * M8_BM), ntiles = cdiv(tokens, N);
  const int total = mtiles * ntiles;

  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) {
      mbar_init(full(s), 2);
      mbar_init(empty(s), 1);
    }
    for (int s = 0; s < P8_SLOTS; ++s) {
      mbar_init(sffull(s), 4);
      mbar_init(sfempty(s), 1);
    }
    for (int a = 0; a < P8_MAX_SETS; ++a) mbar_init(setfree(a), 1);
    for (int a = 0; a < 2; ++a) {
      mbar_init(tfull(a), 1);
      mbar_init(tempty(a), 8);
    }
    mbar_init(drain, 1);
    mbar_init(rawfull, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc_pair(smem_u32(holder), 512);
  tc_fence_before();
  cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem = *holder;
  pdl_wait();
  pdl_trigger();
  auto tile_at = [&](int it, int& mt, int& nt) {
    if (tokens_fast) {
      nt = it % ntiles;
      mt = it / ntiles;
    } else {
      mt = it % mtiles;
      nt = it / mtiles;
    }
  };

  if (warp == 0) {
    if (elect_one()) {
      int stage = 0;
      uint32_t ph = 0, issued = 0, issued_par = 0;
      const uint32_t full0 = mapa(full(0), 0);
      for (int it = pair; it < total; it += npairs) {
        int mt, nt;
        tile_at(it, mt, nt);
        const int wrow = mt * 2 * M8_BM + (int)rank * M8_BM, xrow = nt * N + (int)rank * (N / 2);
#pragma unroll 4
        for (int g = 0; g < G; ++g) {
          wait_through(empty(stage), ph ^ 1u, abort_flag, 411);
          issued |= 1u << stage;
          issued_par = (issued_par & ~(1u << stage)) | (ph << stage);
          const uint32_t fbar = full0 + 8u * (uint32_t)stage;
          mbar_expect_tx_cluster(fbar, (uint32_t)stage_bytes);
          const uint32_t dst = smem_u32(smem + stage * stage_bytes);
          tma_load_2d_pair(dst, &tmW, fbar, g * 128, wrow);
          tma_load_2d_pair(dst + M8_A, &tmX, fbar, g * 128, xrow);
          if (++stage == stages) { stage = 0; ph ^= 1u; }
        }
      }
      // our copies have landed once the leader's full barrier has completed, or once our own
      // empty barrier shows that the leader consumed them
      for (int s = 0; s < stages; ++s)
        if (issued & (1u << s)) mbar_wait_drain(rank == 0 ? full(s) : empty(s), (issued_par >> s) & 1u, 412);
    }
    __syncwarp();
  } else if (warp == 1) {
    if (rank == 0 && elect_one()) {
      const uint32_t idesc = idesc_mx8(2 * M8_BM, N);
      const uint64_t wd0 = sdesc(smem_u32(smem), 16, 1024), xd0 = sdesc(smem_u32(smem) + M8_A, 16, 1024);
      int stage = 0, lt = 0;
      uint32_t ph = 0;
      const int sets = min(P8_MAX_SETS, (512 - 2 * N) / 12);
      int set = 0;
      uint32_t sph = 1, ss = 0;     // parity of the set's last use; ring slots so far, over all tiles
      for (int it = pair; it < total; it += npairs, ++lt) {
        const int acc = lt & 1;
        wait_through(tempty(acc), ((uint32_t)(lt >> 1) & 1u) ^ 1u, abort_flag, 413);
        tc_fence_after();
        const uint32_t d = tmem + (uint32_t)(acc * N);
        for (int c = 0; c < nchunk; ++c) {
          const int slot = (int)(ss % P8_SLOTS);
          if (c % P8_SLOT == 0) wait_through_cluster(sffull(slot), (ss / P8_SLOTS) & 1u, abort_flag, 414);
          wait_through(setfree(set), sph, abort_flag, 415);     // the products that read this set last
          tc_fence_after();
          const uint32_t sfa = tmem + (uint32_t)(2 * N + 12 * set), sfb = sfa + 4;
          const uint32_t src = smem_u32(sf + (slot * P8_SLOT + c % P8_SLOT) * P8_SF_BYTES);
          copy_scales_pair(sfa, sdesc_scales(src));
          copy_scales_pair(sfb, sdesc_scales(src + 512));
          if (N > 128) copy_scales_pair(sfb + 4, sdesc_scales(src + 1024));
          auto group = [&](int j, int steps) {      // the products of group j of the chunk, 32 channels a step
            wait_through(full(stage), ph, abort_flag, 416);
            tc_fence_after();
            const uint64_t wd = wd0 + (uint32_t)(stage * (stage_bytes >> 4)), xd = xd0 + (uint32_t)(stage * (stage_bytes >> 4));
            const uint32_t id = with_byte(idesc, j);
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (k < steps) mma_mx8_pair(d, wd + 2 * k, xd + 2 * k, id, sfa, sfb, (c | j | k) != 0);
            mma_commit_pair(empty(stage), 0x3);
            if (++stage == stages) { stage = 0; ph ^= 1u; }
          };
          const int left = cin - 512 * c;
          if (left >= 512) {
#pragma unroll
            for (int j = 0; j < 4; ++j) group(j, 4);
          } else {
#pragma unroll 1
            for (int j = 0; 128 * j < left; ++j) group(j, min(4, (left - 128 * j) / 32));
          }
          mma_commit_pair(setfree(set), 0x1);
          if (++set == sets) { set = 0; sph ^= 1u; }
          if (c % P8_SLOT == P8_SLOT - 1 || c == nchunk - 1) {
            mma_commit_pair(sfempty(slot), 0x3);
            ++ss;
          }
        }
        mma_commit_pair(tfull(acc), 0x3);
      }
      mma_commit_pair(drain, 0x1);
      mbar_wait_drain(drain, 0, 417);
    }
    __syncwarp();
  } else if (warp >= 6) {
    // The tile's scale bytes, N rows of G bytes one after another, come in by one bulk copy (N and
    // so the start are multiples of 16; the up to 15 bytes behind the last whole 16 of X's scales by
    // plain loads).  Each warp then builds its 128 tokens' words (n = 128 half + 32 j + lane) of every
    // other ring slot, ahead of the products, which hides the next tile's copy.
    const int half = (warp - 6) & 1, odd = (warp - 6) >> 1;
    const uint32_t sffull0 = mapa(sffull(0), 0);
    uint32_t ss = 0, par = 0;
    bool ok = true;
    for (int it = pair; it < total; it += npairs, par ^= 1u) {
      // The four warps are done with the tile before, and they leave together once a wait of any of them has
      // given up: a warp that left alone would keep the others at the barrier, which has no limit.
      if (!named_and(1, 128, ok)) break;
      int mt, nt;
      tile_at(it, mt, nt);
      const int wblock = 2 * mt + (int)rank, rows = min(N, tokens - nt * N);
      const uint8_t* src = Xs + (size_t)nt * N * G;
      const uint32_t bytes = (uint32_t)(rows * G), bulk = bytes & ~15u;
      if (warp == 6) {
        if (bulk && elect_one()) {
          mbar_expect_tx(rawfull, bulk);
          bulk_load(smem_u32(xraw), src, bulk, rawfull);
        }
        if (!bulk && lane == 0) mbar_arrive(rawfull);
        for (int i = lane; i < G; i += 32) wraw[i] = wblock * M8_BM < cout ? __ldg(Ws + (size_t)wblock * G + i) : 127;
      } else if (warp == 7 && bulk + lane < bytes) {
        xraw[bulk + lane] = __ldg(src + bulk + lane);
      }
      named_sync(1, 128);
      ok = warp_all(mbar_wait(rawfull, par, abort_flag, 420));
      const uint8_t* row[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int n = half * 128 + j * 32 + lane;
        row[j] = n < rows ? xraw + n * G : nullptr;
      }
      for (int c0 = 0; c0 < nchunk && ok; c0 += P8_SLOT, ++ss) {
        if ((int)(ss & 1u) != odd) continue;
        const int slot = (int)(ss % P8_SLOTS);
        ok = warp_all(mbar_wait(sfempty(slot), (ss / P8_SLOTS + 1) & 1u, abort_flag, 418));
        if (!ok) break;
#pragma unroll
        for (int i = 0; i < P8_SLOT; ++i) {
          const int c = c0 + i;
          if (c >= nchunk) break;
          uint8_t* dst = sf + (slot * P8_SLOT + i) * P8_SF_BYTES;
          uint32_t w[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) w[j] = row[j] ? scale_word(row[j], 4 * c, G) : 0x7f7f7f7fu;
          reinterpret_cast<uint4*>(dst + 512 + 512 * half)[lane] = make_uint4(w[0], w[1], w[2], w[3]);
          if (half == 0) {
            const uint32_t a = scale_word(wraw, 4 * c, G);
            reinterpret_cast<uint4*>(dst)[lane] = make_uint4(a, a, a, a);
          }
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive_release_cluster(sffull0 + 8u * (uint32_t)slot);
      }
      if (!ok && warp == 6) mbar_wait_drain(rawfull, par, 421);     // nothing of ours in flight when the CTA ends
    }
  } else {
    const int q = warp & 3;
    const uint32_t tempty_leader0 = mapa(tempty(0), 0), tempty_leader1 = mapa(tempty(1), 0);
    int lt = 0;
    for (int it = pair; it < total; it += npairs, ++lt) {
      const int acc = lt & 1;
      if (!warp_all(mbar_wait(tfull(acc), (uint32_t)(lt >> 1) & 1u, abort_flag, 419))) break;
      tc_fence_after();
      int mt, nt;
      tile_at(it, mt, nt);
      const int o = mt * 2 * M8_BM + (int)rank * M8_BM + q * 32 + lane;
      const uint32_t base = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(acc * N);
      const int nmax = tokens - nt * N < N ? tokens - nt * N : N;
      // 16 tokens a step; the next step's accumulators are on their way while this one's are stored
      OUT* out = Y + (size_t)nt * N * cout + o;
      auto store16 = [&](const uint32_t(&r)[16], int n0) {
        if (o < cout) {
          if (n0 + 16 <= nmax) {
#pragma unroll
            for (int i = 0; i < 16; ++i) out[(size_t)i * cout] = from_f32<OUT>(__uint_as_float(r[i]));
          } else {
#pragma unroll
            for (int i = 0; i < 16; ++i)
              if (n0 + i < nmax) out[(size_t)i * cout] = from_f32<OUT>(__uint_as_float(r[i]));
          }
        }
        out += 16 * (size_t)cout;
      };
      uint32_t ra[16], rb[16];
      tmem_ld16(base, ra);
#pragma unroll 1
      for (int n0 = 0; n0 < nmax; n0 += 32) {
        tmem_ld_wait();
        if (n0 + 16 < nmax) tmem_ld16(base + (uint32_t)(n0 + 16), rb);
        store16(ra, n0);
        if (n0 + 16 >= nmax) break;
        tmem_ld_wait();
        if (n0 + 32 < nmax) tmem_ld16(base + (uint32_t)(n0 + 32), ra);
        store16(rb, n0 + 16);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(acc ? tempty_leader1 : tempty_leader0);
    }
  }
  tc_fence_before();
  cluster_sync_all();   // neither CTA leaves while the other may still signal its barriers
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
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

// How the split kernel cuts a product: tokens a tile, CTAs an SM, CTAs a tile (the C_in split).
// Up to 32 tokens a ring stage is small and two CTAs share an SM, one's loads covering the other's
// set-up and epilogue, unless there are so few CTAs that each can have a deep ring for itself.
// The split is the largest that leaves every CTA three groups and all CTAs at once on the GPU:
// 0.88 of the slots, since a GPC's SMs are not a multiple of every cluster size.  One token,
// 4096 x 4096: 10.3 us without a split, 5.7 with 8; 4096 x 11008: 10.6 with 3 (258 CTAs), 14.5 with 4
// (344, a second round); 13824 x 5120: 14.5 with 6 (240 CTAs), 20.6 with 7 (280).
struct SplitPlan {
  int NT, per_sm, S;
  long long tiles;
};
SplitPlan split_plan(int cout, int cin, int tokens) {
  SplitPlan p;
  p.NT = tokens >= 128 ? 128 : (tokens + 15) / 16 * 16;
  p.per_sm = p.NT <= 32 ? 2 : 1;
  p.tiles = (long long)cdiv(cout, M8_BM) * cdiv(tokens, p.NT);
  const int G = cdiv(cin, 128);
  p.S = 8;
  while (p.S > 1 && (p.S == 7 || 3 * p.S > G || 100 * p.tiles * p.S > 88LL * p.per_sm * num_sms())) --p.S;
  if (p.tiles * p.S <= num_sms()) p.per_sm = 1;
  return p;
}

// XT = uint8_t: quantised activations X with scales Xs; otherwise the activations (Xs unused).
template <typename OUT, typename XT, bool PERM>
lcp_status split_t(const XT* X, const int32_t* perm, int B, const uint8_t* Xs, const uint8_t* Wq, const uint8_t* Ws, OUT* Y,
                   int cout, int cin, int tokens, const SplitPlan& p, bool w_early, cudaStream_t st) {
  CUtensorMap mW, mX;
  TC_TRY(make_map8(&mW, Wq, cin, cout, M8_BM, "mm8 W"));
  if (sizeof(XT) == 1) TC_TRY(make_map8(&mX, X, cin, tokens, p.NT, "mm8 X"));
  else mX = mW;      // not used
  const int stage_bytes = M8_A + p.NT * 128;
  int stages = (p.per_sm == 2 ? M8_HALF_RING : M8_RING) / stage_bytes;
  if (stages > M8_MAX_STAGES) stages = M8_MAX_STAGES;
  const int smem = stages * stage_bytes + M8_SF * 1024 + (PERM ? M8_FUSED_WARPS * Q8_STAGE * 4 : 0) + 1024 + 512;
  const auto kernel = mm8_split_kernel<OUT, XT, PERM>;
  TC_TRY(set_smem(kernel, smem, "mm8"));
  return launch_kernel(kernel, dim3((unsigned)(p.tiles * p.S)), dim3(m8_threads<XT>()), (size_t)smem, st, p.S, true, "mm8",
                       mW, mX, X, perm, B - 1, Xs, Ws, Y, cout, cin, tokens, p.NT, stages, p.S, w_early ? 1 : 0);
}

template <typename OUT>
lcp_status pair_t(const uint8_t* Xq, const uint8_t* Xs, const uint8_t* Wq, const uint8_t* Ws, OUT* Y, int cout, int cin,
                  int tokens, int N, cudaStream_t st) {
  CUtensorMap mW, mX;
  TC_TRY(make_map8(&mW, Wq, cin, cout, M8_BM, "mm8 W"));
  TC_TRY(make_map8(&mX, Xq, cin, tokens, N / 2, "mm8 X"));
  const int stage_bytes = M8_A + N * 64;
  const int raw = N * cdiv(cin, 128);
  const int fixed = P8_SLOTS * P8_SLOT * P8_SF_BYTES + P8_MAX_G + raw + 1024 + 512;
  int stages = (227 * 1024 - fixed) / stage_bytes;
  if (stages > P8_MAX_STAGES) stages = P8_MAX_STAGES;
  const int smem = stages * stage_bytes + fixed;
  const long long total = (long long)cdiv(cout, 2 * M8_BM) * cdiv(tokens, N);
  const int most = num_sms() / 2;
  const int pairs = total < most ? (int)total : most;
  TC_TRY(set_smem(mm8_pair_kernel<OUT>, smem, "mm8"));
  return launch_kernel(mm8_pair_kernel<OUT>, dim3((unsigned)(2 * pairs)), dim3(P8_THREADS), (size_t)smem, st, 2, true,
                       "mm8", mW, mX, Xs, Ws, Y, cout, cin, tokens, N, stages, raw, tokens <= cout ? 1 : 0);
}

// Tokens a tile of the pair kernel: the width whose rounds over the SM pairs cost least.  A round
// costs, in nanoseconds, 95 + N a group (2048 x 4096 x 4096: 5.4 us a round of 32 groups at N = 64, 6.5
// at 128, 11 at 240) but at least the 17 N that storing a tile takes, and some 600 to change tiles; the
// last round's store shows (700 x 512 x 4096: 13.0 us with the 16 tokens a tile that the model without
// the 600 picks, 8.1 with its 96).
int pair_width(int cout, int cin, int tokens) {
  const int G = cdiv(cin, 128), pairs = num_sms() / 2;
  int best = 16;
  long long cost = -1;
  for (int N = 16; N <= P8_MAX_N && N * G <= P8_RAW; N += 16) {
    const long long tiles = (long long)cdiv(cout, 2 * M8_BM) * cdiv(tokens, N);
    const long long round = std::max((long long)G * (95 + N), 17LL * N) + 600;
    const long long c = (tiles + pairs - 1) / pairs * round + 11 * N;
    if (cost < 0 || c < cost) {
      cost = c;
      best = N;
    }
  }
  return best;
}

// Above 128 tokens the pair kernel is ahead at every size measured (200 x 4096 x 4096: 10.9 us
// against 12.2); between 65 and 128 it is where the split kernel has nothing to split, for want of
// SMs or of channels (128 x 4096 x 11008: 15.0 against 17.8; 128 x 512 x 4096: 4.5 against 7.1; but
// 128 x 11008 x 4096: 19.8 against 16.5).
template <typename OUT>
lcp_status mm8_t(const uint8_t* Xq, const uint8_t* Xs, const uint8_t* Wq, const uint8_t* Ws, OUT* Y, int cout, int cin,
                 int tokens, bool w_early, cudaStream_t st) {
  const SplitPlan p = split_plan(cout, cin, tokens);
  const int G = cdiv(cin, 128);
  if (G <= P8_MAX_G && (tokens > 128 || (tokens > 64 && (p.S == 1 || G <= 8))))
    return pair_t(Xq, Xs, Wq, Ws, Y, cout, cin, tokens, pair_width(cout, cin, tokens), st);
  return split_t<OUT, uint8_t, false>(Xq, nullptr, 1, Xs, Wq, Ws, Y, cout, cin, tokens, p, w_early, st);
}

template <typename OUT, typename XT>
lcp_status fused_t(const XT* X, const int32_t* perm, int B, const uint8_t* Wq, const uint8_t* Ws, OUT* Y, int cout, int cin,
                   int tokens, cudaStream_t st) {
  const SplitPlan p = split_plan(cout, cin, tokens);
  if (perm) return split_t<OUT, XT, true>(X, perm, B, nullptr, Wq, Ws, Y, cout, cin, tokens, p, false, st);
  return split_t<OUT, XT, false>(X, perm, 1, nullptr, Wq, Ws, Y, cout, cin, tokens, p, false, st);
}

}  // namespace

lcp_status tc_error_mm8(int* site, int reset) { return read_tc_error(site, reset); }

lcp_status launch_mm8(const uint8_t* Xq, const uint8_t* Xs, const uint8_t* Wq, const uint8_t* Ws, void* Y, int cout,
                      int cin, int tokens, lcp_dtype ydt, bool w_early, cudaStream_t st) {
  if (ydt == LCP_F32) return mm8_t(Xq, Xs, Wq, Ws, static_cast<float*>(Y), cout, cin, tokens, w_early, st);
  return mm8_t(Xq, Xs, Wq, Ws, static_cast<__nv_bfloat16*>(Y), cout, cin, tokens, w_early, st);
}

bool linear8_fused(int tokens) { return tokens <= M8_FUSED_TOKENS; }

lcp_status launch_linear8_fused(const void* X, const int32_t* perm, int B, const uint8_t* Wq, const uint8_t* Ws, void* Y,
                                int cout, int cin, int tokens, lcp_dtype dt, lcp_dtype ydt, cudaStream_t st) {
  const float* xf = static_cast<const float*>(X);
  const __nv_bfloat16* xb = static_cast<const __nv_bfloat16*>(X);
  float* yf = static_cast<float*>(Y);
  __nv_bfloat16* yb = static_cast<__nv_bfloat16*>(Y);
  if (dt == LCP_F32)
    return ydt == LCP_F32 ? fused_t(xf, perm, B, Wq, Ws, yf, cout, cin, tokens, st)
                          : fused_t(xf, perm, B, Wq, Ws, yb, cout, cin, tokens, st);
  return ydt == LCP_F32 ? fused_t(xb, perm, B, Wq, Ws, yf, cout, cin, tokens, st)
                        : fused_t(xb, perm, B, Wq, Ws, yb, cout, cin, tokens, st);
}

}  // namespace lcp
