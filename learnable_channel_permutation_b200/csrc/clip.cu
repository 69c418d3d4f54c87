// The global 2-norm of many gradient tensors, the gradients clipped by it, and
// one AdamW update of many tensors with the clipping factor applied to the
// gradient on the way.
//
//   norm = sqrt(sum over all tensors of g^2)
//   f    = min(1, max_norm / (norm + 1e-6))
//   g <- f g                       (clip)
//   AdamW with f g as the gradient (adamw; the formulas of adamw.cu)
//
// A norm that is not finite is passed on: NaN makes every clipped gradient NaN,
// infinity makes f zero.  max_norm infinite: f = 1, whatever the norm.
//
// Bound by HBM (three float32 operations a value).  The squares and their sums
// are float64: no gradient overflows or underflows in them, and the sum of a
// whole model's gradients keeps more digits than the float32 result.
//
// Work: the tensors are cut into chunks of 8192 or 2048 values, in list order; CTA c of
// G takes chunks c, c + G, ... and leaves one partial sum.  The kernel that needs
// the norm adds the partials in a fixed order in every CTA, so the result does
// not depend on timing and the workspace holds nothing that has to be cleared.
// The second pass walks the chunks backwards: the end of the list is what the
// first pass left in L2.  Everything but those kKeep bytes is read and written
// with streaming accesses, so that it stays there (a 7B model's logits, 291 MB:
// 143 us without, 138 with 64 to 80 MB kept, 140 with 112).  That is one table of
// kCapLarge tensors: a longer list takes each pass table by table, front first,
// every table with an end of its own, and little of what is left in L2 is met again.

#include <algorithm>
#include <atomic>
#include <type_traits>

#include <cooperative_groups.h>

#include "lcp_internal.cuh"

namespace lcp {
namespace {

constexpr int kThreads = 256;
constexpr int kChunk = 8192, kShortChunk = 2048;      // values of a chunk (use_short_chunks)
// Short lists: one cluster does both passes in one launch (below).
constexpr int kSmallThreads = 1024, kSmallCluster = 16, kSmallChunk = 4096;
constexpr double kClipEps = 1e-6;
constexpr long long kKeep = 80LL << 20;   // bytes of the list's end that the first pass leaves in L2

// The tensors of one launch, in its parameters: nothing is copied to the device
// before the launch and a captured graph holds its own list.  The capacity is
// the smallest of the instantiated ones, since a launch carries all of it.
template <int CAP> struct GradTable {
  const void* g[CAP];
  void* out[CAP];
  long long n[CAP];
  int first[CAP + 1];     // chunk index of each tensor's first chunk
  unsigned char bf16[CAP];
  int count;
};
template <int CAP> struct AdamTable {
  float* L[CAP];
  const float* g[CAP];
  float* m[CAP];
  float* v[CAP];
  long long n[CAP];
  int first[CAP + 1];
  int count;
};
constexpr int kCapSmall = 16, kCapMid = 80, kCapLarge = 640;    // 640 AdamTable entries: 28 KB of a launch's 32 KB at most

template <typename Table> __device__ __forceinline__ int tensor_of(const Table& t, int chunk) {
  int lo = 0, hi = t.count - 1;       // first[lo] <= chunk < first[hi + 1]
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (t.first[mid] <= chunk) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

template <int NTHR> __device__ __forceinline__ double block_sum(double v) {
  __shared__ double warp_sum[NTHR / 32];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if (threadIdx.x % 32 == 0) warp_sum[threadIdx.x / 32] = v;
  __syncthreads();
  double s = 0.0;
#pragma unroll
  for (int w = 0; w < NTHR / 32; ++w) s += warp_sum[w];
  return s;
}

// Values before the first 16-byte boundary of p (elements of E bytes).
template <int E> __device__ __forceinline__ int head_of(const void* p) {
  return (int)((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15) / E;
}

__device__ __forceinline__ double sq(float x) { return (double)x * (double)x; }
__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// CONST: the launch does not write the gradients, so they may be read on the read-only path (norm of
// 262144 values 2.7 us, 2.8 without).
template <int NTHR, bool CONST, typename T> __device__ __forceinline__ double chunk_squares(const T* p, int n, bool stream) {
  constexpr int V = 16 / sizeof(T);
  double s0 = 0.0, s1 = 0.0;
  int head = head_of<sizeof(T)>(p);
  if (head > n) head = n;
  const int vecs = (n - head) / V;
  const uint4* q = reinterpret_cast<const uint4*>(p + head);
#pragma unroll 4
  for (int i = threadIdx.x; i < vecs; i += NTHR) {
    const uint4 u = stream ? __ldcs(q + i) : CONST ? __ldg(q + i) : q[i];
    if constexpr (sizeof(T) == 4) {
      s0 += sq(__uint_as_float(u.x)) + sq(__uint_as_float(u.y));
      s1 += sq(__uint_as_float(u.z)) + sq(__uint_as_float(u.w));
    } else {
      s0 += sq(bf_lo(u.x)) + sq(bf_hi(u.x)) + sq(bf_lo(u.y)) + sq(bf_hi(u.y));
      s1 += sq(bf_lo(u.z)) + sq(bf_hi(u.z)) + sq(bf_lo(u.w)) + sq(bf_hi(u.w));
    }
  }
  const int rest = n - vecs * V;     // the head, then what follows the last whole vector
  if ((int)threadIdx.x < rest) {
    const int i = (int)threadIdx.x < head ? (int)threadIdx.x : (int)threadIdx.x + vecs * V;
    s0 += sq(to_f32(p[i]));
  }
  return s0 + s1;
}

template <typename Table> struct is_adam { static constexpr bool value = false; };
template <int CAP> struct is_adam<AdamTable<CAP>> { static constexpr bool value = true; };

// Chunk c of a list: its tensor, where it starts in it and its length.
struct ChunkAt {
  int i, n;
  long long at;
};
template <int CHUNK, typename Table> __device__ __forceinline__ ChunkAt chunk_at(const Table& t, int c) {
  ChunkAt r;
  r.i = tensor_of(t, c);
  r.at = (long long)(c - t.first[r.i]) * CHUNK;
  r.n = (int)(t.n[r.i] - r.at < CHUNK ? t.n[r.i] - r.at : CHUNK);
  return r;
}
template <typename Table> __device__ __forceinline__ bool is_bf16(const Table& t, int i) {
  if constexpr (is_adam<Table>::value) return false;
  else return t.bf16[i];
}
template <int NTHR, bool CONST, typename Table>
__device__ __forceinline__ double squares_of(const Table& t, const ChunkAt& a, bool stream) {
  if (is_bf16(t, a.i)) return chunk_squares<NTHR, CONST>(reinterpret_cast<const __nv_bfloat16*>(t.g[a.i]) + a.at, a.n, stream);
  return chunk_squares<NTHR, CONST>(reinterpret_cast<const float*>(t.g[a.i]) + a.at, a.n, stream);
}

template <int CHUNK, typename Table>
__global__ void __launch_bounds__(kThreads, kClipCtasPerSm)
squares_kernel(const __grid_constant__ Table t, double* __restrict__ partials, long long keep) {
  pdl_wait();
  pdl_trigger();
  double s = 0.0;
  const int chunks = t.first[t.count];
  for (int c = blockIdx.x; c < chunks; c += gridDim.x) {
    const ChunkAt a = chunk_at<CHUNK>(t, c);
    s += squares_of<kThreads, true>(t, a, (long long)(chunks - c) * CHUNK * (is_bf16(t, a.i) ? 2 : 4) > keep);
  }
  s = block_sum<kThreads>(s);
  if (threadIdx.x == 0) partials[blockIdx.x] = s;
}

// The norm from the partials, the same in every CTA.
__device__ __forceinline__ double norm_of(const double* __restrict__ partials, int np) {
  double s = 0.0;
  for (int i = threadIdx.x; i < np; i += kThreads) s += partials[i];
  return sqrt(block_sum<kThreads>(s));
}
__device__ __forceinline__ float factor_of(double norm, double max_norm) {
  const double f = max_norm / (norm + kClipEps);
  return f > 1.0 || isinf(max_norm) ? 1.f : (float)f;     // NaN stays NaN, where clipping was asked for
}

__global__ void __launch_bounds__(kThreads)
norm_kernel(const double* __restrict__ partials, int np, float* __restrict__ norm) {
  pdl_wait();
  pdl_trigger();
  const double v = norm_of(partials, np);
  if (threadIdx.x == 0) norm[0] = (float)v;
}

__device__ __forceinline__ uint32_t scale_pair(uint32_t w, float f) {
  const __nv_bfloat162 r = __floats2bfloat162_rn(bf_lo(w) * f, bf_hi(w) * f);
  return *reinterpret_cast<const uint32_t*>(&r);
}

// out = f g over one chunk; g and out may be the same array.
template <int NTHR, typename T> __device__ __forceinline__ void chunk_scale(const T* g, T* out, int n, float f) {
  constexpr int V = 16 / sizeof(T);
  int head = head_of<sizeof(T)>(g);
  if (head > n) head = n;
  if (head_of<sizeof(T)>(out) != head_of<sizeof(T)>(g)) {     // no common 16-byte boundary
    for (int i = threadIdx.x; i < n; i += NTHR) out[i] = from_f32<T>(to_f32(g[i]) * f);
    return;
  }
  const int vecs = (n - head) / V;
  const uint4* q = reinterpret_cast<const uint4*>(g + head);
  uint4* w = reinterpret_cast<uint4*>(out + head);
#pragma unroll 4
  for (int i = threadIdx.x; i < vecs; i += NTHR) {
    uint4 u = __ldcs(q + i);
    if constexpr (sizeof(T) == 4) {
      u.x = __float_as_uint(__uint_as_float(u.x) * f);
      u.y = __float_as_uint(__uint_as_float(u.y) * f);
      u.z = __float_as_uint(__uint_as_float(u.z) * f);
      u.w = __float_as_uint(__uint_as_float(u.w) * f);
    } else {
      u.x = scale_pair(u.x, f);
      u.y = scale_pair(u.y, f);
      u.z = scale_pair(u.z, f);
      u.w = scale_pair(u.w, f);
    }
    __stcs(w + i, u);
  }
  const int rest = n - vecs * V;
  if ((int)threadIdx.x < rest) {
    const int i = (int)threadIdx.x < head ? (int)threadIdx.x : (int)threadIdx.x + vecs * V;
    out[i] = from_f32<T>(to_f32(g[i]) * f);
  }
}

// AdamW of one chunk with f g as the gradient.
template <int NTHR>
__device__ __forceinline__ void chunk_adamw(float* L, const float* g, float* m, float* w, int n, float f, const AdamCoef& c) {
  const int phase = head_of<4>(L);
  const bool same = head_of<4>(g) == phase && head_of<4>(m) == phase && head_of<4>(w) == phase;
  const int head = same ? (phase < n ? phase : n) : n;     // no common 16-byte boundary: value by value
  const int vecs = (n - head) / 4;
#pragma unroll 2
  for (int q = threadIdx.x; q < vecs; q += NTHR) {
    float4 l4 = __ldcs(reinterpret_cast<float4*>(L + head) + q);
    float4 g4 = __ldcs(reinterpret_cast<const float4*>(g + head) + q);
    float4 m4 = __ldcs(reinterpret_cast<float4*>(m + head) + q);
    float4 v4 = __ldcs(reinterpret_cast<float4*>(w + head) + q);
    adam1(l4.x, g4.x * f, m4.x, v4.x, c);
    adam1(l4.y, g4.y * f, m4.y, v4.y, c);
    adam1(l4.z, g4.z * f, m4.z, v4.z, c);
    adam1(l4.w, g4.w * f, m4.w, v4.w, c);
    __stcs(reinterpret_cast<float4*>(L + head) + q, l4);
    __stcs(reinterpret_cast<float4*>(m + head) + q, m4);
    __stcs(reinterpret_cast<float4*>(w + head) + q, v4);
  }
  for (int r = threadIdx.x; r < n - vecs * 4; r += NTHR) {
    const int e = r < head ? r : r + vecs * 4;
    float l1 = L[e], m1 = m[e], v1 = w[e];
    adam1(l1, g[e] * f, m1, v1, c);
    L[e] = l1;
    m[e] = m1;
    w[e] = v1;
  }
}

// The second pass over one chunk: clipping, or the update.
template <int NTHR, int CAP>
__device__ __forceinline__ void apply(const GradTable<CAP>& t, const ChunkAt& a, float f, const AdamCoef&) {
  if (t.bf16[a.i])
    chunk_scale<NTHR>(reinterpret_cast<const __nv_bfloat16*>(t.g[a.i]) + a.at,
                      reinterpret_cast<__nv_bfloat16*>(t.out[a.i]) + a.at, a.n, f);
  else
    chunk_scale<NTHR>(reinterpret_cast<const float*>(t.g[a.i]) + a.at, reinterpret_cast<float*>(t.out[a.i]) + a.at, a.n, f);
}
template <int NTHR, int CAP>
__device__ __forceinline__ void apply(const AdamTable<CAP>& t, const ChunkAt& a, float f, const AdamCoef& c) {
  chunk_adamw<NTHR>(t.L[a.i] + a.at, t.g[a.i] + a.at, t.m[a.i] + a.at, t.v[a.i] + a.at, a.n, f, c);
}

// CTAs an SM that the second pass keeps its registers to: clipping, the whole grid (six of eight CTAs
// resident, a 7B model's logits: 154 us instead of 138); the update, five (with none asked for, seven
// layers' logits: 13.7 us instead of 11.6).
template <typename Table> constexpr int apply_ctas() { return is_adam<Table>::value ? 5 : kClipCtasPerSm; }

template <int CHUNK, typename Table>
__global__ void __launch_bounds__(kThreads, apply_ctas<Table>())
apply_kernel(const __grid_constant__ Table t, const double* __restrict__ partials, int np, double max_norm,
             float* __restrict__ norm, AdamCoef c) {
  pdl_wait();
  pdl_trigger();
  const double v = norm_of(partials, np);
  const float f = factor_of(v, max_norm);
  if (blockIdx.x == 0 && threadIdx.x == 0) norm[0] = (float)v;
  for (int k = t.first[t.count] - 1 - (int)blockIdx.x; k >= 0; k -= gridDim.x) apply<kThreads>(t, chunk_at<CHUNK>(t, k), f, c);
}

// A short list in one launch: one cluster, a chunk for each CTA, takes both passes.  The CTAs'
// sums meet in distributed shared memory (added in rank order by every CTA), and the second pass
// finds the gradients in the L1 that the first filled.  APPLY false: the norm alone.
template <typename Table, bool APPLY>
__global__ void __launch_bounds__(kSmallThreads)
small_kernel(const __grid_constant__ Table t, double max_norm, float* __restrict__ norm, AdamCoef c) {
  namespace cg = cooperative_groups;
  __shared__ double mine;
  pdl_wait();
  pdl_trigger();
  const cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank(), ctas = (int)cluster.num_blocks();
  ChunkAt a = {0, 0, 0};
  double s = 0.0;
  if (rank < t.first[t.count]) {
    a = chunk_at<kSmallChunk>(t, rank);
    s = squares_of<kSmallThreads, !APPLY>(t, a, false);      // clipped in place further down
  }
  s = block_sum<kSmallThreads>(s);
  if (threadIdx.x == 0) mine = s;
  cluster.sync();
  double sum = 0.0;
  for (int r = 0; r < ctas; ++r) sum += *cluster.map_shared_rank(&mine, r);
  cluster.barrier_arrive();      // this CTA has read the others' sums
  const double v = sqrt(sum);
  if (rank == 0 && threadIdx.x == 0) norm[0] = (float)v;
  if (APPLY && a.n > 0) apply<kSmallThreads>(t, a, factor_of(v, max_norm), c);
  cluster.barrier_wait();        // no CTA ends while another may still read its sum
}

long long chunks_of(long long n, int chunk) { return (n + chunk - 1) / chunk; }
// Short chunks where long ones would leave SMs without any (one layer's logits, 128 chunks instead of 32:
// 4.5 us instead of 6.2 clipped, 5.5 instead of 9.3 updated; but seven layers', 962 instead of 241: 8.8
// instead of 7.5).
template <typename Desc> bool use_short_chunks(const Desc* d, int count, int sms) {
  long long chunks = 0;
  for (int i = 0; i < count && chunks <= 2 * sms; ++i) chunks += chunks_of(d[i].n, kShortChunk);
  return chunks <= 2 * sms;
}

void add(GradTable<kCapLarge>& t, const lcp_grad& d) {
  t.g[t.count] = d.g;
  t.out[t.count] = d.out;
  t.bf16[t.count] = d.dtype == LCP_BF16;
}
void add(AdamTable<kCapLarge>& t, const lcp_adamw_tensor& d) {
  t.L[t.count] = d.L;
  t.g[t.count] = d.dL;
  t.m[t.count] = d.m;
  t.v[t.count] = d.v;
}
template <typename To, typename From> void shrink(To& to, const From& from) {
  for (int i = 0; i < from.count; ++i) {
    to.g[i] = from.g[i];
    to.n[i] = from.n[i];
    to.first[i] = from.first[i];
    if constexpr (is_adam<To>::value) {
      to.L[i] = from.L[i];
      to.m[i] = from.m[i];
      to.v[i] = from.v[i];
    } else {
      to.out[i] = from.out[i];
      to.bf16[i] = from.bf16[i];
    }
  }
  to.first[from.count] = from.first[from.count];
  to.count = from.count;
}

// Puts tensors from d[*at] on into t until it is full (those without values take no place), moves
// *at behind them and returns their chunk count.
template <typename Table, typename Desc> int fill(Table& t, const Desc* d, int count, int chunk, int* at) {
  long long chunks = 0;
  t.count = 0;
  for (; *at < count && t.count < kCapLarge; ++*at) {
    const Desc& x = d[*at];
    if (x.n == 0) continue;
    t.n[t.count] = x.n;
    t.first[t.count] = (int)chunks;
    add(t, x);
    ++t.count;
    chunks += chunks_of(x.n, chunk);
  }
  t.first[t.count] = (int)chunks;
  return (int)chunks;
}

// Launches with the table by address (launch_kernel's by-value arguments would copy its 28 KB twice).
template <typename... Args>
lcp_status launch_with(const void* kernel, int grid, int threads, int cluster, cudaStream_t st, const char* what,
                       const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  unsigned na = 0;
  if (cluster > 1) {
    attr[na].id = cudaLaunchAttributeClusterDimension;
    attr[na].val.clusterDim.x = (unsigned)cluster;
    attr[na].val.clusterDim.y = attr[na].val.clusterDim.z = 1;
    ++na;
  }
  if (pdl_enabled()) {
    attr[na].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[na].val.programmaticStreamSerializationAllowed = 1;
    ++na;
  }
  cfg.attrs = attr;
  cfg.numAttrs = na;
  void* ptrs[] = {const_cast<void*>(static_cast<const void*>(&args))...};
  const cudaError_t e = cudaLaunchKernelExC(&cfg, kernel, ptrs);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return fail(LCP_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
  }
  return check_launch(what);
}

template <typename K> lcp_status allow_cluster(K kernel, std::atomic<unsigned long long>& done, const char* what) {
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 64 && (done.load(std::memory_order_relaxed) >> dev & 1ull)) return LCP_OK;     // a bit for each device
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return fail(LCP_ERR_CUDA, "%s: cudaFuncSetAttribute: %s", what, cudaGetErrorString(e));
  }
  if (dev < 64) done.fetch_or(1ull << dev, std::memory_order_relaxed);
  return LCP_OK;
}

// Calls go with the smallest table type that holds t.
template <template <int> class T, typename Go> lcp_status with_table(const T<kCapLarge>& t, Go go) {
  if (t.count <= kCapSmall) {
    static thread_local T<kCapSmall> s;
    shrink(s, t);
    return go(s);
  }
  if (t.count <= kCapMid) {
    static thread_local T<kCapMid> m;
    shrink(m, t);
    return go(m);
  }
  return go(t);
}

// One cluster for the whole list, a chunk for each CTA.
template <bool APPLY, template <int> class T>
lcp_status run_small(const T<kCapLarge>& t, int chunks, double max_norm, float* norm, const AdamCoef& c, cudaStream_t st,
                     const char* what) {
  static_assert(kCapSmall >= kSmallCluster, "a list of 16 chunks has at most 16 tensors");
  static thread_local T<kCapSmall> s;
  shrink(s, t);
  const auto kernel = small_kernel<T<kCapSmall>, APPLY>;
  int ctas = 1;
  while (ctas < chunks) ctas *= 2;
  if (ctas > 8) {
    static std::atomic<unsigned long long> done{0};
    const lcp_status r = allow_cluster(kernel, done, what);
    if (r != LCP_OK) return r;
  }
  return launch_with(reinterpret_cast<const void*>(kernel), ctas, kSmallThreads, ctas, st, what, s, max_norm, norm, c);
}

// Both passes over the list in two launches for each kCapLarge tensors (APPLY false: the first alone,
// and the norm).
template <bool APPLY, int CHUNK, template <int> class T, typename Desc>
lcp_status run_passes(T<kCapLarge>& t, const Desc* d, int count, double max_norm, float* norm, double* partials,
                      const AdamCoef& c, int sms, cudaStream_t st, const char* what) {
  int np = 0, tables = 0, chunks = 0, at = 0;
  while (at < count) {
    chunks = fill(t, d, count, CHUNK, &at);
    if (!t.count) break;
    const int grid = std::min(chunks, kClipCtasPerSm * sms);
    const double* out = partials + np;
    const lcp_status r = with_table<T>(t, [&](const auto& x) {
      return launch_with(reinterpret_cast<const void*>(squares_kernel<CHUNK, std::decay_t<decltype(x)>>), grid, kThreads, 1,
                         st, what, x, out, kKeep);
    });
    if (r != LCP_OK) return r;
    np += grid;
    ++tables;
  }
  if (!APPLY || np == 0)      // np 0: nothing but empty tensors, and the norm is zero
    return launch_kernel(norm_kernel, dim3(1), dim3(kThreads), 0, st, 1, true, what, (const double*)partials, np, norm);
  at = 0;
  for (int k = 0; k < tables; ++k) {
    if (tables > 1) chunks = fill(t, d, count, CHUNK, &at);     // a single table is still there
    const lcp_status r = with_table<T>(t, [&](const auto& x) {
      return launch_with(reinterpret_cast<const void*>(apply_kernel<CHUNK, std::decay_t<decltype(x)>>),
                         std::min(chunks, kClipCtasPerSm * sms), kThreads, 1, st, what, x, partials, np, max_norm, norm, c);
    });
    if (r != LCP_OK) return r;
  }
  return LCP_OK;
}

template <bool APPLY, template <int> class T, typename Desc>
lcp_status run_list(const Desc* d, int count, double max_norm, float* norm, void* ws, const AdamCoef& c, cudaStream_t st,
                    const char* what) {
  static thread_local T<kCapLarge> t;       // 28 KB: off the caller's stack
  // Short lists take one launch of one cluster, for a launch less on the host.  One call after another from
  // the host, clipping and update, one launch and two: 4096 values 4.3 / 6.1 and 4.8 / 6.4 us, 65536 values 5.6 / 6.1
  // and 6.5 / 6.4, which is the border.  In a captured graph, where that launch costs less, two are ahead from some
  // 32768 values on: 4096 values 2.9 / 3.9 and 4.2 / 4.4 us, 32768 3.9 / 4.0 and 5.0 / 4.5, 65536 5.4 / 3.9 and
  // 6.3 / 4.6.
  long long small = 0;
  for (int i = 0; i < count && small <= kSmallCluster; ++i) small += chunks_of(d[i].n, kSmallChunk);
  if (small > 0 && small <= kSmallCluster) {
    int at = 0;
    const int chunks = fill(t, d, count, kSmallChunk, &at);
    return run_small<APPLY, T>(t, chunks, max_norm, norm, c, st, what);
  }
  const int sms = device_sms();
  double* partials = static_cast<double*>(ws);
  if (use_short_chunks(d, count, sms))
    return run_passes<APPLY, kShortChunk, T>(t, d, count, max_norm, norm, partials, c, sms, st, what);
  return run_passes<APPLY, kChunk, T>(t, d, count, max_norm, norm, partials, c, sms, st, what);
}

}  // namespace

size_t clip_workspace(int count) {
  // one partial for each CTA of each launch
  const size_t launches = (size_t)count / kCapLarge + 1;
  return launches * (size_t)kClipCtasPerSm * device_sms() * sizeof(double);
}

lcp_status launch_grad_norm(const lcp_grad* d, int count, float* norm, void* ws, cudaStream_t st) {
  return run_list<false, GradTable>(d, count, 1.0, norm, ws, AdamCoef{}, st, "grad_norm");
}

lcp_status launch_grad_clip(const lcp_grad* d, int count, double max_norm, float* norm, void* ws, cudaStream_t st) {
  return run_list<true, GradTable>(d, count, max_norm, norm, ws, AdamCoef{}, st, "grad_clip");
}

lcp_status launch_adamw_list(const lcp_adamw_tensor* d, int count, const lcp_adamw_params& opt, int step, double max_norm,
                             float* norm, void* ws, cudaStream_t st) {
  const AdamCoef c = adam_coef(opt.lr, opt.beta1, opt.beta2, opt.eps, opt.weight_decay, step);
  return run_list<true, AdamTable>(d, count, max_norm, norm, ws, c, st, "adamw_list");
}

}  // namespace lcp
