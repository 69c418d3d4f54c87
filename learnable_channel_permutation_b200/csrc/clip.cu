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
// infinity makes f zero.
//
// Bound by HBM (three float32 operations a value).  The squares and their sums
// are float64: no gradient overflows or underflows in them, and the sum of a
// whole model's gradients keeps more digits than the float32 result.
//
// Work: the tensors are cut into chunks of kChunk values, in list order; CTA c of
// G takes chunks c, c + G, ... and leaves one partial sum.  The kernel that needs
// the norm adds the partials in a fixed order in every CTA, so the result does
// not depend on timing and the workspace holds nothing that has to be cleared.
// The second pass walks the chunks backwards: the end of the list is what the
// first pass left in L2.  Everything but those kKeep bytes is read and written
// with streaming accesses, so that it stays there (a 7B model's logits, 291 MB:
// 143 us without, 138 with 64 to 80 MB kept, 140 with 112).

#include <type_traits>

#include "lcp_internal.cuh"

namespace lcp {
namespace {

constexpr int kThreads = 256;
constexpr int kChunk = 8192;      // values of a chunk
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
constexpr int kCapSmall = 16, kCapLarge = 640;    // 640 AdamTable entries: 28 KB of the 32 KB a launch may carry

template <typename Table> __device__ __forceinline__ int tensor_of(const Table& t, int chunk) {
  int lo = 0, hi = t.count - 1;       // first[lo] <= chunk < first[hi + 1]
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (t.first[mid] <= chunk) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

__device__ __forceinline__ double block_sum(double v) {
  __shared__ double warp_sum[kThreads / 32];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if (threadIdx.x % 32 == 0) warp_sum[threadIdx.x / 32] = v;
  __syncthreads();
  double s = 0.0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) s += warp_sum[w];
  return s;
}

// Values before the first 16-byte boundary of p (elements of E bytes).
template <int E> __device__ __forceinline__ int head_of(const void* p) {
  return (int)((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15) / E;
}

__device__ __forceinline__ double sq(float x) { return (double)x * (double)x; }
__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

template <typename T> __device__ __forceinline__ double chunk_squares(const T* p, int n, bool stream) {
  constexpr int V = 16 / sizeof(T);
  double s0 = 0.0, s1 = 0.0;
  int head = head_of<sizeof(T)>(p);
  if (head > n) head = n;
  const int vecs = (n - head) / V;
  const uint4* q = reinterpret_cast<const uint4*>(p + head);
#pragma unroll 4
  for (int i = threadIdx.x; i < vecs; i += kThreads) {
    const uint4 u = stream ? __ldcs(q + i) : __ldg(q + i);
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

template <typename Table>
__global__ void __launch_bounds__(kThreads)
squares_kernel(const __grid_constant__ Table t, double* __restrict__ partials, long long keep) {
  pdl_wait();
  pdl_trigger();
  double s = 0.0;
  const int chunks = t.first[t.count];
  for (int c = blockIdx.x; c < chunks; c += gridDim.x) {
    const int i = tensor_of(t, c);
    const long long at = (long long)(c - t.first[i]) * kChunk;
    const int n = (int)(t.n[i] - at < kChunk ? t.n[i] - at : kChunk);
    bool bf = false;
    if constexpr (!is_adam<Table>::value) bf = t.bf16[i];
    const bool stream = (long long)(chunks - c) * kChunk * (bf ? 2 : 4) > keep;
    if (bf) s += chunk_squares(reinterpret_cast<const __nv_bfloat16*>(t.g[i]) + at, n, stream);
    else s += chunk_squares(reinterpret_cast<const float*>(t.g[i]) + at, n, stream);
  }
  s = block_sum(s);
  if (threadIdx.x == 0) partials[blockIdx.x] = s;
}

// The norm from the partials, the same in every CTA.
__device__ __forceinline__ double norm_of(const double* __restrict__ partials, int np) {
  double s = 0.0;
  for (int i = threadIdx.x; i < np; i += kThreads) s += partials[i];
  return sqrt(block_sum(s));
}
__device__ __forceinline__ float factor_of(double norm, double max_norm) {
  const double f = max_norm / (norm + kClipEps);
  return f > 1.0 ? 1.f : (float)f;     // NaN stays NaN
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
template <typename T> __device__ __forceinline__ void chunk_scale(const T* g, T* out, int n, float f) {
  constexpr int V = 16 / sizeof(T);
  int head = head_of<sizeof(T)>(g);
  if (head > n) head = n;
  if (head_of<sizeof(T)>(out) != head_of<sizeof(T)>(g)) {     // no common 16-byte boundary
    for (int i = threadIdx.x; i < n; i += kThreads) out[i] = from_f32<T>(to_f32(g[i]) * f);
    return;
  }
  const int vecs = (n - head) / V;
  const uint4* q = reinterpret_cast<const uint4*>(g + head);
  uint4* w = reinterpret_cast<uint4*>(out + head);
#pragma unroll 4
  for (int i = threadIdx.x; i < vecs; i += kThreads) {
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

template <int CAP>
__global__ void __launch_bounds__(kThreads)
scale_kernel(const __grid_constant__ GradTable<CAP> t, const double* __restrict__ partials, int np, double max_norm,
             float* __restrict__ norm) {
  pdl_wait();
  pdl_trigger();
  const double v = norm_of(partials, np);
  const float f = factor_of(v, max_norm);
  if (norm && blockIdx.x == 0 && threadIdx.x == 0) norm[0] = (float)v;
  const int chunks = t.first[t.count];
  for (int c = chunks - 1 - (int)blockIdx.x; c >= 0; c -= gridDim.x) {
    const int i = tensor_of(t, c);
    const long long at = (long long)(c - t.first[i]) * kChunk;
    const int n = (int)(t.n[i] - at < kChunk ? t.n[i] - at : kChunk);
    if (t.bf16[i])
      chunk_scale(reinterpret_cast<const __nv_bfloat16*>(t.g[i]) + at, reinterpret_cast<__nv_bfloat16*>(t.out[i]) + at, n, f);
    else
      chunk_scale(reinterpret_cast<const float*>(t.g[i]) + at, reinterpret_cast<float*>(t.out[i]) + at, n, f);
  }
}

template <int CAP>
__global__ void __launch_bounds__(kThreads)
adamw_list_kernel(const __grid_constant__ AdamTable<CAP> t, const double* __restrict__ partials, int np, double max_norm,
                  float* __restrict__ norm, AdamCoef c) {
  pdl_wait();
  pdl_trigger();
  const double v = norm_of(partials, np);
  const float f = factor_of(v, max_norm);
  if (norm && blockIdx.x == 0 && threadIdx.x == 0) norm[0] = (float)v;
  const int chunks = t.first[t.count];
  for (int k = chunks - 1 - (int)blockIdx.x; k >= 0; k -= gridDim.x) {
    const int i = tensor_of(t, k);
    const long long at = (long long)(k - t.first[i]) * kChunk;
    const int n = (int)(t.n[i] - at < kChunk ? t.n[i] - at : kChunk);
    float* L = t.L[i] + at;
    const float* g = t.g[i] + at;
    float* m = t.m[i] + at;
    float* w = t.v[i] + at;
    const int phase = head_of<4>(L);
    const bool same = head_of<4>(g) == phase && head_of<4>(m) == phase && head_of<4>(w) == phase;
    const int head = same ? (phase < n ? phase : n) : n;     // no common 16-byte boundary: value by value
    const int vecs = (n - head) / 4;
#pragma unroll 2
    for (int q = threadIdx.x; q < vecs; q += kThreads) {
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
    for (int r = threadIdx.x; r < n - vecs * 4; r += kThreads) {
      const int e = r < head ? r : r + vecs * 4;
      float l1 = L[e], m1 = m[e], v1 = w[e];
      adam1(l1, g[e] * f, m1, v1, c);
      L[e] = l1;
      m[e] = m1;
      w[e] = v1;
    }
  }
}

int sm_count() {
  int sms = 148, dev = 0;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  return sms;
}
long long chunks_of(long long n) { return (n + kChunk - 1) / kChunk; }
int grid_of(long long chunks) {
  const long long most = (long long)kClipCtasPerSm * sm_count();
  return (int)(chunks < most ? chunks : most);
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

// Cuts the list into launches of at most kCapLarge tensors (those without values
// take no place) and calls `go` with each table.
template <typename Table, typename Small, typename Desc, typename Go>
lcp_status each_table(const Desc* d, int count, Go go) {
  static thread_local Table t;       // 28 KB: off the caller's stack
  static thread_local Small s;
  t.count = 0;
  long long chunks = 0;
  auto flush = [&]() -> lcp_status {
    if (!t.count) return LCP_OK;
    t.first[t.count] = (int)chunks;
    const int grid = grid_of(chunks);
    lcp_status r;
    if (t.count <= kCapSmall) {
      shrink(s, t);
      r = go(s, grid);
    } else {
      r = go(t, grid);
    }
    t.count = 0;
    chunks = 0;
    return r;
  };
  for (int i = 0; i < count; ++i) {
    if (d[i].n == 0) continue;
    const long long c = chunks_of(d[i].n);
    if (t.count == kCapLarge) {
      const lcp_status r = flush();
      if (r != LCP_OK) return r;
    }
    t.n[t.count] = d[i].n;
    t.first[t.count] = (int)chunks;
    add(t, d[i]);
    ++t.count;
    chunks += c;
  }
  return flush();
}

template <typename Table, typename Small, typename Desc>
lcp_status squares(const Desc* d, int count, double* partials, int* np, cudaStream_t st) {
  *np = 0;
  return each_table<Table, Small>(d, count, [&](const auto& t, int grid) {
    using T = std::decay_t<decltype(t)>;
    const lcp_status r = launch_kernel(squares_kernel<T>, dim3((unsigned)grid), dim3(kThreads), 0, st, 1, true, "grad_norm",
                                       t, partials + *np, kKeep);
    *np += grid;
    return r;
  });
}

}  // namespace

size_t clip_workspace(int count) {
  // one partial for each CTA of each launch
  const size_t launches = (size_t)count / kCapLarge + 1;
  return launches * (size_t)kClipCtasPerSm * sm_count() * sizeof(double);
}

lcp_status launch_grad_norm(const lcp_grad* d, int count, float* norm, void* ws, cudaStream_t st) {
  double* partials = static_cast<double*>(ws);
  int np = 0;
  lcp_status r = squares<GradTable<kCapLarge>, GradTable<kCapSmall>>(d, count, partials, &np, st);
  if (r != LCP_OK) return r;
  return launch_kernel(norm_kernel, dim3(1), dim3(kThreads), 0, st, 1, true, "grad_norm", (const double*)partials, np, norm);
}

lcp_status launch_grad_clip(const lcp_grad* d, int count, double max_norm, float* norm, void* ws, cudaStream_t st) {
  double* partials = static_cast<double*>(ws);
  int np = 0;
  lcp_status r = squares<GradTable<kCapLarge>, GradTable<kCapSmall>>(d, count, partials, &np, st);
  if (r != LCP_OK) return r;
  if (np == 0)      // nothing but empty tensors: the norm is zero
    return launch_kernel(norm_kernel, dim3(1), dim3(kThreads), 0, st, 1, true, "grad_clip", (const double*)partials, 0, norm);
  return each_table<GradTable<kCapLarge>, GradTable<kCapSmall>>(d, count, [&](const auto& t, int grid) {
    using T = std::decay_t<decltype(t)>;
    constexpr int cap = sizeof(T::bf16);
    return launch_kernel(scale_kernel<cap>, dim3((unsigned)grid), dim3(kThreads), 0, st, 1, true, "grad_clip", t,
                         (const double*)partials, np, max_norm, norm);
  });
}

lcp_status launch_adamw_list(const lcp_adamw_tensor* d, int count, const lcp_adamw_params& opt, int step, double max_norm,
                             float* norm, void* ws, cudaStream_t st) {
  double* partials = static_cast<double*>(ws);
  int np = 0;
  lcp_status r = squares<AdamTable<kCapLarge>, AdamTable<kCapSmall>>(d, count, partials, &np, st);
  if (r != LCP_OK) return r;
  if (np == 0)
    return launch_kernel(norm_kernel, dim3(1), dim3(kThreads), 0, st, 1, true, "adamw_list", (const double*)partials, 0, norm);
  const AdamCoef c = adam_coef(opt.lr, opt.beta1, opt.beta2, opt.eps, opt.weight_decay, step);
  return each_table<AdamTable<kCapLarge>, AdamTable<kCapSmall>>(d, count, [&](const auto& t, int grid) {
    using T = std::decay_t<decltype(t)>;
    constexpr int cap = sizeof(T::n) / sizeof(long long);
    return launch_kernel(adamw_list_kernel<cap>, dim3((unsigned)grid), dim3(kThreads), 0, st, 1, true, "adamw_list", t,
                         (const double*)partials, np, max_norm, norm, c);
  });
}

}  // namespace lcp
