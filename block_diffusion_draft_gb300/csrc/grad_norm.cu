// grad_norm.cu -- the global norm of many gradients, and clipping by it.
//
//   norm = sqrt(sum over all tensors of g^2);  norm > max: g becomes g * (max / norm)
//
// HBM bounds it: the norm reads every gradient once; clipping, which needs the
// norm first, reads them again and writes them.  The tensors are cut into
// chunks of 32 KB (2048 16-byte pieces) in one line, which the CTAs take in turn,
// so that all of them are near one another in memory (a run of its own for each
// CTA was 5% slower); the second pass goes backwards and so begins with what the
// first one left in L2.  One decoder layer's gradients in bf16 (386 MB): the
// norm 59 us (6.5 TB/s), clipped into other buffers 187 us (of another alignment:
// 460 to 525, in stores of 2 bytes).
//
// A thread adds the squares of up to 64 values in fp32 (relative error below
// 64 * 2^-24) and everything above that in fp64, in an order that depends on
// the sizes alone: the norm is the same in every run.  64 squares whose fp32
// sum leaves [2^-80, 2^100) are added again in fp64, so that values up to the
// largest and down to the smallest count.
#include <algorithm>
#include <utility>
#include <vector>

#include "../../include/dflash_attn.h"
#include "handles.h"
#include "internal.h"
#include "ptx.cuh"

namespace df {
namespace {

constexpr int kThreads = 256;
constexpr int kVecs = 8;                       // 16-byte pieces of a thread in a chunk
constexpr int kChunk = kThreads * kVecs;       // pieces of a chunk
// Tensors of one launch, whose table goes by value: few, so that a small call's
// launch copies little (1.6 KB instead of 28: 0.8 us each), or many.
constexpr int kFew = 56, kMany = 1000;
constexpr int kCtasPerSm = 4;
constexpr double kBig = 1.2676506002282294e30;    // 2^100
constexpr double kSmall = 8.271806125530277e-25;  // 2^-80

template <int N>
struct GradTable {
  const void* g[N];
  void* out[N];
  long long n[N];    // elements, bit 62 set: fp32
  int first[N + 1];  // its first chunk
  int tensors;
};
constexpr long long kWide = 1LL << 62;

// Elements in front of the first 16-byte boundary, whole 16-byte pieces, and
// chunks of a tensor.
struct Cut {
  int head;
  long long vecs;
  int chunks;
};

__host__ __device__ inline Cut cut(const void* p, long long n, bool wide) {
  const int es = wide ? 4 : 2, per = 16 / es;
  Cut c;
  c.head = (int)((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15) / es;
  if (c.head > n) c.head = (int)n;
  c.vecs = (n - c.head) / per;
  c.chunks = n == 0 ? 0 : (int)((c.vecs + kChunk - 1) / kChunk);
  if (n > 0 && c.chunks == 0) c.chunks = 1;
  return c;
}

// 16 bytes that this CTA reads once
DF_DEV uint4 load_once(const uint4* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p)
               : "memory");
  return v;
}

DF_DEV float bf_lo(uint32_t v) { return __uint_as_float(v << 16); }
DF_DEV float bf_hi(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }

DF_DEV float square4(uint4 v, bool wide) {
  if (wide) {
    const float a = __uint_as_float(v.x), b = __uint_as_float(v.y);
    const float c = __uint_as_float(v.z), d = __uint_as_float(v.w);
    return (a * a + b * b) + (c * c + d * d);
  }
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  float s[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) s[i] = bf_lo(w[i]) * bf_lo(w[i]) + bf_hi(w[i]) * bf_hi(w[i]);
  return (s[0] + s[1]) + (s[2] + s[3]);
}

DF_DEV double square4_f64(uint4 v, bool wide) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  double s = 0.;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (wide) {
      const double a = __uint_as_float(w[i]);
      s += a * a;
    } else {
      const double a = bf_lo(w[i]), b = bf_hi(w[i]);
      s += a * a + b * b;
    }
  }
  return s;
}

DF_DEV float load_one(const void* p, long long i, bool wide) {
  return wide ? static_cast<const float*>(p)[i]
              : __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
}

// index of the i-th element outside the 16-byte pieces (in front of them, then
// behind them), or -1
DF_DEV long long edge_index(const Cut& c, long long n, int per, int i) {
  if (i < c.head) return i;
  const long long at = c.head + c.vecs * per + (i - c.head);
  return at < n ? at : -1;
}

template <int N>
DF_DEV int find_tensor(const GradTable<N>& t, int chunk) {
  int lo = 0, hi = t.tensors - 1;  // the last one whose first chunk is not above
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (t.first[mid] <= chunk) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

DF_DEV double block_sum(double v, double* sm) {
#pragma unroll
  for (int o = 16; o > 0; o /= 2) v += __shfl_xor_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = v;
  __syncthreads();
  double s = 0.;
  for (int w = 0; w < kThreads / 32; ++w) s += sm[w];
  return s;
}

// A chunk of a tensor: what a thread of it reads and writes.
struct Chunk {
  const void* g;
  void* out;
  long long n, v0;  // elements; this thread's first piece
  Cut cu;
  bool wide;
};

template <int N>
DF_DEV Chunk chunk_at(const GradTable<N>& t, int k, int c) {
  Chunk x;
  x.g = t.g[k];
  x.out = t.out[k];
  x.wide = (t.n[k] & kWide) != 0;
  x.n = t.n[k] & ~kWide;
  x.cu = cut(x.g, x.n, x.wide);
  x.v0 = (long long)(c - t.first[k]) * kChunk + threadIdx.x;
  return x;
}

DF_DEV void load_chunk(const Chunk& x, uint4 (&v)[kVecs]) {
  const uint4* v4 = reinterpret_cast<const uint4*>(static_cast<const char*>(x.g) +
                                                   x.cu.head * (x.wide ? 4 : 2));
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const long long at = x.v0 + i * kThreads;
    v[i] = make_uint4(0, 0, 0, 0);
    if (at < x.cu.vecs) v[i] = load_once(v4 + at);
  }
}

// The squares of a thread's part of a chunk.
DF_DEV double chunk_square(const Chunk& x, const uint4 (&v)[kVecs]) {
  double acc = 0.;
  if (x.v0 == threadIdx.x && threadIdx.x < 16) {  // the first chunk takes the edges, too
    const long long at = edge_index(x.cu, x.n, x.wide ? 4 : 8, threadIdx.x);
    if (at >= 0) {
      const double e = load_one(x.g, at, x.wide);
      acc = e * e;
    }
  }
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < kVecs; ++i) s += square4(v[i], x.wide);
  if (s >= (float)kSmall && s < (float)kBig) return acc + s;
  uint32_t any = 0;
#pragma unroll
  for (int i = 0; i < kVecs; ++i) any |= v[i].x | v[i].y | v[i].z | v[i].w;
  if (any & (x.wide ? 0x7fffffffu : 0x7fff7fffu))
#pragma unroll
    for (int i = 0; i < kVecs; ++i) acc += square4_f64(v[i], x.wide);
  return acc;
}

template <int N>
__global__ void __launch_bounds__(kThreads, kCtasPerSm)
    grad_square_kernel(const __grid_constant__ GradTable<N> t, double* partial) {
  __shared__ double sm[kThreads / 32];
  grid_dep_sync();
  const int total = t.first[t.tensors];
  double acc = 0.;
  int k = 0;
  for (int c = blockIdx.x; c < total; c += gridDim.x) {
    if (c >= t.first[k + 1]) k = find_tensor(t, c);
    const Chunk x = chunk_at(t, k, c);
    uint4 v[kVecs];
    load_chunk(x, v);
    acc += chunk_square(x, v);
  }
  const double s = block_sum(acc, sm);
  if (threadIdx.x == 0) partial[blockIdx.x] = s;
}

// the squared norm from the first pass' sums, the same in every CTA
DF_DEV double total_square(const double* partial, int n) {
  __shared__ double sm[kThreads / 32];
  double v = 0.;
  for (int i = threadIdx.x; i < n; i += kThreads) v += __ldcg(partial + i);
  const double s = block_sum(v, sm);
  __syncthreads();
  return s;
}

__global__ void __launch_bounds__(kThreads)
    grad_norm_kernel(const double* partial, int n, float* norm) {
  grid_dep_sync();
  const double s = total_square(partial, n);
  if (threadIdx.x == 0) *norm = (float)sqrt(s);
}

DF_DEV uint32_t scale_word(uint32_t w, bool wide, float a, float b) {
  if (wide) return __float_as_uint(__uint_as_float(w) * a * b);
  return pack_bf16x2(bf_lo(w) * a * b, bf_hi(w) * a * b);
}

DF_DEV void store_one(void* p, long long i, bool wide, float v) {
  if (wide) static_cast<float*>(p)[i] = v;
  else static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16(v);
}

// What a norm does to the gradients: a factor in two steps, the second one for
// factors below the normal fp32 numbers.
struct Factor {
  bool clip;
  float a, b;
};

DF_DEV Factor factor_of(double norm, double max_norm) {
  // (false where the norm is NaN: the gradients stay as they are, as with an
  // infinite one)
  Factor f;
  f.clip = norm > max_norm && norm <= 1.7976931348623157e308;
  const double x = f.clip ? max_norm / norm : 1.;
  const bool tiny = x < 1e-30;
  f.a = (float)(tiny ? x * 18446744073709551616. : x);
  f.b = tiny ? 5.421010862427522e-20f : 1.f;
  return f;
}

DF_DEV void scale_chunk(const Chunk& x, const uint4 (&v)[kVecs], Factor f) {
  char* o = static_cast<char*>(x.out) + x.cu.head * (x.wide ? 4 : 2);
  const bool whole = (reinterpret_cast<uintptr_t>(o) & 15) == 0;
  if (x.v0 == threadIdx.x && threadIdx.x < 16) {
    const long long at = edge_index(x.cu, x.n, x.wide ? 4 : 8, threadIdx.x);
    if (at >= 0) store_one(x.out, at, x.wide, load_one(x.g, at, x.wide) * f.a * f.b);
  }
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const long long at = x.v0 + i * kThreads;
    if (at >= x.cu.vecs) continue;
    const uint32_t w[4] = {scale_word(v[i].x, x.wide, f.a, f.b),
                           scale_word(v[i].y, x.wide, f.a, f.b),
                           scale_word(v[i].z, x.wide, f.a, f.b),
                           scale_word(v[i].w, x.wide, f.a, f.b)};
    if (whole) {
      __stcs(reinterpret_cast<uint4*>(o) + at, make_uint4(w[0], w[1], w[2], w[3]));
    } else if (x.wide) {
#pragma unroll
      for (int j = 0; j < 4; ++j) reinterpret_cast<uint32_t*>(o)[at * 4 + j] = w[j];
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        reinterpret_cast<uint16_t*>(o)[at * 8 + 2 * j] = (uint16_t)w[j];
        reinterpret_cast<uint16_t*>(o)[at * 8 + 2 * j + 1] = (uint16_t)(w[j] >> 16);
      }
    }
  }
}

template <int N>
__global__ void __launch_bounds__(kThreads, kCtasPerSm)
    grad_scale_kernel(const __grid_constant__ GradTable<N> t, const double* partial, int n_partial,
                      double max_norm, float* norm, int in_place) {
  const int total = t.first[t.tensors];
  int c = total - 1 - (int)blockIdx.x;  // (the grid has at most a CTA per chunk)
  int k = find_tensor(t, c);
  grid_dep_sync();
  // the first chunk is on its way while the norm is added up
  uint4 v[kVecs];
  Chunk x = chunk_at(t, k, c);
  load_chunk(x, v);
  const double nm = sqrt(total_square(partial, n_partial));
  if (norm != nullptr && blockIdx.x == 0 && threadIdx.x == 0) *norm = (float)nm;
  const Factor f = factor_of(nm, max_norm);
  if (!f.clip && in_place) return;
  while (true) {
    scale_chunk(x, v, f);
    c -= (int)gridDim.x;
    if (c < 0) break;
    if (c < t.first[k]) k = find_tensor(t, c);
    x = chunk_at(t, k, c);
    load_chunk(x, v);
  }
}

// Few chunks: one launch of one cluster does all of it, the CTAs' sums going
// from one's shared memory to the others'.  mode 0: the norm, 1: clip in place,
// 2: into other tensors.
constexpr int kClusterCtas = 8, kClusterChunks = 32;

template <int N>
__global__ void __launch_bounds__(kThreads)
    grad_cluster_kernel(const __grid_constant__ GradTable<N> t, int mode, double max_norm,
                        float* norm) {
  __shared__ double sm[kThreads / 32];
  __shared__ double sums[kClusterCtas];
  const int rank = (int)cluster_ctarank(), total = t.first[t.tensors];
  cluster_arrive();  // (waited for before anything goes to another CTA's memory)
  grid_dep_sync();
  double acc = 0.;
  uint4 v[kVecs];
  Chunk x{};
  for (int c = rank; c < total; c += kClusterCtas) {
    x = chunk_at(t, find_tensor(t, c), c);
    load_chunk(x, v);
    acc += chunk_square(x, v);
  }
  const double s = block_sum(acc, sm);
  cluster_wait();
  if (threadIdx.x < kClusterCtas)
    st_cluster_u64(cluster_map(smem_u32(&sums[rank]), threadIdx.x),
                   (unsigned long long)__double_as_longlong(s));
  cluster_sync();  // (nothing goes to another CTA's memory after it)
  double square = 0.;
  for (int i = 0; i < kClusterCtas; ++i) square += sums[i];
  const double nm = sqrt(square);
  if (rank == 0 && threadIdx.x == 0) *norm = (float)nm;
  if (mode == 0) return;
  const Factor f = factor_of(nm, max_norm);
  if (!f.clip && mode == 1) return;
  for (int c = rank; c < total; c += kClusterCtas) {
    if (total > kClusterCtas) {  // (otherwise it is the one that was read)
      x = chunk_at(t, find_tensor(t, c), c);
      load_chunk(x, v);
    }
    scale_chunk(x, v, f);
  }
}

// Checks of both entry points; total_chunks gets the chunks of all tensors.
int check_grads(int n, const void* const* g, void* const* out, const int64_t* counts,
                const int32_t* dtypes, const float* norm, const void* ws, size_t ws_bytes,
                size_t need) {
  if (n < 0 || n > (1 << 20)) return api_fail(DFLASH_ERR_ARG, "tensors must be in [0, 2^20]");
  if (n > 0 && (g == nullptr || counts == nullptr || dtypes == nullptr))
    return api_fail(DFLASH_ERR_ARG, "null list");
  if (norm == nullptr || ws == nullptr) return api_fail(DFLASH_ERR_ARG, "null norm or workspace");
  if (ws_bytes < need)
    return api_fail(DFLASH_ERR_CAPACITY, "workspace of %zu bytes, %zu needed", ws_bytes, need);
  if ((reinterpret_cast<uintptr_t>(norm) & 3) != 0 || (reinterpret_cast<uintptr_t>(ws) & 15) != 0)
    return api_fail(DFLASH_ERR_ARG, "norm or workspace not aligned");
  for (int i = 0; i < n; ++i) {
    if (dtypes[i] != DFLASH_BF16 && dtypes[i] != DFLASH_FP32)
      return api_fail(DFLASH_ERR_ARG, "tensor %d: dtype must be DFLASH_BF16 or DFLASH_FP32", i);
    if (counts[i] < 0 || counts[i] > (1LL << 40))
      return api_fail(DFLASH_ERR_ARG, "tensor %d: count out of range", i);
    if (counts[i] == 0) continue;
    const uintptr_t m = dtypes[i] == DFLASH_BF16 ? 1 : 3;
    if (g[i] == nullptr || (out != nullptr && out[i] == nullptr))
      return api_fail(DFLASH_ERR_ARG, "tensor %d is null", i);
    if (((uintptr_t)g[i] & m) != 0 || (out != nullptr && ((uintptr_t)out[i] & m) != 0))
      return api_fail(DFLASH_ERR_ARG, "tensor %d is not aligned to its type", i);
  }
  return DFLASH_OK;
}

// What is written must not overlap anything else that is written or read (the
// second pass would read scaled values): only a tensor clipped in place.
int check_overlap(int n, const void* const* g, void* const* out, const int64_t* counts,
                  const int32_t* dtypes) {
  struct Range {
    uintptr_t lo, hi;
    int i;
    bool written;
  };
  std::vector<Range> r;
  try {
    r.reserve(2 * (size_t)n);
  } catch (...) {
    return api_fail(DFLASH_ERR_MEMORY, "host allocation failed");
  }
  for (int i = 0; i < n; ++i) {
    if (counts[i] == 0) continue;
    const uintptr_t bytes = (uintptr_t)counts[i] * (dtypes[i] == DFLASH_BF16 ? 2 : 4);
    void* o = out != nullptr ? out[i] : const_cast<void*>(g[i]);
    r.push_back({(uintptr_t)o, (uintptr_t)o + bytes, i, true});
    if (o != g[i]) r.push_back({(uintptr_t)g[i], (uintptr_t)g[i] + bytes, i, false});
  }
  std::sort(r.begin(), r.end(), [](const Range& a, const Range& b) { return a.lo < b.lo; });
  uintptr_t end = 0, written_end = 0;  // of everything, and of what is written, so far
  for (const Range& x : r) {
    if (x.lo < written_end || (x.written && x.lo < end))
      return api_fail(DFLASH_ERR_ARG, "tensor %d overlaps another one", x.i);
    end = std::max(end, x.hi);
    if (x.written) written_end = std::max(written_end, x.hi);
  }
  return DFLASH_OK;
}

int num_sms(int* sms) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev);
  return e == cudaSuccess ? DFLASH_OK : api_fail(DFLASH_ERR_CUDA, "%s", cudaGetErrorString(e));
}

// fills t with tensors from i on, as many as it holds; returns the next one
template <int N>
int fill_table(GradTable<N>& t, int i, int n, const void* const* g, void* const* out,
               const int64_t* counts, const int32_t* dtypes) {
  t.tensors = 0;
  t.first[0] = 0;
  long long chunks = 0;
  for (; i < n && t.tensors < N; ++i) {
    if (counts[i] == 0) continue;
    const bool wide = dtypes[i] == DFLASH_FP32;
    const Cut c = cut(g[i], counts[i], wide);
    if (chunks + c.chunks > (1LL << 30)) break;
    const int k = t.tensors++;
    t.g[k] = g[i];
    t.out[k] = out != nullptr ? out[i] : const_cast<void*>(g[i]);
    t.n[k] = counts[i] | (wide ? kWide : 0);
    chunks += c.chunks;
    t.first[k + 1] = (int)chunks;
  }
  return i;
}

constexpr int kMaxSms = 256;

size_t workspace_bytes(int n) {
  const size_t launches = (size_t)n / kMany + 2;
  return launches * kMaxSms * kCtasPerSm * sizeof(double);
}

template <int N>
int run_norm(int n, const void* const* g, void* const* out, const int64_t* counts,
             const int32_t* dtypes, bool clip, double max_norm, float* norm, void* ws,
             size_t ws_bytes, cudaStream_t s) {
  if (int r = check_grads(n, g, out, counts, dtypes, norm, ws, ws_bytes, workspace_bytes(n)))
    return r;
  if (clip)
    if (int r = check_overlap(n, g, out, counts, dtypes)) return r;
  int sms = 0;
  if (int r = num_sms(&sms)) return r;
  const int ctas = std::min(sms, kMaxSms) * kCtasPerSm;
  double* partial = static_cast<double*>(ws);
  GradTable<N> t;
  int n_partial = 0;
  cudaError_t e = cudaSuccess;
  if (n > 0 && fill_table(t, 0, n, g, out, counts, dtypes) == n && t.tensors > 0 &&
      t.first[t.tensors] <= kClusterChunks) {
    e = launch_pdl_cluster(grad_cluster_kernel<N>, dim3(kClusterCtas), dim3(kThreads), 0, s,
                           (unsigned)kClusterCtas, t, !clip ? 0 : out == nullptr ? 1 : 2,
                           max_norm, norm);
    return e == cudaSuccess ? DFLASH_OK
                            : api_fail(DFLASH_ERR_CUDA, "gradient norm launch: %s",
                                       cudaGetErrorString(e));
  }
  const int max_partial = (int)(ws_bytes / sizeof(double));
  for (int i = 0; i < n && e == cudaSuccess;) {
    i = fill_table(t, i, n, g, out, counts, dtypes);
    if (t.tensors == 0) break;
    const int grid = std::min(ctas, t.first[t.tensors]);
    if (n_partial + grid > max_partial)
      return api_fail(DFLASH_ERR_CAPACITY, "workspace too small");
    e = launch_pdl(grad_square_kernel<N>, dim3(grid), dim3(kThreads), 0, s, t, partial + n_partial);
    n_partial += grid;
  }
  if (e == cudaSuccess && (!clip || n_partial == 0))
    e = launch_pdl(grad_norm_kernel, dim3(1), dim3(kThreads), 0, s, partial, n_partial, norm);
  for (int i = 0; clip && n_partial > 0 && i < n && e == cudaSuccess;) {
    const bool first = i == 0;
    i = fill_table(t, i, n, g, out, counts, dtypes);
    if (t.tensors == 0) break;
    const int grid = std::min(ctas, t.first[t.tensors]);
    e = launch_pdl(grad_scale_kernel<N>, dim3(grid), dim3(kThreads), 0, s, t, partial, n_partial,
                   max_norm, first ? norm : nullptr, out == nullptr ? 1 : 0);
  }
  return e == cudaSuccess ? DFLASH_OK
                          : api_fail(DFLASH_ERR_CUDA, "gradient norm launch: %s",
                                     cudaGetErrorString(e));
}

}  // namespace
}  // namespace df

using namespace df;

extern "C" {

int dflash_grad_norm_workspace(int n_tensors, size_t* bytes) {
  if (bytes == nullptr) return api_fail(DFLASH_ERR_ARG, "bytes is null");
  if (n_tensors < 0 || n_tensors > (1 << 20))
    return api_fail(DFLASH_ERR_ARG, "tensors must be in [0, 2^20]");
  *bytes = workspace_bytes(n_tensors);
  return DFLASH_OK;
}

int dflash_grad_norm(int n_tensors, const void* const* grads, const int64_t* counts,
                     const int32_t* dtypes, float* norm, void* workspace, size_t workspace_bytes,
                     dflash_stream stream) {
  return (n_tensors <= kFew ? run_norm<kFew> : run_norm<kMany>)(
      n_tensors, grads, nullptr, counts, dtypes, false, 0., norm, workspace, workspace_bytes,
      static_cast<cudaStream_t>(stream));
}

int dflash_clip_grad_norm(int n_tensors, const void* const* grads, void* const* out,
                          const int64_t* counts, const int32_t* dtypes, double max_norm,
                          float* norm, void* workspace, size_t workspace_bytes,
                          dflash_stream stream) {
  if (!(max_norm >= 0.)) return api_fail(DFLASH_ERR_ARG, "max_norm must be >= 0");
  return (n_tensors <= kFew ? run_norm<kFew> : run_norm<kMany>)(
      n_tensors, grads, out, counts, dtypes, true, max_norm, norm, workspace, workspace_bytes,
      static_cast<cudaStream_t>(stream));
}

}  // extern "C"
