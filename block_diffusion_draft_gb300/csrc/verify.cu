// verify.cu -- verification of drafted tokens against the target's
// probabilities, from given uniform numbers.
//
// Sequence b has drafted x_0 .. x_{n-1} from distributions q_i; the target
// gives p_0 .. p_n.  Draft i is accepted while u_i q_i(x_i) < p_i(x_i).  At
// the first rejection a the next token is drawn from max(p_a - q_a, 0), with
// every draft accepted from p_n; both by inversion: the first token whose
// cumulative weight exceeds u * (sum of the weights).  Accepted tokens and
// that one are then distributed as the target's own samples.
//
// Weights are sums of up to 2^19 numbers that are compared with one another,
// so they are whole multiples of 2^-44 in 64-bit integers (a probability is
// cut off below): sums are exact and the same in every order, so the split of
// a row over warps and CTAs cannot move a token's border.  A weight's cut-off
// is below 2^-44, far under the 2^-24 relative step of the inputs.  64-bit
// float sums would cost more here: this GPU's fp64 rate is about 1/30 of its
// integer rate.
//
// Only two rows of a sequence's probabilities decide (one when everything is
// accepted or the drafts have no distribution), so that is all that is read:
// 2 * vocab * 4 bytes.  A cluster of CTAs takes a sequence; every CTA finds
// the rejection itself (a gather of n probabilities), each warp sums its
// contiguous share of the row, the CTAs exchange their sums through
// distributed shared memory, and the one warp whose share holds the drawn
// point goes over it again (from L2) to find the token.  Latency bounds a
// call of few sequences, HBM one of many.
#include <algorithm>
#include <atomic>

#include "internal.h"
#include "ptx.cuh"

namespace df {
namespace {

constexpr int kWarps = 16;
constexpr int kThreads = kWarps * 32;
constexpr int kMaxCluster = 8;
constexpr unsigned long long kOne = 1ull << 44;

// min(max(p, 0), 1) in multiples of 2^-44, cut off below; NaN counts as 0
DF_DEV unsigned long long fixed(float p) {
  if (!(p > 0.f)) return 0ull;
  if (p >= 1.f) return kOne;
  const uint32_t b = __float_as_uint(p);
  // p = mant * 2^(field - 150): mant * 2^21 is p * 2^44 for field 127
  const uint32_t k = 127u - (b >> 23);
  const unsigned long long m = (unsigned long long)((b & 0x7fffffu) | 0x800000u) << 21;
  return k > 63u ? 0ull : m >> k;
}

template <typename T>
DF_DEV float prob(const T* p, long long i);
template <>
DF_DEV float prob<float>(const float* p, long long i) { return __ldg(p + i); }
template <>
DF_DEV float prob<uint16_t>(const uint16_t* p, long long i) {
  return __uint_as_float((uint32_t)__ldg(p + i) << 16);
}

// E consecutive probabilities of a row (16 bytes), zero past its end
template <typename T, bool VEC>
DF_DEV void load_row(const T* row, int i, int vocab, float (&x)[16 / sizeof(T)]) {
  constexpr int E = 16 / sizeof(T);
  if (VEC && i + E <= vocab) {
    const uint4 w = __ldg(reinterpret_cast<const uint4*>(row + i));
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if constexpr (sizeof(T) == 4) {
        x[e] = __uint_as_float(u[e]);
      } else {
        x[2 * e] = __uint_as_float(u[e] << 16);
        x[2 * e + 1] = __uint_as_float(u[e] & 0xffff0000u);
      }
    }
  } else {
#pragma unroll
    for (int e = 0; e < E; ++e) x[e] = i + e < vocab ? prob<T>(row, i + e) : 0.f;
  }
}

// what a pass draws from: the target's row, less the draft's row or with one
// token taken out
template <typename T>
struct Row {
  const T* p;
  const T* q;   // or null
  int out;      // token without weight, or -1
};

template <typename T, bool VEC>
DF_DEV void weights(const Row<T>& r, int i, int vocab,
                    unsigned long long (&w)[16 / sizeof(T)]) {
  constexpr int E = 16 / sizeof(T);
  float x[E];
  load_row<T, VEC>(r.p, i, vocab, x);
  if (r.q != nullptr) {
    float y[E];
    load_row<T, VEC>(r.q, i, vocab, y);
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const long long d = (long long)fixed(x[e]) - (long long)fixed(y[e]);
      w[e] = d > 0 ? (unsigned long long)d : 0ull;
    }
  } else {
#pragma unroll
    for (int e = 0; e < E; ++e) w[e] = i + e == r.out ? 0ull : fixed(x[e]);
  }
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(kThreads)
    verify_kernel(const __grid_constant__ VerifyArgs a, int cluster) {
  constexpr int E = 16 / sizeof(T), STEP = 32 * E;
  __shared__ unsigned long long warp_sum[2][kWarps];
  __shared__ unsigned long long cta_sum[2];
  __shared__ int first_bad;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = cluster > 1 ? (int)cluster_ctarank() : 0;
  const int b = blockIdx.x / cluster;
  grid_dep_sync();

  // the first rejected draft
  int n = a.n_draft;
  if (a.seq_drafts != nullptr) n = min(max(__ldg(a.seq_drafts + b), 0), n);
  if (threadIdx.x == 0) first_bad = n;
  __syncthreads();
  const T* target = static_cast<const T*>(a.target) + (long long)b * a.target_batch;
  const T* draft = a.draft == nullptr
                       ? nullptr
                       : static_cast<const T*>(a.draft) + (long long)b * a.draft_batch;
  const int* drafts = a.draft_tokens + (long long)b * a.n_draft;
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const int x = __ldg(drafts + i);
    const double u = (double)__ldg(a.u_accept + (long long)b * a.n_draft + i);
    bool ok = x >= 0 && x < a.vocab;
    if (ok) {
      const double p = (double)prob<T>(target, (long long)i * a.target_row + x);
      const double q = draft == nullptr ? 1.0
                                        : (double)prob<T>(draft, (long long)i * a.draft_row + x);
      ok = u * q < p;  // 24-bit factors: the product is exact
    }
    if (!ok) atomicMin(&first_bad, i);
  }
  __syncthreads();
  const int k = first_bad;
  int* tokens = a.tokens + (long long)b * (a.n_draft + 1);
  if (rank == 0) {
    if (threadIdx.x == 0) a.accepted[b] = k;
    for (int i = threadIdx.x; i <= a.n_draft; i += kThreads)
      if (i != k) tokens[i] = i < k ? __ldg(drafts + i) : -1;
  }

  Row<T> r;
  r.p = target + (long long)k * a.target_row;
  r.q = k < n && draft != nullptr ? draft + (long long)k * a.draft_row : nullptr;
  r.out = k < n && draft == nullptr ? __ldg(drafts + k) : -1;
  // this warp's share of the row: whole steps, in order
  const int shares = cluster * kWarps;
  const int steps = (a.vocab + STEP - 1) / STEP;
  const int mine = rank * kWarps + warp;
  const int s0 = (int)((long long)mine * steps / shares);
  const int s1 = (int)((long long)(mine + 1) * steps / shares);

  // pass 1 only when the difference left no weight at all: the target's row
  for (int pass = 0; pass < 2; ++pass) {
    unsigned long long sum = 0ull;
#pragma unroll 4
    for (int s = s0; s < s1; ++s) {
      unsigned long long w[E];
      weights<T, VEC>(r, s * STEP + lane * E, a.vocab, w);
#pragma unroll
      for (int e = 0; e < E; ++e) sum += w[e];
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    if (lane == 0) warp_sum[pass][warp] = sum;
    __syncthreads();
    if (threadIdx.x == 0) {
      unsigned long long t = 0ull;
      for (int i = 0; i < kWarps; ++i) t += warp_sum[pass][i];
      cta_sum[pass] = t;
    }
    unsigned long long before = 0ull, total = 0ull;
    if (cluster > 1) {
      __syncwarp();
      cluster_sync();
      for (int c = 0; c < cluster; ++c) {
        const unsigned long long t =
            ld_cluster_u64(cluster_map(smem_u32(&cta_sum[pass]), (uint32_t)c));
        if (c < rank) before += t;
        total += t;
      }
    } else {
      __syncthreads();
      total = cta_sum[pass];
    }
    if (total == 0ull && (r.q != nullptr || r.out >= 0)) {
      r.q = nullptr;
      r.out = -1;
      continue;
    }
    if (total == 0ull) {
      if (rank == 0 && threadIdx.x == 0) tokens[k] = -1;
      break;
    }
    const float u = __ldg(a.u_sample + b);
    unsigned long long t = u > 0.f ? (unsigned long long)((double)min(u, 1.f) * (double)total) : 0ull;
    t = min(t, total - 1ull);
    for (int i = 0; i < warp; ++i) before += warp_sum[pass][i];
    if (t >= before && t - before < sum) {
      // the drawn point lies in this warp's share: the first token whose
      // cumulative weight exceeds it
      for (int s = s0; s < s1; ++s) {
        unsigned long long w[E], own = 0ull;
        const int i = s * STEP + lane * E;
        weights<T, VEC>(r, i, a.vocab, w);
#pragma unroll
        for (int e = 0; e < E; ++e) own += w[e];
        unsigned long long upto = own;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const unsigned long long o = __shfl_up_sync(0xffffffffu, upto, d);
          if (lane >= d) upto += o;
        }
        const unsigned over = __ballot_sync(0xffffffffu, before + upto > t);
        if (over != 0u) {
          if (lane == __ffs(over) - 1) {
            unsigned long long c = before + upto - own;
            int e = 0;
#pragma unroll
            for (int f = 0; f < E - 1; ++f) {
              c += w[f];
              if (c <= t) e = f + 1;
            }
            tokens[k] = i + e;
          }
          break;
        }
        before += __shfl_sync(0xffffffffu, upto, 31);
      }
    }
    break;
  }
  if (cluster > 1) {
    // no CTA leaves while another may still read its sum
    __syncwarp();
    cluster_sync();
  }
}

template <typename T, bool VEC>
cudaError_t launch_t(const VerifyArgs& a, int cluster, cudaStream_t s) {
  return launch_pdl_cluster(verify_kernel<T, VEC>, dim3((unsigned)(a.batch * cluster)),
                            dim3(kThreads), 0, s, (unsigned)cluster, a, cluster);
}

}  // namespace

int launch_verify(const VerifyArgs& a, int bf16, int num_sms, cudaStream_t s) {
  // CTAs per sequence: enough for the whole GPU, as long as a warp keeps a
  // step of 32 16-byte loads
  const int step = 32 * (bf16 ? 8 : 4);
  int cluster = 1;
  while (cluster < kMaxCluster && (long long)a.batch * cluster < 2LL * num_sms &&
         (long long)cluster * kWarps * step < a.vocab)
    cluster *= 2;
  const size_t size = bf16 ? 2 : 4;
  auto rows16 = [&](const void* p, long long batch, long long row, int rows) {
    return ((uintptr_t)p & 15) == 0 && (a.batch == 1 || (size_t)batch * size % 16 == 0) &&
           (rows == 1 || (size_t)row * size % 16 == 0);
  };
  const bool vec =
      rows16(a.target, a.target_batch, a.target_row, a.n_draft + 1) &&
      (a.draft == nullptr || rows16(a.draft, a.draft_batch, a.draft_row, a.n_draft));
  if (bf16)
    return vec ? launch_t<uint16_t, true>(a, cluster, s) : launch_t<uint16_t, false>(a, cluster, s);
  return vec ? launch_t<float, true>(a, cluster, s) : launch_t<float, false>(a, cluster, s);
}

}  // namespace df
