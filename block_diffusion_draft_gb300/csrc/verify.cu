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
// point goes over it again (from L2) to find the step, eight steps' loads at a
// time, and then the token.  Latency bounds a call of few sequences, HBM one of
// many.
#include <algorithm>
#include <atomic>

#include "internal.h"
#include "ptx.cuh"

namespace df {
namespace {

constexpr int kWarps = 16;
constexpr int kThreads = kWarps * 32;
// 16 CTAs are the most that this GPU puts into a cluster, beyond the portable 8:
// one sequence of 15 drafts and 150000 tokens takes 11.6 us, with 8 14.4 us.
constexpr int kMaxCluster = 16;

// min(max(p, 0), 1) in multiples of 2^-44, cut off below, as hi * 2^22 + lo; NaN
// counts as 0.  Adding 2 towards zero leaves the multiples of 2^-22 in the
// mantissa; what is left over is exact, and adding 2^-21 to it leaves its
// multiples of 2^-44.  (Conversions to 64-bit integers took 35 us, shifts of the
// mantissa 29 us where this takes 21 us, on 32 sequences of 15 drafts and 150000
// tokens.)
struct Fixed {
  int hi, lo;
};

DF_DEV Fixed fixed(float p) {
  p = fminf(fmaxf(p, 0.f), 1.f);
  const float t = __fadd_rz(p, 2.f);
  const float rest = __fadd_rn(p, -__fadd_rn(t, -2.f));
  constexpr float unit = 4.76837158203125e-07f;  // 2^-21
  Fixed f;
  f.hi = __float_as_int(t) - 0x40000000;
  f.lo = __float_as_int(__fadd_rz(rest, unit)) - 0x35000000;
  return f;
}

// floor(min(max(u, 0), 1) * total) without rounding, NaN as 0, for a total below
// 2^63: u is a 24-bit number times a power of two, their product has 87 bits.  (In
// 64-bit floats it is rounded to 53, up to the next whole number at times.)
DF_DEV unsigned long long scaled(float u, unsigned long long total) {
  if (!(u > 0.f)) return 0ull;
  const uint32_t bits = __float_as_uint(fminf(u, 1.f)), field = bits >> 23;
  const unsigned long long m = (bits & 0x7fffffu) | (field != 0u ? 0x800000u : 0u);
  const int shift = 150 - (int)max(field, 1u);  // 23 to 149
  const unsigned long long hi = __umul64hi(m, total);
  if (shift >= 64) return hi >> min(shift - 64, 63);  // (hi < 2^23)
  return hi << (64 - shift) | (m * total) >> shift;
}

DF_DEV long long whole(int hi, int lo) { return (long long)hi * (1 << 22) + lo; }

template <typename T>
DF_DEV float prob(const T* p, long long i);
template <>
DF_DEV float prob<float>(const float* p, long long i) { return __ldcg(p + i); }
template <>
DF_DEV float prob<uint16_t>(const uint16_t* p, long long i) {
  return __uint_as_float((uint32_t)__ldcg(p + i) << 16);
}

// E = 16 / sizeof(T) probabilities of a row, `by` apart, zero past its end: 16
// bytes in one load where the row's start is aligned and they are neighbours
template <typename T, bool VEC>
DF_DEV void load_row(const T* row, int i, int by, int vocab, float (&x)[16 / sizeof(T)]) {
  constexpr int E = 16 / sizeof(T);
  if (VEC && i + E <= vocab) {
    const uint4 w = __ldcg(reinterpret_cast<const uint4*>(row + i));
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
    for (int e = 0; e < E; ++e) x[e] = i + e * by < vocab ? prob<T>(row, i + e * by) : 0.f;
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
DF_DEV void weights(const Row<T>& r, int i, int by, int vocab,
                    unsigned long long (&w)[16 / sizeof(T)]) {
  constexpr int E = 16 / sizeof(T);
  float x[E];
  load_row<T, VEC>(r.p, i, by, vocab, x);
  if (r.q != nullptr) {
    float y[E];
    load_row<T, VEC>(r.q, i, by, vocab, y);
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const Fixed f = fixed(x[e]), g = fixed(y[e]);
      const long long d = whole(f.hi - g.hi, f.lo - g.lo);
      w[e] = d > 0 ? (unsigned long long)d : 0ull;
    }
  } else {
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const Fixed f = fixed(x[e]);
      w[e] = i + e * by == r.out ? 0ull : (unsigned long long)whole(f.hi, f.lo);
    }
  }
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(kThreads)
    verify_kernel(const __grid_constant__ VerifyArgs a, int cluster) {
  constexpr int E = 16 / sizeof(T), STEP = 32 * E;
  __shared__ unsigned long long warp_sum[2][kWarps];
  __shared__ unsigned long long cta_sum[2][kMaxCluster];
  __shared__ int first_bad;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = cluster > 1 ? (int)cluster_ctarank() : 0;
  const int b = blockIdx.x / cluster;
  // what a CTA exchanges with its cluster goes to CTAs that must have started
  if (cluster > 1) cluster_arrive();
  grid_dep_sync();

  // the first rejected draft
  const T* target = static_cast<const T*>(a.target) + (long long)b * a.target_batch;
  const T* draft = a.draft == nullptr
                       ? nullptr
                       : static_cast<const T*>(a.draft) + (long long)b * a.draft_batch;
  const int* drafts = a.draft_tokens + (long long)b * a.n_draft;
  const float u_sample = __ldcg(a.u_sample + b);
  const int n_seq = a.seq_drafts != nullptr ? __ldcg(a.seq_drafts + b) : a.n_draft;
  if (threadIdx.x == 0) first_bad = a.n_draft;
  __syncthreads();
  for (int i = threadIdx.x; i < a.n_draft; i += kThreads) {
    const int x = __ldcg(drafts + i);
    const double u = (double)__ldcg(a.u_accept + (long long)b * a.n_draft + i);
    bool ok = x >= 0 && x < a.vocab && i < n_seq;
    if (ok) {
      const double p = (double)prob<T>(target, (long long)i * a.target_row + x);
      const double q = draft == nullptr ? 1.0
                                        : (double)prob<T>(draft, (long long)i * a.draft_row + x);
      ok = u * q < p;  // 24-bit factors: the product is exact
    }
    if (!ok) atomicMin(&first_bad, i);
  }
  __syncthreads();
  const int n = min(max(n_seq, 0), a.n_draft);
  const int k = first_bad;
  int* tokens = a.tokens + (long long)b * (a.n_draft + 1);
  if (rank == 0) {
    if (threadIdx.x == 0) a.accepted[b] = k;
    for (int i = threadIdx.x; i <= a.n_draft; i += kThreads)
      if (i != k) tokens[i] = i < k ? __ldcg(drafts + i) : -1;
  }

  Row<T> r;
  r.p = target + (long long)k * a.target_row;
  r.q = k < n && draft != nullptr ? draft + (long long)k * a.draft_row : nullptr;
  r.out = k < n && draft == nullptr ? __ldcg(drafts + k) : -1;
  // this warp's share of the row: whole steps, in order
  const int shares = cluster * kWarps;
  const int steps = (a.vocab + STEP - 1) / STEP;
  const int mine = rank * kWarps + warp;
  const int s0 = (int)((long long)mine * steps / shares);
  const int s1 = (int)((long long)(mine + 1) * steps / shares);

  // pass 1 only when the difference left no weight at all: the target's row
  for (int pass = 0; pass < 2; ++pass) {
    unsigned long long sum = 0ull;
    // (the order of a sum does not matter: a step's elements side by side where
    // they are loaded one by one)
    const int first = VEC ? lane * E : lane, by = VEC ? 1 : 32;
#pragma unroll 4
    for (int s = s0; s < s1; ++s) {
      unsigned long long w[E];
      weights<T, VEC>(r, s * STEP + first, by, a.vocab, w);
#pragma unroll
      for (int e = 0; e < E; ++e) sum += w[e];
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    if (lane == 0) warp_sum[pass][warp] = sum;
    __syncthreads();
    if (cluster > 1 && pass == 0) cluster_wait();
    if (warp == 0) {
      unsigned long long t = lane < kWarps ? warp_sum[pass][lane] : 0ull;
#pragma unroll
      for (int d = kWarps / 2; d > 0; d >>= 1) t += __shfl_xor_sync(0xffffffffu, t, d);
      // to every CTA of the cluster, this one among them
      if (cluster == 1) {
        if (lane == 0) cta_sum[pass][0] = t;
      } else {
        if (lane < cluster)
          st_cluster_u64(cluster_map(smem_u32(&cta_sum[pass][rank]), (uint32_t)lane), t);
      }
    }
    if (cluster > 1) {
      __syncwarp();
      cluster_sync();
    } else {
      __syncthreads();
    }
    unsigned long long before = 0ull, total = 0ull;
    for (int c = 0; c < cluster; ++c) {
      const unsigned long long t = cta_sum[pass][c];
      if (c < rank) before += t;
      total += t;
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
    const unsigned long long t = min(scaled(u_sample, total), total - 1ull);
    for (int i = 0; i < warp; ++i) before += warp_sum[pass][i];
    if (t >= before && t - before < sum) {
      // the drawn point lies in this warp's share: the step that holds it, and
      // there the first token whose cumulative weight exceeds it
      constexpr int AHEAD = 8;
      int step = s0;
      for (bool found = false; !found; ) {
        unsigned long long own[AHEAD];
#pragma unroll
        for (int j = 0; j < AHEAD; ++j) {
          own[j] = 0ull;
          if (step + j < s1) {
            unsigned long long w[E];
            weights<T, VEC>(r, (step + j) * STEP + first, by, a.vocab, w);
#pragma unroll
            for (int e = 0; e < E; ++e) own[j] += w[e];
          }
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1)
#pragma unroll
          for (int j = 0; j < AHEAD; ++j) own[j] += __shfl_xor_sync(0xffffffffu, own[j], d);
#pragma unroll
        for (int j = 0; j < AHEAD; ++j) {
          if (found) continue;
          if (t < before + own[j] || step + 1 >= s1) {
            found = true;
          } else {
            before += own[j];
            ++step;
          }
        }
      }
      unsigned long long w[E], own = 0ull;
      const int i = step * STEP + lane * E;
      weights<T, VEC>(r, i, 1, a.vocab, w);
#pragma unroll
      for (int e = 0; e < E; ++e) own += w[e];
      unsigned long long upto = own;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const unsigned long long o = __shfl_up_sync(0xffffffffu, upto, d);
        if (lane >= d) upto += o;
      }
      const unsigned over = __ballot_sync(0xffffffffu, before + upto > t);
      if (over != 0u && lane == __ffs(over) - 1) {
        unsigned long long c = before + upto - own;
        int e = 0;
#pragma unroll
        for (int f = 0; f < E - 1; ++f) {
          c += w[f];
          if (c <= t) e = f + 1;
        }
        tokens[k] = i + e;
      }
    }
    break;
  }
}

template <typename T, bool VEC>
cudaError_t launch_t(const VerifyArgs& a, int cluster, cudaStream_t s) {
  static std::atomic<unsigned long long> done{0};
  if (!done_on_device(done)) {
    const cudaError_t e = cudaFuncSetAttribute(
        verify_kernel<T, VEC>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    mark_device(done);
  }
  return launch_pdl_cluster(verify_kernel<T, VEC>, dim3((unsigned)(a.batch * cluster)),
                            dim3(kThreads), 0, s, (unsigned)cluster, a, cluster);
}

}  // namespace

int launch_verify(const VerifyArgs& a, int bf16, int num_sms, cudaStream_t s) {
  // CTAs per sequence: as many as run at a time (two per SM), as long as a
  // warp keeps a step of 32 16-byte loads (128 sequences of 50001 tokens in two
  // waves of four CTAs each took 26 us, in one of two 21 us)
  const int step = 32 * (bf16 ? 8 : 4);
  int cluster = 1;
  while (cluster < kMaxCluster && (long long)a.batch * cluster * 2 <= 2LL * num_sms &&
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
