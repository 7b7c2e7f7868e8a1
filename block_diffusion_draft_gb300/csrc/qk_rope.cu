// qk_rope.cu -- per-head RMSNorm and rotation of queries and keys in one pass,
// and its gradient, for training around the packed attention core.
//
// Per head (d channels) of a row at position p, with r = 1 / sqrt(mean(x^2) + eps):
//   z = g * x * r,  y_j = z_j cos - z_{j+d/2} sin,  y_{j+d/2} = z_{j+d/2} cos + z_j sin
// and back, with w the gradient of y turned by -p, u = g * w and s = sum(u * x):
//   dx = r * (u - x * r^2 * s / d),   dg = sum over rows and heads of w * x * r.
// Both sums (x^2 and u * x) go through one reduction.
//
// HBM bounds it: every value is read and written once.  A lane holds four
// channels of either half of a head, so a pair's two channels meet in one
// lane without an exchange and every access is a contiguous half head.
#include <algorithm>

#include "internal.h"
#include "ptx.cuh"

namespace df {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;

DF_DEV void load4(const float* p, float (&v)[4]) {
  const float4 t = *reinterpret_cast<const float4*>(p);
  v[0] = t.x, v[1] = t.y, v[2] = t.z, v[3] = t.w;
}

DF_DEV void load4(const __nv_bfloat16* p, float (&v)[4]) {
  const uint2 t = *reinterpret_cast<const uint2*>(p);
  v[0] = __uint_as_float(t.x << 16), v[1] = __uint_as_float(t.x & 0xffff0000u);
  v[2] = __uint_as_float(t.y << 16), v[3] = __uint_as_float(t.y & 0xffff0000u);
}

DF_DEV void store4(float* p, const float (&v)[4]) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
}

DF_DEV void store4(__nv_bfloat16* p, const float (&v)[4]) {
  *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
}

template <typename T>
DF_DEV T* head_ptr(const HeadView& h, int b, int r) {
  return reinterpret_cast<T*>(h.p) + b * h.batch + r * h.row;
}

// (row of the call, which of q and k, first head) of a warp's item: `per`
// heads of one row
struct Item {
  int b, r, kind, head;
};

DF_DEV Item item_at(const QkRopeArgs& a, long long i, int per) {
  const int cq = (a.heads[0] + per - 1) / per, ck = (a.heads[1] + per - 1) / per;
  const int row = (int)(i / (cq + ck)), c = (int)(i - (long long)row * (cq + ck));
  Item t;
  t.kind = c >= cq;
  t.head = (t.kind ? c - cq : c) * per;
  t.b = row / a.rows;
  t.r = row - t.b * a.rows;
  return t;
}

DF_DEV const float2* rope_row(const QkRopeArgs& a, const Item& t) {
  int pos = __ldg(a.positions + (long long)t.b * a.rows + t.r);
  if (pos < 0 || pos >= a.max_pos) {
    record_error(a.err, 2 /* DFLASH_DEV_POSITION */);
    pos = min(max(pos, 0), a.max_pos - 1);
  }
  return a.rope + (long long)pos * (a.d / 2);
}

template <typename T>
DF_DEV void load_gain(const QkRopeArgs& a, int kind, int j, float (&v)[4]) {
  if (a.gain[kind] != nullptr)
    load4(static_cast<const T*>(a.gain[kind]) + j, v);
  else
    load4(a.gain32[kind] + j, v);
}

// Heads of D channels whose tensors allow 4-channel accesses.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) qk_rope_kernel(const __grid_constant__ QkRopeArgs a) {
  constexpr int L = D / 8, G = 32 / L, U = 4;
  const int lane = threadIdx.x & 31, l = lane % L, g = lane / L;
  grid_dep_sync();
  const long long i = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (i >= a.items) return;
  const Item t = item_at(a, i, G * U);
  const int n = a.heads[t.kind];
  const T* src = head_ptr<const T>(a.x[t.kind], t.b, t.r) + 4 * l;
  float lo[U][4], hi[U][4];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int h = t.head + u * G + g;
    if (h < n) {
      load4(src + h * a.x[t.kind].head, lo[u]);
      load4(src + h * a.x[t.kind].head + D / 2, hi[u]);
    }
  }
  const float2* rp = rope_row(a, t) + 4 * l;
  const float4 c01 = __ldg(reinterpret_cast<const float4*>(rp));
  const float4 c23 = __ldg(reinterpret_cast<const float4*>(rp) + 1);
  const float cs[4] = {c01.x, c01.z, c23.x, c23.z}, sn[4] = {c01.y, c01.w, c23.y, c23.w};
  float ga[4], gb[4];
  load_gain<T>(a, t.kind, 4 * l, ga);
  load_gain<T>(a, t.kind, 4 * l + D / 2, gb);
  T* dst = head_ptr<T>(a.out[t.kind], t.b, t.r) + 4 * l;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int h = t.head + u * G + g;
    float ss = 0.f;
    if (h < n)
#pragma unroll
      for (int j = 0; j < 4; ++j) ss += lo[u][j] * lo[u][j] + hi[u][j] * hi[u][j];
#pragma unroll
    for (int o = L / 2; o > 0; o /= 2) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    if (h >= n) continue;
    const float r = 1.f / sqrtf(ss * (1.f / D) + a.eps);
    float ya[4], yb[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float za = lo[u][j] * r * ga[j], zb = hi[u][j] * r * gb[j];
      ya[j] = za * cs[j] - zb * sn[j];
      yb[j] = zb * cs[j] + za * sn[j];
    }
    store4(dst + h * a.out[t.kind].head, ya);
    store4(dst + h * a.out[t.kind].head + D / 2, yb);
  }
}

// The CTA's sums for the gains' gradients: lanes of a warp that hold the same
// channels (L apart), then the warps in order, to partial[CTA][kind][d].
template <int D>
DF_DEV void store_gain_sums(const QkRopeArgs& a, float (&acc)[2][8]) {
  constexpr int L = D / 8;
  __shared__ float red[kWarps][2][D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int k = 0; k < 2; ++k)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float v = acc[k][j];
#pragma unroll
      for (int o = 16; o >= L; o /= 2) v += __shfl_xor_sync(0xffffffffu, v, o);
      if (lane < L) red[warp][k][4 * lane + (j & 3) + (j >> 2) * (D / 2)] = v;
    }
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * D; i += kThreads) {
    float v = 0.f;
    for (int w = 0; w < kWarps; ++w) v += (&red[w][0][0])[i];
    a.partial[(size_t)blockIdx.x * 2 * D + i] = v;
  }
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads)
    qk_rope_bwd_kernel(const __grid_constant__ QkRopeArgs a) {
  constexpr int L = D / 8, G = 32 / L, U = 2;
  const int lane = threadIdx.x & 31, l = lane % L, g = lane / L;
  grid_dep_sync();
  float acc[2][8] = {};
  for (long long i = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5); i < a.items;
       i += (long long)gridDim.x * kWarps) {
    const Item t = item_at(a, i, G * U);
    const int n = a.heads[t.kind];
    const T* src = head_ptr<const T>(a.x[t.kind], t.b, t.r) + 4 * l;
    const T* dsrc = head_ptr<const T>(a.dy[t.kind], t.b, t.r) + 4 * l;
    float xa[U][4], xb[U][4], wa[U][4], wb[U][4];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = t.head + u * G + g;
      if (h < n) {
        load4(src + h * a.x[t.kind].head, xa[u]);
        load4(src + h * a.x[t.kind].head + D / 2, xb[u]);
        load4(dsrc + h * a.dy[t.kind].head, wa[u]);
        load4(dsrc + h * a.dy[t.kind].head + D / 2, wb[u]);
      }
    }
    const float2* rp = rope_row(a, t) + 4 * l;
    const float4 c01 = __ldg(reinterpret_cast<const float4*>(rp));
    const float4 c23 = __ldg(reinterpret_cast<const float4*>(rp) + 1);
    const float cs[4] = {c01.x, c01.z, c23.x, c23.z}, sn[4] = {c01.y, c01.w, c23.y, c23.w};
    float ga[4], gb[4];
    load_gain<T>(a, t.kind, 4 * l, ga);
    load_gain<T>(a, t.kind, 4 * l + D / 2, gb);
    T* dst = head_ptr<T>(a.out[t.kind], t.b, t.r) + 4 * l;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = t.head + u * G + g;
      float ss = 0.f, ux = 0.f;
      if (h < n)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float da = wa[u][j], db = wb[u][j];
          wa[u][j] = da * cs[j] + db * sn[j];
          wb[u][j] = db * cs[j] - da * sn[j];
          ss += xa[u][j] * xa[u][j] + xb[u][j] * xb[u][j];
          ux += wa[u][j] * ga[j] * xa[u][j] + wb[u][j] * gb[j] * xb[u][j];
        }
#pragma unroll
      for (int o = L / 2; o > 0; o /= 2) {
        ss += __shfl_xor_sync(0xffffffffu, ss, o);
        ux += __shfl_xor_sync(0xffffffffu, ux, o);
      }
      if (h >= n) continue;
      const float r = 1.f / sqrtf(ss * (1.f / D) + a.eps);
      const float m = r * r * ux * (1.f / D);
      float da[4], db[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        da[j] = r * (wa[u][j] * ga[j] - xa[u][j] * m);
        db[j] = r * (wb[u][j] * gb[j] - xb[u][j] * m);
        const float pa = wa[u][j] * xa[u][j] * r, pb = wb[u][j] * xb[u][j] * r;
        // (selects, so that the sums stay in registers)
        acc[0][j] += t.kind ? 0.f : pa;
        acc[0][4 + j] += t.kind ? 0.f : pb;
        acc[1][j] += t.kind ? pa : 0.f;
        acc[1][4 + j] += t.kind ? pb : 0.f;
      }
      store4(dst + h * a.out[t.kind].head, da);
      store4(dst + h * a.out[t.kind].head + D / 2, db);
    }
  }
  store_gain_sums<D>(a, acc);
}

// Any even head size up to 256 and any alignment, fp32: a warp takes a head,
// a lane the pairs lane, lane + 32, ...
constexpr int kPairs = 4;

template <bool BWD>
__global__ void __launch_bounds__(kThreads)
    qk_rope_any_kernel(const __grid_constant__ QkRopeArgs a) {
  __shared__ float red[BWD ? kWarps : 1][2][256];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, half = a.d / 2;
  grid_dep_sync();
  float acc[2][2 * kPairs] = {};
  for (long long i = (long long)blockIdx.x * kWarps + warp; i < a.items;
       i += (long long)gridDim.x * kWarps) {
    const Item t = item_at(a, i, 1);
    const float* x = head_ptr<const float>(a.x[t.kind], t.b, t.r) + t.head * a.x[t.kind].head;
    const float* dy = BWD ? head_ptr<const float>(a.dy[t.kind], t.b, t.r) +
                                t.head * a.dy[t.kind].head
                          : nullptr;
    const float* gain = a.gain[t.kind] != nullptr ? static_cast<const float*>(a.gain[t.kind])
                                                  : a.gain32[t.kind];
    const float2* rp = rope_row(a, t);
    float xa[kPairs], xb[kPairs], wa[kPairs], wb[kPairs], ga[kPairs], gb[kPairs];
    float2 cs[kPairs];
    float ss = 0.f, ux = 0.f;
#pragma unroll
    for (int q = 0; q < kPairs; ++q) {
      const int j = lane + 32 * q;
      xa[q] = xb[q] = wa[q] = wb[q] = ga[q] = gb[q] = 0.f;
      cs[q] = make_float2(1.f, 0.f);
      if (j < half) {
        xa[q] = x[j], xb[q] = x[j + half], ga[q] = gain[j], gb[q] = gain[j + half];
        cs[q] = __ldg(rp + j);
        if (BWD) {
          const float da = dy[j], db = dy[j + half];
          wa[q] = da * cs[q].x + db * cs[q].y;
          wb[q] = db * cs[q].x - da * cs[q].y;
        }
      }
      ss += xa[q] * xa[q] + xb[q] * xb[q];
      ux += wa[q] * ga[q] * xa[q] + wb[q] * gb[q] * xb[q];
    }
#pragma unroll
    for (int o = 16; o > 0; o /= 2) {
      ss += __shfl_xor_sync(0xffffffffu, ss, o);
      if (BWD) ux += __shfl_xor_sync(0xffffffffu, ux, o);
    }
    const float r = 1.f / sqrtf(ss / a.d + a.eps), m = r * r * ux / a.d;
    float* out = head_ptr<float>(a.out[t.kind], t.b, t.r) + t.head * a.out[t.kind].head;
#pragma unroll
    for (int q = 0; q < kPairs; ++q) {
      const int j = lane + 32 * q;
      if (j >= half) continue;
      if (BWD) {
        out[j] = r * (wa[q] * ga[q] - xa[q] * m);
        out[j + half] = r * (wb[q] * gb[q] - xb[q] * m);
        const float pa = wa[q] * xa[q] * r, pb = wb[q] * xb[q] * r;
        acc[0][q] += t.kind ? 0.f : pa;
        acc[0][kPairs + q] += t.kind ? 0.f : pb;
        acc[1][q] += t.kind ? pa : 0.f;
        acc[1][kPairs + q] += t.kind ? pb : 0.f;
      } else {
        const float za = xa[q] * r * ga[q], zb = xb[q] * r * gb[q];
        out[j] = za * cs[q].x - zb * cs[q].y;
        out[j + half] = zb * cs[q].x + za * cs[q].y;
      }
    }
  }
  if constexpr (BWD) {
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int q = 0; q < kPairs; ++q) {
        const int j = lane + 32 * q;
        if (j >= half) continue;
        red[warp][k][j] = acc[k][q];
        red[warp][k][j + half] = acc[k][kPairs + q];
      }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * a.d; i += kThreads) {
      const int k = i / a.d, j = i - k * a.d;
      float v = 0.f;
      for (int w = 0; w < kWarps; ++w) v += red[w][k][j];
      a.partial[(size_t)blockIdx.x * 2 * a.d + i] = v;
    }
  }
}

// The gains' gradients from the CTAs' sums, always in the same order: 32
// channels per CTA, 32 slices of the CTAs each.
__global__ void __launch_bounds__(1024)
    qk_rope_gain_kernel(const float* partial, int n, int d, float* dq_gain, float* dk_gain) {
  __shared__ float red[32][33];
  grid_dep_sync();
  const int c = threadIdx.x & 31, s = threadIdx.x >> 5, col = blockIdx.x * 32 + c;
  float v = 0.f;
  if (col < 2 * d)
#pragma unroll 8
    for (int i = s; i < n; i += 32) v += __ldcg(partial + (size_t)i * 2 * d + col);
  red[s][c] = v;
  __syncthreads();
  if (s == 0 && col < 2 * d) {
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) sum += red[i][c];
    float* out = col < d ? dq_gain : dk_gain;
    if (out != nullptr) out[col < d ? col : col - d] = sum;
  }
}

bool vector_view(const HeadView& v, size_t elem) {
  const long long m = 16 / (long long)elem - 1;
  return ((reinterpret_cast<uintptr_t>(v.p) & 15) | ((v.batch | v.row | v.head) & m)) == 0;
}

long long n_items(const QkRopeArgs& a, int per) {
  const int chunks = (a.heads[0] + per - 1) / per + (a.heads[1] + per - 1) / per;
  return (long long)a.batch * a.rows * chunks;
}

template <typename T, int D>
cudaError_t launch_heads(QkRopeArgs a, bool bwd, int max_ctas, int* ctas, cudaStream_t s) {
  a.items = n_items(a, 32 / (D / 8) * (bwd ? 2 : 4));
  const long long need = (a.items + kWarps - 1) / kWarps;
  *ctas = (int)(bwd ? std::min<long long>(need, max_ctas) : need);
  return bwd ? launch_pdl(qk_rope_bwd_kernel<T, D>, dim3(*ctas), dim3(kThreads), 0, s, a)
             : launch_pdl(qk_rope_kernel<T, D>, dim3(*ctas), dim3(kThreads), 0, s, a);
}

}  // namespace

// Four CTAs of 256 threads per SM keep enough loads in flight.
int qk_rope_max_ctas(int num_sms) { return 4 * num_sms; }

int launch_qk_rope(const QkRopeArgs& args, int bf16, bool bwd, int num_sms, float* dq_gain,
                   float* dk_gain, cudaStream_t s) {
  QkRopeArgs a = args;
  const int max_ctas = qk_rope_max_ctas(num_sms);
  int ctas = 0;
  bool wide = true;
  for (int k = 0; k < 2; ++k) {
    if (a.heads[k] == 0) continue;
    const size_t es = bf16 ? 2 : 4;
    wide = wide && vector_view(a.x[k], es) && vector_view(a.out[k], es) &&
           (!bwd || vector_view(a.dy[k], es)) &&
           (reinterpret_cast<uintptr_t>(a.gain[k]) & 15) == 0;
  }
  cudaError_t e;
  if (bf16) {
    e = launch_heads<__nv_bfloat16, 128>(a, bwd, max_ctas, &ctas, s);
  } else if (wide && a.d == 64) {
    e = launch_heads<float, 64>(a, bwd, max_ctas, &ctas, s);
  } else if (wide && a.d == 128) {
    e = launch_heads<float, 128>(a, bwd, max_ctas, &ctas, s);
  } else {
    a.items = n_items(a, 1);
    ctas = (int)std::min<long long>((a.items + kWarps - 1) / kWarps, max_ctas);
    e = bwd ? launch_pdl(qk_rope_any_kernel<true>, dim3(ctas), dim3(kThreads), 0, s, a)
            : launch_pdl(qk_rope_any_kernel<false>, dim3(ctas), dim3(kThreads), 0, s, a);
  }
  if (e != cudaSuccess || !bwd) return (int)e;
  return (int)launch_pdl(qk_rope_gain_kernel, dim3((2 * a.d + 31) / 32), dim3(1024), 0, s,
                         a.partial, ctas, a.d, dq_gain, dk_gain);
}

}  // namespace df
