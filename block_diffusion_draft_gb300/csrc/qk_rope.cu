// qk_rope.cu -- per-head RMSNorm and rotation of queries and keys in one pass,
// and its gradient, for training around the packed attention core.
//
// Per head (d channels) of a row at position p, with r = 1 / sqrt(mean(x^2) + eps):
//   z = g * x * r,  y_j = z_j cos - z_{j+d/2} sin,  y_{j+d/2} = z_{j+d/2} cos + z_j sin
// and back, with w the gradient of y turned by -p, u = g * w and s = sum(u * x):
//   dx = r * (u - x * r^2 * s / d),   dg = sum over rows and heads of w * x * r.
// Both sums (x^2 and u * x) go through one reduction.
//
// HBM bounds it: every value is read and written once.  A lane holds channels of
// either half of a head, so a pair's two channels meet in one lane without an
// exchange and every access is a contiguous half head.
#include <algorithm>

#include "internal.h"
#include "ptx.cuh"

namespace df {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;

// Four channels as they lie in memory, and as two pairs of numbers (the fp32
// units take two at a time, and instructions are what this kernel has to save
// next to bytes).
template <typename T>
struct Quad;
template <>
struct Quad<float> {
  float4 r;
  DF_DEV void load(const float* p) { r = *reinterpret_cast<const float4*>(p); }
  DF_DEV float2 pair(int i) const {
    return i == 0 ? make_float2(r.x, r.y) : make_float2(r.z, r.w);
  }
  static DF_DEV void store(float* p, float2 a, float2 b) {
    *reinterpret_cast<float4*>(p) = make_float4(a.x, a.y, b.x, b.y);
  }
};
template <>
struct Quad<__nv_bfloat16> {
  uint2 r;
  DF_DEV void load(const __nv_bfloat16* p) { r = *reinterpret_cast<const uint2*>(p); }
  DF_DEV float2 pair(int i) const {
    const uint32_t w = i == 0 ? r.x : r.y;
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  }
  static DF_DEV void store(__nv_bfloat16* p, float2 a, float2 b) {
    *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(a.x, a.y), pack_bf16x2(b.x, b.y));
  }
};

DF_DEV float2 neg(float2 a) { return make_float2(-a.x, -a.y); }
DF_DEV float2 both(float a) { return make_float2(a, a); }

template <typename T>
DF_DEV T* head_ptr(const HeadView& h, int b, int r) {
  return reinterpret_cast<T*>(h.p) + b * h.batch + r * h.row;
}

// A warp's unit of work: `per` heads from `head` on of row r of sequence b.
struct Item {
  int b, r, head;
};

DF_DEV Item item_at(const QkRopeArgs& a, int kind, int i, int per) {
  const int row = a.chunks[kind].quotient(i);
  Item t;
  t.head = (i - row * a.chunks[kind].d) * per;
  t.b = a.by_rows.quotient(row);
  t.r = row - t.b * a.rows;
  return t;
}

// the position of an item's row, moved into the table
DF_DEV int position(const QkRopeArgs& a, const Item& t) {
  const int pos = __ldg(a.positions + (long long)t.b * a.rows + t.r);
  if (pos >= 0 && pos < a.max_pos) return pos;
  record_error(a.err, 2 /* DFLASH_DEV_POSITION */);
  return pos < 0 ? 0 : a.max_pos - 1;
}

DF_DEV const float2* rope_row(const QkRopeArgs& a, const Item& t) {
  return a.rope + (long long)position(a, t) * (a.d / 2);
}

template <typename T>
DF_DEV void load_gain(const QkRopeArgs& a, int kind, int j, float2 (&v)[2]) {
  Quad<T> q;
  Quad<float> f;
  if (a.gain[kind] != nullptr) q.load(static_cast<const T*>(a.gain[kind]) + j);
  else f.load(a.gain32[kind] + j);
#pragma unroll
  for (int i = 0; i < 2; ++i) v[i] = a.gain[kind] != nullptr ? q.pair(i) : f.pair(i);
}

// cosines and sines of four neighbouring pairs
DF_DEV void load_turn(const float2* p, float2 (&cs)[2], float2 (&sn)[2]) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p));
  const float4 b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  cs[0] = make_float2(a.x, a.z), sn[0] = make_float2(a.y, a.w);
  cs[1] = make_float2(b.x, b.z), sn[1] = make_float2(b.y, b.w);
}

// Groups of heads that a warp of the forward holds at a time: their loads are in
// flight together.  8192 rows of 32 + 8 heads, bf16: 34.5, 32.9, 34.5 us with 2,
// 4, 8 groups (cold; 28 us, 6.0 TB/s, among other calls).
constexpr int kForward = 4;
// Heads of D channels whose tensors allow 4-channel accesses.  The CTAs below
// `a.split` take the queries, the others the keys.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? 5 : 4)
    qk_rope_kernel(const __grid_constant__ QkRopeArgs a) {
  constexpr int L = D / 8, G = 32 / L, U = kForward;
  const int lane = threadIdx.x & 31, l = lane % L, g = lane / L;
  const int kind = (int)blockIdx.x >= a.split;
  const int i = ((int)blockIdx.x - (kind ? a.split : 0)) * kWarps + (threadIdx.x >> 5);
  grid_dep_sync();
  if (i >= a.items[kind]) return;
  const Item t = item_at(a, kind, i, G * U);
  const int n = a.heads[kind];
  const T* src = head_ptr<const T>(a.x[kind], t.b, t.r) + 4 * l;
  Quad<T> lo[U], hi[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int h = min(t.head + u * G + g, n - 1);
    lo[u].load(src + h * a.x[kind].head);
    hi[u].load(src + h * a.x[kind].head + D / 2);
  }
  // gain times cosine and sine, the same for all heads of the row
  float2 ac[2], as[2], bc[2], bs[2];
  load_turn(rope_row(a, t) + 4 * l, ac, as);
  {
    float2 ga[2], gb[2];
    load_gain<T>(a, kind, 4 * l, ga);
    load_gain<T>(a, kind, 4 * l + D / 2, gb);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      bc[j] = mul_f32x2(gb[j], ac[j]);
      bs[j] = neg(mul_f32x2(gb[j], as[j]));
      ac[j] = mul_f32x2(ga[j], ac[j]);
      as[j] = mul_f32x2(ga[j], as[j]);
    }
  }
  T* dst = head_ptr<T>(a.out[kind], t.b, t.r) + 4 * l;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    float2 s2 = make_float2(0.f, 0.f);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      s2 = fma_f32x2(lo[u].pair(j), lo[u].pair(j), s2);
      s2 = fma_f32x2(hi[u].pair(j), hi[u].pair(j), s2);
    }
    float ss = s2.x + s2.y;
#pragma unroll
    for (int o = L / 2; o > 0; o /= 2) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    const int h = t.head + u * G + g;
    if (h >= n) continue;
    const float2 r = both(rsqrtf(ss * (1.f / D) + a.eps));
    float2 ya[2], yb[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const float2 xa = lo[u].pair(j), xb = hi[u].pair(j);
      ya[j] = mul_f32x2(r, fma_f32x2(xa, ac[j], mul_f32x2(xb, bs[j])));
      yb[j] = mul_f32x2(r, fma_f32x2(xb, bc[j], mul_f32x2(xa, as[j])));
    }
    Quad<T>::store(dst + h * a.out[kind].head, ya[0], ya[1]);
    Quad<T>::store(dst + h * a.out[kind].head + D / 2, yb[0], yb[1]);
  }
}

// 16 bytes of a head, as numbers in pairs
template <typename T>
struct Wide;
template <>
struct Wide<float> {
  static constexpr int N = 4;
  uint4 r;
  DF_DEV float2 pair(int i) const {
    return i == 0 ? make_float2(__uint_as_float(r.x), __uint_as_float(r.y))
                  : make_float2(__uint_as_float(r.z), __uint_as_float(r.w));
  }
  DF_DEV void set(const float2 (&v)[2]) {
    r = make_uint4(__float_as_uint(v[0].x), __float_as_uint(v[0].y), __float_as_uint(v[1].x),
                   __float_as_uint(v[1].y));
  }
};
template <>
struct Wide<__nv_bfloat16> {
  static constexpr int N = 8;
  uint4 r;
  DF_DEV float2 pair(int i) const {
    const uint32_t w = i == 0 ? r.x : i == 1 ? r.y : i == 2 ? r.z : r.w;
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  }
  DF_DEV void set(const float2 (&v)[4]) {
    r = make_uint4(pack_bf16x2(v[0].x, v[0].y), pack_bf16x2(v[1].x, v[1].y),
                   pack_bf16x2(v[2].x, v[2].y), pack_bf16x2(v[3].x, v[3].y));
  }
};

DF_DEV void copy16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src)
               : "memory");
}

DF_DEV void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
DF_DEV void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Stages, groups of heads of an item, CTAs per SM: 8192 rows of 32 + 8 heads,
// bf16, cold and with the gains' kernel, took 51.0 us with (2, 4, 3), 51.9 with (2,
// 2, 4), 52.3 with (3, 2, 3), 56 with (3, 1, 5), 80 and more where the CTAs' registers
// or rings leave too few warps; 46 us with (2, 4, 3) among other calls.
constexpr int kStages = 2, kSteps = 4, kCtasPerSm = 3;
constexpr int kBackWarps = 4, kBackThreads = kBackWarps * 32;

// One stage of a warp's ring: its lanes' pieces of x and of the gradient of y
// for kSteps groups of heads, and the row's cosines and sines.
template <int D>
struct Stage {
  uint4 piece[kSteps][4][32];
  float4 turn[D / 4];
};

// where the turns of a lane's pairs lie, so that eight lanes' reads at a time
// fall into different banks (P reads of 16 bytes each)
template <int P>
DF_DEV int turn_at(int q) {
  return q / P * P + (q % P + q / P / (8 / P)) % P;
}

// The gradient.  A lane holds 16 bytes of either half of a head (8 lanes share
// a head of 128 bf16 channels: half the exchanges of the forward's split), a
// warp takes kSteps groups of such heads of one row at a time.  Every lane
// copies what it will need kStages - 1 items ahead into a ring of its warp's,
// which needs no barrier: held in registers, those bytes left too few warps.
template <typename T, int D>
__global__ void __launch_bounds__(kBackThreads, kCtasPerSm)
    qk_rope_bwd_kernel(const __grid_constant__ QkRopeArgs a) {
  constexpr int N = Wide<T>::N, P = N / 2;  // channels and pairs of numbers of a piece
  constexpr int L = D / 2 / N, G = 32 / L;  // lanes of a head, heads of a group
  extern __shared__ uint4 smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, l = lane % L, g = lane / L;
  Stage<D>* ring = reinterpret_cast<Stage<D>*>(smem) + warp * kStages;
  const int kind = (int)blockIdx.x >= a.split;
  const int step = (kind ? (int)gridDim.x - a.split : a.split) * kBackWarps;
  const int n = a.heads[kind], items = a.items[kind];
  const int first = ((int)blockIdx.x - (kind ? a.split : 0)) * kBackWarps + warp;
  const long long x_group = G * a.x[kind].head, dy_group = G * a.dy[kind].head;
  grid_dep_sync();
  // copies of an item into a stage; one group each, also for none
  auto issue = [&](int i, int pos, int stage) {
    if (i < items) {
      const Item t = item_at(a, kind, i, G * kSteps);
      Stage<D>& s = ring[stage];
      const int h = t.head + g;
      const T* x = head_ptr<const T>(a.x[kind], t.b, t.r) + h * a.x[kind].head + N * l;
      const T* dy = head_ptr<const T>(a.dy[kind], t.b, t.r) + h * a.dy[kind].head + N * l;
#pragma unroll
      for (int u = 0; u < kSteps; ++u) {
        if (h + u * G < n) {
          copy16(&s.piece[u][0][lane], x + u * x_group);
          copy16(&s.piece[u][1][lane], x + u * x_group + D / 2);
          copy16(&s.piece[u][2][lane], dy + u * dy_group);
          copy16(&s.piece[u][3][lane], dy + u * dy_group + D / 2);
        }
      }
      if (lane < D / 4)
        copy16(&s.turn[turn_at<P>(lane)], a.rope + (long long)pos * (D / 2) + 2 * lane);
    }
    copy_commit();
  };
  auto pos_of = [&](int i) {
    return i < items ? position(a, item_at(a, kind, i, G * kSteps)) : 0;
  };
  int next = 0;  // the position of the item to copy next
  {
    int pos[kStages];
#pragma unroll
    for (int k = 0; k < kStages; ++k) pos[k] = pos_of(first + k * step);
#pragma unroll
    for (int k = 0; k < kStages - 1; ++k) issue(first + k * step, pos[k], k);
    next = pos[kStages - 1];
  }
  float2 ga[P], gb[P], acc[2 * P] = {};
#pragma unroll
  for (int j = 0; j < P; ++j) {
    const int c = N * l + 2 * j;
    if (a.gain[kind] != nullptr) {
      const T* w = static_cast<const T*>(a.gain[kind]) + c;
      ga[j] = make_float2((float)w[0], (float)w[1]);
      gb[j] = make_float2((float)w[D / 2], (float)w[D / 2 + 1]);
    } else {
      const float* w = a.gain32[kind] + c;
      ga[j] = make_float2(w[0], w[1]);
      gb[j] = make_float2(w[D / 2], w[D / 2 + 1]);
    }
  }
  int stage = 0;
  for (int i = first; i < items; i += step) {
    copy_wait<kStages - 2>();
    __syncwarp();  // (the turns are other lanes' copies; the stage before is read)
    const int ahead = i + (kStages - 1) * step;
    issue(ahead, next, stage == 0 ? kStages - 1 : stage - 1);
    next = pos_of(ahead + step);
    const Stage<D>& s = ring[stage];
    if (++stage == kStages) stage = 0;
    const Item t = item_at(a, kind, i, G * kSteps);
    T* out = head_ptr<T>(a.out[kind], t.b, t.r) + (t.head + g) * a.out[kind].head + N * l;
    float2 cs[P], sn[P];
#pragma unroll
    for (int j = 0; j < P; ++j) {
      const float4 v = s.turn[turn_at<P>(l * P + j)];
      cs[j] = make_float2(v.x, v.z), sn[j] = make_float2(v.y, v.w);
    }
#pragma unroll
    for (int u = 0; u < kSteps; ++u) {
      Wide<T> xa, xb, da, db, ya, yb;
      xa.r = s.piece[u][0][lane];
      xb.r = s.piece[u][1][lane];
      da.r = s.piece[u][2][lane];
      db.r = s.piece[u][3][lane];
      float2 wa[P], wb[P], s2 = make_float2(0.f, 0.f), u2 = s2;
#pragma unroll
      for (int j = 0; j < P; ++j) {
        const float2 va = xa.pair(j), vb = xb.pair(j), ea = da.pair(j), eb = db.pair(j);
        wa[j] = fma_f32x2(ea, cs[j], mul_f32x2(eb, sn[j]));
        wb[j] = fma_f32x2(eb, cs[j], mul_f32x2(neg(ea), sn[j]));
        s2 = fma_f32x2(va, va, s2);
        s2 = fma_f32x2(vb, vb, s2);
        u2 = fma_f32x2(mul_f32x2(ga[j], wa[j]), va, u2);
        u2 = fma_f32x2(mul_f32x2(gb[j], wb[j]), vb, u2);
      }
      float ss = s2.x + s2.y, ux = u2.x + u2.y;
#pragma unroll
      for (int o = L / 2; o > 0; o /= 2) {
        ss += __shfl_xor_sync(0xffffffffu, ss, o);
        ux += __shfl_xor_sync(0xffffffffu, ux, o);
      }
      if (t.head + u * G + g >= n) continue;
      // (r times a sum of products with x, and r times x, are of ordinary size
      // whatever x's is; r * r * r leaves fp32's normal numbers above an rms of 4e12)
      const float r = rsqrtf(ss * (1.f / D) + a.eps);
      const float2 r2 = both(r), m2 = both(r * (-r * ux * (1.f / D)));
#pragma unroll
      for (int j = 0; j < P; ++j) {
        const float2 na = mul_f32x2(r2, xa.pair(j)), nb = mul_f32x2(r2, xb.pair(j));
        acc[j] = fma_f32x2(wa[j], na, acc[j]);
        acc[P + j] = fma_f32x2(wb[j], nb, acc[P + j]);
        wa[j] = fma_f32x2(mul_f32x2(r2, wa[j]), ga[j], mul_f32x2(na, m2));
        wb[j] = fma_f32x2(mul_f32x2(r2, wb[j]), gb[j], mul_f32x2(nb, m2));
      }
      ya.set(wa);
      yb.set(wb);
      T* at = out + u * (G * a.out[kind].head);
      *reinterpret_cast<uint4*>(at) = ya.r;
      *reinterpret_cast<uint4*>(at + D / 2) = yb.r;
    }
  }
  // the CTA's sums: lanes that hold the same channels (L apart), then the
  // warps in order
  copy_wait<0>();
  __syncthreads();
  float* red = reinterpret_cast<float*>(smem);  // [kBackWarps][D]
#pragma unroll
  for (int j = 0; j < 2 * N; ++j) {
    float v = (j & 1) ? acc[j >> 1].y : acc[j >> 1].x;
#pragma unroll
    for (int o = 16; o >= L; o /= 2) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (lane < L) red[warp * D + N * lane + (j % N) + (j / N) * (D / 2)] = v;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < D; i += kBackThreads) {
    float v = 0.f;
    for (int w = 0; w < kBackWarps; ++w) v += red[w * D + i];
    a.partial[(size_t)blockIdx.x * D + i] = v;
  }
}

// Any even head size up to 256 and any alignment, fp32: a warp takes a head,
// a lane the pairs lane, lane + 32, ...  With one head in flight per warp it is far
// from its bytes: 8192 rows of 32 + 8 heads of 80, 121 us, backward 143 (floors 31, 46).
constexpr int kPairs = 4;

template <bool BWD>
__global__ void __launch_bounds__(kThreads)
    qk_rope_any_kernel(const __grid_constant__ QkRopeArgs a) {
  __shared__ float red[BWD ? kWarps : 1][256];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, half = a.d / 2;
  const int kind = (int)blockIdx.x >= a.split;
  const int ctas = kind ? (int)gridDim.x - a.split : a.split;
  grid_dep_sync();
  const float* gain = a.gain[kind] != nullptr ? static_cast<const float*>(a.gain[kind])
                                              : a.gain32[kind];
  float acc[2 * kPairs] = {};
  for (int i = ((int)blockIdx.x - (kind ? a.split : 0)) * kWarps + warp; i < a.items[kind];
       i += ctas * kWarps) {
    const Item t = item_at(a, kind, i, 1);
    const float* x = head_ptr<const float>(a.x[kind], t.b, t.r) + t.head * a.x[kind].head;
    const float* dy =
        BWD ? head_ptr<const float>(a.dy[kind], t.b, t.r) + t.head * a.dy[kind].head : nullptr;
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
    float* out = head_ptr<float>(a.out[kind], t.b, t.r) + t.head * a.out[kind].head;
#pragma unroll
    for (int q = 0; q < kPairs; ++q) {
      const int j = lane + 32 * q;
      if (j >= half) continue;
      if (BWD) {
        out[j] = r * (wa[q] * ga[q] - xa[q] * m);
        out[j + half] = r * (wb[q] * gb[q] - xb[q] * m);
        acc[q] += wa[q] * xa[q] * r;
        acc[kPairs + q] += wb[q] * xb[q] * r;
      } else {
        const float za = xa[q] * r * ga[q], zb = xb[q] * r * gb[q];
        out[j] = za * cs[q].x - zb * cs[q].y;
        out[j + half] = zb * cs[q].x + za * cs[q].y;
      }
    }
  }
  if constexpr (BWD) {
#pragma unroll
    for (int q = 0; q < kPairs; ++q) {
      const int j = lane + 32 * q;
      if (j >= half) continue;
      red[warp][j] = acc[q];
      red[warp][j + half] = acc[kPairs + q];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < a.d; i += kThreads) {
      float v = 0.f;
      for (int w = 0; w < kWarps; ++w) v += red[w][i];
      a.partial[(size_t)blockIdx.x * a.d + i] = v;
    }
  }
}

// The gains' gradients from the CTAs' sums (the first `split` CTAs: the
// queries'), always in the same order: 16 channels per CTA, 64 slices of the
// CTAs each.
constexpr int kGainCols = 16, kGainSlices = 64;

__global__ void __launch_bounds__(kGainCols * kGainSlices)
    qk_rope_gain_kernel(const float* partial, int split, int n, int d, float* dq_gain,
                        float* dk_gain) {
  __shared__ float red[kGainSlices][kGainCols + 1];
  const int c = threadIdx.x % kGainCols, s = threadIdx.x / kGainCols;
  const int col = blockIdx.x * kGainCols + c, kind = blockIdx.y;
  grid_dep_sync();
  float v = 0.f;
  if (col < d)
#pragma unroll 8
    for (int i = (kind ? split : 0) + s; i < (kind ? n : split); i += kGainSlices)
      v += __ldcg(partial + (size_t)i * d + col);
  red[s][c] = v;
  __syncthreads();
  if (s == 0 && col < d) {
    // (eight sums, then those: with one after the other their roundings were
    // most of the fp32 gradients' error)
    float sum[8] = {};
#pragma unroll
    for (int i = 0; i < kGainSlices; ++i) sum[i & 7] += red[i][c];
#pragma unroll
    for (int o = 4; o > 0; o /= 2)
#pragma unroll
      for (int i = 0; i < o; ++i) sum[i] += sum[i + o];
    float* out = kind ? dk_gain : dq_gain;
    if (out != nullptr) out[col] = sum[0];
  }
}

bool vector_view(const HeadView& v, size_t elem) {
  const long long m = 16 / (long long)elem - 1;
  return ((reinterpret_cast<uintptr_t>(v.p) & 15) | ((v.batch | v.row | v.head) & m)) == 0;
}

// Items of `per` heads, and the CTAs of either kind: as many as there is work
// for, in proportion to it where `most` are less.
int share(QkRopeArgs& a, int per, int warps, long long most) {
  long long need[2];
  a.by_rows = Divisor(a.rows);
  for (int k = 0; k < 2; ++k) {
    a.chunks[k] = Divisor((a.heads[k] + per - 1) / per);
    a.items[k] = a.heads[k] > 0 ? a.batch * a.rows * a.chunks[k].d : 0;
    need[k] = (a.items[k] + warps - 1) / warps;
  }
  const long long all = need[0] + need[1];
  if (all > most)
    for (int k = 0; k < 2; ++k)
      if (need[k] > 0) need[k] = std::max(1LL, need[k] * (most - 1) / all);
  a.split = (int)need[0];
  return (int)(need[0] + need[1]);
}

template <typename T, int D>
cudaError_t launch_heads(QkRopeArgs& a, bool bwd, int num_sms, int* ctas, cudaStream_t s) {
  if (!bwd) {
    *ctas = share(a, 32 / (D / 8) * kForward, kWarps, 1LL << 30);
    return launch_pdl(qk_rope_kernel<T, D>, dim3(*ctas), dim3(kThreads), 0, s, a);
  }
  constexpr size_t bytes = sizeof(Stage<D>) * kStages * kBackWarps;
  static std::atomic<unsigned long long> attr_done{0};
  if (!done_on_device(attr_done)) {
    const cudaError_t e = cudaFuncSetAttribute(
        qk_rope_bwd_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e != cudaSuccess) return e;
    mark_device(attr_done);
  }
  *ctas = share(a, 32 / (D / 2 / Wide<T>::N) * kSteps, kBackWarps, qk_rope_max_ctas(num_sms));
  return launch_pdl(qk_rope_bwd_kernel<T, D>, dim3(*ctas), dim3(kBackThreads), bytes, s, a);
}

}  // namespace

int qk_rope_max_ctas(int num_sms) { return kCtasPerSm * num_sms; }

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
    e = launch_heads<__nv_bfloat16, 128>(a, bwd, num_sms, &ctas, s);
  } else if (wide && a.d == 64) {
    e = launch_heads<float, 64>(a, bwd, num_sms, &ctas, s);
  } else if (wide && a.d == 128) {
    e = launch_heads<float, 128>(a, bwd, num_sms, &ctas, s);
  } else {
    ctas = share(a, 1, kWarps, max_ctas);
    e = bwd ? launch_pdl(qk_rope_any_kernel<true>, dim3(ctas), dim3(kThreads), 0, s, a)
            : launch_pdl(qk_rope_any_kernel<false>, dim3(ctas), dim3(kThreads), 0, s, a);
  }
  if (e != cudaSuccess || !bwd) return (int)e;
  return (int)launch_pdl(qk_rope_gain_kernel, dim3((a.d + kGainCols - 1) / kGainCols, 2),
                         dim3(kGainCols * kGainSlices), 0, s,
                         a.partial, a.split, ctas, a.d, dq_gain, dk_gain);
}

}  // namespace df
