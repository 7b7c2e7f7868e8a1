// q8_cache.cu -- writing rows into an 8-bit draft KV cache and reading them
// back (formats: q8.cuh).
//
// Both kernels move each byte once and compute a handful of integer
// operations per channel, so HBM bounds them at large sizes and launch
// latency at small ones.  Sixteen lanes take one (row, kv head): a lane
// handles eight channels of K and of V, so that a warp's accesses to the bf16
// rows are whole 256-byte runs and those to the codes whole 128-byte lines.
// When writing, a group's four lanes agree on its largest magnitude with two
// shuffles.
#include <algorithm>

#include "q8.cuh"

namespace df {
namespace {

constexpr int kThreads = 256;
constexpr int kItems = kThreads / 16;  // (row, kv head) pairs that a CTA has in work
// CTAs of a large append, per SM: four times what runs at a time, so that they do
// not end together.  32768 rows of 8 KV heads (407 MB) take 84 us, 4.8 TB/s, with
// 24, 92 us with 6 and 118 us with a CTA per 16 items, each of which then looks
// at the ranges by itself.
constexpr int kAppendCtas = 24;

// The (row, kv head) that item `it` of a call stands for: row `local` of
// sequence b, which is row r of the call's packed rows and row `store` of the
// (sequence, kv head)-major storage.
struct Item {
  int b, h, local;
  long long r;
  size_t store;
};

DF_DEV Item item_of(const Q8Rows& t, const Q8Store& st, long long it) {
  Item w;
  w.r = (uint32_t)it / (uint32_t)st.n_kv;  // (a cache has fewer than 2^31 of them)
  w.h = (int)(it - w.r * st.n_kv);
  int lo = 0, hi = t.n;  // off: prefix sums of the sequences' rows
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (t.off[mid] <= w.r) lo = mid; else hi = mid;
  }
  w.b = lo;
  w.local = (int)(w.r - t.off[lo]);
  w.store = ((size_t)lo * st.n_kv + w.h) * st.cap + t.first[lo] + w.local;
  return w;
}

struct Coded {
  uint2 codes;
  uint32_t byte;
};

template <int FMT>
DF_DEV Coded encode8(uint4 x) {
  constexpr uint32_t m = 0x7fff7fffu;
  const uint32_t a2 = __vmaxu2(__vmaxu2(x.x & m, x.y & m), __vmaxu2(x.z & m, x.w & m));
  uint32_t amax = max(a2 & 0xffffu, a2 >> 16);
  amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
  amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
  Coded r;
  r.byte = q8_scale_byte<FMT>(amax);
  r.codes = make_uint2(0u, 0u);
  if (r.byte != kQ8NanByte) {
    const float inv = __uint_as_float((254u - max(r.byte, 1u)) << 23);  // 2^-e
    r.codes.x = q8_encode2<FMT>(x.x, inv) | (q8_encode2<FMT>(x.y, inv) << 16);
    r.codes.y = q8_encode2<FMT>(x.z, inv) | (q8_encode2<FMT>(x.w, inv) << 16);
  }
  return r;
}

// Smallest and largest scale bytes that a group of 16 lanes has met of K and of
// V in one (sequence, kv head); zero groups do not count.
struct Span {
  int* range;  // of the (sequence, kv head), or null
  int4 seen;   // this lane's
  int4 known;  // as the range was when the first row came

  // Into the range.  Only a lane whose span is wider than the range issues
  // atomics, and looks at the range again before: of the many lanes that find
  // a range empty at the same time only the first ones need to.
  DF_DEV void flush(bool writer) {
#pragma unroll
    for (int d = 4; d <= 8; d <<= 1) {
      seen.x = min(seen.x, __shfl_xor_sync(0xffffffffu, seen.x, d));
      seen.y = max(seen.y, __shfl_xor_sync(0xffffffffu, seen.y, d));
      seen.z = min(seen.z, __shfl_xor_sync(0xffffffffu, seen.z, d));
      seen.w = max(seen.w, __shfl_xor_sync(0xffffffffu, seen.w, d));
    }
    if (!writer || range == nullptr) return;
    auto wider = [&]() {
      return seen.x < known.x || seen.y > known.y || seen.z < known.z || seen.w > known.w;
    };
    if (!wider()) return;
    known = __ldcg(reinterpret_cast<const int4*>(range));
    if (seen.x < known.x) atomicMin(range, seen.x);
    if (seen.y > known.y) atomicMax(range + 1, seen.y);
    if (seen.z < known.z) atomicMin(range + 2, seen.z);
    if (seen.w > known.w) atomicMax(range + 3, seen.w);
  }
};

// Ranges of the sequences whose rows begin anew.
__global__ void q8_reset_kernel(const __grid_constant__ Q8Store st,
                                const __grid_constant__ Q8Rows t) {
  grid_dep_sync();
  const int i = blockIdx.x * blockDim.x + threadIdx.x;  // (sequence, head)
  if (i >= t.n * st.n_kv) return;
  const int b = i / st.n_kv;
  if (t.first[b] == 0 && t.off[b + 1] > t.off[b])
    reinterpret_cast<int4*>(st.range)[i] = make_int4(255, 0, 255, 0);
}

// A CTA takes `per` items per group of lanes, kItems apart: with a power of two
// of up to 16 KV heads a group stays with one head, and its span goes to the
// range once.
template <int FMT>
__global__ void __launch_bounds__(kThreads)
    q8_append_kernel(const __grid_constant__ Q8Store st, const __grid_constant__ Q8Rows t,
                     const __grid_constant__ Q8Source src, int per) {
  const int lane16 = threadIdx.x & 15;
  const long long items = (long long)t.off[t.n] * st.n_kv;
  long long it = (long long)blockIdx.x * per * kItems + (threadIdx.x >> 4);
  Span span;
  span.range = nullptr;
  span.seen = make_int4(255, 0, 255, 0);
  span.known = span.seen;
  grid_dep_sync();
#pragma unroll 2
  for (int i = 0; i < per; ++i, it += kItems) {
    const bool live = it < items;
    const Item w = item_of(t, st, live ? it : 0);
    const long long row = src.packed ? w.r : (long long)w.local;
    const long long base = (long long)w.b * src.seq_stride + (long long)w.h * src.head_stride +
                           lane16 * 8;
    const uint4 k = __ldcg(reinterpret_cast<const uint4*>(src.k + base + row * src.k_row_stride));
    const uint4 v = __ldcg(reinterpret_cast<const uint4*>(src.v + base + row * src.v_row_stride));
    int* range = st.range + ((size_t)w.b * st.n_kv + w.h) * 4;
    if (__any_sync(0xffffffffu, live && range != span.range)) {
      span.flush(lane16 == 0);
      span.range = live ? range : nullptr;
      span.seen = make_int4(255, 0, 255, 0);
      span.known = __ldcg(reinterpret_cast<const int4*>(range));
    }
    const Coded ck = encode8<FMT>(k), cv = encode8<FMT>(v);
    if (!live) continue;
    if (ck.byte != 0u) span.seen.x = min(span.seen.x, (int)ck.byte);
    if (cv.byte != 0u) span.seen.z = min(span.seen.z, (int)cv.byte);
    span.seen.y = max(span.seen.y, (int)ck.byte);
    span.seen.w = max(span.seen.w, (int)cv.byte);
    *reinterpret_cast<uint2*>(st.k + w.store * 128 + lane16 * 8) = ck.codes;
    *reinterpret_cast<uint2*>(st.v + w.store * 128 + lane16 * 8) = cv.codes;
    if ((lane16 & 3) == 0) {
      st.ks[w.store * 4 + (lane16 >> 2)] = (uint8_t)ck.byte;
      st.vs[w.store * 4 + (lane16 >> 2)] = (uint8_t)cv.byte;
    }
  }
  span.flush(lane16 == 0);
}

template <int FMT>
__global__ void __launch_bounds__(kThreads)
    q8_read_kernel(const __grid_constant__ Q8Store st, const __grid_constant__ Q8Rows t,
                   uint16_t* k_dst, uint16_t* v_dst) {
  const int lane16 = threadIdx.x & 15;
  const long long it = (long long)blockIdx.x * kItems + (threadIdx.x >> 4);
  const bool live = it < (long long)t.off[t.n] * st.n_kv;
  const Item w = item_of(t, st, live ? it : 0);
  grid_dep_sync();
  if (!live) return;
  const uint2 ck = *reinterpret_cast<const uint2*>(st.k + w.store * 128 + lane16 * 8);
  const uint2 cv = *reinterpret_cast<const uint2*>(st.v + w.store * 128 + lane16 * 8);
  const uint32_t bk = st.ks[w.store * 4 + (lane16 >> 2)];
  const uint32_t bv = st.vs[w.store * 4 + (lane16 >> 2)];
  const size_t to = (size_t)it * 128 + lane16 * 8;
  *reinterpret_cast<uint4*>(k_dst + to) = bf16_decode8<FMT>(ck.x, ck.y, bf16_scale(bk));
  *reinterpret_cast<uint4*>(v_dst + to) = bf16_decode8<FMT>(cv.x, cv.y, bf16_scale(bv));
}

unsigned blocks_of(const Q8Rows& t, const Q8Store& st) {
  return (unsigned)(((long long)t.off[t.n] * st.n_kv + kItems - 1) / kItems);
}

}  // namespace

int launch_q8_append(int fmt, const Q8Store& st, const Q8Rows& t, const Q8Source& src,
                     int num_sms, cudaStream_t s) {
  if (t.off[t.n] == 0) return cudaSuccess;
  bool anew = false;
  for (int b = 0; b < t.n; ++b) anew = anew || (t.first[b] == 0 && t.off[b + 1] > t.off[b]);
  if (anew) {
    const cudaError_t e = launch_pdl(q8_reset_kernel, dim3((t.n * st.n_kv + 255) / 256),
                                     dim3(256), 0, s, st, t);
    if (e != cudaSuccess) return e;
  }
  const unsigned blocks = blocks_of(t, st);
  const unsigned per = std::max(1u, blocks / (unsigned)(num_sms * kAppendCtas));
  const dim3 grid((blocks + per - 1) / per), block(kThreads);
  return fmt == Q8_E4M3
             ? launch_pdl(q8_append_kernel<Q8_E4M3>, grid, block, 0, s, st, t, src, (int)per)
             : launch_pdl(q8_append_kernel<Q8_INT8>, grid, block, 0, s, st, t, src, (int)per);
}

int launch_q8_read(int fmt, const Q8Store& st, const Q8Rows& t, void* k_dst, void* v_dst,
                   cudaStream_t s) {
  if (t.off[t.n] == 0) return cudaSuccess;
  const dim3 grid(blocks_of(t, st)), block(kThreads);
  uint16_t* k = static_cast<uint16_t*>(k_dst);
  uint16_t* v = static_cast<uint16_t*>(v_dst);
  return fmt == Q8_E4M3 ? launch_pdl(q8_read_kernel<Q8_E4M3>, grid, block, 0, s, st, t, k, v)
                        : launch_pdl(q8_read_kernel<Q8_INT8>, grid, block, 0, s, st, t, k, v);
}

}  // namespace df
