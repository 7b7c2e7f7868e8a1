// q8_cache.cu -- writing rows into an 8-bit draft KV cache and reading them
// back (formats: q8.cuh).
//
// Both kernels move each byte once and compute a handful of integer
// operations per channel, so HBM bounds them at large sizes and launch
// latency at small ones.  A warp's accesses to the bf16 rows are whole runs of
// 128 bytes and more, those to the codes of 64 and more.
//
// Reading, sixteen lanes take one (row, kv head), eight channels of K and of V
// each.  Writing, which has the larger share of arithmetic, eight lanes do, and
// a lane takes channels 8 l .. 8 l + 7 of either half: the largest magnitudes of
// the two groups that it meets travel as one word through the two shuffles
// by which a group's four lanes agree.  (With sixteen lanes the instructions
// bounded an append of 32768 rows of 8 KV heads: 52 us, 40 us now.)
#include <algorithm>

#include "q8.cuh"

namespace df {
namespace {

constexpr int kThreads = 256;
constexpr int kReadItems = kThreads / 16;  // (row, kv head) pairs that a CTA reads
constexpr int kItems = kThreads / 8;       // and that it has in work when writing
// CTAs of a large append, per SM: three times what runs at a time, so that they
// do not end together, and few enough that not each looks at the ranges for
// itself.  32768 rows of 8 KV heads, appended and read (407 MB): 72 us with 12;
// in one comparison 76 us with 12, 77 us with 8, 83 us with 24, 100 us with 48.
constexpr int kAppendCtas = 12;

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

// A lane's sixteen channels of a row: codes of its chunk in either half, and
// the scale bytes of the two groups.
struct Coded {
  uint2 codes[2];
  uint32_t byte[2];
};

DF_DEV uint32_t max_magnitude(uint4 x) {  // the larger in each half word
  constexpr uint32_t m = 0x7fff7fffu;
  const uint32_t a = __vmaxu2(__vmaxu2(x.x & m, x.y & m), __vmaxu2(x.z & m, x.w & m));
  return max(a & 0xffffu, a >> 16);
}

template <int FMT>
DF_DEV Coded encode16(uint4 x0, uint4 x1) {
  uint32_t amax = max_magnitude(x0) | max_magnitude(x1) << 16;
  amax = __vmaxu2(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
  amax = __vmaxu2(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
  const uint32_t top[2] = {amax & 0xffffu, amax >> 16};
  uint4 x[2] = {x0, x1};
  Coded r;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if (top[i] > kBf16MaxStored) {  // seldom: magnitudes down to 2^126
      x[i].x = q8_clamp2(x[i].x), x[i].y = q8_clamp2(x[i].y);
      x[i].z = q8_clamp2(x[i].z), x[i].w = q8_clamp2(x[i].w);
    }
    r.byte[i] = q8_scale_byte<FMT>(top[i]);
    const float inv = __uint_as_float((254u - max(r.byte[i], 1u)) << 23);  // 2^-e
    r.codes[i] = make_uint2(q8_encode4<FMT>(x[i].x, x[i].y, inv),
                            q8_encode4<FMT>(x[i].z, x[i].w, inv));
    if (r.byte[i] == kQ8NanByte) r.codes[i] = make_uint2(0u, 0u);
  }
  return r;
}

// Codes and scales to their row.  Lanes 0 and 4 of eight know two groups' scale
// bytes each: 0 and 2, 1 and 3.
DF_DEV void put(const Coded& c, uint8_t* codes, uint8_t* scales, int lane8, bool live) {
  uint32_t bytes = c.byte[0] | c.byte[1] << 16;
  bytes |= __shfl_xor_sync(0xffffffffu, bytes, 4) << 8;
  if (!live) return;
  *reinterpret_cast<uint2*>(codes + lane8 * 8) = c.codes[0];
  *reinterpret_cast<uint2*>(codes + 64 + lane8 * 8) = c.codes[1];
  if (lane8 == 0) *reinterpret_cast<uint32_t*>(scales) = bytes;
}

// Smallest and largest scale bytes that eight lanes have met of K and of V in
// one (sequence, kv head); zero groups do not count.
struct Span {
  int* range;  // of the (sequence, kv head), or null
  int4 seen;   // this lane's
  int4 known;  // as the range was when the first row came

  DF_DEV void see(const Coded& k, const Coded& v) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      // (a zero group's 0 becomes the largest number)
      seen.x = (int)min((uint32_t)seen.x, k.byte[i] - 1u);
      seen.y = max(seen.y, (int)k.byte[i]);
      seen.z = (int)min((uint32_t)seen.z, v.byte[i] - 1u);
      seen.w = max(seen.w, (int)v.byte[i]);
    }
  }

  // Into the range.  Only a lane whose span is wider than the range issues
  // atomics, and looks at the range again before: of the many lanes that find
  // a range empty at the same time only the first ones need to.
  DF_DEV void flush(bool writer) {
    seen.x = min(seen.x, __shfl_xor_sync(0xffffffffu, seen.x, 4));
    seen.y = max(seen.y, __shfl_xor_sync(0xffffffffu, seen.y, 4));
    seen.z = min(seen.z, __shfl_xor_sync(0xffffffffu, seen.z, 4));
    seen.w = max(seen.w, __shfl_xor_sync(0xffffffffu, seen.w, 4));
    if (!writer || range == nullptr) return;
    seen.x = min(seen.x + 1, 255);
    seen.z = min(seen.z + 1, 255);
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

// Ranges of the sequences whose rows begin anew.  Not in a CUDA graph: when it
// is replayed the sequence may hold other rows behind the ones it writes, so
// there a range only widens.
__global__ void q8_reset_kernel(const __grid_constant__ Q8Store st,
                                const __grid_constant__ Q8Rows t) {
  grid_dep_sync();
  const int i = blockIdx.x * blockDim.x + threadIdx.x;  // (sequence, head)
  if (i >= t.n * st.n_kv) return;
  const int b = i / st.n_kv;
  if (t.first[b] == 0 && t.off[b + 1] > t.off[b])
    reinterpret_cast<int4*>(st.range)[i] = make_int4(255, 0, 255, 0);
}

// A CTA takes `per` items per eight lanes, kItems apart: with a power of two of
// up to 32 KV heads they stay with one head, goes on by whole rows (without looking
// its place up again until its sequence ends), and its span goes to the range
// once.
template <int FMT>
__global__ void __launch_bounds__(kThreads, 4)
    q8_append_kernel(const __grid_constant__ Q8Store st, const __grid_constant__ Q8Rows t,
                     const __grid_constant__ Q8Source src, int per) {
  const int lane8 = threadIdx.x & 7;
  const long long items = (long long)t.off[t.n] * st.n_kv;
  long long it = (long long)blockIdx.x * per * kItems + (threadIdx.x >> 3);
  const int step = kItems % st.n_kv == 0 ? kItems / st.n_kv : 0;  // rows, 0: not whole
  Span span;
  span.range = nullptr;
  span.seen = make_int4(254, 0, 254, 0);
  span.known = make_int4(255, 0, 255, 0);
  // the item's place: its row, the first one behind its sequence's, its (lane's)
  // source and destination, its range
  long long row = 0, end = 0;
  const uint16_t *k_src = src.k, *v_src = src.v;
  size_t store = 0;
  int* range = st.range;
  auto look_up = [&]() {
    const Item w = item_of(t, st, it);
    const long long base = (long long)w.b * src.seq_stride + (long long)w.h * src.head_stride +
                           lane8 * 8;
    const long long r = src.packed ? w.r : (long long)w.local;
    row = w.r;
    end = t.off[w.b + 1];
    k_src = src.k + base + r * src.k_row_stride;
    v_src = src.v + base + r * src.v_row_stride;
    store = w.store;
    range = st.range + ((size_t)w.b * st.n_kv + w.h) * 4;
  };
  if (it < items) look_up();
  grid_dep_sync();
#pragma unroll 2
  for (int i = 0; i < per; ++i) {
    const bool live = it < items;
    uint4 k0 = make_uint4(0u, 0u, 0u, 0u), k1 = k0, v0 = k0, v1 = k0;
    if (live) {
      k0 = __ldcg(reinterpret_cast<const uint4*>(k_src));
      k1 = __ldcg(reinterpret_cast<const uint4*>(k_src + 64));
      v0 = __ldcg(reinterpret_cast<const uint4*>(v_src));
      v1 = __ldcg(reinterpret_cast<const uint4*>(v_src + 64));
    }
    if (__any_sync(0xffffffffu, live && range != span.range)) {
      span.flush(lane8 == 0);
      span.range = live ? range : nullptr;
      span.seen = make_int4(254, 0, 254, 0);
      span.known = __ldcg(reinterpret_cast<const int4*>(range));
    }
    const Coded ck = encode16<FMT>(k0, k1), cv = encode16<FMT>(v0, v1);
    if (live) span.see(ck, cv);
    put(ck, st.k + store * 128, st.ks + store * 4, lane8, live);
    put(cv, st.v + store * 128, st.vs + store * 4, lane8, live);
    it += kItems;
    row += step;
    if (step != 0 && row < end) {
      k_src += step * src.k_row_stride;
      v_src += step * src.v_row_stride;
      store += step;
    } else if (i + 1 < per && it < items) {
      look_up();
    }
  }
  span.flush(lane8 == 0);
}

template <int FMT>
__global__ void __launch_bounds__(kThreads)
    q8_read_kernel(const __grid_constant__ Q8Store st, const __grid_constant__ Q8Rows t,
                   uint16_t* k_dst, uint16_t* v_dst) {
  const int lane16 = threadIdx.x & 15;
  const long long it = (long long)blockIdx.x * kReadItems + (threadIdx.x >> 4);
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

unsigned blocks_of(const Q8Rows& t, const Q8Store& st, int items) {
  return (unsigned)(((long long)t.off[t.n] * st.n_kv + items - 1) / items);
}

}  // namespace

int launch_q8_append(int fmt, const Q8Store& st, const Q8Rows& t, const Q8Source& src,
                     bool anew, int num_sms, cudaStream_t s) {
  if (t.off[t.n] == 0) return cudaSuccess;
  bool any = false;
  for (int b = 0; b < t.n; ++b) any = any || (t.first[b] == 0 && t.off[b + 1] > t.off[b]);
  if (anew && any) {
    const cudaError_t e = launch_pdl(q8_reset_kernel, dim3((t.n * st.n_kv + 255) / 256),
                                     dim3(256), 0, s, st, t);
    if (e != cudaSuccess) return e;
  }
  const unsigned blocks = blocks_of(t, st, kItems);
  const unsigned per = std::max(1u, blocks / (unsigned)(num_sms * kAppendCtas));
  const dim3 grid((blocks + per - 1) / per), block(kThreads);
  return fmt == Q8_E4M3
             ? launch_pdl(q8_append_kernel<Q8_E4M3>, grid, block, 0, s, st, t, src, (int)per)
             : launch_pdl(q8_append_kernel<Q8_INT8>, grid, block, 0, s, st, t, src, (int)per);
}

int launch_q8_read(int fmt, const Q8Store& st, const Q8Rows& t, void* k_dst, void* v_dst,
                   cudaStream_t s) {
  if (t.off[t.n] == 0) return cudaSuccess;
  const dim3 grid(blocks_of(t, st, kReadItems)), block(kThreads);
  uint16_t* k = static_cast<uint16_t*>(k_dst);
  uint16_t* v = static_cast<uint16_t*>(v_dst);
  return fmt == Q8_E4M3 ? launch_pdl(q8_read_kernel<Q8_E4M3>, grid, block, 0, s, st, t, k, v)
                        : launch_pdl(q8_read_kernel<Q8_INT8>, grid, block, 0, s, st, t, k, v);
}

}  // namespace df
