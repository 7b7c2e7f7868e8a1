// attn_q8.cu -- attention of the draft's block queries over an 8-bit cache
// (formats: q8.cuh) on tcgen05.
//
//   S = scale * Q K^T over the keys a row sees, O = softmax(S) V
//
// A query tile is up to 64 rows (tokens x query heads of one KV head).  The
// key tiles (128 keys) of every (sequence, query tile, kv head) -- a pair --
// stand in one line; CTA c, one per SM, takes places [c U, (c + 1) U) of it:
// segments of one pair after another.  Every SM gets the same work whatever
// the lengths, and a pair that lies across CTAs is merged afterwards.
//
// The products are taken transposed, keys and channels on the MMA's 128 rows
// and the queries on its 64 columns:
//
//   S^T(g) = K(g) Q^T       A: K in TMEM, key = lane;  B: Q in shared memory
//   O^T   += V(g)^T P(g)^T  A: V, B: P, both in shared memory as [key][...]
//
// so the MMAs do no padded rows, a tile's sums over keys happen in the tensor
// core, and a decoded K row goes from registers to TMEM without touching
// shared memory.
//
// The codes of a tile are 33 KB against the 64 KB of a bf16 tile, so HBM asks
// for a tile every 0.76 us per SM.  A tile takes 1.06 us (2200 cycles; one pair
// per SM, 9 to 257 tiles): the two steps that it spends on its way through the
// decoding warps (16384 codes each of K and V, 270 instructions per warp) follow
// one another without a gap, while the softmax warps wait a third of their time.
// About 6100 warp instructions a tile keep the issue slots 63% busy; shared
// memory moves about 178 KB a tile (copies in, codes out, V in and out, P in and
// out, Q out).  74 us for 4 sequences of 32800 keys (8 KV heads): 3.8 TB/s.  The
// scalar state that does not fit the register split is spilled: 24 and 32 bytes
// a thread in the two instances.
//
// Rows beyond 64 per KV head are other query tiles, for which the keys are
// copied and decoded again: 32 sequences of 512 to 8192 keys take 88 us with 64
// rows, 157 us with 68 to 128, 300 us with 256.  Heads that are decoded to bf16
// take 1.4 to 1.5 times as long (131 us, and 100 us for the 4 long sequences).
//
//   warps 0-15   softmax, thread = key (TMEM lane) and a quarter of the queries
//   warps 16-23  decode: K from the ring into TMEM, V into the tensor core's
//                128-byte-swizzled layout in shared memory, two stages each
//   warp 24      TMEM allocator; issues S^T(g) and O^T
//   warp 25      copies codes (by TMA, swizzled, because a thread reads a row of
//                its own) and scales: a slot of the ring has half of K(g) and
//                half of V(g - 1)
//   warps 26-27  the next segment's queries and tables
//   warps 28-31  those queries to the products' type; the last segment's O out
//
// All of them run on across segments.  Tried and slower, each pair of times
// without the fences of the hand-overs below: eight softmax warps with 32 queries
// a thread (fewer instructions, 78 us when this took 74 us), and eight warps each
// for K and V beside them (78 us); K decoded by the softmax warps (96 us); codes
// read from the ring one step ahead (76 us against 70 us); Q and O handled by the
// softmax warps (a segment cost 13000 cycles instead of 6500); the merge in the
// CTA that comes last (29 us against 21 us for one block over 4128 keys).
//
// Softmax.  m_q, the reference of query q's exponentials, is shared by all
// threads and moves only when a score exceeds it by more than 2^8: each thread
// looks at its own scores, a barrier per tile makes the finding common, and
// then (the first tile of a segment, and seldom later) the tile's largest
// scores are taken over the keys and O is rescaled.
//
// Hand-overs.  Every buffer goes from its writers to its readers and back
// through an mbarrier's phase.  Where one side is the async proxy (copies, the
// tensor core's reads of shared memory) and the other a thread's own loads or
// stores, the thread puts fence.proxy.async between its accesses and its
// arrival: the storing warps for Q, V and P, the decoding warps for a slot of
// the ring that they have read.  What the tensor core has read or a copy has
// written is handed over by the commit or by the transaction bytes.  In TMEM the
// tcgen05 fences stand on both sides.  The fences of V, P and the slots cost 4%
// on 4 sequences of 32800 keys (74 us against 70 us); a fence in the warp that
// issues the MMAs alone is none for what the other warps have stored.
//
// Rows behind the sequence's end decode to zero in V, so nothing stale can
// reach O through a zero probability.  A group that reads NaN is decoded as
// zero too; the queries that see its key remember it and return NaN (in V's
// case in the group's channels), the others are untouched.
#include <algorithm>
#include <atomic>

#include "q8.cuh"

namespace df {
namespace {

constexpr int HD = 128;
constexpr int TK = 128;                   // keys per tile
constexpr int QR = kQ8TileRows;           // query rows per tile (64)
constexpr int kSoftmaxWarps = 16;
constexpr int kDecodeWarps = 8;
constexpr int kWarpMma = kSoftmaxWarps + kDecodeWarps;
constexpr int kWarpCopy = kWarpMma + 1, kWarpQ = kWarpMma + 2;  // (and the next one)
constexpr int kWarpOut = kWarpQ + 2;
constexpr int kThreads = (kWarpOut + 4) * 32;
// registers per thread: 64 at launch, and the same total after the split
constexpr int kSoftmaxRegs = 72, kDecodeRegs = 56, kOtherRegs = 56;
static_assert(4 * kSoftmaxRegs + 2 * kDecodeRegs + 2 * kOtherRegs <= 8 * 64, "register split");
constexpr int HK = TK / 2;                // keys of half a tile
constexpr int RING = 5;                   // slots of half a tile's K and V codes
constexpr uint32_t CODES = HK * HD, SCALES = HK * 4;  // of one of the two
constexpr uint32_t SLOT = 2 * CODES, SLOT_SC = 2 * SCALES, SLOT_META = 64;
constexpr uint32_t VT = TK * HD * 2;      // a decoded V tile
constexpr uint32_t VHALF = VT / 2;        // 64 channels of it
constexpr uint32_t PT = TK * QR * 2;      // a P tile
constexpr uint32_t QT = QR * HD * 2;      // a Q tile
constexpr uint32_t QHALF = QT / 2;
constexpr uint32_t S_COL = 0, O_COL = 2 * QR, K_COL = O_COL + 2 * QR, TMEM_COLS = 512;
constexpr uint32_t OFF_P = 2 * VT, OFF_Q = OFF_P + 2 * PT;
constexpr uint32_t OFF_RING = OFF_Q + 2 * QT, OFF_SC = OFF_RING + RING * SLOT;
constexpr uint32_t OFF_META = OFF_SC + RING * SLOT_SC;
constexpr uint32_t OFF_NAN = OFF_META + RING * SLOT_META, OFF_BAR = OFF_NAN + 8 * TK;
constexpr uint32_t OFF_SEG = OFF_BAR + 512;   // [2] SegmentTable
constexpr uint32_t OFF_ROWS = OFF_SEG + 2 * 1536;  // [4 + 3 * 4 + 8][QR] words
constexpr size_t kSmem = 1024 + OFF_ROWS + 24 * QR * 4;
static_assert(OFF_RING % 1024 == 0 && OFF_BAR % 16 == 0, "alignment");
constexpr float kRescale = 8.f;           // log2 units
constexpr float kLift = 7.f;              // fp16 P = 2^(score - m + 7)
// What a segment costs beside its tiles, in tiles: places of the line that a
// pair takes up without having a tile there.  (A tile takes 2200 cycles, a
// segment 6400 and more where segments are short: 32 sequences of 512 to 8192
// keys take 97, 93, 89, 89 and 90 us with 2, 3, 4, 5 and 6, 4 of 32800 keys 74 us
// with each, 7 of up to 1500 with a window 21 to 24 us, the least with 2.)
constexpr int kPairCost = 4;
constexpr uint32_t kNanK = 16;            // the key reads NaN in K

// ---------------------------------------------------------------- segments
// A CTA's tiles of one pair: what the CTA does of it.
struct Segment {
  int b, h, qt;
  int rows;           // query rows of the tile
  int len;
  int lo, hi;         // keys any row of the query tile sees, within the segment
  int lo_all, hi_all; // keys every row of the query tile sees
  bool same;          // all of them see the same keys
  int t0, t1;         // the tiles that hold [lo, hi) (none: t0 = t1)
  int slot;           // partial slot, or -1 if the segment is the whole pair
};

// Tiles of one of sequence b's pairs: at least one, so that every row is
// written by some CTA.
__host__ __device__ inline int tiles_of(const Q8Plan& p, int b) {
  const int n = (p.len[b] + TK - 1) / TK - p.lo[b] / TK;
  return n > 0 ? n : 1;
}

// the keys that block row t of a sequence of `len` keys sees
DF_DEV int2 seen_by(const Q8AttnArgs& a, int len, int t) {
  const long long at = (long long)len - a.q_len + t;
  long long lo = 0, hi = len;
  if (a.window > 0) {
    lo = max(lo, at - a.window + 1);
    hi = min(hi, at + a.window);
  }
  if (a.causal) hi = min(hi, at + 1);
  return make_int2((int)lo, (int)max(hi, 0LL));
}

// Walks a CTA's segments.  A pair's places in the line are kPairCost empty ones
// and its tiles.
struct Walk {
  int x, end, b;
  bool begun;
  DF_DEV Walk(const Q8AttnArgs& a, const Q8Plan& p) {
    x = (int)blockIdx.x * p.share;
    end = min(x + p.share, p.first[a.batch]);
    b = p.start[blockIdx.x];
    begun = false;
  }
  DF_DEV bool next(const Q8AttnArgs& a, const Q8Plan& p, Segment& w) {
    int n, pair, i0, i1;
    do {
      if (x >= end) return false;
      while (x >= p.first[b + 1]) ++b;
      n = tiles_of(p, b);
      const int rel = x - p.first[b];
      pair = rel / (n + kPairCost);
      const int from = rel - pair * (n + kPairCost), to = min(n + kPairCost, from + end - x);
      x += to - from;
      i0 = max(0, from - kPairCost);
      i1 = max(0, to - kPairCost);
    } while (i0 == i1);
    w.b = b;
    w.qt = pair / a.st.n_kv;
    w.h = pair - w.qt * a.st.n_kv;
    w.slot = i0 == 0 && i1 == n ? -1 : 2 * (int)blockIdx.x + (begun ? 1 : 0);
    begun = true;
    const int r0 = w.qt * QR;
    w.rows = min(QR, a.q_len * a.groups - r0);
    w.len = p.len[b];
    // both ends of what a row sees grow along the rows
    const int2 s0 = seen_by(a, w.len, r0 / a.groups);
    const int2 s1 = seen_by(a, w.len, (r0 + w.rows - 1) / a.groups);
    const int t = p.lo[b] / TK;
    w.lo = max(s0.x, (t + i0) * TK);
    w.hi = min(s1.y, (t + i1) * TK);
    w.lo_all = s1.x;
    w.hi_all = s0.y;
    w.same = s0.x == s1.x && s0.y == s1.y;
    w.t0 = w.lo / TK;
    w.t1 = w.hi > w.lo ? (w.hi + TK - 1) / TK : w.t0;
    return true;
  }
};

// output (and log-sum-exp) row of row r of (b, h)'s tokens x heads
DF_DEV int out_row(const Q8AttnArgs& a, int b, int h, int r) {
  const int t = r / a.groups, g = r - t * a.groups;
  return (b * a.q_len + t) * (a.st.n_kv * a.groups) + h * a.groups + g;
}

DF_DEV float2 fma_f32x2(float2 a, float2 b, float2 c) {
  unsigned long long pa, pb, pc, pd;
  asm("mov.b64 %0, {%1, %2};" : "=l"(pa) : "f"(a.x), "f"(a.y));
  asm("mov.b64 %0, {%1, %2};" : "=l"(pb) : "f"(b.x), "f"(b.y));
  asm("mov.b64 %0, {%1, %2};" : "=l"(pc) : "f"(c.x), "f"(c.y));
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(pd) : "l"(pa), "l"(pb), "l"(pc));
  float2 d;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(d.x), "=f"(d.y) : "l"(pd));
  return d;
}

DF_DEV uint32_t pack_f16x2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

DF_DEV float nan_f() { return __uint_as_float(0x7fffffffu); }

// How the codes of a (sequence, kv head) are decoded (q8.cuh): to fp16 in
// units of 2^(k0 - 127), 2^(v0 - 127), or to bf16.
struct Mode {
  bool half;
  int k0, v0;
};

DF_DEV Mode mode_of(const Q8Store& st, int b, int h) {
  const int4 r = __ldcg(reinterpret_cast<const int4*>(st.range) + (size_t)b * st.n_kv + h);
  Mode m;
  m.half = (r.y == 0 || r.y - r.x <= kHalfSpan) && (r.w == 0 || r.w - r.z <= kHalfSpan) &&
           max(r.y, r.w) < (int)kQ8NanByte;
  m.k0 = max(r.y - kHalfTop, kHalfMinUnit);
  m.v0 = max(r.w - kHalfTop, kHalfMinUnit);
  return m;
}

// What a slot of the ring holds: step u's slots hold K of tile u and V of
// tile u - 1 (the tiles of all the CTA's segments are numbered through).
constexpr int kHasK = 1, kHasV = 2, kHalfK = 4, kHalfV = 8, kEdgeV = 16, kEnd = 32;
struct SlotMeta {
  int flags, k0, v0, unused;
  int k_key, k_lo, k_hi, unused2;  // first key, and the live ones
  int v_key, v_lo, v_hi, unused3;
};
static_assert(sizeof(SlotMeta) <= SLOT_META, "slot meta");

// A segment as the other warps need it, written, with a double-buffered Q tile,
// while the one before is worked on.
struct SegmentTable {
  int n, t0, rows, slot;       // n: tiles, -1 behind the last segment
  int lo, hi, lo_all, hi_all;
  int same, half, k0, v0;
  int uneven;                  // the rows' scores have scales sc, not `scale`, or may be 2^20
  float scale;                 // of a score, in log2 units
  int top[4], low[4];          // exponents of the rows, per warp
  int2 seen[QR];               // keys a row sees
  int dst[QR], nan[QR];        // output row; NaN marks
  float sc[QR];
};
static_assert(sizeof(SegmentTable) <= 1536 && sizeof(SegmentTable) % 8 == 0, "segment table");

// Shared memory of a CTA.  Barriers come in pairs by the parity of g, the
// CTA's running tile number over all its segments, or of the segment.
struct Shared {
  uint8_t *v, *p, *q;      // [2] decoded V tiles, P tiles, Q tiles
  uint8_t *ring, *ring_sc; // [RING] K and V codes, scales
  uint8_t* meta;           // [RING]
  uint8_t* nan_bits;       // [K, V][4][TK]
  uint8_t* seg;            // [2] SegmentTable
  float *m, *off, *alpha;  // [2 by segment][QR], [QR], [QR]
  float *top, *sum;        // [4][QR] per quarter of the keys; [2 by segment][QR][4]
  int2* out_rows;          // [4 by warp][QR]
  int* open;               // [2] rows without a key so far
  volatile int* nan_tile;  // [4] the last tile of this number (mod 4) with a NaN
  volatile int* abort;
  uint64_t *ring_full, *ring_empty;  // [RING]
  uint64_t *k_full, *v_full;         // by tile, as the next three
  uint64_t *s_full;        // S(g) and PV(g - 2) complete: K(g)'s stage, and V(g)'s and P(g)'s,
                           // are free
  uint64_t *p_full;        // P(g) written, and S(g) read
  uint64_t *o_done;        // PV(g) complete
  uint64_t *o_last;        // by segment, of those with tiles: its last PV complete
  uint64_t *l_full;        // by segment: the softmax is through, its m and sums written
  uint64_t *q_raw;         // by segment: its query rows and what is known of them
  uint64_t *q_full;        // by segment: its table and Q tile are complete
  uint64_t *o_free;        // by segment: its rows are written
  DF_DEV SegmentTable& table(int i) const {
    return *reinterpret_cast<SegmentTable*>(seg + (i & 1) * 1536);
  }
};

// The library's bounded wait, written small: five kinds of warps run their
// loops side by side, and those loops have to stay in the instruction caches
// together.
DF_DEV bool wait(uint64_t* bar, uint32_t parity, const Shared& sm, int* err) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = global_ns();
  while (!mbar_try_wait(bar, parity)) {
    if (*sm.abort) return false;
    if (global_ns() - t0 > kWaitLimitNs) {
      *sm.abort = 1;
      record_error(err, 1 /* DFLASH_DEV_WAIT_TIMEOUT */);
      return false;
    }
  }
  return true;
}

// The same for warps that wait for long, without taking issue slots.
DF_DEV bool patient_wait(uint64_t* bar, uint32_t parity, const Shared& sm, int* err) {
  const uint64_t t0 = global_ns();
  while (!__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) {
    if (__any_sync(0xffffffffu, *sm.abort != 0)) return false;
    if (__any_sync(0xffffffffu, global_ns() - t0 > kWaitLimitNs)) {
      *sm.abort = 1;
      record_error(err, 1 /* DFLASH_DEV_WAIT_TIMEOUT */);
      return false;
    }
    __nanosleep(100);
  }
  return true;
}

DF_DEV bool warp_wait(uint64_t* bar, uint32_t parity, const Shared& sm, int* err) {
  return __all_sync(0xffffffffu, wait(bar, parity, sm, err));
}

// A value that is the same in all lanes, for the compiler to know it: it then
// keeps it in uniform registers, branches without reconvergence and issues
// what takes uniform operands (tensor memory accesses, copies, MMAs) directly
// (74 us against 83 us on 4 sequences of 32800 keys).
template <typename T>
DF_DEV T uniform(T x) {
  return __shfl_sync(0xffffffffu, x, 0);
}

// Meets the n threads of barrier `id`: whether `x` holds for all of them.  (If
// a wait runs out in one warp and not in another, both still do the same.)
DF_DEV bool all_of(int id, int n, bool x) {
  uint32_t y;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "bar.red.and.pred q, %2, %3, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(y)
      : "r"((uint32_t)x), "r"(id), "r"(n)
      : "memory");
  return y != 0u;
}

// One arrival per warp, after what its threads did in TMEM.
DF_DEV void warp_arrive(uint64_t* bar, int lane) {
  tc_fence_before();
  __syncwarp();
  if (lane == 0) mbar_arrive(bar);
}

template <int N>
DF_DEV void reg_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

template <int N>
DF_DEV void reg_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// ---------------------------------------------------------------- decode
// A row's scale bytes for one tile: zero where the segment has no such key,
// and NaN groups taken out; their bits (kNanK, or V's groups) go to `bits`.
DF_DEV uint32_t live_scales(uint32_t s, bool is_k, bool live, uint32_t& bits) {
  if (!live) return 0u;
  const uint32_t nan = __vcmpeq4(s, 0xffffffffu);
  if (nan != 0u)
    bits |= is_k ? kNanK
                 : (nan & 1u) | ((nan >> 7) & 2u) | ((nan >> 14) & 4u) | ((nan >> 21) & 8u);
  return s & ~nan;
}

// K: this thread's half (64 channels, `ch`) of its row as 32 columns of its
// TMEM lane, 16 at a time.
template <int FMT, bool HALF16>
DF_DEV void decode_k(const uint4 (&c)[4], uint32_t bytes, int ch, int unit0, uint32_t col) {
  HalfScales hs{};
  if (HALF16) hs = half_scales(bytes, unit0);
#pragma unroll
  for (int o = 0; o < 2; ++o) {
    const int g = ch * 2 + o;
    uint32_t v[16];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint4 x = c[2 * o + i];
      uint4 a, b;
      if (HALF16) {
        half_decode16<FMT>(x, hs, half_select(g), a, b);
      } else {
        const float s = bf16_scale((bytes >> (g * 8)) & 0xffu);
        a = bf16_decode8<FMT>(x.x, x.y, s);
        b = bf16_decode8<FMT>(x.z, x.w, s);
      }
      v[8 * i] = a.x, v[8 * i + 1] = a.y, v[8 * i + 2] = a.z, v[8 * i + 3] = a.w;
      v[8 * i + 4] = b.x, v[8 * i + 5] = b.y, v[8 * i + 6] = b.z, v[8 * i + 7] = b.w;
    }
    tmem_st16_nowait(col + o * 16, v);
  }
  tmem_st_wait();
}

// V: the same half of a row, to `at`, its first chunk's place in a tile: chunk c
// of a half lies at c ^ (row & 7) of the row's 128 bytes.  Eight lanes write
// eight rows' chunks to different banks.
template <int FMT, bool HALF16>
DF_DEV void decode_v(const uint4 (&c)[4], uint32_t bytes, int ch, int unit0, uint8_t* tile,
                     uint32_t at) {
  HalfScales hs{};
  if (HALF16) hs = half_scales(bytes, unit0);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int g = ch * 2 + (i >> 1);
    uint4 a, b;
    if (HALF16) {
      half_decode16<FMT>(c[i], hs, half_select(g), a, b);
    } else {
      const float s = bf16_scale((bytes >> (g * 8)) & 0xffu);
      a = bf16_decode8<FMT>(c[i].x, c[i].y, s);
      b = bf16_decode8<FMT>(c[i].z, c[i].w, s);
    }
    *reinterpret_cast<uint4*>(tile + (at ^ (uint32_t)(2 * i * 16))) = a;
    *reinterpret_cast<uint4*>(tile + (at ^ (uint32_t)((2 * i + 1) * 16))) = b;
  }
}

// Step u: K(u), then V(u - 1).  A slot is free as soon as its codes are in
// registers: it is released behind K's, because the fence before that waits for
// the loads of V's (released before K's: 76 us against 74 us on 4 sequences of
// 32800 keys).  One wait besides the slot's is enough: s_full(u - 1) frees
// V(u - 1)'s stage, and K(u + 1)'s for the next step.
template <int FMT>
DF_DEV void decode_all(const Shared& sm, int* err, uint32_t tmem, int warp, int lane) {
  const int quarter = warp & 3, half = quarter >> 1, ch = warp >> 2;
  const int rr = (quarter & 1) * 32 + lane;  // the thread's row within the slot
  const uint32_t v_at = ch * VHALF + (quarter * 32 + lane) * 128 + ((rr & 7) << 4);
  const uint32_t k_col = tmem + ((uint32_t)(quarter * 32) << 16) + K_COL + ch * 32;
  int slot = half;
  uint32_t phase = 0;
  for (int u = 0;; ++u) {
    if (!warp_wait(&sm.ring_full[slot], phase, sm, err)) return;
    const SlotMeta* meta = reinterpret_cast<const SlotMeta*>(sm.meta + slot * SLOT_META);
    const uint8_t* codes = sm.ring + slot * SLOT;
    const uint8_t* scales = sm.ring_sc + slot * SLOT_SC;
    const int4 head = *reinterpret_cast<const int4*>(meta);
    const int flags = uniform(head.x);
    int4 k_live, v_live;
    uint4 kc[4], vc[4];
    uint32_t kb = *reinterpret_cast<const uint32_t*>(scales + rr * 4);
    uint32_t vb = *reinterpret_cast<const uint32_t*>(scales + SCALES + rr * 4);
#pragma unroll
    for (int i = 0; i < 4; ++i)  // (16-byte chunk c of a row lies at c ^ (rr & 7))
      kc[i] = *reinterpret_cast<const uint4*>(codes + rr * HD + (((ch * 4 + i) ^ (rr & 7)) << 4));
#pragma unroll
    for (int i = 0; i < 4; ++i)
      vc[i] = *reinterpret_cast<const uint4*>(codes + CODES + rr * HD +
                                              (((ch * 4 + i) ^ (rr & 7)) << 4));
    v_live = *(reinterpret_cast<const int4*>(meta) + 2);
    if ((flags & (kHasK | kHalfK)) == kHasK) k_live = *(reinterpret_cast<const int4*>(meta) + 1);
    if (flags & kHasK) {
      const uint32_t col = k_col + (u & 1) * 64;
      tc_fence_after();
      if (flags & kHalfK) {
        decode_k<FMT, true>(kc, kb, ch, head.y, col);
      } else {
        const int key = k_live.x + rr;
        uint32_t bits = 0u;
        kb = live_scales(kb, true, key >= k_live.y && key < k_live.z, bits);
        // (the softmax of tile u - 4, which read these marks, is behind PV(u - 4))
        if (ch == 0) sm.nan_bits[(u & 3) * TK + quarter * 32 + lane] = (uint8_t)bits;
        if (bits != 0u) sm.nan_tile[u & 3] = u;
        decode_k<FMT, false>(kc, kb, ch, 0, col);
      }
      warp_arrive(&sm.k_full[u & 1], lane);
    }
    // the slot's codes are in registers, K's have been used
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.ring_empty[slot]);
    if (flags & kHasV) {
      const int g = u - 1;
      if (!warp_wait(&sm.s_full[g & 1], (g >> 1) & 1, sm, err)) return;
      uint8_t* tile = sm.v + (g & 1) * VT;
      const int key = v_live.x + rr;
      const bool live = key >= v_live.y && key < v_live.z;
      if (flags & kHalfV) {
        if ((flags & kEdgeV) && !live) {  // codes and scales of zero
          constexpr uint32_t zero = FMT == Q8_INT8 ? 0x80808080u : 0u;
          for (int i = 0; i < 4; ++i) vc[i] = make_uint4(zero, zero, zero, zero);
          vb = 0u;
        }
        decode_v<FMT, true>(vc, vb, ch, head.z, tile, v_at);
      } else {
        uint32_t bits = 0u;
        vb = live_scales(vb, false, live, bits);
        if (ch == 0) sm.nan_bits[(4 + (g & 3)) * TK + quarter * 32 + lane] = (uint8_t)bits;
        if (bits != 0u) sm.nan_tile[g & 3] = g;
        decode_v<FMT, false>(vc, vb, ch, 0, tile, v_at);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.v_full[g & 1]);
    }
    if (flags & kEnd) return;
    slot += 2;
    if (slot >= RING) {
      slot -= RING;
      phase ^= 1u;
    }
  }
}

// ---------------------------------------------------------------- copies
DF_DEV bool elect_one() {
  uint32_t is;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(is));
  return is != 0u;
}

DF_DEV void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar,
                      uint64_t policy) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], "
      "[%1], %2, [%3], %4;" ::"r"(smem_u32(dst)),
      "l"(src), "r"(bytes), "r"(smem_u32(bar)), "l"(policy)
      : "memory");
}

// The ring (one elected lane copies).  On an abort the copies in flight are
// still waited for, with a limit: no CTA may leave before they have landed.
DF_DEV void copy_codes(const Q8AttnArgs& a, const Q8Plan& p, const CUtensorMap* tm_k,
                       const CUtensorMap* tm_v, const Shared& sm) {
  const uint64_t once = policy_evict_first();
  Walk walk(a, p);
  Segment w{};
  Mode mode{};
  SlotMeta m{};
  int t = -1, k_row = 0, v_row = 0, slot = 0, n = 0;
  uint32_t phase = 1;
  bool alive = true;
  while (alive && !(m.flags & kEnd)) {
    // the last step's K is this step's V
    m.flags = (m.flags & kHasK) ? kHasV | ((m.flags & kHalfK) ? kHalfV : 0) : 0;
    m.v0 = mode.v0;
    m.v_key = m.k_key, m.v_lo = m.k_lo, m.v_hi = m.k_hi;
    v_row = k_row;
    ++t;
    bool more = true;
    while (more && t >= w.t1) {
      more = walk.next(a, p, w);
      t = w.t0;
      if (more && w.t0 < w.t1) mode = mode_of(a.st, w.b, w.h);
    }
    if (more) {
      m.flags |= kHasK | (mode.half ? kHalfK : 0);
      m.k0 = mode.k0;
      m.k_key = t * TK, m.k_lo = w.lo, m.k_hi = w.hi;
      k_row = (w.b * a.st.n_kv + w.h) * a.st.cap + t * TK;
    } else {
      m.flags |= kEnd;
    }
#pragma unroll 1
    for (int half = 0; half < 2; ++half) {
      alive = warp_wait(&sm.ring_empty[slot], phase, sm, a.err);
      if (!alive) break;
      if (elect_one()) {
        uint64_t* bar = &sm.ring_full[slot];
        uint8_t* codes = sm.ring + slot * SLOT;
        uint8_t* scales = sm.ring_sc + slot * SLOT_SC;
        SlotMeta x = m;
        x.k_key += half * HK;
        x.v_key += half * HK;
        if (x.v_key < x.v_lo || x.v_key + HK > x.v_hi) x.flags |= kEdgeV;
        int4* meta = reinterpret_cast<int4*>(sm.meta + slot * SLOT_META);
        meta[0] = make_int4(x.flags, x.k0, x.v0, 0);
        meta[1] = make_int4(x.k_key, x.k_lo, x.k_hi, 0);
        meta[2] = make_int4(x.v_key, x.v_lo, x.v_hi, 0);
        mbar_arrive_expect_tx(bar, ((m.flags & kHasK ? 1 : 0) + (m.flags & kHasV ? 1 : 0)) *
                                       (CODES + SCALES));
        if (m.flags & kHasK) {
          const int row = k_row + half * HK;
          tma_load_2d(codes, tm_k, bar, 0, row, once);
          bulk_load(scales, a.st.ks + (size_t)row * 4, SCALES, bar, once);
        }
        if (m.flags & kHasV) {
          const int row = v_row + half * HK;
          tma_load_2d(codes + CODES, tm_v, bar, 0, row, once);
          bulk_load(scales + SCALES, a.st.vs + (size_t)row * 4, SCALES, bar, once);
        }
      }
      __syncwarp();
      ++n;
      if (++slot == RING) {
        slot = 0;
        phase ^= 1u;
      }
    }
  }
  const uint64_t t0 = global_ns();
  for (int i = max(0, n - RING); i < n; ++i)
    while (!mbar_try_wait(&sm.ring_full[i % RING], (i / RING) & 1) &&
           global_ns() - t0 < kWaitLimitNs) {
    }
  __syncwarp();
}

// ---------------------------------------------------------------- queries
// 16-byte chunk c of a row of segment seg's Q tile: 128-byte rows of one half of
// the channels each, chunks at c ^ (row & 7)
DF_DEV uint4* q_chunk(const Shared& sm, int seg, int row, int c) {
  return reinterpret_cast<uint4*>(sm.q + (seg & 1) * QT + (c >> 3) * QHALF + row * 128 +
                                  (((c & 7) ^ (row & 7)) << 4));
}

// Two warps fetch the segments' query rows, a row per lane, and write their
// tables.
DF_DEV void fetch_queries(const Q8AttnArgs& a, const Q8Plan& p, const Shared& sm, int warp,
                          int lane) {
  Walk walk(a, p);
  for (int seg = 0;; ++seg) {
    Segment w;
    const bool more = walk.next(a, p, w);
    SegmentTable& tab = sm.table(seg);
    // segment seg - 2 is finished with
    if (seg >= 2 && !patient_wait(&sm.o_free[seg & 1], ((seg >> 1) & 1) ^ 1, sm, a.err)) return;
    if (!more) {
      if (warp == 0 && lane == 0) tab.n = -1;
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.q_raw[seg & 1]);
      return;
    }
    const int row = warp * 32 + lane;
    const bool real = row < w.rows;
    const int x = w.qt * QR + (real ? row : 0), t = x / a.groups, g = x - t * a.groups;
    const uint16_t* q = a.q + (long long)w.b * a.q_seq + (long long)w.h * a.q_head +
                        (long long)g * a.q_group + (long long)t * a.q_tok;
    if (real) {
#pragma unroll
      for (int c = 0; c < 16; ++c)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                         smem_u32(q_chunk(sm, seg, row, c))),
                     "l"(q + c * 8)
                     : "memory");
    } else {
#pragma unroll
      for (int c = 0; c < 16; ++c) *q_chunk(sm, seg, row, c) = make_uint4(0u, 0u, 0u, 0u);
    }
    int2 seen = make_int2(0, 0);
    if (real) {
      seen = seen_by(a, w.len, t);
      seen.x = max(seen.x, w.lo);
      seen.y = min(seen.y, w.hi);
    }
    tab.seen[row] = seen;
    tab.dst[row] = (w.b * a.q_len + t) * (a.st.n_kv * a.groups) + w.h * a.groups + g;
    if (warp == 0 && lane == 0) {
      const Mode mode = mode_of(a.st, w.b, w.h);
      tab.n = w.t1 - w.t0;
      tab.t0 = w.t0;
      tab.rows = w.rows;
      tab.slot = w.slot;
      tab.lo = w.lo;
      tab.hi = w.hi;
      tab.lo_all = w.lo_all;
      tab.hi_all = w.hi_all;
      tab.same = w.same ? 1 : 0;
      tab.half = mode.half ? 1 : 0;
      tab.k0 = mode.k0;
      tab.v0 = mode.v0;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.q_raw[seg & 1]);
  }
}

// The Q tile of a fetched segment in the products' type, by four warps, half a
// row per lane: bf16 rows as they are, or fp16 rows scaled by the power of two
// that brings the tile's largest magnitude to [2^13, 2^14); a row whose own
// largest is below 2^-10 of that gets its own power of two.  Either is exact
// but for what is below 2^-17 of the row's largest, and that is off by 2^-28 of
// it at most.  A row that is not finite becomes zero and is marked.
DF_DEV void convert_queries(const Q8AttnArgs& a, const Shared& sm, int seg, int warp, int lane) {
  SegmentTable& tab = sm.table(seg);
  const int row = warp * 16 + (lane >> 1), c0 = (lane & 1) * 8;
  const bool half = uniform(tab.half) != 0;
  uint32_t top2 = 0u;
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    const uint4 y = *q_chunk(sm, seg, row, c0 + c);
    constexpr uint32_t m = 0x7fff7fffu;
    top2 = __vmaxu2(top2, __vmaxu2(__vmaxu2(y.x & m, y.y & m), __vmaxu2(y.z & m, y.w & m)));
  }
  uint32_t most = max(top2 & 0xffffu, top2 >> 16);
  most = max(most, __shfl_xor_sync(0xffffffffu, most, 1));
  const bool finite = most < 0x7f80u;
  // exponent field of the row's largest magnitude (0: a zero row)
  int field = most == 0u || !finite ? 0 : max((int)(most >> 7), 14);
  int top = __reduce_max_sync(0xffffffffu, field);
  int low = __reduce_min_sync(0xffffffffu, field == 0 ? 255 : field);
  if (lane == 0) {
    tab.top[warp] = top;
    tab.low[warp] = low;
  }
  named_bar_sync(2, 128);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    top = max(top, tab.top[i]);
    low = min(low, tab.low[i]);
  }
  top = max(top, 14);
  // a.scale * 2^(f - 140 + k0 - 127), kept finite and above zero
  const float k_unit = __uint_as_float((uint32_t)tab.k0 << 23);
  auto scale_of = [&](int f) {
    if (!half) return a.scale;
    const float y = a.scale * __uint_as_float((uint32_t)(f - 13) << 23) * k_unit;
    return fminf(fmaxf(y, 1.1754944e-38f), 3.4028235e38f);
  };
  if (field == 0 || field >= top - 10) field = top;
  if (c0 == 0) {
    tab.sc[row] = scale_of(field);
    tab.nan[row] = finite ? 0 : (int)kNanK;
  }
  if (warp == 0 && lane == 0) {
    // Even rows have one scale and scores below 2^20: fp16, |S| < 2^35, so
    // that scale <= 2^-15; bf16, |S| < 2^(top - 126) 2^(9 + k0 + 5 - 127) 2^7 (the
    // largest scale byte of K is k0 + 5 at most, or 255 with a NaN), scale <= 1.
    tab.uneven = half ? low < top - 10 || scale_of(top) > 3.0517578125e-05f
                      : top + tab.k0 > 252;
    tab.scale = scale_of(top);
  }
  if (half || !finite) {
    const float up = __uint_as_float((uint32_t)(267 - field) << 23);
#pragma unroll 4
    for (int c = 0; c < 8; ++c) {
      uint4* at = q_chunk(sm, seg, row, c0 + c);
      const uint4 v = *at;
      uint32_t y[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int k = 0; k < 4; ++k)
        y[k] = pack_f16x2(__uint_as_float(y[k] << 16) * up,
                          __uint_as_float(y[k] & 0xffff0000u) * up);
      *at = finite ? make_uint4(y[0], y[1], y[2], y[3]) : make_uint4(0u, 0u, 0u, 0u);
    }
  }
  fence_proxy_async_smem();
}

// ---------------------------------------------------------------- products
// One elected lane each: with elect.sync the compiler knows that a single
// thread issues, and keeps the descriptors in uniform registers (behind a test
// of the lane number the eight MMAs of a product took 800-950 cycles to issue).
// Q, V and P reach the tensor core through the async proxy: every thread that
// stores a part of them fences its own stores before it arrives.
// One warp issues both products, and PV(g - 2) before S(g): the tensor core
// takes them in that order, so one barrier tells of both.  (The O buffer of a
// segment is free when its table is there.)
DF_DEV void issue_all(const Shared& sm, int* err, uint32_t tmem) {
  const uint64_t desc_q = sdesc_sw128(smem_u32(sm.q), 16, 1024);
  const uint64_t desc_v = sdesc_sw128(smem_u32(sm.v), VHALF, 1024);
  const uint64_t desc_p = sdesc_sw128(smem_u32(sm.p), 16, 1024);
  // tiles whose S is issued and PV not: the last `pending` before g, with the
  // segment, whether it begins with the tile, and the instruction descriptor
  struct Tile {
    int seg, first, last;
    uint32_t idesc;
  } older{}, newer{};
  int pending = 0, g = 0;
  auto issue_pv = [&]() {
    const Tile x = pending == 2 ? older : newer;
    const int st = (g - pending) & 1;
    const uint32_t ph = ((g - pending) >> 1) & 1;
    --pending;
    if (!warp_wait(&sm.v_full[st], ph, sm, err) || !warp_wait(&sm.p_full[st], ph, sm, err))
      return false;
    tc_fence_after();
    const uint64_t dv = desc_v + (uint32_t)(st * (VT >> 4));
    const uint64_t dp = desc_p + (uint32_t)(st * (PT >> 4));
    if (elect_one()) {
#pragma unroll
      for (int kk = 0; kk < TK / 16; ++kk)
        tc_mma_bf16(tmem + O_COL + (x.seg & 1) * QR, dv + ((kk * 16 * 128) >> 4), dp + ((kk * 16 * 128) >> 4),
                    x.idesc, (!x.first || kk > 0) ? 1u : 0u);
      tc_commit(&sm.o_done[st]);
      if (x.last) tc_commit(&sm.o_last[x.seg & 1]);
    }
    __syncwarp();
    return true;
  };
  // Each step issues the oldest pending PV, or a tile's S, or goes to the next
  // segment (whose table waits for the end of the segment before the last).
  int seg = -1, left = 0;
  Tile cur{};
#pragma unroll 1
  while (true) {
    if (pending == 2 || (pending == 1 && left == 0 && newer.seg < seg) ||
        (pending == 1 && left < 0)) {
      if (!issue_pv()) return;
      continue;
    }
    if (left < 0) return;
    if (left == 0) {
      ++seg;
      if (!warp_wait(&sm.q_full[seg & 1], (seg >> 1) & 1, sm, err)) return;
      const SegmentTable& tab = sm.table(seg);
      left = uniform(tab.n);
      const bool half = uniform(tab.half) != 0;
      __syncwarp();
      if (elect_one()) mbar_arrive(&sm.o_free[seg & 1]);  // (the table has been read)
      const uint32_t mask = half ? ~((1u << 7) | (1u << 10)) : ~0u;  // fp16 operands
      cur.seg = seg;
      cur.first = 1;
      cur.idesc = (idesc_bf16(128, QR, true) | (1u << 15)) & mask;  // A MN-major, too
      continue;
    }
    const int st = g & 1;
    // (S(g - 2) has been read: PV(g - 2) waited for P(g - 2))
    if (!warp_wait(&sm.k_full[st], (g >> 1) & 1, sm, err)) return;
    tc_fence_after();
    const uint64_t dq = desc_q + (uint32_t)((seg & 1) * (QT >> 4));
    const uint32_t idesc = cur.idesc & ~((1u << 15) | (1u << 16));
    if (elect_one()) {
#pragma unroll
      for (int kk = 0; kk < HD / 16; ++kk)
        tc_mma_bf16_ta(tmem + S_COL + st * QR, tmem + K_COL + st * 64 + kk * 8,
                       dq + (((kk >> 2) * QHALF + (kk & 3) * 32) >> 4), idesc,
                       kk > 0 ? 1u : 0u);
      tc_commit(&sm.s_full[st]);
    }
    __syncwarp();
    cur.last = left == 1 ? 1 : 0;
    older = newer;
    newer = cur;
    cur.first = 0;
    ++pending;
    ++g;
    --left;
  }
}

// ---------------------------------------------------------------- softmax
// A softmax thread: TMEM lane r (a key of the tile; a channel of O), and of
// the queries every kParts-th group of eight from `part` on.
constexpr int kParts = kSoftmaxWarps / 4, NQ = QR / kParts;  // its queries: NQ
struct Place {
  int r, part, lane, quarter, tid;
  uint32_t trow;  // the lane's TMEM address
  uint32_t p_at;  // its first chunk's place in a P tile: chunk c at c ^ (r & 7)
  DF_DEV int query(int i) const { return ((i >> 3) * kParts + part) * 8 + (i & 7); }
};

constexpr int kSoftmaxThreads = kSoftmaxWarps * 32;
DF_DEV void softmax_sync() { named_bar_sync(1, kSoftmaxThreads); }

DF_DEV void load_columns8(uint32_t col, uint32_t* r) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
                 "=r"(r[6]), "=r"(r[7])
               : "r"(col));
}

// Waits for two such loads.  The registers go through the wait, so that nothing
// that takes their values can be placed before it.
DF_DEV void columns16_wait(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                 "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                 "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
}

// this thread's columns (query(0), query(1), ...) of the 64 at `col` of its lane
DF_DEV void load_columns(uint32_t col, int part, float (&v)[NQ]) {
  uint32_t r[NQ];
#pragma unroll
  for (int j = 0; j < NQ / 8; ++j) load_columns8(col + (j * kParts + part) * 8, r + 8 * j);
  columns16_wait(r);
#pragma unroll
  for (int i = 0; i < NQ; ++i) v[i] = __uint_as_float(r[i]);
}

DF_DEV void store_columns8(uint32_t col, const float* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(col),
      "r"(__float_as_uint(v[0])), "r"(__float_as_uint(v[1])), "r"(__float_as_uint(v[2])),
      "r"(__float_as_uint(v[3])), "r"(__float_as_uint(v[4])), "r"(__float_as_uint(v[5])),
      "r"(__float_as_uint(v[6])), "r"(__float_as_uint(v[7]))
      : "memory");
}

DF_DEV float score_of(float s, float scale) { return fminf(__fmul_rn(s, scale), 3.4028235e38f); }

// largest of the warp's x
DF_DEV float warp_max(float x) {
  float y;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
  return y;
}

// Sum v[i] over the warp's lanes: lane i (modulo NQ) returns the i-th (each
// exchange but the first halves the values a lane still holds).
DF_DEV float sum_lanes(float (&v)[NQ], int lane) {
#pragma unroll
  for (int d = 16; d >= NQ; d >>= 1)
#pragma unroll
    for (int i = 0; i < NQ; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], d);
#pragma unroll
  for (int d = NQ / 2; d > 0; d >>= 1) {
    const bool up = (lane & d) != 0;
#pragma unroll
    for (int i = 0; i < d; ++i) {
      const float keep = up ? v[i + d] : v[i], send = up ? v[i] : v[i + d];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, send, d);
    }
  }
  return v[0];
}

// One segment's tiles.  l: this thread's key's share of the queries' sums.
// False if a wait ran out: the loop then still runs to its end, on whatever it
// reads and without waiting, because the warps meet at a barrier in every
// tile.
template <bool HALF16>
DF_DEV bool softmax_segment(SegmentTable& tab, int seg, const Shared& sm, int* err,
                            const Place& at, float (&l)[NQ], int& g) {
  constexpr float lift = HALF16 ? kLift : 0.f;
  const float scale = tab.scale;
  const int n = uniform(tab.n), t0 = uniform(tab.t0), key0 = t0 * TK + at.r;
  // every row sees all of the tiles [clear0, clear1)
  const int clear0 = uniform((tab.lo_all + TK - 1) / TK) - t0;
  const int clear1 = uniform(tab.hi_all / TK) - t0;
  const bool uneven = uniform(tab.uneven) != 0;
  const uint32_t o_col = at.trow + O_COL + (seg & 1) * QR;
  float* row_m = sm.m + (seg & 1) * QR;
  bool ok = true, open = true;  // open: some row has no reference yet
  float off[NQ];                // lift - m of this thread's queries
#pragma unroll
  for (int i = 0; i < NQ; ++i) off[i] = 0.f;
#pragma unroll 1
  for (int t = 0; t < n; ++t, ++g) {
    const int st = g & 1;
    ok = warp_wait(&sm.s_full[st], (g >> 1) & 1, sm, err) && ok;
    tc_fence_after();
    const uint32_t s_col = at.trow + S_COL + st * QR;
    const int key = key0 + t * TK;
    const bool edge = t < clear0 || t >= clear1;
    float v[NQ];
    auto scores = [&]() {  // the unseen at -inf
      load_columns(s_col, at.part, v);
      if (edge) {
        if (uniform(tab.same)) {
          const bool dead = key < tab.lo || key >= tab.hi;
#pragma unroll
          for (int i = 0; i < NQ; ++i) v[i] = dead ? -INFINITY : v[i];
        } else {
#pragma unroll
          for (int i = 0; i < NQ; ++i) {
            const int2 b = tab.seen[at.query(i)];
            if (key < b.x || key >= b.y) v[i] = -INFINITY;
          }
        }
      }
    };
    auto relate = [&]() {
      if (uneven) {
        // not fused: the largest score becomes its row's reference exactly,
        // however large it is
#pragma unroll
        for (int i = 0; i < NQ; ++i) v[i] = __fadd_rn(score_of(v[i], tab.sc[at.query(i)]), off[i]);
      } else {
#pragma unroll
        for (int i = 0; i < NQ; i += 2) {
          const float2 y = fma_f32x2(make_float2(v[i], v[i + 1]), make_float2(scale, scale),
                                     make_float2(off[i], off[i + 1]));
          v[i] = y.x, v[i + 1] = y.y;
        }
      }
    };
    uint8_t* p_tile = sm.p + st * PT;
    // rounded to the products' type (2^-11 relative in fp16, 2^-8 in bf16), the
    // one rounding of the probabilities; their sums take them unrounded
    auto store_p = [&]() {
#pragma unroll
      for (int j = 0; j < NQ / 8; ++j) {
        uint32_t y[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int i = 8 * j + 2 * k;
          y[k] = HALF16 ? pack_f16x2(v[i], v[i + 1]) : pack_bf16x2(v[i], v[i + 1]);
        }
        *reinterpret_cast<uint4*>(p_tile + (at.p_at ^ (uint32_t)(j * kParts * 16))) =
            make_uint4(y[0], y[1], y[2], y[3]);
      }
    };
    bool moves = open;
    if (!open) {
      scores();
      relate();
      float top = v[0];
#pragma unroll
      for (int i = 1; i < NQ - 1; i += 2) top = max3f(top, v[i], v[i + 1]);
      top = fmaxf(top, v[NQ - 1]);
#pragma unroll
      for (int i = 0; i < NQ; ++i) v[i] = fast_exp2(v[i]);
      store_p();
      moves = !all_of(1, kSoftmaxThreads, !(top > lift + kRescale));
    }
    if (moves) {
      // references from this tile's scores on, and what depended on the old
#pragma unroll 1
      for (int pass = 0;; ++pass) {
        scores();
        if (pass == 1) break;
        const int mine = at.query(at.lane & (NQ - 1));
        float highest = 0.f;
#pragma unroll
        for (int i = 0; i < NQ; ++i) {
          const float x = warp_max(v[i]);
          if (at.lane == i) highest = x;
        }
        if (at.lane < NQ) sm.top[at.quarter * QR + mine] = score_of(highest, tab.sc[mine]);
        softmax_sync();
        if (at.tid < QR) {
          const int q = at.tid;
          const float old = t == 0 ? -INFINITY : row_m[q];
          const float m = fmaxf(fmaxf(old, fmaxf(sm.top[q], sm.top[QR + q])),
                                fmaxf(sm.top[2 * QR + q], sm.top[3 * QR + q]));
          row_m[q] = m;
          sm.off[q] = lift - (m == -INFINITY ? 0.f : m);
          sm.alpha[q] = old == -INFINITY ? 1.f : fast_exp2(old - m);
          const bool none = __any_sync(0xffffffffu, q < tab.rows && m == -INFINITY);
          if (at.lane == 0) sm.open[at.tid >> 5] = none ? 1 : 0;
        }
        softmax_sync();
        open = uniform(sm.open[0] | sm.open[1]) != 0;
#pragma unroll
        for (int i = 0; i < NQ; ++i) off[i] = sm.off[at.query(i)];
        if (t > 0) {
          ok = warp_wait(&sm.o_done[st ^ 1], ((g - 1) >> 1) & 1, sm, err) && ok;
          tc_fence_after();
          load_columns(o_col, at.part, v);
#pragma unroll
          for (int i = 0; i < NQ; ++i) {
            const float al = sm.alpha[at.query(i)];
            v[i] *= al;
            l[i] *= al;
          }
#pragma unroll
          for (int j = 0; j < NQ / 8; ++j)
            store_columns8(o_col + (j * kParts + at.part) * 8, v + 8 * j);
          tmem_st_wait();
        }
      }
      relate();
#pragma unroll
      for (int i = 0; i < NQ; ++i) v[i] = fast_exp2(v[i]);
      store_p();
    }
#pragma unroll
    for (int i = 0; i < NQ; i += 2) {
      const float2 s = add_f32x2(make_float2(l[i], l[i + 1]), make_float2(v[i], v[i + 1]));
      l[i] = s.x;
      l[i + 1] = s.y;
    }
    if (!HALF16) {
      // V(g)'s NaN marks, and K(g)'s, which the same warps set before
      ok = warp_wait(&sm.v_full[st], (g >> 1) & 1, sm, err) && ok;
      const int bits = sm.nan_tile[g & 3] == g ? sm.nan_bits[(g & 3) * TK + at.r] |
                                                     sm.nan_bits[(4 + (g & 3)) * TK + at.r]
                                               : 0;
      if (bits != 0) {
#pragma unroll 1
        for (int i = 0; i < NQ; ++i) {
          const int q = at.query(i);
          const int2 b = tab.seen[q];
          if (key >= b.x && key < b.y) atomicOr(tab.nan + q, bits);
        }
      }
    }
    fence_proxy_async_smem();
    warp_arrive(&sm.p_full[st], at.lane);
  }
  return ok;
}

DF_DEV void softmax_all(const Shared& sm, int* err, uint32_t tmem, int warp, int lane) {
  Place at;
  at.quarter = warp & 3;
  at.r = at.quarter * 32 + lane;
  at.part = warp >> 2;
  at.lane = lane;
  at.tid = warp * 32 + lane;
  at.trow = tmem + ((uint32_t)(at.quarter * 32) << 16);
  at.p_at = at.r * (QR * 2) + ((at.part ^ (at.r & 7)) << 4);
  int g = 0;
  for (int seg = 0;; ++seg) {
    if (!all_of(1, kSoftmaxThreads, warp_wait(&sm.q_full[seg & 1], (seg >> 1) & 1, sm, err)))
      return;
    SegmentTable& tab = sm.table(seg);
    const int n = uniform(tab.n);
    if (n < 0) return;
    if (n > 0) {
      float l[NQ];
#pragma unroll
      for (int i = 0; i < NQ; ++i) l[i] = 0.f;
      // (after a wait that ran out the sums are zero, and the rows, too)
      const bool ok = uniform(tab.half) ? softmax_segment<true>(tab, seg, sm, err, at, l, g)
                               : softmax_segment<false>(tab, seg, sm, err, at, l, g);
      const float share = sum_lanes(l, lane);
      if (lane < NQ)
        sm.sum[((seg & 1) * QR + at.query(lane)) * 4 + at.quarter] = ok ? share : 0.f;
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.l_full[seg & 1]);
  }
}

// ---------------------------------------------------------------- output
// What an accumulator of P V is multiplied by.
DF_DEV float v_unit(bool half, int v0) { return half ? __uint_as_float((uint32_t)v0 << 23) : 1.f; }

DF_DEV uint16_t bf16_bits(float x) { return __bfloat16_as_ushort(__float2bfloat16_rn(x)); }

DF_DEV float row_lse(float M, float L, bool half) {
  return L == 0.f ? -INFINITY : (M + (__log2f(L) - (half ? kLift : 0.f))) * 0.6931471805599453f;
}

// A segment's rows out of TMEM, to the output or unnormalised to the segment's
// partial slot, by four warps (thread = channel) while the softmax is at the
// next segment.  Lane i works out what queries i and i + 32 need.
// o_phase: bit i is the phase of o_last[i].
DF_DEV void write_rows(const Q8AttnArgs& a, const Shared& sm, uint32_t tmem, int seg, int quarter,
                       int lane, uint32_t& o_phase) {
  const int st = seg & 1;
  const uint32_t phase = (seg >> 1) & 1;
  const SegmentTable& tab = sm.table(seg);
  const int n = uniform(tab.n), rows = uniform(tab.rows), slot = uniform(tab.slot);
  const bool half = tab.half != 0;
  int2* row = sm.out_rows + quarter * QR;  // factor and output row (or part row)
  bool ok = patient_wait(&sm.l_full[st], phase, sm, a.err);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int q = i * 32 + lane;
    const float4 s = *reinterpret_cast<const float4*>(sm.sum + (st * QR + q) * 4);
    const float M = n > 0 ? sm.m[st * QR + q] : -INFINITY;
    float L = n > 0 && ok ? (s.x + s.y) + (s.z + s.w) : 0.f;
    const int nan = L == 0.f ? 0 : tab.nan[q];
    if (nan & (int)kNanK) L = nan_f();
    float f = L == 0.f ? 0.f : slot >= 0 ? 1.f : v_unit(half, tab.v0) / L;
    if ((nan & (int)kNanK) || ((nan >> quarter) & 1)) f = nan_f();
    row[q] = make_int2(__float_as_int(f), slot >= 0 ? slot * QR + q : tab.dst[q]);
    if (quarter == 0 && q < rows) {
      if (slot >= 0) {
        __stcg(a.part_ml + (size_t)slot * 2 * QR + q, M);
        __stcg(a.part_ml + (size_t)slot * 2 * QR + QR + q, L);
      } else if (a.lse != nullptr) {
        a.lse[tab.dst[q]] = row_lse(M, L, half);
      }
    }
  }
  if (n > 0) {
    ok = warp_wait(&sm.o_last[st], (o_phase >> st) & 1, sm, a.err) && ok;
    o_phase ^= 1u << st;
  }
  tc_fence_after();
  const uint32_t col = tmem + ((uint32_t)(quarter * 32) << 16) + O_COL + st * QR;
  const int d = quarter * 32 + lane;
  __syncwarp();
#pragma unroll 1
  for (int j = 0; j < rows; j += 16) {
    uint32_t v[16];
    load_columns8(col + j, v);
    load_columns8(col + j + 8, v + 8);
    columns16_wait(v);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int2 r = row[j + i];
      const float f = __int_as_float(r.x);
      // (an O that was never written may hold anything)
      const float x = f == 0.f || !ok ? 0.f : __uint_as_float(v[i]) * f;
      if (j + i < rows) {
        if (slot >= 0)
          __stcg(a.part_o + (size_t)r.y * HD + d, x);
        else
          a.out[(size_t)r.y * HD + d] = bf16_bits(x);
      }
    }
  }
  warp_arrive(&sm.o_free[st], lane);
}

// These warps convert a segment's queries ahead of the one in work, and write
// the rows of the one behind it.
DF_DEV void convert_and_write(const Q8AttnArgs& a, const Shared& sm, uint32_t tmem, int warp,
                              int lane) {
  int ready = 0;     // segments converted
  bool more = true;  // none seen without one
  uint32_t o_phase = 0u;
  for (int seg = 0;; ++seg) {
    for (; more && ready <= seg + 1; ++ready) {
      if (!all_of(2, 128, patient_wait(&sm.q_raw[ready & 1], (ready >> 1) & 1, sm, a.err)))
        return;
      more = uniform(sm.table(ready).n) >= 0;
      if (more) convert_queries(a, sm, ready, warp, lane);
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.q_full[ready & 1]);
    }
    if (!more && seg == ready - 1) return;
    write_rows(a, sm, tmem, seg, warp, lane, o_phase);
  }
}

template <int FMT>
__global__ void __launch_bounds__(kThreads, 1)
    attn_q8_kernel(const __grid_constant__ CUtensorMap tm_k,
                   const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ Q8AttnArgs a,
                   const __grid_constant__ Q8Plan plan) {
  extern __shared__ uint8_t smem_raw[];
  // (an offset from the array, not a cast: the compiler has to know that all
  // of this is shared memory)
  uint8_t* smem = smem_raw + ((0u - smem_u32(smem_raw)) & 1023u);
  Shared sm;
  sm.v = smem;
  sm.p = smem + OFF_P;
  sm.q = smem + OFF_Q;
  sm.ring = smem + OFF_RING;
  sm.ring_sc = smem + OFF_SC;
  sm.meta = smem + OFF_META;
  sm.nan_bits = smem + OFF_NAN;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + OFF_BAR);
  sm.ring_full = bars;
  sm.ring_empty = bars + RING;
  sm.k_full = sm.ring_empty + RING;
  sm.v_full = sm.k_full + 2;
  sm.s_full = sm.v_full + 2;
  sm.p_full = sm.s_full + 2;
  sm.o_done = sm.p_full + 2;
  sm.o_last = sm.o_done + 2;
  sm.l_full = sm.o_last + 2;
  sm.q_full = sm.l_full + 2;
  sm.o_free = sm.q_full + 2;
  sm.q_raw = sm.o_free + 2;
  int* words = reinterpret_cast<int*>(bars + 32);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(words);
  sm.abort = words + 1;
  sm.nan_tile = words + 4;
  sm.open = words + 8;
  sm.seg = smem + OFF_SEG;
  float* rows = reinterpret_cast<float*>(smem + OFF_ROWS);
  sm.m = rows;
  sm.off = rows + 2 * QR;
  sm.alpha = rows + 3 * QR;
  sm.top = rows + 4 * QR;
  sm.sum = rows + 8 * QR;
  sm.out_rows = reinterpret_cast<int2*>(rows + 16 * QR);

  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < RING; ++s) {
      mbar_init(&sm.ring_full[s], 1);
      mbar_init(&sm.ring_empty[s], kDecodeWarps / 2);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.k_full[i], kDecodeWarps);
      mbar_init(&sm.v_full[i], kDecodeWarps);
      mbar_init(&sm.s_full[i], 1);
      mbar_init(&sm.p_full[i], kSoftmaxWarps);
      mbar_init(&sm.o_done[i], 1);
      mbar_init(&sm.o_last[i], 1);
      mbar_init(&sm.l_full[i], kSoftmaxWarps);
      mbar_init(&sm.q_raw[i], 2);
      mbar_init(&sm.q_full[i], 4);
      mbar_init(&sm.o_free[i], 4 + 1);
    }
    for (int i = 0; i < 4; ++i) sm.nan_tile[i] = -1;
    *sm.abort = 0;
    fence_mbar_init();
    prefetch_tmap(&tm_k);
    prefetch_tmap(&tm_v);
  }
  if (warp == kWarpMma) {
    tmem_alloc(tmem_slot, TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = uniform(*tmem_slot);
  grid_dep_sync();

  if (warp < kSoftmaxWarps) {
    reg_inc<kSoftmaxRegs>();
    softmax_all(sm, a.err, tmem, warp, lane);
  } else if (warp < kWarpMma) {
    reg_dec<kDecodeRegs>();
    decode_all<FMT>(sm, a.err, tmem, warp - kSoftmaxWarps, lane);
  } else {
    reg_dec<kOtherRegs>();
    if (warp >= kWarpOut) {
      convert_and_write(a, sm, tmem, warp - kWarpOut, lane);
    } else if (warp == kWarpCopy) {
      copy_codes(a, plan, &tm_k, &tm_v, sm);
    } else if (warp >= kWarpQ) {
      fetch_queries(a, plan, sm, warp - kWarpQ, lane);
    } else {
      issue_all(sm, a.err, tmem);
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == kWarpMma) {
    tc_fence_after();
    tmem_dealloc(tmem, TMEM_COLS);
  }
}

// ---------------------------------------------------------------- merge
// Rows of pairs that lie across CTAs: a column of blocks for every place where
// one CTA's share ends, which merges the pair that it cuts if it is the pair's
// first cut; one warp per query row, lane i holding the i-th CTA's reference
// and sum (at most kQ8MaxSplits = 32), four channels per lane.  The parts are
// summed in order, each rescaled to the largest reference: the result does not
// depend on which CTA finished when.  512 bytes per part and row through L2.
constexpr int kMergeWarps = 8;
__global__ void __launch_bounds__(kMergeWarps * 32)
    q8_merge_kernel(const __grid_constant__ Q8AttnArgs a, const __grid_constant__ Q8Plan p) {
  const int lane = threadIdx.x & 31;
  const int cta = blockIdx.x + 1, x = cta * p.share;
  const int b = p.start[cta];
  const int n = tiles_of(p, b), places = n + kPairCost;
  const int pair = (x - p.first[b]) / places, begin = p.first[b] + pair * places;
  const int x0 = begin + kPairCost, c0 = x0 / p.share;
  const int ns = (x0 + n - 1) / p.share - c0 + 1;
  grid_dep_sync();
  if (x <= x0 || c0 != cta - 1) return;
  const int qt = pair / a.st.n_kv, h = pair - qt * a.st.n_kv;
  const int q = blockIdx.y * kMergeWarps + (threadIdx.x >> 5);
  if (qt * QR + q >= a.q_len * a.groups) return;
  // the pair is its first CTA's last segment (slot 1, unless the CTA begins
  // with it), and the others' first
  const int slot0 = 2 * c0 + (c0 * p.share < begin ? 1 : 0);
  const int slot = lane == 0 ? slot0 : 2 * (c0 + lane);
  float m = -INFINITY, l = 0.f;
  if (lane < ns) {
    m = __ldcg(a.part_ml + (size_t)slot * 2 * QR + q);
    l = __ldcg(a.part_ml + (size_t)slot * 2 * QR + QR + q);
  }
  if (l == 0.f) m = -INFINITY;
  float M = m;
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, d));
  const unsigned some = __ballot_sync(0xffffffffu, l != 0.f);  // parts that saw a key
  const float f = l == 0.f ? 0.f : (m == M ? 1.f : fast_exp2(m - M));
  const float fl = l == 0.f ? 0.f : f * l;
  float L = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i0 = 0; i0 < ns; i0 += 8) {
    float4 y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int k = i0 + i;
      if (k < ns)
        y[i] = __ldcg(reinterpret_cast<const float4*>(
                          a.part_o + ((size_t)(k == 0 ? slot0 : 2 * (c0 + k)) * QR + q) * HD) +
                      lane);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int k = i0 + i;
      if (k < ns) {
        const float fi = __shfl_sync(0xffffffffu, f, k);
        L += __shfl_sync(0xffffffffu, fl, k);
        if ((some >> k) & 1u) {
          o.x += fi * y[i].x;
          o.y += fi * y[i].y;
          o.z += fi * y[i].z;
          o.w += fi * y[i].w;
        }
      }
    }
  }
  const Mode mode = mode_of(a.st, b, h);
  const size_t row = (size_t)out_row(a, b, h, qt * QR + q);
  const float s = L == 0.f ? 0.f : v_unit(mode.half, mode.v0) / L;
  *reinterpret_cast<uint2*>(a.out + row * HD + lane * 4) =
      make_uint2(pack_bf16x2(o.x * s, o.y * s), pack_bf16x2(o.z * s, o.w * s));
  if (lane == 0 && a.lse != nullptr) a.lse[row] = row_lse(M, L, mode.half);
}

cudaError_t set_attrs() {
  static std::atomic<unsigned long long> done{0};
  if (done_on_device(done)) return cudaSuccess;
  for (const void* f : {(const void*)attn_q8_kernel<Q8_E4M3>, (const void*)attn_q8_kernel<Q8_INT8>}) {
    const cudaError_t e =
        cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
    if (e != cudaSuccess) return e;
  }
  mark_device(done);
  return cudaSuccess;
}

}  // namespace

size_t q8_attention_slots(int num_sms) { return (size_t)2 * num_sms; }

bool plan_q8_attention(Q8Plan& p, int batch, int n_kv, int n_q_tiles, int num_sms) {
  // one CTA per SM, equal shares of the line; a pair's parts are merged by the
  // lanes of a warp, so a share is at least 1/32 of the longest pair (whose
  // ends may both lie inside a share: 1/30)
  num_sms = std::min(num_sms, kQ8MaxCtas);
  long long total = 0;
  int longest = 1;
  for (int b = 0; b < batch; ++b) {
    p.first[b] = (int)total;
    const int n = tiles_of(p, b);
    longest = std::max(longest, n);
    total += (long long)(n + kPairCost) * n_kv * n_q_tiles;
    if (total >= (1LL << 30)) return false;
  }
  p.first[batch] = (int)total;
  p.share = (int)std::max<long long>((total + num_sms - 1) / num_sms,
                                     (longest + kQ8MaxSplits - 3) / (kQ8MaxSplits - 2));
  int b = 0;
  for (int c = 0; (long long)c * p.share < total; ++c) {
    while ((long long)c * p.share >= p.first[b + 1]) ++b;
    p.start[c] = (uint16_t)b;
  }
  return true;
}

int launch_q8_attention(int fmt, const CUtensorMap& tm_k, const CUtensorMap& tm_v,
                        const Q8AttnArgs& a, const Q8Plan& p, cudaStream_t s) {
  if (const cudaError_t e = set_attrs()) return e;
  const int total = p.first[a.batch];
  const dim3 grid((unsigned)((total - 1) / p.share + 1)), block(kThreads);
  const cudaError_t e =
      fmt == Q8_E4M3 ? launch_pdl(attn_q8_kernel<Q8_E4M3>, grid, block, kSmem, s, tm_k, tm_v, a, p)
                     : launch_pdl(attn_q8_kernel<Q8_INT8>, grid, block, kSmem, s, tm_k, tm_v, a, p);
  if (e != cudaSuccess) return e;
  bool cut = false;
  for (unsigned c = 1; c < grid.x && !cut; ++c) {
    const int b = p.start[c], places = tiles_of(p, b) + kPairCost;
    cut = ((int)c * p.share - p.first[b]) % places > kPairCost;
  }
  if (!cut) return cudaSuccess;
  return launch_pdl(q8_merge_kernel, dim3(grid.x - 1, QR / kMergeWarps), dim3(kMergeWarps * 32), 0,
                    s, a, p);
}

}  // namespace df
