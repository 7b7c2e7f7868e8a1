// attn_q8.cu -- attention of the draft's block queries over an 8-bit cache
// (formats: q8.cuh) on tcgen05.
//
//   S = scale * Q K^T over the keys a row sees, O = softmax(S) V
//
// The key tiles (128 keys) of every (sequence, query tile, kv head) -- a pair
// -- stand in one line; CTA c, one per SM, takes tiles [c U, (c + 1) U) of it:
// segments of one pair after another.  Every SM gets the same number of tiles
// whatever the lengths, and a pair that lies across CTAs is merged afterwards.
//
// The codes of a tile are 33 KB against the 64 KB of a bf16 tile, so HBM asks
// for a tile every 0.74 us per SM; on the way to the tensor core every code
// becomes a 16-bit number in shared memory.  Most warps do nothing else.  The two
// MMAs are the longest queue, about 2560 cycles a tile:
//
//   warps 0-7    softmax, two threads per TMEM lane (accumulator row); the Q
//                tile into TMEM at a segment's start, O out at its end
//   warps 8-15   decode: a tile's codes of K, then of V, from the ring to the
//                tile in the tensor core's 128-byte-swizzled layout, two
//                stages of each
//   warp 16      TMEM allocator; S(g) = Q K(g)^T
//   warp 17      O += P(g) V(g)
//   warp 18      bulk copies of codes and scales, half a tile of K or V per
//                slot of a nine-slot ring (59 KB in flight beside the two
//                slots being decoded), and of a segment's query rows
//
// All of them run on across segments, so a segment's start costs its Q and the
// last one's O, not a pipeline.  Prefetching codes into the decode warps'
// registers instead of a ring left those warps waiting for the newest load
// whenever they needed the oldest (127 us against 112 us on 32 sequences of 512
// to 8192 keys, before the other steps); decoding K and V by the same eight
// warps left the issue slots half empty; one warp for both products let PV
// wait for the next tile's K.
//
// Shared memory is what the decode warps and the tensor core compete for
// (bulk writes, code reads, tile writes and tile reads: about 1500 cycles a
// tile), so Q and P are read from TMEM (A operands).  TMEM columns: S
// double-buffered [0, 256), O [256, 384), Q as 16-bit pairs [384, 448); P(g)
// overwrites the first 64 columns of S(g).
//
// The MMA has 128 rows.  A query tile of at most 64 (32) rows is held two
// (four) times: copy c of a row takes the c-th 64 (32) keys of every tile as
// an online softmax of its own (its P is zero elsewhere), and the copies are
// merged at the end, so that all four softmax warps work on a short block.
//
// Rows behind the sequence's end decode to zero, so nothing stale can reach O
// through a zero probability.  A group that reads NaN is decoded as zero too;
// the rows that see its key remember it and return NaN (in V's case in the
// group's channels), the others are untouched.
#include <algorithm>
#include <atomic>

#include "q8.cuh"

namespace df {
namespace {

constexpr int HD = 128;
constexpr int TK = 128;                   // keys per tile
constexpr int kSoftmaxWarps = 8;
constexpr int kDecodeWarps = 8;
constexpr int kWarpS = kSoftmaxWarps + kDecodeWarps, kWarpPV = kWarpS + 1;
constexpr int kWarpCopy = kWarpS + 2;
constexpr int kThreads = (kWarpCopy + 2) * 32;  // (a multiple of four warps)
constexpr int RING = 9;                   // slots of half a tile's K or V codes
constexpr int HK = TK / 2;                // keys of a slot
constexpr uint32_t SLOT = HK * HD + HK * 4;
constexpr uint32_t TILE = TK * HD * 2;    // one decoded tile
constexpr uint32_t HALF = TILE / 2;       // 64 channels of it
constexpr uint32_t O_COL = 256, Q_COL = 384, TMEM_COLS = 512;
// staged query rows (at most 64) and, between segments, 32 channels of the
// lanes' O on their way out
constexpr uint32_t Q_PITCH = HD * 2 + 16;
constexpr int X_LD = 36;
constexpr uint32_t QX_BYTES = 128 * X_LD * 4;
static_assert(QX_BYTES >= 64 * Q_PITCH, "query rows");
constexpr size_t kSmem = 1024 + 4 * TILE + RING * SLOT + QX_BYTES + 4 * TK + 512 + 9 * TK * 4;
constexpr float kRescale = 8.f;           // log2 units
constexpr float kLift = 7.f;              // fp16 P = 2^(score - max + 7)
constexpr uint32_t kNanK = 16;            // the key reads NaN in K

// ---------------------------------------------------------------- segments
// A CTA's tiles [x, end) of one pair: what the CTA does of it.
struct Segment {
  int b, h, qt;
  int tokens, rows;   // real block rows and query rows of the tile
  int len;
  int lo, hi;         // keys any row of the query tile sees, within the segment
  int t0, t1;         // the tiles that hold them (none: t0 = t1)
  int slot;           // partial slot, or -1 if the segment is the whole pair
};

// Tiles of one of sequence b's pairs: at least one, so that every row is
// written by some CTA.
__host__ __device__ inline int tiles_of(const Q8Plan& p, int b) {
  const int n = (p.len[b] + TK - 1) / TK - p.lo[b] / TK;
  return n > 0 ? n : 1;
}

// the sequence whose tiles x lies in
DF_DEV int sequence_at(const Q8Plan& p, int batch, int x) {
  int lo = 0, hi = batch;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (p.first[mid] <= x) lo = mid; else hi = mid;
  }
  return lo;
}

// Walks a CTA's segments.
struct Walk {
  int x, end, b;
  bool begun;
  DF_DEV Walk(const Q8AttnArgs& a, const Q8Plan& p) {
    x = (int)blockIdx.x * p.share;
    end = min(x + p.share, p.first[a.batch]);
    b = sequence_at(p, a.batch, x);
    begun = false;
  }
  DF_DEV bool next(const Q8AttnArgs& a, const Q8Plan& p, Segment& w) {
    if (x >= end) return false;
    while (x >= p.first[b + 1]) ++b;
    const int n = tiles_of(p, b), rel = x - p.first[b];
    const int pair = rel / n, i0 = rel - pair * n, i1 = min(n, i0 + end - x);
    w.b = b;
    w.qt = pair / a.st.n_kv;
    w.h = pair - w.qt * a.st.n_kv;
    w.slot = i0 == 0 && i1 == n ? -1 : 2 * (int)blockIdx.x + (begun ? 1 : 0);
    x += i1 - i0;
    begun = true;
    const int tok0 = w.qt * a.tile_tokens;
    w.tokens = min(a.tile_tokens, a.q_len - tok0);
    w.rows = w.tokens * a.groups;
    w.len = p.len[b];
    const int q0 = w.len - a.q_len + tok0, q1 = q0 + w.tokens - 1;
    int k0 = 0, k1 = w.len;
    if (a.window > 0) {
      k0 = (int)max(0LL, (long long)q0 - a.window + 1);
      k1 = (int)min((long long)k1, (long long)q1 + a.window);
    }
    if (a.causal) k1 = min(k1, q1 + 1);
    const int t = p.lo[b] / TK;
    w.lo = max(k0, (t + i0) * TK);
    w.hi = min(k1, (t + i1) * TK);
    w.t0 = w.lo / TK;
    w.t1 = w.hi > w.lo ? (w.hi + TK - 1) / TK : w.t0;
    return true;
  }
};

// output (and log-sum-exp) row of query row qr of a tile
DF_DEV size_t out_row(const Q8AttnArgs& a, int b, int h, int qt, int tokens, int qr) {
  const int g = qr / tokens, t = qr - g * tokens;
  const size_t token = (size_t)b * a.q_len + qt * a.tile_tokens + t;
  return token * (a.st.n_kv * a.groups) + h * a.groups + g;
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

// what an accumulator of P V is multiplied by, and what P is lifted by
DF_DEV float v_unit(const Mode& m) { return m.half ? __uint_as_float((uint32_t)m.v0 << 23) : 1.f; }
DF_DEV float lift_of(const Mode& m) { return m.half ? kLift : 0.f; }

// Shared memory of a CTA.  Barriers come in pairs by the parity of g, the
// CTA's running tile number over all its segments.
struct Shared {
  uint8_t *k, *v;          // [2] decoded tiles each
  uint8_t* ring;           // [RING][codes | scales]
  uint8_t* qx;             // [64][Q_PITCH] query rows; [128][X_LD] floats
  uint8_t* nan_bits;       // [K, V][2][TK]
  float* pair;             // [2][2][128] by tile parity: what a lane's two
                           // threads tell one another
  float *row_m, *row_l;    // [128], [2][128]
  float* row_f;            // [128] what a lane's O counts in its row
  int* row_nan;            // [128]
  uint64_t *ring_full, *ring_empty;  // [RING]
  uint64_t *k_full, *v_full;         // [2]
  uint64_t *s_full;        // S(g) complete: K(g)'s stage is free
  uint64_t *p_full;
  uint64_t *o_done;        // PV(g) complete: V(g)'s stage and S(g)'s buffer are free
  int4* mode;              // [2] by segment: half, k0, v0
  uint64_t *q_staged;      // per segment: its mode and query rows are in shared memory
  uint64_t *q_full;        // per segment: Q is in TMEM
  uint64_t *o_free;        // per segment: O has been read, the exchange is over
  volatile int* abort;
  volatile int* nan_tile;  // [2] the last tile of this parity with a NaN
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

DF_DEV bool warp_wait(uint64_t* bar, uint32_t parity, const Shared& sm, int* err) {
  return __all_sync(0xffffffffu, wait(bar, parity, sm, err));
}

// ---------------------------------------------------------------- decode
// A decode lane's share of its warp's 16 rows of half a tile: it owns two rows
// and takes 16 codes of each in each of two passes.  Lanes 0-3 of eight take
// the one half of an even row, lanes 4-7 the other half of the odd row, so
// that the eight 16-byte reads and stores of a phase fall into different
// banks.
struct DecodeLane {
  int row[2];          // rows of the half tile
  int src[2];          // pass 0 within a ring slot; pass 1 is 64 bytes away (xor)
  int dst[2];          // pass 0's first store within a tile; the second is 16
                       // bytes away (xor), pass 1 in the other half
  uint32_t group[2];   // scale byte of each pass
};

DF_DEV DecodeLane decode_lane(int warp, int lane) {  // warp: 0..7 of its group
  DecodeLane l;
  const int sub = (lane >> 2) & 1, u4 = lane & 3;
  for (int o = 0; o < 2; ++o) {
    const int r = (warp & 3) * 16 + o * 8 + (lane >> 3) * 2 + sub;
    l.row[o] = r;
    l.src[o] = r * HD + sub * 64 + u4 * 16;
    l.dst[o] = sub * (int)HALF + ((warp >> 2) * HK + r) * 128 + ((2 * u4) ^ (r & 7)) * 16;
  }
  for (int p = 0; p < 2; ++p) l.group[p] = (uint32_t)((sub ^ p) * 2 + (u4 >> 1));
  return l;
}

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

// A warp's rows of half a tile, as they come out of a ring slot.
struct Codes {
  uint4 c[2][2];
  uint32_t bytes[2];
};

DF_DEV void read_codes(Codes& x, const uint8_t* slot, const DecodeLane& l) {
#pragma unroll
  for (int o = 0; o < 2; ++o) {
    x.bytes[o] = *reinterpret_cast<const uint32_t*>(slot + HK * HD + l.row[o] * 4);
#pragma unroll
    for (int p = 0; p < 2; ++p)
      x.c[o][p] = *reinterpret_cast<const uint4*>(slot + (l.src[o] ^ (p * 64)));
  }
}

// Decode them (first key key0) into `tile`.
template <int FMT, bool HALF16>
DF_DEV void decode_rows(Codes& x, uint8_t* tile, const DecodeLane& l, bool is_k, int key0, int lo,
                        int hi, int unit0, uint32_t (&bits)[2]) {
  if (HALF16 && (key0 < lo || key0 + HK > hi)) {
#pragma unroll
    for (int o = 0; o < 2; ++o)
      if (key0 + l.row[o] < lo || key0 + l.row[o] >= hi) {  // codes and scale of zero
        constexpr uint32_t zero = FMT == Q8_INT8 ? 0x80808080u : 0u;
        x.c[o][0] = x.c[o][1] = make_uint4(zero, zero, zero, zero);
        x.bytes[o] = 0u;
      }
  }
#pragma unroll
  for (int o = 0; o < 2; ++o) {
    HalfScales hs;
    if (HALF16)
      hs = half_scales(x.bytes[o], unit0);
    else
      x.bytes[o] = live_scales(x.bytes[o], is_k, key0 + l.row[o] >= lo && key0 + l.row[o] < hi,
                               bits[o]);
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      const uint4 c = x.c[o][p];
      uint4 a, b;
      if (HALF16) {
        half_decode16<FMT>(c, hs, half_select(l.group[p]), a, b);
      } else {
        const float s = bf16_scale((x.bytes[o] >> (l.group[p] * 8)) & 0xffu);
        a = bf16_decode8<FMT>(c.x, c.y, s);
        b = bf16_decode8<FMT>(c.z, c.w, s);
      }
      const int dst = l.dst[o] ^ (p * (int)HALF);
      *reinterpret_cast<uint4*>(tile + dst) = a;
      *reinterpret_cast<uint4*>(tile + (dst ^ 16)) = b;
    }
  }
}

// One segment's tiles: K, then V.  A slot is free as soon as its codes are in
// registers, before the tile's stage is: the ring stays in flight.
template <int FMT, bool HALF16>
DF_DEV bool decode_segment(const Segment& w, const Mode& mode, const Shared& sm, int* err,
                           int half, int lane, const DecodeLane& l, int& g) {
  for (int t = w.t0; t < w.t1; ++t, ++g) {
    const int st = g & 1;
#pragma unroll 1
    for (int kv = 0; kv < 2; ++kv) {
      const bool is_k = kv == 0;
      const int n = 4 * g + 2 * kv + half, slot = n % RING;
      if (!warp_wait(&sm.ring_full[slot], (n / RING) & 1, sm, err)) return false;
      Codes x;
      read_codes(x, sm.ring + slot * SLOT, l);
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.ring_empty[slot]);
      if (!warp_wait(is_k ? &sm.s_full[st] : &sm.o_done[st], ((g >> 1) & 1) ^ 1, sm, err))
        return false;
      uint32_t bits[2] = {0u, 0u};
      decode_rows<FMT, HALF16>(x, (is_k ? sm.k : sm.v) + st * TILE, l, is_k, t * TK + half * HK,
                               w.lo, w.hi, is_k ? mode.k0 : mode.v0, bits);
      if (!HALF16) {
        // The softmax of tile g - 2 has read these marks before PV(g - 2) was
        // issued; K's marks wait for that here.
        if (is_k && !warp_wait(&sm.o_done[st], ((g >> 1) & 1) ^ 1, sm, err)) return false;
        if ((lane & 3) == 0)
          for (int o = 0; o < 2; ++o)
            sm.nan_bits[(2 * kv + st) * TK + half * HK + l.row[o]] = (uint8_t)bits[o];
        if ((bits[0] | bits[1]) != 0u) sm.nan_tile[st] = g;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(is_k ? &sm.k_full[st] : &sm.v_full[st]);
    }
  }
  return true;
}

template <int FMT>
DF_DEV void decode_all(const Q8AttnArgs& a, const Q8Plan& p, const Shared& sm, int warp,
                       int lane) {
  const DecodeLane l = decode_lane(warp, lane);
  Walk walk(a, p);
  Segment w;
  int g = 0;
  while (walk.next(a, p, w)) {
    if (w.t1 == w.t0) continue;
    const Mode m = mode_of(a.st, w.b, w.h);
    if (!(m.half ? decode_segment<FMT, true>(w, m, sm, a.err, warp >> 2, lane, l, g)
                 : decode_segment<FMT, false>(w, m, sm, a.err, warp >> 2, lane, l, g)))
      return;
  }
}

// ---------------------------------------------------------------- copies
DF_DEV void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar,
                      uint64_t policy) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], "
      "[%1], %2, [%3], %4;" ::"r"(smem_u32(dst)),
      "l"(src), "r"(bytes), "r"(smem_u32(bar)), "l"(policy)
      : "memory");
}

// Lane 0 copies the tiles, every lane its query rows; how the segment is
// decoded goes to the softmax warps with them.  On an abort the copies
// in flight are still waited for, with a limit: no CTA may leave before they
// have landed.
DF_DEV void copy_all(const Q8AttnArgs& a, const Q8Plan& p, const Shared& sm, bool stage_q,
                     int lane) {
  const uint64_t once = policy_evict_first();
  Walk walk(a, p);
  Segment w;
  int n = 0, seg = 0;
  bool alive = true;
  while (alive && walk.next(a, p, w)) {
    if (w.t1 == w.t0) continue;
    // the rows of segment seg - 1 have been read, and the exchange that
    // followed (of segment seg - 2's O) is over
    if (seg == 1) alive = warp_wait(sm.q_full, 0, sm, a.err);
    if (seg >= 2) alive = warp_wait(sm.o_free, seg & 1, sm, a.err);
    if (!alive) break;
    if (lane == 0) {
      const Mode m = mode_of(a.st, w.b, w.h);
      sm.mode[seg & 1] = make_int4(m.half ? 1 : 0, m.k0, m.v0, 0);
      if (stage_q)
        mbar_arrive_expect_tx(sm.q_staged, (uint32_t)w.rows * HD * 2);
      else
        mbar_arrive(sm.q_staged);
    }
    if (stage_q) {
      __syncwarp();
      const uint16_t* q = a.q + (long long)w.b * a.q_seq + (long long)w.h * a.q_head;
      for (int r = lane; r < w.rows; r += 32) {
        const int g = r / w.tokens, t = w.qt * a.tile_tokens + r - g * w.tokens;
        bulk_load(sm.qx + r * Q_PITCH, q + (long long)g * a.q_group + (long long)t * a.q_tok,
                  HD * 2, sm.q_staged, once);
      }
    }
    ++seg;
    if (lane == 0) {
      const size_t row0 = ((size_t)w.b * a.st.n_kv + w.h) * a.st.cap;
      for (int t = w.t0; t < w.t1 && alive; ++t) {
#pragma unroll 1
        for (int i = 0; i < 4; ++i) {
          const int slot = n % RING;
          alive = wait(&sm.ring_empty[slot], ((n / RING) & 1) ^ 1, sm, a.err);
          if (!alive) break;
          const size_t row = row0 + (size_t)t * TK + (i & 1) * HK;
          uint8_t* dst = sm.ring + slot * SLOT;
          mbar_arrive_expect_tx(&sm.ring_full[slot], SLOT);
          bulk_load(dst, (i < 2 ? a.st.k : a.st.v) + row * HD, HK * HD, &sm.ring_full[slot],
                    once);
          bulk_load(dst + HK * HD, (i < 2 ? a.st.ks : a.st.vs) + row * 4, HK * 4,
                    &sm.ring_full[slot], once);
          ++n;
        }
      }
    }
    alive = __shfl_sync(0xffffffffu, (int)alive, 0) != 0;
  }
  if (lane == 0) {
    const uint64_t t0 = global_ns();
    for (int i = max(0, n - RING); i < n; ++i)
      while (!mbar_try_wait(&sm.ring_full[i % RING], (i / RING) & 1) &&
             global_ns() - t0 < kWaitLimitNs) {
      }
    while (seg > 0 && !mbar_try_wait(sm.q_staged, (seg - 1) & 1) &&
           global_ns() - t0 < kWaitLimitNs) {
    }
  }
  __syncwarp();
}

// ---------------------------------------------------------------- products
// One lane each.  The decode warps' stores, ordered before this by a tile's
// barrier, become visible to the tensor core through the issuing thread's
// proxy fence (in a decode warp the fence would wait for its loads as well).
DF_DEV uint32_t f16_mask(const Mode& m) { return m.half ? ~((1u << 7) | (1u << 10)) : ~0u; }

DF_DEV void issue_s(const Q8AttnArgs& a, const Q8Plan& p, const Shared& sm, uint32_t tmem) {
  const uint64_t desc0 = sdesc_sw128(smem_u32(sm.k), 16, 1024);
  Walk walk(a, p);
  Segment w;
  int g = 0, seg = 0;
  while (walk.next(a, p, w)) {
    if (w.t1 == w.t0) continue;
    const uint32_t idesc = idesc_bf16(128, TK, false) & f16_mask(mode_of(a.st, w.b, w.h));
    if (!wait(sm.q_full, seg & 1, sm, a.err)) return;
    for (int t = w.t0; t < w.t1; ++t, ++g) {
      const int st = g & 1;
      // (S(g)'s buffer is free once PV(g - 2) has read P(g - 2))
      if (!wait(&sm.k_full[st], (g >> 1) & 1, sm, a.err) ||
          !wait(&sm.o_done[st], ((g >> 1) & 1) ^ 1, sm, a.err))
        return;
      fence_proxy_async_smem();
      tc_fence_after();
      const uint64_t desc = desc0 + (uint32_t)(st * (TILE >> 4));  // (in 16-byte units)
#pragma unroll
      for (int kk = 0; kk < HD / 16; ++kk)
        tc_mma_bf16_ta(tmem + (uint32_t)(st * TK), tmem + Q_COL + kk * 8,
                       desc + (((kk >> 2) * HALF + (kk & 3) * 32) >> 4), idesc,
                       kk > 0 ? 1u : 0u);
      tc_commit(&sm.s_full[st]);
    }
    ++seg;
  }
}

DF_DEV void issue_pv(const Q8AttnArgs& a, const Q8Plan& p, const Shared& sm, uint32_t tmem) {
  const uint64_t desc0 = sdesc_sw128(smem_u32(sm.v), HALF, 1024);
  Walk walk(a, p);
  Segment w;
  int g = 0, seg = 0;
  while (walk.next(a, p, w)) {
    if (w.t1 == w.t0) continue;
    const uint32_t idesc = idesc_bf16(128, HD, true) & f16_mask(mode_of(a.st, w.b, w.h));
    if (!wait(sm.o_free, (seg & 1) ^ 1, sm, a.err)) return;
    for (int t = w.t0; t < w.t1; ++t, ++g) {
      const int st = g & 1;
      if (!wait(&sm.v_full[st], (g >> 1) & 1, sm, a.err)) return;
      fence_proxy_async_smem();
      if (!wait(&sm.p_full[st], (g >> 1) & 1, sm, a.err)) return;
      tc_fence_after();
      const uint64_t desc = desc0 + (uint32_t)(st * (TILE >> 4));
#pragma unroll
      for (int kk = 0; kk < TK / 16; ++kk)
        tc_mma_bf16_ta(tmem + O_COL, tmem + (uint32_t)(st * TK) + kk * 8,
                       desc + ((kk * 16 * 128) >> 4), idesc, (t > w.t0 || kk > 0) ? 1u : 0u);
      tc_commit(&sm.o_done[st]);
    }
    ++seg;
  }
}

// ---------------------------------------------------------------- softmax
struct SoftmaxRow {
  float sc;          // of a score, in log2 units
  int k_lo, k_hi;    // the keys it sees
  float m, l;        // running max (log2 units) and sum of P
  int nan;           // V groups that read NaN (bits 0-3), kNanK
};

// Where a softmax thread works: TMEM lane r = query row qr in copy `seg` of it;
// of what the lane has to do, thread hh = 0, 1 takes the one half.
struct Place {
  int r, qr, seg, hh, lane, quarter;
  uint32_t trow;  // the lane's TMEM address
};

// wait for the other thread of every lane of this warp (and for this warp's)
DF_DEV void pair_sync(const Place& at) { named_bar_sync(2 + at.quarter, 64); }

// One arrival per warp, after what its threads did in TMEM.
DF_DEV void warp_arrive(uint64_t* bar, int lane) {
  tc_fence_before();
  __syncwarp();
  if (lane == 0) mbar_arrive(bar);
}

// This thread's half of its query row as the A operand of S: 32 columns of
// bf16 pairs, or of fp16 pairs scaled by the power of two that brings the
// row's largest magnitude to [2^13, 2^14): exact but for what is 2^-30 of it.
template <int COPIES>
DF_DEV void load_q(const Q8AttnArgs& a, const Segment& w, const Mode& mode, const Shared& sm,
                   const Place& at, SoftmaxRow& row) {
  const bool real = at.qr < w.rows;
  uint4 y[8];
  if (COPIES > 1) {
    const uint4* src = reinterpret_cast<const uint4*>(sm.qx + at.qr * Q_PITCH) + at.hh * 8;
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = real ? src[i] : make_uint4(0u, 0u, 0u, 0u);
  } else {
    const int g = at.qr / w.tokens, t = w.qt * a.tile_tokens + at.qr - g * w.tokens;
    const uint4* src = reinterpret_cast<const uint4*>(
                           a.q + (real ? (long long)w.b * a.q_seq + (long long)w.h * a.q_head +
                                             (long long)g * a.q_group + (long long)t * a.q_tok
                                       : 0)) + at.hh * 8;
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = real ? __ldcg(src + i) : make_uint4(0u, 0u, 0u, 0u);
  }
  uint32_t top2 = 0u;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t m = 0x7fff7fffu;
    top2 = __vmaxu2(top2, __vmaxu2(__vmaxu2(y[i].x & m, y[i].y & m),
                                   __vmaxu2(y[i].z & m, y[i].w & m)));
  }
  int top = (int)max(top2 & 0xffffu, top2 >> 16);
  pair_sync(at);  // (the last tile's exchange has been read)
  sm.pair[at.hh * 128 + at.r] = __int_as_float(top);
  pair_sync(at);
  top = max(top, __float_as_int(sm.pair[(at.hh ^ 1) * 128 + at.r]));
  const bool finite = top < 0x7f80;
  if (!finite) row.nan = kNanK;  // the row is NaN if it sees a key
  const int field = max(top >> 7, 14);
  const float up = __uint_as_float((uint32_t)(267 - field) << 23);
  if (mode.half) {
    // a.scale * 2^(field - 140 + k0 - 127), in two steps
    row.sc *= __uint_as_float((uint32_t)(field - 13) << 23);
    row.sc *= __uint_as_float((uint32_t)mode.k0 << 23);
  }
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    uint32_t x[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const uint4 z = y[c * 4 + (i >> 2)];
      uint32_t v = (i & 3) == 0 ? z.x : (i & 3) == 1 ? z.y : (i & 3) == 2 ? z.z : z.w;
      if (!finite) v = 0u;
      if (mode.half)
        v = pack_f16x2(__uint_as_float(v << 16) * up, __uint_as_float(v & 0xffff0000u) * up);
      x[i] = v;
    }
    tmem_st16_nowait(at.trow + Q_COL + at.hh * 32 + c * 16, x);
  }
  tmem_st_wait();
  pair_sync(at);  // the exchange is free again
}

// W consecutive columns of this thread's TMEM lane (16 or 32), or stores
template <int W>
DF_DEV void tmem_load(uint32_t taddr, float (&v)[W]) {
  if constexpr (W == 32) {
    tmem_ld32(taddr, v);
  } else {
    uint32_t r[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
          "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
    tmem_ld_wait();
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
  }
}

template <int W>
DF_DEV void tmem_store(uint32_t taddr, const uint32_t (&v)[W]) {
  if constexpr (W == 8) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(
            taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
        : "memory");
  } else if constexpr (W == 16) {
    tmem_st16_nowait(taddr, v);
  } else {
    tmem_st32_nowait(taddr, v);
  }
}

// One segment's tiles: online softmax of this thread's keys of its row's copy,
// P into TMEM.  False if a wait ran out: the loop then still runs to its end,
// on whatever it reads and without waiting, because the threads of a lane
// meet at a barrier in every tile.
template <int COPIES, bool HALF16>
DF_DEV bool softmax_segment(const Segment& w, const Shared& sm, int* err, const Place& at,
                            SoftmaxRow& row, int& g) {
  constexpr int NT = TK / COPIES / 2;   // keys of a tile that this thread handles
  constexpr int W = NT < 32 ? NT : 32;  // held at a time
  constexpr int CH = NT / W;            // (two times 32 are read twice)
  constexpr float lift = HALF16 ? kLift : 0.f;
  const float2 sc2 = make_float2(row.sc, row.sc);
  const int key0 = at.seg * 2 * NT + at.hh * NT;
  bool ok = true;
  for (int t = w.t0; t < w.t1; ++t, ++g) {
    const int st = g & 1;
    ok = warp_wait(&sm.s_full[st], (g >> 1) & 1, sm, err) && ok;
    tc_fence_after();
    const uint32_t s_col = at.trow + st * TK;
    const int k0 = t * TK + key0;
    const bool edge = !(k0 >= row.k_lo && k0 + NT <= row.k_hi);
    float s[W];
    auto load = [&](int c) {  // the unseen at -inf
      tmem_load<W>(s_col + key0 + c * W, s);
      if (edge) {
#pragma unroll
        for (int i = 0; i < W; ++i) {
          const int key = k0 + c * W + i;
          if (key < row.k_lo || key >= row.k_hi) s[i] = -INFINITY;
        }
      }
    };
    float tmax = -INFINITY;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      load(c);
      float pm[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        pm[e] = max3f(s[e], s[e + 4], s[e + 8]);
#pragma unroll
        for (int i = 12; i < W; i += 8)
          pm[e] = i + 4 < W ? max3f(pm[e], s[e + i], s[e + (i + 4) % W]) : fmaxf(pm[e], s[e + i]);
      }
      tmax = fmaxf(tmax, fmaxf(fmaxf(pm[0], pm[1]), fmaxf(pm[2], pm[3])));
    }
    tmax *= row.sc;
    // the lane's largest over both threads' keys; both have read their scores
    sm.pair[(st * 2 + at.hh) * 128 + at.r] = tmax;
    pair_sync(at);
    tmax = fmaxf(tmax, sm.pair[(st * 2 + (at.hh ^ 1)) * 128 + at.r]);
    // the maximum grows only by more than 2^kRescale at a time (fp16 P up to
    // 2^(kRescale + kLift))
    float alpha = 1.f;
    if (row.m == -INFINITY || tmax > row.m + kRescale) {
      if (row.m != -INFINITY) alpha = fast_exp2(row.m - tmax);
      row.m = tmax;
    }
    // O is touched only to rescale it, and only then must PV(g-1) be complete:
    // S(g) was issued after PV(g-2), so a parity wait on o_done is exact.  (A
    // row without keys so far has P = 0 and needs no rescaling.)
    if (t > w.t0 && __any_sync(0xffffffffu, alpha != 1.f)) {
      ok = warp_wait(&sm.o_done[st ^ 1], ((g - 1) >> 1) & 1, sm, err) && ok;
      tc_fence_after();
#pragma unroll 1
      for (int c = 0; c < 4; ++c) {
        float o[16];
        uint32_t x[16];
        const uint32_t col = at.trow + O_COL + at.hh * 64 + c * 16;
        tmem_load<16>(col, o);
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = __float_as_uint(o[i] * alpha);
        tmem_store<16>(col, x);
      }
    }
    const float off = lift - (row.m == -INFINITY ? 0.f : row.m);
    const float2 off2 = make_float2(off, off);
    float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
    uint32_t p[NT / 2];
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      if (CH > 1) load(c);
#pragma unroll
      for (int i = 0; i < W / 2; ++i) {
        float2 e = fma_f32x2(make_float2(s[2 * i], s[2 * i + 1]), sc2, off2);
        e.x = fast_exp2(e.x);
        e.y = fast_exp2(e.y);
        sum[i & 1] = add_f32x2(sum[i & 1], e);
        p[c * (W / 2) + i] = HALF16 ? pack_f16x2(e.x, e.y) : pack_bf16x2(e.x, e.y);
      }
    }
    if (CH > 1) pair_sync(at);  // the scores under P have been read again
    // P over the first 64 columns of S: this copy's keys, zero for the others'
    tmem_store<NT / 2>(s_col + key0 / 2, p);
    if (COPIES > 1) {
      uint32_t zero[NT / 2];
#pragma unroll
      for (int i = 0; i < NT / 2; ++i) zero[i] = 0u;
#pragma unroll
      for (int c = 0; c < COPIES; ++c)
        if (c != at.seg) tmem_store<NT / 2>(s_col + c * NT + at.hh * (NT / 2), zero);
    }
    row.l = row.l * alpha + ((sum[0].x + sum[0].y) + (sum[1].x + sum[1].y));
    if (!HALF16) {
      // PV(g) needs V(g) anyway; its NaN marks are complete then (K's are, as
      // S(g) is)
      ok = warp_wait(&sm.k_full[st], (g >> 1) & 1, sm, err) && ok;
      ok = warp_wait(&sm.v_full[st], (g >> 1) & 1, sm, err) && ok;
      if (sm.nan_tile[st] == g) {
        for (int i = 0; i < NT; ++i)
          if (k0 + i >= row.k_lo && k0 + i < row.k_hi)
            row.nan |= sm.nan_bits[st * TK + key0 + i] | sm.nan_bits[(2 + st) * TK + key0 + i];
      }
    }
    tmem_st_wait();
    warp_arrive(&sm.p_full[st], at.lane);
  }
  return ok;
}

DF_DEV float row_lse(float M, float L, const Mode& mode) {
  return L == 0.f ? -INFINITY : (M + (__log2f(L) - lift_of(mode))) * 0.6931471805599453f;
}

// A segment's rows out of TMEM, 32 channels at a time through shared memory:
// the copies of a row are merged (log-sum-exp rescaling, in order), and the
// row goes to the output, or unnormalised to the segment's partial slot.
// `have`: O holds something.
template <int COPIES>
DF_DEV void finish_segment(const Q8AttnArgs& a, const Segment& w, const Mode& mode,
                           const Shared& sm, const Place& at, bool have, const SoftmaxRow& row) {
  constexpr int RW = 128 / COPIES, N = kSoftmaxWarps * 32;
  pair_sync(at);  // (the segment before has been read)
  if (at.hh == 0) {
    sm.row_m[at.r] = row.m;
    sm.row_nan[at.r] = 0;
  }
  sm.row_l[at.hh * 128 + at.r] = row.l;
  pair_sync(at);
  if (row.nan != 0) atomicOr(sm.row_nan + at.r, row.nan);
  named_bar_sync(1, N);
  if (at.hh == 0 && at.seg == 0 && at.qr < w.rows) {
    float M = -INFINITY, L = 0.f;
    int nan = 0;
#pragma unroll
    for (int c = 0; c < COPIES; ++c) {
      M = fmaxf(M, sm.row_m[c * RW + at.qr]);
      nan |= sm.row_nan[c * RW + at.qr];
    }
    float f[COPIES];
#pragma unroll
    for (int c = 0; c < COPIES; ++c) {
      const int x = c * RW + at.qr;
      const float m = sm.row_m[x], l = sm.row_l[x] + sm.row_l[128 + x];
      f[c] = l == 0.f ? 0.f : m == M ? 1.f : fast_exp2(m - M);  // l = 0: no key seen
      if (l != 0.f) L += f[c] * l;
    }
    if (L == 0.f) nan = 0;
    if (nan & kNanK) L = nan_f();
    sm.row_nan[at.qr] = nan;
    if (w.slot >= 0) {
      __stcg(a.part_ml + (size_t)w.slot * 256 + at.qr, M);
      __stcg(a.part_ml + (size_t)w.slot * 256 + 128 + at.qr, L);
    } else if (a.lse != nullptr) {
      a.lse[out_row(a, w.b, w.h, w.qt, w.tokens, at.qr)] = row_lse(M, L, mode);
    }
    const float scale = w.slot >= 0 ? 1.f : L == 0.f ? 0.f : v_unit(mode) / L;
#pragma unroll
    for (int c = 0; c < COPIES; ++c) sm.row_f[c * RW + at.qr] = f[c] == 0.f ? 0.f : f[c] * scale;
  }
  // This thread's share of what goes out: four channels of the rows r0, r0 +
  // 32, ... in every pass.
  float* x = reinterpret_cast<float*>(sm.qx);
  constexpr int ITEMS = RW / 32;
  const int r0 = at.hh * 16 + at.quarter * 4 + (at.lane >> 3), c4 = (at.lane & 7) * 4;
  size_t to[ITEMS];
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    const int qr = r0 + i * 32;
    to[i] = qr >= w.rows ? 0
            : (w.slot >= 0 ? (size_t)w.slot * 128 + qr
                           : out_row(a, w.b, w.h, w.qt, w.tokens, qr)) * HD + c4;
  }
#pragma unroll 1
  for (int c = 0; c < HD / 32; ++c) {
    if (have) {
      float o[16];
      tmem_load<16>(at.trow + O_COL + c * 32 + at.hh * 16, o);
      float4* d = reinterpret_cast<float4*>(x + at.r * X_LD + at.hh * 16);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        d[i] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
    }
    named_bar_sync(1, N);
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      const int qr = r0 + i * 32;
      if (qr >= w.rows) continue;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
      if (have) {
#pragma unroll
        for (int k = 0; k < COPIES; ++k) {
          const float f = sm.row_f[k * RW + qr];
          const float4 y = *reinterpret_cast<const float4*>(x + (k * RW + qr) * X_LD + c4);
          if (f != 0.f) {
            o.x += f * y.x;
            o.y += f * y.y;
            o.z += f * y.z;
            o.w += f * y.w;
          }
        }
      }
      const int nan = sm.row_nan[qr];
      if (((nan >> c) & 1) || (nan & kNanK)) o.x = o.y = o.z = o.w = nan_f();
      if (w.slot >= 0)
        __stcg(reinterpret_cast<float4*>(a.part_o + to[i] + c * 32), o);
      else
        *reinterpret_cast<uint2*>(a.out + to[i] + c * 32) =
            make_uint2(pack_bf16x2(o.x, o.y), pack_bf16x2(o.z, o.w));
    }
    named_bar_sync(1, N);
  }
}

// The keys this thread's row sees in a segment.
DF_DEV SoftmaxRow begin_row(const Q8AttnArgs& a, const Segment& w, int qr) {
  const int g = qr / w.tokens, t = w.qt * a.tile_tokens + qr - g * w.tokens;
  SoftmaxRow row{a.scale, w.lo, w.hi, -INFINITY, 0.f, 0};
  const long long at = (long long)w.len - a.q_len + t;
  if (a.window > 0) {
    row.k_lo = (int)max((long long)row.k_lo, at - a.window + 1);
    row.k_hi = (int)min((long long)row.k_hi, at + a.window);
  }
  if (a.causal) row.k_hi = (int)min((long long)row.k_hi, at + 1);
  return row;
}

template <int COPIES>
DF_DEV void softmax_all(const Q8AttnArgs& a, const Q8Plan& p, const Shared& sm, uint32_t tmem,
                        int warp, int lane) {
  constexpr int RW = 128 / COPIES;
  Place at;
  at.r = (warp & 3) * 32 + lane;
  at.qr = at.r % RW;
  at.seg = at.r / RW;
  at.hh = warp >> 2;
  at.lane = lane;
  at.quarter = warp & 3;
  at.trow = tmem + ((uint32_t)((warp & 3) * 32) << 16);
  Walk walk(a, p);
  Segment w{};
  int g = 0, staged = 0;
  bool ok = true;
  // Begin a segment: its Q goes into TMEM as soon as the last S of the one
  // before has completed (its softmax has waited for it), before that one's O
  // is read out, so that the first S of the segment does not wait for it.
  Mode mode{};
  SoftmaxRow row{};
  auto begin = [&]() {
    row = begin_row(a, w, at.qr);
    if (w.t1 == w.t0) return;
    ok = warp_wait(sm.q_staged, staged & 1, sm, a.err) && ok;
    const int4 m = sm.mode[staged & 1];
    mode.half = m.x != 0;
    mode.k0 = m.y;
    mode.v0 = m.z;
    ++staged;
    load_q<COPIES>(a, w, mode, sm, at, row);
    warp_arrive(sm.q_full, lane);
  };
  bool more = walk.next(a, p, w);
  if (more) begin();
  while (more) {
    const bool have = w.t1 > w.t0;
    if (have)
      ok = (mode.half ? softmax_segment<COPIES, true>(w, sm, a.err, at, row, g)
                      : softmax_segment<COPIES, false>(w, sm, a.err, at, row, g)) && ok;
    const Segment done = w;
    const Mode done_mode = mode;
    SoftmaxRow done_row = row;
    const int last = g - 1;
    more = walk.next(a, p, w);
    if (more) begin();
    if (have) {
      ok = warp_wait(&sm.o_done[last & 1], (last >> 1) & 1, sm, a.err) && ok;
      tc_fence_after();
    }
    if (!ok) done_row.m = -INFINITY, done_row.l = 0.f;
    finish_segment<COPIES>(a, done, done_mode, sm, at, have, done_row);
    if (have) warp_arrive(sm.o_free, lane);
  }
}

template <int FMT, int COPIES>
__global__ void __launch_bounds__(kThreads, 1)
    attn_q8_kernel(const __grid_constant__ Q8AttnArgs a, const __grid_constant__ Q8Plan plan) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Shared sm;
  sm.k = smem;
  sm.v = smem + 2 * TILE;
  sm.ring = smem + 4 * TILE;
  sm.qx = sm.ring + RING * SLOT;
  sm.nan_bits = sm.qx + QX_BYTES;
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm.nan_bits + 4 * TK);
  sm.ring_full = bars;
  sm.ring_empty = bars + RING;
  sm.k_full = sm.ring_empty + RING;
  sm.v_full = sm.k_full + 2;
  sm.s_full = sm.v_full + 2;
  sm.p_full = sm.s_full + 2;
  sm.o_done = sm.p_full + 2;
  sm.q_staged = sm.o_done + 2;
  sm.q_full = sm.q_staged + 1;
  sm.o_free = sm.q_full + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm.o_free + 1);
  sm.mode = reinterpret_cast<int4*>(bars + 48);
  sm.abort = reinterpret_cast<volatile int*>(tmem_slot + 1);
  sm.nan_tile = sm.abort + 1;
  sm.pair = reinterpret_cast<float*>(bars + 64);
  sm.row_m = sm.pair + 4 * 128;
  sm.row_l = sm.row_m + 128;
  sm.row_nan = reinterpret_cast<int*>(sm.row_l + 2 * 128);
  sm.row_f = sm.row_l + 3 * 128;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
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
      sm.nan_tile[i] = -1;
    }
    mbar_init(sm.q_staged, 1);
    mbar_init(sm.q_full, kSoftmaxWarps);
    mbar_init(sm.o_free, kSoftmaxWarps);
    *sm.abort = 0;
    fence_mbar_init();
  }
  if (warp == kWarpS) {
    tmem_alloc(tmem_slot, TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  grid_dep_sync();

  if (warp < kSoftmaxWarps) {
    softmax_all<COPIES>(a, plan, sm, tmem, warp, lane);
  } else if (warp < kWarpS) {
    decode_all<FMT>(a, plan, sm, warp - kSoftmaxWarps, lane);
  } else if (warp == kWarpCopy) {
    copy_all(a, plan, sm, COPIES > 1, lane);
  } else if (lane == 0) {
    if (warp == kWarpS) issue_s(a, plan, sm, tmem);
    if (warp == kWarpPV) issue_pv(a, plan, sm, tmem);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == kWarpS) {
    tc_fence_after();
    tmem_dealloc(tmem, TMEM_COLS);
  }
}

// ---------------------------------------------------------------- merge
// Rows of pairs that lie across CTAs: one warp per query row, lane i holding
// the i-th CTA's max and sum (at most kQ8MaxSplits = 32), four channels per
// lane.  The parts are summed in order, each rescaled to the largest max: the
// result does not depend on which CTA finished when.  512 bytes per part and
// row through L2.
__global__ void __launch_bounds__(128)
    q8_merge_kernel(const __grid_constant__ Q8AttnArgs a, const __grid_constant__ Q8Plan p) {
  const int lane = threadIdx.x & 31;
  const int rows_max = a.tile_tokens * a.groups;
  const int per_seq = a.n_q_tiles * a.st.n_kv * rows_max;
  const int idx = blockIdx.x * 4 + (threadIdx.x >> 5);
  const int b = idx / per_seq;
  grid_dep_sync();
  if (b >= a.batch) return;
  const int r = idx - b * per_seq;
  const int pair = r / rows_max, qr = r - pair * rows_max;
  const int n = tiles_of(p, b), x0 = p.first[b] + pair * n;
  const int c0 = x0 / p.share, ns = (x0 + n - 1) / p.share - c0 + 1;
  if (ns == 1) return;
  const int qt = pair / a.st.n_kv, h = pair - qt * a.st.n_kv;
  const int tokens = min(a.tile_tokens, a.q_len - qt * a.tile_tokens);
  if (qr >= tokens * a.groups) return;
  // the pair is its first CTA's last segment (slot 1, unless the CTA begins
  // with it), and the others' first
  const int slot0 = 2 * c0 + (x0 % p.share != 0 ? 1 : 0);
  const int slot = lane == 0 ? slot0 : 2 * (c0 + lane);
  float m = -INFINITY, l = 0.f;
  if (lane < ns) {
    m = __ldcg(a.part_ml + (size_t)slot * 256 + qr);
    l = __ldcg(a.part_ml + (size_t)slot * 256 + 128 + qr);
  }
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
    for (int i = 0; i < 8; ++i)
      if (i0 + i < ns)
        y[i] = __ldcg(reinterpret_cast<const float4*>(
                          a.part_o + ((size_t)(i0 + i == 0 ? slot0 : 2 * (c0 + i0 + i)) * 128 +
                                      qr) * HD) + lane);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (i0 + i < ns) {
        const float fi = __shfl_sync(0xffffffffu, f, i0 + i);
        L += __shfl_sync(0xffffffffu, fl, i0 + i);
        if ((some >> (i0 + i)) & 1u) {
          o.x += fi * y[i].x;
          o.y += fi * y[i].y;
          o.z += fi * y[i].z;
          o.w += fi * y[i].w;
        }
      }
    }
  }
  const Mode mode = mode_of(a.st, b, h);
  const size_t row = out_row(a, b, h, qt, tokens, qr);
  const float s = L == 0.f ? 0.f : v_unit(mode) / L;
  *reinterpret_cast<uint2*>(a.out + row * HD + lane * 4) =
      make_uint2(pack_bf16x2(o.x * s, o.y * s), pack_bf16x2(o.z * s, o.w * s));
  if (lane == 0 && a.lse != nullptr) a.lse[row] = row_lse(M, L, mode);
}

template <int FMT>
const void* kernel_of(int copies) {
  return copies == 4   ? (const void*)attn_q8_kernel<FMT, 4>
         : copies == 2 ? (const void*)attn_q8_kernel<FMT, 2>
                       : (const void*)attn_q8_kernel<FMT, 1>;
}

cudaError_t set_attrs() {
  static std::atomic<unsigned long long> done{0};
  if (done_on_device(done)) return cudaSuccess;
  for (int copies = 1; copies <= 4; copies *= 2)
    for (const void* f : {kernel_of<Q8_E4M3>(copies), kernel_of<Q8_INT8>(copies)}) {
      const cudaError_t e =
          cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
      if (e != cudaSuccess) return e;
    }
  mark_device(done);
  return cudaSuccess;
}

template <int FMT>
cudaError_t launch_tiles(const Q8AttnArgs& a, const Q8Plan& p, unsigned ctas, cudaStream_t s) {
  const int rows = a.tile_tokens * a.groups;
  const dim3 grid(ctas), block(kThreads);
  if (rows <= 32) return launch_pdl(attn_q8_kernel<FMT, 4>, grid, block, kSmem, s, a, p);
  if (rows <= 64) return launch_pdl(attn_q8_kernel<FMT, 2>, grid, block, kSmem, s, a, p);
  return launch_pdl(attn_q8_kernel<FMT, 1>, grid, block, kSmem, s, a, p);
}

}  // namespace

size_t q8_attention_slots(int num_sms) { return (size_t)2 * num_sms; }

bool plan_q8_attention(Q8Plan& p, int batch, int n_kv, int n_q_tiles, int num_sms) {
  // one CTA per SM, equal shares of the tiles; a pair's parts are merged by
  // the lanes of a warp, so a share is at least 1/32 of the longest pair
  // (whose ends may both lie inside a share: 1/30)
  long long total = 0;
  int longest = 1;
  for (int b = 0; b < batch; ++b) {
    p.first[b] = (int)total;
    const int n = tiles_of(p, b);
    longest = std::max(longest, n);
    total += (long long)n * n_kv * n_q_tiles;
    if (total >= (1LL << 31) - 1) return false;
  }
  p.first[batch] = (int)total;
  p.share = (int)std::max<long long>((total + num_sms - 1) / num_sms,
                                     (longest + kQ8MaxSplits - 3) / (kQ8MaxSplits - 2));
  return true;
}

int launch_q8_attention(int fmt, const Q8AttnArgs& a, const Q8Plan& p, cudaStream_t s) {
  if (const cudaError_t e = set_attrs()) return e;
  const int total = p.first[a.batch];
  const unsigned ctas = (unsigned)((total - 1) / p.share + 1);
  const cudaError_t e = fmt == Q8_E4M3 ? launch_tiles<Q8_E4M3>(a, p, ctas, s)
                                       : launch_tiles<Q8_INT8>(a, p, ctas, s);
  if (e != cudaSuccess) return e;
  bool split = false;
  for (int b = 0; b < a.batch && !split; ++b) {
    const int n = tiles_of(p, b);
    // a pair lies within one CTA if its first tile's place in the share
    // leaves room for all of it; shares that are multiples of n keep it so
    split = n > 1 && (p.share % n != 0 || p.first[b] % n != 0);
  }
  if (!split) return cudaSuccess;
  const long long rows =
      (long long)a.batch * a.n_q_tiles * a.st.n_kv * a.tile_tokens * a.groups;
  return launch_pdl(q8_merge_kernel, dim3((unsigned)((rows + 3) / 4)), dim3(128), 0, s, a, p);
}

}  // namespace df
