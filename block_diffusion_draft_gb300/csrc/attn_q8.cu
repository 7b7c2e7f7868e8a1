// attn_q8.cu -- attention of the draft's block queries over an 8-bit cache
// (formats: q8.cuh) on tcgen05.
//
//   S = scale * Q K^T over the keys a row sees, O = softmax(S) V
//
// One CTA owns one work unit: a (sequence, kv head, query tile) and a range of
// its 128-key tiles.  The codes of a tile are 33 KB against the 64 KB of a
// bf16 tile, so HBM asks for a tile every 0.74 us per SM; between HBM and the
// tensor core every code has to become bf16 in shared memory.  That, not the
// MMAs (1024 cycles a tile) nor HBM, is the longest queue of an SM, so eight
// of the thirteen warps do nothing else:
//
//   warps 0-3   softmax, one TMEM lane (accumulator row) per thread
//   warps 4-11  load codes into registers (the next tile's loads are issued
//               as the current tile's registers are consumed), convert them
//               and write the bf16 K and V tiles in the tensor core's
//               128-byte-swizzled layout, three stages
//   warp 12     TMEM allocator + MMA issuer:  S(j) = Q K(j)^T, O += P(j) V(j),
//               S(j+1) issued before P(j) is waited for
//
// Shared-memory traffic is what the converters compete with the tensor core
// for, so Q and P are read from TMEM (A operands) and codes never pass
// through shared memory.  TMEM columns: S double-buffered [0, 256), O [256,
// 384), Q as bf16 pairs [384, 448); P(j) overwrites the first 64 columns of
// S(j).
//
// The MMA has 128 rows.  A query tile of at most 64 (32) rows is held two
// (four) times: copy c of a row takes the c-th 64 (32) keys of every tile as
// an online softmax of its own (its P is zero elsewhere), and the copies are
// merged at the end, so that all four softmax warps work on a short block.
//
// Rows behind the sequence's end (and before the unit's first key) decode to
// zero, so nothing stale can reach O through a zero probability.  A V group
// that reads NaN is decoded as zero too; the rows that see its key remember
// the group and return NaN in its channels, the others are untouched.
#include <algorithm>
#include <atomic>
#include <queue>
#include <vector>

#include "q8.cuh"

namespace df {
namespace {

constexpr int HD = 128;
constexpr int TK = 128;                   // keys per tile
constexpr int NST = 3;                    // K/V stages
constexpr int kConvWarps = 8;
constexpr int kThreads = (4 + kConvWarps + 1) * 32;
constexpr uint32_t TILE = TK * HD * 2;    // one bf16 tile
constexpr uint32_t HALF = TILE / 2;       // 64 channels of it
constexpr uint32_t O_COL = 256, Q_COL = 384, TMEM_COLS = 512;
constexpr int O_LD = HD + 4;              // floats per row of the output staging
constexpr size_t kSmem = 1024 + 2 * NST * TILE + NST * TK + 512 + 4 * TK * 4;
constexpr float kRescale = 8.f;           // log2 units

struct Unit {
  int b, h, qt;
  int tokens, rows;   // real block rows and query rows of the tile
  int len;
  int lo, hi;         // the unit's keys
  int t0, t1;         // its key tiles
  int ns, slot;       // units of the (sequence, tile, head); partial slot or -1
};

DF_DEV Unit unit_of(const Q8AttnArgs& a, const Q8Plan& p, int u) {
  Unit w;
  int lo = 0, hi = a.batch;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (p.unit_off[mid] <= u) lo = mid; else hi = mid;
  }
  w.b = p.order[lo];
  w.ns = p.n_split[w.b];
  const int r = u - p.unit_off[lo];
  const int pair = r / w.ns, c = r - pair * w.ns;
  w.qt = pair / a.st.n_kv;
  w.h = pair - w.qt * a.st.n_kv;
  w.slot = p.slot_off[lo] < 0 ? -1 : p.slot_off[lo] + r;
  const int tok0 = w.qt * a.tile_tokens;
  w.tokens = min(a.tile_tokens, a.q_len - tok0);
  w.rows = w.tokens * a.groups;
  w.len = p.len[w.b];
  const int first = p.lo[w.b] / TK, n = (w.len + TK - 1) / TK - first;
  w.t0 = first + (int)((long long)c * n / w.ns);
  w.t1 = first + (int)((long long)(c + 1) * n / w.ns);
  // keys any row of the query tile sees
  const int i0 = w.len - a.q_len + tok0, i1 = i0 + w.tokens - 1;
  int k0 = 0, k1 = w.len;
  if (a.window > 0) {
    k0 = (int)max(0LL, (long long)i0 - a.window + 1);
    k1 = (int)min((long long)k1, (long long)i1 + a.window);
  }
  if (a.causal) k1 = min(k1, i1 + 1);
  w.lo = max(k0, w.t0 * TK);
  w.hi = min(k1, w.t1 * TK);
  if (w.hi <= w.lo) {
    w.t1 = w.t0;
  } else {
    w.t0 = w.lo / TK;
    w.t1 = (w.hi + TK - 1) / TK;
  }
  return w;
}

// output (and log-sum-exp) row of query row qr of the tile
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

// One unit of a converter thread: the two octets of rows it owns in a tile.
// In each of its two passes a lane takes 16 codes of its row: lanes 0-3 of
// eight read the one half of an even row, lanes 4-7 the other half of the odd
// row, so that the eight 16-byte stores of a phase fall into different banks.
struct Codes {
  uint4 c[2][2];   // [octet][pass]
  uint32_t s[2];   // [octet] the row's four scale bytes
};

struct ConvLane {
  int row[2];      // row of the tile, per octet
  int half[2];     // 64-channel half, per pass
  int u4;          // 16-code unit within the half
};

DF_DEV ConvLane conv_lane(int cw, int lane) {
  ConvLane l;
  const int sub = (lane >> 2) & 1;
  for (int o = 0; o < 2; ++o) l.row[o] = cw * 16 + o * 8 + (lane >> 3) * 2 + sub;
  l.half[0] = sub;
  l.half[1] = sub ^ 1;
  l.u4 = lane & 3;
  return l;
}

DF_DEV void conv_load(Codes& x, const uint8_t* codes, const uint8_t* scales, const ConvLane& l) {
#pragma unroll
  for (int o = 0; o < 2; ++o) {
#pragma unroll
    for (int p = 0; p < 2; ++p)
      x.c[o][p] = __ldcg(reinterpret_cast<const uint4*>(codes + (size_t)l.row[o] * HD +
                                                        l.half[p] * 64 + l.u4 * 16));
    x.s[o] = __ldcg(reinterpret_cast<const uint32_t*>(scales + (size_t)l.row[o] * 4));
  }
}

// Convert and store one tile.  V: NaN groups decode to zero, their bits go to
// nan_bits[row] and the tile's tag to *nan_tile.
template <int FMT, bool V>
DF_DEV void conv_store(const Codes& x, uint8_t* tile, const ConvLane& l, int k0, int lo, int hi,
                       uint8_t* nan_bits, volatile int* nan_tile, int tag) {
#pragma unroll
  for (int o = 0; o < 2; ++o) {
    const int row = l.row[o];
    const bool live = k0 + row >= lo && k0 + row < hi;
    if (V) {
      uint32_t bits = 0;
      if (live && __vcmpeq4(x.s[o], 0xffffffffu) != 0u) {
        const uint32_t e = __vcmpeq4(x.s[o], 0xffffffffu);
        bits = (e & 1u) | ((e >> 7) & 2u) | ((e >> 14) & 4u) | ((e >> 21) & 8u);
        *nan_tile = tag;
      }
      if (l.u4 == 0) nan_bits[row] = (uint8_t)bits;
    }
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      const int half = l.half[p];
      const uint32_t byte = (x.s[o] >> ((half * 2 + (l.u4 >> 1)) * 8)) & 0xffu;
      Q8Scale s = q8_scale<FMT>(byte);
      if (!live || (V && byte == kQ8NanByte)) s = q8_zero();
      uint8_t* dst = tile + half * HALF + row * 128;
      const uint4 c = x.c[o][p];
      *reinterpret_cast<uint4*>(dst + (((2 * l.u4) ^ (row & 7)) * 16)) =
          q8_decode8<FMT>(c.x, c.y, s);
      *reinterpret_cast<uint4*>(dst + (((2 * l.u4 + 1) ^ (row & 7)) * 16)) =
          q8_decode8<FMT>(c.z, c.w, s);
    }
  }
}

template <int FMT, int COPIES>
__global__ void __launch_bounds__(kThreads, 1)
    attn_q8_kernel(const __grid_constant__ Q8AttnArgs a, const __grid_constant__ Q8Plan plan) {
  constexpr int RW = 128 / COPIES;  // rows of the query tile
  constexpr int NC = TK / COPIES;   // keys of a tile that one thread handles
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sK = smem;
  uint8_t* sV = sK + NST * TILE;
  uint8_t* nan_bits = sV + NST * TILE;  // [NST][TK]
  uint64_t* bars = reinterpret_cast<uint64_t*>(nan_bits + NST * TK);
  uint64_t* kv_full = bars;             // [NST]
  uint64_t* kv_empty = kv_full + NST;   // [NST]
  uint64_t* s_full = kv_empty + NST;    // [2]
  uint64_t* p_full = s_full + 2;        // [2]
  uint64_t* o_done = p_full + 2;        // [2]: PV(j) completes o_done[j & 1]
  uint64_t* q_full = o_done + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(q_full + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* nan_tile = abort_flag + 1;  // [NST]
  float* row_m = reinterpret_cast<float*>(bars + 64);  // [128] each
  float* row_l = row_m + 128;
  int* row_nan = reinterpret_cast<int*>(row_l + 128);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Unit w = unit_of(a, plan, blockIdx.x);
  const int T = w.t1 - w.t0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < NST; ++s) {
      mbar_init(&kv_full[s], kConvWarps);
      mbar_init(&kv_empty[s], 1);
      nan_tile[s] = -1;
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 128);
      mbar_init(&o_done[i], 1);
    }
    mbar_init(q_full, 128);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 12) {
    tmem_alloc(tmem_slot, TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  grid_dep_sync();

  if (warp >= 4 && warp < 4 + kConvWarps) {
    // ---------------------------------------------------------- converters
    const ConvLane l = conv_lane(warp - 4, lane);
    const size_t row0 = ((size_t)w.b * a.st.n_kv + w.h) * a.st.cap + (size_t)w.t0 * TK;
    const uint8_t* kc = a.st.k + row0 * HD;
    const uint8_t* vc = a.st.v + row0 * HD;
    const uint8_t* ks = a.st.ks + row0 * 4;
    const uint8_t* vs = a.st.vs + row0 * 4;
    Codes xk, xv;
    if (T > 0) {
      conv_load(xv, vc, vs, l);
      conv_load(xk, kc, ks, l);
    }
    for (int j = 0; j < T; ++j) {
      const int s = j % NST;
      if (!__all_sync(0xffffffffu,
                      mbar_wait(&kv_empty[s], ((j / NST) & 1) ^ 1, abort_flag, a.err)))
        break;
      const int k0 = (w.t0 + j) * TK;
      conv_store<FMT, true>(xv, sV + s * TILE, l, k0, w.lo, w.hi, nan_bits + s * TK,
                            nan_tile + s, j);
      if (j + 1 < T) conv_load(xv, vc + (size_t)(j + 1) * TK * HD, vs + (j + 1) * TK * 4, l);
      conv_store<FMT, false>(xk, sK + s * TILE, l, k0, w.lo, w.hi, nullptr, nullptr, j);
      if (j + 1 < T) conv_load(xk, kc + (size_t)(j + 1) * TK * HD, ks + (j + 1) * TK * 4, l);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&kv_full[s]);
    }
  } else if (warp == 12) {
    // ---------------------------------------------------------- MMA issuer
    if (lane == 0 && T > 0) {
      constexpr uint32_t idesc_s = idesc_bf16(128, TK, false);
      constexpr uint32_t idesc_o = idesc_bf16(128, HD, true);
      bool alive = mbar_wait(q_full, 0, abort_flag, a.err);
      auto issue_s = [&](int j) {
        const int s = j % NST;
        if (!mbar_wait(&kv_full[s], (j / NST) & 1, abort_flag, a.err)) return false;
        tc_fence_after();
        const uint32_t k_base = smem_u32(sK + s * TILE);
#pragma unroll
        for (int kk = 0; kk < HD / 16; ++kk)
          tc_mma_bf16_ta(tmem + (uint32_t)((j & 1) * TK), tmem + Q_COL + kk * 8,
                         sdesc_sw128(k_base + (kk >> 2) * HALF + (kk & 3) * 32, 16, 1024),
                         idesc_s, kk > 0 ? 1u : 0u);
        tc_commit(&s_full[j & 1]);
        return true;
      };
      if (alive) alive = issue_s(0);
      for (int j = 0; j < T && alive; ++j) {
        if (j + 1 < T && !issue_s(j + 1)) break;
        if (!mbar_wait(&p_full[j & 1], (j >> 1) & 1, abort_flag, a.err)) break;
        tc_fence_after();
        const int s = j % NST;
        const uint32_t v_base = smem_u32(sV + s * TILE);
#pragma unroll
        for (int kk = 0; kk < TK / 16; ++kk)
          tc_mma_bf16_ta(tmem + O_COL, tmem + (uint32_t)((j & 1) * TK) + kk * 8,
                         sdesc_sw128(v_base + kk * 16 * 128, HALF, 1024), idesc_o,
                         (j > 0 || kk > 0) ? 1u : 0u);
        tc_commit(&o_done[j & 1]);
        tc_commit(&kv_empty[s]);
      }
    }
    __syncwarp();
  } else {
    // ---------------------------------------------------------- softmax
    const int r = warp * 32 + lane;          // TMEM lane
    const int qr = r % RW, seg = r / RW;     // query row and copy
    const uint32_t trow = tmem + ((uint32_t)(warp * 32) << 16);
    const bool real = qr < w.rows;
    int k_lo = w.lo, k_hi = w.hi;
    {
      const int g = qr / w.tokens, t = w.qt * a.tile_tokens + qr - g * w.tokens;
      const long long at = (long long)w.len - a.q_len + t;
      if (a.window > 0) {
        k_lo = (int)max((long long)k_lo, at - a.window + 1);
        k_hi = (int)min((long long)k_hi, at + a.window);
      }
      if (a.causal) k_hi = (int)min((long long)k_hi, at + 1);
      // the query row as the A operand: bf16 pairs in 64 columns
      const uint4* src = reinterpret_cast<const uint4*>(
          a.q + (real ? (long long)w.b * a.q_seq + (long long)w.h * a.q_head +
                            (long long)g * a.q_group + (long long)t * a.q_tok
                      : 0));
      if (T > 0) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t x[32];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint4 y = real ? __ldcg(src + c * 8 + i) : make_uint4(0u, 0u, 0u, 0u);
            x[4 * i] = y.x;
            x[4 * i + 1] = y.y;
            x[4 * i + 2] = y.z;
            x[4 * i + 3] = y.w;
          }
          tmem_st32_nowait(trow + Q_COL + c * 32, x);
        }
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(q_full);
      }
    }
    float m_run = -INFINITY, l_run = 0.f;
    int nan_run = 0;
    bool ok = true;
    const float2 sc2 = make_float2(a.scale, a.scale);
    for (int j = 0; j < T; ++j) {
      const int sb = j & 1;
      // (the tile's barrier is complete by then; waiting on it too orders the
      // converters' NaN marks before their use here)
      if (!__all_sync(0xffffffffu,
                      mbar_wait(&s_full[sb], (j >> 1) & 1, abort_flag, a.err) &&
                          mbar_wait(&kv_full[j % NST], (j / NST) & 1, abort_flag, a.err))) {
        ok = false;
        break;
      }
      tc_fence_after();
      const uint32_t s_col = trow + sb * TK;
      const int k0 = (w.t0 + j) * TK + seg * NC;
      const bool edge = !(k0 >= k_lo && k0 + NC <= k_hi);
      // Scores of 32 keys at a time (a thread's registers hold one chunk of
      // a 128-key row, not the row): the largest first, then the
      // exponentials, so the columns are read from TMEM twice when NC > 32.
      float s[32];
      auto load = [&](int c) {
        tmem_ld32(s_col + seg * NC + c * 32, s);
        if (edge) {
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const int key = k0 + c * 32 + i;
            if (key < k_lo || key >= k_hi) s[i] = -INFINITY;
          }
        }
      };
      float tmax = -INFINITY;
#pragma unroll
      for (int c = 0; c < NC / 32; ++c) {
        load(c);
        float pm[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          pm[e] = max3f(s[e], s[e + 4], s[e + 8]);
          pm[e] = max3f(pm[e], s[e + 12], s[e + 16]);
          pm[e] = max3f(pm[e], s[e + 20], s[e + 24]);
          pm[e] = fmaxf(pm[e], s[e + 28]);
        }
        tmax = fmaxf(tmax, fmaxf(fmaxf(pm[0], pm[1]), fmaxf(pm[2], pm[3])));
      }
      tmax *= a.scale;
      float m_new = m_run, alpha = 1.f;
      bool rescale = false;
      if (m_run == -INFINITY || tmax > m_run + kRescale) m_new = fmaxf(m_run, tmax);
      if (m_new != m_run) {
        alpha = m_run == -INFINITY ? 0.f : fast_exp2(m_run - m_new);
        rescale = j > 0;
      }
      const float mm = m_new == -INFINITY ? 0.f : m_new;
      const float2 neg_m = make_float2(-mm, -mm);
      float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
      uint32_t p[NC / 2];
#pragma unroll
      for (int c = 0; c < NC / 32; ++c) {
        if (NC > 32) load(c);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          float2 e = fma_f32x2(make_float2(s[2 * i], s[2 * i + 1]), sc2, neg_m);
          e.x = fast_exp2(e.x);
          e.y = fast_exp2(e.y);
          sum[i & 1] = add_f32x2(sum[i & 1], e);
          p[c * 16 + i] = pack_bf16x2(e.x, e.y);
        }
      }
      // P: this copy's keys, zero for the others' (64 columns in all); the
      // thread has read all of its scores
#pragma unroll
      for (int c = 0; c < COPIES; ++c) {
        uint32_t x[16];
#pragma unroll
        for (int n = 0; n < NC / 32; ++n) {
#pragma unroll
          for (int i = 0; i < 16; ++i) x[i] = c == seg ? p[n * 16 + i] : 0u;
          tmem_st16_nowait(s_col + c * (NC / 2) + n * 16, x);
        }
      }
      l_run = l_run * alpha + ((sum[0].x + sum[0].y) + (sum[1].x + sum[1].y));
      m_run = m_new;
      if (nan_tile[j % NST] == j) {
        for (int i = 0; i < NC; ++i)
          if (k0 + i >= k_lo && k0 + i < k_hi)
            nan_run |= nan_bits[(j % NST) * TK + seg * NC + i];
      }
      // O is touched only to rescale it, and only then must PV(j-1) be
      // complete: having seen S(j) complete, PV(j-2) is (one thread issues
      // every MMA in order), so a parity wait on o_done is exact
      if (__any_sync(0xffffffffu, rescale)) {
        if (!__all_sync(0xffffffffu, mbar_wait(&o_done[(j - 1) & 1], ((j - 1) >> 1) & 1,
                                               abort_flag, a.err))) {
          ok = false;
          break;
        }
        tc_fence_after();
        const float f = rescale ? alpha : 1.f;
#pragma unroll
        for (int c = 0; c < HD / 32; ++c) {
          float o[32];
          tmem_ld32(trow + O_COL + c * 32, o);
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] *= f;
          tmem_st32(trow + O_COL + c * 32, o);
        }
      }
      tmem_st_wait();
      tc_fence_before();
      mbar_arrive(&p_full[sb]);
    }
    if (ok && T > 0)
      ok = __all_sync(0xffffffffu, mbar_wait(&o_done[(T - 1) & 1], ((T - 1) >> 1) & 1,
                                             abort_flag, a.err));
    tc_fence_after();
    // every MMA has read its operands: the K stages hold the rows' O now
    float* so = reinterpret_cast<float*>(sK);
    if (ok && T > 0) {
#pragma unroll
      for (int c = 0; c < HD / 32; ++c) {
        float o[32];
        tmem_ld32(trow + O_COL + c * 32, o);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          *reinterpret_cast<float4*>(so + r * O_LD + c * 32 + 4 * i) =
              make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
      }
    }
    row_m[r] = ok ? m_run : -INFINITY;
    row_l[r] = ok ? l_run : 0.f;
    row_nan[r] = nan_run;
  }

  // ------------------------------------------------------------ finish
  // every thread: merge the copies of a row (log-sum-exp rescaling), four
  // channels per item, and write the row or the unit's partial of it
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 12) tmem_dealloc(tmem, TMEM_COLS);
  const float* so = reinterpret_cast<const float*>(sK);
  for (int it = threadIdx.x; it < w.rows * (HD / 4); it += kThreads) {
    const int qr = it / (HD / 4), c4 = it - qr * (HD / 4);
    float M = -INFINITY;
    int nan = 0;
#pragma unroll
    for (int c = 0; c < COPIES; ++c) {
      M = fmaxf(M, row_m[c * RW + qr]);
      nan |= row_nan[c * RW + qr];
    }
    float L = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int c = 0; c < COPIES; ++c) {
      const int x = c * RW + qr;
      const float m = row_m[x], l = row_l[x];
      // no key seen: no weight, whatever O holds (a NaN score leaves m at
      // -inf but makes l NaN)
      if (m == -INFINITY && l == 0.f) continue;
      const float f = m == M ? 1.f : fast_exp2(m - M);
      const float4 y = *reinterpret_cast<const float4*>(so + x * O_LD + c4 * 4);
      L += f * l;
      o.x += f * y.x;
      o.y += f * y.y;
      o.z += f * y.z;
      o.w += f * y.w;
    }
    if ((nan >> (c4 / 8)) & 1) o.x = o.y = o.z = o.w = __int_as_float(0x7fffffff);
    if (w.slot >= 0) {
      __stcg(reinterpret_cast<float4*>(a.part_o + ((size_t)w.slot * 128 + qr) * HD) + c4, o);
      if (c4 == 0) {
        __stcg(a.part_ml + (size_t)w.slot * 256 + qr, M);
        __stcg(a.part_ml + (size_t)w.slot * 256 + 128 + qr, L);
      }
    } else {
      const size_t row = out_row(a, w.b, w.h, w.qt, w.tokens, qr);
      const float inv = L == 0.f ? 0.f : 1.f / L;
      *reinterpret_cast<uint2*>(a.out + row * HD + c4 * 4) =
          make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
      if (c4 == 0 && a.lse != nullptr)
        a.lse[row] = L == 0.f ? -INFINITY : (M + __log2f(L)) * 0.6931471805599453f;
    }
  }
}

// ---------------------------------------------------------------- merge
// Split rows: one warp per query row, lane i holding split i's max and sum
// (at most 32 splits), four channels per lane.  The splits are summed in
// order, each rescaled to the largest max: the result does not depend on
// which unit finished when.  512 bytes per split and row through L2.
__global__ void __launch_bounds__(128)
    q8_merge_kernel(const __grid_constant__ Q8AttnArgs a, const __grid_constant__ Q8Plan p) {
  const int lane = threadIdx.x & 31;
  const int rows_max = a.tile_tokens * a.groups;
  const int per_seq = a.n_q_tiles * a.st.n_kv * rows_max;
  const int idx = blockIdx.x * 4 + (threadIdx.x >> 5);
  const int i = idx / per_seq;
  grid_dep_sync();
  if (i >= a.batch || p.slot_off[i] < 0) return;
  const int r = idx - i * per_seq;
  const int pair = r / rows_max, qr = r - pair * rows_max;
  const int qt = pair / a.st.n_kv, h = pair - qt * a.st.n_kv;
  const int b = p.order[i], ns = p.n_split[b];
  const int tokens = min(a.tile_tokens, a.q_len - qt * a.tile_tokens);
  if (qr >= tokens * a.groups) return;
  const size_t slot0 = (size_t)p.slot_off[i] + (size_t)pair * ns;
  float m = -INFINITY, l = 0.f;
  if (lane < ns) {
    m = __ldcg(a.part_ml + (slot0 + lane) * 256 + qr);
    l = __ldcg(a.part_ml + (slot0 + lane) * 256 + 128 + qr);
  }
  float M = m;
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, d));
  const bool none = m == -INFINITY && l == 0.f;
  const float f = none ? 0.f : (m == M ? 1.f : fast_exp2(m - M));
  const float fl = none ? 0.f : f * l;
  float L = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  const float4* src = reinterpret_cast<const float4*>(a.part_o + (slot0 * 128 + qr) * HD) + lane;
  for (int c0 = 0; c0 < ns; c0 += 8) {
    float4 y[8];
#pragma unroll
    for (int c = 0; c < 8; ++c)
      if (c0 + c < ns) y[c] = __ldcg(src + (size_t)(c0 + c) * 128 * (HD / 4));
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      if (c0 + c < ns) {
        const float fc = __shfl_sync(0xffffffffu, f, c0 + c);
        L += __shfl_sync(0xffffffffu, fl, c0 + c);
        if (!__shfl_sync(0xffffffffu, (int)none, c0 + c)) {
          o.x += fc * y[c].x;
          o.y += fc * y[c].y;
          o.z += fc * y[c].z;
          o.w += fc * y[c].w;
        }
      }
    }
  }
  const size_t row = out_row(a, b, h, qt, tokens, qr);
  const float inv = L == 0.f ? 0.f : 1.f / L;
  *reinterpret_cast<uint2*>(a.out + row * HD + lane * 4) =
      make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
  if (lane == 0 && a.lse != nullptr)
    a.lse[row] = L == 0.f ? -INFINITY : (M + __log2f(L)) * 0.6931471805599453f;
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
cudaError_t launch_units(const Q8AttnArgs& a, const Q8Plan& p, int units, cudaStream_t s) {
  const int rows = a.tile_tokens * a.groups;
  const dim3 grid(units), block(kThreads);
  if (rows <= 32) return launch_pdl(attn_q8_kernel<FMT, 4>, grid, block, kSmem, s, a, p);
  if (rows <= 64) return launch_pdl(attn_q8_kernel<FMT, 2>, grid, block, kSmem, s, a, p);
  return launch_pdl(attn_q8_kernel<FMT, 1>, grid, block, kSmem, s, a, p);
}

}  // namespace

size_t q8_attention_slots(int num_sms) { return (size_t)4 * num_sms; }

void plan_q8_attention(Q8Plan& p, int batch, int n_kv, int n_q_tiles, int num_sms) {
  // Units of at most U tiles for about m = 1..4 units per SM, dispatched
  // largest first.  A unit costs its tiles plus about two for its start, and
  // one more when its rows are merged afterwards; list scheduling gives the
  // makespan of each m, and the smallest one is taken.
  const int pairs = n_kv * n_q_tiles;
  std::vector<int> np(batch), ns(batch), best(batch, 1);
  long long total = 0;
  for (int b = 0; b < batch; ++b) {
    np[b] = std::max(1, (p.len[b] + TK - 1) / TK - p.lo[b] / TK);
    total += (long long)pairs * np[b];
  }
  const long long slots = (long long)q8_attention_slots(num_sms);
  double best_t = 1e300;
  for (int m = 0; m <= 4; ++m) {
    // m = 0: no splits
    const long long share = (long long)m * num_sms;
    const long long U = m == 0 ? (1LL << 40) : std::max<long long>(1, (total + share - 1) / share);
    long long split_units = 0;
    for (int b = 0; b < batch; ++b) {
      ns[b] = (int)std::min<long long>({(np[b] + U - 1) / U, (long long)np[b],
                                        (long long)kQ8MaxSplits});
      if (ns[b] > 1) split_units += (long long)pairs * ns[b];
    }
    if (split_units > slots) continue;
    std::vector<std::pair<double, int>> cost(batch);
    for (int b = 0; b < batch; ++b)
      cost[b] = {(double)((np[b] + ns[b] - 1) / ns[b]) + 2.0 + (ns[b] > 1 ? 1.0 : 0.0), b};
    std::sort(cost.begin(), cost.end(), [](const auto& x, const auto& y) {
      return x.first > y.first || (x.first == y.first && x.second < y.second);
    });
    std::priority_queue<double, std::vector<double>, std::greater<double>> load;
    for (int i = 0; i < num_sms; ++i) load.push(0.0);
    double t = split_units > 0 ? 3.0 : 0.0;  // the merge kernel
    double end = 0.0;
    for (const auto& c : cost)
      for (int i = 0; i < pairs * ns[c.second]; ++i) {
        const double l = load.top() + c.first;
        load.pop();
        load.push(l);
        end = std::max(end, l);
      }
    t += end;
    if (t < best_t - 1e-9) {
      best_t = t;
      best = ns;
    }
  }
  std::vector<std::pair<double, int>> order(batch);
  for (int b = 0; b < batch; ++b) {
    p.n_split[b] = best[b];
    order[b] = {(double)np[b] / best[b], b};
  }
  std::sort(order.begin(), order.end(), [](const auto& x, const auto& y) {
    return x.first > y.first || (x.first == y.first && x.second < y.second);
  });
  p.unit_off[0] = 0;
  int slot = 0;
  for (int i = 0; i < batch; ++i) {
    const int b = order[i].second, units = pairs * p.n_split[b];
    p.order[i] = b;
    p.unit_off[i + 1] = p.unit_off[i] + units;
    p.slot_off[i] = p.n_split[b] > 1 ? slot : -1;
    if (p.n_split[b] > 1) slot += units;
  }
}

int launch_q8_attention(int fmt, const Q8AttnArgs& a, const Q8Plan& p, cudaStream_t s) {
  if (const cudaError_t e = set_attrs()) return e;
  const int units = p.unit_off[a.batch];
  const cudaError_t e = fmt == Q8_E4M3 ? launch_units<Q8_E4M3>(a, p, units, s)
                                       : launch_units<Q8_INT8>(a, p, units, s);
  if (e != cudaSuccess) return e;
  bool split = false;
  for (int i = 0; i < a.batch; ++i) split = split || p.slot_off[i] >= 0;
  if (!split) return cudaSuccess;
  const long long rows =
      (long long)a.batch * a.n_q_tiles * a.st.n_kv * a.tile_tokens * a.groups;
  return launch_pdl(q8_merge_kernel, dim3((unsigned)((rows + 3) / 4)), dim3(128), 0, s, a, p);
}

}  // namespace df
