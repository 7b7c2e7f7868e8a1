// linear_ce.cu -- cross entropy of a linear head over a large vocabulary,
// and its gradients, without the logits of more than a piece of it.
//
//   z = x w^T,  nll = logsumexp(z) - z_t,
//   dx = d * (sum_v p_v w_v - w_t),  dw_v = sum_rows d * (p_v - [v = t]) * x.
//
// Rows without a target are taken out first (compact, gather), so that they
// cost nothing and nothing of theirs reaches a sum.  One GEMM kernel with
// different operand layouts and epilogues does the products:
//   LSE   x w^T of all columns; per row and 128 columns the largest logit and
//         the sum of exponentials relative to it
//   EXP   x w^T of one piece of columns; e = 2^(z log2 e - ref) in bf16 with a
//         reference per row, and their sums
//   ACC   sum_v e_v w_v of the piece, added to an fp32 buffer
//   GRAD  x w^T of one piece again, now with the row's lse known:
//         d * (p - [v = t]) in bf16
//   OUT   its transpose times x: dw's rows of the piece
// The exponentials need no row maximum: a sum of products is linear in them,
// so dx needs the logits once (EXP, ACC: 4 N V H operations) and is divided by
// the row's sum at the end.  The reference is the target's logit; a row in
// whose piece an exponential relative to it would be above 2^80 (a logit 80 ln 2
// above it) is done again with its largest logit: a second launch of EXP, which
// ends at once otherwise (6 us) and looks at every row tile where one row of the
// piece needs it (2048 rows x 64000 with dx: 1.33 ms, 1.81 with one such row, 2.10
// with one in every tile).
// Where the whole vocabulary is one piece, GRAD's product is saved: EXP keeps 8
// more bits of every exponential, which scaled by the row's sum and rounded to
// bf16 once are what GRAD computes (2048 rows x 64000, hidden 4096, with dw: 2.58
// -> 2.08 ms).
//
// The target's column is left out of every sum of exponentials and added
// where the results are written: 1 - p_t is then a quotient of sums without
// cancellation, also for a row that is sure of its target.
//
// The tensor cores bound it with many rows, one read of w for each product with
// few.  A pair of CTAs (cta_group::2) shares a tile of 256 rows x 256 columns:
// each CTA stages 128 rows of either operand, 64 bytes a clock for 4096
// multiply-adds, half of what a CTA with a tile of 128 x 256 of its own stages.
// One persistent pair per two SMs; a warp issues copies, a warp MMAs, eight read
// the accumulator, of which there are two, so that a tile's epilogue runs
// beside the next one's products.  Up to 128 rows a CTA has a tile of its own
// (the padding to 256 would cost more MMA time than the read of w).
// Finer row tiles of a pair gain little: one of 192 rows took 90% of a whole one's
// time, with the rows as either operand.
// Measured (hidden 4096): 4096 rows x 150000 with dx 5.4 to 6.1 ms, 1.87 to 1.65
// PFLOP/s by what the power limit leaves; 2048 x 38912: EXP 345 us, ACC 348, OUT
// 331, tensor pipe 86 to 89% active; 16 rows x 150000, forward: 185 us, 6.6 TB/s.
#include <algorithm>

#include "../../include/dflash_attn.h"
#include "handles.h"
#include "internal.h"
#include "ptx.cuh"

namespace df {
namespace {

constexpr int BM = 128, BN = 256, BK = 64;
constexpr int kEpiWarps = 8;   // two for each quarter of TMEM's lanes, 128 columns each
constexpr int kThreads = 64 + 32 * kEpiWarps;  // and the producer's and the MMA's warp
constexpr int HN = BN / 2;     // columns of an epilogue warp, and of the sums that it writes
constexpr uint32_t A_BYTES = BM * BK * 2;
constexpr uint32_t SLAB = 4096;  // 32 rows of 128 bytes: what a warp stores at a time
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kNegInf = -__builtin_huge_valf();
// Binades that a logit may lie above its row's reference: 2^24 such exponentials,
// and their products with weights below 2^20, stay in fp32's range.
constexpr float kRefSlack = 80.f;

// The factor of a row's own target, -d (1 - p_t), is by far the largest of its
// column, so what its rounding to bf16 changes is most of dw's error beyond the
// last rounding.  A column that is one row's target (own = kOwnOne + row) is
// multiplied by what that rounding took away, which puts it back exactly; the
// other factors of the column move by no more than their own rounding.
constexpr unsigned long long kOwnOne = 1ull << 40;

enum Epi { LSE = 0, EXP = 1, GRAD = 2, ACC = 3, OUT = 4 };

// CG CTAs work on one tile of CG * 128 rows and 256 columns.  Shared memory
// holds the ring and the slabs of ACC's epilogue, which adds by bulk copies (the
// others store from registers: without fences and waits for slabs OUT's short
// tiles are 6% faster).
template <int EPI, int CG>
struct Geo {
  static constexpr uint32_t B_BYTES = BN / CG * BK * 2;
  static constexpr uint32_t STAGE = A_BYTES + B_BYTES;
  static constexpr uint32_t SLABS = EPI == ACC ? kEpiWarps * SLAB : 0;
  static constexpr size_t FIXED = 1024 + SLABS + 256;
  static constexpr int STAGES = (int)((232448 - FIXED) / STAGE);
  static constexpr size_t SMEM = FIXED + STAGES * STAGE;
};

struct CeGemm {
  const int* n_rows;   // device: rows with a target
  int m_tiles;         // OUT: tiles of the piece's columns
  int n_tiles, n_kb, splits;
  Divisor by_group;    // kGroup * n_tiles
  int v0;              // first column of the piece
  int vocab, hidden;
  int rows_pad;
  uint8_t* g;          // EXP, GRAD: [rows_pad][g_pitch] bf16
  uint8_t* low;        // EXP: null, or [rows_pad][g_pitch] the exponentials' next 8 bits
  int g_pitch;
  const float* ref2;   // EXP: the rows' references before the piece; GRAD: their lse, log2 units
  float* raised;       // EXP: [pieces left][rows_pad] references after the piece and later ones
  int pieces_left;     // this one included
  const int* target;
  const float* d;      // GRAD, OUT: gradients of the rows' nll
  const float* miss;   // GRAD, OUT: 1 - p_t
  const unsigned long long* own;  // OUT: [vocab] rows with this target (see kOwnOne)
  float* part_m;       // [rows_pad][parts], log2 units: of 128 columns each
  float* part_s;
  int parts;
  int* any;            // EXP: whether a reference was raised
  int repair;          // EXP: only the row tiles with a raised reference, with that
  int add;             // ACC: the buffer holds earlier pieces
  float* acc;          // repair: [splits][rows_pad][acc_pitch] earlier pieces' products, or null
  int acc_pitch, acc_slices;
  __nv_bfloat16* dw;   // OUT: [vocab][hidden]
  float* nll;          // GRAD, OUT: [all_rows] where a wait that ran out leaves NaN (the kernels
  float* lse;          // before them leave it to the one that writes nll)
  int all_rows;
  int* err;
};

// ------------------------------------------------------------ PTX for pairs
template <int CG>
DF_DEV void tmem_alloc_cg(uint32_t* dst, uint32_t cols) {
  if (CG == 1) {
    tmem_alloc(dst, cols);
    tmem_relinquish();
  } else {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(dst)),
                 "r"(cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
}

template <int CG>
DF_DEV void tmem_dealloc_cg(uint32_t t, uint32_t cols) {
  if (CG == 1)
    tmem_dealloc(t, cols);
  else
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(t), "r"(cols)
                 : "memory");
}

// A box into this CTA's shared memory; its bytes are counted on the barrier at
// shared::cluster address `bar` (with pairs: the first CTA's).
template <int CG>
DF_DEV void load_box(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y) {
  if (CG == 1)
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(bar)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes."
        "cta_group::2 [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(bar)
        : "memory");
}

template <int CG>
DF_DEV void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  if (CG == 1)
    tc_mma_bf16(d, a, b, idesc, acc);
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}

// one arrival on `bar` (with pairs: in both CTAs) once all MMAs so far are done
template <int CG>
DF_DEV void commit(uint64_t* bar) {
  if (CG == 1)
    tc_commit(bar);
  else
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster."
        "b64 [%0], %1;" ::"r"(smem_u32(bar)),
        "h"((uint16_t)3)
        : "memory");
}

// Arrival on another CTA's barrier that hands over tensor memory alone, ordered
// by the tcgen05 fence before it: a release would wait for the epilogue's stores
// to global memory first.
DF_DEV void arrive_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar)
               : "memory");
}

DF_DEV void store_box(const CUtensorMap* map, const void* src, int x, int y) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::
                   "l"(map),
               "r"(x), "r"(y), "r"(smem_u32(src))
               : "memory");
}

DF_DEV void add_box(const CUtensorMap* map, const void* src, int x, int y) {
  asm volatile(
      "cp.reduce.async.bulk.tensor.2d.global.shared::cta.add.tile.bulk_group [%0, {%1, %2}], "
      "[%3];" ::"l"(map),
      "r"(x), "r"(y), "r"(smem_u32(src))
      : "memory");
}

DF_DEV void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
template <int N>
DF_DEV void bulk_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}
DF_DEV void bulk_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// 32 fp32 columns of this thread's TMEM lane: the load, and the wait, through
// which the values go so that no use of them comes before it
DF_DEV void tmem_wait32(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                 "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                 "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]),
                 "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                 "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]),
                 "+r"(r[30]), "+r"(r[31])::"memory");
}

// D fp32, A and B bf16, K-major or MN-major each
constexpr uint32_t idesc_ce(int m, int n, bool a_mn, bool b_mn) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((a_mn ? 1u : 0u) << 15) |
         ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

// ------------------------------------------------------------------- GEMM
struct Tile {
  int m, n, split, k0, k1;
};

// Tiles in groups of 8 row tiles, column tiles outside: the CTAs that run at
// the same time share their operands in L2.
constexpr int kGroup = 8;

DF_DEV Tile tile_at(const CeGemm& p, int m_tiles, int n_kb, int u) {
  Tile t;
  t.split = 0, t.k0 = 0, t.k1 = n_kb;
  if (p.splits > 1) {
    const int per_split = m_tiles * p.n_tiles;
    t.split = u / per_split;
    u -= t.split * per_split;
    t.k0 = n_kb * t.split / p.splits;
    t.k1 = n_kb * (t.split + 1) / p.splits;
  }
  const int g = p.by_group.quotient(u), left = m_tiles - g * kGroup;
  const int rem = u - g * p.by_group.d;
  t.n = left >= kGroup ? rem / kGroup : rem / left;
  t.m = g * kGroup + rem - t.n * min(left, kGroup);
  return t;
}

// Whether a repair has to compute this row tile again: one of its rows has
// another reference than before.  For a whole warp or for one thread.
template <int CG>
DF_DEV bool raised(const CeGemm& p, const Tile& t, int first, int step) {
  bool any = false;
  for (int i = first; i < CG * BM; i += step) {
    const int row = t.m * CG * BM + i;
    any |= row < __ldcg(p.n_rows) && __ldcg(p.raised + row) != __ldcg(p.ref2 + row);
  }
  return any;
}

// A logit far above the row's reference: it becomes the reference of this
// piece's repair and of all pieces behind it (the largest such one, whatever the
// order).
DF_DEV void raise(const CeGemm& p, int row, float top) {
  for (int i = 0; i < p.pieces_left; ++i) {
    int* at = reinterpret_cast<int*>(p.raised + (size_t)i * p.rows_pad + row);
    int old = *reinterpret_cast<volatile int*>(at);
    while (__int_as_float(old) < top) {
      const int seen = atomicCAS(at, old, __float_as_int(top));
      if (seen == old) break;
      old = seen;
    }
  }
  *p.any = 1;  // (every writer stores the same)
}

// A pair's last row tile of at most 128 rows is half a tile: each CTA takes 64
// rows, of which the tensor memory's lanes 0-63 hold columns 0-127 of the tile
// and lanes 64-127 the others.  The MMA takes as long as a whole tile's, with less
// power; copies and epilogue are half.
template <int EPI, int CG>
DF_DEV bool half_tile(const Tile& t, int rows) {
  return CG == 2 && EPI != OUT && rows - t.m * CG * BM <= BM;
}

// What a warp stores by bulk copies goes through a slab of 4 KB of its own, in
// the layout of the 128-byte swizzle: 16-byte chunk c of row r at place
// c ^ (r % 8).  It is filled once the copy that last read it has.
DF_DEV void slab_begin(int lane) {
  if (lane == 0) bulk_wait_read<0>();
  __syncwarp();
}

// 32 bytes: a whole sector
DF_DEV void store32(void* p, const uint32_t (&v)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]),
               "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

DF_DEV void slab_put(uint8_t* slab, int lane, int chunk, uint4 v) {
  *reinterpret_cast<uint4*>(slab + lane * 128 + ((chunk ^ (lane & 7)) << 4)) = v;
}

template <int EPI, int CG>
__global__ void __launch_bounds__(kThreads, 1)
    ce_gemm_kernel(const __grid_constant__ CUtensorMap tm_a,
                   const __grid_constant__ CUtensorMap tm_a64,  // the same in boxes of 64 rows
                   const __grid_constant__ CUtensorMap tm_b,
                   const __grid_constant__ CUtensorMap tm_out,  // ACC
                   const __grid_constant__ CeGemm p) {
  using G = Geo<EPI, CG>;
  constexpr bool kAmn = EPI == OUT, kBmn = EPI == ACC || EPI == OUT;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* slabs = smem + G::STAGES * G::STAGE;
  uint64_t* full = reinterpret_cast<uint64_t*>(slabs + G::SLABS);
  uint64_t* empty = full + G::STAGES;
  uint64_t* acc_full = empty + G::STAGES;  // [2]
  uint64_t* acc_empty = acc_full + 2;      // [2]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acc_empty + 2);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = CG == 2 ? (int)(blockIdx.x & 1) : 0;
  const int first = blockIdx.x / CG, stride = gridDim.x / CG;

  if (threadIdx.x == 0) {
    for (int s = 0; s < G::STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], kEpiWarps * CG);
    }
    *abort_flag = 0;
    fence_mbar_init();
    prefetch_tmap(&tm_a);
    prefetch_tmap(&tm_a64);
    prefetch_tmap(&tm_b);
    prefetch_tmap(&tm_out);
  }
  if (warp == 1) tmem_alloc_cg<CG>(tmem_slot, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (CG == 2) cluster_sync();
  const uint32_t tmem = *tmem_slot;
  grid_dep_sync();
  const bool repair = EPI == EXP && p.repair != 0;
  const int rows = repair && __ldcg(p.any) == 0 ? 0 : __ldcg(p.n_rows);
  const int m_tiles = EPI == OUT ? p.m_tiles : (rows + CG * BM - 1) / (CG * BM);
  const int n_kb = EPI == OUT ? (rows + BK - 1) / BK : p.n_kb;
  const int units = m_tiles * p.n_tiles * p.splits;

  if (warp == 0) {
    if (lane == 0) {
      uint32_t s = 0, ph = 0;
      bool alive = true;
      for (int u = first; alive && u < units; u += stride) {
        const Tile t = tile_at(p, m_tiles, n_kb, u);
        if (repair && !raised<CG>(p, t, 0, 1)) continue;
        const bool small = half_tile<EPI, CG>(t, rows);
        const int m0 = t.m * CG * BM + rank * (small ? BM / 2 : BM), n0 = t.n * BN + rank * (BN / CG);
        for (int kb = t.k0; kb < t.k1; ++kb) {
          if (!mbar_wait(&empty[s], ph ^ 1, abort_flag, p.err)) {
            alive = false;
            break;
          }
          // (the first CTA's barrier counts the bytes of both)
          if (rank == 0)
            mbar_arrive_expect_tx(&full[s], CG * (G::STAGE - (small ? A_BYTES / 2 : 0)));
          const uint32_t bar =
              CG == 2 ? cluster_map(smem_u32(&full[s]), 0) : smem_u32(&full[s]);
          const uint32_t a = smem_u32(smem + s * G::STAGE), b = a + A_BYTES;
          if (kAmn) {
#pragma unroll
            for (int i = 0; i < BM / 64; ++i)
              load_box<CG>(a + i * 8192, &tm_a, bar, m0 + 64 * i, kb * BK);
          } else {
            load_box<CG>(a, small ? &tm_a64 : &tm_a, bar, kb * BK, m0);
          }
          if (kBmn) {
#pragma unroll
            for (int i = 0; i < BN / CG / 64; ++i)
              load_box<CG>(b + i * 8192, &tm_b, bar, n0 + 64 * i,
                           (EPI == ACC ? p.v0 : 0) + kb * BK);
          } else {
            load_box<CG>(b, &tm_b, bar, kb * BK, p.v0 + n0);
          }
          if (++s == (uint32_t)G::STAGES) s = 0, ph ^= 1;
        }
      }
    }
  } else if (warp == 1) {
    if (lane == 0 && rank == 0) {
      uint32_t s = 0, ph = 0, tc = 0;
      bool alive = true;
      for (int u = first; alive && u < units; u += stride) {
        const Tile t = tile_at(p, m_tiles, n_kb, u);
        if (t.k0 >= t.k1 || (repair && !raised<CG>(p, t, 0, 1))) continue;
        const uint32_t buf = tc & 1, use = tc >> 1;
        ++tc;
        if (!mbar_wait(&acc_empty[buf], (use & 1) ^ 1, abort_flag, p.err)) break;
        tc_fence_after();
        const uint32_t idesc = half_tile<EPI, CG>(t, rows) ? idesc_ce(BM, BN, kAmn, kBmn)
                                                           : idesc_ce(CG * BM, BN, kAmn, kBmn);
        const uint32_t d = tmem + buf * BN;
        for (int kb = t.k0; kb < t.k1; ++kb) {
          if (!mbar_wait(&full[s], ph, abort_flag, p.err)) {
            alive = false;
            break;
          }
          tc_fence_after();
          const uint32_t a = smem_u32(smem + s * G::STAGE), b = a + A_BYTES;
          const uint64_t da = kAmn ? sdesc_sw128(a, 8192, 1024) : sdesc_sw128(a, 16, 1024);
          const uint64_t db = kBmn ? sdesc_sw128(b, 8192, 1024) : sdesc_sw128(b, 16, 1024);
          // a K step of 16: 2 groups of 8 rows, or 32 bytes of every row
#pragma unroll
          for (int kk = 0; kk < BK / 16; ++kk)
            mma<CG>(d, da + (uint64_t)(kk * (kAmn ? 2048 : 32) >> 4),
                    db + (uint64_t)(kk * (kBmn ? 2048 : 32) >> 4), idesc,
                    (kb > t.k0 || kk > 0) ? 1u : 0u);
          commit<CG>(&empty[s]);
          if (++s == (uint32_t)G::STAGES) s = 0, ph ^= 1;
        }
        commit<CG>(&acc_full[buf]);
      }
    }
  } else {
    const int q = warp & 3, half = (warp - 2) >> 2;
    uint8_t* slab = slabs + (warp - 2) * SLAB;
    // a row's part of an epilogue that looks at logits; the next tile's is
    // read before this one's logits are waited for
    struct Row {
      int tgt = -1;
      float ref = 0.f, sc = 0.f, miss = 0.f;
    };
    auto first_row = [&](const Tile& t) {  // of this warp
      return half_tile<EPI, CG>(t, rows) ? t.m * CG * BM + rank * (BM / 2) + (q & 1) * 32
                                         : (t.m * CG + rank) * BM + q * 32;
    };
    auto row_of = [&](const Tile& t) {
      Row r;
      const int row = first_row(t) + lane;
      if (EPI == OUT) {  // (here a row is a column of the vocabulary)
        r.sc = 1.f;
        if (p.v0 + row < p.vocab) {
          const unsigned long long own = __ldcg(p.own + p.v0 + row);
          if (own >= kOwnOne && own < 2 * kOwnOne) {
            const int c = (int)(own - kOwnOne);
            const float g = __ldcg(p.d + c) * __ldcg(p.miss + c);
            const float rounded = __bfloat162float(__float2bfloat16(g));
            if (rounded != 0.f) r.sc = g / rounded;
          }
        }
      }
      if (EPI <= GRAD && row < rows) {
        r.tgt = __ldcg(p.target + row);
        if (EPI != LSE) r.ref = __ldcg((repair ? p.raised : p.ref2) + row);
        if (EPI == GRAD) {
          r.sc = __ldcg(p.d + row);
          r.miss = __ldcg(p.miss + row);
        }
      }
      return r;
    };
    if (repair && rows > 0 && p.acc != nullptr) {
      // what the rows hold of earlier pieces follows their references
      const int warps = gridDim.x * kEpiWarps;
      for (int r = blockIdx.x * kEpiWarps + warp - 2; r < rows; r += warps) {
        const float was = __ldcg(p.ref2 + r), now = __ldcg(p.raised + r);
        if (was == now) continue;
        const float f = fast_exp2(was - now);
        for (int s = 0; s < p.acc_slices; ++s) {
          float* v = p.acc + ((size_t)s * p.rows_pad + r) * p.acc_pitch;
          for (int i = lane; i < p.acc_pitch; i += 32) v[i] *= f;
        }
      }
    }
    uint32_t tc = 0;
    Tile next{};
    Row next_row;
    if (first < units) {
      next = tile_at(p, m_tiles, n_kb, first);
      next_row = row_of(next);
    }
    for (int u = first; u < units; u += stride) {
      const Tile t = next;
      const Row mine = next_row;
      if (u + stride < units) {
        next = tile_at(p, m_tiles, n_kb, u + stride);
        next_row = row_of(next);
      }
      if (repair && !__any_sync(0xffffffffu, raised<CG>(p, t, lane, 32))) continue;
      const bool any = t.k0 < t.k1;  // otherwise the tile is zero
      const bool small = half_tile<EPI, CG>(t, rows);
      const int row0 = first_row(t), row = row0 + lane;
      const bool live = EPI == ACC || EPI == OUT || row < rows;
      const int x0 = t.n * BN + (small ? q >> 1 : half) * HN;  // first column of this warp
      const int cols = p.vocab - p.v0 - x0;  // logits: columns that exist
      const int tgt = mine.tgt - p.v0 - x0;  // the target's among them
      const float sc = mine.sc, miss = mine.miss;
      float ref = mine.ref;
      const uint32_t buf = tc & 1, use = tc >> 1;
      if (any) {
        ++tc;
        if (!__all_sync(0xffffffffu, mbar_wait(&acc_full[buf], use & 1, abort_flag, p.err)))
          break;
        tc_fence_after();
      }
      if (small && half) {  // the other four warps have all of it
        __syncwarp();
        if (any && lane == 0) arrive_cluster(cluster_map(smem_u32(&acc_empty[buf]), 0));
        continue;
      }
      const uint32_t trow =
          tmem + ((uint32_t)(q * 32) << 16) + buf * BN + (small ? 0 : half * HN);
      float mx = kNegInf, sum = 0.f;
#pragma unroll 1
      for (int c = 0; c < HN / 32; ++c) {
        float v[32];
        if (any) {
          uint32_t raw[32];
          tmem_ld32_nowait(trow + c * 32, raw);
          tmem_wait32(raw);
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(raw[i]);
          if (c == HN / 32 - 1) {  // read: back to the MMA warp
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
              if (CG == 2) arrive_cluster(cluster_map(smem_u32(&acc_empty[buf]), 0));
              else mbar_arrive(&acc_empty[buf]);
            }
          }
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = 0.f;
        }
        if (EPI <= GRAD) {
          // logits of the target and of columns that do not exist: -inf
          const bool has = tgt >= c * 32 && tgt < c * 32 + 32;
          if (c * 32 + 32 > cols || __any_sync(0xffffffffu, has)) {
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (c * 32 + i >= cols || c * 32 + i == tgt) v[i] = kNegInf;
          }
          if (EPI != GRAD) {
            float m[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
            for (int i = 4; i < 32; ++i) m[i & 3] = fmaxf(m[i & 3], v[i]);
            const float top = fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3])) * kLog2e;
            if (EPI == LSE) {
              const float now = fmaxf(mx, top);
              if (now > kNegInf) sum *= fast_exp2(mx - now);
              ref = now > kNegInf ? now : 0.f;
            }
            mx = fmaxf(mx, top);
          }
          float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            v[i] = fast_exp2(fmaf(v[i], kLog2e, -ref));
            if (EPI != GRAD) s[i & 3] += v[i];
          }
          sum += (s[0] + s[1]) + (s[2] + s[3]);
          if (EPI == LSE) continue;
          if (EPI == GRAD) {
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] *= sc;
            if (__any_sync(0xffffffffu, has)) {
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (c * 32 + i == tgt) v[i] = -sc * miss;
            }
          }
          if (!live) {
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = 0.f;
          }
        }
        if (EPI == EXP || EPI == GRAD) {
          const size_t at = (size_t)row * p.g_pitch + x0 + c * 32;
          if (EPI == EXP && p.low != nullptr) {
            // 24 bits of every number: rounded there, the upper 16 rounded from
            // those to a bf16 number, and the byte below as what is left (a
            // signed number: carries are in the upper ones)
            uint32_t lo[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              uint32_t b[4];
#pragma unroll
              for (int i = 0; i < 4; ++i) b[i] = __float_as_uint(v[4 * j + i]) + 0x80u;
              lo[j] = __byte_perm(__byte_perm(b[0], b[1], 0x0051), __byte_perm(b[2], b[3], 0x0051),
                                  0x5410);
#pragma unroll
              for (int i = 0; i < 4; ++i) v[4 * j + i] = __uint_as_float(b[i] + 0x8000u);
            }
            store32(p.low + at, lo);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              uint32_t h[8];
#pragma unroll
              for (int i = 0; i < 8; ++i)
                h[i] = __byte_perm(__float_as_uint(v[16 * k + 2 * i]),
                                   __float_as_uint(v[16 * k + 2 * i + 1]), 0x7632);
              store32(p.g + 2 * at + 32 * k, h);
            }
          } else {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              uint32_t h[8];
#pragma unroll
              for (int i = 0; i < 8; ++i)
                h[i] = pack_bf16x2(v[16 * k + 2 * i], v[16 * k + 2 * i + 1]);
              store32(p.g + 2 * at + 32 * k, h);
            }
          }
          continue;
        }
        if (EPI == OUT) {
          const int x = x0 + c * 32;
          if (p.v0 + row < p.vocab) {
            __nv_bfloat16* at = p.dw + (size_t)(p.v0 + row) * p.hidden + x;
            const bool sectors = (reinterpret_cast<uintptr_t>(at) & 31) == 0;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              uint32_t h[8];
#pragma unroll
              for (int i = 0; i < 8; ++i)
                h[i] = pack_bf16x2(v[16 * k + 2 * i] * sc, v[16 * k + 2 * i + 1] * sc);
              if (sectors && x + 16 * k + 16 <= p.hidden) {
                store32(at + 16 * k, h);
              } else {
                uint4* at4 = reinterpret_cast<uint4*>(at + 16 * k);
                if (x + 16 * k < p.hidden) at4[0] = make_uint4(h[0], h[1], h[2], h[3]);
                if (x + 16 * k + 8 < p.hidden) at4[1] = make_uint4(h[4], h[5], h[6], h[7]);
              }
            }
          }
          continue;
        }
        if (EPI == ACC) {
          slab_begin(lane);
#pragma unroll
          for (int j = 0; j < 8; ++j)
            slab_put(slab, lane, j,
                     make_uint4(__float_as_uint(v[4 * j]), __float_as_uint(v[4 * j + 1]),
                                __float_as_uint(v[4 * j + 2]), __float_as_uint(v[4 * j + 3])));
          fence_proxy_async_smem();
          __syncwarp();
          const int x = x0 + c * 32;
          if (lane == 0 && x < p.hidden) {
            if (p.add) add_box(&tm_out, slab, x, t.split * p.rows_pad + row0);
            else store_box(&tm_out, slab, x, t.split * p.rows_pad + row0);
            bulk_commit();
          }
        }
      }
      if (EPI == LSE || EPI == EXP) {
        if (live) {
          const size_t at = (size_t)row * p.parts + (p.v0 + x0) / HN;
          if (EPI == LSE) p.part_m[at] = mx;
          p.part_s[at] = sum;
          // (a repair's references are its largest logits)
          if (EPI == EXP && !repair && mx - ref > kRefSlack) raise(p, row, mx);
        }
      }
    }
    if (EPI == ACC && lane == 0) bulk_wait_all();
  }

  tc_fence_before();
  __syncthreads();
  if ((EPI == GRAD || EPI == OUT) && *abort_flag)
    for (int r = threadIdx.x; r < p.all_rows; r += kThreads)
      p.nll[r] = p.lse[r] = __int_as_float(0x7fc00000);
  // no CTA leaves while its pair's copies, products or arrivals may reach it
  if (CG == 2) cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_cg<CG>(tmem, 512);
  }
}

// ------------------------------------------------------------ small kernels
struct CeRows {
  int rows, vocab, hidden, rows_pad;
  const __nv_bfloat16* x;
  const __nv_bfloat16* w;
  long long x_stride, w_stride;
  const int* targets;
  const float* d_nll;  // null: forward only
  int scan;            // the gather numbers the rows itself
  int* n;              // rows with a target
  int* err;
  int* any;            // [pieces]: whether a repair has anything to do
  int pieces;
  int* place;          // [rows]: compact row or -1
  int* target;         // compact
  float* z_t;          // compact: the target's logit
  float* ref2;         // compact: [pieces + 1][rows_pad] references before each piece and at
                       // the end, log2 units
  float* d;            // compact
  unsigned long long* own;  // [vocab] or null: rows with this target, kOwnOne + row each
  __nv_bfloat16* xc;   // [rows_pad][pitch]
  int pitch;           // hidden rounded up: rows on 128-byte boundaries
};

DF_DEV bool has_target(const CeRows& a, int r) {
  const int t = __ldg(a.targets + r);
  return t >= 0 && t < a.vocab;
}

DF_DEV void store_counts(const CeRows& a, int n) {
  *a.n = n;
  *a.err = 0;
  for (int i = 0; i < a.pieces; ++i) a.any[i] = 0;
}

// Compact numbers of the rows that have a target, in their order.
__global__ void __launch_bounds__(1024) ce_compact_kernel(const __grid_constant__ CeRows a) {
  __shared__ int warp_n[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  grid_dep_sync();
  int base = 0;
  for (int r0 = 0; r0 < a.rows; r0 += 1024) {
    const int r = r0 + threadIdx.x;
    const bool has = r < a.rows && has_target(a, r);
    const uint32_t b = __ballot_sync(0xffffffffu, has);
    if (lane == 0) warp_n[warp] = __popc(b);
    __syncthreads();
    int at = base + __popc(b & ((1u << lane) - 1u));
    for (int w = 0; w < 32; ++w) {
      at += w < warp ? warp_n[w] : 0;
      base += warp_n[w];
    }
    if (r < a.rows) a.place[r] = has ? at : -1;
    __syncthreads();
  }
  if (threadIdx.x == 0) store_counts(a, base);
}

DF_DEV float dot8(uint4 a, uint4 b) {
  const uint32_t u[4] = {a.x, a.y, a.z, a.w}, v[4] = {b.x, b.y, b.z, b.w};
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    s += __uint_as_float(u[i] << 16) * __uint_as_float(v[i] << 16);
    s += __uint_as_float(u[i] & 0xffff0000u) * __uint_as_float(v[i] & 0xffff0000u);
  }
  return s;
}

// One CTA per row: its place, its copy of x, its target's logit.  The compact
// rows that fill the last 256 are zero.
constexpr int kRowThreads = 256;

__global__ void __launch_bounds__(kRowThreads) ce_gather_kernel(const __grid_constant__ CeRows a) {
  __shared__ float sm[8];
  __shared__ int before[8], all[8];
  grid_dep_sync();
  const int row = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int n8 = a.hidden / 8;
  int n, c = -1;
  if (a.scan) {  // the rows with a target in front of this one, and all of them
    int mine = 0, sum = 0;
    for (int r = threadIdx.x; r < a.rows; r += kRowThreads) {
      const int has = has_target(a, r) ? 1 : 0;
      sum += has;
      mine += r < row ? has : 0;
    }
    mine = __reduce_add_sync(0xffffffffu, mine);
    sum = __reduce_add_sync(0xffffffffu, sum);
    if (lane == 0) before[warp] = mine, all[warp] = sum;
    __syncthreads();
    n = mine = 0;
    for (int w = 0; w < 8; ++w) n += all[w], mine += before[w];
    if (row < a.rows) {
      c = has_target(a, row) ? mine : -1;
      if (threadIdx.x == 0) a.place[row] = c;
    }
    if (row == 0 && threadIdx.x == 0) store_counts(a, n);
  } else {
    n = __ldcg(a.n);
    if (row < a.rows) c = __ldcg(a.place + row);
  }
  if (a.own != nullptr)
    for (long long v = (long long)row * kRowThreads + threadIdx.x; v < a.vocab;
         v += (long long)gridDim.x * kRowThreads)
      a.own[v] = 0;
  if (row < 256 && n + row < (n + 255) / 256 * 256) {
    uint4* dst = reinterpret_cast<uint4*>(a.xc + (size_t)(n + row) * a.pitch);
    for (int i = threadIdx.x; i < n8; i += kRowThreads) dst[i] = make_uint4(0, 0, 0, 0);
  }
  if (c < 0) return;
  const int t = __ldg(a.targets + row);
  const uint4* x = reinterpret_cast<const uint4*>(a.x + row * a.x_stride);
  const uint4* w = reinterpret_cast<const uint4*>(a.w + t * a.w_stride);
  uint4* dst = reinterpret_cast<uint4*>(a.xc + (size_t)c * a.pitch);
  float s = 0.f;
  for (int i = threadIdx.x; i < n8; i += kRowThreads) {
    const uint4 v = __ldg(x + i);
    s += dot8(v, __ldg(w + i));
    dst[i] = v;
  }
#pragma unroll
  for (int o = 16; o > 0; o /= 2) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (lane == 0) sm[warp] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    float z = 0.f;
    for (int i = 0; i < 8; ++i) z += sm[i];
    a.target[c] = t;
    a.z_t[c] = z;
    for (int i = 0; i <= a.pieces; ++i) a.ref2[(size_t)i * a.rows_pad + c] = z * kLog2e;
    if (a.d_nll != nullptr) a.d[c] = __ldg(a.d_nll + row);
  }
}

struct CeSums {
  const float* part_m;  // [rows_pad][parts]
  const float* part_s;
  const float* refs;    // gradient: [piece][rows_pad] the references of the sums, log2 units
  int parts, piece_parts;
  float* nll;           // [rows]
  float* lse;
  const float* acc;     // gradient: [slices][rows_pad][pitch]
  int slices;
  __nv_bfloat16* dx;
  float* miss;          // compact: 1 - p_t
  float* lse2;          // compact: lse in log2 units
  float* scale;         // compact: 1 / sum of the exponentials, with the last reference
};

// (m, s) and (m2, s2), sums relative to a reference each, as one
DF_DEV void join(float& m, float& s, float m2, float s2) {
  if (s2 == 0.f) return;
  const float top = fmaxf(m, m2);
  s = s * fast_exp2(m - top) + s2 * fast_exp2(m2 - top);
  m = top;
}

// nll and lse of a row from the tiles' sums, joined in a fixed order, and with a
// gradient dx = d * (acc / sum - (1 - p_t) * w_t): a thread has 8 channels, a row
// as many CTAs as that takes.  The products and w_t are on their way while the
// sums are joined.
constexpr int kAhead = 4;  // slices of the products

__global__ void __launch_bounds__(kRowThreads)
    ce_finish_kernel(const __grid_constant__ CeRows a, const __grid_constant__ CeSums s) {
  __shared__ float sm[8], ss[8];
  grid_dep_sync();
  const int row = blockIdx.x, c = __ldcg(a.place + row);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int i = blockIdx.y * kRowThreads + threadIdx.x;  // of the channels' groups of 8
  const bool mine = s.dx != nullptr && i < a.hidden / 8;
  const bool one = threadIdx.x == 0 && blockIdx.y == 0;
  const float nan = __int_as_float(0x7fc00000);
  const bool failed = __ldcg(a.err) != 0;  // a wait ran out: no number is right
  uint4* out = reinterpret_cast<uint4*>(s.dx + (size_t)row * a.hidden);
  if (c < 0) {
    if (one) s.nll[row] = s.lse[row] = failed ? nan : 0.f;
    if (mine) out[i] = make_uint4(0, 0, 0, 0);
    return;
  }
  float4 u[kAhead][2];
  uint4 wt = make_uint4(0, 0, 0, 0);
  auto load = [&](int k0) {
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      if (k0 + k >= s.slices) break;
      const float4* p = reinterpret_cast<const float4*>(
                            s.acc + ((size_t)(k0 + k) * a.rows_pad + c) * a.pitch) + 2 * i;
      u[k][0] = __ldcg(p), u[k][1] = __ldcg(p + 1);
    }
  };
  if (mine) {
    wt = __ldg(reinterpret_cast<const uint4*>(a.w + __ldcg(a.target + c) * a.w_stride) + i);
    load(0);
  }
  float m = kNegInf, sum = 0.f;
  const float* pm = s.part_m + (size_t)c * s.parts;
  const float* ps = s.part_s + (size_t)c * s.parts;
  if (s.refs == nullptr) {
    for (int t = threadIdx.x; t < s.parts; t += kRowThreads)
      join(m, sum, __ldcg(pm + t), __ldcg(ps + t));
  } else {
    for (int k = 0, t0 = 0; t0 < s.parts; ++k, t0 += s.piece_parts) {
      float piece = 0.f;
      for (int t = t0 + threadIdx.x; t < min(t0 + s.piece_parts, s.parts); t += kRowThreads)
        piece += __ldcg(ps + t);
      join(m, sum, __ldcg(s.refs + (size_t)k * a.rows_pad + c), piece);
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o /= 2) {
    const float m2 = __shfl_xor_sync(0xffffffffu, m, o), s2 = __shfl_xor_sync(0xffffffffu, sum, o);
    join(m, sum, m2, s2);
  }
  if (lane == 0) sm[warp] = m, ss[warp] = sum;
  __syncthreads();
  m = sm[0], sum = ss[0];
  for (int w = 1; w < 8; ++w) join(m, sum, sm[w], ss[w]);
  const float z = __ldcg(a.z_t + c), z2 = z * kLog2e;
  const float top = sum == 0.f ? z2 : fmaxf(m, z2);
  const float others = sum == 0.f ? 0.f : sum * fast_exp2(m - top);  // relative to `top`
  const float total = others + fast_exp2(z2 - top);
  if (one) {
    // where the target leads, log1p keeps what is left of a small loss
    // (an infinite one leaves NaN: the difference is otherwise zero there)
    const float nll = (top == z2 ? log1pf(others) : logf(total)) + (top - z2) * kLn2;
    s.nll[row] = failed ? nan : nll;
    s.lse[row] = failed ? nan : nll + z;
    if (s.dx != nullptr) {
      s.miss[c] = others / total;
      s.lse2[c] = top + log2f(total);
    }
  }
  if (s.dx == nullptr) return;
  // the products are relative to the row's last reference, the exponentials'
  // sum up to 2^104: their quotient is an ordinary number, to which d comes last
  const float d = __ldcg(a.d + c);
  const float last = __ldcg(a.ref2 + (size_t)a.pieces * a.rows_pad + c);
  const float f = failed ? nan : fast_exp2(last - top) / total;
  const float g = others / total;
  if (one) {
    s.scale[c] = f;
    // (whole numbers: the sum does not depend on the rows' order)
    if (a.own != nullptr) atomicAdd(a.own + __ldcg(a.target + c), kOwnOne + (unsigned)c);
  }
  if (!mine) return;
  float v[8] = {};
  for (int k0 = 0; k0 < s.slices; k0 += kAhead) {
    if (k0 > 0) load(k0);
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      if (k0 + k >= s.slices) break;
      v[0] += u[k][0].x, v[1] += u[k][0].y, v[2] += u[k][0].z, v[3] += u[k][0].w;
      v[4] += u[k][1].x, v[5] += u[k][1].y, v[6] += u[k][1].z, v[7] += u[k][1].w;
    }
  }
  const uint32_t t[4] = {wt.x, wt.y, wt.z, wt.w};
  uint32_t o[4];
#pragma unroll
  for (int j = 0; j < 4; ++j)
    o[j] = pack_bf16x2(d * (v[2 * j] * f - g * __uint_as_float(t[j] << 16)),
                       d * (v[2 * j + 1] * f - g * __uint_as_float(t[j] & 0xffff0000u)));
  out[i] = make_uint4(o[0], o[1], o[2], o[3]);
}

// The kept exponentials of a piece that is the whole vocabulary, with their
// sums known: 24-bit numbers times the row's scale and weight, rounded to bf16
// once, the target's in its place.  A row and 4 * 2048 columns per CTA.
constexpr int kScaleCols = 8, kScaleSteps = 4;

__global__ void __launch_bounds__(kRowThreads)
    ce_scale_kernel(const __grid_constant__ CeRows a, __nv_bfloat16* g, const uint8_t* low,
                    int pitch, const float* scale, const float* miss) {
  grid_dep_sync();
  const int row = blockIdx.x;
  const int col0 = (blockIdx.y * kScaleSteps * kRowThreads + threadIdx.x) * kScaleCols;
  if (row >= __ldcg(a.n)) return;
  uint4* at = reinterpret_cast<uint4*>(g + (size_t)row * pitch);
  const uint2* lat = reinterpret_cast<const uint2*>(low + (size_t)row * pitch);
  uint4 hi[kScaleSteps];
  uint2 lo[kScaleSteps];
#pragma unroll
  for (int k = 0; k < kScaleSteps; ++k) {
    const int col = col0 + k * kRowThreads * kScaleCols;
    if (col < pitch) {
      hi[k] = at[col / kScaleCols];
      lo[k] = __ldcg(lat + col / kScaleCols);
    }
  }
  const float s = __ldcg(scale + row), d = __ldcg(a.d + row), own = -d * __ldcg(miss + row);
  const int target = __ldcg(a.target + row);
#pragma unroll
  for (int k = 0; k < kScaleSteps; ++k) {
    const int col = col0 + k * kRowThreads * kScaleCols;
    if (col >= pitch) break;
    const uint32_t h[4] = {hi[k].x, hi[k].y, hi[k].z, hi[k].w};
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t up = (i & 1) ? h[i >> 1] & 0xffff0000u : h[i >> 1] << 16;
      const int down = (int)(int8_t)((i < 4 ? lo[k].x : lo[k].y) >> (8 * (i & 3)));
      v[i] = __uint_as_float(up + (uint32_t)(down * 256)) * s * d;
      if (col + i == target) v[i] = own;
    }
    at[col / kScaleCols] = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                      pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
  }
}

// ----------------------------------------------------------------- the host
// Bytes of a piece's bf16 exponentials: what the caller's workspace grows to (half
// as much again where their next 8 bits are kept).  Three pieces of 512 MB instead
// of two of 1 GB make no difference in time.  From one piece to two dw takes a
// fourth product: with dx and dw 3328 rows x 150000, hidden 4096, one piece, 7.45 to
// 7.9 ms (floor 7.07 at the sustained rate), 4096 rows, two, 11.4 to 12.5 (8.70).
constexpr size_t kPieceBytes = 1ull << 30;
constexpr int kMaxSplits = 16;
// Up to here every CTA of the gather counts the targets in front of its row
// itself (16 KB from L2 each): a launch less.
constexpr int kScanRows = 4096;

struct Plan {
  int cg, rows_pad, pitch, n_tiles;
  int piece, pieces;   // columns of a piece (a multiple of 256)
  int splits;          // of ACC's K
  bool keep;           // dw from the exponentials that dx was made from
  size_t any, place, target, z_t, ref2, d, miss, lse2, scale, own, xc, part_m, part_s, g,
      low, acc, total;
};

// Splits of K for the products of few tiles: whole waves, and about 24
// k-blocks' time for each wave's beginning and end.
int acc_splits(int tiles, int n_kb, int units) {
  double best_t = 1e30;
  int best = 1;
  for (int sp = 1; sp <= std::min(kMaxSplits, std::max(1, n_kb / 8)); ++sp) {
    const int waves = (tiles * sp + units - 1) / units;
    const double t = waves * ((double)n_kb / sp + 24.) + 4. * sp;
    if (t < best_t - 1e-9) best_t = t, best = sp;
  }
  return best;
}

// The plan of a call goes by its sizes alone, so that the workspace can be
// asked for without a GPU; 152 SMs are what it is made for.
constexpr int kPlanSms = 152;

Plan make_plan(int rows, int vocab, int hidden, int grads) {
  Plan p{};
  p.cg = rows <= BM ? 1 : 2;
  p.rows_pad = (rows + 255) / 256 * 256;
  p.pitch = (hidden + 63) / 64 * 64;
  p.n_tiles = (vocab + BN - 1) / BN;
  const size_t most =
      std::max<size_t>(4096, kPieceBytes / (2 * (size_t)p.rows_pad) / BN * BN);
  p.pieces = (int)(((size_t)p.n_tiles * BN + most - 1) / most);
  p.piece = (p.n_tiles + p.pieces - 1) / p.pieces * BN;
  p.pieces = (p.n_tiles * BN + p.piece - 1) / p.piece;
  p.keep = grads == 2 && p.pieces == 1;
  const int m_tiles = (rows + p.cg * BM - 1) / (p.cg * BM), h_tiles = (hidden + BN - 1) / BN;
  p.splits = acc_splits(m_tiles * h_tiles, p.piece / BK, kPlanSms / p.cg);
  size_t at = 256;  // n, err
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += (bytes + 255) / 256 * 256;
    return here;
  };
  const size_t pad = (size_t)p.rows_pad;
  p.any = take((size_t)p.pieces * 4);
  p.place = take((size_t)rows * 4);
  p.target = take(pad * 4);
  p.z_t = take(pad * 4);
  p.ref2 = take(pad * (p.pieces + 1) * 4);
  p.xc = take(pad * p.pitch * 2);
  if (grads == 0) p.part_m = take(pad * p.n_tiles * 2 * 4);
  p.part_s = take(pad * p.n_tiles * 2 * 4);
  if (grads > 0) {
    p.d = take(pad * 4);
    p.miss = take(pad * 4);
    p.lse2 = take(pad * 4);
    p.scale = take(pad * 4);
    p.g = take(pad * p.piece * 2);
    if (p.keep) p.low = take(pad * p.piece);
    if (grads == 2) p.own = take((size_t)vocab * 8);
    p.acc = take(pad * p.splits * p.pitch * 4);
  }
  p.total = at;
  return p;
}

int make_map(CUtensorMap* m, const void* p, bool f32, long long rows, long long cols,
             long long pitch, int box_cols, int box_rows) {
  return make_tmap_2d(m, p, f32 ? 4 : 2, rows, cols, pitch, box_cols, box_rows);
}

template <int EPI, int CG>
cudaError_t launch_gemm(const CUtensorMap& a, const CUtensorMap& a64, const CUtensorMap& b,
                        const CUtensorMap& out, const CeGemm& p, int units, int sms,
                        cudaStream_t s) {
  static std::atomic<unsigned long long> attr_done{0};
  if (!done_on_device(attr_done)) {
    const cudaError_t e = cudaFuncSetAttribute(
        ce_gemm_kernel<EPI, CG>, cudaFuncAttributeMaxDynamicSharedMemorySize,
        (int)Geo<EPI, CG>::SMEM);
    if (e != cudaSuccess) return e;
    mark_device(attr_done);
  }
  const int grid = std::max(1, std::min(units, sms / CG)) * CG;
  CeGemm q = p;
  q.by_group = Divisor(kGroup * p.n_tiles);
  return launch_pdl_cluster(ce_gemm_kernel<EPI, CG>, dim3(grid), dim3(kThreads),
                            Geo<EPI, CG>::SMEM, s, (unsigned)CG, a, a64, b, out, q);
}

template <int EPI>
cudaError_t launch_gemm(int cg, const CUtensorMap& a, const CUtensorMap& a64,
                        const CUtensorMap& b, const CUtensorMap& out, const CeGemm& p, int units,
                        int sms, cudaStream_t s) {
  return cg == 1 ? launch_gemm<EPI, 1>(a, a64, b, out, p, units, sms, s)
                 : launch_gemm<EPI, 2>(a, a64, b, out, p, units, sms, s);
}

struct Call {
  int rows, vocab, hidden;
  const void* x;
  int64_t x_stride;
  const void* w;
  int64_t w_stride;
  const int32_t* targets;
  const float* d_nll;
  float* nll;
  float* lse;
  void* dx;
  void* dw;
};

int device_sms(int* sms) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev);
  return e == cudaSuccess ? DFLASH_OK : api_fail(DFLASH_ERR_CUDA, "%s", cudaGetErrorString(e));
}

int check_sizes(int rows, int vocab, int hidden) {
  if (rows < 0 || vocab <= 0 || hidden <= 0)
    return api_fail(DFLASH_ERR_ARG, "rows must be >= 0, vocab and hidden positive");
  if (hidden % 8 != 0) return api_fail(DFLASH_ERR_SHAPE, "hidden must be a multiple of 8");
  if (rows > (1 << 20) || vocab > (1 << 24) || hidden > (1 << 16))
    return api_fail(DFLASH_ERR_SHAPE, "at most 2^20 rows, 2^24 columns and hidden 2^16");
  return DFLASH_OK;
}

bool misaligned(const void* p, uintptr_t m) { return (reinterpret_cast<uintptr_t>(p) & m) != 0; }

int check_call(const Call& c, bool grad, const void* ws, size_t ws_bytes) {
  if (int r = check_sizes(c.rows, c.vocab, c.hidden)) return r;
  if (c.rows > 0 && (c.x == nullptr || c.targets == nullptr || c.nll == nullptr ||
                     c.lse == nullptr || (grad && (c.d_nll == nullptr || c.dx == nullptr))))
    return api_fail(DFLASH_ERR_ARG, "null tensor");
  if (c.w == nullptr) return api_fail(DFLASH_ERR_ARG, "null head");
  if (misaligned(c.x, 15) || misaligned(c.w, 15) || misaligned(c.dx, 15) || misaligned(c.dw, 15))
    return api_fail(DFLASH_ERR_ARG, "bf16 tensors must be 16-byte aligned");
  if (misaligned(c.targets, 3) || misaligned(c.d_nll, 3) || misaligned(c.nll, 3) ||
      misaligned(c.lse, 3))
    return api_fail(DFLASH_ERR_ARG, "32-bit tensors must be aligned to their type");
  if ((c.rows > 1 && (c.x_stride < c.hidden || c.x_stride % 8 != 0)) ||
      (c.vocab > 1 && (c.w_stride < c.hidden || c.w_stride % 8 != 0)))
    return api_fail(DFLASH_ERR_ARG, "row strides must be multiples of 8, at least hidden");
  if (c.x_stride > (1LL << 32) || c.w_stride > (1LL << 32))
    return api_fail(DFLASH_ERR_SHAPE, "row strides must be at most 2^32");
  if (ws == nullptr || misaligned(ws, 255))
    return api_fail(DFLASH_ERR_ARG, "workspace null or not on a 256-byte boundary");
  size_t need = 0;
  if (int r = dflash_linear_ce_workspace(c.rows, c.vocab, c.hidden, grad ? (c.dw ? 2 : 1) : 0,
                                         &need))
    return r;
  if (ws_bytes < need)
    return api_fail(DFLASH_ERR_CAPACITY, "workspace of %zu bytes, %zu needed", ws_bytes, need);
  return DFLASH_OK;
}

int run(const Call& c, bool grad, void* ws, size_t ws_bytes, cudaStream_t s) {
  if (int r = check_call(c, grad, ws, ws_bytes)) return r;
  int sms = 0;
  if (int r = device_sms(&sms)) return r;
  cudaError_t e = cudaSuccess;
  auto done = [&](const char* what) {
    return e == cudaSuccess ? DFLASH_OK
                            : api_fail(DFLASH_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
  };
  if (c.rows == 0) {
    if (c.dw != nullptr)
      e = cudaMemsetAsync(c.dw, 0, (size_t)c.vocab * c.hidden * 2, s);
    return done("memset");
  }
  const Plan p = make_plan(c.rows, c.vocab, c.hidden, !grad ? 0 : c.dw == nullptr ? 1 : 2);
  char* base = static_cast<char*>(ws);
  auto f32 = [&](size_t at) { return reinterpret_cast<float*>(base + at); };
  auto i32 = [&](size_t at) { return reinterpret_cast<int*>(base + at); };
  const int pad = p.rows_pad, H = c.hidden, V = c.vocab;

  CeRows a{};
  a.rows = c.rows;
  a.vocab = V;
  a.hidden = H;
  a.rows_pad = pad;
  a.x = static_cast<const __nv_bfloat16*>(c.x);
  a.w = static_cast<const __nv_bfloat16*>(c.w);
  a.x_stride = c.x_stride;
  a.w_stride = c.w_stride;
  a.targets = c.targets;
  a.d_nll = c.d_nll;
  a.n = i32(0);
  a.err = i32(4);
  a.scan = c.rows <= kScanRows;
  a.any = i32(p.any);
  a.pieces = p.pieces;
  a.place = i32(p.place);
  a.target = i32(p.target);
  a.z_t = f32(p.z_t);
  a.ref2 = f32(p.ref2);
  a.d = f32(p.d);
  a.xc = reinterpret_cast<__nv_bfloat16*>(base + p.xc);
  a.pitch = p.pitch;
  if (c.dw != nullptr) a.own = reinterpret_cast<unsigned long long*>(base + p.own);

  // maps: x by rows and by channels, w the same, a piece's exponentials, the
  // fp32 products
  const long long w_pitch = V > 1 ? c.w_stride : H;
  CUtensorMap x_k, x_k64, w_k, x_mn, w_mn, g_k, g_k64, g_mn, acc_out;
  int bad = make_map(&x_k, a.xc, false, pad, H, p.pitch, 64, BM) |
            make_map(&x_k64, a.xc, false, pad, H, p.pitch, 64, BM / 2) |
            make_map(&w_k, c.w, false, V, H, w_pitch, 64, BN / p.cg);
  if (grad) {
    const void* g = base + p.g;
    bad |= make_map(&w_mn, c.w, false, V, H, w_pitch, 64, 64) |
           make_map(&g_k, g, false, pad, p.piece, p.piece, 64, BM) |
           make_map(&g_k64, g, false, pad, p.piece, p.piece, 64, BM / 2) |
           make_map(&acc_out, base + p.acc, true, (long long)pad * p.splits, H, p.pitch, 32, 32);
    if (c.dw != nullptr)
      bad |= make_map(&x_mn, a.xc, false, pad, H, p.pitch, 64, 64) |
             make_map(&g_mn, g, false, pad, p.piece, p.piece, 64, 64);
  }
  if (bad != 0) return api_fail(DFLASH_ERR_CUDA, "tensor map encoding failed");

  CeGemm gm{};
  gm.n_rows = a.n;
  gm.n_kb = (H + BK - 1) / BK;
  gm.splits = 1;
  gm.vocab = V;
  gm.hidden = H;
  gm.rows_pad = pad;
  gm.ref2 = a.ref2;
  gm.target = a.target;
  gm.part_m = f32(p.part_m);
  gm.part_s = f32(p.part_s);
  gm.g = reinterpret_cast<uint8_t*>(base + p.g);
  gm.g_pitch = p.piece;
  gm.parts = p.n_tiles * 2;
  gm.nll = c.nll;
  gm.lse = c.lse;
  gm.all_rows = c.rows;
  gm.err = a.err;
  CeSums sums{};
  sums.part_m = gm.part_m;
  sums.part_s = gm.part_s;
  sums.parts = p.n_tiles * 2;
  sums.piece_parts = p.piece / HN;
  sums.nll = c.nll;
  sums.lse = c.lse;
  const int m_tiles = (c.rows + p.cg * BM - 1) / (p.cg * BM);
  const int h_tiles = (H + BN - 1) / BN;
  const dim3 b1024(1024), b256(kRowThreads);

  if (!a.scan) e = launch_pdl(ce_compact_kernel, dim3(1), b1024, 0, s, a);
  if (e == cudaSuccess) e = launch_pdl(ce_gather_kernel, dim3(pad), b256, 0, s, a);
  if (!grad) {
    gm.n_tiles = p.n_tiles;
    if (e == cudaSuccess)
      e = launch_gemm<LSE>(p.cg, x_k, x_k64, w_k, x_k, gm, m_tiles * p.n_tiles, sms, s);
    if (e == cudaSuccess) e = launch_pdl(ce_finish_kernel, dim3(c.rows), b256, 0, s, a, sums);
    return done("cross entropy launch");
  }

  sums.refs = a.ref2 + pad;
  sums.acc = f32(p.acc);
  sums.slices = p.splits;
  sums.dx = static_cast<__nv_bfloat16*>(c.dx);
  sums.miss = f32(p.miss);
  sums.lse2 = f32(p.lse2);
  sums.scale = f32(p.scale);
  for (int i = 0; i < p.pieces && e == cudaSuccess; ++i) {
    const int v0 = i * p.piece, tiles = std::min(p.piece, V - v0 + BN - 1) / BN;
    CeGemm ex = gm;
    ex.v0 = v0;
    ex.n_tiles = tiles;
    ex.ref2 = a.ref2 + (size_t)i * pad;
    ex.raised = a.ref2 + (size_t)(i + 1) * pad;
    ex.pieces_left = p.pieces - i;
    ex.any = a.any + i;
    if (p.keep) ex.low = reinterpret_cast<uint8_t*>(base + p.low);
    e = launch_gemm<EXP>(p.cg, x_k, x_k64, w_k, x_k, ex, m_tiles * tiles, sms, s);
    ex.repair = 1;
    if (i > 0) {
      ex.acc = f32(p.acc);
      ex.acc_pitch = p.pitch;
      ex.acc_slices = p.splits;
    }
    if (e == cudaSuccess)
      e = launch_gemm<EXP>(p.cg, x_k, x_k64, w_k, x_k, ex, m_tiles * tiles, sms, s);
    CeGemm ac = gm;
    ac.v0 = v0;
    ac.n_tiles = h_tiles;
    ac.n_kb = tiles * BN / BK;
    ac.splits = p.splits;
    ac.add = i > 0;
    if (e == cudaSuccess)
      e = launch_gemm<ACC>(p.cg, g_k, g_k64, w_mn, acc_out, ac, m_tiles * h_tiles * p.splits, sms, s);
  }
  const int shares = (H / 8 + kRowThreads - 1) / kRowThreads;
  if (e == cudaSuccess)
    e = launch_pdl(ce_finish_kernel, dim3(c.rows, shares), b256, 0, s, a, sums);
  for (int i = 0; c.dw != nullptr && i < p.pieces && e == cudaSuccess; ++i) {
    const int v0 = i * p.piece, tiles = std::min(p.piece, V - v0 + BN - 1) / BN;
    if (p.keep) {
      e = launch_pdl(ce_scale_kernel, dim3(pad, (p.piece + kScaleSteps * kScaleCols * kRowThreads - 1) /
                                     (kScaleSteps * kScaleCols * kRowThreads)),
                     b256, 0, s, a, reinterpret_cast<__nv_bfloat16*>(base + p.g),
                     reinterpret_cast<const uint8_t*>(base + p.low), p.piece, f32(p.scale),
                     f32(p.miss));
    } else {
      CeGemm gr = gm;
      gr.v0 = v0;
      gr.n_tiles = tiles;
      gr.ref2 = f32(p.lse2);
      gr.d = a.d;
      gr.miss = f32(p.miss);
      e = launch_gemm<GRAD>(p.cg, x_k, x_k64, w_k, x_k, gr, m_tiles * tiles, sms, s);
    }
    CeGemm ow = gm;
    ow.v0 = v0;
    ow.m_tiles = (tiles * BN + p.cg * BM - 1) / (p.cg * BM);
    ow.n_tiles = h_tiles;
    ow.d = a.d;
    ow.miss = f32(p.miss);
    ow.own = a.own;
    ow.dw = static_cast<__nv_bfloat16*>(c.dw);
    if (e == cudaSuccess)
      e = launch_gemm<OUT>(p.cg, g_mn, g_mn, x_mn, g_mn, ow, ow.m_tiles * h_tiles, sms, s);
  }
  return done("cross entropy launch");
}

}  // namespace
}  // namespace df

using namespace df;

extern "C" {

int dflash_linear_ce_workspace(int rows, int vocab, int hidden, int grads, size_t* bytes) {
  if (bytes == nullptr) return api_fail(DFLASH_ERR_ARG, "bytes is null");
  if (grads < 0 || grads > 2) return api_fail(DFLASH_ERR_ARG, "grads must be 0, 1 or 2");
  if (int r = check_sizes(rows, vocab, hidden)) return r;
  *bytes = make_plan(std::max(rows, 1), vocab, hidden, grads).total;
  return DFLASH_OK;
}

int dflash_linear_ce(int rows, int vocab, int hidden, const void* x, int64_t x_stride,
                     const void* w, int64_t w_stride, const int32_t* targets, float* nll,
                     float* lse, void* workspace, size_t workspace_bytes, dflash_stream stream) {
  return run({rows, vocab, hidden, x, x_stride, w, w_stride, targets, nullptr, nll, lse, nullptr,
              nullptr},
             false, workspace, workspace_bytes, static_cast<cudaStream_t>(stream));
}

int dflash_linear_ce_grad(int rows, int vocab, int hidden, const void* x, int64_t x_stride,
                          const void* w, int64_t w_stride, const int32_t* targets,
                          const float* d_nll, float* nll, float* lse, void* dx, void* dw,
                          void* workspace, size_t workspace_bytes, dflash_stream stream) {
  return run({rows, vocab, hidden, x, x_stride, w, w_stride, targets, d_nll, nll, lse, dx, dw},
             true, workspace, workspace_bytes, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
