// gated_ffn.cu -- the dense gated feed-forward block with a choice of activation,
// forward and backward, on tcgen05 with CTA pairs:
//   z = x Wg, u = x Wu, h = act(z) u, y = h Wd
//   (Shazeer, "GLU Variants Improve Transformer", 2020);
//   dh = dy Wd^T, du = dh act(z), dz = dh u act'(z),
//   dx = du Wu^T + dz Wg^T, dWd = h^T dy, dWu = du^T x, dWg = dz^T x.
//
// Every product is one persistent GEMM kernel with its elementwise work in the
// epilogue: both projections, activation and product in the first (gate and up
// weights are the two halves of one 256-wide operand), the activation's backward
// behind dh, the sum of dx in one accumulator over both products, and the three
// weight gradients in one launch.
//
// A pair of CTAs (two SMs) owns a 256 x 256 tile: each CTA loads 128 rows of A and
// 128 rows of B a 64-wide k-block, tcgen05.mma.cta_group::2 multiplies both halves
// of B with both halves of A, and each CTA accumulates its 128 rows in its own
// TMEM (two accumulators: the epilogue of a tile overlaps the next tile).  A k-block
// then costs an SM 32 KB from L2 for 128 x 256 outputs, against 48 KB with a CTA a
// tile.
//
// Roles (320 threads): warp 0 loads by TMA, warp 1 allocates TMEM and in the first
// CTA of the pair issues the MMAs, warps 2..9 are the epilogue (two warps a quarter
// of the TMEM lanes, each half of the columns).
//
// Measured at d = 2048, F = 8192: 16384 tokens forward 1.22 to 1.28 ms (1.29 to 1.35
// PFLOP/s), a training step of 8192 tokens 2.01 to 2.09 ms.  In a loop the power cap
// bounds the products (tensor pipe 97 to 98% active at 1.46 GHz).
//
// Every wait is bounded: on timeout the CTA flags TW_ERR_TIMEOUT, stops its roles, lets
// its copies land and meets its pair at the last barrier.
#include "tmap.h"
#include "pdl.cuh"
#include "cluster.cuh"
#include "gated_act.cuh"
#include "tw_common.cuh"
#include "tw_internal.h"

namespace tw {
namespace {

constexpr int kBM = 128;  // rows of A (and of B) a CTA
constexpr int kBN = 256;  // columns of a tile
constexpr int kBK = 64;   // 64 bf16 = one 128-byte swizzle row
constexpr int kHalfBytes = kBM * kBK * 2;       // one operand's share of a stage
constexpr int kStageBytes = 2 * kHalfBytes;
constexpr int kEpiWarps = 8;
constexpr int kThreads = 64 + 32 * kEpiWarps;
constexpr int kTmemCols = 2 * kBN;

// Staging of the elementwise epilogues: slabs of a warp's 32 rows x 32 columns of a
// bf16 matrix, moved by TMA (64-byte swizzle).
constexpr int kSlabBytes = 32 * 32 * 2;

struct Tail {
  uint64_t full[6];
  uint64_t empty[6];
  uint64_t tmem_full[2];
  uint64_t tmem_empty[2];
  uint64_t drain;
  uint64_t loaded[kEpiWarps];
  uint32_t tmem_base;
  int abort;
  int never;
};
// Shared memory: the operands' ring, then each epilogue warp's slabs.
template <class Epi>
struct Layout {
  static constexpr size_t kRing = (size_t)Epi::kStages * kStageBytes;
  static constexpr size_t kStaging = (size_t)kEpiWarps * Epi::kSlabs * kSlabBytes;
  static constexpr size_t kSmem = 1024 + kRing + kStaging + sizeof(Tail);
  static_assert(kSmem <= 227 * 1024, "shared memory budget");
};

// ------------------------------------------------------------- pair helpers --
// Address of `bar` in the first CTA of the pair.
TW_DEV uint32_t leader_addr(const uint64_t* bar) {
  return place_in(smem_u32(bar), 0);
}
// Load into this CTA's shared memory; the bytes are counted on the leader's barrier.
TW_DEV void tma_load_pair(void* dst, const CUtensorMap* map, uint32_t leader_bar, int c0, int c1) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4}], [%2];"
      ::"r"(smem_u32(dst)), "l"(reinterpret_cast<uint64_t>(map)), "r"(leader_bar), "r"(c0), "r"(c1)
      : "memory");
}
TW_DEV void tmem_alloc_pair(uint32_t* result, uint32_t cols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;"
               ::"r"(smem_u32(result)), "r"(cols) : "memory");
}
TW_DEV void tmem_relinquish_pair() {
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
TW_DEV void tmem_dealloc_pair(uint32_t addr, uint32_t cols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols)
               : "memory");
}
TW_DEV void umma_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}\n"
      ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(accumulate) : "memory");
}
// Arrive on `bar` of both CTAs when the MMAs issued so far have completed.
TW_DEV void umma_commit_pair(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
      " [%0], %1;"
      ::"r"(smem_u32(bar)), "h"((uint16_t)3) : "memory");
}
TW_DEV void arrive_leader(uint32_t leader_bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(leader_bar)
               : "memory");
}
// Bounded wait for arrivals from both CTAs.
TW_DEV bool wait_pair(uint64_t* bar, uint32_t parity, volatile int* abort, uint64_t timeout_ns) {
  uint64_t t0 = 0;
  for (uint32_t i = 0;; ++i) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}\n"
        : "=r"(ok) : "r"(smem_u32(bar)), "r"(parity), "r"(20000u) : "memory");
    if (ok) return true;
    if ((i & 31u) == 31u) {
      if (*abort) return false;
      const uint64_t now = globaltimer_ns();
      if (t0 == 0) t0 = now;
      else if (now - t0 > timeout_ns) return false;
    }
  }
}

// ----------------------------------------------------------------- staging --
TW_DEV void tma_load_own(uint32_t dst, const CUtensorMap* map, uint64_t* bar, int c0, int c1) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4}], [%2];"
      ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1)
      : "memory");
}
TW_DEV void tma_store(const CUtensorMap* map, uint32_t src, int c0, int c1) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%2, %3}], [%1];"
               ::"l"(reinterpret_cast<uint64_t>(map)), "r"(src), "r"(c0), "r"(c1) : "memory");
}
TW_DEV void stores_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
template <int PENDING>
TW_DEV void stores_read() {  // all but the newest PENDING groups have read their slabs
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(PENDING) : "memory");
}
TW_DEV void stores_done() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }
TW_DEV void fence_async_proxy() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
// A lane's row of a slab: 16-byte chunk q (8 columns) in its swizzled place.
TW_DEV uint32_t slab_chunk(uint32_t slab, int lane, int q) {
  return slab + lane * 64 + ((q ^ ((lane >> 1) & 3)) << 4);
}
// Chunks first and first + 1 of a lane's row: 16 columns.
TW_DEV void slab_write16(uint32_t slab, int lane, int first, const uint32_t (&w)[8]) {
#pragma unroll
  for (int q = 0; q < 2; ++q)
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};"
                 ::"r"(slab_chunk(slab, lane, first + q)), "r"(w[4 * q]), "r"(w[4 * q + 1]),
                   "r"(w[4 * q + 2]), "r"(w[4 * q + 3]) : "memory");
}
TW_DEV void slab_write(uint32_t slab, int lane, const uint32_t (&w)[16]) {
#pragma unroll
  for (int q = 0; q < 4; ++q)
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};"
                 ::"r"(slab_chunk(slab, lane, q)), "r"(w[4 * q]), "r"(w[4 * q + 1]),
                   "r"(w[4 * q + 2]), "r"(w[4 * q + 3]) : "memory");
}
TW_DEV void slab_read(uint32_t slab, int lane, uint32_t (&w)[16]) {
#pragma unroll
  for (int q = 0; q < 4; ++q)
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(w[4 * q]), "=r"(w[4 * q + 1]), "=r"(w[4 * q + 2]), "=r"(w[4 * q + 3])
                 : "r"(slab_chunk(slab, lane, q)) : "memory");
}

// An fp32 row of a double slab: 32 columns, 128 bytes, 128-byte swizzle.
TW_DEV void slab_write_f32(uint32_t slab, int lane, const uint32_t (&w)[32]) {
#pragma unroll
  for (int q = 0; q < 8; ++q)
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};"
                 ::"r"(slab + lane * 128 + ((q ^ (lane & 7)) << 4)), "r"(w[4 * q]),
                   "r"(w[4 * q + 1]), "r"(w[4 * q + 2]), "r"(w[4 * q + 3]) : "memory");
}

struct Maps {
  CUtensorMap a[3], b[3];
  CUtensorMap e[5];  // of the epilogue, boxes of 32 columns x 32 rows
  CUtensorMap o[4];  // results, the same boxes
};

// ------------------------------------------------------------------- tiles --
// One launch's tiles.  Order: groups of kGroupM tile rows, within a group down the
// rows first, so the pairs at work share few rows of A and few of B in L2 (groups of 1
// to 16 rows measure alike at these sizes; the weights of larger ones leave L2).  When the
// last round of tiles would leave half of the pairs idle, its tiles are cut into
// two of 128 columns (`full` tiles before them; MN-major B only), each in about 0.75 of
// a whole one's time.  A launch of few tiles, all of them cut so, also divides the
// reduction into `splits`.
constexpr int kGroupM = 8;
struct Tile {
  int product, m, col, width;  // tile row; first column (of units: dual B), columns
  int k0, k1, k_half;          // k-blocks, and half of the whole reduction's
};
struct Tiles {
  int m, n, products, kblocks, full, count, splits;
  TW_DEV Tile at(int i, int n_step) const {
    Tile t;
    const int split = i % splits;
    i /= splits;
    t.k0 = split * kblocks / splits;
    t.k1 = (split + 1) * kblocks / splits;
    t.k_half = kblocks / 2;
    int tile = i, part = 0;
    t.width = kBN;
    if (i >= full) {
      tile = full + ((i - full) >> 1);
      part = (i - full) & 1;
      t.width = kBN / 2;
    }
    t.product = tile / (m * n);
    const int k = tile - t.product * (m * n);
    const int group = k / (kGroupM * n), in = k - group * (kGroupM * n);
    const int rows = m - group * kGroupM < kGroupM ? m - group * kGroupM : kGroupM;
    const int tn = in / rows;
    t.m = group * kGroupM + in - tn * rows;
    t.col = tn * n_step + part * (kBN / 2);
    return t;
  }
};

// Two products' tiles in one launch: `lead` (product 0, the longer units) and then `rest`
// (products 1 on).
struct LeadTiles {
  Tiles lead, rest;
  int count;
  TW_DEV Tile at(int i, int n_step) const {
    if (i < lead.count) return lead.at(i, n_step);
    Tile t = rest.at(i - lead.count, n_step);
    ++t.product;
    return t;
  }
};

// What an epilogue warp works with.
struct EpiWarp {
  int warp, lane, q, half, rank;  // index among the epilogue warps; lane quarter; column half
  int pair, pairs;
  uint32_t slabs;     // its staging
  uint64_t* loaded;   // its barrier of staged loads
  volatile int* abort;
  uint64_t timeout_ns;
  TW_DEV int row0(const Tile& t) const { return t.m * 2 * kBM + rank * kBM + q * 32; }
  TW_DEV uint32_t slab(int i) const { return slabs + i * kSlabBytes; }
};

// ---------------------------------------------------------------- epilogues --
// Operand layout of a product:
//   kDualB  B is gate (first CTA) beside up (second CTA), 128 units each
//   kAMN    A is MN-major: A[m][k] read from a [K][M] row-major tensor
//   kBMN    B is MN-major: B[n][k] read from a [K][N] row-major tensor
//   kDualK  the reduction runs over (a[0], b[0]) and then (a[1], b[1])
//   kGroup  independent products of one shape, (a[p], b[p]) -> out[p]
//   kStages, kSlabs  stages of the ring, and staging slabs of an epilogue warp
// begin() comes before the first tile, run() once a tile (false: a wait ran out),
// end() after the last.
template <bool DUALB, bool AMN, bool BMN, bool DUALK, bool GROUP, int STAGES, int SLABS>
struct Operands {
  static constexpr bool kDualB = DUALB, kAMN = AMN, kBMN = BMN, kDualK = DUALK, kGroup = GROUP;
  static constexpr bool kMixed = false;
  static constexpr int kStages = STAGES, kSlabs = SLABS;
  using Set = Tiles;
  static constexpr int kStep = DUALB ? 128 : kBN;  // output columns a tile
};

// Counters of the launch behind this one, cleared by one warp.
TW_DEV void clear(const EpiWarp& w, uint32_t* words, int n) {
  if (w.pair == 0 && w.rank == 0 && w.warp == 0)
    for (int i = w.lane; i < n; i += 32) words[i] = 0u;
}

// Two slabs in turns: a warp's 32 x 32 of one matrix after the other goes into the slab
// whose last store but one has been read, and from there to global memory.
struct Turns {
  int turn;
  TW_DEV uint32_t take(const EpiWarp& w, int first) {
    if (w.lane == 0) stores_read<1>();
    __syncwarp();
    return w.slab(first + turn);
  }
  TW_DEV void give(const EpiWarp& w, const CUtensorMap* to, int first, int col, int row) {
    fence_async_proxy();
    __syncwarp();
    if (w.lane == 0) {  // rows and columns past the end are not stored
      tma_store(to, w.slab(first + turn), col, row);
      stores_commit();
    }
    turn ^= 1;
  }
};

// h = act(z) u from the unrounded z and u; with KEEP z and u are kept (bf16) for the
// backward, through the same two slabs, which leaves the ring its six stages (a slab for
// each of the three leaves five; the two measure alike: a step of 1003 tokens at 1024 x 4096
// takes 97 to 104 us from one machine to the next).
template <bool KEEP>
struct EpiGateUp : Operands<true, false, false, false, false, 6, 2> {
  int T, F, act;
  uint32_t* arrived;  // the next product's arrival counters, cleared here
  int n_arrived;
  // maps.e: h, z, u
  using State = Turns;
  TW_DEV void begin(State& s, const EpiWarp& w, const Maps&, const Tiles&) const {
    s.turn = 0;
    clear(w, arrived, n_arrived);
  }
  template <int ACT>
  TW_DEV void rows(State& s, const EpiWarp& w, const Maps& maps, uint32_t taddr,
                   const Tile& t) const {
    const int row0 = w.row0(t);
    if (row0 >= T) return;  // uniform over the warp, as all conditions below
#pragma unroll 1
    for (int c = w.half * 64; c < w.half * 64 + 64; c += 32) {
      const int col = t.col + c;
      if (col >= F) break;
      uint32_t zr[32], ur[32], out[16];
      __syncwarp();
      tmem_ld_32x32b_x32(taddr + c, zr);
      tmem_ld_32x32b_x32(taddr + 128 + c, ur);
      tmem_ld_wait();
      if (KEEP) {
#pragma unroll
        for (int i = 0; i < 16; ++i)
          out[i] = pack_bf16x2(__uint_as_float(zr[2 * i]), __uint_as_float(zr[2 * i + 1]));
        slab_write(s.take(w, 0), w.lane, out);
        s.give(w, &maps.e[1], 0, col, row0);
#pragma unroll
        for (int i = 0; i < 16; ++i)
          out[i] = pack_bf16x2(__uint_as_float(ur[2 * i]), __uint_as_float(ur[2 * i + 1]));
        slab_write(s.take(w, 0), w.lane, out);
        s.give(w, &maps.e[2], 0, col, row0);
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        float a0, a1, da;
        activate<ACT>(__uint_as_float(zr[2 * i]), a0, da);
        activate<ACT>(__uint_as_float(zr[2 * i + 1]), a1, da);
        out[i] = pack_bf16x2(a0 * __uint_as_float(ur[2 * i]), a1 * __uint_as_float(ur[2 * i + 1]));
      }
      slab_write(s.take(w, 0), w.lane, out);
      s.give(w, &maps.e[0], 0, col, row0);
    }
  }
  TW_DEV bool run(State& s, const EpiWarp& w, const Maps& maps, const Tiles&, uint32_t taddr,
                  const Tile& t, int) const {
    switch (act) {
      case TW_ACT_RELU: rows<TW_ACT_RELU>(s, w, maps, taddr, t); break;
      case TW_ACT_SILU: rows<TW_ACT_SILU>(s, w, maps, taddr, t); break;
      case TW_ACT_GELU: rows<TW_ACT_GELU>(s, w, maps, taddr, t); break;
      default: rows<TW_ACT_GELU_TANH>(s, w, maps, taddr, t); break;
    }
    return true;
  }
  TW_DEV void end(State&, const EpiWarp& w) const {
    if (w.lane == 0) stores_done();
  }
};

// From dh and the kept z and u: h again (bf16, the operand of dWd: keeping z and u
// alone holds a third less between the passes), du = dh act(z), dz = dh u act'(z).
// z and u are bf16 because they are as large as all else that a step holds; with the
// operands' own roundings the gradients are 0.0035 off in the 2-norm, against 0.0024
// that the rounding of operands and results alone costs.  Bound by the TMA unit, which
// moves five matrices beside the operands: 437,000 cycles at 8192 x 2048 x 8192, 291,000
// without them, 432,000 without the activation's arithmetic.
// Slabs: z, u, loaded for the next 32 columns as soon as these are in registers; h,
// du, dz.
struct EpiBackward : Operands<false, false, false, false, false, 4, 5> {
  int T, F, act;
  uint32_t* arrived;  // as in EpiGateUp
  int n_arrived;
  // maps.e: h, z, u, du, dz
  struct State {
    uint32_t chunk;            // 32-column chunks worked on; the barrier's phase is chunk & 1
    int next_tile;             // the chunk to load next (next_tile >= count: none):
    int next_c;                // its column in the warp's half of the tile,
    int next_col, next_row;    // the half's first column and the warp's first row
  };
  TW_DEV void place(State& s, const EpiWarp& w, const Tiles& tiles) const {
    const Tile t = tiles.at(s.next_tile, kStep);
    s.next_col = t.col + w.half * 128;
    s.next_row = w.row0(t);
  }
  // Moves on to the first chunk at or behind next_c that has rows and columns.
  TW_DEV void seek(State& s, const EpiWarp& w, const Tiles& tiles) const {
    while (s.next_tile < tiles.count) {
      if (s.next_c < 128 && s.next_row < T && s.next_col + s.next_c < F) return;
      s.next_tile += w.pairs;
      s.next_c = 0;
      if (s.next_tile < tiles.count) place(s, w, tiles);
    }
  }
  TW_DEV void load_next(State& s, const EpiWarp& w, const Maps& maps, const Tiles& tiles) const {
    if (s.next_tile >= tiles.count) return;
    if (w.lane == 0) {
      mbar_arrive_expect_tx(w.loaded, 2 * kSlabBytes);
      tma_load_own(w.slab(0), &maps.e[1], w.loaded, s.next_col + s.next_c, s.next_row);
      tma_load_own(w.slab(1), &maps.e[2], w.loaded, s.next_col + s.next_c, s.next_row);
    }
    s.next_c += 32;
    seek(s, w, tiles);
  }
  TW_DEV void begin(State& s, const EpiWarp& w, const Maps& maps, const Tiles& tiles) const {
    clear(w, arrived, n_arrived);
    s.chunk = 0;
    s.next_tile = w.pair;
    s.next_c = 0;
    if (s.next_tile < tiles.count) place(s, w, tiles);
    seek(s, w, tiles);
    load_next(s, w, maps, tiles);
  }
  template <int ACT>
  TW_DEV bool rows(State& s, const EpiWarp& w, const Maps& maps, const Tiles& tiles,
                   uint32_t taddr, const Tile& t) const {
    const int row0 = w.row0(t);
    if (row0 >= T) return true;  // uniform over the warp, as all conditions below
#pragma unroll 1
    for (int c = w.half * 128; c < w.half * 128 + 128; c += 32) {
      const int col = t.col + c;
      if (col >= F) break;
      uint32_t zw[16], uw[16];
      bool ok = mbar_wait(w.loaded, s.chunk & 1u, w.abort, w.timeout_ns);
      if (!__all_sync(0xFFFFFFFFu, ok)) return false;
      slab_read(w.slab(0), w.lane, zw);
      slab_read(w.slab(1), w.lane, uw);
      ++s.chunk;
      __syncwarp();  // all lanes have read
      load_next(s, w, maps, tiles);
#pragma unroll
      for (int part = 0; part < 2; ++part) {  // 16 columns at a time, for the registers
        uint32_t r[16], hw[8], duw[8], dzw[8];
        __syncwarp();
        tmem_ld_x16(taddr + c + part * 16, r);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float dh0 = __uint_as_float(r[2 * i]), dh1 = __uint_as_float(r[2 * i + 1]);
          const uint32_t zp = zw[part * 8 + i], up = uw[part * 8 + i];
          const float u0 = bf16_lo(up), u1 = bf16_hi(up);
          float a0, a1, d0, d1;
          activate<ACT>(bf16_lo(zp), a0, d0);
          activate<ACT>(bf16_hi(zp), a1, d1);
          hw[i] = pack_bf16x2(a0 * u0, a1 * u1);
          duw[i] = pack_bf16x2(dh0 * a0, dh1 * a1);
          dzw[i] = pack_bf16x2(dh0 * u0 * d0, dh1 * u1 * d1);
        }
        if (part == 0) {  // the last stores have read their slabs
          if (w.lane == 0) stores_read<0>();
          __syncwarp();
        }
        slab_write16(w.slab(2), w.lane, part * 2, hw);
        slab_write16(w.slab(3), w.lane, part * 2, duw);
        slab_write16(w.slab(4), w.lane, part * 2, dzw);
      }
      fence_async_proxy();
      __syncwarp();
      if (w.lane == 0) {
        tma_store(&maps.e[0], w.slab(2), col, row0);
        tma_store(&maps.e[3], w.slab(3), col, row0);
        tma_store(&maps.e[4], w.slab(4), col, row0);
        stores_commit();
      }
    }
    return true;
  }
  TW_DEV bool run(State& s, const EpiWarp& w, const Maps& maps, const Tiles& tiles, uint32_t taddr,
                  const Tile& t, int) const {
    switch (act) {
      case TW_ACT_RELU: return rows<TW_ACT_RELU>(s, w, maps, tiles, taddr, t);
      case TW_ACT_SILU: return rows<TW_ACT_SILU>(s, w, maps, tiles, taddr, t);
      case TW_ACT_GELU: return rows<TW_ACT_GELU>(s, w, maps, tiles, taddr, t);
      default: return rows<TW_ACT_GELU_TANH>(s, w, maps, tiles, taddr, t);
    }
  }
  TW_DEV void end(State&, const EpiWarp& w) const {
    if (w.lane == 0) stores_done();
  }
};

// 32 bf16 columns of one row, stored 8 at a time as far as they exist.
TW_DEV void store_bf16(uint16_t* dst, const uint32_t (&w)[16], int left) {
#pragma unroll
  for (int q = 0; q < 4; ++q)
    if (left > 8 * q)
      reinterpret_cast<uint4*>(dst)[q] =
          make_uint4(w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]);
}

// Plain results [M][N], rounded once to bf16 or stored in fp32: 32 x 32 at a time
// through two slabs in turns (fp32: one of twice the size).  Stores of a row a lane
// straight from registers bound short reductions by the epilogue (a step of 64 tokens at
// 2048 x 8192: 130 us against 112).
struct StoreState {
  int turn;
  bool wide;  // the newest store is fp32, out of both slabs
};
template <class Ops>
struct EpiStore : Ops {
  int M, N;
  bool bf16;
  void* out[3];
  int first_map;     // maps.o of its first product
  float* parts;      // partial sums and arrival counters of a divided reduction
  uint32_t* arrived;
  using State = StoreState;
  TW_DEV void begin(State& s, const EpiWarp&, const Maps&, const Tiles&) const {
    s.turn = 0;
    s.wide = false;
  }
  // 32 columns of this lane's row.
  TW_DEV void store(const Tile& t, int row, int col, const uint32_t (&r)[32]) const {
    if (row >= M) return;
    const size_t off = (size_t)row * N + col;
    if (bf16) {
      uint32_t v[16];
#pragma unroll
      for (int i = 0; i < 16; ++i)
        v[i] = pack_bf16x2(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1]));
      store_bf16(static_cast<uint16_t*>(out[t.product]) + off, v, N - col);
    } else {
      float4* dst = reinterpret_cast<float4*>(static_cast<float*>(out[t.product]) + off);
#pragma unroll
      for (int q = 0; q < 8; ++q)
        if (N - col > 4 * q)
          dst[q] = make_float4(__uint_as_float(r[4 * q]), __uint_as_float(r[4 * q + 1]),
                               __uint_as_float(r[4 * q + 2]), __uint_as_float(r[4 * q + 3]));
    }
  }
  // A divided reduction (width 128: 64 columns a warp).  Every part writes its sums;
  // the warp that arrives last at its place adds all parts in their order, so the
  // result does not depend on which one that is, and no one waits.
  TW_DEV void join(const EpiWarp& w, const Tiles& tiles, uint32_t taddr, const Tile& t,
                   int index) const {
    constexpr int kPlace = 2 * 8 * 32 * 4;  // floats of a warp's 32 x 64 sums
    const int S = tiles.splits, unit = index / S, split = index - unit * S;
    const int place = (unit * 2 + w.rank) * kEpiWarps + w.warp;
    const int col0 = t.col + w.half * 64;
    if (col0 >= N) return;  // uniform
    float4* mine = reinterpret_cast<float4*>(parts + ((size_t)place * S + split) * kPlace) + w.lane;
#pragma unroll 1
    for (int c = 0; c < 2; ++c) {
      uint32_t r[32];
      __syncwarp();
      tmem_ld_32x32b_x32(taddr + w.half * 64 + c * 32, r);
      tmem_ld_wait();
#pragma unroll
      for (int q = 0; q < 8; ++q)
        mine[(c * 8 + q) * 32] =
            make_float4(__uint_as_float(r[4 * q]), __uint_as_float(r[4 * q + 1]),
                        __uint_as_float(r[4 * q + 2]), __uint_as_float(r[4 * q + 3]));
    }
    __threadfence();
    __syncwarp();
    uint32_t before = 0;
    if (w.lane == 0) before = atomicAdd(&arrived[place], 1u);
    before = __shfl_sync(0xFFFFFFFFu, before, 0);
    if ((int)before != S - 1) return;
    __threadfence();
    const float4* all = reinterpret_cast<const float4*>(parts + (size_t)place * S * kPlace) + w.lane;
#pragma unroll 1
    for (int c = 0; c < 2; ++c) {
      float4 v[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) v[q] = __ldcg(all + (c * 8 + q) * 32);
#pragma unroll 1
      for (int k = 1; k < S; ++k) {
        float4 o[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) o[q] = __ldcg(all + (size_t)k * (kPlace / 4) + (c * 8 + q) * 32);
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          v[q].x += o[q].x; v[q].y += o[q].y; v[q].z += o[q].z; v[q].w += o[q].w;
        }
      }
      uint32_t r[32];
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        r[4 * q] = __float_as_uint(v[q].x);
        r[4 * q + 1] = __float_as_uint(v[q].y);
        r[4 * q + 2] = __float_as_uint(v[q].z);
        r[4 * q + 3] = __float_as_uint(v[q].w);
      }
      if (col0 + c * 32 < N) store(t, w.row0(t) + w.lane, col0 + c * 32, r);
    }
  }
  TW_DEV bool run(State& s, const EpiWarp& w, const Maps& maps, const Tiles& tiles, uint32_t taddr,
                  const Tile& t, int index) const {
    if (tiles.splits > 1) {
      join(w, tiles, taddr, t, index);
      return true;
    }
    const int row0 = w.row0(t), part = t.width / 2;
    if (row0 >= M) return true;  // uniform over the warp, as all conditions below
    const CUtensorMap* to = &maps.o[first_map + t.product];
#pragma unroll 1
    for (int c = w.half * part; c < w.half * part + part; c += 32) {
      const int col = t.col + c;
      if (col >= N) break;
      uint32_t r[32];
      __syncwarp();
      tmem_ld_32x32b_x32(taddr + c, r);
      // The last stores from this slab have read it.  Where dx and the weight gradients share
      // a launch, a bf16 chunk may follow an fp32 one, whose store reads both slabs.
      if (w.lane == 0) {
        if (bf16 && !s.wide) stores_read<1>();
        else stores_read<0>();
      }
      s.wide = !bf16;
      __syncwarp();
      tmem_ld_wait();
      const uint32_t slab = w.slab(bf16 ? s.turn : 0);
      if (bf16) {
        uint32_t v[16];
#pragma unroll
        for (int i = 0; i < 16; ++i)
          v[i] = pack_bf16x2(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1]));
        slab_write(slab, w.lane, v);
      } else {
        slab_write_f32(slab, w.lane, r);
      }
      fence_async_proxy();
      __syncwarp();
      if (w.lane == 0) {  // rows and columns past the end are not stored
        tma_store(to, slab, col, row0);
        stores_commit();
      }
      s.turn ^= 1;
    }
    return true;
  }
  TW_DEV void end(State&, const EpiWarp& w) const {
    if (w.lane == 0) stores_done();
  }
};
using OpsDown = Operands<false, false, true, false, false, 6, 2>;
using OpsDx = Operands<false, false, true, true, false, 6, 2>;
using OpsGrads = Operands<false, true, true, false, true, 6, 2>;

// dx and the weight gradients in one launch, where dx has few tiles: the weight
// gradients fill the pairs that it leaves idle (a step of 1003 tokens, d = 1024, F = 4096:
// 106.6 -> 102.7 us).  Both write through the same slabs, each in its own type.  Operands of the weight gradients:
// a[2] and e[2] (dWd), e[0] and e[3] (dWu), e[1] and e[3] (dWg).
struct EpiInputs : Operands<false, false, true, true, false, 6, 2> {
  static constexpr bool kMixed = true;
  using Set = LeadTiles;
  EpiStore<OpsDx> dx;
  EpiStore<OpsGrads> grads;
  using State = StoreState;
  TW_DEV void begin(State& s, const EpiWarp&, const Maps&, const LeadTiles&) const {
    s.turn = 0;
    s.wide = false;
  }
  TW_DEV bool run(State& s, const EpiWarp& w, const Maps& maps, const LeadTiles& tiles,
                  uint32_t taddr, const Tile& t, int index) const {
    if (t.product == 0) return dx.run(s, w, maps, tiles.lead, taddr, t, index);
    Tile one = t;
    --one.product;
    return grads.run(s, w, maps, tiles.rest, taddr, one, index - tiles.lead.count);
  }
  TW_DEV void end(State& s, const EpiWarp& w) const { dx.end(s, w); }
};

// ------------------------------------------------------------------- kernel --
template <class Epi>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    pair_gemm_kernel(const __grid_constant__ Maps maps, const typename Epi::Set tiles,
                     const Epi epi, int32_t* status, unsigned long long timeout_ns,
                     int withhold_loads) {
  constexpr int kStages = Epi::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* slabs = smem + Layout<Epi>::kRing;
  auto* sm = reinterpret_cast<Tail*>(slabs + Layout<Epi>::kStaging);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)cta_rank();
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  const int count = tiles.count;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&sm->full[s], 1);
      mbar_init(&sm->empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&sm->tmem_full[a], 1);
      mbar_init(&sm->tmem_empty[a], 2 * kEpiWarps);
    }
    mbar_init(&sm->drain, 1);
    for (int w = 0; w < kEpiWarps; ++w) mbar_init(&sm->loaded[w], 1);
    sm->abort = 0;
    sm->never = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc_pair(&sm->tmem_base, kTmemCols);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_meet();
  tc_fence_after();
  const uint32_t tmem_base = sm->tmem_base;
  volatile int* abort = &sm->abort;
  pdl_wait();
  pdl_launch_next();

  if (warp == 0) {
    if (elect_one()) {
      // ------------------------------------------------------ TMA producer --
      uint32_t it = 0;
      bool ok = true;
      // withhold_loads (a test of the bounded waits): no operand is loaded
      for (int tile = pair; tile < count && ok && !withhold_loads; tile += pairs) {
        const Tile t = tiles.at(tile, Epi::kStep);
        const int m0 = t.m * 2 * kBM + rank * kBM;
        // dual B: this CTA's weight, 128 units; otherwise its half of the columns
        const int n0 = Epi::kDualB ? t.col : t.col + rank * (t.width / 2);
        const bool narrow = Epi::kBMN && t.width < kBN;
        const bool grads = Epi::kMixed && t.product > 0;
        const uint32_t bytes = 2 * (kHalfBytes + (narrow ? kHalfBytes / 2 : kHalfBytes));
        for (int kb = t.k0; kb < t.k1; ++kb) {
          const uint32_t s = it % kStages;
          if (!mbar_wait(&sm->empty[s], ((it / kStages) & 1u) ^ 1u, abort, timeout_ns)) {
            ok = false;
            break;
          }
          uint8_t* a = smem + (size_t)s * kStageBytes;
          uint8_t* b = a + kHalfBytes;
          const uint32_t bar = leader_addr(&sm->full[s]);
          if (rank == 0) mbar_arrive_expect_tx(&sm->full[s], bytes);
          const bool second = Epi::kDualK && !grads && kb >= t.k_half;
          const int k0 = (second ? kb - t.k_half : kb) * kBK;
          const CUtensorMap* ma = &maps.a[Epi::kGroup ? t.product : second ? 1 : 0];
          const CUtensorMap* mb =
              &maps.b[Epi::kGroup ? t.product : Epi::kDualB ? rank : second ? 1 : 0];
          if (grads) {
            ma = t.product == 1 ? &maps.a[2] : &maps.e[t.product - 2];
            mb = t.product == 1 ? &maps.e[2] : &maps.e[3];
          }
          if (Epi::kAMN || grads) {  // boxes of 64 k-rows x 64 columns
            tma_load_pair(a, ma, bar, m0, k0);
            tma_load_pair(a + kHalfBytes / 2, ma, bar, m0 + 64, k0);
          } else {
            tma_load_pair(a, ma, bar, k0, m0);
          }
          if (Epi::kBMN) {
            tma_load_pair(b, mb, bar, n0, k0);
            if (!narrow) tma_load_pair(b + kHalfBytes / 2, mb, bar, n0 + 64, k0);
          } else {
            tma_load_pair(b, mb, bar, k0, n0);
          }
          ++it;
        }
      }
      if (!ok) {
        *abort = 1;
        set_status(status, kStatusTimeout);
        // copies in flight land within microseconds; the pair leaves together,
        // after this wait in both CTAs
        const uint64_t t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < 1000000u) {}
      }
    }
  } else if (warp == 1) {
    if (rank == 0 && elect_one()) {
      // -------------------------------------------------------- MMA issuer --
      uint32_t it = 0, tl = 0;
      bool ok = true;
      for (int tile = pair; tile < count && ok; tile += pairs, ++tl) {
        const uint32_t acc = tl & 1u;
        if (!wait_pair(&sm->tmem_empty[acc], ((tl >> 1) & 1u) ^ 1u, abort, timeout_ns)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t d = tmem_base + acc * kBN;
        const Tile t = tiles.at(tile, Epi::kStep);
        const bool amn = Epi::kAMN || (Epi::kMixed && t.product > 0);
        const uint32_t idesc = idesc_bf16_f32(2 * kBM, t.width, amn, Epi::kBMN);
        for (int kb = t.k0; kb < t.k1; ++kb) {
          const uint32_t s = it % kStages;
          if (!mbar_wait(&sm->full[s], (it / kStages) & 1u, abort, timeout_ns)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t a = smem_u32(smem + (size_t)s * kStageBytes), b = a + kHalfBytes;
#pragma unroll
          for (int kk = 0; kk < kBK / 16; ++kk) {
            // K-major: 16 k further along the swizzled row; MN-major: 16 k-rows
            // further, boxes of 64 columns 8 KB apart
            const uint64_t ad = amn ? sdesc_mnmajor_sw128(a + kk * 2048, kBK * 64 * 2)
                                    : sdesc_kmajor_sw128(a + kk * 32);
            const uint64_t bd = Epi::kBMN ? sdesc_mnmajor_sw128(b + kk * 2048, kBK * 64 * 2)
                                          : sdesc_kmajor_sw128(b + kk * 32);
            umma_pair(d, ad, bd, idesc, kb != t.k0 || kk != 0 ? 1u : 0u);
          }
          umma_commit_pair(&sm->empty[s]);
          ++it;
        }
        if (!ok) break;
        umma_commit_pair(&sm->tmem_full[acc]);
      }
      if (!ok) {
        *abort = 1;
        set_status(status, kStatusTimeout);
      }
      // every MMA issued here has completed once `drain` flips
      umma_commit_pair(&sm->drain);
      mbar_wait(&sm->drain, 0, &sm->never, kWaitTimeoutNs);
    }
  } else {
    // ---------------------------------------------------------- epilogue -----
    EpiWarp w;
    w.warp = warp - 2;
    w.lane = lane;
    w.q = warp & 3;  // TMEM lane quarter this warp may access
    w.half = w.warp >> 2;
    w.rank = rank;
    w.pair = pair;
    w.pairs = pairs;
    w.slabs = smem_u32(slabs) + w.warp * Epi::kSlabs * kSlabBytes;
    w.loaded = &sm->loaded[w.warp];
    w.abort = abort;
    w.timeout_ns = timeout_ns;
    typename Epi::State state;
    epi.begin(state, w, maps, tiles);
    uint32_t tl = 0;
    for (int tile = pair; tile < count; tile += pairs, ++tl) {
      const Tile t = tiles.at(tile, Epi::kStep);
      const uint32_t acc = tl & 1u;
      bool ok = mbar_wait(&sm->tmem_full[acc], (tl >> 1) & 1u, abort, timeout_ns);
      ok = __all_sync(0xFFFFFFFFu, ok);
      if (ok) {
        tc_fence_after();
        ok = epi.run(state, w, maps, tiles,
                     tmem_base + ((uint32_t)(w.q * 32) << 16) + acc * kBN, t, tile);
      }
      if (!ok) {
        *abort = 1;
        if (lane == 0) {
          set_status(status, kStatusTimeout);
          const uint64_t t0 = globaltimer_ns();  // as in the producer
          while (globaltimer_ns() - t0 < 1000000u) {}
        }
        break;
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive_leader(leader_addr(&sm->tmem_empty[acc]));
    }
    epi.end(state, w);
  }
  tc_fence_before();
  __syncwarp();
  __syncthreads();
  cluster_meet();  // no CTA leaves while the other may still arrive on its barriers
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, kTmemCols);
  }
}

// --------------------------------------------------------------------- host --
int most_pairs() { return num_sms() / 2 > 0 ? num_sms() / 2 : 1; }

// Half tiles and divided reductions: a step of 1003 tokens (d 1024, F 4096: 16 tiles of y
// and of dx for 74 pairs) 148 us without them, 137 with (before the later steps).  A part
// keeps 8 k-blocks, about what its join costs.
constexpr int kMinSplitBlocks = 8;
constexpr int kMaxSplits = 8;

// How a product's tiles are dealt out (narrow: with MN-major B).
Tiles plan_tiles(int m, int n, int products, int kblocks, bool narrow) {
  const long long count = (long long)m * n * products;
  Tiles t{m, n, products, kblocks, (int)count, (int)count, 1};
  const int most = most_pairs(), rest = (int)(count % most);
  if (narrow && rest > 0 && 2 * rest <= most) {
    t.full = (int)count - rest;
    t.count = t.full + 2 * rest;
    if (t.full == 0) {
      while (2 * t.splits <= kMaxSplits && 2 * t.splits * t.count <= most &&
             kblocks / (2 * t.splits) >= kMinSplitBlocks)
        t.splits *= 2;
      t.count *= t.splits;
    }
  }
  return t;
}

// Arrival counters and partial sums of a divided reduction, in bytes.
int counters_of(const Tiles& t) { return t.splits > 1 ? t.count / t.splits * 2 * kEpiWarps : 0; }
size_t counter_bytes(const Tiles& t) { return ((size_t)counters_of(t) * 4 + 255) & ~size_t(255); }
size_t split_bytes(const Tiles& t) {
  return t.splits > 1 ? counter_bytes(t) + (size_t)t.count * 2 * kBM * (kBN / 2) * 4 : 0;
}

template <class Epi>
cudaError_t launch_pairs(const Maps& maps, const typename Epi::Set& t, const Epi& epi,
                         unsigned long long withheld_wait_ns, int32_t* status,
                         cudaStream_t stream) {
  if (t.count == 0) return cudaSuccess;
  constexpr size_t smem = Layout<Epi>::kSmem;
  cudaError_t e = set_smem_limit(reinterpret_cast<const void*>(pair_gemm_kernel<Epi>), (int)smem);
  if (e != cudaSuccess) return e;
  const int pairs = t.count < most_pairs() ? t.count : most_pairs();
  return launch_pdl(pair_gemm_kernel<Epi>, dim3(2 * pairs), dim3(kThreads), smem, stream, maps, t,
                    epi, status, withheld_wait_ns ? withheld_wait_ns : kWaitTimeoutNs,
                    withheld_wait_ns ? 1 : 0);
}

// K-major operand: boxes of 64 columns (k) x 128 rows.
bool map_k(CUtensorMap* m, const void* base, uint64_t rows, uint64_t cols) {
  return make_tmap_bf16(m, base, rows, cols, kBK, kBM);
}
// MN-major operand, a [K][MN] row-major tensor: boxes of 64 columns x 64 k-rows.
bool map_mn(CUtensorMap* m, const void* base, uint64_t k_rows, uint64_t cols) {
  return make_tmap_bf16(m, base, k_rows, cols, 64, kBK);
}

// A matrix of the staged epilogues: 32 x 32 boxes.
bool map_slab(CUtensorMap* m, const void* base, uint64_t rows, uint64_t cols) {
  return make_tmap_bf16_sw64(m, base, rows, cols, 32);
}

bool map_result(CUtensorMap* m, const void* base, uint64_t rows, uint64_t cols, bool bf16) {
  return bf16 ? make_tmap_bf16_sw64(m, base, rows, cols, 32)
              : make_tmap_f32(m, base, rows, cols, 32);
}

int div_up(int a, int b) { return a / b + (a % b != 0); }

Tiles down_tiles(int T, int d, int F) {
  return plan_tiles(div_up(T, 2 * kBM), div_up(d, kBN), 1, div_up(F, kBK), true);
}
Tiles dx_tiles(int T, int d, int F) {
  return plan_tiles(div_up(T, 2 * kBM), div_up(d, kBN), 1, 2 * div_up(F, kBK), true);
}
// The tiles' count of any product fits an int.
bool too_large(int T, int d, int F) {
  const long long mt = div_up(T, 2 * kBM), mf = div_up(F, 2 * kBM);
  const long long nf = div_up(F, 128), nd = div_up(d, kBN);
  return mt * nf > 0x3FFFFFFF || mt * nd > 0x3FFFFFFF || 3 * mf * nd > 0x3FFFFFFF;
}

}  // namespace

size_t gated_forward_split_bytes(int T, int d, int F) {
  return T <= kGatedFewMaxT || too_large(T, d, F) ? 0 : split_bytes(down_tiles(T, d, F));
}
size_t gated_backward_split_bytes(int T, int d, int F) {
  return T == 0 || too_large(T, d, F) ? 0 : split_bytes(dx_tiles(T, d, F));
}

cudaError_t launch_gated_forward(const void* x, const void* Wg_t, const void* Wu_t, const void* Wd,
                                 int T, int d, int F, tw_act act, uint16_t* h, uint16_t* z,
                                 uint16_t* u, void* y, tw_dtype y_dtype, void* split,
                                 int32_t* status, cudaStream_t stream) {
  if (too_large(T, d, F)) return cudaErrorInvalidValue;
  const unsigned long long withheld = take_withheld_ffn_wait();
  if (T <= kGatedFewMaxT)
    return launch_gated_few(x, Wg_t, Wu_t, Wd, T, d, F, act, h, z, u, y, y_dtype, withheld, status,
                            stream);
  Maps m1{}, m2{};
  if (!map_k(&m1.a[0], x, T, d) || !map_k(&m1.b[0], Wg_t, F, d) || !map_k(&m1.b[1], Wu_t, F, d) ||
      !map_slab(&m1.e[0], h, T, F) || (z && !map_slab(&m1.e[1], z, T, F)) ||
      (z && !map_slab(&m1.e[2], u, T, F)) || !map_k(&m2.a[0], h, T, F) ||
      !map_mn(&m2.b[0], Wd, F, d) || !map_result(&m2.o[0], y, T, d, y_dtype == TW_BF16))
    return cudaErrorInvalidValue;
  const Tiles t1 = plan_tiles(div_up(T, 2 * kBM), div_up(F, 128), 1, div_up(d, kBK), false);
  const Tiles t2 = down_tiles(T, d, F);
  auto gate_up = [&](auto epi) {
    epi.T = T;
    epi.F = F;
    epi.act = act;
    epi.arrived = static_cast<uint32_t*>(split);
    epi.n_arrived = counters_of(t2);
    return launch_pairs(m1, t1, epi, withheld, status, stream);
  };
  cudaError_t e = z ? gate_up(EpiGateUp<true>{}) : gate_up(EpiGateUp<false>{});
  if (e != cudaSuccess) return e;
  EpiStore<OpsDown> e2;
  e2.M = T;
  e2.N = d;
  e2.bf16 = y_dtype == TW_BF16;
  e2.out[0] = e2.out[1] = e2.out[2] = y;
  e2.first_map = 0;
  e2.arrived = static_cast<uint32_t*>(split);
  e2.parts = reinterpret_cast<float*>(static_cast<char*>(split) + counter_bytes(t2));
  return launch_pairs(m2, t2, e2, withheld, status, stream);
}

cudaError_t launch_gated_backward(const void* x, const void* dy, const void* Wg_t, const void* Wu_t,
                                  const void* Wd, int T, int d, int F, tw_act act,
                                  const uint16_t* z, const uint16_t* u, uint16_t* h, uint16_t* du,
                                  uint16_t* dz, void* dx, tw_dtype dx_dtype, void* dWg_t,
                                  void* dWu_t, void* dWd, tw_dtype dw_dtype, void* split,
                                  int32_t* status, cudaStream_t stream) {
  if (too_large(T, d, F)) return cudaErrorInvalidValue;
  const unsigned long long withheld = take_withheld_ffn_wait();
  Maps m1{}, m2{}, m3{};
  if (!map_k(&m1.a[0], dy, T, d) || !map_k(&m1.b[0], Wd, F, d) || !map_k(&m2.a[0], du, T, F) ||
      !map_k(&m2.a[1], dz, T, F) || !map_mn(&m2.b[0], Wu_t, F, d) ||
      !map_mn(&m2.b[1], Wg_t, F, d) || !map_mn(&m3.a[0], h, T, F) || !map_mn(&m3.a[1], du, T, F) ||
      !map_mn(&m3.a[2], dz, T, F) || !map_mn(&m3.b[0], dy, T, d) || !map_mn(&m3.b[1], x, T, d) ||
      !map_mn(&m3.b[2], x, T, d) || !map_slab(&m1.e[0], h, T, F) || !map_slab(&m1.e[1], z, T, F) ||
      !map_slab(&m1.e[2], u, T, F) || !map_slab(&m1.e[3], du, T, F) ||
      !map_slab(&m1.e[4], dz, T, F) || !map_result(&m2.o[0], dx, T, d, dx_dtype == TW_BF16))
    return cudaErrorInvalidValue;
  void* const grads[3] = {dWd, dWu_t, dWg_t};
  for (int i = 0; i < 3; ++i)
    if (!map_result(&m3.o[i], grads[i], F, d, dw_dtype == TW_BF16)) return cudaErrorInvalidValue;
  EpiBackward e1;
  e1.T = T;
  e1.F = F;
  e1.act = act;
  const Tiles t2 = dx_tiles(T, d, F);
  e1.arrived = static_cast<uint32_t*>(split);
  e1.n_arrived = counters_of(t2);
  const int nd = div_up(d, kBN);
  cudaError_t e = launch_pairs(
      m1, plan_tiles(div_up(T, 2 * kBM), div_up(F, kBN), 1, div_up(d, kBK), false), e1, withheld,
      status, stream);
  if (e != cudaSuccess) return e;
  EpiStore<OpsDx> e2;
  e2.M = T;
  e2.N = d;
  e2.bf16 = dx_dtype == TW_BF16;
  e2.out[0] = e2.out[1] = e2.out[2] = dx;
  e2.first_map = 0;
  e2.arrived = static_cast<uint32_t*>(split);
  e2.parts = reinterpret_cast<float*>(static_cast<char*>(split) + counter_bytes(t2));
  EpiStore<OpsGrads> e3;
  e3.M = F;
  e3.N = d;
  e3.bf16 = dw_dtype == TW_BF16;
  for (int i = 0; i < 3; ++i) e3.out[i] = grads[i];
  e3.first_map = 0;
  e3.arrived = nullptr;
  e3.parts = nullptr;
  Tiles t3 = plan_tiles(div_up(F, 2 * kBM), nd, 3, div_up(T, kBK), true);
  if (t3.splits > 1) {  // small weights: no room is kept for their partial sums
    t3.count /= t3.splits;
    t3.splits = 1;
  }
  if (t2.full == 0) {  // dx leaves pairs idle: one launch for both
    const LeadTiles both{t2, t3, t2.count + t3.count};
    Maps m{};
    m.a[0] = m2.a[0];
    m.a[1] = m2.a[1];
    m.a[2] = m3.a[0];
    m.b[0] = m2.b[0];
    m.b[1] = m2.b[1];
    m.e[0] = m3.a[1];
    m.e[1] = m3.a[2];
    m.e[2] = m3.b[0];
    m.e[3] = m3.b[1];
    EpiInputs e4;
    e4.dx = e2;
    e4.grads = e3;
    e4.grads.first_map = 1;
    m.o[0] = m2.o[0];
    for (int i = 0; i < 3; ++i) m.o[1 + i] = m3.o[i];
    return launch_pairs(m, both, e4, withheld, status, stream);
  }
  e = launch_pairs(m2, t2, e2, withheld, status, stream);
  if (e != cudaSuccess) return e;
  return launch_pairs(m3, t3, e3, withheld, status, stream);
}

}  // namespace tw
