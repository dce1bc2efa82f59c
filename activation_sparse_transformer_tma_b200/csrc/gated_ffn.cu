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
// of the TMEM lanes, each half of the columns).  Every wait is bounded: on timeout
// the CTA flags TW_ERR_TIMEOUT, stops its roles, lets its copies land and meets its
// pair at the last barrier.
#include "tmap.h"
#include "pdl.cuh"
#include "tw_common.cuh"
#include "tw_internal.h"

namespace tw {
namespace {

constexpr int kBM = 128;  // rows of A (and of B) a CTA
constexpr int kBN = 256;  // columns of a tile
constexpr int kBK = 64;   // 64 bf16 = one 128-byte swizzle row
constexpr int kStages = 6;
constexpr int kHalfBytes = kBM * kBK * 2;       // one operand's share of a stage
constexpr int kStageBytes = 2 * kHalfBytes;
constexpr int kEpiWarps = 8;
constexpr int kThreads = 64 + 32 * kEpiWarps;
constexpr int kTmemCols = 2 * kBN;

struct Tail {
  uint64_t full[kStages];
  uint64_t empty[kStages];
  uint64_t tmem_full[2];
  uint64_t tmem_empty[2];
  uint64_t drain;
  uint32_t tmem_base;
  int abort;
  int never;
};
constexpr size_t kSmem = 1024 + (size_t)kStages * kStageBytes + sizeof(Tail);
static_assert(kSmem <= 227 * 1024, "shared memory budget");

// ------------------------------------------------------------- pair helpers --
TW_DEV uint32_t pair_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
TW_DEV void pair_sync() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
// Address of `bar` in the first CTA of the pair.
TW_DEV uint32_t leader_addr(const uint64_t* bar) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(smem_u32(bar)));
  return r;
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

// -------------------------------------------------------------- activations --
// act(z) and act'(z).  exp and the division are the approximate instructions: the
// results are rounded to bf16.
template <int ACT>
TW_DEV void activate(float z, float& a, float& da) {
  if (ACT == TW_ACT_RELU) {
    a = z > 0.f ? z : 0.f;
    da = z > 0.f ? 1.f : 0.f;
    if (z != z) a = da = z;
  } else if (ACT == TW_ACT_SILU) {
    const float p = __fdividef(1.f, 1.f + __expf(-z));
    a = z * p;
    da = p * fmaf(z, 1.f - p, 1.f);
  } else if (ACT == TW_ACT_GELU) {
    const float cdf = 0.5f * (1.f + erff(z * 0.70710678f));
    a = z * cdf;
    da = fmaf(z * 0.39894228f, __expf(-0.5f * z * z), cdf);
  } else {
    // 0.5 (1 + tanh(k)) = 1 / (1 + exp(-2k)) =: p, k = sqrt(2/pi) (z + 0.044715 z^3)
    const float p =
        __fdividef(1.f, 1.f + __expf(-1.5957691f * z * fmaf(0.044715f * z, z, 1.f)));
    a = z * p;
    da = fmaf(z * p * (1.f - p), 1.5957691f * fmaf(0.134145f * z, z, 1.f), p);
  }
}

// ---------------------------------------------------------------- epilogues --
// Operand layout of a product:
//   kDualB  B is gate (first CTA) beside up (second CTA), 128 units each
//   kAMN    A is MN-major: A[m][k] read from a [K][M] row-major tensor
//   kBMN    B is MN-major: B[n][k] read from a [K][N] row-major tensor
//   kDualK  the reduction runs over (a[0], b[0]) and then (a[1], b[1])
//   kGroup  independent products of one shape, (a[p], b[p]) -> out[p]
template <bool DUALB, bool AMN, bool BMN, bool DUALK, bool GROUP>
struct Operands {
  static constexpr bool kDualB = DUALB, kAMN = AMN, kBMN = BMN, kDualK = DUALK, kGroup = GROUP;
};

// 32 bf16 columns of one row, stored 8 at a time as far as they exist.
TW_DEV void store_bf16(uint16_t* dst, const uint32_t (&w)[16], int left) {
#pragma unroll
  for (int q = 0; q < 4; ++q)
    if (left > 8 * q)
      reinterpret_cast<uint4*>(dst)[q] =
          make_uint4(w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]);
}
TW_DEV void load_bf16(const uint16_t* src, uint32_t (&w)[16], int left) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    if (left > 8 * q) v = reinterpret_cast<const uint4*>(src)[q];
    w[4 * q] = v.x; w[4 * q + 1] = v.y; w[4 * q + 2] = v.z; w[4 * q + 3] = v.w;
  }
}

// h = act(z) u from the unrounded z and u; z and u are kept (bf16) for the backward
// where it asks for them.
struct EpiGateUp : Operands<true, false, false, false, false> {
  int T, F, act;
  uint16_t *h, *z, *u;
  template <int ACT>
  TW_DEV void rows(uint32_t taddr, int row, int tile_n, int half) const {
#pragma unroll 1
    for (int c = half * 64; c < half * 64 + 64; c += 32) {
      const int col = tile_n * 128 + c;
      if (col >= F) break;  // uniform
      uint32_t zr[32], ur[32];
      __syncwarp();
      tmem_ld_32x32b_x32(taddr + c, zr);
      tmem_ld_32x32b_x32(taddr + 128 + c, ur);
      tmem_ld_wait();
      if (row >= T) continue;
      const size_t off = (size_t)row * F + col;
      uint32_t w[16];
      if (z) {
#pragma unroll
        for (int i = 0; i < 16; ++i)
          w[i] = pack_bf16x2(__uint_as_float(zr[2 * i]), __uint_as_float(zr[2 * i + 1]));
        store_bf16(z + off, w, F - col);
#pragma unroll
        for (int i = 0; i < 16; ++i)
          w[i] = pack_bf16x2(__uint_as_float(ur[2 * i]), __uint_as_float(ur[2 * i + 1]));
        store_bf16(u + off, w, F - col);
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        float a0, a1, da;
        activate<ACT>(__uint_as_float(zr[2 * i]), a0, da);
        activate<ACT>(__uint_as_float(zr[2 * i + 1]), a1, da);
        w[i] = pack_bf16x2(a0 * __uint_as_float(ur[2 * i]), a1 * __uint_as_float(ur[2 * i + 1]));
      }
      store_bf16(h + off, w, F - col);
    }
  }
  TW_DEV void run(uint32_t taddr, int row, int tile_n, int half, int) const {
    switch (act) {
      case TW_ACT_RELU: rows<TW_ACT_RELU>(taddr, row, tile_n, half); break;
      case TW_ACT_SILU: rows<TW_ACT_SILU>(taddr, row, tile_n, half); break;
      case TW_ACT_GELU: rows<TW_ACT_GELU>(taddr, row, tile_n, half); break;
      default: rows<TW_ACT_GELU_TANH>(taddr, row, tile_n, half); break;
    }
  }
};

// From dh and the kept z and u: h again (bf16, the operand of dWd: keeping z and u
// alone holds a third less between the passes), du = dh act(z), dz = dh u act'(z).
struct EpiBackward : Operands<false, false, false, false, false> {
  int T, F, act;
  const uint16_t *z, *u;
  uint16_t *h, *du, *dz;
  template <int ACT>
  TW_DEV void rows(uint32_t taddr, int row, int tile_n, int half) const {
#pragma unroll 1
    for (int c = half * 128; c < half * 128 + 128; c += 32) {
      const int col = tile_n * kBN + c;
      if (col >= F) break;  // uniform
      uint32_t r[32];
      __syncwarp();
      tmem_ld_32x32b_x32(taddr + c, r);
      tmem_ld_wait();
      if (row >= T) continue;
      const size_t off = (size_t)row * F + col;
      uint32_t zw[16], uw[16], hw[16];
      load_bf16(z + off, zw, F - col);
      load_bf16(u + off, uw, F - col);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float dh0 = __uint_as_float(r[2 * i]), dh1 = __uint_as_float(r[2 * i + 1]);
        const float u0 = bf16_lo(uw[i]), u1 = bf16_hi(uw[i]);
        float a0, a1, d0, d1;
        activate<ACT>(bf16_lo(zw[i]), a0, d0);
        activate<ACT>(bf16_hi(zw[i]), a1, d1);
        hw[i] = pack_bf16x2(a0 * u0, a1 * u1);
        uw[i] = pack_bf16x2(dh0 * a0, dh1 * a1);
        zw[i] = pack_bf16x2(dh0 * u0 * d0, dh1 * u1 * d1);
      }
      store_bf16(h + off, hw, F - col);
      store_bf16(du + off, uw, F - col);
      store_bf16(dz + off, zw, F - col);
    }
  }
  TW_DEV void run(uint32_t taddr, int row, int tile_n, int half, int) const {
    switch (act) {
      case TW_ACT_RELU: rows<TW_ACT_RELU>(taddr, row, tile_n, half); break;
      case TW_ACT_SILU: rows<TW_ACT_SILU>(taddr, row, tile_n, half); break;
      case TW_ACT_GELU: rows<TW_ACT_GELU>(taddr, row, tile_n, half); break;
      default: rows<TW_ACT_GELU_TANH>(taddr, row, tile_n, half); break;
    }
  }
};

// Plain results [M][N], rounded once to bf16 or stored in fp32.
template <class Ops>
struct EpiStore : Ops {
  int M, N;
  bool bf16;
  void* out[3];
  TW_DEV void run(uint32_t taddr, int row, int tile_n, int half, int product) const {
#pragma unroll 1
    for (int c = half * 128; c < half * 128 + 128; c += 32) {
      const int col = tile_n * kBN + c;
      if (col >= N) break;  // uniform
      uint32_t r[32];
      __syncwarp();
      tmem_ld_32x32b_x32(taddr + c, r);
      tmem_ld_wait();
      if (row >= M) continue;
      const size_t off = (size_t)row * N + col;
      if (bf16) {
        uint32_t w[16];
#pragma unroll
        for (int i = 0; i < 16; ++i)
          w[i] = pack_bf16x2(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1]));
        store_bf16(static_cast<uint16_t*>(out[product]) + off, w, N - col);
      } else {
        float4* dst = reinterpret_cast<float4*>(static_cast<float*>(out[product]) + off);
#pragma unroll
        for (int q = 0; q < 8; ++q)
          if (N - col > 4 * q)
            dst[q] = make_float4(__uint_as_float(r[4 * q]), __uint_as_float(r[4 * q + 1]),
                                 __uint_as_float(r[4 * q + 2]), __uint_as_float(r[4 * q + 3]));
      }
    }
  }
};
using OpsDown = Operands<false, false, true, false, false>;
using OpsDx = Operands<false, false, true, true, false>;
using OpsGrads = Operands<false, true, true, false, true>;

struct Maps {
  CUtensorMap a[3], b[3];
};

// Tiles of one launch.  Order: groups of kGroupM tile rows, within a group down
// the rows first, so the pairs at work share few rows of A and few of B in L2.
constexpr int kGroupM = 8;
struct Tiles {
  int m, n, products, kblocks;
  TW_DEV int count() const { return m * n * products; }
  TW_DEV void at(int tile, int& product, int& tm, int& tn) const {
    product = tile / (m * n);
    const int t = tile - product * (m * n);
    const int group = t / (kGroupM * n), in = t - group * (kGroupM * n);
    const int rows = m - group * kGroupM < kGroupM ? m - group * kGroupM : kGroupM;
    tn = in / rows;
    tm = group * kGroupM + in - tn * rows;
  }
};

// ------------------------------------------------------------------- kernel --
template <class Epi>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    pair_gemm_kernel(const __grid_constant__ Maps maps, const Tiles tiles, const Epi epi,
                     int32_t* status, unsigned long long timeout_ns) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  auto* sm = reinterpret_cast<Tail*>(smem + (size_t)kStages * kStageBytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)pair_rank();
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  const int count = tiles.count(), kblocks = tiles.kblocks;

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
  pair_sync();
  tc_fence_after();
  const uint32_t tmem_base = sm->tmem_base;
  volatile int* abort = &sm->abort;
  pdl_wait();
  pdl_launch_next();

  if (warp == 0) {
    if (lane == 0) {
      // ------------------------------------------------------ TMA producer --
      uint32_t it = 0;
      bool ok = true;
      for (int tile = pair; tile < count && ok; tile += pairs) {
        int product, tm, tn;
        tiles.at(tile, product, tm, tn);
        const int m0 = tm * 2 * kBM + rank * kBM;
        // dual B: this CTA's weight, 128 units; otherwise its half of the columns
        const int n0 = Epi::kDualB ? tn * 128 : tn * kBN + rank * 128;
        for (int kb = 0; kb < kblocks; ++kb) {
          const uint32_t s = it % kStages;
          if (!mbar_wait(&sm->empty[s], ((it / kStages) & 1u) ^ 1u, abort, timeout_ns)) {
            ok = false;
            break;
          }
          uint8_t* a = smem + (size_t)s * kStageBytes;
          uint8_t* b = a + kHalfBytes;
          const uint32_t bar = leader_addr(&sm->full[s]);
          if (rank == 0) mbar_arrive_expect_tx(&sm->full[s], 2 * kStageBytes);
          const bool second = Epi::kDualK && kb >= kblocks / 2;
          const int k0 = (second ? kb - kblocks / 2 : kb) * kBK;
          const CUtensorMap* ma = &maps.a[Epi::kGroup ? product : second ? 1 : 0];
          const CUtensorMap* mb =
              &maps.b[Epi::kGroup ? product : Epi::kDualB ? rank : second ? 1 : 0];
          if (Epi::kAMN) {  // boxes of 64 k-rows x 64 columns
            tma_load_pair(a, ma, bar, m0, k0);
            tma_load_pair(a + kHalfBytes / 2, ma, bar, m0 + 64, k0);
          } else {
            tma_load_pair(a, ma, bar, k0, m0);
          }
          if (Epi::kBMN) {
            tma_load_pair(b, mb, bar, n0, k0);
            tma_load_pair(b + kHalfBytes / 2, mb, bar, n0 + 64, k0);
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
    if (lane == 0 && rank == 0) {
      // -------------------------------------------------------- MMA issuer --
      constexpr uint32_t idesc = idesc_bf16_f32(2 * kBM, kBN, Epi::kAMN, Epi::kBMN);
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
        for (int kb = 0; kb < kblocks; ++kb) {
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
            const uint64_t ad = Epi::kAMN ? sdesc_mnmajor_sw128(a + kk * 2048, kBK * 64 * 2)
                                          : sdesc_kmajor_sw128(a + kk * 32);
            const uint64_t bd = Epi::kBMN ? sdesc_mnmajor_sw128(b + kk * 2048, kBK * 64 * 2)
                                          : sdesc_kmajor_sw128(b + kk * 32);
            umma_pair(d, ad, bd, idesc, (kb | kk) != 0 ? 1u : 0u);
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
    const int q = warp & 3;           // TMEM lane quarter this warp may access
    const int half = (warp - 2) >> 2;  // of the tile's columns
    uint32_t tl = 0;
    for (int tile = pair; tile < count; tile += pairs, ++tl) {
      int product, tm, tn;
      tiles.at(tile, product, tm, tn);
      const uint32_t acc = tl & 1u;
      bool ok = mbar_wait(&sm->tmem_full[acc], (tl >> 1) & 1u, abort, timeout_ns);
      ok = __all_sync(0xFFFFFFFFu, ok);
      if (!ok) {
        *abort = 1;
        if (lane == 0) set_status(status, kStatusTimeout);
        break;
      }
      tc_fence_after();
      const int row = tm * 2 * kBM + rank * kBM + q * 32 + lane;
      epi.run(tmem_base + ((uint32_t)(q * 32) << 16) + acc * kBN, row, tn, half, product);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive_leader(leader_addr(&sm->tmem_empty[acc]));
    }
  }
  tc_fence_before();
  __syncwarp();
  __syncthreads();
  pair_sync();  // no CTA leaves while the other may still arrive on its barriers
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, kTmemCols);
  }
}

// --------------------------------------------------------------------- host --
template <class Epi>
cudaError_t launch_pairs(const Maps& maps, const Tiles& t, const Epi& epi, int32_t* status,
                         cudaStream_t stream) {
  const long long count = (long long)t.m * t.n * t.products;
  if (count == 0) return cudaSuccess;
  if (count > 0x3FFFFFFF) return cudaErrorInvalidValue;
  cudaError_t e =
      set_smem_limit(reinterpret_cast<const void*>(pair_gemm_kernel<Epi>), (int)kSmem);
  if (e != cudaSuccess) return e;
  const int most = num_sms() / 2;
  const int pairs = count < most ? (int)count : most;
  return launch_pdl(pair_gemm_kernel<Epi>, dim3(2 * pairs), dim3(kThreads), kSmem, stream, maps, t,
                    epi, status, kWaitTimeoutNs);
}

// K-major operand: boxes of 64 columns (k) x 128 rows.
bool map_k(CUtensorMap* m, const void* base, uint64_t rows, uint64_t cols) {
  return make_tmap_bf16(m, base, rows, cols, kBK, kBM);
}
// MN-major operand, a [K][MN] row-major tensor: boxes of 64 columns x 64 k-rows.
bool map_mn(CUtensorMap* m, const void* base, uint64_t k_rows, uint64_t cols) {
  return make_tmap_bf16(m, base, k_rows, cols, 64, kBK);
}

int div_up(int a, int b) { return a / b + (a % b != 0); }

}  // namespace

cudaError_t launch_gated_forward(const void* x, const void* Wg_t, const void* Wu_t, const void* Wd,
                                 int T, int d, int F, tw_act act, uint16_t* h, uint16_t* z,
                                 uint16_t* u, void* y, tw_dtype y_dtype, int32_t* status,
                                 cudaStream_t stream) {
  Maps m1{}, m2{};
  if (!map_k(&m1.a[0], x, T, d) || !map_k(&m1.b[0], Wg_t, F, d) || !map_k(&m1.b[1], Wu_t, F, d) ||
      !map_k(&m2.a[0], h, T, F) || !map_mn(&m2.b[0], Wd, F, d))
    return cudaErrorInvalidValue;
  EpiGateUp e1;
  e1.T = T;
  e1.F = F;
  e1.act = act;
  e1.h = h;
  e1.z = z;
  e1.u = u;
  const int mt = div_up(T, 2 * kBM);
  cudaError_t e = launch_pairs(m1, Tiles{mt, div_up(F, 128), 1, div_up(d, kBK)}, e1, status, stream);
  if (e != cudaSuccess) return e;
  EpiStore<OpsDown> e2;
  e2.M = T;
  e2.N = d;
  e2.bf16 = y_dtype == TW_BF16;
  e2.out[0] = e2.out[1] = e2.out[2] = y;
  return launch_pairs(m2, Tiles{mt, div_up(d, kBN), 1, div_up(F, kBK)}, e2, status, stream);
}

cudaError_t launch_gated_backward(const void* x, const void* dy, const void* Wg_t, const void* Wu_t,
                                  const void* Wd, int T, int d, int F, tw_act act,
                                  const uint16_t* z, const uint16_t* u, uint16_t* h, uint16_t* du,
                                  uint16_t* dz, void* dx, tw_dtype dx_dtype, void* dWg_t,
                                  void* dWu_t, void* dWd, tw_dtype dw_dtype, int32_t* status,
                                  cudaStream_t stream) {
  Maps m1{}, m2{}, m3{};
  if (!map_k(&m1.a[0], dy, T, d) || !map_k(&m1.b[0], Wd, F, d) || !map_k(&m2.a[0], du, T, F) ||
      !map_k(&m2.a[1], dz, T, F) || !map_mn(&m2.b[0], Wu_t, F, d) ||
      !map_mn(&m2.b[1], Wg_t, F, d) || !map_mn(&m3.a[0], h, T, F) || !map_mn(&m3.a[1], du, T, F) ||
      !map_mn(&m3.a[2], dz, T, F) || !map_mn(&m3.b[0], dy, T, d) || !map_mn(&m3.b[1], x, T, d) ||
      !map_mn(&m3.b[2], x, T, d))
    return cudaErrorInvalidValue;
  EpiBackward e1;
  e1.T = T;
  e1.F = F;
  e1.act = act;
  e1.z = z;
  e1.u = u;
  e1.h = h;
  e1.du = du;
  e1.dz = dz;
  const int mt = div_up(T, 2 * kBM), nd = div_up(d, kBN);
  cudaError_t e =
      launch_pairs(m1, Tiles{mt, div_up(F, kBN), 1, div_up(d, kBK)}, e1, status, stream);
  if (e != cudaSuccess) return e;
  EpiStore<OpsDx> e2;
  e2.M = T;
  e2.N = d;
  e2.bf16 = dx_dtype == TW_BF16;
  e2.out[0] = e2.out[1] = e2.out[2] = dx;
  e = launch_pairs(m2, Tiles{mt, nd, 1, 2 * div_up(F, kBK)}, e2, status, stream);
  if (e != cudaSuccess) return e;
  EpiStore<OpsGrads> e3;
  e3.M = F;
  e3.N = d;
  e3.bf16 = dw_dtype == TW_BF16;
  e3.out[0] = dWd;
  e3.out[1] = dWu_t;
  e3.out[2] = dWg_t;
  return launch_pairs(m3, Tiles{div_up(F, 2 * kBM), nd, 3, div_up(T, kBK)}, e3, status, stream);
}

}  // namespace tw
