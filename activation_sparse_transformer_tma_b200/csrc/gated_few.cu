// gated_few.cu -- the dense gated FFN of few tokens (T <= kGatedFewMaxT): h = act(x Wg)
// (x Wu), then y = h Wd, on tcgen05 with the operand roles swapped.
//
// With few tokens both products are bound by reading the weights once (3 d F bf16).
// Here 128 rows of weights are the MMA's M side (64 units' gate rows above the same
// units' up rows; for y, 128 output columns, read MN-major from Wd) and the tokens,
// rounded up to 16, its N side, so nothing is spent on absent tokens.
//
// The tiles alone (128 of 64 units at F = 8192, 16 of 128 columns at d = 2048) do
// not occupy the SMs, so the reduction is split over a cluster of S CTAs.  Each
// streams its share of the 64-wide k-blocks through a TMA ring into its TMEM
// accumulator; then every CTA sends each other CTA its part of the tokens through
// distributed shared memory and adds its own tokens' S partial sums in rank order,
// so the result does not depend on timing.  The exchange takes the ring's place.
//
// Measured at d = 2048, F = 8192, weights not in L2 (100.7 MB, 15.6 us at the measured
// copy rate): 1 token 24.5 us, 16: 25.3, 37: 29.2, 64: 31.4, 96: 36.6 (4.1 to 2.8 TB/s); at 112
// as long as the tile kernels.
//
// The second kernel is launched while the first runs (programmatic dependent
// launch).  It starts to read Wd at once -- the
// first kernel has waited for whatever came before it, and does not write Wd -- and
// waits for the first kernel before it reads h.
//
// Roles (320 threads): warp 0 loads by TMA, warp 1 allocates TMEM and issues the
// MMAs, warps 2..9 read TMEM (warp w owns lanes 32 (w % 4)..) and finish the tokens; with
// four of them the finish of 37 tokens took 5 us of the call's 33.  Every mbarrier wait is
// bounded; the cluster barriers are reached by every thread after bounded work.
#include "tmap.h"
#include "pdl.cuh"
#include "cluster.cuh"
#include "gated_act.cuh"
#include "tw_common.cuh"
#include "tw_internal.h"

namespace tw {
namespace {

constexpr int kBK = 64;
constexpr int kRows = 128;                 // rows of weights a tile (MMA M)
constexpr int kUnits = 64;                 // units a gate-up tile
constexpr int kWBytes = kRows * kBK * 2;   // weights a stage
constexpr int kMaxStages = 6;
constexpr int kEndWarps = 8;                // two a quarter of the TMEM lanes
constexpr int kThreads = 64 + 32 * kEndWarps;
constexpr int kMaxCluster = 8;             // portable cluster size

struct Tail {
  uint64_t full[kMaxStages];
  uint64_t empty[kMaxStages];
  uint64_t done;
  uint32_t tmem_base;
  int abort;
  int never;
};

struct Few {
  int T, N;          // tokens, and rounded up to 16 (x box rows)
  int width;         // output columns: F units, or d
  int kblocks;       // of the whole reduction
  int stages, stage_bytes;
  uint32_t tmem_cols;
  int act;
  bool y_bf16;
  uint16_t *h, *z, *u;  // gate-up
  void* y;              // down
};

TW_DEV float activated(int act, float z) {
  float a, da;
  switch (act) {
    case TW_ACT_RELU: activate<TW_ACT_RELU>(z, a, da); break;
    case TW_ACT_SILU: activate<TW_ACT_SILU>(z, a, da); break;
    case TW_ACT_GELU: activate<TW_ACT_GELU>(z, a, da); break;
    default: activate<TW_ACT_GELU_TANH>(z, a, da); break;
  }
  return a;
}

// DOWN: y = h Wd (w0 = Wd, tokens = h); otherwise h = act(x Wg) (x Wu) (w0, w1, tokens = x).
template <bool DOWN>
__global__ void __launch_bounds__(kThreads, 1)
    gated_few_kernel(const __grid_constant__ CUtensorMap w0, const __grid_constant__ CUtensorMap w1,
                     const __grid_constant__ CUtensorMap tokens, const Few f, int32_t* status,
                     unsigned long long timeout_ns, int withhold_loads) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  auto* sm = reinterpret_cast<Tail*>(smem + (size_t)f.stages * f.stage_bytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)cta_rank(), ranks = (int)cta_count();
  const int tile = blockIdx.x / ranks;
  const int k_first = rank * f.kblocks / ranks, k_last = (rank + 1) * f.kblocks / ranks;
  const int n = k_last - k_first;
  volatile int* abort = &sm->abort;

  if (threadIdx.x == 0) {
    for (int s = 0; s < f.stages; ++s) {
      mbar_init(&sm->full[s], 1);
      mbar_init(&sm->empty[s], 1);
    }
    mbar_init(&sm->done, 1);
    sm->abort = 0;
    sm->never = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(&sm->tmem_base, f.tmem_cols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm->tmem_base;

  if (warp == 0) {
    if (elect_one()) {
      auto stage = [&](int i) { return smem + (size_t)(i % f.stages) * f.stage_bytes; };
      auto weights = [&](int i) {
        uint8_t* a = stage(i);
        uint64_t* bar = &sm->full[i % f.stages];
        const int k0 = (k_first + i) * kBK;
        mbar_arrive_expect_tx(bar, (uint32_t)f.stage_bytes);
        if (DOWN) {  // two boxes of 64 k-rows x 64 columns
          tma_load_2d(a, &w0, bar, tile * kRows, k0);
          tma_load_2d(a + kWBytes / 2, &w0, bar, tile * kRows + 64, k0);
        } else {
          tma_load_2d(a, &w0, bar, k0, tile * kUnits);
          tma_load_2d(a + kWBytes / 2, &w1, bar, k0, tile * kUnits);
        }
      };
      auto rows = [&](int i) {
        tma_load_2d(stage(i) + kWBytes, &tokens, &sm->full[i % f.stages], (k_first + i) * kBK, 0);
      };
      // withhold_loads (a test of the bounded waits): nothing is issued
      const int loads = withhold_loads ? 0 : n, early = loads < f.stages ? loads : f.stages;
      if (DOWN) {
        for (int i = 0; i < early; ++i) weights(i);
        pdl_wait();
        for (int i = 0; i < early; ++i) rows(i);
      } else {
        pdl_wait();
        for (int i = 0; i < early; ++i) {
          weights(i);
          rows(i);
        }
      }
      pdl_launch_next();
      int i = early;
      for (; i < loads; ++i) {
        if (!mbar_wait(&sm->empty[i % f.stages], ((i / f.stages) & 1u) ^ 1u, abort, timeout_ns)) {
          *abort = 1;
          set_status(status, kStatusTimeout);
          break;
        }
        weights(i);
        rows(i);
      }
      // copies of a run given up still land before the CTA leaves
      if (*abort)
        for (int j = i > f.stages ? i - f.stages : 0; j < i; ++j)
          mbar_wait(&sm->full[j % f.stages], (j / f.stages) & 1u, &sm->never, kWaitTimeoutNs);
    }
    __syncwarp();
  } else if (warp == 1) {
    pdl_wait();
    pdl_launch_next();
    if (elect_one()) {
      const uint32_t idesc = idesc_bf16_f32(kRows, f.N, DOWN, false);
      bool ok = true;
      for (int i = 0; i < n; ++i) {
        const int s = i % f.stages;
        if (!mbar_wait(&sm->full[s], (i / f.stages) & 1u, abort, timeout_ns)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t a = smem_u32(smem + (size_t)s * f.stage_bytes), b = a + kWBytes;
#pragma unroll
        for (int kk = 0; kk < kBK / 16; ++kk)
          umma_f16_ss(tmem,
                      DOWN ? sdesc_mnmajor_sw128(a + kk * 2048, kBK * 64 * 2)
                           : sdesc_kmajor_sw128(a + kk * 32),
                      sdesc_kmajor_sw128(b + kk * 32), idesc, (i | kk) != 0 ? 1u : 0u);
        umma_commit(&sm->empty[s]);
      }
      if (!ok) {
        *abort = 1;
        set_status(status, kStatusTimeout);
      }
      umma_commit(&sm->done);  // every MMA issued has completed once it flips
      mbar_wait(&sm->done, 0, &sm->never, kWaitTimeoutNs);
    }
    __syncwarp();
  } else {
    pdl_wait();
    pdl_launch_next();
    bool ok = mbar_wait(&sm->done, 0, &sm->never, 2 * timeout_ns);
    if (!__all_sync(0xFFFFFFFFu, ok)) {
      *abort = 1;
      if (lane == 0) set_status(status, kStatusTimeout);
    }
  }
  __syncthreads();
  tc_fence_after();
  // all the cluster's products are done: the rings are free for the exchange
  cluster_meet();
  const int part = f.N / ranks, pairs = part / 2;  // tokens a CTA finishes, and pairs of them
  const uint32_t exchange = smem_u32(smem);
  if (warp >= 2 && !*abort) {
    const int row = (warp & 3) * 32 + lane;
    const uint32_t taddr = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    // two tokens at a time to the CTA that finishes them (part is even); a source's
    // sums of token pair p and row r are at [source][p][r]
    const uint32_t mine = exchange + ((rank * pairs * kRows + row) << 3);
    for (int c = ((warp - 2) >> 2) * 16; c < f.N; c += 32) {
      int to = c / part, p = (c - to * part) / 2;
      uint32_t place = place_in(mine, to);
      uint32_t r[16];
      tmem_ld_x16(taddr + c, r);
      tmem_ld_wait();
#pragma unroll
      for (int k = 0; k < 16; k += 2) {
        store_in(place + p * (kRows * 8), r[k], r[k + 1]);
        if (++p == pairs) {
          p = 0;
          if (++to < ranks) place = place_in(mine, to);
        }
      }
    }
    tc_fence_before();
  }
  __syncwarp();
  cluster_meet();
  if (warp >= 2 && !*abort) {
    const int th = threadIdx.x - 64;
    const float2* sums = reinterpret_cast<const float2*>(smem);
    auto total = [&](int p, int row) {
      float2 v = make_float2(0.f, 0.f);
      for (int s = 0; s < ranks; ++s) {
        const float2 o = sums[(s * pairs + p) * kRows + row];
        v.x += o.x;
        v.y += o.y;
      }
      return v;
    };
    if (DOWN) {
      const int row = th & (kRows - 1), col = tile * kRows + row;
      if (col < f.width)
        for (int p = th / kRows; p < pairs; p += 32 * kEndWarps / kRows) {
          const float2 v = total(p, row);
          const float v2[2] = {v.x, v.y};
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const int t = rank * part + 2 * p + k;
            if (t >= f.T) continue;
            const size_t to = (size_t)t * f.width + col;
            if (f.y_bf16) static_cast<uint16_t*>(f.y)[to] = f32_to_bf16(v2[k]);
            else static_cast<float*>(f.y)[to] = v2[k];
          }
        }
    } else {
      const int row = th & (kUnits - 1), unit = tile * kUnits + row;
      if (unit < f.width)
        for (int p = th / kUnits; p < pairs; p += 32 * kEndWarps / kUnits) {
          const float2 z = total(p, row), u = total(p, kUnits + row);
          const float z2[2] = {z.x, z.y}, u2[2] = {u.x, u.y};
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const int t = rank * part + 2 * p + k;
            if (t >= f.T) continue;
            const size_t to = (size_t)t * f.width + unit;
            f.h[to] = f32_to_bf16(activated(f.act, z2[k]) * u2[k]);
            if (f.z) {
              f.z[to] = f32_to_bf16(z2[k]);
              f.u[to] = f32_to_bf16(u2[k]);
            }
          }
        }
    }
  }
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, f.tmem_cols);
  }
}

// Cluster size: up to two CTAs for every SM, as far as whole k-blocks go round (1 token at
// 2048 x 8192: 26.2 us with two gate-up CTAs an SM, 29.8 with one).
int cluster_of(int tiles, int kblocks) {
  int s = 1;
  while (s < kMaxCluster && 2 * s * tiles <= 2 * num_sms() && 2 * s <= kblocks) s *= 2;
  return s;
}

template <bool DOWN>
cudaError_t launch_few(const CUtensorMap& w0, const CUtensorMap& w1, const CUtensorMap& tokens,
                       Few f, int tiles, unsigned long long withheld_wait_ns, int32_t* status,
                       cudaStream_t stream) {
  f.N = (f.T + 15) / 16 * 16;
  f.stage_bytes = kWBytes + f.N * kBK * 2;
  // two CTAs on an SM, of one kernel or of both (1 token: 24.8 us; with a deeper ring and
  // an SM each 40; with smaller rings, for a third CTA, 25.0 to 28.6)
  const int room = 106 * 1024;
  f.stages = room / f.stage_bytes < kMaxStages ? room / f.stage_bytes : kMaxStages;
  static_assert(kRows * kGatedFewMaxT * 4 <= 106 / (16 + kGatedFewMaxT / 8) *
                                                 (16 + kGatedFewMaxT / 8) * 1024,
                "the exchange fits the ring of the most tokens");
  f.tmem_cols = 32;
  while ((int)f.tmem_cols < f.N) f.tmem_cols *= 2;
  const size_t smem = 1024 + (size_t)f.stages * f.stage_bytes + sizeof(Tail);
  cudaError_t e =
      set_smem_limit(reinterpret_cast<const void*>(gated_few_kernel<DOWN>), (int)smem);
  if (e != cudaSuccess) return e;
  const int s = cluster_of(tiles, f.kblocks);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(tiles * s);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = s;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, gated_few_kernel<DOWN>, w0, w1, tokens, f, status,
                            withheld_wait_ns ? withheld_wait_ns : kWaitTimeoutNs,
                            withheld_wait_ns ? 1 : 0);
}

}  // namespace

cudaError_t launch_gated_few(const void* x, const void* Wg_t, const void* Wu_t, const void* Wd,
                             int T, int d, int F, tw_act act, uint16_t* h, uint16_t* z, uint16_t* u,
                             void* y, tw_dtype y_dtype, unsigned long long withheld_wait_ns,
                             int32_t* status, cudaStream_t stream) {
  const uint32_t n = (uint32_t)((T + 15) / 16 * 16);
  CUtensorMap mx, mg, mu, mh, md;
  if (!make_tmap_bf16(&mx, x, T, d, kBK, n) || !make_tmap_bf16(&mg, Wg_t, F, d, kBK, kUnits) ||
      !make_tmap_bf16(&mu, Wu_t, F, d, kBK, kUnits) || !make_tmap_bf16(&mh, h, T, F, kBK, n) ||
      !make_tmap_bf16(&md, Wd, F, d, 64, kBK))
    return cudaErrorInvalidValue;
  Few f{};
  f.T = T;
  f.act = act;
  f.h = h;
  f.z = z;
  f.u = u;
  f.y = y;
  f.y_bf16 = y_dtype == TW_BF16;
  f.width = F;
  f.kblocks = (d + kBK - 1) / kBK;
  cudaError_t e = launch_few<false>(mg, mu, mx, f, (F + kUnits - 1) / kUnits, withheld_wait_ns,
                                    status, stream);
  if (e != cudaSuccess) return e;
  f.width = d;
  f.kblocks = (F + kBK - 1) / kBK;
  return launch_few<true>(md, md, mh, f, (d + kRows - 1) / kRows, withheld_wait_ns, status,
                          stream);
}

}  // namespace tw
