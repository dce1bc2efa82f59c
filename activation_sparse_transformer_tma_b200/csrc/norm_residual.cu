// norm_residual.cu -- the RMS norms before and after a block, fused with the
// block's gate, its residual scale and the residual sum (Zhang and Sennrich,
// "Root Mean Square Layer Normalization", 2019), forward and backward:
//   o = y rstd_post w_post,  r' = a r + s gate o,  n = r' rstd_pre w_pre.
//
// Both directions read and write each element once and are bound by memory:
// 12 bytes an element forward and 18 backward for bf16 y and n and an fp32
// residual stream.
//   * A team of 32 to 512 threads holds one row in registers, four groups of 4
//     columns a thread (4 (tid + h team)), so every access is contiguous over a
//     warp.  With two groups a thread, twice the team, the instructions that a row
//     costs whatever its width (two reductions, addresses, waits) bounded the
//     kernels: 68 instructions an element forward and 85 backward.
//   * Rows arrive by asynchronous copies, up to three rows ahead.  The thread that
//     copies is the thread that reads, so waiting for its own copies is all the
//     synchronisation the ring needs.
//   * The backward sums the weights' gradients over a CTA's rows in registers and
//     over its teams in shared memory, and leaves one partial row; a second kernel
//     adds the partial rows in a fixed order.  No atomics: the result does not
//     depend on timing.
#include "pdl.cuh"
#include "tw_common.cuh"
#include "tw_internal.h"

namespace tw {
namespace {

constexpr int kQ = 4;  // groups of 4 columns a thread

// Threads of a CTA for a team size.  Forward: two CTAs of 256 threads on an SM at 128
// registers.  Backward: one CTA, of 384 threads at 168 registers where several teams
// fit in it.
constexpr int fwd_threads(int team) { return team > 256 ? team : 256; }
constexpr int bwd_threads(int team) { return team <= 128 ? 384 : team; }

// Four columns as a thread holds them: 8 bytes in bf16, 16 in fp32.
TW_DEV void unpack4(const uint2 w, float (&x)[4]) {
  x[0] = bf16_lo(w.x); x[1] = bf16_hi(w.x); x[2] = bf16_lo(w.y); x[3] = bf16_hi(w.y);
}
TW_DEV uint2 pack4(const float (&x)[4]) {
  return make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]));
}
TW_DEV float4 vec4(const float (&x)[4]) { return make_float4(x[0], x[1], x[2], x[3]); }

// The thread's columns of a row in global memory; i is the first group's index.
// The type is tested once a row and array, not once a group.
template <int TEAM>
TW_DEV void load_row(const void* base, bool bf16, size_t i, const bool (&in)[kQ],
                     float (&x)[kQ][4]) {
  if (bf16) {
    const uint16_t* p = static_cast<const uint16_t*>(base) + i;
#pragma unroll
    for (int h = 0; h < kQ; ++h)
      if (in[h]) unpack4(*reinterpret_cast<const uint2*>(p + h * 4 * TEAM), x[h]);
  } else {
    const float* p = static_cast<const float*>(base) + i;
#pragma unroll
    for (int h = 0; h < kQ; ++h)
      if (in[h]) {
        const float4 w = *reinterpret_cast<const float4*>(p + h * 4 * TEAM);
        x[h][0] = w.x; x[h][1] = w.y; x[h][2] = w.z; x[h][3] = w.w;
      }
  }
}
template <int TEAM>
TW_DEV void store_row(void* base, bool bf16, size_t i, const bool (&in)[kQ],
                      const float (&x)[kQ][4]) {
  if (bf16) {
    uint16_t* p = static_cast<uint16_t*>(base) + i;
#pragma unroll
    for (int h = 0; h < kQ; ++h)
      if (in[h]) *reinterpret_cast<uint2*>(p + h * 4 * TEAM) = pack4(x[h]);
  } else {
    float* p = static_cast<float*>(base) + i;
#pragma unroll
    for (int h = 0; h < kQ; ++h)
      if (in[h]) *reinterpret_cast<float4*>(p + h * 4 * TEAM) = vec4(x[h]);
  }
}

// The same columns in the ring: group h of all threads, contiguous over the threads.
template <int TEAM, int N>
TW_DEV void copy_row(uint32_t array, const void* base, bool bf16, size_t i,
                     const bool (&in)[kQ]) {
  if (bf16) {
    const uint16_t* p = static_cast<const uint16_t*>(base) + i;
    const uint32_t to = array + threadIdx.x * 8;
#pragma unroll
    for (int h = 0; h < kQ; ++h)
      if (in[h])
        asm volatile("cp.async.ca.shared.global [%0], [%1], 8;"
                     ::"r"(to + h * N * 8), "l"(p + h * 4 * TEAM) : "memory");
  } else {
    const float* p = static_cast<const float*>(base) + i;
    const uint32_t to = array + threadIdx.x * 16;
#pragma unroll
    for (int h = 0; h < kQ; ++h)
      if (in[h])
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;"
                     ::"r"(to + h * N * 16), "l"(p + h * 4 * TEAM) : "memory");
  }
}
// Columns past d read what is in their place: zeros that zero_past() left there.
template <int N>
TW_DEV void read_row(uint32_t array, bool bf16, float (&x)[kQ][4]) {
  if (bf16) {
    const uint32_t at = array + threadIdx.x * 8;
#pragma unroll
    for (int h = 0; h < kQ; ++h) {
      uint2 w;
      asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];"
                   : "=r"(w.x), "=r"(w.y) : "r"(at + h * N * 8) : "memory");
      unpack4(w, x[h]);
    }
  } else {
    const uint32_t at = array + threadIdx.x * 16;
#pragma unroll
    for (int h = 0; h < kQ; ++h)
      asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                   : "=f"(x[h][0]), "=f"(x[h][1]), "=f"(x[h][2]), "=f"(x[h][3])
                   : "r"(at + h * N * 16) : "memory");
  }
}
TW_DEV void copy_float(uint32_t to, const float* from) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(to), "l"(from) : "memory");
}
TW_DEV float read_float(uint32_t at) {
  float x;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(x) : "r"(at) : "memory");
  return x;
}
TW_DEV void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// The oldest of `stages` groups has landed.
TW_DEV void copies_wait(int stages) {
  if (stages >= 4) asm volatile("cp.async.wait_group 3;" ::: "memory");
  else if (stages == 3) asm volatile("cp.async.wait_group 2;" ::: "memory");
  else if (stages == 2) asm volatile("cp.async.wait_group 1;" ::: "memory");
  else asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// A ring of `stages` rows: a row's copies are issued stages - 1 rows ahead, into the
// place of the row just read (with one stage: at its own turn).  Offsets of the
// arrays within a stage, in bytes; an absent array has no room.
struct Ring {
  int y, r, dr, dn, gate, p, bytes, stages;
};

// Rows narrower than the team's columns: a thread clears its places past d, which no
// copy writes.
template <int N>
TW_DEV void zero_past(uint32_t base, const Ring& ring, int array, bool bf16,
                      const bool (&in)[kQ]) {
  if (array < 0 || in[kQ - 1]) return;
  for (int s = 0; s < ring.stages; ++s) {
#pragma unroll
    for (int h = 0; h < kQ; ++h) {
      const uint32_t at =
          base + s * ring.bytes + array + (h * N + threadIdx.x) * (bf16 ? 8 : 16);
      if (in[h]) continue;
      if (bf16) asm volatile("st.shared.v2.u32 [%0], {%1, %1};" ::"r"(at), "r"(0u) : "memory");
      else asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(at), "r"(0u) : "memory");
    }
  }
}

struct Block {
  int T, d, gate_group;
  float a, s, eps, inv_d;
  bool y_bf16, r_bf16, n_bf16, w_bf16;
  const void *w_post, *gate, *w_pre;
};

// Threads of one row, and this thread's groups of columns; N threads in the CTA.
template <int TEAM, int N>
struct Team {
  static constexpr int W = TEAM / 32;
  int index, tid, turn;
  bool in[kQ];
  TW_DEV explicit Team(int d) {
    index = threadIdx.x / TEAM;
    tid = threadIdx.x % TEAM;
    turn = 0;
#pragma unroll
    for (int h = 0; h < kQ; ++h) in[h] = 4 * (tid + h * TEAM) < d;
  }
  // Sums of K values over the team, in a fixed order.  `slots` holds K floats per
  // warp of the CTA and alternates between two arrays: a thread that writes an
  // array again has passed the barrier of the other one, so all have read it.
  template <int K>
  TW_DEV void sum(float (&v)[K], float (*slots)[K * 16]) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
      for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(0xFFFFFFFFu, v[k], o);
    if (W == 1) return;
    float* at = slots[turn] + index * (W * K);
    turn ^= 1;
    if ((threadIdx.x & 31) == 0) {
#pragma unroll
      for (int k = 0; k < K; ++k) at[k * W + (tid >> 5)] = v[k];
    }
    if (TEAM == N) __syncthreads();
    else asm volatile("bar.sync %0, %1;" ::"r"(1 + index), "r"(TEAM) : "memory");
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (W == 2) {
        const float2 a = *reinterpret_cast<const float2*>(at + k * W);
        v[k] = a.x + a.y;
      } else {
        v[k] = 0.f;
#pragma unroll
        for (int w = 0; w < W / 4; ++w) {
          const float4 a = reinterpret_cast<const float4*>(at + k * W)[w];
          v[k] += (a.x + a.y) + (a.z + a.w);
        }
      }
    }
  }
};

// 1/sqrt(sum / d + eps): the approximate instruction is within 2 ulp.
TW_DEV float inverse_norm(float sum, const Block& b) { return rsqrtf(fmaf(sum, b.inv_d, b.eps)); }

template <int TEAM>
__global__ void __launch_bounds__(fwd_threads(TEAM), TEAM <= 256 ? 2 : 1)
    norm_forward_kernel(const Block b, const void* y, const void* r, void* r_out, void* n_out,
                        float* rstd_post, float* rstd_pre, const Ring ring) {
  extern __shared__ __align__(16) uint8_t rows[];
  __shared__ __align__(16) float slots[2][16];
  constexpr int N = fwd_threads(TEAM), TEAMS = N / TEAM;
  Team<TEAM, N> tm(b.d);
  const long long stride = (long long)gridDim.x * TEAMS;
  const long long first = (long long)blockIdx.x * TEAMS + tm.index;
  const uint32_t base = smem_u32(rows);
  zero_past<N>(base, ring, ring.y, b.y_bf16, tm.in);
  zero_past<N>(base, ring, ring.r, b.r_bf16, tm.in);
  zero_past<N>(base, ring, ring.gate, b.w_bf16, tm.in);
  pdl_wait();
  pdl_launch_next();
  const bool gate_rows = b.gate && b.gate_group < b.T;
  auto fetch = [&](int stage, long long row) {
    if (row < b.T) {
      const uint32_t to = base + stage * ring.bytes;
      const size_t i = (size_t)row * b.d + 4 * tm.tid;
      if (y) copy_row<TEAM, N>(to + ring.y, y, b.y_bf16, i, tm.in);
      copy_row<TEAM, N>(to + ring.r, r, b.r_bf16, i, tm.in);
      if (gate_rows)
        copy_row<TEAM, N>(to + ring.gate, b.gate, b.w_bf16,
                       (size_t)((int)row / b.gate_group) * b.d + 4 * tm.tid, tm.in);
    }
    copies_commit();
  };
  for (int k = 0; k + 1 < ring.stages; ++k) fetch(k, first + k * stride);

  // c = block_scale * gate * w_post of this thread's columns; without gate rows
  // it is kept over the thread's rows.  Columns past d: everything is zero there.
  float c[kQ][4] = {}, wpre[kQ][4] = {};
  if (y && !gate_rows) {
    float gt[kQ][4];
#pragma unroll
    for (int h = 0; h < kQ; ++h)
#pragma unroll
      for (int k = 0; k < 4; ++k) c[h][k] = gt[h][k] = 1.f;
    if (b.w_post) load_row<TEAM>(b.w_post, b.w_bf16, 4 * tm.tid, tm.in, c);
    if (b.gate) load_row<TEAM>(b.gate, b.w_bf16, 4 * tm.tid, tm.in, gt);
#pragma unroll
    for (int h = 0; h < kQ; ++h)
#pragma unroll
      for (int k = 0; k < 4; ++k) c[h][k] *= b.s * gt[h][k];
  }
  if (b.w_pre) load_row<TEAM>(b.w_pre, b.w_bf16, 4 * tm.tid, tm.in, wpre);

  int stage = 0;
  for (long long row = first; row < b.T; row += stride) {
    // into the stage read before
    fetch(stage == 0 ? ring.stages - 1 : stage - 1, row + (ring.stages - 1) * stride);
    copies_wait(ring.stages);
    const uint32_t from = base + stage * ring.bytes;
    if (++stage == ring.stages) stage = 0;
    const size_t i = (size_t)row * b.d + 4 * tm.tid;
    float rv[kQ][4];
    read_row<N>(from + ring.r, b.r_bf16, rv);
    if (y) {
      float yv[kQ][4];
      read_row<N>(from + ring.y, b.y_bf16, yv);
      if (gate_rows) {
        float w[kQ][4];
#pragma unroll
        for (int h = 0; h < kQ; ++h)
#pragma unroll
          for (int k = 0; k < 4; ++k) w[h][k] = 1.f;
        read_row<N>(from + ring.gate, b.w_bf16, c);
        if (b.w_post) load_row<TEAM>(b.w_post, b.w_bf16, 4 * tm.tid, tm.in, w);
#pragma unroll
        for (int h = 0; h < kQ; ++h)
#pragma unroll
          for (int k = 0; k < 4; ++k) c[h][k] *= b.s * w[h][k];
      }
      float p = 1.f;
      if (b.w_post) {
        float ss[1] = {0.f};
#pragma unroll
        for (int h = 0; h < kQ; ++h)
#pragma unroll
          for (int k = 0; k < 4; ++k) ss[0] = fmaf(yv[h][k], yv[h][k], ss[0]);
        tm.sum(ss, slots);
        p = inverse_norm(ss[0], b);
        if (rstd_post && tm.tid == 0) rstd_post[row] = p;
      }
#pragma unroll
      for (int h = 0; h < kQ; ++h)
#pragma unroll
        for (int k = 0; k < 4; ++k) rv[h][k] = fmaf(yv[h][k] * p, c[h][k], b.a * rv[h][k]);
      store_row<TEAM>(r_out, b.r_bf16, i, tm.in, rv);
    }
    if (b.w_pre) {
      float ss[1] = {0.f};
#pragma unroll
      for (int h = 0; h < kQ; ++h)
#pragma unroll
        for (int k = 0; k < 4; ++k) ss[0] = fmaf(rv[h][k], rv[h][k], ss[0]);
      tm.sum(ss, slots);
      const float p = inverse_norm(ss[0], b);
      if (rstd_pre && tm.tid == 0) rstd_pre[row] = p;
#pragma unroll
      for (int h = 0; h < kQ; ++h)
#pragma unroll
        for (int k = 0; k < 4; ++k) rv[h][k] *= p * wpre[h][k];
      store_row<TEAM>(n_out, b.n_bf16, i, tm.in, rv);
    }
  }
}

// ----------------------------------------------------------------- backward --
// Rows are dealt out in items: at most rows_per_item consecutive rows of one gate
// group (per_group items cover a group).  An item belongs to a CTA, whose teams
// share its rows, or to one team (by_team: short groups, and where a CTA is one
// team); either way the gate row's gradient is complete, or one partial of
// per_group, when the item is done.
struct Items {
  int group, rows_per_item, per_group, count;
  bool by_team;
};

struct BackwardArgs {
  const void *dn, *dr_out, *y, *r_out;
  const float *rstd_post, *rstd_pre;
  void *dy, *dr;
  float* dgate;      // where an item's gate gradient goes: row (per_group == 1 ? group : item)
  float* part_post;  // [CTAs][d]
  float* part_pre;   // [CTAs][d]
};

// Shared memory behind the ring (byte offsets): w_pre in fp32; with gate rows, w_post in
// fp32 where teams have their own items (-1 in the widest rows, which leave no room, and
// for a CTA's items, too few to repay the copy: 8192 x 200 in groups of 31 takes 22.3 us
// with it, 20.8 without), the sums of dw_post over the items done (of a thread, or of the
// CTA's columns) and the teams' sums of an item.  Sums over the teams behind the loop
// take the ring's place.
struct Extra {
  int wpre, wpost, post, comb;
};

// Over an item the gate is one row, so one sum A = sum_t G yh serves both the gate
// and w_post: dgate = s w_post A and dw_post += s gate A.
//
// One reduction a row: with H = dr_out + rstd_pre e, the second mean is
//   sum f yh = sum F H yh - rstd_pre mean(e rh) sum F rh yh,   F = s gate w_post,
// so its sums need no result of the first (a second reduction behind the first cost
// about 1 us of 67 for 8192 x 2048).  The terms are those that G is summed from.
//
// One CTA of 384 threads an SM: 60 us for 8192 x 2048 (302 MB, 5.0 TB/s) against 66
// with 256 threads; 512 spill registers and leave room for one row a team (92 us).
// Two CTAs' worth of rounds cost more (69 us): what a CTA does once, its first rows'
// latency and its partial row, is 8 us.
template <int TEAM>
__global__ void __launch_bounds__(bwd_threads(TEAM), 1)
    norm_backward_kernel(const Block b, const BackwardArgs g, const Items it, const Ring ring,
                         const Extra extra) {
  extern __shared__ __align__(16) uint8_t rows[];
  __shared__ __align__(16) float slots[2][3 * 16];
  constexpr int N = bwd_threads(TEAM), TEAMS = N / TEAM;
  Team<TEAM, N> tm(b.d);
  const int units = it.by_team ? gridDim.x * TEAMS : gridDim.x;
  const int unit = it.by_team ? blockIdx.x * TEAMS + tm.index : blockIdx.x;
  const int first = it.by_team ? 0 : tm.index;  // this team's first row of an item
  const int stride = it.by_team ? 1 : TEAMS;
  const uint32_t base = smem_u32(rows);
  const bool gate_rows = b.gate && it.group < b.T;
  const bool gate_ring = TEAM <= 256 && gate_rows && ring.gate >= 0;
  const bool wpost_kept = TEAM <= 256 && extra.wpost >= 0;
  zero_past<N>(base, ring, ring.y, b.y_bf16, tm.in);
  zero_past<N>(base, ring, ring.r, b.r_bf16, tm.in);
  zero_past<N>(base, ring, ring.gate, b.w_bf16, tm.in);
  zero_past<N>(base, ring, ring.dr, b.r_bf16, tm.in);
  zero_past<N>(base, ring, ring.dn, b.n_bf16, tm.in);
  pdl_wait();
  pdl_launch_next();

  auto group_of = [&](int item) { return it.per_group == 1 ? item : item / it.per_group; };
  auto range = [&](int item, int& row0, int& row1) {
    const int group = group_of(item), part = item - group * it.per_group;
    // group * it.group < T, so only the ends can pass T (and, added up, 2^31)
    const long long g0 = (long long)group * it.group;
    const long long g1 = g0 + it.group < b.T ? g0 + it.group : b.T;
    long long r0 = g0 + (long long)part * it.rows_per_item;
    if (r0 > g1) r0 = g1;
    row0 = (int)r0;
    row1 = (int)(r0 + it.rows_per_item < g1 ? r0 + it.rows_per_item : g1);
  };
  // The row to copy next: this team's rows of its items in order, `ring.stages - 1`
  // rows ahead of the one in hand.
  long long ahead_item = unit, ahead_row = 0;
  int ahead_end = 0;
  bool ahead_new = true;  // at the first row of an item
  auto seek = [&]() {     // the first item from ahead_item on that has a row for this team
    for (; ahead_item < it.count; ahead_item += units) {
      int n0;
      range((int)ahead_item, n0, ahead_end);
      ahead_row = (long long)n0 + first;
      if (ahead_row < ahead_end) break;
    }
    ahead_new = true;
  };
  auto fetch = [&](int stage) {
    if (ahead_item < it.count) {
      const uint32_t to = base + stage * ring.bytes;
      const size_t i = (size_t)ahead_row * b.d + 4 * tm.tid;
      if (g.dn) {
        copy_row<TEAM, N>(to + ring.dn, g.dn, b.n_bf16, i, tm.in);
        copy_row<TEAM, N>(to + ring.r, g.r_out, b.r_bf16, i, tm.in);
      }
      if (g.dr_out) copy_row<TEAM, N>(to + ring.dr, g.dr_out, b.r_bf16, i, tm.in);
      if (g.y) copy_row<TEAM, N>(to + ring.y, g.y, b.y_bf16, i, tm.in);
      if (gate_ring && ahead_new)
        copy_row<TEAM, N>(to + ring.gate, b.gate, b.w_bf16,
                       (size_t)group_of((int)ahead_item) * b.d + 4 * tm.tid, tm.in);
      if (g.rstd_post) copy_float(to + ring.p + threadIdx.x * 4, g.rstd_post + ahead_row);
      if (g.rstd_pre) copy_float(to + ring.p + (N + threadIdx.x) * 4, g.rstd_pre + ahead_row);
      ahead_new = false;
      ahead_row += stride;
      if (ahead_row >= ahead_end) {
        ahead_item += units;
        seek();
      }
    }
    copies_commit();
  };
  seek();
  for (int k = 0; k + 1 < ring.stages; ++k) fetch(k);

  auto ones = [&](float (&x)[kQ][4]) {
#pragma unroll
    for (int h = 0; h < kQ; ++h)
#pragma unroll
      for (int k = 0; k < 4; ++k) x[h][k] = tm.in[h] ? 1.f : 0.f;
  };
  // A thread's own floats behind the ring.
  auto mine = [&](int array, int h) {
    return reinterpret_cast<float4*>(rows + array) + h * N + threadIdx.x;
  };
  // Sums over the teams: every thread leaves its columns in an area, and after a barrier
  // a thread takes strips of 4 columns, strip i being columns 4i..4i+3.
  constexpr int kStrips = kQ * TEAM;
  auto leave = [&](int array, const float (&v)[kQ][4]) {
#pragma unroll
    for (int h = 0; h < kQ; ++h) *mine(array, h) = vec4(v[h]);
  };
  auto strip_sum = [&](int array, int i, float (&v)[4]) {
    const float4* at = reinterpret_cast<const float4*>(rows + array) + (i / TEAM) * N + i % TEAM;
    v[0] = v[1] = v[2] = v[3] = 0.f;
#pragma unroll 4
    for (int t = 0; t < TEAMS; ++t) {
      const float4 o = at[t * TEAM];
      v[0] += o.x; v[1] += o.y; v[2] += o.z; v[3] += o.w;
    }
  };
  auto strip_load = [&](const void* w, size_t at, float (&v)[4]) {
    v[0] = v[1] = v[2] = v[3] = 1.f;
    if (!w) return;
    if (b.w_bf16) {
      unpack4(*reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(w) + at), v);
    } else {
      const float4 o = *reinterpret_cast<const float4*>(static_cast<const float*>(w) + at);
      v[0] = o.x; v[1] = o.y; v[2] = o.z; v[3] = o.w;
    }
  };
  // s x times y of a strip to global memory.
  auto strip_store = [&](float* to, int i, const float (&x)[4], const float (&y)[4]) {
    *reinterpret_cast<float4*>(to + 4 * i) = make_float4(
        b.s * x[0] * y[0], b.s * x[1] * y[1], b.s * x[2] * y[2], b.s * x[3] * y[3]);
  };

  const bool keep_post = g.part_post && gate_rows;
  // every team writes the same values; a thread reads the columns that it wrote
  float4* wpre = reinterpret_cast<float4*>(rows + extra.wpre) + tm.tid;
  auto keep = [&](float4* to, const void* from) {
    float w[kQ][4] = {};
    load_row<TEAM>(from, b.w_bf16, 4 * tm.tid, tm.in, w);
#pragma unroll
    for (int h = 0; h < kQ; ++h) to[h * TEAM] = vec4(w[h]);
  };
  if (b.w_pre) keep(wpre, b.w_pre);
  float4* wpost = reinterpret_cast<float4*>(rows + extra.wpost) + tm.tid;
  if (wpost_kept) keep(wpost, b.w_post);
  auto read_wpost = [&](float (&w)[kQ][4]) {
    ones(w);
    if (wpost_kept) {
#pragma unroll
      for (int h = 0; h < kQ; ++h) {
        const float4 o = wpost[h * TEAM];
        w[h][0] = o.x; w[h][1] = o.y; w[h][2] = o.z; w[h][3] = o.w;
      }
    } else if (b.w_post) {
      load_row<TEAM>(b.w_post, b.w_bf16, 4 * tm.tid, tm.in, w);
    }
  };
  if (keep_post) {
#pragma unroll
    for (int h = 0; h < kQ; ++h) *mine(extra.post, h) = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  float apre[kQ][4] = {}, A[kQ][4] = {}, F[kQ][4];  // F = s gate w_post
  int stage = 0;
  for (long long next_item = unit; next_item < it.count; next_item += units) {
    const int item = (int)next_item;
    int row0, row1;
    range(item, row0, row1);
    const int group = group_of(item);
    const size_t gate_at = (size_t)group * b.d + 4 * tm.tid;
    bool new_item = true;
    uint32_t from = base;  // the stage of the row in hand
    for (long long row = (long long)row0 + first; row < row1; row += stride) {
      fetch(stage == 0 ? ring.stages - 1 : stage - 1);  // into the stage read before
      copies_wait(ring.stages);
      from = base + stage * ring.bytes;
      if (++stage == ring.stages) stage = 0;
      if (new_item && g.y) {
        float w[kQ][4];
        read_wpost(w);
        ones(F);
        if (gate_ring) read_row<N>(from + ring.gate, b.w_bf16, F);
        else if (b.gate) load_row<TEAM>(b.gate, b.w_bf16, gate_at, tm.in, F);
#pragma unroll
        for (int h = 0; h < kQ; ++h)
#pragma unroll
          for (int k = 0; k < 4; ++k) F[h][k] *= b.s * w[h][k];
      }
      new_item = false;
      const size_t i = (size_t)row * b.d + 4 * tm.tid;
      float G[kQ][4] = {}, e[kQ][4] = {}, yh[kQ][4] = {};  // e: rh until the sums are known
      float ppre = 0.f, ppost = 1.f;
      float sums[3] = {0.f, 0.f, 0.f};
      if (g.dr_out) read_row<N>(from + ring.dr, b.r_bf16, G);
      if (g.dy) {
        read_row<N>(from + ring.y, b.y_bf16, yh);
        if (b.w_post) {
          ppost = read_float(from + ring.p + threadIdx.x * 4);
#pragma unroll
          for (int h = 0; h < kQ; ++h)
#pragma unroll
            for (int k = 0; k < 4; ++k) yh[h][k] *= ppost;
        }
      }
      if (g.dn) {
        float dn[kQ][4];
        ppre = read_float(from + ring.p + (N + threadIdx.x) * 4);
        read_row<N>(from + ring.dn, b.n_bf16, dn);
        read_row<N>(from + ring.r, b.r_bf16, e);
#pragma unroll
        for (int h = 0; h < kQ; ++h) {
          const float4 w4 = wpre[h * TEAM];
          const float w[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float rh = e[h][k] * ppre;
            apre[h][k] = fmaf(dn[h][k], rh, apre[h][k]);
            const float ee = dn[h][k] * w[k];
            sums[0] = fmaf(ee, rh, sums[0]);
            G[h][k] = fmaf(ppre, ee, G[h][k]);  // H
            e[h][k] = rh;
          }
        }
      }
      if (b.w_post) {
#pragma unroll
        for (int h = 0; h < kQ; ++h)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float fy = F[h][k] * yh[h][k];
            sums[1] = fmaf(G[h][k], fy, sums[1]);
            sums[2] = fmaf(e[h][k], fy, sums[2]);
          }
      }
      if (g.dn || b.w_post) tm.sum(sums, slots);
      const float c = ppre * (sums[0] * b.inv_d);
      float out[kQ][4];
#pragma unroll
      for (int h = 0; h < kQ; ++h)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          G[h][k] = fmaf(-c, e[h][k], G[h][k]);
          out[h][k] = g.dy ? b.a * G[h][k] : G[h][k];  // no residual scale without a block
        }
      store_row<TEAM>(g.dr, b.r_bf16, i, tm.in, out);
      if (g.dy) {
        const float inner = fmaf(-c, sums[2], sums[1]) * b.inv_d;
#pragma unroll
        for (int h = 0; h < kQ; ++h)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            A[h][k] = fmaf(G[h][k], yh[h][k], A[h][k]);
            out[h][k] = F[h][k] * G[h][k];
            if (b.w_post) out[h][k] = ppost * fmaf(-yh[h][k], inner, out[h][k]);
          }
        store_row<TEAM>(g.dy, b.y_bf16, i, tm.in, out);
      }
    }
    if (gate_rows) {
      float* to = g.dgate + (size_t)(it.per_group == 1 ? group : item) * b.d;
      if (it.by_team) {
        float w[kQ][4], gt[kQ][4];
        read_wpost(w);
        ones(gt);
        // an item of one row still has its gate row in the ring (8192 x 2048 with a gate
        // row each: 92 us for the call, 109 with gate and w_post from global memory)
        if (gate_ring && row1 - row0 == 1) read_row<N>(from + ring.gate, b.w_bf16, gt);
        else load_row<TEAM>(b.gate, b.w_bf16, gate_at, tm.in, gt);
#pragma unroll
        for (int h = 0; h < kQ; ++h) {
          if (keep_post) {
            float4 o = *mine(extra.post, h);
            o.x = fmaf(b.s * gt[h][0], A[h][0], o.x);
            o.y = fmaf(b.s * gt[h][1], A[h][1], o.y);
            o.z = fmaf(b.s * gt[h][2], A[h][2], o.z);
            o.w = fmaf(b.s * gt[h][3], A[h][3], o.w);
            *mine(extra.post, h) = o;
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) w[h][k] *= b.s * A[h][k];
        }
        store_row<TEAM>(to, false, 4 * tm.tid, tm.in, w);
      } else {
        __syncthreads();  // the last item's sums have been taken
        leave(extra.comb, A);
        __syncthreads();
        for (int i = threadIdx.x; i < kStrips && 4 * i < b.d; i += N) {
          float w[4], gt[4], v[4];
          strip_load(b.w_post, 4 * i, w);
          strip_load(b.gate, (size_t)group * b.d + 4 * i, gt);
          strip_sum(extra.comb, i, v);
          strip_store(to, i, w, v);
          if (keep_post) {  // the strip is this thread's in every item
            float4* o = reinterpret_cast<float4*>(rows + extra.post) + i;
            *o = make_float4(fmaf(b.s * gt[0], v[0], o->x), fmaf(b.s * gt[1], v[1], o->y),
                             fmaf(b.s * gt[2], v[2], o->z), fmaf(b.s * gt[3], v[3], o->w));
          }
        }
      }
#pragma unroll
      for (int h = 0; h < kQ; ++h)
#pragma unroll
        for (int k = 0; k < 4; ++k) A[h][k] = 0.f;
    }
  }
  // Without gate rows A runs over all the CTA's rows, and gives both gradients here.
  constexpr int kVector = 4 * 4 * kQ * N;  // bytes of an area
  __syncthreads();  // the ring's rows have been read
  if (g.part_pre) leave(0, apre);
  if (!gate_rows) leave(kVector, A);
  __syncthreads();
  for (int i = threadIdx.x; i < kStrips && 4 * i < b.d; i += N) {
    const size_t part_at = (size_t)blockIdx.x * b.d;
    float w[4], gt[4], v[4];
    if (!gate_rows) {
      strip_load(b.w_post, 4 * i, w);
      strip_load(b.gate, 4 * i, gt);
    }
    if (g.part_pre) {
      strip_sum(0, i, v);
      *reinterpret_cast<float4*>(g.part_pre + part_at + 4 * i) = vec4(v);
    }
    if (keep_post) {
      if (it.by_team) {
        strip_sum(extra.post, i, v);
      } else {
        const float4 o = reinterpret_cast<const float4*>(rows + extra.post)[i];
        v[0] = o.x; v[1] = o.y; v[2] = o.z; v[3] = o.w;
      }
      *reinterpret_cast<float4*>(g.part_post + part_at + 4 * i) = vec4(v);
    } else if (!gate_rows) {
      strip_sum(kVector, i, v);
      if (b.gate) strip_store(g.dgate + part_at, i, w, v);
      if (g.part_post) strip_store(g.part_post + part_at, i, gt, v);
    }
  }
}

// One sum of partial rows: out[row][c] = sum of `each` consecutive rows of `part`.
struct RowSum {
  const float* part;
  float* out;
  int rows, each;
};
struct RowSums {
  RowSum s[3];
  int first[4];  // prefix sums of the CTAs
  int count, d;
};

// 32 columns of an output row each: by a CTA, its partial rows dealt over 16 warps and
// their sums added in order, or, with few partial rows (a group's items), by a warp.
constexpr int kSumWarps = 16;
constexpr int kFewParts = 16;
__global__ void __launch_bounds__(kSumWarps * 32) norm_sum_kernel(const RowSums a) {
  __shared__ float sums[kSumWarps][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int strips = (a.d + 31) / 32;
  int i = 0;
  while (i + 1 < a.count && (int)blockIdx.x >= a.first[i + 1]) ++i;
  const RowSum& s = a.s[i];
  const bool few = s.each <= kFewParts;
  int unit = blockIdx.x - a.first[i];
  if (few) unit = unit * kSumWarps + warp;
  const int row = unit / strips, c = (unit - row * strips) * 32 + lane;
  pdl_wait();
  pdl_launch_next();
  const int first = few ? 0 : warp, step = few ? 1 : kSumWarps;
  float v = 0.f;
  if (row < s.rows && c < a.d) {
    const float* p = s.part + (size_t)row * s.each * a.d + c;
    for (int k0 = first; k0 < s.each; k0 += 8 * step) {
      float x[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int k = k0 + j * step;
        x[j] = k < s.each ? p[(size_t)k * a.d] : 0.f;
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) v += x[j];
    }
  }
  if (!few) {
    sums[warp][lane] = v;
    __syncthreads();
    if (warp != 0) return;
    v = 0.f;
#pragma unroll
    for (int k = 0; k < kSumWarps; ++k) v += sums[k][lane];
  }
  if (row < s.rows && c < a.d) s.out[(size_t)row * a.d + c] = v;
}

int team_size_of(int d) {
  int team = 32;
  while (team * 4 * kQ < d) team *= 2;
  return team;
}

// The backward's launch: CTAs, and how rows are dealt out, for T > 0.  The same rule sizes
// the workspace, from T, d and gate_group alone (sms: the SMs of the current device).
struct Plan {
  Items it;
  int ctas, threads, team;
};
// What an item costs beside its rows, in rows of one team: a team on its own stores its
// sums, a CTA's teams meet twice and add theirs.
constexpr int kTeamItem = 1, kCtaItem = 2;

Plan make_plan(int T, int d, int gate_group, int sms) {
  Plan p;
  p.team = team_size_of(d);
  p.threads = bwd_threads(p.team);
  const int teams = p.threads / p.team;
  const long long T64 = T;
  const int group = gate_group <= 0 || gate_group > T ? T : gate_group;
  const int groups = (int)((T64 + group - 1) / group);
  p.it.group = group;
  // The rounds of items times their length: groups whole to a team each, or cut into `per`
  // items for CTAs.  (8192 x 2048, groups of 31: 2 rounds of CTAs, where teams of their own
  // took 87 us for the call; groups of 100: 5 items each, where whole groups on 82 of 148
  // CTAs took 109.)
  const long long teams_all = (long long)sms * teams;
  long long best = groups > 1 ? (groups + teams_all - 1) / teams_all * ((long long)group + kTeamItem)
                              : 0;
  long long rows = group;
  bool by_team = groups > 1;
  const long long most = (group + (long long)teams - 1) / teams;  // a row for each team
  for (long long rounds = 1; rounds <= 16; ++rounds) {
    long long per = rounds * sms / groups;  // as many items as the rounds hold
    per = per < 1 ? 1 : per > most ? most : per;
    const long long length = (group + per - 1) / per, items = groups * ((group + length - 1) / length);
    const long long cost = (items + sms - 1) / sms * ((length + teams - 1) / teams + kCtaItem);
    if (best == 0 || cost < best) {
      best = cost;
      rows = length;
      by_team = false;
    }
    // without gate rows a CTA has one item, whose partial row is the CTA's
    if (per == most || groups == 1) break;
  }
  p.it.by_team = by_team || teams == 1;
  p.it.rows_per_item = (int)rows;
  p.it.per_group = (int)((group + rows - 1) / rows);
  p.it.count = groups * p.it.per_group;
  const int units = (int)(p.it.by_team ? ((long long)p.it.count + teams - 1) / teams : p.it.count);
  p.ctas = units < sms ? units : sms;
  return p;
}

size_t align256(size_t n) { return (n + 255) & ~size_t(255); }

// Workspace: the CTAs' partial rows of dw_pre and dw_post, and the partial rows of
// gate gradients where a group has several items.
struct Parts {
  size_t pre, post, gate, bytes;
};
Parts parts_of(const Plan& p, int d, bool gate) {
  Parts q;
  const size_t row = sizeof(float) * (size_t)d;
  q.pre = 0;
  q.post = align256(p.ctas * row);
  q.gate = 2 * q.post;
  q.bytes = q.gate + (gate && p.it.per_group > 1 ? align256(p.it.count * row) : 0);
  return q;
}

Block device_block(const tw_norm_block& b) {
  Block k;
  k.T = b.T;
  k.d = b.d;
  k.gate_group = b.gate_group;
  k.a = b.res_scale;
  k.s = b.block_scale;
  k.eps = b.eps;
  k.inv_d = 1.f / (float)b.d;
  k.y_bf16 = b.y_dtype == TW_BF16;
  k.r_bf16 = b.r_dtype == TW_BF16;
  k.n_bf16 = b.n_dtype == TW_BF16;
  k.w_bf16 = b.w_dtype == TW_BF16;
  k.w_post = b.w_post;
  k.gate = b.gate;
  k.w_pre = b.w_pre;
  return k;
}

// Shared memory of an SM for the rings, beside 1 KB a CTA that the system takes and
// the kernels' own arrays.
constexpr int kSmemSm = 224 * 1024;

// The ring for the arrays that a call has (bytes of an element, 0 if absent).
Ring make_ring(int threads, int y, int r, int dr, int dn, int gate, bool p, int room) {
  Ring q;
  int at = 0;
  auto take = [&](int size) {
    const int here = size ? at : -1;
    at += 4 * kQ * threads * size;
    return here;
  };
  q.y = take(y);
  q.r = take(r);
  q.dr = take(dr);
  q.dn = take(dn);
  q.gate = take(gate);
  q.p = at;
  if (p) at += 2 * threads * 4;
  q.bytes = at;
  q.stages = room / at < 1 ? 1 : room / at > 4 ? 4 : room / at;
  return q;
}

template <int TEAM>
cudaError_t forward_team(const Block& k, const void* y, const void* r, void* r_out, void* n_out,
                         float* rstd_post, float* rstd_pre, cudaStream_t stream) {
  constexpr int N = fwd_threads(TEAM), TEAMS = N / TEAM, per_sm = TEAM <= 256 ? 2 : 1;
  const long long want = ((long long)k.T + TEAMS - 1) / TEAMS;
  // CTAs for four rounds: one round of CTAs with more rows each takes 74 us for 16384 x
  // 2048 against 65, and eight take 75
  const long long most = (long long)num_sms() * per_sm * 4;
  const bool gate_rows = k.gate && k.gate_group < k.T;
  const int w = k.w_bf16 ? 2 : 4;
  const Ring ring = make_ring(N, !y ? 0 : k.y_bf16 ? 2 : 4, k.r_bf16 ? 2 : 4, 0, 0,
                              gate_rows ? w : 0, false, kSmemSm / per_sm - 1024);
  const size_t smem = (size_t)ring.bytes * ring.stages;
  cudaError_t e =
      set_smem_limit(reinterpret_cast<const void*>(norm_forward_kernel<TEAM>), (int)smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(norm_forward_kernel<TEAM>, dim3((unsigned)(want < most ? want : most)),
                    dim3(N), smem, stream, k, y, r, r_out, n_out, rstd_post, rstd_pre,
                    ring);
}

template <int TEAM>
cudaError_t backward_team(const Block& k, const BackwardArgs& g, const Plan& p,
                          cudaStream_t stream) {
  constexpr int N = bwd_threads(TEAM);
  const int r = k.r_bf16 ? 2 : 4, w = k.w_bf16 ? 2 : 4;
  const bool gate_rows = k.gate && p.it.group < k.T;
  const int vector = 4 * 4 * kQ * N;  // fp32 columns of every thread
  const int wpre = k.w_pre ? 4 * 4 * kQ * TEAM : 0;
  const int wpost =
      gate_rows && k.w_post && p.it.by_team && TEAM <= 256 ? 4 * 4 * kQ * TEAM : 0;
  const int post = gate_rows && g.part_post ? vector : 0;
  const int comb = gate_rows && !p.it.by_team ? vector : 0;
  // the widest rows' gate rows and w_post are read when they are needed, not ahead: with
  // fp32 arrays they would not fit
  const Ring ring = make_ring(N, !g.y ? 0 : k.y_bf16 ? 2 : 4, g.dn ? r : 0,
                              g.dr_out ? r : 0, !g.dn ? 0 : k.n_bf16 ? 2 : 4,
                              gate_rows && TEAM <= 256 ? w : 0, true,
                              kSmemSm - wpre - wpost - post - comb);
  // the last sums over the teams take the ring's place
  int at = ring.bytes * ring.stages;
  if (at < 2 * vector) at = 2 * vector;
  Extra x;
  x.wpre = at;
  x.wpost = wpost ? x.wpre + wpre : -1;
  x.post = x.wpre + wpre + wpost;
  x.comb = x.post + post;
  at = x.comb + comb;
  cudaError_t e = set_smem_limit(reinterpret_cast<const void*>(norm_backward_kernel<TEAM>), at);
  if (e != cudaSuccess) return e;
  return launch_pdl(norm_backward_kernel<TEAM>, dim3(p.ctas), dim3(p.threads), (size_t)at, stream,
                    k, g, p.it, ring, x);
}

}  // namespace

cudaError_t launch_norm_forward(const tw_norm_block& b, const void* y, const void* r, void* r_out,
                                void* n_out, float* rstd_post, float* rstd_pre,
                                cudaStream_t stream) {
  const Block k = device_block(b);
  auto run = [&](auto f) { return f(k, y, r, r_out, n_out, rstd_post, rstd_pre, stream); };
  switch (team_size_of(b.d)) {
    case 32: return run(forward_team<32>);
    case 64: return run(forward_team<64>);
    case 128: return run(forward_team<128>);
    case 256: return run(forward_team<256>);
    default: return run(forward_team<512>);
  }
}

size_t norm_backward_ws_bytes(int T, int d, int gate_group) {
  return parts_of(make_plan(T, d, gate_group, num_sms()), d, gate_group > 0).bytes;
}

cudaError_t launch_norm_backward(const tw_norm_block& b, const void* dn, const void* dr_out,
                                 const void* y, const void* r_out, const float* rstd_post,
                                 const float* rstd_pre, void* dy, void* dr, float* dw_post,
                                 float* dgate, float* dw_pre, void* ws, cudaStream_t stream) {
  const Block k = device_block(b);
  const Plan p = make_plan(b.T, b.d, b.gate ? b.gate_group : 0, num_sms());
  const Parts q = parts_of(p, b.d, b.gate != nullptr);
  auto at = [&](size_t off) { return reinterpret_cast<float*>(static_cast<char*>(ws) + off); };
  BackwardArgs g;
  g.dn = dn;
  g.dr_out = dr_out;
  g.y = y;
  g.r_out = r_out;
  g.rstd_post = rstd_post;
  g.rstd_pre = rstd_pre;
  g.dy = dy;
  g.dr = dr;
  g.part_pre = dw_pre ? at(q.pre) : nullptr;
  g.part_post = dw_post ? at(q.post) : nullptr;
  const bool gate_parts = dgate && p.it.per_group > 1;
  g.dgate = gate_parts ? at(q.gate) : dgate;
  cudaError_t e;
  switch (p.team) {
    case 32: e = backward_team<32>(k, g, p, stream); break;
    case 64: e = backward_team<64>(k, g, p, stream); break;
    case 128: e = backward_team<128>(k, g, p, stream); break;
    case 256: e = backward_team<256>(k, g, p, stream); break;
    default: e = backward_team<512>(k, g, p, stream); break;
  }
  if (e != cudaSuccess) return e;
  RowSums s;
  s.count = 0;
  s.d = b.d;
  s.first[0] = 0;
  auto add = [&](const float* part, float* out, int rows, int each) {
    s.s[s.count] = RowSum{part, out, rows, each};
    const long long units = (long long)rows * ((b.d + 31) / 32);
    const long long ctas = each <= kFewParts ? (units + kSumWarps - 1) / kSumWarps : units;
    s.first[s.count + 1] = s.first[s.count] + (int)ctas;
    ++s.count;
  };
  if (dw_pre) add(g.part_pre, dw_pre, 1, p.ctas);
  if (dw_post) add(g.part_post, dw_post, 1, p.ctas);
  if (gate_parts) add(g.dgate, dgate, p.it.count / p.it.per_group, p.it.per_group);
  if (s.count == 0) return cudaSuccess;
  return launch_pdl(norm_sum_kernel, dim3((unsigned)s.first[s.count]), dim3(kSumWarps * 32), 0,
                    stream, s);
}

}  // namespace tw
