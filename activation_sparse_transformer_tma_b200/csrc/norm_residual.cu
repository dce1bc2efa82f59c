// norm_residual.cu -- the RMS norms before and after a block, fused with the
// block's gate, its residual scale and the residual sum (Zhang and Sennrich,
// "Root Mean Square Layer Normalization", 2019), forward and backward:
//   o = y rstd_post w_post,  r' = a r + s gate o,  n = r' rstd_pre w_pre.
//
// Both directions read and write each element once and are bound by memory:
// 12 bytes an element forward and 18 backward for bf16 y and n and an fp32
// residual stream.  A team of 32 ceil(d / 256) threads holds one row in
// registers, two groups of 4 columns a thread (4 tid and 4 (tid + team)), so every
// access is contiguous over a warp (16 bytes a lane in fp32, 8 in bf16) and the
// weights of a thread's columns, and in the backward their gradients, stay in
// registers over all its rows.  A row needs two reductions over d, the second of
// them on the first's result; the next row's loads are issued before them.
//
// Backward: the gradients of the weights are sums over tokens.  Each CTA sums its
// rows in registers and over its teams in shared memory, and leaves one partial
// row; a second kernel adds the partial rows in a fixed order.  No atomics: the
// result does not depend on timing.
#include "pdl.cuh"
#include "tw_common.cuh"
#include "tw_internal.h"

namespace tw {
namespace {

// Four columns of a row, as loaded.
template <bool BF>
struct Quad;
template <>
struct Quad<true> {
  uint2 w;
  TW_DEV void load(const void* base, size_t i) {
    w = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(base) + i);
  }
  TW_DEV void zero() { w = make_uint2(0u, 0u); }
  TW_DEV void get(float (&x)[4]) const {
    x[0] = bf16_lo(w.x); x[1] = bf16_hi(w.x); x[2] = bf16_lo(w.y); x[3] = bf16_hi(w.y);
  }
};
template <>
struct Quad<false> {
  float4 w;
  TW_DEV void load(const void* base, size_t i) {
    w = *reinterpret_cast<const float4*>(static_cast<const float*>(base) + i);
  }
  TW_DEV void zero() { w = make_float4(0.f, 0.f, 0.f, 0.f); }
  TW_DEV void get(float (&x)[4]) const { x[0] = w.x; x[1] = w.y; x[2] = w.z; x[3] = w.w; }
};

TW_DEV void load4(const void* base, bool bf16, size_t i, float (&x)[4]) {
  if (bf16) {
    Quad<true> q;
    q.load(base, i);
    q.get(x);
  } else {
    Quad<false> q;
    q.load(base, i);
    q.get(x);
  }
}
TW_DEV void store4(void* base, bool bf16, size_t i, const float (&x)[4]) {
  if (bf16)
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(base) + i) =
        make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]));
  else
    *reinterpret_cast<float4*>(static_cast<float*>(base) + i) = make_float4(x[0], x[1], x[2], x[3]);
}

struct Block {
  int T, d, gate_group;
  float a, s, eps, inv_d;
  bool y_bf16, r_bf16, n_bf16, w_bf16;
  const void *w_post, *gate, *w_pre;
};

// Threads of one row, and this thread's two groups of columns.
struct Team {
  int size, index, tid, warps;
  int col[2];
  bool in[2];
  TW_DEV Team(int d, int team_size) {
    size = team_size;
    index = threadIdx.x / team_size;
    tid = threadIdx.x - index * team_size;
    warps = team_size >> 5;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      col[h] = 4 * (tid + h * team_size);
      in[h] = col[h] < d;
    }
  }
  // Sum over the team, in a fixed order.  `slots` holds one float per warp of the
  // CTA and alternates between two arrays: a thread that writes an array again has
  // passed the barrier of the other one, so all have read it.
  TW_DEV float sum(float v, float (*slots)[32], int& turn) const {
    v = warp_sum(v);
    if (warps == 1) return v;
    float* at = slots[turn] + index * warps;
    turn ^= 1;
    if ((threadIdx.x & 31) == 0) at[tid >> 5] = v;
    asm volatile("bar.sync %0, %1;" ::"r"(1 + index), "r"(size) : "memory");
    v = 0.f;
    for (int w = 0; w < warps; ++w) v += at[w];
    return v;
  }
};

template <bool YB, bool RB>
struct ForwardRow {
  Quad<YB> y[2];
  Quad<RB> r[2];
  TW_DEV void load(const Team& tm, const void* yp, const void* rp, size_t row, int d) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      y[h].zero();
      r[h].zero();
      if (tm.in[h]) {
        if (yp) y[h].load(yp, row * d + tm.col[h]);
        r[h].load(rp, row * d + tm.col[h]);
      }
    }
  }
};

template <bool YB, bool RB, int MAXT>
__global__ void __launch_bounds__(MAXT, MAXT <= 256 ? 3 : 1)
    norm_forward_kernel(const Block b, const void* y, const void* r, void* r_out, void* n_out,
                        float* rstd_post, float* rstd_pre, int team_size) {
  __shared__ float slots[2][32];
  const Team tm(b.d, team_size);
  const int teams = blockDim.x / team_size;
  const long long stride = (long long)gridDim.x * teams;
  long long row = (long long)blockIdx.x * teams + tm.index;
  int turn = 0;
  pdl_wait();
  pdl_launch_next();
  // c = block_scale * gate * w_post of this thread's columns, kept over its rows
  // unless tokens have gate rows of their own
  float c[2][4], wpre[2][4];
  const bool gate_rows = b.gate && b.gate_group < b.T;
  auto scales = [&](size_t gate_row) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (!tm.in[h]) continue;
      float w[4] = {1.f, 1.f, 1.f, 1.f}, gt[4] = {1.f, 1.f, 1.f, 1.f};
      if (b.w_post) load4(b.w_post, b.w_bf16, tm.col[h], w);
      if (b.gate) load4(b.gate, b.w_bf16, gate_row * b.d + tm.col[h], gt);
#pragma unroll
      for (int k = 0; k < 4; ++k) c[h][k] = b.s * gt[k] * w[k];
    }
  };
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int k = 0; k < 4; ++k) c[h][k] = wpre[h][k] = 0.f;
  if (y && !gate_rows) scales(0);
  if (b.w_pre) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
      if (tm.in[h]) load4(b.w_pre, b.w_bf16, tm.col[h], wpre[h]);
  }
  ForwardRow<YB, RB> next;
  if (row < b.T) next.load(tm, y, r, row, b.d);
  for (; row < b.T; row += stride) {
    const ForwardRow<YB, RB> cur = next;
    if (row + stride < b.T) next.load(tm, y, r, row + stride, b.d);
    float rv[2][4];
#pragma unroll
    for (int h = 0; h < 2; ++h) cur.r[h].get(rv[h]);
    if (y) {
      if (gate_rows) scales((size_t)((int)row / b.gate_group));
      float yv[2][4];
#pragma unroll
      for (int h = 0; h < 2; ++h) cur.y[h].get(yv[h]);
      float p = 1.f;
      if (b.w_post) {
        float ss = 0.f;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int k = 0; k < 4; ++k) ss = fmaf(yv[h][k], yv[h][k], ss);
        p = 1.f / sqrtf(fmaf(tm.sum(ss, slots, turn), b.inv_d, b.eps));
        if (rstd_post && tm.tid == 0) rstd_post[row] = p;
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int k = 0; k < 4; ++k) rv[h][k] = fmaf(yv[h][k] * p, c[h][k], b.a * rv[h][k]);
        if (tm.in[h]) store4(r_out, RB, (size_t)row * b.d + tm.col[h], rv[h]);
      }
    }
    if (b.w_pre) {
      float ss = 0.f;
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int k = 0; k < 4; ++k) ss = fmaf(rv[h][k], rv[h][k], ss);
      const float p = 1.f / sqrtf(fmaf(tm.sum(ss, slots, turn), b.inv_d, b.eps));
      if (rstd_pre && tm.tid == 0) rstd_pre[row] = p;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float nv[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) nv[k] = rv[h][k] * p * wpre[h][k];
        if (tm.in[h]) store4(n_out, b.n_bf16, (size_t)row * b.d + tm.col[h], nv);
      }
    }
  }
}

// ----------------------------------------------------------------- backward --
// Rows are dealt out in items: at most rows_per_item consecutive rows of one gate
// group (per_group items cover a group).  An item belongs to a CTA, whose teams
// share its rows, or with short groups (by_team) to one team; either way the gate
// row's gradient is complete, or one partial of per_group, when the item is done.
struct Items {
  int group, rows_per_item, per_group, count;
  bool by_team;
};

template <bool YB, bool RB, bool NB>
struct BackwardRow {
  Quad<YB> y[2];
  Quad<RB> r[2], dr[2];
  Quad<NB> dn[2];
  float ppost, ppre;
};

struct BackwardArgs {
  const void *dn, *dr_out, *y, *r_out;
  const float *rstd_post, *rstd_pre;
  void *dy, *dr;
  float* dgate;      // where an item's gate gradient goes: row (per_group == 1 ? group : item)
  float* part_post;  // [CTAs][d]
  float* part_pre;   // [CTAs][d]
};

template <bool YB, bool RB, bool NB, int MAXT>
__global__ void __launch_bounds__(MAXT, 1)
    norm_backward_kernel(const Block b, const BackwardArgs g, const Items it, int team_size) {
  __shared__ float slots[2][32];
  __shared__ float4 comb[MAXT * 2];  // the other teams' sums of one vector
  const Team tm(b.d, team_size);
  const int teams = blockDim.x / team_size;
  const int units = it.by_team ? gridDim.x * teams : gridDim.x;
  const int unit = it.by_team ? blockIdx.x * teams + tm.index : blockIdx.x;
  const int first = it.by_team ? 0 : tm.index;   // this team's first row of an item
  const int stride = it.by_team ? 1 : teams;
  int turn = 0;
  pdl_wait();
  pdl_launch_next();

  float wpost[2][4], wpre[2][4], gate[2][4];
  float apost[2][4], apre[2][4], agate[2][4];
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      wpost[h][k] = gate[h][k] = 1.f;
      wpre[h][k] = apost[h][k] = apre[h][k] = agate[h][k] = 0.f;
    }
#pragma unroll
  for (int h = 0; h < 2; ++h)
    if (tm.in[h]) {
      if (b.w_post) load4(b.w_post, b.w_bf16, tm.col[h], wpost[h]);
      if (b.w_pre) load4(b.w_pre, b.w_bf16, tm.col[h], wpre[h]);
    }

  auto range = [&](int item, int& row0, int& row1) {
    const int group = item / it.per_group, part = item - group * it.per_group;
    // group * it.group < T, so only the ends can pass T (and, added up, 2^31)
    const long long g0 = (long long)group * it.group;
    const long long g1 = g0 + it.group < b.T ? g0 + it.group : b.T;
    long long r0 = g0 + (long long)part * it.rows_per_item;
    if (r0 > g1) r0 = g1;
    row0 = (int)r0;
    row1 = (int)(r0 + it.rows_per_item < g1 ? r0 + it.rows_per_item : g1);
  };
  using Row = BackwardRow<YB, RB, NB>;
  auto load = [&](Row& w, int row) {
    const size_t at = (size_t)row * b.d;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      w.y[h].zero();
      w.r[h].zero();
      w.dr[h].zero();
      w.dn[h].zero();
      if (tm.in[h]) {
        const size_t i = at + tm.col[h];
        if (g.y) w.y[h].load(g.y, i);
        if (g.dn) {
          w.dn[h].load(g.dn, i);
          w.r[h].load(g.r_out, i);
        }
        if (g.dr_out) w.dr[h].load(g.dr_out, i);
      }
    }
    w.ppost = g.rstd_post ? g.rstd_post[row] : 1.f;
    w.ppre = g.rstd_pre ? g.rstd_pre[row] : 0.f;
  };
  // Adds a vector over the teams into the first team's registers (all threads).
  auto combine = [&](float (&v)[2][4]) {
    if (teams == 1) return;
    __syncthreads();
    if (tm.index > 0) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
        comb[((tm.index - 1) * team_size + tm.tid) * 2 + h] =
            make_float4(v[h][0], v[h][1], v[h][2], v[h][3]);
    }
    __syncthreads();
    if (tm.index == 0)
      for (int t = 0; t + 1 < teams; ++t)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float4 o = comb[(t * team_size + tm.tid) * 2 + h];
          v[h][0] += o.x; v[h][1] += o.y; v[h][2] += o.z; v[h][3] += o.w;
        }
  };

  Row next;
  bool have = false;  // `next` holds the row that comes next
  for (long long next_item = unit; next_item < it.count; next_item += units) {
    const int item = (int)next_item;
    int row0, row1;
    range(item, row0, row1);
    const int group = item / it.per_group;
    if (b.gate) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (tm.in[h]) load4(b.gate, b.w_bf16, (size_t)group * b.d + tm.col[h], gate[h]);
    }
    for (long long at_row = (long long)row0 + first; at_row < row1; at_row += stride) {
      const int row = (int)at_row;
      if (!have) load(next, row);
      const Row cur = next;
      have = false;
      if (stride < row1 - row) {
        load(next, row + stride);
        have = true;
      } else if (units < it.count - item) {
        int n0, n1;
        range(item + units, n0, n1);
        if (first < n1 - n0) {
          load(next, n0 + first);
          have = true;
        }
      }
      float G[2][4];
#pragma unroll
      for (int h = 0; h < 2; ++h) cur.dr[h].get(G[h]);
      if (g.dn) {
        float dn[2][4], rh[2][4];
        float inner = 0.f;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          cur.dn[h].get(dn[h]);
          cur.r[h].get(rh[h]);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            rh[h][k] *= cur.ppre;
            apre[h][k] = fmaf(dn[h][k], rh[h][k], apre[h][k]);
            dn[h][k] *= wpre[h][k];
            inner = fmaf(dn[h][k], rh[h][k], inner);
          }
        }
        inner = tm.sum(inner, slots, turn) * b.inv_d;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            G[h][k] = fmaf(cur.ppre, fmaf(-rh[h][k], inner, dn[h][k]), G[h][k]);
      }
      const size_t at = (size_t)row * b.d;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float out[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) out[k] = b.a * G[h][k];
        if (tm.in[h]) store4(g.dr, RB, at + tm.col[h], out);
      }
      if (g.dy) {
        float yh[2][4], f[2][4];
        float inner = 0.f;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          cur.y[h].get(yh[h]);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            yh[h][k] *= cur.ppost;
            const float sg = b.s * G[h][k], kk = sg * gate[h][k];
            agate[h][k] = fmaf(sg, yh[h][k] * wpost[h][k], agate[h][k]);
            apost[h][k] = fmaf(kk, yh[h][k], apost[h][k]);
            f[h][k] = kk * wpost[h][k];
            inner = fmaf(f[h][k], yh[h][k], inner);
          }
        }
        if (b.w_post) {
          inner = tm.sum(inner, slots, turn) * b.inv_d;
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int k = 0; k < 4; ++k) f[h][k] = cur.ppost * fmaf(-yh[h][k], inner, f[h][k]);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (tm.in[h]) store4(g.dy, YB, at + tm.col[h], f[h]);
      }
    }
    if (b.gate) {
      if (!it.by_team) combine(agate);
      if (it.by_team || tm.index == 0) {
        float* to = g.dgate + (size_t)(it.per_group == 1 ? group : item) * b.d;
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (tm.in[h]) store4(to, false, tm.col[h], agate[h]);
      }
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int k = 0; k < 4; ++k) agate[h][k] = 0.f;
    }
  }
  if (g.part_pre) {
    combine(apre);
    if (tm.index == 0)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (tm.in[h]) store4(g.part_pre + (size_t)blockIdx.x * b.d, false, tm.col[h], apre[h]);
  }
  if (g.part_post) {
    combine(apost);
    if (tm.index == 0)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (tm.in[h]) store4(g.part_post + (size_t)blockIdx.x * b.d, false, tm.col[h], apost[h]);
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
  int first[4];  // prefix sums of the output rows
  int count, d;
};

// 32 columns of one output row a CTA, its partial rows dealt over 16 warps and
// their 16 sums added in order.
constexpr int kSumWarps = 16;
__global__ void __launch_bounds__(kSumWarps * 32) norm_sum_kernel(const RowSums a) {
  __shared__ float sums[kSumWarps][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int strips = (a.d + 31) / 32;
  const int at = blockIdx.x / strips, c = (blockIdx.x - at * strips) * 32 + lane;
  int i = 0;
  while (i + 1 < a.count && at >= a.first[i + 1]) ++i;
  const RowSum& s = a.s[i];
  const int row = at - a.first[i];
  pdl_wait();
  pdl_launch_next();
  float v = 0.f;
  if (c < a.d) {
    const float* p = s.part + (size_t)row * s.each * a.d + c;
    for (int k = warp; k < s.each; k += kSumWarps) v += p[(size_t)k * a.d];
  }
  sums[warp][lane] = v;
  __syncthreads();
  if (warp == 0 && c < a.d) {
    v = 0.f;
#pragma unroll
    for (int k = 0; k < kSumWarps; ++k) v += sums[k][lane];
    s.out[(size_t)row * a.d + c] = v;
  }
}

int team_size_of(int d) { return 32 * ((d + 255) / 256); }

// The backward's launch: CTAs, and how rows are dealt out.  The same rule sizes the
// workspace, from T, d and gate_group alone (sms: the SMs of the current device).
struct Plan {
  Items it;
  int ctas, threads, team;
};
constexpr int kBwdThreads = 512;
// Groups shorter than this go to one team each: a CTA's teams would share too few
// rows of one, and meet at a barrier after each.
constexpr int kShortGroup = 32;

Plan make_plan(int T, int d, int gate_group, int sms) {
  Plan p;
  p.team = team_size_of(d);
  const int teams = p.team >= kBwdThreads ? 1 : kBwdThreads / p.team;
  p.threads = teams * p.team;
  const long long T64 = T;
  const int group = gate_group <= 0 || gate_group > T ? (T > 0 ? T : 1) : gate_group;
  const int groups = (int)((T64 + group - 1) / group);
  p.it.group = group;
  p.it.by_team = group < kShortGroup && groups > 1;
  if (p.it.by_team) {
    p.it.per_group = 1;
    p.it.rows_per_item = group;
  } else {
    // enough items for every SM; an item has a row for each team at least
    long long per = groups >= sms ? 1 : (sms + groups - 1) / groups;
    const long long most = (group + teams - 1) / teams;
    if (per > most) per = most;
    p.it.rows_per_item = (int)((group + per - 1) / per);
    p.it.per_group = (group + p.it.rows_per_item - 1) / p.it.rows_per_item;
  }
  p.it.count = groups * p.it.per_group;
  const int units = p.it.by_team ? (p.it.count + teams - 1) / teams : p.it.count;
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

template <bool YB, bool RB>
cudaError_t forward_dtyped(const Block& k, const void* y, const void* r, void* r_out, void* n_out,
                           float* rstd_post, float* rstd_pre, cudaStream_t stream) {
  const int team = team_size_of(k.d);
  const int teams = team >= 256 ? 1 : 256 / team;
  const long long want = ((long long)k.T + teams - 1) / teams;
  const long long most = (long long)num_sms() * (team <= 256 ? 3 : 1024 / team);
  const dim3 grid((unsigned)(want < most ? want : most)), block(teams * team);
  if (team <= 256)
    return launch_pdl(norm_forward_kernel<YB, RB, 256>, grid, block, 0, stream, k, y, r, r_out,
                      n_out, rstd_post, rstd_pre, team);
  return launch_pdl(norm_forward_kernel<YB, RB, 1024>, grid, block, 0, stream, k, y, r, r_out,
                    n_out, rstd_post, rstd_pre, team);
}

template <bool YB, bool RB, bool NB>
cudaError_t backward_dtyped(const Block& k, const BackwardArgs& g, const Plan& p,
                            cudaStream_t stream) {
  if (p.threads <= kBwdThreads)
    return launch_pdl(norm_backward_kernel<YB, RB, NB, kBwdThreads>, dim3(p.ctas),
                      dim3(p.threads), 0, stream, k, g, p.it, p.team);
  return launch_pdl(norm_backward_kernel<YB, RB, NB, 1024>, dim3(p.ctas), dim3(p.threads), 0,
                    stream, k, g, p.it, p.team);
}

}  // namespace

cudaError_t launch_norm_forward(const tw_norm_block& b, const void* y, const void* r, void* r_out,
                                void* n_out, float* rstd_post, float* rstd_pre,
                                cudaStream_t stream) {
  const Block k = device_block(b);
  if (k.y_bf16)
    return k.r_bf16 ? forward_dtyped<true, true>(k, y, r, r_out, n_out, rstd_post, rstd_pre, stream)
                    : forward_dtyped<true, false>(k, y, r, r_out, n_out, rstd_post, rstd_pre, stream);
  return k.r_bf16 ? forward_dtyped<false, true>(k, y, r, r_out, n_out, rstd_post, rstd_pre, stream)
                  : forward_dtyped<false, false>(k, y, r, r_out, n_out, rstd_post, rstd_pre, stream);
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
  const int kind = (k.y_bf16 ? 4 : 0) | (k.r_bf16 ? 2 : 0) | (k.n_bf16 ? 1 : 0);
  switch (kind) {
    case 0: e = backward_dtyped<false, false, false>(k, g, p, stream); break;
    case 1: e = backward_dtyped<false, false, true>(k, g, p, stream); break;
    case 2: e = backward_dtyped<false, true, false>(k, g, p, stream); break;
    case 3: e = backward_dtyped<false, true, true>(k, g, p, stream); break;
    case 4: e = backward_dtyped<true, false, false>(k, g, p, stream); break;
    case 5: e = backward_dtyped<true, false, true>(k, g, p, stream); break;
    case 6: e = backward_dtyped<true, true, false>(k, g, p, stream); break;
    default: e = backward_dtyped<true, true, true>(k, g, p, stream); break;
  }
  if (e != cudaSuccess) return e;
  RowSums s;
  s.count = 0;
  s.d = b.d;
  s.first[0] = 0;
  auto add = [&](const float* part, float* out, int rows, int each) {
    s.s[s.count] = RowSum{part, out, rows, each};
    s.first[s.count + 1] = s.first[s.count] + rows;
    ++s.count;
  };
  if (dw_pre) add(g.part_pre, dw_pre, 1, p.ctas);
  if (dw_post) add(g.part_post, dw_post, 1, p.ctas);
  if (gate_parts) add(g.dgate, dgate, p.it.count / p.it.per_group, p.it.per_group);
  if (s.count == 0) return cudaSuccess;
  const unsigned strips = (unsigned)(b.d + 31) / 32;
  return launch_pdl(norm_sum_kernel, dim3(strips * (unsigned)s.first[s.count]),
                    dim3(kSumWarps * 32), 0, stream, s);
}

}  // namespace tw
