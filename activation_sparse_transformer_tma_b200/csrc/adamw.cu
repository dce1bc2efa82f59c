// adamw.cu -- one AdamW step over many tensors, with fp32 or 8-bit moments
// (Loshchilov and Hutter, "Decoupled Weight Decay Regularization", 2019):
//   m = b1 m + (1 - b1) g;  v = b2 v + (1 - b2) g^2;
//   p = p (1 - lr wd) - lr/(1 - b1^t) m / (sqrt(v/(1 - b2^t)) + eps).
//
// Every element is read and written once, so the step is bound by memory.  A
// warp owns a block of 256 elements: lane l holds elements 4l..4l+3 of each
// half, so every access of a warp is one contiguous run of 16-byte (fp32),
// 8-byte (bf16) or 4-byte (codes) pieces, and the largest magnitude of a block
// of 8-bit states is one warp reduction.  The maximum is taken over the bits of
// |m| and v as integers: these order like the values, and a NaN is above all
// of them, so that it is not lost.
//
// 8-bit codes: m = s c|c| (int8), sqrt(v) = s c^2 (uint8).  The square law
// keeps the relative step at 2/c (1.6% and 0.8% at the block's largest value)
// over a range of 127^2 and 255^2; a linear code would round every value under
// 1/254 of the block's largest to zero, and a v rounded to zero would divide by
// eps.  The moments are rounded to nearest once a step; the update itself uses
// them unrounded.
//
// One block a warp and five CTAs of eight warps on an SM: more blocks a warp (16,
// 32 or 64 a CTA) were 2 to 20% slower, since a warp's loads do not overlap its
// own arithmetic, and forcing six CTAs on an SM spilled registers.  Measured on the
// three 8192 x 2048 matrices of a 2B layer: fp32 moments, fp32 masters and
// gradients, bf16 weights (30 bytes an element) 223 us, 6.8 TB/s; 8-bit moments, bf16
// gradients, with the values written (20 bytes) 161 to 173 us, 5.8 to 6.2 TB/s, with three quarters
// of the issue slots busy, and without them (16 bytes) 137 us, 5.9 TB/s.
//
// With device scalars one thread of a CTA reads them and works out the bias corrections in
// fp64, in front of the CTA's loads: 224, 174 and 153 us for the same three.
//
// The tensors' descriptors travel as kernel parameters: nothing has to stay
// alive after the call and a captured step replays with them.
#include "pdl.cuh"
#include "tw_common.cuh"
#include "tw_internal.h"

#include <cmath>

namespace tw {
namespace {

constexpr int kBlock = TW_ADAMW_BLOCK;
constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kBlocksPerCta = kWarps;  // one block a warp
constexpr int kCtasPerSm = 5;          // 48 registers a thread
static_assert(kBlock == 256, "a warp holds a block as two halves of 4 elements a lane");

struct Tensor {
  int64_t n;
  void* p;
  float* master;
  const void* g;
  void* m;
  void* v;
  float* m_scale;
  float* v_scale;
  void* m_values;
  void* v_values;
  double decay;
  float keep;  // 1 - lr * decay, unless lr_dev is given
  uint32_t p_bf16 : 1, g_bf16 : 1, values_bf16 : 1, small : 1;
};

struct Scalars {
  double lr, beta1, beta2;
  double bias1, bias2;  // 1 - beta^step, unless step_dev is given
  float eps, b1, c1, b2, c2;
  float size, rsqrt_bias2;  // lr / bias1 and 1 / sqrt(bias2) without device scalars
  bool dynamic;             // any device scalar
  const float* lr_dev;
  const int32_t* step_dev;
  const float* grad_scale;
};

template <int CAP>
struct Batch {
  int count;
  int32_t first_cta[CAP + 1];  // prefix sums of the tensors' CTAs
  Scalars s;
  Tensor t[CAP];
};

// Four consecutive elements; `valid` of them exist (4: one vector access).
TW_DEV void load4(const void* base, bool bf16, int64_t i, int valid, float (&x)[4]) {
  if (valid == 4) {
    if (bf16) {
      const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(base) + i);
      x[0] = bf16_lo(w.x); x[1] = bf16_hi(w.x); x[2] = bf16_lo(w.y); x[3] = bf16_hi(w.y);
    } else {
      const float4 w = *reinterpret_cast<const float4*>(static_cast<const float*>(base) + i);
      x[0] = w.x; x[1] = w.y; x[2] = w.z; x[3] = w.w;
    }
    return;
  }
#pragma unroll
  for (int k = 0; k < 4; ++k)
    x[k] = k >= valid ? 0.f
           : bf16     ? bf16_to_f32(static_cast<const uint16_t*>(base)[i + k])
                      : static_cast<const float*>(base)[i + k];
}
TW_DEV void store4(void* base, bool bf16, int64_t i, int valid, const float (&x)[4]) {
  if (valid == 4) {
    if (bf16)
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(base) + i) =
          make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]));
    else
      *reinterpret_cast<float4*>(static_cast<float*>(base) + i) =
          make_float4(x[0], x[1], x[2], x[3]);
    return;
  }
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if (k < valid) {
      if (bf16) static_cast<uint16_t*>(base)[i + k] = f32_to_bf16(x[k]);
      else static_cast<float*>(base)[i + k] = x[k];
    }
}
// Four codes as one word, the first in the lowest byte.
TW_DEV uint32_t load_codes(const void* base, int64_t i, int valid) {
  if (valid == 4) return *reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(base) + i);
  uint32_t w = 0;
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if (k < valid) w |= (uint32_t) static_cast<const uint8_t*>(base)[i + k] << (8 * k);
  return w;
}
TW_DEV void store_codes(void* base, int64_t i, int valid, uint32_t w) {
  if (valid == 4) {
    *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(base) + i) = w;
    return;
  }
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if (k < valid) static_cast<uint8_t*>(base)[i + k] = (uint8_t)(w >> (8 * k));
}

// The approximate instructions, values below 2^-126 as zero (their exact handling
// was a seventh of the 8-bit form's instructions).
TW_DEV float sqrt_approx(float x) {
  float r;
  asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
TW_DEV float reciprocal_approx(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Codes and floats without conversion instructions, which run at a quarter of
// the rate: a byte in the low mantissa bits of 2^23 is that integer above 2^23,
// and adding 1.5 * 2^23 rounds a small float to the nearest integer, in two's
// complement in the low bits.
constexpr float kMagic = 12582912.f;  // 1.5 * 2^23
TW_DEV float byte_above_2_23(uint32_t word, int k) {
  return __uint_as_float(__byte_perm(word, 0x4B000000u, 0x7440u + k));
}
TW_DEV uint32_t pack_bytes(const float (&a)[4]) {
  const uint32_t lo = __byte_perm(__float_as_uint(a[0]), __float_as_uint(a[1]), 0x0040);
  const uint32_t hi = __byte_perm(__float_as_uint(a[2]), __float_as_uint(a[3]), 0x0040);
  return __byte_perm(lo, hi, 0x5410);
}

struct Step {
  float gscale, b1, c1, b2, c2, rsqrt_bias2, eps, size, keep;
};

// One block of 256 elements by one warp (FULL: all of them exist).  With 8-bit moments the square roots
// and the division are the approximate instructions (2 ulp, against codes
// that are off by up to 0.8%): the IEEE forms' extra instructions, not memory,
// bounded that form.
template <bool SMALL, bool FULL>
TW_DEV void step_block(const Tensor& t, const Step& st, int64_t block, int lane) {
  const int64_t at[2] = {block * kBlock + lane * 4, block * kBlock + 128 + lane * 4};
  int valid[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int64_t left = t.n - at[h];
    valid[h] = FULL || left >= 4 ? 4 : left > 0 ? (int)left : 0;
  }
  const void* from = t.master ? static_cast<const void*>(t.master) : t.p;
  const bool from_bf16 = t.p_bf16 && !t.master;
  float g[2][4], p[2][4], m[2][4], v[2][4];
  uint32_t mc[2], vc[2];
  float ms = 0.f, vs = 0.f;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    load4(t.g, t.g_bf16, at[h], valid[h], g[h]);
    load4(from, from_bf16, at[h], valid[h], p[h]);
    if (SMALL) {
      mc[h] = load_codes(t.m, at[h], valid[h]);
      vc[h] = load_codes(t.v, at[h], valid[h]);
    } else {
      load4(t.m, false, at[h], valid[h], m[h]);
      load4(t.v, false, at[h], valid[h], v[h]);
    }
  }
  if (SMALL) {
    ms = t.m_scale[block];
    vs = t.v_scale[block];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float c = byte_above_2_23(mc[h] ^ 0x80808080u, k) - 8388736.f;  // 2^23 + 128
        m[h][k] = c * fabsf(c) * ms;
        const float b = byte_above_2_23(vc[h], k) - 8388608.f;
        const float root = b * b * vs;
        v[h][k] = root * root;
      }
  }
  float root[2][4];
  uint32_t mtop = 0, vtop = 0;
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float gs = g[h][k] * st.gscale;
      const float mn = m[h][k] = fmaf(st.b1, m[h][k], st.c1 * gs);
      const float vn = v[h][k] = fmaf(st.b2, v[h][k], st.c2 * gs * gs);
      const float r = root[h][k] = SMALL ? sqrt_approx(vn) : sqrtf(vn);
      const float den = fmaf(r, st.rsqrt_bias2, st.eps);
      const float q = SMALL ? mn * reciprocal_approx(den) : __fdiv_rn(mn, den);
      p[h][k] = fmaf(p[h][k], st.keep, -st.size * q);
      // elements past n take no part in the block's maximum, whatever a
      // block scale of NaN made of them
      if (SMALL && k < valid[h]) {
        mtop = max(mtop, __float_as_uint(mn) & 0x7FFFFFFFu);
        vtop = max(vtop, __float_as_uint(r));
      }
    }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if (t.master) store4(t.master, false, at[h], valid[h], p[h]);
    store4(t.p, t.p_bf16, at[h], valid[h], p[h]);
    if (!SMALL) {
      store4(t.m, false, at[h], valid[h], m[h]);
      store4(t.v, false, at[h], valid[h], v[h]);
    }
  }
  if (!SMALL) return;
  const float mmax = __uint_as_float(__reduce_max_sync(0xFFFFFFFFu, mtop));
  const float vmax = __uint_as_float(__reduce_max_sync(0xFFFFFFFFu, vtop));
  // below 2^-127 the reciprocal is infinite: such a block of m is held as zero
  const float minv = mmax < 5.9e-39f ? 0.f : 1.f / mmax;
  const float vinv = vmax == 0.f ? 0.f : 1.f / vmax;
  // a block with a value that is not finite has a scale of NaN, and no part of it
  // decodes to a number
  ms = !(mmax < INFINITY) ? NAN : minv == 0.f ? 0.f : mmax * (1.f / 16129.f);
  vs = !(vmax < INFINITY) ? NAN : vmax * (1.f / 65025.f);
  if (lane == 0) {
    t.m_scale[block] = ms;
    t.v_scale[block] = vs;
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float mw[4], vw[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      mw[k] = copysignf(127.f * sqrt_approx(fabsf(m[h][k]) * minv), m[h][k]) + kMagic;
      // at least code 1 where v is not zero: one position below it rounds up to it
      const float pos = 255.f * sqrt_approx(root[h][k] * vinv);
      vw[k] = (root[h][k] > 0.f ? fmaxf(pos, 1.f) : pos) + kMagic;
    }
    store_codes(t.m, at[h], valid[h], pack_bytes(mw));
    store_codes(t.v, at[h], valid[h], pack_bytes(vw));
    if (t.m_values) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float c = mw[k] - kMagic, b = vw[k] - kMagic;
        mw[k] = c * fabsf(c) * ms;
        const float r = b * b * vs;
        vw[k] = r * r;
      }
      store4(t.m_values, t.values_bf16, at[h], valid[h], mw);
      store4(t.v_values, t.values_bf16, at[h], valid[h], vw);
    }
  }
}

template <int CAP>
__global__ void __launch_bounds__(kThreads, kCtasPerSm)
    adamw_kernel(const __grid_constant__ Batch<CAP> b) {
  __shared__ Step dynamic;
  const int cta = blockIdx.x;
  int lo = 0, hi = b.count - 1;  // the last tensor whose first CTA is not past this one
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (b.first_cta[mid] <= cta) lo = mid;
    else hi = mid - 1;
  }
  const Tensor& t = b.t[lo];
  pdl_wait();
  pdl_launch_next();
  const Scalars& s = b.s;
  Step st;
  st.gscale = 1.f;
  st.b1 = s.b1;
  st.c1 = s.c1;
  st.b2 = s.b2;
  st.c2 = s.c2;
  st.eps = s.eps;
  st.rsqrt_bias2 = s.rsqrt_bias2;
  st.size = s.size;
  st.keep = t.keep;
  if (s.dynamic) {
    if (threadIdx.x == 0) {
      double bias1 = s.bias1, bias2 = s.bias2;
      if (s.step_dev) {
        // beta^step by squaring, in fp64: 1 - beta^step loses digits in fp32
        const int32_t at = *s.step_dev;
        double p1 = 1.0, p2 = 1.0, q1 = s.beta1, q2 = s.beta2;
        for (int32_t e = at < 1 ? 1 : at; e > 0; e >>= 1) {
          if (e & 1) {
            p1 *= q1;
            p2 *= q2;
          }
          q1 *= q1;
          q2 *= q2;
        }
        bias1 = 1.0 - p1;
        bias2 = 1.0 - p2;
      }
      const double lr = s.lr_dev ? (double)*s.lr_dev : s.lr;
      dynamic.gscale = s.grad_scale ? *s.grad_scale : 1.f;
      dynamic.rsqrt_bias2 = (float)(1.0 / sqrt(bias2));
      dynamic.size = (float)(lr / bias1);
      dynamic.keep = (float)(1.0 - lr * t.decay);
    }
    __syncthreads();
    st.gscale = dynamic.gscale;
    st.rsqrt_bias2 = dynamic.rsqrt_bias2;
    st.size = dynamic.size;
    st.keep = dynamic.keep;
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t i = (int64_t)(cta - b.first_cta[lo]) * kBlocksPerCta + warp;
  if (i * kBlock >= t.n) return;
  const bool full = t.n - i * kBlock >= kBlock;
  if (t.small) {
    if (full) step_block<true, true>(t, st, i, lane);
    else step_block<true, false>(t, st, i, lane);
  } else {
    if (full) step_block<false, true>(t, st, i, lane);
    else step_block<false, false>(t, st, i, lane);
  }
}

// Kernel parameters end at 32,764 bytes; the small form keeps the usual step
// of one layer within the 4 KB that every launch copies cheaply.
constexpr int kFew = 32, kMany = 256;
static_assert(sizeof(Batch<kFew>) <= 4096 && sizeof(Batch<kMany>) <= 32764, "parameter space");

// Takes tensors from `at` on, as many as fit; returns the next one to take.
template <int CAP>
cudaError_t launch_some(const tw_adamw_tensor* tensors, int count, int* at, const Scalars& s,
                        cudaStream_t stream) {
  Batch<CAP> b;
  b.s = s;
  int n = 0;
  int64_t ctas = 0;
  while (*at < count && n < CAP) {
    const tw_adamw_tensor& t = tensors[*at];
    const int64_t blocks = (t.n + kBlock - 1) / kBlock;
    const int64_t need = (blocks + kBlocksPerCta - 1) / kBlocksPerCta;
    if (ctas + need > 0x7FFFFFFF) break;
    ++*at;
    if (t.n == 0) continue;
    Tensor& d = b.t[n];
    d.n = t.n;
    d.p = t.p;
    d.master = t.master;
    d.g = t.g;
    d.m = t.m;
    d.v = t.v;
    d.m_scale = t.m_scale;
    d.v_scale = t.v_scale;
    d.m_values = t.m_values;
    d.v_values = t.v_values;
    d.decay = t.weight_decay;
    d.keep = (float)(1.0 - s.lr * t.weight_decay);
    d.p_bf16 = t.p_dtype == TW_BF16;
    d.g_bf16 = t.g_dtype == TW_BF16;
    d.values_bf16 = t.values_dtype == TW_BF16;
    d.small = t.state_bits == 8;
    b.first_cta[n++] = (int32_t)ctas;
    ctas += need;
  }
  if (n == 0) return cudaSuccess;
  b.first_cta[n] = (int32_t)ctas;
  b.count = n;
  return launch_pdl(adamw_kernel<CAP>, dim3((unsigned)ctas), dim3(kThreads), 0, stream, b);
}

}  // namespace

cudaError_t launch_adamw(const tw_adamw_tensor* tensors, int count, const tw_adamw_args& a,
                         cudaStream_t stream) {
  Scalars s;
  s.lr = a.lr;
  s.beta1 = a.beta1;
  s.beta2 = a.beta2;
  s.bias1 = a.step_dev ? 1.0 : 1.0 - std::pow(a.beta1, a.step);
  s.bias2 = a.step_dev ? 1.0 : 1.0 - std::pow(a.beta2, a.step);
  s.eps = (float)a.eps;
  s.b1 = (float)a.beta1;
  s.c1 = (float)(1.0 - a.beta1);
  s.b2 = (float)a.beta2;
  s.c2 = (float)(1.0 - a.beta2);
  s.size = (float)(s.lr / s.bias1);
  s.rsqrt_bias2 = (float)(1.0 / std::sqrt(s.bias2));
  s.dynamic = a.lr_dev || a.step_dev || a.grad_scale;
  s.lr_dev = a.lr_dev;
  s.step_dev = a.step_dev;
  s.grad_scale = a.grad_scale;
  for (int at = 0; at < count;) {
    const cudaError_t e = count - at <= kFew
                              ? launch_some<kFew>(tensors, count, &at, s, stream)
                              : launch_some<kMany>(tensors, count, &at, s, stream);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace tw
