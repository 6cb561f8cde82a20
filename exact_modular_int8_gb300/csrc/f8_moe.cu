// f8_moe.cu -- a whole mixture-of-experts layer for a few tokens.
//
//   p = softmax(x Wr^T); the top_k largest (ties: the lower index), weighted by
//   p or, renormalised, by p over their sum
//   y = sum_e w_e (silu(x G_e^T) * (x U_e^T)) D_e^T
//
// G and U are the upper and lower halves of W13 [E][2I][H], D is W2 [E][H][I],
// both E4M3 with one fp32 scale per 128 x 128 tile.  With a few tokens the
// work is reading the chosen experts' weights once.
//
// The products run on warp-level MMAs (m16n8k16, fp16 operands, fp32 sums)
// with the weights as the 16-row operand and up to eight tokens as columns:
// E4M3 is exact in fp16, and the MMA's order of k is free as long as both
// operands agree, so a lane's 16 consecutive bytes of a weight row feed four
// MMAs without any shuffle.  tcgen05 would want the tokens padded to its tiles
// and quantised to E4M3 too; here the pass is bound by memory.  Activations
// enter as fp16 scaled by a power of two per row (their largest magnitude in
// [2^14, 2^15)): exact for bf16 and fp16 entries within 2^-29 of the row's
// largest, off by at most 2^-40 of it below.  The gated product h is kept in
// fp32 and rounded to fp16 the same way when it enters the second product
// (relative 2^-12 per entry, an eighth of a bf16 result's rounding).  Each
// 128-block's sum is scaled in fp32 and added to fp32 sums.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <cstdint>
#include <mutex>

#include "f8_kernels.h"

namespace rg {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kMaxT = RG_MOE_MAX_TOKENS;
constexpr int kMaxK = RG_MOE_MAX_TOP_K;
constexpr int kMaxE = RG_MOE_MAX_EXPERTS;
constexpr int kSlots = kMaxT * kMaxK;

struct MoeWs {
  float* logits;     // [T][E]
  __half* xs;        // [T][H] x times 2^n
  float* x_inv;      // [T] 2^-n
  float* h;          // [T * top_k][I]
  uint32_t* h_max;   // [T * top_k] largest |h|, as bits
  float* part;       // [T * top_k][H] the experts' outputs
};

struct MoeParams {
  const void* X;
  const void* WR;
  const uint8_t* W13;
  const float* S13;
  const uint8_t* W2;
  const float* S2;
  void* Y;
  int T, H, I, E, top_k;
  int type;  // of X, WR and Y
  int renorm;
  MoeWs w;
};

template <typename T>
__device__ __forceinline__ float to_f(T v);
template <>
__device__ __forceinline__ float to_f(__half v) { return __half2float(v); }
template <>
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void from_f(float v, __half& o) { o = __float2half_rn(v); }
__device__ __forceinline__ void from_f(float v, __nv_bfloat16& o) { o = __float2bfloat16_rn(v); }

// The power of two that brings a largest magnitude (as bits) to [2^14, 2^15),
// and its inverse.  Zero, inf and NaN rows are left alone; the exponent is
// bounded so that both stay normal.
__device__ __forceinline__ float2 pow2_scale(uint32_t max_bits) {
  int e = (int)(max_bits >> 23) - 127;
  if (max_bits == 0 || e == 128) return make_float2(1.0f, 1.0f);
  e = max(e, -110);
  return make_float2(__int_as_float((127 + 14 - e) << 23), __int_as_float((127 - 14 + e) << 23));
}

// ---------------------------------------------------------------------------
// Phase 1: router logits, scaled fp16 copies of the tokens
// ---------------------------------------------------------------------------
template <typename T>
__device__ void router_phase(const MoeParams& p, int cta, int ctas) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const T* X = static_cast<const T*>(p.X);
  const T* WR = static_cast<const T*>(p.WR);
  for (int i = cta * kWarps + warp; i < p.T * (p.E + 1); i += ctas * kWarps) {
    const int t = i / (p.E + 1), e = i - t * (p.E + 1);
    const T* x = X + (long long)t * p.H;
    if (e < p.E) {
      const T* w = WR + (long long)e * p.H;
      float s = 0.0f;
      for (int k = lane * 8; k < p.H; k += 256) {  // H is a multiple of 16
        const uint4 a = __ldg(reinterpret_cast<const uint4*>(x + k)), b = __ldg(reinterpret_cast<const uint4*>(w + k));
        const T* av = reinterpret_cast<const T*>(&a);
        const T* bv = reinterpret_cast<const T*>(&b);
#pragma unroll
        for (int j = 0; j < 8; ++j) s = fmaf(to_f(av[j]), to_f(bv[j]), s);
      }
#pragma unroll
      for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
      if (lane == 0) p.w.logits[t * p.E + e] = s;
    } else {
      uint32_t m = 0;
      for (int k = lane; k < p.H; k += 32) m = max(m, __float_as_uint(to_f(x[k])) & 0x7FFFFFFFu);
      m = __reduce_max_sync(0xFFFFFFFFu, m);
      const float2 sc = pow2_scale(m);
      for (int k = lane; k < p.H; k += 32) p.w.xs[(long long)t * p.H + k] = __float2half_rn(to_f(x[k]) * sc.x);
      if (lane == 0) p.w.x_inv[t] = sc.y;
      for (int j = lane; j < p.top_k; j += 32) p.w.h_max[t * p.top_k + j] = 0;
    }
  }
}

// ---------------------------------------------------------------------------
// Top-k and the tokens' order by expert, formed by every CTA for itself
// ---------------------------------------------------------------------------
struct Routing {
  float gate[kSlots];            // by slot = token * top_k + j
  short expert[kSlots];
  short order[kSlots];           // slots, grouped by expert
  short start[kMaxE + 1];        // of each expert's group
  short active[kMaxE];           // experts with tokens
  short fill[kMaxE];
  int counts[kMaxE];
  int num_active;
};

// Order of floats as unsigned integers; NaN sorts by its bits (the softmax
// makes every weight of such a token NaN whichever experts it takes).
__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t b = __float_as_uint(v);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

__device__ void form_routing(const MoeParams& p, Routing& r) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int e = threadIdx.x; e < p.E; e += kThreads) {
    r.counts[e] = 0;
    r.fill[e] = 0;
  }
  __syncthreads();
  constexpr int PER = (kMaxE + 31) / 32;
  for (int t = warp; t < p.T; t += kWarps) {
    const float* lg = p.w.logits + t * p.E;
    float v[PER];
    float mx = -INFINITY;
    bool nan = false;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      v[i] = i * 32 + lane < p.E ? __ldcg(lg + i * 32 + lane) : -INFINITY;
      mx = fmaxf(mx, v[i]);
      nan |= v[i] != v[i];
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, o));
    nan = __any_sync(0xFFFFFFFFu, nan);
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < PER; ++i) sum += i * 32 + lane < p.E ? expf(v[i] - mx) : 0.0f;
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    uint32_t taken = 0;  // bit i: this lane's entry i is chosen
    float mine = 0.0f, total = 0.0f;
    int my_expert = 0;
    for (int j = 0; j < p.top_k; ++j) {
      uint32_t key = 0;
      int at = 0;
      bool any = false;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const uint32_t k = order_key(v[i] + 0.0f);  // -0 ties with +0
        if (i * 32 + lane < p.E && !(taken >> i & 1u) && (!any || k > key)) {
          key = k;
          at = i;
          any = true;
        }
      }
      // the largest key, then the lowest expert that has it
      const uint32_t best = __reduce_max_sync(0xFFFFFFFFu, any ? key : 0u);
      const uint32_t cand = any && key == best ? (uint32_t)(at * 32 + lane) : 0xFFFFFFFFu;
      const uint32_t e = __reduce_min_sync(0xFFFFFFFFu, cand);
      float pe = 0.0f;
      if (cand == e) {
        taken |= 1u << at;
#pragma unroll
        for (int i = 0; i < PER; ++i)
          if (i == at) pe = expf(v[i] - mx) / sum;
      }
      pe = __shfl_sync(0xFFFFFFFFu, pe, (int)(e & 31u));
      total += pe;
      if (lane == j) {
        mine = pe;
        my_expert = (int)e;
      }
    }
    if (lane < p.top_k) {
      float g = p.renorm ? mine / total : mine;
      if (nan) g = __int_as_float(0x7FC00000);
      const int slot = t * p.top_k + lane;
      r.gate[slot] = g;
      r.expert[slot] = (short)my_expert;
      atomicAdd(&r.counts[my_expert], 1);
    }
  }
  __syncthreads();
  if (warp == 0) {  // exclusive sums of the counts, and the experts that have any
    int base = 0, nact = 0;
    for (int e0 = 0; e0 < p.E; e0 += 32) {
      const int e = e0 + lane, c = e < p.E ? r.counts[e] : 0;
      int s = c;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xFFFFFFFFu, s, o);
        if (lane >= o) s += u;
      }
      const uint32_t has = __ballot_sync(0xFFFFFFFFu, c > 0);
      if (e < p.E) {
        r.start[e] = (short)(base + s - c);
        if (c > 0) r.active[nact + __popc(has & ((1u << lane) - 1u))] = (short)e;
      }
      base += __shfl_sync(0xFFFFFFFFu, s, 31);
      nact += __popc(has);
    }
    if (lane == 0) {
      r.start[p.E] = (short)base;
      r.num_active = nact;
    }
  }
  __syncthreads();
  // slots in their own order within each expert's group
  for (int e = threadIdx.x; e < p.E; e += kThreads) {
    if (r.counts[e] == 0) continue;
    int at = r.start[e];
    for (int s = 0; s < p.T * p.top_k; ++s)
      if (r.expert[s] == e) r.order[at++] = (short)s;
  }
  __syncthreads();
}

// ---------------------------------------------------------------------------
// The product core: 16 weight rows times up to 8 NT columns over the 128-blocks
// kb0, kb0 + step, ... of k.
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint32_t e4m3x2_to_h2(uint32_t two) {  // the low 16 bits: two E4M3 values
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)two));
  return h;
}
__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Columns (tokens) of the second operand, 16 consecutive k at a time, as eight
// fp16 pairs.
struct HalfColumns {  // fp16 rows
  const __half* base[8];
  __device__ __forceinline__ void load(int nt, int k, bool live, uint32_t (&b)[8]) const {
    uint4 u = make_uint4(0, 0, 0, 0), v = u;
    if (live) {
      u = __ldcg(reinterpret_cast<const uint4*>(base[nt] + k));
      v = __ldcg(reinterpret_cast<const uint4*>(base[nt] + k) + 1);
    }
    b[0] = u.x; b[1] = u.y; b[2] = u.z; b[3] = u.w;
    b[4] = v.x; b[5] = v.y; b[6] = v.z; b[7] = v.w;
  }
};
struct FloatColumns {  // fp32 rows, scaled and rounded to fp16 here
  const float* base[8];
  float scale[8];
  __device__ __forceinline__ void load(int nt, int k, bool live, uint32_t (&b)[8]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
      if (live) f = __ldcg(reinterpret_cast<const float4*>(base[nt] + k) + i);
      const __half2 lo = __floats2half2_rn(f.x * scale[nt], f.y * scale[nt]);
      const __half2 hi = __floats2half2_rn(f.z * scale[nt], f.w * scale[nt]);
      b[2 * i] = *reinterpret_cast<const uint32_t*>(&lo);
      b[2 * i + 1] = *reinterpret_cast<const uint32_t*>(&hi);
    }
  }
};

// row_lo / row_hi: this lane's two weight rows (null: zeros), K long (a multiple
// of 16); s_lo / s_hi: their scales along k.
template <int NT, typename Cols>
__device__ __forceinline__ void rows_product(const uint8_t* row_lo, const uint8_t* row_hi, const float* s_lo,
                                             const float* s_hi, int K, int kb0, int step, const Cols& cols,
                                             float (&tot)[NT][4]) {
  const int t4 = threadIdx.x & 3;
  const int nkb = (K + 127) / 128;
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i) tot[n][i] = 0.0f;
  for (int kb = kb0; kb < nkb; kb += step) {
    float acc[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[n][i] = 0.0f;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int k = kb * 128 + half * 64 + t4 * 16;
      const bool live = k < K;
      uint4 lo = make_uint4(0, 0, 0, 0), hi = lo;
      if (live && row_lo) lo = __ldg(reinterpret_cast<const uint4*>(row_lo + k));
      if (live && row_hi) hi = __ldg(reinterpret_cast<const uint4*>(row_hi + k));
      const uint32_t wl[4] = {lo.x, lo.y, lo.z, lo.w}, wh[4] = {hi.x, hi.y, hi.z, hi.w};
      uint32_t a[4][4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        a[j][0] = e4m3x2_to_h2(wl[j]);
        a[j][1] = e4m3x2_to_h2(wh[j]);
        a[j][2] = e4m3x2_to_h2(wl[j] >> 16);
        a[j][3] = e4m3x2_to_h2(wh[j] >> 16);
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        uint32_t b[8];
        cols.load(n, k, live, b);
#pragma unroll
        for (int j = 0; j < 4; ++j) mma_f16(acc[n], a[j], b[2 * j], b[2 * j + 1]);
      }
    }
    const float s0 = __ldg(s_lo + kb), s1 = __ldg(s_hi + kb);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      tot[n][0] = fmaf(acc[n][0], s0, tot[n][0]);
      tot[n][1] = fmaf(acc[n][1], s0, tot[n][1]);
      tot[n][2] = fmaf(acc[n][2], s1, tot[n][2]);
      tot[n][3] = fmaf(acc[n][3], s1, tot[n][3]);
    }
  }
}

constexpr int kRedLd = 8 * 8 + 4;  // columns of a warp's partial sums, padded
struct Smem {
  Routing r;
  float red[kWarps][16][kRedLd];
};

// ---------------------------------------------------------------------------
// Phase 2: h = silu(x G^T) * (x U^T), eight columns of h per unit (their eight
// gate rows and eight up rows are one 16-row operand); warps split k.
// ---------------------------------------------------------------------------
template <int NT>
__device__ void up_unit(const MoeParams& p, Smem& sm, int e, int r0, int first, int n_tok) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
  const Routing& r = sm.r;
  HalfColumns cols;
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int c = min(n * 8 + g, n_tok - 1);  // columns past the last repeat it and are not stored
    cols.base[n] = p.w.xs + (long long)(r.order[first + c] / p.top_k) * p.H;
  }
  const int hb = (p.H + 127) / 128, ib = (2 * p.I + 127) / 128;
  const uint8_t* W = p.W13 + (long long)e * 2 * p.I * p.H;
  const float* S = p.S13 + (long long)e * ib * hb;
  const int row = r0 + g;
  float tot[NT][4];
  rows_product<NT>(W + (long long)row * p.H, W + (long long)(p.I + row) * p.H, S + (long long)(row / 128) * hb,
                   S + (long long)((p.I + row) / 128) * hb, p.H, warp, kWarps, cols, tot);
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    *reinterpret_cast<float2*>(&sm.red[warp][g][n * 8 + 2 * t4]) = make_float2(tot[n][0], tot[n][1]);
    *reinterpret_cast<float2*>(&sm.red[warp][g + 8][n * 8 + 2 * t4]) = make_float2(tot[n][2], tot[n][3]);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 8 * n_tok; i += kThreads) {
    const int c = i >> 3, rr = i & 7;
    float a = 0.0f, u = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      a += sm.red[w][rr][c];
      u += sm.red[w][rr + 8][c];
    }
    const int slot = r.order[first + c];
    const float inv = p.w.x_inv[slot / p.top_k];
    a *= inv;
    u *= inv;
    const float h = a / (1.0f + expf(-a)) * u;
    p.w.h[(long long)slot * p.I + r0 + rr] = h;
    atomicMax(&p.w.h_max[slot], __float_as_uint(h) & 0x7FFFFFFFu);  // a maximum: the order does not matter
  }
  __syncthreads();
}

// ---------------------------------------------------------------------------
// Phase 3: an expert's output for its tokens, 16 rows of D per unit.
// ---------------------------------------------------------------------------
template <int NT>
__device__ void down_unit(const MoeParams& p, Smem& sm, int e, int r0, int first, int n_tok) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
  const Routing& r = sm.r;
  FloatColumns cols;
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int slot = r.order[first + min(n * 8 + g, n_tok - 1)];
    cols.base[n] = p.w.h + (long long)slot * p.I;
    cols.scale[n] = pow2_scale(__ldcg(&p.w.h_max[slot])).x;
  }
  const int hb = (p.H + 127) / 128, ib = (p.I + 127) / 128;
  const uint8_t* W = p.W2 + (long long)e * p.H * p.I + (long long)(r0 + g) * p.I;
  const float* S = p.S2 + ((long long)e * hb + r0 / 128) * ib;
  float tot[NT][4];
  rows_product<NT>(W, W + 8LL * p.I, S, S, p.I, warp, kWarps, cols, tot);
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    *reinterpret_cast<float2*>(&sm.red[warp][g][n * 8 + 2 * t4]) = make_float2(tot[n][0], tot[n][1]);
    *reinterpret_cast<float2*>(&sm.red[warp][g + 8][n * 8 + 2 * t4]) = make_float2(tot[n][2], tot[n][3]);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 16 * n_tok; i += kThreads) {
    const int c = i >> 4, rr = i & 15;
    float y = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) y += sm.red[w][rr][c];
    const int slot = r.order[first + c];
    p.w.part[(long long)slot * p.H + r0 + rr] = y * pow2_scale(__ldcg(&p.w.h_max[slot])).y;
  }
  __syncthreads();
}

template <bool UP>
__device__ void expert_phase(const MoeParams& p, Smem& sm, int cta, int ctas) {
  const int groups = UP ? p.I / 8 : p.H / 16;
  const int units = sm.r.num_active * groups;
  for (int u = cta; u < units; u += ctas) {
    const int a = u / groups, e = sm.r.active[a], r0 = (u - a * groups) * (UP ? 8 : 16);
    const int first = sm.r.start[e], n = sm.r.counts[e];
#define RG_MOE_UNIT(NT) (UP ? up_unit<NT>(p, sm, e, r0, first, n) : down_unit<NT>(p, sm, e, r0, first, n))
    if (n <= 8) RG_MOE_UNIT(1);
    else if (n <= 16) RG_MOE_UNIT(2);
    else if (n <= 32) RG_MOE_UNIT(4);
    else RG_MOE_UNIT(8);
#undef RG_MOE_UNIT
  }
}

// Phase 4: the weighted sum of each token's experts, in the order of their ranks.
template <typename T>
__device__ void combine_phase(const MoeParams& p, const Routing& r, int cta, int ctas) {
  T* Y = static_cast<T*>(p.Y);
  for (long long i = (long long)cta * kThreads + threadIdx.x; i < (long long)p.T * p.H; i += (long long)ctas * kThreads) {
    const int t = (int)(i / p.H), c = (int)(i - (long long)t * p.H);
    float y = 0.0f;
    for (int j = 0; j < p.top_k; ++j) {
      const int slot = t * p.top_k + j;
      y = fmaf(r.gate[slot], __ldcg(&p.w.part[(long long)slot * p.H + c]), y);
    }
    T o;
    from_f(y, o);
    Y[i] = o;
  }
}

__global__ void __launch_bounds__(kThreads) moe_phase_kernel(MoeParams p, int phase) {
  extern __shared__ __align__(16) uint8_t raw[];
  Smem& sm = *reinterpret_cast<Smem*>(raw);
  if (phase == 0) {
    if (p.type == RG_TYPE_F16) router_phase<__half>(p, blockIdx.x, gridDim.x);
    else router_phase<__nv_bfloat16>(p, blockIdx.x, gridDim.x);
    return;
  }
  form_routing(p, sm.r);
  if (phase == 1) expert_phase<true>(p, sm, blockIdx.x, gridDim.x);
  else if (phase == 2) expert_phase<false>(p, sm, blockIdx.x, gridDim.x);
  else if (p.type == RG_TYPE_F16) combine_phase<__half>(p, sm.r, blockIdx.x, gridDim.x);
  else combine_phase<__nv_bfloat16>(p, sm.r, blockIdx.x, gridDim.x);
}

size_t up256(size_t x) { return (x + 255) & ~size_t(255); }

// Workspace after the call block; base may be null (sizes only).
size_t layout(long long T, long long H, long long I, long long E, long long top_k, uint8_t* base, MoeWs* w) {
  size_t off = 0;
  auto take = [&](size_t bytes) {
    uint8_t* q = base ? base + off : nullptr;
    off = up256(off + bytes);
    return q;
  };
  const size_t slots = (size_t)(T * top_k);
  MoeWs m;
  m.logits = reinterpret_cast<float*>(take((size_t)T * E * 4));
  m.xs = reinterpret_cast<__half*>(take((size_t)T * H * 2));
  m.x_inv = reinterpret_cast<float*>(take((size_t)T * 4));
  m.h = reinterpret_cast<float*>(take(slots * I * 4));
  m.h_max = reinterpret_cast<uint32_t*>(take(slots * 4));
  m.part = reinterpret_cast<float*>(take(slots * H * 4));
  if (w) *w = m;
  return off;
}

}  // namespace

size_t moe_f8_scratch_bytes(long long T, long long H, long long I, long long E, long long top_k) {
  return layout(T, H, I, E, top_k, nullptr, nullptr);
}

cudaError_t launch_moe_f8(const MoeArgs& a, void* scratch, cudaStream_t st) {
  MoeParams p{a.X, a.WR, a.W13, a.S13, a.W2, a.S2, a.Y, (int)a.T, (int)a.H, (int)a.I, (int)a.E, (int)a.top_k, a.type,
              a.renorm ? 1 : 0, {}};
  layout(a.T, a.H, a.I, a.E, a.top_k, static_cast<uint8_t*>(scratch), &p.w);
  static std::once_flag once;
  static cudaError_t attr = cudaSuccess;
  std::call_once(once, [] {
    attr = cudaFuncSetAttribute(moe_phase_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(Smem));
  });
  if (attr != cudaSuccess) return attr;
  const int grid = 304;
  for (int phase = 0; phase < 4; ++phase) {
    moe_phase_kernel<<<grid, kThreads, sizeof(Smem), st>>>(p, phase);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace rg
