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
// [2^14, 2^15)): exact for bf16 and fp16 entries within 2^-28 of the row's
// largest, off by at most 2^-39 of it below.  The gated product h is kept in
// fp32 and enters the second product, scaled the same way, as the sum of two
// fp16 terms: h to 11 bits and what that leaves out.  Together they are within
// 2^-23 of the entry or 2^-39 of the row's largest, as fp32 is, for twice that
// product's MMAs (with the first term alone, 11 bits, 64 tokens took 311 us
// instead of 317 and one token 28.7 instead of 30.1).  Each 128-block's sum is
// scaled in fp32 and added to fp32 sums.
//
// 64 tokens through 128 experts of 4096 x 1024 (top 8): 300 to 308 us, the weights
// at the copy rate 237; the two products stream at 6.3 TB/s, and the grid's
// meetings wait for the slowest SM, 10% behind the median.  One token through 8 of
// 64 experts of 2048 x 1024: 30 us (7.6): router 4, routing 1.4, first product 9,
// second 5, two meetings of the grid 4 and 1.4, sum 1, launches.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <cmath>
#include <cstdint>
#include <mutex>

#include "f8_kernels.h"

namespace rg {
namespace {

constexpr int kWarps = 16;
constexpr int kThreads = 32 * kWarps;
constexpr int kRouterWarps = 16;
constexpr int kRouterThreads = 32 * kRouterWarps;
constexpr int kMaxT = RG_MOE_MAX_TOKENS;
constexpr int kMaxK = RG_MOE_MAX_TOP_K;
constexpr int kMaxE = RG_MOE_MAX_EXPERTS;
constexpr int kSlots = kMaxT * kMaxK;
// column tiles of eight tokens per pass over the weights (a kernel with four
// spills registers: 64 tokens in 300 against 290 us, and no faster where experts
// get more than 16 tokens)
constexpr int kMaxNT = 2;
constexpr int kMinRing = 3, kMaxRing = 8;  // weight pieces (16 rows x 128 k) per warp, on their way or in use
constexpr int kTightRing = 2;              // where one token's operands leave no room for kMinRing
constexpr int kPiece = 16 * 128 + 16;      // and the two scales of its rows
constexpr int kMaxStride = 32;             // words between two slots' maxima
constexpr int kSmemBytes = 231424;         // all of an SM's

struct MoeWs {
  float* gate;       // [T * top_k] weights, and
  int* expert;       // experts, by slot = token * top_k + rank
  float* h;          // [T * top_k][I]
  uint32_t* h_max;   // [T * top_k][kMaxStride] largest |h|, as bits, in the first word
  unsigned* arrived;  // CTAs that have reached the grid's barriers
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
  int ks_up, ks_down;    // warps that split k in the two products
  int cap_up, cap_down;  // tokens per pass
  int ring;              // pieces per warp
  int red_ld;            // columns of the warps' partial sums, padded
  int together;          // segments are staged together
  int red_off, cols_off, ring_off;  // shared memory beyond struct Smem
  unsigned long long wait_ns;
  DevPlan* plan;
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
// and its inverse.  A row with an inf or NaN is scaled as if its largest were
// finite, so that its other entries stay finite in fp16; a row of zeros is left
// alone; the exponent is bounded so that both stay normal.
__device__ __forceinline__ float2 pow2_scale(uint32_t max_bits) {
  if (max_bits == 0) return make_float2(1.0f, 1.0f);
  const int e = min(max((int)(max_bits >> 23) - 127, -110), 127);
  return make_float2(__int_as_float((127 + 14 - e) << 23), __int_as_float((127 - 14 + e) << 23));
}

// ---------------------------------------------------------------------------
// Kernel 1: the router.  A cluster of eight CTAs takes eight tokens: its CTAs
// form the logits of a share of the experts each (tiles of 8 or 16 experts x 8
// tokens, a CTA's warps splitting k; the products of 16-bit entries are exact in
// the MMA's fp32), then one token's top-k each, reading the logits from each
// other's shared memory.  It also clears the words that kernel 2 starts from.
// ---------------------------------------------------------------------------
template <typename T>
__device__ __forceinline__ void mma_t(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                      uint32_t b1);
template <>
__device__ __forceinline__ void mma_t<__half>(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma_t<__nv_bfloat16>(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                                     uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Order of floats as unsigned integers; NaN sorts by its bits (the softmax
// makes every weight of such a token NaN whichever experts it takes).
__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t b = __float_as_uint(v);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// Softmax and top-k of one token by a warp; logit(e) gives its logits.
template <int PER, typename F>  // E <= 32 PER
__device__ __forceinline__ void choose(const MoeParams& p, int t, F&& logit) {
  const int lane = threadIdx.x & 31;
  float v[PER];
  float mx = -INFINITY;
  bool nan = false;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    v[i] = i * 32 + lane < p.E ? logit(i * 32 + lane) : -INFINITY;
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
  float mine = 0.0f;   // lane j: the logit and the expert of rank j
  int my_expert = 0;
  for (int j = 0; j < p.top_k; ++j) {
    uint32_t key = 0;
    float best_v = 0.0f;
    int at = 0;
    bool any = false;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const uint32_t k = order_key(v[i] + 0.0f);  // -0 ties with +0
      if (i * 32 + lane < p.E && !(taken >> i & 1u) && (!any || k > key)) {
        key = k;
        best_v = v[i];
        at = i;
        any = true;
      }
    }
    // the largest key, then the lowest expert that has it
    const uint32_t best = __reduce_max_sync(0xFFFFFFFFu, any ? key : 0u);
    const uint32_t cand = any && key == best ? (uint32_t)(at * 32 + lane) : 0xFFFFFFFFu;
    const uint32_t e = __reduce_min_sync(0xFFFFFFFFu, cand);
    if (cand == e) taken |= 1u << at;
    best_v = __shfl_sync(0xFFFFFFFFu, best_v, (int)(e & 31u));
    if (lane == j) {
      mine = best_v;
      my_expert = (int)e;
    }
  }
  const float prob = lane < p.top_k ? expf(mine - mx) / sum : 0.0f;
  float total = prob;
#pragma unroll
  for (int o = 16; o; o >>= 1) total += __shfl_xor_sync(0xFFFFFFFFu, total, o);
  if (lane < p.top_k) {
    const float w = p.renorm ? prob / total : prob;
    p.w.gate[t * p.top_k + lane] = nan ? __int_as_float(0x7FC00000) : w;
    p.w.expert[t * p.top_k + lane] = my_expert;
    p.w.h_max[(t * p.top_k + lane) * kMaxStride] = 0;
  }
}

template <typename T>
__global__ void __cluster_dims__(8, 1, 1) __launch_bounds__(kRouterThreads) moe_router_kernel(MoeParams p) {
  __shared__ float red[kRouterWarps][16][8];
  __shared__ float logits[8][kMaxE / 8];  // [token][16-expert (8-expert) tiles of this CTA]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
  const T* X = static_cast<const T*>(p.X);
  const T* WR = static_cast<const T*>(p.WR);
  const int rank = (int)(blockIdx.x & 7u), t0 = (int)(blockIdx.x >> 3) * 8;
  wait_for_predecessor();
  allow_dependents();
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    p.plan->status = 0;
    p.plan->timeout_where = 0;
    *p.w.arrived = 0;
  }
  // logits of this CTA's tiles; rows past the last repeat it, and nothing reads their results
  const int rows = p.E > 64 ? 16 : 8;  // experts per tile: all eight CTAs busy from 57 experts on
  const T* xb = X + (long long)min(t0 + g, p.T - 1) * p.H;
  for (int tile = rank, local = 0; tile * rows < p.E; tile += 8, ++local) {
    const T* wa = WR + (long long)min(tile * rows + g, p.E - 1) * p.H;
    const T* wb = WR + (long long)min(tile * rows + g + 8, p.E - 1) * p.H;
    float c[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
    for (int k = warp * 32 + t4 * 8; k - t4 * 8 < p.H; k += kRouterWarps * 32) {  // H is a multiple of 16
      uint4 a = make_uint4(0, 0, 0, 0), b = a, x = a;
      if (k < p.H) {
        a = __ldg(reinterpret_cast<const uint4*>(wa + k));
        if (rows == 16) b = __ldg(reinterpret_cast<const uint4*>(wb + k));
        x = __ldg(reinterpret_cast<const uint4*>(xb + k));
      }
      mma_t<T>(c, a.x, b.x, a.y, b.y, x.x, x.y);
      mma_t<T>(c, a.z, b.z, a.w, b.w, x.z, x.w);
    }
    red[warp][g][2 * t4] = c[0];
    red[warp][g][2 * t4 + 1] = c[1];
    red[warp][g + 8][2 * t4] = c[2];
    red[warp][g + 8][2 * t4 + 1] = c[3];
    __syncthreads();
    if ((int)threadIdx.x < 8 * rows) {
      const int e = threadIdx.x % rows, t = threadIdx.x / rows;
      float s = 0.0f;
#pragma unroll
      for (int w = 0; w < kRouterWarps; ++w) s += red[w][e][t];
      logits[t][local * rows + e] = s;
    }
    __syncthreads();
  }
  const int t = t0 + rank;  // this CTA's token
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
  if (t < p.T && warp == 0) {
    auto logit = [&](int e) {
      const int tile = e / rows;
      const uint32_t at = (uint32_t)__cvta_generic_to_shared(&logits[rank][(tile >> 3) * rows + e % rows]);
      uint32_t remote;
      float v;
      asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(at), "r"(tile & 7));
      asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(remote));
      return v;
    };
    if (p.E <= 128) choose<4>(p, t, logit);
    else choose<kMaxE / 32>(p, t, logit);
  }
  __syncwarp();  // the barrier below is for whole warps
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// ---------------------------------------------------------------------------
// Kernel 2.  The tokens' order by expert, formed by every CTA for itself.
// ---------------------------------------------------------------------------
struct Routing {
  short expert[kSlots];          // by slot = token * top_k + rank
  short order[kSlots];           // slots, grouped by expert
  short start[kMaxE + 1];        // of each expert's group
  short active[kMaxE];           // experts with tokens
  short fill[kMaxE];
  int counts[kMaxE];
  int units[kMaxE + 1];          // of a product phase: first unit of each active expert
  int num_active;
  int first_active;              // of a product phase: the active expert of this CTA's first unit
  int go;                        // the grid's barrier was passed
};

__device__ void form_routing(const MoeParams& p, Routing& r) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int e = threadIdx.x; e < p.E; e += kThreads) {
    r.counts[e] = 0;
    r.fill[e] = 0;
  }
  __syncthreads();
  for (int s = threadIdx.x; s < p.T * p.top_k; s += kThreads) {
    const int e = __ldg(p.w.expert + s);
    r.expert[s] = (short)e;
    atomicAdd(&r.counts[e], 1);
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
    __syncwarp();
    // Slots in their own order within each expert's group, 32 at a time.  The
    // order has to be the same in every CTA: passes over an expert take tokens by it.
    for (int s0 = 0; s0 < p.T * p.top_k; s0 += 32) {
      const int s = s0 + lane;
      const bool live = s < p.T * p.top_k;
      const int e = live ? r.expert[s] : -1;
      const uint32_t same = __match_any_sync(0xFFFFFFFFu, e);
      const int before = __popc(same & ((1u << lane) - 1u));
      const int at = live ? r.start[e] + r.fill[e] : 0;
      __syncwarp();
      if (live) {
        r.order[at + before] = (short)s;
        if (before == 0) r.fill[e] += (short)__popc(same);
      }
      __syncwarp();
    }
  }
  __syncthreads();
}

// All CTAs of the (cooperative) grid, bounded in time.
__device__ bool grid_barrier(const MoeParams& p, Routing& r, unsigned target) {
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    atomicAdd(p.w.arrived, 1u);
    unsigned long long t0 = 0;
    int ok = 1;
    for (uint32_t i = 1;; ++i) {
      unsigned n;
      asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(n) : "l"(p.w.arrived) : "memory");
      if (n >= target) break;
      if ((i & 63u) == 0) {
        unsigned long long now;
        asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(now));
        if (!t0) t0 = now;
        if (now - t0 > p.wait_ns) {
          ok = 0;
          atomicCAS(&p.plan->status, 0, RG_ERR_TIMEOUT);
          atomicCAS(&p.plan->timeout_where, 0, 41);
          break;
        }
      }
    }
    r.go = ok;
  }
  __syncthreads();
  return r.go != 0;
}

// ---------------------------------------------------------------------------
// The products.  A unit is 16 weight rows times the (up to cap) tokens of one
// pass over an expert.  A group of ks warps works on a unit, each on every ks-th
// 128-block of k, and the groups of all CTAs share the units out evenly, in
// contiguous ranges per CTA, so that a CTA stages an expert's tokens in shared
// memory once.  Every warp copies the weights it will use itself, ring - 1
// pieces ahead of their use and across units (cp.async, 2 KB a piece and warp: at
// least 64 KB on their way per SM, where the latency times the bandwidth of
// this memory needs about 45).
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint32_t e4m3x2_to_h2(uint32_t two) {  // the low 16 bits: two E4M3 values
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)two));
  return h;
}
__device__ __forceinline__ uint32_t su32(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool live) {
  const int n = live ? 16 : 0;  // zeros where there is nothing to read
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}

// The units of one pass over one expert, as far as they are this CTA's.
struct Segment {
  int base, end;  // unit of row block 0, and the one after the segment's last
  int first, n;   // tokens of the order,
  int c0;         // staged in columns c0 onwards
};
// Shared memory: this, then the warps' partial sums, the staged tokens and the
// rings of weight pieces, laid out by the host for the call's shape.
struct Smem {
  Routing r;
  float col_scale[8 * kMaxNT];   // of the staged columns: takes a sum back from the operand's power of two
  Segment segs[8 * kMaxNT];      // the staged segments
  short slot[8 * kMaxNT];        // the slots of the staged columns
};
constexpr int kFixedBytes = ((int)sizeof(Smem) + 127) / 128 * 128;
// the widest layer: two pieces per warp, one column tile, one token of two terms
static_assert(kFixedBytes + kWarps * 16 * 20 * 4 + kWarps * kTightRing * kPiece + (RG_MOE_MAX_WIDTH / 128) * 512 + 16 <=
                  kSmemBytes,
              "shared memory");
// Bytes of a staged token of K entries, one fp16 term or two: a multiple of 128
// and 16, so that the lanes' loads of eight tokens do not conflict.
__host__ __device__ constexpr int token_bytes(int K, bool two_terms) {
  return (K + 127) / 128 * (two_terms ? 512 : 256) + 16;
}

template <bool UP>
struct Phase {
  const MoeParams& p;
  Smem& sm;
  const int warp, lane, g, t4;
  const int K, nkb, ks, groups, group, kpart, rows_per_expert;
  int u0, u1;            // this CTA's units
  // the next piece to copy
  int pu, pkb, pa, prb;  // unit, 128-block, active expert, its row block
  const uint8_t* p_lo;
  const uint8_t* p_hi;
  const float* p_s;      // the even lanes' (gate, or all) or the odd lanes' (up) row scales
  uint8_t* const cols;   // staged tokens
  float* const red;      // [warps][16][red_ld]
  const uint32_t ring;   // this warp's pieces
  int slot;              // the next piece to use
  int parity;            // half of the reduction buffer

  __device__ Phase(const MoeParams& pp, Smem& s, uint8_t* base)
      : p(pp), sm(s), warp(threadIdx.x >> 5), lane(threadIdx.x & 31), g((threadIdx.x & 31) >> 2),
        t4(threadIdx.x & 3), K(UP ? pp.H : pp.I), nkb((K + 127) / 128), ks(UP ? pp.ks_up : pp.ks_down),
        groups(kWarps / ks), group((threadIdx.x >> 5) / ks), kpart((threadIdx.x >> 5) % ks),
        rows_per_expert(UP ? pp.I / 8 : pp.H / 16),
        cols(base + pp.cols_off), red(reinterpret_cast<float*>(base + pp.red_off)),
        ring(su32(base + pp.ring_off) + (threadIdx.x >> 5) * pp.ring * kPiece), slot(0), parity(0) {}

  __device__ int cap() const { return UP ? p.cap_up : p.cap_down; }

  // Units of the active experts, and this CTA's range of them.
  __device__ void plan_units(int cta, int ctas) {
    Routing& r = sm.r;
    __syncthreads();
    if (warp == 0) {
      int base = 0;
      for (int a0 = 0; a0 < r.num_active; a0 += 32) {
        const int a = a0 + lane;
        const int n = a < r.num_active ? (r.counts[r.active[a]] + cap() - 1) / cap() * rows_per_expert : 0;
        int s = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int v = __shfl_up_sync(0xFFFFFFFFu, s, o);
          if (lane >= o) s += v;
        }
        if (a < r.num_active) r.units[a] = base + s - n;
        base += __shfl_sync(0xFFFFFFFFu, s, 31);
      }
      if (lane == 0) r.units[r.num_active] = base;
    }
    __syncthreads();
    const long long total = r.units[r.num_active];
    u0 = (int)(total * cta / ctas);
    u1 = (int)(total * (cta + 1) / ctas);
    for (int a = threadIdx.x; a < r.num_active; a += kThreads)
      if (r.units[a] <= u0 && u0 < r.units[a + 1]) r.first_active = a;
    __syncthreads();
    pu = u0 + group;
    pkb = kpart;
    pa = u0 < u1 ? r.first_active : 0;
    if (pu < u1) point_expert();
  }

  // The expert of unit pu: its weights and scales, and pu's row block.
  __device__ __forceinline__ void point_expert() {
    const Routing& r = sm.r;
    while (pu >= r.units[pa + 1]) ++pa;
    prb = (pu - r.units[pa]) % rows_per_expert;
    point();
  }
  // Row block prb's weights and scales.  A lane copies 16 bytes of rows lane / 8 +
  // 4 j of the 16 (whole 128-byte lines per eight lanes); the even lanes' scales
  // are the gate's (or all rows'), the odd lanes' the up rows'.
  __device__ __forceinline__ void point() {
    const long long e = sm.r.active[pa];
    if constexpr (UP) {  // eight gate rows, eight up rows
      p_lo = p.W13 + (e * 2 * p.I + (lane >> 3) + prb * 8) * K;
      p_hi = p_lo + (long long)p.I * K;
      p_s = p.S13 + (e * ((2 * p.I + 127) / 128) + (((lane & 1) * p.I + prb * 8) >> 7)) * nkb;
    } else {
      p_lo = p.W2 + (e * p.H + (lane >> 3) + prb * 16) * K;
      p_hi = p_lo + 8LL * K;
      p_s = p.S2 + (e * ((p.H + 127) / 128) + (prb >> 3)) * nkb;
    }
  }
  __device__ __forceinline__ void next_unit() {
    pu += groups;
    if (pu >= u1) return;
    if (pu >= sm.r.units[pa + 1]) {
      point_expert();
    } else {
      prb += groups;
      while (prb >= rows_per_expert) prb -= rows_per_expert;  // the next pass over the same expert
      point();
    }
  }

  // Starts the copy of the next piece into ring slot s (an empty group at the
  // end).  Row r's 16-byte chunk c lies at r * 128 + (c ^ 4 (r & 1)) * 16, which
  // the MMA lanes read without bank conflicts.
  __device__ __forceinline__ void copy_next(int s) {
    if (pu < u1) {
      const uint32_t at = ring + s * kPiece;
      const int c = lane & 7, k = pkb * 128 + c * 16;
      const bool live = k < K;
      const uint32_t dst = at + (lane >> 3) * 128 + ((c ^ ((lane >> 3) & 1) << 2) << 4);
      const long long down4 = 4LL * K;
      const uint8_t* lo = live ? p_lo + k : p_lo;
      const uint8_t* hi = live ? p_hi + k : p_hi;
      copy16(dst, lo, live);
      copy16(dst + 4 * 128, lo + down4, live);
      copy16(dst + 8 * 128, hi, live);
      copy16(dst + 12 * 128, hi + down4, live);
      if (lane < 2) copy4(at + 16 * 128 + lane * 4, p_s + pkb);
      pkb += ks;
      if (pkb >= nkb) {
        pkb = kpart;
        next_unit();
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  }

  // All but the newest ring - 2 copies of this lane have landed.
  __device__ __forceinline__ void wait_oldest() {
    switch (p.ring) {
      case 2: asm volatile("cp.async.wait_group 0;" ::: "memory"); break;
      case 3: asm volatile("cp.async.wait_group 1;" ::: "memory"); break;
      case 4: asm volatile("cp.async.wait_group 2;" ::: "memory"); break;
      case 5: asm volatile("cp.async.wait_group 3;" ::: "memory"); break;
      case 6: asm volatile("cp.async.wait_group 4;" ::: "memory"); break;
      case 7: asm volatile("cp.async.wait_group 5;" ::: "memory"); break;
      default: asm volatile("cp.async.wait_group 6;" ::: "memory"); break;
    }
  }

  __device__ int stride() const { return token_bytes(K, !UP); }

  // The operands of the staged columns' slots: fp16 scaled by the power of two that
  // col_scale undoes, zeros past K; in the second product each 128-block's first
  // terms, then its second ones.  A warp makes a token's row; in the second product,
  // which need not find its largest entry first, all warps share the rows.
  __device__ void stage(int used) {
    static_assert(kWarps == 16 && 8 * kMaxNT <= kWarps, "a column to a warp at least");
    const int sh = UP || used > 8 ? 0 : used > 4 ? 1 : used > 2 ? 2 : used > 1 ? 3 : 4;
    const int c = warp >> sh;
    if (c < used) {
      const int s = sm.slot[c];
      uint8_t* out = cols + c * stride();
      if constexpr (UP) {
        const long long at = (long long)(s / p.top_k) * K;
        if (p.type == RG_TYPE_F16) stage_token(static_cast<const __half*>(p.X) + at, out, c);
        else stage_token(static_cast<const __nv_bfloat16*>(p.X) + at, out, c);
      } else {
        const float* h = p.w.h + (long long)s * K;
        const float2 sc = pow2_scale(__ldcg(&p.w.h_max[s * kMaxStride]));
        if (lane == 0) sm.col_scale[c] = sc.y;
#pragma unroll 4
        for (int k = (warp & ((1 << sh) - 1)) * 256 + lane * 8; k < nkb * 128; k += 256 << sh) {
          float4 a = make_float4(0.f, 0.f, 0.f, 0.f), b = a;
          if (k < K) {
            a = __ldcg(reinterpret_cast<const float4*>(h + k));
            b = __ldcg(reinterpret_cast<const float4*>(h + k) + 1);
          }
          const uint2 t[4] = {half_terms(a.x, a.y, sc.x), half_terms(a.z, a.w, sc.x), half_terms(b.x, b.y, sc.x),
                              half_terms(b.z, b.w, sc.x)};
          uint4* to = reinterpret_cast<uint4*>(out + (k & ~127) * 4 + (k & 127) * 2);
          to[0] = make_uint4(t[0].x, t[1].x, t[2].x, t[3].x);
          to[16] = make_uint4(t[0].y, t[1].y, t[2].y, t[3].y);
        }
      }
    }
  }
  static __device__ __forceinline__ uint32_t half_pair(float a, float b, float scale) {
    const __half2 h = __floats2half2_rn(a * scale, b * scale);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  // Both terms of two entries.  The difference is exact in fp32; an inf or NaN has
  // its first term alone.
  static __device__ __forceinline__ uint2 half_terms(float a, float b, float scale) {
    const float x = a * scale, y = b * scale;
    const __half2 h = __floats2half2_rn(x, y);
    const float2 f = __half22float2(h);
    const __half2 l = __floats2half2_rn(fabsf(f.x) <= 65504.0f ? x - f.x : 0.0f, fabsf(f.y) <= 65504.0f ? y - f.y : 0.0f);
    return make_uint2(*reinterpret_cast<const uint32_t*>(&h), *reinterpret_cast<const uint32_t*>(&l));
  }
  template <typename T>
  __device__ __forceinline__ void stage_token(const T* x, uint8_t* out, int c) {
    uint32_t m = 0;
#pragma unroll 8
    for (int k = lane * 8; k < K; k += 256) {  // K is a multiple of 16
      const uint4 a = __ldg(reinterpret_cast<const uint4*>(x + k));
      const T* v = reinterpret_cast<const T*>(&a);
#pragma unroll
      for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(to_f(v[j])) & 0x7FFFFFFFu);
    }
    const float2 sc = pow2_scale(__reduce_max_sync(0xFFFFFFFFu, m));
    if (lane == 0) sm.col_scale[c] = sc.y;
#pragma unroll 4
    for (int k = lane * 8; k < nkb * 128; k += 256) {  // the row again, now from near
      uint4 a = make_uint4(0, 0, 0, 0);
      if (k < K) a = __ldg(reinterpret_cast<const uint4*>(x + k));
      const T* v = reinterpret_cast<const T*>(&a);
      *reinterpret_cast<uint4*>(out + k * 2) =
          make_uint4(half_pair(to_f(v[0]), to_f(v[1]), sc.x), half_pair(to_f(v[2]), to_f(v[3]), sc.x),
                     half_pair(to_f(v[4]), to_f(v[5]), sc.x), half_pair(to_f(v[6]), to_f(v[7]), sc.x));
    }
  }

  // Token first + c's sums (staged column c0 + c) of row pair `row` of row block rb,
  // by whole warps; the lanes that differ in the bits of `lanes` hold the rows of
  // one token.
  __device__ __forceinline__ void store(int rb, int row, int first, int c0, int c, bool live, float lo, float hi,
                                        int lanes) {
    const int s = live ? sm.r.order[first + c] : 0;
    if constexpr (UP) {
      uint32_t m = 0;
      if (live) {
        const float a = lo * sm.col_scale[c0 + c], u = hi * sm.col_scale[c0 + c];
        const float h = a / (1.0f + expf(-a)) * u;
        p.w.h[(long long)s * p.I + rb * 8 + row] = h;
        m = __float_as_uint(h) & 0x7FFFFFFFu;
      }
      // one maximum per column (their order does not matter), each slot's in a
      // sector of its own: a maximum per entry into adjacent words kept one L2
      // slice busy for longer than all the weights took
      m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, lanes));
      m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2 * lanes));
      m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 4 * lanes));
      if (live && row == 0) atomicMax(&p.w.h_max[s * kMaxStride], m);
    } else if (live) {
      const float back = sm.col_scale[c0 + c];
      float* out = p.w.part + (long long)s * p.H + rb * 16 + row;
      out[0] = lo * back;
      out[8] = hi * back;
    }
  }

  // One unit, of staged segment q.  (What the segment is is read where it is used:
  // the loop over k has no registers for it.)
  template <int NT>
  __device__ void unit(int q, int at) {
    const volatile Segment& seg = sm.segs[q];
    float tot[NT][4];
#pragma unroll
    for (int i = 0; i < NT; ++i) tot[i][0] = tot[i][1] = tot[i][2] = tot[i][3] = 0.0f;
    // columns past the last repeat it and are not stored
    uint32_t col[NT];
    {
      const int n = seg.n, c0 = seg.c0;
#pragma unroll
    for (int i = 0; i < NT; ++i) col[i] = su32(cols) + (c0 + min(i * 8 + g, n - 1)) * stride() + t4 * 32;
    }
    for (int kb = kpart; kb < nkb; kb += ks) {
      wait_oldest();
      __syncwarp();
      const uint32_t piece = ring + slot * kPiece;
      float acc[NT][4], odd[NT][4];  // two chains of MMAs, even and odd k groups
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.0f;
        odd[i][0] = odd[i][1] = odd[i][2] = odd[i][3] = 0.0f;
      }
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const uint32_t at = piece + g * 128 + (((half * 4 + t4) ^ (g & 1) << 2) << 4);
        const uint4 lo = lds16(at), hi = lds16(at + 8 * 128);
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
        for (int i = 0; i < NT; ++i) {
#pragma unroll
          for (int term = 0; term < (UP ? 1 : 2); ++term) {
            const uint32_t xa = col[i] + kb * (UP ? 256 : 512) + term * 256 + half * 128;
            const uint4 x0 = lds16(xa), x1 = lds16(xa + 16);
            mma_t<__half>(acc[i], a[0][0], a[0][1], a[0][2], a[0][3], x0.x, x0.y);
            mma_t<__half>(odd[i], a[1][0], a[1][1], a[1][2], a[1][3], x0.z, x0.w);
            mma_t<__half>(acc[i], a[2][0], a[2][1], a[2][2], a[2][3], x1.x, x1.y);
            mma_t<__half>(odd[i], a[3][0], a[3][1], a[3][2], a[3][3], x1.z, x1.w);
          }
        }
      }
      float s0, s1;
      asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(s0), "=f"(s1) : "r"(piece + 16 * 128) : "memory");
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        tot[i][0] = fmaf(acc[i][0] + odd[i][0], s0, tot[i][0]);
        tot[i][1] = fmaf(acc[i][1] + odd[i][1], s0, tot[i][1]);
        tot[i][2] = fmaf(acc[i][2] + odd[i][2], s1, tot[i][2]);
        tot[i][3] = fmaf(acc[i][3] + odd[i][3], s1, tot[i][3]);
      }
      // the slot before this one: all lanes have read it since they met above
      copy_next(slot == 0 ? p.ring - 1 : slot - 1);
      slot = slot + 1 == p.ring ? 0 : slot + 1;
    }
    const int rb = at - seg.base, first = seg.first, n = seg.n, c0 = seg.c0;
    if (ks == 1) {
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int c = i * 8 + 2 * t4 + j;
          store(rb, g, first, c0, c, c < n, tot[i][j], tot[i][2 + j], 4);
        }
      return;
    }
    // units alternate between two halves of the buffer, so that one meeting of the
    // group per unit is enough
    const int ld = p.red_ld;
    float* part = red + (size_t)group * ks * 16 * ld + parity * ((ld - 4) / 2);
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      *reinterpret_cast<float2*>(&part[(kpart * 16 + g) * ld + i * 8 + 2 * t4]) = make_float2(tot[i][0], tot[i][1]);
      *reinterpret_cast<float2*>(&part[(kpart * 16 + g + 8) * ld + i * 8 + 2 * t4]) = make_float2(tot[i][2], tot[i][3]);
    }
    asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(ks * 32) : "memory");
    for (int c1 = kpart * 4; c1 < n; c1 += ks * 4) {  // four tokens' eight row pairs per warp
      const int c = c1 + (lane >> 3), row = lane & 7;
      float lo = 0.0f, hi = 0.0f;
      if (c < n)
        for (int w = 0; w < ks; ++w) {
          lo += part[(w * 16 + row) * ld + c];
          hi += part[(w * 16 + row + 8) * ld + c];
        }
      store(rb, row, first, c0, c, c < n, lo, hi, 1);
    }
    parity ^= 1;
  }

  // The segment of unit `at` (of active expert a or a later one, which a becomes).
  __device__ __forceinline__ Segment segment(int at, int& a) const {
    const Routing& r = sm.r;
    while (at >= r.units[a + 1]) ++a;
    const int pass = (at - r.units[a]) / rows_per_expert, e = r.active[a];
    Segment s;
    s.base = r.units[a] + pass * rows_per_expert;
    s.end = min(s.base + rows_per_expert, u1);
    s.first = r.start[e] + pass * cap();
    s.n = min(r.counts[e] - pass * cap(), cap());
    s.c0 = 0;
    return s;
  }

  template <typename F>
  __device__ bool run(int cta, int ctas, F&& before_use) {
    plan_units(cta, ctas);
    slot = 0;
    for (int s = 0; s < p.ring - 1; ++s) copy_next(s);
    if (!before_use()) return false;
    // While experts get few tokens, segments whose tokens fit into the staged columns
    // together are staged together: a CTA that meets the border between two experts
    // would otherwise do one part after the other, and the grid waits for it (7 tokens,
    // 2 of 16 experts of 1808 x 1552: 39.1 us, 45.7 one after the other; 8 tokens, 4 of
    // 16 of 2048 x 1024: 38.8 and 45.5; 32 tokens, 4 of 64: 88.3 and 93.2).  With more
    // than two tokens to an expert one after the other is faster (48 tokens, 8 of 128
    // experts of 4096 x 1024: 291.6 us, together 301; 64 tokens: 308 and 316).
    int mine = u0 + group;
    for (int at = u0, a = u0 < u1 ? sm.r.first_active : 0; at < u1;) {
      __syncthreads();
      int end = at, used = 0;
      int k = 0;
      while (end < u1) {
        Segment g1 = segment(end, a);
        if (used && (!p.together || used + g1.n > cap())) break;
        g1.c0 = used;
        if (threadIdx.x == 0) sm.segs[k] = g1;
        if ((int)threadIdx.x < g1.n) sm.slot[used + threadIdx.x] = sm.r.order[g1.first + threadIdx.x];
        used += g1.n;
        end = g1.end;
        ++k;
      }
      __syncthreads();
      stage(used);
      __syncthreads();
      for (int q = 0; q < k; ++q) {
        const int last = sm.segs[q].end;
        for (; mine < last; mine += groups) {
          if (sm.segs[q].n <= 8) unit<1>(q, mine);
          else unit<kMaxNT>(q, mine);
        }
      }
      at = end;
    }
    return true;
  }
};

// Phase 4: the weighted sum of each token's experts, in the order of their ranks.
template <typename T>
__device__ void combine_phase(const MoeParams& p, int cta, int ctas) {
  T* Y = static_cast<T*>(p.Y);
  for (long long i = (long long)cta * kThreads + threadIdx.x; i < (long long)p.T * p.H; i += (long long)ctas * kThreads) {
    const int t = (int)(i / p.H), c = (int)(i - (long long)t * p.H);
    float y = 0.0f;
    for (int j = 0; j < p.top_k; ++j) {
      const int slot = t * p.top_k + j;
      y = fmaf(__ldg(&p.w.gate[slot]), __ldcg(&p.w.part[(long long)slot * p.H + c]), y);
    }
    T o;
    from_f(y, o);
    Y[i] = o;
  }
}

// Kernel 2 (cooperative, one CTA per SM): routing, the two products, the sum.
__global__ void __launch_bounds__(kThreads, 1) moe_experts_kernel(const __grid_constant__ MoeParams p) {
  extern __shared__ __align__(128) uint8_t raw[];
  Smem& sm = *reinterpret_cast<Smem*>(raw);
  const int cta = blockIdx.x, ctas = gridDim.x;
  wait_for_predecessor();
  form_routing(p, sm.r);
  {
    Phase<true> up(p, sm, raw);
    up.run(cta, ctas, [] { return true; });
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  bool ok;
  {
    // the second product's first weights are on their way while the grid meets
    Phase<false> down(p, sm, raw);
    ok = down.run(cta, ctas, [&] { return grid_barrier(p, sm.r, (unsigned)ctas); });
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  if (!ok || !grid_barrier(p, sm.r, 2u * (unsigned)ctas)) return;
  if (p.type == RG_TYPE_F16) combine_phase<__half>(p, cta, ctas);
  else combine_phase<__nv_bfloat16>(p, cta, ctas);
}

size_t up256(size_t x) { return (x + 255) & ~size_t(255); }

// Workspace after the call block; base may be null (sizes only).
size_t layout(long long T, long long H, long long I, long long top_k, uint8_t* base, MoeWs* w) {
  size_t off = 0;
  auto take = [&](size_t bytes) {
    uint8_t* q = base ? base + off : nullptr;
    off = up256(off + bytes);
    return q;
  };
  const size_t slots = (size_t)(T * top_k);
  MoeWs m;
  m.gate = reinterpret_cast<float*>(take(slots * 4));
  m.expert = reinterpret_cast<int*>(take(slots * 4));
  m.h = reinterpret_cast<float*>(take(slots * I * 4));
  m.h_max = reinterpret_cast<uint32_t*>(take(slots * 4 * kMaxStride));
  m.arrived = reinterpret_cast<unsigned*>(take(4));
  m.part = reinterpret_cast<float*>(take(slots * H * 4));
  if (w) *w = m;
  return off;
}

}  // namespace

size_t moe_f8_scratch_bytes(long long T, long long H, long long I, long long top_k) {
  return layout(T, H, I, top_k, nullptr, nullptr);
}

// Warps that split k: as many (a power of two) as leave each eight 128-blocks
// (with two, the work around a unit took as long as the unit).  Fixed by the
// widths alone, so that a token's sums do not depend on what comes with it.
int k_split(long long K) {
  const long long nkb = (K + 127) / 128;
  int ks = 1;
  while (ks < 8 && nkb >= 16 * ks) ks *= 2;
  return ks;
}
// The call's shared memory: in each product room for the tokens that nearly every
// expert gets in one pass (the mean of even routing and two deviations), as far
// as it goes, at least three pieces per warp (two where one token leaves no
// room for three: I above 24960), and what is left to deeper rings.
void plan_smem(MoeParams& p) {
  const int bytes_up = token_bytes(p.H, false), bytes_down = token_bytes(p.I, true);
  const int wide = bytes_up > bytes_down ? bytes_up : bytes_down, ring1 = kWarps * kPiece;
  const double mean = (double)p.T * p.top_k / p.E;
  int want = (int)std::ceil(mean + 2.0 * std::sqrt(mean));
  if (want > 8) want = (want + 7) / 8 * 8;
  if (want > 8 * kMaxNT) want = 8 * kMaxNT;
  if (want > p.T) want = p.T;
  auto tiles = [](int n) { return n <= 8 ? 1 : kMaxNT; };
  auto ld = [&](int n) { return 16 * tiles(n) + 4; };  // two halves, see unit()
  p.ring = kMinRing;
  auto room_for = [&](int n) { return kSmemBytes - kFixedBytes - p.ring * ring1 - kWarps * 16 * 4 * ld(n); };
  if (wide > room_for(1)) p.ring = kTightRing;
  if (want > 8 && wide > room_for(want)) want = 8;  // the second column tile's sums take room too
  auto most = [&](int bytes) {
    int n = want;
    while (n * bytes > room_for(n)) n = n > 8 ? (n - 1) / 8 * 8 : n - 1;
    return n;
  };
  int n_up = most(bytes_up), n_down = most(bytes_down);
  const int tokens = n_up > n_down ? n_up : n_down;
  while (n_up * bytes_up > room_for(tokens)) --n_up;
  while (n_down * bytes_down > room_for(tokens)) --n_down;
  const int used = n_up * bytes_up > n_down * bytes_down ? n_up * bytes_up : n_down * bytes_down;
  int room = room_for(tokens);
  for (; p.ring < kMaxRing && room - used >= ring1; ++p.ring) room -= ring1;
  auto fit = [&](int bytes) {
    int n = room / bytes;
    if (n > 8) n = n / 8 * 8;
    return n > 8 * tiles(tokens) ? 8 * tiles(tokens) : n;
  };
  p.together = p.T * p.top_k <= 2 * p.E;
  p.cap_up = fit(bytes_up);
  p.cap_down = fit(bytes_down);
  p.red_ld = ld(tokens);
  p.red_off = kFixedBytes;
  p.cols_off = p.red_off + kWarps * 16 * 4 * p.red_ld;
  p.ring_off = kSmemBytes - p.ring * ring1;
}

cudaError_t launch_moe_f8(const MoeArgs& a, DevPlan* plan, void* scratch, cudaStream_t st,
                          unsigned long long wait_ns) {
  MoeParams p{a.X, a.WR, a.W13, a.S13, a.W2, a.S2, a.Y, (int)a.T, (int)a.H, (int)a.I, (int)a.E, (int)a.top_k, a.type,
              a.renorm ? 1 : 0, k_split(a.H), k_split(a.I), 0, 0, 0, 0, 0, 0, 0, 0, wait_ns, plan, {}};
  plan_smem(p);
  layout(a.T, a.H, a.I, a.top_k, static_cast<uint8_t*>(scratch), &p.w);
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  {
    static std::mutex mu;
    static int known[64];
    std::lock_guard<std::mutex> lock(mu);
    if (!known[dev]) {
      e = cudaFuncSetAttribute(moe_experts_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
      if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
      if (e != cudaSuccess) return e;
      known[dev] = sms;
    }
    sms = known[dev];
  }
  const unsigned blocks = 8u * (unsigned)((p.T + 7) / 8);
  e = launch_dependent(p.type == RG_TYPE_F16 ? moe_router_kernel<__half> : moe_router_kernel<__nv_bfloat16>,
                       dim3(blocks), dim3(kRouterThreads), 0, st, p);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)sms);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeCooperative;
  attr[0].val.cooperative = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, moe_experts_kernel, p);
}

}  // namespace rg
