// gl_moe.cu -- a whole mixture-of-experts layer for a few tokens: router,
// gated experts, weighted sum.
//
//   logits[t, e] = sum_h x[t, h] router[e, h],  p = softmax over e
//   idx[t, :], w[t, :] = the k largest p (ties: lowest e), optionally
//                        divided by their sum
//   h[t, i, f] = act(x_t W1_e[f]) * (x_t W1_e[F + f]),  e = idx[t, i]
//   y[t, n] = sum_i w[t, i] sum_f h[t, i, f] W2_e[n, f]
//
// Bound by HBM: every expert that some token reaches has its 3 H F weights
// read once, whatever T (up to 128) is.  So the weights are the M operand of
// the tensor-core products (tiles of 128 weight rows x 128 contraction
// elements, streamed by TMA through a deep ring) and the tokens are the N
// operand (16 .. 128 columns).
//
// Two launches:
//
// route_kernel (one cluster of 8 CTAs): each CTA forms the logits over its
// eighth of H, the sums meet through distributed shared memory, one warp per
// token picks its experts; the first CTA sorts the (token, expert) slots by
// expert and clears the counters of the second launch.
//
// experts_kernel (cooperative, one CTA per SM) runs two phases, W1 then W2.
// The phase's tiles x contraction blocks form one long list, and every CTA
// takes an equal contiguous piece of it (in blocks, not tiles: with one token
// there are fewer tiles than it takes to fill the SMs evenly; W1's tiles stay
// whole where that costs less than the exchange).  A tile cut by a border is
// summed from fp32 partials in the workspace, in CTA order, so results do not
// depend on timing.  The second phase's weights are loaded
// ahead while the first phase finishes: only the h operand, which has its own
// producer thread, waits for the experts' h to be complete.  After the second
// phase and a grid barrier, the slots are weighted and summed in fp32 and
// rounded once.  h is rounded to bf16 in between: it is an operand of the
// second product.
//
// Measured (time of both launches against the weights' bytes at the copy
// bandwidth): 13 tokens, top 8 of 128 experts of 7168 x 2048 970-993 us (978);
// 64 tokens, top 6 of 64 experts of 2048 x 1408 187-196 us (169); one token, top
// 2 of 8 experts of 4096 x 14336 120-122 us (108); one token, top 6 of 64 of
// 2048 x 1408 37 us (16).  The last is a chain of latencies: routing 6.6 us, 3 us
// to the second kernel, its set-up and first weights 3.9, W1 10.5, h to the
// other CTAs 3.9, W2 4.5, grid barrier and weighted sum 3.5.
#include <cuda_bf16.h>

#include <algorithm>
#include <cstring>
#include <new>

#include "gl_act.cuh"
#include "gl_internal.h"
#include "gl_ptx.cuh"

namespace gl {
namespace {

constexpr int kMaxT = GL_MOE_MAX_TOKENS;
constexpr int kMaxE = GL_MOE_MAX_EXPERTS;
constexpr int kMaxSlots = GL_MOE_MAX_TOKENS * GL_MOE_MAX_TOP_K;
constexpr int kMaxCtas = 256;  // counters are laid out for up to this many CTAs
constexpr int kPG = GL_MOE_MAX_PER_GROUP;  // experts whose tensor maps a launch carries (32 KB of parameters)

// ------------------------------------------------------------- the workspace
// Counters (cleared by route_kernel) and the plan (written by it).
struct Plan {
  int grid_bar;
  int n_act;             // experts that some token reaches
  int skip;              // the status word was set, or the routing is bad: nothing is written
  int pad[61];
  int ready[kMaxE];      // finished h tiles of each active expert
  int cut[kMaxCtas];     // arrivals at the W1 tile that starts in CTA c and ends in a later one
  int act_e[kMaxE];      // active experts, ascending
  int act_off[kMaxE + 1];  // their first slots
  int slot_tok[kMaxSlots];  // token of each sorted slot
  int slot_act[kMaxSlots];  // active-expert index of each sorted slot
  int pos_of[kMaxSlots];    // sorted slot of (token, choice); -1: none
};

__host__ __device__ constexpr int64_t up256(int64_t b) { return (b + 255) / 256 * 256; }
__host__ __device__ constexpr int ceil16(int n) { return (n + 15) / 16 * 16; }

struct Layout {
  int64_t h, p, part1, part2, bytes;
};
Layout layout_for(int T, int k, int H, int F, int ctas) {
  Layout l;
  const int64_t S = static_cast<int64_t>(T) * k, nt = ceil16(T);
  l.h = up256(sizeof(Plan));
  l.p = l.h + up256(S * F * 2);
  l.part1 = l.p + up256(S * H * 4);
  l.part2 = l.part1 + up256(2 * ctas * nt * 128 * 4);
  l.bytes = l.part2 + up256(ctas * nt * 128 * 4);
  return l;
}

// ------------------------------------------------------------------- routing
constexpr int kRouteCtas = 8;
constexpr int kRouteThreads = 512;
constexpr int kRouteWarps = kRouteThreads / 32;

struct RouteParams {
  const __nv_bfloat16* x;
  const __nv_bfloat16* router;  // null: idx and w are inputs
  int* idx;
  float* w;
  int32_t* status;
  Plan* plan;
  int T, E, k, H;
  int renorm;
};

__device__ __forceinline__ void mma_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float route_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

__device__ __forceinline__ void st_cluster_u16(uint32_t addr, uint16_t v) {
  asm volatile("st.shared::cluster.u16 [%0], %1;" ::"r"(addr), "h"(v) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }
__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

// How a CTA's warps share its logits: units of 16 experts x 32 tokens, and,
// while there are fewer of them than warps, `ks` parts of the CTA's slice of H.
struct RouteSplit {
  int et, tg, ks;
};
__host__ __device__ __forceinline__ RouteSplit route_split(int T, int E) {
  RouteSplit r;
  r.et = (E + 15) / 16;
  r.tg = (T + 31) / 32;
  const int units = r.et * r.tg;
  r.ks = units >= kRouteWarps ? 1 : kRouteWarps / units;
  return r;
}

// Logits of all tokens over this CTA's part of H into part[ks][T][E].  A
// thread takes 8 consecutive elements of its expert row and of its token row
// and uses them as the k pairs of two MMAs: the order of a contraction is
// free, as long as both operands share it.  TILES: token tiles of 8 per unit;
// the fewer there are, the more of the slice is loaded at once (a warp's chain
// of loads is what this takes: one token over 128 experts of 7168 x 2048 ran
// 133 us with four tiles and two steps at once, 129 us with one and four).
template <int TILES, int UNROLL>
__device__ __forceinline__ void route_logits(const RouteParams& p, const RouteSplit& sp, float* part, int rank, int warp,
                                             int lane) {
  const int g = lane >> 2, t4 = lane & 3;
  const int slice = (p.H + kRouteCtas * 32 - 1) / (kRouteCtas * 32) * 32;
  const int sub = (slice / 32 + sp.ks - 1) / sp.ks * 32;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  for (int u = warp; u < sp.et * sp.tg * sp.ks; u += kRouteWarps) {
    const int e0 = u % sp.et * 16, n0 = u / sp.et % sp.tg * 32, ks = u / (sp.et * sp.tg);
    const int end = min(p.H, (rank + 1) * slice);
    const int k0 = min(end, rank * slice + ks * sub), k1 = min(end, k0 + sub);
    const bool r0 = e0 + g < p.E, r1 = e0 + g + 8 < p.E;
    const __nv_bfloat16* w0 = p.router + static_cast<int64_t>(e0 + g) * p.H;
    const __nv_bfloat16* w1 = w0 + static_cast<int64_t>(8) * p.H;
    float c[TILES][4] = {};
#pragma unroll UNROLL
    for (int kk = k0 + t4 * 8; kk - t4 * 8 < k1; kk += 32) {
      const bool in = kk < k1;
      const uint4 a = (in && r0) ? __ldg(reinterpret_cast<const uint4*>(w0 + kk)) : zero;
      const uint4 b = (in && r1) ? __ldg(reinterpret_cast<const uint4*>(w1 + kk)) : zero;
      uint4 v[TILES];
#pragma unroll
      for (int j = 0; j < TILES; ++j) {
        const int t = n0 + j * 8 + g;
        v[j] = (in && t < p.T) ? __ldg(reinterpret_cast<const uint4*>(p.x + static_cast<int64_t>(t) * p.H + kk)) : zero;
      }
#pragma unroll
      for (int j = 0; j < TILES; ++j) {
        mma_16816(c[j], a.x, b.x, a.y, b.y, v[j].x, v[j].y);
        mma_16816(c[j], a.z, b.z, a.w, b.w, v[j].z, v[j].w);
      }
    }
    float* dst = part + ks * p.T * p.E;
#pragma unroll
    for (int j = 0; j < TILES; ++j) {
      const int t = n0 + j * 8 + t4 * 2;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int tt = t + (i & 1), e = e0 + g + (i >> 1) * 8;
        if (tt < p.T && e < p.E) dst[tt * p.E + e] = c[j][i];
      }
    }
  }
}

// One warp picks token t's experts, from the sums of all CTAs' parts, and
// leaves them in the first CTA's s_idx too.  Keys order by value, equal ones
// by the lower index; a NaN orders last but stays a candidate, so that k valid
// experts always come out (and the token's weights become NaN).  Of s_skip the
// first CTA's counts.
__device__ __forceinline__ void route_pick(const RouteParams& p, const float* part, const short* s_idx,
                                           const int* s_skip, int t, int lane) {
  constexpr int kPer = kMaxE / 32;
  const int per = (p.E + 31) >> 5;
  float v[kPer];
  uint32_t key[kPer];
  float m = __int_as_float(0xff800000);
  const bool skip = __float_as_int(ld_cluster_f32(mapa_shared(smem_u32(s_skip), 0))) != 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = lane + i * 32;
    v[i] = 0.0f;
    key[i] = 0u;
    if (i < per && e < p.E) {
      const uint32_t at = smem_u32(part + t * p.E + e);
      float f[kRouteCtas];
#pragma unroll
      for (int c = 0; c < kRouteCtas; ++c) f[c] = ld_cluster_f32(mapa_shared(at, c));
#pragma unroll
      for (int c = 0; c < kRouteCtas; ++c) v[i] += f[c];
      m = fmaxf(m, v[i]);
      const uint32_t b = __float_as_uint(v[i] + 0.0f);  // -0 and 0 are equal
      key[i] = (v[i] != v[i]) ? 1u : ((b & 0x80000000u) ? ~b : (b | 0x80000000u));
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  float z = 0.0f;
#pragma unroll
  for (int i = 0; i < kPer; ++i)
    if (i < per && lane + i * 32 < p.E) z += expf(v[i] - m);
  z = route_sum(z);
  float mine = 0.0f;
  int pick = 0;
  for (int n = 0; n < p.k; ++n) {
    uint32_t bk = 0u;
    int be = 0;
    float bv = 0.0f;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (i < per && key[i] > bk) {
        bk = key[i];
        be = lane + i * 32;
        bv = v[i];
      }
    const uint32_t top = __reduce_max_sync(0xffffffffu, bk);
    const int e = static_cast<int>(__reduce_min_sync(0xffffffffu, bk == top ? static_cast<uint32_t>(be) : 0xffffffffu));
    const float l = __shfl_sync(0xffffffffu, bv, e & 31);  // the expert's own lane holds it
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (lane + i * 32 == e) key[i] = 0u;
    if (lane == n) {
      mine = expf(l - m);
      pick = e;
    }
  }
  const float total = route_sum(mine);
  // z is NaN when any logit is: so are then the weights, renormalised or not
  const float denom = p.renorm ? (z == z ? total : z) : z;
  if (lane < p.k) {
    if (!skip) {
      p.idx[t * p.k + lane] = pick;
      p.w[t * p.k + lane] = mine / denom;
    }
    st_cluster_u16(mapa_shared(smem_u32(s_idx + t * p.k + lane), 0), static_cast<uint16_t>(pick));
  }
}

__global__ void __cluster_dims__(kRouteCtas, 1, 1) __maxnreg__(80)
    route_kernel(const RouteParams p) {
  extern __shared__ float part[];  // logits over this CTA's part of H; then the first CTA's histograms
  __shared__ short s_idx[kMaxSlots];
  __shared__ int s_cnt[kMaxE + 1], s_act[kMaxE + 1], s_bad, s_skip;
  const int rank = static_cast<int>(cluster_ctarank());
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  grid_launch_dependents();  // experts_kernel may set itself up meanwhile
  // The status word is read once, by one thread: a call beside this one may set it
  // meanwhile, and where threads or CTAs went by different values, some would wait
  // at barriers for others that had left.  A set word only holds back the outputs:
  // here s_skip (the word itself, copied while the logits are formed), in the next
  // kernel the plan's copy.
  const bool reader = rank == 0 && tid == 0;
  if (reader) cp_async4(smem_u32(&s_skip), p.status);
  Plan* pl = p.plan;
  const int S = p.T * p.k;
  const bool few = p.T <= kRouteWarps;  // the first CTA picks for all tokens
  if (tid == 0) s_bad = 0;
  __syncthreads();
  if (rank == kRouteCtas - 1) {
    for (int i = tid; i < kMaxE; i += kRouteThreads) pl->ready[i] = 0;
    for (int i = tid; i < kMaxCtas; i += kRouteThreads) pl->cut[i] = 0;
    if (tid == 0) pl->grid_bar = 0;
  }
  if (p.router != nullptr) {
    const RouteSplit sp = route_split(p.T, p.E);
    if (p.T <= 8) route_logits<1, 4>(p, sp, part, rank, warp, lane);
    else route_logits<4, 2>(p, sp, part, rank, warp, lane);
    if (sp.ks > 1) {
      __syncthreads();
      for (int i = tid; i < p.T * p.E; i += kRouteThreads) {
        float v = part[i];
        for (int k = 1; k < sp.ks; ++k) v += part[k * p.T * p.E + i];
        part[i] = v;
      }
    }
    if (reader) cp_async_wait_all();
    cluster_sync();
    if (few) {
      if (rank == 0 && warp < p.T) route_pick(p, part, s_idx, &s_skip, warp, lane);
    } else {
      for (int t = rank + kRouteCtas * warp; t < p.T; t += kRouteCtas * kRouteWarps)
        route_pick(p, part, s_idx, &s_skip, t, lane);
    }
  } else if (rank == 0) {
    if (reader) cp_async_wait_all();
    for (int s = tid; s < S; s += kRouteThreads) {
      const int e = p.idx[s];
      const bool ok = e >= -1 && e < p.E;
      if (!ok) s_bad = 1;
      s_idx[s] = static_cast<short>(ok ? e : -1);
    }
    __syncthreads();
    for (int t = tid; t < p.T; t += kRouteThreads)  // one expert twice for one token
      for (int i = 1; i < p.k; ++i)
        for (int j = 0; j < i; ++j)
          if (s_idx[t * p.k + i] >= 0 && s_idx[t * p.k + i] == s_idx[t * p.k + j]) s_bad = 1;
  }
  // The first CTA goes on once the picks are in its s_idx, the others leave
  // once their logits have been read.
  cluster_arrive();
  if (rank != 0) {
    cluster_wait();
    return;
  }
  if (few) __syncthreads();
  else cluster_wait();
  if (S <= 32) {
    // one warp holds all slots: positions by comparison with every other slot
    if (warp == 0) {
      const int e = lane < S ? s_idx[lane] : -1;
      const uint32_t same = __match_any_sync(0xffffffffu, e);
      const bool first = e >= 0 && (same & ((1u << lane) - 1)) == 0;
      int pos = __popc(same & ((1u << lane) - 1)), j = 0;
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        const int ei = __shfl_sync(0xffffffffu, first ? e : -1, i);
        const int ni = __popc(__shfl_sync(0xffffffffu, same, i));
        if (ei >= 0 && ei < e) {
          pos += ni;
          ++j;
        }
      }
      const int n_act = __popc(__ballot_sync(0xffffffffu, first)), n = __popc(__ballot_sync(0xffffffffu, e >= 0));
      if (e >= 0) {
        pl->slot_tok[pos] = lane / p.k;
        pl->slot_act[pos] = j;
        if (first) {
          pl->act_e[j] = e;
          pl->act_off[j] = pos;
        }
      }
      if (lane < S) pl->pos_of[lane] = e >= 0 ? pos : -1;
      if (lane == 0) {
        pl->n_act = n_act;
        pl->act_off[n_act] = n;
        pl->skip = s_skip | s_bad;
        if (s_bad) atomicOr(p.status, GL_DEV_BAD_INDEX);
      }
    }
    if (few) cluster_wait();
    return;
  }
  // More: sort the slots by expert (ascending), stable in the token: a histogram
  // per chunk of 32 slots, prefixes over the chunks and then over the experts.
  uint16_t* hist = reinterpret_cast<uint16_t*>(part);  // [chunks][E]
  const int chunks = (S + 31) >> 5;
  for (int i = tid; i < chunks * p.E; i += kRouteThreads) hist[i] = 0;
  __syncthreads();
  for (int c = warp; c < chunks; c += kRouteWarps) {
    const int s = c * 32 + lane;
    const int e = s < S ? s_idx[s] : -1;
    const uint32_t same = __match_any_sync(0xffffffffu, e);
    if (e >= 0 && (same & ((1u << lane) - 1)) == 0) hist[c * p.E + e] = static_cast<uint16_t>(__popc(same));
  }
  __syncthreads();
  int cnt = 0;
  if (tid < kMaxE) {
    if (tid < p.E)
      for (int c = 0; c < chunks; ++c) {
        const int h = hist[c * p.E + tid];
        hist[c * p.E + tid] = static_cast<uint16_t>(cnt);
        cnt += h;
      }
    s_cnt[tid] = cnt;
    s_act[tid] = cnt > 0;
  }
  __syncthreads();
  if (warp == 0) {  // exclusive scans of the counts and of the active flags, 8 experts a lane
    constexpr int kPer = kMaxE / 32;
    int c = 0, a = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      c += s_cnt[lane * kPer + i];
      a += s_act[lane * kPer + i];
    }
    int ci = c, ai = a;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int cu = __shfl_up_sync(0xffffffffu, ci, o), au = __shfl_up_sync(0xffffffffu, ai, o);
      if (lane >= o) {
        ci += cu;
        ai += au;
      }
    }
    c = ci - c;
    a = ai - a;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int nc = s_cnt[lane * kPer + i], na = s_act[lane * kPer + i];
      s_cnt[lane * kPer + i] = c;
      s_act[lane * kPer + i] = a;
      c += nc;
      a += na;
    }
    if (lane == 31) {
      s_cnt[kMaxE] = c;
      s_act[kMaxE] = a;
    }
  }
  __syncthreads();
  if (tid < p.E && cnt > 0) {
    pl->act_e[s_act[tid]] = tid;
    pl->act_off[s_act[tid]] = s_cnt[tid];
  }
  for (int c = warp; c < chunks; c += kRouteWarps) {
    const int s = c * 32 + lane;
    const int e = s < S ? s_idx[s] : -1;
    const uint32_t same = __match_any_sync(0xffffffffu, e);
    if (s < S) {
      int pos = -1;
      if (e >= 0) {
        pos = s_cnt[e] + hist[c * p.E + e] + __popc(same & ((1u << lane) - 1));
        pl->slot_tok[pos] = s / p.k;
        pl->slot_act[pos] = s_act[e];
      }
      pl->pos_of[s] = pos;
    }
  }
  if (tid == 0) {
    pl->n_act = s_act[kMaxE];
    pl->act_off[s_act[kMaxE]] = s_cnt[kMaxE];
    pl->skip = s_skip | s_bad;
    if (s_bad) atomicOr(p.status, GL_DEV_BAD_INDEX);
  }
  if (few) cluster_wait();
}

// Dynamic shared memory of route_kernel.
int route_smem(int T, int E, int k, bool router) {
  const int hist = (T * k + 31) / 32 * E * 2;
  return std::max(hist, router ? route_split(T, E).ks * T * E * 4 : 0);
}

// ------------------------------------------------------------------- experts
constexpr int kThreads = 256;  // warps: 0 weights, 1 tokens / h, 2 MMA, 3 -, 4-7 epilogue
// A block is 128 weight rows x 128 contraction elements (two boxes of one
// 128-byte swizzle row).  The MMA thread spends some 0.2 us per block on its
// barriers beside the MMAs' 0.1 us per 64 elements: with blocks of 64 that is
// little less than the 0.37 us an SM's share of HBM takes, and the W2 blocks
// already loaded when h arrives took 4 us to work off.
constexpr int kBK = 128;
constexpr int kABytes = 128 * kBK * 2;
constexpr int kHalf = kABytes / 2;  // one 64-element box of it
constexpr int kChunk = 16;     // slots per epilogue step
constexpr int kMaxStages = 5;  // 160 KB of weights in flight: with six the SMs' shares of HBM drift apart
// (8 experts of 4096 x 14336, one token: 125 against 122 us), with three they wait (127)
constexpr int kBarBytes = 256;
constexpr int kExBytes = kChunk * 64 * 4;

struct ExpertParams {
  CUtensorMap x;   // {H, T} box {64, nt}
  CUtensorMap w1;  // stacked {H, F, 2E} box {64, 64, 1}
  CUtensorMap w2;  // stacked {F, H, E} box {64, 128, 1}
  CUtensorMap h;   // {F, S} box {64, 16}
  Plan* plan;
  int32_t* status;
  __nv_bfloat16* hbuf;
  float* pbuf;
  float* part1;
  float* part2;
  const float* w;
  __nv_bfloat16* y;
  int T, k, H, F;
  int act;
  int nt;      // token columns of the W1 products: T rounded up to 16
  int stages;
  uint64_t wait_ns;
  int hold_loads;
};

template <bool PG>
struct ExpertMaps {
  CUtensorMap w1[kPG];  // {H, F, 2} box {64, 64, 1}
  CUtensorMap w2[kPG];  // {F, H, 1} box {64, 128, 1}
  __device__ const CUtensorMap* m1(int e) const { return &w1[e]; }
  __device__ const CUtensorMap* m2(int e) const { return &w2[e]; }
};
template <>
struct ExpertMaps<false> {
  int unused;
  __device__ const CUtensorMap* m1(int) const { return nullptr; }
  __device__ const CUtensorMap* m2(int) const { return nullptr; }
};

// One phase's list of blocks: unit u = (active expert, tile) has `kb` blocks;
// of the list's grains of `grain` blocks (one, or a whole tile's) CTA c takes
// [c total / ctas, (c + 1) total / ctas).
struct Phase {
  int tiles;      // tiles per expert
  int kb;         // blocks per tile
  int grain;      // blocks that stay together
  int64_t total;  // grains
  int ctas;       // CTAs with work
  __device__ int64_t begin(int c) const { return total * c / ctas * grain; }
  // the CTA that takes block b
  __device__ int owner(int64_t b) const { return static_cast<int>(((b / grain + 1) * ctas - 1) / total); }
};

__device__ __forceinline__ Phase make_phase(int n_act, int tiles, int kb, int ctas, bool whole) {
  Phase f;
  f.tiles = tiles;
  f.kb = kb;
  f.grain = whole ? kb : 1;
  f.total = static_cast<int64_t>(n_act) * tiles * (whole ? 1 : kb);
  f.ctas = static_cast<int>(f.total < ctas ? f.total : ctas);
  return f;
}

// Whether the W1 tiles are better left whole: the slowest CTA's extra blocks
// against the exchange of a cut tile's partials (two trips through L2 and an
// atomic, about as long as kCutBlocks blocks take to stream).
constexpr int kCutBlocks = 4;
__device__ __forceinline__ bool keep_whole(int units, int kb, int ctas) {
  const int64_t most = static_cast<int64_t>((units + ctas - 1) / ctas) * kb;
  return most <= static_cast<int64_t>(units) * kb / ctas + kCutBlocks;
}

// Blocks [lo, hi) of one tile: what a CTA accumulates at a time.
struct Segment {
  int j, tile;  // active expert, tile
  int lo, hi;
  int64_t first;  // block number of the tile's block 0
};

// Walks the segments of CTA c: f(segment) -> continue?
template <typename Fn>
__device__ __forceinline__ bool for_segments(const Phase& ph, int c, Fn f) {
  if (c >= ph.ctas) return true;
  int64_t b = ph.begin(c);
  const int64_t e = ph.begin(c + 1);
  while (b < e) {
    const int64_t u = b / ph.kb;
    Segment s;
    s.j = static_cast<int>(u / ph.tiles);
    s.tile = static_cast<int>(u - static_cast<int64_t>(s.j) * ph.tiles);
    s.first = u * ph.kb;
    s.lo = static_cast<int>(b - s.first);
    s.hi = static_cast<int>(e - s.first < ph.kb ? e - s.first : ph.kb);
    if (!f(s)) return false;
    b = s.first + s.hi;
  }
  return true;
}

__device__ __forceinline__ void report_abort(volatile int* abort_flag, int32_t* status) {
  if (!*abort_flag) {
    *abort_flag = 1;
    atomicOr(status, GL_DEV_TIMEOUT);
  }
}

__device__ __forceinline__ int ld_acquire(const int* p) {
  int v;
  asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
// A release by one thread after a barrier covers the writes of all the
// barrier's threads, an acquire before one their reads.
__device__ __forceinline__ int atom_acq_rel_add1(int* p) {
  int v;
  asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], 1;" : "=r"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ void red_release_add(int* p, int n) {
  asm volatile("red.release.gpu.global.add.s32 [%0], %1;" ::"l"(p), "r"(n) : "memory");
}
// Orders generic-proxy accesses to global memory before later ones of the
// async proxy (TMA) and the other way round.
__device__ __forceinline__ void fence_proxy_async_all() { asm volatile("fence.proxy.async;" ::: "memory"); }

// Wait until *p reaches `want` (another CTA's releases), bounded.
__device__ __forceinline__ bool wait_count(const int* p, int want, const volatile int* abort, uint64_t limit_ns) {
  if (ld_acquire(p) >= want) return true;
  const uint64_t t0 = globaltimer_ns();
  while (true) {
    if (ld_acquire(p) >= want) return true;
    if (*abort) return false;
    if (globaltimer_ns() - t0 > limit_ns) return false;
  }
}

__device__ __forceinline__ float4 add4(float4 a, float4 b) {
  return make_float4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w);
}

__device__ __forceinline__ void bar_epilogue() { asm volatile("bar.sync 1, 128;" ::: "memory"); }
// The same barrier with a vote: the epilogue warps go on together or give up
// together, whatever each of their waits returned.
__device__ __forceinline__ bool bar_epilogue_all(bool ok) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %1, 0;\n\t"
      "bar.red.and.pred q, 1, 128, p;\n\t"
      "selp.b32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(ok))
      : "memory");
  return r != 0;
}

template <bool PG>
__global__ void __launch_bounds__(kThreads, 1)
    experts_kernel(const __grid_constant__ ExpertParams p, const __grid_constant__ ExpertMaps<PG> pg) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int stage_bytes = kABytes + p.nt * kBK * 2;
  uint8_t* tail = smem + p.stages * stage_bytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(tail);
  uint64_t* empty = full + kMaxStages;
  uint64_t* tfull = empty + kMaxStages;
  uint64_t* tempty = tfull + 2;
  uint64_t* mma_done = tempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma_done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* flag = abort_flag + 1;  // one word that thread 0 of a group hands to the others
  static_assert((2 * kMaxStages + 5) * 8 + 12 <= kBarBytes, "barriers");
  float* ex = reinterpret_cast<float*>(tail + kBarBytes);  // [kChunk][64] second factors of a tile
  int* act_e = reinterpret_cast<int*>(tail + kBarBytes + kExBytes);
  int* act_off = act_e + kMaxE;
  uint8_t* slot_tok = reinterpret_cast<uint8_t*>(act_off + kMaxE + 4);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cta = static_cast<int>(blockIdx.x);
  if (warp == 3 && lane == 0) {
    tma_prefetch_desc(&p.x);
    tma_prefetch_desc(&p.h);
    if (!PG) {
      tma_prefetch_desc(&p.w1);
      tma_prefetch_desc(&p.w2);
    }
  }
  if (tid == 0) {
    *abort_flag = 0;
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(&full[s], 2);  // the weights' producer and the tokens' producer
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], 4);
    }
    mbar_init(mma_done, 1);
    fence_barrier_init();
  }
  if (warp == 2) {
    tmem_alloc(tmem_slot, 256);  // two 128 x 128 fp32 accumulators
    tmem_relinquish();
  }
  grid_dependency_wait();  // route_kernel's results from here on
  // the plan: all of it at once, whatever part is in use, so that its loads overlap
  const int skip = p.plan->skip;  // one value for the whole grid: its CTAs and warps wait for one another
  const int n_act = p.plan->n_act;
  static_assert(kThreads == kMaxE, "one expert a thread");
  act_e[tid] = p.plan->act_e[tid];
  act_off[tid] = p.plan->act_off[tid];
  if (tid == 0) act_off[kMaxE] = p.plan->act_off[kMaxE];
  for (int i = tid; i < p.T * p.k; i += kThreads) slot_tok[i] = static_cast<uint8_t>(p.plan->slot_tok[i]);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  if (skip != 0) {
    if (warp == 2) tmem_dealloc(tmem_base, 256);
    return;
  }
  const int ctas = static_cast<int>(gridDim.x);
  const int tiles1 = (p.F + 63) / 64, kb1 = (p.H + kBK - 1) / kBK;
  const Phase f1 = make_phase(n_act, tiles1, kb1, ctas, keep_whole(n_act * tiles1, kb1, ctas));
  const Phase f2 = make_phase(n_act, (p.H + 127) / 128, (p.F + kBK - 1) / kBK, ctas, false);

  // Before a producer leaves: wait for its last copies to land (the stage also
  // waits for the other producer, which may have given up: one bound for all).
  auto drain = [&](int stage, uint32_t phase, int issued) {
    if (p.hold_loads) return;  // none issued
    const int inflight = issued < p.stages ? issued : p.stages;
    const uint64_t deadline = globaltimer_ns() + kWaitLimitNs;
    for (int i = 0; i < inflight; ++i) {
      if (--stage < 0) { stage = p.stages - 1; phase ^= 1u; }
      mbar_wait_until(&full[stage], phase, deadline);
    }
  };

  if (warp == 0) {
    // ===================== weights =====================
    if (lane == 0) {
      const uint64_t policy = l2_policy_evict_first();
      int stage = 0, issued = 0;
      uint32_t phase = 0;
      auto walk = [&](const Phase& f, auto load) {
        for_segments(f, cta, [&](const Segment& s) {
          const int e = act_e[s.j];
          for (int kb = s.lo; kb < s.hi; ++kb) {
            if (!mbar_wait(&empty[stage], phase ^ 1u, abort_flag, p.wait_ns)) {
              report_abort(abort_flag, p.status);
              return false;
            }
            if (!p.hold_loads) {
              mbar_arrive_expect_tx(&full[stage], kABytes);
              load(smem + stage * stage_bytes, &full[stage], e, s.tile, kb);
            }
            ++issued;
            if (++stage == p.stages) { stage = 0; phase ^= 1u; }
          }
          return true;
        });
      };
      walk(f1, [&](uint8_t* dst, uint64_t* bar, int e, int tile, int kb) {
        const CUtensorMap* m = PG ? pg.m1(e) : &p.w1;
        const int z = PG ? 0 : 2 * e;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          tma_load_3d_hint(dst + c * kHalf, m, bar, kb * kBK + c * 64, tile * 64, z, policy);
          tma_load_3d_hint(dst + c * kHalf + kHalf / 2, m, bar, kb * kBK + c * 64, tile * 64, z + 1, policy);
        }
      });
      if (!*abort_flag)
        walk(f2, [&](uint8_t* dst, uint64_t* bar, int e, int tile, int kb) {
#pragma unroll
          for (int c = 0; c < 2; ++c)
            tma_load_3d_hint(dst + c * kHalf, PG ? pg.m2(e) : &p.w2, bar, kb * kBK + c * 64, tile * 128, PG ? 0 : e, policy);
        });
      drain(stage, phase, issued);
    }
  } else if (warp == 1) {
    // ===================== tokens, then h =====================
    if (lane == 0) {
      int stage = 0, issued = 0;
      uint32_t phase = 0;
      int ready_j = -1;
      auto walk = [&](const Phase& f, bool second) {
        return for_segments(f, cta, [&](const Segment& s) {
          const int off = act_off[s.j];
          const int rows = second ? ceil16(act_off[s.j + 1] - off) : p.nt;
          if (second && ready_j != s.j) {
            // h of this expert: all of its tiles are written
            if (!wait_count(&p.plan->ready[s.j], f1.tiles, abort_flag, p.wait_ns)) {
              report_abort(abort_flag, p.status);
              return false;
            }
            fence_proxy_async_all();
            ready_j = s.j;
          }
          for (int kb = s.lo; kb < s.hi; ++kb) {
            if (!mbar_wait(&empty[stage], phase ^ 1u, abort_flag, p.wait_ns)) {
              report_abort(abort_flag, p.status);
              return false;
            }
            uint8_t* dst = smem + stage * stage_bytes + kABytes;
            if (!p.hold_loads) {
              mbar_arrive_expect_tx(&full[stage], rows * kBK * 2);
#pragma unroll
              for (int c = 0; c < 2; ++c) {
                uint8_t* to = dst + c * p.nt * 128;
                if (!second) {
                  tma_load_2d(to, &p.x, &full[stage], kb * kBK + c * 64, 0);
                } else {
                  for (int r = 0; r < rows; r += 16)
                    tma_load_2d(to + r * 128, &p.h, &full[stage], kb * kBK + c * 64, off + r);
                }
              }
            }
            ++issued;
            if (++stage == p.stages) { stage = 0; phase ^= 1u; }
          }
          return true;
        });
      };
      if (walk(f1, false)) walk(f2, true);
      drain(stage, phase, issued);
    }
  } else if (warp == 2) {
    // ===================== MMA =====================
    // One thread waits, issues and commits (the whole warp at the barriers is
    // slower by a fifth per block).
    if (lane == 0) {
      int stage = 0, it = 0;
      uint32_t phase = 0;
      auto walk = [&](const Phase& f, bool second) {
        return for_segments(f, cta, [&](const Segment& s) {
          const int n = second ? ceil16(act_off[s.j + 1] - act_off[s.j]) : p.nt;
          const uint32_t idesc = idesc_bf16_f32(128, n, 0, 0);
          const int buf = it & 1;
          const uint32_t tph = (it >> 1) & 1;
          ++it;
          if (!mbar_wait(&tempty[buf], tph ^ 1u, abort_flag, p.wait_ns)) {
            report_abort(abort_flag, p.status);
            return false;
          }
          tc_fence_after();
          for (int kb = s.lo; kb < s.hi; ++kb) {
            if (!mbar_wait(&full[stage], phase, abort_flag, p.wait_ns)) {
              report_abort(abort_flag, p.status);
              return false;
            }
            tc_fence_after();
            const uint32_t sa = smem_u32(smem + stage * stage_bytes);
            const uint64_t ad = smem_desc_sw128(sa, 16, 1024);
            const uint64_t bd = smem_desc_sw128(sa + kABytes, 16, 1024);
            const uint32_t b_half = static_cast<uint32_t>(p.nt) * 8;  // 16-byte units of one box of tokens
#pragma unroll
            for (int ks = 0; ks < 8; ++ks)
              mma_bf16_ss(tmem_base + buf * 128, desc_add(ad, (ks >> 2) * (kHalf / 16) + (ks & 3) * 2),
                          desc_add(bd, (ks >> 2) * b_half + (ks & 3) * 2), idesc, (kb > s.lo || ks > 0) ? 1u : 0u);
            tc_commit(&empty[stage]);
            if (kb == s.hi - 1) tc_commit(&tfull[buf]);
            if (++stage == p.stages) { stage = 0; phase ^= 1u; }
          }
          return true;
        });
      };
      if (walk(f1, false)) walk(f2, true);
      tc_commit(mma_done);
      mbar_wait_bounded(mma_done, 0);  // no MMA in flight past this point
    }
    __syncwarp();
  } else if (warp >= 4) {
    // ===================== epilogue =====================
    const int q = warp & 3;             // TMEM lane quarter
    const int row = q * 32 + lane;      // weight row of the tile
    const int et = tid - 128;           // 0..127
    int it = 0;
    auto store_h = [&](int slot, int f, float u0, float u1) {
      float a[1] = {u0};
      act_values(p.act, a);
      if (f < p.F) p.hbuf[static_cast<int64_t>(slot) * p.F + f] = __float2bfloat16_rn(a[0] * u1);
    };
    // Finished tiles of expert ready_j that are not yet announced: other CTAs' TMA
    // reads h, so the announcement takes a proxy fence and a release.  It is made
    // once per expert: per tile it cost more than a tile's products where tokens are
    // short (20 tokens, top 4 of 129 experts of 272 x 8312: 263 us instead of 190).
    int ready_j = 0, ready_n = 0;
    auto announce = [&]() {
      if (ready_n == 0) return;
      fence_proxy_async_all();
      bar_epilogue();
      if (et == 0) red_release_add(&p.plan->ready[ready_j], ready_n);
      ready_n = 0;
    };
    const bool ok = for_segments(f1, cta, [&](const Segment& s) {
      if (s.j != ready_j) announce();
      ready_j = s.j;
      const int buf = it & 1;
      const uint32_t tph = (it >> 1) & 1;
      ++it;
      const bool done = mbar_wait(&tfull[buf], tph, abort_flag, p.wait_ns);
      if (!done) report_abort(abort_flag, p.status);
      if (!bar_epilogue_all(done)) return false;
      tc_fence_after();
      const uint32_t acc = tmem_base + buf * 128 + (static_cast<uint32_t>(q * 32) << 16);
      const int off = act_off[s.j], n = act_off[s.j + 1] - off;
      const bool whole = s.lo == 0 && s.hi == f1.kb;
      const int f0 = s.tile * 64;
      // a cut tile: this CTA's partial is its first (0) or its last (1) segment
      float* part = p.part1 + static_cast<int64_t>(2 * cta + (s.first + s.lo == f1.begin(cta) ? 0 : 1)) * p.nt * 128;
      for (int s0 = 0; s0 < n; s0 += kChunk) {
        uint32_t r[kChunk];
#pragma unroll
        for (int i = 0; i < kChunk; ++i) tmem_ld_32x32b_x1(acc + slot_tok[off + min(s0 + i, n - 1)], r[i]);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < kChunk; ++i) asm volatile("" : "+r"(r[i]));
        if (s0 + kChunk >= n) {  // accumulator read
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&tempty[buf]);
        }
        if (whole) {
          // rows 64..127 of the tile are the second factors of rows 0..63
          if (row >= 64) {
#pragma unroll
            for (int i = 0; i < kChunk; ++i) ex[i * 64 + row - 64] = __uint_as_float(r[i]);
          }
          bar_epilogue();
          if (row < 64) {
#pragma unroll
            for (int i = 0; i < kChunk; ++i)
              if (s0 + i < n) store_h(off + s0 + i, f0 + row, __uint_as_float(r[i]), ex[i * 64 + row]);
          }
          bar_epilogue();
        } else {
#pragma unroll
          for (int i = 0; i < kChunk; ++i)
            if (s0 + i < n) part[(s0 + i) * 128 + row] = __uint_as_float(r[i]);
        }
      }
      if (!whole) {
        // the last CTA to arrive at a cut tile adds the partials, in CTA order
        const int c0 = f1.owner(s.first), c1 = f1.owner(s.first + f1.kb - 1);
        bar_epilogue();
        if (et == 0) *flag = atom_acq_rel_add1(&p.plan->cut[c0]) == c1 - c0;
        bar_epilogue();
        if (!*flag) return true;
        const int r64 = et & 63;
        constexpr int kSlots = 4;  // of every other slot, the partials asked for at once
        for (int i0 = et >> 6; i0 < n; i0 += 2 * kSlots) {
          float u0[kSlots] = {}, u1[kSlots] = {};
          for (int c = c0; c <= c1; ++c) {
            const int which = (c == c0 && s.first != f1.begin(c0)) ? 1 : 0;
            const float* src = p.part1 + (static_cast<int64_t>(2 * c + which) * p.nt + i0) * 128 + r64;
#pragma unroll
            for (int i = 0; i < kSlots; ++i) {
              const int o = min(2 * i, n - 1 - i0) * 128;
              u0[i] += __ldcg(src + o);
              u1[i] += __ldcg(src + o + 64);
            }
          }
#pragma unroll
          for (int i = 0; i < kSlots; ++i)
            if (i0 + 2 * i < n) store_h(off + i0 + 2 * i, f0 + r64, u0[i], u1[i]);
        }
      }
      ++ready_n;
      return true;
    });
    if (ok) announce();
    if (ok)
      for_segments(f2, cta, [&](const Segment& s) {
        const int buf = it & 1;
        const uint32_t tph = (it >> 1) & 1;
        ++it;
        const bool done = mbar_wait(&tfull[buf], tph, abort_flag, p.wait_ns);
        if (!done) report_abort(abort_flag, p.status);
        if (!bar_epilogue_all(done)) return false;
        tc_fence_after();
        const uint32_t acc = tmem_base + buf * 128 + (static_cast<uint32_t>(q * 32) << 16);
        const int off = act_off[s.j], n = act_off[s.j + 1] - off;
        const int col = s.tile * 128 + row;
        // the segment that starts a tile writes the slots' rows; a later one (a CTA's first) its partial
        float* dst = s.lo == 0 ? p.pbuf + static_cast<int64_t>(off) * p.H + col
                               : p.part2 + static_cast<int64_t>(cta) * p.nt * 128 + row;
        const int64_t pitch = s.lo == 0 ? p.H : 128;
        const bool in = s.lo > 0 || col < p.H;
        for (int s0 = 0; s0 < n; s0 += kChunk) {
          uint32_t r[kChunk];
          tmem_ld_32x32b_x16(acc + s0, r);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < kChunk; ++i) asm volatile("" : "+r"(r[i]));
          if (s0 + kChunk >= n) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&tempty[buf]);
          }
#pragma unroll
          for (int i = 0; i < kChunk; ++i)
            if (in && s0 + i < n) dst[(s0 + i) * pitch] = __uint_as_float(r[i]);
        }
        return true;
      });
  }

  tc_fence_before();
  __syncthreads();
  // ===================== weighted sum =====================
  // An item is 128 columns of 8 / wpt tokens: wpt warps share a token's choices
  // (few tokens would leave warps idle and chain the loads of all choices in
  // one).  Lane i holds the token's choice i: its slot, the slot's row in a
  // partial, the CTAs that its tile is cut between, its weight.  (The first
  // ones are looked up before the barrier.)
  struct Choice {
    int pos, s, c0, c1;
    float w;
  };
  const int wpt = p.T == 1 ? 8 : p.T == 2 ? 4 : p.T <= 4 ? 2 : 1;
  const int tpi = 8 / wpt, sub = warp % wpt;
  const int tiles = f2.tiles, items = tiles * ((p.T + tpi - 1) / tpi);
  auto look_up = [&](int item) {
    Choice c{-1, 0, 0, 0, 0.0f};
    const int tile = item % tiles, t = item / tiles * tpi + warp / wpt;
    if (item < items && t < p.T && lane < p.k) {
      c.pos = p.plan->pos_of[t * p.k + lane];
      const float w = p.w[t * p.k + lane];
      c.w = c.pos >= 0 ? w : 0.0f;  // an absent choice's weight may be anything: 0 times a NaN is one
      if (c.pos >= 0) {
        const int j = p.plan->slot_act[c.pos];
        const int64_t first = (static_cast<int64_t>(j) * tiles + tile) * f2.kb;
        c.s = c.pos - act_off[j];
        c.c0 = f2.owner(first);
        c.c1 = f2.owner(first + f2.kb - 1);
      }
    }
    return c;
  };
  if (tid == 0 && !*abort_flag) red_release_add(&p.plan->grid_bar, 1);
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc(tmem_base, 256);
  }
  Choice ch = look_up(cta);
  if (tid == 0) {
    const bool all = !*abort_flag && wait_count(&p.plan->grid_bar, ctas, abort_flag, p.wait_ns);
    if (!all) report_abort(abort_flag, p.status);
    *flag = all;
  }
  __syncthreads();
  if (!*flag) return;
  for (int item = cta; item < items; item += ctas) {
    const int tile = item % tiles, t = item / tiles * tpi + warp / wpt;
    const int col = tile * 128 + lane * 4;
    float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (t < p.T) {
#pragma unroll 4
      for (int i = sub; i < p.k; i += wpt) {
        const int pi = __shfl_sync(0xffffffffu, ch.pos, i), si = __shfl_sync(0xffffffffu, ch.s, i);
        const int b = __shfl_sync(0xffffffffu, ch.c0, i), e = __shfl_sync(0xffffffffu, ch.c1, i);
        const float wi = __shfl_sync(0xffffffffu, ch.w, i);
        const bool in = pi >= 0 && col < p.H;
        // the tile's first segment, and the partials of up to two more CTAs at once
        const float4 zero = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        const float* more = p.part2 + (static_cast<int64_t>(b) * p.nt + si) * 128 + lane * 4;
        const int64_t pitch = static_cast<int64_t>(p.nt) * 128;
        float4 v = in ? __ldcg(reinterpret_cast<const float4*>(p.pbuf + static_cast<int64_t>(pi) * p.H + col)) : zero;
        const float4 a1 = in && b + 1 <= e ? __ldcg(reinterpret_cast<const float4*>(more + pitch)) : zero;
        const float4 a2 = in && b + 2 <= e ? __ldcg(reinterpret_cast<const float4*>(more + 2 * pitch)) : zero;
        v = add4(add4(v, a1), a2);
        if (in)
          for (int c = b + 3; c <= e; ++c) v = add4(v, __ldcg(reinterpret_cast<const float4*>(more + (c - b) * pitch)));
        sum.x = fmaf(wi, v.x, sum.x);
        sum.y = fmaf(wi, v.y, sum.y);
        sum.z = fmaf(wi, v.z, sum.z);
        sum.w = fmaf(wi, v.w, sum.w);
      }
    }
    if (wpt > 1) {  // add the shares of the token's warps, in order
      float4* share = reinterpret_cast<float4*>(ex);
      __syncthreads();
      share[warp * 32 + lane] = sum;
      __syncthreads();
      if (sub == 0)
        for (int i = 1; i < wpt; ++i) sum = add4(sum, share[(warp + i) * 32 + lane]);
    }
    if (sub == 0 && t < p.T && col < p.H) {  // H % 8 == 0: four columns are all in or all out
      __nv_bfloat162 lo = __floats2bfloat162_rn(sum.x, sum.y), hi = __floats2bfloat162_rn(sum.z, sum.w);
      uint2 o;
      o.x = *reinterpret_cast<uint32_t*>(&lo);
      o.y = *reinterpret_cast<uint32_t*>(&hi);
      *reinterpret_cast<uint2*>(p.y + static_cast<int64_t>(t) * p.H + col) = o;
    }
    if (item + ctas < items) ch = look_up(item + ctas);
  }
}

bool map_bf16(CUtensorMap* m, const void* base, int rank, uint64_t d0, uint64_t d1, uint64_t d2, uint32_t b0,
              uint32_t b1) {
  const uint64_t dims[3] = {d0, d1, d2};
  const uint64_t strides[2] = {d0 * 2, d0 * d1 * 2};
  const uint32_t box[3] = {b0, b1, 1};
  return encode_tmap(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, base, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

constexpr int kTailBytes = kBarBytes + kExBytes + (2 * kMaxE + 4) * 4 + kMaxSlots;

template <bool PG>
gl_status launch_experts(const ExpertParams& prm, const ExpertMaps<PG>& pg, int grid, int smem, cudaStream_t stream) {
  auto kern = experts_kernel<PG>;
  if (set_max_smem(reinterpret_cast<const void*>(kern), smem) != cudaSuccess) return GL_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeCooperative;  // the CTAs wait for one another: all resident, or none
  attr[0].val.cooperative = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, prm, pg) == cudaSuccess ? GL_OK : GL_ERR_CUDA;
}

}  // namespace

int64_t moe_workspace_bytes(int T, int k, int H, int F) {
  return layout_for(T, k, H, F, std::min(num_sms(), kMaxCtas)).bytes;
}

gl_status launch_moe(const MoeCall& c) {
  const int ctas = std::min(num_sms(), kMaxCtas);
  const Layout l = layout_for(c.T, c.k, c.H, c.F, ctas);
  uint8_t* ws = static_cast<uint8_t*>(c.workspace);
  RouteParams r;
  r.x = static_cast<const __nv_bfloat16*>(c.x);
  r.router = static_cast<const __nv_bfloat16*>(c.router);
  r.idx = c.idx;
  r.w = c.w;
  r.status = c.status;
  r.plan = reinterpret_cast<Plan*>(ws);
  r.T = c.T;
  r.E = c.E;
  r.k = c.k;
  r.H = c.H;
  r.renorm = c.renorm;

  ExpertParams p;
  memset(&p, 0, sizeof(p));
  p.plan = r.plan;
  p.status = c.status;
  p.hbuf = reinterpret_cast<__nv_bfloat16*>(ws + l.h);
  p.pbuf = reinterpret_cast<float*>(ws + l.p);
  p.part1 = reinterpret_cast<float*>(ws + l.part1);
  p.part2 = reinterpret_cast<float*>(ws + l.part2);
  p.w = c.w;
  p.y = static_cast<__nv_bfloat16*>(c.y);
  p.T = c.T;
  p.k = c.k;
  p.H = c.H;
  p.F = c.F;
  p.act = act_inner(c.act);
  p.nt = ceil16(c.T);
  const int stage_bytes = kABytes + p.nt * kBK * 2;
  p.stages = std::min(kMaxStages, (232448 - 1024 - kTailBytes) / stage_bytes);
  p.wait_ns = c.wait_ns ? c.wait_ns : kWaitLimitNs;
  p.hold_loads = c.hold_loads;
  const int smem = 1024 + p.stages * stage_bytes + kTailBytes;
  bool ok = map_bf16(&p.x, c.x, 2, c.H, c.T, 1, 64, p.nt) &&
            map_bf16(&p.h, p.hbuf, 2, c.F, static_cast<uint64_t>(c.T) * c.k, 1, 64, 16);
  const bool stacked = c.w1.mode == GL_STACKED && c.w2.mode == GL_STACKED;
  ExpertMaps<true>* pg = nullptr;
  if (stacked) {
    ok = ok && map_bf16(&p.w1, c.w1.base, 3, c.H, c.F, 2ull * c.E, 64, 64) &&
         map_bf16(&p.w2, c.w2.base, 3, c.F, c.H, c.E, 64, 128);
  } else {
    pg = new (std::nothrow) ExpertMaps<true>;
    if (pg == nullptr) return GL_ERR_CUDA;
    memset(pg, 0, sizeof(*pg));
    for (int e = 0; e < c.E && ok; ++e) {
      const int64_t n = static_cast<int64_t>(c.H) * c.F * 2;
      const void* a = c.w1.mode == GL_STACKED ? static_cast<const uint8_t*>(c.w1.base) + 2 * n * e : c.w1.ptrs[e];
      const void* b = c.w2.mode == GL_STACKED ? static_cast<const uint8_t*>(c.w2.base) + n * e : c.w2.ptrs[e];
      ok = map_bf16(&pg->w1[e], a, 3, c.H, c.F, 2, 64, 64) && map_bf16(&pg->w2[e], b, 3, c.F, c.H, 1, 64, 128);
    }
  }
  gl_status st = ok ? GL_OK : GL_ERR_UNSUPPORTED;
  if (ok) {
    const int rsmem = route_smem(c.T, c.E, c.k, c.router != nullptr);
    if (set_max_smem(reinterpret_cast<const void*>(route_kernel), kMaxT * kMaxE * 4) != cudaSuccess) {
      st = GL_ERR_CUDA;
    } else {
      route_kernel<<<kRouteCtas, kRouteThreads, rsmem, c.stream>>>(r);
      if (cudaGetLastError() != cudaSuccess) st = GL_ERR_CUDA;
      else if (stacked) st = launch_experts<false>(p, ExpertMaps<false>{0}, ctas, smem, c.stream);
      else st = launch_experts<true>(p, *pg, ctas, smem, c.stream);
    }
  }
  delete pg;
  return st;
}

}  // namespace gl
