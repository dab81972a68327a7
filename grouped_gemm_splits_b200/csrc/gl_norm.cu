// gl_norm.cu -- root-mean-square norm with the residual's addition, bf16 and /
// or MXFP8 output, and its backward pass.
//
// Forward, per row of n columns (all in fp32 from bf16 inputs):
//   s = x (+ residual),  rstd = 1 / sqrt(sum(s^2) / n + eps),  y = s * rstd * gamma
// and s, y (bf16), rstd (fp32) and the MXFP8 form of y are written, each value
// rounded once: the codes come from the fp32 y, not from its bf16 copy, and
// the norm is taken of the fp32 sum, not of its bf16 copy.
//
// Backward, with xh = s * rstd and g = dy * gamma:
//   dx = rstd * (g - xh * mean(g * xh)) (+ dsum),  dgamma[c] (+)= sum over rows of dy * xh
//
// One row is held in registers by one block (or by one warp when it is short),
// so every input is read once.  A thread owns the 8-column vectors tid,
// tid + threads, ...: four neighbouring lanes hold one 32-column MXFP8 block.
//
// Bound by HBM: 6-8 bytes per element move.  Each thread copies its own
// vectors of the rows to come into its own places of a shared-memory ring
// (cp.async) and reads them back itself, so loads are in flight whatever the
// block is doing and the ring needs no barrier; with the loads at the head of
// each row instead, 65536 x 7168 to MXFP8 ran 810 us (47% of HBM, warps waiting
// for loads).  The arithmetic is done on pairs of columns (f32x2
// instructions), gamma stays in registers.
//
// How much is in flight: enough threads for the arithmetic (768-1024 per SM)
// and no more rows than that takes.  More blocks or a deeper ring make reads
// and writes meet in DRAM: 32768 x 4096 to MXFP8 took 147 us with two blocks of
// 512 and two rows each in flight, 155 us with three rows, 179 us with four
// blocks of 256 (two vectors a thread) and three rows; the floor is 144 us.
// Without a residual the same threads have one tensor to load, and a row's two
// reductions are what they wait for: two rows a turn share them, and the ring
// holds twice the rows (16384 x 7168 to bf16: 74 us, with one row a turn 98, with
// the shorter ring 103; floor 72.  To MXFP8 90 us of 54: 76% of the issue slots are taken).
// Measured with it: 65536 x 7168 to MXFP8 511 us (floor 504), to bf16 571
// (574); 32768 x 2048 81 (72) and 88 (82); backward 32768 x 4096 164 (164).
#include <cuda_bf16.h>

#include <algorithm>

#include "gl_internal.h"
#include "gl_ptx.cuh"

namespace gl {
namespace {

constexpr int kMaxThreads = 1024;  // two vectors a thread: GL_NORM_MAX_COLS = 16384 columns
static_assert(GL_NORM_MAX_COLS == kMaxThreads * 16, "a row fits one block");
constexpr int kWarpRowThreads = 256;  // eight rows per block when a warp takes a row
constexpr int kWarpRowCols = 256;     // up to here: one vector a lane

// ------------------------------------------------------- pairs of fp32 values
typedef uint64_t f2;
__device__ __forceinline__ f2 f2_make(float a, float b) {
  f2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 f2_get(f2 v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ f2 f2_add(f2 a, f2 b) {
  f2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f2 f2_mul(f2 a, f2 b) {
  f2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f2 f2_fma(f2 a, f2 b, f2 c) {
  f2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
// two bf16 values
__device__ __forceinline__ f2 f2_of_bf16(uint32_t w) {
  return f2_make(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
__device__ __forceinline__ uint32_t bf16_of_f2(f2 v) {
  const float2 t = f2_get(v);
  __nv_bfloat162 h = __floats2bfloat162_rn(t.x, t.y);
  return *reinterpret_cast<uint32_t*>(&h);
}

// One vector: eight bf16 values, or four pairs.
struct Words {
  uint32_t w[4];
};
__device__ __forceinline__ Words words(const uint4& v) { return Words{{v.x, v.y, v.z, v.w}}; }
__device__ __forceinline__ uint4 pack_vec(const f2 (&v)[4]) {
  return make_uint4(bf16_of_f2(v[0]), bf16_of_f2(v[1]), bf16_of_f2(v[2]), bf16_of_f2(v[3]));
}

__device__ __forceinline__ uint32_t e4m3x4(f2 a, f2 b) {
  const float2 u = f2_get(a), v = f2_get(b);
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(u.y), "f"(u.x));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(v.y), "f"(v.x));
  return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
}

// Biased exponent e + 127 of the smallest power of two with amax <= 448 * 2^e.
// 448 = 1.75 * 2^8: the mantissa above 1.75 moves to the next exponent.
__device__ __forceinline__ int e8m0_of(float amax) {
  if (amax == 0.0f) return 127;
  const uint32_t b = __float_as_uint(amax);
  return max(0, static_cast<int>((b + 0x1FFFFFu) >> 23) - 8);
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// 1 / sqrt(a): rsqrtf and one Newton step, a dozen instructions fewer in every
// thread than a square root and a division.  Zero and infinity stay rsqrtf's.
__device__ __forceinline__ float inv_sqrt(float a) {
  const float r = rsqrtf(a), e = fmaf(-a * r, r, 1.0f);
  return fabsf(e) < 1.0f ? fmaf(0.5f * r, e, r) : r;
}

// Sums over the threads that share a row, of N rows at once.  `part` is one of
// two buffers used in turn, so one barrier per turn is enough.
template <bool WARP_ROW, int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float (*part)[32]) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = warp_sum(v[i]);
  if (WARP_ROW) return;
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (lane == 0) part[i][threadIdx.x >> 5] = v[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = warp_sum(lane < static_cast<int>(blockDim.x >> 5) ? part[i][lane] : 0.0f);
}

template <bool WARP_ROW>
__device__ __forceinline__ float row_sum(float v, float* part) {
  float a[1] = {v};
  row_sums<WARP_ROW>(a, reinterpret_cast<float(*)[32]>(part));
  return a[0];
}

struct NormParams {
  const void* x;
  const void* residual;
  const void* gamma;
  float eps;
  int64_t rows;
  int cols;
  void* sum;
  void* y;
  float* rstd;
  uint8_t* codes;
  uint8_t* scales;
  int mma_scales;
};

// The ring: TENSORS tensors x DEPTH rows, one 16-byte place per thread and
// vector.  A thread refills a place only after it has used what it read there.
template <int VPT, int TENSORS, int DEPTH>
struct Ring {
  uint32_t base;  // this thread's first place
  uint32_t pitch;  // bytes from one vector of the block to the next
  __device__ __forceinline__ uint32_t place(int slot, int tensor, int j) const {
    return base + ((slot * TENSORS + tensor) * VPT + j) * pitch;
  }
  static constexpr int bytes(int threads) { return DEPTH * TENSORS * VPT * threads * 16; }
};

// x, residual and the outputs may be the same buffers: a thread has read all
// of its row's vectors before it writes any, and no other thread touches them.
template <int VPT, bool WARP_ROW, bool MX, bool RES, int ROWS, int DEPTH>
__global__ void __launch_bounds__(WARP_ROW ? kWarpRowThreads : kMaxThreads)
    rmsnorm_kernel(const NormParams p) {
  extern __shared__ __align__(16) uint8_t ring_s[];
  __shared__ float part[2][ROWS][32];
  const int tpr = WARP_ROW ? 32 : static_cast<int>(blockDim.x);
  const int t = WARP_ROW ? static_cast<int>(threadIdx.x & 31) : static_cast<int>(threadIdx.x);
  const int rpb = WARP_ROW ? kWarpRowThreads / 32 : 1;
  const int nv = p.cols >> 3;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * rpb;
  const int64_t row0 = static_cast<int64_t>(blockIdx.x) * rpb + (WARP_ROW ? (threadIdx.x >> 5) : 0);
  const Ring<VPT, RES ? 2 : 1, DEPTH> ring{smem_u32(ring_s) + threadIdx.x * 16, blockDim.x * 16};
  const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(p.x);
  const __nv_bfloat16* res = static_cast<const __nv_bfloat16*>(p.residual);
  auto fetch = [&](int64_t row, int slot) {
    if (row < p.rows) {
#pragma unroll
      for (int j = 0; j < VPT; ++j) {
        const int c = t + j * tpr;
        if (c < nv) {
          const int64_t at = row * p.cols + c * 8;
          cp_async16(ring.place(slot, 0, j), x + at);
          if (RES) cp_async16(ring.place(slot, 1, j), res + at);
        }
      }
    }
    cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < DEPTH; ++i) fetch(row0 + i * stride, i);
  f2 g[VPT][4];
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int c = t + j * tpr;
    const Words w = words(c < nv ? __ldg(reinterpret_cast<const uint4*>(p.gamma) + c) : make_uint4(0, 0, 0, 0));
#pragma unroll
    for (int i = 0; i < 4; ++i) g[j][i] = f2_of_bf16(w.w[i]);
  }
  const float inv_n = 1.0f / static_cast<float>(p.cols);
  const int64_t atoms = (p.rows + 127) >> 7;  // MMA layout: atoms per k-group
  int slot = 0, buf = 0;
  for (int64_t turn = row0; turn < p.rows; turn += ROWS * stride, buf ^= 1) {
    f2 v[ROWS][VPT][4];
    float sum[ROWS];
    cp_async_wait<DEPTH - ROWS>();
#pragma unroll
    for (int n = 0; n < ROWS; ++n) {  // behind the last row: what the place holds, for no output
      f2 ss = 0;
#pragma unroll
      for (int j = 0; j < VPT; ++j) {
        if (t + j * tpr < nv) {
          const Words a = words(lds16(ring.place(slot + n, 0, j)));
#pragma unroll
          for (int i = 0; i < 4; ++i) v[n][j][i] = f2_of_bf16(a.w[i]);
          if (RES) {
            const Words r = words(lds16(ring.place(slot + n, 1, j)));
#pragma unroll
            for (int i = 0; i < 4; ++i) v[n][j][i] = f2_add(v[n][j][i], f2_of_bf16(r.w[i]));
          }
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) v[n][j][i] = 0;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) ss = f2_fma(v[n][j][i], v[n][j][i], ss);
      }
      const float2 s2 = f2_get(ss);
      sum[n] = s2.x + s2.y;
    }
    row_sums<WARP_ROW>(sum, part[buf]);
#pragma unroll
    for (int n = 0; n < ROWS; ++n) fetch(turn + (DEPTH + n) * stride, slot + n);
    slot = slot + ROWS == DEPTH ? 0 : slot + ROWS;
#pragma unroll
    for (int n = 0; n < ROWS; ++n) {
      const int64_t row = turn + n * stride;
      if (n > 0 && row >= p.rows) break;
      const int64_t base = row * p.cols;
      const float rstd = inv_sqrt(fmaf(sum[n], inv_n, p.eps));
      if (t == 0 && p.rstd != nullptr) p.rstd[row] = rstd;
      const f2 rr = f2_make(rstd, rstd);
      const int64_t srow = !MX ? 0 : p.mma_scales ? (row >> 7) * 512 + (row & 31) * 16 + ((row & 127) >> 5) * 4
                                                  : row * (p.cols >> 5);
#pragma unroll
      for (int j = 0; j < VPT; ++j) {
        const int c = t + j * tpr;
        const bool in = c < nv;
        f2(&u)[4] = v[n][j];
        if (in && p.sum != nullptr)
          __stcs(reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.sum) + base + c * 8), pack_vec(u));
#pragma unroll
        for (int i = 0; i < 4; ++i) u[i] = f2_mul(f2_mul(u[i], rr), g[j][i]);
        if (in && p.y != nullptr)
          __stcs(reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.y) + base + c * 8), pack_vec(u));
        if (MX) {
          float amax = 0.0f;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 w = f2_get(u[i]);
            amax = fmaxf(amax, fmaxf(fabsf(w.x), fabsf(w.y)));
          }
          amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
          amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
          const int e = e8m0_of(amax);
          const float inv = __uint_as_float(static_cast<uint32_t>(254 - e) << 23);  // 2^-(e - 127)
          const f2 ii = f2_make(inv, inv);
          if (in) {
            const uint2 q = make_uint2(e4m3x4(f2_mul(u[0], ii), f2_mul(u[1], ii)),
                                       e4m3x4(f2_mul(u[2], ii), f2_mul(u[3], ii)));
            __stcs(reinterpret_cast<uint2*>(p.codes + base + c * 8), q);
            if ((c & 3) == 0) {
              const int kb = c >> 2;
              p.scales[srow + (p.mma_scales ? static_cast<int64_t>(kb >> 2) * atoms * 512 + (kb & 3) : kb)] =
                  static_cast<uint8_t>(e);
            }
          }
        }
      }
    }
  }
}

struct NormBwdParams {
  const void* dy;
  const void* sum;
  const void* gamma;
  const float* rstd;
  const void* dsum;
  int64_t rows;
  int cols;
  void* dx;
  float* part;  // [grid, cols] sums of dy * xh over a block's rows
};

template <int VPT, bool WARP_ROW, int DEPTH>
__global__ void __launch_bounds__(WARP_ROW ? kWarpRowThreads : kMaxThreads)
    rmsnorm_bwd_kernel(const NormBwdParams p) {
  extern __shared__ __align__(16) uint8_t ring_s[];
  __shared__ float part[2][32];
  __shared__ __align__(16) float acc_s[WARP_ROW ? VPT * 256 : 4];
  const int tpr = WARP_ROW ? 32 : static_cast<int>(blockDim.x);
  const int t = WARP_ROW ? static_cast<int>(threadIdx.x & 31) : static_cast<int>(threadIdx.x);
  const int rpb = WARP_ROW ? kWarpRowThreads / 32 : 1;
  const int nv = p.cols >> 3;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * rpb;
  const int64_t row0 = static_cast<int64_t>(blockIdx.x) * rpb + (WARP_ROW ? (threadIdx.x >> 5) : 0);
  const Ring<VPT, 3, DEPTH> ring{smem_u32(ring_s) + threadIdx.x * 16, blockDim.x * 16};
  const __nv_bfloat16* dy = static_cast<const __nv_bfloat16*>(p.dy);
  const __nv_bfloat16* sum = static_cast<const __nv_bfloat16*>(p.sum);
  const __nv_bfloat16* dsum = static_cast<const __nv_bfloat16*>(p.dsum);
  auto fetch = [&](int64_t row, int slot) {
    if (row < p.rows) {
#pragma unroll
      for (int j = 0; j < VPT; ++j) {
        const int c = t + j * tpr;
        if (c < nv) {
          const int64_t at = row * p.cols + c * 8;
          cp_async16(ring.place(slot, 0, j), dy + at);
          cp_async16(ring.place(slot, 1, j), sum + at);
          if (dsum != nullptr) cp_async16(ring.place(slot, 2, j), dsum + at);
        }
      }
    }
    cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < DEPTH; ++i) fetch(row0 + i * stride, i);
  Words g[VPT];
  f2 acc[VPT][4];
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int c = t + j * tpr;
    g[j] = words(c < nv ? __ldg(reinterpret_cast<const uint4*>(p.gamma) + c) : make_uint4(0, 0, 0, 0));
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[j][i] = 0;
  }
  const float inv_n = 1.0f / static_cast<float>(p.cols);
  float next_rstd = row0 < p.rows ? __ldg(p.rstd + row0) : 0.0f;
  int slot = 0, buf = 0;
  for (int64_t row = row0; row < p.rows; row += stride, buf ^= 1) {
    const int64_t base = row * p.cols;
    const float rstd = next_rstd;
    if (row + stride < p.rows) next_rstd = __ldg(p.rstd + row + stride);
    const f2 rr = f2_make(rstd, rstd);
    f2 dot2 = 0;
    cp_async_wait<DEPTH - 1>();
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      if (t + j * tpr < nv) {
        const Words d = words(lds16(ring.place(slot, 0, j))), x = words(lds16(ring.place(slot, 1, j)));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const f2 dh = f2_mul(f2_of_bf16(d.w[i]), f2_mul(f2_of_bf16(x.w[i]), rr));
          acc[j][i] = f2_add(acc[j][i], dh);
          dot2 = f2_fma(dh, f2_of_bf16(g[j].w[i]), dot2);
        }
      }
    }
    const float2 d2 = f2_get(dot2);
    const float dot = row_sum<WARP_ROW>(d2.x + d2.y, part[buf]) * inv_n;
    // dx = rstd * (dy gamma - s rstd dot) + dsum; the row is read a second time
    // from the ring (keeping it in registers would halve the threads per SM)
    const f2 md = f2_make(-dot * rstd, -dot * rstd);
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int c = t + j * tpr;
      if (c < nv) {
        const Words d = words(lds16(ring.place(slot, 0, j))), x = words(lds16(ring.place(slot, 1, j)));
        const Words e = words(dsum != nullptr ? lds16(ring.place(slot, 2, j)) : make_uint4(0, 0, 0, 0));
        f2 o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const f2 gd = f2_mul(f2_of_bf16(d.w[i]), f2_of_bf16(g[j].w[i]));
          o[i] = f2_fma(f2_fma(f2_of_bf16(x.w[i]), md, gd), rr, f2_of_bf16(e.w[i]));
        }
        __stcs(reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.dx) + base + c * 8), pack_vec(o));
      }
    }
    fetch(row + DEPTH * stride, slot);
    slot = slot + 1 == DEPTH ? 0 : slot + 1;
  }
  grid_launch_dependents();
  float* out = p.part + static_cast<int64_t>(blockIdx.x) * p.cols;
  if (WARP_ROW) {  // the block's eight warps hold the same columns: add them in warp order
    for (int w = 0; w < kWarpRowThreads / 32; ++w) {
      if (static_cast<int>(threadIdx.x >> 5) == w) {
#pragma unroll
        for (int j = 0; j < VPT; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            f2* at = reinterpret_cast<f2*>(acc_s) + (t + j * 32) * 4 + i;
            *at = w == 0 ? acc[j][i] : f2_add(*at, acc[j][i]);
          }
      }
      __syncthreads();
    }
    for (int c = threadIdx.x; c < p.cols; c += kWarpRowThreads) out[c] = acc_s[c];
  } else {
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int c = t + j * tpr;
      if (c < nv) {
        *reinterpret_cast<ulonglong2*>(out + c * 8) = make_ulonglong2(acc[j][0], acc[j][1]);
        *reinterpret_cast<ulonglong2*>(out + c * 8 + 4) = make_ulonglong2(acc[j][2], acc[j][3]);
      }
    }
  }
}

// dgamma[c] (+)= the blocks' partial sums, in a fixed order: 32 warps take the
// blocks w, w + 32, ... of 32 columns, four at a time, then the 32 sums are
// added.
constexpr int kDgThreads = 1024;
__global__ void __launch_bounds__(kDgThreads)
    rmsnorm_dgamma_kernel(const float* __restrict__ part, int blocks, int cols, float* __restrict__ dgamma,
                          int accumulate) {
  __shared__ float sm[32][33];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  const float old = (w == 0 && c < cols && accumulate) ? dgamma[c] : 0.0f;
  float s = 0.0f;
  grid_dependency_wait();
  if (c < cols) {
    int b = w;
    for (; b + 96 < blocks; b += 128) {
      float v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = part[static_cast<int64_t>(b + 32 * i) * cols + c];
      s += (v[0] + v[1]) + (v[2] + v[3]);
    }
    for (; b < blocks; b += 32) s += part[static_cast<int64_t>(b) * cols + c];
  }
  sm[w][lane] = s;
  __syncthreads();
  s = warp_sum(sm[lane][w]);  // warp w: the sums of column w
  __syncthreads();
  if (lane == 0) sm[0][w] = s;
  __syncthreads();
  if (w == 0 && c < cols) dgamma[c] = old + sm[0][lane];
}

struct NormPlan {
  bool warp_row;
  int vpt, threads, rows_per_block;
};

// Short rows go to one warp each, up to 8192 columns to a block of one vector
// a thread (two or four vectors were slower at every width: fewer threads per
// row in flight), wider ones to a block of two.
NormPlan plan_for(int cols) {
  const int nv = cols >> 3;
  NormPlan pl;
  pl.warp_row = cols <= kWarpRowCols;
  pl.vpt = nv <= kMaxThreads ? 1 : 2;
  pl.threads = pl.warp_row ? kWarpRowThreads : ((nv + pl.vpt - 1) / pl.vpt + 31) / 32 * 32;
  pl.rows_per_block = pl.warp_row ? kWarpRowThreads / 32 : 1;
  return pl;
}

// Blocks of one wave.  Forward: 768 threads per SM of the small blocks, up to
// 1024 of the larger; backward (more arithmetic, three reads to one write): 1024.
int per_sm(const NormPlan& pl, bool backward) {
  return std::max(1, (backward || pl.threads > 256 ? 1024 : 768) / pl.threads);
}
int blocks_for(const NormPlan& pl, int64_t rows, bool backward) {
  const int64_t need = (rows + pl.rows_per_block - 1) / pl.rows_per_block;
  return static_cast<int>(std::min<int64_t>(need, static_cast<int64_t>(num_sms()) * per_sm(pl, backward)));
}

template <int VPT, bool WARP_ROW, bool MX, bool RES, int ROWS, int DEPTH>
gl_status run_fwd(const NormPlan& pl, int grid, const NormParams& p, cudaStream_t s) {
  auto kern = rmsnorm_kernel<VPT, WARP_ROW, MX, RES, ROWS, DEPTH>;
  const int smem = Ring<VPT, RES ? 2 : 1, DEPTH>::bytes(pl.threads);
  if (set_max_smem(reinterpret_cast<const void*>(kern), smem) != cudaSuccess) return GL_ERR_CUDA;
  kern<<<grid, pl.threads, smem, s>>>(p);
  return cudaGetLastError() == cudaSuccess ? GL_OK : GL_ERR_CUDA;
}

// Two rows in flight per block, three where an SM holds one block only; without
// a residual twice that, for the same bytes, and two rows a turn (rows of two
// vectors a thread stay at three: 8192 x 12288 took 68 us with them, 73 with six).
template <bool MX, bool RES>
gl_status launch_fwd(const NormPlan& pl, int grid, const NormParams& p, cudaStream_t s) {
  constexpr int R = RES ? 1 : 2;
  if (pl.warp_row) return run_fwd<1, true, MX, RES, R, 2 * R>(pl, grid, p, s);
  if (pl.vpt == 2) return run_fwd<2, false, MX, RES, 1, 3>(pl, grid, p, s);
  return per_sm(pl, false) > 1 ? run_fwd<1, false, MX, RES, R, 2 * R>(pl, grid, p, s)
                               : run_fwd<1, false, MX, RES, R, 3 * R>(pl, grid, p, s);
}

template <int VPT, bool WARP_ROW>
gl_status run_bwd(const NormPlan& pl, int grid, const NormBwdParams& p, cudaStream_t s) {
  constexpr int kDepth = 2;
  auto kern = rmsnorm_bwd_kernel<VPT, WARP_ROW, kDepth>;
  const int smem = Ring<VPT, 3, kDepth>::bytes(pl.threads);
  if (set_max_smem(reinterpret_cast<const void*>(kern), smem) != cudaSuccess) return GL_ERR_CUDA;
  kern<<<grid, pl.threads, smem, s>>>(p);
  return cudaGetLastError() == cudaSuccess ? GL_OK : GL_ERR_CUDA;
}

}  // namespace

gl_status launch_rmsnorm(const void* x, const void* residual, const void* gamma, float eps, int64_t rows, int cols,
                         void* sum, void* y, float* rstd, uint8_t* codes, uint8_t* scales, int scale_layout,
                         cudaStream_t stream) {
  const NormPlan pl = plan_for(cols);
  NormParams p{x, residual, gamma, eps, rows, cols, sum, y, rstd, codes, scales, scale_layout == GL_SCALES_MMA};
  const int grid = blocks_for(pl, rows, false);
  if (residual != nullptr)
    return codes != nullptr ? launch_fwd<true, true>(pl, grid, p, stream) : launch_fwd<false, true>(pl, grid, p, stream);
  return codes != nullptr ? launch_fwd<true, false>(pl, grid, p, stream) : launch_fwd<false, false>(pl, grid, p, stream);
}

int64_t rmsnorm_bwd_blocks(int64_t rows, int cols) { return blocks_for(plan_for(cols), rows, true); }

gl_status launch_rmsnorm_bwd(const void* dy, const void* sum, const void* gamma, const float* rstd, const void* dsum,
                             int64_t rows, int cols, void* dx, float* dgamma, int accumulate, float* part,
                             cudaStream_t stream) {
  const NormPlan pl = plan_for(cols);
  const int grid = static_cast<int>(rmsnorm_bwd_blocks(rows, cols));
  NormBwdParams p{dy, sum, gamma, rstd, dsum, rows, cols, dx, part};
  if (grid > 0) {
    const gl_status st = pl.warp_row ? run_bwd<1, true>(pl, grid, p, stream)
                         : pl.vpt == 1 ? run_bwd<1, false>(pl, grid, p, stream)
                                       : run_bwd<2, false>(pl, grid, p, stream);
    if (st != GL_OK) return st;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((cols + 31) / 32);
  cfg.blockDim = dim3(kDgThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];  // its blocks may start while the last of the rows are worked on
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = grid > 0;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, rmsnorm_dgamma_kernel, static_cast<const float*>(part), grid, cols, dgamma,
                            accumulate) == cudaSuccess
             ? GL_OK
             : GL_ERR_CUDA;
}

}  // namespace gl
