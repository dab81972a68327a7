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
// Bound by HBM: 6-8 bytes per element move and some 20 instructions run.
#include <cuda_bf16.h>

#include <algorithm>

#include "gl_internal.h"

namespace gl {
namespace {

constexpr int kMaxThreads = 1024;  // two vectors a thread: GL_NORM_MAX_COLS = 16384 columns
static_assert(GL_NORM_MAX_COLS == kMaxThreads * 16, "a row fits one block");
constexpr int kWarpRowThreads = 256;  // eight rows per block when a warp takes a row

__device__ __forceinline__ void unpack8(const uint4& w, float (&v)[8]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(u[i] << 16);
    v[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
  uint32_t u[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    u[i] = *reinterpret_cast<uint32_t*>(&h);
  }
  return make_uint4(u[0], u[1], u[2], u[3]);
}

__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
}

// Biased exponent e + 127 of the smallest power of two with amax <= 448 * 2^e.
// 448 = 1.75 * 2^8: the mantissa above 1.75 moves to the next exponent.
__device__ __forceinline__ int e8m0_of(float amax) {
  if (amax == 0.0f) return 127;
  const uint32_t b = __float_as_uint(amax);
  return max(0, static_cast<int>((b + 0x1FFFFFu) >> 23) - 8);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Sum over the threads that share a row.  `part` is one of two buffers used in
// turn, so one barrier per row is enough.
template <bool WARP_ROW>
__device__ __forceinline__ float row_sum(float v, float* part) {
  v = warp_sum(v);
  if (WARP_ROW) return v;
  const int lane = threadIdx.x & 31;
  if (lane == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  return warp_sum(lane < static_cast<int>(blockDim.x >> 5) ? part[lane] : 0.0f);
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

// x, residual and the outputs may be the same buffers: a thread reads all of
// its row's vectors before it writes any, and no other thread touches them.
template <int VPT, bool WARP_ROW, bool MX>
__global__ void __launch_bounds__(WARP_ROW ? kWarpRowThreads : kMaxThreads)
    rmsnorm_kernel(const NormParams p) {
  __shared__ float part[2][32];
  const int tpr = WARP_ROW ? 32 : static_cast<int>(blockDim.x);
  const int t = WARP_ROW ? static_cast<int>(threadIdx.x & 31) : static_cast<int>(threadIdx.x);
  const int rpb = WARP_ROW ? kWarpRowThreads / 32 : 1;
  const int nv = p.cols >> 3;
  int buf = 0;
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * rpb + (WARP_ROW ? (threadIdx.x >> 5) : 0); row < p.rows;
       row += static_cast<int64_t>(gridDim.x) * rpb, buf ^= 1) {
    const int64_t base = row * p.cols;
    float v[VPT][8];
    float ss = 0.0f;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int c = t + j * tpr;
      if (c < nv) {
        unpack8(*reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.x) + base + c * 8), v[j]);
        if (p.residual != nullptr) {
          float r[8];
          unpack8(*reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.residual) + base + c * 8), r);
#pragma unroll
          for (int i = 0; i < 8; ++i) v[j][i] += r[i];
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[j][i] = 0.0f;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fmaf(v[j][i], v[j][i], ss);
    }
    ss = row_sum<WARP_ROW>(ss, part[buf]);
    const float rstd = 1.0f / sqrtf(ss / static_cast<float>(p.cols) + p.eps);
    if (t == 0 && p.rstd != nullptr) p.rstd[row] = rstd;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int c = t + j * tpr;
      const bool in = c < nv;
      if (in && p.sum != nullptr)
        *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.sum) + base + c * 8) = pack8(v[j]);
      float g[8] = {};
      if (in) unpack8(__ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.gamma) + c * 8)), g);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[j][i] = v[j][i] * rstd * g[i];
      if (in && p.y != nullptr)
        *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.y) + base + c * 8) = pack8(v[j]);
      if (MX) {
        float amax = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(v[j][i]));
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        const int e = e8m0_of(amax);
        const float inv = __uint_as_float(static_cast<uint32_t>(254 - e) << 23);  // 2^-(e - 127)
        if (in) {
          uint2 q;
          q.x = e4m3x4(v[j][0] * inv, v[j][1] * inv, v[j][2] * inv, v[j][3] * inv);
          q.y = e4m3x4(v[j][4] * inv, v[j][5] * inv, v[j][6] * inv, v[j][7] * inv);
          *reinterpret_cast<uint2*>(p.codes + base + c * 8) = q;
          if ((c & 3) == 0) {
            const int kb = c >> 2;
            const int64_t at = p.mma_scales ? (static_cast<int64_t>(kb >> 2) * ((p.rows + 127) >> 7) + (row >> 7)) * 512 +
                                                  (row & 31) * 16 + ((row & 127) >> 5) * 4 + (kb & 3)
                                            : row * (p.cols >> 5) + kb;
            p.scales[at] = static_cast<uint8_t>(e);
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

template <int VPT, bool WARP_ROW>
__global__ void __launch_bounds__(WARP_ROW ? kWarpRowThreads : kMaxThreads)
    rmsnorm_bwd_kernel(const NormBwdParams p) {
  __shared__ float part[2][32];
  __shared__ float acc_s[WARP_ROW ? VPT * 256 : 1];
  const int tpr = WARP_ROW ? 32 : static_cast<int>(blockDim.x);
  const int t = WARP_ROW ? static_cast<int>(threadIdx.x & 31) : static_cast<int>(threadIdx.x);
  const int rpb = WARP_ROW ? kWarpRowThreads / 32 : 1;
  const int nv = p.cols >> 3;
  float acc[VPT][8] = {};
  int buf = 0;
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * rpb + (WARP_ROW ? (threadIdx.x >> 5) : 0); row < p.rows;
       row += static_cast<int64_t>(gridDim.x) * rpb, buf ^= 1) {
    const int64_t base = row * p.cols;
    const float rstd = p.rstd[row];
    uint4 dyw[VPT], sw[VPT];
    float dot = 0.0f;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int c = t + j * tpr;
      dyw[j] = sw[j] = make_uint4(0, 0, 0, 0);
      if (c < nv) {
        dyw[j] = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.dy) + base + c * 8);
        sw[j] = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.sum) + base + c * 8);
      }
    }
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int c = t + j * tpr;
      if (c < nv) {
        float d[8], s[8], g[8];
        unpack8(dyw[j], d);
        unpack8(sw[j], s);
        unpack8(__ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.gamma) + c * 8)), g);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float dh = d[i] * (s[i] * rstd);
          acc[j][i] += dh;
          dot = fmaf(dh, g[i], dot);
        }
      }
    }
    dot = row_sum<WARP_ROW>(dot, part[buf]) / static_cast<float>(p.cols);
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int c = t + j * tpr;
      if (c < nv) {
        float d[8], s[8], g[8], r[8] = {};
        unpack8(dyw[j], d);
        unpack8(sw[j], s);
        unpack8(__ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.gamma) + c * 8)), g);
        if (p.dsum != nullptr)
          unpack8(*reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.dsum) + base + c * 8), r);
#pragma unroll
        for (int i = 0; i < 8; ++i) d[i] = rstd * (d[i] * g[i] - (s[i] * rstd) * dot) + r[i];
        *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.dx) + base + c * 8) = pack8(d);
      }
    }
  }
  float* out = p.part + static_cast<int64_t>(blockIdx.x) * p.cols;
  if (WARP_ROW) {  // the block's eight warps hold the same columns: add them in warp order
    for (int w = 0; w < kWarpRowThreads / 32; ++w) {
      if (static_cast<int>(threadIdx.x >> 5) == w) {
#pragma unroll
        for (int j = 0; j < VPT; ++j)
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int at = (t + j * 32) * 8 + i;
            acc_s[at] = (w == 0 ? 0.0f : acc_s[at]) + acc[j][i];
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
        *reinterpret_cast<float4*>(out + c * 8) = make_float4(acc[j][0], acc[j][1], acc[j][2], acc[j][3]);
        *reinterpret_cast<float4*>(out + c * 8 + 4) = make_float4(acc[j][4], acc[j][5], acc[j][6], acc[j][7]);
      }
    }
  }
}

// dgamma[c] (+)= the blocks' partial sums, in a fixed order: eight warps take
// the blocks w, w + 8, ... of 32 columns, then the eight sums are added.
__global__ void __launch_bounds__(256)
    rmsnorm_dgamma_kernel(const float* __restrict__ part, int blocks, int cols, float* __restrict__ dgamma,
                          int accumulate) {
  __shared__ float sm[8][32];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float s = 0.0f;
  if (c < cols)
    for (int b = w; b < blocks; b += 8) s += part[static_cast<int64_t>(b) * cols + c];
  sm[w][lane] = s;
  __syncthreads();
  if (w == 0 && c < cols) {
    s = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) s += sm[i][lane];
    dgamma[c] = accumulate ? dgamma[c] + s : s;
  }
}

struct NormPlan {
  bool warp_row;
  int vpt, threads, rows_per_block;
};

// Rows of up to 1024 columns go to one warp each.  Longer rows take a block of
// two vectors a thread.
NormPlan plan_for(int cols) {
  const int nv = cols >> 3;
  NormPlan pl;
  pl.warp_row = nv <= 128;
  if (pl.warp_row) {
    pl.vpt = nv <= 32 ? 1 : nv <= 64 ? 2 : 4;
    pl.threads = kWarpRowThreads;
    pl.rows_per_block = kWarpRowThreads / 32;
  } else {
    pl.vpt = 2;
    pl.threads = ((nv + pl.vpt - 1) / pl.vpt + 31) / 32 * 32;
    pl.rows_per_block = 1;
  }
  return pl;
}

int blocks_for(const NormPlan& pl, int64_t rows, int threads_per_sm) {
  const int64_t need = (rows + pl.rows_per_block - 1) / pl.rows_per_block;
  const int64_t fit = static_cast<int64_t>(num_sms()) * std::max(1, threads_per_sm / pl.threads);
  return static_cast<int>(std::min(need, fit));
}

template <bool MX>
void launch_fwd(const NormPlan& pl, int grid, const NormParams& p, cudaStream_t s) {
  if (pl.warp_row) {
    if (pl.vpt == 1) rmsnorm_kernel<1, true, MX><<<grid, pl.threads, 0, s>>>(p);
    else if (pl.vpt == 2) rmsnorm_kernel<2, true, MX><<<grid, pl.threads, 0, s>>>(p);
    else rmsnorm_kernel<4, true, MX><<<grid, pl.threads, 0, s>>>(p);
  } else {
    rmsnorm_kernel<2, false, MX><<<grid, pl.threads, 0, s>>>(p);
  }
}

constexpr int kFwdThreadsPerSm = 2048;
constexpr int kBwdThreadsPerSm = 1024;

}  // namespace

gl_status launch_rmsnorm(const void* x, const void* residual, const void* gamma, float eps, int64_t rows, int cols,
                         void* sum, void* y, float* rstd, uint8_t* codes, uint8_t* scales, int scale_layout,
                         cudaStream_t stream) {
  const NormPlan pl = plan_for(cols);
  NormParams p{x, residual, gamma, eps, rows, cols, sum, y, rstd, codes, scales, scale_layout == GL_SCALES_MMA};
  const int grid = blocks_for(pl, rows, kFwdThreadsPerSm);
  if (codes != nullptr) launch_fwd<true>(pl, grid, p, stream);
  else launch_fwd<false>(pl, grid, p, stream);
  return cudaGetLastError() == cudaSuccess ? GL_OK : GL_ERR_CUDA;
}

int64_t rmsnorm_bwd_blocks(int64_t rows, int cols) { return blocks_for(plan_for(cols), rows, kBwdThreadsPerSm); }

gl_status launch_rmsnorm_bwd(const void* dy, const void* sum, const void* gamma, const float* rstd, const void* dsum,
                             int64_t rows, int cols, void* dx, float* dgamma, int accumulate, float* part,
                             cudaStream_t stream) {
  const NormPlan pl = plan_for(cols);
  const int grid = static_cast<int>(rmsnorm_bwd_blocks(rows, cols));
  NormBwdParams p{dy, sum, gamma, rstd, dsum, rows, cols, dx, part};
  if (grid > 0) {
    if (pl.warp_row) {
      if (pl.vpt == 1) rmsnorm_bwd_kernel<1, true><<<grid, pl.threads, 0, stream>>>(p);
      else if (pl.vpt == 2) rmsnorm_bwd_kernel<2, true><<<grid, pl.threads, 0, stream>>>(p);
      else rmsnorm_bwd_kernel<4, true><<<grid, pl.threads, 0, stream>>>(p);
    } else {
      rmsnorm_bwd_kernel<2, false><<<grid, pl.threads, 0, stream>>>(p);
    }
    if (cudaGetLastError() != cudaSuccess) return GL_ERR_CUDA;
  }
  rmsnorm_dgamma_kernel<<<(cols + 31) / 32, 256, 0, stream>>>(part, grid, cols, dgamma, accumulate);
  return cudaGetLastError() == cudaSuccess ? GL_OK : GL_ERR_CUDA;
}

}  // namespace gl
