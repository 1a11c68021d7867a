// Layer norm over the rows of the residual stream, in front of the block's projections, and its
// backward pass.
//
// Forward, per row of D channels: h = x + residual (rounded to the element type, so that the stored
// row is the one that is normalised), mean = sum h / D, rstd = 1 / sqrt(sum (h - mean)^2 / D + eps),
// y = (h - mean) rstd g + b; h's 8-bit checkpoint in the same pass.
// Backward, with xh = (h - mean) rstd and e = dy g: dx = rstd (e - mean(e) - xh mean(e xh)) + dh,
// dg = sum over rows of dy xh, db = sum over rows of dy.
//
// Both are HBM-bound streams.  A row is held in the registers of one block, NE values per thread, so
// it is read once; the statistics are two sums over the block, the variance taken about the mean.
#include <algorithm>

#include "act8.cuh"

namespace gdn2 {
namespace {

constexpr int NE = 16;  // values per thread and row: 512 threads hold LN_MAX_WIDTH of them
static_assert(512 * NE == LN_MAX_WIDTH, "a block holds the widest row");

// Threads of a block for a row: whole warps, so that every group of 32 channels lies in one warp.
int row_threads(int width) { return std::max(1, (width + 32 * NE - 1) / (32 * NE)) * 32; }

// Sums of `a` and `b` over the block, in a fixed order; `red` is one of two buffers used in turn, so
// one barrier is enough.
__device__ __forceinline__ void block_sum2(float &a, float &b, float2 *red) {
  a = warp_allreduce_sum(a);
  b = warp_allreduce_sum(b);
  if (blockDim.x == 32) return;
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = make_float2(a, b);
  __syncthreads();
  a = b = 0.f;
  for (int w = 0; w < (int)blockDim.x / 32; ++w) {
    a += red[w].x;
    b += red[w].y;
  }
}

template <typename T, int VEC>
__global__ void __launch_bounds__(512) norm_fwd_kernel(const NormFwdArgs a) {
  constexpr int NV = NE / VEC;
  __shared__ float2 red[2][16];
  const int D = a.width, groups = (D + ACT_GROUP - 1) / ACT_GROUP;
  const float inv_d = 1.f / (float)D;
  for (long long row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const size_t base = (size_t)row * D;
    LaneVec<T, VEC> rx[NV], rr[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = (v * blockDim.x + threadIdx.x) * VEC;
      if (c < D) {
        rx[v] = *reinterpret_cast<const LaneVec<T, VEC> *>(static_cast<const T *>(a.x) + base + c);
        if (a.residual) rr[v] = *reinterpret_cast<const LaneVec<T, VEC> *>(static_cast<const T *>(a.residual) + base + c);
      }
    }
    float f[NV][VEC], sum = 0.f, sq = 0.f, none = 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = (v * blockDim.x + threadIdx.x) * VEC;
      if (c < D) {
        widen(rx[v], f[v]);
        if (a.residual) {
          float r[VEC];
          widen(rr[v], r);
#pragma unroll
          for (int i = 0; i < VEC; ++i) f[v][i] += r[i];
          narrow(f[v], rx[v]);
          *reinterpret_cast<LaneVec<T, VEC> *>(static_cast<T *>(a.h) + base + c) = rx[v];
          widen(rx[v], f[v]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) f[v][i] = 0.f;
      }
#pragma unroll
      for (int i = 0; i < VEC; ++i) sum += f[v][i];
    }
    if (a.codes) {
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int c = (v * blockDim.x + threadIdx.x) * VEC;
        uint32_t s;
        const LaneVec<int8_t, VEC> q = act8_encode<VEC>(f[v], s);
        if (c < D) {
          *reinterpret_cast<LaneVec<int8_t, VEC> *>(a.codes + base + c) = q;
          if (c % ACT_GROUP == 0) a.scales[(size_t)row * groups + c / ACT_GROUP] = (uint8_t)s;
        }
      }
    }
    block_sum2(sum, none, red[0]);
    const float mean = sum * inv_d;
#pragma unroll
    for (int v = 0; v < NV; ++v)
      if ((v * blockDim.x + threadIdx.x) * VEC < D)
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          f[v][i] -= mean;
          sq = fmaf(f[v][i], f[v][i], sq);
        }
    block_sum2(sq, none, red[1]);
    const float rstd = 1.f / sqrtf(sq * inv_d + a.eps);
    if (threadIdx.x == 0 && a.mean) {
      a.mean[row] = mean;
      a.rstd[row] = rstd;
    }
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = (v * blockDim.x + threadIdx.x) * VEC;
      if (c < D) {
        float p[VEC];
        load_f32(a.weight + c, p);
#pragma unroll
        for (int i = 0; i < VEC; ++i) f[v][i] *= rstd * p[i];
        if (a.bias) {
          load_f32(a.bias + c, p);
#pragma unroll
          for (int i = 0; i < VEC; ++i) f[v][i] += p[i];
        }
        narrow(f[v], rx[v]);
        *reinterpret_cast<LaneVec<T, VEC> *>(static_cast<T *>(a.y) + base + c) = rx[v];
      }
    }
  }
}

// One row of partial sums per block in `parts`: [gridDim.x][2][D] (dweight, dbias).
template <typename T, typename S, int VEC>
__global__ void __launch_bounds__(512) norm_bwd_kernel(const NormBwdArgs a, float *parts) {
  constexpr int NV = NE / VEC;
  constexpr bool Q = sizeof(S) == 1;  // h is held in 8 bits
  __shared__ float2 red[2][16];
  const int D = a.width, groups = (D + ACT_GROUP - 1) / ACT_GROUP;
  const float inv_d = 1.f / (float)D;
  float g[NV][VEC], dg[NV][VEC], db[NV][VEC];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int c = (v * blockDim.x + threadIdx.x) * VEC;
#pragma unroll
    for (int i = 0; i < VEC; ++i) g[v][i] = dg[v][i] = db[v][i] = 0.f;
    if (c < D) load_f32(a.weight + c, g[v]);
  }
  int turn = 0;
  for (long long row = blockIdx.x; row < a.rows; row += gridDim.x, turn ^= 1) {
    const size_t base = (size_t)row * D;
    const float mean = a.mean[row], rstd = a.rstd[row];
    LaneVec<T, VEC> ry[NV], rh[NV];
    LaneVec<S, VEC> rs[NV];
    float unit[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = (v * blockDim.x + threadIdx.x) * VEC;
      if (c < D) {
        ry[v] = *reinterpret_cast<const LaneVec<T, VEC> *>(static_cast<const T *>(a.dy) + base + c);
        rs[v] = *reinterpret_cast<const LaneVec<S, VEC> *>(static_cast<const S *>(a.h) + base + c);
        if (Q) unit[v] = act8_unit(a.scales[(size_t)row * groups + c / ACT_GROUP]);
        if (a.dh) rh[v] = *reinterpret_cast<const LaneVec<T, VEC> *>(static_cast<const T *>(a.dh) + base + c);
      }
    }
    float xh[NV][VEC], e[NV][VEC], s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v)
      if ((v * blockDim.x + threadIdx.x) * VEC < D) {
        if constexpr (Q) widen(rs[v], unit[v], xh[v]);
        else widen(rs[v], xh[v]);
        widen(ry[v], e[v]);
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          xh[v][i] = (xh[v][i] - mean) * rstd;
          dg[v][i] = fmaf(e[v][i], xh[v][i], dg[v][i]);
          db[v][i] += e[v][i];
          e[v][i] *= g[v][i];
          s1 += e[v][i];
          s2 = fmaf(e[v][i], xh[v][i], s2);
        }
      }
    block_sum2(s1, s2, red[turn]);
    s1 *= inv_d;
    s2 *= inv_d;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = (v * blockDim.x + threadIdx.x) * VEC;
      if (c < D) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) e[v][i] = rstd * (e[v][i] - s1 - xh[v][i] * s2);
        if (a.dh) {
          widen(rh[v], xh[v]);
#pragma unroll
          for (int i = 0; i < VEC; ++i) e[v][i] += xh[v][i];
        }
        narrow(e[v], ry[v]);
        *reinterpret_cast<LaneVec<T, VEC> *>(static_cast<T *>(a.dx) + base + c) = ry[v];
      }
    }
  }
  float *p = parts + (size_t)blockIdx.x * 2 * D;
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int c = (v * blockDim.x + threadIdx.x) * VEC;
    if (c < D) {
      store_f32(dg[v], p + c);
      store_f32(db[v], p + D + c);
    }
  }
}

// Blocks of the backward: enough to fill the GPU, one row at least for each.
int bwd_blocks(long long rows, int width) {
  return (int)std::max<long long>(1, std::min<long long>(rows, (long long)sm_count() * std::max(1, 512 / row_threads(width))));
}

// 16-byte vectors where every row starts on one, single values elsewhere.
template <typename T>
bool vector_rows(int width) { return width * sizeof(T) % 16 == 0; }

template <typename T>
cudaError_t fwd_t(const NormFwdArgs &a, cudaStream_t stream) {
  if (a.rows == 0) return cudaSuccess;
  const unsigned grid = (unsigned)std::min<long long>(a.rows, 1 << 30);
  const int threads = row_threads(a.width);
  note_launch();
  if (vector_rows<T>(a.width)) norm_fwd_kernel<T, 16 / sizeof(T)><<<grid, threads, 0, stream>>>(a);
  else norm_fwd_kernel<T, 1><<<grid, threads, 0, stream>>>(a);
  return cudaGetLastError();
}

template <typename T, typename S>
cudaError_t bwd_t(const NormBwdArgs &a, float *parts, cudaStream_t stream) {
  const int blocks = bwd_blocks(a.rows, a.width), threads = row_threads(a.width);
  note_launch();
  if (vector_rows<T>(a.width)) norm_bwd_kernel<T, S, 16 / sizeof(T)><<<blocks, threads, 0, stream>>>(a, parts);
  else norm_bwd_kernel<T, S, 1><<<blocks, threads, 0, stream>>>(a, parts);
  const cudaError_t err = cudaGetLastError();
  if (err != cudaSuccess) return err;
  return launch_colsum({parts, blocks, 2 * a.width, {a.dweight, a.dbias, nullptr}, {a.width, 2 * a.width, 2 * a.width}},
                       stream);
}

}  // namespace

cudaError_t launch_norm_fwd(const NormFwdArgs &a, bool bf16, cudaStream_t stream) {
  return bf16 ? fwd_t<__nv_bfloat16>(a, stream) : fwd_t<float>(a, stream);
}

size_t norm_bwd_workspace_bytes(long long rows, int width) {
  return (size_t)bwd_blocks(rows, width) * 2 * width * sizeof(float);
}

cudaError_t launch_norm_bwd(const NormBwdArgs &a, bool bf16, void *ws, cudaStream_t stream) {
  float *parts = static_cast<float *>(ws);
  if (a.scales) return bf16 ? bwd_t<__nv_bfloat16, int8_t>(a, parts, stream) : bwd_t<float, int8_t>(a, parts, stream);
  return bf16 ? bwd_t<__nv_bfloat16, __nv_bfloat16>(a, parts, stream) : bwd_t<float, float>(a, parts, stream);
}

}  // namespace gdn2
