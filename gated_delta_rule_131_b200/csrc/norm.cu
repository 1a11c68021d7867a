// Layer norm over the rows of the residual stream, in front of the block's projections, and its
// backward pass.
//
// Forward, per row of D channels: h = x + residual (rounded to the element type, so that the stored
// row is the one that is normalised), mean = sum h / D, rstd = 1 / sqrt(sum (h - mean)^2 / D + eps),
// y = (h - mean) rstd g + b; h's 8-bit checkpoint in the same pass.
// Backward, with xh = (h - mean) rstd and e = dy g: dx = rstd (e - mean(e) - xh mean(e xh)) + dh,
// dg = sum over rows of dy xh, db = sum over rows of dy.
//
// Both are HBM-bound streams.  A row is held in the registers of `span` threads, NE values each, so it
// is read once; the statistics are sums over those threads, the variance taken about the mean.  Threads
// walk rows in turn and load the next one before the sums of this one meet, or, where the registers do not
// hold two, ask for its lines in the L2 (see EARLY).  A column's sums over rows are fp32 sums in one register over the
// rows of a group (rows / (148 * groups) of them, at most), then over a block's groups, then over the blocks.
//
// 8192 x 2048 bf16: forward with a residual 25 us, 134 MB at 5.3 TB/s (fp32 46 us, 5.8 TB/s); backward
// with dh 33 us, 134 MB at 4.1 TB/s, of which about 5 us are the second launch (fp32 51 us, 5.2 TB/s);
// from 8 bits 31 us.  Both are bound by latency: two barriers a row forward, one backward, at 50 to 63 %
// of the issue slots; 16 values per thread halve the sums' share (8: 37 us backward, 33 forward).
// The backward of that layer was slower with a ring of three rows filled by asynchronous copies in
// 1024-thread blocks (39 us), two rows at a time (50 us), dh loaded a row ahead (35 us), and its second
// launch took twice as long with fp64 sums of the columns.
//
// Widths that are no multiple of 16 bytes move value by value, far from the bytes they need: backward with dh
// 8192 x 2047 57 us in bf16, 68 from 8 bits, 60 in fp32, 72 from 8 bits; 4096 x 8191 239, 309, 194 and 247
// us, where 8192 wide takes 57, 55, 100 and 90.  ptxas reports spills of the backward's forms for them (140 to
// 350 bytes stored by a thread with 16 values, 36 to 52 with 8 from 8 bits) and of the fp32 form of 16
// values in 16-byte vectors (44 and 60 bytes).
#include <algorithm>
#include <utility>

#include "act8.cuh"

namespace gdn2 {
namespace {

// Calls f(0), f(1), .. with compile-time indices.
template <typename F, int... I>
__device__ __forceinline__ void each_(F f, std::integer_sequence<int, I...>) {
  (f(std::integral_constant<int, I>()), ...);
}
template <int N, typename F>
__device__ __forceinline__ void each(F f) { each_(f, std::make_integer_sequence<int, N>()); }

// How a row lies in its threads: vector v of thread `tid` covers the VEC columns from (v * span + tid) *
// VEC, so that a warp's accesses lie side by side and one warp holds every group of 32 channels.  FULL:
// the row fills its threads, and nothing has to be checked.
template <int VEC, int NE, bool FULL> struct Row {
  static constexpr int N = NE / VEC;
  int D, span, tid;
  __device__ __forceinline__ int col(int v) const { return (v * span + tid) * VEC; }
  __device__ __forceinline__ bool inside(int v) const { return FULL || col(v) < D; }
  // Values past the row's end are zeros.
  template <typename S> __device__ __forceinline__ void load(LaneVec<S, VEC> (&r)[N], const S *row) const {
#pragma unroll
    for (int v = 0; v < N; ++v) {
      if (!FULL) r[v] = LaneVec<S, VEC>{};
      if (inside(v)) r[v].load(row + col(v));
    }
  }
  template <typename S> __device__ __forceinline__ void store(const LaneVec<S, VEC> (&r)[N], S *row) const {
#pragma unroll
    for (int v = 0; v < N; ++v)
      if (inside(v)) r[v].store(row + col(v));
  }
  // Asks for the row's lines in the L2, each once.
  template <typename S> __device__ __forceinline__ void ask(const S *row) const {
    const uintptr_t begin = reinterpret_cast<uintptr_t>(row), end = reinterpret_cast<uintptr_t>(row + D);
    for (uintptr_t p = (begin & ~(uintptr_t)127) + 128 * tid; p < end; p += 128 * span)
      asm volatile("prefetch.global.L2 [%0];" ::"l"(p < begin ? begin : p));
  }
  template <typename S> static __device__ __forceinline__ void get(const LaneVec<S, VEC> (&r)[N], Pairs<NE> &f) {
    each<N>([&](auto v) { widen<v * VEC, VEC>(r[v], f); });
  }
  template <typename S> static __device__ __forceinline__ void put(const Pairs<NE> &f, LaneVec<S, VEC> (&r)[N]) {
    each<N>([&](auto v) { narrow<v * VEC, VEC>(f, r[v]); });
  }
  __device__ __forceinline__ void weights(const float *p, Pairs<NE> &f) const {
    each<N>([&](auto v) {
      if (inside(v)) load_f32<v * VEC, VEC>(p + col(v), f);
    });
  }
  // The row's weights, kept in shared memory as [NE / 4][span] float4 where a lane's vector is longer
  // than one: read from there they cost no bank conflicts, while a warp's 16-byte loads 32 or 64 bytes
  // apart would take the L1 twice or four times as long (backward 8192 x 2048: 34 us instead of 32).
  static constexpr bool STAGED = VEC > 4;
  __device__ __forceinline__ void stage(const float *p, float4 *s) const {
    Pairs<NE> f;
    fill(f, 0.f);
    weights(p, f);
#pragma unroll
    for (int k = 0; k < NE / 4; ++k)
      s[k * span + tid] = make_float4(f.p[2 * k].x, f.p[2 * k].y, f.p[2 * k + 1].x, f.p[2 * k + 1].y);
  }
  __device__ __forceinline__ void staged(const float4 *s, Pairs<NE> &f) const {
#pragma unroll
    for (int k = 0; k < NE / 4; ++k) {
      const float4 q = s[k * span + tid];
      f.p[2 * k] = make_float2(q.x, q.y);
      f.p[2 * k + 1] = make_float2(q.z, q.w);
    }
  }
};

// The sums of NV (1 or 2) values over a row's threads, in a fixed order; `group` is the row's place in
// the block and `red` its block's [warp][2].  A warp folds two values onto its odd and even lanes while
// it sums.  Two buffers in turn make one barrier enough; each group has its own (0 is __syncthreads').
template <int NV>
__device__ __forceinline__ void row_sum(float (&v)[NV], float (*red)[2], int group, int span) {
  const int lane = threadIdx.x & 31;
  float s = v[0];
  if constexpr (NV == 2) {
    const bool odd = lane & 1;
    s = (odd ? v[1] : v[0]) + __shfl_xor_sync(0xffffffffu, odd ? v[0] : v[1], 1);
  }
#pragma unroll
  for (int m = NV; m < 32; m <<= 1) s += __shfl_xor_sync(0xffffffffu, s, m);
  if (span == 32) {
    if constexpr (NV == 2) v[1] = __shfl_sync(0xffffffffu, s, 1);
    v[0] = __shfl_sync(0xffffffffu, s, 0);
    return;
  }
  if (lane < NV) red[threadIdx.x >> 5][lane] = s;
  asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(span) : "memory");
  const float2 *r = reinterpret_cast<const float2 *>(red[group * (span >> 5)]);
  float2 t = r[0];
#pragma unroll 4
  for (int w = 1; w < span >> 5; ++w) t = __fadd2_rn(t, r[w]);
  v[0] = t.x;
  if constexpr (NV == 2) v[1] = t.y;
}

// One row at a time per block.
template <typename T, int VEC, int NE, bool FULL>
__global__ void __launch_bounds__(512) norm_fwd_kernel(const NormFwdArgs a) {
  using R = Row<VEC, NE, FULL>;
  __shared__ __align__(8) float red[2][16][2];
  const R row{a.width, (int)blockDim.x, (int)threadIdx.x};
  const int D = a.width, groups = (D + ACT_GROUP - 1) / ACT_GROUP;
  const float inv_d = 1.f / (float)D;
  const T *px = static_cast<const T *>(a.x), *pr = static_cast<const T *>(a.residual);
  LaneVec<T, VEC> rx[R::N], rr[R::N];
  row.load(rx, px + (size_t)blockIdx.x * D);
  if (pr) row.load(rr, pr + (size_t)blockIdx.x * D);
  for (long long at = blockIdx.x; at < a.rows; at += gridDim.x) {
    const size_t base = (size_t)at * D;
    Pairs<NE> f;
    R::get(rx, f);
    if (pr) {
      Pairs<NE> r;
      R::get(rr, r);
#pragma unroll
      for (int i = 0; i < NE / 2; ++i) f.p[i] = __fadd2_rn(f.p[i], r.p[i]);
      R::put(f, rx);
      row.store(rx, static_cast<T *>(a.h) + base);
      R::get(rx, f);
    }
    if (a.codes)
      each<R::N>([&](auto v) {
        uint32_t sc;
        const LaneVec<int8_t, VEC> code = act8_encode<v * VEC>(rx[v], f, row.inside(v), sc);
        if (row.inside(v)) {
          const int c = row.col(v);
          code.store(a.codes + base + c);
          if (c % ACT_GROUP == 0) a.scales[(size_t)at * groups + c / ACT_GROUP] = (uint8_t)sc;
        }
      });
    if (at + gridDim.x < a.rows) {
      row.load(rx, px + base + (size_t)gridDim.x * D);
      if (pr) row.load(rr, pr + base + (size_t)gridDim.x * D);
    }
    float s[1] = {total(f)};
    row_sum(s, red[0], 0, blockDim.x);
    const float mean = s[0] * inv_d;
#pragma unroll
    for (int i = 0; i < NE / 2; ++i) f.p[i] = __fadd2_rn(f.p[i], splat(-mean));
    if (!FULL) each<R::N>([&](auto v) {
      if (!row.inside(v))
#pragma unroll
        for (int i = 0; i < VEC; ++i) f.set(v * VEC + i, 0.f);
    });
    s[0] = dot(f, f);
    row_sum(s, red[1], 0, blockDim.x);
    const float rstd = 1.f / sqrtf(s[0] * inv_d + a.eps);
    if (threadIdx.x == 0 && a.mean) {
      a.mean[at] = mean;
      a.rstd[at] = rstd;
    }
    each<R::N>([&](auto v) {
      if (!row.inside(v)) return;
      const int c = row.col(v);
      Pairs<VEC + VEC % 2> g, b;
      load_f32<0, VEC>(a.weight + c, g);
      if (a.bias) load_f32<0, VEC>(a.bias + c, b);
      else fill(b, 0.f);
      if constexpr (VEC == 1) {
        f.set(v, fmaf(f.get(v) * rstd, g.get(0), b.get(0)));
      } else {
#pragma unroll
        for (int i = 0; i < VEC / 2; ++i)
          f.p[v * VEC / 2 + i] = __ffma2_rn(__fmul2_rn(f.p[v * VEC / 2 + i], splat(rstd)), g.p[i], b.p[i]);
      }
      LaneVec<T, VEC> y;
      narrow<v * VEC, VEC>(f, y);
      y.store(static_cast<T *>(a.y) + base + c);
    });
  }
}

// A block holds `groups` = blockDim.x / span rows at a time.  The groups' weight gradients are added at
// the end, so that a block leaves one row of partial sums in `parts`: [gridDim.x][2][D] (dweight, dbias).
// Without `parts` the grid is one cluster, which adds them itself.
template <typename T, typename S, int VEC, int NE, bool FULL>
__global__ void __launch_bounds__(512) norm_bwd_kernel(const NormBwdArgs a, float *parts, int span) {
  constexpr bool Q = sizeof(S) == 1;  // h is held in 8 bits
  // The registers hold the next row, or its lines are asked for (4096 x 8191 bf16 237 us, without 315; fp32
  // from 8 bits 247 and 315; rows of 32-byte vectors are no faster for it: 4096 x 8192 fp32 99 us either way,
  // from 8 bits 91 us and 90 without).
  constexpr bool EARLY = NE == 8 || (VEC > 1 && sizeof(T) == 2), ASK = !EARLY && !FULL;
  using R = Row<VEC, NE, FULL>;
  extern __shared__ __align__(16) float sums[];  // the weights where R::STAGED; at the end [group][2][D]
  __shared__ __align__(8) float red[2][16][2];
  const int D = a.width, scales = (D + ACT_GROUP - 1) / ACT_GROUP;
  const int group = threadIdx.x / span, groups = blockDim.x / span;
  const R row{D, span, (int)threadIdx.x - group * span};
  const float inv_d = 1.f / (float)D;
  Pairs<NE> g, dg, db;
  fill(g, 0.f);
  fill(dg, 0.f);
  fill(db, 0.f);
  if (R::STAGED) {
    if (group == 0) row.stage(a.weight, reinterpret_cast<float4 *>(sums));
    __syncthreads();
  } else if (NE == 8) {
    row.weights(a.weight, g);
  }
  LaneVec<T, VEC> ry[R::N], rh[R::N];
  LaneVec<S, VEC> rs[R::N];
  uint8_t sc[R::N];
  float mean = 0.f, rstd = 0.f;
  auto load = [&](long long at) {
    const size_t base = (size_t)at * D;
    row.load(ry, static_cast<const T *>(a.dy) + base);
    row.load(rs, static_cast<const S *>(a.h) + base);
    if (Q)
#pragma unroll
      for (int v = 0; v < R::N; ++v)
        sc[v] = row.inside(v) ? a.scales[(size_t)at * scales + row.col(v) / ACT_GROUP] : 0;
    mean = a.mean[at];
    rstd = a.rstd[at];
  };
  auto ask = [&](long long at) {
    row.ask(static_cast<const T *>(a.dy) + (size_t)at * D);
    row.ask(static_cast<const S *>(a.h) + (size_t)at * D);
  };
  const long long step = (long long)gridDim.x * groups;
  long long at = (long long)blockIdx.x * groups + group;
  if (EARLY && at < a.rows) load(at);
  for (int turn = 0; at < a.rows; at += step, turn ^= 1) {
    const size_t base = (size_t)at * D;
    if (!EARLY) load(at);
    Pairs<NE> xh, e;
    if constexpr (Q) each<R::N>([&](auto v) { widen<v * VEC, VEC>(rs[v], act8_unit(sc[v]), xh); });
    else R::get(rs, xh);
    R::get(ry, e);
    if (a.dh) row.load(rh, static_cast<const T *>(a.dh) + base);
    const float m = -mean, r = rstd;
    if (at + step < a.rows) {
      if (EARLY) load(at + step);
      if (ASK) ask(at + step);
    }
    if constexpr (R::STAGED) row.staged(reinterpret_cast<const float4 *>(sums), g);
    else if (NE == 16) row.weights(a.weight, g);  // 8 values fit the registers for good, 16 do not
    float2 t1 = make_float2(0.f, 0.f), t2 = t1;
#pragma unroll
    for (int i = 0; i < NE / 2; ++i) {
      xh.p[i] = __fmul2_rn(__fadd2_rn(xh.p[i], splat(m)), splat(r));
      dg.p[i] = __ffma2_rn(e.p[i], xh.p[i], dg.p[i]);
      db.p[i] = __fadd2_rn(db.p[i], e.p[i]);
      e.p[i] = __fmul2_rn(e.p[i], g.p[i]);  // zero past the row's end, and so are its terms below
      t1 = __fadd2_rn(t1, e.p[i]);
      t2 = __ffma2_rn(e.p[i], xh.p[i], t2);
    }
    float s[2] = {t1.x + t1.y, t2.x + t2.y};
    row_sum(s, red[turn], group, span);
    const float2 k1 = splat(-s[0] * inv_d), k2 = splat(-s[1] * inv_d);
    if (a.dh) {
      Pairs<NE> dh;
      R::get(rh, dh);
#pragma unroll
      for (int i = 0; i < NE / 2; ++i)
        e.p[i] = __ffma2_rn(splat(r), __ffma2_rn(xh.p[i], k2, __fadd2_rn(e.p[i], k1)), dh.p[i]);
    } else {
#pragma unroll
      for (int i = 0; i < NE / 2; ++i)
        e.p[i] = __fmul2_rn(splat(r), __ffma2_rn(xh.p[i], k2, __fadd2_rn(e.p[i], k1)));
    }
    R::put(e, rh);
    row.store(rh, static_cast<T *>(a.dx) + base);
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  float *p = parts ? parts + (size_t)blockIdx.x * 2 * D : sums;
  float *mine = groups == 1 ? p : sums + (size_t)group * 2 * D;
  if (R::STAGED) __syncthreads();  // every group has read its last weights
  each<R::N>([&](auto v) {
    if (row.inside(v)) {
      store_f32<v * VEC, VEC>(dg, mine + row.col(v));
      store_f32<v * VEC, VEC>(db, mine + D + row.col(v));
    }
  });
  if (groups > 1) {
    __syncthreads();
    for (int c = threadIdx.x; c < 2 * D; c += blockDim.x) {
      float t = sums[c];
      for (int q = 1; q < groups; ++q) t += sums[(size_t)q * 2 * D + c];
      p[c] = t;
    }
  }
  if (!parts) cluster_sum(sums, 2 * D, a.dweight, D, a.dbias);
}

constexpr int FWD_THREADS = 1024;  // per SM
static_assert(512 * 16 == LN_MAX_WIDTH, "512 threads hold the widest row");
// Threads of a row: whole warps of ne values per thread.
int row_threads(int width, int ne) { return (width + 32 * ne - 1) / (32 * ne) * 32; }

template <typename T, int VEC, int NE, bool FULL>
cudaError_t fwd_launch(const NormFwdArgs &a, cudaStream_t stream) {
  const int span = row_threads(a.width, NE);
  const long long fill = (long long)sm_count() * std::min(16, std::max(1, FWD_THREADS / span));
  note_launch();
  norm_fwd_kernel<T, VEC, NE, FULL><<<(unsigned)std::min<long long>(a.rows, fill), span, 0, stream>>>(a);
  return cudaGetLastError();
}

// 16-byte vectors where every row starts on one, else single values.  (32-byte vectors, which the
// backward takes, are no faster here: 8192 x 2048 with a residual 25 us either way.)
template <typename T>
cudaError_t fwd_t(const NormFwdArgs &a, cudaStream_t stream) {
  if (a.rows == 0) return cudaSuccess;
  constexpr int V = 16 / sizeof(T);
  if (a.width % (32 * 16) == 0) return fwd_launch<T, V, 16, true>(a, stream);
  if (a.width % V == 0) return fwd_launch<T, V, 16, false>(a, stream);
  return a.width <= 4096 ? fwd_launch<T, 1, 8, false>(a, stream) : fwd_launch<T, 1, 16, false>(a, stream);
}

// The backward's blocks of up to 512 threads: as many rows at a time as they hold (barriers 1 to 15 are
// the groups', one warp needs none), one block per SM.  What one cluster of blocks holds at a time, with
// sums of one row or of at most 1024 channels per block, goes without the second launch: 13.3 us a call,
// 17.3 with it, at the same 4.0 us of the GPU's time (8 x 2048).  With more sums to add, 32 x 2048 in
// blocks of four rows, the GPU took 6.4 us for 4.3.
struct NormBwdPlan {
  int ne, span, groups, blocks;
  bool cluster;
};
NormBwdPlan norm_bwd_plan(long long rows, int width, bool bf16) {
  NormBwdPlan p;
  // 16 values per thread halve the sums' share of the work; fp32 vectors and single values take their
  // registers twice, and rows that 8 hold are faster so (8192 x 2048 fp32: 51 us, with 16: 66 us)
  p.ne = width > 4096 || (bf16 && width % 8 == 0) ? 16 : 8;
  p.span = row_threads(width, p.ne);
  const int most = p.span == 32 ? 16 : std::min(512 / p.span, 15);
  const long long sms = sm_count();
  p.cluster = rows <= CLUSTER_BLOCKS || (rows <= CLUSTER_BLOCKS * most && rows * width <= CLUSTER_BLOCKS * 1024);
  const long long per = p.cluster ? CLUSTER_BLOCKS : sms;
  p.groups = (int)std::max(1ll, std::min<long long>(most, (rows + per - 1) / per));
  p.blocks = p.cluster ? CLUSTER_BLOCKS : (int)std::min((rows + p.groups - 1) / p.groups, sms);
  return p;
}

template <typename T, typename S, int VEC, int NE, bool FULL>
cudaError_t bwd_launch(const NormBwdArgs &a, const NormBwdPlan &p, float *parts, cudaStream_t stream) {
  const auto kernel = norm_bwd_kernel<T, S, VEC, NE, FULL>;
  static std::atomic<uint64_t> allowed;
  // at most 512 threads' worth of groups: 512 * NE columns, twice
  const cudaError_t err = allow_smem((const void *)kernel, 512 * NE * 2 * (int)sizeof(float), allowed);
  if (err != cudaSuccess) return err;
  note_launch();
  const int sums = p.groups > 1 || p.cluster ? p.groups * 2 * a.width : 0;
  const int smem = std::max(sums, VEC > 4 ? p.span * NE : 0) * (int)sizeof(float);
  if (p.cluster) return launch_cluster(kernel, p.span * p.groups, smem, stream, a, parts, p.span);
  kernel<<<p.blocks, p.span * p.groups, smem, stream>>>(a, parts, p.span);
  return cudaGetLastError();
}

// 32-byte vectors where a row fills its threads and everything lies on such boundaries (half the
// instructions for loads and addresses: 8192 x 2048 in 32 us, 37 us without), 16-byte ones where every
// row starts on one, else single values.
template <typename T, typename S>
cudaError_t bwd_t(const NormBwdArgs &a, float *parts, cudaStream_t stream) {
  constexpr int V = 16 / sizeof(T), FEW = sizeof(T) == 4 ? 8 : 16;  // see norm_bwd_plan
  const NormBwdPlan p = norm_bwd_plan(a.rows, a.width, sizeof(T) == 2);
  const bool full = a.width % (32 * p.ne) == 0 &&
                    on32((const char *)a.dy, (const char *)a.dh, (const char *)a.dx, a.scales ? nullptr : (const char *)a.h);
  cudaError_t err;
  if (a.width % V != 0)
    err = p.ne == 8 ? bwd_launch<T, S, 1, 8, false>(a, p, parts, stream) : bwd_launch<T, S, 1, 16, false>(a, p, parts, stream);
  else if (p.ne == FEW)
    err = full ? bwd_launch<T, S, 2 * V, FEW, true>(a, p, parts, stream) : bwd_launch<T, S, V, FEW, false>(a, p, parts, stream);
  else
    err = full ? bwd_launch<T, S, 2 * V, 16, true>(a, p, parts, stream) : bwd_launch<T, S, V, 16, false>(a, p, parts, stream);
  if (err != cudaSuccess || p.cluster) return err;
  return launch_colsum({parts, p.blocks, 2 * a.width, {a.dweight, a.dbias, nullptr}, {a.width, 2 * a.width, 2 * a.width}},
                       stream);
}

}  // namespace

cudaError_t launch_norm_fwd(const NormFwdArgs &a, bool bf16, cudaStream_t stream) {
  return bf16 ? fwd_t<__nv_bfloat16>(a, stream) : fwd_t<float>(a, stream);
}

size_t norm_bwd_workspace_bytes(long long rows, int width, bool bf16) {
  const NormBwdPlan p = norm_bwd_plan(rows, width, bf16);
  return p.cluster ? 0 : (size_t)p.blocks * 2 * width * sizeof(float);
}

cudaError_t launch_norm_bwd(const NormBwdArgs &a, bool bf16, void *ws, cudaStream_t stream) {
  float *parts = static_cast<float *>(ws);
  if (a.scales) return bf16 ? bwd_t<__nv_bfloat16, int8_t>(a, parts, stream) : bwd_t<float, int8_t>(a, parts, stream);
  return bf16 ? bwd_t<__nv_bfloat16, __nv_bfloat16>(a, parts, stream) : bwd_t<float, float>(a, parts, stream);
}

}  // namespace gdn2
