// Backward of the work around the mixer in its block: of the output gate behind it (RMS norm times
// SiLU gate) and of the short convolutions, SiLU, L2 norm and gates in front of it.  The forward is
// defined in block.cu; here its inputs are read again (in their type, or held in 8 bits) and what the
// gradients need of the forward is formed anew, in fp32.
//
// Figures in this file are of short runs (15 calls back to back) at high clocks, unless they are said to be
// of long ones (half a second and more, at the clocks that the power limit leaves).
#include <algorithm>
#include <climits>
#include <type_traits>

#include "act8.cuh"

namespace gdn2 {
namespace {

constexpr int CE = 8;  // channels per lane of the pointwise passes
constexpr int CC = 4;  // channels per lane of the convolution paths
constexpr float L2_EPS = 1e-6f, RMS_EPS = 1e-5f;

__device__ __forceinline__ float ex2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// sigmoid(x) = 1 / (1 + 2^(-x log2 e)) of a pair; 0 and 1 at the far ends.
__device__ __forceinline__ float2 sigmoid2(float2 x) {
  const float2 m = __fmul2_rn(x, splat(-1.4426950408889634f));
  const float2 den = __fadd2_rn(make_float2(ex2_approx(m.x), ex2_approx(m.y)), splat(1.f));
  return make_float2(rcp_approx(den.x), rcp_approx(den.y));
}
__device__ __forceinline__ float rsqrt_approx(float x) {
  float y;
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// 1 - s of a pair.
__device__ __forceinline__ float2 one_minus2(float2 s) { return __ffma2_rn(s, splat(-1.f), splat(1.f)); }

// N channels of a lane, as loaded: words of WB bytes at most (16, or 32 on such boundaries).
template <typename S, int N, int WB = 16> struct Lane {
  static constexpr int VEC = N * (int)sizeof(S) > WB ? WB / (int)sizeof(S) : N, WORDS = N / VEC;
  LaneVec<S, VEC> v[WORDS];
  __device__ __forceinline__ void load(const S *p) {
#pragma unroll
    for (int i = 0; i < WORDS; ++i) v[i].load(p + i * VEC);
  }
  __device__ __forceinline__ void load_cached(const S *p) {
#pragma unroll
    for (int i = 0; i < WORDS; ++i) v[i].load_cached(p + i * VEC);
  }
  __device__ __forceinline__ void store(S *p) const {
#pragma unroll
    for (int i = 0; i < WORDS; ++i) v[i].store(p + i * VEC);
  }
  template <int I = 0> __device__ __forceinline__ void get(Pairs<N> &f, float unit) const {
    if constexpr (sizeof(S) == 1) widen<I * VEC, VEC>(v[I], unit, f);
    else widen<I * VEC, VEC>(v[I], f);
    if constexpr (I + 1 < WORDS) get<I + 1>(f, unit);
  }
  template <int I = 0> __device__ __forceinline__ void put(const Pairs<N> &f) {
    narrow<I * VEC, VEC>(f, v[I]);
    if constexpr (I + 1 < WORDS) put<I + 1>(f);
  }
};

// d <- sign d p (1 - p), p = sigmoid(x): p (1 - p) = e / (1 + e)^2 with e = 2^-(|x| log2 e), which neither
// cancels nor overflows.  Each channel has a reciprocal of its own: one of the pair's product would carry a
// channel's NaN to the other (and saved nothing: the prologue's 1.3B layer 114.9 us either way, packed from
// 8 bits 516 us for 517).
template <int N> __device__ __forceinline__ void gate_bwd(const Pairs<N> &x, Pairs<N> &d, float sign) {
#pragma unroll
  for (int c = 0; c < N / 2; ++c) {
    const float2 e = make_float2(ex2_approx(-1.4426950408889634f * fabsf(x.p[c].x)),
                                 ex2_approx(-1.4426950408889634f * fabsf(x.p[c].y)));
    const float2 den = __fadd2_rn(e, splat(1.f));
    const float2 p = make_float2(rcp_approx(den.x), rcp_approx(den.y));
    d.p[c] = __fmul2_rn(__fmul2_rn(d.p[c], e), __fmul2_rn(p, __fmul2_rn(p, splat(sign))));
  }
}

// Sum over the G lanes of a row (G a power of two, the lanes aligned within their warp).
template <int G>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
  for (int m = 1; m < G; m <<= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
  return x;
}

// Asynchronous copy of BYTES (4, 8 or 16) from global to shared memory.
template <int BYTES>
__device__ __forceinline__ void cp_async(void *smem, const void *gmem) {
  const uint32_t s = (uint32_t)__cvta_generic_to_shared(smem);
  if constexpr (BYTES == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(s), "l"(gmem) : "memory");
  else asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(s), "l"(gmem), "n"(BYTES) : "memory");
}
// ---------------------------------------------------------------------------------------- epilogue
//
// y = oh g s with oh = o r, r = 1 / sqrt(mean o^2 + eps), s = z sigmoid(z).  With e = dy g s:
// do = r (e - oh mean(e oh)), dz = dy g oh sigmoid(z) (1 + z (1 - sigmoid(z))), dg = sum over rows of
// dy oh s.
//
// A row of d_v values is held by G lanes, one 32-byte vector of dy each (16 bf16 or 8 fp32 values); a block
// takes tiles of whole rows in turn, loads the next one while it works on this, and keeps its dg in
// registers until the end.  Each value is read once and written once.  1.3B layer (8192 x 16 x 128 bf16) 34
// us, 168 MB at 4.9 TB/s; 12345 x 32 x 256 from 8 bits 162 us, 815 MB at 5.0 TB/s (168 us and 4.8 TB/s in
// long runs); fp32 layer 58 us.  Bound by latency at 16 warps per SM: the exponential and the reciprocal
// keep the special function units 37 % busy, issue slots are 41 to 49 % used.  More warps need fewer
// registers than the three rows of values take: 8 values per lane at 24 or 32 warps ran 35 and 34 us, and
// 171 and 163 us.

template <typename T> constexpr int EPI_CHANNELS = 32 / sizeof(T);  // per lane: one 32-byte vector
constexpr int EPI_THREADS = 256, EPI_BLOCKS = 2;                    // blocks per SM: 128 registers

template <typename T, typename S, int DV, int WB>
__global__ void __launch_bounds__(EPI_THREADS, EPI_BLOCKS) epilogue_bwd_kernel(const EpilogueBwdArgs a, float *parts) {
  constexpr int EC = EPI_CHANNELS<T>, G = DV / EC, GROUPS = EPI_THREADS / G, TILE = EPI_THREADS * EC;  // whole rows
  constexpr bool Q = sizeof(S) == 1;
  __shared__ float red[GROUPS][DV];
  const int grp = threadIdx.x / G, c = (threadIdx.x % G) * EC;
  const unsigned off = threadIdx.x * EC;  // a lane's place in every tile
  Pairs<EC> g, dg;
  fill(dg, 0.f);
#pragma unroll
  for (int i = 0; i < EC; ++i) g.set(i, a.g[c + i]);
  const long long total = a.rows * DV, step = (long long)gridDim.x * TILE;
  Lane<S, EC, WB> ro, rz;
  Lane<T, EC, WB> ry;
  uint8_t so = 0, sz = 0;
  auto load = [&](long long base) {  // (marked to leave the L2 first, the loads cost 3 % here)
    ro.load_cached(static_cast<const S *>(a.o) + base + off);
    rz.load_cached(static_cast<const S *>(a.z) + base + off);
    ry.load_cached(static_cast<const T *>(a.dy) + base + off);
    if (Q) {
      so = a.o_scales[base / ACT_GROUP + off / ACT_GROUP];
      sz = a.z_scales[base / ACT_GROUP + off / ACT_GROUP];
    }
  };
  auto inside = [&](long long base) { return base + off < total; };
  auto tile = [&](long long base, auto checked) {
    const bool live = !decltype(checked)::value || inside(base);
    Pairs<EC> o, z, e;
    if (live) {
      ro.get(o, Q ? act8_unit(so) : 0.f);
      rz.get(z, Q ? act8_unit(sz) : 0.f);
      ry.get(e, 0.f);
    } else {  // the sums shuffle whole warps
      fill(o, 0.f);
      fill(z, 0.f);
      fill(e, 0.f);
    }
    if (inside(base + step)) load(base + step);
    const float r = rsqrt_approx(row_sum<G>(dot(o, o)) * (1.f / DV) + RMS_EPS);
#pragma unroll
    for (int i = 0; i < EC / 2; ++i) {
      const float2 sg = sigmoid2(z.p[i]), s = __fmul2_rn(z.p[i], sg);
      o.p[i] = __fmul2_rn(o.p[i], splat(r));  // oh
      const float2 yo = __fmul2_rn(e.p[i], o.p[i]), yg = __fmul2_rn(e.p[i], g.p[i]);
      dg.p[i] = __ffma2_rn(yo, s, dg.p[i]);
      z.p[i] = __fmul2_rn(__fmul2_rn(yo, g.p[i]), __ffma2_rn(s, one_minus2(sg), sg));  // dz
      e.p[i] = __fmul2_rn(yg, s);
    }
    const float m = row_sum<G>(dot(e, o)) * (-1.f / DV);
    if (live) {
#pragma unroll
      for (int i = 0; i < EC / 2; ++i) e.p[i] = __fmul2_rn(splat(r), __ffma2_rn(o.p[i], splat(m), e.p[i]));
      Lane<T, EC, WB> out;
      out.put(e);
      out.store(static_cast<T *>(a.dout) + base + off);
      out.put(z);
      out.store(static_cast<T *>(a.dz) + base + off);
    }
  };
  long long base = (long long)blockIdx.x * TILE;
  if (inside(base)) load(base);
  for (; base + TILE <= total; base += step) tile(base, std::false_type());
  if (base < total) tile(base, std::true_type());
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
#pragma unroll
  for (int i = 0; i < EC; ++i) red[grp][c + i] = dg.get(i);
  __syncthreads();
  for (int k = threadIdx.x; k < DV; k += EPI_THREADS) {
    float s = 0.f;
#pragma unroll 8
    for (int w = 0; w < GROUPS; ++w) s += red[w][k];
    if (parts) parts[(size_t)blockIdx.x * DV + k] = s;
    else red[0][k] = s;
  }
  if (!parts) cluster_sum(red[0], DV, a.dg, DV, nullptr);  // the grid is one cluster
}

// Up to two tiles a block of one cluster go without the second launch: 12.0 us a call, 16.2 with it, at
// 3.9 us of the GPU's time for 3.5 at most (128 x 256 fp32).  Four tiles took 5.4 us of it for 4.0.
struct EpiloguePlan {
  int blocks;
  bool cluster;
};
EpiloguePlan epilogue_plan(long long rows, int dv, int channels) {
  const long long per = EPI_THREADS / (dv / channels), tiles = (rows + per - 1) / per;
  if (tiles <= 2 * CLUSTER_BLOCKS) return {CLUSTER_BLOCKS, true};
  return {(int)std::min<long long>(tiles, (long long)sm_count() * EPI_BLOCKS), false};
}

template <typename T, typename S, int WB>
cudaError_t epilogue_t(const EpilogueBwdArgs &a, float *parts, cudaStream_t stream) {
  const EpiloguePlan p = epilogue_plan(a.rows, a.dv, EPI_CHANNELS<T>);
  const auto kernel = a.dv == 64    ? epilogue_bwd_kernel<T, S, 64, WB>
                      : a.dv == 128 ? epilogue_bwd_kernel<T, S, 128, WB>
                                    : epilogue_bwd_kernel<T, S, 256, WB>;
  note_launch();
  if (p.cluster) return launch_cluster(kernel, EPI_THREADS, 0, stream, a, parts);
  kernel<<<p.blocks, EPI_THREADS, 0, stream>>>(a, parts);
  const cudaError_t err = cudaGetLastError();
  if (err != cudaSuccess) return err;
  return launch_colsum({parts, p.blocks, a.dv, {a.dg, nullptr, nullptr}, {a.dv, a.dv, a.dv}}, stream);
}

template <typename T, typename S>
cudaError_t epilogue_t(const EpilogueBwdArgs &a, float *parts, cudaStream_t stream) {
  const bool wide = on32((const char *)a.dy, (const char *)a.dout, (const char *)a.dz,
                         sizeof(S) == 1 ? nullptr : (const char *)a.o, sizeof(S) == 1 ? nullptr : (const char *)a.z);
  return wide ? epilogue_t<T, S, 32>(a, parts, stream) : epilogue_t<T, S, 16>(a, parts, stream);
}

// ---------------------------------------------------------------------------------------- prologue
//
// Convolution paths, per channel: y_t = sum_j w_j x_{t-j} (w_j = conv[K-1-j], terms inside the
// sequence), s = y sigmoid(y), and for q and k the unit row n s, n = 1 / sqrt(sum s^2 + eps).
// ds = n d - n^3 s (s . d) (v: ds = d); dy = ds sigmoid(y) (1 + y (1 - sigmoid(y)));
// dx_t = sum_j w_j dy_{t+j}, dw_j = sum_t dy_t x_{t-j}, inside the sequence both.
// Gates: alpha = sigmoid(-x), b and w = sigmoid(x): dx = +- d p (1 - p), p = sigmoid(x).
//
// A block holds up to 512 neighbouring channels of one path, 4 per lane, so that d / 4 lanes hold one
// (token, head) row, and walks a run of R tokens forwards.  dx_t is complete once dy_{t+K-1} is known,
// so three unfinished dx and the three previous x stay in registers beside the taps and their
// gradients; each run walks K - 1 tokens further than it writes.  The taps' gradients of a run leave as
// one row of partial sums; within it they are sums of sums over 256 tokens, so that a long run's
// rounding does not grow with its length.
//
// The convolutions are bound by arithmetic (about 125 instructions per lane and token for 16 bytes read
// and 8 written), so the gates, pure streams, are blocks of their own: the runs take seven eighths of the
// SMs' room (three quarters: 119 us, all of it: 118), and the gates' blocks the rest and what the runs
// leave.  1.3B layer 115 us, 604 MB at 5.2 TB/s (the runs alone 100 us, the gates alone 49), in long runs
// 125 us and 4.8 TB/s; 15003 packed tokens x 32 heads, d_v = 256, from 8 bits 517 us, 2474 MB at 4.8 TB/s,
// in long runs 566 us and 4.4 TB/s; the layer in fp32 190 us, 1208 MB at 6.4 TB/s.  ptxas reports small
// spills of the four-tap forms (4 to 40 bytes stored by a thread; none in bf16 from 8 bits) and none of those
// with fewer taps.  What was slower: 8 channels per lane (spills, 185 us), the gates in the
// convolution's lanes (142 us), run length and path varying inside a block, with the norm's lanes known
// only at run time (138 us), shorter runs in several rounds (154 to 184 us), a fifth block per SM (128 us).

constexpr int CT = 128;           // threads of a block, at most
constexpr int CONV_BLOCKS = 4;    // blocks of that many threads per SM
constexpr int GATE_TILES = 32;    // blocks of the gates per SM, at most
constexpr int SUM_BATCHES = 64;   // load batches after which the taps' gradients move to their second level
constexpr int CS = 2;             // load batches in a lane's ring (one is used, the other in flight; a third: no gain)

struct PathBwd {  // a convolution path and the gate that goes with it
  const void *x, *d, *gx, *gd;
  void *dx, *gdx;
  const uint8_t *scales, *gscales;
  const float *W;
  int dim, col;  // col: the path's first column in a row of partial sums
  float sign;        // of the gate's derivative
  int blocks;        // of one run's channels
};
struct ConvBwdArgs {
  PathBwd path[3];
  const int32_t *cu;
  float *parts;  // [runs][ncols]
  int ncols, N, T, H, K, R;
  long long tokens, runs;
  int gate_blocks;
};

// A lane's ring: per batch and token x and d, each [thread].
template <typename T, typename S> struct Ring {
  static constexpr int CU = 4;  // tokens per batch
  static constexpr int XB = CC * (int)sizeof(S), DB = CC * (int)sizeof(T);
  static constexpr int X = 0, D = X + XB * CT, TOKEN = D + DB * CT, BATCH = TOKEN * CU;
};

// Vectors that a lane of the gates has in flight: 128 bytes of each input.
template <typename T> __host__ __device__ constexpr int gate_unroll() { return sizeof(T) == 2 ? 8 : 4; }
// The gates: tiles of U vectors per lane over the three paths end to end, taken in turn by the blocks.
template <typename T, typename S>
__device__ __forceinline__ void gates_bwd(const ConvBwdArgs &a, int block) {
  constexpr bool Q = sizeof(S) == 1;
  constexpr int U = gate_unroll<T>();
  const long long live = a.cu ? min((long long)a.cu[a.N], a.tokens) : a.tokens;
  const int span = blockDim.x * U;
  const long long nk = max(0ll, live) * a.H * (a.path[0].dim / CE), nv = max(0ll, live) * a.H * (a.path[2].dim / CE);
  const long long tk = (nk + span - 1) / span, tiles = 2 * tk + (nv + span - 1) / span;
  for (long long t = block; t < tiles; t += a.gate_blocks) {
    const int k = t < tk ? 0 : t < 2 * tk ? 1 : 2;
    const PathBwd &P = a.path[k];
    const long long b = (t - k * tk) * span;
    const S *x = static_cast<const S *>(P.gx) + b * CE;
    const T *d = static_cast<const T *>(P.gd) + b * CE;
    T *dx = static_cast<T *>(P.gdx) + b * CE;
    const int n = (int)min((k < 2 ? nk : nv) - b, (long long)span);
    Lane<S, CE> rx[U];
    Lane<T, CE> rd[U];
    uint8_t sc[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = u * blockDim.x + threadIdx.x;
      if (i < n) {
        rx[u].load(x + i * CE);
        rd[u].load(d + i * CE);
        if (Q) sc[u] = P.gscales[b / (ACT_GROUP / CE) + i / (ACT_GROUP / CE)];
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = u * blockDim.x + threadIdx.x;
      if (i < n) {
        Pairs<CE> xf, df;
        rx[u].get(xf, Q ? act8_unit(sc[u]) : 0.f);
        rd[u].get(df, 0.f);
        gate_bwd(xf, df, P.sign);
        rd[u].put(df);
        rd[u].store(dx + i * CE);
      }
    }
  }
}

// One block's run of one path; G: lanes of a row whose norm is taken, 0 for a path without one.  FOUR:
// there are four taps; where there are fewer, the others' products are left out, not formed with zeros
// (0 * NaN would carry a NaN to tokens that the taps do not join).  The common four-tap form so pays
// nothing for them.
template <typename T, typename S, int G, bool FOUR>
__device__ __forceinline__ void conv_bwd(const ConvBwdArgs &a, const PathBwd &P, int blk, long long run, uint8_t *ring,
                                         float4 (*far)[CT]) {
  using RB = Ring<T, S>;
  constexpr int CU = RB::CU;
  constexpr bool Q = sizeof(S) == 1;
  const long long t0 = run * a.R;
  const int K = a.K;
  const bool has1 = FOUR || K > 1, has2 = FOUR || K > 2;  // the last tap is there where FOUR
  const unsigned stride = (unsigned)a.H * P.dim;  // elements between tokens; a run's offsets fit 32 bits
  const unsigned ch = (blk * blockDim.x + threadIdx.x) * CC;
  if (ch >= stride) return;  // whole groups leave together
  const int lane = threadIdx.x & 31;
  const unsigned gmask = G == 0 || G == 32 ? 0xffffffffu : ((1u << (G & 31)) - 1u) << (lane & ~(G - 1));
  const long long live = a.cu ? min((long long)a.cu[a.N], a.tokens) : a.tokens;  // rows behind it are not touched
  const size_t at0 = (size_t)t0 * stride;

  Pairs<CC> w[4], dw[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    fill(dw[j], 0.f);
#pragma unroll
    for (int i = 0; i < CC; ++i) w[j].set(i, j < K ? P.W[(size_t)(ch + i) * K + K - 1 - j] : 0.f);
    far[j][threadIdx.x] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  auto second_level = [&] {  // far += dw, a lane's own words only
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float4 s = far[j][threadIdx.x];
      s.x += dw[j].p[0].x;
      s.y += dw[j].p[0].y;
      s.z += dw[j].p[1].x;
      s.w += dw[j].p[1].y;
      far[j][threadIdx.x] = s;
    }
  };
  const int ntok = (int)max(0ll, min((long long)a.R, live - t0));           // tokens of the run
  const int nload = (int)max(0ll, min((long long)a.R + K - 1, live - t0));  // and those its dx reach
  if (ntok > 0) {
    // the sequence holding t0: its first token s0, and the next sequence's start nbr (beyond: none);
    // both relative to t0, as all token indices below
    long long s0, nb;
    int n = 0;
    if (!a.cu) {
      s0 = -(t0 % a.T);
      nb = s0 + a.T;
    } else {
      int lo = 0, hi = a.N - 1;
      while (lo < hi) {  // largest n < N with cu[n] <= t0
        const int mid = (lo + hi + 1) >> 1;
        if (a.cu[mid] <= t0) lo = mid; else hi = mid - 1;
      }
      n = lo;
      s0 = a.cu[n] - t0;
      nb = a.cu[n + 1] - t0;
      if (nb <= 0) nb = INT_MAX;
    }
    int nbr = (int)min(nb, (long long)INT_MAX);
    Pairs<CC> x1, x2, x3, p1, p2, p3;  // x_{t-j}; unfinished dx_{t-j}
    auto clear = [&] {
      fill(x1, 0.f);
      fill(x2, 0.f);
      fill(x3, 0.f);
      fill(p1, 0.f);
      fill(p2, 0.f);
      fill(p3, 0.f);
    };
    clear();
    auto before = [&](int j, Pairs<CC> &f) {
      if (-j < max(s0, -t0)) return;
      const size_t at = at0 + ch - (size_t)j * stride;
      Lane<S, CC> r;
      r.load(static_cast<const S *>(P.x) + at);
      r.get(f, Q ? act8_unit(P.scales[at / ACT_GROUP]) : 0.f);
    };
    before(1, x1);
    before(2, x2);
    before(3, x3);
    const S *const x = static_cast<const S *>(P.x) + at0;
    const T *const d = static_cast<const T *>(P.d) + at0;
    T *const dx = static_cast<T *>(P.dx) + at0;
    const uint8_t *const sc = P.scales + at0 / ACT_GROUP;
    uint8_t ahead[CU];  // scale bytes of the batch in flight
    const int nbatch = (nload + CU - 1) / CU;
    auto issue = [&](int bt) {  // copies of batch bt, committed as one group
      uint8_t *slot = ring + (bt % CS) * RB::BATCH;
#pragma unroll
      for (int u = 0; u < CU; ++u) {
        const int i = bt * CU + u;
        if (i < nload) {
          const unsigned o = (unsigned)i * stride + ch;
          uint8_t *to = slot + u * RB::TOKEN;
          cp_async<RB::XB>(to + RB::X + threadIdx.x * RB::XB, x + o);
          cp_async<RB::DB>(to + RB::D + threadIdx.x * RB::DB, d + o);
          if (Q) ahead[u] = sc[o / ACT_GROUP];
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    int lo = 0;  // first token of the run in the current sequence
    // One token, or two whose sums meet together: nine shuffles instead of twelve, and one's arithmetic
    // fills the other's waits (1.3B layer 115 us; one at a time 118).
    auto token = [&](int i, const uint8_t *from, uint32_t units, auto checked, auto count) {
      constexpr bool CHECK = decltype(checked)::value;
      constexpr int NT = decltype(count)::value;
      Pairs<CC> xt[NT], y[NT], g[NT], ds[NT];
      Lane<T, CC> rd;
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const Pairs<CC> &h1 = t == 1 ? xt[0] : x1, &h2 = t == 1 ? x1 : x2, &h3 = t == 1 ? x2 : x3;
        Lane<S, CC> rx;
        rx.v[0] = *reinterpret_cast<const LaneVec<S, CC> *>(from + t * RB::TOKEN + RB::X + threadIdx.x * RB::XB);
        rd.v[0] = *reinterpret_cast<const LaneVec<T, CC> *>(from + t * RB::TOKEN + RB::D + threadIdx.x * RB::DB);
        rx.get(xt[t], Q ? act8_unit(units >> 8 * t & 255) : 0.f);
        rd.get(g[t], 0.f);
#pragma unroll
        for (int c = 0; c < CC / 2; ++c) {
          float2 v = __fmul2_rn(w[0].p[c], xt[t].p[c]);
          if (has1) v = __ffma2_rn(w[1].p[c], h1.p[c], v);
          if (has2) v = __ffma2_rn(w[2].p[c], h2.p[c], v);
          if (FOUR) v = __ffma2_rn(w[3].p[c], h3.p[c], v);
          const float2 sg = sigmoid2(v);
          y[t].p[c] = __fmul2_rn(v, sg);
          ds[t].p[c] = __ffma2_rn(y[t].p[c], one_minus2(sg), sg);  // derivative of SiLU
        }
      }
      if constexpr (G > 0) {
        // all sums in one pass: even lanes end with sum y^2, odd ones with sum y d, of the first token
        // where lane & 2 is 0
        const bool odd = lane & 1, second = NT == 2 && lane & 2;
        float part[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const float ss = dot(y[t], y[t]), sd = dot(y[t], g[t]);
          part[t] = (odd ? sd : ss) + __shfl_xor_sync(gmask, odd ? ss : sd, 1);
        }
        float s = part[0];
        if constexpr (NT == 2) s = (second ? part[1] : part[0]) + __shfl_xor_sync(gmask, second ? part[0] : part[1], 2);
#pragma unroll
        for (int m = 2 * NT; m < G; m <<= 1) s += __shfl_xor_sync(gmask, s, m);
        const float other = __shfl_xor_sync(gmask, s, 1);
        const float n = rsqrt_approx((odd ? other : s) + L2_EPS), k = -n * n * n * (odd ? s : other);
        float nrm[2] = {n, n}, k3[2] = {k, k};
        if constexpr (NT == 2) {
          const float on = __shfl_xor_sync(gmask, n, 2), ok = __shfl_xor_sync(gmask, k, 2);
          nrm[0] = second ? on : n;
          k3[0] = second ? ok : k;
          nrm[1] = second ? n : on;
          k3[1] = second ? k : ok;
        }
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int c = 0; c < CC / 2; ++c)
            g[t].p[c] = __ffma2_rn(splat(k3[t]), y[t].p[c], __fmul2_rn(splat(nrm[t]), g[t].p[c]));
      }
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const unsigned o = (unsigned)(i + t) * stride + ch;
#pragma unroll
        for (int c = 0; c < CC / 2; ++c) g[t].p[c] = __fmul2_rn(g[t].p[c], ds[t].p[c]);  // dy
        if (!CHECK || i < ntok) {
#pragma unroll
          for (int c = 0; c < CC / 2; ++c) {
            dw[0].p[c] = __ffma2_rn(g[t].p[c], xt[t].p[c], dw[0].p[c]);
            dw[1].p[c] = __ffma2_rn(g[t].p[c], x1.p[c], dw[1].p[c]);
            dw[2].p[c] = __ffma2_rn(g[t].p[c], x2.p[c], dw[2].p[c]);
            dw[3].p[c] = __ffma2_rn(g[t].p[c], x3.p[c], dw[3].p[c]);
          }
        }
#pragma unroll
        for (int c = 0; c < CC / 2; ++c) {
          y[t].p[c] = FOUR ? __ffma2_rn(w[3].p[c], g[t].p[c], p3.p[c]) : p3.p[c];  // dx of the third token before
          p3.p[c] = has2 ? __ffma2_rn(w[2].p[c], g[t].p[c], p2.p[c]) : p2.p[c];
          p2.p[c] = has1 ? __ffma2_rn(w[1].p[c], g[t].p[c], p1.p[c]) : p1.p[c];
          p1.p[c] = __fmul2_rn(w[0].p[c], g[t].p[c]);
        }
        x3 = x2;
        x2 = x1;
        x1 = xt[t];
        if (i + t - 3 >= lo) {
          rd.put(y[t]);
          rd.store(dx + (o - 3 * stride));
        }
      }
    };
    // What is unfinished before token i is complete where its sequence ends at i.
    auto flush = [&](int i) {
      auto put = [&](int j, const Pairs<CC> &f) {
        if (i - j < lo || i - j >= ntok) return;
        Lane<T, CC> r;
        r.put(f);
        r.store(dx + ((unsigned)(i - j) * stride + ch));
      };
      put(3, p3);
      put(2, p2);
      put(1, p1);
    };
#pragma unroll
    for (int bt = 0; bt < CS - 1; ++bt) issue(bt);
    int i = 0;
    bool more = true;
    for (int bt = 0; bt < nbatch && more; ++bt) {
      uint32_t now = 0;  // this batch's scale bytes
      if (Q)
#pragma unroll
        for (int u = 0; u < CU; ++u) now |= (uint32_t)ahead[u] << 8 * u;
      if (bt % SUM_BATCHES == SUM_BATCHES - 1) {
        second_level();
#pragma unroll
        for (int j = 0; j < 4; ++j) fill(dw[j], 0.f);
      }
      issue(bt + CS - 1);  // into the slot that batch bt - 1 used
      asm volatile("cp.async.wait_group %0;" ::"n"(CS - 1) : "memory");
      const int ib = bt * CU;
      const uint8_t *slot = ring + (bt % CS) * RB::BATCH;
      if (ib + CU <= ntok && nbr >= ib + CU) {  // a full batch inside one sequence: no checks
#pragma unroll
        for (int u = 0; u < CU; u += 2)
          token(ib + u, slot + u * RB::TOKEN, now >> 8 * u, std::false_type(), std::integral_constant<int, 2>());
        i = ib + CU;
      } else {
#pragma unroll 1
        for (int u = 0; u < CU; ++u) {
          i = ib + u;
          if (i >= nload) break;
          if (i == nbr) {  // a new sequence starts here (uniform in the group)
            if (i >= ntok) {
              more = false;
              break;
            }
            flush(i);
            lo = i;
            clear();
            if (!a.cu) {
              nbr = (int)min((long long)nbr + a.T, (long long)INT_MAX);
            } else {
              const long long t = t0 + i;
              int m = n + 1;  // cu[m] == t; skip empty sequences
              while (m + 1 < a.N && a.cu[m + 1] <= t) ++m;
              n = m;
              nb = m + 1 <= a.N ? (long long)a.cu[m + 1] : LLONG_MAX;
              nbr = nb <= t ? INT_MAX : (int)min(nb - t0, (long long)INT_MAX);
            }
          }
          token(i, slot + u * RB::TOKEN, now >> 8 * u, std::true_type(), std::integral_constant<int, 1>());
          ++i;
        }
      }
    }
    flush(i);
    asm volatile("cp.async.wait_group 0;" ::: "memory");
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  second_level();
  float *part = a.parts + (size_t)run * a.ncols + P.col + (size_t)ch * K;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float4 q = far[j][threadIdx.x];
    const float s[CC] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int c = 0; c < CC; ++c)
      if (j < K) part[c * K + K - 1 - j] = s[c];
  }
}

template <typename T, typename S, bool FOUR>
__global__ void __launch_bounds__(CT, CONV_BLOCKS) prologue_bwd_kernel(const ConvBwdArgs a) {
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ float4 far[4][CT];
  // the block's run and path; all of it is uniform in the block but the lane's channel
  const int per_run = a.path[0].blocks + a.path[1].blocks + a.path[2].blocks;
  const long long cb = blockIdx.x;
  if (cb >= a.runs * per_run) {
    gates_bwd<T, S>(a, (int)(cb - a.runs * per_run));
    return;
  }
  const long long run = cb / per_run;
  int blk = (int)(cb % per_run), path = 0;
  while (path < 2 && blk >= a.path[path].blocks) blk -= a.path[path++].blocks;
  if (path == 2) conv_bwd<T, S, 0, FOUR>(a, a.path[2], blk, run, ring, far);
  else if (a.path[0].dim == 64) conv_bwd<T, S, 64 / CC, FOUR>(a, a.path[path], blk, run, ring, far);
  else conv_bwd<T, S, 128 / CC, FOUR>(a, a.path[path], blk, run, ring, far);
}

// How the work is cut; the same for the workspace's size and the launch.  Runs are as many as let all
// blocks of CT threads be resident at once (a second round of a few blocks would double the time), each of
// at least four tokens and at most what keeps a run's offsets in 32 bits.  Blocks of fewer threads (heads of
// under 512 channels in all) are counted by their threads, but each takes the shared memory of CT: of one
// head's 16 blocks an SM holds 9 at once in bf16 and 5 in fp32, and such calls run in two to four rounds
// (15003 tokens x 64 in bf16: 29 us, bytes for 5).
struct ConvBwdPlan {
  int threads, blocks[3], R, ncols;
  long long runs;
};
ConvBwdPlan conv_bwd_plan(long long tokens, int H, int dk, int dv, int K) {
  ConvBwdPlan p;
  const long long most = (1ll << 29) / ((long long)H * std::max(dk, dv)) / 4 * 4 - 4;
  const int dim[3] = {dk, dk, dv};
  p.threads = (int)std::min<long long>(CT, ((long long)H * std::max(dk, dv) / CC + 31) / 32 * 32);
  int per_run = 0;
  for (int i = 0; i < 3; ++i) per_run += p.blocks[i] = (H * dim[i] / CC + p.threads - 1) / p.threads;
  const long long slots = (long long)sm_count() * CONV_BLOCKS * (CT / p.threads);
  const long long runs = std::max(1ll, slots * 7 / 8 / per_run), R = ((tokens + runs - 1) / runs + 3) / 4 * 4;
  p.R = (int)std::min(R, most);
  p.runs = (tokens + p.R - 1) / p.R;
  p.ncols = H * (2 * dk + dv) * K;
  return p;
}

template <typename T, typename S, bool FOUR>
cudaError_t prologue_t(const PrologueBwdArgs &p, float *parts, cudaStream_t stream) {
  const ConvBwdPlan pl = conv_bwd_plan(p.tokens, p.H, p.dk, p.dv, p.K);
  const int dim[3] = {p.dk, p.dk, p.dv};
  ConvBwdArgs a{};
  int col = 0;
  ColSumArgs sum{parts, (int)pl.runs, pl.ncols, {}, {}};
  for (int i = 0; i < 3; ++i) {
    const int g = 3 + i;  // alpha with q, b with k, w with v
    a.path[i] = PathBwd{p.x[i], p.d[i], p.x[g], p.d[g], p.dx[i], p.dx[g], p.scales[i], p.scales[g], p.W[i],
                        dim[i], col, i == 0 ? -1.f : 1.f, pl.blocks[i]};
    col += p.H * dim[i] * p.K;
    sum.out[i] = p.dW[i];
    sum.end[i] = col;
  }
  a.cu = p.cu;
  a.parts = parts;
  a.ncols = pl.ncols;
  a.N = p.B;
  a.T = p.T;
  a.H = p.H;
  a.K = p.K;
  a.R = pl.R;
  a.tokens = p.tokens;
  a.runs = pl.runs;
  const long long span = pl.threads * gate_unroll<T>(), rows = p.tokens * p.H;
  const long long tiles = 2 * ((rows * p.dk / CE + span - 1) / span) + (rows * p.dv / CE + span - 1) / span;
  a.gate_blocks = (int)std::min<long long>(tiles, (long long)sm_count() * GATE_TILES);
  constexpr int smem = CS * Ring<T, S>::BATCH;
  static std::atomic<uint64_t> allowed;
  cudaError_t err = allow_smem((const void *)prologue_bwd_kernel<T, S, FOUR>, smem, allowed);
  if (err != cudaSuccess) return err;
  note_launch();
  const long long blocks = pl.runs * (pl.blocks[0] + pl.blocks[1] + pl.blocks[2]);
  prologue_bwd_kernel<T, S, FOUR><<<(unsigned)(blocks + a.gate_blocks), pl.threads, smem, stream>>>(a);
  if ((err = cudaGetLastError()) != cudaSuccess) return err;
  return launch_colsum(sum, stream);
}

template <typename T, typename S>
cudaError_t prologue_t(const PrologueBwdArgs &p, float *parts, cudaStream_t stream) {
  return p.K == 4 ? prologue_t<T, S, true>(p, parts, stream) : prologue_t<T, S, false>(p, parts, stream);
}

}  // namespace

size_t epilogue_bwd_workspace_bytes(long long rows, int dv, bool bf16) {
  const EpiloguePlan p = epilogue_plan(rows, dv, bf16 ? EPI_CHANNELS<__nv_bfloat16> : EPI_CHANNELS<float>);
  return p.cluster ? 0 : (size_t)p.blocks * dv * sizeof(float);
}

cudaError_t launch_epilogue_bwd(const EpilogueBwdArgs &a, bool bf16, void *ws, cudaStream_t stream) {
  float *parts = static_cast<float *>(ws);
  if (a.o_scales)
    return bf16 ? epilogue_t<__nv_bfloat16, int8_t>(a, parts, stream) : epilogue_t<float, int8_t>(a, parts, stream);
  return bf16 ? epilogue_t<__nv_bfloat16, __nv_bfloat16>(a, parts, stream) : epilogue_t<float, float>(a, parts, stream);
}

size_t prologue_bwd_workspace_bytes(long long tokens, int H, int dk, int dv, int K) {
  const ConvBwdPlan p = conv_bwd_plan(tokens, H, dk, dv, K);
  return (size_t)p.runs * p.ncols * sizeof(float);
}

cudaError_t launch_prologue_bwd(const PrologueBwdArgs &a, bool bf16, void *ws, cudaStream_t stream) {
  float *parts = static_cast<float *>(ws);
  if (a.scales[0])
    return bf16 ? prologue_t<__nv_bfloat16, int8_t>(a, parts, stream) : prologue_t<float, int8_t>(a, parts, stream);
  return bf16 ? prologue_t<__nv_bfloat16, __nv_bfloat16>(a, parts, stream) : prologue_t<float, float>(a, parts, stream);
}

}  // namespace gdn2
