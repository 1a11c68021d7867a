// Backward of the work around the mixer in its block: of the output gate behind it (RMS norm times
// SiLU gate) and of the short convolutions, SiLU, L2 norm and gates in front of it.  The forward is
// defined in block.cu; here its inputs are read again (in their type, or held in 8 bits) and what the
// gradients need of the forward is formed anew, in fp32.
#include <algorithm>
#include <climits>

#include "act8.cuh"

namespace gdn2 {
namespace {

constexpr int CE = 8;  // channels per lane
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
// sigmoid(x) = 1 / (1 + 2^(-x log2 e)); 0 and 1 at the far ends.
__device__ __forceinline__ float sigmoid(float x) { return rcp_approx(1.f + ex2_approx(-1.4426950408889634f * x)); }

// The CE channels of a lane, as loaded: 16-byte words in the element type, one 8-byte word of codes.
template <typename S> struct Lane {
  static constexpr int VEC = sizeof(S) == 4 ? 4 : CE;
  LaneVec<S, VEC> v[CE / VEC];
  __device__ __forceinline__ void load(const S *p) {
#pragma unroll
    for (int i = 0; i < CE / VEC; ++i) v[i] = reinterpret_cast<const LaneVec<S, VEC> *>(p)[i];
  }
  __device__ __forceinline__ void store(S *p) const {
#pragma unroll
    for (int i = 0; i < CE / VEC; ++i) reinterpret_cast<LaneVec<S, VEC> *>(p)[i] = v[i];
  }
  __device__ __forceinline__ void get(float (&f)[CE], float unit) const {
#pragma unroll
    for (int i = 0; i < CE / VEC; ++i) {
      float t[VEC];
      if constexpr (sizeof(S) == 1) widen(v[i], unit, t);
      else widen(v[i], t);
#pragma unroll
      for (int k = 0; k < VEC; ++k) f[i * VEC + k] = t[k];
    }
  }
  __device__ __forceinline__ void put(const float (&f)[CE]) {
#pragma unroll
    for (int i = 0; i < CE / VEC; ++i) {
      float t[VEC];
#pragma unroll
      for (int k = 0; k < VEC; ++k) t[k] = f[i * VEC + k];
      narrow(t, v[i]);
    }
  }
};

// Sum over the G lanes of a row (G a power of two, the lanes aligned within their warp).
template <int G>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
  for (int m = 1; m < G; m <<= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
  return x;
}

// ---------------------------------------------------------------------------------------- epilogue
//
// y = oh g s with oh = o r, r = 1 / sqrt(mean o^2 + eps), s = z sigmoid(z).  With e = dy g s:
// do = r (e - oh mean(e oh)), dz = dy g oh sigmoid(z) (1 + z (1 - sigmoid(z))), dg = sum over rows of
// dy oh s.  A row of d_v values is held by G = d_v / 8 lanes, 8 per lane; groups of lanes take rows in
// turn and keep their dg in registers.  HBM-bound: each value is read once and written once.

constexpr int ER = 2;  // rows whose loads a lane has in flight

template <typename T, typename S, int DV>
__global__ void __launch_bounds__(256) epilogue_bwd_kernel(const EpilogueBwdArgs a, float *parts) {
  constexpr int G = DV / CE, GROUPS = 256 / G;
  constexpr bool Q = sizeof(S) == 1;
  __shared__ float red[GROUPS][DV];
  const int grp = threadIdx.x / G, c = (threadIdx.x % G) * CE;
  float g[CE], dg[CE];
#pragma unroll
  for (int i = 0; i < CE; ++i) {
    g[i] = a.g[c + i];
    dg[i] = 0.f;
  }
  const long long step = (long long)gridDim.x * GROUPS * ER;
  for (long long row0 = (long long)blockIdx.x * GROUPS * ER; row0 < a.rows; row0 += step) {
    Lane<S> ro[ER], rz[ER];
    Lane<T> ry[ER];
    float uo[ER], uz[ER];
#pragma unroll
    for (int u = 0; u < ER; ++u) {
      const long long row = row0 + u * GROUPS + grp;
      if (row < a.rows) {
        const size_t at = (size_t)row * DV + c;
        ro[u].load(static_cast<const S *>(a.o) + at);
        rz[u].load(static_cast<const S *>(a.z) + at);
        ry[u].load(static_cast<const T *>(a.dy) + at);
        if (Q) {
          uo[u] = act8_unit(a.o_scales[at / ACT_GROUP]);
          uz[u] = act8_unit(a.z_scales[at / ACT_GROUP]);
        }
      }
    }
#pragma unroll
    for (int u = 0; u < ER; ++u) {
      const long long row = row0 + u * GROUPS + grp;
      const bool live = row < a.rows;
      float o[CE], z[CE], e[CE], ss = 0.f, eo = 0.f;
      if (live) {
        ro[u].get(o, uo[u]);
        rz[u].get(z, uz[u]);
        ry[u].get(e, 0.f);
#pragma unroll
        for (int i = 0; i < CE; ++i) ss = fmaf(o[i], o[i], ss);
      }
      ss = row_sum<G>(ss);
      const float r = rsqrtf(ss * (1.f / DV) + RMS_EPS);
      if (live) {
#pragma unroll
        for (int i = 0; i < CE; ++i) {
          const float sg = sigmoid(z[i]), s = z[i] * sg, oh = o[i] * r, yo = e[i] * oh;
          dg[i] = fmaf(yo, s, dg[i]);
          z[i] = yo * g[i] * fmaf(s, 1.f - sg, sg);  // dz
          e[i] *= g[i] * s;
          eo = fmaf(e[i], oh, eo);
          o[i] = oh;
        }
      }
      eo = row_sum<G>(eo) * (1.f / DV);
      if (live) {
#pragma unroll
        for (int i = 0; i < CE; ++i) e[i] = r * (e[i] - o[i] * eo);
        const size_t at = (size_t)row * DV + c;
        ry[u].put(e);
        ry[u].store(static_cast<T *>(a.dout) + at);
        ry[u].put(z);
        ry[u].store(static_cast<T *>(a.dz) + at);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < CE; ++i) red[grp][c + i] = dg[i];
  __syncthreads();
  for (int k = threadIdx.x; k < DV; k += 256) {
    float s = 0.f;
    for (int w = 0; w < GROUPS; ++w) s += red[w][k];
    parts[(size_t)blockIdx.x * DV + k] = s;
  }
}

int epilogue_blocks(long long rows, int dv) {
  const long long per = (long long)256 / (dv / CE) * ER;
  return (int)std::max<long long>(1, std::min<long long>((rows + per - 1) / per, (long long)sm_count() * 4));
}

template <typename T, typename S>
cudaError_t epilogue_t(const EpilogueBwdArgs &a, float *parts, cudaStream_t stream) {
  const int blocks = epilogue_blocks(a.rows, a.dv);
  note_launch();
  if (a.dv == 64) epilogue_bwd_kernel<T, S, 64><<<blocks, 256, 0, stream>>>(a, parts);
  else if (a.dv == 128) epilogue_bwd_kernel<T, S, 128><<<blocks, 256, 0, stream>>>(a, parts);
  else epilogue_bwd_kernel<T, S, 256><<<blocks, 256, 0, stream>>>(a, parts);
  const cudaError_t err = cudaGetLastError();
  if (err != cudaSuccess) return err;
  return launch_colsum({parts, blocks, a.dv, {a.dg, nullptr, nullptr}, {a.dv, a.dv, a.dv}}, stream);
}

// ---------------------------------------------------------------------------------------- prologue
//
// Convolution paths, per channel: y_t = sum_j w_j x_{t-j} (w_j = conv[K-1-j], terms inside the
// sequence), s = y sigmoid(y), and for q and k the unit row n s, n = 1 / sqrt(sum s^2 + eps).
// ds = n d - n^3 s (s . d) (v: ds = d); dy = ds sigmoid(y) (1 + y (1 - sigmoid(y)));
// dx_t = sum_j w_j dy_{t+j}, dw_j = sum_t dy_t x_{t-j}, inside the sequence both.
//
// A group of d / 8 lanes holds one (token, head) row, 8 channels per lane, and walks a run of R tokens
// of one head forwards.  dx_t is complete once dy_{t+K-1} is known, so three unfinished dx and the
// three previous x stay in registers beside the taps and their gradients; each run walks K - 1 tokens
// further than it writes.  The taps' gradients of a run leave as one row of partial sums.

constexpr int CT = 128;  // threads of a block
constexpr int CS = 3;    // load batches in a lane's ring (two in flight while one is used)

struct ConvBwdPath {
  const void *x;
  const uint8_t *scales;
  const float *W;
  const void *d;
  void *dx;
  int dim, l2, col;  // col: the path's first column in a row of partial sums
  long long blocks;  // of its runs
};
struct GateBwdPath {
  const void *x;
  const uint8_t *scales;
  const void *d;
  void *dx;
  int dim;
  float sign;
};
struct ConvBwdArgs {
  ConvBwdPath conv[3];
  GateBwdPath gate[3];
  const int32_t *cu;
  float *parts;  // [runs][ncols]
  int ncols, N, T, H, K, R;
  long long tokens, runs;
  int gate_blocks;
};

__device__ __forceinline__ void cp_async(void *smem, const void *gmem, int bytes, int src) {
  const uint32_t s = (uint32_t)__cvta_generic_to_shared(smem);
  if (bytes == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(s), "l"(gmem) : "memory");
  else if (bytes == 8) asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(s), "l"(gmem) : "memory");
  else asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(s), "l"(gmem), "r"(src) : "memory");
}

// One batch of a block's ring, [token][word][thread] for each of its arrays.
template <typename T, typename S> struct Ring {
  static constexpr int CU = 16 / (int)sizeof(T) / 2;  // tokens per batch: 4 (bf16), 2 (fp32)
  static constexpr bool Q = sizeof(S) == 1;
  static constexpr int XW = Q ? 1 : CE * (int)sizeof(S) / 16, DW = CE * (int)sizeof(T) / 16;
  static constexpr int XB = Q ? 8 : 16;  // bytes of a word of x
  static constexpr int X = 0, D = X + CU * XW * XB * CT, SC = D + CU * DW * 16 * CT;
  static constexpr int BYTES = SC + (Q ? CU * 4 * CT : 0);
};

// The gates: alpha = sigmoid(-x), b and w = sigmoid(x); each has dx = +- d p (1 - p), p = sigmoid(x),
// formed as 2^-|..| / (1 + 2^-|..|)^2, which neither cancels nor overflows.
template <typename T, typename S>
__device__ void gate_bwd(const ConvBwdArgs &a, int block) {
  constexpr bool Q = sizeof(S) == 1;
  constexpr int U = 2;
  const long long live = a.cu ? min((long long)a.cu[a.N], a.tokens) : a.tokens;
#pragma unroll 1
  for (int k = 0; k < 3; ++k) {
    const GateBwdPath P = k == 0 ? a.gate[0] : k == 1 ? a.gate[1] : a.gate[2];
    const long long nvec = live * a.H * (P.dim / CE);
    for (long long b = (long long)block * (CT * U); b < nvec; b += (long long)a.gate_blocks * (CT * U)) {
      Lane<S> rx[U];
      Lane<T> rd[U];
      float unit[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const long long i = b + u * CT + threadIdx.x;
        if (i < nvec) {
          rx[u].load(static_cast<const S *>(P.x) + i * CE);
          rd[u].load(static_cast<const T *>(P.d) + i * CE);
          if (Q) unit[u] = act8_unit(P.scales[i / (ACT_GROUP / CE)]);
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const long long i = b + u * CT + threadIdx.x;
        if (i < nvec) {
          float x[CE], d[CE];
          rx[u].get(x, unit[u]);
          rd[u].get(d, 0.f);
#pragma unroll
          for (int c = 0; c < CE; ++c) {
            const float e = ex2_approx(-1.4426950408889634f * fabsf(x[c])), p = rcp_approx(1.f + e);
            d[c] *= P.sign * e * p * p;
          }
          rd[u].put(d);
          rd[u].store(static_cast<T *>(P.dx) + i * CE);
        }
      }
    }
  }
}

template <typename T, typename S>
__global__ void __launch_bounds__(CT, 3) prologue_bwd_kernel(const ConvBwdArgs a) {
  using RB = Ring<T, S>;
  constexpr int CU = RB::CU;
  constexpr bool Q = RB::Q;
  extern __shared__ __align__(16) uint8_t ring[];
  long long blk = blockIdx.x;
  int path = 0;
  while (path < 3 && blk >= a.conv[path].blocks) blk -= a.conv[path++].blocks;
  if (path == 3) {
    gate_bwd<T, S>(a, (int)blk);
    return;
  }
  const ConvBwdPath P = path == 0 ? a.conv[0] : path == 1 ? a.conv[1] : a.conv[2];
  const int G = P.dim / CE, K = a.K;
  const long long gid = (blk * CT + threadIdx.x) / G;
  if (gid >= a.runs * a.H) return;  // whole groups leave together
  const int lane = threadIdx.x & 31, gl = lane & (G - 1);
  const unsigned gmask = G == 32 ? 0xffffffffu : ((1u << G) - 1u) << (lane & ~(G - 1));
  const int h = (int)(gid % a.H);
  const long long run = gid / a.H, t0 = run * a.R;
  const long long live = a.cu ? min((long long)a.cu[a.N], a.tokens) : a.tokens;  // rows behind it are not touched
  const size_t stride = (size_t)a.H * P.dim, first = (size_t)t0 * stride + (size_t)h * P.dim + gl * CE;
  const int ch = h * P.dim + gl * CE;
  float *part = a.parts + (size_t)run * a.ncols + P.col + (size_t)ch * K;

  float w[4][CE], dw[4][CE];
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int i = 0; i < CE; ++i) {
      w[j][i] = j < K ? P.W[(size_t)(ch + i) * K + K - 1 - j] : 0.f;
      dw[j][i] = 0.f;
    }
  const int ntok = (int)max(0ll, min((long long)a.R, live - t0));      // tokens of the run
  const int nload = (int)max(0ll, min((long long)a.R + K - 1, live - t0));  // and those its dx reach
  if (ntok > 0) {
    // the sequence holding t0: its first token s0, and the next sequence's start nb (beyond: none)
    long long s0, nb;
    int n = 0;
    if (!a.cu) {
      s0 = t0 - t0 % a.T;
      nb = s0 + a.T;
    } else {
      int lo = 0, hi = a.N - 1;
      while (lo < hi) {  // largest n < N with cu[n] <= t0
        const int mid = (lo + hi + 1) >> 1;
        if (a.cu[mid] <= t0) lo = mid; else hi = mid - 1;
      }
      n = lo;
      s0 = a.cu[n];
      nb = a.cu[n + 1];
      if (nb <= t0) nb = LLONG_MAX;
    }
    const S *x = static_cast<const S *>(P.x);
    const T *d = static_cast<const T *>(P.d) + first;
    T *dx = static_cast<T *>(P.dx) + first;
    float x1[CE], x2[CE], x3[CE], p1[CE], p2[CE], p3[CE];  // x_{t-j}; unfinished dx_{t-j}
#pragma unroll
    for (int i = 0; i < CE; ++i) x1[i] = x2[i] = x3[i] = p1[i] = p2[i] = p3[i] = 0.f;
#pragma unroll
    for (int j = 1; j <= 3; ++j)
      if (t0 - j >= max(s0, 0ll)) {
        const size_t at = first - (size_t)j * stride;
        Lane<S> r;
        r.load(x + at);
        r.get(j == 1 ? x1 : (j == 2 ? x2 : x3), Q ? act8_unit(P.scales[at / ACT_GROUP]) : 0.f);
      }
    const int nbatch = (nload + CU - 1) / CU;
    const size_t scale_end = (size_t)a.tokens * stride / ACT_GROUP;
    auto issue = [&](int bt) {  // copies of batch bt, committed as one group
      uint8_t *slot = ring + (bt % CS) * RB::BYTES;
#pragma unroll
      for (int u = 0; u < CU; ++u) {
        const int i = bt * CU + u;
        if (i < nload) {
          const size_t at = first + (size_t)i * stride;
#pragma unroll
          for (int v = 0; v < RB::XW; ++v)
            cp_async(slot + RB::X + ((u * RB::XW + v) * CT + threadIdx.x) * RB::XB,
                     reinterpret_cast<const uint8_t *>(x + at) + v * RB::XB, RB::XB, RB::XB);
#pragma unroll
          for (int v = 0; v < RB::DW; ++v)
            cp_async(slot + RB::D + ((u * RB::DW + v) * CT + threadIdx.x) * 16,
                     reinterpret_cast<const uint8_t *>(d + (size_t)i * stride) + v * 16, 16, 16);
          if (Q) {  // the aligned word that holds the group's scale byte, up to the array's end
            const size_t sa = at / ACT_GROUP & ~(size_t)3;
            cp_async(slot + RB::SC + (u * CT + threadIdx.x) * 4, P.scales + sa, 4, (int)min((size_t)4, scale_end - sa));
          }
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    int lo = 0;  // first token of the run in the current sequence (relative to t0, as all below)
    int nbr = (int)min(nb - t0, (long long)INT_MAX);
    auto put = [&](int i, const float (&f)[CE]) {
      Lane<T> r;
      r.put(f);
      r.store(dx + (size_t)i * stride);
    };
    auto token = [&](int i, int u, const uint8_t *slot, bool checked) {
      float xt[CE], y[CE], g[CE];
      {
        Lane<S> rx;
        Lane<T> rd;
        float unit = 0.f;
#pragma unroll
        for (int v = 0; v < RB::XW; ++v)
          rx.v[v] = *reinterpret_cast<const LaneVec<S, Lane<S>::VEC> *>(
              slot + RB::X + ((u * RB::XW + v) * CT + threadIdx.x) * RB::XB);
#pragma unroll
        for (int v = 0; v < RB::DW; ++v)
          rd.v[v] = *reinterpret_cast<const LaneVec<T, Lane<T>::VEC> *>(
              slot + RB::D + ((u * RB::DW + v) * CT + threadIdx.x) * 16);
        if (Q) {
          const size_t sa = (first + (size_t)i * stride) / ACT_GROUP;
          unit = act8_unit(slot[RB::SC + (u * CT + threadIdx.x) * 4 + (sa & 3)]);
        }
        rx.get(xt, unit);
        rd.get(g, 0.f);
      }
      float ss = 0.f, sd = 0.f;
      float ds[CE];  // derivative of SiLU at y
#pragma unroll
      for (int c = 0; c < CE; ++c) {
        float v = w[0][c] * xt[c];
        v = fmaf(w[1][c], x1[c], v);
        v = fmaf(w[2][c], x2[c], v);
        v = fmaf(w[3][c], x3[c], v);
        const float sg = sigmoid(v);
        y[c] = v * sg;
        ds[c] = fmaf(y[c], 1.f - sg, sg);
        ss = fmaf(y[c], y[c], ss);
        sd = fmaf(y[c], g[c], sd);
      }
      if (P.l2) {
#pragma unroll
        for (int m = 16; m > 0; m >>= 1)
          if (m < G) {
            ss += __shfl_xor_sync(gmask, ss, m);
            sd += __shfl_xor_sync(gmask, sd, m);
          }
        const float nrm = rsqrtf(ss + L2_EPS), k3 = nrm * nrm * nrm * sd;
#pragma unroll
        for (int c = 0; c < CE; ++c) g[c] = fmaf(-k3, y[c], nrm * g[c]);
      }
#pragma unroll
      for (int c = 0; c < CE; ++c) g[c] *= ds[c];  // dy
      if (!checked || i < ntok) {
#pragma unroll
        for (int c = 0; c < CE; ++c) {
          dw[0][c] = fmaf(g[c], xt[c], dw[0][c]);
          dw[1][c] = fmaf(g[c], x1[c], dw[1][c]);
          dw[2][c] = fmaf(g[c], x2[c], dw[2][c]);
          dw[3][c] = fmaf(g[c], x3[c], dw[3][c]);
        }
      }
#pragma unroll
      for (int c = 0; c < CE; ++c) {
        y[c] = fmaf(w[3][c], g[c], p3[c]);  // dx of the third token before
        p3[c] = fmaf(w[2][c], g[c], p2[c]);
        p2[c] = fmaf(w[1][c], g[c], p1[c]);
        p1[c] = w[0][c] * g[c];
        x3[c] = x2[c];
        x2[c] = x1[c];
        x1[c] = xt[c];
      }
      if (!checked || i - 3 >= lo) put(i - 3, y);
    };
    // What is unfinished before token i is complete where its sequence ends at i.
    auto flush = [&](int i) {
      if (i - 3 >= lo && i - 3 < ntok) put(i - 3, p3);
      if (i - 2 >= lo && i - 2 < ntok) put(i - 2, p2);
      if (i - 1 >= lo && i - 1 < ntok) put(i - 1, p1);
    };
#pragma unroll
    for (int bt = 0; bt < CS - 1; ++bt) issue(bt);
    int i = 0;
    bool more = true;
    for (int bt = 0; bt < nbatch && more; ++bt) {
      issue(bt + CS - 1);  // into the slot that batch bt - 1 used
      asm volatile("cp.async.wait_group %0;" ::"n"(CS - 1) : "memory");
      const int ib = bt * CU;
      const uint8_t *slot = ring + (bt % CS) * RB::BYTES;
      if (ib - 3 >= lo && ib + CU <= ntok && nbr >= ib + CU) {  // a full batch inside one sequence: no checks
#pragma unroll
        for (int u = 0; u < CU; ++u) token(ib + u, u, slot, false);
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
#pragma unroll
            for (int c = 0; c < CE; ++c) x1[c] = x2[c] = x3[c] = p1[c] = p2[c] = p3[c] = 0.f;
            const long long t = t0 + i;
            if (!a.cu) {
              nb += a.T;
            } else {
              int m = n + 1;  // cu[m] == t; skip empty sequences
              while (m + 1 < a.N && a.cu[m + 1] <= t) ++m;
              n = m;
              nb = m + 1 <= a.N ? (long long)a.cu[m + 1] : LLONG_MAX;
              if (nb <= t) nb = LLONG_MAX;
            }
            nbr = (int)min(nb - t0, (long long)INT_MAX);
          }
          token(i, u, slot, true);
          ++i;
        }
      }
    }
    flush(i);
    asm volatile("cp.async.wait_group 0;" ::: "memory");
  }
#pragma unroll
  for (int c = 0; c < CE; ++c)
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (j < K) part[c * K + K - 1 - j] = dw[j][c];
}

// Tokens of a run, so that the convolution paths' lanes fill the resident blocks once: at least one
// load batch, and the same on the host for the workspace's size and the launch.
struct ConvBwdPlan {
  int R;
  long long runs, blocks[3];
  int ncols;
};
ConvBwdPlan conv_bwd_plan(long long tokens, int H, int dk, int dv, int K, bool bf16) {
  ConvBwdPlan p;
  const int CU = bf16 ? 4 : 2;
  const long long lanes = (long long)sm_count() * 3 * CT, work = tokens * H * (long long)(2 * dk + dv) / CE;
  const long long per = (work + lanes - 1) / lanes;
  p.R = (int)std::min<long long>(std::max<long long>((per + CU - 1) / CU * CU, CU), 1 << 20);
  p.runs = (tokens + p.R - 1) / p.R;
  const int dim[3] = {dk, dk, dv};
  for (int i = 0; i < 3; ++i) p.blocks[i] = (p.runs * H * (dim[i] / CE) + CT - 1) / CT;
  p.ncols = H * (2 * dk + dv) * K;
  return p;
}

template <typename T, typename S>
cudaError_t prologue_t(const PrologueBwdArgs &p, float *parts, cudaStream_t stream) {
  const ConvBwdPlan pl = conv_bwd_plan(p.tokens, p.H, p.dk, p.dv, p.K, sizeof(T) == 2);
  const int dim[6] = {p.dk, p.dk, p.dv, p.dk, p.dk, p.dv};
  ConvBwdArgs a{};
  int col = 0;
  ColSumArgs sum{parts, (int)pl.runs, pl.ncols, {}, {}};
  for (int i = 0; i < 3; ++i) {
    a.conv[i] = ConvBwdPath{p.x[i], p.scales[i], p.W[i], p.d[i], p.dx[i], dim[i], i < 2, col, pl.blocks[i]};
    col += p.H * dim[i] * p.K;
    sum.out[i] = p.dW[i];
    sum.end[i] = col;
    a.gate[i] = GateBwdPath{p.x[3 + i], p.scales[3 + i], p.d[3 + i], p.dx[3 + i], dim[3 + i], i == 0 ? -1.f : 1.f};
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
  const long long gvec = p.tokens * p.H * (long long)(std::max(p.dk, p.dv) / CE);
  a.gate_blocks = (int)std::max<long long>(1, std::min<long long>((gvec + 2 * CT - 1) / (2 * CT), (long long)sm_count() * 8));
  constexpr int smem = CS * Ring<T, S>::BYTES;
  cudaError_t err = cudaFuncSetAttribute(prologue_bwd_kernel<T, S>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (err != cudaSuccess) return err;
  const long long blocks = pl.blocks[0] + pl.blocks[1] + pl.blocks[2] + a.gate_blocks;
  note_launch();
  prologue_bwd_kernel<T, S><<<(unsigned)blocks, CT, smem, stream>>>(a);
  if ((err = cudaGetLastError()) != cudaSuccess) return err;
  return launch_colsum(sum, stream);
}

}  // namespace

size_t epilogue_bwd_workspace_bytes(long long rows, int dv) {
  return (size_t)epilogue_blocks(rows, dv) * dv * sizeof(float);
}

cudaError_t launch_epilogue_bwd(const EpilogueBwdArgs &a, bool bf16, void *ws, cudaStream_t stream) {
  float *parts = static_cast<float *>(ws);
  if (a.o_scales)
    return bf16 ? epilogue_t<__nv_bfloat16, int8_t>(a, parts, stream) : epilogue_t<float, int8_t>(a, parts, stream);
  return bf16 ? epilogue_t<__nv_bfloat16, __nv_bfloat16>(a, parts, stream) : epilogue_t<float, float>(a, parts, stream);
}

size_t prologue_bwd_workspace_bytes(long long tokens, int H, int dk, int dv, int K, bool bf16) {
  const ConvBwdPlan p = conv_bwd_plan(tokens, H, dk, dv, K, bf16);
  return (size_t)p.runs * p.ncols * sizeof(float);
}

cudaError_t launch_prologue_bwd(const PrologueBwdArgs &a, bool bf16, void *ws, cudaStream_t stream) {
  float *parts = static_cast<float *>(ws);
  if (a.scales[0])
    return bf16 ? prologue_t<__nv_bfloat16, int8_t>(a, parts, stream) : prologue_t<float, int8_t>(a, parts, stream);
  return bf16 ? prologue_t<__nv_bfloat16, __nv_bfloat16>(a, parts, stream) : prologue_t<float, float>(a, parts, stream);
}

}  // namespace gdn2
