// Activation checkpoints in 8 bits (format: act8.cuh): packing, unpacking, and the column sums that
// finish the weight gradients of the training operators.
//
// Packing and unpacking are HBM-bound streams: each value is read once and written once.  Six tensors of
// the 1.3B layer (100.7 M bf16 values) packed and read back: 98 us in short runs, 100 us in long ones, 610
// MB at 6.1 TB/s, 0.93 of a copy.  What a value costs is conversion: the group's largest is found on the
// bf16 pairs as integers, two to an instruction, and the rounding, the products and the widening run in
// fp32 pairs.
#include <algorithm>
#include <atomic>

#include "act8.cuh"

namespace gdn2 {
namespace {

constexpr int NU = 4;  // vectors that a lane has in flight

// Rows whose width is a multiple of 32: groups lie end to end over the whole tensor, so a lane's
// vector index needs no row.  A block takes tiles of 256 * NU vectors; one tensor per grid row.
template <typename T, int VEC>
__global__ void __launch_bounds__(256) act_pack_flat_kernel(const ActArgs a) {
  constexpr int LPG = ACT_GROUP / VEC;
  const ActTensor &t = a.t[blockIdx.y];
  const long long nvec = t.rows * t.width / VEC;  // a multiple of the lanes of a group
  for (long long b = (long long)blockIdx.x * (256 * NU); b < nvec; b += (long long)gridDim.x * (256 * NU)) {
    const T *x = static_cast<const T *>(t.x) + b * VEC;
    int8_t *codes = t.codes + b * VEC;
    uint8_t *scales = t.scales + b / LPG;
    const int n = (int)min(nvec - b, (long long)(256 * NU));
    LaneVec<T, VEC> r[NU];
#pragma unroll
    for (int u = 0; u < NU; ++u) {
      const int i = u * 256 + threadIdx.x;
      if (i < n) r[u].load(x + i * VEC);
    }
#pragma unroll
    for (int u = 0; u < NU; ++u) {
      const int i = u * 256 + threadIdx.x;
      Pairs<VEC> f;
      widen<0, VEC>(r[u], f);
      uint32_t s;
      const LaneVec<int8_t, VEC> v = act8_encode<0>(r[u], f, i < n, s);
      if (i < n) {
        v.store(codes + i * VEC);
        if (i % LPG == 0) scales[i / LPG] = (uint8_t)s;
      }
    }
  }
}

template <typename T, int VEC>
__global__ void __launch_bounds__(256) act_unpack_flat_kernel(const ActArgs a) {
  constexpr int LPG = ACT_GROUP / VEC;
  const ActTensor &t = a.t[blockIdx.y];
  const long long nvec = t.rows * t.width / VEC;
  for (long long b = (long long)blockIdx.x * (256 * NU); b < nvec; b += (long long)gridDim.x * (256 * NU)) {
    const int8_t *codes = t.codes + b * VEC;
    const uint8_t *scales = t.scales + b / LPG;
    T *x = static_cast<T *>(t.x) + b * VEC;
    const int n = (int)min(nvec - b, (long long)(256 * NU));
    LaneVec<int8_t, VEC> r[NU];
    uint32_t s[NU];
#pragma unroll
    for (int u = 0; u < NU; ++u) {
      const int i = u * 256 + threadIdx.x;
      if (i < n) {
        r[u].load(codes + i * VEC);
        s[u] = scales[i / LPG];
      }
    }
#pragma unroll
    for (int u = 0; u < NU; ++u) {
      const int i = u * 256 + threadIdx.x;
      if (i < n) {
        Pairs<VEC> f;
        widen<0, VEC>(r[u], act8_unit(s[u]), f);
        LaneVec<T, VEC> v;
        narrow<0, VEC>(f, v);
        v.store(x + i * VEC);
      }
    }
  }
}

// How rows of `width` channels are cut into segments of `span` of them, a warp's at a time.  A row may have
// 2^31 - 1 channels: columns, which run past its end by up to a segment, are unsigned.
struct Segments {
  unsigned width, per_row, groups;
  __host__ __device__ Segments(int w, unsigned span)
      : width((unsigned)w), per_row((width + span - 1) / span), groups((width + ACT_GROUP - 1) / ACT_GROUP) {}
};

// Rows that end inside a group but start on 16-byte boundaries: a warp takes 32 * VEC * NU channels of
// one row at a time.
template <typename T, int VEC, bool PACK>
__global__ void __launch_bounds__(256) act_rows_kernel(const ActArgs a) {
  constexpr unsigned SPAN = 32 * VEC * NU;
  const ActTensor &t = a.t[blockIdx.y];
  const Segments g(t.width, SPAN);
  const unsigned lane = threadIdx.x & 31;
  const long long tasks = t.rows * g.per_row, step = (long long)gridDim.x * 8;
  for (long long k = (long long)blockIdx.x * 8 + (threadIdx.x >> 5); k < tasks; k += step) {
    const long long row = k / g.per_row;
    const unsigned c0 = (unsigned)(k - row * g.per_row) * SPAN + lane * VEC;
    T *x = static_cast<T *>(t.x) + (size_t)row * g.width;
    int8_t *codes = t.codes + (size_t)row * g.width;
    uint8_t *scales = t.scales + (size_t)row * g.groups;
    LaneVec<T, VEC> r[NU];
    LaneVec<int8_t, VEC> q[NU];
    uint32_t s[NU];
#pragma unroll
    for (int u = 0; u < NU; ++u) {
      const unsigned c = c0 + u * 32 * VEC;  // VEC divides the width: a vector is inside the row or outside
      if (c < g.width) {
        if constexpr (PACK) {
          r[u].load(x + c);
        } else {
          q[u].load(codes + c);
          s[u] = scales[c / ACT_GROUP];
        }
      }
    }
#pragma unroll
    for (int u = 0; u < NU; ++u) {
      const unsigned c = c0 + u * 32 * VEC;
      Pairs<VEC> f;
      if constexpr (PACK) {
        widen<0, VEC>(r[u], f);
        uint32_t sc;
        const LaneVec<int8_t, VEC> v = act8_encode<0>(r[u], f, c < g.width, sc);
        if (c < g.width) {
          v.store(codes + c);
          if (c % ACT_GROUP == 0) scales[c / ACT_GROUP] = (uint8_t)sc;
        }
      } else if (c < g.width) {
        widen<0, VEC>(q[u], act8_unit(s[u]), f);
        LaneVec<T, VEC> v;
        narrow<0, VEC>(f, v);
        v.store(x + c);
      }
    }
  }
}

// Rows that start anywhere: a warp takes 256 channels of one row at a time, 8 consecutive ones per lane
// (read one by one, through the L1), so that two shuffles settle a group's scale.  The codes leave as
// aligned 4-byte words, each put together from two neighbours; only a segment's ragged ends leave as
// bytes.  (One channel per lane takes five shuffles per channel: 16384 x 1001 bf16, two tensors, 134 us
// with the reading back; this form 89 us, and 76 with unsigned columns.)
template <typename T>
__global__ void __launch_bounds__(256) act_pack_any_kernel(const ActArgs a) {
  constexpr int V = 8, SPAN = 32 * V;
  const ActTensor &t = a.t[blockIdx.y];
  const Segments g(t.width, SPAN);
  const int lane = threadIdx.x & 31;
  const long long tasks = t.rows * g.per_row, step = (long long)gridDim.x * 8;
  for (long long k = (long long)blockIdx.x * 8 + (threadIdx.x >> 5); k < tasks; k += step) {
    const long long row = k / g.per_row;
    const unsigned first = (unsigned)(k - row * g.per_row) * SPAN, c = first + lane * V;
    const T *x = static_cast<const T *>(t.x) + (size_t)row * g.width + c;
    LaneVec<T, V> r;
#pragma unroll
    for (int i = 0; i < V; ++i) r.e[i] = c + i < g.width ? x[i] : T(0.f);
    Pairs<V> f;
    widen<0, V>(r, f);
    uint32_t sc;
    const LaneVec<int8_t, V> q = act8_encode<0>(r, f, true, sc);
    if (c < g.width && c % ACT_GROUP == 0) t.scales[(size_t)row * g.groups + c / ACT_GROUP] = (uint8_t)sc;
    int8_t *out = t.codes + (size_t)row * g.width + first;
    const int n = (int)min((unsigned)SPAN, g.width - first), s = (int)(reinterpret_cast<uintptr_t>(out) & 3);
    const uint32_t w0 = reinterpret_cast<const uint32_t *>(&q)[0], w1 = reinterpret_cast<const uint32_t *>(&q)[1];
    const uint32_t before = __shfl_up_sync(0xffffffffu, w1, 1);
    auto put = [&](int at, uint32_t word) {  // the word of bytes at .. at + 3 of the segment
      if (at >= 0 && at + 4 <= n) {
        *reinterpret_cast<uint32_t *>(out + at) = word;
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (at + i >= 0 && at + i < n) out[at + i] = (int8_t)(word >> 8 * i);
      }
    };
    put(lane * V - s, __funnelshift_rc(before, w0, 32 - 8 * s));
    put(lane * V - s + 4, __funnelshift_rc(w0, w1, 32 - 8 * s));
    if (lane == 31 && s > 0) put(SPAN - s, w1 >> (32 - 8 * s));
  }
}

template <typename T>
__global__ void __launch_bounds__(256) act_unpack_any_kernel(const ActArgs a) {
  constexpr unsigned SPAN = 32 * 2 * NU;
  const ActTensor &t = a.t[blockIdx.y];
  const Segments g(t.width, SPAN);
  const unsigned lane = threadIdx.x & 31;
  const long long tasks = t.rows * g.per_row, step = (long long)gridDim.x * 8;
  for (long long k = (long long)blockIdx.x * 8 + (threadIdx.x >> 5); k < tasks; k += step) {
    const long long row = k / g.per_row;
    const unsigned c0 = (unsigned)(k - row * g.per_row) * SPAN + lane;
    const int8_t *codes = t.codes + (size_t)row * g.width;
    const uint8_t *scales = t.scales + (size_t)row * g.groups;
    T *x = static_cast<T *>(t.x) + (size_t)row * g.width;
    int8_t q[2 * NU];
    uint8_t s[2 * NU];
#pragma unroll
    for (int u = 0; u < 2 * NU; ++u) {
      const unsigned c = c0 + 32 * u;
      if (c < g.width) {
        q[u] = codes[c];
        s[u] = scales[c / ACT_GROUP];
      }
    }
#pragma unroll
    for (int u = 0; u < 2 * NU; ++u) {
      const unsigned c = c0 + 32 * u;
      if (c < g.width) x[c] = from_f32<T>((float)q[u] * act8_unit(s[u]));
    }
  }
}

// Which kernel serves the call: one launch handles tensors of one kind.  16-byte vectors where every
// row starts on one (width * element size a multiple of 16), single values elsewhere.
template <typename T, bool PACK>
cudaError_t act_t(const ActArgs &all, cudaStream_t stream) {
  constexpr int V = 16 / sizeof(T);
  for (int kind = 0; kind < 3; ++kind) {  // 0: whole groups, 1: aligned rows, 2: any width
    ActArgs a{};
    long long most = 0;
    for (int i = 0; i < all.count; ++i) {
      const ActTensor &t = all.t[i];
      const int k = t.width % ACT_GROUP == 0 ? 0 : t.width % V == 0 ? 1 : 2;
      if (k != kind || t.rows == 0) continue;
      a.t[a.count++] = t;
      const long long span = kind < 2 ? 32 * NU * V : 256;
      most = std::max(most, kind == 0 ? (t.rows * t.width + 8 * span - 1) / (8 * span)
                                      : (t.rows * ((t.width + span - 1) / span) + 7) / 8);
    }
    if (a.count == 0) continue;
    const dim3 grid((unsigned)std::min<long long>(most, 1 << 20), a.count);
    note_launch();
    if (kind == 0) {
      if (PACK) act_pack_flat_kernel<T, V><<<grid, 256, 0, stream>>>(a);
      else act_unpack_flat_kernel<T, V><<<grid, 256, 0, stream>>>(a);
    } else if (kind == 1) {
      act_rows_kernel<T, V, PACK><<<grid, 256, 0, stream>>>(a);
    } else {
      if (PACK) act_pack_any_kernel<T><<<grid, 256, 0, stream>>>(a);
      else act_unpack_any_kernel<T><<<grid, 256, 0, stream>>>(a);
    }
    const cudaError_t err = cudaGetLastError();
    if (err != cudaSuccess) return err;
  }
  return cudaSuccess;
}

// Column sums, 3 to 5 us behind the kernel that wrote the rows, most of it the launch and one round trip
// to the L2.  A block sums 32 columns (lane = column): warp w takes the rows w, w + W, ... of its W
// warps, eight loads in flight and added as a tree, then the first warp adds the warps' sums in order.
constexpr int SUM_WARPS = 32;
__global__ void __launch_bounds__(32 * SUM_WARPS) colsum_kernel(const ColSumArgs a) {
  __shared__ float part[SUM_WARPS][32];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, W = blockDim.x >> 5;
  const int col = blockIdx.x * 32 + lane;
  float s = 0.f;
  if (col < a.ncols) {
    const float *p = a.parts + col;
    for (int r = warp; r < a.nparts; r += 8 * W) {
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = r + i * W < a.nparts ? p[(size_t)(r + i * W) * a.ncols] : 0.f;
      s += ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]));
    }
  }
  part[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && col < a.ncols) {
    for (int w = 1; w < W; ++w) s += part[w][lane];
    const int k = col < a.end[0] ? 0 : col < a.end[1] ? 1 : 2;
    if (a.out[k]) a.out[k][col - (k ? a.end[k - 1] : 0)] = s;
  }
}

}  // namespace

int sm_count() {
  static std::atomic<int> known[64];  // by device; 0: not asked yet
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) {
    cudaGetLastError();  // no device: the sizes are host arithmetic only
    return 148;
  }
  if ((sms = known[dev].load(std::memory_order_relaxed)) > 0) return sms;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms <= 0) {
    cudaGetLastError();
    return 148;
  }
  known[dev].store(sms, std::memory_order_relaxed);
  return sms;
}

cudaError_t allow_smem(const void *kernel, int bytes, std::atomic<uint64_t> &devices) {
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  const uint64_t bit = dev >= 0 && dev < 64 ? 1ull << dev : 0;
  if (devices.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (err == cudaSuccess) devices.fetch_or(bit, std::memory_order_relaxed);
  return err;
}

cudaError_t launch_colsum(const ColSumArgs &a, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3((unsigned)((a.ncols + 31) / 32));
  cfg.blockDim = dim3(32 * std::min(SUM_WARPS, (a.nparts + 7) / 8));  // one round of eight loads, or more
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  note_launch();
  return cudaLaunchKernelEx(&cfg, colsum_kernel, a);
}

cudaError_t launch_act_pack(const ActArgs &a, bool bf16, cudaStream_t stream) {
  return bf16 ? act_t<__nv_bfloat16, true>(a, stream) : act_t<float, true>(a, stream);
}

cudaError_t launch_act_unpack(const ActArgs &a, bool bf16, cudaStream_t stream) {
  return bf16 ? act_t<__nv_bfloat16, false>(a, stream) : act_t<float, false>(a, stream);
}

}  // namespace gdn2
