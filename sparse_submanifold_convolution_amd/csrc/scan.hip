// Gated linear recurrence along the rows of ragged samples, and its backward pass.
//
// Per channel, along a sample's rows (from its last row where reversed), with a_t = sigmoid(gate_t):
//   h_t = a_t h_{t-1} + b_t,   b_t = (1 - a_t) x_t  (mix)  or  x_t  (sum),   h before the first row: the sample's h0.
// Backward, with D_t the gradient of h_t and c_t what row t hands to the row before it:
//   D_t = dy_t + c_{t+1},  c_t = a_t D_t,  c past the last row: the gradient of the final state;
//   dx_t = (1 - a_t) D_t  or  D_t,   dgate_t = a_t (1 - a_t) D_t (h_{t-1} - x_t)  or  a_t (1 - a_t) D_t h_{t-1},
//   dh0 = c of the first row.
//
// Both directions compose maps v -> A v + B, which is associative: a thread walks L rows of a 16-byte vector of channels,
// the CL lanes beside it the neighbouring channels; 256 / CL threads deep the workgroup's tile is joined by shuffles and
// LDS, and tiles are joined over the launch.  A sample's first row has A = 0, and A = 0 drops whatever came before it, so
// samples never touch each other, not even through an infinity or a NaN.
//
// States, products and sums are fp32.  The backward pass forms h again from the inputs and the states at the tiles'
// borders, which the forward pass hands out, so y is not read and its rounding does not matter.

#include <hip/hip_runtime.h>

#include "ssc_internal.h"
#include "vec.h"

namespace ssc {

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kScanRows = 8;  // rows a thread walks

struct ScanParams {
  const void *x, *gate, *dy;
  void *y, *dx, *dgate;
  const int32_t* off;
  const float *h0, *dlast;
  float *last, *dh0;
  float* carries;  // [tiles][C]: h before each tile's first row
  float2* agg;     // [tiles][C]: a tile's map (A, B)
  float* back;     // [tiles][C], backward: c behind each tile's last row
  int64_t n, x_row, gate_row;
  int32_t c, batch, tiles, groups, rev;
};

// What a row is, from its sample: the sample's number times 4, with kFirst and kLast; kNone outside of all samples.
constexpr int kFirst = 1, kLast = 2, kNone = -1;

__device__ __forceinline__ int row_info(const ScanParams& p, int64_t t) {
  if (t >= p.n) return kNone;
  const int row = int(p.rev ? p.n - 1 - t : t);
  // the last sample that does not begin past the row; empty ones before it begin there as well
  int lo = 0, hi = p.batch;  // off[lo] <= row < off[hi], were both so
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (p.off[mid] <= row)
      lo = mid;
    else
      hi = mid;
  }
  int begin = p.off[lo], end = p.off[lo + 1];
  begin = begin < 0 ? 0 : begin;
  end = end > p.n ? int(p.n) : end;
  if (row < begin || row >= end) return kNone;
  const int first = p.rev ? end - 1 : begin, last = p.rev ? begin : end - 1;
  return 4 * lo + (row == first ? kFirst : 0) + (row == last ? kLast : 0);
}

// sigmoid(g) as its smaller side q in [0, 1/2], with the sign of g: q = e / (1 + e), e = exp(-|g|).  One side of the pair
// (a, 1 - a) is q and the other 1 - q, so both keep their relative error however near to 0 or 1 they are.
template <typename T>
__device__ __forceinline__ float gate_side(float g) {
  float q;
  if constexpr (sizeof(T) == 4) {
    const float e = expf(-fabsf(g));
    q = e / (1.f + e);
  } else {
    // the hardware's exponential and reciprocal, off by 2^-22 or so: a 16-bit gate is itself known to 2^-11 at best
    const float e = __builtin_amdgcn_exp2f(-fabsf(g) * kLog2e);
    q = e * __builtin_amdgcn_rcpf(1.f + e);
  }
  return __uint_as_float(__float_as_uint(q) | (__float_as_uint(g) & 0x80000000u));
}
__device__ __forceinline__ float decay_of(float side) {
  const float q = fabsf(side);
  return int(__float_as_uint(side)) < 0 ? q : 1.f - q;
}
__device__ __forceinline__ float keep_of(float side) {
  const float q = fabsf(side);
  return int(__float_as_uint(side)) < 0 ? 1.f - q : q;
}

// The map (A, B) of a value, and its factor after an earlier map's: A = 0 drops what came before, a NaN among it too
__device__ __forceinline__ float after(float A, float B, float v) { return A == 0.f ? B : fmaf(A, v, B); }
__device__ __forceinline__ float times(float A, float a) { return A == 0.f ? 0.f : A * a; }

template <int CL, int V>
struct Tile {
  static constexpr int kChunks = 256 / CL, kRows = kChunks * kScanRows;
  // Joins the threads' maps along the rows (BACK: against them): on return (A, B) is the map of the wave's threads before
  // this one, and tot holds each wave's.
  template <bool BACK>
  __device__ static __forceinline__ void join(float (&A)[V], float (&B)[V], float (*tot)[2][CL * V]) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, col = threadIdx.x % CL;
#pragma unroll
    for (int d = CL; d < 64; d <<= 1)
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float a = BACK ? __shfl_down(A[v], d) : __shfl_up(A[v], d);
        const float b = BACK ? __shfl_down(B[v], d) : __shfl_up(B[v], d);
        if (BACK ? lane + d < 64 : lane >= d) {
          B[v] = after(A[v], B[v], b);
          A[v] = times(A[v], a);
        }
      }
    if (BACK ? lane < CL : lane >= 64 - CL)
#pragma unroll
      for (int v = 0; v < V; ++v) {
        tot[wave][0][col * V + v] = A[v];
        tot[wave][1][col * V + v] = B[v];
      }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const float a = BACK ? __shfl_down(A[v], CL) : __shfl_up(A[v], CL);
      const float b = BACK ? __shfl_down(B[v], CL) : __shfl_up(B[v], CL);
      const bool some = BACK ? lane + CL < 64 : lane >= CL;
      A[v] = some ? a : 1.f;
      B[v] = some ? b : 0.f;
    }
  }
  // the value that reaches this thread's rows, from what reaches the tile
  template <bool BACK>
  __device__ static __forceinline__ void enter(float (&v)[V], const float (&A)[V], const float (&B)[V],
                                               const float (*tot)[2][CL * V]) {
    const int wave = threadIdx.x >> 6, col = threadIdx.x % CL;
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      const int w = BACK ? 3 - i : i;
      if (BACK ? w > wave : w < wave)
#pragma unroll
        for (int k = 0; k < V; ++k) v[k] = after(tot[w][0][col * V + k], tot[w][1][col * V + k], v[k]);
    }
#pragma unroll
    for (int k = 0; k < V; ++k) v[k] = after(A[k], B[k], v[k]);
  }
  // the whole tile's map, channel by channel
  template <bool BACK>
  __device__ static __forceinline__ float2 whole(const float (*tot)[2][CL * V], int ch) {
    float A = 1.f, B = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int w = BACK ? 3 - i : i;
      const float a = tot[w][0][ch], b = tot[w][1][ch];
      B = after(a, b, B);
      A = times(a, A);
    }
    return make_float2(A, B);
  }
};

template <int V>
__device__ __forceinline__ void load_state(const float* src, float (&f)[V]) {
#pragma unroll
  for (int v = 0; v < V; v += 4) {
    const float4 q = *reinterpret_cast<const float4*>(src + v);
    f[v] = q.x;
    f[v + 1] = q.y;
    f[v + 2] = q.z;
    f[v + 3] = q.w;
  }
}
template <int V>
__device__ __forceinline__ void store_state(float* dst, const float (&f)[V]) {
#pragma unroll
  for (int v = 0; v < V; v += 4) *reinterpret_cast<float4*>(dst + v) = make_float4(f[v], f[v + 1], f[v + 2], f[v + 3]);
}

// Samples with no rows hand on the state (or its gradient) that reaches them; the tiles share them out.
template <int CL, int V>
__device__ __forceinline__ void empty_samples(const ScanParams& p, int tile, int c0, bool mine, const float* from, float* to) {
  constexpr int CH = 256 / CL;
  if (!to || !mine) return;
  for (int64_t b = int64_t(tile) * CH + threadIdx.x / CL; b < p.batch; b += int64_t(p.tiles) * CH) {
    int begin = p.off[b], end = p.off[b + 1];
    begin = begin < 0 ? 0 : begin;
    end = end > p.n ? int(p.n) : end;
    if (begin < end) continue;
    float f[V];
#pragma unroll
    for (int v = 0; v < V; ++v) f[v] = 0.f;
    if (from) load_state(from + b * p.c + c0, f);
    store_state(to + b * p.c + c0, f);
  }
}

// SUM: only the tile's map is formed (to p.agg).  Otherwise y and the final states, from the states in p.carries.
template <typename T, int CL, bool MIX, bool SUM>
__global__ void __launch_bounds__(256, 2) scan_fwd(ScanParams p) {
  constexpr int V = Vec<T>::N, L = kScanRows;
  using TL = Tile<CL, V>;
  __shared__ int info[TL::kRows];
  __shared__ float tot[4][2][CL * V];
  const int group = blockIdx.x % p.groups, tile = blockIdx.x / p.groups;
  const int chunk = threadIdx.x / CL, c0 = (group * CL + threadIdx.x % CL) * V;
  const bool mine = c0 < p.c;
  const int64_t t0 = int64_t(tile) * TL::kRows + chunk * L;
  u32x4 xv[L], gv[L];
#pragma unroll
  for (int i = 0; i < L; ++i) {
    xv[i] = gv[i] = u32x4{0, 0, 0, 0};
    if (mine && t0 + i < p.n) {
      const int64_t row = p.rev ? p.n - 1 - (t0 + i) : t0 + i;
      xv[i] = *reinterpret_cast<const u32x4*>(static_cast<const T*>(p.x) + row * p.x_row + c0);
      gv[i] = *reinterpret_cast<const u32x4*>(static_cast<const T*>(p.gate) + row * p.gate_row + c0);
    }
  }
  for (int r = threadIdx.x; r < TL::kRows; r += 256) info[r] = row_info(p, int64_t(tile) * TL::kRows + r);
  __syncthreads();

  float a[L][V], b[L][V], A[V], B[V];
#pragma unroll
  for (int v = 0; v < V; ++v) A[v] = 1.f, B[v] = 0.f;
#pragma unroll
  for (int i = 0; i < L; ++i) {
    const int what = info[chunk * L + i];
    float g[V], x[V];
    Vec<T>::unpack(gv[i], g);
    Vec<T>::unpack(xv[i], x);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const float side = gate_side<T>(g[v]);
      a[i][v] = decay_of(side);
      b[i][v] = MIX ? keep_of(side) * x[v] : x[v];
    }
    if (what == kNone || (what & kFirst)) {
      float h[V];
#pragma unroll
      for (int v = 0; v < V; ++v) h[v] = 0.f;
      if (what != kNone && p.h0 && mine) load_state(p.h0 + int64_t(what >> 2) * p.c + c0, h);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        b[i][v] = what == kNone ? 0.f : (p.h0 ? fmaf(a[i][v], h[v], b[i][v]) : b[i][v]);
        a[i][v] = 0.f;
        A[v] = 0.f;
        B[v] = 0.f;
      }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      B[v] = fmaf(a[i][v], B[v], b[i][v]);
      A[v] *= a[i][v];
    }
  }
  TL::template join<false>(A, B, tot);
  __syncthreads();
  if constexpr (SUM) {
    for (int ch = threadIdx.x; ch < CL * V; ch += 256) {
      const int c = group * CL * V + ch;
      if (c < p.c) p.agg[int64_t(tile) * p.c + c] = TL::template whole<false>(tot, ch);
    }
  } else {
    empty_samples<CL, V>(p, tile, c0, mine, p.h0, p.last);
    float h[V];
#pragma unroll
    for (int v = 0; v < V; ++v) h[v] = 0.f;
    if (p.tiles > 1 && mine) load_state(p.carries + int64_t(tile) * p.c + c0, h);
    TL::template enter<false>(h, A, B, tot);
#pragma unroll
    for (int i = 0; i < L; ++i) {
      const int what = info[chunk * L + i];
      if (what == kNone || (what & kFirst))
#pragma unroll
        for (int v = 0; v < V; ++v) h[v] = 0.f;
#pragma unroll
      for (int v = 0; v < V; ++v) h[v] = fmaf(a[i][v], h[v], b[i][v]);
      if (!mine || t0 + i >= p.n) continue;
      const int64_t row = p.rev ? p.n - 1 - (t0 + i) : t0 + i;
      *reinterpret_cast<u32x4*>(static_cast<T*>(p.y) + row * p.c + c0) = Vec<T>::pack(h);
      if (what != kNone && (what & kLast)) store_state(p.last + int64_t(what >> 2) * p.c + c0, h);
    }
  }
}

// SUM: the tile's map of c (from its end to its beginning) to p.agg.  Otherwise the gradients, from the states in
// p.carries and the c in p.back.
template <typename T, int CL, bool MIX, bool SUM>
__global__ void __launch_bounds__(256, 2) scan_bwd(ScanParams p) {
  constexpr int V = Vec<T>::N, L = kScanRows;
  using TL = Tile<CL, V>;
  __shared__ int info[TL::kRows];
  __shared__ float tot[4][2][CL * V], totb[4][2][CL * V];
  const int group = blockIdx.x % p.groups, tile = blockIdx.x / p.groups;
  const int chunk = threadIdx.x / CL, c0 = (group * CL + threadIdx.x % CL) * V;
  const bool mine = c0 < p.c;
  const int64_t t0 = int64_t(tile) * TL::kRows + chunk * L;
  u32x4 xv[SUM ? 1 : L], gv[L], uv[L];
#pragma unroll
  for (int i = 0; i < L; ++i) {
    gv[i] = uv[i] = u32x4{0, 0, 0, 0};
    if constexpr (!SUM) xv[i] = u32x4{0, 0, 0, 0};
    if (mine && t0 + i < p.n) {
      const int64_t row = p.rev ? p.n - 1 - (t0 + i) : t0 + i;
      gv[i] = *reinterpret_cast<const u32x4*>(static_cast<const T*>(p.gate) + row * p.gate_row + c0);
      uv[i] = *reinterpret_cast<const u32x4*>(static_cast<const T*>(p.dy) + row * p.c + c0);
      if constexpr (!SUM) xv[i] = *reinterpret_cast<const u32x4*>(static_cast<const T*>(p.x) + row * p.x_row + c0);
    }
  }
  for (int r = threadIdx.x; r < TL::kRows; r += 256) info[r] = row_info(p, int64_t(tile) * TL::kRows + r);
  __syncthreads();

  float side[L][V], u[SUM ? 1 : L][V], A[V], B[V];
#pragma unroll
  for (int i = 0; i < L; ++i) {
    float g[V];
    Vec<T>::unpack(gv[i], g);
#pragma unroll
    for (int v = 0; v < V; ++v) side[i][v] = gate_side<T>(g[v]);
  }
  // what a row adds to c where the sample ends with it
  auto end_of = [&](int what, float (&f)[V]) {
#pragma unroll
    for (int v = 0; v < V; ++v) f[v] = 0.f;
    if (what != kNone && p.dlast && mine) load_state(p.dlast + int64_t(what >> 2) * p.c + c0, f);
  };
  float Ab[V], Bb[V];
#pragma unroll
  for (int v = 0; v < V; ++v) Ab[v] = 1.f, Bb[v] = 0.f;
#pragma unroll
  for (int i = L - 1; i >= 0; --i) {
    const int what = info[chunk * L + i];
    float dy[V];
    Vec<T>::unpack(uv[i], dy);
    if (what == kNone || (what & kLast)) {
      end_of(what, Bb);
#pragma unroll
      for (int v = 0; v < V; ++v) Ab[v] = 0.f;
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const float a = what == kNone ? 0.f : decay_of(side[i][v]);
      Bb[v] = what == kNone ? 0.f : a * (dy[v] + Bb[v]);
      Ab[v] *= a;
    }
  }
  TL::template join<true>(Ab, Bb, totb);
  if constexpr (SUM) {
    __syncthreads();
    for (int ch = threadIdx.x; ch < CL * V; ch += 256) {
      const int c = group * CL * V + ch;
      if (c < p.c) p.agg[int64_t(tile) * p.c + c] = TL::template whole<true>(totb, ch);
    }
  } else {
    // the states again
#pragma unroll
    for (int v = 0; v < V; ++v) A[v] = 1.f, B[v] = 0.f;
    auto first_of = [&](int what, float (&f)[V]) {
#pragma unroll
      for (int v = 0; v < V; ++v) f[v] = 0.f;
      if (what != kNone && p.h0 && mine) load_state(p.h0 + int64_t(what >> 2) * p.c + c0, f);
    };
#pragma unroll
    for (int i = 0; i < L; ++i) {
      const int what = info[chunk * L + i];
      float x[V];
      Vec<T>::unpack(xv[i], x);
      if (what == kNone || (what & kFirst)) {
        first_of(what, B);
#pragma unroll
        for (int v = 0; v < V; ++v) A[v] = 0.f;
      }
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float a = what == kNone ? 0.f : decay_of(side[i][v]);
        B[v] = what == kNone ? 0.f : fmaf(a, B[v], MIX ? keep_of(side[i][v]) * x[v] : x[v]);
        A[v] *= a;
      }
    }
    TL::template join<false>(A, B, tot);
    __syncthreads();
    empty_samples<CL, V>(p, tile, c0, mine, p.dlast, p.dh0);
    float h[V], c[V];
#pragma unroll
    for (int v = 0; v < V; ++v) h[v] = c[v] = 0.f;
    if (p.tiles > 1 && mine) {
      load_state(p.carries + int64_t(tile) * p.c + c0, h);
      load_state(p.back + int64_t(tile) * p.c + c0, c);
    }
    TL::template enter<false>(h, A, B, tot);
    TL::template enter<true>(c, Ab, Bb, totb);
#pragma unroll
    for (int i = 0; i < L; ++i) {
      const int what = info[chunk * L + i];
      float x[V];
      Vec<T>::unpack(xv[i], x);
      if (what == kNone || (what & kFirst)) first_of(what, h);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        u[i][v] = MIX ? h[v] - x[v] : h[v];
        h[v] = what == kNone ? 0.f : fmaf(decay_of(side[i][v]), h[v], MIX ? keep_of(side[i][v]) * x[v] : x[v]);
      }
    }
#pragma unroll
    for (int i = L - 1; i >= 0; --i) {
      const int what = info[chunk * L + i];
      float dy[V], dx[V], dg[V];
      Vec<T>::unpack(uv[i], dy);
      if (what == kNone || (what & kLast)) end_of(what, c);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float q = fabsf(side[i][v]), d = dy[v] + c[v];
        dx[v] = what == kNone ? 0.f : (MIX ? keep_of(side[i][v]) * d : d);
        dg[v] = what == kNone ? 0.f : q * (1.f - q) * d * u[i][v];
        c[v] = decay_of(side[i][v]) * d;
      }
      if (!mine || t0 + i >= p.n) continue;
      const int64_t row = p.rev ? p.n - 1 - (t0 + i) : t0 + i;
      *reinterpret_cast<u32x4*>(static_cast<T*>(p.dx) + row * p.c + c0) = Vec<T>::pack(dx);
      *reinterpret_cast<u32x4*>(static_cast<T*>(p.dgate) + row * p.c + c0) = Vec<T>::pack(dg);
      if (p.dh0 && what != kNone && (what & kFirst)) store_state(p.dh0 + int64_t(what >> 2) * p.c + c0, c);
    }
  }
}

// What reaches each tile, from the tiles' maps: a thread a channel
template <bool BACK>
__global__ void __launch_bounds__(64) scan_tiles(const float2* agg, float* into, int tiles, int c) {
  const int ch = blockIdx.x * 64 + threadIdx.x;
  if (ch >= c) return;
  float v = 0.f;
#pragma unroll 8
  for (int i = 0; i < tiles; ++i) {
    const int64_t at = int64_t(BACK ? tiles - 1 - i : i) * c + ch;
    into[at] = v;
    const float2 m = agg[at];
    v = after(m.x, m.y, v);
  }
}

int esize(int32_t dtype) { return dtype == SSC_F32 ? 4 : 2; }
bool bad(const void* ptr) { return !ptr || !aligned16(ptr); }

struct ScanPlan {
  int lanes;  // a row's vectors side by side in a workgroup
  int64_t tiles, groups;
};
ScanPlan scan_plan(const ssc_scan_shape& a) {
  const int vecs = a.channels * esize(a.dtype) / 16;
  ScanPlan s{};
  s.lanes = vecs <= 4 ? 4 : (vecs <= 8 ? 8 : 16);
  const int64_t rows = int64_t(256 / s.lanes) * kScanRows;
  s.tiles = a.n > 0 ? (a.n + rows - 1) / rows : 1;
  s.groups = (vecs + s.lanes - 1) / s.lanes;
  return s;
}

int scan_check(const ssc_scan_shape* a) {
  if (!a) return SSC_ERR_INVALID_ARG;
  if (a->dtype != SSC_F32 && a->dtype != SSC_F16 && a->dtype != SSC_BF16) return SSC_ERR_UNSUPPORTED;
  if (a->n < 0 || a->n > SSC_MAX_SEQ_ROWS || a->channels < 1 || a->batch < 1 || a->batch > SSC_MAX_ATTN_BATCH)
    return SSC_ERR_INVALID_ARG;
  const int vec = 16 / esize(a->dtype);
  if (a->channels > SSC_MAX_SEQ_CHANNELS || a->channels % vec != 0) return SSC_ERR_UNSUPPORTED;
  if (a->form != SSC_SCAN_MIX && a->form != SSC_SCAN_SUM) return SSC_ERR_UNSUPPORTED;
  for (int64_t v : {a->x_row_stride, a->gate_row_stride})
    if (v < 0 || v > (1LL << 40) || v % vec != 0) return SSC_ERR_INVALID_ARG;
  const ScanPlan s = scan_plan(*a);
  // HIP takes fewer than 2^32 threads in a dimension of a launch
  return s.tiles * s.groups * 256 < (1LL << 32) ? SSC_OK : SSC_ERR_UNSUPPORTED;
}

ScanParams scan_params(const ssc_scan_shape& a, const ScanPlan& s) {
  ScanParams p{};
  p.n = a.n;
  p.x_row = a.x_row_stride;
  p.gate_row = a.gate_row_stride;
  p.c = a.channels;
  p.batch = a.batch;
  p.tiles = int32_t(s.tiles);
  p.groups = int32_t(s.groups);
  p.rev = a.reverse != 0;
  return p;
}

size_t carry_bytes(const ssc_scan_shape& a) {
  const ScanPlan s = scan_plan(a);
  return size_t(s.tiles) * size_t(a.channels) * 4;
}

struct ScanWs {
  size_t agg = 0, into = 0, total = 0;
};
ScanWs scan_ws(const ssc_scan_shape& a) {
  const size_t n = align_up(carry_bytes(a), 256);
  ScanWs w;
  w.into = 2 * n;
  w.total = 3 * n;
  return w;
}

template <typename T, int CL, bool MIX>
void scan_launch(const ScanParams& p, bool back, hipStream_t s) {
  const unsigned grid = unsigned(int64_t(p.tiles) * p.groups), per = unsigned((p.c + 63) / 64);
  if (!back) {
    if (p.tiles > 1) {
      scan_fwd<T, CL, MIX, true><<<grid, 256, 0, s>>>(p);
      scan_tiles<false><<<per, 64, 0, s>>>(p.agg, p.carries, p.tiles, p.c);
    }
    scan_fwd<T, CL, MIX, false><<<grid, 256, 0, s>>>(p);
  } else {
    if (p.tiles > 1) {
      scan_bwd<T, CL, MIX, true><<<grid, 256, 0, s>>>(p);
      scan_tiles<true><<<per, 64, 0, s>>>(p.agg, p.back, p.tiles, p.c);
    }
    scan_bwd<T, CL, MIX, false><<<grid, 256, 0, s>>>(p);
  }
}

template <typename T, int CL>
void scan_form(const ScanParams& p, bool mix, bool back, hipStream_t s) {
  if (mix)
    scan_launch<T, CL, true>(p, back, s);
  else
    scan_launch<T, CL, false>(p, back, s);
}

template <typename T>
void scan_lanes(const ScanParams& p, int lanes, bool mix, bool back, hipStream_t s) {
  if (lanes == 4)
    scan_form<T, 4>(p, mix, back, s);
  else if (lanes == 8)
    scan_form<T, 8>(p, mix, back, s);
  else
    scan_form<T, 16>(p, mix, back, s);
}

int scan_run(const ssc_scan_shape& a, const ScanPlan& sp, const ScanParams& p, bool back, void* stream) {
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  const bool mix = a.form == SSC_SCAN_MIX;
  (void)hipGetLastError();
  if (a.dtype == SSC_F32)
    scan_lanes<float>(p, sp.lanes, mix, back, s);
  else if (a.dtype == SSC_F16)
    scan_lanes<_Float16>(p, sp.lanes, mix, back, s);
  else
    scan_lanes<__bf16>(p, sp.lanes, mix, back, s);
  return hipGetLastError() == hipSuccess ? SSC_OK : SSC_ERR_HIP;
}

}  // namespace

}  // namespace ssc

using namespace ssc;

extern "C" size_t ssc_gated_scan_carry_bytes(const ssc_scan_shape* shape) {
  return scan_check(shape) == SSC_OK ? carry_bytes(*shape) : 0;
}

extern "C" size_t ssc_gated_scan_workspace_bytes(const ssc_scan_shape* shape) {
  return scan_check(shape) == SSC_OK ? scan_ws(*shape).total : 0;
}

extern "C" int ssc_gated_scan_fwd(const ssc_scan_shape* shape, const void* x, const void* gate, const int32_t* offsets,
                                  const float* h0, void* y, float* last, float* carries, void* workspace,
                                  size_t workspace_bytes, void* stream) {
  const int st = scan_check(shape);
  if (st != SSC_OK) return st;
  const ssc_scan_shape& a = *shape;
  if (a.n > 0 && (bad(x) || bad(gate) || bad(y))) return SSC_ERR_INVALID_ARG;
  if (bad(offsets) || bad(last) || !aligned16(h0) || !aligned16(carries) || bad(workspace)) return SSC_ERR_INVALID_ARG;
  const ScanWs w = scan_ws(a);
  if (workspace_bytes < w.total) return SSC_ERR_WORKSPACE;
  const ScanPlan sp = scan_plan(a);
  ScanParams p = scan_params(a, sp);
  char* ws = static_cast<char*>(workspace);
  p.x = x;
  p.gate = gate;
  p.off = offsets;
  p.h0 = h0;
  p.y = y;
  p.last = last;
  p.agg = reinterpret_cast<float2*>(ws + w.agg);
  p.carries = carries ? carries : reinterpret_cast<float*>(ws + w.into);
  return scan_run(a, sp, p, false, stream);
}

extern "C" int ssc_gated_scan_bwd(const ssc_scan_shape* shape, const void* x, const void* gate, const float* carries,
                                  const void* dy, const int32_t* offsets, const float* h0, const float* dlast, void* dx,
                                  void* dgate, float* dh0, void* workspace, size_t workspace_bytes, void* stream) {
  const int st = scan_check(shape);
  if (st != SSC_OK) return st;
  const ssc_scan_shape& a = *shape;
  if (a.n > 0 && (bad(x) || bad(gate) || bad(dy) || bad(dx) || bad(dgate))) return SSC_ERR_INVALID_ARG;
  if (bad(offsets) || bad(carries) || !aligned16(h0) || !aligned16(dlast) || !aligned16(dh0) || bad(workspace))
    return SSC_ERR_INVALID_ARG;
  const ScanWs w = scan_ws(a);
  if (workspace_bytes < w.total) return SSC_ERR_WORKSPACE;
  const ScanPlan sp = scan_plan(a);
  ScanParams p = scan_params(a, sp);
  char* ws = static_cast<char*>(workspace);
  p.x = x;
  p.gate = gate;
  p.dy = dy;
  p.off = offsets;
  p.h0 = h0;
  p.dlast = dlast;
  p.dx = dx;
  p.dgate = dgate;
  p.dh0 = dh0;
  p.agg = reinterpret_cast<float2*>(ws + w.agg);
  p.back = reinterpret_cast<float*>(ws + w.into);
  p.carries = const_cast<float*>(carries);
  return scan_run(a, sp, p, true, stream);
}
