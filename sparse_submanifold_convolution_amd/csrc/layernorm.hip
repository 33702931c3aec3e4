// Layer norm of feature rows, with the sum of a residual stream and dropout in the same pass, its backward pass, and
// dropout by itself.
//
// Forward, per row of C channels:  s = x  or  s = residual + dropout(x);
//   mean = sum s / C,  r = 1 / sqrt(sum (s - mean)^2 / C + eps),  y = (s - mean) r w + b.
// Backward, with z = (s - mean) r and g = dy w:
//   ds = r (g - mean g - z mean(g z)) [+ the output gradient of s],  dx = ds through the same dropout,
//   dw = sum over rows of dy z,  db = sum over rows of dy.
//
// L lanes own a row (a part of a wave, a wave, or a workgroup of 256 for rows of over 4 KiB), V 16-byte vectors a lane,
// so a row is read once and its mean, its centred sum of squares and its result are formed from registers: the variance
// is a sum of squares of differences, which rows far from zero keep exact.  Statistics are formed again in the backward
// pass, which holds the whole row anyway, so nothing but s is kept between the passes.  y is formed from s before it is
// rounded; the backward pass reads s as rounded, whose error of half a step is no more than that of its other inputs.
// Sums are fp32, results are rounded once, and the weight gradients are summed in a fixed order.

#include <hip/hip_runtime.h>

#include "dropout.h"
#include "ssc_internal.h"
#include "vec.h"

namespace ssc {

namespace {

struct NormParams {
  const void *x, *res, *w, *b, *dy, *ds;
  void *y, *s, *dx, *dres;
  int64_t n, x_row, res_row;
  int32_t c;
  float eps;
  Drop drop;
  float* part;  // backward: [gridDim.x][2][C] partial sums of dw and db
};

// Sums over the row's L lanes.  A workgroup's (L = 256) go through LDS, in one of two places in turn: `turn` counts them.
template <int L, int K>
__device__ __forceinline__ void row_sums(float (&v)[K], float (*lds)[4][2], int& turn) {
#pragma unroll
  for (int d = 1; d < (L < 64 ? L : 64); d <<= 1)
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] += __shfl_xor(v[k], d);
  if constexpr (L > 64) {
    const int wave = threadIdx.x >> 6;
    float(*at)[2] = lds[turn & 1];
    ++turn;
    if ((threadIdx.x & 63) == 0)
#pragma unroll
      for (int k = 0; k < K; ++k) at[wave][k] = v[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = (at[0][k] + at[1][k]) + (at[2][k] + at[3][k]);
  }
}

// Differences from the mean (zeros past the row) in place of the row's values; returns r.
template <int L, int V, int N>
__device__ __forceinline__ float centre(float (&f)[V][N], const bool (&mine)[V], float inv_c, float eps, float (*lds)[4][2],
                                        int& turn) {
  float sum[1] = {0.f};
#pragma unroll
  for (int i = 0; i < V; ++i)
#pragma unroll
    for (int j = 0; j < N; ++j) sum[0] += f[i][j];
  row_sums<L>(sum, lds, turn);
  const float mean = sum[0] * inv_c;
  float sq[1] = {0.f};
#pragma unroll
  for (int i = 0; i < V; ++i)
#pragma unroll
    for (int j = 0; j < N; ++j) {
      f[i][j] = mine[i] ? f[i][j] - mean : 0.f;
      sq[0] = fmaf(f[i][j], f[i][j], sq[0]);
    }
  row_sums<L>(sq, lds, turn);
  return 1.f / sqrtf(fmaf(sq[0], inv_c, eps));
}

template <typename T, int L, int V, bool RES, bool DROP>
__global__ void __launch_bounds__(256, 4) norm_fwd(NormParams p) {
  constexpr int N = Vec<T>::N;
  __shared__ float lds[L > 64 ? 2 : 1][4][2];
  int turn = 0;
  const int sub = threadIdx.x % L;
  const int64_t row = (int64_t(blockIdx.x) * 256 + threadIdx.x) / L;
  if (row >= p.n) return;
  DropKey key;
  if constexpr (DROP) key.load(p.drop.rng);
  bool mine[V];
  u32x4 xv[V], rv[RES ? V : 1];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = (sub + i * L) * N;
    mine[i] = e < p.c;
    xv[i] = u32x4{0, 0, 0, 0};
    if (mine[i]) xv[i] = *reinterpret_cast<const u32x4*>(static_cast<const T*>(p.x) + row * p.x_row + e);
    if constexpr (RES) {
      rv[i] = u32x4{0, 0, 0, 0};
      if (mine[i]) rv[i] = *reinterpret_cast<const u32x4*>(static_cast<const T*>(p.res) + row * p.res_row + e);
    }
  }
  float f[V][N];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int64_t at = row * p.c + (sub + i * L) * N;
    Vec<T>::unpack(xv[i], f[i]);
    if constexpr (DROP) drop(f[i], at, p.drop, key);
    if constexpr (RES) {
      float r[N];
      Vec<T>::unpack(rv[i], r);
#pragma unroll
      for (int j = 0; j < N; ++j) f[i][j] += r[j];
      if (mine[i]) *reinterpret_cast<u32x4*>(static_cast<T*>(p.s) + at) = Vec<T>::pack(f[i]);
    }
  }
  const float r = centre<L>(f, mine, 1.f / float(p.c), p.eps, lds, turn);
#pragma unroll
  for (int i = 0; i < V; ++i) {
    if (!mine[i]) continue;
    const int e = (sub + i * L) * N;
    float w[N], b[N];
    if (p.w) Vec<T>::unpack(*reinterpret_cast<const u32x4*>(static_cast<const T*>(p.w) + e), w);
    if (p.b) Vec<T>::unpack(*reinterpret_cast<const u32x4*>(static_cast<const T*>(p.b) + e), b);
#pragma unroll
    for (int j = 0; j < N; ++j) {
      float v = f[i][j] * r;
      if (p.w) v *= w[j];
      if (p.b) v += b[j];
      f[i][j] = v;
    }
    *reinterpret_cast<u32x4*>(static_cast<T*>(p.y) + row * p.c + e) = Vec<T>::pack(f[i]);
  }
}

// Waves per SIMD that the backward kernel's registers are held to, by the elements of a lane.  Its grid is what then fits
// the chip at once: with 2,048 workgroups in two and two thirds rounds a tenth of the time went to the last one.
constexpr int bwd_waves(int esize, int vecs) {
  const int elements = vecs * 16 / esize;
  return elements <= 8 ? 4 : (elements <= 16 ? 3 : (esize == 2 ? 2 : 1));
}

// Rows are taken in turn by the grid's groups; dw and db of the group's channels stay in registers (DW) and are added
// over the workgroup's groups at the end.
template <typename T, int L, int V, bool RES, bool DROP, bool DW>
__global__ void __launch_bounds__(256, bwd_waves(sizeof(T), V)) norm_bwd(NormParams p) {
  constexpr int N = Vec<T>::N, GPB = 256 / L;
  __shared__ float lds[L > 64 ? 2 : 1][4][2];
  int turn = 0;
  const int sub = threadIdx.x % L, grp = threadIdx.x / L;
  const float inv_c = 1.f / float(p.c);
  DropKey key;
  if constexpr (DROP) key.load(p.drop.rng);
  bool mine[V];
  u32x4 wv[V];
  float dw[DW ? V : 1][N], db[DW ? V : 1][N];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = (sub + i * L) * N;
    mine[i] = e < p.c;
    wv[i] = u32x4{0, 0, 0, 0};
    if (p.w && mine[i]) wv[i] = *reinterpret_cast<const u32x4*>(static_cast<const T*>(p.w) + e);
    if constexpr (DW)
#pragma unroll
      for (int j = 0; j < N; ++j) dw[i][j] = db[i][j] = 0.f;
  }
  u32x4 xv[V], gv[V], uv[RES ? V : 1];
  auto load = [&](int64_t row) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = (sub + i * L) * N;
      xv[i] = gv[i] = u32x4{0, 0, 0, 0};
      if constexpr (RES) uv[i] = u32x4{0, 0, 0, 0};
      if (mine[i]) {
        xv[i] = *reinterpret_cast<const u32x4*>(static_cast<const T*>(p.x) + row * p.x_row + e);
        gv[i] = *reinterpret_cast<const u32x4*>(static_cast<const T*>(p.dy) + row * p.c + e);
        if constexpr (RES)
          if (p.ds) uv[i] = *reinterpret_cast<const u32x4*>(static_cast<const T*>(p.ds) + row * p.c + e);
      }
    }
  };
  const int64_t step = int64_t(gridDim.x) * GPB;
  for (int64_t row = int64_t(blockIdx.x) * GPB + grp; row < p.n; row += step) {
    load(row);
    float f[V][N], g[V][N], u[RES ? V : 1][N];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      Vec<T>::unpack(xv[i], f[i]);
      Vec<T>::unpack(gv[i], g[i]);
      if constexpr (RES) Vec<T>::unpack(uv[i], u[i]);
    }
    const float r = centre<L>(f, mine, inv_c, p.eps, lds, turn);
    float sums[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < V; ++i) {
      float w[N];
      Vec<T>::unpack(wv[i], w);
#pragma unroll
      for (int j = 0; j < N; ++j) {
        f[i][j] *= r;
        if constexpr (DW) {
          dw[i][j] = fmaf(g[i][j], f[i][j], dw[i][j]);
          db[i][j] += g[i][j];
        }
        if (p.w) g[i][j] *= w[j];
        sums[0] += g[i][j];
        sums[1] = fmaf(g[i][j], f[i][j], sums[1]);
      }
    }
    row_sums<L>(sums, lds, turn);
    const float mg = sums[0] * inv_c, mz = sums[1] * inv_c;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if (!mine[i]) continue;
      const int64_t at = row * p.c + (sub + i * L) * N;
#pragma unroll
      for (int j = 0; j < N; ++j) g[i][j] = r * (g[i][j] - mg - f[i][j] * mz);
      if constexpr (RES) {
#pragma unroll
        for (int j = 0; j < N; ++j) g[i][j] += u[i][j];
        if (p.dres) *reinterpret_cast<u32x4*>(static_cast<T*>(p.dres) + at) = Vec<T>::pack(g[i]);
      }
      if (p.dx) {
        if constexpr (DROP) drop(g[i], at, p.drop, key);
        *reinterpret_cast<u32x4*>(static_cast<T*>(p.dx) + at) = Vec<T>::pack(g[i]);
      }
    }
  }
  if constexpr (DW) {
    // the workgroup's groups in a fixed order: within a wave by lane distance, then the four waves
    float* out = p.part + int64_t(blockIdx.x) * 2 * p.c;
    if constexpr (L > 64) {
#pragma unroll
      for (int i = 0; i < V; ++i)
#pragma unroll
        for (int j = 0; j < N; ++j)
          if (mine[i]) {
            const int e = (sub + i * L) * N + j;
            out[e] = dw[i][j];
            out[p.c + e] = db[i][j];
          }
    } else {
      __shared__ float red[4][2][L * N];
      const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        if (i > 0) __syncthreads();
#pragma unroll
        for (int j = 0; j < N; ++j) {
          float a = dw[i][j], b = db[i][j];
#pragma unroll
          for (int d = L; d < 64; d <<= 1) {
            a += __shfl_xor(a, d);
            b += __shfl_xor(b, d);
          }
          if (lane < L) {
            red[wave][0][sub * N + j] = a;
            red[wave][1][sub * N + j] = b;
          }
        }
        __syncthreads();
        for (int t = threadIdx.x; t < 2 * L * N; t += 256) {
          const int k = t / (L * N), e = t % (L * N), at = i * L * N + e;
          if (at < p.c) out[k * p.c + at] = (red[0][k][e] + red[1][k][e]) + (red[2][k][e] + red[3][k][e]);
        }
      }
    }
  }
}

// The weight gradients: a column's partial sums over the row blocks.  A workgroup is 16 columns x 16 shares of the blocks.
template <typename T>
__global__ void __launch_bounds__(256) norm_dw(const float* part, int nparts, int c, T* dw, T* db) {
  const int col = blockIdx.x * 16 + threadIdx.x % 16, share = threadIdx.x / 16;
  T* out = blockIdx.y ? db : dw;
  if (!out) return;
  const float* src = part + (blockIdx.y ? c : 0) + col;
  float v = 0.f;
  if (col < c) {
#pragma unroll 8
    for (int64_t b = share; b < nparts; b += 16) v += src[b * 2 * c];
  }
  __shared__ float red[16][17];
  red[share][threadIdx.x % 16] = v;
  __syncthreads();
  if (share == 0 && col < c) {
    float s = 0.f;
    for (int i = 0; i < 16; ++i) s += red[i][threadIdx.x];
    out[col] = T(s);
  }
}

// Dropout by itself: element by element, U vectors a thread on their way together.
struct DropParams {
  const void *x, *res;
  void* y;
  int64_t n;  // elements
  Drop drop;
};

constexpr int kDropVecs = 4;

template <typename T, bool RES, bool DROP>
__global__ void __launch_bounds__(256) dropout_kernel(DropParams p) {
  constexpr int N = Vec<T>::N;
  const int64_t whole = p.n / N, first = int64_t(blockIdx.x) * 256 * kDropVecs + threadIdx.x;
  const T* x = static_cast<const T*>(p.x);
  const T* res = static_cast<const T*>(p.res);
  T* y = static_cast<T*>(p.y);
  DropKey key;
  if constexpr (DROP) key.load(p.drop.rng);
  u32x4 xv[kDropVecs], rv[RES ? kDropVecs : 1];
#pragma unroll
  for (int i = 0; i < kDropVecs; ++i) {
    const int64_t v = first + i * 256;
    xv[i] = u32x4{0, 0, 0, 0};
    if (v < whole) xv[i] = *reinterpret_cast<const u32x4*>(x + v * N);
    if constexpr (RES) {
      rv[i] = u32x4{0, 0, 0, 0};
      if (v < whole) rv[i] = *reinterpret_cast<const u32x4*>(res + v * N);
    }
  }
#pragma unroll
  for (int i = 0; i < kDropVecs; ++i) {
    const int64_t v = first + i * 256;
    float f[N], r[N];
    if (v < whole) {
      Vec<T>::unpack(xv[i], f);
      if constexpr (DROP) drop(f, v * N, p.drop, key);
      if constexpr (RES) {
        Vec<T>::unpack(rv[i], r);
#pragma unroll
        for (int j = 0; j < N; ++j) f[j] += r[j];
      }
      *reinterpret_cast<u32x4*>(y + v * N) = Vec<T>::pack(f);
    } else if (v == whole) {
      // the elements past the last whole vector
      const int left = int(p.n - whole * N);
#pragma unroll
      for (int j = 0; j < N; ++j) f[j] = j < left ? float(x[whole * N + j]) : 0.f;
      if constexpr (DROP) drop(f, whole * N, p.drop, key);
#pragma unroll
      for (int j = 0; j < N; ++j)
        if (j < left) {
          if constexpr (RES) f[j] += float(res[whole * N + j]);
          y[whole * N + j] = T(f[j]);
        }
    }
  }
}

int esize(int32_t dtype) { return dtype == SSC_F32 ? 4 : 2; }
bool bad(const void* ptr) { return !ptr || !aligned16(ptr); }
bool known(int32_t dtype) { return dtype == SSC_F32 || dtype == SSC_F16 || dtype == SSC_BF16; }

// lanes of a row, and vectors of a lane
struct RowForm {
  int lanes, vecs;
};
RowForm row_form(int64_t channels, int32_t dtype) {
  const int v = int(channels * esize(dtype) / 16);
  for (int l = 4; l <= 64; l *= 2)
    if (v <= l) return {l, 1};
  if (v <= 128) return {64, 2};
  if (v <= 256) return {64, 4};
  if (v <= 512) return {256, 2};
  if (v <= 1024) return {256, 4};
  return {256, 8};
}

// Workgroups of the backward grid: as many as fit the chip's 256 CUs at once, no more than the rows need
int64_t row_blocks(const ssc_layer_norm_shape& a) {
  const RowForm f = row_form(a.channels, a.dtype);
  const int gpb = 256 / f.lanes;
  const int64_t need = (a.n + gpb - 1) / gpb, most = 256 * bwd_waves(esize(a.dtype), f.vecs);
  return need < 1 ? 1 : (need < most ? need : most);
}

int norm_check(const ssc_layer_norm_shape* a) {
  if (!a) return SSC_ERR_INVALID_ARG;
  if (!known(a->dtype)) return SSC_ERR_UNSUPPORTED;
  if (a->n < 0 || a->n > SSC_MAX_SEQ_ROWS || a->channels < 1) return SSC_ERR_INVALID_ARG;
  const int vec = 16 / esize(a->dtype);
  if (a->channels > SSC_MAX_SEQ_CHANNELS || a->channels % vec != 0) return SSC_ERR_UNSUPPORTED;
  if (!(a->eps >= 0.f && a->eps < INFINITY) || drop_threshold(a->p) < 0 || a->layer < 0) return SSC_ERR_INVALID_ARG;
  for (int64_t v : {a->x_row_stride, a->residual_row_stride})
    if (v < 0 || v > (1LL << 40) || v % vec != 0) return SSC_ERR_INVALID_ARG;
  // HIP takes fewer than 2^32 threads in a dimension of a launch; dropout numbers its elements in 32 bits of eights
  const RowForm f = row_form(a->channels, a->dtype);
  if ((a->n * f.lanes + 255) / 256 * 256 >= (1LL << 32)) return SSC_ERR_UNSUPPORTED;
  if (drop_threshold(a->p) > 0 && a->n * a->channels > kMaxDropElements) return SSC_ERR_UNSUPPORTED;
  return SSC_OK;
}

Drop drop_of(double p, int32_t layer, const int64_t* rng) {
  const int t = drop_threshold(p);
  return Drop{rng, uint32_t(layer), uint32_t(t), drop_scale(t)};
}

bool bad_rng(const int64_t* rng) { return !rng || (reinterpret_cast<uintptr_t>(rng) & 7u); }

NormParams norm_params(const ssc_layer_norm_shape& a, const int64_t* rng) {
  NormParams p{};
  p.n = a.n;
  p.x_row = a.x_row_stride;
  p.res_row = a.residual_row_stride;
  p.c = a.channels;
  p.eps = a.eps;
  p.drop = drop_of(a.p, a.layer, rng);
  return p;
}

struct NormCall {
  int64_t grid;
  bool back, res, drop, dw;
  hipStream_t s;
};

template <typename T, int L, int V>
void norm_launch(const NormCall& c, const NormParams& p) {
  const unsigned grid = unsigned(c.grid);
  if (!c.back) {
    if (c.drop)
      norm_fwd<T, L, V, true, true><<<grid, 256, 0, c.s>>>(p);
    else if (c.res)
      norm_fwd<T, L, V, true, false><<<grid, 256, 0, c.s>>>(p);
    else
      norm_fwd<T, L, V, false, false><<<grid, 256, 0, c.s>>>(p);
  } else if (c.dw) {
    if (c.drop)
      norm_bwd<T, L, V, true, true, true><<<grid, 256, 0, c.s>>>(p);
    else if (c.res)
      norm_bwd<T, L, V, true, false, true><<<grid, 256, 0, c.s>>>(p);
    else
      norm_bwd<T, L, V, false, false, true><<<grid, 256, 0, c.s>>>(p);
  } else {
    if (c.drop)
      norm_bwd<T, L, V, true, true, false><<<grid, 256, 0, c.s>>>(p);
    else if (c.res)
      norm_bwd<T, L, V, true, false, false><<<grid, 256, 0, c.s>>>(p);
    else
      norm_bwd<T, L, V, false, false, false><<<grid, 256, 0, c.s>>>(p);
  }
}

template <typename T>
void norm_rows(const RowForm& f, const NormCall& c, const NormParams& p) {
  if (f.lanes == 4)
    norm_launch<T, 4, 1>(c, p);
  else if (f.lanes == 8)
    norm_launch<T, 8, 1>(c, p);
  else if (f.lanes == 16)
    norm_launch<T, 16, 1>(c, p);
  else if (f.lanes == 32)
    norm_launch<T, 32, 1>(c, p);
  else if (f.lanes == 64 && f.vecs == 1)
    norm_launch<T, 64, 1>(c, p);
  else if (f.lanes == 64 && f.vecs == 2)
    norm_launch<T, 64, 2>(c, p);
  else if (f.lanes == 64)
    norm_launch<T, 64, 4>(c, p);
  else if (f.vecs == 2)
    norm_launch<T, 256, 2>(c, p);
  else if (f.vecs == 4)
    norm_launch<T, 256, 4>(c, p);
  else if constexpr (sizeof(T) == 4)
    norm_launch<T, 256, 8>(c, p);
}
static_assert(SSC_MAX_SEQ_CHANNELS == 8192, "the widest row is 8 vectors of fp32, 4 of 16 bits, for each of 256 lanes");

void norm_dispatch(const ssc_layer_norm_shape& a, const NormCall& c, const NormParams& p) {
  const RowForm f = row_form(a.channels, a.dtype);
  if (a.dtype == SSC_F32)
    norm_rows<float>(f, c, p);
  else if (a.dtype == SSC_F16)
    norm_rows<_Float16>(f, c, p);
  else
    norm_rows<__bf16>(f, c, p);
}

template <typename T>
void dw_launch(const float* part, int64_t nparts, int c, void* dw, void* db, hipStream_t s) {
  norm_dw<T><<<dim3(unsigned((c + 15) / 16), 2), 256, 0, s>>>(part, int(nparts), c, static_cast<T*>(dw), static_cast<T*>(db));
}

template <typename T>
void dropout_launch(const DropParams& p, hipStream_t s) {
  const int64_t per = 256 * kDropVecs * Vec<T>::N;
  const unsigned grid = unsigned((p.n + per - 1) / per);
  if (p.drop.t > 0) {
    if (p.res)
      dropout_kernel<T, true, true><<<grid, 256, 0, s>>>(p);
    else
      dropout_kernel<T, false, true><<<grid, 256, 0, s>>>(p);
  } else if (p.res) {
    dropout_kernel<T, true, false><<<grid, 256, 0, s>>>(p);
  } else {
    dropout_kernel<T, false, false><<<grid, 256, 0, s>>>(p);
  }
}

}  // namespace

}  // namespace ssc

using namespace ssc;

extern "C" int ssc_layer_norm_fwd(const ssc_layer_norm_shape* shape, const void* x, const void* residual,
                                  const void* weight, const void* bias, const int64_t* rng, void* y, void* s,
                                  void* stream) {
  const int st = norm_check(shape);
  if (st != SSC_OK) return st;
  const ssc_layer_norm_shape& a = *shape;
  const bool drops = drop_threshold(a.p) > 0;
  if (a.n == 0) return SSC_OK;
  if (drops && !residual) return SSC_ERR_INVALID_ARG;
  if (bad(x) || bad(y) || !aligned16(residual) || !aligned16(weight) || !aligned16(bias)) return SSC_ERR_INVALID_ARG;
  if (residual ? bad(s) : s != nullptr) return SSC_ERR_INVALID_ARG;
  if (drops && bad_rng(rng)) return SSC_ERR_INVALID_ARG;
  NormParams p = norm_params(a, rng);
  p.x = x;
  p.res = residual;
  p.w = weight;
  p.b = bias;
  p.y = y;
  p.s = s;
  const int gpb = 256 / row_form(a.channels, a.dtype).lanes;
  (void)hipGetLastError();
  norm_dispatch(a, NormCall{(a.n + gpb - 1) / gpb, false, residual != nullptr, drops, false, reinterpret_cast<hipStream_t>(stream)}, p);
  return hipGetLastError() == hipSuccess ? SSC_OK : SSC_ERR_HIP;
}

extern "C" size_t ssc_layer_norm_workspace_bytes(const ssc_layer_norm_shape* shape) {
  if (norm_check(shape) != SSC_OK) return 0;
  const size_t bytes = size_t(row_blocks(*shape)) * 2 * size_t(shape->channels) * 4;
  return bytes < 256 ? 256 : bytes;
}

extern "C" int ssc_layer_norm_bwd(const ssc_layer_norm_shape* shape, const void* s, const void* dy, const void* ds,
                                  const void* weight, const int64_t* rng, void* dx, void* dresidual, void* dweight,
                                  void* dbias, void* workspace, size_t workspace_bytes, void* stream) {
  const int st = norm_check(shape);
  if (st != SSC_OK) return st;
  const ssc_layer_norm_shape& a = *shape;
  const bool drops = drop_threshold(a.p) > 0;
  const void* ptrs[6] = {ds, weight, dx, dresidual, dweight, dbias};
  for (const void* v : ptrs)
    if (!aligned16(v)) return SSC_ERR_INVALID_ARG;
  if (!dx && !dresidual && !dweight && !dbias) return SSC_OK;
  if (a.n > 0) {
    if (bad(s) || bad(dy)) return SSC_ERR_INVALID_ARG;
    if (drops && dx && bad_rng(rng)) return SSC_ERR_INVALID_ARG;
  }
  const bool dw = dweight || dbias;
  if (dw) {
    if (bad(workspace)) return SSC_ERR_INVALID_ARG;
    if (workspace_bytes < ssc_layer_norm_workspace_bytes(shape)) return SSC_ERR_WORKSPACE;
  } else if (a.n == 0) {
    return SSC_OK;
  }
  NormParams p = norm_params(a, rng);
  p.x = s;
  p.w = weight;
  p.dy = dy;
  p.ds = ds;
  p.dx = dx;
  p.dres = dresidual;
  p.part = static_cast<float*>(workspace);
  hipStream_t str = reinterpret_cast<hipStream_t>(stream);
  (void)hipGetLastError();
  // n == 0 with weight gradients still runs: its one workgroup writes zero sums
  norm_dispatch(a, NormCall{row_blocks(a), true, ds || dresidual || drops, drops && dx, dw, str}, p);
  if (dw) {
    if (a.dtype == SSC_F32)
      dw_launch<float>(p.part, row_blocks(a), a.channels, dweight, dbias, str);
    else if (a.dtype == SSC_F16)
      dw_launch<_Float16>(p.part, row_blocks(a), a.channels, dweight, dbias, str);
    else
      dw_launch<__bf16>(p.part, row_blocks(a), a.channels, dweight, dbias, str);
  }
  return hipGetLastError() == hipSuccess ? SSC_OK : SSC_ERR_HIP;
}

extern "C" int ssc_dropout(int64_t elements, int32_t dtype, double p, int32_t layer, const void* x, const void* residual,
                           const int64_t* rng, void* y, void* stream) {
  if (!known(dtype)) return SSC_ERR_UNSUPPORTED;
  if (elements < 0 || drop_threshold(p) < 0 || layer < 0) return SSC_ERR_INVALID_ARG;
  if (elements > kMaxDropElements) return SSC_ERR_UNSUPPORTED;
  if (elements == 0) return SSC_OK;
  if (bad(x) || bad(y) || !aligned16(residual)) return SSC_ERR_INVALID_ARG;
  if (drop_threshold(p) > 0 && bad_rng(rng)) return SSC_ERR_INVALID_ARG;
  const DropParams d{x, residual, y, elements, drop_of(p, layer, rng)};
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  (void)hipGetLastError();
  if (dtype == SSC_F32)
    dropout_launch<float>(d, s);
  else if (dtype == SSC_F16)
    dropout_launch<_Float16>(d, s);
  else
    dropout_launch<__bf16>(d, s);
  return hipGetLastError() == hipSuccess ? SSC_OK : SSC_ERR_HIP;
}
