// Norm of the queries and keys of each head with the position rotation in the same pass, and its backward pass.
//
// For every row i and head h, x = q[i][h] (or k[i][h]) of D elements:
//   r = 1 / sqrt(mean(x^2) + eps),  u = x r w,  and pair j of the head, (u_a, u_b), turns by the angle
//   2 pi turns[j] positions[i][axis[j]]:  y_a = u_a cos - u_b sin,  y_b = u_a sin + u_b cos.
// Pairs are (2j, 2j + 1) (interleaved) or (j, j + P) (halves); the D - 2P dimensions past them are not turned.
// Backward, with g the output gradient turned back: dw = sum over rows of g x r, and with u = g w,
//   dx = r (u - x r mean(u x r)).
//
// A group of L lanes (a power of two) owns one row's head, 16 bytes a lane, and walks several heads of its row, so a
// row's cosines and sines are computed once per group.  Turns are multiplied and reduced to [-1/2, 1/2] in 64 bits:
// the phase of a position near 2^31 is as exact as that of position 1.  Sums, the norm and the rotation are fp32 and
// the result is rounded once.  Each element is read once and written once (backward: read twice, written once).  629k rows
// of 16 + 16 heads of 64, bf16, interleaved: forward 0.95 ms (5.4 TB/s), backward 1.50 ms (5.2 TB/s), bound by memory: a
// 1 GiB copy reaches 5.2 TB/s.  The halves layout's lanes form every angle of their elements and exchange partners, in
// registers for two waves per SIMD: 2.9 and 4.3 TB/s in 16 bits (fp32, half as many elements a lane: 5.3 and 5.0); heads
// that do not fill a power of two of vectors leave lanes idle (80, bf16, interleaved: 4.2 and 3.6 TB/s).

#include <hip/hip_runtime.h>

#include "ssc_internal.h"

namespace ssc {

namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

template <typename T>
struct Vec {
  static constexpr int N = 8;
  __device__ static __forceinline__ void unpack(const u32x4& v, float (&f)[8]) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if constexpr (__is_same(T, __bf16)) {
        f[2 * e] = __uint_as_float(v[e] << 16);
        f[2 * e + 1] = __uint_as_float(v[e] & 0xffff0000u);
      } else {
        f[2 * e] = float(__builtin_bit_cast(_Float16, uint16_t(v[e] & 0xffffu)));
        f[2 * e + 1] = float(__builtin_bit_cast(_Float16, uint16_t(v[e] >> 16)));
      }
    }
  }
  __device__ static __forceinline__ u32x4 pack(const float (&f)[8]) {
    u32x4 v;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const f32x2 p{f[2 * e], f[2 * e + 1]};
      if constexpr (__is_same(T, __bf16))
        v[e] = __builtin_bit_cast(uint32_t, __builtin_convertvector(p, bf16x2));
      else
        v[e] = __builtin_bit_cast(uint32_t, __builtin_convertvector(p, f16x2));
    }
    return v;
  }
};

template <>
struct Vec<float> {
  static constexpr int N = 4;
  __device__ static __forceinline__ void unpack(const u32x4& v, float (&f)[4]) {
#pragma unroll
    for (int e = 0; e < 4; ++e) f[e] = __uint_as_float(v[e]);
  }
  __device__ static __forceinline__ u32x4 pack(const float (&f)[4]) {
    u32x4 v;
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = __float_as_uint(f[e]);
    return v;
  }
};

struct RopeParams {
  const void *q, *k, *qw, *kw, *dqo, *dko;
  void *qo, *ko;  // outputs: forward the turned rows, backward the input gradients
  const int32_t* pos;
  const double* turns;
  const int32_t* axis;
  int64_t n, q_row, q_head, k_row, k_head, pos_row;
  int32_t hq, hk, d, axes, pairs, chunks;  // chunks: groups sharing a row
  int32_t per_head;                        // weights are [heads][D], else [D]
  float eps;
  float* part;  // backward: [gridDim.x][hq + hk][D] partial weight gradients
};

// cosine and sine of each of the lane's elements' pair angles; (1, 0) past the pairs.  Interleaved: one entry a pair.
template <typename T, bool HALVES, int NA>
__device__ __forceinline__ void angles(const RopeParams& p, int64_t row, int sub, float (&co)[NA], float (&si)[NA]) {
#pragma unroll
  for (int j = 0; j < NA; ++j) {
    const int e = sub * NA + j;  // interleaved: NA = N / 2 pairs a lane; halves: NA = N elements
    const int pair = HALVES ? (e < p.pairs ? e : e - p.pairs) : e;
    const bool turned = HALVES ? e < 2 * p.pairs : e < p.pairs;
    co[j] = 1.f;
    si[j] = 0.f;
    if (turned) {
      int a = p.axis[pair];
      a = a < 0 ? 0 : (a < p.axes ? a : p.axes - 1);
      double t = double(p.pos[row * p.pos_row + a]) * p.turns[pair];
      t -= rint(t);
      if constexpr (sizeof(T) == 4) {
        sincospif(2.f * float(t), &si[j], &co[j]);
      } else {
        // the hardware's sine and cosine take revolutions; their error is far below a 16-bit result's rounding
        si[j] = __builtin_amdgcn_sinf(float(t));
        co[j] = __builtin_amdgcn_cosf(float(t));
      }
    }
  }
}

// turns the lane's elements by the angles (back: by their negatives)
template <bool HALVES, bool BACK, int N, int NA>
__device__ __forceinline__ void turn(float (&f)[N], const float (&co)[NA], const float (&si)[NA], int pairs, int sub) {
  if constexpr (!HALVES) {
#pragma unroll
    for (int j = 0; j < N / 2; ++j) {
      const float s = BACK ? -si[j] : si[j];
      const float a = f[2 * j], b = f[2 * j + 1];
      f[2 * j] = a * co[j] - b * s;
      f[2 * j + 1] = a * s + b * co[j];
    }
  } else {
    // the partner of a vector in the first half is `pairs` elements up, of one in the second half as many down
    const int step = pairs / N;
    const bool low = sub < step;
    const int other = sub + (low ? step : -step);
    const int lane = int(threadIdx.x & 63) - sub;
    const bool turned = sub < 2 * step;
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const float o = __shfl(f[j], lane + (turned ? other : sub));
      const float s = (low != BACK) ? -si[j] : si[j];
      if (turned) f[j] = f[j] * co[j] + o * s;
    }
  }
}

template <int L>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int d = 1; d < L; d <<= 1) v += __shfl_xor(v, d);
  return v;
}

// Lanes of a group past the head's vectors compute on zeros and store nothing.
template <typename T, int L, bool HALVES, bool NORM>
__global__ void __launch_bounds__(256) rope_fwd(RopeParams p) {
  constexpr int N = Vec<T>::N, NA = HALVES ? N : N / 2;
  const int sub = threadIdx.x % L;
  const int64_t g = (int64_t(blockIdx.x) * 256 + threadIdx.x) / L;
  const int64_t row = g / p.chunks;
  const int chunk = int(g - row * p.chunks);
  if (row >= p.n) return;
  const bool mine = sub * N < p.d;
  const float inv_d = 1.f / float(p.d);
  const int heads = p.hq + p.hk;
  float co[NA], si[NA];
  // heads chunk, chunk + chunks, ...: four at a time, their loads issued together and the first ones' before the angles
  constexpr int B = 4;
  for (int h0 = chunk; h0 < heads; h0 += B * p.chunks) {
    u32x4 v[B];
#pragma unroll
    for (int i = 0; i < B; ++i) {
      const int h = h0 + i * p.chunks;
      const bool isq = h < p.hq;
      const T* src = isq ? static_cast<const T*>(p.q) + row * p.q_row + h * p.q_head
                         : static_cast<const T*>(p.k) + row * p.k_row + (h - p.hq) * p.k_head;
      v[i] = u32x4{0, 0, 0, 0};
      if (mine && h < heads) v[i] = *reinterpret_cast<const u32x4*>(src + sub * N);
    }
    if (h0 == chunk) {
#pragma unroll
      for (int j = 0; j < NA; ++j) co[j] = 1.f, si[j] = 0.f;
      if (p.pairs > 0) angles<T, HALVES, NA>(p, row, sub, co, si);
    }
#pragma unroll
    for (int i = 0; i < B; ++i) {
      const int h = h0 + i * p.chunks;
      if (h >= heads) break;
      const bool isq = h < p.hq;
      const int hh = isq ? h : h - p.hq;
      T* dst = isq ? static_cast<T*>(p.qo) + (row * p.hq + hh) * p.d : static_cast<T*>(p.ko) + (row * p.hk + hh) * p.d;
      const T* w = static_cast<const T*>(isq ? p.qw : p.kw);
      float f[N];
      Vec<T>::unpack(v[i], f);
      if constexpr (NORM) {
        float sq = 0.f;
#pragma unroll
        for (int j = 0; j < N; ++j) sq = fmaf(f[j], f[j], sq);
        const float r = 1.f / sqrtf(group_sum<L>(sq) * inv_d + p.eps);
#pragma unroll
        for (int j = 0; j < N; ++j) f[j] *= r;
        if (w) {
          float wf[N];
          Vec<T>::unpack(mine ? *reinterpret_cast<const u32x4*>(w + (p.per_head ? hh * p.d : 0) + sub * N)
                              : u32x4{0, 0, 0, 0}, wf);
#pragma unroll
          for (int j = 0; j < N; ++j) f[j] *= wf[j];
        }
      }
      if (p.pairs > 0) turn<HALVES, false>(f, co, si, p.pairs, sub);
      if (mine) *reinterpret_cast<u32x4*>(dst + sub * N) = Vec<T>::pack(f);
    }
  }
}

constexpr int kRopeHeads = 4;  // heads a backward group keeps weight-gradient sums for

// blockIdx.y: heads y * kRopeHeads ..; the block's groups take rows in turn and the weight gradients' sums stay in
// registers.  All loads of a row's heads are issued before its angles are formed: with a head's loads waited for one
// after another the pass ran at 3.0 TB/s.
template <typename T, int L, bool HALVES, bool NORM, bool DW>
__global__ void __launch_bounds__(256) rope_bwd(RopeParams p) {
  constexpr int N = Vec<T>::N, NA = HALVES ? N : N / 2, GPB = 256 / L;
  const int sub = threadIdx.x % L, grp = threadIdx.x / L;
  const int h0 = blockIdx.y * kRopeHeads, heads = p.hq + p.hk;
  const bool mine = sub * N < p.d;
  const float inv_d = 1.f / float(p.d);
  float acc[kRopeHeads][N], wf[kRopeHeads][N];
#pragma unroll
  for (int i = 0; i < kRopeHeads; ++i) {
    const int h = h0 + i;
    const bool isq = h < p.hq;
    const int hh = isq ? h : h - p.hq;
    const T* w = static_cast<const T*>(isq ? p.qw : p.kw);
#pragma unroll
    for (int j = 0; j < N; ++j) acc[i][j] = 0.f, wf[i][j] = 1.f;
    if (NORM && w && h < heads && mine)
      Vec<T>::unpack(*reinterpret_cast<const u32x4*>(w + (p.per_head ? hh * p.d : 0) + sub * N), wf[i]);
  }
  // a head past the last reads the last's rows and writes nothing; so does one whose output gradient is not given
  const T *src[kRopeHeads], *up[kRopeHeads];
  T* out[kRopeHeads];
  int64_t srow[kRopeHeads], urow[kRopeHeads];
  bool on[kRopeHeads];
#pragma unroll
  for (int i = 0; i < kRopeHeads; ++i) {
    const int h = h0 + i < heads ? h0 + i : heads - 1;
    const bool isq = h < p.hq;
    const int hh = isq ? h : h - p.hq;
    const T* u = static_cast<const T*>(isq ? p.dqo : p.dko);
    T* o = static_cast<T*>(isq ? p.qo : p.ko);
    on[i] = h0 + i < heads && u;
    src[i] = (isq ? static_cast<const T*>(p.q) + hh * p.q_head : static_cast<const T*>(p.k) + hh * p.k_head) + sub * N;
    srow[i] = isq ? p.q_row : p.k_row;
    up[i] = u + hh * p.d + sub * N;
    urow[i] = int64_t(isq ? p.hq : p.hk) * p.d;
    out[i] = o ? o + hh * p.d + sub * N : nullptr;
  }
  for (int64_t row = int64_t(blockIdx.x) * GPB + grp; row < p.n; row += int64_t(gridDim.x) * GPB) {
    // all of the row's loads are on their way before the angles are formed
    u32x4 gv[kRopeHeads], xv[kRopeHeads];
#pragma unroll
    for (int i = 0; i < kRopeHeads; ++i) {
      gv[i] = xv[i] = u32x4{0, 0, 0, 0};
      if (mine && on[i]) {
        gv[i] = *reinterpret_cast<const u32x4*>(up[i] + row * urow[i]);
        if constexpr (NORM) xv[i] = *reinterpret_cast<const u32x4*>(src[i] + row * srow[i]);
      }
    }
    float co[NA], si[NA];
#pragma unroll
    for (int j = 0; j < NA; ++j) co[j] = 1.f, si[j] = 0.f;
    if (p.pairs > 0) angles<T, HALVES, NA>(p, row, sub, co, si);
#pragma unroll
    for (int i = 0; i < kRopeHeads; ++i) {
      float g[N];
      Vec<T>::unpack(gv[i], g);
      if (p.pairs > 0) turn<HALVES, true>(g, co, si, p.pairs, sub);
      if constexpr (NORM) {
        float x[N];
        Vec<T>::unpack(xv[i], x);
        float sq = 0.f, dot = 0.f;
#pragma unroll
        for (int j = 0; j < N; ++j) {
          sq = fmaf(x[j], x[j], sq);
          dot = fmaf(g[j] * wf[i][j], x[j], dot);
        }
        sq = group_sum<L>(sq);
        dot = group_sum<L>(dot);
        const float r = 1.f / sqrtf(sq * inv_d + p.eps), s = dot * r * inv_d;
#pragma unroll
        for (int j = 0; j < N; ++j) {
          const float xn = x[j] * r;
          if constexpr (DW) acc[i][j] = fmaf(g[j], on[i] ? xn : 0.f, acc[i][j]);
          g[j] = r * (g[j] * wf[i][j] - xn * s);
        }
      }
      if (mine && on[i] && out[i]) *reinterpret_cast<u32x4*>(out[i] + row * urow[i]) = Vec<T>::pack(g);
    }
  }
  if constexpr (DW) {
    // the block's groups in a fixed order: within a wave by lane distance, then the four waves
    __shared__ float red[4][kRopeHeads][L * N];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
#pragma unroll
    for (int i = 0; i < kRopeHeads; ++i)
#pragma unroll
      for (int j = 0; j < N; ++j) {
        float v = acc[i][j];
#pragma unroll
        for (int d = L; d < 64; d <<= 1) v += __shfl_xor(v, d);
        if (lane < L) red[wave][i][sub * N + j] = v;
      }
    __syncthreads();
    for (int t = threadIdx.x; t < kRopeHeads * p.d; t += 256) {
      const int i = t / p.d, e = t - i * p.d, h = h0 + i;
      if (h < heads)
        p.part[(int64_t(blockIdx.x) * heads + h) * p.d + e] = (red[0][i][e] + red[1][i][e]) + (red[2][i][e] + red[3][i][e]);
    }
  }
}

// The weight gradients: column c's partial sums over the row blocks (and, for one weight shared by all heads, over the
// heads), queries' columns first, then the keys'.  A workgroup is 16 columns x 16 shares of the partial rows.
template <typename T>
__global__ void __launch_bounds__(256) rope_dw(const float* part, int nparts, int hq, int hk, int d, int per_head, T* dqw,
                                               T* dkw) {
  const int qcols = dqw ? (per_head ? hq * d : d) : 0, kcols = dkw ? (per_head ? hk * d : d) : 0;
  int c = blockIdx.x * 16 + threadIdx.x % 16;
  const int ph = threadIdx.x / 16;
  const bool isq = c < qcols;
  T* dw = isq ? dqw : dkw;
  if (!isq) c -= qcols;
  const bool any = isq || c < kcols;
  float v = 0.f;
  if (any) {
    const int reps = per_head ? 1 : (isq ? hq : hk), h0 = isq ? 0 : hq;
    for (int64_t b = ph; b < nparts; b += 16)
      for (int r = 0; r < reps; ++r) v += part[(b * (hq + hk) + h0 + r) * d + c];
  }
  __shared__ float red[16][17];
  red[ph][threadIdx.x % 16] = v;
  __syncthreads();
  if (ph == 0 && any) {
    float s = 0.f;
    for (int i = 0; i < 16; ++i) s += red[i][threadIdx.x];
    dw[c] = T(s);
  }
}

int esize(int32_t dtype) { return dtype == SSC_F32 ? 4 : 2; }
bool bad(const void* ptr) { return !ptr || !aligned16(ptr); }

int lanes_of(const ssc_norm_rope_shape& a) {
  const int vecs = a.head_dim * esize(a.dtype) / 16;
  int l = 4;
  while (l < vecs) l <<= 1;
  return l;
}

// Groups that share a row's heads in the forward pass: a group walks up to 8 (the angles are then a small part of its
// work), fewer when the rows alone do not give the chip 4096 waves (22.4k rows x 8 heads: 14.7 us with twice as many,
// 13.4 us)
int64_t fwd_chunks(const ssc_norm_rope_shape& a) {
  const int64_t heads = a.heads_q + a.heads_kv;
  int64_t chunks = (heads + 7) / 8;
  while (chunks < heads && a.n * chunks * lanes_of(a) < 262144) chunks *= 2;
  return chunks > heads ? heads : chunks;
}

// row blocks of the backward grid: enough workgroups to fill the chip, no more than the rows need
int64_t row_blocks(const ssc_norm_rope_shape& a) {
  const int64_t ny = (a.heads_q + a.heads_kv + kRopeHeads - 1) / kRopeHeads;
  const int gpb = 256 / lanes_of(a);
  int64_t want = 2048 / ny, need = (a.n + gpb - 1) / gpb;
  if (want < 1) want = 1;
  return need < want ? (need < 1 ? 1 : need) : want;
}

int rope_check(const ssc_norm_rope_shape* a) {
  if (!a) return SSC_ERR_INVALID_ARG;
  if (a->dtype != SSC_F32 && a->dtype != SSC_F16 && a->dtype != SSC_BF16) return SSC_ERR_UNSUPPORTED;
  if (a->n < 0 || a->n > SSC_MAX_ATTN_ROWS || a->heads_q < 0 || a->heads_kv < 0 || a->head_dim < 1)
    return SSC_ERR_INVALID_ARG;
  if (a->heads_q > 1024 || a->heads_kv > 1024) return SSC_ERR_UNSUPPORTED;
  const int e = esize(a->dtype), vec = 16 / e;
  if (a->head_dim > 256 || a->head_dim % vec != 0) return SSC_ERR_UNSUPPORTED;
  if (a->pairs < 0 || 2 * int64_t(a->pairs) > a->head_dim) return SSC_ERR_INVALID_ARG;
  if (a->pairs > 0 && (a->axes < 1 || a->axes > SSC_MAX_ROPE_AXES || a->pos_row_stride < 0)) return SSC_ERR_INVALID_ARG;
  if (a->layout != SSC_ROPE_INTERLEAVED && a->layout != SSC_ROPE_HALVES) return SSC_ERR_UNSUPPORTED;
  if (a->layout == SSC_ROPE_HALVES && a->pairs % vec != 0) return SSC_ERR_UNSUPPORTED;
  if (a->norm && !(a->eps >= 0.f && a->eps < INFINITY)) return SSC_ERR_INVALID_ARG;
  // HIP takes fewer than 2^32 threads in a dimension of a launch
  if ((a->n * fwd_chunks(*a) * lanes_of(*a) + 255) / 256 * 256 >= (1LL << 32)) return SSC_ERR_UNSUPPORTED;
  const int64_t st[4] = {a->q_row_stride, a->q_head_stride, a->k_row_stride, a->k_head_stride};
  for (int64_t v : st)
    if (v < 0 || v > (1LL << 40) || v % vec != 0) return SSC_ERR_INVALID_ARG;
  return SSC_OK;
}

RopeParams rope_params(const ssc_norm_rope_shape& a) {
  RopeParams p{};
  p.n = a.n;
  p.q_row = a.q_row_stride;
  p.q_head = a.q_head_stride;
  p.k_row = a.k_row_stride;
  p.k_head = a.k_head_stride;
  p.pos_row = a.pos_row_stride;
  p.hq = a.heads_q;
  p.hk = a.heads_kv;
  p.d = a.head_dim;
  p.axes = a.axes;
  p.pairs = a.pairs;
  p.per_head = a.weight_per_head;
  p.eps = a.eps;
  return p;
}

template <typename T, int L, bool HALVES>
void fwd_lanes(const ssc_norm_rope_shape& a, RopeParams& p, hipStream_t s) {
  p.chunks = int32_t(fwd_chunks(a));
  const int64_t threads = a.n * p.chunks * L;
  const unsigned grid = unsigned((threads + 255) / 256);
  if (a.norm)
    rope_fwd<T, L, HALVES, true><<<grid, 256, 0, s>>>(p);
  else
    rope_fwd<T, L, HALVES, false><<<grid, 256, 0, s>>>(p);
}

template <typename T, int L, bool HALVES>
void bwd_lanes(const ssc_norm_rope_shape& a, const RopeParams& p, bool dw, hipStream_t s) {
  const dim3 grid(unsigned(row_blocks(a)), unsigned((a.heads_q + a.heads_kv + kRopeHeads - 1) / kRopeHeads));
  if (!a.norm)
    rope_bwd<T, L, HALVES, false, false><<<grid, 256, 0, s>>>(p);
  else if (dw)
    rope_bwd<T, L, HALVES, true, true><<<grid, 256, 0, s>>>(p);
  else
    rope_bwd<T, L, HALVES, true, false><<<grid, 256, 0, s>>>(p);
}

template <typename T, int L>
void rope_layout(const ssc_norm_rope_shape& a, RopeParams& p, bool back, bool dw, hipStream_t s) {
  const bool halves = a.layout == SSC_ROPE_HALVES;
  if (back) {
    if (halves)
      bwd_lanes<T, L, true>(a, p, dw, s);
    else
      bwd_lanes<T, L, false>(a, p, dw, s);
  } else {
    if (halves)
      fwd_lanes<T, L, true>(a, p, s);
    else
      fwd_lanes<T, L, false>(a, p, s);
  }
}

template <typename T>
void rope_dispatch(const ssc_norm_rope_shape& a, RopeParams& p, bool back, bool dw, hipStream_t s) {
  const int l = lanes_of(a);
  if (l == 4)
    rope_layout<T, 4>(a, p, back, dw, s);
  else if (l == 8)
    rope_layout<T, 8>(a, p, back, dw, s);
  else if (l == 16)
    rope_layout<T, 16>(a, p, back, dw, s);
  else if (l == 32)
    rope_layout<T, 32>(a, p, back, dw, s);
  else if constexpr (sizeof(T) == 4)
    rope_layout<T, 64>(a, p, back, dw, s);
}

template <typename T>
void launch_dw(const ssc_norm_rope_shape& a, const float* part, void* dqw, void* dkw, hipStream_t s) {
  const int per = a.weight_per_head ? a.head_dim : 0;
  const int cols = (dqw ? (per ? a.heads_q * per : a.head_dim) : 0) + (dkw ? (per ? a.heads_kv * per : a.head_dim) : 0);
  rope_dw<T><<<unsigned((cols + 15) / 16), 256, 0, s>>>(part, int(row_blocks(a)), a.heads_q, a.heads_kv, a.head_dim,
                                                        a.weight_per_head, static_cast<T*>(dqw), static_cast<T*>(dkw));
}

}  // namespace

}  // namespace ssc

using namespace ssc;

extern "C" int ssc_qk_norm_rope_fwd(const ssc_norm_rope_shape* shape, const void* q, const void* k,
                                    const int32_t* positions, const double* turns, const int32_t* axis,
                                    const void* q_weight, const void* k_weight, void* q_out, void* k_out,
                                    void* stream) {
  const int st = rope_check(shape);
  if (st != SSC_OK) return st;
  const ssc_norm_rope_shape& a = *shape;
  if (a.n == 0 || a.heads_q + a.heads_kv == 0) return SSC_OK;
  if (a.heads_q > 0 && (bad(q) || bad(q_out))) return SSC_ERR_INVALID_ARG;
  if (a.heads_kv > 0 && (bad(k) || bad(k_out))) return SSC_ERR_INVALID_ARG;
  if (a.pairs > 0 && (!positions || (reinterpret_cast<uintptr_t>(positions) & 3u) || bad(turns) || bad(axis)))
    return SSC_ERR_INVALID_ARG;
  if (!aligned16(q_weight) || !aligned16(k_weight) || (!a.norm && (q_weight || k_weight))) return SSC_ERR_INVALID_ARG;
  RopeParams p = rope_params(a);
  p.q = q;
  p.k = k;
  p.qw = q_weight;
  p.kw = k_weight;
  p.qo = q_out;
  p.ko = k_out;
  p.pos = positions;
  p.turns = turns;
  p.axis = axis;
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  (void)hipGetLastError();
  if (a.dtype == SSC_F32)
    rope_dispatch<float>(a, p, false, false, s);
  else if (a.dtype == SSC_F16)
    rope_dispatch<_Float16>(a, p, false, false, s);
  else
    rope_dispatch<__bf16>(a, p, false, false, s);
  return hipGetLastError() == hipSuccess ? SSC_OK : SSC_ERR_HIP;
}

extern "C" size_t ssc_qk_norm_rope_workspace_bytes(const ssc_norm_rope_shape* shape) {
  if (rope_check(shape) != SSC_OK) return 0;
  const size_t bytes = size_t(row_blocks(*shape)) * size_t(shape->heads_q + shape->heads_kv) * size_t(shape->head_dim) * 4;
  return bytes < 256 ? 256 : bytes;
}

extern "C" int ssc_qk_norm_rope_bwd(const ssc_norm_rope_shape* shape, const void* q, const void* k,
                                    const int32_t* positions, const double* turns, const int32_t* axis,
                                    const void* q_weight, const void* k_weight, const void* dq_out,
                                    const void* dk_out, void* dq, void* dk, void* dq_weight, void* dk_weight,
                                    void* workspace, size_t workspace_bytes, void* stream) {
  const int st = rope_check(shape);
  if (st != SSC_OK) return st;
  const ssc_norm_rope_shape& a = *shape;
  if (a.heads_q + a.heads_kv == 0) return SSC_OK;
  const void* ptrs[6] = {q_weight, k_weight, dq, dk, dq_weight, dk_weight};
  for (const void* x : ptrs)
    if (!aligned16(x)) return SSC_ERR_INVALID_ARG;
  if (!a.norm && (q_weight || k_weight || dq_weight || dk_weight)) return SSC_ERR_INVALID_ARG;
  if ((dq_weight && !q_weight) || (dk_weight && !k_weight)) return SSC_ERR_INVALID_ARG;
  if (a.n > 0) {
    if (a.heads_q > 0 && (dq || dq_weight) && (bad(q) || bad(dq_out))) return SSC_ERR_INVALID_ARG;
    if (a.heads_kv > 0 && (dk || dk_weight) && (bad(k) || bad(dk_out))) return SSC_ERR_INVALID_ARG;
    if (a.pairs > 0 && (!positions || (reinterpret_cast<uintptr_t>(positions) & 3u) || bad(turns) || bad(axis)))
      return SSC_ERR_INVALID_ARG;
  }
  const bool dw = dq_weight || dk_weight;
  if (dw) {
    if (bad(workspace)) return SSC_ERR_INVALID_ARG;
    if (workspace_bytes < ssc_qk_norm_rope_workspace_bytes(shape)) return SSC_ERR_WORKSPACE;
  }
  RopeParams p = rope_params(a);
  p.q = q;
  p.k = k;
  p.qw = q_weight;
  p.kw = k_weight;
  p.dqo = (dq || dq_weight) ? dq_out : nullptr;
  p.dko = (dk || dk_weight) ? dk_out : nullptr;
  p.qo = dq;
  p.ko = dk;
  p.pos = positions;
  p.turns = turns;
  p.axis = axis;
  p.part = static_cast<float*>(workspace);
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  (void)hipGetLastError();
  // n == 0 with weight gradients still runs: its one row block writes zero sums
  if (a.n > 0 || dw) {
    if (a.dtype == SSC_F32)
      rope_dispatch<float>(a, p, true, dw, s);
    else if (a.dtype == SSC_F16)
      rope_dispatch<_Float16>(a, p, true, dw, s);
    else
      rope_dispatch<__bf16>(a, p, true, dw, s);
  }
  if (dw) {
    if (a.dtype == SSC_F32)
      launch_dw<float>(a, p.part, dq_weight, dk_weight, s);
    else if (a.dtype == SSC_F16)
      launch_dw<_Float16>(a, p.part, dq_weight, dk_weight, s);
    else
      launch_dw<__bf16>(a, p.part, dq_weight, dk_weight, s);
  }
  return hipGetLastError() == hipSuccess ? SSC_OK : SSC_ERR_HIP;
}
