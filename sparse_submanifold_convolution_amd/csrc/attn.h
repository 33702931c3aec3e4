// Ragged cross attention on gfx950: kernels shared by the element types' translation units.
//
// Rows of sample b (q rows [qoff[b], qoff[b+1]), key rows [koff[b], koff[b+1])) attend that sample's keys.  Every
// product is a 32x32 MFMA tile with one side resident in registers as the tile's columns and the other streamed
// through LDS as its rows:
//   forward        columns = queries, rows = keys:     S^T = K Q^T, then O^T += V^T P^T
//   dQ             columns = queries, rows = keys:     S^T, dP^T = V dO^T, then dQ^T += K^T dS^T
//   dK and dV      columns = keys,    rows = queries:  S = Q K^T, dP = dO V^T, then dV^T += dO^T P, dK^T += Q^T dS
// A 32x32 result holds column (lane mod 32) and rows 8 (r/4) + 4 (lane/32) + r mod 4 in register r, so softmax
// statistics of a query column are one lane's registers and one exchange between the half-waves, and the packed
// results are at once the second product's B operand: the reduction order inside an MFMA is free as long as both
// operands agree on it, so the A operand's rows are read from LDS in the order the registers have them (by the LDS
// transpose read for 16-bit types, by single words for fp32).  Nothing goes through LDS between the two products.
//
// Query heads sharing a key head are packed along the rows: row r of a sample and key head hk is token r / G,
// head hk * G + r mod G (G = heads_q / heads_kv).  dK and dV of a shared head thereby sum over its query heads in a
// fixed order, and one query token's G heads share a tile.
#pragma once

#include <hip/hip_runtime.h>

#include "ssc_internal.h"

namespace ssc {
namespace attn {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kTile = 64;  // streamed rows per LDS stage

struct Params {
  const void *q, *k, *v, *out, *dout;
  void *o, *dq, *dk, *dv;
  float* lse;          // [hq][nq]
  float* delta;        // [hq][nq], backward: sum over d of dout * out
  const uint32_t* bound;  // backward, fp16: bits of max |dout row|^2 and max |v row|^2
  const int32_t *qoff, *koff;
  const uint8_t* mask;
  int64_t nq, nk;
  int64_t q_row, q_head, k_row, k_head, v_row, v_head;  // strides in elements
  int32_t batch, hq, hk, d, G;
  uint32_t gmul;
  int32_t gshift;      // r / G = (r * gmul) >> gshift for r < 2^31
  float scale;
  int32_t tiles, nsplit;
  float *part_a, *part_b;  // splits: partial sums [nsplit][rows][d]; forward part_b: [nsplit][rows][2] (max, sum)
};

template <typename T>
struct Elt;

template <>
struct Elt<float> {
  using frag_t = u32x4;               // 4 reduction indices per lane
  static constexpr int kVec = 4;      // elements of a 16-byte chunk
  static constexpr int kSteps = 4;    // fragments covering 32 streamed rows
  __device__ static __forceinline__ f32x16 mma(const u32x4& a, const u32x4& b, f32x16 c) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      c = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(a[j]), __uint_as_float(b[j]), c, 0, 0, 0);
    return c;
  }
  // fragment s of a 32x32 result: its registers 4s .. 4s+3
  __device__ static __forceinline__ u32x4 pack(const f32x16& p, int s) {
    u32x4 f;
#pragma unroll
    for (int j = 0; j < 4; ++j) f[j] = __float_as_uint(p[4 * s + j]);
    return f;
  }
};

template <>
struct Elt<_Float16> {
  using frag_t = u32x4;
  static constexpr int kVec = 8;
  static constexpr int kSteps = 2;
  __device__ static __forceinline__ f32x16 mma(const u32x4& a, const u32x4& b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0,
                                                  0);
  }
  __device__ static __forceinline__ uint32_t pack2(float a, float b) {
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{a, b}, f16x2));
  }
  __device__ static __forceinline__ u32x4 pack(const f32x16& p, int s) {
    u32x4 f;
#pragma unroll
    for (int j = 0; j < 4; ++j) f[j] = pack2(p[8 * s + 2 * j], p[8 * s + 2 * j + 1]);
    return f;
  }
  __device__ static __forceinline__ float lo(uint32_t u) {
    return float(__builtin_bit_cast(_Float16, uint16_t(u & 0xffffu)));
  }
  __device__ static __forceinline__ float hi(uint32_t u) { return float(__builtin_bit_cast(_Float16, uint16_t(u >> 16))); }
};

template <>
struct Elt<__bf16> {
  using frag_t = u32x4;
  static constexpr int kVec = 8;
  static constexpr int kSteps = 2;
  __device__ static __forceinline__ f32x16 mma(const u32x4& a, const u32x4& b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                   0, 0);
  }
  __device__ static __forceinline__ uint32_t pack2(float a, float b) {
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{a, b}, bf16x2));
  }
  __device__ static __forceinline__ u32x4 pack(const f32x16& p, int s) {
    u32x4 f;
#pragma unroll
    for (int j = 0; j < 4; ++j) f[j] = pack2(p[8 * s + 2 * j], p[8 * s + 2 * j + 1]);
    return f;
  }
  __device__ static __forceinline__ float lo(uint32_t u) { return __uint_as_float(u << 16); }
  __device__ static __forceinline__ float hi(uint32_t u) { return __uint_as_float(u & 0xffff0000u); }
};

// Exponent offset of the 16-bit probabilities.  fp16 is subnormal below 2^-14, which rows over thousands of keys
// reach, so its probabilities are held times a power of two that keeps the largest (1) below fp16's 65504; sums
// accumulated from them are scaled back exactly.  bf16 and fp32 have fp32's exponents.
template <typename T>
constexpr int kPExp = __is_same(T, _Float16) ? 14 : 0;

// Sixteen-byte chunks of an LDS row are permuted by row so that both kinds of read spread over all 64 banks: 16
// consecutive rows of one chunk (operand rows), and four consecutive rows of four neighbouring chunks (transpose
// reads).  CPR chunks make a row; 16 chunks span the banks once.
template <int CPR>
__device__ __forceinline__ int swz(int row, int chunk) {
  if constexpr (CPR % 16 == 0) {
    return chunk ^ (((row & 3) << 2) | ((row >> 2) & 3));
  } else if constexpr (CPR % 8 == 0) {
    const int p = (row >> 1) & 7;
    return chunk ^ (((p & 1) << 2) | (p >> 1));
  } else {
    return chunk ^ ((row >> 2) & 3);
  }
}

__device__ __forceinline__ s16x4 lds_tr16(const void* p) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)(const_cast<void*>(p)));
}

// Geometry of one LDS tile of kTile streamed rows and DP (head size rounded up to 32) elements, and its reads
template <typename T, int DP>
struct TileOf {
  static constexpr int kVec = Elt<T>::kVec;
  static constexpr int CPR = DP / kVec;            // chunks per row
  static constexpr int kBytes = kTile * CPR * 16;
  static constexpr int kFrags = DP / (2 * kVec);   // operand fragments along the head dimension
  static constexpr int kBlocks = DP / 32;          // 32-wide blocks of the head dimension

  // rows r0 .. r0+31 as MFMA rows, reduction indices of fragment f (chunk 2f + lane/32)
  __device__ static __forceinline__ u32x4 rows(const char* tile, int r0, int f) {
    const int lane = threadIdx.x & 63;
    const int row = r0 + (lane & 31);
    return *reinterpret_cast<const u32x4*>(tile + (row * CPR + swz<CPR>(row, 2 * f + (lane >> 5))) * 16);
  }
  // head-dimension elements 32 cb .. +31 as MFMA rows, streamed rows of fragment s of the block at r0 as the reduction
  __device__ static __forceinline__ u32x4 cols(const char* tile, int r0, int s, int cb) {
    const int lane = threadIdx.x & 63;
    if constexpr (sizeof(T) == 4) {
      u32x4 f;
      const int col = 32 * cb + (lane & 31);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int row = r0 + 8 * s + 4 * (lane >> 5) + j;
        f[j] = *reinterpret_cast<const uint32_t*>(tile + (row * CPR + swz<CPR>(row, col >> 2)) * 16 + (col & 3) * 4);
      }
      return f;
    } else {
      const int i = lane & 15;
      const int chunk = 4 * cb + 2 * ((lane >> 4) & 1) + ((i >> 1) & 1);
      union {
        s16x4 h[2];
        u32x4 f;
      } u;
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const int row = r0 + 16 * s + 8 * b + 4 * (lane >> 5) + (i >> 2);
        u.h[b] = lds_tr16(tile + (row * CPR + swz<CPR>(row, chunk)) * 16 + (i & 1) * 8);
      }
      return u.f;
    }
  }
};

// A tile on its way from memory to LDS, NT threads: 16-byte chunks in registers
template <typename T, int DP, int NT>
struct Stage {
  using TL = TileOf<T, DP>;
  static constexpr int kTotal = kTile * TL::CPR;
  static constexpr int N = (kTotal + NT - 1) / NT;
  u32x4 r[N];
  __device__ static __forceinline__ int item(int i) { return int(threadIdx.x) + i * NT; }
  __device__ static __forceinline__ bool any(int i) { return kTotal % NT == 0 || item(i) < kTotal; }
  // ptr(row): address of row `row` of the tile, called for rows below `rows` only; dchunks: chunks the head fills
  template <typename F>
  __device__ __forceinline__ void load(int rows, int dchunks, F ptr) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int row = item(i) / TL::CPR, c = item(i) % TL::CPR;
      r[i] = u32x4{0, 0, 0, 0};
      if (any(i) && row < rows && c < dchunks)
        r[i] = *reinterpret_cast<const u32x4*>(ptr(row) + c * TL::kVec);
    }
  }
  __device__ __forceinline__ void store(char* tile) const {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int row = item(i) / TL::CPR, c = item(i) % TL::CPR;
      if (any(i)) *reinterpret_cast<u32x4*>(tile + (row * TL::CPR + swz<TL::CPR>(row, c)) * 16) = r[i];
    }
  }
  // clears the chunks of rows whose key is masked, whatever memory held there
  __device__ __forceinline__ void clear(const uint8_t* keep) {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (!keep[i]) r[i] = u32x4{0, 0, 0, 0};
  }
};

__device__ __forceinline__ int64_t clamp_off(const int32_t* off, int i, int64_t n) {
  const int64_t v = off[i];
  return v < 0 ? 0 : (v > n ? n : v);
}

// One tile of the rows of one sample.  The rows split into batch + 2 segments: those before off[0], the samples',
// those from off[batch]; the first and the last belong to no sample and have no counterpart rows.
struct Segment {
  int64_t begin;   // first row
  int32_t len;     // rows
  int64_t other;   // first row of the sample on the other side
  int32_t other_len;
  int32_t tile;    // tile number inside the segment
};

// Finds tile t of the concatenated segments, each holding ceil(len * mult / cols) tiles; false past the last.
__device__ __forceinline__ bool find_segment(const int32_t* off, int64_t n, const int32_t* other_off, int64_t other_n,
                                             int batch, int mult, int cols, int t, Segment* seg) {
  const int lane = threadIdx.x & 63;
  int before = 0;
  for (int base = 0; base < batch + 2; base += 64) {
    const int s = base + lane;
    int64_t b = 0, e = 0;
    if (s < batch + 2) {
      b = s == 0 ? 0 : clamp_off(off, s - 1, n);
      e = s == batch + 1 ? n : clamp_off(off, s, n);
      if (e < b) e = b;
    }
    int incl = int(((e - b) * mult + cols - 1) / cols);
    const int mine = incl;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int o = __shfl_up(incl, d);
      if (lane >= d) incl += o;
    }
    const int total = __shfl(incl, 63);
    if (t - before < total) {
      const uint64_t past = __ballot(incl > t - before);
      const int w = __ffsll((unsigned long long)past) - 1;
      const int sw = __builtin_amdgcn_readfirstlane(base + w);
      // every lane reads the same values again: uniform, so they sit in scalar registers
      const int64_t bw = sw == 0 ? 0 : clamp_off(off, sw - 1, n);
      const int64_t ew = sw == batch + 1 ? n : clamp_off(off, sw, n);
      seg->begin = bw;
      seg->len = int(ew > bw ? ew - bw : 0);
      seg->tile = __builtin_amdgcn_readfirstlane(t - before - __shfl(incl - mine, w));
      seg->other = 0;
      seg->other_len = 0;
      if (sw >= 1 && sw <= batch) {
        const int64_t ob = clamp_off(other_off, sw - 1, other_n), oe = clamp_off(other_off, sw, other_n);
        seg->other = ob;
        seg->other_len = int(oe > ob ? oe - ob : 0);
      }
      return true;
    }
    before += total;
  }
  return false;
}

__device__ __forceinline__ uint32_t div_g(uint32_t r, const Params& p) {
  return uint32_t((uint64_t(r) * p.gmul) >> p.gshift);
}

// Workgroup ids reach the 8 XCDs round-robin; consecutive work items go to one XCD, so the tiles that stream the
// same sample and head share its L2.
__device__ __forceinline__ int64_t xcd_item(int64_t items) {
  const int64_t per = (items + 7) / 8;
  return int64_t(blockIdx.x % 8u) * per + blockIdx.x / 8u;
}
inline unsigned xcd_grid(int64_t items) { return unsigned((items + 7) / 8 * 8); }

// the tiles [first, last) of `len` streamed rows that split `s` of `n` takes
__device__ __forceinline__ void split_range(int len, int s, int n, int* first, int* last) {
  const int tiles = (len + kTile - 1) / kTile, per = (tiles + n - 1) / n;
  *first = s * per < tiles ? s * per : tiles;
  *last = *first + per < tiles ? *first + per : tiles;
}

__device__ __forceinline__ float half_swap(float v) { return __shfl_xor(v, 32); }

// ---------------------------------------------------------------------------
// forward
// ---------------------------------------------------------------------------

template <typename T, int DP, int NW, int QB, bool MASK>
__global__ void __launch_bounds__(NW * 64) fwd_kernel(Params p) {
  using TL = TileOf<T, DP>;
  using E = Elt<T>;
  constexpr int NT = NW * 64, TC = NW * QB * 32;
  __shared__ __align__(16) char lk[2][TL::kBytes];
  __shared__ __align__(16) char lv[2][TL::kBytes];
  __shared__ unsigned long long lvalid[2];
  const int64_t item = xcd_item(int64_t(p.tiles) * p.hk * p.nsplit);
  if (item >= int64_t(p.tiles) * p.hk * p.nsplit) return;
  const int tile = int(item % p.tiles), hk = int(item / p.tiles % p.hk), split = int(item / p.tiles / p.hk);
  Segment sg;
  if (!find_segment(p.qoff, p.nq, p.koff, p.nk, p.batch, p.G, TC, tile, &sg)) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, half = lane >> 5;
  const int dchunks = p.d / TL::kVec;
  // the running maximum is taken on unscaled scores: a negative scale's sign goes into the queries (exactly), and a
  // scale of zero clears them (a masked score's -inf times 0 would be NaN)
  const float c = p.scale == 0.f ? 1.f : fabsf(p.scale) * kLog2e;
  const uint32_t clear = p.scale == 0.f ? 0u : ~0u;
  const uint32_t flip = p.scale < 0.f ? (sizeof(T) == 4 ? 0x80000000u : 0x80008000u) : 0u;

  // this lane's query columns
  int64_t row[QB];
  int head[QB];
  bool live[QB];
  u32x4 qf[QB][TL::kFrags];
#pragma unroll
  for (int b = 0; b < QB; ++b) {
    const uint32_t r = uint32_t(sg.tile) * TC + (wave * QB + b) * 32 + (lane & 31);
    live[b] = r < uint32_t(sg.len) * uint32_t(p.G);
    const uint32_t rc = live[b] ? r : 0u, tok = div_g(rc, p);
    row[b] = sg.begin + tok;
    head[b] = hk * p.G + int(rc - tok * uint32_t(p.G));
    const T* qp = static_cast<const T*>(p.q) + row[b] * p.q_row + head[b] * p.q_head;
#pragma unroll
    for (int f = 0; f < TL::kFrags; ++f) {
      const int ch = 2 * f + half;
      qf[b][f] = u32x4{0, 0, 0, 0};
      if (live[b] && ch < dchunks) {
        qf[b][f] = *reinterpret_cast<const u32x4*>(qp + ch * TL::kVec);
#pragma unroll
        for (int e = 0; e < 4; ++e) qf[b][f][e] = (qf[b][f][e] & clear) ^ flip;
      }
    }
  }

  f32x16 o[QB][TL::kBlocks];
  float m[QB], l[QB];
#pragma unroll
  for (int b = 0; b < QB; ++b) {
    m[b] = -INFINITY;
    l[b] = 0.f;
#pragma unroll
    for (int d = 0; d < TL::kBlocks; ++d) o[b][d] = f32x16{};
  }

  int t0, t1;
  split_range(sg.other_len, split, p.nsplit, &t0, &t1);
  const T* kp = static_cast<const T*>(p.k) + sg.other * p.k_row + hk * p.k_head;
  const T* vp = static_cast<const T*>(p.v) + sg.other * p.v_row + hk * p.v_head;
  Stage<T, DP, NT> sk, sv;
  uint8_t keep[Stage<T, DP, NT>::N];
  bool kept = false;  // the key of streamed row `lane`
  auto load = [&](int t) {
    const int64_t k0 = int64_t(t) * kTile;
    const int rows = sg.other_len - t * kTile;
    sk.load(rows, dchunks, [&](int r) { return kp + (k0 + r) * p.k_row; });
    sv.load(rows, dchunks, [&](int r) { return vp + (k0 + r) * p.v_row; });
    if constexpr (MASK) {
      const uint8_t* mp = p.mask + sg.other + k0;
#pragma unroll
      for (int i = 0; i < Stage<T, DP, NT>::N; ++i) {
        const int r = Stage<T, DP, NT>::item(i) / TL::CPR;
        keep[i] = (r < rows && r < kTile) ? mp[r] : 0;
      }
      kept = lane < rows && mp[lane] != 0;
    }
  };
  if (t0 < t1) load(t0);
  for (int t = t0; t < t1; ++t) {
    const int buf = (t - t0) & 1;
    if constexpr (MASK) {
      sk.clear(keep);
      sv.clear(keep);
      const uint64_t w = __ballot(kept);
      if (threadIdx.x == 0) lvalid[buf] = w;
    }
    sk.store(lk[buf]);
    sv.store(lv[buf]);
    __syncthreads();
    const int rows = sg.other_len - t * kTile;
    uint64_t valid = rows >= kTile ? ~0ull : (1ull << rows) - 1;
    if constexpr (MASK) valid = lvalid[buf];
    if (t + 1 < t1) load(t + 1);
    if (MASK && valid == 0) continue;

    f32x16 s[QB][2];
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) {
#pragma unroll
      for (int b = 0; b < QB; ++b) s[b][kb] = f32x16{};
#pragma unroll
      for (int f = 0; f < TL::kFrags; ++f) {
        const u32x4 a = TL::rows(lk[buf], 32 * kb, f);
#pragma unroll
        for (int b = 0; b < QB; ++b) s[b][kb] = E::mma(a, qf[b][f], s[b][kb]);
      }
    }
    if (~valid != 0) {
#pragma unroll
      for (int kb = 0; kb < 2; ++kb) {
        const uint32_t w = uint32_t(valid >> (32 * kb)) >> (4 * half);
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const bool on = (w >> (8 * (r / 4) + r % 4)) & 1u;
#pragma unroll
          for (int b = 0; b < QB; ++b) s[b][kb][r] = on ? s[b][kb][r] : -INFINITY;
        }
      }
    }
#pragma unroll
    for (int b = 0; b < QB; ++b) {
      float mx = s[b][0][0];
#pragma unroll
      for (int kb = 0; kb < 2; ++kb)
#pragma unroll
        for (int r = 0; r < 16; ++r) mx = fmaxf(mx, s[b][kb][r]);
      mx = fmaxf(mx, half_swap(mx)) * c;
      const float mn = fmaxf(m[b], mx);
      const float ref = mn == -INFINITY ? 0.f : mn;  // nothing attended yet
      const float al = __builtin_amdgcn_exp2f(m[b] - ref);
      m[b] = mn;
      l[b] *= al;
      const float sh = float(kPExp<T>) - ref;
#pragma unroll
      for (int kb = 0; kb < 2; ++kb)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const float e = __builtin_amdgcn_exp2f(fmaf(s[b][kb][r], c, sh));
          s[b][kb][r] = e;
          l[b] += e;
        }
#pragma unroll
      for (int d = 0; d < TL::kBlocks; ++d)
#pragma unroll
        for (int r = 0; r < 16; ++r) o[b][d][r] *= al;
    }
#pragma unroll
    for (int kb = 0; kb < 2; ++kb)
#pragma unroll
      for (int st = 0; st < E::kSteps; ++st) {
        u32x4 pf[QB];
#pragma unroll
        for (int b = 0; b < QB; ++b) pf[b] = E::pack(s[b][kb], st);
#pragma unroll
        for (int d = 0; d < TL::kBlocks; ++d) {
          const u32x4 a = TL::cols(lv[buf], 32 * kb, st, d);
#pragma unroll
          for (int b = 0; b < QB; ++b) o[b][d] = E::mma(a, pf[b], o[b][d]);
        }
      }
  }

#pragma unroll
  for (int b = 0; b < QB; ++b) {
    const float total = l[b] + half_swap(l[b]);
    if (!live[b]) continue;
    const bool some = total != 0.f;  // NaN counts
    if (p.nsplit > 1) {
      const int64_t at = (int64_t(split) * p.nq + row[b]) * p.hq + head[b];
      if (half == 0) {
        p.part_b[2 * at] = m[b];
        p.part_b[2 * at + 1] = total;
      }
      if (some) {
        float* op = p.part_a + at * p.d;
#pragma unroll
        for (int d = 0; d < TL::kBlocks; ++d)
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            const int e = 32 * d + 8 * g + 4 * half;
            if (e < p.d) *reinterpret_cast<float4*>(op + e) = make_float4(o[b][d][4 * g], o[b][d][4 * g + 1], o[b][d][4 * g + 2], o[b][d][4 * g + 3]);
          }
      }
      continue;
    }
    const float inv = some ? 1.f / total : 0.f;
    if (half == 0) p.lse[int64_t(head[b]) * p.nq + row[b]] = some ? (m[b] - float(kPExp<T>)) * kLn2 + logf(total) : -INFINITY;
    T* op = static_cast<T*>(p.o) + (row[b] * p.hq + head[b]) * p.d;
#pragma unroll
    for (int d = 0; d < TL::kBlocks; ++d)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const int e = 32 * d + 8 * g + 4 * half;
        if (e < p.d) {
          const float f0 = o[b][d][4 * g] * inv, f1 = o[b][d][4 * g + 1] * inv, f2 = o[b][d][4 * g + 2] * inv,
                      f3 = o[b][d][4 * g + 3] * inv;
          if constexpr (sizeof(T) == 4)
            *reinterpret_cast<float4*>(op + e) = make_float4(f0, f1, f2, f3);
          else
            *reinterpret_cast<uint2*>(op + e) = make_uint2(E::pack2(f0, f1), E::pack2(f2, f3));
        }
      }
  }
}

// Joins the splits of the forward pass: a wave per (row, head)
template <typename T>
__global__ void __launch_bounds__(256) fwd_join_kernel(Params p) {
  const int lane = threadIdx.x & 63;
  const int64_t rh = int64_t(blockIdx.x) * 4 + (threadIdx.x >> 6), n = p.nq * p.hq;
  if (rh >= n) return;
  float mx = -INFINITY;
  for (int s = 0; s < p.nsplit; ++s) mx = fmaxf(mx, p.part_b[2 * (s * n + rh)]);
  const float ref = mx == -INFINITY ? 0.f : mx;
  float total = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
  for (int s = 0; s < p.nsplit; ++s) {
    const float ls = p.part_b[2 * (s * n + rh) + 1];
    if (ls == 0.f) continue;
    const float w = __builtin_amdgcn_exp2f(p.part_b[2 * (s * n + rh)] - ref);
    total += w * ls;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (lane + 64 * e < p.d) acc[e] += w * p.part_a[(s * n + rh) * p.d + lane + 64 * e];
  }
  const bool some = total != 0.f;
  const float inv = some ? 1.f / total : 0.f;
  T* op = static_cast<T*>(p.o) + rh * p.d;
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (lane + 64 * e < p.d) op[lane + 64 * e] = T(acc[e] * inv);
  if (lane == 0)
    p.lse[(rh % p.hq) * p.nq + rh / p.hq] = some ? (mx - float(kPExp<T>)) * kLn2 + logf(total) : -INFINITY;
}

// ---------------------------------------------------------------------------
// backward
// ---------------------------------------------------------------------------

// delta[h][i] = sum over d of dout * out: a wave per four (row, head) pairs of 16 lanes.  fp16: also the largest
// |dout row|^2 and |v row|^2 (maxima: any order gives the same), which bound dS for its scaling to fp16's range.
template <typename T>
__global__ void __launch_bounds__(256) delta_kernel(Params p, uint32_t* bound) {
  constexpr int kVec = Elt<T>::kVec;
  const int sub = threadIdx.x & 15;
  const int64_t id = int64_t(blockIdx.x) * 16 + (threadIdx.x >> 4), nd = p.nq * p.hq;
  const int chunks = p.d / kVec;
  float acc = 0.f, sq = 0.f;
  const bool isq = id < nd;
  const int64_t vi = id - nd;
  const bool isv = sizeof(T) == 2 && bound && !isq && vi < p.nk * p.hk && (!p.mask || p.mask[vi / p.hk]);
  if (isq || isv) {
    const T* a = isq ? static_cast<const T*>(p.dout) + id * p.d
                     : static_cast<const T*>(p.v) + vi / p.hk * p.v_row + vi % p.hk * p.v_head;
    const T* o = static_cast<const T*>(p.out) + id * p.d;
    for (int ch = sub; ch < chunks; ch += 16) {
      const u32x4 x = *reinterpret_cast<const u32x4*>(a + ch * kVec);
      u32x4 y = u32x4{0, 0, 0, 0};
      if (isq) y = *reinterpret_cast<const u32x4*>(o + ch * kVec);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if constexpr (sizeof(T) == 4) {
          acc = fmaf(__uint_as_float(x[e]), __uint_as_float(y[e]), acc);
        } else {
          const float x0 = Elt<T>::lo(x[e]), x1 = Elt<T>::hi(x[e]);
          acc = fmaf(x0, Elt<T>::lo(y[e]), acc);
          acc = fmaf(x1, Elt<T>::hi(y[e]), acc);
          sq = fmaf(x0, x0, fmaf(x1, x1, sq));
        }
      }
    }
  }
#pragma unroll
  for (int d = 1; d < 16; d <<= 1) {
    acc += __shfl_xor(acc, d);
    sq += __shfl_xor(sq, d);
  }
  if (isq && sub == 0) p.delta[id % p.hq * p.nq + id / p.hq] = acc;
  if (sizeof(T) == 2 && bound) {
    float mq = isq && sq < INFINITY ? sq : 0.f, mv = isv && sq < INFINITY ? sq : 0.f;
#pragma unroll
    for (int d = 16; d < 64; d <<= 1) {
      mq = fmaxf(mq, __shfl_xor(mq, d));
      mv = fmaxf(mv, __shfl_xor(mv, d));
    }
    if ((threadIdx.x & 63) == 0) {
      if (mq > 0.f) atomicMax(&bound[0], __float_as_uint(mq));
      if (mv > 0.f) atomicMax(&bound[1], __float_as_uint(mv));
    }
  }
}

// clears the two bounds before the maxima
static __global__ void bound_clear_kernel(uint32_t* bound) {
  if (threadIdx.x < 2) bound[threadIdx.x] = 0u;
}

// Power of two for dS in fp16: |dS| <= |dP - delta| <= 2 |dout row| |v row| (out lies within the values it averages),
// so with b2 = max |dout row|^2 max |v row|^2 < 2^e the scaled dS stays below 2^(1 + e/2 + s) <= 2^15.5 < 65504 for
// s = 14 - floor(e / 2).  The rest of fp16's range (steps of 2^-24) is then all below the largest possible entry.
template <typename T>
__device__ __forceinline__ int ds_exp(const Params& p) {
  if constexpr (kPExp<T> == 0) {
    return 0;
  } else {
    const float b2 = __uint_as_float(p.bound[0]) * __uint_as_float(p.bound[1]);
    if (!(b2 > 0.f) || !(b2 < INFINITY)) return 0;
    int e;
    (void)frexpf(b2, &e);
    const int s = 14 - (e >> 1);
    return s < -30 ? -30 : (s > 60 ? 60 : s);
  }
}

// Loads resident columns (rows of a [n][head][d] tensor) as B fragments
template <typename T, int DP>
__device__ __forceinline__ void load_cols(const T* ptr, bool live, int dchunks, u32x4 (&f)[TileOf<T, DP>::kFrags]) {
  const int half = (threadIdx.x & 63) >> 5;
#pragma unroll
  for (int i = 0; i < TileOf<T, DP>::kFrags; ++i) {
    f[i] = u32x4{0, 0, 0, 0};
    if (live && 2 * i + half < dchunks) f[i] = *reinterpret_cast<const u32x4*>(ptr + (2 * i + half) * TileOf<T, DP>::kVec);
  }
}

// Writes a column block's transposed sums times f: rows of `dst` (T) or of fp32 partial sums
template <typename T, int DP>
__device__ __forceinline__ void store_cols(T* dst, float* part, const f32x16 (&o)[TileOf<T, DP>::kBlocks], int d, float f) {
  const int half = (threadIdx.x & 63) >> 5;
#pragma unroll
  for (int b = 0; b < TileOf<T, DP>::kBlocks; ++b)
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const int e = 32 * b + 8 * g + 4 * half;
      if (e >= d) continue;
      const float f0 = o[b][4 * g] * f, f1 = o[b][4 * g + 1] * f, f2 = o[b][4 * g + 2] * f, f3 = o[b][4 * g + 3] * f;
      if (part) {
        *reinterpret_cast<float4*>(part + e) = make_float4(f0, f1, f2, f3);
      } else if constexpr (sizeof(T) == 4) {
        *reinterpret_cast<float4*>(dst + e) = make_float4(f0, f1, f2, f3);
      } else {
        *reinterpret_cast<uint2*>(dst + e) = make_uint2(Elt<T>::pack2(f0, f1), Elt<T>::pack2(f2, f3));
      }
    }
}

template <typename T, int DP, int NW, int QB, bool MASK>
__global__ void __launch_bounds__(NW * 64) dq_kernel(Params p) {
  using TL = TileOf<T, DP>;
  using E = Elt<T>;
  constexpr int NT = NW * 64, TC = NW * QB * 32;
  __shared__ __align__(16) char lk[2][TL::kBytes];
  __shared__ __align__(16) char lv[2][TL::kBytes];
  __shared__ unsigned long long lvalid[2];
  const int64_t item = xcd_item(int64_t(p.tiles) * p.hk * p.nsplit);
  if (item >= int64_t(p.tiles) * p.hk * p.nsplit) return;
  const int tile = int(item % p.tiles), hk = int(item / p.tiles % p.hk), split = int(item / p.tiles / p.hk);
  Segment sg;
  if (!find_segment(p.qoff, p.nq, p.koff, p.nk, p.batch, p.G, TC, tile, &sg)) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, half = lane >> 5;
  const int dchunks = p.d / TL::kVec;
  const float c = p.scale * kLog2e;
  const int dse = ds_exp<T>(p);
  const float dsmul = ldexpf(1.f, dse - kPExp<T>);  // probabilities carry 2^kPExp

  int64_t row[QB];
  int head[QB];
  bool live[QB];
  u32x4 qf[QB][TL::kFrags], df[QB][TL::kFrags];
  float sh[QB], del[QB];
  f32x16 acc[QB][TL::kBlocks];
#pragma unroll
  for (int b = 0; b < QB; ++b) {
    const uint32_t r = uint32_t(sg.tile) * TC + (wave * QB + b) * 32 + (lane & 31);
    live[b] = r < uint32_t(sg.len) * uint32_t(p.G);
    const uint32_t rc = live[b] ? r : 0u, tok = div_g(rc, p);
    row[b] = sg.begin + tok;
    head[b] = hk * p.G + int(rc - tok * uint32_t(p.G));
    load_cols<T, DP>(static_cast<const T*>(p.q) + row[b] * p.q_row + head[b] * p.q_head, live[b], dchunks, qf[b]);
    load_cols<T, DP>(static_cast<const T*>(p.dout) + (row[b] * p.hq + head[b]) * p.d, live[b], dchunks, df[b]);
    const int64_t at = int64_t(head[b]) * p.nq + row[b];
    const float lse = live[b] ? p.lse[at] : -INFINITY;
    sh[b] = lse == -INFINITY ? -INFINITY : float(kPExp<T>) - lse * kLog2e;  // rows with no key: probabilities 0
    del[b] = live[b] ? p.delta[at] : 0.f;
#pragma unroll
    for (int d = 0; d < TL::kBlocks; ++d) acc[b][d] = f32x16{};
  }

  int t0, t1;
  split_range(sg.other_len, split, p.nsplit, &t0, &t1);
  const T* kp = static_cast<const T*>(p.k) + sg.other * p.k_row + hk * p.k_head;
  const T* vp = static_cast<const T*>(p.v) + sg.other * p.v_row + hk * p.v_head;
  Stage<T, DP, NT> sk, sv;
  uint8_t keep[Stage<T, DP, NT>::N];
  bool kept = false;
  auto load = [&](int t) {
    const int64_t k0 = int64_t(t) * kTile;
    const int rows = sg.other_len - t * kTile;
    sk.load(rows, dchunks, [&](int r) { return kp + (k0 + r) * p.k_row; });
    sv.load(rows, dchunks, [&](int r) { return vp + (k0 + r) * p.v_row; });
    if constexpr (MASK) {
      const uint8_t* mp = p.mask + sg.other + k0;
#pragma unroll
      for (int i = 0; i < Stage<T, DP, NT>::N; ++i) {
        const int r = Stage<T, DP, NT>::item(i) / TL::CPR;
        keep[i] = (r < rows && r < kTile) ? mp[r] : 0;
      }
      kept = lane < rows && mp[lane] != 0;
    }
  };
  if (t0 < t1) load(t0);
  for (int t = t0; t < t1; ++t) {
    const int buf = (t - t0) & 1;
    if constexpr (MASK) {
      sk.clear(keep);
      sv.clear(keep);
      const uint64_t w = __ballot(kept);
      if (threadIdx.x == 0) lvalid[buf] = w;
    }
    sk.store(lk[buf]);
    sv.store(lv[buf]);
    __syncthreads();
    const int rows = sg.other_len - t * kTile;
    uint64_t valid = rows >= kTile ? ~0ull : (1ull << rows) - 1;
    if constexpr (MASK) valid = lvalid[buf];
    if (t + 1 < t1) load(t + 1);
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) {
      const uint32_t vw = uint32_t(valid >> (32 * kb));
      if (vw == 0) continue;
      f32x16 s[QB], dp[QB];
#pragma unroll
      for (int b = 0; b < QB; ++b) s[b] = dp[b] = f32x16{};
#pragma unroll
      for (int f = 0; f < TL::kFrags; ++f) {
        const u32x4 a = TL::rows(lk[buf], 32 * kb, f), v = TL::rows(lv[buf], 32 * kb, f);
#pragma unroll
        for (int b = 0; b < QB; ++b) {
          s[b] = E::mma(a, qf[b][f], s[b]);
          dp[b] = E::mma(v, df[b][f], dp[b]);
        }
      }
#pragma unroll
      for (int b = 0; b < QB; ++b)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const float pr = __builtin_amdgcn_exp2f(fmaf(s[b][r], c, sh[b]));
          s[b][r] = pr * ((dp[b][r] - del[b]) * dsmul);
        }
      if (~vw != 0) {
        const uint32_t w = vw >> (4 * half);
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const bool on = (w >> (8 * (r / 4) + r % 4)) & 1u;
#pragma unroll
          for (int b = 0; b < QB; ++b) s[b][r] = on ? s[b][r] : 0.f;
        }
      }
#pragma unroll
      for (int st = 0; st < E::kSteps; ++st) {
        u32x4 pf[QB];
#pragma unroll
        for (int b = 0; b < QB; ++b) pf[b] = E::pack(s[b], st);
#pragma unroll
        for (int d = 0; d < TL::kBlocks; ++d) {
          const u32x4 a = TL::cols(lk[buf], 32 * kb, st, d);
#pragma unroll
          for (int b = 0; b < QB; ++b) acc[b][d] = E::mma(a, pf[b], acc[b][d]);
        }
      }
    }
  }
  const float f = ldexpf(p.scale, -dse);
#pragma unroll
  for (int b = 0; b < QB; ++b) {
    if (!live[b]) continue;
    const int64_t at = (row[b] * p.hq + head[b]) * p.d;
    store_cols<T, DP>(static_cast<T*>(p.dq) + at, p.nsplit > 1 ? p.part_a + int64_t(split) * p.nq * p.hq * p.d + at : nullptr,
                      acc[b], p.d, f);
  }
}

template <typename T, int DP, int NW, bool MASK>
__global__ void __launch_bounds__(NW * 64) dkv_kernel(Params p) {
  using TL = TileOf<T, DP>;
  using E = Elt<T>;
  constexpr int NT = NW * 64, TC = NW * 32;
  __shared__ __align__(16) char lq[2][TL::kBytes];
  __shared__ __align__(16) char ld[2][TL::kBytes];
  __shared__ __align__(16) float lsh[2][kTile], ldel[2][kTile];
  const int64_t item = xcd_item(int64_t(p.tiles) * p.hk * p.nsplit);
  if (item >= int64_t(p.tiles) * p.hk * p.nsplit) return;
  const int tile = int(item % p.tiles), hk = int(item / p.tiles % p.hk), split = int(item / p.tiles / p.hk);
  Segment sg;
  if (!find_segment(p.koff, p.nk, p.qoff, p.nq, p.batch, 1, TC, tile, &sg)) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, half = lane >> 5;
  const int dchunks = p.d / TL::kVec;
  const float c = p.scale * kLog2e;
  const int dse = ds_exp<T>(p);
  const float dsmul = ldexpf(1.f, dse - kPExp<T>);

  const int col = sg.tile * TC + wave * 32 + (lane & 31);
  const bool live = col < sg.len;
  const int64_t row = sg.begin + (live ? col : 0);
  const bool on = live && (!MASK || p.mask[row] != 0);
  u32x4 kf[TL::kFrags], vf[TL::kFrags];
  load_cols<T, DP>(static_cast<const T*>(p.k) + row * p.k_row + hk * p.k_head, on, dchunks, kf);
  load_cols<T, DP>(static_cast<const T*>(p.v) + row * p.v_row + hk * p.v_head, on, dchunks, vf);
  f32x16 dk[TL::kBlocks], dv[TL::kBlocks];
#pragma unroll
  for (int d = 0; d < TL::kBlocks; ++d) dk[d] = dv[d] = f32x16{};

  const int qrows = sg.other_len * p.G;  // (token, head) rows
  int t0, t1;
  split_range(qrows, split, p.nsplit, &t0, &t1);
  const T* qp = static_cast<const T*>(p.q) + sg.other * p.q_row + int64_t(hk) * p.G * p.q_head;
  const T* dp_ = static_cast<const T*>(p.dout) + (sg.other * p.hq + int64_t(hk) * p.G) * p.d;
  Stage<T, DP, NT> sq, sd;
  float rsh = -INFINITY, rdel = 0.f;
  auto load = [&](int t) {
    const int r0 = t * kTile, rows = qrows - r0;
    sq.load(rows, dchunks, [&](int r) {
      const uint32_t tok = div_g(uint32_t(r0 + r), p);
      return qp + int64_t(tok) * p.q_row + int64_t(uint32_t(r0 + r) - tok * uint32_t(p.G)) * p.q_head;
    });
    sd.load(rows, dchunks, [&](int r) {
      const uint32_t tok = div_g(uint32_t(r0 + r), p);
      return dp_ + (int64_t(tok) * p.hq + int64_t(uint32_t(r0 + r) - tok * uint32_t(p.G))) * p.d;
    });
    rsh = -INFINITY;
    rdel = 0.f;
    if (lane < rows) {
      const uint32_t tok = div_g(uint32_t(r0 + lane), p);
      const int64_t at = int64_t(hk * p.G + int(uint32_t(r0 + lane) - tok * uint32_t(p.G))) * p.nq + sg.other + tok;
      const float lse = p.lse[at];
      rsh = lse == -INFINITY ? -INFINITY : float(kPExp<T>) - lse * kLog2e;
      rdel = p.delta[at];
    }
  };
  if (t0 < t1) load(t0);
  for (int t = t0; t < t1; ++t) {
    const int buf = (t - t0) & 1;
    sq.store(lq[buf]);
    sd.store(ld[buf]);
    if (wave == 0) {
      lsh[buf][lane] = rsh;
      ldel[buf][lane] = rdel;
    }
    __syncthreads();
    if (t + 1 < t1) load(t + 1);
#pragma unroll
    for (int qb = 0; qb < 2; ++qb) {
      f32x16 s{}, dp{};
#pragma unroll
      for (int f = 0; f < TL::kFrags; ++f) {
        s = E::mma(TL::rows(lq[buf], 32 * qb, f), kf[f], s);
        dp = E::mma(TL::rows(ld[buf], 32 * qb, f), vf[f], dp);
      }
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const float4 sh4 = *reinterpret_cast<const float4*>(&lsh[buf][32 * qb + 8 * g + 4 * half]);
        const float4 de4 = *reinterpret_cast<const float4*>(&ldel[buf][32 * qb + 8 * g + 4 * half]);
        const float sh[4] = {sh4.x, sh4.y, sh4.z, sh4.w}, de[4] = {de4.x, de4.y, de4.z, de4.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float pr = __builtin_amdgcn_exp2f(fmaf(s[4 * g + j], c, sh[j]));
          s[4 * g + j] = pr;
          dp[4 * g + j] = pr * ((dp[4 * g + j] - de[j]) * dsmul);
        }
      }
#pragma unroll
      for (int st = 0; st < E::kSteps; ++st) {
        const u32x4 pf = E::pack(s, st), sf = E::pack(dp, st);
#pragma unroll
        for (int d = 0; d < TL::kBlocks; ++d) {
          dv[d] = E::mma(TL::cols(ld[buf], 32 * qb, st, d), pf, dv[d]);
          dk[d] = E::mma(TL::cols(lq[buf], 32 * qb, st, d), sf, dk[d]);
        }
      }
    }
  }
  if (!live) return;
  // a masked key has no gradient, whatever its zeroed column collected
  const float fk = on ? ldexpf(p.scale, -dse) : 0.f, fv = on ? ldexpf(1.f, -kPExp<T>) : 0.f;
  if (!on)
#pragma unroll
    for (int d = 0; d < TL::kBlocks; ++d) dk[d] = dv[d] = f32x16{};
  const int64_t at = (row * p.hk + hk) * p.d, sp = int64_t(split) * p.nk * p.hk * p.d + at;
  if (p.dk) store_cols<T, DP>(static_cast<T*>(p.dk) + at, p.nsplit > 1 ? p.part_a + sp : nullptr, dk, p.d, fk);
  if (p.dv) store_cols<T, DP>(static_cast<T*>(p.dv) + at, p.nsplit > 1 ? p.part_b + sp : nullptr, dv, p.d, fv);
}

// dst[i] = the sum of the splits' partial sums, in split order; four elements a thread
template <typename T>
__global__ void __launch_bounds__(256) sum_splits_kernel(const float* part, int64_t n4, int nsplit, T* dst) {
  const int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x;
  if (i >= n4) return;
  const float4* src = reinterpret_cast<const float4*>(part);
  float4 a = src[i];
  for (int s = 1; s < nsplit; ++s) {
    const float4 b = src[int64_t(s) * n4 + i];
    a.x += b.x;
    a.y += b.y;
    a.z += b.z;
    a.w += b.w;
  }
  if constexpr (sizeof(T) == 4)
    reinterpret_cast<float4*>(dst)[i] = a;
  else
    reinterpret_cast<uint2*>(dst)[i] = make_uint2(Elt<T>::pack2(a.x, a.y), Elt<T>::pack2(a.z, a.w));
}

// what the host decides before a launch
struct FwdPlan {
  int nw, qb, tiles, nsplit;
};
struct BwdPlan {
  int q_nw, q_qb, q_tiles, q_split;   // dQ
  int k_nw, k_tiles, k_split;         // dK and dV
};

// launches of one element type (defined once per type)
template <typename T>
int launch_fwd(const Params& p, const FwdPlan& f, hipStream_t s);
template <typename T>
int launch_bwd(Params p, const BwdPlan& b, float* part_q, float* part_k, float* part_v, uint32_t* bound, hipStream_t s);

// ---------------------------------------------------------------------------
// launches
// ---------------------------------------------------------------------------

template <typename T, int DP, int NW, int QB>
void launch_fwd_tile(const Params& p, hipStream_t s) {
  const unsigned grid = xcd_grid(int64_t(p.tiles) * p.hk * p.nsplit);
  if (p.mask)
    fwd_kernel<T, DP, NW, QB, true><<<grid, NW * 64, 0, s>>>(p);
  else
    fwd_kernel<T, DP, NW, QB, false><<<grid, NW * 64, 0, s>>>(p);
}

template <typename T, int DP>
void launch_fwd_dim(const Params& p, const FwdPlan& f, hipStream_t s) {
  if (f.nw == 1)
    launch_fwd_tile<T, DP, 1, 1>(p, s);
  else
    launch_fwd_tile<T, DP, 4, 1>(p, s);
}

template <typename T, int DP, int NW, int QB>
void launch_dq_tile(const Params& p, hipStream_t s) {
  const unsigned grid = xcd_grid(int64_t(p.tiles) * p.hk * p.nsplit);
  if (p.mask)
    dq_kernel<T, DP, NW, QB, true><<<grid, NW * 64, 0, s>>>(p);
  else
    dq_kernel<T, DP, NW, QB, false><<<grid, NW * 64, 0, s>>>(p);
}

template <typename T, int DP>
void launch_dq_dim(const Params& p, const BwdPlan& b, hipStream_t s) {
  if (b.q_nw == 1)
    launch_dq_tile<T, DP, 1, 1>(p, s);
  else
    launch_dq_tile<T, DP, 4, 1>(p, s);
}

template <typename T, int DP>
void launch_dkv_dim(const Params& p, hipStream_t s) {
  const unsigned grid = xcd_grid(int64_t(p.tiles) * p.hk * p.nsplit);
  if (p.mask)
    dkv_kernel<T, DP, 4, true><<<grid, 256, 0, s>>>(p);
  else
    dkv_kernel<T, DP, 4, false><<<grid, 256, 0, s>>>(p);
}

template <typename T>
int launch_fwd_impl(const Params& p, const FwdPlan& f, hipStream_t s) {
  if (p.d <= 32)
    launch_fwd_dim<T, 32>(p, f, s);
  else if (p.d <= 64)
    launch_fwd_dim<T, 64>(p, f, s);
  else if (p.d <= 96)
    launch_fwd_dim<T, 96>(p, f, s);
  else
    launch_fwd_dim<T, 128>(p, f, s);
  if (p.nsplit > 1) fwd_join_kernel<T><<<unsigned((p.nq * p.hq + 3) / 4), 256, 0, s>>>(p);
  return hipGetLastError() == hipSuccess ? SSC_OK : SSC_ERR_HIP;
}

template <typename T>
int launch_bwd_impl(Params p, const BwdPlan& b, float* part_q, float* part_k, float* part_v, uint32_t* bound,
                    hipStream_t s) {
  const bool scaled = kPExp<T> != 0;
  if (scaled) bound_clear_kernel<<<1, 64, 0, s>>>(bound);
  p.bound = bound;
  const int64_t groups = p.nq * p.hq + (scaled ? p.nk * p.hk : 0);
  if (groups > 0) delta_kernel<T><<<unsigned((groups + 15) / 16), 256, 0, s>>>(p, scaled ? bound : nullptr);
  if (p.dq && p.nq > 0) {
    p.tiles = b.q_tiles;
    p.nsplit = b.q_split;
    p.part_a = part_q;
    if (p.d <= 32)
      launch_dq_dim<T, 32>(p, b, s);
    else if (p.d <= 64)
      launch_dq_dim<T, 64>(p, b, s);
    else if (p.d <= 96)
      launch_dq_dim<T, 96>(p, b, s);
    else
      launch_dq_dim<T, 128>(p, b, s);
    if (p.nsplit > 1) {
      const int64_t n4 = p.nq * p.hq * p.d / 4;
      sum_splits_kernel<T><<<unsigned((n4 + 255) / 256), 256, 0, s>>>(part_q, n4, p.nsplit, static_cast<T*>(p.dq));
    }
  }
  if ((p.dk || p.dv) && p.nk > 0) {
    p.tiles = b.k_tiles;
    p.nsplit = b.k_split;
    p.part_a = part_k;
    p.part_b = part_v;
    if (p.d <= 32)
      launch_dkv_dim<T, 32>(p, s);
    else if (p.d <= 64)
      launch_dkv_dim<T, 64>(p, s);
    else if (p.d <= 96)
      launch_dkv_dim<T, 96>(p, s);
    else
      launch_dkv_dim<T, 128>(p, s);
    if (p.nsplit > 1) {
      const int64_t n4 = p.nk * p.hk * p.d / 4;
      const unsigned grid = unsigned((n4 + 255) / 256);
      if (p.dk) sum_splits_kernel<T><<<grid, 256, 0, s>>>(part_k, n4, p.nsplit, static_cast<T*>(p.dk));
      if (p.dv) sum_splits_kernel<T><<<grid, 256, 0, s>>>(part_v, n4, p.nsplit, static_cast<T*>(p.dv));
    }
  }
  return hipGetLastError() == hipSuccess ? SSC_OK : SSC_ERR_HIP;
}

}  // namespace attn
}  // namespace ssc
