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
//
// WIN: windowed attention.  Token i of a sample sits at place t = i + (keys - tokens) of the sample's keys and sees the
// keys j <= t + right with j >= t - left or j < sinks.  A workgroup streams only the rows that one of its columns sees:
// the sinks' tiles, then tiles that begin with the first row of its columns' windows and end with the last one's, so
// rows that no column sees are not read.  Tiles that every column of a wave sees whole skip the comparison; the others
// turn a column's bounds into a word of a bit per streamed row.
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
// streamed rows of an LDS tile: 32 for fp32, whose 64 would not fit the registers on their way
constexpr int tile_rows(int esize) { return esize == 4 ? 32 : 64; }

struct Params {
  const void *q, *k, *v, *out, *dout;
  void *o, *dq, *dk, *dv;
  float* lse;          // [hq][nq]
  float* delta;        // [hq][nq], backward: sum over d of dout * out, as the dQ pass corrects it
  // backward, fp16: maxima of |dout row|^2 and |v row|^2 by key head and piece of rows (see piece_rows)
  const float *top_q, *top_k;
  int32_t q_piece, k_piece, q_pieces, k_pieces;  // rows of a piece, pieces
  const int32_t *qoff, *koff;
  const uint8_t* mask;
  int64_t nq, nk;
  int64_t q_row, q_head, k_row, k_head, v_row, v_head;  // strides in elements
  int32_t batch, hq, hk, d, G;
  uint32_t gmul;
  int32_t gshift;      // r / G = (r * gmul) >> gshift for r < 2^31
  float scale;
  int32_t tiles, nsplit;
  int32_t left, right, sinks;  // WIN
  // splits: partial sums [nsplit][rows][d]; forward part_b: [nsplit][rows][2] (max, sum); dQ part_e: [nsplit][rows][2]
  float *part_a, *part_b, *part_e;
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
  // acc + the products of the elements two words hold
  __device__ static __forceinline__ float dot(uint32_t a, uint32_t b, float acc) {
    return fmaf(__uint_as_float(a), __uint_as_float(b), acc);
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
  // acc + the two elements a word holds
  __device__ static __forceinline__ float sum(uint32_t a, float acc) {
    return __builtin_amdgcn_fdot2(__builtin_bit_cast(f16x2, a), f16x2{_Float16(1.f), _Float16(1.f)}, acc, false);
  }
  __device__ static __forceinline__ float dot(uint32_t a, uint32_t b, float acc) {
    return fmaf(hi(a), hi(b), fmaf(lo(a), lo(b), acc));
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
  // acc + the two elements a word holds
  __device__ static __forceinline__ float sum(uint32_t a, float acc) {
    return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, a), bf16x2{__bf16(1.f), __bf16(1.f)}, acc, false);
  }
  __device__ static __forceinline__ float dot(uint32_t a, uint32_t b, float acc) {
    return fmaf(hi(a), hi(b), fmaf(lo(a), lo(b), acc));
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

// Probabilities and dS are rounded to a 16-bit type for the second products, whose operands they are: results have about
// 1.4 times the error of ones only rounded at the end.  Their remainders as a second operand would take that out with two
// to three more products on the backward pass's eight.
//
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

// Geometry of one LDS tile of kRows streamed rows and DP (head size rounded up to 32) elements, and its reads
template <typename T, int DP, int R = tile_rows(sizeof(T))>
struct TileOf {
  static constexpr int kVec = Elt<T>::kVec;
  static constexpr int CPR = DP / kVec;            // chunks per row
  static constexpr int kRows = R, kGroups = R / 32;
  static constexpr int kBytes = kRows * CPR * 16;
  static constexpr int kFrags = DP / (2 * kVec);   // operand fragments along the head dimension
  static constexpr int kBlocks = DP / 32;          // 32-wide blocks of the head dimension

  // whether fragment f lies past the head's `dchunks` chunks; 16-bit products are too short to gain from a branch
  __device__ static __forceinline__ bool skip(int f, int dchunks) { return sizeof(T) == 4 && 2 * f >= dchunks; }
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

__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const void* base, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, int(bytes), 0x00027000);
}

// Tiles of R rows, one after another: where the next one starts and how many bytes its rows span (row strides are
// bounded so that a whole tile's fit 32 bits)
template <int R>
struct Walk {
  const char* at;
  int64_t step;
  uint32_t row_bytes, head_bytes, full;
  __device__ __forceinline__ void init(int64_t row, uint32_t head) {
    row_bytes = uint32_t(row);
    head_bytes = head;
    full = uint32_t(R - 1) * row_bytes + head;
    step = R * row;
  }
  __device__ __forceinline__ uint32_t span(int rows) const {
    return rows >= R ? full : uint32_t(rows - 1) * row_bytes + head_bytes;
  }
};

// A tile on its way from memory to LDS, NT threads (a workgroup, or one wave): 16-byte chunks in registers.  The loads go through a buffer
// descriptor that ends with the sample's last row, so rows past it (and chunks past the head) read as zeros with no
// branch, and a thread's offsets inside a tile are computed once for all tiles.
template <typename T, int DP, int NT, int R = tile_rows(sizeof(T))>
struct Stage {
  using TL = TileOf<T, DP, R>;
  static constexpr int kTotal = TL::kRows * TL::CPR;
  static constexpr int N = (kTotal + NT - 1) / NT;
  u32x4 r[N];
  uint32_t off[N];
  __device__ static __forceinline__ int item(int i) { return int(threadIdx.x) % NT + i * NT; }
  __device__ static __forceinline__ bool any(int i) { return kTotal % NT == 0 || item(i) < kTotal; }
  // row_bytes: from one row to the next; dchunks: chunks the head fills
  __device__ __forceinline__ void init(uint32_t row_bytes, int dchunks) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int row = item(i) / TL::CPR, c = item(i) % TL::CPR;
      off[i] = (any(i) && c < dchunks) ? uint32_t(row) * row_bytes + uint32_t(c) * 16u : 0xFFFFFFF0u;
    }
  }
  // the rows at `base` that the next `span` bytes hold
  __device__ __forceinline__ void load(const void* base, uint32_t span) {
    const auto rsrc = buffer_of(base, span);
#pragma unroll
    for (int i = 0; i < N; ++i) r[i] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rsrc, int(off[i]), 0, 0));
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

// a value every lane holds alike, in scalar registers
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ int64_t uniform(int64_t v) {
  return int64_t(uint64_t(uint32_t(uniform(int(v >> 32)))) << 32 | uint32_t(uniform(int(v))));
}

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
  int32_t index;   // of the segment: 0 before the first sample, b + 1 for sample b
};

// Finds tile t of the segments; false where there is none.  Segment s of rows b .. e - 1 owns the tiles from
// floor(b mult / cols) + s up to the next segment's, which are enough for its rows (ceil(x - y) <= floor(x) - floor(y) + 1)
// and number the tiles of a launch without a table of where a segment's begin; it leaves the last of them idle where one
// less would do.  The segment is the last one whose first tile is not past t: each lane looks at one of 64 candidates, and
// in the last round (the only one up to 62 samples) at all of its offsets side by side.  A walk over the samples, 64 at a
// time, took a time that grew with them (windows of 17 keys, 4 heads of 64, bf16, forward: 16,384 samples of 16 rows
// 23 ms, and now 0.87; 1,024 of 256 rows 251 us, and 154).
// most: tiles of the samples' first `most` rows only, as many for each sample where that is fewer in all.
__device__ __forceinline__ bool find_segment(const int32_t* off, int64_t n, const int32_t* other_off, int64_t other_n,
                                             int batch, int mult, int cols, int t, Segment* seg, int most = 0x7FFFFFFF) {
  const int lane = threadIdx.x & 63;
  const int per = int64_t(most) * batch < n ? (most + cols - 1) / cols : 0;
  int at = 0, end = batch + 2;
  if (per > 0) {
    at = t / per + 1;
    if (at > batch) return false;
    end = at + 1;
  }
  for (int step = 0; step != 1;) {
    step = (end - at + 63) / 64;
    const int s = at + lane * step;
    const bool in = s < end;
    const int lo = s < 1 ? 0 : (s - 1 < batch ? s - 1 : batch), hi = s < batch ? s : batch;
    int64_t b = clamp_off(off, lo, n), e = 0, ob = 0, oe = 0;
    if (step == 1) {
      e = clamp_off(off, hi, n);
      ob = clamp_off(other_off, lo, other_n);
      oe = clamp_off(other_off, hi, other_n);
    }
    if (s == 0) b = 0;
    const int first = per > 0 ? (s - 1) * per : int(b * mult / cols) + s;
    const int k = __popcll(__ballot(in && first <= t)) - 1, w = uniform(k < 0 ? 0 : k);
    if (step == 1) {
      if (s == batch + 1) e = n;
      if (e < b) e = b;
      const int len = int(e - b), olen = s >= 1 && s <= batch && oe > ob ? int(oe - ob) : 0;
      // rows are below 2^28: offsets fit an int
      seg->begin = __builtin_amdgcn_readlane(int(b), w);
      seg->len = __builtin_amdgcn_readlane(len, w);
      seg->tile = t - __builtin_amdgcn_readlane(first, w);
      seg->other = __builtin_amdgcn_readlane(int(ob), w);
      seg->other_len = __builtin_amdgcn_readlane(olen, w);
      seg->index = uniform(at) + w;
    } else {
      at += w * step;
      end = at + step < end ? at + step : end;
    }
  }
  if (most != 0x7FFFFFFF && (seg->index < 1 || seg->index > batch)) return false;
  const int rows = seg->len < most ? seg->len : most;
  return seg->tile >= 0 && int64_t(seg->tile) * cols < int64_t(rows) * mult;
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

// the share [first, last) of `tiles` streamed tiles that split `s` of `n` takes
__device__ __forceinline__ void split_range(int tiles, int s, int n, int* first, int* last) {
  const int per = (tiles + n - 1) / n;
  *first = s * per < tiles ? s * per : tiles;
  *last = *first + per < tiles ? *first + per : tiles;
}

// bits 0 .. n - 1
__device__ __forceinline__ uint64_t below(int n) { return n <= 0 ? 0ull : (n >= 64 ? ~0ull : (1ull << n) - 1); }

// The key rows that a workgroup's query columns see (WIN): the sinks' tiles, then the window's, each R rows.  Where the
// two meet they are one run of tiles from row 0.
struct Seen {
  int sink_tiles, sink_end, first, end, tiles;
  // place0, place1: of the first and the last column
  __device__ __forceinline__ void init(const Params& p, int place0, int place1, int keys, int R) {
    end = place1 + p.right + 1;
    end = end < 0 ? 0 : (end < keys ? end : keys);
    first = place0 - p.left;
    first = first < 0 ? 0 : (first < end ? first : end);
    sink_end = p.sinks < end ? p.sinks : end;
    if (first <= sink_end) first = sink_end = 0;
    sink_tiles = (sink_end + R - 1) / R;
    tiles = sink_tiles + (end - first + R - 1) / R;
  }
  __device__ __forceinline__ int row(int t, int R) const { return t < sink_tiles ? t * R : first + (t - sink_tiles) * R; }
  __device__ __forceinline__ int rows(int t, int R) const { return (t < sink_tiles ? sink_end : end) - row(t, R); }
};

// bit k: whether the column at `place` sees key row0 + k
__device__ __forceinline__ uint64_t sees(const Params& p, int place, int row0) {
  return below(place + p.right + 1 - row0) & (~below(place - p.left - row0) | below(p.sinks - row0));
}

// Waves per SIMD the registers are held to.  Two waves overlap their matrix and vector phases: with one (and
// accumulators in the second register half) the passes ran at 0.5 to 0.7 of their speed.  Some forms keep more than these
// limits hold and put registers into scratch, by the compiler's report: dQ over few rows with heads of 33 to 64 (6 to 45
// registers a lane, most with a mask) and masked over 96 (1 to 4), dQ with heads of 65 to 96 (16 to 19 with a mask, 4 in
// fp16 without), and fp32 with heads over 96: the masked few-rows forward 36, dQ over few rows 41 to 90, dK and dV 57.
struct Cfg {
  int fwd_occ, dq_occ, dkv_occ;
};
constexpr Cfg tile_cfg(int esize, int dp) {
  return dp <= 64 ? Cfg{2, 2, 2} : esize == 4 ? Cfg{1, 1, 1} : Cfg{2, dp == 96 ? 2 : 1, 2};
}
// Waves of a forward workgroup: eight for 16-bit heads of over 96, whose tiles (64 KiB) then serve both waves of every
// SIMD (2 x 11.2k rows, 8 heads of 128, bf16: 1.08 -> 1.01 ms); narrower heads run alike with four.
constexpr int fwd_waves(int esize, int dp) { return esize == 2 && dp == 128 ? 8 : 4; }

// keeps a wave's LDS writes before the reads that follow; the hardware serves them in order
__device__ __forceinline__ void wave_fence() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

__device__ __forceinline__ float half_swap(float v) { return __shfl_xor(v, 32); }

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

// ---------------------------------------------------------------------------
// forward
// ---------------------------------------------------------------------------

// Forward exponentials are taken against a reference at most kSlack (a power of two's exponent) below the row's
// maximum, with an offset that keeps the largest inside fp16's 65504.
template <typename T>
constexpr int kFwdExp = __is_same(T, _Float16) ? 8 : 0;
constexpr float kSlack = 7.f;

// factor from scores, and their maxima, to exponents of two
__device__ __forceinline__ float exp_unit(const Params& p) { return p.scale == 0.f ? 1.f : fabsf(p.scale) * kLog2e; }
// ln sum exp of a row from its reference score and its sum
template <typename T>
__device__ __forceinline__ float lse_of(const Params& p, float m, float total) {
  return fmaf(m, fabsf(p.scale), logf(total) - float(kFwdExp<T>) * kLn2);
}

// Online softmax: per tile of keys s = q k^T, the reference m follows the row's maximum, p = 2^(c s - m), l += sum p,
// o += p v; out = o / l and lse = m + ln l.  A wave keeps 32 query columns: their fragments, sums and statistics are
// registers, and one tile of 64 keys costs it 16 MFMA (head of 64) against about 200 vector instructions, so both units
// bound it, and power: self attention of 2 x 11.2k rows, 16 heads of 64, bf16, takes 1.15 ms (0.9 PFLOP/s; MFMA 44 %
// and vector issue 70 % of the cycles), 22.4k rows over 4,099 keys, 8 heads of 128, fp16, 0.40 ms (0.93 PFLOP/s).
//
// Two forms.  Rows: the workgroup's waves own different columns and share the streamed tiles, double buffered in LDS
// with one barrier a tile.  FEW (a sample's rows fit 32 columns: single tokens while serving): the waves share the
// columns and take the tiles in turn, each through an LDS tile of its own with no barrier, and join their sums at the
// end; four rows pooling 0.8M keys, 4 heads of 64, run at 5.2 TB/s.
template <typename T, int DP, int NW, bool MASK, bool FEW, bool WIN>
__global__ void __launch_bounds__(NW * 64, FEW ? 2 : tile_cfg(sizeof(T), DP).fwd_occ) fwd_kernel(Params p) {
  using TL = TileOf<T, DP>;
  using E = Elt<T>;
  constexpr int NT = FEW ? 64 : NW * 64, TC = FEW ? 32 : NW * 32, BUFS = FEW ? NW : 2;
  __shared__ __align__(16) char lds[2 * BUFS * TL::kBytes];
  __shared__ unsigned long long lvalid[BUFS];
  __shared__ float lml[FEW ? 2 * NW * 32 : 1];
  const int64_t item = xcd_item(int64_t(p.tiles) * p.hk * p.nsplit);
  if (item >= int64_t(p.tiles) * p.hk * p.nsplit) return;
  const int tile = int(item % p.tiles), hk = int(item / p.tiles % p.hk), split = int(item / p.tiles / p.hk);
  Segment sg;
  if (!find_segment(p.qoff, p.nq, p.koff, p.nk, p.batch, p.G, TC, tile, &sg)) return;
  const int lane = threadIdx.x & 63, wave = uniform(int(threadIdx.x >> 6)), half = lane >> 5;
  const int dchunks = p.d / TL::kVec;
  // the running maximum is taken on unscaled scores: a negative scale's sign goes into the queries (exactly), and a
  // scale of zero clears them (a masked score's -inf times 0 would be NaN)
  const float c = exp_unit(p);
  const uint32_t clear = p.scale == 0.f ? 0u : ~0u;
  const uint32_t flip = p.scale < 0.f ? (sizeof(T) == 4 ? 0x80000000u : 0x80008000u) : 0u;

  // this lane's query columns
  u32x4 qf[TL::kFrags];
  const uint32_t r = uint32_t(sg.tile) * TC + (FEW ? 0 : wave * 32) + (lane & 31);
  const bool live = r < uint32_t(sg.len) * uint32_t(p.G);
  const uint32_t rc = live ? r : 0u, tok = div_g(rc, p);
  const int64_t row = sg.begin + tok;
  const int head = hk * p.G + int(rc - tok * uint32_t(p.G));
  load_cols<T, DP>(static_cast<const T*>(p.q) + row * p.q_row + head * p.q_head, live, dchunks, qf);
#pragma unroll
  for (int f = 0; f < TL::kFrags; ++f)
#pragma unroll
    for (int e = 0; e < 4; ++e) qf[f][e] = (qf[f][e] & clear) ^ flip;

  f32x16 o[TL::kBlocks];
  float m = -INFINITY, l = 0.f;
#pragma unroll
  for (int d = 0; d < TL::kBlocks; ++d) o[d] = f32x16{};

  int t0, t1;
  Seen seen;
  int place = 0, place0 = 0, place1 = 0;  // of this lane's column, of the wave's first and last ones
  if constexpr (WIN) {
    const int shift = sg.other_len - sg.len, lastr = int(uint32_t(sg.len) * uint32_t(p.G)) - 1;
    auto at = [&](int c) { return int(div_g(uint32_t(c < lastr ? c : lastr), p)) + shift; };
    const int c0 = sg.tile * TC, w0 = c0 + (FEW ? 0 : wave * 32);
    place = at(w0 + (lane & 31));
    place0 = at(w0);
    place1 = at(w0 + 31);
    seen.init(p, at(c0), at(c0 + TC - 1), sg.other_len, TL::kRows);
  }
  split_range(WIN ? seen.tiles : (sg.other_len + TL::kRows - 1) / TL::kRows, split, p.nsplit, &t0, &t1);
  constexpr int step = FEW ? NW : 1;
  if (FEW) t0 += wave;
  const uint32_t head_bytes = uint32_t(p.d) * uint32_t(sizeof(T));
  Walk<TL::kRows> wk, wv;
  wk.init(p.k_row * int64_t(sizeof(T)), head_bytes);
  wv.init(p.v_row * int64_t(sizeof(T)), head_bytes);
  const char* k0 = reinterpret_cast<const char*>(static_cast<const T*>(p.k) + sg.other * p.k_row + hk * p.k_head);
  const char* v0 = reinterpret_cast<const char*>(static_cast<const T*>(p.v) + sg.other * p.v_row + hk * p.v_head);
  wk.at = k0 + t0 * wk.step;
  wv.at = v0 + t0 * wv.step;
  Stage<T, DP, NT> sk, sv;
  sk.init(wk.row_bytes, dchunks);
  sv.init(wv.row_bytes, dchunks);
  uint8_t keep[Stage<T, DP, NT>::N];
  bool kept = false;  // the key of streamed row `lane`
  auto load = [&](int t) {
    const int rows = WIN ? seen.rows(t, TL::kRows) : sg.other_len - t * TL::kRows;
    if constexpr (WIN) {
      wk.at = k0 + int64_t(seen.row(t, TL::kRows)) * wk.row_bytes;
      wv.at = v0 + int64_t(seen.row(t, TL::kRows)) * wv.row_bytes;
    }
    sk.load(wk.at, wk.span(rows));
    sv.load(wv.at, wv.span(rows));
    if constexpr (!WIN) {
      wk.at += step * wk.step;
      wv.at += step * wv.step;
    }
    if constexpr (MASK) {
      const uint8_t* mp = p.mask + sg.other + (WIN ? int64_t(seen.row(t, TL::kRows)) : int64_t(t) * TL::kRows);
#pragma unroll
      for (int i = 0; i < Stage<T, DP, NT>::N; ++i) {
        const int r = Stage<T, DP, NT>::item(i) / TL::CPR;
        keep[i] = (r < rows && r < TL::kRows) ? mp[r] : 0;
      }
      kept = lane < rows && lane < TL::kRows && mp[lane] != 0;
    }
  };
  if (t0 < t1) load(t0);
  for (int t = t0, n = 0; t < t1; t += step, ++n) {
    const int buf = FEW ? wave : n & 1;
    char* lk = lds + buf * 2 * TL::kBytes;
    char* lv = lk + TL::kBytes;
    constexpr uint64_t kAll = ~0ull >> (64 - TL::kRows);
    uint64_t valid = 0;
    if constexpr (MASK) {
      sk.clear(keep);
      sv.clear(keep);
      valid = __ballot(kept);
      if (!FEW && threadIdx.x == 0) lvalid[buf] = valid;
    }
    sk.store(lk);
    sv.store(lv);
    if constexpr (FEW)
      wave_fence();  // LDS serves a wave's accesses in order
    else
      __syncthreads();
    const int rows = WIN ? seen.rows(t, TL::kRows) : sg.other_len - t * TL::kRows;
    if constexpr (!MASK)
      valid = rows >= TL::kRows ? kAll : (1ull << rows) - 1;
    else if constexpr (!FEW)
      valid = lvalid[buf];
    if (t + step < t1) load(t + step);
    if (MASK && valid == 0) continue;
    bool part = valid != kAll;  // some row is not seen by some column
    if constexpr (WIN) {
      const int row0 = seen.row(t, TL::kRows);
      if (row0 < place1 - p.left || row0 + TL::kRows - 1 > place0 + p.right) {
        valid &= sees(p, place, row0);
        if (!__any(valid != 0)) continue;
        part = true;
      }
    }

    f32x16 s[TL::kGroups];
#pragma unroll
    for (int kb = 0; kb < TL::kGroups; ++kb) {
      s[kb] = f32x16{};
#pragma unroll
      for (int f = 0; f < TL::kFrags; ++f) {
        if (TL::skip(f, dchunks)) break;
        const u32x4 a = TL::rows(lk, 32 * kb, f);
        s[kb] = E::mma(a, qf[f], s[kb]);
      }
    }
    if (part) {
#pragma unroll
      for (int kb = 0; kb < TL::kGroups; ++kb) {
        const uint32_t w = uint32_t(valid >> (32 * kb)) >> (4 * half);
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const bool on = (w >> (8 * (r / 4) + r % 4)) & 1u;
          s[kb][r] = on ? s[kb][r] : -INFINITY;
        }
      }
    }
    float mx = s[0][0];
#pragma unroll
    for (int kb = 0; kb < TL::kGroups; ++kb)
#pragma unroll
      for (int r = 0; r < 16; ++r) mx = fmaxf(mx, s[kb][r]);
    mx = fmaxf(mx, half_swap(mx));
    // The reference point of the exponentials follows the running maximum only when a row's has grown past what the
    // type holds (2^kSlack): any reference gives the same quotient, and most tiles then skip the rescaling.
    if (__any((mx - m) * c > kSlack)) {
      const float mn = fmaxf(m, mx);
      const float al = m == mn ? 1.f : __builtin_amdgcn_exp2f((m - mn) * c);  // -inf stays: nothing attended yet
      m = mn;
      l *= al;
#pragma unroll
      for (int d = 0; d < TL::kBlocks; ++d)
#pragma unroll
        for (int r = 0; r < 16; ++r) o[d][r] *= al;
    }
    const float ref = m == -INFINITY ? 0.f : m;
    const float sh = float(kFwdExp<T>) - ref * c;
#pragma unroll
    for (int kb = 0; kb < TL::kGroups; ++kb)
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        // fp32 subtracts before it scales, which rounds the difference and not the score
        const float e = __builtin_amdgcn_exp2f(sizeof(T) == 4 ? (s[kb][r] - ref) * c : fmaf(s[kb][r], c, sh));
        s[kb][r] = e;
        l += e;
      }
#pragma unroll
    for (int kb = 0; kb < TL::kGroups; ++kb)
#pragma unroll
      for (int st = 0; st < E::kSteps; ++st) {
        const u32x4 pf = E::pack(s[kb], st);
#pragma unroll
        for (int d = 0; d < TL::kBlocks; ++d) {
          const u32x4 a = TL::cols(lv, 32 * kb, st, d);
          o[d] = E::mma(a, pf, o[d]);
        }
      }
  }

  if constexpr (FEW) {
    // The waves' references differ: each wave's sums are brought to the largest, then added in wave order.  2 NW
    // threads share a column's elements.
    float total = l + half_swap(l);
    if (half == 0) {
      lml[wave * 32 + lane] = m;
      lml[(NW + wave) * 32 + lane] = total;
    }
    __syncthreads();
    float mx = -INFINITY;
#pragma unroll
    for (int w = 0; w < NW; ++w) mx = fmaxf(mx, lml[w * 32 + (lane & 31)]);
    const float al = m == mx ? 1.f : __builtin_amdgcn_exp2f((m - mx) * c);
    float* mine = reinterpret_cast<float*>(lds) + wave * DP * 33;
#pragma unroll
    for (int d = 0; d < TL::kBlocks; ++d)
#pragma unroll
      for (int r = 0; r < 16; ++r) mine[(32 * d + 8 * (r / 4) + 4 * half + r % 4) * 33 + (lane & 31)] = o[d][r] * al;
    __syncthreads();
    constexpr int TPC = 2 * NW;
    const int col = threadIdx.x / TPC, e0 = threadIdx.x % TPC;
    const uint32_t r = uint32_t(sg.tile) * TC + col;
    if (r >= uint32_t(sg.len) * uint32_t(p.G)) return;
    const uint32_t tok = div_g(r, p);
    const int64_t orow = sg.begin + tok;
    const int ohead = hk * p.G + int(r - tok * uint32_t(p.G));
    mx = -INFINITY;
#pragma unroll
    for (int w = 0; w < NW; ++w) mx = fmaxf(mx, lml[w * 32 + col]);
    total = 0.f;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      const float mw = lml[w * 32 + col];
      total += lml[(NW + w) * 32 + col] * (mw == mx ? 1.f : __builtin_amdgcn_exp2f((mw - mx) * c));
    }
    const bool some = total != 0.f;  // NaN counts
    const float inv = p.nsplit > 1 ? 1.f : (some ? 1.f / total : 0.f);
    const int64_t at = (int64_t(split) * p.nq + orow) * p.hq + ohead;
    for (int e = e0; e < p.d; e += TPC) {
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < NW; ++w) v += reinterpret_cast<const float*>(lds)[w * DP * 33 + e * 33 + col];
      if (p.nsplit > 1)
        p.part_a[at * p.d + e] = v;
      else
        static_cast<T*>(p.o)[(orow * p.hq + ohead) * p.d + e] = T(v * inv);
    }
    if (e0 == 0) {
      if (p.nsplit > 1) {
        p.part_b[2 * at] = mx;
        p.part_b[2 * at + 1] = total;
      } else {
        p.lse[int64_t(ohead) * p.nq + orow] = some ? lse_of<T>(p, mx, total) : -INFINITY;
      }
    }
    return;
  }

  const float total = l + half_swap(l);
  if (!live) return;
  const bool some = total != 0.f;  // NaN counts
  if (p.nsplit > 1) {
    const int64_t at = (int64_t(split) * p.nq + row) * p.hq + head;
    if (half == 0) {
      p.part_b[2 * at] = m;
      p.part_b[2 * at + 1] = total;
    }
    store_cols<T, DP>(nullptr, p.part_a + at * p.d, o, p.d, 1.f);
    return;
  }
  if (half == 0)
    p.lse[int64_t(head) * p.nq + row] = some ? lse_of<T>(p, m, total) : -INFINITY;
  store_cols<T, DP>(static_cast<T*>(p.o) + (row * p.hq + head) * p.d, nullptr, o, p.d, some ? 1.f / total : 0.f);
}

constexpr int kMaxSplit = 128;

// up to this many splits a wave joins a row's one after another, four rows a workgroup
constexpr int kFewSplits = 8;

// Joins the splits of the forward pass.  Many splits (WIDE): a workgroup per (row, head), the weights formed side by
// side, the four waves adding their splits' rows and the wave sums added in order.  Few: a wave per (row, head).
template <typename T, bool WIDE>
__global__ void __launch_bounds__(256) fwd_join_kernel(Params p) {
  __shared__ float lw[4][WIDE ? kMaxSplit : 64], lsum[WIDE ? 4 : 1][SSC_MAX_HEAD_DIM];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  constexpr int M = WIDE ? kMaxSplit / 64 : 1;
  const int64_t n = p.nq * p.hq, rh = WIDE ? int64_t(blockIdx.x) : int64_t(blockIdx.x) * 4 + wave;
  if (!WIDE && rh >= n) return;
  float mx = -INFINITY, ms[M], ls[M];
#pragma unroll
  for (int i = 0; i < M; ++i) {
    const int s = lane + 64 * i;
    ms[i] = s < p.nsplit ? p.part_b[2 * (s * n + rh)] : -INFINITY;
    ls[i] = s < p.nsplit ? p.part_b[2 * (s * n + rh) + 1] : 0.f;
    mx = fmaxf(mx, ms[i]);
  }
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) mx = fmaxf(mx, __shfl_xor(mx, d));
  float total = 0.f;
#pragma unroll
  for (int i = 0; i < M; ++i) {
    const float w = ms[i] == mx ? 1.f : __builtin_amdgcn_exp2f((ms[i] - mx) * exp_unit(p));
    total += w * ls[i];
    lw[wave][lane + 64 * i] = w;
  }
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) total += __shfl_xor(total, d);
  const bool some = total != 0.f;
  const float inv = some ? 1.f / total : 0.f;
  wave_fence();
  float acc[2] = {0.f, 0.f};
#pragma unroll 4
  for (int s = WIDE ? wave : 0; s < p.nsplit; s += WIDE ? 4 : 1) {
    const float w = lw[wave][s];
#pragma unroll
    for (int e = 0; e < 2; ++e)
      if (lane + 64 * e < p.d) acc[e] = fmaf(w, p.part_a[(s * n + rh) * p.d + lane + 64 * e], acc[e]);
  }
  T* op = static_cast<T*>(p.o) + rh * p.d;
  if constexpr (WIDE) {
#pragma unroll
    for (int e = 0; e < 2; ++e) lsum[wave][lane + 64 * e] = acc[e];
    __syncthreads();
    const int e = threadIdx.x;
    if (e < p.d) op[e] = T(((lsum[0][e] + lsum[1][e]) + (lsum[2][e] + lsum[3][e])) * inv);
  } else {
#pragma unroll
    for (int e = 0; e < 2; ++e)
      if (lane + 64 * e < p.d) op[lane + 64 * e] = T(acc[e] * inv);
  }
  if (lane == 0 && (!WIDE || wave == 0))
    p.lse[(rh % p.hq) * p.nq + rh / p.hq] = some ? lse_of<T>(p, mx, total) : -INFINITY;
}

// ---------------------------------------------------------------------------
// backward
// ---------------------------------------------------------------------------

// fp16: dS carries a power of two that keeps it inside the type's range.  It follows the largest |dout row|^2 and
// |v row|^2 of the sample and key head that dS belongs to, so that a sample's and a head's gradients do not depend on the
// values of others.  The maxima are formed by pieces: the rows of segment s within block g (`rows` of them) of one side
// are piece g + s, which numbers the pieces in row order with no table of where a segment's begin, and each piece is one
// workgroup's per key head.  Numbers that no row has (empty segments leave them) are never written nor read.
// Blocks of a side times key heads, at most.  Fewer leave the launch short of loads on their way (backward pass of 2 x 300k
// keys of 4 heads, 8 rows each: 992 us with 128, 810 with 256, 715 with 512, 687 with 1,024), more are more to read for
// every workgroup of a single key head (100k rows of 16 heads over 77 keys: 743 us with 512, 775 with 1,024, 851 with
// 2,048; with four loads on their way together 686 with 512).
constexpr int kPieceBlocks = 512;
inline int piece_rows(int64_t rows, int64_t heads_kv, int64_t rows_least) {
  const int64_t blocks = kPieceBlocks / heads_kv > 0 ? kPieceBlocks / heads_kv : 1, n = (rows + blocks - 1) / blocks;
  return int(n > rows_least ? n : rows_least);
}
inline int piece_count(int64_t rows, int piece, int64_t batch) { return int((rows + piece - 1) / piece + batch + 2); }

// The maxima of piece blockIdx.x (the query side's first, then the key side's) and key head blockIdx.y.  16 lanes a (row,
// head), four rows on their way at a time; infinite or NaN rows are left out and spoil the results they reach, masked
// ones are left out.  Rows of no sample have no maxima.
template <typename T>
__global__ void __launch_bounds__(256) top_kernel(Params p, float* top_q, float* top_k) {
  __shared__ float lmax[4];
  const int lane = threadIdx.x & 63, sub = threadIdx.x & 15, hk = blockIdx.y, chunks = p.d / 8;
  const bool isq = int(blockIdx.x) < p.q_pieces;
  const int piece = isq ? blockIdx.x : blockIdx.x - p.q_pieces, rows = isq ? p.q_piece : p.k_piece;
  const int32_t* off = isq ? p.qoff : p.koff;
  const int64_t n = isq ? p.nq : p.nk;
  // the piece's segment is the last one whose first piece is not past it: each lane looks at one of 64 candidates
  int seg = 0, end = p.batch + 2;
  while (end - seg > 1) {
    const int step = (end - seg + 63) / 64, s = seg + lane * step;
    const int first = s < end ? (s == 0 ? 0 : int(clamp_off(off, s - 1, n)) / rows + s) : 0x7FFFFFFF;
    const int k = __popcll(__ballot(first <= piece)) - 1;
    seg += (k < 0 ? 0 : k) * step;
    end = seg + step < end ? seg + step : end;
  }
  seg = uniform(seg);
  if (seg == 0 || seg > p.batch) return;
  const int64_t block = int64_t(piece - seg) * rows, begin = clamp_off(off, seg - 1, n), stop = clamp_off(off, seg, n);
  const int64_t lo = begin > block ? begin : block, hi = stop < block + rows ? stop : block + rows;
  if (lo >= hi) return;
  const int items = int(hi - lo) * (isq ? p.G : 1);
  float most = 0.f;
  // whole waves iterate together: the groups' sums cross lanes
  for (int base = 0; base < items; base += 4 * 16) {
    u32x4 x[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int i = base + u * 16 + int(threadIdx.x >> 4);
      x[u] = u32x4{0, 0, 0, 0};
      if (i < items && sub < chunks) {
        const int tok = isq ? int(div_g(uint32_t(i), p)) : i;
        const int64_t row = lo + tok;
        const T* a = isq ? static_cast<const T*>(p.dout) + (row * p.hq + hk * p.G + (i - tok * p.G)) * p.d
                         : static_cast<const T*>(p.v) + row * p.v_row + hk * p.v_head;
        if (isq || !p.mask || p.mask[row]) x[u] = *reinterpret_cast<const u32x4*>(a + sub * 8);
      }
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      float sq = 0.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) sq = Elt<T>::dot(x[u][e], x[u][e], sq);
#pragma unroll
      for (int d = 1; d < 16; d <<= 1) sq += __shfl_xor(sq, d);
      if (sq < INFINITY) most = fmaxf(most, sq);
    }
  }
#pragma unroll
  for (int d = 16; d < 64; d <<= 1) most = fmaxf(most, __shfl_xor(most, d));
  if (lane == 0) lmax[threadIdx.x >> 6] = most;
  __syncthreads();
  if (threadIdx.x == 0)
    (isq ? top_q + int64_t(hk) * p.q_pieces : top_k + int64_t(hk) * p.k_pieces)[piece] =
        fmaxf(fmaxf(lmax[0], lmax[1]), fmaxf(lmax[2], lmax[3]));
}
static_assert(SSC_MAX_HEAD_DIM <= 16 * 8, "a row is one vector a lane");

// the largest of the pieces of rows [begin, begin + len) of segment `index`
__device__ __forceinline__ float top_of(const float* top, int rows, int64_t begin, int len, int index) {
  const int last = int((begin + len - 1) / rows) + index;
  float m = 0.f;
  // four loads on their way together; past the last piece they repeat it
  for (int i = int(begin / rows) + index; i <= last; i += 256) {
    float x[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int at = i + 64 * u + int(threadIdx.x & 63);
      x[u] = top[at < last ? at : last];
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) m = fmaxf(m, x[u]);
  }
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) m = fmaxf(m, __shfl_xor(m, d));
  return m;
}

// Power of two for dS in fp16 of one sample and key head (q: the sample's query rows, k: its key rows): |dS| <=
// |dP - delta| <= 2 |dout row| |v row| (out lies within the values it averages), so with b2 = max |dout row|^2
// max |v row|^2 < 2^e the scaled dS stays below 2^(1 + e/2 + s) <= 2^15.5 < 65504 for s = 14 - floor(e / 2).  The rest of
// fp16's range (steps of 2^-24) is then all below the largest possible entry.
template <typename T>
__device__ __forceinline__ int ds_exp(const Params& p, int hk, int index, int64_t q_begin, int q_len, int64_t k_begin,
                                      int k_len) {
  if constexpr (kPExp<T> == 0) {
    return 0;
  } else {
    if (q_len <= 0 || k_len <= 0) return 0;  // nothing attends
    const float b2 = top_of(p.top_q + int64_t(hk) * p.q_pieces, p.q_piece, q_begin, q_len, index) *
                     top_of(p.top_k + int64_t(hk) * p.k_pieces, p.k_piece, k_begin, k_len, index);
    if (!(b2 > 0.f) || !(b2 < INFINITY)) return 0;
    int e;
    (void)frexpf(b2, &e);
    const int s = 14 - (e >> 1);
    return s < -30 ? -30 : (s > 60 ? 60 : s);
  }
}

// dP - delta times dS's power of two, which only fp16 has; `ndel` is -delta times it already
template <typename T>
__device__ __forceinline__ float less_delta(float dp, float ndel, float mul) {
  return kPExp<T> == 0 ? dp + ndel : fmaf(dp, mul, ndel);
}

// dq_i = scale sum_j dS_ij k_j, and the exact delta.  The forward result that delta = dout . out is formed from was
// rounded to 16 bits, and that error meets every key of the row with one sign: where attention is peaked it outweighs dS
// itself.  The sum of a row's dS is zero, so the sum e of the dS formed with the rounded delta is the error, and
// dq = scale (sum dS k - e sum P k).  With the sum of the values of dS as they are rounded for the product in e's place,
// their rounding goes out along the keys' mean as well (the error of dq against 64 bits fell from 2.1 to 1.4 times that
// of a result only rounded at the end, for about 5 % of this pass).  The second sum is one more product on operands that
// are at hand; the dK pass reads delta + e.  fp32 needs none of it.
//
// Forms, tiles and bounds as the forward pass: 2 x 11.2k rows, 16 heads of 64, bf16, 2.0 ms (four products at
// 1.0 PFLOP/s, MFMA busy 48 % of the cycles).  Heads of 72 to 96 stream 32-row tiles, whose smaller stage leaves
// registers for a second wave per SIMD (8 heads of 96: 2.0 -> 1.6 ms).
template <typename T, int DP, int NW, bool MASK, bool FEW, bool WIN>
__global__ void __launch_bounds__(NW * 64, FEW ? 2 : tile_cfg(sizeof(T), DP).dq_occ) dq_kernel(Params p) {
  constexpr int R = sizeof(T) == 4 || (!FEW && DP == 96) ? 32 : 64;
  using TL = TileOf<T, DP, R>;
  using E = Elt<T>;
  constexpr int NT = FEW ? 64 : NW * 64, TC = FEW ? 32 : NW * 32, BUFS = FEW ? NW : 2;
  constexpr bool kFix = sizeof(T) == 2;
  __shared__ __align__(16) char lds[2 * BUFS * TL::kBytes];
  __shared__ unsigned long long lvalid[BUFS];
  __shared__ float le[FEW ? (2 * NW + 1) * 32 : 1];  // the waves' sums of dS, of its rounded values, then delta
  const int64_t item = xcd_item(int64_t(p.tiles) * p.hk * p.nsplit);
  if (item >= int64_t(p.tiles) * p.hk * p.nsplit) return;
  const int tile = int(item % p.tiles), hk = int(item / p.tiles % p.hk), split = int(item / p.tiles / p.hk);
  Segment sg;
  if (!find_segment(p.qoff, p.nq, p.koff, p.nk, p.batch, p.G, TC, tile, &sg)) return;
  const int lane = threadIdx.x & 63, wave = uniform(int(threadIdx.x >> 6)), half = lane >> 5;
  const int dchunks = p.d / TL::kVec;
  const float c = p.scale * kLog2e;
  const int dse = ds_exp<T>(p, hk, sg.index, sg.begin, sg.len, sg.other, sg.other_len);
  const float dsmul = ldexpf(1.f, dse - kPExp<T>);  // probabilities carry 2^kPExp

  u32x4 qf[TL::kFrags], df[TL::kFrags];
  f32x16 acc[TL::kBlocks], mean[TL::kBlocks];
  const uint32_t r = uint32_t(sg.tile) * TC + (FEW ? 0 : wave * 32) + (lane & 31);
  const bool live = r < uint32_t(sg.len) * uint32_t(p.G);
  const uint32_t rc = live ? r : 0u, tok = div_g(rc, p);
  const int64_t row = sg.begin + tok;
  const int head = hk * p.G + int(rc - tok * uint32_t(p.G));
  load_cols<T, DP>(static_cast<const T*>(p.q) + row * p.q_row + head * p.q_head, live, dchunks, qf);
  load_cols<T, DP>(static_cast<const T*>(p.dout) + (row * p.hq + head) * p.d, live, dchunks, df);
  u32x4 of[TL::kFrags];
  load_cols<T, DP>(static_cast<const T*>(p.out) + (row * p.hq + head) * p.d, live, dchunks, of);
  float del = 0.f, esum = 0.f, rsum = 0.f;
#pragma unroll
  for (int f = 0; f < TL::kFrags; ++f)
#pragma unroll
    for (int e = 0; e < 4; ++e) del = E::dot(df[f][e], of[f][e], del);
  del += half_swap(del);
  const float ndel = -del * dsmul;
  const float lse = live ? p.lse[int64_t(head) * p.nq + row] : -INFINITY;
  const float sh = lse == -INFINITY ? -INFINITY : float(kPExp<T>) - lse * kLog2e;  // rows with no key: probabilities 0
#pragma unroll
  for (int d = 0; d < TL::kBlocks; ++d) {
    acc[d] = f32x16{};
    if constexpr (kFix) mean[d] = f32x16{};
  }

  int t0, t1;
  Seen seen;
  int place = 0, place0 = 0, place1 = 0;  // of this lane's column, of the wave's first and last ones
  if constexpr (WIN) {
    const int shift = sg.other_len - sg.len, lastr = int(uint32_t(sg.len) * uint32_t(p.G)) - 1;
    auto at = [&](int c) { return int(div_g(uint32_t(c < lastr ? c : lastr), p)) + shift; };
    const int c0 = sg.tile * TC, w0 = c0 + (FEW ? 0 : wave * 32);
    place = at(w0 + (lane & 31));
    place0 = at(w0);
    place1 = at(w0 + 31);
    seen.init(p, at(c0), at(c0 + TC - 1), sg.other_len, TL::kRows);
  }
  split_range(WIN ? seen.tiles : (sg.other_len + TL::kRows - 1) / TL::kRows, split, p.nsplit, &t0, &t1);
  constexpr int step = FEW ? NW : 1;
  if (FEW) t0 += wave;
  const uint32_t head_bytes = uint32_t(p.d) * uint32_t(sizeof(T));
  Walk<TL::kRows> wk, wv;
  wk.init(p.k_row * int64_t(sizeof(T)), head_bytes);
  wv.init(p.v_row * int64_t(sizeof(T)), head_bytes);
  const char* k0 = reinterpret_cast<const char*>(static_cast<const T*>(p.k) + sg.other * p.k_row + hk * p.k_head);
  const char* v0 = reinterpret_cast<const char*>(static_cast<const T*>(p.v) + sg.other * p.v_row + hk * p.v_head);
  wk.at = k0 + t0 * wk.step;
  wv.at = v0 + t0 * wv.step;
  Stage<T, DP, NT, R> sk, sv;
  sk.init(wk.row_bytes, dchunks);
  sv.init(wv.row_bytes, dchunks);
  uint8_t keep[Stage<T, DP, NT, R>::N];
  bool kept = false;
  auto load = [&](int t) {
    const int rows = WIN ? seen.rows(t, TL::kRows) : sg.other_len - t * TL::kRows;
    if constexpr (WIN) {
      wk.at = k0 + int64_t(seen.row(t, TL::kRows)) * wk.row_bytes;
      wv.at = v0 + int64_t(seen.row(t, TL::kRows)) * wv.row_bytes;
    }
    sk.load(wk.at, wk.span(rows));
    sv.load(wv.at, wv.span(rows));
    if constexpr (!WIN) {
      wk.at += step * wk.step;
      wv.at += step * wv.step;
    }
    if constexpr (MASK) {
      const uint8_t* mp = p.mask + sg.other + (WIN ? int64_t(seen.row(t, TL::kRows)) : int64_t(t) * TL::kRows);
#pragma unroll
      for (int i = 0; i < Stage<T, DP, NT, R>::N; ++i) {
        const int r = Stage<T, DP, NT, R>::item(i) / TL::CPR;
        keep[i] = (r < rows && r < TL::kRows) ? mp[r] : 0;
      }
      kept = lane < rows && lane < TL::kRows && mp[lane] != 0;
    }
  };
  if (t0 < t1) load(t0);
  for (int t = t0, n = 0; t < t1; t += step, ++n) {
    const int buf = FEW ? wave : n & 1;
    char* lk = lds + buf * 2 * TL::kBytes;
    char* lv = lk + TL::kBytes;
    constexpr uint64_t kAll = ~0ull >> (64 - TL::kRows);
    uint64_t valid = 0;
    if constexpr (MASK) {
      sk.clear(keep);
      sv.clear(keep);
      valid = __ballot(kept);
      if (!FEW && threadIdx.x == 0) lvalid[buf] = valid;
    }
    sk.store(lk);
    sv.store(lv);
    if constexpr (FEW)
      wave_fence();
    else
      __syncthreads();
    const int rows = WIN ? seen.rows(t, TL::kRows) : sg.other_len - t * TL::kRows;
    if constexpr (!MASK)
      valid = rows >= TL::kRows ? kAll : (1ull << rows) - 1;
    else if constexpr (!FEW)
      valid = lvalid[buf];
    if (t + step < t1) load(t + step);
    bool bounds = false;  // WIN: the columns see different rows
    if constexpr (WIN) {
      const int row0 = seen.row(t, TL::kRows);
      bounds = row0 < place1 - p.left || row0 + TL::kRows - 1 > place0 + p.right;
      if (bounds) valid &= sees(p, place, row0);
    }
#pragma unroll
    for (int kb = 0; kb < TL::kGroups; ++kb) {
      const uint32_t vw = uint32_t(valid >> (32 * kb));
      if (WIN ? !__any(vw != 0) : vw == 0) continue;
      f32x16 s{}, dp{};
#pragma unroll
      for (int f = 0; f < TL::kFrags; ++f) {
        if (TL::skip(f, dchunks)) break;
        const u32x4 a = TL::rows(lk, 32 * kb, f), v = TL::rows(lv, 32 * kb, f);
        s = E::mma(a, qf[f], s);
        dp = E::mma(v, df[f], dp);
      }
#pragma unroll
      for (int r = 0; r < 16; ++r) s[r] = __builtin_amdgcn_exp2f(fmaf(s[r], c, sh));
      if (WIN ? bounds || __any(~vw != 0) : ~vw != 0) {
        const uint32_t w = vw >> (4 * half);
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const bool on = (w >> (8 * (r / 4) + r % 4)) & 1u;
          s[r] = on ? s[r] : 0.f;
        }
      }
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        dp[r] = s[r] * less_delta<T>(dp[r], ndel, dsmul);
        if constexpr (kFix) esum += dp[r];
      }
#pragma unroll
      for (int st = 0; st < E::kSteps; ++st) {
        const u32x4 sf = E::pack(dp, st);
        u32x4 pf;
        if constexpr (kFix) {
          pf = E::pack(s, st);
#pragma unroll
          for (int j = 0; j < 4; ++j) rsum = E::sum(sf[j], rsum);
        }
#pragma unroll
        for (int d = 0; d < TL::kBlocks; ++d) {
          const u32x4 a = TL::cols(lk, 32 * kb, st, d);
          acc[d] = E::mma(a, sf, acc[d]);
          if constexpr (kFix) mean[d] = E::mma(a, pf, mean[d]);
        }
      }
    }
  }
  // dS carries 2^dse and P 2^kPExp: the sums in units of delta are esum 2^-dse and rsum 2^-dse
  const float f = ldexpf(p.scale, -dse), unit = ldexpf(1.f, -dse), punit = ldexpf(1.f, dse - kPExp<T>);
  if constexpr (FEW) {
    // the waves' sums, added in wave order; 2 NW threads share a column's elements
    float* all = reinterpret_cast<float*>(lds);
    float* mine = all + wave * DP * 33;
    const float e = kFix ? esum + half_swap(esum) : 0.f, re = kFix ? rsum + half_swap(rsum) : 0.f;
    if (half == 0) {
      le[wave * 32 + lane] = e;
      le[(NW + wave) * 32 + lane] = re;
      if (wave == 0) le[2 * NW * 32 + lane] = del;
    }
    constexpr int TPC = 2 * NW;
    const int col = threadIdx.x / TPC, e0 = threadIdx.x % TPC;
    const uint32_t r = uint32_t(sg.tile) * TC + col;
    const bool here = r < uint32_t(sg.len) * uint32_t(p.G);
    const uint32_t tok = div_g(r, p);
    const int64_t orow = sg.begin + tok;
    const int ohead = hk * p.G + int(r - tok * uint32_t(p.G));
    const int64_t rh = orow * p.hq + ohead, sp = int64_t(split) * p.nq * p.hq + rh;
    float sums[DP / TPC] = {};
    float es = 0.f, rs = 0.f;
#pragma unroll
    for (int pass = 0; pass < (kFix ? 2 : 1); ++pass) {
      __syncthreads();  // the tiles, or the first pass's sums, are read out
#pragma unroll
      for (int d = 0; d < TL::kBlocks; ++d)
#pragma unroll
        for (int i = 0; i < 16; ++i)
          mine[(32 * d + 8 * (i / 4) + 4 * half + i % 4) * 33 + (lane & 31)] = pass == 0 ? acc[d][i] : mean[d][i];
      __syncthreads();
      if (pass == 0) {
#pragma unroll
        for (int w = 0; w < NW; ++w) es += le[w * 32 + col], rs += le[(NW + w) * 32 + col];
        es *= unit;
        rs *= unit;
      }
#pragma unroll
      for (int i = 0; i < DP / TPC; ++i) {
        const int x = e0 + TPC * i;
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < NW; ++w) v += all[w * DP * 33 + x * 33 + col];
        if (p.nsplit > 1 && here && x < p.d && p.dq) {
          if (pass == 0)
            p.part_a[sp * p.d + x] = v * f;
          else
            p.part_b[sp * p.d + x] = v * ldexpf(p.scale, -kPExp<T>);
        }
        sums[i] = pass == 0 ? v : fmaf(-rs * punit, v, sums[i]);
      }
    }
    if (!here) return;
    if (e0 == 0 && p.nsplit > 1) {
      if constexpr (kFix) p.part_e[2 * sp] = es, p.part_e[2 * sp + 1] = rs;
    }
    if (p.nsplit == 1 && p.dq) {
#pragma unroll
      for (int i = 0; i < DP / TPC; ++i)
        if (e0 + TPC * i < p.d) static_cast<T*>(p.dq)[rh * p.d + e0 + TPC * i] = T(sums[i] * f);
    }
    if (e0 == 0 && split == 0) p.delta[int64_t(ohead) * p.nq + orow] = le[2 * NW * 32 + col] + (p.nsplit > 1 ? 0.f : es);
    return;
  }
  const float e = kFix ? esum + half_swap(esum) : 0.f, re = kFix ? rsum + half_swap(rsum) : 0.f;
  if (!live) return;
  const int64_t rh = row * p.hq + head, at = rh * p.d;
  if (p.nsplit > 1) {
    const int64_t sp = int64_t(split) * p.nq * p.hq;
    if (p.dq) {
      store_cols<T, DP>(nullptr, p.part_a + sp * p.d + at, acc, p.d, f);
      if constexpr (kFix) store_cols<T, DP>(nullptr, p.part_b + sp * p.d + at, mean, p.d, ldexpf(p.scale, -kPExp<T>));
    }
    if (half == 0) {
      if constexpr (kFix) p.part_e[2 * (sp + rh)] = e * unit, p.part_e[2 * (sp + rh) + 1] = re * unit;
      if (split == 0) p.delta[int64_t(head) * p.nq + row] = del;
    }
    return;
  }
  if (half == 0) p.delta[int64_t(head) * p.nq + row] = del + e * unit;
  if (!p.dq) return;
  if constexpr (kFix)
#pragma unroll
    for (int d = 0; d < TL::kBlocks; ++d)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[d][r] = fmaf(-(re * unit) * punit, mean[d][r], acc[d][r]);
  store_cols<T, DP>(static_cast<T*>(p.dq) + at, nullptr, acc, p.d, f);
}

// Joins the splits of dQ, in the two forms of the forward join.  e and re are the
// splits' sums of dS and of its rounded values (see dq_kernel).
template <typename T, bool WIDE>
__global__ void __launch_bounds__(256) dq_join_kernel(Params p) {
  __shared__ float la[WIDE ? 4 : 1][SSC_MAX_HEAD_DIM], lm[WIDE ? 4 : 1][SSC_MAX_HEAD_DIM];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t n = p.nq * p.hq, rh = WIDE ? int64_t(blockIdx.x) : int64_t(blockIdx.x) * 4 + wave;
  if (!WIDE && rh >= n) return;
  float e = 0.f, re = 0.f;
  if constexpr (sizeof(T) == 2) {
#pragma unroll
    for (int i = 0; i < kMaxSplit / 64; ++i)
      if (lane + 64 * i < p.nsplit) {
        e += p.part_e[2 * ((lane + 64 * i) * n + rh)];
        re += p.part_e[2 * ((lane + 64 * i) * n + rh) + 1];
      }
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) e += __shfl_xor(e, d), re += __shfl_xor(re, d);
    if (lane == 0 && (!WIDE || wave == 0)) p.delta[(rh % p.hq) * p.nq + rh / p.hq] += e;
  }
  if (!p.dq) return;
  float a[2] = {0.f, 0.f}, m[2] = {0.f, 0.f};
#pragma unroll 4
  for (int s = WIDE ? wave : 0; s < p.nsplit; s += WIDE ? 4 : 1)
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (lane + 64 * i < p.d) {
        a[i] += p.part_a[(s * n + rh) * p.d + lane + 64 * i];
        if constexpr (sizeof(T) == 2) m[i] += p.part_b[(s * n + rh) * p.d + lane + 64 * i];
      }
  T* op = static_cast<T*>(p.dq) + rh * p.d;
  if constexpr (WIDE) {
#pragma unroll
    for (int i = 0; i < 2; ++i) la[wave][lane + 64 * i] = a[i], lm[wave][lane + 64 * i] = m[i];
    __syncthreads();
    const int i = threadIdx.x;
    if (i < p.d) {
      const float as = (la[0][i] + la[1][i]) + (la[2][i] + la[3][i]), mm = (lm[0][i] + lm[1][i]) + (lm[2][i] + lm[3][i]);
      op[i] = T(fmaf(-re, mm, as));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (lane + 64 * i < p.d) op[lane + 64 * i] = T(fmaf(-re, m[i], a[i]));
  }
}

// dv_j = sum_i P_ij dout_i and dk_j = scale sum_i dS_ij q_i of 32 key columns a wave, over tiles of query rows (head after
// head of the group), double buffered in LDS.  Both of a tile's score blocks are formed before the first block's
// weights, so the matrix units have work while the vector units form those.  Bound as the forward pass, with 32 MFMA a
// tile: 2 x 11.2k rows, 16 heads of 64, bf16, 2.0 ms (four products at 1.0 PFLOP/s, MFMA busy 49 % of the cycles).  A
// software pipeline over 32-row blocks measured the same for heads of 64 and 10 to 60 % longer for 32 and for fp32.
// DK, DV: the gradients a launch forms.
//
// WIN: a key past the sinks is seen by the tokens of places j - right .. j + left, which its workgroup streams.  The
// sinks are seen by all later tokens: they are columns of a launch of their own (SINK), of single waves, whose long
// streams are split and whose sums are joined by sink_join_kernel.
template <typename T, int DP, int NW, bool MASK, bool DK, bool DV, bool WIN, bool SINK>
__global__ void __launch_bounds__(NW * 64, SINK ? 1 : tile_cfg(sizeof(T), DP).dkv_occ) dkv_kernel(Params p) {
  constexpr int R = sizeof(T) == 4 || DP > 64 ? 32 : 64;
  using TL = TileOf<T, DP, R>;
  using E = Elt<T>;
  constexpr int NT = NW * 64, TC = NW * 32, KS = E::kSteps, G = TL::kGroups;
  __shared__ __align__(16) char lds[2][2 * TL::kBytes];
  __shared__ __align__(16) float lsh[2][R], ldel[2][R];
  const int64_t item = xcd_item(int64_t(p.tiles) * p.hk * p.nsplit);
  if (item >= int64_t(p.tiles) * p.hk * p.nsplit) return;
  const int tile = int(item % p.tiles), hk = int(item / p.tiles % p.hk), split = int(item / p.tiles / p.hk);
  Segment sg;
  if (!find_segment(p.koff, p.nk, p.qoff, p.nq, p.batch, 1, TC, tile, &sg, SINK ? p.sinks : 0x7FFFFFFF)) return;
  const int lane = threadIdx.x & 63, wave = uniform(int(threadIdx.x >> 6)), half = lane >> 5;
  const int dchunks = p.d / TL::kVec;
  // WIN: a scale of zero clears the keys instead (an unseen score's -inf times 0 would be NaN)
  const float c = WIN && p.scale == 0.f ? 1.f : p.scale * kLog2e;
  const int dse = DK ? ds_exp<T>(p, hk, sg.index, sg.other, sg.other_len, sg.begin, sg.len) : 0;
  const float dsmul = ldexpf(1.f, dse - kPExp<T>);

  const int col = sg.tile * TC + wave * 32 + (lane & 31);
  const bool live = col < sg.len && (!WIN || (SINK ? col < p.sinks : col >= p.sinks || sg.index == 0 || sg.index > p.batch));
  const int64_t row = sg.begin + (live ? col : 0);
  const bool on = live && (!MASK || p.mask[row] != 0);
  u32x4 kf[TL::kFrags], vf[DK ? TL::kFrags : 1];
  load_cols<T, DP>(static_cast<const T*>(p.k) + row * p.k_row + hk * p.k_head, on && !(WIN && p.scale == 0.f), dchunks, kf);
  if constexpr (DK) load_cols<T, DP>(static_cast<const T*>(p.v) + row * p.v_row + hk * p.v_head, on, dchunks, vf);
  f32x16 dk[DK ? TL::kBlocks : 1], dv[DV ? TL::kBlocks : 1];
  auto clear = [&]() {
#pragma unroll
    for (int d = 0; d < TL::kBlocks; ++d) {
      if constexpr (DK) dk[d] = f32x16{};
      if constexpr (DV) dv[d] = f32x16{};
    }
  };
  clear();
  // waves whose columns all lie past the sample's keys only help to stage
  const bool busy = WIN ? __any(live) : sg.tile * TC + wave * 32 < sg.len;
  // WIN: only the tokens that see one of the workgroup's columns; tokens [see0, see1) see this lane's
  int see0 = 0, see1 = 0, full0 = 0, full1 = 0;
  if constexpr (WIN) {
    const int shift = sg.len - sg.other_len, tokens = sg.other_len;
    const int j0 = SINK || sg.tile * TC > p.sinks ? sg.tile * TC : p.sinks;
    const int j1 = (sg.tile + 1) * TC < sg.len ? (sg.tile + 1) * TC : sg.len;
    int lo = j0 - p.right - shift, hi = SINK ? tokens : j1 - 1 + p.left - shift + 1;
    lo = lo < 0 ? 0 : lo;
    hi = hi < tokens ? hi : tokens;
    const int w0 = sg.tile * TC + wave * 32;
    see0 = col - p.right - shift - lo;
    see1 = SINK ? 0x3FFFFFFF : col + p.left - shift + 1 - lo;
    full0 = w0 + 31 - p.right - shift - lo;  // rows [full0, full1) of the stream are seen by all of the wave's columns
    full1 = SINK ? 0x3FFFFFFF : w0 + p.left - shift + 1 - lo;
    sg.other += lo;
    sg.other_len = j0 < j1 && hi > lo ? hi - lo : 0;
  }

  // the sample's queries, head after head of the group: tile n is head n / tiles, its tile n mod tiles
  const int tiles = (sg.other_len + R - 1) / R;
  int n0, n1;
  split_range(tiles * p.G, split, p.nsplit, &n0, &n1);
  const uint32_t head_bytes = uint32_t(p.d) * uint32_t(sizeof(T));
  Walk<R> wq, wd;
  wq.init(p.q_row * int64_t(sizeof(T)), head_bytes);
  wd.init(int64_t(p.hq) * head_bytes, head_bytes);
  Stage<T, DP, NT, R> sq, sd;
  sq.init(wq.row_bytes, dchunks);
  sd.init(wd.row_bytes, dchunks);
  const float *lse_at = nullptr, *del_at = nullptr;
  int g = n0 < n1 ? n0 / tiles : 0, left = n0 < n1 ? sg.other_len - (n0 - g * tiles) * R : 0;  // rows of head g to load
  auto seek = [&]() {
    const int64_t r0 = sg.other + (sg.other_len - left), head = hk * p.G + g;
    wq.at = reinterpret_cast<const char*>(static_cast<const T*>(p.q) + r0 * p.q_row + head * p.q_head);
    wd.at = reinterpret_cast<const char*>(static_cast<const T*>(p.dout) + (r0 * p.hq + head) * p.d);
    lse_at = p.lse + head * p.nq + r0;
    del_at = p.delta + head * p.nq + r0;
  };
  float rlse = 0.f, rdel = 0.f;
  int rows = 0;  // of the tile on its way
  const uint32_t lane_off = wave == 0 && lane < R ? lane * 4 : 0xFFFFFFF0u;
  auto load = [&]() {
    sq.load(wq.at, wq.span(left));
    sd.load(wd.at, wd.span(left));
    const uint32_t bytes = uint32_t(left < R ? left : R) * 4;
    rlse = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(buffer_of(lse_at, bytes), int(lane_off), 0, 0));
    // dV alone needs no delta
    if constexpr (DK) rdel = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(buffer_of(del_at, bytes), int(lane_off), 0, 0));
    rows = left;
    left -= R;
    wq.at += wq.step;
    wd.at += wd.step;
    lse_at += R;
    del_at += R;
    if (left <= 0) {
      left = sg.other_len;
      ++g;
      seek();
    }
  };
  auto store = [&](int buf) {
    sq.store(lds[buf]);
    sd.store(lds[buf] + TL::kBytes);
    if (wave == 0 && lane < R) {
      // rows past the sample and rows with no key: weights 0
      lsh[buf][lane] = lane >= rows || rlse == -INFINITY ? -INFINITY : float(kPExp<T>) - rlse * kLog2e;
      ldel[buf][lane] = -rdel * dsmul;
    }
  };
  const int n = n1 - n0;
  int done = WIN && n > 0 ? (n0 - g * tiles) * R : 0;  // first row of the tile at hand
  if (n > 0) {
    seek();
    load();
  }
  for (int i = 0; i < n; ++i) {
    const int buf = i & 1;
    store(buf);
    __syncthreads();
    if (i + 1 < n) load();
    if (!busy) continue;  // for the whole pass
    const char* tq = lds[buf];
    const char* td = tq + TL::kBytes;
    uint64_t vis = ~0ull;
    bool part = false;  // WIN: some column does not see some of the tile's rows
    if constexpr (WIN) {
      const int r0 = done;
      done = done + R < sg.other_len ? done + R : 0;  // the next head's rows begin anew
      part = r0 < full0 || r0 + R > full1;
      if (part) {
        vis = below(see1 - r0) & ~below(see0 - r0);
        if (!__any(vis != 0)) continue;
      }
    }
    f32x16 s[G], dp[G];
#pragma unroll
    for (int b = 0; b < G; ++b) {
      s[b] = dp[b] = f32x16{};
#pragma unroll
      for (int f = 0; f < TL::kFrags; ++f) {
        if (TL::skip(f, dchunks)) break;
        s[b] = E::mma(TL::rows(tq, 32 * b, f), kf[f], s[b]);
        if constexpr (DK) dp[b] = E::mma(TL::rows(td, 32 * b, f), vf[f], dp[b]);
      }
    }
    if constexpr (WIN)
      if (part) {
        // what is not seen gets no weight (c times this is -inf) and no dP, whatever an unseen key's rows hold
        const float never = c < 0.f ? INFINITY : -INFINITY;
#pragma unroll
        for (int b = 0; b < G; ++b) {
          const uint32_t w = uint32_t(vis >> (32 * b)) >> (4 * half);
#pragma unroll
          for (int r = 0; r < 16; ++r) {
            const bool on = (w >> (8 * (r / 4) + r % 4)) & 1u;
            s[b][r] = on ? s[b][r] : never;
            if constexpr (DK) dp[b][r] = on ? dp[b][r] : 0.f;
          }
        }
      }
#pragma unroll
    for (int b = 0; b < G; ++b) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4 sh4 = *reinterpret_cast<const float4*>(&lsh[buf][32 * b + 8 * i + 4 * half]);
        float4 de4{};
        if constexpr (DK) de4 = *reinterpret_cast<const float4*>(&ldel[buf][32 * b + 8 * i + 4 * half]);
        const float sh[4] = {sh4.x, sh4.y, sh4.z, sh4.w}, de[4] = {de4.x, de4.y, de4.z, de4.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float pr = __builtin_amdgcn_exp2f(fmaf(s[b][4 * i + j], c, sh[j]));
          s[b][4 * i + j] = pr;
          if constexpr (DK) dp[b][4 * i + j] = pr * less_delta<T>(dp[b][4 * i + j], de[j], dsmul);
        }
      }
#pragma unroll
      for (int st = 0; st < KS; ++st) {
        u32x4 pf, sf;
        if constexpr (DV) pf = E::pack(s[b], st);
        if constexpr (DK) sf = E::pack(dp[b], st);
#pragma unroll
        for (int d = 0; d < TL::kBlocks; ++d) {
          if constexpr (DV) dv[d] = E::mma(TL::cols(td, 32 * b, st, d), pf, dv[d]);
          if constexpr (DK) dk[d] = E::mma(TL::cols(tq, 32 * b, st, d), sf, dk[d]);
        }
      }
    }
  }

  if (!live) return;
  // a masked key has no gradient, whatever its zeroed column collected
  if (!on) clear();
  const int64_t o = (row * p.hk + hk) * p.d;
  // a sink's partial sums are numbered by its tile's columns
  const int64_t sp = SINK ? (((int64_t(split) * p.tiles + tile) * TC + (lane & 31)) * p.hk + hk) * p.d
                          : int64_t(split) * p.nk * p.hk * p.d + o;
  if constexpr (DK)
    store_cols<T, DP>(static_cast<T*>(p.dk) + o, p.nsplit > 1 ? p.part_a + sp : nullptr, dk, p.d, ldexpf(p.scale, -dse));
  if constexpr (DV)
    store_cols<T, DP>(static_cast<T*>(p.dv) + o, p.nsplit > 1 ? p.part_b + sp : nullptr, dv, p.d, ldexpf(1.f, -kPExp<T>));
}

// dK (blockIdx.y 0) and dV (1): the splits' partial sums added in split order; four elements a thread
template <typename T>
__global__ void __launch_bounds__(64) sum_splits_kernel(const float* part_k, const float* part_v, int64_t n4, int nsplit,
                                                        T* dk, T* dv) {
  const int64_t i = int64_t(blockIdx.x) * 64 + threadIdx.x;
  T* dst = blockIdx.y ? dv : dk;
  if (i >= n4 || !dst) return;
  const float4* src = reinterpret_cast<const float4*>(blockIdx.y ? part_v : part_k);
  float4 a = src[i];
#pragma unroll 8
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

constexpr int kSinkCols = 32;  // keys of a sink launch's tile: one wave's columns

// The sinks' dK (blockIdx.y 0) and dV (1): a workgroup adds a sink tile's partial sums of one key head in split order
template <typename T>
__global__ void __launch_bounds__(256) sink_join_kernel(Params p, const float* part_k, const float* part_v) {
  const int tile = blockIdx.x % p.tiles, hk = blockIdx.x / p.tiles;
  T* dst = static_cast<T*>(blockIdx.y ? p.dv : p.dk);
  const float* src = blockIdx.y ? part_v : part_k;
  Segment sg;
  if (!dst || !find_segment(p.koff, p.nk, p.qoff, p.nq, p.batch, 1, kSinkCols, tile, &sg, p.sinks)) return;
  const int end = sg.len < p.sinks ? sg.len : p.sinks, cols = end - sg.tile * kSinkCols;
  for (int i = threadIdx.x; i < kSinkCols * p.d; i += 256) {
    const int col = i / p.d, e = i - col * p.d;
    if (col >= cols) break;
    float v = 0.f;
#pragma unroll 8
    for (int s = 0; s < p.nsplit; ++s)
      v += src[(((int64_t(s) * p.tiles + tile) * kSinkCols + col) * p.hk + hk) * p.d + e];
    dst[((sg.begin + sg.tile * kSinkCols + col) * p.hk + hk) * p.d + e] = T(v);
  }
}

// what the host decides before a launch
struct FwdPlan {
  bool few;  // a sample's rows fit one tile of 32 columns (see fwd_kernel)
  int tiles, nsplit;
};
struct BwdPlan {
  bool q_few;
  int q_tiles, q_split;  // dQ
  int k_tiles, k_split;  // dK and dV
  int s_tiles, s_split;  // dK and dV of windowed attention's sinks
};

// the backward pass's regions of the workspace
struct BwdParts {
  float *q_sum, *q_mean, *q_err, *k_sum, *v_sum, *sink_k, *sink_v;
  float *top_q, *top_k;
};

// launches of one element type (defined once per type)
template <typename T>
int launch_fwd(const Params& p, const FwdPlan& f, hipStream_t s);
template <typename T>
int launch_bwd(Params p, const BwdPlan& b, const BwdParts& w, hipStream_t s);
// of windowed attention
template <typename T>
int launch_win_fwd(const Params& p, const FwdPlan& f, hipStream_t s);
template <typename T>
int launch_win_bwd(Params p, const BwdPlan& b, const BwdParts& w, hipStream_t s);

// ---------------------------------------------------------------------------
// launches
// ---------------------------------------------------------------------------

template <typename T, int DP, bool FEW, bool WIN>
void launch_fwd_tile(const Params& p, hipStream_t s) {
  constexpr int NW = FEW ? 4 : fwd_waves(sizeof(T), DP);
  const unsigned grid = xcd_grid(int64_t(p.tiles) * p.hk * p.nsplit);
  if (p.mask)
    fwd_kernel<T, DP, NW, true, FEW, WIN><<<grid, NW * 64, 0, s>>>(p);
  else
    fwd_kernel<T, DP, NW, false, FEW, WIN><<<grid, NW * 64, 0, s>>>(p);
}

template <typename T, int DP, bool WIN>
void launch_fwd_dim(const Params& p, const FwdPlan& f, hipStream_t s) {
  if (f.few)
    launch_fwd_tile<T, DP, true, WIN>(p, s);
  else
    launch_fwd_tile<T, DP, false, WIN>(p, s);
}

template <typename T, int DP, bool FEW, bool WIN>
void launch_dq_tile(const Params& p, hipStream_t s) {
  const unsigned grid = xcd_grid(int64_t(p.tiles) * p.hk * p.nsplit);
  if (p.mask)
    dq_kernel<T, DP, 4, true, FEW, WIN><<<grid, 256, 0, s>>>(p);
  else
    dq_kernel<T, DP, 4, false, FEW, WIN><<<grid, 256, 0, s>>>(p);
}

template <typename T, int DP, bool WIN>
void launch_dq_dim(const Params& p, const BwdPlan& b, hipStream_t s) {
  if (b.q_few)
    launch_dq_tile<T, DP, true, WIN>(p, s);
  else
    launch_dq_tile<T, DP, false, WIN>(p, s);
}

template <typename T, int DP, bool DK, bool DV, bool WIN, bool SINK>
void launch_dkv_tile(const Params& p, hipStream_t s) {
  constexpr int NW = SINK ? kSinkCols / 32 : 4;
  const unsigned grid = xcd_grid(int64_t(p.tiles) * p.hk * p.nsplit);
  if (p.mask)
    dkv_kernel<T, DP, NW, true, DK, DV, WIN, SINK><<<grid, NW * 64, 0, s>>>(p);
  else
    dkv_kernel<T, DP, NW, false, DK, DV, WIN, SINK><<<grid, NW * 64, 0, s>>>(p);
}

// The sums of both gradients of a 16-bit head of over 96 leave registers for one wave per SIMD only; a pass for each,
// which forms the scores again, runs with two (dK and dV of 2 x 11.2k rows, 8 heads of 128: 3.3 -> 2.8 ms).
template <typename T, int DP, bool WIN, bool SINK>
void launch_dkv_dim(const Params& p, hipStream_t s) {
  if constexpr (sizeof(T) == 4 || DP <= 96) {
    if (p.dk && p.dv) {
      launch_dkv_tile<T, DP, true, true, WIN, SINK>(p, s);
      return;
    }
  }
  if (p.dk) launch_dkv_tile<T, DP, true, false, WIN, SINK>(p, s);
  if (p.dv) launch_dkv_tile<T, DP, false, true, WIN, SINK>(p, s);
}

template <typename T>
void launch_fwd_join(const Params& p, hipStream_t s) {
  if (p.nsplit > kFewSplits)
    fwd_join_kernel<T, true><<<unsigned(p.nq * p.hq), 256, 0, s>>>(p);
  else
    fwd_join_kernel<T, false><<<unsigned((p.nq * p.hq + 3) / 4), 256, 0, s>>>(p);
}

template <typename T>
void launch_dq_join(const Params& p, hipStream_t s) {
  if (p.nsplit > kFewSplits)
    dq_join_kernel<T, true><<<unsigned(p.nq * p.hq), 256, 0, s>>>(p);
  else
    dq_join_kernel<T, false><<<unsigned((p.nq * p.hq + 3) / 4), 256, 0, s>>>(p);
}

template <typename T, bool WIN = false>
int launch_fwd_impl(const Params& p, const FwdPlan& f, hipStream_t s) {
  if (p.d <= 32)
    launch_fwd_dim<T, 32, WIN>(p, f, s);
  else if (p.d <= 64)
    launch_fwd_dim<T, 64, WIN>(p, f, s);
  else if (p.d <= 96)
    launch_fwd_dim<T, 96, WIN>(p, f, s);
  else
    launch_fwd_dim<T, 128, WIN>(p, f, s);
  if (p.nsplit > 1) launch_fwd_join<T>(p, s);
  return hipGetLastError() == hipSuccess ? SSC_OK : SSC_ERR_HIP;
}

template <typename T, bool WIN = false>
int launch_bwd_impl(Params p, const BwdPlan& b, const BwdParts& w, hipStream_t s) {
  if constexpr (kPExp<T> != 0) {
    p.top_q = w.top_q;
    p.top_k = w.top_k;
    if ((p.dq || p.dk) && p.nq > 0 && p.nk > 0)
      top_kernel<T><<<dim3(unsigned(p.q_pieces + p.k_pieces), unsigned(p.hk)), 256, 0, s>>>(p, w.top_q, w.top_k);
  }
  // dK reads the delta that the dQ pass forms, so that pass runs for either
  if ((p.dq || p.dk) && p.nq > 0) {
    p.tiles = b.q_tiles;
    p.nsplit = b.q_split;
    p.part_a = w.q_sum;
    p.part_b = w.q_mean;
    p.part_e = w.q_err;
    if (p.d <= 32)
      launch_dq_dim<T, 32, WIN>(p, b, s);
    else if (p.d <= 64)
      launch_dq_dim<T, 64, WIN>(p, b, s);
    else if (p.d <= 96)
      launch_dq_dim<T, 96, WIN>(p, b, s);
    else
      launch_dq_dim<T, 128, WIN>(p, b, s);
    if (p.nsplit > 1) launch_dq_join<T>(p, s);
  }
  if ((p.dk || p.dv) && p.nk > 0) {
    p.tiles = b.k_tiles;
    p.nsplit = b.k_split;
    p.part_a = w.k_sum;
    p.part_b = w.v_sum;
    if (p.d <= 32)
      launch_dkv_dim<T, 32, WIN, false>(p, s);
    else if (p.d <= 64)
      launch_dkv_dim<T, 64, WIN, false>(p, s);
    else if (p.d <= 96)
      launch_dkv_dim<T, 96, WIN, false>(p, s);
    else
      launch_dkv_dim<T, 128, WIN, false>(p, s);
    if (p.nsplit > 1) {
      const int64_t n4 = p.nk * p.hk * p.d / 4;
      sum_splits_kernel<T><<<dim3(unsigned((n4 + 63) / 64), 2), 64, 0, s>>>(w.k_sum, w.v_sum, n4, p.nsplit,
                                                                            static_cast<T*>(p.dk), static_cast<T*>(p.dv));
    }
    if constexpr (WIN) {
      if (p.sinks > 0) {
        p.tiles = b.s_tiles;
        p.nsplit = b.s_split;
        p.part_a = w.sink_k;
        p.part_b = w.sink_v;
        if (p.d <= 32)
          launch_dkv_dim<T, 32, WIN, true>(p, s);
        else if (p.d <= 64)
          launch_dkv_dim<T, 64, WIN, true>(p, s);
        else if (p.d <= 96)
          launch_dkv_dim<T, 96, WIN, true>(p, s);
        else
          launch_dkv_dim<T, 128, WIN, true>(p, s);
        if (p.nsplit > 1)
          sink_join_kernel<T><<<dim3(unsigned(p.tiles * p.hk), 2), 256, 0, s>>>(p, w.sink_k, w.sink_v);
      }
    }
  }
  return hipGetLastError() == hipSuccess ? SSC_OK : SSC_ERR_HIP;
}

}  // namespace attn
}  // namespace ssc
