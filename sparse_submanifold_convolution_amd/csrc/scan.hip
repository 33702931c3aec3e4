// Gated linear recurrence along the rows of ragged samples, and its backward pass.
//
// Per channel, along a sample's rows (from its last row where reversed), with a_t = sigmoid(gate_t):
//   h_t = a_t h_{t-1} + b_t,   b_t = (1 - a_t) x_t  (mix)  or  x_t  (sum),   h before the first row: the sample's h0.
// Backward, with D_t the gradient of h_t and c_t what row t hands to the row before it:
//   D_t = dy_t + c_{t+1},  c_t = a_t D_t,  c past the last row: the gradient of the final state;
//   dx_t = (1 - a_t) D_t  or  D_t,   dgate_t = a_t (1 - a_t) D_t (h_{t-1} - x_t)  or  a_t (1 - a_t) D_t h_{t-1},
//   dh0 = c of the first row.
//
// Both directions compose maps v -> A v + B, which is associative.  A thread walks L rows of four channels, CL lanes beside
// it the neighbouring channels, and the 256 / CL threads along the rows are joined by shuffles and LDS: a tile of
// 256 L / CL rows by 4 CL channels, read once.  Tiles are joined as they run: each publishes its map and takes what
// others have published (see look_back).  Which words a tile takes is fixed, so sums have one order and results repeat.
// Tiles take their numbers from a counter in the order they start: a tile only waits for tiles that run already and that
// never wait for it.  A published word is its own flag: it was cleared to all ones, a NaN that no result is given, and is
// written once, so no order between words matters.
//
// Bound by memory where rows are wide: 629k rows x 1,024 channels, bf16, forward 0.76 ms (5.1 TB/s), backward 1.39 ms
// (4.6 TB/s); narrow ones by the exchange between tiles (800k rows x 64 channels: 0.11 and 0.18 ms, 2.8 TB/s).  In three
// launches, with the inputs read twice and the tiles joined in between, the forward pass would move 5 tensors, not 3.
//
// A sample's first row drops whatever came before it (A = -0, which no product of decays is), so samples never touch each
// other, not even through an infinity or a NaN.  States, products and sums are fp32.  The backward pass forms h again from the inputs and
// the values at the tiles' borders, which the forward pass hands out: y is not read and its rounding does not matter.

#include <hip/hip_runtime.h>

#include "ssc_internal.h"
#include "vec.h"

namespace ssc {

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kFour = 4;  // channels of a thread
// Tiles of a bunch, and bunches that a tile looks back over: what is known moves on by 56 tiles with each exchange between
// tiles, of about 2 us, and a tile takes 3.5 + 8 words on average.  A plain row of 16 tiles (16 words) left narrow rows
// waiting (800k rows x 64 channels, bf16: forward 196 us, now 108; x 256: 301 and 299), three bunches did as well (142 us),
// and bunches of 16 take more words and registers than they save (x 256 backward: 524 -> 798 us).
constexpr int kBunch = 8, kBunches = 7;
// Rows of a thread.  Forward, 16 bits: 16 keep 128 registers of decays and inputs, at three waves per SIMD; 8 leave room for
// four, but tiles half as long (800k rows x 256 channels: 341 us, with 16 rows 299).  The backward pass keeps three values
// an element and fp32 twice the raw rows.  With few tiles shorter ones spread the work.
constexpr int kBackRows = 8;
constexpr int fwd_rows(int esize, bool few) { return esize == 2 && !few ? 16 : 8; }

struct ScanParams {
  const void *x, *gate, *dy;
  void *y, *dx, *dgate;
  const int32_t* off;
  const float *h0, *dlast;
  float *last, *dh0;
  float* carries;        // h before the first row of each tile of the backward pass
  uint32_t* ticket;
  // words between tiles, by the order of work, A in the low half: the tiles' maps [tiles][C], the maps of bunches of tiles
  // and the values that reach them [bunches][C]
  uint64_t *maps, *bunches, *values;
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

// a = sigmoid(g) and 1 - a.  The smaller of the two is q = e / (1 + e), e = exp(-|g|), and the other 1 - q: both keep
// their relative error however near to 0 or 1 they are.
template <typename T>
__device__ __forceinline__ void sides(float g, float& a, float& keep) {
  float q;
  if constexpr (sizeof(T) == 4) {
    const float e = expf(-fabsf(g));
    q = e / (1.f + e);
  } else {
    // the hardware's exponential and reciprocal, off by 2^-22 or so: a 16-bit gate is itself known to 2^-11 at best
    const float e = __builtin_amdgcn_exp2f(-fabsf(g) * kLog2e);
    q = e * __builtin_amdgcn_rcpf(1.f + e);
  }
  const float big = 1.f - q;
  a = g < 0.f ? q : big;
  keep = g < 0.f ? big : q;
}

// Ends the compiler's knowledge of a register's value, at no instruction: what is unpacked from it is then unpacked again
// in the next walk over the rows, instead of being held from one to the next in twice the registers.
__device__ __forceinline__ void afresh(uint2& r) { asm("" : "+v"(r.x), "+v"(r.y)); }
__device__ __forceinline__ void afresh(float4&) {}

// Where a thread's rows of a [n][C] tensor lie: a base that the workgroup shares, which steps from row to row in scalar
// registers, and the thread's offset from it, which 32 bits hold (row strides are bounded for it).
struct Lane {
  const char* base;
  int64_t step;
  uint32_t off;
  // first: the tile's first place; place: the thread's first place in it; rows: the tile's; col: the thread's first channel
  __device__ __forceinline__ void init(const void* ptr, int64_t row_bytes, const ScanParams& p, int64_t first, int place, int rows,
                                       int col_bytes) {
    // reversed, places walk down from the tile's end; its lowest row may lie before row 0, where no place of it is taken
    const int64_t low = p.rev ? p.n - first - rows : first;
    base = static_cast<const char*>(ptr) + low * row_bytes;
    step = p.rev ? -row_bytes : row_bytes;
    off = uint32_t(p.rev ? rows - 1 - place : place) * uint32_t(row_bytes) + uint32_t(col_bytes);
  }
  template <typename R>
  __device__ __forceinline__ R get(int i) const {
    return *reinterpret_cast<const R*>(base + i * step + off);
  }
  template <typename R>
  __device__ __forceinline__ void put(int i, const R& v) const {
    *reinterpret_cast<R*>(const_cast<char*>(base) + i * step + off) = v;
  }
};

// a value every lane holds alike, in a scalar register
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// The map (A, B) of a value, and its factor after an earlier map's.  A = -0 drops what came before, a NaN among it too; a
// product of decays that underflows is +0 and still hands on a NaN.
constexpr float kDrop = -0.f;
__device__ __forceinline__ bool drops(float A) { return __float_as_uint(A) == 0x80000000u; }
__device__ __forceinline__ float after(float A, float B, float v) { return drops(A) ? B : fmaf(A, v, B); }
__device__ __forceinline__ float times(float A, float a) { return drops(A) ? A : A * a; }

// four elements of a row
template <typename T>
struct Four {
  typedef uint2 raw;
  __device__ static __forceinline__ raw none() { return make_uint2(0, 0); }
  __device__ static __forceinline__ void unpack(const raw& r, float (&f)[4]) {
    const uint32_t w[2] = {r.x, r.y};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if constexpr (__is_same(T, __bf16)) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
      } else {
        f[2 * i] = float(__builtin_bit_cast(_Float16, uint16_t(w[i] & 0xffffu)));
        f[2 * i + 1] = float(__builtin_bit_cast(_Float16, uint16_t(w[i] >> 16)));
      }
    }
  }
  __device__ static __forceinline__ raw pack(const float (&f)[4]) {
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const f32x2 p{f[2 * i], f[2 * i + 1]};
      if constexpr (__is_same(T, __bf16))
        w[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(p, bf16x2));
      else
        w[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(p, f16x2));
    }
    return make_uint2(w[0], w[1]);
  }
};
template <>
struct Four<float> {
  typedef float4 raw;
  __device__ static __forceinline__ raw none() { return make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ static __forceinline__ void unpack(const raw& r, float (&f)[4]) {
    f[0] = r.x;
    f[1] = r.y;
    f[2] = r.z;
    f[3] = r.w;
  }
  __device__ static __forceinline__ raw pack(const float (&f)[4]) { return make_float4(f[0], f[1], f[2], f[3]); }
};

__device__ __forceinline__ void load_state(const float* src, float (&f)[4]) {
  Four<float>::unpack(*reinterpret_cast<const float4*>(src), f);
}
__device__ __forceinline__ void store_state(float* dst, const float (&f)[4]) {
  *reinterpret_cast<float4*>(dst) = make_float4(f[0], f[1], f[2], f[3]);
}

// The threads' maps of a tile: 256 / CL threads along the rows, 4 CL channels
template <int CL>
struct Tile {
  static constexpr int kCh = 4 * CL;
  // Joins the threads' maps along the rows (BACK: against them): on return (A, B) is the map of the wave's threads before
  // this one, and tot holds each wave's.
  template <bool BACK>
  __device__ static __forceinline__ void join(float (&A)[4], float (&B)[4], float (*tot)[2][kCh]) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, col = threadIdx.x % CL;
#pragma unroll
    for (int d = CL; d < 64; d <<= 1)
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const float a = BACK ? __shfl_down(A[v], d) : __shfl_up(A[v], d);
        const float b = BACK ? __shfl_down(B[v], d) : __shfl_up(B[v], d);
        if (BACK ? lane + d < 64 : lane >= d) {
          B[v] = after(A[v], B[v], b);
          A[v] = times(A[v], a);
        }
      }
    if (BACK ? lane < CL : lane >= 64 - CL) {
      store_state(&tot[wave][0][col * 4], A);
      store_state(&tot[wave][1][col * 4], B);
    }
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const float a = BACK ? __shfl_down(A[v], CL) : __shfl_up(A[v], CL);
      const float b = BACK ? __shfl_down(B[v], CL) : __shfl_up(B[v], CL);
      const bool some = BACK ? lane + CL < 64 : lane >= CL;
      A[v] = some ? a : 1.f;
      B[v] = some ? b : 0.f;
    }
  }
  // the value that reaches this thread's rows, from what reaches the tile
  template <bool BACK>
  __device__ static __forceinline__ void enter(float (&v)[4], const float (&A)[4], const float (&B)[4],
                                               const float (*tot)[2][kCh]) {
    const int wave = threadIdx.x >> 6, col = threadIdx.x % CL;
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      const int w = BACK ? 3 - i : i;
      if (BACK ? w > wave : w < wave) {
        float a[4], b[4];
        load_state(&tot[w][0][col * 4], a);
        load_state(&tot[w][1][col * 4], b);
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = after(a[k], b[k], v[k]);
      }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = after(A[k], B[k], v[k]);
  }
  // one channel's map of the whole tile
  template <bool BACK>
  __device__ static __forceinline__ void whole(const float (*tot)[2][kCh], int ch, float* A, float* B) {
    *A = 1.f;
    *B = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int w = BACK ? 3 - i : i;
      const float a = tot[w][0][ch], b = tot[w][1][ch];
      *B = after(a, b, *B);
      *A = times(a, *A);
    }
  }
};

// Words on their way between tiles
constexpr uint32_t kNotYet = 0xFFFFFFFFu;
__device__ __forceinline__ uint32_t word_of(float f) {
  const uint32_t u = __float_as_uint(f);
  return u == kNotYet ? 0x7FC00000u : u;
}

// Waits for n of K words `step` apart, of which the first lies at `head` and the k-th at at + k step, and composes their
// maps in order.
template <int K>
__device__ __forceinline__ void take_words(const uint64_t* head, const uint64_t* at, int64_t step, int n, float& A, float& B) {
  uint64_t w[K];
  bool done;
  do {
    done = true;
#pragma unroll
    for (int k = 0; k < K; ++k)
      if (k < n) w[k] = __hip_atomic_load(k == 0 ? head : at + k * step, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
#pragma unroll
    for (int k = 0; k < K; ++k)
      if (k < n) done &= uint32_t(w[k]) != kNotYet;
    if (!done) __builtin_amdgcn_s_sleep(1);
  } while (!done);
  A = 1.f;
  B = 0.f;
#pragma unroll
  for (int k = 0; k < K; ++k)
    if (k < n) {
      const float a = __uint_as_float(uint32_t(w[k])), b = __uint_as_float(uint32_t(w[k] >> 32));
      B = after(a, b, B);
      A = times(a, A);
    }
}
__device__ __forceinline__ void give_word(uint64_t* at, float A, float B) {
  __hip_atomic_store(at, uint64_t(__float_as_uint(B)) << 32 | word_of(A), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// The value that reaches tile `order` (of the order of work), for the thread's own channels.  Tiles come in bunches of
// kBunch.  Per channel, a lane of the first wave publishes the tile's map and composes those of the bunch's tiles before
// it, and the last tile's publishes the bunch's; a lane of the second wave composes the maps of the kBunches bunches
// before this one upon the value that reached the first of them, and the first tile's publishes the value that reaches the
// bunch.  A value is a word whose A hands nothing on.
template <int CL, bool BACK>
__device__ __forceinline__ void look_back(const ScanParams& p, int order, int group, const float (*tot)[2][4 * CL],
                                          float (*link)[2][4 * CL], float (&v)[4]) {
  constexpr int CH = 4 * CL;
  const int lane = threadIdx.x & 63, wave = uniform(int(threadIdx.x >> 6)), ch = group * CH + lane;
  const int bunch = order / kBunch, place = order % kBunch;
  const bool here = lane < CH && ch < p.c;
  if (wave < 2 && here) {
    float A, B;
    if (wave == 0) {
      float mA, mB;
      Tile<CL>::template whole<BACK>(tot, lane, &mA, &mB);
      uint64_t* mine = p.maps + int64_t(order) * p.c + ch;
      give_word(mine, mA, mB);
      const uint64_t* from = mine - int64_t(place) * p.c;
      take_words<kBunch - 1>(from, from, p.c, place, A, B);
      if (place == kBunch - 1) give_word(p.bunches + int64_t(bunch) * p.c + ch, times(mA, A), after(mA, mB, B));
    } else {
      // the value that reached bunch `from`, then that bunch and those after it
      const int from = bunch > kBunches ? bunch - kBunches : 0;
      take_words<kBunches + 1>(p.values + int64_t(from) * p.c + ch, p.bunches + (int64_t(from) - 1) * p.c + ch, p.c,
                               bunch - from + 1, A, B);
      if (place == 0 && bunch > 0) give_word(p.values + int64_t(bunch) * p.c + ch, A, B);
    }
    link[wave][0][lane] = A;
    link[wave][1][lane] = B;
  }
  __syncthreads();
  const int col = threadIdx.x % CL;
  if (group * CH + col * 4 < p.c)
#pragma unroll
    for (int w = 1; w >= 0; --w) {
      float a[4], b[4];
      load_state(&link[w][0][col * 4], a);
      load_state(&link[w][1][col * 4], b);
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = after(a[k], b[k], v[k]);
    }
}

// The tile's number in the order of work, for all threads
__device__ __forceinline__ int take_ticket(const ScanParams& p, int* slot) {
  if (p.tiles == 1) return int(blockIdx.x);
  if (threadIdx.x == 0) *slot = int(__hip_atomic_fetch_add(p.ticket, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT));
  __syncthreads();
  return uniform(*slot);
}

// Samples with no rows hand on the state (or its gradient) that reaches them; the tiles share them out.
template <int CL>
__device__ __forceinline__ void empty_samples(const ScanParams& p, int tile, int c0, bool mine, const float* from, float* to) {
  constexpr int CH = 256 / CL;
  if (!to || !mine) return;
  for (int64_t b = int64_t(tile) * CH + threadIdx.x / CL; b < p.batch; b += int64_t(p.tiles) * CH) {
    int begin = p.off[b], end = p.off[b + 1];
    begin = begin < 0 ? 0 : begin;
    end = end > p.n ? int(p.n) : end;
    if (begin < end) continue;
    float f[4] = {0.f, 0.f, 0.f, 0.f};
    if (from) load_state(from + b * p.c + c0, f);
    store_state(to + b * p.c + c0, f);
  }
}

// LB: rows of the backward pass's threads, whose tiles are as many times shorter as L is larger
template <typename T, int CL, int L, int LB, bool MIX>
__global__ void __launch_bounds__(256, sizeof(T) == 2 ? 3 : 2) scan_fwd(ScanParams p) {
  using TL = Tile<CL>;
  using F = Four<T>;
  constexpr int kRows = 256 / CL * L;
  __shared__ __align__(16) int info[kRows];
  __shared__ __align__(16) float tot[4][2][4 * CL], link[2][2][4 * CL];
  __shared__ __align__(16) float apart[2][256][4];
  __shared__ int slot;
  const int work = take_ticket(p, &slot), group = work % p.groups, tile = work / p.groups;
  const int chunk = threadIdx.x / CL, c0 = (group * CL + threadIdx.x % CL) * 4;
  const bool mine = c0 < p.c;
  const int64_t first = int64_t(tile) * kRows, t0 = first + chunk * L;
  const bool whole = first + kRows <= p.n;  // every row of the tile exists
  const int rows = t0 >= p.n ? 0 : (p.n - t0 < L ? int(p.n - t0) : L);
  // lanes past the last channel compute on the first ones and keep nothing
  const int col = (mine ? c0 : 0) * int(sizeof(T));
  Lane xl, gl;
  xl.init(p.x, p.x_row * int64_t(sizeof(T)), p, first, chunk * L, kRows, col);
  gl.init(p.gate, p.gate_row * int64_t(sizeof(T)), p, first, chunk * L, kRows, col);
  typename F::raw xv[L], gv[L];
  if (whole) {
#pragma unroll
    for (int i = 0; i < L; ++i) {
      xv[i] = xl.get<typename F::raw>(i);
      gv[i] = gl.get<typename F::raw>(i);
    }
  } else {
#pragma unroll
    for (int i = 0; i < L; ++i) {
      xv[i] = gv[i] = F::none();
      if (i < rows) {
        xv[i] = xl.get<typename F::raw>(i);
        gv[i] = gl.get<typename F::raw>(i);
      }
    }
  }
  for (int r = threadIdx.x; r < kRows; r += 256) info[r] = row_info(p, int64_t(tile) * kRows + r);
  __syncthreads();
  int any = 0;
#pragma unroll
  for (int i = 0; i < L; ++i) any |= info[chunk * L + i];
  const bool plain = !__any((any & 3) != 0);  // no row of the wave begins or ends a sample, or is of none

  float a[L][4], b[L][4], A[4] = {1.f, 1.f, 1.f, 1.f}, B[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < L; ++i) {
    float g[4], x[4];
    F::unpack(gv[i], g);
    F::unpack(xv[i], x);
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      float keep;
      sides<T>(g[v], a[i][v], keep);
      b[i][v] = MIX ? keep * x[v] : x[v];
    }
    if (!plain) {
      const int what = info[chunk * L + i];
      if (what & kFirst) {  // kNone has all bits
        float h[4] = {0.f, 0.f, 0.f, 0.f};
        if (what != kNone && p.h0 && mine) load_state(p.h0 + int64_t(what >> 2) * p.c + c0, h);
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          b[i][v] = what == kNone ? 0.f : fmaf(a[i][v], h[v], b[i][v]);
          a[i][v] = B[v] = 0.f;
          A[v] = kDrop;
        }
      }
    }
    // a NaN decay makes A one where it should stay -0, but B as well
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      B[v] = fmaf(a[i][v], B[v], b[i][v]);
      A[v] *= a[i][v];
    }
  }
  TL::template join<false>(A, B, tot);
  // the thread's map waits in LDS while registers hold the words between tiles: with 28 bytes of a lane's registers in
  // scratch instead of 64, three waves a SIMD are worth having (629k rows x 1,024 channels: 816 -> 763 us)
  store_state(&apart[0][threadIdx.x][0], A);
  store_state(&apart[1][threadIdx.x][0], B);
  __syncthreads();
  empty_samples<CL>(p, tile, c0, mine, p.h0, p.last);
  float h[4] = {0.f, 0.f, 0.f, 0.f};
  if (p.tiles > 1) look_back<CL, false>(p, tile, group, tot, link, h);
  load_state(&apart[0][threadIdx.x][0], A);
  load_state(&apart[1][threadIdx.x][0], B);
  TL::template enter<false>(h, A, B, tot);
  if (!mine) return;
  constexpr int kParts = L / LB, kPart = 256 / CL / kParts;
  if (p.carries && chunk % kPart == 0 && rows > 0)
    store_state(p.carries + (int64_t(tile) * kParts + chunk / kPart) * p.c + c0, h);
  Lane yl;
  yl.init(p.y, p.c * int64_t(sizeof(T)), p, first, chunk * L, kRows, col);
#pragma unroll
  for (int i = 0; i < L; ++i) {
    int what = 0;
    if (!plain) {
      what = info[chunk * L + i];
      if (what & kFirst)
#pragma unroll
        for (int v = 0; v < 4; ++v) h[v] = 0.f;
    }
#pragma unroll
    for (int v = 0; v < 4; ++v) h[v] = fmaf(a[i][v], h[v], b[i][v]);
    if (!whole && i >= rows) break;
    yl.put(i, F::pack(h));
    if (!plain && what != kNone && (what & kLast)) store_state(p.last + int64_t(what >> 2) * p.c + c0, h);
  }
}

template <typename T, int CL, int L, bool MIX>
__global__ void __launch_bounds__(256, sizeof(T) == 2 ? 3 : 2) scan_bwd(ScanParams p) {
  using TL = Tile<CL>;
  using F = Four<T>;
  constexpr int kRows = 256 / CL * L;
  __shared__ __align__(16) int info[kRows];
  __shared__ __align__(16) float tot[4][2][4 * CL], totb[4][2][4 * CL], link[2][2][4 * CL];
  __shared__ int slot;
  const int work = take_ticket(p, &slot), group = work % p.groups, order = work / p.groups, tile = p.tiles - 1 - order;
  const int chunk = threadIdx.x / CL, c0 = (group * CL + threadIdx.x % CL) * 4;
  const bool mine = c0 < p.c;
  const int64_t first = int64_t(tile) * kRows, t0 = first + chunk * L;
  const bool whole = first + kRows <= p.n;
  const int rows = t0 >= p.n ? 0 : (p.n - t0 < L ? int(p.n - t0) : L);
  const int col = (mine ? c0 : 0) * int(sizeof(T));
  Lane xl, gl, ul;
  xl.init(p.x, p.x_row * int64_t(sizeof(T)), p, first, chunk * L, kRows, col);
  gl.init(p.gate, p.gate_row * int64_t(sizeof(T)), p, first, chunk * L, kRows, col);
  ul.init(p.dy, p.c * int64_t(sizeof(T)), p, first, chunk * L, kRows, col);
  typename F::raw xv[L], gv[L], uv[L];
  if (whole) {
#pragma unroll
    for (int i = 0; i < L; ++i) {
      gv[i] = gl.get<typename F::raw>(i);
      uv[i] = ul.get<typename F::raw>(i);
      xv[i] = xl.get<typename F::raw>(i);
    }
  } else {
#pragma unroll
    for (int i = 0; i < L; ++i) {
      xv[i] = gv[i] = uv[i] = F::none();
      if (i < rows) {
        gv[i] = gl.get<typename F::raw>(i);
        uv[i] = ul.get<typename F::raw>(i);
        xv[i] = xl.get<typename F::raw>(i);
      }
    }
  }
  float h[4] = {0.f, 0.f, 0.f, 0.f};
  if (tile > 0 && mine) load_state(p.carries + int64_t(tile) * p.c + c0, h);
  for (int r = threadIdx.x; r < kRows; r += 256) info[r] = row_info(p, int64_t(tile) * kRows + r);
  __syncthreads();
  int any = 0;
#pragma unroll
  for (int i = 0; i < L; ++i) any |= info[chunk * L + i];
  const bool plain = !__any((any & 3) != 0);

  float a[L][4], keep[L][4], u[L][4];
#pragma unroll
  for (int i = 0; i < L; ++i) {
    float g[4];
    F::unpack(gv[i], g);
#pragma unroll
    for (int v = 0; v < 4; ++v) sides<T>(g[v], a[i][v], keep[i][v]);
  }
  // rows of no sample become rows of zeros, which begin and hand on nothing
  if (!plain) {
#pragma unroll
    for (int i = 0; i < L; ++i)
      if (info[chunk * L + i] == kNone) {
        xv[i] = uv[i] = F::none();
#pragma unroll
        for (int v = 0; v < 4; ++v) a[i][v] = keep[i][v] = 0.f;
      }
  }
  // the value that a sample's first row (its last one, in the other direction) begins with
  auto begin = [&](const float* from, int what, float (&f)[4]) {
#pragma unroll
    for (int v = 0; v < 4; ++v) f[v] = 0.f;
    if (what != kNone && from && mine) load_state(from + int64_t(what >> 2) * p.c + c0, f);
  };
  float A[4] = {1.f, 1.f, 1.f, 1.f}, B[4] = {0.f, 0.f, 0.f, 0.f};
  float Ab[4] = {1.f, 1.f, 1.f, 1.f}, Bb[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = L - 1; i >= 0; --i) {
    float dy[4];
    F::unpack(uv[i], dy);
    if (!plain) {
      const int what = info[chunk * L + i];
      if (what & kLast) {  // kNone has all bits
        begin(p.dlast, what, Bb);
#pragma unroll
        for (int v = 0; v < 4; ++v) Ab[v] = kDrop;
      }
    }
    // a NaN decay makes A one where it should stay -0, but B as well
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      Bb[v] = a[i][v] * (dy[v] + Bb[v]);
      Ab[v] *= a[i][v];
    }
  }
#pragma unroll
  for (int i = 0; i < L; ++i) {
    float x[4];
    F::unpack(xv[i], x);
    if (!plain) {
      const int what = info[chunk * L + i];
      if (what & kFirst) {
        begin(p.h0, what, B);
#pragma unroll
        for (int v = 0; v < 4; ++v) A[v] = kDrop;
      }
    }
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      B[v] = fmaf(a[i][v], B[v], MIX ? keep[i][v] * x[v] : x[v]);
      A[v] *= a[i][v];
    }
  }
  TL::template join<true>(Ab, Bb, totb);
  TL::template join<false>(A, B, tot);
  __syncthreads();
  empty_samples<CL>(p, tile, c0, mine, p.dlast, p.dh0);
  float c[4] = {0.f, 0.f, 0.f, 0.f};
  if (p.tiles > 1) look_back<CL, true>(p, order, group, totb, link, c);
  TL::template enter<false>(h, A, B, tot);
  TL::template enter<true>(c, Ab, Bb, totb);
  if (!mine) return;
#pragma unroll
  for (int i = 0; i < L; ++i) {
    float x[4];
    afresh(xv[i]);
    F::unpack(xv[i], x);
    if (!plain) {
      const int what = info[chunk * L + i];
      if (what & kFirst) begin(p.h0, what, h);
    }
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      u[i][v] = MIX ? h[v] - x[v] : h[v];
      h[v] = fmaf(a[i][v], h[v], MIX ? keep[i][v] * x[v] : x[v]);
    }
  }
  Lane dxl, dgl;
  dxl.init(p.dx, p.c * int64_t(sizeof(T)), p, first, chunk * L, kRows, col);
  dgl.init(p.dgate, p.c * int64_t(sizeof(T)), p, first, chunk * L, kRows, col);
#pragma unroll
  for (int i = L - 1; i >= 0; --i) {
    float dy[4], dx[4], dg[4];
    afresh(uv[i]);
    F::unpack(uv[i], dy);
    if (!plain) {
      const int what = info[chunk * L + i];
      if (what & kLast) begin(p.dlast, what, c);
    }
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const float d = dy[v] + c[v], kd = keep[i][v] * d;
      dx[v] = MIX ? kd : d;
      dg[v] = kd * u[i][v] * a[i][v];
      c[v] = a[i][v] * d;
    }
    if (!whole && i >= rows) continue;
    dxl.put(i, F::pack(dx));
    dgl.put(i, F::pack(dg));
    if (!plain && p.dh0) {
      const int what = info[chunk * L + i];
      if (what != kNone && (what & kFirst)) store_state(p.dh0 + int64_t(what >> 2) * p.c + c0, c);
    }
  }
}

// Clears the words between tiles (in 16-byte pieces; first, per: the first bunch's values) and the counter
__global__ void __launch_bounds__(256) scan_clear(uint4* words, int64_t n, int64_t first, int64_t per, uint32_t* ticket) {
  const int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x;
  // what reaches the first bunch is zero
  if (i < n) words[i] = i >= first && i < first + per ? make_uint4(0, 0, 0, 0) : make_uint4(kNotYet, kNotYet, kNotYet, kNotYet);
  if (i == 0) *ticket = 0;
}

int esize(int32_t dtype) { return dtype == SSC_F32 ? 4 : 2; }
bool bad(const void* ptr) { return !ptr || !aligned16(ptr); }

// Forms of a call
struct ScanPlan {
  bool few;   // see kFewTiles
  int lanes;  // of a tile's row
  int64_t fwd_tiles, bwd_tiles, groups;  // tiles along the rows, groups of channels
};
constexpr int64_t kFewTiles = 512;

int64_t scan_tiles(int64_t n, int lanes, int rows) {
  const int64_t per = int64_t(256 / lanes) * rows;
  return n > 0 ? (n + per - 1) / per : 1;
}
ScanPlan scan_plan(const ssc_scan_shape& a) {
  const int vecs = a.channels / kFour;
  ScanPlan s{};
  s.lanes = vecs <= 8 ? 8 : 16;
  s.groups = (vecs + s.lanes - 1) / s.lanes;
  s.bwd_tiles = scan_tiles(a.n, s.lanes, kBackRows);
  s.few = s.bwd_tiles * s.groups < kFewTiles;
  s.fwd_tiles = scan_tiles(a.n, s.lanes, fwd_rows(esize(a.dtype), s.few));
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
    if (v < 0 || v > SSC_MAX_SCAN_ROW_STRIDE || v % vec != 0) return SSC_ERR_INVALID_ARG;
  const ScanPlan s = scan_plan(*a);
  // HIP takes fewer than 2^32 threads in a dimension of a launch
  return s.bwd_tiles * s.groups * 256 < (1LL << 32) ? SSC_OK : SSC_ERR_UNSUPPORTED;
}

ScanParams scan_params(const ssc_scan_shape& a, const ScanPlan& s, bool back) {
  ScanParams p{};
  p.n = a.n;
  p.x_row = a.x_row_stride;
  p.gate_row = a.gate_row_stride;
  p.c = a.channels;
  p.batch = a.batch;
  p.tiles = int32_t(back ? s.bwd_tiles : s.fwd_tiles);
  p.groups = int32_t(s.groups);
  p.rev = a.reverse != 0;
  return p;
}

size_t carry_bytes(const ssc_scan_shape& a) {
  const ScanPlan s = scan_plan(a);
  return size_t(s.bwd_tiles) * size_t(a.channels) * 4;
}

// words between the tiles of a pass: their maps, the bunches' and the values that reach the bunches
int64_t bunch_count(int64_t tiles) { return (tiles + kBunch - 1) / kBunch; }
int64_t word_count(int64_t tiles, int64_t channels) { return (tiles + 2 * bunch_count(tiles)) * channels; }
constexpr size_t kTicketBytes = 256;  // the counter lies first

size_t scan_ws(const ssc_scan_shape& a) {
  const ScanPlan s = scan_plan(a);
  const int64_t most = s.fwd_tiles > s.bwd_tiles ? s.fwd_tiles : s.bwd_tiles;
  return kTicketBytes + (most > 1 ? size_t(word_count(most, a.channels)) * 8 : 0);  // a single tile exchanges nothing
}

void set_words(ScanParams* p, void* workspace) {
  p->ticket = static_cast<uint32_t*>(workspace);
  p->maps = reinterpret_cast<uint64_t*>(static_cast<char*>(workspace) + kTicketBytes);
  p->bunches = p->maps + int64_t(p->tiles) * p->c;
  p->values = p->bunches + bunch_count(p->tiles) * p->c;
}

template <typename T, int CL, int L>
void scan_launch(const ScanParams& p, bool mix, bool back, hipStream_t s) {
  const unsigned grid = unsigned(int64_t(p.tiles) * p.groups);
  if (back) {
    if (mix)
      scan_bwd<T, CL, kBackRows, true><<<grid, 256, 0, s>>>(p);
    else
      scan_bwd<T, CL, kBackRows, false><<<grid, 256, 0, s>>>(p);
  } else {
    if (mix)
      scan_fwd<T, CL, L, kBackRows, true><<<grid, 256, 0, s>>>(p);
    else
      scan_fwd<T, CL, L, kBackRows, false><<<grid, 256, 0, s>>>(p);
  }
}

template <typename T, int CL>
void scan_rows(const ScanPlan& f, const ScanParams& p, bool mix, bool back, hipStream_t s) {
  if (f.few)
    scan_launch<T, CL, fwd_rows(sizeof(T), true)>(p, mix, back, s);
  else
    scan_launch<T, CL, fwd_rows(sizeof(T), false)>(p, mix, back, s);
}

template <typename T>
void scan_form(const ScanPlan& f, const ScanParams& p, bool mix, bool back, hipStream_t s) {
  if (f.lanes == 8)
    scan_rows<T, 8>(f, p, mix, back, s);
  else
    scan_rows<T, 16>(f, p, mix, back, s);
}

int scan_run(const ssc_scan_shape& a, const ScanPlan& sp, const ScanParams& p, bool back, void* stream) {
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  const bool mix = a.form == SSC_SCAN_MIX;
  (void)hipGetLastError();
  if (p.tiles > 1) {
    const int64_t pieces = word_count(p.tiles, p.c) / 2;  // channels come in fours
    scan_clear<<<unsigned((pieces + 255) / 256), 256, 0, s>>>(reinterpret_cast<uint4*>(p.maps), pieces,
                                                           (p.values - p.maps) / 2, p.c / 2, p.ticket);
  }
  if (a.dtype == SSC_F32)
    scan_form<float>(sp, p, mix, back, s);
  else if (a.dtype == SSC_F16)
    scan_form<_Float16>(sp, p, mix, back, s);
  else
    scan_form<__bf16>(sp, p, mix, back, s);
  return hipGetLastError() == hipSuccess ? SSC_OK : SSC_ERR_HIP;
}

}  // namespace

}  // namespace ssc

using namespace ssc;

extern "C" size_t ssc_gated_scan_carry_bytes(const ssc_scan_shape* shape) {
  return scan_check(shape) == SSC_OK ? carry_bytes(*shape) : 0;
}

extern "C" size_t ssc_gated_scan_workspace_bytes(const ssc_scan_shape* shape) {
  return scan_check(shape) == SSC_OK ? scan_ws(*shape) : 0;
}

extern "C" int ssc_gated_scan_fwd(const ssc_scan_shape* shape, const void* x, const void* gate, const int32_t* offsets,
                                  const float* h0, void* y, float* last, float* carries, void* workspace,
                                  size_t workspace_bytes, void* stream) {
  const int st = scan_check(shape);
  if (st != SSC_OK) return st;
  const ssc_scan_shape& a = *shape;
  if (a.n > 0 && (bad(x) || bad(gate) || bad(y))) return SSC_ERR_INVALID_ARG;
  if (bad(offsets) || bad(last) || !aligned16(h0) || !aligned16(carries) || bad(workspace)) return SSC_ERR_INVALID_ARG;
  if (workspace_bytes < scan_ws(a)) return SSC_ERR_WORKSPACE;
  const ScanPlan sp = scan_plan(a);
  ScanParams p = scan_params(a, sp, false);
  set_words(&p, workspace);
  p.x = x;
  p.gate = gate;
  p.off = offsets;
  p.h0 = h0;
  p.y = y;
  p.last = last;
  p.carries = carries;
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
  if (workspace_bytes < scan_ws(a)) return SSC_ERR_WORKSPACE;
  const ScanPlan sp = scan_plan(a);
  ScanParams p = scan_params(a, sp, true);
  set_words(&p, workspace);
  p.x = x;
  p.gate = gate;
  p.dy = dy;
  p.off = offsets;
  p.h0 = h0;
  p.dlast = dlast;
  p.dx = dx;
  p.dgate = dgate;
  p.dh0 = dh0;
  p.carries = const_cast<float*>(carries);
  return scan_run(a, sp, p, true, stream);
}
