// Ragged cross attention and windowed attention: argument checks, launch plans and the C entry points (kernels in attn.h).

#include "attn.h"

namespace ssc {
namespace attn {

template <>
int launch_fwd<float>(const Params&, const FwdPlan&, hipStream_t);
template <>
int launch_fwd<_Float16>(const Params&, const FwdPlan&, hipStream_t);
template <>
int launch_fwd<__bf16>(const Params&, const FwdPlan&, hipStream_t);
template <>
int launch_bwd<float>(Params, const BwdPlan&, const BwdParts&, hipStream_t);
template <>
int launch_bwd<_Float16>(Params, const BwdPlan&, const BwdParts&, hipStream_t);
template <>
int launch_bwd<__bf16>(Params, const BwdPlan&, const BwdParts&, hipStream_t);
template <>
int launch_win_fwd<float>(const Params&, const FwdPlan&, hipStream_t);
template <>
int launch_win_fwd<_Float16>(const Params&, const FwdPlan&, hipStream_t);
template <>
int launch_win_fwd<__bf16>(const Params&, const FwdPlan&, hipStream_t);
template <>
int launch_win_bwd<float>(Params, const BwdPlan&, const BwdParts&, hipStream_t);
template <>
int launch_win_bwd<_Float16>(Params, const BwdPlan&, const BwdParts&, hipStream_t);
template <>
int launch_win_bwd<__bf16>(Params, const BwdPlan&, const BwdParts&, hipStream_t);

namespace {

int esize(int32_t dtype) { return dtype == SSC_F32 ? 4 : 2; }

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

constexpr int64_t kCUs = 256;

// Splits of the streamed axis where the workgroups of the rows alone do not fill the chip: about `want` workgroups,
// each of at least `least` tiles.
int pick_split(int64_t wgs, int64_t want, int64_t stream_tiles, int64_t least) {
  if (wgs < 1) wgs = 1;
  int64_t n = want / wgs;
  const int64_t most = stream_tiles / least;
  if (n > most) n = most;
  if (n > kMaxSplit) n = kMaxSplit;
  return n < 1 ? 1 : int(n);
}

// A window as the kernels take it: a bound that is none is past every row.
struct Window {
  int64_t left, right, sinks;
};
constexpr int64_t kNoBound = int64_t(1) << 30;

// rows of the streamed side that a workgroup's `span` rows of the other side see, of `all`
int64_t seen_rows(const Window* w, int64_t span, int64_t all) {
  if (!w) return all;
  const int64_t n = w->left + w->right + span + w->sinks;
  return n < all ? n : all;
}

// workgroups of a pass: its tiles (an average over the samples) and heads
int64_t busy_wgs(int64_t rows, int64_t cols, const ssc_attn_shape& a) {
  const int64_t tiles = ceil_div(rows, cols);
  return (tiles > a.batch ? tiles : a.batch) * a.heads_kv;
}

// Splits of the forward and dQ passes.  Rows: two workgroups a CU fill the chip; a split is worth its share of the join
// from four 16-bit tiles on, and from one fp32 tile, whose products take about eight times as long; from four too where a
// window leaves few of them (2000 fp32 rows of four heads of 64, in a graph: 28.2 us in splits of four, 28.8 of one and
// 37 in no split; ragged 40 wide: 19.9, 25.3 and 20.2; 1500 of 128: 38.7, 55.6 and 74).  Few rows: as many workgroups as
// fit at once by their LDS, a whole number of times the rows', each wave with two tiles or more.
int row_split(bool few, int64_t wgs, int64_t kv_tiles, const ssc_attn_shape& a, const Window* w) {
  const int e = esize(a.dtype);
  // a window's few tiles of narrow 16-bit heads are over before a join would be (17 tiles: 13.4 us a call in one split,
  // 16.0 in two; 33 tiles in a graph: 16.3 and, in four, 11.9)
  if (few && w && e == 2 && a.head_dim <= 64 && kv_tiles < 24) return 1;
  if (few) return pick_split(wgs, a.head_dim <= 64 ? 2 * kCUs : kCUs, kv_tiles, 8);
  return wgs >= kCUs ? 1 : pick_split(wgs, 2 * kCUs, kv_tiles, e == 4 && !w ? 1 : 4);
}

FwdPlan fwd_plan(const ssc_attn_shape& a, const Window* w = nullptr) {
  const int64_t rows = a.nq * (a.heads_q / a.heads_kv);
  FwdPlan f{};
  f.few = rows <= 32 * int64_t(a.batch);
  const int64_t cols = f.few ? 32 : 32 * fwd_waves(esize(a.dtype), a.head_dim > 96 ? 128 : 96);
  const int64_t kv_tiles = ceil_div(seen_rows(w, cols, ceil_div(a.nk, a.batch)), tile_rows(esize(a.dtype)));
  f.tiles = int(rows / cols + a.batch + 2);
  f.nsplit = row_split(f.few, busy_wgs(rows, cols, a), kv_tiles, a, w);
  return f;
}

BwdPlan bwd_plan(const ssc_attn_shape& a, const Window* w = nullptr) {
  const int64_t rows = a.nq * (a.heads_q / a.heads_kv);
  BwdPlan b{};
  b.q_few = rows <= 32 * int64_t(a.batch);
  const int64_t qc = b.q_few ? 32 : 128, kc = 128, G = a.heads_q / a.heads_kv, tokens = ceil_div(a.nq, a.batch);
  const int64_t kv_tiles = ceil_div(seen_rows(w, qc, ceil_div(a.nk, a.batch)), tile_rows(esize(a.dtype)));
  const int64_t q_all = ceil_div(ceil_div(rows, a.batch), tile_rows(esize(a.dtype)));
  const int64_t q_tiles = w ? ceil_div(seen_rows(w, kc, tokens) * G, tile_rows(esize(a.dtype))) : q_all;
  b.q_tiles = int(rows / qc + a.batch + 2);
  b.k_tiles = int(a.nk / kc + a.batch + 2);
  b.q_split = row_split(b.q_few, busy_wgs(rows, qc, a), kv_tiles, a, w);
  // dK and dV of short encoder sequences: few column tiles over long streams, split into several rounds of workgroups
  // so that the last round's idle CUs and the samples' different lengths matter little (fp32, whose blocks are long:
  // half as many rounds).  A window's fp32 splits take four tiles, as in row_split (the sizes there: 24.8 us, 26.5 in
  // splits of two; 38.5 and 39.3; 40.4 and 47.9).
  const int64_t wgs = busy_wgs(a.nk, kc, a), want = (a.dtype == SSC_F32 ? 4 : 8) * kCUs;
  b.k_split = wgs >= want ? 1 : pick_split(wgs, want, q_tiles, a.dtype == SSC_F32 ? (w ? 4 : 2) : 8);
  if (w && w->sinks > 0) {
    // the sinks' launch is of single waves over all of a sample's tokens: about eight of them a CU, each with one fp32
    // tile at least (ragged fp32 training, 838 tokens of three heads: 27 us with two)
    const int64_t sinks = w->sinks < a.nk ? w->sinks : a.nk, all = sinks * a.batch < a.nk ? sinks * a.batch : a.nk;
    b.s_tiles = int(all / kSinkCols + a.batch + 2);
    b.s_split = pick_split(busy_wgs(all, kSinkCols, a), 8 * kCUs, q_all, a.dtype == SSC_F32 ? 1 : 8);
  }
  return b;
}

Params base_params(const ssc_attn_shape& a) {
  Params p{};
  p.nq = a.nq;
  p.nk = a.nk;
  p.q_row = a.q_row_stride;
  p.q_head = a.q_head_stride;
  p.k_row = a.k_row_stride;
  p.k_head = a.k_head_stride;
  p.v_row = a.v_row_stride;
  p.v_head = a.v_head_stride;
  p.batch = a.batch;
  p.hq = a.heads_q;
  p.hk = a.heads_kv;
  p.d = a.head_dim;
  p.G = a.heads_q / a.heads_kv;
  int l = 0;
  while ((1 << l) < p.G) ++l;
  p.gmul = uint32_t((uint64_t(1) << (31 + l)) / uint64_t(p.G) + 1);
  p.gshift = 31 + l;
  p.scale = a.scale;
  // a piece's workgroup has four rows on their way for each of its 16 groups of lanes
  p.q_piece = piece_rows(a.nq, a.heads_kv, 64 / p.G > 0 ? 64 / p.G : 1);
  p.k_piece = piece_rows(a.nk, a.heads_kv, 64);
  p.q_pieces = piece_count(a.nq, p.q_piece, a.batch);
  p.k_pieces = piece_count(a.nk, p.k_piece, a.batch);
  return p;
}

struct Ws {
  size_t part_q = 0, mean_q = 0, err_q = 0, part_k = 0, part_v = 0, delta = 0, top_q = 0, top_k = 0, total = 0;
  size_t sink_k = 0, sink_v = 0;
};

Ws ws_layout(const ssc_attn_shape& a, bool backward, const Window* win = nullptr) {
  Ws w;
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off = align_up(off + bytes, 256);
    return o;
  };
  const size_t qn = size_t(a.nq) * a.heads_q, kn = size_t(a.nk) * a.heads_kv, d = size_t(a.head_dim);
  if (!backward) {
    const FwdPlan f = fwd_plan(a, win);
    if (f.nsplit > 1) {
      w.part_q = take(size_t(f.nsplit) * qn * d * 4);
      w.part_k = take(size_t(f.nsplit) * qn * 2 * 4);
    }
  } else {
    const BwdPlan b = bwd_plan(a, win);
    if (a.dtype == SSC_F16) {
      const Params p = base_params(a);
      w.top_q = take(size_t(p.q_pieces) * size_t(a.heads_kv) * 4);
      w.top_k = take(size_t(p.k_pieces) * size_t(a.heads_kv) * 4);
    }
    w.delta = take(qn * 4);
    if (b.q_split > 1) {
      w.part_q = take(size_t(b.q_split) * qn * d * 4);
      if (a.dtype != SSC_F32) {
        w.mean_q = take(size_t(b.q_split) * qn * d * 4);
        w.err_q = take(size_t(b.q_split) * qn * 8);
      }
    }
    if (b.k_split > 1) {
      w.part_k = take(size_t(b.k_split) * kn * d * 4);
      w.part_v = take(size_t(b.k_split) * kn * d * 4);
    }
    if (b.s_split > 1) {
      const size_t rows = size_t(b.s_split) * size_t(b.s_tiles) * kSinkCols * size_t(a.heads_kv);
      w.sink_k = take(rows * d * 4);
      w.sink_v = take(rows * d * 4);
    }
  }
  w.total = off < 256 ? 256 : off;
  return w;
}

// whether a pass of `waves` waves a workgroup fits a launch: HIP takes fewer than 2^32 threads in a dimension
bool launches(int64_t tiles, int64_t nsplit, int64_t waves, const ssc_attn_shape& a) {
  return ceil_div(tiles * a.heads_kv * nsplit, 8) * 8 * waves * 64 < (1LL << 32);
}

int check_shape(const ssc_attn_shape* a, const Window* w = nullptr) {
  if (!a) return SSC_ERR_INVALID_ARG;
  if (a->dtype != SSC_F32 && a->dtype != SSC_F16 && a->dtype != SSC_BF16) return SSC_ERR_UNSUPPORTED;
  if (a->nq < 0 || a->nk < 0 || a->batch < 1 || a->heads_q < 1 || a->heads_kv < 1 || a->head_dim < 1)
    return SSC_ERR_INVALID_ARG;
  if (a->nq > SSC_MAX_ATTN_ROWS || a->nk > SSC_MAX_ATTN_ROWS || a->batch > SSC_MAX_ATTN_BATCH)
    return SSC_ERR_INVALID_ARG;
  if (a->heads_q > 1024 || a->heads_q % a->heads_kv != 0) return SSC_ERR_UNSUPPORTED;
  const int e = esize(a->dtype);
  if (a->head_dim > SSC_MAX_HEAD_DIM || (a->head_dim * e) % 16 != 0) return SSC_ERR_UNSUPPORTED;
  if (a->nq * (a->heads_q / a->heads_kv) > (1LL << 30)) return SSC_ERR_UNSUPPORTED;
  const float s = a->scale;
  if (!(s - s == 0.f)) return SSC_ERR_INVALID_ARG;  // infinite or NaN
  const int64_t rows[3] = {a->q_row_stride, a->k_row_stride, a->v_row_stride};
  const int64_t heads[3] = {a->q_head_stride, a->k_head_stride, a->v_head_stride};
  for (int64_t v : rows)
    if (v < 0 || v > SSC_MAX_ATTN_ROW_STRIDE || (v * e) % 16 != 0) return SSC_ERR_INVALID_ARG;
  for (int64_t v : heads)
    if (v < 0 || v > (1LL << 40) || (v * e) % 16 != 0) return SSC_ERR_INVALID_ARG;
  const FwdPlan f = fwd_plan(*a, w);
  const BwdPlan b = bwd_plan(*a, w);
  // The joins and the sums of splits run only where the rows' workgroups do not fill the chip, far below the limit, and
  // the pieces of top_kernel number at most 2 (kPieceBlocks + batch + 3).
  if (!launches(f.tiles, f.nsplit, f.few ? 4 : fwd_waves(esize(a->dtype), a->head_dim > 96 ? 128 : 96), *a) ||
      !launches(b.q_tiles, b.q_split, 4, *a) || !launches(b.k_tiles, b.k_split, 4, *a))
    return SSC_ERR_UNSUPPORTED;
  // the join of the sinks' splits has a workgroup of four waves a tile and key head
  if (b.s_tiles > 0 && (!launches(b.s_tiles, b.s_split, 1, *a) || !launches(b.s_tiles, 1, 4, *a))) return SSC_ERR_UNSUPPORTED;
  return SSC_OK;
}

int check_window(const ssc_attn_window* in, Window* w) {
  if (!in || in->left < -1 || in->right < -1 || in->sinks < 0 || in->left > SSC_MAX_ATTN_ROWS ||
      in->right > SSC_MAX_ATTN_ROWS || in->sinks > SSC_MAX_ATTN_ROWS)
    return SSC_ERR_INVALID_ARG;
  w->left = in->left < 0 ? kNoBound : in->left;
  w->right = in->right < 0 ? kNoBound : in->right;
  w->sinks = in->sinks;
  return SSC_OK;
}

bool bad(const void* ptr) { return !ptr || !aligned16(ptr); }

void set_window(Params* p, const Window* w) {
  if (!w) return;
  p->left = int32_t(w->left);
  p->right = int32_t(w->right);
  p->sinks = int32_t(w->sinks);
}

// the forward call, of windowed attention where there is a window
int run_fwd(const ssc_attn_shape& a, const Window* win, const void* q, const void* k, const void* v,
            const int32_t* q_offsets, const int32_t* kv_offsets, const uint8_t* kv_mask, void* out, float* lse,
            void* workspace, size_t workspace_bytes, void* stream) {
  if (a.nq == 0) return SSC_OK;
  if (bad(q) || bad(out) || bad(lse) || bad(q_offsets) || bad(kv_offsets)) return SSC_ERR_INVALID_ARG;
  if (a.nk > 0 && (bad(k) || bad(v))) return SSC_ERR_INVALID_ARG;
  const Ws w = ws_layout(a, false, win);
  if (bad(workspace)) return SSC_ERR_INVALID_ARG;
  if (workspace_bytes < w.total) return SSC_ERR_WORKSPACE;
  const FwdPlan f = fwd_plan(a, win);
  Params p = base_params(a);
  char* ws = static_cast<char*>(workspace);
  p.q = q;
  p.k = k;
  p.v = v;
  p.o = out;
  p.lse = lse;
  p.qoff = q_offsets;
  p.koff = kv_offsets;
  p.mask = kv_mask;
  p.tiles = f.tiles;
  p.nsplit = f.nsplit;
  p.part_a = reinterpret_cast<float*>(ws + w.part_q);
  p.part_b = reinterpret_cast<float*>(ws + w.part_k);
  set_window(&p, win);
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  (void)hipGetLastError();
  if (a.dtype == SSC_F32) return win ? launch_win_fwd<float>(p, f, s) : launch_fwd<float>(p, f, s);
  if (a.dtype == SSC_F16) return win ? launch_win_fwd<_Float16>(p, f, s) : launch_fwd<_Float16>(p, f, s);
  return win ? launch_win_fwd<__bf16>(p, f, s) : launch_fwd<__bf16>(p, f, s);
}

int run_bwd(const ssc_attn_shape& a, const Window* win, const void* q, const void* k, const void* v, const void* out,
            const float* lse, const void* dout, const int32_t* q_offsets, const int32_t* kv_offsets,
            const uint8_t* kv_mask, void* dq, void* dk, void* dv, void* workspace, size_t workspace_bytes, void* stream) {
  if (a.nq == 0 && a.nk == 0) return SSC_OK;
  if (bad(q_offsets) || bad(kv_offsets)) return SSC_ERR_INVALID_ARG;
  if (a.nq > 0 && (bad(q) || bad(out) || bad(lse) || bad(dout))) return SSC_ERR_INVALID_ARG;
  if (a.nk > 0 && (bad(k) || bad(v))) return SSC_ERR_INVALID_ARG;
  if (!aligned16(dq) || !aligned16(dk) || !aligned16(dv)) return SSC_ERR_INVALID_ARG;
  if (!dq && !dk && !dv) return SSC_OK;
  const Ws w = ws_layout(a, true, win);
  if (bad(workspace)) return SSC_ERR_INVALID_ARG;
  if (workspace_bytes < w.total) return SSC_ERR_WORKSPACE;
  const BwdPlan b = bwd_plan(a, win);
  Params p = base_params(a);
  char* ws = static_cast<char*>(workspace);
  p.q = q;
  p.k = k;
  p.v = v;
  p.out = out;
  p.dout = dout;
  p.dq = dq;
  p.dk = dk;
  p.dv = dv;
  p.lse = const_cast<float*>(lse);
  p.delta = reinterpret_cast<float*>(ws + w.delta);
  p.qoff = q_offsets;
  p.koff = kv_offsets;
  p.mask = kv_mask;
  set_window(&p, win);
  const BwdParts parts{reinterpret_cast<float*>(ws + w.part_q), reinterpret_cast<float*>(ws + w.mean_q),
                       reinterpret_cast<float*>(ws + w.err_q),  reinterpret_cast<float*>(ws + w.part_k),
                       reinterpret_cast<float*>(ws + w.part_v), reinterpret_cast<float*>(ws + w.sink_k),
                       reinterpret_cast<float*>(ws + w.sink_v), reinterpret_cast<float*>(ws + w.top_q),
                       reinterpret_cast<float*>(ws + w.top_k)};
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  (void)hipGetLastError();
  if (a.dtype == SSC_F32) return win ? launch_win_bwd<float>(p, b, parts, s) : launch_bwd<float>(p, b, parts, s);
  if (a.dtype == SSC_F16) return win ? launch_win_bwd<_Float16>(p, b, parts, s) : launch_bwd<_Float16>(p, b, parts, s);
  return win ? launch_win_bwd<__bf16>(p, b, parts, s) : launch_bwd<__bf16>(p, b, parts, s);
}

}  // namespace
}  // namespace attn
}  // namespace ssc

using namespace ssc;
using namespace ssc::attn;

extern "C" size_t ssc_cross_attn_workspace_bytes(const ssc_attn_shape* shape, int32_t backward) {
  if (check_shape(shape) != SSC_OK) return 0;
  return ws_layout(*shape, backward != 0).total;
}

extern "C" int ssc_cross_attn_fwd(const ssc_attn_shape* shape, const void* q, const void* k, const void* v,
                                  const int32_t* q_offsets, const int32_t* kv_offsets, const uint8_t* kv_mask,
                                  void* out, float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  const int st = check_shape(shape);
  if (st != SSC_OK) return st;
  return run_fwd(*shape, nullptr, q, k, v, q_offsets, kv_offsets, kv_mask, out, lse, workspace, workspace_bytes, stream);
}

extern "C" int ssc_cross_attn_bwd(const ssc_attn_shape* shape, const void* q, const void* k, const void* v,
                                  const void* out, const float* lse, const void* dout, const int32_t* q_offsets,
                                  const int32_t* kv_offsets, const uint8_t* kv_mask, void* dq, void* dk, void* dv,
                                  void* workspace, size_t workspace_bytes, void* stream) {
  const int st = check_shape(shape);
  if (st != SSC_OK) return st;
  return run_bwd(*shape, nullptr, q, k, v, out, lse, dout, q_offsets, kv_offsets, kv_mask, dq, dk, dv, workspace,
                 workspace_bytes, stream);
}

extern "C" size_t ssc_window_attn_workspace_bytes(const ssc_attn_shape* shape, const ssc_attn_window* window,
                                                  int32_t backward) {
  Window w;
  if (check_window(window, &w) != SSC_OK || check_shape(shape, &w) != SSC_OK) return 0;
  return ws_layout(*shape, backward != 0, &w).total;
}

extern "C" int ssc_window_attn_fwd(const ssc_attn_shape* shape, const ssc_attn_window* window, const void* q,
                                   const void* k, const void* v, const int32_t* q_offsets, const int32_t* kv_offsets,
                                   const uint8_t* kv_mask, void* out, float* lse, void* workspace,
                                   size_t workspace_bytes, void* stream) {
  Window w;
  int st = check_window(window, &w);
  if (st == SSC_OK) st = check_shape(shape, &w);
  if (st != SSC_OK) return st;
  return run_fwd(*shape, &w, q, k, v, q_offsets, kv_offsets, kv_mask, out, lse, workspace, workspace_bytes, stream);
}

extern "C" int ssc_window_attn_bwd(const ssc_attn_shape* shape, const ssc_attn_window* window, const void* q,
                                   const void* k, const void* v, const void* out, const float* lse, const void* dout,
                                   const int32_t* q_offsets, const int32_t* kv_offsets, const uint8_t* kv_mask,
                                   void* dq, void* dk, void* dv, void* workspace, size_t workspace_bytes, void* stream) {
  Window w;
  int st = check_window(window, &w);
  if (st == SSC_OK) st = check_shape(shape, &w);
  if (st != SSC_OK) return st;
  return run_bwd(*shape, &w, q, k, v, out, lse, dout, q_offsets, kv_offsets, kv_mask, dq, dk, dv, workspace,
                 workspace_bytes, stream);
}
