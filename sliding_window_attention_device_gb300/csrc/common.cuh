// Internal definitions shared by the bdattn kernels and host code.
#pragma once

#include <cstdint>
#include <utility>
#include "bdattn.h"  // include/ is on the include path

namespace bd {

constexpr int kTile = 128;          // q rows / K-V rows per tile (forward, classification)
constexpr int kSms = 152;           // SMs of a GB300
constexpr int kBwdQ = 64;           // q rows per backward iteration
constexpr uint64_t kWaitLimitNs = 2000000000ull;  // pipeline wait limit (2 s)
constexpr int kAbortBits = BD_STATUS_TIMEOUT;      // other CTAs' errors that end a wait early

// Geometry as the kernels see it (scale resolved, table offsets computed).
struct Geom {
  int B, Hq, Hkv, D, G;
  int S_full, L, row_offset, kv_offset, S_kv, window;
  float scale;
  int kv_tm;                      // k, v, dk, dv token-major: [S_kv][B][Hkv][D]
  uint32_t drop_t;                // dropout: keep iff a pair's 16-bit draw >= drop_t; 0: no dropout
  float drop_scale;               // dropout: factor of a kept weight, 2^16 / (2^16 - drop_t)
  uint32_t seed_lo, seed_hi;      // dropout: Philox key
  int nqt, nkt, nkw;              // 128-row q tiles, 128-row K/V tiles, bitmap words per q tile
  int off[BD_SEG_NOFF];           // word offsets of the table regions
  int n_sink;                     // first keys of a document that stay visible past the window (0: none)
  // sink tables only (sink_tab = 1): the regions behind the ordinary table
  int sink_tab;
  int sk_off;                     // word offset of the sink header (kSinkHdrWords), then the units, then the sums
  int sk_units, sk_sums, sk_slots;  // capacities of the unit list, the sum list and the partial slots
  int sk_rows;                    // key rows of a partial slot
  int sk_split;                   // 128-row q tiles of a unit
  int sk_heads;                   // query heads of a unit (G, unless the work is cut finely)
  int sk_fine;                    // 1: few tiles, so units are cut by q rows and heads alike
  float* sk_part;                 // partial slots of a backward, in the caller's workspace
};

__host__ __device__ inline int cdiv(int a, int b) { return (a + b - 1) / b; }
__host__ __device__ inline int align4(int x) { return (x + 3) & ~3; }

// Table layout: each region starts on a 16-byte boundary.
__host__ __device__ inline void seg_layout(int B, int L, int S_kv, int* off, int* nqt, int* nkt, int* nkw) {
  *nqt = cdiv(L, kTile);
  *nkt = cdiv(S_kv, kTile);
  *nkw = cdiv(*nkt, 32);
  int o = 0;
  off[BD_SEG_OFF_HDR] = o;        o = align4(o + B * BD_SEG_HDR_WORDS);
  off[BD_SEG_OFF_CU_Q] = o;       o = align4(o + B * (L + 1));
  off[BD_SEG_OFF_CU_K] = o;       o = align4(o + B * (L + 1));
  off[BD_SEG_OFF_ROW_LO] = o;     o = align4(o + B * L);
  off[BD_SEG_OFF_QT_KRANGE] = o;  o = align4(o + B * (*nqt) * 2);
  off[BD_SEG_OFF_KT_QRANGE] = o;  o = align4(o + B * (*nkt) * 2);
  off[BD_SEG_OFF_FULL_BITS] = o;  o = align4(o + B * (*nqt) * (*nkw));
  off[BD_SEG_OFF_FWD_WORK] = o;   o = align4(o + B * (*nqt));
  off[BD_SEG_OFF_BWD_WORK] = o;   o = align4(o + B * (*nkt));
  off[BD_SEG_OFF_COUNTS] = o;     o = align4(o + 8);
  off[BD_SEG_OFF_TOTAL] = o;
}

// Header words that record the geometry the table was built for.
constexpr int kHdrRowOffset = 16, kHdrL = 17, kHdrKvOffset = 18, kHdrSkv = 19, kHdrWindow = 20,
              kHdrSfull = 21, kHdrMagic = 22,
              kHdrKvChunk = 23,  // 1: table built for one K/V chunk (no K/V range requirement)
              kHdrSink = 24,     // n_sink the table was built for (0 in ordinary tables)
              kHdrSinkTab = 25,  // 1: the sink regions follow the table
              kHdrSinkCut = 28;  // and what these were laid out for: B, G, sk_units, sk_rows
constexpr int kSegMagic = 0x62646174;  // "bdat"

// Whether a batch row's header was written for this geometry: three 16-byte
// loads and no branch between them (each a trip to L2 that a CTA starts with).
__device__ __forceinline__ bool seg_hdr_ok(const Geom& g, const int32_t* hdr) {
  const int4 a = *reinterpret_cast<const int4*>(hdr + kHdrRowOffset);
  const int4 c = *reinterpret_cast<const int4*>(hdr + kHdrWindow);
  const int4 e = *reinterpret_cast<const int4*>(hdr + kHdrSink);
  return (a.x == g.row_offset) & (a.y == g.L) & (a.z == g.kv_offset) & (a.w == g.S_kv) & (c.x == g.window) &
         (c.y == g.S_full) & (c.z == kSegMagic) & (e.x == g.n_sink) & (e.y == g.sink_tab || g.sink_tab == 0);
}

// The kernels' kSink: ordinary, with sinks, with sinks and a window below kTile.
constexpr int kNoSink = 0, kSinkLong = 1, kSinkShort = 2;

// ---- sink tables -----------------------------------------------------------
// A sink's gradient sums over all later rows of its document: with a window W,
// the rows that attend a K/V tile are a short range, except that a tile that
// holds sinks is attended to the document's end. The backward therefore works
// on units, K/V tile by q rows: a tile's first unit (the primary) covers its
// window rows, or sk_split 128-row q tiles where that is more, and the rows
// behind it are cut into units of sk_split q tiles. Only sinks of the tile's
// last document have such rows. A tile with one unit writes its dk / dv
// directly; the units of a tile with several write those sinks' key rows,
// [rbase, rbase + sk_rows), as fp32 partials into slots of the workspace, which
// a last kernel adds in slot order, and the primary writes the other rows.
// Where the tiles are too few to occupy the SMs (sk_fine), every tile's rows are
// cut into units of sk_split q tiles and sk_heads query heads of the group, and
// all 128 key rows of a tile with several units go through slots: one head dim
// 256 unit of 8 heads and 8 q tiles is 0.4 ms of products in sequence.
constexpr int kSinkHdrWords = 8;   // n_units, n_sums, n_slots
constexpr int kSinkUnitWords = 8;  // item (b * nkt + kt), q_begin, q_end (local rows), primary, slot (-1:
                                   // none), rbase, first head of the group, heads
constexpr int kSinkSumWords = 4;   // item, first slot, slots, rbase

// Row index of (batch row b, kv head hk, K/V buffer row j) in k, v, dk, dv.
__host__ __device__ inline size_t kv_row(const Geom& g, int b, int hk, int j) {
  return g.kv_tm ? (static_cast<size_t>(j) * g.B + b) * g.Hkv + hk
                 : (static_cast<size_t>(b) * g.Hkv + hk) * g.S_kv + j;
}

// Exchange plan layout (BD_PLAN_OFF_* regions, each on a 16-byte boundary).
// Returns the total words, or -1 when a size is out of range.
constexpr int kPlanMagic = 0x62647870;  // "bdxp"
constexpr int kPlanMaxRanks = 1024;
__host__ __device__ inline long long plan_layout(int B, int W, int L, int* off) {
  if (B < 1 || W < 1 || L < 1 || W > kPlanMaxRanks) return -1;
  if (static_cast<long long>(W) * L > 0x7fffffffLL || static_cast<long long>(B) * W > (1 << 24)) return -1;
  long long o = 0;
  long long sz[BD_PLAN_OFF_TOTAL] = {BD_PLAN_HDR_WORDS, W, W, W, W, static_cast<long long>(W) * W, W, W, W, W,
                                     static_cast<long long>(W) * L, 2LL * B * W};
  for (int i = 0; i < BD_PLAN_OFF_TOTAL; ++i) {
    off[i] = static_cast<int>(o);
    o = (o + sz[i] + 3) & ~3LL;
    if (o > 0x7fffffffLL) return -1;
  }
  off[BD_PLAN_OFF_TOTAL] = static_cast<int>(o);
  return o;
}

// The allowed key interval [lo, hi] (global positions) of a real local row i:
// hi = p, lo = max(doc_start, p - W + 1).
__device__ __forceinline__ int row_lo_window(int doc_start, int p, int window) {
  return (window > 0 && p - window + 1 > doc_start) ? p - window + 1 : doc_start;
}

// Capacities of a sink table and its partial slots. A tile has several units
// only if its last document has more than (sk_split - 2) * kTile local rows, so
// at most L / that many documents count, each with its sinks (n <= 128) in at
// most two tiles; a document's rows are cut once for each of the two. Cut
// finely, any tile may have several: its window's q tiles and its sinks' tails.
__host__ __device__ inline void sink_sizes(Geom* g) {
  const bool on = g->window > 0 && g->n_sink > 0;
  g->sk_rows = g->n_sink > 0 ? g->n_sink : 1;
  g->sk_heads = g->G;
  g->sk_fine = 0;
  const int w_tiles = g->window > 0 ? g->window / kTile + 1 : g->nqt;
  g->sk_split = w_tiles > 8 ? w_tiles : 8;  // a unit about as long as a window's, and not short
  // tiles with a unit: those reachable by position through the window, and the
  // straddling document's sinks
  const long long hi = static_cast<long long>(g->row_offset) + g->L - 1 - g->kv_offset;
  const long long lo = g->window > 0 ? static_cast<long long>(g->row_offset) - g->window + 1 - g->kv_offset : 0;
  const long long a = lo > 0 ? lo : 0;
  const long long z = hi < g->S_kv - 1 ? hi : static_cast<long long>(g->S_kv) - 1;
  const long long seen = z < a ? 0 : z / kTile - a / kTile + 1;
  long long reach = seen + (on ? 2 : 0);
  if (reach > g->nkt) reach = g->nkt;
  // Half the SMs or fewer with a tile, and four or more (head, q tile) steps in
  // the longest unit: cut to an SM's share of all the steps, by heads first.
  const int slices = g->D == 512 ? 4 : 1;
  const long long ctas = g->B * (seen > 0 ? seen : 1) * g->Hkv * slices;
  const int longest = g->nqt < g->sk_split ? g->nqt : g->sk_split;  // q tiles
  if (on && 2 * ctas <= kSms && static_cast<long long>(g->G) * longest >= 4) {
    const int near = w_tiles + 1 < g->nqt ? w_tiles + 1 : g->nqt;
    const long long steps = static_cast<long long>(g->B) * g->Hkv * slices * g->G * (seen * near + g->nqt);
    const long long share = steps / kSms > 1 ? steps / kSms : 1;
    const int by = share < g->G ? static_cast<int>((g->G + share - 1) / share) : 1;  // groups of heads
    g->sk_fine = 1;
    g->sk_rows = kTile;
    g->sk_heads = cdiv(g->G, by);
    const long long split = share / g->sk_heads;
    g->sk_split = split < 1 ? 1 : split < longest ? static_cast<int>(split) : longest;
  }
  const int hs = cdiv(g->G, g->sk_heads);
  long long t = 0, e = 0;  // tiles with several units; units beyond the first of a tile
  if (g->sk_fine) {
    const long long win = w_tiles + 2 < g->nqt ? w_tiles + 2 : g->nqt;
    t = reach;
    e = hs * (reach + (reach * (win + 2) + 2LL * g->nqt) / g->sk_split + 2);
  } else if (on) {
    t = 2LL * (g->L / ((g->sk_split - 2) * kTile) + 1);
    if (t > g->nkt) t = g->nkt;
    e = t + 2LL * (g->L / (g->sk_split * kTile)) + 2;
  }
  g->sk_sums = static_cast<int>(g->B * t);
  g->sk_slots = static_cast<int>(g->B * (t + e));
  g->sk_units = static_cast<int>(g->B * (reach + e));
}

// Words of the sink regions (each region a multiple of 4 words).
__host__ __device__ inline long long sink_words(const Geom& g) {
  return kSinkHdrWords + static_cast<long long>(g.sk_units) * kSinkUnitWords +
         static_cast<long long>(g.sk_sums) * kSinkSumWords;
}

// Sink passes of q tile qt. The rows of a document see its sinks before their
// window; only the q tile's first document has sinks that its rows' windows have
// left behind (a document that starts inside the q tile does so behind the first
// row's window), and those lie in at most two K/V tiles (n <= 128): [*x0, *x0 +
// *nx). A q tile walks these first, seeing that document's sinks only, then its
// window's tiles, seeing the window only (and, for W < kTile, the sinks of the
// documents that start inside it: RowKeys); a tile may come up in both walks.
// Where a sink tile's sinks fit 32 columns from a 16-column boundary on, col[] is
// the first of them and the pass works on 32 keys instead of 128, else -1. ds:
// the document start of the q tile's first row (row_lo).
__device__ inline void sink_passes(const Geom& g, int ds, int qt, int n_real, int* x0, int* nx, int* col) {
  *x0 = *nx = 0;
  col[0] = col[1] = -1;
  const int first = qt * kTile;
  if (g.window <= 0 || g.n_sink <= 0 || first >= n_real) return;
  const int last = first + kTile - 1 < n_real - 1 ? first + kTile - 1 : n_real - 1;
  const int lo = g.row_offset + last - g.window + 1;  // no row of the document sees a window key before it
  if (ds < 0 || lo <= ds) return;
  const int a = ds > g.kv_offset ? ds - g.kv_offset : 0;
  int e = (ds + g.n_sink < lo ? ds + g.n_sink : lo) - 1 - g.kv_offset;
  if (e > g.S_kv - 1) e = g.S_kv - 1;
  if (e < a) return;
  *x0 = a / kTile;
  *nx = e / kTile - *x0 + 1;
  for (int k = 0; k < *nx; ++k) {
    const int c_a = k == 0 ? a % kTile : 0, c_e = k == *nx - 1 ? e % kTile : kTile - 1;
    const int c0 = (c_a & ~15) < kTile - 32 ? (c_a & ~15) : kTile - 32;
    if (c_e - c0 < 32) col[k] = c0;
  }
}

// The keys a row sees beside its window [jlo, ...]: buffer rows [slo, shi], its
// document's sinks before the window (slo > shi: none). `inner`: they are seen in
// the window passes, as the document starts inside the q tile that starts at
// global position p0 (only with W < kTile does that leave any), not in the sink
// passes.
struct RowKeys {
  int slo = 1, shi = 0;
  bool inner = false;
};
template <int kSink>
__device__ __forceinline__ RowKeys row_sinks(const Geom& g, int doc_start, int jlo, int p0) {
  RowKeys k;
  const int d = doc_start - g.kv_offset;
  if (g.window <= 0 || g.n_sink <= 0 || d >= jlo) return k;
  k.slo = d;
  k.shi = (d + g.n_sink < jlo ? d + g.n_sink : jlo) - 1;
  if (k.shi > g.S_kv - 1) k.shi = g.S_kv - 1;  // a K/V chunk may end among them
  if constexpr (kSink == kSinkShort) k.inner = doc_start > p0;
  return k;
}

// Keep bits [c0, c0 + 32) of a row's 128, c0 a multiple of 16.
__device__ __forceinline__ uint32_t keep_bits32(const uint32_t (&km)[4], int c0) {
  const int w = c0 >> 5;
  const uint32_t lo = w == 0 ? km[0] : w == 1 ? km[1] : w == 2 ? km[2] : km[3];
  const uint32_t hi = w == 0 ? km[1] : w == 1 ? km[2] : km[3];
  return (c0 & 16) ? (lo >> 16) | (hi << 16) : lo;
}

// Units of a sink table, or -1 when the table is not one for this geometry. The
// regions' places and the units' heads, rows and slots follow from the batch and
// the heads too, which the ordinary table does not depend on; with B, G, sk_units
// and sk_rows alike and the counts within capacity the units say the rest.
__device__ __forceinline__ int sink_n_units(const Geom& g, const int32_t* seg) {
  const int32_t* hdr = seg + g.off[BD_SEG_OFF_HDR];
  const int4 cut = *reinterpret_cast<const int4*>(hdr + kHdrSinkCut);  // one trip with the header's other words
  if (!(seg_hdr_ok(g, hdr) & (hdr[kHdrSinkTab] == 1) & (cut.x == g.B) & (cut.y == g.G) & (cut.z == g.sk_units) &
        (cut.w == g.sk_rows)))
    return -1;
  const int4 n = *reinterpret_cast<const int4*>(seg + g.sk_off);
  return n.x <= g.sk_units && n.y <= g.sk_sums && n.z <= g.sk_slots ? n.x : -1;
}

// Where key row r of a unit's tile goes: >= 0 a row of the unit's partial slot,
// -1 straight to dk / dv, -2 nowhere (the tile's primary unit writes it).
__device__ __forceinline__ int unit_part_row(const Geom& g, int slot, int primary, int rbase, int r) {
  if (slot < 0) return -1;
  if (r >= rbase && r < rbase + g.sk_rows) return r - rbase;
  return primary ? -1 : -2;
}
// A slot row of dk (which = 0) or dv (1) of kv head hk.
__device__ __forceinline__ float* unit_part(const Geom& g, int slot, int hk, int which, int row) {
  return g.sk_part + (((static_cast<size_t>(slot) * g.Hkv + hk) * 2 + which) * g.sk_rows + row) * g.D;
}

// The end of the rows (global positions, from key on) that attend key `key` of
// document [ds, de): the document's end for a sink, else the window's.
__device__ __forceinline__ int sink_row_end(const Geom& g, int key, int ds, int de) {
  if (g.window <= 0 || key - ds < g.n_sink) return de;
  return key + g.window < de ? key + g.window : de;
}

// Number of 128-row K/V tiles some local row can attend by position alone:
// a row p in [row_offset, row_offset + L) attends keys s <= p and, with a
// window W, s > p - W. Every tile the segment table marks as attended lies in
// this range, so a backward grid of B x this many tiles covers them all.
__host__ __device__ inline int kv_tiles_reachable(const Geom& g) {
  const long long hi = static_cast<long long>(g.row_offset) + g.L - 1 - g.kv_offset;
  const long long lo = g.window > 0 ? static_cast<long long>(g.row_offset) - g.window + 1 - g.kv_offset : 0;
  const long long a = lo > 0 ? lo : 0;
  const long long e = hi < g.S_kv - 1 ? hi : static_cast<long long>(g.S_kv) - 1;
  return e < a ? 0 : static_cast<int>(e / kTile - a / kTile + 1);
}

#ifdef __CUDACC__
// Programmatic dependent launch. Every kernel of the library is launched with
// programmatic stream serialization and starts with pdl_begin(): it waits
// (griddepcontrol.wait) until the grids before it in the stream have completed
// and their memory is visible -- so it touches no global memory before that --
// and then lets the next grid launch (griddepcontrol.launch_dependents). A
// dependent grid launches only once every CTA of this one has started, so its
// CTAs take only resources this grid leaves free; what it gains is that its
// CTAs are already resident when this grid ends, instead of launching then.
__device__ __forceinline__ void pdl_begin() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

template <class... Exp, class... Act>
inline cudaError_t launch_pdl(void (*kernel)(Exp...), dim3 grid, dim3 block, size_t smem, cudaStream_t st,
                              Act&&... args) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Act>(args)...);
}

// Zero dK / dV rows of the K/V tiles no local row attends. The backward work
// list holds the n_att attended tiles first; the (position, kv head) pairs of
// the rest, x = (z - n_att) * Hkv + hk, are taken by writer w of n_w as
// x = w, w + n_w, ...; threads t = 0..nthr-1 share each tile. The stores are
// marked streaming (evict-first) as nothing reads these lines again soon.
__device__ inline void zero_unattended_kv(const int32_t* seg, const Geom& g, int n_att, int w, int n_w, int t, int nthr,
                                          void* dk, void* dv, int grads_bf16, int32_t* status) {
  const int n_items = g.B * g.nkt;
  const long long n_pairs = static_cast<long long>(n_items - n_att) * g.Hkv;
  const size_t row_bytes = static_cast<size_t>(g.D) * (grads_bf16 ? 2 : 4);  // a multiple of 16
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  for (long long x = w; x < n_pairs; x += n_w) {
    const int z = n_att + static_cast<int>(x / g.Hkv), hk = static_cast<int>(x % g.Hkv);
    const int wi = seg[g.off[BD_SEG_OFF_BWD_WORK] + z];
    if (wi < 0 || wi >= n_items) {
      if (t == 0) atomicOr(status, BD_STATUS_BOUNDS);
      continue;
    }
    const int b = wi / g.nkt, r0 = (wi % g.nkt) * kTile;
    const int r1 = r0 + kTile < g.S_kv ? r0 + kTile : g.S_kv;
    const size_t vpr = row_bytes / 16;  // 16-byte pieces per row
    const size_t n16 = static_cast<size_t>(r1 - r0) * vpr;
    uint4* pk = static_cast<uint4*>(dk);
    uint4* pv = static_cast<uint4*>(dv);
    if (!g.kv_tm) {  // the tile's rows are contiguous
      const size_t off = kv_row(g, b, hk, r0) * vpr;
      for (size_t i = t; i < n16; i += nthr) {
        __stcs(pk + off + i, zero);
        __stcs(pv + off + i, zero);
      }
    } else {  // token-major: one row of this kv head per token
      for (size_t i = t; i < n16; i += nthr) {
        const size_t off = kv_row(g, b, hk, r0 + static_cast<int>(i / vpr)) * vpr + i % vpr;
        __stcs(pk + off, zero);
        __stcs(pv + off, zero);
      }
    }
  }
}
#endif

}  // namespace bd
