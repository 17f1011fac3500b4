// K1 (segmentation) and K2 (128x128 tile classification) of the block-diagonal
// CP attention path.
//
// K1 follows blockdiag_cp.kernels `_cp_blockdiag_varlen` / `_varlen_seg_for_rank`
// (NeMo AutoModel API): padding is a contiguous tail so the real local rows
// are a prefix [0, n_real); one varlen segment per document the local rows
// touch, q segment = its local rows, k segment = [doc_start, last local q + 1).
// Only the first segment can start before the shard (the straddle); every later
// segment starts inside it. The reference builds this on the host after a
// .tolist() copy; here one CTA per batch row builds it on the device, so no host
// synchronisation is needed: one pass over the row for the layout, the padding
// and the straddle, two over the local rows that count and place the segments
// with warp ballots. A chain of trips to L2 and block barriers bounds it, not the
// bytes: as few of both as the steps' order allows, and blocks no wider than the
// row needs. K1 and K2 together 5.5 us at 256 positions, 8 at 2 x 4096, 12 at
// 16384 (12, 22 and 26 with a block scan and a binary search per row and tile).
// Ids that fall, 16384 rows in documents of 128: 25 us for 15 (91 with a scan and a
// barrier per document); where only what is behind the shard falls, no more than
// rising ones (131,072 positions, 16384 of them local: 35 us).
//
// K2 marks every (128-row q tile, 128-row K/V tile) as full, partial or empty.
// A real row p may attend the keys [lo(p), p] with lo(p) = max(doc_start(p),
// p - W + 1); lo and hi are non-decreasing in p, so the non-empty K/V tiles
// of a q tile form one contiguous range, and so do the q rows of a K/V tile.
// The forward and backward kernels only visit those ranges (empty tiles are
// never loaded) and mask only the partial tiles. Tables with sinks also list the
// backward's units (common.cuh), in a CTA beside the classification's two: 1 to 3
// us more.
#include <cstdint>

#include "common.cuh"

namespace bd {

namespace {

// Every thread of the block gets the sum of `v`.
__device__ int block_add(int v, int* s_red) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, nw = blockDim.x >> 5;
  v = __reduce_add_sync(0xffffffffu, v);
  __syncthreads();
  if (lane == 0) s_red[w] = v;
  __syncthreads();
  return __reduce_add_sync(0xffffffffu, lane < nw ? s_red[lane] : 0);
}

// Exclusive prefix sum of `v` over the block; *total receives the sum.
__device__ int block_exclusive_scan(int v, int* s_red, int* total) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, nw = blockDim.x >> 5;
  int incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += t;
  }
  __syncthreads();
  if (lane == 31) s_red[w] = incl;
  __syncthreads();
  const int x = lane < nw ? s_red[lane] : 0;  // every warp sums the warps before it
  *total = __reduce_add_sync(0xffffffffu, x);
  return __reduce_add_sync(0xffffffffu, lane < w ? x : 0) + incl - v;
}

}  // namespace

// The sink-only rows of K/V tile kt of batch row b (local rows [sb, se), none
// if sb >= se) and the tile row rbase from which its last document's keys start.
// A superset: the kernels mask pair by pair.
__device__ void sink_tile_rows(const Geom& g, const int32_t* seg, int b, int kt, int* sb, int* se, int* rbase) {
  *sb = *se = *rbase = 0;
  if (g.window <= 0 || g.n_sink <= 0) return;
  const int32_t* hdr = seg + g.off[BD_SEG_OFF_HDR] + b * BD_SEG_HDR_WORDS;
  const int32_t* cu_q = seg + g.off[BD_SEG_OFF_CU_Q] + b * (g.L + 1);
  const int ro = g.row_offset, n_seg = hdr[BD_SEG_N_SEG], s_first = hdr[BD_SEG_S_FIRST];
  if (n_seg <= 0) return;
  const int s_lo = g.kv_offset + kt * kTile;
  const int s_hi = g.kv_offset + min(kt * kTile + kTile - 1, g.S_kv - 1);
  const int k_lo = max(s_lo, s_first), k_hi = min(s_hi, hdr[BD_SEG_REAL_END] - 1);
  if (k_hi < k_lo) return;
  // the document [ds, de) of the tile's last key
  int k = 0;
  if (k_hi >= ro) {
    int a = 0, e = n_seg - 1;
    while (a < e) {
      const int mid = (a + e + 1) >> 1;
      if (ro + cu_q[mid] <= k_hi) a = mid; else e = mid - 1;
    }
    k = a;
  }
  const int ds = k == 0 ? s_first : ro + cu_q[k], de = ro + cu_q[k + 1];
  const int first = max(ds, k_lo);  // its first key in the tile
  int beg = 0x3fffffff, end = 0;
  if (first - ds < g.n_sink) {
    beg = max(0, first + g.window - ro);
    end = de - ro;
  }
  *rbase = first - s_lo;
  if (g.window < kTile && ds > k_lo) {  // earlier documents of the tile may have such rows inside it
    const int beg2 = max(0, k_lo + g.window - ro), end2 = ds - ro;
    if (beg2 < end2) {
      beg = min(beg, beg2);
      end = max(end, end2);
    }
  }
  if (beg < end) {
    *sb = beg;
    *se = end;
  }
}

// The local rows with a window pair in K/V tile kt: [*wb, *we), from the tile's
// first position on, up to where the window or the last key's document ends.
__device__ void window_tile_rows(const Geom& g, const int32_t* seg, int b, int kt, int* wb, int* we) {
  const int32_t* hdr = seg + g.off[BD_SEG_OFF_HDR] + b * BD_SEG_HDR_WORDS;
  const int32_t* cu_q = seg + g.off[BD_SEG_OFF_CU_Q] + b * (g.L + 1);
  const int ro = g.row_offset, n_real = hdr[BD_SEG_N_REAL], n_seg = hdr[BD_SEG_N_SEG];
  const int s_lo = g.kv_offset + kt * kTile;
  const int s_hi = g.kv_offset + min(kt * kTile + kTile - 1, g.S_kv - 1);
  const int i_begin = max(0, s_lo - ro);
  int end = n_real;
  if (n_seg == 0 || s_hi < hdr[BD_SEG_S_FIRST]) {
    end = 0;
  } else if (s_hi < ro + n_real) {  // the document of s_hi ends the rows
    int k = 0;
    if (s_hi >= ro) {
      int a = 0, e = n_seg - 1;
      while (a < e) {
        const int mid = (a + e + 1) >> 1;
        if (ro + cu_q[mid] <= s_hi) a = mid; else e = mid - 1;
      }
      k = a;
    }
    end = cu_q[k + 1];
  }
  if (g.window > 0) end = static_cast<int>(min(static_cast<long long>(end), static_cast<long long>(s_hi) + g.window - ro));
  *wb = i_begin < end ? i_begin : 0;
  *we = i_begin < end ? end : 0;
}

// One CTA per batch row; each warp takes a contiguous piece of it, 32 positions
// at a time, so that runs are found with ballots.
__global__ void __launch_bounds__(1024) seg_build_kernel(const int32_t* __restrict__ doc, Geom g,
                                                         int32_t* __restrict__ seg, int32_t* status, int kv_chunk) {
  pdl_begin();
  __shared__ int s_red[32];
  __shared__ int s_w[4][32];
  const int b = blockIdx.x, tid = threadIdx.x, nthr = blockDim.x;
  const int lane = tid & 31, warp = tid >> 5, n_warps = nthr >> 5;
  const int ro = g.row_offset, L = g.L;
  const int32_t* row = doc + static_cast<size_t>(b) * g.S_full;
  int32_t* hdr = seg + g.off[BD_SEG_OFF_HDR] + b * BD_SEG_HDR_WORDS;
  int32_t* cu_q = seg + g.off[BD_SEG_OFF_CU_Q] + b * (L + 1);
  int32_t* cu_k = seg + g.off[BD_SEG_OFF_CU_K] + b * (L + 1);
  int32_t* rowlo = seg + g.off[BD_SEG_OFF_ROW_LO] + b * L;

  // One pass over the whole row: ids >= 0 and no document after padding; the
  // shard's first padding row (L if none); the start of the run that holds the
  // shard's first position; whether ids fall from one document to the next up to
  // the shard's end.
  int flags = 0, first_pad = L, s_first = 0;  // flags: 1 bad layout, 2 falling ids
  {
    const int piece = cdiv(cdiv(g.S_full, 32), n_warps) * 32;
    const int e = min(g.S_full, (warp + 1) * piece);
    int fall = g.S_full;  // the first position this thread sees ids fall at
#pragma unroll 8
    for (int p = warp * piece + lane; p < e; p += 32) {
      const int c = row[p], prev = p > 0 ? row[p - 1] : c;
      if (c < 0 || (c != 0 && prev == 0)) flags |= 1;
      if (c != 0 && c < prev) fall = min(fall, p);
      if (c == 0 && p >= ro) first_pad = min(first_pad, p - ro);
      if (p <= ro && c != prev) s_first = p;
    }
    if (fall < ro + L) flags |= 2;
  }
  flags = __reduce_or_sync(0xffffffffu, flags);
  first_pad = __reduce_min_sync(0xffffffffu, first_pad);
  s_first = __reduce_max_sync(0xffffffffu, s_first);
  if (lane == 0) {
    s_w[0][warp] = flags;
    s_w[1][warp] = first_pad;
    s_w[2][warp] = s_first;
  }
  __syncthreads();
  flags = __reduce_or_sync(0xffffffffu, lane < n_warps ? s_w[0][lane] : 0);
  const int n_real = __reduce_min_sync(0xffffffffu, lane < n_warps ? s_w[1][lane] : L);
  s_first = __reduce_max_sync(0xffffffffu, lane < n_warps ? s_w[2][lane] : 0);
  if (n_real == 0) s_first = ro;
  int bad = flags & 1;

  // Segments: they start at local row 0 and at every real row whose id differs
  // from the previous one. First the pieces' counts and last starts, then their
  // places; each row's document start is the last start at or before it.
  const int piece = cdiv(cdiv(n_real, 32), n_warps) * 32;
  const int r0 = min(n_real, warp * piece), r1 = min(n_real, r0 + piece);
  auto starts = [&](int i0) -> unsigned {
    const int i = i0 + lane;
    return __ballot_sync(0xffffffffu, i < r1 && (i == 0 || row[ro + i] != row[ro + i - 1]));
  };
  int count = 0, last = -1;
#pragma unroll 4
  for (int i0 = r0; i0 < r1; i0 += 32) {
    const unsigned m = starts(i0);
    count += __popc(m);
    if (m) last = i0 + 31 - __clz(m);
  }
  if (lane == 0) {
    s_w[3][warp] = count;
    s_red[warp] = last;
  }
  __syncthreads();
  const int cnt_l = lane < n_warps ? s_w[3][lane] : 0;
  const int n_seg = __reduce_add_sync(0xffffffffu, cnt_l);
  int at = __reduce_add_sync(0xffffffffu, lane < warp ? cnt_l : 0);
  int cur = __reduce_max_sync(0xffffffffu, lane < warp ? s_red[lane] : -1);  // last start before this piece
#pragma unroll 4
  for (int i0 = r0; i0 < r1; i0 += 32) {
    const unsigned m = starts(i0);
    const int i = i0 + lane;
    const unsigned upto = m & (0xffffffffu >> (31 - lane));
    if (i < r1) {
      if (m >> lane & 1u) cu_q[at + __popc(upto) - 1] = i;
      const int st = upto ? i0 + 31 - __clz(upto) : cur;  // 0: the straddling document
      rowlo[i] = st == 0 ? s_first : ro + st;
    }
    at += __popc(m);
    if (m) cur = i0 + 31 - __clz(m);
  }
  for (int i = n_real + tid; i < L; i += nthr) rowlo[i] = -1;  // padding rows
  if (tid == 0) cu_q[n_seg] = n_real;
  __syncthreads();  // cu_q visible to the whole block

  // Each local document id must not occur before its own run. Ids that never fall
  // up to the shard's end cannot, nor ids that rise in the shard from one above
  // every id before it; otherwise every run that starts before the shard's end is
  // compared with the ids of the local segments that start behind it, a warp per
  // run and no barrier between them.
  if (flags & 2) {
    bool open = false;
    if (n_seg > 0) {
      const int id0 = row[ro];
#pragma unroll 8
      for (int p = tid; p < s_first; p += nthr) open |= row[p] >= id0;
      for (int k = tid + 1; k < n_seg; k += nthr) open |= row[ro + cu_q[k]] <= row[ro + cu_q[k - 1]];
    }
    if (!__syncthreads_or(open)) flags &= ~2;
  }
  if (flags & 2) {
    bool hit = false;
    const int e = ro + n_real;
    for (int p0 = warp * 32; p0 < e; p0 += n_warps * 32) {
      const int p = p0 + lane, c = p < e ? row[p] : 0;
      unsigned m = __ballot_sync(0xffffffffu, p < e && (p == 0 || c != row[p - 1]));
      if (m == 0) continue;
      // With many segments from the first one on that does not start before these 32
      // positions (finding it is a chain of loads: with 128 segments 34 us for 25, with
      // 4096 890 for 1,615).
      int k0 = 0, k1 = n_seg > 512 ? n_seg : 0;
      while (k0 < k1) {
        const int mid = (k0 + k1) >> 1;
        if ((mid == 0 ? s_first : ro + cu_q[mid]) < p0) k0 = mid + 1; else k1 = mid;
      }
      for (; m; m &= m - 1) {
        const int q = p0 + __ffs(m) - 1, id = __shfl_sync(0xffffffffu, c, __ffs(m) - 1);
#pragma unroll 4
        for (int k = k0 + lane; k < n_seg; k += 32)
          hit |= q < (k == 0 ? s_first : ro + cu_q[k]) && row[ro + cu_q[k]] == id;
      }
    }
    bad |= __syncthreads_or(hit);
  }

  // cu_k and the maxima.
  const int real_end = ro + n_real;
  int mq = 0, mk = 0, mt = 0;
  for (int k = tid; k < n_seg; k += nthr) {
    const int q0 = cu_q[k], q1 = cu_q[k + 1];
    const int st = (k == 0) ? s_first : ro + q0;
    cu_k[k] = st - s_first;
    const int sq = q1 - q0, sk = ro + q1 - st;
    mq = max(mq, sq);
    mk = max(mk, sk);
    if (k >= 1) mt = max(mt, sq);
  }
  mq = __reduce_max_sync(0xffffffffu, mq);
  mk = __reduce_max_sync(0xffffffffu, mk);
  mt = __reduce_max_sync(0xffffffffu, mt);
  __syncthreads();
  if (lane == 0) {
    s_w[0][warp] = mq;
    s_w[1][warp] = mk;
    s_w[2][warp] = mt;
  }
  __syncthreads();
  if (warp != 0) return;
  mq = __reduce_max_sync(0xffffffffu, lane < n_warps ? s_w[0][lane] : 0);
  mk = __reduce_max_sync(0xffffffffu, lane < n_warps ? s_w[1][lane] : 0);
  mt = __reduce_max_sync(0xffffffffu, lane < n_warps ? s_w[2][lane] : 0);

  if (tid == 0) {
    cu_k[n_seg] = real_end - s_first;
    // the first row's sinks are needed too (a no-op without a window)
    const int need_lo = n_real == 0 ? ro : g.n_sink > 0 ? s_first : row_lo_window(s_first, ro, g.window);
    // a chunk of the K/V range need not hold every key the rows may attend
    const int kv_bad = !kv_chunk && n_real > 0 && (need_lo < g.kv_offset || real_end > g.kv_offset + g.S_kv);
    const int row_status = (bad ? BD_STATUS_LAYOUT : 0) | (kv_bad ? BD_STATUS_KV_RANGE : 0);
    hdr[BD_SEG_N_REAL] = n_real;
    hdr[BD_SEG_N_SEG] = n_seg;
    hdr[BD_SEG_S_FIRST] = s_first;
    hdr[BD_SEG_REAL_END] = real_end;
    hdr[BD_SEG_MAX_Q] = mq;
    hdr[BD_SEG_MAX_K] = mk;
    hdr[BD_SEG_FIRST_Q] = n_seg >= 1 ? cu_q[1] : 0;
    hdr[BD_SEG_FIRST_K] = n_seg >= 2 ? ro + cu_q[1] - s_first : (n_seg == 1 ? real_end - s_first : 0);
    hdr[BD_SEG_MAX_TAIL] = mt;
    hdr[BD_SEG_KV_NEED_LO] = need_lo;
    hdr[BD_SEG_ROW_STATUS] = row_status;
    for (int x = 11; x < kHdrRowOffset; ++x) hdr[x] = 0;
    hdr[kHdrRowOffset] = ro;
    hdr[kHdrL] = L;
    hdr[kHdrKvOffset] = g.kv_offset;
    hdr[kHdrSkv] = g.S_kv;
    hdr[kHdrWindow] = g.window;
    hdr[kHdrSfull] = g.S_full;
    hdr[kHdrKvChunk] = kv_chunk;
    hdr[kHdrMagic] = kSegMagic;
    hdr[kHdrSink] = g.n_sink;
    hdr[kHdrSinkTab] = g.sink_tab;
    const int cut[4] = {g.B, g.G, g.sk_units, g.sk_rows};
    for (int x = kHdrSinkTab + 1; x < BD_SEG_HDR_WORDS; ++x)
      hdr[x] = g.sink_tab && x >= kHdrSinkCut ? cut[x - kHdrSinkCut] : 0;
    if (row_status) atomicOr(status, row_status);
  }
}

// The backward's units of a sink table (one CTA; see common.cuh), longest
// first; partial slots numbered in tile order, so the order in which the last
// kernel adds them does not depend on the run. s_hist: nbins ints of histogram.
__device__ void build_sink_units(const Geom& g, int32_t* __restrict__ seg, int nbins, int32_t* status, int* s_hist,
                                 int* s_red) {
  const int tid = threadIdx.x, nthr = blockDim.x;
  int32_t* hdr = seg + g.sk_off;
  int32_t* units = hdr + kSinkHdrWords;
  int32_t* sums = units + static_cast<size_t>(g.sk_units) * kSinkUnitWords;
  const int n_items = g.B * g.nkt, span = g.sk_split * kTile;
  const int hs = cdiv(g.G, g.sk_heads);
  // units of a tile: rows [beg, end0), then pieces of `span` up to end, each for every
  // group of sk_heads heads; returns their number
  auto ranges = [&](int item, int* beg, int* end0, int* end, int* rbase) -> int {
    const int b = item / g.nkt, kt = item % g.nkt;
    int wb, we, sb, se;
    window_tile_rows(g, seg, b, kt, &wb, &we);
    sink_tile_rows(g, seg, b, kt, &sb, &se, rbase);
    if (wb >= we) {
      wb = sb;
      we = sb;
    } else if (sb < se) {
      wb = min(wb, sb);
    }
    *beg = wb;
    *end = max(we, se);
    if (*beg >= *end) return 0;
    const int first = (wb / kTile) * kTile + span;
    if (g.sk_fine) *rbase = 0;
    *end0 = min(*end, g.sk_fine ? first : max(first, cdiv(we, kTile) * kTile));
    return (1 + cdiv(*end - *end0, span)) * hs;
  };
  // unit x of the tile: rows [*ub, *ue), the group's heads [*h0, *h0 + *nh); returns its bin
  auto unit_of = [&](int x, int beg, int end0, int end, int* ub, int* ue, int* h0, int* nh) -> int {
    const int y = x / hs;
    *ub = y == 0 ? beg : end0 + (y - 1) * span;
    *ue = y == 0 ? end0 : min(end, end0 + y * span);
    *h0 = (x % hs) * g.sk_heads;
    *nh = min(g.sk_heads, g.G - *h0);
    return nbins - 1 - min((*ue - 1) / kBwdQ - *ub / kBwdQ + 1, nbins - 1);
  };
  for (int x = tid; x < nbins; x += nthr) s_hist[x] = 0;
  __syncthreads();
  int n_units = 0;
  for (int item = tid; item < n_items; item += nthr) {
    int beg, end0, end, rbase;
    const int n = ranges(item, &beg, &end0, &end, &rbase);
    for (int x = 0; x < n; ++x) {
      int ub, ue, h0, nh;
      atomicAdd(&s_hist[unit_of(x, beg, end0, end, &ub, &ue, &h0, &nh)], 1);
    }
    n_units += n;
  }
  n_units = block_add(n_units, s_red);
  int carry = 0;  // exclusive scan of the histogram, in chunks of blockDim
  for (int c0 = 0; c0 < nbins; c0 += nthr) {
    const int x = c0 + tid;
    const int v = x < nbins ? s_hist[x] : 0;
    int tot;
    const int ex = block_exclusive_scan(v, s_red, &tot);
    __syncthreads();
    if (x < nbins) s_hist[x] = carry + ex;
    carry += tot;
    __syncthreads();
  }
  int n_sums = 0, n_slots = 0;
  bool over = n_units > g.sk_units;
  for (int c0 = 0; c0 < n_items; c0 += nthr) {
    const int item = c0 + tid;
    int beg = 0, end0 = 0, end = 0, rbase = 0, n = 0;
    if (item < n_items) n = ranges(item, &beg, &end0, &end, &rbase);
    const int multi = n > 1;
    int tot_sums, tot_slots;
    const int sum = n_sums + block_exclusive_scan(multi, s_red, &tot_sums);
    const int slot0 = n_slots + block_exclusive_scan(multi ? n : 0, s_red, &tot_slots);
    if (multi && (sum >= g.sk_sums || slot0 + n > g.sk_slots)) over = true;
    if (multi && sum < g.sk_sums) {
      int32_t* e = sums + static_cast<size_t>(sum) * kSinkSumWords;
      e[0] = item;
      e[1] = slot0;
      e[2] = n;
      e[3] = rbase;
    }
    for (int x = 0; x < n; ++x) {
      int ub, ue, h0, nh;
      const int pos = atomicAdd(&s_hist[unit_of(x, beg, end0, end, &ub, &ue, &h0, &nh)], 1);
      if (pos >= g.sk_units) continue;
      int32_t* u = units + static_cast<size_t>(pos) * kSinkUnitWords;
      u[0] = item;
      u[1] = ub;
      u[2] = ue;
      u[3] = x == 0;
      u[4] = multi ? slot0 + x : -1;
      u[5] = rbase;
      u[6] = h0;
      u[7] = nh;
    }
    n_sums += tot_sums;
    n_slots += tot_slots;
  }
  over = __syncthreads_or(over ? 1 : 0) != 0;
  if (tid == 0) {
    // an overflow would be an error of the capacities: nothing is run on the table
    hdr[0] = over ? -1 : n_units;
    hdr[1] = over ? -1 : n_sums;
    hdr[2] = n_slots;
    for (int x = 3; x < kSinkHdrWords; ++x) hdr[x] = 0;
    if (over) atomicOr(status, BD_STATUS_BOUNDS);
  }
}

// Items (n of them, key(item) in [0, nbins)) in descending order of their keys:
// a counting sort, the order within a key left open.
template <class Key>
__device__ void list_longest_first(int n, int nbins, Key key, int32_t* out, int* s_hist, int* s_red) {
  const int tid = threadIdx.x, nthr = blockDim.x;
  for (int x = tid; x < nbins; x += nthr) s_hist[x] = 0;
  __syncthreads();
  for (int it = tid; it < n; it += nthr) atomicAdd(&s_hist[nbins - 1 - min(key(it), nbins - 1)], 1);
  __syncthreads();
  int carry = 0;  // exclusive scan of the histogram, in chunks of blockDim
  for (int c0 = 0; c0 < nbins; c0 += nthr) {
    const int x = c0 + tid;
    const int v = x < nbins ? s_hist[x] : 0;
    int tot;
    const int ex = block_exclusive_scan(v, s_red, &tot);
    if (x < nbins) s_hist[x] = carry + ex;
    carry += tot;
  }
  __syncthreads();
  for (int it = tid; it < n; it += nthr) out[atomicAdd(&s_hist[nbins - 1 - min(key(it), nbins - 1)], 1)] = it;
}

// CTA 0 classifies the q tiles (their K/V tiles, the full ones, the forward's
// longest-first list), CTA 1 the K/V tiles (their q rows, the backward's list);
// CTA 2, launched for sink tables, lists the backward's units. None needs
// anything of the others'. Dynamic shared memory: nbins ints of histogram.
__global__ void __launch_bounds__(1024) classify_kernel(Geom g, int32_t* __restrict__ seg, int nbins,
                                                        int32_t* status) {
  pdl_begin();
  extern __shared__ int s_hist[];
  __shared__ int s_red[32];
  if (blockIdx.x == 2) {
    build_sink_units(g, seg, nbins, status, s_hist, s_red);
    return;
  }
  const int tid = threadIdx.x, nthr = blockDim.x;
  const int ro = g.row_offset, W = g.window;
  int32_t* counts = seg + g.off[BD_SEG_OFF_COUNTS];

  if (blockIdx.x == 0) {
    // Per q tile: the range of K/V tiles and which of them are full.
    int n_full = 0, n_part = 0;
    const int n_items = g.B * g.nqt;
    for (int item = tid; item < n_items; item += nthr) {
      const int b = item / g.nqt, qt = item % g.nqt, first = qt * kTile;
      const int n_real = seg[g.off[BD_SEG_OFF_HDR] + b * BD_SEG_HDR_WORDS + BD_SEG_N_REAL];
      const int32_t* rowlo = seg + g.off[BD_SEG_OFF_ROW_LO] + b * g.L;
      int32_t* qk = seg + g.off[BD_SEG_OFF_QT_KRANGE] + 2 * item;
      int32_t* bits = seg + g.off[BD_SEG_OFF_FULL_BITS] + item * g.nkw;
      int kt_lo = 0, kt_hi = -1, f_lo = 0, f_hi = -1;  // f: the full tiles, an interval
      if (first < n_real) {
        const int last = min(first + kTile - 1, n_real - 1);
        const int j_lo = max(row_lo_window(rowlo[first], ro + first, W) - g.kv_offset, 0);
        const int j_hi = min(ro + last - g.kv_offset, g.S_kv - 1);
        if (j_lo <= j_hi) {
          kt_lo = j_lo / kTile;
          kt_hi = j_hi / kTile;
          if (first + kTile - 1 < n_real) {  // every row is real
            // the tile starts at or behind the last row's first key and ends at or before the first row
            const int a = max(row_lo_window(rowlo[last], ro + last, W) - g.kv_offset, 0);
            const int e = min(ro + first - g.kv_offset + 1, g.S_kv);  // keys [a, e)
            f_lo = max(kt_lo, cdiv(a, kTile));
            f_hi = min(kt_hi, (e > 0 ? e / kTile : 0) - 1);
          }
          const int full = max(0, f_hi - f_lo + 1);
          n_full += full;
          n_part += kt_hi - kt_lo + 1 - full;
        }
      }
      for (int w = 0; w < g.nkw; ++w) {
        const int x = max(f_lo - 32 * w, 0), y = min(f_hi - 32 * w, 31);
        bits[w] = x <= y ? static_cast<int32_t>((0xffffffffu >> (31 - y)) & (0xffffffffu << x)) : 0;
      }
      qk[0] = kt_lo;
      qk[1] = kt_hi;
    }
    n_full = block_add(n_full, s_red);
    n_part = block_add(n_part, s_red);
    if (tid == 0) {
      counts[0] = n_full;
      counts[1] = n_part;
      counts[2] = g.B * g.nqt * g.nkt - n_full - n_part;
      for (int x = 4; x < 8; ++x) counts[x] = 0;
    }
    __syncthreads();  // ranges written above are read below by other threads
    list_longest_first(n_items, nbins, [&](int item) {
      const int32_t* qk = seg + g.off[BD_SEG_OFF_QT_KRANGE] + item * 2;
      int key = qk[1] >= qk[0] ? qk[1] - qk[0] + 1 : 0;
      if (g.n_sink > 0) {
        const int b = item / g.nqt;
        int x0, nx, col[2];
        sink_passes(g, seg[g.off[BD_SEG_OFF_ROW_LO] + b * g.L + item % g.nqt * kTile], item % g.nqt,
                    seg[g.off[BD_SEG_OFF_HDR] + b * BD_SEG_HDR_WORDS + BD_SEG_N_REAL], &x0, &nx, col);
        key += nx;
      }
      return key;
    }, seg + g.off[BD_SEG_OFF_FWD_WORK], s_hist, s_red);
    return;
  }

  // Per K/V tile: the local q rows whose allowed keys meet it.
  int n_kv_att = 0;
  const int n_items = g.B * g.nkt;
  for (int item = tid; item < n_items; item += nthr) {
    const int b = item / g.nkt, kt = item % g.nkt;
    int32_t* kq = seg + g.off[BD_SEG_OFF_KT_QRANGE] + 2 * item;
    int wb, we, sb, se, rbase;
    window_tile_rows(g, seg, b, kt, &wb, &we);
    if (g.n_sink > 0) {
      sink_tile_rows(g, seg, b, kt, &sb, &se, &rbase);
      if (sb < se) {
        wb = wb < we ? min(wb, sb) : sb;
        we = max(we, se);
      }
    }
    kq[0] = wb;
    kq[1] = we;
    n_kv_att += wb < we ? 1 : 0;
  }
  n_kv_att = block_add(n_kv_att, s_red);
  if (tid == 0) counts[3] = n_kv_att;  // these K/V tiles lead the backward work list
  __syncthreads();
  list_longest_first(n_items, nbins, [&](int item) {
    const int32_t* kq = seg + g.off[BD_SEG_OFF_KT_QRANGE] + item * 2;
    return kq[1] > kq[0] ? (kq[1] - 1) / kBwdQ - kq[0] / kBwdQ + 1 : 0;
  }, seg + g.off[BD_SEG_OFF_BWD_WORK], s_hist, s_red);
}

cudaError_t launch_seg_build(const int32_t* doc, const Geom& g, int32_t* seg, int32_t* status, cudaStream_t st,
                             int kv_chunk) {
  // blocks no wider than their work: a barrier of 8 warps is cheaper than one of 32
  auto threads = [](long long items) {
    int n = 128;
    while (n < 1024 && n < items) n *= 2;
    return dim3(n);
  };
  if (const cudaError_t le = launch_pdl(seg_build_kernel, dim3(g.B), threads(g.S_full / 8), 0, st, doc, g, seg, status,
                                        kv_chunk);
      le != cudaSuccess) return le;
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  // histogram bins of the work-list sort: 48 KB of shared memory at most, the
  // kernel's static words included (longer items share the last bin)
  int nbins = (g.nkt > cdiv(g.L, kBwdQ) ? g.nkt : cdiv(g.L, kBwdQ)) + 1;
  if (nbins > 12288 - 64) nbins = 12288 - 64;
  const int widest = g.nkt > g.nqt ? g.nkt : g.nqt;
  if (const cudaError_t le = launch_pdl(classify_kernel, dim3(g.sink_tab ? 3 : 2),
                                        threads(static_cast<long long>(g.B) * widest),
                                        static_cast<size_t>(nbins) * 4, st, g, seg, nbins, status);
      le != cudaSuccess) return le;
  return cudaGetLastError();
}

}  // namespace bd
