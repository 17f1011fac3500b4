// Geometry of the paged cache as its kernels see it.
#pragma once

#include <cstdint>

#include "common.cuh"

namespace bd {

struct PagedGeom {
  int B, Hq, Hkv, D, G;
  int n_pages, page_size, max_pages;
  int page_shift;  // log2 of page_size, or -1 when it is no power of two
  int window, n_sink;
  float scale;
};

// The rotation of new queries and keys, and how their rows lie.
struct RopeGeom {
  int rot, adjacent, n_pos;
  long long q_stride, k_stride, v_stride;  // 16-byte pieces from a token's row to the next one's
};

// A cache held in 4 bits (cache row r: D / 2 bytes of codes, D / 16 block scales).
struct Cache4 {
  uint8_t *k_codes, *v_codes, *k_blocks, *v_blocks;
  float k_gain, v_gain;
};

// A page id of the table, or -1 for one that names no page.
__device__ __forceinline__ int page_of(const PagedGeom& g, const int32_t* table, int b, int pos, int* off) {
  const int pi = g.page_shift >= 0 ? pos >> g.page_shift : pos / g.page_size;
  *off = pos - pi * g.page_size;
  return table[static_cast<size_t>(b) * g.max_pages + pi];
}

// Row of (page, kv head, token) in the cache; below 2^31 by the host's checks.
__device__ __forceinline__ uint32_t page_row(const PagedGeom& g, int page, int hk, int off) {
  return (static_cast<uint32_t>(page) * g.Hkv + hk) * g.page_size + off;
}

constexpr uint32_t kNoRow = 0xffffffffu;  // no place in the cache

// Token t of the ragged tokens whose offsets are cu [B + 1]: sequence a's are
// [cu[a], cu[a + 1]), its last ones, up to position seq_lens[a] - 1. Gives the
// token's position (-1: t is no token of a) and the cache row of kv head 0 (kNoRow:
// none, because the table names no page). True where something is out of range;
// then there is no position and no row. cu may hold anything.
__device__ __forceinline__ bool token_place(const PagedGeom& g, const int32_t* cu, const int32_t* seq_lens,
                                            const int32_t* page_table, int a, int t, int n_tokens, int* pos_out,
                                            uint32_t* row) {
  *pos_out = -1;
  *row = kNoRow;
  const int begin = cu[a], end = cu[a + 1];
  if (t < begin || t >= end) return false;
  // among offsets that fall, a range that reaches past all new tokens is no
  // sequence's: its tokens would go to places of earlier ones
  const long long pos = static_cast<long long>(seq_lens[a]) - (static_cast<long long>(end) - t);
  if (begin < 0 || end > min(cu[g.B], n_tokens) || pos < 0 || pos >= static_cast<long long>(g.max_pages) * g.page_size)
    return true;
  int off;
  const int page = page_of(g, page_table, a, static_cast<int>(pos), &off);
  if (page != -1 && (page < 0 || page >= g.n_pages)) return true;
  if (page != -1) *row = page_row(g, page, 0, off);  // -1: no page, the token is not kept
  *pos_out = static_cast<int>(pos);
  return false;
}

// Decode: CTAs, warps per CTA, keys per warp step and query heads per CTA.
constexpr int kDecWarps = 4;
constexpr int kDecKeys = 16;
__host__ __device__ inline int dec_ctas(int D) { return D <= 256 ? 2 * kSms : kSms; }
__host__ __device__ inline int dec_head_tiles(int D, int G) { return D <= 256 && G > 8 ? 2 : 1; }
// Whether a CTA takes whole rows, by the most keys that the table's capacity and
// the window let a new token see (the lengths are on the device): few, or not
// very many and there are rows for most SMs.
__host__ __device__ inline long long most_visible(const PagedGeom& g) {
  const long long n = static_cast<long long>(g.max_pages) * g.page_size;
  const long long w = static_cast<long long>(g.window) + g.n_sink;
  return g.window > 0 && n > w ? w : n;
}
__host__ __device__ inline bool dec_whole_rows(const PagedGeom& g) {
  const long long n = most_visible(g);
  if (g.D > 256) return n <= 128;
  const int heads = 8 * dec_head_tiles(g.D, g.G);
  const long long rows = static_cast<long long>(g.B) * g.Hkv * ((g.G + heads - 1) / heads);
  return n <= 512 || (n <= 2048 && rows >= 128);
}
// The same over 4-bit pages, whose steps cost a CTA by their bytes: keys count D / 128
// times from D 128 on. In us, whole and cut: 8 rows of 608 keys at D 128 6.4 and 8.4, of
// 1,024 8.0 and 8.4; at D 256 9.9 and 9.1, 13.9 and 9.3; at D 512 256 keys 8.8 and 10.7.
// 128 rows of 2,048 at D 128 14.4 and 19.4 (ragged 14.0 and 16.4), of 4,096 24.2 and 26.1
// (23.6 and 19.0); of 1,024 at D 256 15.1 and 19.7 (14.5 and 16.5). The limit is one for
// ragged rows. Rows that a window shorter than all sequences makes equally long would be
// faster whole beyond it: 128 rows at D 128 with a window of 2,560 17.4 and 21.4, of 4,096
// 25.0 and 26.3, at D 256 of 1,280 18.4 and 20.9, of 2,048 26.8 and 26.8.
__host__ __device__ constexpr int dec4_ctas(int D, int nt) {
  return D * nt <= 128 || (D == 256 && nt == 1) ? 2 * kSms : kSms;
}
__host__ __device__ inline bool dec4_whole_rows(const PagedGeom& g) {
  const long long n = most_visible(g) * (g.D > 128 ? g.D / 128 : 1);
  const int heads = 8 * dec_head_tiles(g.D, g.G);
  const long long rows = static_cast<long long>(g.B) * g.Hkv * ((g.G + heads - 1) / heads);
  return n <= 1024 || (n <= 2176 && rows >= 128);  // (a window of 1024 and sinks at D 256)
}
constexpr size_t kDecNoWorkspace = 16;  // what the size query answers then: nothing is kept there
// Workspace: per CTA a descriptor (8 ints), then two partials of (m, l) and O
// for each of its heads.
__host__ __device__ inline size_t dec_desc_bytes(int D) { return static_cast<size_t>(dec_ctas(D)) * 32; }
__host__ __device__ inline size_t dec4_desc_bytes(int D, int nt) { return static_cast<size_t>(dec4_ctas(D, nt)) * 32; }
__host__ __device__ inline size_t dec_part_floats(int D, int heads) { return static_cast<size_t>(heads) * (D + 4); }

}  // namespace bd
