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

// Decode: CTAs, warps per CTA, keys per warp step and query heads per CTA.
constexpr int kDecWarps = 4;
constexpr int kDecKeys = 16;
__host__ __device__ inline int dec_ctas(int D) { return D <= 256 ? 2 * kSms : kSms; }
__host__ __device__ inline int dec_head_tiles(int D, int G) { return D <= 256 && G > 8 ? 2 : 1; }
// Whether a CTA takes whole rows, by the most keys that the table's capacity and
// the window let a new token see (the lengths are on the device): few, or not
// very many and there are rows for most SMs.
__host__ __device__ inline bool dec_whole_rows(const PagedGeom& g) {
  long long n = static_cast<long long>(g.max_pages) * g.page_size;
  if (g.window > 0 && n > static_cast<long long>(g.window) + g.n_sink) n = static_cast<long long>(g.window) + g.n_sink;
  if (g.D > 256) return n <= 128;
  const int heads = 8 * dec_head_tiles(g.D, g.G);
  const long long rows = static_cast<long long>(g.B) * g.Hkv * ((g.G + heads - 1) / heads);
  return n <= 512 || (n <= 2048 && rows >= 128);
}
constexpr size_t kDecNoWorkspace = 16;  // what the size query answers then: nothing is kept there
// Workspace: per CTA a descriptor (8 ints), then two partials of (m, l) and O
// for each of its heads.
__host__ __device__ inline size_t dec_desc_bytes(int D) { return static_cast<size_t>(dec_ctas(D)) * 32; }
__host__ __device__ inline size_t dec_part_floats(int D, int heads) { return static_cast<size_t>(heads) * (D + 4); }

}  // namespace bd
