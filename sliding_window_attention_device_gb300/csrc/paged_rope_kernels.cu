// New tokens rotated by their position on the way into the paged cache, in bf16 or
// in 4 bits, and cached 4-bit tokens read back as bf16 rows.
//
// A pair (a, b) of a head's first rot numbers turns by its position's angle:
// a' = a c - b s, b' = b c + a s, with c and s from row pos of a table. Every
// operation is rounded by itself (no fused multiply-add), so that the 4-bit codes,
// which jump at the borders between two of them, are those of the same formula
// written out in 32-bit steps.
//
// Bytes bound the large calls: everything is read and written once, whole sectors by
// neighbouring threads. In front of them is a chain of small loads (offsets, length, page)
// that finds where a token goes: one warp per CTA runs it, 32 offsets a trip, while the
// CTA's first pieces of q, k and v are already on their way, and a CTA takes up to 32
// tokens: into bf16 pages as many as let all CTAs be on the SMs at once, up to 38,912
// tokens; the others below are several waves. 13,800 tokens of 32 + 2 x 8 heads, D 128, 340 MB:
// 57 us, 5.9 TB/s (of a plain copy's 6.6 in the same run); without the rotation 55. 64
// single tokens 3.5 us, 3 of them that chain and a launch. Threads in flight count for more
// than loads of a thread: two heads at a time at 64 registers 58 us, three at 80 64.
//   Into 4 bits, keys and values cost instructions rather than bytes: 13,500 tokens of
// 2 x 8 heads alone 22 us for 71 MB (17 without the rotation), with 32 query heads 55 us
// for 292 MB. They have CTAs of their own, in front (among those of the queries 57 to 61,
// the queries in the same CTAs 70).
//   Reading back is bound by the rows written: 55,700 tokens, 8 heads, 292 MB 48 us, 6.1
// TB/s; 16 numbers a thread, in two stores 32 bytes apart, 63; 16 CTAs per SM, one wave,
// instead of 64 of fewer tokens 58, as few waves end unevenly.
#include <cuda_bf16.h>
#include <cstdint>

#include "fp4.cuh"
#include "paged.cuh"
#include "sm100_ptx.cuh"

namespace bd {
namespace {

constexpr int kRopeThreads = 128;
constexpr int kRopeCtas = 8;   // of the append, on an SM at once
constexpr int kRopeTok = 32;   // tokens of a CTA at most
constexpr int kReadBatch = 2;  // pieces that a thread has in flight

__device__ __forceinline__ void unpack8(const uint4& u, float (&x)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                    pack_bf16x2(x[6], x[7]));
}
__device__ __forceinline__ void load8(const float* p, float (&x)[8]) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}
__device__ __forceinline__ void load4(const float* p, float* x) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p));
  x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
}
__device__ __forceinline__ float turn_a(float a, float b, float c, float s) {
  return __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
}
__device__ __forceinline__ float turn_b(float a, float b, float c, float s) {
  return __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
}

// The sequence of token t among offsets cu: the last one that starts at or before
// it. The whole warp asks: 32 offsets a trip.
__device__ __forceinline__ int warp_find_sequence(const int32_t* cu, int B, int t) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = B;
  while (n > 1) {
    const int step = (n + 31) / 32, x = lane * step;
    const unsigned yes = __ballot_sync(0xffffffffu, x < n && cu[lo + x] <= t);
    const int k = max(__popc(yes) - 1, 0) * step;
    lo += k;
    n = min(step, n - k);
  }
  return lo;
}

// Positions (-1: no token, or one out of range) and cache rows of a CTA's tokens.
struct Tokens {
  int pos[kRopeTok];
  uint32_t row[kRopeTok];
  int skip;
};
// Warp 0 finds the sequences of the CTA's first and last token, then lane i token i's
// place; ends with a barrier.
__device__ __forceinline__ void find_tokens(const PagedGeom& g, const int32_t* cu, const int32_t* seq_lens,
                                            const int32_t* page_table, int n_tokens, int tok, int cta, int n_pos,
                                            Tokens* s, int32_t* status) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, t0 = cta * tok;
  if (warp == 0) {
    if (lane == 0) s->skip = *reinterpret_cast<const volatile int*>(status) != 0;
    int a = 0, e = 0;
    if (t0 < n_tokens) {
      a = warp_find_sequence(cu, g.B, t0);
      e = tok == 1 ? a : warp_find_sequence(cu, g.B, min(t0 + tok, n_tokens) - 1);
    }
    const int t = t0 + lane;
    int pos = -1;
    uint32_t row = kNoRow;
    if (lane < tok && t < n_tokens) {
      while (a < e) {
        const int mid = (a + e + 1) >> 1;
        if (cu[mid] <= t) a = mid; else e = mid - 1;
      }
      bool bad = token_place(g, cu, seq_lens, page_table, a, t, n_tokens, &pos, &row);
      if (pos >= n_pos) {
        bad = true;
        pos = -1;
      }
      if (bad) atomicOr(status, BD_STATUS_BOUNDS);
    }
    if (lane < kRopeTok) {
      s->pos[lane] = pos;
      s->row[lane] = row;
    }
  } else if (blockIdx.x == 0) {  // the offsets as a whole: from 0, never falling, to n_tokens at most
    const int x0 = threadIdx.x - 32;
    bool bad = x0 == 0 && (cu[0] != 0 || cu[g.B] > n_tokens);
    for (int x = x0; x < g.B; x += kRopeThreads - 32) bad |= cu[x + 1] < cu[x];
    if (bad) atomicOr(status, BD_STATUS_BOUNDS);
  }
  __syncthreads();
}

// What a thread has of a token's heads: head h of token i, and on to the next one that
// its threads (of one place in the head) take.
struct Item {
  int i, h;
  __device__ __forceinline__ void go(int by, int H) {
    h += by;
    while (h >= H) {
      h -= H;
      ++i;
    }
  }
};

// Heads that stay bf16: the queries, and (kKv) keys and values. A head is D / 16 items
// of two 16-byte pieces; in the rotated part an item holds the two pieces that turn
// against each other (pairs in two halves), elsewhere two pieces half the part apart, so
// that neighbouring threads touch neighbouring pieces. A thread keeps its item's place in
// the head, and so its cosines and sines, over all heads of a token; its first item is on
// its way before the tokens' places are known, the next one while one is worked on.
template <bool kKv>
__device__ __forceinline__ void rope_heads(const uint4* q_new, const uint4* k_new, const uint4* v_new,
                                           const float* cos_sin, const RopeGeom& r, const int32_t* cu_new,
                                           const int32_t* seq_lens, const int32_t* page_table, const PagedGeom& g,
                                           int n_tokens, int tok, int cta, uint4* q_out, uint4* k_out, uint4* k_pages,
                                           uint4* v_pages, Tokens* s, int32_t* status) {
  const int jn = g.D / 16, vpr = g.D / 8, n_r = r.rot / 16, groups = kRopeThreads / jn;
  const int j = threadIdx.x & (jn - 1);
  const int Hq = q_new != nullptr ? g.Hq : 0, Hkv = g.Hkv, H = kKv ? Hq + 2 * Hkv : Hq;
  const bool turns = j < n_r;
  const int p0 = turns ? j : 2 * n_r + (j - n_r), p1 = turns ? j + n_r : p0 + (jn - n_r);
  const int t0 = cta * tok, n_here = min(tok, n_tokens - t0);

  Item at{0, 0};
  at.go(threadIdx.x / jn, H);
  uint4 next0 = make_uint4(0, 0, 0, 0), next1 = next0;
  auto load = [&](const Item& of) {
    if (of.i >= n_here) return;
    const size_t t = static_cast<size_t>(t0) + of.i;
    const uint4* src = !kKv || of.h < Hq ? q_new + t * r.q_stride + of.h * vpr
                       : of.h < Hq + Hkv ? k_new + t * r.k_stride + (of.h - Hq) * vpr
                                         : v_new + t * r.v_stride + (of.h - Hq - Hkv) * vpr;
    next0 = src[p0];
    next1 = src[p1];
  };
  load(at);
  find_tokens(g, cu_new, seq_lens, page_table, n_tokens, tok, cta, r.rot > 0 ? r.n_pos : 0x7fffffff, s, status);
  if (s->skip) return;
  float co[8], si[8];
  int of = -1;  // token that these are of
  for (Item next = at; at.i < n_here; at = next) {
    uint4 x0 = next0, x1 = next1;
    next.go(groups, H);
    load(next);
    const int i = at.i, h = at.h, pos = s->pos[i];
    if (pos < 0) continue;
    const bool is_q = !kKv || h < Hq, is_k = !is_q && h < Hq + Hkv;
    if (turns && (is_q || is_k)) {
      if (of != i) {
        const float* cs = cos_sin + static_cast<size_t>(pos) * r.rot;
        of = i;
        if (!r.adjacent) {
          load8(cs + 8 * j, co);
          load8(cs + r.rot / 2 + 8 * j, si);
        } else {
          load4(cs + 4 * p0, co);
          load4(cs + 4 * p1, co + 4);
          load4(cs + r.rot / 2 + 4 * p0, si);
          load4(cs + r.rot / 2 + 4 * p1, si + 4);
        }
      }
      float a[8], b[8];
      unpack8(x0, a);
      unpack8(x1, b);
      if (!r.adjacent) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float ya = turn_a(a[e], b[e], co[e], si[e]), yb = turn_b(a[e], b[e], co[e], si[e]);
          a[e] = ya;
          b[e] = yb;
        }
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float y0 = turn_a(a[2 * e], a[2 * e + 1], co[e], si[e]);
          const float y1 = turn_b(a[2 * e], a[2 * e + 1], co[e], si[e]);
          const float y2 = turn_a(b[2 * e], b[2 * e + 1], co[4 + e], si[4 + e]);
          const float y3 = turn_b(b[2 * e], b[2 * e + 1], co[4 + e], si[4 + e]);
          a[2 * e] = y0;
          a[2 * e + 1] = y1;
          b[2 * e] = y2;
          b[2 * e + 1] = y3;
        }
      }
      x0 = pack8(a);
      x1 = pack8(b);
    }
    const size_t t = static_cast<size_t>(t0) + i;
    uint4* dst;
    if (is_q) {
      dst = q_out + (t * Hq + h) * vpr;
    } else {
      const int hk = h - Hq - (is_k ? 0 : Hkv);
      if (is_k && k_out != nullptr) {
        uint4* ko = k_out + (t * Hkv + hk) * vpr;
        ko[p0] = x0;
        ko[p1] = x1;
      }
      const uint32_t row = s->row[i];
      if (row == kNoRow) continue;
      dst = (is_k ? k_pages : v_pages) + (static_cast<size_t>(row) + static_cast<size_t>(hk) * g.page_size) * vpr;
    }
    dst[p0] = x0;
    dst[p1] = x1;
  }
}

// Keys and values that become 4 bits. An item is a block of 16 numbers, two
// neighbouring pieces, so that the largest of a block is one thread's; a rotated key's
// partners are read a second time, out of L1. The next item's pieces are on their way
// while one is worked on.
__device__ __forceinline__ void rope_blocks(const uint4* k_new, const uint4* v_new, const float* cos_sin,
                                            const RopeGeom& r, const int32_t* cu_new, const int32_t* seq_lens,
                                            const int32_t* page_table, const PagedGeom& g, int n_tokens, int tok,
                                            int cta, uint4* k_out, const Cache4& c4, Tokens* s, int32_t* status) {
  const int jn = g.D / 16, vpr = g.D / 8, n_r = r.rot / 16, groups = kRopeThreads / jn;
  const int j = threadIdx.x & (jn - 1), Hkv = g.Hkv, H = 2 * Hkv;
  const int t0 = cta * tok, n_here = min(tok, n_tokens - t0);
  // Of my pieces' pairs (halves): how far the partner piece is, whether I am their first
  // number (a' = a c - b s) or their second (b' = b c + a s), and where their cosines are.
  const bool lower0 = 2 * j < n_r, lower1 = 2 * j + 1 < n_r;
  const int pair0 = lower0 ? 2 * j : 2 * j - n_r, pair1 = lower1 ? 2 * j + 1 : 2 * j + 1 - n_r;

  Item at{0, 0};
  at.go(threadIdx.x / jn, H);
  uint4 next0 = make_uint4(0, 0, 0, 0), next1 = next0;
  // keys first in one token, values first in the next: where a warp's heads are the same ones of every token, all
  // warps then have as many keys, which cost more (54.7 us for 55.6)
  auto is_key = [&](const Item& of) { return (of.h < Hkv) == ((of.i & 1) == 0); };
  auto source = [&](const Item& of) {
    const size_t t = static_cast<size_t>(t0) + of.i;
    const int hk = of.h >= Hkv ? of.h - Hkv : of.h;
    return is_key(of) ? k_new + t * r.k_stride + hk * vpr : v_new + t * r.v_stride + hk * vpr;
  };
  auto load = [&](const Item& of) {
    if (of.i >= n_here) return;
    const uint4* src = source(of) + 2 * j;
    next0 = src[0];
    next1 = src[1];
  };
  load(at);
  find_tokens(g, cu_new, seq_lens, page_table, n_tokens, tok, cta, r.rot > 0 ? r.n_pos : 0x7fffffff, s, status);
  if (s->skip) return;
  for (Item next = at; at.i < n_here; at = next) {
    float x[16];
    {
      float a[8], b[8];
      unpack8(next0, a);
      unpack8(next1, b);
#pragma unroll
      for (int z = 0; z < 8; ++z) x[z] = a[z], x[8 + z] = b[z];
    }
    next.go(groups, H);
    load(next);
    const int pos = s->pos[at.i];
    if (pos < 0) continue;
    const bool is_k = is_key(at);
    const int hk = at.h >= Hkv ? at.h - Hkv : at.h;
    if (is_k && j < n_r) {
      const float* cs = cos_sin + static_cast<size_t>(pos) * r.rot;
      if (!r.adjacent) {
        const uint4* src = source(at);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int pair = e == 0 ? pair0 : pair1;
          const bool lower = e == 0 ? lower0 : lower1;
          const float sign = lower ? -1.0f : 1.0f;  // (a product with it is exact)
          float o[8], c[8], sn[8];
          unpack8(src[lower ? pair + n_r : pair], o);
          load8(cs + 8 * pair, c);
          load8(cs + r.rot / 2 + 8 * pair, sn);
#pragma unroll
          for (int z = 0; z < 8; ++z)
            x[8 * e + z] = __fmaf_rn(__fmul_rn(o[z], sn[z]), sign, __fmul_rn(x[8 * e + z], c[z]));
        }
      } else {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float c[4], sn[4];
          load4(cs + 8 * j + 4 * e, c);
          load4(cs + r.rot / 2 + 8 * j + 4 * e, sn);
#pragma unroll
          for (int z = 0; z < 4; ++z) {
            const float a = x[8 * e + 2 * z], b = x[8 * e + 2 * z + 1];
            x[8 * e + 2 * z] = turn_a(a, b, c[z], sn[z]);
            x[8 * e + 2 * z + 1] = turn_b(a, b, c[z], sn[z]);
          }
        }
      }
    }
    if (is_k && k_out != nullptr) {
      uint4* ko = k_out + ((static_cast<size_t>(t0) + at.i) * Hkv + hk) * vpr + 2 * j;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float y[8];
#pragma unroll
        for (int z = 0; z < 8; ++z) y[z] = x[8 * e + z];
        ko[e] = pack8(y);
      }
    }
    const uint32_t row = s->row[at.i];
    if (row == kNoRow) continue;
    uint8_t scale;
    const uint2 codes = block_to_4_bits(x, is_k ? c4.k_gain : c4.v_gain, &scale);  // (the gains' inverses)
    const size_t block = (static_cast<size_t>(row) + static_cast<size_t>(hk) * g.page_size) * jn + j;
    reinterpret_cast<uint2*>(is_k ? c4.k_codes : c4.v_codes)[block] = codes;
    (is_k ? c4.k_blocks : c4.v_blocks)[block] = scale;
  }
}

// bf16 pages: every CTA takes `tok` tokens with all their heads.
__global__ void __launch_bounds__(kRopeThreads, kRopeCtas)
    paged_rope_kernel(const uint4* q_new, const uint4* __restrict__ k_new, const uint4* __restrict__ v_new,
                      const float* __restrict__ cos_sin, const RopeGeom r, const int32_t* __restrict__ cu_new,
                      const int32_t* __restrict__ seq_lens, const int32_t* __restrict__ page_table, const PagedGeom g,
                      int n_tokens, int tok, uint4* q_out, uint4* k_out, uint4* __restrict__ k_pages,
                      uint4* __restrict__ v_pages, int32_t* status) {
  pdl_begin();
  __shared__ Tokens s;
  rope_heads<true>(q_new, k_new, v_new, cos_sin, r, cu_new, seq_lens, page_table, g, n_tokens, tok, blockIdx.x, q_out,
                   k_out, k_pages, v_pages, &s, status);
}

// 4-bit pages: the first kv_ctas CTAs take keys and values, kv_tok tokens each, the
// others queries.
__global__ void __launch_bounds__(kRopeThreads, kRopeCtas)
    paged4_rope_kernel(const uint4* q_new, const uint4* __restrict__ k_new, const uint4* __restrict__ v_new,
                       const float* __restrict__ cos_sin, const RopeGeom r, const int32_t* __restrict__ cu_new,
                       const int32_t* __restrict__ seq_lens, const int32_t* __restrict__ page_table, const PagedGeom g,
                       int n_tokens, int tok, int kv_tok, int kv_ctas, uint4* q_out, uint4* k_out, const Cache4 c4,
                       int32_t* status) {
  pdl_begin();
  __shared__ Tokens s;
  if (static_cast<int>(blockIdx.x) < kv_ctas)
    rope_blocks(k_new, v_new, cos_sin, r, cu_new, seq_lens, page_table, g, n_tokens, kv_tok, blockIdx.x, k_out, c4, &s,
                status);
  else
    rope_heads<false>(q_new, k_new, v_new, cos_sin, r, cu_new, seq_lens, page_table, g, n_tokens, tok,
                      blockIdx.x - kv_ctas, q_out, nullptr, nullptr, nullptr, &s, status);
}

// The last tokens of each sequence, as rows [n_tokens, Hkv, D]. A thread takes 8 numbers
// of K and the same ones of V, 16 bytes of each row written whole by neighbouring threads.
__global__ void __launch_bounds__(kRopeThreads)
    paged4_read_kernel(const Cache4 c4, const int32_t* __restrict__ cu, const int32_t* __restrict__ seq_lens,
                       const int32_t* __restrict__ page_table, const PagedGeom g, int n_tokens, int tok,
                       uint4* __restrict__ k_out, uint4* __restrict__ v_out, int32_t* status) {
  pdl_begin();
  __shared__ Tokens s;
  find_tokens(g, cu, seq_lens, page_table, n_tokens, tok, blockIdx.x, 0x7fffffff, &s, status);
  if (s.skip) return;
  const int vpr = g.D / 8, t0 = blockIdx.x * tok, n_here = min(tok, n_tokens - t0);
  const int p = threadIdx.x & (vpr - 1), groups = kRopeThreads / vpr;
  Item at{0, 0};
  at.go(threadIdx.x / vpr, g.Hkv);
  while (at.i < n_here) {
    uint32_t code[kReadBatch][2], scale[kReadBatch][2];
    Item it[kReadBatch];
#pragma unroll
    for (int u = 0; u < kReadBatch; ++u) {
      it[u] = at;
      code[u][0] = code[u][1] = scale[u][0] = scale[u][1] = 0;
      if (at.i >= n_here) continue;
      const uint32_t row = s.row[at.i];
      if (row != kNoRow) {
        const size_t r = static_cast<size_t>(row) + static_cast<size_t>(at.h) * g.page_size;
        code[u][0] = __ldg(reinterpret_cast<const uint32_t*>(c4.k_codes) + r * vpr + p);
        code[u][1] = __ldg(reinterpret_cast<const uint32_t*>(c4.v_codes) + r * vpr + p);
        scale[u][0] = __ldg(c4.k_blocks + r * (vpr / 2) + p / 2);
        scale[u][1] = __ldg(c4.v_blocks + r * (vpr / 2) + p / 2);
      }
      at.go(groups, g.Hkv);
    }
#pragma unroll
    for (int u = 0; u < kReadBatch; ++u) {
      if (it[u].i >= n_here || s.pos[it[u].i] < 0) continue;
      const size_t dst = ((static_cast<size_t>(t0) + it[u].i) * g.Hkv + it[u].h) * vpr + p;
#pragma unroll
      for (int z = 0; z < 2; ++z) {
        const float by = floats_of(e4m3_values(scale[u][z])).x, gain = z == 0 ? c4.k_gain : c4.v_gain;
        uint32_t w[4];
        e2m1_values(code[u][z], w);
        float f[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 y = floats_of(w[e]);
          f[2 * e] = y.x * by * gain;  // the first product is exact
          f[2 * e + 1] = y.y * by * gain;
        }
        (z == 0 ? k_out : v_out)[dst] = pack8(f);
      }
    }
  }
}

// Tokens a CTA takes, of `items` items each: enough for its threads; and where there are
// more, so many that `share` CTAs per SM are launched, as finding the tokens' places is
// paid per CTA; kRopeTok at most. The append into bf16 pages asks for the 8 that an SM
// holds; the one into 4 bits for 8 of keys and values and 16 of queries, and the read for
// 64, which run in several waves.
int tokens_per_cta(int n_tokens, int items, int share) {
  const int least = (kRopeThreads + items - 1) / items, ctas = kSms * share;
  int tok = (n_tokens - 1) / ctas + 1;
  tok = tok < least ? least : tok;
  return tok > kRopeTok ? kRopeTok : tok;
}
int ctas_of(int n_tokens, int tok) { return n_tokens == 0 ? 1 : (n_tokens - 1) / tok + 1; }
}  // namespace

cudaError_t launch_paged_rope(const void* q_new, const void* k_new, const void* v_new, const float* cos_sin,
                              const RopeGeom& r, const int32_t* cu_new, const int32_t* seq_lens,
                              const int32_t* page_table, const PagedGeom& g, int n_tokens, void* q_out, void* k_out,
                              void* k_pages, void* v_pages, const Cache4* c4, int32_t* status, cudaStream_t st) {
  const uint4 *q = static_cast<const uint4*>(q_new), *k = static_cast<const uint4*>(k_new),
              *v = static_cast<const uint4*>(v_new);
  uint4 *qo = static_cast<uint4*>(q_out), *ko = static_cast<uint4*>(k_out);
  const int Hq = q != nullptr ? g.Hq : 0, jn = g.D / 16;
  cudaError_t le;
  if (c4 == nullptr) {
    const int tok = tokens_per_cta(n_tokens, (Hq + 2 * g.Hkv) * jn, kRopeCtas);
    le = launch_pdl(paged_rope_kernel, dim3(ctas_of(n_tokens, tok)), dim3(kRopeThreads), 0, st, q, k, v, cos_sin, r,
                    cu_new, seq_lens, page_table, g, n_tokens, tok, qo, ko, static_cast<uint4*>(k_pages),
                    static_cast<uint4*>(v_pages), status);
  } else {
    const Cache4 inv{c4->k_codes, c4->v_codes, c4->k_blocks, c4->v_blocks, 1.0f / c4->k_gain, 1.0f / c4->v_gain};
    const int kv_tok = tokens_per_cta(n_tokens, 2 * g.Hkv * jn, kRopeCtas);
    const int tok = Hq > 0 ? tokens_per_cta(n_tokens, Hq * jn, 2 * kRopeCtas) : 1;
    const int kv_ctas = ctas_of(n_tokens, kv_tok), q_ctas = Hq > 0 ? ctas_of(n_tokens, tok) : 0;
    le = launch_pdl(paged4_rope_kernel, dim3(kv_ctas + q_ctas), dim3(kRopeThreads), 0, st, q, k, v, cos_sin, r, cu_new,
                    seq_lens, page_table, g, n_tokens, tok, kv_tok, kv_ctas, qo, ko, inv, status);
  }
  if (le != cudaSuccess) return le;
  return cudaGetLastError();
}

cudaError_t launch_paged4_read(const Cache4& c4, const int32_t* cu, const int32_t* seq_lens, const int32_t* page_table,
                               const PagedGeom& g, int n_tokens, void* k_out, void* v_out, int32_t* status,
                               cudaStream_t st) {
  const int tok = tokens_per_cta(n_tokens, g.Hkv * (g.D / 8), 64);
  const unsigned grid = static_cast<unsigned>(ctas_of(n_tokens, tok));
  if (const cudaError_t le =
          launch_pdl(paged4_read_kernel, dim3(grid), dim3(kRopeThreads), 0, st, c4, cu, seq_lens, page_table, g,
                     n_tokens, tok, static_cast<uint4*>(k_out), static_cast<uint4*>(v_out), status);
      le != cudaSuccess)
    return le;
  return cudaGetLastError();
}

}  // namespace bd
