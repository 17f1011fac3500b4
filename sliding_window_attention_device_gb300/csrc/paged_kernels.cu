// Paged K/V cache: writing new tokens into it, and attention of one new token
// per sequence over it.
//
// The cache holds pages of page_size tokens, [n_pages][Hkv][page_size][D]: the
// keys a kv head reads of a page are one contiguous block. Sequence b's token at
// position s lies in page page_table[b][s / page_size]. The new token, at
// position len - 1, sees key s iff there is no window, or len - 1 - s < window,
// or s < n_sink.
#include <cuda_bf16.h>
#include <cstdint>

#include "paged.cuh"
#include "sm100_ptx.cuh"

namespace bd {

// ------------------------------------------------------------------ append
// One CTA copies `tok` consecutive tokens: the first threads find each token's
// sequence (binary search in cu_new), page and cache row, then all copy
// 16-byte pieces, K and V together. Reads and writes every new element once: the
// bytes bound it. 19,200 tokens of 12 prompts (8 kv heads, D 128, 157 MB in all),
// new data each time: 27 us, 5.8 TB/s; 64 single tokens 3 us, a launch's cost. The
// offsets' check (CTA 0, and each token's own range) costs nothing beside these.
constexpr int kAppendThreads = 256;
constexpr int kAppendTok = 16;

__global__ void __launch_bounds__(kAppendThreads)
    paged_append_kernel(const uint4* __restrict__ k_new, const uint4* __restrict__ v_new,
                        const int32_t* __restrict__ cu_new, const int32_t* __restrict__ seq_lens,
                        const int32_t* __restrict__ page_table, const PagedGeom g, int n_tokens, int tok,
                        uint4* __restrict__ k_pages, uint4* __restrict__ v_pages, int32_t* status) {
  pdl_begin();
  __shared__ uint32_t s_row[kAppendTok];  // cache row of kv head 0, or 0xffffffff: not stored
  __shared__ int s_skip;
  const int t0 = blockIdx.x * tok;
  if (threadIdx.x == 0) s_skip = *reinterpret_cast<const volatile int*>(status) != 0;
  if (blockIdx.x == 0) {  // the offsets as a whole: from 0, never falling, to n_tokens at most
    bool bad = threadIdx.x == 0 && (cu_new[0] != 0 || cu_new[g.B] > n_tokens);
    for (int x = threadIdx.x; x < g.B; x += kAppendThreads) bad |= cu_new[x + 1] < cu_new[x];
    if (bad) atomicOr(status, BD_STATUS_BOUNDS);
  }
  if (threadIdx.x < static_cast<unsigned>(tok)) {
    const int t = t0 + static_cast<int>(threadIdx.x);
    uint32_t row = 0xffffffffu;
    if (t < n_tokens) {
      int a = 0, e = g.B - 1;  // the last sequence that starts at or before t
      while (a < e) {
        const int mid = (a + e + 1) >> 1;
        if (cu_new[mid] <= t) a = mid; else e = mid - 1;
      }
      const int begin = cu_new[a], end = cu_new[a + 1];
      if (begin <= t && t < end) {
        // among offsets that fall, a range that reaches past all new tokens is no
        // sequence's: its tokens would go to places of earlier ones
        const long long pos = static_cast<long long>(seq_lens[a]) - (end - t);
        int bad = begin < 0 || end > min(cu_new[g.B], n_tokens) || pos < 0 ||
                  pos >= static_cast<long long>(g.max_pages) * g.page_size;
        if (!bad) {
          int off;
          const int page = page_of(g, page_table, a, static_cast<int>(pos), &off);
          if (page >= 0 && page < g.n_pages) row = page_row(g, page, 0, off);
          else bad = page != -1;  // -1: no page, the token is not kept
        }
        if (bad) atomicOr(status, BD_STATUS_BOUNDS);
      }
    }
    s_row[threadIdx.x] = row;
  }
  __syncthreads();
  if (s_skip) return;
  const int vpr = g.D / 8, vpt = g.Hkv * vpr;  // 16-byte pieces of a row, of a token
  const int n = min(tok, n_tokens - t0) * vpt;
  const size_t src0 = static_cast<size_t>(t0) * vpt;
#pragma unroll 2
  for (int x = threadIdx.x; x < n; x += kAppendThreads) {
    const int i = x / vpt, y = x - i * vpt, hk = y / vpr;
    const uint32_t row = s_row[i];
    if (row == 0xffffffffu) continue;
    const uint4 kk = __ldg(k_new + src0 + x), vv = __ldg(v_new + src0 + x);
    const size_t dst = (static_cast<size_t>(row) + static_cast<size_t>(hk) * g.page_size) * vpr + (y - hk * vpr);
    k_pages[dst] = kk;
    v_pages[dst] = vv;
  }
}

cudaError_t launch_paged_append(const void* k_new, const void* v_new, const int32_t* cu_new, const int32_t* seq_lens,
                                const int32_t* page_table, const PagedGeom& g, int n_tokens, void* k_pages,
                                void* v_pages, int32_t* status, cudaStream_t st) {
  // a token per CTA until the CTAs fill the machine four times over; then two
  // pieces of K and of V per thread (at 8 kv heads, D 128, 19,200 tokens: 1 token
  // a CTA 33 us, 2 28, 4 27, 8 27.5, 16 29.5)
  int most = 2 * kAppendThreads / (g.Hkv * (g.D / 8));
  most = most < 1 ? 1 : most > kAppendTok ? kAppendTok : most;
  int tok = (n_tokens + 4 * kSms - 1) / (4 * kSms);
  tok = tok < 1 ? 1 : tok > most ? most : tok;
  // (no tokens: one CTA, for the offsets' check)
  const unsigned grid = n_tokens == 0 ? 1u : static_cast<unsigned>((n_tokens - 1) / tok + 1);
  if (const cudaError_t le =
          launch_pdl(paged_append_kernel, dim3(grid), dim3(kAppendThreads), 0, st, static_cast<const uint4*>(k_new),
                     static_cast<const uint4*>(v_new), cu_new, seq_lens, page_table, g, n_tokens, tok,
                     static_cast<uint4*>(k_pages), static_cast<uint4*>(v_pages), status);
      le != cudaSuccess)
    return le;
  return cudaGetLastError();
}

// ------------------------------------------------------------------ decode
// out = softmax(scale q K^T) V of one query row per head over the sequence's
// visible keys. A K or V row is read once for up to 16 query heads of its kv head
// (8 at D 512), so the cache's bytes bound it, not the products. A larger group
// reads the cache again for each such block: 16 sequences of 8,000 keys, 4 kv
// heads, D 128: G 8 39 us, 16 46, 32 74, 64 132.
//
// A (sequence, kv head, block of up to 16 query heads) is a row of work; its
// visible keys, sinks first, then the window, are numbered without a gap and cut
// into steps of 16. The steps of all rows form one line that is dealt out to
// the CTAs in equal pieces, so ragged lengths leave no CTA idle; each warp takes
// every fourth step of a piece:
//   K and V rows gathered with 16-byte cp.async into the warp's own ring of
//   16-key items (K, V, K, V, ...), as many in flight as the ring holds;
//   S^T (16 keys x 8 heads) = K Q^T and O^T (16 d x 8 heads) += V^T P^T by
//   mma.sync m16n8k16: the keys, not the few query heads, are the wide side, a
//   warp's softmax needs no other warp, and no step waits for a barrier. (The
//   tensor rate is not what bounds this: one mma covers 512 bytes of cache.)
//   Softmax statistics and O in fp32. P enters the product as two bf16 numbers,
//   the second of what the first left (off by 2^-16): a second mma on the same V
//   fragments, which the bytes hide. With one number, out is off by 0.0020 to 0.0024
//   over a tensor where its own rounding is 0.0017; at most 6% less time where a
//   CTA's chain is all there is (8 x 500 keys 8.0 us for 8.5), else within 3%.
// Where sequences are short, or not long and rows many (dec_whole_rows), a CTA
// takes a whole row instead: no line, no second kernel. The host decides it, and
// knows the table's capacity and the window but not the lengths: short sequences
// under a large table take the cut line (100 keys, D 64, alone 7.8 us for 4.1;
// 8 kv heads, D 128, 64 x 100 keys 13.0 for 8.6, 64 x 500 22.4 for 19.1). At 1,028
// visible keys (window 1024) and 8 kv heads, D 128: 16 sequences 14.6 us whole, 16.4
// cut; 64 42.5 and 56.3; but 4 sequences 14.0 and 11.1. At 4,100 keys about even, and
// cut pieces are the safer choice for ragged lengths.
// A step's chain (scores, maximum, exponentials, P V) is what bounds a CTA alone:
// so the score products run in four chains, the maximum is raised only when a
// score passes it by 2^8 (one vote instead of three rounds of shuffles), and a
// page id is loaded a step before it is used (D 64, whole rows of 4,100 keys: 48
// -> 34 us). With all SMs at work the cache's bytes bound it: 16 ragged sequences
// up to 32,768 keys, 8 kv heads, D 128, 1.06 GB in 172 us, 6.2 TB/s; one sequence
// of 131,072 keys, 4 kv heads, 268 MB in 51 us (7 us of these start and join).
// Rings of 4 items or 6, 2 or 3 CTAs an SM, 4 or 8 warps a CTA: within 3%.
// At the end of a row's piece the warps join through shared memory. A row
// inside one CTA is written at once; of a row cut over CTAs each leaves (m, l,
// O) in the workspace, and paged_join_kernel adds them in CTA order.
template <int D, int NT>
struct DecCfg {
  static constexpr int kItem = kDecKeys * D * 2;  // bytes of 16 K or V rows
  static constexpr int kItems = D == 64 ? 12 : D == 128 ? 6 : 3;
  static constexpr int kHeads = 8 * NT;
  static constexpr bool kQSmem = D > 128;  // Q fragments in shared memory instead of registers
  static constexpr int kRing = kDecWarps * kItems * kItem;
  static constexpr int kQBytes = kQSmem ? NT * (D / 16) * 32 * 8 : 0;
  static constexpr int kOStride = D + 4;  // fp32 row of a warp's O in its ring (4: no bank conflicts)
  static constexpr int kMl = kDecWarps * kHeads * 8;
  static constexpr int kSmem = kRing + kQBytes + kMl;
  static_assert(kHeads * kOStride * 4 <= kItems * kItem, "a warp's O fits its ring");
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool valid) {
  const int n = valid ? 16 : 0;  // 0: the 16 bytes are set to zero
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The two values of a bf16 pair.
__device__ __forceinline__ float bf16_lo(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t u) { return __uint_as_float(u & 0xffff0000u); }

// The visible keys of a sequence: sinks [0, ns), then [lo, lo + n - ns).
struct Visible {
  int n, ns, lo;
};
__device__ __forceinline__ Visible visible_keys(const PagedGeom& g, const int32_t* seq_lens, int b, bool* bad) {
  Visible v{0, 0, 0};
  const int len = seq_lens[b];
  if (len < 0 || len > static_cast<long long>(g.max_pages) * g.page_size) {
    *bad = true;  // taken as empty
    return v;
  }
  v.lo = g.window > 0 && len > g.window ? len - g.window : 0;
  v.ns = min(g.n_sink, v.lo);
  v.n = len - v.lo + v.ns;
  return v;
}

// What exponents are taken against: the maximum, or 0 where every score so far
// is -inf, whose weights are then 0 and not NaN.
__device__ __forceinline__ float exp_base(float m) { return m == -INFINITY ? 0.f : m; }
// O's factor and the log-sum-exp of a row with maximum m (log2) and sum l: out 0
// and -inf where nothing weighs (l = 0), NaN where a score is.
__device__ __forceinline__ float row_inv(float l) { return l == 0.f ? 0.f : 1.0f / l; }
__device__ __forceinline__ float row_lse(float m, float l) {
  return l == 0.f ? -INFINITY : (m + __log2f(l)) * 0.6931471805599453f;
}

struct DecDesc {  // a row that starts in a CTA's piece and ends in a later one
  int b, hk, hb, slot, last_cta, pad[3];
};

template <int D, int NT>
__global__ void __launch_bounds__(kDecWarps * 32)
    paged_decode_kernel(const __nv_bfloat16* __restrict__ q, const __nv_bfloat16* __restrict__ k_pages,
                        const __nv_bfloat16* __restrict__ v_pages, const int32_t* __restrict__ page_table,
                        const int32_t* __restrict__ seq_lens, const PagedGeom g, int whole_rows,
                        __nv_bfloat16* __restrict__ out, float* __restrict__ lse, DecDesc* __restrict__ desc,
                        float* __restrict__ part, int32_t* status) {
  pdl_begin();
  using C = DecCfg<D, NT>;
  constexpr int kThreads = kDecWarps * 32, kHeads = C::kHeads, kKs = D / 16;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ long long s_sum[kThreads];
  __shared__ int s_b, s_skip;
  __shared__ long long s_at;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int n_hb = (g.G + kHeads - 1) / kHeads, rows_b = g.Hkv * n_hb;

  bool bad = false;
  int b = 0;
  long long per = 1, at = 0, end = 0, in_b = 0;  // steps [at, end) of the line; step of sequence b that `at` is
  if (whole_rows) {
    // ---- one row per CTA
    b = blockIdx.x / rows_b;
    const int row = blockIdx.x % rows_b;
    const Visible v = visible_keys(g, seq_lens, b, &bad);
    if (tid == 0) {  // read once: another CTA may set a bit between two threads' reads
      if (bad) atomicOr(status, BD_STATUS_BOUNDS);
      s_skip = *reinterpret_cast<const volatile int*>(status) != 0;
    }
    __syncthreads();
    if (s_skip) return;
    const int steps = (v.n + kDecKeys - 1) / kDecKeys;
    if (steps == 0) {
      const int heads = min(kHeads, g.G - row % n_hb * kHeads);
      const size_t r0 = static_cast<size_t>(b) * g.Hq + row / n_hb * g.G + row % n_hb * kHeads;
      uint4* o4 = reinterpret_cast<uint4*>(out + r0 * D);
      for (int i = tid; i < heads * (D / 8); i += kThreads) o4[i] = make_uint4(0, 0, 0, 0);
      if (tid < heads) lse[r0 + tid] = -INFINITY;
      return;
    }
    in_b = static_cast<long long>(row) * steps;
    end = steps;
  } else {
    // ---- an equal piece of the line of steps
    // thread t sums the steps of sequences [t * span, (t + 1) * span)
    const int span = (g.B + kThreads - 1) / kThreads;
    long long mine = 0;
    for (int x = tid * span; x < min(g.B, (tid + 1) * span); ++x) {
      const Visible v = visible_keys(g, seq_lens, x, &bad);
      mine += static_cast<long long>((v.n + kDecKeys - 1) / kDecKeys) * rows_b;
    }
    if (bad) atomicOr(status, BD_STATUS_BOUNDS);
    if (tid == 0) s_skip = *reinterpret_cast<const volatile int*>(status) != 0;
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long t = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += t;
    }
    if (lane == 31) s_sum[warp] = incl;
    const bool any_bad = __syncthreads_or(bad) != 0;  // every CTA sees every length: then none writes
    long long total = 0, before = incl - mine;
#pragma unroll
    for (int w = 0; w < kDecWarps; ++w) {
      if (w < warp) before += s_sum[w];
      total += s_sum[w];
    }
    if (tid == 0) desc[blockIdx.x].last_cta = -1;
    if (s_skip || any_bad) return;
    // no fewer than one step per warp
    per = (total + gridDim.x - 1) / gridDim.x;
    if (per < kDecWarps) per = kDecWarps;
    at = per * blockIdx.x;
    end = min(at + per, total);

    // sequences without a visible key: zeros and -inf, shared out over the CTAs
    for (int x = blockIdx.x; x < g.B; x += gridDim.x) {
      bool y = false;
      if (visible_keys(g, seq_lens, x, &y).n > 0) continue;
      uint4* o4 = reinterpret_cast<uint4*>(out + static_cast<size_t>(x) * g.Hq * D);
      for (int i = tid; i < g.Hq * (D / 8); i += kThreads) o4[i] = make_uint4(0, 0, 0, 0);
      for (int i = tid; i < g.Hq; i += kThreads) lse[static_cast<size_t>(x) * g.Hq + i] = -INFINITY;
    }
    if (at >= end) return;
    // the thread whose sequences hold the first step finds the one
    if (at >= before && at < before + mine) {
      long long sum = before;
      int x = tid * span;
      for (;; ++x) {
        const Visible v = visible_keys(g, seq_lens, x, &bad);
        const long long n = static_cast<long long>((v.n + kDecKeys - 1) / kDecKeys) * rows_b;
        if (at < sum + n) break;
        sum += n;
      }
      s_b = x;
      s_at = at - sum;
    }
    __syncthreads();
    b = s_b;
    in_b = s_at;
  }

  uint8_t* ring = smem + warp * C::kItems * C::kItem;
  const uint32_t ring_a = smem_u32(ring);
  uint2* qs = reinterpret_cast<uint2*>(smem + C::kRing);
  float* ml = reinterpret_cast<float*>(smem + C::kRing + C::kQBytes);  // [warp][head] m, l
  const float sl2 = g.scale * 1.4426950408889634f;

  bool first_piece = true;
  while (at < end) {
    const Visible v = visible_keys(g, seq_lens, b, &bad);
    const int steps = (v.n + kDecKeys - 1) / kDecKeys;
    if (in_b >= static_cast<long long>(steps) * rows_b) {
      ++b;
      in_b = 0;
      continue;
    }
    const int row = static_cast<int>(in_b / steps), t0 = static_cast<int>(in_b - static_cast<long long>(row) * steps);
    const int hk = row / n_hb, hb = row % n_hb;
    const int t1 = static_cast<int>(min(static_cast<long long>(steps), t0 + (end - at)));
    const int heads = min(kHeads, g.G - hb * kHeads);  // query heads of this row
    const int h0 = hk * g.G + hb * kHeads;

    // ---- this warp's steps t0 + warp, t0 + warp + 4, ...
    const int n_mine = t1 - t0 > warp ? (t1 - t0 - warp + kDecWarps - 1) / kDecWarps : 0;
    // the page and place of key lane % 16 of my i-th step (-1: no such key); the
    // page is loaded a step before it is looked at
    auto page_at = [&](int i, int* off) -> int {
      const int x = (t0 + warp + i * kDecWarps) * kDecKeys + (lane & 15);
      if (i >= n_mine || x >= v.n) {
        *off = -1;
        return 0;
      }
      return page_of(g, page_table, b, x < v.ns ? x : v.lo + (x - v.ns), off);
    };
    int off_next, page_next = page_at(0, &off_next);
    uint32_t row_cur = 0xffffffffu;  // cache row of that key of the step being copied (0xffffffff: none)
    // item y: K (even) or V (odd) of my step y / 2
    auto issue = [&](int y) {
      if (y < 2 * n_mine) {
        if ((y & 1) == 0) {
          row_cur = 0xffffffffu;
          if (off_next >= 0) {
            if (page_next >= 0 && page_next < g.n_pages) row_cur = page_row(g, page_next, hk, off_next);
            else atomicOr(status, BD_STATUS_BOUNDS);
          }
          page_next = page_at((y >> 1) + 1, &off_next);
        }
        const __nv_bfloat16* base = (y & 1) ? v_pages : k_pages;
        const uint32_t dst = ring_a + (y % C::kItems) * C::kItem;
        constexpr int kPieces = D / 8;  // 16-byte pieces of a row
#pragma unroll
        for (int x = 0; x < kDecKeys * kPieces / 32; ++x) {
          const int piece = (x * 32 + lane) % kPieces, r = (x * 32 + lane) / kPieces;
          const uint32_t src = __shfl_sync(0xffffffffu, row_cur, r);
          const bool ok = src != 0xffffffffu;
          cp_async16(dst + r * (D * 2) + ((piece ^ (r & 7)) << 4),
                     base + static_cast<size_t>(ok ? src : 0u) * D + piece * 8, ok);
        }
      }
      cp_async_commit();
    };
#pragma unroll 1
    for (int y = 0; y < C::kItems - 1; ++y) issue(y);

    // Q^T fragments (behind the first copies): head lane / 4 of each 8, d pairs of each 16
    uint32_t qf[C::kQSmem ? 1 : NT][C::kQSmem ? 1 : kKs][2];
    const __nv_bfloat16* qb = q + (static_cast<size_t>(b) * g.Hq + h0) * D;
    if constexpr (C::kQSmem) {
      for (int x = tid; x < NT * kKs * 32; x += kThreads) {
        const int nt = x / (kKs * 32), ks = x / 32 % kKs, l = x % 32, h = nt * 8 + (l >> 2);
        const uint32_t* p = reinterpret_cast<const uint32_t*>(qb + h * D + ks * 16 + (l & 3) * 2);
        qs[x] = h < heads ? make_uint2(p[0], p[4]) : make_uint2(0, 0);
      }
      __syncthreads();
    } else {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const int h = nt * 8 + (lane >> 2);
        const uint32_t* p = reinterpret_cast<const uint32_t*>(qb + h * D + (lane & 3) * 2);
#pragma unroll
        for (int ks = 0; ks < kKs; ++ks) {
          qf[nt][ks][0] = h < heads ? p[ks * 8] : 0u;
          qf[nt][ks][1] = h < heads ? p[ks * 8 + 4] : 0u;
        }
      }
    }

    float acc[NT][kKs][4];
    float m[NT][2], l[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      m[nt][0] = m[nt][1] = -INFINITY;
      l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
      for (int ks = 0; ks < kKs; ++ks)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[nt][ks][e] = 0.f;
    }
#pragma unroll 1
    for (int i = 0; i < n_mine; ++i) {
      // K item: S^T = K Q^T, in kChains sums so that no product waits for the one before
      cp_async_wait<C::kItems - 2>();
      __syncwarp();
      constexpr int kChains = kKs >= 8 ? 4 : 2;
      float sc[kChains][NT][4];
#pragma unroll
      for (int c = 0; c < kChains; ++c)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) sc[c][nt][e] = 0.f;
      {
        const uint32_t a0 = ring_a + (2 * i % C::kItems) * C::kItem;
        const int r = (lane & 7) + ((lane >> 3) & 1) * 8;
        const uint32_t row_a = a0 + r * (D * 2);
#pragma unroll
        for (int ks = 0; ks < kKs; ++ks) {
          uint32_t a[4];
          ldsm4(a, row_a + (((ks * 2 + (lane >> 4)) ^ (r & 7)) << 4));
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            if constexpr (C::kQSmem) {
              const uint2 bq = qs[(nt * kKs + ks) * 32 + lane];
              mma16816(sc[ks % kChains][nt], a, bq.x, bq.y);
            } else {
              mma16816(sc[ks % kChains][nt], a, qf[nt][ks][0], qf[nt][ks][1]);
            }
          }
        }
      }
      issue(2 * i + C::kItems - 1);
      // online softmax over the 16 keys; this thread: keys lane / 4 and + 8, heads 2 (lane % 4) and + 1.
      // The running maximum is raised, and O and the sum rescaled, only when a
      // score passes it by 2^8.
      const int x0 = (t0 + warp + i * kDecWarps) * kDecKeys + (lane >> 2);
      const bool in0 = x0 < v.n, in1 = x0 + 8 < v.n;
      uint32_t pb[NT][2], pl[NT][2];  // P's upper bf16 half and what it leaves
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float x[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float sum = sc[0][nt][e] + sc[1][nt][e];
          if constexpr (kChains == 4) sum += sc[2][nt][e] + sc[3][nt][e];
          x[e] = (e < 2 ? in0 : in1) ? sum * sl2 : -INFINITY;
        }
        float m0 = fmaxf(x[0], x[2]), m1 = fmaxf(x[1], x[3]);
        if (__any_sync(0xffffffffu, m0 > m[nt][0] + 8.0f || m1 > m[nt][1] + 8.0f)) {
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) {
            m0 = fmaxf(m0, __shfl_xor_sync(0xffffffffu, m0, o));
            m1 = fmaxf(m1, __shfl_xor_sync(0xffffffffu, m1, o));
          }
          m0 = fmaxf(m0, m[nt][0]);
          m1 = fmaxf(m1, m[nt][1]);
          const float al0 = fast_exp2(m[nt][0] - exp_base(m0)), al1 = fast_exp2(m[nt][1] - exp_base(m1));
          l[nt][0] *= al0;
          l[nt][1] *= al1;
#pragma unroll
          for (int ks = 0; ks < kKs; ++ks) {
            acc[nt][ks][0] *= al0;
            acc[nt][ks][1] *= al1;
            acc[nt][ks][2] *= al0;
            acc[nt][ks][3] *= al1;
          }
          m[nt][0] = m0;
          m[nt][1] = m1;
        }
        const float b0 = exp_base(m[nt][0]), b1 = exp_base(m[nt][1]);
        const float p0 = fast_exp2(x[0] - b0), p1 = fast_exp2(x[1] - b1);
        const float p2 = fast_exp2(x[2] - b0), p3 = fast_exp2(x[3] - b1);
        l[nt][0] += p0 + p2;
        l[nt][1] += p1 + p3;
        const uint32_t u0 = pack_bf16x2(p0, p1), u1 = pack_bf16x2(p2, p3);
        pb[nt][0] = transpose8x8(u0);  // keys along the product's inner side
        pb[nt][1] = transpose8x8(u1);
        pl[nt][0] = transpose8x8(pack_bf16x2(p0 - bf16_lo(u0), p1 - bf16_hi(u0)));
        pl[nt][1] = transpose8x8(pack_bf16x2(p2 - bf16_lo(u1), p3 - bf16_hi(u1)));
      }
      // V item: O^T += V^T P^T
      cp_async_wait<C::kItems - 2>();
      __syncwarp();
      {
        const uint32_t a0 = ring_a + ((2 * i + 1) % C::kItems) * C::kItem;
        const int r = (lane & 7) + (lane >> 4) * 8;
        const uint32_t row_a = a0 + r * (D * 2);
#pragma unroll
        for (int ks = 0; ks < kKs; ++ks) {
          uint32_t a[4];
          ldsm4_t(a, row_a + (((ks * 2 + ((lane >> 3) & 1)) ^ (r & 7)) << 4));
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            mma16816(acc[nt][ks], a, pb[nt][0], pb[nt][1]);
            mma16816(acc[nt][ks], a, pl[nt][0], pl[nt][1]);
          }
        }
      }
      issue(2 * i + C::kItems);
    }
    cp_async_wait<0>();
    __syncwarp();

    // ---- join the warps: each leaves O in its ring, m and l behind the rings
    float* ow = reinterpret_cast<float*>(ring);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) {
        l[nt][0] += __shfl_xor_sync(0xffffffffu, l[nt][0], o);
        l[nt][1] += __shfl_xor_sync(0xffffffffu, l[nt][1], o);
      }
      const int h = nt * 8 + (lane & 3) * 2;
      if (lane < 4) {
        ml[(warp * kHeads + h) * 2] = m[nt][0];
        ml[(warp * kHeads + h) * 2 + 1] = l[nt][0];
        ml[(warp * kHeads + h + 1) * 2] = m[nt][1];
        ml[(warp * kHeads + h + 1) * 2 + 1] = l[nt][1];
      }
#pragma unroll
      for (int ks = 0; ks < kKs; ++ks) {
        float* o = ow + h * C::kOStride + ks * 16 + (lane >> 2);
        o[0] = acc[nt][ks][0];
        o[C::kOStride] = acc[nt][ks][1];
        o[8] = acc[nt][ks][2];
        o[C::kOStride + 8] = acc[nt][ks][3];
      }
    }
    __syncthreads();
    const bool whole = t0 == 0 && t1 == steps;
    const int slot = 2 * blockIdx.x + (first_piece ? 0 : 1);
    float* pt = part + static_cast<size_t>(slot) * dec_part_floats(D, kHeads);  // [head] m, l, -, -; then [head][D] O
    for (int x = tid; x < heads * (D / 4); x += kThreads) {
      const int h = x / (D / 4), d = (x % (D / 4)) * 4;
      float mm = -INFINITY;
#pragma unroll
      for (int w = 0; w < kDecWarps; ++w) mm = fmaxf(mm, ml[(w * kHeads + h) * 2]);
      const float base = exp_base(mm);
      float ll = 0.f;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kDecWarps; ++w) {
        const float f = fast_exp2(ml[(w * kHeads + h) * 2] - base);
        ll += f * ml[(w * kHeads + h) * 2 + 1];
        const float4 y = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(
                                                              smem + w * C::kItems * C::kItem) + h * C::kOStride + d);
        o.x = fmaf(f, y.x, o.x);
        o.y = fmaf(f, y.y, o.y);
        o.z = fmaf(f, y.z, o.z);
        o.w = fmaf(f, y.w, o.w);
      }
      if (whole) {
        const float inv = row_inv(ll);
        const size_t r = static_cast<size_t>(b) * g.Hq + h0 + h;
        *reinterpret_cast<uint2*>(out + r * D + d) =
            make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
        if (d == 0) lse[r] = row_lse(mm, ll);
      } else {
        *reinterpret_cast<float4*>(pt + kHeads * 4 + h * D + d) = o;
        if (d == 0) *reinterpret_cast<float4*>(pt + h * 4) = make_float4(mm, ll, 0.f, 0.f);
      }
    }
    if (!whole && t0 == 0 && tid == 0) {  // the row starts here and goes on
      DecDesc d{b, hk, hb, slot, static_cast<int>((at + steps - 1) / per), {0, 0, 0}};
      desc[blockIdx.x] = d;
    }
    __syncthreads();  // the rings are free again
    first_piece = false;
    at += t1 - t0;
    in_b += t1 - t0;
  }
}

// A row cut over CTAs: log-sum-exp weights over their partials. One CTA per (CTA
// the row starts in, head); each of its warps runs over every eighth partial,
// eight loads in flight, with a running maximum, and the warps are added in
// order: the same bits in every run.
constexpr int kJoinWarps = 8;

template <int D, int NT>
__global__ void __launch_bounds__(kJoinWarps * 32)
    paged_join_kernel(const PagedGeom g, int heads, const DecDesc* __restrict__ desc, const float* __restrict__ part,
                      __nv_bfloat16* __restrict__ out, float* __restrict__ lse, const int32_t* status) {
  pdl_begin();
  constexpr int kHeads = 8 * NT, kVec = (D + 127) / 128;  // float4 per lane
  constexpr int kBatch = D <= 128 ? 8 : D <= 256 ? 4 : 2;
  const int c0 = blockIdx.x / heads, h = blockIdx.x % heads;
  const DecDesc d = desc[c0];
  if (d.last_cta < 0 || h >= g.G - d.hb * kHeads) return;
  if (__syncthreads_or(*reinterpret_cast<const volatile int*>(status) != 0)) return;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  __shared__ float s_m[kJoinWarps], s_l[kJoinWarps];
  __shared__ float4 s_o[kJoinWarps][D / 4];
  const int n = d.last_cta - c0 + 1;
  auto part_of = [&](int i) {
    return part + static_cast<size_t>(i == 0 ? d.slot : 2 * (c0 + i)) * dec_part_floats(D, kHeads);
  };
  float mm = -INFINITY, ll = 0.f;
  float4 o[kVec];
#pragma unroll
  for (int e = 0; e < kVec; ++e) o[e] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i0 = warp; i0 < n; i0 += kJoinWarps * kBatch) {
    float pm[kBatch], pl[kBatch], bm = mm;
    float4 y[kBatch][kVec];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int i = i0 + k * kJoinWarps;
      pm[k] = -INFINITY;
      pl[k] = 0.f;
#pragma unroll
      for (int e = 0; e < kVec; ++e) y[k][e] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (i < n) {
        const float* p = part_of(i);
        const float2 x = *reinterpret_cast<const float2*>(p + h * 4);
        pm[k] = x.x;
        pl[k] = x.y;
#pragma unroll
        for (int e = 0; e < kVec; ++e)
          if (e * 128 + lane * 4 < D)
            y[k][e] = *reinterpret_cast<const float4*>(p + kHeads * 4 + h * D + e * 128 + lane * 4);
      }
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k) bm = fmaxf(bm, pm[k]);
    const float base = exp_base(bm), f0 = fast_exp2(mm - base);
    mm = bm;
    ll *= f0;
#pragma unroll
    for (int e = 0; e < kVec; ++e) {
      o[e].x *= f0;
      o[e].y *= f0;
      o[e].z *= f0;
      o[e].w *= f0;
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const float f = fast_exp2(pm[k] - base);
      ll = fmaf(f, pl[k], ll);
#pragma unroll
      for (int e = 0; e < kVec; ++e) {
        o[e].x = fmaf(f, y[k][e].x, o[e].x);
        o[e].y = fmaf(f, y[k][e].y, o[e].y);
        o[e].z = fmaf(f, y[k][e].z, o[e].z);
        o[e].w = fmaf(f, y[k][e].w, o[e].w);
      }
    }
  }
  if (lane == 0) {
    s_m[warp] = mm;
    s_l[warp] = ll;
  }
#pragma unroll
  for (int e = 0; e < kVec; ++e)
    if (e * 128 + lane * 4 < D) s_o[warp][e * 32 + lane] = o[e];
  __syncthreads();
  mm = s_m[0];
#pragma unroll
  for (int w = 1; w < kJoinWarps; ++w) mm = fmaxf(mm, s_m[w]);
  const float base = exp_base(mm);
  float f[kJoinWarps];
  ll = 0.f;
#pragma unroll
  for (int w = 0; w < kJoinWarps; ++w) {
    f[w] = fast_exp2(s_m[w] - base);
    ll = fmaf(f[w], s_l[w], ll);
  }
  const float inv = row_inv(ll);
  const size_t r = static_cast<size_t>(d.b) * g.Hq + d.hk * g.G + d.hb * kHeads + h;
  for (int x = tid; x < D / 4; x += kJoinWarps * 32) {
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) {
      const float4 y = s_o[w][x];
      a.x = fmaf(f[w], y.x, a.x);
      a.y = fmaf(f[w], y.y, a.y);
      a.z = fmaf(f[w], y.z, a.z);
      a.w = fmaf(f[w], y.w, a.w);
    }
    *reinterpret_cast<uint2*>(out + r * D + x * 4) =
        make_uint2(pack_bf16x2(a.x * inv, a.y * inv), pack_bf16x2(a.z * inv, a.w * inv));
  }
  if (tid == 0) lse[r] = row_lse(mm, ll);
}

namespace {
template <int D, int NT>
cudaError_t launch_decode_dn(const void* q, const void* k_pages, const void* v_pages, const int32_t* page_table,
                             const int32_t* seq_lens, const PagedGeom& g, void* out, float* lse, void* workspace,
                             int32_t* status, cudaStream_t st) {
  using C = DecCfg<D, NT>;
  auto kern = paged_decode_kernel<D, NT>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (e != cudaSuccess) return e;
  DecDesc* desc = static_cast<DecDesc*>(workspace);
  float* part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + dec_desc_bytes(D));
  const bool whole = dec_whole_rows(g);
  const int n_hb = (g.G + C::kHeads - 1) / C::kHeads, heads = g.G < C::kHeads ? g.G : C::kHeads;
  const unsigned ctas = static_cast<unsigned>(whole ? g.B * g.Hkv * n_hb : dec_ctas(D));
  __nv_bfloat16* o = static_cast<__nv_bfloat16*>(out);
  if (const cudaError_t le = launch_pdl(kern, dim3(ctas), dim3(kDecWarps * 32), C::kSmem, st,
                                        static_cast<const __nv_bfloat16*>(q),
                                        static_cast<const __nv_bfloat16*>(k_pages),
                                        static_cast<const __nv_bfloat16*>(v_pages), page_table, seq_lens, g,
                                        static_cast<int>(whole), o, lse, desc, part, status);
      le != cudaSuccess)
    return le;
  if (whole) return cudaGetLastError();
  if (const cudaError_t le = launch_pdl(paged_join_kernel<D, NT>, dim3(ctas * heads), dim3(kJoinWarps * 32), 0, st, g, heads,
                                        static_cast<const DecDesc*>(desc), static_cast<const float*>(part), o, lse,
                                        static_cast<const int32_t*>(status));
      le != cudaSuccess)
    return le;
  return cudaGetLastError();
}
}  // namespace

size_t paged_decode_workspace_bytes(const PagedGeom& g) {
  if (dec_whole_rows(g)) return kDecNoWorkspace;
  return dec_desc_bytes(g.D) + 2 * static_cast<size_t>(dec_ctas(g.D)) *
                                   dec_part_floats(g.D, 8 * dec_head_tiles(g.D, g.G)) * 4;
}

cudaError_t launch_paged_decode(const void* q, const void* k_pages, const void* v_pages, const int32_t* page_table,
                                const int32_t* seq_lens, const PagedGeom& g, void* out, float* lse, void* workspace,
                                int32_t* status, cudaStream_t st) {
  const bool two = dec_head_tiles(g.D, g.G) == 2;
#define BD_DECODE(D, NT) \
  launch_decode_dn<D, NT>(q, k_pages, v_pages, page_table, seq_lens, g, out, lse, workspace, status, st)
  switch (g.D) {
    case 64: return two ? BD_DECODE(64, 2) : BD_DECODE(64, 1);
    case 128: return two ? BD_DECODE(128, 2) : BD_DECODE(128, 1);
    case 256: return two ? BD_DECODE(256, 2) : BD_DECODE(256, 1);
    case 512: return BD_DECODE(512, 1);
    default: return cudaErrorInvalidValue;
  }
#undef BD_DECODE
}

}  // namespace bd
