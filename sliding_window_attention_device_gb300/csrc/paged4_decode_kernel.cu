// Decode over a 4-bit paged cache: out = softmax(scale q K^T) V of one query row per
// head over its sequence's visible keys, K and V as e2m1 codes with one e4m3 scale
// per 16 numbers of a row.
//
// Rows of work, whole rows where sequences are short, and the join are those of the
// decode over bf16 pages (paged_kernels.cu). What differs:
//   Values are made in registers. A value, code times scale, has at most 6 significant
// bits and lies between 2^-10 and 2688: exact in fp16. So the products are fp16 mma.sync
// m16n8k16 with fp32 sums; q, whose range fp16 lacks, is scaled by a power of two per
// head that its scores are multiplied with afterwards; P is taken against the maximum
// less 7 (in log2), so the largest weight is between 2^7 and 2^15 and fp16's smallest
// step, 2^-24, is at most 2^-31 of it; and each weight is two fp16 numbers, the second of
// what the first left, off by 2^-22 of it or by 2^-32 of the largest: out is then off by
// its own rounding only. The second one costs a second product with V, but where a row
// has at most 4 heads (kFold): they stand twice among a product's 8 columns, which hold
// first parts in one half and second parts in the other. 16 sequences to 32,768 keys with 4
// heads 66.7 us folded, 72.8 with two products (D 64 44.9 and 47.5); 32 with a window of
// 1024 at D 256 and 2 heads 22.4 and 24.0. One number per weight took 67 us for 8 heads
// (two: 75) and 92 for 16 (110).
//   The order of d within a product and of keys within a step is free as long as both
// factors share it. So lane (g, c) = (lane / 4, lane % 4) of the K product reads a
// quarter of a key's row, D / 8 bytes, from shared memory at once and makes its part of
// all A fragments from it; and of the V product a piece of D / 16 bytes of four keys'
// rows, whose codes are put side by side key by key before they are converted. No
// transposing load, no shuffle; 16-byte pieces are swizzled so that the loads touch every
// bank as often.
//   A step is 32 keys of a warp (16 from D 256 on), beginning at a multiple of that; a
// step of the window whose keys are all visible needs no masks, and where pages are
// multiples of 16 tokens its 16-key halves are pieces of the cache, one address each (one
// per row elsewhere: pages of 200 at D 128 50 us for 48). The sinks' steps are masked ones
// also where they are whole: meant for a few of them.
//   The line of all rows' steps is cut for each row by itself where rows are few, into
// equal pieces otherwise, with a charge for each row's start (kRowStart): a CTA that
// goes from one row to the next waits for a page number, for keys and for its warps.
//
// What bounds it. 16 keys of D 128 are 2,304 bytes, 392 clocks of an SM's quarter at the
// copy rate, and 325 instructions (measured; 64 conversions, 64 products with scales, 24
// mma, 12 loads from shared memory, the rest copies, softmax and addresses). With one
// number per weight, 16 mma and no copies the work took 327 clocks, and 8 mma more are
// some 65: conversions, half-precision products and mma.sync hardly overlap on the SM. So
// instructions and bytes bound it about alike. 16 ragged sequences to 32,768 keys, 8 kv
// heads of 8 heads each, D 128, 312 MB: 75 us, 4.2 TB/s (the bf16 pages of the same keys:
// 172 us); D 64, 156 MB 50 us; D 256, 313 MB 76; D 512 68. With 16 heads each D 64 72,
// D 128 110, D 256 109. A call with few steps is 3 us of a launch, page number, keys and
// softmax, one after the other, and 2 to 3 of the join: one sequence of 1,000 keys 8 us,
// of 131,072 (75 MB) 26.
//   Tried and not kept, for the 312 MB, all with one number per weight: bulk copies by
// one lane 79 us for 67 (many small ones); K and V as items of their own 77 for 74; 24
// warps an SM at 80 registers 105;
// every warp with a piece of the line of its own 69 for 72, but 28 for 22 at 1,028 keys
// of D 256. Two CTAs an SM, but for 16 heads at D 128 (91 us with one and 236 registers,
// 113 with two) and D 256, and for D 512.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cstdint>

#include "fp4.cuh"
#include "paged_decode.cuh"
#include "sm100_ptx.cuh"

namespace bd {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kSpan = 8;  // sequences of a lane where a warp sums up all of them
// What a row's start in a CTA's midst costs, in steps (312 MB over 128 rows with 0, 12,
// 24 and 48: 77.7, 74.7, 74.9 and 77.4 us; head dim 512: 78.7, 70.6, 67.9 and 69.9).
constexpr int kRowStart = 24;
// How the line is cut: a row per CTA; or equal pieces, rows that are cut being named by
// the CTA they start in, or, where there are no more rows than CTAs, by their number.
enum { kWholeRows = 0, kCutByCta = 1, kCutByRow = 2 };
constexpr float kRefShift = 7.0f;  // log2: weights are taken against the maximum less this
constexpr float kRaise = 15.0f;    // and may grow up to 2^this, within fp16's range

template <int D, int NT>
struct Cfg {
  static constexpr int kGroups = D <= 128 ? 2 : 1;  // groups of 16 keys of a step
  static constexpr int kStep = 16 * kGroups;
  static constexpr int kCodeRow = D / 2, kBlockRow = D / 16;  // bytes of a key's codes and scales
  // a step in the ring: K codes, V codes, K scales, V scales
  static constexpr int kVCodes = kStep * kCodeRow, kKBlocks = 2 * kVCodes, kVBlocks = kKBlocks + kStep * kBlockRow;
  static constexpr int kItem = kVBlocks + kStep * kBlockRow;
  static constexpr int kItems = D == 64 || (D <= 256 && NT == 2) ? 4 : D == 128 ? 3 : 2;
  static constexpr int kHeads = 8 * NT;
  static constexpr bool kQSmem = D > 128;  // Q fragments in shared memory instead of registers
  static constexpr int kRing = kWarps * kItems * kItem;
  static constexpr int kQBytes = kQSmem ? NT * (D / 16) * 32 * 8 : 0;
  static constexpr int kOStride = D + 4;  // fp32 row of a warp's O in its ring
  static constexpr int kMl = kWarps * kHeads * 8;
  static constexpr int kSmem = kRing + kQBytes + kMl;
  static constexpr int kCtas = dec4_ctas(D, NT) / kSms;  // per SM
  static_assert(kHeads * kOStride * 4 <= kItems * kItem, "a warp's O fits its ring");
  static_assert(kItem % 16 == 0 && (kSmem + 2048) * kCtas <= 227 * 1024, "");
};

// Where 16-byte piece j of row r lies in its row: the lanes of one load then touch
// every bank as often (once at D 128 and 256).
template <int D>
__device__ __forceinline__ int swizzle(int r) {
  if (D == 128) return r & 2;
  if (D == 256) return ((r & 3) << 1) | ((r >> 2) & 1);
  if (D == 512) return (r & 1) | ((r & 2) << 1);
  return 0;
}
// The key of a step that is index i of a product's 16 (8 + i likewise).
__device__ __forceinline__ int key_of(int i) { return (i & 1) ? ((i >> 1) + 4) ^ 1 : i >> 1; }

template <int kBytes>
__device__ __forceinline__ void cp_async_block(uint32_t dst, const void* src, bool valid) {
  if constexpr (kBytes == 16)
    cp_async16(dst, src, valid);
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(kBytes),
                 "r"(valid ? kBytes : 0)
                 : "memory");
}

template <int kBytes>
__device__ __forceinline__ void cp_async_all(uint32_t dst, const void* src) {
  if constexpr (kBytes == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(kBytes) : "memory");
}

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_f16_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ uint32_t half_twice(uint32_t h2, int upper) {
  const __half2 x = *reinterpret_cast<const __half2*>(&h2), y = upper ? __high2half2(x) : __low2half2(x);
  return *reinterpret_cast<const uint32_t*>(&y);
}
__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  const __half2 x = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&x);
}
// N words (1, 2, 4, 8, 16) of shared memory; pieces of 16 bytes lie at swizzled places.
template <int N>
__device__ __forceinline__ void load_words(const uint8_t* row, int byte, int swz, uint32_t (&w)[N]) {
  if constexpr (N == 1) {
    w[0] = *reinterpret_cast<const uint32_t*>(row + ((((byte >> 4) ^ swz) << 4) | (byte & 15)));
  } else if constexpr (N == 2) {
    const uint2 x = *reinterpret_cast<const uint2*>(row + ((((byte >> 4) ^ swz) << 4) | (byte & 15)));
    w[0] = x.x, w[1] = x.y;
  } else {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const uint4 x = *reinterpret_cast<const uint4*>(row + ((((byte >> 4) + i) ^ swz) << 4));
      w[4 * i] = x.x, w[4 * i + 1] = x.y, w[4 * i + 2] = x.z, w[4 * i + 3] = x.w;
    }
  }
}
// N scale bytes (1, 2, 4, 8), two to an entry.
template <int N>
__device__ __forceinline__ void load_scales(const uint8_t* p, uint32_t (&s)[(N + 1) / 2]) {
  if constexpr (N == 1) {
    s[0] = *p;
  } else if constexpr (N == 2) {
    s[0] = *reinterpret_cast<const uint16_t*>(p);
  } else {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const uint32_t x = *reinterpret_cast<const uint32_t*>(p + 4 * i);
      s[2 * i] = x & 0xffffu;
      s[2 * i + 1] = x >> 16;
    }
  }
}

// The steps of a sequence: the runs of kStep positions, counted from its first token,
// that hold a visible key; those of the sinks, then those of the window. Where both
// end and begin in one run it is a step of each.
template <int kStep>
struct Steps {
  int n, sinks;  // all of them; those of the sinks
  int first;     // the window's first run
  int lo, ns, len;
  __device__ __forceinline__ Steps(const PagedGeom& g, const int32_t* seq_lens, int b, bool* bad) {
    const Visible v = visible_keys(g, seq_lens, b, bad);
    lo = v.lo;
    ns = v.ns;
    len = v.lo + (v.n - v.ns);
    sinks = (ns + kStep - 1) / kStep;
    first = lo / kStep;
    n = sinks + (len + kStep - 1) / kStep - first;
  }
  // positions [base + a, base + e) of step t
  __device__ __forceinline__ int base(int t) const { return (t < sinks ? t : first + (t - sinks)) * kStep; }
  __device__ __forceinline__ int a(int t, int base) const { return t < sinks ? 0 : max(lo - base, 0); }
  __device__ __forceinline__ int e(int t, int base) const { return min((t < sinks ? ns : len) - base, kStep); }
};

// q of one head in fp16: q times 2^(14 - e), e the exponent of its largest number,
// whose scores are then to be multiplied by 2^(e - 14). Numbers 2^-28 of the largest
// and below lose bits that no fp32 sum would keep. With an infinity or NaN among them
// the finite ones are taken as zeros, which changes no such score.
struct QScale {
  float to_half, back;
  bool all_finite;
  __device__ __forceinline__ explicit QScale(uint32_t amax_bits) {
    all_finite = amax_bits < 0x7f800000u;
    int e = static_cast<int>(amax_bits >> 23) - 127;
    e = e < -100 ? -100 : e;
    if (!all_finite) e = 14;
    to_half = __uint_as_float(static_cast<uint32_t>(14 - e + 127) << 23);
    back = __uint_as_float(static_cast<uint32_t>(e - 14 + 127) << 23);
  }
  __device__ __forceinline__ float operator()(float q) const {
    return all_finite || !isfinite(q) ? q * to_half : 0.f;
  }
};
// Neither 0 nor infinite, so that a score of -inf stays one and 0 stays 0.
__device__ __forceinline__ float finite_scale(float x) { return fminf(fmaxf(x, 1.1754944e-38f), 3.4028235e38f); }
__device__ __forceinline__ float bf_lo(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float bf_hi(uint32_t u) { return __uint_as_float(u & 0xffff0000u); }
__device__ __forceinline__ uint32_t max_abs(uint32_t top, uint32_t pair) {
  return max(top, max((pair << 16) & 0x7fffffffu, pair & 0x7fff0000u));
}

template <int D, int NT, bool kFold>
__global__ void __launch_bounds__(kThreads, Cfg<D, NT>::kCtas)
    paged4_decode_kernel(const __nv_bfloat16* __restrict__ q, const Cache4 c4, const int32_t* __restrict__ page_table,
                         const int32_t* __restrict__ seq_lens, const PagedGeom g, int mode,
                         __nv_bfloat16* __restrict__ out, float* __restrict__ lse, DecDesc* __restrict__ desc,
                         float* __restrict__ part, int32_t* status) {
  pdl_begin();
  using C = Cfg<D, NT>;
  static_assert(!kFold || NT == 1, "");
  constexpr int kHeads = C::kHeads, kKs = D / 16;
  constexpr int kParts = kFold ? 1 : 2;  // columns that P's two parts take of their own
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ long long s_sum[kWarps];
  __shared__ int s_b, s_skip;
  __shared__ long long s_at;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int n_hb = (g.G + kHeads - 1) / kHeads, rows_b = g.Hkv * n_hb;

  if (tid == 0) s_skip = *reinterpret_cast<const volatile int*>(status) != 0;  // looked at behind a barrier
  bool bad = false;
  int b = 0;
  // [at, end) of the line is this CTA's; what of sequence b's part lies before it; where
  // aligned, the last CTA of a row that starts here
  long long per = 1, at = 0, end = 0, in_b = 0;
  bool aligned = false;
  int last_cta = 0;
  if (mode == kWholeRows) {
    // ---- one row per CTA
    b = blockIdx.x / rows_b;
    const int row = blockIdx.x % rows_b;
    const int steps = Steps<C::kStep>(g, seq_lens, b, &bad).n;
    if (bad) {
      if (tid == 0) atomicOr(status, BD_STATUS_BOUNDS);
      return;
    }
    if (steps == 0) {
      __syncthreads();
      if (s_skip) return;
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
    // ---- a piece of the line. Where rows are few, each is cut for itself into pieces of
    // no more than `per` steps (aligned): a CTA has one row. Else the line is cut into
    // equal pieces, wherever rows end: a row that starts in a CTA's midst costs it what
    // kRowStart steps take, so that many count for a row's start.
    const unsigned ctas = gridDim.x;
    auto div_up = [](long long x, unsigned n) {
      return x < 0x7fff0000LL ? (static_cast<unsigned>(x) + n - 1) / n : (x + n - 1) / n;
    };
    if (mode == kCutByCta && tid == 0) desc[blockIdx.x].last_cta = -1;
    long long place = 0;  // of the CTA's piece among its sequence's: CTAs if aligned, else steps with starts
    if (g.B <= 32 * kSpan) {
      // every warp for itself, lane x the steps of sequences [x * span, (x + 1) * span)
      const int span = (g.B + 31) / 32, x0 = lane * span, x1 = min(g.B, x0 + span);
      const int n_first = x0 < x1 ? Steps<C::kStep>(g, seq_lens, x0, &bad).n : 0;
      auto sum_of = [&](auto f) {
        auto n = f(n_first);
#pragma unroll 1
        for (int x = x0 + 1; x < x1; ++x) n += f(Steps<C::kStep>(g, seq_lens, x, &bad).n);
        return n;
      };
      // a lane's steps are below 2^30: summed up in two halves
      const unsigned my_steps = sum_of([](int n) { return static_cast<unsigned>(n); });
      const long long steps = (static_cast<long long>(__reduce_add_sync(0xffffffffu, my_steps >> 16)) << 16) +
                              __reduce_add_sync(0xffffffffu, my_steps & 0xffffu);
      const int rows = rows_b * __reduce_add_sync(0xffffffffu, sum_of([](int n) { return n > 0 ? 1 : 0; }));
      if (__any_sync(0xffffffffu, bad)) {  // every CTA sees every length: none writes
        if (bad) atomicOr(status, BD_STATUS_BOUNDS);
        return;
      }
      // sum ceil(steps / per) <= steps / per + rows, so this is enough for one CTA per piece
      per = max(div_up(steps * rows_b + static_cast<long long>(rows) * kRowStart, ctas),
                static_cast<long long>(kWarps));
      if (rows < static_cast<int>(ctas)) {
        const long long p = max(div_up(steps * rows_b, ctas - rows), static_cast<long long>(kWarps));
        if (p <= per) {
          aligned = true;
          per = p;
        }
      }
      auto share = [&](int n) -> long long {
        return n == 0 ? 0 : rows_b * (aligned ? div_up(n, static_cast<unsigned>(per)) : n + kRowStart);
      };
      place = aligned ? blockIdx.x : per * blockIdx.x;
      const long long mine = sum_of(share);
      long long incl = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long t = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += t;
      }
      end = __shfl_sync(0xffffffffu, incl, 31);
      // the first lane whose sequences end behind the place has it
      const unsigned behind = __ballot_sync(0xffffffffu, place < incl);
      const int owner = behind != 0 ? __ffs(behind) - 1 : 31;
      long long sum = incl - mine;
      int x = x0;
      if (span > 1 && lane == owner) {
#pragma unroll 1
        for (; x + 1 < x1; ++x) {
          const long long n = share(Steps<C::kStep>(g, seq_lens, x, &bad).n);
          if (place < sum + n) break;
          sum += n;
        }
      }
      b = __shfl_sync(0xffffffffu, x, owner);
      at = place;
      place = __shfl_sync(0xffffffffu, place - sum, owner);
    } else {
      // thread t sums the steps of sequences [t * span, (t + 1) * span)
      const int span = (g.B + kThreads - 1) / kThreads, x0 = tid * span, x1 = min(g.B, x0 + span);
      auto share = [&](int n) -> long long { return n == 0 ? 0 : static_cast<long long>(rows_b) * (n + kRowStart); };
      long long mine = 0;
      for (int x = x0; x < x1; ++x) mine += share(Steps<C::kStep>(g, seq_lens, x, &bad).n);
      if (bad) atomicOr(status, BD_STATUS_BOUNDS);
      long long incl = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long t = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += t;
      }
      if (lane == 31) s_sum[warp] = incl;
      if (__syncthreads_or(bad)) return;
      long long before = incl - mine;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        if (w < warp) before += s_sum[w];
        end += s_sum[w];
      }
      per = max(div_up(end, ctas), static_cast<long long>(kWarps));
      at = per * blockIdx.x;
      // the thread whose sequences hold the place finds the one
      if (at >= before && at < before + mine) {
        long long sum = before;
        int x = x0;
        for (;; ++x) {
          const long long n = share(Steps<C::kStep>(g, seq_lens, x, &bad).n);
          if (at < sum + n) break;
          sum += n;
        }
        s_b = x;
        s_at = at - sum;
      }
      __syncthreads();
      b = s_b;
      place = s_at;
    }
    in_b = place;
    if (aligned) {
      if (at < end) {  // `end` CTAs have a piece
        const int n = Steps<C::kStep>(g, seq_lens, b, &bad).n;
        const int pieces = static_cast<int>(div_up(n, static_cast<unsigned>(per)));
        const int row = static_cast<int>(place) / pieces, i = static_cast<int>(place) - row * pieces;
        last_cta = static_cast<int>(blockIdx.x) + pieces - 1;  // (where the row starts)
        in_b = static_cast<long long>(row) * n + min(i * per, static_cast<long long>(n));
        at = 0;
        end = min(per, n - min(i * per, static_cast<long long>(n)));
      }
    } else {
      end = min(at + per, end);
    }
  }
  const int row_start = mode == kWholeRows || aligned ? 0 : kRowStart;  // what a row costs in front of its steps

  uint8_t* ring = smem + warp * C::kItems * C::kItem;
  const uint32_t ring_a = smem_u32(ring);
  uint2* qs = reinterpret_cast<uint2*>(smem + C::kRing);
  float* ml = reinterpret_cast<float*>(smem + C::kRing + C::kQBytes);  // [warp][head] m, l
  __shared__ float s_back[kHeads];  // (kQSmem) what a head's scores are multiplied with
  const float sl2 = g.scale * 1.4426950408889634f * c4.k_gain;
  const bool whole_groups = g.page_size % 16 == 0;  // 16 keys of a step are one piece of a page
  const int gr = lane >> 2, cl = lane & 3;  // a product's row (or head) and column pair of this lane

  bool first_piece = true;
  while (at < end) {
    const Steps<C::kStep> sq(g, seq_lens, b, &bad);
    const int steps = sq.n;
    const int cost = steps == 0 ? 0 : steps + row_start;
    if (in_b >= static_cast<long long>(cost) * rows_b) {
      in_b -= static_cast<long long>(cost) * rows_b;
      ++b;
      continue;
    }
    const int row = static_cast<int>(in_b < 0x7fffffffLL ? static_cast<unsigned>(in_b) / static_cast<unsigned>(cost)
                                                         : in_b / cost);
    const int c0 = static_cast<int>(in_b - static_cast<long long>(row) * cost);
    const int c1 = static_cast<int>(min(static_cast<long long>(cost), c0 + (end - at)));
    const int t0 = max(c0 - row_start, 0), t1 = max(c1 - row_start, 0);  // steps [t0, t1) of the row
    if (t0 == t1) {
      at += c1 - c0;
      in_b += c1 - c0;
      continue;
    }
    const int hk = row / n_hb, hb = row % n_hb;
    const int heads = min(kHeads, g.G - hb * kHeads);  // query heads of this row
    const int h0 = hk * g.G + hb * kHeads;

    // ---- q, on its way before the first page is known. Index 2 c, 2 c + 1, 2 c + 8,
    // 2 c + 9 of product ks is d = c D / 4 + 4 ks + 0..3. In registers, a lane holds
    // what its part of the products takes, of head g; else a warp takes whole heads.
    constexpr int kQLoads = C::kQSmem ? kKs * 4 / 32 : kKs;
    constexpr int kQHeads = C::kQSmem ? (kHeads + kWarps - 1) / kWarps : NT;
    uint32_t qf[kQHeads][kQLoads][2];
    {
      const __nv_bfloat16* qb = q + (static_cast<size_t>(b) * g.Hq + h0) * D;
#pragma unroll
      for (int y = 0; y < kQHeads; ++y) {
        const int h = C::kQSmem ? warp + y * kWarps : y * 8 + gr;
        const int hq = kFold ? h & 3 : h;  // folded: heads 0 to 3 once more in columns 4 to 7
        const bool has = hq < heads;
        if constexpr (C::kQSmem) {
#pragma unroll
          for (int x = 0; x < kQLoads; ++x) {
            const int i = x * 32 + lane;  // (ks, c)
            uint2 u = make_uint2(0u, 0u);
            if (has) u = *reinterpret_cast<const uint2*>(qb + hq * D + (i & 3) * (D / 4) + 4 * (i >> 2));
            qf[y][x][0] = u.x, qf[y][x][1] = u.y;
          }
        } else {
#pragma unroll
          for (int ks = 0; ks < kKs; ks += 2) {
            uint4 u = make_uint4(0u, 0u, 0u, 0u);
            if (has) u = *reinterpret_cast<const uint4*>(qb + hq * D + cl * (D / 4) + 4 * ks);
            qf[y][ks][0] = u.x, qf[y][ks][1] = u.y, qf[y][ks + 1][0] = u.z, qf[y][ks + 1][1] = u.w;
          }
        }
      }
    }

    // ---- this warp's steps: t0 + warp, t0 + warp + kWarps, ...
    // Steps [full0, full0 + n_full), of the window, see all of their keys.
    constexpr int kStep = C::kStep;
    const int full0 = sq.sinks + (sq.lo % kStep != 0);
    const int n_full = max(steps - (sq.len % kStep != 0) - full0, 0);
    auto is_full = [&](int t) { return static_cast<unsigned>(t - full0) < static_cast<unsigned>(n_full); };
    const int32_t* pages = page_table + static_cast<size_t>(b) * g.max_pages;
    const int key = lane % kStep;
    // The page of this lane's key of step t (-1: no such key) and its place in it, looked
    // up a step before they are used.
    auto page_at = [&](int t, int* off) -> int {
      if (t >= t1) return -1;
      const int base = sq.base(t), pos = base + key;
      if (!is_full(t) && (key < sq.a(t, base) || key >= sq.e(t, base))) return -1;
      const int i = g.page_shift >= 0 ? pos >> g.page_shift : pos / g.page_size;
      *off = pos - i * g.page_size;
      return pages[i];
    };
    int off_next = 0, t_next = t0 + warp, page_next = page_at(t_next, &off_next);
    int put = 0;  // place of the ring that step t_next goes to
    constexpr int kPieces = C::kCodeRow / 16, kRowsAtOnce = 32 / kPieces;  // 16-byte pieces of a row; rows of 32 pieces
    const int piece = lane % kPieces, r_piece = lane / kPieces;
    auto issue = [&]() {  // the next of my steps into the ring
      if (t_next < t1) {
        const int t = t_next, page = page_next, off = off_next;
        t_next += kWarps;
        page_next = page_at(t_next, &off_next);
        const uint32_t dst = ring_a + put * C::kItem;
        put = put + 1 == C::kItems ? 0 : put + 1;
        const bool in_cache = static_cast<unsigned>(page) < static_cast<unsigned>(g.n_pages);
        uint32_t row = page_row(g, page, hk, off);  // of this lane's key
        if (is_full(t) && __all_sync(0xffffffffu, in_cache)) {
          if (whole_groups) {  // 16 rows are one piece of the cache
#pragma unroll
            for (int q = 0; q < C::kGroups; ++q) {
              const uint32_t row0 = __shfl_sync(0xffffffffu, row, 16 * q);
              const size_t from = static_cast<size_t>(row0) * C::kCodeRow + lane * 16;
              const uint8_t *kf = c4.k_codes + from, *vf = c4.v_codes + from;
#pragma unroll
              for (int x = 0; x < 16 / kRowsAtOnce; ++x) {
                const int r = x * kRowsAtOnce + r_piece;
                const uint32_t to = dst + (16 * q + r) * C::kCodeRow + ((piece ^ swizzle<D>(r)) << 4);
                cp_async_all<16>(to, kf + x * 512);
                cp_async_all<16>(to + C::kVCodes, vf + x * 512);
              }
            }
          } else {  // a row at a time
#pragma unroll
            for (int x = 0; x < kStep / kRowsAtOnce; ++x) {
              const int r = x * kRowsAtOnce + r_piece;
              const size_t from = static_cast<size_t>(__shfl_sync(0xffffffffu, row, r)) * C::kCodeRow + piece * 16;
              const uint32_t to = dst + r * C::kCodeRow + ((piece ^ swizzle<D>(r)) << 4);
              cp_async_all<16>(to, c4.k_codes + from);
              cp_async_all<16>(to + C::kVCodes, c4.v_codes + from);
            }
          }
          if constexpr (C::kGroups == 2) {  // a lane's key, both scales
            const size_t block = static_cast<size_t>(row) * C::kBlockRow;
            cp_async_all<C::kBlockRow>(dst + C::kKBlocks + lane * C::kBlockRow, c4.k_blocks + block);
            cp_async_all<C::kBlockRow>(dst + C::kVBlocks + lane * C::kBlockRow, c4.v_blocks + block);
          } else if constexpr (C::kBlockRow == 16) {  // lanes 0 to 15 K's, the others V's
            cp_async_all<16>(dst + C::kKBlocks + lane * 16,
                             (lane < 16 ? c4.k_blocks : c4.v_blocks) + static_cast<size_t>(row) * 16);
          } else {
            static_assert(C::kBlockRow == 32, "");
            const size_t block = static_cast<size_t>(__shfl_sync(0xffffffffu, row, lane >> 1)) * 32 + (lane & 1) * 16;
            cp_async_all<16>(dst + C::kKBlocks + lane * 16, c4.k_blocks + block);
            cp_async_all<16>(dst + C::kVBlocks + lane * 16, c4.v_blocks + block);
          }
        } else {  // the sinks' steps, the window's first and last: zeros for keys that are not to be seen
          const int base = sq.base(t);
          const bool seen = key >= sq.a(t, base) && key < sq.e(t, base);
          if (seen && !in_cache) atomicOr(status, BD_STATUS_BOUNDS);
          if (!seen || !in_cache) row = kNoRow;
#pragma unroll 1
          for (int r = r_piece; r < kStep; r += kRowsAtOnce) {
            const uint32_t src = __shfl_sync(0xffffffffu, row, r);
            const bool ok = src != kNoRow;
            const size_t from = static_cast<size_t>(ok ? src : 0u) * C::kCodeRow + piece * 16;
            const uint32_t to = dst + r * C::kCodeRow + ((piece ^ swizzle<D>(r)) << 4);
            cp_async16(to, c4.k_codes + from, ok);
            cp_async16(to + C::kVCodes, c4.v_codes + from, ok);
          }
          constexpr int kBlockPieces = C::kBlockRow > 16 ? C::kBlockRow / 16 : 1, kBytes = C::kBlockRow / kBlockPieces;
#pragma unroll 1
          for (int y = lane; y < 2 * kStep * kBlockPieces; y += 32) {  // K's scales, then V's
            const int z = y % (kStep * kBlockPieces);
            const uint32_t src = __shfl_sync(0xffffffffu, row, z / kBlockPieces);
            const bool ok = src != kNoRow;
            const uint8_t* p = (y < kStep * kBlockPieces ? c4.k_blocks : c4.v_blocks) +
                               static_cast<size_t>(ok ? src : 0u) * C::kBlockRow + z % kBlockPieces * kBytes;
            cp_async_block<kBytes>(dst + C::kKBlocks + y * kBytes, p, ok);
          }
        }
      }
      cp_async_commit();
    };
#pragma unroll 1
    for (int y = 0; y < C::kItems - 1; ++y) issue();

    // Q fragments from what was loaded
    float back[NT][2];  // of heads 2 c and 2 c + 1
    if constexpr (C::kQSmem) {
#pragma unroll
      for (int y = 0; y < kQHeads; ++y) {
        const int h = warp + y * kWarps;
        if (h >= kHeads) break;
        uint32_t top = 0;
#pragma unroll
        for (int x = 0; x < kQLoads; ++x) top = max_abs(max_abs(top, qf[y][x][0]), qf[y][x][1]);
        top = __reduce_max_sync(0xffffffffu, top);
        const QScale scale(top);
#pragma unroll
        for (int x = 0; x < kQLoads; ++x) {
          const int i = x * 32 + lane;
          qs[((h >> 3) * kKs + (i >> 2)) * 32 + (h & 7) * 4 + (i & 3)] =
              make_uint2(pack_half2(scale(bf_lo(qf[y][x][0])), scale(bf_hi(qf[y][x][0]))),
                         pack_half2(scale(bf_lo(qf[y][x][1])), scale(bf_hi(qf[y][x][1]))));
        }
        if (lane == 0) s_back[h] = finite_scale(scale.back * sl2);
      }
      __syncthreads();
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        back[nt][0] = s_back[nt * 8 + cl * 2];
        back[nt][1] = s_back[nt * 8 + cl * 2 + 1];
      }
    } else {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        uint32_t top = 0;
#pragma unroll
        for (int ks = 0; ks < kKs; ++ks) top = max_abs(max_abs(top, qf[nt][ks][0]), qf[nt][ks][1]);
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const QScale scale(top);
#pragma unroll
        for (int ks = 0; ks < kKs; ++ks)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            qf[nt][ks][e] = pack_half2(scale(bf_lo(qf[nt][ks][e])), scale(bf_hi(qf[nt][ks][e])));
        back[nt][0] = finite_scale(__shfl_sync(0xffffffffu, scale.back, cl * 8) * sl2);
        back[nt][1] = finite_scale(__shfl_sync(0xffffffffu, scale.back, cl * 8 + 4) * sl2);
      }
    }

    float acc[NT][kKs][4];
    // m: what exponents are taken against, the maximum less kRefShift or up to kRaise below
    // the next scores; neg_base: -m, or 0; limit: m + kRaise
    float m[NT][2], l[NT][2], neg_base[NT][2], limit[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      m[nt][0] = m[nt][1] = limit[nt][0] = limit[nt][1] = -INFINITY;
      neg_base[nt][0] = neg_base[nt][1] = 0.f;
      l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
      for (int ks = 0; ks < kKs; ++ks)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[nt][ks][e] = 0.f;
    }
    int take = 0;  // place of the ring of step t
#pragma unroll 1
    for (int t = t0 + warp; t < t1; t += kWarps) {
      cp_async_wait<C::kItems - 2>();
      __syncwarp();
      issue();  // into the place that every lane has read a step ago
      const uint8_t* item = ring + take * C::kItem;
      take = take + 1 == C::kItems ? 0 : take + 1;
      // ---- S^T = K Q^T of each group, in kChains sums so that no product waits for the one before
      constexpr int kGroups = C::kGroups, kChains = kGroups == 2 ? 2 : kKs >= 8 ? 4 : 2;
      float x[kGroups][NT][4];
#pragma unroll
      for (int q = 0; q < kGroups; ++q) {
        float sc[kChains][NT][4];
        constexpr int kW = D / 32, kB = D / 64;  // words and scales of a lane's quarter of a row
        uint32_t w0[kW], w1[kW], s0[(kB + 1) / 2], s1[(kB + 1) / 2];
        const int r0 = 16 * q + key_of(gr), swz = swizzle<D>(r0);  // (row r0 + 8 has the same)
        load_words<kW>(item + r0 * C::kCodeRow, cl * (D / 8), swz, w0);
        load_words<kW>(item + (r0 + 8) * C::kCodeRow, cl * (D / 8), swz, w1);
        load_scales<kB>(item + C::kKBlocks + r0 * C::kBlockRow + cl * kB, s0);
        load_scales<kB>(item + C::kKBlocks + (r0 + 8) * C::kBlockRow + cl * kB, s1);
#pragma unroll
        for (int w = 0; w < kW; ++w) {
          const int blk = w / 2;
          const uint32_t f0 = half_twice(e4m3_values(s0[blk / 2]), blk & 1);
          const uint32_t f1 = half_twice(e4m3_values(s1[blk / 2]), blk & 1);
          uint32_t x0[4], x1[4];
          e2m1_values(w0[w], x0);
          e2m1_values(w1[w], x1);
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int ks = 2 * w + e;
            const uint32_t a[4] = {mul_h2(x0[2 * e], f0), mul_h2(x1[2 * e], f1), mul_h2(x0[2 * e + 1], f0),
                                   mul_h2(x1[2 * e + 1], f1)};
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              uint2 bq;
              if constexpr (C::kQSmem) bq = qs[(nt * kKs + ks) * 32 + lane];
              else bq = make_uint2(qf[nt % kQHeads][ks % kQLoads][0], qf[nt % kQHeads][ks % kQLoads][1]);
              if (ks < kChains) mma_f16_first(sc[ks][nt], a, bq.x, bq.y);
              else mma_f16(sc[ks % kChains][nt], a, bq.x, bq.y);
            }
          }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            x[q][nt][y] = sc[0][nt][y] + sc[1][nt][y];
            if constexpr (kChains == 4) x[q][nt][y] += sc[2][nt][y] + sc[3][nt][y];
          }
      }
      // ---- online softmax; this thread: keys key_of(g) and + 8 of each group, heads 2 c and + 1.
      // The reference is raised, and O and the sum rescaled, only when a score
      // passes it by kRaise.
      if (!is_full(t)) {
        const int base = sq.base(t), a = sq.a(t, base), e = sq.e(t, base);
#pragma unroll
        for (int q = 0; q < kGroups; ++q) {
          const int k0 = 16 * q + key_of(gr);
          const bool in0 = k0 >= a && k0 < e, in1 = k0 + 8 >= a && k0 + 8 < e;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int y = 0; y < 4; ++y)
              if (!(y < 2 ? in0 : in1)) x[q][nt][y] = -INFINITY;
        }
      }
      auto top_of = [&](int nt, int h) {
        float top = fmaxf(x[0][nt][h], x[0][nt][2 + h]);
        if constexpr (kGroups == 2) top = fmax3(top, x[1][nt][h], x[1][nt][2 + h]);
        return top * back[nt][h];
      };
      bool above = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) above |= top_of(nt, 0) > limit[nt][0] || top_of(nt, 1) > limit[nt][1];
      if (__any_sync(0xffffffffu, above)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float top = top_of(nt, h);
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            const float now = fmaxf(top - kRefShift, m[nt][h]), neg = -exp_base(now);
            const float f = fast_exp2(m[nt][h] + neg);
            l[nt][h] *= f;
#pragma unroll
            for (int j = 0; j < kKs; ++j) {
              acc[nt][j][h] *= f;
              acc[nt][j][2 + h] *= f;
            }
            m[nt][h] = now;
            neg_base[nt][h] = neg;
            limit[nt][h] = now + kRaise;
          }
      }
      // P in two fp16 parts, the second of what the first left; folded, columns 4 to 7 hold the second ones
      uint32_t pb[kGroups][NT][kParts][2];
#pragma unroll
      for (int q = 0; q < kGroups; ++q)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float p[4];
#pragma unroll
          for (int y = 0; y < 4; ++y) p[y] = fast_exp2(fmaf(x[q][nt][y], back[nt][y & 1], neg_base[nt][y & 1]));
          l[nt][0] += p[0] + p[2];
          l[nt][1] += p[1] + p[3];
#pragma unroll
          for (int z = 0; z < 2; ++z) {  // keys along the product's inner side
            const uint32_t first = pack_half2(p[2 * z], p[2 * z + 1]);
            const float2 f = floats_of(first);
            const uint32_t second = pack_half2(p[2 * z] - f.x, p[2 * z + 1] - f.y);
            if constexpr (kFold) {
              pb[q][nt][0][z] = transpose8x8(cl < 2 ? first : second);
            } else {
              pb[q][nt][0][z] = transpose8x8(first);
              pb[q][nt][kParts - 1][z] = transpose8x8(second);
            }
          }
        }
      // ---- O^T += V^T P^T: rows g and g + 8 of product j are d = g D / 8 + 2 j and + 1
#pragma unroll
      for (int q = 0; q < kGroups; ++q) {
        constexpr int kW = D / 64, kB = D / 128 > 0 ? D / 128 : 1;  // words and scales of a lane's eighth of a row
        uint32_t w[4][kW], s[4][(kB + 1) / 2];
#pragma unroll
        for (int k = 0; k < 4; ++k) {  // keys 2 c, 2 c + 1, 2 c + 8, 2 c + 9 of the product
          const int r = 16 * q + key_of(2 * cl + (k & 1)) + (k >> 1) * 8;
          load_words<kW>(item + C::kVCodes + r * C::kCodeRow, gr * (D / 16), swizzle<D>(r), w[k]);
          load_scales<kB>(item + C::kVBlocks + r * C::kBlockRow + gr * (D / 8) / 16, s[k]);
        }
#pragma unroll
        for (int y = 0; y < kW; ++y) {
          const int blk = y / 2;
          // the two keys' scales side by side
          const uint32_t pick = blk & 1 ? 0x51 : 0x40;
          const uint32_t f0 = e4m3_values(__byte_perm(s[0][blk / 2], s[1][blk / 2], pick));
          const uint32_t f1 = e4m3_values(__byte_perm(s[2][blk / 2], s[3][blk / 2], pick));
          constexpr uint32_t kLow = 0x0f0f0f0fu;
          uint32_t v[4][4];  // [d even, d odd of keys 0, 1; of keys 2, 3][byte]
          e2m1_values((w[0][y] & kLow) | ((w[1][y] << 4) & ~kLow), v[0]);
          e2m1_values(((w[0][y] >> 4) & kLow) | (w[1][y] & ~kLow), v[1]);
          e2m1_values((w[2][y] & kLow) | ((w[3][y] << 4) & ~kLow), v[2]);
          e2m1_values(((w[2][y] >> 4) & kLow) | (w[3][y] & ~kLow), v[3]);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t a[4] = {mul_h2(v[0][e], f0), mul_h2(v[1][e], f0), mul_h2(v[2][e], f1), mul_h2(v[3][e], f1)};
#pragma unroll
            for (int part = 0; part < kParts; ++part)
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
                mma_f16(acc[nt][4 * y + e], a, pb[q][nt][part][0], pb[q][nt][part][1]);
          }
        }
      }
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
      const int h = nt * 8 + cl * 2;
      if (lane < 4) {
        ml[(warp * kHeads + h) * 2] = m[nt][0];
        ml[(warp * kHeads + h) * 2 + 1] = l[nt][0];
        ml[(warp * kHeads + h + 1) * 2] = m[nt][1];
        ml[(warp * kHeads + h + 1) * 2 + 1] = l[nt][1];
      }
#pragma unroll
      for (int j = 0; j < kKs; ++j) {
        float* o = ow + h * C::kOStride + gr * (D / 8) + 2 * j;
        *reinterpret_cast<float2*>(o) = make_float2(acc[nt][j][0], acc[nt][j][2]);
        *reinterpret_cast<float2*>(o + C::kOStride) = make_float2(acc[nt][j][1], acc[nt][j][3]);
      }
    }
    __syncthreads();
    if (s_skip) return;
    const bool whole = t0 == 0 && t1 == steps;
    const int slot = 2 * blockIdx.x + (first_piece ? 0 : 1);
    float* pt = part + static_cast<size_t>(slot) * dec_part_floats(D, kHeads);  // [head] m, l, -, -; then [head][D] O
    for (int x = tid; x < heads * (D / 4); x += kThreads) {
      const int h = x / (D / 4), d = (x % (D / 4)) * 4;
      float mm = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, ml[(w * kHeads + h) * 2]);
      const float base = exp_base(mm);
      float ll = 0.f;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float f = fast_exp2(ml[(w * kHeads + h) * 2] - base);
        ll += f * ml[(w * kHeads + h) * 2 + 1];
        auto add = [&](float f, int column) {
          const float4 y = *reinterpret_cast<const float4*>(
              reinterpret_cast<const float*>(smem + w * C::kItems * C::kItem) + column * C::kOStride + d);
          o.x = fmaf(f, y.x, o.x);
          o.y = fmaf(f, y.y, o.y);
          o.z = fmaf(f, y.z, o.z);
          o.w = fmaf(f, y.w, o.w);
        };
        add(f, h);
        if constexpr (kFold) add(fast_exp2(ml[(w * kHeads + h + 4) * 2] - base), h + 4);
      }
      o.x *= c4.v_gain, o.y *= c4.v_gain, o.z *= c4.v_gain, o.w *= c4.v_gain;
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
    if (t0 == 0 && tid == 0 && (mode == kCutByRow || !whole)) {  // the row starts here, and may go on
      DecDesc d{b, hk, hb, slot, 
                whole ? -1 : aligned ? last_cta : static_cast<int>((at - c0 + cost - 1) / per),
                static_cast<int>(blockIdx.x), {0, 0}};
      desc[mode == kCutByRow ? b * rows_b + row : blockIdx.x] = d;
    }
    __syncthreads();  // the rings are free again
    first_piece = false;
    at += c1 - c0;
    in_b += c1 - c0;
  }
  if (mode == kWholeRows) return;
  // sequences without a visible key: zeros and -inf, shared out over the CTAs
  for (int x = blockIdx.x; x < g.B; x += gridDim.x) {
    if (Steps<C::kStep>(g, seq_lens, x, &bad).n > 0) continue;
    __syncthreads();
    if (s_skip) return;
    uint4* o4 = reinterpret_cast<uint4*>(out + static_cast<size_t>(x) * g.Hq * D);
    for (int i = tid; i < g.Hq * (D / 8); i += kThreads) o4[i] = make_uint4(0, 0, 0, 0);
    for (int i = tid; i < g.Hq; i += kThreads) lse[static_cast<size_t>(x) * g.Hq + i] = -INFINITY;
    if (mode == kCutByRow)
      for (int i = tid; i < rows_b; i += kThreads) desc[x * rows_b + i].last_cta = -1;
  }
}

template <int D, int NT, bool kFold = false>
cudaError_t launch_dn(const void* q, const Cache4& c4, const int32_t* page_table, const int32_t* seq_lens,
                      const PagedGeom& g, void* out, float* lse, void* workspace, int32_t* status, cudaStream_t st) {
  using C = Cfg<D, NT>;
  auto kern = paged4_decode_kernel<D, NT, kFold>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (e != cudaSuccess) return e;
  DecDesc* desc = static_cast<DecDesc*>(workspace);
  float* part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + dec4_desc_bytes(D, NT));
  const bool whole = dec4_whole_rows(g);
  const int n_hb = (g.G + C::kHeads - 1) / C::kHeads;
  const long long rows = static_cast<long long>(g.B) * g.Hkv * n_hb;
  const unsigned ctas = static_cast<unsigned>(whole ? rows : dec4_ctas(D, NT));
  const bool by_row = rows <= dec4_ctas(D, NT);
  const int mode = whole ? kWholeRows : by_row ? kCutByRow : kCutByCta;
  if (const cudaError_t le = launch_pdl(kern, dim3(ctas), dim3(kThreads), C::kSmem, st,
                                        static_cast<const __nv_bfloat16*>(q), c4, page_table, seq_lens, g, mode,
                                        static_cast<__nv_bfloat16*>(out), lse, desc, part, status);
      le != cudaSuccess)
    return le;
  if (whole) return cudaGetLastError();
  // 16 warps to a row and head where it is cut over 16 CTAs or more (4 rows, 76 CTAs each:
  // 24.4 us for 25.6), 8 elsewhere (128 rows: 66.8 for 70.4)
  return launch_paged_join(D, NT, rows * 16 <= dec4_ctas(D, NT), g,
                           by_row ? static_cast<int>(rows) : dec4_ctas(D, NT), desc, part, out, lse, status, st);
}
}  // namespace

size_t paged4_decode_workspace_bytes(const PagedGeom& g) {
  if (dec4_whole_rows(g)) return kDecNoWorkspace;
  const int nt = dec_head_tiles(g.D, g.G);
  return dec4_desc_bytes(g.D, nt) + 2 * static_cast<size_t>(dec4_ctas(g.D, nt)) * dec_part_floats(g.D, 8 * nt) * 4;
}

cudaError_t launch_paged4_decode(const void* q, const Cache4& c4, const int32_t* page_table, const int32_t* seq_lens,
                                 const PagedGeom& g, void* out, float* lse, void* workspace, int32_t* status,
                                 cudaStream_t st) {
  const bool two = dec_head_tiles(g.D, g.G) == 2, fold = g.G <= 4;
#define BD_DECODE4(...) launch_dn<__VA_ARGS__>(q, c4, page_table, seq_lens, g, out, lse, workspace, status, st)
  switch (g.D) {
    case 64: return two ? BD_DECODE4(64, 2) : fold ? BD_DECODE4(64, 1, true) : BD_DECODE4(64, 1);
    case 128: return two ? BD_DECODE4(128, 2) : fold ? BD_DECODE4(128, 1, true) : BD_DECODE4(128, 1);
    case 256: return two ? BD_DECODE4(256, 2) : fold ? BD_DECODE4(256, 1, true) : BD_DECODE4(256, 1);
    case 512: return fold ? BD_DECODE4(512, 1, true) : BD_DECODE4(512, 1);
    default: return cudaErrorInvalidValue;
  }
#undef BD_DECODE4
}

}  // namespace bd
