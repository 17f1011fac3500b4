// Last kernel of the backward with sink tokens: dk / dv of the key rows that
// several units of a K/V tile touch (see common.cuh).
//
// A sink's gradient sums over every later row of its document, so the backward
// cuts those rows into units (and, where the tiles are too few for the SMs, all
// rows and the heads); each leaves its fp32 share of the shared key rows in a
// slot of the workspace. Here every such row is the sum of its tile's slots,
// added in slot order -- the same order in every run, no atomics -- and rounded
// once to the gradient type. With n_sink rows per unit the cost is the launch; a
// finely cut backward moves whole 128-row tiles through L2. A backward with bf16
// gradients does it in the launch that rounds dq (359 -> 349 us at 2 x 32 heads x
// 4096 rows, D 128).
#include <cuda_bf16.h>
#include <cstdint>

#include "common.cuh"
#include "sm100_ptx.cuh"

namespace bd {

constexpr int kSumThreads = 256;

// CTA `cta` of `ctas`: its share of the sums.
__device__ __forceinline__ void sum_slots(const int32_t* __restrict__ seg, const Geom& g, void* __restrict__ dk,
                                          void* __restrict__ dv, int grads_bf16, long long cta, long long ctas) {
  if (sink_n_units(g, seg) < 0) return;  // reported by the main kernel
  const int n_sums = seg[g.sk_off + 1] < g.sk_sums ? seg[g.sk_off + 1] : g.sk_sums;
  const int32_t* sums = seg + g.sk_off + kSinkHdrWords + static_cast<size_t>(g.sk_units) * kSinkUnitWords;
  const int vpr = g.D / 4, per = g.sk_rows * vpr;  // 4-element pieces of a row, of a slot's dk or dv
  const int cuts = (2 * per + kSumThreads - 1) / kSumThreads;  // CTAs' worth of pieces of a (sum, kv head)
  const size_t slot_step = static_cast<size_t>(g.Hkv) * 2 * per;
  for (long long x = cta; x < static_cast<long long>(n_sums) * g.Hkv * cuts; x += ctas) {
    const int y = static_cast<int>(x % cuts) * kSumThreads + threadIdx.x;
    if (y >= 2 * per) continue;
    const int32_t* e = sums + (x / cuts / g.Hkv) * kSinkSumWords;
    const int hk = static_cast<int>(x / cuts % g.Hkv), item = e[0], slot0 = e[1], n = e[2], rbase = e[3];
    if (item < 0 || item >= g.B * g.nkt || slot0 < 0 || n < 0 || slot0 + n > g.sk_slots) continue;
    const int b = item / g.nkt, kt = item % g.nkt;
    const int which = y / per, row = y % per / vpr, c4 = y % vpr;
    const int r = rbase + row, j = kt * kTile + r;
    if (r >= kTile || j >= g.S_kv) continue;
    const float4* p = reinterpret_cast<const float4*>(unit_part(g, slot0, hk, which, row)) + c4;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
    for (int k = 0; k < n; ++k) {
      const float4 v = p[k * slot_step];
      a.x += v.x;
      a.y += v.y;
      a.z += v.z;
      a.w += v.w;
    }
    void* out = which ? dv : dk;
    const size_t at = kv_row(g, b, hk, j) * vpr + c4;
    if (grads_bf16)
      static_cast<uint2*>(out)[at] = make_uint2(pack_bf16x2(a.x, a.y), pack_bf16x2(a.z, a.w));
    else
      static_cast<float4*>(out)[at] = a;
  }
}

__global__ void __launch_bounds__(kSumThreads) sink_sum_kernel(const int32_t* __restrict__ seg, const Geom g,
                                                               void* __restrict__ dk, void* __restrict__ dv,
                                                               int grads_bf16, const int32_t* status) {
  pdl_begin();
  if (*reinterpret_cast<const volatile int*>(status) != 0) return;
  sum_slots(seg, g, dk, dv, grads_bf16, blockIdx.x, gridDim.x);
}

// The sums and, by the other CTAs, dq = the fp32 accumulator rounded to bf16
// (n8 pieces of 8): one launch ends a backward with bf16 gradients.
__global__ void __launch_bounds__(kSumThreads)
    sink_finalize_kernel(const int32_t* __restrict__ seg, const Geom g, int sum_ctas, void* __restrict__ dk,
                         void* __restrict__ dv, const float4* __restrict__ dq_acc, uint4* __restrict__ dq,
                         long long n8, const int32_t* status) {
  pdl_begin();
  if (*reinterpret_cast<const volatile int*>(status) != 0) return;
  if (static_cast<int>(blockIdx.x) < sum_ctas) {
    sum_slots(seg, g, dk, dv, 1, blockIdx.x, sum_ctas);
    return;
  }
  const long long step = static_cast<long long>(gridDim.x - sum_ctas) * kSumThreads;
  for (long long t = static_cast<long long>(blockIdx.x - sum_ctas) * kSumThreads + threadIdx.x; t < n8; t += step) {
    const float4 a = dq_acc[2 * t], c = dq_acc[2 * t + 1];
    dq[t] = make_uint4(pack_bf16x2(a.x, a.y), pack_bf16x2(a.z, a.w), pack_bf16x2(c.x, c.y), pack_bf16x2(c.z, c.w));
  }
}

static int sum_ctas(const Geom& g) {
  const long long n = static_cast<long long>(g.sk_sums) * g.Hkv *
                      ((2LL * g.sk_rows * g.D / 4 + kSumThreads - 1) / kSumThreads);
  return static_cast<int>(n < kSms * 8 ? n : kSms * 8);
}

cudaError_t launch_sink_sum(const int32_t* seg, const Geom& g, void* dk, void* dv, int bf16, int32_t* status,
                            cudaStream_t st) {
  const int n = sum_ctas(g);
  if (n == 0) return cudaSuccess;  // every tile has one unit
  if (const cudaError_t le = launch_pdl(sink_sum_kernel, dim3(n), dim3(kSumThreads), 0, st, seg, g, dk, dv, bf16, status);
      le != cudaSuccess) return le;
  return cudaGetLastError();
}

cudaError_t launch_sink_finalize(const int32_t* seg, const Geom& g, void* dk, void* dv, void* workspace, void* dq,
                                 int32_t* status, cudaStream_t st) {
  const long long n8 = static_cast<long long>(g.B) * g.Hq * g.L * g.D / 8;
  const long long want = (n8 + kSumThreads - 1) / kSumThreads;
  const int sums = sum_ctas(g), conv = static_cast<int>(want < kSms * 16 ? want : kSms * 16);
  if (const cudaError_t le = launch_pdl(sink_finalize_kernel, dim3(sums + conv), dim3(kSumThreads), 0, st, seg, g, sums,
                                        dk, dv, static_cast<const float4*>(workspace), static_cast<uint4*>(dq), n8,
                                        static_cast<const int32_t*>(status));
      le != cudaSuccess) return le;
  return cudaGetLastError();
}

}  // namespace bd
