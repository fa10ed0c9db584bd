// Attention of several query rows per sequence over the paged cache: causal
// prompts (pa_prefill_attention) and trees of drafted tokens
// (pa_tree_attention).
//   out[t][h] = sum_p softmax_p(scale q[t][h] . k_p) v_p
// over the cache positions p that token t of its sequence attends: all
// positions up to its own (prompt), or the whole prefix and the drafted tokens
// its mask names (tree).  A row that attends nothing gives zeros.
//
// One warp per (token, query head): 4 head dimensions a lane, the running
// maximum and sum of the softmax in one pass over the positions.
#include <algorithm>
#include <cstring>

#include "device_common.cuh"
#include "pa_internal.h"

namespace pa {
namespace {

struct AttendParams {
  const uint8_t* q;
  uint8_t* out;
  const uint8_t* k_cache;
  const uint8_t* v_cache;
  const int32_t* tables;
  const uint64_t* mask;     // tree: per packed row, or null (causal)
  const float* k_scale;
  const float* v_scale;
  uint32_t* err;
  int64_t rows;             // (tokens of this launch) x query heads
  float sl2;                // scale * log2(e)
  int32_t layer, H, G, num_blocks, mbps, bshift;
  AttendItems items;
};

template <int KV, int ACT>
__device__ __forceinline__ void load4(const uint8_t* p, int64_t el, float (&x)[4]) {
  if constexpr (KV == kFP8) {
    const uint32_t r = *reinterpret_cast<const uint32_t*>(p + el);
    const uint32_t a = dev::e4m3x2_to_f16x2(static_cast<uint16_t>(r)), b = dev::e4m3x2_to_f16x2(static_cast<uint16_t>(r >> 16));
    x[0] = dev::f16lo_to_f32(a);
    x[1] = dev::f16hi_to_f32(a);
    x[2] = dev::f16lo_to_f32(b);
    x[3] = dev::f16hi_to_f32(b);
  } else {
    const uint2 r = *reinterpret_cast<const uint2*>(p + el * 2);
    if constexpr (ACT == kBF16) {
      x[0] = dev::bf16lo_to_f32(r.x);
      x[1] = dev::bf16hi_to_f32(r.x);
      x[2] = dev::bf16lo_to_f32(r.y);
      x[3] = dev::bf16hi_to_f32(r.y);
    } else {
      x[0] = dev::f16lo_to_f32(r.x);
      x[1] = dev::f16hi_to_f32(r.x);
      x[2] = dev::f16lo_to_f32(r.y);
      x[3] = dev::f16hi_to_f32(r.y);
    }
  }
}

template <int KV, int ACT>
__global__ void __launch_bounds__(256) attend_kernel(const __grid_constant__ AttendParams prm) {
  dev::grid_dep_wait();
  const int lane = threadIdx.x & 31;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  if (row >= prm.rows) return;
  const int32_t hq = prm.H * prm.G;
  const int32_t tok = static_cast<int32_t>(row / hq), qh = static_cast<int32_t>(row % hq), h = qh / prm.G;
  const AttendItems& I = prm.items;
  int lo = 0, hi = I.n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (I.q0[mid] <= tok) lo = mid; else hi = mid - 1;
  }
  const int32_t t = tok - I.q0[lo], m = I.q0[lo + 1] - I.q0[lo], len = I.kv_len[lo], past = len - m;
  const int32_t end = prm.mask ? len : past + t + 1;
  const uint64_t mask = prm.mask ? prm.mask[I.row0 + tok] : 0;
  float q[4], o[4] = {0.f, 0.f, 0.f, 0.f}, mx = -INFINITY, l = 0.f;
  const int64_t qel = (static_cast<int64_t>(I.row0 + tok) * hq + qh) * kHeadDim + lane * 4;
  load4<kBF16, ACT>(prm.q, qel, q);
  const float sl2 = prm.sl2 * (KV == kFP8 ? prm.k_scale[prm.layer * prm.H + h] : 1.f);
  const int32_t* table = prm.tables + static_cast<int64_t>(I.row[lo]) * prm.mbps;
  for (int32_t p = 0; p < end; ++p) {
    if (prm.mask && p >= past && !(mask >> (p - past) & 1)) continue;
    int32_t phys = table[p >> prm.bshift];
    if (static_cast<uint32_t>(phys) >= static_cast<uint32_t>(prm.num_blocks)) {
      if (lane == 0) atomicOr(prm.err, kErrBadBlock);
      phys = 0;
    }
    const int64_t el = ((((static_cast<int64_t>(prm.layer) * prm.num_blocks + phys) * prm.H + h) << prm.bshift) +
                        (p & ((1 << prm.bshift) - 1))) * kHeadDim + lane * 4;
    float k[4], v[4];
    load4<KV, ACT>(prm.k_cache, el, k);
    load4<KV, ACT>(prm.v_cache, el, v);
    float s = q[0] * k[0] + q[1] * k[1] + q[2] * k[2] + q[3] * k[3];
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
    s *= sl2;
    const float mn = fmaxf(mx, s);
    const float c = mx == -INFINITY ? 0.f : dev::exp2_approx(mx - mn);
    const float e = mn == -INFINITY ? 0.f : dev::exp2_approx(s - mn);
    l = l * c + e;
#pragma unroll
    for (int x = 0; x < 4; ++x) o[x] = o[x] * c + e * v[x];
    mx = mn;
  }
  const float inv = (l > 0.f ? 1.f / l : 0.f) * (KV == kFP8 ? prm.v_scale[prm.layer * prm.H + h] : 1.f);
  uint2 r;
  if constexpr (ACT == kBF16)
    r = make_uint2(dev::pack_bf16(o[0] * inv, o[1] * inv), dev::pack_bf16(o[2] * inv, o[3] * inv));
  else
    r = make_uint2(dev::pack_f16(o[0] * inv, o[1] * inv), dev::pack_f16(o[2] * inv, o[3] * inv));
  *reinterpret_cast<uint2*>(prm.out + qel * 2) = r;
}

}  // namespace

cudaError_t launch_attend(const PoolView& pool, const CacheMaps&, const AttendArgs& a, const AttendItems& items,
                          int num_sms, cudaStream_t stream, int* launches) {
  static thread_local AttendParams prm;
  prm.q = static_cast<const uint8_t*>(a.q);
  prm.out = static_cast<uint8_t*>(a.out);
  prm.k_cache = static_cast<const uint8_t*>(pool.k_cache);
  prm.v_cache = static_cast<const uint8_t*>(pool.v_cache);
  prm.tables = a.tables;
  prm.mask = a.mask;
  prm.k_scale = pool.k_scale;
  prm.v_scale = pool.v_scale;
  prm.err = pool.err;
  prm.rows = static_cast<int64_t>(items.q0[items.n]) * a.num_q_heads;
  prm.sl2 = a.scale * 1.4426950408889634f;
  prm.layer = a.layer;
  prm.H = pool.num_kv_heads;
  prm.G = a.num_q_heads / pool.num_kv_heads;
  prm.num_blocks = pool.num_blocks;
  prm.mbps = pool.mbps;
  prm.bshift = pool.block_size == 32 ? 5 : 4;
  prm.items = items;
  const dim3 grid(static_cast<unsigned>((prm.rows + 7) / 8));
  ++*launches;
  if (pool.kv_dtype == kFP8)
    return pool.act_dtype == kBF16 ? launch_pdl(attend_kernel<kFP8, kBF16>, grid, dim3(256), 0, stream, prm)
                                   : launch_pdl(attend_kernel<kFP8, kFP16>, grid, dim3(256), 0, stream, prm);
  return pool.act_dtype == kBF16 ? launch_pdl(attend_kernel<kBF16, kBF16>, grid, dim3(256), 0, stream, prm)
                                 : launch_pdl(attend_kernel<kFP16, kFP16>, grid, dim3(256), 0, stream, prm);
}

}  // namespace pa
