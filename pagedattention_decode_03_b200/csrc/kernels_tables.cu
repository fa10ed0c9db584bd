// Device-side bookkeeping of a serving step whose request lengths live on the
// GPU:
//   * build_tables   -- block tables and the slot map of the new tokens from
//                       request lengths and a list of free block ids
//                       ("Managing the KV Cache", Block Tables and Sharing and
//                       Answer Key item 2, as the host block manager does it);
//   * append_slots   -- K/V rows into the cache slots that map names (FP8 pools
//                       quantise as pa_append_kv does, "Managing the KV Cache",
//                       Quantized KV).
#include <algorithm>
#include <cstring>

#include "device_common.cuh"
#include "pa_internal.h"

namespace pa {
namespace {

// ------------------------------------------------------------ build_tables
// need_i = ceil(new_i / B) - ceil(old_i / B) fresh blocks and new_i - old_i new
// tokens of request i; exclusive sums of both over the requests place a
// request's ids in the free list and its tokens in the slot map.  Every CTA
// computes both sums for itself in shared memory (n is at most kTablesMaxSeqs:
// a few loads a thread, cheaper than a second launch or a grid-wide wait), then
// takes its grid-strided part of the fresh table entries and of the slots,
// finding each one's request by a binary search in the sums.
// A slot's block is read from the free list when it is fresh, so no CTA waits
// for the table entries another one writes.  Bound by latency: lengths, sums, ids and
// slots follow one another (64 requests 3.6 us, 509 prompts with 1 M slots 7.9 us; the
// slots alone are 4 MB, 0.7 us).

struct TablesParams {
  const int32_t* old_lens;
  const int32_t* new_lens;
  const int32_t* free_blocks;
  const int32_t* free_head;
  int32_t* free_head_out;
  int32_t* tables;
  int32_t* cu;
  int32_t* slots;
  int32_t* ticket;   // zero between launches
  uint32_t* err;
  int32_t n, num_free, mbps, bshift, num_blocks, cap;  // bshift: log2(block_size)
};

// Largest i with pre[i] <= x (pre[0] = 0, ascending, n entries).
__device__ __forceinline__ int last_at_or_below(const int32_t* pre, int n, int32_t x) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (pre[mid] <= x) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// SPT: consecutive slots of a thread, which share a search and mostly a block.
template <int SPT, int kTablesThreads>
__global__ void __launch_bounds__(kTablesThreads) build_tables_kernel(const __grid_constant__ TablesParams prm) {
  constexpr int kTablesWarps = kTablesThreads / 32;
  extern __shared__ int32_t sm[];
  int32_t* tok = sm;                  // [n + 1] tokens before request i
  int32_t* blk = sm + prm.n + 1;      // [n + 1] fresh blocks before request i
  int32_t* old = blk + prm.n + 1;     // [n] length before the step
  __shared__ int64_t warp_tok[kTablesWarps], warp_blk[kTablesWarps];
  __shared__ int32_t head_s, fail_s;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int32_t B = 1 << prm.bshift;
  dev::grid_dep_wait();
  dev::grid_dep_launch();

  // each thread sums its run of consecutive requests, then a scan over threads
  const int per = (prm.n + kTablesThreads - 1) / kTablesThreads;
  const int i0 = min(prm.n, tid * per), i1 = min(prm.n, i0 + per);
  const int64_t max_len = min(static_cast<int64_t>(prm.mbps) << prm.bshift, static_cast<int64_t>(kMaxLen));
  int64_t st = 0, sb = 0;
  for (int i = i0; i < i1; ++i) {
    int32_t a = prm.old_lens[i], b = prm.new_lens[i];
    if (a < 0 || b < a || b > max_len) {  // the request is left as it is
      atomicOr(prm.err, kErrBadLen);
      a = b = 0;
    }
    old[i] = a;
    tok[i] = b - a;
    blk[i] = static_cast<int32_t>(((static_cast<int64_t>(b) + B - 1) >> prm.bshift) -
                                  ((static_cast<int64_t>(a) + B - 1) >> prm.bshift));
    st += tok[i];
    sb += blk[i];
  }
  int64_t ct = st, cb = sb;  // inclusive over the warp's lanes
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t ut = __shfl_up_sync(0xffffffffu, ct, o), ub = __shfl_up_sync(0xffffffffu, cb, o);
    if (lane >= o) {
      ct += ut;
      cb += ub;
    }
  }
  if (lane == 31) {
    warp_tok[warp] = ct;
    warp_blk[warp] = cb;
  }
  if (tid == 0) head_s = *prm.free_head;
  __syncthreads();
  int64_t bt = 0, bb = 0, tt = 0, tb = 0;  // before this warp; totals
#pragma unroll
  for (int w = 0; w < kTablesWarps; ++w) {
    if (w < warp) {
      bt += warp_tok[w];
      bb += warp_blk[w];
    }
    tt += warp_tok[w];
    tb += warp_blk[w];
  }
  const int32_t head = head_s;
  if (tid == 0) {
    // all or nothing: too few free ids, or a slot map too short for the tokens
    uint32_t bad = 0;
    if (head < 0 || head > prm.num_free || tb > prm.num_free - head) bad |= kErrNoBlocks;
    if (tt > prm.cap) bad |= kErrBadLen;
    fail_s = bad != 0;
    if (bad) atomicOr(prm.err, bad);
  }
  int64_t et = bt + ct - st, eb = bb + cb - sb;
  for (int i = i0; i < i1; ++i) {
    const int32_t dt = tok[i], db = blk[i];
    tok[i] = static_cast<int32_t>(et);
    blk[i] = static_cast<int32_t>(eb);
    et += dt;
    eb += db;
  }
  if (tid == 0) {
    tok[prm.n] = static_cast<int32_t>(tt);
    blk[prm.n] = static_cast<int32_t>(tb);
  }
  __syncthreads();
  const bool failed = fail_s != 0;

  if (blockIdx.x == 0)
    for (int i = tid; i <= prm.n; i += kTablesThreads) prm.cu[i] = failed ? 0 : tok[i];

  const int64_t gid = static_cast<int64_t>(blockIdx.x) * kTablesThreads + tid;
  const int64_t gsize = static_cast<int64_t>(gridDim.x) * kTablesThreads;
  const int32_t total = failed ? 0 : tok[prm.n];
  const bool aligned = (reinterpret_cast<uintptr_t>(prm.slots) & 15) == 0;
  for (int64_t t0 = gid * SPT; t0 < prm.cap; t0 += gsize * SPT) {
    int i = t0 < total ? last_at_or_below(tok, prm.n, static_cast<int32_t>(t0)) : 0;
    int32_t lb0 = -1, i_of = -1, phys = 0;
#pragma unroll
    for (int q = 0; q < SPT; q += 4) {
      int32_t v[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int64_t t = t0 + q + k;
        v[k] = -1;
        if (t >= total) continue;
        while (tok[i + 1] <= t) ++i;
        const int32_t pos = old[i] + static_cast<int32_t>(t) - tok[i];
        const int32_t lb = pos >> prm.bshift;
        if (lb != lb0 || i != i_of) {
          const int32_t have = (old[i] + B - 1) >> prm.bshift;
          phys = lb < have ? prm.tables[static_cast<int64_t>(i) * prm.mbps + lb]
                           : prm.free_blocks[head + blk[i] + lb - have];
          lb0 = lb;
          i_of = i;
          if (static_cast<uint32_t>(phys) >= static_cast<uint32_t>(prm.num_blocks)) atomicOr(prm.err, kErrBadBlock);
        }
        if (static_cast<uint32_t>(phys) < static_cast<uint32_t>(prm.num_blocks))
          v[k] = (phys << prm.bshift) + (pos & (B - 1));
      }
      if (aligned && t0 + q + 4 <= prm.cap) {
        *reinterpret_cast<int4*>(prm.slots + t0 + q) = make_int4(v[0], v[1], v[2], v[3]);
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (t0 + q + k < prm.cap) prm.slots[t0 + q + k] = v[k];
      }
    }
  }
  if (!failed)
    // (from the last thread on: in a small call others than those that list slots)
    for (int64_t e = gsize - 1 - gid; e < blk[prm.n]; e += gsize) {
      const int i = last_at_or_below(blk, prm.n, static_cast<int32_t>(e));
      const int32_t have = (old[i] + B - 1) >> prm.bshift;
      prm.tables[static_cast<int64_t>(i) * prm.mbps + have + (e - blk[i])] = prm.free_blocks[head + e];
    }
  // Every CTA has read the head before it counts itself in here, so the last one
  // may replace it even where both pointers name the same word.
  if (tid == 0) {
    bool last = gridDim.x == 1;
    if (!last) {
      __threadfence();
      last = atomicAdd(prm.ticket, 1) == static_cast<int32_t>(gridDim.x) - 1;
      if (last) *prm.ticket = 0;
    }
    if (last) *prm.free_head_out = failed ? head : head + blk[prm.n];
  }
}

// ------------------------------------------------------------ append_slots
// A copy bound by HBM: one thread moves 16 bytes of a 16-bit row (32 bytes of
// the source where it quantises to 16 bytes of FP8 codes), K and V together.
// The source loads do not depend on the slot, so all three are in flight at once.
// 32,749 rows of 8 heads to FP8: 35.0 us, 5.75 TB/s of the 6.47 that a copy reaches.
struct SlotsParams {
  const uint8_t* k_new;  // [T][H][128] act dtype
  const uint8_t* v_new;
  uint8_t* k_cache;
  uint8_t* v_cache;
  const float* k_inv;    // [L][H] fp32 (FP8 pools)
  const float* v_inv;
  const int32_t* slots;  // [T]
  uint32_t* err;
  int64_t layer_off;     // elements before this layer
  int64_t jobs;          // T * H * chunks of a row
  int32_t H, bshift, layer;
  int64_t num_slots;     // num_blocks * block_size
};

template <int ACT>
__device__ __forceinline__ uint2 quantise8(uint4 x, float inv) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint16_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float lo = ACT == kBF16 ? dev::bf16lo_to_f32(w[i]) : dev::f16lo_to_f32(w[i]);
    const float hi = ACT == kBF16 ? dev::bf16hi_to_f32(w[i]) : dev::f16hi_to_f32(w[i]);
    c[i] = dev::f32x2_to_e4m3x2(__fmul_rn(lo, inv), __fmul_rn(hi, inv));
  }
  return make_uint2(c[0] | (static_cast<uint32_t>(c[1]) << 16), c[2] | (static_cast<uint32_t>(c[3]) << 16));
}

template <int KV, int ACT>
__global__ void __launch_bounds__(256) append_slots_kernel(const __grid_constant__ SlotsParams prm) {
  dev::grid_dep_wait();
  dev::grid_dep_launch();
  constexpr int kChunks = KV == kFP8 ? 8 : 16;  // of one row
  const int64_t job = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (job >= prm.jobs) return;
  const int c = static_cast<int>(job % kChunks);
  const int64_t row = job / kChunks;
  const int32_t h = static_cast<int32_t>(row % prm.H);
  const int64_t t = row / prm.H;
  const int32_t slot = prm.slots[t];
  const uint4* ks = reinterpret_cast<const uint4*>(prm.k_new) + row * 16;
  const uint4* vs = reinterpret_cast<const uint4*>(prm.v_new) + row * 16;
  const int64_t blk = slot >> prm.bshift;
  const int64_t off = slot & ((1 << prm.bshift) - 1);
  const int64_t dst = prm.layer_off + (((blk * prm.H + h) << prm.bshift) + off) * kHeadDim;
  const bool ok = slot >= 0 && slot < prm.num_slots;
  if constexpr (KV == kFP8) {
    const uint4 k0 = __ldcs(ks + 2 * c), k1 = __ldcs(ks + 2 * c + 1);
    const uint4 v0 = __ldcs(vs + 2 * c), v1 = __ldcs(vs + 2 * c + 1);
    const float ki = prm.k_inv[prm.layer * prm.H + h], vi = prm.v_inv[prm.layer * prm.H + h];
    if (ok) {
      const uint2 ka = quantise8<ACT>(k0, ki), kb = quantise8<ACT>(k1, ki);
      const uint2 va = quantise8<ACT>(v0, vi), vb = quantise8<ACT>(v1, vi);
      *reinterpret_cast<uint4*>(prm.k_cache + dst + c * 16) = make_uint4(ka.x, ka.y, kb.x, kb.y);
      *reinterpret_cast<uint4*>(prm.v_cache + dst + c * 16) = make_uint4(va.x, va.y, vb.x, vb.y);
    }
  } else {
    const uint4 k0 = __ldcs(ks + c), v0 = __ldcs(vs + c);
    if (ok) {
      *reinterpret_cast<uint4*>(prm.k_cache + dst * 2 + c * 16) = k0;
      *reinterpret_cast<uint4*>(prm.v_cache + dst * 2 + c * 16) = v0;
    }
  }
  if (slot != -1 && !ok && c == 0 && h == 0) atomicOr(prm.err, kErrBadBlock);
}

}  // namespace

cudaError_t launch_build_tables(const PoolView& pool, int n, const int32_t* old_lens, const int32_t* new_lens,
                                const int32_t* free_blocks, int num_free, const int32_t* free_head,
                                int32_t* free_head_out, int32_t* tables, int32_t* cu, int32_t* slots, int cap,
                                int num_sms, cudaStream_t stream) {
  TablesParams prm;
  prm.old_lens = old_lens;
  prm.new_lens = new_lens;
  prm.free_blocks = free_blocks;
  prm.free_head = free_head;
  prm.free_head_out = free_head_out;
  prm.tables = tables;
  prm.cu = cu;
  prm.slots = slots;
  prm.ticket = pool.counters;
  prm.err = pool.err;
  prm.n = n;
  prm.num_free = num_free;
  prm.mbps = pool.mbps;
  prm.bshift = pool.block_size == 32 ? 5 : 4;
  prm.num_blocks = pool.num_blocks;
  prm.cap = cap;
  const size_t smem = (static_cast<size_t>(n) * 3 + 2) * sizeof(int32_t);
  // Few slots: 4 a thread, for the shortest way through one CTA's, of 128 threads
  // where they are enough.  Many: 16, one block's worth, so that a search and a block
  // id serve them all: 509 prompts with 1 M slots 7.9 us; 4 a thread on two or four
  // CTAs an SM took 8.4 and 10.9 us.
  const bool many = cap > num_sms * 512 * 4, few = n <= 128 && cap <= 512;
  auto* kernel = many ? build_tables_kernel<16, 512> : few ? build_tables_kernel<4, 128> : build_tables_kernel<4, 512>;
  const int threads = few ? 128 : 512;
  // (48 KB need no asking for, but the kernel's static arrays, under 1 KB, count as well)
  if (smem > 47 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               static_cast<int>((kTablesMaxSeqs * 3 + 2) * sizeof(int32_t)));
    if (e != cudaSuccess) return e;
  }
  const int64_t per = static_cast<int64_t>(threads) * (many ? 16 : 4);
  const int grid = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(num_sms, (cap + per - 1) / per)));
  return launch_with(many || stream != nullptr, kernel, dim3(grid), dim3(threads), smem, stream, prm);
}

cudaError_t launch_append_slots(const PoolView& pool, int layer, int T, const int32_t* slots, const void* k_new,
                                const void* v_new, cudaStream_t stream) {
  SlotsParams prm;
  prm.k_new = static_cast<const uint8_t*>(k_new);
  prm.v_new = static_cast<const uint8_t*>(v_new);
  prm.k_cache = static_cast<uint8_t*>(pool.k_cache);
  prm.v_cache = static_cast<uint8_t*>(pool.v_cache);
  prm.k_inv = pool.k_inv;
  prm.v_inv = pool.v_inv;
  prm.slots = slots;
  prm.err = pool.err;
  prm.layer_off = static_cast<int64_t>(layer) * pool.num_blocks * pool.num_kv_heads * pool.block_size * kHeadDim;
  prm.H = pool.num_kv_heads;
  prm.bshift = pool.block_size == 32 ? 5 : 4;
  prm.layer = layer;
  prm.num_slots = static_cast<int64_t>(pool.num_blocks) * pool.block_size;
  const bool fp8 = pool.kv_dtype == kFP8;
  prm.jobs = static_cast<int64_t>(T) * prm.H * (fp8 ? 8 : 16);
  const int64_t blocks = (prm.jobs + 255) / 256;
  if (blocks > INT32_MAX) return cudaErrorInvalidValue;
  const dim3 grid(static_cast<unsigned>(blocks));
  // On the legacy default stream only a call that takes the GPU longer than the host
  // overlaps: the launch itself is dearer then (64 rows 5.6 -> 7.5 us a call; 32,749
  // rows 36.9 -> 35.0 us).
  const bool overlap = stream != nullptr || blocks > 1024;
  auto* kernel = !fp8 ? append_slots_kernel<kBF16, kBF16>
                 : pool.act_dtype == kBF16 ? append_slots_kernel<kFP8, kBF16> : append_slots_kernel<kFP8, kFP16>;
  return launch_with(overlap, kernel, grid, dim3(256), 0, stream, prm);
}

}  // namespace pa
