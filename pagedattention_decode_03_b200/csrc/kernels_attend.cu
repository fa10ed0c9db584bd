// Attention of several query rows per sequence over the paged cache: causal
// prompts (pa_prefill_attention) and trees of drafted tokens
// (pa_tree_attention), on the 5th-generation tensor cores (tcgen05).
//   out[t][h] = sum_p softmax_p(scale q[t][h] . k_p) v_p
// over the cache positions p that token t of its sequence attends: all
// positions up to its own (prompt), or the whole prefix and the drafted tokens
// its mask names (tree).  A row that attends nothing gives zeros.
//
// A tile of queries is 128 rows of one KV head: 128 / G tokens x the G query
// heads that share it (row = token * G + head in group), so a KV tile is read
// once for the whole group and a tree's few tokens still fill rows.  Per tile
// of 128 cache positions
//   S[128 rows][128 positions] = Q K^T        (A, B from shared memory)
//   O[128 rows][128 d]        += P V          (A = P from tensor memory,
//                                              B = the V tile read MN-major)
// with fp32 S and O in tensor memory; P, 16-bit, overlays S.  One CTA per SM
// runs two softmax streams so that one stream's exponentials overlap the other
// one's products:
//   pair  the streams are two query tiles over the same KV tiles (256 rows a
//         KV read: prompts, wide trees);
//   dual  both streams serve one query tile and take every other KV tile; their
//         results are joined in the epilogue (few rows: bound by the KV read).
// Roles: warp 0 claims work and loads queries, warps 0 and 2 issue the KV tiles'
// TMA copies, warp 1 issues the MMAs, warp 3 zeroes V rows past a length, warps
// 4-7 and 8-11 are the two softmax streams (a thread owns a row: its running
// maximum and sum need no exchange), warps 12-15 convert FP8 codes to fp16 (exact,
// one instruction a pair; bf16 queries then become fp16 times a power of two a row).
// Work units are claimed from a counter, longest first.  Where there are too
// few units for the SMs the positions are split into chunks whose partial
// results (O, maximum, sum) a second kernel joins.
// Measured on one B200 (64 query / 8 KV heads unless named): prompts of 9,001 and
// 7,003 tokens, bf16, 2.02 ms = 1.06 PFLOP/s under the power limit (1.2 in a burst);
// chunks over FP8 caches 0.90 PFLOP/s; trees of 40 to 64 drafts, 32 heads, fp16, 104 us
// = 5.5 TB/s in a burst, 124 us sustained; eight trees of 20 to 33 drafts over 31,000
// FP8 tokens 355 us, where the conversion is what a tile waits for.  A pair of tiles of
// the long prompts takes 3,620 cycles, of which the tensor core needs 2,048; a stream
// waits 1,390 for its S, loads it in 185, makes weights and maximum in 1,650, stores and
// hands over in 150, and spends 7,900 a unit on the epilogue and the next unit's start,
// 245 a tile here.
// Every wait is bounded; one that gives up sets PA_DEVERR_TIMEOUT, and the CTA
// waits for its copies and MMAs, frees its tensor memory and returns.
#include <algorithm>
#include <cmath>
#include <cstring>
#include <mutex>
#include <type_traits>

#include "device_common.cuh"
#include "pa_internal.h"

namespace pa {
namespace {

constexpr uint32_t kWaitLimit = 1u << 22;
constexpr float kLog2e = 1.4426950408889634f;
constexpr int kTile = 128;                      // rows of a query tile, positions of a KV tile
constexpr int kHalf = kTile * 128;              // one 64-element d-half of a 16-bit tile (16 KB)
constexpr int kGroup = 8 * 128;                 // 8 tokens of one d-half in a KV tile (1 KB)
constexpr int kOperand = 2 * kHalf;             // a 16-bit tile (32 KB)
constexpr int kLoaders = 2;                     // warps that issue a tile's copies, 8 / kLoaders blocks each
constexpr int kRaw = kTile * 128;               // an FP8 tile (16 KB)
constexpr int kPartFloats = kHeadDim + 2;       // of one row: O, maximum, sum, each a line of rows
// A row's weights are 2^(score - reference + kBias); its reference follows the
// running maximum only when that passes it by kLazy (in log2 units).  bf16 has
// fp32's range, so any lag will do; fp16 weights stay under 2^(kLazy + kBias) =
// 2^15, and are normal numbers down to 2^-26 of the reference's.
// They are rounded once to the operands' type.  A second product with what that leaves
// out, as the decode makes it for bf16, took bf16 results from 2.1e-3 of their norm to
// 1.65e-3, where their own rounding alone is 1.64e-3 (fp16: 2.6e-4 to 2.1e-4), and long
// prompts from 2.02 to 2.91 ms, 47 trees from 44 to 55 us, FP8 trees from 365 to 520 us.
template <int MMA>
constexpr float kLazy = MMA == kBF16 ? 8.f : 3.f;
template <int MMA>
constexpr float kBias = MMA == kBF16 ? 0.f : 12.f;
// From here on the rounding of a scaled score takes up what the weights' type has room
// for (a step of fp32 is 1/8 at 2^20; fp16 weights pass their largest number from scores
// of 2^24 on, bf16 ones from 2^31): the rest of such a unit is computed apart.
constexpr float kFar = 1 << 20;

// Ring depths: up to 224 KB of the SM's 227.
template <bool PAIR, bool FP8>
struct Ring {
  static constexpr int kQ = PAIR ? 2 : 1;
  static constexpr int kStages = FP8 ? (PAIR ? 3 : 4) : 5;
  static constexpr int kRawStages = FP8 ? (PAIR ? 4 : 3) : 0;
  static constexpr int kThreads = FP8 ? 512 : 384;
  // Registers a thread: at launch (65,536 over the threads), then by role.  The
  // softmax keeps a whole row of S; the shares add up to the launch's total.
  static constexpr int kRegsLaunch = FP8 ? 128 : 168;
  static constexpr int kRegsControl = FP8 ? 64 : 120;
  static constexpr int kRegsSoftmax = FP8 ? 184 : 192;
  static constexpr int kRegsConvert = FP8 ? 80 : 0;
  static_assert(kRegsControl + 2 * kRegsSoftmax + kRegsConvert <= kRegsLaunch * (kThreads / 128), "register shares");
  static constexpr int kOffKv = kQ * kOperand;
  static constexpr int kOffRaw = kOffKv + kStages * kOperand;
  static constexpr int kOffMeta = kOffRaw + kRawStages * kRaw;
};

// What the roles of a CTA know of a work unit.
struct Unit {
  int32_t seq_row;      // row of the block tables; < 0: no more work
  int32_t h;            // KV head
  int32_t tok0;         // packed row of the unit's first token
  int32_t t0, m;        // first token within its sequence's query tokens, and their number
  int32_t past, kv_len; // positions before the query tokens; all positions
  int32_t tile0;        // first KV tile (pair: 0)
  int32_t n0, n1;       // KV tiles of stream 0 / 1 (dual: n0 = all tiles)
  int32_t part;         // partial index of the unit (dual)
  int32_t direct;       // the unit has all its positions here and writes the output
  int32_t end0, end1;   // 16-position steps that any row attends in the stream's last tile (dual: the last tile)
};

struct Meta {
  uint64_t kv_full[6], kv_empty[6], raw_full[6], raw_empty[6];
  uint64_t q_full[2], q_empty[2], s_full[2], p_full[2], o_full[2], o_free[2], ml[2];
  uint64_t sched_full[2], sched_empty[2], done, clean_go, clean_done, q_ready[2];
  Unit unit[2];
  uint32_t tmem;
  int32_t abort;
  // [unit % 4][stream][row]: queries are held as q 2^-exp (FP8 caches, bf16).  The
  // queries of two units may be converted while a stream still works on the one
  // before them (units of one or two tiles); a third waits for its epilogue.
  int8_t q_exp[4][2][kTile];
  int32_t rows[kLoaders][8][8 / kLoaders];  // cache rows of the last 8 tiles' blocks
  float mlv[2][2][2][kTile];  // [unit parity][stream][max, sum][row] (dual)
};

template <bool PAIR, bool FP8>
constexpr size_t smem_bytes() {
  return 1024 + Ring<PAIR, FP8>::kOffMeta + sizeof(Meta) - (PAIR ? sizeof(Meta::mlv) : 0);
}

// Launch parameters, with room for CAP sequences: a call of few does not carry
// the tables of many (10 KB: 1 to 2 us a launch on the host).
template <int CAP>
struct Params {
  uint8_t* out;
  const int32_t* tables;
  const uint64_t* mask;     // tree: per packed row, or null (causal)
  const float* k_scale;
  const float* v_scale;
  float* partials;
  int32_t* counter;         // zero between launches
  uint32_t* err;
  float sl2;                // scale * log2(e)
  int32_t layer, H, gshift, num_blocks, mbps, bshift;  // gshift: log2(G); bshift: log2(block_size / 16)
  int32_t units;            // work units, all heads
  int32_t chunk;            // KV tiles of a chunk
  int32_t part_rows;        // rows of a partial
  int32_t n, row0;
  int32_t row[CAP];
  int32_t kv_len[CAP];
  int32_t q0[CAP];         // first query token, and
  int32_t m[CAP];          // how many
  int32_t pre[CAP + 1];    // prefix of (query tiles x chunks), per KV head
};

// ------------------------------------------------------------------- tcgen05
constexpr uint32_t kLayoutSW128 = 2;

// Shared-memory operand: start address, leading and stride byte offsets in
// 16-byte units, version 1, 128-byte swizzle.
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t lbo, uint32_t sbo) {
  return static_cast<uint64_t>((addr >> 4) & 0x3FFFu) | (static_cast<uint64_t>((lbo >> 4) & 0x3FFFu) << 16) |
         (static_cast<uint64_t>((sbo >> 4) & 0x3FFFu) << 32) | (uint64_t{1} << 46) |
         (static_cast<uint64_t>(kLayoutSW128) << 61);
}
// kind::f16, fp32 accumulators, M = 128, N; B K-major or MN-major.
constexpr uint32_t kNegateA = 1u << 13;
__host__ __device__ constexpr uint32_t instr_desc(bool bf16, bool b_mn, int N) {
  return (1u << 4) | (uint32_t(bf16) << 7) | (uint32_t(bf16) << 10) | (uint32_t(b_mn) << 16) |
         (uint32_t(N >> 3) << 17) | (uint32_t(128 >> 4) << 24);
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(acc))
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(acc))
      : "memory");
}
__device__ __forceinline__ void commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
               : "memory");
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// 32 columns of this thread's lane; the values are valid after tmem_wait.
__device__ __forceinline__ void tmem_ld32(uint32_t a, float (&v)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]),
        "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]),
        "=f"(v[16]), "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]),
        "=f"(v[24]), "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
      : "r"(a)
      : "memory");
}
// Waits for this thread's tensor-memory loads; v passes through, so no use of
// it can be scheduled before the wait.
__device__ __forceinline__ void tmem_wait(float (&v)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]),
                 "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]),
                 "+f"(v[15]), "+f"(v[16]), "+f"(v[17]), "+f"(v[18]), "+f"(v[19]), "+f"(v[20]), "+f"(v[21]),
                 "+f"(v[22]), "+f"(v[23]), "+f"(v[24]), "+f"(v[25]), "+f"(v[26]), "+f"(v[27]), "+f"(v[28]),
                 "+f"(v[29]), "+f"(v[30]), "+f"(v[31])::"memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t a, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(a),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t a, const uint32_t (&v)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(a), "r"(v[0]), "r"(v[1]),
               "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}
// 16 columns of this thread's lane, waited for.
__device__ __forceinline__ void tmem_ld16(uint32_t a, float (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]),
        "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
      : "r"(a)
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

template <int ACT>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  return ACT == kBF16 ? dev::pack_bf16(lo, hi) : dev::pack_f16(lo, hi);
}

// Two fp32 in one 64-bit register, and the packed operations on them.
__device__ __forceinline__ uint64_t pack_f32x2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpack_f32x2(uint64_t x, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(x));
}
__device__ __forceinline__ uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add_f32x2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

template <int N>
__device__ __forceinline__ void regs_more() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_less() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// Weight of a part of a row with maximum m and sum l, against the maximum of all
// parts: 0 for a part that attended nothing, NaN for one with a NaN in it (whose
// maximum may be -inf).
__device__ __forceinline__ float stream_weight(float m, float l, float all) {
  return l == 0.f ? 0.f : (l == l ? dev::exp2_approx(m - all) : l);
}

// Columns of a 32-column chunk whose first n are allowed.
__device__ __forceinline__ uint32_t low_bits(int32_t n) {
  return n >= 32 ? 0xffffffffu : (n <= 0 ? 0u : (1u << n) - 1u);
}

// ------------------------------------------------------------------- kernel
// Up to this many sequences a launch carries 1.3 KB of parameters instead of 10.  Room
// for 128 (2.9 KB) took calls of 1 to 48 sequences 0.5 us longer (16: 8.98 to 9.44 us) and
// saved those of 49 to 128 as much (64: 12.99 to 12.44 us): small calls go first.
constexpr int kSmallCap = 48;

template <int KV, int ACT, bool PAIR, int CAP>
__global__ void __launch_bounds__(Ring<PAIR, KV == kFP8>::kThreads, 1)
    attend_kernel(const __grid_constant__ Params<CAP> prm, const __grid_constant__ CUtensorMap tmk,
                  const __grid_constant__ CUtensorMap tmv, const __grid_constant__ CUtensorMap tmq) {
  constexpr bool kFp8 = KV == kFP8;
  constexpr int MMA = kFp8 ? kFP16 : ACT;        // type of the products' operands
  constexpr bool kScaleQ = kFp8 && ACT == kBF16;
  constexpr bool kSpec = MMA == kBF16;
  using R = Ring<PAIR, kFp8>;
  constexpr int kLead = PAIR ? 1 : 2;           // K tiles copied ahead of the V tile of step i
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* sm = smem_raw + (-dev::smem_u32(smem_raw) & 1023u);
  Meta& mt = *reinterpret_cast<Meta*>(sm + R::kOffMeta);
  const uint32_t base = dev::smem_u32(sm);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto bar = [&](const uint64_t& b) {
    return base + static_cast<uint32_t>(reinterpret_cast<const uint8_t*>(&b) - sm);
  };
  volatile int32_t* abort = &mt.abort;
  constexpr int kSchedConsumers = kLoaders + 8 + (kFp8 ? 4 : 1);  // warps that read a unit

  if (threadIdx.x == 0) {
    for (int s = 0; s < 6; ++s) {
      dev::mbar_init(bar(mt.kv_full[s]), kFp8 ? 4 : kLoaders);
      dev::mbar_init(bar(mt.kv_empty[s]), 1);
      dev::mbar_init(bar(mt.raw_full[s]), kLoaders);
      dev::mbar_init(bar(mt.raw_empty[s]), 4);
    }
    for (int x = 0; x < 2; ++x) {
      dev::mbar_init(bar(mt.q_full[x]), 1);
      dev::mbar_init(bar(mt.q_empty[x]), 1);
      dev::mbar_init(bar(mt.s_full[x]), 1);
      dev::mbar_init(bar(mt.p_full[x]), 4);
      dev::mbar_init(bar(mt.o_full[x]), 1);
      dev::mbar_init(bar(mt.o_free[x]), PAIR ? 4 : 8);
      dev::mbar_init(bar(mt.ml[x]), 4);
      dev::mbar_init(bar(mt.sched_full[x]), 1);
      dev::mbar_init(bar(mt.sched_empty[x]), kSchedConsumers);
    }
    dev::mbar_init(bar(mt.done), 1);
    dev::mbar_init(bar(mt.q_ready[0]), 4);
    dev::mbar_init(bar(mt.q_ready[1]), 4);
    dev::mbar_init(bar(mt.clean_go), 1);
    dev::mbar_init(bar(mt.clean_done), 1);
    mt.abort = 0;
    dev::fence_mbar_init();
    dev::tma_prefetch_desc(&tmk);
    dev::tma_prefetch_desc(&tmv);
    dev::tma_prefetch_desc(&tmq);
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dev::smem_u32(&mt.tmem)),
                 "n"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(&mt.tmem);
  // (each role waits for the kernel before this one before its first bounded wait,
  // so that kernel's time does not count against the limit; the schedule's first
  // unit comes from the parameters alone)

  // A warp's bounded wait, one outcome for all lanes; false ends the role.
  auto wait = [&](uint64_t& b, uint32_t parity) {
    const uint32_t a = bar(b);
    bool ok = false;
    for (uint32_t i = 0; i < kWaitLimit; ++i) {
      if (dev::mbar_try_wait(a, parity)) {
        ok = true;
        break;
      }
      if (*abort) break;
    }
    ok = __all_sync(0xffffffffu, ok);
    if (!ok && lane == 0 && *abort == 0) {
      *abort = 1;
      atomicOr(prm.err, kErrTimeout);
    }
    return ok;
  };
  uint32_t unit_i = 0;
  // The next unit, by the warps that consume the schedule.
  auto next_unit = [&](Unit& u) {
    if (!wait(mt.sched_full[unit_i & 1], (unit_i >> 1) & 1)) return false;
    u = mt.unit[unit_i & 1];
    __syncwarp();
    if (lane == 0) arrive(bar(mt.sched_empty[unit_i & 1]));
    ++unit_i;
    return u.seq_row >= 0;
  };

  // 16-bit tiles: the unit's last KV tile ends inside a block.
  auto needs_clean = [](const Unit& u, int32_t n) {
    const int32_t valid = u.kv_len - (u.tile0 + n - 1) * kTile;
    return !kFp8 && valid < kTile && (valid & 15);
  };

  // ------------------------------------------------------------------ loaders
  // KV tiles in ring order: K(0 .. kLead-1), then V(i), K(i + kLead), ...  One
  // warp gets a copy out every ~60 ns (a lane at a time), so kLoaders warps share
  // each tile's blocks and a block comes as one box.  A 16-bit box lies as
  // [8-token groups][2 d-halves][8 tokens][128 B]: the groups of a d-half are then
  // evenly spaced over the whole tile, as the MMA wants its rows.
  constexpr uint32_t kDepth = kFp8 ? R::kRawStages : R::kStages;
  uint32_t ring_i = 0;
  auto load_unit = [&](const Unit& u, auto between) {
    const int part = warp >> 1;                                      // warps 0, 2
    const int32_t n = max(u.n0, u.n1);
    const int32_t* table = prm.tables + static_cast<int64_t>(u.seq_row) * prm.mbps;
    const int32_t blocks = (u.kv_len + (16 << prm.bshift) - 1) >> (4 + prm.bshift);
    const int32_t per_log = 3 - prm.bshift, share = (1 << per_log) / kLoaders;   // blocks a tile, and of this warp
    const int32_t bytes = (kFp8 ? 2048 : 4096) << prm.bshift;                    // of a block
    int32_t id = 0, id_base = -64;                                   // cache rows of blocks id_base + lane
    auto copy = [&](int32_t i, bool is_v) {
      const int32_t b0 = (u.tile0 + i) << per_log, nb = max(0, min(share, blocks - b0 - part * share));
      if (!is_v) {  // the tile's cache rows, kept for its V copy
        if (b0 >= id_base + 32 || id_base < 0) {
          id_base = b0;
          const int32_t b = b0 + lane;
          int32_t v = b < blocks && b < prm.mbps ? table[b] : 0;
          if (static_cast<uint32_t>(v) >= static_cast<uint32_t>(prm.num_blocks)) {
            atomicOr(prm.err, kErrBadBlock);
            v = 0;
          }
          id = ((prm.layer * prm.num_blocks + v) * prm.H + u.h) << (4 + prm.bshift);
        }
        const int32_t row = __shfl_sync(0xffffffffu, id, (b0 - id_base + part * share + lane) & 31);
        if (lane < share) mt.rows[part][i & 7][lane] = row;
        __syncwarp();
      }
      const uint32_t st = ring_i % kDepth, par = ((ring_i / kDepth) & 1) ^ 1;
      if (!wait(kFp8 ? mt.raw_empty[st] : mt.kv_empty[st], par)) return false;
      const uint32_t full = bar(kFp8 ? mt.raw_full[st] : mt.kv_full[st]);
      if (lane == 0) dev::mbar_arrive_expect_tx(full, nb * bytes);
      __syncwarp();  // the bytes are expected before any copy is issued
      if (lane < nb) {
        const int32_t row = mt.rows[part][i & 7][lane];
        const uint32_t dst = base + (kFp8 ? R::kOffRaw + st * kRaw : R::kOffKv + st * kOperand) + (part * share + lane) * bytes;
        if (kFp8)
          dev::tma_load_2d(dst, is_v ? &tmv : &tmk, 0, row, full);
        else
          dev::tma_load_4d(dst, is_v ? &tmv : &tmk, 0, 0, 0, row >> 3, full);
      }
      ++ring_i;
      return true;
    };
    for (int32_t i = 0; i < min(kLead, n); ++i)
      if (!copy(i, false)) return false;
    if (!between()) return false;
    for (int32_t i = 0; i < n; ++i) {
      if (!copy(i, true)) return false;
      if (i + kLead < n && !copy(i + kLead, false)) return false;
    }
    return true;
  };
  // copies already issued land before the CTA can exit
  auto load_drain = [&]() {
    for (uint32_t k = ring_i > kDepth ? ring_i - kDepth : 0; k < ring_i; ++k)
      dev::mbar_wait_bounded(bar(kFp8 ? mt.raw_full[k % kDepth] : mt.kv_full[k % kDepth]), (k / kDepth) & 1, kWaitLimit);
  };

  if (warp < 4) {
  regs_less<R::kRegsControl>();
  if (warp == 2) {
    dev::grid_dep_wait();
    Unit u;
    while (next_unit(u) && load_unit(u, [] { return true; })) {
    }
    load_drain();
  } else if (warp == 0) {
    // ===================================== schedule, queries, and a loader
    uint32_t sched_i = 0, q_i[2] = {0, 0};
    int32_t w = blockIdx.x, w_next = 0;
    bool ok = true;
    const int32_t total = prm.units;
    const int32_t tq = kTile >> prm.gshift;       // tokens of a query tile
    for (bool begun = false;; begun = true) {
      Unit u;
      u.seq_row = -1;
      if (w < total) {
        const int32_t wi = w / prm.H;
        u.h = w - wi * prm.H;
        int lo = 0, hi = prm.n - 1;
        while (lo < hi) {
          const int mid = (lo + hi + 1) >> 1;
          if (prm.pre[mid] <= wi) lo = mid; else hi = mid - 1;
        }
        u.seq_row = prm.row[lo];
        u.m = prm.m[lo];
        u.kv_len = prm.kv_len[lo];
        u.past = u.kv_len - u.m;
        const int32_t ut = tq * R::kQ;                               // tokens of a unit
        const int32_t qt = (u.m + ut - 1) / ut;
        const int32_t r = wi - prm.pre[lo], ch = (prm.pre[lo + 1] - prm.pre[lo]) / qt;
        const int32_t c = r % ch;
        u.t0 = (qt - 1 - r / ch) * ut;                               // the longest first
        u.tok0 = prm.row0 + prm.q0[lo] + u.t0;
        u.tile0 = c * prm.chunk;
        u.part = w;
        u.direct = 1;
        int32_t nx[2] = {0, 0}, end[2] = {0, 0};
#pragma unroll
        for (int x = 0; x < R::kQ; ++x) {
          if (u.t0 + x * tq >= u.m) break;
          const int32_t last = prm.mask ? u.kv_len - 1 : u.past + min(u.t0 + (x + 1) * tq, u.m) - 1;
          const int32_t nt = last / kTile + 1;
          nx[x] = max(0, min(nt - u.tile0, prm.chunk));
          end[x] = min(8, (last >> 4) + 1 - (u.tile0 + nx[x] - 1) * 8);
          if (nt > prm.chunk) u.direct = 0;
        }
        u.n0 = nx[0];
        u.n1 = nx[1];
        u.end0 = end[0];
        u.end1 = end[1];
      }
      if (!begun) dev::grid_dep_wait();
      // the next claim is on its way while this unit is copied
      if (lane == 0 && w < total) {
        const int32_t v = atomicAdd(prm.counter, 1);
        if (v == total - 1) *prm.counter = 0;     // the last claim of all: `units` claims in total
        w_next = static_cast<int32_t>(gridDim.x) + v;
      }
      const int32_t n = u.seq_row < 0 ? 0 : max(u.n0, u.n1);
      if (u.seq_row < 0 || n > 0) {                                  // an empty chunk is skipped
        if (!(ok = wait(mt.sched_empty[sched_i & 1], ((sched_i >> 1) & 1) ^ 1))) break;
        if (lane == 0) {
          mt.unit[sched_i & 1] = u;
          arrive(bar(mt.sched_full[sched_i & 1]));
        }
        ++sched_i;
      }
      if (u.seq_row < 0) break;
      if (n > 0) {
        // query tiles, [2 d-halves][128 rows][128 B], row = token * G + head: after the
        // first K tiles, which need not wait for the tiles of the unit before
        auto load_q = [&]() {
#pragma unroll
          for (int x = 0; x < R::kQ; ++x) {
            if ((x == 0 ? u.n0 : u.n1) == 0) continue;
            if (!wait(mt.q_empty[x], (q_i[x] & 1) ^ 1)) return false;
            if (lane == 0) {
              const uint32_t dst = base + x * kOperand, b = bar(mt.q_full[x]);
              dev::mbar_arrive_expect_tx(b, kOperand);
              dev::tma_load_3d(dst, &tmq, 0, u.h << prm.gshift, u.tok0 + x * tq, b);
              dev::tma_load_3d(dst + kHalf, &tmq, 64, u.h << prm.gshift, u.tok0 + x * tq, b);
            }
            ++q_i[x];
          }
          return true;
        };
        if (!(ok = load_unit(u, load_q))) break;
      }
      w = __shfl_sync(0xffffffffu, w_next, 0);
    }
    dev::grid_dep_launch();
    load_drain();
    for (int x = 0; x < R::kQ; ++x)
      if (q_i[x]) dev::mbar_wait_bounded(bar(mt.q_full[x]), (q_i[x] - 1) & 1, kWaitLimit);
  } else if (warp == 1) {
    // ===================================================================== MMA
    // One thread runs the whole role: what it does between two MMAs is time the
    // tensor core may stand still.
    if (dev::elect_one()) {
      constexpr bool kBf = MMA == kBF16;
      constexpr uint32_t kIdO = instr_desc(kBf, true, 128);
      // (under a negative scale S is made of -Q, and scaled by its magnitude)
      const uint32_t id_s = instr_desc(kBf, false, 0) | (prm.sl2 < 0.f ? kNegateA : 0u);
      const uint64_t q_desc = smem_desc(base, 16, 1024), k_desc = smem_desc(base + R::kOffKv, 16, 2 * kGroup),
                     v_desc = smem_desc(base + R::kOffKv, kGroup, 2 * kGroup);
      uint32_t st = 0, ph = 0;                          // ring stage of the next tile, and its phase
      uint32_t q_i[2] = {0, 0}, p_i[2] = {0, 0}, o_i[2] = {0, 0}, clean_i = 0;
      bool ok = true;
      dev::grid_dep_wait();
      auto wait1 = [&](uint64_t& b, uint32_t parity) {
        const uint32_t a = bar(b);
        for (uint32_t i = 0; i < kWaitLimit; ++i) {
          if (dev::mbar_try_wait(a, parity)) return true;
          if (*abort) break;
        }
        if (*abort == 0) {
          *abort = 1;
          atomicOr(prm.err, kErrTimeout);
        }
        return ok = false;
      };
      auto advance = [&]() {                            // to the next tile of the ring, which has landed
        const uint32_t s = st;
        if (++st == R::kStages) {
          st = 0;
          ph ^= 1;
        }
        return s;
      };
      // steps: 16-position steps that any row attends; what lies behind them is not computed
      auto issue_s = [&](int x, uint32_t s, int32_t steps) {
        fence_after();
        const uint32_t id = id_s + (static_cast<uint32_t>(steps * 2) << 17);   // N = 16 steps
        const uint64_t qd = q_desc + (PAIR ? x : 0) * (kOperand >> 4), kd = k_desc + s * (kOperand >> 4);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {
          mma_ss(tmem + x * 128, qd + (((kk >> 2) * kHalf + (kk & 3) * 32) >> 4),
                 kd + (((kk >> 2) * kGroup + (kk & 3) * 32) >> 4), id, kk > 0);
        }
        commit(bar(mt.s_full[x]));
      };
      auto issue_pv = [&](int x, uint32_t s, int32_t steps, bool acc) {
        fence_after();
        const uint64_t vd = v_desc + s * (kOperand >> 4);
        if (steps >= 8) {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            mma_ts(tmem + 256 + x * 128, tmem + x * 128 + j * 8, vd + j * (4096 >> 4), kIdO, acc || j > 0);
        } else {
          for (int j = 0; j < steps; ++j)
            mma_ts(tmem + 256 + x * 128, tmem + x * 128 + j * 8, vd + j * (4096 >> 4), kIdO, acc || j > 0);
        }
      };
      for (;;) {
        if (!wait1(mt.sched_full[unit_i & 1], (unit_i >> 1) & 1)) break;
        const Unit& un = mt.unit[unit_i & 1];
        const int32_t seq_row = un.seq_row, n0 = un.n0, n1 = un.n1, n = max(n0, n1);
        const int32_t end0 = un.end0, end1 = un.end1;
        const bool clean = needs_clean(un, n);
        arrive(bar(mt.sched_empty[unit_i & 1]));
        ++unit_i;
        if (seq_row < 0) break;
        // V of tile i: landed, and its rows past the length zeroed
        auto take_v = [&](int32_t i) {
          if (!wait1(mt.kv_full[st], ph)) return st;
          if (clean && i == n - 1) {
            arrive(bar(mt.clean_go));
            wait1(mt.clean_done, clean_i & 1);
            ++clean_i;
          }
          return advance();
        };
        auto take_k = [&]() { return wait1(mt.kv_full[st], ph) ? advance() : st; };
        if constexpr (PAIR) {
          const int32_t nx[2] = {n0, n1}, end[2] = {end0, end1};
          const uint32_t k0 = take_k();
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            if (!ok || nx[x] == 0 || !wait1(kScaleQ ? mt.q_ready[x] : mt.q_full[x], q_i[x] & 1)) continue;
            ++q_i[x];
            issue_s(x, k0, nx[x] == 1 ? end[x] : 8);
            if (nx[x] == 1) commit(bar(mt.q_empty[x]));
          }
          if (!ok) break;
          commit(bar(mt.kv_empty[k0]));
          for (int32_t j = 0; ok && j < n; ++j) {
            const uint32_t v = take_v(j), k = j + 1 < n ? take_k() : 0;
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              if (!ok || j >= nx[x]) continue;
              if (j == 0 && !wait1(mt.o_free[x], (o_i[x]++ & 1) ^ 1)) continue;
              if (!wait1(mt.p_full[x], p_i[x] & 1)) continue;
              ++p_i[x];
              issue_pv(x, v, j == nx[x] - 1 ? end[x] : 8, j > 0);
              if (x == 1 || j >= nx[1]) commit(bar(mt.kv_empty[v]));
              if (j == nx[x] - 1) commit(bar(mt.o_full[x]));
              if (j + 1 < nx[x]) {
                issue_s(x, k, j + 1 == nx[x] - 1 ? end[x] : 8);
                if (j + 1 == nx[x] - 1) commit(bar(mt.q_empty[x]));
              }
              if (j + 1 < n && (x == 1 || j >= nx[1])) commit(bar(mt.kv_empty[k]));
            }
          }
        } else {
          if (!wait1(kScaleQ ? mt.q_ready[0] : mt.q_full[0], q_i[0] & 1)) break;
          ++q_i[0];
          for (int32_t i = 0; ok && i < min(2, n); ++i) {
            const uint32_t k = take_k();
            if (!ok) break;
            issue_s(i, k, i == n - 1 ? end0 : 8);
            commit(bar(mt.kv_empty[k]));
            if (i == n - 1) commit(bar(mt.q_empty[0]));
          }
          if (!ok || !wait1(mt.o_free[0], (o_i[0]++ & 1) ^ 1)) break;
          for (int32_t i = 0; i < n; ++i) {
            const int x = i & 1;
            const uint32_t v = take_v(i);
            if (!ok || !wait1(mt.p_full[x], p_i[x]++ & 1)) break;
            issue_pv(x, v, i == n - 1 ? end0 : 8, i > 1);
            commit(bar(mt.kv_empty[v]));
            if (i >= n - 2) commit(bar(mt.o_full[x]));
            if (i + 2 < n) {
              const uint32_t k = take_k();
              if (!ok) break;
              issue_s(x, k, i + 2 == n - 1 ? end0 : 8);
              commit(bar(mt.kv_empty[k]));
              if (i + 2 == n - 1) commit(bar(mt.q_empty[0]));
            }
          }
        }
        if (!ok) break;
      }
      // every MMA issued has finished before the tensor memory is released
      commit(bar(mt.done));
      dev::mbar_wait_bounded(bar(mt.done), 0, kWaitLimit);
    }
    __syncwarp();
  } else if (!kFp8) {
    // ============================================== V rows past the length
    // Their weights are 0, and 0 x NaN is NaN: zeroed where a block is partly filled.
    uint32_t kv_i = 0, clean_i = 0;
    dev::grid_dep_wait();
    Unit u;
    while (next_unit(u)) {
      const int32_t n = max(u.n0, u.n1);
      kv_i += 2 * n;                                    // the last V is the unit's last tile in the ring
      if (!needs_clean(u, n)) continue;
      if (!wait(mt.clean_go, clean_i & 1)) break;
      ++clean_i;
      const int32_t valid = u.kv_len - (u.tile0 + n - 1) * kTile;
      uint8_t* v = sm + R::kOffKv + ((kv_i - 1) % R::kStages) * kOperand;
      for (int c = lane; c < (16 - (valid & 15)) * 16; c += 32) {
        const int t = valid + (c >> 4);
        *reinterpret_cast<uint4*>(v + (t >> 3) * 2 * kGroup + (c & 1) * kGroup + (t & 7) * 128 + ((c >> 1) & 7) * 16) =
            make_uint4(0, 0, 0, 0);
      }
      dev::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) arrive(bar(mt.clean_done));
    }
  }
  } else if (warp < 12) {
    regs_more<R::kRegsSoftmax>();
    // ======================================================= softmax, epilogue
    const int x = (warp >> 2) - 1;                     // stream
    const int r = (warp & 3) * 32 + lane;              // row, and TMEM lane
    const uint32_t tl = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const uint32_t ts = tl + x * 128, to = tl + 256 + x * 128;
    const int32_t tq = kTile >> prm.gshift, G = 1 << prm.gshift;
    uint32_t s_i = 0, o_i[2] = {0, 0}, ml_i = 0, q_i = 0;
    dev::grid_dep_wait();
    Unit u;
    while (next_unit(u)) {
      const int32_t n = PAIR ? (x == 0 ? u.n0 : u.n1) : u.n0;   // this stream's last step + 1
      if (PAIR && n == 0) continue;
      const int32_t t = u.t0 + (PAIR ? x : 0) * tq + (r >> prm.gshift), g = r & (G - 1);
      const bool row_ok = t < u.m;
      const bool warp_ok = u.t0 + (PAIR ? x : 0) * tq + (((warp & 3) * 32) >> prm.gshift) < u.m;
      const int32_t tc = min(t, u.m - 1);               // rows behind the last token read its limits
      const int32_t tok = u.tok0 + (t - u.t0);
      uint64_t bits = 0;
      int32_t lim;        // causal: positions allowed; tree: prefix positions, all allowed
      if (prm.mask) {
        lim = u.past;
        bits = prm.mask[u.tok0 + (tc - u.t0)];
        if (u.m < 64) bits &= (uint64_t{1} << u.m) - 1;
      } else {
        lim = u.past + tc + 1;
      }
      const int32_t lim_min = __reduce_min_sync(0xffffffffu, lim);
      float sl2 = fabsf(prm.sl2), vs = 1.f;
      if constexpr (kFp8) {
        sl2 *= prm.k_scale[prm.layer * prm.H + u.h];
        vs = prm.v_scale[prm.layer * prm.H + u.h];
      }
      const bool neg = kFp8 && sl2 < 0.f;               // (a negative K scale)
      if constexpr (!kScaleQ)
        if (sl2 == 0.f) sl2 = 1e-30f;                   // equal weights; a masked -inf x sl2 stays -inf
      float mref = -INFINITY, l = 0.f;
      bool ok = true, far = false;
      int32_t i = PAIR ? 0 : x;
      auto next_scores = [&]() {
        if (!(ok = wait(mt.s_full[x], s_i & 1))) return false;
        ++s_i;
        fence_after();
        if constexpr (kScaleQ) {
          if (i < (PAIR ? 1 : 2)) {                     // S is made from the converted queries
            sl2 = ldexpf(sl2, mt.q_exp[q_i & 3][PAIR ? x : 0][r]);
            if (sl2 == 0.f) sl2 = 1e-30f;               // (a row of zeros)
          }
        }
        return true;
      };
      for (; !neg && i < n; i += PAIR ? 1 : 2) {
        if (!next_scores()) break;
        if (warp_ok) {
          const int32_t p0 = (u.tile0 + i) * kTile;
          const bool masked = p0 + kTile > lim_min;
          // the whole row of S in registers; P overlays it as it is made
          float y[4][32];
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_ld32(ts + c * 32, y[c]);
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_wait(y[c]);
          if (masked) {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const int32_t k0 = lim - (p0 + c * 32);   // columns from the chunk's first to the limit
              uint32_t a = low_bits(k0);
              if (prm.mask && k0 < 32)
                a |= k0 >= 0 ? static_cast<uint32_t>(bits << k0) : (k0 > -64 ? static_cast<uint32_t>(bits >> -k0) : 0u);
#pragma unroll
              for (int k = 0; k < 32; ++k) y[c][k] = a >> k & 1 ? y[c][k] : -INFINITY;
            }
          }
          // Weights of the row against the reference, their sum, and (MAX) the row's
          // maximum on the way: it runs beside the exponentials, which the
          // special-function unit bounds.
          const uint64_t sl2x2 = pack_f32x2(sl2, sl2);
          float top;                             // of the scaled scores; -inf where nothing is allowed
          auto weights = [&](auto with_max) {
            constexpr bool MAX = decltype(with_max)::value;
            const float mr = mref == -INFINITY ? 0.f : kBias<MMA> - mref;
            const uint64_t mrx2 = pack_f32x2(mr, mr);
            uint64_t ls[2] = {0, 0};
            float mc[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              uint32_t pk[16];
#pragma unroll
              for (int k = 0; k < 32; k += 2) {
                float e0, e1;
                unpack_f32x2(fma_f32x2(pack_f32x2(y[c][k], y[c][k + 1]), sl2x2, mrx2), e0, e1);
                e0 = dev::exp2_approx(e0);
                e1 = dev::exp2_approx(e1);
                if (MAX) {
                  float& m = mc[(k >> 1) & 3];
                  m = fmaxf(m, fmaxf(y[c][k], y[c][k + 1]));
                }
                ls[(k >> 1) & 1] = add_f32x2(ls[(k >> 1) & 1], pack_f32x2(e0, e1));
                pk[k >> 1] = pack2<MMA>(e0, e1);
              }
              tmem_st16(ts + c * 16, pk);        // over columns of S chunk c / 2, which is in registers
            }
            if (MAX) top = sl2 * fmaxf(fmaxf(mc[0], mc[1]), fmaxf(mc[2], mc[3]));
            float l0, l1;
            unpack_f32x2(add_f32x2(ls[0], ls[1]), l0, l1);
            return l0 + l1;
          };
          // A tile whose maximum does not pass the reference by kLazy, as nearly all
          // after a row's first do, is done with the weights it was given at once.
          const bool known = kSpec && __all_sync(0xffffffffu, !row_ok || mref > -INFINITY);
          bool done = false;
          if (known) {
            if constexpr (kSpec) {
              const float sum = weights(std::true_type{});
              done = !__any_sync(0xffffffffu, row_ok && top > mref + kLazy<MMA>);
              if (done) l += sum;
            }
          } else {
            float mc[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) mc[k] = -INFINITY;
#pragma unroll
            for (int k = 0; k < 128; k += 2) mc[(k >> 1) & 7] = fmaxf(mc[(k >> 1) & 7], fmaxf(y[k >> 5][k & 31], y[k >> 5][(k & 31) + 1]));
#pragma unroll
            for (int k = 1; k < 8; ++k) mc[0] = fmaxf(mc[0], mc[k]);
            top = sl2 * mc[0];
          }
          if (!done) {
            // stores to tensor memory are asynchronous, and not ordered among
            // themselves: weights stored above are over before they are stored again
            if constexpr (kSpec) tmem_wait_st();
            // the reference moves, and O is scaled to the new one, after the P V of the
            // step before (complete: S came after it)
            const bool move = top > mref + kLazy<MMA> || (mref == -INFINITY && top > -INFINITY);
            float corr = 1.f;
            if (move) {
              corr = mref == -INFINITY ? 0.f : dev::exp2_approx(mref - top);
              mref = top;
              l *= corr;
            }
            if (__any_sync(0xffffffffu, move)) {
              if (i >= (PAIR ? 1 : 2)) {
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                  float o[16];
                  tmem_ld16(to + c * 16, o);
#pragma unroll
                  for (int k = 0; k < 16; ++k) o[k] *= corr;
                  tmem_st16(to + c * 16, reinterpret_cast<const uint32_t(&)[16]>(o));
                }
              }
              if (__any_sync(0xffffffffu, row_ok && fabsf(mref) >= kFar && mref > -INFINITY)) {
                if constexpr (kSpec) {                  // scores that weights lie over
#pragma unroll
                  for (int c = 0; c < 4; ++c)
                    tmem_st16(ts + c * 16, reinterpret_cast<const uint32_t(&)[16]>(y[c >> 1][(c & 1) * 16]));
                }
                tmem_wait_st();
                far = true;
                break;
              }
            }
            l += weights(std::false_type{});
          }
          tmem_wait_st();
        }
        fence_before();
        __syncwarp();
        if (lane == 0) arrive(bar(mt.p_full[x]));
      }
      // This tile and the unit's others where a reference is far: scores are scaled and
      // rounded before they are taken from it, which is exact, so the largest weighs 1; no
      // lag, 16 columns at a time from tensor memory.  (A small loop of its own: code in
      // the one above costs prompts percents even where it does not run.)
      for (bool here = far; (far || neg) && i < n; i += PAIR ? 1 : 2, here = false) {
        if (!here && !next_scores()) break;
        const int32_t p0 = (u.tile0 + i) * kTile;
        auto scores = [&](int c, float (&z)[16]) {
          tmem_ld16(ts + c * 16, z);
          const int32_t k0 = lim - (p0 + c * 16);
          uint32_t a = low_bits(k0);
          if (prm.mask && k0 < 32)
            a |= k0 >= 0 ? static_cast<uint32_t>(bits << k0) : (k0 > -64 ? static_cast<uint32_t>(bits >> -k0) : 0u);
#pragma unroll
          for (int k = 0; k < 16; ++k) z[k] = a >> k & 1 ? __fmul_rn(z[k], sl2) : -INFINITY;
        };
        float top = -INFINITY;
#pragma unroll 1
        for (int c = 0; c < 8; ++c) {
          float z[16];
          scores(c, z);
#pragma unroll
          for (int k = 0; k < 16; ++k) top = fmaxf(top, z[k]);
        }
        const bool move = top > mref;
        float corr = 1.f;
        if (move) {
          corr = mref == -INFINITY ? 0.f : dev::exp2_approx(mref - top);
          mref = top;
          l *= corr;
        }
        if (i >= (PAIR ? 1 : 2) && __any_sync(0xffffffffu, move)) {
#pragma unroll 1
          for (int c = 0; c < 8; ++c) {
            float o[16];
            tmem_ld16(to + c * 16, o);
#pragma unroll
            for (int k = 0; k < 16; ++k) o[k] *= corr;
            tmem_st16(to + c * 16, reinterpret_cast<const uint32_t(&)[16]>(o));
          }
        }
        const float ref = mref == -INFINITY ? 0.f : mref;
#pragma unroll 1
        for (int c = 0; c < 8; ++c) {                   // P over columns that have been read
          float z[16];
          uint32_t pk[8];
          scores(c, z);
#pragma unroll
          for (int k = 0; k < 16; k += 2) {
            const float e0 = dev::exp2_approx(__fsub_rn(z[k], ref) + kBias<MMA>);
            const float e1 = dev::exp2_approx(__fsub_rn(z[k + 1], ref) + kBias<MMA>);
            l += e0 + e1;
            pk[k >> 1] = pack2<MMA>(e0, e1);
          }
          tmem_st8(ts + c * 8, pk);
        }
        tmem_wait_st();
        fence_before();
        __syncwarp();
        if (lane == 0) arrive(bar(mt.p_full[x]));
      }
      if (!ok) break;
      ++q_i;
      // ---- epilogue
      uint16_t* out = reinterpret_cast<uint16_t*>(prm.out) +
                      ((static_cast<int64_t>(tok) * prm.H + u.h) * G + g) * kHeadDim;
      // partial: [130][part_rows], so that a warp's rows lie side by side
      const int64_t pr = prm.part_rows;
      float* part = prm.partials + u.part * pr * kPartFloats + r;
      const bool direct = PAIR || u.direct;   // (pairs are taken where no positions are split)
      const bool wide = (reinterpret_cast<uintptr_t>(prm.out) & 31) == 0;  // `out` itself may be 16-byte aligned
      auto put = [&](int c, const float (&o)[32]) {  // columns 32c.. of this row
        if (!row_ok) return;
        if (direct) {
#pragma unroll
          for (int k = 0; k < 32; k += 16) {        // whole 32-byte sectors: a row is a line of its own
            uint32_t v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = pack2<ACT>(o[k + 2 * e], o[k + 2 * e + 1]);
            if (wide) {
              dev::st_global_v8(out + c * 32 + k, v);
            } else {
              *reinterpret_cast<uint4*>(out + c * 32 + k) = make_uint4(v[0], v[1], v[2], v[3]);
              *reinterpret_cast<uint4*>(out + c * 32 + k + 8) = make_uint4(v[4], v[5], v[6], v[7]);
            }
          }
        } else {
#pragma unroll
          for (int k = 0; k < 32; ++k) part[(c * 32 + k) * pr] = o[k];
        }
      };
      if constexpr (PAIR) {
        if (!wait(mt.o_full[x], o_i[x] & 1)) break;
        ++o_i[x];
        fence_after();
        const float f = l != 0.f ? vs / l : 0.f;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          float o[32];
          tmem_ld32(to + c * 32, o);
          tmem_wait(o);
#pragma unroll
          for (int k = 0; k < 32; ++k) o[k] = l != 0.f ? o[k] * f : 0.f;   // (a NaN row stays one)
          put(c, o);
        }
        fence_before();
        __syncwarp();
        if (lane == 0) arrive(bar(mt.o_free[x]));
      } else {
        // join the two streams; stream x writes d-half x
        bool all = true;
#pragma unroll
        for (int y = 0; y < 2; ++y)
          if (all && y < n) {
            all = wait(mt.o_full[y], o_i[y] & 1);
            ++o_i[y];
          }
        if (!all) break;
        fence_after();
        float(&mlv)[2][2][kTile] = mt.mlv[ml_i & 1];
        mlv[x][0][r] = mref;
        mlv[x][1][r] = l;
        __syncwarp();
        if (lane == 0) arrive(bar(mt.ml[x]));
        if (!wait(mt.ml[x ^ 1], ml_i & 1)) break;
        ++ml_i;
        const float m2 = mlv[x ^ 1][0][r], l2 = mlv[x ^ 1][1][r];
        const float mm = fmaxf(mref, m2);
        float w0 = stream_weight(mref, l, mm), w1 = stream_weight(m2, l2, mm);
        const float lsum = l * w0 + l2 * w1;
        const float f = vs * (direct && lsum != 0.f ? 1.f / lsum : 1.f);
        w0 *= f;
        w1 *= f;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float a[32], b[32];
          tmem_ld32(to + x * 64 + c * 32, a);
          tmem_ld32(tl + 256 + (x ^ 1) * 128 + x * 64 + c * 32, b);
          tmem_wait(a);
          tmem_wait(b);
#pragma unroll
          for (int k = 0; k < 32; ++k) a[k] = (w0 != 0.f ? a[k] * w0 : 0.f) + (w1 != 0.f ? b[k] * w1 : 0.f);
          put(x * 2 + c, a);
        }
        fence_before();
        __syncwarp();
        if (lane == 0) arrive(bar(mt.o_free[0]));
        if (!direct && row_ok && x == 0) {
          part[kHeadDim * pr] = mm;
          part[(kHeadDim + 1) * pr] = lsum;
        }
      }
    }
  } else if constexpr (kFp8) {
    regs_less<R::kRegsConvert>();
    // ==================================================== FP8 codes to fp16 tiles
    uint32_t raw_i = 0, q_i[2] = {0, 0};
    const int tid = threadIdx.x - 384;
    dev::grid_dep_wait();
    Unit u;
    bool ok = true;
    while (ok && next_unit(u)) {
      const int32_t n = max(u.n0, u.n1);
      auto convert = [&](int32_t i, bool is_v) {
        const uint32_t rs = raw_i % (kFp8 ? R::kRawStages : 1), ks = raw_i % R::kStages;
        if (!wait(mt.raw_full[rs], (raw_i / (kFp8 ? R::kRawStages : 1)) & 1)) return false;
        if (!wait(mt.kv_empty[ks], ((raw_i / R::kStages) & 1) ^ 1)) return false;
        const int32_t valid = min(kTile, u.kv_len - (u.tile0 + i) * kTile);
        // 16 codes, 16c .., of tokens t, t + 16, ...: every address is one of three
        // bases plus a constant, and all loads are out before the first store.  Eight
        // lanes hold eight tokens, which the swizzle spreads over the banks.  All four
        // warps share a tile: what counts is how soon one is ready.
        const int t = (tid & 7) + (tid >> 6) * 8, c = (tid >> 3) & 7, f = c >> 2;
        const uint8_t* src = sm + R::kOffRaw + rs * kRaw + t * 128 + ((c ^ (t & 7)) << 4);
        uint4 raw[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) raw[k] = *reinterpret_cast<const uint4*>(src + k * 2048);
        if (is_v && valid < kTile) {
#pragma unroll
          for (int k = 0; k < 8; ++k)
            if (k * 16 + t >= valid) raw[k] = make_uint4(0, 0, 0, 0);
        }
        uint8_t* row = sm + R::kOffKv + ks * kOperand + (t >> 3) * 2 * kGroup + f * kGroup + (t & 7) * 128;
        uint8_t* d0 = row + (((2 * (c & 3)) ^ (t & 7)) << 4);
        uint8_t* d1 = row + (((2 * (c & 3) + 1) ^ (t & 7)) << 4);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const uint32_t w[4] = {raw[k].x, raw[k].y, raw[k].z, raw[k].w};
          uint32_t o[8];
#pragma unroll
          for (int q = 0; q < 8; ++q) o[q] = dev::e4m3x2_to_f16x2(static_cast<uint16_t>(w[q >> 1] >> ((q & 1) * 16)));
          *reinterpret_cast<uint4*>(d0 + k * 4 * kGroup) = make_uint4(o[0], o[1], o[2], o[3]);
          *reinterpret_cast<uint4*>(d1 + k * 4 * kGroup) = make_uint4(o[4], o[5], o[6], o[7]);
        }
        dev::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          arrive(bar(mt.kv_full[ks]));
          arrive(bar(mt.raw_empty[rs]));
        }
        ++raw_i;
        return true;
      };
      if constexpr (kScaleQ) {
        // bf16 queries as fp16 times a power of two a row: the row's largest value
        // goes to [2^14, 2^15), so all that is lost is under 2^-38 of it
#pragma unroll
        for (int x = 0; x < R::kQ; ++x) {
          if (!ok || (x == 0 ? u.n0 : u.n1) == 0 || !(ok = wait(mt.q_full[x], q_i[x] & 1))) continue;
          uint8_t* q = sm + x * kOperand + tid * 128;
          uint32_t top = 0;                        // of |q|: bf16 magnitudes compare as integers
#pragma unroll 4
          for (int c = 0; c < 16; ++c) {
            const uint4 v = *reinterpret_cast<const uint4*>(q + (c >> 3) * kHalf + (((c & 7) ^ (tid & 7)) << 4));
            top = __vmaxu2(top, __vmaxu2(__vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu),
                                         __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu)));
          }
          top = max(top & 0xffffu, top >> 16) >> 7;                       // biased exponent
          const int e = max(static_cast<int>(top) - 127 - 14, -126);
          const float f = __int_as_float((127 - e) << 23);                // 2^-e
          mt.q_exp[q_i[x] & 3][x][tid] = static_cast<int8_t>(e);
#pragma unroll 4
          for (int c = 0; c < 16; ++c) {
            uint4* at = reinterpret_cast<uint4*>(q + (c >> 3) * kHalf + (((c & 7) ^ (tid & 7)) << 4));
            const uint4 v = *at;
            auto half2 = [&](uint32_t w) { return dev::pack_f16(dev::bf16lo_to_f32(w) * f, dev::bf16hi_to_f32(w) * f); };
            *at = make_uint4(half2(v.x), half2(v.y), half2(v.z), half2(v.w));
          }
          ++q_i[x];
          dev::fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) arrive(bar(mt.q_ready[x]));
        }
      }
      for (int32_t i = 0; ok && i < min(kLead, n); ++i) ok = convert(i, false);
      for (int32_t i = 0; ok && i < n; ++i) {
        ok = convert(i, true);
        if (ok && i + kLead < n) ok = convert(i + kLead, false);
      }
    }
  }
  fence_before();
  __syncthreads();
  fence_after();
  if (warp == 1)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(512) : "memory");
}

// ------------------------------------------------------------- joining chunks
// A thread takes one row and D d of one query tile, a warp 32 rows side by side,
// and the loads of several chunks are under way together: they are all this kernel
// waits for.  The chunks' O are weighted by 2^(their maximum - the row's) and
// divided by the sum.  Tiles that had one chunk are done already.
template <int ACT, int D, int CAP>
__global__ void __launch_bounds__(256) attend_merge_kernel(const __grid_constant__ Params<CAP> prm) {
  constexpr int kCtas = 64 / D, kBatch = 32 / D;  // CTAs of a query tile; chunks whose loads are under way together
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, G = 1 << prm.gshift;
  const int32_t b = blockIdx.x, dq = b % kCtas, v = b / kCtas;
  const int32_t h = v % prm.H, tq = kTile >> prm.gshift;
  int32_t tile = v / prm.H, it = 0, qt = 0;       // the tile's sequence, and its place there (few sequences are split)
  for (; it < prm.n; ++it) {
    qt = (prm.m[it] + tq - 1) / tq;
    if (tile < qt) break;
    tile -= qt;
  }
  if (it == prm.n) return;
  const int32_t m = prm.m[it], past = prm.kv_len[it] - m, t0 = tile * tq;
  const int32_t last = prm.mask ? prm.kv_len[it] - 1 : past + min(t0 + tq, m) - 1;
  const int32_t nt = last / kTile + 1;
  if (nt <= prm.chunk) return;
  const int32_t chunks = (nt + prm.chunk - 1) / prm.chunk, ch = (prm.pre[it + 1] - prm.pre[it]) / qt;
  const int64_t w = static_cast<int64_t>(prm.pre[it] + (qt - 1 - tile) * ch) * prm.H + h;
  const int32_t r = (warp & 3) * 32 + lane, t = t0 + (r >> prm.gshift);
  dev::grid_dep_wait();
  dev::grid_dep_launch();
  if (t >= m) return;
  const int64_t pr = prm.part_rows, step = prm.H * pr * kPartFloats;   // to the next chunk
  const float* part = prm.partials + w * pr * kPartFloats + r;
  const int d0 = dq * 2 * D + (warp >> 2) * D;
  float mx = -INFINITY, o[D], l = 0.f;            // the sum so far, against the running maximum
#pragma unroll
  for (int k = 0; k < D; ++k) o[k] = 0.f;
  for (int c0 = 0; c0 < chunks; c0 += kBatch) {
    float mc[kBatch], lc[kBatch], vc[kBatch][D];
#pragma unroll
    for (int c = 0; c < kBatch; ++c) {
      const bool in = c0 + c < chunks;
      const float* p = part + (c0 + c) * step;
      mc[c] = in ? __ldcg(p + kHeadDim * pr) : -INFINITY;
      lc[c] = in ? __ldcg(p + (kHeadDim + 1) * pr) : 0.f;
#pragma unroll
      for (int k = 0; k < D; ++k) vc[c][k] = in ? __ldcg(p + (d0 + k) * pr) : 0.f;
    }
    float top = mx;
#pragma unroll
    for (int c = 0; c < kBatch; ++c) top = fmaxf(top, mc[c]);
    const float corr = mx == -INFINITY ? 0.f : dev::exp2_approx(mx - top);
    mx = top;
    l *= corr;
#pragma unroll
    for (int k = 0; k < D; ++k) o[k] *= corr;
#pragma unroll
    for (int c = 0; c < kBatch; ++c) {
      const float wc = stream_weight(mc[c], lc[c], mx);
      l += wc * lc[c];
#pragma unroll
      for (int k = 0; k < D; ++k) o[k] += wc * vc[c][k];
    }
  }
  const float inv = l != 0.f ? 1.f / l : 0.f;
  uint32_t* out = reinterpret_cast<uint32_t*>(
      prm.out + 2 * (((static_cast<int64_t>(prm.row0 + prm.q0[it] + t) * prm.H + h) * G + (r & (G - 1))) * kHeadDim + d0));
  uint32_t res[D / 2];
#pragma unroll
  for (int k = 0; k < D / 2; ++k) res[k] = pack2<ACT>(o[2 * k] * inv, o[2 * k + 1] * inv);
#pragma unroll
  for (int k = 0; k < D / 2; k += 4)
    *reinterpret_cast<uint4*>(out + k) = make_uint4(res[k], res[k + 1], res[k + 2], res[k + 3]);
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encoder() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(p);
  });
  return fn;
}

template <int KV, int ACT, bool PAIR, int CAP>
cudaError_t run(const Params<CAP>& prm, const AttendMaps& maps, const CUtensorMap& tmq, int num_sms, cudaStream_t stream) {
  using R = Ring<PAIR, KV == kFP8>;
  constexpr size_t smem = smem_bytes<PAIR, KV == kFP8>();
  static_assert(smem <= 227 * 1024, "attention exceeds the shared memory of an SM");
  static uint64_t configured = 0;  // bit per device: dynamic shared memory attribute set
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !(configured >> dev & 1u)) {
    e = cudaFuncSetAttribute(attend_kernel<KV, ACT, PAIR, CAP>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    // the warpgroups' register shares come out of what the launch holds
    cudaFuncAttributes attr;
    e = cudaFuncGetAttributes(&attr, attend_kernel<KV, ACT, PAIR, CAP>);
    if (e != cudaSuccess) return e;
    if (attr.numRegs < R::kRegsLaunch) return cudaErrorInvalidConfiguration;
    if (dev < 64) configured |= uint64_t{1} << dev;
  }
  return launch_overlapped(attend_kernel<KV, ACT, PAIR, CAP>, dim3(std::min(num_sms, prm.units)), dim3(R::kThreads), smem, stream,
                    prm, maps.k, maps.v, tmq);
}

template <bool PAIR, int CAP>
cudaError_t dispatch(const PoolView& pool, const Params<CAP>& prm, const AttendMaps& maps, const CUtensorMap& tmq,
                     int num_sms, cudaStream_t stream) {
  const bool bf = pool.act_dtype == kBF16;
  if (pool.kv_dtype == kFP8)
    return bf ? run<kFP8, kBF16, PAIR, CAP>(prm, maps, tmq, num_sms, stream)
              : run<kFP8, kFP16, PAIR, CAP>(prm, maps, tmq, num_sms, stream);
  return bf ? run<kBF16, kBF16, PAIR, CAP>(prm, maps, tmq, num_sms, stream)
            : run<kFP16, kFP16, PAIR, CAP>(prm, maps, tmq, num_sms, stream);
}

int ceil_div(int64_t a, int64_t b) { return static_cast<int>((a + b - 1) / b); }

template <int CAP>
cudaError_t launch(const PoolView& pool, const AttendMaps& maps, const AttendArgs& a, const AttendItems& items,
                   int num_sms, cudaStream_t stream, int* launches) {
  EncodeTiledFn encode = encoder();
  if (!encode) return cudaErrorNotSupported;
  static thread_local Params<CAP> prm;
  static thread_local int order[CAP];
  const int H = pool.num_kv_heads, G = a.num_q_heads / H;
  const int tq = kTile / G;
  const int n = items.n;
  // Pairs of query tiles read (and convert) each KV tile once for 256 rows: taken where
  // few of them stay half empty and there is one for each SM.  As pairs and as single
  // tiles, us: ragged prompts of 32 heads 911 and 1,066, long ones 2,020 and 2,272, FP8
  // chunks 960 and 1,000; 47 trees of 64 drafts 116 and 135, of 5 to 16 drafts 46 and 43;
  // eight FP8 trees of 20 to 33 drafts, 80 pairs, 543 and 350: one tile's two streams,
  // with the positions split, keep more SMs busy.  The border is not exact: 128 pairs of
  // 33 drafts are 534 and 614, 160 pairs of FP8 chunks 311 and 254 (two rounds of pairs).
  int64_t singles = 0, pairs = 0;
  int max_rows = 0;
  for (int i = 0; i < n; ++i) {
    const int m = items.q0[i + 1] - items.q0[i];
    singles += ceil_div(m, tq);
    pairs += ceil_div(m, 2 * tq);
    max_rows = std::max(max_rows, m * G);
  }
  const bool pair = 16 * pairs <= 9 * singles && pairs * H >= num_sms;
  const int ut = pair ? 2 * tq : tq;

  prm.out = static_cast<uint8_t*>(a.out);
  prm.tables = a.tables;
  prm.mask = a.mask;
  prm.k_scale = pool.k_scale;
  prm.v_scale = pool.v_scale;
  prm.partials = pool.partials;
  prm.counter = pool.counters;
  prm.err = pool.err;
  prm.sl2 = a.scale * kLog2e;
  prm.layer = a.layer;
  prm.H = H;
  prm.gshift = G == 8 ? 3 : G == 4 ? 2 : G == 2 ? 1 : 0;
  prm.num_blocks = pool.num_blocks;
  prm.mbps = pool.mbps;
  prm.bshift = pool.block_size == 32 ? 1 : 0;
  prm.n = n;
  prm.row0 = items.row0;
  prm.part_rows = std::min(kTile, (max_rows + 7) / 8 * 8);

  // KV tiles of a chunk: all of a sequence's, unless the units are too few for
  // the SMs; then the smallest chunk that gives each SM one, if that saves more
  // tiles than joining the chunks costs (a second kernel).  Two units of one tree, a tile
  // 1.0 us (FP8 1.25): 7 tiles 13.8 us whole and 10.9 split (16.7 and 12.4), 40 tiles
  // 46 and 13.8 (58 and 15.6), 4 tiles 10.8 whole.
  auto count = [&](int chunk) {
    int64_t u = 0;
    for (int i = 0; i < n; ++i)
      u += static_cast<int64_t>(ceil_div(items.q0[i + 1] - items.q0[i], ut)) *
           ceil_div(ceil_div(items.kv_len[i], kTile), chunk);
    return u * H;
  };
  int most = 1;
  for (int i = 0; i < n; ++i) most = std::max(most, ceil_div(items.kv_len[i], kTile));
  int chunk = most;
  constexpr int kMinChunk = 2, kJoin = 5;
  const int64_t room = pool.partial_slots * kPartialSlotFloats / (static_cast<int64_t>(prm.part_rows) * kPartFloats);
  const int64_t want = std::min<int64_t>(num_sms, room);
  if (!pair && count(most) < want && most >= kMinChunk + kJoin) {
    int lo = kMinChunk, hi = most;                // the smallest chunk with count <= want
    while (lo < hi) {
      const int mid = (lo + hi) / 2;
      if (count(mid) <= want) hi = mid; else lo = mid + 1;
    }
    if (lo + kJoin <= most) chunk = lo;
  }
  prm.chunk = chunk;
  const int64_t units = count(chunk);
  if (units >= INT32_MAX / 4) return cudaErrorInvalidValue;
  prm.units = static_cast<int32_t>(units);

  // the longest sequences first
  for (int i = 0; i < n; ++i) order[i] = i;
  std::stable_sort(order, order + n, [&](int x, int y) { return items.kv_len[x] > items.kv_len[y]; });
  prm.pre[0] = 0;
  for (int k = 0; k < n; ++k) {
    const int i = order[k];
    prm.row[k] = items.row[i];
    prm.kv_len[k] = items.kv_len[i];
    prm.q0[k] = items.q0[i];
    prm.m[k] = items.q0[i + 1] - items.q0[i];
    prm.pre[k + 1] = prm.pre[k] + ceil_div(prm.m[k], ut) * ceil_div(ceil_div(prm.kv_len[k], kTile), chunk);
  }

  // q as [tokens][H_q][128], boxes of 128 / G tokens x G heads x 64
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(kHeadDim), static_cast<cuuint64_t>(a.num_q_heads),
                              static_cast<cuuint64_t>(a.total_tokens)};
  const cuuint64_t strides[2] = {kHeadDim * 2, static_cast<cuuint64_t>(a.num_q_heads) * kHeadDim * 2};
  const cuuint32_t box[3] = {64u, static_cast<cuuint32_t>(G), static_cast<cuuint32_t>(tq)};
  const cuuint32_t estr[3] = {1, 1, 1};
  CUtensorMap tmq;
  if (encode(&tmq, CU_TENSOR_MAP_DATA_TYPE_UINT16, 3, const_cast<void*>(a.q), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return cudaErrorInvalidValue;
  cudaError_t e = pair ? dispatch<true, CAP>(pool, prm, maps, tmq, num_sms, stream)
                       : dispatch<false, CAP>(pool, prm, maps, tmq, num_sms, stream);
  if (e != cudaSuccess) return e;
  ++*launches;
  if (chunk < most) {
    // Few tiles: more CTAs a tile (one of 32K tokens, 8 heads: 34 us in all with 8 d
    // a thread, 37 with 16; 32 to 64 tiles of 4K to 8K: 23 and 69 us with 8, 22 and
    // 66 with 16).
    int64_t tiles = 0;
    for (int i = 0; i < n; ++i) tiles += ceil_div(items.q0[i + 1] - items.q0[i], ut);
    tiles *= H;
    const bool bf = pool.act_dtype == kBF16;
    auto join = [&](auto d) {
      constexpr int D = decltype(d)::value;
      const dim3 grid(static_cast<unsigned>(tiles * (64 / D)));
      return bf ? launch_overlapped(attend_merge_kernel<kBF16, D, CAP>, grid, dim3(256), 0, stream, prm)
                : launch_overlapped(attend_merge_kernel<kFP16, D, CAP>, grid, dim3(256), 0, stream, prm);
    };
    if constexpr (CAP == kSmallCap)   // (more sequences are more tiles than that)
      e = tiles < 32 ? join(std::integral_constant<int, 8>{}) : join(std::integral_constant<int, 16>{});
    else
      e = join(std::integral_constant<int, 16>{});
    if (e != cudaSuccess) return e;
    ++*launches;
  }
  return cudaSuccess;
}

}  // namespace

cudaError_t launch_attend(const PoolView& pool, const AttendMaps& maps, const AttendArgs& args,
                          const AttendItems& items, int num_sms, cudaStream_t stream, int* launches) {
  return items.n <= kSmallCap ? launch<kSmallCap>(pool, maps, args, items, num_sms, stream, launches)
                              : launch<kAttendItemsCap>(pool, maps, args, items, num_sms, stream, launches);
}

}  // namespace pa
