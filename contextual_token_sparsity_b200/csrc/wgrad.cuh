// wgrad.cuh - weight gradient of a linear layer whose input is held in an
// 8-bit checkpoint: dW[n, c] += sum_r dy[r, n] xhat[r, c] over the kept rows.
//
// A tensor-core GEMM with M = n, N = d, K = kept rows, both operands MN-major.
// The checkpoint's codes are turned into bf16 operand tiles inside the kernel:
// code x 2^k is exact in bf16, so the products are those of the restored rows
// without a bf16 copy of them in memory (3 bytes per value less traffic and
// K d x 2 bytes less memory than restoring first).
//
// Persistent clusters of two CTAs take 256 x 256 output tiles with 2-SM
// instructions (tcgen05.mma.cta_group::2, M = N = 256, K = 16).  CTA r of a
// pair holds columns [128 r, +128) of the tile's dy and of its codes.  Per stage
// of 64 kept rows:
//   warp 0      TMA: a 64 x 128 tile of dy (two 128-byte-swizzled boxes, 16 KB);
//   12 warps    three teams of four warps, each team every third stage: codes
//               (loaded to registers a turn ahead) -> bf16 B tile (64 rows of
//               128 columns, the MN-major swizzled image), rows past the kept
//               ones zero;
//   warp 2      passes a landed dy tile on to the leader, after clearing the rows
//               past the kept ones in the last stage (they may hold anything);
//   warp 1      (leader) MMA issue into one of two 256-column accumulators;
//   warps 20-23 read-out of a finished accumulator, one TMEM lane quadrant each.
// A conversion is five instructions per two values (no table, no fp32 detour).
// The converting warps sit on three of the SM's four schedulers (warp % 4 != 1):
// sharing the issuer's scheduler stretched its few instructions between two MMAs
// and with them every stage, 765 cycles against 613 without conversions.
//
// The tensor core's fp32 accumulation truncates: measured against fp64, sums
// over K rows are off by 1.0e-6 (random signs) and 2.2e-6 (one sign) at K = 1024,
// 2.1e-6 and 5.6e-6 at K = 2048, 9.1e-6 and 3.5e-5 at K = 8192.  So an accumulator
// takes at most 2048 rows and is then added into dW with TMA reduce-adds (fp32,
// round to nearest, done at L2), while the MMAs fill the other one.  The adds of
// one tile are issued by one CTA pair, each accumulator's after those of the one
// before have completed, so their order and the result are fixed.
//
// Few tiles leave most SMs idle while every pair walks over all rows.  Then the
// rows of one item are split over the `splits` (2 or 4) pairs of a larger cluster,
// accumulator by accumulator; the pairs add theirs into dW in turn, each after the
// one before it has completed (a barrier in the next pair's CTA), so the order of
// the adds stays fixed.  512 x 512 over 8192 rows: 25 us so, 50 without.
//
// Measured: 8192 rows, 4096 x 11008, e4m3: 591 us in a single launch under the profiler
// (1.25 PFLOP/s, tensor pipe 71 % busy), 664 to 683 us in long loops, where the power
// limit lowers the clock; 4928 rows, 4096 x 4096, int8: 145 and 155 to 169 us.  Restoring
// the rows to memory first and a library product take 579 us in loops of the first: what
// this kernel saves is the copy, not time.
//
// Every wait is bounded in time; a wait that runs out records LEMO_ERR_TIMEOUT
// and makes both CTAs of the pair drain what they issued, free their tensor
// memory and return.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>

#include <type_traits>

#include "ckpt.cuh"
#include "common.cuh"
#include "gemm.cuh"

namespace lemo {
namespace wgrad {

using gemm::bulk_commit;
using gemm::bulk_wait_all;
using gemm::bulk_wait_read1;
using gemm::sdesc;
using gemm::stage_row;
using gemm::tma_reduce_add_2d;
using gemm::umma_pair;
using score::cluster_sync;
using score::cta_rank;
using score::map_to_rank;
using score::mbar_arrive;
using score::mbar_arrive_cluster;
using score::mbar_arrive_expect_tx;
using score::mbar_init;
using score::mbar_try_wait;
using score::smem_u32;
using score::tc_fence_after;
using score::tc_fence_before;
using score::tmem_ld16;
using score::tmem_wait_ld;

constexpr int TM = 256, TN = 256;   // output tile of a pair
constexpr int HALF = 128;           // columns of each operand held by one CTA
constexpr int KB = 64;              // kept rows per stage
constexpr int CHUNK = 32;           // stages per accumulator: 2048 rows
constexpr int STAGES = 6;           // dy tiles and bf16 tiles in flight
constexpr int A_BYTES = KB * HALF * 2;
constexpr int B_BYTES = KB * HALF * 2;
constexpr int TEAMS = 3;            // teams of workers that take alternate stages
constexpr int TEAM = 4;             // warps per team
constexpr int WORKERS = TEAMS * TEAM;
constexpr int FIRST_WORKER = 4;     // warps 4 .. 19 but those of scheduler 1
constexpr int FIRST_READER = FIRST_WORKER + WORKERS / 3 * 4;
constexpr int READERS = 4;          // warps that read accumulators: one per lane quadrant
constexpr int THREADS = 32 * (FIRST_READER + READERS);
constexpr int ROWS_PER_WORKER = KB / TEAM;
constexpr int STEPS = ROWS_PER_WORKER / 4;  // a warp takes 4 rows at a time
constexpr int BOX = 32;             // columns of an output box (32 rows, 128 bytes each)
constexpr int STG_BYTES = 32 * BOX * 4;
constexpr int TMEM_COLS = 512;
constexpr uint64_t kDrainNs = 2000000000ull;  // bound of the waits for copies and MMAs in flight, at the end

struct Smem {
    uint64_t a_full[STAGES];     // each CTA: its dy tile landed
    uint64_t ready[STAGES];      // leader: both CTAs' dy and bf16 tiles are in place
    uint64_t used[STAGES];       // each CTA: the pair's MMAs of a stage completed
    uint64_t acc_full[2];        // each CTA: accumulator holds a finished chunk
    uint64_t acc_empty[2];       // leader: both CTAs' readers read an accumulator
    uint64_t done;               // each CTA: every MMA of the leader completed
    uint64_t turn;               // each CTA: the adds before this CTA's next ones completed
    uint32_t tmem_base;
    int abort_flag;
};
constexpr int OFF_B = STAGES * A_BYTES;
constexpr int OFF_STG = OFF_B + STAGES * B_BYTES;
constexpr int OFF_BAR = OFF_STG + READERS * 2 * STG_BYTES;
constexpr int SMEM_BYTES = OFF_BAR + (int)sizeof(Smem) + 1024 /*align slack*/;
static_assert(SMEM_BYTES <= 232448, "exceeds the 227 KB of shared memory per CTA");
static_assert(A_BYTES % 1024 == 0 && B_BYTES % 1024 == 0 && STG_BYTES % 1024 == 0,
              "swizzled tiles are 1024-byte aligned");

struct Args {
    ckpt::View c;
    int n, d;
    int tiles_m, tiles_n;
    int whole, items;            // items below `whole` are 256 x 256 tiles, the others 256 x 128 halves
    int splits;                  // pairs of a cluster; above 1 a cluster takes one item
    const int32_t* kept_total;
    int64_t rows;
    uint64_t spin_limit_ns;
    int withhold;                // test hook: the first cluster's first stage never becomes ready
};

__device__ __forceinline__ void abort_pair(Smem* sm) {
    *reinterpret_cast<volatile int*>(&sm->abort_flag) = 1;
    const uint32_t peer = map_to_rank(smem_u32(&sm->abort_flag), cta_rank() ^ 1u);
    asm volatile("st.relaxed.cluster.shared::cluster.u32 [%0], %1;" ::"r"(peer), "r"(1) : "memory");
}

__device__ __noinline__ bool wait_slow(uint64_t* bar, uint32_t parity, Smem* sm, uint64_t limit_ns) {
    const uint64_t t0 = globaltimer_ns();
    for (uint32_t n = 1;; ++n) {
        if (mbar_try_wait(bar, parity)) return true;
        if ((n & 63) == 0) {
            if (*reinterpret_cast<volatile int*>(&sm->abort_flag)) return false;
            if (globaltimer_ns() - t0 > limit_ns) {
                raise_error(LEMO_ERR_TIMEOUT);
                abort_pair(sm);
                return false;
            }
        }
    }
}

__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, Smem* sm, uint64_t limit_ns) {
    if (mbar_try_wait(bar, parity)) return true;
    return wait_slow(bar, parity, sm, limit_ns);
}

// warp-uniform result
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, Smem* sm,
                                          uint64_t limit_ns) {
    const bool ok = wait(bar, parity, sm, limit_ns);
    return __all_sync(0xffffffffu, ok);
}

__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap* tm, int x, int y,
                                         uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(tm)), "r"(x), "r"(y), "r"(smem_u32(bar))
        : "memory");
}

// Whether the phase of the given parity has completed, without waiting.
__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}\n"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}

__device__ __forceinline__ void st_shared(uint32_t addr, uint4 v) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z),
                 "r"(v.w)
                 : "memory");
}

// Arrive once on this barrier in both CTAs of the pair when every MMA issued so
// far by this thread has completed.
__device__ __forceinline__ void umma_commit_pair(uint64_t* bar, uint16_t pair_mask) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
        " [%0], %1;" ::"r"(smem_u32(bar)),
        "h"(pair_mask)
        : "memory");
}

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
// (a & b) | c in one instruction
__device__ __forceinline__ uint32_t and_or(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t d;
    asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}

// a + b as a x 1 + b (one instruction of the FMA pipe)
__device__ __forceinline__ uint32_t add_bf16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(0x3f803f80u), "r"(b));
    return d;
}

// Four codes to four bf16 values (two words), exactly, with the group's scale
// 2^k as a pair of equal bf16 factors.  The even codes make one word and the odd
// codes the other, which needs no byte permutation: columns 1 and 2 of every four
// change places in the B tile, and the readers put them back.
// e4m3: the code's exponent and mantissa bits moved to bits 4..10 of a bf16 read
//   as value x 2^-120 (subnormal codes as subnormal bf16), so the factor is
//   2^(k + 120).  Left shifts are written as products: they then run on the FMA
//   pipe, the integer pipe being the busiest.
// int8: with the code's low 7 bits l and sign bit s, (128 + l) - (128 + 128 s) is
//   the value; both terms are a bf16 +-128 with bits of the code or'ed in, and the
//   sum is exact.

// bf16 +-128 twice, kept in registers: (x & constant) | constant is one
// instruction only if one of the two constants is.
struct Consts {
    uint32_t plus, minus;
    __device__ __forceinline__ Consts() {
        asm volatile("mov.b32 %0, 0x43004300;" : "=r"(plus));
        asm volatile("mov.b32 %0, 0xc300c300;" : "=r"(minus));
    }
};

template <int FORMAT>
__device__ __forceinline__ void to_bf16x4(uint32_t q, uint32_t f, const Consts& c, uint32_t& even,
                                          uint32_t& odd) {
    if constexpr (FORMAT == ckpt::kE4M3) {
        even = mul_bf16x2(((q * 16u) & 0x07f007f0u) | ((q * 256u) & 0x80008000u), f);
        odd = mul_bf16x2(((q >> 4) & 0x07f007f0u) | (q & 0x80008000u), f);
    } else {
        const uint32_t o = q >> 8;
        even = mul_bf16x2(add_bf16x2(and_or(q, 0x007f007fu, c.plus), and_or(q, 0x00800080u, c.minus)), f);
        odd = mul_bf16x2(add_bf16x2(and_or(o, 0x007f007fu, c.plus), and_or(o, 0x00800080u, c.minus)), f);
    }
}

// Scale bytes up to this one have a bf16 factor in both formats (2^(134 - 7) is
// bf16's largest power of two); larger ones, and the NaN marker, take two factors.
constexpr uint32_t kOneFactor = 134;

template <int FORMAT>
__device__ __forceinline__ uint32_t factor(uint32_t code) {
    // exponent fields code + 120 (e4m3) or code (int8) in both halves
    return code * 0x00800080u + (FORMAT == ckpt::kE4M3 ? 0x3c003c00u : 0u);
}

template <int FORMAT>
__device__ __forceinline__ uint32_t second_factor(uint32_t code, uint32_t& f) {
    const uint32_t e = FORMAT == ckpt::kE4M3 ? code + 120u : code;
    const uint32_t e1 = e < 254u ? e : 254u;
    f = e1 * 0x00800080u;
    return code == 255u ? 0x7fff7fffu : (127u + e - e1) * 0x00800080u;
}

// Instruction descriptor: D fp32, A and B bf16, both MN-major, M = 256, N = n.
__device__ __forceinline__ constexpr uint32_t idesc(int n) {
    return (1u << 4) | (1u << 7) | (1u << 10) | (1u << 15) | (1u << 16) | ((uint32_t)(n >> 3) << 17) |
           ((uint32_t)(TM >> 4) << 24);
}

// One item of a pair: rows [n0, +256), columns [c0, +width) of dW, each CTA
// converting width / 2 of the columns.  When the last round of tiles would
// leave at least half of the pairs idle the host cuts its tiles in two
// (4928 x 4096 x 4096 has 256 tiles for 74 pairs: 3.5 rounds instead of 4), and
// a tile whose columns end within its first half is one anyway.
struct Item {
    int n0, c0, width;  // width 0: nothing there
};

// Tiles go in groups of GROUP row tiles, column by column: the group's dy stays in
// L2 while the codes stream past it (8192 x 4096 x 11008: 654 MB read from DRAM,
// 948 MB with all 16 row tiles in one group; 671 against 689 us).
constexpr int GROUP = 8;

__device__ __forceinline__ Item item_of(const Args& a, int i) {
    Item r;
    int t = i, half = 0;
    r.width = TN;
    if (i >= a.whole) {
        t = a.whole + ((i - a.whole) >> 1);
        half = (i - a.whole) & 1;
        r.width = HALF;
    }
    const int group = t / (GROUP * a.tiles_n), first = group * GROUP;
    const int rows = min(GROUP, a.tiles_m - first), in = t - first * a.tiles_n;
    r.n0 = (first + in % rows) * TM;
    r.c0 = (in / rows) * TN + half * HALF;
    if (a.d - r.c0 <= HALF) r.width = HALF;
    if (r.c0 >= a.d) r.width = 0;
    return r;
}

template <int FORMAT>
__global__ void __launch_bounds__(THREADS, 1)
    wgrad_kernel(const __grid_constant__ CUtensorMap tm_dy, const __grid_constant__ CUtensorMap tm_dw,
                 const Args a) {
    pdl_entry();
    const int64_t K = ckpt::clamp_rows(a.kept_total, a.rows);
    const int kblocks = (int)((K + KB - 1) / KB);
    const int splits = a.splits, split = (blockIdx.x >> 1) % splits;
    const int cluster = blockIdx.x / (2 * splits), nclusters = gridDim.x / (2 * splits);
    if (kblocks == 0 || cluster >= a.items) return;  // the whole cluster leaves together
    // stages of one accumulator; split s takes accumulators s, s + splits, ...
    const int chunk_kb = splits == 1 ? CHUNK : max(1, min(CHUNK, (kblocks + splits - 1) / splits));
    const int next_kb = splits * chunk_kb;

    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* base = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    Smem* sm = reinterpret_cast<Smem*>(base + OFF_BAR);
    const uint32_t sbase = smem_u32(base);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t crank = cta_rank(), rank = crank & 1u, leader_rank = crank & ~1u;
    const uint16_t pair_mask = (uint16_t)(3u << leader_rank);
    const bool leader = rank == 0;
    const uint64_t lim = a.spin_limit_ns;

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&sm->a_full[s], 1);
            // (test hook: an arrival more than there will be)
            mbar_init(&sm->ready[s], 2 * (TEAM + 1) + (a.withhold && cluster == 0 && s == 0 ? 1 : 0));
            mbar_init(&sm->used[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&sm->acc_full[b], 1);
            mbar_init(&sm->acc_empty[b], 2 * READERS);
        }
        mbar_init(&sm->done, 1);
        mbar_init(&sm->turn, READERS);
        sm->abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_u32(&sm->tmem_base)),
                     "r"(TMEM_COLS));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
    }
    tc_fence_before();
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem_base = sm->tmem_base;

    // the stage behind kb among those of this split
    auto after = [&](int kb) { return (kb + 1) % chunk_kb ? kb + 1 : kb + 1 + next_kb - chunk_kb; };

    if (warp == 0) {
        // ------------------------------------------------------------ TMA producer
        if (lane == 0) {
            uint32_t it = 0, s = 0, ph = 0;  // stage, its slot and the slot's phase
            bool ok = true;
            for (int i = cluster; ok && i < a.items; i += nclusters) {
                const Item im = item_of(a, i);
                if (im.width == 0) continue;
                const int n0 = im.n0 + (int)rank * HALF;
                for (int kb = split * chunk_kb; kb < kblocks; kb = after(kb), ++it) {
                    if (!(ok = wait(&sm->used[s], ph ^ 1, sm, lim))) break;
                    const uint32_t sa = sbase + s * A_BYTES;
                    mbar_arrive_expect_tx(&sm->a_full[s], A_BYTES);
                    tma_load(sa, &tm_dy, n0, kb * KB, &sm->a_full[s]);
                    tma_load(sa + A_BYTES / 2, &tm_dy, n0 + 64, kb * KB, &sm->a_full[s]);
                    if (++s == STAGES) {
                        s = 0;
                        ph ^= 1;
                    }
                }
            }
            // every load in flight lands before the CTA leaves, also where another warp gave up
            for (uint32_t j = it > STAGES ? it - STAGES : 0; j < it; ++j) {
                const uint64_t t0 = globaltimer_ns();
                while (!mbar_try_wait(&sm->a_full[j % STAGES], (j / STAGES) & 1) &&
                       globaltimer_ns() - t0 < kDrainNs) {
                }
            }
        }
    } else if (warp == 2) {
        // ------------------------------------------------------------ dy tiles for the leader
        const uint32_t ready_c = map_to_rank(smem_u32(&sm->ready[0]), leader_rank);
        uint32_t s = 0, ph = 0;
        bool ok = true;
        for (int i = cluster; ok && i < a.items; i += nclusters) {
            if (item_of(a, i).width == 0) continue;
            for (int kb = split * chunk_kb; kb < kblocks; kb = after(kb)) {
                if (!(ok = wait_warp(&sm->a_full[s], ph, sm, lim))) break;
                const int valid = (int)min((int64_t)KB, K - (int64_t)kb * KB);
                if (valid < KB) {
                    // a row is 16 vectors: 8 in each 64-column half
                    for (int v = valid * 16 + lane; v < KB * 16; v += 32) {
                        const int row = v >> 4;
                        st_shared(sbase + s * A_BYTES + ((v >> 3) & 1) * (A_BYTES / 2) + row * 128 +
                                      (v & 7) * 16,
                                  make_uint4(0u, 0u, 0u, 0u));
                    }
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                }
                if (lane == 0) mbar_arrive_cluster(ready_c + s * 8);
                if (++s == STAGES) {
                    s = 0;
                    ph ^= 1;
                }
            }
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issuer
        if (lane == 0 && leader) {
            // descriptors of slot 0; a slot is A_BYTES (B_BYTES) further, a K step 2048 bytes
            const uint64_t da0 = sdesc(sbase, A_BYTES / 2), db0 = sdesc(sbase + OFF_B, B_BYTES / 2);
            // One MMA keeps the pipe busy for ~137 cycles and the pipe queues about two, so what
            // this thread does between two MMAs has to fit in ~270 cycles: the next stage is
            // tested for in the middle of this one's MMAs, and waited for only if that failed.
            uint32_t s = 0, ready_ph = 0, buf = 0, empty_ph = 1;
            bool ok = true, seen = false;  // seen: `ready` of the stage at hand was observed
            for (int i = cluster; ok && i < a.items; i += nclusters) {
                const Item im = item_of(a, i);
                if (im.width == 0) continue;
                const uint32_t id = im.width == TN ? idesc(TN) : idesc(HALF);
                for (int k0 = split * chunk_kb; ok && k0 < kblocks; k0 += next_kb) {
                    if (!(ok = wait(&sm->acc_empty[buf], empty_ph, sm, lim))) break;
                    const uint32_t d_tmem = tmem_base + buf * TN;
                    const int k1 = min(k0 + chunk_kb, kblocks);
                    for (int kb = k0; kb < k1; ++kb) {
                        const uint64_t da = da0 + s * (A_BYTES >> 4), db = db0 + s * (B_BYTES >> 4);
                        if (!seen && !(ok = wait(&sm->ready[s], ready_ph, sm, lim))) break;
                        tc_fence_after();
                        umma_pair(d_tmem, da, db, id, kb > k0 ? 1u : 0u);
                        umma_pair(d_tmem, da + (2048 >> 4), db + (2048 >> 4), id, 1u);
                        const uint32_t used_now = s;
                        s = s + 1 == STAGES ? 0u : s + 1;
                        ready_ph ^= s == 0 ? 1u : 0u;
                        seen = mbar_test(&sm->ready[s], ready_ph);
                        umma_pair(d_tmem, da + 2 * (2048 >> 4), db + 2 * (2048 >> 4), id, 1u);
                        umma_pair(d_tmem, da + 3 * (2048 >> 4), db + 3 * (2048 >> 4), id, 1u);
                        umma_commit_pair(&sm->used[used_now], pair_mask);
                    }
                    if (!ok) break;
                    umma_commit_pair(&sm->acc_full[buf], pair_mask);
                    buf ^= 1;
                    empty_ph ^= buf == 0 ? 1u : 0u;
                }
            }
            umma_commit_pair(&sm->done, pair_mask);
        }
        if (lane == 0) {
            // bounded: every MMA the leader issued completes before TMEM is freed
            const uint64_t t0 = globaltimer_ns();
            while (!mbar_try_wait(&sm->done, 0)) {
                if (globaltimer_ns() - t0 > kDrainNs) {
                    raise_error(LEMO_ERR_TIMEOUT);
                    break;
                }
            }
        }
    } else if (warp >= FIRST_WORKER && warp < FIRST_READER && warp % 4 != 1) {
        // ------------------------------------------------------------ workers
        const int w = (warp - FIRST_WORKER) / 4 * 3 + (warp % 4 ? warp % 4 - 1 : 0);  // 0 .. 11
        const int team = w / TEAM, q = w % TEAM;
        const uint32_t ready_c = map_to_rank(smem_u32(&sm->ready[0]), leader_rank);
        const int64_t turn_scales = (int64_t)TEAMS * KB * a.c.ld_scales;
        const int64_t turn_data = (int64_t)TEAMS * KB * a.c.ld;
        const int full_blocks = (int)(K / KB);
        const Consts consts;
        uint32_t turn = 0;        // stages this team has taken: stage = team + TEAMS turn
        uint32_t it = 0;          // stages before this item
        bool ok = true;
        for (int i = cluster; ok && i < a.items; i += nclusters) {
            const Item im = item_of(a, i);
            if (im.width == 0) continue;
            const bool wide = im.width == TN;
            // A lane turns 16 columns (chunk) of 4 rows, 4 apart (wide: 128 columns per CTA), or
            // of 2 rows, 8 apart (64 columns).  Wide, lanes of the two 64-column halves take
            // neighbouring rows: their swizzles differ in the lowest bit, so the 16-byte stores
            // of a quarter warp fall into 8 different bank groups.
            const int chunk = wide ? lane & 7 : lane & 3, h = chunk >> 2;
            const int row0 = q * ROWS_PER_WORKER + (wide ? (lane >> 3) ^ h : lane >> 2);
            const int gap = wide ? 4 : 8;
            uint32_t b_off[2][2];  // [step parity][vector] (64 columns: steps are 8 rows, one parity)
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    b_off[j][e] = h * (B_BYTES / 2) + (row0 + 4 * j) * 128 +
                                  (((2 * (chunk & 3) + e) ^ ((row0 + 4 * j) & 7)) << 4);
            // Converts this warp's rows of a stage.  `one`: one factor per scale is enough and
            // every row is kept; otherwise the lane's rows from `left` on are zero.
            auto convert = [&](auto wide_c, auto one, uint32_t bt, int left, const uint4* val,
                               const uint32_t* codes) {
                constexpr int N = wide_c.value ? STEPS : STEPS / 2, GAP = wide_c.value ? 4 : 8;
#pragma unroll
                for (int j = 0; j < N; ++j) {
                    const uint4 v = val[j];
                    uint32_t f = factor<FORMAT>(codes[j]), f2 = 0u;
                    if constexpr (!one.value) f2 = second_factor<FORMAT>(codes[j], f);
                    uint4 o0, o1;
                    to_bf16x4<FORMAT>(v.x, f, consts, o0.x, o0.y);
                    to_bf16x4<FORMAT>(v.y, f, consts, o0.z, o0.w);
                    to_bf16x4<FORMAT>(v.z, f, consts, o1.x, o1.y);
                    to_bf16x4<FORMAT>(v.w, f, consts, o1.z, o1.w);
                    if constexpr (!one.value) {
                        o0 = make_uint4(mul_bf16x2(o0.x, f2), mul_bf16x2(o0.y, f2),
                                        mul_bf16x2(o0.z, f2), mul_bf16x2(o0.w, f2));
                        o1 = make_uint4(mul_bf16x2(o1.x, f2), mul_bf16x2(o1.y, f2),
                                        mul_bf16x2(o1.z, f2), mul_bf16x2(o1.w, f2));
                        if (GAP * j >= left) o0 = o1 = make_uint4(0u, 0u, 0u, 0u);
                    }
                    const int par = wide_c.value ? j & 1 : 0, up = (wide_c.value ? j >> 1 : j) * 8 * 128;
                    st_shared(bt + b_off[par][0] + up, o0);
                    st_shared(bt + b_off[par][1] + up, o1);
                }
            };
            const int col = im.c0 + (int)rank * (im.width / 2) + 16 * chunk;
            const bool in = col < a.d;
            // a run of consecutive stages: all of them, or one accumulator's
            for (int run = split * chunk_kb; ok && run < kblocks; run += next_kb) {
                const int run_end = splits == 1 ? kblocks : min(run + chunk_kb, kblocks);
                int kb = run + (int)((team + TEAMS - it % TEAMS) % TEAMS);    // this team's next stage
                const int64_t first = (int64_t)kb * KB + row0;
                const uint8_t* sp = a.c.scales + (in ? col / ckpt::kGroup : 0) + first * a.c.ld_scales;
                const uint8_t* dp = a.c.data + (in ? col : 0) + first * a.c.ld;
                const int64_t step_scales = gap * a.c.ld_scales, step_data = gap * a.c.ld;
                int left = (int)K - kb * KB - row0;  // rows from this lane's first
                uint4 val[STEPS];       // codes and scale bytes of the team's next stage
                uint32_t codes[STEPS];
                // (columns past d are read from column 0: whatever they become is not stored)
                auto load = [&]() {
                    if (kb < full_blocks) {
#pragma unroll
                        for (int j = 0; j < STEPS; ++j) {
                            if (j >= STEPS / 2 && !wide) break;
                            val[j] = __ldg(reinterpret_cast<const uint4*>(dp + j * step_data));
                            codes[j] = __ldg(sp + j * step_scales);
                        }
                        return;
                    }
#pragma unroll
                    for (int j = 0; j < STEPS; ++j) {
                        const bool on = gap * j < left && (wide || j < STEPS / 2);
                        val[j] = on ? __ldg(reinterpret_cast<const uint4*>(dp + j * step_data)) : make_uint4(0u, 0u, 0u, 0u);
                        codes[j] = on ? __ldg(sp + j * step_scales) : 3u;
                    }
                };
                load();
                for (; kb < run_end; ++turn) {
                    // the MMAs of the stage STAGES before have read the slot
                    const uint32_t s = team + (turn & 1) * TEAMS;
                    if (!(ok = wait_warp(&sm->used[s], ((turn >> 1) & 1) ^ 1, sm, lim))) break;
                    const uint32_t bt = sbase + OFF_B + s * B_BYTES;
                    uint32_t most = 0;
#pragma unroll
                    for (int j = 0; j < STEPS; ++j)
                        if (wide || j < STEPS / 2) most = max(most, codes[j]);
                    const bool one = kb < full_blocks && !__any_sync(0xffffffffu, most > kOneFactor);
                    if (wide && one)
                        convert(std::true_type{}, std::true_type{}, bt, left, val, codes);
                    else if (wide)
                        convert(std::true_type{}, std::false_type{}, bt, left, val, codes);
                    else if (one)
                        convert(std::false_type{}, std::true_type{}, bt, left, val, codes);
                    else
                        convert(std::false_type{}, std::false_type{}, bt, left, val, codes);
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                    if (lane == 0) mbar_arrive_cluster(ready_c + s * 8);
                    sp += turn_scales;
                    dp += turn_data;
                    left -= TEAMS * KB;
                    kb += TEAMS;
                    load();
                }
                it += (uint32_t)(run_end - run);
                if (splits == 1) break;
            }
        }
    } else if (warp >= FIRST_READER) {
        // ------------------------------------------------------------ accumulator readers
        const int q = warp & 3;  // TMEM lane quadrant
        const uint32_t lane_addr = tmem_base + ((uint32_t)(q * 32) << 16);
        const uint32_t my_stg = sbase + OFF_STG + (warp - FIRST_READER) * 2 * STG_BYTES;
        const uint32_t empty_c = map_to_rank(smem_u32(&sm->acc_empty[0]), leader_rank);
        // the same CTA of the next pair: its adds come after these
        const uint32_t turn_c = map_to_rank(smem_u32(&sm->turn), (crank + 2) % (2 * splits));
        uint32_t buf = 0, full_ph = 0, turn_ph = 0;
        bool ok = true;
        for (int i = cluster; ok && i < a.items; i += nclusters) {
            const Item im = item_of(a, i);
            if (im.width == 0) continue;
            const int out_n = im.n0 + (int)rank * HALF + q * 32;
            for (int k0 = split * chunk_kb; k0 < kblocks; k0 += next_kb) {
                if (!(ok = wait_warp(&sm->acc_full[buf], full_ph, sm, lim))) break;
                tc_fence_after();
                // The adds of the accumulator before have completed (this warp's own, or those
                // of the pair before): one element's adds keep their order.
                if (lane == 0) bulk_wait_all();
                if (splits > 1 && k0 > 0) {
                    if (!(ok = wait_warp(&sm->turn, turn_ph, sm, lim))) break;
                    turn_ph ^= 1;
                }
#pragma unroll 1
                for (int ch = 0; ch < im.width; ch += BOX) {
                    uint32_t r[BOX];
                    tmem_ld16(lane_addr + buf * TN + ch, &r[0]);
                    tmem_ld16(lane_addr + buf * TN + ch + 16, &r[16]);
                    tmem_wait_ld();
                    if (ch + BOX == im.width) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive_cluster(empty_c + buf * 8);
                    }
                    const uint32_t box = my_stg + ((ch / BOX) & 1) * STG_BYTES;
                    if (lane == 0) bulk_wait_read1();  // the box before last has been read
                    __syncwarp();
#pragma unroll
                    for (int j = 1; j < BOX; j += 4) {  // columns 1 and 2 of every four
                        const uint32_t x = r[j];
                        r[j] = r[j + 1];
                        r[j + 1] = x;
                    }
                    stage_row(box, lane, r);
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                    if (lane == 0) {
                        if (im.c0 + ch < a.d && out_n < a.n)
                            tma_reduce_add_2d(&tm_dw, box, im.c0 + ch, out_n);
                        bulk_commit();
                    }
                }
                if (splits > 1 && k0 + chunk_kb < kblocks && lane == 0) {
                    bulk_wait_all();
                    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(turn_c)
                                 : "memory");
                }
                buf ^= 1;
                full_ph ^= buf == 0 ? 1u : 0u;
            }
        }
        if (lane == 0) bulk_wait_all();  // every reduce-add landed before the CTA exits
        __syncwarp();
    }

    // ---------------------------------------------------------------- teardown
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem_base),
                     "r"(TMEM_COLS));
    }
    cluster_sync();  // no CTA leaves while its peer may still signal its barriers
}

}  // namespace wgrad
}  // namespace lemo
