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
// pair holds columns [128 r, +128) of the tile's dy and of its codes.
//   warp 0     TMA: per 64 rows a 64 x 128 tile of dy (two 128-byte-swizzled
//              boxes, 16 KB) and the 64 x 128 codes (8 KB) into a ring;
//   warp 1     (leader) MMA issue into one of two 256-column accumulators;
//   warps 2-9  per 64 rows: codes -> bf16 B tile in its own ring (64 rows of
//              128 columns, the MN-major swizzled image), zeroing the rows past
//              the kept ones in both operands; and, per 1024 rows, read-out of
//              the finished accumulator.
// The tensor core's fp32 accumulation truncates: measured against fp64, a sum
// over K rows of one sign is off by 2.2e-6 at K = 1024 and 3.5e-5 at K = 8192.
// So an accumulator takes at most 1024 rows; its 128 x 128 values per warp pair are
// then added (round to nearest) to 128 fp32 registers per thread, while the MMAs
// fill the other accumulator.
//
// Every wait is bounded in time; a wait that runs out records LEMO_ERR_TIMEOUT
// and makes both CTAs of the pair drain what they issued, free their tensor
// memory and return.  One TMA reduce-add per output element and call, so the
// result does not depend on timing.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>

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
using score::add_f32x2;
using score::cluster_sync;
using score::cta_rank;
using score::map_to_rank;
using score::mbar_arrive_cluster;
using score::mbar_arrive_expect_tx;
using score::mbar_init;
using score::mbar_try_wait;
using score::smem_u32;
using score::tc_fence_after;
using score::tc_fence_before;
using score::tmem_ld16;
using score::tmem_wait_ld;
using score::umma_commit_pair;

constexpr int TM = 256, TN = 256;   // output tile of a pair
constexpr int HALF = 128;           // columns of each operand held by one CTA
constexpr int KB = 64;              // kept rows per stage
constexpr int CHUNK = 16;           // stages per accumulator: 1024 rows
constexpr int IN_STAGES = 4;        // dy tile + codes
constexpr int B_STAGES = 3;         // bf16 tiles made from codes
constexpr int A_BYTES = KB * HALF * 2;
constexpr int Q_BYTES = KB * HALF;
constexpr int IN_BYTES = A_BYTES + Q_BYTES;
constexpr int B_BYTES = KB * HALF * 2;
constexpr int WORKERS = 8;          // warps that make B tiles and read accumulators
constexpr int THREADS = 32 * (2 + WORKERS);
constexpr int ROWS_PER_WORKER = KB / WORKERS;
constexpr int STG_BYTES = 32 * 128;
constexpr int STG_PER_WARP = 2 * STG_BYTES;
constexpr int TMEM_COLS = 512;

struct Smem {
    uint64_t full[IN_STAGES];    // each CTA: its dy tile and codes of a stage landed
    uint64_t ready[B_STAGES];    // leader: both CTAs' workers finished a stage's operands
    uint64_t used[IN_STAGES];    // each CTA: the pair's MMAs of a stage completed
    uint64_t acc_full[2];        // each CTA: accumulator holds a finished chunk
    uint64_t acc_empty[2];       // leader: both CTAs' workers read an accumulator
    uint64_t done;               // each CTA: every MMA of the leader completed
    uint32_t tmem_base;
    int abort_flag;
};
constexpr int OFF_B = IN_STAGES * IN_BYTES;
constexpr int OFF_STG = OFF_B + B_STAGES * B_BYTES;
constexpr int OFF_BAR = OFF_STG + WORKERS * STG_PER_WARP;
constexpr int SMEM_BYTES = OFF_BAR + (int)sizeof(Smem) + 1024 /*align slack*/;
static_assert(SMEM_BYTES <= 232448, "exceeds the 227 KB of shared memory per CTA");
static_assert(IN_BYTES % 1024 == 0 && B_BYTES % 1024 == 0, "swizzled tiles are 1024-byte aligned");

struct Args {
    ckpt::View c;
    int n, d;
    int tiles_m, tiles_n;
    const int32_t* kept_total;
    int64_t rows;
    uint64_t spin_limit_ns;
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

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ uint32_t sub_bf16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// Four codes to four bf16 values (two words), exactly.
// e4m3: the code's exponent and mantissa bits moved to bits 4..10 of a bf16
//   read as value x 2^-120 (subnormal codes as subnormal bf16), so
//   x 2^120 x 2^(code - 127) follows, in two factors whose exponents fit.
// int8: magnitude m and sign s: (s 128 + s m) - s 128 is exact, then x 2^(code - 127).
struct Scale {
    uint32_t f1, f2;
};

__device__ __forceinline__ Scale make_scale(uint32_t code, int format) {
    Scale s;
    if (format == ckpt::kE4M3) {
        const uint32_t e = code + 120u;  // exponent field of 2^(code - 7)
        const uint32_t e1 = e < 254u ? e : 254u;
        s.f1 = e1 << 7;
        s.f2 = (127u + e - e1) << 7;
    } else {
        s.f1 = code << 7;
        s.f2 = 0u;
    }
    if (code == 255u) s.f1 = 0x7fffu;
    s.f1 |= s.f1 << 16;
    s.f2 |= s.f2 << 16;
    return s;
}

__device__ __forceinline__ void to_bf16x4(uint32_t q, Scale s, int format, uint32_t& lo,
                                          uint32_t& hi) {
    if (format == ckpt::kE4M3) {
        const uint32_t a = __byte_perm(q, 0u, 0x1404), b = __byte_perm(q, 0u, 0x3424);
        lo = (a & 0x80008000u) | ((a >> 4) & 0x07f007f0u);
        hi = (b & 0x80008000u) | ((b >> 4) & 0x07f007f0u);
        lo = mul_bf16x2(mul_bf16x2(lo, s.f1), s.f2);
        hi = mul_bf16x2(mul_bf16x2(hi, s.f1), s.f2);
    } else {
        const uint32_t neg = (q >> 7) & 0x01010101u;
        const uint32_t mag = (q ^ (neg * 255u)) + neg;  // bytes stay below 128: no carries
        const uint32_t sa = (__byte_perm(q, 0u, 0x1404) & 0x80008000u) | 0x43004300u;
        const uint32_t sb = (__byte_perm(q, 0u, 0x3424) & 0x80008000u) | 0x43004300u;
        lo = mul_bf16x2(sub_bf16x2(sa | __byte_perm(mag, 0u, 0x4140), sa), s.f1);
        hi = mul_bf16x2(sub_bf16x2(sb | __byte_perm(mag, 0u, 0x4342), sb), s.f1);
    }
}

// Instruction descriptor: D fp32, A and B bf16, both MN-major, M = 256, N = 256.
constexpr uint32_t kIdesc = (1u << 4) | (1u << 7) | (1u << 10) | (1u << 15) | (1u << 16) |
                            ((uint32_t)(TN >> 3) << 17) | ((uint32_t)(TM >> 4) << 24);

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(THREADS, 1)
    wgrad_kernel(const __grid_constant__ CUtensorMap tm_dy, const __grid_constant__ CUtensorMap tm_q,
                 const __grid_constant__ CUtensorMap tm_dw, const Args a) {
    pdl_entry();
    const int64_t K = ckpt::clamp_rows(a.kept_total, a.rows);
    const int kblocks = (int)((K + KB - 1) / KB);
    const int total = a.tiles_m * a.tiles_n;
    const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;
    if (kblocks == 0 || pair >= total) return;  // both CTAs of the pair leave together

    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* base = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    Smem* sm = reinterpret_cast<Smem*>(base + OFF_BAR);
    const uint32_t sbase = smem_u32(base);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cta_rank();
    const bool leader = rank == 0;
    const uint64_t lim = a.spin_limit_ns;

    if (threadIdx.x == 0) {
        for (int s = 0; s < IN_STAGES; ++s) {
            mbar_init(&sm->full[s], 1);
            mbar_init(&sm->used[s], 1);
        }
        for (int s = 0; s < B_STAGES; ++s) mbar_init(&sm->ready[s], 2 * WORKERS);
        for (int b = 0; b < 2; ++b) {
            mbar_init(&sm->acc_full[b], 1);
            mbar_init(&sm->acc_empty[b], 2 * WORKERS);
        }
        mbar_init(&sm->done, 1);
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

    if (warp == 0) {
        // ------------------------------------------------------------ TMA producer
        if (lane == 0) {
            uint32_t it = 0;
            bool ok = true;
            for (int t = pair; ok && t < total; t += npairs) {
                const int n0 = (t % a.tiles_m) * TM + (int)rank * HALF;
                const int c0 = (t / a.tiles_m) * TN + (int)rank * HALF;
                for (int kb = 0; kb < kblocks; ++kb, ++it) {
                    const uint32_t s = it % IN_STAGES, ph = (it / IN_STAGES) & 1;
                    if (!(ok = wait(&sm->used[s], ph ^ 1, sm, lim))) break;
                    mbar_arrive_expect_tx(&sm->full[s], IN_BYTES);
                    const uint32_t sa = sbase + s * IN_BYTES;
                    tma_load(sa, &tm_dy, n0, kb * KB, &sm->full[s]);
                    tma_load(sa + A_BYTES / 2, &tm_dy, n0 + 64, kb * KB, &sm->full[s]);
                    tma_load(sa + A_BYTES, &tm_q, c0, kb * KB, &sm->full[s]);
                }
            }
            if (!ok) {  // every load in flight lands before the CTA leaves
                const uint32_t first = it > IN_STAGES ? it - IN_STAGES : 0;
                for (uint32_t j = first; j < it; ++j) {
                    const uint64_t t0 = globaltimer_ns();
                    while (!mbar_try_wait(&sm->full[j % IN_STAGES], (j / IN_STAGES) & 1) &&
                           globaltimer_ns() - t0 < lim) {
                    }
                }
            }
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issuer
        if (lane == 0 && leader) {
            uint32_t it = 0, ci = 0;
            bool ok = true;
            for (int t = pair; ok && t < total; t += npairs) {
                for (int kb = 0; ok && kb < kblocks; ++kb, ++it) {
                    const int in_chunk = kb % CHUNK;
                    const uint32_t buf = ci & 1;
                    if (in_chunk == 0 &&
                        !(ok = wait(&sm->acc_empty[buf], ((ci >> 1) & 1) ^ 1, sm, lim)))
                        break;
                    if (!(ok = wait(&sm->ready[it % B_STAGES], (it / B_STAGES) & 1, sm, lim))) break;
                    tc_fence_after();
                    const uint32_t sa = sbase + (it % IN_STAGES) * IN_BYTES;
                    const uint32_t sb = sbase + OFF_B + (it % B_STAGES) * B_BYTES;
#pragma unroll
                    for (int k = 0; k < KB / 16; ++k)
                        umma_pair(tmem_base + buf * TN, sdesc(sa + k * 2048, A_BYTES / 2),
                                  sdesc(sb + k * 2048, B_BYTES / 2), kIdesc,
                                  (in_chunk > 0 || k > 0) ? 1u : 0u);
                    umma_commit_pair(&sm->used[it % IN_STAGES]);
                    if (in_chunk == CHUNK - 1 || kb == kblocks - 1) {
                        umma_commit_pair(&sm->acc_full[buf]);
                        ++ci;
                    }
                }
            }
            umma_commit_pair(&sm->done);
        }
        if (lane == 0) {
            // bounded: every MMA the leader issued completes before TMEM is freed
            const uint64_t t0 = globaltimer_ns();
            while (!mbar_try_wait(&sm->done, 0)) {
                if (globaltimer_ns() - t0 > lim) {
                    raise_error(LEMO_ERR_TIMEOUT);
                    break;
                }
            }
        }
    } else {
        // ------------------------------------------------------------ workers
        const int w = warp - 2;
        const int q = warp & 3, colhalf = w >> 2;  // TMEM lane quadrant, half of the columns
        const uint32_t lane_addr = tmem_base + ((uint32_t)(q * 32) << 16) + colhalf * HALF;
        const uint32_t my_stg = sbase + OFF_STG + w * STG_PER_WARP;
        const uint32_t ready_c = map_to_rank(smem_u32(&sm->ready[0]), 0);
        const uint32_t empty_c = map_to_rank(smem_u32(&sm->acc_empty[0]), 0);
        const int format = a.c.format;
        // a lane turns 16 columns (chunk) of rows row0 and row0 + 4 of every stage
        const int row0 = w * ROWS_PER_WORKER + (lane >> 3), chunk = lane & 7;
        float acc[HALF];
#pragma unroll
        for (int i = 0; i < HALF; ++i) acc[i] = 0.f;
        uint32_t it = 0, ci = 0, nst = 0;  // stages, chunks read, staged boxes
        bool ok = true;
        int pending = 0;                   // chunks whose MMAs were fed but not read yet
        bool pending_last = false;
        int out_n = 0, out_c = 0;          // output of the tile being read

        // Reads the oldest pending accumulator; writes the tile out after its last one.
        auto read_chunk = [&]() -> bool {
            const uint32_t buf = ci & 1;
            if (!wait_warp(&sm->acc_full[buf], (ci >> 1) & 1, sm, lim)) return false;
            tc_fence_after();
            const uint32_t tb = lane_addr + buf * TN;
#pragma unroll
            for (int ch = 0; ch < HALF; ch += 16) {
                uint32_t r[16];
                tmem_ld16(tb + ch, &r[0]);
                tmem_wait_ld();
                if (ch + 16 == HALF) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_cluster(empty_c + buf * 8);
                }
#pragma unroll
                for (int i = 0; i < 16; i += 2)
                    add_f32x2(acc[ch + i], acc[ch + i + 1], __uint_as_float(r[i]),
                              __uint_as_float(r[i + 1]));
            }
            ++ci;
            --pending;
            if (!pending_last) return true;
#pragma unroll
            for (int ch = 0; ch < HALF; ch += 32) {
                const int col = out_c + ch;
                const uint32_t sb = my_stg + (nst & 1) * STG_BYTES;
                if (lane == 0 && nst >= 2) bulk_wait_read1();
                __syncwarp();
                uint32_t r[32];
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    r[i] = __float_as_uint(acc[ch + i]);
                    acc[ch + i] = 0.f;
                }
                stage_row(sb, lane, r);
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) {
                    if (col < a.d && out_n < a.n) tma_reduce_add_2d(&tm_dw, sb, col, out_n);
                    bulk_commit();
                }
                ++nst;
            }
            return true;
        };

        for (int t = pair; ok && t < total; t += npairs) {
            const int tn0 = (t % a.tiles_m) * TM, tc0 = (t / a.tiles_m) * TN;
            const int grp = (tc0 + (int)rank * HALF) / ckpt::kGroup + (chunk >> 1);
            const bool has_grp = tc0 + (int)rank * HALF + 16 * chunk < a.d;
            const uint8_t* scol = a.c.scales + (has_grp ? grp : 0);
            auto load_codes = [&](int kb, uint32_t* c) {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int64_t r = (int64_t)kb * KB + row0 + 4 * j;
                    c[j] = r < K && has_grp ? __ldg(scol + r * a.c.ld_scales) : 3u;
                }
            };
            uint32_t codes[2][2];  // scale bytes of the next two stages
            load_codes(0, codes[0]);
            load_codes(1, codes[1]);
            for (int kb = 0; kb < kblocks; ++kb, ++it) {
                const uint32_t s = it % IN_STAGES, b = it % B_STAGES;
                if (!(ok = wait_warp(&sm->full[s], (it / IN_STAGES) & 1, sm, lim))) break;
                // the MMAs of stage it - B_STAGES have read this B slot
                if (it >= B_STAGES) {
                    const uint32_t u = it - B_STAGES;
                    if (!(ok = wait_warp(&sm->used[u % IN_STAGES], (u / IN_STAGES) & 1, sm, lim)))
                        break;
                }
                const int valid = (int)min((int64_t)KB, K - (int64_t)kb * KB);
                uint8_t* in = base + s * IN_BYTES;
                uint8_t* bt = base + OFF_B + b * B_BYTES;
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int row = row0 + 4 * j;
                    const uint4 v = *reinterpret_cast<const uint4*>(in + A_BYTES + row * HALF + 16 * chunk);
                    const Scale sc = make_scale(codes[0][j], format);
                    uint4 o[2];
                    to_bf16x4(v.x, sc, format, o[0].x, o[0].y);
                    to_bf16x4(v.y, sc, format, o[0].z, o[0].w);
                    to_bf16x4(v.z, sc, format, o[1].x, o[1].y);
                    to_bf16x4(v.w, sc, format, o[1].z, o[1].w);
                    if (row >= valid) {
                        o[0] = o[1] = make_uint4(0u, 0u, 0u, 0u);
                        // this row of dy: 8 lanes clear its 16 vectors
                        uint8_t* ar = in + (row >> 3) * 1024 + (row & 7) * 128 + 16 * chunk;
                        *reinterpret_cast<uint4*>(ar) = o[0];
                        *reinterpret_cast<uint4*>(ar + A_BYTES / 2) = o[0];
                    }
                    // 16-byte vectors 2 (chunk % 4) and + 1 of the row's 64-column half; the two
                    // halves store them in opposite order, so a quarter warp hits 8 banks groups
                    const int h = chunk >> 2;
                    uint8_t* br = bt + h * (B_BYTES / 2) + (row >> 3) * 1024 + (row & 7) * 128;
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int half = e ^ h;
                        *reinterpret_cast<uint4*>(br + (((2 * (chunk & 3) + half) ^ (row & 7)) << 4)) =
                            half ? o[1] : o[0];
                    }
                }
                codes[0][0] = codes[1][0];
                codes[0][1] = codes[1][1];
                load_codes(kb + 2, codes[1]);
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(ready_c + b * 8);
                // Once a few stages of this chunk are fed, the chunk before is (nearly) done.
                if (pending && (kb % CHUNK == B_STAGES || kb == kblocks - 1 ||
                                kb % CHUNK == CHUNK - 1)) {
                    if (!(ok = read_chunk())) break;
                }
                if (kb % CHUNK == CHUNK - 1 || kb == kblocks - 1) {
                    pending = 1;
                    pending_last = kb == kblocks - 1;
                    out_n = tn0 + (int)rank * HALF + q * 32;
                    out_c = tc0 + colhalf * HALF;
                }
            }
        }
        if (ok && pending) read_chunk();
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
