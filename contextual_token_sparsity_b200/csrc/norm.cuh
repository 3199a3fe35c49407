// norm.cuh - the norms before and after a sublayer on the kept tokens, fused
// with the token movement around it:
//
//   gather   y[r] = norm(x[kept[r]]) w + b                 (pre-norm, selective load)
//   scatter  x[kept[r]] += scale gate (norm(y[r]) w + b)   (post-norm, gate, residual scale,
//                                                           in-place addition)
//
// and their backward passes.  With v a row of d values, vhat = (v - mean) rstd
// (mean = 0 for RMS; mean = 0, rstd = 1 without a norm) and g the gradient of
// vhat:
//
//   dv = rstd (g - vhat mean(g vhat) - mean(g))            (no last term for RMS)
//
// gather:   g = dy w;  dx[t] += dv;  dw += sum_r dy vhat;  db += sum_r dy
// scatter:  dz = scale dx[t];  g = dz gate w;  dy[r] = dv;
//           S1 = scale sum_r dx vhat, S2 = scale sum_r dx:  dw += gate S1, db += gate S2,
//           dgate += w S1 + b S2   (per-channel gate: three sums from two)
//           a gate of one value per token and channel goes into S1 and S2, and
//           its gradient rows are dz (vhat w + b).
//
// All rows are bf16; every kernel here is bound by HBM.  One CTA per SM takes
// rows in a fixed order: a producer warp copies the rows that a stage needs
// (cp.async.bulk, whole rows) into a ring in shared memory, up to ~200 KB in
// flight per SM whatever the register use, and each of NG groups of G threads
// takes R rows of a stage at once.  A thread owns the same V vectors of 8 columns in
// every row, so weights stay in registers, column sums are per-thread registers,
// and R rows share one reduction over the group (its latency, ~300 cycles, is what
// a single row per turn was bound by).  The CTAs' column sums are added by a
// second kernel in CTA order, so every result is deterministic.
//
// Measured on the copy rate's scale (6545 GB/s): gather of 8192 x 4096 RMS 27.6 us
// (74 %), with an e4m3 checkpoint of the rows 35 us (74 %, issue slots 57 % busy), its
// backward pass from bf16 rows 53.7 us (76 %) and from the checkpoint 52.8 us (68 %);
// layer norm with bias 31.3, 42.7, 55.4 and 63.2 us;
// scatter of 16384 x 5120 RMS with a gate per token 103 us (99 %), its backward pass
// 142 us (90 %).  Calls of less than 250 MB do not reach the copy rate: a plain copy
// of 8192 x 4096 rows runs at 5.0 TB/s.  The backward passes with a mean spill registers
// (17 warps: 96 each) and are furthest from it: scatter with a channel gate 52 us (59 %) at
// 8192 x 4096, 100 (31 %) at 4096 x 8192 and 101 (30 %) at 2048 x 16384.
#pragma once

#include "ckpt.cuh"
#include "common.cuh"
#include "score.cuh"

namespace lemo {
namespace norm {

using ckpt::add2;
using ckpt::F2;
using ckpt::fma2;
using ckpt::mul2;
using ckpt::pack8;
using ckpt::two;
using ckpt::unf2;
using ckpt::unpack8;
using score::mbar_arrive;
using score::mbar_arrive_expect_tx;
using score::mbar_init;
using score::mbar_try_wait;
using score::smem_u32;

enum Kind : int { kNoNorm = 0, kRms = 1, kLayer = 2 };

constexpr int kMaxParts = 296;  // CTAs that leave column sums in the workspace, at most
constexpr int kMaxD = 16384;
constexpr int kMaxStages = 8;
constexpr int kMaxRows = 32;    // rows of a stage: one per lane of the producer warp
constexpr int kMaxWarps = 20;   // consumer warps
constexpr int kMaxSmem = 220 * 1024;
constexpr uint64_t kDrainNs = 2000000000ull;  // bound of the wait for copies in flight, at the end

// G threads per group, V vectors per thread, R rows per group and stage.
template <int G_, int V_, int R_>
struct Shape {
    static constexpr int G = G_, V = V_, R = R_;
    static constexpr int kConsumers = G > 512 ? G : 512;
    static constexpr int kThreads = kConsumers + 32;  // and the producer warp
    static constexpr int kGroups = kConsumers / G;
    static constexpr int kWarps = G / 32;
    static constexpr int kRows = kGroups * R;         // rows of a stage
    static constexpr bool kNarrow = G * V <= 128;     // rows of up to 1024 values
    static_assert(kRows <= kMaxRows && kConsumers / 32 <= kMaxWarps, "");
};

struct Args {
    int kind;
    int d, dvec;
    float inv_d, eps, scale;
    // rows indexed by token: x forward (read by gather, updated by scatter); the residual
    // gradient dx backward (updated by gather, read by scatter)
    uint4* x;
    int64_t ld_x, x_rows;
    // rows indexed by kept row: y forward (written by gather, read by scatter); dy backward
    // (read by gather, written by scatter)
    uint4* y;
    int64_t ld_y;
    int64_t src_rows;         // backward from bf16 token rows: how many there are
    const uint4* w;           // or nullptr (ones)
    const uint4* b;           // or nullptr (zeros)
    const uint4* gate;        // or nullptr (ones)
    int64_t ld_gate;          // 0: one row for all
    uint4* dgate_rows;
    int64_t ld_dgate;
    float2* stats;            // (mean, rstd) per kept row; forward: optional output
    const int32_t* kept_idx;  // or nullptr: row r is token r
    const int32_t* kept_total;
    int64_t rows;             // rows of every kept-row buffer
    int pad_to;
    ckpt::View c;             // forward: optional output; backward: source when format >= 0
    float* part;              // [grid][2][d] column sums
    // the ring
    int streams, stages;
    struct {
        const uint8_t* base;
        int64_t ld;           // bytes between rows
        uint32_t bytes, off;  // bytes copied, offset in the row's slot
        int by_token;         // indexed by token (else by kept row)
    } in[3];
    uint32_t slot;            // bytes of one row's slot
    uint64_t spin_limit_ns;
    int withhold;         // test hook: the first CTA's first slot never becomes free again
};

struct Smem {
    uint64_t full[kMaxStages];
    uint64_t empty[kMaxStages];
    int32_t token[kMaxStages][kMaxRows];  // -1: no row, or refused
    float2 stats[kMaxStages][kMaxRows];
    float red[2][kMaxWarps][8];           // per consumer warp, two alternating buffers
    int32_t nothing[kMaxRows];            // -1: the tokens of a warp that gave up
    int abort_flag;
};
constexpr int kRing = 5120;  // offset of the ring
static_assert(sizeof(Smem) <= kRing, "the ring starts behind the barriers");

__device__ __noinline__ bool wait_slow(uint64_t* bar, uint32_t parity, Smem* sm, uint64_t limit_ns) {
    const uint64_t t0 = globaltimer_ns();
    for (uint32_t n = 1;; ++n) {
        if (mbar_try_wait(bar, parity)) return true;
        if ((n & 63) == 0) {
            if (*reinterpret_cast<volatile int*>(&sm->abort_flag)) return false;
            if (globaltimer_ns() - t0 > limit_ns) {
                raise_error(LEMO_ERR_TIMEOUT);
                *reinterpret_cast<volatile int*>(&sm->abort_flag) = 1;
                return false;
            }
        }
    }
}

// Warp-uniform: every lane waits for the phase of the given parity (false: gave up).
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, Smem* sm, uint64_t limit_ns) {
    bool ok = mbar_try_wait(bar, parity);
    if (!ok) ok = wait_slow(bar, parity, sm, limit_ns);
    return __all_sync(0xffffffffu, ok);
}

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
            dst),
        "l"(src), "r"(bytes), "r"(smem_u32(bar))
        : "memory");
}

__device__ __forceinline__ uint4 ld_shared(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(addr));
    return v;
}
__device__ __forceinline__ uint2 ld_shared8(uint32_t addr) {
    uint2 v;
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
    return v;
}

// Sums of N values (a power of two, at most 8) over the threads of a group,
// returned to all of them in p.  Inside a warp the values are folded onto lanes
// (N - 1 shuffles instead of 5 N); `red` has two alternating buffers, so one
// barrier per call is enough.
template <typename S, int N>
__device__ __forceinline__ void group_sum(float (&p)[N], Smem* sm, int& flip) {
    const int lane = threadIdx.x & 31;
    int m = 16, idx = 0;
#pragma unroll
    for (int n = N; n > 1; n /= 2, m /= 2) {
        const bool hi = lane & m;
        idx += hi ? n / 2 : 0;
#pragma unroll
        for (int i = 0; i < n / 2; ++i) {
            const float send = hi ? p[i] : p[i + n / 2], keep = hi ? p[i + n / 2] : p[i];
            p[i] = keep + __shfl_xor_sync(0xffffffffu, send, m);
        }
    }
    const int low = m;  // lanes that differ below 2 m hold the same value
#pragma unroll
    for (; m > 0; m /= 2) p[0] += __shfl_xor_sync(0xffffffffu, p[0], m);
    float total = p[0];  // of value idx
    if constexpr (S::kWarps > 1) {
        if ((lane & (2 * low - 1)) == 0) sm->red[flip][threadIdx.x >> 5][idx] = total;
        asm volatile("bar.sync %0, %1;" ::"r"(1 + (int)(threadIdx.x / S::G)), "n"(S::G) : "memory");
        const int w0 = threadIdx.x / S::G * S::kWarps;
        total = 0.f;
        for (int w = lane / N; w < S::kWarps; w += 32 / N) total += sm->red[flip][w0 + w][lane % N];
#pragma unroll
        for (int o = N; o < 32; o *= 2) total += __shfl_xor_sync(0xffffffffu, total, o);
        flip ^= 1;
#pragma unroll
        for (int i = 0; i < N; ++i) p[i] = __shfl_sync(0xffffffffu, total, i);
    } else {
        // value i sits on the lane whose upper bits spell i, highest first
#pragma unroll
        for (int i = 0; i < N; ++i) {
            int src = 0;
#pragma unroll
            for (int n = N, bit = 16; n > 1; n /= 2, bit /= 2) src |= (i & (n / 2)) ? bit : 0;
            p[i] = __shfl_sync(0xffffffffu, total, src);
        }
    }
}

__device__ __forceinline__ uint4 ld_or(const uint4* p, int c, bool in, uint32_t other) {
    return p && in ? __ldg(p + c) : make_uint4(other, other, other, other);
}
constexpr uint32_t kOnes = 0x3f803f80u;  // two bf16 ones

// How K rows are dealt.  Narrow rows (up to 1024 values): a CTA takes `m`
// neighbouring rows per stage (as few as give every CTA the same number of stages),
// and a slot keeps the rows of a stream together, so that rows that
// are neighbours in memory come with one copy: 16384 x 512 was bound by the number
// of copies, 18.4 us forward with one per row, 15.2 so.  Wide rows go round the CTAs one by one,
// each with its streams together: at 8192 x 5120 43 us forward so, 45 as above.
template <typename S>
struct Deal {
    int64_t K;
    int m;
    __device__ __forceinline__ explicit Deal(int64_t k) : K(k) {
        m = S::kRows;
        if (S::kNarrow && k > 0) {  // the same number of rows in each of a CTA's stages
            const int64_t share = (k + gridDim.x - 1) / gridDim.x, stages = (share + m - 1) / m;
            m = (int)((share + stages - 1) / stages);
        }
    }
    __device__ __forceinline__ int64_t row(int64_t st, int j) const {
        return S::kNarrow ? (st * gridDim.x + blockIdx.x) * m + j
                          : blockIdx.x + (st * S::kRows + j) * (int64_t)gridDim.x;
    }
    __device__ __forceinline__ bool any(int64_t st) const { return row(st, 0) < K; }
    __device__ __forceinline__ bool has(int64_t st, int j) const { return j < m && row(st, j) < K; }
};

// Shared-memory address of stream k of row j in slot s.
template <typename S>
__device__ __forceinline__ uint32_t slot_addr(const Args& a, uint32_t ring, int s, int k, int j) {
    if (S::kNarrow)
        return ring + (uint32_t)(s * S::kRows) * a.slot + S::kRows * a.in[k].off + j * a.in[k].bytes;
    return ring + (uint32_t)(s * S::kRows + j) * a.slot + a.in[k].off;
}

// The producer warp: lane j brings row j of a stage; narrow rows that follow one
// another in memory come with the first of them.  `coded`: the consumers read the
// row's scale bytes from global memory right after the copies landed, so they are
// asked for with them (8192 x 4096 backward from a checkpoint: 57.4 -> 53.6 us).
template <typename S>
__device__ __forceinline__ void produce(const Args& a, Smem* sm, uint32_t ring, const Deal<S>& deal,
                                        bool ascending, bool want_stats, bool coded) {
    constexpr int NR = S::kRows;
    const int lane = threadIdx.x & 31;
    int s = 0;
    uint32_t ph = 0;
    bool ok = true;
    int64_t st = 0;
    for (; deal.any(st); ++st) {
        // this stage's tokens and statistics, read while the slot may still be in use
        const int64_t r = deal.row(st, lane);
        int64_t t = -1;
        float2 stat = make_float2(0.f, 1.f);
        if (deal.has(st, lane)) {
            t = a.kept_idx ? a.kept_idx[r] : r;
            bool good = t >= 0 && t < a.x_rows && t < a.src_rows;
            // two rows of one token would race in the kernels that update token rows
            if (ascending && a.kept_idx && r > 0) good = good && a.kept_idx[r - 1] < t;
            if (!good) {
                raise_error(LEMO_ERR_INVALID_ARG);
                t = -1;
            }
            if (want_stats) stat = a.stats[r];
        }
        if (!(ok = wait_warp(&sm->empty[s], ph ^ 1, sm, a.spin_limit_ns))) break;
        const uint32_t rows = __ballot_sync(0xffffffffu, t >= 0);
        const int64_t t_before = __shfl_up_sync(0xffffffffu, t, 1);
        // rows (of kept-row streams) and tokens that do not continue those of the lane before
        const bool follows = lane > 0 && t >= 0 && ((rows >> (lane - 1)) & 1u);
        const uint32_t breaks_r = __ballot_sync(0xffffffffu, !follows);
        const uint32_t breaks_t = __ballot_sync(0xffffffffu, !(follows && t == t_before + 1));
        if (lane < NR) {
            sm->token[s][lane] = (int32_t)t;
            sm->stats[s][lane] = stat;
        }
        __syncwarp();
        if (lane == 0) {
            uint32_t bytes = 0;
            for (int i = 0; i < a.streams; ++i) bytes += a.in[i].bytes;
            mbar_arrive_expect_tx(&sm->full[s], bytes * (uint32_t)__popc(rows));
        }
        __syncwarp();
        if (t >= 0) {
            if (coded) {
                const uint8_t* scales = a.c.scales + r * a.c.ld_scales;
                const int last = (a.d - 1) / ckpt::kGroup;
                for (int j = 0; j < last + 128; j += 128)
                    asm volatile("prefetch.global.L2 [%0];" ::"l"(scales + min(j, last)));
            }
            for (int i = 0; i < a.streams; ++i) {
                const int64_t at = a.in[i].by_token ? t : r;
                uint32_t bytes = a.in[i].bytes;
                if (S::kNarrow && a.in[i].ld == bytes) {
                    const uint32_t breaks = a.in[i].by_token ? breaks_t : breaks_r;
                    if (!((breaks >> lane) & 1u)) continue;  // came with a row before
                    const uint32_t rest = lane < 31 ? breaks >> (lane + 1) : 0u;
                    bytes *= rest ? (uint32_t)__ffs(rest) : 32u - lane;
                }
                bulk_load(slot_addr<S>(a, ring, s, i, lane), a.in[i].base + at * a.in[i].ld, bytes,
                          &sm->full[s]);
            }
        }
        if (++s == a.stages) {
            s = 0;
            ph ^= 1;
        }
    }
    // every copy in flight lands before the CTA leaves, also where its consumers gave up
    for (int64_t j = st > a.stages ? st - a.stages : 0; j < st; ++j) {
        const uint64_t t0 = globaltimer_ns();
        while (!mbar_try_wait(&sm->full[j % a.stages], (uint32_t)(j / a.stages) & 1) &&
               globaltimer_ns() - t0 < kDrainNs) {
        }
    }
}

template <typename S>
__device__ __forceinline__ void init_ring(const Args& a, Smem* sm) {
    if (threadIdx.x < kMaxRows) sm->nothing[threadIdx.x] = -1;
    if (threadIdx.x == 0) {
        for (int s = 0; s < a.stages; ++s) {
            mbar_init(&sm->full[s], 1);
            // (test hook: an arrival more than there will be)
            mbar_init(&sm->empty[s], S::kConsumers / 32 + (a.withhold && blockIdx.x == 0 && s == 0 ? 1 : 0));
        }
        sm->abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncthreads();
}

// Zero rows [K, K_pad) of the kept-row output.
template <typename S>
__device__ __forceinline__ void zero_tail(const Args& a, int64_t K, int64_t K_pad) {
    const int64_t n = (K_pad - K) * a.dvec;
    for (int64_t i = blockIdx.x * (int64_t)S::kThreads + threadIdx.x; i < n;
         i += (int64_t)gridDim.x * S::kThreads)
        a.y[(K + i / a.dvec) * a.ld_y + i % a.dvec] = make_uint4(0u, 0u, 0u, 0u);
}

// ---------------------------------------------------------------------------
// Forward.  Streams: gather x; scatter y, x, (gate rows).  FULL: any norm, with
// or without a bias; otherwise no mean and no bias.
// ---------------------------------------------------------------------------
template <typename S, bool POST, bool FULL>
__global__ void __launch_bounds__(S::kThreads, 1) forward_kernel(const __grid_constant__ Args a) {
    constexpr int G = S::G, V = S::V, R = S::R, NG = S::kGroups;
    extern __shared__ __align__(128) uint8_t smem_raw[];
    Smem* sm = reinterpret_cast<Smem*>(smem_raw);
    init_ring<S>(a, sm);
    pdl_entry();
    const uint32_t ring = smem_u32(smem_raw) + kRing;
    const int64_t K = ckpt::clamp_rows(a.kept_total, a.rows);
    if (!POST) {
        const int64_t K_pad = ckpt::clamp_pad(K, a.pad_to, a.rows);
        if (K_pad > K) zero_tail<S>(a, K, K_pad);
    }
    const Deal<S> deal(K);
    if (threadIdx.x >= S::kConsumers) {
        produce<S>(a, sm, ring, deal, POST, false, false);
        return;
    }
    const int group = threadIdx.x / G, i = threadIdx.x % G;
    int flip = 0;
    uint4 w[V], b[FULL ? V : 1], gate[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int c = v * G + i;
        w[v] = ld_or(a.w, c, c < a.dvec, kOnes);
        if (FULL) b[v] = ld_or(a.b, c, c < a.dvec, 0u);
        if (POST) gate[v] = ld_or(a.ld_gate == 0 ? a.gate : nullptr, c, c < a.dvec, kOnes);
    }
    int s = 0;
    uint32_t ph = 0;
    // A warp whose wait ran out (reported) goes through the rest of its stages without rows: its
    // group's barriers need it.
    bool alive = true;
    for (int64_t st = 0; deal.any(st); ++st) {
        alive = alive && wait_warp(&sm->full[s], ph, sm, a.spin_limit_ns);
        // row q of this group is row q NG + group of the stage
        const int32_t* tokens = alive ? &sm->token[s][group] : sm->nothing;
        const uint32_t base0 = slot_addr<S>(a, ring, s, 0, group);
        auto at = [&](int k, int q, int c) {  // vector c of stream k
            return S::kNarrow ? slot_addr<S>(a, ring, s, k, q * NG + group) + 16 * c
                              : base0 + a.in[k].off + q * (NG * a.slot) + 16 * c;
        };
        uint4 in[R][V];
#pragma unroll
        for (int q = 0; q < R; ++q)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int c = v * G + i;
                in[q][v] = tokens[q * NG] >= 0 && c < a.dvec ? ld_shared(at(0, q, c)) : make_uint4(0u, 0u, 0u, 0u);
            }
        float mean[R], rstd[R];
#pragma unroll
        for (int q = 0; q < R; ++q) {
            mean[q] = 0.f;
            rstd[q] = 1.f;
        }
        if (FULL && a.kind == kLayer) {
#pragma unroll
            for (int q = 0; q < R; ++q) {
                F2 sum = two(0.f);
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    F2 f[4];
                    unpack8(in[q][v], f);
                    sum = add2(sum, add2(add2(f[0], f[1]), add2(f[2], f[3])));
                }
                mean[q] = unf2(sum).x + unf2(sum).y;
            }
            group_sum<S, R>(mean, sm, flip);
#pragma unroll
            for (int q = 0; q < R; ++q) mean[q] *= a.inv_d;
        }
        if (a.kind != kNoNorm) {
#pragma unroll
            for (int q = 0; q < R; ++q) {
                const F2 minus = two(-mean[q]);
                F2 sum = two(0.f), sum2 = two(0.f);
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    if (v * G + i >= a.dvec) continue;
                    F2 f[4];
                    unpack8(in[q][v], f);
                    if (FULL) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) f[j] = add2(f[j], minus);
                    }
                    sum = fma2(f[1], f[1], fma2(f[0], f[0], sum));
                    sum2 = fma2(f[3], f[3], fma2(f[2], f[2], sum2));
                }
                sum = add2(sum, sum2);
                rstd[q] = unf2(sum).x + unf2(sum).y;
            }
            group_sum<S, R>(rstd, sm, flip);
#pragma unroll
            for (int q = 0; q < R; ++q) rstd[q] = rsqrtf(rstd[q] * a.inv_d + a.eps);
        }
        if (a.stats && i == 0) {
#pragma unroll
            for (int q = 0; q < R; ++q)
                if (tokens[q * NG] >= 0) a.stats[deal.row(st, q * NG + group)] = make_float2(mean[q], rstd[q]);
        }
        uint4* out[R];
        uint8_t *data[R], *scales[R];
#pragma unroll
        for (int q = 0; q < R; ++q) {
            const int64_t r = deal.row(st, q * NG + group);
            out[q] = POST ? a.x + (int64_t)tokens[q * NG] * a.ld_x : a.y + r * a.ld_y;
            data[q] = a.c.data + r * a.c.ld;
            scales[q] = a.c.scales + r * a.c.ld_scales;
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = v * G + i;
            F2 wf[4], bf[4];
            unpack8(w[v], wf);
            if (FULL) unpack8(b[v], bf);
#pragma unroll
            for (int q = 0; q < R; ++q) {
                if (tokens[q * NG] < 0) continue;  // the same for the whole group
                if (a.c.format >= 0) ckpt::save8(data[q], scales[q], a.c.format, c, c < a.dvec, in[q][v]);
                if (c >= a.dvec) continue;
                F2 f[4];
                unpack8(in[q][v], f);
                const F2 minus = two(-mean[q]), rs = two(rstd[q]);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    f[j] = FULL ? fma2(mul2(add2(f[j], minus), rs), wf[j], bf[j])
                                : mul2(mul2(f[j], rs), wf[j]);
                if (POST) {
                    F2 gf[4], xf[4];
                    unpack8(a.streams == 3 ? ld_shared(at(2, q, c)) : gate[v], gf);
                    unpack8(ld_shared(at(1, q, c)), xf);
#pragma unroll
                    for (int j = 0; j < 4; ++j) xf[j] = fma2(two(a.scale), mul2(gf[j], f[j]), xf[j]);
                    out[q][c] = pack8(xf);
                } else {
                    out[q][c] = pack8(f);
                }
            }
        }
        __syncwarp();
        if ((threadIdx.x & 31) == 0) mbar_arrive(&sm->empty[s]);
        if (++s == a.stages) {
            s = 0;
            ph ^= 1;
        }
    }
}

// ---------------------------------------------------------------------------
// Backward.  Streams: the normalised row (bf16, or codes: CODED); gather dy;
// scatter dx, (gate rows).  FULL: any norm, and the sums of dy (dn) too;
// otherwise no mean and only the sums with vhat.  Both passes over a row read it
// from shared memory: holding 2 R V raw vectors per thread over the reduction cost
// more in registers than the second read.  The row of dx that a gather updates is
// loaded to registers before the first pass and used after the second.
// ---------------------------------------------------------------------------
template <typename S, bool POST, bool FULL, bool CODED>
__global__ void __launch_bounds__(S::kThreads, 1) backward_kernel(const __grid_constant__ Args a) {
    constexpr int G = S::G, V = S::V, R = S::R, NG = S::kGroups;
    extern __shared__ __align__(128) uint8_t smem_raw[];
    Smem* sm = reinterpret_cast<Smem*>(smem_raw);
    init_ring<S>(a, sm);
    pdl_entry();
    const uint32_t ring = smem_u32(smem_raw) + kRing;
    const int64_t K = ckpt::clamp_rows(a.kept_total, a.rows);
    if (POST) {
        const int64_t K_pad = ckpt::clamp_pad(K, a.pad_to, a.rows);
        if (K_pad > K) zero_tail<S>(a, K, K_pad);
    }
    const Deal<S> deal(K);
    if (threadIdx.x >= S::kConsumers) {
        produce<S>(a, sm, ring, deal, !POST, a.kind != kNoNorm, CODED);
        return;
    }
    const int group = threadIdx.x / G, i = threadIdx.x % G;
    int flip = 0;
    // Four vectors per thread leave no registers for the weights: they come from L1 then.
    constexpr bool kHoldW = V <= 2;
    uint4 w[kHoldW ? V : 1];
    F2 s1[4 * V], s2[FULL ? 4 * V : 1];
#pragma unroll
    for (int v = 0; v < (kHoldW ? V : 1); ++v) w[v] = ld_or(a.w, v * G + i, v * G + i < a.dvec, kOnes);
    auto weight = [&](int v, F2* f) {
        unpack8(kHoldW ? w[kHoldW ? v : 0] : ld_or(a.w, v * G + i, true, kOnes), f);
    };
#pragma unroll
    for (int j = 0; j < 4 * V; ++j) {
        s1[j] = two(0.f);
        if (FULL) s2[j] = two(0.f);
    }
    // scale bytes of this group's next rows
    uint32_t code[CODED ? R : 1][V];
    auto load_codes = [&](int64_t st) {
        if constexpr (CODED) {
#pragma unroll
            for (int q = 0; q < R; ++q) {
                const int64_t r = deal.row(st, q * NG + group);
                const bool on = deal.has(st, q * NG + group);
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const int c = v * G + i;
                    code[q][v] =
                        on && c < a.dvec ? __ldg(a.c.scales + r * a.c.ld_scales + (c >> 2)) : 127u;
                }
            }
        }
    };
    load_codes(0);
    int s = 0;
    uint32_t ph = 0;
    // A warp whose wait ran out (reported) goes through the rest of its stages without rows: its
    // group's barriers need it.
    bool alive = true;
    for (int64_t st = 0; deal.any(st); ++st) {
        alive = alive && wait_warp(&sm->full[s], ph, sm, a.spin_limit_ns);
        // row q of this group is row q NG + group of the stage
        const int32_t* tokens = alive ? &sm->token[s][group] : sm->nothing;
        const float2* stats = &sm->stats[s][group];  // (mean, rstd)
        const uint32_t base0 = slot_addr<S>(a, ring, s, 0, group);
        auto at = [&](int k, int q, int c) {  // vector c of stream k
            return S::kNarrow ? slot_addr<S>(a, ring, s, k, q * NG + group) + 16 * c
                              : base0 + a.in[k].off + q * (NG * a.slot) + 16 * c;
        };
        uint4* out[R];
#pragma unroll
        for (int q = 0; q < R; ++q)
            out[q] = POST ? a.y + deal.row(st, q * NG + group) * a.ld_y : a.x + (int64_t)tokens[q * NG] * a.ld_x;
        uint4 xin[POST ? 1 : R][V];
        if constexpr (!POST) {
#pragma unroll
            for (int q = 0; q < R; ++q)
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const int c = v * G + i;
                    if (tokens[q * NG] >= 0 && c < a.dvec) xin[q][v] = out[q][c];
                }
        }
        auto vhat = [&](int q, int v, F2* f) {
            const int c = v * G + i;
            const float2 m = stats[q * NG];
            if constexpr (CODED) {
                // without a mean, rstd goes into the power-of-two scale: the same values
                ckpt::decode8(ld_shared8(at(0, q, 0) + 8 * c), code[q][v], a.c.format, f, FULL ? 1.f : m.y);
            } else {
                unpack8(ld_shared(at(0, q, c)), f);
            }
            if (FULL) {
#pragma unroll
                for (int j = 0; j < 4; ++j) f[j] = mul2(add2(f[j], two(-m.x)), two(m.y));
            } else if (!CODED) {
#pragma unroll
                for (int j = 0; j < 4; ++j) f[j] = mul2(f[j], two(m.y));
            }
        };
        // Gradient of the row's output (POST: dx).  The residual scale goes into rstd below and
        // into the column sums at the end, a gate of one row into the weights.
        auto grad = [&](int q, int v, F2* f) {
            unpack8(ld_shared(at(1, q, v * G + i)), f);
        };
        auto token_gate = [&](int q, int v, F2* f) {
            unpack8(ld_shared(at(2, q, v * G + i)), f);
        };
        // weights of vector v, times the gate of one row
        auto weight_gate = [&](int v, F2* f) {
            weight(v, f);
            if (POST && a.ld_gate == 0 && a.gate) {
                F2 gf[4];
                unpack8(__ldg(a.gate + v * G + i), gf);
#pragma unroll
                for (int j = 0; j < 4; ++j) f[j] = mul2(f[j], gf[j]);
            }
        };
        F2 p1[R], p2[R];
#pragma unroll
        for (int q = 0; q < R; ++q) p1[q] = p2[q] = two(0.f);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = v * G + i;
            if (c >= a.dvec) continue;
            F2 wf[4];
            weight_gate(v, wf);
#pragma unroll
            for (int q = 0; q < R; ++q) {
                if (tokens[q * NG] < 0) continue;  // no row: nothing goes into the sums
                F2 vv[4], gg[4];
                vhat(q, v, vv);
                grad(q, v, gg);
                if (POST && a.ld_gate) {
                    if (a.dgate_rows) {
                        F2 bf[4];
                        unpack8(ld_or(a.b, c, true, 0u), bf);
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            bf[j] = mul2(mul2(gg[j], two(a.scale)), fma2(vv[j], wf[j], bf[j]));
                        a.dgate_rows[deal.row(st, q * NG + group) * a.ld_dgate + c] = pack8(bf);
                    }
                    F2 gf[4];
                    token_gate(q, v, gf);
#pragma unroll
                    for (int j = 0; j < 4; ++j) gg[j] = mul2(gg[j], gf[j]);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    s1[4 * v + j] = fma2(gg[j], vv[j], s1[4 * v + j]);
                    if (FULL) s2[4 * v + j] = add2(s2[4 * v + j], gg[j]);
                    gg[j] = mul2(gg[j], wf[j]);
                    p1[q] = fma2(gg[j], vv[j], p1[q]);
                    if (FULL) p2[q] = add2(p2[q], gg[j]);
                }
            }
        }
        constexpr int P = FULL ? 2 * R : R;  // mean(g vhat), and mean(g) behind it
        float p[P];
#pragma unroll
        for (int q = 0; q < R; ++q) {
            p[q] = unf2(p1[q]).x + unf2(p1[q]).y;
            if (FULL) p[P - R + q] = unf2(p2[q]).x + unf2(p2[q]).y;
        }
        if (a.kind != kNoNorm) group_sum<S, P>(p, sm, flip);
#pragma unroll
        for (int q = 0; q < P; ++q)
            p[q] = a.kind == kNoNorm || (q >= R && a.kind != kLayer) ? 0.f : -p[q] * a.inv_d;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = v * G + i;
            if (c >= a.dvec) continue;
            F2 wf[4];
            weight_gate(v, wf);
#pragma unroll
            for (int q = 0; q < R; ++q) {
                if (tokens[q * NG] < 0) continue;
                F2 vv[4], gg[4];
                vhat(q, v, vv);
                grad(q, v, gg);
                if (POST && a.ld_gate) {
                    F2 gf[4];
                    token_gate(q, v, gf);
#pragma unroll
                    for (int j = 0; j < 4; ++j) gg[j] = mul2(gg[j], gf[j]);
                }
                const F2 rs = two(POST ? stats[q * NG].y * a.scale : stats[q * NG].y);
                const F2 c1 = two(p[q]), c2 = two(FULL ? p[P - R + q] : 0.f);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    gg[j] = fma2(vv[j], c1, mul2(gg[j], wf[j]));
                    if (FULL) gg[j] = add2(gg[j], c2);
                }
                if constexpr (POST) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) gg[j] = mul2(gg[j], rs);
                    out[q][c] = pack8(gg);
                } else {
                    F2 xf[4];
                    unpack8(xin[q][v], xf);
#pragma unroll
                    for (int j = 0; j < 4; ++j) gg[j] = fma2(gg[j], rs, xf[j]);
                    out[q][c] = pack8(gg);
                }
            }
        }
        __syncwarp();
        if ((threadIdx.x & 31) == 0) mbar_arrive(&sm->empty[s]);
        load_codes(st + 1);
        if (++s == a.stages) {
            s = 0;
            ph ^= 1;
        }
    }
    if (!a.part) return;
    // Column sums of this CTA (zeros where it had no row): its groups in order, through the ring
    // (every copy was consumed).
    float f1[8 * V], f2s[FULL ? 8 * V : 1];
#pragma unroll
    for (int j = 0; j < 4 * V; ++j) {
        f1[2 * j] = unf2(s1[j]).x;
        f1[2 * j + 1] = unf2(s1[j]).y;
        if (FULL) {
            f2s[2 * j] = unf2(s2[j]).x;
            f2s[2 * j + 1] = unf2(s2[j]).y;
        }
    }
    if constexpr (NG > 1) {
        float* acc = reinterpret_cast<float*>(smem_raw + kRing);
        for (int gi = 0; gi < NG; ++gi) {
            asm volatile("bar.sync 15, %0;" ::"n"(S::kConsumers) : "memory");
            if (gi == group) {
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const int c = v * G + i;
                    if (c >= a.dvec) continue;
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        // column 8 c + j at [j][c]: neighbouring threads in neighbouring words
                        const int at = j * a.dvec + c;
                        f1[8 * v + j] += gi ? acc[at] : 0.f;
                        acc[at] = f1[8 * v + j];
                        if (FULL) {
                            f2s[8 * v + j] += gi ? acc[a.d + at] : 0.f;
                            acc[a.d + at] = f2s[8 * v + j];
                        }
                    }
                }
            }
        }
        if (group != NG - 1) return;
    }
    float* part = a.part + (int64_t)blockIdx.x * 2 * a.d;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int c = v * G + i;
        if (c >= a.dvec) continue;
#pragma unroll
        for (int j = 0; j < 8; j += 4) {
            *reinterpret_cast<float4*>(part + 8 * c + j) =
                make_float4(f1[8 * v + j], f1[8 * v + j + 1], f1[8 * v + j + 2], f1[8 * v + j + 3]);
            if (FULL)
                *reinterpret_cast<float4*>(part + a.d + 8 * c + j) = make_float4(
                    f2s[8 * v + j], f2s[8 * v + j + 1], f2s[8 * v + j + 2], f2s[8 * v + j + 3]);
        }
    }
}

struct SumArgs {
    const float* part;  // [parts][2][d]
    int d, parts, second;  // second: the sums of dy (dn) are there too
    float scale;           // of all sums
    const uint16_t* w;     // of dgate
    const uint16_t* b;
    const uint16_t* gate;  // per channel, or nullptr
    float* dw;
    float* db;
    float* dgate;
};

constexpr int kSumCols = 32, kSumSlices = 32, kSumBatch = 5;

__device__ __forceinline__ float bf(const uint16_t* p, int c, float other) {
    return p ? __uint_as_float((uint32_t)p[c] << 16) : other;
}

// Adds the CTAs' column sums in CTA order within 32 slices, then the slices in
// order.  All loads are independent and a thread's are issued kSumBatch rows at a
// time (148 CTAs are one batch), so the kernel is one memory latency long.
__global__ void __launch_bounds__(kSumCols * kSumSlices) column_sums_kernel(const SumArgs a) {
    pdl_entry();
    __shared__ float2 acc[kSumSlices][kSumCols];
    const int col = threadIdx.x % kSumCols, slice = threadIdx.x / kSumCols;
    const int c = blockIdx.x * kSumCols + col;
    const bool last = slice == 0 && c < a.d;  // the thread that adds column c up
    float dw = 0.f, db = 0.f, dg = 0.f, gate = 1.f, w = 1.f, b = 0.f;
    if (last) {
        if (a.dw) dw = a.dw[c];
        if (a.db) db = a.db[c];
        if (a.dgate) dg = a.dgate[c];
        gate = bf(a.gate, c, 1.f);
        w = bf(a.w, c, 1.f);
        b = bf(a.b, c, 0.f);
    }
    float2 s = make_float2(0.f, 0.f);
    if (c < a.d) {
        for (int p0 = slice; p0 < a.parts; p0 += kSumSlices * kSumBatch) {
            float x[kSumBatch], y[kSumBatch];
#pragma unroll
            for (int j = 0; j < kSumBatch; ++j) {
                const int p = p0 + j * kSumSlices;
                const float* row = a.part + (int64_t)p * 2 * a.d;
                x[j] = p < a.parts ? row[c] : 0.f;
                y[j] = p < a.parts && a.second ? row[a.d + c] : 0.f;
            }
#pragma unroll
            for (int j = 0; j < kSumBatch; ++j) {
                s.x += x[j];
                s.y += y[j];
            }
        }
    }
    acc[slice][col] = s;
    __syncthreads();
    if (!last) return;
#pragma unroll
    for (int j = 1; j < kSumSlices; ++j) {
        s.x += acc[j][col].x;
        s.y += acc[j][col].y;
    }
    s.x *= a.scale;
    s.y *= a.scale;
    if (a.dw) a.dw[c] = dw + gate * s.x;
    if (a.db) a.db[c] = db + gate * s.y;
    if (a.dgate) a.dgate[c] = dg + (w * s.x + b * s.y);
}

}  // namespace norm
}  // namespace lemo
