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
//           S1 = sum_r dz vhat, S2 = sum_r dz:  dw += gate S1, db += gate S2,
//           dgate += w S1 + b S2   (per-channel gate: three sums from two)
//           a gate of one value per token and channel goes into S1 and S2, and
//           its gradient rows are dz (vhat w + b).
//
// All rows are bf16 and are bound by HBM.  A row belongs to a group of G
// threads; a thread owns the same V vectors of 8 columns in every row, so
// weights stay in registers, column sums are per-thread registers, and a row
// costs one or two reductions over the group.  Rows are dealt to CTAs in a
// fixed order and the per-CTA column sums are added by a second kernel in CTA
// order, so every result is deterministic.
#pragma once

#include "ckpt.cuh"
#include "common.cuh"

namespace lemo {
namespace norm {

using ckpt::pack8;
using ckpt::unpack8;

enum Kind : int { kNoNorm = 0, kRms = 1, kLayer = 2 };

constexpr int kMaxParts = 296;  // CTAs that leave column sums in the workspace
constexpr int kMaxD = 16384;

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
    // backward: the normalised rows, from their bf16 source or from a checkpoint
    const uint4* src;
    int64_t ld_src, src_rows;
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
};

template <int G, int V>
struct Shape {
    static constexpr int kThreads = G > 256 ? G : 256;
    static constexpr int kGroups = kThreads / G;
    static constexpr int kWarps = G / 32;
};

// Sums of two values over the G threads of a group, returned to all of them.
// `red` holds two alternating buffers, so one barrier per call is enough.
template <int G, int V>
__device__ __forceinline__ float2 group_sum(float a, float b, float2 (*red)[Shape<G, V>::kWarps],
                                            int& flip) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        a += __shfl_xor_sync(0xffffffffu, a, o);
        b += __shfl_xor_sync(0xffffffffu, b, o);
    }
    if constexpr (G == 32) {
        return make_float2(a, b);
    } else {
        const int warp = (threadIdx.x % G) >> 5;
        if ((threadIdx.x & 31) == 0) red[flip][warp] = make_float2(a, b);
        asm volatile("bar.sync %0, %1;" ::"r"(1 + (int)(threadIdx.x / G)), "n"(G) : "memory");
        a = b = 0.f;
#pragma unroll
        for (int i = 0; i < Shape<G, V>::kWarps; ++i) {
            a += red[flip][i].x;
            b += red[flip][i].y;
        }
        flip ^= 1;
        return make_float2(a, b);
    }
}

// Token of kept row r, or -1 (reported) when it is out of range or, for the
// kernels that update x in place, not above the one before it (two rows of one
// token would race).
__device__ __forceinline__ int64_t token_of(const Args& a, int64_t r, bool ascending, bool report) {
    const int64_t t = a.kept_idx ? a.kept_idx[r] : r;
    bool ok = t >= 0 && t < a.x_rows;
    if (ascending && a.kept_idx && r > 0) ok = ok && a.kept_idx[r - 1] < t;
    if (!ok && report) raise_error(LEMO_ERR_INVALID_ARG);
    return ok ? t : -1;
}

__device__ __forceinline__ uint4 ld_or(const uint4* p, int c, bool in, uint32_t other) {
    return p && in ? __ldg(p + c) : make_uint4(other, other, other, other);
}
constexpr uint32_t kOnes = 0x3f803f80u;  // two bf16 ones

// ---------------------------------------------------------------------------
// Forward
// ---------------------------------------------------------------------------
template <int G, int V, bool POST>
__global__ void __launch_bounds__(Shape<G, V>::kThreads) forward_kernel(const Args a) {
    pdl_entry();
    using S = Shape<G, V>;
    __shared__ float2 red_s[S::kGroups][2][S::kWarps];
    const int group = threadIdx.x / G, i = threadIdx.x % G;
    int flip = 0;
    const int64_t K = ckpt::clamp_rows(a.kept_total, a.rows);
    const int64_t K_pad = POST ? K : ckpt::clamp_pad(K, a.pad_to, a.rows);
    uint4 w[V], b[V], gate[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int c = v * G + i;
        w[v] = ld_or(a.w, c, c < a.dvec, kOnes);
        b[v] = ld_or(a.b, c, c < a.dvec, 0u);
        if (POST) gate[v] = ld_or(a.ld_gate == 0 ? a.gate : nullptr, c, c < a.dvec, kOnes);
    }
    for (int64_t r = blockIdx.x + (int64_t)gridDim.x * group; r < K_pad;
         r += (int64_t)gridDim.x * S::kGroups) {
        if (r >= K) {
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int c = v * G + i;
                if (c < a.dvec) a.y[r * a.ld_y + c] = make_uint4(0u, 0u, 0u, 0u);
            }
            continue;
        }
        const int64_t t = token_of(a, r, POST, i == 0);
        if (t < 0) continue;
        const uint4* row = POST ? a.y + r * a.ld_y : a.x + t * a.ld_x;
        uint4 in[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = v * G + i;
            in[v] = c < a.dvec ? row[c] : make_uint4(0u, 0u, 0u, 0u);
        }
        float mean = 0.f, rstd = 1.f;
        if (a.kind != kNoNorm) {
            if (a.kind == kLayer) {
                float s = 0.f;
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    float f[8];
                    unpack8(in[v], f);
#pragma unroll
                    for (int j = 0; j < 8; ++j) s += f[j];
                }
                mean = group_sum<G, V>(s, 0.f, red_s[group], flip).x * a.inv_d;
            }
            float s = 0.f;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                float f[8];
                unpack8(in[v], f);
                if (v * G + i < a.dvec) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) s += (f[j] - mean) * (f[j] - mean);
                }
            }
            rstd = 1.f / sqrtf(group_sum<G, V>(s, 0.f, red_s[group], flip).x * a.inv_d + a.eps);
        }
        if (a.stats && i == 0) a.stats[r] = make_float2(mean, rstd);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = v * G + i;
            if (a.c.format >= 0) {
                const uint32_t code = ckpt::scale_code(in[v], a.c.format);
                if (c < a.dvec) ckpt::store8(a.c, r, c, in[v], code);
            }
            if (c >= a.dvec) continue;
            float f[8], wf[8], bf[8];
            unpack8(in[v], f);
            unpack8(w[v], wf);
            unpack8(b[v], bf);
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] = (f[j] - mean) * rstd * wf[j] + bf[j];
            if (POST) {
                float gf[8], xf[8];
                unpack8(a.gate && a.ld_gate ? __ldg(a.gate + r * a.ld_gate + c) : gate[v], gf);
                uint4* xp = a.x + t * a.ld_x + c;
                unpack8(*xp, xf);
#pragma unroll
                for (int j = 0; j < 8; ++j) xf[j] += a.scale * (gf[j] * f[j]);
                *xp = pack8(xf);
            } else {
                a.y[r * a.ld_y + c] = pack8(f);
            }
        }
    }
}

// ---------------------------------------------------------------------------
// Backward
// ---------------------------------------------------------------------------
template <int G, int V, bool POST>
__global__ void __launch_bounds__(Shape<G, V>::kThreads) backward_kernel(const Args a) {
    pdl_entry();
    using S = Shape<G, V>;
    __shared__ float2 red_s[S::kGroups][2][S::kWarps];
    __shared__ float acc_s[S::kGroups > 1 ? 2 * 8 * G * V : 1];
    const int group = threadIdx.x / G, i = threadIdx.x % G;
    int flip = 0;
    const int64_t K = ckpt::clamp_rows(a.kept_total, a.rows);
    const int64_t K_pad = POST ? ckpt::clamp_pad(K, a.pad_to, a.rows) : K;
    float s1[8 * V], s2[8 * V];
#pragma unroll
    for (int j = 0; j < 8 * V; ++j) s1[j] = s2[j] = 0.f;
    for (int64_t r = blockIdx.x + (int64_t)gridDim.x * group; r < K_pad;
         r += (int64_t)gridDim.x * S::kGroups) {
        if (r >= K) {
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int c = v * G + i;
                if (c < a.dvec) a.y[r * a.ld_y + c] = make_uint4(0u, 0u, 0u, 0u);
            }
            continue;
        }
        int64_t t = token_of(a, r, !POST, i == 0);
        if (!POST && a.c.format < 0 && t >= a.src_rows) {
            if (i == 0) raise_error(LEMO_ERR_INVALID_ARG);
            t = -1;
        }
        if (t < 0) continue;
        float mean = 0.f, rstd = 1.f;
        if (a.kind != kNoNorm) {
            const float2 st = a.stats[r];
            mean = st.x;
            rstd = st.y;
        }
        // vhat and g of this row
        float vh[8 * V], g[8 * V];
        float p1 = 0.f, p2 = 0.f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = v * G + i;
            float* vv = vh + 8 * v;
            float* gg = g + 8 * v;
            if (c >= a.dvec) {
#pragma unroll
                for (int j = 0; j < 8; ++j) vv[j] = gg[j] = 0.f;
                continue;
            }
            if (a.c.format >= 0)
                ckpt::load8(a.c, r, c, vv);
            else
                unpack8(__ldg(a.src + (POST ? r : t) * a.ld_src + c), vv);
            float wf[8];
            unpack8(ld_or(a.w, c, true, kOnes), wf);
            unpack8(POST ? a.x[t * a.ld_x + c] : a.y[r * a.ld_y + c], gg);
#pragma unroll
            for (int j = 0; j < 8; ++j) vv[j] = (vv[j] - mean) * rstd;
            if (POST) {
                float gf[8];
                unpack8(ld_or(a.gate ? a.gate + r * a.ld_gate : nullptr, c, true, kOnes), gf);
                float bf[8], dgf[8];
                if (a.dgate_rows) unpack8(ld_or(a.b, c, true, 0u), bf);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float dz = a.scale * gg[j], dn = dz * gf[j];
                    const float sum = a.ld_gate ? dn : dz;
                    s1[8 * v + j] += sum * vv[j];
                    s2[8 * v + j] += sum;
                    if (a.dgate_rows) dgf[j] = dz * (vv[j] * wf[j] + bf[j]);
                    gg[j] = dn * wf[j];
                }
                if (a.dgate_rows) a.dgate_rows[r * a.ld_dgate + c] = pack8(dgf);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    s1[8 * v + j] += gg[j] * vv[j];
                    s2[8 * v + j] += gg[j];
                    gg[j] *= wf[j];
                }
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                p1 += gg[j] * vv[j];
                p2 += gg[j];
            }
        }
        float c1 = 0.f, c2 = 0.f;
        if (a.kind != kNoNorm) {
            const float2 p = group_sum<G, V>(p1, p2, red_s[group], flip);
            c1 = p.x * a.inv_d;
            c2 = a.kind == kLayer ? p.y * a.inv_d : 0.f;
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = v * G + i;
            if (c >= a.dvec) continue;
            float f[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] = rstd * (g[8 * v + j] - vh[8 * v + j] * c1 - c2);
            if (POST) {
                a.y[r * a.ld_y + c] = pack8(f);
            } else {
                uint4* xp = a.x + t * a.ld_x + c;
                float xf[8];
                unpack8(*xp, xf);
#pragma unroll
                for (int j = 0; j < 8; ++j) f[j] += xf[j];
                *xp = pack8(f);
            }
        }
    }
    if (!a.part || blockIdx.x >= K) return;
    // column sums of this CTA: its groups in order
    if constexpr (S::kGroups > 1) {
        for (int gi = 0; gi < S::kGroups; ++gi) {
            __syncthreads();
            if (gi == group) {
#pragma unroll
                for (int j = 0; j < 8 * V; ++j) {
                    const int at = j * G + i;
                    acc_s[at] = gi ? acc_s[at] + s1[j] : s1[j];
                    acc_s[8 * G * V + at] = gi ? acc_s[8 * G * V + at] + s2[j] : s2[j];
                }
            }
        }
        if (group != S::kGroups - 1) return;
#pragma unroll
        for (int j = 0; j < 8 * V; ++j) {
            s1[j] = acc_s[j * G + i];
            s2[j] = acc_s[8 * G * V + j * G + i];
        }
    }
    float* part = a.part + (int64_t)blockIdx.x * 2 * a.d;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int c = v * G + i;
        if (c >= a.dvec) continue;
#pragma unroll
        for (int j = 0; j < 8; j += 4) {
            *reinterpret_cast<float4*>(part + 8 * c + j) =
                make_float4(s1[8 * v + j], s1[8 * v + j + 1], s1[8 * v + j + 2], s1[8 * v + j + 3]);
            *reinterpret_cast<float4*>(part + a.d + 8 * c + j) =
                make_float4(s2[8 * v + j], s2[8 * v + j + 1], s2[8 * v + j + 2], s2[8 * v + j + 3]);
        }
    }
}

struct SumArgs {
    const float* part;  // [parts][2][d]
    int d, max_parts;
    const int32_t* kept_total;
    int64_t rows;
    const uint16_t* w;     // of dgate
    const uint16_t* b;
    const uint16_t* gate;  // per channel, or nullptr
    float* dw;
    float* db;
    float* dgate;
};

constexpr int kSumCols = 32, kSumSlices = 16;

__device__ __forceinline__ float bf(const uint16_t* p, int c, float other) {
    return p ? __uint_as_float((uint32_t)p[c] << 16) : other;
}

// Adds the CTAs' column sums in CTA order within 16 slices, then the slices in order.
__global__ void __launch_bounds__(kSumCols * kSumSlices) column_sums_kernel(const SumArgs a) {
    pdl_entry();
    __shared__ float2 acc[kSumSlices][kSumCols];
    int64_t K = *a.kept_total;
    if (K > a.rows) K = a.rows;
    if (K <= 0) return;
    const int parts = K < a.max_parts ? (int)K : a.max_parts;
    const int col = threadIdx.x % kSumCols, slice = threadIdx.x / kSumCols;
    const int c = blockIdx.x * kSumCols + col;
    float2 s = make_float2(0.f, 0.f);
    if (c < a.d) {
        for (int p = slice; p < parts; p += kSumSlices) {
            const float* row = a.part + (int64_t)p * 2 * a.d;
            s.x += row[c];
            s.y += row[a.d + c];
        }
    }
    acc[slice][col] = s;
    __syncthreads();
    if (slice != 0 || c >= a.d) return;
#pragma unroll
    for (int j = 1; j < kSumSlices; ++j) {
        s.x += acc[j][col].x;
        s.y += acc[j][col].y;
    }
    const float gate = bf(a.gate, c, 1.f);
    if (a.dw) a.dw[c] += gate * s.x;
    if (a.db) a.db[c] += gate * s.y;
    if (a.dgate) a.dgate[c] += bf(a.w, c, 1.f) * s.x + bf(a.b, c, 0.f) * s.y;
}

}  // namespace norm
}  // namespace lemo
