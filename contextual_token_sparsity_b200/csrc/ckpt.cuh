// ckpt.cuh - activation checkpoints in 8 bits: the codec, saving and
// restoring rows, and the gated MLP whose backward pass reads its gate and up
// activations from their checkpoints.
//
// Format.  A row of d values is cut into groups of 32 columns (the last may be
// short).  A group has one scale 2^k, stored as the byte k + 127, and one code
// per value: e4m3 (largest 448) or int8 (largest 127).  k is the smallest
// integer >= -124 that brings the group's largest magnitude to the format's
// largest, so nothing saturates, and q = rne(v / 2^k).  The values are bf16
// and the scale is a power of two, so v / 2^k is exact and the only error is
// the one rounding to the code's grid; q 2^k has at most 8 significant bits
// and is at least 2^-133 in magnitude, so it is exact in bf16 too (a code that
// would stand for 2^128 is taken one lower).  A group
// that holds an infinity or a NaN stores the scale byte 255 and restores as
// NaN throughout.
//
// Four neighbouring lanes hold one group (8 bf16 each in one 16-byte vector),
// so its maximum costs two shuffles on packed 16-bit magnitudes (bf16
// magnitudes order like integers).  The kernels are bound by HBM, with the issue
// slots next: values are taken as packed fp32 pairs throughout, the scale byte is
// one add and one shift of the magnitude, and the rare cases (infinities, NaN, the
// largest scale) share one branch.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"

namespace lemo {
namespace ckpt {

constexpr int kGroup = 32;       // columns per scale
constexpr int kMinCode = 3;      // 2^-124, the smallest scale

enum Format : int { kNone = -1, kE4M3 = 0, kInt8 = 1 };

// A checkpoint as the kernels see it.
struct View {
    int format;       // Format
    uint8_t* data;    // [rows, ld], one code per value
    int64_t ld;
    uint8_t* scales;  // [rows, ld_scales], one byte per group
    int64_t ld_scales;
};

// (a product: it runs on the FMA pipe, the integer pipe being the busiest here)
__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w * 65536u); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// Two fp32 values worked on by one instruction.
struct F2 {
    uint64_t v;
};
__device__ __forceinline__ F2 f2(float lo, float hi) {
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ float2 unf2(F2 a) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a.v));
    return r;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}
__device__ __forceinline__ F2 two(float x) { return f2(x, x); }

// The eight bf16 values of a vector as four fp32 pairs, and back.
__device__ __forceinline__ void unpack8(uint4 v, F2* f) {
    f[0] = f2(bf_lo(v.x), bf_hi(v.x));
    f[1] = f2(bf_lo(v.y), bf_hi(v.y));
    f[2] = f2(bf_lo(v.z), bf_hi(v.z));
    f[3] = f2(bf_lo(v.w), bf_hi(v.w));
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    const __nv_bfloat162 r = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t pack2(F2 a) {
    const float2 f = unf2(a);
    return pack2(f.x, f.y);
}
__device__ __forceinline__ uint4 pack8(const F2* f) {
    return make_uint4(pack2(f[0]), pack2(f[1]), pack2(f[2]), pack2(f[3]));
}

__device__ __forceinline__ uint32_t e4m3x4(F2 a, F2 b) {
    const float2 x = unf2(a), y = unf2(b);
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(x.y), "f"(x.x));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(y.y), "f"(y.x));
    return (uint32_t)lo | ((uint32_t)hi << 16);
}

// Low bytes of the four floats: rne(t) for |t| <= 127 where they are t + 1.5 2^23.
constexpr float kMagic = 12582912.f;
__device__ __forceinline__ uint32_t low_bytes(F2 a, F2 b) {
    const float2 x = unf2(a), y = unf2(b);
    return __byte_perm(__byte_perm(__float_as_uint(x.x), __float_as_uint(x.y), 0x0040),
                       __byte_perm(__float_as_uint(y.x), __float_as_uint(y.y), 0x0040), 0x5410);
}

// Maximum of the magnitudes of two bf16 pairs (signs arbitrary), NaN if there is one.
__device__ __forceinline__ uint32_t max_abs2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// Codes of this lane's 8 values (zeros where it has none) and the scale byte of
// the group of four lanes that it belongs to.  Called by whole warps.
// Largest magnitude = 1.man 2^(exp - 127); 448 = (1 + 96/128) 2^8 and
// 127 = (1 + 126/128) 2^6: the byte is exp - 8 or exp - 6, one more where man is
// above 96 or 126, i.e. where adding 31 or 1 carries.  u = 128 (byte + 8 or 6).
__device__ __forceinline__ uint2 quantise8(uint4 v, int format, uint32_t& code) {
    uint32_t m = max_abs2(max_abs2(v.x, v.y), max_abs2(v.z, v.w));
    m = max_abs2(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = max_abs2(m, __shfl_xor_sync(0xffffffffu, m, 2));
    const int mag = (int)(max_abs2(m, __byte_perm(m, 0u, 0x1032)) & 0x7fffu);
    const int bias = format == kE4M3 ? 8 : 6;
    const uint32_t u = (uint32_t)max(mag + (format == kE4M3 ? 31 : 1), (kMinCode + bias) << 7) & 0xff80u;
    code = (u >> 7) - bias;
    F2 inv = two(__uint_as_float(((254u + bias) << 23) - u * 65536u));  // 2^-k
    F2 f[4];
    unpack8(v, f);
    if (u >= 0x7f80u) {  // not finite, or the one scale under which 2^128 is next to the largest value
        if (mag >= 0x7f80) {
            code = 255u;
            inv = two(__uint_as_float(0x7fffffffu));  // the codes become e4m3 NaN, or any int8
        } else {
            const float most = (format == kE4M3 ? 240.f : 63.f) * __uint_as_float(code << 23);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 t = unf2(f[i]);
                f[i] = f2(fminf(fmaxf(t.x, -most), most), fminf(fmaxf(t.y, -most), most));
            }
        }
    }
    if (format == kE4M3) {
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = mul2(f[i], inv);
        return make_uint2(e4m3x4(f[0], f[1]), e4m3x4(f[2], f[3]));
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = fma2(f[i], inv, two(kMagic));
    return make_uint2(low_bytes(f[0], f[1]), low_bytes(f[2], f[3]));
}

__device__ __forceinline__ void decode4(uint32_t q, F2 s, int format, F2* f) {
    if (format == kE4M3) {
        uint32_t h0, h1;
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h0) : "h"((uint16_t)(q & 0xffffu)));
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h1) : "h"((uint16_t)(q >> 16)));
        const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&h0));
        const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&h1));
        f[0] = mul2(f2(a.x, a.y), s);
        f[1] = mul2(f2(b.x, b.y), s);
    } else {
        // q ^ 0x80 = value + 128 as an unsigned byte; 2^23 + that, minus both offsets
        const uint32_t u = q ^ 0x80808080u;
        const F2 bias = two(-8388736.f);
        f[0] = mul2(add2(f2(__uint_as_float(__byte_perm(u, 0x4b000000u, 0x7440)),
                            __uint_as_float(__byte_perm(u, 0x4b000000u, 0x7441))), bias), s);
        f[1] = mul2(add2(f2(__uint_as_float(__byte_perm(u, 0x4b000000u, 0x7442)),
                            __uint_as_float(__byte_perm(u, 0x4b000000u, 0x7443))), bias), s);
    }
}

// The 8 values (exact in bf16) of two words of codes, times `by`.
__device__ __forceinline__ void decode8(uint2 q, uint32_t code, int format, F2* f, float by = 1.f) {
    const F2 s = two((code == 255u ? __uint_as_float(0x7fffffffu) : __uint_as_float(code << 23)) * by);
    decode4(q.x, s, format, f);
    decode4(q.y, s, format, f + 2);
}

// Quantises vector `vec` of a row (`in`: the lane has one) whose codes and scales
// start at `data` and `scales`.  Called by whole warps.
__device__ __forceinline__ void save8(uint8_t* data, uint8_t* scales, int format, int vec, bool in,
                                      uint4 v) {
    uint32_t code;
    const uint2 q = quantise8(v, format, code);
    if (!in) return;
    *reinterpret_cast<uint2*>(data + 8 * vec) = q;
    if ((vec & 3) == 0) scales[vec >> 2] = (uint8_t)code;
}

// Rows that exist on the device: kept_total clamped to the buffers' rows.
__device__ __forceinline__ int64_t clamp_rows(const int32_t* kept_total, int64_t rows) {
    int64_t K = *kept_total;
    if (K > rows) {
        if (blockIdx.x == 0 && threadIdx.x == 0) raise_error(LEMO_ERR_CAPACITY);
        K = rows;
    }
    return K < 0 ? 0 : K;
}

// End of the zero tail: K rounded up to pad_to, clamped to the buffers' rows.
__device__ __forceinline__ int64_t clamp_pad(int64_t K, int pad_to, int64_t rows) {
    const int64_t p = (K + pad_to - 1) / pad_to * pad_to;
    if (p > rows) {
        if (blockIdx.x == 0 && threadIdx.x == 0) raise_error(LEMO_ERR_CAPACITY);
        return rows;
    }
    return p;
}

struct RowsArgs {
    const uint4* x;           // save: source rows
    uint4* y;                 // restore: destination rows
    int64_t ld;               // of x or y, in 16-byte vectors
    int64_t x_rows;
    int dvec;
    const int32_t* kept_idx;  // save: source row ids (nullptr = 0, 1, 2, ...)
    const int32_t* kept_total;
    int64_t rows;
    int pad_to;
    View c;
};

constexpr int kThreads = 256;
constexpr int kUnroll = 4;  // vectors per lane in flight

// Item w of a grid of warps is chunk w % chunks (32 vectors) of row w / chunks; a
// warp's next item is nwarps further: all warps together walk through neighbouring
// memory, and they end at the same time.
struct Walk {
    int64_t r, dr;
    int c, dc, chunks;
    __device__ __forceinline__ Walk(int64_t w, int64_t nwarps, int n) : chunks(n) {
        r = w / n;
        c = (int)(w - r * n);
        dr = nwarps / n;
        dc = (int)(nwarps - dr * n);
    }
    __device__ __forceinline__ void next() {
        r += dr;
        c += dc;
        if (c >= chunks) {
            c -= chunks;
            ++r;
        }
    }
};

// One warp per row, 128 vectors (32 groups) at a time: 16384 x 4096 takes 32.1 us
// (97 % of the rate of a copy; 35.8 with 256 vectors, 42 as a walk over items, which
// looks a row's id up for each).
__global__ void __launch_bounds__(kThreads) save_kernel(const RowsArgs a) {
    pdl_entry();
    const int64_t K = clamp_rows(a.kept_total, a.rows);
    const int lane = threadIdx.x & 31;
    const int64_t nwarps = ((int64_t)gridDim.x * kThreads) >> 5;
    for (int64_t r = ((int64_t)blockIdx.x * kThreads + threadIdx.x) >> 5; r < K; r += nwarps) {
        const int64_t t = a.kept_idx ? a.kept_idx[r] : r;
        if (t < 0 || t >= a.x_rows) {
            if (lane == 0) raise_error(LEMO_ERR_INVALID_ARG);
            continue;
        }
        // lane's pointers: its vectors are 32 apart
        const uint4* src = a.x + t * a.ld + lane;
        uint8_t* data = a.c.data + r * a.c.ld + 8 * lane;
        uint8_t* scales = a.c.scales + r * a.c.ld_scales + (lane >> 2);
        for (int left = a.dvec - lane; left + lane > 0; left -= 32 * kUnroll) {
            uint4 v[kUnroll];
#pragma unroll
            for (int u = 0; u < kUnroll; ++u)
                v[u] = 32 * u < left ? __ldcs(src + 32 * u) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                if (32 * u >= left + lane) break;  // warp-uniform
                uint32_t code;
                const uint2 q = quantise8(v[u], a.c.format, code);
                if (32 * u >= left) continue;
                *reinterpret_cast<uint2*>(data + 256 * u) = q;
                if ((lane & 3) == 0) scales[8 * u] = (uint8_t)code;
            }
            src += 32 * kUnroll;
            data += 256 * kUnroll;
            scales += 8 * kUnroll;
        }
    }
}

// A walk over items: 16384 x 4096 takes 35.6 us (87 % of the rate of a copy; 39.3
// with a warp per row, whose rounds of whole rows end unevenly).
__global__ void __launch_bounds__(kThreads) restore_kernel(const RowsArgs a) {
    pdl_entry();
    const int64_t K = clamp_rows(a.kept_total, a.rows);
    const int64_t K_pad = clamp_pad(K, a.pad_to, a.rows);
    const int lane = threadIdx.x & 31;
    const int64_t nwarps = ((int64_t)gridDim.x * kThreads) >> 5;
    Walk at(((int64_t)blockIdx.x * kThreads + threadIdx.x) >> 5, nwarps, (a.dvec + 31) / 32);
    while (at.r < K_pad) {
        int64_t r[kUnroll];
        int c[kUnroll];
        uint2 q[kUnroll];
        uint32_t code[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            r[u] = at.r;
            c[u] = at.c * 32 + lane;
            at.next();
            q[u] = make_uint2(0u, 0u);  // a row of the tail: zeros
            code[u] = 127u;
            if (r[u] < K && c[u] < a.dvec) {
                q[u] = __ldcs(reinterpret_cast<const uint2*>(a.c.data + r[u] * a.c.ld) + c[u]);
                code[u] = __ldg(a.c.scales + r[u] * a.c.ld_scales + (c[u] >> 2));
            }
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            if (r[u] >= K_pad || c[u] >= a.dvec) continue;
            F2 f[4];
            decode8(q[u], code[u], a.c.format, f);
            a.y[r[u] * a.ld + c[u]] = pack8(f);
        }
    }
}

// ---------------------------------------------------------------------------
// Gated MLP activation: a = SiLU(g) u forward, both inputs checkpointed on the
// way; backward from the checkpoints with s = 1 / (1 + e^-g):
//   dg = da u s (1 + g (1 - s)),  du = da g s,  a = g s u (recomputed).
// Element-wise, bound by HBM: 8.06 bytes per value forward, 10.06 backward.  At
// 8192 x 11008 with e4m3 checkpoints: forward 125 us (89 % of the rate of a copy,
// issue slots next; 129 with a sigmoid from e^-|g| and a choice by g's sign),
// backward 149 us (93 %).
// ---------------------------------------------------------------------------
struct GatedArgs {
    const uint4* g;
    const uint4* u;
    int64_t ld_g, ld_u;       // in 16-byte vectors, as all strides here
    uint4* a;
    int64_t ld_a;
    const uint4* da;
    int64_t ld_da;
    uint4* dg;
    int64_t ld_dg;
    uint4* du;
    int64_t ld_du;
    int dvec;
    const int32_t* kept_total;
    int64_t rows;
    int pad_to;
    View cg, cu;
};

// s = 1 / (1 + e^-g) of a pair, as 2^-24 (1 / (2^-24 h^2 + 2^-24)) with
// h = e^(-g / 2).  The hardware exponential and reciprocal flush results below 2^-126
// to 0: the powers of two keep the quotient above that while s is above 2^-149, and
// where h^2 overflows s is 0 anyway.  No choice by the sign of g is needed.
__device__ __forceinline__ F2 sigmoid2(F2 g) {
    const float2 z = unf2(mul2(g, two(-0.72134752f)));
    float hx, hy, rx, ry;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(hx) : "f"(z.x));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(hy) : "f"(z.y));
    const F2 h = f2(hx, hy);
    const float2 d = unf2(fma2(mul2(h, two(0x1p-24f)), h, two(0x1p-24f)));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(rx) : "f"(d.x));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(ry) : "f"(d.y));
    return mul2(f2(rx, ry), two(0x1p-24f));
}

// A warp takes 32 vectors of a row at a time, with the loads of kPairs (backward
// kBackPairs) such items in flight.  Forward (before the present sigmoid) 129 us with 2 and 141 with 1: the
// arithmetic of one covers the other's loads.  Backward 172 us with 2 and 150 with 1: it
// has five streams, and twice the places in memory at a time cost the DRAM more than
// the loads in flight bring (the same with three CTAs of more registers per SM instead
// of four, 168 us).
constexpr int kPairs = 2, kBackPairs = 1;

__global__ void __launch_bounds__(kThreads, 4) gated_kernel(const GatedArgs p) {
    pdl_entry();
    const int64_t K = clamp_rows(p.kept_total, p.rows);
    const int64_t K_pad = clamp_pad(K, p.pad_to, p.rows);
    const int lane = threadIdx.x & 31;
    const int chunks = (p.dvec + 31) / 32;
    const int64_t nwarps = ((int64_t)gridDim.x * kThreads) >> 5;
    Walk at(((int64_t)blockIdx.x * kThreads + threadIdx.x) >> 5, nwarps, chunks);
    while (at.r < K_pad) {
        int64_t r[kPairs];
        int c[kPairs];
        uint4 g[kPairs], u[kPairs];
#pragma unroll
        for (int k = 0; k < kPairs; ++k) {
            r[k] = at.r;
            c[k] = at.c * 32 + lane;
            at.next();
            g[k] = u[k] = make_uint4(0u, 0u, 0u, 0u);
            if (r[k] < K && c[k] < p.dvec) {
                g[k] = __ldg(p.g + r[k] * p.ld_g + c[k]);
                u[k] = __ldg(p.u + r[k] * p.ld_u + c[k]);
            }
        }
#pragma unroll
        for (int k = 0; k < kPairs; ++k) {
            if (r[k] >= K_pad) break;
            const bool in = c[k] < p.dvec;
            if (r[k] < K) {
                if (p.cg.format >= 0)
                    save8(p.cg.data + r[k] * p.cg.ld, p.cg.scales + r[k] * p.cg.ld_scales, p.cg.format, c[k],
                          in, g[k]);
                if (p.cu.format >= 0)
                    save8(p.cu.data + r[k] * p.cu.ld, p.cu.scales + r[k] * p.cu.ld_scales, p.cu.format, c[k],
                          in, u[k]);
            }
            F2 gf[4], uf[4];  // a row of the tail: zeros, SiLU(0) 0 = 0
            unpack8(g[k], gf);
            unpack8(u[k], uf);
#pragma unroll
            for (int i = 0; i < 4; ++i) gf[i] = mul2(mul2(gf[i], sigmoid2(gf[i])), uf[i]);
            if (in) p.a[r[k] * p.ld_a + c[k]] = pack8(gf);
        }
    }
}

__global__ void __launch_bounds__(kThreads, 4) gated_backward_kernel(const GatedArgs p) {
    pdl_entry();
    const int64_t K = clamp_rows(p.kept_total, p.rows);
    const int64_t K_pad = clamp_pad(K, p.pad_to, p.rows);
    const int lane = threadIdx.x & 31;
    const int chunks = (p.dvec + 31) / 32;
    const int64_t nwarps = ((int64_t)gridDim.x * kThreads) >> 5;
    Walk at(((int64_t)blockIdx.x * kThreads + threadIdx.x) >> 5, nwarps, chunks);
    while (at.r < K_pad) {
        int64_t r[kBackPairs];
        int c[kBackPairs];
        uint4 da[kBackPairs];
        uint2 qg[kBackPairs], qu[kBackPairs];
        uint32_t sg[kBackPairs], su[kBackPairs];
#pragma unroll
        for (int k = 0; k < kBackPairs; ++k) {
            r[k] = at.r;
            c[k] = at.c * 32 + lane;
            at.next();
            da[k] = make_uint4(0u, 0u, 0u, 0u);
            qg[k] = qu[k] = make_uint2(0u, 0u);  // a row of the tail: zeros
            sg[k] = su[k] = 127u;
            if (r[k] < K && c[k] < p.dvec) {
                da[k] = __ldg(p.da + r[k] * p.ld_da + c[k]);
                qg[k] = __ldg(reinterpret_cast<const uint2*>(p.cg.data + r[k] * p.cg.ld) + c[k]);
                qu[k] = __ldg(reinterpret_cast<const uint2*>(p.cu.data + r[k] * p.cu.ld) + c[k]);
                sg[k] = __ldg(p.cg.scales + r[k] * p.cg.ld_scales + (c[k] >> 2));
                su[k] = __ldg(p.cu.scales + r[k] * p.cu.ld_scales + (c[k] >> 2));
            }
        }
#pragma unroll
        for (int k = 0; k < kBackPairs; ++k) {
            if (r[k] >= K_pad || c[k] >= p.dvec) continue;
            F2 g[4], u[4], d[4], act[4];
            decode8(qg[k], sg[k], p.cg.format, g);  // code 0 is value 0 in both formats
            decode8(qu[k], su[k], p.cu.format, u);
            unpack8(da[k], d);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const F2 s = sigmoid2(g[i]), gs = mul2(g[i], s);
                act[i] = mul2(gs, u[i]);
                // s + g s (1 - s)
                const F2 slope = fma2(gs, add2(two(1.f), mul2(s, two(-1.f))), s);
                const F2 du = mul2(d[i], gs);
                g[i] = mul2(mul2(d[i], u[i]), slope);
                u[i] = du;
            }
            p.dg[r[k] * p.ld_dg + c[k]] = pack8(g);
            p.du[r[k] * p.ld_du + c[k]] = pack8(u);
            if (p.a) p.a[r[k] * p.ld_a + c[k]] = pack8(act);
        }
    }
}

}  // namespace ckpt
}  // namespace lemo
