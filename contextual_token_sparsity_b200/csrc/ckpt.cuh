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
// magnitudes order like integers).
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

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

__device__ __forceinline__ void unpack8(uint4 v, float* f) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = bf_lo(w[i]);
        f[2 * i + 1] = bf_hi(w[i]);
    }
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    const __nv_bfloat162 r = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&r);
}

__device__ __forceinline__ uint4 pack8(const float* f) {
    return make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7]));
}

// Scale byte of the group of four lanes that this lane belongs to, from the
// lane's 8 values (zeros where it has none).  Called by whole warps.
__device__ __forceinline__ uint32_t scale_code(uint4 v, int format) {
    constexpr uint32_t kMag = 0x7fff7fffu;
    uint32_t m = __vmaxu2(__vmaxu2(v.x & kMag, v.y & kMag), __vmaxu2(v.z & kMag, v.w & kMag));
    m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 2));
    const uint32_t mag = max(m & 0xffffu, m >> 16);
    if (mag >= 0x7f80u) return 255u;
    // magnitude = 1.man 2^(exp - 127); 448 = 1.75 2^8, 127 = (1 + 126/128) 2^6
    const int exp = (int)(mag >> 7), man = (int)(mag & 127u);
    const int code = format == kE4M3 ? exp - 8 + (man > 96) : exp - 6 + (man > 126);
    return (uint32_t)max(code, kMinCode);
}

__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
    return (uint32_t)lo | ((uint32_t)hi << 16);
}

// rne(t) for |t| <= 127 as the low byte of t + 1.5 2^23.
__device__ __forceinline__ uint32_t int8x4(float a, float b, float c, float d) {
    constexpr float kMagic = 12582912.f;
    const uint32_t x = __float_as_uint(a + kMagic), y = __float_as_uint(b + kMagic);
    const uint32_t z = __float_as_uint(c + kMagic), w = __float_as_uint(d + kMagic);
    return __byte_perm(__byte_perm(x, y, 0x0040), __byte_perm(z, w, 0x0040), 0x5410);
}

// Codes of 8 values under the group's scale byte.
__device__ __forceinline__ uint2 encode8(uint4 v, uint32_t code, int format) {
    if (code == 255u) {
        const uint32_t q = format == kE4M3 ? 0x7f7f7f7fu : 0u;
        return make_uint2(q, q);
    }
    const float inv = __uint_as_float((254u - code) << 23);  // 2^-k
    float f[8];
    unpack8(v, f);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] *= inv;
    // the one scale of each format under which a magnitude next to 2^128 could round up to 2^128
    const float most = format == kE4M3 ? 240.f : 63.f;
    if (code == (format == kE4M3 ? 247u : 249u)) {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = fminf(fmaxf(f[i], -most), most);
    }
    if (format == kE4M3)
        return make_uint2(e4m3x4(f[0], f[1], f[2], f[3]), e4m3x4(f[4], f[5], f[6], f[7]));
    return make_uint2(int8x4(f[0], f[1], f[2], f[3]), int8x4(f[4], f[5], f[6], f[7]));
}

__device__ __forceinline__ void decode4(uint32_t q, float s, int format, float* f) {
    if (format == kE4M3) {
        uint32_t h0, h1;
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h0) : "h"((uint16_t)(q & 0xffffu)));
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h1) : "h"((uint16_t)(q >> 16)));
        const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&h0));
        const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&h1));
        f[0] = a.x * s;
        f[1] = a.y * s;
        f[2] = b.x * s;
        f[3] = b.y * s;
    } else {
        // q ^ 0x80 = value + 128 as an unsigned byte; 2^23 + that, minus both offsets
        const uint32_t u = q ^ 0x80808080u;
        constexpr float kBias = 8388608.f + 128.f;
        f[0] = (__uint_as_float(__byte_perm(u, 0x4b000000u, 0x7440)) - kBias) * s;
        f[1] = (__uint_as_float(__byte_perm(u, 0x4b000000u, 0x7441)) - kBias) * s;
        f[2] = (__uint_as_float(__byte_perm(u, 0x4b000000u, 0x7442)) - kBias) * s;
        f[3] = (__uint_as_float(__byte_perm(u, 0x4b000000u, 0x7443)) - kBias) * s;
    }
}

// The 8 values (exact in bf16) of two words of codes.
__device__ __forceinline__ void decode8(uint2 q, uint32_t code, int format, float* f) {
    const float s = code == 255u ? __uint_as_float(0x7fffffffu) : __uint_as_float(code << 23);
    decode4(q.x, s, format, f);
    decode4(q.y, s, format, f + 4);
}

__device__ __forceinline__ void store8(const View& c, int64_t r, int vec, uint4 v, uint32_t code) {
    *reinterpret_cast<uint2*>(c.data + r * c.ld + 8 * (int64_t)vec) = encode8(v, code, c.format);
    if ((vec & 3) == 0) c.scales[r * c.ld_scales + (vec >> 2)] = (uint8_t)code;
}

__device__ __forceinline__ void load8(const View& c, int64_t r, int vec, float* f) {
    const uint2 q = __ldg(reinterpret_cast<const uint2*>(c.data + r * c.ld + 8 * (int64_t)vec));
    decode8(q, __ldg(c.scales + r * c.ld_scales + (vec >> 2)), c.format, f);
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

// One warp per row, 32 vectors (8 groups) at a time.
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
        const uint4* src = a.x + t * a.ld;
        for (int c0 = 0; c0 < a.dvec; c0 += 32) {
            const int c = c0 + lane;
            const uint4 v = c < a.dvec ? __ldg(src + c) : make_uint4(0u, 0u, 0u, 0u);
            const uint32_t code = scale_code(v, a.c.format);
            if (c < a.dvec) store8(a.c, r, c, v, code);
        }
    }
}

__global__ void __launch_bounds__(kThreads) restore_kernel(const RowsArgs a) {
    pdl_entry();
    const int64_t K = clamp_rows(a.kept_total, a.rows);
    const int64_t K_pad = clamp_pad(K, a.pad_to, a.rows);
    const int lane = threadIdx.x & 31;
    const int64_t nwarps = ((int64_t)gridDim.x * kThreads) >> 5;
    for (int64_t r = ((int64_t)blockIdx.x * kThreads + threadIdx.x) >> 5; r < K_pad; r += nwarps) {
        uint4* dst = a.y + r * a.ld;
        for (int c = lane; c < a.dvec; c += 32) {
            uint4 v = make_uint4(0u, 0u, 0u, 0u);
            if (r < K) {
                float f[8];
                load8(a.c, r, c, f);
                v = pack8(f);
            }
            dst[c] = v;
        }
    }
}

// ---------------------------------------------------------------------------
// Gated MLP activation: a = SiLU(g) u forward, both inputs checkpointed on the
// way; backward from the checkpoints with s = 1 / (1 + e^-g):
//   dg = da u s (1 + g (1 - s)),  du = da g s,  a = g s u (recomputed).
// Element-wise, bound by HBM: 8.06 bytes per value forward, 10.06 backward.
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

// 1 / (1 + e^-g) from e^-|g| <= 1, so that nothing overflows for large -g.
__device__ __forceinline__ float sigmoid(float g) {
    const float t = __expf(-fabsf(g));
    return __fdividef(g >= 0.f ? 1.f : t, 1.f + t);
}

__global__ void __launch_bounds__(kThreads) gated_kernel(const GatedArgs p) {
    pdl_entry();
    const int64_t K = clamp_rows(p.kept_total, p.rows);
    const int64_t K_pad = clamp_pad(K, p.pad_to, p.rows);
    const int lane = threadIdx.x & 31;
    const int chunks = (p.dvec + 31) / 32;
    const int64_t nwarps = ((int64_t)gridDim.x * kThreads) >> 5;
    for (int64_t w = ((int64_t)blockIdx.x * kThreads + threadIdx.x) >> 5; w < K_pad * chunks;
         w += nwarps) {
        const int64_t r = w / chunks;
        const int c = (int)(w - r * chunks) * 32 + lane;
        const bool in = c < p.dvec;
        uint4 out = make_uint4(0u, 0u, 0u, 0u);
        if (r < K) {
            const uint4 g = in ? __ldg(p.g + r * p.ld_g + c) : out;
            const uint4 u = in ? __ldg(p.u + r * p.ld_u + c) : out;
            if (p.cg.format >= 0) {
                const uint32_t code = scale_code(g, p.cg.format);
                if (in) store8(p.cg, r, c, g, code);
            }
            if (p.cu.format >= 0) {
                const uint32_t code = scale_code(u, p.cu.format);
                if (in) store8(p.cu, r, c, u, code);
            }
            float gf[8], uf[8];
            unpack8(g, gf);
            unpack8(u, uf);
#pragma unroll
            for (int i = 0; i < 8; ++i) gf[i] = gf[i] * sigmoid(gf[i]) * uf[i];
            out = pack8(gf);
        }
        if (in) p.a[r * p.ld_a + c] = out;
    }
}

__global__ void __launch_bounds__(kThreads) gated_backward_kernel(const GatedArgs p) {
    pdl_entry();
    const int64_t K = clamp_rows(p.kept_total, p.rows);
    const int64_t K_pad = clamp_pad(K, p.pad_to, p.rows);
    const int lane = threadIdx.x & 31;
    const int chunks = (p.dvec + 31) / 32;
    const int64_t nwarps = ((int64_t)gridDim.x * kThreads) >> 5;
    for (int64_t w = ((int64_t)blockIdx.x * kThreads + threadIdx.x) >> 5; w < K_pad * chunks;
         w += nwarps) {
        const int64_t r = w / chunks;
        const int c = (int)(w - r * chunks) * 32 + lane;
        if (c >= p.dvec) continue;
        float dg[8], du[8], act[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) dg[i] = du[i] = act[i] = 0.f;
        if (r < K) {
            float g[8], u[8], da[8];
            unpack8(__ldg(p.da + r * p.ld_da + c), da);
            load8(p.cg, r, c, g);
            load8(p.cu, r, c, u);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float s = sigmoid(g[i]), gs = g[i] * s;
                act[i] = gs * u[i];
                du[i] = da[i] * gs;
                dg[i] = da[i] * u[i] * (s + gs * (1.f - s));
            }
        }
        p.dg[r * p.ld_dg + c] = pack8(dg);
        p.du[r * p.ld_du + c] = pack8(du);
        if (p.a) p.a[r * p.ld_a + c] = pack8(act);
    }
}

}  // namespace ckpt
}  // namespace lemo
