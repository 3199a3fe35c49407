// wgrad.cuh - weight gradient of a linear layer whose input is held in an
// 8-bit checkpoint: dW[n, c] += sum_r dy[r, n] xhat[r, c] over the kept rows.
#pragma once

#include "ckpt.cuh"
#include "common.cuh"

namespace lemo {
namespace wgrad {

struct Args {
    ckpt::View c;
    const uint16_t* dy;
    int64_t ld_dy;
    float* dw;
    int64_t ld_dw;
    int n, d;
    const int32_t* kept_total;
    int64_t rows;
};

constexpr int kTile = 64, kDepth = 16;

// 64 x 64 outputs per CTA of 256 threads, 4 x 4 per thread, fp32.
__global__ void __launch_bounds__(256) simple_kernel(const Args a) {
    pdl_entry();
    __shared__ float sa[kDepth][kTile], sb[kDepth][kTile];
    const int64_t K = ckpt::clamp_rows(a.kept_total, a.rows);
    const int n0 = blockIdx.y * kTile, d0 = blockIdx.x * kTile;
    const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
    float acc[4][4] = {};
    for (int64_t r0 = 0; r0 < K; r0 += kDepth) {
        const int row = threadIdx.x / 16, col = (threadIdx.x % 16) * 4;
        const int64_t r = r0 + row;
        for (int j = 0; j < 4; ++j)
            sa[row][col + j] = r < K && n0 + col + j < a.n
                                   ? __uint_as_float((uint32_t)a.dy[r * a.ld_dy + n0 + col + j] << 16)
                                   : 0.f;
        float f[4] = {0.f, 0.f, 0.f, 0.f};
        if (r < K && d0 + col < a.d) {
            const uint32_t q = *reinterpret_cast<const uint32_t*>(a.c.data + r * a.c.ld + d0 + col);
            const uint32_t code = a.c.scales[r * a.c.ld_scales + (d0 + col) / ckpt::kGroup];
            const float s = code == 255u ? __uint_as_float(0x7fffffffu) : __uint_as_float(code << 23);
            ckpt::decode4(q, s, a.c.format, f);
        }
        for (int j = 0; j < 4; ++j) sb[row][col + j] = f[j];
        __syncthreads();
        for (int k = 0; k < kDepth; ++k)
            for (int x = 0; x < 4; ++x)
                for (int y = 0; y < 4; ++y) acc[x][y] += sa[k][ty * 4 + x] * sb[k][tx * 4 + y];
        __syncthreads();
    }
    for (int x = 0; x < 4; ++x)
        for (int y = 0; y < 4; ++y)
            if (n0 + ty * 4 + x < a.n && d0 + tx * 4 + y < a.d)
                a.dw[(int64_t)(n0 + ty * 4 + x) * a.ld_dw + d0 + tx * 4 + y] += acc[x][y];
}

}  // namespace wgrad
}  // namespace lemo
