// norm.cu - the layer's pre-norm: the residual's addition with the
// root-mean-square norm, its backward pass, and the read-back of MXFP8 rows.
//
// With s = x + r (r the residual, or 0), per row of H elements:
//   rstd = 1 / sqrt(mean(s^2) + eps)        y = s * rstd * gain
// and in the backward, with xh = s * rstd, a = gain * dy and dsum the gradient
// that reaches the sum past the norm (the residual branch), or 0:
//   dx = dsum + rstd * (a - xh * mean(a * xh))      dgain = sum over rows of dy * xh
// (dx is the gradient of x and of r alike). All sums are held in fp32; each
// output is rounded once.
#include <algorithm>

#include "common.cuh"
#include "moves.cuh"
#include "quant.cuh"

namespace mok {

namespace {

// Sum over the CTA of one value per thread, the same in every thread and in
// every run (shuffles, then the warps' sums in order). `red` holds one float
// per warp; two alternating buffers let one barrier serve each call.
__device__ __forceinline__ float block_sum(float v, float* red) {
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    const int nw = (int)blockDim.x >> 5;
    float s = 0.f;
    for (int w = 0; w < nw; ++w) s += red[w];
    return s;
}

struct NormParams {
    int T, H;
    const __nv_bfloat16* x;
    int64_t ldx;
    const __nv_bfloat16* r;   // or NULL
    int64_t ldr;
    const float* gain;
    float eps;
    __nv_bfloat16* sum;       // any of the outputs may be NULL
    __nv_bfloat16* y;
    uint8_t* y_q;
    uint8_t* y_sf;
    uint8_t* sum_q;
    uint8_t* sum_sf;
    float* rstd;
};

// One CTA per row; thread i holds the 8-element vectors i, i + blockDim.x, ...
// (VPT of them), so the row is read once and stays in registers between the
// sum of squares and the scaling. Lanes 4j..4j+3 of a vector round hold one
// 32-element MXFP8 block.
template <int VPT>
__global__ void __launch_bounds__(1024)
rmsnorm_kernel(const NormParams p) {
    __shared__ float red[32];
    pdl_wait();
    pdl_allow_next();
    const int64_t t = blockIdx.x;
    const int nv = p.H / 8;
    float f[VPT][8];
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int v = threadIdx.x + i * blockDim.x;
        if (v < nv) {
            unpack8(*reinterpret_cast<const uint4*>(p.x + t * p.ldx + 8 * v), f[i]);
            if (p.r) {
                float g[8];
                unpack8(*reinterpret_cast<const uint4*>(p.r + t * p.ldr + 8 * v), g);
#pragma unroll
                for (int j = 0; j < 8; ++j) f[i][j] += g[j];
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) f[i][j] = 0.f;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) ss = fmaf(f[i][j], f[i][j], ss);
    }
    const float rstd = 1.0f / sqrtf(block_sum(ss, red) / (float)p.H + p.eps);
    if (p.rstd && threadIdx.x == 0) p.rstd[t] = rstd;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int v = threadIdx.x + i * blockDim.x;
        const bool in = v < nv;
        const uint4 sb = pack8(f[i]);   // the sum as it is carried on (BF16)
        if (in && p.sum) *reinterpret_cast<uint4*>(p.sum + t * p.H + 8 * v) = sb;
        if (p.sum_q) {
            float b[8];
            unpack8(sb, b);
            uint2 o;
            const uint32_t code = quantize8(b, o);
            if (in) {
                *reinterpret_cast<uint2*>(p.sum_q + t * p.H + 8 * v) = o;
                if ((v & 3) == 0) p.sum_sf[t * (p.H / 32) + v / 4] = (uint8_t)code;
            }
        }
        if (p.y || p.y_q) {
            float y[8];
            if (in) {
                const float4 g0 = __ldg(reinterpret_cast<const float4*>(p.gain + 8 * v));
                const float4 g1 = __ldg(reinterpret_cast<const float4*>(p.gain + 8 * v) + 1);
                const float g[8] = {g0.x, g0.y, g0.z, g0.w, g1.x, g1.y, g1.z, g1.w};
#pragma unroll
                for (int j = 0; j < 8; ++j) y[j] = f[i][j] * rstd * g[j];
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) y[j] = 0.f;
            }
            const uint4 yb = pack8(y);
            if (in && p.y) *reinterpret_cast<uint4*>(p.y + t * p.H + 8 * v) = yb;
            if (p.y_q) {
                // quantised from the BF16 values, so the bytes are those of
                // mok_quantize_rows on y
                float b[8];
                unpack8(yb, b);
                uint2 o;
                const uint32_t code = quantize8(b, o);
                if (in) {
                    *reinterpret_cast<uint2*>(p.y_q + t * p.H + 8 * v) = o;
                    if ((v & 3) == 0) p.y_sf[t * (p.H / 32) + v / 4] = (uint8_t)code;
                }
            }
        }
    }
}

struct NormBwdParams {
    int T, H;
    const __nv_bfloat16* dy;
    const __nv_bfloat16* s;    // the sum in BF16, or
    const uint8_t* s_q;        // its MXFP8 rows
    const uint8_t* s_sf;
    const __nv_bfloat16* dsum; // or NULL
    const float* rstd;
    const float* gain;
    __nv_bfloat16* dx;
    float* part;               // [gridDim.x, H]: dgain of each CTA's rows
    float* dgain;              // [H]
};

// CTA b takes rows b, b + gridDim.x, ...; its threads keep their columns'
// dgain in registers over all of its rows and write one partial row at the
// end, which rmsnorm_dgain_kernel adds up in CTA order.
template <int VPT, bool CK>
__global__ void __launch_bounds__(1024)
rmsnorm_bwd_kernel(const NormBwdParams p) {
    __shared__ float red[2][32];
    pdl_wait();
    pdl_allow_next();
    const int nv = p.H / 8;
    float dg[VPT][8];
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) dg[i][j] = 0.f;
    int it = 0;
    for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x, ++it) {
        const float rstd = __ldg(p.rstd + t);
        float a[VPT][8], xh[VPT][8];
        float dot = 0.f;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int v = threadIdx.x + i * blockDim.x;
            if (v < nv) {
                float dy[8];
                unpack8(__ldg(reinterpret_cast<const uint4*>(p.dy + t * p.H + 8 * v)), dy);
                if constexpr (CK) {
                    const uint2 q = __ldg(reinterpret_cast<const uint2*>(p.s_q + t * p.H + 8 * v));
                    dequantize8(q, __ldg(p.s_sf + t * (p.H / 32) + v / 4), xh[i]);
                } else {
                    unpack8(__ldg(reinterpret_cast<const uint4*>(p.s + t * p.H + 8 * v)), xh[i]);
                }
                const float4 g0 = __ldg(reinterpret_cast<const float4*>(p.gain + 8 * v));
                const float4 g1 = __ldg(reinterpret_cast<const float4*>(p.gain + 8 * v) + 1);
                const float g[8] = {g0.x, g0.y, g0.z, g0.w, g1.x, g1.y, g1.z, g1.w};
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    xh[i][j] *= rstd;
                    dg[i][j] = fmaf(dy[j], xh[i][j], dg[i][j]);
                    a[i][j] = dy[j] * g[j];
                    dot = fmaf(a[i][j], xh[i][j], dot);
                }
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) a[i][j] = xh[i][j] = 0.f;
            }
        }
        const float mean = block_sum(dot, red[it & 1]) / (float)p.H;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int v = threadIdx.x + i * blockDim.x;
            if (v < nv) {
                float d[8];
                if (p.dsum) {
                    unpack8(__ldg(reinterpret_cast<const uint4*>(p.dsum + t * p.H + 8 * v)), d);
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j) d[j] = 0.f;
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) d[j] = fmaf(rstd, a[i][j] - xh[i][j] * mean, d[j]);
                *reinterpret_cast<uint4*>(p.dx + t * p.H + 8 * v) = pack8(d);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int v = threadIdx.x + i * blockDim.x;
        if (v < nv) {
            float* o = p.part + (int64_t)blockIdx.x * p.H + 8 * v;
            *reinterpret_cast<float4*>(o) = make_float4(dg[i][0], dg[i][1], dg[i][2], dg[i][3]);
            *reinterpret_cast<float4*>(o + 4) = make_float4(dg[i][4], dg[i][5], dg[i][6], dg[i][7]);
        }
    }
}

// dgain[h] = sum over the P partial rows, in a fixed order: 8 warps take the
// rows w, w + 8, ..., then the warps' sums are added in order. 32 columns a CTA.
__global__ void __launch_bounds__(256)
rmsnorm_dgain_kernel(const float* __restrict__ part, int P, int H, float* __restrict__ dgain) {
    __shared__ float red[8][32];
    pdl_wait();
    pdl_allow_next();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int h = blockIdx.x * 32 + lane;
    float s = 0.f;
    if (h < H)
        for (int b = warp; b < P; b += 8) s += part[(int64_t)b * H + h];
    red[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && h < H) {
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < 8; ++w) v += red[w][lane];
        dgain[h] = v;
    }
}

// BF16 rows from MXFP8 rows: 8 elements a thread.
__global__ void __launch_bounds__(256)
dequantize_rows_kernel(const uint8_t* __restrict__ q, const uint8_t* __restrict__ sf, int64_t n8,
                       __nv_bfloat16* __restrict__ x) {
    pdl_wait();
    pdl_allow_next();
    for (int64_t v = (int64_t)blockIdx.x * 256 + threadIdx.x; v < n8; v += (int64_t)gridDim.x * 256) {
        float f[8];
        dequantize8(__ldg(reinterpret_cast<const uint2*>(q) + v), __ldg(sf + v / 4), f);
        reinterpret_cast<uint4*>(x)[v] = pack8(f);
    }
}

int sm_count() {
    int dev = 0, n = 0;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
    return n > 0 ? n : 1;
}

// Threads and vectors per thread of a CTA that holds one row.
struct RowShape {
    int threads, vpt;
};
RowShape row_shape(int H) {
    const int nv = H / 8;
    const int vpt = nv <= 512 ? 1 : nv <= 1024 ? 2 : nv <= 4096 ? 4 : 8;
    return {std::max(32, (int)align_up(ceil_div(nv, vpt), 32)), vpt};
}

template <bool CK>
cudaError_t run_bwd(const NormBwdParams& p, int grid, RowShape r, cudaStream_t s) {
    switch (r.vpt) {
        case 1: return launch_after(rmsnorm_bwd_kernel<1, CK>, dim3(grid), dim3(r.threads), 0, s, p);
        case 2: return launch_after(rmsnorm_bwd_kernel<2, CK>, dim3(grid), dim3(r.threads), 0, s, p);
        case 4: return launch_after(rmsnorm_bwd_kernel<4, CK>, dim3(grid), dim3(r.threads), 0, s, p);
        default: return launch_after(rmsnorm_bwd_kernel<8, CK>, dim3(grid), dim3(r.threads), 0, s, p);
    }
}

}  // namespace

int rmsnorm_bwd_partials(int T) { return std::min(T, 2 * sm_count()); }

cudaError_t launch_rmsnorm(int T, int H, const mok_rmsnorm_args& a, cudaStream_t s) {
    NormParams p{};
    p.T = T;
    p.H = H;
    p.x = static_cast<const __nv_bfloat16*>(a.x);
    p.ldx = a.ldx;
    p.r = static_cast<const __nv_bfloat16*>(a.residual);
    p.ldr = a.ldr;
    p.gain = a.gain;
    p.eps = a.eps;
    p.sum = static_cast<__nv_bfloat16*>(a.sum);
    p.y = static_cast<__nv_bfloat16*>(a.y);
    p.y_q = static_cast<uint8_t*>(a.y_q);
    p.y_sf = static_cast<uint8_t*>(a.y_sf);
    p.sum_q = static_cast<uint8_t*>(a.sum_q);
    p.sum_sf = static_cast<uint8_t*>(a.sum_sf);
    p.rstd = a.rstd;
    const RowShape r = row_shape(H);
    switch (r.vpt) {
        case 1: return launch_after(rmsnorm_kernel<1>, dim3(T), dim3(r.threads), 0, s, p);
        case 2: return launch_after(rmsnorm_kernel<2>, dim3(T), dim3(r.threads), 0, s, p);
        case 4: return launch_after(rmsnorm_kernel<4>, dim3(T), dim3(r.threads), 0, s, p);
        default: return launch_after(rmsnorm_kernel<8>, dim3(T), dim3(r.threads), 0, s, p);
    }
}

cudaError_t launch_rmsnorm_backward(int T, int H, const mok_rmsnorm_bwd_args& a, cudaStream_t s) {
    NormBwdParams p{};
    p.T = T;
    p.H = H;
    p.dy = static_cast<const __nv_bfloat16*>(a.dy);
    p.s = static_cast<const __nv_bfloat16*>(a.sum);
    p.s_q = static_cast<const uint8_t*>(a.sum_q);
    p.s_sf = static_cast<const uint8_t*>(a.sum_sf);
    p.dsum = static_cast<const __nv_bfloat16*>(a.dsum);
    p.rstd = a.rstd;
    p.gain = a.gain;
    p.dx = static_cast<__nv_bfloat16*>(a.dx);
    p.part = static_cast<float*>(a.workspace);
    p.dgain = a.dgain;
    const int P = rmsnorm_bwd_partials(T);
    const RowShape r = row_shape(H);
    cudaError_t e = a.sum_q ? run_bwd<true>(p, P, r, s) : run_bwd<false>(p, P, r, s);
    if (e != cudaSuccess) return e;
    return launch_after(rmsnorm_dgain_kernel, dim3(ceil_div(H, 32)), dim3(256), 0, s, (const float*)p.part, P, H,
                        p.dgain);
}

cudaError_t launch_dequantize_rows(const void* q, const void* sf, int T, int H, void* x, cudaStream_t s) {
    const int64_t n8 = (int64_t)T * H / 8;
    const int grid = (int)std::min<int64_t>((n8 + 255) / 256, (int64_t)sm_count() * 16);
    return launch_after(dequantize_rows_kernel, dim3(grid), dim3(256), 0, s, static_cast<const uint8_t*>(q),
                        static_cast<const uint8_t*>(sf), n8, static_cast<__nv_bfloat16*>(x));
}

}  // namespace mok
