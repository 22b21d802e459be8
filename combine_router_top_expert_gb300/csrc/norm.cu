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
// every run: shuffles in each warp, then over the warps' sums. `red` holds a float
// per warp; two alternating buffers let one barrier serve each call.
__device__ __forceinline__ float block_sum(float v, float* red) {
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    const int lane = threadIdx.x & 31;
    if (lane == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    v = lane < ((int)blockDim.x >> 5) ? red[lane] : 0.f;
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    return v;
}

// 8 BF16 values as four pairs.
__device__ __forceinline__ void unpack_pairs(const uint4& v, float2 (&f)[4]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = make_float2(bf16_lo(w[i]), bf16_hi(w[i]));
}
__device__ __forceinline__ uint4 pack_pairs(const float2 (&f)[4]) {
    return make_uint4(pack_bf16x2(f[0].x, f[0].y), pack_bf16x2(f[1].x, f[1].y), pack_bf16x2(f[2].x, f[2].y),
                      pack_bf16x2(f[3].x, f[3].y));
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }
// 8 fp32 values as four pairs.
__device__ __forceinline__ void load8(const float* p, float2 (&f)[4]) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
    f[0] = make_float2(a.x, a.y);
    f[1] = make_float2(a.z, a.w);
    f[2] = make_float2(b.x, b.y);
    f[3] = make_float2(b.z, b.w);
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

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async8(uint32_t dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ uint4 ld_shared16(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ uint2 ld_shared8(uint32_t a) {
    uint2 v;
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
    return v;
}

// One CTA per row; thread i holds the 8-element vectors i, i + blockDim.x, ...
// (VPT of them), so the row is read once and stays in registers between the sum
// of squares and the scaling. Lanes 4j..4j+3 of a vector round hold one
// 32-element MXFP8 block. Several CTAs share an SM and hide each other's waits
// (T = 4096, H = 7168, MXFP8 output: 37 us; CTAs that loop over rows with the next
// one prefetched to shared memory took 44).
template <int VPT>
__global__ void __launch_bounds__(VPT <= 2 ? 512 : 1024, VPT <= 2 ? 4 : 1)
rmsnorm_kernel(const NormParams p) {
    __shared__ __align__(16) float red[32];
    pdl_wait();
    pdl_allow_next();
    const int64_t t = blockIdx.x;
    const int nv = p.H / 8;
    uint4 x[VPT], r[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int v = threadIdx.x + i * blockDim.x;
        x[i] = r[i] = make_uint4(0, 0, 0, 0);
        if (v < nv) {
            x[i] = *reinterpret_cast<const uint4*>(p.x + t * p.ldx + 8 * v);
            if (p.r) r[i] = *reinterpret_cast<const uint4*>(p.r + t * p.ldr + 8 * v);
        }
    }
    float2 f[VPT][4], ss2 = both(0.f);   // packed fp32 pairs: half the instructions
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        float2 g[4];
        unpack_pairs(x[i], f[i]);
        unpack_pairs(r[i], g);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            f[i][j] = __fadd2_rn(f[i][j], g[j]);
            ss2 = __ffma2_rn(f[i][j], f[i][j], ss2);
        }
    }
    const float rstd = 1.0f / sqrtf(block_sum(ss2.x + ss2.y, red) / (float)p.H + p.eps);
    if (p.rstd && threadIdx.x == 0) p.rstd[t] = rstd;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int v = threadIdx.x + i * blockDim.x;
        const bool in = v < nv;
        const uint4 sb = pack_pairs(f[i]);   // the sum as it is carried on (BF16)
        if (in && p.sum) *reinterpret_cast<uint4*>(p.sum + t * p.H + 8 * v) = sb;
        if (p.sum_q) {
            uint2 o;
            const uint32_t code = quantize8_bf16(sb, o);
            if (in) {
                *reinterpret_cast<uint2*>(p.sum_q + t * p.H + 8 * v) = o;
                if ((v & 3) == 0) p.sum_sf[t * (p.H / 32) + v / 4] = (uint8_t)code;
            }
        }
        if (p.y || p.y_q) {
            float2 g[4] = {};
            if (in) load8(p.gain + 8 * v, g);
#pragma unroll
            for (int j = 0; j < 4; ++j) g[j] = __fmul2_rn(__fmul2_rn(f[i][j], both(rstd)), g[j]);
            const uint4 yb = pack_pairs(g);
            if (in && p.y) *reinterpret_cast<uint4*>(p.y + t * p.H + 8 * v) = yb;
            if (p.y_q) {
                // quantised from the BF16 values, so the bytes are those of
                // mok_quantize_rows on y
                uint2 o;
                const uint32_t code = quantize8_bf16(yb, o);
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
//
// A row's block-wide sum stands between its loads and its stores, so the loads
// of the next rows have to be in flight meanwhile: each thread copies its own
// vectors of STAGES - 1 rows ahead to shared memory (cp.async; nobody else reads
// them, so no barrier is needed). Up to H = 8192 what the second half needs stays
// in registers; longer rows read their buffers twice. Rows too long for two buffers (STAGES = 0) are read from memory each time.
template <int VPT, bool CK, int STAGES>
__global__ void __launch_bounds__(1024, 1)
rmsnorm_bwd_kernel(const NormBwdParams p) {
    constexpr bool PF = STAGES > 0;
    extern __shared__ __align__(16) unsigned char bwd_smem[];
    __shared__ float red[2][32];
    constexpr int kSlots = 3 * VPT;   // 16-byte slots of a thread per row: dy, dsum, s
    pdl_wait();
    pdl_allow_next();
    const int H = p.H, nv = H / 8, nt = (int)blockDim.x, tid = (int)threadIdx.x;
    const int rows = (p.T - (int)blockIdx.x + (int)gridDim.x - 1) / (int)gridDim.x;   // this CTA's
    const int64_t stride = (int64_t)gridDim.x * H;
    const float inv_h = 1.0f / (float)H;
    const bool has_dsum = p.dsum != nullptr;
    // running pointers: the row to load next (dy, dsum, s), its scale codes and
    // rstd, the row to write (dx)
    const int64_t at = (int64_t)blockIdx.x * H + 8 * tid;
    const __nv_bfloat16* dy = p.dy + at;
    const __nv_bfloat16* dsum = p.dsum + at;
    const __nv_bfloat16* s16 = p.s + at;
    const uint8_t* s8 = p.s_q + at;
    const uint8_t* sf = p.s_sf + at / 32;
    const float* rstdp = p.rstd + blockIdx.x;
    __nv_bfloat16* dx = p.dx + at;
    // slot i of buffer b: consecutive threads side by side
    const uint32_t smem0 = (uint32_t)__cvta_generic_to_shared(bwd_smem) + tid * 16;
    auto slot = [&](int b, int i) { return smem0 + (uint32_t)((b * kSlots + i) * nt) * 16; };
    auto advance = [&]() {
        dy += stride;
        if (has_dsum) dsum += stride;
        if constexpr (CK) s8 += stride;
        else s16 += stride;
    };
    // PF: start the copies of row n (if there is one) into buffer b
    auto issue = [&](int n, int b) {
        if (n < rows) {
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const int o = 8 * i * nt;
                if (tid + i * nt < nv) {
                    cp_async16(slot(b, i), dy + o);
                    if (has_dsum) cp_async16(slot(b, VPT + i), dsum + o);
                    if constexpr (CK) cp_async8(slot(b, 2 * VPT + i), s8 + o);
                    else cp_async16(slot(b, 2 * VPT + i), s16 + o);
                }
            }
            advance();
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    auto load_codes = [&](uint32_t (&code)[VPT], float& rstd) {
        rstd = __ldg(rstdp);
        rstdp += gridDim.x;
        if constexpr (CK) {
#pragma unroll
            for (int i = 0; i < VPT; ++i)
                if (tid + i * nt < nv) code[i] = __ldg(sf + i * nt / 4);
            sf += stride / 32;
        }
    };
    // 8 elements of the sum and of dy
    auto fetch = [&](int b, int i, uint32_t code, float2 (&s)[4], float2 (&g)[4]) {
        const int o = 8 * i * nt;
        unpack_pairs(PF ? ld_shared16(slot(b, i)) : *reinterpret_cast<const uint4*>(dy + o), g);
        if constexpr (CK) {
            float f[8];
            dequantize8(PF ? ld_shared8(slot(b, 2 * VPT + i)) : *reinterpret_cast<const uint2*>(s8 + o), code, f);
#pragma unroll
            for (int j = 0; j < 4; ++j) s[j] = make_float2(f[2 * j], f[2 * j + 1]);
        } else {
            unpack_pairs(PF ? ld_shared16(slot(b, 2 * VPT + i)) : *reinterpret_cast<const uint4*>(s16 + o), s);
        }
    };
    constexpr bool kKeep = VPT == 1;   // gain, s and u stay in registers over the sum
    float2 dg[VPT][4], gk[4], sk[4], uk[4];
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) dg[i][j] = both(0.f);
#pragma unroll
    for (int j = 0; j < 4; ++j) gk[j] = sk[j] = uk[j] = both(0.f);
    if (kKeep && tid < nv) load8(p.gain + 8 * tid, gk);

    if constexpr (PF) {
#pragma unroll
        for (int n = 0; n < STAGES - 1; ++n) issue(n, n);
    }
    uint32_t code[VPT] = {}, code_next[VPT] = {};
    float rstd = 0.f, rstd_next = 0.f;
    if (rows > 0) load_codes(code, rstd);
    int b = 0;   // buffer of this row
#pragma unroll 1
    for (int n = 0; n < rows; ++n) {
        if (n + 1 < rows) load_codes(code_next, rstd_next);
        if constexpr (PF) {
            // into the buffer of the row before this one (this thread is done with it)
            issue(n + STAGES - 1, b == 0 ? STAGES - 1 : b - 1);
            asm volatile("cp.async.wait_group %0;" ::"n"(STAGES - 1) : "memory");
        }
        float2 dot = both(0.f);
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            if (tid + i * nt < nv) {
                float2 s[4], d[4], g[4];
                fetch(b, i, code[i], s, d);
                if constexpr (!kKeep) load8(p.gain + 8 * (tid + i * nt), g);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 u = __fmul2_rn(d[j], kKeep ? gk[j] : g[j]);
                    dg[i][j] = __ffma2_rn(__fmul2_rn(d[j], both(rstd)), s[j], dg[i][j]);
                    dot = __ffma2_rn(u, s[j], dot);
                    if constexpr (kKeep) {
                        sk[j] = s[j];
                        uk[j] = u;
                    }
                }
            }
        }
        // dx = dsum + rstd u - c s with c = rstd^3 sum(u s) / H
        const float c = -rstd * (rstd * (rstd * (block_sum(dot.x + dot.y, red[n & 1]) * inv_h)));
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            if (tid + i * nt < nv) {
                const int o = 8 * i * nt;
                float2 d[4] = {};
                if (has_dsum) unpack_pairs(PF ? ld_shared16(slot(b, VPT + i)) : *reinterpret_cast<const uint4*>(dsum + o), d);
                float2 s[4], u[4];
                if constexpr (!kKeep) {
                    float2 g[4];
                    fetch(b, i, code[i], s, u);
                    load8(p.gain + 8 * (tid + i * nt), g);
#pragma unroll
                    for (int j = 0; j < 4; ++j) u[j] = __fmul2_rn(u[j], g[j]);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 w = __ffma2_rn(both(rstd), kKeep ? uk[j] : u[j], d[j]);
                    d[j] = __ffma2_rn(both(c), kKeep ? sk[j] : s[j], w);
                }
                *reinterpret_cast<uint4*>(dx + o) = pack_pairs(d);
            }
        }
        dx += stride;
        if constexpr (PF) {
            if (++b == STAGES) b = 0;
        } else {
            advance();
        }
        rstd = rstd_next;
#pragma unroll
        for (int i = 0; i < VPT; ++i) code[i] = code_next[i];
    }
    if constexpr (PF) asm volatile("cp.async.wait_group 0;" ::: "memory");
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int v = tid + i * nt;
        if (v < nv) {
            float* o = p.part + (int64_t)blockIdx.x * H + 8 * v;
            *reinterpret_cast<float4*>(o) = make_float4(dg[i][0].x, dg[i][0].y, dg[i][1].x, dg[i][1].y);
            *reinterpret_cast<float4*>(o + 4) = make_float4(dg[i][2].x, dg[i][2].y, dg[i][3].x, dg[i][3].y);
        }
    }
}

// dgain[h] = sum over the P partial rows, in a fixed order: 32 warps take the
// rows w, w + 32, ... (eight loads in flight), then the warps' sums are added in
// order. 32 columns a CTA.
__global__ void __launch_bounds__(1024)
rmsnorm_dgain_kernel(const float* __restrict__ part, int P, int H, float* __restrict__ dgain) {
    __shared__ float red[32][33];
    pdl_wait();
    pdl_allow_next();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int h = blockIdx.x * 32 + lane;
    float s = 0.f;
    if (h < H) {
        for (int b0 = warp; b0 < P; b0 += 8 * 32) {
            float v[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const int b = b0 + 32 * u;
                v[u] = b < P ? part[(int64_t)b * H + h] : 0.f;
            }
#pragma unroll
            for (int u = 0; u < 8; ++u) s += v[u];
        }
    }
    red[warp][lane] = s;
    __syncthreads();
    // warp w: the sum of column w over the 32 warps' sums
    float v = red[lane][warp];
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    if (lane == 0 && blockIdx.x * 32 + warp < H) dgain[blockIdx.x * 32 + warp] = v;
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
    const int vpt = nv <= 512 ? 1 : nv <= 1024 ? 2 : nv <= 4096 ? 4 : 8;   // at most 512 threads up to H = 16384
    return {std::max(32, (int)align_up(ceil_div(nv, vpt), 32)), vpt};
}

// The backward's CTA: 1024 threads at most, four prefetched rows of dy, dsum and
// s while they fit shared memory, else two, else none; about 1024 threads an SM.
struct BwdShape {
    int threads, vpt, stages, smem, per_sm;
};
BwdShape bwd_shape(int H) {
    const int nv = H / 8, vpt = nv <= 1024 ? 1 : nv <= 2048 ? 2 : nv <= 4096 ? 4 : 8;
    BwdShape b{std::max(32, (int)align_up(ceil_div(nv, vpt), 32)), vpt, 0, 0, 1};
    const int row = 3 * vpt * b.threads * 16, room = 216 * 1024;
    b.per_sm = std::max(1, std::min(1024 / b.threads, 8));
    b.stages = vpt == 1 && 4 * row * b.per_sm <= room ? 4 : vpt == 2 && 2 * row <= room ? 2 : 0;
    b.smem = b.stages * row;
    return b;
}

template <int VPT, bool CK, int STAGES>
cudaError_t run_bwd(const NormBwdParams& p, int grid, const BwdShape& b, cudaStream_t s) {
    auto kern = rmsnorm_bwd_kernel<VPT, CK, STAGES>;
    if (b.smem > 40 * 1024) ensure_smem_attr(reinterpret_cast<const void*>(kern), b.smem);
    return launch_after(kern, dim3(grid), dim3(b.threads), b.smem, s, p);
}
template <bool CK>
cudaError_t run_bwd(const NormBwdParams& p, int grid, const BwdShape& b, cudaStream_t s) {
    if (b.stages == 4) return run_bwd<1, CK, 4>(p, grid, b, s);   // H <= 8192: one vector a thread
    if (b.stages == 2) return run_bwd<2, CK, 2>(p, grid, b, s);
    return b.vpt == 4 ? run_bwd<4, CK, 0>(p, grid, b, s) : run_bwd<8, CK, 0>(p, grid, b, s);
}

}  // namespace

int rmsnorm_bwd_partials(int T, int H) {
    const BwdShape b = bwd_shape(H);
    // with rows prefetched, a CTA that has two is hardly slower than with one
    return std::min(b.stages ? ceil_div(T, 2) : T, b.per_sm * sm_count());
}

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
    const int P = rmsnorm_bwd_partials(T, H);
    const BwdShape b = bwd_shape(H);
    cudaError_t e = a.sum_q ? run_bwd<true>(p, P, b, s) : run_bwd<false>(p, P, b, s);
    if (e != cudaSuccess) return e;
    return launch_after(rmsnorm_dgain_kernel, dim3(ceil_div(H, 32)), dim3(1024), 0, s, (const float*)p.part, P, H,
                        p.dgain);
}

cudaError_t launch_dequantize_rows(const void* q, const void* sf, int T, int H, void* x, cudaStream_t s) {
    const int64_t n8 = (int64_t)T * H / 8;
    const int grid = (int)std::min<int64_t>((n8 + 255) / 256, (int64_t)sm_count() * 16);
    return launch_after(dequantize_rows_kernel, dim3(grid), dim3(256), 0, s, static_cast<const uint8_t*>(q),
                        static_cast<const uint8_t*>(sf), n8, static_cast<__nv_bfloat16*>(x));
}

}  // namespace mok
