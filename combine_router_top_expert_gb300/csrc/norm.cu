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

constexpr int kBwdGroups = 8;   // row groups of a CTA of the backward, at most

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

// The same over the threads of one group (nt threads, whole warps; `id` <
// kBwdGroups names it).
__device__ __forceinline__ float group_sum(float v, float* red, int id, int nt) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    if (nt == 32) return v;
    if (lane == 0) red[((int)threadIdx.x % nt) >> 5] = v;
    __syncwarp();
    asm volatile("bar.sync %0, %1;" ::"r"(id + 1), "r"(nt) : "memory");
    v = lane < (nt >> 5) ? red[lane] : 0.f;
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
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
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
// (T = 4096, H = 7168, the sum out as BF16, y as MXFP8: 32 us, 93% of the copy
// rate, so the bytes bound it; CTAs that loop over rows with the next one prefetched
// to shared memory took 44). Longer rows, BF16 in and out: T = 2048, H = 16384 42 us
// (94%), T = 1024, H = 32768 49 (81%), T = 512, H = 65536 (VPT = 8 spills) 64 (62%).
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
    int group;                 // threads of a row group
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

// A row belongs to a group of `group` threads (whole warps); a CTA has one or
// more groups, and all groups of the grid take rows in turn. A thread keeps its
// columns' dgain in registers over all of its rows; at the end the CTA's groups
// are added up in shared memory and one partial row goes to rmsnorm_dgain_kernel,
// which adds those of all CTAs in order.
//
// A row's group-wide sum stands between its loads and its stores, so the loads of
// the next rows have to be in flight meanwhile: each thread copies its own vectors
// of the rows ahead to shared memory (cp.async; nobody else reads them, so no
// barrier is needed). Up to H = 8192 what the second half needs stays in
// registers; longer rows read their buffers twice. Rows too long for two buffers
// (STAGES = 0) are read from memory each time, and spill. BF16 sums: T = 2048, H = 16384
// 68 us (two buffers, 58% of the copy rate), T = 1024, H = 32768 75 (none, 53%), T = 512,
// H = 65536 124 (32%).
//
// T = 4096, H = 7168 with dsum, both kernels: 40.0 us for a BF16 sum (87% of the
// copy rate; the launches, the first rows' way in and the gain gradient take the
// rest), 42.5 for MXFP8 rows (72%): their 12% fewer bytes are paid back in the
// instructions that unpack them between a row's loads and its barrier. Slower were
// two rows to a barrier (spills, 61 us), 448 threads with two vectors each, two
// CTAs an SM (50), and the second half of a row behind the first half of the next
// over mbarriers (55).
template <int VPT, bool CK, int STAGES>
__global__ void __launch_bounds__(1024, 1)
rmsnorm_bwd_kernel(const NormBwdParams p) {
    constexpr bool PF = STAGES > 0;
    extern __shared__ __align__(16) unsigned char bwd_smem[];
    __shared__ float red[kBwdGroups][2][32];
    constexpr int kSlots = 3 * VPT;   // 16-byte slots of a thread per row: dy, dsum, s
    pdl_wait();
    pdl_allow_next();
    const int H = p.H, nv = H / 8, nt = p.group;
    const int grp = (int)threadIdx.x / nt, tid = (int)threadIdx.x % nt, groups = (int)blockDim.x / nt;
    const int first = (int)blockIdx.x * groups + grp, total = (int)gridDim.x * groups;
    const int rows = first < p.T ? (p.T - 1 - first) / total + 1 : 0;   // this group's
    const int64_t stride = (int64_t)total * H;
    const float inv_h = 1.0f / (float)H;
    const bool has_dsum = p.dsum != nullptr;
    // running element offsets of this thread's first vector: in the row to load
    // next and in the row at hand
    int64_t in = (int64_t)first * H + 8 * tid, out = in;
    uint32_t next = first;   // row whose rstd is loaded next
    // slot i of buffer b: consecutive threads side by side
    const uint32_t smem0 = (uint32_t)__cvta_generic_to_shared(bwd_smem) + threadIdx.x * 16;
    auto slot = [&](int b, int i) { return smem0 + (uint32_t)((b * kSlots + i) * (int)blockDim.x) * 16; };
    // behind the ring, the scale codes of the same rows: a byte for four threads,
    // copied four at a time by every 16th thread where their address allows
    unsigned char* codes = bwd_smem + (size_t)STAGES * kSlots * blockDim.x * 16;
    auto code_slot = [&](int b, int i) { return codes + ((b * VPT + i) * (int)blockDim.x + (int)threadIdx.x) / 4; };
    const bool ring_codes = PF && CK && (H & 127) == 0 && (reinterpret_cast<uintptr_t>(p.s_sf) & 3) == 0;
    // PF: start the copies of row n (if there is one) into buffer b, as one group
    // of copies
    auto issue = [&](int n, int b) {
        if (n < rows) {
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const int o = 8 * i * nt;
                if (tid + i * nt < nv) {
                    cp_async16(slot(b, i), p.dy + in + o);
                    if (has_dsum) cp_async16(slot(b, VPT + i), p.dsum + in + o);
                    if constexpr (CK) {
                        cp_async8(slot(b, 2 * VPT + i), p.s_q + in + o);
                        if (ring_codes && (tid & 15) == 0)
                            cp_async4((uint32_t)__cvta_generic_to_shared(code_slot(b, i)), p.s_sf + (in + o) / 32);
                    } else {
                        cp_async16(slot(b, 2 * VPT + i), p.s + in + o);
                    }
                }
            }
            in += stride;
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    auto load_rstd = [&](int n) {
        float v = 0.f;
        if (n < rows) {
            v = __ldg(p.rstd + next);
            next += total;
        }
        return v;
    };
    // 8 elements of the sum over their common factor, which is returned: a block's
    // scale goes into the factors of its elements (`out` is the offset of the row at
    // hand)
    auto fetch_s = [&](int b, int i, float2 (&s)[4]) {
        const int o = 8 * i * nt;
        if constexpr (CK) {
            const uint32_t code = ring_codes ? *code_slot(b, i) : __ldg(p.s_sf + (out + o) / 32);
            const uint2 q = PF ? ld_shared8(slot(b, 2 * VPT + i)) : *reinterpret_cast<const uint2*>(p.s_q + in + o);
#pragma unroll
            for (int j = 0; j < 4; ++j) s[j] = e4m3_pair(q, j);
            return e8m0_scale(code);
        } else {
            unpack_pairs(PF ? ld_shared16(slot(b, 2 * VPT + i)) : *reinterpret_cast<const uint4*>(p.s + in + o), s);
            return 1.0f;
        }
    };
    auto fetch_dy = [&](int b, int i, float2 (&d)[4]) {
        unpack_pairs(PF ? ld_shared16(slot(b, i)) : *reinterpret_cast<const uint4*>(p.dy + in + 8 * i * nt), d);
    };
    constexpr bool kKeep = VPT == 1;   // the gain and the row's s stay in registers over the sum
    float2 dg[VPT][4], gk[4], sk[4];
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) dg[i][j] = both(0.f);
#pragma unroll
    for (int j = 0; j < 4; ++j) gk[j] = sk[j] = both(0.f);
    float fk = 1.f;   // factor of sk
    if (kKeep && tid < nv) load8(p.gain + 8 * tid, gk);

    constexpr int kAhead = PF ? STAGES - 1 : 0;   // rows in flight beyond this one
    if constexpr (PF) {
#pragma unroll
        for (int n = 0; n < kAhead; ++n) issue(n, n);
    }
    float rstd = load_rstd(0);
    int b = 0;   // this row's buffer
#pragma unroll 1
    for (int n = 0; n < rows; ++n) {
        const float rstd_next = load_rstd(n + 1);
        if constexpr (PF) {
            // into the buffer of the row before this one (this thread is done with it)
            issue(n + kAhead, b == 0 ? STAGES - 1 : b - 1);
            asm volatile("cp.async.wait_group %0;" ::"n"(kAhead) : "memory");
            if constexpr (CK) __syncwarp();   // the codes are other lanes' copies
        }
        float dot = 0.f;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            if (tid + i * nt < nv) {
                float2 s[4], d[4], g[4], dot2 = both(0.f);
                const float f = fetch_s(b, i, s), rf = CK ? rstd * f : rstd;
                fetch_dy(b, i, d);
                if constexpr (!kKeep) load8(p.gain + 8 * (tid + i * nt), g);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 u = __fmul2_rn(d[j], kKeep ? gk[j] : g[j]);
                    dg[i][j] = __ffma2_rn(__fmul2_rn(d[j], both(rf)), s[j], dg[i][j]);
                    dot2 = __ffma2_rn(u, s[j], dot2);
                    if constexpr (kKeep) sk[j] = s[j];
                }
                dot = CK ? fmaf(f, dot2.x + dot2.y, dot) : dot + (dot2.x + dot2.y);
                if constexpr (CK && kKeep) fk = f;
            }
        }
        dot = group_sum(dot, red[grp][n & 1], grp, nt);
        // dx = dsum + rstd u - c s with u = gain dy, c = rstd^3 sum(u s) / H
        const float c = -rstd * (rstd * (rstd * (dot * inv_h)));
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            if (tid + i * nt < nv) {
                const int o = 8 * i * nt;
                float2 d[4] = {}, s[4], u[4], g[4];
                if (has_dsum)
                    unpack_pairs(PF ? ld_shared16(slot(b, VPT + i)) : *reinterpret_cast<const uint4*>(p.dsum + in + o), d);
                fetch_dy(b, i, u);
                float f = fk;
                if constexpr (!kKeep) {
                    f = fetch_s(b, i, s);
                    load8(p.gain + 8 * (tid + i * nt), g);
                }
                const float cf = CK ? c * f : c;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 w = __fmul2_rn(u[j], kKeep ? gk[j] : g[j]);
                    d[j] = __ffma2_rn(both(rstd), w, d[j]);
                    d[j] = __ffma2_rn(both(cf), kKeep ? sk[j] : s[j], d[j]);
                }
                *reinterpret_cast<uint4*>(p.dx + out + o) = pack_pairs(d);
            }
        }
        out += stride;
        if constexpr (!PF) in = out;
        if constexpr (PF) b = b + 1 == STAGES ? 0 : b + 1;
        // the next copies may overwrite codes that other lanes have just read again
        if constexpr (PF && CK && !kKeep) __syncwarp();
        rstd = rstd_next;
    }
    if constexpr (PF) asm volatile("cp.async.wait_group 0;" ::: "memory");
    float* part = p.part + (int64_t)blockIdx.x * H;
    if (groups > 1) {
        // the groups' sums, added in group order (VPT = 1: H floats fit the ring)
        __syncthreads();
        float* sum = reinterpret_cast<float*>(bwd_smem);
        if (tid < nv) {
#pragma unroll
            for (int j = 0; j < 4; ++j) *reinterpret_cast<float2*>(sum + grp * H + 8 * tid + 2 * j) = dg[0][j];
        }
        __syncthreads();
        for (int h = threadIdx.x; h < H; h += blockDim.x) {
            float v = 0.f;
            for (int g = 0; g < groups; ++g) v += sum[g * H + h];
            part[h] = v;
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int v = tid + i * nt;
        if (v < nv) {
            *reinterpret_cast<float4*>(part + 8 * v) = make_float4(dg[i][0].x, dg[i][0].y, dg[i][1].x, dg[i][1].y);
            *reinterpret_cast<float4*>(part + 8 * v + 4) = make_float4(dg[i][2].x, dg[i][2].y, dg[i][3].x, dg[i][3].y);
        }
    }
}

// dgain[h] = sum over the P partial rows, in a fixed order: 8 warps take the rows
// w, w + 8, ... (ten loads in flight), then the warps' sums are added in order. 64
// columns a CTA. The CTAs are small enough (32 registers a thread) to be resident
// beside the backward's CTA of 896 threads, so that they wait there for its end.
constexpr int kDgainCols = 64;
__global__ void __launch_bounds__(256, 8)
rmsnorm_dgain_kernel(const float* __restrict__ part, int P, int H, float* __restrict__ dgain) {
    __shared__ float2 red[8][32];
    pdl_wait();
    pdl_allow_next();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int h = blockIdx.x * kDgainCols + 2 * lane;
    float2 s = both(0.f);
    if (h < H) {
        for (int b0 = warp; b0 < P; b0 += 10 * 8) {
            float2 v[10];
#pragma unroll
            for (int u = 0; u < 10; ++u) {
                const int b = b0 + 8 * u;
                v[u] = b < P ? __ldcg(reinterpret_cast<const float2*>(part + (int64_t)b * H + h)) : both(0.f);
            }
#pragma unroll
            for (int u = 0; u < 10; ++u) s = __fadd2_rn(s, v[u]);
        }
    }
    red[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && h < H) {
#pragma unroll
        for (int w = 1; w < 8; ++w) s = __fadd2_rn(s, red[w][lane]);
        dgain[h] = s.x;   // (4-byte aligned)
        dgain[h + 1] = s.y;
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

// Threads and vectors per thread of a CTA that holds one row.
struct RowShape {
    int threads, vpt;
};
RowShape row_shape(int H) {
    const int nv = H / 8;
    const int vpt = nv <= 512 ? 1 : nv <= 1024 ? 2 : nv <= 4096 ? 4 : 8;   // at most 512 threads up to H = 16384
    return {std::max(32, (int)align_up(ceil_div(nv, vpt), 32)), vpt};
}

// The backward's CTA, one per SM: groups of at most 1024 threads, as many as fit
// 1024 threads (kBwdGroups at most); four prefetched rows a group while they fit
// shared memory, else two, else none.
struct BwdShape {
    int group, groups, vpt, stages, smem;
};
BwdShape bwd_shape(int H) {
    const int nv = H / 8, vpt = nv <= 1024 ? 1 : nv <= 2048 ? 2 : nv <= 4096 ? 4 : 8;
    BwdShape b{std::max(32, (int)align_up(ceil_div(nv, vpt), 32)), 1, vpt, 0, 0};
    b.groups = std::max(1, std::min(1024 / b.group, kBwdGroups));
    b.stages = vpt == 1 ? 4 : vpt == 2 ? 2 : 0;
    b.smem = b.stages * vpt * b.group * b.groups * (3 * 16) + b.stages * vpt * b.group * b.groups / 4;   // 197632 at most
    return b;
}

template <int VPT, bool CK, int STAGES>
cudaError_t run_bwd(const NormBwdParams& p, int grid, const BwdShape& b, cudaStream_t s) {
    auto kern = rmsnorm_bwd_kernel<VPT, CK, STAGES>;
    if (b.smem > 40 * 1024) ensure_smem_attr(reinterpret_cast<const void*>(kern), b.smem);
    return launch_after(kern, dim3(grid), dim3(b.group * b.groups), b.smem, s, p);
}
template <bool CK>
cudaError_t run_bwd(const NormBwdParams& p, int grid, const BwdShape& b, cudaStream_t s) {
    switch (b.vpt) {
        case 1: return run_bwd<1, CK, 4>(p, grid, b, s);
        case 2: return run_bwd<2, CK, 2>(p, grid, b, s);
        case 4: return run_bwd<4, CK, 0>(p, grid, b, s);
        default: return run_bwd<8, CK, 0>(p, grid, b, s);
    }
}

}  // namespace

int rmsnorm_bwd_partials(int T, int H) { return std::min(ceil_div(T, bwd_shape(H).groups), sm_count()); }

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
    p.group = b.group;
    cudaError_t e = a.sum_q ? run_bwd<true>(p, P, b, s) : run_bwd<false>(p, P, b, s);
    if (e != cudaSuccess) return e;
    return launch_after(rmsnorm_dgain_kernel, dim3(ceil_div(H, kDgainCols)), dim3(256), 0, s, (const float*)p.part, P, H,
                        p.dgain);
}

cudaError_t launch_dequantize_rows(const void* q, const void* sf, int T, int H, void* x, cudaStream_t s) {
    const int64_t n8 = (int64_t)T * H / 8;
    const int grid = (int)std::min<int64_t>((n8 + 255) / 256, (int64_t)sm_count() * 16);
    return launch_after(dequantize_rows_kernel, dim3(grid), dim3(256), 0, s, static_cast<const uint8_t*>(q),
                        static_cast<const uint8_t*>(sf), n8, static_cast<__nv_bfloat16*>(x));
}

}  // namespace mok
