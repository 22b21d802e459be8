// checkpoint.cu - the training context of the layer in 8 bits: after a
// training forward, save x, the gate/up pre-activations and the expert outputs
// as MXFP8 rows; before the backward, restore the whole context from them.
//
// What the backward reads is a function of three things: the token rows x (the
// gathered rows A are copies of them), the pre-activations G|U (h is
// silu(G) * U), and the unweighted expert outputs y (the partials). So the
// checkpoint holds x [T, H], G|U [T*k, 2I] and y [T*k, H], each quantised along
// its rows in blocks of 32 (E4M3 elements, E8M0 scales), without the padding
// rows, the copies and h. Restored values are exactly those that the bytes
// stand for; h is formed from the restored G and U, so the context is the one
// of a layer whose activations were those values.
#include <algorithm>

#include "common.cuh"
#include "gemm.cuh"
#include "moves.cuh"
#include "quant.cuh"

namespace mok {

namespace {

// One warp takes one row, and CTAs are short, so that a row's end on one SM starts
// the next there (T = 4096, H = 7168, I = 2048, k = 8, save and restore: 550 us with 4
// warps a CTA, 553 with 8; 565 to 596 with 16 to 4 CTAs of 8 warps an SM that stride
// over the rows).
constexpr int kCkThreads = 128;

// Padded segment offsets (each expert's rows start on a 128-row boundary) by the
// CTA's first warp, 8 experts a lane, and the barrier that publishes them.
__device__ __forceinline__ void ck_offsets(const int32_t* counts, int E, int32_t* poff) {
    static_assert(kMaxE == 256, "8 experts a lane");
    if (threadIdx.x < 32) {
        const int lane = threadIdx.x;
        int n[8], sum = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int e = 8 * lane + i;
            n[i] = e < E ? ceil_div(counts[e], kTileM) * kTileM : 0;
            sum += n[i];
        }
        int s = sum;   // inclusive over the lanes
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int o = __shfl_up_sync(0xffffffffu, s, d);
            if (lane >= d) s += o;
        }
        s -= sum;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (8 * lane + i <= E) poff[8 * lane + i] = s;
            s += n[i];
        }
        if (lane == 31 && E == kMaxE) poff[E] = s;
    }
    __syncthreads();
}

// Last e with start[e] <= r (skips empty segments).
__device__ __forceinline__ int segment_of(const int32_t* start, int E, int r) {
    int lo = 0, hi = E - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (start[mid] <= r) lo = mid; else hi = mid - 1;
    }
    return lo;
}

// Vectors of 8 elements that a lane of the save has in flight: a row is read in
// rounds of kCkBatch * 32 vectors, every load of a round issued before the first is
// used. The save reads 1.07 GB and writes 0.4 at T = 4096, H = 7168, I = 2048, k = 8:
// 208 us (the copy rate of this GPU; one load at a time left it waiting, 278 us).
constexpr int kCkBatch = 4;

// One row of n elements (BF16 or fp32) to MXFP8 by one warp. Every lane runs
// every round: quantize8 exchanges the block's maximum among four.
template <typename In>
__device__ __forceinline__ void save_row(const In* src, int n, uint8_t* q, uint8_t* sf) {
    const int lane = threadIdx.x & 31, nv = n / 8;
#pragma unroll 1
    for (int v0 = lane; v0 - lane < nv; v0 += 32 * kCkBatch) {
        uint32_t w[kCkBatch][sizeof(In) * 2];
#pragma unroll
        for (int u = 0; u < kCkBatch; ++u) {
            const int v = v0 + 32 * u;
#pragma unroll
            for (int i = 0; i < (int)sizeof(In) * 2; ++i) w[u][i] = 0;
            if (v < nv) {
                if constexpr (sizeof(In) == 4) {
                    tc::ldg_v8(src + 8 * v, w[u]);
                } else {
                    const uint4 x = __ldg(reinterpret_cast<const uint4*>(src) + v);
                    w[u][0] = x.x; w[u][1] = x.y; w[u][2] = x.z; w[u][3] = x.w;
                }
            }
        }
#pragma unroll
        for (int u = 0; u < kCkBatch; ++u) {
            const int v = v0 + 32 * u;
            if (v - lane >= nv) break;   // the same in every lane
            float f[8];
            if constexpr (sizeof(In) == 4) {
#pragma unroll
                for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(w[u][i]);
            } else {
                unpack8(make_uint4(w[u][0], w[u][1], w[u][2], w[u][3]), f);
            }
            uint2 o;
            const uint32_t code = quantize8(f, o);
            if (v < nv) {
                reinterpret_cast<uint2*>(q)[v] = o;
                if ((v & 3) == 0) sf[v / 4] = (uint8_t)code;
            }
        }
    }
}

// One warp per row. Row jobs in order: the T*k rows of G|U (gathered from
// their padded places), the T*k partials, the T tokens.
__global__ void __launch_bounds__(kCkThreads, 8)
checkpoint_save_kernel(const CheckpointParams p) {
    __shared__ int32_t poff[kMaxE + 1], off[kMaxE + 1];
    pdl_wait();
    pdl_allow_next();
    for (int e = threadIdx.x; e <= p.E; e += kCkThreads) off[e] = p.offsets[e];
    ck_offsets(p.counts, p.E, poff);
    const int64_t R = (int64_t)p.T * p.k;
    const int64_t jobs = 2 * R + p.T;
    const int W = 2 * p.I;
    const int64_t j = (int64_t)blockIdx.x * (kCkThreads / 32) + (threadIdx.x >> 5);
    if (j >= jobs) return;
    if (j < R) {
        const int e = segment_of(off, p.E, (int)j);
        const int64_t pr = poff[e] + (j - off[e]);
        save_row(p.gu + pr * W, W, p.gu_q + j * W, p.gu_sf + j * (W / 32));
    } else if (j < 2 * R) {
        const int64_t i = j - R;
        save_row(p.partials + i * p.H, p.H, p.y_q + i * p.H, p.y_sf + i * (p.H / 32));
    } else {
        const int64_t t = j - 2 * R;
        save_row(p.x + t * p.H, p.H, p.x_q + t * p.H, p.x_sf + t * (p.H / 32));
    }
}

// One MXFP8 row of n elements to BF16 by one warp.
__device__ __forceinline__ void load_row_bf16(const uint8_t* q, const uint8_t* sf, int n, __nv_bfloat16* dst) {
    const int lane = threadIdx.x & 31;
    for (int v = lane; v < n / 8; v += 32) {
        float f[8];
        dequantize8(__ldg(reinterpret_cast<const uint2*>(q) + v), __ldg(sf + v / 4), f);
        __stcs(reinterpret_cast<uint4*>(dst) + v, pack8(f));
    }
}

// One warp per row. Row jobs in order: the padded rows (A, G|U and h together;
// pad rows are zero, as the training forward leaves them), the T*k partials,
// the T tokens. Rows past the last segment are left alone. Bound by its writes,
// which no launch reads back at once, so they are streamed (1.76 GB against 0.6 read
// at the save's sizes: 335 us, 7.0 TB/s both ways; 341 with plain stores).
__global__ void __launch_bounds__(kCkThreads)
checkpoint_load_kernel(const CheckpointParams p) {
    __shared__ int32_t poff[kMaxE + 1], off[kMaxE + 1];
    pdl_wait();
    pdl_allow_next();
    for (int e = threadIdx.x; e <= p.E; e += kCkThreads) off[e] = p.offsets[e];
    ck_offsets(p.counts, p.E, poff);
    const int lane = threadIdx.x & 31;
    const int64_t R = (int64_t)p.T * p.k, P = poff[p.E];
    const int64_t jobs = P + R + p.T;
    const int W = 2 * p.I;
    const int64_t j = (int64_t)blockIdx.x * (kCkThreads / 32) + (threadIdx.x >> 5);
    if (j >= jobs) return;
    if (j < P) {
        const int e = segment_of(poff, p.E, (int)j);
        const int64_t local = j - poff[e];
        __nv_bfloat16* A = p.A_out + j * p.H;
        float* gu = p.gu_out + j * W;
        __nv_bfloat16* h = p.h_out + j * p.I;
        if (local >= off[e + 1] - off[e]) {
            const uint4 z = make_uint4(0, 0, 0, 0);
            for (int v = lane; v < p.H / 8; v += 32) reinterpret_cast<uint4*>(A)[v] = z;
            for (int v = lane; v < W / 4; v += 32) reinterpret_cast<uint4*>(gu)[v] = z;
            for (int v = lane; v < p.I / 8; v += 32) reinterpret_cast<uint4*>(h)[v] = z;
            return;
        }
        const int64_t r = off[e] + local;
        const int64_t t = __ldg(p.row_src + r) / p.k;
        load_row_bf16(p.x_q + t * p.H, p.x_sf + t * (p.H / 32), p.H, A);
        for (int v = lane; v < p.I / 8; v += 32) {
            float g[8], u[8], hv[8];
            uint32_t w[8];
            dequantize8(__ldg(reinterpret_cast<const uint2*>(p.gu_q + r * W) + v),
                        __ldg(p.gu_sf + r * (W / 32) + v / 4), g);
            dequantize8(__ldg(reinterpret_cast<const uint2*>(p.gu_q + r * W + p.I) + v),
                        __ldg(p.gu_sf + r * (W / 32) + p.I / 32 + v / 4), u);
#pragma unroll
            for (int i = 0; i < 8; ++i) hv[i] = silu_f(g[i]) * u[i];
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(g[i]);
            __stcs(reinterpret_cast<uint4*>(gu + 8 * v), make_uint4(w[0], w[1], w[2], w[3]));
            __stcs(reinterpret_cast<uint4*>(gu + 8 * v) + 1, make_uint4(w[4], w[5], w[6], w[7]));
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(u[i]);
            __stcs(reinterpret_cast<uint4*>(gu + p.I + 8 * v), make_uint4(w[0], w[1], w[2], w[3]));
            __stcs(reinterpret_cast<uint4*>(gu + p.I + 8 * v) + 1, make_uint4(w[4], w[5], w[6], w[7]));
            __stcs(reinterpret_cast<uint4*>(h) + v, pack8(hv));
        }
    } else if (j < P + R) {
        const int64_t i = j - P;
        load_row_bf16(p.y_q + i * p.H, p.y_sf + i * (p.H / 32), p.H, p.partials_out + i * p.H);
    } else {
        const int64_t t = j - P - R;
        load_row_bf16(p.x_q + t * p.H, p.x_sf + t * (p.H / 32), p.H, p.x_out + t * p.H);
    }
}

dim3 ck_grid(int64_t jobs) { return dim3((unsigned)((jobs + kCkThreads / 32 - 1) / (kCkThreads / 32))); }

}  // namespace

cudaError_t launch_checkpoint_save(const CheckpointParams& p, cudaStream_t s) {
    return launch_after(checkpoint_save_kernel, ck_grid((int64_t)p.T * (2 * p.k + 1)), dim3(kCkThreads), 0, s, p);
}

cudaError_t launch_checkpoint_load(const CheckpointParams& p, cudaStream_t s) {
    return launch_after(checkpoint_load_kernel, ck_grid(padded_rows_max(p.T, p.E, p.k) + (int64_t)p.T * (p.k + 1)),
                        dim3(kCkThreads), 0, s, p);
}

}  // namespace mok
