// sort.cu - tokens sorted by experts that the caller chose, and back.
//
// With e[i] the expert of entry i = t*k + j (token t, slot j; any value outside
// 0..E-1 drops the entry) and r = slot_row[i] the entry's place in the order
// (expert, i):
//   sort            xs[r] = x[t]
//   unsort          out[t] = sum_j w[t,j] * y[slot_row[t*k+j]]      (w = 1: sort's gradient)
//   its gradient    dy[r] = w[t,j] * dout[t],   dw[t,j] = <dout[t], y[r]>
// Sums run in fp32, j ascending; dropped entries add nothing and have dw = 0.
//
// The row moves are bound by memory, and a row is touched once by each: T = 4096,
// H = 7168, k = 8, BF16, sort 79 us (6.7 TB/s), unsort 81 (6.5), its gradient 146 (6.8).
// Small calls are bound by their launches: T = 7, k = 8, layout, sort and unsort 5.6 us
// together in a graph.
#include <algorithm>

#include <cuda_fp16.h>

#include "common.cuh"
#include "moves.cuh"

namespace mok {

namespace {

constexpr int kSortThreads = 256;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortMaxBlocks = 128;

// Entries of a block: whole rounds of kSortThreads, at most kSortMaxBlocks blocks.
int64_t sort_block_entries(int64_t n) {
    const int64_t rounds = (n + (int64_t)kSortThreads * kSortMaxBlocks - 1) / ((int64_t)kSortThreads * kSortMaxBlocks);
    return std::max<int64_t>(rounds, 1) * kSortThreads;
}
int sort_blocks(int64_t n) { return (int)((n + sort_block_entries(n) - 1) / sort_block_entries(n)); }
// Up to this many entries one block counts and places them in one launch (4096 tokens' 32768
// entries: count 4.6 us, place 7.8, each by itself).
constexpr int kSortOneBlock = 2048;

// hist[e * blocks + b] = entries of expert e among block b's (whole numbers, so
// the order of the atomics does not matter).
__global__ void __launch_bounds__(kSortThreads)
sort_count_kernel(const int32_t* __restrict__ idx, int64_t n, int64_t per, int E, int32_t* __restrict__ hist) {
    extern __shared__ int32_t cnt[];
    pdl_wait();
    pdl_allow_next();
    for (int e = threadIdx.x; e < E; e += kSortThreads) cnt[e] = 0;
    __syncthreads();
    const int64_t i0 = blockIdx.x * per, i1 = min(i0 + per, n);
    for (int64_t i = i0 + threadIdx.x; i < i1; i += kSortThreads) {
        const int e = idx[i];
        if ((unsigned)e < (unsigned)E) atomicAdd(&cnt[e], 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += kSortThreads) hist[(int64_t)e * gridDim.x + blockIdx.x] = cnt[e];
}

// Places block b's entries. `hist` == NULL: a single block, which counts itself.
// The entries of a round (one a thread) are ranked by their lane among the same
// expert's in their warp, then by their warp: no atomic decides an order.
__global__ void __launch_bounds__(kSortThreads)
sort_place_kernel(const int32_t* __restrict__ idx, int64_t n, int64_t per, int E, const int32_t* __restrict__ hist,
                  int32_t* __restrict__ counts, int32_t* __restrict__ offsets, int32_t* __restrict__ row_src,
                  int32_t* __restrict__ slot_row) {
    extern __shared__ int32_t sh[];
    int32_t* next = sh;            // [E]: place of the expert's next entry of this block
    int32_t* tot = sh + E;         // [E]
    int32_t* wcnt = tot + E;       // [kSortWarps][E]
    __shared__ int32_t scan[kSortWarps + 1];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, b = blockIdx.x, nb = gridDim.x;
    const int64_t i0 = b * per, i1 = min(i0 + per, n);
    pdl_wait();
    pdl_allow_next();
    for (int i = tid; i < (2 + kSortWarps) * E; i += kSortThreads) sh[i] = 0;
    __syncthreads();
    if (hist == nullptr) {
        for (int64_t i = tid; i < n; i += kSortThreads) {
            const int e = idx[i];
            if ((unsigned)e < (unsigned)E) atomicAdd(&tot[e], 1);
        }
    } else {
        for (int e = warp; e < E; e += kSortWarps) {
            int before = 0, all = 0;
            for (int j = lane; j < nb; j += 32) {
                const int v = hist[(int64_t)e * nb + j];
                all += v;
                before += j < b ? v : 0;
            }
#pragma unroll
            for (int d = 16; d >= 1; d >>= 1) {
                all += __shfl_xor_sync(0xffffffffu, all, d);
                before += __shfl_xor_sync(0xffffffffu, before, d);
            }
            if (lane == 0) {
                tot[e] = all;
                next[e] = before;
            }
        }
    }
    __syncthreads();
    // exclusive sums over the experts, kSortThreads at a time
    int base = 0;
    for (int e0 = 0; e0 < E; e0 += kSortThreads) {
        const int e = e0 + tid, v = e < E ? tot[e] : 0;
        int s = v;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int o = __shfl_up_sync(0xffffffffu, s, d);
            if (lane >= d) s += o;
        }
        if (lane == 31) scan[warp + 1] = s;
        __syncthreads();
        if (tid == 0) {
            scan[0] = 0;
            for (int w = 1; w <= kSortWarps; ++w) scan[w] += scan[w - 1];
        }
        __syncthreads();
        const int off = base + scan[warp] + s - v;
        if (e < E) {
            next[e] += off;
            if (b == 0) {
                counts[e] = v;
                offsets[e] = off;
            }
        }
        base += scan[kSortWarps];
        __syncthreads();
    }
    if (b == 0 && tid == 0) offsets[E] = base;

    for (int64_t r0 = i0; r0 < i1; r0 += kSortThreads) {
        const int64_t i = r0 + tid;
        int e = i < i1 ? idx[i] : -1;
        if ((unsigned)e >= (unsigned)E) e = -1;
        const unsigned same = __match_any_sync(0xffffffffu, e);
        const int rank = __popc(same & ((1u << lane) - 1));
        if (e >= 0 && rank == 0) wcnt[warp * E + e] = __popc(same);
        __syncthreads();
        if (i < i1) {
            int32_t row = -1;
            if (e >= 0) {
                row = next[e] + rank;
                for (int w = 0; w < warp; ++w) row += wcnt[w * E + e];
                row_src[row] = (int32_t)i;
            }
            slot_row[i] = row;
            if (i >= base) row_src[i] = -1;   // behind the last sorted row
        }
        __syncthreads();
        if (e >= 0 && rank == 0) {
            atomicAdd(&next[e], __popc(same));
            wcnt[warp * E + e] = 0;
        }
        __syncthreads();
    }
}

// ------------------------------------------------------------------ elements

template <int ELEM>
struct Elem;   // 16 bytes of a type as fp32 values and back
template <>
struct Elem<MOK_ELEM_BF16> {
    static constexpr int kN = 8;
    static __device__ __forceinline__ void unpack(const uint4& v, float (&f)[8]) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = bf16_lo(w[i]);
            f[2 * i + 1] = bf16_hi(w[i]);
        }
    }
    static __device__ __forceinline__ uint4 pack(const float (&f)[8]) {
        return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                          pack_bf16x2(f[6], f[7]));
    }
};
template <>
struct Elem<MOK_ELEM_F16> {
    static constexpr int kN = 8;
    static __device__ __forceinline__ void unpack(const uint4& v, float (&f)[8]) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 t = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
            f[2 * i] = t.x;
            f[2 * i + 1] = t.y;
        }
    }
    static __device__ __forceinline__ uint4 pack(const float (&f)[8]) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __half2 h = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};
template <>
struct Elem<MOK_ELEM_F32> {
    static constexpr int kN = 4;
    static __device__ __forceinline__ void unpack(const uint4& v, float (&f)[4]) {
        f[0] = __uint_as_float(v.x);
        f[1] = __uint_as_float(v.y);
        f[2] = __uint_as_float(v.z);
        f[3] = __uint_as_float(v.w);
    }
    static __device__ __forceinline__ uint4 pack(const float (&f)[4]) {
        return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
    }
};

// Rows move as 16-byte vectors whatever their type: nv of them a row. A thread
// holds one vector of the token and writes it to the token's places, so x is read once
// whatever k.
__global__ void __launch_bounds__(256)
sort_rows_kernel(const uint4* __restrict__ x, int64_t ldx, const int32_t* __restrict__ slot_row, int k, int nv,
                 uint4* __restrict__ out) {
    pdl_wait();
    pdl_allow_next();
    const int64_t t = blockIdx.x;
    const int32_t* rows = slot_row + t * k;
    for (int v = blockIdx.y * blockDim.x + threadIdx.x; v < nv; v += gridDim.y * blockDim.x) {
        const uint4 a = __ldg(x + t * ldx + v);
        for (int j = 0; j < k; ++j) {
            const int r = __ldg(rows + j);
            if (r >= 0) out[(int64_t)r * nv + v] = a;
        }
    }
}

// Entries of a token at a time, their loads in flight together. T = 4096, H = 7168, k = 8:
// four in the sum (82 us, 96% of the copy rate; eight take registers that other CTAs' loads
// need, 97), eight in its gradient, which holds the token's gradient meanwhile (146 us).
constexpr int kSumEntries = 4, kBwdEntries = 8;

// Rows (or -1) of N entries of a token from j0 on.
template <int N>
__device__ __forceinline__ void entry_rows(const int32_t* rows, int k, int j0, int (&r)[N]) {
#pragma unroll
    for (int j = 0; j < N; ++j) r[j] = j0 + j < k ? __ldg(rows + j0 + j) : -1;
}

template <int ELEM>
__global__ void __launch_bounds__(256)
unsort_rows_kernel(const uint4* __restrict__ y, const int32_t* __restrict__ slot_row, const float* __restrict__ w,
                   int k, int nv, uint4* __restrict__ out) {
    using L = Elem<ELEM>;
    pdl_wait();
    pdl_allow_next();
    const int64_t t = blockIdx.x;
    const int32_t* rows = slot_row + t * k;
    for (int v = blockIdx.y * blockDim.x + threadIdx.x; v < nv; v += gridDim.y * blockDim.x) {
        float acc[L::kN];
#pragma unroll
        for (int i = 0; i < L::kN; ++i) acc[i] = 0.f;
        for (int j0 = 0; j0 < k; j0 += kSumEntries) {
            int r[kSumEntries];
            float c[kSumEntries];
            uint4 a[kSumEntries];
            entry_rows(rows, k, j0, r);
#pragma unroll
            for (int j = 0; j < kSumEntries; ++j)
                if (r[j] >= 0) {
                    a[j] = __ldg(y + (int64_t)r[j] * nv + v);
                    c[j] = w ? __ldg(w + t * k + j0 + j) : 1.0f;
                }
#pragma unroll
            for (int j = 0; j < kSumEntries; ++j) {
                if (r[j] < 0) continue;
                float f[L::kN];
                L::unpack(a[j], f);
#pragma unroll
                for (int i = 0; i < L::kN; ++i) acc[i] = fmaf(c[j], f[i], acc[i]);
            }
        }
        out[t * nv + v] = L::pack(acc);
    }
}

// A CTA per token: its gradient is read once for up to kBwdEntries entries.
template <int ELEM>
__global__ void __launch_bounds__(256)
unsort_rows_backward_kernel(const uint4* __restrict__ dout, const uint4* __restrict__ y,
                            const int32_t* __restrict__ slot_row, const float* __restrict__ w, int k, int nv,
                            uint4* __restrict__ dy, float* __restrict__ dw) {
    using L = Elem<ELEM>;
    __shared__ float red[8][kBwdEntries];
    pdl_wait();
    pdl_allow_next();
    const int64_t t = blockIdx.x;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int j0 = 0; j0 < k; j0 += kBwdEntries) {
        int r[kBwdEntries];
        float c[kBwdEntries], dot[kBwdEntries];
        entry_rows(slot_row + t * k, k, j0, r);
#pragma unroll
        for (int j = 0; j < kBwdEntries; ++j) {
            c[j] = j0 + j < k ? __ldg(w + t * k + j0 + j) : 0.f;
            dot[j] = 0.f;
        }
        for (int v = threadIdx.x; v < nv; v += blockDim.x) {
            const uint4 dv = __ldg(dout + t * nv + v);
            uint4 a[kBwdEntries];
#pragma unroll
            for (int j = 0; j < kBwdEntries; ++j)
                if (r[j] >= 0) a[j] = __ldg(y + (int64_t)r[j] * nv + v);
            float d[L::kN];
            L::unpack(dv, d);
#pragma unroll
            for (int j = 0; j < kBwdEntries; ++j) {
                if (r[j] < 0) continue;
                float f[L::kN], g[L::kN];
                L::unpack(a[j], f);
#pragma unroll
                for (int i = 0; i < L::kN; ++i) {
                    dot[j] = fmaf(d[i], f[i], dot[j]);
                    g[i] = c[j] * d[i];
                }
                dy[(int64_t)r[j] * nv + v] = L::pack(g);
            }
        }
#pragma unroll
        for (int j = 0; j < kBwdEntries; ++j) {
#pragma unroll
            for (int s = 16; s >= 1; s >>= 1) dot[j] += __shfl_xor_sync(0xffffffffu, dot[j], s);
            if (lane == 0) red[warp][j] = dot[j];
        }
        __syncthreads();
        if (threadIdx.x < kBwdEntries && j0 + threadIdx.x < k) {
            float s = 0.f;
            for (int i = 0; i < (int)blockDim.x / 32; ++i) s += red[i][threadIdx.x];
            dw[t * k + j0 + threadIdx.x] = s;
        }
        __syncthreads();
    }
}

}  // namespace

int elem_bytes(int elem) { return elem == MOK_ELEM_F32 ? 4 : 2; }

size_t sort_workspace_bytes(int64_t n, int E) { return (size_t)sort_blocks(n) * E * 4; }

cudaError_t launch_sort_layout(const int32_t* idx, int64_t n, int E, int32_t* counts, int32_t* offsets,
                               int32_t* row_src, int32_t* slot_row, void* ws, cudaStream_t s) {
    const size_t smem = (size_t)(2 + kSortWarps) * E * 4;
    const bool one = n <= kSortOneBlock;
    const int64_t per = one ? std::max<int64_t>(n, 1) : sort_block_entries(n);
    const int nb = one ? 1 : sort_blocks(n);
    int32_t* hist = one ? nullptr : static_cast<int32_t*>(ws);
    cudaError_t e = cudaSuccess;
    if (!one) e = launch_after(sort_count_kernel, dim3(nb), dim3(kSortThreads), (size_t)E * 4, s, idx, n, per, E, hist);
    if (e == cudaSuccess)
        e = launch_after(sort_place_kernel, dim3(nb), dim3(kSortThreads), smem, s, idx, n, per, E,
                         (const int32_t*)hist, counts, offsets, row_src, slot_row);
    return e;
}

namespace {
// CTAs of a row-moving kernel: a thread a vector, one CTA a token where there are
// many tokens, the row cut over several where there are few.
void row_grid(int T, int nv, dim3& grid, dim3& block) {
    const int threads = std::min(256, ceil_div(nv, 32) * 32);
    const int parts = ceil_div(nv, threads);
    block = dim3(threads);
    grid = dim3(T, std::min(parts, 65535));
}
}  // namespace

cudaError_t launch_sort_rows(int elem, const void* x, int64_t ldx, const int32_t* slot_row, int T, int H, int k,
                             void* out, cudaStream_t s) {
    const int per = 16 / elem_bytes(elem), nv = H / per;
    dim3 grid, block;
    row_grid(T, nv, grid, block);
    return launch_after(sort_rows_kernel, grid, block, 0, s, static_cast<const uint4*>(x), ldx / per, slot_row, k, nv,
                        static_cast<uint4*>(out));
}

cudaError_t launch_unsort_rows(int elem, const void* y, const int32_t* slot_row, const float* w, int T, int H, int k,
                               void* out, cudaStream_t s) {
    const int nv = H / (16 / elem_bytes(elem));
    dim3 grid, block;
    row_grid(T, nv, grid, block);
    auto kern = elem == MOK_ELEM_BF16 ? unsort_rows_kernel<MOK_ELEM_BF16>
              : elem == MOK_ELEM_F16 ? unsort_rows_kernel<MOK_ELEM_F16> : unsort_rows_kernel<MOK_ELEM_F32>;
    return launch_after(kern, grid, block, 0, s, static_cast<const uint4*>(y), slot_row, w, k, nv,
                        static_cast<uint4*>(out));
}

cudaError_t launch_unsort_rows_backward(int elem, const void* dout, const void* y, const int32_t* slot_row,
                                        const float* w, int T, int H, int k, void* dy, float* dw, cudaStream_t s) {
    const int nv = H / (16 / elem_bytes(elem));
    auto kern = elem == MOK_ELEM_BF16 ? unsort_rows_backward_kernel<MOK_ELEM_BF16>
              : elem == MOK_ELEM_F16 ? unsort_rows_backward_kernel<MOK_ELEM_F16>
                                     : unsort_rows_backward_kernel<MOK_ELEM_F32>;
    return launch_after(kern, dim3(T), dim3(std::min(256, ceil_div(nv, 32) * 32)), 0, s,
                        static_cast<const uint4*>(dout), static_cast<const uint4*>(y), slot_row, w, k, nv,
                        static_cast<uint4*>(dy), dw);
}

}  // namespace mok
