// Joins the parts of attention items that were split along the keys.
//
// Part p of a row holds o_p (its own softmax over its keys) and s_p = log2 of
// its sum of exponentials. With M = max_p s_p and w_p = 2^{s_p - M}:
//     o = sum_p w_p o_p / sum_p w_p,   lse = ln 2 (M + log2 sum_p w_p).
// CTA (b, y) looks at the boundary between the ranges of CTAs b and b + 1 of the
// kernel before. If it cuts an item, the CTAs of all boundaries inside that
// item share its rows, four rows per warp at a time, the parts in order (so the
// result does not depend on timing). Bound by latency: a cut, then the parts'
// rows, each a read from L2; four rows of a part are in flight together. 6 us after
// 256 decode rows x 8 heads, 9 us for 16 items of ten parts, 14 us for pairs of row
// tiles; eight parts in flight, or half the rows per warp, changed nothing.
#include "kda_attn.cuh"

namespace kda {
namespace {

constexpr int kCombineWarps = 8;
constexpr int kBatch = 4;  // rows of a warp at a time

template <typename T, int D>
__global__ void __launch_bounds__(kCombineWarps * 32)
    kda_attn_combine_kernel(const AttnSplit sp, const int Hkv, const int G, const int tile_rows,
                            T* o, float* lse, int* d_status) {
    pdl_wait();
    const int b = blockIdx.x + 1;
    const AttnCut cut = attn_cuts(sp, D)[b];
    if (cut.ntok == 0 || cut.tile == 0) return;  // no work, or the boundary is an item's too
    // CTAs with a part: the ranges of the item's first and last tile.
    const int c0 = (int)(cut.u0 / cut.each);
    const int c1 = (int)((cut.u0 + (long long)(cut.n - 1) * cut.cost) / cut.each);
    // The first part may be its range's first too.
    const AttnCut start = attn_cuts(sp, D)[c0];
    const int late = !(start.u0 == cut.u0 && start.tile == 0);
    const int lane = threadIdx.x & 31, rows = cut.ntok * G, per = tile_rows / G;
    const int first = ((b - 1 - c0) * gridDim.y + blockIdx.y) * kCombineWarps + (threadIdx.x >> 5);
    const int step = (c1 - c0) * gridDim.y * kCombineWarps;
    const size_t slot = attn_slot_floats(sp.rows, D);
    constexpr int V = D / 32;
    int flags = 0;
    for (int i0 = first * kBatch; i0 < rows; i0 += step * kBatch) {
        // Rows of a pair of tiles: the first holds tile_rows / G tokens.
        int row[kBatch];
        float m[kBatch], sum[kBatch], acc[kBatch][V];
#pragma unroll
        for (int k = 0; k < kBatch; k++) {
            const int i = min(i0 + k, rows - 1), tok = i / G;
            row[k] = tok / per * tile_rows + tok % per * G + i % G;
            m[k] = -INFINITY;
            sum[k] = 0.f;
#pragma unroll
            for (int e = 0; e < V; e++) acc[k][e] = 0.f;
        }
#pragma unroll 2
        for (int c = c0; c <= c1; c++) {
            const float* p = sp.ws + slot * (2 * (size_t)c + (c == c0 ? late : 0));
            float x[kBatch], y[kBatch][V];
#pragma unroll
            for (int k = 0; k < kBatch; k++) {
                x[k] = p[(size_t)sp.rows * D + row[k]];
#pragma unroll
                for (int e = 0; e < V; e++) y[k][e] = p[(size_t)row[k] * D + lane + 32 * e];
            }
#pragma unroll
            for (int k = 0; k < kBatch; k++) {
                if (x[k] == -INFINITY) continue;  // a part in which this row sees nothing
                const float mn = x[k] > m[k] ? x[k] : m[k];  // NaN stays in x and the sums
                const float a = m[k] == -INFINITY ? 0.f : exp2f(m[k] - mn), w = exp2f(x[k] - mn);
                m[k] = mn;
                sum[k] = sum[k] * a + w;
#pragma unroll
                for (int e = 0; e < V; e++) acc[k][e] = acc[k][e] * a + w * y[k][e];
            }
        }
#pragma unroll
        for (int k = 0; k < kBatch; k++) {
            if (i0 + k >= rows) break;
            const size_t at = ((size_t)cut.tok0 + (i0 + k) / G) * Hkv * G + (size_t)cut.h * G + (i0 + k) % G;
            const float inv = sum[k] == 0.f ? 0.f : 1.f / sum[k];
#pragma unroll
            for (int e = 0; e < V; e++) {
                const float y = acc[k][e] * inv;
                flags |= finite_flag(y);
                o[at * D + lane + 32 * e] = from_f32<T>(y);
            }
            if (lse && lane == 0)
                lse[at] = sum[k] == 0.f ? -INFINITY : (m[k] + log2f(sum[k])) * 0.69314718056f;
        }
    }
    report_flags(d_status, flags);
}

// The same for wide rows (D = 512), M and the weights first, so that no part's load waits for
// another's. Every part of which a row sees keys counts, with a weight that underflowed to 0 too, and
// with one of 0 where its scores are all -Inf: what is not finite in it stays, as 0 x NaN. A row
// without weight in any part is zeros. The parts of an item, where the workspace has them.
template <int D>
struct Parts {
    const AttnSplit& sp;
    int c0, c1, late, row_tile, G;
    __device__ __forceinline__ const float* at(int c) const {
        return sp.ws + attn_slot_floats(sp.rows, D) * (2 * (size_t)c + (c == c0 ? late : 0));
    }
    __device__ __forceinline__ int row(int r) const {  // of the tile, of the item's row r
        const int tok = r / G, per = row_tile / G;
        return tok / per * row_tile + tok % per * G + r % G;
    }
    __device__ __forceinline__ float sum_of(int c, int row) const { return at(c)[(size_t)sp.rows * D + row]; }
    // The largest of all parts' sums, by a warp.
    __device__ __forceinline__ float largest(int row) const {
        float m = -INFINITY;
        for (int c = c0 + (threadIdx.x & 31); c <= c1; c += 32) m = fmaxf(m, sum_of(c, row));
#pragma unroll
        for (int k = 16; k > 0; k >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, k));
        return m;
    }
    // A part's weight; below 0 for one of which the row sees no key. NaN stays.
    __device__ __forceinline__ float weight(int c, int row, float m) const {
        const float x = sum_of(c, row);
        return x == -INFINITY ? -1.f : x == kAttnNoWeight ? 0.f : exp2f(x - m);
    }
};
__device__ __forceinline__ void add(float4& acc, float w, const float* y) {
    const float4 v = *reinterpret_cast<const float4*>(y);
    acc.x = fmaf(w, v.x, acc.x);
    acc.y = fmaf(w, v.y, acc.y);
    acc.z = fmaf(w, v.z, acc.z);
    acc.w = fmaf(w, v.w, acc.w);
}
template <typename T>
__device__ __forceinline__ int put(T* dst, float4 acc, float inv) {
    float y[4] = {acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv};
    T out[4];
    int flags = 0;
#pragma unroll
    for (int e = 0; e < 4; e++) {
        if (inv == 0.f) y[e] = 0.f;  // a row of no weight
        flags |= finite_flag(y[e]);
        out[e] = from_f32<T>(y[e]);
    }
    if constexpr (sizeof(T) == 4) *reinterpret_cast<float4*>(dst) = *reinterpret_cast<float4*>(out);
    else *reinterpret_cast<uint2*>(dst) = *reinterpret_cast<uint2*>(out);
    return flags;
}

// Few parts: a warp takes a row. Many (more than kFewParts): a CTA takes 128 channels of a row, its
// warps every eighth part each, added up in their order. Bound by the latency of a row's loads, first
// the sums, then the parts. Measured with the attention before it, when chosen: 76 parts (2 x 4 drafts over
// 262 k tokens) 182 us, with a warp a row 187 and through the kernel above 206; 1 request of 65536 keys x 64
// heads 33 against 57; 5 parts (3 requests to 700 keys) 18.5 us, shared by a CTA's warps 25. Now 171, 33 and 15.3.
constexpr int kFewParts = 16;

template <typename T, int D>
__global__ void __launch_bounds__(kCombineWarps * 32, 4)
    kda_attn_combine_wide_kernel(const AttnSplit sp, const int Hkv, const int G, const int tile_rows,
                                 T* o, float* lse, int* d_status) {
    __shared__ float4 s_acc[kCombineWarps][32];
    __shared__ float s_sum[kCombineWarps];
    pdl_wait();
    const int b = blockIdx.x + 1;
    const AttnCut cut = attn_cuts(sp, D)[b];
    if (cut.ntok == 0 || cut.tile == 0) return;  // no work, or the boundary is an item's too
    const int c0 = (int)(cut.u0 / cut.each);
    const int c1 = (int)((cut.u0 + (long long)(cut.n - 1) * cut.cost) / cut.each);
    const AttnCut start = attn_cuts(sp, D)[c0];
    const Parts<D> parts{sp, c0, c1, !(start.u0 == cut.u0 && start.tile == 0), tile_rows, G};
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, rows = cut.ntok * G;
    const int cta = (b - 1 - c0) * gridDim.y + blockIdx.y, ctas = (c1 - c0) * gridDim.y;
    constexpr int Q = D / 128;
    auto out_row = [&](int r) {
        return ((size_t)cut.tok0 + r / G) * Hkv * G + (size_t)cut.h * G + r % G;
    };
    int flags = 0;
    if (c1 - c0 < kFewParts) {
        for (int r = cta * kCombineWarps + warp; r < rows; r += ctas * kCombineWarps) {
            const int row = parts.row(r);
            const float m = parts.largest(row);
            const float w = lane <= c1 - c0 ? parts.weight(c0 + lane, row, m) : 0.f;
            float4 acc[Q];
#pragma unroll
            for (int q = 0; q < Q; q++) acc[q] = make_float4(0.f, 0.f, 0.f, 0.f);
            float sum = 0.f;
#pragma unroll 2
            for (int k = 0; k <= c1 - c0; k++) {
                const float wk = __shfl_sync(0xffffffffu, w, k);
                if (wk < 0.f) continue;
                sum += wk;
#pragma unroll
                for (int q = 0; q < Q; q++) add(acc[q], wk, parts.at(c0 + k) + (size_t)row * D + 128 * q + lane * 4);
            }
            const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
            for (int q = 0; q < Q; q++) flags |= put(o + out_row(r) * D + 128 * q + lane * 4, acc[q], inv);
            if (lse && lane == 0) lse[out_row(r)] = sum == 0.f ? -INFINITY : (m + log2f(sum)) * 0.69314718056f;
        }
    } else {
        for (int i = cta; i < rows * Q; i += ctas) {
            const int r = i / Q, row = parts.row(r), col = i % Q * 128 + lane * 4;
            const float m = parts.largest(row);
            float sum = 0.f;
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int cb = c0 + warp; cb <= c1; cb += 32 * kCombineWarps) {
                const int n = min((c1 - cb) / kCombineWarps + 1, 32);  // parts cb, cb + 8, ...
                const float w = lane < n ? parts.weight(cb + kCombineWarps * lane, row, m) : 0.f;
#pragma unroll 4  // (8: registers spill)
                for (int k = 0; k < n; k++) {
                    const float wk = __shfl_sync(0xffffffffu, w, k);
                    if (wk < 0.f) continue;
                    sum += wk;
                    add(acc, wk, parts.at(cb + kCombineWarps * k) + (size_t)row * D + col);
                }
            }
            __syncthreads();  // what was there is read
            s_acc[warp][lane] = acc;
            if (lane == 0) s_sum[warp] = sum;
            __syncthreads();
            if (warp == 0) {
                for (int k = 1; k < kCombineWarps; k++) {
                    const float4 y = s_acc[k][lane];
                    acc.x += y.x;
                    acc.y += y.y;
                    acc.z += y.z;
                    acc.w += y.w;
                    sum += s_sum[k];
                }
                flags |= put(o + out_row(r) * D + col, acc, sum == 0.f ? 0.f : 1.f / sum);
                if (lse && lane == 0 && i % Q == 0)
                    lse[out_row(r)] = sum == 0.f ? -INFINITY : (m + log2f(sum)) * 0.69314718056f;
            }
        }
    }
    report_flags(d_status, flags);
}

}  // namespace

cudaError_t launch_attn_combine(const AttnSplit& sp, int Hkv, int G, int d, int rows_per_tile,
                                void* o, float* lse, kda_dtype_t io, int* d_status,
                                cudaStream_t stream) {
    if (sp.ctas < 2) return cudaSuccess;
    // Two passes of the CTAs of one boundary over the rows of a slot.
    const int per = 2 * kCombineWarps * kBatch;
    const dim3 grid((unsigned)(sp.ctas - 1), (unsigned)((sp.rows + per - 1) / per));
    auto go = [&](auto kernel, auto* out) {
        return launch_dependent(kernel, grid, dim3(kCombineWarps * 32), 0, stream, sp, Hkv, G,
                                rows_per_tile, out, lse, d_status);
    };
    if (d == 512) {
        // A warp for each row, as one boundary may have to do all of an item.
        const dim3 wide((unsigned)(sp.ctas - 1), (unsigned)((sp.rows + kCombineWarps - 1) / kCombineWarps));
        auto go = [&](auto kernel, auto* out) {
            return launch_dependent(kernel, wide, dim3(kCombineWarps * 32), 0, stream, sp, Hkv, G,
                                    rows_per_tile, out, lse, d_status);
        };
        return io == KDA_BF16 ? go(kda_attn_combine_wide_kernel<__nv_bfloat16, 512>, static_cast<__nv_bfloat16*>(o))
                              : go(kda_attn_combine_wide_kernel<float, 512>, static_cast<float*>(o));
    }
    if (io == KDA_BF16) {
        auto* out = static_cast<__nv_bfloat16*>(o);
        return d == 128 ? go(kda_attn_combine_kernel<__nv_bfloat16, 128>, out)
                        : go(kda_attn_combine_kernel<__nv_bfloat16, 64>, out);
    }
    auto* out = static_cast<float*>(o);
    return d == 128 ? go(kda_attn_combine_kernel<float, 128>, out)
                    : go(kda_attn_combine_kernel<float, 64>, out);
}

}  // namespace kda
