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

// The same for wide rows (D = 512): a warp finds M and the weights of a row first, a part per
// lane, so that no part's load waits for another's. It takes all channels of a row that
// has few parts, 128 of one that has many; 8 loads are in flight either way.
// Q: quarters of a row that a warp takes.
template <typename T, int D, int Q>
__device__ __forceinline__ int join_rows(const AttnSplit& sp, const AttnCut& cut, int c0, int c1, int late, int first,
                                         int step, int Hkv, int G, int tile_rows, T* o, float* lse) {
    constexpr int COLS = D / 128 / Q;  // warps of a row
    const int lane = threadIdx.x & 31, units = cut.ntok * G * COLS, per = tile_rows / G;
    const size_t slot = attn_slot_floats(sp.rows, D);
    auto part = [&](int c) { return sp.ws + slot * (2 * (size_t)c + (c == c0 ? late : 0)); };
    int flags = 0;
    for (int i = first; i < units; i += step) {
        const int r = i / COLS, col = i % COLS * 128 + lane * 4, tok = r / G;
        const int row = tok / per * tile_rows + tok % per * G + r % G;
        float m = -INFINITY;
        for (int c = c0 + lane; c <= c1; c += 32) m = fmaxf(m, part(c)[(size_t)sp.rows * D + row]);
#pragma unroll
        for (int k = 16; k > 0; k >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, k));
        float sum = 0.f;
        float4 acc[Q];
#pragma unroll
        for (int q = 0; q < Q; q++) acc[q] = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int cb = c0; cb <= c1; cb += 32) {
            const int n = min(c1 - cb + 1, 32);
            // (a part in which this row sees nothing has weight 0 and is not read; NaN stays)
            float w = 0.f;
            if (lane < n) {
                const float x = part(cb + lane)[(size_t)sp.rows * D + row];
                w = x == -INFINITY ? 0.f : exp2f(x - m);
            }
            sum += w;
#pragma unroll 8 / Q
            for (int k = 0; k < n; k++) {
                const float wk = __shfl_sync(0xffffffffu, w, k);
                if (wk == 0.f) continue;
                const float* y = part(cb + k) + (size_t)row * D + col;
#pragma unroll
                for (int q = 0; q < Q; q++) {
                    const float4 v = *reinterpret_cast<const float4*>(y + 128 * q);
                    acc[q].x = fmaf(wk, v.x, acc[q].x);
                    acc[q].y = fmaf(wk, v.y, acc[q].y);
                    acc[q].z = fmaf(wk, v.z, acc[q].z);
                    acc[q].w = fmaf(wk, v.w, acc[q].w);
                }
            }
        }
#pragma unroll
        for (int k = 16; k > 0; k >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, k);
        const size_t at = ((size_t)cut.tok0 + tok) * Hkv * G + (size_t)cut.h * G + r % G;
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
        for (int q = 0; q < Q; q++) {
            const float y[4] = {acc[q].x * inv, acc[q].y * inv, acc[q].z * inv, acc[q].w * inv};
            T out[4];
#pragma unroll
            for (int e = 0; e < 4; e++) {
                flags |= finite_flag(y[e]);
                out[e] = from_f32<T>(y[e]);
            }
            T* dst = o + at * D + col + 128 * q;
            if constexpr (sizeof(T) == 4) *reinterpret_cast<float4*>(dst) = *reinterpret_cast<float4*>(out);
            else *reinterpret_cast<uint2*>(dst) = *reinterpret_cast<uint2*>(out);
        }
        if (lse && lane == 0 && i % COLS == 0)
            lse[at] = sum == 0.f ? -INFINITY : (m + log2f(sum)) * 0.69314718056f;
    }
    return flags;
}

template <typename T, int D>
__global__ void __launch_bounds__(kCombineWarps * 32, 4)
    kda_attn_combine_wide_kernel(const AttnSplit sp, const int Hkv, const int G, const int tile_rows,
                                 T* o, float* lse, int* d_status) {
    pdl_wait();
    const int b = blockIdx.x + 1;
    const AttnCut cut = attn_cuts(sp, D)[b];
    if (cut.ntok == 0 || cut.tile == 0) return;  // no work, or the boundary is an item's too
    const int c0 = (int)(cut.u0 / cut.each);
    const int c1 = (int)((cut.u0 + (long long)(cut.n - 1) * cut.cost) / cut.each);
    const AttnCut start = attn_cuts(sp, D)[c0];
    const int late = !(start.u0 == cut.u0 && start.tile == 0);
    const int first = ((b - 1 - c0) * gridDim.y + blockIdx.y) * kCombineWarps + (threadIdx.x >> 5);
    const int step = (c1 - c0) * gridDim.y * kCombineWarps;
    const int flags = c1 - c0 < 4
                          ? join_rows<T, D, D / 128>(sp, cut, c0, c1, late, first, step, Hkv, G, tile_rows, o, lse)
                          : join_rows<T, D, 1>(sp, cut, c0, c1, late, first, step, Hkv, G, tile_rows, o, lse);
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
