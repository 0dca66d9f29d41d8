// Joins the parts of attention items that were split along the keys.
//
// Part p of a row holds o_p (its own softmax over its keys) and s_p = log2 of
// its sum of exponentials. With M = max_p s_p and w_p = 2^{s_p - M}:
//     o = sum_p w_p o_p / sum_p w_p,   lse = ln 2 (M + log2 sum_p w_p).
// CTA b looks at the boundary between the ranges of CTAs b and b + 1 of the kernel
// before. If it cuts an item, the CTAs of all boundaries inside that item
// share its rows, one row per warp at a time, the parts in order (so the result
// does not depend on timing). Bound by latency: a part's row is d floats from L2.
#include "kda_attn.cuh"

namespace kda {
namespace {

constexpr int kCombineThreads = 256;

template <typename T, int D>
__global__ void __launch_bounds__(kCombineThreads)
    kda_attn_combine_kernel(const AttnShape s, const AttnSplit sp, const int tile_rows, T* o,
                            float* lse, int* d_status) {
    __shared__ long long s_sum[kCombineThreads / 32];
    pdl_wait();
    const long long each = attn_units_each<kCombineThreads>(s, sp.ctas, sp.least, s_sum);
    const int b = blockIdx.x + 1;
    AttnWalk walk;
    AttnReq q;
    int r, h, t, tile;
    long long in;
    if (!attn_find<true>(s, walk, b * each, &r, &q, &in)) return;
    attn_unit_item(s, q, in, &h, &t, &tile);
    if (tile == 0) return;  // the boundary is an item's too
    const long long u0 = b * each - tile, u1 = u0 + attn_item_units(s, q, t);
    const int c0 = (int)(u0 / each), c1 = (int)((u1 - 1) / each);  // CTAs with a part
    const int tok0 = t * q.tok, ntok = min(q.tok, q.q_len - tok0);
    const int lane = threadIdx.x & 31;
    const int warps = (c1 - c0) * (kCombineThreads / 32);  // of all CTAs of this item
    const size_t slot = attn_slot_floats(sp.rows, D);
    constexpr int V = D / 32;
    int flags = 0;
    for (int i = (b - 1 - c0) * (kCombineThreads / 32) + (threadIdx.x >> 5); i < ntok * s.G; i += warps) {
        // Rows of a pair of tiles: the first holds tile_rows / G tokens.
        const int per = tile_rows / s.G, tok = i / s.G, g = i % s.G;
        const int row = tok / per * tile_rows + tok % per * s.G + g;
        float m = -INFINITY, sum = 0.f, acc[V] = {};
        for (int c = c0; c <= c1; c++) {
            const float* p = sp.ws + slot * (2 * (size_t)c + (u0 > c * each ? 1 : 0));
            const float x = p[(size_t)sp.rows * D + row];
            float y[V];
#pragma unroll
            for (int e = 0; e < V; e++) y[e] = p[(size_t)row * D + lane + 32 * e];
            if (x == -INFINITY) continue;  // a part in which this row sees nothing
            const float mn = x > m ? x : m;  // NaN stays in x and the sums
            const float a = m == -INFINITY ? 0.f : exp2f(m - mn), w = exp2f(x - mn);
            m = mn;
            sum = sum * a + w;
#pragma unroll
            for (int e = 0; e < V; e++) acc[e] = acc[e] * a + w * y[e];
        }
        const size_t at = ((size_t)q.q0 + tok0 + tok) * s.Hkv * s.G + (size_t)h * s.G + g;
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
        for (int e = 0; e < V; e++) {
            const float y = acc[e] * inv;
            flags |= finite_flag(y);
            o[at * D + lane + 32 * e] = from_f32<T>(y);
        }
        if (lse && lane == 0)
            lse[at] = sum == 0.f ? -INFINITY : (m + log2f(sum)) * 0.69314718056f;
    }
    report_flags(d_status, flags);
}

}  // namespace

cudaError_t launch_attn_combine(const AttnShape& s, const AttnSplit& sp, int d, int rows_per_tile,
                                void* o, float* lse, kda_dtype_t io, int* d_status,
                                cudaStream_t stream) {
    if (sp.ctas < 2) return cudaSuccess;
    const dim3 grid((unsigned)(sp.ctas - 1)), block(kCombineThreads);
    auto go = [&](auto kernel, auto* out) {
        return launch_dependent(kernel, grid, block, 0, stream, s, sp, rows_per_tile, out, lse,
                                d_status);
    };
    if (io == KDA_BF16) {
        auto* out = static_cast<__nv_bfloat16*>(o);
        return d == 128 ? go(kda_attn_combine_kernel<__nv_bfloat16, 128>, out)
                        : go(kda_attn_combine_kernel<__nv_bfloat16, 64>, out);
    }
    auto* out = static_cast<float*>(o);
    return d == 128 ? go(kda_attn_combine_kernel<float, 128>, out)
                    : go(kda_attn_combine_kernel<float, 64>, out);
}

int attn_sms() {
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
        cudaGetLastError();
        return 0;
    }
    return n;
}

}  // namespace kda
