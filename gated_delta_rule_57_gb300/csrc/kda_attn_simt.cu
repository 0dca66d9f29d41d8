// Softmax attention of fp32 inputs on the CUDA cores, with every product and sum in 32 bits.
//
//     x_ij = scale log2(e) q_i . k_j (j <= position of i),  m_i = max_j x_ij,
//     l_i = sum_j 2^{x_ij - m_i},  o_i = sum_j 2^{x_ij - m_i} v_j / l_i
//
// in one pass over the keys: when a key tile raises m_i, the sums so far are
// multiplied by 2^{m_old - m_new}. A CTA of 256 threads holds 64 rows and takes
// 64 keys at a time through shared memory; thread (y, x) computes rows
// 4y .. 4y + 3 against keys x + 16 i, and the same rows of the output. Two CTAs
// per SM, so that one's loads and softmax pass beside the other's products; long
// rows are cut into ranges as the header of kda_attn.cuh says. Bound by the FFMA
// pipe and shared memory: 8 loads of 16 bytes feed 64 FFMA in the first product and
// 8 or 12 feed 64 or 128 in the second. Three prompts of up to 1021 tokens (8 / 2
// heads, d = 64): 51.5 us, FFMA pipe 41 % active.
#include <algorithm>

#include "kda_attn.cuh"
#include "kda_host.cuh"

namespace kda {
namespace {

constexpr int kRows = 64, kKeys = 64, kThreadsSimt = 256;

constexpr int kCtasPerSm = 2;

struct SimtParams {
    AttnShape s;
    AttnSplit sp;
    const void* q;
    const void* k;
    const void* v;
    const int* block_table;
    void* o;
    float* lse;
    long long q_stride, k_stride, v_stride;
    int num_pages, page, max_pages;
    float scale;
    int* d_status;
};

template <int D>
constexpr size_t simt_smem() {
    return (size_t)3 * kRows * (D + 4) * 4;
}

__device__ __forceinline__ float4 load4(const float* p) {
    return *reinterpret_cast<const float4*>(p);
}

template <int D>
__global__ void __launch_bounds__(kThreadsSimt, kCtasPerSm) kda_attn_simt_kernel(const SimtParams p) {
    constexpr int LD = D + 4, LP = kKeys + 4, C4 = D / 64;  // C4: float4 columns per thread
    extern __shared__ __align__(16) float sm[];
    float* sq = sm;
    float* sk = sq + kRows * LD;  // also the probabilities, once the scores are done
    float* sv = sk + kKeys * LD;
    float* sp = sk;

    __shared__ long long s_groups[kAttnGroups], s_sum[kThreadsSimt / 32];
    pdl_wait();
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    const AttnShape& s = p.s;
    const float* gq = static_cast<const float*>(p.q);
    const float* gk = static_cast<const float*>(p.k);
    const float* gv = static_cast<const float*>(p.v);
    float* go = static_cast<float*>(p.o);
    const float c = p.scale * 1.44269504089f;  // scores in base 2
    int flags = 0;
    AttnWalk walk;
    struct {
        int r, t, h;
        AttnReq q;
    } it{};
    long long in, each = 0;
    const bool split = p.sp.ws != nullptr;
    if (split) {
        each = attn_cost_each<kThreadsSimt>(s, p.sp.ctas, p.sp.least, s_groups, s_sum);
        __syncthreads();
    }
    // Whole items: numbers blockIdx.x, + gridDim.x, ...; split ones: tiles
    // that start in [cur, end), a key costing 1. Every warp walks by itself, to the same places.
    long long cur = split ? blockIdx.x * each : blockIdx.x;
    const long long end = cur + each;
    long long start = cur;
    if (split) walk = attn_walk_at(s, s_groups, cur);
    bool have = false;
    int tile = 0;
    while (!split || cur < end) {
        if (!have) {
            const bool first = split && cur == start;
            if (!(split ? attn_first_tile(s, walk, &cur, &it.r, &it.q, &it.h, &it.t, &tile) && cur < end
                        : attn_find<false>(s, walk, cur, &it.r, &it.q, &in))) {
                if (first && tid == 0) attn_cuts(p.sp, D)[blockIdx.x] = AttnCut{};
                break;
            }
            if (first) start = cur;
            if (!split) {
                it.t = it.q.nqt - 1 - (int)(in / s.Hkv);
                it.h = (int)(in % s.Hkv);
            }
        }
        const int G = s.G, tok0 = it.t * it.q.tok;
        const int rows = min(it.q.tok, it.q.q_len - tok0) * G;
        const int tiles = attn_item_tiles(s, it.q, it.t);
        // Keys [key0, keys) of the item are this CTA's.
        const long long u0 = cur - tile * kKeys;
        const int last = split ? attn_tiles_until(s, it.q, u0, tiles, end) : tiles;
        const int key0 = tile * kKeys, keys = min(attn_item_keys(it.q, it.t), last * kKeys);
        float* part = nullptr;
        if (split) {
            if (cur == start && tid == 0)
                attn_cuts(p.sp, D)[blockIdx.x] =
                    AttnCut{each, u0, it.q.q0 + tok0, rows / G, it.h, tile, tiles, kKeys};
            if (last - tile < tiles)
                part = p.sp.ws + attn_slot_floats(p.sp.rows, D) * (2 * blockIdx.x + (cur > start ? 1 : 0));
        }
        const size_t first = (size_t)it.q.q0 + tok0;  // packed token of row 0
        __syncthreads();
        for (int i = tid; i < kRows * (D / 4); i += kThreadsSimt) {
            const int r = i / (D / 4), c = (i % (D / 4)) * 4;
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
            if (r < rows)
                x = load4(gq + (first + r / G) * p.q_stride + (size_t)(it.h * G + r % G) * D + c);
            *reinterpret_cast<float4*>(sq + r * LD + c) = x;
        }
        // Keys that each of this thread's rows sees.
        int lim[4];
        float m[4], l[4], acc[4][C4 * 4];
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const int r = ty * 4 + i;
            lim[i] = r < rows ? max(it.q.kv - it.q.q_len + tok0 + r / G + 1, 0) : 0;
            m[i] = -INFINITY;
            l[i] = 0.f;
#pragma unroll
            for (int c = 0; c < C4 * 4; c++) acc[i][c] = 0.f;
        }
        const int seen_by_all = max(it.q.kv - it.q.q_len + tok0 + 1, 0);
        for (int k0 = key0; k0 < keys; k0 += kKeys) {
            __syncthreads();  // the tile before is read
            for (int i = tid; i < kKeys * (D / 4); i += kThreadsSimt) {
                const int j = i / (D / 4), c = (i % (D / 4)) * 4, at = k0 + j;
                float4 xk = make_float4(0.f, 0.f, 0.f, 0.f), xv = xk;
                if (at < keys) {
                    if (p.block_table) {
                        const int id = p.block_table[(size_t)it.r * p.max_pages + at / p.page];
                        if (id >= 0 && id < p.num_pages) {
                            const size_t row = ((size_t)id * s.Hkv + it.h) * p.page + at % p.page;
                            xk = load4(gk + row * D + c);
                            xv = load4(gv + row * D + c);
                        } else {
                            flags |= KDA_DEV_PAGES;
                        }
                    } else {
                        const size_t row = (size_t)it.q.q0 + at;
                        xk = load4(gk + row * p.k_stride + (size_t)it.h * D + c);
                        xv = load4(gv + row * p.v_stride + (size_t)it.h * D + c);
                    }
                }
                *reinterpret_cast<float4*>(sk + j * LD + c) = xk;
                *reinterpret_cast<float4*>(sv + j * LD + c) = xv;
            }
            __syncthreads();
            float x[4][4] = {};
#pragma unroll 4
            for (int e = 0; e < D; e += 4) {
                float4 a[4], b[4];
#pragma unroll
                for (int i = 0; i < 4; i++)
                    a[i] = *reinterpret_cast<const float4*>(sq + (ty * 4 + i) * LD + e);
#pragma unroll
                for (int i = 0; i < 4; i++)
                    b[i] = *reinterpret_cast<const float4*>(sk + (tx + 16 * i) * LD + e);
#pragma unroll
                for (int i = 0; i < 4; i++)
#pragma unroll
                    for (int j = 0; j < 4; j++) {
                        x[i][j] = fmaf(a[i].x, b[j].x, x[i][j]);
                        x[i][j] = fmaf(a[i].y, b[j].y, x[i][j]);
                        x[i][j] = fmaf(a[i].z, b[j].z, x[i][j]);
                        x[i][j] = fmaf(a[i].w, b[j].w, x[i][j]);
                    }
            }
            __syncthreads();  // sk becomes sp
#pragma unroll
            for (int i = 0; i < 4; i++) {
                float mx = -INFINITY;
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    x[i][j] = k0 + tx + 16 * j < lim[i] ? x[i][j] * c : -INFINITY;
                    mx = fmaxf(mx, x[i][j]);
                }
#pragma unroll
                for (int o = 8; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
                const float mn = fmaxf(m[i], mx);
                const float ref = mn == -INFINITY ? 0.f : mn;  // a row that sees nothing yet
                const float corr = exp2f(m[i] - ref);
                m[i] = mn;
                l[i] *= corr;
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    const float e = exp2f(x[i][j] - ref);
                    l[i] += e;  // of this thread's keys
                    sp[(ty * 4 + i) * LP + tx + 16 * j] = e;
                }
#pragma unroll
                for (int c = 0; c < C4 * 4; c++) acc[i][c] *= corr;
            }
            __syncthreads();
            // Rows may see only part of this tile: the other keys add nothing,
            // whatever their values hold.
            const bool edge = k0 + kKeys > seen_by_all;
            auto add = [&](bool guard) {
#pragma unroll 2
                for (int j = 0; j < kKeys; j += 4) {
                    float4 e[4];
#pragma unroll
                    for (int i = 0; i < 4; i++)
                        e[i] = *reinterpret_cast<const float4*>(sp + (ty * 4 + i) * LP + j);
#pragma unroll
                    for (int jj = 0; jj < 4; jj++)
#pragma unroll
                        for (int c = 0; c < C4; c++) {
                            const float4 b = *reinterpret_cast<const float4*>(
                                sv + (j + jj) * LD + tx * 4 + 64 * c);
#pragma unroll
                            for (int i = 0; i < 4; i++) {
                                const float w = jj == 0 ? e[i].x : jj == 1 ? e[i].y : jj == 2 ? e[i].z : e[i].w;
                                if (guard && k0 + j + jj >= lim[i]) continue;
                                acc[i][c * 4] = fmaf(w, b.x, acc[i][c * 4]);
                                acc[i][c * 4 + 1] = fmaf(w, b.y, acc[i][c * 4 + 1]);
                                acc[i][c * 4 + 2] = fmaf(w, b.z, acc[i][c * 4 + 2]);
                                acc[i][c * 4 + 3] = fmaf(w, b.w, acc[i][c * 4 + 3]);
                            }
                        }
                }
            };
            if (edge) add(true);
            else add(false);
        }
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const int r = ty * 4 + i;
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], o);
            if (r >= rows) continue;
            const size_t at = (first + r / G) * s.Hkv * G + it.h * G + r % G;
            float* dst = part ? part + (size_t)r * D : go + at * D;
            const float inv = l[i] > 0.f ? 1.f / l[i] : (l[i] == 0.f ? 0.f : l[i]);  // NaN stays
#pragma unroll
            for (int c = 0; c < C4; c++) {
                const float4 y = make_float4(acc[i][c * 4] * inv, acc[i][c * 4 + 1] * inv,
                                             acc[i][c * 4 + 2] * inv, acc[i][c * 4 + 3] * inv);
                flags |= finite_flag(y.x) | finite_flag(y.y) | finite_flag(y.z) | finite_flag(y.w);
                *reinterpret_cast<float4*>(dst + tx * 4 + 64 * c) = y;
            }
            if (tx == 0) {
                if (part)
                    part[(size_t)p.sp.rows * D + r] =
                        l[i] == 0.f ? -INFINITY : m[i] + log2f(l[i]);
                else if (p.lse)
                    p.lse[at] = l[i] == 0.f ? -INFINITY : (m[i] + log2f(l[i])) * 0.69314718056f;
            }
        }
        if (split) {
            cur = last < tiles ? end
                               : u0 + attn_cost_before(s, it.q, it.t + 1) - attn_cost_before(s, it.q, it.t);
            tile = 0;
            if (++it.t == it.q.nqt) {
                it.t = 0;
                it.h++;
            }
            have = it.h < s.Hkv;
        } else {
            cur += gridDim.x;
        }
    }
    if (blockIdx.x == 0)  // lengths of requests this CTA had no work of
        for (int i = tid; i < s.N; i += kThreadsSimt) walk.bad |= attn_request(s, i).bad != 0;
    if (walk.bad) flags |= KDA_DEV_LENGTH;
    report_flags(p.d_status, flags);
}

template <int D>
cudaError_t launch_t(const AttnArgs& a) {
    const int G = a.Hq / a.Hkv;
    SimtParams p{};
    p.s = {a.cu_q, a.kv_len, a.N, a.total_q, a.max_q,
           attn_kv_cap(a), a.Hkv, G, kRows / G,
           kRows / G, kKeys, 1, 1, 0};
    p.q = a.q;
    p.k = a.k;
    p.v = a.v;
    p.block_table = a.block_table;
    p.o = a.o;
    p.lse = a.lse;
    p.q_stride = a.q_stride;
    p.k_stride = a.k_stride;
    p.v_stride = a.v_stride;
    p.num_pages = a.num_pages;
    p.page = a.page;
    p.max_pages = a.max_pages;
    p.scale = a.scale;
    p.d_status = a.d_status;
    cudaError_t e = cudaFuncSetAttribute(kda_attn_simt_kernel<D>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)simt_smem<D>());
    if (e != cudaSuccess) return e;
    const int nsm = device_sms();
    p.sp = attn_simt_split(a.N, a.total_q, a.max_q, a.kv_len ? p.s.kv_cap : a.max_q, !a.kv_len, a.Hq,
                           a.Hkv, nsm);
    if (p.sp.ctas && a.ws && a.ws_bytes >= attn_split_bytes(p.sp, D)) p.sp.ws = a.ws;
    const long long grid = p.sp.ws ? p.sp.ctas : std::min(attn_items_bound(p.s), 1LL << 20);
    e = launch_dependent(kda_attn_simt_kernel<D>, dim3((unsigned)grid), dim3(kThreadsSimt),
                         simt_smem<D>(), a.stream, p);
    if (e != cudaSuccess || !p.sp.ws) return e;
    return launch_attn_combine(p.sp, a.Hkv, G, D, kRows, a.o, a.lse, KDA_F32, a.d_status, a.stream);
}

}  // namespace

// Ranges unless rows have a key tile or two, or there are enough items to fill the
// SMs evenly. Measured, ranges against whole items, us (8 / 2 heads): d = 64, prompts
// of 200 19/24, 500 32/45, 1000 50/84, 16 x 1000 499/538; d = 128, one token over
// 256 keys 22/46, 4000 58/631.
AttnSplit attn_simt_split(int N, int total_q, int max_q, long long max_keys, bool, int Hq, int Hkv,
                          int nsm) {
    AttnSplit sp{};
    if (N == 0 || total_q == 0 || max_q == 0 || Hkv == 0 || nsm == 0) return sp;
    const int G = Hq / Hkv, tok = kRows / G;
    if (max_keys <= KDA_ATTN_SHORT_KEYS / 16) return sp;
    if ((long long)total_q / tok * Hkv >= 16LL * kCtasPerSm * nsm) return sp;
    sp.ctas = kCtasPerSm * nsm;
    sp.least = kKeys;
    sp.rows = (std::min(max_q, tok) * G + 3) & ~3;  // whole 16-byte vectors
    return sp;
}

cudaError_t launch_attn_simt(const AttnArgs& a) {
    return a.d == 128 ? launch_t<128>(a) : launch_t<64>(a);
}

}  // namespace kda
