// Attention over a paged cache of latents on the CUDA cores, every product and sum in 32 bits.
//
//     x_ij = scale log2(e) q_i . c_j,  p_ij = 2^{x_ij - m_i},  o_i = sum_j p_ij c_j[0 .. 511] / l_i
//
// with one cached row c_j of 512 latent channels and DR rotated ones for all heads. One
// pass over the keys with a running maximum m_i and sum l_i. A CTA of 256 threads holds
// 32 rows (token, head) and takes 32 keys at a time through shared memory, the next 32
// on their way (cp.async) meanwhile; the same tile is keys, then values.
//   Scores: a warp has 4 rows x 32 keys, a thread 4 x 16 of them over every 16th 16-byte vector
//     of the channels, 20 loads for 256 multiply-adds; the 16 lanes of half a warp then add up,
//     each step giving half of a lane's scores away, so that each ends with 4 whole ones of one row.
//   Outputs: a thread has 8 rows x 8 channels, 4 loads for 64 multiply-adds.
// Two of them run in one instruction (fma.rn.f32x2). Where a call has no more than 8 rows a
// tile (single tokens of few heads) the row tile is 8. Long rows are cut into ranges
// as the header of kda_attn.cuh says.
//
// Bound by shared memory and the FMA pipes alike: 20 loads of 16 bytes a lane take 80 clocks of its 128
// bytes a clock, 256 multiply-adds 64 clocks. A mixed step of 9 requests to 2049 keys (two chunks of 33
// tokens among single ones, 8 heads) takes 55 us, 26 TFLOP/s of 74; with 4 x 4 scores a thread (8 loads for 64,
// four lanes adding up, every lane's exponentials four times) 68. Warps whose rows are not there leave the pipes to
// the others: 64 requests of 2048 keys x 16 heads 142 us, 213 without.
#include <algorithm>
#include <atomic>

#include "kda_attn.cuh"
#include "kda_host.cuh"

namespace kda {
namespace {

constexpr int kKeys = 32, kThreads = 256, kDL = kLatentDim;

struct LatentSimtParams {
    AttnShape s;
    AttnSplit sp;
    const float* q;
    const float* cache;
    const int* block_table;
    float* o;
    float* lse;
    long long q_stride, q_head;
    int num_pages, page, max_pages;
    float scale;
    int* d_status;
};

// RT rows of a row tile: 32, or 8 where no more are needed.
template <int DR, int RT>
struct SimtCfg {
    static constexpr int DQ = kDL + DR, LD = DQ + 16;  // rows 16 banks apart
    static constexpr int LP = RT + 4;                  // floats between keys of the probabilities
    static constexpr int P = kKeys * LP * 4 > kAttnGroups * 8 ? kKeys * LP : kAttnGroups * 2;  // floats
    static constexpr size_t SMEM = ((size_t)(RT + 2 * kKeys) * LD + P) * 4;
};

__device__ __forceinline__ void copy16(float* dst, const float* src, bool there) {
    const int n = there ? 16 : 0;  // the rest is zeros
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                     (uint32_t)__cvta_generic_to_shared(dst)),
                 "l"(src), "r"(n)
                 : "memory");
}
__device__ __forceinline__ void copies_end() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ float4 ld4(const float* p) { return *reinterpret_cast<const float4*>(p); }

__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n\t.reg .b64 a, b, c, d;\n\t"
        "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
        "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}

template <int DR, int RT>
__global__ void __launch_bounds__(kThreads, 1) kda_latent_simt_kernel(const LatentSimtParams p) {
    using C = SimtCfg<DR, RT>;
    constexpr int LD = C::LD, LP = C::LP;
    constexpr int RI = RT / 8, RO = RT / 4;  // rows of a thread in the first, in the second product
    constexpr int NV = RI;                   // scores that a thread ends up with, of one row
    constexpr int SPAN = 16 / RI;            // lanes of such a row in a half warp
    extern __shared__ __align__(16) float sm[];
    float* sq = sm;
    float* skv = sq + RT * LD;              // two tiles
    float* sp = skv + 2 * kKeys * LD;       // probabilities [key][row]
    long long* groups = reinterpret_cast<long long*>(sp);  // before the first item
    __shared__ long long s_sum[kThreads / 32];
    __shared__ float s_corr[RT];
    __shared__ int s_lim[RT];

    pdl_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int part = lane & 15, key16 = lane & 16;  // scores: channels 4 part + 64 i, keys key16 .. + 15
    const int row1 = RI * warp + part / SPAN, key1 = key16 + part % SPAN * NV;  // softmax: row, first key
    const int r0 = (tid >> 6) * RO, c4 = (tid & 63) * 4;  // outputs: rows r0 .., channels c4 .., 256 + c4 ..
    const int log2_page = __ffs(p.page) - 1;
    const AttnShape& s = p.s;
    const float c = p.scale * 1.44269504089f;
    int flags = 0;
    AttnWalk walk;
    struct {
        int r, t, h;
        AttnReq q;
    } it{};
    long long in, each = 0;
    const bool split = p.sp.ws != nullptr;
    if (split) {
        each = attn_cost_each<kThreads>(s, p.sp.ctas, p.sp.least, groups, s_sum);
        __syncthreads();
    }
    long long cur = split ? blockIdx.x * each : blockIdx.x;
    const long long end = cur + each;
    long long start = cur;
    if (split) walk = attn_walk_at(s, groups, cur);
    bool have = false;
    int tile = 0;
    while (!split || cur < end) {
        if (!have) {
            const bool first = split && cur == start;
            if (!(split ? attn_first_tile(s, walk, &cur, &it.r, &it.q, &it.h, &it.t, &tile) && cur < end
                        : attn_find<false>(s, walk, cur, &it.r, &it.q, &in))) {
                if (first && tid == 0) attn_cuts(p.sp, kDL)[blockIdx.x] = AttnCut{};
                break;
            }
            if (first) start = cur;
            if (!split && it.q.bad) {
                cur += gridDim.x;
                continue;
            }
            if (!split) {
                it.t = it.q.nqt - 1 - (int)(in / s.Hkv);
                it.h = (int)(in % s.Hkv);
            }
        }
        const int G = s.G, tok0 = it.t * it.q.tok;
        const int rows = min(it.q.tok, it.q.q_len - tok0) * G;
        const int tiles = attn_item_tiles(s, it.q, it.t);
        const long long u0 = cur - (long long)tile * kKeys;
        const int last = split ? attn_tiles_until(s, it.q, u0, tiles, end) : tiles;
        const int key0 = tile * kKeys, keys = min(attn_item_keys(it.q, it.t), last * kKeys);
        float* dst = nullptr;
        if (split) {
            if (cur == start && tid == 0)
                attn_cuts(p.sp, kDL)[blockIdx.x] =
                    AttnCut{each, u0, it.q.q0 + tok0, rows / G, it.h, tile, tiles, kKeys};
            if (last - tile < tiles)
                dst = p.sp.ws + attn_slot_floats(p.sp.rows, kDL) * (2 * blockIdx.x + (cur > start ? 1 : 0));
        }
        const size_t first = (size_t)it.q.q0 + tok0;  // packed token of row 0
        __syncthreads();  // the item before is done with shared memory
        if (const int r = tid >> 3; r < RT) {  // eight threads a row
            const bool there = r < rows;
            const float* src = there ? p.q + (first + r / G) * p.q_stride + (size_t)(it.h * G + r % G) * p.q_head : p.q;
            for (int x = (tid & 7) * 4; x < C::DQ; x += 32) copy16(sq + r * LD + x, there ? src + x : src, there);
        }
        const int seen0 = it.q.kv - it.q.q_len + tok0;  // keys that row 0's token sees, less one
        if (tid < RT) s_lim[tid] = tid < rows ? max(seen0 + tid / G + 1, 0) : 0;
        auto fetch = [&](int k0, int buf) {
            if (k0 < keys) {  // eight threads a key
                const int j = tid >> 3, at = k0 + j;
                const float* src = p.cache;
                bool there = at < keys;
                if (there) {
                    const int id = p.block_table[(size_t)it.r * p.max_pages + (at >> log2_page)];
                    there = id >= 0 && id < p.num_pages;
                    if (there) src += (((size_t)id << log2_page) + (at & (p.page - 1))) * C::DQ;
                    else flags |= KDA_DEV_PAGES;
                }
                float* dst = skv + (buf * kKeys + j) * LD;
                for (int x = (tid & 7) * 4; x < C::DQ; x += 32) copy16(dst + x, there ? src + x : src, there);
            }
            copies_end();
        };
        float m = -INFINITY, l = 0.f;  // (l: of this lane's keys)
        float2 acc[RO][4];
#pragma unroll
        for (int i = 0; i < RO; i++)
#pragma unroll
            for (int e = 0; e < 4; e++) acc[i][e] = make_float2(0.f, 0.f);
        fetch(key0, 0);
        int buf = 0;
        for (int k0 = key0; k0 < keys; k0 += kKeys, buf ^= 1) {
            fetch(k0 + kKeys, buf ^ 1);
            copies_wait<1>();
            __syncthreads();
            const float* kv = skv + buf * kKeys * LD;
            if (RI * warp < rows) {  // (warps without rows leave the pipes to the others)
                float v[16 * RI];
                {
                    float2 y[RI][16];
#pragma unroll
                    for (int i = 0; i < RI; i++)
#pragma unroll
                        for (int j = 0; j < 16; j++) y[i][j] = make_float2(0.f, 0.f);
#pragma unroll 1
                    for (int e = part * 4; e < C::DQ; e += 64) {
                        float4 a[RI];
#pragma unroll
                        for (int i = 0; i < RI; i++) a[i] = ld4(sq + (RI * warp + i) * LD + e);
#pragma unroll
                        for (int j = 0; j < 16; j++) {
                            const float4 b = ld4(kv + (key16 + j) * LD + e);
#pragma unroll
                            for (int i = 0; i < RI; i++) {
                                y[i][j] = fma2(make_float2(a[i].x, a[i].y), make_float2(b.x, b.y), y[i][j]);
                                y[i][j] = fma2(make_float2(a[i].z, a[i].w), make_float2(b.z, b.w), y[i][j]);
                            }
                        }
                    }
#pragma unroll
                    for (int i = 0; i < RI; i++)
#pragma unroll
                        for (int j = 0; j < 16; j++) v[16 * i + j] = y[i][j].x + y[i][j].y;
                }
                // The 16 lanes' sums meet: at each step a lane gives half of its scores away and adds up
                // the other half, so that it ends with NV whole ones.
#pragma unroll
                for (int o = 8, n = 8 * RI; o > 0; o >>= 1, n >>= 1) {
                    const bool up = part & o;
#pragma unroll
                    for (int k = 0; k < n; k++) {
                        const float give = up ? v[k] : v[k + n];
                        v[k] = (up ? v[k + n] : v[k]) + __shfl_xor_sync(0xffffffffu, give, o);
                    }
                }
                const int lim = s_lim[row1];
                float mx = -INFINITY;
#pragma unroll
                for (int j = 0; j < NV; j++) {
                    v[j] = k0 + key1 + j < lim ? v[j] * c : -INFINITY;
                    mx = fmaxf(mx, v[j]);
                }
#pragma unroll
                for (int o = 1; o < SPAN; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
                const float mn = fmaxf(m, mx);
                const float ref = mn == -INFINITY ? 0.f : mn;  // a row that sees nothing yet
                const float corr = exp2f(m - ref);
                m = mn;
                l *= corr;
#pragma unroll
                for (int j = 0; j < NV; j++) {
                    const float e = exp2f(v[j] - ref);
                    l += e;
                    sp[(key1 + j) * LP + row1] = e;
                }
                if (lane % SPAN == 0 && lane < 16) s_corr[row1] = corr;
            }
            __syncthreads();
#pragma unroll
            for (int i = 0; i < RO; i++) {
                const float f = s_corr[r0 + i];
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    acc[i][e].x *= f;
                    acc[i][e].y *= f;
                }
            }
            // Keys that only some rows see add nothing to the others, whatever they hold.
            const bool edge = k0 + kKeys > seen0 + 1;
            auto add = [&](bool guard, int nk) {
#pragma unroll 4
                for (int j = 0; j < nk; j++) {
                    const float4 v0 = ld4(kv + j * LD + c4), v1 = ld4(kv + j * LD + 256 + c4);
                    float w[RO];
                    if constexpr (RO == 8) {
                        const float4 p0 = ld4(sp + j * LP + r0), p1 = ld4(sp + j * LP + r0 + 4);
                        w[0] = p0.x, w[1] = p0.y, w[2] = p0.z, w[3] = p0.w;
                        w[4] = p1.x, w[5] = p1.y, w[6] = p1.z, w[7] = p1.w;
                    } else {
#pragma unroll
                        for (int i = 0; i < RO; i++) w[i] = sp[j * LP + r0 + i];
                    }
#pragma unroll
                    for (int i = 0; i < RO; i++) {
                        if (guard && k0 + j >= s_lim[r0 + i]) continue;
                        const float2 ww = make_float2(w[i], w[i]);
                        acc[i][0] = fma2(ww, make_float2(v0.x, v0.y), acc[i][0]);
                        acc[i][1] = fma2(ww, make_float2(v0.z, v0.w), acc[i][1]);
                        acc[i][2] = fma2(ww, make_float2(v1.x, v1.y), acc[i][2]);
                        acc[i][3] = fma2(ww, make_float2(v1.z, v1.w), acc[i][3]);
                    }
                }
            };
            if (r0 < rows) {
                if (edge) add(true, min(keys - k0, kKeys));
                else add(false, kKeys);
            }
            __syncthreads();  // the tile may be written again
        }
        copies_wait<0>();
        __syncthreads();  // (an item without keys: limits are written)
#pragma unroll
        for (int o = 1; o < SPAN; o <<= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
        l += __shfl_xor_sync(0xffffffffu, l, 16);
        if (lane % SPAN == 0 && lane < 16) {
            s_corr[row1] = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);  // NaN stays
            if (row1 < rows) {
                const size_t at = (first + row1 / G) * s.Hkv * G + it.h * G + row1 % G;
                if (dst)
                    dst[(size_t)p.sp.rows * kDL + row1] =
                        l != 0.f ? m + log2f(l) : key0 < s_lim[row1] ? kAttnNoWeight : -INFINITY;
                else if (p.lse) p.lse[at] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718056f;
            }
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < RO; i++) {
            const int row = r0 + i;
            if (row >= rows) break;
            const float inv = s_corr[row];
            const size_t at = (first + row / G) * s.Hkv * G + it.h * G + row % G;
            float* o = dst ? dst + (size_t)row * kDL : p.o + at * kDL;
            float4 y[2];
#pragma unroll
            for (int e = 0; e < 2; e++) {
                const float2 a = acc[i][2 * e], b = acc[i][2 * e + 1];
                // (a row of no weight: zeros; in a part 0 x NaN stays, as the row may have weight in others)
                y[e] = inv == 0.f && !dst ? make_float4(0.f, 0.f, 0.f, 0.f)
                                          : make_float4(a.x * inv, a.y * inv, b.x * inv, b.y * inv);
                // (of parts the join looks at the joined rows)
                if (!dst) flags |= finite_flag(y[e].x) | finite_flag(y[e].y) | finite_flag(y[e].z) | finite_flag(y[e].w);
            }
            *reinterpret_cast<float4*>(o + c4) = y[0];
            *reinterpret_cast<float4*>(o + 256 + c4) = y[1];
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
        for (int i = tid; i < s.N; i += kThreads) walk.bad |= attn_request<true>(s, i).bad != 0;
    if (walk.bad) flags |= KDA_DEV_LENGTH;
    report_flags(p.d_status, flags);
}

template <int DR, int RT>
cudaError_t launch_t(const AttnArgs& a) {
    using C = SimtCfg<DR, RT>;
    LatentSimtParams p{};
    const int blocks = latent_head_blocks(a.Hq, RT), G = a.Hq / blocks, tok = RT / G;
    int dev = 0;
    const int nsm = device_sms(&dev);
    if (nsm == 0) return cudaErrorNoDevice;
    p.s = {a.cu_q, a.kv_len, a.N, a.total_q, a.max_q, attn_kv_cap(a), blocks, G, tok, tok, kKeys, 1, 1, 0};
    p.q = static_cast<const float*>(a.q);
    p.cache = static_cast<const float*>(a.k);
    p.block_table = a.block_table;
    p.o = static_cast<float*>(a.o);
    p.lse = a.lse;
    p.q_stride = a.q_stride;
    p.q_head = a.q_head;
    p.num_pages = a.num_pages;
    p.page = a.page;
    p.max_pages = a.max_pages;
    p.scale = a.scale;
    p.d_status = a.d_status;
    static std::atomic<uint64_t> ready{0};
    cudaError_t e = allow_shared(kda_latent_simt_kernel<DR, RT>, C::SMEM, ready, dev);
    if (e != cudaSuccess) return e;
    p.sp = latent_simt_split(a.N, a.total_q, a.max_q, p.s.kv_cap, a.Hq, nsm);
    if (p.sp.ctas && a.ws && a.ws_bytes >= attn_split_bytes(p.sp, kDL)) p.sp.ws = a.ws;
    const long long grid = p.sp.ws ? p.sp.ctas : std::min(attn_items_bound(p.s), (long long)nsm);  // one per SM
    e = launch_dependent(kda_latent_simt_kernel<DR, RT>, dim3((unsigned)grid), dim3(kThreads), C::SMEM,
                         a.stream, p);
    if (e != cudaSuccess || !p.sp.ws) return e;
    return launch_attn_combine(p.sp, blocks, G, kDL, RT, a.o, a.lse, KDA_F32, a.d_status, a.stream);
}

}  // namespace

AttnSplit latent_simt_split(int N, int total_q, int max_q, long long max_keys, int Hq, int nsm) {
    AttnSplit sp{};
    if (N == 0 || total_q == 0 || max_q == 0 || Hq == 0 || nsm == 0) return sp;
    const int rt = latent_simt_rows(max_q, Hq), blocks = latent_head_blocks(Hq, rt), G = Hq / blocks, tok = rt / G;
    // Ranges, unless the keys are so few that their join costs more. Measured, ranges against whole
    // items, us: of 32 keys 4 requests x 8 heads 12.0/9.3, 64 x 32 heads 17/15; of 64 keys
    // 13.9/13.7 and 27/22; of 128 keys 14/23 and 34/36, 1024 requests x 16 heads 169/169; 4864 of 256
    // keys x 16 heads 1313/1334.
    if (max_keys <= KDA_LATENT_SHORT_KEYS / 4) return sp;
    sp.ctas = nsm;
    sp.least = kKeys;
    sp.rows = (std::min(max_q, tok) * G + 3) & ~3;  // whole 16-byte vectors
    return sp;
}

cudaError_t launch_latent_simt(const AttnArgs& a) {
    // (8 rows against 32, us: 1 request of 2048 keys x 4 heads 12/14, 4 of 4096 x 1 head 20/28, 64 of 100 x 2
    // heads 16/20, 9 of 2000 x 6 28/31; with 8 heads there is no difference, 16 of 2048 44/43)
    if (latent_simt_rows(a.max_q, a.Hq) == 8) return a.dr ? launch_t<64, 8>(a) : launch_t<0, 8>(a);
    return a.dr ? launch_t<64, 32>(a) : launch_t<0, 32>(a);
}

}  // namespace kda
