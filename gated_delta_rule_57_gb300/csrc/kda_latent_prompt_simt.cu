// Latent attention over packed prompts (expanded heads) on the CUDA cores, every product
// and sum in 32 bits.
//
//     x_ij = scale log2(e) (q_i . k_j + r_i . s_j),  p_ij = 2^{x_ij - m_i},  o_i = sum_j p_ij v_j / l_i
//
// with r_i the last DR channels of a query and s_j key channels that all heads share. One
// pass over the keys with a running maximum m_i and sum l_i. A CTA of 256 threads holds
// 16 RI rows (tokens of one head) and takes 64 keys at a time through shared memory. The
// keys of the next tile are on their way (cp.async) from the softmax on, its values
// from the end of the second product on. Queries (once an item) and probabilities stand
// transposed, so that a thread's rows are vectors; two multiply-adds run in one
// instruction (fma.rn.f32x2): two rows of a score, two channels of an output.
//
// Bound by shared memory, whose 128 bytes a clock bring one operand vector a lane in 4 clocks a warp,
// and by the FMA pipes (128 multiply-adds a clock). So a thread's tile is large: the two halves of a
// CTA take half of the channels each, RI x 8 scores a thread (RI = 8: 16 vectors, 64 clocks, for 256
// multiply-adds a lane, 64 clocks), and exchange half of their sums; then RI rows x 8 channels of the outputs (the
// same ratio). With all channels in each thread and RI x 4 scores (12 vectors for 128) 4 prompts of 2048
// tokens x 32 heads took 3780 us where this takes 3490 (49 TFLOP/s of 74, and a tenth more above the
// diagonal); 3 prompts to 1021 tokens of 8 heads 98 and 93; but 64 of 64 tokens x 16 heads, at RI = 4, 110
// and 121, 16 of 300 x 8 159 and 155.
#include <algorithm>
#include <atomic>

#include "kda_attn.cuh"
#include "kda_host.cuh"

namespace kda {
namespace {

constexpr int kThreads = 256, kKeys = 64, kD = 128, kLV = kD + 4;
constexpr int kKeysT = 8;  // keys of a thread's scores

struct PromptSimtParams {
    AttnShape s;
    AttnSplit sp;
    const float* q;
    const float* k;
    const float* k_r;
    const float* v;
    float* o;
    float* lse;
    long long q_stride, q_head, k_stride, k_head, kr_stride, v_stride, v_head;
    float scale;
    int* d_status;
};

template <int DR, int RI>
struct SimtCfg {
    static constexpr int DQ = kD + DR, LK = DQ + 4, ROWS = 16 * RI;
    static constexpr int LR = ROWS + 4;  // of the queries' channels and of the probabilities' keys
    static constexpr size_t SMEM = (size_t)(DQ * LR + kKeys * LK + kKeys * kLV + kKeys * LR) * 4;
    static_assert(kKeys * LR >= kThreads * RI / 2 * kKeysT, "half of the scores fit the probabilities");
    static_assert(kKeys * LR * 4 >= kAttnGroups * 8, "groups fit the probabilities");
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

template <int DR, int RI>
__global__ void __launch_bounds__(kThreads, 1) kda_latent_prompt_simt_kernel(const PromptSimtParams p) {
    using C = SimtCfg<DR, RI>;
    constexpr int DQ = C::DQ, LK = C::LK, LR = C::LR, ROWS = C::ROWS;
    constexpr int RS = RI / 2;  // rows of a thread's softmax
    extern __shared__ __align__(16) float sm[];
    float* sq = sm;  // [channel][row]
    float* sk = sq + DQ * LR;
    float* sv = sk + kKeys * LK;
    float* sp = sv + kKeys * kLV;  // probabilities [key][row]
    long long* groups = reinterpret_cast<long long*>(sp);  // before the first item
    __shared__ long long s_sum[kThreads / 32];
    __shared__ float s_factor[ROWS];  // of the rows' outputs: of a tile, at last 1 / l

    pdl_wait();
    const int tid = threadIdx.x;
    const int tx = tid & 15, ty = tid >> 4;  // outputs: channels 4 tx .., 64 + 4 tx ..; rows RI ty ..
    // scores: half of the channels, keys kx + 8 j, rows RI ky ..; softmax: of those rows RS from row0 on
    const int half = tid >> 7, kx = tid & 7, ky = tid >> 3 & 15, row0 = RI * ky + RS * half;
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
    // Whole items: numbers blockIdx.x, + gridDim.x, ...; split ones: tiles that start in
    // [cur, end). Every warp walks by itself, to the same places.
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
                if (first && tid == 0) attn_cuts(p.sp, kD)[blockIdx.x] = AttnCut{};
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
        const int tok0 = it.t * it.q.tok;
        const int rows = min(it.q.tok, it.q.q_len - tok0);
        const int tiles = attn_item_tiles(s, it.q, it.t);
        const long long u0 = cur - (long long)tile * kKeys;
        const int last = split ? attn_tiles_until(s, it.q, u0, tiles, end) : tiles;
        const int key0 = tile * kKeys, keys = min(attn_item_keys(it.q, it.t), last * kKeys);
        float* part = nullptr;
        if (split) {
            if (cur == start && tid == 0)
                attn_cuts(p.sp, kD)[blockIdx.x] = AttnCut{each, u0, it.q.q0 + tok0, rows, it.h, tile, tiles, kKeys};
            if (last - tile < tiles)
                part = p.sp.ws + attn_slot_floats(p.sp.rows, kD) * (2 * blockIdx.x + (cur > start ? 1 : 0));
        }
        const size_t first = (size_t)it.q.q0 + tok0;  // packed token of row 0
        __syncthreads();  // the item before is done with shared memory
        // Rows of 128 channels, a warp a row; of DR channels, 16 lanes a row.
        const int wr = tid >> 5, wx = (tid & 31) * 4, hx = tx * 4;
        auto copy_rows = [&](float* dst, int ld, const float* src, long long stride, int n, int there) {
#pragma unroll 1
            for (int j = wr; j < n; j += kThreads / 32)
                copy16(dst + j * ld + wx, j < there ? src + j * stride + wx : src, j < there);
        };
        auto copy_ends = [&](float* dst, int ld, const float* src, long long stride, int n, int there) {
            if constexpr (DR > 0)
#pragma unroll 1
                for (int j = ty; j < n; j += kThreads / 16)
                    copy16(dst + j * ld + hx, j < there ? src + j * stride + hx : src, j < there);
        };
        const float* kh = p.k + (size_t)it.q.q0 * p.k_stride + it.h * p.k_head;
        const float* rh = DR > 0 ? p.k_r + (size_t)it.q.q0 * p.kr_stride : nullptr;
        const float* vh = p.v + (size_t)it.q.q0 * p.v_stride + it.h * p.v_head;
        auto fetch_keys = [&](int k0) {
            if (k0 < keys) {
                copy_rows(sk, LK, kh + k0 * p.k_stride, p.k_stride, kKeys, keys - k0);
                if (DR > 0) copy_ends(sk + kD, LK, rh + k0 * p.kr_stride, p.kr_stride, kKeys, keys - k0);
            }
            copies_end();
        };
        auto fetch_values = [&](int k0) {
            if (k0 < keys) copy_rows(sv, kLV, vh + k0 * p.v_stride, p.v_stride, kKeys, keys - k0);
            copies_end();
        };
        fetch_keys(key0);
        fetch_values(key0);
        // Queries: a lane a row, so that writing them transposed meets no bank twice.
        const float* qh = p.q + first * p.q_stride + it.h * p.q_head;
        for (int i = tid; i < ROWS * (DQ / 4); i += kThreads) {
            const int r = i % ROWS, e = i / ROWS * 4;
            const float4 x = r < rows ? ld4(qh + r * p.q_stride + e) : make_float4(0.f, 0.f, 0.f, 0.f);
            sq[e * LR + r] = x.x;
            sq[(e + 1) * LR + r] = x.y;
            sq[(e + 2) * LR + r] = x.z;
            sq[(e + 3) * LR + r] = x.w;
        }
        const int seen0 = it.q.kv - it.q.q_len + tok0;  // position of row 0
        auto lim = [&](int r) { return r < rows ? seen0 + r + 1 : 0; };  // keys that row r sees
        float m[RS], l[RS];
        float2 acc[RI][4];
#pragma unroll
        for (int i = 0; i < RS; i++) {
            m[i] = -INFINITY;
            l[i] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < RI; i++)
#pragma unroll
            for (int e = 0; e < 4; e++) acc[i][e] = make_float2(0.f, 0.f);
        for (int k0 = key0; k0 < keys; k0 += kKeys) {
            copies_wait<1>();  // the keys
            __syncthreads();
            // In small row tiles, for short prompts, warps without rows leave the pipes to the
            // others, and keys that are not there are left out. (27 prompts of 5 tokens x 40 heads 103 -> 76 us, 16
            // of 200 x 8 108 -> 101; in large ones the tests alone cost 2 to 4 %.)
            const bool live = RI > 4 || 4 * RI * (tid >> 5 & 3) < rows;
            float x[RS][kKeysT];
            {
                float2 y[RI / 2][kKeysT];  // of two rows
#pragma unroll
                for (int i = 0; i < RI / 2; i++)
#pragma unroll
                    for (int j = 0; j < kKeysT; j++) y[i][j] = make_float2(0.f, 0.f);
                const float* ka = sk + kx * LK + half * (DQ / 2);
                const float* qa = sq + half * (DQ / 2) * LR + RI * ky;
#pragma unroll 1
                for (int e = live ? 0 : DQ / 2; e < DQ / 2; e += 4) {
                    float b[kKeysT][4];
#pragma unroll
                    for (int j = 0; j < kKeysT; j++)
                        *reinterpret_cast<float4*>(b[j]) = ld4(ka + 8 * j * LK + e);
#pragma unroll
                    for (int c = 0; c < 4; c++)
#pragma unroll
                        for (int i = 0; i < RI / 4; i++) {
                            const float4 a = ld4(qa + (e + c) * LR + 4 * i);
#pragma unroll
                            for (int j = 0; j < kKeysT; j++) {
                                const float2 bb = make_float2(b[j][c], b[j][c]);
                                y[2 * i][j] = fma2(make_float2(a.x, a.y), bb, y[2 * i][j]);
                                y[2 * i + 1][j] = fma2(make_float2(a.z, a.w), bb, y[2 * i + 1][j]);
                            }
                        }
                }
                // The halves' sums meet: each thread keeps RS of its rows and gives the others away.
                float2* give = reinterpret_cast<float2*>(sp);
#pragma unroll
                for (int i = 0; i < RS / 2; i++)
#pragma unroll
                    for (int j = 0; j < kKeysT; j++)
                        give[(kKeysT * i + j) * kThreads + tid] = half ? y[i][j] : y[RS / 2 + i][j];
                __syncthreads();
#pragma unroll
                for (int i = 0; i < RS / 2; i++)
#pragma unroll
                    for (int j = 0; j < kKeysT; j++) {
                        const float2 mine = half ? y[RS / 2 + i][j] : y[i][j];
                        const float2 got = give[(kKeysT * i + j) * kThreads + (tid ^ kThreads / 2)];
                        x[2 * i][j] = (mine.x + got.x) * c;
                        x[2 * i + 1][j] = (mine.y + got.y) * c;
                    }
            }
            fetch_keys(k0 + kKeys);
            const bool edge = k0 + kKeys > seen0 + 1;  // some row does not see all of the tile
            if (edge) {
#pragma unroll
                for (int i = 0; i < RS; i++)
#pragma unroll
                    for (int j = 0; j < kKeysT; j++) x[i][j] = k0 + kx + 8 * j < lim(row0 + i) ? x[i][j] : -INFINITY;
            }
#pragma unroll
            for (int i = 0; i < RS; i++) {
                float mx = x[i][0];
#pragma unroll
                for (int j = 1; j < kKeysT; j++) mx = fmaxf(mx, x[i][j]);
#pragma unroll
                for (int o = 4; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
                const float mn = fmaxf(m[i], mx);
                const float ref = mn == -INFINITY ? 0.f : mn;  // a row that sees nothing yet
                const float corr = exp2f(m[i] - ref);
                m[i] = mn;
                l[i] *= corr;
#pragma unroll
                for (int j = 0; j < kKeysT; j++) {
                    x[i][j] = exp2f(x[i][j] - ref);
                    l[i] += x[i][j];  // of this thread's keys
                }
                if (kx == 0) s_factor[row0 + i] = corr;
            }
            __syncthreads();  // what was given is read
#pragma unroll
            for (int j = 0; j < kKeysT; j++) {
                float* at = sp + (kx + 8 * j) * LR + row0;
                if constexpr (RS == 4)
                    *reinterpret_cast<float4*>(at) = make_float4(x[0][j], x[1][j], x[2][j], x[3][j]);
                else
                    *reinterpret_cast<float2*>(at) = make_float2(x[0][j], x[1][j]);
            }
            copies_wait<1>();  // the values
            // 0 x NaN: where some rows do not see all keys and a value is not finite, a row
            // takes only the keys that it sees.
            bool guard = false;
            __syncthreads();
#pragma unroll
            for (int i = 0; i < RI; i++) {
                const float corr = s_factor[RI * ty + i];
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    acc[i][e].x *= corr;
                    acc[i][e].y *= corr;
                }
            }
            if (edge) {
                bool odd = false;
                for (int i = tid; i < kKeys * (kD / 4); i += kThreads) {
                    const float4 y = ld4(sv + i / (kD / 4) * kLV + (i % (kD / 4)) * 4);
                    odd |= (finite_flag(y.x) | finite_flag(y.y) | finite_flag(y.z) | finite_flag(y.w)) != 0;
                }
                guard = __syncthreads_or(odd);
            }
            auto add = [&](bool guarded, int nk) {
#pragma unroll 4
                for (int j = 0; j < nk; j++) {
                    const float4 v0 = ld4(sv + j * kLV + tx * 4), v1 = ld4(sv + j * kLV + 64 + tx * 4);
                    float w[RI];
#pragma unroll
                    for (int i = 0; i < RI; i += 4)
                        *reinterpret_cast<float4*>(w + i) = ld4(sp + j * LR + RI * ty + i);
#pragma unroll
                    for (int i = 0; i < RI; i++) {
                        if (guarded && k0 + j >= lim(RI * ty + i)) continue;
                        const float2 ww = make_float2(w[i], w[i]);
                        acc[i][0] = fma2(ww, make_float2(v0.x, v0.y), acc[i][0]);
                        acc[i][1] = fma2(ww, make_float2(v0.z, v0.w), acc[i][1]);
                        acc[i][2] = fma2(ww, make_float2(v1.x, v1.y), acc[i][2]);
                        acc[i][3] = fma2(ww, make_float2(v1.z, v1.w), acc[i][3]);
                    }
                }
            };
            if (RI > 4 || 2 * RI * (tid >> 5) < rows) {
                if (guard) add(true, kKeys);
                else add(false, RI == 4 ? min(keys - k0, kKeys) : kKeys);
            }
            __syncthreads();
            fetch_values(k0 + kKeys);
        }
        copies_wait<0>();
#pragma unroll
        for (int i = 0; i < RS; i++) {
            const int r = row0 + i;
#pragma unroll
            for (int o = 4; o > 0; o >>= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], o);
            if (kx != 0) continue;
            s_factor[r] = l[i] > 0.f ? 1.f / l[i] : (l[i] == 0.f ? 0.f : l[i]);  // NaN stays
            if (r >= rows) continue;
            if (part) part[(size_t)p.sp.rows * kD + r] = l[i] == 0.f ? -INFINITY : m[i] + log2f(l[i]);
            else if (p.lse)
                p.lse[(first + r) * s.Hkv + it.h] = l[i] == 0.f ? -INFINITY : (m[i] + log2f(l[i])) * 0.69314718056f;
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < RI; i++) {
            const int r = RI * ty + i;
            if (r >= rows) break;
            float* dst = part ? part + (size_t)r * kD : p.o + ((first + r) * s.Hkv + it.h) * kD;
            const float inv = s_factor[r];
            const float y[8] = {acc[i][0].x * inv, acc[i][0].y * inv, acc[i][1].x * inv, acc[i][1].y * inv,
                                acc[i][2].x * inv, acc[i][2].y * inv, acc[i][3].x * inv, acc[i][3].y * inv};
#pragma unroll
            for (int e = 0; e < 8; e++) flags |= finite_flag(y[e]);
            *reinterpret_cast<float4*>(dst + tx * 4) = make_float4(y[0], y[1], y[2], y[3]);
            *reinterpret_cast<float4*>(dst + 64 + tx * 4) = make_float4(y[4], y[5], y[6], y[7]);
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

template <int DR, int RI>
cudaError_t launch_t(const AttnArgs& a) {
    using C = SimtCfg<DR, RI>;
    int dev = 0;
    const int nsm = device_sms(&dev);
    if (nsm == 0) return cudaErrorNoDevice;
    PromptSimtParams p{};
    p.s = {a.cu_q, nullptr, a.N, a.total_q, a.max_q, 0, a.Hq, 1, C::ROWS, C::ROWS, kKeys, 1, 1, 0};
    p.q = static_cast<const float*>(a.q);
    p.k = static_cast<const float*>(a.k);
    p.k_r = static_cast<const float*>(a.k_r);
    p.v = static_cast<const float*>(a.v);
    p.o = static_cast<float*>(a.o);
    p.lse = a.lse;
    p.q_stride = a.q_stride;
    p.q_head = a.q_head;
    p.k_stride = a.k_stride;
    p.k_head = a.k_head;
    p.kr_stride = a.kr_stride;
    p.v_stride = a.v_stride;
    p.v_head = a.v_head;
    p.scale = a.scale;
    p.d_status = a.d_status;
    static std::atomic<uint64_t> ready{0};
    cudaError_t e = allow_shared(kda_latent_prompt_simt_kernel<DR, RI>, C::SMEM, ready, dev);
    if (e != cudaSuccess) return e;
    // Ranges unless rows have few key tiles, or there are enough items to fill the SMs evenly.
    // Measured, ranges against whole items, us: 2 prompts of 256 tokens x 8 heads 34/44, 8 x 16 heads
    // 109/116, 32 x 16 heads 399/409, 4 of 2048 x 32 heads 3484/3488; of 128 tokens 2 x 8 heads 25/26,
    // 16 x 16 heads 83/78.
    if (a.max_q > 2 * kKeys && (long long)a.total_q / C::ROWS * a.Hq < 16LL * nsm) {
        p.sp.ctas = nsm;
        p.sp.least = kKeys;
        p.sp.rows = std::min((a.max_q + 3) & ~3, C::ROWS);  // whole 16-byte vectors
        if (a.ws && a.ws_bytes >= attn_split_bytes(p.sp, kD)) p.sp.ws = a.ws;
    }
    // Whole items: a CTA for each, which evens out long ones, or one per SM, which walks over the
    // requests once instead of for every item. Measured, a CTA an item against one per SM, us: 8
    // prompts of 2048 x 32 heads 6940/7130, 40 of 100 .. 1000 x 32 4320/4550, 64 of 128 x 32 563/525; 200
    // of 1 .. 128 x 16 658/595, 256 of 33 x 32 992/757, 1000 of 128 x 8 3770/2030, 4864 of 64 x 2 7400/1030.
    const long long most = a.N > 64 ? nsm : 1 << 20;
    const long long grid = p.sp.ws ? p.sp.ctas : std::min(attn_items_bound(p.s), most);
    e = launch_dependent(kda_latent_prompt_simt_kernel<DR, RI>, dim3((unsigned)grid), dim3(kThreads), C::SMEM,
                         a.stream, p);
    if (e != cudaSuccess || !p.sp.ws) return e;
    return launch_attn_combine(p.sp, a.Hq, 1, kD, C::ROWS, a.o, a.lse, KDA_F32, a.d_status, a.stream);
}

}  // namespace

cudaError_t launch_latent_prompt_simt(const AttnArgs& a) {
    // Row tiles of 64 or 128. Small ones waste less of a short prompt, on keys behind the diagonal and
    // in the last tile; large ones read keys and values half as often. Measured, 64 against 128, us: 64
    // prompts of 64 tokens x 16 heads 121/174, 64 of 128 286/287, 16 of 200 x 8 heads 108/113, 16 of 300
    // 156/195; 8 of 512 x 16 heads 335/312, 4 of 2048 x 32 heads 4210/3484.
    if (a.max_q <= 384) return a.dr ? launch_t<64, 4>(a) : launch_t<0, 4>(a);
    return a.dr ? launch_t<64, 8>(a) : launch_t<0, 8>(a);
}

}  // namespace kda
