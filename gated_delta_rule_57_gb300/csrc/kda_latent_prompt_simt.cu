// Latent attention over packed prompts (expanded heads) on the CUDA cores, every product
// and sum in 32 bits.
//
//     x_ij = scale log2(e) (q_i . k_j + r_i . s_j),  p_ij = 2^{x_ij - m_i},  o_i = sum_j p_ij v_j / l_i
//
// with r_i the last DR channels of a query and s_j key channels that all heads share. One
// pass over the keys with a running maximum m_i and sum l_i. A CTA of 256 threads holds
// 16 RI rows (tokens of one head) and takes 64 keys at a time through shared memory. Thread
// (y, x) has rows RI y .. against keys x + 16 j, then the same rows of 8 output channels.
// The keys of the next tile are on their way (cp.async) from the softmax on, its values
// from the end of the second product on; the rows of a warp are its own, so P needs no
// barrier. Two products run in one instruction (fma.rn.f32x2): even and odd channels
// of a score, two neighbouring channels of an output.
//
// Bound by shared memory in the first product (at RI = 8 12 loads of 16 bytes a lane, 48 clocks
// a warp, for 128 multiply-adds, 32 clocks) and by the FMA pipes in the second. Three prompts to 1021
// tokens of 8 heads take 98 us, 28 TFLOP/s of 74; with loads between the products instead of
// beside them, single multiply-adds and 64-row tiles they took 141.
#include <algorithm>
#include <atomic>

#include "kda_attn.cuh"
#include "kda_host.cuh"

namespace kda {
namespace {

constexpr int kThreads = 256, kKeys = 64, kD = 128, kLP = kKeys + 4, kLV = kD + 4;

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
    static constexpr int DQ = kD + DR, LQ = DQ + 4, ROWS = 16 * RI;
    static constexpr size_t SMEM = (size_t)((ROWS + kKeys) * LQ + kKeys * kLV + ROWS * kLP) * 4;
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
    constexpr int DQ = C::DQ, LQ = C::LQ, ROWS = C::ROWS;
    extern __shared__ __align__(16) float sm[];
    float* sq = sm;
    float* sk = sq + ROWS * LQ;
    float* sv = sk + kKeys * LQ;
    float* sp = sv + kKeys * kLV;  // probabilities
    long long* groups = reinterpret_cast<long long*>(sp);  // before the first item
    static_assert(kAttnGroups * 8 <= ROWS * kLP * 4, "groups fit the probabilities");
    __shared__ long long s_sum[kThreads / 32];

    pdl_wait();
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
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
        const float* qh = p.q + first * p.q_stride + it.h * p.q_head;
        copy_rows(sq, LQ, qh, p.q_stride, ROWS, rows);
        copy_ends(sq + kD, LQ, qh + kD, p.q_stride, ROWS, rows);
        const float* kh = p.k + (size_t)it.q.q0 * p.k_stride + it.h * p.k_head;
        const float* rh = DR > 0 ? p.k_r + (size_t)it.q.q0 * p.kr_stride : nullptr;
        const float* vh = p.v + (size_t)it.q.q0 * p.v_stride + it.h * p.v_head;
        auto fetch_keys = [&](int k0) {
            if (k0 < keys) {
                copy_rows(sk, LQ, kh + k0 * p.k_stride, p.k_stride, kKeys, keys - k0);
                if (DR > 0) copy_ends(sk + kD, LQ, rh + k0 * p.kr_stride, p.kr_stride, kKeys, keys - k0);
            }
            copies_end();
        };
        auto fetch_values = [&](int k0) {
            if (k0 < keys) copy_rows(sv, kLV, vh + k0 * p.v_stride, p.v_stride, kKeys, keys - k0);
            copies_end();
        };
        fetch_keys(key0);
        fetch_values(key0);
        // Row i of this thread is RI ty + i; it sees keys up to its own position.
        const int seen0 = it.q.kv - it.q.q_len + tok0;  // position of row 0
        float m[RI], l[RI];
        float2 acc[RI][4];
#pragma unroll
        for (int i = 0; i < RI; i++) {
            m[i] = -INFINITY;
            l[i] = 0.f;
#pragma unroll
            for (int e = 0; e < 4; e++) acc[i][e] = make_float2(0.f, 0.f);
        }
        auto lim = [&](int i) {
            const int r = RI * ty + i;
            return r < rows ? seen0 + r + 1 : 0;
        };
        for (int k0 = key0; k0 < keys; k0 += kKeys) {
            copies_wait<1>();  // the keys
            __syncthreads();
            float x[RI][4];
            {
                float2 y[RI][4];
#pragma unroll
                for (int i = 0; i < RI; i++)
#pragma unroll
                    for (int j = 0; j < 4; j++) y[i][j] = make_float2(0.f, 0.f);
#pragma unroll 2
                for (int e = 0; e < DQ; e += 4) {
                    float4 b[4];
#pragma unroll
                    for (int j = 0; j < 4; j++) b[j] = ld4(sk + (tx + 16 * j) * LQ + e);
#pragma unroll
                    for (int i = 0; i < RI; i++) {
                        const float4 a = ld4(sq + (RI * ty + i) * LQ + e);
#pragma unroll
                        for (int j = 0; j < 4; j++) {
                            y[i][j] = fma2(make_float2(a.x, a.y), make_float2(b[j].x, b[j].y), y[i][j]);
                            y[i][j] = fma2(make_float2(a.z, a.w), make_float2(b[j].z, b[j].w), y[i][j]);
                        }
                    }
                }
#pragma unroll
                for (int i = 0; i < RI; i++)
#pragma unroll
                    for (int j = 0; j < 4; j++) x[i][j] = (y[i][j].x + y[i][j].y) * c;
            }
            __syncthreads();
            fetch_keys(k0 + kKeys);
            const bool edge = k0 + kKeys > seen0 + 1;  // some row does not see all of the tile
            if (edge) {
#pragma unroll
                for (int i = 0; i < RI; i++)
#pragma unroll
                    for (int j = 0; j < 4; j++) x[i][j] = k0 + tx + 16 * j < lim(i) ? x[i][j] : -INFINITY;
            }
            __syncwarp();  // P of the tile before is read
#pragma unroll
            for (int i = 0; i < RI; i++) {
                float mx = fmaxf(fmaxf(x[i][0], x[i][1]), fmaxf(x[i][2], x[i][3]));
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
                    sp[(RI * ty + i) * kLP + tx + 16 * j] = e;
                }
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    acc[i][e].x *= corr;
                    acc[i][e].y *= corr;
                }
            }
            copies_wait<1>();  // the values
            // 0 x NaN: where some rows do not see all keys and a value is not finite, a row
            // takes only the keys that it sees.
            bool guard = false;
            __syncthreads();
            if (edge) {
                bool odd = false;
                for (int i = tid; i < kKeys * (kD / 4); i += kThreads) {
                    const float4 y = ld4(sv + i / (kD / 4) * kLV + (i % (kD / 4)) * 4);
                    odd |= (finite_flag(y.x) | finite_flag(y.y) | finite_flag(y.z) | finite_flag(y.w)) != 0;
                }
                guard = __syncthreads_or(odd);
            }
            if (!guard) {
#pragma unroll 2
                for (int j = 0; j < kKeys; j += 4) {
                    float4 v0[4], v1[4];
#pragma unroll
                    for (int k = 0; k < 4; k++) {
                        v0[k] = ld4(sv + (j + k) * kLV + tx * 4);
                        v1[k] = ld4(sv + (j + k) * kLV + 64 + tx * 4);
                    }
#pragma unroll
                    for (int i = 0; i < RI; i++) {
                        const float4 w4 = ld4(sp + (RI * ty + i) * kLP + j);
                        const float w[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
                        for (int k = 0; k < 4; k++) {
                            const float2 ww = make_float2(w[k], w[k]);
                            acc[i][0] = fma2(ww, make_float2(v0[k].x, v0[k].y), acc[i][0]);
                            acc[i][1] = fma2(ww, make_float2(v0[k].z, v0[k].w), acc[i][1]);
                            acc[i][2] = fma2(ww, make_float2(v1[k].x, v1[k].y), acc[i][2]);
                            acc[i][3] = fma2(ww, make_float2(v1[k].z, v1[k].w), acc[i][3]);
                        }
                    }
                }
            } else {
                for (int j = 0; j < kKeys; j++) {
                    const float4 v0 = ld4(sv + j * kLV + tx * 4), v1 = ld4(sv + j * kLV + 64 + tx * 4);
#pragma unroll
                    for (int i = 0; i < RI; i++) {
                        if (k0 + j >= lim(i)) continue;
                        const float w = sp[(RI * ty + i) * kLP + j];
                        const float2 ww = make_float2(w, w);
                        acc[i][0] = fma2(ww, make_float2(v0.x, v0.y), acc[i][0]);
                        acc[i][1] = fma2(ww, make_float2(v0.z, v0.w), acc[i][1]);
                        acc[i][2] = fma2(ww, make_float2(v1.x, v1.y), acc[i][2]);
                        acc[i][3] = fma2(ww, make_float2(v1.z, v1.w), acc[i][3]);
                    }
                }
            }
            __syncthreads();
            fetch_values(k0 + kKeys);
        }
        copies_wait<0>();
#pragma unroll
        for (int i = 0; i < RI; i++) {
            const int r = RI * ty + i;
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], o);
            if (r >= rows) continue;
            const size_t at = (first + r) * s.Hkv + it.h;
            float* dst = part ? part + (size_t)r * kD : p.o + at * kD;
            const float inv = l[i] > 0.f ? 1.f / l[i] : (l[i] == 0.f ? 0.f : l[i]);  // NaN stays
            const float y[8] = {acc[i][0].x * inv, acc[i][0].y * inv, acc[i][1].x * inv, acc[i][1].y * inv,
                                acc[i][2].x * inv, acc[i][2].y * inv, acc[i][3].x * inv, acc[i][3].y * inv};
#pragma unroll
            for (int e = 0; e < 8; e++) flags |= finite_flag(y[e]);
            *reinterpret_cast<float4*>(dst + tx * 4) = make_float4(y[0], y[1], y[2], y[3]);
            *reinterpret_cast<float4*>(dst + 64 + tx * 4) = make_float4(y[4], y[5], y[6], y[7]);
            if (tx == 0) {
                if (part) part[(size_t)p.sp.rows * kD + r] = l[i] == 0.f ? -INFINITY : m[i] + log2f(l[i]);
                else if (p.lse) p.lse[at] = l[i] == 0.f ? -INFINITY : (m[i] + log2f(l[i])) * 0.69314718056f;
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
        for (int i = tid; i < s.N; i += kThreads) walk.bad |= attn_request(s, i).bad != 0;
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
    // Measured, ranges against whole items, us: 2 prompts of 256 tokens x 8 heads 33/73, 8 x 16 heads
    // 121/144, 32 x 16 heads 396/407, 4 of 2048 x 32 heads 3790/3770; of 128 tokens 2 x 8 heads 32/41, but
    // 16 x 16 heads 93/81.
    if (a.max_q > 2 * kKeys && (long long)a.total_q / C::ROWS * a.Hq < 16LL * nsm) {
        p.sp.ctas = nsm;
        p.sp.least = kKeys;
        p.sp.rows = std::min((a.max_q + 3) & ~3, C::ROWS);  // whole 16-byte vectors
        if (a.ws && a.ws_bytes >= attn_split_bytes(p.sp, kD)) p.sp.ws = a.ws;
    }
    // Whole items: a CTA for each, which evens out long ones, or one per SM, which walks over the
    // requests once instead of for every item. Measured, a CTA an item against one per SM, us: 8
    // prompts of 2048 x 32 heads 7500/7730, 40 of 100 .. 1000 x 32 4570/4860, 64 of 128 x 32 565/564; 200
    // of 1 .. 128 x 16 719/694, 256 of 33 x 32 919/695, 1000 of 128 x 8 3250/2110, 4864 of 64 x 2 6710/916.
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
    // prompts of 64 tokens x 16 heads 110/167, 64 of 128 270/286, 16 of 200 x 8 heads 112/119, 16 of 300
    // 160/205; 8 of 512 x 16 heads 344/329, 4 of 2048 x 32 heads 4460/3790.
    if (a.max_q <= 384) return a.dr ? launch_t<64, 4>(a) : launch_t<0, 4>(a);
    return a.dr ? launch_t<64, 8>(a) : launch_t<0, 8>(a);
}

}  // namespace kda
