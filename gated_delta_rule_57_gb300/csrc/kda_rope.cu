// Rotation by position on the way to a paged cache: queries and keys rotated, keys and
// values written to their slots (kda_kv_append_rope), or a token's latent and its
// rotated key part (kda_latent_append). One kernel.
//
//     (a, b) -> (a cos t - b sin t, a sin t + b cos t),   t = position * frequency
//
// Angles. A frequency is held in turns a token, as a 64-bit fraction f / 2^64: the
// product position * f modulo 2^64 is then exact at any position, and no 64-bit floating
// point is needed (a rate of 1/64 here). The nearest quarter turn is taken off in whole numbers
// and turned back by signs and an exchange, so that what is rounded to fp32 is an eighth of a turn
// at most, to 2^-34: cos and sin are off by less than 3.1 x 2^-24 of themselves and 4e-10, near
// their zeros too. (A fraction of half a turn rounded to fp32 is off by 9.4e-8 rad. 65536 latents
// below take 115.5 us, 114.8 so, and 116.6 with all bits of the eighth, by a 64-bit conversion.)
//
// A token's angles are turned into cos and sin once (rot / 2 pairs, a thread each) and
// kept in shared memory for all its heads, while the token's first loads are on their
// way. The token's work is laid out as items of two 16-byte vectors, a few for each of its
// threads (with one vector where pairs are neighbours, the latents below took 180 us).
//
// Bound by HBM: every byte is read and written once. Measured in bf16, calls one after another from a
// graph, with outputs made beforehand: 65536 tokens of 32 query and 8 key heads of 128 channels 237 us,
// 6.8 TB/s; 65536 latents with 32 query heads, expanded, 115 us, 6.0 TB/s; 256 tokens 3.1 and 2.7 us, the
// latency of a launch, a load, the angles and a store.
#include "kda_host.cuh"
#include "kda_internal.cuh"

namespace kda {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeBatch = 4;   // items in flight per thread
constexpr int kRopeMaxRot = 128;

// Heads of a tensor: token t, head h starts at ptr + t * tok + h * head (in vectors).
struct RopeHeads {
    uint4* p;
    long long tok, head;
};
struct RopeParams {
    RopeHeads q, q_out, k, k_out, v;  // k_out: may be null
    uint4* k_cache;
    uint4* v_cache;
    // Slot (page, offset), head h of the caches starts at page * c_page + h * c_head +
    // offset * c_row (+ k_at for keys), in vectors.
    long long c_page, c_head, c_row, k_at;
    const int* slot;
    const int* pos;
    const long long* turns;
    int T, Hq, Hk, Hv;
    int v_vec, v_half;     // vectors of a head of v; half of those of all its heads
    int pairs;             // rot / 2
    int turned, items;     // items of a head of q or k: turned ones, all
    uint32_t items_magic, v_magic;  // of the divisions by items and v_vec
    int neighbours;        // pairs are neighbours, not halves
    int tpt_log2;          // threads of a token
    long long slots;
    int page;
    int* d_status;
};

// x / n for x * n < 2^32, magic = ceil(2^32 / n) (0: n is 1).
__device__ __forceinline__ int divide(int x, uint32_t magic) {
    return magic ? (int)__umulhi((uint32_t)x, magic) : x;
}
uint32_t magic_of(int n) { return n <= 1 ? 0u : (uint32_t)(((1ull << 32) + n - 1) / n); }

template <typename T>
struct Vec {
    static constexpr int N = 16 / sizeof(T);
    float x[N];
    __device__ explicit Vec(uint4 u) {
        if constexpr (N == 4) {
            x[0] = __uint_as_float(u.x);
            x[1] = __uint_as_float(u.y);
            x[2] = __uint_as_float(u.z);
            x[3] = __uint_as_float(u.w);
        } else {
            const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int i = 0; i < 4; i++) {
                x[2 * i] = __uint_as_float(w[i] << 16);
                x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
            }
        }
    }
    __device__ uint4 pack() const {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; i++) {
            if constexpr (N == 4) {
                w[i] = __float_as_uint(x[i]);
            } else {
                const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
                w[i] = *reinterpret_cast<const uint32_t*>(&b);
            }
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};

// HALVES: a pair's channels are rot / 2 apart, else neighbours.
template <typename T, bool HALVES>
__global__ void __launch_bounds__(kRopeThreads, 4) kda_rope_kernel(const RopeParams p) {
    constexpr int N = Vec<T>::N;
    // cos and sin of the tokens' pairs (a token has at least 32 threads), an item's N in the
    // order of its use: two pairs a vector, vector c of item i at c * turned + i, so that
    // neighbouring lanes read neighbouring vectors.
    __shared__ float4 s_cs[kRopeThreads / 32][kRopeMaxRot / 4];
    pdl_wait();
    const int tpt = 1 << p.tpt_log2;
    const int sub = threadIdx.x >> p.tpt_log2, i0 = threadIdx.x & (tpt - 1);
    const long long t64 = (long long)blockIdx.x * (kRopeThreads >> p.tpt_log2) + sub;
    const bool live = t64 < p.T;
    const int t = live ? (int)t64 : 0;
    const int slot = p.slot[t];
    const int half = p.turned;  // vectors of half of a head's turned channels
    // Items 0 .. nqk - 1: of queries and keys, a head after the other. A turned one i of a
    // head has vectors i and i + half, the others copy one vector. Then values, vectors i and
    // i + v_half.
    const int nqk = (p.Hq + p.Hk) * p.items, n = live ? nqk + p.v_half : 0;
    uint4 a[kRopeBatch], b[kRopeBatch];
    auto load = [&](int e0) {
#pragma unroll
        for (int j = 0; j < kRopeBatch; j++) {
            const int e = e0 + j * tpt;
            if (e < nqk) {
                const int h = divide(e, p.items_magic), i = e - h * p.items;
                const uint4* src = h >= p.Hq ? p.k.p + t * p.k.tok + (h - p.Hq) * p.k.head
                                             : p.q.p + t * p.q.tok + h * p.q.head;
                src += i < p.turned ? i : i + half;  // (what is copied follows both halves)
                a[j] = __ldcs(src);
                if (i < p.turned) b[j] = __ldcs(src + half);
            } else if (e < n) {
                const uint4* src = p.v.p + t * p.v.tok + (e - nqk);
                a[j] = __ldcs(src);
                b[j] = __ldcs(src + p.v_half);
            }
        }
    };
    load(live ? i0 : n);
    if (p.pairs > 0) {  // while they are on their way
        const unsigned long long pos = (unsigned long long)(long long)p.pos[t];
        for (int i = i0; i < p.pairs; i += tpt) {
            const unsigned long long turn = pos * (unsigned long long)p.turns[i];
            const uint32_t rest = (uint32_t)(turn >> 30);  // signed: less the nearest quarter
            const uint32_t quarter = (uint32_t)(turn >> 62) + (rest >> 31);
            float s, c;
            sincospif((float)(int)rest * 0x1p-33f, &s, &c);
            if (quarter & 1) {
                const float x = c;
                c = -s;
                s = x;
            }
            if (quarter & 2) c = -c, s = -s;
            int u = i / N, w = i % N;
            if (!HALVES) {  // pair i is in vector i / (N / 2)
                u = i / (N / 2);
                w = i % (N / 2) + (u < half ? 0 : N / 2);
                u -= u < half ? 0 : half;
            }
            reinterpret_cast<float2*>(&s_cs[sub][(w >> 1) * p.turned + u])[w & 1] = make_float2(c, s);
        }
        __syncthreads();
    }
    const bool stored = live && slot >= 0 && slot < p.slots;
    const int id = stored ? slot / p.page : 0, off = stored ? slot - id * p.page : 0;
    const long long at = id * p.c_page + off * p.c_row;
    for (int e0 = i0; e0 < n;) {
#pragma unroll
        for (int j = 0; j < kRopeBatch; j++) {
            const int e = e0 + j * tpt;
            if (e >= n) continue;
            if (e >= nqk) {
                if (!stored) continue;
                int v = e - nqk, h = divide(v, p.v_magic);
                p.v_cache[at + h * p.c_head + (v - h * p.v_vec)] = a[j];
                v += p.v_half;
                h = divide(v, p.v_magic);
                p.v_cache[at + h * p.c_head + (v - h * p.v_vec)] = b[j];
                continue;
            }
            const int h = divide(e, p.items_magic), i = e - h * p.items;
            const bool turned = i < p.turned;
            if (turned) {
                const float4* cs = &s_cs[sub][i];
                Vec<T> u(a[j]), w(b[j]);
#pragma unroll
                for (int c = 0; c < N; c += 2) {
                    const float4 x = cs[(c >> 1) * p.turned];
                    // two pairs: of channels c and c + 1 of both vectors, or four of one of them
                    float* y = c < N / 2 ? u.x + 2 * c : w.x + 2 * c - N;
                    float& a0 = HALVES ? u.x[c] : y[0];
                    float& b0 = HALVES ? w.x[c] : y[1];
                    float& a1 = HALVES ? u.x[c + 1] : y[2];
                    float& b1 = HALVES ? w.x[c + 1] : y[3];
                    const float c0 = a0, c1 = a1;
                    a0 = c0 * x.x - b0 * x.y;
                    b0 = c0 * x.y + b0 * x.x;
                    a1 = c1 * x.z - b1 * x.w;
                    b1 = c1 * x.w + b1 * x.z;
                }
                a[j] = u.pack();
                b[j] = w.pack();
            }
            auto put = [&](uint4* dst) {
                dst += turned ? i : i + half;
                *dst = a[j];
                if (turned) dst[half] = b[j];
            };
            if (h < p.Hq) {
                put(p.q_out.p + t * p.q_out.tok + h * p.q_out.head);
            } else {
                if (stored) put(p.k_cache + at + (h - p.Hq) * p.c_head + p.k_at);
                if (p.k_out.p) put(p.k_out.p + t * p.k_out.tok + (h - p.Hq) * p.k_out.head);
            }
        }
        e0 += tpt * kRopeBatch;
        load(e0);
    }
    report_flags(p.d_status, live && slot >= p.slots ? KDA_DEV_PAGES : 0);
}

// Rows of one tensor: row t starts at p + t * stride bytes and has `row` bytes.
struct Rows {
    const void* p;
    size_t row, stride;
    int n;
    size_t span() const { return n > 0 ? (n - 1) * stride + row : 0; }
};
// Do any of the rows of a and b overlap? Exact where the strides agree (views of one
// projection); else true where their spans meet.
bool rows_meet(const Rows& a, const Rows& b) {
    if (!overlaps(a.p, a.span(), b.p, b.span())) return false;
    if (a.stride != b.stride || a.row > a.stride || b.row > b.stride) return true;
    const long long d = (long long)reinterpret_cast<uintptr_t>(b.p) - (long long)reinterpret_cast<uintptr_t>(a.p);
    const long long s = (long long)a.stride, m = ((d % s) + s) % s;
    return m < (long long)a.row || m + (long long)b.row > s;
}

cudaError_t launch_rope(RopeParams& p, kda_dtype_t io, cudaStream_t stream) {
    p.v_half = p.Hv * p.v_vec / 2;  // (v_vec is even)
    const int work = (p.Hq + p.Hk) * p.items + p.v_half;
    // Threads of a token: as few as two batches of items each allow, and more while the
    // call has too few tokens for two CTAs an SM. Measured as above with 32, 64, 128, 256, us: 65536 tokens
    // of 32 + 8 + 8 heads 238/236/240/318, of 8 + 1 + 1 heads 68/89/132/223, latents with 32 query heads
    // 115/131/174/244 (absorbed 115/130/173/242); 256 tokens 6.6/4.3/3.2/3.2, 3.6/2.9/2.7/2.6,
    // 4.4/3.4/3.1/2.7.
    int dev = 0;
    const long long fill = 2LL * device_sms(&dev) * kRopeThreads;
    p.tpt_log2 = 5;
    while (p.tpt_log2 < 8 && ((work >> p.tpt_log2) > 2 * kRopeBatch || ((long long)p.T << p.tpt_log2) < fill)) p.tpt_log2++;
    p.items_magic = magic_of(p.items);
    p.v_magic = magic_of(p.v_vec);
    const int per = kRopeThreads >> p.tpt_log2;
    const dim3 grid((unsigned)((p.T + per - 1) / per));
    auto kernel = io == KDA_BF16
                      ? (p.neighbours ? kda_rope_kernel<__nv_bfloat16, false> : kda_rope_kernel<__nv_bfloat16, true>)
                      : (p.neighbours ? kda_rope_kernel<float, false> : kda_rope_kernel<float, true>);
    return launch_dependent(kernel, grid, dim3(kRopeThreads), 0, stream, p);
}

// Items of a head of d channels of which the first rot are turned; V channels a vector.
void head_items(RopeParams* p, int d, int rot, int neighbours, int V) {
    p->pairs = rot / 2;
    p->neighbours = neighbours != 0;
    p->turned = rot / 2 / V;
    p->items = p->turned + (d - rot) / V;
}

kda_status_t check_stride(long long s, long long least, size_t esz, long long most = 1LL << 30) {
    if (s < least || s > most) return fail(KDA_ERR_INVALID_ARG, "a stride is too small or too large");
    if (s * (long long)esz % 16) return fail(KDA_ERR_INVALID_ARG, "strides must be 16-byte multiples");
    return KDA_OK;
}

}  // namespace
}  // namespace kda

using namespace kda;

extern "C" {

kda_status_t kda_kv_append_rope(const void* q, const void* k, const void* v, const int* slot_map,
                                const int* positions, const long long* turns, void* k_cache,
                                void* v_cache, void* q_out, void* k_out, int T, int Hq, int Hkv, int d,
                                int rot, int neighbours, long long q_stride, long long k_stride,
                                long long v_stride, long long q_out_stride, long long k_out_stride,
                                int num_pages, int page_size, kda_dtype_t io, int* d_status,
                                void* stream) {
    NvtxRange nvtx_range("kda_kv_append_rope");
    if (T < 0 || Hq < 0 || Hkv < 0 || num_pages < 0 || page_size < 1)
        return fail(KDA_ERR_INVALID_ARG, "T, Hq, Hkv and num_pages must be >= 0, page_size positive");
    if (io != KDA_BF16 && io != KDA_F32) return fail(KDA_ERR_INVALID_ARG, "unknown io dtype");
    if (d != 64 && d != 128) return fail(KDA_ERR_UNSUPPORTED, "d must be 64 or 128");
    if (rot < 16 || rot > d || rot % 16)
        return fail(KDA_ERR_UNSUPPORTED, "rot must be a multiple of 16 in 16 .. d");
    if (T > (1 << 30)) return fail(KDA_ERR_INVALID_ARG, "T must be at most 2^30");
    if (Hq > (1 << 16) || Hkv > (1 << 16)) return fail(KDA_ERR_INVALID_ARG, "at most 65536 heads");
    if ((long long)num_pages * page_size >= (1LL << 31))
        return fail(KDA_ERR_INVALID_ARG, "num_pages * page_size must be below 2^31");
    if (T == 0 || (Hq == 0 && Hkv == 0)) return KDA_OK;
    const size_t esz = io == KDA_BF16 ? 2 : 4;
    if ((Hq > 0 && (!q || !q_out)) || (Hkv > 0 && (!k || !v || ((!k_cache || !v_cache) && num_pages > 0))) ||
        !slot_map || !positions || !turns)
        return fail(KDA_ERR_INVALID_ARG, "a NULL pointer");
    for (const void* x : {q, k, v, (const void*)k_cache, (const void*)v_cache, (const void*)q_out, (const void*)k_out})
        if (!aligned16(x)) return fail(KDA_ERR_INVALID_ARG, "pointers must be 16-byte aligned");
    if (reinterpret_cast<uintptr_t>(turns) & 7u)
        return fail(KDA_ERR_INVALID_ARG, "turns must be 8-byte aligned");
    if (!aligned4(slot_map) || !aligned4(positions) || !aligned4(d_status))
        return fail(KDA_ERR_INVALID_ARG, "slot_map, positions and d_status must be 4-byte aligned");
    const size_t rq = (size_t)Hq * d * esz, rk = (size_t)Hkv * d * esz;
    kda_status_t st = KDA_OK;
    if (Hq > 0)
        for (long long s : {q_stride, q_out_stride})
            if ((st = check_stride(s, (long long)Hq * d, esz)) != KDA_OK) return st;
    if (Hkv > 0)
        for (long long s : {k_stride, v_stride})
            if ((st = check_stride(s, (long long)Hkv * d, esz)) != KDA_OK) return st;
    if (k_out && (st = check_stride(k_out_stride, (long long)Hkv * d, esz)) != KDA_OK) return st;
    size_t n_c;
    if (!mul_ok(&n_c, num_pages, page_size, (size_t)Hkv * d, esz))
        return fail(KDA_ERR_INVALID_ARG, "tensor size overflow");
    const size_t t4 = (size_t)T * 4;
    const Rows in_q{q, rq, q_stride * esz, Hq ? T : 0}, in_k{k, rk, k_stride * esz, Hkv ? T : 0},
        in_v{v, rk, v_stride * esz, Hkv ? T : 0}, s{slot_map, t4, t4, 1}, ps{positions, t4, t4, 1},
        tn{turns, (size_t)rot * 4, (size_t)rot * 4, 1};
    const Rows kc{k_cache, n_c, n_c, 1}, vc{v_cache, n_c, n_c, 1},
        qo{q_out, rq, q_out_stride * esz, Hq ? T : 0}, ko{k_out, rk, k_out_stride * esz, k_out && Hkv ? T : 0};
    const bool q_in_place = q == q_out && q_stride == q_out_stride;
    const bool k_in_place = k == k_out && k_stride == k_out_stride;
    bool meet = (!q_in_place && rows_meet(qo, in_q)) || (!k_in_place && rows_meet(ko, in_k));
    meet |= rows_meet(qo, in_k) || rows_meet(ko, in_q);
    for (const Rows& o : {kc, vc})
        for (const Rows& x : {in_q, in_k}) meet |= rows_meet(o, x);
    for (const Rows& o : {kc, vc, qo, ko})
        for (const Rows& x : {in_v, s, ps, tn}) meet |= rows_meet(o, x);
    if (meet) return fail(KDA_ERR_INVALID_ARG, "a cache, q_out or k_out overlaps an input");
    if (rows_meet(kc, vc) || rows_meet(kc, qo) || rows_meet(vc, qo) || rows_meet(kc, ko) || rows_meet(vc, ko) ||
        rows_meet(qo, ko))
        return fail(KDA_ERR_INVALID_ARG, "the caches, q_out and k_out overlap");
    const int V = (int)(16 / esz), dv = d / V;
    RopeParams p{};
    p.q = {static_cast<uint4*>(const_cast<void*>(q)), q_stride / V, dv};
    p.q_out = {static_cast<uint4*>(q_out), q_out_stride / V, dv};
    p.k = {static_cast<uint4*>(const_cast<void*>(k)), k_stride / V, dv};
    p.k_out = {static_cast<uint4*>(k_out), k_out_stride / V, dv};
    p.v = {static_cast<uint4*>(const_cast<void*>(v)), v_stride / V, dv};
    p.k_cache = static_cast<uint4*>(k_cache);
    p.v_cache = static_cast<uint4*>(v_cache);
    p.c_row = dv;
    p.c_head = (long long)page_size * dv;
    p.c_page = (long long)Hkv * p.c_head;
    p.slot = slot_map;
    p.pos = positions;
    p.turns = turns;
    p.T = T;
    p.Hq = Hq;
    p.Hk = p.Hv = Hkv;
    p.v_vec = dv;
    head_items(&p, d, rot, neighbours, V);
    p.slots = (long long)num_pages * page_size;
    p.page = page_size;
    p.d_status = d_status;
    return launched(launch_rope(p, io, static_cast<cudaStream_t>(stream)));
}

kda_status_t kda_latent_append(const void* c, const void* k_r, const void* q_r, const int* slot_map,
                               const int* positions, const long long* turns, void* cache,
                               void* q_out, void* k_out, int T, int Hq, int dl, int dr,
                               int neighbours, long long c_stride, long long kr_stride,
                               long long qr_stride, long long qr_head, long long q_out_stride,
                               long long q_out_head, long long k_out_stride, int num_pages,
                               int page_size, kda_dtype_t io, int* d_status, void* stream) {
    NvtxRange nvtx_range("kda_latent_append");
    if (T < 0 || Hq < 0 || num_pages < 0 || page_size < 1)
        return fail(KDA_ERR_INVALID_ARG, "T, Hq and num_pages must be >= 0, page_size positive");
    if (io != KDA_BF16 && io != KDA_F32) return fail(KDA_ERR_INVALID_ARG, "unknown io dtype");
    if (dl != 512) return fail(KDA_ERR_UNSUPPORTED, "the latent must have 512 channels");
    if (dr != 0 && dr != 64) return fail(KDA_ERR_UNSUPPORTED, "dr must be 0 or 64");
    if (T > (1 << 30)) return fail(KDA_ERR_INVALID_ARG, "T must be at most 2^30");
    if (Hq > (1 << 16)) return fail(KDA_ERR_INVALID_ARG, "at most 65536 heads");
    if ((long long)num_pages * page_size >= (1LL << 31))
        return fail(KDA_ERR_INVALID_ARG, "num_pages * page_size must be below 2^31");
    if (dr == 0 && (Hq != 0 || k_out))
        return fail(KDA_ERR_INVALID_ARG, "without a rotated part there are no q_r and k_out");
    if (T == 0) return KDA_OK;
    const size_t esz = io == KDA_BF16 ? 2 : 4;
    if (!c || !slot_map || (!cache && num_pages > 0) || (dr > 0 && (!k_r || !positions || !turns)) ||
        (Hq > 0 && (!q_r || !q_out)))
        return fail(KDA_ERR_INVALID_ARG, "a NULL pointer");
    for (const void* x : {c, dr ? k_r : nullptr, Hq ? q_r : nullptr, (const void*)cache,
                          Hq ? (const void*)q_out : nullptr, (const void*)k_out})
        if (!aligned16(x)) return fail(KDA_ERR_INVALID_ARG, "pointers must be 16-byte aligned");
    if (dr && (reinterpret_cast<uintptr_t>(turns) & 7u))
        return fail(KDA_ERR_INVALID_ARG, "turns must be 8-byte aligned");
    if (!aligned4(slot_map) || (dr && !aligned4(positions)) || !aligned4(d_status))
        return fail(KDA_ERR_INVALID_ARG, "slot_map, positions and d_status must be 4-byte aligned");
    kda_status_t st = check_stride(c_stride, dl, esz);
    if (st == KDA_OK && dr) st = check_stride(kr_stride, dr, esz);
    if (st == KDA_OK && k_out) st = check_stride(k_out_stride, dr, esz);
    if (st != KDA_OK) return st;
    if (Hq > 0)
        for (int i = 0; i < 2; i++) {
            const long long head = i ? q_out_head : qr_head, tok = i ? q_out_stride : qr_stride;
            if ((st = check_stride(head, dr, esz, 1LL << 40)) != KDA_OK) return st;
            if ((st = check_stride(tok, dr, esz)) != KDA_OK) return st;
            if (tok < (Hq - 1) * head + dr && head < (T - 1) * tok + dr)
                return fail(KDA_ERR_INVALID_ARG, "heads and tokens of q_r or q_out overlap");
        }
    size_t n_c;
    if (!mul_ok(&n_c, num_pages, page_size, (size_t)(dl + dr), esz))
        return fail(KDA_ERR_INVALID_ARG, "tensor size overflow");
    const size_t t4 = (size_t)T * 4, nr = dr * esz;
    auto heads = [&](const void* p, long long tok, long long head) {
        const size_t row = Hq ? ((Hq - 1) * head + dr) * esz : 0;
        if (tok * esz >= row) return Rows{p, row, tok * esz, Hq ? T : 0};
        const size_t all = row + (T - 1) * tok * esz;  // tokens inside heads
        return Rows{p, all, all, 1};
    };
    const Rows in_c{c, dl * esz, c_stride * esz, T}, in_k{k_r, nr, kr_stride * esz, dr ? T : 0},
        in_q = heads(q_r, qr_stride, qr_head), s{slot_map, t4, t4, 1}, ps{positions, t4, t4, dr ? 1 : 0},
        tn{turns, (size_t)dr * 4, (size_t)dr * 4, dr ? 1 : 0};
    const Rows cc{cache, n_c, n_c, 1}, qo = heads(q_out, q_out_stride, q_out_head),
        ko{k_out, nr, k_out_stride * esz, k_out ? T : 0};
    const bool q_in_place = q_r == q_out && qr_stride == q_out_stride && qr_head == q_out_head;
    const bool k_in_place = k_r == k_out && kr_stride == k_out_stride;
    bool meet = !q_in_place && rows_meet(qo, in_q);
    meet |= !k_in_place && rows_meet(ko, in_k);
    meet |= rows_meet(cc, in_q) || rows_meet(cc, in_k) || rows_meet(qo, in_k) || rows_meet(ko, in_q);
    for (const Rows& o : {cc, qo, ko})
        for (const Rows& x : {in_c, s, ps, tn}) meet |= rows_meet(o, x);
    if (meet) return fail(KDA_ERR_INVALID_ARG, "the cache, q_out or k_out overlaps an input");
    if (rows_meet(cc, qo) || rows_meet(cc, ko) || rows_meet(qo, ko))
        return fail(KDA_ERR_INVALID_ARG, "the cache, q_out and k_out overlap");
    const int V = (int)(16 / esz);
    RopeParams p{};
    p.q = {static_cast<uint4*>(const_cast<void*>(q_r)), qr_stride / V, qr_head / V};
    p.q_out = {static_cast<uint4*>(q_out), q_out_stride / V, q_out_head / V};
    p.k = {static_cast<uint4*>(const_cast<void*>(k_r)), kr_stride / V, 0};
    p.k_out = {static_cast<uint4*>(k_out), k_out_stride / V, 0};
    p.v = {static_cast<uint4*>(const_cast<void*>(c)), c_stride / V, 0};
    p.k_cache = p.v_cache = static_cast<uint4*>(cache);
    p.c_row = (dl + dr) / V;
    p.c_page = (long long)page_size * p.c_row;
    p.k_at = dl / V;
    p.slot = slot_map;
    p.pos = positions;
    p.turns = turns;
    p.T = T;
    p.Hq = Hq;
    p.Hk = dr ? 1 : 0;
    p.Hv = 1;
    p.v_vec = dl / V;
    head_items(&p, dr, dr, neighbours, V);
    p.slots = (long long)num_pages * page_size;
    p.page = page_size;
    p.d_status = d_status;
    return launched(launch_rope(p, io, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
