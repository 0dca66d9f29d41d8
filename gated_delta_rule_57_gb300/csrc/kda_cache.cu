// Paged key/value cache of the softmax-attention layers: the plan of a step
// (block tables, slot map and free list from request lengths) and the write of
// new keys and values to their slots. Kernels and entry points.
#include <algorithm>
#include <atomic>

#include "kda_host.cuh"
#include "kda_internal.cuh"

namespace kda {
namespace {

// ---------------------------------------------------------------------------
// Plan. Request r goes from a = old[r] to b = new[r] tokens and from
// held = ceil(a / page) to want = ceil(b / page) pages. With
//   T(r) = sum_{i < r} max(b_i - a_i, 0)        tokens before r
//   G(r) = sum_{i < r} max(want_i - held_i, 0)  pages taken before r
//   F(r) = sum_{i < r} max(held_i - want_i, 0)  pages given back before r
// its j-th page is ring[head + G(r) + j - held], its pages from want on go to
// ring[head + count + F(r) + ...], and its new token i has slot
// table[r][(a + i) / page] * page + (a + i) % page. The free pages are a ring,
// so what is taken and what is given back never share an entry and no order
// among threads is needed: one launch. Every CTA scans all lengths itself
// (N ints from L2 and two block scans, about 1 us) rather than wait for another
// launch to do it, then takes its share of the tokens and pages, each found by
// a binary search in the prefix sums in shared memory.
// Bound by latency (the bytes of the larger step are 0.3 us of HBM time): 4.0 us for 256
// requests that gain a token each, 10.9 us for 2048 mixed ones with 253 k new tokens (2048
// that gain a token each: 9.6 us, so it is the scans and their loads, not the tokens).
// ---------------------------------------------------------------------------
constexpr int kPlanThreads = 512;
constexpr int kPlanMaxN = 16384;           // three prefix arrays in shared memory
constexpr unsigned kLenCap = 1u << 30;     // lengths and sums saturate here

__device__ __forceinline__ unsigned sat_add(unsigned a, unsigned b) {
    const unsigned s = a + b;  // both at most 2^30
    return s < kLenCap ? s : kLenCap;
}

// Exclusive saturating scan over the block of one value per thread; `total`
// gets the sum. s_warp: one word per warp.
__device__ __forceinline__ unsigned block_scan(unsigned x, unsigned* s_warp, unsigned* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    unsigned inc = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const unsigned y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc = sat_add(inc, y);
    }
    __syncthreads();  // s_warp of the scan before is read
    if (lane == 31) s_warp[warp] = inc;
    __syncthreads();
    unsigned before = 0, sum = 0;
#pragma unroll
    for (int w = 0; w < kPlanThreads / 32; w++) {
        if (w == warp) before = sum;
        sum = sat_add(sum, s_warp[w]);
    }
    *total = sum;
    unsigned ex = __shfl_up_sync(0xffffffffu, inc, 1);
    if (lane == 0) ex = 0;
    return sat_add(before, ex);
}

// Largest r in [0, n) with pre[r] <= x (pre[0] = 0, non-decreasing).
__device__ __forceinline__ int find(const unsigned* pre, int n, unsigned x) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (pre[mid] <= x) lo = mid;
        else hi = mid;
    }
    return lo;
}

struct PlanParams {
    const int* old_len;
    const int* new_len;
    int* table;
    int* ring;
    const int* ring_in;
    int* ring_out;
    int* kv_len;
    int* cu;
    int* slot;
    int N, max_pages, num_pages, page, max_tokens;
    int* d_status;
};

// EACH: requests of a thread in a round of kPlanThreads * EACH; a call of one round holds
// their lengths in registers for both passes (2048 requests: 10.9 us against 13.0 us when
// each pass reads them again), a call of several reads them twice. Rounds of 8 a thread:
// 2049 requests 10.9 us, 8192 27.0, 16384 46.0; one round of 32 a thread, whose lengths
// do not fit the registers, 54.2, 81.2 and 123.
template <int EACH>
__global__ void __launch_bounds__(kPlanThreads) kda_kv_plan_kernel(const PlanParams p) {
    extern __shared__ unsigned s_pre[];
    unsigned* s_tok = s_pre;
    unsigned* s_take = s_tok + p.N + 1;
    unsigned* s_back = s_take + p.N + 1;
    __shared__ unsigned s_warp[kPlanThreads / 32];
    __shared__ unsigned s_taken;

    pdl_wait();
    const int tid = threadIdx.x, N = p.N;
    const unsigned page = p.page, P = p.num_pages;
    int flags = 0;
    int h = p.ring_in[0], c = p.ring_in[1];
    if (h < 0 || h >= (int)P || c < 0 || c > (int)P) {
        flags |= KDA_DEV_PAGES;
        h = h < 0 ? 0 : h % (int)P;
        c = c < 0 ? 0 : ((unsigned)c > P ? (int)P : c);
    }
    const unsigned head = h, count = c;
    auto length = [&](const int* len, int r) {
        const int x = len[r];
        if (x < 0 || x > (int)kLenCap) flags |= KDA_DEV_LENGTH;
        return x < 0 ? 0u : min((unsigned)x, kLenCap);
    };
    auto pages = [&](unsigned x) { return (x + page - 1) / page; };
    // Taken only where the table's row holds them.
    auto takes = [&](unsigned held, unsigned want) {
        return want > held && want <= (unsigned)p.max_pages ? want - held : 0u;
    };
    // Left as it was: its row is too short, or (a prefix property, so every
    // later request that needs as much is refused too) the free pages or the
    // room for tokens run out.
    auto refused = [&](int r, unsigned a, unsigned b, unsigned held, unsigned want) {
        return want > (unsigned)p.max_pages || (want > held && s_take[r + 1] > count) ||
               (b > a && s_tok[r + 1] > (unsigned)p.max_tokens);
    };

    // A round: each thread owns EACH consecutive requests, from r0 on.
    constexpr int kRound = kPlanThreads * EACH;
    unsigned a[EACH], b[EACH], held[EACH], want[EACH];
    auto load = [&](int r0) {
#pragma unroll
        for (int e = 0; e < EACH; e++) {
            a[e] = b[e] = 0;
            if (r0 + e < N) {
                a[e] = length(p.old_len, r0 + e);
                b[e] = length(p.new_len, r0 + e);
            }
        }
#pragma unroll
        for (int e = 0; e < EACH; e++) {
            held[e] = pages(a[e]);
            want[e] = pages(b[e]);
        }
    };
    unsigned tokens = 0, needed = 0, given = 0, sum;  // of the rounds so far
    if (tid == 0) s_taken = 0;
    for (int base = 0; base < N; base += kRound) {
        const int r0 = base + tid * EACH;
        load(r0);
        unsigned tok = 0, take = 0;
#pragma unroll
        for (int e = 0; e < EACH; e++) {
            tok = sat_add(tok, b[e] > a[e] ? b[e] - a[e] : 0u);
            take = sat_add(take, takes(held[e], want[e]));
        }
        tok = sat_add(tokens, block_scan(tok, s_warp, &sum));
        tokens = sat_add(tokens, sum);
        take = sat_add(needed, block_scan(take, s_warp, &sum));
        needed = sat_add(needed, sum);
#pragma unroll
        for (int e = 0; e < EACH; e++) {
            if (r0 + e < N) {
                s_tok[r0 + e] = tok;
                s_take[r0 + e] = take;
            }
            tok = sat_add(tok, b[e] > a[e] ? b[e] - a[e] : 0u);
            take = sat_add(take, takes(held[e], want[e]));
        }
    }
    if (tid == 0) {
        s_tok[N] = tokens;
        s_take[N] = needed;
        if (tokens >= kLenCap) flags |= KDA_DEV_LENGTH;
    }
    __syncthreads();
    for (int base = 0; base < N; base += kRound) {
        const int r0 = base + tid * EACH;
        if (N > kRound) load(r0);
        unsigned gives[EACH], back = 0;
#pragma unroll
        for (int e = 0; e < EACH; e++) {
            const int r = r0 + e;
            gives[e] = 0;
            if (r >= N) continue;
            const bool no = refused(r, a[e], b[e], held[e], want[e]);
            if (no) flags |= KDA_DEV_PAGES;
            else if (want[e] > held[e]) atomicMax(&s_taken, s_take[r + 1]);
            // Entries past the row's end were never pages.
            if (!no && want[e] < held[e] && want[e] < (unsigned)p.max_pages)
                gives[e] = min(held[e], (unsigned)p.max_pages) - want[e];
            back = sat_add(back, gives[e]);
            if (blockIdx.x == 0) {
                p.kv_len[r] = (int)(no ? a[e] : b[e]);
                p.cu[r] = (int)s_tok[r];
            }
        }
        back = sat_add(given, block_scan(back, s_warp, &sum));
        given = sat_add(given, sum);
#pragma unroll
        for (int e = 0; e < EACH; e++) {
            if (r0 + e < N) s_back[r0 + e] = back;
            back = sat_add(back, gives[e]);
        }
    }
    if (tid == 0) s_back[N] = given;
    __syncthreads();
    const unsigned taken = s_taken;
    // More pages given back than the ring has room for: an id was held twice.
    if (given > P - count) {
        flags |= KDA_DEV_PAGES;
        given = P - count;
    }
    if (blockIdx.x == 0 && tid == 0) {
        p.cu[N] = (int)tokens;
        p.ring_out[0] = (int)((head + taken) % P);
        p.ring_out[1] = (int)(count - taken + given);
    }

    const unsigned after = head + count < P ? head + count : head + count - P;  // the ring's end
    const unsigned first = blockIdx.x * kPlanThreads + tid, step = gridDim.x * kPlanThreads;
    for (unsigned t = first; t < (unsigned)p.max_tokens; t += step) {
        int slot = -1;
        if (t < tokens) {
            const int r = find(s_tok, N, t);
            const unsigned a = length(p.old_len, r), b = a + (s_tok[r + 1] - s_tok[r]);
            const unsigned held = pages(a), want = pages(b);
            if (!refused(r, a, b, held, want)) {
                const unsigned at = a + t - s_tok[r], j = at / page;
                const int id = j < held ? p.table[(size_t)r * p.max_pages + j]
                                        : p.ring[(head + s_take[r] + j - held) % P];
                if (id >= 0 && id < (int)P) slot = id * (int)page + (int)(at % page);
                else flags |= KDA_DEV_PAGES;
            }
        }
        p.slot[t] = slot;
    }
    for (unsigned i = first; i < taken; i += step) {
        const int r = find(s_take, N, i);
        p.table[(size_t)r * p.max_pages + pages(length(p.old_len, r)) + i - s_take[r]] =
            p.ring[(head + i) % P];
    }
    for (unsigned i = first; i < given; i += step) {
        const int r = find(s_back, N, i);
        p.ring[(after + i) % P] =
            p.table[(size_t)r * p.max_pages + pages(length(p.new_len, r)) + i - s_back[r]];
    }
    report_flags(p.d_status, flags);
}

// ---------------------------------------------------------------------------
// Append. A warp takes one token: its keys and values of all heads are two
// contiguous rows, read with 16-byte loads and written as one d-row per head.
// Bound by HBM (every byte is read once and written once): 65536 tokens of 8 x 128
// bf16 in 79.3 us, 6.77 TB/s; 256 tokens in 2.1 us.
// ---------------------------------------------------------------------------
constexpr int kAppendWarps = 8;
constexpr int kAppendBatch = 8;  // 16-byte loads in flight per lane

struct AppendParams {
    const uint4* k;
    const uint4* v;
    const int* slot;
    uint4* kc;
    uint4* vc;
    long long k_stride, v_stride;  // between tokens, in 16-byte vectors
    int T, Hkv, page;
    int vec_log2;                  // log2 of the 16-byte vectors of one head's row
    long long slots;               // num_pages * page
    int* d_status;
};

__global__ void __launch_bounds__(kAppendWarps * 32) kda_kv_append_kernel(const AppendParams p) {
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const int t = blockIdx.x * kAppendWarps + (threadIdx.x >> 5);
    if (t >= p.T) return;
    const int s = p.slot[t];
    const int row = p.Hkv << p.vec_log2;  // vectors of one token's keys
    const uint4* k = p.k + (size_t)t * p.k_stride;
    const uint4* v = p.v + (size_t)t * p.v_stride;
    int flags = 0;
    if (s < 0 || s >= p.slots) {
        if (s >= 0) flags = KDA_DEV_PAGES;
        report_flags(p.d_status, flags);
        return;
    }
    const int id = s / p.page, off = s - id * p.page;
    for (int i0 = lane; i0 < 2 * row; i0 += 32 * kAppendBatch) {
        uint4 x[kAppendBatch];
#pragma unroll
        for (int e = 0; e < kAppendBatch; e++) {
            const int i = i0 + 32 * e;
            if (i < 2 * row) x[e] = __ldcs(i < row ? k + i : v + (i - row));
        }
#pragma unroll
        for (int e = 0; e < kAppendBatch; e++) {
            const int i = i0 + 32 * e;
            if (i < 2 * row) {
                const int j = i < row ? i : i - row, head = j >> p.vec_log2;
                const size_t at = ((size_t)((size_t)id * p.Hkv + head) * p.page + off)
                                  << p.vec_log2;
                (i < row ? p.kc : p.vc)[at + (j & ((1 << p.vec_log2) - 1))] = x[e];
            }
        }
    }
}

}  // namespace
}  // namespace kda

using namespace kda;

extern "C" {

kda_status_t kda_kv_plan(const int* old_len, const int* new_len, int* block_table,
                         int* free_pages, const int* ring_in, int* ring_out, int* kv_len,
                         int* cu_new, int* slot_map, int N, int max_pages, int num_pages,
                         int page_size, int max_tokens, int* d_status, void* stream) {
    NvtxRange nvtx_range("kda_kv_plan");
    if (N < 0 || max_pages < 0 || num_pages < 1 || page_size < 1 || max_tokens < 0)
        return fail(KDA_ERR_INVALID_ARG, "N, max_pages and max_tokens must be >= 0, num_pages and "
                                         "page_size positive");
    if ((long long)num_pages * page_size >= (1LL << 31))
        return fail(KDA_ERR_INVALID_ARG, "num_pages * page_size must be below 2^31");
    if (max_tokens > (int)kLenCap || max_pages > (int)kLenCap)
        return fail(KDA_ERR_INVALID_ARG, "max_tokens and max_pages must be at most 2^30");
    if (N > kPlanMaxN) return fail(KDA_ERR_UNSUPPORTED, "at most 16384 requests");
    const size_t n4 = (size_t)N * 4;
    struct Buf {
        const void* p;
        size_t n;
        bool out;
    };
    const Buf bufs[] = {{old_len, n4, false},
                        {new_len, n4, false},
                        {ring_in, 8, false},
                        {block_table, n4 * max_pages, true},
                        {free_pages, (size_t)num_pages * 4, true},
                        {ring_out, 8, true},
                        {kv_len, n4, true},
                        {cu_new, n4 + 4, true},
                        {slot_map, (size_t)max_tokens * 4, true}};
    for (const Buf& b : bufs) {
        if (b.n && !b.p) return fail(KDA_ERR_INVALID_ARG, "a NULL pointer");
        if (!aligned4(b.p)) return fail(KDA_ERR_INVALID_ARG, "pointers must be 4-byte aligned");
    }
    if (d_status && !aligned4(d_status))
        return fail(KDA_ERR_INVALID_ARG, "d_status must be 4-byte aligned");
    for (const Buf& o : bufs)
        for (const Buf& b : bufs)
            if (o.out && &o != &b && overlaps(o.p, o.n, b.p, b.n))
                return fail(KDA_ERR_INVALID_ARG, "an output overlaps another argument");
    PlanParams p{old_len, new_len, block_table, free_pages, ring_in, ring_out, kv_len, cu_new,
                 slot_map, N, max_pages, num_pages, page_size, max_tokens, d_status};
    const size_t smem = 3 * ((size_t)N + 1) * 4;
    auto kernel = N <= kPlanThreads        ? kda_kv_plan_kernel<1>
                  : N <= 4 * kPlanThreads ? kda_kv_plan_kernel<4>
                                          : kda_kv_plan_kernel<8>;
    int dev = -1;
    const long long most = std::max(device_sms(&dev), 1);
    // Past 48 KB, of which the static part takes some (only the last kernel gets there).
    if (smem > 47 * 1024) {
        static std::atomic<uint64_t> ready{0};
        const cudaError_t e = allow_shared(kernel, 3 * ((size_t)kPlanMaxN + 1) * 4, ready, dev);
        if (e != cudaSuccess) return launched(e);
    }
    // A CTA for 2048 tokens' slots: 253 k tokens took 13.0 us so, as with 512 or
    // 1024, and 18.5 us with 4096; fewer tokens leave the scans, alike for any grid.
    long long grid = ((long long)max_tokens + 4 * kPlanThreads - 1) / (4 * kPlanThreads);
    grid = grid < 1 ? 1 : (grid > most ? most : grid);
    return launched(launch_dependent(kernel, dim3((unsigned)grid), dim3(kPlanThreads),
                                     smem, static_cast<cudaStream_t>(stream), p));
}

kda_status_t kda_kv_append(const void* k, const void* v, const int* slot_map, void* k_cache,
                           void* v_cache, int T, int Hkv, int d, long long k_stride,
                           long long v_stride, int num_pages, int page_size, kda_dtype_t io,
                           int* d_status, void* stream) {
    NvtxRange nvtx_range("kda_kv_append");
    if (T < 0 || Hkv < 0 || num_pages < 0 || page_size < 1)
        return fail(KDA_ERR_INVALID_ARG, "T, Hkv and num_pages must be >= 0, page_size positive");
    if (io != KDA_BF16 && io != KDA_F32) return fail(KDA_ERR_INVALID_ARG, "unknown io dtype");
    if (d != 64 && d != 128) return fail(KDA_ERR_UNSUPPORTED, "d must be 64 or 128");
    if (T > (1 << 30)) return fail(KDA_ERR_INVALID_ARG, "T must be at most 2^30");
    if (Hkv > (1 << 16)) return fail(KDA_ERR_INVALID_ARG, "Hkv must be at most 65536");
    if ((long long)num_pages * page_size >= (1LL << 31))
        return fail(KDA_ERR_INVALID_ARG, "num_pages * page_size must be below 2^31");
    if (T == 0 || Hkv == 0) return KDA_OK;
    const size_t esz = io == KDA_BF16 ? 2 : 4;
    if (!k || !v || !slot_map || ((!k_cache || !v_cache) && num_pages > 0))
        return fail(KDA_ERR_INVALID_ARG, "a NULL pointer");
    for (const void* q : {k, v, (const void*)k_cache, (const void*)v_cache})
        if (!aligned16(q)) return fail(KDA_ERR_INVALID_ARG, "pointers must be 16-byte aligned");
    if (!aligned4(slot_map) || (d_status && !aligned4(d_status)))
        return fail(KDA_ERR_INVALID_ARG, "slot_map and d_status must be 4-byte aligned");
    for (long long s : {k_stride, v_stride}) {
        if (s < (long long)Hkv * d || s > (1LL << 40))
            return fail(KDA_ERR_INVALID_ARG, "token strides must be at least Hkv * d");
        if (s * esz % 16) return fail(KDA_ERR_INVALID_ARG, "token strides must be 16-byte multiples");
    }
    size_t n_c;
    if (!mul_ok(&n_c, num_pages, page_size, (size_t)Hkv * d, esz))
        return fail(KDA_ERR_INVALID_ARG, "tensor size overflow");
    const size_t row = (size_t)Hkv * d;
    const size_t n_k = ((size_t)(T - 1) * k_stride + row) * esz, n_v = ((size_t)(T - 1) * v_stride + row) * esz;
    for (const void* c : {(const void*)k_cache, (const void*)v_cache})
        if (overlaps(c, n_c, k, n_k) || overlaps(c, n_c, v, n_v) ||
            overlaps(c, n_c, slot_map, (size_t)T * 4))
            return fail(KDA_ERR_INVALID_ARG, "a cache overlaps an input");
    if (overlaps(k_cache, n_c, v_cache, n_c))
        return fail(KDA_ERR_INVALID_ARG, "k_cache overlaps v_cache");
    int vec_log2 = 2;
    while ((16u << vec_log2) < d * esz) vec_log2++;
    AppendParams p{static_cast<const uint4*>(k), static_cast<const uint4*>(v), slot_map,
                   static_cast<uint4*>(k_cache), static_cast<uint4*>(v_cache),
                   k_stride * (long long)esz / 16, v_stride * (long long)esz / 16, T, Hkv,
                   page_size, vec_log2, (long long)num_pages * page_size, d_status};
    return launched(launch_dependent(kda_kv_append_kernel,
                                     dim3((unsigned)((T + kAppendWarps - 1) / kAppendWarps)),
                                     dim3(kAppendWarps * 32), 0, static_cast<cudaStream_t>(stream), p));
}

}  // extern "C"
