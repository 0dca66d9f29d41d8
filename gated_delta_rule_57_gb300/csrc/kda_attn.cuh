// Softmax attention over packed prompts and over the paged cache: parameters
// and the division of the work, shared by the kernels.
//
// Rows. The G = Hq / Hkv query heads of a key head read the same keys, so a
// row tile holds (token, head of the group) pairs, token-major: row
// i * G + g of a tile is token i, head h * G + g. A key tile is then read
// once for all of them, and a causal boundary costs G times fewer masked rows.
//
// Items. An item is one row tile (or a pair of them) of one request and one key
// head; it needs the key tiles 0 .. n - 1 of its request, n by the last token
// it holds. Lengths live on the device, so the kernels find their items
// themselves: items are numbered request by request, and a walk over the
// requests (32 at a time, one per lane) turns a number into an item.
//   Whole items: CTA c takes item c; in bf16 the CTAs that run then take over, in
//     order, those that have not started, in fp32 items c + grid, ... Inside a
//     request the longest (last tokens) come first and the key heads run fastest,
//     so concurrent CTAs share the keys of one request in L2 and the short items
//     fill the end.
//   Split items: the key tiles of all items laid end to end are cut into
//     ranges of equal cost, one per CTA, so few rows over a long cache use every
//     SM and ragged lengths balance exactly (a tile belongs to the range that
//     its first unit of cost is in). An item cut by a boundary leaves
//     partial results in the workspace (at most two per CTA) that
//     kda_attn_combine joins.
#pragma once

#include "kda_internal.cuh"

namespace kda {

struct AttnArgs {
    const void* q;
    const void* k;  // packed keys, or the key cache
    const void* v;
    const int* cu_q;         // [N + 1]
    const int* kv_len;       // [N], or null: packed prompts
    const int* block_table;  // [N, max_pages], or null
    void* o;
    float* lse;  // may be null
    int N, total_q, max_q, Hq, Hkv, d;
    long long q_stride, k_stride, v_stride;  // elements between tokens
    int num_pages, page, max_pages;
    float scale;
    float* ws;      // partial results, or null: whole items
    size_t ws_bytes;
    int* d_status;
    cudaStream_t stream;
};

// What the device side needs to divide the work.
struct AttnShape {
    const int* cu_q;
    const int* kv_len;
    int N, total_q, max_q, kv_cap;  // kv_cap: keys of a request, at most
    int Hkv, G;
    int tok1, tok2;  // tokens of an item: tok1 for requests that fit it, else tok2
    int kt;          // keys of a key tile
    int cost1, cost2;  // of a key of either kind of item, in any unit
    int extra;         // keys whose cost an item adds by starting and ending
};

// One request: its packed tokens, keys, and items.
struct AttnReq {
    int q0, q_len, kv;  // first packed token, new tokens, keys
    int tok, nqt;       // tokens per item, items per key head
    int cost;           // of a key
    int bad;            // lengths outside what the call was sized for
};

__device__ __forceinline__ AttnReq attn_request(const AttnShape& s, int r) {
    AttnReq q;
    q.q0 = s.cu_q[r];
    int n = s.cu_q[r + 1] - q.q0;
    q.bad = q.q0 < 0 || n < 0 || n > s.max_q || (long long)q.q0 + n > s.total_q;
    if (q.bad) n = 0;
    q.q_len = n;
    q.kv = n;
    if (s.kv_len) {
        const int x = s.kv_len[r];
        q.kv = min(max(x, 0), s.kv_cap);
        q.bad |= x != q.kv;
    }
    q.tok = n <= s.tok1 ? s.tok1 : s.tok2;
    q.nqt = (n + q.tok - 1) / q.tok;
    q.cost = n <= s.tok1 ? s.cost1 : s.cost2;
    return q;
}

// Keys that the last token of item t of a request sees (0: none).
__device__ __forceinline__ int attn_item_keys(const AttnReq& q, int t) {
    const int last = min((t + 1) * q.tok, q.q_len);
    return max(q.kv - q.q_len + last, 0);
}

// Key tiles of item t of a request, at least one.
__device__ __forceinline__ int attn_item_tiles(const AttnShape& s, const AttnReq& q, int t) {
    return max((attn_item_keys(q, t) + s.kt - 1) / s.kt, 1);
}

// Cost. A key tile costs q.cost kt; item t of a request is counted as
//     q.cost (max(kv - q_len, 0) + (t + 1) tok + kt - 1 + extra),
// its keys rounded up to where its last tile must end and what it costs beside
// them: never less than its tiles', and linear in t, so that the cost before
// an item is a product and not a sum of quotients (those, by Euclid's steps,
// took 1200 clocks each time). Tile k of an item starts at k q.cost kt.
__device__ __forceinline__ long long attn_cost_before(const AttnShape& s, const AttnReq& q, int t) {
    const long long first = (long long)max(q.kv - q.q_len, 0) + s.kt - 1 + s.extra;
    return ((long long)t * first + (long long)q.tok * t * (t + 1) / 2) * q.cost;
}

// A walk over the requests, a warp together, that finds the request of an item
// (or of a unit of cost) of a non-decreasing sequence of numbers.
struct AttnWalk {
    int r0 = 0;          // the 32 requests r0 .. r0 + 31 are looked at
    long long base = 0;  // items (cost) before them
    bool bad = false;    // some request so far had a bad length (lane-wise)
};

// False when there is no item (unit of cost) `idx`. *in: its number in the request.
template <bool COST>
__device__ __forceinline__ bool attn_find(const AttnShape& s, AttnWalk& w, long long idx, int* req,
                                          AttnReq* rq, long long* in) {
    const int lane = threadIdx.x & 31;
    for (; w.r0 < s.N; w.r0 += 32) {
        const int r = w.r0 + lane;
        AttnReq q{};
        if (r < s.N) q = attn_request(s, r);
        w.bad |= q.bad != 0;
        const long long mine =
            (COST ? attn_cost_before(s, q, q.nqt) : q.nqt) * s.Hkv;
        long long inc = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += y;
        }
        const long long total = __shfl_sync(0xffffffffu, inc, 31);
        if (idx < w.base + total) {
            const unsigned m = __ballot_sync(0xffffffffu, idx < w.base + inc);
            const int src = __ffs(m) - 1;
            *req = w.r0 + src;
            rq->q0 = __shfl_sync(0xffffffffu, q.q0, src);
            rq->q_len = __shfl_sync(0xffffffffu, q.q_len, src);
            rq->kv = __shfl_sync(0xffffffffu, q.kv, src);
            rq->tok = __shfl_sync(0xffffffffu, q.tok, src);
            rq->nqt = __shfl_sync(0xffffffffu, q.nqt, src);
            rq->cost = __shfl_sync(0xffffffffu, q.cost, src);
            rq->bad = 0;
            *in = idx - w.base - __shfl_sync(0xffffffffu, inc - mine, src);
            return true;
        }
        w.base += total;
    }
    return false;
}

// a / b, in 32 bits where that does (a quarter of the time).
__device__ __forceinline__ int attn_quotient(long long a, long long b) {
    return (unsigned long long)a < 1ull << 32 && b < 1LL << 32 ? (int)((uint32_t)a / (uint32_t)b) : (int)(a / b);
}

// Split items: the items of a request run key head by key head, row tile by row
// tile. The first key tile that starts at or after `cur`, by a warp together:
// its request, key head, row tile and number in the item. cur moves to its
// start. False when there is none.
__device__ __forceinline__ bool attn_first_tile(const AttnShape& s, AttnWalk& w, long long* cur,
                                                int* r, AttnReq* q, int* h, int* t, int* tile) {
    long long in;
    while (attn_find<true>(s, w, *cur, r, q, &in)) {
        const long long base = *cur - in, per = attn_cost_before(s, *q, q->nqt);
        *h = attn_quotient(in, per);
        const long long rest = in - *h * per;
        // cost_before(lo) <= rest < cost_before(hi); 32 places at a time
        int lo = 0, hi = q->nqt;
        while (hi - lo > 1) {
            const int step = (hi - lo + 31) >> 5, x = lo + (int)(threadIdx.x & 31) * step;
            const bool below = x < hi && attn_cost_before(s, *q, x) <= rest;
            lo += (__popc(__ballot_sync(0xffffffffu, below)) - 1) * step;
            hi = min(lo + step, hi);
        }
        const int each = s.kt * q->cost;
        const long long before = attn_cost_before(s, *q, lo);
        *tile = attn_quotient(rest - before + each - 1, each);
        if (*tile >= attn_item_tiles(s, *q, lo)) {  // the next item's first
            *tile = 0;
            if (++lo == q->nqt) {
                lo = 0;
                ++*h;
            }
        }
        *t = lo;
        *cur = base + *h * per + (*tile ? before + (long long)*tile * each : attn_cost_before(s, *q, lo));
        if (*h < s.Hkv) return true;
    }
    return false;
}
// Tiles of an item of `n` that starts at u0 that start before `end`.
__device__ __forceinline__ int attn_tiles_until(const AttnShape& s, const AttnReq& q, long long u0,
                                                int n, long long end) {
    const int each = s.kt * q.cost;
    const long long room = end - u0;
    return room >= (long long)n * each ? n : attn_quotient(room + each - 1, each);
}

// Sums of the cost of 32 requests each, for a walk to start from.
constexpr int kAttnGroups = 256;

// Cost of a CTA's range, by the whole block: that of all requests over `ctas`, but
// at least `least`. groups[i]: cost of requests 32 i .. 32 i + 31;
// s_sum: one word per warp. The caller synchronises before groups is read.
template <int THREADS>
__device__ __forceinline__ long long attn_cost_each(const AttnShape& s, int ctas, int least,
                                                     long long* groups, long long* s_sum) {
    long long sum = 0;
    for (int r0 = threadIdx.x & ~31; r0 < s.N; r0 += THREADS) {
        const int r = r0 + (threadIdx.x & 31);
        long long mine = 0;
        if (r < s.N) {
            const AttnReq q = attn_request(s, r);
            mine = attn_cost_before(s, q, q.nqt) * s.Hkv;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
        if ((threadIdx.x & 31) == 0 && (r0 >> 5) < kAttnGroups) groups[r0 >> 5] = mine;
        sum += mine;
    }
    if ((threadIdx.x & 31) == 0) s_sum[threadIdx.x >> 5] = sum;
    __syncthreads();
    sum = 0;
    for (int w = 0; w < THREADS / 32; w++) sum += s_sum[w];
    const long long each = (sum + ctas - 1) / ctas;
    return each < least ? least : each;
}

// A walk that starts at the 32 requests that hold unit of cost `idx` (or, beyond the
// groups there are sums of, at the first ones without).
__device__ __forceinline__ AttnWalk attn_walk_at(const AttnShape& s, const long long* groups,
                                                 long long idx) {
    const int n = min((s.N + 31) >> 5, kAttnGroups);
    AttnWalk w;
    int i = 0;
    for (; i < n && w.base + groups[i] <= idx; i++) w.base += groups[i];
    w.r0 = 32 * i;
    return w;
}

// Partial results of split items in the workspace: slot 2 c holds the part of
// CTA c's range that starts where the range does, slot 2 c + 1 the one that
// ends where it does. Per slot: rows x d outputs (each the softmax over its
// part), then rows log-sums in base 2. After the slots, one AttnCut per CTA.
struct AttnSplit {
    float* ws;      // null: whole items
    int ctas;       // CTAs the tiles are divided among
    int least;      // cost of a range, at least (no less than a tile's)
    int rows;       // rows of a slot
};
// The first tile of a CTA's range.
struct AttnCut {
    long long each;  // cost of a range
    long long u0;    // cost before the tile's item
    int tok0, ntok;  // the item's tokens (ntok 0: no tile in the range)
    int h, tile, n;  // key head; the tile's number in the item; tiles of the item
    int cost;        // of a tile
};
inline __host__ __device__ size_t attn_slot_floats(int rows, int d) { return (size_t)rows * (d + 1); }
inline __host__ __device__ AttnCut* attn_cuts(const AttnSplit& sp, int d) {
    return reinterpret_cast<AttnCut*>(sp.ws + 2 * (size_t)sp.ctas * attn_slot_floats(sp.rows, d));
}
inline size_t attn_split_bytes(const AttnSplit& sp, int d) {
    return sp.ctas * (2 * attn_slot_floats(sp.rows, d) * sizeof(float) + sizeof(AttnCut));
}

// Joins the parts of the split items (io: type of o); G query heads per key head.
cudaError_t launch_attn_combine(const AttnSplit& sp, int Hkv, int G, int d, int rows_per_tile,
                                void* o, float* lse, kda_dtype_t io, int* d_status,
                                cudaStream_t stream);
cudaError_t launch_attn_tc(const AttnArgs& a);    // bf16
cudaError_t launch_attn_simt(const AttnArgs& a);  // fp32

// How a call on `nsm` SMs divides a kernel's work: CTAs and rows of a slot of its
// split form, or ctas = 0 for whole items. max_keys: no request has more keys.
AttnSplit attn_tc_split(int N, int total_q, int max_q, long long max_keys, bool prompt, int Hq,
                        int Hkv, int nsm);
AttnSplit attn_simt_split(int N, int total_q, int max_q, long long max_keys, bool prompt, int Hq,
                          int Hkv, int nsm);

// Keys a request can have: what a row of the block table holds, up to 2^30, so that
// key numbers a few tiles past the end stay inside 32 bits.
inline int attn_kv_cap(const AttnArgs& a) {
    const long long row = (long long)a.max_pages * a.page;
    return (int)(row < (1LL << 30) ? row : 1LL << 30);
}

// Most items there can be: every request may leave one partly filled.
inline long long attn_items_bound(const AttnShape& s) {
    return ((long long)s.total_q / s.tok2 + s.N) * s.Hkv;
}

}  // namespace kda
