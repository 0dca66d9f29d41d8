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
//   Whole items: CTA c takes items c, c + grid, ...; inside a request the
//     longest (last tokens) come first and the key heads run fastest, so
//     concurrent CTAs share the keys of one request in L2 and the short
//     items fill the end.
//   Split items: the key tiles of all items laid end to end are cut into
//     equal ranges, one per CTA, so few rows over a long cache use every SM
//     and ragged lengths balance exactly. An item cut by a boundary leaves
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

cudaError_t launch_attn_simt(const AttnArgs& a, kda_dtype_t io);

// What the device side needs to divide the work.
struct AttnShape {
    const int* cu_q;
    const int* kv_len;
    int N, total_q, max_q, kv_cap;  // kv_cap: tokens a block-table row can hold
    int Hkv, G;
    int tok1, tok2;  // tokens of an item: tok1 for requests that fit it, else tok2
    int kt;          // keys of a key tile
};

// One request: its packed tokens, keys, and items.
struct AttnReq {
    int q0, q_len, kv;  // first packed token, new tokens, keys
    int tok, nqt;       // tokens per item, items per key head
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
    return q;
}

// Keys that the last token of item t of a request sees (0: none).
__device__ __forceinline__ int attn_item_keys(const AttnReq& q, int t) {
    const int last = min((t + 1) * q.tok, q.q_len);
    return max(q.kv - q.q_len + last, 0);
}

// The next whole item of a sequence of increasing item numbers: a walk over
// the requests, a warp together. Items of a request: tiles from the last to
// the first, key heads inside.
struct AttnWalk {
    int r0 = 0;          // the 32 requests r0 .. r0 + 31 are looked at
    long long base = 0;  // items before them
    bool bad = false;    // some request so far had a bad length (lane-wise)
};

struct AttnItem {
    int r, t, h;
    AttnReq q;
};

// False when there is no item `idx`. idx must not decrease from call to call.
__device__ __forceinline__ bool attn_find_item(const AttnShape& s, AttnWalk& w, long long idx,
                                               AttnItem* it) {
    const int lane = threadIdx.x & 31;
    for (; w.r0 < s.N; w.r0 += 32) {
        const int r = w.r0 + lane;
        AttnReq q{};
        if (r < s.N) q = attn_request(s, r);
        w.bad |= q.bad != 0;
        const long long mine = (long long)q.nqt * s.Hkv;
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
            it->r = w.r0 + src;
            it->q.q0 = __shfl_sync(0xffffffffu, q.q0, src);
            it->q.q_len = __shfl_sync(0xffffffffu, q.q_len, src);
            it->q.kv = __shfl_sync(0xffffffffu, q.kv, src);
            it->q.tok = __shfl_sync(0xffffffffu, q.tok, src);
            it->q.nqt = __shfl_sync(0xffffffffu, q.nqt, src);
            it->q.bad = 0;
            const int in = (int)(idx - w.base - __shfl_sync(0xffffffffu, inc - mine, src));
            it->t = it->q.nqt - 1 - in / s.Hkv;
            it->h = in % s.Hkv;
            return true;
        }
        w.base += total;
    }
    return false;
}

// Most items there can be, for the grid: every request may leave one tile
// partly filled.
inline long long attn_items_bound(const AttnShape& s) {
    const long long full = (long long)s.total_q / s.tok1;
    const long long some = full + s.N;
    return some * s.Hkv;
}

}  // namespace kda
