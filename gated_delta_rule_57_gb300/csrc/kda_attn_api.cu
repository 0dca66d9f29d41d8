// Entry points of softmax attention: argument checks and dispatch.
#include <limits.h>
#include <math.h>

#include "kda_attn.cuh"
#include "kda_host.cuh"

using namespace kda;

namespace {

constexpr int kMaxGroup = 64;  // query heads of one key head

kda_status_t check_heads(int Hq, int Hkv, int d, kda_dtype_t io) {
    if (io != KDA_BF16 && io != KDA_F32) return fail(KDA_ERR_INVALID_ARG, "unknown io dtype");
    if (Hq < 0 || Hkv < 0) return fail(KDA_ERR_INVALID_ARG, "Hq and Hkv must be >= 0");
    if (Hkv == 0 ? Hq != 0 : Hq % Hkv != 0)
        return fail(KDA_ERR_INVALID_ARG, "Hq must be a multiple of Hkv");
    if (d != 64 && d != 128) return fail(KDA_ERR_UNSUPPORTED, "d must be 64 or 128");
    if (Hkv > 0 && Hq / Hkv > kMaxGroup)
        return fail(KDA_ERR_UNSUPPORTED, "at most 64 query heads per key head");
    if (Hq > (1 << 16)) return fail(KDA_ERR_INVALID_ARG, "Hq must be at most 65536");
    return KDA_OK;
}

// What both entry points check alike; n_k and n_v: bytes that k and v span.
kda_status_t run(AttnArgs& a, kda_dtype_t io, size_t n_k, size_t n_v) {
    const size_t esz = io == KDA_BF16 ? 2 : 4;
    const size_t row = (size_t)a.Hq * a.d;
    if (!(a.scale > 0.f) || !isfinite(a.scale))
        return fail(KDA_ERR_INVALID_ARG, "scale must be positive and finite");
    if (a.total_q > (1 << 30) || a.N > (1 << 30))
        return fail(KDA_ERR_INVALID_ARG, "at most 2^30 tokens and requests");
    if (!a.q || !a.cu_q || !a.o) return fail(KDA_ERR_INVALID_ARG, "a NULL pointer");
    for (const void* p : {a.q, a.k, a.v, (const void*)a.o, (const void*)a.ws})
        if (!aligned16(p)) return fail(KDA_ERR_INVALID_ARG, "pointers must be 16-byte aligned");
    for (const void* p : {(const void*)a.cu_q, (const void*)a.kv_len, (const void*)a.block_table,
                          (const void*)a.lse, (const void*)a.d_status})
        if (!aligned4(p)) return fail(KDA_ERR_INVALID_ARG, "int and lse pointers must be 4-byte aligned");
    if (a.q_stride < (long long)row || a.q_stride > (1LL << 37))
        return fail(KDA_ERR_INVALID_ARG, "q's token stride must be at least Hq * d");
    if (a.q_stride * esz % 16)
        return fail(KDA_ERR_INVALID_ARG, "token strides must be 16-byte multiples");
    const size_t n_q = ((size_t)(a.total_q - 1) * a.q_stride + row) * esz;
    const size_t n_o = (size_t)a.total_q * row * esz;
    const size_t n_l = a.lse ? (size_t)a.total_q * a.Hq * 4 : 0;
    struct Buf {
        const void* p;
        size_t n;
    };
    const Buf ins[] = {{a.q, n_q}, {a.k, n_k}, {a.v, n_v}, {a.cu_q, ((size_t)a.N + 1) * 4},
                       {a.kv_len, a.kv_len ? (size_t)a.N * 4 : 0},
                       {a.block_table, a.block_table ? (size_t)a.N * a.max_pages * 4 : 0}};
    const Buf outs[] = {{a.o, n_o}, {a.lse, n_l}, {a.ws, a.ws_bytes}};
    for (int i = 0; i < 3; i++) {
        for (const Buf& b : ins)
            if (overlaps(outs[i].p, outs[i].n, b.p, b.n))
                return fail(KDA_ERR_INVALID_ARG, "o, lse or the workspace overlaps an input");
        for (int j = 0; j < i; j++)
            if (overlaps(outs[i].p, outs[i].n, outs[j].p, outs[j].n))
                return fail(KDA_ERR_INVALID_ARG, "o, lse and the workspace overlap");
    }
    return launched(io == KDA_BF16 ? launch_attn_tc(a) : launch_attn_simt(a));
}

}  // namespace

extern "C" {

size_t kda_attn_workspace_size(int N, int total_q, int max_q, int Hq, int Hkv, int d,
                               kda_dtype_t io) {
    if (N < 0 || total_q < 0 || max_q < 0 || check_heads(Hq, Hkv, d, io) != KDA_OK)
        return (size_t)-1;
    const int most = max_q < total_q ? max_q : total_q;
    const auto split = io == KDA_BF16 ? attn_tc_split : attn_simt_split;
    return attn_split_bytes(split(N, total_q, most, INT_MAX, false, Hq, Hkv, device_sms()), d);
}

kda_status_t kda_attn_prompt(const void* q, const void* k, const void* v, const int* cu_seqlens,
                             void* o, float* lse, int N, int total, int max_len, int Hq, int Hkv,
                             int d, long long q_stride, long long k_stride, long long v_stride,
                             float scale, kda_dtype_t io, void* workspace, size_t ws_bytes,
                             int* d_status, void* stream) {
    NvtxRange nvtx_range("kda_attn_prompt");
    if (N < 0 || total < 0 || max_len < 0)
        return fail(KDA_ERR_INVALID_ARG, "N, total and max_len must be >= 0");
    kda_status_t st = check_heads(Hq, Hkv, d, io);
    if (st != KDA_OK) return st;
    if (N == 0 || total == 0 || max_len == 0 || Hq == 0) return KDA_OK;
    if (!k || !v) return fail(KDA_ERR_INVALID_ARG, "a NULL pointer");
    const size_t esz = io == KDA_BF16 ? 2 : 4, row = (size_t)Hkv * d;
    for (long long s : {k_stride, v_stride}) {
        if (s < (long long)row || s > (1LL << 37))
            return fail(KDA_ERR_INVALID_ARG, "k's and v's token strides must be at least Hkv * d");
        if (s * esz % 16) return fail(KDA_ERR_INVALID_ARG, "token strides must be 16-byte multiples");
    }
    AttnArgs a{};
    a.q = q;
    a.k = k;
    a.v = v;
    a.cu_q = cu_seqlens;
    a.o = o;
    a.lse = lse;
    a.N = N;
    a.total_q = total;
    a.max_q = max_len < total ? max_len : total;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.d = d;
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.scale = scale;
    a.ws = static_cast<float*>(workspace);
    a.ws_bytes = workspace ? ws_bytes : 0;
    a.d_status = d_status;
    a.stream = static_cast<cudaStream_t>(stream);
    return run(a, io, ((size_t)(total - 1) * k_stride + row) * esz,
               ((size_t)(total - 1) * v_stride + row) * esz);
}

kda_status_t kda_attn_paged(const void* q, const void* k_cache, const void* v_cache,
                            const int* block_table, const int* cu_q, const int* kv_len, void* o,
                            float* lse, int N, int total_q, int max_q, int Hq, int Hkv, int d,
                            long long q_stride, int num_pages, int page_size, int max_pages,
                            float scale, kda_dtype_t io, void* workspace, size_t ws_bytes,
                            int* d_status, void* stream) {
    NvtxRange nvtx_range("kda_attn_paged");
    if (N < 0 || total_q < 0 || max_q < 0 || num_pages < 1 || max_pages < 0 || page_size < 1)
        return fail(KDA_ERR_INVALID_ARG, "sizes must be >= 0, num_pages and page_size positive");
    kda_status_t st = check_heads(Hq, Hkv, d, io);
    if (st != KDA_OK) return st;
    if (page_size < 16 || page_size > 1024 || (page_size & (page_size - 1)))
        return fail(KDA_ERR_UNSUPPORTED, "page_size must be a power of two in 16 .. 1024");
    if ((long long)num_pages * page_size >= (1LL << 31))
        return fail(KDA_ERR_INVALID_ARG, "num_pages * page_size must be below 2^31");
    if (N == 0 || total_q == 0 || max_q == 0 || Hq == 0) return KDA_OK;
    if (!kv_len || (max_pages > 0 && !block_table) || !k_cache || !v_cache)
        return fail(KDA_ERR_INVALID_ARG, "a NULL pointer");
    size_t n_c;
    if (!mul_ok(&n_c, num_pages, page_size, (size_t)Hkv * d, io == KDA_BF16 ? 2 : 4))
        return fail(KDA_ERR_INVALID_ARG, "tensor size overflow");
    AttnArgs a{};
    a.q = q;
    a.k = k_cache;
    a.v = v_cache;
    a.cu_q = cu_q;
    a.kv_len = kv_len;
    a.block_table = block_table;
    a.o = o;
    a.lse = lse;
    a.N = N;
    a.total_q = total_q;
    a.max_q = max_q < total_q ? max_q : total_q;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.d = d;
    a.q_stride = q_stride;
    a.num_pages = num_pages;
    a.page = page_size;
    a.max_pages = max_pages;
    a.scale = scale;
    a.ws = static_cast<float*>(workspace);
    a.ws_bytes = workspace ? ws_bytes : 0;
    a.d_status = d_status;
    a.stream = static_cast<cudaStream_t>(stream);
    return run(a, io, n_c, n_c);
}

}  // extern "C"
