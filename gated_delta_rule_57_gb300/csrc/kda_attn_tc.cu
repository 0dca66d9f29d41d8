// Softmax attention on the 5th-generation tensor cores (bf16).
//
//     S = Q K^T,  P = 2^{c S - m},  O = P V / l,   c = scale log2 e
//
// with m a running reference of each row's largest c S and l its running sum.
// A raised m multiplies what O and l hold by 2^{m_old - m_new}; m is only
// raised when a row's maximum passes it by more than 8, so P stays below 2^8
// (bf16 and fp32 keep their relative precision there) and after a few key
// tiles O is hardly ever touched.
//
// One CTA per SM, four warpgroups:
//   warps 0..3, 4..7  two softmax groups, one row of S per thread
//   warp 8            issues the products (at DQ = 192: of the first group)
//   warp 9            finds the work and issues the loads
//   warp 10           clears V of what some rows must not see
//   warp 11           adds that to the finished rows which see it (at DQ = 192 warp 10 does,
//                     and this one issues the second group's products)
//   warps 12..15      the results: O / l, merging, stores
// Every wait has a limit, after which the kernel reports KDA_DEV_TIMEOUT.
// A group's loop: S (TMEM, 128 lanes x 128 columns fp32) -> registers, mask,
// maximum, exponentials, P as bf16 pairs into the first half of S's columns, and
// the second product reads P from there as its A operand. While one group
// computes exponentials the tensor core runs the other group's two products.
// The groups hold either the two row tiles of one item, sharing every key and
// value tile (prompts and chunks), or the even and the odd key tiles of one
// row tile (few rows: the two results are merged in TMEM at the end).
//
// Tensor memory (512 columns): S of group 0, S of group 1, O of group 0, O of
// group 1. Shared memory: two Q tiles and a ring of K / V tiles, all "SW128
// row tiles" of 128 rows, filled by TMA. K tiles are the K-major B operand of
// the first product, V tiles the MN-major B operand of the second.
//
// A key past a row's last one gets P = 0 by a select on S. 0 x NaN is NaN, so V is
// cleared in shared memory before the product: past the item's last key (stale cache
// slots, the next prompt) all of it; of the keys that some rows of the item see and
// others do not (fewer than it has tokens, at its end) the values that are not finite.
// Those are noted, and added to the finished o of the rows that see them: p > 0 times
// NaN or Inf is what it was.
//
// What bounds it: for prompts the tensor pipe (78 % active), whose gaps are the chain
// of one group (scores, exponentials, second product) against the other group's two
// products, and shared memory, which the products' operands and the TMA writes
// occupy as long as the products take; for single tokens HBM. Measured (32 / 8
// heads, d = 128): 8 prompts of 8192 tokens 2.46 ms, 1.79 PFLOP/s, alone at 2.07 GHz, and
// 2.74 ms, 1.60 PFLOP/s, back to back at the power limit (1.65 to 1.70 GHz); one token
// of 256 requests over 1.05 M cached tokens 0.61 ms, 7.0 TB/s; 2 x 4 drafts over 262 k
// tokens each 0.31 ms, 6.9 TB/s.
#include <atomic>

#include "kda_attn.cuh"
#include "kda_host.cuh"
#include "sm100_ptx.cuh"
#include "tensor_map.cuh"

namespace kda {
namespace {

using namespace ptx;

constexpr int kTile = 128;         // rows of a row tile, keys of a key tile
constexpr int kThreadsTc = 512;
// Registers per thread: launched with 128 (65536 in all), then by warpgroup.
constexpr int kRegsSoftmax = 192, kRegsOther = 64, kRegsResult = 64;
static_assert(2 * kRegsSoftmax + kRegsOther + kRegsResult <= 4 * 128, "more than launched with");
constexpr int kMmaWarp = 8, kLoadWarp = 9, kEdgeWarp = 10, kMmaWarp1 = 11;
constexpr int kPieces = 4;         // pieces announced ahead
constexpr int kAskAhead = 6;       // key tiles left to load of a whole item when the next is asked for
// Relative time of a key tile for one row tile and for a pair: about 1750 and 2500
// clocks, measured at d = 128 in a step of two prompts' chunks among single tokens.
constexpr int kCostSingle = 5, kCostPair = 7;
// An item beside its key tiles: 4700 clocks of a pair's, measured over 8192 causal tokens.
constexpr int kItemKeys = 256;
// Limit of a wait (about 4 s). The longest is for the results of a piece, while its key
// tiles go by at 1.4 us each: some 2.8 million tiles, 360 million keys.
constexpr long long kWaitClocks = 1LL << 33;
constexpr float kRaise = 8.f;      // log2 growth of a row maximum that moves its reference

// DQ channels of queries and keys, D of values and outputs. DQ > D: the last DQ - D of
// the keys are shared by all heads and have places of their own beside the ring. (Two, and
// three tiles in the ring: all that fits. 96 keys a tile and four of them took 1799 and 488 us for
// the two calls below where these took 1812 and 494.) At 192 and 128 channels 4 prompts of 8192 tokens
// x 32 heads run at 1690 TFLOP/s, bound by the tensor cores; 24 ragged ones to 4096 at 1260: tiles at
// the diagonal and at the ends of prompts take an eighth more, uneven CTAs the rest.
template <int DQ, int D>
struct TcCfg {
    static constexpr int DR = DQ - D;
    static constexpr int TILE_BYTES = kTile * D * 2, Q_BYTES = kTile * DQ * 2;
    static constexpr int SHARED_BYTES = kTile * DR * 2;
    static constexpr int STAGES = DR ? 3 : D == 128 ? 5 : 8;
    // Issuing warps: one for both groups, in a fixed order, or one for each. What such a warp
    // does between two products shows as idle tensor core unless the other's run, but the
    // order keeps the groups half a step apart. Measured, one against two, us (32 heads): DQ = 192,
    // 4 prompts of 8192 1800/1614, 24 ragged 490/460; DQ = D = 128 (8 key heads), 8 of 8192 2465/2855,
    // ragged 318/370, a mixed step over pages 463/521; with 32 key heads, 4 of 8192 1327/1643, 24
    // ragged 1083/1258.
    static constexpr bool TWO_ISSUE = DR > 0;
    static constexpr int TILES = 2 * Q_BYTES + STAGES * TILE_BYTES + 2 * SHARED_BYTES;
};

struct TcAttnParams {
    AttnShape s;
    AttnSplit sp;
    const int* block_table;  // null: packed prompts
    const __nv_bfloat16* v;
    __nv_bfloat16* o;
    float* lse;
    long long v_stride, v_head;
    int num_pages, page, max_pages;
    int box_q;  // tokens of a Q load
    float c;    // scale log2 e
    int* d_status;
};

// A range of key tiles of one item.
struct Piece {
    int r, h;
    int tok0;       // packed token of row 0
    int ntok;       // tokens of the item
    int pos0;       // keys that row 0's token sees, less one (may be negative)
    int key0;       // packed token of key 0 (prompts)
    int kv;         // keys of the request
    int keys;       // keys the item's last token sees
    int kt0, kt1;   // key tiles
    int pair;       // two row tiles (1) or one (0)
    int slot;       // where a part of an item goes; -1: the whole item
    int end;        // no more pieces
};

// Key tiles of a softmax group: tiles kt0 + first, + step, ... (n of them).
struct Share {
    int n, first, step;
};
__device__ __forceinline__ Share group_share(const Piece& p, int w, int tok1) {
    Share g;
    if (p.pair) {
        const int last = min((w + 1) * tok1, p.ntok);  // its last token
        const int keys = last > w * tok1 ? max(p.pos0 + last, 0) : 0;
        g.n = max(min(p.kt1, (keys + kTile - 1) / kTile) - p.kt0, 0);
        g.first = 0;
        g.step = 1;
    } else {
        g.n = (min(p.kt1, (p.keys + kTile - 1) / kTile) - p.kt0 - w + 1) / 2;
        g.n = max(g.n, 0);
        g.first = w;
        g.step = 2;
    }
    return g;
}
__device__ __forceinline__ int piece_tiles(const Piece& p) {
    return max(min(p.kt1, (p.keys + kTile - 1) / kTile) - p.kt0, 0);
}
// Keys that every row of the item sees: those of its first token.
__device__ __forceinline__ int seen_by_all(const Piece& p) { return min(max(p.pos0 + 1, 0), p.keys); }
// The first of a piece's n key tiles with keys that some row does not see; V of this
// one and those after it is cleared.
__device__ __forceinline__ int edge_tile(const Piece& p, int n) {
    return min(max(seen_by_all(p) / kTile - p.kt0, 0), n);
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<uint32_t*>(&v);
}
// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n\t.reg .b64 a, b, c, d;\n\t"
        "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
        "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 a, b, d;\n\t"
        "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "add.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
// A bounded wait by a whole warp, with one outcome for all its lanes.
__device__ __forceinline__ void warp_wait(bool& ok, uint64_t* bar, uint32_t parity) {
    if (ok) ok = mbar_wait(bar, parity, kWaitClocks);
    ok = __all_sync(0xffffffffu, ok);
}

struct Shared {
    uint64_t kv_full[8], kv_empty[8];
    uint64_t v_ready[8];            // a tile of the ring has been seen: V is cleared
    uint64_t q_full, q_empty;
    uint64_t s_full[2], p_full[2][2];  // of each group; P per half of the keys
    // Of each group, for each piece: its references and sums are there, are read;
    // for each piece in which it has key tiles: its O is complete, is read. (A
    // group without tiles runs ahead of the products, so it may not count in
    // what they wait for.)
    uint64_t ml_full[2], ml_free[2], o_full[2], o_free[2];
    uint64_t piece_full[kPieces], piece_empty[kPieces];
    uint64_t odd_full[kPieces];     // all V tiles of a piece are cleared
    uint64_t rows_full[kPieces];    // all its rows are written
    uint64_t next_full;             // the number of the next whole item
    uint64_t drained[2];            // all products (of a group) have ended
    alignas(16) uint4 next;
    Piece pieces[kPieces];
    // Keys of a piece with values that were cleared: bit i, key seen_by_all + i.
    uint32_t odd[kPieces][8];
    union {
        float2 ml[2][kTile];            // reference and sum of each row
        long long groups[kAttnGroups];  // before the first piece
    };
    long long sum[kThreadsTc / 32];
    uint32_t tmem;
};
template <int DQ, int D>
constexpr int tc_smem() {
    return TcCfg<DQ, D>::TILES + (int)sizeof(Shared);
}
static_assert(tc_smem<128, 128>() <= 227 * 1024 && tc_smem<192, 128>() <= 227 * 1024, "shared memory of a CTA");

// Values of key j of a piece; null where its page id is out of range (such pages
// read as zeros).
__device__ __forceinline__ const __nv_bfloat16* values_at(const TcAttnParams& p, const Piece& pc,
                                                          int d, int j) {
    if (!p.block_table)
        return p.v + (size_t)(pc.key0 + j) * p.v_stride + (size_t)pc.h * p.v_head;
    const int id = p.block_table[(size_t)pc.r * p.max_pages + j / p.page];
    if (id < 0 || id >= p.num_pages) return nullptr;
    return p.v + (((size_t)id * p.s.Hkv + pc.h) * p.page + j % p.page) * d;
}

// Sign bits set where a bf16 of a pair has all exponent bits: NaN or Inf.
__device__ __forceinline__ uint32_t odd_pair(uint32_t x) {
    return ((x & 0x7f807f80u) + 0x00800080u) & 0x80008000u;
}
__device__ __forceinline__ uint32_t odd_vector(uint4 x) {
    return odd_pair(x.x) | odd_pair(x.y) | odd_pair(x.z) | odd_pair(x.w);
}
__device__ __forceinline__ uint32_t finite_pair(uint32_t x) {  // zeros for the others
    const uint32_t odd = odd_pair(x);
    return x & ~((odd >> 15 & 0x00010001u) * 0xffffu);
}

// Clears a V tile, a warp together: rows from r1 on, and what is not finite in rows
// [r0, r1). odd: a bit for each such row, row r0 being bit `bit0`.
template <int D>
__device__ __forceinline__ void clear_values(unsigned char* v, int r0, int r1, uint32_t* odd,
                                             int bit0) {
    const int lane = threadIdx.x & 31;
    uint32_t any = 0;
#pragma unroll
    for (int half = 0; half < D / 64; half++) {
        const unsigned char* t = v + half * (kTile * 128);
#pragma unroll 2  // (short prompts 8.5 us, 8.9 with one at a time; four: ragged ones +0.3 %)
        for (int b = r0 * 128 + lane * 16; b < r1 * 128; b += 512)
            any |= odd_vector(*reinterpret_cast<const uint4*>(t + b));
    }
    if (__any_sync(0xffffffffu, any)) {
        for (int half = 0; half < D / 64; half++)
            for (int b = r0 * 128 + lane * 16; b < r1 * 128; b += 512) {
                uint4& x = *reinterpret_cast<uint4*>(v + half * (kTile * 128) + b);
                if (!odd_vector(x)) continue;
                x = make_uint4(finite_pair(x.x), finite_pair(x.y), finite_pair(x.z), finite_pair(x.w));
                const int bit = bit0 + b / 128 - r0;
                atomicOr(odd + (bit >> 5), 1u << (bit & 31));
            }
    }
#pragma unroll
    for (int half = 0; half < D / 64; half++)
        for (int b = r1 * 128 + lane * 16; b < kTile * 128; b += 512)
            *reinterpret_cast<uint4*>(v + half * (kTile * 128) + b) = make_uint4(0, 0, 0, 0);
}

// Adds the cleared values to the rows that see them, by a warp once the rows are
// written. odd: lane i holds word i of the piece's bits (zero from lane 8 on). Rows see
// more keys from one to the next, so each value is read once for a row tile.
template <int D>
__device__ __forceinline__ int add_cleared(const TcAttnParams& p, const Piece& pc, uint32_t odd,
                                           float* part) {
    const int lane = threadIdx.x & 31, all = seen_by_all(pc), G = p.s.G, tok1 = p.s.tok1;
    constexpr int E = D / 32;
    int flags = 0;
    for (int w = 0; w <= pc.pair; w++) {
        float sum[E];  // of columns lane + 32 e: zero, or not finite
#pragma unroll
        for (int e = 0; e < E; e++) sum[e] = 0.f;
        int i = 0;  // cleared keys below all + i are in the sums
        for (int r = 0; r < tok1 * G; r++) {
            const int tok = w * tok1 + r / G;
            if (tok >= pc.ntok) break;
            const int sees = min(pc.pos0 + tok + 1 - all, 256);
            for (; i < sees; i++) {
                if (!(__shfl_sync(0xffffffffu, odd, i >> 5) >> (i & 31) & 1)) continue;
                const __nv_bfloat16* v = values_at(p, pc, D, all + i);
                if (!v) continue;
#pragma unroll
                for (int e = 0; e < E; e++) {
                    const float x = __bfloat162float(v[lane + 32 * e]);
                    if (finite_flag(x)) sum[e] += x;
                }
            }
            const size_t at = ((size_t)pc.tok0 + tok) * p.s.Hkv * G + (size_t)pc.h * G + r % G;
#pragma unroll
            for (int e = 0; e < E; e++) {
                if (!finite_flag(sum[e])) continue;
                flags = KDA_DEV_NONFINITE;
                const int c = lane + 32 * e;
                if (part) part[(size_t)(w * kTile + r) * D + c] += sum[e];
                else p.o[at * D + c] = __float2bfloat16_rn(__bfloat162float(p.o[at * D + c]) + sum[e]);
            }
        }
    }
    return flags;
}

// r: of the shared key channels, where there are any.
template <int DR>
struct TcMaps {
    CUtensorMap q, k, v, r;
};
template <>
struct TcMaps<0> {
    CUtensorMap q, k, v;
};

template <int DQ, int D, bool EARLY>
__global__ void __launch_bounds__(kThreadsTc, 1)
    kda_attn_tc_kernel(const __grid_constant__ TcMaps<DQ - D> maps, const __grid_constant__ TcAttnParams p) {
    using C = TcCfg<DQ, D>;
    constexpr int NS = C::STAGES, HALVES = D / 64;
    constexpr uint32_t TM_S = 0, TM_O = 256;
    extern __shared__ __align__(1024) unsigned char sm[];  // 128-byte swizzle: 1024-byte tiles
    unsigned char* sq = sm;                        // two Q tiles
    unsigned char* skv = sm + 2 * C::Q_BYTES;      // the ring
    // Shared key channels: of even and odd key tiles. They come and go with their key tile:
    // a place's last user is at least as far back as that of the ring's place (three tiles).
    unsigned char* srope = skv + NS * C::TILE_BYTES;
    Shared& sh = *reinterpret_cast<Shared*>(sm + C::TILES);
    if (smem_addr(sm) & 1023u) {  // never, by the declaration above
        if (threadIdx.x == 0 && p.d_status) atomicOr(p.d_status, KDA_DEV_TIMEOUT);
        return;
    }

    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // uniform, and known to be
    if (warp == 1) {
        if (lane < NS) {
            mbar_init(&sh.kv_full[lane], 1);
            // read by the products, seen by the V warp
            mbar_init(&sh.kv_empty[lane], C::TWO_ISSUE ? 3 : 2);
            mbar_init(&sh.v_ready[lane], 1);
        }
        if (lane < 2) {
            mbar_init(&sh.s_full[lane], 1);
            mbar_init(&sh.p_full[lane][0], 128);
            mbar_init(&sh.p_full[lane][1], 128);
            mbar_init(&sh.o_full[lane], 1);
            mbar_init(&sh.ml_full[lane], 128);
            mbar_init(&sh.ml_free[lane], 128);
            mbar_init(&sh.o_free[lane], 128);
            mbar_init(&sh.drained[lane], 1);
        }
        if (lane < kPieces) {
            mbar_init(&sh.piece_full[lane], 1);
            // softmax 8, products and V 3 (TWO_ISSUE: products 2, V), results 4
            mbar_init(&sh.piece_empty[lane], 15);
            mbar_init(&sh.odd_full[lane], 1);
            mbar_init(&sh.rows_full[lane], 4);
        }
        if (lane == 0) {
            mbar_init(&sh.next_full, 1);
            mbar_init(&sh.q_full, 1);
            mbar_init(&sh.q_empty, C::TWO_ISSUE ? 2 : 1);
            prefetch_tensormap(&maps.q);
            prefetch_tensormap(&maps.k);
            prefetch_tensormap(&maps.v);
            if constexpr (C::DR > 0) prefetch_tensormap(&maps.r);
        }
        fence_mbarrier_init();
    }
    if (warp == 0) {
        tmem_alloc(&sh.tmem, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    pdl_wait();
    // Cost of this CTA's range (split items); also the barrier after the setup.
    long long each = 0;
    if (p.sp.ws) each = attn_cost_each<kThreadsTc>(p.s, p.sp.ctas, p.sp.least, sh.groups, sh.sum);
    __syncthreads();
    tc_fence_after();
    const uint32_t tbase = sh.tmem;
    const int G = p.s.G, tok1 = p.s.tok1;
    int flags = 0;
    bool ok = true;

    if (warp >= 8 && warp < 12) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOther));
        if (warp == kLoadWarp) {
            // ------------------------------------------------------------ work and loads
            int stage = 0, kv_phase = 0, q_phase = 0, np = 0;
            int asked = 0;  // for further items
            int nk = 0;     // key tiles so far
            // Paged: a tile is `per` pages (or part of one); lane `pg` of each half
            // loads one. Their ids are read a tile or more ahead of their use.
            const int log2_page = __ffs(p.page) - 1;
            const int per = p.block_table && p.page < kTile ? kTile >> log2_page : 1;
            const int pg = lane & (per - 1), half = lane / per;
            auto page_id = [&](const Piece& pc, int kt) {
                // past the keys, or no page: beyond the cache, which loads zeros
                int id = p.num_pages;
                const int j = kt * kTile + (pg << log2_page);  // first key of the lane's part
                if (half < HALVES && j < pc.kv) {
                    id = p.block_table[(size_t)pc.r * p.max_pages + (j >> log2_page)];
                    if (id < 0 || id >= p.num_pages) {
                        id = p.num_pages;
                        flags |= KDA_DEV_PAGES;
                    }
                }
                return id;
            };
            auto load_kv = [&](const Piece& pc, const CUtensorMap* map, int kt, int id, bool keys) {
                warp_wait(ok, &sh.kv_empty[stage], kv_phase ^ 1);
                if (!ok) return;
                unsigned char* dst = skv + stage * C::TILE_BYTES;
                uint64_t* bar = &sh.kv_full[stage];
                if (lane == 0)
                    mbar_arrive_expect_tx(bar, C::TILE_BYTES + (keys ? C::SHARED_BYTES : 0));
                __syncwarp();
                if constexpr (C::DR > 0) {
                    if (keys) {
                        if (lane == HALVES)
                            tma_load_3d(srope + (nk & 1) * C::SHARED_BYTES, &maps.r, bar, 0, 0, pc.key0 + kt * kTile);
                        nk++;
                    }
                }
                if (half < HALVES) {
                    dst += half * (kTile * 128);
                    if (!p.block_table)
                        tma_load_3d(dst, map, bar, 64 * half, pc.h, pc.key0 + kt * kTile);
                    else
                        tma_load_4d(dst + (pg << log2_page) * 128, map, bar, 64 * half,
                                    (kt * kTile) & (p.page - 1), pc.h, id);
                }
                if (++stage == NS) {
                    stage = 0;
                    kv_phase ^= 1;
                }
            };
            auto announce = [&](const Piece& pc) {
                const int i = np % kPieces;
                warp_wait(ok, &sh.piece_empty[i], ((np / kPieces) & 1) ^ 1);
                if (!ok) return;
                if (lane == 0) {
                    sh.pieces[i] = pc;
                    mbar_arrive(&sh.piece_full[i]);
                }
                np++;
                __syncwarp();
            };
            // Whole items: another one is asked for when this one's last loads are due (at its first
            // ones, a CTA with a long item takes a further one away from those about to end), or,
            // EARLY, before this one is looked up: see launch_t.
            auto ask = [&] {
                if (lane == 0) {
                    mbar_arrive_expect_tx(&sh.next_full, 16);
                    clc_try_cancel(&sh.next, &sh.next_full);
                }
                asked++;
                __syncwarp();
            };
            auto process = [&](const Piece& pc) {
                announce(pc);
                const int n = piece_tiles(pc), lead = pc.pair ? 1 : 2;
                if (n == 0 || !ok) return false;
                warp_wait(ok, &sh.q_empty, q_phase ^ 1);
                if (!ok) return false;
                q_phase ^= 1;
                if (lane == 0)
                    mbar_arrive_expect_tx(&sh.q_full, (1 + pc.pair) * (DQ / 64) * p.box_q * G * 128);
                __syncwarp();
                if (lane < DQ / 64 * (1 + pc.pair)) {
                    const int w = lane / (DQ / 64), half = lane % (DQ / 64);
                    tma_load_3d(sq + w * C::Q_BYTES + half * (kTile * 128), &maps.q, &sh.q_full,
                                64 * half, pc.h * G, pc.tok0 + w * tok1);
                }
                // Ids of tiles j, j + 1, j + 2 in id[0..2].
                int id[3] = {0, 0, 0};
                if (p.block_table) {
#pragma unroll
                    for (int j = 0; j < 3; j++) id[j] = page_id(pc, pc.kt0 + j);
                }
                load_kv(pc, &maps.k, pc.kt0, id[0], true);
                if (lead == 2 && n > 1) load_kv(pc, &maps.k, pc.kt0 + 1, id[1], true);
                for (int j = 0; j < n; j++) {
                    if (!EARLY && !p.sp.ws && j == max(n - kAskAhead, 0)) ask();
                    load_kv(pc, &maps.v, pc.kt0 + j, id[0], false);
                    if (j + lead < n) load_kv(pc, &maps.k, pc.kt0 + j + lead, lead == 1 ? id[1] : id[2], true);
                    id[0] = id[1];
                    id[1] = id[2];
                    if (p.block_table && j + 3 < n) id[2] = page_id(pc, pc.kt0 + j + 3);
                }
                return true;
            };
            auto piece_of = [&](int r, const AttnReq& q, int h, int t) {
                Piece pc;
                pc.r = r;
                pc.h = h;
                const int at = t * q.tok;
                pc.tok0 = q.q0 + at;
                pc.ntok = min(q.tok, q.q_len - at);
                pc.pos0 = q.kv - q.q_len + at;
                pc.key0 = q.q0;
                pc.kv = q.kv;
                pc.keys = attn_item_keys(q, t);
                pc.kt0 = 0;
                pc.kt1 = attn_item_tiles(p.s, q, t);
                pc.pair = q.tok > tok1;
                pc.slot = -1;
                pc.end = 0;
                return pc;
            };
            // Whole items: a CTA per item, of which those that run take over the ones
            // that have not started, in their order (longest rows of a request first),
            // asking ahead. Split ones: the tiles that start in [cur, end), item by item.
            AttnReq q{};
            int r = 0, h = 0, t = 0, tile = 0;
            long long in;
            const bool split = p.sp.ws != nullptr;
            long long cur = split ? blockIdx.x * each : blockIdx.x;
            const long long end = cur + each;
            long long start = cur;
            bool have = false;  // (q, h, t, tile) is where `cur` is
            // One CTA reports on the lengths of all requests: the one that has item 0.
            // CTA 0 is not always that, as one that has not started may be taken over.
            bool reports = blockIdx.x == 0;
            AttnWalk walk;
            if (split) {
                walk = attn_walk_at(p.s, sh.groups, cur);
                AttnCut cut{each, 0, 0, 0, 0, 0, 0, 0};
                have = attn_first_tile(p.s, walk, &cur, &r, &q, &h, &t, &tile) && cur < end;
                start = cur;
                if (have) {
                    cut.cost = q.cost * kTile;
                    cut.u0 = cur - (long long)tile * cut.cost;
                    cut.tok0 = q.q0 + t * q.tok;
                    cut.ntok = min(q.tok, q.q_len - t * q.tok);
                    cut.h = h;
                    cut.tile = tile;
                    cut.n = attn_item_tiles(p.s, q, t);
                }
                if (lane == 0) attn_cuts(p.sp, D)[blockIdx.x] = cut;
                if (!have) cur = end;
            }
            while (ok && (!split || cur < end)) {
                if (!split) {
                    if (EARLY) ask();
                    if (cur < walk.base) walk = AttnWalk{};
                }
                if (!have) {
                    have = split ? attn_first_tile(p.s, walk, &cur, &r, &q, &h, &t, &tile)
                                 : attn_find<false>(p.s, walk, cur, &r, &q, &in);
                    if (!split && have) {
                        t = q.nqt - 1 - (int)(in / p.s.Hkv);
                        h = (int)(in % p.s.Hkv);
                        have = !q.bad;
                    }
                }
                bool asks = false;  // for the next item, among its loads
                if (have) {
                    Piece pc = piece_of(r, q, h, t);
                    if (split) {
                        const int n = pc.kt1;
                        const long long u0 = cur - (long long)tile * q.cost * kTile;
                        pc.kt0 = tile;
                        pc.kt1 = attn_tiles_until(p.s, q, u0, n, end);
                        if (pc.kt1 - pc.kt0 < n) pc.slot = 2 * blockIdx.x + (cur > start ? 1 : 0);
                        cur = pc.kt1 < n ? end
                                         : u0 + attn_cost_before(p.s, q, t + 1) - attn_cost_before(p.s, q, t);
                        tile = 0;
                        if (++t == q.nqt) {
                            t = 0;
                            h++;
                        }
                        have = h < p.s.Hkv;
                    }
                    asks = process(pc);
                } else if (split) {
                    break;
                }
                if (!split) {
                    if (!EARLY && !asks) ask();
                    have = false;
                    warp_wait(ok, &sh.next_full, (asked - 1) & 1);
                    const int x = ok ? __shfl_sync(0xffffffffu, clc_answer(&sh.next), 0) : -1;
                    if (x < 0) break;
                    cur = x;
                    reports |= x == 0;
                    // the answer is read before the next one is written
                    fence_proxy_async_smem();
                    __syncwarp();
                }
            }
            if (reports) {  // lengths of requests this CTA had no work of too
                for (int i = lane; i < p.s.N; i += 32) walk.bad |= attn_request<true>(p.s, i).bad != 0;
                if (walk.bad) flags |= KDA_DEV_LENGTH;
            }
            Piece last{};
            last.end = 1;
            announce(last);
            if (!ok) {
                flags |= KDA_DEV_TIMEOUT;
                // copies in flight land before the CTA leaves
                for (int i = 0; i < NS; i++)
                    mbar_wait(&sh.kv_full[i], (i < stage ? kv_phase : kv_phase ^ 1), 1LL << 24);
                mbar_wait(&sh.q_full, q_phase ^ 1, 1LL << 24);
                if (asked) mbar_wait(&sh.next_full, (asked - 1) & 1, 1LL << 24);
            }
        } else if (C::TWO_ISSUE && (warp == kMmaWarp || warp == kMmaWarp1)) {
            // ------------------------------------------------------------ products, a warp a group
            // Both warps see every tile of the ring go by, in its order, and give it back:
            // after the products of theirs that read it, or at once. All of it is uniform,
            // so that stages and descriptors stay in uniform registers, and one elected lane
            // issues.
            const int w = warp == kMmaWarp ? 0 : 1;
            int stage = 0, kv_phase = 0, np = 0;
            int nq = 0, tiles = 0, uses = 0;  // row tiles, key tiles of the group, pieces with any, so far
            constexpr uint32_t idesc_s = idesc_bf16(kTile, kTile, 0, 0);
            constexpr uint32_t idesc_o = idesc_bf16(kTile, D, 0, 1);
            const uint64_t dq = desc_kmajor(smem_addr(sq));
            const uint64_t dk = desc_kmajor(smem_addr(skv)), dv = desc_mnmajor(smem_addr(skv), kTile);
            constexpr uint32_t TILE = C::TILE_BYTES >> 4, QTILE = C::Q_BYTES >> 4;  // in descriptor units
            const uint64_t dr = desc_kmajor(smem_addr(srope));
            uint32_t rope = 0;  // place of the next key tile's shared channels
            const uint32_t ds = tbase + TM_S + w * kTile, dout = tbase + TM_O + w * D;
            auto next = [&] {
                if (++stage == NS) {
                    stage = 0;
                    kv_phase ^= 1;
                }
            };
            auto wait = [&](uint64_t* bar, uint32_t parity) {
                if (!__all_sync(0xffffffffu, mbar_wait(bar, parity, kWaitClocks))) ok = false;
                return ok;
            };
            auto uniform = [](int x) { return __shfl_sync(0xffffffffu, x, 0); };
            auto commit = [&](uint64_t* bar) {
                if (elect_one()) mma_commit(bar);
                __syncwarp();
            };
            // A tile of the other group's: there, so that its barrier's phase is this one. (Given
            // back behind this warp's products, so that what the ring gives back, and the
            // shared channels of earlier tiles with it, is read.)
            auto skip = [&] {
                if (!wait(&sh.kv_full[stage], kv_phase)) return false;
                commit(&sh.kv_empty[stage]);
                next();
                return true;
            };
            // S = Q K^T with the ring's next tile; `last` of the piece for these rows.
            auto scores = [&](uint32_t qtile, bool last) {
                if (!wait(&sh.kv_full[stage], kv_phase)) return false;
                tc_fence_after();
                const uint64_t a = dq + qtile * QTILE, b = dk + stage * TILE;
                if (elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < D / 16; kk++)
                        mma_bf16(ds, a + kstep_kmajor(kTile, kk), b + kstep_kmajor(kTile, kk), idesc_s, kk > 0);
                    if (C::DR) {
                        const uint64_t ar = a + kstep_kmajor(kTile, D / 16);
                        const uint64_t br = dr + rope * (C::SHARED_BYTES >> 4);
#pragma unroll
                        for (int kk = 0; kk < C::DR / 16; kk++)
                            mma_bf16(ds, ar + kstep_kmajor(kTile, kk), br + kstep_kmajor(kTile, kk), idesc_s, 1);
                    }
                    mma_commit(&sh.s_full[w]);
                    mma_commit(&sh.kv_empty[stage]);
                    if (last) mma_commit(&sh.q_empty);
                }
                __syncwarp();
                next();
                return true;
            };
            // O += P V with the ring's next tile, one half of its keys after the other.
            auto outputs = [&](uint32_t add, bool last) {
                if (!wait(&sh.v_ready[stage], kv_phase)) return false;
                const uint64_t b = dv + stage * TILE;
#pragma unroll
                for (int half = 0; half < 2; half++) {
                    if (!wait(&sh.p_full[w][half], tiles & 1)) return false;
                    tc_fence_after();
                    if (elect_one()) {
#pragma unroll
                        for (int i = 0; i < kTile / 32; i++) {
                            const int kk = half * (kTile / 32) + i;
                            mma_bf16_ta(dout, ds + 8 * kk, b + kstep_mnmajor(kk), idesc_o, kk > 0 ? 1 : add);
                        }
                        if (half) {
                            mma_commit(&sh.kv_empty[stage]);
                            if (last) mma_commit(&sh.o_full[w]);
                        }
                    }
                    __syncwarp();
                }
                tiles++;
                next();
                return true;
            };
            while (ok) {
                const int i = np % kPieces;
                if (!wait(&sh.piece_full[i], (np / kPieces) & 1)) break;
                const Piece& pc = sh.pieces[i];
                const int end = uniform(pc.end), n = uniform(piece_tiles(pc)), pair = uniform(pc.pair);
                const int mine = uniform(group_share(pc, w, tok1).n);
                if (lane == 0) mbar_arrive(&sh.piece_empty[i]);
                np++;
                if (end) break;
                if (n == 0) continue;
                if (!wait(&sh.q_full, nq++ & 1)) break;
                if (mine == 0) commit(&sh.q_empty);
                if (pair) {
                    // Two row tiles on every key tile.
                    if (!(mine > 0 ? scores(w, mine == 1) : skip())) break;
                    rope ^= 1;
                    // What O held is read.
                    if (mine > 0 && !wait(&sh.o_free[w], (uses++ & 1) ^ 1)) break;
                    for (int j = 0; j < n && ok; j++) {
                        if (!(j < mine ? outputs(j > 0, j + 1 == mine) : skip())) break;
                        if (j + 1 == n) break;
                        if (!(j + 1 < mine ? scores(w, j + 2 == mine) : skip())) break;
                        rope ^= 1;
                    }
                } else {
                    // One row tile, key tiles in turn to the two groups; two of them lead.
                    for (int j = 0; j < 2 && j < n && ok; j++) {
                        if (!(j == w ? scores(0, mine == 1) : skip())) break;
                        rope ^= 1;
                    }
                    if (!ok || (mine > 0 && !wait(&sh.o_free[w], (uses++ & 1) ^ 1))) break;
                    for (int j = 0; j < n && ok; j++) {
                        const bool own = (j & 1) == w;
                        if (!(own ? outputs(j > 1, j + 2 >= n) : skip())) break;
                        if (j + 2 >= n) continue;
                        if (!(own ? scores(0, j + 4 >= n) : skip())) break;
                        rope ^= 1;
                    }
                }
            }
            // Products in flight, which write the tensor memory that is freed below and
            // arrive on this CTA's barriers, end before it leaves.
            commit(&sh.drained[w]);
            if (!__all_sync(0xffffffffu, mbar_wait(&sh.drained[w], 0, 1LL << 24))) ok = false;
            if (!ok) flags |= KDA_DEV_TIMEOUT;
        } else if (!C::TWO_ISSUE && warp == kMmaWarp) {
            // ------------------------------------------------------------ products
            // What this warp does between two products shows as idle tensor core.
            // All of it is uniform, so that stages and descriptors stay in uniform
            // registers, and one elected lane issues.
            int stage = 0, kv_phase = 0, q_phase = 0, np = 0;
            int tiles0 = 0, tiles1 = 0;  // parities of the groups' tiles so far
            constexpr uint32_t idesc_s = idesc_bf16(kTile, kTile, 0, 0);
            constexpr uint32_t idesc_o = idesc_bf16(kTile, D, 0, 1);
            const uint64_t dq = desc_kmajor(smem_addr(sq));
            const uint64_t dk = desc_kmajor(smem_addr(skv)), dv = desc_mnmajor(smem_addr(skv), kTile);
            constexpr uint32_t TILE = C::TILE_BYTES >> 4;  // a tile in descriptor units
            auto next = [&] {
                if (++stage == NS) {
                    stage = 0;
                    kv_phase ^= 1;
                }
            };
            auto wait = [&](uint64_t* bar, uint32_t parity) {
                if (!__all_sync(0xffffffffu, mbar_wait(bar, parity, kWaitClocks))) ok = false;
                return ok;
            };
            auto uniform = [](int x) { return __shfl_sync(0xffffffffu, x, 0); };
            auto scores = [&](int w, uint32_t qtile, uint32_t kstage) {  // S_w = Q_w K^T
                const uint64_t a = dq + qtile * TILE, b = dk + kstage * TILE;
                if (elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < D / 16; kk++)
                        mma_bf16(tbase + TM_S + w * kTile, a + kstep_kmajor(kTile, kk),
                                 b + kstep_kmajor(kTile, kk), idesc_s, kk > 0);
                    mma_commit(&sh.s_full[w]);
                }
                __syncwarp();
            };
            // O_w += P_w V over one half of the key tile
            auto outputs = [&](int w, uint32_t vstage, int half, uint32_t add) {
                const uint64_t b = dv + vstage * TILE;
                if (elect_one()) {
#pragma unroll
                    for (int i = 0; i < kTile / 32; i++) {
                        const int kk = half * (kTile / 32) + i;
                        mma_bf16_ta(tbase + TM_O + w * D, tbase + TM_S + w * kTile + 8 * kk,
                                    b + kstep_mnmajor(kk), idesc_o, kk > 0 ? 1 : add);
                    }
                }
                __syncwarp();
            };
            auto commit = [&](uint64_t* bar) {
                if (elect_one()) mma_commit(bar);
                __syncwarp();
            };
            struct Next {  // the piece after this one
                int end, n, pair, n0, n1;
            };
            auto take = [&](Next& x) {  // from the queue
                const int i = np % kPieces;
                if (!wait(&sh.piece_full[i], (np / kPieces) & 1)) return false;
                const Piece& pc = sh.pieces[i];
                x.end = uniform(pc.end);
                x.n = uniform(piece_tiles(pc));
                x.pair = uniform(pc.pair);
                x.n0 = uniform(group_share(pc, 0, tok1).n);
                x.n1 = uniform(group_share(pc, 1, tok1).n);
                if (lane == 0) mbar_arrive(&sh.piece_empty[i]);
                np++;
                return true;
            };
            // Group w's O may be written: what it held is read. Waited for once per
            // piece in which the group has key tiles.
            int uses0 = 0, uses1 = 0;
            auto o_free = [&](int w) { return wait(&sh.o_free[w], ((w ? uses1++ : uses0++) & 1) ^ 1); };
            auto half_by_half = [&](int w, int parity, uint32_t vs, uint32_t add) {
                if (!wait(&sh.p_full[w][0], parity)) return false;
                tc_fence_after();
                outputs(w, vs, 0, add);
                if (!wait(&sh.p_full[w][1], parity)) return false;
                tc_fence_after();
                outputs(w, vs, 1, 1);
                return true;
            };
            Next x{};
            take(x);
            bool primed = false;  // x's first scores are on their way
            while (ok && !x.end) {
                const int n = x.n;
                if (n == 0) {
                    if (!take(x)) break;
                    continue;
                }
                if (x.pair) {
                    // Two row tiles on every key tile. The last tile's step starts the
                    // next piece's first scores, if that is a pair too, as any other
                    // step starts the next tile's.
                    const int n0 = x.n0, n1 = x.n1;
                    if (!primed) {
                        if (!wait(&sh.q_full, q_phase)) break;
                        q_phase ^= 1;
                        if (!wait(&sh.kv_full[stage], kv_phase)) break;
                        tc_fence_after();
                        if (n0 > 0) scores(0, 0, stage);
                        if (n1 > 0) scores(1, 1, stage);
                        commit(&sh.kv_empty[stage]);
                        next();
                        if (n == 1) commit(&sh.q_empty);
                    }
                    primed = false;
                    for (int j = 0; j < n; j++) {
                        const int vs = stage;
                        if (!wait(&sh.v_ready[vs], kv_phase)) break;
                        next();
                        bool s0 = j + 1 < n0, s1 = j + 1 < n1;  // scores to start
                        if (j + 1 == n) {
                            if (!take(x)) break;
                            primed = !x.end && x.pair && x.n > 0;
                            s0 = primed && x.n0 > 0;
                            s1 = primed && x.n1 > 0;
                        }
                        const bool more = j + 1 < n || primed;
                        const int ks = stage;
                        bool have = false;
                        auto keys = [&] {  // the key tile (and the rows) of the next scores
                            if (have) return true;
                            have = true;
                            if (j + 1 == n) {
                                if (!wait(&sh.q_full, q_phase)) return false;
                                q_phase ^= 1;
                            }
                            if (!wait(&sh.kv_full[ks], kv_phase)) return false;
                            tc_fence_after();
                            return true;
                        };
                        if (j == 0 && n0 > 0 && !o_free(0)) break;
                        if (j < n0) {
                            if (!half_by_half(0, tiles0, vs, j > 0)) break;
                            tiles0 ^= 1;
                            if (j + 1 == n0) commit(&sh.o_full[0]);
                        }
                        if (s0) {
                            if (!keys()) break;
                            scores(0, 0, ks);
                        }
                        if (j == 0 && n1 > 0 && !o_free(1)) break;
                        if (j < n1) {
                            if (!half_by_half(1, tiles1, vs, j > 0)) break;
                            tiles1 ^= 1;
                            if (j + 1 == n1) commit(&sh.o_full[1]);
                        }
                        if (s1) {
                            if (!keys()) break;
                            scores(1, 1, ks);
                        }
                        commit(&sh.kv_empty[vs]);
                        if (more) {
                            commit(&sh.kv_empty[ks]);
                            next();
                        }
                        // the rows' last scores are issued
                        if (j + 2 == n || (j + 1 == n && primed && x.n == 1)) commit(&sh.q_empty);
                    }
                } else {
                    // One row tile, key tiles in turn to the two groups.
                    if (!wait(&sh.q_full, q_phase)) break;
                    q_phase ^= 1;
                    for (int j = 0; j < 2 && j < n; j++) {
                        if (!wait(&sh.kv_full[stage], kv_phase)) break;
                        tc_fence_after();
                        scores(j, 0, stage);
                        commit(&sh.kv_empty[stage]);
                        next();
                    }
                    if (n <= 2) commit(&sh.q_empty);
                    if (!ok || !o_free(0) || (n > 1 && !o_free(1))) break;
                    for (int j = 0; j < n && ok; j++) {
                        const int vs = stage, w = j & 1;
                        if (!wait(&sh.v_ready[vs], kv_phase)) break;
                        next();
                        const bool more = j + 2 < n;
                        const int ks = stage;
                        if (!half_by_half(w, w ? tiles1 : tiles0, vs, j > 1)) break;
                        tiles0 ^= w ^ 1;
                        tiles1 ^= w;
                        commit(&sh.kv_empty[vs]);
                        if (more) {
                            if (!wait(&sh.kv_full[ks], kv_phase)) break;
                            tc_fence_after();
                            scores(w, 0, ks);
                            commit(&sh.kv_empty[ks]);
                            next();
                            if (j + 3 == n) commit(&sh.q_empty);
                        } else {
                            commit(&sh.o_full[w]);
                        }
                    }
                    if (!ok || !take(x)) break;
                }
            }
            // Products in flight, which write the tensor memory that is freed below and
            // arrive on this CTA's barriers, end before it leaves.
            commit(&sh.drained[0]);
            if (!__all_sync(0xffffffffu, mbar_wait(&sh.drained[0], 0, 1LL << 24))) ok = false;
            if (!ok) flags |= KDA_DEV_TIMEOUT;
        } else if (warp == kEdgeWarp) {
            // ------------------------------------------------------------ V at the edge
            // It sees every tile of the ring go by (so that no phase of a barrier
            // passes unseen) and clears the V tiles of a piece from its edge on. The
            // products wait for V through this warp: one wait for every tile, where a
            // second one for those at the edge cost long prompts 0.5 %.
            int stage = 0, kv_phase = 0, np = 0;
            while (ok) {
                const int i = np % kPieces;
                warp_wait(ok, &sh.piece_full[i], (np / kPieces) & 1);
                if (!ok) break;
                const Piece pc = sh.pieces[i];
                __syncwarp();
                if (!C::TWO_ISSUE && lane == 0) mbar_arrive(&sh.piece_empty[i]);
                if (pc.end) break;
                if (lane < 8) sh.odd[i][lane] = 0;  // (those of the piece before are done with)
                __syncwarp();
                const int n = piece_tiles(pc), edge = edge_tile(pc, n), all = seen_by_all(pc);
                int j = 0;                             // the next V tile
                int v_at = pc.pair || n == 1 ? 1 : 2;  // and its place: one or two K tiles lead
                for (int at = 0; at < 2 * n; at++) {
                    warp_wait(ok, &sh.kv_full[stage], kv_phase);
                    if (!ok) break;
                    if (at == v_at) {
                        if (j >= edge) {
                            const int base = (pc.kt0 + j) * kTile;
                            const int r0 = max(all - base, 0), r1 = min(pc.keys - base, kTile);
                            clear_values<D>(skv + stage * C::TILE_BYTES, r0, r1, sh.odd[i],
                                            base + r0 - all);
                            fence_proxy_async_smem();
                        }
                        j++;
                        v_at = min(v_at + 2, 2 * n - 1);
                    }
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(&sh.v_ready[stage]);
                        mbar_arrive(&sh.kv_empty[stage]);
                    }
                    if (++stage == NS) {
                        stage = 0;
                        kv_phase ^= 1;
                    }
                }
                __syncwarp();
                if (!C::TWO_ISSUE) {
                    if (lane == 0) mbar_arrive(&sh.odd_full[i]);
                } else {  // what was cleared is added to the finished rows that see it
                    const uint32_t odd = lane < 8 ? sh.odd[i][lane] : 0;
                    if (__any_sync(0xffffffffu, odd != 0)) {
                        warp_wait(ok, &sh.rows_full[i], (np / kPieces) & 1);
                        if (ok)
                            flags |= add_cleared<D>(
                                p, pc, odd,
                                pc.slot >= 0 ? p.sp.ws + attn_slot_floats(p.sp.rows, D) * pc.slot : nullptr);
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sh.piece_empty[i]);
                }
                np++;
            }
            if (!ok) flags |= KDA_DEV_TIMEOUT;
        } else {
            // ------------------------------------------------------------ cleared values
            // In a warp of its own: beside the results' code it cost ragged prompts 3 %
            // without ever running.
            for (int np = 0; ok; np++) {
                const int i = np % kPieces;
                warp_wait(ok, &sh.piece_full[i], (np / kPieces) & 1);
                if (!ok) break;
                const Piece& pc = sh.pieces[i];  // (stays until this warp is done with it)
                if (pc.end) break;
                warp_wait(ok, &sh.odd_full[i], (np / kPieces) & 1);
                warp_wait(ok, &sh.rows_full[i], (np / kPieces) & 1);
                if (!ok) break;
                const uint32_t odd = lane < 8 ? sh.odd[i][lane] : 0;
                if (__any_sync(0xffffffffu, odd != 0))
                    flags |= add_cleared<D>(
                        p, pc, odd,
                        pc.slot >= 0 ? p.sp.ws + attn_slot_floats(p.sp.rows, D) * pc.slot : nullptr);
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.piece_empty[i]);
            }
            if (!ok) flags |= KDA_DEV_TIMEOUT;
        }
    } else if (warp < 8) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
        // ------------------------------------------------------------ softmax
        const int w = warp >> 2, quarter = warp & 3;
        const int row = 32 * quarter + lane;  // of the row tile, and the TMEM lane
        const int rtok = row / G;
        const uint32_t ts = tmem_at(tbase, 32 * quarter, TM_S + w * kTile);
        const uint32_t to = tmem_at(tbase, 32 * quarter, TM_O + w * D);
        int mine = 0;  // key tiles of this group so far
        auto wait = [&](uint64_t* bar, uint32_t parity) {
            warp_wait(ok, bar, parity);
            return ok;
        };
        for (int np = 0; ok; np++) {
            const int i = np % kPieces;
            if (!wait(&sh.piece_full[i], (np / kPieces) & 1)) break;
            const Piece& pc = sh.pieces[i];
            const int end = pc.end, pair = pc.pair, kt0 = pc.kt0;
            const Share g = group_share(pc, w, tok1);
            const int tok = (pair ? w * tok1 : 0) + rtok;
            const bool live = row < tok1 * G && tok < pc.ntok;
            // Keys this row sees; a row of nothing masks nothing (never stored).
            const int lim = live ? max(pc.pos0 + tok + 1, 0) : 0x7fffffff;
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.piece_empty[i]);
            if (end) break;
            const bool warp_live = __any_sync(0xffffffffu, live);
            float m = -INFINITY, l = 0.f;  // reference (c S) and sum
            for (int n = 0; n < g.n; n++) {
                const int base = (kt0 + g.first + n * g.step) * kTile;
                if (!wait(&sh.s_full[w], mine & 1)) break;
                tc_fence_after();
                if (warp_live) {
                    uint32_t xr[kTile];
                    float* x = reinterpret_cast<float*>(xr);
                    // The second half is on its way while the first is looked at.
                    tmem_ld64_async(ts, xr);
                    tmem_wait_ld();
                    tmem_landed<64>(xr);
                    tmem_ld64_async(ts + 64, xr + 64);
                    const bool edge = __any_sync(0xffffffffu, base + kTile > lim);
                    float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int b = 0; b < kTile; b += 64) {
                        if (b > 0) {
                            tmem_wait_ld();
                            tmem_landed<64>(xr + 64);
                        }
                        if (edge) {
#pragma unroll
                            for (int e = b; e < b + 64; e++)
                                x[e] = base + e < lim ? x[e] : -INFINITY;
                        }
#pragma unroll
                        for (int e = b; e < b + 64; e += 8)
#pragma unroll
                            for (int i = 0; i < 4; i++)
                                mx[i] = fmaxf(fmaxf(mx[i], x[e + i]), x[e + i + 4]);
                    }
                    const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * p.c;
                    if (n == 0) {
                        m = top;
                    } else if (__any_sync(0xffffffffu, live && top > m + kRaise)) {
                        const float mn = fmaxf(m, top);
                        const float a = mn == -INFINITY ? 1.f : ex2(m - mn);
                        m = mn;
                        l *= a;
                        // (S of this tile is there, so the products before it are done)
#pragma unroll
                        for (int b = 0; b < D; b += 32) {
                            float y[32];
                            tmem_ld32(to + b, y);
#pragma unroll
                            for (int e = 0; e < 32; e++) y[e] *= a;
                            tmem_st16(to + b, y);
                            tmem_st16(to + b + 16, y + 16);
                        }
                    }
                    const float ref = m == -INFINITY ? 0.f : m;
                    const float2 c2 = make_float2(p.c, p.c), ref2 = make_float2(-ref, -ref);
                    float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                    for (int b = 0; b < kTile; b += 32) {
                        float pk[16];
#pragma unroll
                        for (int e = 0; e < 32; e += 2) {
                            float2 u = fma2(make_float2(x[b + e], x[b + e + 1]), c2, ref2);
                            u.x = ex2(u.x);
                            u.y = ex2(u.y);
                            sum[(e >> 1) & 1] = add2(sum[(e >> 1) & 1], u);
                            // to bf16, as the product wants P in V's type (the sum is of
                            // the unrounded): o is off by 1.8e-3 to 2.3e-3 of its norm,
                            // 1.6e-3 to 1.7e-3 with P in fp32
                            pk[e / 2] = __uint_as_float(pack2(u.x, u.y));
                        }
                        tmem_st16(ts + b / 2, pk);
                        if (b == kTile / 2 - 32) {  // the second product may start on this half
                            tmem_wait_st();
                            tc_fence_before();
                            mbar_arrive(&sh.p_full[w][0]);
                        }
                    }
                    l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
                    tmem_wait_st();
                } else {
                    mbar_arrive(&sh.p_full[w][0]);
                }
                mine++;
                tc_fence_before();
                mbar_arrive(&sh.p_full[w][1]);
            }
            if (!wait(&sh.ml_free[w], (np & 1) ^ 1)) break;  // of the piece before
            sh.ml[w][row] = make_float2(m, l);
            mbar_arrive(&sh.ml_full[w]);
        }
        if (!ok) flags |= KDA_DEV_TIMEOUT;
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsResult));
        // ------------------------------------------------------------ results
        const int row = tid & 127;  // of the row tile, and the TMEM lane
        const int rtok = row / G, rhead = row % G;
        const uint32_t to = tmem_at(tbase, row & 96, TM_O);
        int done[2] = {0, 0};  // pieces with key tiles of each group so far
        for (int np = 0; ok; np++) {
            const int i = np % kPieces;
            warp_wait(ok, &sh.piece_full[i], (np / kPieces) & 1);
            if (!ok) break;
            const Piece pc = sh.pieces[i];
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.piece_empty[i]);
            if (pc.end) break;
            float* part = pc.slot >= 0 ? p.sp.ws + attn_slot_floats(p.sp.rows, D) * pc.slot : nullptr;
            const int n[2] = {group_share(pc, 0, tok1).n, group_share(pc, 1, tok1).n};
            // Two row tiles, one after the other; or the two halves of one.
#pragma unroll
            for (int w = 0; w < 2; w++) {
                if (w == 1 && !pc.pair) break;
                // Weights of O_w (and of O_1), and whether they hold anything: what a group
                // of no weight at all accumulated (0 x NaN) is left out, but a weight that
                // is zero only in 32 bits keeps the NaN or Inf of a seen value.
                float a0, a1 = 0.f;
                bool any0, any1 = false;
                float m, l;
                {
                    warp_wait(ok, &sh.ml_full[w], np & 1);
                    const float2 x = sh.ml[w][row];
                    mbar_arrive(&sh.ml_free[w]);
                    m = x.x;
                    l = x.y;
                    any0 = n[w] > 0 && l != 0.f;
                    if (n[w] > 0) warp_wait(ok, &sh.o_full[w], done[w]++ & 1);
                }
                if (w == 0 && !pc.pair) {
                    warp_wait(ok, &sh.ml_full[1], np & 1);
                    const float2 x = sh.ml[1][row];
                    mbar_arrive(&sh.ml_free[1]);
                    if (n[1] > 0) warp_wait(ok, &sh.o_full[1], done[1]++ & 1);
                    any1 = n[1] > 0 && x.y != 0.f;
                    const float mn = fmaxf(m, x.x);
                    a0 = m == -INFINITY ? 0.f : ex2(m - mn);
                    a1 = x.x == -INFINITY ? 0.f : ex2(x.x - mn);
                    // a NaN sum keeps its NaN through either weight
                    l = (l == 0.f ? 0.f : l * a0) + (x.y == 0.f ? 0.f : x.y * a1);
                    m = mn;
                    const float inv = l == 0.f ? 0.f : 1.f / l;
                    a0 *= inv;
                    a1 *= inv;
                } else {
                    a0 = l == 0.f ? 0.f : 1.f / l;
                }
                if (!ok) break;
                tc_fence_after();
                const int tok = w * tok1 + rtok, srow = w * kTile + row;
                const bool live = row < tok1 * G && tok < pc.ntok;
                const size_t at = ((size_t)pc.tok0 + tok) * p.s.Hkv * G + (size_t)pc.h * G + rhead;
                float fin = 0.f;  // NaN once a value is not finite
                if (__any_sync(0xffffffffu, live)) {
                    for (int b = 0; b < D; b += 16) {
                        float y[16];
                        if (n[w] > 0) {
                            tmem_ld16(to + w * D + b, y);
#pragma unroll
                            for (int e = 0; e < 16; e++) y[e] = any0 ? y[e] * a0 : 0.f;
                        } else {
#pragma unroll
                            for (int e = 0; e < 16; e++) y[e] = 0.f;
                        }
                        if (w == 0 && !pc.pair && n[1] > 0) {
                            float z[16];
                            tmem_ld16(to + D + b, z);
#pragma unroll
                            for (int e = 0; e < 16; e++) y[e] += any1 ? z[e] * a1 : 0.f;
                        }
#pragma unroll
                        for (int e = 0; e < 16; e++) fin = fmaf(y[e], 0.f, fin);
                        if (live) {
                            if (part) {
                                float4* dst = reinterpret_cast<float4*>(part + (size_t)srow * D + b);
#pragma unroll
                                for (int e = 0; e < 4; e++)
                                    dst[e] = make_float4(y[4 * e], y[4 * e + 1], y[4 * e + 2],
                                                         y[4 * e + 3]);
                            } else {
                                uint4* dst = reinterpret_cast<uint4*>(p.o + at * D + b);
#pragma unroll
                                for (int e = 0; e < 2; e++)
                                    dst[e] = make_uint4(pack2(y[8 * e], y[8 * e + 1]),
                                                        pack2(y[8 * e + 2], y[8 * e + 3]),
                                                        pack2(y[8 * e + 4], y[8 * e + 5]),
                                                        pack2(y[8 * e + 6], y[8 * e + 7]));
                            }
                        }
                    }
                }
                // The groups may go on to the next piece.
                tc_fence_before();
                if (n[w] > 0) mbar_arrive(&sh.o_free[w]);
                if (!pc.pair && n[1] > 0) mbar_arrive(&sh.o_free[1]);
                if (live) {
                    if (part)
                        part[(size_t)p.sp.rows * D + srow] = l == 0.f ? -INFINITY : m + log2f(l);
                    else if (p.lse)
                        p.lse[at] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718056f;
                }
                if (live && !(fin == 0.f)) flags |= KDA_DEV_NONFINITE;
            }
            if (!ok) break;
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.rows_full[i]);
        }
        if (!ok) flags |= KDA_DEV_TIMEOUT;
    }
    __syncwarp();
    report_flags(p.d_status, flags);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 0) tmem_dealloc(tbase, 512);
}

// Rows of packed tokens: [tokens][heads][d], boxes of 64 x heads x tokens.
bool make_rows(CUtensorMap* m, const void* ptr, int d, int heads, int tokens, long long stride,
               long long head, int box_heads, int box_tokens) {
    auto enc = tensor_map_encoder();
    if (!enc) return false;
    cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)tokens};
    cuuint64_t strides[2] = {(cuuint64_t)head * 2, (cuuint64_t)stride * 2};
    cuuint32_t box[3] = {64, (cuuint32_t)box_heads, (cuuint32_t)box_tokens};
    cuuint32_t es[3] = {1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(ptr), dims, strides, box,
               es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A cache: [pages][heads][page][d], boxes of 64 x (page or 128) tokens.
bool make_cache(CUtensorMap* m, const void* ptr, int d, int page, int heads, int pages) {
    auto enc = tensor_map_encoder();
    if (!enc) return false;
    cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)page, (cuuint64_t)heads, (cuuint64_t)pages};
    cuuint64_t strides[3] = {(cuuint64_t)d * 2, (cuuint64_t)page * d * 2,
                             (cuuint64_t)heads * page * d * 2};
    cuuint32_t box[4] = {64, (cuuint32_t)(page < kTile ? page : kTile), 1, 1};
    cuuint32_t es[4] = {1, 1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(ptr), dims, strides, box,
               es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int DQ, int D>
cudaError_t launch_t(const AttnArgs& a) {
    const int G = a.Hq / a.Hkv, tok1 = kTile / G;
    int dev = 0;
    const int nsm = device_sms(&dev);
    if (nsm == 0) return cudaErrorNoDevice;
    TcAttnParams p{};
    p.s = {a.cu_q, a.kv_len, a.N, a.total_q, a.max_q,
           attn_kv_cap(a), a.Hkv, G, tok1, 2 * tok1,
           kTile, kCostSingle, kCostPair, kItemKeys};
    p.sp = attn_tc_split(a.N, a.total_q, a.max_q, a.kv_len ? p.s.kv_cap : a.max_q, !a.kv_len, DQ > D,
                         a.Hq, a.Hkv, nsm);
    if (p.sp.ctas && a.ws && a.ws_bytes >= attn_split_bytes(p.sp, D)) p.sp.ws = a.ws;
    p.block_table = a.block_table;
    p.v = static_cast<const __nv_bfloat16*>(a.v);
    p.o = static_cast<__nv_bfloat16*>(a.o);
    p.lse = a.lse;
    p.v_stride = a.v_stride;
    p.v_head = a.v_head;
    p.num_pages = a.num_pages;
    p.page = a.page;
    p.max_pages = a.max_pages;
    p.box_q = a.max_q < tok1 ? a.max_q : tok1;
    p.c = a.scale * 1.44269504089f;
    p.d_status = a.d_status;

    TcMaps<DQ - D> m;
    bool ok = make_rows(&m.q, a.q, DQ, a.Hq, a.total_q, a.q_stride, a.q_head, G, p.box_q);
    if (a.kv_len)
        ok = ok && make_cache(&m.k, a.k, D, a.page, a.Hkv, a.num_pages) &&
             make_cache(&m.v, a.v, D, a.page, a.Hkv, a.num_pages);
    else
        ok = ok && make_rows(&m.k, a.k, D, a.Hkv, a.total_q, a.k_stride, a.k_head, 1, kTile) &&
             make_rows(&m.v, a.v, D, a.Hkv, a.total_q, a.v_stride, a.v_head, 1, kTile);
    if constexpr (DQ > D) ok = ok && make_rows(&m.r, a.k_r, DQ - D, 1, a.total_q, a.kr_stride, DQ - D, 1, kTile);
    if (!ok) return cudaErrorInvalidValue;
    // Whole items, when the next one is asked for. With keys of up to two tiles the answer's way shows if
    // it is asked for among the loads; with more, a CTA with a long item took a further one that others
    // could have begun. Measured, early against late, us (heads of 128 channels): 4864 prompts of 64 tokens x 2
    // heads 321/332, 1000 of 128 x 8 246/251, 500 of 200 x 8 190/191, of 1 to 128 x 8 on 2 2000 223/221; 256
    // of 384 x 8 235/222, 8192 tokens x 8 119/88 (x 8 of 192 channels 182/146).
    const bool early = !p.sp.ws && (a.kv_len ? p.s.kv_cap : a.max_q) <= 2 * kTile;
    auto kernel = early ? kda_attn_tc_kernel<DQ, D, true> : kda_attn_tc_kernel<DQ, D, false>;
    static std::atomic<uint64_t> ready[2];
    cudaError_t e = allow_shared(kernel, tc_smem<DQ, D>(), ready[early], dev);
    if (e != cudaSuccess) return e;
    const long long grid = p.sp.ws ? p.sp.ctas : attn_items_bound(p.s);
    if (grid >= 1LL << 31) return cudaErrorInvalidValue;
    e = launch_dependent(kernel, dim3((unsigned)grid), dim3(kThreadsTc), tc_smem<DQ, D>(), a.stream,
                         m, p);
    if (e != cudaSuccess || !p.sp.ws) return e;
    return launch_attn_combine(p.sp, a.Hkv, G, D, kTile, a.o, a.lse, KDA_BF16, a.d_status, a.stream);
}

}  // namespace

// Whole items or ranges. Ranges balance any lengths, but cost a second launch,
// the parts' stores and a longer start: about 10 us over single tokens, 25 us over
// pairs of row tiles, and with one issuing warp a tile takes a quarter longer in them. Measured,
// ranges against whole items, us (Hq / Hkv heads; 32 / 8 where none are given):
//                                             d = 128      d = 64
//   one token, 1 x 1024                         16/12       17/12
//     1 x 2048, 1 x 4096                  18/17, 21/28  19/16, 22/24
//     16 x 2048, 64 x 2048                36/27, 94/86  23/15, 57/54
//     lengths to 8192, 32 requests                92/95       56/64
//     256 requests                              606/588     322/322
//   prompts, 2048, 4 x 2048              55/31, 141/106 45/27, 117/86
//     8192                                      340/311     293/265
//     8 / 2, 4096, 8192                    51/48, 109/88  43/45, 95/82
//     4 / 1, 3000, 4096, 8192     35/40, 42/49, 70/87  27/34, 31/44, 58/80
//     4 / 4, 8192, 12288, 16384 72/87, 120/127, 186/170  60/80, 102/116, 155/152
//     5 / 5, 8192, 12288                  96/102, 167/129  68/80, 119/116
//     6 / 6, 4096, 8192, 12288    48/49, 93/89, 166/135  38/44, 79/80, 136/116
//     2 / 2, 8192 alone, with 3000 and 500    50/87, 54/86  39/80, 43/80
//   512 new tokens over 32768                   195/323     148/304
//   2 x 4096 over 16384                       1145/1125     913/917
// The rule is within 5 % of the better side of these. With shared key channels (192 of them, two issuing
// warps) there is no such quarter: 6 heads x 8192 132/147, 8 x 4096 67/77, 7 x 8192 149/148, 8 x 8192
// 166/148, 4 x 16384 284/284, 6 x 12288 248/217.
AttnSplit attn_tc_split(int N, int total_q, int max_q, long long max_keys, bool prompt, bool shared,
                        int Hq, int Hkv, int nsm) {
    AttnSplit sp{};
    if (N == 0 || total_q == 0 || max_q == 0 || Hkv == 0 || nsm == 0) return sp;
    const int G = Hq / Hkv, tok1 = kTile / G;
    if (max_keys <= KDA_ATTN_SHORT_KEYS) return sp;
    const long long items = (long long)total_q / (2 * tok1) * Hkv;
    if (max_q > tok1) {
        // Prompts: half the longest item is the mean one. Whole unless the longest
        // passes an even share of all of them by more than what ranges cost, 17 tiles.
        const long long longest = (max_keys + kTile - 1) / kTile, share = longest * items / (2 * nsm);
        if (prompt ? longest - share - (shared ? 0 : share / 4) <= 17 : items >= 8LL * nsm) return sp;
    }
    sp.ctas = nsm;
    sp.least = 2 * kCostPair * kTile;
    sp.rows = max_q <= tok1 ? (max_q * G + 3) & ~3 : 2 * kTile;  // whole 16-byte vectors
    return sp;
}

cudaError_t launch_attn_tc(const AttnArgs& a) {
    if (a.dr) return launch_t<192, 128>(a);
    return a.d == 128 ? launch_t<128, 128>(a) : launch_t<64, 64>(a);
}

}  // namespace kda
