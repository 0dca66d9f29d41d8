// Attention over a paged cache of latents on the 5th-generation tensor cores (bf16): all
// heads share one cached row c_j a token, 512 latent channels and DR rotated ones.
//
//     S = Q C^T,  P = 2^{c S - m},  O^T = C_l^T P^T,  o = O / l,   c = scale log2 e
//
// with C_l the latent channels, m a running reference of each row's largest c S (raised
// only when the maximum passes it by more than 8) and l its running sum.
//
// Layout. A row of O has 512 fp32 channels: 64 rows take half of the tensor memory if the
// channels are its lanes, four accumulators of 128 channels x 64 rows, and two tiles of scores
// fit beside them; of 32 rows two O do. So the first product has the rows (token, head) as M (64, of
// which 32 or 64 count) and 32 keys as N, the second the channels as M (4 x 128) and the rows as
// N. One tile of 32 cached rows in shared memory is the K-major B operand of the first and the
// MN-major A operand of the second; P goes through shared memory as its B operand. At few rows
// the second product is as narrow as they are (a multiple of 16).
//
// One CTA per SM:
//   warps 0..3   softmax, one row of S per thread (64-row accumulators use 16 lanes of
//                each warp's 32), and the edge (below)
//   warps 4..7   the results
//   warps 8, 9   issue the first and the second products
//   warp 10      issues the loads
//   warp 11      finds the work, ahead of the loads: from a request's lengths to its first
//                tile takes some 5000 clocks, which stood between any two items before
//
// A key past a row's last one gets P = 0 by a select on S. 0 x NaN is NaN, so before the
// second product the softmax warps clear in shared memory what some rows must not see:
// rows of keys past the item's last (stale slots) whole; of the keys that only some rows
// see the values that are not finite. Those are noted and added to the rows that see them.
//
// What bounds it. Few rows: HBM. 256 single tokens of 32 heads over 1.06 M cached tokens take 201 us,
// 6.1 TB/s (90 % of a copy's rate; some 15 us are the start, the parts and their join). Full
// tiles: the products, whose operands come out of shared memory. An MMA of 64 x 32 takes 30 clocks, one of
// 128 x 64 49, so a tile of 64 rows and 32 keys 36 x 30 + 8 x 49 = 1470, which is 880 TFLOP/s;
// 2 x 4 draft tokens of 32 heads over 262147 keys take 171 us, 850 TFLOP/s with the join. Tiles of 64 keys
// would take 2080 clocks for twice the keys, but only two of them fit beside 64 rows, and
// their loads are then waited for (202 us against 182 at the time). 16 heads fill half of a tile's 32 rows,
// which costs nothing while HBM is the bound.
#include <atomic>

#include "kda_attn.cuh"
#include "kda_host.cuh"
#include "sm100_ptx.cuh"
#include "tensor_map.cuh"

namespace kda {
namespace {

using namespace ptx;

constexpr int kThreadsTc = 384;
constexpr int kScoreWarp = 8, kOutWarp = 9, kLoadWarp = 10, kPlanWarp = 11;
constexpr int kDL = kLatentDim;
constexpr int kUnits = kDL / 128;        // units of a tile's latents
constexpr int kPieces = 4;               // pieces announced ahead
constexpr int kAskAhead = 4;             // tiles left to load of an item when the next one is asked for
constexpr int kItemKeys = 256;           // what an item costs beside its keys, in keys
constexpr long long kWaitClocks = 1LL << 33;  // limit of a wait (about 4 s)
// Log2 growth of a row maximum that moves its reference: P then stays below 2^8, and a raise costs a
// pass over the results.
constexpr float kRaise = 8.f;
constexpr int kMaxTiles = 6;             // key tiles in shared memory, at most
constexpr int kKeys = 32;                // keys of a key tile

// RT rows of a row tile.
template <int DR, int RT>
struct TcCfg {
    static constexpr int BLOCKS = (kDL + DR) / 64;             // of 64 channels, of a row
    static constexpr int QBLOCK = RT * 128, KBLOCK = kKeys * 128;  // bytes of one
    static constexpr int Q = BLOCKS * QBLOCK, TILE = BLOCKS * KBLOCK;
    static constexpr int P = RT * 128;
    static constexpr int NT = (225 * 1024 - Q - P) / TILE;      // key tiles in shared memory
    static constexpr int TILES = Q + NT * TILE + P;
    static constexpr int NO = RT == 32 ? 2 : 1;                 // results in tensor memory
    static constexpr uint32_t TM_O = 0, TM_S = NO * kUnits * RT;  // its columns
    static_assert(NT >= 2 && NT <= kMaxTiles, "key tiles");
};

struct LatentTcParams {
    AttnShape s;
    AttnSplit sp;
    const int* block_table;
    const __nv_bfloat16* cache;
    __nv_bfloat16* o;
    float* lse;
    int num_pages, page, max_pages;
    int box_q;  // tokens of a Q load
    float c;    // scale log2 e
    int* d_status;
};

// A range of key tiles of one item.
struct Piece {
    int r, h;
    int tok0, ntok;  // packed token of row 0; tokens
    int pos0;        // keys that row 0's token sees, less one (may be negative)
    int kv, keys;    // keys of the request; those that the item's last token sees
    int kt0, kt1;    // key tiles
    int slot;        // where a part of an item goes; -1: the whole item
    int end;         // no more pieces
};
__device__ __forceinline__ int piece_tiles(const Piece& p) {
    return max(min(p.kt1, (p.keys + kKeys - 1) / kKeys) - p.kt0, 0);
}
// Keys that every row of the item sees: those of its first token.
__device__ __forceinline__ int seen_by_all(const Piece& p) { return min(max(p.pos0 + 1, 0), p.keys); }

struct Shared {
    uint64_t full[kMaxTiles], empty[kMaxTiles];  // of each key tile in shared memory
    uint64_t s_full[2], s_read[2], p_full, pv_done;
    uint64_t q_full, q_empty;
    uint64_t piece_full[kPieces], piece_empty[kPieces], piece_taken[kPieces];  // (taken: its last loads are due)
    uint64_t sums_full[kPieces], o_full[kPieces];  // of a piece: its rows' sums, its products
    uint64_t o_free[2];   // a result in tensor memory is read
    uint64_t next_full;   // the number of the next whole item
    uint64_t drained[2];  // all products of either kind have ended
    alignas(16) uint4 next;
    Piece pieces[kPieces];
    alignas(16) float factor[64];        // of the rows of a raised reference
    alignas(16) float inv[kPieces][64];  // 1 / l of a piece's rows; 0: a row without weight, or none
    int row_at[64];                      // row of o of the tile's rows, from its first
    uint32_t odd[kPieces][2];  // bit i: key seen_by_all + i has values that were cleared
    long long sum[kThreadsTc / 32];
    uint32_t tmem;
};
template <typename C>
constexpr int tc_smem() {
    static_assert(C::TILES + sizeof(Shared) <= 227 * 1024, "shared memory of a CTA");
    static_assert(kAttnGroups * 8 <= C::P, "cost groups fit P's tile");
    return C::TILES + (int)sizeof(Shared);
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
__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_addr(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}
// A bounded wait by a whole warp, with one outcome for all its lanes.
__device__ __forceinline__ void warp_wait(bool& ok, uint64_t* bar, uint32_t parity) {
    if (ok) ok = mbar_wait(bar, parity, kWaitClocks);
    ok = __all_sync(0xffffffffu, ok);
}
__device__ __forceinline__ bool warp_test(uint64_t* bar, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_test(bar, parity));
}
// The four softmax warps together.
__device__ __forceinline__ void wg_sync() { asm volatile("barrier.cta.sync 1, 128;" ::: "memory"); }
__device__ __forceinline__ bool wg_or(bool x) {
    uint32_t y;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.or.pred q, 1, 128, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(y)
        : "r"((uint32_t)x)
        : "memory");
    return y != 0;
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

template <int DR, int RT>
__global__ void __launch_bounds__(kThreadsTc, 1)
    kda_latent_tc_kernel(const __grid_constant__ CUtensorMap map_q,
                         const __grid_constant__ CUtensorMap map_c,
                         const __grid_constant__ LatentTcParams p) {
    using C = TcCfg<DR, RT>;
    constexpr int NT = C::NT;
    extern __shared__ __align__(1024) unsigned char sm[];  // 128-byte swizzle: 1024-byte tiles
    unsigned char* sq = sm;
    unsigned char* skv = sm + C::Q;
    unsigned char* sp = skv + NT * C::TILE;
    Shared& sh = *reinterpret_cast<Shared*>(sm + C::TILES);
    long long* groups = reinterpret_cast<long long*>(sp);  // before the first piece
    if (smem_addr(sm) & 1023u) {  // never, by the declaration above
        if (threadIdx.x == 0 && p.d_status) atomicOr(p.d_status, KDA_DEV_TIMEOUT);
        return;
    }
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // uniform, and known to be
    const int G = p.s.G, Hq = p.s.Hkv * G;
    if (warp == kLoadWarp) {
        if (lane < NT) {
            mbar_init(&sh.full[lane], 1);
            mbar_init(&sh.empty[lane], 1);
        }
        if (lane < 2) {
            mbar_init(&sh.s_full[lane], 1);
            mbar_init(&sh.s_read[lane], 4);
            mbar_init(&sh.drained[lane], 1);
            mbar_init(&sh.o_free[lane], 128);
        }
        if (lane < kPieces) {
            mbar_init(&sh.piece_full[lane], 1);
            mbar_init(&sh.piece_empty[lane], 11);  // softmax 4, products 2, results 4, loads
            mbar_init(&sh.piece_taken[lane], 1);
            mbar_init(&sh.sums_full[lane], 128);
            mbar_init(&sh.o_full[lane], 1);
        }
        if (lane == 0) {
            mbar_init(&sh.p_full, 128);
            mbar_init(&sh.pv_done, 1);
            mbar_init(&sh.q_full, 1);
            mbar_init(&sh.q_empty, 1);
            mbar_init(&sh.next_full, 1);
            prefetch_tensormap(&map_q);
            prefetch_tensormap(&map_c);
        }
        fence_mbarrier_init();
    }
    if (warp == kScoreWarp) {
        tmem_alloc(&sh.tmem, 512);
        tmem_relinquish();
    }
    if (tid < RT) sh.row_at[tid] = tid / G * Hq + tid % G;
    tc_fence_before();
    pdl_wait();
    // Cost of this CTA's range (split items); also the barrier after the setup.
    long long each = 0;
    if (p.sp.ws) each = attn_cost_each<kThreadsTc>(p.s, p.sp.ctas, p.sp.least, groups, sh.sum);
    __syncthreads();
    // The join's CTAs may take their places and wait. (Not before this CTA has its tensor memory: a kernel that
    // took some and waited for this one could hold what this one needs.)
    pdl_launch();
    tc_fence_after();
    const uint32_t tbase = sh.tmem;
    int flags = 0;
    bool ok = true;

    if (warp == kLoadWarp) {
        // ------------------------------------------------------------ loads
        int tile = 0, slot = 0, phase = 0;  // key tiles so far; the next one's place
        int nq = 0;                         // row tiles so far
        bool q_pending = false;
        const int log2_page = __ffs(p.page) - 1;
        const int log2_per = p.page < kKeys ? __ffs(kKeys) - 1 - log2_page : 0, per = 1 << log2_per;  // pages of a tile
        auto page_id = [&](const Piece& pc, int kt) {  // of part `lane` of a tile
            int id = p.num_pages;  // past the keys, or no page: beyond the cache, which loads zeros
            const int j = kt * kKeys + (lane << log2_page);
            if (lane < per && j < pc.kv) {
                id = p.block_table[(size_t)pc.r * p.max_pages + (j >> log2_page)];
                if (id < 0 || id >= p.num_pages) {
                    id = p.num_pages;
                    flags |= KDA_DEV_PAGES;
                }
            }
            return id;
        };
        auto load_q = [&](const Piece& pc) {
            if (lane == 0) mbar_arrive_expect_tx(&sh.q_full, C::BLOCKS * p.box_q * G * 128);
            __syncwarp();
            if (lane < C::BLOCKS)
                tma_load_3d(sq + lane * C::QBLOCK, &map_q, &sh.q_full, 64 * lane, pc.h * G, pc.tok0);
            nq++;
            q_pending = false;
        };
        // A free place for a tile; the rows of a new piece are loaded as soon as theirs is.
        auto wait_place = [&](const Piece& pc, uint64_t* bar, uint32_t parity) {
            if (q_pending) {
                const long long t0 = clock64();
                while (ok && q_pending && !warp_test(bar, parity)) {
                    if (warp_test(&sh.q_empty, (nq & 1) ^ 1)) load_q(pc);
                    else if (clock64() - t0 > kWaitClocks) ok = false;
                    ok = __all_sync(0xffffffffu, ok);
                }
            }
            warp_wait(ok, bar, parity);
            return ok;
        };
        int id_ahead = 0;
        bool ahead = false;  // id_ahead: of the next piece's first tile
        for (int np = 0; ok; np++) {
            const int i = np % kPieces;
            warp_wait(ok, &sh.piece_full[i], (np / kPieces) & 1);
            if (!ok) break;
            const Piece pc = sh.pieces[i];
            __syncwarp();
            const int n = piece_tiles(pc);
            if (lane == 0) {
                if (n <= kAskAhead) mbar_arrive(&sh.piece_taken[i]);
                mbar_arrive(&sh.piece_empty[i]);
            }
            if (pc.end) break;
            if (n == 0) continue;
            q_pending = true;
            int id = ahead ? id_ahead : page_id(pc, pc.kt0);
            ahead = false;
            for (int j = 0; j < n; j++) {
                if (lane == 0 && j > 0 && j == n - kAskAhead) mbar_arrive(&sh.piece_taken[i]);
                const int kt = pc.kt0 + j;
                int next_id = 0;
                if (j + 1 < n) {
                    next_id = page_id(pc, kt + 1);
                } else if (const int k = (np + 1) % kPieces; warp_test(&sh.piece_full[k], ((np + 1) / kPieces) & 1)) {
                    const Piece& nx = sh.pieces[k];
                    ahead = !nx.end && piece_tiles(nx) > 0;
                    if (ahead) id_ahead = page_id(nx, nx.kt0);
                }
                if (!wait_place(pc, &sh.empty[slot], phase ^ 1)) break;
                if (lane == 0) mbar_arrive_expect_tx(&sh.full[slot], C::TILE);
                __syncwarp();
                // All blocks together, so that DRAM sees whole rows.
                for (int i0 = 0; i0 < C::BLOCKS << log2_per; i0 += 32) {
                    const int x = i0 + lane, blk = x >> log2_per, part = x & (per - 1);
                    const int page = __shfl_sync(0xffffffffu, id, part);
                    if (blk < C::BLOCKS)
                        tma_load_3d(skv + slot * C::TILE + blk * C::KBLOCK + (part << log2_page) * 128, &map_c,
                                    &sh.full[slot], 64 * blk, (kt * kKeys) & (p.page - 1), page);
                }
                tile++;
                if (++slot == NT) {
                    slot = 0;
                    phase ^= 1;
                }
                if (q_pending) {
                    warp_wait(ok, &sh.q_empty, (nq & 1) ^ 1);
                    if (!ok) break;
                    load_q(pc);
                }
                id = next_id;
            }
        }
        if (!ok) {
            flags |= KDA_DEV_TIMEOUT;
            // copies in flight land before the CTA leaves
            for (int i = 0; i < NT && i < tile; i++) {
                slot = (slot ? slot : NT) - 1;  // the last tiles, backwards
                phase ^= slot == NT - 1;
                mbar_wait(&sh.full[slot], phase, 1LL << 24);
            }
            if (nq) mbar_wait(&sh.q_full, (nq - 1) & 1, 1LL << 24);
        }
    } else if (warp == kPlanWarp) {
        // ------------------------------------------------------------ work
        int np = 0, asked = 0;  // pieces announced; items asked for
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
        auto piece_of = [&](int r, const AttnReq& q, int h, int t) {
            Piece pc;
            pc.r = r;
            pc.h = h;
            const int at = t * q.tok;
            pc.tok0 = q.q0 + at;
            pc.ntok = min(q.tok, q.q_len - at);
            pc.pos0 = q.kv - q.q_len + at;
            pc.kv = q.kv;
            pc.keys = attn_item_keys(q, t);
            pc.kt0 = 0;
            pc.kt1 = attn_item_tiles(p.s, q, t);
            pc.slot = -1;
            pc.end = 0;
            return pc;
        };
        // Whole items, taken over from CTAs that have not started, or the tiles that start
        // in [cur, end), item by item.
        AttnReq q{};
        int r = 0, h = 0, t = 0, first = 0;
        long long in;
        const bool split = p.sp.ws != nullptr;
        long long cur = split ? blockIdx.x * each : blockIdx.x;
        const long long end = cur + each;
        long long start = cur;
        bool have = false;  // (q, h, t, first) is where `cur` is
        // One CTA reports on the lengths of all requests: the one that has item 0.
        bool reports = blockIdx.x == 0;
        AttnWalk walk;
        if (split) {
            walk = attn_walk_at(p.s, groups, cur);
            AttnCut cut{each, 0, 0, 0, 0, 0, 0, 0};
            have = attn_first_tile(p.s, walk, &cur, &r, &q, &h, &t, &first) && cur < end;
            start = cur;
            if (have) {
                cut.cost = q.cost * kKeys;
                cut.u0 = cur - (long long)first * cut.cost;
                cut.tok0 = q.q0 + t * q.tok;
                cut.ntok = min(q.tok, q.q_len - t * q.tok);
                cut.h = h;
                cut.tile = first;
                cut.n = attn_item_tiles(p.s, q, t);
            }
            if (lane == 0) attn_cuts(p.sp, kDL)[blockIdx.x] = cut;
            if (!have) cur = end;
        }
        while (ok && (!split || cur < end)) {
            if (!split && cur < walk.base) walk = AttnWalk{};
            if (!have) {
                have = split ? attn_first_tile(p.s, walk, &cur, &r, &q, &h, &t, &first)
                             : attn_find<false>(p.s, walk, cur, &r, &q, &in);
                if (!split && have) {
                    t = q.nqt - 1 - (int)(in / p.s.Hkv);
                    h = (int)(in % p.s.Hkv);
                    have = !q.bad;
                }
            }
            if (have) {
                Piece pc = piece_of(r, q, h, t);
                if (split) {
                    const int n = pc.kt1;
                    const long long u0 = cur - (long long)first * q.cost * kKeys;
                    pc.kt0 = first;
                    pc.kt1 = attn_tiles_until(p.s, q, u0, n, end);
                    if (pc.kt1 - pc.kt0 < n) pc.slot = 2 * blockIdx.x + (cur > start ? 1 : 0);
                    cur = pc.kt1 < n ? end
                                     : u0 + attn_cost_before(p.s, q, t + 1) - attn_cost_before(p.s, q, t);
                    first = 0;
                    if (++t == q.nqt) {
                        t = 0;
                        h++;
                    }
                    have = h < p.s.Hkv;
                }
                announce(pc);
                // Another item is asked for when this one's last loads are due: not before, or it
                // would wait here while other CTAs have nothing to do.
                if (!split) warp_wait(ok, &sh.piece_taken[(np - 1) % kPieces], ((np - 1) / kPieces) & 1);
            } else if (split) {
                break;
            }
            if (!split && ok) {
                have = false;
                if (lane == 0) {
                    mbar_arrive_expect_tx(&sh.next_full, 16);
                    clc_try_cancel(&sh.next, &sh.next_full);
                }
                asked++;
                __syncwarp();
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
            if (asked) mbar_wait(&sh.next_full, (asked - 1) & 1, 1LL << 24);  // an answer on its way lands
        }
    } else if (warp == kScoreWarp || warp == kOutWarp) {
        // ------------------------------------------------------------ products
        // What a warp does between two products shows as idle tensor core, so the two kinds
        // have a warp each, and a tile's are issued in one go, by one lane, from
        // registers known to be uniform.
        const bool scores = warp == kScoreWarp;
        constexpr uint32_t idesc_s = idesc_bf16(64, kKeys, 0, 0);  // (rows past RT: whatever follows)
        const uint64_t dq = desc_kmajor(smem_addr(sq)), dk = desc_kmajor(smem_addr(skv));
        const uint64_t dp = desc_kmajor(smem_addr(sp)), dv = desc_mnmajor(smem_addr(skv), kKeys);
        constexpr uint32_t QBLOCK = C::QBLOCK >> 4, KBLOCK = C::KBLOCK >> 4, TILE = C::TILE >> 4;  // descriptor units
        int t = 0, slot = 0, phase = 0, nq = 0;  // tiles so far; the next one's place; pieces with tiles
        auto wait = [&](uint64_t* bar, uint32_t parity) {
            if (!__all_sync(0xffffffffu, mbar_wait(bar, parity, kWaitClocks))) ok = false;
            return ok;
        };
        for (int np = 0; ok; np++) {
            const int i = np % kPieces;
            if (!wait(&sh.piece_full[i], (np / kPieces) & 1)) break;
            const Piece& pc = sh.pieces[i];
            const int end = __shfl_sync(0xffffffffu, pc.end, 0);
            const int n = __shfl_sync(0xffffffffu, piece_tiles(pc), 0);
            const int nrow = __shfl_sync(0xffffffffu, (pc.ntok * G + 15) & ~15, 0);
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.piece_empty[i]);
            if (end) break;
            if (scores) {
                if (n > 0 && !wait(&sh.q_full, nq++ & 1)) break;
                for (int j = 0; j < n; j++, t++) {
                    if (!wait(&sh.full[slot], phase)) break;
                    if (!wait(&sh.s_read[t & 1], ((t >> 1) & 1) ^ 1)) break;
                    tc_fence_after();
                    const uint64_t b = dk + (uint32_t)slot * TILE;
                    const uint32_t d = tbase + C::TM_S + (t & 1) * kKeys;
                    if (elect_one()) {
#pragma unroll
                        for (int c = 0; c < C::BLOCKS; c++)
#pragma unroll
                            for (int kk = 0; kk < 4; kk++)
                                mma_bf16(d, dq + (uint32_t)c * QBLOCK + 2 * kk, b + (uint32_t)c * KBLOCK + 2 * kk, idesc_s,
                                         c > 0 || kk > 0);
                        mma_commit(&sh.s_full[t & 1]);
                        if (j + 1 == n) mma_commit(&sh.q_empty);
                    }
                    __syncwarp();
                    if (++slot == NT) {
                        slot = 0;
                        phase ^= 1;
                    }
                }
            } else {
                const uint32_t idesc = idesc_bf16(128, 16, 1, 0) + (((uint32_t)(nrow >> 3) - 2) << 17);
                const int buf = nq % C::NO;
                const uint32_t d = tbase + C::TM_O + buf * kUnits * RT;
                if (n > 0 && !wait(&sh.o_free[buf], ((nq++ / C::NO) & 1) ^ 1)) break;
                for (int j = 0; j < n; j++, t++) {
                    if (!wait(&sh.p_full, t & 1)) break;
                    tc_fence_after();
                    const uint64_t a = dv + (uint32_t)slot * TILE;
                    if (elect_one()) {
#pragma unroll
                        for (int u = 0; u < kUnits; u++)
#pragma unroll
                            for (int kk = 0; kk < kKeys / 16; kk++)
                                mma_bf16(d + u * RT, a + (uint32_t)u * 2 * KBLOCK + kstep_mnmajor(kk),
                                         dp + 2 * kk, idesc, j > 0 || kk > 0);
                        mma_commit(&sh.empty[slot]);
                        mma_commit(&sh.pv_done);
                        if (j + 1 == n) mma_commit(&sh.o_full[i]);
                    }
                    __syncwarp();
                    if (++slot == NT) slot = 0;
                }
            }
        }
        // Products in flight, which write the tensor memory that is freed below and
        // arrive on this CTA's barriers, end before it leaves.
        if (elect_one()) mma_commit(&sh.drained[scores]);
        __syncwarp();
        if (!__all_sync(0xffffffffu, mbar_wait(&sh.drained[scores], 0, 1LL << 24))) ok = false;
        if (!ok) flags |= KDA_DEV_TIMEOUT;
    } else if (warp < 4) {
        // ------------------------------------------------------------ softmax
        // Row 16 w + i of a 64-row accumulator is lane 32 w + i.
        const int row = 16 * warp + (lane & 15), rtok = row / G;
        const bool rows_here = 16 * warp < RT;
        const uint32_t tlane = tmem_at(tbase, 32 * warp, 0);
        int t = 0, slot = 0, phase = 0, buf = 0;  // tiles so far; the current one's place; O's
        // These warps meet at barriers, so after a wait that gave up they go on without
        // waiting to where all of them stop.
        for (int np = 0;; np++) {
            const int i = np % kPieces;
            warp_wait(ok, &sh.piece_full[i], (np / kPieces) & 1);
            if (tid < 2) sh.odd[i][tid] = 0;  // (its last piece is done with)
            if (wg_or(!ok)) {
                ok = false;
                break;
            }
            const Piece pc = sh.pieces[i];
            if (pc.end) break;
            const int n = piece_tiles(pc), all = seen_by_all(pc);
            const bool live = lane < 16 && row < pc.ntok * G;  // (at most RT rows)
            // Keys this row sees; a row of nothing masks nothing (never stored).
            const int lim = live ? max(pc.pos0 + rtok + 1, 0) : 0x7fffffff;
            const uint32_t to = tlane + C::TM_O + buf * kUnits * RT;
            float m = -INFINITY, l = 0.f;  // reference (c S) and sum
            for (int j = 0; j < n; j++, t++) {
                const int base = (pc.kt0 + j) * kKeys;
                warp_wait(ok, &sh.s_full[t & 1], (t >> 1) & 1);
                tc_fence_after();
                float x[kKeys];
                float top = -INFINITY;
                if (rows_here) {
                    tmem_ld32(tlane + C::TM_S + (t & 1) * kKeys, x);
                    tc_fence_before();
                    if (lane == 0) mbar_arrive(&sh.s_read[t & 1]);
                    if (__any_sync(0xffffffffu, base + kKeys > lim)) {
#pragma unroll
                        for (int e = 0; e < kKeys; e++) x[e] = base + e < lim ? x[e] : -INFINITY;
                    }
                    float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int e = 0; e < kKeys; e += 8)
#pragma unroll
                        for (int k = 0; k < 4; k++) mx[k] = fmaxf(fmaxf(mx[k], x[e + k]), x[e + k + 4]);
                    top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * p.c;
                } else if (lane == 0) {
                    mbar_arrive(&sh.s_read[t & 1]);
                }
                if (j == 0) {
                    m = top;
                } else if (wg_or(live && top > m + kRaise)) {
                    const float mn = live ? fmaxf(m, top) : m;
                    const float a = mn == -INFINITY ? 1.f : ex2(m - mn);
                    m = mn;
                    l *= a;
                    if (lane < 16 && rows_here) sh.factor[row] = a;
                    wg_sync();
                    warp_wait(ok, &sh.pv_done, (t - 1) & 1);  // the sums so far
                    tc_fence_after();
#pragma unroll 1
                    for (int b = 0; b < kUnits * RT; b += 32) {
                        float y[32];
                        tmem_ld32(to + b, y);
#pragma unroll
                        for (int e = 0; e < 32; e++) y[e] *= sh.factor[(b & (RT - 1)) + e];
                        tmem_st16(to + b, y);
                        tmem_st16(to + b + 16, y + 16);
                    }
                    tmem_wait_st();
                }
                if (rows_here) {
                    const float ref = m == -INFINITY ? 0.f : m;
                    float sum[4] = {0.f, 0.f, 0.f, 0.f};
                    uint32_t pk[kKeys / 2];
#pragma unroll
                    for (int e = 0; e < kKeys; e += 2) {
                        const float u = ex2(fmaf(x[e], p.c, -ref)), v = ex2(fmaf(x[e + 1], p.c, -ref));
                        sum[e & 2] += u;
                        sum[(e & 2) + 1] += v;
                        // to bf16, as the product wants P in the values' type (the sum is of the unrounded)
                        pk[e / 2] = pack2(u, v);
                    }
                    l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
                    if (t > 0) warp_wait(ok, &sh.pv_done, (t - 1) & 1);  // P of the tile before is read
                    if (lane < 16) {
#pragma unroll
                        for (int b = 0; b < kKeys / 8; b++)
                            *reinterpret_cast<uint4*>(sp + row * 128 + ((b ^ (row & 7)) << 4)) =
                                make_uint4(pk[4 * b], pk[4 * b + 1], pk[4 * b + 2], pk[4 * b + 3]);
                    }
                }
                if (base + kKeys > all) {
                    // Keys that some rows must not see: 16 threads a key.
                    warp_wait(ok, &sh.full[slot], phase);  // (the copies, seen by this thread)
                    const int k0 = max(all - base, 0), k1 = pc.keys - base;
                    for (int k = k0 + tid / 16; k < kKeys; k += 8) {
                        bool odd = false;
#pragma unroll
                        for (int b = 0; b < 4; b++) {
                            const int v = (tid & 15) + 16 * b;  // vector of the key's 64
                            uint4* at = reinterpret_cast<uint4*>(
                                skv + slot * C::TILE + (v >> 3) * C::KBLOCK + k * 128 + (v & 7) * 16);
                            if (k >= k1) {
                                *at = make_uint4(0, 0, 0, 0);
                            } else {
                                const uint4 y = *at;
                                if (odd_vector(y)) {
                                    odd = true;
                                    *at = make_uint4(finite_pair(y.x), finite_pair(y.y), finite_pair(y.z),
                                                     finite_pair(y.w));
                                }
                            }
                        }
                        const int bit = base + k - all;
                        if (odd) atomicOr(&sh.odd[i][bit >> 5 & 1], 1u << (bit & 31));
                    }
                }
                fence_proxy_async_smem();
                tc_fence_before();
                mbar_arrive(&sh.p_full);
                if (++slot == NT) {
                    slot = 0;
                    phase ^= 1;
                }
            }
            // What the results need, and the rows' sums. (The slot is used again once these warps
            // and the results' are done with the piece.)
            if (lane < 16 && rows_here) sh.inv[i][row] = !live || l == 0.f ? 0.f : 1.f / l;
            if (live) {
                if (pc.slot >= 0)
                    p.sp.ws[attn_slot_floats(p.sp.rows, kDL) * pc.slot + (size_t)p.sp.rows * kDL + row] =
                        l != 0.f ? m + log2f(l) : pc.kt0 * kKeys < lim ? kAttnNoWeight : -INFINITY;
                else if (p.lse)
                    p.lse[(size_t)pc.tok0 * Hq + (size_t)pc.h * G + sh.row_at[row]] =
                        l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718056f;
            }
            mbar_arrive(&sh.sums_full[i]);
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.piece_empty[i]);
            if (n > 0 && ++buf == C::NO) buf = 0;
        }
        if (!ok) flags |= KDA_DEV_TIMEOUT;
    } else {
        // ------------------------------------------------------------ results
        // In warps of their own, so that the next piece's scores need not wait (nor, at 32
        // rows, its products: there are two results in tensor memory).
        const uint32_t tlane = tmem_at(tbase, 32 * (warp & 3), 0);
        int buf = 0;
        uint32_t o_phase = 0;  // of the pieces' products, a bit a slot
        for (int np = 0; ok; np++) {
            const int i = np % kPieces;
            warp_wait(ok, &sh.piece_full[i], (np / kPieces) & 1);
            if (!ok) break;
            const Piece pc = sh.pieces[i];
            if (pc.end) break;
            const int n = piece_tiles(pc), all = seen_by_all(pc), rows = pc.ntok * G;
            warp_wait(ok, &sh.sums_full[i], (np / kPieces) & 1);
            if (n > 0) {
                warp_wait(ok, &sh.o_full[i], o_phase >> i & 1);
                o_phase ^= 1u << i;
            }
            if (!ok) break;
            tc_fence_after();
            const uint32_t to = tlane + C::TM_O + buf * kUnits * RT;
            const size_t at0 = (size_t)pc.tok0 * Hq + (size_t)pc.h * G;
            float* part = pc.slot >= 0 ? p.sp.ws + attn_slot_floats(p.sp.rows, kDL) * pc.slot : nullptr;
            // Rows without any weight: zeros, whatever their accumulators hold. In a part 0 times that,
            // 0 or NaN, as the row may have weight in others.
            bool empty_row = false;
            for (int r = lane; r < rows; r += 32) empty_row |= sh.inv[i][r] == 0.f;
            const bool nothing = n == 0 || (!part && __any_sync(0xffffffffu, empty_row));
            const bool in_order = p.s.Hkv == 1 || pc.ntok == 1;  // rows of o
            const uint32_t odd[2] = {sh.odd[i][0], sh.odd[i][1]};
            float fin = 0.f;  // NaN once a value is not finite (of parts the join looks at the joined rows)
#pragma unroll 1
            for (int b = 0; b < kUnits * RT; b += 32) {
                const int u = b / RT, r0 = b & (RT - 1);
                const int ch = 128 * u + 32 * (warp & 3) + lane;
                if (r0 >= rows) continue;
                float y[32];
                if (n > 0) tmem_ld32(to + b, y);
#pragma unroll
                for (int e = 0; e < 32; e += 4) {
                    const float4 f = *reinterpret_cast<const float4*>(&sh.inv[i][r0 + e]);
                    const float g[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
                    for (int k = 0; k < 4; k++) y[e + k] *= g[k];
                }
                if (nothing) {
#pragma unroll
                    for (int e = 0; e < 32; e++) y[e] = n > 0 && sh.inv[i][r0 + e] != 0.f ? y[e] : 0.f;
                }
                if (odd[0] | odd[1]) {
                    for (int k = 0; k < 64; k++) {
                        if (!(odd[k >> 5] >> (k & 31) & 1)) continue;
                        const int key = all + k;
                        const int id = p.block_table[(size_t)pc.r * p.max_pages + key / p.page];
                        if (id < 0 || id >= p.num_pages) continue;
                        const float v =
                            __bfloat162float(p.cache[((size_t)id * p.page + key % p.page) * (kDL + DR) + ch]);
                        if (!finite_flag(v)) continue;
                        // (a row of no weight stays zeros)
#pragma unroll
                        for (int e = 0; e < 32; e++)
                            if (key < pc.pos0 + (r0 + e) / G + 1 && (part || sh.inv[i][r0 + e] != 0.f)) y[e] += v;
                    }
                }
                if (part) {
                    float* dst = part + (size_t)r0 * kDL + ch;
#pragma unroll
                    for (int e = 0; e < 32; e++)
                        if (r0 + e < rows) dst[e * kDL] = y[e];
                } else {
                    // Two rows at a time: even lanes store two channels of the first, odd
                    // lanes of the second.
                    const bool up = lane & 1;
                    __nv_bfloat16* dst = p.o + at0 * kDL + (ch & ~1);
#pragma unroll
                    for (int e = 0; e < 32; e += 2) {
                        const float other = __shfl_xor_sync(0xffffffffu, up ? y[e] : y[e + 1], 1);
                        const float lo = up ? other : y[e], hi = up ? y[e + 1] : other;
                        const int rr = r0 + e + up;
                        if (rr < rows) {
                            fin = fmaf(lo, 0.f, fmaf(hi, 0.f, fin));
                            const int at = in_order ? rr : sh.row_at[rr];
                            *reinterpret_cast<uint32_t*>(dst + (size_t)at * kDL) = pack2(lo, hi);
                        }
                    }
                }
            }
            if (!(fin == 0.f)) flags |= KDA_DEV_NONFINITE;
            tc_fence_before();
            if (n > 0) {
                mbar_arrive(&sh.o_free[buf]);
                if (++buf == C::NO) buf = 0;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.piece_empty[i]);
        }
        if (!ok) flags |= KDA_DEV_TIMEOUT;
    }
    __syncwarp();
    report_flags(p.d_status, flags);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kScoreWarp) tmem_dealloc(tbase, 512);
}

// Rows of queries, [tokens][heads][d], boxes of 64 x heads x tokens.
bool make_rows(CUtensorMap* m, const AttnArgs& a, int d, int box_heads, int box_tokens) {
    auto enc = tensor_map_encoder();
    if (!enc) return false;
    cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)a.Hq, (cuuint64_t)a.total_q};
    cuuint64_t strides[2] = {(cuuint64_t)a.q_head * 2, (cuuint64_t)a.q_stride * 2};
    cuuint32_t box[3] = {64, (cuuint32_t)box_heads, (cuuint32_t)box_tokens};
    cuuint32_t es[3] = {1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(a.q), dims, strides, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The cache, [pages][page][d], boxes of 64 x (page or kKeys) tokens.
bool make_cache(CUtensorMap* m, const AttnArgs& a, int d) {
    auto enc = tensor_map_encoder();
    if (!enc) return false;
    cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)a.page, (cuuint64_t)a.num_pages};
    cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)a.page * d * 2};
    cuuint32_t box[3] = {64, (cuuint32_t)(a.page < kKeys ? a.page : kKeys), 1};
    cuuint32_t es[3] = {1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(a.k), dims, strides, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int DR, int RT>
cudaError_t launch_t(const AttnArgs& a) {
    using C = TcCfg<DR, RT>;
    const int blocks = latent_head_blocks(a.Hq, RT), G = a.Hq / blocks, tok = RT / G;
    int dev = 0;
    const int nsm = device_sms(&dev);
    if (nsm == 0) return cudaErrorNoDevice;
    LatentTcParams p{};
    p.s = {a.cu_q, a.kv_len, a.N, a.total_q, a.max_q, attn_kv_cap(a), blocks, G, tok, tok, kKeys, 1, 1, kItemKeys};
    p.sp = latent_tc_split(a.N, a.total_q, a.max_q, p.s.kv_cap, a.Hq, nsm);
    if (p.sp.ctas && a.ws && a.ws_bytes >= attn_split_bytes(p.sp, kDL)) p.sp.ws = a.ws;
    p.block_table = a.block_table;
    p.cache = static_cast<const __nv_bfloat16*>(a.k);
    p.o = static_cast<__nv_bfloat16*>(a.o);
    p.lse = a.lse;
    p.num_pages = a.num_pages;
    p.page = a.page;
    p.max_pages = a.max_pages;
    p.box_q = a.max_q < tok ? a.max_q : tok;
    p.c = a.scale * 1.44269504089f;
    p.d_status = a.d_status;
    CUtensorMap mq, mc;
    if (!make_rows(&mq, a, kDL + DR, G, p.box_q) || !make_cache(&mc, a, kDL + DR)) return cudaErrorInvalidValue;
    auto kernel = kda_latent_tc_kernel<DR, RT>;
    static std::atomic<uint64_t> ready{0};
    cudaError_t e = allow_shared(kernel, tc_smem<C>(), ready, dev);
    if (e != cudaSuccess) return e;
    const long long grid = p.sp.ws ? p.sp.ctas : attn_items_bound(p.s);
    if (grid >= 1LL << 31) return cudaErrorInvalidValue;
    e = launch_dependent(kernel, dim3((unsigned)grid), dim3(kThreadsTc), tc_smem<C>(), a.stream, mq, mc, p);
    if (e != cudaSuccess || !p.sp.ws) return e;
    return launch_attn_combine(p.sp, blocks, G, kDL, RT, a.o, a.lse, KDA_BF16, a.d_status, a.stream);
}

}  // namespace

AttnSplit latent_tc_split(int N, int total_q, int max_q, long long max_keys, int Hq, int nsm) {
    AttnSplit sp{};
    if (N == 0 || total_q == 0 || max_q == 0 || Hq == 0 || nsm == 0) return sp;
    const int rt = latent_tc_rows(max_q, Hq), blocks = latent_head_blocks(Hq, rt), G = Hq / blocks, tok = rt / G;
    // Whole items, given out as CTAs become free, or ranges of one cost. Ranges end together,
    // but cost some 6 us for the parts, their join and more pieces; whole items end up to one
    // item apart. Measured, ranges against whole, us, 152 SMs, one token a request, 16 heads (32 are alike).
    // Requests of equal length, and of lengths drawn from 1 up to it:
    //   256 keys, 256 requests         30/22
    //   512       40, 256, 608         20/18, 46/36, 75/69        20/18, 34/29, 57/49
    //   1024      40, 152, 400         22/28, 42/37, 95/85        21/28, 33/30, 65/60
    //   1536      76, 152, 608         41/39, 56/50, 176/170      27/37, 45/43, 107/108
    //   2048      152, 608, 4864       68/62, 225/220             50/52, 131/135, 873/865
    //   4096, 8192  608; 1216          406/399; 1546/1538         239/263; 839/896
    // What a request may have is not what it has, and one long request among many short ones is a chain on
    // one SM, of 21 ns a key: 1215 to 2048 keys and one of 131072 283/2712, 1216 with logarithms drawn, to 8192
    // 227/306, to 32768 673/1007. So beyond 2048 keys whole items need so many that this chain is at most
    // half as long as they take (5 us each and more): 20000 to 300 keys in tables of 2048 1355/1050, 256 of 67
    // heads (17152 items) to 8192 11605/9376; 4864 to 8192, logarithms drawn, 864/884 and 3000 to 300 in tables
    // of 32768, 171/160, are ranges.
    const long long items = (long long)total_q / (max_q < tok ? max_q : tok) * blocks;  // at least
    if (max_keys <= KDA_LATENT_SHORT_KEYS || (max_keys <= 512 && 2 * items >= nsm)) return sp;
    if ((max_keys < 2048 && items >= nsm) || items >= max_keys / 128 * nsm) return sp;
    sp.ctas = nsm;
    sp.least = 128;  // keys of a range: 3 requests to 700 keys x 8 heads 17.3 us, with 256 20.3, with 64 17.9
    sp.rows = ((max_q < tok ? max_q : tok) * G + 3) & ~3;  // whole 16-byte vectors
    return sp;
}

cudaError_t launch_latent_tc(const AttnArgs& a) {
    // Row tiles of 32 where calls have no more rows, with room for five key tiles and two results
    // (against 64 with four and one: 256 requests of 4096 keys x 16 heads 194 us against 202, 64 x 32 heads 66
    // against 69, 3 of 700 x 8 heads 15.7 against 16.4); of 64 above, as a tile's products are bound by
    // its reads from shared memory, the same for 64 rows as for 32.
    if (latent_tc_rows(a.max_q, a.Hq) == 32) return a.dr ? launch_t<64, 32>(a) : launch_t<0, 32>(a);
    return a.dr ? launch_t<64, 64>(a) : launch_t<0, 64>(a);
}

}  // namespace kda
