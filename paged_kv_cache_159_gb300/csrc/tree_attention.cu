// tree_attention.cu -- attention of a few new tokens per sequence over a paged cache: trees (or chains)
// of drafted tokens, and single tokens with a sliding window and sink tokens.
//
// What is computed ("传统 Attention 的 KV Cache 问题" (pyllm.pages.dev) §1.1; the mask: "理解 KV Cache"
// (steinslab.io) §1.2's M, a row of it per drafted token).  The last P of a sequence's L positions are new,
// C = L - P cached.  Row i's output is sum_j softmax_j(scale q_i . k_j) v_j over the positions j that it sees:
//   chain (no mask):  j <= p and (j > p - window or j < sinks), p = C + i;
//   tree:             new position C + j where bit j of the row's mask is set, and cached j < C with
//                     j > p - window or j < sinks, p = C + (bits set) - 1: the row's place behind its ancestors.
// A row that sees nothing is zeros.
//
// Schedule.  A unit is (sequence, KV head, up to MR rows): rows are (token, head of the group) pairs, MR = 16 or
// 32 by the most rows that a sequence may have; more take the kernel of tree_tcgen05.cu (MOST_MMA_ROWS).  A unit's
// visible blocks (those of the sinks, then from the window's first on) make tiles of 64 keys, and the tiles of all
// units, laid end to end, are cut evenly over a one-wave grid (a unit counts for UNIT_COST tiles more than it has).
// Every CTA finds its share from the device's lengths.  A unit in one CTA is written there; a cut one leaves a
// partial (max, sum, output) per CTA, which a second launch merges in order: the placement of blocks changes no bit.
//
// A CTA: one warp copies (a tensor copy per bf16 block of K and V, 128-byte swizzle; a bulk copy per FP8 or
// INT4 block) into a ring of tiles, WR x WK warps multiply (mma.sync m16n8k16, queries as the 16 rows): WR
// groups of 16 rows, the tile's keys divided over WK warps, whose states meet at a unit's end.  FP8 and INT4
// tiles are expanded to f16 once a CTA (exactly), q goes to f16 with a power of two per row, P is f16 times 2^8.  Over
// bf16 pools P is bf16, 8 bits, since both factors of a product have one type and V is bf16 (the plain decode does the same;
// P in two bf16 terms would be twice the products): outputs are 0.0020 to 0.0023 off in norm, where their own rounding
// alone is 0.0017.
//
// Masked places.  Scores are masked by select.  A V element that no row of the warp sees is taken as zero (a
// register mask), since 0 x NaN is NaN; where some rows see a position and others do not, and its V is not
// finite, its products leave the tensor core and are added row by row.
//
// What bounds it (32 / 8 heads of 128, bf16 pool, in a graph, merge included):
//   * 256 sequences of up to 16384, window 1024, 4 sinks: 175 us, 6.05 TB/s of the visible keys' bytes, 0.89 of a copy's
//     rate: the reading.
//   * 64 sequences of 2048 with 8 drafts (32 rows): 103 us, 5.3 TB/s.  The two CTAs of an SM take 1.28 us a tile, by the
//     latency of a tile's steps in the two warps that share its keys (issue slots 29 % used, tensor pipe 31 %, DRAM 71 %;
//     some four spilled registers a warp and tile, at 168 a thread, are part of it); a unit costs three tiles besides (q, the
//     epilogue), and the merge takes 7 us.
//   * one sequence of 13 drafts: 14 us, latency: lengths, table, tiles, partials, merge one after another.
//
// Both launches may start while the one before drains (programmatic dependent launch): they wait before they
// read, and load coherently.
#include <algorithm>
#include <atomic>
#include <cmath>

#include "tree_common.cuh"

namespace pkv {
namespace tree {

__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// A tile as the copying warp writes it down; a segment's first tile says what unit it is of.
struct TileNote {
    int got, pos[TB];                                              // loaded blocks; first position of each
    int L, P, row0, h, m, left, unit, place;                       // left: tiles of the segment; place: the unit's, bit 31: not from its first tile
};

template <int D, int KIND, int WR, int WK>
struct Shape {
    static constexpr int NC = WR * WK, NT = NC * 32 + 32, MR = 16 * WR;
    static constexpr int BT = BS * D * 2;                          // a block of K or V in 16 bits
    static constexpr int TILE = KIND == BF16 ? BT : KIND == FP8 ? BS * D : int4::tile_bytes(D);      // as stored
    static constexpr int STAGE = 2 * TB * TILE;
    // 16-bit tiles that FP8 and INT4 are expanded to: one where every warp expands its own keys, else two
    static constexpr int WIDE = 2 * TB * BT;
    static constexpr int NWIDE = KIND == BF16 ? 0 : WK == TB ? 1 : 2;
    static constexpr int QB = MR * D * 2;                          // a unit's rows of q, the next one's while this one's are in registers
    static constexpr int ROOM = 110 * 1024;                        // two CTAs per SM
    static constexpr int NS_ = (ROOM - NWIDE * WIDE - QB) / STAGE;
    static constexpr int NS = NS_ > 8 ? 8 : NS_;
    static constexpr int RING = NWIDE * WIDE;                      // (STAGE of a quantised pool is a multiple of 128)
    static constexpr int Q = RING + NS * STAGE;
    static constexpr int ML = Q + QB;                              // (max, sum) of the key warps' rows
    static constexpr int INFO = ML + NC * 16 * 8;                  // TileNote of every stage
    static constexpr int BAR = INFO + (NS * (int)sizeof(TileNote) + 7) / 8 * 8;
    static constexpr int ALLOC = BAR + 8 * (2 * NS + 4) + 1024;    // + alignment slack
    static_assert(NS >= 2 && ALLOC + 256 <= 113 * 1024, "shared memory");
    static_assert(TB % WK == 0 && STAGE % 128 == 0, "");
};

template <int D, int KIND, int WR, int WK>
__global__ void __launch_bounds__(Shape<D, KIND, WR, WK>::NT, 2)
tree_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap, const Params p)
{
    using S = Shape<D, KIND, WR, WK>;
    constexpr int NC = S::NC, MR = S::MR, NS = S::NS, BT = S::BT, NB = TB / WK, KS = D / 16, NN = D / 8;
    constexpr float SHIFT = KIND == BF16 ? 0.f : 8.f;              // P is held as P 2^SHIFT
    extern __shared__ uint8_t smem_raw[];
    __shared__ ShareScratch<S::NT> scratch;
    uint8_t *sm = smem_raw + ((1024u - (dev::smem_u32(smem_raw) & 1023u)) & 1023u);
    const uint32_t base = dev::smem_u32(sm);
    const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(dev::FULL, tid >> 5, 0);
    auto full = [&](int s) { return base + S::BAR + 8 * s; };
    auto empty = [&](int s) { return base + S::BAR + 8 * (NS + s); };
    const uint32_t meet = base + S::BAR + 8 * (2 * NS), never = meet + 8, q_full = meet + 16, q_free = meet + 24;
    TileNote *info = reinterpret_cast<TileNote *>(sm + S::INFO);
    auto wait_all = [&](uint32_t bar, int phase) { return (bool)__all_sync(dev::FULL, wait_bar(bar, (uint32_t)phase & 1u)); };
    if (tid == 0) {
        for (int s = 0; s < NS; ++s) {
            dev::mbar_init(full(s), 1);
            dev::mbar_init(empty(s), NC);
        }
        dev::mbar_init(meet, NC);
        dev::mbar_init(never, 1);
        dev::mbar_init(q_full, 32);                                // the copying warp's lanes
        dev::mbar_init(q_free, NC);
        dev::fence_barrier_init();
    }
    pdl_launch();
    pdl_wait();

    const Share my = share_of<S::NT, D>(p, scratch);
    if (my.tiles == 0) return;

    if (warp == NC) {
        // ============ the copying warp: lane k < TB takes block k of a tile, K and V; all of them a unit's rows of q
        Walk walk(p, my);
        bool ok = true;
        int n = 0;                                                 // tiles issued
        for (int u = 0; ok && n < my.tiles; ++u) {
            const Segment g = walk.next(p);
            // the table's entries of 32 blocks (8 tiles from `chunk` on), and of the 32 after them
            auto fetch = [&](int t0) {
                const int v = TB * t0 + lane;
                return v < walk.sq.nvb && v < TB * g.t1 ? __ldcg(p.tables + (size_t)walk.b * p.MB + walk.block(v)) : -2;
            };
            int chunk = g.t0, ids = fetch(chunk), nxt = fetch(chunk + 8);
            // rows of q, 16 bytes a lane, chunks swizzled within 64 columns (rows beyond the unit's hold what they held)
            if (u > 0) ok = wait_all(q_free, u - 1);
            if (!ok) break;
            {
                constexpr int CH = D / 8, STEP = 32 / CH;          // chunks of a row; rows a pass
                const int rows = min(MR, walk.sq.P * p.group - g.m * MR), c = lane % CH;
                int x = lane / CH, y = g.m * MR + x, i = y / p.group, hh = y - i * p.group;
                const uint16_t *src = p.q + ((size_t)walk.sq.row0 * p.Hq + (size_t)g.h * p.group) * D + 8 * c;
#pragma unroll 1
                for (; x < rows; x += STEP) {
                    const uint32_t dst = base + S::Q + (c >> 3) * (MR * 128) + x * 128 + (((c & 7) ^ (x & 7)) << 4);
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src + ((size_t)i * p.Hq + hh) * D) : "memory");
                    hh += STEP;
                    while (hh >= p.group) {
                        hh -= p.group;
                        ++i;
                    }
                }
                asm volatile("cp.async.mbarrier.arrive.noinc.shared.b64 [%0];" ::"r"(q_full) : "memory");
            }
#pragma unroll 1
            for (int t = g.t0; t < g.t1 && n < my.tiles; ++t, ++n) {
                if (t - chunk == 8) {
                    chunk = t;
                    ids = nxt;
                    nxt = fetch(t + 8);
                }
                const int cur = __shfl_sync(dev::FULL, ids, TB * (t - chunk) + (lane & (TB - 1))), s = n % NS;
                if (n >= NS) ok = wait_all(empty(s), (n - NS) / NS);
                if (!ok) break;
                const bool want = lane < TB && cur != -2, good = lane < TB && cur >= 0 && cur < p.num_blocks;
                if (want && !good) dev::flag_error(p.err, PKV_DEVERR_BLOCK_ID);
                const unsigned got = __ballot_sync(dev::FULL, good);
                TileNote &note = info[s];
                if (lane < TB) note.pos[lane] = walk.block(TB * t + lane) * BS;
                if (lane == 0) {
                    note.got = (int)got;
                    if (t == g.t0) {
                        note.L = walk.sq.L;
                        note.P = walk.sq.P;
                        note.row0 = walk.sq.row0;
                        note.h = g.h;
                        note.m = g.m;
                        note.left = g.t1 - t;
                        note.unit = walk.sq.nt;
                        note.place = walk.unit0 | (t > 0 ? INT_MIN : 0);
                    }
                }
                __syncwarp();
                if (lane == 0) dev::mbar_arrive_expect_tx(full(s), (uint32_t)(2 * S::TILE * __popc(got)));
                __syncwarp();
                if (good) {
                    const uint32_t dk = base + S::RING + s * S::STAGE + lane * S::TILE, dv = dk + TB * S::TILE;
                    const int tile = cur * p.Hkv + g.h;
                    if constexpr (KIND != BF16) {
                        dev::bulk_g2s(dk, p.key_cache + (size_t)tile * S::TILE, S::TILE, full(s));
                        dev::bulk_g2s(dv, p.value_cache + (size_t)tile * S::TILE, S::TILE, full(s));
                    } else if constexpr (D == 128) {
                        tc::tma_load_4d(dk, &kmap, 0, 0, 0, tile, full(s));
                        tc::tma_load_4d(dv, &vmap, 0, 0, 0, tile, full(s));
                    } else {
                        tc::tma_load_3d(dk, &kmap, 0, 0, tile, full(s));
                        tc::tma_load_3d(dv, &vmap, 0, 0, tile, full(s));
                    }
                }
            }
        }
        if (!ok && lane == 0) dev::flag_error(p.err, PKV_DEVERR_TIMEOUT);
        // no copy may land after the CTA has left: wait (bounded) for the last one of every stage
        asm volatile("cp.async.wait_all;" ::: "memory");
#pragma unroll 1
        for (int x = max(0, n - NS); x < n; ++x) (void)wait_bar(full(x % NS), (uint32_t)((x / NS) & 1));
        return;
    }

    // ============ the multiplying warps: rows 16 wr .. of the unit, blocks NB wk .. of every tile
    const int wr = warp / WK, wk = warp % WK, gid = lane >> 2, t4 = lane & 3;
    uint32_t meet_phase = 0;
    bool ok = true;
    auto sync_warps = [&]() {                                      // all multiplying warps, bounded
        __syncwarp();
        if (lane == 0) dev::mbar_arrive(meet);
        ok = wait_all(meet, (int)meet_phase);
        meet_phase ^= 1u;
        return ok;
    };
    if (p.test_stall) ok = __all_sync(dev::FULL, dev::mbar_wait_bounded_ns(never, 0, dev::TEST_EXPIRE_NS));
    int n = 0;                                                     // tiles seen
    bool cut_begins = false;
    int cut[META] = {};
    for (int u = 0; ok && n < my.tiles; ++u) {
        const bool at_first = n == 0;                              // the share's first segment
        ok = wait_all(full(n % NS), n / NS) && wait_all(q_full, u);
        if (!ok) break;
        const TileNote &first = info[n % NS];
        Seq sq;                                                    // (what the masks need of it)
        sq.L = first.L;
        sq.P = first.P;
        sq.C = sq.L - sq.P;
        sq.row0 = first.row0;
        const int h = first.h, mt = first.m, left = first.left, unit = first.unit, place0 = first.place;
        const int rows = sq.P * p.group - mt * MR;                 // of this unit, at most MR of them here
        uint32_t qa[KS][4];
#pragma unroll
        for (int k = 0; k < KS; ++k) {
            const int row = 16 * wr + (lane & 15), chunk = 2 * k + (lane >> 4);
            dev::ldsm_x4(base + S::Q + (chunk >> 3) * (MR * 128) + row * 128 + (((chunk & 7) ^ (row & 7)) << 4), qa[k]);
        }
        __syncwarp();
        if (lane == 0) dev::mbar_arrive(q_free);
        // this lane's two rows
        int place[2], draft[2], head[2];                           // p of the row; its token; its head in the group
        bool live[2];
        unsigned long long word[2];                                // the first of its mask
        float sc[2] = {p.score_scale, p.score_scale};
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int x = 16 * wr + gid + 8 * e;
            live[e] = x < rows;
            const int y = mt * MR + (live[e] ? x : 0);
            draft[e] = y / p.group;
            head[e] = y - draft[e] * p.group;
            place[e] = p.mask && !p.window ? 0 : place_of(p, sq, draft[e]);
            word[e] = first_word(p, sq, draft[e]);
        }
        if constexpr (KIND != BF16) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                uint32_t top = 0;
#pragma unroll
                for (int k = 0; k < KS; ++k) {
                    const uint32_t m2 = __vmaxu2(qa[k][e] & 0x7fff7fffu, qa[k][e + 2] & 0x7fff7fffu);
                    top = max(top, max(m2 & 0xffffu, m2 >> 16));
                }
                top = max(top, __shfl_xor_sync(dev::FULL, top, 1));
                top = max(top, __shfl_xor_sync(dev::FULL, top, 2));
                const int up = q_exponent(top);
                const float f = q_factor(up);
                sc[e] = row_scale(sc[e], up);
#pragma unroll
                for (int k = 0; k < KS; ++k)
#pragma unroll
                    for (int x = e; x < 4; x += 2) qa[k][x] = dev::pack_f16x2(dev::bf16_lo(qa[k][x]) * f, dev::bf16_hi(qa[k][x]) * f);
            }
        }
        float acc[NN][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
        for (int x = 0; x < NN; ++x)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[x][e] = 0.f;
        // positions up to which, and from which on, all rows of the unit see the cache
        const int i0 = mt * MR / p.group, i1 = min(sq.P - 1, (mt * MR + min(rows, MR) - 1) / p.group);
        const int to = all_to(p, sq, i0), from = all_from(p, sq, i1);

#pragma unroll 1
        for (const int end = n + left; n < end; ++n) {
            const int s = n % NS;
            ok = wait_all(full(s), n / NS);
            if (!ok) break;
            const unsigned got = (unsigned)info[s].got;
            int pos[NB];                                           // first position of each of this warp's blocks
#pragma unroll
            for (int k = 0; k < NB; ++k) pos[k] = info[s].pos[wk * NB + k];
            const uint8_t *stage = sm + S::RING + s * S::STAGE;
            uint32_t kt = base + S::RING + s * S::STAGE;           // the tile in 16 bits: TB blocks of K, TB of V
            const bool at_end = n == end - 1;
            if constexpr (KIND != BF16) {
                uint8_t *wide = sm + (S::NWIDE == 2 ? (n & 1) * S::WIDE : 0);
                kt = base + (S::NWIDE == 2 ? (n & 1) * S::WIDE : 0);
#pragma unroll
                for (int x = warp; x < 2 * TB; x += NC) {          // (block x % TB, K or V)
                    const int k = x % TB;
                    if ((got >> k) & 1u) widen<D, KIND>(stage + x * S::TILE, wide + x * BT, BS * 128, x < TB, lane);
                }
                __syncwarp();
                if (lane == 0) dev::mbar_arrive(empty(s));
                if (WK != TB && !sync_warps()) break;
            }
            const uint32_t vt = kt + TB * BT;
            bool edge = false;
#pragma unroll
            for (int k = 0; k < NB; ++k) {
                edge |= !((got >> (wk * NB + k)) & 1u) || pos[k] + BS > to || (pos[k] < from && pos[k] + BS > p.sinks);
            }
            // ---- S = Q K^T
            float x[2 * NB][4];
#pragma unroll
            for (int k = 0; k < NB; ++k) {
                const uint32_t kb = kt + (wk * NB + k) * BT;
#pragma unroll
                for (int e = 0; e < 4; ++e) x[2 * k][e] = x[2 * k + 1][e] = 0.f;
                const int row = ((lane >> 4) & 1) * 8 + (lane & 7);
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) {
                    const int chunk = 2 * ks + ((lane >> 3) & 1);
                    uint32_t f[4];
                    dev::ldsm_x4(kb + (chunk >> 3) * (BS * 128) + row * 128 + (((chunk & 7) ^ (row & 7)) << 4), f);
                    if constexpr (KIND == BF16) {
                        dev::mma_bf16_16816(x[2 * k], qa[ks], f[0], f[1]);
                        dev::mma_bf16_16816(x[2 * k + 1], qa[ks], f[2], f[3]);
                    } else {
                        dev::mma_f16_16816(x[2 * k], qa[ks], f[0], f[1]);
                        dev::mma_f16_16816(x[2 * k + 1], qa[ks], f[2], f[3]);
                    }
                }
            }
#pragma unroll
            for (int k = 0; k < 2 * NB; ++k)
#pragma unroll
                for (int e = 0; e < 4; ++e) x[k][e] *= sc[e >> 1];
            // ---- the mask of each 16 keys: bit j of see[k], row gid in the lower half, gid + 8 in the upper
            uint32_t see[NB];
            if (__builtin_expect(edge, 0)) {
#pragma unroll
                for (int k = 0; k < NB; ++k) {
                    see[k] = 0;
                    const uint32_t valid = (got >> (wk * NB + k)) & 1u ? ones(sq.L - pos[k]) : 0u;
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        if (live[e]) see[k] |= seen16(p, sq, draft[e], place[e], word[e], pos[k], valid) << (16 * e);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
#pragma unroll
                        for (int j = 0; j < 2; ++j)
                            if (!((see[k] >> (8 * j + 2 * t4 + (e & 1) + 16 * (e >> 1))) & 1u)) x[2 * k + j][e] = -INFINITY;
                }
            }
            // ---- running maximum and sum, P
            float top[2] = {m[0], m[1]};
#pragma unroll
            for (int k = 0; k < 2 * NB; ++k) {
                top[0] = tc::fmax3(top[0], x[k][0], x[k][1]);
                top[1] = tc::fmax3(top[1], x[k][2], x[k][3]);
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                top[e] = fmaxf(top[e], __shfl_xor_sync(dev::FULL, top[e], 1));
                top[e] = fmaxf(top[e], __shfl_xor_sync(dev::FULL, top[e], 2));
            }
            if (__any_sync(dev::FULL, top[0] > m[0] || top[1] > m[1])) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float f = top[e] > m[e] ? dev::fast_exp2(m[e] - top[e]) : 1.f;
                    m[e] = top[e];
                    l[e] *= f;
#pragma unroll
                    for (int c = 0; c < NN; ++c) {
                        acc[c][2 * e] *= f;
                        acc[c][2 * e + 1] *= f;
                    }
                }
            }
            const float ref[2] = {m[0] == -INFINITY ? 0.f : m[0] - SHIFT, m[1] == -INFINITY ? 0.f : m[1] - SHIFT};
#pragma unroll
            for (int k = 0; k < 2 * NB; ++k)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    x[k][e] = dev::fast_exp2(x[k][e] - ref[e >> 1]);
                    l[e >> 1] += x[k][e];
                }
            // ---- O += P V
#pragma unroll
            for (int k = 0; k < NB; ++k) {
                auto pack = [&](float lo, float hi) { return KIND == BF16 ? dev::pack_bf16x2(lo, hi) : dev::pack_f16x2(lo, hi); };
                const uint32_t pa[4] = {pack(x[2 * k][0], x[2 * k][1]), pack(x[2 * k][2], x[2 * k][3]),
                                        pack(x[2 * k + 1][0], x[2 * k + 1][1]), pack(x[2 * k + 1][2], x[2 * k + 1][3])};
                const int row = ((lane >> 3) & 1) * 8 + (lane & 7);
                const uint32_t vb = vt + (wk * NB + k) * BT;
                auto load_v = [&](int dd, uint32_t (&f)[4]) {      // 16 columns from 16 dd on
                    const int chunk = 2 * dd + (lane >> 4);
                    dev::ldsm_x4_trans(vb + (chunk >> 3) * (BS * 128) + row * 128 + (((chunk & 7) ^ (row & 7)) << 4), f);
                };
                auto mma = [&](float (&d)[4], uint32_t b0, uint32_t b1) {
                    if constexpr (KIND == BF16) dev::mma_bf16_16816(d, pa, b0, b1);
                    else dev::mma_f16_16816(d, pa, b0, b1);
                };
                if (!edge) {
#pragma unroll
                    for (int dd = 0; dd < NN / 2; ++dd) {
                        uint32_t f[4];
                        load_v(dd, f);
                        mma(acc[2 * dd], f[0], f[1]);
                        mma(acc[2 * dd + 1], f[2], f[3]);
                    }
                    continue;
                }
                // V only where a row sees it (a padding row sees nothing, and hides nothing)
                const uint32_t any2 = __reduce_or_sync(dev::FULL, see[k]);
                const uint32_t all2 = __reduce_and_sync(dev::FULL, (live[0] ? see[k] : see[k] | 0xffffu) | (live[1] ? 0u : 0xffff0000u));
                const uint32_t any = (any2 | any2 >> 16) & 0xffffu, all = all2 & (all2 >> 16) & 0xffffu;
                uint32_t keep = any;
                if (any & ~all) {
                    // positions that some rows do not see: those whose V is not finite go row by row
                    constexpr uint32_t EXP = KIND == BF16 ? 0x7f80u : 0x7c00u;
                    uint32_t lo = 0, hi = 0;                       // largest exponents of keys 2 t4, + 1; + 8, + 9
#pragma unroll 2
                    for (int dd = 0; dd < NN / 2; ++dd) {
                        uint32_t f[4];
                        load_v(dd, f);
                        lo = __vmaxu2(lo, __vmaxu2(f[0] & (EXP | EXP << 16), f[2] & (EXP | EXP << 16)));
                        hi = __vmaxu2(hi, __vmaxu2(f[1] & (EXP | EXP << 16), f[3] & (EXP | EXP << 16)));
                    }
                    uint32_t odd = ((lo & 0xffffu) == EXP ? 1u : 0u) | ((lo >> 16) == EXP ? 2u : 0u) | ((hi & 0xffffu) == EXP ? 0x100u : 0u) |
                                   ((hi >> 16) == EXP ? 0x200u : 0u);
                    odd <<= 2 * t4;
                    odd = __reduce_or_sync(dev::FULL, odd) & any & ~all;
                    keep &= ~odd;
#pragma unroll 1
                    while (odd) {
                        const int j = __ffs(odd) - 1, from = (lane & ~3) | ((j & 7) >> 1);
                        odd &= odd - 1;
                        float pj[2];
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const float c = j & 8 ? (j & 1 ? x[2 * k + 1][2 * e + 1] : x[2 * k + 1][2 * e])
                                                  : (j & 1 ? x[2 * k][2 * e + 1] : x[2 * k][2 * e]);
                            pj[e] = __shfl_sync(dev::FULL, c, from);
                        }
#pragma unroll
                        for (int c = 0; c < NN; ++c) {
                            uint32_t w;
                            asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w) : "r"(vb + (c >> 3) * (BS * 128) + j * 128 + (((c & 7) ^ (j & 7)) << 4) + t4 * 4));
                            float2 v;
                            if constexpr (KIND == BF16) v = make_float2(dev::bf16_lo(w), dev::bf16_hi(w));
                            else v = __half22float2(*reinterpret_cast<const __half2 *>(&w));
#pragma unroll
                            for (int e = 0; e < 2; ++e)
                                if ((see[k] >> (j + 16 * e)) & 1u) {
                                    acc[c][2 * e] = fmaf(pj[e], v.x, acc[c][2 * e]);
                                    acc[c][2 * e + 1] = fmaf(pj[e], v.y, acc[c][2 * e + 1]);
                                }
                        }
                    }
                }
                auto halves = [&](int j) { return ((keep >> j) & 1u ? 0xffffu : 0u) | ((keep >> (j + 1)) & 1u ? 0xffff0000u : 0u); };
                const uint32_t k0 = halves(2 * t4), k1 = halves(2 * t4 + 8);
#pragma unroll
                for (int dd = 0; dd < NN / 2; ++dd) {
                    uint32_t f[4];
                    load_v(dd, f);
                    mma(acc[2 * dd], f[0] & k0, f[1] & k1);
                    mma(acc[2 * dd + 1], f[2] & k0, f[3] & k1);
                }
            }
            // (the last tile of a segment keeps its stage for the key warps' states)
            if (KIND == BF16 && (WK == 1 || !at_end)) {
                __syncwarp();
                if (lane == 0) dev::mbar_arrive(empty(s));
            }
        }
        if (!ok) break;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            l[e] += __shfl_xor_sync(dev::FULL, l[e], 1);
            l[e] += __shfl_xor_sync(dev::FULL, l[e], 2);
        }
        // ---- the key warps' states: each joins all of them for its share of the columns
        constexpr int NS4 = NN / WK;                               // 8-column groups of a warp's share
        float o[NS4][4];
        if constexpr (WK > 1) {
            const int s = (n - 1) % NS;
            uint8_t *buf = KIND == BF16 ? sm + S::RING + s * S::STAGE : sm + (S::NWIDE == 2 ? ((n - 1) & 1) * S::WIDE : 0);
            float4 *all = reinterpret_cast<float4 *>(buf);         // [warp][NN][32]
            float2 *ml = reinterpret_cast<float2 *>(sm + S::ML);   // [warp][16]
            if (!sync_warps()) break;                              // the tile is read
#pragma unroll
            for (int c = 0; c < NN; ++c)
                if (c / NS4 != wk) all[(warp * NN + c) * 32 + lane] = make_float4(acc[c][0], acc[c][1], acc[c][2], acc[c][3]);
            if (t4 == 0) {
                ml[warp * 16 + gid] = make_float2(m[0], l[0]);
                ml[warp * 16 + gid + 8] = make_float2(m[1], l[1]);
            }
            if (!sync_warps()) break;
            float2 st[WK][2];
            float M[2] = {-INFINITY, -INFINITY};
#pragma unroll
            for (int w = 0; w < WK; ++w)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    st[w][e] = ml[(wr * WK + w) * 16 + gid + 8 * e];
                    M[e] = fmaxf(M[e], st[w][e].x);
                }
#pragma unroll
            for (int c = 0; c < NS4; ++c)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[c][e] = 0.f;
            l[0] = l[1] = 0.f;
#pragma unroll
            for (int w = 0; w < WK; ++w) {
                float f[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    f[e] = M[e] == -INFINITY ? 1.f : dev::fast_exp2(st[w][e].x - M[e]);
                    l[e] = fmaf(st[w][e].y, f[e], l[e]);
                }
#pragma unroll
                for (int c = 0; c < NS4; ++c) {
                    float4 v;
                    if (w == wk) {
#pragma unroll
                        for (int x = 0; x < WK; ++x)               // (a constant index)
                            if (x == wk) v = make_float4(acc[x * NS4 + c][0], acc[x * NS4 + c][1], acc[x * NS4 + c][2], acc[x * NS4 + c][3]);
                    } else {
                        v = all[((wr * WK + w) * NN + wk * NS4 + c) * 32 + lane];
                    }
                    o[c][0] = fmaf(v.x, f[0], o[c][0]);
                    o[c][1] = fmaf(v.y, f[0], o[c][1]);
                    o[c][2] = fmaf(v.z, f[1], o[c][2]);
                    o[c][3] = fmaf(v.w, f[1], o[c][3]);
                }
            }
            m[0] = M[0];
            m[1] = M[1];
            if constexpr (KIND == BF16) {
                dev::fence_proxy_async_smem();                     // these accesses before the next copy into the stage
                __syncwarp();
                if (lane == 0) dev::mbar_arrive(empty(s));
            } else if (!sync_warps()) {                            // the buffer is read
                break;
            }
        } else {
#pragma unroll
            for (int c = 0; c < NN; ++c)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[c][e] = acc[c][e];
        }
        const int c0 = wk * NS4;
        if (left == unit) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                if (!live[e]) continue;
                const float inv = l[e] == 0.f ? 0.f : p.out_scale / l[e];
                uint32_t *dst = reinterpret_cast<uint32_t *>(p.out + ((size_t)(sq.row0 + draft[e]) * p.Hq + (size_t)h * p.group + head[e]) * D) + t4;
#pragma unroll
                for (int c = 0; c < NS4; ++c) dst[4 * (c0 + c)] = dev::pack_bf16x2(o[c][2 * e] * inv, o[c][2 * e + 1] * inv);
            }
        } else {
            const int slot = at_first ? 0 : 1;
            if (place0 >= 0) {
                // the unit goes on in the next CTAs, up to the one that holds its last task
                cut_begins = true;
                cut[0] = min(rows, MR);
                cut[1] = stream_of(place0 + p.unit_cost + unit - 1, my.W, my.streams);
                cut[2] = slot;
                cut[3] = sq.row0;
                cut[4] = h;
                cut[5] = mt;
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                if (!live[e]) continue;
                const size_t pr = ((size_t)blockIdx.x * 2 + slot) * MR + 16 * wr + gid + 8 * e;
                const size_t s0 = (size_t)blockIdx.x * 2 + slot;
#pragma unroll
                for (int c = 0; c < NS4; ++c)                      // columns 8 (c0 + c) + 2 t4, + 1
                    *reinterpret_cast<float2 *>(p.part_o + ((s0 * (D / 4) + 2 * (c0 + c) + (t4 >> 1)) * MR + (pr - s0 * MR)) * 4 + 2 * (t4 & 1)) =
                        make_float2(o[c][2 * e], o[c][2 * e + 1]);
                if (wk == 0 && t4 == 0) reinterpret_cast<float2 *>(p.part_ml)[pr] = make_float2(m[e], l[e]);
            }
        }
    }
    if (!ok && lane == 0) dev::flag_error(p.err, PKV_DEVERR_TIMEOUT);
    if (warp == 0 && lane < META) {
        int v = 0;
#pragma unroll
        for (int x = 0; x < META; ++x)
            if (x == lane) v = cut[x];
        p.meta[(size_t)blockIdx.x * META + lane] = ok && cut_begins ? v : 0;
    }
}

// Merge the partials of cut units: block (c, y) the rows MERGE_ROWS y .. of the unit that begins in stream c.  A warp takes
// 8 rows and D / 4 columns of them, lane (row, c) columns 4 (c + 4 i) of its quarter ..: every load is four runs of 128
// bytes.  Bound by the latency of the loads (four parts in flight): 6 to 8 us for the 304 parts of 16 or 32 rows, 8 to 13 us
// for 152 of 256 rows (40 MB at most, of which DRAM sees little).
constexpr int MERGE_ROWS = 8, MERGE_WARPS = 4;
template <int D>
__global__ void __launch_bounds__(MERGE_WARPS * 32) tree_merge_kernel(const Params p)
{
    constexpr int NG = D / 4 / 4 / MERGE_WARPS, BATCH = 4;         // groups of 4 columns a lane; parts in flight
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, row = blockIdx.y * MERGE_ROWS + (lane & 7), c0 = blockIdx.x;
    const int g0 = warp * 4 * NG + (lane >> 3);
    pdl_launch();
    pdl_wait();
    const ::int4 *meta = reinterpret_cast<const ::int4 *>(p.meta + (size_t)c0 * META);
    const ::int4 a = __ldcg(meta);
    if (row >= a.x) return;
    const ::int4 u = __ldcg(meta + 1);
    const int c1 = a.y, row0 = a.w, h = u.x, y = u.y * p.rows_unit + row, i = y / p.group, hh = y - i * p.group;
    float M = -INFINITY, den = 0.f;
    float4 num[NG];
#pragma unroll
    for (int x = 0; x < NG; ++x) num[x] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
    for (int c = c0; c <= c1; c += BATCH) {
        float2 ml[BATCH];
        float4 o[BATCH][NG];
#pragma unroll
        for (int k = 0; k < BATCH; ++k) {
            ml[k] = make_float2(-INFINITY, 0.f);
#pragma unroll
            for (int x = 0; x < NG; ++x) o[k][x] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (c + k <= c1) {
                const size_t slot = (size_t)(c + k) * 2 + (c + k == c0 ? a.z : 0);
                ml[k] = __ldcg(reinterpret_cast<const float2 *>(p.part_ml) + slot * p.rows_unit + row);
#pragma unroll
                for (int x = 0; x < NG; ++x)
                    o[k][x] = __ldcg(reinterpret_cast<const float4 *>(p.part_o) + (slot * (D / 4) + g0 + 4 * x) * p.rows_unit + row);
            }
        }
        float top = M;
#pragma unroll
        for (int k = 0; k < BATCH; ++k) top = fmaxf(top, ml[k].x);
        // (a part without a position that the row sees has the maximum -infinity, or a NaN sum, which stays)
        const float f = M == top ? 1.f : dev::fast_exp2(M - top);
        den *= f;
#pragma unroll
        for (int x = 0; x < NG; ++x) num[x] = make_float4(num[x].x * f, num[x].y * f, num[x].z * f, num[x].w * f);
#pragma unroll
        for (int k = 0; k < BATCH; ++k) {
            const float w = ml[k].x == top ? 1.f : dev::fast_exp2(ml[k].x - top);
            den = fmaf(ml[k].y, w, den);
#pragma unroll
            for (int x = 0; x < NG; ++x)
                num[x] = make_float4(fmaf(o[k][x].x, w, num[x].x), fmaf(o[k][x].y, w, num[x].y), fmaf(o[k][x].z, w, num[x].z),
                                     fmaf(o[k][x].w, w, num[x].w));
        }
        M = top;
    }
    const float inv = den == 0.f ? 0.f : p.out_scale / den;
    uint16_t *dst = p.out + ((size_t)(row0 + i) * p.Hq + (size_t)h * p.group + hh) * D;
#pragma unroll
    for (int x = 0; x < NG; ++x)
        *reinterpret_cast<uint2 *>(dst + 4 * (g0 + 4 * x)) = make_uint2(dev::pack_bf16x2(num[x].x * inv, num[x].y * inv), dev::pack_bf16x2(num[x].z * inv, num[x].w * inv));
}

// ------------------------------------------------------------------------------------
// Host side.
// ------------------------------------------------------------------------------------
// SMs of the current device, asked for once for each.
int sm_count()
{
    static std::atomic<int> known[64];
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    if (dev < 64 && (n = known[dev].load(std::memory_order_relaxed)) > 0) return n;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    if (dev < 64) known[dev].store(n, std::memory_order_relaxed);
    return n;
}

// Rows per unit by the most rows of a sequence and KV head: 16 or 32 on mma.sync, above that the tcgen05 kernel's.
constexpr int MOST_MMA_ROWS = 32;
int rows_per_unit(int max_q, int group, bool few)
{
    const int rows = max_q * group;
    return rows <= 16 ? 16 : rows <= MOST_MMA_ROWS || few ? 32 : tcgen05_tokens(group) * group;
}

// Few tiles: even with the tables full, 32 rows at a time, no more of them than the mma.sync grid has CTAs.  Then a call is
// the kernels' latency, which is less without tensor memory and twenty warps (13 drafts of 4 heads behind 60 positions,
// 8 KV heads, in a graph: 12.6 us against 15.4; behind 1500, where there are more, 16.0 against 14.9).  Not every CTA gets
// one of them, since the units' cost is dealt out with the tiles: of 96 tiles on 96 CTAs (16 units of 6) a third have none
// and a third two; where short units stand beside a long one a CTA may get three.
bool few_tiles(const pkv_pool_desc &d, int batch, int max_blocks, int max_q, int group)
{
    const int64_t tiles = (int64_t)batch * d.num_kv_heads * ((max_blocks + TB - 1) / TB) * (((int64_t)max_q * group + 31) / 32);
    return tiles <= (int64_t)2 * sm_count();
}

// What a unit costs besides its tiles, in tiles (see places_of).  64 ragged sequences with 8 drafts: 65 us, 73 with a cost of
// 1; 37 ragged trees on tcgen05: 70, 73 with 6, 78 with 10.
constexpr int UNIT_COST = 3, UNIT_COST_TCGEN05 = 3;

struct Room { int grid, rows; size_t o, ml, q, up, bytes; };
Room room(const pkv_pool_desc &d, int batch, int max_q, int num_q_heads, bool few)
{
    const int D = d.head_dim, group = num_q_heads / d.num_kv_heads;
    Room r;
    r.rows = rows_per_unit(max_q, group, few);
    r.grid = sm_count() * (r.rows <= MOST_MMA_ROWS ? 2 : 1);
    r.o = ((size_t)r.grid * META * 4 + 255) / 256 * 256;
    r.ml = r.o + ((size_t)r.grid * 2 * r.rows * D * 4 + 255) / 256 * 256;
    r.q = r.ml + ((size_t)r.grid * 2 * r.rows * 2 * 4 + 255) / 256 * 256;
    const size_t q_rows = r.rows > MOST_MMA_ROWS && d.kv_dtype != PKV_KV_BF16 ? (size_t)batch * max_q * num_q_heads : 0;
    r.up = r.q + (q_rows * D * 2 + 255) / 256 * 256;
    r.bytes = r.up + (q_rows + 255) / 256 * 256;
    return r;
}

template <int D, int KIND, int WR, int WK>
cudaError_t launch(const CUtensorMap &km, const CUtensorMap &vm, const Params &p, int grid, cudaStream_t s)
{
    using S = Shape<D, KIND, WR, WK>;
    auto kernel = tree_kernel<D, KIND, WR, WK>;
    // (an attribute of the function on the current device: once for each of them)
    static std::atomic<uint64_t> asked{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 64 || !((asked.load() >> dev) & 1u)) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, S::ALLOC);
        if (e != cudaSuccess) return e;
        if (dev < 64) asked.fetch_or(1ull << dev);
    }
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(S::NT);
    cfg.dynamicSmemBytes = S::ALLOC;
    cfg.stream = s;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, kernel, km, vm, p);
    return e;
}

template <int D>
cudaError_t launch_merge(const Params &p, int grid, cudaStream_t s)
{
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)grid, (unsigned)((p.rows_unit + MERGE_ROWS - 1) / MERGE_ROWS));
    cfg.blockDim = dim3(MERGE_WARPS * 32);
    cfg.stream = s;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, tree_merge_kernel<D>, p);
}

template <int D, int KIND>
cudaError_t launch_rows(int mr, const CUtensorMap &km, const CUtensorMap &vm, const Params &p, int grid, cudaStream_t s)
{
    if (mr == 16) return launch<D, KIND, 1, 4>(km, vm, p, grid, s);
    return launch<D, KIND, 2, 2>(km, vm, p, grid, s);
}

bool aligned(const void *ptr, uintptr_t a) { return (reinterpret_cast<uintptr_t>(ptr) & (a - 1)) == 0; }

// Both entry points; cu_q null: one row per sequence.
int run(pkv_pool *pool, const void *q, const void *key_cache, const void *value_cache, const int32_t *block_tables,
        const int32_t *seq_lens, const int32_t *cu_q, const int64_t *tree_mask, int32_t batch, int32_t num_q_heads,
        int32_t max_blocks, int32_t total_q, int32_t max_q, float scale, int32_t window, int32_t sinks, void *out,
        void *workspace, size_t workspace_bytes, void *stream)
{
    const int st = check_attached(pool);
    if (st != PKV_OK) return st;
    const pkv_pool_desc &d = pool->desc;
    if (batch < 0 || batch > MOST_BATCH || num_q_heads < 1 || max_blocks < 1 || max_blocks > MOST_TABLE_BLOCKS || total_q < 0 ||
        max_q < 1 || max_q > MOST_NEW || !std::isfinite(scale) || window < 0 || sinks < 0)
        return PKV_ERR_INVALID;
    if (num_q_heads % d.num_kv_heads || num_q_heads / d.num_kv_heads > 16) return PKV_ERR_INVALID;
    if ((int64_t)batch * max_blocks * d.num_kv_heads >= (int64_t)1 << 31) return PKV_ERR_INVALID;
    if (tree_mask && window > 0 && window < max_q) return PKV_ERR_INVALID;
    if (batch == 0 || total_q == 0) return PKV_OK;
    if (!q || !key_cache || !value_cache || !block_tables || !seq_lens || !out || !workspace) return PKV_ERR_INVALID;
    // (rows are written while other CTAs still read theirs)
    const uint64_t q_bytes = (uint64_t)total_q * num_q_heads * d.head_dim * 2;
    const uint64_t qa = reinterpret_cast<uintptr_t>(q), oa = reinterpret_cast<uintptr_t>(out);
    if (qa < oa + q_bytes && oa < qa + q_bytes) return PKV_ERR_INVALID;
    if (!aligned(q, 16) || !aligned(key_cache, 16) || !aligned(value_cache, 16) || !aligned(out, 16) || !aligned(block_tables, 4) ||
        !aligned(seq_lens, 4) || !aligned(cu_q, 4) || !aligned(tree_mask, 8) || !aligned(workspace, 256))
        return PKV_ERR_INVALID;
    const int D = d.head_dim, group = num_q_heads / d.num_kv_heads;
    const Room rm = room(d, batch, max_q, num_q_heads, few_tiles(d, batch, max_blocks, max_q, group));
    // (places of all units, with their cost, in 31 bits)
    const int64_t units = (int64_t)batch * d.num_kv_heads * (((int64_t)max_q * group + rm.rows - 1) / rm.rows);
    if (units * ((max_blocks + TB - 1) / TB + std::max(UNIT_COST, UNIT_COST_TCGEN05)) >= (int64_t)1 << 31) return PKV_ERR_INVALID;
    const bool many = rm.rows > MOST_MMA_ROWS;
    if (rm.grid < 1) return PKV_ERR_CUDA;
    if (workspace_bytes < rm.bytes) return PKV_ERR_INVALID;
    CUtensorMap qm{}, km{}, vm{};
    if (d.kv_dtype == PKV_KV_BF16) {
        const uint64_t tiles = (uint64_t)d.num_blocks * d.num_kv_heads;
        bool ok;
        // a block in one copy, 64 columns after the other; for the tcgen05 kernel K's halves by themselves
        const uint64_t dims[3] = {(uint64_t)D, BS, tiles}, strides[2] = {(uint64_t)D * 2, (uint64_t)D * 2 * BS};
        const uint32_t box[3] = {64, BS, 1};
        const uint64_t dims4[4] = {64, BS, 2, tiles}, strides4[3] = {256, 128, 256 * BS};
        const uint32_t box4[4] = {64, BS, 2, 1};
        auto map = [&](CUtensorMap *m, const void *cache, bool whole) {
            return whole ? encode_tiled(m, cache, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, dims4, strides4, box4, CU_TENSOR_MAP_SWIZZLE_128B)
                         : encode_tiled_3d(m, cache, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
        };
        ok = map(&km, key_cache, D == 128 && !many) && map(&vm, value_cache, D == 128);
        if (!ok) return PKV_ERR_CUDA;
    }
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    const void *q_tiles = q;                                       // what the tcgen05 kernel copies
    uint64_t q_rows = (uint64_t)total_q;
    if (many && d.kv_dtype != PKV_KV_BF16) {
        q_tiles = ws + rm.q;
        q_rows = (uint64_t)batch * max_q;
    }
    if (many) {
        // eight tokens' rows of a KV head's group
        const uint64_t dims[3] = {(uint64_t)D, (uint64_t)num_q_heads, q_rows}, strides[2] = {(uint64_t)D * 2, (uint64_t)num_q_heads * D * 2};
        const uint32_t box[3] = {64, (uint32_t)group, 8};
        if (!encode_tiled_3d(&qm, q_tiles, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B)) return PKV_ERR_CUDA;
    }
    const int most = max_blocks * BS;                              // no position is beyond
    Params p;
    p.q = static_cast<const uint16_t *>(q);
    p.q16 = reinterpret_cast<uint16_t *>(ws + rm.q);
    p.q_up = reinterpret_cast<int8_t *>(ws + rm.up);
    p.key_cache = static_cast<const uint8_t *>(key_cache);
    p.value_cache = static_cast<const uint8_t *>(value_cache);
    p.tables = block_tables;
    p.lens = seq_lens;
    p.cu = cu_q;
    p.mask = reinterpret_cast<const unsigned long long *>(tree_mask);
    p.out = static_cast<uint16_t *>(out);
    p.part_o = reinterpret_cast<float *>(ws + rm.o);
    p.part_ml = reinterpret_cast<float *>(ws + rm.ml);
    p.meta = reinterpret_cast<int32_t *>(ws);
    p.err = pool->d_err;
    p.B = batch;
    p.MB = max_blocks;
    p.Hq = num_q_heads;
    p.Hkv = d.num_kv_heads;
    p.group = group;
    p.num_blocks = d.num_blocks;
    p.total_q = total_q;
    p.max_q = max_q;
    p.words = (max_q + 63) / 64;
    p.window = window >= most ? 0 : window;
    p.sinks = std::min(sinks, most);
    p.rows_unit = rm.rows;
    p.unit_cost = many ? UNIT_COST_TCGEN05 : UNIT_COST;
    p.test_stall = test_expire() == PKV_TEST_EXPIRE_DECODE;
    p.score_scale = scale * d.k_scale * LOG2E;
    p.out_scale = d.v_scale;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (many) e = launch_tcgen05(D, d.kv_dtype, qm, km, vm, p, rm.grid, s);
    else if (d.kv_dtype == PKV_KV_BF16) e = D == 128 ? launch_rows<128, BF16>(rm.rows, km, vm, p, rm.grid, s) : launch_rows<64, BF16>(rm.rows, km, vm, p, rm.grid, s);
    else if (d.kv_dtype == PKV_KV_FP8E4M3) e = D == 128 ? launch_rows<128, FP8>(rm.rows, km, vm, p, rm.grid, s) : launch_rows<64, FP8>(rm.rows, km, vm, p, rm.grid, s);
    else e = D == 128 ? launch_rows<128, INT4>(rm.rows, km, vm, p, rm.grid, s) : launch_rows<64, INT4>(rm.rows, km, vm, p, rm.grid, s);
    if (e == cudaSuccess && max_blocks > TB)                       // (with a tile at most no unit is cut)
        e = D == 128 ? launch_merge<128>(p, rm.grid, s) : launch_merge<64>(p, rm.grid, s);
    return e == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

}  // namespace tree
}  // namespace pkv

extern "C" size_t pkv_tree_workspace_bytes(const pkv_pool *pool, int32_t batch, int32_t num_q_heads, int32_t max_q)
{
    using namespace pkv::tree;
    if (!pool || batch < 1 || batch > MOST_BATCH || num_q_heads < 1 || num_q_heads % pool->desc.num_kv_heads || max_q < 1 || max_q > MOST_NEW)
        return 0;
    const int g = num_q_heads / pool->desc.num_kv_heads;
    if (g > 16 || sm_count() < 1) return 0;
    // (which kernel a call takes depends on its max_blocks as well)
    return std::max(room(pool->desc, batch, max_q, num_q_heads, false).bytes, room(pool->desc, batch, max_q, num_q_heads, true).bytes);
}

extern "C" int pkv_paged_attention_tree(pkv_pool *pool, const void *q, const void *key_cache, const void *value_cache,
                                        const int32_t *block_tables, const int32_t *seq_lens, const int32_t *cu_q,
                                        const int64_t *tree_mask, int32_t batch, int32_t num_q_heads, int32_t max_blocks,
                                        int32_t total_q, int32_t max_q, float scale, int32_t window, int32_t sinks, void *out,
                                        void *workspace, size_t workspace_bytes, void *stream)
{
    if (batch > 0 && total_q > 0 && !cu_q) return PKV_ERR_INVALID;
    return pkv::tree::run(pool, q, key_cache, value_cache, block_tables, seq_lens, cu_q, tree_mask, batch, num_q_heads, max_blocks,
                          total_q, max_q, scale, window, sinks, out, workspace, workspace_bytes, stream);
}

extern "C" int pkv_paged_attention_window(pkv_pool *pool, const void *q, const void *key_cache, const void *value_cache,
                                          const int32_t *block_tables, const int32_t *seq_lens, int32_t batch, int32_t num_q_heads,
                                          int32_t max_blocks, float scale, int32_t window, int32_t sinks, void *out,
                                          void *workspace, size_t workspace_bytes, void *stream)
{
    return pkv::tree::run(pool, q, key_cache, value_cache, block_tables, seq_lens, nullptr, nullptr, batch, num_q_heads, max_blocks,
                          batch, 1, scale, window, sinks, out, workspace, workspace_bytes, stream);
}
