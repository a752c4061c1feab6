// tree_tcgen05.cu -- the attention of tree_attention.cu for many rows per KV head, on the tcgen05 tensor cores.
//
// Above some 64 rows (tokens times the group's heads) the products bind, not the reading of K and V: 256 rows on
// mma.sync ran at a tenth of what the fifth-generation tensor cores give.  A unit is (sequence, KV head, 256 rows)
// as two q-tiles of 128, of which the second rests where a unit has no more than 128 rows; a tile is 64 keys of
// the unit's visible blocks.  The work is divided as in tree_attention.cu: every CTA of a one-wave grid takes an
// even share of all tiles, and partial states of cut units are merged by the same second launch.
//
// Twenty warps, one CTA per SM.  Warps 0-3 and 4-7: softmax of q-tiles 0 and 1, a row per thread; 8, 9 issue S = Q K^T
// of the q-tiles (M 128, N 64) and 10, 11 O += P V (M 128, N D, P from tensor memory); 12, 13 bring K, 16, 17 V, 14 Q.
// S is double-buffered in tensor memory and P overwrites it, O stays there; S of tile J waits for P V of tile J - 2
// of its q-tile.  One issuing thread per product and q-tile, since a thread issues a tcgen05.mma only every 36 to 60 ns.
//   * bf16 pools: tensor copies with 128-byte swizzle straight into the operand rings.
//   * FP8 and INT4 pools: bulk copies of the blocks as stored into staging rings, expanded (exactly) to f16 operand
//     tiles by two warps for K and two for V; q to f16 by a power of two per row (warp 14), P in f16 times 2^8.  Four
//     expanding warps beside eight of softmax need registers moved between warpgroups (setmaxnreg: 96 a thread at
//     launch, 144 for softmax, 64 for the others, which is the same sum).
//   * V that must not meet the tensor core is zeroed in its operand tile before P V, by the warps that bring V:
//     what is not there, and, of positions that some rows of the unit do not see, those that are not finite
//     (0 x NaN is NaN); the softmax threads of rows that do see such a position add its product themselves.
// All waits are bounded (about 1 s, then PKV_DEVERR_TIMEOUT, and the copies in flight are waited for).
#include <atomic>

#include "tree_common.cuh"

namespace pkv {
namespace tree {

__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

constexpr int BM = 128, BN = TB * BS, TC_THREADS = 640;
constexpr int REG_LAUNCH = 96, REG_SOFTMAX = 144, REG_OTHER = 64;
static_assert(256 * REG_SOFTMAX + 384 * REG_OTHER <= TC_THREADS * REG_LAUNCH, "registers that the launch has");
constexpr uint32_t NEGATE_A = 1u << 13;        // instruction descriptor: A enters the product negated
constexpr uint32_t TMEM_COLS = 512;            // S (and P over it): 2 buffers x 2 q-tiles x 64, O: 2 x D
constexpr int LEAD = 16;                       // ring of tiles' masks: more than any warp runs ahead of another

template <int D, int KIND>
struct Tc {
    static constexpr int H = D / 64;
    static constexpr int NS = KIND == BF16 ? (D == 128 ? 5 : 8) : (D == 128 ? 3 : 4);       // operand tiles of K and V
    static constexpr int TILE = KIND == BF16 ? BS * D * 2 : KIND == FP8 ? BS * D : int4::tile_bytes(D);
    static constexpr int RAW = TB * TILE;
    static constexpr int NSG = KIND == BF16 ? 0 : KIND == FP8 && D == 128 ? 4 : D == 128 ? 6 : 8;     // staging tiles
    static constexpr int QHALF = 2 * BM * 128, KHALF = BN * 128, KSTAGE = H * KHALF;
    static constexpr int K = H * QHALF, V = K + NS * KSTAGE, SK = V + NS * KSTAGE, SV = SK + NSG * RAW;
    static constexpr int QEXP = SV + NSG * RAW;                    // int8 [256]
    static constexpr int INFO = QEXP + (KIND == BF16 ? 0 : 256);      // u64 sure, live, bad [LEAD], then int got [LEAD]
    static constexpr int BAR = INFO + LEAD * 28;
    static constexpr int NRAW = KIND == BF16 ? NS : NSG;
    static constexpr int BARS = 3 + 4 * NS + 4 + 4 + 4 + 2 + 1 + NRAW + 3 * NSG;
    static constexpr int ALLOC = BAR + BARS * 8 + 16 + 1024;
    static_assert(ALLOC <= 227 * 1024 && NS + NSG + 3 < LEAD && RAW % 128 == 0 && BAR % 8 == 0, "shared memory");
};

template <int N>
__device__ __forceinline__ void more_registers() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void fewer_registers() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

// Element (token t, column d) of a block of V as the operand tiles hold it (without the pool's scale).
template <int D, int KIND>
__device__ __forceinline__ float v_element(const uint8_t *tile, int t, int d)
{
    if constexpr (KIND == BF16) {
        return __uint_as_float((uint32_t)__ldcg(reinterpret_cast<const uint16_t *>(tile) + t * D + d) << 16);
    } else if constexpr (KIND == FP8) {
        return int4::scale_value(__ldcg(tile + t * D + d));        // (E4M3, as the INT4 pools' scales are)
    } else {
        using P = int4::Place<D>;
        const int o = d >> 3, i = d & 7;
        const uint32_t w = __ldcg(reinterpret_cast<const uint16_t *>(tile + P::v_word(t, o) + (i >> 2) * P::VSTEP));
        return ((float)((w >> (4 * (i & 3))) & 15u) - 8.f) * int4::scale_value(__ldcg(tile + P::v_scale(t, o)));
    }
}

// Zero the rows of a block of V (16 tokens, its operand tile in 16 bits) that must not meet the tensor core, by a
// warp: those that are not there, and those that are not finite while some row of the unit does not see
// them, which are returned.
template <int D, int KIND, int HALF>
__device__ __forceinline__ uint32_t clean_v(uint8_t *dst, uint32_t there16, uint32_t sure16, int lane)
{
    if (sure16 == 0xffffu) return 0;
    constexpr uint32_t EXP = KIND == BF16 ? 0x7f80u : 0x7c00u;
    constexpr int CHUNKS = D / 16;                                 // half a row a lane
    const int row = lane >> 1, part = lane & 1;
    uint4 *at = reinterpret_cast<uint4 *>(dst + (D == 128 ? part * HALF : 0) + row * 128 + (D == 128 ? 0 : part * 64));
    bool odd = false;
#pragma unroll
    for (int c = 0; c < CHUNKS; ++c) {
        const uint4 v = at[c];
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) odd |= (w[e] & EXP) == EXP || ((w[e] >> 16) & EXP) == EXP;
    }
    odd |= __shfl_xor_sync(dev::FULL, (int)odd, 1) != 0;
    const bool is = (there16 >> row) & 1u, keep_out = is && !((sure16 >> row) & 1u) && odd;
    if (!is || keep_out) {
#pragma unroll
        for (int c = 0; c < CHUNKS; ++c) at[c] = make_uint4(0u, 0u, 0u, 0u);
    }
    const uint32_t both = __ballot_sync(dev::FULL, keep_out);
    uint32_t rows = 0;
    if (both)
        for (int r = 0; r < BS; ++r) rows |= ((both >> (2 * r)) & 1u) << r;
    return rows;
}

template <int D, int KIND>
__global__ void __launch_bounds__(TC_THREADS, 1)
tree_tcgen05_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                    const __grid_constant__ CUtensorMap vmap, const Params p)
{
    using L = Tc<D, KIND>;
    constexpr int H = L::H, NS = L::NS, NSG = L::NSG;
    constexpr bool WIDE = KIND != BF16;
    constexpr float SHIFT = WIDE ? 8.f : 0.f, TAU = WIDE ? 7.f : 8.f;      // P 2^SHIFT, at most 2^TAU above the running max
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = smem_raw + ((1024u - (dev::smem_u32(smem_raw) & 1023u)) & 1023u);
    const uint32_t base = dev::smem_u32(sm);
    const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(dev::FULL, tid >> 5, 0);
    unsigned long long *sure = reinterpret_cast<unsigned long long *>(sm + L::INFO), *there = sure + LEAD;
    uint32_t *bad = reinterpret_cast<uint32_t *>(there + LEAD);    // [LEAD][2]
    volatile int *got_k = reinterpret_cast<volatile int *>(bad + 2 * LEAD);
    int8_t *qexp = reinterpret_cast<int8_t *>(sm + L::QEXP);
    const uint32_t bars = base + L::BAR;
    const uint32_t q_full = bars, q_ready = bars + 8, q_free = bars + 16;
    auto k_full = [&](int s) { return bars + 8 * (3 + s); };
    auto v_full = [&](int s) { return bars + 8 * (3 + NS + s); };
    auto k_free = [&](int s) { return bars + 8 * (3 + 2 * NS + s); };
    auto v_free = [&](int s) { return bars + 8 * (3 + 3 * NS + s); };
    auto s_full = [&](int w, int J) { return bars + 8 * (3 + 4 * NS + 2 * w + (J & 1)); };
    auto p_full = [&](int w, int J) { return bars + 8 * (7 + 4 * NS + 2 * w + (J & 1)); };
    auto pv_done = [&](int w, int J) { return bars + 8 * (11 + 4 * NS + 2 * w + (J & 1)); };
    auto o_free = [&](int w) { return bars + 8 * (15 + 4 * NS + w); };
    const uint32_t never = bars + 8 * (17 + 4 * NS);
    auto v_raw = [&](int x) { return bars + 8 * (18 + 4 * NS + x); };
    auto k_raw = [&](int x) { return bars + 8 * (18 + 4 * NS + L::NRAW + x); };
    auto raw_free = [&](bool isk, int x) { return bars + 8 * (18 + 4 * NS + L::NRAW + NSG + (isk ? 0 : NSG) + x); };
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sm + L::BAR + L::BARS * 8);

    if (tid == 0) {
        dev::mbar_init(q_full, 1);
        dev::mbar_init(q_ready, 1);
        dev::mbar_init(q_free, WIDE ? 10 : 2);                     // both S issuers (and the softmax warps: exponents)
        for (int s = 0; s < NS; ++s) {
            dev::mbar_init(k_full(s), WIDE ? 2 : 1);               // the expanding warps, or the copy
            dev::mbar_init(v_full(s), 2);                          // the expanding warps; the copy, and warp 17's look
            dev::mbar_init(k_free(s), 2);                          // both q-tiles' S
            dev::mbar_init(v_free(s), 2);                          // both q-tiles' P V
        }
        for (int w = 0; w < 2; ++w) {
            for (int x = 0; x < 2; ++x) {
                dev::mbar_init(s_full(w, x), 1);
                dev::mbar_init(p_full(w, x), 4);                   // the q-tile's softmax warps
                dev::mbar_init(pv_done(w, x), 1);
            }
            dev::mbar_init(o_free(w), 4);
        }
        dev::mbar_init(never, 1);
        for (int x = 0; x < L::NRAW; ++x) dev::mbar_init(v_raw(x), 1);
        for (int x = 0; x < NSG; ++x) {
            dev::mbar_init(k_raw(x), 1);
            dev::mbar_init(raw_free(true, x), 1);
            dev::mbar_init(raw_free(false, x), 1);
        }
        dev::fence_barrier_init();
    }
    pdl_launch();
    pdl_wait();
    const Share my = share_of<TC_THREADS, D>(p, *reinterpret_cast<ShareScratch<TC_THREADS> *>(sm));      // (Q's room, not yet in use)
    if (my.first >= my.last) return;
    if (warp == 15) tc::tmem_alloc(dev::smem_u32(tmem_slot), TMEM_COLS);
    tc::fence_before_sync();
    dev::fence_proxy_async_smem();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    auto tS = [&](int b, int w) { return tmem + (uint32_t)((2 * b + w) * BN); };
    auto tO = [&](int w) { return tmem + 256u + (uint32_t)(w * D); };
    const int nt = (int)(my.last - my.first), tokens = p.rows_unit / p.group;

    // (a warpgroup's registers are moved before its warps part)
    if (warp < 8) {
        more_registers<REG_SOFTMAX>();
        // ============ softmax and output: a row per thread, all keys of a tile, all columns
        const int w = warp >> 2, q4 = warp & 3, rg = w * BM + 32 * q4 + lane;      // row of the unit
        const uint32_t lane_off = (uint32_t)(32 * q4) << 16;
        Walk walk(p, my);
        int J = 0, Jw = 0, uq = 0;
        bool ok = true, cut_begins = false;
        int cut[META] = {};
        for (long long r = my.first; ok && r < my.last; ++uq) {
            const Segment g = walk.at(p, r);
            const Seq &sq = walk.sq;
            const int i0 = g.m * tokens, i1 = min(sq.P, i0 + tokens) - 1, rows = (i1 + 1 - i0) * p.group;
            const bool whole = g.t0 == 0 && g.t1 == sq.nt;
            const int slot = r == my.first ? 0 : 1;
            if (g.t0 == 0 && !whole) {
                cut_begins = true;
                cut[0] = rows;
                cut[1] = stream_of(r + sq.nt - 1, my.W, my.streams);
                cut[2] = slot;
                cut[3] = sq.row0;
                cut[4] = g.h;
                cut[5] = g.m;
            }
            const bool live = rg < rows;
            float sc = fabsf(p.score_scale);
            if constexpr (WIDE) {
                ok = __all_sync(dev::FULL, dev::mbar_wait_bounded(q_ready, (uint32_t)(uq & 1)));
                if (!ok) break;
                if (live) sc = row_scale(sc, qexp[rg]);
                __syncwarp();
                if (lane == 0) dev::mbar_arrive(q_free);
            }
            if (rows <= BM * w) {                                  // this q-tile rests
                J += g.t1 - g.t0;
                r += g.t1 - g.t0;
                continue;
            }
            const int token = i0 + (live ? rg / p.group : 0), hh = live ? rg - (token - i0) * p.group : 0;
            const int place = p.mask && p.window ? place_of(p, sq, token) : sq.C + token;
            sc = sc == sc ? fmaxf(sc, 1e-37f) : sc;                // (masked scores stay -infinity)
            const int to = all_to(p, sq, i0), from = all_from(p, sq, i1);
            float m = -INFINITY, l = 0.f;
            for (int t = g.t0; t < g.t1; ++t, ++J, ++Jw) {
                ok = __all_sync(dev::FULL, dev::mbar_wait_bounded(s_full(w, Jw), (uint32_t)((Jw >> 1) & 1)));
                if (!ok) break;
                tc::fence_after_sync();
                float x[BN];
                {
                    uint32_t v0[32], v1[32];
                    tc::tmem_ld32(tS(Jw & 1, w) + lane_off, v0);
                    tc::tmem_ld32(tS(Jw & 1, w) + lane_off + 32, v1);
                    tc::tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        x[i] = __uint_as_float(v0[i]);
                        x[32 + i] = __uint_as_float(v1[i]);
                    }
                }
                const int got = got_k[J % LEAD];
                bool edge = got != (1 << TB) - 1;
#pragma unroll
                for (int k = 0; k < TB; ++k) {
                    const int p0 = walk.block(TB * t + k) * BS;
                    edge |= p0 + BS > to || (p0 < from && p0 + BS > p.sinks);
                }
                if (edge) {
#pragma unroll
                    for (int k = 0; k < TB; ++k) {
                        const int p0 = walk.block(TB * t + k) * BS;
                        const uint32_t see = live ? seen16(p, sq, token, place, p0, (got >> k) & 1 ? ones(sq.L - p0) : 0u) : 0u;
#pragma unroll
                        for (int c = 0; c < BS; ++c)
                            if (!((see >> c) & 1u)) x[BS * k + c] = -INFINITY;
                    }
                }
                float mx4[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
                for (int c = 4; c < BN; c += 8)
#pragma unroll
                    for (int e = 0; e < 4; ++e) mx4[e] = c + 4 + e < BN ? tc::fmax3(mx4[e], x[c + e], x[c + 4 + e]) : fmaxf(mx4[e], x[c + e]);
                const float top = tc::fmax3(mx4[0], mx4[1], fmaxf(mx4[2], mx4[3]));
                const float d = (top - m) * sc;
                const bool raise = d > TAU || (m == -INFINITY && top > m), rescale = raise && m != -INFINITY;
                const float f = rescale ? dev::fast_exp2(-d) : 1.f;
                if (raise) m = top;
                const float nm = m == -INFINITY ? 0.f : -m, ns = nm * sc + SHIFT;
                uint32_t pw[BN / 2];
                const float2 sc2 = make_float2(sc, sc);
                float2 ps[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
                auto put = [&](int e, float2 v) {
                    const float2 pe = make_float2(dev::fast_exp2(v.x), dev::fast_exp2(v.y));
                    ps[e & 1] = tc::fadd2(ps[e & 1], pe);
                    pw[e] = WIDE ? dev::pack_f16x2(pe.x, pe.y) : dev::pack_bf16x2(pe.x, pe.y);
                };
                // m's product with the scale may join the exponents while its rounding is below 2^-16
                if (!__any_sync(dev::FULL, fabsf(ns) > 256.f)) {
                    const float2 ns2 = make_float2(ns, ns);
#pragma unroll
                    for (int e = 0; e < BN / 2; ++e) put(e, tc::ffma2(make_float2(x[2 * e], x[2 * e + 1]), sc2, ns2));
                } else {
                    const float2 nm2 = make_float2(nm, nm), sh2 = make_float2(SHIFT, SHIFT);
#pragma unroll
                    for (int e = 0; e < BN / 2; ++e) put(e, tc::ffma2(tc::fadd2(make_float2(x[2 * e], x[2 * e + 1]), nm2), sc2, sh2));
                }
                const float2 ps2 = tc::fadd2(ps[0], ps[1]);
                l = l * f + (ps2.x + ps2.y);
                tc::tmem_st32(tS(Jw & 1, w) + lane_off, pw);       // over this tile's S, which is read
                if (__any_sync(dev::FULL, rescale)) {
                    ok = __all_sync(dev::FULL, dev::mbar_wait_bounded(pv_done(w, Jw - 1), (uint32_t)(((Jw - 1) >> 1) & 1)));
                    if (!ok) break;
                    tc::fence_after_sync();
#pragma unroll 1
                    for (int c = 0; c < D / 32; ++c) {
                        uint32_t v[32];
                        tc::tmem_ld32(tO(w) + lane_off + 32 * c, v);
                        tc::tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 32; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * f);
                        tc::tmem_st32(tO(w) + lane_off + 32 * c, v);
                    }
                }
                tc::tmem_wait_st();
                unsigned long long odd = 0;                        // positions whose V was kept from the tensor core
                if (edge) {
                    ok = __all_sync(dev::FULL, dev::mbar_wait_bounded(v_full(J % NS), (uint32_t)((J / NS) & 1)));
                    if (!ok) break;
                    const volatile uint32_t *vb = bad + 2 * (J % LEAD);
                    odd = vb[0] | (unsigned long long)vb[1] << 32;
                }
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) dev::mbar_arrive(p_full(w, Jw));
                if (edge) {
                    if (odd) {                                     // their products, where this row sees them
                        ok = __all_sync(dev::FULL, dev::mbar_wait_bounded(pv_done(w, Jw), (uint32_t)((Jw >> 1) & 1)));
                        if (!ok) break;
                        tc::fence_after_sync();
                        for (unsigned long long left = odd; left; left &= left - 1) {
                            const int j = __ffsll((long long)left) - 1, k = j / BS;
                            const int blk = walk.block(TB * t + k), id = __ldcg(p.tables + (size_t)walk.b * p.MB + blk);
                            const uint8_t *tile = p.value_cache + ((size_t)id * p.Hkv + g.h) * L::TILE;
                            const uint32_t see = live ? seen16(p, sq, token, place, blk * BS, ones(sq.L - blk * BS)) : 0u;
                            float pj = 0.f;
#pragma unroll
                            for (int e = 0; e < BN / 2; ++e)
                                if (e == j >> 1) {
                                    if constexpr (WIDE) {
                                        const float2 h = __half22float2(*reinterpret_cast<const __half2 *>(&pw[e]));
                                        pj = j & 1 ? h.y : h.x;
                                    } else {
                                        pj = j & 1 ? dev::bf16_hi(pw[e]) : dev::bf16_lo(pw[e]);
                                    }
                                }
                            const bool mine = (see >> (j % BS)) & 1u;
#pragma unroll 1
                            for (int c = 0; c < D; c += 32) {
                                uint32_t v[32];
                                tc::tmem_ld32(tO(w) + lane_off + c, v);
                                tc::tmem_wait_ld();
#pragma unroll
                                for (int e = 0; e < 32; ++e) {
                                    const float y = v_element<D, KIND>(tile, j % BS, c + e);
                                    if (mine) v[e] = __float_as_uint(fmaf(pj, y, __uint_as_float(v[e])));
                                }
                                tc::tmem_st32(tO(w) + lane_off + c, v);
                                tc::tmem_wait_st();
                            }
                        }
                        tc::fence_before_sync();                   // (before the next p_full, or the output below)
                    }
                }
            }
            if (!ok) break;
            ok = __all_sync(dev::FULL, dev::mbar_wait_bounded(pv_done(w, Jw - 1), (uint32_t)(((Jw - 1) >> 1) & 1)));
            if (!ok) break;
            tc::fence_after_sync();
            const float inv = l == 0.f ? 0.f : p.out_scale / l;
            uint16_t *dst = p.out + ((size_t)(sq.row0 + token) * p.Hq + (size_t)g.h * p.group + hh) * D;
            const size_t pr = ((size_t)blockIdx.x * 2 + slot) * p.rows_unit + rg;
            if (!whole && live) reinterpret_cast<float2 *>(p.part_ml)[pr] = make_float2(m == -INFINITY ? m : m * sc, l);
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
                uint32_t v[32];
                tc::tmem_ld32(tO(w) + lane_off + 32 * c, v);
                tc::tmem_wait_ld();
                if (live && whole) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        uint32_t o4[4];
#pragma unroll
                        for (int y = 0; y < 4; ++y)
                            o4[y] = dev::pack_bf16x2(__uint_as_float(v[8 * e + 2 * y]) * inv, __uint_as_float(v[8 * e + 2 * y + 1]) * inv);
                        *reinterpret_cast<uint4 *>(dst + 32 * c + 8 * e) = make_uint4(o4[0], o4[1], o4[2], o4[3]);
                    }
                } else if (live) {
                    uint4 *o = reinterpret_cast<uint4 *>(p.part_o + pr * D + 32 * c);
#pragma unroll
                    for (int e = 0; e < 8; ++e) o[e] = make_uint4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
                }
                __syncwarp();
            }
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) dev::mbar_arrive(o_free(w));
            r += g.t1 - g.t0;
        }
        if (!ok && lane == 0) dev::flag_error(p.err, PKV_DEVERR_TIMEOUT);
        if (warp == 0 && lane < META) {
            int v = 0;
#pragma unroll
            for (int x = 0; x < META; ++x)
                if (x == lane) v = cut[x];
            p.meta[(size_t)blockIdx.x * META + lane] = ok && cut_begins ? v : 0;
        }
    } else {
        fewer_registers<REG_OTHER>();
    if (warp == 12 || warp == 16) {
        // ============ K (12) and V (16): the copies, and for FP8 and INT4 half of each tile's expansion
        const bool isk = warp == 12;
        Walk walk(p, my);
        Segment g = walk.at(p, my.first);
        long long r = my.first;
        int t = g.t0, chunk = t, n = 0;                            // n: tiles issued
        // table entries of 32 blocks (8 tiles from `chunk` on), and of the 32 after them
        auto fetch = [&](int t0) {
            const int v = TB * t0 + lane;
            return v < walk.sq.nvb && v < TB * g.t1 ? __ldcg(p.tables + (size_t)walk.b * p.MB + walk.block(v)) : -2;
        };
        int cur = fetch(t), nxt = fetch(t + 8);
        auto issue = [&]() {
            const int id = __shfl_sync(dev::FULL, cur, TB * (t - chunk) + (lane & 3));
            const bool good = lane < TB && id >= 0 && id < p.num_blocks;
            if (isk && lane < TB && id != -2 && !good) dev::flag_error(p.err, PKV_DEVERR_BLOCK_ID);
            const unsigned got = __ballot_sync(dev::FULL, good);
            bool edge = false;
            if (isk) {
                if (lane == 0) got_k[n % LEAD] = (int)got;
            } else {
                // the positions that are there, and those that every row of the unit sees
                const int p0 = walk.block(TB * t + (lane & 3)) * BS, i0 = g.m * tokens, i1 = min(walk.sq.P, i0 + tokens) - 1;
                const uint32_t l16 = good ? ones(walk.sq.L - p0) : 0u;
                uint32_t s16 = l16 & ones(all_to(p, walk.sq, i0) - p0);
                if (p.window) s16 &= ~ones(all_from(p, walk.sq, i1) - p0) | ones(p.sinks - p0);
                edge = __any_sync(dev::FULL, lane < TB && s16 != 0xffffu);
                unsigned long long a = (unsigned long long)l16 << (16 * (lane & 3)), z = (unsigned long long)s16 << (16 * (lane & 3));
                if (lane >= TB) a = z = 0;
#pragma unroll
                for (int o = 1; o < TB; o <<= 1) {
                    a |= __shfl_xor_sync(dev::FULL, a, o);
                    z |= __shfl_xor_sync(dev::FULL, z, o);
                }
                if (lane == 0) {
                    there[n % LEAD] = a;
                    sure[n % LEAD] = z;
                    if (!WIDE && !edge) bad[2 * (n % LEAD)] = bad[2 * (n % LEAD) + 1] = 0;
                }
            }
            const int tile = id * p.Hkv + g.h;
            if constexpr (WIDE) {
                const uint32_t bar = isk ? k_raw(n % NSG) : v_raw(n % NSG);
                if (lane == 0) dev::mbar_arrive_expect_tx(bar, (uint32_t)(__popc(got) * L::TILE));
                __syncwarp();
                if (good) dev::bulk_g2s(base + (isk ? L::SK : L::SV) + (n % NSG) * L::RAW + lane * L::TILE,
                                        (isk ? p.key_cache : p.value_cache) + (size_t)tile * L::TILE, L::TILE, bar);
            } else {
                // (V that needs looking at lands on v_raw, and warp 17 passes it on; it passes every tile, so that it is
                // never a ring behind)
                const int s = n % NS;
                const uint32_t bar = isk ? k_full(s) : edge ? v_raw(s) : v_full(s);
                if (lane == 0) {
                    dev::mbar_arrive_expect_tx(bar, (uint32_t)(__popc(got) * L::TILE));
                    if (!isk) dev::mbar_arrive(edge ? v_full(s) : v_raw(s));
                }
                __syncwarp();
                if (good) {
                    const uint32_t dst = base + (isk ? L::K : L::V) + s * L::KSTAGE + lane * (BS * 128);
                    for (int hf = 0; hf < H; ++hf) tc::tma_load_3d(dst + hf * L::KHALF, isk ? &kmap : &vmap, hf * 64, 0, tile, bar);
                }
            }
            ++n;
            ++r;
            if (r < my.last) {
                if (++t == g.t1) {
                    g = walk.at(p, r);
                    t = chunk = g.t0;
                    cur = fetch(t);
                    nxt = fetch(t + 8);
                } else if (t - chunk == 8) {
                    chunk = t;
                    cur = nxt;
                    nxt = fetch(t + 8);
                }
            }
        };
        bool ok = true;
        int J = 0;
        if constexpr (WIDE) {
            for (; J < nt; ++J) {
                while (ok && n < nt && n < J + NSG) {
                    if (n >= NSG) ok = __all_sync(dev::FULL, dev::mbar_wait_bounded(raw_free(isk, n % NSG), (uint32_t)(((n - NSG) / NSG) & 1)));
                    if (ok) issue();
                }
                ok = ok && __all_sync(dev::FULL, dev::mbar_wait_bounded(isk ? k_raw(J % NSG) : v_raw(J % NSG), (uint32_t)((J / NSG) & 1)));
                if (ok && J >= NS) ok = __all_sync(dev::FULL, dev::mbar_wait_bounded(isk ? k_free(J % NS) : v_free(J % NS), (uint32_t)(((J - NS) / NS) & 1)));
                if (!ok) break;
                const uint8_t *src = sm + (isk ? L::SK : L::SV) + (J % NSG) * L::RAW;
                uint8_t *dst = sm + (isk ? L::K : L::V) + (J % NS) * L::KSTAGE;
                if (isk) {
                    const int got = got_k[J % LEAD];
                    for (int k = 0; k < 2; ++k)
                        if ((got >> k) & 1) widen<D, KIND, L::KHALF>(src + k * L::TILE, dst + k * (BS * 128), true, lane);
                } else {
                    const unsigned long long l = there[J % LEAD], z = sure[J % LEAD];
                    uint32_t b = 0;
                    for (int k = 0; k < 2; ++k) {
                        if ((l >> (16 * k)) & 0xffffu) widen<D, KIND, L::KHALF>(src + k * L::TILE, dst + k * (BS * 128), false, lane);
                        __syncwarp();
                        b |= clean_v<D, KIND, L::KHALF>(dst + k * (BS * 128), (uint32_t)(l >> (16 * k)) & 0xffffu, (uint32_t)(z >> (16 * k)) & 0xffffu, lane) << (16 * k);
                    }
                    if (lane == 0) bad[2 * (J % LEAD)] = b;
                }
                dev::fence_proxy_async_smem();                     // expanded rows -> tensor core
                __syncwarp();
                if (lane == 0) dev::mbar_arrive(isk ? k_full(J % NS) : v_full(J % NS));
            }
            // no copy may land after the CTA has left
            for (int x = J; x < n; ++x) (void)dev::mbar_wait_bounded(isk ? k_raw(x % NSG) : v_raw(x % NSG), (uint32_t)((x / NSG) & 1));
        } else {
            for (; J < nt; ++J) {
                if (J >= NS) ok = __all_sync(dev::FULL, dev::mbar_wait_bounded(isk ? k_free(J % NS) : v_free(J % NS), (uint32_t)(((J - NS) / NS) & 1)));
                if (!ok) break;
                issue();
            }
            for (int x = max(0, n - NS); x < n; ++x) {
                (void)dev::mbar_wait_bounded(isk ? k_full(x % NS) : v_raw(x % NS), (uint32_t)((x / NS) & 1));
                if (!isk) (void)dev::mbar_wait_bounded(v_full(x % NS), (uint32_t)((x / NS) & 1));
            }
        }
        if (!ok && lane == 0) dev::flag_error(p.err, PKV_DEVERR_TIMEOUT);
    } else if (warp == 13 || warp == 17) {
        // ============ the other half of K's (13) and V's (17) expansion; bf16: V that needs looking at (17)
        const bool isk = warp == 13;
        bool ok = true;
        for (int J = 0; J < nt && (WIDE || !isk); ++J) {
            if constexpr (WIDE) {
                ok = __all_sync(dev::FULL, dev::mbar_wait_bounded(isk ? k_raw(J % NSG) : v_raw(J % NSG), (uint32_t)((J / NSG) & 1)));
                if (ok && J >= NS) ok = __all_sync(dev::FULL, dev::mbar_wait_bounded(isk ? k_free(J % NS) : v_free(J % NS), (uint32_t)(((J - NS) / NS) & 1)));
                if (!ok) break;
                const uint8_t *src = sm + (isk ? L::SK : L::SV) + (J % NSG) * L::RAW;
                uint8_t *dst = sm + (isk ? L::K : L::V) + (J % NS) * L::KSTAGE;
                if (isk) {
                    const int got = got_k[J % LEAD];
                    for (int k = 2; k < TB; ++k)
                        if ((got >> k) & 1) widen<D, KIND, L::KHALF>(src + k * L::TILE, dst + k * (BS * 128), true, lane);
                } else {
                    const unsigned long long l = there[J % LEAD], z = sure[J % LEAD];
                    uint32_t b = 0;
                    for (int k = 2; k < TB; ++k) {
                        if ((l >> (16 * k)) & 0xffffu) widen<D, KIND, L::KHALF>(src + k * L::TILE, dst + k * (BS * 128), false, lane);
                        __syncwarp();
                        b |= clean_v<D, KIND, L::KHALF>(dst + k * (BS * 128), (uint32_t)(l >> (16 * k)) & 0xffffu, (uint32_t)(z >> (16 * k)) & 0xffffu, lane) << (16 * (k - 2));
                    }
                    if (lane == 0) bad[2 * (J % LEAD) + 1] = b;
                }
                dev::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    dev::mbar_arrive(isk ? k_full(J % NS) : v_full(J % NS));
                    dev::mbar_arrive(raw_free(isk, J % NSG));
                }
            } else {
                ok = __all_sync(dev::FULL, dev::mbar_wait_bounded(v_raw(J % NS), (uint32_t)((J / NS) & 1)));
                if (!ok) break;
                const unsigned long long l = there[J % LEAD], z = sure[J % LEAD];
                if (z != ~0ull) {
                    uint8_t *dst = sm + L::V + (J % NS) * L::KSTAGE;
                    unsigned long long b = 0;
                    for (int k = 0; k < TB; ++k)
                        b |= (unsigned long long)clean_v<D, KIND, L::KHALF>(dst + k * (BS * 128), (uint32_t)(l >> (16 * k)) & 0xffffu,
                                                                           (uint32_t)(z >> (16 * k)) & 0xffffu, lane) << (16 * k);
                    if (lane == 0) {
                        bad[2 * (J % LEAD)] = (uint32_t)b;
                        bad[2 * (J % LEAD) + 1] = (uint32_t)(b >> 32);
                    }
                    dev::fence_proxy_async_smem();                 // zeroed rows -> tensor core
                    __syncwarp();
                }
                if (lane == 0) dev::mbar_arrive(v_full(J % NS));
            }
        }
        if (!ok && lane == 0) dev::flag_error(p.err, PKV_DEVERR_TIMEOUT);
    } else if (warp == 14) {
        // ============ Q: eight tokens a copy, once the S before is done with its room; FP8 and INT4: to f16 in place
        Walk walk(p, my);
        int uq = 0;
        bool pending = false;
        bool ok = __all_sync(dev::FULL, !p.test_stall || lane != 0 || dev::mbar_wait_bounded_ns(never, 0, dev::TEST_EXPIRE_NS));
        for (long long r = my.first; ok && r < my.last; ++uq) {
            const Segment g = walk.at(p, r);
            const int i0 = g.m * tokens, copies = (min(tokens, walk.sq.P - i0) + 7) / 8;
            if (uq > 0) ok = __all_sync(dev::FULL, dev::mbar_wait_bounded(q_free, (uint32_t)((uq - 1) & 1)));
            if (!ok) break;
            if (lane == 0) dev::mbar_arrive_expect_tx(q_full, (uint32_t)(copies * H * 64 * p.group * 8 * 2));
            __syncwarp();
            for (int x = lane; x < copies * H; x += 32) {
                const int hf = x % H, c = x / H;
                tc::tma_load_3d(base + hf * L::QHALF + c * (8 * p.group * 128), &qmap, hf * 64, g.h * p.group, walk.sq.row0 + i0 + 8 * c, q_full);
            }
            pending = true;
            if constexpr (WIDE) {
                ok = __all_sync(dev::FULL, dev::mbar_wait_bounded(q_full, (uint32_t)(uq & 1)));
                if (!ok) break;
                pending = false;
                const int rows = copies * 8 * p.group;
                for (int row = lane; row < rows; row += 32) {
                    uint4 *src = reinterpret_cast<uint4 *>(sm + row * 128);
                    uint32_t top = 0;
                    for (int x = 0; x < 8 * H; ++x) {              // (chunks in the row's swizzled order)
                        const uint4 v = src[(x >> 3) * (L::QHALF / 16) + ((x ^ row) & 7)];
                        const uint32_t m2 = __vmaxu2(__vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu), __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu));
                        top = max(top, max(m2 & 0xffffu, m2 >> 16));
                    }
                    const int up = q_exponent(top);
                    const float f = q_factor(up);
                    for (int x = 0; x < 8 * H; ++x) {
                        uint4 *at = src + (x >> 3) * (L::QHALF / 16) + ((x ^ row) & 7);
                        uint4 v = *at;
                        uint32_t *w = reinterpret_cast<uint32_t *>(&v);
#pragma unroll
                        for (int e = 0; e < 4; ++e) w[e] = dev::pack_f16x2(dev::bf16_lo(w[e]) * f, dev::bf16_hi(w[e]) * f);
                        *at = v;
                    }
                    qexp[row] = (int8_t)up;
                }
                dev::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) dev::mbar_arrive(q_ready);
            }
            r += g.t1 - g.t0;
        }
        if (!ok && lane == 0) dev::flag_error(p.err, PKV_DEVERR_TIMEOUT);
        // no copy may land after the CTA has left
        if (pending) (void)dev::mbar_wait_bounded(q_full, (uint32_t)((ok ? uq - 1 : uq) & 1));
    } else if (warp >= 8 && warp < 12) {
        // ============ the products: warps 8, 9 S and 10, 11 P V of q-tiles 0, 1
        if (lane == 0) {
            const bool is_s = warp < 10;
            const int w = warp & 1;
            Walk walk(p, my);
            int J = 0, Jw = 0, uq = 0, uw = 0;                     // tiles and units, and those of this q-tile
            bool ok = true;
            auto wait = [&](uint32_t bar, int par) {
                if (ok && !dev::mbar_wait_bounded(bar, (uint32_t)par & 1u)) ok = false;
                return ok;
            };
            const uint32_t IDS = (WIDE ? tc::idesc_f16(BM, BN, 0) : tc::idesc_bf16(BM, BN, 0)) | (p.score_scale < 0.f ? NEGATE_A : 0u);
            constexpr uint32_t IDO = WIDE ? tc::idesc_f16(BM, D, 1) : tc::idesc_bf16(BM, D, 1);
            const uint64_t dQ = tc::desc_add(tc::smem_desc_sw128(base, 16, 1024), (uint32_t)w * 16384);
            const uint64_t dK = tc::smem_desc_sw128(base + L::K, 16, 1024), dV = tc::smem_desc_sw128(base + L::V, L::KHALF, 1024);
            for (long long r = my.first; ok && r < my.last; ++uq) {
                const Segment g = walk.at(p, r);
                const bool active = min(tokens, walk.sq.P - g.m * tokens) * p.group > BM * w;
                if (is_s && !wait(WIDE ? q_ready : q_full, uq)) break;
                for (int t = g.t0; t < g.t1; ++t, ++J) {
                    const int st = J % NS;
                    if (!wait(is_s ? k_full(st) : v_full(st), J / NS)) break;
                    if (!active) {
                        dev::mbar_arrive(is_s ? k_free(st) : v_free(st));
                        continue;
                    }
                    if (is_s) {
                        // P V of the tile before last has read P, and the softmax its S
                        if (Jw >= 2 && !wait(pv_done(w, Jw), (Jw - 2) >> 1)) break;
                        tc::fence_after_sync();
                        const uint64_t dk = tc::desc_add(dK, (uint32_t)st * L::KSTAGE);
#pragma unroll
                        for (int k = 0; k < 4 * H; ++k) {
                            const uint32_t hf = k >> 2, kk = (k & 3) * 32;
                            tc::mma_bf16(tS(Jw & 1, w), tc::desc_add(dQ, hf * L::QHALF + kk), tc::desc_add(dk, hf * L::KHALF + kk), IDS, k > 0);
                        }
                        tc::commit(s_full(w, Jw));
                        tc::commit(k_free(st));
                        if (t == g.t1 - 1) tc::commit(q_free);
                    } else {
                        if (!wait(p_full(w, Jw), Jw >> 1)) break;
                        if (t == g.t0 && uw > 0 && !wait(o_free(w), uw - 1)) break;      // the unit before has been read
                        tc::fence_after_sync();
                        const uint64_t dv = tc::desc_add(dV, (uint32_t)st * L::KSTAGE);
                        const uint32_t tp = tS(Jw & 1, w);
#pragma unroll
                        for (int k = 0; k < BN / 16; ++k)
                            tc::mma_bf16_ts(tO(w), tp + (uint32_t)(k * 8), tc::desc_add(dv, k * 16 * 128), IDO, t > g.t0 || k > 0);
                        tc::commit(v_free(st));
                        tc::commit(pv_done(w, Jw));
                    }
                    ++Jw;
                }
                if (is_s && !active && ok) dev::mbar_arrive(q_free);
                if (active) ++uw;
                r += g.t1 - g.t0;
            }
            if (!ok) dev::flag_error(p.err, PKV_DEVERR_TIMEOUT);
        }
    }
    }
    tc::fence_before_sync();
    __syncthreads();
    if (warp == 15) {
        tc::fence_after_sync();
        tc::tmem_dealloc(tmem, TMEM_COLS);
    }
}

template <int D, int KIND>
cudaError_t launch(const CUtensorMap &qm, const CUtensorMap &km, const CUtensorMap &vm, const Params &p, int grid, cudaStream_t s)
{
    auto kernel = tree_tcgen05_kernel<D, KIND>;
    // (an attribute of the function on the current device: once for each of them)
    static std::atomic<uint64_t> asked{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 64 || !((asked.load() >> dev) & 1u)) {
        // the registers that the warps share out are those of the launch
        cudaFuncAttributes a;
        e = cudaFuncGetAttributes(&a, kernel);
        if (e == cudaSuccess && a.numRegs < REG_LAUNCH) e = cudaErrorInvalidConfiguration;
        if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Tc<D, KIND>::ALLOC);
        if (e != cudaSuccess) return e;
        if (dev < 64) asked.fetch_or(1ull << dev);
    }
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(TC_THREADS);
    cfg.dynamicSmemBytes = Tc<D, KIND>::ALLOC;
    cfg.stream = s;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, qm, km, vm, p);
}

cudaError_t launch_tcgen05(int D, int kind, const CUtensorMap &qm, const CUtensorMap &km, const CUtensorMap &vm, const Params &p,
                           int grid, cudaStream_t s)
{
    if (kind == BF16) return D == 128 ? launch<128, BF16>(qm, km, vm, p, grid, s) : launch<64, BF16>(qm, km, vm, p, grid, s);
    if (kind == FP8) return D == 128 ? launch<128, FP8>(qm, km, vm, p, grid, s) : launch<64, FP8>(qm, km, vm, p, grid, s);
    return D == 128 ? launch<128, INT4>(qm, km, vm, p, grid, s) : launch<64, INT4>(qm, km, vm, p, grid, s);
}

}  // namespace tree
}  // namespace pkv
