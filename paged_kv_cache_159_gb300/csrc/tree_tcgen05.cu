// tree_tcgen05.cu -- the attention of tree_attention.cu for many rows per KV head, on the tcgen05 tensor cores.
//
// Above 32 rows (tokens times the group's heads) the products and the softmax bind, not the reading of K and V: 16 trees
// of 61 tokens of 64 / 8 heads (488 rows a KV head, FP8) took 1080 us on mma.sync.  A unit is (sequence, KV head, 256 rows)
// as two q-tiles of 128, of which the second rests where a unit has no more than 128 rows; a tile is 64 keys of
// the unit's visible blocks.  The work is divided as in tree_attention.cu: every CTA of a one-wave grid takes an
// even share of all tiles, and partial states of cut units are merged by the same second launch.
//
// Twenty warps, one CTA per SM.  Warps 0-3 and 4-7: softmax of q-tiles 0 and 1, a row per thread; 8, 9 issue S = Q K^T
// of the q-tiles (M 128, N 64) and 10, 11 O += P V (M 128, N D, P from tensor memory); 12, 13 (16) bring K, 18, 19 (17) V, 14 Q;
// 15 goes through the CTA's share ahead of them all and writes down each tile (its blocks, positions, masks and unit) in
// a ring that the others read.  (Each of them going through it alone cost the two loaders, with a microsecond a
// tile, twice what the copies take, and the others a microsecond or more a unit.)  S is double-buffered in tensor memory and P
// overwrites it, O stays there; S of tile J waits for P V of tile J - 2 of its q-tile.  One issuing thread per product and
// q-tile, since a thread issues a tcgen05.mma only every 36 to 60 ns.
//   * bf16 pools: tensor copies with 128-byte swizzle straight into the operand rings.
//   * FP8 and INT4 pools: bulk copies of the blocks as stored into staging rings, expanded (exactly) to f16 operand
//     tiles by three warps for K and three for V, which take half tiles in turn; P in f16 times 2^8.  q goes to f16 by a power of two per row in a launch of its
//     own (in the kernel, a warp took 8 us a unit for it).  Six
//     expanding warps beside eight of softmax need registers moved between warpgroups (setmaxnreg: 96 a thread at
//     launch, 144 for softmax, 64 for the others, which is the same sum).
//   * V that must not meet the tensor core is zeroed in its operand tile before P V, by the warps that bring V:
//     what is not there, and, of positions that some rows of the unit do not see, those that are not finite
//     (0 x NaN is NaN); the softmax threads of rows that do see such a position add its product themselves.
// What bounds it (head_dim 128, in a graph, all launches):
//   * those 16 trees behind up to 8192 positions: 221 us, 738 TFLOP/s.  A CTA has 136 tiles of 64 keys and both q-tiles at
//     1.28 us (the slope of the time over contexts of 4096 to 16384): 174 us.  Besides, 2.7 pieces of units a CTA at 6 to 7 us
//     (edge tiles, epilogue, refill), and q to f16 and the merge, 14 and 13 us by themselves.  Of a tile, 0.95 us are the
//     softmax's, the rest is S and P handed over; the expansion of E4M3 does not set the pace, since over a bf16 pool a tile
//     takes 1.42 us and the call, without a launch for q, 203.  The tensor pipe is busy 41 % of the time, the issue slots
//     53 %.  The softmax threads also store P to local memory, a tile's 32 words a thread, for the rare path that picks
//     one of them by its number.
//   * 37 trees of up to 25 tokens behind up to 4096, 28 / 4 heads, INT4: 72 us.  A CTA has 30 tiles
//     of mostly one q-tile (91 rows a unit on average), at 1.2 us the latency of its chain (below), and two units' own cost.
//   * bf16, one q-tile: 0.85 to 1.2 us a tile, the latency of S, softmax, P V in turn over two S buffers.
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
constexpr int LEAD = 16, STEP = 32 / TB;       // tiles that warp 15 writes down ahead, and at a time

// A tile as warp 15 writes it down.
struct TileInfo {
    unsigned long long there, sure;            // bit per key: it is there; every row of the unit sees it
    int tile[TB], pos[TB];                     // blocks: (block id * Hkv + head), -1 where there is none; first position
    uint32_t bad[2];                           // bit per key: V kept from the tensor core (written by the V warps)
    int b, L, P, row0;                         // the sequence
    int hm, left, unit, t_place;               // KV head and (from bit 24) row tile; tiles left in the segment, in the unit;
                                               // the unit's place, bit 31: the segment begins after its first tile
    __device__ __forceinline__ int h() const { return hm & 0xffffff; }
    __device__ __forceinline__ int m() const { return hm >> 24; }
};
static_assert(sizeof(TileInfo) == 88, "room");

template <int D, int KIND>
struct Tc {
    static constexpr int H = D / 64;
    static constexpr int NS = KIND == BF16 ? (D == 128 ? 5 : 8) : (D == 128 ? 3 : 4);       // operand tiles of K and V
    static constexpr int TILE = KIND == BF16 ? BS * D * 2 : KIND == FP8 ? BS * D : int4::tile_bytes(D);
    static constexpr int RAW = TB * TILE;
    static constexpr int NSG = KIND == BF16 ? 0 : KIND == FP8 && D == 128 ? 3 : 6;     // staging tiles
    static constexpr int QHALF = 2 * BM * 128, KHALF = BN * 128, KSTAGE = H * KHALF;
    // K: [64 columns][64 keys], a copy per block and half row; V: block by block [64 columns][16 keys], as P V takes it,
    // a copy per block
    static constexpr int VHALF = BS * 128, VBLOCK = H * VHALF;
    static constexpr int K = H * QHALF, V = K + NS * KSTAGE, SK = V + NS * KSTAGE, SV = SK + NSG * RAW;
    static constexpr int INFO = SV + NSG * RAW;                    // TileInfo [LEAD]
    static constexpr int BAR = INFO + LEAD * (int)sizeof(TileInfo);
    static constexpr int NRAW = KIND == BF16 ? 1 : NSG;            // landings that a V (K) warp looks at, each its own
    static constexpr int BARS = 2 + 4 * NS + 4 + 4 + 4 + 2 + 1 + 2 * LEAD + (KIND == BF16 ? 2 : 4) * NRAW;
    static constexpr int ALLOC = BAR + BARS * 8 + 8 + 1024;
    static_assert(NSG % 3 == 0, "a staging place is one warp's");
    static_assert(ALLOC <= 227 * 1024 && NS < LEAD && NSG < LEAD && RAW % 128 == 0 && BAR % 8 == 0, "shared memory");
};

// 8 consecutive columns of this thread's lane (see tmem_ld32).
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr));
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8])
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]), "r"(r[1]),
                 "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}

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
    uint32_t lo = 0, hi = 0;                                       // the largest exponents
#pragma unroll 2
    for (int c = 0; c < CHUNKS; ++c) {
        const uint4 v = at[c];
        const uint32_t w[4] = {v.x & (EXP | EXP << 16), v.y & (EXP | EXP << 16), v.z & (EXP | EXP << 16), v.w & (EXP | EXP << 16)};
        const uint32_t m = __vmaxu2(__vmaxu2(w[0], w[1]), __vmaxu2(w[2], w[3]));
        lo = max(lo, m & 0xffffu);
        hi = max(hi, m >> 16);
    }
    bool odd = max(lo, hi) == EXP;
    odd |= __shfl_xor_sync(dev::FULL, (int)odd, 1) != 0;
    const bool is = (there16 >> row) & 1u, keep_out = is && !((sure16 >> row) & 1u) && odd;
    if (!is || keep_out) {
#pragma unroll 1
        for (int c = 0; c < CHUNKS; ++c) at[c] = make_uint4(0u, 0u, 0u, 0u);
    }
    const uint32_t both = __ballot_sync(dev::FULL, keep_out);
    uint32_t rows = 0;
    if (both)
#pragma unroll 1
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
    TileInfo *info = reinterpret_cast<TileInfo *>(sm + L::INFO);
    const uint32_t bars = base + L::BAR;
    const uint32_t q_full = bars, q_free = bars + 8;
    auto k_full = [&](int s) { return bars + 8 * (2 + s); };
    auto v_full = [&](int s) { return bars + 8 * (2 + NS + s); };
    auto k_free = [&](int s) { return bars + 8 * (2 + 2 * NS + s); };
    auto v_free = [&](int s) { return bars + 8 * (2 + 3 * NS + s); };
    auto s_full = [&](int w, int J) { return bars + 8 * (2 + 4 * NS + 2 * w + (J & 1)); };
    auto p_full = [&](int w, int J) { return bars + 8 * (6 + 4 * NS + 2 * w + (J & 1)); };
    auto pv_done = [&](int w, int J) { return bars + 8 * (10 + 4 * NS + 2 * w + (J & 1)); };
    auto o_free = [&](int w) { return bars + 8 * (14 + 4 * NS + w); };
    const uint32_t never = bars + 8 * (16 + 4 * NS);
    auto told = [&](int J) { return bars + 8 * (17 + 4 * NS + J % LEAD); };                // tile J is written down
    auto untold = [&](int J) { return bars + 8 * (17 + 4 * NS + LEAD + J % LEAD); };      // and nobody reads it any more
    auto raw = [&](int x, int i) { return bars + 8 * (17 + 4 * NS + 2 * LEAD + x * L::NRAW + i); };       // landings of loader x
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sm + L::BAR + L::BARS * 8);

    if (tid == 0) {
        dev::mbar_init(q_full, 1);
        dev::mbar_init(q_free, 2);                                 // both S issuers
        for (int s = 0; s < NS; ++s) {
            dev::mbar_init(k_full(s), 2);                          // two warps each
            dev::mbar_init(v_full(s), 2);
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
        for (int J = 0; J < LEAD; ++J) {
            dev::mbar_init(told(J), 1);
            dev::mbar_init(untold(J), 2);                          // both P V issuers
        }
        for (int x = 0; x < (WIDE ? 4 : 2); ++x)
            for (int i = 0; i < L::NRAW; ++i) dev::mbar_init(raw(x, i), 1);
        dev::fence_barrier_init();
    }
    pdl_launch();
    pdl_wait();
    const Share my = share_of<TC_THREADS, D>(p, *reinterpret_cast<ShareScratch<TC_THREADS> *>(sm));      // (Q's room, not yet in use)
    if (my.tiles == 0) return;
    if (warp == 15) tc::tmem_alloc(dev::smem_u32(tmem_slot), TMEM_COLS);
    tc::fence_before_sync();
    dev::fence_proxy_async_smem();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    auto tS = [&](int b, int w) { return tmem + (uint32_t)((2 * b + w) * BN); };
    auto tO = [&](int w) { return tmem + 256u + (uint32_t)(w * D); };
    const int nt = my.tiles, tokens = p.rows_unit / p.group;
    auto wait = [&](uint32_t bar, int phase) { return wait_bar(bar, (uint32_t)phase & 1u); };
    auto wait_all = [&](uint32_t bar, int phase) { return (bool)__all_sync(dev::FULL, wait_bar(bar, (uint32_t)phase & 1u)); };

    // (a warpgroup's registers are moved before its warps part)
    if (warp < 8) {
        more_registers<REG_SOFTMAX>();
        // ============ softmax and output: a row per thread, all keys of a tile, all columns
        const int w = warp >> 2, q4 = warp & 3, rg = w * BM + 32 * q4 + lane;      // row of the unit
        const uint32_t lane_off = (uint32_t)(32 * q4) << 16;
        int Jw = 0;                                                // this q-tile's tiles (two for a unit that it rests in)
        bool ok = true, cut_begins = false;
        int cut[META] = {};
        for (int J = 0; ok && J < nt;) {
            ok = wait_all(told(J), J / LEAD);
            if (!ok) break;
            Seq sq;                                                // (what the masks need of it)
            const TileInfo &u = info[J % LEAD];
            sq.L = u.L;
            sq.P = u.P;
            sq.C = u.L - u.P;
            sq.row0 = u.row0;
            const int b = u.b, h = u.h(), mt = u.m(), left = u.left, unit = u.unit, place0 = u.t_place;
            const int i0 = mt * tokens, i1 = min(sq.P, i0 + tokens) - 1, rows = (i1 + 1 - i0) * p.group;
            const bool whole = left == unit;
            const int slot = J == 0 ? 0 : 1;
            if (place0 >= 0 && !whole) {
                cut_begins = true;
                cut[0] = rows;
                cut[1] = stream_of(place0 + p.unit_cost + unit - 1, my.W, my.streams);
                cut[2] = slot;
                cut[3] = sq.row0;
                cut[4] = h;
                cut[5] = mt;
            }
            if (rows <= BM * w) {                                  // this q-tile rests
                // two tiles of nothing: after the first the unit's slot may be written over, and when the second
                // is done the unit is past, so that of the barriers waited for next none is more than a phase away
                for (int i = 0; i < 2 && ok; ++i, ++Jw) {
                    ok = wait_all(s_full(w, Jw), Jw >> 1);
                    if (ok && lane == 0) dev::mbar_arrive(p_full(w, Jw));
                }
                ok = ok && wait_all(pv_done(w, Jw - 1), (Jw - 1) >> 1);
                J += left;
                continue;
            }
            const bool live = rg < rows;
            const int token = i0 + (live ? rg / p.group : 0), hh = live ? rg - (token - i0) * p.group : 0;
            const int place = p.mask && p.window ? place_of(p, sq, token) : sq.C + token;
            const unsigned long long word = first_word(p, sq, token);
            float sc = fabsf(p.score_scale);
            if (WIDE && live) sc = row_scale(sc, __ldcg(p.q_up + ((size_t)b * p.max_q + token) * p.Hq + h * p.group + hh));
            sc = fmaxf(sc, 1e-37f);                                // (masked scores stay -infinity)
            float m = -INFINITY, l = 0.f;
            for (const int end = J + left; J < end; ++J, ++Jw) {
                ok = wait_all(s_full(w, Jw), Jw >> 1);
                if (!ok) break;
                tc::fence_after_sync();
                const volatile TileInfo &ti = info[J % LEAD];
                const bool edge = ti.sure != ~0ull;
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
                if (__builtin_expect(edge, 0)) {
                    const unsigned long long there = ti.there;
                    unsigned long long see = 0;
                    const int p0 = ti.pos[0];
                    if (ti.pos[TB - 1] == p0 + (TB - 1) * BS) {
                        if (live) see = seen64(p, sq, token, place, word, p0, there);
                    } else {
#pragma unroll 1
                        for (int k = 0; live && k < TB; ++k)
                            see |= (unsigned long long)seen16(p, sq, token, place, word, ti.pos[k], (uint32_t)(there >> (BS * k)) & 0xffffu) << (BS * k);
                    }
                    const uint32_t lo = (uint32_t)see, hi = (uint32_t)(see >> 32);
#pragma unroll
                    for (int c = 0; c < 32; ++c) {
                        if (!((lo >> c) & 1u)) x[c] = -INFINITY;
                        if (!((hi >> c) & 1u)) x[32 + c] = -INFINITY;
                    }
                }
                float mx4[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
                for (int c = 4; c < BN; c += 8)
#pragma unroll
                    for (int e = 0; e < 4; ++e) mx4[e] = c + 4 + e < BN ? tc::fmax3(mx4[e], x[c + e], x[c + 4 + e]) : fmaxf(mx4[e], x[c + e]);
                const float top = tc::fmax3(mx4[0], mx4[1], fmaxf(mx4[2], mx4[3]));
                const float d = (top - m) * sc;
                const bool raise = live && (d > TAU || (m == -INFINITY && top > m)), rescale = raise && m != -INFINITY;
                const float f = rescale ? dev::fast_exp2(-d) : 1.f;
                if (raise) m = top;
                // m's product with the scale may join the exponents while its rounding is below 2^-16; else m goes first
                const float nm = m == -INFINITY ? 0.f : -m;
                float ns = nm * sc + SHIFT;
                if (__builtin_expect(__any_sync(dev::FULL, live && fabsf(ns) > 256.f), 0)) {        // (what a row beyond the unit holds decides nothing)
                    const float2 nm2 = make_float2(nm, nm);
#pragma unroll
                    for (int e = 0; e < BN / 2; ++e) {
                        const float2 v = tc::fadd2(make_float2(x[2 * e], x[2 * e + 1]), nm2);
                        x[2 * e] = v.x;
                        x[2 * e + 1] = v.y;
                    }
                    ns = SHIFT;
                }
                uint32_t pw[BN / 2];
                const float2 sc2 = make_float2(sc, sc), ns2 = make_float2(ns, ns);
                float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                for (int e = 0; e < BN / 2; ++e) {
                    const float2 v = tc::ffma2(make_float2(x[2 * e], x[2 * e + 1]), sc2, ns2);
                    const float2 pe = make_float2(dev::fast_exp2(v.x), dev::fast_exp2(v.y));
                    sum[e & 1] = tc::fadd2(sum[e & 1], pe);
                    pw[e] = WIDE ? dev::pack_f16x2(pe.x, pe.y) : dev::pack_bf16x2(pe.x, pe.y);
                }
                const float2 sum2 = tc::fadd2(sum[0], sum[1]);
                l = l * f + (sum2.x + sum2.y);
                tc::tmem_st32(tS(Jw & 1, w) + lane_off, pw);       // over this tile's S, which is read
                if (__builtin_expect(__any_sync(dev::FULL, rescale), 0)) {
                    ok = wait_all(pv_done(w, Jw - 1), (Jw - 1) >> 1);
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
                if (__builtin_expect(edge, 0)) {
                    ok = wait_all(v_full(J % NS), J / NS);
                    if (!ok) break;
                    odd = ti.bad[0] | (unsigned long long)ti.bad[1] << 32;
                }
                int tiles[TB] = {}, ps[TB] = {};                   // (what is read below: the tile may be gone by then)
                if (__builtin_expect(odd != 0, 0)) {
#pragma unroll
                    for (int k = 0; k < TB; ++k) {
                        tiles[k] = ti.tile[k];
                        ps[k] = ti.pos[k];
                    }
                }
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) dev::mbar_arrive(p_full(w, Jw));
                if (__builtin_expect(odd != 0, 0)) {               // their products, where this row sees them
                    {
                        ok = wait_all(pv_done(w, Jw), Jw >> 1);
                        if (!ok) break;
                        tc::fence_after_sync();
                        for (unsigned long long rest = odd; rest; rest &= rest - 1) {
                            const int j = __ffsll((long long)rest) - 1;
                            int at = 0, p0 = 0;
#pragma unroll
                            for (int k = 0; k < TB; ++k)
                                if (k == j / BS) {
                                    at = tiles[k];
                                    p0 = ps[k];
                                }
                            const uint8_t *tile = p.value_cache + (size_t)at * L::TILE;
                            const uint32_t see = live ? seen16(p, sq, token, place, word, p0, ones(sq.L - p0)) : 0u;
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
                            for (int c = 0; c < D; c += 8) {
                                uint32_t v[8];
                                tmem_ld8(tO(w) + lane_off + c, v);
                                tc::tmem_wait_ld();
#pragma unroll
                                for (int e = 0; e < 8; ++e) {
                                    const float y = v_element<D, KIND>(tile, j % BS, c + e);
                                    if (mine) v[e] = __float_as_uint(fmaf(pj, y, __uint_as_float(v[e])));
                                }
                                tmem_st8(tO(w) + lane_off + c, v);
                                tc::tmem_wait_st();
                            }
                        }
                        tc::fence_before_sync();                   // (before the next p_full, or the output below)
                    }
                }
            }
            if (!ok) break;
            ok = wait_all(pv_done(w, Jw - 1), (Jw - 1) >> 1);
            if (!ok) break;
            tc::fence_after_sync();
            const float inv = l == 0.f ? 0.f : p.out_scale / l;
            uint16_t *dst = p.out + ((size_t)(sq.row0 + token) * p.Hq + (size_t)h * p.group + hh) * D;
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
                    // (a warp's lanes are consecutive rows: 512 bytes a store)
                    uint4 *o = reinterpret_cast<uint4 *>(p.part_o) + (((size_t)blockIdx.x * 2 + slot) * (D / 4) + 8 * c) * p.rows_unit + rg;
#pragma unroll
                    for (int e = 0; e < 8; ++e) o[(size_t)e * p.rows_unit] = make_uint4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
                }
                __syncwarp();
            }
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) dev::mbar_arrive(o_free(w));
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
    if (warp == 15) {
        // ============ the tiles of the share, written down for the others, up to eight at a time: a block a lane
        Walk walk(p, my);
        bool ok = true;
        int J = 0;
        while (J < nt) {
            const Segment g = walk.next(p);
            // the table's entry of this lane's block, a step ahead of its use
            auto fetch = [&](int t0) {
                const int v = TB * t0 + lane;
                return v < walk.sq.nvb && v < TB * g.t1 ? __ldcg(p.tables + (size_t)walk.b * p.MB + walk.block(v)) : -2;
            };
            const int i0 = g.m * tokens, i1 = min(walk.sq.P, i0 + tokens) - 1, to = all_to(p, walk.sq, i0), from = all_from(p, walk.sq, i1);
            int next = fetch(g.t0);
            for (int t = g.t0; t < g.t1; t += STEP) {
                const int id = next, n = min(STEP, g.t1 - t), i = lane / TB, k = lane % TB;
                next = fetch(t + STEP);
                ok = __all_sync(dev::FULL, i >= n || J + i < LEAD || wait(untold(J + i), (J + i - LEAD) / LEAD));
                if (!ok) break;
                const bool good = id >= 0 && id < p.num_blocks;
                if (id != -2 && !good) dev::flag_error(p.err, PKV_DEVERR_BLOCK_ID);
                if (i < n) {
                    const int p0 = walk.block(TB * t + lane) * BS;
                    const uint32_t l16 = good ? ones(walk.sq.L - p0) : 0u;
                    uint32_t s16 = l16 & ones(to - p0);
                    if (p.window) s16 &= ~ones(from - p0) | ones(p.sinks - p0);
                    TileInfo &u = info[(J + i) % LEAD];
                    u.tile[k] = good ? id * p.Hkv + g.h : -1;
                    u.pos[k] = p0;
                    reinterpret_cast<uint16_t *>(&u.there)[k] = (uint16_t)l16;
                    reinterpret_cast<uint16_t *>(&u.sure)[k] = (uint16_t)s16;
                    if (k == 0) {
                        u.L = walk.sq.L;
                        u.P = walk.sq.P;
                        u.row0 = walk.sq.row0;
                        u.b = walk.b;
                        u.hm = g.h | g.m << 24;
                        u.left = g.t1 - t - i;
                        u.unit = walk.sq.nt;
                        u.t_place = walk.unit0 | (g.t0 > 0 ? INT_MIN : 0);
                    }
                }
                __syncwarp();
                if (i < n && k == 0) dev::mbar_arrive(told(J + i));
                J += n;
            }
            if (!ok) break;
        }
        if (!ok && lane == 0) dev::flag_error(p.err, PKV_DEVERR_TIMEOUT);
    } else if (warp == 12 || warp == 13 || warp == 18 || warp == 19 || (WIDE && (warp == 16 || warp == 17))) {
        // ============ K (12, 13, 16) and V (18, 19, 17): a job is two blocks of a tile
        const bool isk = warp < 14 || warp == 16;
        bool ok = true;
        // the copies of job (J, half) to dst, landing on bar: lane i < 2 the i-th block's
        auto issue = [&](int J, int half, uint32_t dst, uint32_t bar) {
            const int tile = lane < 2 ? info[J % LEAD].tile[2 * half + lane] : -1;
            const int got = __popc(__ballot_sync(dev::FULL, tile >= 0));
            if (lane == 0) dev::mbar_arrive_expect_tx(bar, (uint32_t)(got * L::TILE));
            __syncwarp();
            if (tile >= 0) {
                if constexpr (WIDE) {
                    dev::bulk_g2s(dst + (2 * half + lane) * L::TILE, (isk ? p.key_cache : p.value_cache) + (size_t)tile * L::TILE, L::TILE, bar);
                } else {
                    if (isk || H == 1) {
                        for (int hf = 0; hf < H; ++hf)
                            tc::tma_load_3d(dst + hf * L::KHALF + (2 * half + lane) * (BS * 128), isk ? &kmap : &vmap, hf * 64, 0, tile, bar);
                    } else {
                        tc::tma_load_4d(dst + (2 * half + lane) * L::VBLOCK, &vmap, 0, 0, 0, tile, bar);
                    }
                }
            }
        };
        auto full = [&](int J) { return isk ? k_full(J % NS) : v_full(J % NS); };
        auto room = [&](int J) { return J < NS || wait_all(isk ? k_free(J % NS) : v_free(J % NS), (J - NS) / NS); };
        // what of a job's V must not meet the tensor core (see clean_v)
        auto look = [&](int J, int half) {
            TileInfo &u = info[J % LEAD];
            uint8_t *dst = sm + L::V + (J % NS) * L::KSTAGE;
            uint32_t b = 0;
#pragma unroll 1
            for (int k = 0; k < 2; ++k)
                b |= clean_v<D, KIND, L::VHALF>(dst + (2 * half + k) * L::VBLOCK, (uint32_t)(u.there >> (BS * (2 * half + k))) & 0xffffu,
                                                (uint32_t)(u.sure >> (BS * (2 * half + k))) & 0xffffu, lane) << (BS * k);
            if (lane == 0) u.bad[half] = b;
        };
        auto needs_look = [&](int J, int half) {
            return !isk && __builtin_expect((uint32_t)(info[J % LEAD].sure >> (32 * half)) != 0xffffffffu, 0);
        };
        if constexpr (WIDE) {
            // three warps take the jobs in turn, each with its own 2 NSG / 3 staging places
            const int which = warp < 16 ? warp - 12 : warp == 16 || warp == 17 ? 2 : warp - 18, jobs = 2 * nt;
            auto raw_of = [&](int q) { return raw((isk ? 2 : 0) + (q & 1), (q >> 1) % NSG); };
            int n = which, q = which;                              // jobs issued, and done with
            for (; q < jobs; q += 3) {
                for (; n < jobs && n < q + 2 * NSG; n += 3) {
                    ok = wait_all(told(n >> 1), (n >> 1) / LEAD);
                    if (!ok) break;                                // (n stays: only what was issued is waited for below)
                    issue(n >> 1, n & 1, base + (isk ? L::SK : L::SV) + ((n >> 1) % NSG) * L::RAW, raw_of(n));
                }
                const int J = q >> 1, half = q & 1;
                ok = ok && wait_all(raw_of(q), J / NSG) && room(J);
                if (!ok) break;
                const uint8_t *src = sm + (isk ? L::SK : L::SV) + (J % NSG) * L::RAW + 2 * half * L::TILE;
                uint8_t *dst = sm + (isk ? L::K : L::V) + (J % NS) * L::KSTAGE + 2 * half * (isk ? BS * 128 : L::VBLOCK);
                // (a block that is not there is expanded as well: whatever it holds is masked, or zeroed below)
#pragma unroll
                for (int k = 0; k < 2; ++k)
                    widen<D, KIND>(src + k * L::TILE, dst + k * (isk ? BS * 128 : L::VBLOCK), isk ? L::KHALF : L::VHALF, isk, lane);
                if (needs_look(J, half)) {
                    __syncwarp();
                    look(J, half);
                } else if (!isk && lane == 0) {
                    info[J % LEAD].bad[half] = 0;
                }
                dev::fence_proxy_async_smem();                     // expanded rows -> tensor core (and read before the next copy)
                __syncwarp();
                if (lane == 0) dev::mbar_arrive(full(J));
            }
            // no copy may land after the CTA has left
            for (; q < n; q += 3) (void)wait(raw_of(q), (q >> 1) / NSG);
        } else {
            const int half = warp & 1;
            int looks = 0, J = 0;
            bool looking = false;                                  // the copy that raw() is for may be under way
            for (; J < nt; ++J) {
                ok = wait_all(told(J), J / LEAD) && room(J);
                if (!ok) break;
                const bool l = needs_look(J, half);
                if (!isk && lane == 0 && !l) info[J % LEAD].bad[half] = 0;
                issue(J, half, base + (isk ? L::K : L::V) + (J % NS) * L::KSTAGE, l ? raw(half, 0) : full(J));
                if (l) {
                    looking = true;
                    ok = wait_all(raw(half, 0), looks);
                    if (!ok) break;
                    looking = false;
                    ++looks;
                    look(J, half);
                    dev::fence_proxy_async_smem();                 // zeroed rows -> tensor core
                    __syncwarp();
                    if (lane == 0) dev::mbar_arrive(full(J));
                }
            }
            if (looking) (void)wait(raw(half, 0), looks);
            for (int i = max(0, J - NS); i < J; ++i) (void)wait(full(i), i / NS);
        }
        if (!ok && lane == 0) dev::flag_error(p.err, PKV_DEVERR_TIMEOUT);
    } else if (warp == 14) {
        // ============ Q: eight tokens a copy, once the S before is done with its room
        int uq = 0;                                                // units whose rows were asked for
        bool ok = true;
        for (int J = 0; J < nt; ++uq) {
            // (in this order: a tile is waited for only once the one before it has been told, so that its barrier is
            // not more than a phase away)
            if (uq > 0) ok = wait_all(q_free, uq - 1);
            ok = ok && wait_all(told(J), J / LEAD);
            // (the failure path's test: the share's last unit does not get its rows, behind units that did)
            if (ok && p.test_stall && J + info[J % LEAD].left >= nt) ok = wait_all(never, 0);
            if (!ok) break;
            const TileInfo &u = info[J % LEAD];
            const int i0 = u.m() * tokens, copies = (min(tokens, u.P - i0) + 7) / 8, h = u.h(), left = u.left;
            const int row0 = WIDE ? u.b * p.max_q : u.row0;        // (q16 has room for max_q tokens of each sequence)
            if (lane == 0) dev::mbar_arrive_expect_tx(q_full, (uint32_t)(copies * H * 64 * p.group * 8 * 2));
            __syncwarp();
            for (int i = lane; i < copies * H; i += 32) {
                const int hf = i % H, c = i / H;
                tc::tma_load_3d(base + hf * L::QHALF + c * (8 * p.group * 128), &qmap, hf * 64, h * p.group, row0 + i0 + 8 * c, q_full);
            }
            J += left;
        }
        if (!ok && lane == 0) dev::flag_error(p.err, PKV_DEVERR_TIMEOUT);
        // no copy may land after the CTA has left: those of the last unit asked for, however the loop ended
        if (uq > 0) (void)wait(q_full, uq - 1);
    } else if (warp < 12 && lane == 0) {
        // ============ the products: warps 8, 9 S and 10, 11 P V of q-tiles 0, 1
        const bool is_s = warp < 10;
        const int w = warp & 1;
        int Jw = 0, uq = 0, uw = 0;                                // this q-tile's tiles; units, and those of this q-tile
        bool ok = true;
        const uint32_t IDS = (WIDE ? tc::idesc_f16(BM, BN, 0) : tc::idesc_bf16(BM, BN, 0)) | (p.score_scale < 0.f ? NEGATE_A : 0u);
        constexpr uint32_t IDO = WIDE ? tc::idesc_f16(BM, D, 1) : tc::idesc_bf16(BM, D, 1);
        const uint64_t dQ = tc::desc_add(tc::smem_desc_sw128(base, 16, 1024), (uint32_t)w * 16384);
        const uint64_t dKV = is_s ? tc::smem_desc_sw128(base + L::K, 16, 1024) : tc::smem_desc_sw128(base + L::V, L::VHALF, 1024);
        // Per tile three waits: the operand tile; S: P V of the tile before last has read P (and the softmax its S), P V:
        // P is there; P V at a unit's start: the unit before has been read
        for (int J = 0; ok && J < nt; ++uq) {
            ok = wait(told(J), J / LEAD) && (!is_s || wait(q_full, uq));
            if (!ok) break;
            const TileInfo &u = info[J % LEAD];
            const int end = J + u.left, J0 = J;
            const bool active = min(tokens, u.P - u.m() * tokens) * p.group > BM * w;
            // a unit that this q-tile rests in: a tile of nothing before it, which its softmax passes on when it has
            // read the unit, and one behind it
            for (int i = active ? 1 : 0; ok && (i == 0 || J < end || i == 2);) {
                const bool nothing = !active && (J == end || i == 0);
                const int st = J % NS;
                if (!nothing) ok = wait(is_s ? k_full(st) : v_full(st), J / NS);
                if (nothing || active) {
                    if (is_s) ok = ok && (Jw < 2 || wait(pv_done(w, Jw), (Jw - 2) >> 1));
                    else ok = ok && wait(p_full(w, Jw), Jw >> 1) && (!active || J > J0 || uw == 0 || wait(o_free(w), uw - 1));
                }
                if (!ok) break;
                if (nothing) {
                    dev::mbar_arrive(is_s ? s_full(w, Jw) : pv_done(w, Jw));
                    ++Jw;
                    if (i == 2) break;
                    i = 1;
                    continue;
                }
                if (!active) {
                    dev::mbar_arrive(is_s ? k_free(st) : v_free(st));
                    if (!is_s) dev::mbar_arrive(untold(J));
                    if (++J == end) i = 2;
                    continue;
                }
                tc::fence_after_sync();
                const uint64_t d = tc::desc_add(dKV, (uint32_t)st * L::KSTAGE);
                const uint32_t ts = tS(Jw & 1, w);
                if (is_s) {
#pragma unroll
                    for (int k = 0; k < 4 * H; ++k) {
                        const uint32_t hf = k >> 2, kk = (k & 3) * 32;
                        tc::mma_bf16(ts, tc::desc_add(dQ, hf * L::QHALF + kk), tc::desc_add(d, hf * L::KHALF + kk), IDS, k > 0);
                    }
                    tc::commit(s_full(w, Jw));
                    tc::commit(k_free(st));
                    if (J == end - 1) tc::commit(q_free);
                } else {
#pragma unroll
                    for (int k = 0; k < BN / 16; ++k)
                        tc::mma_bf16_ts(tO(w), ts + (uint32_t)(k * 8), tc::desc_add(d, (uint32_t)(k * L::VBLOCK)), IDO, J > J0 || k > 0);
                    tc::commit(v_free(st));
                    tc::commit(pv_done(w, Jw));
                    dev::mbar_arrive(untold(J));
                }
                ++Jw;
                ++J;
            }
            if (ok && is_s && !active) dev::mbar_arrive(q_free);
            if (active) ++uw;
        }
        if (!ok) dev::flag_error(p.err, PKV_DEVERR_TIMEOUT);
    }
    }
    tc::fence_before_sync();
    __syncthreads();
    if (warp == 15) {
        tc::fence_after_sync();
        tc::tmem_dealloc(tmem, TMEM_COLS);
    }
}

// q to f16 [batch][max_q][Hq][D] by a power of two per row and head, a warp each (see q_exponent).  Reads and writes q
// once.
constexpr int Q_WARPS = 8;
template <int D>
__global__ void __launch_bounds__(Q_WARPS * 32) tree_q_kernel(const Params p)
{
    pdl_launch();
    pdl_wait();
    const int lane = threadIdx.x & 31, b = blockIdx.y;
    const Seq s = seq_at(p, b);
    if (s.rt == 0) return;
    constexpr int N = D / 64, R = 4;                               // a lane's words of a row; rows in flight
    const int step = gridDim.x * Q_WARPS, end = s.P * p.Hq;
    for (int r0 = blockIdx.x * Q_WARPS + (threadIdx.x >> 5); r0 < end; r0 += R * step) {
        uint32_t w[R][N];
#pragma unroll
        for (int x = 0; x < R; ++x)
#pragma unroll
            for (int i = 0; i < N; ++i)
                w[x][i] = r0 + x * step < end ? __ldcg(reinterpret_cast<const uint32_t *>(p.q + ((size_t)s.row0 * p.Hq + r0 + x * step) * D) + lane + 32 * i) : 0u;
#pragma unroll
        for (int x = 0; x < R; ++x) {
            if (r0 + x * step >= end) break;
            const size_t row = (size_t)b * p.max_q * p.Hq + r0 + x * step;
            uint32_t top = 0;
#pragma unroll
            for (int i = 0; i < N; ++i) top = max(top, max(w[x][i] & 0x7fffu, (w[x][i] >> 16) & 0x7fffu));
            top = __reduce_max_sync(dev::FULL, top);
            const int up = q_exponent(top);
            const float f = q_factor(up);
#pragma unroll
            for (int i = 0; i < N; ++i)
                reinterpret_cast<uint32_t *>(p.q16 + row * D)[lane + 32 * i] = dev::pack_f16x2(dev::bf16_lo(w[x][i]) * f, dev::bf16_hi(w[x][i]) * f);
            if (lane == 0) p.q_up[row] = (int8_t)up;
        }
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
    cfg.stream = s;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    if (KIND != BF16) {
        // (a warp has up to four rows)
        cfg.gridDim = dim3((unsigned)((p.max_q * p.Hq + 4 * Q_WARPS - 1) / (4 * Q_WARPS)), (unsigned)p.B);
        cfg.blockDim = dim3(Q_WARPS * 32);
        e = cudaLaunchKernelEx(&cfg, tree_q_kernel<D>, p);
        if (e != cudaSuccess) return e;
    }
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(TC_THREADS);
    cfg.dynamicSmemBytes = Tc<D, KIND>::ALLOC;
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
