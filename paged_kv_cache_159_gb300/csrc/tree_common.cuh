// tree_common.cuh -- what the kernels of tree_attention.cu and tree_tcgen05.cu share: the call's parameters,
// a sequence's visible blocks and work, the even split of all work over the grid, the masks of 16 keys, and the
// expansion of FP8 and INT4 blocks to f16.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <climits>

#include "int4.cuh"
#include "pkv_internal.h"
#include "tc_device.cuh"

namespace pkv {
namespace tree {

constexpr int BS = 16;                 // tokens per block
constexpr int TB = 4;                  // blocks per tile
constexpr int MOST_BATCH = 4096;
constexpr int MOST_NEW = 256;          // new tokens per sequence
constexpr float LOG2E = 1.4426950408889634f;
enum { BF16 = 0, FP8 = 1, INT4 = 2 };

struct Params {
    const uint16_t *q;
    uint16_t *q16;                         // tcgen05 over FP8 and INT4 pools: q in f16 [batch][max_q][Hq][D], and its
    int8_t *q_up;                          // rows' exponents [batch][max_q][Hq]
    const uint8_t *key_cache, *value_cache;
    const int32_t *tables, *lens, *cu;     // cu null: one row per sequence
    const unsigned long long *mask;        // [total_q][words], or null
    uint16_t *out;
    float *part_o, *part_ml;               // [streams][2][D / 4][rows_unit][4], [streams][2][rows_unit][2]
    int32_t *meta;                         // [streams][META]: the cut unit that begins in a stream
    uint32_t *err;
    int B, MB, Hq, Hkv, group, num_blocks, total_q, max_q, words, window, sinks, rows_unit, unit_cost, test_stall;
    float score_scale, out_scale;
};

constexpr int META = 8;                    // rows (0: none), last stream, first slot, first row of q, KV head, row tile

// A sequence: its lengths, its visible blocks (list entry v is block v < sb ? v : v - sb + b1) and its tasks.
struct Seq {
    int L, P, C, row0;
    int sb, b1, nvb;               // blocks of the sinks, first block of the window, entries of the list
    int nt, rt;                    // tiles and row tiles of a unit (0: nothing to do)
    int bad;                       // 1: flagged, its rows are zeros; 2: flagged, it has no rows to write
};

__device__ __forceinline__ Seq seq_at(const Params &p, int b)
{
    Seq s;
    s.L = __ldcg(p.lens + b);
    s.row0 = b;
    int end = b + 1;
    if (p.cu) {
        s.row0 = __ldcg(p.cu + b);
        end = __ldcg(p.cu + b + 1);
    }
    s.nt = s.rt = s.bad = s.sb = s.b1 = s.nvb = 0;
    s.P = s.C = 0;
    if (s.row0 < 0 || end < s.row0 || end > p.total_q) {
        s.bad = 2;
        return s;
    }
    s.P = end - s.row0;
    if (s.P == 0) return s;
    if (s.P > p.max_q || s.L < s.P || s.L > p.MB * BS) {
        s.bad = 1;
        return s;
    }
    s.C = s.L - s.P;
    const int blocks = (s.L + BS - 1) / BS;
    if (p.window) {
        // a tree's row without a bit stands at C - 1
        const int lo = max(0, s.C - p.window + (p.mask ? 0 : 1));
        s.sb = min(blocks, (p.sinks + BS - 1) / BS);
        s.b1 = max(lo / BS, s.sb);
    }
    s.nvb = s.sb + max(0, blocks - s.b1);
    s.nt = (s.nvb + TB - 1) / TB;
    s.rt = (s.P * p.group + p.rows_unit - 1) / p.rows_unit;
    return s;
}

// The work is laid out unit after unit, a unit's unit_cost (what it costs besides its tiles, in tiles: its rows, its
// edges, its output) and then its tiles; sequence after sequence, KV head after KV head, row tile after row tile.  (The
// host refuses shapes whose places could pass 31 bits.)
__device__ __forceinline__ int units_of(const Params &p, const Seq &s) { return s.rt * p.Hkv; }
__device__ __forceinline__ int places_of(const Params &p, const Seq &s) { return units_of(p, s) * (s.nt + p.unit_cost); }

// floor(W c / G), the even split of W places over G streams, in 32 bits: a 64-bit division is some hundred instructions.
__device__ __forceinline__ int share(int W, int G, int c)
{
    const int q = W / G;
    return q * c + (W - q * G) * c / G;
}


// ---- the split of the work
// Share of one stream of the grid: places first .. last - 1 of W, which hold `tiles` tiles; the first of them is in
// sequence b, whose places begin at U0.
struct Share {
    int first, last, W, U0, tiles, b, streams;
};
template <int NT>
struct ShareScratch {
    long long wsum[NT / 32];
    int U0, b, tiles[2];           // tiles before the share's first and last place
};

// By the whole block: a thread sums some sequences, the block scans (places in the upper half, tiles in the lower).
// Zeroes the rows of invalid sequences.
template <int NT, int D>
__device__ __forceinline__ Share share_of(const Params &p, ShareScratch<NT> &x)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (p.B + NT - 1) / NT, b0 = min(p.B, tid * per), b1 = min(p.B, b0 + per);
    long long run = 0;
    int bad = 0;
#pragma unroll 1
    for (int b = b0; b < b1; ++b) {
        const Seq s = seq_at(p, b);
        bad |= s.bad;
        if (s.rt) run += ((long long)places_of(p, s) << 32) + units_of(p, s) * s.nt;
    }
    long long incl = run;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long v = __shfl_up_sync(dev::FULL, incl, o);
        if (lane >= o) incl += v;
    }
    if (lane == 31) x.wsum[warp] = incl;
    const int any_bad = __syncthreads_or(bad);
    long long before = incl - run, all = 0;
#pragma unroll 1
    for (int w = 0; w < NT / 32; ++w) {
        if (w < warp) before += x.wsum[w];
        all += x.wsum[w];
    }
    Share h;
    h.W = (int)(all >> 32);
    h.streams = min((int)gridDim.x, max((int)all, 1));
    h.first = (int)blockIdx.x < h.streams ? share(h.W, h.streams, blockIdx.x) : h.W;
    h.last = (int)blockIdx.x < h.streams ? share(h.W, h.streams, blockIdx.x + 1) : h.W;
    int at = (int)(before >> 32), tiles = (int)before;
    if (h.first < at + (int)(run >> 32) && h.last > at) {
        // one of the two may fall into this thread's sequences
#pragma unroll 1
        for (int b = b0; b < b1; ++b) {
            const Seq s = seq_at(p, b);
            if (!s.rt) continue;
            const int n = places_of(p, s), len = s.nt + p.unit_cost;
            auto tiles_to = [&](int place) {
                const int u = (place - at) / len;
                return tiles + u * s.nt + max(0, place - at - u * len - p.unit_cost);
            };
            if (h.first >= at && h.first < at + n) {
                x.b = b;
                x.U0 = at;
                x.tiles[0] = tiles_to(h.first);
            }
            if (h.last > at && h.last <= at + n) x.tiles[1] = tiles_to(h.last);
            at += n;
            tiles += units_of(p, s) * s.nt;
        }
    }
    __syncthreads();
    if (any_bad) {
        if (tid == 0 && blockIdx.x == 0) dev::flag_error(p.err, PKV_DEVERR_SEQ_LEN);
#pragma unroll 1
        for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
            const Seq s = seq_at(p, b);
            uint4 *dst = reinterpret_cast<uint4 *>(p.out + (size_t)s.row0 * p.Hq * D);
            if (s.bad == 1)
#pragma unroll 1
                for (size_t e = tid; e < (size_t)s.P * p.Hq * (D / 8); e += NT) dst[e] = make_uint4(0u, 0u, 0u, 0u);
        }
    }
    h.tiles = h.b = h.U0 = 0;
    if (h.first < h.last) {
        h.b = x.b;
        h.U0 = x.U0;
        h.tiles = x.tiles[1] - x.tiles[0];
    }
    if (h.tiles == 0 && tid < META) p.meta[(size_t)blockIdx.x * META + tid] = 0;
    return h;
}

// The segments of a share: tiles t0 .. t1 - 1 of one unit (KV head h, row tile m of sequence b), one after another.
// (A share that ends among a unit's cost has no tile of it: its reader counts tiles.)  Sequences without rows are
// stepped over one at a time, each a trip to L2: 64 sequences of 8 drafts behind 504 positions (32 / 8 heads of 128, bf16)
// take 39 us in a batch of 64 slots, 45 in one of 1024 and 87 in one of 4096.
struct Segment { int h, m, t0, t1; };
struct Walk {
    Seq sq;
    int b, U0, place, last, unit0;             // unit0: the current unit's first place
    __device__ __forceinline__ Walk(const Params &p, const Share &s) : sq(seq_at(p, s.b)), b(s.b), U0(s.U0), place(s.first), last(s.last), unit0(0) {}
    __device__ __forceinline__ Segment next(const Params &p)
    {
#pragma unroll 1
        while (b + 1 < p.B && (!sq.rt || place >= U0 + places_of(p, sq))) {
            if (sq.rt) U0 += places_of(p, sq);
            sq = seq_at(p, ++b);
        }
        const int len = max(sq.nt + p.unit_cost, 1), unit = (place - U0) / len;
        unit0 = U0 + unit * len;
        Segment g;
        g.t0 = max(0, place - unit0 - p.unit_cost);
        g.t1 = max(g.t0 + 1, min(sq.nt, last - unit0 - p.unit_cost));
        g.h = unit / max(sq.rt, 1);
        g.m = unit - g.h * sq.rt;
        place = unit0 + p.unit_cost + g.t1;
        return g;
    }
    // The logical block of entry v of the list.
    __device__ __forceinline__ int block(int v) const { return v < sq.sb ? v : v - sq.sb + sq.b1; }
};

// The stream that holds place r of W: a guess, off by one at most, put right.
__device__ __forceinline__ int stream_of(int r, int W, int streams)
{
    int c = min(streams - 1, (int)((float)(r + 1) * (float)streams / (float)W));
#pragma unroll 1
    while (c > 0 && share(W, streams, c) > r) --c;
#pragma unroll 1
    while (c + 1 < streams && share(W, streams, c + 1) <= r) ++c;
    return c;
}

// ---- masks
__device__ __forceinline__ uint32_t ones(int c) { return (1u << min(max(c, 0), BS)) - 1u; }

// A row's place: chain, the token's position; tree, C + (bits set) - 1.
__device__ __forceinline__ int place_of(const Params &p, const Seq &s, int token)
{
    if (!p.mask) return s.C + token;
    const unsigned long long *bits = p.mask + (size_t)(s.row0 + token) * p.words;
    int c = 0;
#pragma unroll 1
    for (int w = 0; w < p.words; ++w) {
        const int left = s.P - 64 * w;
        if (left > 0) c += __popcll(__ldcg(bits + w) & (left >= 64 ? ~0ull : (1ull << left) - 1));
    }
    return s.C + c - 1;
}

// The first word of a row's mask (0 for a chain), loaded ahead of its use.
__device__ __forceinline__ unsigned long long first_word(const Params &p, const Seq &s, int token)
{
    return p.mask ? __ldcg(p.mask + (size_t)(s.row0 + token) * p.words) : 0ull;
}

// Which of the 16 positions from p0 on a row sees, `valid` those that are there; w0: its mask's first word.
__device__ __forceinline__ uint32_t seen16(const Params &p, const Seq &s, int token, int place, unsigned long long w0, int p0, uint32_t valid)
{
    uint32_t c = valid & ones((p.mask ? s.C : s.C + token + 1) - p0), d = 0;
    if (p.mask && p0 + BS > s.C) {
        const int off = p0 - s.C;                              // bit of the first position
        unsigned long long w;
        if (off < 0) {
            w = w0 << -off;
        } else if (off < 64 && p.words == 1) {
            w = w0 >> off;
        } else {
            const unsigned long long *bits = p.mask + (size_t)(s.row0 + token) * p.words;
            const int i = off >> 6, sh = off & 63;
            w = i < p.words ? __ldcg(bits + i) >> sh : 0ull;
            if (sh && i + 1 < p.words) w |= __ldcg(bits + i + 1) << (64 - sh);
        }
        d = (uint32_t)w & valid & ~ones(s.C - p0);
    }
    if (p.window) c &= ~ones(place - p.window + 1 - p0) | ones(p.sinks - p0);
    return c | d;
}

// The same for the 64 consecutive positions from p0 on.
__device__ __forceinline__ unsigned long long ones64(int c) { return c <= 0 ? 0ull : c >= 64 ? ~0ull : (1ull << c) - 1; }
__device__ __forceinline__ unsigned long long seen64(const Params &p, const Seq &s, int token, int place, unsigned long long w0, int p0,
                                                     unsigned long long valid)
{
    unsigned long long c = valid & ones64((p.mask ? s.C : s.C + token + 1) - p0), d = 0;
    if (p.mask && p0 + 64 > s.C) {
        const int off = p0 - s.C, sh = off & 63;
        if (off < 0) {
            d = w0 << -off;                                        // (off > -64)
        } else if (p.words == 1) {
            d = off < 64 ? w0 >> off : 0ull;
        } else {
            const unsigned long long *bits = p.mask + (size_t)(s.row0 + token) * p.words;
            const int i = off >> 6;
            d = i < p.words ? __ldcg(bits + i) >> sh : 0ull;
            if (sh && i + 1 < p.words) d |= __ldcg(bits + i + 1) << (64 - sh);
        }
        d &= valid & ~ones64(s.C - p0);
    }
    if (p.window) c &= ~ones64(place - p.window + 1 - p0) | ones64(p.sinks - p0);
    return c | d;
}

// Positions up to which (all_to), and from which on or among the sinks (all_from), every row of tokens i0 .. i1
// sees the cache.
__device__ __forceinline__ int all_to(const Params &p, const Seq &s, int i0) { return p.mask ? s.C : s.C + i0 + 1; }
__device__ __forceinline__ int all_from(const Params &p, const Seq &s, int i1)
{
    return p.window ? s.C + (p.mask ? s.P - 1 : i1) - p.window + 1 : INT_MIN;
}

// q to f16 by a power of two per row that brings its largest element (magnitude bits `top`) into [2^14, 2^15): exact
// for elements of 2^-24 of it and more.  The exponent; NO_SCALE for a row with an infinity or NaN, which becomes NaN
// as a whole: its scores are NaN, and the select of the masked ones takes NaN away where the row sees nothing (a NaN
// in the row's scale would come back behind that select, where the scale is applied after it).
constexpr int NO_SCALE = -128;
__device__ __forceinline__ int q_exponent(uint32_t top)
{
    const int ex = (int)(top >> 7);
    return ex == 255 ? NO_SCALE : top == 0 ? 0 : min(126, 141 - max(ex, 1));
}
__device__ __forceinline__ float q_factor(int up) { return __uint_as_float(up == NO_SCALE ? 0x7fffffffu : (uint32_t)(127 + up) << 23); }
// The score scale of such a row.
__device__ __forceinline__ float row_scale(float sc, int up) { return up == NO_SCALE ? sc : sc * __uint_as_float((uint32_t)(127 - up) << 23); }

// Expand one block (16 tokens) of K or V to f16 in the swizzled layout, by a warp; half: bytes from a row's first 64
// columns to its others.
template <int D, int KIND>
__device__ __forceinline__ void widen(const uint8_t *src, uint8_t *dst, int half, bool isk, int lane)
{
    auto at = [&](int row, int chunk) {
        return reinterpret_cast<uint4 *>(dst + (chunk >> 3) * half + row * 128 + (((chunk & 7) ^ (row & 7)) << 4));
    };
    if constexpr (KIND == FP8) {
        constexpr int PR = D / 16;                                 // 16-byte pieces of a row
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
            const int e = i * 32 + lane, row = e / PR, cc = e % PR;
            const uint4 x = *reinterpret_cast<const uint4 *>(src + e * 16);
            const uint32_t w[4] = {x.x, x.y, x.z, x.w};
            uint32_t h[8];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                h[2 * k] = dev::e4m3x2_to_f16x2((uint16_t)w[k]);
                h[2 * k + 1] = dev::e4m3x2_to_f16x2((uint16_t)(w[k] >> 16));
            }
            // (lanes of the upper 64 columns store their second half first: no bank conflict)
            const bool odd = cc >= 4;
            const uint4 lo = make_uint4(h[0], h[1], h[2], h[3]), hi = make_uint4(h[4], h[5], h[6], h[7]);
            *at(row, 2 * cc + (odd ? 1 : 0)) = odd ? hi : lo;
            *at(row, 2 * cc + (odd ? 0 : 1)) = odd ? lo : hi;
        }
    } else if constexpr (KIND == INT4) {
        constexpr int NG = D / 32;
        const int c = lane & 3;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const int r = 8 * x + (lane >> 2);
            const int t = isk ? (r & 8) | ((r >> 1) & 3) | ((r & 1) << 2) : r, oc = !isk && D == 128 ? c ^ (r & 2) : c;
            uint32_t w[NG], sb = 0, vs[NG];
            const uint8_t *row = src + r * (D / 2) + c * (4 * NG);
            if constexpr (NG == 4) {
                const uint4 v = *reinterpret_cast<const uint4 *>(row);
                w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
            } else {
                const uint2 v = *reinterpret_cast<const uint2 *>(row);
                w[0] = v.x; w[1] = v.y;
            }
            if (isk) {
                if constexpr (NG == 4) sb = *reinterpret_cast<const uint32_t *>(src + 8 * D + r * NG);
                else sb = *reinterpret_cast<const uint16_t *>(src + 8 * D + r * NG);
            } else {
#pragma unroll
                for (int j = 0; j < NG; ++j) vs[j] = *reinterpret_cast<const uint32_t *>(src + 8 * D + (r & 3) * (4 * NG) + 4 * j);
            }
#pragma unroll
            for (int j = 0; j < NG; ++j) {
                const uint32_t codes = isk ? w[j] : __byte_perm(w[j >> 1], w[NG / 2 + (j >> 1)], (j & 1) ? 0x7632u : 0x5410u);
                const uint32_t scale = isk ? (sb >> (8 * j)) & 0xffu : (vs[j] >> (8 * (r >> 2))) & 0xffu;
                *at(t, 4 * j + oc) = int4::expand_octet<__half2>(codes, scale);
            }
        }
    }
}

// A bounded wait in few instructions: warps of different code share the instruction cache, and what the unrolled
// waits of pkv_device.cuh, 64-bit divisions and the like added to the tcgen05 kernel (100 KB of code, a hit rate of 82 %)
// made a tile's softmax take 1.2 to 2.9 us instead of 0.5.
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity)
{
    if (__builtin_expect(dev::mbar_try_wait(bar, parity), 1)) return true;
    const unsigned long long t0 = dev::globaltimer();
#pragma unroll 1
    while (!dev::mbar_try_wait_suspend(bar, parity, dev::WAIT_SUSPEND_NS))
        if (dev::globaltimer() - t0 > dev::WAIT_NS) return false;
    return true;
}

// ---- host
// Launch the tcgen05 kernel (tree_tcgen05.cu): maps of q and, for bf16 pools, of K and V.
cudaError_t launch_tcgen05(int D, int kind, const CUtensorMap &qm, const CUtensorMap &km, const CUtensorMap &vm, const Params &p,
                           int grid, cudaStream_t s);
// Its rows per unit: tokens, a multiple of eight, times the group's heads.
inline int tcgen05_tokens(int group) { return 256 / group / 8 * 8; }

}  // namespace tree
}  // namespace pkv
