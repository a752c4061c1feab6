// decode_int4.cuh -- single-query attention over an INT4 pool.
//
// With k = scale_kj (n - 8) per group j of 32 columns (the pool's k_scale goes into the score
// scale), and likewise v:
//   S_t   = sum_j scale_tj sum_{d in j} q_d (n_td - 8)
//   O_d   = sum_t (p_t scale_tj(d)) (n_td - 8)
// with tokens (S^T = K Q^T) or columns (O^T = V^T P^T) as the 16 rows of a tensor-core product
// and the group's query heads as its 8 columns, so each code is unpacked once per step whatever
// the group.  Unpacking is most of the work of the integer pipe (half rate), so codes go to
// the f16 tensor cores as they are: a nibble n at the low bits of an f16 is the subnormal n 2^-24,
// one nibble up it is n 2^-20, so one and makes an operand register of two codes (after one shift
// by 8 for the other half of a word).
//   * K: each query head is scaled by a power of two of its own (exact) to a largest magnitude in
//     [2^14, 2^15), and the columns at the upper nibbles by 2^-4 of that, which evens out the two
//     factors: exact for every bf16 element of at least 2^-24 of the head's largest.  Heads are columns
//     of the product, so an infinity or NaN in one stays there.  The -8 of every code is the
//     accumulators' start value, -8 2^-24 sum_{d in j} q_d.
//   * Group j's partial sums are multiplied with scale_tj in fp32 as they join S.
//   * V: a second product with the constant -8 2^-24 (-8 2^-20) takes the offset out step by step,
//     so that the accumulators stay as small as the sums they stand for.
//   * The tensor core cuts a product's terms 25 bits below the largest exponent among them, and counts
//     a subnormal's as 2^-14: a term of a code is cut 2^-15 of a code unit (the lower nibble of a byte; the
//     upper 2^-19), so a group's score is off by at most 2^-9 of its largest |q| in code units, and an
//     output by 2^-9 (2^-13) of a code unit of the largest p scale of every block.
//   * p scale is formed per group in f16: p 2^8 <= 2^15 (the running max is raised past 2^7) and
//     scale 2^-8 (the scale byte moved to f16's fields) <= 1.75; both products round to 11 bits, or
//     to 2^-25 where they are subnormal: a position loses that much of the largest p's 2^8.
//
// Schedule.  A 16-token block of one head is 2 x 17 D / 2 bytes, little work to hand between
// warps, so nothing is: a warp copies its own tiles (cp.async into a ring of its own, two pairs of
// blocks ahead), computes a pair at a time, and writes its result from registers; it waits for no
// other warp, and the CTA meets only to scan seq_lens.  Teams of HG warps, one per KV head, take the
// same blocks at about the same time, since the heads' tiles of a block lie together in memory.  The
// blocks of all (layer, sequence, head group) units are laid end to end and cut evenly over
// the teams of a one-wave grid.  A team that holds a whole unit writes its output; a cut unit
// leaves a partial (max, sum, unnormalised output) per team, and a second launch merges them
// in team order: placement of the blocks changes no bit.  Both launches may start while the one
// before them drains (programmatic dependent launch) and wait for it before they read, by loads that
// are coherent: a non-coherent one takes its data to be the same from the kernel's start on.
//
// What it measured (GB300; us a pass in a graph over three states, 32 / 8 heads, D 128, K/V of 64 x
// 2048 positions, 143.7 MB, and of the ragged batch, 592.9 MB; the measured copy peak gives 21.2
// and 87.3): streaming alone 28.0 and 97.3; the first version, on the other pools' schedule with
// a producer warp and bulk copies of 1088 bytes, 67 and 228; own copies and the merge launch 44 and
// 148; subnormal operands and pairs of blocks, 43.7 and 139; twelve warps, 41.0 and 132; now 39.6 and
// 122.4.  Not kept: E4M3 products for K (58 and 181), loads
// straight to registers (48 and 159: too few bytes in flight), four pairs in the ring (no change),
// V's codes as whole bytes less their upper nibbles (119, but the cut of whole bytes grows with the
// nibble taken out).
// What bounds it: waits of the three warps that a scheduler has.  No pipe is full on average (64 x 2048: issue
// slots 52 % busy, integer pipe 49 %, tensor 33 %), but the warps are all unpacking or all multiplying: per issued
// instruction a warp spends 1.35 waiting for a fixed latency and 0.97 for a pipe, and 0.93 warps are
// ready a clock.  The merge launch comes on top (7.9 us by itself from cold caches).
#pragma once

#include "decode_kernels.cuh"
#include "int4.cuh"

namespace pkv {
namespace decode {

// Warps of a CTA, one CTA per SM, by the registers that a warp's state needs (168 a thread at 12 warps,
// 128 at 16; 16 columns hold twice the state).  At D 128 sixteen warps spill and are slower (43.7 against
// 41.0 us for 64 x 2048, 139 against 132 for the ragged batch).
template <int D, int NH>
constexpr int int4_warps() { return D == 128 ? (NH == 1 ? 12 : 8) : (NH == 1 ? 16 : 12); }
constexpr int I4_NST = 3;                           // pairs of blocks in a warp's ring
constexpr int I4_MERGE_WARPS = 8;

// KV heads of a team: all of them up to 8, else the largest divisor up to 8.
__host__ __device__ constexpr int int4_team(int Hkv)
{
    int h = Hkv < 8 ? Hkv : 8;
    while (Hkv % h) --h;
    return h;
}

template <int D, int NH>
struct Int4Compute {
    static constexpr int TILE = int4::tile_bytes(D);
    static constexpr int NG = D / 32;               // column groups
    static constexpr int ROWB = D / 2;              // bytes of a row's codes
    static constexpr int SCALES = 8 * D;            // byte offset of a tile's scales
    static constexpr uint32_t LO = 0x000F000Fu, HI = 0x00F000F0u;     // nibbles 0 and 1 of each half
    static constexpr float OFF = 8.0f;              // p is held as p 2^8, p = 2^(score - reference)
    static constexpr float TAU = 7.0f;              // raise the reference to the max beyond 2^7

    uint32_t qb[NG][NH][4];       // Q^T fragments of group j: 2 words of each k-step
    float c0[NG][NH][4];          // -8 2^-24 sum_{d in j} q_d of this lane's columns, for both rows
    float acc[2 * NG][NH][4];
    float R[NH][2], l[NH][2];     // reference of the scores (before their scale), sum of p 2^8
    float base_sc = 0.f;          // scale * k_scale * log2(e)
    float sc[NH][2];              // score scale of this lane's columns (with the head's power of two), positive
    float thr[NH][2];             // the reference is raised where a score less it passes this: TAU / sc, -infinity at first
    uint32_t ok, oks, ov, ovs;    // byte offsets in a tile of this lane's K words, K scales, V words, V scales

    __device__ __forceinline__ void setup(int lane)
    {
        const int gid = lane >> 2, tid = lane & 3;
        ok = lane * (4 * NG);                        // row gid (8 NG bytes to four lanes), word tid NG
        oks = SCALES + gid * NG;
        ov = TILE + tid * ROWB + (D == 128 ? gid ^ ((tid & 2) << 1) : gid) * (2 * NG);
        ovs = TILE + SCALES + tid * (4 * NG);
        asm volatile("" : "+r"(ok), "+r"(oks), "+r"(ov), "+r"(ovs));      // (not formed anew for every block)
    }

    // Shared-memory loads at a 32-bit address.
    template <int N>
    __device__ static __forceinline__ void lds(uint32_t a, uint32_t (&w)[N])
    {
        if constexpr (N == 4)
            asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(a));
        else if constexpr (N == 2)
            asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(a));
        else
            asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w[0]) : "r"(a));
    }
    __device__ static __forceinline__ uint32_t lds16(uint32_t a)
    {
        uint16_t x;
        asm volatile("ld.shared.b16 %0, [%1];" : "=h"(x) : "r"(a));
        return x;
    }

    __device__ void start(const uint16_t *qs, int group, int lane)
    {
        const int gid = lane >> 2, tid = lane & 3;
        float amax[NH], up[NH];
        uint4 raw[NG][NH];
#pragma unroll
        for (int h = 0; h < NH; ++h) amax[h] = 0.f;
#pragma unroll
        for (int j = 0; j < NG; ++j)
#pragma unroll
            for (int h = 0; h < NH; ++h) {
                const int head = 8 * h + gid;
                uint4 x = make_uint4(0u, 0u, 0u, 0u);
                if (head < group) x = *reinterpret_cast<const uint4 *>(qs + head * D + 32 * j + 8 * tid);
                raw[j][h] = x;
                const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) amax[h] = fmaxf(amax[h], fmaxf(fabsf(dev::bf16_lo(w[i])), fabsf(dev::bf16_hi(w[i]))));
            }
#pragma unroll
        for (int h = 0; h < NH; ++h) {
            amax[h] = fmaxf(amax[h], __shfl_xor_sync(dev::FULL, amax[h], 1));         // (head 8 h + gid: this quad's lanes)
            amax[h] = fmaxf(amax[h], __shfl_xor_sync(dev::FULL, amax[h], 2));
            int e = 0;                               // amax * 2^e in [2^14, 2^15)
            if (amax[h] > 0.f) e = 14 - (((int)(__float_as_uint(amax[h]) >> 23) & 0xff) - 127);
            e = max(-126, min(126, e));
            up[h] = copysignf(__uint_as_float((uint32_t)(127 + e) << 23), base_sc);   // (q takes a negative scale's sign)
            // (at a scale of zero a masked score still has to come out as -infinity; the upper end keeps
            // R * sc finite, and from there on any two scores that differ are further apart than f16 reaches)
            const float s = fminf(fmaxf(fabsf(base_sc) * 0x1p24f * __uint_as_float((uint32_t)(127 - e) << 23), 1e-37f), 1e30f);
            sc[h][0] = __shfl_sync(dev::FULL, s, 8 * tid);           // (columns 2 tid, + 1: lanes 4 times that)
            sc[h][1] = __shfl_sync(dev::FULL, s, 8 * tid + 4);
        }
#pragma unroll
        for (int j = 0; j < NG; ++j)
#pragma unroll
            for (int h = 0; h < NH; ++h) {
                const uint32_t w[4] = {raw[j][h].x, raw[j][h].y, raw[j][h].z, raw[j][h].w};
                float x[8], sum = 0.f;               // columns 32 j + 8 tid + i of head 8 h + gid
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    x[2 * i] = dev::bf16_lo(w[i]) * up[h];
                    x[2 * i + 1] = dev::bf16_hi(w[i]) * up[h];
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {        // pair i of a word: codes i and i + 4, at the upper nibbles for odd i
                    const float f = (i & 1) ? 0x1p-4f : 1.f;
                    const uint32_t v = dev::pack_f16x2(x[i] * f, x[i + 4] * f);
                    const float2 y = __half22float2(*reinterpret_cast<const __half2 *>(&v));
                    sum += (y.x + y.y) * ((i & 1) ? 16.f : 1.f);
                    qb[j][h][i] = v;
                }
                sum += __shfl_xor_sync(dev::FULL, sum, 1);
                sum += __shfl_xor_sync(dev::FULL, sum, 2);
                // head 8 h + n's sum lies in lanes 4 n .. 4 n + 3; this lane's columns are 2 tid, + 1
                sum *= -8.f * 0x1p-24f;
                c0[j][h][0] = c0[j][h][2] = __shfl_sync(dev::FULL, sum, 8 * tid);
                c0[j][h][1] = c0[j][h][3] = __shfl_sync(dev::FULL, sum, 8 * tid + 4);
                // kept as they are: the compiler would otherwise form them anew for every block
#pragma unroll
                for (int i = 0; i < 4; ++i) asm volatile("" : "+r"(qb[j][h][i]), "+f"(c0[j][h][i]));
            }
#pragma unroll
        for (int mt = 0; mt < 2 * NG; ++mt)
#pragma unroll
            for (int h = 0; h < NH; ++h)
#pragma unroll
                for (int c = 0; c < 4; ++c) acc[mt][h][c] = 0.f;
#pragma unroll
        for (int h = 0; h < NH; ++h) {
            R[h][0] = R[h][1] = l[h][0] = l[h][1] = 0.f;
            thr[h][0] = thr[h][1] = -INFINITY;
        }
    }

    __device__ static __forceinline__ uint32_t hmul(uint32_t a, uint32_t b)
    {
        const __half2 d = __hmul2(*reinterpret_cast<const __half2 *>(&a), *reinterpret_cast<const __half2 *>(&b));
        return *reinterpret_cast<const uint32_t *>(&d);
    }
    // D = A B + C with a C that stays
    __device__ static __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, const float (&c)[4])
    {
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
            : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
    }

    // S^T - R of one tile: stored rows gid, gid + 8 (tokens t0, t0 + 8); columns 8 h + 2 tid, + 1.
    // (R joins as the sum's start, which takes no instruction more.  Subtracting a rounded R * sc
    // later would leave the product's rounding in the exponent, more than f16 holds from scores of 2^28 on.)
    __device__ __forceinline__ void scores(uint32_t tiles, float (&s)[NH][4])
    {
        uint32_t k0[NG], k1[NG], b0, b1;
        lds(tiles + ok, k0);
        lds(tiles + ok + 8 * ROWB, k1);
        if constexpr (NG == 4) {
            uint32_t t[1];
            lds(tiles + oks, t);
            b0 = t[0];
            lds(tiles + oks + 8 * NG, t);
            b1 = t[0];
        } else {
            b0 = lds16(tiles + oks);
            b1 = lds16(tiles + oks + 8 * NG);
        }
        float ks0[NG], ks1[NG];
#pragma unroll
        for (int j = 0; j < NG; j += 2) {
            const uint32_t x = dev::e4m3x2_to_f16x2((uint16_t)(b0 >> (8 * j)));
            const uint32_t y = dev::e4m3x2_to_f16x2((uint16_t)(b1 >> (8 * j)));
            const float2 fx = __half22float2(*reinterpret_cast<const __half2 *>(&x));
            const float2 fy = __half22float2(*reinterpret_cast<const __half2 *>(&y));
            ks0[j] = fx.x; ks0[j + 1] = fx.y;
            ks1[j] = fy.x; ks1[j + 1] = fy.y;
        }
#pragma unroll
        for (int j = 0; j < NG; ++j) {
            const uint32_t x = k0[j], y = k1[j], x8 = x >> 8, y8 = y >> 8;
            const uint32_t a0[4] = {x & LO, y & LO, x & HI, y & HI}, a1[4] = {x8 & LO, y8 & LO, x8 & HI, y8 & HI};
#pragma unroll
            for (int h = 0; h < NH; ++h) {
                float d[4];
                mma_f16(d, a0, qb[j][h][0], qb[j][h][1], c0[j][h]);
                dev::mma_f16_16816(d, a1, qb[j][h][2], qb[j][h][3]);
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const float f = c < 2 ? ks0[j] : ks1[j];
                    s[h][c] = fmaf(d[c], f, j == 0 ? -R[h][c & 1] : s[h][c]);
                }
            }
        }
    }

    // O^T += V^T (P scale)^T of one tile; pb: tokens tid, tid + 4 of head gid in word 0, tid + 8,
    // tid + 12 in word 1.  MASK: tokens from ntok on count nothing, whatever they hold.
    template <bool MASK>
    __device__ __forceinline__ void outputs(uint32_t tiles, int ntok, int tid, const uint32_t (&pb)[NH][2])
    {
        uint32_t vs[NG];                             // scales of group j: tokens tid, + 4, + 8, + 12
        lds(tiles + ovs, vs);
        if constexpr (MASK) {
            uint32_t mask = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) mask |= tid + 4 * i < ntok ? 0xffu << (8 * i) : 0u;
#pragma unroll
            for (int j = 0; j < NG; ++j) vs[j] &= mask;
        }
        uint32_t w[4][NG / 2];                       // tokens tid + 4 i: 16-bit word of group j in half j & 1
#pragma unroll
        for (int i = 0; i < 4; ++i) lds(tiles + ov + 4 * i * ROWB, w[i]);
#pragma unroll
        for (int j = 0; j < NG; ++j) {
            const uint32_t sel = (j & 1) ? 0x7632u : 0x5410u;
            const uint32_t x = __byte_perm(w[0][j >> 1], w[1][j >> 1], sel);      // tokens tid, tid + 4
            const uint32_t y = __byte_perm(w[2][j >> 1], w[3][j >> 1], sel);      // tokens tid + 8, tid + 12
            const uint32_t x8 = x >> 8, y8 = y >> 8;
            const uint32_t a0[4] = {x & LO, x & HI, y & LO, y & HI}, a1[4] = {x8 & LO, x8 & HI, y8 & LO, y8 & HI};
            constexpr uint32_t EIGHT[4] = {0x80088008u, 0x80808080u, 0x80088008u, 0x80808080u};     // -8 2^-24, -8 2^-20
            // scale 2^-8: the scale bytes at bits 7-14 of each half
            const uint32_t s0 = __byte_perm(vs[j], 0u, 0x4140u) * 128u, s1 = __byte_perm(vs[j], 0u, 0x4342u) * 128u;
#pragma unroll
            for (int h = 0; h < NH; ++h) {
                const uint32_t b0 = hmul(pb[h][0], s0), b1 = hmul(pb[h][1], s1);
                dev::mma_f16_16816(acc[2 * j][h], EIGHT, b0, b1);
                dev::mma_f16_16816(acc[2 * j + 1][h], EIGHT, b0, b1);
                dev::mma_f16_16816(acc[2 * j][h], a0, b0, b1);
                dev::mma_f16_16816(acc[2 * j + 1][h], a1, b0, b1);
            }
        }
    }

    // Two blocks (32 positions), K, V, K, V tiles at the shared-memory address given; FULL: all of them valid, else the first n0 of the first
    // tile and the first n1 of the second (n0 + n1 > 0), the rest masked by select.
    template <bool FULL>
    __device__ __forceinline__ void pair(uint32_t tiles, int n0, int n1, int lane)
    {
        const int gid = lane >> 2, tid = lane & 3;           // (of masked pairs only)
        float s[2][NH][4];
        scores(tiles, s[0]);
        scores(tiles + 2 * TILE, s[1]);
        // ---- mask, lazy running max
        const int t0 = (gid >> 1) + 4 * (gid & 1);
        bool need = false;
#pragma unroll
        for (int h = 0; h < NH; ++h) {
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    if (!FULL && !(t0 + 8 * (c >> 1) < (x ? n1 : n0))) s[x][h][c] = -INFINITY;
                }
#pragma unroll
            for (int r = 0; r < 2; ++r)
                need |= fmaxf(fmaxf(s[0][h][r], s[0][h][r + 2]), fmaxf(s[1][h][r], s[1][h][r + 2])) > thr[h][r];
        }
        if (__any_sync(dev::FULL, need)) {
#pragma unroll
            for (int h = 0; h < NH; ++h)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    float mx = fmaxf(fmaxf(s[0][h][r], s[0][h][r + 2]), fmaxf(s[1][h][r], s[1][h][r + 2]));
                    mx = fmaxf(mx, __shfl_xor_sync(dev::FULL, mx, 4));
                    mx = fmaxf(mx, __shfl_xor_sync(dev::FULL, mx, 8));
                    mx = fmaxf(mx, __shfl_xor_sync(dev::FULL, mx, 16));
                    const bool first = thr[h][r] == -INFINITY;
                    // (no maximum: every score is NaN and so is the sum, which a reference of 0 carries on)
                    const float up = mx > -INFINITY ? (first ? mx : fmaxf(mx, 0.f)) : 0.f;
                    const float alpha = first ? 0.f : dev::fast_exp2(-up * sc[h][r]);
                    R[h][r] += up;                           // (its rounding is one of the later scores', none of the maximum's)
                    thr[h][r] = __fdividef(TAU, sc[h][r]);
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        s[x][h][r] -= up;
                        s[x][h][r + 2] -= up;
                    }
                    l[h][r] *= alpha;
#pragma unroll
                    for (int mt = 0; mt < 2 * NG; ++mt) {
                        acc[mt][h][r] *= alpha;
                        acc[mt][h][r + 2] *= alpha;
                    }
                }
        }
        // ---- P 2^8 = exp2((S - R) sc + 8), transposed
        uint32_t pb[2][NH][2];
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int h = 0; h < NH; ++h) {
                const float p0 = dev::fast_exp2(fmaf(s[x][h][0], sc[h][0], OFF)), p1 = dev::fast_exp2(fmaf(s[x][h][1], sc[h][1], OFF));
                const float p2 = dev::fast_exp2(fmaf(s[x][h][2], sc[h][0], OFF)), p3 = dev::fast_exp2(fmaf(s[x][h][3], sc[h][1], OFF));
                l[h][0] += p0 + p2;
                l[h][1] += p1 + p3;
                pb[x][h][0] = dev::movmatrix_trans(dev::pack_f16x2(p0, p1));
                pb[x][h][1] = dev::movmatrix_trans(dev::pack_f16x2(p2, p3));
            }
        outputs<!FULL>(tiles, n0, tid, pb[0]);
        outputs<!FULL>(tiles + 2 * TILE, n1, tid, pb[1]);
    }

    // The state's rows (query heads 0 .. group - 1): f(row, reference, sum, group j, four consecutive
    // columns from 32 j + 4 gid).
    template <class F>
    __device__ __forceinline__ void rows(int group, int lane, F f)
    {
        const int tid = lane & 3;
#pragma unroll
        for (int h = 0; h < NH; ++h)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                float x = l[h][r];
                x += __shfl_xor_sync(dev::FULL, x, 4);
                x += __shfl_xor_sync(dev::FULL, x, 8);
                x += __shfl_xor_sync(dev::FULL, x, 16);
                const int row = 8 * h + 2 * tid + r;
                const float max = x == 0.f ? -INFINITY : R[h][r] * sc[h][r];      // (no sum: nothing valid, any reference)
                if (row < group) {
#pragma unroll
                    for (int j = 0; j < NG; ++j)
                        // back from n 2^-24 (n 2^-20), and scale 2^-8 (p 2^8 is in the sum as well)
                        f(row, max, x, j, make_float4(acc[2 * j][h][r] * 0x1p32f, acc[2 * j][h][r + 2] * 0x1p28f,
                                                          acc[2 * j + 1][h][r] * 0x1p32f, acc[2 * j + 1][h][r + 2] * 0x1p28f));
                }
            }
    }
};

// Shared memory of a CTA: the warps' rings, then prefix [B + 1], lens [B] and the scan's sums.
template <int D, int NH>
__host__ __device__ constexpr size_t int4_ring_bytes() { return (size_t)int4_warps<D, NH>() * I4_NST * 4 * int4::tile_bytes(D); }

// A unit (layer l, sequence b, KV head h): its length and blocks, the task it starts at.
struct Int4Unit { int l, b, h, L, nb; long long U0; };

// Not inlined: once per unit and 32 tasks, so that the streaming loop stays small.
static __device__ __noinline__ Int4Unit int4_unit_at(long long r, const int32_t *prefix, const int32_t *lens, int B, int layers, int HG, int hh)
{
    Int4Unit u;
    const int W1 = prefix[B];
    u.l = layers > 1 ? (int)div_nonneg(r, W1) : 0;
    const int rl = (int)(r - (long long)u.l * W1);
    u.b = find_seq(prefix, B, rl);
    u.L = lens[u.b];
    u.nb = (u.L + BS - 1) / BS;
    const int hg = (rl - prefix[u.b]) / u.nb;
    u.h = hg * HG + hh;
    u.U0 = (long long)u.l * W1 + prefix[u.b] + (long long)hg * u.nb;
    return u;
}

// The even split of W tasks over T teams.
__host__ __device__ __forceinline__ long long int4_start(long long W, int T, int t) { return W * t / T; }

__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

__device__ __forceinline__ void cp16(uint32_t dst, const void *src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp16_if(uint32_t dst, const void *src, int yes)
{
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %2, 0;\n\t@p cp.async.cg.shared.global [%0], [%1], 16;\n\t}" ::"r"(dst), "l"(src), "r"(yes) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// p.part_o [teams][2][HG][group][D], p.part_ml [teams][2][HG][group][2], p.prefix_n [B + 2]: the
// tasks before each sequence within a layer, then the number of teams.
// APPEND: the new tokens' rows are written first.
template <int D, int NH, bool APPEND>
__global__ void __launch_bounds__(int4_warps<D, NH>() * 32, 1) decode_int4_kernel(const DecodeParams p)
{
    constexpr int NST = I4_NST, NW = int4_warps<D, NH>(), NT = NW * 32;
    constexpr int TILE = int4::tile_bytes(D);
    constexpr int CH = TILE / 16;                  // 16-byte pieces of a tile
    extern __shared__ __align__(128) uint8_t smem[];
    int32_t *prefix = reinterpret_cast<int32_t *>(smem + int4_ring_bytes<D, NH>()), *lens = prefix + p.B + 1;
    int32_t *wsum = lens + p.B;                    // [NW]
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(dev::FULL, tid >> 5, 0);         // (known to be the same in every lane)
    const int Hkv = p.Hkv, group = p.group, HG = int4_team(Hkv), HGN = Hkv / HG;
    pdl_launch();
    pdl_wait();

    // ---- tasks per sequence (head groups x blocks; 0 for an invalid length), scanned
    {
        const int per = (p.B + NT - 1) / NT;
        const int b0 = min(p.B, tid * per), b1 = min(p.B, b0 + per);
        int run = 0;
        for (int b = b0; b < b1; ++b) {
            const int L = __ldcg(p.seq_lens + b);
            const bool ok = L >= 1 && L <= p.MB * BS;
            lens[b] = L;
            if (!ok && blockIdx.x == 0) {
                dev::flag_error(p.err, PKV_DEVERR_SEQ_LEN);
                for (int l = 0; l < p.layers; ++l)
                    for (int e = 0; e < p.Hq * D; ++e) p.out[((size_t)l * p.B + b) * p.Hq * D + e] = 0;
            }
            prefix[b] = run;
            run += ok ? HGN * ((L + BS - 1) / BS) : 0;
        }
        int incl = run;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(dev::FULL, incl, o);
            if (lane >= o) incl += v;
        }
        if (lane == 31) wsum[warp] = incl;
        __syncthreads();
        int base = incl - run, total = 0;
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            if (w < warp) base += wsum[w];
            total += wsum[w];
        }
        for (int b = b0; b < b1; ++b) prefix[b] += base;
        if (tid == 0) prefix[p.B] = total;
        __syncthreads();
    }
    const int W1 = prefix[p.B];
    const long long W = (long long)W1 * p.layers;
    const int teams = (int)min((W + 1) / 2, (long long)((int)gridDim.x * NW / HG));
    if (blockIdx.x == 0) {                         // for the merge
        for (int b = tid; b <= p.B; b += NT) p.prefix_n[b] = prefix[b];
        if (tid == 0) p.prefix_n[p.B + 1] = teams;
    }
    const int gw = blockIdx.x * NW + warp, team = gw / HG, hh = gw - team * HG;
    if (team >= teams) return;
    const long long s = int4_start(W, teams, team), e = int4_start(W, teams, team + 1);
    const int n = (int)(e - s);

    using U = Int4Unit;
    auto unit_of = [&](long long r) { return int4_unit_at(r, prefix, lens, p.B, p.layers, HG, hh); };
    // Tile of task s + i ((layer * blocks + block) * Hkv + head, -1 for a bad entry), for a chunk of
    // 32 tasks, lane x holding task 32 chunk + x.  fetch() starts the table loads two chunks ahead
    // of their use, finish() checks the entries.
    struct Pending { int id, base; };
    auto fetch = [&](int chunk) {
        Pending q{-1, -1};
        const int i = chunk * 32 + lane;
        if (i < n) {
            const U u = unit_of(s + i);
            q.id = __ldcg(p.block_tables + (size_t)u.b * p.MB + (int)(s + i - u.U0));
            q.base = u.l * p.num_blocks * Hkv + u.h;
        }
        return q;
    };
    auto finish = [&](const Pending &q) {
        if (q.base < 0) return -1;
        if (q.id < 0 || q.id >= p.num_blocks) {
            dev::flag_error(p.err, PKV_DEVERR_BLOCK_ID);
            return -1;
        }
        return q.base + q.id * Hkv;
    };
    Pending f0 = fetch(0), f1 = fetch(1), pend = fetch(2);
    int cur = finish(f0), nxt = finish(f1), at = 32;  // tiles of tasks at - 32 .. at - 1, at .. at + 31
    // The ring holds NST pairs of tasks: consecutive blocks of a unit, the second one absent at the
    // end of a run of odd length.  The copy cursor: task s + ii, in a unit whose tasks here end
    // before s + ihi and in all before s + iend.  Bad entries copy tile 0 and count as absent.
    constexpr uint32_t STAGE = 4 * TILE, RING = NST * STAGE;
    const uint32_t ring = dev::smem_u32(smem) + warp * RING;
    const uint8_t *kbase = p.key_cache + lane * 16, *vbase = p.value_cache + lane * 16;
    int ii = 0;
    U iu = unit_of(s);
    int iend = __shfl_sync(dev::FULL, (int)min((long long)INT_MAX, iu.U0 + iu.nb - s), 0), ihi = min(n, iend);
    uint32_t io = 0;                               // its stage's offset
    unsigned good = 0;                             // a bit per tile, the pair copied last at bits 0 and 1
    // the last CH % 32 pieces of a tile: lanes 0 .. 4 REST - 1 take those of the pair's four tiles at once
    constexpr int REST = CH % 32;
    static_assert(4 * REST <= 32, "one copy for the rests");
    const int rt = lane / REST;                    // tile of the pair (K, V, K, V)
    const uint8_t *rbase = ((rt & 1) ? p.value_cache : p.key_cache) + (CH / 32 * 32 + lane % REST) * 16;
    const uint32_t rdst = ring + rt * TILE + (CH / 32 * 32 + lane % REST) * 16;
    const int rest = lane < 4 * REST;
    auto copy_tile = [&](int t, uint32_t dst) {
        const uint8_t *k = kbase + (size_t)(unsigned)t * TILE, *v = vbase + (size_t)(unsigned)t * TILE;
#pragma unroll
        for (int c = 0; c + 32 <= CH; c += 32) {
            cp16(dst + c * 16, k + c * 16);
            cp16(dst + TILE + c * 16, v + c * 16);
        }
    };
    auto issue = [&]() {
        good <<= 2;
        if (ii < n) {
            if (ii >= at) {                        // cur is used up
                cur = nxt;
                nxt = finish(pend);
                pend = fetch((at >> 5) + 2);
                at += 32;
            }
            const int t0 = __shfl_sync(dev::FULL, cur, ii & 31);
            const uint32_t dst = ring + io + lane * 16;
            int last = t0;
            ++ii;
            int t1 = -1;
            const bool two = ii < ihi;
            if (two) {
                t1 = __shfl_sync(dev::FULL, ii < at ? cur : nxt, ii & 31);
                last = t1;
                ++ii;
            }
            if (APPEND && ii == iend && last >= 0) {   // the new token's row goes in before its block is read
                const size_t src = (((size_t)iu.l * p.B + iu.b) * Hkv + iu.h) * D;
                int4::write_row_pair<D>(p.k_new + src, p.v_new + src, p.inv_k_scale, p.inv_v_scale, (iu.L - 1) % BS,
                                        const_cast<uint8_t *>(p.key_cache) + (size_t)last * TILE,
                                        const_cast<uint8_t *>(p.value_cache) + (size_t)last * TILE, lane);
                __threadfence();
                __syncwarp();
            }
            copy_tile(max(t0, 0), dst);
            if (two) copy_tile(max(t1, 0), dst + 2 * TILE);
            cp16_if(rdst + io, rbase + (size_t)(unsigned)max((rt & 2) ? t1 : t0, 0) * TILE, rest);
            good |= (t0 >= 0 ? 1u : 0u) | (t1 >= 0 ? 2u : 0u);
            if (ii == ihi && ii < n) {
                iu = unit_of(s + ii);
                iend = __shfl_sync(dev::FULL, (int)min((long long)INT_MAX, iu.U0 + iu.nb - s), 0);
                ihi = min(n, iend);
            }
            io = io + STAGE == RING ? 0u : io + STAGE;
        }
        cp_commit();                               // a group per step, empty past the end
    };
#pragma unroll 1
    for (int i = 0; i < NST - 1; ++i) issue();

    Int4Compute<D, NH> cmp;
    cmp.base_sc = p.score_scale;
    cmp.setup(lane);
    uint32_t co = ring;                            // address of the next pair to compute
    for (long long lo = s; lo < e;) {
        const U u = unit_of(lo);
        const long long U1 = u.U0 + u.nb, hi = min(e, U1);
        const size_t lb = (size_t)u.l * p.B + u.b;
        cmp.start(p.q + (lb * p.Hq + (size_t)u.h * group) * D, group, lane);
        int left = u.L - (int)(lo - u.U0) * BS;    // positions from this pair on, up to the run's end
        left = __shfl_sync(dev::FULL, min(left, (int)(hi - lo) * BS), 0);
        for (; left > 0; left -= 2 * BS) {
            cp_wait<NST - 2>();                    // this pair has landed (this lane's pieces)
            __syncwarp();                          // every lane's; and the stage before it is read
            issue();
            const unsigned g = (good >> (2 * (NST - 1))) & 3u;
            if (left >= 2 * BS && g == 3u) {
                cmp.template pair<true>(co, BS, BS, lane);
            } else {
                const int n0 = (g & 1u) ? min(left, BS) : 0, n1 = (g & 2u) ? max(0, min(left - BS, BS)) : 0;
                if (n0 + n1 > 0) cmp.template pair<false>(co, n0, n1, lane);
            }
            co = co + STAGE == ring + RING ? ring : co + STAGE;
        }
        const int gid = lane >> 2;
        if (lo == u.U0 && hi == U1) {
            uint16_t *out = p.out + (lb * p.Hq + (size_t)u.h * group) * D + 4 * gid;
            cmp.rows(group, lane, [&](int row, float, float sum, int j, float4 v) {
                const float inv = sum > 0.f ? p.out_scale / sum : 0.f;
                *reinterpret_cast<uint2 *>(out + row * D + 32 * j) =
                    make_uint2(dev::pack_bf16x2(v.x * inv, v.y * inv), dev::pack_bf16x2(v.z * inv, v.w * inv));
            });
        } else {
            const size_t prow = (((size_t)team * 2 + (lo == s ? 0 : 1)) * HG + hh) * group;
            cmp.rows(group, lane, [&](int row, float m, float sum, int j, float4 v) {
                *reinterpret_cast<float4 *>(p.part_o + (prow + row) * D + 32 * j + 4 * gid) = v;
                if (j == 0 && gid == 0) *reinterpret_cast<float2 *>(p.part_ml + (prow + row) * 2) = make_float2(m, sum);
            });
        }
        lo = hi;
    }
    cp_wait<0>();
}

// Merge the partials of cut units.  S warps of a CTA per output row, each taking every S-th partial;
// the row's first warp combines the S results.  Or (S = 1) R rows of one KV head to a warp.  Either way
// 8 partials are in flight at a time.
template <int D, int S, int R>
__global__ void __launch_bounds__(I4_MERGE_WARPS * 32) decode_int4_merge_kernel(const DecodeParams p)
{
    static_assert(S == 1 || R == 1, "one way or the other");
    constexpr int DPL = D / 32, BATCH = 8 / R;
    __shared__ float part[S > 1 ? I4_MERGE_WARPS : 1][D + 2];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, HG = int4_team(p.Hkv), sub = warp % S;
    const long long row = ((long long)blockIdx.x * (I4_MERGE_WARPS / S) + warp / S) * R;
    pdl_launch();
    pdl_wait();
    bool cut = false;
    float M[R], den[R], num[R][DPL];
#pragma unroll
    for (int q = 0; q < R; ++q) {
        M[q] = -INFINITY;
        den[q] = 0.f;
#pragma unroll
        for (int x = 0; x < DPL; ++x) num[q][x] = 0.f;
    }
    if (row < (long long)p.layers * p.B * p.Hq) {
        const int lb = (int)div_nonneg(row, p.Hq), hq = (int)(row - (long long)lb * p.Hq), l = lb / p.B, b = lb - l * p.B;
        const int h = hq / p.group, hg = h / HG, hh = h - hg * HG;
        const int P0 = __ldcg(p.prefix_n + b), P1 = __ldcg(p.prefix_n + b + 1), W1 = __ldcg(p.prefix_n + p.B), T = __ldcg(p.prefix_n + p.B + 1);
        const int nb = (P1 - P0) / (p.Hkv / HG);
        const long long W = (long long)W1 * p.layers, U0 = (long long)l * W1 + P0 + (long long)hg * nb;
        // team of task r: the last t with W t / T <= r
        auto owner = [&](long long r) { return (int)div_nonneg((r + 1) * T - 1, W); };
        const int c0 = nb ? owner(U0) : 0, c1 = nb ? owner(U0 + nb - 1) : 0;
        cut = c0 < c1;                                       // (not an invalid length, nor a whole unit)
        const int first_slot = cut && int4_start(W, T, c0) < U0 ? 1 : 0;
        for (int c = c0 + sub; cut && c <= c1; c += BATCH * S) {
            float2 ml[R][BATCH];
            float o[R][BATCH][DPL];
#pragma unroll
            for (int i = 0; i < BATCH; ++i)
#pragma unroll
                for (int q = 0; q < R; ++q) {
                    const int cc = c + i * S;
                    ml[q][i] = make_float2(-INFINITY, 0.f);
#pragma unroll
                    for (int x = 0; x < DPL; ++x) o[q][i][x] = 0.f;
                    if (cc <= c1) {
                        const size_t pr = (((size_t)cc * 2 + (cc == c0 ? first_slot : 0)) * HG + hh) * p.group + (hq - h * p.group) + q;
                        ml[q][i] = __ldcg(reinterpret_cast<const float2 *>(p.part_ml) + pr);
                        if constexpr (DPL == 4) {
                            const float4 v = __ldcg(reinterpret_cast<const float4 *>(p.part_o + pr * D) + lane);
                            o[q][i][0] = v.x; o[q][i][1] = v.y; o[q][i][2] = v.z; o[q][i][3] = v.w;
                        } else {
                            const float2 v = __ldcg(reinterpret_cast<const float2 *>(p.part_o + pr * D) + lane);
                            o[q][i][0] = v.x; o[q][i][1] = v.y;
                        }
                    }
                }
#pragma unroll
            for (int q = 0; q < R; ++q) {
                float Mn = M[q];
#pragma unroll
                for (int i = 0; i < BATCH; ++i) Mn = fmaxf(Mn, ml[q][i].x);
                if (Mn == -INFINITY) continue;               // nothing valid so far (bad table entries)
                const float a = dev::fast_exp2(M[q] - Mn);
                den[q] *= a;
#pragma unroll
                for (int x = 0; x < DPL; ++x) num[q][x] *= a;
#pragma unroll
                for (int i = 0; i < BATCH; ++i) {
                    const float w = dev::fast_exp2(ml[q][i].x - Mn);
                    den[q] = fmaf(ml[q][i].y, w, den[q]);
#pragma unroll
                    for (int x = 0; x < DPL; ++x) num[q][x] = fmaf(o[q][i][x], w, num[q][x]);
                }
                M[q] = Mn;
            }
        }
    }
    if constexpr (S > 1) {
#pragma unroll
        for (int x = 0; x < DPL; ++x) part[warp][lane * DPL + x] = num[0][x];
        if (lane == 0) {
            part[warp][D] = M[0];
            part[warp][D + 1] = den[0];
        }
        __syncthreads();
        if (sub == 0) {
            float Mn = M[0];
#pragma unroll
            for (int i = 1; i < S; ++i) Mn = fmaxf(Mn, part[warp + i][D]);
            const float a = Mn == -INFINITY ? 0.f : dev::fast_exp2(M[0] - Mn);
            den[0] *= a;
#pragma unroll
            for (int x = 0; x < DPL; ++x) num[0][x] *= a;
#pragma unroll
            for (int i = 1; i < S; ++i) {
                const float w = Mn == -INFINITY ? 0.f : dev::fast_exp2(part[warp + i][D] - Mn);
                den[0] = fmaf(part[warp + i][D + 1], w, den[0]);
#pragma unroll
                for (int x = 0; x < DPL; ++x) num[0][x] = fmaf(part[warp + i][lane * DPL + x], w, num[0][x]);
            }
        }
    }
    if (!cut || sub) return;
#pragma unroll
    for (int q = 0; q < R; ++q) {
        const float inv = den[q] > 0.f ? p.out_scale / den[q] : 0.f;
        uint16_t *dst = p.out + (row + q) * D + lane * DPL;
        if constexpr (DPL == 4)
            *reinterpret_cast<uint2 *>(dst) = make_uint2(dev::pack_bf16x2(num[q][0] * inv, num[q][1] * inv),
                                                         dev::pack_bf16x2(num[q][2] * inv, num[q][3] * inv));
        else
            *reinterpret_cast<uint32_t *>(dst) = dev::pack_bf16x2(num[q][0] * inv, num[q][1] * inv);
    }
}

// Either report CTAs per SM (launch == false) or launch.
template <int D>
cudaError_t dispatch_int4(const Plan &pl, int group, bool launch, int *per_sm, cudaStream_t s, const LaunchArgs *a)
{
    const bool wide = group > 8, append = launch && a->p.k_new;
    auto kernel = wide ? (append ? decode_int4_kernel<D, 2, true> : decode_int4_kernel<D, 2, false>)
                       : (append ? decode_int4_kernel<D, 1, true> : decode_int4_kernel<D, 1, false>);
    const int threads = pl.nw * 32;
    cudaError_t e = prepare(kernel, pl.smem, threads, launch ? nullptr : per_sm);
    if (e != cudaSuccess || !launch) return e;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)pl.grid);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = pl.smem;
    cfg.stream = s;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, kernel, a->p);
    if (e != cudaSuccess || a->p.MB == 1) return e;           // one block: no unit is cut
    // the merge: by a unit's average share of the teams, as many warps to a row as leave each about a
    // batch of its partials, or four rows to a warp where most units are whole or cut once (8192 rows
    // of the ragged batch: 3.7 us a launch less than a warp each)
    const int HG = int4_team(a->p.Hkv);
    const long long rows = (long long)a->p.layers * a->p.B * a->p.Hq, units = (long long)a->p.layers * a->p.B * (a->p.Hkv / HG);
    const long long parts = (long long)pl.grid * pl.nw / HG / units;
    cfg.blockDim = dim3(I4_MERGE_WARPS * 32);
    cfg.dynamicSmemBytes = 0;
    auto merge = [&](auto s_, auto r_) {
        constexpr int S = decltype(s_)::value, R = decltype(r_)::value, PER = I4_MERGE_WARPS / S * R;
        cfg.gridDim = dim3((unsigned)((rows + PER - 1) / PER));
        return cudaLaunchKernelEx(&cfg, decode_int4_merge_kernel<D, S, R>, a->p);
    };
    using One = std::integral_constant<int, 1>;
    if (parts > 32) return merge(std::integral_constant<int, 8>{}, One{});
    if (parts > 8) return merge(std::integral_constant<int, 4>{}, One{});
    if (parts <= 1 && group % 4 == 0) return merge(One{}, std::integral_constant<int, 4>{});
    return merge(One{}, One{});
}

// Warps of a CTA for a group size, and a CTA's shared memory for a batch.
template <int D>
void int4_shape(int group, int B, int *warps, size_t *smem)
{
    const bool wide = group > 8;
    *warps = wide ? int4_warps<D, 2>() : int4_warps<D, 1>();
    *smem = (wide ? int4_ring_bytes<D, 2>() : int4_ring_bytes<D, 1>()) + ((size_t)2 * B + 1 + *warps) * 4;
}

}  // namespace decode
}  // namespace pkv
