// decode_int4.cuh -- single-query attention over an INT4 pool: the compute of the persistent
// stream-K decode kernel (decode_kernels.cuh) for tiles of 4-bit codes.
//
// With k = scale_kj (n - 8) per group j of 32 columns (the pool's k_scale goes into the score
// scale), and likewise v:
//   S_t   = sum_j scale_tj (sum_{d in j} q_d n_td - 8 sum_{d in j} q_d)
//   O_d   = sum_t (p_t scale_tj(d)) (n_td - 8)
// Both products run on the f16 tensor cores (m16n8k16, fp32 accumulation) with tokens (S^T = K
// Q^T) or columns (O^T = V^T P^T) as the 16 rows and the group's query heads as the 8 columns,
// so each code is unpacked once per step whatever the group.
//   * K codes become 64 + n by one and-or on the packed word (nibble at mantissa bits 4-7 of
//     an f16 with exponent 2^6); the excess 72 sum q of every group is a constant of the unit
//     and enters as the accumulators' start value, so S needs no subtraction per element.  The
//     fp32 sums then carry 72 / 8 times the magnitude, 2^-20 of the largest partial sum.
//   * Group j's partial sums (two k-steps) are multiplied with scale_tj in fp32 as they join S.
//   * p scale is formed per group in f16: p <= 2^7 (the running max is raised past that) and
//     scale <= 448, below f16's largest value; p and p scale each round to 11 bits, and the
//     scales are exact.
//   * V codes become n - 8 exactly (1024 + n or 64 + n, minus a constant, in f16): here an
//     excess in the accumulators would be large against outputs that average out.
//   * q is taken to f16 with a power of two per unit that brings its largest magnitude to
//     [128, 256): exact for every bf16 element above 2^-25 of the largest.
// What bounds it: instruction issue.  At HBM speed an SM receives 42 elements a clock and can
// issue 128 lane instructions, 3 an element; unpacking, the products, scales and softmax of
// a 16-token block take about 2.
#pragma once

#include "decode_kernels.cuh"

namespace pkv {
namespace decode {

template <int D, int NH>
struct Int4Compute {
    static constexpr bool SWIZZLED = false;         // tiles hold their own bank-conflict-free order
    static constexpr bool IDENTITY_SLOTS = true;    // merge-area column d at d
    static constexpr int FORMAT = PKV_KV_INT4;
    static constexpr int TILE = int4::tile_bytes(D);
    static constexpr int NG = D / 32;               // column groups
    static constexpr int ROWB = D / 2;              // bytes of a row's codes
    static constexpr int SCALES = 8 * D;            // byte offset of a tile's scales
    static constexpr float TAU = 7.0f;              // raise the running max beyond 2^7
    static constexpr uint32_t F16_64 = 0x54005400u, F16_1024 = 0x64006400u;      // {64, 64}, {1024, 1024}

    uint32_t qb[NG][2][NH][2];    // Q^T fragments: group, k-step, heads, word
    float c0[NG][NH][2];          // -72 sum_{d in j} q_d of this lane's columns
    float acc[2 * NG][NH][4];
    float m[NH][2], l[NH][2];
    float base_sc = 0.f;          // scale * k_scale * log2(e)
    float sc = 0.f;               // the unit's score scale (with the queries' power of two)

    // Output column of O^T row r (0..15) of m-tile mt: codes 2 (mt & 1) + (r >> 3) of word r & 7.
    __device__ static int dcol(int mt, int r) { return 32 * (mt >> 1) + 4 * (r & 7) + 2 * (mt & 1) + (r >> 3); }
    __device__ static int slot_of_d(int d) { return d; }

    __device__ void start(const uint16_t *qs, int group, int lane)
    {
        const int gid = lane >> 2, tid = lane & 3;
        float amax = 0.f;
        uint4 raw[NG][NH];
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
                for (int i = 0; i < 4; ++i) amax = fmaxf(amax, fmaxf(fabsf(dev::bf16_lo(w[i])), fabsf(dev::bf16_hi(w[i]))));
            }
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(dev::FULL, amax, o));
        int e = 0;                                   // amax * 2^e in [128, 256)
        if (amax > 0.f) e = 7 - (((int)(__float_as_uint(amax) >> 23) & 0xff) - 127);
        e = max(-126, min(126, e));
        const float up = __uint_as_float((uint32_t)(127 + e) << 23);
        sc = base_sc * __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
        for (int j = 0; j < NG; ++j)
#pragma unroll
            for (int h = 0; h < NH; ++h) {
                const uint32_t w[4] = {raw[j][h].x, raw[j][h].y, raw[j][h].z, raw[j][h].w};
                float x[8], sum = 0.f;               // columns 32 j + 8 tid + i of head 8 h + gid
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    x[2 * i] = dev::bf16_lo(w[i]) * up;
                    x[2 * i + 1] = dev::bf16_hi(w[i]) * up;
                }
#pragma unroll
                for (int s = 0; s < 2; ++s)
#pragma unroll
                    for (int b = 0; b < 2; ++b) {    // pair 2 s + b of a word: codes 2 s + b and + 4
                        const uint32_t f = dev::pack_f16x2(x[2 * s + b], x[2 * s + b + 4]);
                        qb[j][s][h][b] = f;
                        const float2 v = __half22float2(*reinterpret_cast<const __half2 *>(&f));
                        sum += v.x + v.y;
                    }
                sum += __shfl_xor_sync(dev::FULL, sum, 1);
                sum += __shfl_xor_sync(dev::FULL, sum, 2);
                // head 8 h + n's sum lies in lanes 4 n .. 4 n + 3; this lane's columns are 2 tid, + 1
                c0[j][h][0] = -72.f * __shfl_sync(dev::FULL, sum, 8 * tid);
                c0[j][h][1] = -72.f * __shfl_sync(dev::FULL, sum, 8 * tid + 4);
            }
#pragma unroll
        for (int mt = 0; mt < 2 * NG; ++mt)
#pragma unroll
            for (int h = 0; h < NH; ++h)
#pragma unroll
                for (int c = 0; c < 4; ++c) acc[mt][h][c] = 0.f;
#pragma unroll
        for (int h = 0; h < NH; ++h) {
            m[h][0] = m[h][1] = -INFINITY;
            l[h][0] = l[h][1] = 0.f;
        }
    }

    __device__ static __forceinline__ uint32_t hsub(uint32_t a, uint32_t b)
    {
        const __half2 d = __hsub2(*reinterpret_cast<const __half2 *>(&a), *reinterpret_cast<const __half2 *>(&b));
        return *reinterpret_cast<const uint32_t *>(&d);
    }
    __device__ static __forceinline__ uint32_t hmul(uint32_t a, uint32_t b)
    {
        const __half2 d = __hmul2(*reinterpret_cast<const __half2 *>(&a), *reinterpret_cast<const __half2 *>(&b));
        return *reinterpret_cast<const uint32_t *>(&d);
    }
    // 64 + n of the nibbles at bits 4-7 of each half
    __device__ static __forceinline__ uint32_t up64(uint32_t w) { return (w & 0x00F000F0u) | F16_64; }
    // 1024 + n of the nibbles at bits 0-3 of each half
    __device__ static __forceinline__ uint32_t up1024(uint32_t w) { return (w & 0x000F000Fu) | F16_1024; }

    // NG consecutive 32-bit words.
    __device__ static __forceinline__ void load_words(const uint8_t *src, uint32_t (&w)[NG])
    {
        if constexpr (NG == 4) {
            const uint4 x = *reinterpret_cast<const uint4 *>(src);
            w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
        } else {
            const uint2 x = *reinterpret_cast<const uint2 *>(src);
            w[0] = x.x; w[1] = x.y;
        }
    }

    // One 16-token block; PARTIAL: only tokens < ntok are valid (the rest masked by select).
    template <bool PARTIAL>
    __device__ __forceinline__ void block_impl(const uint8_t *kt, const uint8_t *vt, int ntok, int lane)
    {
        const int gid = lane >> 2, tid = lane & 3;
        // ---- S^T = K Q^T: stored rows gid, gid + 8 (tokens t0, t0 + 8); columns 8 h + 2 tid, + 1
        const int t0 = (gid >> 1) + 4 * (gid & 1);
        uint32_t k0[NG], k1[NG];
        load_words(kt + gid * ROWB + tid * (4 * NG), k0);
        load_words(kt + (gid + 8) * ROWB + tid * (4 * NG), k1);
        float ks0[NG], ks1[NG];
        {
            const uint8_t *src = kt + SCALES + gid * NG;
            uint32_t b0, b1;
            if constexpr (NG == 4) {
                b0 = *reinterpret_cast<const uint32_t *>(src);
                b1 = *reinterpret_cast<const uint32_t *>(src + 8 * NG);
            } else {
                b0 = *reinterpret_cast<const uint16_t *>(src);
                b1 = *reinterpret_cast<const uint16_t *>(src + 8 * NG);
            }
#pragma unroll
            for (int j = 0; j < NG; j += 2) {
                const uint32_t x = dev::e4m3x2_to_f16x2((uint16_t)(b0 >> (8 * j)));
                const uint32_t y = dev::e4m3x2_to_f16x2((uint16_t)(b1 >> (8 * j)));
                const float2 fx = __half22float2(*reinterpret_cast<const __half2 *>(&x));
                const float2 fy = __half22float2(*reinterpret_cast<const __half2 *>(&y));
                ks0[j] = fx.x; ks0[j + 1] = fx.y;
                ks1[j] = fy.x; ks1[j + 1] = fy.y;
            }
        }
        float s[NH][4];
#pragma unroll
        for (int j = 0; j < NG; ++j) {
            const uint32_t a0[4] = {up64(k0[j] << 4), up64(k1[j] << 4), up64(k0[j]), up64(k1[j])};
            const uint32_t a1[4] = {up64(k0[j] >> 4), up64(k1[j] >> 4), up64(k0[j] >> 8), up64(k1[j] >> 8)};
#pragma unroll
            for (int h = 0; h < NH; ++h) {
                float d[4] = {c0[j][h][0], c0[j][h][1], c0[j][h][0], c0[j][h][1]};
                dev::mma_f16_16816(d, a0, qb[j][0][h][0], qb[j][0][h][1]);
                dev::mma_f16_16816(d, a1, qb[j][1][h][0], qb[j][1][h][1]);
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const float f = c < 2 ? ks0[j] : ks1[j];
                    s[h][c] = j == 0 ? d[c] * f : fmaf(d[c], f, s[h][c]);
                }
            }
        }
        // ---- scale, mask, lazy running max
        bool need = false;
#pragma unroll
        for (int h = 0; h < NH; ++h) {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const float x = s[h][c] * sc;
                s[h][c] = (!PARTIAL || t0 + 8 * (c >> 1) < ntok) ? x : -INFINITY;
            }
            need |= fmaxf(s[h][0], s[h][2]) > m[h][0] + TAU;
            need |= fmaxf(s[h][1], s[h][3]) > m[h][1] + TAU;
        }
        if (__any_sync(dev::FULL, need)) {
#pragma unroll
            for (int h = 0; h < NH; ++h)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    float mx = fmaxf(s[h][r], s[h][r + 2]);
                    mx = fmaxf(mx, __shfl_xor_sync(dev::FULL, mx, 4));
                    mx = fmaxf(mx, __shfl_xor_sync(dev::FULL, mx, 8));
                    mx = fmaxf(mx, __shfl_xor_sync(dev::FULL, mx, 16));
                    const float mn = fmaxf(m[h][r], mx);
                    const float alpha = dev::fast_exp2(m[h][r] - mn);
                    m[h][r] = mn;
                    l[h][r] *= alpha;
#pragma unroll
                    for (int mt = 0; mt < 2 * NG; ++mt) {
                        acc[mt][h][r] *= alpha;
                        acc[mt][h][r + 2] *= alpha;
                    }
                }
        }
        // ---- P = exp2(S - m), transposed: tokens tid, tid + 4 of head gid in word 0, tid + 8,
        //      tid + 12 in word 1
        uint32_t pb[NH][2];
#pragma unroll
        for (int h = 0; h < NH; ++h) {
            const float p0 = dev::fast_exp2(s[h][0] - m[h][0]), p1 = dev::fast_exp2(s[h][1] - m[h][1]);
            const float p2 = dev::fast_exp2(s[h][2] - m[h][0]), p3 = dev::fast_exp2(s[h][3] - m[h][1]);
            l[h][0] += p0 + p2;
            l[h][1] += p1 + p3;
            pb[h][0] = dev::movmatrix_trans(dev::pack_f16x2(p0, p1));
            pb[h][1] = dev::movmatrix_trans(dev::pack_f16x2(p2, p3));
        }
        // ---- O^T += V^T (P scale)^T
        uint32_t vs[NG];                             // scales of group j: tokens tid, + 4, + 8, + 12
        load_words(vt + SCALES + tid * (4 * NG), vs);
        if constexpr (PARTIAL) {                     // a NaN scale past the end would survive p = 0
            uint32_t mask = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) mask |= tid + 4 * i < ntok ? 0xffu << (8 * i) : 0u;
#pragma unroll
            for (int j = 0; j < NG; ++j) vs[j] &= mask;
        }
        uint32_t w[4][NG / 2];                       // tokens tid + 4 i: 16-bit word of group j in half j & 1
        {
            const int c = D == 128 ? gid ^ ((tid & 2) << 1) : gid;
            const uint8_t *src = vt + tid * ROWB + c * (2 * NG);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (NG == 4) {
                    const uint2 x = *reinterpret_cast<const uint2 *>(src + 4 * i * ROWB);
                    w[i][0] = x.x; w[i][1] = x.y;
                } else {
                    w[i][0] = *reinterpret_cast<const uint32_t *>(src + 4 * i * ROWB);
                }
            }
        }
#pragma unroll
        for (int j = 0; j < NG; ++j) {
            const uint32_t sel = (j & 1) ? 0x7632u : 0x5410u;
            const uint32_t x = __byte_perm(w[0][j >> 1], w[1][j >> 1], sel);      // tokens tid, tid + 4
            const uint32_t y = __byte_perm(w[2][j >> 1], w[3][j >> 1], sel);      // tokens tid + 8, tid + 12
            const uint32_t x8 = x >> 8, y8 = y >> 8;
            constexpr uint32_t C1032 = 0x64086408u, C72 = 0x54805480u;
            const uint32_t a0[4] = {hsub(up1024(x), C1032), hsub(up64(x), C72), hsub(up1024(y), C1032), hsub(up64(y), C72)};
            const uint32_t a1[4] = {hsub(up1024(x8), C1032), hsub(up64(x8), C72), hsub(up1024(y8), C1032), hsub(up64(y8), C72)};
            const uint32_t s0 = dev::e4m3x2_to_f16x2((uint16_t)vs[j]), s1 = dev::e4m3x2_to_f16x2((uint16_t)(vs[j] >> 16));
#pragma unroll
            for (int h = 0; h < NH; ++h) {
                const uint32_t b0 = hmul(pb[h][0], s0), b1 = hmul(pb[h][1], s1);
                dev::mma_f16_16816(acc[2 * j][h], a0, b0, b1);
                dev::mma_f16_16816(acc[2 * j + 1][h], a1, b0, b1);
            }
        }
    }

    __device__ void block(const uint8_t *kt, const uint8_t *vt, int ntok, float /*score_scale*/, int lane)
    {
        if (ntok == BS) block_impl<false>(kt, vt, BS, lane);
        else block_impl<true>(kt, vt, ntok, lane);
    }

    // Write this warp's (max, sum) rows and accumulators into the merge area ([head][d]).
    __device__ void dump(float *ml, float *accs, int group, int lane)
    {
        const int gid = lane >> 2, tid = lane & 3;
#pragma unroll
        for (int h = 0; h < NH; ++h)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                float x = l[h][r];
                x += __shfl_xor_sync(dev::FULL, x, 4);
                x += __shfl_xor_sync(dev::FULL, x, 8);
                x += __shfl_xor_sync(dev::FULL, x, 16);
                const int head = 8 * h + 2 * tid + r;
                if (head < group) {
                    if (gid == 0) {
                        ml[head * 2] = m[h][r];
                        ml[head * 2 + 1] = x;
                    }
                    float *row = accs + head * (D + ACC_PAD);
#pragma unroll
                    for (int mt = 0; mt < 2 * NG; ++mt) {
                        row[dcol(mt, gid)] = acc[mt][h][r];
                        row[dcol(mt, gid + 8)] = acc[mt][h][r + 2];
                    }
                }
            }
    }
};

template <int D, int NW, int NS, int NH>
__global__ void __launch_bounds__((NW + 2) * 32, 8 / NW) decode_int4_kernel(const DecodeParams p)
{
    Int4Compute<D, NH> cmp;
    cmp.base_sc = p.score_scale;
    decode_body<D, NW, NS, 1>(p, cmp, nullptr, nullptr);
}

// Either report CTAs per SM (launch == false) or launch.
template <int D>
cudaError_t dispatch_int4(const Plan &pl, int group, bool launch, int *per_sm, cudaStream_t s, const LaunchArgs *a)
{
    auto go = [&](auto kernel) -> cudaError_t {
        const int threads = (pl.nw + 2) * 32;
        cudaError_t e = prepare(kernel, pl.smem, threads, launch ? nullptr : per_sm);
        if (e != cudaSuccess || !launch) return e;
        kernel<<<pl.grid, threads, pl.smem, s>>>(a->p);
        return cudaGetLastError();
    };
    auto by_ring = [&](auto nh) -> cudaError_t {
        constexpr int NH = decltype(nh)::value;
        if (pl.nw == 4 && pl.ns == 4) return go(decode_int4_kernel<D, 4, 4, NH>);
        if (pl.nw == 4 && pl.ns == 8) return go(decode_int4_kernel<D, 4, 8, NH>);
        if (pl.nw == 8 && pl.ns == 4) return go(decode_int4_kernel<D, 8, 4, NH>);
        return cudaErrorInvalidConfiguration;
    };
    return group > 8 ? by_ring(std::integral_constant<int, 2>{}) : by_ring(std::integral_constant<int, 1>{});
}

}  // namespace decode
}  // namespace pkv
