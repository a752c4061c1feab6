// int4.cuh -- the INT4 pool format: layout of a tile, quantisation of a row.
//
// "KV Cache 与推理优化" (note.yj-dis.top), section "KV 量化": K/V stored in few bits with
// scales, the arithmetic in higher precision.  A tile (16 tokens of one KV head, K or V) is
// 8 D bytes of codes followed by D / 2 bytes of scales.  Each token's row has a scale (E4M3)
// per group of 32 columns and a 4-bit code n per column: the element is
//     pool scale * scale * (n - 8),   n - 8 in -7 .. 7.
//
// The places follow from how the decode kernel's tensor-core products read them, so that a
// lane fetches whole words and unpacks without moving bits between lanes:
//   * K is the row operand of S^T = K Q^T (rows: tokens; k: columns).  Lane (gid, tid) needs
//     the columns 32 j + 8 tid .. + 7 of mma rows gid and gid + 8 for every group j: they
//     are consecutive 32-bit words, word tid * (D / 32) + j of a row.  Mma row r holds token
//     t(r) with r = (t & 8) | (t & 3) << 1 | (t >> 2 & 1), and rows are stored in that order.
//   * V is the row operand of O^T = V^T P^T (rows: columns d; k: tokens).  Lane (gid, tid)
//     needs the columns 32 j + 4 gid .. + 3 of tokens tid, tid + 4, tid + 8, tid + 12: 16-bit
//     words gid * (D / 32) + j of those rows, pairs of which interleave into f16 pairs (t,
//     t + 4).  At D 128 the rows are 64 bytes, so four of them would share banks: rows
//     with t & 2 set are stored with their halves swapped (gid ^ 4).
//   * A lane's scales are consecutive as well: K byte r * (D / 32) + j; V byte
//     (t & 3) * (D / 8) + 4 j + (t >> 2), four tokens of one group to a word.
// Every byte belongs to one token, so tokens are written independently of each other.
#pragma once

#include <cuda_fp16.h>

#include <cstdint>
#include <type_traits>

#include "pkv_device.cuh"
#include "tc_device.cuh"

namespace pkv {
namespace int4 {

constexpr int GROUP = 32;                     // columns per scale

// Rows (of one head) up to which append and gather take an octet a thread, above it a quarter of a row:
// append / gather at D 128, us: 2048 rows 1.8 / 1.9 against 2.6 / 2.2, 8192 rows 2.7 / 2.5 against 3.2 / 2.5,
// 16384 rows 3.9 / 3.3 against 3.9 / 3.2, 65536 rows 11.0 / 8.5 against 8.9 / 6.7.
constexpr int64_t FEW_ROWS = 8192;

__host__ __device__ constexpr int tile_bytes(int D) { return 8 * D + D / 2; }

// Byte offsets within a tile of token t's octet o (columns 8 o .. 8 o + 7): the 32-bit word
// of K; the two 16-bit words of V (columns 8 o .. + 3 at the first, + 4 .. + 7 VSTEP bytes
// on); the scale of group o / 4.
template <int D>
struct Place {
    static constexpr int NG = D / GROUP;
    static constexpr int VSTEP = 2 * NG;
    __device__ static int k_row(int t) { return (t & 8) | ((t & 3) << 1) | ((t >> 2) & 1); }
    __device__ static int k_word(int t, int o) { return k_row(t) * (D / 2) + ((o & 3) * NG + (o >> 2)) * 4; }
    __device__ static int k_scale(int t, int o) { return 8 * D + k_row(t) * NG + (o >> 2); }
    __device__ static int v_word(int t, int o)
    {
        const int c = 2 * (o & 3);
        return t * (D / 2) + ((D == 128 ? c ^ ((t & 2) << 1) : c) * NG + (o >> 2)) * 2;
    }
    __device__ static int v_scale(int t, int o) { return 8 * D + (t & 3) * (4 * NG) + 4 * (o >> 2) + (t >> 2); }
};

// The value of a scale byte (E4M3, exact in fp32).
__device__ __forceinline__ float scale_value(uint32_t byte)
{
    const uint32_t h = dev::e4m3x2_to_f16x2((uint16_t)byte);
    return __low2float(*reinterpret_cast<const __half2 *>(&h));
}

__device__ __forceinline__ float2 mul2(float2 a, float2 b)
{
    float2 d;
    asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmul.rn.f32x2 z, x, y;\n\tmov.b64 {%0, %1}, z;\n\t}"
        : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}

// (n - 8) * scale of the codes at bits 0-3 of each half of w, as a pair of bf16 (128 + n by an and-or,
// then exact arithmetic) or of f16 (1024 + n).
__device__ __forceinline__ uint32_t expand_pair(uint32_t w, __nv_bfloat162 scale)
{
    const uint32_t x = (w & 0x000F000Fu) | 0x43004300u;
    const __nv_bfloat162 v = __hmul2(__hsub2(*reinterpret_cast<const __nv_bfloat162 *>(&x), __float2bfloat162_rn(136.f)), scale);
    return *reinterpret_cast<const uint32_t *>(&v);
}
__device__ __forceinline__ uint32_t expand_pair(uint32_t w, __half2 scale)
{
    const uint32_t x = (w & 0x000F000Fu) | 0x64006400u;
    const __half2 v = __hmul2(__hsub2(*reinterpret_cast<const __half2 *>(&x), __float2half2_rn(1032.f)), scale);
    return *reinterpret_cast<const uint32_t *>(&v);
}

// Octet of codes (column i at bits 4 i) to 8 elements, T their pair type.
template <class T>
__device__ __forceinline__ uint4 expand_octet(uint32_t codes, uint32_t scale_byte)
{
    T s;
    if constexpr (std::is_same<T, __half2>::value) s = __float2half2_rn(scale_value(scale_byte));
    else s = __float2bfloat162_rn(scale_value(scale_byte));
    // halves hold columns 0-3 and 4-7: pairs (0, 4), (1, 5), (2, 6), (3, 7)
    const uint32_t a = expand_pair(codes, s), b = expand_pair(codes >> 4, s), c = expand_pair(codes >> 8, s),
                   d = expand_pair(codes >> 12, s);
    return make_uint4(__byte_perm(a, b, 0x5410u), __byte_perm(c, d, 0x5410u), __byte_perm(a, b, 0x7632u),
                      __byte_perm(c, d, 0x7632u));
}

// Quantise octets of rows (8 bf16 each; whole warps call it, the 4 consecutive lanes of a group
// share its maximum): the 8 codes, column 8 o + i at bits 4 i, and the group's scale byte.
//   y = fl32(x * fl32(1 / pool scale)),  a = max |y| over the group (NaN ignored),
//   scale = E4M3(fl32(a * fl32(1 / 7))) rounded to nearest even, saturating,
//   n = clamp(rint(fl32(y * fl32(1 / scale))), -7, 7) + 8   (8 where the scale is 0 or y NaN).
// Rounding the scale to nearest moves a by at most 1/16, so |y| / scale < 7.5 and the clamp
// costs no more than half a step; where the scale is neither saturated nor subnormal it
// changes nothing.  Bound by instruction issue, so the common case does without the clamp and
// NaN, and a warp that holds either takes the plain steps below: the maximum is taken on the bits
// of x, two at a time (multiplying is monotonic), and the rest in packed fp32 pairs.  Adding 1.5 2^23
// rounds to the nearest integer (ties to even); four codes join as one exact integer below 2^16.
static __device__ __noinline__ uint32_t quantise_plain(uint4 x, float inv_pool, uint32_t *scale_byte)
{
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    float y[8], a = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        y[i] = __fmul_rn((i & 1) ? dev::bf16_hi(w[i >> 1]) : dev::bf16_lo(w[i >> 1]), inv_pool);
        a = fmaxf(a, fabsf(y[i]));
    }
    a = fmaxf(a, __shfl_xor_sync(dev::FULL, a, 1));
    a = fmaxf(a, __shfl_xor_sync(dev::FULL, a, 2));
    *scale_byte = dev::e4m3x2_satfinite(a * (1.0f / 7.0f), 0.f) & 0xffu;
    const float s = scale_value(*scale_byte), r = s > 0.f ? __frcp_rn(s) : 0.f;
    uint32_t codes = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float v = __fmul_rn(y[i], r);
        v = v == v ? fminf(fmaxf(v, -7.f), 7.f) : 0.f;
        codes |= (uint32_t)(__float2int_rn(v) + 8) << (4 * i);
    }
    return codes;
}

template <int N>
__device__ __forceinline__ void quantise(const uint4 (&x)[N], const float (&inv_pool)[N], uint32_t (&codes)[N],
                                         uint32_t (&scale_byte)[N])
{
    float r[N];
    bool rare = false;
#pragma unroll
    for (int k = 0; k < N; ++k) {
        constexpr uint32_t ABS = 0x7fff7fffu;
        const uint32_t m2 = __vmaxu2(__vmaxu2(x[k].x & ABS, x[k].y & ABS), __vmaxu2(x[k].z & ABS, x[k].w & ABS));
        uint32_t top = max(m2 & 0xffffu, m2 >> 16);
        top = max(top, __shfl_xor_sync(dev::FULL, top, 1));
        top = max(top, __shfl_xor_sync(dev::FULL, top, 2));
        const float a = __uint_as_float(top << 16) * inv_pool[k];
        scale_byte[k] = dev::e4m3x2_satfinite(a * (1.0f / 7.0f), 0.f) & 0xffu;
        const float s = scale_value(scale_byte[k]);
        r[k] = s > 0.f ? __frcp_rn(s) : 0.f;
        rare |= !(a * r[k] < 7.5f);                    // (NaN among them)
    }
    if (__any_sync(dev::FULL, rare)) {
#pragma unroll
        for (int k = 0; k < N; ++k) codes[k] = quantise_plain(x[k], inv_pool[k], &scale_byte[k]);
        return;
    }
#pragma unroll
    for (int k = 0; k < N; ++k) {
        const uint32_t w[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
        float q[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float2 n[2];                               // n + 8
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint32_t b = w[2 * h + i];
                const float2 y = mul2(make_float2(dev::bf16_lo(b), dev::bf16_hi(b)), make_float2(inv_pool[k], inv_pool[k]));
                // (a packed product would be fused with the packed sum, although both say .rn)
                const float2 v = make_float2(__fmul_rn(y.x, r[k]), __fmul_rn(y.y, r[k]));
                n[i] = tc::fadd2(tc::fadd2(v, make_float2(12582912.f, 12582912.f)), make_float2(-12582904.f, -12582904.f));
            }
            const float2 t = tc::ffma2(n[1], make_float2(256.f, 256.f), n[0]);
            q[h] = fmaf(t.y, 16.f, t.x) + 8388608.f;
        }
        codes[k] = __byte_perm(__float_as_uint(q[0]), __float_as_uint(q[1]), 0x5410u);
    }
}

// Token t's octet o of a K or V tile.
template <int D>
__device__ __forceinline__ void store_k(uint8_t *tile, int t, int o, uint32_t codes, uint32_t scale_byte)
{
    using P = Place<D>;
    *reinterpret_cast<uint32_t *>(tile + P::k_word(t, o)) = codes;
    if ((o & 3) == 0) tile[P::k_scale(t, o)] = (uint8_t)scale_byte;
}

template <int D>
__device__ __forceinline__ void store_v(uint8_t *tile, int t, int o, uint32_t codes, uint32_t scale_byte)
{
    using P = Place<D>;
    uint8_t *w = tile + P::v_word(t, o);
    *reinterpret_cast<uint16_t *>(w) = (uint16_t)codes;
    *reinterpret_cast<uint16_t *>(w + P::VSTEP) = (uint16_t)(codes >> 16);
    if ((o & 3) == 0) tile[P::v_scale(t, o)] = (uint8_t)scale_byte;
}

// Lane c of the four that share a row takes octets 4 j + c, one of every group j: 4 NG consecutive
// bytes of the row in K (octet c's words) as in V (the 16-bit words of quads 2 c and 2 c + 1, which are
// octet c's, or c ^ 2's where the row's halves are swapped).  So a row moves in a few wide accesses.
template <int NG>
__device__ __forceinline__ void load_words(const uint8_t *src, uint32_t (&w)[NG])
{
    if constexpr (NG == 4) {
        const uint4 x = __ldg(reinterpret_cast<const uint4 *>(src));
        w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
    } else {
        const uint2 x = __ldg(reinterpret_cast<const uint2 *>(src));
        w[0] = x.x; w[1] = x.y;
    }
}
template <int NG>
__device__ __forceinline__ void store_words(uint8_t *dst, const uint32_t (&w)[NG])
{
    if constexpr (NG == 4) *reinterpret_cast<uint4 *>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
    else *reinterpret_cast<uint2 *>(dst) = make_uint2(w[0], w[1]);
}

// The (layer, token, head) row of lane i of [layers, tokens, heads, LANES]: with 32-bit arithmetic wherever
// the whole range fits (a 64-bit division is some seventy instructions, more than the rest of an
// octet's work).
template <int LANES, class I>
struct Row {
    int h;
    int64_t layer, t;
    __device__ __forceinline__ Row(I i, I num_tokens, I num_kv_heads)
    {
        const I row = i / LANES, lt = row / num_kv_heads, l = lt < num_tokens ? (I)0 : lt / num_tokens;
        h = (int)(row - lt * num_kv_heads);
        layer = (int64_t)l;
        t = (int64_t)(lt - l * num_tokens);
    }
};

// One warp writes token t's K and V rows (bf16, 16-byte aligned) into their tiles: lanes 0 ..
// D / 8 - 1 take K's octets, lanes 16 .. 16 + D / 8 - 1 V's.
template <int D>
__device__ __forceinline__ void write_row_pair(const uint16_t *k, const uint16_t *v, float inv_k, float inv_v, int t,
                                               uint8_t *ktile, uint8_t *vtile, int lane)
{
    const int o = lane & 15;
    const bool isv = lane >= 16, mine = o < D / 8;
    uint4 x[1] = {make_uint4(0u, 0u, 0u, 0u)};
    if (mine) x[0] = *reinterpret_cast<const uint4 *>((isv ? v : k) + 8 * o);
    const float inv[1] = {isv ? inv_v : inv_k};
    uint32_t codes[1], sb[1];
    quantise(x, inv, codes, sb);
    if (!mine) return;
    if (isv) store_v<D>(vtile, t, o, codes[0], sb[0]);
    else store_k<D>(ktile, t, o, codes[0], sb[0]);
}

}  // namespace int4
}  // namespace pkv
