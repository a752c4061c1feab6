// kv_gather.cu -- read K/V rows of the paged pool back as bf16, by slot.
//
// The inverse of kv_append: "理解 KV Cache：Attention、P/D 分离与 vLLM 的页式显存管理"
// (steinslab.io) §3.3 gives the address (physical block = slot / 16, offset = slot % 16), and
// its title's P/D separation is the use: the rows that a prefill instance wrote are handed to
// a decode instance, or moved into a pool of another type, whatever the pool stores them in.
//
// A thread reads octets (8 columns of a row) of K and V and writes 16 bytes of each.  An FP8 element
// becomes bf16(fl32(pool scale * value)), an INT4 one bf16(fl32((n - 8) * fl32(scale * pool scale))): at most
// two fp32 roundings before the one to bf16, none where the pool scale is a power of two.
// Bound by DRAM (a row's reads are 17 D / 32 bytes for INT4, D for FP8 or 2 D, its writes 2 D): INT4,
// 131072 tokens of 8 heads, D 128, 680.5 MB, take 102.1 us, 6.66 TB/s (an octet a thread 131 us, four 120); of a bf16 pool 158.8 us, 6.77 TB/s,
// of an FP8 one 121.4 us, 6.64 TB/s.
#include <cuda_runtime.h>

#include <type_traits>

#include "int4.cuh"
#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {
namespace {

constexpr int THREADS = 256;
constexpr int ROW_THREADS = 128;              // of the INT4 kernel

__device__ __forceinline__ uint4 pack8(const float (&x)[8])
{
    return make_uint4(dev::pack_bf16x2(x[0], x[1]), dev::pack_bf16x2(x[2], x[3]), dev::pack_bf16x2(x[4], x[5]),
                      dev::pack_bf16x2(x[6], x[7]));
}

// Octet o of token t of a tile: its stored words (load), and its 8 bf16 (expand).
template <int FORMAT, int D>
struct Octet {
    uint4 w;                              // bf16: the octet; FP8: codes in x, y
    __device__ __forceinline__ void load(const uint8_t *tile, int t, int o)
    {
        if constexpr (FORMAT == PKV_KV_BF16) {
            w = __ldg(reinterpret_cast<const uint4 *>(tile + t * (2 * D)) + o);
        } else {
            const uint2 c = __ldg(reinterpret_cast<const uint2 *>(tile + t * D) + o);
            w.x = c.x;
            w.y = c.y;
        }
    }
    __device__ __forceinline__ uint4 expand(float scale) const
    {
        if constexpr (FORMAT == PKV_KV_BF16) {
            return w;
        } else {
            float x[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t h = dev::e4m3x2_to_f16x2((uint16_t)((i < 2 ? w.x : w.y) >> (16 * (i & 1))));
                const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
                x[2 * i] = f.x * scale;
                x[2 * i + 1] = f.y * scale;
            }
            return pack8(x);
        }
    }
};

// A thread takes UNROLL octets a block's width apart, their loads in flight together.  I: the index
// type, 32 bits where the octets' count allows.
template <int FORMAT, int D, int UNROLL, class I>
__global__ void __launch_bounds__(THREADS) kv_gather_kernel(
    const int64_t *__restrict__ slots, I num_tokens, I total, I num_kv_heads, int64_t num_slots,
    float k_scale, float v_scale, const uint8_t *__restrict__ key_cache, const uint8_t *__restrict__ value_cache,
    uint4 *__restrict__ k, uint4 *__restrict__ v, uint32_t *err)
{
    constexpr int64_t TILE = 16 * D * (FORMAT == PKV_KV_BF16 ? 2 : 1);
    const I i0 = (I)blockIdx.x * (I)(THREADS * UNROLL) + threadIdx.x;
    Octet<FORMAT, D> ko[UNROLL], vo[UNROLL];
    bool in[UNROLL];
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
        // (no branches, so that the loads go out together: skipped rows read slot 0)
        const I i = i0 + (I)(THREADS * u);
        const I j = i < total ? i : total - 1;
        const int4::Row<D / 8, I> r(j, num_tokens, num_kv_heads);
        const int o = (int)(j % (D / 8));
        const int64_t slot = __ldg(slots + r.t);
        const bool valid = slot >= 0 && slot < num_slots;
        in[u] = valid && i < total;
        if (slot >= num_slots) dev::flag_error(err, PKV_DEVERR_SLOT);
        const int64_t at = valid ? slot : 0;
        const int64_t tile = ((r.layer * (num_slots >> 4) + (at >> 4)) * (int64_t)num_kv_heads + r.h) * TILE;
        ko[u].load(key_cache + tile, (int)(at & 15), o);
        vo[u].load(value_cache + tile, (int)(at & 15), o);
    }
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
        if (!in[u]) continue;
        const I i = i0 + (I)(THREADS * u);
        __stcs(k + i, ko[u].expand(k_scale));
        __stcs(v + i, vo[u].expand(v_scale));
    }
}

// Octet of codes (column i at bits 4 i), times s: the nibble at bits 4 i joins 2^23's mantissa in
// place; less 2^23 + 8 16^i it is (n - 8) 16^i, exactly, and the multiplier's 16^-i brings it back.
__device__ __forceinline__ uint4 expand_octet(uint32_t codes, float s)
{
    const float m[4] = {s, s * 0x1p-4f, s * 0x1p-8f, s * 0x1p-12f};
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t bits = ((i < 4 ? codes : codes >> 16) & (15u << (4 * (i & 3)))) | 0x4B000000u;
        x[i] = (__uint_as_float(bits) - (8388608.f + (float)(8 << (4 * (i & 3))))) * m[i & 3];
    }
    return pack8(x);
}

// INT4: a thread takes 8 columns of GP groups of its row, K and V: of all groups where there are rows enough,
// so that they are 4 NG consecutive bytes in each (int4.cuh) and come in a few wide loads; of one for few
// rows, which leaves a thread less to do in turn.
template <int D, int GP, class I>
__global__ void __launch_bounds__(ROW_THREADS) kv_gather_int4_kernel(
    const int64_t *__restrict__ slots, I num_tokens, I total, I num_kv_heads, int64_t num_slots,
    float k_scale, float v_scale, const uint8_t *__restrict__ key_cache, const uint8_t *__restrict__ value_cache,
    uint4 *__restrict__ k, uint4 *__restrict__ v, uint32_t *err)
{
    using P = int4::Place<D>;
    constexpr int NG = P::NG, LANES = 4 * NG / GP;             // lanes of a row
    static_assert(GP == 1 || GP == NG, "one group or all");
    const I i = (I)blockIdx.x * (I)ROW_THREADS + threadIdx.x;
    if (i >= total) return;
    const int o = (int)(threadIdx.x % LANES);                  // its octet, or its octet of every group
    const int4::Row<LANES, I> r(i, num_tokens, num_kv_heads);
    const int64_t slot = __ldg(slots + r.t);
    if (slot >= num_slots) dev::flag_error(err, PKV_DEVERR_SLOT);
    if (slot < 0 || slot >= num_slots) return;
    const int t = (int)(slot & 15);
    const int64_t tile = ((r.layer * (num_slots >> 4) + (slot >> 4)) * (int64_t)num_kv_heads + r.h) * int4::tile_bytes(D);
    const uint8_t *kt = key_cache + tile, *vt = value_cache + tile;
    const size_t row = (size_t)(i / LANES) * (D / 8);
    if constexpr (GP == 1) {
        const uint32_t kw = __ldg(reinterpret_cast<const uint32_t *>(kt + P::k_word(t, o)));
        const uint16_t *vp = reinterpret_cast<const uint16_t *>(vt + P::v_word(t, o));
        const uint32_t vw = __ldg(vp) | ((uint32_t)__ldg(vp + P::VSTEP / 2) << 16);
        const uint32_t ks = __ldg(kt + P::k_scale(t, o)), vs = __ldg(vt + P::v_scale(t, o));
        __stcs(k + row + o, expand_octet(kw, int4::scale_value(ks) * k_scale));
        __stcs(v + row + o, expand_octet(vw, int4::scale_value(vs) * v_scale));
    } else {
        uint32_t kw[NG], vw[NG], vs[NG], ks;
        int4::load_words(kt + P::k_word(t, o), kw);
        int4::load_words(vt + t * (D / 2) + o * (4 * NG), vw);        // (in storage order)
        int4::load_words(vt + 8 * D + (t & 3) * (4 * NG), vs);        // (of tokens t & 3, + 4, + 8, + 12)
        if constexpr (NG == 4) ks = __ldg(reinterpret_cast<const uint32_t *>(kt + P::k_scale(t, 0)));
        else ks = __ldg(reinterpret_cast<const uint16_t *>(kt + P::k_scale(t, 0)));
        const int vo = D == 128 ? o ^ (t & 2) : o;                    // the octet that V's words are
#pragma unroll
        for (int j = 0; j < NG; ++j)
            __stcs(k + row + 4 * j + o, expand_octet(kw[j], int4::scale_value((ks >> (8 * j)) & 0xffu) * k_scale));
#pragma unroll
        for (int j = 0; j < NG; ++j) {
            const uint32_t codes = __byte_perm(vw[j >> 1], vw[NG / 2 + (j >> 1)], (j & 1) ? 0x7632u : 0x5410u);
            __stcs(v + row + 4 * j + vo, expand_octet(codes, int4::scale_value((vs[j] >> (8 * (t >> 2))) & 0xffu) * v_scale));
        }
    }
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int gather_impl(pkv_pool *pool, int layers, const int64_t *slot_mapping, int32_t num_tokens, const void *key_cache,
                const void *value_cache, void *k, void *v, void *stream)
{
    int st = check_attached(pool);
    if (st != PKV_OK) return st;
    if (num_tokens < 0) return PKV_ERR_INVALID;
    if (num_tokens == 0) return PKV_OK;
    if (!k || !v || !slot_mapping || !key_cache || !value_cache) return PKV_ERR_INVALID;
    if (!aligned16(k) || !aligned16(v) || !aligned16(key_cache) || !aligned16(value_cache) ||
        (reinterpret_cast<uintptr_t>(slot_mapping) & 7u))
        return PKV_ERR_INVALID;
    const pkv_pool_desc &d = pool->desc;
    const int64_t total = (int64_t)layers * num_tokens * d.num_kv_heads * (d.head_dim / 8);
    auto launch = [&](auto format, auto dim, auto unroll, auto index) {
        constexpr int U = decltype(unroll)::value;
        using I = decltype(index);
        kv_gather_kernel<decltype(format)::value, decltype(dim)::value, U, I>
            <<<(unsigned)((total + THREADS * U - 1) / (THREADS * U)), THREADS, 0, static_cast<cudaStream_t>(stream)>>>(
                slot_mapping, (I)num_tokens, (I)total, (I)d.num_kv_heads, (int64_t)d.num_blocks * d.block_size, d.k_scale,
                d.v_scale, static_cast<const uint8_t *>(key_cache), static_cast<const uint8_t *>(value_cache),
                static_cast<uint4 *>(k), static_cast<uint4 *>(v), pool->d_err);
    };
    auto run = [&](auto format, auto dim) {
        // few octets: one a thread, to spread them over the SMs; many: four in flight
        if (total < (int64_t)1 << 18) launch(format, dim, std::integral_constant<int, 1>{}, uint32_t{});
        else if (total < (int64_t)1 << 31) launch(format, dim, std::integral_constant<int, 4>{}, uint32_t{});
        else launch(format, dim, std::integral_constant<int, 4>{}, uint64_t{});
    };
    auto by_dim = [&](auto format) {
        if (d.head_dim == 128) run(format, std::integral_constant<int, 128>{});
        else run(format, std::integral_constant<int, 64>{});
    };
    auto int4_rows = [&](auto dim, auto groups, auto index) {
        constexpr int D = decltype(dim)::value, GP = decltype(groups)::value;
        using I = decltype(index);
        const int64_t lanes = total / GP;
        kv_gather_int4_kernel<D, GP, I>
            <<<(unsigned)((lanes + ROW_THREADS - 1) / ROW_THREADS), ROW_THREADS, 0, static_cast<cudaStream_t>(stream)>>>(
                slot_mapping, (I)num_tokens, (I)lanes, (I)d.num_kv_heads, (int64_t)d.num_blocks * d.block_size, d.k_scale,
                d.v_scale, static_cast<const uint8_t *>(key_cache), static_cast<const uint8_t *>(value_cache),
                static_cast<uint4 *>(k), static_cast<uint4 *>(v), pool->d_err);
    };
    auto by_int4 = [&](auto dim) {
        constexpr int NG = decltype(dim)::value / 32;
        const int64_t rows = total / (d.head_dim / 8);
        if (rows <= int4::FEW_ROWS) int4_rows(dim, std::integral_constant<int, 1>{}, uint32_t{});
        else if (rows < (int64_t)1 << 29) int4_rows(dim, std::integral_constant<int, NG>{}, uint32_t{});
        else int4_rows(dim, std::integral_constant<int, NG>{}, uint64_t{});
    };
    if (d.kv_dtype == PKV_KV_BF16) by_dim(std::integral_constant<int, PKV_KV_BF16>{});
    else if (d.kv_dtype == PKV_KV_FP8E4M3) by_dim(std::integral_constant<int, PKV_KV_FP8E4M3>{});
    else if (d.head_dim == 128) by_int4(std::integral_constant<int, 128>{});
    else by_int4(std::integral_constant<int, 64>{});
    return cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

}  // namespace
}  // namespace pkv

extern "C" int pkv_kv_gather(pkv_pool *pool, const int64_t *slot_mapping, int32_t num_tokens, const void *key_cache,
                             const void *value_cache, void *k, void *v, void *stream)
{
    return pkv::gather_impl(pool, 1, slot_mapping, num_tokens, key_cache, value_cache, k, v, stream);
}

extern "C" int pkv_kv_gather_layers(pkv_pool *pool, const int64_t *slot_mapping, int32_t num_tokens,
                                    const void *key_cache, const void *value_cache, void *k, void *v, void *stream)
{
    if (!pool) return PKV_ERR_INVALID;
    return pkv::gather_impl(pool, pool->desc.num_layers, slot_mapping, num_tokens, key_cache, value_cache, k, v, stream);
}
