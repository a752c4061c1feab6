// kv_gather.cu -- read K/V rows of the paged pool back as bf16, by slot.
//
// The inverse of kv_append: "理解 KV Cache：Attention、P/D 分离与 vLLM 的页式显存管理"
// (steinslab.io) §3.3 gives the address (physical block = slot / 16, offset = slot % 16), and
// its title's P/D separation is the use: the rows that a prefill instance wrote are handed to
// a decode instance, or moved into a pool of another type, whatever the pool stores them in.
//
// A thread per octet (8 columns of a row), K and V by the same thread, so that every output
// row is written in 16-byte pieces by consecutive lanes.  An FP8 element becomes bf16(fl32(pool scale *
// value)), an INT4 one bf16(fl32((n - 8) * fl32(scale * pool scale))): at most two fp32 roundings before
// the one to bf16, none where the pool scale is a power of two.
// Bound by DRAM (a row's reads are 17 D / 32 bytes for INT4, D for FP8 or 2 D, its writes 2 D) and, for INT4,
// nearly by instruction issue: 131072 tokens of 8 heads, D 128, 680.5 MB, take 120 us, 5.66 TB/s;
// 157 us with 64-bit indexing and one octet a thread.
#include <cuda_runtime.h>

#include <type_traits>

#include "int4.cuh"
#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {
namespace {

constexpr int THREADS = 256;

__device__ __forceinline__ uint4 pack8(const float (&x)[8])
{
    return make_uint4(dev::pack_bf16x2(x[0], x[1]), dev::pack_bf16x2(x[2], x[3]), dev::pack_bf16x2(x[4], x[5]),
                      dev::pack_bf16x2(x[6], x[7]));
}

// Octet o of token t of a tile: its stored words (load), and its 8 bf16 (expand).
template <int FORMAT, int D, bool IS_K>
struct Octet {
    uint4 w;                              // bf16: the octet; FP8: codes in x, y; INT4: codes in x, the scale byte in y
    __device__ __forceinline__ void load(const uint8_t *tile, int t, int o)
    {
        if constexpr (FORMAT == PKV_KV_BF16) {
            w = __ldg(reinterpret_cast<const uint4 *>(tile + t * (2 * D)) + o);
        } else if constexpr (FORMAT == PKV_KV_FP8E4M3) {
            const uint2 c = __ldg(reinterpret_cast<const uint2 *>(tile + t * D) + o);
            w.x = c.x;
            w.y = c.y;
        } else {
            using P = int4::Place<D>;
            if constexpr (IS_K) {
                w.x = __ldg(reinterpret_cast<const uint32_t *>(tile + P::k_word(t, o)));
                w.y = __ldg(tile + P::k_scale(t, o));
            } else {
                const uint8_t *s = tile + P::v_word(t, o);
                w.x = __ldg(reinterpret_cast<const uint16_t *>(s));
                w.z = __ldg(reinterpret_cast<const uint16_t *>(s + P::VSTEP));
                w.y = __ldg(tile + P::v_scale(t, o));
            }
        }
    }
    __device__ __forceinline__ uint4 expand(float scale) const
    {
        if constexpr (FORMAT == PKV_KV_BF16) {
            return w;
        } else if constexpr (FORMAT == PKV_KV_FP8E4M3) {
            float x[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t h = dev::e4m3x2_to_f16x2((uint16_t)((i < 2 ? w.x : w.y) >> (16 * (i & 1))));
                const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
                x[2 * i] = f.x * scale;
                x[2 * i + 1] = f.y * scale;
            }
            return pack8(x);
        } else {
            const uint32_t codes = IS_K ? w.x : (w.x | (w.z << 16));
            // the nibble at bits 4 i joins 2^23's mantissa in place; less 2^23 + 8 16^i it is (n - 8) 16^i,
            // exactly, and the multiplier's 16^-i brings it back
            const float s = int4::scale_value(w.y) * scale;
            const float m[4] = {s, s * 0x1p-4f, s * 0x1p-8f, s * 0x1p-12f};
            float x[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t bits = ((i < 4 ? codes : codes >> 16) & (15u << (4 * (i & 3)))) | 0x4B000000u;
                x[i] = (__uint_as_float(bits) - (8388608.f + (float)(8 << (4 * (i & 3))))) * m[i & 3];
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
    constexpr int64_t TILE = FORMAT == PKV_KV_INT4 ? int4::tile_bytes(D) : 16 * D * (FORMAT == PKV_KV_BF16 ? 2 : 1);
    const I i0 = (I)blockIdx.x * (I)(THREADS * UNROLL) + threadIdx.x;
    Octet<FORMAT, D, true> ko[UNROLL];
    Octet<FORMAT, D, false> vo[UNROLL];
    bool in[UNROLL];
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
        // (no branches, so that the loads go out together: skipped rows read slot 0)
        const I i = i0 + (I)(THREADS * u);
        const int4::Row<D, I> r(i < total ? i : total - 1, num_tokens, num_kv_heads);
        const int64_t slot = __ldg(slots + r.t);
        const bool valid = slot >= 0 && slot < num_slots;
        in[u] = valid && i < total;
        if (slot >= num_slots) dev::flag_error(err, PKV_DEVERR_SLOT);
        const int64_t at = valid ? slot : 0;
        const int64_t tile = ((r.layer * (num_slots >> 4) + (at >> 4)) * (int64_t)num_kv_heads + r.h) * TILE;
        ko[u].load(key_cache + tile, (int)(at & 15), r.o);
        vo[u].load(value_cache + tile, (int)(at & 15), r.o);
    }
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
        if (!in[u]) continue;
        const I i = i0 + (I)(THREADS * u);
        __stcs(k + i, ko[u].expand(k_scale));
        __stcs(v + i, vo[u].expand(v_scale));
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
    if (d.kv_dtype == PKV_KV_BF16) by_dim(std::integral_constant<int, PKV_KV_BF16>{});
    else if (d.kv_dtype == PKV_KV_FP8E4M3) by_dim(std::integral_constant<int, PKV_KV_FP8E4M3>{});
    else by_dim(std::integral_constant<int, PKV_KV_INT4>{});
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
