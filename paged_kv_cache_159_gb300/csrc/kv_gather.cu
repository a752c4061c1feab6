// kv_gather.cu -- read K/V rows of the paged pool back as bf16, by slot.
//
// The inverse of kv_append: "理解 KV Cache：Attention、P/D 分离与 vLLM 的页式显存管理"
// (steinslab.io) §3.3 gives the address (physical block = slot / 16, offset = slot % 16), and
// its title's P/D separation is the use: the rows that a prefill instance wrote are handed to
// a decode instance, or moved into a pool of another type, whatever the pool stores them in.
//
// A thread per octet (8 columns of a row), K and V by the same thread, so that every output
// row is written in 16-byte pieces by consecutive lanes.  FP8 and INT4 elements become
// bf16(fl32(pool scale * value)): E4M3 values, and scale * (n - 8) of INT4, are exact in fp32,
// so each element is rounded twice, and only once where the pool scale is a power of two.
// Bound by DRAM: a row's reads are 17 D / 32 bytes (INT4), D (FP8) or 2 D, its writes 2 D.
#include <cuda_runtime.h>

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

// Octet o of token t of a tile.
template <int FORMAT, int D, bool IS_K>
__device__ __forceinline__ uint4 read_octet(const uint8_t *tile, int t, int o, float scale)
{
    if constexpr (FORMAT == PKV_KV_BF16) {
        return __ldg(reinterpret_cast<const uint4 *>(tile + t * (2 * D)) + o);
    } else if constexpr (FORMAT == PKV_KV_FP8E4M3) {
        const uint2 c = __ldg(reinterpret_cast<const uint2 *>(tile + t * D) + o);
        float x[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t h = dev::e4m3x2_to_f16x2((uint16_t)((i < 2 ? c.x : c.y) >> (16 * (i & 1))));
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
            x[2 * i] = f.x * scale;
            x[2 * i + 1] = f.y * scale;
        }
        return pack8(x);
    } else {
        using P = int4::Place<D>;
        uint32_t codes, sb;
        if constexpr (IS_K) {
            codes = __ldg(reinterpret_cast<const uint32_t *>(tile + P::k_word(t, o)));
            sb = __ldg(tile + P::k_scale(t, o));
        } else {
            const uint8_t *w = tile + P::v_word(t, o);
            codes = __ldg(reinterpret_cast<const uint16_t *>(w)) |
                    ((uint32_t)__ldg(reinterpret_cast<const uint16_t *>(w + P::VSTEP)) << 16);
            sb = __ldg(tile + P::v_scale(t, o));
        }
        const float s = int4::scale_value(sb);
        float x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = ((float)((int)((codes >> (4 * i)) & 15u) - 8) * s) * scale;
        return pack8(x);
    }
}

template <int FORMAT, int D>
__global__ void __launch_bounds__(THREADS) kv_gather_kernel(
    const int64_t *__restrict__ slots, int64_t num_tokens, int layers, int num_kv_heads, int64_t num_slots,
    float k_scale, float v_scale, const uint8_t *__restrict__ key_cache, const uint8_t *__restrict__ value_cache,
    uint4 *__restrict__ k, uint4 *__restrict__ v, uint32_t *err)
{
    constexpr int OCTETS = D / 8;
    constexpr int64_t TILE = FORMAT == PKV_KV_INT4 ? int4::tile_bytes(D) : 16 * D * (FORMAT == PKV_KV_BF16 ? 2 : 1);
    const int64_t total = layers * num_tokens * num_kv_heads * OCTETS;
    for (int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; i < total; i += (int64_t)gridDim.x * blockDim.x) {
        const int64_t row = i / OCTETS, lt = row / num_kv_heads;       // (layer, token, head); (layer, token)
        const int o = (int)(i - row * OCTETS), h = (int)(row - lt * num_kv_heads);
        const int64_t layer = lt / num_tokens, t = lt - layer * num_tokens;
        const int64_t slot = __ldg(slots + t);
        if (slot >= num_slots) dev::flag_error(err, PKV_DEVERR_SLOT);
        if (slot < 0 || slot >= num_slots) continue;
        const int64_t tile = ((layer * (num_slots >> 4) + (slot >> 4)) * num_kv_heads + h) * TILE;
        const int off = (int)(slot & 15);
        k[i] = read_octet<FORMAT, D, true>(key_cache + tile, off, o, k_scale);
        v[i] = read_octet<FORMAT, D, false>(value_cache + tile, off, o, v_scale);
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
    int64_t blocks = (total + THREADS - 1) / THREADS;
    if (blocks > 65535LL * 32) blocks = 65535LL * 32;
    auto run = [&](auto kernel) {
        kernel<<<(unsigned)blocks, THREADS, 0, static_cast<cudaStream_t>(stream)>>>(
            slot_mapping, num_tokens, layers, d.num_kv_heads, (int64_t)d.num_blocks * d.block_size, d.k_scale,
            d.v_scale, static_cast<const uint8_t *>(key_cache), static_cast<const uint8_t *>(value_cache),
            static_cast<uint4 *>(k), static_cast<uint4 *>(v), pool->d_err);
    };
    const bool wide = d.head_dim == 128;
    if (d.kv_dtype == PKV_KV_BF16) {
        if (wide) run(kv_gather_kernel<PKV_KV_BF16, 128>);
        else run(kv_gather_kernel<PKV_KV_BF16, 64>);
    } else if (d.kv_dtype == PKV_KV_FP8E4M3) {
        if (wide) run(kv_gather_kernel<PKV_KV_FP8E4M3, 128>);
        else run(kv_gather_kernel<PKV_KV_FP8E4M3, 64>);
    } else {
        if (wide) run(kv_gather_kernel<PKV_KV_INT4, 128>);
        else run(kv_gather_kernel<PKV_KV_INT4, 64>);
    }
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
