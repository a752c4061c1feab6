// kv_append.cu -- scatter each new token's K/V rows into its slot of the paged pool.
//
// "理解 KV Cache：Attention、P/D 分离与 vLLM 的页式显存管理" (steinslab.io) §1.3 treats the
// KV cache as an append-only log: each decode step adds one K/V record per token and layer.
// §3.3 gives the address: physical block = slot / block_size, offset = slot % block_size,
// and §3.2 the per-block layout [num_kv_heads, block_size, head_dim].  FP8 pools follow the
// "KV 量化" section of "KV Cache 与推理优化" (note.yj-dis.top): 1-byte storage, scaled.
//
// Work split: one thread per 16-byte piece of a (layer, token, head) row, K and V handled by
// the same thread; consecutive threads cover consecutive bytes of a row, so reads of k/v are
// fully coalesced and each row lands as whole 16-byte stores.  The op moves a few hundred
// KB per step and layer and is launch-latency bound; it shares the decode's stream.  With
// several layers (k, v [layers, tokens, Hkv, D], caches stacked layer-major) one launch
// writes every layer: a token has the same slot in each, since a block spans all layers.
#include <cuda_runtime.h>

#include <type_traits>

#include "int4.cuh"
#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {
namespace {

using dev::flag_error;

// Destination piece of source piece i, or -1 (padding slot) / -2 (slot beyond the pool).
// i runs over [layers, tokens, Hkv, chunks]; the cache is [layers, NB, Hkv, 16, chunks].
__device__ __forceinline__ int64_t dst_piece(int64_t i, const int64_t *__restrict__ slots,
                                             int64_t num_tokens, int num_kv_heads,
                                             int chunks_per_row, int64_t num_slots)
{
    const int64_t per_token = (int64_t)num_kv_heads * chunks_per_row;
    const int64_t lt = i / per_token;                  // layer * num_tokens + t
    const int64_t r = i - lt * per_token;              // = h * chunks_per_row + c
    const int64_t layer = lt / num_tokens, t = lt - layer * num_tokens;
    const int64_t slot = __ldg(slots + t);
    if (slot < 0) return -1;
    if (slot >= num_slots) return -2;
    const int64_t blk = slot >> 4, off = slot & 15;
    const int64_t h = r / chunks_per_row, c = r - h * chunks_per_row;
    return (((layer * (num_slots >> 4) + blk) * num_kv_heads + h) * 16 + off) * chunks_per_row + c;
}

// bf16 pool: 16-byte bit copies.
__global__ void __launch_bounds__(256) kv_append_bf16_kernel(
    const uint4 *__restrict__ k, const uint4 *__restrict__ v, const int64_t *__restrict__ slots,
    int64_t num_tokens, int layers, int num_kv_heads, int chunks_per_row, int64_t num_slots,
    uint4 *__restrict__ key_cache, uint4 *__restrict__ value_cache, uint32_t *err)
{
    const int64_t total = layers * num_tokens * num_kv_heads * chunks_per_row;
    for (int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; i < total;
         i += (int64_t)gridDim.x * blockDim.x) {
        const int64_t dst = dst_piece(i, slots, num_tokens, num_kv_heads, chunks_per_row, num_slots);
        if (dst == -2) flag_error(err, PKV_DEVERR_SLOT);
        if (dst < 0) continue;
        key_cache[dst] = __ldg(k + i);
        value_cache[dst] = __ldg(v + i);
    }
}

using dev::e4m3x2_satfinite;

// 8 bf16 values scaled by inv then encoded: 16 bytes in, 8 bytes out.
__device__ __forceinline__ uint2 encode8(uint4 x, float inv)
{
    uint2 o;
    o.x = e4m3x2_satfinite(dev::bf16_lo(x.x) * inv, dev::bf16_hi(x.x) * inv) |
          (e4m3x2_satfinite(dev::bf16_lo(x.y) * inv, dev::bf16_hi(x.y) * inv) << 16);
    o.y = e4m3x2_satfinite(dev::bf16_lo(x.z) * inv, dev::bf16_hi(x.z) * inv) |
          (e4m3x2_satfinite(dev::bf16_lo(x.w) * inv, dev::bf16_hi(x.w) * inv) << 16);
    return o;
}

// FP8 pool: read 8 bf16, write 8 codes.
__global__ void __launch_bounds__(256) kv_append_fp8_kernel(
    const uint4 *__restrict__ k, const uint4 *__restrict__ v, const int64_t *__restrict__ slots,
    int64_t num_tokens, int layers, int num_kv_heads, int chunks_per_row, int64_t num_slots,
    float inv_k, float inv_v, uint2 *__restrict__ key_cache, uint2 *__restrict__ value_cache,
    uint32_t *err)
{
    const int64_t total = layers * num_tokens * num_kv_heads * chunks_per_row;
    for (int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; i < total;
         i += (int64_t)gridDim.x * blockDim.x) {
        const int64_t dst = dst_piece(i, slots, num_tokens, num_kv_heads, chunks_per_row, num_slots);
        if (dst == -2) flag_error(err, PKV_DEVERR_SLOT);
        if (dst < 0) continue;
        key_cache[dst] = encode8(__ldg(k + i), inv_k);
        value_cache[dst] = encode8(__ldg(v + i), inv_v);
    }
}

// INT4 pool: four lanes share a 32-column group and its maximum (two shuffles), each with 8 columns
// (16 bytes of bf16), K and V by the same thread.  A thread takes GP groups of its row: all of them where
// there are rows enough, so that its codes are 4 NG consecutive bytes of K as of V (int4.cuh) and
// leave in one store each; one of them for few rows, which leaves a thread less to do in turn.
// I: the index type, 32 bits where the lanes' count allows.  Bound by DRAM, instruction issue close behind:
// append and gather of 16411 tokens of 8 heads, D 128, 170 MB, take 28.8 us together, 5.92 TB/s (36.7 with an
// octet a thread).
constexpr int ROW_THREADS = 128;

template <int D, int GP, class I>
__global__ void __launch_bounds__(ROW_THREADS) kv_append_int4_kernel(
    const uint4 *__restrict__ k, const uint4 *__restrict__ v, const int64_t *__restrict__ slots,
    I num_tokens, I total, I num_kv_heads, int64_t num_slots, float inv_k, float inv_v,
    uint8_t *__restrict__ key_cache, uint8_t *__restrict__ value_cache, uint32_t *err)
{
    using P = int4::Place<D>;
    constexpr int NG = P::NG, LANES = 4 * NG / GP;             // lanes of a row
    static_assert(GP == 1 || GP == NG, "one group or all");
    const I i = (I)blockIdx.x * (I)ROW_THREADS + threadIdx.x, j = i < total ? i : total - 1;    // (whole warps: the shuffles)
    const int o = (int)(threadIdx.x % LANES);                  // its octet, or its octet of every group
    const size_t at = (size_t)(j / LANES) * (D / 8) + o;
    uint4 x[2 * GP];
    float inv[2 * GP];
#pragma unroll
    for (int g = 0; g < GP; ++g) {
        x[g] = __ldcs(k + at + 4 * g);
        x[GP + g] = __ldcs(v + at + 4 * g);
        inv[g] = inv_k;
        inv[GP + g] = inv_v;
    }
    const int4::Row<LANES, I> r(j, num_tokens, num_kv_heads);
    const int64_t slot = __ldg(slots + r.t);
    if (slot >= num_slots) flag_error(err, PKV_DEVERR_SLOT);
    uint32_t codes[2 * GP], sb[2 * GP];
    int4::quantise(x, inv, codes, sb);
    if (i >= total || slot < 0 || slot >= num_slots) return;
    const int t = (int)(slot & 15);
    const int64_t tile = ((r.layer * (num_slots >> 4) + (slot >> 4)) * (int64_t)num_kv_heads + r.h) * int4::tile_bytes(D);
    uint8_t *kt = key_cache + tile, *vt = value_cache + tile;
    if constexpr (GP == 1) {
        int4::store_k<D>(kt, t, o, codes[0], sb[0]);
        int4::store_v<D>(vt, t, o, codes[1], sb[1]);
    } else {
        uint32_t kw[NG], vw[NG], ks = 0, vs = 0;
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            kw[g] = codes[g];
            ks |= sb[g] << (8 * g);
            vs |= sb[NG + g] << (8 * g);
        }
#pragma unroll
        for (int g = 0; g < NG; g += 2) {
            vw[g / 2] = __byte_perm(codes[NG + g], codes[NG + g + 1], 0x5410u);
            vw[(NG + g) / 2] = __byte_perm(codes[NG + g], codes[NG + g + 1], 0x7632u);
        }
        int4::store_words(kt + P::k_word(t, o), kw);
        int4::store_words(vt + P::v_word(t, o), vw);
        if (o == 0) {
            if constexpr (NG == 4) *reinterpret_cast<uint32_t *>(kt + P::k_scale(t, 0)) = ks;
            else *reinterpret_cast<uint16_t *>(kt + P::k_scale(t, 0)) = (uint16_t)ks;
        }
        if (o < NG) vt[P::v_scale(t, 4 * o)] = (uint8_t)(vs >> (8 * o));
    }
}

template <int D>
void append_int4(const pkv_pool *pool, int layers, const void *k, const void *v, const int64_t *slots, int32_t num_tokens,
                 void *key_cache, void *value_cache, cudaStream_t s)
{
    const pkv_pool_desc &d = pool->desc;
    const int64_t rows = (int64_t)layers * num_tokens * d.num_kv_heads;
    auto run = [&](auto groups, auto index) {
        constexpr int GP = decltype(groups)::value, LANES = D / 8 / GP;
        using I = decltype(index);
        const int64_t total = rows * LANES;
        kv_append_int4_kernel<D, GP, I><<<(unsigned)((total + ROW_THREADS - 1) / ROW_THREADS), ROW_THREADS, 0, s>>>(
            static_cast<const uint4 *>(k), static_cast<const uint4 *>(v), slots, (I)num_tokens, (I)total, (I)d.num_kv_heads,
            (int64_t)d.num_blocks * d.block_size, pool->inv_k_scale, pool->inv_v_scale, static_cast<uint8_t *>(key_cache),
            static_cast<uint8_t *>(value_cache), pool->d_err);
    };
    constexpr int NG = int4::Place<D>::NG;
    if (rows <= int4::FEW_ROWS) run(std::integral_constant<int, 1>{}, uint32_t{});
    else if (rows < (int64_t)1 << 29) run(std::integral_constant<int, NG>{}, uint32_t{});
    else run(std::integral_constant<int, NG>{}, uint64_t{});
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int append_impl(pkv_pool *pool, int layers, const void *k, const void *v,
                const int64_t *slot_mapping, int32_t num_tokens, void *key_cache,
                void *value_cache, void *stream)
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
    const int chunks = d.head_dim / 8;                 // 8 bf16 source values per chunk
    const int64_t total = (int64_t)layers * num_tokens * d.num_kv_heads * chunks;
    const int threads = 256;
    int64_t blocks = (total + threads - 1) / threads;
    if (blocks > 65535LL * 32) blocks = 65535LL * 32;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int64_t num_slots = (int64_t)d.num_blocks * d.block_size;
    if (d.kv_dtype == PKV_KV_BF16) {
        kv_append_bf16_kernel<<<(unsigned)blocks, threads, 0, s>>>(
            static_cast<const uint4 *>(k), static_cast<const uint4 *>(v), slot_mapping,
            num_tokens, layers, d.num_kv_heads, chunks, num_slots, static_cast<uint4 *>(key_cache),
            static_cast<uint4 *>(value_cache), pool->d_err);
    } else if (d.kv_dtype == PKV_KV_INT4) {
        if (d.head_dim == 128) append_int4<128>(pool, layers, k, v, slot_mapping, num_tokens, key_cache, value_cache, s);
        else append_int4<64>(pool, layers, k, v, slot_mapping, num_tokens, key_cache, value_cache, s);
    } else {
        kv_append_fp8_kernel<<<(unsigned)blocks, threads, 0, s>>>(
            static_cast<const uint4 *>(k), static_cast<const uint4 *>(v), slot_mapping,
            num_tokens, layers, d.num_kv_heads, chunks, num_slots, pool->inv_k_scale,
            pool->inv_v_scale, static_cast<uint2 *>(key_cache), static_cast<uint2 *>(value_cache),
            pool->d_err);
    }
    return cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

}  // namespace
}  // namespace pkv

extern "C" int pkv_kv_append(pkv_pool *pool, const void *k, const void *v,
                             const int64_t *slot_mapping, int32_t num_tokens, void *key_cache,
                             void *value_cache, void *stream)
{
    return pkv::append_impl(pool, 1, k, v, slot_mapping, num_tokens, key_cache, value_cache, stream);
}

extern "C" int pkv_kv_append_layers(pkv_pool *pool, const void *k, const void *v,
                                    const int64_t *slot_mapping, int32_t num_tokens,
                                    void *key_cache, void *value_cache, void *stream)
{
    if (!pool) return PKV_ERR_INVALID;
    return pkv::append_impl(pool, pool->desc.num_layers, k, v, slot_mapping, num_tokens, key_cache,
                            value_cache, stream);
}
