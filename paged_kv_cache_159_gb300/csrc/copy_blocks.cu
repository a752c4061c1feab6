// copy_blocks.cu -- copy whole physical blocks of the paged pool (every layer, K and V).
//
// "KV Cache 与推理优化" (note.yj-dis.top), PagedAttention section: a prefix block is stored
// once and shared by every request that references it; when a request diverges it gets its
// own copy before it writes (copy-on-write).  pkv_cow_prepare picks the (shared, fresh)
// pairs on the host; this kernel makes the fresh blocks byte-identical to the shared ones.
//
// Layout ("理解 KV Cache" §3.2): a cache is [layers, NB, Hkv, 16, D], so one block of one
// layer is a contiguous Hkv * 16 * D elements (32 KiB bf16 at Hkv 8, D 128).  One CTA copies
// one (pair, layer) for K and for V with 16-byte loads, 8 in flight per thread before the
// stores, streaming (evict-first) since the copied block is written again by the append.
#include <cuda_runtime.h>

#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {
namespace {

constexpr int CB_THREADS = 256;
constexpr int CB_UNROLL = 8;

__global__ void __launch_bounds__(CB_THREADS) copy_blocks_kernel(
    const int32_t *__restrict__ src, const int32_t *__restrict__ dst, int layers, int num_blocks,
    int64_t block_words, uint4 *__restrict__ key_cache, uint4 *__restrict__ value_cache,
    uint32_t *err)
{
    const int pair = blockIdx.x / layers, layer = blockIdx.x - pair * layers;
    const int s = __ldg(src + pair), d = __ldg(dst + pair);
    if (s < 0 || s >= num_blocks || d < 0 || d >= num_blocks) {
        if (threadIdx.x == 0 && layer == 0) dev::flag_error(err, PKV_DEVERR_BLOCK_ID);
        return;
    }
    const int64_t base = (int64_t)layer * num_blocks * block_words;
    for (int kv = 0; kv < 2; ++kv) {
        uint4 *cache = kv ? value_cache : key_cache;
        const uint4 *from = cache + base + (int64_t)s * block_words;
        uint4 *to = cache + base + (int64_t)d * block_words;
        for (int64_t i0 = 0; i0 < block_words; i0 += (int64_t)CB_THREADS * CB_UNROLL) {
            uint4 w[CB_UNROLL];
#pragma unroll
            for (int u = 0; u < CB_UNROLL; ++u) {
                const int64_t i = i0 + (int64_t)u * CB_THREADS + threadIdx.x;
                if (i < block_words) w[u] = __ldcs(from + i);
            }
#pragma unroll
            for (int u = 0; u < CB_UNROLL; ++u) {
                const int64_t i = i0 + (int64_t)u * CB_THREADS + threadIdx.x;
                if (i < block_words) __stcs(to + i, w[u]);
            }
        }
    }
}

// Move blocks and point the block tables at their new places: the device side of a compaction
// (pkv_pool_compact picks the moves on the host).  All (move, layer, K or V) blocks are laid end
// to end and cut into pieces of MV_WORDS 16-byte words, one per CTA, so that blocks of any size
// (1 KiB to 512 KiB a layer) keep every thread busy; a thread's MV_UNROLL loads are in flight
// before its stores.  The CTAs past the pieces look every table entry up in src, which is
// descending, by bisection: log2(moves) cached loads per entry instead of a map of the pool.
// Entries change to ids that are not in src, so running it again changes nothing.  Bound by DRAM: 400
// blocks of 8 bf16 layers (419 MB read and written in all) take 66.5 us, 6.31 TB/s.
constexpr int MV_THREADS = 256;
constexpr int MV_UNROLL = 8;
constexpr int MV_WORDS = MV_THREADS * MV_UNROLL;

__global__ void __launch_bounds__(MV_THREADS) move_blocks_kernel(
    const int32_t *__restrict__ src, const int32_t *__restrict__ dst, int moves, int layers, int num_blocks,
    uint32_t block_words, unsigned pieces, uint4 *__restrict__ key_cache, uint4 *__restrict__ value_cache,
    int32_t *__restrict__ tables, int64_t entries, uint32_t *err)
{
    if (blockIdx.x < pieces) {
        const int64_t first = (int64_t)blockIdx.x * MV_WORDS, all = (int64_t)moves * layers * 2 * block_words;
        const uint32_t unit0 = (uint32_t)(first / block_words), rem0 = (uint32_t)(first - (int64_t)unit0 * block_words);
        const uint4 *from[MV_UNROLL];
        uint4 *to[MV_UNROLL], w[MV_UNROLL];
#pragma unroll
        for (int u = 0; u < MV_UNROLL; ++u) {
            const uint32_t off = (uint32_t)u * MV_THREADS + threadIdx.x;
            to[u] = nullptr;
            if (first + off >= all) continue;
            const uint32_t r = rem0 + off, du = r / block_words, unit = unit0 + du;
            const uint32_t ml = unit >> 1, move = ml / (uint32_t)layers, layer = ml - move * (uint32_t)layers;
            const int s = __ldg(src + move), d = __ldg(dst + move);
            if (s < 0 || s >= num_blocks || d < 0 || d >= num_blocks) {
                dev::flag_error(err, PKV_DEVERR_BLOCK_ID);
                continue;
            }
            uint4 *cache = (unit & 1u) ? value_cache : key_cache;
            const int64_t base = (int64_t)layer * num_blocks, word = r - du * block_words;
            from[u] = cache + (base + s) * block_words + word;
            to[u] = cache + (base + d) * block_words + word;
        }
#pragma unroll
        for (int u = 0; u < MV_UNROLL; ++u)
            if (to[u]) w[u] = __ldcs(from[u]);
#pragma unroll
        for (int u = 0; u < MV_UNROLL; ++u)
            if (to[u]) *to[u] = w[u];
        return;
    }
    const int64_t i = (int64_t)(blockIdx.x - pieces) * MV_THREADS + threadIdx.x;
    if (i >= entries) return;
    const int id = tables[i];
    int lo = 0, hi = moves;                            // the first src at or below id
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (__ldg(src + mid) > id) lo = mid + 1;
        else hi = mid;
    }
    if (lo < moves && __ldg(src + lo) == id) {
        const int d = __ldg(dst + lo);
        if (id >= 0 && id < num_blocks && d >= 0 && d < num_blocks) tables[i] = d;
    }
}

}  // namespace
}  // namespace pkv

extern "C" int pkv_move_blocks(pkv_pool *pool, void *key_cache, void *value_cache, const int32_t *src,
                               const int32_t *dst, int32_t num_moves, int32_t *block_tables, int64_t num_entries,
                               void *stream)
{
    int st = pkv::check_attached(pool);
    if (st != PKV_OK) return st;
    if (num_moves < 0 || num_entries < 0 || num_entries >= (int64_t)1 << 36) return PKV_ERR_INVALID;
    if (num_moves == 0) return PKV_OK;
    if (!key_cache || !value_cache || !src || !dst || (num_entries > 0 && !block_tables)) return PKV_ERR_INVALID;
    if ((reinterpret_cast<uintptr_t>(key_cache) & 15u) || (reinterpret_cast<uintptr_t>(value_cache) & 15u) ||
        (reinterpret_cast<uintptr_t>(src) & 3u) || (reinterpret_cast<uintptr_t>(dst) & 3u) ||
        (reinterpret_cast<uintptr_t>(block_tables) & 3u))
        return PKV_ERR_INVALID;
    const pkv_pool_desc &d = pool->desc;
    const int64_t block_words = (int64_t)d.num_kv_heads * pkv::tile_bytes(d) / 16;
    const int64_t units = (int64_t)num_moves * d.num_layers * 2;
    if (units >= (int64_t)1 << 31 || block_words >= (int64_t)1 << 31) return PKV_ERR_INVALID;
    const int64_t pieces = (units * block_words + pkv::MV_WORDS - 1) / pkv::MV_WORDS;
    const int64_t grid = pieces + (num_entries + pkv::MV_THREADS - 1) / pkv::MV_THREADS;
    if (grid >= (int64_t)1 << 31) return PKV_ERR_INVALID;
    pkv::move_blocks_kernel<<<(unsigned)grid, pkv::MV_THREADS, 0, static_cast<cudaStream_t>(stream)>>>(
        src, dst, num_moves, d.num_layers, d.num_blocks, (uint32_t)block_words, (unsigned)pieces,
        static_cast<uint4 *>(key_cache), static_cast<uint4 *>(value_cache), block_tables, num_entries, pool->d_err);
    return cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

extern "C" int pkv_copy_blocks(pkv_pool *pool, void *key_cache, void *value_cache,
                               const int32_t *src, const int32_t *dst, int32_t num_pairs,
                               void *stream)
{
    int st = pkv::check_attached(pool);
    if (st != PKV_OK) return st;
    if (num_pairs < 0) return PKV_ERR_INVALID;
    if (num_pairs == 0) return PKV_OK;
    if (!key_cache || !value_cache || !src || !dst) return PKV_ERR_INVALID;
    if ((reinterpret_cast<uintptr_t>(key_cache) & 15u) || (reinterpret_cast<uintptr_t>(value_cache) & 15u) ||
        (reinterpret_cast<uintptr_t>(src) & 3u) || (reinterpret_cast<uintptr_t>(dst) & 3u))
        return PKV_ERR_INVALID;
    const pkv_pool_desc &d = pool->desc;
    const int layers = d.num_layers;
    if ((int64_t)num_pairs * layers >= (int64_t)1 << 31) return PKV_ERR_INVALID;
    const int64_t block_words = (int64_t)d.num_kv_heads * pkv::tile_bytes(d) / 16;
    pkv::copy_blocks_kernel<<<(unsigned)(num_pairs * layers), pkv::CB_THREADS, 0,
                              static_cast<cudaStream_t>(stream)>>>(
        src, dst, layers, d.num_blocks, block_words, static_cast<uint4 *>(key_cache),
        static_cast<uint4 *>(value_cache), pool->d_err);
    return cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}
