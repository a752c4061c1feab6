// draft_pages.cu -- page bookkeeping of a loop that appends and drafts on the GPU: block tables and
// slots extended from lengths, and the rows of an accepted draft path moved to where they belong.
//
// "理解 KV Cache" (steinslab.io) §3.3: slot = table[pos / 16] * 16 + pos % 16; §3.5: blocks are taken
// from the free pool in order as a sequence grows.  "KV Cache 与推理优化" (note.yj-dis.top),
// PagedAttention: one table a request, blocks on demand.  The host's pkv_build_block_tables and
// pkv_slot_mapping_chunks do the same from host arrays; these kernels do it from device arrays, so
// that a captured graph can step without the host.
#include <cuda_runtime.h>

#include "int4.cuh"
#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {
namespace {

constexpr int BS = 16;

// ------------------------------------------------------------------------------------
// extend_tables.  One CTA looks at every sequence (a thread for up to four), scans the numbers of
// blocks that they need, and fills the empty entries from the reserve: entry i of all that are empty,
// in the order of sequences and positions, gets reserve[cursor + i].  It is the only one to write the
// tables, so no CTA can see an entry half a step old.  Then the rows' slots: by the same CTA up to
// FEW_SLOTS, by a launch over all SMs above.
// Bound by latency: lengths, two entries a sequence, the reserve and the slots' entries are four dependent
// trips to L2: 3.9 us (64 sequences, 8 rows each, in a graph).  512 prompts of 1 to 2000 rows, 501483 in all: 8.6 us in
// two launches, 6.0 MB of slots and positions (one SM stores 64 bytes a cycle, which would be 47 us at 2 GHz).
// ------------------------------------------------------------------------------------
constexpr int EXT_THREADS = 1024;
constexpr int EXT_MOST = 4096;                  // sequences
constexpr int FEW_SLOTS = 8192;
constexpr int ROW_THREADS = 256, ROWS_EACH = 4;

struct ExtendParams {
    const int32_t *lens, *cu;
    int32_t *tables;
    const int32_t *reserve;
    int32_t *state;                             // the reserve's cursor; whether the last call was refused
    int32_t *new_lens;
    int64_t *slots;
    int32_t *positions;                         // or null
    uint32_t *err;
    int B, MB, total, reserve_len, num_blocks;
};

// The sequence of row r: the last b in [lo, hi) with cu[b] <= r.
__device__ __forceinline__ int seq_of(const int32_t *cu, int lo, int hi, int r)
{
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (cu[mid] <= r) lo = mid;
        else hi = mid;
    }
    return lo;
}

// Slot and position of row r of sequence b, whose length with its rows is `end`.
__device__ __forceinline__ void write_slot(const ExtendParams &p, int r, int b, int cu1, int end)
{
    const int pos = end - (cu1 - r);
    const int id = p.tables[(size_t)b * p.MB + pos / BS];
    const bool ok = id >= 0 && id < p.num_blocks;
    if (!ok) dev::flag_error(p.err, PKV_DEVERR_BLOCK_ID);
    p.slots[r] = ok ? (int64_t)id * BS + pos % BS : -1;
    if (p.positions) p.positions[r] = pos;
}

__device__ __forceinline__ void write_padding(const ExtendParams &p, int r)
{
    p.slots[r] = -1;
    if (p.positions) p.positions[r] = 0;
}

__global__ void __launch_bounds__(EXT_THREADS) extend_tables_kernel(const ExtendParams p, int write_rows)
{
    extern __shared__ int shared_ints[];                 // 3 B + 1
    int *first = shared_ints, *base = first + p.B, *cu = base + p.B;
    __shared__ int wsum[EXT_THREADS / 32];
    constexpr int EACH = EXT_MOST / EXT_THREADS;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (p.B + EXT_THREADS - 1) / EXT_THREADS, b0 = min(p.B, tid * per), b1 = min(p.B, b0 + per);
    const int cursor = p.state[0];
    // lengths, and the entries that a sequence's rows fall into: the empty ones are those from `first` on
    int n[EACH], L[EACH], end[EACH];
    bool bad = false;
    int run = 0;
#pragma unroll
    for (int k = 0; k < EACH; ++k) {
        n[k] = 0;
        const int b = b0 + k;
        if (b >= b1) continue;
        const int c0 = p.cu[b], c1 = p.cu[b + 1];
        L[k] = p.lens[b];
        cu[b] = c0;
        if (b == p.B - 1) cu[p.B] = c1;
        const int64_t e = (int64_t)L[k] + c1 - c0;
        if (c0 < 0 || c1 < c0 || c1 > p.total || (b == 0 && c0 != 0) || L[k] < 0 || e > (int64_t)p.MB * BS) {
            bad = true;
            continue;
        }
        end[k] = (int)e;
        const int lo = L[k] / BS, hi = ((int)e + BS - 1) / BS;
        const int32_t *row = p.tables + (size_t)b * p.MB;
        int f = hi;
        if (c1 > c0) {
            const int head = row[lo], tail = row[hi - 1];
            if (head < 0) {
                f = lo;
            } else if (tail < 0) {
                int x = lo, y = hi - 1;                  // row[x] is filled, row[y] empty
                while (y - x > 1) {
                    const int mid = (x + y) >> 1;
                    if (row[mid] < 0) y = mid;
                    else x = mid;
                }
                f = y;
            }
        }
        first[b] = f;
        n[k] = hi - f;
        if (c1 == c0) n[k] = 0;
        run += n[k];
    }
    int incl = run;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(dev::FULL, incl, o);
        if (lane >= o) incl += v;
    }
    if (lane == 31) wsum[warp] = incl;
    const int any_bad = __syncthreads_or(bad);
    int at = incl - run, total = 0;
#pragma unroll
    for (int w = 0; w < EXT_THREADS / 32; ++w) {
        if (w < warp) at += wsum[w];
        total += wsum[w];
    }
    const bool dry = cursor < 0 || total > p.reserve_len - cursor;
    const bool refuse = any_bad || dry;
#pragma unroll
    for (int k = 0; k < EACH; ++k) {
        const int b = b0 + k;
        if (b >= b1) continue;
        base[b] = at;
        at += n[k];
        p.new_lens[b] = refuse ? L[k] : end[k];
    }
    if (tid == 0) {
        if (!refuse) p.state[0] = cursor + total;
        p.state[1] = refuse;
        if (any_bad) dev::flag_error(p.err, PKV_DEVERR_SEQ_LEN);
        else if (dry) dev::flag_error(p.err, PKV_DEVERR_RESERVE);
    }
    __syncthreads();
    if (!refuse) {
        for (int i = tid; i < total; i += EXT_THREADS) {
            const int id = p.reserve[cursor + i], b = seq_of(base, 0, p.B, i);      // (the last of equals: one that needs blocks)
            const bool ok = id >= 0 && id < p.num_blocks;
            if (!ok) dev::flag_error(p.err, PKV_DEVERR_BLOCK_ID);
            p.tables[(size_t)b * p.MB + first[b] + (i - base[b])] = ok ? id : -1;
        }
        __syncthreads();
    }
    if (!write_rows) return;
    const int rows = refuse ? 0 : cu[p.B];
    for (int r = tid; r < p.total; r += EXT_THREADS) {
        if (r < rows) {
            const int b = seq_of(cu, 0, p.B, r);
            write_slot(p, r, b, cu[b + 1], p.new_lens[b]);
        } else {
            write_padding(p, r);
        }
    }
}

__global__ void __launch_bounds__(ROW_THREADS) extend_rows_kernel(const ExtendParams p)
{
    const int r0 = blockIdx.x * (ROW_THREADS * ROWS_EACH);
    const int rows = p.state[1] ? 0 : p.cu[p.B];
    __shared__ int range[2];
    if (threadIdx.x < 2) {
        const int r = threadIdx.x ? r0 + min(ROW_THREADS * ROWS_EACH, p.total - r0) - 1 : r0;
        range[threadIdx.x] = rows > 0 ? seq_of(p.cu, 0, p.B, min(r, rows - 1)) : 0;
    }
    __syncthreads();
    const int lo = range[0], hi = range[1] + 1;
#pragma unroll
    for (int k = 0; k < ROWS_EACH; ++k) {
        const int r = r0 + k * ROW_THREADS + threadIdx.x;
        if (r >= p.total) return;
        if (r < rows) {
            const int b = seq_of(p.cu, lo, hi, r);
            write_slot(p, r, b, p.cu[b + 1], p.new_lens[b]);
        } else {
            write_padding(p, r);
        }
    }
}

// ------------------------------------------------------------------------------------
// accept_rows.  A warp per (layer, sequence, KV head, K or V).  Row path[j] of the sequence's new rows goes
// to place j.  The path is strictly increasing, so path[j] >= j: in chunks of ACC_ROWS in order, all of a
// chunk read before any of it is written, no row is overwritten that a later one comes from.  A row is
// bytes of its own in every pool type, so stored bits move as they are; in INT4 tiles a row's place and the
// order of V's halves follow from its token.
// Bound by latency (path, table entries, rows) up to some hundred rows: 2.4 us (5 trees, FP8, one layer, in a graph);
// then by DRAM: 7.5 us for 64 trees in 8 layers.
// ------------------------------------------------------------------------------------
constexpr int ACC_WARPS = 8, ACC_ROWS = 8;

struct AcceptParams {
    uint8_t *caches[2];
    const int32_t *tables, *lens, *cu, *path, *count;
    int32_t *new_lens;
    uint32_t *err;
    int B, MB, Hkv, max_path, num_blocks;
};

// PIECES: 16-byte pieces of a row (INT4: of its codes).
template <int PIECES, int D, bool I4>
__global__ void __launch_bounds__(ACC_WARPS * 32) accept_rows_kernel(const AcceptParams p)
{
    constexpr int NP = (ACC_ROWS * PIECES + 31) / 32, TILE = I4 ? int4::tile_bytes(D) : PIECES * 16 * BS, NG = D / 32;
    static_assert(!I4 || (PIECES * 16 == D / 2 && ACC_ROWS * NG <= 32), "a piece and a scale a lane");
    const int lane = threadIdx.x & 31;
    const unsigned w = blockIdx.x * ACC_WARPS + (threadIdx.x >> 5), bh = w >> 1;
    if (bh >= (unsigned)p.B * p.Hkv) return;
    const int kv = (int)(w & 1u), b = (int)(bh / p.Hkv), h = (int)(bh - (unsigned)b * p.Hkv), layer = blockIdx.y;
    const bool first = layer == 0 && h == 0 && kv == 0;
    const int L = p.lens[b], P = p.cu[b + 1] - p.cu[b], n = p.count[b];
    const int64_t most = (int64_t)p.MB * BS;
    if (P < 0 || L < P || L > most) {
        if (first && lane == 0) dev::flag_error(p.err, PKV_DEVERR_SEQ_LEN);
        return;
    }
    const int C = L - P;
    const int32_t *path = p.path + (size_t)b * p.max_path, *row = p.tables + (size_t)b * p.MB;
    // the whole path is looked at before anything moves
    bool bad = n < 0 || n > P || n > p.max_path, lost = false;
    if (!bad)
        for (int j = lane; j < n; j += 32) {
            const int x = path[j], before = j ? path[j - 1] : -1;
            if (x <= before || x >= P) {
                bad = true;
            } else {
                const int a = row[(C + x) / BS], z = row[(C + j) / BS];
                lost |= a < 0 || a >= p.num_blocks || z < 0 || z >= p.num_blocks;
            }
        }
    bad = __any_sync(dev::FULL, bad);
    lost = __any_sync(dev::FULL, lost);
    if (bad || lost) {
        if (first && lane == 0) dev::flag_error(p.err, bad ? PKV_DEVERR_PATH : PKV_DEVERR_BLOCK_ID);
        return;
    }
    if (first && lane == 0) p.new_lens[b] = C + n;
    uint8_t *cache = p.caches[kv];
    auto tile_of = [&](int pos) { return cache + (((size_t)layer * p.num_blocks + row[pos / BS]) * p.Hkv + h) * TILE; };
    for (int j0 = 0; j0 < n; j0 += ACC_ROWS) {
        uint4 v[NP];
        uint8_t *to[NP];
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const int e = i * 32 + lane, j = j0 + e / PIECES, c = e % PIECES;
            to[i] = nullptr;
            if (e >= ACC_ROWS * PIECES || j >= n || path[j] == j) continue;
            const int s = C + path[j], d = C + j, ts = s % BS, td = d % BS;
            if constexpr (I4) {
                const int rs = kv ? ts : int4::Place<D>::k_row(ts), rd = kv ? td : int4::Place<D>::k_row(td);
                const int cd = kv && D == 128 ? c ^ ((ts ^ td) & 2) : c;         // V's halves are swapped where t & 2
                v[i] = *reinterpret_cast<const uint4 *>(tile_of(s) + rs * (D / 2) + c * 16);
                to[i] = tile_of(d) + rd * (D / 2) + cd * 16;
            } else {
                v[i] = *reinterpret_cast<const uint4 *>(tile_of(s) + (ts * PIECES + c) * 16);
                to[i] = tile_of(d) + (td * PIECES + c) * 16;
            }
        }
        uint8_t sv = 0, *sto = nullptr;
        if constexpr (I4) {
            const int j = j0 + lane / NG, g = lane % NG;
            if (lane < ACC_ROWS * NG && j < n && path[j] != j) {
                const int s = C + path[j], d = C + j, ts = s % BS, td = d % BS;
                using Pl = int4::Place<D>;
                sv = tile_of(s)[kv ? Pl::v_scale(ts, 4 * g) : Pl::k_scale(ts, 4 * g)];
                sto = tile_of(d) + (kv ? Pl::v_scale(td, 4 * g) : Pl::k_scale(td, 4 * g));
            }
        }
        __syncwarp();                                    // all of the chunk is read
#pragma unroll
        for (int i = 0; i < NP; ++i)
            if (to[i]) *reinterpret_cast<uint4 *>(to[i]) = v[i];
        if (sto) *sto = sv;
        __syncwarp();
    }
}

bool aligned(const void *ptr, uintptr_t a) { return (reinterpret_cast<uintptr_t>(ptr) & (a - 1)) == 0; }

bool overlap(const int32_t *a, uint64_t na, const int32_t *b, uint64_t nb)
{
    const uint64_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + nb * 4 && y < x + na * 4;
}

}  // namespace
}  // namespace pkv

extern "C" int pkv_extend_tables(pkv_pool *pool, const int32_t *seq_lens, const int32_t *cu_q, int32_t batch,
                                 int32_t max_blocks, int32_t total_q, int32_t *block_tables, const int32_t *reserve,
                                 int32_t reserve_len, int32_t *state, int32_t *new_lens, int64_t *slots_out,
                                 int32_t *positions_out, void *stream)
{
    using namespace pkv;
    const int st = check_attached(pool);
    if (st != PKV_OK) return st;
    if (batch < 0 || batch > EXT_MOST || max_blocks < 1 || max_blocks > MOST_TABLE_BLOCKS || total_q < 0 || reserve_len < 0)
        return PKV_ERR_INVALID;
    if (batch == 0) return total_q == 0 ? PKV_OK : PKV_ERR_INVALID;
    if (!seq_lens || !cu_q || !block_tables || !state || !new_lens || (reserve_len > 0 && !reserve) || (total_q > 0 && !slots_out))
        return PKV_ERR_INVALID;
    if (!aligned(seq_lens, 4) || !aligned(cu_q, 4) || !aligned(block_tables, 4) || !aligned(reserve, 4) || !aligned(state, 4) ||
        !aligned(new_lens, 4) || !aligned(slots_out, 8) || !aligned(positions_out, 4))
        return PKV_ERR_INVALID;
    ExtendParams p{seq_lens, cu_q, block_tables, reserve, state, new_lens, slots_out, positions_out, pool->d_err,
                   batch, max_blocks, total_q, reserve_len, pool->desc.num_blocks};
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int smem = (3 * batch + 1) * (int)sizeof(int);
    // (beyond what a launch may have without asking; asked for each time, since the answer is the device's)
    if (smem > 40 * 1024 &&
        cudaFuncSetAttribute(extend_tables_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
        return PKV_ERR_CUDA;
    const bool few = total_q <= FEW_SLOTS;
    extend_tables_kernel<<<1, EXT_THREADS, smem, s>>>(p, few);
    if (!few) {
        const unsigned grid = (unsigned)(((int64_t)total_q + ROW_THREADS * ROWS_EACH - 1) / (ROW_THREADS * ROWS_EACH));
        extend_rows_kernel<<<grid, ROW_THREADS, 0, s>>>(p);
    }
    return cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

extern "C" int pkv_accept_rows(pkv_pool *pool, void *key_cache, void *value_cache, const int32_t *block_tables,
                               const int32_t *seq_lens, const int32_t *cu_q, const int32_t *path,
                               const int32_t *num_accepted, int32_t batch, int32_t max_blocks, int32_t max_path,
                               int32_t *lens_out, void *stream)
{
    using namespace pkv;
    const int st = check_attached(pool);
    if (st != PKV_OK) return st;
    if (batch < 0 || max_blocks < 1 || max_blocks > MOST_TABLE_BLOCKS || max_path < 1) return PKV_ERR_INVALID;
    if (batch == 0) return PKV_OK;
    if (!key_cache || !value_cache || !block_tables || !seq_lens || !cu_q || !path || !num_accepted || !lens_out)
        return PKV_ERR_INVALID;
    if (!aligned(key_cache, 16) || !aligned(value_cache, 16) || !aligned(block_tables, 4) || !aligned(seq_lens, 4) ||
        !aligned(cu_q, 4) || !aligned(path, 4) || !aligned(num_accepted, 4) || !aligned(lens_out, 4))
        return PKV_ERR_INVALID;
    // every warp reads the inputs; one of a sequence writes its new length
    const uint64_t n = (uint64_t)batch;
    if (overlap(lens_out, n, seq_lens, n) || overlap(lens_out, n, num_accepted, n) || overlap(lens_out, n, cu_q, n + 1) ||
        overlap(lens_out, n, path, n * max_path) || overlap(lens_out, n, block_tables, n * max_blocks))
        return PKV_ERR_INVALID;
    const pkv_pool_desc &d = pool->desc;
    AcceptParams p{{static_cast<uint8_t *>(key_cache), static_cast<uint8_t *>(value_cache)}, block_tables, seq_lens, cu_q,
                   path, num_accepted, lens_out, pool->d_err, batch, max_blocks, d.num_kv_heads, max_path, d.num_blocks};
    const int64_t warps = (int64_t)batch * d.num_kv_heads * 2;
    if (warps >= (int64_t)1 << 31) return PKV_ERR_INVALID;
    const dim3 grid((unsigned)((warps + ACC_WARPS - 1) / ACC_WARPS), (unsigned)d.num_layers);
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    auto go = [&](auto kernel) { kernel<<<grid, ACC_WARPS * 32, 0, s>>>(p); };
    const bool wide = d.head_dim == 128;
    if (d.kv_dtype == PKV_KV_BF16) wide ? go(accept_rows_kernel<16, 128, false>) : go(accept_rows_kernel<8, 64, false>);
    else if (d.kv_dtype == PKV_KV_FP8E4M3) wide ? go(accept_rows_kernel<8, 128, false>) : go(accept_rows_kernel<4, 64, false>);
    else wide ? go(accept_rows_kernel<4, 128, true>) : go(accept_rows_kernel<2, 64, true>);
    return cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}
