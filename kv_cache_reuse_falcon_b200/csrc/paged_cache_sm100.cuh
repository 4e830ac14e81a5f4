// Rows into and out of a paged KV pool: the write of a ragged batch's rows
// into the requests' pages, and the eviction of the rows that collected the
// least attention weight.  (A paged pool: a unipin_kvpool whose slots are
// pages; row j of request r is row j % n_cap of page page_table[r][j / n_cap].)
#pragma once

#include <cstdint>
#include <cuda_bf16.h>

#include "e4m3.cuh"
#include "paged_common.cuh"
#include "sm100_ptx.cuh"
#include "unipin.h"

namespace unipin {

// ------------------------------------------------------------------- write

struct PgWriteParams {
    const uint4* k;        // [T, H, D] bf16 viewed as 16-byte vectors
    const uint4* v;
    uint8_t* pool_k;       // the layer's planes [S, H, ps, D]
    uint8_t* pool_v;
    const int* cu;         // [B + 1]
    const int* new_lens;   // [B] rows to write
    const int* table;      // [B, max_pages]
    const int* first;      // [B] cache row of the first one
    float* key_weights;    // the layer's [S, H, ps] or null: the written rows' weights become 0
    int H, D, S, ps, max_pages, max_new, total_tokens;
    PgDiv page_of, token_of;   // division by the rows of a page, and by a token's vectors
    float inv_k, inv_v;    // E4M3
    int* status;
};

constexpr int kPgWriteThreads = 256;
constexpr int kPgWriteVecs = 4;   // vectors of K and of V per thread

// Memory bound: each row of K and V read once and written once.  A thread takes 16-byte vectors of
// the packed token rows (consecutive threads: consecutive vectors of a token, all heads), so the
// reads are contiguous; a head's D elements of a row are contiguous in the pool.  Four vectors of
// each tensor are loaded before the first is stored.  Divisions are multiplications (PgDiv) and places
// 32-bit: with 64-bit divisions the instructions and not the memory were the bound (603 us in place of
// 519).  Measured (B200): the history of 256 requests, 32 .. 4096 rows, H = 8, D = 128, into E4M3 (3.26 GB)
// 519 us, 6.28 TB/s, 96% of the rate of a copy; one row of 32 requests 2.2 us, a launch.
// Grid (blocks of rows, B).
template <bool kE4M3>
__global__ void __launch_bounds__(kPgWriteThreads) paged_write_kernel(const PgWriteParams p)
{
    const int b = blockIdx.y;
    const int n = p.new_lens[b];
    const int start = p.cu[b];
    const long long len = (long long)p.cu[b + 1] - start;
    const int first = p.first[b];
    if (n < 0 || n > len || n > p.max_new || first < 0 || start < 0 ||
        (long long)start + n > (long long)p.total_tokens ||
        (long long)first + n > min((long long)p.max_pages * p.ps, 0x7fffffffll)) {
        if (threadIdx.x == 0 && blockIdx.x == 0) report(p.status, (int)UNIPIN_ERR_OUT_OF_RANGE);
        return;
    }
    const int vpr = p.D / 8;                  // vectors of a head's row (a power of two)
    const int vpr_shift = 31 - __clz(vpr);
    const int vpt = p.H * vpr;                // vectors of a token
    // the block's first token, and where in it the block begins; behind it 32 bits are enough
    const long long base = (long long)blockIdx.x * (kPgWriteThreads * kPgWriteVecs);
    const int j0 = (int)(base / vpt);
    const int rest0 = (int)(base - (long long)j0 * vpt) + threadIdx.x;
    const uint4* k = p.k + (long long)start * vpt + base + threadIdx.x;
    const uint4* v = p.v + (long long)start * vpt + base + threadIdx.x;
    uint4 kk[kPgWriteVecs], vv[kPgWriteVecs];
    int j[kPgWriteVecs], rest[kPgWriteVecs];
#pragma unroll
    for (int i = 0; i < kPgWriteVecs; ++i) {
        const int y = rest0 + i * kPgWriteThreads;
        j[i] = p.token_of(y);
        rest[i] = y - j[i] * vpt;
        j[i] += j0;
        if (j[i] < n) {
            kk[i] = __ldg(k + i * kPgWriteThreads);
            vv[i] = __ldg(v + i * kPgWriteThreads);
        }
    }
#pragma unroll
    for (int i = 0; i < kPgWriteVecs; ++i) {
        if (j[i] >= n) break;
        const int h = rest[i] >> vpr_shift, c = rest[i] & (vpr - 1);
        const int row = first + j[i];
        const int pg = p.page_of(row);
        const int page = __ldg(p.table + (size_t)b * p.max_pages + pg);
        if (page < 0 || page >= p.S) {
            report(p.status, (int)UNIPIN_ERR_OUT_OF_RANGE);
            continue;
        }
        const size_t at = ((size_t)page * p.H + h) * p.ps + (row - pg * p.ps);
        const size_t dst = at * vpr + c;
        if (kE4M3) {
            reinterpret_cast<uint2*>(p.pool_k)[dst] = e4m3x8_from_bf16(kk[i], p.inv_k);
            reinterpret_cast<uint2*>(p.pool_v)[dst] = e4m3x8_from_bf16(vv[i], p.inv_v);
        } else {
            reinterpret_cast<uint4*>(p.pool_k)[dst] = kk[i];
            reinterpret_cast<uint4*>(p.pool_v)[dst] = vv[i];
        }
        if (p.key_weights && c == 0) p.key_weights[at] = 0.f;
    }
}

// ------------------------------------------------------------------- evict
//
// Of request r's n cached rows of a key/value head, budget stay if n > budget: the first n_sinks, the
// last n_recent, and of the rows between the ones with the largest weight, equal weights by the
// lowest row.  The kept rows move to rows 0 .. budget - 1 in their order.
//
// paged_evict_select_kernel: one block per (request, head).  The weights of the middle rows become
// order-preserving 32-bit keys; the need-th largest is found by radix selection, eight bits a pass
// (a histogram of the keys that still match; the lanes of a warp with one digit add once: the first
// digits of attention weights are nearly all equal), from a copy in shared memory where it fits.  Then
// each warp counts what stays of its consecutive share of the rows, one scan over the warps gives each
// its place (and its share of the ties, in row order), and it writes the rows' numbers there.
// paged_evict_move_kernel: moves a slice of the bytes of every K or V row, or the weights.  Rows move
// towards the front and in order within a slice, and slices do not touch each other, so the move is in
// place with one barrier per step, and slices, heads and requests give the blocks that fill the memory.
// Bound: memory (the weights once, the kept rows read and written once) where there are many requests;
// else the chain of the four selection passes.  Measured (B200), both kernels: 32 requests of 1500 .. 8192
// rows to 2048, H = 8, D = 128 (514 MB), none of them evicted before, 118 us (4.4 TB/s in all; the selection
// alone 30, issue slots 63% busy, the move 86, DRAM 64%); one of 1000 rows to 500, D = 64, 10.3 us.  With the
// kept rows' numbers loaded in their own step and not the one before, 122 and 12.4 us where a graph that
// repeats the call took 107 and 10.6.

struct PgEvictParams {
    uint8_t* pool_k;       // the layer's planes [S, H, ps, D]
    uint8_t* pool_v;
    float* key_weights;    // the layer's [S, H, ps]
    const int* table;      // [R, max_pages]
    const int* lens;       // [R]
    int* kept;             // [R, H, budget]
    int* new_lens;         // [R]
    int H, S, ps, max_pages, max_len, budget, n_sinks, n_recent;
    int row_bytes;
    PgDiv page_of;         // division by ps
    int keys_cap;          // keys that fit the shared-memory copy
    int* status;
};

constexpr int kPgSelThreads = 1024;      // of a selection block, and where no request is long
constexpr int kPgSelThreadsShort = 256;
constexpr int kPgMoveThreads = 256;

// Larger float, larger key; -0 counts as 0 and NaN as less than every number.
__device__ __forceinline__ uint32_t pg_order_key(float w)
{
    if (w != w) return 0u;
    const uint32_t b = __float_as_uint(w + 0.f);
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

// A request that evicts: its length is in range, above the budget, and every page of its rows exists.
__device__ __forceinline__ bool pg_evict_len_ok(const PgEvictParams& p, int n)
{
    return n >= 0 && n <= p.max_len && (long long)n <= (long long)p.max_pages * p.ps;
}

template <int kThreads>
__global__ void __launch_bounds__(kThreads) paged_evict_select_kernel(const PgEvictParams p)
{
    extern __shared__ uint32_t s_keys[];
    __shared__ uint32_t hist[256];
    __shared__ uint32_t s_prefix, s_need;
    __shared__ int w_keep[kThreads / 32], w_tie[kThreads / 32];
    const int r = blockIdx.y, h = blockIdx.x;
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int n = p.lens[r];
    const int* table = p.table + (size_t)r * p.max_pages;
    int* kept = p.kept + ((size_t)r * p.H + h) * p.budget;
    bool bad = !pg_evict_len_ok(p, n);
    if (!bad && n > 0)
        for (int i = tid, last = p.page_of(n - 1); i <= last; i += kThreads) {   // (n + ps may pass 31 bits)
            const int page = table[i];
            bad |= page < 0 || page >= p.S;
        }
    if (__syncthreads_or(bad)) {
        // nothing moves; the caller sees no kept row and a length of -1
        for (int i = tid; i < p.budget; i += kThreads) kept[i] = -1;
        if (tid == 0) {
            report(p.status, (int)UNIPIN_ERR_OUT_OF_RANGE);
            if (h == 0) p.new_lens[r] = -1;
        }
        return;
    }
    if (tid == 0 && h == 0) p.new_lens[r] = min(n, p.budget);
    if (n <= p.budget) {
        for (int i = tid; i < p.budget; i += kThreads) kept[i] = i < n ? i : -1;
        return;
    }
    auto slot = [&](int j) -> float* {
        const int pg = p.page_of(j);
        return p.key_weights + ((size_t)__ldg(table + pg) * p.H + h) * p.ps + (j - pg * p.ps);
    };
    const int m0 = p.n_sinks, mid = n - p.n_sinks - p.n_recent;   // n > budget >= n_sinks + n_recent
    uint32_t need = (uint32_t)(p.budget - p.n_sinks - p.n_recent);   // 0 <= need < mid
    const bool cached = mid <= p.keys_cap;
    auto key = [&](int i) -> uint32_t { return cached ? s_keys[i] : pg_order_key(*slot(m0 + i)); };
    if (cached)
        for (int i = tid; i < mid; i += kThreads) s_keys[i] = pg_order_key(*slot(m0 + i));
    uint32_t prefix = 0, mask = 0;
    const bool any = need > 0;
    if (any) {
        for (int shift = 24; shift >= 0; shift -= 8) {
            for (int i = tid; i < 256; i += kThreads) hist[i] = 0;
            __syncthreads();
            for (int i0 = 0; i0 < mid; i0 += kThreads) {
                const int i = i0 + tid;
                const uint32_t x = i < mid ? key(i) : 0u;
                const bool in = i < mid && (x & mask) == prefix;
                const uint32_t digit = in ? (x >> shift) & 255u : 256u;
                const uint32_t same = __match_any_sync(0xffffffffu, digit);
                if (in && lane == __ffs(same) - 1) atomicAdd(&hist[digit], (uint32_t)__popc(same));
            }
            __syncthreads();
            if (warp == 0) {
                // lane i: digits 255 - 8 i .. 248 - 8 i, from the largest down
                uint32_t c[8], sum = 0;
#pragma unroll
                for (int d = 0; d < 8; ++d) sum += c[d] = hist[255 - 8 * lane - d];
                uint32_t incl = sum;
#pragma unroll
                for (int off = 1; off < 32; off <<= 1) {
                    const uint32_t up = __shfl_up_sync(0xffffffffu, incl, off);
                    if (lane >= off) incl += up;
                }
                uint32_t above = incl - sum;
                if (above < need && need <= incl) {       // one lane
#pragma unroll
                    for (int d = 0; d < 8; ++d) {
                        if (above < need && need <= above + c[d]) {
                            s_prefix = prefix | ((uint32_t)(255 - 8 * lane - d) << shift);
                            s_need = need - above;
                            break;
                        }
                        above += c[d];
                    }
                }
            }
            __syncthreads();
            prefix = s_prefix;
            need = s_need;
            mask |= 255u << shift;
        }
    } else {
        __syncthreads();
    }
    // every key above `prefix` stays, and the first `need` rows whose key equals it
    const int share = ((n + kThreads - 1) / kThreads) * 32;     // rows of a warp, whole groups of 32
    const int j0 = min(warp * share, n), j1 = min(j0 + share, n);
    auto look = [&](int j, bool& keep, bool& tie) {
        keep = tie = false;
        if (j >= j1) return;
        if (j < m0 || j >= n - p.n_recent) {
            keep = true;
        } else if (any) {
            const uint32_t x = key(j - m0);
            keep = x > prefix;
            tie = x == prefix;
        }
    };
    int n_keep = 0, n_tie = 0;
    for (int j = j0; j < j1; j += 32) {
        bool keep, tie;
        look(j + lane, keep, tie);
        n_keep += __popc(__ballot_sync(0xffffffffu, keep));
        n_tie += __popc(__ballot_sync(0xffffffffu, tie));
    }
    if (lane == 0) {
        w_keep[warp] = n_keep;
        w_tie[warp] = n_tie;
    }
    __syncthreads();
    int ties = 0, at = 0;    // ties and kept rows before this warp's
    {
        const bool is = lane < kThreads / 32;
        const int tw = is ? w_tie[lane] : 0, kw = is ? w_keep[lane] : 0;
        int incl = tw;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int up = __shfl_up_sync(0xffffffffu, incl, off);
            if (lane >= off) incl += up;
        }
        const int stay = kw + max(min((int)need - (incl - tw), tw), 0);   // rows of warp `lane` that stay
        int kept_incl = stay;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int up = __shfl_up_sync(0xffffffffu, kept_incl, off);
            if (lane >= off) kept_incl += up;
        }
        ties = __shfl_sync(0xffffffffu, incl - tw, warp);
        at = __shfl_sync(0xffffffffu, kept_incl - stay, warp);
    }
    for (int j = j0; j < j1; j += 32) {
        bool keep, tie;
        look(j + lane, keep, tie);
        const uint32_t below = (1u << lane) - 1u;
        const uint32_t tb = __ballot_sync(0xffffffffu, tie);
        if (tie && ties + __popc(tb & below) < (int)need) keep = true;
        ties += __popc(tb);
        const uint32_t kb = __ballot_sync(0xffffffffu, keep);
        if (keep) kept[at + __popc(kb & below)] = j + lane;
        at += __popc(kb);
    }
}

// kVec: 16-byte vectors of a row slice.  Grid (2 x slices + 1, H, R): K's slices, then V's, then the weights.
template <int kVec>
__global__ void __launch_bounds__(kPgMoveThreads) paged_evict_move_kernel(const PgEvictParams p)
{
    constexpr int kUnroll = 4;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int r = blockIdx.z, h = blockIdx.y;
    const int n = p.lens[r];
    if (p.new_lens[r] < 0 || n <= p.budget) return;
    const int* table = p.table + (size_t)r * p.max_pages;
    const int* kept = p.kept + ((size_t)r * p.H + h) * p.budget;
    auto row_at = [&](int j) -> size_t {
        const int pg = p.page_of(j);
        return ((size_t)__ldg(table + pg) * p.H + h) * p.ps + (j - pg * p.ps);
    };
    // row kept[i] to row i for all i, `rows` of them per step and load, in order
    auto move = [&](int rows, int row, auto load, auto store) {
        int next[kUnroll];         // kept[] a step ahead: its latency is not added to the rows'
        auto ahead = [&](int i0) {
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                const int i = i0 + u * rows + row;
                next[u] = i < p.budget ? kept[i] : i;
            }
        };
        ahead(0);
        for (int i0 = 0; i0 < p.budget; i0 += rows * kUnroll) {
            decltype(load(size_t(0))) x[kUnroll];
            bool moves[kUnroll];
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                moves[u] = next[u] != i0 + u * rows + row;
                if (moves[u]) x[u] = load(row_at(next[u]));
            }
            ahead(i0 + rows * kUnroll);
            __syncthreads();       // every load of the step precedes its stores
#pragma unroll
            for (int u = 0; u < kUnroll; ++u)
                if (moves[u]) store(row_at(i0 + u * rows + row), x[u]);
        }
    };
    const int slices = gridDim.x / 2;
    if ((int)blockIdx.x == 2 * slices) {
        move(kPgMoveThreads, threadIdx.x, [&](size_t at) { return p.key_weights[at]; },
             [&](size_t at, float w) { p.key_weights[at] = w; });
        return;
    }
    uint8_t* pool = (int)blockIdx.x < slices ? p.pool_k : p.pool_v;
    const size_t col = ((size_t)(blockIdx.x % slices) * kVec + threadIdx.x % kVec) * 16;
    move(kPgMoveThreads / kVec, threadIdx.x / kVec,
         [&](size_t at) { return *reinterpret_cast<const uint4*>(pool + at * p.row_bytes + col); },
         [&](size_t at, uint4 x) { *reinterpret_cast<uint4*>(pool + at * p.row_bytes + col) = x; });
}

}  // namespace unipin
