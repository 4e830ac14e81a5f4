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
// each tensor are loaded before the first is stored.
// Grid (blocks of rows, B).
template <bool kE4M3>
__global__ void __launch_bounds__(kPgWriteThreads) paged_write_kernel(const PgWriteParams p)
{
    const int b = blockIdx.y;
    const int n = p.new_lens[b];
    const int start = p.cu[b];
    const int len = p.cu[b + 1] - start;
    const int first = p.first[b];
    if (n < 0 || n > len || n > p.max_new || first < 0 || start < 0 ||
        (long long)start + n > (long long)p.total_tokens ||
        (long long)first + n > (long long)p.max_pages * p.ps) {
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
// (a histogram of the keys that still match), from a copy in shared memory where it fits.  A pass
// over the rows in order then writes the kept rows' indices (ballots and a block-wide prefix give
// each its place; ties are counted in row order), and moves the weights: a row moves only towards
// the front, and a step's loads all precede its stores, so it can be done in place.
// paged_evict_move_kernel: the same move for a slice of the bytes of every K or V row.  Rows move in
// order within a slice and slices do not touch each other, so the move is in place with one barrier
// per step, and slices, heads and requests give the blocks that fill the memory.
// Bound: memory (the weights once, the kept rows read and written once).

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

constexpr int kPgSelThreads = 1024;
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

__global__ void __launch_bounds__(kPgSelThreads) paged_evict_select_kernel(const PgEvictParams p)
{
    extern __shared__ uint32_t s_keys[];
    __shared__ uint32_t hist[256];
    __shared__ uint32_t s_prefix, s_need;
    __shared__ int w_keep[32], w_tie[32];
    const int r = blockIdx.y, h = blockIdx.x;
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int n = p.lens[r];
    const int* table = p.table + (size_t)r * p.max_pages;
    int* kept = p.kept + ((size_t)r * p.H + h) * p.budget;
    bool bad = !pg_evict_len_ok(p, n);
    if (!bad)
        for (int i = tid; i < (n + p.ps - 1) / p.ps; i += kPgSelThreads) {
            const int page = table[i];
            bad |= page < 0 || page >= p.S;
        }
    if (__syncthreads_or(bad)) {
        // nothing moves; the caller sees no kept row and a length of -1
        for (int i = tid; i < p.budget; i += kPgSelThreads) kept[i] = -1;
        if (tid == 0) {
            report(p.status, (int)UNIPIN_ERR_OUT_OF_RANGE);
            if (h == 0) p.new_lens[r] = -1;
        }
        return;
    }
    if (tid == 0 && h == 0) p.new_lens[r] = min(n, p.budget);
    if (n <= p.budget) {
        for (int i = tid; i < p.budget; i += kPgSelThreads) kept[i] = i < n ? i : -1;
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
        for (int i = tid; i < mid; i += kPgSelThreads) s_keys[i] = pg_order_key(*slot(m0 + i));
    uint32_t prefix = 0, mask = 0;
    if (need > 0) {
        for (int shift = 24; shift >= 0; shift -= 8) {
            for (int i = tid; i < 256; i += kPgSelThreads) hist[i] = 0;
            __syncthreads();
            for (int i = tid; i < mid; i += kPgSelThreads) {
                const uint32_t x = key(i);
                if ((x & mask) == prefix) atomicAdd(&hist[(x >> shift) & 255u], 1u);
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
    }
    // every key above `prefix` stays, and the first `need` rows whose key equals it
    const bool any = p.budget - p.n_sinks - p.n_recent > 0;
    uint32_t ties = 0;       // ties seen before this step
    int at = 0;              // rows kept before this step
    __syncthreads();
    for (int j0 = 0; j0 < n; j0 += kPgSelThreads) {
        const int j = j0 + tid;
        bool keep = false, tie = false;
        float w = 0.f;
        if (j < n) {
            w = *slot(j);
            if (j < m0 || j >= n - p.n_recent) {
                keep = true;
            } else if (any) {
                const uint32_t x = pg_order_key(w);
                keep = x > prefix;
                tie = x == prefix;
            }
        }
        const uint32_t tb = __ballot_sync(0xffffffffu, tie);
        if (lane == 0) w_tie[warp] = __popc(tb);
        __syncthreads();
        int tbase = (int)ties, tall = 0;
        for (int x = 0; x < 32; ++x) {
            const int c = w_tie[x];
            if (x < warp) tbase += c;
            tall += c;
        }
        if (tie && (uint32_t)(tbase + __popc(tb & ((1u << lane) - 1u))) < need) keep = true;
        const uint32_t kb = __ballot_sync(0xffffffffu, keep);
        if (lane == 0) w_keep[warp] = __popc(kb);
        __syncthreads();       // also: every load of this step precedes its stores
        int kbase = at, kall = 0;
        for (int x = 0; x < 32; ++x) {
            const int c = w_keep[x];
            if (x < warp) kbase += c;
            kall += c;
        }
        if (keep) {
            const int i = kbase + __popc(kb & ((1u << lane) - 1u));
            kept[i] = j;
            if (i != j) *slot(i) = w;
        }
        ties += (uint32_t)tall;
        at += kall;
        // the next step's ballot counts overwrite w_tie only after every thread has read them
        // (the barrier above), and w_keep after the next step's first barrier
    }
}

// kVec: 16-byte vectors of a row slice.  Grid (2 x slices, H, R): K's slices, then V's.
template <int kVec>
__global__ void __launch_bounds__(kPgMoveThreads) paged_evict_move_kernel(const PgEvictParams p)
{
    constexpr int kRowsStep = kPgMoveThreads / kVec;
    constexpr int kUnroll = 4;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int r = blockIdx.z, h = blockIdx.y;
    const int n = p.lens[r];
    if (p.new_lens[r] < 0 || n <= p.budget) return;
    const int slices = gridDim.x / 2;
    uint8_t* pool = blockIdx.x < (unsigned)slices ? p.pool_k : p.pool_v;
    const int slice = blockIdx.x % slices;
    const int* table = p.table + (size_t)r * p.max_pages;
    const int* kept = p.kept + ((size_t)r * p.H + h) * p.budget;
    const int c = threadIdx.x % kVec, row = threadIdx.x / kVec;
    const size_t col = ((size_t)slice * kVec + c) * 16;
    auto addr = [&](int j) -> uint4* {
        const int pg = p.page_of(j);
        const size_t at = ((size_t)__ldg(table + pg) * p.H + h) * p.ps + (j - pg * p.ps);
        return reinterpret_cast<uint4*>(pool + at * p.row_bytes + col);
    };
    for (int i0 = 0; i0 < p.budget; i0 += kRowsStep * kUnroll) {
        uint4 x[kUnroll];
        bool move[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int i = i0 + u * kRowsStep + row;
            const int j = i < p.budget ? kept[i] : i;
            move[u] = j != i;
            if (move[u]) x[u] = *addr(j);
        }
        __syncthreads();       // every load of the step precedes its stores
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
            if (move[u]) *addr(i0 + u * kRowsStep + row) = x[u];
    }
}

}  // namespace unipin
