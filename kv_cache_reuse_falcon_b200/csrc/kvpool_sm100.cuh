// Pool write: copies the past K/V rows of each segment from the packed
// token-major layout [T, H, D] into the head-major pool [L, S, H, n_cap, D]
// at the segment's slot ([review] §2.4: retrieval writes the history K/V into
// the shared pool; [notes] §6: pool shape [L, S, H, n, D]).
//
// Memory-bound byte copy.  Each thread moves 16-byte vectors; consecutive
// threads walk one pool row after another, so the pool side (the write) is
// fully contiguous and each token-major source row is read as whole 32-byte
// sectors.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>

#include "e4m3.cuh"
#include "unipin.h"

namespace unipin {

struct PoolWriteParams {
    const uint4* k;        // [T, H, D] bf16 viewed as 16-byte vectors
    const uint4* v;
    uint4* pool_k;         // [L, S, H, n_cap, D]
    uint4* pool_v;
    const int* cu;
    const int* past;
    const int* slots;
    int H, D, S, n_cap, layer;
    int total_tokens;      // T
    int* status;
};

__global__ void __launch_bounds__(256) kvpool_write_kernel(const PoolWriteParams p)
{
    const int b = blockIdx.z;
    const int h = blockIdx.y;
    const int n = p.past[b];
    const int slot = p.slots[b];
    const int start = p.cu[b];
    const int len = p.cu[b + 1] - start;
    if (n < 0 || n > p.n_cap || n > len || slot < 0 || slot >= p.S || start < 0 ||
        (long long)start + n > (long long)p.total_tokens) {
        if (threadIdx.x == 0 && blockIdx.x == 0 && p.status) atomicCAS(p.status, 0, (int)UNIPIN_ERR_OUT_OF_RANGE);
        return;
    }
    const int vpr = p.D / 8;   // 16-byte vectors per row
    const long long total = (long long)n * vpr;
    const long long src_row0 = (long long)start * p.H + h;                                  // in rows of D
    const long long dst_row0 = (((long long)p.layer * p.S + slot) * p.H + h) * (long long)p.n_cap;
    for (long long idx = (long long)blockIdx.x * blockDim.x + threadIdx.x; idx < total;
         idx += (long long)gridDim.x * blockDim.x) {
        const long long j = idx / vpr;
        const int c = (int)(idx - j * vpr);
        const long long src = (src_row0 + j * p.H) * vpr + c;
        const long long dst = (dst_row0 + j) * vpr + c;
        const uint4 kv = __ldg(p.k + src);
        const uint4 vv = __ldg(p.v + src);
        p.pool_k[dst] = kv;
        p.pool_v[dst] = vv;
    }
}

// E4M3 pools (conversions in e4m3.cuh).

struct PoolWriteE4M3Params {
    const uint4* k;        // [T, H, D] bf16 viewed as 16-byte vectors
    const uint4* v;
    uint2* pool_k;         // [L, S, H, n_cap, D] E4M3 codes viewed as 8-byte vectors
    uint2* pool_v;
    const int* cu;
    const int* past;
    const int* slots;
    int H, D, S, n_cap, layer;
    int total_tokens;
    float inv_k, inv_v;    // float32 reciprocals of the pool's scales
    int* status;
};

// The rows and grid of kvpool_write_kernel; each thread turns 8 elements into 8 codes.
__global__ void __launch_bounds__(256) kvpool_write_e4m3_kernel(const PoolWriteE4M3Params p)
{
    const int b = blockIdx.z;
    const int h = blockIdx.y;
    const int n = p.past[b];
    const int slot = p.slots[b];
    const int start = p.cu[b];
    const int len = p.cu[b + 1] - start;
    if (n < 0 || n > p.n_cap || n > len || slot < 0 || slot >= p.S || start < 0 ||
        (long long)start + n > (long long)p.total_tokens) {
        if (threadIdx.x == 0 && blockIdx.x == 0 && p.status) atomicCAS(p.status, 0, (int)UNIPIN_ERR_OUT_OF_RANGE);
        return;
    }
    const int vpr = p.D / 8;
    const long long total = (long long)n * vpr;
    const long long src_row0 = (long long)start * p.H + h;
    const long long dst_row0 = (((long long)p.layer * p.S + slot) * p.H + h) * (long long)p.n_cap;
    for (long long idx = (long long)blockIdx.x * blockDim.x + threadIdx.x; idx < total;
         idx += (long long)gridDim.x * blockDim.x) {
        const long long j = idx / vpr;
        const int c = (int)(idx - j * vpr);
        const long long src = (src_row0 + j * p.H) * vpr + c;
        const long long dst = (dst_row0 + j) * vpr + c;
        p.pool_k[dst] = e4m3x8_from_bf16(__ldg(p.k + src), p.inv_k);
        p.pool_v[dst] = e4m3x8_from_bf16(__ldg(p.v + src), p.inv_v);
    }
}

struct PoolDequantParams {
    const uint2* pool_k;   // [L, S, H, n_cap, D] E4M3 codes viewed as 8-byte vectors
    const uint2* pool_v;
    uint4* out_k;          // [R, H, n_cap, D] bfloat16 viewed as 16-byte vectors: a pool with L = 1, S = R
    uint4* out_v;
    int* out_slots;        // [R]: r, or -1 where request r's slot or length is out of range
    const int* past;
    const int* slots;
    int H, D, S, n_cap, layer;
    float k_scale, v_scale;
};

// Rows 0..n_r-1 of request r's slot (layer `layer`, every head) expanded into
// slot r of a bfloat16 pool; the rank decode then reads that pool.  Grid:
// (row-vector chunks, H, R).
__global__ void __launch_bounds__(256) kvpool_dequant_kernel(const PoolDequantParams p)
{
    const int r = blockIdx.z;
    const int h = blockIdx.y;
    const int n = p.past[r];
    const int slot = p.slots[r];
    const bool ok = slot >= 0 && slot < p.S && n >= 0 && n <= p.n_cap;
    if (blockIdx.x == 0 && h == 0 && threadIdx.x == 0) p.out_slots[r] = ok ? r : -1;
    if (!ok) return;   // the decode rejects the request (zero rows, status)
    const int vpr = p.D / 8;
    const long long total = (long long)n * vpr;
    const long long src_row0 = (((long long)p.layer * p.S + slot) * p.H + h) * (long long)p.n_cap;
    const long long dst_row0 = ((long long)r * p.H + h) * (long long)p.n_cap;
    for (long long idx = (long long)blockIdx.x * blockDim.x + threadIdx.x; idx < total;
         idx += (long long)gridDim.x * blockDim.x) {
        const long long j = idx / vpr;
        const int c = (int)(idx - j * vpr);
        const long long src = (src_row0 + j) * vpr + c;
        const long long dst = (dst_row0 + j) * vpr + c;
        p.out_k[dst] = bf16x8_from_e4m3(__ldg(p.pool_k + src), p.k_scale);
        p.out_v[dst] = bf16x8_from_e4m3(__ldg(p.pool_v + src), p.v_scale);
    }
}

}  // namespace unipin
