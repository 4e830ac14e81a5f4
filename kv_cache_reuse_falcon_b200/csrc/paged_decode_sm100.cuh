// One new token per request over a paged KV pool, split over the cache's
// length and joined.
//
// A paged pool is a unipin_kvpool whose slots are pages: [L, S pages, H_kv,
// n_cap rows of a page, D].  Row j of request r lies in page
// page_table[r][j / n_cap] at offset j % n_cap.  With pos the new token's
// position (n_r when its own key is passed apart, n_r - 1 when it is the last
// cached row) the token sees the cached rows
//   j < n_r  with  pos - j < window  or  j < n_sinks,
// i.e. the rows [0, ns) and [lo, n_r), lo = max(0, pos - window + 1), ns =
// min(n_sinks, lo): "visible rows" v = 0 .. vis - 1 below, in that order.
//   o_h = sum_v softmax_v(scale q_h . k_v) v_v       (and its own key, if any)
//   key_weights[row v] += sum over the group's heads of the weight of v.
//
// Bound: memory.  Each visible K and V row is read once for the G query heads
// that share it: 2 D elements for 4 D G flops.  So the kernel is built around
// loads in flight, not around the tensor cores:
//   - a work item is (request, key/value head, 16 query heads of the group,
//     chunk of visible rows); a warp takes every fourth tile of 16 rows of its
//     block's chunk on its own, with no barrier in its loop;
//   - each lane copies with cp.async exactly the bytes its MMA fragments need
//     into its own slots of a ring of stages and reads them back itself, so the
//     ring needs no barrier, no swizzle and no padding (lane-contiguous 16-byte
//     slots), works for any page size, and a page that ends inside a tile costs
//     nothing;
//   - S = Q K^T by mma.m16n8k16 with the query heads as M (16, or 8 used) and
//     eight keys as N.  The sum over d may be taken in any order, so lane (g, t)
//     takes consecutive elements of key g as its share of the K index and Q is
//     loaded in the same order: no shuffle, no ldmatrix;
//   - O += P V the same way: P's fragment is S's accumulator layout; lane (g, t)
//     holds consecutive elements of the value rows 2t, 2t+1, 2t+8, 2t+9, and a
//     byte permute pairs two rows per register.
// mma.sync and not tcgen05: at 16 query rows or fewer per key the tensor work is
// under a tenth of the tensor cores' rate at the full memory rate, and a TMEM
// accumulator would put a chain of barriers (load, S, softmax, P, P.V) into
// every tile.
// Scores, row maxima, row sums and O are float32.  P is rounded to the type of
// V's fragment (bfloat16; float16 over E4M3 codes), as in the prefill: one
// rounding of relative size <= 2^-8 (2^-11) per weight, independent of the others.
//
// E4M3 pools: attention reads code c as bf16(value(c) * scale).  Where both
// scales are powers of two that is value(c) * scale exactly, so the codes go to
// the tensor cores as float16 (exact), the scales are applied to the scores and
// to O, and q goes to float16 after a power-of-two scaling of its row that puts
// the row's largest element into [2^9, 2^10): bfloat16 has 8 significant bits,
// float16 11, so only elements below 2^-33 of the row's largest can lose bits.
// Other scales take the float32 product and its rounding to bfloat16 per element.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "e4m3.cuh"
#include "sm100_ptx.cuh"
#include "unipin.h"

namespace unipin {

constexpr int kPgWarps = 4;
constexpr int kPgThreads = 32 * kPgWarps;
constexpr int kPgKeys = 16;                      // rows of a warp's tile
constexpr int kPgSpan = kPgWarps * kPgKeys;      // rows a block takes per step
constexpr float kPgLog2e = 1.4426950408889634f;
constexpr float kPgRescaleLog2 = 8.0f;           // O is rescaled only when a row max grows by > 2^8

enum PgMode { kPgBf16 = 0, kPgE4M3Pow2 = 1, kPgE4M3Any = 2 };

template <int D, int kMode>
struct PgCfg {
    static constexpr int kElt = kMode == kPgBf16 ? 2 : 1;
    static constexpr int kRowBytes = D * kElt;
    // a lane's share of a K row (a quarter) and of a V row (an eighth), in pieces of at most 16 bytes
    static constexpr int kKB = kRowBytes / 4 < 16 ? kRowBytes / 4 : 16;
    static constexpr int kKPieces = kRowBytes / 4 / kKB;
    static constexpr int kKElems = kKB / kElt;
    static constexpr int kVB = kRowBytes / 8 < 16 ? kRowBytes / 8 : 16;
    static constexpr int kVPieces = kRowBytes / 8 / kVB;
    static constexpr int kVElems = kVB / kElt;
    static constexpr int kStageBytes = 32 * kRowBytes;      // K and V of 16 rows
    // Enough bytes in flight per SM for the memory latency (about 64 KB): 2 blocks of 4 warps
    // at the widest row, more blocks at narrower ones.
    static constexpr int kStages = kRowBytes >= 256 ? 3 : 4;
    static constexpr int kRingBytes = kPgWarps * kStages * kStageBytes;
    static constexpr int kJoinBytes = kPgWarps * 16 * (D + 2) * 4;   // the warps' O, m, l at the end
    static constexpr int kSmemBytes = kRingBytes > kJoinBytes ? kRingBytes : kJoinBytes;
};

struct PgParams {
    const __nv_bfloat16* q;        // [R, H, D]
    const __nv_bfloat16* k_self;   // [R, H_kv, D] or null
    const __nv_bfloat16* v_self;
    const uint8_t* pool_k;         // the layer's planes: [S, H_kv, ps, D]
    const uint8_t* pool_v;
    const int* table;              // [R, max_pages]
    const int* lens;               // [R]
    void* out;                     // [R, H, D]
    float* key_weights;            // the layer's [S, H_kv, ps] or null
    float* part_o;                 // [R * H, nsplit, D]
    float* part_ml;                // [R * H, nsplit, 2]: (m in log2 units, l); l = -1: rejected
    float* scores;                 // [R * H, vmax] log2-unit scores of the visible rows (key_weights)
    int R, H, Hkv, G, S, ps, max_pages, max_len;
    int window, n_sinks;
    int chunk, nsplit, vmax;
    int out_fp32;
    float sl2;                     // scale * log2(e), times k_scale over power-of-two E4M3 pools
    float sl2_self;                // scale * log2(e)
    float k_scale, v_scale;        // E4M3
    int* status;
};

// The visible rows of request r.
struct PgRows {
    int n, ns, lo, vis;
    bool ok;
    __device__ int row(int v) const { return v < ns ? v : v - ns + lo; }
};

__device__ __forceinline__ PgRows pg_rows(const PgParams& p, int r)
{
    PgRows x;
    x.n = p.lens[r];
    x.ok = x.n >= 0 && x.n <= p.max_len && (long long)x.n <= (long long)p.max_pages * p.ps;
    const int pos = p.k_self ? x.n : x.n - 1;
    x.lo = pos - p.window + 1;                 // window >= 1, so no overflow
    if (x.lo < 0) x.lo = 0;
    x.ns = min(p.n_sinks, x.lo);
    x.vis = x.ok ? x.ns + x.n - x.lo : 0;
    return x;
}

template <int kBytes>
__device__ __forceinline__ void pg_copy(uint32_t dst, const void* src, bool live)
{
    const int n = live ? kBytes : 0;           // 0: the slot is filled with zeros
    if constexpr (kBytes == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(kBytes), "r"(n)
                     : "memory");
}

__device__ __forceinline__ void pg_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

template <int N>
__device__ __forceinline__ void pg_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// N bytes of this lane's slot into 32-bit registers.
template <int kBytes>
__device__ __forceinline__ void pg_read(uint32_t addr, uint32_t* r)
{
    if constexpr (kBytes == 16)
        asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
    else if constexpr (kBytes == 8)
        asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "r"(addr) : "memory");
    else
        asm volatile("ld.shared.b32 %0, [%1];" : "=r"(r[0]) : "r"(addr) : "memory");
}

// D (16 x 8, f32) += A (16 x 16) B (16 x 8); bfloat16 or float16 operands.
template <bool kHalf>
__device__ __forceinline__ void pg_mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                       uint32_t b1)
{
    if constexpr (kHalf)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                     "{%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                     "{%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pg_prmt(uint32_t a, uint32_t b, uint32_t sel)
{
    return __byte_perm(a, b, sel);
}

// Two E4M3 codes (the low two bytes) as float16 pair: exact.
__device__ __forceinline__ uint32_t pg_half2_from_e4m3(uint32_t codes)
{
    uint32_t h2;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"((uint16_t)codes));
    return h2;
}

// Two E4M3 codes as the bfloat16 pair attention reads: bf16(value * scale).
__device__ __forceinline__ uint32_t pg_bf2_from_e4m3(uint32_t codes, float scale)
{
    const uint32_t h2 = pg_half2_from_e4m3(codes);
    const __half2 h = *reinterpret_cast<const __half2*>(&h2);
    return pack_bf16x2(__fmul_rn(__low2float(h), scale), __fmul_rn(__high2float(h), scale));
}

template <int kMode>
__device__ __forceinline__ uint32_t pg_expand(uint32_t codes, float scale)
{
    return kMode == kPgE4M3Pow2 ? pg_half2_from_e4m3(codes) : pg_bf2_from_e4m3(codes, scale);
}

__device__ __forceinline__ uint32_t pg_pack_p(float lo, float hi, bool half)
{
    if (half) {
        const __half2 h = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
    return pack_bf16x2(lo, hi);
}

// Lane `lane` of a warp owns elements lane * E .. of a row of D: stores them as fp32 or bf16.
template <int E>
__device__ __forceinline__ void pg_store_row(void* out, int out_fp32, size_t at, const float (&o)[E])
{
    if (out_fp32) {
        float* dst = static_cast<float*>(out) + at;
        if constexpr (E == 4) *reinterpret_cast<float4*>(dst) = make_float4(o[0], o[1], o[2], o[3]);
        else if constexpr (E == 2) *reinterpret_cast<float2*>(dst) = make_float2(o[0], o[1]);
        else dst[0] = o[0];
    } else {
        __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(out) + at;
        if constexpr (E == 4)
            *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]));
        else if constexpr (E == 2) *reinterpret_cast<uint32_t*>(dst) = pack_bf16x2(o[0], o[1]);
        else dst[0] = __float2bfloat16_rn(o[0]);
    }
}

// q . k_self in log2 units of query row (r, h); every lane gets it.
template <int D>
__device__ __forceinline__ float pg_self_score(const PgParams& p, int r, int h, int lane)
{
    constexpr int E = D / 32;
    const __nv_bfloat16* q = p.q + ((size_t)r * p.H + h) * D + lane * E;
    const __nv_bfloat16* k = p.k_self + ((size_t)r * p.Hkv + h / p.G) * D + lane * E;
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) s = fmaf(__bfloat162float(q[e]), __bfloat162float(k[e]), s);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
    return s * p.sl2_self;
}

// One warp finishes query row (r, h): o (this lane's elements, relative to m) and l of the cached
// rows, the own key merged in, divided and stored.  A row that sees nothing is zeros.
template <int D>
__device__ __forceinline__ void pg_finish_row(const PgParams& p, int r, int h, int lane, float m, float l,
                                              float (&o)[D / 32])
{
    constexpr int E = D / 32;
    float a = 1.f, b = 0.f;
    if (p.k_self) {
        const float ss = pg_self_score<D>(p, r, h, lane);
        const float mf = fmaxf(m, ss);
        a = m == -INFINITY ? 0.f : ex2_approx(m - mf);
        b = ss == -INFINITY ? 0.f : ex2_approx(ss - mf);
        if (ss != ss) b = ss;                 // a NaN score makes the row NaN
    }
    const float total = l * a + b;
    const float inv = total == 0.f ? 0.f : 1.f / total;
    float res[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
        float x = a == 0.f ? 0.f : o[e] * a;
        if (b != 0.f)
            x = fmaf(b, __bfloat162float(p.v_self[((size_t)r * p.Hkv + h / p.G) * D + lane * E + e]), x);
        res[e] = x * inv;
    }
    pg_store_row<E>(p.out, p.out_fp32, ((size_t)r * p.H + h) * D + lane * E, res);
}

template <int D>
__device__ __forceinline__ void pg_zero_row(const PgParams& p, int r, int h, int lane)
{
    float z[D / 32];
#pragma unroll
    for (int e = 0; e < D / 32; ++e) z[e] = 0.f;
    pg_store_row<D / 32>(p.out, p.out_fp32, ((size_t)r * p.H + h) * D + lane * (D / 32), z);
}

// Grid (nsplit, H_kv * column groups, R).  kWide: the block's query heads may be more than 8 (rows 8..15
// of the MMA carry heads too).
template <int D, int kMode, bool kWide>
__global__ void __launch_bounds__(kPgThreads) paged_decode_kernel(const PgParams p)
{
    using C = PgCfg<D, kMode>;
    constexpr bool kHalf = kMode == kPgE4M3Pow2;
    constexpr int NT = D / 8;                       // n-tiles of O
    extern __shared__ __align__(16) uint8_t smem[];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int g = lane / 4, t = lane % 4;
    const int r = blockIdx.z;
    const int groups = (p.G + 15) / 16;
    const int hkv = blockIdx.y / groups;
    const int cg = blockIdx.y - hkv * groups;
    const int h0 = hkv * p.G + cg * 16;             // first query head of the block
    const int nh = min(16, p.G - cg * 16);
    const PgRows rows = pg_rows(p, r);
    const bool split = p.part_ml != nullptr;
    const int v0 = blockIdx.x * p.chunk;
    if (v0 >= rows.vis && (split || blockIdx.x > 0) && rows.ok) return;   // the join asks for chunks < vis only
    if (!rows.ok && blockIdx.x > 0) return;
    const int v1 = min(v0 + p.chunk, rows.vis);
    bool bad = !rows.ok;

    // ---- Q fragments: row g (and g + 8), in the order the K fragments take d
    constexpr int QP = C::kKElems / 2;              // pairs per K piece
    uint32_t qa[C::kKPieces][QP], qb[kWide ? C::kKPieces : 1][QP];
    float fac0 = p.sl2, fac1 = p.sl2;               // score factor of rows g and g + 8
    {
        const __nv_bfloat16* q0 = p.q + ((size_t)r * p.H + h0 + g) * D;
        const __nv_bfloat16* q1 = q0 + 8 * (size_t)D;
#pragma unroll
        for (int c = 0; c < C::kKPieces; ++c)
#pragma unroll
            for (int i = 0; i < QP; ++i) {
                const int d = (c * 4 + t) * C::kKElems + 2 * i;
                qa[c][i] = g < nh ? *reinterpret_cast<const uint32_t*>(q0 + d) : 0u;
                if (kWide) qb[c][i] = g + 8 < nh ? *reinterpret_cast<const uint32_t*>(q1 + d) : 0u;
            }
        if constexpr (kHalf) {
            auto to_half = [&](auto& qq, float& fac) {
                float top = 0.f;
#pragma unroll
                for (int c = 0; c < C::kKPieces; ++c)
#pragma unroll
                    for (int i = 0; i < QP; ++i) {
                        top = fmaxf(top, fabsf(__uint_as_float(qq[c][i] << 16)));
                        top = fmaxf(top, fabsf(__uint_as_float(qq[c][i] & 0xffff0000u)));
                    }
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                int e = (int)((__float_as_uint(top) >> 23) & 255) - 127;   // top in [2^e, 2^(e+1))
                if (top == 0.f || e == 128) e = 9;
                e = max(e, -100);                                          // keeps both powers finite
                const float up = __uint_as_float((uint32_t)(9 - e + 127) << 23);   // 2^(9-e), 9-e in [-118, 109]
#pragma unroll
                for (int c = 0; c < C::kKPieces; ++c)
#pragma unroll
                    for (int i = 0; i < QP; ++i) {
                        const __half2 h = __floats2half2_rn(__uint_as_float(qq[c][i] << 16) * up,
                                                            __uint_as_float(qq[c][i] & 0xffff0000u) * up);
                        qq[c][i] = *reinterpret_cast<const uint32_t*>(&h);
                    }
                fac *= __uint_as_float((uint32_t)(e - 9 + 127) << 23);
            };
            to_half(qa, fac0);
            if (kWide) to_half(qb, fac1);
        }
    }

    float o[NT][4];
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;

    const uint32_t ring = smem_u32(smem) + warp * C::kStages * C::kStageBytes;
    const int ntile = rows.ok && v1 > v0 ? (v1 - v0 + kPgSpan - 1 - warp * kPgKeys) / kPgSpan : 0;   // this warp's tiles
    const int* table = p.table + (size_t)r * p.max_pages;
    const uint32_t last = (uint32_t)p.S * p.Hkv * (uint32_t)p.ps;   // rows of the layer (host: fits 32 bits)

    // lane's key of tile i: its row in the layer's plane, or `last` where there is none
    auto key_row = [&](int i) -> uint32_t {
        const int v = v0 + i * kPgSpan + warp * kPgKeys + (lane & 15);
        if (i >= ntile || v >= v1) return last;
        const int j = rows.row(v);
        const int pg = j / p.ps;
        const int page = __ldg(table + pg);
        if (page < 0 || page >= p.S) {
            bad = true;
            return last;
        }
        return ((uint32_t)page * p.Hkv + hkv) * (uint32_t)p.ps + (uint32_t)(j - pg * p.ps);
    };
    auto issue = [&](int i, uint32_t row) {
        const uint32_t st = ring + (i % C::kStages) * C::kStageBytes;
#pragma unroll
        for (int x = 0; x < 2; ++x) {               // K rows g, g + 8
            const uint32_t kr = __shfl_sync(0xffffffffu, row, g + 8 * x);
            const uint8_t* src = p.pool_k + (size_t)(kr < last ? kr : 0u) * C::kRowBytes + t * C::kKB;
#pragma unroll
            for (int c = 0; c < C::kKPieces; ++c)
                pg_copy<C::kKB>(st + (x * C::kKPieces + c) * 32 * C::kKB + lane * C::kKB, src + c * 4 * C::kKB,
                                kr < last);
        }
        const uint32_t sv = st + 2 * C::kKPieces * 32 * C::kKB;
#pragma unroll
        for (int x = 0; x < 4; ++x) {               // V rows 2t, 2t + 1, 2t + 8, 2t + 9
            const uint32_t vr = __shfl_sync(0xffffffffu, row, 2 * t + (x & 1) + 8 * (x >> 1));
            const uint8_t* src = p.pool_v + (size_t)(vr < last ? vr : 0u) * C::kRowBytes + g * C::kVB;
#pragma unroll
            for (int c = 0; c < C::kVPieces; ++c)
                pg_copy<C::kVB>(sv + (x * C::kVPieces + c) * 32 * C::kVB + lane * C::kVB, src + c * 8 * C::kVB,
                                vr < last);
        }
    };

#pragma unroll
    for (int i = 0; i < C::kStages - 1; ++i) {
        issue(i, key_row(i));
        pg_commit();
    }
    uint32_t next_row = key_row(C::kStages - 1);
    for (int i = 0; i < ntile; ++i) {
        pg_wait<C::kStages - 2>();                  // tile i has landed (this lane's own copies)
        issue(i + C::kStages - 1, next_row);        // into the stage that tile i - 1 has left
        pg_commit();
        next_row = key_row(i + C::kStages);         // its page lookup overlaps this tile's work
        const uint32_t st = ring + (i % C::kStages) * C::kStageBytes;
        float s[2][4];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            uint32_t kf[C::kKPieces][C::kKB / 4];
#pragma unroll
            for (int c = 0; c < C::kKPieces; ++c)
                pg_read<C::kKB>(st + (x * C::kKPieces + c) * 32 * C::kKB + lane * C::kKB, kf[c]);
#pragma unroll
            for (int e = 0; e < 4; ++e) s[x][e] = 0.f;
#pragma unroll
            for (int c = 0; c < C::kKPieces; ++c)
#pragma unroll
                for (int i2 = 0; i2 < QP; i2 += 2) {
                    uint32_t b0, b1;
                    if constexpr (kMode == kPgBf16) {
                        b0 = kf[c][i2];
                        b1 = kf[c][i2 + 1];
                    } else {                        // four codes per register
                        b0 = pg_expand<kMode>(kf[c][i2 / 2], p.k_scale);
                        b1 = pg_expand<kMode>(kf[c][i2 / 2] >> 16, p.k_scale);
                    }
                    pg_mma<kHalf>(s[x], qa[c][i2], kWide ? qb[c][i2] : 0u, qa[c][i2 + 1], kWide ? qb[c][i2 + 1] : 0u,
                                  b0, b1);
                }
        }
        const int vt = v0 + i * kPgSpan + warp * kPgKeys;   // visible index of the tile's first key
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            s[x][0] *= fac0;
            s[x][1] *= fac0;
            s[x][2] *= fac1;
            s[x][3] *= fac1;
        }
        if (p.scores) {
            // rows g (and g + 8) of the group's scores, two keys per lane
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const int v = vt + 8 * x + 2 * t;
#pragma unroll
                for (int half = 0; half < (kWide ? 2 : 1); ++half) {
                    if (g + 8 * half >= nh) continue;
                    float* dst = p.scores + ((size_t)r * p.H + h0 + g + 8 * half) * p.vmax + v;
                    if (v + 1 < v1) *reinterpret_cast<float2*>(dst) = make_float2(s[x][2 * half], s[x][2 * half + 1]);
                    else if (v < v1) *dst = s[x][2 * half];
                }
            }
        }
        if (vt + kPgKeys > v1) {                    // the chunk ends inside the tile
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (vt + 8 * x + 2 * t + (e & 1) >= v1) s[x][e] = -INFINITY;
        }
        float t0 = fmaxf(fmaxf(s[0][0], s[0][1]), fmaxf(s[1][0], s[1][1]));
        float t1 = kWide ? fmaxf(fmaxf(s[0][2], s[0][3]), fmaxf(s[1][2], s[1][3])) : -INFINITY;
        if (__any_sync(0xffffffffu, t0 > m0 + kPgRescaleLog2 || t1 > m1 + kPgRescaleLog2)) {
            t0 = fmaxf(t0, __shfl_xor_sync(0xffffffffu, t0, 1));
            t0 = fmaxf(t0, __shfl_xor_sync(0xffffffffu, t0, 2));
            const float n0 = fmaxf(m0, t0);
            const float c0 = m0 == -INFINITY ? 0.f : ex2_approx(m0 - n0);
            m0 = n0;
            l0 *= c0;
            float c1 = 0.f;
            if (kWide) {
                t1 = fmaxf(t1, __shfl_xor_sync(0xffffffffu, t1, 1));
                t1 = fmaxf(t1, __shfl_xor_sync(0xffffffffu, t1, 2));
                const float n1 = fmaxf(m1, t1);
                c1 = m1 == -INFINITY ? 0.f : ex2_approx(m1 - n1);
                m1 = n1;
                l1 *= c1;
            }
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                o[j][0] *= c0;
                o[j][1] *= c0;
                if (kWide) {
                    o[j][2] *= c1;
                    o[j][3] *= c1;
                }
            }
        }
        const float u0 = m0 == -INFINITY ? 0.f : m0, u1 = m1 == -INFINITY ? 0.f : m1;
        uint32_t pa[2], pb[2] = {0u, 0u};
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const float e0 = ex2_approx(s[x][0] - u0), e1 = ex2_approx(s[x][1] - u0);
            l0 += e0 + e1;
            pa[x] = pg_pack_p(e0, e1, kHalf);
            if (kWide) {
                const float e2 = ex2_approx(s[x][2] - u1), e3 = ex2_approx(s[x][3] - u1);
                l1 += e2 + e3;
                pb[x] = pg_pack_p(e2, e3, kHalf);
            }
        }
        // ---- O += P V: element j of the lane's share of rows 2t, 2t+1 (b0) and 2t+8, 2t+9 (b1)
        const uint32_t sv = st + 2 * C::kKPieces * 32 * C::kKB;
#pragma unroll
        for (int c = 0; c < C::kVPieces; ++c) {
            uint32_t vf[4][C::kVB / 4];
#pragma unroll
            for (int x = 0; x < 4; ++x)
                pg_read<C::kVB>(sv + (x * C::kVPieces + c) * 32 * C::kVB + lane * C::kVB, vf[x]);
            if constexpr (kMode == kPgBf16) {
#pragma unroll
                for (int j = 0; j < C::kVElems; ++j) {
                    const uint32_t sel = (j & 1) ? 0x7632u : 0x5410u;
                    pg_mma<kHalf>(o[c * C::kVElems + j], pa[0], pb[0], pa[1], pb[1],
                                  pg_prmt(vf[0][j / 2], vf[1][j / 2], sel), pg_prmt(vf[2][j / 2], vf[3][j / 2], sel));
                }
            } else {
#pragma unroll
                for (int j = 0; j < C::kVElems; j += 2) {
                    // bytes (row a [j], row b [j], row a [j+1], row b [j+1])
                    const uint32_t sel = (j & 2) ? 0x7362u : 0x5140u;
                    const uint32_t lo = pg_prmt(vf[0][j / 4], vf[1][j / 4], sel);
                    const uint32_t hi = pg_prmt(vf[2][j / 4], vf[3][j / 4], sel);
                    pg_mma<kHalf>(o[c * C::kVElems + j], pa[0], pb[0], pa[1], pb[1],
                                  pg_expand<kMode>(lo, p.v_scale), pg_expand<kMode>(hi, p.v_scale));
                    pg_mma<kHalf>(o[c * C::kVElems + j + 1], pa[0], pb[0], pa[1], pb[1],
                                  pg_expand<kMode>(lo >> 16, p.v_scale), pg_expand<kMode>(hi >> 16, p.v_scale));
                }
            }
        }
    }
    pg_wait<0>();
    l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
    l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
    if (kWide) {
        l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
        l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
    }

    // ---- the four warps' O, m, l joined through shared memory
    bad = __syncthreads_or(bad);                     // every warp has left its ring
    if (bad && threadIdx.x == 0) report(p.status, (int)UNIPIN_ERR_OUT_OF_RANGE);
    float* so = reinterpret_cast<float*>(smem);      // [warp][16][D]
    float* sml = so + kPgWarps * 16 * D;             // [warp][16][2]
    const float vs = kMode == kPgE4M3Pow2 ? p.v_scale : 1.f;
#pragma unroll
    for (int half = 0; half < (kWide ? 2 : 1); ++half) {
        float* dst = so + (warp * 16 + g + 8 * half) * D;
#pragma unroll
        for (int c = 0; c < C::kVPieces; ++c)
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int j = 0; j < C::kVElems; ++j)
                    dst[(c * 8 + 2 * t + e) * C::kVElems + j] = o[c * C::kVElems + j][2 * half + e] * vs;
        if (t == 0) {
            sml[(warp * 16 + g + 8 * half) * 2] = half ? m1 : m0;
            sml[(warp * 16 + g + 8 * half) * 2 + 1] = half ? l1 : l0;
        }
    }
    __syncthreads();
    constexpr int E = D / 32;
    for (int row = warp; row < nh; row += kPgWarps) {
        const int h = h0 + row;
        float m = -INFINITY, l = 0.f, acc[E];
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = 0.f;
#pragma unroll
        for (int w = 0; w < kPgWarps; ++w) m = fmaxf(m, sml[(w * 16 + row) * 2]);
#pragma unroll
        for (int w = 0; w < kPgWarps; ++w) {
            const float mw = sml[(w * 16 + row) * 2];
            const float f = mw == -INFINITY ? 0.f : ex2_approx(mw - m);
            // a warp without a key contributes nothing; one whose every score is -inf contributes
            // nothing either, but a NaN in it must stay
            l = fmaf(sml[(w * 16 + row) * 2 + 1], mw == -INFINITY ? 1.f : f, l);
#pragma unroll
            for (int e = 0; e < E; ++e)
                acc[e] = fmaf(so[(w * 16 + row) * D + lane * E + e], mw == -INFINITY ? 1.f : f, acc[e]);
        }
        if (split) {
            const size_t at = ((size_t)r * p.H + h) * p.nsplit + blockIdx.x;
            float* po = p.part_o + at * D + lane * E;
#pragma unroll
            for (int e = 0; e < E; ++e) po[e] = acc[e];
            if (lane == 0) {
                p.part_ml[at * 2] = m;
                p.part_ml[at * 2 + 1] = bad ? -1.f : l;
            }
        } else if (bad) {
            pg_zero_row<D>(p, r, h, lane);
        } else {
            pg_finish_row<D>(p, r, h, lane, m, l, acc);
        }
    }
}

// Joins the chunks of each query row, and adds the weights of the cached rows into key_weights.
// Grid (H + H_kv * weight blocks, R), 128 threads: a block x < H finishes query head x of request r; the
// others take kPgWeightRows visible rows of one key/value head each.
constexpr int kPgWeightRows = 1024;

template <int D>
__global__ void __launch_bounds__(kPgThreads) paged_join_kernel(const PgParams p)
{
    constexpr int E = D / 32;
    __shared__ float so[kPgWarps][D];
    __shared__ float sml[kPgWarps][2];
    extern __shared__ float s_lse[];                // [G] (weight blocks)
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int r = blockIdx.y;
    const PgRows rows = pg_rows(p, r);
    const int nchunk = (rows.vis + p.chunk - 1) / p.chunk;
    const bool head_block = blockIdx.x < (unsigned)p.H;
    if (head_block) {
        const int h = blockIdx.x;
        const size_t at = ((size_t)r * p.H + h) * p.nsplit;
        float m = -INFINITY;
        bool bad = !rows.ok;
        for (int c = lane; c < nchunk; c += 32) {
            m = fmaxf(m, p.part_ml[(at + c) * 2]);
            bad |= p.part_ml[(at + c) * 2 + 1] == -1.f;
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
        bad = __any_sync(0xffffffffu, bad);
        if (bad) {
            if (warp == 0) pg_zero_row<D>(p, r, h, lane);
            return;
        }
        float l = 0.f, acc[E];
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = 0.f;
        for (int c = warp; c < nchunk; c += kPgWarps) {
            const float mc = p.part_ml[(at + c) * 2];
            const float f = mc == -INFINITY ? 1.f : ex2_approx(mc - m);   // -inf: zeros (or NaN), kept
            l = fmaf(p.part_ml[(at + c) * 2 + 1], f, l);
#pragma unroll
            for (int e = 0; e < E; ++e) acc[e] = fmaf(p.part_o[(at + c) * D + lane * E + e], f, acc[e]);
        }
#pragma unroll
        for (int e = 0; e < E; ++e) so[warp][lane * E + e] = acc[e];
        if (lane == 0) sml[warp][0] = l;
        __syncthreads();
        if (warp > 0) return;
#pragma unroll
        for (int w = 1; w < kPgWarps; ++w) {
            l += sml[w][0];
#pragma unroll
            for (int e = 0; e < E; ++e) acc[e] += so[w][lane * E + e];
        }
        pg_finish_row<D>(p, r, h, lane, m, l, acc);
        return;
    }
    // ---- weights
    const int nw = (p.vmax + kPgWeightRows - 1) / kPgWeightRows;
    const int x = blockIdx.x - p.H;
    const int hkv = x / nw;
    const int vb = (x - hkv * nw) * kPgWeightRows;
    if (vb >= rows.vis) return;
    bool bad = false;
    for (int gg = warp; gg < p.G; gg += kPgWarps) {
        const int h = hkv * p.G + gg;
        const size_t at = ((size_t)r * p.H + h) * p.nsplit;
        float m = -INFINITY;
        for (int c = lane; c < nchunk; c += 32) {
            m = fmaxf(m, p.part_ml[(at + c) * 2]);
            bad |= p.part_ml[(at + c) * 2 + 1] == -1.f;
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
        const float ss = p.k_self ? pg_self_score<D>(p, r, h, lane) : -INFINITY;
        m = fmaxf(m, ss);
        float l = 0.f;
        for (int c = lane; c < nchunk; c += 32) {
            const float mc = p.part_ml[(at + c) * 2];
            l = fmaf(p.part_ml[(at + c) * 2 + 1], mc == -INFINITY ? 1.f : ex2_approx(mc - m), l);
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) l += __shfl_xor_sync(0xffffffffu, l, off);
        if (ss != -INFINITY) l += ex2_approx(ss - m);
        if (lane == 0) s_lse[gg] = m + log2f(l);    // -inf where the row sees nothing
    }
    if (__syncthreads_or(bad)) return;
    const int* table = p.table + (size_t)r * p.max_pages;
    for (int v = vb + threadIdx.x; v < min(vb + kPgWeightRows, rows.vis); v += kPgThreads) {
        float w = 0.f;
        for (int gg = 0; gg < p.G; ++gg) {
            const float s = p.scores[((size_t)r * p.H + hkv * p.G + gg) * p.vmax + v];
            w += s == -INFINITY ? 0.f : ex2_approx(s - s_lse[gg]);
        }
        const int j = rows.row(v);
        const int page = __ldg(table + j / p.ps);
        float* dst = p.key_weights + ((size_t)page * p.Hkv + hkv) * p.ps + j % p.ps;
        atomicAdd(dst, w);                         // requests may share pages (a common prefix)
    }
}

}  // namespace unipin
