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
//   - the work is cut into units of 128 visible rows (64 at 256-byte rows) of one
//     (request, key/value head, up to 16 query heads of the group); the units of all requests, in
//     order, go to one wave of blocks in equal contiguous shares, whatever the
//     requests' lengths.  (One block per chunk of a request left a third of the
//     time to the blocks' starts and ends.)  A block that holds all of a row's
//     units finishes the row; the others' pieces are joined by a second kernel;
//   - a warp takes 32 (16) rows of each of its block's units on its own, through a ring
//     of stages of its own: no block-wide barrier within a row, and the copies run
//     on across the ends of rows and requests.  Neighbouring lanes copy (cp.async)
//     neighbouring 16-byte chunks of a row, so each sector crosses from L2 once;
//     rows are looked up one by one, so any page size works and a page that ends
//     inside a tile costs nothing; chunk c of row r lies at c ^ f(r), which keeps
//     copies and fragment reads free of bank conflicts;
//   - S^T = K Q^T by mma.m16n8k16 with 16 keys as M and eight query heads as N
//     (K by ldmatrix);
//   - O^T += V^T P^T with 16 head-dim elements as M (V by ldmatrix.trans): P^T's
//     fragment is the transpose of S^T's (movmatrix).  (With the heads as M, half
//     of each product and of O's registers went to rows 8 .. 15 that eight heads or
//     fewer do not fill.)
//   - E4M3 codes come as pairs of codes in a 16-bit element: for K the four codes
//     of a register are four consecutive d, and Q is read in that order; for V a
//     transposed register holds two d of two rows, and a byte permute sorts them.
// mma.sync and not tcgen05: at 16 query rows or fewer per key the tensor work is
// under a tenth of the tensor cores' rate at the full memory rate, and a TMEM
// accumulator would put a chain of barriers (load, S, softmax, P, P.V) into
// every tile.
// Measured (B200, with the join), call by call over rows that are not in L2: 32 requests of 1024 .. 2048 rows,
// H = 8, D = 64, bf16 28.4 us (102 MB: 3.6 TB/s, 55% of the rate of a copy; repeated over the same rows, which
// the L2 holds in good part, 21.6); 256 of 32 .. 4096 under a window of 1024, D = 128, E4M3 100 us (477 MB: 4.8
// TB/s, 73%); 8 of 777 .. 32768, H = 8 over 2, D = 128, with key_weights 40.4 us (150 MB: 3.7 TB/s); one of 500
// rows 10.2 us, 8.2 in a graph.  Repeated in a graph, 32 requests of 1024 .. 2048, H = 8: bf16 D = 32, 64, 128
// 15.4, 21.6 and 41.3 us; E4M3 14.4, 18.0 and 25.7; E4M3 with other scales 16.4, 22.0 and 34.4 (and 136 for
// the window's 99); bf16 D = 64 with 8 and 16 heads over one 12.2 and 14.1.
// What is left is latency: at 12 warps per SM no warp can issue in two of three cycles over bf16 and in half of
// them over E4M3 (issue slots busy 32% and 49%), for the rows' way into the ring (one stage of two in flight
// while the other is used), the chain of a tile and the barriers at a row's end; DRAM is at 55 and 63%.  The
// join is a launch of 7 to 10 us, in part beside the main kernel.  The smallest calls are one chain: lengths,
// page, rows, S, P, O, join of the warps.
// Scores, row maxima, row sums and O are float32.  P is rounded to the type of
// V's fragment (bfloat16; float16 over E4M3 codes with power-of-two scales), as
// in the prefill: one rounding of relative size <= 2^-8 (2^-11, see PgWeights) per
// weight, independent of the others.
//
// E4M3 pools: attention reads code c as bf16(value(c) * scale).  Where both
// scales are powers of two that is value(c) * scale exactly, so the codes go to
// the tensor cores as float16 (exact), the scales are applied to the scores and
// to O, and q goes to float16 after a power-of-two scaling of its row that puts
// the row's largest element into [2^9, 2^10): bfloat16 has 8 significant bits
// and float16's smallest step is 2^-24, so only elements below 2^-26 of the row's
// largest lose bits, and none more than 2^-34 of it.
// Other scales take the float32 product and its rounding to bfloat16 per element.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "e4m3.cuh"
#include "paged_common.cuh"
#include "sm100_ptx.cuh"
#include "unipin.h"

namespace unipin {

constexpr int kPgWarps = 4;
constexpr int kPgThreads = 32 * kPgWarps;
constexpr float kPgLog2e = 1.4426950408889634f;

enum PgMode { kPgBf16 = 0, kPgE4M3Pow2 = 1, kPgE4M3Any = 2 };

// O is rescaled only when a row's maximum grows by more than 2^kRescale, and weights are held as 2^kLift times
// themselves.  In float16 a weight below 2^-14 loses bits and one below 2^-25 is gone, while the row's sum
// still counts it: so the weights use float16's whole range, the largest of a row in [2^14, 2^15].  Then weights
// down to 2^-28 of the largest are rounded by 2^-11 of themselves and smaller ones by 2^-39 of the largest,
// 2^-9 in all for the longest row that a call takes (2^30).
template <int kMode>
struct PgWeights {
    static constexpr float kRescale = kMode == kPgE4M3Pow2 ? 1.0f : 8.0f;
    static constexpr float kLift = kMode == kPgE4M3Pow2 ? 14.0f : 0.0f;
};

template <int D, int kMode>
struct PgCfg {
    static constexpr int kElt = kMode == kPgBf16 ? 2 : 1;
    static constexpr int kRowBytes = D * kElt;
    // rows of a warp's tile: 32 (one look-up per lane; what a tile costs whatever its rows is halved against
    // 16), at the widest rows 16, for three blocks per SM
    static constexpr int kKeys = kRowBytes >= 256 ? 16 : 32;
    static constexpr int kUnit = kPgWarps * kKeys;          // rows of a unit
    static constexpr int kChunks = kRowBytes / 16;          // 16-byte chunks of a row
    static constexpr int kRowsPerCopy = 32 / kChunks;       // rows that one copy of a warp covers
    static constexpr int kStageBytes = 2 * kKeys * kRowBytes;   // K and V of a tile
    // Bytes in flight per SM for the memory latency: about 100 KB (one stage of two or two of three of 12
    // or 16 warps).  Three blocks per SM against two, with a wider join: 24.3 -> 21.7 us (R = 32, D = 64, bf16),
    // 41 -> 38 us (R = 8 with weights, D = 128), 109 -> 98 us (R = 256, window, E4M3).
    static constexpr int kStages = kRowBytes >= 128 ? 2 : (kRowBytes == 64 ? 3 : 4);
    static constexpr int kBlocksPerSm = kRowBytes >= 128 ? 3 : 4;
    static constexpr int kRingBytes = kPgWarps * kStages * kStageBytes;
    static constexpr int kRedHeads = D == 128 ? 2 : 4;                              // heads that the warps join at a time
    static constexpr int kOffQ = kRingBytes;                           // [16][D] bf16
    static constexpr int kOffRed = kOffQ + 16 * D * 2;                 // [warp][kRedHeads][D] fp32
    static constexpr int kOffMl = kOffRed + kPgWarps * kRedHeads * D * 4;   // [warp][16][2] fp32
    static constexpr int kSmemBytes = kOffMl + kPgWarps * 16 * 2 * 4;
    static_assert((kSmemBytes + 1024) * kBlocksPerSm <= 228 * 1024, "shared memory budget");
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
    float* part_o;                 // [2 * blocks, heads of a unit, D]: pieces of rows (see PgPlace), or null
    float* part_ml;                // [2 * blocks, heads of a unit, 2]: (m in log2 units, l); l = -1: rejected
    int* first_unit;               // [R + 1] first unit of each request (block 0 writes it for the join)
    float* row_lse;                // [R * H] log2 of a finished row's weight sum; +inf: rejected (key_weights)
    float* scores;                 // [R * H, vmax] log2-unit scores of the visible rows (key_weights)
    int R, H, Hkv, G, S, ps, max_pages, max_len;
    PgDiv page_of;                 // division by ps
    int unit_shift;                // log2 of a unit's rows
    int window, n_sinks;
    int heads;                     // query heads of a unit: min(G, 16)
    int groups;                    // units' head groups per key/value head
    int vmax;
    int whole;                     // shares end at row ends: nothing is joined
    int shares;                    // blocks of the main kernel
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

// Units of a row with `vis` visible rows (one where there is none: the row is still written).
__device__ __forceinline__ int pg_units(const PgParams& p, int vis)
{
    return max((vis + (1 << p.unit_shift) - 1) >> p.unit_shift, 1);
}

// A place in the sequence of units: request r, key/value head hk, head group cg, unit t of u.
struct PgPlace {
    int r, hk, cg, t, u;
    PgRows rows;
    __device__ void enter(const PgParams& p)
    {
        if (r < p.R) {
            rows = pg_rows(p, r);
            u = pg_units(p, rows.vis);
        }
    }
    // the first unit of the next row
    __device__ void next_row(const PgParams& p)
    {
        t = 0;
        if (++cg < p.groups) return;
        cg = 0;
        if (++hk < p.Hkv) return;
        hk = 0;
        ++r;
        enter(p);
    }
    __device__ void next(const PgParams& p)
    {
        if (++t == u) next_row(p);
    }
};

// Sixteen bytes into shared memory, or zeros.
__device__ __forceinline__ void pg_copy(uint32_t dst, const void* src, bool live)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}

__device__ __forceinline__ void pg_copy(uint32_t dst, const void* src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

__device__ __forceinline__ void pg_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

template <int N>
__device__ __forceinline__ void pg_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Four 8 x 8 matrices of 16-bit elements, one row address per lane.
__device__ __forceinline__ void pg_ldmatrix(uint32_t addr, uint32_t (&r)[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}

__device__ __forceinline__ void pg_ldmatrix_trans(uint32_t addr, uint32_t (&r)[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}

// Where the 16-byte chunk c of row r of a tile lies (in chunks): eight rows' chunk c, and a row's eight
// neighbouring chunks, fall into different bank groups.
template <int kChunks>
__host__ __device__ constexpr int pg_swizzle(int r, int c)
{
    return r * kChunks + (c ^ (kChunks >= 8 ? r & 7 : (kChunks == 4 ? (r >> 1) & 3 : (r >> 2) & 1)));
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

// Four E4M3 codes as two pairs of operands: float16 (exact), or bf16(value * scale), what attention reads.
template <int kMode>
__device__ __forceinline__ void pg_expand(uint32_t codes, float scale, uint32_t& lo, uint32_t& hi)
{
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(lo), "=r"(hi) : "r"(codes));
    if constexpr (kMode == kPgE4M3Any) {
        const __half2 a = *reinterpret_cast<const __half2*>(&lo), b = *reinterpret_cast<const __half2*>(&hi);
        lo = pack_bf16x2(__fmul_rn(__low2float(a), scale), __fmul_rn(__high2float(a), scale));
        hi = pack_bf16x2(__fmul_rn(__low2float(b), scale), __fmul_rn(__high2float(b), scale));
    }
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
// rows, the own key merged in, divided and stored.  A row that sees nothing is zeros.  Returns log2 of
// the sum of the row's weights.
template <int D>
__device__ __forceinline__ float pg_finish_row(const PgParams& p, int r, int h, int lane, float m, float l,
                                              float (&o)[D / 32])
{
    constexpr int E = D / 32;
    float a = 1.f, b = 0.f, mf = m;
    if (p.k_self) {
        const float ss = pg_self_score<D>(p, r, h, lane);
        mf = fmaxf(m, ss);
        a = m == -INFINITY ? 0.f : ex2_approx(m - mf);
        b = ss == -INFINITY ? 0.f : ex2_approx(ss - mf);
        if (ss != ss) b = ss;                 // a NaN score makes the row NaN
    }
    const float total = l * a + b;
    const float inv = total == 0.f ? 0.f : 1.f / total;
    float res[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
        float x = o[e] * a;                       // (a = 0: a NaN or infinite value still shows)
        if (b != 0.f)
            x = fmaf(b, __bfloat162float(p.v_self[((size_t)r * p.Hkv + h / p.G) * D + lane * E + e]), x);
        res[e] = x * inv;
    }
    pg_store_row<E>(p.out, p.out_fp32, ((size_t)r * p.H + h) * D + lane * E, res);
    return mf + log2f(total);                     // -inf where the row sees nothing
}

template <int D>
__device__ __forceinline__ void pg_zero_row(const PgParams& p, int r, int h, int lane)
{
    float z[D / 32];
#pragma unroll
    for (int e = 0; e < D / 32; ++e) z[e] = 0.f;
    pg_store_row<D / 32>(p.out, p.out_fp32, ((size_t)r * p.H + h) * D + lane * (D / 32), z);
}


// Transpose of an 8 x 8 matrix of 16-bit elements, two per lane.
__device__ __forceinline__ uint32_t pg_transpose(uint32_t a)
{
    uint32_t d;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}

struct PgScan {
    int warp_sum[kPgWarps];
    int r, first;
};

// Units of a share: equal shares of all units, the last ones less or none.
__device__ __forceinline__ int pg_share(int total, int shares) { return (total + shares - 1) / shares; }

// The units [x, x1) of share `b` and the place of unit x, by a scan over all requests' lengths, which
// every block makes for itself (4 R bytes; unit numbers fit 31 bits, the host sees to it).  With
// `first_unit` the first unit of every request is written there, and behind them their total.
__device__ __forceinline__ void pg_find(const PgParams& p, PgScan& sc, int* first_unit, int b, int& x, int& x1,
                                        PgPlace& at)
{
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int y_all = p.Hkv * p.groups;
    const int per = (p.R + kPgThreads - 1) / kPgThreads;
    const int r0 = min(tid * per, p.R), r1 = min(r0 + per, p.R);   // this thread's requests
    int sum = 0;
    for (int r = r0; r < r1; ++r) sum += pg_units(p, pg_rows(p, r).vis) * y_all;
    int incl = sum;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += up;
    }
    if (lane == 31) sc.warp_sum[warp] = incl;
    __syncthreads();
    int base = 0, total = 0;
#pragma unroll
    for (int w = 0; w < kPgWarps; ++w) {
        if (w < warp) base += sc.warp_sum[w];
        total += sc.warp_sum[w];
    }
    const int share = pg_share(total, p.shares);
    x = (int)min((long long)b * share, (long long)total);
    x1 = (int)min((long long)x + share, (long long)total);
    int first = base + incl - sum;
    if (first_unit || (first <= x && x < first + sum)) {
        for (int r = r0; r < r1; ++r) {
            const int n = pg_units(p, pg_rows(p, r).vis) * y_all;
            if (first_unit) first_unit[r] = first;
            if (first <= x && x < first + n) {
                sc.r = r;
                sc.first = first;
            }
            first += n;
        }
    }
    if (first_unit && tid == 0) first_unit[p.R] = total;
    __syncthreads();
    if (x >= x1) return;
    at.r = sc.r;
    at.enter(p);
    const int y = (x - sc.first) / at.u;
    at.hk = y / p.groups;
    at.cg = y - at.hk * p.groups;
    at.t = (x - sc.first) - y * at.u;
}

// One wave of blocks, block b: units [b share, (b + 1) share).  kNG: groups of eight query heads (1 or 2).
template <int D, int kMode, int kNG>
__global__ void __launch_bounds__(kPgThreads, PgCfg<D, kMode>::kBlocksPerSm) paged_decode_kernel(const PgParams p)
{
    using C = PgCfg<D, kMode>;
    using W = PgWeights<kMode>;
    constexpr bool kHalf = kMode == kPgE4M3Pow2;
    constexpr int MT = D / 16;                      // k-steps of S^T, m-tiles of O^T
    extern __shared__ __align__(1024) uint8_t smem[];   // (fragment addresses are formed by xor)
    __shared__ PgScan scan;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int g = lane / 4, t = lane % 4;
    PgPlace at;
    int x, x1;
    pg_find(p, scan, blockIdx.x == 0 ? p.first_unit : nullptr, blockIdx.x, x, x1, at);
    // whole rows: from the first that begins in the share to the last that does
    if (p.whole)
        for (; x < x1 && at.t != 0; ++x) at.next(p);
    if (x >= x1) return;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // the join waits for this kernel's end itself
    const uint32_t ring = smem_u32(smem) + warp * C::kStages * C::kStageBytes;
    __nv_bfloat16* sQ = reinterpret_cast<__nv_bfloat16*>(smem + C::kOffQ);
    float* sRed = reinterpret_cast<float*>(smem + C::kOffRed);
    float* sMl = reinterpret_cast<float*>(smem + C::kOffMl);

    // ---- the copies, kStages - 1 units ahead of the products
    PgPlace ld = at;
    int xl = x;
    bool ld_end = false;                            // the share's last unit has been asked for
    uint32_t bad_stages = 0;                        // stages with a page id out of range
    // a tile's rows on their way to `issue`: this lane's row in the layer's plane
    uint32_t row = 0;
    bool row_live = false, row_bad = false;
    auto look_up = [&]() {
        const int v = ld.t * C::kUnit + warp * C::kKeys + lane % C::kKeys;
        row = 0;
        row_live = !ld_end && v < ld.rows.vis;
        row_bad = false;
        if (row_live) {
            const int j = ld.rows.row(v);
            const int pg = p.page_of(j);
            const int page = __ldg(p.table + (size_t)ld.r * p.max_pages + pg);
            row_bad = page < 0 || page >= p.S;
            if (row_bad) row_live = false;
            else row = ((uint32_t)page * p.Hkv + ld.hk) * (uint32_t)p.ps + (uint32_t)(j - pg * p.ps);
        }
        if (!ld_end) {
            ld.next(p);
            ++xl;
            ld_end = xl >= x1 && (!p.whole || ld.t == 0);
        }
    };
    const int cc = lane % C::kChunks, cr = lane / C::kChunks;   // the chunk of the row that this lane copies
    const uint8_t* src_k = p.pool_k + cc * 16;
    const uint8_t* src_v = p.pool_v + cc * 16;
    auto issue = [&](int stage) {
        const uint32_t st = ring + stage * C::kStageBytes;
        const uint32_t live = __ballot_sync(0xffffffffu, row_live);
        const bool bad = __any_sync(0xffffffffu, row_bad);
        bad_stages = (bad_stages & ~(1u << stage)) | ((uint32_t)bad << stage);
#pragma unroll
        for (int i = 0; i < C::kKeys / C::kRowsPerCopy; ++i) {
            const int tr = i * C::kRowsPerCopy + cr;
            const uint64_t at_row = (uint64_t)__shfl_sync(0xffffffffu, row, tr) * C::kRowBytes;
            const uint32_t dst = st + pg_swizzle<C::kChunks>(tr, cc) * 16;
            if (live == 0xffffffffu) {            // (16-row tiles: the upper lanes look up the same rows)
                pg_copy(dst, src_k + at_row);
                pg_copy(dst + C::kStageBytes / 2, src_v + at_row);
            } else {
                pg_copy(dst, src_k + at_row, (live >> tr) & 1u);
                pg_copy(dst + C::kStageBytes / 2, src_v + at_row, (live >> tr) & 1u);
            }
        }
    };

    look_up();
#pragma unroll
    for (int i = 0; i < C::kStages - 1; ++i) {
        issue(i);
        pg_commit();
        look_up();                                  // (the next one's: its page lookup overlaps a unit's work)
    }

    // ---- query rows: this unit's in shared memory, the next row's on the way in a register
    constexpr int kQVecs = (2 * D + kPgThreads - 1) / kPgThreads;   // 16 rows x D / 8 vectors
    // this thread's vectors of the query rows of a place
    auto q_fetch = [&](int r, int hk, int cg, uint4 (&v)[kQVecs]) {
        const int nh = min(p.heads, p.G - cg * 16);
#pragma unroll
        for (int i = 0; i < kQVecs; ++i) {
            const int hh = (threadIdx.x + i * kPgThreads) / (D / 8), c = (threadIdx.x + i * kPgThreads) % (D / 8);
            v[i] = make_uint4(0u, 0u, 0u, 0u);
            if (r < p.R && hh < nh)
                v[i] = __ldg(reinterpret_cast<const uint4*>(p.q + ((size_t)r * p.H + hk * p.G + cg * 16 + hh) * D) + c);
        }
    };
    auto q_store = [&](const uint4 (&v)[kQVecs]) {
#pragma unroll
        for (int i = 0; i < kQVecs; ++i)
            if (threadIdx.x + i * kPgThreads < 2 * D) reinterpret_cast<uint4*>(sQ)[threadIdx.x + i * kPgThreads] = v[i];
    };
    uint4 q_next[kQVecs];
    q_fetch(at.r, at.hk, at.cg, q_next);
    q_store(q_next);
    __syncthreads();

    int stage = 0;
    while (x < x1) {
        // ---- a row: units t .. of (r, y) that are this block's
        const int h0 = at.hk * p.G + at.cg * 16;
        const int nh = min(p.heads, p.G - at.cg * 16);
        const int r = at.r, t_first = at.t, units = p.whole ? at.u - at.t : min(at.u - at.t, x1 - x);
        const PgRows rows = at.rows;
        const bool all = t_first == 0 && units == at.u;   // else a piece of the row
        x += units;
        at.next_row(p);                             // (a share that ends inside a row ends with it)
        q_fetch(at.r, at.hk, at.cg, q_next);
        if (p.k_self && all && threadIdx.x < 2) {   // read when the row is finished
            const size_t own = ((size_t)r * p.Hkv + h0 / p.G) * D;
            asm volatile("prefetch.global.L1 [%0];" ::"l"((threadIdx.x ? p.v_self : p.k_self) + own));
            if (D == 128) asm volatile("prefetch.global.L1 [%0];" ::"l"((threadIdx.x ? p.v_self : p.k_self) + own + 64));
        }

        // Q fragments: head g (and g + 8) as N, d in the order of the K fragments
        uint32_t qf[kNG][MT][2];
        float fac[kNG][2];                          // score factors of heads 2t, 2t + 1 (+ 8)
#pragma unroll
        for (int n = 0; n < kNG; ++n) {
            const __nv_bfloat16* q0 = sQ + (n * 8 + g) * D;
#pragma unroll
            for (int c = 0; c < MT; ++c) {
                if constexpr (kMode == kPgBf16) {
                    qf[n][c][0] = *reinterpret_cast<const uint32_t*>(q0 + c * 16 + 2 * t);
                    qf[n][c][1] = *reinterpret_cast<const uint32_t*>(q0 + c * 16 + 8 + 2 * t);
                } else {
                    const uint2 x2 = *reinterpret_cast<const uint2*>(q0 + c * 16 + 4 * t);
                    qf[n][c][0] = x2.x;
                    qf[n][c][1] = x2.y;
                }
            }
            fac[n][0] = fac[n][1] = p.sl2;
            if constexpr (kHalf) {
                float top = 0.f;
#pragma unroll
                for (int c = 0; c < MT; ++c)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        top = fmaxf(top, fabsf(__uint_as_float(qf[n][c][i] << 16)));
                        top = fmaxf(top, fabsf(__uint_as_float(qf[n][c][i] & 0xffff0000u)));
                    }
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                int e = (int)((__float_as_uint(top) >> 23) & 255) - 127;   // top in [2^e, 2^(e+1))
                if (top == 0.f || e == 128) e = 9;
                e = max(e, -100);                                          // keeps both powers finite
                const float up = __uint_as_float((uint32_t)(9 - e + 127) << 23);   // 2^(9-e), 9-e in [-118, 109]
#pragma unroll
                for (int c = 0; c < MT; ++c)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const __half2 h = __floats2half2_rn(__uint_as_float(qf[n][c][i] << 16) * up,
                                                            __uint_as_float(qf[n][c][i] & 0xffff0000u) * up);
                        qf[n][c][i] = *reinterpret_cast<const uint32_t*>(&h);
                    }
                const float down = __uint_as_float((uint32_t)(e - 9 + 127) << 23);
                fac[n][0] *= __shfl_sync(0xffffffffu, down, 8 * t);        // of head 2t: lane (2t, any)
                fac[n][1] *= __shfl_sync(0xffffffffu, down, 8 * t + 4);
            }
        }

        float o[kNG][MT][4];
        float m[kNG][2], l[kNG][2];                 // of heads 2t, 2t + 1 (+ 8)
#pragma unroll
        for (int n = 0; n < kNG; ++n) {
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[n][i][e] = 0.f;
            m[n][0] = m[n][1] = -INFINITY;
            l[n][0] = l[n][1] = 0.f;
        }
        bool bad = !rows.ok;

        for (int i = 0; i < units; ++i) {
            pg_wait<C::kStages - 2>();              // the unit has landed: this lane's copies,
            __syncwarp();                           // and the other lanes'
            bad |= (bad_stages >> stage) & 1u;
            issue(stage == 0 ? C::kStages - 1 : stage - 1);   // the stage that the unit before has left
            pg_commit();
            look_up();
            const uint32_t st = ring + stage * C::kStageBytes;
            stage = stage + 1 == C::kStages ? 0 : stage + 1;
            const int vt = (t_first + i) * C::kUnit + warp * C::kKeys;   // visible index of the tile's first key
            if (vt >= rows.vis) continue;
            constexpr int KT = C::kKeys / 16;        // m-tiles of S^T, k-steps of O^T
            float s[kNG][KT][4];
#pragma unroll
            for (int n = 0; n < kNG; ++n)
#pragma unroll
                for (int k = 0; k < KT; ++k)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[n][k][e] = 0.f;
            // K: matrices (rows 0-7, 8-15) x (chunk, next chunk)
            const uint32_t ka = st + pg_swizzle<C::kChunks>((lane & 7) + (lane & 8), lane >> 4) * 16;
#pragma unroll
            for (int k = 0; k < KT; ++k) {
                const uint32_t kk = ka + k * 16 * C::kRowBytes;
                if constexpr (kMode == kPgBf16) {
#pragma unroll
                    for (int c = 0; c < MT; ++c) {
                        uint32_t a[4];
                        pg_ldmatrix(kk ^ (c * 32), a);
#pragma unroll
                        for (int n = 0; n < kNG; ++n)
                            pg_mma<kHalf>(s[n][k], a[0], a[1], a[2], a[3], qf[n][c][0], qf[n][c][1]);
                    }
                } else {
#pragma unroll
                    for (int c = 0; c < MT; c += 2) {
                        uint32_t a[4];
                        pg_ldmatrix(kk ^ (c * 16), a);
#pragma unroll
                        for (int i2 = 0; i2 < 2; ++i2) {
                            uint32_t a0, a1, a2, a3;
                            pg_expand<kMode>(a[2 * i2], p.k_scale, a0, a2);
                            pg_expand<kMode>(a[2 * i2 + 1], p.k_scale, a1, a3);
#pragma unroll
                            for (int n = 0; n < kNG; ++n)
                                pg_mma<kHalf>(s[n][k], a0, a1, a2, a3, qf[n][c + i2][0], qf[n][c + i2][1]);
                        }
                    }
                }
            }
            // s[n][k]: keys 16k + (g, g, g + 8, g + 8) of heads 2t, 2t + 1, 2t, 2t + 1 (+ 8 n)
            bool grow = false;
            float top[kNG][2];
#pragma unroll
            for (int n = 0; n < kNG; ++n) {
#pragma unroll
                for (int k = 0; k < KT; ++k)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[n][k][e] *= fac[n][e & 1];
                if (p.scores) {
#pragma unroll
                    for (int k = 0; k < KT; ++k)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int hh = n * 8 + 2 * t + (e & 1), v = vt + k * 16 + g + 8 * (e >> 1);
                            if (hh < nh && v < rows.vis) p.scores[((size_t)r * p.H + h0 + hh) * p.vmax + v] = s[n][k][e];
                        }
                }
                if (vt + C::kKeys > rows.vis) {      // the row ends inside the tile
#pragma unroll
                    for (int k = 0; k < KT; ++k)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (vt + k * 16 + g + 8 * (e >> 1) >= rows.vis) s[n][k][e] = -INFINITY;
                }
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    top[n][e] = fmaxf(s[n][0][e], s[n][0][e + 2]);
#pragma unroll
                    for (int k = 1; k < KT; ++k) top[n][e] = max3f(top[n][e], s[n][k][e], s[n][k][e + 2]);
                    grow |= top[n][e] > m[n][e] + W::kRescale;
                }
            }
            if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
                for (int n = 0; n < kNG; ++n) {
                    float f[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float x2 = top[n][e];
                        x2 = fmaxf(x2, __shfl_xor_sync(0xffffffffu, x2, 4));
                        x2 = fmaxf(x2, __shfl_xor_sync(0xffffffffu, x2, 8));
                        x2 = fmaxf(x2, __shfl_xor_sync(0xffffffffu, x2, 16));
                        const float to = fmaxf(m[n][e], x2);
                        f[e] = m[n][e] == -INFINITY ? 0.f : ex2_approx(m[n][e] - to);
                        m[n][e] = to;
                        l[n][e] *= f[e];
                    }
#pragma unroll
                    for (int i2 = 0; i2 < MT; ++i2)
#pragma unroll
                        for (int e = 0; e < 4; ++e) o[n][i2][e] *= f[e & 1];
                }
            }
            uint32_t pb[kNG][KT][2];
#pragma unroll
            for (int n = 0; n < kNG; ++n) {
                const float u0 = m[n][0] == -INFINITY ? 0.f : m[n][0] - W::kLift;
                const float u1 = m[n][1] == -INFINITY ? 0.f : m[n][1] - W::kLift;
#pragma unroll
                for (int k = 0; k < KT; ++k) {
                    const float e0 = ex2_approx(s[n][k][0] - u0), e1 = ex2_approx(s[n][k][1] - u1);
                    const float e2 = ex2_approx(s[n][k][2] - u0), e3 = ex2_approx(s[n][k][3] - u1);
                    l[n][0] += e0 + e2;
                    l[n][1] += e1 + e3;
                    pb[n][k][0] = pg_transpose(pg_pack_p(e0, e1, kHalf));
                    pb[n][k][1] = pg_transpose(pg_pack_p(e2, e3, kHalf));
                }
            }
            // ---- O^T += V^T P^T
            if constexpr (kMode == kPgBf16) {
                // matrices (rows 0-7) x (chunk, next), then rows 8-15: dims g, g + 8 of a 16
                const uint32_t va = st + C::kStageBytes / 2 +
                                    pg_swizzle<C::kChunks>((lane & 7) + (lane >> 4) * 8, (lane >> 3) & 1) * 16;
#pragma unroll
                for (int k = 0; k < KT; ++k)
#pragma unroll
                    for (int c = 0; c < MT; ++c) {
                        uint32_t a[4];
                        pg_ldmatrix_trans((va + k * 16 * C::kRowBytes) ^ (c * 32), a);
#pragma unroll
                        for (int n = 0; n < kNG; ++n)
                            pg_mma<kHalf>(o[n][c], a[0], a[1], a[2], a[3], pb[n][k][0], pb[n][k][1]);
                    }
            } else {
                // as K, transposed: a register has codes 2g, 2g + 1 of a chunk, of rows 2t and 2t + 1
                const uint32_t va = ka + C::kStageBytes / 2;
#pragma unroll
                for (int k = 0; k < KT; ++k)
#pragma unroll
                    for (int c = 0; c < MT; c += 2) {
                        uint32_t a[4];
                        pg_ldmatrix_trans((va + k * 16 * C::kRowBytes) ^ (c * 16), a);
#pragma unroll
                        for (int i2 = 0; i2 < 2; ++i2) {
                            uint32_t a0, a1, a2, a3;
                            pg_expand<kMode>(__byte_perm(a[2 * i2], 0u, 0x3120u), p.v_scale, a0, a1);
                            pg_expand<kMode>(__byte_perm(a[2 * i2 + 1], 0u, 0x3120u), p.v_scale, a2, a3);
#pragma unroll
                            for (int n = 0; n < kNG; ++n)
                                pg_mma<kHalf>(o[n][c + i2], a0, a1, a2, a3, pb[n][k][0], pb[n][k][1]);
                        }
                    }
            }
        }

        // ---- the warps' O, m, l joined through shared memory, C::kRedHeads heads at a time
        constexpr int E = D / 32;
        [[maybe_unused]] const float vs = kMode == kPgE4M3Pow2 ? p.v_scale : 1.f;
#pragma unroll
        for (int n = 0; n < kNG; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float sum = l[n][e];
                sum += __shfl_xor_sync(0xffffffffu, sum, 4);
                sum += __shfl_xor_sync(0xffffffffu, sum, 8);
                sum += __shfl_xor_sync(0xffffffffu, sum, 16);
                if (g == 0) {
                    sMl[(warp * 16 + n * 8 + 2 * t + e) * 2] = m[n][e] - W::kLift;   // what l and O are relative to
                    sMl[(warp * 16 + n * 8 + 2 * t + e) * 2 + 1] = sum;
                }
            }
        for (int hr = 0; hr < nh; hr += C::kRedHeads) {
#pragma unroll
            for (int n = 0; n < kNG; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int hh = n * 8 + 2 * t + e - hr;
                    if (hh < 0 || hh >= C::kRedHeads) continue;
                    float* dst = sRed + (warp * C::kRedHeads + hh) * D;
#pragma unroll
                    for (int i = 0; i < MT; ++i) {
                        if constexpr (kMode == kPgBf16) {
                            dst[i * 16 + g] = o[n][i][e];
                            dst[i * 16 + 8 + g] = o[n][i][e + 2];
                        } else {
                            *reinterpret_cast<float2*>(dst + i * 16 + 2 * g) =
                                make_float2(o[n][i][e] * vs, o[n][i][e + 2] * vs);
                        }
                    }
                }
            bad = __syncthreads_or(bad);
            if (hr == 0) q_store(q_next);
            for (int hh = warp; hh < min(C::kRedHeads, nh - hr); hh += kPgWarps) {
                const int head = hr + hh;           // within the unit's heads
                float mm = -INFINITY, ll = 0.f, acc[E];
#pragma unroll
                for (int e = 0; e < E; ++e) acc[e] = 0.f;
#pragma unroll
                for (int w = 0; w < kPgWarps; ++w) mm = fmaxf(mm, sMl[(w * 16 + head) * 2]);
#pragma unroll
                for (int w = 0; w < kPgWarps; ++w) {
                    const float mw = sMl[(w * 16 + head) * 2];
                    // a warp without a key contributes nothing; one whose every score is -inf contributes
                    // nothing either, but a NaN in it must stay
                    const float f = mw == -INFINITY ? 1.f : ex2_approx(mw - mm);
                    ll = fmaf(sMl[(w * 16 + head) * 2 + 1], f, ll);
#pragma unroll
                    for (int e = 0; e < E; ++e)
                        acc[e] = fmaf(sRed[(w * C::kRedHeads + hh) * D + lane * E + e], f, acc[e]);
                }
                if (!all) {
                    // a block's first piece, of a row that began before it, goes to slot 2b, its last to 2b + 1
                    const size_t slot = ((size_t)blockIdx.x * 2 + (t_first == 0 ? 1 : 0)) * p.heads + head;
#pragma unroll
                    for (int e = 0; e < E; ++e) p.part_o[slot * D + lane * E + e] = acc[e];
                    if (lane == 0) {
                        p.part_ml[slot * 2] = mm;
                        p.part_ml[slot * 2 + 1] = bad ? -1.f : ll;
                    }
                } else {
                    float lse = INFINITY;
                    if (bad) pg_zero_row<D>(p, r, h0 + head, lane);
                    else lse = pg_finish_row<D>(p, r, h0 + head, lane, mm, ll, acc);
                    if (p.row_lse && lane == 0) p.row_lse[(size_t)r * p.H + h0 + head] = lse;
                }
            }
            __syncthreads();                        // sRed and sMl may be written again
        }
        if (bad && threadIdx.x == 0) report(p.status, (int)UNIPIN_ERR_OUT_OF_RANGE);
    }
    pg_wait<0>();
}

// Joins the pieces of each query row, and adds the weights of the cached rows into key_weights.
// Grid (H + H_kv * weight blocks, R), 128 threads: a block x < H finishes query head x of request r (if it
// is in pieces); the others take kPgWeightRows visible rows of one key/value head each.
constexpr int kPgWeightRows = 512;
constexpr int kPgJoinWarps = 4;

// The pieces of a query row: those of blocks b0 .. b1 (one block: the row is finished already).
struct PgPieces {
    int b0, b1, heads, head;
    __device__ PgPieces(const PgParams& p, int r, int h, int vis)
    {
        const int share = pg_share(p.first_unit[p.R], p.shares);
        const int hk = h / p.G, rest = h - hk * p.G, u = pg_units(p, vis);
        const int start = p.first_unit[r] + (hk * p.groups + rest / 16) * u;
        b0 = start / share;
        b1 = (start + u - 1) / share;
        heads = p.heads;
        head = rest % 16;
    }
    __device__ size_t slot(int b) const { return ((size_t)b * 2 + (b == b0 ? 1 : 0)) * heads + head; }
};

template <int D>
__global__ void __launch_bounds__(32 * kPgJoinWarps) paged_join_kernel(const PgParams p)
{
    constexpr int E = D / 32;
    __shared__ float so[kPgJoinWarps][D];
    __shared__ float sml[kPgJoinWarps];
    extern __shared__ float s_lse[];                // [G] (weight blocks)
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int r = blockIdx.y;
    const PgRows rows = pg_rows(p, r);
    asm volatile("griddepcontrol.wait;" ::: "memory");   // (behind it: what the main kernel wrote)
    if (blockIdx.x < (unsigned)p.H) {
        const int h = blockIdx.x;
        const PgPieces pc(p, r, h, rows.vis);
        if (pc.b0 == pc.b1) return;
        float m = -INFINITY;
        bool bad = !rows.ok;
        for (int b = pc.b0 + lane; b <= pc.b1; b += 32) {
            m = fmaxf(m, p.part_ml[pc.slot(b) * 2]);
            bad |= p.part_ml[pc.slot(b) * 2 + 1] == -1.f;
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
#pragma unroll 4
        for (int b = pc.b0 + warp; b <= pc.b1; b += kPgJoinWarps) {
            const size_t slot = pc.slot(b);
            const float mc = p.part_ml[slot * 2];
            const float f = mc == -INFINITY ? 1.f : ex2_approx(mc - m);   // -inf: zeros (or NaN), kept
            l = fmaf(p.part_ml[slot * 2 + 1], f, l);
#pragma unroll
            for (int e = 0; e < E; ++e) acc[e] = fmaf(p.part_o[slot * D + lane * E + e], f, acc[e]);
        }
#pragma unroll
        for (int e = 0; e < E; ++e) so[warp][lane * E + e] = acc[e];
        if (lane == 0) sml[warp] = l;
        __syncthreads();
        if (warp > 0) return;
#pragma unroll
        for (int w = 1; w < kPgJoinWarps; ++w) {
            l += sml[w];
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
    for (int gg = warp; gg < p.G; gg += kPgJoinWarps) {
        const int h = hkv * p.G + gg;
        const PgPieces pc(p, r, h, rows.vis);
        float lse;
        if (pc.b0 == pc.b1) {
            lse = p.row_lse[(size_t)r * p.H + h];
            bad |= lse == INFINITY;
        } else {
            float m = -INFINITY;
            for (int b = pc.b0 + lane; b <= pc.b1; b += 32) {
                m = fmaxf(m, p.part_ml[pc.slot(b) * 2]);
                bad |= p.part_ml[pc.slot(b) * 2 + 1] == -1.f;
            }
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
            const float ss = p.k_self ? pg_self_score<D>(p, r, h, lane) : -INFINITY;
            m = fmaxf(m, ss);
            float l = 0.f;
            for (int b = pc.b0 + lane; b <= pc.b1; b += 32) {
                const float mc = p.part_ml[pc.slot(b) * 2];
                l = fmaf(p.part_ml[pc.slot(b) * 2 + 1], mc == -INFINITY ? 1.f : ex2_approx(mc - m), l);
            }
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) l += __shfl_xor_sync(0xffffffffu, l, off);
            if (ss != -INFINITY) l += ex2_approx(ss - m);
            lse = m + log2f(l);                     // -inf where the row sees nothing
        }
        if (lane == 0) s_lse[gg] = lse;
    }
    if (__syncthreads_or(bad)) return;
    const int* table = p.table + (size_t)r * p.max_pages;
    static_assert(kPgWeightRows == 4 * 32 * kPgJoinWarps, "four rows per thread");
    const int v = vb + 4 * threadIdx.x;
    if (v >= rows.vis) return;
    float w[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int gg = 0; gg < p.G; ++gg) {
        // (vmax is a multiple of four; scores behind the last row are not used)
        const float4 x4 = *reinterpret_cast<const float4*>(p.scores + ((size_t)r * p.H + hkv * p.G + gg) * p.vmax + v);
        const float s[4] = {x4.x, x4.y, x4.z, x4.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] += s[i] == -INFINITY ? 0.f : ex2_approx(s[i] - s_lse[gg]);
    }
    float* dst[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int j = rows.row(min(v + i, rows.vis - 1));
        const int pg = p.page_of(j);
        dst[i] = p.key_weights + ((size_t)__ldg(table + pg) * p.Hkv + hkv) * p.ps + (j - pg * p.ps);
    }
    // atomic: requests may share pages (a common prefix)
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (v + i < rows.vis) atomicAdd(dst[i], w[i]);
}

}  // namespace unipin
