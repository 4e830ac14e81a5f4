// Gradients of the masked attention under a sliding window with first rows
// that stay visible, on sm_100a.
//
// With P_ij = 2^(s_ij * sl2 - lse_i) (sl2 = scale * log2 e, lse_i the forward's
// row statistic in the same units), O_i = sum_j P_ij v_j and the upstream
// gradient dO, over the allowed pairs (i, j):
//   Dvec_i = dO_i . O_i
//   dS_ij  = P_ij (dO_i . v_j - Dvec_i)
//   dV_j   = sum_i P_ij dO_i,   dK_j = scale * sum_i dS_ij q_i
//   dQ_i   = scale * sum_j dS_ij k_j
// Row i sees the past keys j <= i, j < n_b with min(i, n_b) - j < window or
// j < n_sinks, and a candidate its own key.
//
// win_bwd_prep_kernel: Dvec of every row (dO . O, O as the forward rounded it; where a row sees eight keys or
// fewer, sum_j P_ij dO_i . v_j: there dS is small against dO . O and the rounding of O would be the largest
// error of dQ and dK, 3.5e-3 of a gradient under a window of two in place of 1.7e-3), and for a candidate its own key (the
// only row that sees it): dK and dV of a candidate come from here alone, and the
// weight of that key in dQ (dself) is left for the dQ blocks.
// win_bwd_kernel: blocks of two kinds, the first n_kv of the grid the KV blocks.
//   KV block: 128 past keys of (segment, key/value head).  K and V of the keys
//     stay in shared memory; the 64-row tiles of Q and dO of the rows that see
//     them are streamed, for each of the G query heads in turn:
//       S^T = K Q^T, dP^T = V dO^T;  dV += P^T dO, dK += dS^T Q
//     A long sweep (a tile with sinks is seen by every row) is cut into pieces whose
//     float32 sums are added up, in order, by the piece that ends last.
//   dQ block: 128 rows of (segment, query head).  Q and dO stay, the 64-row tiles
//     of K and V that the rows see are streamed:
//       S = Q K^T, dP = dO V^T;      dQ += dS K
//   So each pair's S and dP are computed twice (7 products instead of 5), and in
//   return no gradient is summed with atomics: under a window every key meets few
//   rows, and adding fp32 dQ tiles into memory (written once to zero, added to
//   once per key tile, read again to be rounded) costs more than the two products,
//   and would leave the order of the additions open.
// Both kinds run one pipeline: resident tiles R0, R1, streamed tiles T0, T1,
//   S = R0 T0^T, dP = R1 T1^T (TMEM, lane = resident row, column = streamed row),
//   P and dS from them by the softmax warps, back into TMEM as bfloat16 over the
//   scores, acc1 += dS T0 and (KV) acc0 += P T1 with P, dS as A from TMEM.
// Warps: 8 softmax warps per stage (two threads per resident row, 32 streamed rows
// each: no row statistic is left to be computed, so they need not meet), then the
// TMA producer and the MMA issuer.  At
// D = 128 two stages of S and dP and one block per SM: while one group of softmax
// warps works on a tile the other's products run.  At D <= 64 one stage and two
// blocks per SM, which also hides a block's first loads and its epilogue.
// P is rounded to bfloat16 (relative 2^-8) as a tensor-core operand of dV; dS goes to the products as the sum of
// two bfloat16 (relative 2^-15), which costs one product per tile in either kind of block: dS carries the
// error of Dvec already (of an output that was rounded twice), and with a third rounding dQ and dK would be
// the least exact of the results (relative error 2.5e-3 in place of 1.8e-3, where the gradients' own rounding
// to bfloat16 is 1.7e-3).  Scores, P, dS and all sums are float32.
// Bound: the chain of a tile (0.8 us of softmax, 0.7 us of products alone on an SM; a third of the softmax is
// the exponentials' rate) at one or two blocks per SM: the tensor pipe is busy 18% of the time at D = 64 and 35%
// at D = 128, the issue slots 35% and 30%.  The first loads and the epilogue of a block are 5 of its 12 us.
// Measured (B200), with the forward: 64 segments of 256 + 128 rows, H = 8, D = 64, window 128,
// 184 us (forward 45, this kernel 124, the prep kernel's exposed part; 304 MB); 8 segments of 700 .. 1500,
// H = 8 over 2, D = 128, window 300, 164 us; one of 186 + 125, H = 8 over 1, D = 128, window 80, 42 us.  A
// persistent block that took its items from a ring of its own took 145 us for this kernel in the first case;
// sweeps with sinks in one piece 190 and 180 us for the first two; pieces' sums stored row by row, as the
// threads hold them, 171 us for the second and 82 us for the third.
// Segments are kept apart: streamed rows behind the segment's (or behind its
// history) are zeroed in shared memory before they meet a zero weight, so what
// another segment holds cannot reach a gradient through 0 * NaN.
#pragma once

#include "sm100_ptx.cuh"
#include "tmem_wide.cuh"
#include "unipin.h"
#include "win_common.cuh"

namespace unipin {

template <int D>
struct WbCfg {
    static constexpr int kBoxElems = D >= 64 ? 64 : D;
    static constexpr int kBoxes = D / kBoxElems;
    static constexpr int kRowBytes = kBoxElems * 2;
    static constexpr uint32_t kLayout = D >= 64 ? kLayoutSw128 : kLayoutSw64;
    static constexpr int kResBox = kWinRes * kRowBytes;
    static constexpr int kResTile = kBoxes * kResBox;
    static constexpr int kStrBox = kWinStr * kRowBytes;
    static constexpr int kStrTile = kBoxes * kStrBox;
    static constexpr int kSlotBytes = 2 * kStrTile;
    static constexpr int kSlots = 4;
    static constexpr int kStages = D == 128 ? 2 : 1;
    static constexpr int kBlocksPerSm = D == 128 ? 1 : 2;
    static constexpr int kSoftWarps = 8 * kStages;
    static constexpr int kThreads = 32 * (kSoftWarps + 2);
    static constexpr int kOffRing = 2 * kResTile;
    static constexpr int kOffStat = kOffRing + kSlots * kSlotBytes;   // per group: 2 buffers of -lse[64], -dvec[64]
    static constexpr int kOffBar = kOffStat + kStages * 2 * 2 * kWinStr * 4;
    static constexpr int kSmemBytes = kOffBar + 256;
    // TMEM columns: stage x has S at 128 x and dP at 128 x + 64; KV: then P of streamed rows 0..31 in the
    // first 16 columns of S, of rows 32..63 in the 16 from column 32 on, the upper part of dS likewise in dP
    // and the lower part in the 16 columns behind each
    static constexpr int kColAcc0 = 128 * kStages;
    static constexpr int kColAcc1 = kColAcc0 + D;
    static constexpr int kTmemCols = D == 128 ? 512 : 256;
    // dQ: the two parts of dS in columns of their own (a dQ block has one sum only): the next S and dP of a
    // stage then wait for its scores to be read, not for the products that read dS.
    static __device__ constexpr int col_apart(int x) { return D == 32 ? 192 : kColAcc0 + 64 * x; }
    static_assert(kColAcc1 + D <= kTmemCols, "TMEM budget");
    static_assert(kSmemBytes * kBlocksPerSm <= 226 * 1024, "shared memory budget");
};

struct WbParams {
    const __nv_bfloat16* q;     // [T, H, D]
    const __nv_bfloat16* k;     // [T, H_kv, D]
    const __nv_bfloat16* v;
    const __nv_bfloat16* o;     // forward output
    const __nv_bfloat16* dout;
    const float* lse;           // [T, H]
    void* dq;                   // [T, H, D] fp32 or bf16
    void* dk;                   // [T, H_kv, D]
    void* dv;
    float* dvec;                // [T, H] workspace
    float* dself;               // [T, H] workspace: dS of a candidate's own key
    float* part;                // workspace: pieces' sums [slot][dV, dK: 2 D / 4][128 rows][4]
    unsigned* counters;         // workspace: ended pieces of (segment, kv head, key tile, dV or dK)
    long long n_counters;
    const int* cu;
    const int* past;
    int B, H, Hkv, G, total_rows, max_rows;
    int tiles, sink_tiles;      // key tiles of max_rows, and how many of them may hold a sink
    int prep_rows;              // rows of a prep kernel's block
    int sink_pieces, win_pieces;   // most pieces of a KV block's sweep with and without sinks
    int window, n_sinks;
    int grad_fp32;
    unsigned n_kv;
    float scale, sl2;
    int* status;
    unsigned long long wait_limit_ns;
};

constexpr int kWbPrepThreads = 256;
constexpr int kWbPrepRows = 16;     // most rows of a block
constexpr int kWbFewKeys = 8;       // most keys of a row whose Dvec is summed over them (see above)
constexpr int kWbPrepHeads = 2;     // query heads of a candidate at a time
constexpr int kWbPrepUnroll = 4;    // query rows of a thread at a time: loads in flight

// Grid (blocks of rows, B); D / 8 lanes per query row, 16 bytes of it each.
template <int D>
__global__ void __launch_bounds__(kWbPrepThreads, 3) win_bwd_prep_kernel(const WbParams p)
{
    constexpr int L = D / 8;
    constexpr int kGroups = kWbPrepThreads / L;
    // the main kernel may start: its loads and first products need nothing from here, and what does waits
    // for this kernel's end
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    for (long long i = ((long long)blockIdx.y * gridDim.x + blockIdx.x) * kWbPrepThreads + threadIdx.x; i < p.n_counters;
         i += (long long)gridDim.x * gridDim.y * kWbPrepThreads)
        p.counters[i] = 0u;
    const int b = blockIdx.y;
    const WinSegment s = win_segment(p.cu, p.past, b, p.max_rows, p.total_rows);
    if (!s.ok && blockIdx.x == 0 && threadIdx.x == 0) report(p.status, (int)UNIPIN_ERR_OUT_OF_RANGE);
    const int r0 = blockIdx.x * p.prep_rows, r1 = min(r0 + p.prep_rows, s.len);
    if (!s.rows_ok || r0 >= r1) return;
    const int c = threadIdx.x % L, grp = threadIdx.x / L;
    if (!s.ok) {                                         // an out-of-range history length: zero gradients
        const float z[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        for (long long x = grp; x < (long long)(r1 - r0) * p.H; x += kGroups)
            win_store8(p.dq, p.grad_fp32, (((size_t)s.tok0 + r0) * p.H + x) * D + c * 8, z);
        for (long long x = grp; x < (long long)(r1 - r0) * p.Hkv; x += kGroups) {
            win_store8(p.dk, p.grad_fp32, (((size_t)s.tok0 + r0) * p.Hkv + x) * D + c * 8, z);
            win_store8(p.dv, p.grad_fp32, (((size_t)s.tok0 + r0) * p.Hkv + x) * D + c * 8, z);
        }
        return;
    }
    auto dot_lanes = [&](float x) {
#pragma unroll
        for (int off = L / 2; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
        return x;
    };
    auto dot8 = [&](uint4 a, uint4 b8) {
        float x[8], y[8], d = 0.f;
        win_unpack8(a, x);
        win_unpack8(b8, y);
#pragma unroll
        for (int e = 0; e < 8; ++e) d = fmaf(x[e], y[e], d);
        return d;
    };
    // Dvec of the block's query rows, which lie side by side
    {
        const long long rows = (long long)(r1 - r0) * p.H;
        const size_t q0 = ((size_t)s.tok0 + r0) * p.H;
        for (long long x0 = grp; x0 - grp < rows; x0 += kGroups * kWbPrepUnroll) {
            uint4 o4[kWbPrepUnroll], g4[kWbPrepUnroll];
#pragma unroll
            for (int i = 0; i < kWbPrepUnroll; ++i) {
                const long long x = x0 + i * kGroups;
                const size_t at = (q0 + (x < rows ? x : 0)) * D + c * 8;
                o4[i] = __ldg(reinterpret_cast<const uint4*>(p.o + at));
                g4[i] = __ldg(reinterpret_cast<const uint4*>(p.dout + at));
            }
#pragma unroll
            for (int i = 0; i < kWbPrepUnroll; ++i) {
                const long long x = x0 + i * kGroups;
                const float d = dot_lanes(dot8(o4[i], g4[i]));
                if (c == 0 && x < rows) p.dvec[q0 + x] = d;
            }
        }
    }
    // rows that see few keys: sum_j P_ij dO_i . v_j itself (each by the lanes that stored its dO . O)
    if (p.window <= kWbFewKeys || min(r0, s.n) < kWbFewKeys) {
        const int rows = (r1 - r0) * p.H;
        for (int x0 = grp; x0 - grp < rows; x0 += kGroups) {
            const int x = min(x0, rows - 1), row = r0 + x / p.H, h = x % p.H;
            // keys below sk and from lo to hi - 1, and a candidate's own
            const int lo = max(min(row, s.n) - p.window + 1, 0), hi = min(row + 1, s.n);
            const int sk = min(min(p.n_sinks, lo), hi);
            const int n = sk + max(hi - lo, 0) + (row >= s.n ? 1 : 0);
            const bool few = x0 < rows && n <= kWbFewKeys;
            if (!__any_sync(0xffffffffu, few)) continue;
            const size_t qr = ((size_t)s.tok0 + row) * p.H + h;
            const uint4 q4 = __ldg(reinterpret_cast<const uint4*>(p.q + qr * D + c * 8));
            const uint4 g4 = __ldg(reinterpret_cast<const uint4*>(p.dout + qr * D + c * 8));
            const float nl = win_neg_lse(p.lse[qr]);
            float d = 0.f;
            const int most = __reduce_max_sync(0xffffffffu, few ? n : 0);
            for (int y0 = 0; y0 < most; y0 += 4) {
                uint4 k4[4], v4[4];
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    int j = y0 + y < sk ? y0 + y : lo + y0 + y - sk;
                    if (j >= hi) j = row;
                    const size_t at = (((size_t)s.tok0 + j) * p.Hkv + h / p.G) * D + c * 8;
                    k4[y] = __ldg(reinterpret_cast<const uint4*>(p.k + at));
                    v4[y] = __ldg(reinterpret_cast<const uint4*>(p.v + at));
                }
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    const float qk = dot_lanes(dot8(q4, k4[y])), gv = dot_lanes(dot8(g4, v4[y]));
                    if (y0 + y < n) d = fmaf(ex2_approx(fmaf(qk, p.sl2, nl)), gv, d);
                }
            }
            if (few && c == 0) p.dvec[qr] = d;
        }
    }
    // candidates: their own key
    __syncthreads();                                     // Dvec of the block's rows
    const int c0 = max(r0, s.n);
    const int pairs = max(r1 - c0, 0) * p.Hkv;           // (at most 16 rows)
    for (int x = grp; x - grp < pairs; x += kGroups) {
        const bool live = x < pairs;
        const int row = c0 + (live ? x / p.Hkv : 0), hk = live ? x % p.Hkv : 0;
        const size_t tok = (size_t)s.tok0 + row, at = (tok * p.Hkv + hk) * D + c * 8;
        const uint4 k4 = __ldg(reinterpret_cast<const uint4*>(p.k + at));
        const uint4 v4 = __ldg(reinterpret_cast<const uint4*>(p.v + at));
        float dk[8], dv[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) dk[e] = dv[e] = 0.f;
#pragma unroll 1
        for (int g0 = 0; g0 < p.G; g0 += kWbPrepHeads) {
            uint4 q4[kWbPrepHeads], g4[kWbPrepHeads];
            float nl[kWbPrepHeads], dvec[kWbPrepHeads];
#pragma unroll
            for (int g = 0; g < kWbPrepHeads; ++g) {
                const size_t qr = tok * p.H + hk * p.G + min(g0 + g, p.G - 1);
                q4[g] = __ldg(reinterpret_cast<const uint4*>(p.q + qr * D + c * 8));
                g4[g] = __ldg(reinterpret_cast<const uint4*>(p.dout + qr * D + c * 8));
                nl[g] = win_neg_lse(p.lse[qr]);
                dvec[g] = p.dvec[qr];
            }
#pragma unroll
            for (int g = 0; g < kWbPrepHeads; ++g) {
                if (g0 + g >= p.G) break;
                const float qk = dot_lanes(dot8(q4[g], k4)), gv = dot_lanes(dot8(g4[g], v4));
                const float w = ex2_approx(fmaf(qk, p.sl2, nl[g]));
                const float ds = w * (gv - dvec[g]);
                if (live && c == 0) p.dself[tok * p.H + hk * p.G + g0 + g] = ds;
                float qf[8], gf[8];
                win_unpack8(q4[g], qf);
                win_unpack8(g4[g], gf);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    dk[e] = fmaf(p.scale * ds, qf[e], dk[e]);
                    dv[e] = fmaf(w, gf[e], dv[e]);
                }
            }
        }
        if (live) {
            win_store8(p.dk, p.grad_fp32, at, dk);
            win_store8(p.dv, p.grad_fp32, at, dv);
        }
    }
}

// What a block works on; every warp derives the same.
struct WbItem {
    int b, h;            // h: key/value head (KV) or query head (dQ)
    int r0;              // first resident row within the segment
    WinSweep sweep;      // the streamed tiles (KV: of each of the G query heads in turn)
    int first, total;    // the block's part of them: its first, and how many
    int piece, pieces;   // KV: which of how many pieces of the tile's sweep
    size_t slot, tile;   // KV: number of the tile's first piece (of the tiles that are cut), and of the tile
};

template <bool kKV>
__device__ __forceinline__ bool wb_item(const WbParams& p, unsigned block, WbItem& it, WinSegment& s)
{
    // tile-major: the longest sweeps (a KV block's first tile sees the most rows, a tile with sinks all) start first
    const int heads = kKV ? p.Hkv : p.H;
    const unsigned bh_count = (unsigned)p.B * heads;
    int t = (int)(block / bh_count);
    const unsigned bh = block - (unsigned)t * bh_count;
    it.b = (int)(bh / heads);
    it.h = (int)(bh - (unsigned)it.b * heads);
    it.piece = 0;
    int most = 1;
    if (kKV) {
        const int sinks = p.sink_tiles * p.sink_pieces;
        if (t < sinks) {
            most = p.sink_pieces;
            it.piece = t % most;
            t /= most;
            it.slot = ((size_t)bh * p.sink_tiles + t) * most;
        } else {
            most = p.win_pieces;
            t -= sinks;
            it.piece = t % most;
            t /= most;
            it.slot = (size_t)bh_count * (p.sink_pieces > 1 ? sinks : 0) + ((size_t)bh * (p.tiles - p.sink_tiles) + t) * most;
            t += p.sink_tiles;
        }
        it.tile = (size_t)bh * p.tiles + t;
    }
    it.r0 = t * kWinRes;
    s = win_segment(p.cu, p.past, it.b, p.max_rows, p.total_rows);
    if (!s.ok || it.r0 >= (kKV ? s.n : s.len)) return false;   // the prep kernel zeroed and reported bad segments
    it.sweep = kKV ? win_row_sweep(it.r0, s, p.window, p.n_sinks) : win_key_sweep(it.r0, s, p.window, p.n_sinks);
    it.total = kKV ? it.sweep.cnt * p.G : it.sweep.cnt;
    it.first = 0;
    it.pieces = 1;
    if (kKV && most > 1) {
        const int all = it.total, each = (all + most - 1) / most;
        it.pieces = (all + each - 1) / each;
        it.first = it.piece * each;
        it.total = min(each, all - it.first);
        if (it.total <= 0) return false;      // a piece behind the sweep's end
    }
    return true;
}

// All ones in the low (high) half where a (b) is negative.
__device__ __forceinline__ uint32_t wb_sign_pair(uint32_t a, uint32_t b)
{
    uint32_t d;
    asm("prmt.b32 %0, %1, %2, 0xffbb;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// One softmax pass over half a streamed tile: P and dS of this thread's resident row over 32 of the 64
// streamed rows, from S and dP in TMEM (32 columns at tS and at tS + 64) and back as bfloat16 pairs: P (KV)
// to tP, dS in two parts to tD (the upper 8 bits) and tL.  read(): the scores have been read; free(): the
// columns written may be (false: a timeout).  `see`: the columns that are allowed pairs.  kKV: -lse and
// -Dvec per column from shared memory, otherwise this row's own.
template <bool kKV, typename Read, typename Free>
__device__ __forceinline__ bool wb_softmax(uint32_t tS, uint32_t tP, uint32_t tD, uint32_t tL, Read read, Free free,
                                           float sl2, const float* nlse, const float* ndvec, float nl, float nd,
                                           uint32_t see)
{
    const uint64_t sc = f2_pack(sl2, sl2);
    const uint64_t nl2 = f2_pack(nl, nl), nd2 = f2_pack(nd, nd);
    const bool full = __all_sync(0xffffffffu, see == ~0u);
    uint32_t sr[32], dr[32], pk[16], dk[16], lk[16];
    if (!__any_sync(0xffffffffu, see != 0u)) {       // no pair of these 32 x 32
#pragma unroll
        for (int i = 0; i < 16; ++i) dk[i] = 0u;
        read();
        if (!free()) return false;
        if (kKV) tmem_st16_nowait(tP, dk);
        tmem_st16_nowait(tL, dk);
        tmem_st16(tD, dk);
        return true;
    }
    tmem_ld32x2(tS, sr, tS + kWinStr, dr);
    read();
#pragma unroll
    for (int e = 0; e < 32; e += 4) {
        uint64_t a[2], b[2];
        if (kKV) {
            const ulonglong2 x = *reinterpret_cast<const ulonglong2*>(nlse + e);
            const ulonglong2 y = *reinterpret_cast<const ulonglong2*>(ndvec + e);
            a[0] = x.x, a[1] = x.y, b[0] = y.x, b[1] = y.y;
        } else {
            a[0] = a[1] = nl2, b[0] = b[1] = nd2;
        }
#pragma unroll
        for (int f = 0; f < 2; ++f) {
            const int i = e + 2 * f;
            float x0, x1, d0, d1;
            f2_unpack(f2_fma(f2_pack(__uint_as_float(sr[i]), __uint_as_float(sr[i + 1])), sc, a[f]), x0, x1);
            f2_unpack(f2_add(f2_pack(__uint_as_float(dr[i]), __uint_as_float(dr[i + 1])), b[f]), d0, d1);
            const float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
            d0 *= p0;
            d1 *= p1;
            // the upper 8 bits of dS, and the rest rounded to as many
            const uint32_t b0 = __float_as_uint(d0), b1 = __float_as_uint(d1);
            dk[i / 2] = __byte_perm(b0, b1, 0x7632);
            lk[i / 2] = pack_bf16x2(d0 - __uint_as_float(b0 & 0xffff0000u), d1 - __uint_as_float(b1 & 0xffff0000u));
            if (kKV) pk[i / 2] = pack_bf16x2(p0, p1);
            if (!full) {
                // bits i, i + 1 of `see` as the signs of two bytes, spread over the pair's halves
                const uint32_t pair = wb_sign_pair(see << (31 - i), see << (30 - i));
                dk[i / 2] &= pair;
                lk[i / 2] &= pair;
                if (kKV) pk[i / 2] &= pair;
            }
        }
        if (kKV && e % 16 == 12) {                   // (as soon as they are there, for the registers)
            const int c = e / 16 * 8;
            tmem_st8_nowait(tP + c, pk + c);
            tmem_st8_nowait(tL + c, lk + c);
            tmem_st8_nowait(tD + c, dk + c);
        }
    }
    if (kKV) {
        tmem_st_wait();
        return true;
    }
    if (!free()) return false;
    tmem_st16_nowait(tL, lk);
    tmem_st16(tD, dk);
    return true;
}

template <int D, bool kKV>
__device__ __forceinline__ void wb_body(const CUtensorMap& tm_r0, const CUtensorMap& tm_r1, const CUtensorMap& tm_s0,
                                        const CUtensorMap& tm_s1, const WbParams& p, unsigned block, uint8_t* smem)
{
    using C = WbCfg<D>;
    const int warp = threadIdx.x / 32;
    const int lane = threadIdx.x % 32;
    if (warp == C::kSoftWarps && lane == 0) {
        tma_prefetch_map(&tm_r0);
        tma_prefetch_map(&tm_r1);
        tma_prefetch_map(&tm_s0);
        tma_prefetch_map(&tm_s1);
    }
    const int seen = status_seen(p.status);
    WbItem it;
    WinSegment s;
    const bool work = wb_item<kKV>(p, block, it, s);
    if (!work || block_timed_out(seen, (int)UNIPIN_ERR_DEVICE_TIMEOUT)) {
        asm volatile("griddepcontrol.wait;" ::: "memory");   // no block ends before the prep kernel
        return;
    }
    const int cnt = it.sweep.cnt;
    const int total = it.total;

    uint8_t* sRes = smem;
    uint8_t* ring = smem + C::kOffRing;
    float* stat = reinterpret_cast<float*>(smem + C::kOffStat);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
    uint64_t* bar_res = bars + 0;
    uint64_t* bar_drain = bars + 1;
    uint64_t* acc_done = bars + 2;
    uint64_t* s_ready = bars + 3;      // [2]
    uint64_t* p_ready = bars + 5;      // [2]
    uint64_t* grp = bars + 7;          // [2]
    uint64_t* s_free = bars + 9;       // [2] dQ: a stage's scores have been read
    uint64_t* p_free = bars + 11;      // [2] .. its dS
    uint64_t* full = bars + 13;        // [kSlots]
    uint64_t* empty = full + C::kSlots;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(empty + C::kSlots);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    volatile int* last_piece = reinterpret_cast<volatile int*>(tmem_slot + 2);   // [2]
    WaitCtl ctl{abort_flag, p.status, p.wait_limit_ns, (int)UNIPIN_ERR_DEVICE_TIMEOUT};
    const bool leader = lane == 0;
    constexpr bool kApart = !kKV;
    // streamed tile i = tile `idx` of query head `g` of the group, into its ring slot
    auto load_tile = [&](int i, int g, int idx) {
        const int st = i % C::kSlots;
        const int head = kKV ? it.h * p.G + g : it.h / p.G;
        const int row = s.tok0 + it.sweep.row(idx);
        uint8_t* dst = ring + st * C::kSlotBytes;
        mbar_arrive_expect_tx(full + st, C::kSlotBytes);
        for (int c = 0; c < C::kBoxes; ++c) {
            tma_load_3d(dst + c * C::kStrBox, &tm_s0, full + st, c * C::kBoxElems, head, row);
            tma_load_3d(dst + C::kStrTile + c * C::kStrBox, &tm_s1, full + st, c * C::kBoxElems, head, row);
        }
    };
    int pg = kKV && it.first > 0 ? it.first / cnt : 0;
    int pi = it.first - pg * cnt;      // producer: next tile's place
    if (warp == C::kSoftWarps) {
        if (leader) {
            mbar_init(bar_res, 1);
            mbar_init(bar_drain, 1);
            mbar_init(acc_done, 1);
            for (int x = 0; x < 2; ++x) {
                mbar_init(s_ready + x, 1);
                mbar_init(p_ready + x, 8);
                mbar_init(grp + x, 8);
                mbar_init(s_free + x, 8);
                mbar_init(p_free + x, 1);
            }
            for (int x = 0; x < C::kSlots; ++x) {
                mbar_init(full + x, 1);
                mbar_init(empty + x, 1);
            }
            *abort_flag = 0;
            fence_mbarrier_init();
            // the first loads need no other warp
            if (total > 0) {
                mbar_arrive_expect_tx(bar_res, 2 * C::kResTile);
                for (int c = 0; c < C::kBoxes; ++c) {
                    tma_load_3d(sRes + c * C::kResBox, &tm_r0, bar_res, c * C::kBoxElems, it.h, s.tok0 + it.r0);
                    tma_load_3d(sRes + C::kResTile + c * C::kResBox, &tm_r1, bar_res, c * C::kBoxElems, it.h,
                                s.tok0 + it.r0);
                }
            }
        }
        for (int i = 0; i < min(total, C::kSlots); ++i) {
            if (leader) load_tile(i, pg, pi);
            if (++pi == cnt) pi = 0, ++pg;
        }
    }
    if (warp == C::kSoftWarps + 1) {
        tmem_alloc(tmem_slot, C::kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = *tmem_slot;

    if (warp == C::kSoftWarps) {
        // ------------------------------------------------------------ producer
        int issued = min(total, C::kSlots);
        for (; issued < total; ++issued) {
            if (!__all_sync(0xffffffffu, mbar_wait(empty + issued % C::kSlots, (issued / C::kSlots - 1) & 1, ctl))) break;
            if (leader) load_tile(issued, pg, pi);
            if (++pi == cnt) pi = 0, ++pg;
        }
        if (leader && total > 0) {
            // every copy lands before the block exits
            mbar_wait_drain(bar_res, 0, p.wait_limit_ns);
            for (int v = (issued > C::kSlots ? issued - C::kSlots : 0); v < issued; ++v)
                mbar_wait_drain(full + v % C::kSlots, (v / C::kSlots) & 1, p.wait_limit_ns);
        }
    } else if (warp == C::kSoftWarps + 1) {
        // --------------------------------------------------------- MMA issuer
        constexpr uint32_t idesc_s = idesc_bf16_f32(kWinRes, kWinStr, false);
        constexpr uint32_t idesc_g = idesc_bf16_f32(kWinRes, D, true);       // A from TMEM, B MN-major
        constexpr int kStepsPerBox = C::kBoxElems / 16;
        const uint64_t d_r0 = smem_desc(smem_u32(sRes), 16, 8 * C::kRowBytes, C::kLayout);
        const uint64_t d_r1 = smem_desc(smem_u32(sRes) + C::kResTile, 16, 8 * C::kRowBytes, C::kLayout);
        const uint64_t d_s0 = smem_desc(smem_u32(ring), 16, 8 * C::kRowBytes, C::kLayout);
        const uint64_t d_s1 = smem_desc(smem_u32(ring) + C::kStrTile, 16, 8 * C::kRowBytes, C::kLayout);
        const uint64_t d_g0 = smem_desc(smem_u32(ring), C::kStrBox, 8 * C::kRowBytes, C::kLayout);
        const uint64_t d_g1 = smem_desc(smem_u32(ring) + C::kStrTile, C::kStrBox, 8 * C::kRowBytes, C::kLayout);
        auto landed = [&](int i) -> bool {
            return i >= total ||
                   __all_sync(0xffffffffu, mbar_wait(full + i % C::kSlots, (i / C::kSlots) & 1, ctl));
        };
        // S and dP of tile i (landed) into its stage, whose P and dS no product reads any more
        auto scores = [&](int i) {
            const int st = i % C::kSlots;
            if (elect_one()) {
                const uint32_t tS = tmem + (i % C::kStages) * 128;
                const uint64_t slot = (uint64_t)((st * C::kSlotBytes) >> 4);
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const int box = kk / kStepsPerBox, in = (kk % kStepsPerBox) * 32;
                    umma_bf16_ss(tS, d_r0 + (uint64_t)((box * C::kResBox + in) >> 4),
                                 d_s0 + slot + (uint64_t)((box * C::kStrBox + in) >> 4), idesc_s, kk > 0 ? 1u : 0u);
                }
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const int box = kk / kStepsPerBox, in = (kk % kStepsPerBox) * 32;
                    umma_bf16_ss(tS + kWinStr, d_r1 + (uint64_t)((box * C::kResBox + in) >> 4),
                                 d_s1 + slot + (uint64_t)((box * C::kStrBox + in) >> 4), idesc_s, kk > 0 ? 1u : 0u);
                }
                umma_commit(s_ready + i % C::kStages);
            }
        };
        bool ok = total == 0 || __all_sync(0xffffffffu, mbar_wait(bar_res, 0, ctl));
        for (int i = 0; ok && i < min(C::kStages, total); ++i) {
            if (!(ok = landed(i))) break;
            tc_fence_after_sync();
            scores(i);
        }
        for (int i = 0; ok && i < total; ++i) {
            const int x = i % C::kStages, st = i % C::kSlots;
            // kSlots > kStages: the later tile's load does not need this tile's slot
            if (!(ok = landed(i + C::kStages))) break;
            if (kApart && i + C::kStages < total) {
                ok = __all_sync(0xffffffffu, mbar_wait(s_free + x, (i / C::kStages) & 1, ctl));
                if (!ok) break;
                tc_fence_after_sync();
                scores(i + C::kStages);
            }
            ok = __all_sync(0xffffffffu, mbar_wait(p_ready + x, (i / C::kStages) & 1, ctl));
            if (!ok) break;
            tc_fence_after_sync();
            if (elect_one()) {
                const uint64_t slot = (uint64_t)((st * C::kSlotBytes) >> 4);
#pragma unroll
                for (int kk = 0; kk < kWinStr / 16; ++kk) {
                    // 16 streamed rows: 8 columns of pairs, those of rows 32.. at column 32
                    const uint32_t tP = tmem + x * 128 + (kk / 2) * 32 + (kk % 2) * 8;
                    const uint32_t tD = kApart ? tmem + C::col_apart(x) + kk * 8 : tP + kWinStr;
                    const uint32_t tL = tD + (kApart ? 32 : 16);
                    const uint64_t off = slot + (uint64_t)((kk * 16 * C::kRowBytes) >> 4);
                    const uint32_t acc = (i > 0 || kk > 0) ? 1u : 0u;
                    if (kKV) umma_bf16_ts(tmem + C::kColAcc0, tP, d_g1 + off, idesc_g, acc);
                    umma_bf16_ts(tmem + C::kColAcc1, tD, d_g0 + off, idesc_g, acc);
                    umma_bf16_ts(tmem + C::kColAcc1, tL, d_g0 + off, idesc_g, 1u);
                }
                umma_commit(empty + st);
                if (kApart) umma_commit(p_free + x);
                if (i + 1 == total) umma_commit(acc_done);
            }
            if (!kApart && i + C::kStages < total) {
                // only products into one accumulator are sure to run in order: S and dP over P and dS wait
                // for the products that read those
                ok = __all_sync(0xffffffffu, mbar_wait(empty + st, (i / C::kSlots) & 1, ctl));
                if (!ok) break;
                tc_fence_after_sync();
                scores(i + C::kStages);
            }
        }
        if (elect_one()) {
            umma_commit(bar_drain);
            mbar_wait_drain(bar_drain, 0, p.wait_limit_ns);
        }
    } else {
        // ------------------------------------------------- softmax + epilogue
        const int x = warp / 8;                      // stage
        const int half = (warp / 4) % 2;             // which 32 streamed rows of a tile
        const int t = (warp % 4) * 32 + lane;        // resident row
        const uint32_t lanes = tmem + (static_cast<uint32_t>((warp % 4) * 32) << 16);
        const int row = it.r0 + t;                   // within the segment
        asm volatile("griddepcontrol.wait;" ::: "memory");   // Dvec, dself and the counters
        const bool live = row < (kKV ? s.n : s.len);
        float nl = 0.f, nd = 0.f;
        // the resident row's allowed streamed rows: r < hi with r >= lo or r < sk
        int lo = 0, hi = 0, sk = 0;
        if (kKV) {
            // rows i >= key, min(i, n) - key < window (or any, for a sink)
            lo = row;
            hi = !live ? 0 : (row < p.n_sinks || s.n - row < p.window ? s.len : row + p.window);
        } else if (live) {
            const size_t at = ((size_t)s.tok0 + row) * p.H + it.h;
            nl = win_neg_lse(p.lse[at]);
            nd = -p.dvec[at];
            lo = max(min(row, s.n) - p.window + 1, 0);
            hi = min(row + 1, s.n);
            sk = p.n_sinks;
        }
        // KV: -lse and -Dvec of a streamed tile's rows: threads 0..63 of the group's first half the one,
        // 64..127 the other; fetched one tile ahead
        int idx = it.first + x, g = 0;               // place of the group's tile
        auto wrap = [&]() {
            while (idx >= cnt && g < p.G) idx -= cnt, ++g;
        };
        wrap();
        auto fetch = [&]() -> float {
            if (!kKV || half != 0 || g >= p.G) return 0.f;
            const int r = it.sweep.row(idx) + t % 64;
            if (r >= s.len) return 0.f;
            const size_t at = ((size_t)s.tok0 + r) * p.H + it.h * p.G + g;
            return t < 64 ? win_neg_lse(p.lse[at]) : -p.dvec[at];
        };
        float ahead = total > 0 ? fetch() : 0.f;
        uint32_t ngrp = 0;
        bool ok = true;
        for (int i = x; i < total; i += C::kStages) {
            const int k = i / C::kStages;
            float* st = stat + ((x * 2 + (k & 1)) * 2) * kWinStr;
            const int row0 = it.sweep.row(idx);
            idx += C::kStages;
            if (kKV) {
                wrap();
                if (half == 0) st[t] = ahead;
                ahead = fetch();
                if (!(ok = warp_group_sync(grp + x, ngrp, ctl, lane))) break;
            }
            const int c0 = row0 + half * 32;         // streamed row of this half's first column
            const uint32_t see = win_see32(lo - c0, hi - c0, sk - c0);
            ok = __all_sync(0xffffffffu, mbar_wait(s_ready + x, k & 1, ctl));
            if (!ok) break;
            tc_fence_after_sync();
            const uint32_t tS = lanes + x * 128 + half * 32;
            const uint32_t tD = kApart ? lanes + C::col_apart(x) + half * 16 : tS + kWinStr;
            auto read = [&]() {
                if (!kApart) return;
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(s_free + x);
            };
            auto free = [&]() -> bool {
                if (!kApart || k == 0) return true;
                if (!__all_sync(0xffffffffu, mbar_wait(p_free + x, (k - 1) & 1, ctl))) return false;
                tc_fence_after_sync();
                return true;
            };
            ok = wb_softmax<kKV>(tS, tS, tD, tD + (kApart ? 32 : 16), read, free, p.sl2, st + half * 32,
                                 st + kWinStr + half * 32, nl, nd, see);
            if (!ok) break;
            // streamed rows that are no row (KV: behind the segment) or no past key (dQ) become zeros
            const int end = (kKV ? s.len : s.n) - row0;
            if (end < kWinStr) {
                // the first half of the group clears T0's rows, the second T1's
                if (t < kWinStr && t >= end && (kKV || half == 0)) {
                    uint8_t* dst = ring + (i % C::kSlots) * C::kSlotBytes + half * C::kStrTile + t * C::kRowBytes;
#pragma unroll
                    for (int c = 0; c < C::kBoxes; ++c)
#pragma unroll
                        for (int a = 0; a < C::kRowBytes; a += 16)
                            *reinterpret_cast<uint4*>(dst + c * C::kStrBox + a) = make_uint4(0u, 0u, 0u, 0u);
                }
                fence_proxy_async_smem();
            }
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(p_ready + x);
        }
        if (ok && total > 0) {
            ok = __all_sync(0xffffffffu, mbar_wait(acc_done, 0, ctl));
            tc_fence_after_sync();
        }
        if (ok) {
            // (the TMEM loads are warp-collective: every lane loads)
            const size_t tok = (size_t)s.tok0 + row;
            if (kKV) {
                // 2 D accumulator columns over the block's groups of warps, dV first
                constexpr int kPart = 2 * D / (2 * C::kStages);
                const int c_first = (x * 2 + half) * kPart;
                const bool is_dk = c_first >= D;
                const float f = is_dk ? p.scale : 1.f;
                void* out = is_dk ? p.dk : p.dv;
                bool store = true;
                float* part = nullptr;
                if (it.pieces > 1) {
                    // this piece's sums; the piece that ends last adds them all up, in order
                    // (four columns of all rows side by side: a warp's accesses are contiguous)
                    part = p.part + it.slot * (2 * kWinRes * D) + ((size_t)c_first / 4 * kWinRes + t) * 4;
                    float* mine = part + (size_t)it.piece * (2 * kWinRes * D);
#pragma unroll
                    for (int c = 0; c < kPart; c += 32) {
                        uint32_t a[32];
                        tmem_ld32(lanes + C::kColAcc0 + c_first + c, a);
#pragma unroll
                        for (int e = 0; e < 32; e += 4)
                            *reinterpret_cast<uint4*>(mine + (c + e) * kWinRes) =
                                make_uint4(a[e], a[e + 1], a[e + 2], a[e + 3]);
                    }
                    __threadfence();
                    ok = warp_group_sync(grp + x, ngrp, ctl, lane);
                    if (ok && threadIdx.x % 256 == 0) {
                        const unsigned ended = atomicAdd(p.counters + it.tile * 2 + x, 1u);
                        __threadfence();
                        last_piece[x] = ended == (unsigned)(it.pieces - 1);
                    }
                    ok = ok && warp_group_sync(grp + x, ngrp, ctl, lane);
                    store = ok && last_piece[x];
                }
#pragma unroll
                for (int c = 0; c < kPart; c += 32) {
                    if (!store) break;
                    uint32_t a[32];
                    if (it.pieces > 1) {
#pragma unroll
                        for (int e = 0; e < 32; ++e) a[e] = 0u;
#pragma unroll 2
                        for (int y = 0; y < it.pieces; ++y) {
                            const float* from = part + (size_t)y * (2 * kWinRes * D) + c * kWinRes;
#pragma unroll
                            for (int e = 0; e < 32; e += 4) {
                                const float4 v = __ldcg(reinterpret_cast<const float4*>(from + e * kWinRes));
                                a[e] = __float_as_uint(__uint_as_float(a[e]) + v.x);
                                a[e + 1] = __float_as_uint(__uint_as_float(a[e + 1]) + v.y);
                                a[e + 2] = __float_as_uint(__uint_as_float(a[e + 2]) + v.z);
                                a[e + 3] = __float_as_uint(__uint_as_float(a[e + 3]) + v.w);
                            }
                        }
                    } else {
                        tmem_ld32(lanes + C::kColAcc0 + c_first + c, a);
                    }
                    if (!live) continue;
#pragma unroll
                    for (int e = 0; e < 32; e += 8) {
                        float o[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) o[i] = f * __uint_as_float(a[e + i]);
                        win_store8(out, p.grad_fp32, (tok * p.Hkv + it.h) * D + (c_first - (is_dk ? D : 0)) + c + e, o);
                    }
                }
            } else {
                const size_t at = tok * p.H + it.h;
                const bool cand = live && row >= s.n;
                const float ds = cand ? p.dself[at] : 0.f;
                // D columns in pieces of 32 over the groups of warps
#pragma unroll
                for (int c0 = 0; c0 < D; c0 += 32) {
                    if ((c0 / 32) % (2 * C::kStages) != x * 2 + half) continue;
                    uint32_t a[32];
                    if (total > 0) {
                        tmem_ld32(lanes + C::kColAcc1 + c0, a);
                    } else {
#pragma unroll
                        for (int e = 0; e < 32; ++e) a[e] = 0u;
                    }
                    if (!live) continue;
#pragma unroll
                    for (int e = 0; e < 32; e += 8) {
                        float o[8], kf[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) o[i] = __uint_as_float(a[e + i]);
                        if (cand) {
                            win_unpack8(__ldg(reinterpret_cast<const uint4*>(
                                            p.k + (tok * p.Hkv + it.h / p.G) * D + c0 + e)), kf);
#pragma unroll
                            for (int i = 0; i < 8; ++i) o[i] = fmaf(ds, kf[i], o[i]);
                        }
#pragma unroll
                        for (int i = 0; i < 8; ++i) o[i] *= p.scale;
                        win_store8(p.dq, p.grad_fp32, at * D + c0 + e, o);
                    }
                }
            }
        }
    }

    tc_fence_before_sync();
    __syncthreads();
    if (warp == C::kSoftWarps + 1) {
        __syncwarp();
        tc_fence_after_sync();
        tmem_dealloc(tmem, C::kTmemCols);
    }
}

// Maps: r = boxes of 128 rows, s = boxes of 64 rows.
template <int D>
__global__ void __launch_bounds__(WbCfg<D>::kThreads, WbCfg<D>::kBlocksPerSm)
    win_bwd_kernel(const __grid_constant__ CUtensorMap tm_qr, const __grid_constant__ CUtensorMap tm_gr,
                   const __grid_constant__ CUtensorMap tm_kr, const __grid_constant__ CUtensorMap tm_vr,
                   const __grid_constant__ CUtensorMap tm_qs, const __grid_constant__ CUtensorMap tm_gs,
                   const __grid_constant__ CUtensorMap tm_ks, const __grid_constant__ CUtensorMap tm_vs,
                   const __grid_constant__ WbParams p)
{
    extern __shared__ __align__(1024) uint8_t smem[];
    if ((smem_u32(smem) & 1023u) != 0) {
        if (threadIdx.x == 0) report(p.status, (int)UNIPIN_ERR_CUDA);
        return;
    }
    if (blockIdx.x < p.n_kv)
        wb_body<D, true>(tm_kr, tm_vr, tm_qs, tm_gs, p, blockIdx.x, smem);
    else
        wb_body<D, false>(tm_qr, tm_gr, tm_ks, tm_vs, p, blockIdx.x - p.n_kv, smem);
}

}  // namespace unipin
