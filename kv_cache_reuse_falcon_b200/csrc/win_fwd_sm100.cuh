// The masked prefill under a sliding window with first rows that stay visible,
// on sm_100a.
//
// Row i of a segment of n past rows and its candidates stands at pos = min(i, n)
// and sees the past keys j <= i, j < n with pos - j < window or j < n_sinks, and
// a candidate its own key:
//   O_i = sum_j softmax_j(scale q_i . k_j) v_j
// One block per (segment, query head, 128 query rows): it visits the 64-key
// tiles of the sinks and of the rows' windows and no others.  Under a window a
// block's sweep is short (window / 64 + 3 tiles), so what the masked prefill's
// engine does for long sweeps (two query tiles per block, one persistent block
// per SM) leaves the SM waiting for one item's first loads, its chain of
// products and softmaxes and its epilogue; here several small blocks share an
// SM and fill each other's gaps (three at D <= 64, two at D = 128).
// Per key tile: S = Q K^T (tcgen05, TMEM: lane = row), the softmax warps (thread
// = row) read S, update the row maximum and sum (float32; O in TMEM is rescaled
// only when a maximum grows by more than 2^8), write P as bfloat16 over S
// (relative 2^-8), O += P V with P as A from TMEM.  At D = 128 S has two stages,
// so the next tile's S is computed while the softmax works; at D <= 64 one, and
// the other blocks' products run meanwhile.
// Warps: 0-3 softmax and epilogue, 4 TMA producer, 5 MMA issuer (owns TMEM).
// Bound: the chain of a tile (S, its load from TMEM, softmax, P's store, P V) with two blocks per SM to fill
// each other's gaps.  At D = 128, 16 segments of 500 .. 2048 past rows and 50 .. 256 candidates, H = 8, window
// 512, are 89 key tiles per SM and 2200 cycles each.  The products take about 660 of these (an M = 128, N = 64
// product from shared memory 50 cycles, where its rate is 32, P V's N = 128 65); the tensor pipe is busy 27% of
// the time, the issue slots 31%, the MUFU 23%, DRAM 22%.  Measured (B200): that case 99 us in a graph (40.4
// GFLOP of allowed pairs: 408 TFLOP/s, 25% of the rate of a large product; 191 MB); 2 segments of 300, D = 64,
// 10.3 us.  Two threads per row at D = 128 took 105 us, MMAs issued behind `lane == 0` and not elect.sync 110.
// The masked prefill's engine with a window took 162 us, but with its MMAs issued behind `lane == 0`; behind
// elect.sync it has not been measured.
// What a row does not see reaches nothing of it: masked scores are replaced, and
// rows of V that are no past key of the segment are zeroed in shared memory.  A
// value that is NaN or infinite can still reach a row of its tile that the mask
// keeps from it, as 0 * NaN in the product P V; so a row whose result is not
// finite is computed again from its visible keys alone (win_row_again).
#pragma once

#include "sm100_ptx.cuh"
#include "tmem_wide.cuh"
#include "unipin.h"
#include "win_common.cuh"

namespace unipin {

constexpr float kWfRescaleLog2 = 8.0f;   // rescale O only when a row max grows by > 2^8

template <int D>
struct WfCfg {
    static constexpr int kBoxElems = D >= 64 ? 64 : D;
    static constexpr int kBoxes = D / kBoxElems;
    static constexpr int kRowBytes = kBoxElems * 2;
    static constexpr uint32_t kLayout = D >= 64 ? kLayoutSw128 : kLayoutSw64;
    static constexpr int kQBox = kWinRes * kRowBytes;
    static constexpr int kQTile = kBoxes * kQBox;
    static constexpr int kKvBox = kWinStr * kRowBytes;
    static constexpr int kKvTile = kBoxes * kKvBox;
    // rings of K and of V tiles; K runs ahead by the stages of S, so at D = 128 it has one slot more
    static constexpr int kKSlots = 3;
    static constexpr int kVSlots = D == 128 ? 2 : 3;
    static constexpr int kStages = D == 128 ? 2 : 1;               // of S
    static constexpr int kBlocksPerSm = D == 128 ? 2 : 3;
    static constexpr int kThreads = 192;
    static constexpr int kOffK = kQTile;
    static constexpr int kOffV = kOffK + kKSlots * kKvTile;
    static constexpr int kOffBar = kOffV + kVSlots * kKvTile;
    static constexpr int kSmemBytes = kOffBar + 256;
    // TMEM columns: the S stages (P over the first half of each), then O
    static constexpr int kColO = kStages * kWinStr;
    static constexpr int kTmemCols = D == 128 ? 256 : 128;
    static_assert(kColO + D <= kTmemCols, "TMEM budget");
    static_assert((kSmemBytes + 1024) * kBlocksPerSm <= 228 * 1024, "shared memory budget");
    static_assert(kTmemCols * kBlocksPerSm <= 512, "TMEM budget");
};

struct WfParams {
    const __nv_bfloat16* q;     // [T, H, D]
    const __nv_bfloat16* k;     // [T, H_kv, D]
    const __nv_bfloat16* v;
    void* out;                  // [T, H, D] fp32 or bf16
    float* lse;                 // [T, H] or null
    const int* cu;
    const int* past;
    int B, H, Hkv, G, total_rows, max_rows;
    int window, n_sinks;
    int out_fp32;
    unsigned blocks;
    float sl2;
    int* status;
    unsigned long long wait_limit_ns;
};

// q . k in log2 units, both rows of D bfloat16.
template <int D>
__device__ __forceinline__ float wf_score(const __nv_bfloat16* q, const __nv_bfloat16* k, float sl2)
{
    float a = 0.f, b = 0.f;
#pragma unroll
    for (int c = 0; c < D / 8; ++c) {
        float x[8], y[8];
        win_unpack8(__ldg(reinterpret_cast<const uint4*>(q) + c), x);
        win_unpack8(__ldg(reinterpret_cast<const uint4*>(k) + c), y);
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
            a = fmaf(x[e], y[e], a);
            b = fmaf(x[e + 1], y[e + 1], b);
        }
    }
    return (a + b) * sl2;
}

// A row whose result is not finite although its statistics are numbers, from its visible keys alone:
// O = sum_j 2^(s_j - lse) v_j, in pieces of eight elements (one thread; rare, so not fast).
template <int D>
__device__ __noinline__ void win_row_again(const WfParams& p, int tok0, int n, int row, int h, float lse)
{
    const size_t tok = (size_t)tok0 + row;
    const __nv_bfloat16* q = p.q + (tok * p.H + h) * D;
    const int hk = h / p.G;
    const int lo = max(min(row, n) - p.window + 1, 0), hi = min(row + 1, n), sk = min(p.n_sinks, lo);
    const float nl = win_neg_lse(lse);
    for (int c = 0; c < D / 8; ++c) {
        float o[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = 0.f;
        auto add = [&](int j) {
            const size_t at = (((size_t)tok0 + j) * p.Hkv + hk) * D;
            const float w = ex2_approx(wf_score<D>(q, p.k + at, p.sl2) + nl);
            float v[8];
            win_unpack8(__ldg(reinterpret_cast<const uint4*>(p.v + at) + c), v);
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e] = fmaf(w, v[e], o[e]);
        };
        for (int j = 0; j < min(sk, hi); ++j) add(j);
        for (int j = lo; j < hi; ++j) add(j);
        if (row >= n) add(row);
        win_store8(p.out, p.out_fp32, (tok * p.H + h) * D + c * 8, o);
    }
}

template <int D>
__global__ void __launch_bounds__(WfCfg<D>::kThreads, WfCfg<D>::kBlocksPerSm)
    win_fwd_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                   const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ WfParams p)
{
    using C = WfCfg<D>;
    extern __shared__ __align__(1024) uint8_t smem[];
    const int warp = threadIdx.x / 32;
    const int lane = threadIdx.x % 32;
    if (warp == 4 && lane == 0) {
        tma_prefetch_map(&tm_q);
        tma_prefetch_map(&tm_k);
        tma_prefetch_map(&tm_v);
    }
    const int seen = status_seen(p.status);
    if ((smem_u32(smem) & 1023u) != 0) {   // the layout needs 1024-byte aligned tiles
        if (threadIdx.x == 0) report(p.status, (int)UNIPIN_ERR_CUDA);
        return;
    }
    // the last rows of the segments, whose sweeps are the longest, come first
    const unsigned block = p.blocks - 1 - blockIdx.x;
    const unsigned bh_count = (unsigned)p.B * p.H;
    const int t0 = (int)(block / bh_count);
    const unsigned bh = block - (unsigned)t0 * bh_count;
    const int b = (int)(bh / p.H), h = (int)(bh - (unsigned)b * p.H);
    const int r0 = t0 * kWinRes;
    const WinSegment s = win_segment(p.cu, p.past, b, p.max_rows, p.total_rows);
    if (!s.ok && t0 == 0 && h == 0 && threadIdx.x == 0) report(p.status, (int)UNIPIN_ERR_OUT_OF_RANGE);
    if (!s.rows_ok || r0 >= s.len || block_timed_out(seen, (int)UNIPIN_ERR_DEVICE_TIMEOUT)) return;
    if (!s.ok) {
        // a history length out of range: zeros
        const float z[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        const int row = r0 + threadIdx.x;
        if (threadIdx.x < kWinRes && row < s.len)
            for (int c = 0; c < D / 8; ++c)
                win_store8(p.out, p.out_fp32, (((size_t)s.tok0 + row) * p.H + h) * D + c * 8, z);
        return;
    }
    const WinSweep sweep = win_key_sweep(r0, s, p.window, p.n_sinks);
    const int total = sweep.cnt;

    uint8_t* sQ = smem;
    uint8_t* sK = smem + C::kOffK;
    uint8_t* sV = smem + C::kOffV;
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
    uint64_t* bar_q = bars + 0;
    uint64_t* bar_drain = bars + 1;
    uint64_t* pv_done = bars + 2;
    uint64_t* s_ready = bars + 3;      // [2]
    uint64_t* p_ready = bars + 5;      // [2]
    uint64_t* k_full = bars + 7;       // [3]
    uint64_t* k_empty = bars + 10;
    uint64_t* v_full = bars + 13;
    uint64_t* v_empty = bars + 16;
    uint64_t* o_done = bars + 19;      // the last P V: O is final
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 20);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    const bool leader = lane == 0;
    WaitCtl ctl{abort_flag, p.status, p.wait_limit_ns, (int)UNIPIN_ERR_DEVICE_TIMEOUT};
    auto load_tile = [&](const CUtensorMap& map, uint8_t* dst, uint64_t* bar, int i) {
        mbar_arrive_expect_tx(bar, C::kKvTile);
        for (int c = 0; c < C::kBoxes; ++c)
            tma_load_3d(dst + c * C::kKvBox, &map, bar, c * C::kBoxElems, h / p.G, s.tok0 + sweep.row(i));
    };
    auto load_k = [&](int i) { load_tile(tm_k, sK + i % C::kKSlots * C::kKvTile, k_full + i % C::kKSlots, i); };
    auto load_v = [&](int i) { load_tile(tm_v, sV + i % C::kVSlots * C::kKvTile, v_full + i % C::kVSlots, i); };
    if (warp == 4 && leader) {
        mbar_init(bar_q, 1);
        mbar_init(bar_drain, 1);
        mbar_init(pv_done, 1);
        mbar_init(o_done, 1);
        for (int x = 0; x < 2; ++x) {
            mbar_init(s_ready + x, 1);
            mbar_init(p_ready + x, 4);
        }
        for (int x = 0; x < 3; ++x) {
            mbar_init(k_full + x, 1);
            mbar_init(k_empty + x, 1);
            mbar_init(v_full + x, 1);
            mbar_init(v_empty + x, 1);
        }
        *abort_flag = 0;
        fence_mbarrier_init();
        // the first loads need no other warp
        if (total > 0) {
            mbar_arrive_expect_tx(bar_q, C::kQTile);
            for (int c = 0; c < C::kBoxes; ++c)
                tma_load_3d(sQ + c * C::kQBox, &tm_q, bar_q, c * C::kBoxElems, h, s.tok0 + r0);
            for (int i = 0; i < min(total, C::kKSlots); ++i) {
                load_k(i);
                if (i < C::kVSlots) load_v(i);
            }
        }
    }
    if (warp == 5) {
        tmem_alloc(tmem_slot, C::kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = *tmem_slot;

    if (warp == 4) {
        // ------------------------------------------------------------ producer
        // in the order in which the slots come free: V of a tile behind the P V of the tile kVSlots before,
        // K behind the (earlier) S of the tile kKSlots before
        int nk = min(total, C::kKSlots), nv = min(total, C::kVSlots);
        bool ok = true;
        while (ok && (nk < total || nv < total)) {
            if (nv < total && nv - C::kVSlots < nk - C::kKSlots) {
                ok = __all_sync(0xffffffffu, mbar_wait(v_empty + nv % C::kVSlots, (nv / C::kVSlots - 1) & 1, ctl));
                if (ok && leader) load_v(nv);
                nv += ok;
            } else if (nk < total) {
                ok = __all_sync(0xffffffffu, mbar_wait(k_empty + nk % C::kKSlots, (nk / C::kKSlots - 1) & 1, ctl));
                if (ok && leader) load_k(nk);
                nk += ok;
            } else {
                ok = __all_sync(0xffffffffu, mbar_wait(v_empty + nv % C::kVSlots, (nv / C::kVSlots - 1) & 1, ctl));
                if (ok && leader) load_v(nv);
                nv += ok;
            }
        }
        if (leader && total > 0) {
            // every copy lands before the block exits
            mbar_wait_drain(bar_q, 0, p.wait_limit_ns);
            for (int i = max(nk - C::kKSlots, 0); i < nk; ++i)
                mbar_wait_drain(k_full + i % C::kKSlots, (i / C::kKSlots) & 1, p.wait_limit_ns);
            for (int i = max(nv - C::kVSlots, 0); i < nv; ++i)
                mbar_wait_drain(v_full + i % C::kVSlots, (i / C::kVSlots) & 1, p.wait_limit_ns);
        }
    } else if (warp == 5) {
        // --------------------------------------------------------- MMA issuer
        constexpr uint32_t idesc_s = idesc_bf16_f32(kWinRes, kWinStr, false);
        constexpr uint32_t idesc_o = idesc_bf16_f32(kWinRes, D, true);      // A from TMEM, B MN-major
        constexpr int kStepsPerBox = C::kBoxElems / 16;
        const uint64_t d_q = smem_desc(smem_u32(sQ), 16, 8 * C::kRowBytes, C::kLayout);
        const uint64_t d_k = smem_desc(smem_u32(sK), 16, 8 * C::kRowBytes, C::kLayout);
        const uint64_t d_v = smem_desc(smem_u32(sV), C::kKvBox, 8 * C::kRowBytes, C::kLayout);
        auto k_landed = [&](int i) -> bool {
            return i >= total ||
                   __all_sync(0xffffffffu, mbar_wait(k_full + i % C::kKSlots, (i / C::kKSlots) & 1, ctl));
        };
        // S of tile i (landed) into its stage, whose P no product reads any more
        auto scores = [&](int i) {
            if (elect_one()) {
                const uint64_t slot = (uint64_t)((i % C::kKSlots * C::kKvTile) >> 4);
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const int box = kk / kStepsPerBox, in = (kk % kStepsPerBox) * 32;
                    umma_bf16_ss(tmem + (i % C::kStages) * kWinStr, d_q + (uint64_t)((box * C::kQBox + in) >> 4),
                                 d_k + slot + (uint64_t)((box * C::kKvBox + in) >> 4), idesc_s, kk > 0 ? 1u : 0u);
                }
                umma_commit(s_ready + i % C::kStages);
                umma_commit(k_empty + i % C::kKSlots);
            }
        };
        bool ok = total == 0 || __all_sync(0xffffffffu, mbar_wait(bar_q, 0, ctl));
        for (int i = 0; ok && i < min(C::kStages, total); ++i) {
            if (!(ok = k_landed(i))) break;
            tc_fence_after_sync();
            scores(i);
        }
        for (int i = 0; ok && i < total; ++i) {
            const int x = i % C::kStages;
            // kKSlots > kStages: K of the later tile does not need this tile's slot.  The softmax has seen
            // this tile's V land before it says that P is there.
            ok = k_landed(i + C::kStages) &&
                 __all_sync(0xffffffffu, mbar_wait(p_ready + x, (i / C::kStages) & 1, ctl));
            if (!ok) break;
            tc_fence_after_sync();
            if (elect_one()) {
                const uint64_t slot = (uint64_t)((i % C::kVSlots * C::kKvTile) >> 4);
#pragma unroll
                for (int kk = 0; kk < kWinStr / 16; ++kk)
                    umma_bf16_ts(tmem + C::kColO, tmem + x * kWinStr + kk * 8,
                                 d_v + slot + (uint64_t)((kk * 16 * C::kRowBytes) >> 4), idesc_o,
                                 (i > 0 || kk > 0) ? 1u : 0u);
                umma_commit(v_empty + i % C::kVSlots);
                umma_commit(pv_done);
                if (i + 1 == total) umma_commit(o_done);
            }
            if (i + C::kStages < total) {
                // only products into one accumulator are sure to run in order: S over P waits for P V
                ok = __all_sync(0xffffffffu, mbar_wait(pv_done, i & 1, ctl));
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
        const int t = threadIdx.x;
        const int row = r0 + t;                      // within the segment
        const bool live = row < s.len;
        const uint32_t lanes = tmem + (static_cast<uint32_t>(warp * 32) << 16);
        const uint32_t tO = lanes + C::kColO;
        const size_t at = ((size_t)s.tok0 + row) * p.H + h;
        const size_t at_kv = ((size_t)s.tok0 + row) * p.Hkv + h / p.G;
        const bool self = live && row >= s.n;        // a candidate: its own key
        const float ss = self ? wf_score<D>(p.q + at * D, p.k + at_kv * D, p.sl2) : -INFINITY;
        // the row sees keys j < hi with j >= lo or j < sk
        const int lo = max(min(row, s.n) - p.window + 1, 0);
        const int hi = live ? min(row + 1, s.n) : 0;
        const float sl2 = p.sl2;
        float m = -INFINITY;     // reference max (log2 units) that P and O are relative to
        float l = 0.f;           // row sum relative to m
        bool odd = false;        // a visible score is NaN or +inf: so is the row
        bool ok = true;
        for (int i = 0; i < total; ++i) {
            const int x = i % C::kStages;
            const uint32_t tS = lanes + x * kWinStr;
            const int row0 = sweep.row(i);
            ok = __all_sync(0xffffffffu, mbar_wait(s_ready + x, (i / C::kStages) & 1, ctl));
            if (!ok) break;
            tc_fence_after_sync();
            uint32_t sc[kWinStr];
            tmem_ld64(tS, sc);
            // a warp's 32 rows by 32 keys at a time: under a short window a good part of a tile's have no
            // pair, and cost nothing
            uint32_t see[2];
            bool some[2];
            float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const int c0 = row0 + 32 * half;
                see[half] = win_see32(lo - c0, hi - c0, p.n_sinks - c0);
                some[half] = __any_sync(0xffffffffu, see[half] != 0u);
                if (!some[half]) continue;
                uint32_t* x = sc + 32 * half;
                if (!__all_sync(0xffffffffu, see[half] == ~0u)) {
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        if (!(see[half] >> e & 1u)) x[e] = 0xff800000u;   // -inf
                }
                float m0 = -INFINITY, m1 = -INFINITY;
#pragma unroll
                for (int e = 0; e < 32; e += 4) {
                    m0 = max3f<true>(m0, __uint_as_float(x[e]), __uint_as_float(x[e + 1]));
                    m1 = max3f<true>(m1, __uint_as_float(x[e + 2]), __uint_as_float(x[e + 3]));
                }
                mx[half] = fmax_nan(m0, m1);
            }
            const float m_tile = fmax_nan(mx[0], mx[1]) * sl2;
            odd = odd || !(m_tile < INFINITY);
            // move the reference max only when some row of the warp would see P > 2^8
            if (__any_sync(0xffffffffu, m_tile > m + kWfRescaleLog2)) {
                const float m_new = fmaxf(m, m_tile);
                const float corr = m == -INFINITY ? 0.f : ex2_approx(m - m_new);
                if (i > 0) {
                    ok = __all_sync(0xffffffffu, mbar_wait(pv_done, (i - 1) & 1, ctl));
                    if (!ok) break;
                    tc_fence_after_sync();
#pragma unroll
                    for (int c = 0; c < D; c += 8) {
                        uint32_t o[8];
                        tmem_ld8(tO + c, o);
#pragma unroll
                        for (int e = 0; e < 8; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * corr);
                        tmem_st8(tO + c, o);
                    }
                }
                l *= corr;
                m = m_new;
            }
            const float m_use = m == -INFINITY ? 0.f : m;
            // 2^x by the MUFU alone: the FMA-pipe polynomial for one pair in four, as in the masked prefill, was
            // slower here, where the MUFU is busy 23% of the time and the polynomial lengthens a tile's chain
            const uint64_t sc2 = f2_pack(sl2, sl2), nm2 = f2_pack(-m_use, -m_use);
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                uint32_t pk[16];
                if (some[half]) {
                    uint64_t acc[2] = {0ull, 0ull};
#pragma unroll
                    for (int c = 0; c < 16; ++c) {
                        const int e = half * 32 + 2 * c;
                        float p0, p1;
                        f2_unpack(f2_fma(f2_pack(__uint_as_float(sc[e]), __uint_as_float(sc[e + 1])), sc2, nm2), p0, p1);
                        p0 = ex2_approx(p0);
                        p1 = ex2_approx(p1);
                        acc[c & 1] = f2_add(acc[c & 1], f2_pack(p0, p1));
                        pk[c] = pack_bf16x2(p0, p1);
                    }
                    float a, c;
                    f2_unpack(f2_add(acc[0], acc[1]), a, c);
                    l += a + c;
                } else {
#pragma unroll
                    for (int c = 0; c < 16; ++c) pk[c] = 0u;
                }
                if (half == 0) tmem_st16_nowait(tS, pk);
                else tmem_st16(tS + 16, pk);
            }
            ok = __all_sync(0xffffffffu, mbar_wait(v_full + i % C::kVSlots, (i / C::kVSlots) & 1, ctl));
            if (!ok) break;
            // rows of V that are no past key of the segment become zeros
            const int end = s.n - row0;
            if (end < kWinStr) {
                if (t < kWinStr && t >= end) {
                    uint8_t* dst = sV + (i % C::kVSlots) * C::kKvTile + t * C::kRowBytes;
#pragma unroll
                    for (int c = 0; c < C::kBoxes; ++c)
#pragma unroll
                        for (int a = 0; a < C::kRowBytes; a += 16)
                            *reinterpret_cast<uint4*>(dst + c * C::kKvBox + a) = make_uint4(0u, 0u, 0u, 0u);
                }
                fence_proxy_async_smem();
            }
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(p_ready + x);
        }
        // the own value (half of it at D = 128, for the registers) is fetched before O is waited for
        constexpr int kAhead = D / 8 < 8 ? D / 8 : 8;
        uint4 own[kAhead];
#pragma unroll
        for (int c = 0; c < kAhead; ++c)
            own[c] = self ? __ldg(reinterpret_cast<const uint4*>(p.v + at_kv * D) + c) : make_uint4(0u, 0u, 0u, 0u);
        if (ok && total > 0) {
            ok = __all_sync(0xffffffffu, mbar_wait(o_done, 0, ctl));
            tc_fence_after_sync();
        }
        if (ok) {
            const float m_fin = fmaxf(m, ss);
            const float a = m == -INFINITY ? 0.f : ex2_approx(m - m_fin);
            const float w = ss == -INFINITY ? 0.f : ex2_approx(ss - m_fin);
            if (odd || !(ss < INFINITY)) l = __int_as_float(0x7fffffff);
            const float denom = l * a + w;
            const float inv = denom == 0.f ? 0.f : 1.f / denom;
            const float lse = m_fin + log2f(denom);
            if (live && p.lse) p.lse[at] = lse;
            float chk = 0.f;     // NaN once an element is not finite
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
                uint32_t o[32];
                if (c * 4 == kAhead) {
#pragma unroll
                    for (int i = 0; i < kAhead; ++i)
                        if (self) own[i] = __ldg(reinterpret_cast<const uint4*>(p.v + at_kv * D) + kAhead + i);
                }
                if (total > 0) {
                    tmem_ld32(tO + c * 32, o);       // warp-collective: every lane loads
                } else {
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[e] = 0u;
                }
                if (!live) continue;
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    float f[8], vf[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) f[e] = __uint_as_float(o[g * 8 + e]) * a;
                    if (self) {
                        win_unpack8(own[(c * 4 + g) % kAhead], vf);
#pragma unroll
                        for (int e = 0; e < 8; ++e) f[e] = fmaf(w, vf[e], f[e]);
                    }
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        f[e] *= inv;
                        chk = fmaf(f[e], 0.f, chk);
                    }
                    win_store8(p.out, p.out_fp32, at * D + c * 32 + g * 8, f);
                }
            }
            if (chk != chk && lse == lse) win_row_again<D>(p, s.tok0, s.n, row, h, lse);
        }
    }

    tc_fence_before_sync();
    __syncthreads();
    if (warp == 5) {
        __syncwarp();
        tc_fence_after_sync();
        tmem_dealloc(tmem, C::kTmemCols);
    }
}

}  // namespace unipin
