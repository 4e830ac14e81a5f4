// What the windowed prefill and its gradients share: segments, the streamed
// tiles of a block, masks as bits, rows of eight elements.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>

#include "sm100_ptx.cuh"

namespace unipin {

constexpr int kWinRes = 128;    // resident rows of a block = TMEM lanes
constexpr int kWinStr = 64;     // rows of a streamed tile

struct WinSegment {
    int tok0, len, n;
    bool rows_ok, ok;           // the rows lie inside the token tensors; so does the history in the rows
};

__device__ __forceinline__ WinSegment win_segment(const int* cu, const int* past, int b, int max_rows, int total_rows)
{
    WinSegment s;
    s.tok0 = cu[b];
    const long long len = (long long)cu[b + 1] - s.tok0;
    s.len = (int)len;
    s.n = past[b];
    s.rows_ok = s.tok0 >= 0 && len >= 0 && len <= max_rows && s.tok0 + len <= (long long)total_rows;
    s.ok = s.rows_ok && s.n >= 0 && s.n <= s.len;
    return s;
}

// The streamed tiles of a block: tile i begins at segment row first + 64 * (i < split ? i : i + jump).
struct WinSweep {
    int first, split, jump, cnt;
    __device__ int row(int i) const { return first + kWinStr * (i < split ? i : i + jump); }
};

// Key tiles that rows r0 .. r0 + 127 see: those of the sinks, then those from the first row's window on.
__device__ __forceinline__ WinSweep win_key_sweep(int r0, const WinSegment& s, int window, int n_sinks)
{
    WinSweep w;
    const int kmax = min(min(r0 + kWinRes, s.len), s.n);             // keys 0 .. kmax - 1
    const int low = max(min(r0, s.n) - window + 1, 0);               // first key of the first row's window
    const int t0 = low / kWinStr, t1 = (kmax + kWinStr - 1) / kWinStr;
    w.first = 0;
    w.split = min((int)(((long long)min(n_sinks, kmax) + kWinStr - 1) / kWinStr), t0);
    w.jump = t0 - w.split;
    w.cnt = w.split + max(t1 - t0, 0);
    return w;
}

// Row tiles that see keys r0 .. r0 + 127 (r0 < n): past rows as far as the last key's window reaches (all
// of them for a tile with a sink), then the candidates' if their window (or a sink) does.
__device__ __forceinline__ WinSweep win_row_sweep(int r0, const WinSegment& s, int window, int n_sinks)
{
    WinSweep w;
    const bool sink = r0 < n_sinks;
    const int last = min(r0 + kWinRes, s.n) - 1;                     // last key
    const int end = sink || s.n - last <= window ? s.n : last + window;
    const bool cand = sink || s.n - last < window;                   // a candidate stands at n
    w.first = r0;
    w.split = (end - r0 + kWinStr - 1) / kWinStr;
    const int c0 = max((s.n - r0) / kWinStr, w.split);
    const int c1 = (s.len - r0 + kWinStr - 1) / kWinStr;
    w.jump = c0 - w.split;
    w.cnt = w.split + (cand ? max(c1 - c0, 0) : 0);
    return w;
}

// Bits c = 0 .. 31 with c < n.
__device__ __forceinline__ uint32_t win_below32(int n)
{
    return n >= 32 ? ~0u : (1u << max(n, 0)) - 1u;
}

// Bits c with c < hi and (c >= lo or c < sk).
__device__ __forceinline__ uint32_t win_see32(int lo, int hi, int sk)
{
    return win_below32(hi) & (~win_below32(lo) | win_below32(sk));
}

// Eight bfloat16 (16 bytes) as floats.
__device__ __forceinline__ void win_unpack8(uint4 x, float (&f)[8])
{
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

// Eight elements at element offset `at`, as float32 or rounded to bfloat16.
__device__ __forceinline__ void win_store8(void* out, int fp32, size_t at, const float (&f)[8])
{
    if (fp32) {
        float4* dst = reinterpret_cast<float4*>(static_cast<float*>(out) + at);
        dst[0] = make_float4(f[0], f[1], f[2], f[3]);
        dst[1] = make_float4(f[4], f[5], f[6], f[7]);
    } else {
        *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(out) + at) =
            make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                       pack_bf16x2(f[6], f[7]));
    }
}

// -lse; a row that gave every score no weight (lse = -inf) keeps zero weights: 2^(s - inf).
__device__ __forceinline__ float win_neg_lse(float lse) { return lse == -INFINITY ? -INFINITY : -lse; }

}  // namespace unipin
