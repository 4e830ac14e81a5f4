// Host side of the paged-pool entry points of include/unipin.h: the write of
// rows into pages, the one-token decode over pages and the eviction.
// Everything is asynchronous on the caller's stream; nothing allocates.
#include <cuda_runtime.h>

#include <climits>
#include <cmath>
#include <cstdint>
#include <mutex>

#include "unipin.h"
#include "host_util.h"
#include "paged_cache_sm100.cuh"
#include "paged_decode_sm100.cuh"

using namespace unipin;

namespace {

std::mutex g_paged_mutex;
bool g_paged_ready[kMaxDevices] = {};

constexpr int kSelKeysCap = 48 * 1024;   // keys of the selection's shared-memory copy (192 KB)
// Rows up to which the selection takes the smaller block (256 threads against 1024: 133 requests of 7 rows,
// H = 8, 13.9 and 33.9 us; 184 of 165, H = 2, 7.7 and 10.8; one of 1000, H = 8, 12.0 and 10.6).
constexpr int kSelShort = 512;

template <int D, int kMode, int kNG>
int set_decode_attr()
{
    return cudaFuncSetAttribute(paged_decode_kernel<D, kMode, kNG>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                PgCfg<D, kMode>::kSmemBytes) == cudaSuccess &&
                   cudaFuncSetAttribute(paged_decode_kernel<D, kMode, kNG>,
                                        cudaFuncAttributePreferredSharedMemoryCarveout,
                                        (int)cudaSharedmemCarveoutMaxShared) == cudaSuccess
               ? UNIPIN_OK
               : UNIPIN_ERR_CUDA;
}

template <int D>
int set_decode_attrs()
{
    int rc = set_decode_attr<D, kPgBf16, 1>();
    if (rc == UNIPIN_OK) rc = set_decode_attr<D, kPgBf16, 2>();
    if (rc == UNIPIN_OK) rc = set_decode_attr<D, kPgE4M3Pow2, 1>();
    if (rc == UNIPIN_OK) rc = set_decode_attr<D, kPgE4M3Pow2, 2>();
    if (rc == UNIPIN_OK) rc = set_decode_attr<D, kPgE4M3Any, 1>();
    if (rc == UNIPIN_OK) rc = set_decode_attr<D, kPgE4M3Any, 2>();
    return rc;
}

// Once per device: check it is an sm_100 part and raise the kernels' shared-memory limits.
int ensure_paged()
{
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return UNIPIN_ERR_CUDA;
    if (dev < 0 || dev >= kMaxDevices) return UNIPIN_ERR_UNSUPPORTED;
    std::lock_guard<std::mutex> lock(g_paged_mutex);
    if (g_paged_ready[dev]) return UNIPIN_OK;
    int major = 0, minor = 0;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess) return UNIPIN_ERR_CUDA;
    if (cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess) return UNIPIN_ERR_CUDA;
    if (major != 10 || minor != 0) return UNIPIN_ERR_UNSUPPORTED;
    int rc = set_decode_attrs<32>();
    if (rc == UNIPIN_OK) rc = set_decode_attrs<64>();
    if (rc == UNIPIN_OK) rc = set_decode_attrs<128>();
    if (rc == UNIPIN_OK && cudaFuncSetAttribute(paged_evict_select_kernel<kPgSelThreads>,
                                                cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                kSelKeysCap * 4) != cudaSuccess)
        rc = UNIPIN_ERR_CUDA;
    if (rc != UNIPIN_OK) return rc;
    g_paged_ready[dev] = true;
    return UNIPIN_OK;
}

// A kernel that may be scheduled while the one before it on the stream drains (it waits for that
// one's results itself, with griddepcontrol.wait).
template <typename P>
int launch_dependent(void (*kernel)(P), dim3 grid, int threads, size_t smem, cudaStream_t s, const P& p)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p) == cudaSuccess ? UNIPIN_OK : UNIPIN_ERR_CUDA;
}

int check_paged_pool(const unipin_kvpool* pool, int H, int layer)
{
    if (!pool) return UNIPIN_ERR_INVALID_ARG;
    if (!supported_d(pool->D)) return UNIPIN_ERR_UNSUPPORTED;
    const int rc = check_pool(pool, H, pool->D, layer);
    if (rc != UNIPIN_OK) return rc;
    // row numbers within a layer are 32-bit
    if ((uint64_t)pool->S * pool->H >= (1ull << 32) / (uint64_t)pool->n_cap) return UNIPIN_ERR_UNSUPPORTED;
    return UNIPIN_OK;
}

size_t elt_bytes(const unipin_kvpool* pool) { return pool->dtype == UNIPIN_POOL_E4M3 ? 1 : 2; }

uint8_t* layer_plane(const unipin_kvpool* pool, void* base, int layer)
{
    return static_cast<uint8_t*>(base) +
           (size_t)layer * pool->S * pool->H * pool->n_cap * pool->D * elt_bytes(pool);
}

float* layer_weights(const unipin_kvpool* pool, float* w, int layer)
{
    return w ? w + (size_t)layer * pool->S * pool->H * pool->n_cap : nullptr;
}

// A power of two with which value * scale is exact in bfloat16 for every E4M3 value.
bool pow2_scale(float s)
{
    int e = 0;
    return std::frexp(s, &e) == 0.5f && e >= -100 && e <= 100;
}

int decode_mode(const unipin_kvpool* pool)
{
    if (pool->dtype != UNIPIN_POOL_E4M3) return kPgBf16;
    return pow2_scale(pool->k_scale) && pow2_scale(pool->v_scale) ? kPgE4M3Pow2 : kPgE4M3Any;
}

struct DecodePlan {
    int vmax;      // most visible rows of a request
    int shares;    // blocks
    bool whole;    // every row within one block: no join kernel
};

struct DecodeShape {
    int blocks_per_sm, unit;
};

DecodeShape decode_shape(const unipin_kvpool* pool)
{
    const int row_bytes = (int)(pool->D * elt_bytes(pool));
    if (row_bytes >= 256) return {PgCfg<128, kPgBf16>::kBlocksPerSm, PgCfg<128, kPgBf16>::kUnit};
    if (row_bytes == 128) return {PgCfg<64, kPgBf16>::kBlocksPerSm, PgCfg<64, kPgBf16>::kUnit};
    return {PgCfg<32, kPgBf16>::kBlocksPerSm, PgCfg<32, kPgBf16>::kUnit};
}

// One wave of blocks.  Rows stay whole (no partials, no second launch) where they are short: up to two units,
// and up to 512 visible rows where the rows fill half of the device's blocks alone.  Whole and split, D = 64,
// H = 8: one request of 256 rows 6.9 and 7.4 us, of 500 8.7 and 7.7 us, of 1000 12.0 and 8.2 us; 32 requests
// of 256 7.9 and 9.7 us, of 500 10.0 and 13.6 us.
DecodePlan decode_plan(const unipin_kvpool* pool, int R, int H, int max_len, int window, int n_sinks, bool weights,
                       int sms)
{
    DecodePlan pl;
    long long vmax = (long long)window + n_sinks;
    if (vmax > max_len) vmax = max_len;
    pl.vmax = (int)vmax;
    const int G = H / pool->H;
    const long long pairs = (long long)R * pool->H * ((G + 15) / 16);
    const DecodeShape shape = decode_shape(pool);
    const long long units = vmax > 0 ? (vmax + shape.unit - 1) / shape.unit : 1;
    const long long slots = (long long)sms * shape.blocks_per_sm;
    pl.whole = !weights && (units <= 2 || (vmax <= 512 && 2 * pairs >= slots));
    const long long most = pl.whole ? pairs : pairs * units;
    pl.shares = (int)(most < slots ? most : slots);
    return pl;
}

size_t align256(size_t n) { return (n + 255) / 256 * 256; }

// Workspace: pieces' O [2 shares, heads, D] and (m, l), the requests' first units [R + 1]; with weights the
// rows' log sums [R * H] and the scores [R * H, vmax padded to 4].
struct DecodeSpace {
    size_t ml, first, lse, scores, bytes;
};

DecodeSpace decode_space(const DecodePlan& pl, int R, int H, int Hkv, int D, bool weights)
{
    DecodeSpace w = {};
    if (pl.whole) return w;
    const int G = H / Hkv;
    const size_t pieces = 2 * (size_t)pl.shares * (G < 16 ? G : 16), rows = (size_t)R * H;
    w.ml = align256(pieces * D * 4);
    w.first = w.ml + align256(pieces * 2 * 4);
    w.lse = w.first + align256(((size_t)R + 1) * 4);
    w.scores = w.lse + (weights ? align256(rows * 4) : 0);
    w.bytes = w.scores + (weights ? align256(rows * ((pl.vmax + 3) / 4 * 4) * 4) : 0);
    return w;
}

template <int D, int kMode>
int launch_decode(bool wide, const PgParams& p, cudaStream_t s)
{
    if (wide)
        paged_decode_kernel<D, kMode, 2><<<p.shares, kPgThreads, PgCfg<D, kMode>::kSmemBytes, s>>>(p);
    else
        paged_decode_kernel<D, kMode, 1><<<p.shares, kPgThreads, PgCfg<D, kMode>::kSmemBytes, s>>>(p);
    return cudaGetLastError() == cudaSuccess ? UNIPIN_OK : UNIPIN_ERR_CUDA;
}

template <int D>
int launch_decode_mode(int mode, bool wide, const PgParams& p, cudaStream_t s)
{
    switch (mode) {
    case kPgBf16: return launch_decode<D, kPgBf16>(wide, p, s);
    case kPgE4M3Pow2: return launch_decode<D, kPgE4M3Pow2>(wide, p, s);
    default: return launch_decode<D, kPgE4M3Any>(wide, p, s);
    }
}

}  // namespace

extern "C" {

int unipin_paged_pool_write(const unipin_kvpool* pool, int layer, const void* k, const void* v,
                            const int* cu_seqlens, const int* new_lens, const int* page_table, int max_pages,
                            const int* first_rows, int B, int max_new, int total_tokens, float* key_weights,
                            int* dev_status, void* stream)
{
    if (!pool || B < 0 || max_new < 0 || total_tokens < 0 || max_pages < 0) return UNIPIN_ERR_INVALID_ARG;
    int rc = check_paged_pool(pool, pool->H, layer);
    if (rc != UNIPIN_OK) return rc;
    if (B == 0 || max_new == 0 || total_tokens == 0) return UNIPIN_OK;
    if (!k || !v || !cu_seqlens || !new_lens || !page_table || !first_rows || max_pages < 1)
        return UNIPIN_ERR_INVALID_ARG;
    if (B > 65535) return UNIPIN_ERR_INVALID_ARG;
    if ((long long)max_new > (long long)max_pages * pool->n_cap) return UNIPIN_ERR_OUT_OF_RANGE;
    if (!aligned16(k) || !aligned16(v)) return UNIPIN_ERR_MISALIGNED;
    const long long per_block = (long long)kPgWriteThreads * kPgWriteVecs;
    const long long blocks = ((long long)max_new * pool->H * (pool->D / 8) + per_block - 1) / per_block;
    if (blocks >= (1ll << 31) || (long long)pool->H * (pool->D / 8) >= (1ll << 30)) return UNIPIN_ERR_INVALID_ARG;
    rc = ensure_paged();
    if (rc != UNIPIN_OK) return rc;
    PgWriteParams p = {};
    p.k = static_cast<const uint4*>(k);
    p.v = static_cast<const uint4*>(v);
    p.pool_k = layer_plane(pool, pool->k, layer);
    p.pool_v = layer_plane(pool, pool->v, layer);
    p.cu = cu_seqlens;
    p.new_lens = new_lens;
    p.table = page_table;
    p.first = first_rows;
    p.key_weights = layer_weights(pool, key_weights, layer);
    p.H = pool->H;
    p.D = pool->D;
    p.S = pool->S;
    p.ps = pool->n_cap;
    p.max_pages = max_pages;
    p.max_new = max_new;
    p.page_of = pg_divisor(pool->n_cap);
    p.token_of = pg_divisor(pool->H * (pool->D / 8));
    p.total_tokens = total_tokens;
    p.status = dev_status;
    const dim3 grid((unsigned)blocks, (unsigned)B, 1);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (pool->dtype == UNIPIN_POOL_E4M3) {
        p.inv_k = 1.f / pool->k_scale;
        p.inv_v = 1.f / pool->v_scale;
        paged_write_kernel<true><<<grid, kPgWriteThreads, 0, s>>>(p);
    } else {
        paged_write_kernel<false><<<grid, kPgWriteThreads, 0, s>>>(p);
    }
    return cudaGetLastError() == cudaSuccess ? UNIPIN_OK : UNIPIN_ERR_CUDA;
}

size_t unipin_paged_decode_workspace_size(const unipin_kvpool* pool, int R, int H, int max_len, int window,
                                          int n_sinks, int with_weights)
{
    if (!pool || pool->H < 1 || H < 1 || H % pool->H != 0 || !supported_d(pool->D) || R < 1 || max_len < 0 ||
        window < 1 || n_sinks < 0)
        return 0;
    const int sms = current_sms() > kNumSmsHint ? current_sms() : kNumSmsHint;
    const bool weights = with_weights != 0;
    return decode_space(decode_plan(pool, R, H, max_len, window, n_sinks, weights, sms), R, H, pool->H, pool->D,
                        weights)
        .bytes;
}

int unipin_paged_decode_attn(const void* q, const void* k_self, const void* v_self, void* out, int out_fp32,
                             const int* page_table, int max_pages, const int* lens, int R, int H, int D, int max_len,
                             int window, int n_sinks, float scale, const unipin_kvpool* pool, int layer,
                             float* key_weights, void* workspace, size_t workspace_bytes, int* dev_status,
                             void* stream)
{
    if (R < 0 || H < 1 || max_len < 0 || max_pages < 0 || window < 1 || n_sinks < 0) return UNIPIN_ERR_INVALID_ARG;
    if (!supported_d(D)) return UNIPIN_ERR_UNSUPPORTED;
    if (!(scale > 0.f) || !std::isfinite(scale)) return UNIPIN_ERR_INVALID_ARG;
    if (!pool || pool->D != D) return UNIPIN_ERR_INVALID_ARG;
    int rc = check_paged_pool(pool, H, layer);
    if (rc != UNIPIN_OK) return rc;
    if ((k_self == nullptr) != (v_self == nullptr)) return UNIPIN_ERR_INVALID_ARG;
    if (R == 0) return UNIPIN_OK;
    if (!q || !out || !lens || ((!page_table || max_pages < 1) && max_len > 0)) return UNIPIN_ERR_INVALID_ARG;
    if ((long long)max_len > (long long)max_pages * pool->n_cap) return UNIPIN_ERR_OUT_OF_RANGE;
    if (!aligned16(q) || !aligned16(k_self) || !aligned16(v_self) || !aligned16(out)) return UNIPIN_ERR_MISALIGNED;
    if (workspace && !aligned16(workspace)) return UNIPIN_ERR_MISALIGNED;
    const int G = H / pool->H, groups = (G + 15) / 16;
    const bool weights = key_weights != nullptr;
    DecodePlan pl = decode_plan(pool, R, H, max_len, window, n_sinks, weights, current_sms());
    // rows and units are numbered with 31 bits
    const long long units = (long long)R * pool->H * groups * ((pl.vmax + 63) / 64 + 1);
    if (R > 65535 || max_len > (1 << 30) || units >= (1ll << 31)) return UNIPIN_ERR_INVALID_ARG;
    if (weights && G > 8192) return UNIPIN_ERR_UNSUPPORTED;   // (the join keeps a group's statistics in shared memory)
    rc = ensure_paged();
    if (rc != UNIPIN_OK) return rc;
    DecodeSpace w = decode_space(pl, R, H, pool->H, D, weights);
    if (!pl.whole && (!workspace || workspace_bytes < w.bytes)) {
        if (weights) return UNIPIN_ERR_INVALID_ARG;     // the scores need a place
        pl.whole = true;                                // slower where few rows are long, same result
    }
    PgParams p = {};
    p.q = static_cast<const __nv_bfloat16*>(q);
    p.k_self = static_cast<const __nv_bfloat16*>(k_self);
    p.v_self = static_cast<const __nv_bfloat16*>(v_self);
    p.pool_k = layer_plane(pool, pool->k, layer);
    p.pool_v = layer_plane(pool, pool->v, layer);
    p.table = page_table;
    p.lens = lens;
    p.out = out;
    p.R = R;
    p.H = H;
    p.Hkv = pool->H;
    p.G = G;
    p.S = pool->S;
    p.ps = pool->n_cap;
    p.page_of = pg_divisor(pool->n_cap);
    p.max_pages = max_pages;
    p.max_len = max_len;
    p.window = window;
    p.n_sinks = n_sinks;
    p.heads = G < 16 ? G : 16;
    p.unit_shift = decode_shape(pool).unit == 64 ? 6 : 7;
    p.groups = groups;
    p.vmax = (pl.vmax + 3) / 4 * 4;
    p.whole = pl.whole ? 1 : 0;
    p.shares = pl.shares;
    p.out_fp32 = out_fp32 ? 1 : 0;
    const int mode = decode_mode(pool);
    p.sl2_self = scale * kPgLog2e;
    p.sl2 = mode == kPgE4M3Pow2 ? p.sl2_self * pool->k_scale : p.sl2_self;
    p.k_scale = pool->k_scale;
    p.v_scale = pool->v_scale;
    p.status = dev_status;
    if (!pl.whole) {
        char* ws = static_cast<char*>(workspace);
        p.part_o = reinterpret_cast<float*>(ws);
        p.part_ml = reinterpret_cast<float*>(ws + w.ml);
        p.first_unit = reinterpret_cast<int*>(ws + w.first);
        if (weights) {
            p.row_lse = reinterpret_cast<float*>(ws + w.lse);
            p.scores = reinterpret_cast<float*>(ws + w.scores);
            p.key_weights = layer_weights(pool, key_weights, layer);
        }
    }
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool wide = G > 8;
    if (D == 32) rc = launch_decode_mode<32>(mode, wide, p, s);
    else if (D == 64) rc = launch_decode_mode<64>(mode, wide, p, s);
    else rc = launch_decode_mode<128>(mode, wide, p, s);
    if (rc != UNIPIN_OK || pl.whole) return rc;
    const long long nw = weights ? (p.vmax + kPgWeightRows - 1) / kPgWeightRows : 0;
    const dim3 jgrid((unsigned)(H + pool->H * nw), (unsigned)R, 1);
    const size_t jsmem = weights ? (size_t)G * 4 : 0;
    if (D == 32) return launch_dependent(paged_join_kernel<32>, jgrid, 32 * kPgJoinWarps, jsmem, s, p);
    if (D == 64) return launch_dependent(paged_join_kernel<64>, jgrid, 32 * kPgJoinWarps, jsmem, s, p);
    return launch_dependent(paged_join_kernel<128>, jgrid, 32 * kPgJoinWarps, jsmem, s, p);
}

int unipin_paged_evict(const unipin_kvpool* pool, int layer, float* key_weights, const int* page_table,
                       int max_pages, const int* lens, int R, int max_len, int budget, int n_sinks, int n_recent,
                       int* kept, int* new_lens, int* dev_status, void* stream)
{
    if (!pool || R < 0 || max_len < 0 || max_pages < 0 || budget < 1 || n_sinks < 0 || n_recent < 0)
        return UNIPIN_ERR_INVALID_ARG;
    if ((long long)n_sinks + n_recent > budget) return UNIPIN_ERR_INVALID_ARG;
    int rc = check_paged_pool(pool, pool->H, layer);
    if (rc != UNIPIN_OK) return rc;
    if (R == 0) return UNIPIN_OK;
    if (!key_weights || !lens || !kept || !new_lens || ((!page_table || max_pages < 1) && max_len > 0) ||
        new_lens == lens)
        return UNIPIN_ERR_INVALID_ARG;
    if ((long long)max_len > (long long)max_pages * pool->n_cap) return UNIPIN_ERR_OUT_OF_RANGE;
    if (R > 65535 || pool->H > 65535 || max_len > (1 << 30) || budget > (1 << 30)) return UNIPIN_ERR_INVALID_ARG;
    rc = ensure_paged();
    if (rc != UNIPIN_OK) return rc;
    PgEvictParams p = {};
    p.pool_k = layer_plane(pool, pool->k, layer);
    p.pool_v = layer_plane(pool, pool->v, layer);
    p.key_weights = layer_weights(pool, key_weights, layer);
    p.table = page_table;
    p.lens = lens;
    p.kept = kept;
    p.new_lens = new_lens;
    p.H = pool->H;
    p.S = pool->S;
    p.ps = pool->n_cap;
    p.max_pages = max_pages;
    p.max_len = max_len;
    p.budget = budget;
    p.n_sinks = n_sinks;
    p.n_recent = n_recent;
    p.row_bytes = (int)(pool->D * elt_bytes(pool));
    p.page_of = pg_divisor(pool->n_cap);
    p.status = dev_status;
    p.keys_cap = max_len < kSelKeysCap ? max_len : kSelKeysCap;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const dim3 sgrid((unsigned)pool->H, (unsigned)R, 1);
    const size_t ssmem = (size_t)p.keys_cap * 4;
    if (max_len <= kSelShort)
        paged_evict_select_kernel<kPgSelThreadsShort><<<sgrid, kPgSelThreadsShort, ssmem, s>>>(p);
    else
        paged_evict_select_kernel<kPgSelThreads><<<sgrid, kPgSelThreads, ssmem, s>>>(p);
    if (cudaGetLastError() != cudaSuccess) return UNIPIN_ERR_CUDA;
    if (max_len <= budget) return UNIPIN_OK;
    if (p.row_bytes >= 64)
        return launch_dependent(paged_evict_move_kernel<4>,
                                dim3((unsigned)(2 * p.row_bytes / 64 + 1), (unsigned)pool->H, (unsigned)R), kPgMoveThreads,
                                0, s, p);
    return launch_dependent(paged_evict_move_kernel<2>, dim3(3, (unsigned)pool->H, (unsigned)R), kPgMoveThreads, 0, s,
                            p);
}

}  // extern "C"
