// kv_api.cu -- the C ABI of the 4-bit KV cache (declared in moeq4.h): argument
// checks, workspace and launches.  The arithmetic runs in kv_cache.cuh and
// kv_attn.cuh.
#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <mutex>
#include <new>

#include "common.cuh"
#include "kv_attn.cuh"
#include "kv_attn_tc.cuh"
#include "kv_cache.cuh"
#include "kv_weights.cuh"

using namespace moeq4;

// the library's per-thread error message (moe_last_error)
void moeq4_set_error(const char* msg);

static int kv_fail(int code, const char* fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof(buf), fmt, ap);
    va_end(ap);
    moeq4_set_error(buf);
    return code;
}

#define KV_CK(call)                                                                \
    do {                                                                           \
        cudaError_t e_ = (call);                                                   \
        if (e_ != cudaSuccess)                                                     \
            return kv_fail(MOE_ERR_CUDA, "%s: %s (%s:%d)", #call, cudaGetErrorString(e_), \
                           __FILE__, __LINE__);                                    \
    } while (0)

#define KV_TRY(expr)                   \
    do {                               \
        int rc_ = (expr);              \
        if (rc_ != MOE_OK) return rc_; \
    } while (0)

static inline bool kv_al(const void* p, uintptr_t n) { return ((uintptr_t)p & (n - 1)) == 0; }

// Launch that may be scheduled before the kernel ahead of it in the stream ends
// (every kernel here begins with kv_begin, which waits for it).
template <typename... P, typename... A>
static cudaError_t kv_launch(int cluster, void (*fn)(P...), dim3 grid, int threads, size_t smem, cudaStream_t s, A... args) {
    cudaLaunchConfig_t lc{};
    lc.gridDim = grid;
    lc.blockDim = dim3(threads);
    lc.dynamicSmemBytes = smem;
    lc.stream = s;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = cluster;
    at[1].val.clusterDim.y = 1;
    at[1].val.clusterDim.z = 1;
    lc.attrs = at;
    lc.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&lc, fn, static_cast<P>(args)...);
}

struct moe_kv {
    MoeKvConfig cfg{};
    int device = 0;
    int n_sms = 0;
    uint8_t* ws = nullptr;
    int* status = nullptr;     // [2]: what kernels report, a bounded wait that gave up
    float* lse = nullptr;      // [max_rows][n_q_heads], where the caller wants none
    float* part = nullptr;     // partial sums of the split attention
    int* count = nullptr;      // arrivals per cut item, zero between calls
    int split_ctas[2] = {0, 0};  // CTAs of the split kernel: 8-row and 16-row tiles
    int split_smem[2] = {0, 0};
    TileCut* cut = nullptr;    // [n_sms]
    unsigned long long wait_ns = kWaitNs;  // bound of the tile kernel's waits
};

// The split kernel of one head size and row-tile count.
typedef void (*SplitFn)(const SplitArgs);
struct SplitKernel {
    SplitFn fn;
    int smem, rows, part_floats;
};
template <int NG, int RT>
static SplitKernel split_of() {
    using Sh = SplitShape<NG, RT>;
    return {k_attn_split<NG, RT>, Sh::kSmem, Sh::kRows, Sh::kRows * (Sh::kD + 2)};
}
typedef void (*TileFn)(const TileArgs);
struct TileKernel {
    TileFn fn, join;
    int smem, part_floats;
};
template <int NG>
static TileKernel tile_of() {
    return {k_attn_tile<NG>, k_attn_join<NG>, TileShape<NG>::kSmem, kTileRows * (TileShape<NG>::kD + 2)};
}
static TileKernel tile_kernel(int ng) {
    static const TileKernel table[4] = {tile_of<1>(), tile_of<2>(), tile_of<3>(), tile_of<4>()};
    return table[ng - 1];
}
typedef void (*WtFn)(const AttnArgs);
struct WtKernel {
    WtFn fn;
    int smem, ctas;
};
template <int NG, bool MANY>
static WtKernel weights_of() {
    return {k_attn_weights<NG, MANY>, WtShape<NG, MANY>::kSmem, WtShape<NG, MANY>::kCtas};
}
static WtKernel weights_kernel(int ng, bool many) {
    static const WtKernel table[4][2] = {{weights_of<1, false>(), weights_of<1, true>()},
                                         {weights_of<2, false>(), weights_of<2, true>()},
                                         {weights_of<3, false>(), weights_of<3, true>()},
                                         {weights_of<4, false>(), weights_of<4, true>()}};
    return table[ng - 1][many];
}
static SplitKernel split_kernel(int ng, int rt) {
    static const SplitKernel table[4][2] = {{split_of<1, 1>(), split_of<1, 2>()},
                                            {split_of<2, 1>(), split_of<2, 2>()},
                                            {split_of<3, 1>(), split_of<3, 2>()},
                                            {split_of<4, 1>(), split_of<4, 2>()}};
    return table[ng - 1][rt - 1];
}

static int kv_check_cfg(const MoeKvConfig* c) {
    if (!c) return kv_fail(MOE_ERR_INVALID_ARG, "moe_kv_create: cfg is NULL");
    if (c->head_dim < 64 || c->head_dim > 256 || c->head_dim % 64)
        return kv_fail(MOE_ERR_UNSUPPORTED_SHAPE, "head_dim must be 64, 128, 192 or 256 (%d)", c->head_dim);
    if (c->n_kv_heads < 1 || c->n_kv_heads > 128 || c->n_q_heads < 1 || c->n_q_heads > 1024 ||
        c->n_q_heads % c->n_kv_heads)
        return kv_fail(MOE_ERR_UNSUPPORTED_SHAPE,
                       "need 1 <= n_kv_heads <= 128 and n_q_heads <= 1024 a multiple of it (%d, %d)",
                       c->n_kv_heads, c->n_q_heads);
    if (c->n_pages < 1 || c->max_pages < 1 || c->max_pages > 32768)
        return kv_fail(MOE_ERR_UNSUPPORTED_SHAPE, "need n_pages >= 1 and max_pages in 1..32768");
    if (c->max_seqs < 1 || c->max_seqs > 4096 || c->max_rows < 1 || c->max_rows > (1 << 20))
        return kv_fail(MOE_ERR_UNSUPPORTED_SHAPE, "need max_seqs in 1..4096 and max_rows in 1..1048576");
    if (c->reserved != 0) return kv_fail(MOE_ERR_INVALID_ARG, "reserved must be zero");
    return MOE_OK;
}

extern "C" size_t moe_kv_page_bytes(int n_kv_heads, int head_dim) {
    if (n_kv_heads < 1 || n_kv_heads > 128 || head_dim < 64 || head_dim > 256 || head_dim % 64) return 0;
    return (size_t)n_kv_heads * KvTile(head_dim / 64).bytes();
}

extern "C" int moe_kv_destroy(moe_kv* kv) {
    if (!kv) return MOE_OK;
    int dev = -1;
    cudaGetDevice(&dev);
    cudaSetDevice(kv->device);
    cudaDeviceSynchronize();
    if (kv->ws) cudaFree(kv->ws);
    if (dev >= 0) cudaSetDevice(dev);
    delete kv;
    return MOE_OK;
}

// Loads a kernel that nothing else here asks about, so that a context's first call
// may be captured.
template <typename F>
static cudaError_t kv_load(F* fn) {
    cudaFuncAttributes fa{};
    return cudaFuncGetAttributes(&fa, fn);
}

extern "C" int moe_kv_create(const MoeKvConfig* cfg, moe_kv** out) {
    if (!out) return kv_fail(MOE_ERR_INVALID_ARG, "moe_kv_create: out is NULL");
    *out = nullptr;
    KV_TRY(kv_check_cfg(cfg));
    moe_kv* kv = new (std::nothrow) moe_kv();
    if (!kv) return kv_fail(MOE_ERR_CUDA, "moe_kv_create: out of host memory");
    kv->cfg = *cfg;
    int optin = 0;
    cudaError_t e = cudaGetDevice(&kv->device);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&kv->n_sms, cudaDevAttrMultiProcessorCount, kv->device);
    if (e == cudaSuccess)
        e = cudaDeviceGetAttribute(&optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, kv->device);
    size_t off = 0;
    auto take = [&](size_t bytes) { const size_t o = off; off = (off + bytes + 255) / 256 * 256; return o; };
    const size_t o_status = take(2 * sizeof(int));
    const size_t o_lse = take((size_t)cfg->max_rows * cfg->n_q_heads * sizeof(float));
    // every kernel's shared memory limit is raised here: no later call changes it
    size_t part = 0, ctas = 0;
    for (int rt = 1; rt <= 2 && e == cudaSuccess; rt++) {
        const SplitKernel k = split_kernel(cfg->head_dim / 64, rt);
        int occ = 0;
        cudaFuncAttributes fa{};
        e = cudaFuncGetAttributes(&fa, k.fn);
        const int most = optin - (int)fa.sharedSizeBytes;
        if (e == cudaSuccess) e = cudaFuncSetAttribute(k.fn, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
        if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&occ, k.fn, kSplitThreads, k.smem);
        if (e == cudaSuccess && occ < 1) e = cudaErrorInvalidConfiguration;
        const size_t n = (size_t)kv->n_sms * (occ > 0 ? occ : 1);
        kv->split_ctas[rt - 1] = (int)n;
        // an item may be cut into as many parts as there are CTAs: their weights and totals
        // (two floats a row) have to fit as well
        kv->split_smem[rt - 1] = std::max(k.smem, (int)n * k.rows * 8);
        if (e == cudaSuccess && kv->split_smem[rt - 1] > most) e = cudaErrorInvalidConfiguration;
        if (2 * n * k.part_floats > part) part = 2 * n * k.part_floats;
        if (n > ctas) ctas = n;
    }
    if (e == cudaSuccess && (int64_t)cfg->max_rows * (cfg->n_q_heads / cfg->n_kv_heads) > kSplitMaxRows) {
        const TileKernel k = tile_kernel(cfg->head_dim / 64);
        e = cudaFuncSetAttribute(k.fn, cudaFuncAttributeMaxDynamicSharedMemorySize, k.smem);
        if (e == cudaSuccess) e = kv_load(k.join);
        part = std::max(part, (size_t)2 * kv->n_sms * k.part_floats);
    }
    const size_t o_part = take(part * sizeof(float));
    const size_t o_count = take(ctas * sizeof(int));
    const size_t o_cut = take((size_t)kv->n_sms * sizeof(TileCut));
    for (int many = 0; many < 2; many++) {
        const WtKernel k = weights_kernel(cfg->head_dim / 64, many);
        if (e == cudaSuccess) e = cudaFuncSetAttribute(k.fn, cudaFuncAttributeMaxDynamicSharedMemorySize, k.smem);
    }
    if (e == cudaSuccess) e = kv_load(k_kv_rows<true, 1>);
    if (e == cudaSuccess) e = kv_load(k_kv_rows<true, 8>);
    if (e == cudaSuccess) e = kv_load(k_kv_rows<false, 1>);
    if (e == cudaSuccess) e = kv_load(k_kv_rows<false, 8>);
    if (e == cudaSuccess) e = cudaMalloc(&kv->ws, off);
    // what begins as zeros: the status, the arrival counts and the cut items
    if (e == cudaSuccess) e = cudaMemsetAsync(kv->ws + o_status, 0, 2 * sizeof(int), cudaStreamPerThread);
    if (e == cudaSuccess) e = cudaMemsetAsync(kv->ws + o_count, 0, ctas * sizeof(int), cudaStreamPerThread);
    if (e == cudaSuccess) e = cudaMemsetAsync(kv->ws + o_cut, 0, (size_t)kv->n_sms * sizeof(TileCut), cudaStreamPerThread);
    if (e == cudaSuccess) e = cudaStreamSynchronize(cudaStreamPerThread);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(k_kv_evict, cudaFuncAttributeMaxDynamicSharedMemorySize, kEvictSmem);
    if (e != cudaSuccess) {
        const int rc = kv_fail(MOE_ERR_CUDA, "moe_kv_create: %s", cudaGetErrorString(e));
        moe_kv_destroy(kv);
        return rc;
    }
    kv->status = reinterpret_cast<int*>(kv->ws + o_status);
    kv->lse = reinterpret_cast<float*>(kv->ws + o_lse);
    kv->part = reinterpret_cast<float*>(kv->ws + o_part);
    kv->count = reinterpret_cast<int*>(kv->ws + o_count);
    kv->cut = reinterpret_cast<TileCut*>(kv->ws + o_cut);
    *out = kv;
    return MOE_OK;
}

static int kv_check_device(const moe_kv* kv, const char* who) {
    int dev = -1;
    KV_CK(cudaGetDevice(&dev));
    if (dev != kv->device)
        return kv_fail(MOE_ERR_INVALID_ARG, "%s: the context belongs to device %d, current is %d", who, kv->device, dev);
    return MOE_OK;
}

extern "C" int moe_kv_check(moe_kv* kv, moe_stream_t stream) {
    if (!kv) return kv_fail(MOE_ERR_INVALID_ARG, "moe_kv_check: NULL context");
    KV_TRY(kv_check_device(kv, "moe_kv_check"));
    int st[2] = {0, 0};
    KV_CK(cudaMemcpyAsync(st, kv->status, sizeof(st), cudaMemcpyDeviceToHost, stream));
    KV_CK(cudaStreamSynchronize(stream));
    if (st[0] == 0 && st[1] == 0) return MOE_OK;
    KV_CK(cudaMemsetAsync(kv->status, 0, sizeof(st), stream));
    if (st[1] != 0)                    // (the tile kernel's; the split kernel and its counts wait for nobody)
        return kv_fail(st[1], "a bounded device wait of an attention call gave up; its outputs are not valid");
    return kv_fail(st[0], "a KV cache kernel met a length, row start or page index outside its limits");
}

extern "C" int moe_kv_set_wait_ns(moe_kv* kv, unsigned long long ns) {
    if (!kv) return kv_fail(MOE_ERR_INVALID_ARG, "moe_kv_set_wait_ns: NULL context");
    if (ns < 1000ull || ns > 60000000000ull)
        return kv_fail(MOE_ERR_INVALID_ARG, "moe_kv_set_wait_ns: %llu ns outside 1 us .. 60 s", ns);
    kv->wait_ns = ns;
    return MOE_OK;
}

static int kv_check_cache(const moe_kv* kv, const MoeKvCache* c, int n_seqs, const char* who) {
    if (!c->pages || !c->page_table || !c->lens) return kv_fail(MOE_ERR_INVALID_ARG, "%s: NULL cache buffer", who);
    if (!kv_al(c->pages, 16)) return kv_fail(MOE_ERR_ALIGNMENT, "%s: pages must be 16-byte aligned", who);
    if (!kv_al(c->page_table, 4) || !kv_al(c->lens, 4) || !kv_al(c->score, 4) || !kv_al(c->pos, 4) ||
        !kv_al(c->seen, 4))
        return kv_fail(MOE_ERR_ALIGNMENT, "%s: misaligned cache buffer", who);
    if (c->pos && !c->seen) return kv_fail(MOE_ERR_INVALID_ARG, "%s: pos needs seen", who);
    if (n_seqs < 0 || n_seqs > kv->cfg.max_seqs)
        return kv_fail(MOE_ERR_UNSUPPORTED_SHAPE, "%s: n_seqs=%d outside 0..%d", who, n_seqs, kv->cfg.max_seqs);
    return MOE_OK;
}

static int kv_check_batch(const moe_kv* kv, const MoeKvBatch* b, const char* who) {
    if (!b->row_start || !kv_al(b->row_start, 4))
        return kv_fail(MOE_ERR_INVALID_ARG, "%s: row_start is NULL or misaligned", who);
    if (b->n_rows < 0 || b->n_rows > kv->cfg.max_rows)
        return kv_fail(MOE_ERR_UNSUPPORTED_SHAPE, "%s: n_rows=%d outside 0..%d", who, b->n_rows, kv->cfg.max_rows);
    if (b->max_q < 1) return kv_fail(MOE_ERR_INVALID_ARG, "%s: max_q must be >= 1", who);
    if (b->reserved != 0) return kv_fail(MOE_ERR_INVALID_ARG, "%s: reserved must be zero", who);
    return MOE_OK;
}

static int kv_check_rows(const void* p, int64_t stride, int heads, int D, const char* who) {
    if (!p) return kv_fail(MOE_ERR_INVALID_ARG, "%s: NULL rows", who);
    if (!kv_al(p, 16)) return kv_fail(MOE_ERR_ALIGNMENT, "%s: rows must be 16-byte aligned", who);
    if (stride < (int64_t)heads * D || stride % 8 || stride > (int64_t)1 << 32)
        return kv_fail(MOE_ERR_INVALID_ARG, "%s: row stride %lld must be a multiple of 8, at least %d", who,
                       (long long)stride, heads * D);
    return MOE_OK;
}

// Whether two row arrays share bytes: their spans meet, and they are not column
// ranges of rows of one stride.
static bool kv_overlap(const void* p, int64_t p_stride, int64_t p_width, const void* q, int64_t q_stride,
                       int64_t q_width, int64_t rows) {
    const int64_t a = (int64_t)(uintptr_t)p / 2, b = (int64_t)(uintptr_t)q / 2;
    if (a + (rows - 1) * p_stride + p_width <= b || b + (rows - 1) * q_stride + q_width <= a) return false;
    if (p_stride != q_stride) return true;
    const int64_t d = ((b - a) % p_stride + p_stride) % p_stride;          // q's first column in p's rows
    return d < p_width || d + q_width > p_stride;
}

static KvArgs kv_args(const moe_kv* kv, const MoeKvCache* c, const MoeKvBatch* b, int n_seqs) {
    KvArgs a{};
    a.pages = static_cast<uint8_t*>(c->pages);
    a.table = c->page_table;
    a.lens = c->lens;
    a.row_start = b ? b->row_start : nullptr;
    a.score = c->score;
    a.pos = c->pos;
    a.seen = c->seen;
    a.status = kv->status;
    a.stop = kv->status + 1;
    a.n_seqs = n_seqs;
    a.n_rows = b ? b->n_rows : 0;
    a.max_q = b ? (b->max_q < b->n_rows ? b->max_q : b->n_rows) : 0;
    a.hq = kv->cfg.n_q_heads;
    a.hkv = kv->cfg.n_kv_heads;
    a.ng = kv->cfg.head_dim / 64;
    a.n_pages = kv->cfg.n_pages;
    a.max_pages = kv->cfg.max_pages;
    return a;
}

static int kv_rows_call(moe_kv* kv, const MoeKvCache* cache, const MoeKvBatch* batch, moe_half* k,
                        int64_t k_stride, moe_half* v, int64_t v_stride, bool read, cudaStream_t s) {
    const char* who = read ? "moe_kv_read_q4" : "moe_kv_append_q4";
    if (!kv || !cache || !batch) return kv_fail(MOE_ERR_INVALID_ARG, "%s: NULL argument", who);
    if (batch->n_seqs == 0 || batch->n_rows == 0) return MOE_OK;
    KV_TRY(kv_check_cache(kv, cache, batch->n_seqs, who));
    KV_TRY(kv_check_batch(kv, batch, who));
    KV_TRY(kv_check_rows(k, k_stride, kv->cfg.n_kv_heads, kv->cfg.head_dim, who));
    KV_TRY(kv_check_rows(v, v_stride, kv->cfg.n_kv_heads, kv->cfg.head_dim, who));
    const int64_t width = (int64_t)kv->cfg.n_kv_heads * kv->cfg.head_dim;
    if (read && kv_overlap(k, k_stride, width, v, v_stride, width, batch->n_rows))
        return kv_fail(MOE_ERR_INVALID_ARG, "%s: k and v overlap", who);
    KV_TRY(kv_check_device(kv, who));
    const KvArgs a = kv_args(kv, cache, batch, batch->n_seqs);
    __half* kp = reinterpret_cast<__half*>(k);
    __half* vp = reinterpret_cast<__half*>(v);
    // 32 groups a warp where that still gives every SM 16 warps, else 4 (append and read in a
    // graph, 8 heads of 128: 64 rows 9.8 us with 32 and 5.3 with 4, 1,024 rows 18.3 and 11.9,
    // 16 chunks of up to 512 21.4 and 28.7)
    const int items = a.hkv * 2 * a.ng;
    const bool many = (int64_t)a.n_rows * ((items + 31) / 32) >= 16 * kv->n_sms;
    const int64_t jobs = (int64_t)a.n_rows * (many ? (items + 31) / 32 : (items + 3) / 4);
    const auto fn = read ? (many ? k_kv_rows<true, 8> : k_kv_rows<true, 1>) : many ? k_kv_rows<false, 8> : k_kv_rows<false, 1>;
    KV_CK(kv_launch(1, fn, dim3((unsigned)((jobs + kKvRowWarps - 1) / kKvRowWarps)), kKvRowThreads, 0, s, a, kp, k_stride, vp,
                    v_stride));
    return MOE_OK;
}

extern "C" int moe_kv_append_q4(moe_kv* kv, const MoeKvCache* cache, const MoeKvBatch* batch,
                                const moe_half* k, int64_t k_stride, const moe_half* v,
                                int64_t v_stride, moe_stream_t stream) {
    return kv_rows_call(kv, cache, batch, const_cast<moe_half*>(k), k_stride, const_cast<moe_half*>(v),
                        v_stride, false, stream);
}

extern "C" int moe_kv_read_q4(moe_kv* kv, const MoeKvCache* cache, const MoeKvBatch* batch, moe_half* k,
                              int64_t k_stride, moe_half* v, int64_t v_stride, moe_stream_t stream) {
    return kv_rows_call(kv, cache, batch, k, k_stride, v, v_stride, true, stream);
}

extern "C" int moe_attn_q4(moe_kv* kv, const MoeKvCache* cache, const MoeKvBatch* batch,
                           const moe_half* q, int64_t q_stride, float scale, int window, int flags,
                           moe_half* out, int64_t out_stride, float* lse, moe_stream_t stream) {
    const char* who = "moe_attn_q4";
    if (!kv || !cache || !batch) return kv_fail(MOE_ERR_INVALID_ARG, "%s: NULL argument", who);
    if (batch->n_seqs == 0 || batch->n_rows == 0) return MOE_OK;
    KV_TRY(kv_check_cache(kv, cache, batch->n_seqs, who));
    KV_TRY(kv_check_batch(kv, batch, who));
    KV_TRY(kv_check_rows(q, q_stride, kv->cfg.n_q_heads, kv->cfg.head_dim, who));
    KV_TRY(kv_check_rows(out, out_stride, kv->cfg.n_q_heads, kv->cfg.head_dim, who));
    const int64_t width = (int64_t)kv->cfg.n_q_heads * kv->cfg.head_dim;
    if (kv_overlap(q, q_stride, width, out, out_stride, width, batch->n_rows))
        return kv_fail(MOE_ERR_INVALID_ARG, "%s: q and out overlap", who);
    if (flags & ~MOE_ATTN_WEIGHTS) return kv_fail(MOE_ERR_INVALID_ARG, "%s: unknown flags 0x%x", who, flags);
    if (window < 0) return kv_fail(MOE_ERR_INVALID_ARG, "%s: window must be >= 0", who);
    // the kernels multiply it by powers of two between 2^-37 and 2^25 and by sums below 2^46:
    // neither the factors (0 times the -infinity of a masked entry) nor the scores leave fp32
    const float mag = std::fabs(scale);
    if (!(scale == 0.f || (mag >= 0x1p-32f && mag <= 0x1p32f)))
        return kv_fail(MOE_ERR_INVALID_ARG, "%s: scale must be 0 or between 2^-32 and 2^32 in size", who);
    if ((flags & MOE_ATTN_WEIGHTS) && !cache->score)
        return kv_fail(MOE_ERR_INVALID_ARG, "%s: MOE_ATTN_WEIGHTS needs cache->score", who);
    if (!kv_al(lse, 4)) return kv_fail(MOE_ERR_ALIGNMENT, "%s: misaligned lse", who);
    KV_TRY(kv_check_device(kv, who));
    AttnArgs a{};
    a.c = kv_args(kv, cache, batch, batch->n_seqs);
    a.q = reinterpret_cast<const __half*>(q);
    a.out = reinterpret_cast<__half*>(out);
    a.lse = lse ? lse : kv->lse;
    a.q_stride = q_stride;
    a.out_stride = out_stride;
    a.scale = scale;
    // as wide as the cache: every entry is seen, as without a window.  (Narrower ones keep
    // "entry - window" of rows before the first entry within 32 bits.)
    a.window = window < kv->cfg.max_pages * kKvPage ? window : 0;
    // sequences of many rows on the tile kernel, of few on the split kernel (each passes over
    // the other's); one sequence needs one of them
    const int64_t most = (int64_t)a.c.max_q * (a.c.hq / a.c.hkv);
    const bool tile = most > kSplitMaxRows;
    if (tile) {
        TileArgs y{a, kv->part, kv->cut, a.c.n_seqs == 1 ? 0 : kSplitMaxRows + 1, kv->wait_ns};
        const TileKernel k = tile_kernel(a.c.ng);
        KV_CK(kv_launch(1, k.fn, dim3(kv->n_sms), kTileThreads, k.smem, stream, y));
        KV_CK(kv_launch(1, k.join, dim3(kv->n_sms, kTileRows / 32, a.c.ng), kJoinThreads, 0, stream, y));
    }
    if (!tile || a.c.n_seqs > 1) {
        const int rt = most <= 8 ? 1 : 2;
        SplitArgs x{a, kv->part, kv->count, kSplitMaxRows};
        KV_CK(kv_launch(1, split_kernel(a.c.ng, rt).fn, dim3(kv->split_ctas[rt - 1]), kSplitThreads,
                        kv->split_smem[rt - 1], stream, x));
    }
    if (flags & MOE_ATTN_WEIGHTS) {
        const WtKernel k = weights_kernel(a.c.ng, most > kWtBlock);
        KV_CK(kv_launch(1, k.fn, dim3(k.ctas * kv->n_sms), kWtThreads, k.smem, stream, a));
    }
    return MOE_OK;
}

extern "C" int moe_kv_evict(moe_kv* kv, const MoeKvCache* cache, int n_seqs, int budget, int n_recent,
                            int32_t* new_lens, moe_stream_t stream) {
    const char* who = "moe_kv_evict";
    if (!kv || !cache) return kv_fail(MOE_ERR_INVALID_ARG, "%s: NULL argument", who);
    if (n_seqs == 0) return MOE_OK;
    if (!new_lens) return kv_fail(MOE_ERR_INVALID_ARG, "%s: NULL argument", who);
    KV_TRY(kv_check_cache(kv, cache, n_seqs, who));
    if (!cache->score || !cache->pos || !cache->seen)
        return kv_fail(MOE_ERR_INVALID_ARG, "%s: needs score, pos and seen", who);
    if (!kv_al(new_lens, 4)) return kv_fail(MOE_ERR_ALIGNMENT, "%s: misaligned new_lens", who);
    if (budget < 1 || n_recent < 0 || n_recent > budget)
        return kv_fail(MOE_ERR_INVALID_ARG, "%s: need 0 <= n_recent <= budget, budget >= 1", who);
    // the first CTA to run writes new_lens while others still read these
    const size_t per_seq = (size_t)kv->cfg.n_kv_heads * kv->cfg.max_pages * kKvPage;
    const struct { const void* p; size_t words; } in[] = {{cache->lens, 1}, {cache->seen, 1},
                                                          {cache->page_table, (size_t)kv->cfg.max_pages},
                                                          {cache->score, per_seq}, {cache->pos, per_seq}};
    for (const auto& b : in) {
        const uintptr_t p = (uintptr_t)b.p, q = (uintptr_t)new_lens;
        if (q < p + 4 * b.words * n_seqs && p < q + 4 * (size_t)n_seqs)
            return kv_fail(MOE_ERR_INVALID_ARG, "%s: new_lens overlaps another buffer of the cache", who);
    }
    if (kv->cfg.max_pages > 8192)
        return kv_fail(MOE_ERR_UNSUPPORTED_SHAPE, "%s: max_pages=%d above 8192", who, kv->cfg.max_pages);
    KV_TRY(kv_check_device(kv, who));
    const KvArgs a = kv_args(kv, cache, nullptr, n_seqs);
    // clusters: what fits the device at once (two CTAs per SM), parts of 2048 entries at least
    // (half of 16,384 entries, 64 pairs of sequence and head: one CTA a pair 146 us, 4 60, 8, which
    // no longer fit at once, 75; 16 of 4,112 entries, 256 pairs: 23 us with one, 129 with 8; 8 pairs
    // of 4,112: 17 to 19 us with 1, 2 or 8)
    const int cap = kv->cfg.max_pages * kKvPage;
    int parts = 1;
    while (parts < 8 && (int64_t)n_seqs * a.hkv * parts * 2 <= 2 * kv->n_sms && cap / (parts * 2) >= 2048) parts *= 2;
    KV_CK(kv_launch(parts, k_kv_evict, dim3(a.hkv * parts, n_seqs), kEvictThreads, evict_smem(evict_part(cap, parts)), stream,
                    a, budget, n_recent, new_lens));
    return MOE_OK;
}
