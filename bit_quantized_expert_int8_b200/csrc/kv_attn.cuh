// kv_attn.cuh -- attention over the 4-bit KV cache.
#pragma once
#include "kv_cache.cuh"

namespace moeq4 {

struct AttnArgs {
    KvArgs c;
    const __half* q;
    __half* out;
    float* lse;                // [n_rows][hq]
    long long q_stride, out_stride;
    float scale;
    int window;
};

// One element of K (part 0) or V (part 1).
__device__ __forceinline__ float kv_value(const uint8_t* tile, const KvTile& t, int part, int e, int d) {
    const int g = d >> 6, c = d & 63;
    const uint32_t w = *reinterpret_cast<const uint32_t*>(tile + t.codes(part, g, e) + (c >> 3) * 4);
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(tile + t.sb(part, g, e)));
    return fmaf(f.x, (float)((w >> (4 * (c & 7))) & 15u), f.y);
}

// One block per (row, query head): 64 entries at a time, scores by one thread
// each, then the running maximum and sum, then 64 entries into the block's
// head_dim columns.
__global__ void __launch_bounds__(256) k_attn_simple(const AttnArgs a) {
    const KvArgs& c = a.c;
    const int r = blockIdx.x, head = blockIdx.y, tid = threadIdx.x;
    const int D = c.ng * 64, h = head / (c.hq / c.hkv);
    const int s = kv_seq_of_row(c, r);
    if (s >= c.n_seqs) return;
    int first;
    const int n = kv_rows(c, s, &first, tid == 0);
    const int i = r - first;
    if (i < 0 || i >= n) return;
    const int p = kv_len(c, s, tid == 0) - n + i;
    const int j0 = a.window > 0 ? max(0, p - a.window + 1) : 0;
    __shared__ float sq[256], sp[kKvPage];
    const KvTile t(c.ng);
    if (tid < D) sq[tid] = __half2float(a.q[(size_t)r * a.q_stride + (size_t)head * D + tid]);
    __syncthreads();
    float m = -INFINITY, l = 0.f, o = 0.f;
    for (int pg = j0 / kKvPage; pg * kKvPage <= p; pg++) {
        const uint8_t* tile = kv_tile(c, s, pg, h);
        if (tid < kKvPage) {
            const int j = pg * kKvPage + tid;
            float x = -INFINITY;
            if (tile && j >= j0 && j <= p) {
                x = 0.f;
                for (int d = 0; d < D; d++) x = fmaf(sq[d], kv_value(tile, t, 0, tid, d), x);
                x *= a.scale;
            }
            sp[tid] = x;
        }
        __syncthreads();
        float mn = m;
        for (int e = 0; e < kKvPage; e++) mn = fmaxf(mn, sp[e]);
        const float ref = mn == -INFINITY ? 0.f : mn;
        const float f = expf(m - ref);
        o *= f;
        l *= f;
        m = mn;
        for (int e = 0; e < kKvPage; e++) {
            if (sp[e] == -INFINITY) continue;
            const float w = expf(sp[e] - ref);
            l += w;
            if (tid < D) o = fmaf(w, kv_value(tile, t, 1, e, tid), o);
        }
        __syncthreads();
    }
    if (tid < D)
        a.out[(size_t)r * a.out_stride + (size_t)head * D + tid] = __float2half_rn(l == 0.f ? 0.f : o / l);
    if (tid == 0) a.lse[(size_t)r * c.hq + head] = l == 0.f ? -INFINITY : m + logf(l);
}

// score[s][h][j] += sum over rows and heads of exp(S - lse): one thread per
// entry.  grid (max_pages, hkv, n_seqs), block 64.
__global__ void __launch_bounds__(kKvPage) k_attn_weights_simple(const AttnArgs a) {
    const KvArgs& c = a.c;
    const int pg = blockIdx.x, h = blockIdx.y, s = blockIdx.z, tid = threadIdx.x;
    const int len = kv_len(c, s, false), j = pg * kKvPage + tid;
    int first;
    const int n = kv_rows(c, s, &first, false);
    if (j >= len || n == 0) return;
    const uint8_t* tile = kv_tile(c, s, pg, h);
    if (!tile) return;
    const int D = c.ng * 64, G = c.hq / c.hkv;
    const KvTile t(c.ng);
    float sum = 0.f;
    for (int i = 0; i < n; i++) {
        const int p = len - n + i;
        if (j > p || (a.window > 0 && j <= p - a.window)) continue;
        for (int u = 0; u < G; u++) {
            const __half* q = a.q + (size_t)(first + i) * a.q_stride + (size_t)(h * G + u) * D;
            float x = 0.f;
            for (int d = 0; d < D; d++) x = fmaf(__half2float(q[d]), kv_value(tile, t, 0, tid, d), x);
            sum += expf(x * a.scale - a.lse[(size_t)(first + i) * c.hq + h * G + u]);
        }
    }
    c.score[((size_t)s * c.hkv + h) * ((size_t)c.max_pages * kKvPage) + j] += sum;
}

}  // namespace moeq4
