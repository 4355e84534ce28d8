// kv_cache.cuh -- the 4-bit KV cache: page layout, appending and reading rows,
// eviction by accumulated attention weight.  Layout and rules in moeq4.h.
#pragma once
#include "common.cuh"
#include "ptx.cuh"

namespace moeq4 {

constexpr int kKvPage = MOE_KV_PAGE;      // entries per page
constexpr int kKvGroupBytes = 32;         // codes of one entry's group of 64 columns

// Byte offsets inside one (page, kv head) tile of 4608 NG bytes.
struct KvTile {
    int ng;
    __host__ __device__ explicit KvTile(int ng_) : ng(ng_) {}
    __host__ __device__ int bytes() const { return 4608 * ng; }
    __host__ __device__ int part(int v) const { return v * 2304 * ng; }          // K 0, V 1
    __host__ __device__ int codes(int v, int g, int e) const { return part(v) + (g * kKvPage + e) * kKvGroupBytes; }
    __host__ __device__ int sb(int v, int g, int e) const { return part(v) + 2048 * ng + (g * kKvPage + e) * 4; }
};

struct KvArgs {
    uint8_t* pages;
    const int32_t* table;      // [n_seqs][max_pages]
    const int32_t* lens;
    const int32_t* row_start;
    float* score;
    int32_t* pos;
    const int32_t* seen;
    int* status;               // what kv_flag reports
    int* stop;                 // a bounded wait gave up
    int n_seqs, n_rows, max_q, hq, hkv, ng, n_pages, max_pages;
};

// The kernels of a decode step follow one another closely: each lets the next
// be scheduled early and waits here for the work before it, so launches overlap.
__device__ __forceinline__ void kv_begin() {
    griddep_launch_dependents();
    griddep_wait();
}

__device__ __forceinline__ void kv_flag(int* status) { atomicCAS(status, 0, MOE_ERR_INVALID_ARG); }

// Entries held by sequence s, clamped to what its page-table row can hold.
__device__ __forceinline__ int kv_len(const KvArgs& a, int s, bool report) {
    const int n = a.lens[s], cap = a.max_pages * kKvPage;
    if (n >= 0 && n <= cap) return n;
    if (report) kv_flag(a.status);
    return n < 0 ? 0 : cap;
}

// Rows of sequence s: first row and count (0 where row_start is not usable).
__device__ __forceinline__ int kv_rows(const KvArgs& a, int s, int* first, bool report) {
    const int r0 = a.row_start[s], r1 = a.row_start[s + 1];
    *first = r0;
    if (r0 >= 0 && r1 >= r0 && r1 <= a.n_rows && r1 - r0 <= a.max_q) return r1 - r0;
    if (report) kv_flag(a.status);
    return 0;
}

// Tile of (sequence s, page slot p, kv head h), or null where the page index
// is outside the pool.
__device__ __forceinline__ uint8_t* kv_tile(const KvArgs& a, int s, int p, int h) {
    const int pg = a.table[(size_t)s * a.max_pages + p];
    if ((unsigned)pg >= (unsigned)a.n_pages) {
        kv_flag(a.status);
        return nullptr;
    }
    return a.pages + ((size_t)pg * a.hkv + h) * (size_t)(4608 * a.ng);
}

// Sequence that owns row r: the count of row_start[1..n] at most r, taken by a
// whole warp with independent loads (a binary search would chain its loads).
__device__ __forceinline__ int kv_seq_of_row(const KvArgs& a, int r) {
    const int lane = threadIdx.x & 31;
    int n = 0;
    for (int j = 1 + lane; j <= a.n_seqs; j += 32) n += a.row_start[j] <= r ? 1 : 0;
    return warp_sum(n);
}

// ------------------------------------------------------ append and read --
// One block per row; eight lanes per group of 64 columns, one 16-byte load
// and one code word each.  READ turns the direction round.
constexpr int kKvRowThreads = 256;

template <bool READ>
__global__ void __launch_bounds__(kKvRowThreads)
k_kv_rows(const KvArgs a, __half* k, long long k_stride, __half* v, long long v_stride) {
    const int r = blockIdx.x;
    kv_begin();
    const int s = kv_seq_of_row(a, r);
    if (s >= a.n_seqs) return;                                  // behind the last sequence
    int first;
    const int n = kv_rows(a, s, &first, threadIdx.x == 0);
    const int i = r - first;
    if (i < 0 || i >= n) return;
    const int e = kv_len(a, s, threadIdx.x == 0) - n + i;
    if (e < 0) {
        if (threadIdx.x == 0) kv_flag(a.status);
        return;
    }
    const KvTile t(a.ng);
    const int pg = a.table[(size_t)s * a.max_pages + e / kKvPage];
    if ((unsigned)pg >= (unsigned)a.n_pages) {
        if (threadIdx.x == 0) kv_flag(a.status);
        return;
    }
    uint8_t* page = a.pages + (size_t)pg * a.hkv * t.bytes();
    const int en = e % kKvPage, w = threadIdx.x & 7;
    const int items = a.hkv * 2 * a.ng;
    for (int base = 0; base < items; base += kKvRowThreads / 8) {
        const int it = base + (threadIdx.x >> 3);
        const bool on = it < items;
        const int part = on ? it / (a.hkv * a.ng) : 0, hg = on ? it % (a.hkv * a.ng) : 0;
        const int h = hg / a.ng, g = hg % a.ng;
        uint8_t* tile = page + (size_t)h * t.bytes();
        uint32_t* cw = reinterpret_cast<uint32_t*>(tile + t.codes(part, g, en)) + w;
        __half2* sb = reinterpret_cast<__half2*>(tile + t.sb(part, g, en));
        uint4* x = reinterpret_cast<uint4*>((part ? v + (size_t)r * v_stride : k + (size_t)r * k_stride) +
                                            (size_t)h * a.ng * 64 + g * 64) + w;
        if (READ) {
            if (!on) continue;
            const float2 f = __half22float2(*sb);
            const uint32_t c = *cw;
            uint4 o;
            uint32_t* ow = reinterpret_cast<uint32_t*>(&o);
#pragma unroll
            for (int q = 0; q < 4; q++) {
                const __half2 p = __floats2half2_rn(fmaf(f.x, (float)((c >> (8 * q)) & 15u), f.y),
                                                    fmaf(f.x, (float)((c >> (8 * q + 4)) & 15u), f.y));
                ow[q] = *reinterpret_cast<const uint32_t*>(&p);
            }
            *x = o;
        } else {
            const uint4 in = on ? *x : make_uint4(0, 0, 0, 0);
            const uint32_t iw[4] = {in.x, in.y, in.z, in.w};
            float f[8];
            bool fin = true;
#pragma unroll
            for (int q = 0; q < 4; q++) {
                const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&iw[q]));
                f[2 * q] = p.x;
                f[2 * q + 1] = p.y;
                fin = fin && fabsf(p.x) <= 65504.f && fabsf(p.y) <= 65504.f;   // false for NaN
            }
            float lo = f[0], hi = f[0];
#pragma unroll
            for (int q = 1; q < 8; q++) {
                lo = fminf(lo, f[q]);
                hi = fmaxf(hi, f[q]);
            }
            int bad = fin ? 0 : 1;
#pragma unroll
            for (int o = 1; o < 8; o <<= 1) {
                lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
                hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
                bad |= __shfl_xor_sync(0xffffffffu, bad, o);
            }
            if (!on) continue;
            const __half sc = __float2half_rn(__fdiv_rn(hi - lo, 15.0f));
            const __half bi = __float2half_rn(lo);
            const float sf = __half2float(sc), bf = __half2float(bi);
            uint32_t c = 0;
            if (!bad && sf != 0.f) {
#pragma unroll
                for (int q = 0; q < 8; q++) {
                    const float u = rintf(__fdiv_rn(f[q] - bf, sf));
                    c |= (uint32_t)fminf(fmaxf(u, 0.f), 15.f) << (4 * q);
                }
            }
            *cw = c;
            if (w == 0) *sb = bad ? __halves2half2(__ushort_as_half(0x7FFF), __ushort_as_half(0x7FFF))
                                  : __halves2half2(sc, bi);
        }
    }
    if (!READ)
        for (int h = threadIdx.x; h < a.hkv; h += kKvRowThreads) {
            const size_t at = ((size_t)s * a.hkv + h) * ((size_t)a.max_pages * kKvPage) + e;
            if (a.score) a.score[at] = 0.f;
            if (a.pos) a.pos[at] = a.seen[s] - n + i;
        }
}

// -------------------------------------------------------------- eviction --
// One block per (kv head, sequence).  The budget-th largest rank of the
// entries is found by a radix selection on an order-preserving 32-bit key
// (11 + 11 + 10 bits, one histogram pass each); a bit per entry then says
// whether it stays.  The r-th staying entry behind the budget moves into the
// r-th free place below it; both are found through prefix counts over the
// words of bits, so no list leaves shared memory.
constexpr int kEvictThreads = 1024;
constexpr int kEvictBins = 2048;

// Rank of an entry: last tokens above all, then by score; NaN below all.
__device__ __forceinline__ uint32_t evict_key(float score, bool recent) {
    if (recent) return 0xFFFFFFFFu;
    if (!(score == score)) return 0u;
    const uint32_t u = __float_as_uint(score + 0.0f);           // -0 -> +0
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// words of bits, prefix counts, histogram, scan scratch
__host__ __device__ constexpr size_t evict_smem(int cap) {
    return (size_t)((cap + 31) / 32) * 8 + kEvictBins * 4 + 64 * 4;
}

__device__ __forceinline__ int block_exclusive_scan(int v, int* s_scan, int* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 31) s_scan[warp] = x;
    __syncthreads();
    if (warp == 0) {
        int t = s_scan[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, t, o);
            if (lane >= o) t += y;
        }
        s_scan[lane] = t;
    }
    __syncthreads();
    *total = s_scan[kEvictThreads / 32 - 1];
    return x - v + (warp ? s_scan[warp - 1] : 0);
}

__global__ void __launch_bounds__(kEvictThreads)
k_kv_evict(const KvArgs a, int budget, int n_recent, int32_t* __restrict__ new_lens) {
    extern __shared__ __align__(16) uint32_t ev_smem[];
    const int h = blockIdx.x, s = blockIdx.y, tid = threadIdx.x;
    const int cap = a.max_pages * kKvPage;
    kv_begin();
    const int len = kv_len(a, s, h == 0 && tid == 0);
    if (h == 0 && tid == 0) new_lens[s] = min(len, budget);
    if (len <= budget) return;
    const int words = (len + 31) / 32;
    uint32_t* bits = ev_smem;
    uint32_t* pre = bits + (cap + 31) / 32;
    uint32_t* hist = pre + (cap + 31) / 32;
    int* s_scan = reinterpret_cast<int*>(hist + kEvictBins);   // 32 words, then 2 of results
    int* s_res = s_scan + 32;
    const size_t at = ((size_t)s * a.hkv + h) * (size_t)cap;
    float* score = a.score + at;
    int32_t* pos = a.pos + at;
    const int since = a.seen[s] - n_recent;

    // the budget-th largest key T, and how many entries equal to T stay
    uint32_t prefix = 0, mask = 0;
    int need = budget;
    for (int pass = 0; pass < 3; pass++) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
        const int nb = pass == 2 ? 1024 : 2048;
        for (int b = tid; b < kEvictBins; b += kEvictThreads) hist[b] = 0;
        __syncthreads();
        for (int e = tid; e < len; e += kEvictThreads) {
            const uint32_t key = evict_key(score[e], pos[e] >= since);
            if ((key & mask) == prefix) atomicAdd(&hist[(key >> shift) & (nb - 1)], 1u);
        }
        __syncthreads();
        // bins from the top, two per thread
        const int b1 = kEvictBins - 1 - 2 * tid, b0 = b1 - 1;
        const int c1 = (int)hist[b1], c0 = (int)hist[b0];
        int total;
        const int above = block_exclusive_scan(c0 + c1, s_scan, &total);
        if (above < need && need <= above + c1) { s_res[0] = b1; s_res[1] = need - above; }
        else if (above + c1 < need && need <= above + c1 + c0) { s_res[0] = b0; s_res[1] = need - above - c1; }
        __syncthreads();
        prefix |= (uint32_t)s_res[0] << shift;
        mask |= (uint32_t)(nb - 1) << shift;
        need = s_res[1];
        __syncthreads();
    }
    // ties at T stay in index order: count them per word first
    const int lane = tid & 31;
    for (int w = tid >> 5; w < words; w += kEvictThreads / 32) {
        const int e = w * 32 + lane;
        const uint32_t key = e < len ? evict_key(score[e], pos[e] >= since) : 0u;
        const uint32_t up = __ballot_sync(0xffffffffu, e < len && key > prefix);
        const uint32_t eq = __ballot_sync(0xffffffffu, e < len && key == prefix);
        if (lane == 0) { bits[w] = up; pre[w] = eq; }
    }
    __syncthreads();
    const int per = (words + kEvictThreads - 1) / kEvictThreads;
    const int w0 = min(tid * per, words), w1 = min(w0 + per, words);
    int n = 0, total;
    for (int w = w0; w < w1; w++) n += __popc(pre[w]);
    int left = need - block_exclusive_scan(n, s_scan, &total);
    for (int w = w0; w < w1; w++) {
        uint32_t eq = pre[w], take = 0;
        while (eq && left > 0) {
            const uint32_t low = eq & (0u - eq);
            take |= low;
            eq ^= low;
            left--;
        }
        bits[w] |= take;
    }
    __syncthreads();
    // free places below the budget (bit 0 there), entries to move at or behind it
    // (bit 1 there): word-wise counts, free places first in the low half
    const auto holes = [&](int w) -> uint32_t {
        const int lo = w * 32;
        if (lo >= budget) return 0u;
        const uint32_t in = budget - lo >= 32 ? 0xFFFFFFFFu : (1u << (budget - lo)) - 1u;
        return ~bits[w] & in;
    };
    const auto movers = [&](int w) -> uint32_t {
        const int lo = w * 32;
        if (lo + 32 <= budget) return 0u;
        const uint32_t out = lo >= budget ? 0xFFFFFFFFu : ~((1u << (budget - lo)) - 1u);
        return bits[w] & out;
    };
    int nh = 0, nm = 0, th, tm;
    for (int w = w0; w < w1; w++) { nh += __popc(holes(w)); nm += __popc(movers(w)); }
    int ph = block_exclusive_scan(nh, s_scan, &th);
    const int pm = block_exclusive_scan(nm, s_scan, &tm);
    for (int w = w0; w < w1; w++) { pre[w] = (uint32_t)ph; ph += __popc(holes(w)); }
    __syncthreads();
    const KvTile t(a.ng);
    int rank = pm;
    const int bw = (budget + 31) / 32;                          // words that hold free places
    for (int w = w0; w < w1; w++) {
        uint32_t m = movers(w);
        while (m) {
            const int src = w * 32 + __ffs(m) - 1;
            m &= m - 1;
            int lo = 0, hi = bw - 1;                            // last word with pre <= rank
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if ((int)pre[mid] <= rank) lo = mid;
                else hi = mid - 1;
            }
            uint32_t f = holes(lo);
            for (int q = rank - (int)pre[lo]; q > 0; q--) f &= f - 1;
            const int dst = lo * 32 + __ffs(f) - 1;
            rank++;
            score[dst] = score[src];
            pos[dst] = pos[src];
            const uint8_t* ts = kv_tile(a, s, src / kKvPage, h);
            uint8_t* td = kv_tile(a, s, dst / kKvPage, h);
            if (!ts || !td) continue;
            for (int part = 0; part < 2; part++)
                for (int g = 0; g < a.ng; g++) {
                    const uint4* cs = reinterpret_cast<const uint4*>(ts + t.codes(part, g, src % kKvPage));
                    uint4* cd = reinterpret_cast<uint4*>(td + t.codes(part, g, dst % kKvPage));
                    cd[0] = cs[0];
                    cd[1] = cs[1];
                    *reinterpret_cast<uint32_t*>(td + t.sb(part, g, dst % kKvPage)) =
                        *reinterpret_cast<const uint32_t*>(ts + t.sb(part, g, src % kKvPage));
                }
        }
    }
}

}  // namespace moeq4
