// kv_cache.cuh -- the 4-bit KV cache: page layout, appending and reading rows,
// eviction by accumulated attention weight.  Layout and rules in moeq4.h.
#pragma once
#include <cooperative_groups.h>

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
// What other kernels of the stream write (pages, rows, lse) is therefore read with
// ordinary or L2 loads only: this kernel may be resident while it is written, and
// loads through the read-only path are not ordered behind the wait.
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

// Sequence that owns row r: the count of row_start[1..n] at most r, taken by a
// whole warp with independent loads (a binary search would chain its loads).
__device__ __forceinline__ int kv_seq_of_row(const KvArgs& a, int r) {
    const int lane = threadIdx.x & 31;
    int n = 0;
    for (int j = 1 + lane; j <= a.n_seqs; j += 32) n += a.row_start[j] <= r ? 1 : 0;
    return warp_sum(n);
}

// ------------------------------------------------------ append and read --
// A warp takes 4 N groups of 64 columns of one row (kv heads x K, V x groups):
// eight lanes a group, four groups at once, N times over with every load in
// flight before the first is used; an append loads its row while it still looks
// for the row's place (sequence, length, page: three dependent reads).  Bound by
// memory (128 bytes a group on the fp16 side, 36 on the other) with many rows, by
// that chain with few: then N = 1 spreads a row over as many warps as it has.
constexpr int kKvRowWarps = 4;
constexpr int kKvRowThreads = kKvRowWarps * 32;

template <bool READ, int N>
__global__ void __launch_bounds__(kKvRowThreads)
k_kv_rows(const KvArgs a, __half* k, long long k_stride, __half* v, long long v_stride) {
    constexpr int kKvRowGroups = 4 * N;
    const int lane = threadIdx.x & 31, w = lane & 7;
    const int items = a.hkv * 2 * a.ng, chunks = (items + kKvRowGroups - 1) / kKvRowGroups;
    const long long job = (long long)blockIdx.x * kKvRowWarps + (threadIdx.x >> 5);
    kv_begin();
    const int r = (int)(job / chunks), it0 = (int)(job % chunks) * kKvRowGroups + (lane >> 3);
    if (r >= a.n_rows) return;
    const int per = a.hkv * a.ng;                                // groups of K, then of V
    const auto row = [&](int it) {
        const bool is_v = it >= per;
        const int hg = is_v ? it - per : it;
        return reinterpret_cast<uint4*>((is_v ? v + (size_t)r * v_stride : k + (size_t)r * k_stride) + (size_t)hg * 64) + w;
    };
    uint4 in[N];
    if constexpr (!READ) {
#pragma unroll
        for (int n = 0; n < N; n++) {
            in[n] = make_uint4(0, 0, 0, 0);
            if (it0 + 4 * n < items) in[n] = *row(it0 + 4 * n);
        }
    }
    const int s = kv_seq_of_row(a, r);
    if (s >= a.n_seqs) return;                                  // behind the last sequence
    int first;
    const bool tell = job % chunks == 0 && lane == 0;
    const int n = kv_rows(a, s, &first, tell);
    const int i = r - first;
    if (i < 0 || i >= n) return;
    const int e = kv_len(a, s, tell) - n + i;
    if (e < 0) {
        if (tell) kv_flag(a.status);
        return;
    }
    const KvTile t(a.ng);
    const int pg = a.table[(size_t)s * a.max_pages + e / kKvPage];
    if ((unsigned)pg >= (unsigned)a.n_pages) {
        if (tell) kv_flag(a.status);
        return;
    }
    const int en = e % kKvPage;
    uint8_t* page = a.pages + (size_t)pg * a.hkv * t.bytes();
    const auto codes = [&](int it) {                            // this lane's code word, and the group's scale
        const int part = it >= per, hg = part ? it - per : it, h = hg / a.ng, g = hg - h * a.ng;
        uint8_t* tile = page + (size_t)h * t.bytes();
        return make_ulonglong2((unsigned long long)(reinterpret_cast<uint32_t*>(tile + t.codes(part, g, en)) + w),
                               (unsigned long long)(tile + t.sb(part, g, en)));
    };
    if constexpr (READ) {
        uint32_t cw[N], sb[N];
#pragma unroll
        for (int q = 0; q < N; q++) {
            if (it0 + 4 * q >= items) continue;
            const ulonglong2 at = codes(it0 + 4 * q);
            cw[q] = *reinterpret_cast<const uint32_t*>(at.x);
            sb[q] = *reinterpret_cast<const uint32_t*>(at.y);
        }
#pragma unroll
        for (int q = 0; q < N; q++) {
            if (it0 + 4 * q >= items) continue;
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&sb[q]));
            uint4 o;
            uint32_t* ow = reinterpret_cast<uint32_t*>(&o);
#pragma unroll
            for (int c = 0; c < 4; c++) {
                const __half2 p = __floats2half2_rn(fmaf(f.x, (float)((cw[q] >> (8 * c)) & 15u), f.y),
                                                    fmaf(f.x, (float)((cw[q] >> (8 * c + 4)) & 15u), f.y));
                ow[c] = *reinterpret_cast<const uint32_t*>(&p);
            }
            *row(it0 + 4 * q) = o;
        }
    } else {
#pragma unroll
        for (int q = 0; q < N; q++) {
            const uint32_t iw[4] = {in[q].x, in[q].y, in[q].z, in[q].w};
            float f[8];
            bool fin = true;
#pragma unroll
            for (int c = 0; c < 4; c++) {
                const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&iw[c]));
                f[2 * c] = p.x;
                f[2 * c + 1] = p.y;
                fin = fin && fabsf(p.x) <= 65504.f && fabsf(p.y) <= 65504.f;       // false for NaN
            }
            float lo = f[0], hi = f[0];
#pragma unroll
            for (int c = 1; c < 8; c++) {
                lo = fminf(lo, f[c]);
                hi = fmaxf(hi, f[c]);
            }
            int bad = fin ? 0 : 1;
#pragma unroll
            for (int o = 1; o < 8; o <<= 1) {
                lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
                hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
                bad |= __shfl_xor_sync(0xffffffffu, bad, o);
            }
            if (it0 + 4 * q >= items) continue;
            const __half sc = __float2half_rn(__fdiv_rn(hi - lo, 15.0f));
            const __half bi = __float2half_rn(lo);
            const float sf = __half2float(sc), bf = __half2float(bi);
            uint32_t c = 0;
            if (!bad && sf != 0.f) {
                // the correctly rounded quotient from the correctly rounded reciprocal and one
                // corrected step (P. Markstein, IBM J. Res. Dev. 34 (1990), theorem on division)
                const float rs = __frcp_rn(sf);
#pragma unroll
                for (int x = 0; x < 8; x++) {
                    const float d = f[x] - bf, q0 = d * rs;
                    const float u = rintf(fmaf(fmaf(-q0, sf, d), rs, q0));
                    c |= (uint32_t)fminf(fmaxf(u, 0.f), 15.f) << (4 * x);
                }
            }
            const ulonglong2 at = codes(it0 + 4 * q);
            *reinterpret_cast<uint32_t*>(at.x) = c;
            if (w == 0)
                *reinterpret_cast<__half2*>(at.y) = bad ? __halves2half2(__ushort_as_half(0x7FFF), __ushort_as_half(0x7FFF))
                                                        : __halves2half2(sc, bi);
        }
        if (job % chunks == 0)
            for (int h = lane; h < a.hkv; h += 32) {
                const size_t at = ((size_t)s * a.hkv + h) * ((size_t)a.max_pages * kKvPage) + e;
                if (a.score) a.score[at] = 0.f;
                if (a.pos) a.pos[at] = a.seen[s] - n + i;
            }
    }
}

// -------------------------------------------------------------- eviction --
// One cluster of CTAs per (kv head, sequence), each with an equal part of the
// entries.  The budget-th largest rank is found by a radix selection on an
// order-preserving 32-bit key (11 + 11 + 10 bits): every CTA counts its part,
// the counts meet in the cluster's first CTA through distributed shared memory,
// which finds the threshold.  A bit per entry then says whether it stays.  The r-th staying entry
// behind the budget moves into the r-th free place below it.  Each CTA of the
// cluster has an equal share of the ranks (and with them of the copying); the CTA
// that holds an entry's bit writes the entry into the list of the CTA that has its
// rank, by a store to distributed shared memory, which nobody waits for.  (Searching
// the other CTAs' prefix counts instead took 21 of 63 us for half of 16384 entries.)
// No list leaves shared memory.  The clusters are as large as fills the device (a cluster
// per pair alone leaves most SMs idle when there are few pairs).
constexpr int kEvictThreads = 512;
constexpr int kEvictBins = 2048;
constexpr int kEvictKeys = 16384;      // entries of a part whose keys are kept in shared memory

// Rank of an entry: last tokens above all, then by score; NaN below all.
__device__ __forceinline__ uint32_t evict_key(float score, bool recent) {
    if (recent) return 0xFFFFFFFFu;
    if (!(score == score)) return 0u;
    const uint32_t u = __float_as_uint(score + 0.0f);           // -0 -> +0
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Entries of one CTA at most, for a cluster of `parts`.
__host__ __device__ constexpr int evict_part(int cap, int parts) { return ((cap + parts - 1) / parts + 31) / 32 * 32; }
// Moves of one CTA that have room in its list at a time: all of a part of kEvictKeys / 2.
__host__ __device__ constexpr int evict_room(int part) { return (part < kEvictKeys / 2 ? part : kEvictKeys / 2) / 2; }
// histogram, the list of moves over the keys of a part (where these fit), bits, prefix counts
__host__ __device__ constexpr size_t evict_smem(int part) {
    return kEvictBins * 4 + (size_t)evict_room(part) * 16 + (size_t)(part / 32) * 4 + (size_t)(part / 32 + 2) * 4;
}

// The most that a part of 524288 entries (max_pages 8192) asks for, alone or in a cluster.
constexpr int kEvictSmem = 204 * 1024;
static_assert(evict_smem(524288) <= kEvictSmem && evict_smem(kEvictKeys) <= kEvictSmem, "eviction's shared memory");

__device__ __forceinline__ int block_exclusive_scan(int v, int* s_scan, int* total) {
    constexpr int W = kEvictThreads / 32;
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
    int before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < W; w++) {
        const int t = s_scan[w];
        before += w < warp ? t : 0;
        all += t;
    }
    *total = all;
    return x - v + before;
}

// What stays in word w of a part that begins at entry e0: free places below the
// budget, and entries to move at or behind it.
__device__ __forceinline__ uint32_t evict_holes(uint32_t bits, int lo, int budget) {
    if (lo >= budget) return 0u;
    return ~bits & (budget - lo >= 32 ? 0xFFFFFFFFu : (1u << (budget - lo)) - 1u);
}
__device__ __forceinline__ uint32_t evict_movers(uint32_t bits, int lo, int budget) {
    if (lo + 32 <= budget) return 0u;
    return bits & (lo >= budget ? 0xFFFFFFFFu : ~((1u << (budget - lo)) - 1u));
}

__global__ void __launch_bounds__(kEvictThreads)
k_kv_evict(const KvArgs a, int budget, int n_recent, int32_t* __restrict__ new_lens) {
    namespace cg = cooperative_groups;
    extern __shared__ __align__(16) uint32_t ev_smem[];
    __shared__ int s_scan[kEvictThreads / 32], s_res[2], s_cnt[3], s_hc[8], s_mc[8];
    const cg::cluster_group cluster = cg::this_cluster();
    const int C = (int)cluster.num_blocks(), me = (int)cluster.block_rank();
    const int h = blockIdx.x / C, s = blockIdx.y, tid = threadIdx.x, lane = tid & 31;
    const int cap = a.max_pages * kKvPage;
    kv_begin();
    const bool first = h == 0 && me == 0 && tid == 0;
    const int len = kv_len(a, s, first);
    if (first) new_lens[s] = min(len, budget);
    if (len <= budget) return;                                  // the whole cluster alike
    const int part_cap = evict_part(cap, C);
    uint32_t* hist = ev_smem;
    uint32_t* keys = hist + kEvictBins;
    int4* list = reinterpret_cast<int4*>(keys);                 // from and its page, to and its page; keys have been used
    uint32_t* bits = keys + 4 * evict_room(part_cap);
    uint32_t* pre = bits + part_cap / 32;
    const bool kept = part_cap <= kEvictKeys;
    const size_t at = ((size_t)s * a.hkv + h) * (size_t)cap;
    float* score = a.score + at;
    int32_t* pos = a.pos + at;
    const int since = a.seen[s] - n_recent;
    const int part = evict_part(len, C);
    const int e0 = min(me * part, len), n = min(len - e0, part), words = (n + 31) / 32;
    const auto key_of = [&](int i) { return evict_key(score[e0 + i], pos[e0 + i] >= since); };
    if (kept)
        for (int i = tid; i < n; i += kEvictThreads) keys[i] = key_of(i);

    // the budget-th largest key T, and how many entries equal to T stay
    uint32_t prefix = 0, mask = 0;
    int need = budget;
    for (int pass = 0; pass < 3; pass++) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
        const uint32_t low = pass == 2 ? 1023u : 2047u;
        for (int b = tid; b < kEvictBins; b += kEvictThreads) hist[b] = 0;
        __syncthreads();
        for (int i = tid; i < n; i += kEvictThreads) {
            const uint32_t key = kept ? keys[i] : key_of(i);
            if ((key & mask) == prefix) atomicAdd(&hist[(key >> shift) & low], 1u);
        }
        __syncthreads();
        if (C > 1) {                                            // the parts' counts meet in the first CTA
            cluster.sync();
            uint32_t* h0 = cluster.map_shared_rank(hist, 0);
            for (int b = tid; me > 0 && b < kEvictBins; b += kEvictThreads)
                if (hist[b]) atomicAdd(h0 + b, hist[b]);
            cluster.sync();
        }
        if (me == 0) {                                          // four bins per thread, from the top
            constexpr int B = kEvictBins / kEvictThreads;
            const int top = kEvictBins - 1 - B * tid;
            int cnt[B], sum = 0, total;
#pragma unroll
            for (int k = 0; k < B; k++) sum += cnt[k] = (int)hist[top - k];
            int above = block_exclusive_scan(sum, s_scan, &total);
#pragma unroll
            for (int k = 0; k < B; k++) {
                if (above < need && need <= above + cnt[k]) {
                    s_res[0] = top - k;
                    s_res[1] = need - above;
                }
                above += cnt[k];
            }
        }
        if (C > 1) cluster.sync();
        else __syncthreads();
        const int* res = cluster.map_shared_rank(s_res, 0);
        prefix |= (uint32_t)res[0] << shift;
        mask |= low << shift;
        need = res[1];
    }
    // ties at T stay in index order
    for (int w = tid >> 5; w < words; w += kEvictThreads / 32) {
        const int i = w * 32 + lane;
        const uint32_t key = i < n ? (kept ? keys[i] : key_of(i)) : 0u;
        const uint32_t up = __ballot_sync(0xffffffffu, i < n && key > prefix);
        const uint32_t eq = __ballot_sync(0xffffffffu, i < n && key == prefix);
        if (lane == 0) { bits[w] = up; pre[w] = eq; }
    }
    __syncthreads();
    const int per = (words + kEvictThreads - 1) / kEvictThreads;
    const int w0 = min(tid * per, words), w1 = min(w0 + per, words);
    int ties = 0, all;
    for (int w = w0; w < w1; w++) ties += __popc(pre[w]);
    const int mine = block_exclusive_scan(ties, s_scan, &all);
    if (tid == 0) s_cnt[0] = all;
    cluster.sync();
    int left = need - mine;
    for (int r = 0; r < me; r++) left -= *cluster.map_shared_rank(&s_cnt[0], r);
    for (int w = w0; w < w1; w++) {
        uint32_t eq = pre[w], take = 0;
        if (__popc(eq) <= left) {
            take = eq;
            left -= __popc(eq);
        }
        for (; take != eq && left > 0; left--) {
            const uint32_t lowest = (eq & ~take) & (0u - (eq & ~take));
            take |= lowest;
        }
        bits[w] |= take;
    }
    // prefix counts: free places at pre[w], entries to move at pre[w + 1] (a word below the
    // budget has none to move, one behind it no free place, so the two never meet)
    int nh = 0, nm = 0, th, tm;
    for (int w = w0; w < w1; w++) {
        nh += __popc(evict_holes(bits[w], e0 + w * 32, budget));
        nm += __popc(evict_movers(bits[w], e0 + w * 32, budget));
    }
    int ph = block_exclusive_scan(nh, s_scan, &th);             // (its barriers: pre has been read)
    int pm = block_exclusive_scan(nm, s_scan, &tm);
    for (int w = w0; w < w1; w++) {
        const int lo = e0 + w * 32;
        if (lo < budget) pre[w] = (uint32_t)ph;
        if (lo + 32 > budget) pre[w + 1] = (uint32_t)pm;
        ph += __popc(evict_holes(bits[w], lo, budget));
        pm += __popc(evict_movers(bits[w], lo, budget));
    }
    if (tid == 0) { s_cnt[1] = th; s_cnt[2] = tm; }
    cluster.sync();
    if (tid < C) {
        s_hc[tid] = *cluster.map_shared_rank(&s_cnt[1], tid);
        s_mc[tid] = *cluster.map_shared_rank(&s_cnt[2], tid);
    }
    __syncthreads();
    int moves = 0, hb = 0, mb = 0;                              // and the ranks before this part
    for (int r = 0; r < C; r++) {
        hb += r < me ? s_hc[r] : 0;
        mb += r < me ? s_mc[r] : 0;
        moves += s_mc[r];
    }
    if (moves == 0) {                                           // alike in the whole cluster
        cluster.sync();                                         // nobody leaves while its counts are being read
        return;
    }
    const int share = (moves + C - 1) / C, room = evict_room(part_cap);
    const KvTile t(a.ng);
    // 2^sh lanes a move: 4 ng of them copy 16 bytes of codes, 2 ng a scale and bias, two the
    // score and the position; four moves a lane in flight
    const int sh = a.ng == 1 ? 3 : a.ng == 2 ? 4 : 5, p = tid & ((1 << sh) - 1);
    size_t unit = 0;                                            // this lane's bytes in a tile, and per entry
    int off = 0, step = 32;
    if (p < 4 * a.ng) {
        off = t.codes(p / (2 * a.ng), (p >> 1) % a.ng, 0) + (p & 1) * 16;
    } else if (p < 6 * a.ng) {
        off = t.sb((p - 4 * a.ng) / a.ng, (p - 4 * a.ng) % a.ng, 0);
        step = 4;
    }
    unit = (size_t)h * t.bytes() + off;
    const size_t page_bytes = (size_t)a.hkv * t.bytes();
    const int32_t* trow = a.table + (size_t)s * a.max_pages;
    for (int k0 = 0; k0 < share; k0 += room) {
        if (k0) cluster.sync();                                 // the lists have been worked through
        // a lane per entry of a word tells the CTA that has its rank where it stands
        for (int w = tid >> 5; w < words; w += kEvictThreads / 32) {
            const int lo = e0 + w * 32;
            const uint32_t holes = evict_holes(bits[w], lo, budget), movers = evict_movers(bits[w], lo, budget);
            if (!(holes | movers)) continue;
            int page = trow[lo / kKvPage];                      // a word lies in one page
            if ((unsigned)page >= (unsigned)a.n_pages) {
                kv_flag(a.status);
                page = -1;
            }
            const auto tell = [&](uint32_t f, int before, int side) {
                if (!(f >> lane & 1u)) return;
                const int g = before + __popc(f & ((1u << lane) - 1u)), r = g / share, slot = g - r * share - k0;
                if (g < moves && slot >= 0 && slot < room)
                    reinterpret_cast<int2*>(cluster.map_shared_rank(list, r) + slot)[side] = make_int2(lo + lane, page);
            };
            if (movers) tell(movers, mb + (int)pre[w + 1], 0);
            if (holes) tell(holes, hb + (int)pre[w], 1);
        }
        cluster.sync();
        const int m = min(room, min(share, moves - me * share) - k0);
        const int each = kEvictThreads >> sh;                   // moves in flight in a step
        for (int i0 = tid >> sh; i0 < m; i0 += 4 * each) {
            uint4 v[4];
#pragma unroll
            for (int k = 0; k < 4; k++) {
                const int i = i0 + k * each;
                if (i >= m) continue;
                const int4 e = list[i];
                const bool ok = (e.y | e.w) >= 0;               // codes of a bad page stay where they are
                const uint8_t* src = a.pages + (size_t)e.y * page_bytes + unit + (e.x % kKvPage) * step;
                if (p < 4 * a.ng) { if (ok) v[k] = *reinterpret_cast<const uint4*>(src); }
                else if (p < 6 * a.ng) { if (ok) v[k].x = *reinterpret_cast<const uint32_t*>(src); }
                else if (p == 6 * a.ng) v[k].x = __float_as_uint(score[e.x]);
                else if (p == 6 * a.ng + 1) v[k].x = (uint32_t)pos[e.x];
            }
#pragma unroll
            for (int k = 0; k < 4; k++) {
                const int i = i0 + k * each;
                if (i >= m) continue;
                const int4 e = list[i];
                const bool ok = (e.y | e.w) >= 0;
                uint8_t* dst = a.pages + (size_t)e.w * page_bytes + unit + (e.z % kKvPage) * step;
                if (p < 4 * a.ng) { if (ok) *reinterpret_cast<uint4*>(dst) = v[k]; }
                else if (p < 6 * a.ng) { if (ok) *reinterpret_cast<uint32_t*>(dst) = v[k].x; }
                else if (p == 6 * a.ng) score[e.z] = __uint_as_float(v[k].x);
                else if (p == 6 * a.ng + 1) pos[e.z] = (int)v[k].x;
            }
        }
    }
}

}  // namespace moeq4
