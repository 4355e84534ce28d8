// kv_attn_tc.cuh -- attention of many rows per kv head over the 4-bit KV cache
// (prompt chunks) on the 5th-generation tensor cores.
//
// Rows of one kv head are its (row, query head) pairs; an item is (sequence,
// tile of 128 rows, kv head).  Per page of 64 entries
//   S[r][j] = q[r] . k[j]       tcgen05, Q and K in shared memory
//   p = exp(S - max)            one row per pair of threads, P over S in tensor memory
//   O[r][d] += P[r] . v[.][d]   tcgen05, P from tensor memory, V in shared memory
// K enters as two fp16 operands, hi = fp16(s c + b) and lo = fp16(s c + b - hi),
// so the scores are as exact as fp32 sums are; the products of lo come first, because
// the tensor cores cut off at the size of the running sum (hi first: twice the error of
// lse, 1.8e-7 of it instead of 0.9e-7 with heads of 256).  (With the raw codes as operands
// and the groups' scales folded in by the softmax threads, as the few-row kernel
// does it, every thread reads every entry's scales from shared memory: 512
// 16-byte broadcasts a tile, 427 us at 4 chunks of up to 512 rows against 360 when two
// operands replaced them; now 338 to 387, as the chunks' lengths fall.)  p enters as
// hi and remainder too; V is rounded to fp16 once, a relative 2^-12 on average, as
// the output is (one more rounding, of p, would make the error 1.7 times that of
// the output's own rounding instead of 1.4).  K and V are scaled by powers of two, so
// that no value leaves fp16's range: K's (per page) divides the softmax scale, V's (held
// until a page exceeds it) leaves at the end; small V are held to 2^-31 of the largest
// that a row of the tile sees.  The row maximum moves only when it grows by more
// than 2^8, and only then is O rescaled.  Groups of V that are not finite enter as
// zeros; rows that see one get a NaN in its columns at the end, so that masked
// rows (p = 0) stay clean.
//
// Roles, meeting at mbarriers (every wait bounded; each barrier that frees a ring
// slot belongs to that slot, so no waiter can fall two phases behind):
//   warps 0..7    softmax: warp w holds rows 32 (w % 4) .. of the tile (TMEM lanes)
//                 and half w / 4 of its entries; the halves of a row exchange
//                 their maximum through shared memory.  They bring Q to tensor memory.
//   warps 8..15   converters: codes from global memory (the next page's loads in
//                 flight while this one is converted) to fp16 operands in shared memory,
//                 128-byte swizzle: K entry-major, V transposed (8 x 4 blocks of
//                 codes turned in registers);
//   warp 16       MMA issuer (one thread): Q K of tile t + 1 is issued before P V of
//                 tile t, so it runs under the softmax of tile t;
//   warp 17       walker (one thread): what the CTA does next, a segment ahead;
//   warps 18, 19  scales and biases of K and of V, pages ahead of the converters:
//                 the powers of two, which entries count, what is not finite.
// Work is cut as in the split kernel: equal runs of pages per CTA.  An item that
// CTA borders cut leaves partial sums in the workspace ([column / 4][row] of four
// floats, so that a warp's 32 rows are one contiguous store); the CTA in which it
// begins describes it, and k_attn_join, launched behind, joins the parts over all
// SMs (one CTA per item would read its 9 parts of 128 KB in 40 us).
#pragma once
#include "kv_attn.cuh"
#include "tcgen05.cuh"
#include "wait.cuh"

namespace moeq4 {

constexpr int kTileRows = 128;
constexpr int kTileSoft = 8;           // softmax warps: 2 per 32 rows
constexpr int kTileConv = 8;           // converter warps
constexpr int kTileWarps = kTileSoft + kTileConv + 4;    // the issuer's warpgroup: one warp works
// Registers: 96 a thread at launch (640 threads); the issuer's warpgroup gives some of
// its own up to the others: 256 x 112 + 256 x 104 + 128 x 48 = 640 x 96.
constexpr int kTileSoftRegs = 112, kTileConvRegs = 104, kTileIssueRegs = 48;
static_assert((kTileSoft * kTileSoftRegs + kTileConv * kTileConvRegs + 4 * kTileIssueRegs) <= kTileWarps * 96, "registers");
constexpr int kTileThreads = kTileWarps * 32;
// Pages an item costs beside its own (0: 58 us for a chunk of 128 rows over 4,096
// entries of 256 columns, 4 and 8: 52) and pages per CTA at least (64 rows of 4 heads
// over 1,000 entries: 6 25 us, 3 to 1 20; a chunk of 128: 1 53 us, 2 52, 12 62).
constexpr int kTileItemCost = 4;
constexpr int kTileMinUnits = 2;
constexpr int kTileMeta = 16;          // pages whose facts are kept for the softmax
constexpr int kTileScales = 4;         // pages whose scales are kept for the converters
constexpr float kTileLift = 6.f;       // p is taken times 2^6: at most 2^14.5 with a maximum 2^8.5 behind

template <int NG>
struct TileShape {
    static constexpr int kD = 64 * NG;
    static constexpr int kK = 2 * NG * kKvPage * 128;           // bytes: hi, then lo
    static constexpr int kV = NG * 64 * 128;                    // columns x entries
    static constexpr int kKRing = 2, kVRing = 2;
    static constexpr int kSmem = kKRing * kK + kVRing * kV + 1024;
    static constexpr uint32_t kO = 0;                           // TMEM columns: O, two score stages, Q
    static constexpr uint32_t kS = kD;
    static constexpr uint32_t kQ = kS + 2 * kKvPage;
    static_assert(kQ + kD / 2 <= 512, "tensor memory");
};

// What the scale warps tell the softmax warps of a page.
struct TileMeta {
    float kinv;                // 1 / K's power of two
    float vexp;                // log2 of V's
    int ok;                    // the page index is usable
    uint32_t bad[4][2];        // per group: entries whose V is not finite
    int any;                   // some are
};

// An item cut by CTA borders: its parts lie in this CTA and the next parts - 1.
struct TileCut {
    int parts;                 // 0: none
    int first, rows, rt, h;    // first row of the sequence, its (row, head) pairs, row tile, kv head
};

struct TileArgs {
    AttnArgs a;
    float* part;               // [2 gridDim.x][128 (D + 2)]: sums, then maximum and total per row
    TileCut* cut;              // [gridDim.x]: the cut item that begins in each CTA
    int min_rows_seq;          // sequences with fewer (row, head) pairs per kv head are not served here
    unsigned long long wait_ns; // bound of every wait inside the kernel
};

struct TileSeq {
    int n, first, len, rows, tiles;
    long long units;
};
// Pages that row tile rt of a sequence reads.
__device__ __forceinline__ void tile_pages(const TileArgs& x, const TileSeq& q, int rt, int* lo, int* n) {
    const int G = x.a.c.hq / x.a.c.hkv, p0 = q.len - q.n;
    const int first = p0 + rt * kTileRows / G, last = p0 + (min((rt + 1) * kTileRows, q.rows) - 1) / G;
    const int j0 = x.a.window > 0 ? max(0, first - x.a.window + 1) : 0;
    *lo = j0 / kKvPage;
    *n = max(1, last / kKvPage + 1 - *lo);
}
__device__ __forceinline__ TileSeq tile_seq(const TileArgs& x, int s, bool report) {
    const KvArgs& c = x.a.c;
    TileSeq q;
    q.n = kv_rows(c, s, &q.first, report);
    q.len = kv_len(c, s, report);
    q.rows = q.n * (c.hq / c.hkv);
    q.tiles = q.rows < x.min_rows_seq ? 0 : (q.rows + kTileRows - 1) / kTileRows;
    q.units = 0;
    for (int rt = 0; rt < q.tiles; rt++) {
        int lo, n;
        tile_pages(x, q, rt, &lo, &n);
        q.units += n + kTileItemCost;
    }
    q.units *= c.hkv;
    return q;
}

// One CTA's run of pages of one item.
struct TileSegment {
    int T;                     // pages; 0: no more work
    int s, first, len, rows;   // sequence, its first row, entries, (row, head) pairs
    int p0;                    // entry of its row 0
    int rt, h, pg0;            // row tile, kv head, first page
    int whole;                 // the item lies in this segment
    int slot;                  // of its partial sums: 1 when it begins here and goes on
};

// Finds a CTA's segments in order.
struct TileWalk {
    long long u, u_end, per, base, rt_base;   // next unit, end of the run; units before the sequence and the row tile
    int s, rt;
    TileSeq q;

    // A warp: units of all sequences, this CTA's run, the sequence it begins in.
    __device__ __forceinline__ void start(const TileArgs& x, int lane) {
        const int n_seqs = x.a.c.n_seqs;
        long long total = 0;
        q.units = 0;
        for (int s0 = 0; s0 < n_seqs; s0 += 32) {
            q.units = 0;
            if (s0 + lane < n_seqs) q = tile_seq(x, s0 + lane, blockIdx.x == 0);
            total += q.units;
        }
        total = warp_sum(total);
        const long long n = total + gridDim.x - 1;
        per = max(n >> 32 ? n / gridDim.x : (long long)((unsigned)n / gridDim.x), (long long)kTileMinUnits);
        u = blockIdx.x * per;
        u_end = min(total, u + per);
        base = rt_base = 0;
        s = rt = 0;
        if (lane == 0) x.cut[blockIdx.x].parts = 0;              // until a cut item begins here
        if (u >= u_end) return;
        int at = 0;
        for (int s0 = 0; s0 < n_seqs; s0 += 32) {
            if (n_seqs > 32) {                                   // else q holds it already
                q.units = 0;
                if (s0 + lane < n_seqs) q = tile_seq(x, s0 + lane, false);
            }
            long long inc = q.units;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long y = __shfl_up_sync(0xffffffffu, inc, o);
                if (lane >= o) inc += y;
            }
            const unsigned hit = __ballot_sync(0xffffffffu, base + inc > u);
            if (hit) {
                at = __ffs(hit) - 1;
                s = s0 + at;
                base += __shfl_sync(0xffffffffu, inc - q.units, at);
                break;
            }
            base += __shfl_sync(0xffffffffu, inc, 31);
        }
        rt_base = base;
        if (lane == 0) q = tile_seq(x, s, false);
    }

    // One thread: the next segment.
    __device__ __forceinline__ TileSegment next(const TileArgs& x) {
        const KvArgs& c = x.a.c;
        TileSegment g{};
        if (u < u_end) {
            int plo, np;
            while (true) {                                       // row tile that holds unit u
                while (rt >= q.tiles) {
                    if (s + 1 >= c.n_seqs) return g;             // (not reached while what lens says stays)
                    base += q.units;
                    q = tile_seq(x, ++s, false);
                    rt = 0;
                    rt_base = base;
                }
                tile_pages(x, q, rt, &plo, &np);
                const long long w = (long long)(np + kTileItemCost) * c.hkv;
                if (u < rt_base + w) break;
                rt_base += w;
                rt++;
            }
            const int h = (int)(u - rt_base) / (np + kTileItemCost);
            // the item's pages stand at units ib .. ie - 1, behind its fixed cost
            const long long ib = rt_base + (long long)h * (np + kTileItemCost) + kTileItemCost, ie = ib + np;
            u = max(u, ib);
            if (u < u_end) {
                g.T = (int)(min(u_end, ie) - u);
                g.s = s;
                g.first = q.first;
                g.len = q.len;
                g.rows = q.rows;
                g.p0 = q.len - q.n;
                g.rt = rt;
                g.h = h;
                g.pg0 = plo + (int)(u - ib);
                u = min(u_end, ie);
                const bool begins = ib >= blockIdx.x * per;
                g.whole = begins && u == ie;
                g.slot = begins;
                if (begins && u < ie)
                    x.cut[blockIdx.x] = TileCut{(int)((ie - 1) / per) - (int)blockIdx.x + 1, q.first, q.rows, rt, h};
                return g;
            }
        }
        return g;
    }
};

template <int NG>
__global__ void __launch_bounds__(kTileThreads, 1) k_attn_tile(const TileArgs x) {
    using Sh = TileShape<NG>;
    constexpr int D = Sh::kD, KT = kKvPage, HK = KT / 2, KR = Sh::kKRing, VR = Sh::kVRing;
    extern __shared__ uint8_t tl_raw[];
    __shared__ __align__(8) uint64_t b_q, b_k[KR], b_kf[KR], b_v[VR], b_pv[VR], b_s[2], b_p[2];
    __shared__ __align__(8) uint64_t b_sc[kTileScales], b_scf[kTileScales];
    __shared__ uint32_t s_tmem;
    __shared__ float s_mx[2][2][kTileRows], s_sum[2][NG + 1][kTileRows];
    // scaled by the page's powers of two: scale then bias of every entry
    __shared__ __align__(16) __half s_sc[kTileScales][2][2][NG][KT];
    __shared__ TileMeta s_meta[kTileMeta];
    __shared__ TileSegment s_seg[2];
    const AttnArgs& a = x.a;
    const KvArgs& c = a.c;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int G = c.hq / c.hkv;
    const uint32_t sbase = (smem_u32(tl_raw) + 1023u) & ~1023u;
    uint8_t* gK = tl_raw + (sbase - smem_u32(tl_raw));
    uint8_t* gV = gK + KR * Sh::kK;
    const uint32_t sK = sbase, sV = sK + KR * Sh::kK;

    kv_begin();
    TileWalk walk;
    if (warp == kTileSoft + kTileConv + 1) {
        walk.start(x, lane);
        if (lane == 0) s_seg[0] = walk.next(x);
    }
    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&s_tmem)), "r"(512)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    if (tid == 0) {
        mbar_init(&b_q, kTileSoft);
        for (int i = 0; i < KR; i++) {
            mbar_init(&b_k[i], kTileConv);
            mbar_init(&b_kf[i], 1);                                         // commits
        }
        for (int i = 0; i < VR; i++) {
            mbar_init(&b_v[i], kTileConv);
            mbar_init(&b_pv[i], 1);
        }
        for (int i = 0; i < 2; i++) {
            mbar_init(&b_s[i], 2);              // the commit, and the issuer for what it saw of the page
            mbar_init(&b_p[i], kTileSoft);
        }
        for (int i = 0; i < kTileScales; i++) {
            mbar_init(&b_sc[i], 2);                                         // the two scale warps
            mbar_init(&b_scf[i], kTileConv);
        }
        fence_mbar_init();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem;
    bool ok = true;
    uint32_t gt = 0;                                    // tiles of earlier segments: phases run on
    // end of a segment: a role that gave up has recorded it, and all leave together
#define TILE_SEGMENTS(seg, g)                                                     \
    for (int seg = 0;; seg++) {                                                   \
        const TileSegment g = s_seg[seg & 1];                                     \
        if (g.T == 0) break;
#define TILE_SEGMENTS_END(g)                                                      \
        gt += g.T;                                                                \
        if (__syncthreads_or(!ok)) break;                                         \
    }

    if (warp < kTileSoft) {
        // ---------------------------------------------------------- softmax --
        reg_alloc<kTileSoftRegs>();
        TILE_SEGMENTS(seg, sg)
            const int T = sg.T, rt = sg.rt, h = sg.h, p0 = sg.p0, pg0 = sg.pg0;
            const int first_pos = p0 + rt * kTileRows / G;      // least and greatest row
            const int last_pos = p0 + (min((rt + 1) * kTileRows, sg.rows) - 1) / G;
            const int last_low = a.window > 0 ? last_pos - a.window + 1 : 0;
            const int q4 = warp & 3, half = warp >> 2, r = 32 * q4 + lane;
            const uint32_t t_row = tmem + ((uint32_t)(32 * q4) << 16);
            // Q to tensor memory: this half's columns of the row, in the order of the code pairs;
            // the sign of the softmax scale goes with it
            {
                const uint32_t flip = a.scale < 0.f ? 0x80008000u : 0u;
                const int qr = rt * kTileRows + r;
                const bool on = qr < sg.rows && a.scale != 0.f;
                const __half* qp = a.q + (size_t)(sg.first + min(qr, sg.rows - 1) / G) * a.q_stride +
                                   (size_t)(h * G + min(qr, sg.rows - 1) % G) * D + half * (NG * 32);
#pragma unroll
                for (int k = 0; k < NG; k++) {
                    uint32_t o[16];
#pragma unroll
                    for (int e = 0; e < 4; e++) {
                        uint4 v = make_uint4(0, 0, 0, 0);
                        if (on) v = *reinterpret_cast<const uint4*>(qp + k * 32 + e * 8);
                        v.x ^= flip; v.y ^= flip; v.z ^= flip; v.w ^= flip;
                        o[4 * e] = __byte_perm(v.x, v.z, 0x5410);
                        o[4 * e + 1] = __byte_perm(v.x, v.z, 0x7632);
                        o[4 * e + 2] = __byte_perm(v.y, v.w, 0x5410);
                        o[4 * e + 3] = __byte_perm(v.y, v.w, 0x7632);
                    }
                    tmem_st16(t_row + Sh::kQ + half * (NG * 16) + k * 16, o);
                }
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&b_q);
            }
            const int rr = min(rt * kTileRows + r, sg.rows - 1);
            const int pos = p0 + rr / G, low = a.window > 0 ? pos - a.window + 1 : 0;
            const float sl2 = a.scale == 0.f ? 1.f : fabsf(a.scale) * kLog2e;
            float poison[NG];                            // NaN where the row saw a V that is not finite
#pragma unroll
            for (int g = 0; g < NG; g++) poison[g] = 0.f;
            float m = -INFINITY, l = 0.f, vexp = 0.f;
            for (int t = 0; t < T; t++) {
                const uint32_t n = gt + t;
                const int st = n & 1;
                const uint32_t t_s = t_row + Sh::kS + st * KT;
                if (ok) ok = __all_sync(0xffffffffu, wait_bar(&b_s[st], (n >> 1) & 1u, c.stop, x.wait_ns));
                if (!ok) {                               // the other half may still come to the barrier
                    named_bar(1 + q4, 64);
                    continue;
                }
                tc_fence_after();
                const TileMeta& meta = s_meta[n % kTileMeta];
                float S[HK];
                {
                    uint32_t a0[16], a1[16];
                    tmem_ld16_nw(t_s + half * HK, a0);
                    tmem_ld16_nw(t_s + half * HK + 16, a1);
                    tmem_ld_wait();
#pragma unroll
                    for (int j = 0; j < 16; j++) {
                        S[j] = __uint_as_float(a0[j]);
                        S[16 + j] = __uint_as_float(a1[j]);
                    }
                }
                const int j0 = (pg0 + t) * kKvPage + half * HK;
                const bool edge = j0 + HK - 1 > first_pos || j0 < last_low || !meta.ok;
                uint32_t vis = 0xFFFFFFFFu;
                if (edge) {
                    vis = 0;
                    const bool page = meta.ok != 0;
#pragma unroll
                    for (int j = 0; j < HK; j++) {
                        if (page && j0 + j <= pos && j0 + j >= low) vis |= 1u << j;
                        else S[j] = -INFINITY;
                    }
                }
                float tp[4] = {S[0], S[1], S[2], S[3]};
#pragma unroll
                for (int j = 4; j < HK; j++) tp[j & 3] = fmaxf(tp[j & 3], S[j]);
                float top = fmaxf(fmaxf(tp[0], tp[1]), fmaxf(tp[2], tp[3]));
                s_mx[st][half][r] = top;
                named_bar(1 + q4, 64);
                const float sc = sl2 * meta.kinv;
                top = fmaxf(top, s_mx[st][half ^ 1][r]) * sc;
                const float du = meta.vexp - vexp;       // V's unit moved (alike in all threads)
                const bool grow = top > m + 8.f;
                if (__any_sync(0xffffffffu, grow) || du != 0.f) {
                    const float m2 = grow ? rintf(top) : m;
                    const float fp = m2 == -INFINITY ? 1.f : exp2_fast(m - m2), f = fp * exp2f(du);
                    m = m2;
                    vexp = meta.vexp;
                    l *= fp;
                    if (t > 0) {                         // O so far: this half's columns of the row
                        ok = __all_sync(0xffffffffu, wait_bar(&b_pv[(n - 1) % VR], ((n - 1) / VR) & 1u, c.stop, x.wait_ns));
                        if (!ok) continue;
                        tc_fence_after();
#pragma unroll
                        for (int k = 0; k < NG * 2; k++) {
                            uint32_t o[16];
                            const uint32_t at = t_row + Sh::kO + half * (NG * 32) + k * 16;
                            tmem_ld16_nw(at, o);
                            tmem_ld_wait();
#pragma unroll
                            for (int e = 0; e < 16; e++) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                            tmem_st16(at, o);
                        }
                    }
                }
                const float ref = m == -INFINITY ? 0.f : m - kTileLift;
                const float2 sc2 = make_float2(sc, sc), ref2 = make_float2(-ref, -ref);
                float2 ls[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                for (int j = 0; j < HK; j += 2) {
                    const float2 e = fma2(make_float2(S[j], S[j + 1]), sc2, ref2);
                    S[j] = exp2_fast(e.x);
                    S[j + 1] = exp2_fast(e.y);
                    ls[(j >> 1) & 1] = add2(ls[(j >> 1) & 1], make_float2(S[j], S[j + 1]));
                }
                l += (ls[0].x + ls[0].y) + (ls[1].x + ls[1].y);
                uint32_t P[16];                          // hi, then the remainder behind it
#pragma unroll
                for (int j = 0; j < 16; j++) P[j] = f2h(S[2 * j], S[2 * j + 1]);
                tmem_st16(t_s + half * (HK / 2), P);
#pragma unroll
                for (int j = 0; j < 16; j++) {
                    const float2 f = h2f(P[j]), d = add2(make_float2(S[2 * j], S[2 * j + 1]), make_float2(-f.x, -f.y));
                    P[j] = f2h(d.x, d.y);
                }
                tmem_st16(t_s + KT / 2 + half * (HK / 2), P);
                if (meta.any)
#pragma unroll
                    for (int g = 0; g < NG; g++)
                        if (meta.bad[g][half] & vis) poison[g] = NAN;
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&b_p[st]);
            }
            // row sums of both halves, then this half's columns
            s_sum[half][NG][r] = l;
#pragma unroll
            for (int g = 0; g < NG; g++) s_sum[half][g][r] = poison[g];
            named_bar(1 + q4, 64);
            if (ok) ok = __all_sync(0xffffffffu, wait_bar(&b_pv[(gt + T - 1) % VR], ((gt + T - 1) / VR) & 1u, c.stop, x.wait_ns));
            tc_fence_after();
            if (ok) {
                const float L = s_sum[0][NG][r] + s_sum[1][NG][r];
                const float M = m == -INFINITY ? m : m - kTileLift;
                const bool row = rt * kTileRows + r < sg.rows;
                float* slot = x.part + (size_t)(2 * blockIdx.x + sg.slot) * (kTileRows * (D + 2));
                const int head = h * G + rr % G;
                const float f = L == 0.f ? 0.f : 1.f / L, back = exp2f(-vexp);
                __half* out = a.out + (size_t)(sg.first + rr / G) * a.out_stride + (size_t)head * D;
#pragma unroll
                for (int k = 0; k < NG * 2; k++) {
                    const int col = half * (NG * 32) + k * 16;
                    uint32_t o[16];
                    tmem_ld16_nw(t_row + Sh::kO + col, o);
                    tmem_ld_wait();
                    const float bad = s_sum[0][col / 64][r] + s_sum[1][col / 64][r];
                    if (!row) continue;
                    float v[16];
#pragma unroll
                    for (int e = 0; e < 16; e++) v[e] = fmaf(__uint_as_float(o[e]), back, bad);
                    if (sg.whole) {
#pragma unroll
                        for (int e = 0; e < 2; e++)
                            *reinterpret_cast<uint4*>(out + col + 8 * e) =
                                make_uint4(f2h(v[8 * e] * f, v[8 * e + 1] * f), f2h(v[8 * e + 2] * f, v[8 * e + 3] * f),
                                           f2h(v[8 * e + 4] * f, v[8 * e + 5] * f), f2h(v[8 * e + 6] * f, v[8 * e + 7] * f));
                    } else {
#pragma unroll
                        for (int e = 0; e < 4; e++)
                            *reinterpret_cast<float4*>(slot + ((size_t)(col / 4 + e) * kTileRows + r) * 4) =
                                make_float4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
                    }
                }
                if (half == 0 && row) {
                    if (sg.whole) {
                        a.lse[(size_t)(sg.first + rr / G) * c.hq + head] = lse_of(M, L);
                    } else {
                        slot[kTileRows * D + r] = M;
                        slot[kTileRows * D + kTileRows + r] = L;
                    }
                }
            }
            tc_fence_before();
        TILE_SEGMENTS_END(sg)
    } else if (warp < kTileSoft + kTileConv) {
        // ------------------------------------------------------- converters --
        reg_alloc<kTileConvRegs>();
        TILE_SEGMENTS(seg, sg)
            const int T = sg.T, h = sg.h, pg0 = sg.pg0;
            constexpr int CT = kTileConv * 32, NK = (NG + 1) / 2;       // 128 NG pieces of K and of V a page
            const int ct = tid - kTileSoft * 32;
            const int32_t* trow = c.table + (size_t)sg.s * c.max_pages;
            // a page's codes; those of the next page are loaded as soon as a part has been
            // converted, so K's come while V is converted and V's while K is
            uint4 rk[NK];                                // 32 codes of an entry
            uint32_t rv[NK][8];                          // a code word of 8 entries
            const auto page_at = [&](int t) {            // -1: behind the last entry
                const int pg = pg0 + t;
                return t < T && pg * kKvPage < sg.len ? trow[pg] : -1;
            };
            // codes of a page that does not exist may be anything: its scales are zero
            const auto tile_at = [&](int id) {
                return c.pages + ((size_t)((unsigned)id < (unsigned)c.n_pages ? id : 0) * c.hkv + h) * (size_t)(4608 * NG);
            };
            const auto load_k = [&](const uint8_t* tile) {
#pragma unroll
                for (int i = 0; i < NK; i++)
                    if (i * CT + ct < 128 * NG) rk[i] = reinterpret_cast<const uint4*>(tile)[i * CT + ct];
            };
            const auto load_v = [&](const uint8_t* tile) {
#pragma unroll
                for (int i = 0; i < NK; i++) {
                    const int n = i * CT + ct;           // columns 8 vw + 4 (n & 1) .. of entries 8 vk ..
                    const uint8_t* v = tile + 2304 * NG + (n >> 7) * 2048 + ((n >> 4) & 7) * 256 + ((n >> 1) & 7) * 4;
                    if (n < 128 * NG)
#pragma unroll
                        for (int e = 0; e < 8; e++) rv[i][e] = *reinterpret_cast<const uint32_t*>(v + e * 32);
                }
            };
            int id = page_at(0), id2 = page_at(1);       // pages t and t + 1
            load_k(tile_at(id));
            load_v(tile_at(id));
            for (int t = 0; t < T; t++) {
                const uint32_t n = gt + t;
                const int sl = n % kTileScales;
                // the page's scales, and K's slot once Q K of the slot's last page has ended
                if (ok)
                    ok = __all_sync(0xffffffffu, wait_bar(&b_sc[sl], (n / kTileScales) & 1u, c.stop, x.wait_ns) &&
                                                     (n < KR || wait_bar(&b_kf[n % KR], ((n / KR) - 1) & 1u, c.stop, x.wait_ns)));
                if (!ok) break;
                uint8_t* gk = gK + (n % KR) * Sh::kK;
#pragma unroll
                for (int i = 0; i < NK; i++) {
                    const int nn = i * CT + ct, g = nn >> 7, r = (nn >> 1) & 63, hf = nn & 1;
                    if (nn < 128 * NG) {
                        const __half2 s2 = __half2half2(s_sc[sl][0][0][g][r]), b2 = __half2half2(s_sc[sl][0][1][g][r]);
                        const float2 fs = __half22float2(s2), fb = __half22float2(b2);
                        const uint32_t word[4] = {rk[i].x, rk[i].y, rk[i].z, rk[i].w};
#pragma unroll
                        for (int k = 0; k < 4; k++) {
                            uint32_t cd[4], hi[4], lo[4];
                            codes_exact(word[k], cd);
#pragma unroll
                            for (int e = 0; e < 4; e++) {
                                const __half2 hv = __hfma2(*reinterpret_cast<const __half2*>(&cd[e]), s2, b2);
                                hi[e] = *reinterpret_cast<const uint32_t*>(&hv);
                                const float2 f = h2f(hi[e]), x2 = fma2(h2f(cd[e]), fs, fb);
                                const float2 d = add2(x2, make_float2(-f.x, -f.y));
                                lo[e] = f2h(d.x, d.y);
                            }
                            uint8_t* at = gk + g * (KT * 128) + r * 128 + (((hf * 4 + k) ^ (r & 7)) << 4);
                            *reinterpret_cast<uint4*>(at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                            *reinterpret_cast<uint4*>(at + NG * KT * 128) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                        }
                    }
                }
                fence_proxy_async_shared();
                __syncwarp();
                if (lane == 0) mbar_arrive(&b_k[n % KR]);
                id = id2;
                id2 = page_at(t + 2);
                const uint8_t* next = tile_at(id);
                if (t + 1 < T) load_k(next);
                // V, transposed, once P V of the slot's last page has ended
                if (n >= VR) ok = __all_sync(0xffffffffu, wait_bar(&b_pv[n % VR], ((n / VR) - 1) & 1u, c.stop, x.wait_ns));
                if (!ok) break;
                uint8_t* gv = gV + (n % VR) * Sh::kV;
#pragma unroll
                for (int i = 0; i < NK; i++) {
                    const int nn = i * CT + ct, g = nn >> 7, vk = (nn >> 4) & 7, vw = (nn >> 1) & 7, hf = nn & 1;
                    if (nn < 128 * NG) {
                        const uint4 sv = *reinterpret_cast<const uint4*>(&s_sc[sl][1][0][g][8 * vk]);
                        const uint4 bv = *reinterpret_cast<const uint4*>(&s_sc[sl][1][1][g][8 * vk]);
                        const uint32_t s2[4] = {sv.x, sv.y, sv.z, sv.w}, b2[4] = {bv.x, bv.y, bv.z, bv.w};
                        uint32_t o[4][4];                // [column][entries 2e, 2e + 1]
#pragma unroll
                        for (int e = 0; e < 4; e++) {
                            uint32_t cd[4];
                            codes_exact(__byte_perm(rv[i][2 * e], rv[i][2 * e + 1], hf ? 0x7632 : 0x5410), cd);
#pragma unroll
                            for (int k = 0; k < 4; k++) {
                                const __half2 v = __hfma2(*reinterpret_cast<const __half2*>(&cd[k]),
                                                          *reinterpret_cast<const __half2*>(&s2[e]),
                                                          *reinterpret_cast<const __half2*>(&b2[e]));
                                o[k][e] = *reinterpret_cast<const uint32_t*>(&v);
                            }
                        }
                        uint8_t* dst = gv + g * (64 * 128) + (8 * vw + 4 * hf) * 128;
#pragma unroll
                        for (int k = 0; k < 4; k++)
                            *reinterpret_cast<uint4*>(dst + k * 128 + ((vk ^ (4 * hf + k)) << 4)) =
                                make_uint4(o[k][0], o[k][1], o[k][2], o[k][3]);
                    }
                }
                fence_proxy_async_shared();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&b_v[n % VR]);
                    mbar_arrive(&b_scf[sl]);
                }
                if (t + 1 < T) load_v(next);
            }
        TILE_SEGMENTS_END(sg)
    } else {
        // ---------------------------------------------- MMA issuer and walker --
        reg_dealloc<kTileIssueRegs>();
        TILE_SEGMENTS(seg, sg)
            const int T = sg.T;
        if (warp == kTileSoft + kTileConv + 1) {
            if (lane == 0) s_seg[(seg + 1) & 1] = walk.next(x);
        } else if (warp > kTileSoft + kTileConv + 1) {
            // ----------------------------------------------------- scales --
            const int v = warp - (kTileSoft + kTileConv + 2);           // K, V
            const int32_t* trow = c.table + (size_t)sg.s * c.max_pages;
            const int last_pos = sg.p0 + (min((sg.rt + 1) * kTileRows, sg.rows) - 1) / G;
            const int first_low = a.window > 0 ? sg.p0 + sg.rt * kTileRows / G - a.window + 1 : 0;
            constexpr int N = 2 * NG;                                   // words a lane: entry 32 (i % 2) + lane of group i / 2
            uint32_t f[N];
            bool there = false;
            const auto load = [&](int t) {
                const int pg = sg.pg0 + t;
                const bool held = pg * kKvPage < sg.len;
                const int id = held ? trow[pg] : -1;
                there = (unsigned)id < (unsigned)c.n_pages;
                if (held && !there && v == 0 && lane == 0) kv_flag(c.status);
                const uint8_t* at = c.pages + ((size_t)(there ? id : 0) * c.hkv + sg.h) * (size_t)(4608 * NG) + (2304 * v + 2048) * NG;
#pragma unroll
                for (int i = 0; i < N; i++) f[i] = reinterpret_cast<const uint32_t*>(at)[i * 32 + lane];
            };
            int vexp = 0;                                // log2 of V's factor
            float vtop = 0.f;                            // largest value it admits
            load(0);
            for (int t = 0; t < T; t++) {
                const uint32_t n = gt + t;
                const int sl = n % kTileScales;
                TileMeta& meta = s_meta[n % kTileMeta];
                const int j = (sg.pg0 + t) * kKvPage + lane;
                const bool in0 = there && j <= last_pos && j >= first_low;
                const bool in1 = there && j + 32 <= last_pos && j + 32 >= first_low;
                float mx = 0.f;
                uint32_t bad = 0;
#pragma unroll
                for (int i = 0; i < N; i++) {
                    const float2 x2 = h2f(f[i]);
                    const bool in = i & 1 ? in1 : in0, fin = fabsf(x2.x) <= 65504.f && fabsf(x2.y) <= 65504.f;
                    if (in && fin) mx = fmaxf(mx, fmaf(15.f, fabsf(x2.x), fabsf(x2.y)));
                    if (in && !fin) bad |= 1u << i;
                }
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
                // K: the page's largest value to 2^13..2^14.  V: the first to 2^10..2^11, and anew
                // when a page exceeds 2^15
                int e;
                if (v == 0) {
                    e = mx > 0.f ? 13 - exponent_of(mx) : 0;
                } else {
                    if (mx > vtop) {
                        vexp = 10 - exponent_of(mx);
                        vtop = 32768.f * pow2(-vexp);
                    }
                    e = vexp;
                }
                if (n >= kTileScales)
                    ok = __all_sync(0xffffffffu, wait_bar(&b_scf[sl], ((n / kTileScales) - 1) & 1u, c.stop, x.wait_ns));
                if (!ok) break;
                const float up = pow2(e);
                bool any = false;
#pragma unroll
                for (int i = 0; i < N; i++) {
                    const float2 x2 = h2f(f[i]);
                    // entries that no row of the tile sees count as zero, whatever they hold, and
                    // values of V that are not finite too (their rows learn of them)
                    const bool take = (i & 1 ? in1 : in0) && !(v == 1 && ((bad >> i) & 1u));
                    s_sc[sl][v][0][i >> 1][32 * (i & 1) + lane] = __float2half_rn(take ? x2.x * up : 0.f);
                    s_sc[sl][v][1][i >> 1][32 * (i & 1) + lane] = __float2half_rn(take ? x2.y * up : 0.f);
                    if (v == 1) {
                        const uint32_t word = __ballot_sync(0xffffffffu, (bad >> i) & 1u);
                        any = any || word;
                        if (lane == 0) meta.bad[i >> 1][i & 1] = word;
                    }
                }
                if (lane == 0) {
                    if (v == 0) {
                        meta.kinv = pow2(-e);
                        meta.ok = there;
                    } else {
                        meta.vexp = (float)e;
                        meta.any = any;
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&b_sc[sl]);
                if (t + 1 < T) load(t + 1);
            }
        } else if (warp == kTileSoft + kTileConv && lane == 0) {
            constexpr uint32_t id_s = kTcIdescF16 | ((uint32_t)(KT >> 3) << 17);
            constexpr uint32_t id_o = kTcIdescF16 | ((uint32_t)(D >> 3) << 17);
            // descriptors: the high half is the same for all, the low half (address) moves
            const uint32_t dhi = (uint32_t)(tc_sdesc_sw128(0) >> 32);
            const auto pv = [&](int t) {
                const uint32_t n = gt + t;
                const int st = n & 1;
                if (!wait_bar(&b_v[n % VR], (n / VR) & 1u, c.stop, x.wait_ns) ||
                    !wait_bar(&b_p[st], (n >> 1) & 1u, c.stop, x.wait_ns))
                    return false;
                tc_fence_after();
                const uint32_t dv = (uint32_t)tc_sdesc_sw128(sV + (n % VR) * Sh::kV), pa = tmem + Sh::kS + st * KT;
                tc_mma_ts(tmem + Sh::kO, pa, tc_desc(dv, dhi), id_o, t > 0 ? 1u : 0u);
#pragma unroll
                for (int k = 1; k < KT / 8; k++)         // hi, then the remainder
                    tc_mma_ts_acc(tmem + Sh::kO, pa + 8 * k, tc_desc(dv + 2u * (k % (KT / 16)), dhi), id_o);
                mma_commit(&b_pv[n % VR]);
                return true;
            };
            if (!wait_bar(&b_q, seg & 1u, c.stop, x.wait_ns)) ok = false;
            int done = 0, asked = 0;                     // tiles whose P V and whose Q K have been issued
            for (int t = 0; ok && t < T; t++) {
                const uint32_t n = gt + t;
                const int st = n & 1;
                if (!wait_bar(&b_k[n % KR], (n / KR) & 1u, c.stop, x.wait_ns) ||
                    // the stage's P of tile t - 2 has been used
                    (t >= 2 && !wait_bar(&b_pv[(n - 2) % VR], ((n - 2) / VR) & 1u, c.stop, x.wait_ns))) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t dk = (uint32_t)tc_sdesc_sw128(sK + (n % KR) * Sh::kK), ds = tmem + Sh::kS + st * KT;
#pragma unroll
                for (int z = 0; z < 2; z++)              // lo, then hi
#pragma unroll
                    for (int g = 0; g < NG; g++)
#pragma unroll
                        for (int k = 0; k < 4; k++) {
                            const uint32_t da = tmem + Sh::kQ + g * 32 + 8 * k;
                            const uint64_t db = tc_desc(dk + ((((1 - z) * NG + g) * KT * 128) >> 4) + 2u * k, dhi);
                            if (z + g + k == 0) tc_mma_ts(ds, da, db, id_s, 0u);
                            else tc_mma_ts_acc(ds, da, db, id_s);
                        }
                mma_commit(&b_s[st]);
                mma_commit(&b_kf[n % KR]);
                mbar_arrive(&b_s[st]);
                asked = t + 1;
                if (t > 0) {
                    if (!pv(t - 1)) { ok = false; break; }
                    done = t;
                }
            }
            if (ok && !pv(T - 1)) ok = false;
            else if (ok) done = T;
            // every commit has arrived before the segment ends
            if (done > 0) mma_drain_wait(&b_pv[(gt + done - 1) % VR], ((gt + done - 1) / VR) & 1u);
            if (!ok && asked > 0) mma_drain_wait(&b_kf[(gt + asked - 1) % KR], ((gt + asked - 1) / KR) & 1u);
        }
        TILE_SEGMENTS_END(sg)
    }
#undef TILE_SEGMENTS
#undef TILE_SEGMENTS_END
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
    }
}

// Joins the parts of the item that begins in CTA blockIdx.x: rows 32 blockIdx.y ..
// of its tile, one per lane, 64 columns a CTA, 8 a warp, eight parts at a time with
// all their loads in flight (the weights first and then 16 columns a warp, two
// passes where heads are wide, made a chunk of 128 rows over 4,096 entries of 256
// columns 60 us; now 53).
constexpr int kJoinThreads = 256;
constexpr int kJoinParts = 8;

template <int NG>
__global__ void __launch_bounds__(kJoinThreads) k_attn_join(const TileArgs x) {
    constexpr int D = 64 * NG;
    constexpr size_t kSlot = (size_t)kTileRows * (D + 2);
    kv_begin();
    const TileCut c = x.cut[blockIdx.x];
    const int r = blockIdx.y * 32 + (threadIdx.x & 31), rr = c.rt * kTileRows + r;
    if (c.parts <= 0 || rr >= c.rows) return;
    const int col = blockIdx.z * 64 + (threadIdx.x >> 5) * 8;
    float M = -INFINITY, L = 0.f, o[8];
#pragma unroll
    for (int e = 0; e < 8; e++) o[e] = 0.f;
    for (int b0 = 0; b0 < c.parts; b0 += kJoinParts) {
        float m[kJoinParts], l[kJoinParts];
        float4 v[kJoinParts][2];
#pragma unroll
        for (int k = 0; k < kJoinParts; k++) {
            const int b = b0 + k;
            m[k] = -INFINITY;
            l[k] = 0.f;
            v[k][0] = v[k][1] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (b < c.parts) {
                // the first part is its CTA's second slot, the others their CTAs' first
                const float* at = x.part + (size_t)(2 * ((int)blockIdx.x + b) + (b == 0 ? 1 : 0)) * kSlot;
                m[k] = at[kTileRows * D + r];
                l[k] = at[kTileRows * D + kTileRows + r];
#pragma unroll
                for (int e = 0; e < 2; e++)
                    v[k][e] = *reinterpret_cast<const float4*>(at + ((size_t)(col / 4 + e) * kTileRows + r) * 4);
            }
        }
        float top = M;
#pragma unroll
        for (int k = 0; k < kJoinParts; k++) top = fmaxf(top, m[k]);
        const float ref = top == -INFINITY ? 0.f : top, back = exp2_fast(M - ref);
        M = top;
        L *= back;
#pragma unroll
        for (int e = 0; e < 8; e++) o[e] *= back;
#pragma unroll
        for (int k = 0; k < kJoinParts; k++) {
            const float f = m[k] == -INFINITY && l[k] == 0.f ? 0.f : exp2_fast(m[k] - ref);
            L = fmaf(f, l[k], L);
#pragma unroll
            for (int e = 0; e < 2; e++) {
                o[4 * e] = fmaf(f, v[k][e].x, o[4 * e]);
                o[4 * e + 1] = fmaf(f, v[k][e].y, o[4 * e + 1]);
                o[4 * e + 2] = fmaf(f, v[k][e].z, o[4 * e + 2]);
                o[4 * e + 3] = fmaf(f, v[k][e].w, o[4 * e + 3]);
            }
        }
    }
    const int G = x.a.c.hq / x.a.c.hkv, head = c.h * G + rr % G;
    const float inv = L == 0.f ? 0.f : 1.f / L;
    const size_t row = (size_t)c.first + rr / G;
    *reinterpret_cast<uint4*>(x.a.out + row * x.a.out_stride + (size_t)head * D + col) =
        make_uint4(f2h(o[0] * inv, o[1] * inv), f2h(o[2] * inv, o[3] * inv), f2h(o[4] * inv, o[5] * inv), f2h(o[6] * inv, o[7] * inv));
    if (col == 0) x.a.lse[row * x.a.c.hq + head] = lse_of(M, L);
}

}  // namespace moeq4
