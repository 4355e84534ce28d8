// kv_attn_tc.cuh -- attention of many rows per kv head over the 4-bit KV cache
// (prompt chunks) on the 5th-generation tensor cores.
//
// Rows of one kv head are its (row, query head) pairs; an item is (sequence,
// tile of 128 rows, kv head).  Per tile of KT entries and group g of 64 columns
//   acc_g[r][j] = q_g[r] . (c_g[j] - 8)            tcgen05, Q and codes in shared memory
//   S = sum_g s_jg acc_g + (b_jg + 8 s_jg) sum(q_g[r])                    CUDA cores
//   p = exp(S - max),  P_g = fp16(p s_jg)          into tensor memory, over acc
//   O_g[r][d] += P_g[r] . (c_g[.][d] - 8)          tcgen05, P from tensor memory
//   B_g[r] += p (b_jg + 8 s_jg)                                           CUDA cores
// and out = (O_g + B_g) / sum p.  The codes are exact operands, so the scores are
// as exact as fp32 sums are; the one rounding is that of p s to fp16 (relative
// 2^-12 per entry, averaged over the entries seen: below the rounding of the
// output itself).  Codes are centred (c - 8) so that this rounding is weighed
// with values around zero.  P is kept in range by a power of two per CTA (unit)
// from the largest scale of V in a tile; the row maximum moves only when it grows
// by more than 2^8, and only then is O rescaled.
//
// Roles, meeting at mbarriers (every wait bounded):
//   warps 0..15   scores and softmax: warp w holds rows 32 (w % 4) .. of the tile
//                 (TMEM lanes) and quarter w / 4 of its entries; the four quarters
//                 of a row exchange their maximum through shared memory;
//   warps 16..19  converters: codes from global memory (the next tile's loads in
//                 flight while one is converted) to fp16 operands in shared memory,
//                 128-byte swizzle: K entry-major, V transposed (8 x 8 blocks of
//                 codes turned in registers); scales and biases to fp32;
//   warp 20       MMA issuer (one thread): Q K of tile t + 1 is issued before P V of
//                 tile t, so it runs under the softmax of tile t.
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
constexpr int kTileSoft = 16;          // softmax warps: 4 per 32 rows
constexpr int kTileWarps = kTileSoft + 5;
constexpr int kTileThreads = kTileWarps * 32;
constexpr int kTileSlots = 3;
constexpr int kTileItemCost = 4;       // pages an item costs beside its own
constexpr int kTileMinUnits = 6;       // pages per CTA at least

template <bool B>
struct BoolC {
    static constexpr bool value = B;
};

template <int NG>
struct TileShape {
    static constexpr int kD = 64 * NG;
    static constexpr int KT = NG <= 2 ? 64 : 32;                // entries per tile
    static constexpr int kSub = kKvPage / KT;                   // tiles per page
    static constexpr int kHK = KT / 4;                          // entries per softmax thread
    static constexpr int kQ = NG * kTileRows * 128;             // bytes
    static constexpr int kK = NG * KT * 128;
    static constexpr int kV = NG * 64 * 128;                    // 64 columns x KT entries, rows of 128 bytes
    static constexpr int kScale = NG * KT * 8;                  // (scale, bias + 8 scale) of K or V
    static constexpr int kSlot = kK + kV;
    static constexpr int kSmem = kQ + kTileSlots * (kSlot + 2 * kScale) + 1024;
    static constexpr uint32_t kO = 0;                           // TMEM columns: O, then two score stages
    static constexpr uint32_t kS = NG * 64;
    static constexpr uint32_t kStage = NG * KT;
    static_assert(kS + 2 * kStage <= 512, "tensor memory");
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

template <int NG>
__global__ void __launch_bounds__(kTileThreads, 1) k_attn_tile(const TileArgs x) {
    using Sh = TileShape<NG>;
    constexpr int D = Sh::kD, KT = Sh::KT, HK = Sh::kHK;
    extern __shared__ uint8_t tl_raw[];
    __shared__ __align__(8) uint64_t b_q, b_full[kTileSlots], b_s[2], b_p[2], b_pv[2];
    __shared__ uint32_t s_tmem;
    __shared__ float s_mx[2][4][kTileRows], s_qs[NG][kTileRows];
    __shared__ float s_vmax[kTileSlots][4];
    __shared__ int s_ok[kTileSlots];
    __shared__ long long s_base0, s_total, s_per;
    __shared__ TileSeq s_q;
    __shared__ int s_seq;
    const AttnArgs& a = x.a;
    const KvArgs& c = a.c;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int G = c.hq / c.hkv;
    const uint32_t sbase = (smem_u32(tl_raw) + 1023u) & ~1023u;
    uint8_t* gbase = tl_raw + (sbase - smem_u32(tl_raw));
    const uint32_t sQ = sbase, sSlots = sbase + Sh::kQ;
    uint8_t* gQ = gbase;
    float(*s_sum)[NG + 1][kTileRows] = reinterpret_cast<float(*)[NG + 1][kTileRows]>(gQ);   // once Q has been used
    uint8_t* gSlots = gbase + Sh::kQ;
    float2* gScale = reinterpret_cast<float2*>(gSlots + kTileSlots * Sh::kSlot);   // [slot][K, V][g][entry]

    kv_begin();
    if (warp == 0) {
        long long total = 0;
        TileSeq q{};
        for (int s0 = 0; s0 < c.n_seqs; s0 += 32) {
            q.units = 0;
            if (s0 + lane < c.n_seqs) q = tile_seq(x, s0 + lane, blockIdx.x == 0);
            total += q.units;
        }
        total = warp_sum(total);
        const long long per = max((total + gridDim.x - 1) / gridDim.x, (long long)kTileMinUnits);
        const long long u = blockIdx.x * per;
        long long base = 0;
        if (u < total)
            for (int s0 = 0; s0 < c.n_seqs; s0 += 32) {
                if (c.n_seqs > 32) {
                    q.units = 0;
                    if (s0 + lane < c.n_seqs) q = tile_seq(x, s0 + lane, false);
                }
                long long inc = q.units;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const long long y = __shfl_up_sync(0xffffffffu, inc, o);
                    if (lane >= o) inc += y;
                }
                const unsigned hit = __ballot_sync(0xffffffffu, base + inc > u);
                if (hit) {
                    if (lane == __ffs(hit) - 1) {
                        s_q = q;
                        s_seq = s0 + lane;
                        s_base0 = base + inc - q.units;
                    }
                    break;
                }
                base += __shfl_sync(0xffffffffu, inc, 31);
            }
        if (lane == 0) {
            s_total = total;
            s_per = per;
        }
    }
    __syncthreads();
    const long long total = s_total, per = s_per;
    long long u = blockIdx.x * per, base = s_base0;
    const long long u_end = min(total, u + per);
    if (u >= u_end) {
        if (tid == 0) x.cut[blockIdx.x].parts = 0;
        return;
    }
    int s = s_seq;
    TileSeq q = s_q;
    bool cut = false;                                   // an item begins here and goes on in the next CTA

    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&s_tmem)), "r"(512)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    if (tid == 0) {
        mbar_init(&b_q, kTileSoft);
        for (int i = 0; i < kTileSlots; i++) mbar_init(&b_full[i], 4);      // converter warps
        for (int i = 0; i < 2; i++) {
            mbar_init(&b_s[i], 1);                                          // commits
            mbar_init(&b_p[i], kTileSoft);                                  // softmax warps
            mbar_init(&b_pv[i], 1);
        }
        fence_mbar_init();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem;
    bool ok = true;
    uint32_t gt = 0, seg = 0;                           // tiles of earlier segments, and those: phases run on
    int rt = 0;                                         // row tile of the sequence, and the units before it
    long long rt_base = base;

    while (u < u_end) {
        int plo, np;
        while (true) {                                  // row tile that holds unit u
            while (rt >= q.tiles) {
                base += q.units;
                s++;
                q = tile_seq(x, s, false);
                rt = 0;
                rt_base = base;
            }
            tile_pages(x, q, rt, &plo, &np);
            const long long w = (long long)(np + kTileItemCost) * c.hkv;
            if (u < rt_base + w) break;
            rt_base += w;
            rt++;
        }
        const int h = (int)((u - rt_base) / (np + kTileItemCost));
        const long long ib = rt_base + (long long)h * (np + kTileItemCost) + kTileItemCost, ie = ib + np;
        u = max(u, ib);
        if (u >= u_end) break;
        const int pg0 = plo + (int)(u - ib), pg1 = plo + (int)(min(u_end, ie) - ib);
        u = min(u_end, ie);
        const int p0 = q.len - q.n;
        const int T = (pg1 - pg0) * Sh::kSub;           // tiles of this segment
        const int first_pos = p0 + rt * kTileRows / G;  // least and greatest row
        const int last_pos = p0 + (min((rt + 1) * kTileRows, q.rows) - 1) / G;
        const int first_low = a.window > 0 ? first_pos - a.window + 1 : 0;
        const int last_low = a.window > 0 ? last_pos - a.window + 1 : 0;

        if (warp < kTileSoft) {
            // ------------------------------------------------------ softmax --
            const int q4 = warp & 3, part = warp >> 2, r = 32 * q4 + lane;
            // Q: rows of 64 columns per group, columns in the order of the code pairs; the sign
            // of the softmax scale goes with it
            {
                const uint32_t flip = a.scale < 0.f ? 0x80008000u : 0u;
                constexpr int N = 2 * NG;               // 16-byte chunks per thread, all in flight
                uint4 v[N];
#pragma unroll
                for (int k = 0; k < N; k++) {
                    const int i = tid + k * (kTileSoft * 32), ch = i & 7, rr = rt * kTileRows + ((i >> 3) & (kTileRows - 1));
                    v[k] = make_uint4(0, 0, 0, 0);
                    if (rr < q.rows && a.scale != 0.f)
                        v[k] = *reinterpret_cast<const uint4*>(a.q + (size_t)(q.first + rr / G) * a.q_stride +
                                                               (size_t)(h * G + rr % G) * D + (i >> 10) * 64 + ch * 8);
                }
#pragma unroll
                for (int k = 0; k < N; k++) {
                    const int i = tid + k * (kTileSoft * 32), ch = i & 7, r = (i >> 3) & (kTileRows - 1), g = i >> 10;
                    v[k].x ^= flip; v[k].y ^= flip; v[k].z ^= flip; v[k].w ^= flip;
                    *reinterpret_cast<uint4*>(gQ + g * (kTileRows * 128) + r * 128 + ((ch ^ (r & 7)) << 4)) =
                        make_uint4(__byte_perm(v[k].x, v[k].z, 0x5410), __byte_perm(v[k].x, v[k].z, 0x7632),
                                   __byte_perm(v[k].y, v[k].w, 0x5410), __byte_perm(v[k].y, v[k].w, 0x7632));
                    const float2 f0 = h2f(v[k].x), f1 = h2f(v[k].y), f2 = h2f(v[k].z), f3 = h2f(v[k].w);
                    float sum = ((f0.x + f0.y) + (f1.x + f1.y)) + ((f2.x + f2.y) + (f3.x + f3.y));
                    sum += __shfl_xor_sync(0xffffffffu, sum, 1);
                    sum += __shfl_xor_sync(0xffffffffu, sum, 2);
                    sum += __shfl_xor_sync(0xffffffffu, sum, 4);
                    if (ch == 0) s_qs[g][r] = sum;
                }
                fence_proxy_async_shared();
                __syncwarp();
                if (lane == 0) mbar_arrive(&b_q);
                named_bar(5, kTileSoft * 32);           // the rows' sums
            }
            const uint32_t t_row = tmem + ((uint32_t)(32 * q4) << 16);
            const int rr = min(rt * kTileRows + r, q.rows - 1);
            const int pos = p0 + rr / G, low = a.window > 0 ? pos - a.window + 1 : 0;
            const float sl2 = a.scale == 0.f ? 1.f : fabsf(a.scale) * kLog2e;
            float qs[NG], B[NG];
#pragma unroll
            for (int g = 0; g < NG; g++) {
                qs[g] = s_qs[g][r];
                B[g] = 0.f;
            }
            float m = -INFINITY, l = 0.f, unit = 0.f, vtop = 0.f;   // vtop: largest |scale| the unit admits
            for (int t = 0; t < T; t++) {
                const uint32_t n = gt + t;
                const int slot = n % kTileSlots, st = n & 1;
                const uint32_t t_s = t_row + Sh::kS + st * Sh::kStage;
                if (ok) ok = __all_sync(0xffffffffu, fused_wait_bar(&b_full[slot], (n / kTileSlots) & 1u, c.stop) &&
                                                         fused_wait_bar(&b_s[st], (n >> 1) & 1u, c.stop));
                if (!ok) {                               // the others may still come to the barrier
                    named_bar(1 + q4, 128);
                    continue;
                }
                tc_fence_after();
                const float4* sk = reinterpret_cast<const float4*>(gScale + (size_t)slot * 2 * NG * KT) + part * (HK / 2);
                const float4* sv = sk + NG * KT / 2;
                float S[HK];
                {
                    uint32_t acc[NG][HK];
#pragma unroll
                    for (int g = 0; g < NG; g++)
#pragma unroll
                        for (int b = 0; b < HK / 8; b++) tmem_ld8_nw(t_s + g * KT + part * HK + b * 8, acc[g] + b * 8);
                    tmem_ld_wait();
#pragma unroll
                    for (int j = 0; j < HK; j++) S[j] = 0.f;
#pragma unroll
                    for (int g = 0; g < NG; g++)
#pragma unroll
                        for (int j = 0; j < HK / 2; j++) {
                            const float4 f = sk[g * (KT / 2) + j];      // two entries
                            S[2 * j] = fmaf(f.x, __uint_as_float(acc[g][2 * j]), fmaf(f.y, qs[g], S[2 * j]));
                            S[2 * j + 1] = fmaf(f.z, __uint_as_float(acc[g][2 * j + 1]), fmaf(f.w, qs[g], S[2 * j + 1]));
                        }
                }
                const int j0 = (pg0 + t / Sh::kSub) * kKvPage + (t % Sh::kSub) * KT + part * HK;
                const bool edge = j0 + HK - 1 > first_pos || j0 < last_low || !s_ok[slot];
                uint32_t vis = 0xFFFFFFFFu;
                if (edge) {
                    vis = 0;
                    const bool page = s_ok[slot] != 0;
#pragma unroll
                    for (int j = 0; j < HK; j++) {
                        if (page && j0 + j <= pos && j0 + j >= low) vis |= 1u << j;
                        else S[j] = -INFINITY;
                    }
                }
                float top = S[0];
#pragma unroll
                for (int j = 1; j < HK; j++) top = fmaxf(top, S[j]);
                s_mx[st][part][r] = top;
                named_bar(1 + q4, 128);
                top = fmaxf(fmaxf(s_mx[st][0][r], s_mx[st][1][r]), fmaxf(s_mx[st][2][r], s_mx[st][3][r])) * sl2;
                // a scale of V beyond the present unit (alike in all threads)
                const float* vm = s_vmax[slot];
                const float vmax = fmaxf(fmaxf(vm[0], vm[1]), fmaxf(vm[2], vm[3]));
                float du = 0.f;
                if (vmax > vtop && vmax < 1e30f) {
                    du = fmaxf(fminf(3.f - floorf(log2f(vmax)), 60.f), -60.f) - unit;
                    vtop = 127.f * exp2f(-(unit + du));
                }
                const bool grow = top > m + 8.f;
                if (__any_sync(0xffffffffu, grow) || du != 0.f) {
                    const float m2 = grow ? top : m;
                    const float f = (m2 == -INFINITY ? 1.f : exp2_fast(m - m2)) * exp2f(du);
                    m = m2;
                    unit += du;
                    l *= f;
#pragma unroll
                    for (int g = 0; g < NG; g++) B[g] *= f;
                    if (t > 0) {                         // O so far: this quarter's columns of the row
                        ok = __all_sync(0xffffffffu, fused_wait_bar(&b_pv[(n - 1) & 1], ((n - 1) >> 1) & 1u, c.stop));
                        if (!ok) continue;
                        tc_fence_after();
#pragma unroll
                        for (int k = 0; k < NG; k++) {
                            uint32_t o[16];
                            const uint32_t at = t_row + Sh::kO + part * (NG * 16) + k * 16;
                            tmem_ld16_nw(at, o);
                            tmem_ld_wait();
#pragma unroll
                            for (int e = 0; e < 16; e++) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                            tmem_st16(at, o);
                        }
                    }
                }
                const float ref = m == -INFINITY ? 0.f : m - unit;
#pragma unroll
                for (int j = 0; j < HK; j++) S[j] = exp2_fast(fmaf(S[j], sl2, -ref));
                float ls[4] = {S[0], S[1], S[2], S[3]};
#pragma unroll
                for (int j = 4; j < HK; j++) ls[j & 3] += S[j];
                l += (ls[0] + ls[1]) + (ls[2] + ls[3]);
                const auto store = [&](auto some) {
                    constexpr bool EDGE = decltype(some)::value;
#pragma unroll
                    for (int g = 0; g < NG; g++) {
                        uint32_t P[HK / 2];
                        float b2[2] = {0.f, 0.f};
#pragma unroll
                        for (int j = 0; j < HK / 2; j++) {
                            const float4 f = sv[g * (KT / 2) + j];
                            // an entry out of sight may hold a NaN scale
                            const bool v0 = !EDGE || ((vis >> (2 * j)) & 1u), v1 = !EDGE || ((vis >> (2 * j + 1)) & 1u);
                            P[j] = f2h(v0 ? S[2 * j] * f.x : 0.f, v1 ? S[2 * j + 1] * f.z : 0.f);
                            if (v0) b2[0] = fmaf(S[2 * j], f.y, b2[0]);
                            if (v1) b2[1] = fmaf(S[2 * j + 1], f.w, b2[1]);
                        }
                        B[g] += b2[0] + b2[1];
                        const uint32_t at = t_s + g * (KT / 2) + part * (HK / 2);
                        if (HK == 16) tmem_st8(at, P);
                        else tmem_st4(at, P);
                    }
                };
                if (edge) store(BoolC<true>{});
                else store(BoolC<false>{});
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&b_p[st]);
            }
            // row sums of the four quarters, then this quarter's columns
            s_sum[part][NG][r] = l;
#pragma unroll
            for (int g = 0; g < NG; g++) s_sum[part][g][r] = B[g];
            named_bar(1 + q4, 128);
            if (ok) ok = __all_sync(0xffffffffu, fused_wait_bar(&b_pv[(gt + T - 1) & 1], ((gt + T - 1) >> 1) & 1u, c.stop));
            tc_fence_after();
            if (ok) {
                const float L = (s_sum[0][NG][r] + s_sum[1][NG][r]) + (s_sum[2][NG][r] + s_sum[3][NG][r]);
                const float M = m == -INFINITY ? m : m - unit;
                const bool whole = u == ie && ib >= blockIdx.x * per;
                const bool row = rt * kTileRows + r < q.rows;
                const int c0 = (int)(ib / per);
                float* slot = x.part + (size_t)(2 * blockIdx.x + (c0 == (int)blockIdx.x ? 1 : 0)) * (kTileRows * (D + 2));
                const int head = h * G + rr % G;
                const float f = L == 0.f ? 0.f : 1.f / L;
                __half* out = a.out + (size_t)(q.first + rr / G) * a.out_stride + (size_t)head * D;
#pragma unroll
                for (int k = 0; k < NG; k++) {
                    const int col = part * (NG * 16) + k * 16;
                    uint32_t o[16];
                    tmem_ld16_nw(t_row + Sh::kO + col, o);
                    tmem_ld_wait();
                    const int g = col / 64;
                    const float bb = (s_sum[0][g][r] + s_sum[1][g][r]) + (s_sum[2][g][r] + s_sum[3][g][r]);
                    if (!row) continue;
                    float v[16];
#pragma unroll
                    for (int e = 0; e < 16; e++) v[e] = __uint_as_float(o[e]) + bb;
                    if (whole) {
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
                if (part == 0 && row) {
                    if (whole) {
                        a.lse[(size_t)(q.first + rr / G) * c.hq + head] = L == 0.f ? -INFINITY : (M + log2f(L)) * kLn2;
                    } else {
                        slot[kTileRows * D + r] = M;
                        slot[kTileRows * D + kTileRows + r] = L;
                    }
                }
            }
            tc_fence_before();
        } else if (warp < kTileSoft + 4) {
            // --------------------------------------------------- converters --
            const int ct = tid - kTileSoft * 32, cw = warp - kTileSoft;
            const int32_t* trow = c.table + (size_t)s * c.max_pages;
            const int vw = ct & 7, vk = (ct >> 3) % (KT / 8), vg = (ct >> 3) / (KT / 8);   // V: 8 x 8 codes each
            const int eg = ct / KT, ee = ct % KT;                                          // scale and bias of one entry
            // a tile's raw bytes, two sets in turn: the next tile's loads are in flight while
            // one is converted
            struct Raw {
                uint4 k[2];
                uint32_t v[8], ks, vs;
                bool page;
            } raw[2];
            const auto page_at = [&](int t) {            // -1: behind the last entry
                const int pg = pg0 + t / Sh::kSub;
                return t < T && pg * kKvPage < q.len ? trow[pg] : -1;
            };
            int id = page_at(0);                         // of the next tile to load, read one ahead
            const auto load = [&](Raw& w, int t) {
                w.page = (unsigned)id < (unsigned)c.n_pages;
                if (!w.page) {
                    if (ct == 0 && (pg0 + t / Sh::kSub) * kKvPage < q.len) kv_flag(c.status);
                    w.k[0] = w.k[1] = make_uint4(0, 0, 0, 0);
#pragma unroll
                    for (int i = 0; i < 8; i++) w.v[i] = 0;
                    w.ks = w.vs = 0;
                } else {
                    const uint8_t* tile = c.pages + ((size_t)id * c.hkv + h) * (size_t)(4608 * NG);
                    const int sub = (t % Sh::kSub) * KT;
#pragma unroll
                    for (int i = 0; i < 2; i++) {
                        const int n = i * 128 + ct, g = n / (KT * 2);
                        if (g < NG)
                            w.k[i] = __ldg(reinterpret_cast<const uint4*>(tile + g * 2048 + sub * 32 + (n % (KT * 2)) * 16));
                    }
                    if (vg < NG) {
                        const uint8_t* v = tile + 2304 * NG + vg * 2048 + (sub + vk * 8) * 32 + vw * 4;
#pragma unroll
                        for (int i = 0; i < 8; i++) w.v[i] = __ldg(reinterpret_cast<const uint32_t*>(v + i * 32));
                    }
                    if (eg < NG) {
                        const uint8_t* sp = tile + 2048 * NG + (eg * kKvPage + sub + ee) * 4;
                        w.ks = __ldg(reinterpret_cast<const uint32_t*>(sp));
                        w.vs = __ldg(reinterpret_cast<const uint32_t*>(sp + 2304 * NG));
                    }
                }
                id = page_at(t + 1);
            };
            const auto convert = [&](const Raw& w, int t) {
                const uint32_t n = gt + t;
                const int slot = n % kTileSlots;
                // the slot's last user, P V of tile t - 3, has ended (tiles of earlier segments: all have)
                if (t >= kTileSlots)
                    ok = __all_sync(0xffffffffu, fused_wait_bar(&b_pv[(n - kTileSlots) & 1],
                                                                ((n - kTileSlots) >> 1) & 1u, c.stop));
                if (!ok) return;
                uint8_t* gk = gSlots + slot * Sh::kSlot;
                uint8_t* gv = gk + Sh::kK;
#pragma unroll
                for (int i = 0; i < 2; i++) {
                    const int nn = i * 128 + ct, g = nn / (KT * 2), r = (nn >> 1) % KT, hf = nn & 1;
                    if (g < NG) {
                        const uint32_t word[4] = {w.k[i].x, w.k[i].y, w.k[i].z, w.k[i].w};
#pragma unroll
                        for (int k = 0; k < 4; k++)
                            *reinterpret_cast<uint4*>(gk + g * (KT * 128) + r * 128 + (((hf * 4 + k) ^ (r & 7)) << 4)) =
                                codes_centred(word[k]);
                    }
                }
                if (vg < NG) {
#pragma unroll
                    for (int hf = 0; hf < 2; hf++) {     // columns 0..3, then 4..7 of the block
                        uint4 e[4];                      // entries 2i, 2i + 1
#pragma unroll
                        for (int i = 0; i < 4; i++)
                            e[i] = codes_centred(__byte_perm(w.v[2 * i], w.v[2 * i + 1], hf ? 0x7632 : 0x5410));
                        uint8_t* dst = gv + vg * (64 * 128) + (8 * vw + 4 * hf) * 128;
                        const int z = 4 * hf;
                        *reinterpret_cast<uint4*>(dst + ((vk ^ z) << 4)) = make_uint4(e[0].x, e[1].x, e[2].x, e[3].x);
                        *reinterpret_cast<uint4*>(dst + 128 + ((vk ^ (z + 1)) << 4)) = make_uint4(e[0].y, e[1].y, e[2].y, e[3].y);
                        *reinterpret_cast<uint4*>(dst + 256 + ((vk ^ (z + 2)) << 4)) = make_uint4(e[0].z, e[1].z, e[2].z, e[3].z);
                        *reinterpret_cast<uint4*>(dst + 384 + ((vk ^ (z + 3)) << 4)) = make_uint4(e[0].w, e[1].w, e[2].w, e[3].w);
                    }
                }
                // scales: entries that no row of the tile sees count as zero, whatever they hold
                float vm = 0.f;
                if (eg < NG) {
                    const int j = (pg0 + t / Sh::kSub) * kKvPage + (t % Sh::kSub) * KT + ee;
                    const bool in = w.page && j <= last_pos && j >= first_low;
                    const float2 fk = in ? h2f(w.ks) : make_float2(0.f, 0.f), fv = in ? h2f(w.vs) : make_float2(0.f, 0.f);
                    float2* sc = gScale + (size_t)slot * 2 * NG * KT + eg * KT + ee;
                    sc[0] = make_float2(fk.x, fmaf(8.f, fk.x, fk.y));
                    sc[NG * KT] = make_float2(fv.x, fmaf(8.f, fv.x, fv.y));
                    vm = fabsf(fv.x);
                }
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) vm = fmaxf(vm, __shfl_xor_sync(0xffffffffu, vm, o));
                if (lane == 0) s_vmax[slot][cw] = vm;
                if (ct == 0) s_ok[slot] = w.page;
                fence_proxy_async_shared();
                __syncwarp();
                if (lane == 0) mbar_arrive(&b_full[slot]);
            };
            load(raw[0], 0);
            for (int t = 0; ok && t < T; t += 2) {
                if (t + 1 < T) load(raw[1], t + 1);
                convert(raw[0], t);
                if (t + 2 < T) load(raw[0], t + 2);
                if (ok && t + 1 < T) convert(raw[1], t + 1);
            }
        } else if (lane == 0) {
            // --------------------------------------------------- MMA issuer --
            constexpr uint32_t id_s = kTcIdescF16 | ((uint32_t)(KT >> 3) << 17);
            constexpr uint32_t id_o = kTcIdescF16 | (8u << 17);
            const uint64_t dq = tc_sdesc_sw128(sQ);
            const auto pv = [&](int t) {
                const uint32_t n = gt + t;
                const int slot = n % kTileSlots, st = n & 1;
                if (!fused_wait_bar(&b_p[st], (n >> 1) & 1u, c.stop)) return false;
                tc_fence_after();
                const uint64_t dv = tc_sdesc_sw128(sSlots + slot * Sh::kSlot + Sh::kK);
#pragma unroll
                for (int g = 0; g < NG; g++)
#pragma unroll
                    for (int k = 0; k < KT / 16; k++)
                        tc_mma_ts(tmem + Sh::kO + g * 64, tmem + Sh::kS + st * Sh::kStage + g * (KT / 2) + 8 * k,
                                  dv + (uint64_t)((g * 64 * 128) >> 4) + 2u * k, id_o, t > 0 || k > 0 ? 1u : 0u);
                mma_commit(&b_pv[st]);
                return true;
            };
            if (!fused_wait_bar(&b_q, seg & 1u, c.stop)) ok = false;
            int done = 0, asked = 0;                     // tiles whose P V and whose Q K have been issued
            for (int t = 0; ok && t < T; t++) {
                const uint32_t n = gt + t;
                const int slot = n % kTileSlots, st = n & 1;
                if (!fused_wait_bar(&b_full[slot], (n / kTileSlots) & 1u, c.stop) ||
                    // the stage's P of tile t - 2 has been used
                    (t >= 2 && !fused_wait_bar(&b_pv[st], ((n - 2) >> 1) & 1u, c.stop))) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint64_t dk = tc_sdesc_sw128(sSlots + slot * Sh::kSlot);
#pragma unroll
                for (int g = 0; g < NG; g++)
#pragma unroll
                    for (int k = 0; k < 4; k++)
                        tc_mma_ss(tmem + Sh::kS + st * Sh::kStage + g * KT, dq + (uint64_t)((g * kTileRows * 128) >> 4) + 2u * k,
                                  dk + (uint64_t)((g * KT * 128) >> 4) + 2u * k, id_s, k > 0 ? 1u : 0u);
                mma_commit(&b_s[st]);
                asked = t + 1;
                if (t > 0) {
                    if (!pv(t - 1)) { ok = false; break; }
                    done = t;
                }
            }
            if (ok && !pv(T - 1)) ok = false;
            else if (ok) done = T;
            // every commit has arrived before the segment ends
            if (done > 0) mma_drain_wait(&b_pv[(gt + done - 1) & 1], ((gt + done - 1) >> 1) & 1u);
            if (!ok && asked > 0) mma_drain_wait(&b_s[(gt + asked - 1) & 1], ((gt + asked - 1) >> 1) & 1u);
        }
        gt += T;
        seg++;
        if (ib >= blockIdx.x * per && u < ie) {         // the item goes on in the next CTA
            cut = true;
            if (tid == 0) x.cut[blockIdx.x] = TileCut{(int)((ie - 1) / per) - (int)blockIdx.x + 1, q.first, q.rows, rt, h};
        }
        // a role that gave up has recorded it: all leave together; shared memory is free then
        if (__syncthreads_or(!ok)) {
            cut = false;
            break;
        }
    }
    if (tid == 0 && !cut) x.cut[blockIdx.x].parts = 0;
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
    }
}

// Joins the parts of the item that begins in CTA blockIdx.x: rows 32 blockIdx.y ..
// of its tile, one per lane, 16 columns a warp at a time.
constexpr int kJoinThreads = 256;

template <int NG>
__global__ void __launch_bounds__(kJoinThreads) k_attn_join(const TileArgs x) {
    constexpr int D = 64 * NG;
    constexpr size_t kSlot = (size_t)kTileRows * (D + 2);
    kv_begin();
    const TileCut c = x.cut[blockIdx.x];
    const int r = blockIdx.y * 32 + (threadIdx.x & 31), rr = c.rt * kTileRows + r;
    if (c.parts <= 0 || rr >= c.rows) return;
    const int G = x.a.c.hq / x.a.c.hkv, head = c.h * G + rr % G;
    // the first part is its CTA's second slot, the others their CTAs' first
    const auto at = [&](int b) { return x.part + (size_t)(2 * ((int)blockIdx.x + b) + (b == 0 ? 1 : 0)) * kSlot; };
    float M = -INFINITY, L = 0.f;
#pragma unroll 8
    for (int b = 0; b < c.parts; b++) M = fmaxf(M, at(b)[kTileRows * D + r]);
    const float ref = M == -INFINITY ? 0.f : M;
#pragma unroll 8
    for (int b = 0; b < c.parts; b++) {
        const float mb = at(b)[kTileRows * D + r], lb = at(b)[kTileRows * D + kTileRows + r];
        L = fmaf(mb == -INFINITY && lb == 0.f ? 0.f : exp2_fast(mb - ref), lb, L);
    }
    const float inv = L == 0.f ? 0.f : 1.f / L;
    const size_t row = (size_t)c.first + rr / G;
    for (int col = (threadIdx.x >> 5) * 16; col < D; col += kJoinThreads / 32 * 16) {
        float o[16];
#pragma unroll
        for (int e = 0; e < 16; e++) o[e] = 0.f;
#pragma unroll 4
        for (int b = 0; b < c.parts; b++) {
            const float mb = at(b)[kTileRows * D + r], lb = at(b)[kTileRows * D + kTileRows + r];
            const float f = mb == -INFINITY && lb == 0.f ? 0.f : exp2_fast(mb - ref);
#pragma unroll
            for (int e = 0; e < 4; e++) {
                const float4 v = *reinterpret_cast<const float4*>(at(b) + ((size_t)(col / 4 + e) * kTileRows + r) * 4);
                o[4 * e] = fmaf(f, v.x, o[4 * e]);
                o[4 * e + 1] = fmaf(f, v.y, o[4 * e + 1]);
                o[4 * e + 2] = fmaf(f, v.z, o[4 * e + 2]);
                o[4 * e + 3] = fmaf(f, v.w, o[4 * e + 3]);
            }
        }
        __half* out = x.a.out + row * x.a.out_stride + (size_t)head * D + col;
#pragma unroll
        for (int e = 0; e < 2; e++)
            *reinterpret_cast<uint4*>(out + 8 * e) =
                make_uint4(f2h(o[8 * e] * inv, o[8 * e + 1] * inv), f2h(o[8 * e + 2] * inv, o[8 * e + 3] * inv),
                           f2h(o[8 * e + 4] * inv, o[8 * e + 5] * inv), f2h(o[8 * e + 6] * inv, o[8 * e + 7] * inv));
    }
    if (threadIdx.x < 32) x.a.lse[row * x.a.c.hq + head] = L == 0.f ? -INFINITY : (M + log2f(L)) * kLn2;
}

}  // namespace moeq4
