// kv_weights.cuh -- the weight that each cache entry received from a call's
// rows, added to its score: score[s][h][j] += sum over rows r and the query
// heads of kv head h of exp(S_rj - lse_r).
//
// The weights need the rows' final lse, so the scores are formed a second time,
// from K alone (half of the cache's bytes).  Entries are the rows of the
// tensor-core products here (m16n8k16: 16 entries x 8 query rows), so a warp
// unpacks its entries' codes once, keeps them as operands in registers and runs
// over all query rows, which come in blocks of 64 through shared memory; each
// thread sums its entries' weights over rows in a register, and every score is
// written by one thread: the result does not depend on the order in which CTAs
// run.  With few rows the kernel is bound by reading K, with many by the fold of
// the groups' sums (S = sum_g s_g q_g . (c_g - 8) + (b_g + 8 s_g) sum(q_g)) and the
// exponentials.  A unit is what the eight warps of a CTA hold at once: 256 entries
// (128 with wide heads) when rows are few; 64 when there are many (MANY), each 16
// held by two warps that take every second 8 rows and add up at the end, because
// the entries alone do not fill the device (256 rows over 2,900 entries: 96 units of
// 256, 127 us; 368 of 64).  CTAs take equal runs of units, over all sequences and kv
// heads.
#pragma once
#include "kv_attn.cuh"

namespace moeq4 {

constexpr int kWtWarps = 8;
constexpr int kWtThreads = kWtWarps * 32;
constexpr int kWtBlock = 64;           // query rows in shared memory

template <int NG, bool MANY>
struct WtShape {
    static constexpr int kD = 64 * NG;
    static constexpr int kSets = NG <= 2 && !MANY ? 2 : 1;      // 16 entries each, per warp
    static constexpr int kGroups = MANY ? 4 : 8;                // warps with entries of their own
    static constexpr int kSplit = kWtWarps / kGroups;           // warps that share the rows of the same entries
    static constexpr int kUnit = kGroups * 16 * kSets;          // entries a CTA holds: 4, 2 or 1 pages
    static constexpr int kQ = NG * 2 * 32 * 16;                 // operands of 8 query rows, bytes
    static constexpr int kSmem = kWtBlock / 8 * kQ;
};

struct WtSeq {
    int n, first, len, units;          // units of one kv head
    int lo;                            // first entry any row sees, rounded down to a unit
};
template <int UNIT>
__device__ __forceinline__ WtSeq wt_seq(const AttnArgs& a, int s) {
    const KvArgs& c = a.c;
    WtSeq q;
    q.n = kv_rows(c, s, &q.first, false);
    q.len = kv_len(c, s, false);
    const int p0 = q.len - q.n;
    q.lo = (a.window > 0 ? max(0, p0 - a.window + 1) : 0) / UNIT * UNIT;
    q.units = q.n == 0 ? 0 : (max(0, q.len - q.lo) + UNIT - 1) / UNIT;
    return q;
}

template <int NG, bool MANY>
__global__ void __launch_bounds__(kWtThreads, 2) k_attn_weights(const AttnArgs a) {
    using Sh = WtShape<NG, MANY>;
    constexpr int D = Sh::kD, SETS = Sh::kSets, UNIT = Sh::kUnit;
    extern __shared__ __align__(128) uint8_t wt_smem[];
    __shared__ __align__(16) float s_qs[kWtBlock / 8][NG][8];
    __shared__ __align__(16) float s_lse[kWtBlock];
    __shared__ __align__(16) int s_pos[kWtBlock];
    __shared__ float s_part[kWtWarps][16];
    __shared__ long long s_total, s_base0;
    __shared__ int s_seq;
    const KvArgs& c = a.c;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g8 = lane >> 2, t4 = lane & 3;
    const int G = c.hq / c.hkv;
    kv_begin();
    // units of all sequences and kv heads, this CTA's run and the sequence it begins in
    if (warp == 0) {
        long long total = 0;
        for (int s0 = 0; s0 < c.n_seqs; s0 += 32)
            total += s0 + lane < c.n_seqs ? (long long)wt_seq<UNIT>(a, s0 + lane).units * c.hkv : 0;
        total = warp_sum(total);
        const long long per = (total + gridDim.x - 1) / gridDim.x, u = blockIdx.x * per;
        long long base = 0;
        int found = 0;
        for (int s0 = 0; u < total && s0 < c.n_seqs; s0 += 32) {
            const long long w = s0 + lane < c.n_seqs ? (long long)wt_seq<UNIT>(a, s0 + lane).units * c.hkv : 0;
            long long inc = w;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long y = __shfl_up_sync(0xffffffffu, inc, o);
                if (lane >= o) inc += y;
            }
            const unsigned hit = __ballot_sync(0xffffffffu, base + inc > u);
            if (hit) {
                const int at = __ffs(hit) - 1;
                found = s0 + at;
                base += __shfl_sync(0xffffffffu, inc - w, at);
                break;
            }
            base += __shfl_sync(0xffffffffu, inc, 31);
        }
        if (lane == 0) {
            s_total = total;
            s_base0 = base;
            s_seq = found;
        }
    }
    __syncthreads();
    const long long total = s_total, per = (total + gridDim.x - 1) / gridDim.x;
    long long u = blockIdx.x * per, base = s_base0;
    const long long u_end = min(total, u + per);
    if (u >= u_end) return;
    int s = s_seq, h_now = -1, s_now = -1, blk_now = -1;
    WtSeq q = wt_seq<UNIT>(a, s);
    const uint32_t qb = smem_u32(wt_smem);
    const float sl2 = a.scale * kLog2e;

    for (; u < u_end; u++) {
        while (u >= base + (long long)q.units * c.hkv) {
            base += (long long)q.units * c.hkv;
            s++;
            q = wt_seq<UNIT>(a, s);
        }
        const int h = (int)((u - base) / q.units);
        const int e0 = q.lo + (int)((u - base) % q.units) * UNIT;        // first entry of the unit
        const int j0 = e0 + warp % Sh::kGroups * (16 * SETS);            // of this warp
        const int p0 = q.len - q.n, rows = q.n * G;
        // this warp's entries lie in one page
        const int pg = j0 / kKvPage;
        const int id = j0 < q.len ? c.table[(size_t)s * c.max_pages + pg] : -1;
        const bool in = (unsigned)id < (unsigned)c.n_pages;
        if (!in && j0 < q.len && lane == 0) kv_flag(c.status);
        uint32_t kf[SETS][NG][4][4];                                     // operand: step m, register
        float2 sb[SETS][NG][2];                                          // scale, bias + 8 scale of entries g8, g8 + 8
        {
            const uint8_t* tile = c.pages + ((size_t)(in ? id : 0) * c.hkv + h) * (size_t)(4608 * NG);
            uint2 w[SETS][NG][2];
            uint32_t f[SETS][NG][2];
#pragma unroll
            for (int z = 0; z < SETS; z++)
#pragma unroll
                for (int g = 0; g < NG; g++)
#pragma unroll
                    for (int k = 0; k < 2; k++) {
                        const int e = (j0 + 16 * z + 8 * k + g8) % kKvPage;
                        w[z][g][k] = make_uint2(0, 0);
                        f[z][g][k] = 0;
                        if (in) {
                            w[z][g][k] = __ldg(reinterpret_cast<const uint2*>(tile + (g * kKvPage + e) * 32 + t4 * 8));
                            f[z][g][k] = __ldg(reinterpret_cast<const uint32_t*>(tile + 2048 * NG + (g * kKvPage + e) * 4));
                        }
                    }
#pragma unroll
            for (int z = 0; z < SETS; z++)
#pragma unroll
                for (int g = 0; g < NG; g++)
#pragma unroll
                    for (int k = 0; k < 2; k++) {
                        const uint4 x0 = codes_centred(w[z][g][k].x), x1 = codes_centred(w[z][g][k].y);
                        kf[z][g][0][k] = x0.x; kf[z][g][1][k] = x0.y; kf[z][g][2][k] = x0.z; kf[z][g][3][k] = x0.w;
                        kf[z][g][0][2 + k] = x1.x; kf[z][g][1][2 + k] = x1.y; kf[z][g][2][2 + k] = x1.z; kf[z][g][3][2 + k] = x1.w;
                        const float2 v = h2f(f[z][g][k]);
                        sb[z][g][k] = make_float2(v.x, fmaf(8.f, v.x, v.y));
                    }
        }
        float sum[SETS][2];
#pragma unroll
        for (int z = 0; z < SETS; z++) sum[z][0] = sum[z][1] = 0.f;

        // rows that see any of the unit's entries: p0 + i >= e0, and low <= last entry
        const int i0 = max(0, e0 - p0);
        const int i1 = a.window > 0 ? (int)min((long long)q.n - 1, (long long)min(e0 + UNIT, q.len) - 1 + a.window - 1 - p0) : q.n - 1;
        const int blk0 = i0 * G / kWtBlock, blk1 = i1 < i0 ? blk0 - 1 : (i1 * G + G - 1) / kWtBlock;
        for (int blk = blk0; blk <= blk1; blk++) {
            if (s != s_now || h != h_now || blk != blk_now) {            // alike in the whole CTA
                __syncthreads();
                // query rows into operand order: thread 4 r + t takes 16 columns of each group of row r
                const int t = tid & 3, r = tid >> 2, rr = blk * kWtBlock + r;
                const bool on = rr < rows;
                const int row = q.first + min(rr, rows - 1) / G, head = h * G + min(rr, rows - 1) % G;
                const float lse_now = t == 0 && on ? a.lse[(size_t)row * c.hq + head] : -INFINITY;
#pragma unroll
                for (int g = 0; g < NG; g++) {
                    uint4 v0 = make_uint4(0, 0, 0, 0), v1 = v0;
                    if (on) {
                        const __half* qp = a.q + (size_t)row * a.q_stride + (size_t)head * D + g * 64 + t * 16;
                        v0 = *reinterpret_cast<const uint4*>(qp);
                        v1 = *reinterpret_cast<const uint4*>(qp + 8);
                    }
                    // two steps of 16 columns per 16 bytes
                    uint4* dst = reinterpret_cast<uint4*>(wt_smem + (r >> 3) * Sh::kQ) + (g * 2) * 32 + (r & 7) * 4 + t;
                    dst[0] = make_uint4(__byte_perm(v0.x, v0.z, 0x5410), __byte_perm(v1.x, v1.z, 0x5410),
                                        __byte_perm(v0.x, v0.z, 0x7632), __byte_perm(v1.x, v1.z, 0x7632));
                    dst[32] = make_uint4(__byte_perm(v0.y, v0.w, 0x5410), __byte_perm(v1.y, v1.w, 0x5410),
                                         __byte_perm(v0.y, v0.w, 0x7632), __byte_perm(v1.y, v1.w, 0x7632));
                    const uint32_t w[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
                    float qsum = 0.f;
#pragma unroll
                    for (int k = 0; k < 8; k++) {
                        const float2 f = h2f(w[k]);
                        qsum += f.x + f.y;
                    }
                    qsum += __shfl_xor_sync(0xffffffffu, qsum, 1);
                    qsum += __shfl_xor_sync(0xffffffffu, qsum, 2);
                    if (t == 0) s_qs[r >> 3][g][r & 7] = qsum;
                }
                if (t == 0) {
                    s_lse[r] = lse_now == -INFINITY ? INFINITY : lse_now * kLog2e;   // such rows add nothing
                    s_pos[r] = p0 + min(rr, rows - 1) / G;
                }
                s_now = s;
                h_now = h;
                blk_now = blk;
                __syncthreads();
            }
            if (!in) continue;
            const int tiles = min(kWtBlock, rows - blk * kWtBlock + 7) / 8;
            // PAIR row tiles side by side: their products and exponentials hide each other's latency
            constexpr int PAIR = MANY ? 2 : 1;
            for (int rt0 = warp / Sh::kGroups * PAIR; rt0 < tiles; rt0 += Sh::kSplit * PAIR) {
                const int r0 = rt0 * 8, r1 = min(r0 + 8 * PAIR, rows - blk * kWtBlock) - 1;
                const int pmin = s_pos[r0], pmax = s_pos[r1];
                if (pmax < j0) continue;                                 // all before these entries
                if (a.window > 0 && pmin - a.window + 1 > j0 + 16 * SETS - 1) continue;
                const bool edge = j0 + 16 * SETS - 1 > pmin || (a.window > 0 && j0 < pmax - a.window + 1);
                float S[PAIR][SETS][4];
#pragma unroll
                for (int y = 0; y < PAIR; y++)
#pragma unroll
                    for (int z = 0; z < SETS; z++)
#pragma unroll
                        for (int k = 0; k < 4; k++) S[y][z][k] = 0.f;
#pragma unroll
                for (int g = 0; g < NG; g++)
#pragma unroll
                    for (int y = 0; y < PAIR; y++) {
                        // rows behind the block's last are zero there, and add nothing
                        const uint4 b0 = lds128(qb + (rt0 + y) * Sh::kQ + ((g * 2) * 32 + lane) * 16);
                        const uint4 b1 = lds128(qb + (rt0 + y) * Sh::kQ + ((g * 2 + 1) * 32 + lane) * 16);
                        const float2 qs = *reinterpret_cast<const float2*>(&s_qs[rt0 + y][g][2 * t4]);
#pragma unroll
                        for (int z = 0; z < SETS; z++) {
                            const uint32_t(&k)[4][4] = kf[z][g];
                            float(&S4)[4] = S[y][z];
                            float d[4];
                            mma_f16(d, k[0][0], k[0][1], k[0][2], k[0][3], b0.x, b0.y, 0.f, 0.f, 0.f, 0.f);
                            mma_f16(d, k[1][0], k[1][1], k[1][2], k[1][3], b0.z, b0.w);
                            mma_f16(d, k[2][0], k[2][1], k[2][2], k[2][3], b1.x, b1.y);
                            mma_f16(d, k[3][0], k[3][1], k[3][2], k[3][3], b1.z, b1.w);
                            const float2 f0 = sb[z][g][0], f1 = sb[z][g][1];
                            S4[0] = fmaf(f0.x, d[0], fmaf(f0.y, qs.x, S4[0]));
                            S4[1] = fmaf(f0.x, d[1], fmaf(f0.y, qs.y, S4[1]));
                            S4[2] = fmaf(f1.x, d[2], fmaf(f1.y, qs.x, S4[2]));
                            S4[3] = fmaf(f1.x, d[3], fmaf(f1.y, qs.y, S4[3]));
                        }
                    }
#pragma unroll
                for (int y = 0; y < PAIR; y++) {
                    const float2 lse = *reinterpret_cast<const float2*>(&s_lse[r0 + 8 * y + 2 * t4]);
#pragma unroll
                    for (int z = 0; z < SETS; z++) {
                        const float(&S4)[4] = S[y][z];
                        float w[4] = {exp2_fast(fmaf(S4[0], sl2, -lse.x)), exp2_fast(fmaf(S4[1], sl2, -lse.y)),
                                      exp2_fast(fmaf(S4[2], sl2, -lse.x)), exp2_fast(fmaf(S4[3], sl2, -lse.y))};
                        if (edge) {
                            const int2 p = *reinterpret_cast<const int2*>(&s_pos[r0 + 8 * y + 2 * t4]);
#pragma unroll
                            for (int k = 0; k < 4; k++) {
                                const int j = j0 + 16 * z + 8 * (k >> 1) + g8, at = k & 1 ? p.y : p.x;
                                if (j > at || (a.window > 0 && j <= at - a.window)) w[k] = 0.f;
                            }
                        }
                        sum[z][0] += w[0] + w[1];
                        sum[z][1] += w[2] + w[3];
                    }
                }
            }
        }
        if (Sh::kSplit > 1) {                                            // the partner's sums, to the first of the two
            if (warp >= Sh::kGroups) {
#pragma unroll
                for (int k = 0; k < 2; k++) {
                    float v = sum[0][k];
                    v += __shfl_xor_sync(0xffffffffu, v, 1);
                    v += __shfl_xor_sync(0xffffffffu, v, 2);
                    if (t4 == 0) s_part[warp][8 * k + g8] = v;
                }
            }
            __syncthreads();
        }
        if (in && blk1 >= blk0 && warp < Sh::kGroups) {
            float* score = c.score + ((size_t)s * c.hkv + h) * ((size_t)c.max_pages * kKvPage);
#pragma unroll
            for (int z = 0; z < SETS; z++)
#pragma unroll
                for (int k = 0; k < 2; k++) {
                    float v = sum[z][k];
                    v += __shfl_xor_sync(0xffffffffu, v, 1);
                    v += __shfl_xor_sync(0xffffffffu, v, 2);
                    const int j = j0 + 16 * z + 8 * k + g8;
                    if (Sh::kSplit > 1) v += s_part[warp + Sh::kGroups][8 * k + g8];
                    if (t4 == 0 && j < q.len) score[j] += v;
                }
        }
        if (Sh::kSplit > 1) __syncthreads();                             // s_part is free again
    }
}

}  // namespace moeq4
