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
// run.  Scores are S = sum_g s_g q_g . (c_g - 8) + (b_g + 8 s_g) sum(q_g).
//
// A unit is what the eight warps of a CTA hold at once.  Few rows (one block, up to
// kWtBlock (row, head) pairs): 256 entries, 128 with wide heads; the queries stay in
// shared memory while sequence and kv head do, and reading K is the bound.  More
// (MANY): 64 entries, each 16 held by two warps that take every second pair of row
// tiles and add up at the end, because the entries alone do not fill the device (256
// rows of 5 heads over 2,900 entries: 96 units of 256, 127 us; 368 of 64).  Blocks of
// rows then come by asynchronous copies, two blocks ahead, and ldmatrix deals them to
// the threads as they lie, with the codes of K dealt to match: bringing every block
// into operand order in registers, for every unit, was 40 % of the instructions (the
// whole call 150 us, now 132, of which 50 are this kernel).  What bounds it there is
// issue (51 % of the slots; 28 % of the tensor pipe, 14 % of the exponentials'), with
// three CTAs per SM; two take 153 us.  CTAs take equal runs of units, over all
// sequences and kv heads.
#pragma once
#include "kv_attn.cuh"

namespace moeq4 {

constexpr int kWtWarps = 8;
constexpr int kWtThreads = kWtWarps * 32;
constexpr int kWtBlock = 64;           // query rows in shared memory
constexpr uint32_t kOnes = 0x3C003C00u; // fp16 1, 1

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool on) {     // else zeros
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void ldmatrix4(uint32_t& r0, uint32_t& r1, uint32_t& r2, uint32_t& r3, uint32_t at) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3) : "r"(at) : "memory");
}

template <int NG, bool MANY>
struct WtShape {
    static constexpr int kD = 64 * NG;
    static constexpr int kSets = NG <= 2 && !MANY ? 2 : 1;      // 16 entries each, per warp
    static constexpr int kGroups = MANY ? 4 : 8;                // warps with entries of their own
    static constexpr int kSplit = kWtWarps / kGroups;           // warps that share the rows of the same entries
    static constexpr int kUnit = kGroups * 16 * kSets;          // entries a CTA holds: 4, 2 or 1 pages
    static constexpr int kQ = NG * 2 * 32 * 16;                 // operands of 8 query rows, bytes
    static constexpr int kBufs = MANY ? 3 : 1;                  // blocks of query rows in shared memory
    static constexpr int kBlock = kWtBlock / 8 * kQ;
    static constexpr int kSmem = kBufs * kBlock;
    static constexpr int kCtas = MANY && NG <= 2 ? 3 : 2;       // per SM
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
__global__ void __launch_bounds__(kWtThreads, WtShape<NG, MANY>::kCtas) k_attn_weights(const AttnArgs a) {
    using Sh = WtShape<NG, MANY>;
    constexpr int D = Sh::kD, SETS = Sh::kSets, UNIT = Sh::kUnit;
    extern __shared__ __align__(128) uint8_t wt_smem[];
    __shared__ __align__(16) float s_qs[Sh::kBufs][kWtBlock / 8][NG][8];
    __shared__ __align__(16) float s_lse[Sh::kBufs][kWtBlock];
    __shared__ __align__(16) int s_pos[Sh::kBufs][kWtBlock];
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
    int s = s_seq, h_now = -1, s_now = -1;
    WtSeq q = wt_seq<UNIT>(a, s);
    const uint32_t sb_q = smem_u32(wt_smem);
    // this thread's row and chunk for ldmatrix; kBlock and D leave its bits 4..6 alone
    const uint32_t at_q = sb_q + (lane & 7) * (D * 2) + (((lane >> 3) ^ (lane & 7)) << 4);
    const float sl2 = a.scale * kLog2e;

    for (; u < u_end; u++) {
        while (u >= base + (long long)q.units * c.hkv) {
            if (s + 1 >= c.n_seqs) return;                       // (not reached while what lens says stays)
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
        if constexpr (MANY) {
            // Columns 2 t4, 2 t4 + 1 of every 8, byte t4 of every word, as ldmatrix deals query
            // rows to the threads: no block of them is put into another order.
            const uint8_t* tile = c.pages + ((size_t)(in ? id : 0) * c.hkv + h) * (size_t)(4608 * NG);
#pragma unroll
            for (int g = 0; g < NG; g++)
#pragma unroll
                for (int k = 0; k < 2; k++) {
                    const int e = (j0 + 8 * k + g8) % kKvPage;
                    uint4 w[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
                    uint32_t f = 0;
                    if (in) {
                        w[0] = *reinterpret_cast<const uint4*>(tile + (g * kKvPage + e) * 32);
                        w[1] = *reinterpret_cast<const uint4*>(tile + (g * kKvPage + e) * 32 + 16);
                        f = *reinterpret_cast<const uint32_t*>(tile + 2048 * NG + (g * kKvPage + e) * 4);
                    }
#pragma unroll
                    for (int i = 0; i < 2; i++) {
                        const int sel = t4 | (4 + t4) << 4;
                        const uint4 x = codes_centred(__byte_perm(__byte_perm(w[i].x, w[i].y, sel), __byte_perm(w[i].z, w[i].w, sel), 0x5410));
                        kf[0][g][2 * i][k] = __byte_perm(x.x, x.y, 0x5410);
                        kf[0][g][2 * i][2 + k] = __byte_perm(x.z, x.w, 0x5410);
                        kf[0][g][2 * i + 1][k] = __byte_perm(x.x, x.y, 0x7632);
                        kf[0][g][2 * i + 1][2 + k] = __byte_perm(x.z, x.w, 0x7632);
                    }
                    const float2 v = h2f(f);
                    sb[0][g][k] = make_float2(v.x, fmaf(8.f, v.x, v.y));
                }
        } else {
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
                            w[z][g][k] = *reinterpret_cast<const uint2*>(tile + (g * kKvPage + e) * 32 + t4 * 8);
                            f[z][g][k] = *reinterpret_cast<const uint32_t*>(tile + 2048 * NG + (g * kKvPage + e) * 4);
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
        // MANY: query rows by 16-byte asynchronous copies, chunk x of row r at x ^ (r % 8); block
        // i + 2 is on its way and the facts of block i + 1 are formed while block i is computed
        const auto fetch = [&](int i) {
            if (blk0 + i <= blk1) {
                const int rr = (blk0 + i) * kWtBlock + (tid >> 2), at = min(rr, rows - 1);
                const size_t row = q.first + at / G, head = h * G + at % G;
                const uint8_t* src = reinterpret_cast<const uint8_t*>(a.q + row * a.q_stride + head * D);
                const uint32_t dst = sb_q + i % Sh::kBufs * Sh::kBlock + (tid >> 2) * (D * 2);
#pragma unroll
                for (int k = 0; k < 2 * NG; k++) {
                    const int x = 4 * k + (tid & 3);
                    cp_async16(dst + (x ^ ((tid >> 2) & 7)) * 16, src + x * 16, rr < rows);
                }
                if ((tid & 3) == 0) cp_async4(smem_u32(&s_lse[i % Sh::kBufs][tid >> 2]), a.lse + row * c.hq + head);
            }
            cp_async_commit();
        };
        const auto operand = [&](int y, int rt, int g, uint32_t (&b)[8]) {       // of 8 rows of buffer y, a group
            const uint32_t at = y * Sh::kBlock + rt * 8 * (D * 2) + g * 128;
            ldmatrix4(b[0], b[1], b[2], b[3], at_q + at);
            ldmatrix4(b[4], b[5], b[6], b[7], (at_q ^ 64u) + at);
        };
        const auto facts = [&](int i) {              // sums of the queries, lse and positions
            const int y = i % Sh::kBufs;
#pragma unroll
            for (int g = 0; g < NG; g++) {
                uint32_t b[8];
                operand(y, warp, g, b);
                float d[4] = {0.f, 0.f, 0.f, 0.f};   // a product with ones
#pragma unroll
                for (int m = 0; m < 4; m++) mma_f16(d, kOnes, kOnes, kOnes, kOnes, b[2 * m], b[2 * m + 1]);
                if (g8 == 0) *reinterpret_cast<float2*>(&s_qs[y][warp][g][2 * t4]) = make_float2(d[0], d[1]);
            }
            if (tid < kWtBlock) {
                const int rr = (blk0 + i) * kWtBlock + tid;
                const float l = s_lse[y][tid];
                s_lse[y][tid] = rr >= rows || l == -INFINITY ? INFINITY : l * kLog2e;   // such rows add nothing
                s_pos[y][tid] = p0 + min(rr, rows - 1) / G;
            }
        };
        if (MANY && blk0 <= blk1) {
            fetch(0);
            fetch(1);
            cp_async_wait<1>();
            __syncthreads();
            facts(0);
        }
        for (int blk = blk0; blk <= blk1; blk++) {
            const int i = blk - blk0, buf = MANY ? i % Sh::kBufs : 0;
            if constexpr (MANY) {
                cp_async_wait<0>();
                __syncthreads();
                fetch(i + 2);
                if (blk < blk1) facts(i + 1);
            } else if (s != s_now || h != h_now) {                       // alike in the whole CTA; one block
                __syncthreads();
                // query rows into operand order: thread 4 r + t takes 16 columns of each group of row r
                const int t = tid & 3, r = tid >> 2;
                const bool on = r < rows;
                const int row = q.first + min(r, rows - 1) / G, head = h * G + min(r, rows - 1) % G;
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
                    if (t == 0) s_qs[0][r >> 3][g][r & 7] = qsum;
                }
                if (t == 0) {
                    s_lse[0][r] = lse_now == -INFINITY ? INFINITY : lse_now * kLog2e;    // such rows add nothing
                    s_pos[0][r] = p0 + min(r, rows - 1) / G;
                }
                s_now = s;
                h_now = h;
                __syncthreads();
            }
            if (!in) continue;
            const int tiles = min(kWtBlock, rows - blk * kWtBlock + 7) / 8;
            // whether every row of the block sees all of the entries
            const int last = min(kWtBlock, rows - blk * kWtBlock) - 1;
            const bool clear = s_pos[buf][0] >= j0 + 16 * SETS - 1 && (a.window == 0 || s_pos[buf][last] - a.window < j0);
            // PAIR row tiles side by side: their products and exponentials hide each other's latency
            constexpr int PAIR = MANY ? 2 : 1;
            for (int rt0 = warp / Sh::kGroups * PAIR; rt0 < tiles; rt0 += Sh::kSplit * PAIR) {
                const int r0 = rt0 * 8;
                bool edge = false;
                if (!clear) {
                    const int pmin = s_pos[buf][r0], pmax = s_pos[buf][min(r0 + 8 * PAIR, last + 1) - 1];
                    if (pmax < j0) continue;                             // all before these entries
                    if (a.window > 0 && pmin - a.window + 1 > j0 + 16 * SETS - 1) continue;
                    edge = j0 + 16 * SETS - 1 > pmin || (a.window > 0 && j0 < pmax - a.window + 1);
                }
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
                        uint32_t b[8];
                        if constexpr (MANY) {
                            operand(buf, rt0 + y, g, b);
                        } else {
                            const uint4 b0 = lds128(sb_q + (rt0 + y) * Sh::kQ + ((g * 2) * 32 + lane) * 16);
                            const uint4 b1 = lds128(sb_q + (rt0 + y) * Sh::kQ + ((g * 2 + 1) * 32 + lane) * 16);
                            b[0] = b0.x; b[1] = b0.y; b[2] = b0.z; b[3] = b0.w;
                            b[4] = b1.x; b[5] = b1.y; b[6] = b1.z; b[7] = b1.w;
                        }
                        const float2 qs = *reinterpret_cast<const float2*>(&s_qs[buf][rt0 + y][g][2 * t4]);
#pragma unroll
                        for (int z = 0; z < SETS; z++) {
                            const uint32_t(&k)[4][4] = kf[z][g];
                            float(&S4)[4] = S[y][z];
                            float d[4];
                            mma_f16(d, k[0][0], k[0][1], k[0][2], k[0][3], b[0], b[1], 0.f, 0.f, 0.f, 0.f);
                            mma_f16(d, k[1][0], k[1][1], k[1][2], k[1][3], b[2], b[3]);
                            mma_f16(d, k[2][0], k[2][1], k[2][2], k[2][3], b[4], b[5]);
                            mma_f16(d, k[3][0], k[3][1], k[3][2], k[3][3], b[6], b[7]);
                            const float2 f0 = sb[z][g][0], f1 = sb[z][g][1];
                            S4[0] = fmaf(f0.x, d[0], fmaf(f0.y, qs.x, S4[0]));
                            S4[1] = fmaf(f0.x, d[1], fmaf(f0.y, qs.y, S4[1]));
                            S4[2] = fmaf(f1.x, d[2], fmaf(f1.y, qs.x, S4[2]));
                            S4[3] = fmaf(f1.x, d[3], fmaf(f1.y, qs.y, S4[3]));
                        }
                    }
#pragma unroll
                for (int y = 0; y < PAIR; y++) {
                    const float2 lse = *reinterpret_cast<const float2*>(&s_lse[buf][r0 + 8 * y + 2 * t4]);
#pragma unroll
                    for (int z = 0; z < SETS; z++) {
                        const float(&S4)[4] = S[y][z];
                        float w[4] = {exp2_fast(fmaf(S4[0], sl2, -lse.x)), exp2_fast(fmaf(S4[1], sl2, -lse.y)),
                                      exp2_fast(fmaf(S4[2], sl2, -lse.x)), exp2_fast(fmaf(S4[3], sl2, -lse.y))};
                        if (edge) {
                            const int2 p = *reinterpret_cast<const int2*>(&s_pos[buf][r0 + 8 * y + 2 * t4]);
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
