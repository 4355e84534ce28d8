// kv_attn.cuh -- attention over the 4-bit KV cache.
#pragma once
#include "kv_cache.cuh"
#include "ptx.cuh"

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

// Scores and running sums are in units of log2: exp(S) = exp2(S log2 e).
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float exp2_fast(float x) {       // 2^x, 2 ulp; 0 for x = -inf
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// D (16 x 8, fp32) += A (16 x 16, fp16) B (16 x 8, fp16); lane = 4 g + t holds
// A rows g (a0, a2) and g + 8 (a1, a3), columns 2t, 2t + 1 (a0, a1) and 8 more
// (a2, a3); B column g, rows alike; D rows g (c0, c1) and g + 8, columns 2t, 2t + 1.
__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Nibbles i and i + 4 of w as the fp16 pair (64 + code, 64 + code'): the code
// lands in mantissa bits 4..7 of 64, so one shift and one masked or serve two
// codes and no subtraction is needed.  The constant 64 leaves the sums through
// the bias: s c + b = s (64 + c) + (b - 64 s).  64 rather than 1024 (code in the
// lowest bits) keeps the cancelling part of the fp32 sums 16 times smaller.
template <int I>
__device__ __forceinline__ uint32_t code_pair(uint32_t w) {
    const uint32_t v = I == 0 ? w << 4 : I == 1 ? w : I == 2 ? w >> 4 : w >> 8;
    return (v & 0x00F000F0u) | 0x54005400u;
}
constexpr float kCodeOff = 64.f;

__device__ __forceinline__ float2 h2f(uint32_t v) { return __half22float2(*reinterpret_cast<const __half2*>(&v)); }
__device__ __forceinline__ uint32_t f2h(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }
__device__ __forceinline__ uint2 lds64(uint32_t a) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
    return v;
}

// ------------------------------------------------------- split attention --
// Few rows per kv head (single tokens): bound by reading the cache, so every
// byte of it is read once by one warp and used from registers.
//
// An item is (sequence, tile of 8 RT rows, kv head); its rows are the
// (row, query head) pairs that read the kv head, so a group's query heads share
// each entry.  The pages of all items form one list of units; CTA c takes units
// [c per, (c + 1) per), whatever items they belong to, so ragged batches are
// even.  Eight warps: warps 0-3 take the four 16-entry parts of even pages of a
// segment, warps 4-7 of odd ones, each through its own ring of cp.async stages
// with no barrier between warps.  Per 16 entries a warp forms
//   S = sum_g s_g (q_g . (64 + c_g)) + (b_g - 64 s_g) sum(q_g)
// with tensor-core products of the raw codes (m16n8k16, rows = query rows,
// columns = entries), keeps a running maximum (moved only when it grows by
// more than 2^8: the sums are rescaled rarely) and adds
//   O += sum_j p_j s_jg (64 + c_j),   B_g += sum_j p_j (b_jg - 64 s_jg)
// where p s enters as two fp16 parts (hi, lo: 22 bits; with 8 rows the lower
// half of the 16-row tile carries lo).  p s is kept in fp16's range by a power
// of two per warp (vs), raised or lowered when needed.  The warps' sums meet in
// shared memory; an item cut by CTA borders goes through partial sums in the
// workspace, joined in a fixed order by the last CTA to arrive (one counter per
// item start, reset by that CTA).
constexpr int kSplitWarps = 8;
constexpr int kSplitThreads = kSplitWarps * 32;
constexpr int kSplitStages = 4;
constexpr int kSplitMinUnits = 4;      // pages per CTA at least: fewer partial sums in small calls

template <int NG, int RT>
struct SplitShape {
    static constexpr int kRows = 8 * RT;
    static constexpr int kD = 64 * NG;
    static constexpr int kBlock = 1152 * NG;                         // 16 entries: K and V, codes and s, b
    static constexpr int kRing = kSplitWarps * kSplitStages * kBlock;
    static constexpr int kJoin = kSplitWarps * kRows * kD * 4;       // the warps' sums, over the ring
    static constexpr int kSmem = (kRing > kJoin ? kRing : kJoin);
};

struct SplitArgs {
    AttnArgs a;
    float* part;               // [2 gridDim.x][kRows][D + 2]: sums, maximum, total
    int* count;                // [gridDim.x], zero between calls
    int max_rows_seq;          // sequences with more (row, head) pairs per kv head are not served here
};

// What one sequence asks of the split kernel.
struct SplitSeq {
    int n, first, len, plo, np, tiles, units;
};
template <int ROWS>
__device__ __forceinline__ SplitSeq split_seq(const SplitArgs& x, int s, bool report) {
    const KvArgs& c = x.a.c;
    SplitSeq q;
    q.n = kv_rows(c, s, &q.first, report);
    q.len = kv_len(c, s, report);
    const int rows = q.n * (c.hq / c.hkv), p0 = q.len - q.n;
    const int lo = x.a.window > 0 ? max(0, p0 - x.a.window + 1) : 0;
    q.plo = lo / kKvPage;
    q.np = max(1, (q.len + kKvPage - 1) / kKvPage - q.plo);
    q.tiles = rows > x.max_rows_seq ? 0 : (rows + ROWS - 1) / ROWS;
    q.units = q.tiles * c.hkv * q.np;
    return q;
}

template <int NG, int RT>
__global__ void __launch_bounds__(kSplitThreads, NG * RT <= 2 ? 2 : 1) k_attn_split(const SplitArgs x) {
    using Sh = SplitShape<NG, RT>;
    constexpr int R = Sh::kRows, D = Sh::kD;
    extern __shared__ __align__(128) uint8_t sp_smem[];
    __shared__ float s_m[kSplitWarps][R], s_l[kSplitWarps][R];
    __shared__ int s_last;
    const AttnArgs& a = x.a;
    const KvArgs& c = a.c;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g8 = lane >> 2, t4 = lane & 3;
    const int G = c.hq / c.hkv;
    const int cap_pages = c.max_pages;

    // units of all sequences, then this CTA's range
    long long total = 0;
    for (int s0 = 0; s0 < c.n_seqs; s0 += 32) {
        const int s = s0 + lane;
        total += s < c.n_seqs ? split_seq<R>(x, s, blockIdx.x == 0 && warp == 0).units : 0;
    }
    total = warp_sum(total);
    long long per = (total + gridDim.x - 1) / gridDim.x;
    if (per < kSplitMinUnits) per = kSplitMinUnits;
    long long u = blockIdx.x * per;
    const long long u_end = min(total, u + per);
    if (u >= u_end) return;

    // sequence that holds unit u, and the units before it
    int s = 0;
    long long s_base = 0;
    for (int s0 = 0; s0 < c.n_seqs; s0 += 32) {
        const int sl = s0 + lane;
        const int w = sl < c.n_seqs ? split_seq<R>(x, sl, false).units : 0;
        long long inc = w;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += y;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, s_base + inc > u);
        if (hit) {
            const int at = __ffs(hit) - 1;
            s = s0 + at;
            s_base += __shfl_sync(0xffffffffu, inc - w, at);
            break;
        }
        s_base += __shfl_sync(0xffffffffu, inc, 31);
    }
    SplitSeq q = split_seq<R>(x, s, false);

    const uint32_t ring = smem_u32(sp_smem) + warp * (kSplitStages * Sh::kBlock);
    const int sub = warp & 3, par = warp >> 2;
    const float sl2 = a.scale * kLog2e;

    while (u < u_end) {
        while (u >= s_base + q.units) {                      // sequences without units are passed over
            s_base += q.units;
            s++;
            q = split_seq<R>(x, s, false);
        }
        const int item = (int)((u - s_base) / q.np);
        const long long ib = s_base + (long long)item * q.np, ie = ib + q.np;
        const int rt = item / c.hkv, h = item % c.hkv;
        const int pg0 = q.plo + (int)(u - ib);
        const int pg1 = q.plo + (int)(min(u_end, ie) - ib);
        const int pend = (q.len + kKvPage - 1) / kKvPage;    // pages that hold entries
        const int p0 = q.len - q.n;
        const int rows = q.n * G;
        u = min(u_end, ie);

        // queries of this tile: row g8 (and g8 + 8) of the 16-row operand
        uint32_t qa[NG][4][2 * RT];
        float qs[NG][RT];
        int pos[RT], low[RT];
#pragma unroll
        for (int z = 0; z < RT; z++) {
            const int r = rt * R + g8 + 8 * z, rr = min(r, rows - 1);
            const int i = rr / G, head = h * G + rr % G;
            const __half* qp = a.q + (size_t)(q.first + i) * a.q_stride + (size_t)head * D;
            pos[z] = p0 + i;
            low[z] = a.window > 0 ? p0 + i - a.window + 1 : 0;
#pragma unroll
            for (int g = 0; g < NG; g++) {
                uint4 v0 = make_uint4(0, 0, 0, 0), v1 = v0;
                if (r < rows) {
                    v0 = *reinterpret_cast<const uint4*>(qp + g * 64 + t4 * 16);
                    v1 = *reinterpret_cast<const uint4*>(qp + g * 64 + t4 * 16 + 8);
                }
                // columns (m, m + 4) of each 8, as the code pairs come
                qa[g][0][z] = __byte_perm(v0.x, v0.z, 0x5410);
                qa[g][1][z] = __byte_perm(v0.x, v0.z, 0x7632);
                qa[g][2][z] = __byte_perm(v0.y, v0.w, 0x5410);
                qa[g][3][z] = __byte_perm(v0.y, v0.w, 0x7632);
                qa[g][0][RT + z] = __byte_perm(v1.x, v1.z, 0x5410);
                qa[g][1][RT + z] = __byte_perm(v1.x, v1.z, 0x7632);
                qa[g][2][RT + z] = __byte_perm(v1.y, v1.w, 0x5410);
                qa[g][3][RT + z] = __byte_perm(v1.y, v1.w, 0x7632);
                const uint32_t w[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
                float sum = 0.f;
#pragma unroll
                for (int k = 0; k < 8; k++) {
                    const float2 f = h2f(w[k]);
                    sum += f.x + f.y;
                }
                sum += __shfl_xor_sync(0xffffffffu, sum, 1);
                sum += __shfl_xor_sync(0xffffffffu, sum, 2);
                qs[g][z] = sum;
            }
        }
        const int first_pos = p0 + (rt * R) / G;             // least and greatest row of the tile
        const int last_low = a.window > 0 ? p0 + (min(rt * R + R, rows) - 1) / G - a.window + 1 : 0;

        float O[NG * 8][4];
        float B[NG][RT], m[RT], l[RT];
        float vs = 1.f, top_ps = 0.f;                        // unit not chosen yet: any p s is above it
#pragma unroll
        for (int j = 0; j < NG * 8; j++)
#pragma unroll
            for (int k = 0; k < 4; k++) O[j][k] = 0.f;
#pragma unroll
        for (int z = 0; z < RT; z++) {
            m[z] = -INFINITY;
            l[z] = 0.f;
#pragma unroll
            for (int g = 0; g < NG; g++) B[g][z] = 0.f;
        }

        // stage k of this warp holds its 16 entries of page pg0 + par + 2 k
        unsigned ok = 0;                                     // bit: the stage's page is usable
        const int32_t* trow = c.table + (size_t)s * cap_pages;
        const auto fetch = [&](int pg, int st) {
            ok &= ~(1u << st);
            if (pg < pg1 && pg < pend) {
                const int id = trow[pg];
                if ((unsigned)id < (unsigned)c.n_pages) {
                    ok |= 1u << st;
                    const uint8_t* src = c.pages + ((size_t)id * c.hkv + h) * (size_t)(4608 * NG);
                    const uint32_t dst = ring + st * Sh::kBlock;
                    const int e = lane >> 1;                 // V rows: entries 2t, 2t + 1, 8 more as rows t, 4 + t
                    const int vr = (e & 8) + ((e & 1) << 2) + ((e & 7) >> 1);
#pragma unroll
                    for (int g = 0; g < NG; g++) {
                        cp_async16(dst + g * 512 + lane * 16, src + g * 2048 + sub * 512 + lane * 16);
                        cp_async16(dst + 576 * NG + g * 512 + vr * 32 + (lane & 1) * 16,
                                   src + 2304 * NG + g * 2048 + sub * 512 + lane * 16);
                    }
                    if (lane < 8 * NG) {
                        const int v = lane / (4 * NG), k = lane % (4 * NG);
                        cp_async16(dst + v * 576 * NG + 512 * NG + k * 16,
                                   src + v * 2304 * NG + 2048 * NG + (k >> 2) * 256 + sub * 64 + (k & 3) * 16);
                    }
                } else if (lane == 0) {
                    kv_flag(c.status);
                }
            }
            cp_async_commit();
        };
#pragma unroll
        for (int st = 0; st < kSplitStages - 1; st++) fetch(pg0 + par + 2 * st, st);

        int st = 0;
        for (int pg = pg0 + par; pg < pg1; pg += 2) {
            fetch(pg + 2 * (kSplitStages - 1), (st + kSplitStages - 1) % kSplitStages);
            cp_async_wait<kSplitStages - 1>();
            __syncwarp();
            const uint32_t kb = ring + st * Sh::kBlock, vb = kb + 576 * NG;
            const bool page_ok = (ok >> st) & 1u;
            st = (st + 1) % kSplitStages;
            const int j0 = pg * kKvPage + sub * 16;
            if (!page_ok || j0 >= q.len) continue;           // nothing here (all lanes alike)

            float S[2][2 * RT];
#pragma unroll
            for (int nt = 0; nt < 2; nt++) {
#pragma unroll
                for (int k = 0; k < 2 * RT; k++) S[nt][k] = 0.f;
#pragma unroll
                for (int g = 0; g < NG; g++) {
                    const uint2 kw = lds64(kb + g * 512 + (8 * nt + g8) * 32 + t4 * 8);
                    float d[4] = {0.f, 0.f, 0.f, 0.f};
                    const uint32_t z0 = 0;
                    mma_f16(d, qa[g][0][0], RT == 2 ? qa[g][0][RT - 1] : z0, qa[g][0][RT], RT == 2 ? qa[g][0][2 * RT - 1] : z0,
                            code_pair<0>(kw.x), code_pair<0>(kw.y));
                    mma_f16(d, qa[g][1][0], RT == 2 ? qa[g][1][RT - 1] : z0, qa[g][1][RT], RT == 2 ? qa[g][1][2 * RT - 1] : z0,
                            code_pair<1>(kw.x), code_pair<1>(kw.y));
                    mma_f16(d, qa[g][2][0], RT == 2 ? qa[g][2][RT - 1] : z0, qa[g][2][RT], RT == 2 ? qa[g][2][2 * RT - 1] : z0,
                            code_pair<2>(kw.x), code_pair<2>(kw.y));
                    mma_f16(d, qa[g][3][0], RT == 2 ? qa[g][3][RT - 1] : z0, qa[g][3][RT], RT == 2 ? qa[g][3][2 * RT - 1] : z0,
                            code_pair<3>(kw.x), code_pair<3>(kw.y));
                    const uint2 sb = lds64(kb + 512 * NG + g * 64 + (8 * nt + 2 * t4) * 4);
                    const float2 f0 = h2f(sb.x), f1 = h2f(sb.y);
                    const float o0 = fmaf(-kCodeOff, f0.x, f0.y), o1 = fmaf(-kCodeOff, f1.x, f1.y);
#pragma unroll
                    for (int z = 0; z < RT; z++) {
                        S[nt][2 * z] = fmaf(f0.x, d[2 * z], fmaf(o0, qs[g][z], S[nt][2 * z]));
                        S[nt][2 * z + 1] = fmaf(f1.x, d[2 * z + 1], fmaf(o1, qs[g][z], S[nt][2 * z + 1]));
                    }
                }
            }
            // entries of this lane: j0 + 2 t4, + 1, + 8, + 9
            const bool edge = j0 + 15 > first_pos || j0 < last_low;
            unsigned vis[RT];
            float p[RT][4];
            bool grow = false;
            float top[RT];
#pragma unroll
            for (int z = 0; z < RT; z++) {
                vis[z] = 0xFu;
                float* pz = p[z];
                pz[0] = S[0][2 * z] * sl2;
                pz[1] = S[0][2 * z + 1] * sl2;
                pz[2] = S[1][2 * z] * sl2;
                pz[3] = S[1][2 * z + 1] * sl2;
                if (edge) {
                    vis[z] = 0;
#pragma unroll
                    for (int k = 0; k < 4; k++) {
                        const int j = j0 + 2 * t4 + (k & 1) + 8 * (k >> 1);
                        if (j <= pos[z] && j >= low[z]) vis[z] |= 1u << k;
                        else pz[k] = -INFINITY;
                    }
                }
                top[z] = fmaxf(fmaxf(pz[0], pz[1]), fmaxf(pz[2], pz[3]));
                top[z] = fmaxf(top[z], __shfl_xor_sync(0xffffffffu, top[z], 1));
                top[z] = fmaxf(top[z], __shfl_xor_sync(0xffffffffu, top[z], 2));
                grow = grow || top[z] > m[z] + 8.f;
            }
            if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
                for (int z = 0; z < RT; z++) {
                    const float m2 = fmaxf(m[z], top[z]);
                    const float f = m2 == -INFINITY ? 1.f : exp2_fast(m[z] - m2);
                    m[z] = m2;
                    l[z] *= f;
#pragma unroll
                    for (int g = 0; g < NG; g++) B[g][z] *= f;
#pragma unroll
                    for (int j = 0; j < NG * 8; j++) {
                        O[j][2 * z] *= f;
                        O[j][2 * z + 1] *= f;
                        if (RT == 1) {
                            O[j][2] *= f;
                            O[j][3] *= f;
                        }
                    }
                }
            }
#pragma unroll
            for (int z = 0; z < RT; z++) {
                const float ref = m[z] == -INFINITY ? 0.f : m[z];
#pragma unroll
                for (int k = 0; k < 4; k++) p[z][k] = exp2_fast(p[z][k] - ref);
                l[z] += (p[z][0] + p[z][1]) + (p[z][2] + p[z][3]);
            }
            // the weighted sum, one group of 64 columns at a time
#pragma unroll
            for (int g = 0; g < NG; g++) {
                const uint2 sb0 = lds64(vb + 512 * NG + g * 64 + t4 * 8);
                const uint2 sb1 = lds64(vb + 512 * NG + g * 64 + 32 + t4 * 8);
                const float2 f[4] = {h2f(sb0.x), h2f(sb0.y), h2f(sb1.x), h2f(sb1.y)};   // scale, bias
                float e[RT][4];
#pragma unroll
                for (int z = 0; z < RT; z++)
#pragma unroll
                    for (int k = 0; k < 4; k++)
                        e[z][k] = !edge || ((vis[z] >> k) & 1u) ? p[z][k] * f[k].x : 0.f;
                uint32_t hi[RT][2], lo[RT][2];
                float big = 0.f;
#pragma unroll
                for (int z = 0; z < RT; z++)
#pragma unroll
                    for (int k = 0; k < 4; k++) big = fmaxf(big, fabsf(e[z][k]));
                if (__any_sync(0xffffffffu, big > top_ps)) {
                    // above fp16's range in the present unit (or the first entries): the unit
                    // becomes the power of two that brings the largest p s to 16..32
#pragma unroll
                    for (int o = 1; o < 32; o <<= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, o));
                    if (big < 1e30f) {                       // an infinite scale: nothing finite to keep
                        const float v2 = exp2f(fminf(4.f - floorf(log2f(big)), 100.f));
                        const float k = top_ps == 0.f ? 1.f : v2 / vs;
                        vs = v2;
                        top_ps = 16384.f / v2;
#pragma unroll
                        for (int z = 0; z < RT; z++)
#pragma unroll
                            for (int gg = 0; gg < NG; gg++) B[gg][z] *= k;
#pragma unroll
                        for (int j = 0; j < NG * 8; j++)
#pragma unroll
                            for (int w = 0; w < 4; w++) O[j][w] *= k;
                    }
                }
#pragma unroll
                for (int z = 0; z < RT; z++) {
#pragma unroll
                    for (int k = 0; k < 4; k++) {
                        e[z][k] *= vs;
                        if (!edge || ((vis[z] >> k) & 1u))
                            B[g][z] = fmaf(p[z][k] * vs, fmaf(-kCodeOff, f[k].x, f[k].y), B[g][z]);
                    }
#pragma unroll
                    for (int k = 0; k < 2; k++) {
                        hi[z][k] = f2h(e[z][2 * k], e[z][2 * k + 1]);
                        const float2 r = h2f(hi[z][k]);
                        lo[z][k] = f2h(e[z][2 * k] - r.x, e[z][2 * k + 1] - r.y);
                    }
                }
                const uint32_t va = vb + g * 512 + t4 * 32 + g8 * 4;
                const uint32_t w0 = lds32(va), w1 = lds32(va + 128), w2 = lds32(va + 256), w3 = lds32(va + 384);
#pragma unroll
                for (int k = 0; k < 2; k++) {
                    const uint32_t c0 = __byte_perm(w0, w1, k ? 0x7632 : 0x5410);
                    const uint32_t c1 = __byte_perm(w2, w3, k ? 0x7632 : 0x5410);
                    const uint32_t e0[4] = {code_pair<0>(c0), code_pair<1>(c0), code_pair<2>(c0), code_pair<3>(c0)};
                    const uint32_t e1[4] = {code_pair<0>(c1), code_pair<1>(c1), code_pair<2>(c1), code_pair<3>(c1)};
#pragma unroll
                    for (int j = 0; j < 4; j++) {
                        float(&o)[4] = O[g * 8 + k * 4 + j];
                        if (RT == 1) {
                            mma_f16(o, hi[0][0], lo[0][0], hi[0][1], lo[0][1], e0[j], e1[j]);
                        } else {
                            mma_f16(o, hi[0][0], hi[RT - 1][0], hi[0][1], hi[RT - 1][1], e0[j], e1[j]);
                            mma_f16(o, lo[0][0], lo[RT - 1][0], lo[0][1], lo[RT - 1][1], e0[j], e1[j]);
                        }
                    }
                }
            }
            __syncwarp();
        }
        cp_async_wait<0>();

        // join the warps: sums to shared memory (over the ring), relative to each warp's maximum
        const float inv = 1.f / vs;                          // a power of two
#pragma unroll
        for (int z = 0; z < RT; z++) {
            l[z] += __shfl_xor_sync(0xffffffffu, l[z], 1);
            l[z] += __shfl_xor_sync(0xffffffffu, l[z], 2);
#pragma unroll
            for (int g = 0; g < NG; g++) {
                B[g][z] += __shfl_xor_sync(0xffffffffu, B[g][z], 1);
                B[g][z] += __shfl_xor_sync(0xffffffffu, B[g][z], 2);
            }
            if (t4 == 0) {
                s_m[warp][g8 + 8 * z] = m[z];
                s_l[warp][g8 + 8 * z] = l[z];
            }
        }
        __syncthreads();                                     // every warp has left its ring
        float* join = reinterpret_cast<float*>(sp_smem);
#pragma unroll
        for (int z = 0; z < RT; z++)
#pragma unroll
            for (int g = 0; g < NG; g++) {
                float* dst = join + ((size_t)warp * R + g8 + 8 * z) * D + g * 64 + t4 * 16;
#pragma unroll
                for (int j = 0; j < 8; j++) {
                    const float(&o)[4] = O[g * 8 + j];
                    dst[j] = ((RT == 1 ? o[0] + o[2] : o[2 * z]) + B[g][z]) * inv;
                    dst[8 + j] = ((RT == 1 ? o[1] + o[3] : o[2 * z + 1]) + B[g][z]) * inv;
                }
            }
        __syncthreads();
        const bool whole = u == ie && ib >= blockIdx.x * per;
        const int c0 = (int)(ib / per), c1 = (int)((ie - 1) / per);
        float* slot = x.part + (size_t)(2 * blockIdx.x + (c0 == (int)blockIdx.x ? 1 : 0)) * (R * (D + 2));
        const auto store_row = [&](int r, int d, const float (&o)[8], float M, float L) {
            const int i = r / G, head = h * G + r % G;
            const float f = L == 0.f ? 0.f : 1.f / L;
            uint4 v;
            v.x = f2h(o[0] * f, o[1] * f);
            v.y = f2h(o[2] * f, o[3] * f);
            v.z = f2h(o[4] * f, o[5] * f);
            v.w = f2h(o[6] * f, o[7] * f);
            *reinterpret_cast<uint4*>(a.out + (size_t)(q.first + i) * a.out_stride + (size_t)head * D + d) = v;
            if (d == 0) a.lse[(size_t)(q.first + i) * c.hq + head] = L == 0.f ? -INFINITY : (M + log2f(L)) * kLn2;
        };
        for (int k = tid; k < R * (D / 8); k += kSplitThreads) {
            const int r = k / (D / 8), d = (k % (D / 8)) * 8;
            if (rt * R + r >= rows) continue;
            float M = -INFINITY, L = 0.f, o[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int w = 0; w < kSplitWarps; w++) M = fmaxf(M, s_m[w][r]);
            const float ref = M == -INFINITY ? 0.f : M;
#pragma unroll
            for (int w = 0; w < kSplitWarps; w++) {
                if (s_m[w][r] == -INFINITY && s_l[w][r] == 0.f) continue;
                const float f = exp2_fast(s_m[w][r] - ref);
                const float4* src = reinterpret_cast<const float4*>(join + ((size_t)w * R + r) * D + d);
                const float4 v0 = src[0], v1 = src[1];
                L = fmaf(f, s_l[w][r], L);
                o[0] = fmaf(f, v0.x, o[0]); o[1] = fmaf(f, v0.y, o[1]);
                o[2] = fmaf(f, v0.z, o[2]); o[3] = fmaf(f, v0.w, o[3]);
                o[4] = fmaf(f, v1.x, o[4]); o[5] = fmaf(f, v1.y, o[5]);
                o[6] = fmaf(f, v1.z, o[6]); o[7] = fmaf(f, v1.w, o[7]);
            }
            if (whole) {
                store_row(rt * R + r, d, o, M, L);
            } else {
                float4* dst = reinterpret_cast<float4*>(slot + (size_t)r * D + d);
                dst[0] = make_float4(o[0], o[1], o[2], o[3]);
                dst[1] = make_float4(o[4], o[5], o[6], o[7]);
                if (d == 0) {
                    slot[R * D + r] = M;
                    slot[R * D + R + r] = L;
                }
            }
        }
        if (!whole) {
            __threadfence();
            __syncthreads();
            if (tid == 0) s_last = atomicAdd(x.count + c0, 1) == c1 - c0;
            __syncthreads();
            if (s_last) {
                __threadfence();
                for (int k = tid; k < R * (D / 8); k += kSplitThreads) {
                    const int r = k / (D / 8), d = (k % (D / 8)) * 8;
                    if (rt * R + r >= rows) continue;
                    float M = -INFINITY, L = 0.f, o[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
                    const auto at = [&](int b) { return x.part + (size_t)(2 * b + (b == c0 ? 1 : 0)) * (R * (D + 2)); };
                    for (int b = c0; b <= c1; b++) M = fmaxf(M, __ldcg(at(b) + R * D + r));
                    const float ref = M == -INFINITY ? 0.f : M;
#pragma unroll 4
                    for (int b = c0; b <= c1; b++) {
                        const float* src = at(b);
                        const float mb = __ldcg(src + R * D + r), lb = __ldcg(src + R * D + R + r);
                        const float4 v0 = __ldcg(reinterpret_cast<const float4*>(src + (size_t)r * D + d));
                        const float4 v1 = __ldcg(reinterpret_cast<const float4*>(src + (size_t)r * D + d) + 1);
                        const bool none = mb == -INFINITY && lb == 0.f;
                        const float f = none ? 0.f : exp2_fast(mb - ref);
                        L = fmaf(f, lb, L);
                        o[0] = fmaf(f, v0.x, o[0]); o[1] = fmaf(f, v0.y, o[1]);
                        o[2] = fmaf(f, v0.z, o[2]); o[3] = fmaf(f, v0.w, o[3]);
                        o[4] = fmaf(f, v1.x, o[4]); o[5] = fmaf(f, v1.y, o[5]);
                        o[6] = fmaf(f, v1.z, o[6]); o[7] = fmaf(f, v1.w, o[7]);
                    }
                    store_row(rt * R + r, d, o, M, L);
                }
                if (tid == 0) x.count[c0] = 0;
            }
        }
        __syncthreads();                                     // the ring and s_m are free again
    }
}

// One element of K (part 0) or V (part 1).
__device__ __forceinline__ float kv_value(const uint8_t* tile, const KvTile& t, int part, int e, int d) {
    const int g = d >> 6, c = d & 63;
    const uint32_t w = *reinterpret_cast<const uint32_t*>(tile + t.codes(part, g, e) + (c >> 3) * 4);
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(tile + t.sb(part, g, e)));
    return fmaf(f.x, (float)((w >> (4 * (c & 7))) & 15u), f.y);
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
