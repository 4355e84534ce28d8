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

// Scores and running sums are in units of log2: exp(S) = exp2(S log2 e).
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float exp2_fast(float x) {       // 2^x, 2 ulp; 0 for x = -inf
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// D = C + A B on 16 x 8 fp32 (A 16 x 16, B 16 x 8, fp16); lane = 4 g + t holds
// A rows g (a0, a2) and g + 8 (a1, a3), columns 2t, 2t + 1 (a0, a1) and 8 more
// (a2, a3); B column g, rows alike; C and D rows g (0, 1) and g + 8 (2, 3),
// columns 2t, 2t + 1.
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1, float c0, float c1, float c2, float c3) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%10, %11, %12, %13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
}
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1) {
    mma_f16(d, a0, a1, a2, a3, b0, b1, d[0], d[1], d[2], d[3]);
}

// Nibbles i and i + 4 of w as a pair of fp16 operands, i = 0..3.  fp16's
// subnormals and first binade are linear in their bits, so a code in bits 0..3 is
// the number code * 2^-24 as it stands and one in bits 4..7 is 16 times that: a
// mask makes an operand, exactly, with no exponent to set and no offset to take
// out again.  The factors 2^24 and 16 leave through the query operand.
__device__ __forceinline__ void code_pairs(uint32_t w, uint32_t (&o)[4]) {
    const uint32_t u = w >> 8;
    o[0] = w & 0x000F000Fu;
    o[1] = w & 0x00F000F0u;
    o[2] = u & 0x000F000Fu;
    o[3] = u & 0x00F000F0u;
}
constexpr float kCodeUnit = 16777216.f;       // 2^24: operands of even pairs are code / 2^24, of odd ones 16 times it

__device__ __forceinline__ float2 h2f(uint32_t v) { return __half22float2(*reinterpret_cast<const __half2*>(&v)); }
__device__ __forceinline__ uint32_t f2h(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n\t.reg .b64 x, y, z;\n\t"
        "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
        "fma.rn.f32x2 x, x, y, z;\n\tmov.b64 {%0, %1}, x;\n\t}\n"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 x, y;\n\t"
        "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
        "add.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}\n"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}

// floor(log2 x) of a positive normal x, and 2^e for -126 <= e <= 127.
__device__ __forceinline__ int exponent_of(float x) { return (int)(__float_as_uint(x) >> 23) - 127; }
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// log sum exp of a row with total L = sum 2^(S - M).  The running maxima are whole
// numbers (the next to the true one), so that they and the powers of two in the
// totals add up exactly and only log2 of 1 <= L < 2 is rounded (with fractions left
// in M and a large L the sum of the two cost lse 5e-7).
__device__ __forceinline__ float lse_of(float M, float L) {
    if (L == 0.f) return -INFINITY;
    const int e = exponent_of(L);
    return (M + (float)e + log2f(L * pow2(-e))) * kLn2;
}

// The same pairs as fp16 c - 8.
__device__ __forceinline__ uint4 codes_centred(uint32_t w) {
    const uint32_t u = w >> 8;
    const uint32_t v[4] = {(w & 0x000F000Fu) | 0x64006400u, (w & 0x00F000F0u) | 0x54005400u,
                           (u & 0x000F000Fu) | 0x64006400u, (u & 0x00F000F0u) | 0x54005400u};
    const __half2 o0 = __float2half2_rn(-1032.f), o1 = __float2half2_rn(-72.f);   // -(1024 + 8), -(64 + 8)
    uint32_t r[4];
#pragma unroll
    for (int k = 0; k < 4; k++) {
        const __half2 h = __hadd2(*reinterpret_cast<const __half2*>(&v[k]), k & 1 ? o1 : o0);
        r[k] = *reinterpret_cast<const uint32_t*>(&h);
    }
    return make_uint4(r[0], r[1], r[2], r[3]);
}

// And as fp16 c.
__device__ __forceinline__ void codes_exact(uint32_t w, uint32_t (&o)[4]) {
    const uint32_t u = w >> 8;
    const uint32_t v[4] = {(w & 0x000F000Fu) | 0x64006400u, (w & 0x00F000F0u) | 0x54005400u,
                           (u & 0x000F000Fu) | 0x64006400u, (u & 0x00F000F0u) | 0x54005400u};
    const __half2 o0 = __float2half2_rn(-1024.f), o1 = __float2half2_rn(-64.f);
#pragma unroll
    for (int k = 0; k < 4; k++) {
        const __half2 h = __hadd2(*reinterpret_cast<const __half2*>(&v[k]), k & 1 ? o1 : o0);
        o[k] = *reinterpret_cast<const uint32_t*>(&h);
    }
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
// Few rows per kv head (single tokens): every byte of the cache is read once per 8
// or 16 rows by one warp and used from registers.
//
// An item is (sequence, tile of 8 RT rows, kv head); its rows are the
// (row, query head) pairs that read the kv head, so a group's query heads share
// each entry.  The pages of all items form one list of units; CTA c takes units
// [c per, (c + 1) per), whatever items they belong to, so ragged batches are
// even; an item counts kSplitItemCost pages more than it has, for its start and
// end.  Four warps: two take the halves of every second page of a segment, each
// through its own ring of cp.async stages with no barrier between warps.  Per 32
// entries a warp forms
//   S = sum_g s_g (q_g . c_g) + b_g sum(q_g)
// with tensor-core products of the raw codes (m16n8k16: rows = query rows,
// columns = entries; q is taken times a power of two per row that brings its
// largest to 1024..2048, so that 16 q, for the even pairs, stays exact), keeps a
// running maximum (moved only when it grows by more than 2^8, so the sums are
// rescaled rarely) and adds
//   O += sum_j p_j s_jg (c_j - 8),   B_g += sum_j p_j (b_jg + 8 s_jg).
// Codes of V are centred: raw ones (0..15) would let O grow to many times the
// result, and the tensor cores' accumulation, which cuts off, would cost 8e-4 of it
// over 131,072 entries.  These products are taken transposed (rows = columns of V,
// columns = query rows): the scores' registers are then the second operand as they
// stand, and 8 query rows fill a tile.  p s enters as one fp16 value (a relative
// 2^-12 per entry on average; a second one for the remainder made the kernel 8 %
// slower), kept in fp16's range by a power of two per warp (unit) that is chosen at
// the first entries and lowered when a later p s would leave the range, so that p s is
// held to 2^-29 of the largest that the warp's rows have met; it is part
// of the exponent that p is formed with.  The warps' sums meet in shared memory; an
// item cut by CTA borders goes through partial sums in the workspace, joined in a
// fixed order by the last CTA to arrive (one counter per item start, reset by that
// CTA).
//
// What bounds it is instruction issue and latency, about 690 instructions per 32
// entries of 128 columns and three warps a scheduler (54 % of the issue slots): 64
// tokens with up to 16,384 entries take 162 to 169 us, as their lengths fall (3.6 TB/s of
// the cache, 0.56 of the copy rate), one with 131,072 50 us (3.0 TB/s, the start and the join of the parts
// included; the loop alone streams 4.6 TB/s).
constexpr int kSplitWarps = 4;
constexpr int kSplitThreads = kSplitWarps * 32;
// Ring stages.  64 tokens with a window of 1024 (heads of 256): 3 stages, which leave
// room for one CTA per SM, 100 us, 2 stages and two CTAs 83.  64 tokens of up to 16,384
// entries (heads of 128): 3 stages and two CTAs 171 us, 2 and three 169, 4 CTAs of 128
// registers 5 % more.
constexpr int kSplitStages = 2;
// An item's start and end in pages.  64 tokens with up to 16,384 entries: 0 184 us, 2
// to 8 alike (169).
constexpr int kSplitItemCost = 4;
// (row, head) pairs per kv head of a sequence; with more the tile kernel takes over.
// This kernel reads the cache anew for every 16 of them, that one computes 128 whatever
// there are: 16 sequences of up to 4,096 entries, heads of 128, here and there: 16 pairs
// 36 and 97 us, 32 53 and 97, 64 84 and 99, 80 99 and 103; heads of 64, 64 pairs: 51 and
// 79; of 256: 65 and 70.  (Over a few hundred entries of one sequence the tile kernel
// would win from 32 on, 15 us against 18.)
constexpr int kSplitMaxRows = 64;

template <int NG, int RT>
struct SplitShape {
    static constexpr int kRows = 8 * RT;
    static constexpr int kD = 64 * NG;
    static constexpr int kHalf = 2304 * NG;                          // 32 entries: K and V, codes and s, b
    static constexpr int kRing = kSplitWarps * kSplitStages * kHalf;
    static constexpr int kJoinRow = kD + 4;                          // floats; 4 more against bank conflicts
    static constexpr int kJoin = kSplitWarps * kRows * kJoinRow * 4; // the warps' sums, over the ring
    static constexpr int kQ = NG * 4 * 32 * 16;                      // query operand, 16 rows (zeros behind 8)
    static constexpr int kSmem = (kRing > kJoin ? kRing : kJoin) + kQ;
    // CTAs per SM that the registers are bounded for; as many fit, but for <4, 1>, where
    // 82 KB of shared memory a CTA let two in
    static constexpr int kCtas = NG * RT <= 4 ? 3 : 2;
};

struct SplitArgs {
    AttnArgs a;
    float* part;               // [2 gridDim.x][kRows][D + 2]: sums, maximum, total
    int* count;                // [gridDim.x], zero between calls
    int max_rows_seq;          // sequences with more (row, head) pairs per kv head are not served here
};

// What one sequence asks of the split kernel.
struct SplitSeq {
    int n, first, len, plo, np, tiles, units;     // np pages an item
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
    q.units = q.tiles * c.hkv * (q.np + kSplitItemCost);
    return q;
}

// A warp's running sums of one segment.  Lane (g, t) holds, of group gg and rows
// 8 z + 2t (even k) and 8 z + 2t + 1 (odd k), columns 8 g + jj (k < 2) and
// 8 g + 4 + jj in O[z][4 gg + jj][k]; B, m and l belong to row 8 z + g.
template <int NG, int RT>
struct SplitAcc {
    float O[RT][NG * 4][4];
    float B[NG][RT], m[RT], l[RT];
    float unit;                // all sums are taken times 2^unit
    bool chosen;
};

// The value that row 2t (k = 0) or 2t + 1 (k = 1) of a warp has, from row g's.
__device__ __forceinline__ float row_value(float v, int k) {
    return __shfl_sync(0xffffffffu, v, 8 * (threadIdx.x & 3) + 4 * k);
}

// 32 entries (kb: their K block, V block behind it) from entry j0 on.  EDGE:
// some row does not see some of them.
template <int NG, int RT, bool EDGE>
__device__ __forceinline__ void split_block(SplitAcc<NG, RT>& A, uint32_t kb, uint32_t qb, const float (&qs)[NG][RT],
                                            const float (&sl2)[RT], int j0, const int (&pos)[RT], const int (&low)[RT]) {
    const int lane = threadIdx.x & 31, g8 = lane >> 2, t4 = lane & 3;
    const uint32_t vb = kb + 1152 * NG;
    float p[RT][8];
#pragma unroll
    for (int z = 0; z < RT; z++)
#pragma unroll
        for (int k = 0; k < 8; k++) p[z][k] = 0.f;
#pragma unroll
    for (int g = 0; g < NG; g++) {
        uint32_t qa[4][4];
#pragma unroll
        for (int mm = 0; mm < 4; mm++) {
            const uint4 v = lds128(qb + ((g * 4 + mm) * 32 + lane) * 16);
            qa[mm][0] = v.x; qa[mm][1] = v.y; qa[mm][2] = v.z; qa[mm][3] = v.w;
        }
#pragma unroll
        for (int nt = 0; nt < 4; nt++) {
            const uint2 kw = lds64(kb + g * 1024 + (8 * nt + g8) * 32 + t4 * 8);
            uint32_t b0[4], b1[4];
            code_pairs(kw.x, b0);
            code_pairs(kw.y, b1);
            float d[4];
            mma_f16(d, qa[0][0], qa[0][1], qa[0][2], qa[0][3], b0[0], b1[0], 0.f, 0.f, 0.f, 0.f);
            mma_f16(d, qa[1][0], qa[1][1], qa[1][2], qa[1][3], b0[1], b1[1]);
            mma_f16(d, qa[2][0], qa[2][1], qa[2][2], qa[2][3], b0[2], b1[2]);
            mma_f16(d, qa[3][0], qa[3][1], qa[3][2], qa[3][3], b0[3], b1[3]);
            const uint2 sb = lds64(kb + 1024 * NG + g * 128 + (8 * nt + 2 * t4) * 4);
            const float2 f0 = h2f(sb.x), f1 = h2f(sb.y);
#pragma unroll
            for (int z = 0; z < RT; z++) {
                p[z][2 * nt] = fmaf(f0.x, d[2 * z], fmaf(f0.y, qs[g][z], p[z][2 * nt]));
                p[z][2 * nt + 1] = fmaf(f1.x, d[2 * z + 1], fmaf(f1.y, qs[g][z], p[z][2 * nt + 1]));
            }
        }
    }
    // this lane's entries: j0 + 8 (k / 2) + 2 t4 + k % 2
    unsigned vis[RT];
    bool grow = false;
    float top[RT];
#pragma unroll
    for (int z = 0; z < RT; z++) {
        vis[z] = 0xFFu;
#pragma unroll
        for (int k = 0; EDGE && k < 8; k++) {
            const int j = j0 + 8 * (k >> 1) + 2 * t4 + (k & 1);
            if (j > pos[z] || j < low[z]) {
                vis[z] &= ~(1u << k);
                p[z][k] = -INFINITY;
            }
        }
        top[z] = fmaxf(fmaxf(fmaxf(p[z][0], p[z][1]), fmaxf(p[z][2], p[z][3])),
                       fmaxf(fmaxf(p[z][4], p[z][5]), fmaxf(p[z][6], p[z][7])));
        top[z] = fmaxf(top[z], __shfl_xor_sync(0xffffffffu, top[z], 1));
        top[z] = fmaxf(top[z], __shfl_xor_sync(0xffffffffu, top[z], 2));
        top[z] *= sl2[z];                                    // sl2 > 0
        grow = grow || top[z] > A.m[z] + 8.f;
    }
    if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
        for (int z = 0; z < RT; z++) {
            const float m2 = rintf(fmaxf(A.m[z], top[z]));
            const float f = m2 == -INFINITY ? 1.f : exp2_fast(A.m[z] - m2);
            A.m[z] = m2;
            A.l[z] *= f;
            const float f0 = row_value(f, 0), f1 = row_value(f, 1);
#pragma unroll
            for (int g = 0; g < NG; g++) A.B[g][z] *= f;
#pragma unroll
            for (int j = 0; j < NG * 4; j++) {
                A.O[z][j][0] *= f0;
                A.O[z][j][1] *= f1;
                A.O[z][j][2] *= f0;
                A.O[z][j][3] *= f1;
            }
        }
    }
#pragma unroll
    for (int z = 0; z < RT; z++) {
        const float ref = A.m[z] == -INFINITY ? 0.f : A.m[z] - A.unit;
#pragma unroll
        for (int k = 0; k < 8; k++) p[z][k] = exp2_fast(fmaf(p[z][k], sl2[z], -ref));
        A.l[z] += ((p[z][0] + p[z][1]) + (p[z][2] + p[z][3])) + ((p[z][4] + p[z][5]) + (p[z][6] + p[z][7]));
    }
    // the weighted sum, 16 entries at a time
#pragma unroll
    for (int b = 0; b < 2; b++) {
        uint32_t sb[NG][4], hi[NG][RT][2];
#pragma unroll
        for (int g = 0; g < NG; g++) {
            const uint2 s0 = lds64(vb + 1024 * NG + g * 128 + b * 64 + t4 * 8);
            const uint2 s1 = lds64(vb + 1024 * NG + g * 128 + b * 64 + 32 + t4 * 8);
            sb[g][0] = s0.x; sb[g][1] = s0.y; sb[g][2] = s1.x; sb[g][3] = s1.y;
        }
        const auto seen = [&](int z, int k) { return !EDGE || ((vis[z] >> (4 * b + k)) & 1u); };
        // p s of every group, and whether all of them fit (up to 2^15)
        const auto parts = [&]() {
            __half2 big = __float2half2_rn(0.f);
#pragma unroll
            for (int g = 0; g < NG; g++)
#pragma unroll
                for (int z = 0; z < RT; z++)
#pragma unroll
                    for (int k = 0; k < 2; k++) {
                        const float2 f0 = h2f(sb[g][2 * k]), f1 = h2f(sb[g][2 * k + 1]);
                        // an entry out of sight may hold a NaN scale
                        const float e0 = seen(z, 2 * k) ? p[z][4 * b + 2 * k] * f0.x : 0.f;
                        const float e1 = seen(z, 2 * k + 1) ? p[z][4 * b + 2 * k + 1] * f1.x : 0.f;
                        hi[g][z][k] = f2h(e0, e1);
                        big = __hmax2(big, __habs2(*reinterpret_cast<const __half2*>(&hi[g][z][k])));
                    }
            return fmaxf(__low2float(big), __high2float(big)) <= 32768.f;
        };
        const bool fits = parts();
        if (__any_sync(0xffffffffu, !fits || !A.chosen)) {
            // the unit becomes the one that brings the largest finite p s to 16..32 (an infinite
            // one belongs to the rows that see it, and must not keep the others' in fp16's way)
            float mx = 0.f;
#pragma unroll
            for (int g = 0; g < NG; g++)
#pragma unroll
                for (int z = 0; z < RT; z++)
#pragma unroll
                    for (int k = 0; k < 4; k++) {
                        const float v = p[z][4 * b + k] * h2f(sb[g][k]).x;
                        if (seen(z, k)) mx = fmaxf(mx, fabsf(fmaf(v, 0.f, v)));  // v, or NaN, which fmaxf passes over
                    }
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            if (mx > 0.f) {                              // else nothing here, or nothing finite to keep
                const float du = fmaxf(fminf(4.f - floorf(log2f(mx)), 60.f - A.unit), -60.f - A.unit);
                const float f = exp2f(du);
                A.unit += du;
                A.chosen = true;
#pragma unroll
                for (int z = 0; z < RT; z++) {
                    A.l[z] *= f;
#pragma unroll
                    for (int g = 0; g < NG; g++) A.B[g][z] *= f;
#pragma unroll
                    for (int k = 0; k < 8; k++) p[z][k] *= f;
#pragma unroll
                    for (int j = 0; j < NG * 4; j++)
#pragma unroll
                        for (int k = 0; k < 4; k++) A.O[z][j][k] *= f;
                }
                parts();
            }
        }
#pragma unroll
        for (int g = 0; g < NG; g++) {
#pragma unroll
            for (int k = 0; k < 4; k++) {
                const float2 f = h2f(sb[g][k]);
                const float mid = fmaf(8.f, f.x, f.y);
#pragma unroll
                for (int z = 0; z < RT; z++)
                    if (seen(z, k)) A.B[g][z] = fmaf(p[z][4 * b + k], mid, A.B[g][z]);
            }
            const uint32_t va = vb + g * 1024 + b * 512 + t4 * 32 + g8 * 4;
            const uint32_t w0 = lds32(va), w1 = lds32(va + 128), w2 = lds32(va + 256), w3 = lds32(va + 384);
            const uint4 a0 = codes_centred(__byte_perm(w0, w1, 0x5410)), a1 = codes_centred(__byte_perm(w0, w1, 0x7632));
            const uint4 a2 = codes_centred(__byte_perm(w2, w3, 0x5410)), a3 = codes_centred(__byte_perm(w2, w3, 0x7632));
#pragma unroll
            for (int z = 0; z < RT; z++) {
                float(*o)[4] = &A.O[z][g * 4];
                mma_f16(o[0], a0.x, a1.x, a2.x, a3.x, hi[g][z][0], hi[g][z][1]);
                mma_f16(o[1], a0.y, a1.y, a2.y, a3.y, hi[g][z][0], hi[g][z][1]);
                mma_f16(o[2], a0.z, a1.z, a2.z, a3.z, hi[g][z][0], hi[g][z][1]);
                mma_f16(o[3], a0.w, a1.w, a2.w, a3.w, hi[g][z][0], hi[g][z][1]);
            }
        }
    }
}

template <int NG, int RT>
__global__ void __launch_bounds__(kSplitThreads, SplitShape<NG, RT>::kCtas) k_attn_split(const SplitArgs x) {
    using Sh = SplitShape<NG, RT>;
    constexpr int R = Sh::kRows, D = Sh::kD, JR = Sh::kJoinRow;
    extern __shared__ __align__(128) uint8_t sp_smem[];
    __shared__ float s_m[kSplitWarps][R], s_l[kSplitWarps][R], s_qs[NG][R], s_sl2[R];
    __shared__ long long s_base0, s_total, s_per;
    __shared__ SplitSeq s_q;
    __shared__ int s_seq, s_last;
    const AttnArgs& a = x.a;
    const KvArgs& c = a.c;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g8 = lane >> 2, t4 = lane & 3;
    const int G = c.hq / c.hkv;
    uint8_t* q_smem = sp_smem + Sh::kSmem - Sh::kQ;

    kv_begin();
    // units of all sequences, this CTA's range and the sequence it begins in
    if (warp == 0) {
        long long total = 0;
        SplitSeq q{};
        for (int s0 = 0; s0 < c.n_seqs; s0 += 32) {
            q.units = 0;
            if (s0 + lane < c.n_seqs) q = split_seq<R>(x, s0 + lane, blockIdx.x == 0);
            total += q.units;
        }
        total = warp_sum(total);
        const long long n = total + gridDim.x - 1;
        const long long per = max(n >> 32 ? n / gridDim.x : (long long)((unsigned)n / gridDim.x), 1LL);
        const long long u = blockIdx.x * per;
        long long base = 0;
        if (u < total)
            for (int s0 = 0; s0 < c.n_seqs; s0 += 32) {
                if (c.n_seqs > 32) {                         // else q holds it already
                    q.units = 0;
                    if (s0 + lane < c.n_seqs) q = split_seq<R>(x, s0 + lane, false);
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
    long long u = blockIdx.x * per, s_base = s_base0;
    const long long u_end = min(total, u + per);
    if (u >= u_end) return;
    int s = s_seq;
    SplitSeq q = s_q;

    const uint32_t ring = smem_u32(sp_smem) + warp * (kSplitStages * Sh::kHalf);
    const int half = warp & 1, par = warp >> 1;
    constexpr int kStep = kSplitWarps / 2;                   // pages a round
    // this lane's parts of a fetch: codes of V go to rows in the order that the products
    // want (entries 2t, 2t + 1, 8 + 2t, 9 + 2t as rows t, 4 + t, 8 + t, 12 + t); scales and
    // biases, 16 bytes each
    const size_t page_bytes = (size_t)c.hkv * (4608 * NG);
    const int ve = lane >> 1;
    const uint32_t v_dst = 1152 * NG + ((ve & 8) + ((ve & 1) << 2) + ((ve & 7) >> 1)) * 32 + (lane & 1) * 16;
    uint32_t sb_dst[(NG + 1) / 2];
    int sb_src[(NG + 1) / 2];
#pragma unroll
    for (int k = 0; k < (NG + 1) / 2; k++) {
        const int n = k * 32 + lane, v = n / (8 * NG), i = n % (8 * NG);
        sb_dst[k] = v * 1152 * NG + 1024 * NG + i * 16;
        sb_src[k] = v * 2304 * NG + 2048 * NG + (i >> 3) * 256 + half * 128 + (i & 7) * 16 - half * 1024 - lane * 16;
    }

    while (u < u_end) {
        while (u >= s_base + q.units) {                      // sequences without units are passed over
            if (s + 1 >= c.n_seqs) return;                   // (not reached while what lens says stays)
            s_base += q.units;
            s++;
            q = split_seq<R>(x, s, false);
        }
        const int item = (int)(u - s_base) / (q.np + kSplitItemCost);        // within one sequence: 32 bits
        // the item's pages stand at units ib .. ie - 1, behind its fixed cost
        const long long ib = s_base + (long long)item * (q.np + kSplitItemCost) + kSplitItemCost, ie = ib + q.np;
        u = max(u, ib);
        if (u >= u_end) break;
        const int rt = item / c.hkv, h = item % c.hkv;
        const int pg0 = q.plo + (int)(u - ib);
        const int pend = (q.len + kKvPage - 1) / kKvPage;    // pages that hold entries
        const int pg1 = min(q.plo + (int)(min(u_end, ie) - ib), pend);
        const int p0 = q.len - q.n;
        const int rows = q.n * G;
        u = min(u_end, ie);

        // queries of the tile: threads 4 r + t take 16 columns of each group of row r
        const int qt = tid & 3, qr = tid >> 2;
        uint4 qv[NG][2];
#pragma unroll
        for (int g = 0; g < NG; g++) {
            qv[g][0] = qv[g][1] = make_uint4(0, 0, 0, 0);
            if (qr < R && rt * R + qr < rows) {
                const int rr = rt * R + qr;
                const __half* qp = a.q + (size_t)(q.first + rr / G) * a.q_stride + (size_t)(h * G + rr % G) * D + g * 64 + qt * 16;
                qv[g][0] = *reinterpret_cast<const uint4*>(qp);
                qv[g][1] = *reinterpret_cast<const uint4*>(qp + 8);
            }
        }
        // the stage holds this warp's half of page pg0 + par + kStep k
        unsigned ok = 0;                                     // bit: the stage's page is usable
        const int32_t* trow = c.table + (size_t)s * c.max_pages;
        int id = pg0 + par < pg1 ? trow[pg0 + par] : -1;     // page of the next fetch, read one ahead
        const uint8_t* pool = c.pages + (size_t)h * (4608 * NG) + half * 1024 + lane * 16;
        const auto fetch = [&](int pg, int st) {
            ok &= ~(1u << st);
            if (pg < pg1) {
                if ((unsigned)id < (unsigned)c.n_pages) {
                    ok |= 1u << st;
                    const uint8_t* src = pool + (size_t)id * page_bytes;
                    const uint32_t dst = ring + st * Sh::kHalf;
#pragma unroll
                    for (int g = 0; g < NG; g++)
#pragma unroll
                        for (int b = 0; b < 2; b++) {
                            cp_async16(dst + lane * 16 + g * 1024 + b * 512, src + g * 2048 + b * 512);
                            cp_async16(dst + v_dst + g * 1024 + b * 512, src + 2304 * NG + g * 2048 + b * 512);
                        }
#pragma unroll
                    for (int k = 0; k < (NG + 1) / 2; k++)
                        if (k * 32 + lane < 16 * NG) cp_async16(dst + sb_dst[k], src + sb_src[k]);
                } else if (lane == 0) {
                    kv_flag(c.status);
                }
                if (pg + kStep < pg1) id = trow[pg + kStep];
            }
            cp_async_commit();
        };
#pragma unroll
        for (int st = 0; st < kSplitStages - 1; st++) fetch(pg0 + par + kStep * st, st);

        // into the operand order of code_pairs: per group, 4 steps of 16 columns; lane
        // (g8, t4) holds columns 16 t4 + m (+ 4, + 8, + 12) of rows g8, g8 + 8
        if (tid < R * 4) {
            const int t = qt, r = qr;
            float mx = 0.f;
#pragma unroll
            for (int g = 0; g < NG; g++) {
                const uint32_t w[8] = {qv[g][0].x, qv[g][0].y, qv[g][0].z, qv[g][0].w, qv[g][1].x, qv[g][1].y, qv[g][1].z, qv[g][1].w};
#pragma unroll
                for (int k = 0; k < 8; k++) {
                    const float2 f = h2f(w[k]);
                    mx = fmaxf(mx, fmaxf(fabsf(f.x), fabsf(f.y)));
                }
            }
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
            // the sign of the softmax scale goes into the query: maxima are then taken of S itself
            const float mag = mx > 0.f && mx < 1e30f ? exp2f(10.f - floorf(log2f(mx))) : 1.f;
            const float up = a.scale > 0.f ? mag : a.scale < 0.f ? -mag : 0.f;
            if (t == 0) s_sl2[r] = a.scale == 0.f ? 1.f : fabsf(a.scale) * kLog2e * (kCodeUnit / 16.f) / mag;
#pragma unroll
            for (int g = 0; g < NG; g++) {
                uint32_t* dst = reinterpret_cast<uint32_t*>(q_smem) + ((g * 4) * 32 + (r & 7) * 4 + t) * 4 + (r >> 3);
                float sum = 0.f;
#pragma unroll
                for (int e = 0; e < 2; e++) {
                    const uint4 x4 = qv[g][e];
                    const uint32_t w[4] = {__byte_perm(x4.x, x4.z, 0x5410), __byte_perm(x4.x, x4.z, 0x7632),
                                           __byte_perm(x4.y, x4.w, 0x5410), __byte_perm(x4.y, x4.w, 0x7632)};
#pragma unroll
                    for (int mm = 0; mm < 4; mm++) {
                        const float2 f = h2f(w[mm]);
                        sum += f.x * up + f.y * up;
                        const float u16 = mm & 1 ? up : 16.f * up;
                        dst[mm * 128 + e * 2] = f2h(f.x * u16, f.y * u16);
                        if (RT == 1) dst[mm * 128 + e * 2 + 1] = 0;
                    }
                }
                sum += __shfl_xor_sync(0xffffffffu, sum, 1);
                sum += __shfl_xor_sync(0xffffffffu, sum, 2);
                if (t == 0) s_qs[g][r] = sum * (16.f / kCodeUnit);
            }
        }
        __syncthreads();

        float qs[NG][RT], sl2[RT];
        int pos[RT], low[RT];
#pragma unroll
        for (int z = 0; z < RT; z++) {
            pos[z] = p0 + min(rt * R + g8 + 8 * z, rows - 1) / G;
            low[z] = a.window > 0 ? pos[z] - a.window + 1 : 0;
            sl2[z] = s_sl2[g8 + 8 * z];
#pragma unroll
            for (int g = 0; g < NG; g++) qs[g][z] = s_qs[g][g8 + 8 * z];
        }
        const int first_pos = p0 + (rt * R) / G;             // least and greatest row of the tile
        const int last_low = a.window > 0 ? p0 + (min(rt * R + R, rows) - 1) / G - a.window + 1 : 0;

        SplitAcc<NG, RT> A;
        A.unit = 0.f;
        A.chosen = false;
#pragma unroll
        for (int z = 0; z < RT; z++) {
            A.m[z] = -INFINITY;
            A.l[z] = 0.f;
#pragma unroll
            for (int g = 0; g < NG; g++) A.B[g][z] = 0.f;
#pragma unroll
            for (int j = 0; j < NG * 4; j++)
#pragma unroll
                for (int k = 0; k < 4; k++) A.O[z][j][k] = 0.f;
        }
        const uint32_t qb = smem_u32(q_smem);
        int st = 0;
        for (int pg = pg0 + par; pg < pg1; pg += kStep) {
            fetch(pg + kStep * (kSplitStages - 1), st == 0 ? kSplitStages - 1 : st - 1);
            cp_async_wait<kSplitStages - 1>();
            __syncwarp();
            const uint32_t kb = ring + st * Sh::kHalf;
            const bool page_ok = (ok >> st) & 1u;
            st = st == kSplitStages - 1 ? 0 : st + 1;
            const int j0 = pg * kKvPage + half * 32;
            if (!page_ok || j0 >= q.len) continue;           // nothing here (all lanes alike)
            if (j0 + 31 > first_pos || j0 < last_low) split_block<NG, RT, true>(A, kb, qb, qs, sl2, j0, pos, low);
            else split_block<NG, RT, false>(A, kb, qb, qs, sl2, j0, pos, low);
            __syncwarp();
        }
        cp_async_wait<0>();

        // join the warps: sums to shared memory (over the ring), relative to each warp's maximum
#pragma unroll
        for (int z = 0; z < RT; z++) {
            A.l[z] += __shfl_xor_sync(0xffffffffu, A.l[z], 1);
            A.l[z] += __shfl_xor_sync(0xffffffffu, A.l[z], 2);
#pragma unroll
            for (int g = 0; g < NG; g++) {
                A.B[g][z] += __shfl_xor_sync(0xffffffffu, A.B[g][z], 1);
                A.B[g][z] += __shfl_xor_sync(0xffffffffu, A.B[g][z], 2);
            }
            if (t4 == 0) {
                s_m[warp][g8 + 8 * z] = A.m[z] == -INFINITY ? A.m[z] : A.m[z] - A.unit;
                s_l[warp][g8 + 8 * z] = A.l[z];
            }
        }
        __syncthreads();                                     // every warp has left its ring
        float* join = reinterpret_cast<float*>(sp_smem);
#pragma unroll
        for (int z = 0; z < RT; z++)
#pragma unroll
            for (int g = 0; g < NG; g++)
#pragma unroll
                for (int k = 0; k < 2; k++) {                // rows 2t and 2t + 1
                    const float bb = row_value(A.B[g][z], k);
                    float4* dst = reinterpret_cast<float4*>(join + ((size_t)warp * R + 8 * z + 2 * t4 + k) * JR + g * 64 + g8 * 8);
                    const float(*v)[4] = &A.O[z][g * 4];
                    dst[0] = make_float4(v[0][k] + bb, v[1][k] + bb, v[2][k] + bb, v[3][k] + bb);
                    dst[1] = make_float4(v[0][2 + k] + bb, v[1][2 + k] + bb, v[2][2 + k] + bb,
                                         v[3][2 + k] + bb);
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
            if (d == 0) a.lse[(size_t)(q.first + i) * c.hq + head] = lse_of(M, L);
        };
        const auto add = [](float (&o)[8], float f, float4 v0, float4 v1) {
            o[0] = fmaf(f, v0.x, o[0]); o[1] = fmaf(f, v0.y, o[1]);
            o[2] = fmaf(f, v0.z, o[2]); o[3] = fmaf(f, v0.w, o[3]);
            o[4] = fmaf(f, v1.x, o[4]); o[5] = fmaf(f, v1.y, o[5]);
            o[6] = fmaf(f, v1.z, o[6]); o[7] = fmaf(f, v1.w, o[7]);
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
                if (s_m[w][r] == -INFINITY && s_l[w][r] == 0.f) continue;   // the warp's entries are not seen
                const float f = exp2_fast(s_m[w][r] - ref);
                const float4* src = reinterpret_cast<const float4*>(join + ((size_t)w * R + r) * JR + d);
                L = fmaf(f, s_l[w][r], L);
                add(o, f, src[0], src[1]);
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
                // every part's maximum and total at once, then its weight, then the sums of up to
                // sixteen parts in flight per thread
                __threadfence();
                const int parts = c1 - c0 + 1;
                float* pf = reinterpret_cast<float*>(sp_smem);           // [parts][R] weight (first the maximum)
                float* pl = pf + parts * R;                              // [parts][R] total
                const auto at = [&](int b) { return x.part + (size_t)(2 * (c0 + b) + (b == 0 ? 1 : 0)) * (R * (D + 2)); };
                for (int k = tid; k < parts * R; k += kSplitThreads) {
                    const float* src = at(k / R) + R * D + k % R;
                    pf[k] = __ldcg(src);
                    pl[k] = __ldcg(src + R);
                }
                __syncthreads();
                for (int r = warp; r < R; r += kSplitWarps) {
                    float M = -INFINITY, L = 0.f;
                    for (int b = lane; b < parts; b += 32) M = fmaxf(M, pf[b * R + r]);
#pragma unroll
                    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
                    const float ref = M == -INFINITY ? 0.f : M;
                    for (int b = lane; b < parts; b += 32) {
                        const float mb = pf[b * R + r], lb = pl[b * R + r];
                        const float f = mb == -INFINITY && lb == 0.f ? 0.f : exp2_fast(mb - ref);
                        pf[b * R + r] = f;
                        L = fmaf(f, lb, L);
                    }
                    L = warp_sum(L);
                    if (lane == 0) {
                        s_m[0][r] = M;
                        s_l[0][r] = L;
                    }
                }
                __syncthreads();
                for (int k = tid; k < R * (D / 4); k += kSplitThreads) {
                    const int r = k / (D / 4), d = (k % (D / 4)) * 4;
                    if (rt * R + r >= rows) continue;
                    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
                    for (int b0 = 0; b0 < parts; b0 += 16) {
                        float4 v[16];
#pragma unroll
                        for (int e = 0; e < 16; e++)
                            v[e] = b0 + e < parts ? __ldcg(reinterpret_cast<const float4*>(at(b0 + e) + (size_t)r * D + d))
                                                  : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                        for (int e = 0; e < 16; e++) {
                            const float f = b0 + e < parts ? pf[(b0 + e) * R + r] : 0.f;
                            o.x = fmaf(f, v[e].x, o.x);
                            o.y = fmaf(f, v[e].y, o.y);
                            o.z = fmaf(f, v[e].z, o.z);
                            o.w = fmaf(f, v[e].w, o.w);
                        }
                    }
                    const int i = (rt * R + r) / G, head = h * G + (rt * R + r) % G;
                    const float M = s_m[0][r], L = s_l[0][r], f = L == 0.f ? 0.f : 1.f / L;
                    *reinterpret_cast<uint2*>(a.out + (size_t)(q.first + i) * a.out_stride + (size_t)head * D + d) =
                        make_uint2(f2h(o.x * f, o.y * f), f2h(o.z * f, o.w * f));
                    if (d == 0) a.lse[(size_t)(q.first + i) * c.hq + head] = lse_of(M, L);
                }
                if (tid == 0) x.count[c0] = 0;
            }
        }
        __syncthreads();                                     // the ring and s_m are free again
    }
}

}  // namespace moeq4
