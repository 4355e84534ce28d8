"""The 4-bit KV cache in 64 bits, entry by entry (numpy; shares no code with the
CUDA library).  Layout and rules as include/moeq4.h states them."""
import numpy as np

PAGE = 64


def tile_bytes(D):
    return 4608 * (D // 64)


def entry(tile, D, part, e):
    """One entry's K (part 0) or V (part 1) from a tile's bytes, float64 [D]."""
    ng = D // 64
    out = np.empty(D)
    for g in range(ng):
        o = part * 2304 * ng + (g * PAGE + e) * 32
        byte = tile[o:o + 32]
        code = np.empty(64)
        code[0::2] = byte & 15                       # little-endian words: low nibble first
        code[1::2] = byte >> 4
        o = part * 2304 * ng + 2048 * ng + (g * PAGE + e) * 4
        s, b = tile[o:o + 4].view(np.float16).astype(np.float64)
        with np.errstate(invalid="ignore"):
            out[64 * g:64 * g + 64] = s * code + b
    return out


def sequence(pages, table, n, Hkv, D):
    """K and V float64 [Hkv][n][D] of a sequence's first n entries; pages uint8
    [n_pages][Hkv][tile]."""
    ng = D // 64
    kv = np.empty((2, Hkv, n, D))
    for p in range((n + PAGE - 1) // PAGE):
        m = min(PAGE, n - p * PAGE)
        t = pages[table[p]]
        for part in (0, 1):
            o = part * 2304 * ng
            b = t[:, o:o + 2048 * ng].reshape(Hkv, ng, PAGE, 32)
            c = np.stack((b & 15, b >> 4), -1).reshape(Hkv, ng, PAGE, 64).astype(np.float64)
            f = np.ascontiguousarray(t[:, o + 2048 * ng:o + 2304 * ng]).view(np.float16)
            f = f.reshape(Hkv, ng, PAGE, 2).astype(np.float64)
            with np.errstate(invalid="ignore"):
                x = f[..., :1] * c + f[..., 1:]
            kv[part, :, p * PAGE:p * PAGE + m] = x.transpose(0, 2, 1, 3).reshape(Hkv, PAGE, D)[:, :m]
    return kv[0], kv[1]


def value_spread(pages, table, V, D):
    """|V - (bias + 8 scale)| of a sequence's entries: the part scale * (code - 8)
    of each value, in size."""
    Hkv, n = V.shape[:2]
    ng = D // 64
    out = np.empty_like(V)
    for p in range((n + PAGE - 1) // PAGE):
        m = min(PAGE, n - p * PAGE)
        f = np.ascontiguousarray(pages[table[p]][:, 4352 * ng:]).view(np.float16).astype(np.float64)
        f = f.reshape(Hkv, ng, PAGE, 2)[:, :, :m]
        with np.errstate(invalid="ignore"):
            mid = np.repeat((f[..., 1] + 8 * f[..., 0]).transpose(0, 2, 1), 64, axis=2)
            out[:, p * PAGE:p * PAGE + m] = np.abs(V[:, p * PAGE:p * PAGE + m] - mid)
    return out


def attention(q, K, V, scale, window, n_entries):
    """q [n][Hq][D] of a sequence with n_entries entries: out [n][Hq][D], lse
    [n][Hq] and the weight each entry received [Hkv][n_entries]."""
    n, Hq, D = q.shape
    Hkv = K.shape[0]
    G = Hq // Hkv
    out = np.zeros((n, Hq, D))
    lse = np.full((n, Hq), -np.inf)
    got = np.zeros((Hkv, n_entries))
    for i in range(n):
        p = n_entries - n + i
        j0 = max(0, p - window + 1) if window else 0
        if p < 0 or j0 > p:
            continue
        for a in range(Hq):
            h = a // G
            S = K[h, j0:p + 1] @ q[i, a] * scale
            m = S.max()
            w = np.exp(S - m)
            lse[i, a] = m + np.log(w.sum())
            w /= w.sum()
            out[i, a] = w @ V[h, j0:p + 1]
            got[h, j0:p + 1] += w
    return out, lse, got


def quantise(x):
    """x float16 [..., 64]: the stored bytes of each group, uint8 [..., 32] codes
    and [..., 4] scale and bias (fp32 arithmetic, as the format defines it)."""
    v = x.astype(np.float32)
    bad = ~np.isfinite(v).all(-1, keepdims=True)
    v = np.where(bad, np.float32(0), v)
    lo, hi = v.min(-1, keepdims=True), v.max(-1, keepdims=True)
    s = ((hi - lo) / np.float32(15)).astype(np.float16)
    b = lo.astype(np.float16)
    with np.errstate(divide="ignore", invalid="ignore"):
        c = np.rint((v - b.astype(np.float32)) / s.astype(np.float32))
    c = np.where((s == 0) | bad, 0, np.clip(np.nan_to_num(c), 0, 15)).astype(np.uint8)
    sb = np.concatenate((s, b), -1).view(np.uint16)
    sb = np.where(bad, np.uint16(0x7FFF), sb)
    return c[..., 0::2] | (c[..., 1::2] << 4), np.ascontiguousarray(sb).view(np.uint8)


def append(pages, table, at, k, v):
    """Writes one row's K and V (float16 [Hkv][D]) at entry `at`."""
    Hkv, D = k.shape
    ng = D // 64
    t = pages[table[at // PAGE]]
    e = at % PAGE
    for part, x in ((0, k), (1, v)):
        codes, sb = quantise(x.reshape(Hkv, ng, 64))
        for g in range(ng):
            o = part * 2304 * ng + (g * PAGE + e) * 32
            t[:, o:o + 32] = codes[:, g]
            o = part * 2304 * ng + 2048 * ng + (g * PAGE + e) * 4
            t[:, o:o + 4] = sb[:, g]


def evict(pages, table, n, seen, score, pos, budget, recent):
    """One sequence; score and pos [Hkv][cap], changed in place with the pages.
    Returns the new length."""
    if n <= budget:
        return n
    Hkv = score.shape[0]
    ng = pages.shape[-1] // 4608
    for h in range(Hkv):
        def rank(j):
            s = score[h, j]
            late = pos[h, j] >= seen - recent
            return (0 if late else 1, 0 if (late or s == s) else 1, 0.0 if (late or s != s) else -float(s), j)
        stay = sorted(sorted(range(n), key=rank)[:budget])
        free = sorted(set(range(budget)) - set(stay))
        move = [j for j in stay if j >= budget]
        assert len(free) == len(move)
        for dst, src in zip(free, move):
            score[h, dst], pos[h, dst] = score[h, src], pos[h, src]
            ts, td = pages[table[src // PAGE], h], pages[table[dst // PAGE], h]
            a, b = src % PAGE, dst % PAGE
            for part in (0, 1):
                for g in range(ng):
                    o = part * 2304 * ng + g * PAGE * 32
                    td[o + 32 * b:o + 32 * b + 32] = ts[o + 32 * a:o + 32 * a + 32]
                    o = part * 2304 * ng + 2048 * ng + g * PAGE * 4
                    td[o + 4 * b:o + 4 * b + 4] = ts[o + 4 * a:o + 4 * a + 4]
    return budget
