"""4-bit KV cache on the GPU against the 64-bit reference (tests/kv_ref.py).

Tolerances.  Stored bytes, positions, lengths and moved entries are equal.  The
attention forms products of fp16 queries and integer codes in fp32: with unit
normal K and V and queries of 1.5 sigma, a score's partial sums stay below
about 40 (codes carry an offset of up to 64, 72 * 0.35 * 1.5), so the rounding
of a few dozen accumulation steps leaves about 1e-5 on a score and 4e-5 at the
far end of its distribution.  The weighted sum adds 16-entry steps of at most
79 * 0.35 * 2^-24 each, 3e-5 over 4096 entries.  Hence 1e-4 absolute on lse,
1e-4 relative (1e-6 absolute) on accumulated weights, and on the output 1e-4
beside the half step 2^-11 of its rounding to fp16 (2^-25 below the normal
range).

One more operand is rounded to fp16, off by at most half a step, 2^-11 of its size.
With up to 64 (row, head) pairs per kv head it is p s, the weight times a group's
scale: an output is sum_j p_j s_j (code_j - 8) + p_j (bias_j + 8 s_j) over sum p, so
it moves by at most 2^-11 sum_j w_j |s_j (code_j - 8)| with w = p / sum p.  With more
it is V itself, scale * code + bias: at most 2^-11 sum_j w_j |v_j|.  Both are
attentions of absolute values, which the reference forms (spread).
"""
import math

import numpy as np
import pytest
import torch

import kv_ref
from bit_quantized_expert_int8_b200 import build, moeq4
from bit_quantized_expert_int8_b200.config import KvConfig

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    moeq4.load()


def cu(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def random_pages(rng, n_pages, Hkv, D, sigma=1.0):
    ng = D // 64
    pages = np.empty((n_pages, Hkv, kv_ref.tile_bytes(D)), np.uint8)
    for part in (0, 1):
        x = (rng.standard_normal((n_pages, Hkv, ng, 64, 64)) * sigma).astype(np.float16)
        c, sb = kv_ref.quantise(x)
        o = part * 2304 * ng
        pages[:, :, o:o + 2048 * ng] = c.reshape(n_pages, Hkv, -1)
        pages[:, :, o + 2048 * ng:o + 2304 * ng] = sb.reshape(n_pages, Hkv, -1)
    return pages


class Case:
    """A cache and a batch on both sides."""

    def __init__(self, seed, D, Hq, Hkv, lens, rows, spare_rows=0, extra_pages=1, state=False, sigma=1.0,
                 max_pages=None):
        rng = self.rng = np.random.default_rng(seed)
        self.D, self.Hq, self.Hkv, self.n = D, Hq, Hkv, len(lens)
        self.lens, self.rows = np.array(lens, np.int32), np.array(rows, np.int32)
        self.max_pages = max_pages or max(1, -(-max(lens) // 64))
        self.n_pages = self.n * self.max_pages + extra_pages
        self.pages = random_pages(rng, self.n_pages, Hkv, D, sigma)
        self.table = rng.permutation(self.n_pages)[:self.n * self.max_pages].reshape(self.n, -1).astype(np.int32)
        self.start = np.concatenate(([0], np.cumsum(self.rows))).astype(np.int32)
        self.n_rows = int(self.start[-1]) + spare_rows
        self.cap = self.max_pages * 64
        self.score = self.pos = self.seen = None
        if state:
            self.score = rng.random((self.n, Hkv, self.cap)).astype(np.float32)
            self.pos = np.tile(np.arange(self.cap, dtype=np.int32), (self.n, Hkv, 1))
            self.seen = self.lens.copy()
        self.upload()

    def upload(self):
        self.kv = moeq4.Kv(KvConfig(self.Hq, self.Hkv, self.D, self.n_pages, self.max_pages,
                                    max_seqs=max(1, self.n), max_rows=max(1, self.n_rows)))
        opt = {k: None if getattr(self, k) is None else cu(getattr(self, k)) for k in ("score", "pos", "seen")}
        self.g = dict(pages=cu(self.pages), table=cu(self.table), lens=cu(self.lens), start=cu(self.start), **opt)
        self.cache = moeq4.KvCache(self.kv, self.g["pages"], self.g["table"], self.g["lens"], **opt)
        self.batch = moeq4.KvBatch(self.kv, self.g["start"], self.n_rows, max(1, int(self.rows.max(initial=0))))

    def queries(self):
        return (self.rng.standard_normal((self.n_rows, self.Hq, self.D)) * 1.5).astype(np.float16)

    def reference(self, q, scale, window=0):
        out, spread = np.zeros((2, self.n_rows, self.Hq, self.D))
        lse = np.full((self.n_rows, self.Hq), -np.inf)
        got = np.zeros((self.n, self.Hkv, self.cap))
        for s in range(self.n):
            a, b, n = self.start[s], self.start[s + 1], int(self.lens[s])
            if a == b:
                continue
            K, V = kv_ref.sequence(self.pages, self.table[s], n, self.Hkv, self.D)
            out[a:b], lse[a:b], got[s, :, :n] = kv_ref.attention(q[a:b].astype(np.float64), K, V, scale, window, n)
            spread[a:b] = self.spread(s, q[a:b], K, V, scale, window, n)
        return out, lse, got, spread

    def spread(self, s, q, K, V, scale, window, n):
        few = q.shape[0] * self.Hq // self.Hkv <= 64
        U = kv_ref.value_spread(self.pages, self.table[s], V, self.D) if few else np.abs(V)
        return kv_ref.attention(q.astype(np.float64), K, U, scale, window, n)[0]

    def attend(self, q, scale, window=0, weights=False, **kw):
        out = torch.full((self.n_rows, self.Hq, self.D), 7.0, dtype=torch.float16, device=DEV)
        lse = torch.full((self.n_rows, self.Hq), 7.0, device=DEV)
        moeq4.moe_attn_q4(self.kv, self.cache, self.batch, cu(q), out, lse=lse, scale=scale, window=window,
                          weights=weights, **kw)
        moeq4.moe_kv_check(self.kv)
        return out.cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)


def close(out, lse, ref, rows=None):
    ro, rl, rs = ref[0][:rows], ref[1][:rows], ref[3][:rows]
    out, lse = out[:rows], lse[:rows]
    assert np.isfinite(out).all()
    off = np.abs(out - ro) - (2.0 ** -11 * np.abs(ro) + 2.0 ** -11 * rs + 2.0 ** -25 + 1e-4)
    assert (off <= 0).all(), off.max()
    dead = np.isneginf(rl)
    assert (np.isneginf(lse) == dead).all()
    assert (np.abs(lse[~dead] - rl[~dead]) <= 1e-4).all(), np.abs(lse[~dead] - rl[~dead]).max()


SHAPES = [
    # D, Hq, Hkv, lens, rows, window
    (64, 1, 1, [1], [1], 0),
    (128, 8, 8, [5], [1], 0),
    (128, 16, 8, [64, 65, 63], [1, 1, 1], 0),
    (128, 32, 8, [300, 1, 1000, 129], [1, 1, 1, 1], 0),
    (64, 9, 3, [700, 10], [1, 1], 0),
    (192, 10, 2, [333, 511], [1, 2], 0),
    (256, 16, 2, [500, 77], [1, 1], 0),
    (256, 5, 1, [260, 1500], [1, 1], 100),
    (128, 22, 2, [400, 90], [1, 1], 0),                # 11 heads a kv head
    (128, 20, 1, [200], [1], 0),                       # 20 heads a kv head
    (128, 8, 2, [700, 70, 300], [3, 4, 2], 0),         # a few rows each
    (64, 4, 2, [100, 0, 50], [0, 0, 5], 0),            # sequences without rows or entries
    (128, 4, 2, [2, 40], [5, 1], 0),                   # rows before the first entry
    (128, 8, 4, [1000, 64, 65], [1, 1, 1], 1),
    (128, 8, 4, [1000, 64, 65], [1, 3, 2], 64),
    (128, 8, 4, [900], [7], 333),
    (128, 8, 2, [600], [600], 0),                      # a whole prompt
    (128, 8, 2, [900, 130, 64], [33, 130, 1], 0),      # chunks of several prompts
    (64, 6, 2, [500, 333], [100, 77], 50),
    (256, 4, 2, [700], [129], 0),
    (192, 6, 3, [300, 260], [64, 65], 0),
    (128, 16, 1, [400], [40], 0),
    (128, 3, 1, [517], [200], 129),
    (256, 8, 8, [1100], [70], 600),
    (128, 8, 2, [700, 65, 130], [16, 17, 5], 0),       # 64, 68 and 20 rows a kv head
    (192, 7, 1, [450, 40], [9, 8], 30),                # 63 and 56
    (64, 2, 2, [190, 70], [64, 65], 0),
    (64, 200, 1, [300, 70], [2, 1], 0),                # more heads than a tile has rows
    (64, 1024, 1, [130], [1], 0),
    (128, 8, 2, [300, 90], [1, 40], 2 ** 31 - 1),      # the widest window: all entries
]


@pytest.mark.parametrize("D,Hq,Hkv,lens,rows,window", SHAPES)
def test_attention(D, Hq, Hkv, lens, rows, window):
    c = Case(11 + D + Hq + sum(lens), D, Hq, Hkv, lens, rows)
    q = c.queries()
    out, lse = c.attend(q, 1 / math.sqrt(D), window)
    close(out, lse, c.reference(q, 1 / math.sqrt(D), window))


@pytest.mark.parametrize("D,Hq,Hkv,lens,rows,window", SHAPES)
def test_attention_weights(D, Hq, Hkv, lens, rows, window):
    c = Case(12 + D + Hq + sum(lens), D, Hq, Hkv, lens, rows, state=True)
    q = c.queries()
    ref = c.reference(q, 1 / math.sqrt(D), window)
    out, lse = c.attend(q, 1 / math.sqrt(D), window, weights=True)
    close(out, lse, ref)
    want = c.score.astype(np.float64) + ref[2]
    got = c.g["score"].cpu().numpy().astype(np.float64)
    assert (np.abs(got - want) <= 1e-4 * ref[2] + 2.0 ** -23 * np.abs(want) + 1e-6).all(), np.abs(got - want).max()
    for s in range(c.n):                               # nothing behind a sequence's last entry changes
        assert np.array_equal(got[s, :, lens[s]:], c.score[s, :, lens[s]:].astype(np.float64))


@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 64, 64, 3])
@pytest.mark.parametrize("Hq,lens,rows", [(4, [2, 40], [5, 1]), (4, [30, 0, 100], [60, 5, 7]), (16, [70, 5], [200, 9])])
def test_window_with_rows_before_the_first_entry(Hq, lens, rows, window):
    """Rows that stand before the first entry see nothing, those behind them all
    that the window shows, however wide it is."""
    c = Case(13 + Hq + sum(lens), 128, Hq, 2, lens, rows, state=True)
    q = c.queries()
    ref = c.reference(q, 0.09, window)
    out, lse = c.attend(q, 0.09, window, weights=True)
    close(out, lse, ref)
    want = c.score.astype(np.float64) + ref[2]
    got = c.g["score"].cpu().numpy().astype(np.float64)
    assert (np.abs(got - want) <= 1e-4 * ref[2] + 2.0 ** -23 * np.abs(want) + 1e-6).all(), np.abs(got - want).max()


@pytest.mark.parametrize("D,Hq,Hkv,lens,rows", [
    (128, 16, 4, [5000, 3000], [1, 1]), (256, 8, 4, [4000], [1]), (64, 8, 4, [4000], [4]),
    (128, 8, 4, [3000], [20]), (128, 8, 4, [3000], [100]), (256, 4, 4, [2500], [130]), (64, 8, 4, [2500], [120])])
def test_precision_over_long_sequences(D, Hq, Hkv, lens, rows):
    """Norms of the errors, where a bound on each element has to allow for all of an
    element's roundings at once.  Output: two roundings to fp16 (p s or V, and the output
    itself), each 2^-11 sqrt(1/3 / 2.164) = 1.92e-4 of a value with evenly distributed log,
    2.7e-4 together; a third one would make it 3.3e-4.  lse (8 to 10): a score's partial
    sums, below 40 * 0.09, are rounded to 2^-24 of that a few dozen times, 1e-6 to 5e-6 in
    all.  Weights: exp of that error."""
    c = Case(90 + D + sum(rows), D, Hq, Hkv, lens, rows, state=True)
    c.score[:] = 0
    c.upload()
    q = c.queries()
    ref = c.reference(q, 1 / math.sqrt(D))
    out, lse = c.attend(q, 1 / math.sqrt(D), weights=True)
    got = c.g["score"].cpu().numpy().astype(np.float64)

    def off(x, y):
        return np.linalg.norm(x - y) / np.linalg.norm(y)

    assert off(out, ref[0]) <= 3.2e-4
    assert off(lse, ref[1]) <= 5e-7
    assert off(got, ref[2]) <= 2e-6


def test_rows_of_the_first_sequence_begin_later():
    """row_start need not begin at 0: rows before it belong to nobody."""
    for rows in ([1, 2], [40, 50]):
        c = Case(83, 128, 8, 2, [200, 90], rows, spare_rows=6, state=True)
        q, n = c.queries(), sum(rows)
        kv = c.rng.standard_normal((2, c.n_rows, 2, 128)).astype(np.float16)
        batch = moeq4.KvBatch(c.kv, cu(c.start + 3), c.n_rows, max(rows))
        moeq4.moe_kv_append_q4(c.kv, c.cache, batch, cu(kv[0]), cu(kv[1]))
        for s in range(2):
            for i in range(rows[s]):
                r, at = c.start[s] + 3 + i, c.lens[s] - rows[s] + i
                kv_ref.append(c.pages, c.table[s], at, kv[0][r], kv[1][r])
        assert np.array_equal(c.g["pages"].cpu().numpy(), c.pages)
        ref = c.reference(np.roll(q, -3, axis=0), 0.09)
        c.batch = batch
        out, lse = c.attend(q, 0.09)
        close(out[3:], lse[3:], ref, n)
        assert (out[:3] == 7).all() and (out[n + 3:] == 7).all() and (lse[:3] == 7).all() and (lse[n + 3:] == 7).all()
        back = torch.full((2, c.n_rows, 2, 128), 7.0, dtype=torch.float16, device=DEV)
        moeq4.moe_kv_read_q4(c.kv, c.cache, batch, back[0], back[1])
        moeq4.moe_kv_check(c.kv)
        assert (back[:, :3] == 7).all() and (back[:, n + 3:] == 7).all() and (back[:, 3:n + 3] != 7).any()


def test_long_sequences_and_split_work():
    c = Case(21, 128, 16, 4, [9000, 3, 2500, 640], [1, 1, 1, 1], state=True)
    q = c.queries()
    ref = c.reference(q, 0.11)
    out, lse = c.attend(q, 0.11, weights=True)
    close(out, lse, ref)
    again = c.attend(q, 0.11)                          # and the same bits on every run
    assert np.array_equal(out, again[0]) and np.array_equal(lse, again[1])


def test_many_sequences():
    rng = np.random.default_rng(5)
    lens = rng.integers(1, 200, 300).tolist()
    c = Case(22, 64, 4, 2, lens, [1] * 300)
    q = c.queries()
    out, lse = c.attend(q, 0.125)
    close(out, lse, c.reference(q, 0.125))


@pytest.mark.parametrize("scale", [0.0, -0.3, 1.0])
def test_scales(scale):
    c = Case(23, 128, 8, 2, [200, 90], [1, 20])
    q = (c.queries().astype(np.float32) * 0.3).astype(np.float16)
    out, lse = c.attend(q, scale)
    close(out, lse, c.reference(q, scale))


@pytest.mark.parametrize("rows", [[1, 9], [40, 70]])
@pytest.mark.parametrize("scale", [2.0 ** -32, -(2.0 ** 32), 2.0 ** 32])
def test_smallest_and_largest_scales(scale, rows):
    """The least scale makes every entry count alike, the largest one leaves one entry a row."""
    c = Case(74, 128, 8, 2, [200, 90], rows)
    q = c.queries()
    if abs(scale) > 1:                                           # scores of a few million: below 2^28
        q = (q.astype(np.float64) * 2.0 ** -14).astype(np.float16)
    ref = c.reference(q, scale)
    out, lse = c.attend(q, scale)
    rl = ref[1]
    # lse is as large as the scores are: their partial sums (at most 40, see above) are
    # rounded a few dozen times, which is below 1e-5 of a score of a few units
    assert (np.abs(lse - rl) <= 1e-4 + 1e-5 * np.abs(rl)).all()
    assert (np.abs(out - ref[0]) <= 2.0 ** -11 * (np.abs(ref[0]) + ref[3]) + 2.0 ** -25 + 1e-4).all()


@pytest.mark.parametrize("scale", [2.0 ** -33, -1e-30, 2.0 ** 33, -3e38, 1e-45])
def test_scales_out_of_range_are_refused(scale):
    c = Case(75, 128, 8, 2, [20], [2])
    q = cu(c.queries())
    out = torch.full_like(q, 7)
    refused(moeq4.MOE_ERR_INVALID_ARG, moeq4.moe_attn_q4, c.kv, c.cache, c.batch, q, out, scale=scale)
    assert (out == 7).all()


@pytest.mark.parametrize("sigma", [1e-4, 300.0])
def test_small_and_large_values(sigma):
    """V of any size: the output's error scales with it."""
    c = Case(24, 128, 8, 2, [300, 90], [1, 30], sigma=sigma)
    q = (c.queries().astype(np.float64) / sigma).clip(-60000, 60000).astype(np.float16)
    ref = c.reference(q, 0.09)
    out, lse = c.attend(q, 0.09)
    # q / sigma is rounded to fp16 (subnormal for 300) on both sides alike; the
    # code offset makes partial sums of the bias part about as large as above.
    # At 1e-4 the output itself is in fp16's subnormal range, where a half step is 2^-25
    assert (np.abs(out - ref[0]) <= 2.0 ** -11 * (np.abs(ref[0]) + ref[3]) + 2.0 ** -25 + 1e-4 * sigma).all()
    assert (np.abs(lse - ref[1]) <= 1e-4).all()


def test_mixed_value_scales():
    """Entries whose V is a million times smaller than others' must not push the
    others out of range, wherever they stand."""
    c = Case(25, 128, 4, 1, [640], [1])
    big = random_pages(c.rng, c.n_pages, 1, 128, 100.0)
    for j, p in enumerate(c.table[0]):
        if j in (3, 7):
            o = 2304 * 2
            c.pages[p, :, o:] = big[p, :, o:]
        if j in (0, 5):
            o = 2304 * 2 + 2048 * 2
            sb = c.pages[p, :, o:].copy().view(np.float16)
            c.pages[p, :, o:] = (sb.astype(np.float64) * 1e-4).astype(np.float16).view(np.uint8)
    c.upload()
    q = c.queries()
    ref = c.reference(q, 0.05)
    out, lse = c.attend(q, 0.05)
    assert (np.abs(out - ref[0]) <= 2.0 ** -11 * (np.abs(ref[0]) + ref[3]) + 1e-4 * 100).all()
    # with the large pages masked away the small ones alone have to be exact
    c2 = Case(25, 128, 4, 1, [640], [1])
    for p in c2.table[0]:
        o = 2304 * 2 + 2048 * 2
        sb = c2.pages[p, :, o:].copy().view(np.float16)
        c2.pages[p, :, o:] = (sb.astype(np.float64) * 2.0 ** -10).astype(np.float16).view(np.uint8)
    c2.upload()
    ref = c2.reference(q, 0.05)
    out, lse = c2.attend(q, 0.05)
    assert (np.abs(out - ref[0]) <= 2.0 ** -11 * (np.abs(ref[0]) + ref[3]) + 2.0 ** -25 + 1e-4 * 2.0 ** -10).all()


@pytest.mark.parametrize("rows,window", [([1, 1], 0), ([1, 1], 20), ([9, 40], 0), ([9, 40], 20), ([130, 140], 30)])
def test_masked_entries_may_hold_anything(rows, window):
    """NaN and infinite scales behind the last entry, before the window and in
    pages that no row sees leave no trace."""
    c = Case(26, 128, 8, 2, [150, 201], rows, extra_pages=2)
    q = c.queries()
    ref = c.reference(q, 0.09, window)
    bad = np.frombuffer(np.array([np.nan, np.inf, -np.inf, 65504], np.float16).tobytes(), np.uint8)
    used = {}
    for s in range(c.n):
        first = c.lens[s] - rows[s]
        lo = max(0, first - window + 1) if window else 0
        for j in range(lo, int(c.lens[s])):
            used.setdefault(int(c.table[s, j // 64]), set()).add(j % 64)
    ng = 2
    for p in range(c.n_pages):
        for e in range(64):
            if e in used.get(p, ()):
                continue
            for part in (0, 1):
                for g in range(ng):
                    o = part * 2304 * ng + 2048 * ng + (g * 64 + e) * 4
                    c.pages[p, :, o:o + 4] = np.roll(bad, 2 * ((e + g) % 4))[:4]
    c.upload()
    out, lse = c.attend(q, 0.09, window)
    close(out, lse, ref)


def test_nan_reaches_only_the_rows_that_see_it():
    c = Case(27, 128, 4, 2, [100], [30])
    k = np.zeros((2, 128), np.float16)
    k[1, 3] = np.nan
    kv_ref.append(c.pages, c.table[0], 85, k, k)       # rows 15.. of 30 see entry 85; kv head 1 only
    c.upload()
    out, lse = c.attend(c.queries(), 0.09)
    assert np.isfinite(out[:15]).all() and np.isfinite(out[:, :2]).all() and np.isfinite(lse[:, :2]).all()
    assert np.isnan(out[15:, 2:]).all() and np.isnan(lse[15:, 2:]).all()


def scale_v(pages, table, j, factor, groups=(0, 1)):
    """Entry j's V times a factor (its scales and biases; 128 columns, all kv heads)."""
    for g in groups:
        o = 2304 * 2 + 2048 * 2 + (g * 64 + j % 64) * 4
        sb = pages[table[j // 64], :, o:o + 4].copy().view(np.float16).astype(np.float64)
        with np.errstate(over="ignore"):
            pages[table[j // 64], :, o:o + 4] = (sb * factor).astype(np.float16).view(np.uint8)


@pytest.mark.parametrize("rows,window", [([1, 1], 0), ([9, 40], 20), ([70, 80], 0), ([130, 140], 30)])
def test_masked_entries_add_no_weight(rows, window):
    """As above with weights: NaN scales outside the rows' range leave scores alone too."""
    c = Case(26, 128, 8, 2, [150, 201], rows, extra_pages=2, state=True)
    q = c.queries()
    ref = c.reference(q, 0.09, window)
    ng = 2
    for s in range(c.n):
        first = c.lens[s] - rows[s]
        lo = max(0, first - window + 1) if window else 0
        for j in [*range(lo), *range(int(c.lens[s]), c.cap)]:
            for o in range(2048 * ng + (j % 64) * 4, 4608 * ng, 256):
                if o % (2304 * ng) >= 2048 * ng:
                    c.pages[c.table[s, j // 64], :, o:o + 4] = np.array([np.nan, np.inf], np.float16).view(np.uint8)
    c.upload()
    out, lse = c.attend(q, 0.09, window, weights=True)
    close(out, lse, ref)
    want = c.score.astype(np.float64) + ref[2]
    got = c.g["score"].cpu().numpy().astype(np.float64)
    assert (np.abs(got - want) <= 1e-4 * ref[2] + 2.0 ** -23 * np.abs(want) + 1e-6).all()


@pytest.mark.parametrize("what", ["k", "v"])
@pytest.mark.parametrize("rows", [30, 80, 200])
def test_nan_reaches_only_the_rows_that_see_it_with_many_rows(rows, what):
    """A row appended with NaN in kv head 1: that head's rows behind it get NaN (in V's
    group of 64 columns alone), all others what they would get anyway."""
    c = Case(27, 128, 4, 2, [300], [rows], state=True)
    q = c.queries()
    at, i = 300 - rows // 2, rows - rows // 2                    # row i stands at entry `at`
    new = c.rng.standard_normal((2, 2, 128)).astype(np.float16)
    kv_ref.append(c.pages, c.table[0], at, *new)
    ref = c.reference(q, 0.09)
    new[0 if what == "k" else 1][1, 3] = np.nan
    kv_ref.append(c.pages, c.table[0], at, *new)
    c.upload()
    out, lse = c.attend(q, 0.09, weights=True)
    cols = slice(0, 128 if what == "k" else 64)
    assert np.isnan(out[i:, 2:, cols]).all()
    out[i:, 2:, cols] = ref[0][i:, 2:, cols]
    if what == "k":
        assert np.isnan(lse[i:, 2:]).all()
        lse[i:, 2:] = ref[1][i:, 2:]
    close(out, lse, ref)
    got = c.g["score"].cpu().numpy()[0].astype(np.float64)
    want = c.score[0].astype(np.float64) + ref[2][0]
    assert (np.abs(got - want)[0] <= 1e-4 * ref[2][0, 0] + 2.0 ** -23 * want[0] + 1e-6).all()
    if what == "k":
        assert np.isnan(got[1, :300]).all()                      # a weight of every entry is NaN
    else:
        assert (np.abs(got - want)[1] <= 1e-4 * ref[2][0, 1] + 2.0 ** -23 * want[1] + 1e-6).all()


@pytest.mark.parametrize("D,Hq,Hkv,rows", [(128, 16, 8, 256), (64, 16, 16, 130), (256, 8, 8, 200)])
def test_v_that_grows_and_shrinks_between_pages(D, Hq, Hkv, rows):
    """V a thousand times larger, and smaller, from one page to the next, with many rows
    and several pages a CTA: what has been summed follows the unit that V is held in."""
    c = Case(80 + D, D, Hq, Hkv, [2000], [rows])
    ng = D // 64
    factor = 10.0 ** np.array([0, -3, 0, 2, -1, 3, 0, -3])       # V of 1e-3 to 1e3
    for p in range(c.max_pages):
        o = 2304 * ng + 2048 * ng
        t = c.pages[c.table[0, p], :, o:]
        t[:] = (t.copy().view(np.float16).astype(np.float64) * factor[p % 8]).astype(np.float16).view(np.uint8)
    c.upload()
    q = c.queries()
    ref = c.reference(q, 0.7 / math.sqrt(D))
    out, lse = c.attend(q, 0.7 / math.sqrt(D))
    # the terms are as large as the largest V, 1000
    assert (np.abs(out - ref[0]) <= 2.0 ** -11 * (np.abs(ref[0]) + ref[3]) + 2.0 ** -25 + 1e-4 * 1000).all()
    assert (np.abs(lse - ref[1]) <= 1e-4).all()
    # as a whole: two roundings to fp16, each sqrt(E e^2 / E x^2) = 2^-11 sqrt(1/3 / 2.164) = 1.92e-4
    # of a value with evenly distributed log, 2.7e-4 together; three would be 3.3e-4
    assert np.linalg.norm(out - ref[0]) <= 3.2e-4 * np.linalg.norm(ref[0])


@pytest.mark.parametrize("bad", [np.inf, np.nan])
@pytest.mark.parametrize("rows", [8, 16, 30, 70, 140])          # 8 and 16 rows a tile, 128 on the tile kernel
def test_v_out_of_range_stays_with_the_rows_that_see_it(rows, bad):
    """The last entry's V is not finite, in one group of 64 columns: other rows, and
    the last row's other group, stay right beside V whose scale is near the largest."""
    c = Case(76, 128, 2, 2, [400], [rows])
    tile = c.pages[c.table[0, 6]]                                # entries 384 to 399
    ng = 2
    for g in range(ng):
        o = 2304 * ng + g * 2048
        tile[:, o + 32:o + 16 * 32] &= 0x11                      # codes 0 and 1
        o = 2304 * ng + 2048 * ng + g * 256
        tile[:, o + 4:o + 16 * 4] = np.tile(np.array([50000, 0], np.float16).view(np.uint8), 15)
    q = c.queries()
    ref = c.reference(q, 0.09)
    o = 2304 * ng + 2048 * ng + 15 * 4
    tile[:, o:o + 4] = np.array([bad, 0], np.float16).view(np.uint8)
    c.upload()
    out, lse = c.attend(q, 0.09)
    assert not np.isfinite(out[-1, :, :64]).any()
    out[-1, :, :64] = ref[0][-1, :, :64]
    assert np.isfinite(out).all()
    # 2^-11 of the spread, and sums of 16-entry steps as in the tolerances above, of values
    # 50000 times as large
    assert (np.abs(out - ref[0]) <= 2.0 ** -11 * (np.abs(ref[0]) + ref[3]) + 1e-4 * 50000).all()
    assert (np.abs(lse - ref[1]) <= 1e-4).all()


def test_rows_behind_the_last_sequence_stay():
    for rows in ([1, 2], [40, 3]):
        c = Case(28, 128, 8, 2, [200, 90], rows, spare_rows=5)
        q = c.queries()
        out, lse = c.attend(q, 0.09)
        n = sum(rows)
        close(out, lse, c.reference(q, 0.09), n)
        assert (out[n:] == 7).all() and (lse[n:] == 7).all()


def test_strided_rows_and_no_lse():
    c = Case(29, 128, 8, 2, [200, 90], [3, 20])
    q = c.queries()
    wide = torch.zeros((c.n_rows, 13, 128), dtype=torch.float16, device=DEV)
    wide[:, 2:10] = cu(q)
    outw = torch.full((c.n_rows, 11, 128), 3.0, dtype=torch.float16, device=DEV)
    moeq4.moe_attn_q4(c.kv, c.cache, c.batch, wide[:, 2:10], outw[:, 1:9], scale=0.09)
    out, lse = c.attend(q, 0.09)
    assert np.array_equal(outw[:, 1:9].cpu().numpy().astype(np.float64), out)
    assert (outw[:, 0] == 3).all() and (outw[:, 9:] == 3).all()


def test_shared_pages():
    """Two sequences with the same prefix pages."""
    c = Case(30, 128, 8, 2, [300, 200], [1, 1])
    c.table[1, :3] = c.table[0, :3]
    c.upload()
    q = c.queries()
    out, lse = c.attend(q, 0.09)
    close(out, lse, c.reference(q, 0.09))


def test_pool_offsets_beyond_32_bits():
    D, Hkv = 256, 8
    per = moeq4.kv_page_bytes(Hkv, D)
    n_pages = (1 << 32) // per + 600
    kv = moeq4.Kv(KvConfig(8, Hkv, D, n_pages, 4, max_seqs=1, max_rows=1))
    pool = torch.empty(n_pages * per, dtype=torch.uint8, device=DEV)
    rng = np.random.default_rng(31)
    small = random_pages(rng, 4, Hkv, D)
    at = [n_pages - 1, 5, n_pages - 3, (1 << 31) // per + 1]
    for i, p in enumerate(at):
        pool[p * per:(p + 1) * per] = cu(small[i].reshape(-1))
    table = cu(np.array([at], np.int32))
    cache = moeq4.KvCache(kv, pool, table, cu(np.array([250], np.int32)))
    batch = moeq4.KvBatch(kv, cu(np.array([0, 1], np.int32)), 1, 1)
    q = rng.standard_normal((1, 8, D)).astype(np.float16)
    k = rng.standard_normal((1, Hkv, D)).astype(np.float16)
    moeq4.moe_kv_append_q4(kv, cache, batch, cu(k), cu(k))
    kv_ref.append(small, [0, 1, 2, 3], 249, k[0], k[0])
    out = torch.zeros((1, 8, D), dtype=torch.float16, device=DEV)
    lse = torch.zeros((1, 8), device=DEV)
    moeq4.moe_attn_q4(kv, cache, batch, cu(q), out, lse=lse, scale=0.06)
    moeq4.moe_kv_check(kv)
    K, V = kv_ref.sequence(small, [0, 1, 2, 3], 250, Hkv, D)
    U = kv_ref.value_spread(small, [0, 1, 2, 3], V, D)
    ref = (*kv_ref.attention(q.astype(np.float64), K, V, 0.06, 0, 250),
           kv_ref.attention(q.astype(np.float64), K, U, 0.06, 0, 250)[0])
    close(out.cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64), ref)
    assert np.array_equal(pool[at[3] * per:(at[3] + 1) * per].cpu().numpy(), small[3].reshape(-1))


# ------------------------------------------------------- append and read --
@pytest.mark.parametrize("D,Hkv,lens,rows", [
    (64, 1, [1], [1]), (128, 8, [70, 64, 200], [1, 1, 1]), (128, 3, [100, 5, 64, 130], [60, 5, 0, 70]),
    (192, 2, [65], [65]), (256, 5, [300, 299], [300, 1])])
def test_append_and_read(D, Hkv, lens, rows):
    c = Case(41 + D, D, Hkv, Hkv, lens, rows, spare_rows=2, state=True)
    c.seen += 1000
    c.upload()
    qkv = c.rng.standard_normal((c.n_rows, 3 * Hkv + 1, D)).astype(np.float16)
    qkv[0, 0, :64] = 1.5                               # a constant group
    qkv[0, Hkv, :] = 0
    if c.n_rows > 3:
        qkv[1, 0, 5] = np.inf
        qkv[1, -1, 7] = np.nan
        qkv[2, 1 % Hkv] *= np.float16(6e-6)            # subnormal scales
        qkv[2, 2 * Hkv + 1] = np.where(np.arange(D) % 2, 65504, -65504)
    k, v = qkv[:, :Hkv], qkv[:, 2 * Hkv + 1:]
    g = cu(qkv)
    moeq4.moe_kv_append_q4(c.kv, c.cache, c.batch, g[:, :Hkv], g[:, 2 * Hkv + 1:])
    ko = torch.full((c.n_rows, Hkv, D), 7.0, dtype=torch.float16, device=DEV)
    vo = torch.full((c.n_rows, Hkv + 1, D), 7.0, dtype=torch.float16, device=DEV)
    moeq4.moe_kv_read_q4(c.kv, c.cache, c.batch, ko, vo[:, :Hkv])
    moeq4.moe_kv_check(c.kv)
    for s in range(c.n):
        for i in range(rows[s]):
            at, r = lens[s] - rows[s] + i, c.start[s] + i
            kv_ref.append(c.pages, c.table[s], at, k[r], v[r])
            c.score[s, :, at] = 0
            c.pos[s, :, at] = c.seen[s] - rows[s] + i
    assert np.array_equal(c.g["pages"].cpu().numpy(), c.pages)
    assert np.array_equal(c.g["score"].cpu().numpy(), c.score)
    assert np.array_equal(c.g["pos"].cpu().numpy(), c.pos)
    for s in range(c.n):
        K, V = kv_ref.sequence(c.pages, c.table[s], lens[s], Hkv, D)
        a, b = c.start[s], c.start[s + 1]
        for X, got in ((K, ko), (V, vo[:, :Hkv])):
            # scale * code + bias in fp32, then one rounding to fp16
            want = X[:, lens[s] - rows[s]:].transpose(1, 0, 2).astype(np.float32).astype(np.float16)
            assert np.array_equal(got[a:b].cpu().numpy(), want, equal_nan=True)
    n = int(c.start[-1])
    assert (ko[n:] == 7).all() and (vo[:, Hkv:] == 7).all() and (vo[n:] == 7).all()


@pytest.mark.parametrize("seed", range(4))
def test_append_many_values(seed):
    """Scales over fp16's whole range, and groups built on half steps: the codes
    are those of the correctly rounded fp32 quotient, bit for bit."""
    c = Case(45 + seed, 128, 8, 8, [1500], [1500])
    rng = c.rng
    if seed < 2:
        kv = rng.standard_normal((2, 1500, 8, 128)) * np.exp2(rng.integers(-14, 11, (2, 1500, 8, 1)))
        if seed:
            kv = kv + np.exp2(rng.integers(-6, 12, (2, 1500, 8, 1))) * rng.standard_normal((2, 1500, 8, 1))
        kv = kv.clip(-65504, 65504).astype(np.float16)
    else:                                              # lo + s (code / 2): quotients at and next to .5
        s = rng.integers(1024, 2048, (2, 1500, 8, 2, 1)) * np.exp2(rng.integers(-12, -8, (2, 1500, 8, 2, 1)))
        x = rng.integers(0, 31, (2, 1500, 8, 2, 64)) * 0.5
        x[..., 0], x[..., 1] = 0, 15
        lo = 0 if seed == 2 else rng.integers(-2048, 2048, (2, 1500, 8, 2, 1))
        kv = (lo + s * x).astype(np.float16).reshape(2, 1500, 8, 128)
    moe_k, moe_v = cu(kv[0]), cu(kv[1])
    moeq4.moe_kv_append_q4(c.kv, c.cache, c.batch, moe_k, moe_v)
    moeq4.moe_kv_check(c.kv)
    got = c.g["pages"].cpu().numpy()[c.table[0]]       # [pages][8][tile]
    for part in (0, 1):
        codes, sb = kv_ref.quantise(kv[part].reshape(1500, 8, 2, 64))
        pad = np.zeros((24 * 64 - 1500, 8, 2, 36), np.uint8)
        want = np.concatenate((np.concatenate((codes, sb), -1), pad)).reshape(24, 64, 8, 2, 36).transpose(0, 2, 3, 1, 4)
        o = part * 4608
        have = np.concatenate((got[:, :, o:o + 4096].reshape(24, 8, 2, 64, 32),
                               got[:, :, o + 4096:o + 4608].reshape(24, 8, 2, 64, 4)), -1)
        have[-1, :, :, 1500 - 23 * 64:] = 0
        assert np.array_equal(have, want)


# --------------------------------------------------------------- eviction --
def check_evict(c, budget, recent):
    new = torch.full((c.n,), -5, dtype=torch.int32, device=DEV)
    moeq4.moe_kv_evict(c.kv, c.cache, c.n, budget, recent, new)
    moeq4.moe_kv_check(c.kv)
    want = [kv_ref.evict(c.pages, c.table[s], int(c.lens[s]), int(c.seen[s]), c.score[s], c.pos[s], budget, recent)
            for s in range(c.n)]
    assert new.cpu().tolist() == want
    assert np.array_equal(c.g["pos"].cpu().numpy(), c.pos)
    assert np.array_equal(c.g["score"].cpu().numpy(), c.score, equal_nan=True)
    assert np.array_equal(c.g["pages"].cpu().numpy(), c.pages)
    return new


@pytest.mark.parametrize("D,Hkv,lens,budget,recent", [
    (64, 1, [2], 1, 0), (64, 1, [2], 1, 1), (128, 8, [100, 64, 65, 1, 0], 64, 10), (128, 2, [700, 333], 200, 200),
    (192, 1, [3000], 2999, 0), (256, 2, [500, 501], 1, 0), (128, 3, [1500, 1025], 1024, 100),
    (64, 2, [5000, 4096], 33, 31)])
def test_evict(D, Hkv, lens, budget, recent):
    check_evict(Case(51 + D, D, Hkv, Hkv, lens, [1] * len(lens), state=True), budget, recent)


@pytest.mark.parametrize("kind", ["ties", "zeros", "nan", "inf", "negative", "shuffled", "all recent"])
def test_evict_orders(kind):
    c = Case(52, 128, 4, 2, [900, 400], [1, 1], state=True)
    s = c.score
    recent = 50
    if kind == "ties":
        s[:] = np.floor(s * 4) / 4
    elif kind == "zeros":
        s[:] = np.where(s < 0.9, np.where(s < 0.4, 0.0, -0.0), s)
    elif kind == "nan":
        s[:] = np.where(s < 0.5, np.float32(np.nan), s)
        s[1, 0] = np.nan
    elif kind == "inf":
        s[:] = np.where(s < 0.2, -np.inf, np.where(s > 0.8, np.inf, s))
    elif kind == "negative":
        s[:] = s - 0.5
    elif kind == "shuffled":
        c.pos = c.rng.permuted(c.pos[..., :900], axis=-1)
        c.pos = np.concatenate((c.pos, np.full((2, 2, c.cap - 900), 5, np.int32)), -1)
    else:
        c.pos[:] = 2000
        recent = 256
    c.upload()
    check_evict(c, 256, recent)


def test_evict_many_entries_one_head():
    check_evict(Case(53, 64, 1, 1, [70000], [1], state=True), 30000, 1000)


def test_evict_more_moves_than_a_list_holds():
    check_evict(Case(54, 64, 1, 1, [140000], [1], state=True), 70000, 10)


@pytest.mark.parametrize("kind", ["equal", "descending", "ascending", "ties", "zeros", "nan", "all recent", "one move"])
@pytest.mark.parametrize("entries", [4500, 8300, 16500])        # clusters of 2, 4 and 8 CTAs
def test_evict_orders_across_parts(entries, kind):
    """Orders whose borders, ties or lack of any move lie across the parts of a cluster."""
    c = Case(55, 64, 2, 2, [entries, entries - 300], [1, 1], state=True)
    s, budget, recent = c.score, entries // 2 + 5, 0
    if kind == "equal":                                          # the first `budget` entries stay: nothing moves
        s[:] = 0.25
    elif kind == "descending":
        s[:] = -np.arange(c.cap, dtype=np.float32)
    elif kind == "ascending":                                    # as many moves as there can be
        s[:] = np.arange(c.cap, dtype=np.float32)
    elif kind == "ties":
        s[:] = np.floor(s * 3)
    elif kind == "zeros":
        s[:] = np.where(s < 0.9, np.where(s < 0.4, 0.0, -0.0), s)
    elif kind == "nan":
        s[:] = np.where(s < 0.6, np.float32(np.nan), s)
        s[1, 0] = np.nan
    elif kind == "all recent":
        c.pos[:] = 3 * entries
        recent = budget
    else:
        s[:] = 0.25
        s[:, :, 3] = 0.0
        s[1, 1, 3] = 0.25                                        # and one (sequence, head) without any
    c.upload()
    check_evict(c, budget, recent)
    if kind in ("equal", "descending"):                          # nothing has changed: the same again, many times
        new = torch.zeros(c.n, dtype=torch.int32, device=DEV)
        for _ in range(50):
            moeq4.moe_kv_evict(c.kv, c.cache, c.n, budget, recent, new)
        moeq4.moe_kv_check(c.kv)
        for name in ("pos", "score", "pages"):
            assert np.array_equal(c.g[name].cpu().numpy(), getattr(c, name))


# ------------------------------------------------------ a run of them all --
def test_bounded_decode_steps():
    """Prompt chunk, then decode steps with a bounded cache: append, attention
    with weights, eviction, as a serving loop makes them."""
    rng = np.random.default_rng(61)
    n, Hq, Hkv, D, max_pages, budget, recent = 3, 8, 2, 128, 4, 150, 16
    rows0 = [140, 200, 20]
    kv = moeq4.Kv(KvConfig(Hq, Hkv, D, n * max_pages, max_pages, max_seqs=n, max_rows=sum(rows0)))
    pages = rng.integers(0, 256, (n * max_pages, Hkv, kv_ref.tile_bytes(D)), dtype=np.uint8)
    table = rng.permutation(n * max_pages).reshape(n, -1).astype(np.int32)
    score = np.zeros((n, Hkv, max_pages * 64), np.float32)
    pos = np.full((n, Hkv, max_pages * 64), -1, np.int32)
    lens, seen = np.zeros(n, np.int32), np.zeros(n, np.int32)
    gp, gt, gs, gpos, gseen = cu(pages), cu(table), cu(score), cu(pos), cu(seen)
    glens = [cu(lens), cu(lens)]
    caches = [moeq4.KvCache(kv, gp, gt, x, score=gs, pos=gpos, seen=gseen) for x in glens]
    score64 = score.astype(np.float64)
    for step in range(4):
        rows = np.array(rows0 if step == 0 else [1] * n, np.int32)
        start = np.concatenate(([0], np.cumsum(rows))).astype(np.int32)
        qkv = (rng.standard_normal((start[-1], Hq + 2 * Hkv, D)) * 1.2).astype(np.float16)
        g, grows = cu(qkv), cu(rows)
        batch = moeq4.KvBatch(kv, cu(start), int(start[-1]), int(rows.max()))
        now, nxt = step % 2, 1 - step % 2
        glens[now] += grows
        gseen += grows
        out = torch.empty((int(start[-1]), Hq, D), dtype=torch.float16, device=DEV)
        lse = torch.empty((int(start[-1]), Hq), device=DEV)
        moeq4.moe_kv_append_q4(kv, caches[now], batch, g[:, Hq:Hq + Hkv], g[:, Hq + Hkv:])
        moeq4.moe_attn_q4(kv, caches[now], batch, g[:, :Hq], out, lse=lse, scale=0.09, weights=True)
        moeq4.moe_kv_evict(kv, caches[now], n, budget, recent, glens[nxt])
        moeq4.moe_kv_check(kv)
        lens = lens + rows
        seen = seen + rows
        # the reference goes on from the library's scores: a near tie may fall either way
        got = gs.cpu().numpy()
        for s in range(n):
            a, b = start[s], start[s + 1]
            for i in range(rows[s]):
                at = lens[s] - rows[s] + i
                kv_ref.append(pages, table[s], at, qkv[a + i, Hq:Hq + Hkv], qkv[a + i, Hq + Hkv:])
                score64[s, :, at] = 0
                pos[s, :, at] = seen[s] - rows[s] + i
            K, V = kv_ref.sequence(pages, table[s], int(lens[s]), Hkv, D)
            ro, rl, w = kv_ref.attention(qkv[a:b, :Hq].astype(np.float64), K, V, 0.09, 0, int(lens[s]))
            U = np.abs(V) if rows[s] * Hq // Hkv > 16 else kv_ref.value_spread(pages, table[s], V, D)
            rs = kv_ref.attention(qkv[a:b, :Hq].astype(np.float64), K, U, 0.09, 0, int(lens[s]))[0]
            close(out[a:b].cpu().numpy().astype(np.float64), lse[a:b].cpu().numpy().astype(np.float64), (ro, rl, w, rs))
            score64[s, :, :lens[s]] += w
            lens[s] = kv_ref.evict(pages, table[s], int(lens[s]), int(seen[s]), score64[s], pos[s], budget, recent)
        assert glens[nxt].cpu().tolist() == lens.tolist()
        assert np.array_equal(gpos.cpu().numpy(), pos)
        assert np.array_equal(gp.cpu().numpy(), pages)
        for s in range(n):
            d = np.abs(got[s, :, :lens[s]] - score64[s, :, :lens[s]])
            assert (d <= 1e-4 * score64[s, :, :lens[s]] + 1e-6).all()


def test_graph_replays_follow_the_lengths():
    """A captured step is replayed while lens and seen advance on the device."""
    c = Case(62, 128, 8, 2, [150, 61], [1, 1], state=True)
    q = torch.zeros((2, 8, 128), dtype=torch.float16, device=DEV)
    k = torch.zeros((2, 2, 128), dtype=torch.float16, device=DEV)
    out = torch.zeros_like(q)
    lse = torch.zeros((2, 8), device=DEV)
    lens = c.g["lens"]

    def step():
        moeq4.moe_kv_append_q4(c.kv, c.cache, c.batch, k, k)
        moeq4.moe_attn_q4(c.kv, c.cache, c.batch, q, out, lse=lse, scale=0.09, weights=True)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    c.upload()
    lens = c.g["lens"]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    score = c.score.astype(np.float64)
    for n in ([150, 61], [170, 64], [190, 65]):
        c.lens[:] = n
        lens.copy_(cu(c.lens))
        qn, kn = c.queries(), c.rng.standard_normal((2, 2, 128)).astype(np.float16)
        q.copy_(cu(qn))
        k.copy_(cu(kn))
        graph.replay()
        for s in range(2):
            kv_ref.append(c.pages, c.table[s], n[s] - 1, kn[s], kn[s])
            score[s, :, n[s] - 1] = 0
        ref = c.reference(qn, 0.09)
        score += ref[2]
        close(out.cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64), ref)
        got = c.g["score"].cpu().numpy()
        assert (np.abs(got - score) <= 1e-4 * score + 1e-6).all()
    moeq4.moe_kv_check(c.kv)


def test_another_stream():
    c = Case(63, 128, 8, 2, [5000, 61], [1, 1])
    q = c.queries()
    st = torch.cuda.Stream()
    gq = cu(q)
    out = torch.zeros((2, 8, 128), dtype=torch.float16, device=DEV)
    lse = torch.zeros((2, 8), device=DEV)
    st.wait_stream(torch.cuda.current_stream())
    moeq4.moe_attn_q4(c.kv, c.cache, c.batch, gq, out, lse=lse, scale=0.09, stream=st)
    moeq4.moe_kv_check(c.kv, st)
    close(out.cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64), c.reference(q, 0.09))


@pytest.mark.parametrize("seed", range(3))
def test_many_ragged_sequences(seed):
    """Sequences of few and of many rows in one call, and a larger max_q than any has."""
    rng = np.random.default_rng(100 + seed)
    n = [45, 70, 33][seed]
    rows = [int(x) for x in rng.choice([0, 1, 2, 5, 17, 40, 150], n)]
    lens = [int(r + x) for r, x in zip(rows, rng.integers(0, 400, n))]
    D, Hq, Hkv = [(64, 6, 2), (128, 4, 2), (192, 3, 1)][seed]
    c = Case(66 + seed, D, Hq, Hkv, lens, rows, spare_rows=7, state=True)
    q = c.queries()
    ref = c.reference(q, 0.1, 90)
    c.batch = moeq4.KvBatch(c.kv, c.g["start"], c.n_rows, c.n_rows)
    out, lse = c.attend(q, 0.1, 90, weights=True)
    close(out, lse, ref, int(c.start[-1]))
    want = c.score.astype(np.float64) + ref[2]
    got = c.g["score"].cpu().numpy().astype(np.float64)
    assert (np.abs(got - want) <= 1e-4 * ref[2] + 2.0 ** -23 * np.abs(want) + 1e-6).all()


@pytest.mark.parametrize("D,Hq,Hkv,lens,rows", [(128, 8, 2, [700, 300], [1, 1]), (128, 8, 2, [300, 129], [40, 33]),
                                                (256, 4, 2, [200, 64], [50, 3])])
def test_calls_behind_one_another_see_what_was_written(D, Hq, Hkv, lens, rows):
    """Appends and attentions in one graph, launches overlapping, nothing between
    them: each attention sees the rows just written, also where an earlier one
    has read the same entries."""
    c = Case(73, D, Hq, Hkv, lens, rows, state=True)
    m, n = 12, c.n_rows
    k, v = (c.rng.standard_normal((2, m, n, Hkv, D)) * 1.2).astype(np.float16)
    k, v, q = cu(k), cu(v), cu(c.queries())

    def outputs():
        return torch.zeros((m, n, Hq, D), dtype=torch.float16, device=DEV), torch.zeros((m, n, Hq), device=DEV)

    def step(i, out, lse):
        moeq4.moe_kv_append_q4(c.kv, c.cache, c.batch, k[i], v[i])
        moeq4.moe_attn_q4(c.kv, c.cache, c.batch, q, out[i], lse=lse[i], scale=0.09, weights=True)

    alone, got = outputs(), outputs()
    score = c.g["score"].clone()
    for i in range(m):
        step(i, *alone)
        torch.cuda.synchronize()
    after = c.g["score"].clone()
    assert not torch.equal(alone[0][0], alone[0][1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for i in range(m):
            step(i, *got)
    for _ in range(20):
        c.g["score"].copy_(score)
        got[0].zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got[0], alone[0]) and torch.equal(got[1], alone[1]) and torch.equal(c.g["score"], after)
    moeq4.moe_kv_check(c.kv)


def test_two_contexts_on_two_streams():
    """Calls of two contexts at once give what each gives alone."""
    cs = [Case(67, 128, 8, 2, [3000, 700], [1, 60], state=True), Case(68, 128, 16, 4, [900, 2000], [150, 1], state=True)]
    qs = [cu(c.queries()) for c in cs]
    alone, outs, scores = [], [], []
    for c, q in zip(cs, qs):
        out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device=DEV)
        moeq4.moe_attn_q4(c.kv, c.cache, c.batch, q, out, lse=lse, scale=0.09, weights=True)
        alone.append((out, lse, c.g["score"].clone()))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for rep in range(8):
        for c, q, st in zip(cs, qs, streams):
            with torch.cuda.stream(st):
                c.g["score"].copy_(cu(c.score))
                out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device=DEV)
                moeq4.moe_attn_q4(c.kv, c.cache, c.batch, q, out, lse=lse, scale=0.09, weights=True)
                outs.append((out, lse))
                scores.append(c.g["score"].clone())
    torch.cuda.synchronize()
    for i, (out, lse) in enumerate(outs):
        want = alone[i % 2]
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1]) and torch.equal(scores[i], want[2])


def test_first_call_captured():
    """A fresh context's first calls are captured, with many rows and an eviction, and
    replayed on new contents."""
    c = Case(69, 128, 8, 2, [700, 400], [100, 60], state=True)
    e = Case(69, 128, 8, 2, [700, 400], [100, 60], state=True)      # the same, for eager calls
    k, v = torch.randn((2, 160, 2, 128), dtype=torch.float16, device=DEV)
    q = cu(c.queries())

    def step(x, out, lse, new):
        moeq4.moe_kv_append_q4(x.kv, x.cache, x.batch, k, v)
        moeq4.moe_attn_q4(x.kv, x.cache, x.batch, q, out, lse=lse, scale=0.09, weights=True)
        moeq4.moe_kv_evict(x.kv, x.cache, 2, 350, 20, new)

    def outputs():
        return torch.zeros_like(q), torch.zeros((160, 8), device=DEV), torch.zeros(2, dtype=torch.int32, device=DEV)

    got, want = outputs(), outputs()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(c, *got)
    for rep in range(3):
        k.mul_(-1.5)
        q.neg_()
        graph.replay()
        step(e, *want)
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
        for name in ("pages", "score", "pos"):
            assert torch.equal(c.g[name].view(torch.uint8), e.g[name].view(torch.uint8)), name
    moeq4.moe_kv_check(c.kv)


def test_bounded_wait_gives_up_and_context_recovers():
    """With a bound of 1 us the tile kernel's waits run out before the first page has
    been converted: it leaves, the check tells once, and the next call is right."""
    c = Case(78, 128, 16, 4, [3000, 2000], [128, 100], state=True)
    q = c.queries()
    ref = c.reference(q, 0.09)
    refused(moeq4.MOE_ERR_INVALID_ARG, moeq4.moe_kv_set_wait_ns, c.kv, 999)
    refused(moeq4.MOE_ERR_INVALID_ARG, moeq4.moe_kv_set_wait_ns, c.kv, 60_000_000_001)
    moeq4.moe_kv_set_wait_ns(c.kv, 1000)
    out = torch.zeros((c.n_rows, 16, 128), dtype=torch.float16, device=DEV)
    moeq4.moe_attn_q4(c.kv, c.cache, c.batch, cu(q), out, scale=0.09)
    refused(moeq4.MOE_ERR_TIMEOUT, moeq4.moe_kv_check, c.kv)
    moeq4.moe_kv_check(c.kv)                                     # reported once
    moeq4.moe_kv_set_wait_ns(c.kv, 2_000_000_000)
    out, lse = c.attend(q, 0.09, weights=True)
    close(out, lse, ref)


def test_queries_and_outputs_in_the_same_rows():
    c = Case(70, 128, 8, 2, [300, 90], [1, 40])
    q = c.queries()
    both = torch.full((41, 16, 128), 7.0, dtype=torch.float16, device=DEV)
    both[:, 8:] = cu(q)
    lse = torch.empty((41, 8), device=DEV)
    moeq4.moe_attn_q4(c.kv, c.cache, c.batch, both[:, 8:], both[:, :8], lse=lse, scale=0.09)
    close(both[:, :8].cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64), c.reference(q, 0.09))
    assert np.array_equal(both[:, 8:].cpu().numpy(), q)


def test_nothing_to_do():
    c = Case(64, 64, 2, 1, [10], [1])
    q = torch.zeros((0, 2, 64), dtype=torch.float16, device=DEV)
    k = torch.zeros((0, 1, 64), dtype=torch.float16, device=DEV)
    b = moeq4.KvBatch(c.kv, cu(np.zeros(2, np.int32)), 0, 1)
    moeq4.moe_attn_q4(c.kv, c.cache, b, q, q.clone())
    moeq4.moe_kv_append_q4(c.kv, c.cache, b, k, k)
    b = moeq4.KvBatch(c.kv, cu(np.zeros(1, np.int32)), 1, 1)
    q = torch.zeros((1, 2, 64), dtype=torch.float16, device=DEV)
    out = torch.full_like(q, 7)
    moeq4.moe_attn_q4(c.kv, c.cache, b, q, out)
    moeq4.moe_kv_check(c.kv)
    assert (out == 7).all() and np.array_equal(c.g["pages"].cpu().numpy(), c.pages)


# --------------------------------------------------------------- refusals --
def refused(code, f, *a, **kw):
    with pytest.raises(moeq4.MoeError) as ei:
        f(*a, **kw)
    assert ei.value.code == code, ei.value
    assert str(ei.value)


def test_refusals():
    c = Case(71, 128, 8, 2, [100, 50], [1, 2], state=True)
    inv, ali, shp = moeq4.MOE_ERR_INVALID_ARG, moeq4.MOE_ERR_ALIGNMENT, moeq4.MOE_ERR_UNSUPPORTED_SHAPE
    q, out = torch.zeros((2, 3, 8, 128), dtype=torch.float16, device=DEV)
    k = torch.zeros((3, 2, 128), dtype=torch.float16, device=DEV)
    att = moeq4.moe_attn_q4
    refused(inv, att, c.kv, c.cache, c.batch, q[:2], out)                       # too few rows
    refused(inv, att, c.kv, c.cache, c.batch, q[:, :4], out)                    # too few heads
    refused(inv, att, c.kv, c.cache, c.batch, q.float(), out)
    refused(inv, att, c.kv, c.cache, c.batch, q.transpose(0, 1), out)
    refused(inv, att, c.kv, c.cache, c.batch, q, out, window=-1)
    refused(inv, att, c.kv, c.cache, c.batch, q, out, scale=math.nan)
    refused(inv, att, c.kv, c.cache, c.batch, q, out, scale=math.inf)
    refused(inv, att, c.kv, c.cache, c.batch, q, out, lse=torch.zeros(3, device=DEV))
    odd = torch.zeros(3 * 8 * 128 + 8, dtype=torch.float16, device=DEV)[1:1 + 3 * 8 * 128].view(3, 8, 128)
    refused(ali, att, c.kv, c.cache, c.batch, odd, out)
    gap = torch.zeros((3, 8 * 128 + 4), dtype=torch.float16, device=DEV)[:, :1024].view(3, 8, 128)
    refused(inv, att, c.kv, c.cache, c.batch, gap, out)                         # stride not a multiple of 8
    refused(inv, moeq4.KvBatch, c.kv, c.g["start"].long(), 3, 2)
    refused(shp, att, c.kv, c.cache, moeq4.KvBatch(c.kv, c.g["start"], 4, 2),
            torch.zeros((4, 8, 128), dtype=torch.float16, device=DEV), torch.zeros((4, 8, 128), dtype=torch.float16, device=DEV))
    refused(inv, att, c.kv, c.cache, moeq4.KvBatch(c.kv, c.g["start"], 3, 0), q, out)
    refused(inv, att, c.kv, c.cache, c.batch, q, q)                             # in place
    flat = torch.zeros((3, 12, 128), dtype=torch.float16, device=DEV)
    refused(inv, att, c.kv, c.cache, c.batch, flat[:, :8], flat[:, 4:])         # columns that overlap
    refused(inv, moeq4.moe_kv_read_q4, c.kv, c.cache, c.batch, k, k)
    refused(inv, att, c.kv, c.cache, c.batch, q.cpu(), out)
    refused(inv, att, c.kv, c.cache, c.batch, q, out.cpu())
    refused(inv, moeq4.moe_kv_append_q4, c.kv, c.cache, c.batch, k, k.cpu())
    refused(inv, moeq4.KvBatch, c.kv, c.g["start"].cpu(), 3, 2)
    refused(inv, moeq4.KvCache, c.kv, c.g["pages"].cpu(), c.g["table"], c.g["lens"])
    other = Case(71, 128, 8, 2, [100, 50], [1, 2], max_pages=9)
    refused(inv, att, c.kv, other.cache, c.batch, q, out)                       # pages of another layout
    bare = moeq4.KvCache(c.kv, c.g["pages"], c.g["table"], c.g["lens"])
    refused(inv, att, c.kv, bare, c.batch, q, out, weights=True)
    refused(inv, moeq4.KvCache, c.kv, c.g["pages"][1:], c.g["table"], c.g["lens"])
    refused(inv, moeq4.KvCache, c.kv, c.g["pages"], c.g["table"][:1], c.g["lens"])
    refused(inv, moeq4.KvCache, c.kv, c.g["pages"], c.g["table"], c.g["lens"], score=c.g["score"][:1])
    big = moeq4.KvBatch(c.kv, cu(np.zeros(4, np.int32)), 3, 1)
    refused(inv, att, c.kv, c.cache, big, q, out)                               # more sequences than the cache has
    nopos = moeq4.KvCache(c.kv, c.g["pages"], c.g["table"], c.g["lens"], pos=c.g["pos"])
    refused(inv, moeq4.moe_kv_append_q4, c.kv, nopos, c.batch, k, k)            # pos without seen
    new = torch.zeros(2, dtype=torch.int32, device=DEV)
    ev = moeq4.moe_kv_evict
    refused(inv, ev, c.kv, c.cache, 2, 0, 0, new)
    refused(inv, ev, c.kv, c.cache, 2, 10, 11, new)
    refused(inv, ev, c.kv, c.cache, 2, 10, -1, new)
    refused(inv, ev, c.kv, c.cache, 2, 10, 1, c.g["lens"])
    refused(inv, ev, c.kv, c.cache, 2, 10, 1, new[:1])
    refused(inv, ev, c.kv, bare, 2, 10, 1, new)
    refused(shp, ev, c.kv, c.cache, -1, 10, 1, new)
    huge = moeq4.Kv(KvConfig(2, 1, 64, 1, 8193))
    cap = 8193 * 64
    hc = moeq4.KvCache(huge, torch.zeros(4608, dtype=torch.uint8, device=DEV),
                       torch.zeros((1, 8193), dtype=torch.int32, device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV),
                       score=torch.zeros(cap, device=DEV), pos=torch.zeros(cap, dtype=torch.int32, device=DEV),
                       seen=torch.zeros(1, dtype=torch.int32, device=DEV))
    refused(shp, ev, huge, hc, 1, 10, 1, new)
    moeq4.moe_kv_check(c.kv)


def test_evict_refuses_new_lens_over_what_it_reads():
    c = Case(79, 128, 4, 2, [100, 50], [1, 1], state=True)
    for name in ("seen", "table", "score", "pos"):
        over = c.g[name].view(torch.int32).view(-1)
        for part in (over[:2], over[-2:]):
            refused(moeq4.MOE_ERR_INVALID_ARG, moeq4.moe_kv_evict, c.kv, c.cache, 2, 10, 1, part)
    for name in ("seen", "table", "score", "pos", "pages"):
        assert np.array_equal(c.g[name].cpu().numpy(), getattr(c, name))


@pytest.mark.parametrize("rows", [[1, 2], [40, 70]])
@pytest.mark.parametrize("what", ["page", "negative page", "start", "start past rows", "max_q", "long", "negative len"])
def test_bad_device_values_are_reported_and_skipped(what, rows):
    """The kernels check what they read: nothing outside the pool is touched, the
    other sequence is served, and moe_kv_check tells."""
    c = Case(72, 128, 8, 2, [300, 190], rows, spare_rows=3, state=True)
    q = c.queries()
    ref = c.reference(q, 0.09)
    k = torch.zeros((c.n_rows, 2, 128), dtype=torch.float16, device=DEV)
    n0 = rows[0]
    batch = c.batch
    if what == "page":
        c.g["table"][1, 2] = c.n_pages
    elif what == "negative page":
        c.g["table"][1, 0] = -1
    elif what == "start":
        c.g["start"][2] = n0 - 1
    elif what == "start past rows":
        c.g["start"][2] = c.n_rows + 1
    elif what == "max_q":
        batch = moeq4.KvBatch(c.kv, c.g["start"], c.n_rows, rows[1] - 1)
    elif what == "long":
        c.g["lens"][1] = c.cap + 1
    else:
        c.g["lens"][1] = -3
    out = torch.full((c.n_rows, 8, 128), 7.0, dtype=torch.float16, device=DEV)
    lse = torch.full((c.n_rows, 8), 7.0, device=DEV)
    moeq4.moe_attn_q4(c.kv, c.cache, batch, cu(q), out, lse=lse, scale=0.09, weights=True)
    refused(moeq4.MOE_ERR_INVALID_ARG, moeq4.moe_kv_check, c.kv)
    moeq4.moe_kv_check(c.kv)                            # reported once
    if what != "start":                                 # there row n0 - 1 belongs to nobody
        close(out.cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64), ref, n0)
    if what in ("start past rows", "max_q"):
        assert (out[n0:] == 7).all()
    moeq4.moe_kv_append_q4(c.kv, c.cache, batch, k, k)
    if what != "negative page":                         # page 0 of the table: not where the rows go
        refused(moeq4.MOE_ERR_INVALID_ARG, moeq4.moe_kv_check, c.kv)
    moeq4.moe_kv_check(c.kv)
    if what in ("page", "negative page", "long"):
        new = torch.zeros(2, dtype=torch.int32, device=DEV)
        moeq4.moe_kv_evict(c.kv, c.cache, 2, 100, 10, new)
        assert new.cpu().tolist() == [100, 100]
        refused(moeq4.MOE_ERR_INVALID_ARG, moeq4.moe_kv_check, c.kv)
