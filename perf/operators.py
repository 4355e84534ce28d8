"""Measured cases of the operators on a KV cache held in 4 bits: appending rows,
attention of single tokens and of prompt chunks, attention that also accumulates
the weight each cache entry received, and eviction by that weight.

The cache is a pool of pages of 64 entries; a page holds, per kv head, a tile of
4608 * NG bytes (NG = head_dim / 64 groups of 64 columns):
  K codes [NG][64 entries][32 bytes], K scale and bias fp16 [NG][64][2],
  V codes and V scale and bias in the same order;
value = scale * code + bias, column c of a group in nibble c % 8 of its 32-bit
word c / 8.  A sequence's entry j is entry j % 64 of page page_table[s][j / 64].
"""
import math

import torch

own = False

PAGE = 64


# ------------------------------------------------------------------ cases --
def listed():
    return [
        # one decode step's new K/V rows of 64 sequences
        dict(name="append step 64 seqs", op="append", seqs=64, rows=1, ragged=False, hq=32, hkv=8, d=128, lo=500, hi=4000),
        # K/V rows of a batch of prompt chunks
        dict(name="append 16 x 512 rows", op="append", seqs=16, rows=512, ragged=True, hq=32, hkv=8, d=128, lo=600, hi=2000),
        # the first tokens of a single chat: latency is all
        dict(name="attn 1 token of 500", op="attn", seqs=1, rows=1, ragged=False, hq=16, hkv=8, d=128, lo=500, hi=500, window=0, weights=False),
        # a serving batch of ragged lengths
        dict(name="attn 64 tokens to 16384", op="attn", seqs=64, rows=1, ragged=False, hq=32, hkv=8, d=128, lo=300, hi=16384, window=0, weights=False),
        # one very long context
        dict(name="attn 1 token of 131072", op="attn", seqs=1, rows=1, ragged=False, hq=32, hkv=8, d=128, lo=131072, hi=131072, window=0, weights=False),
        # a local (sliding window) layer with wide heads, large batch
        dict(name="attn 64 tokens window 1024", op="attn", seqs=64, rows=1, ragged=False, hq=16, hkv=8, d=256, lo=200, hi=6000, window=1024, weights=False),
        # one prompt chunk of 128 tokens against a 4096-token cache
        dict(name="attn chunk 128 of 4096", op="attn", seqs=1, rows=128, ragged=False, hq=16, hkv=8, d=256, lo=4096, hi=4096, window=0, weights=False),
        # several prompts' chunks together, ragged
        dict(name="attn chunks 4 x 512", op="attn", seqs=4, rows=512, ragged=True, hq=32, hkv=8, d=128, lo=2000, hi=8192, window=0, weights=False),
        # decode step of a bounded cache: the weights feed the eviction
        dict(name="weights 16 tokens to 8192", op="attn", seqs=16, rows=1, ragged=False, hq=32, hkv=8, d=128, lo=2000, hi=8192, window=0, weights=True),
        # prompt chunk of a bounded cache
        dict(name="weights chunk 256 of 2900", op="attn", seqs=1, rows=256, ragged=False, hq=40, hkv=8, d=128, lo=2900, hi=2900, window=0, weights=True),
        # steady decode: 16 entries over the budget
        dict(name="evict 16 of 4112", op="evict", seqs=32, hq=32, hkv=8, d=128, lo=4112, hi=4112, budget=4096, recent=128),
        # a prompt cut to half its length
        dict(name="evict half of 16384", op="evict", seqs=8, hq=32, hkv=8, d=128, lo=12000, hi=16384, budget=8192, recent=512),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    d = rng.choice([64, 128, 128, 192, 256])
    hkv = rng.choice([1, 2, 4, 8, 8])
    hq = hkv * rng.choice([1, 2, 3, 4, 5, 8])
    kind = rng.choice(["append", "append", "token", "token", "token", "chunk", "chunk", "evict"])
    if kind == "append":
        seqs = _log(rng, 1, 64)
        rows = rng.choice([1, _log(rng, 1, 512)])
        rows = max(1, min(rows, 8192 // seqs))
        lo = rows + rng.randint(0, 500)
        return dict(op="append", seqs=seqs, rows=rows, ragged=rng.random() < 0.5, hq=hq, hkv=hkv, d=d,
                    lo=lo, hi=lo + _log(rng, 1, 2000))
    if kind == "evict":
        seqs = _log(rng, 1, 16)
        hi = _log(rng, 100, 12000)
        budget = max(2, int(hi * rng.uniform(0.3, 0.99)))
        return dict(op="evict", seqs=seqs, hq=hq, hkv=hkv, d=d, lo=max(1, hi - rng.randint(0, hi // 2)), hi=hi,
                    budget=budget, recent=rng.randint(0, budget // 2))
    if kind == "token":
        seqs = _log(rng, 1, 48)
        hi = _log(rng, 1, 60000)
        hi = max(1, min(hi, 120000 // seqs))
        rows = 1 if rng.random() < 0.8 else min(hi, rng.randint(2, 6))
        return dict(op="attn", seqs=seqs, rows=rows, ragged=rows > 1, hq=hq, hkv=hkv, d=d,
                    lo=max(rows, int(hi * rng.uniform(0.05, 1.0))), hi=hi,
                    window=rng.choice([0, 0, _log(rng, 16, 4000)]), weights=rng.random() < 0.3)
    seqs = _log(rng, 1, 6)
    rows = _log(rng, 7, 512)
    hi = rows + _log(rng, 1, 6000)
    hi = min(hi, max(rows, 8000 // seqs))
    return dict(op="attn", seqs=seqs, rows=rows, ragged=rng.random() < 0.7, hq=hq, hkv=hkv, d=d,
                lo=rows + int((hi - rows) * rng.random()), hi=hi,
                window=rng.choice([0, 0, _log(rng, 16, 4000)]), weights=rng.random() < 0.3)


def _sizes(case, seed):
    """Lengths (entries held, new rows included) and rows of each sequence."""
    g = torch.Generator().manual_seed(seed % (1 << 40) + 17)
    n = case["seqs"]
    lens = torch.randint(case["lo"], case["hi"] + 1, (n,), generator=g)
    lens[0] = case["hi"]
    rows = torch.full((n,), case.get("rows", 1))
    if case.get("ragged"):
        # the same for every seed: the outputs keep their shape
        rows = torch.randint(1, case["rows"] + 1, (n,), generator=torch.Generator().manual_seed(n + case["hi"]))
        rows[0] = case["rows"]
    return lens, rows


# ----------------------------------------------------------------- inputs --
def _quantise(x):
    """x fp16 [..., 64] -> codes (whole fp32 0..15), scale and bias fp16 [..., 1]."""
    v = x.float()
    lo, hi = v.amin(-1, keepdim=True), v.amax(-1, keepdim=True)
    s, b = ((hi - lo) / 15).half(), lo.half()
    c = torch.round((v - b.float()) / s.float()).clamp(0, 15)
    return torch.where(s == 0, torch.zeros_like(c), c), s, b


def _pack(c):
    """codes [..., 64] -> int32 [..., 8], column c in nibble c % 8 of word c / 8."""
    w = c.to(torch.int64).view(*c.shape[:-1], 8, 8) << (4 * torch.arange(8, device=c.device))
    w = w.sum(-1)
    return torch.where(w >= 1 << 31, w - (1 << 32), w).to(torch.int32)


def _random_pages(n_pages, hkv, ng, gen, dev):
    """Pages of normal K and V values, quantised."""
    words = torch.empty((n_pages, hkv, 2, ng, 576), dtype=torch.int32, device=dev)
    step = max(1, (1 << 25) // (hkv * 2 * ng * 4096))
    for p in range(0, n_pages, step):
        m = min(step, n_pages - p)
        x = torch.randn((m, hkv, 2, ng, PAGE, 64), generator=gen, device=dev, dtype=torch.float16)
        c, s, b = _quantise(x)
        words[p:p + m, ..., :512] = _pack(c).view(m, hkv, 2, ng, 512)
        words[p:p + m, ..., 512:] = torch.cat((s, b), -1).view(torch.int32).view(m, hkv, 2, ng, 64)
    # tile order: codes of every group, then scale and bias of every group
    t = torch.cat((words[..., :512].reshape(n_pages, hkv, 2, ng * 512),
                   words[..., 512:].reshape(n_pages, hkv, 2, ng * 64)), -1)
    return t.reshape(n_pages, hkv, 1152 * ng).contiguous()


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev).manual_seed(seed % (1 << 40) + 1)
    lens, rows = _sizes(case, seed)
    n, hkv, d = case["seqs"], case["hkv"], case["d"]
    hq, ng = case["hq"], case["d"] // 64
    max_pages = -(-int(lens.max()) // PAGE)
    n_pages = n * max_pages
    table = torch.randperm(n_pages, generator=gen, device=dev).to(torch.int32).view(n, max_pages)
    st = dict(case=case, n=n, hq=hq, hkv=hkv, d=d, ng=ng, max_pages=max_pages, n_pages=n_pages,
              max_len=int(lens.max()), table=table, lens=lens.to(dev, torch.int32),
              pages=_random_pages(n_pages, hkv, ng, gen, dev), scale=1 / math.sqrt(d))
    n_rows = int(rows.sum())
    start = torch.zeros(n + 1, dtype=torch.int32)
    start[1:] = rows.cumsum(0)
    st.update(rows=n_rows, max_q=int(rows.max()), start=start.to(dev))
    cap = max_pages * PAGE
    if case["op"] == "append":
        qkv = torch.randn((n_rows, hq + 2 * hkv, d), generator=gen, device=dev, dtype=torch.float16)
        st.update(k=qkv[:, hq:hq + hkv], v=qkv[:, hq + hkv:],
                  k_out=torch.zeros((n_rows, hkv, d), dtype=torch.float16, device=dev),
                  v_out=torch.zeros((n_rows, hkv, d), dtype=torch.float16, device=dev))
    elif case["op"] == "attn":
        # queries that lean towards some keys: logits of a few units, as in a trained model
        q = torch.randn((n_rows, hq, d), generator=gen, device=dev, dtype=torch.float16) * 1.5
        st.update(q=q, out=torch.zeros_like(q), lse=torch.zeros((n_rows, hq), device=dev))
        if case["weights"]:
            st.update(score=torch.rand((n, hkv, cap), generator=gen, device=dev) * 0.1)
    else:
        # accumulated weights: a few entries hold most of it; some entries tie at zero
        w = torch.rand((n, hkv, cap), generator=gen, device=dev)
        score = w ** 8 * 20 * (torch.rand((n, hkv, cap), generator=gen, device=dev) > 0.05)
        pos = torch.arange(cap, dtype=torch.int32, device=dev).expand(n, hkv, cap)
        before = torch.stack((score.view(torch.int32), pos))
        now = before.clone()
        st.update(before=before, now=now, score=now[0].view(torch.float32), pos=now[1],
                  seen=st["lens"].clone(), new_lens=torch.zeros_like(st["lens"]))
    if own:
        from bit_quantized_expert_int8_b200 import moeq4
        st["kv"] = moeq4.Kv(moeq4.KvConfig(n_q_heads=hq, n_kv_heads=hkv, head_dim=d, n_pages=n_pages,
                                           max_pages=max_pages, max_seqs=n, max_rows=n_rows))
        st["cache"] = moeq4.KvCache(st["kv"], st["pages"], table, st["lens"], score=st.get("score"),
                                    pos=st.get("pos"), seen=st.get("seen"))
        st["batch"] = moeq4.KvBatch(st["kv"], st["start"], n_rows, st["max_q"])
    return st


# -------------------------------------------------------------- one pass --
def run(state):
    if state["case"]["op"] == "evict":
        # evicting changes scores and positions in place: every pass begins with the same ones
        state["now"].copy_(state["before"])
    if own:
        return _run_own(state)
    return {"append": _plain_append, "attn": _plain_attn, "evict": _plain_evict}[state["case"]["op"]](state)


def _run_own(st):
    from bit_quantized_expert_int8_b200 import moeq4
    case = st["case"]
    if case["op"] == "append":
        moeq4.moe_kv_append_q4(st["kv"], st["cache"], st["batch"], st["k"], st["v"])
        moeq4.moe_kv_read_q4(st["kv"], st["cache"], st["batch"], st["k_out"], st["v_out"])
        return st["k_out"], st["v_out"]
    if case["op"] == "attn":
        moeq4.moe_attn_q4(st["kv"], st["cache"], st["batch"], st["q"], st["out"], lse=st["lse"],
                          scale=st["scale"], window=case["window"], weights=case["weights"])
        return (st["out"], st["lse"], st["score"]) if case["weights"] else (st["out"], st["lse"])
    moeq4.moe_kv_evict(st["kv"], st["cache"], st["n"], case["budget"], case["recent"], st["new_lens"])
    return st["new_lens"], st["pos"], st["score"], st["pages"]


def _places(st):
    """Sequence, row within it and cache entry of every row."""
    r = torch.arange(st["rows"], device=st["start"].device)
    s = torch.searchsorted(st["start"][1:].contiguous(), r, right=True)
    i = r - st["start"][s]
    n = st["start"][s + 1] - st["start"][s]
    return s, i, st["lens"][s] - n + i


def _plain_append(st):
    pages, ng, hkv = st["pages"], st["ng"], st["hkv"]
    s, _, e = _places(st)
    page, e = st["table"][s, e // PAGE].long(), e % PAGE
    got = []
    for x, base, out in ((st["k"], 0, st["k_out"]), (st["v"], 576 * ng, st["v_out"])):
        c, sc, b = _quantise(x.reshape(st["rows"], hkv, ng, 64))
        sb = torch.cat((sc, b), -1).view(torch.int32)                             # [rows][hkv][ng][1]
        h = torch.arange(hkv, device=x.device).view(1, hkv, 1, 1)
        g = torch.arange(ng, device=x.device).view(1, 1, ng, 1)
        w = torch.arange(8, device=x.device).view(1, 1, 1, 8)
        pg, en = page.view(-1, 1, 1, 1), e.view(-1, 1, 1, 1)
        pages[pg, h, base + g * 512 + en * 8 + w] = _pack(c)
        pages[pg, h, base + 512 * ng + g * 64 + en] = sb
        out.copy_((sc.float() * c + b.float()).half().view(st["rows"], hkv, -1))
        got.append(out)
    return tuple(got)


def _values(st, part):
    """K (part 0) or V (part 1) of every sequence, fp32 [n][hkv][entries][d]."""
    n, hkv, ng, mp = st["n"], st["hkv"], st["ng"], st["max_pages"]
    t = st["pages"][st["table"].long()][..., part * 576 * ng:(part + 1) * 576 * ng]   # [n][mp][hkv][576 ng]
    w = t[..., :512 * ng].reshape(n, mp, hkv, ng, PAGE, 8, 1)
    c = ((w >> (4 * torch.arange(8, dtype=torch.int32, device=w.device))) & 15).float().view(n, mp, hkv, ng, PAGE, 64)
    sb = t[..., 512 * ng:].contiguous().view(torch.float16).view(n, mp, hkv, ng, PAGE, 2).float()
    x = sb[..., :1] * c + sb[..., 1:]
    return x.permute(0, 2, 1, 4, 3, 5).reshape(n, hkv, mp * PAGE, ng * 64)


def _plain_attn(st):
    n, hq, hkv, d, mq = st["n"], st["hq"], st["hkv"], st["d"], st["max_q"]
    grp, window = hq // hkv, st["case"]["window"]
    s, i, _ = _places(st)
    q = torch.zeros((n, mq, hq, d), device=st["q"].device)
    q[s, i] = st["q"].float()
    q = q.view(n, mq, hkv, grp, d).permute(0, 2, 1, 3, 4).reshape(n, hkv, mq * grp, d)
    k = _values(st, 0)
    x = (q @ k.transpose(-1, -2) * st["scale"]).view(n, hkv, mq, grp, -1)
    del k
    count = st["start"][1:] - st["start"][:-1]
    p = (st["lens"] - count).view(-1, 1) + torch.arange(mq, device=q.device)              # entry of each row
    j = torch.arange(x.shape[-1], device=q.device)
    seen = (j <= p[..., None]) & (torch.arange(mq, device=q.device) < count.view(-1, 1))[..., None]
    if window:
        seen &= j > p[..., None] - window
    x = x.masked_fill(~seen[:, None, :, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    x = torch.exp(x - m)
    total = x.sum(-1, keepdim=True)
    x = x / torch.where(total == 0, torch.ones_like(total), total)
    o = (x.view(n, hkv, mq * grp, -1) @ _values(st, 1)).view(n, hkv, mq, grp, d)
    o = o.permute(0, 2, 1, 3, 4).reshape(n, mq, hq, d)
    lse = (m + torch.log(total)).squeeze(-1).permute(0, 2, 1, 3).reshape(n, mq, hq)
    st["out"].copy_(o[s, i].half())
    st["lse"].copy_(lse[s, i])
    if not st["case"]["weights"]:
        return st["out"], st["lse"]
    st["score"] += x.sum((2, 3))
    return st["out"], st["lse"], st["score"]


def _entry_words(st, s, h, j):
    """Places in the flat pool of all words of entries j of (sequence s, kv head h)."""
    ng = st["ng"]
    dev = s.device
    g, w = torch.arange(ng, device=dev).view(-1, 1), torch.arange(8, device=dev)
    codes = (g * 512 + w).reshape(-1)
    sb = (512 * ng + g * 64).reshape(-1)
    first = torch.cat((codes, sb, codes + 576 * ng, sb + 576 * ng))
    step = torch.cat((torch.full_like(codes, 8), torch.ones_like(sb)) * 2)
    tile = (st["table"][s, j // PAGE].long() * st["hkv"] + h) * (1152 * ng)
    return tile[:, None] + first + (j % PAGE)[:, None] * step


def _plain_evict(st):
    n, hkv, budget, recent = st["n"], st["hkv"], st["case"]["budget"], st["case"]["recent"]
    score, pos = st["score"], st["pos"]
    cap = score.shape[-1]
    j = torch.arange(cap, device=score.device)
    ln = st["lens"].view(n, 1, 1)
    held = (j < ln).expand(n, hkv, cap)
    safe = held & (pos >= st["seen"].view(n, 1, 1) - recent)
    key = torch.where(safe, torch.full_like(score, math.inf), torch.where(held, score, torch.full_like(score, -math.inf)))
    order = torch.sort(key, dim=-1, descending=True, stable=True).indices
    rank = torch.empty_like(order).scatter_(-1, order, j.expand(n, hkv, cap))
    keep = held & (rank < budget)
    over = (ln > budget).expand(n, hkv, cap)
    hole = torch.nonzero(over & ~keep & (j < budget))
    move = torch.nonzero(over & keep & (j >= budget))
    s, h, a, b = move[:, 0], move[:, 1], move[:, 2], hole[:, 2]
    flat = st["pages"].view(-1)
    flat[_entry_words(st, s, h, b)] = flat[_entry_words(st, s, h, a)]
    score[s, h, b] = score[s, h, a]
    pos[s, h, b] = pos[s, h, a]
    st["new_lens"].copy_(st["lens"].clamp(max=budget))
    return st["new_lens"], pos, score, st["pages"]


# ------------------------------------------------------------------- work --
def work(case):
    """Bytes: queries or new rows, the cache entries that the rows see (72 bytes a
    kv head and 64 columns; K alone is not read twice for the weights), outputs,
    read and written scores.  Lengths are taken at the middle of the case's range."""
    hkv, hq, d, n = case["hkv"], case["hq"], case["d"], case["seqs"]
    mid = (case["lo"] + case["hi"]) / 2
    entry = hkv * d / 64 * 72
    if case["op"] == "append":
        rows = n * (case["rows"] if not case["ragged"] else (1 + case["rows"]) / 2)
        x = rows * hkv * d * 2 * 2
        return {"bytes": 2 * x + 2 * rows * entry, "flops": rows * hkv * d * 2 * 6}
    if case["op"] == "evict":
        over = max(0.0, mid - case["budget"])
        moved = min(over, over * case["budget"] / mid)
        return {"bytes": n * hkv * (mid * 8 + moved * (2 * d / 64 * 72 + 16)), "flops": n * hkv * mid * 4}
    rows = case["rows"] if not case["ragged"] else (1 + case["rows"]) / 2
    read = min(mid, case["window"] + rows - 1) if case["window"] else mid
    see = min(mid, case["window"]) if case["window"] else max(1.0, mid - (rows - 1) / 2)
    flops = 4 * d * n * rows * hq * see
    size = n * (read * entry + rows * hq * (4 * d + 4))
    if case["weights"]:
        size += n * hkv * read * 8
    return {"bytes": size, "flops": flops}


# ------------------------------------------------- the definition, 64 bits --
def exact(case, seed):
    """The operators' definitions entry by entry in 64 bits, sequence by sequence."""
    st = prepare(case, seed)
    dev, ng, hkv, hq, d = "cuda", st["ng"], st["hkv"], st["hq"], st["d"]
    lens, start = st["lens"].tolist(), st["start"].tolist()
    if case["op"] == "append":
        outs = []
        for x in (st["k"], st["v"]):
            v = x.double().reshape(st["rows"], hkv, ng, 64)
            lo, hi = v.min(-1, keepdim=True).values, v.max(-1, keepdim=True).values
            s, b = ((hi - lo) / 15).half().double(), lo
            outs.append((s * ((v - b) / s).round().clamp(0, 15) + b).view(st["rows"], hkv, d))
        return tuple(outs)
    if case["op"] == "evict":
        score = st["score"].double().cpu()
        where, shift = st["pos"].cpu(), st["seen"].tolist()
        for s in range(st["n"]):
            if lens[s] <= case["budget"]:
                continue
            for h in range(hkv):
                v, p = score[s, h, :lens[s]], where[s, h, :lens[s]]
                free = (p < shift[s] - case["recent"]).nonzero().view(-1)
                lose = free[torch.argsort(-v[free], stable=True)[case["budget"] - (lens[s] - len(free)):]]
                gone = torch.zeros(lens[s], dtype=torch.bool)
                gone[lose] = True
                to = gone[:case["budget"]].nonzero().view(-1)
                fr = (~gone[case["budget"]:]).nonzero().view(-1) + case["budget"]
                score[s, h, to] = score[s, h, fr]
        return None, None, score.to(dev), None
    out = torch.zeros((st["rows"], hq, d), dtype=torch.float64, device=dev)
    lse = torch.zeros((st["rows"], hq), dtype=torch.float64, device=dev)
    score = st["score"].double() if case["weights"] else None
    shifts = torch.arange(0, 32, 4, device=dev, dtype=torch.int32)
    for s in range(st["n"]):
        rows = start[s + 1] - start[s]
        tiles = st["pages"][st["table"][s].long()]
        at = (lens[s] - rows + torch.arange(rows, device=dev)).view(-1, 1)
        j = torch.arange(lens[s], device=dev)
        dark = (j > at) | ((j <= at - case["window"]) if case["window"] else torch.zeros_like(j > at))
        for h in range(hkv):
            kv = []
            for part in (0, 1):
                w = tiles[:, h, part * 576 * ng:]
                cols = []
                for g in range(ng):
                    c = w[:, g * 512:(g + 1) * 512].reshape(-1, 8, 1).bitwise_right_shift(shifts).bitwise_and(15)
                    f = w[:, 512 * ng + 64 * g:512 * ng + 64 * (g + 1)].contiguous().view(torch.float16)
                    f = f.reshape(-1, 2).double()
                    cols.append(f[:, :1] * c.reshape(-1, 64).double() + f[:, 1:])
                kv.append(torch.cat(cols, 1)[:lens[s]])
            for u in range(hq // hkv):
                a = h * (hq // hkv) + u
                x = st["q"][start[s]:start[s + 1], a].double() @ kv[0].T / math.sqrt(d)
                x[dark] = -math.inf
                top = torch.logsumexp(x, 1)
                p = torch.exp(x - top[:, None])
                out[start[s]:start[s + 1], a] = p @ kv[1]
                lse[start[s]:start[s + 1], a] = top
                if score is not None:
                    score[s, h, :lens[s]] += p.sum(0)
    return (out, lse, score) if case["weights"] else (out, lse)
