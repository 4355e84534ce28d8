"""Both halves of a decode step behind one another: rows appended to the 4-bit KV
cache, attention over it, and the MoE layer on what attention gives, several layers
in a row with nothing between their kernels.  Each half is compared with its own
reference on the inputs it got; the captured run gives the same bits.
"""
import math

import numpy as np
import pytest
import torch

import kv_ref
import oracle
from bit_quantized_expert_int8_b200 import build, moeq4
from bit_quantized_expert_int8_b200.config import TINY, KvConfig
from gpu_util import assert_half_close, make_layer, np_layer, np_of
from test_gpu_kv import close, cu

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    moeq4.load()


@pytest.mark.parametrize("D,Hkv,rows,lens", [
    (128, 1, [1], [300]),                                # the fused layer kernel
    (64, 4, [1, 1, 1], [100, 1, 257]),                   # a batch of tokens
    (64, 2, [40, 1], [90, 200]),                         # a prompt chunk and a token: both attention kernels
])
def test_attention_and_moe_layers_in_one_step(D, Hkv, rows, lens):
    cfg, n_layers = TINY, 4
    Hq, n, T = cfg.H // D, len(rows), sum(rows)
    rng = np.random.default_rng(D + T)
    L = [make_layer(cfg, seed=50, layer=i, bias_std=1.5) for i in range(n_layers)]
    moe_layers = [moeq4.Layer.from_dict(x) for x in L]
    ctx = moeq4.Context(cfg, T)
    mp = -(-max(lens) // 64)
    kv = moeq4.Kv(KvConfig(Hq, Hkv, D, n * mp, mp, n, T))
    start = np.concatenate(([0], np.cumsum(rows))).astype(np.int32)
    batch = moeq4.KvBatch(kv, cu(start), T, max(rows))
    table = rng.permutation(n * mp).reshape(n, mp).astype(np.int32)
    pages = []                                           # one pool a layer, filled up to the new rows
    for i in range(n_layers):
        p = np.zeros((n * mp, Hkv, kv_ref.tile_bytes(D)), np.uint8)
        for s in range(n):
            for j in range(lens[s] - rows[s]):
                kv_ref.append(p, table[s], j, *rng.standard_normal((2, Hkv, D)).astype(np.float16))
        pages.append(p)
    pools = [cu(p) for p in pages]
    caches = [moeq4.KvCache(kv, p, cu(table), cu(np.array(lens, np.int32))) for p in pools]
    k, v = rng.standard_normal((2, n_layers, T, Hkv, D)).astype(np.float16)
    gk, gv = cu(k), cu(v)
    h0 = rng.standard_normal((T, cfg.H)).astype(np.float16)
    scale = 1 / math.sqrt(D)
    y = torch.empty((T, cfg.H), device=DEV)

    def buffers():
        return (torch.zeros((n_layers + 1, T, cfg.H), dtype=torch.float16, device=DEV),
                torch.zeros((n_layers, T, Hq), device=DEV))

    def attend(i, h, lse):                               # h[i] are the queries, h[i + 1] attention's output
        moeq4.moe_kv_append_q4(kv, caches[i], batch, gk[i], gv[i])
        moeq4.moe_attn_q4(kv, caches[i], batch, h[i].view(T, Hq, D), h[i + 1].view(T, Hq, D), lse=lse[i], scale=scale)

    def experts(i, h):                                   # in place: h + MoE(norm(h))
        moeq4.moe_layer_decode(ctx, moe_layers[i], h[i + 1], T, y, flags=moeq4.MOE_PRENORM)

    h, lse = buffers()
    h[0].copy_(cu(h0))
    for i in range(n_layers):
        torch.cuda.synchronize()
        attend(i, h, lse)
        torch.cuda.synchronize()
        q, out = h[i].cpu().numpy().reshape(T, Hq, D), h[i + 1].cpu().numpy()
        ref = [np.zeros((T, Hq, D)), np.zeros((T, Hq)), None, np.zeros((T, Hq, D))]
        for s in range(n):
            a, b = start[s], start[s + 1]
            for r in range(rows[s]):
                kv_ref.append(pages[i], table[s], lens[s] - rows[s] + r, k[i, a + r], v[i, a + r])
            K, V = kv_ref.sequence(pages[i], table[s], lens[s], Hkv, D)
            few = rows[s] * Hq // Hkv <= 64
            U = kv_ref.value_spread(pages[i], table[s], V, D) if few else np.abs(V)
            x = q[a:b].astype(np.float64)
            ref[0][a:b], ref[1][a:b], _ = kv_ref.attention(x, K, V, scale, 0, lens[s])
            ref[3][a:b] = kv_ref.attention(x, K, U, scale, 0, lens[s])[0]
        close(out.reshape(T, Hq, D).astype(np.float64), lse[i].cpu().numpy().astype(np.float64), ref)
        assert np.array_equal(pools[i].cpu().numpy(), pages[i])
        experts(i, h)
        torch.cuda.synchronize()
        Ln = np_layer(L[i])
        for t in range(T):
            x = out[t].view(np.uint16)
            want = oracle.moe_layer(cfg, Ln, oracle.rmsnorm(x, cfg.rms_eps))["y"]
            assert_half_close(np_of(h[i + 1])[t], oracle.residual_add(x, want), f"layer {i}, token {t}")
    moeq4.moe_kv_check(kv)
    moeq4.moe_ctx_check(ctx)

    again, lse2 = buffers()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for i in range(n_layers):
            attend(i, again, lse2)
            experts(i, again)
    for _ in range(5):
        again.zero_()
        again[0].copy_(cu(h0))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(again, h) and torch.equal(lse2, lse)
    moeq4.moe_kv_check(kv)
    moeq4.moe_ctx_check(ctx)
    ctx.close()
