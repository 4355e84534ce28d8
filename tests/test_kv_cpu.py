"""4-bit KV cache, host side: sizes, refusals that need no GPU, and pins of the
64-bit reference that the GPU tests compare with."""
import ctypes
import os
import re
import types

import numpy as np
import pytest
import torch

import kv_ref
from bit_quantized_expert_int8_b200 import build, moeq4
from bit_quantized_expert_int8_b200.config import KvConfig

GOOD = dict(n_q_heads=8, n_kv_heads=2, head_dim=128, n_pages=4, max_pages=2, max_seqs=2, max_rows=4)


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return moeq4.load()


def test_page_bytes():
    for hkv in (1, 3, 8):
        for d in (64, 128, 192, 256):
            # K and V: half a byte a column and 4 bytes a group of 64, 64 entries
            assert moeq4.kv_page_bytes(hkv, d) == hkv * 2 * 64 * (d // 2 + 4 * (d // 64))
            assert moeq4.kv_page_bytes(hkv, d) == hkv * kv_ref.tile_bytes(d)
    for hkv, d in ((0, 64), (129, 64), (1, 32), (1, 320), (1, 100)):
        assert moeq4.kv_page_bytes(hkv, d) == 0


def test_struct_sizes_match_the_c_layout():
    assert ctypes.sizeof(moeq4.CMoeKvConfig) == 32
    assert ctypes.sizeof(moeq4.CMoeKvCache) == 48
    assert ctypes.sizeof(moeq4.CMoeKvBatch) == 24


@pytest.mark.parametrize("bad", [
    dict(head_dim=96), dict(head_dim=320), dict(head_dim=0), dict(n_q_heads=7), dict(n_q_heads=0),
    dict(n_kv_heads=0), dict(n_kv_heads=129, n_q_heads=129), dict(n_q_heads=1026), dict(n_pages=0),
    dict(max_pages=0), dict(max_pages=32769), dict(max_seqs=0), dict(max_seqs=4097), dict(max_rows=0),
    dict(max_rows=(1 << 20) + 1)])
def test_create_refuses_bad_shapes_without_cuda(bad):
    with pytest.raises(moeq4.MoeError) as ei:
        moeq4.Kv(KvConfig(**{**GOOD, **bad}))
    assert ei.value.code == moeq4.MOE_ERR_UNSUPPORTED_SHAPE
    assert moeq4.last_error()


def test_null_arguments_are_refused():
    lib = moeq4.load()
    assert lib.moe_kv_create(None, None) == moeq4.MOE_ERR_INVALID_ARG
    assert lib.moe_kv_destroy(None) == moeq4.MOE_OK
    assert lib.moe_kv_check(None, None) == moeq4.MOE_ERR_INVALID_ARG
    assert lib.moe_kv_append_q4(None, None, None, None, 0, None, 0, None) == moeq4.MOE_ERR_INVALID_ARG
    assert lib.moe_kv_read_q4(None, None, None, None, 0, None, 0, None) == moeq4.MOE_ERR_INVALID_ARG
    assert lib.moe_attn_q4(None, None, None, None, 0, 1.0, 0, 0, None, 0, None, None) == moeq4.MOE_ERR_INVALID_ARG
    assert lib.moe_kv_evict(None, None, 1, 1, 0, None, None) == moeq4.MOE_ERR_INVALID_ARG


def test_host_tensors_are_refused():
    kv = types.SimpleNamespace(cfg=KvConfig(**GOOD), device=0, handle=None)
    i32 = dict(dtype=torch.int32)
    pages = torch.zeros(4 * moeq4.kv_page_bytes(2, 128), dtype=torch.uint8)
    for f in (lambda: moeq4.KvCache(kv, pages, torch.zeros((2, 2), **i32), torch.zeros(2, **i32)),
              lambda: moeq4.KvBatch(kv, torch.zeros(3, **i32), 2, 1),
              lambda: moeq4._rows(kv, torch.zeros((2, 8, 128), dtype=torch.float16), "q", 2, 8, 128)):
        with pytest.raises(moeq4.MoeError) as ei:
            f()
        assert ei.value.code == moeq4.MOE_ERR_INVALID_ARG and "device" in str(ei.value)


def test_reference_reads_what_it_appends():
    rng = np.random.default_rng(3)
    D, Hkv, n = 128, 2, 70
    pages = rng.integers(0, 256, (3, Hkv, kv_ref.tile_bytes(D)), dtype=np.uint8)
    table = [2, 0]
    k = rng.standard_normal((n, Hkv, D)).astype(np.float16)
    v = rng.standard_normal((n, Hkv, D)).astype(np.float16)
    before = pages[1].copy()
    for j in range(n):
        kv_ref.append(pages, table, j, k[j], v[j])
    assert (pages[1] == before).all()
    K, V = kv_ref.sequence(pages, table, n, Hkv, D)
    for x, X in ((k, K), (v, V)):
        g = x.astype(np.float64).transpose(1, 0, 2).reshape(Hkv, n, 2, 64)
        step = (g.max(-1) - g.min(-1)) / 15
        # half a step, plus the fp16 rounding of the scale over 15 steps and of the fp32 quotient
        room = step * (0.5 + 15 * 2.0 ** -11 + 1e-5)
        assert (np.abs(X.reshape(Hkv, n, 2, 64) - g).max(-1) <= room).all()
    t = pages[table[0]][1]
    assert np.array_equal(kv_ref.entry(t, D, 0, 5), K[1, 5]) and np.array_equal(kv_ref.entry(t, D, 1, 63), V[1, 63])


def test_reference_quantiser_by_hand():
    x = np.zeros((3, 64), np.float16)
    x[0] = np.arange(64) % 16                        # min 0, max 15: scale 1, codes 0..15
    x[1] = 2.5                                       # constant: scale 0, codes 0, bias 2.5
    x[2, 7] = np.inf
    c, sb = kv_ref.quantise(x)
    assert c[0, 0] == 0x10 and c[0, 7] == 0xFE
    assert sb[0].view(np.float16).tolist() == [1.0, 0.0]
    assert not c[1].any() and sb[1].view(np.float16).tolist() == [0.0, 2.5]
    assert not c[2].any() and np.isnan(sb[2].view(np.float16)).all()


def test_reference_attention_closed_forms():
    K = np.zeros((1, 5, 64))
    V = np.arange(5.0)[None, :, None] * np.ones(64)
    q = np.ones((2, 2, 64))
    out, lse, got = kv_ref.attention(q, K, V, 0.125, 0, 5)      # equal scores: means
    assert np.allclose(out[0], 1.5) and np.allclose(out[1], 2.0)
    assert np.allclose(lse[1], np.log(5)) and np.allclose(got.sum(), 4)
    out, lse, got = kv_ref.attention(q, K, V, 0.125, 2, 5)      # two entries each
    assert np.allclose(out[0], 2.5) and np.allclose(out[1], 3.5) and got[0, 0] == 0
    out, lse, got = kv_ref.attention(q, K, V, 0.125, 0, 1)      # the first row stands before entry 0
    assert not out[0].any() and np.isneginf(lse[0]).all() and np.allclose(out[1], 0.0) and np.allclose(lse[1], 0.0)


def test_reference_eviction_by_hand():
    D, Hkv, n = 64, 1, 6
    pages = np.zeros((1, Hkv, kv_ref.tile_bytes(D)), np.uint8)
    rows = np.arange(n, dtype=np.float16)[:, None, None] * np.ones((1, Hkv, D), np.float16)
    for j in range(n):
        kv_ref.append(pages, [0], j, rows[j], rows[j])
    score = np.zeros((1, 64), np.float32)
    score[0, :n] = [5, 0, 3, 0, 1, 0]
    pos = np.arange(64, dtype=np.int32)[None].copy()
    # entry 5 is recent; 0, 2, 4 by score; 1, 3 leave.  4 and 5 move into 1 and 3
    assert kv_ref.evict(pages, [0], n, 6, score, pos, 4, 1) == 4
    assert pos[0, :6].tolist() == [0, 4, 2, 5, 4, 5]
    assert score[0, :4].tolist() == [5, 1, 3, 0]
    assert [kv_ref.entry(pages[0, 0], D, 1, e)[0] for e in range(6)] == [0, 4, 2, 5, 4, 5]


def test_kernels_read_memory_coherently():
    """Every kernel of the KV cache may be resident while the work before it runs:
    none reads global memory through the read-only path (whose loads are not
    ordered behind the wait), by name or by const __restrict__."""
    for path in build.sources():
        if os.path.basename(path).startswith("kv_"):
            with open(path) as f:
                text = re.sub(r"//.*", "", f.read())
            assert not re.search(r"__ldg|\.nc\b|const[^;(),]*\*\s*__restrict__", text), path
