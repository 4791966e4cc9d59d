"""Chunk attention on the host: refused arguments, and its oracle pinned by the
decode's and by closed forms.  CPU only: no call here launches a kernel."""
import numpy as np
import pytest

import mla_prefill_attention_plan_gb300 as mla
import oracle as O
from mla_prefill_attention_plan_gb300 import build as B
from oracle import chunk_oracle as C


@pytest.fixture(scope="module")
def lib():
    B.build()
    return mla.load()


NAMES = "out lse q iro cl kv pt np ps mp uk uv B H T scale".split()
OK = [16, None, 16, 16, 16, 16, 16, 8, 16, 4, 16, 16, 2, 4, 6, 0.1]


def call(chunk_mask=16, mask_words=1, workspace=256, workspace_bytes=1 << 40, **change):
    a = list(OK)
    for k, v in change.items():
        a[NAMES.index(k)] = v
    return mla.mla_chunk_attention(*a, chunk_mask=chunk_mask, mask_words=mask_words, workspace=workspace,
                                   workspace_bytes=workspace_bytes, stream=1)


@pytest.mark.parametrize("change", [
    dict(out=None), dict(out=8), dict(q=None), dict(q=24), dict(iro=None), dict(cl=None), dict(kv=None), dict(kv=2),
    dict(pt=None), dict(np=0), dict(ps=0), dict(mp=0), dict(uk=None), dict(uk=8), dict(uv=None), dict(uv=4), dict(B=0),
    dict(T=-1), dict(scale=0.0), dict(scale=float("nan")), dict(H=16380), dict(T=1 << 22, H=128),
    dict(np=1 << 20, ps=1 << 11), dict(mask_words=0), dict(mask_words=-1), dict(chunk_mask=None, mask_words=2)])
def test_refusals(lib, change):
    assert call(**change) == mla.MLA_ERR_ARG


def test_other_refusals(lib):
    assert call(H=0) == mla.MLA_ERR_GEOMETRY
    need = mla.mla_chunk_attention_workspace_bytes(2, 4, 6)
    assert call(workspace=None) == mla.MLA_ERR_WORKSPACE
    assert call(workspace=128) == mla.MLA_ERR_WORKSPACE
    assert call(workspace_bytes=need - 1) == mla.MLA_ERR_WORKSPACE
    assert call(T=0, workspace=None) == mla.MLA_OK         # nothing to do
    for bad in ((0, 4, 6), (2, 0, 6), (2, 4, -1)):
        assert mla.mla_chunk_attention_workspace_bytes(*bad) == 0


# ------------------------------------------------------------------ the oracle

def inputs(new, cached, H, page, seed=0):
    rng = np.random.default_rng(seed)
    held = [-(-(n + c) // page) for n, c in zip(new, cached)]
    order, at = rng.permutation(sum(held)), 0
    table = np.full((len(new), max(held)), -1, np.int32)
    for b, k in enumerate(held):
        table[b, :k] = order[at: at + k]
        at += k
    iro = np.concatenate([[0], np.cumsum(new)])
    return dict(q=rng.standard_normal((iro[-1], H, 192)), kv=rng.standard_normal((sum(held) * page, 576)), table=table,
                page_size=page, w_uk=rng.standard_normal((H, 512, 128)) * 512 ** -0.5,
                w_uv=rng.standard_normal((H, 128, 512)) * 512 ** -0.5, iro=iro, cached=cached, scale=192 ** -0.5)


def test_no_workspace_for_sizes_that_are_refused(lib):
    most = (1 << 29) - 1
    for heads, tokens in [(16380, 1), (2, 1 << 28), (16, 1 << 25), (16379, 1 << 30), (1, 1 << 29)]:
        assert mla.mla_chunk_attention_workspace_bytes(1, heads, tokens) == 0
        assert call(H=heads, T=tokens) == mla.MLA_ERR_ARG
    assert mla.mla_chunk_attention_workspace_bytes(1, 1, most) >= most * 3200


def test_causal_oracle_is_the_decode_oracle():
    x = inputs([2, 1, 3], [9, 0, 30], 3, 8)
    out, lse, _ = C.chunk_attention(**x)
    full = C.chunk_attention(**x, mask=[1, 3, 1, 1, 3, 7])
    assert np.array_equal(out, full[0]) and np.array_equal(lse, full[1])
    kv = O.bf16_encode(x["kv"])
    x["kv"] = O.decode(kv, "bf16")
    out, lse, _ = C.chunk_attention(**x)
    ref = O.mla_decode(x["q"], kv.reshape(-1, 8, 576), x["table"], 8, x["w_uk"], x["w_uv"], x["iro"], x["cached"],
                       x["scale"])
    rows = ref[0] if isinstance(ref, tuple) else ref
    for (b, h), (tok, o, l) in rows.items():
        np.testing.assert_allclose(out[tok, h], o, rtol=1e-9, atol=1e-12)
        np.testing.assert_allclose(lse[tok, h], l, rtol=1e-9)


def test_a_tree_is_its_paths():
    """Each node of a tree equals the last token of its path, attended causally."""
    x = inputs([5], [7], 2, 16)
    up = [-1, 0, 0, 2, 1]
    mask = []
    for i, u in enumerate(up):
        mask.append(1 << i | (mask[u] if u >= 0 else 0))
    out, lse, _ = C.chunk_attention(**x, mask=mask)
    for i in range(5):
        path = [m for m in range(5) if mask[i] >> m & 1]
        y = dict(x, q=x["q"][path], iro=np.array([0, len(path)]), kv=x["kv"].copy())
        for k, m in enumerate(path):               # the path's rows, one behind the other
            y["kv"][[x["table"][0, 0] * 16 + 7 + k]] = x["kv"][x["table"][0, 0] * 16 + 7 + m]
        o, l, _ = C.chunk_attention(**y)
        np.testing.assert_allclose(out[i], o[-1], rtol=1e-12)
        np.testing.assert_allclose(lse[i], l[-1], rtol=1e-12)


def test_closed_forms():
    x = inputs([2], [0], 2, 4)
    out, lse, _ = C.chunk_attention(**x, mask=[0, 2])
    assert not out[0].any() and np.isneginf(lse[0]).all()
    c = x["kv"][x["table"][0, 0] * 4 + 1]
    np.testing.assert_allclose(out[1], x["w_uv"] @ c[:512])
    out, lse, _ = C.chunk_attention(**x, mask=[0, 2], sink=[0.25])
    assert not out[0].any() and np.allclose(lse[0], 0.25)


def test_more_sequences_than_32_bits_step_over(lib):
    for B in ((1 << 31) - 65535, (1 << 31) - 1):
        assert call(B=B) == mla.MLA_ERR_ARG and mla.mla_chunk_attention_workspace_bytes(B, 4, 6) == 0
    assert mla.mla_chunk_attention_workspace_bytes((1 << 31) - 65536, 4, 6) > 0
