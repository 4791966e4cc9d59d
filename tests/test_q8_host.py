"""The 8-bit cache and key selection on the host: refused arguments, and the
float64 oracle pinned by closed forms and invariants.  CPU only: no call here
launches a kernel."""
import math

import numpy as np
import pytest
import torch

import mla_prefill_attention_plan_gb300 as mla
import oracle as O
from mla_prefill_attention_plan_gb300 import build as B
from oracle import q8


@pytest.fixture(scope="module")
def lib():
    B.build()
    return mla.load()


def _caller(fn, names, ok, **kw):
    def call(**change):
        a = list(ok)
        for k, v in change.items():
            a[names.index(k)] = v
        return fn(*a, stream=1, **kw)   # any non-null handle: these calls fail before using it
    return call


WRITE = ["kv", "sc", "q", "lat", "gamma", "freqs", "iro", "cl", "pt", "np", "ps", "mp", "sb", "B", "H", "T", "L", "eps"]


@pytest.mark.parametrize("change", [
    dict(kv=None), dict(kv=24), dict(sc=None), dict(q=8), dict(lat=None), dict(gamma=20), dict(freqs=None),
    dict(iro=None), dict(cl=None), dict(pt=None), dict(np=0), dict(ps=0), dict(mp=0), dict(sb=0), dict(sb=3),
    dict(sb=256), dict(B=0), dict(H=0), dict(T=-1), dict(L=0), dict(eps=-1.0), dict(eps=float("nan"))])
def test_write_refusals(lib, change):
    ok = [16, 16, 16, 16, 16, 16, 16, 16, 16, 1, 256, 1, 64, 1, 1, 1, 8, 1e-6]
    assert _caller(mla.mla_latent_cache_write_q8, WRITE, ok)(**change) == mla.MLA_ERR_ARG


GATHER = ["ckv", "kr", "kv", "sc", "pt", "np", "ps", "mp", "sb", "bro", "co", "bl", "chunk", "B", "S"]


@pytest.mark.parametrize("change", [
    dict(ckv=None), dict(ckv=8), dict(kr=None), dict(kv=17), dict(sc=None), dict(pt=None), dict(np=0), dict(ps=0),
    dict(mp=0), dict(sb=5), dict(sb=-1), dict(bro=None), dict(co=None), dict(bl=None), dict(chunk=-1), dict(B=0),
    dict(S=0), dict(S=1 << 31)])
def test_gather_refusals(lib, change):
    ok = [16, 16, 16, 16, 16, 1, 16, 1, 4, 16, 16, 16, 0, 1, 8]
    assert _caller(mla.mla_gather_latent_q8, GATHER, ok)(**change) == mla.MLA_ERR_ARG


PREFILL = ["out", "lse", "q", "iro", "cl", "kv", "sc", "pt", "np", "ps", "mp", "sb", "wk", "wuv", "B", "H", "T", "mpl",
           "S", "mc", "scale"]


def test_prefill_refusals(lib):
    ok = [16, None, 16, 16, 16, 16, 16, 16, 1, 16, 1, 4, 16, 16, 1, 4, 8, 8, 32, 1, 0.1]
    call = _caller(mla.mla_prefill_q8, PREFILL, ok, workspace=256, workspace_bytes=16)
    assert call(H=0) == mla.MLA_ERR_GEOMETRY
    for change in (dict(sc=None), dict(sb=3), dict(sb=0), dict(ps=0), dict(kv=8), dict(q=None), dict(S=0), dict(mc=0)):
        assert call(**change) == mla.MLA_ERR_ARG
    assert call() == mla.MLA_ERR_WORKSPACE          # too small


DECODE = ["out", "lse", "q", "iro", "cl", "kv", "sc", "pt", "np", "ps", "mp", "sb", "wuk", "wuv", "B", "H", "T", "mn",
          "L", "parts", "scale"]


def test_decode_refusals(lib):
    ok = [16, None, 16, 16, 16, 16, 16, 16, 1, 16, 1, 4, 16, 16, 1, 4, 1, 1, 8, 1, 0.1]
    call = _caller(mla.mla_decode_q8, DECODE, ok, workspace=256, workspace_bytes=16)
    assert call(H=0) == mla.MLA_ERR_GEOMETRY
    for change in (dict(out=None), dict(out=8), dict(q=4), dict(iro=None), dict(cl=None), dict(kv=None), dict(sc=None),
                   dict(pt=None), dict(np=0), dict(ps=0), dict(mp=0), dict(sb=3), dict(sb=0), dict(wuk=8),
                   dict(wuv=None), dict(B=0), dict(T=-1), dict(mn=-1), dict(L=0), dict(parts=-1), dict(scale=0.0),
                   dict(scale=float("nan")), dict(H=16384), dict(np=1 << 30), dict(T=1 << 28),
                   dict(parts=(1 << 15) + 1)):
        assert call(**change) == mla.MLA_ERR_ARG, change
    assert call() == mla.MLA_ERR_WORKSPACE
    assert call(T=0) == mla.MLA_OK                   # nothing to do
    need = mla.mla_decode_q8_workspace_bytes(4, 1, 1)
    assert need > 0
    assert mla.mla_decode_q8(*ok, stream=1, workspace=128, workspace_bytes=need) == mla.MLA_ERR_WORKSPACE
    # sparse: the list's stride, and no page table needed (then the workspace is what is missing)
    sparse = dict(d_indices=16, stream=1, workspace=256, workspace_bytes=16)
    a = list(ok)
    a[DECODE.index("pt")] = None
    assert mla.mla_decode_q8(*a, indices_stride=0, **sparse) == mla.MLA_ERR_ARG
    assert mla.mla_decode_q8(*a, indices_stride=8, **sparse) == mla.MLA_ERR_WORKSPACE


def test_decode_sizes(lib):
    assert mla.mla_decode_q8_workspace_bytes(0, 1, 1) == 0
    assert mla.mla_decode_q8_workspace_bytes(1, -1, 1) == 0
    assert mla.mla_decode_q8_workspace_bytes(1, 1, 0) == 0
    assert mla.mla_decode_q8_partitions(0, 1, 1, 100) == 1
    assert mla.mla_decode_q8_partitions(1, 16, 1, 1) == 1
    for keys in (1, 255, 257, 5000, 131072, 1 << 30):
        n = mla.mla_decode_q8_partitions(3, 128, 2, keys)
        assert 1 <= n <= 1024
        # a slot of 128 rows for each piece and each of the six tokens
        assert mla.mla_decode_q8_workspace_bytes(128, 6, n) >= (n + 6) * 128 * 1024


SCORES = ["s", "q", "w", "k", "ks", "iro", "cl", "pt", "np", "ps", "mp", "block", "B", "Hi", "T", "mn", "L", "stride",
          "dt"]


def test_scores_refusals(lib):
    ok = [16, 16, 16, 16, None, 16, 16, 16, 1, 16, 1, 4, 1, 8, 2, 1, 8, 2, mla.MLA_BF16]
    call = _caller(mla.mla_index_scores, SCORES, ok)
    assert call(dt=7) == mla.MLA_ERR_DTYPE
    assert call(Hi=0) == mla.MLA_ERR_GEOMETRY
    assert call(Hi=129) == mla.MLA_ERR_GEOMETRY
    for change in (dict(s=None), dict(q=8), dict(w=None), dict(k=20), dict(iro=None), dict(cl=None), dict(pt=None),
                   dict(np=0), dict(ps=0), dict(mp=0), dict(block=0), dict(block=3), dict(block=256), dict(B=0),
                   dict(T=-1), dict(mn=-1), dict(L=0), dict(stride=0), dict(stride=1), dict(np=1 << 30)):
        assert call(**change) == mla.MLA_ERR_ARG, change
    assert call(T=0) == mla.MLA_OK


SELECT = ["i", "c", "s", "iro", "cl", "pt", "np", "ps", "mp", "block", "top", "local", "B", "T", "L", "stride", "width"]


def test_select_refusals(lib):
    ok = [16, 16, 16, 16, 16, 16, 1, 16, 1, 4, 2, 1, 1, 2, 8, 2, 8]
    call = _caller(mla.mla_index_select, SELECT, ok)
    for change in (dict(i=None), dict(c=None), dict(s=None), dict(iro=None), dict(cl=None), dict(pt=None), dict(np=0),
                   dict(ps=0), dict(mp=0), dict(block=0), dict(block=6), dict(block=256), dict(top=0), dict(top=3),
                   dict(local=-1), dict(local=3), dict(B=0), dict(T=-1), dict(L=0), dict(L=9), dict(stride=0),
                   dict(width=7), dict(np=1 << 30), dict(T=1 << 28)):
        assert call(**change) == mla.MLA_ERR_ARG, change
    assert call(T=0) == mla.MLA_OK


# ------------------------------------------------------------------ the oracle

@pytest.mark.parametrize("amax,scale", [(448.0, 1.0), (448.0001, 2.0), (449.0, 2.0), (224.0, 0.5), (1.0, 2.0 ** -8),
                                        (0.0, 2.0 ** -60), (1e-30, 2.0 ** -60), (math.inf, 2.0 ** 120),
                                        (896.0, 2.0), (3.5, 2.0 ** -7)])
def test_block_scale(amax, scale):
    assert q8.block_scale(amax) == scale


def test_block_scale_is_the_smallest():
    rng = np.random.default_rng(0)
    for x in np.exp(rng.uniform(-30, 30, 300)):
        s = q8.block_scale(float(x))
        assert x <= 448 * s and x > 448 * s / 2 and math.log2(s) == round(math.log2(s))


def test_oracle_write_in_pieces_matches_one_call_up_to_requantisation():
    """Writing token by token grows scales; the values differ from those of one
    call only by the requantisation of what was denormal after growth."""
    rng = np.random.default_rng(1)
    sb, ps, n = 8, 16, 13
    y = rng.standard_normal((n, 576)) * np.exp(rng.uniform(-2, 4, (n, 1)))
    zero = np.zeros((1, ps, 576), np.uint8), np.ones((1, ps // sb))
    one = q8.latent_cache_write_q8(*zero, y, [0, n], [0], [[0]], ps, sb)
    c, s = zero
    for i in range(n):
        c, s, _ = q8.latent_cache_write_q8(c, s, y[i: i + 1], [0, 1], [i], [[0]], ps, sb)
    assert np.array_equal(s, one[1])
    a, b = q8.q8_values(c, s, sb)[:n], q8.q8_values(one[0], one[1], sb)[:n]
    assert np.all(np.abs(a - b) <= np.repeat(s.reshape(-1), sb)[:n, None] * 2.0 ** -9)


def test_oracle_decode_equals_the_bf16_oracle_on_the_same_values():
    rng = np.random.default_rng(2)
    ps, H, sb = 8, 3, 4
    codes = rng.integers(0, 0x70, (4, ps, 576)).astype(np.uint8)
    scales = np.full((4, ps // sb), 0.25)
    pt = np.array([[2, 0], [3, 1]])
    q = rng.standard_normal((3, H, 192))
    w_uk, w_uv = rng.standard_normal((H, 512, 128)) * 0.01, rng.standard_normal((H, 128, 512)) * 0.01
    iro, cl = [0, 2, 3], [9, 5]
    out, lse = q8.decode_values(q, q8.q8_values(codes, scales, sb), pt, ps, w_uk, w_uv, iro, cl, 0.05)
    ref = O.mla_decode(q, codes, pt, ps, w_uk, w_uv, iro, cl, 0.05, dtype="e4m3", ckv_scale=0.25)
    for (b, h), (tok, o, l) in ref.items():
        assert np.allclose(out[tok, h], o, rtol=1e-10, atol=1e-12)
        assert np.allclose(lse[tok, h], l, rtol=1e-12)


def test_oracle_select_closed_forms():
    s = np.array([[3.0, 1.0, 3.0, np.nan, 2.0, 0.0]])
    pt = [[1, 0]]
    # Position 10 in blocks of 2: six blocks, the last of one key; ties to the lowest.
    rows, cnt = q8.index_select(s, pt, 8, [0, 1], [10], 2, 2, 0, 6)
    assert rows[0] == [8, 9, 12, 13, -1, -1] and cnt[0] == 4
    rows, cnt = q8.index_select(s, pt, 8, [0, 1], [10], 2, 2, 1, 6)
    assert rows[0] == [8, 9, 2, -1, -1, -1] and cnt[0] == 3
    rows, cnt = q8.index_select(s, pt, 8, [0, 1], [10], 2, 9, 0, 18)
    assert cnt[0] == 11 and rows[0][:11] == list(range(8, 16)) + [0, 1, 2]


def test_oracle_scores_closed_form():
    q, w = np.ones((1, 2, 128)), np.array([[1.0, -2.0]])
    keys = np.zeros((1, 4, 128))
    keys[0, :, 0] = [1, -1, 2, 9]
    got, _ = q8.index_scores(q, w, keys, np.array([1, 1, 0.5, 1]), [[0]], 4, [0, 1], [2], 2, 3)
    assert got[0].tolist() == [0.0, -1.0, -np.inf]


def test_oracle_codes_agree_with_torch():
    rng = np.random.default_rng(4)
    x = rng.standard_normal(4000) * np.exp(rng.uniform(-8, 8, 4000))
    t = torch.from_numpy(np.clip(x, -448, 448)).to(torch.float32)
    assert np.array_equal(O.e4m3_encode(t.double().numpy()), t.to(torch.float8_e4m3fn).view(torch.uint8).numpy())


def test_stream_of_a_call_without_the_private_function(monkeypatch):
    """torch's raw stream lookup is not public: without it the public one serves."""
    monkeypatch.setattr(mla, "_current_stream", None)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 70 + device, raising=False)
    assert mla._stream(None) == 73
    monkeypatch.setattr(mla, "_current_stream", None)
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream")
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: type("S", (), {"cuda_stream": 5})())
    assert mla._stream(None) == 5 and mla._stream(9) == 9
