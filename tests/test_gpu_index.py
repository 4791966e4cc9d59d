"""GPU tests of the key scores and the block selection for sparse decode, and of
the whole chain: write into the 8-bit cache, score, select, decode.

Scores: products of bf16 or e4m3 values are exact in fp32, so what remains is
the rounding of at most 128 + 128 fp32 additions, each within 2^-24 (2^-23 where
the tensor core truncates) of the sum of magnitudes: 256 * 2^-23 = 2^-15 of
sum_h |w| sum |q||k| covers it.  Selections are whole numbers and equal."""
import numpy as np
import pytest
import torch

import mla_prefill_attention_plan_gb300 as mla
import oracle as O
from oracle import q8
from test_gpu_q8 import DEV, Decode, fp8, i32, offsets, pages, status
from workloads import WORKLOADS, make_cache_write_operands, scaled

pytestmark = pytest.mark.gpu
FILL = 3.5


@pytest.fixture(scope="module", autouse=True)
def _built():
    from mla_prefill_attention_plan_gb300 import build
    build.build()
    mla.load()


def run_scores(new, cached, Hi, block, page, eight=False, scales=False, seed=0, extra_stride=0, T_extra=0, junk=True,
               expect=0, max_seq=None):
    rng = np.random.default_rng(seed)
    table, num = pages(new, cached, page, seed)
    iro, T = offsets(new), int(sum(new)) + T_extra
    L = [n + c for n, c in zip(new, cached)]
    max_seq = max(L) if max_seq is None else max_seq
    stride = -(-max_seq // block) + extra_stride
    kind = "e4m3" if eight else "bf16"
    enc = O.e4m3_encode if eight else O.bf16_encode
    q, k = enc(rng.standard_normal((T, Hi, 128))), enc(rng.standard_normal((num, page, 128)))
    w = rng.standard_normal((T, Hi)).astype(np.float32)
    ks = np.exp(rng.uniform(-2, 2, num * page)).astype(np.float32) if scales else None
    q_val, k_val = O.decode(q, kind), O.decode(k, kind)
    if junk:   # NaN keys and scales behind the contexts
        used = np.zeros(num * page, bool)
        for b in range(len(new)):
            j = np.arange(L[b])
            used[table[b, j // page] * page + j % page] = True
        k.reshape(-1, 128)[~used] = 0x7F if eight else 0x7FC0
        if ks is not None:
            ks[~used] = np.nan
    out = torch.full((T, stride), FILL, device=DEV)
    st = status()
    view = (lambda x: torch.from_numpy(x).to(DEV)) if eight else (lambda x: torch.from_numpy(x.view(np.int16)).to(DEV))
    mla.check(mla.mla_index_scores(out, view(q), torch.from_numpy(w).to(DEV), view(k),
                                   None if ks is None else torch.from_numpy(ks).to(DEV), i32(iro), i32(cached),
                                   i32(table), num, page, table.shape[1], block, len(new), Hi, T, max(new), max_seq,
                                   stride, mla.MLA_E4M3 if eight else mla.MLA_BF16, st))
    torch.cuda.synchronize()
    assert st.item() == expect
    with np.errstate(invalid="ignore"):
        ref, mag = q8.index_scores(q_val, w, k_val, ks, table, page, iro, cached, block, stride)
    return out.cpu().double().numpy(), ref, mag


def check_scores(*a, **kw):
    got, ref, mag = run_scores(*a, **kw)
    outside = np.isnan(ref).all(1)
    assert np.all(got[outside] == FILL)
    got, ref, mag = got[~outside], ref[~outside], mag[~outside]
    dead = np.isneginf(ref)
    assert np.all(np.isneginf(got[dead]))
    assert np.all(np.abs(got[~dead] - ref[~dead]) <= 2.0 ** -15 * mag[~dead])


@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("page", [128, 64, 24, 100, 1])
def test_scores_pages(page, eight):
    check_scores([1, 2, 0, 1], [300, 127, 9, 0], 16, 1, page, eight, scales=eight, seed=page)


@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("block", [1, 2, 8, 32, 64, 128])
def test_scores_blocks(block, eight):
    """Maxima inside a warp and across warps; strides longer than needed."""
    check_scores([1, 3, 1], [1000, 255, 127], 8, block, 32, eight, seed=block, extra_stride=5)


@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("Hi", [1, 5, 15, 16, 33, 64, 127, 128])
def test_scores_heads(Hi, eight):
    check_scores([2, 1], [200, 60], Hi, 1, 16, eight, seed=Hi)


@pytest.mark.parametrize("eight", [False, True])
def test_scores_many_new_tokens(eight):
    """Several groups of tokens a sequence, each token with its own limit."""
    check_scores([70, 1, 33], [100, 600, 0], 64, 16, 16, eight, scales=True)


def test_scores_ring_longer_than_its_stages():
    check_scores([1], [8000], 64, 1, 128)
    check_scores([1], [8000], 4, 1, 100)              # rows copied one by one
    check_scores([1], [8000], 4, 1, 100, True)


def test_scores_rows_behind_the_last_sequence():
    check_scores([1, 1], [10, 20], 4, 1, 16, T_extra=2)


def test_scores_nan_key_gives_nan():
    table, num = pages([1], [20], 16)
    k = torch.ones(num, 16, 128, dtype=torch.bfloat16, device=DEV)
    k[int(table[0, 0]), 3, 7] = float("nan")
    q, w = torch.ones(1, 4, 128, dtype=torch.bfloat16, device=DEV), torch.ones(1, 4, device=DEV)
    out = torch.zeros(1, 21, device=DEV)
    mla.check(mla.mla_index_scores(out, q, w, k, None, i32([0, 1]), i32([20]), i32(table), num, 16, 2, 1, 1, 4, 1, 1, 21,
                                   21, mla.MLA_BF16))
    got = out[0].tolist()
    assert np.isnan(got[3]) and [x for i, x in enumerate(got) if i != 3] == [512.0] * 20


def test_scores_status():
    got, ref, mag = run_scores([1, 1], [10, 50], 4, 1, 16, max_seq=20, extra_stride=31, expect=mla.MLA_DEV_BAD_OFFSETS)
    assert np.all(got[1] == FILL) and np.abs(got[0, :11] - ref[0, :11]).max() <= 2.0 ** -15 * mag.max()


@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("block", [1, 16, 64, 128])
@pytest.mark.parametrize("Hi", [1, 16, 17, 32, 40, 64, 100, 128])
def test_scores_several_tokens(Hi, block, eight):
    """Batches of one to eight tokens an MMA, the last ones not full."""
    check_scores([9, 1, 30], [200, 130, 0], Hi, block, 16, eight, scales=True, seed=Hi)


@pytest.mark.parametrize("B", [700, 1500])
def test_scores_many_sequences(B):
    """Runs found among more sequences than a CTA has threads; and, without
    cutting, a CTA for each.  Some sequences are empty, one is long."""
    new = [0 if b % 7 == 3 else 1 for b in range(B)]
    cached = [b % 50 for b in range(B)]
    cached[B // 2] = 2000
    check_scores(new, cached, 3, 4, 16, seed=B)


def test_scores_max_seq_far_above_the_contexts():
    check_scores([1, 3], [500, 130], 8, 2, 16, max_seq=40000, extra_stride=3)
    check_scores([20, 3], [500, 130], 40, 128, 16, max_seq=40000)


@pytest.mark.parametrize("Hi", [3, 16, 24, 40])
def test_scores_infinite_weight(Hi):
    """An infinite weight gives infinity or, where the product is not positive,
    NaN, in its own token only."""
    L = 50
    rng = np.random.default_rng(Hi)
    table, num = pages([2], [L - 2], 16)
    k = torch.from_numpy(rng.standard_normal((num, 16, 128))).to(torch.bfloat16)
    q = torch.from_numpy(rng.standard_normal((2, Hi, 128))).to(torch.bfloat16)
    w = torch.from_numpy(rng.uniform(0.5, 1, (2, Hi))).float()
    w[1, Hi - 1] = float("inf")
    out = torch.zeros(2, L, device=DEV)
    mla.check(mla.mla_index_scores(out, q.to(DEV), w.to(DEV), k.to(DEV), None, i32([0, 2]), i32([L - 2]), i32(table), num,
                                   16, table.shape[1], 1, 1, Hi, 2, 2, L, L, mla.MLA_BF16))
    rows = k.reshape(-1, 128).double()[torch.from_numpy(table[0][np.arange(L) // 16] * 16 + np.arange(L) % 16)]
    pos = (q[1, Hi - 1].double() @ rows.T > 0).numpy()
    got = out.cpu().numpy()
    assert np.isfinite(got[0, :L - 1]).all() and np.isneginf(got[0, L - 1])
    assert np.all(np.isposinf(got[1][pos])) and np.all(np.isnan(got[1][~pos]))


def test_scores_replay_bit_for_bit():
    rng = np.random.default_rng(0)
    new, cached, Hi, page = [3, 1], [500, 900], 32, 64
    table, num = pages(new, cached, page)
    q, k = (torch.from_numpy(rng.standard_normal(x)).to(torch.bfloat16).to(DEV) for x in ((4, Hi, 128), (num, page, 128)))
    w, out = torch.from_numpy(rng.standard_normal((4, Hi))).float().to(DEV), torch.zeros(4, 15, device=DEV)
    args = (out, q, w, k, None, i32(offsets(new)), i32(cached), i32(table), num, page, table.shape[1], 64, 2, Hi, 4, 3, 901,
            15, mla.MLA_BF16)
    mla.check(mla.mla_index_scores(*args))
    torch.cuda.synchronize()
    ref = out.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mla.check(mla.mla_index_scores(*args))
    for _ in range(2):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, ref)


# ------------------------------------------------------------------ selection

def check_select(new, cached, block, top, local, page=16, seed=0, scores=None, T_extra=0, extra_stride=0, width=None):
    rng = np.random.default_rng(seed)
    table, num = pages(new, cached, page, seed)
    iro, T = offsets(new), int(sum(new)) + T_extra
    max_seq = max(n + c for n, c in zip(new, cached))
    stride = -(-max_seq // block) + extra_stride
    if scores is None:
        scores = rng.standard_normal((T, stride))
    elif callable(scores):
        scores = scores(rng, (T, stride))
    scores = scores.astype(np.float32)
    width = top * block if width is None else width
    rows = torch.full((T, width), -7, dtype=torch.int32, device=DEV)
    cnt = torch.full((T,), -7, dtype=torch.int32, device=DEV)
    st = status()
    mla.check(mla.mla_index_select(rows, cnt, torch.from_numpy(scores).to(DEV), i32(iro), i32(cached), i32(table), num,
                                   page, table.shape[1], block, top, local, len(new), T, max_seq, stride, width, st))
    torch.cuda.synchronize()
    assert st.item() == 0
    ref, ref_cnt = q8.index_select(scores, table, page, iro, cached, block, top, local, width)
    got, got_cnt = rows.cpu().numpy(), cnt.cpu().numpy()
    for t in range(T):
        if ref[t] is None:
            assert np.all(got[t] == -7) and got_cnt[t] == -7
        else:
            assert got_cnt[t] == ref_cnt[t] and np.array_equal(got[t], ref[t])


def quantised(rng, shape):
    return rng.integers(-3, 4, shape).astype(np.float64)


def special(rng, shape):
    return rng.choice([np.nan, np.inf, -np.inf, 0.0, -0.0, 1.0, -1.0, 1e-45, 3e38], shape)


@pytest.mark.parametrize("scores", [None, quantised, special, np.ones])
@pytest.mark.parametrize("block", [1, 4, 64, 128])
@pytest.mark.parametrize("local", [0, 1, 3])
def test_select(block, local, scores):
    fn = (lambda rng, s: np.ones(s)) if scores is np.ones else scores
    check_select([1, 3, 0, 1, 1], [700, 260, 8, 0, 1999], block, 5, local, seed=block, scores=fn, width=5 * block + 3)


@pytest.mark.parametrize("top", [1, 2, 63, 64, 999, 1000, 1001, 5000])
def test_select_counts(top):
    check_select([2], [999], 1, top, 1, scores=quantised)


def test_select_many_tokens():
    check_select([170, 40], [50, 3000], 1, 100, 1, page=128, extra_stride=7)


@pytest.mark.parametrize("scores", [None, quantised])
@pytest.mark.parametrize("cached", [9000, 40000, 70000])
def test_select_over_a_cluster(cached, scores):
    """Long rows of few tokens: two to eight CTAs a token, and a short row beside
    them whose last CTAs have nothing."""
    check_select([1, 1], [cached, 30], 1, 2048, 1, page=128, scores=scores)


def test_select_many_sequences():
    """More sequences than are probed at once, some of them empty."""
    new = [0 if b % 7 == 3 else 1 for b in range(1500)]
    check_select(new, [b % 50 for b in range(1500)], 1, 8, 1, scores=quantised)


def test_select_longer_than_shared_memory():
    """400000 scores: a slice no longer fits and is read again for each digit."""
    check_select([1], [399999], 1, 3000, 2, page=256, scores=quantised)


def test_select_rows_behind_the_last_sequence():
    check_select([1, 1], [10, 20], 2, 3, 1, T_extra=3)


def test_select_bad_page():
    rows = torch.zeros(1, 4, dtype=torch.int32, device=DEV)
    cnt, st = torch.zeros(1, dtype=torch.int32, device=DEV), status()
    mla.check(mla.mla_index_select(rows, cnt, torch.arange(20.0, device=DEV).view(1, -1), i32([0, 1]), i32([19]),
                                   i32([[0, 9]]), 2, 16, 2, 1, 4, 0, 1, 1, 20, 20, 4, st))
    torch.cuda.synchronize()
    assert st.item() == mla.MLA_DEV_BAD_PAGE and rows.tolist() == [[-1, -1, -1, -1]] and cnt.item() == 4


@pytest.mark.parametrize("n,L", [(3, 20000), (1, 140000)])
def test_select_replays_bit_for_bit(n, L):
    s = torch.randn(n, L, generator=torch.Generator().manual_seed(0)).to(DEV)
    rows = torch.zeros(n, 2048, dtype=torch.int32, device=DEV)
    cnt = torch.zeros(n, dtype=torch.int32, device=DEV)
    args = (rows, cnt, s, i32(range(n + 1)), i32([L - 1] * n), i32(np.zeros((n, L // 100 + 1))), 1, 100, L // 100 + 1, 1,
            2048, 1, n, n, L, L, 2048)
    mla.check(mla.mla_index_select(*args))
    torch.cuda.synchronize()
    ref = rows.clone()
    assert cnt.tolist() == [2048] * n
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mla.check(mla.mla_index_select(*args))
    for _ in range(2):
        rows.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(rows, ref)


# ------------------------------------------------------------------ together

def test_write_score_select_decode_together():
    """Two decode steps as a serving loop makes them: the new tokens' rows into
    the 8-bit cache, index scores over the paged index keys, the best rows of
    every token, sparse decode with each token as a sequence of its own.  Every
    stage is held to the oracle on the stage before's device results."""
    H, Hi, page, sb, block, top, B = 8, 16, 64, 16, 8, 12, 2
    new, cached = [1, 2], [700, 250]
    d = Decode([n + 2 for n in new], cached, H, page, sb, lo=-7, hi=-6)     # room for both steps
    table, num = d.table, d.num
    rng = np.random.default_rng(9)
    kv, sc = fp8(d.codes), torch.from_numpy(d.scales).to(DEV)
    index_cache = torch.from_numpy(rng.standard_normal((num, page, 128))).to(torch.bfloat16)
    gamma, freqs = make_cache_write_operands(scaled(WORKLOADS["tiny_ragged"], H=H), 1, 1024)[1:]
    w_uk, w_uv = d.w_uk.to(DEV), d.w_uv.to(DEV)
    for step in range(2):
        iro, T = offsets(new), sum(new)
        max_seq = max(n + c for n, c in zip(new, cached))
        lat = torch.from_numpy(rng.standard_normal((T, 576))).to(torch.bfloat16)
        q = torch.from_numpy(rng.standard_normal((T, H, 192))).to(torch.bfloat16)
        iq = torch.from_numpy(rng.standard_normal((T, Hi, 128))).to(torch.bfloat16)
        iw = torch.from_numpy(rng.standard_normal((T, Hi))).float()
        dq, st = q.to(DEV), status()
        mla.check(mla.mla_latent_cache_write_q8(kv, sc, dq, lat.to(DEV), gamma.to(DEV), freqs.to(DEV), i32(iro),
                                                i32(cached), i32(table), num, page, table.shape[1], sb, B, H, T, 1024,
                                                1e-6, st))
        stride = -(-max_seq // block)
        scores = torch.zeros(T, stride, device=DEV)
        mla.check(mla.mla_index_scores(scores, iq.to(DEV), iw.to(DEV), index_cache.to(DEV), None, i32(iro), i32(cached),
                                       i32(table), num, page, table.shape[1], block, B, Hi, T, max(new), max_seq, stride,
                                       mla.MLA_BF16, st))
        rows = torch.zeros(T, top * block, dtype=torch.int32, device=DEV)
        cnt = torch.zeros(T, dtype=torch.int32, device=DEV)
        mla.check(mla.mla_index_select(rows, cnt, scores, i32(iro), i32(cached), i32(table), num, page, table.shape[1],
                                       block, top, 1, B, T, max_seq, stride, top * block, st))
        each = torch.arange(T + 1, dtype=torch.int32, device=DEV)
        parts = mla.mla_decode_q8_partitions(T, H, 1, top * block)
        nbytes = mla.mla_decode_q8_workspace_bytes(H, T, parts)
        ws = torch.empty(nbytes, dtype=torch.uint8, device=DEV)
        out, lse = torch.zeros(T, H, 128, dtype=torch.bfloat16, device=DEV), torch.zeros(T, H, device=DEV)
        mla.check(mla.mla_decode_q8(out, lse, dq, each, i32([0] * T), kv, sc, None, num, page, 0, sb, w_uk, w_uv, T, H, T,
                                    1, top * block, 0, d.scale, d_indices=rows, indices_stride=top * block,
                                    topk_lengths=cnt, workspace=ws, workspace_bytes=nbytes, d_status=st))
        torch.cuda.synchronize()
        assert st.item() == 0
        y = q8.new_rows(O.decode(O.codes(lat), "bf16"), gamma.numpy(), freqs.numpy(), iro, cached, 1e-6)
        codes, scales, pre = q8.latent_cache_write_q8(d.codes, d.scales, y, iro, cached, table, page, sb)
        assert np.array_equal(sc.cpu().numpy(), scales.astype(np.float32))
        d.codes, d.scales = kv.cpu().numpy(), sc.cpu().numpy()
        assert np.mean(d.codes != codes) < 1e-4        # codes next to a rounding border only
        ref, mag = q8.index_scores(O.decode(O.codes(iq), "bf16"), iw.numpy(), O.decode(O.codes(index_cache), "bf16"), None,
                                   table, page, iro, cached, block, stride)
        s = scores.cpu().double().numpy()
        fin = np.isfinite(ref)
        assert np.all(np.abs(s[fin] - ref[fin]) <= 2.0 ** -15 * mag[fin]) and np.all(s[~fin] == ref[~fin])
        lists, counts = q8.index_select(s, table, page, iro, cached, block, top, 1, top * block)
        assert rows.cpu().tolist() == lists and cnt.cpu().tolist() == counts
        ref_out, ref_lse = q8.decode_values(dq.float().cpu().double().numpy(), q8.q8_values(d.codes, d.scales, sb), None,
                                            page, O.decode(O.codes(d.w_uk), "bf16"), O.decode(O.codes(d.w_uv), "bf16"),
                                            np.arange(T + 1), [0] * T, d.scale, rows.cpu().numpy(), cnt.cpu().numpy())
        g = out.float().cpu().double().numpy()
        assert np.linalg.norm(g - ref_out) <= 2.0 ** -8 * np.linalg.norm(ref_out)
        assert np.abs(lse.cpu().double().numpy() - ref_lse).max() <= 5e-3
        cached = [n + c for n, c in zip(new, cached)]
        new = [1, 2] if step else [2, 1]


def test_selected_rows_in_the_bf16_decode():
    """The lists serve mla_decode's sparse form as they are."""
    H, page, B = 4, 32, 2
    new, cached = [1, 1], [300, 90]
    d = Decode(new, cached, H, page, 1, lo=-6, hi=-6)
    kv = torch.from_numpy(q8.q8_values(d.codes, d.scales, 1)).to(torch.bfloat16).view(d.num, page, 576)
    s = torch.randn(2, 301, generator=torch.Generator().manual_seed(1)).to(DEV)
    rows = torch.zeros(2, 64, dtype=torch.int32, device=DEV)
    cnt, st = torch.zeros(2, dtype=torch.int32, device=DEV), status()
    mla.check(mla.mla_index_select(rows, cnt, s, i32(d.iro), i32(cached), i32(d.table), d.num, page, d.table.shape[1], 1,
                                   64, 1, B, 2, 301, 301, 64, st))
    nbytes = mla.mla_decode_workspace_bytes(H, 2, 1)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=DEV)
    out = torch.zeros(2, H, 128, dtype=torch.bfloat16, device=DEV)
    mla.check(mla.mla_decode(out, None, d.q.to(DEV), i32(d.iro), i32(cached), kv.to(DEV), None, d.num, page, 0,
                             d.w_uk.to(DEV), d.w_uv.to(DEV), B, H, 2, 1, 301, 1, d.scale, d_indices=rows,
                             indices_stride=64, topk_lengths=cnt, workspace=ws, workspace_bytes=nbytes, d_status=st))
    torch.cuda.synchronize()
    assert st.item() == 0
    ref, _ = d.reference(lists=rows.cpu().numpy(), topk=cnt.cpu().numpy())
    g = out.float().cpu().double().numpy()
    assert np.abs(g - ref).max() <= 2e-2 and np.abs(g - ref).sum() <= 1e-2 * np.abs(ref).sum()


@pytest.mark.parametrize("B", [3, 2500])
def test_scores_decreasing_offsets(B):
    """The second sequence ends before it begins: reported, the first one scored.
    (A few sequences, whose work is shared out, and so many that each has a CTA.)"""
    page, table = 16, np.arange(2 * B).reshape(B, 2)
    iro = np.concatenate([[0, 4, 2], np.arange(2, B) + 3])            # 4 tokens, -2, 3, then one each
    T = int(iro[-1])
    q, w = torch.ones(T, 4, 128, dtype=torch.bfloat16, device=DEV), torch.ones(T, 4, device=DEV)
    k = torch.ones(2 * B, page, 128, dtype=torch.bfloat16, device=DEV)
    out, st = torch.full((T, 32), FILL, device=DEV), status()
    mla.check(mla.mla_index_scores(out, q, w, k, None, i32(iro), i32([9] * B), i32(table), 2 * B, page, 2, 1, B, 4, T, 4,
                                   32, 32, mla.MLA_BF16, st))
    torch.cuda.synchronize()
    assert st.item() == mla.MLA_DEV_BAD_OFFSETS
    assert torch.all(out[0, :10] == 512.0) and torch.all(out[0, 10:] == float("-inf"))
    if B > 3:
        assert torch.all(out[-1, :10] == 512.0) and torch.all(out[-1, 10:] == float("-inf"))


def test_select_decreasing_offsets():
    iro, scores = [0, 4, 2, 5], torch.randn(5, 32, device=DEV)
    rows, cnt, st = torch.full((5, 8), -7, dtype=torch.int32, device=DEV), torch.zeros(5, dtype=torch.int32, device=DEV), status()
    mla.check(mla.mla_index_select(rows, cnt, scores, i32(iro), i32([9] * 3), i32([[0, 1], [2, 3], [4, 5]]), 6, 16, 2, 1, 8, 1,
                                   3, 5, 32, 32, 8, st))
    torch.cuda.synchronize()
    assert st.item() == mla.MLA_DEV_BAD_OFFSETS and cnt[0].item() == 8


def test_select_leaves_out_what_the_scores_leave_out():
    """The second sequence's context is one token longer than max_seq_len: none of
    its tokens has scores, so none is given a list, the first two positions that
    do exist included."""
    new, cached, max_seq = [1, 3], [10, 18], 20
    table, num = pages(new, cached, 16)
    k = torch.ones(num, 16, 128, dtype=torch.bfloat16, device=DEV)
    q, w = torch.ones(4, 4, 128, dtype=torch.bfloat16, device=DEV), torch.ones(4, 4, device=DEV)
    scores, st = torch.full((4, max_seq), FILL, device=DEV), status()
    iro, cl = i32(offsets(new)), i32(cached)
    mla.check(mla.mla_index_scores(scores, q, w, k, None, iro, cl, i32(table), num, 16, table.shape[1], 1, 2, 4, 4, 3,
                                   max_seq, max_seq, mla.MLA_BF16, st))
    rows, cnt = torch.full((4, 6), -7, dtype=torch.int32, device=DEV), torch.full((4,), -7, dtype=torch.int32, device=DEV)
    mla.check(mla.mla_index_select(rows, cnt, scores, iro, cl, i32(table), num, 16, table.shape[1], 1, 6, 1, 2, 4, max_seq,
                                   max_seq, 6, st))
    torch.cuda.synchronize()
    assert st.item() == mla.MLA_DEV_BAD_OFFSETS
    assert torch.all(scores[1:] == FILL) and torch.all(rows[1:] == -7) and torch.all(cnt[1:] == -7)
    assert cnt[0].item() == 6 and rows[0].min().item() >= 0
