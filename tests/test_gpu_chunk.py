"""GPU tests of chunk attention against the float64 oracle.

Tolerance.  A bf16 rounding is off by at most 2^-8 of the value, on average over
the significand by 0.42 * 2^-8 = 0.00165 (root mean square).  On random rows
three of them reach an output, independent of each other: its own, the weights',
and the projected query's, which moves a score of spread sigma by 0.00165 sigma
(sigma is 1 here).  Together 0.00165 * sqrt(3) = 0.0029 of the output's 2-norm;
twice that is allowed for a whole result, four times for a row of 128 values.  (Small calls have the weights
in two terms; the bound stays.)
The lse is off by no more than the worst score: 2^-8 of scale * sum |q_lat c|
(the oracle's slack), and fp32's part of it."""
import numpy as np
import pytest
import torch

import mla_prefill_attention_plan_gb300 as mla
import oracle as O
from oracle import chunk_oracle as C
from oracle import pages_oracle as P

pytestmark = pytest.mark.gpu
DEV = "cuda"
FILL = 3.5
WHOLE, ROW = 2 * 0.0029, 4 * 0.0029


@pytest.fixture(scope="module", autouse=True)
def _built():
    from mla_prefill_attention_plan_gb300 import build
    build.build()
    mla.load()


def dev(x, kind=np.int32):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(x).astype(kind))).to(DEV)


def bf16(x):
    """(device tensor, the values it holds)."""
    t = torch.from_numpy(np.asarray(x, dtype=np.float32)).to(torch.bfloat16)
    return t.to(DEV), t.double().numpy()


def tree(rng, n):
    seen = []
    for i in range(n):
        up = int(rng.integers(-1, i)) if i else -1
        seen.append(1 << i | (seen[up] if up >= 0 else 0))
    return seen


def words_of(rows, words):
    return np.array([[r >> 32 * w & 0xffffffff for w in range(words)] for r in rows], dtype=np.uint32).view(np.int32)


@pytest.fixture(params=["small", "any"], autouse=True)
def size(request):
    """Calls whose page table holds few tiles have their weights in two terms."""
    Case.reach = 0 if request.param == "small" else 40000


class Case:
    """Inputs of ragged sequences on shuffled pages; rows that no sequence sees are NaN."""

    reach = 0              # positions that the page table has entries for, at least

    def __init__(self, new, cached, H, page, seed=0, mask="tree", sink=False, extra=0, words=None, spread=1.0):
        rng = np.random.default_rng(seed)
        self.new, self.cached, self.H, self.page, self.B = new, cached, H, page, len(new)
        held = [-(-(n + c) // page) for n, c in zip(new, cached)]
        self.num, self.most = sum(held) + 1, max(held + [self.reach // page]) + 1
        order, at = rng.permutation(self.num), 0
        self.table = np.full((self.B, self.most), -1, np.int32)
        for b, k in enumerate(held):
            self.table[b, :k] = order[at: at + k]
            at += k
        self.iro = np.concatenate([[0], np.cumsum(new)])
        self.T = int(self.iro[-1]) + extra
        rows = np.full((self.num * page, 576), np.nan)
        for b in range(self.B):
            j = np.arange(new[b] + cached[b])
            rows[self.table[b, j // page] * page + j % page] = rng.standard_normal((len(j), 576))
        self.kv_d, self.kv = bf16(rows)
        self.q_d, self.q = bf16(rng.standard_normal((self.T, H, 192)) * spread)
        self.uk_d, self.uk = bf16(rng.standard_normal((H, 512, 128)) * 512 ** -0.5)
        self.uv_d, self.uv = bf16(rng.standard_normal((H, 128, 512)) * 512 ** -0.5)
        self.mask = None
        if mask == "tree":
            self.mask = sum((tree(rng, n) for n in new), [])
        elif mask == "any":
            self.mask = [int(rng.integers(0, 2)) and int.from_bytes(rng.bytes(32), "little") for _ in range(self.T)]
        elif isinstance(mask, list):
            self.mask = mask
        self.words = 0
        if self.mask is not None:
            self.words = words or max(1, -(-max(new) // 32))
            self.mask = (self.mask + [0] * self.T)[:self.T]
        self.sink = rng.standard_normal(self.B).astype(np.float32) if sink else None
        self.scale = 192 ** -0.5
        self.make_buffers()

    def make_buffers(self):
        self.out = torch.full((self.T, self.H, 128), FILL, dtype=torch.bfloat16, device=DEV)
        self.lse = torch.full((self.T, self.H), FILL, device=DEV)
        self.st = torch.zeros(1, dtype=torch.int32, device=DEV)
        self.bytes = mla.mla_chunk_attention_workspace_bytes(self.B, self.H, self.T)
        self.ws = torch.randint(0, 256, (self.bytes,), dtype=torch.uint8, device=DEV)
        self.ints = [dev(self.iro), dev(self.cached), dev(self.table)]
        self.mask_d = None if self.mask is None else dev(words_of(self.mask, self.words))
        self.sink_d = None if self.sink is None else torch.from_numpy(self.sink).to(DEV)

    def call(self, lse=True, stream=None, **kw):
        iro, cached, table = self.ints
        a = dict(chunk_mask=self.mask_d, mask_words=self.words, attn_sink=self.sink_d, workspace=self.ws,
                 workspace_bytes=self.bytes, d_status=self.st, stream=stream)
        a.update(kw)
        return mla.mla_chunk_attention(self.out, self.lse if lse else None, self.q_d, iro, cached, self.kv_d, table,
                                       self.num, self.page, self.most, self.uk_d, self.uv_d, self.B, self.H, self.T,
                                       self.scale, **a)

    def oracle(self):
        return C.chunk_attention(self.q, self.kv, self.table, self.page, self.uk, self.uv, self.iro, self.cached,
                                 self.scale, self.mask, self.sink)

    def check(self, **kw):
        mla.check(self.call(**kw))
        torch.cuda.synchronize()
        assert self.st.item() == 0
        self.compare(*self.oracle())

    def compare(self, out, lse, slack):
        got, got_lse = self.out.double().cpu().numpy(), self.lse.double().cpu().numpy()
        outside = np.isnan(lse)
        assert (got[outside] == FILL).all() and (got_lse[outside] == FILL).all()
        got, got_lse, out, lse, slack = (x[~outside] for x in (got, got_lse, out, lse, slack))
        blank = np.isneginf(lse)
        assert np.isneginf(got_lse[blank]).all() and not got[blank].any()
        got, got_lse, out, lse, slack = (x[~blank] for x in (got, got_lse, out, lse, slack))
        if not len(out):
            return
        assert np.isfinite(got).all()
        off, size = np.linalg.norm(got - out, axis=-1), np.linalg.norm(out, axis=-1)
        assert np.linalg.norm(off) <= WHOLE * np.linalg.norm(size), np.linalg.norm(off) / np.linalg.norm(size)
        assert (off <= ROW * size + 1e-6).all(), (off / size).max()
        worst = 2.0 ** -8 * slack + 2.0 ** -20 * (1 + np.abs(lse))
        assert (np.abs(got_lse - lse) <= worst).all(), (np.abs(got_lse - lse) / worst).max()


def test_small_calls_are_closer():
    """At most 0.00165 sqrt(2) = 0.0023 without the weights' rounding, 0.0029 with it:
    over 10^5 values a result is far from the middle of them."""
    off = []
    for Case.reach in (0, 40000):
        c = Case([20], [1000], 64, 64)
        mla.check(c.call())
        out = c.oracle()[0]
        off.append(np.linalg.norm(c.out.double().cpu().numpy() - out) / np.linalg.norm(out))
    assert off[0] < 0.0026 and off[0] < 0.95 * off[1], off


@pytest.mark.parametrize("page", [128, 256, 64, 16, 24, 100, 7, 1])
def test_pages(page):
    Case([3, 1, 5], [300, 255, 40], 4, page, seed=page).check()


@pytest.mark.parametrize("H", [1, 2, 16, 21, 64, 128])
def test_heads(H):
    Case([2, 3], [70, 400], H, 16, seed=H).check()


@pytest.mark.parametrize("cached", [0, 1, 126, 127, 128, 129, 253, 254, 255, 256, 257, 511, 512, 600])
def test_context_lengths_at_the_tiles_edges(cached):
    """New tokens on both sides of a half tile's and a tile's edge."""
    Case([3], [cached], 8, 32, seed=cached).check()


@pytest.mark.parametrize("mask", ["causal", "tree", "any"])
@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 64, 65, 100, 128])
def test_chunk_lengths(n, mask):
    Case([n, 1], [90, 3], 3, 16, seed=n, mask=mask).check()


@pytest.mark.parametrize("mask", ["causal", "tree"])
def test_long_chunks(mask):
    """More new tokens than a tile has keys, rows of several tiles a token."""
    Case([300, 2], [5, 200], 2, 64, mask=mask, words=16 if mask == "tree" else None).check()


def test_no_new_tokens_and_single_ones():
    Case([0, 1, 0, 1, 0], [10, 0, 0, 700, 3], 16, 16).check()


def test_many_short_sequences():
    """Several row tiles a piece, sequences shorter than one key tile."""
    rng = np.random.default_rng(5)
    Case(list(rng.integers(0, 6, 200)), list(rng.integers(0, 60, 200)), 4, 16, mask="any").check()


@pytest.mark.parametrize("mask", ["causal", "any"])
def test_one_long_sequence_cut_into_many_pieces(mask):
    Case([4], [22000], 4, 128, mask=mask).check()


@pytest.mark.parametrize("sink", [True, False])
def test_rows_that_see_nothing(sink):
    Case([4, 2, 1], [0, 0, 9], 5, 16, mask=[0, 1, 0, 6, 0, 2, 0], sink=sink).check()


def test_rows_that_see_nothing_in_a_split_tile():
    """No cached keys, thousands of new ones, of which most rows see few."""
    rng = np.random.default_rng(1)
    n = 3500
    mask = [0 if i % 3 == 0 else 1 << int(rng.integers(n)) | 1 << int(rng.integers(n)) for i in range(n)]
    c = Case([n], [0], 1, 128, mask=mask, words=-(-n // 32))
    c.check()


@pytest.mark.parametrize("mask", ["causal", "tree"])
def test_sinks(mask):
    Case([5, 40, 1], [0, 300, 2000], 16, 64, mask=mask, sink=True).check()


def test_a_sink_that_is_no_logit():
    c = Case([2, 2], [30, 0], 4, 16, sink=True)
    c.sink[:] = [-np.inf, 80.0]
    c.make_buffers()
    c.check()


def test_rows_behind_the_last_sequence_stay():
    Case([3, 2], [50, 10], 4, 16, extra=4).check()


def test_spread_scores():
    """Scores whose maximum moves from tile to tile: references that follow it.
    (sigma is 6: the query's rounding counts six times, so that bound only.)"""
    c = Case([4], [3000], 4, 64, spread=6.0)
    mla.check(c.call())
    out, lse, slack = c.oracle()
    got = c.out.double().cpu().numpy()
    assert np.linalg.norm(got - out) <= 2 * 0.00165 * np.sqrt(2 + 36) * np.linalg.norm(out)
    assert (np.abs(c.lse.double().cpu().numpy() - lse) <= 2.0 ** -8 * slack + 2.0 ** -20 * (1 + np.abs(lse))).all()


def test_a_maximum_that_grows_and_one_far_above():
    """Keys whose scores rise along the context by far more than a reference
    bears, and one key that takes all the weight."""
    c = Case([1], [2000], 1, 64, mask="causal")
    rows = c.kv.copy()
    lat = c.uk[0] @ c.q[0, 0, :128]
    j = np.arange(2001)
    at = c.table[0, j // 64] * 64 + j % 64
    rows[at, :512] += np.outer(np.linspace(-3, 3, 2001), lat / np.linalg.norm(lat)) * 60
    c.kv_d, c.kv = bf16(rows)
    mla.check(c.call())
    out, lse, slack = c.oracle()
    got = c.out.double().cpu().numpy()
    # The scores' error is bounded by the slack; what it does to a softmax by twice that, relative.
    assert np.linalg.norm(got - out) <= (2 * 0.00165 * slack.max() + 2 * 0.0029) * np.linalg.norm(out)
    assert np.abs(c.lse.item() - lse.item()) <= 2.0 ** -8 * slack.max() + 2.0 ** -20 * (1 + abs(lse.item()))


def test_one_key_is_its_own_result():
    """A token that sees itself alone: out = w_uv c, lse = its score."""
    Case([6, 1], [0, 0], 8, 16, mask=[1 << i for i in range(6)] + [1]).check()


def test_causal_equals_the_mask_that_says_so():
    c = Case([7, 33, 2], [100, 255, 0], 16, 16, mask="causal")
    mla.check(c.call())
    d = Case([7, 33, 2], [100, 255, 0], 16, 16, mask=[(2 << i) - 1 for n in (7, 33, 2) for i in range(n)])
    mla.check(d.call())
    assert torch.equal(c.out, d.out) and torch.equal(c.lse, d.lse)


def test_bits_past_the_chunk_mean_nothing():
    c = Case([3, 2], [20, 0], 4, 16, mask=[1, 3, 5, 1, 2])
    mla.check(c.call())
    d = Case([3, 2], [20, 0], 4, 16, mask=[1 | 8 << 20, 3 | 16, 5 | 1 << 60, 1 | 12, 2 | 1 << 33], words=3)
    mla.check(d.call())
    assert torch.equal(c.out, d.out) and torch.equal(c.lse, d.lse)


def test_equal_to_decode_on_single_tokens():
    """mla_decode's result within both calls' roundings."""
    c = Case([1] * 5, [500, 3, 64, 1000, 128], 16, 64, mask="causal", sink=True)
    mla.check(c.call())
    out, lse = torch.zeros_like(c.out), torch.zeros_like(c.lse)
    iro, cached, table = c.ints
    parts = mla.mla_decode_partitions(c.B, c.H, 1, 1001)
    n = mla.mla_decode_workspace_bytes(c.H, c.T, parts)
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)
    kv = torch.nan_to_num(c.kv_d)                    # the decode reads whole tiles
    mla.check(mla.mla_decode(out, lse, c.q_d, iro, cached, kv, table, c.num, c.page, c.most, c.uk_d, c.uv_d, c.B, c.H,
                             c.T, 1, 1001, 0, c.scale, attn_sink=c.sink_d, workspace=ws, workspace_bytes=n,
                             d_status=c.st))
    assert c.st.item() == 0
    a, b = c.out.double(), out.double()
    assert ((a - b).norm() / b.norm()).item() <= 2 * WHOLE and (c.lse - lse).abs().max().item() <= 5e-3


def test_without_lse_and_repeated_calls_are_the_same_bits():
    c = Case([9, 3, 20], [3000, 10, 700], 16, 64)
    c.check()
    out = c.out.clone()
    for _ in range(3):
        c.out.fill_(FILL)
        mla.check(c.call(lse=False))
        assert torch.equal(c.out, out)


def test_captured_replayed_and_on_two_streams():
    """A graph replayed on other inputs, and two calls at once with workspaces of their own."""
    a, b = Case([5, 8], [900, 60], 8, 32, seed=1), Case([6, 7], [80, 1200], 8, 32, seed=2)
    a.check(), b.check()
    want = a.out.clone(), b.out.clone()
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for c in (a, b):
        c.out.fill_(FILL)
    torch.cuda.synchronize()
    mla.check(a.call(stream=s)), mla.check(b.call(stream=t))
    torch.cuda.synchronize()
    assert torch.equal(a.out, want[0]) and torch.equal(b.out, want[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mla.check(a.call())
    for scale in (1.0, 0.5):
        a.q_d.mul_(scale)
        a.q = a.q_d.double().cpu().numpy()
        a.out.fill_(FILL)
        g.replay()
        torch.cuda.synchronize()
        a.compare(*a.oracle())


def test_left_out_sequences():
    """Offsets past the tokens, more tokens than the mask has bits: those rows stay."""
    c = Case([3, 40, 2], [20, 30, 5], 4, 16, words=1)
    mla.check(c.call())
    assert c.st.item() == mla.MLA_DEV_BAD_OFFSETS
    out, lse, slack = c.oracle()
    lse[3:43] = np.nan
    c.compare(out, lse, slack)
    c = Case([3, 4], [20, 30], 4, 16)
    c.T -= 1
    mla.check(c.call())
    assert c.st.item() == mla.MLA_DEV_BAD_OFFSETS
    out, lse, slack = c.oracle()
    lse[3:] = np.nan
    c.compare(out, lse, slack)


@pytest.mark.parametrize("iro", [[0, 5, 3, 7], [1, 3, 5, 7], [0, 3, 7, 1 << 31]])
def test_offsets_that_are_none(iro):
    c = Case([3, 2, 2], [20, 30, 40], 4, 16)
    c.ints[0] = dev(np.array(iro, dtype=np.int64).astype(np.uint32).view(np.int32))
    mla.check(c.call())
    assert c.st.item() == mla.MLA_DEV_BAD_OFFSETS
    if iro[0] == 0 and iro[2] == 7:
        assert (c.out != FILL).any()
    else:
        assert (c.out == FILL).all() and (c.lse == FILL).all()


def test_a_missing_page_is_reported_and_harms_no_other_sequence():
    c = Case([3, 2], [100, 100], 4, 16)
    out, lse, slack = c.oracle()
    for entry in (-1, c.num, 1 << 30):
        table = c.table.copy()
        table[0, 2] = entry
        c.ints[2] = dev(table)
        c.st.zero_(), c.out.fill_(FILL), c.lse.fill_(FILL)
        mla.check(c.call())
        assert c.st.item() == mla.MLA_DEV_BAD_PAGE
        c.out[:3], c.lse[:3] = FILL, FILL
        lse[:3] = np.nan
        c.compare(out, lse, slack)


def test_a_nan_key_is_nan_for_those_who_see_it():
    c = Case([4], [40], 4, 16, mask=[1, 2, 4, 8])
    j = 42                                         # new token 2
    c.kv_d[int(c.table[0, j // 16]) * 16 + j % 16, 530] = float("nan")
    mla.check(c.call())
    nan = torch.isnan(c.out).any(-1).any(-1).tolist()
    assert nan[2] and torch.isnan(c.out[2]).all()


def test_a_timeout_before_stops_the_call():
    c = Case([4], [40], 4, 16)
    c.st.fill_(mla.MLA_DEV_TIMEOUT)
    mla.check(c.call())
    assert (c.out == FILL).all() and (c.lse == FILL).all()


def test_a_speculative_step():
    """The calls of one step in a row: two prompts are continued twice each, drafts are written at their depths,
    attend as trees, the accepted ones move together, what was reserved for the others is given back, the pool is
    compacted, and the next token decodes: as the same tokens do in caches of their own."""
    rng = np.random.default_rng(11)
    page, H, most, pool, B = 8, 4, 8, 40, 4
    L0, parents, n_draft = [19, 24], [0, 0, 1, 1], 6
    up = [-1, 0, 0, 1, 3, 2]
    depth, mask = [], []
    for i, u in enumerate(up):
        depth.append(0 if u < 0 else depth[u] + 1)
        mask.append(1 << i | (mask[u] if u >= 0 else 0))
    kept = [[0, 1, 3], [0, 2, 5], [0], [0, 1, 3, 4]]                      # paths from the root
    ang = np.arange(64)[:, None] * 10000.0 ** (-np.arange(32) / 32)
    freqs = torch.from_numpy(np.stack([np.cos(ang), np.sin(ang)], -1).reshape(64, 64)).float().to(DEV)
    gamma = torch.ones(512, device=DEV)
    kv = torch.full((pool * page, 576), float("nan"), dtype=torch.bfloat16, device=DEV)
    uk, uv = bf16(rng.standard_normal((H, 512, 128)) * 512 ** -0.5), bf16(rng.standard_normal((H, 128, 512)) * 512 ** -0.5)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    table, refs, lengths = dev(np.full((2, most), -1)), dev(np.zeros(pool)), dev([0, 0])
    src, dst, cnt = dev(np.zeros(pool)), dev(np.zeros(pool)), dev([0])
    size = mla.mla_pages_workspace_bytes(pool, B)
    ws = torch.empty(size, dtype=torch.uint8, device=DEV)

    def reserve(t, n, new, b):
        mla.check(mla.mla_pages_reserve(t, refs, n, dev(new), src, dst, cnt, pool, page, most, b, ws, size, st))
        mla.check(mla.mla_pages_copy(kv, page * 1152, 1, 0, src, dst, cnt, pool, pool, st))

    def write(t, n, lat, iro, b, q=None, positions=None):
        rest = (dev(iro), n, t, pool, page, most, b, H, len(lat), 64, 1e-6, 1.0, mla.MLA_BF16, st)
        if positions is None:
            mla.check(mla.mla_latent_cache_write(kv, q, lat, gamma, freqs, *rest))
        else:
            mla.check(mla.mla_latent_cache_write_at(kv, q, lat, gamma, freqs, dev(positions), *rest))

    prompt = bf16(rng.standard_normal((sum(L0), 576)))[0]
    reserve(table, lengths, L0, 2)
    write(table, lengths, prompt, [0, L0[0], sum(L0)], 2)
    lengths = dev(L0)
    t2, n2 = dev(np.zeros((B, most))), dev(np.zeros(B))
    mla.check(mla.mla_pages_fork(t2, n2, table, lengths, refs, dev(parents), pool, most, B, 2, st))
    reserve(t2, n2, [n_draft] * B, B)
    iro = np.arange(B + 1) * n_draft
    drafts = bf16(rng.standard_normal((B * n_draft, 576)))[0]
    q_raw = bf16(rng.standard_normal((B * n_draft, H, 192)))[0]
    q = q_raw.clone()
    at = np.concatenate([[L0[p] + d for d in depth] for p in parents])
    write(t2, n2, drafts, iro, B, q, at)
    words = dev(np.array(mask * B)[:, None])
    out, lse = torch.zeros(B * n_draft, H, 128, dtype=torch.bfloat16, device=DEV), torch.zeros(B * n_draft, H, device=DEV)
    nb = mla.mla_chunk_attention_workspace_bytes(B, H, B * n_draft)
    cws = torch.empty(nb, dtype=torch.uint8, device=DEV)

    def attend(qq, t, n, i, o, l, m=None):
        mla.check(mla.mla_chunk_attention(o, l, qq, dev(i), n, kv, t, pool, page, most, uk[0], uv[0], len(i) - 1, H, len(qq),
                                          192 ** -0.5, chunk_mask=m, mask_words=0 if m is None else 1, workspace=cws,
                                          workspace_bytes=nb, d_status=st))
    attend(q, t2, n2, iro, out, lse, words)
    # The accepted rows, the rest given back, the pool compacted.
    width = max(map(len, kept))
    pad = dev([k + [-1] * (width - len(k)) for k in kept])
    counts = dev([len(k) for k in kept])
    mla.check(mla.mla_cache_keep_rows(kv, 1152, 1, 0, n2, pad, width, counts, t2, pool, page, most, B, st))
    n2 += counts
    mla.check(mla.mla_pages_free(t2, refs, n2, n2, pool, page, most, B, st))
    mla.check(mla.mla_pages_compact(t2, refs, src, dst, cnt, pool, pool, most, B, ws, size, st))
    mla.check(mla.mla_pages_copy(kv, page * 1152, 1, 0, src, dst, cnt, pool, pool, st))
    assert st.item() == 0
    live = int((refs > 0).sum())
    assert (refs[:live] > 0).all() and np.array_equal(np.bincount(t2[t2 >= 0].cpu(), minlength=pool), refs.cpu())
    # Each sequence's rows are those of its text written in a row.
    for b in range(B):
        p = parents[b]
        L = L0[p] + len(kept[b])
        lat = torch.cat([prompt[L0[0] * p: L0[0] * p + L0[p]], drafts[[b * n_draft + k for k in kept[b]]]])
        own = torch.zeros(8 * page, 576, dtype=torch.bfloat16, device=DEV)
        mla.check(mla.mla_latent_cache_write(own, None, lat, gamma, freqs, dev([0, L]), dev([0]), dev([np.arange(8)]), 8, page,
                                             8, 1, H, L, 64, 1e-6, 1.0, mla.MLA_BF16, st))
        j = np.arange(L)
        rows = t2[b].cpu().numpy()[j // page] * page + j % page
        assert torch.equal(kv[rows], own[:L])
        # Each accepted draft saw the prompt and the path behind it: the causal chunk of the kept rows.
        qk = q[[b * n_draft + k for k in kept[b]]].contiguous()
        o, l = torch.zeros(len(kept[b]), H, 128, dtype=torch.bfloat16, device=DEV), torch.zeros(len(kept[b]), H, device=DEV)
        attend(qk, t2[b: b + 1].contiguous(), dev([L0[p]]), [0, len(kept[b])], o, l)
        want = out[[b * n_draft + k for k in kept[b]]].double()
        assert ((o.double() - want).norm() / want.norm()).item() <= 2 * WHOLE
        assert (l - lse[[b * n_draft + k for k in kept[b]]]).abs().max().item() <= 1e-5
    assert st.item() == 0


def poisoned(c, j, columns, value):
    """Context position j of sequence 0 with a value that is no finite number in some columns."""
    row = int(c.table[0, j // c.page]) * c.page + j % c.page
    c.kv_d[row, columns] = value


@pytest.mark.parametrize("page", [64, 16])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("columns", [slice(0, 512), slice(7, 8), slice(511, 512), slice(512, 576), slice(575, 576)])
@pytest.mark.parametrize("mask", ["tree", "causal"])
def test_a_key_that_is_no_number_does_not_reach_who_does_not_see_it(mask, columns, value, page):
    """New token 5 of 9, hidden from the tokens before it and (tree) from its siblings' branches; everything else as
    without it."""
    c = Case([9, 2], [190, 300], 4, page, mask=mask, seed=3)
    out, lse, slack = c.oracle()
    poisoned(c, 195, columns, value)
    mla.check(c.call())
    sees = [i >= 5 if c.mask is None else bool(c.mask[i] >> 5 & 1) for i in range(9)]
    assert any(sees) and not all(sees)
    got, l = c.out.clone(), c.lse.clone()
    for i in range(9):
        if sees[i]:
            if columns.stop <= 512:
                assert torch.isnan(got[i]).all() and torch.isnan(l[i]).all()
            c.out[i], c.lse[i] = FILL, FILL
            lse[i] = np.nan
    c.compare(out, lse, slack)


def test_keys_that_are_no_numbers_in_a_long_chunk():
    """Among 200 new tokens over several groups of 64, each seen by itself alone."""
    n = 200
    c = Case([3, n], [40, 77], 2, 64, mask=[1, 2, 4] + [1 << i for i in range(n)], words=7)
    out, lse, slack = c.oracle()
    odd = [0, 1, 31, 32, 50, 63, 64, 120, 179, 180, 199]
    for m in odd:
        j = 77 + m
        c.kv_d[int(c.table[1, j // 64]) * 64 + j % 64, m % 512] = float("nan") if m % 2 else float("inf")
    mla.check(c.call())
    for m in odd:
        assert torch.isnan(c.out[3 + m]).all() and torch.isnan(c.lse[3 + m]).all()
        c.out[3 + m], c.lse[3 + m] = FILL, FILL
        lse[3 + m] = np.nan
    c.compare(out, lse, slack)


def test_the_largest_numbers_are_numbers():
    """The largest bf16 among a hidden row's values: no part of it reaches the others."""
    c = Case([4], [100], 2, 16, mask=[1, 2, 4, 8])
    out, lse, slack = c.oracle()
    poisoned(c, 102, slice(0, 512), 3.3895e38)
    mla.check(c.call())
    c.out[2], c.lse[2] = FILL, FILL
    lse[2] = np.nan
    c.compare(out, lse, slack)


def test_thousands_of_sequences():
    """More than the plan holds in shared memory, most of them without new tokens."""
    rng = np.random.default_rng(8)
    Case(list((rng.random(5000) < 0.3).astype(int) * rng.integers(1, 4, 5000)), list(rng.integers(0, 20, 5000)), 2, 16,
         mask="any").check()


@pytest.mark.parametrize("empty", [30, 31, 32, 33, 200])
def test_odd_keys_behind_sequences_without_tokens(empty):
    """Tokens 3 and 4 are neighbours in the batch with many sequences between them."""
    new = [4] + [0] * empty + [3, 0, 2]
    c = Case(new, [20] + [1] * empty + [30, 5, 40], 3, 16, mask=[1, 2, 4, 8] + [1, 2, 4] + [1, 2])
    out, lse, slack = c.oracle()
    for b, m, t in ((0, 3, 3), (empty + 1, 1, 5), (empty + 3, 0, 7)):
        j = c.cached[b] + m
        c.kv_d[int(c.table[b, j // 16]) * 16 + j % 16, 5] = float("nan")
        lse[t] = np.nan
    mla.check(c.call())
    for t in (3, 5, 7):
        assert torch.isnan(c.out[t]).all() and torch.isnan(c.lse[t]).all()
        c.out[t], c.lse[t] = FILL, FILL
    c.compare(out, lse, slack)


@pytest.mark.parametrize("B", [1, 4, 20, 60, 250])
def test_a_long_sequence_among_short_ones(B):
    """Row tiles of many parts, of one and of none, however many row tiles there are."""
    rng = np.random.default_rng(B)
    cached = list(rng.integers(0, 400, B))
    cached[B // 2] = 9000
    Case(list(rng.integers(1, 30, B)), cached, 8, 64, seed=B, sink=True).check()


@pytest.mark.parametrize("size", ["any"], indirect=True)
def test_a_call_that_takes_longer_than_a_wait_may(size):
    """Waits are limited to two seconds each, calls are not: 4096 tokens over a context of small pages, which hold the
    same few rows again and again.  out is as over those rows once, with how often each is seen as its weight.
    The products are added up in fp32, at most 2^-23 off each of the 16 steps of a tile; the sums of the weights,
    128 a tile and thread, by half of that to either side, of which eight times the root mean square is allowed."""
    rng = np.random.default_rng(4)
    H, T, pool, cached = 128, 4096, 4096, 800000
    kv_d, kv = bf16(rng.standard_normal((pool, 576)))
    q_d = torch.randn(T, H, 192, device=DEV, generator=torch.Generator(DEV).manual_seed(1)).to(torch.bfloat16)
    uk_d, uk = bf16(rng.standard_normal((H, 512, 128)) * 512 ** -0.5)
    uv_d, uv = bf16(rng.standard_normal((H, 128, 512)) * 512 ** -0.5)
    table = dev(rng.permutation(pool)[np.arange(cached + T) % pool][None])
    iro, lengths, st = dev([0, T]), dev([cached]), dev([0])
    out, lse = torch.full((T, H, 128), FILL, dtype=torch.bfloat16, device=DEV), torch.full((T, H), FILL, device=DEV)
    size = mla.mla_chunk_attention_workspace_bytes(1, H, T)
    ws = torch.empty(size, dtype=torch.uint8, device=DEV)
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    begin.record()
    mla.check(mla.mla_chunk_attention(out, lse, q_d, iro, lengths, kv_d, table, pool, 1, cached + T, uk_d, uv_d, 1, H, T,
                                      192 ** -0.5, workspace=ws, workspace_bytes=size, d_status=st))
    end.record()
    torch.cuda.synchronize()
    assert st.item() == 0
    assert begin.elapsed_time(end) > 2000, "the call no longer takes as long as this test needs it to"
    order = table[0, :pool].cpu().numpy()
    for t, h in ((0, 0), (0, 77), (1777, 5), (T - 1, 127)):
        q, seen = q_d[t, h].double().cpu().numpy(), cached + t + 1
        times = np.empty(pool)
        times[order] = seen // pool + (np.arange(pool) < seen % pool)
        lat = uk[h] @ q[:128]
        s = 192 ** -0.5 * (kv[:, :512] @ lat + kv[:, 512:] @ q[128:])
        w = times * np.exp(s - s.max())
        want = uv[h] @ (w @ kv[:, :512] / w.sum())
        got = out[t, h].double().cpu().numpy()
        assert np.linalg.norm(got - want) <= (ROW + 16 * (seen / 256 + 1) * 2.0 ** -23) * np.linalg.norm(want)
        slack = 192 ** -0.5 * (np.abs(kv[:, :512]) @ np.abs(lat)).max()
        assert abs(lse[t, h].item() - (s.max() + np.log(w.sum()))) <= (
            2.0 ** -8 * slack + 8 * np.sqrt(seen / 2) * 2.0 ** -24)


def infinite_keys(c, js, column, logit):
    """Cached positions js of the only token, head 0, with an infinite value in a latent column, so that their logits
    are logit (+-infinity); (out, lse) of what is left."""
    lat = c.uk[0] @ c.q[0, 0, :128]
    for j in js:
        poisoned(c, j, slice(column, column + 1), float(np.sign(lat[column])) * logit)
    rest = np.setdiff1d(np.arange(c.cached[0] + 1), js)
    at = c.table[0, rest // c.page] * c.page + rest % c.page
    s = c.scale * (c.kv[at, :512] @ lat + c.kv[at, 512:] @ c.q[0, 0, 128:])
    slack = c.scale * (np.abs(c.kv[at, :512]) @ np.abs(lat)).max()
    return s.max() + np.log(np.exp(s - s.max()).sum()), slack


@pytest.mark.parametrize("logit", [-np.inf, np.inf])
@pytest.mark.parametrize("column", [0, 200, 511])
@pytest.mark.parametrize("cached,js", [
    (700, [3]), (700, [699]), (700, range(256)), (700, range(128)), (700, range(256, 512)), (700, range(512, 700)),
    (20000, range(256)), (20000, range(128, 256)), (20000, range(512, 1024)), (20000, [19000]), (20000, range(20000))])
def test_a_cached_key_with_an_infinite_value_is_nan_for_all(cached, js, column, logit):
    """Also where its logit, -infinity, is all that a tile or a part of the line has: softmax of it is 0, and 0 times
    infinity is no number."""
    c = Case([1, 1], [cached, 9], 1, 64, mask="causal", seed=cached + column)
    want, slack = infinite_keys(c, js, column, logit)
    mla.check(c.call())
    assert c.st.item() == 0
    assert torch.isnan(c.out[0]).all() and torch.isfinite(c.out[1]).all() and torch.isfinite(c.lse[1]).all()
    if logit > 0:
        assert torch.isnan(c.lse[0]).all()
    else:
        assert abs(c.lse[0].item() - want) <= 2.0 ** -8 * slack + 2.0 ** -20 * (1 + abs(want))


@pytest.mark.parametrize("B", [1, 160])
def test_no_number_is_forgotten_when_the_maximum_jumps(B):
    """A key of weight 0 with an infinite value, then keys that are above all before them by more than 2^-126 leaves."""
    c = Case([1] * B, [700] * B, 1, 64, mask="causal", seed=2)
    lat = c.uk[0] @ c.q[0, 0, :128]
    j = np.arange(300, 701)
    at = c.table[0, j // 64] * 64 + j % 64
    rows = c.kv.copy()
    rows[at, :512] += 250 / c.scale * lat / (lat @ lat)
    c.kv_d, c.kv = bf16(rows)
    infinite_keys(c, [5], 17, -np.inf)
    mla.check(c.call())
    assert torch.isnan(c.out[0]).all() and torch.isfinite(c.out[1:]).all() and torch.isfinite(c.lse).all()


def test_a_key_that_is_cached_and_no_number():
    """NaN in a latent or rope column, of one sequence's context: nobody else's."""
    for column in (0, 511, 512, 575):
        c = Case([3, 2, 1], [500, 300, 40], 8, 16, sink=True)
        out, lse, slack = c.oracle()
        poisoned(c, 77, slice(column, column + 1), float("nan"))
        mla.check(c.call())
        assert torch.isnan(c.out[:3]).all() and torch.isnan(c.lse[:3]).all()
        c.out[:3], c.lse[:3] = FILL, FILL
        lse[:3] = np.nan
        c.compare(out, lse, slack)


@pytest.mark.parametrize("sink", [True, False])
@pytest.mark.parametrize("long", [0, 1, 1 << 20, 1 << 30])
def test_a_context_longer_than_its_pages_is_left_out(long, sink):
    """A wrong length beside good ones: its rows stay, theirs are right.  (At 0 the context
    ends with the last page of the row.)"""
    c = Case([3, 2, 4], [100, 100, 3], 4, 16, sink=sink)
    out, lse, slack = c.oracle()
    cached = list(c.cached)
    cached[1] = c.most * c.page - 2 + long
    c.ints[1] = dev(cached)
    mla.check(c.call())
    assert c.st.item() == mla.MLA_DEV_BAD_PAGE
    if long:
        assert (c.out[3:5] == FILL).all() and (c.lse[3:5] == FILL).all()
    else:
        assert (c.out[3:5] != FILL).any()            # (pages are missing, but there is room for them)
        c.out[3:5], c.lse[3:5] = FILL, FILL
    lse[3:5] = np.nan
    c.compare(out, lse, slack)


@pytest.mark.parametrize("size", ["any"], indirect=True)
@pytest.mark.parametrize("H,many", [(128, 600), (1, 300)])
def test_more_tiles_than_are_counted(H, many):
    """Contexts of 2^31 keys on one page again and again: for 300 pairs of row tiles of one sequence, and for the one
    row tile of each of 300 sequences, the tiles do not fit 31 bits.  Nothing is worked at, and all rows stay."""
    one = H > 1
    new, page, most = [many] if one else [1] * many, 1 << 16, 1 << 15
    c = Case([2], [30], H, 16, mask="causal")
    T = sum(new)
    iro, cached = dev(np.concatenate([[0], np.cumsum(new)])), dev([(1 << 31) - 8192 - n for n in new])
    kv, table = torch.zeros(page, 576, dtype=torch.bfloat16, device=DEV), dev(np.zeros((len(new), most)))
    q = torch.zeros(T, H, 192, dtype=torch.bfloat16, device=DEV)
    out, lse = torch.full((T, H, 128), FILL, dtype=torch.bfloat16, device=DEV), torch.full((T, H), FILL, device=DEV)
    size = mla.mla_chunk_attention_workspace_bytes(len(new), H, T)
    ws = torch.empty(size, dtype=torch.uint8, device=DEV)
    mla.check(mla.mla_chunk_attention(out, lse, q, iro, cached, kv, table, 1, page, most, c.uk_d, c.uv_d, len(new), H, T,
                                      1.0, workspace=ws, workspace_bytes=size, d_status=c.st))
    assert c.st.item() == mla.MLA_DEV_BAD_OFFSETS
    assert (out == FILL).all() and (lse == FILL).all()
    c.st.zero_()
    c.check()


@pytest.mark.parametrize("value", [np.inf, np.nan])
def test_a_sink_that_is_no_number(value):
    """No weights can be told: NaN, as in the definition, whether a row tile is split (the long context) or not."""
    c = Case([2, 3] + [1] * 160, [20000, 9] + [40] * 160, 4, 64, sink=True)
    c.sink[[0, 1, 50]] = value
    c.make_buffers()
    out, lse, slack = c.oracle()
    mla.check(c.call())
    bad = [0, 1, 2, 3, 4, 5 + 48]
    assert np.isnan(out[bad]).all() and torch.isnan(c.out[bad]).all() and torch.isnan(c.lse[bad]).all()
    c.out[bad], c.lse[bad] = FILL, FILL
    lse[bad] = np.nan
    c.compare(out, lse, slack)


def exact_queries(H):
    """(w_uk, projected): every latent column takes one of the 128 query values, with a sign, so that the projected
    query is a bf16 number and no rounding of it is in a result."""
    uk = np.zeros((H, 512, 128))
    k = np.arange(512)
    uk[:, k, k % 128] = np.where(k // 128 % 2, -1.0, 1.0)
    return bf16(uk)


class Ranked:
    """Sequences of one token each that share their pages, in orders of their own: the keys' logits rise (or fall, or
    go up and down by pages) by far more than a reference bears, many times within the tiles that a pair walks.

    Logits are scale * q . (noise + at[j] u): the queries have u's direction in common.  The projected query is exact
    (exact_queries), so that no rounding of it moves a logit; what is left are the weights' and the output's."""

    def __init__(self, B, L, H, order, reach=40, page=64, seed=0, spikes=0.0):
        rng = np.random.default_rng(seed)
        self.B, self.L, self.H, self.page = B, L, H, page
        pages = -(-(L + 1) // page)
        base = rng.standard_normal(128)
        lat = np.concatenate([base, -base, base, -base])
        noise = rng.standard_normal((pages * page, 576))
        at = np.linspace(-1, 1, pages * page) * reach / 192 ** -0.5 / np.linalg.norm(lat)
        if spikes:
            at[:] = 0.0
            at[rng.choice(len(at), 6, replace=False)] = spikes * (1 - 0.1 * np.arange(6)) / 192 ** -0.5 / np.linalg.norm(lat)
        noise[:, :512] += at[:, None] * lat / np.linalg.norm(lat)
        self.kv_d, self.kv = bf16(noise)
        rows = np.arange(pages)
        self.table = np.stack([{"up": rows, "down": rows[::-1], "mixed": rng.permutation(pages)}[order] for _ in range(B)])
        self.cached = rng.integers(L // 2, L + 1, B)
        self.cached[0] = L
        q = rng.standard_normal((B, H, 192)) * 0.1
        q[..., :128] += base
        self.q_d, self.q = bf16(q)
        self.uk_d, self.uk = exact_queries(H)
        self.uv_d, self.uv = bf16(rng.standard_normal((H, 128, 512)) * 512 ** -0.5)

    def check(self):
        B, H, scale = self.B, self.H, 192 ** -0.5
        out = torch.full((B, H, 128), FILL, dtype=torch.bfloat16, device=DEV)
        lse, st = torch.full((B, H), FILL, device=DEV), dev([0])
        size = mla.mla_chunk_attention_workspace_bytes(B, H, B)
        ws = torch.randint(0, 256, (size,), dtype=torch.uint8, device=DEV)
        mla.check(mla.mla_chunk_attention(out, lse, self.q_d, dev(np.arange(B + 1)), dev(self.cached), self.kv_d,
                                          dev(self.table), len(self.kv) // self.page, self.page, self.table.shape[1],
                                          self.uk_d, self.uv_d, B, H, B, scale, workspace=ws, workspace_bytes=size,
                                          d_status=st))
        assert st.item() == 0
        out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
        off, whole, heaviest = 0.0, 0.0, []
        for b in range(B):
            j = np.arange(self.cached[b] + 1)
            c = self.kv[self.table[b, j // self.page] * self.page + j % self.page]
            for h in range(H):
                lat = self.uk[h] @ self.q[b, h, :128]
                assert np.array_equal(lat, bf16(lat)[1])
                s = scale * (c[:, :512] @ lat + c[:, 512:] @ self.q[b, h, 128:])
                p = np.exp(s - s.max())
                total = p.sum()
                mix = p @ c[:, :512] / total
                want = self.uv[h] @ mix
                # Weights and output are off by 0.00165 each, independent of each other (see above); a weight's
                # part goes by its own key.  A logit is off by at most fp32's 2^-23 of the terms' sizes in each of
                # 36 steps of 16, and a quarter of that again in the exponent.
                each = 0.00165 * np.sqrt(((p[:, None] * (c[:, :512] - mix)) ** 2).sum()) / total
                fp32 = 45 * 2.0 ** -23 * scale * (np.abs(c[:, :512]) @ np.abs(lat)).max()
                moved = fp32 * (p @ np.abs(c[:, :512] - mix)) / total
                bound = 4 * (each + 0.00165 * np.linalg.norm(want)) + 2 * np.linalg.norm(moved)
                miss = np.linalg.norm(out[b, h] - want)
                assert miss <= bound, (b, h, miss, bound)
                assert abs(lse[b, h] - s.max() - np.log(total)) <= fp32 + 2.0 ** -20 * (1 + abs(lse[b, h]))
                off, whole = off + miss ** 2, whole + want @ want
                heaviest.append(1 / total)
        return np.sqrt(off / whole), np.array(heaviest)


@pytest.mark.parametrize("order", ["up", "down", "mixed"])
@pytest.mark.parametrize("B,L", [(160, 2500), (80, 5000), (1, 40000)])
def test_references_that_move_many_times(B, L, order):
    """Whole row tiles that a pair walks alone, and one cut into many parts: no key is lost on the way."""
    off, heaviest = Ranked(B, L, 2, order, reach=40 * max(1.0, L / 10000), seed=L).check()
    assert off <= WHOLE and heaviest.max() < 0.9


@pytest.mark.parametrize("order", ["up", "mixed"])
@pytest.mark.parametrize("B,L", [(160, 2500), (1, 40000)])
def test_a_key_that_takes_all_the_weight(B, L, order):
    """A few keys 100 to 200 above all others and 20 apart: what comes before and behind the highest has no part in
    the result."""
    off, heaviest = Ranked(B, L, 2, order, seed=L, spikes=200.0).check()
    assert off <= WHOLE and (heaviest > 0.999).all()


@pytest.mark.parametrize("H", [129, 160, 256])
def test_more_heads_than_a_row_tile_has_rows(H):
    """A token's heads lie in two or three row tiles."""
    Case([2, 3], [70, 400], H, 16, seed=H, sink=True).check()


@pytest.mark.parametrize("mask", ["tree", "causal"])
def test_contexts_on_shared_pages(mask):
    """Samples of one prompt: 12 sequences hold its 47 full pages in common and one page of their own."""
    c = Case([6] * 12, [3010] * 12, 16, 64, mask=mask)
    c.table[:, :47] = c.table[0, :47]
    c.make_buffers()
    c.check()
