"""GPU tests of the 8-bit latent cache (write, gather, fused prefill, decode)
against the float64 oracle, through the C ABI.

Tolerances.
* Codes: a kernel may differ from the oracle only where the unrounded value is
  within its fp32 error (a few 2^-24 of the value; 2^-20 allowed) of a rounding
  border, so |code - y / s| <= half a step (2^-4 of the value, 2^-10 below the
  normal range) + 2^-20 |y / s|.  Scales are equal: the tests' largest values
  stay 2^-20 away from the borders 448 * 2^k.
* Rotated queries: half a bf16 step, 2^-8 of the value, and the fp32 error of
  the two products, 2^-22 (|re| + |im|).
* Decode, 2-norm over all outputs: three roundings that are no larger than a
  bf16 one (the query terms, the weight terms and the output: each at most 2^-8
  of the value, so sqrt(1/3) 2^-8 in the mean for errors spread evenly, and a
  score error is the query error times the scores' spread, at most 1 here
  unless said) give sqrt(3) * sqrt(1/3) 2^-8 = 2^-8.  LSE: within 5e-3.
"""
import numpy as np
import pytest
import torch

import mla_prefill_attention_plan_gb300 as mla
import oracle as O
from oracle import q8
from workloads import WORKLOADS, make_cache_write_operands, make_inputs, scaled

pytestmark = pytest.mark.gpu
DEV = "cuda"
REL, LSE_ABS = 2.0 ** -8, 5e-3


@pytest.fixture(scope="module", autouse=True)
def _built():
    from mla_prefill_attention_plan_gb300 import build
    build.build()
    mla.load()


def pages(new, cached, page, seed=0, extra=0):
    """Shuffled page table of every sequence's context."""
    rng = np.random.default_rng(seed)
    need = [-(-(n + c) // page) for n, c in zip(new, cached)]
    num = max(1, sum(need) + extra)
    order = rng.permutation(num)
    table = np.full((len(new), max(1, max(need))), -1, np.int64)
    at = 0
    for b, k in enumerate(need):
        table[b, :k] = order[at: at + k]
        at += k
    return table, num


def i32(x):
    return torch.as_tensor(np.asarray(x, np.int32)).to(DEV)


def offsets(new):
    return np.concatenate([[0], np.cumsum(new)]).astype(np.int64)


def status():
    return torch.zeros(1, dtype=torch.int32, device=DEV)


def fp8(codes):
    return torch.from_numpy(np.ascontiguousarray(codes)).to(DEV)


def random_cache(num, page, sb, seed=0, lo=-9, hi=-5, powers=True):
    """Codes of about N(0, 1) / s and scales 2^lo .. 2^hi (or any numbers there)."""
    rng = np.random.default_rng(seed)
    e = rng.integers(lo, hi + 1, (num, page // sb)).astype(np.float64) if powers else rng.uniform(lo, hi, (num, page // sb))
    scales = np.exp2(e).astype(np.float32)
    x = rng.standard_normal((num, page, 576)) / np.repeat(scales, sb, 1)[:, :, None]
    return O.e4m3_encode(x), scales


# ------------------------------------------------------------------ write

def check_write(new, cached, page, sb, H, seed=0, T_extra=0, spread=1.0, with_q=True):
    table, num = pages(new, cached, page, seed, extra=1)
    iro, T = offsets(new), int(sum(new))
    rng = np.random.default_rng(seed)
    codes, scales = random_cache(num, page, sb, seed)
    w = scaled(WORKLOADS["tiny_ragged"], H=H, seed=seed)
    max_seq = max(n + c for n, c in zip(new, cached))
    lat, gamma, freqs = make_cache_write_operands(w, T + T_extra, max_seq)
    # Rope rows of very different sizes make the blocks' scales differ (the
    # latent part is normalised).
    lat[:, 512:] = (lat[:, 512:].float() * torch.from_numpy(np.exp(rng.uniform(0, spread, (T + T_extra, 1)))).float()).bfloat16()
    q = torch.from_numpy(rng.standard_normal((T + T_extra, H, 192))).to(torch.bfloat16)
    kv, sc, dq, st = fp8(codes), torch.from_numpy(scales).to(DEV), q.to(DEV), status()
    mla.check(mla.mla_latent_cache_write_q8(kv, sc, dq if with_q else None, lat.to(DEV), gamma.to(DEV), freqs.to(DEV),
                                            i32(iro), i32(cached), i32(table), num, page, table.shape[1], sb, len(new),
                                            H, T, max_seq, 1e-6, st))
    torch.cuda.synchronize()
    assert st.item() == 0
    y = q8.new_rows(O.decode(O.codes(lat), "bf16"), gamma.numpy(), freqs.numpy(), iro, cached, 1e-6)[:T]
    ref, ref_s, pre = q8.latent_cache_write_q8(codes, scales, y, iro, cached, table, page, sb)
    assert np.array_equal(sc.cpu().numpy(), ref_s.astype(np.float32))
    got = kv.cpu().numpy().reshape(-1, 576)
    written = np.zeros(num * page, bool)
    for b in range(len(new)):
        for i in range(new[b]):
            p, t = cached[b] + i, iro[b] + i
            row = table[b, p // page] * page + p % page
            written[row] = True
            err = np.abs(O.e4m3_decode(got[row]) - pre[t])
            # Half a step of the binade, or half of 2^-9 below the normal range.
            a = np.maximum(np.abs(pre[t]), 2.0 ** -6)
            assert np.all(err <= np.exp2(np.floor(np.log2(a)) - 4) + 2.0 ** -20 * a)
    assert np.array_equal(got[~written], ref.reshape(-1, 576)[~written])   # requantised or untouched
    if with_q:
        g = dq.float().cpu().double().numpy()
        r = O.decode(O.codes(q), "bf16")
        assert np.array_equal(g[..., :128], r[..., :128])
        assert np.array_equal(g[T:], r[T:])
        for b in range(len(new)):
            for i in range(new[b]):
                t = iro[b] + i
                x = O.rope_rotate(r[t, :, 128:], freqs.numpy()[cached[b] + i])
                size = np.abs(r[t, :, 128:]).reshape(H, 32, 2).sum(-1).repeat(2, -1)
                assert np.all(np.abs(g[t, :, 128:] - x) <= 2.0 ** -8 * np.abs(x) + 2.0 ** -22 * size)


@pytest.mark.parametrize("page,sb", [(16, 1), (16, 16), (24, 8), (100, 4), (128, 64), (256, 128), (7, 1), (1, 1)])
def test_write_ragged(page, sb):
    check_write([3, 0, 17, 1], [5, 9, 40, 0], page, sb, H=3, seed=page)


@pytest.mark.parametrize("sb", [1, 32, 128])
def test_write_long_prompts(sb):
    check_write([300, 65], [1000, 127], 128, sb, H=2, seed=sb)


def test_write_grows_scales_and_requantises():
    """Rows with rope parts up to e^6 larger than those before: the blocks'
    scales grow and the earlier rows move with them."""
    check_write([2, 9, 1], [6, 3, 15], 16, 8, H=1, seed=3, spread=6.0)


def test_write_one_token_a_call_without_queries():
    for p in (0, 1, 7, 8):
        check_write([1], [p], 16, 8, H=1, seed=p, with_q=False, spread=4.0)


def test_write_rows_behind_the_last_sequence():
    check_write([2, 3], [4, 0], 16, 4, H=2, T_extra=3)


def _small_write(new, cached, lat, page=16, sb=8, table=None, max_seq=64, T=None, kv=None, sc=None):
    T = sum(new) if T is None else T
    tab, num = pages(new, cached, page)
    tab = tab if table is None else table
    kv = torch.zeros(num, page, 576, dtype=torch.uint8, device=DEV) if kv is None else kv
    sc = torch.ones(num, page // sb, device=DEV) if sc is None else sc
    st = status()
    freqs = torch.zeros(max_seq, 64, device=DEV)
    freqs[:, 0::2] = 1
    mla.check(mla.mla_latent_cache_write_q8(kv, sc, None, lat.to(DEV), torch.ones(512, device=DEV), freqs,
                                            i32(offsets(new)), i32(cached), i32(tab), num, page, tab.shape[1], sb,
                                            len(new), 1, T, max_seq, 0.0, st))
    torch.cuda.synchronize()
    return kv, sc, int(st.item()), tab


def test_write_special_values():
    """A NaN stays out of the scale, a zero row gets the smallest one (with eps
    0 its latents are NaN, as 0 / 0), an infinite rope value the largest."""
    lat = torch.zeros(3, 576, dtype=torch.bfloat16)
    lat[:2, :512] = 1.0
    lat[0, 512] = float("nan")
    lat[1, 512] = float("inf")
    kv, sc, st, tab = _small_write([3], [0], lat, sb=1)
    assert st == 0
    s = sc.view(-1)[tab[0, 0] * 16: tab[0, 0] * 16 + 3].tolist()
    assert s == [q8.block_scale(1.0), 2.0 ** 120, 2.0 ** -60]
    rows = kv.view(-1, 576)[tab[0, 0] * 16: tab[0, 0] * 16 + 3].cpu().numpy()
    assert np.isnan(O.e4m3_decode(rows[0, 512:514])).all()        # the pair's rotation mixes the NaN in
    assert np.all(O.e4m3_decode(rows[0, :512]) * s[0] == 1.0)
    assert O.e4m3_decode(rows[1, 512:513])[0] == 448
    assert np.isnan(O.e4m3_decode(rows[2, :512])).all()


def test_write_replaces_a_scale_that_is_no_number():
    lat = torch.ones(1, 576, dtype=torch.bfloat16)
    sc = torch.full((1, 2), float("nan"), device=DEV)
    kv, sc, st, _ = _small_write([1], [3], lat, sc=sc)
    assert st == 0 and sc[0, 0].item() == q8.block_scale(1.0)
    assert kv[0, :3].abs().sum().item() == 0 and torch.isnan(sc[0, 1])


def test_write_status():
    lat = torch.ones(4, 576, dtype=torch.bfloat16)
    bad = np.array([[5]])
    kv, sc, st, _ = _small_write([2], [0], lat, table=bad)
    assert st == mla.MLA_DEV_BAD_PAGE and kv.abs().sum().item() == 0
    kv, sc, st, _ = _small_write([2], [3], lat, max_seq=4)        # the second position does not exist
    assert st == mla.MLA_DEV_BAD_OFFSETS and int((kv != 0).any(-1).sum()) == 1
    kv, sc, st, _ = _small_write([2], [0], lat, T=4)              # two tokens outside every sequence
    assert st == mla.MLA_DEV_BAD_OFFSETS and int((kv != 0).any(-1).sum()) == 2


# ------------------------------------------------------------------ gather and prefill

@pytest.mark.parametrize("page,sb,powers", [(16, 4, True), (128, 128, True), (24, 1, True), (10, 2, False)])
def test_gather_chunks(page, sb, powers):
    new, cached = [3, 40, 1], [100, 0, 77]
    table, num = pages(new, cached, page)
    codes, scales = random_cache(num, page, sb, seed=page, powers=powers)
    S, mc, B = 64, 4, 3
    bro = torch.zeros(mc, B + 1, dtype=torch.int32, device=DEV)
    co, bl = torch.zeros(mc, B, dtype=torch.int32, device=DEV), torch.zeros(mc, dtype=torch.int32, device=DEV)
    st = status()
    iro = offsets(new)
    mla.check(mla.mla_prefill_plan(bro, co, bl, i32(iro), i32(cached), B, mc, S, st))
    values = q8.q8_values(codes, scales, sb)
    ctx = np.concatenate([values[table[b, np.arange(L) // page] * page + np.arange(L) % page]
                          for b, L in enumerate(n + c for n, c in zip(new, cached))])
    for c in range(mc):
        ckv = torch.full((S, 512), 7.0, dtype=torch.bfloat16, device=DEV)
        kr = torch.full((S, 64), 7.0, dtype=torch.bfloat16, device=DEV)
        mla.check(mla.mla_gather_latent_q8(ckv, kr, fp8(codes), torch.from_numpy(scales).to(DEV), i32(table), num, page,
                                           table.shape[1], sb, bro, co, bl, c, B, S, st))
        torch.cuda.synchronize()
        n = max(0, min(S, len(ctx) - c * S))
        ref = torch.from_numpy(ctx[c * S: c * S + n]).to(torch.float32)
        assert np.array_equal(ref.double().numpy(), ctx[c * S: c * S + n]) or not powers
        got = torch.cat([ckv, kr], 1).cpu()
        if powers:
            assert torch.equal(got[:n].float(), ref)               # exact
        else:
            assert torch.all((got[:n].float() - ref).abs() <= 2.0 ** -8 * ref.abs())
        assert torch.all(got[n:] == 7.0)
    assert st.item() == 0


def test_gather_bad_page_skips_the_row():
    table, num = pages([20], [0], 16)
    codes, scales = random_cache(num, 16, 4)
    table[0, 1] = num
    ckv = torch.zeros(32, 512, dtype=torch.bfloat16, device=DEV)
    kr = torch.zeros(32, 64, dtype=torch.bfloat16, device=DEV)
    st = status()
    mla.check(mla.mla_gather_latent_q8(ckv, kr, fp8(codes), torch.from_numpy(scales).to(DEV), i32(table), num, 16, 2, 4,
                                       i32([[0, 20]]), i32([[0]]), i32([20]), 0, 1, 32, st))
    torch.cuda.synchronize()
    assert st.item() == mla.MLA_DEV_BAD_PAGE
    assert torch.all(ckv[16:] == 0) and torch.all((ckv[:16] != 0).any(1))


def test_prefill_equals_the_bf16_call_on_the_same_values():
    """The gather is exact, so the fused call's result is mla_prefill's on a bf16
    cache of the same values, bit for bit (three chunks)."""
    w = scaled(WORKLOADS["tiny_ragged"], H=4)
    inp = make_inputs(w)
    codes, scales = random_cache(inp["num_pages"], w.page_size, 8, seed=5)
    values = torch.from_numpy(q8.q8_values(codes, scales, 8)).to(torch.bfloat16).view(-1, w.page_size, 576)
    B, T, S, mc = inp["B"], inp["T_q"], w.buffer_token_size, w.max_chunks
    nbytes = mla.mla_prefill_workspace_bytes(B, w.H, T, mc, S, mla.MLA_BF16)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=DEV)
    d = {k: inp[k].to(DEV) for k in ("q", "input_row_offsets", "cache_lengths", "page_table", "w_k", "w_uv")}
    res = []
    for eight in (False, True):
        out = torch.zeros(T, w.H, 128, dtype=torch.bfloat16, device=DEV)
        lse, st = torch.zeros(T, w.H, device=DEV), status()
        head = (out, lse, d["q"], d["input_row_offsets"], d["cache_lengths"])
        tail = (d["w_k"], d["w_uv"], B, w.H, T, inp["max_prompt_len"], S, mc, inp["scale"])
        if eight:
            mla.check(mla.mla_prefill_q8(*head, fp8(codes), torch.from_numpy(scales).to(DEV), d["page_table"],
                                         inp["num_pages"], w.page_size, inp["max_pages"], 8, *tail, workspace=ws,
                                         workspace_bytes=nbytes, d_status=st))
        else:
            mla.check(mla.mla_prefill(*head, values.to(DEV), d["page_table"], inp["num_pages"], w.page_size,
                                      inp["max_pages"], *tail, workspace=ws, workspace_bytes=nbytes, d_status=st))
        torch.cuda.synchronize()
        assert st.item() == 0
        res.append((out.clone(), lse.clone()))
    assert torch.equal(res[0][0].view(torch.int16), res[1][0].view(torch.int16))
    assert torch.equal(res[0][1], res[1][1])


# ------------------------------------------------------------------ decode

class Decode:
    """A decode call's operands on the host and the device."""

    def __init__(self, new, cached, H, page=128, sb=1, seed=0, q_std=1.0, T_extra=0, **cache):
        rng = np.random.default_rng(seed)
        self.new, self.cached, self.H, self.page, self.sb = new, cached, H, page, sb
        self.table, self.num = pages(new, cached, page, seed)
        self.codes, self.scales = random_cache(self.num, page, sb, seed, **cache)
        self.iro, self.T = offsets(new), int(sum(new)) + T_extra
        bf = lambda *s, std=1.0: torch.from_numpy(rng.standard_normal(s) * std).to(torch.bfloat16)
        self.q = bf(self.T, H, 192, std=q_std)
        self.w_uk, self.w_uv = bf(H, 512, 128, std=512 ** -0.5), bf(H, 128, 512, std=512 ** -0.5)
        self.scale = 192 ** -0.5

    def rows(self, b, pos):
        pos = np.asarray(pos)
        return self.table[b, pos // self.page] * self.page + pos % self.page

    def run(self, parts=0, lists=None, topk=None, sink=None, expect=0, lse=True, table=None, max_new=None,
            max_seq=None, iro=None, T=None, stream=None):
        B = len(self.new)
        T = self.T if T is None else T
        max_new = max(self.new) if max_new is None else max_new
        max_seq = max(n + c for n, c in zip(self.new, self.cached)) if max_seq is None else max_seq
        keys = min(lists.shape[1], max_seq) if lists is not None else max_seq
        n = parts or mla.mla_decode_q8_partitions(B, self.H, max_new, keys)
        nbytes = mla.mla_decode_q8_workspace_bytes(self.H, T, n)
        ws = torch.full((nbytes,), 0xFF, dtype=torch.uint8, device=DEV)     # NaN wherever it is read unwritten
        self.out = torch.full((self.T, self.H, 128), 7.0, dtype=torch.bfloat16, device=DEV)
        self.lse = torch.full((self.T, self.H), 7.0, device=DEV) if lse else None
        st = status()
        self.dev = (self.q.to(DEV), i32(self.iro if iro is None else iro), i32(self.cached), fp8(self.codes),
                    torch.from_numpy(self.scales).to(DEV), i32(self.table if table is None else table))
        self.keep = (ws, self.w_uk.to(DEV), self.w_uv.to(DEV), None if lists is None else i32(lists),
                     None if topk is None else i32(topk), None if sink is None else torch.tensor(sink, device=DEV), st)
        q, iro_, cl, kv, sc, pt = self.dev
        self.call = lambda: mla.check(mla.mla_decode_q8(
            self.out, self.lse, q, iro_, cl, kv, sc, pt, self.num, self.page, self.table.shape[1], self.sb,
            self.keep[1], self.keep[2], B, self.H, T, max_new, max_seq, parts, self.scale, d_indices=self.keep[3],
            indices_stride=0 if lists is None else lists.shape[1], topk_lengths=self.keep[4], attn_sink=self.keep[5],
            workspace=ws, workspace_bytes=nbytes, d_status=st, stream=stream))
        torch.cuda.synchronize()
        self.call()
        torch.cuda.synchronize()
        assert st.item() == expect, mla.status_string(int(st.item()))
        return self.out.float().cpu().double().numpy(), None if not lse else self.lse.cpu().double().numpy()

    def reference(self, lists=None, topk=None, sink=None, codes=None, scales=None):
        values = q8.q8_values(self.codes if codes is None else codes, self.scales if scales is None else scales, self.sb)
        return q8.decode_values(O.decode(O.codes(self.q), "bf16"), values, self.table, self.page,
                                O.decode(O.codes(self.w_uk), "bf16"), O.decode(O.codes(self.w_uv), "bf16"), self.iro,
                                self.cached, self.scale, lists, topk, sink)

    def check(self, rel=REL, lse_abs=LSE_ABS, **kw):
        parts = kw.pop("parts", 0)
        out, lse = self.run(parts, **kw)
        compare(out, lse, *self.reference(**kw), rel=rel, lse_abs=lse_abs)


def compare(out, lse, ref, ref_lse, rel=REL, lse_abs=LSE_ABS):
    ok = ~np.isnan(ref_lse)
    assert np.all(out[~ok] == 7.0)                              # tokens outside every sequence
    assert np.isfinite(out[ok]).all()
    assert np.linalg.norm(out[ok] - ref[ok]) <= rel * np.linalg.norm(ref[ok])
    if lse is not None:
        assert np.all(lse[~ok] == 7.0)
        fin = ok & np.isfinite(ref_lse)
        assert np.array_equal(lse[ok & ~fin], ref_lse[ok & ~fin])
        assert np.abs(lse[fin] - ref_lse[fin]).max(initial=0.0) <= lse_abs


@pytest.mark.parametrize("page,sb", [(128, 64), (64, 1), (96, 32), (16, 16), (24, 8), (100, 4), (7, 7), (1, 1), (256, 128)])
@pytest.mark.parametrize("H", [3, 12, 40])
def test_decode_page_sizes(page, sb, H):
    """Runs of 128, 64 and 32 rows, and pages whose rows are copied one by one;
    the kernels of 16, 32 and 64 rows."""
    Decode([1, 2, 1, 0], [300, 127, 0, 50], H, page, sb, seed=page).check()


@pytest.mark.parametrize("H", [1, 16, 17, 32, 33, 64, 100, 128])
def test_decode_heads(H):
    Decode([1, 1, 1], [500, 129, 63], H, 64, 32, seed=H).check()


@pytest.mark.parametrize("parts", [1, 2, 5, 40])
def test_decode_partitions(parts):
    d = Decode([2, 1], [1500, 200], 8, 128, 8)
    out, lse = d.run(parts)
    compare(out, lse, *d.reference())


@pytest.mark.parametrize("H,new", [(16, [20, 3]), (1, [150, 2]), (5, [1, 33])])
def test_decode_many_new_tokens(H, new):
    """Row tiles that hold several tokens, each with its own causal limit."""
    Decode(new, [500, 64], H, 16, 16, seed=H).check(parts=2)


def test_decode_lengths_around_a_tile():
    new = [1] * 10
    Decode(new, [0, 1, 126, 127, 128, 129, 254, 255, 256, 257], 4, 16, 1).check()


@pytest.mark.parametrize("lo,hi", [(-9, 4), (-40, -38), (30, 34)])
def test_decode_scales_far_apart(lo, hi):
    """Block scales over a factor of 2^13, very small and very large ones: the
    weights that the tensor cores see carry the scale.  The queries are divided
    by the largest scale times 448 / 4, so that scores stay of order one."""
    d = Decode([1, 1], [700, 300], 8, 128, 4, lo=lo, hi=hi)
    rng = np.random.default_rng(0)
    d.codes = O.e4m3_encode(rng.standard_normal(d.codes.shape))   # values of the size of their scale
    d.q = (d.q.float() * 2.0 ** -hi).to(torch.bfloat16)
    d.check()


def test_decode_scales_that_are_no_powers_of_two():
    Decode([1, 2], [400, 90], 6, 32, 4, powers=False).check()


@pytest.mark.parametrize("H", [4, 20, 48])
def test_decode_growing_scores(H):
    """Later keys score ever higher, so the running reference moves tile after
    tile.  The scores spread over about 40, so the query terms' error (2^-8 of
    a score's parts) counts: the outputs are held to the worst case
    2 * max |score error| = 2 * 2^-8 * 24, the LSE to half of it."""
    d = Decode([1], [1000], H, 128, 1)
    v = O.e4m3_decode(d.codes).reshape(-1, 576)
    q = O.decode(O.codes(d.q), "bf16")
    u = np.concatenate([np.einsum("hd,hkd->hk", q[0, :, :128], O.decode(O.codes(d.w_uk), "bf16")), q[0, :, 128:]], 1)
    ramp = u.mean(0) / np.linalg.norm(u.mean(0))
    rows = d.rows(0, np.arange(1001))
    x = v * np.repeat(d.scales.reshape(-1), d.sb)[:, None]
    x[rows] += np.linspace(0, 60, 1001)[:, None] * ramp
    for r in rows:
        s = q8.block_scale(np.abs(x[r]).max())
        d.scales.reshape(-1)[r] = s
        d.codes.reshape(-1, 576)[r] = O.e4m3_encode(x[r] / s)
    d.check(rel=2 * 2.0 ** -8 * 24, lse_abs=2.0 ** -8 * 24)


def test_decode_strongly_negative_scores():
    """Every score near -200: no weight may vanish."""
    d = Decode([1], [300], 2, 128, 1)
    d.scale = 1.0
    d.codes[:] = 0
    d.codes[..., 512] = O.e4m3_encode(np.array([-200.0]))[0]
    d.codes[..., :4] = O.e4m3_encode(np.random.default_rng(0).standard_normal((*d.codes.shape[:2], 4)))
    d.scales[:] = 1.0
    d.q[:] = 0
    d.q[..., 128] = 1.0
    d.check()
    assert abs(d.lse[0, 0].item() - (np.log(301) - O.e4m3_decode(d.codes)[0, 0, 512] * -1)) < 1e-3


def test_decode_zero_query():
    d = Decode([1], [200], 2, 128, 1)
    d.q[:] = 0
    d.check()


@pytest.mark.parametrize("page,H", [(128, 4), (16, 40), (100, 4), (128, 9), (100, 9)])
def test_decode_ignores_what_lies_behind_the_context(page, H):
    """Slots behind the context hold NaN codes under NaN scales."""
    new, cached = [1, 3], [130, 61]
    d = Decode(new, cached, H, page, 1)
    ref = d.reference()
    used = np.zeros(d.num * page, bool)
    for b in range(2):
        used[d.rows(b, np.arange(new[b] + cached[b]))] = True
    d.codes.reshape(-1, 576)[~used] = 0x7F
    d.scales.reshape(-1)[~used] = np.nan
    out, lse = d.run(2)
    compare(out, lse, *ref)


@pytest.mark.parametrize("scale_nan", [False, True])
@pytest.mark.parametrize("H", [4, 9, 40])
def test_decode_a_broken_row_reaches_only_tokens_that_see_it(scale_nan, H):
    """The second new token's row is NaN: the first token does not see it, the
    second and third do."""
    d = Decode([3], [140], H, 128, 1)
    ref, ref_lse = d.reference()
    row = d.rows(0, [141])[0]
    if scale_nan:
        d.scales.reshape(-1)[row] = np.nan
    else:
        d.codes.reshape(-1, 576)[row, 5] = 0xFF
    out, lse = d.run(1)
    compare(out[:1], lse[:1], ref[:1], ref_lse[:1])
    assert np.isnan(out[1:]).all()


def test_decode_infinite_query_gives_nan():
    d = Decode([2], [50], 2, 16, 1)
    d.q[1, 1, 3] = float("inf")
    out, _ = d.run(1)
    assert np.isfinite(out[0]).all() and np.isfinite(out[1, 0]).all() and np.isnan(out[1, 1]).all()


def test_decode_rows_behind_the_last_sequence_are_left():
    Decode([1, 2], [20, 70], 4, 16, 1, T_extra=3).check()


@pytest.mark.parametrize("H", [5, 8, 40])
@pytest.mark.parametrize("with_sink", [False, True])
def test_sparse_decode(H, with_sink):
    """Listed rows in any order, the same row twice, counts below the stride
    (what lies past them is never read), an empty list, a single row; several
    tokens share a list."""
    d = Decode([1, 3, 1, 1, 2], [300, 90, 10, 40, 1000], H, 24, 8)
    rng = np.random.default_rng(1)
    lists = np.full((5, 200), 2 ** 30)
    topk = [150, 93, 0, 1, 200]
    for b, k in enumerate(topk):
        lists[b, :k] = d.rows(b, rng.integers(0, d.new[b] + d.cached[b], k))
    sink = None if not with_sink else rng.standard_normal(5).astype(np.float32) * 3
    d.check(parts=2, lists=lists, topk=topk, sink=sink)
    if not with_sink:
        t = int(d.iro[2])
        assert torch.all(d.out[t] == 0) and torch.all(d.lse[t] == float("-inf"))


def test_sparse_decode_whole_stride_and_unused_tables():
    """No counts: the whole stride; neither page table nor context lengths are
    read."""
    d = Decode([1, 1], [200, 300], 4, 128, 1)
    lists = np.stack([d.rows(b, np.arange(130)) for b in range(2)])
    ref = d.reference(lists=lists)
    d.cached = [2 ** 31 - 1, 0]
    d_table = d.table
    out, lse = d.run(0, lists=lists, max_seq=1000)
    compare(out, lse, *ref)
    assert d_table is d.table


def test_dense_decode_with_sink():
    d = Decode([2, 1], [100, 3], 4, 16, 2)
    d.check(sink=np.array([2.0, -1.0], np.float32))
    d.check(sink=np.array([-np.inf, 30.0], np.float32))


def test_decode_status():
    d = Decode([1, 1], [100, 150], 4, 128, 1)
    ref, ref_lse = d.reference()
    table = d.table.copy()
    table[1, 0] = d.num + 5
    out, lse = d.run(1, table=table, expect=mla.MLA_DEV_BAD_PAGE)
    compare(out[:1], lse[:1], ref[:1], ref_lse[:1])
    out, lse = d.run(1, max_seq=101, expect=mla.MLA_DEV_BAD_OFFSETS)   # the second context is longer
    compare(out[:1], lse[:1], ref[:1], ref_lse[:1])
    assert np.all(out[1] == 7.0)
    out, lse = d.run(1, iro=[0, 1, 3], expect=mla.MLA_DEV_BAD_OFFSETS)  # past the call's tokens
    compare(out[:1], lse[:1], ref[:1], ref_lse[:1])
    assert np.all(out[1] == 7.0)
    lists = np.zeros((2, 4), np.int64)
    lists[1, 2] = d.num * 128
    d.run(1, lists=lists, expect=mla.MLA_DEV_BAD_PAGE)
    lists[1, 2] = -1
    d.run(1, lists=lists, expect=mla.MLA_DEV_BAD_PAGE)


def test_decode_after_a_timeout_does_nothing():
    d = Decode([1], [100], 4, 128, 1)
    d.run(1)
    d.out.fill_(7.0)
    d.keep[-1].fill_(mla.MLA_DEV_TIMEOUT)
    d.call()
    torch.cuda.synchronize()
    assert torch.all(d.out == 7.0)


@pytest.mark.parametrize("H", [4, 12, 40])
def test_decode_replays_bit_for_bit(H):
    """Two eager calls, one on another stream, and two replays of a captured one
    give the same bits."""
    d = Decode([1, 2], [900, 333], H, 64, 8)
    d.run()
    ref, ref_lse = d.out.clone(), d.lse.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        d.out.zero_()
        d.call()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert torch.equal(d.out.view(torch.int16), ref.view(torch.int16)) and torch.equal(d.lse, ref_lse)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        d.call()
    for _ in range(2):
        d.out.zero_()
        d.lse.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(d.out.view(torch.int16), ref.view(torch.int16)) and torch.equal(d.lse, ref_lse)


def test_cache_offsets_past_32_bits():
    """A cache of more than 2^32 bytes: write, gather and decode (dense and
    listed) on its last pages."""
    page, H, n = 128, 4, 200
    num = (1 << 32) // (page * 576) + 40
    kv = torch.empty(num, page, 576, dtype=torch.uint8, device=DEV)
    sc = torch.empty(num, page // 64, device=DEV)
    table = np.array([[num - 1, num - 3]])
    for p in table[0]:
        kv[p] = 0
    w = scaled(WORKLOADS["tiny_ragged"], H=H)
    lat, gamma, freqs = make_cache_write_operands(w, n, n)
    st = status()
    mla.check(mla.mla_latent_cache_write_q8(kv, sc, None, lat.to(DEV), gamma.to(DEV), freqs.to(DEV), i32([0, n]), i32([0]),
                                            i32(table), num, page, 2, 64, 1, H, n, n, 1e-6, st))
    codes, scales = kv[[num - 1, num - 3]].cpu().numpy(), sc[[num - 1, num - 3]].cpu().numpy()
    values = q8.q8_values(codes, scales, 64)
    y = q8.new_rows(O.decode(O.codes(lat), "bf16"), gamma.numpy(), freqs.numpy(), [0, n], [0], 1e-6)
    assert np.all(np.abs(values[:n] - y) <= 2.0 ** -4 * np.abs(y) * 1.001 + np.repeat(scales.reshape(-1), 64)[:n, None] * 2.0 ** -10)
    ckv = torch.zeros(n, 512, dtype=torch.bfloat16, device=DEV)
    kr = torch.zeros(n, 64, dtype=torch.bfloat16, device=DEV)
    mla.check(mla.mla_gather_latent_q8(ckv, kr, kv, sc, i32(table), num, page, 2, 64, i32([[0, n]]), i32([[0]]), i32([n]),
                                       0, 1, n, st))
    assert np.array_equal(torch.cat([ckv, kr], 1).float().cpu().double().numpy(), values[:n])
    d = Decode([1], [n - 1], H, page, 64)
    ref = q8.decode_values(O.decode(O.codes(d.q), "bf16"), values, [[0, 1]], page, O.decode(O.codes(d.w_uk), "bf16"),
                           O.decode(O.codes(d.w_uv), "bf16"), [0, 1], [n - 1], d.scale)
    rows = torch.from_numpy(table[0][np.arange(n) // page] * page + np.arange(n) % page).to(torch.int32).to(DEV)
    nbytes = mla.mla_decode_q8_workspace_bytes(H, 1, 2)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=DEV)
    for sparse in (False, True):
        out = torch.zeros(1, H, 128, dtype=torch.bfloat16, device=DEV)
        lse = torch.zeros(1, H, device=DEV)
        mla.check(mla.mla_decode_q8(out, lse, d.q.to(DEV), i32([0, 1]), i32([n - 1]), kv, sc, i32(table), num, page, 2, 64,
                                    d.w_uk.to(DEV), d.w_uv.to(DEV), 1, H, 1, 1, n, 2, d.scale,
                                    d_indices=rows if sparse else None, indices_stride=n if sparse else 0, workspace=ws,
                                    workspace_bytes=nbytes, d_status=st))
        torch.cuda.synchronize()
        assert st.item() == 0
        compare(out.float().cpu().double().numpy(), lse.cpu().double().numpy(), *ref)


# ------------------------------------------------------------------ at the edges of the launch shapes

@pytest.mark.parametrize("H", [65, 192, 256, 320, 576])
def test_decode_many_heads(H):
    """Two to eight row tiles walk a piece together (pairs of them as clusters);
    576 heads are two items a token."""
    Decode([1, 2], [300, 40], H, 64, 16, seed=H).check(parts=3)


@pytest.mark.parametrize("H", [100, 192])
def test_sparse_decode_many_heads(H):
    d = Decode([1, 1], [300, 90], H, 24, 8)
    lists = np.stack([np.resize(d.rows(b, np.arange(91)[::-1]), 150) for b in range(2)])
    d.check(parts=3, lists=lists, topk=[150, 131])


@pytest.mark.parametrize("H", [4, 24, 40])
def test_decode_one_long_sequence(H):
    """A piece for every SM and one sequence: 16 warps share a token's pieces."""
    Decode([1], [40000], H, 128, 64).check()


@pytest.mark.parametrize("H,n", [(16, 30), (40, 16), (9, 100), (128, 40)])
def test_decode_tokens_of_the_last_kernel(H, n):
    """Two to 32 tokens a CTA of the merge, with one or several warps a token."""
    rng = np.random.default_rng(H)
    Decode([1] * n, [int(x) for x in rng.integers(0, 400, n)], H, 16, 4, seed=H).check()


def test_decode_many_pieces_of_several_tokens():
    """Items of two tokens cut into pieces, 128 heads."""
    Decode([2, 1, 2], [1500, 700, 90], 128, 128, 64).check()


def test_decode_mostly_empty_batch():
    """More sequences than tokens, the plan's scan in several turns."""
    new, cached = [0] * 400, [int(x) for x in np.random.default_rng(0).integers(0, 200, 400)]
    for b in (0, 127, 128, 300, 399):
        new[b] = 1 + b % 2
    Decode(new, cached, 8, 16, 1).check()


def test_decode_without_lse():
    d = Decode([1, 2], [300, 140], 40, 128, 8)
    out, lse = d.run(lse=False)
    assert lse is None
    compare(out, None, *d.reference())


def test_decode_max_new_above_every_sequence():
    d = Decode([1, 2], [300, 140], 8, 128, 8)
    compare(*d.run(max_new=50), *d.reference())


def test_decode_overlapping_and_decreasing_offsets():
    """Sequence 1 ends before it begins, sequence 2 begins inside sequence 0:
    both are reported and left out."""
    d = Decode([2, 1, 2], [100, 30, 60], 4, 16, 1)
    ref, ref_lse = d.reference()
    out, lse = d.run(iro=[0, 2, 1, 3], expect=mla.MLA_DEV_BAD_OFFSETS)
    compare(out[:2], lse[:2], ref[:2], ref_lse[:2])
    assert np.all(out[2:] == 7.0) and np.all(lse[2:] == 7.0)


def test_decode_a_piece_without_weight_beside_one_that_is_no_number():
    """All scores of the first piece are -infinity, a scale of the second is NaN."""
    d = Decode([1], [255], 2, 128, 1)
    d.q[:] = 0
    d.q[..., 128] = 2.0 ** 60
    d.codes[:] = 0
    d.scales[:] = 1.0
    first = d.rows(0, np.arange(128))
    d.codes.reshape(-1, 576)[first, 512] = O.e4m3_encode(np.array([-448.0]))[0]
    d.scales.reshape(-1)[first] = 2.0 ** 100
    assert np.all(np.isfinite(d.run(2)[0]))
    d.scales.reshape(-1)[d.rows(0, [200])[0]] = np.nan
    assert np.all(np.isnan(d.run(2)[0]))


def test_decode_two_calls_at_once():
    """Calls with workspaces of their own on two streams, eager and captured."""
    a, b = Decode([1, 2], [900, 333], 16, 64, 8), Decode([1], [5000], 40, 128, 64, seed=1)
    ref = []
    for d in (a, b):
        d.run()
        ref.append((d.out.clone(), d.lse.clone()))
    sides = [torch.cuda.Stream() for _ in range(2)]
    graphs = []
    for d, s in zip((a, b), sides):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            d.call()
        graphs.append(g)
    for how in ("eager", "captured"):
        for d in (a, b):
            d.out.zero_()
            d.lse.zero_()
        torch.cuda.synchronize()
        for _ in range(3):
            for d, g, s in zip((a, b), graphs, sides):
                with torch.cuda.stream(s):
                    d.call() if how == "eager" else g.replay()
        torch.cuda.synchronize()
        for d, (out, lse) in zip((a, b), ref):
            assert torch.equal(d.out.view(torch.int16), out.view(torch.int16)) and torch.equal(d.lse, lse)


@pytest.mark.parametrize("H", [33, 128, 200])
def test_write_heads(H):
    """Query pieces that do not fill a turn of the CTA, fill it, and take two."""
    check_write([2, 5], [9, 60], 16, 4, H)


def test_write_many_sequences():
    """More sequences than 32 * 32, most of them empty."""
    new = [0] * 1100
    for b in (0, 5, 31, 32, 500, 1023, 1024, 1099):
        new[b] = 1 + b % 3
    check_write(new, [b % 40 for b in range(1100)], 16, 4, 2)


def test_write_replays_bit_for_bit():
    page, n = 32, 70
    w = scaled(WORKLOADS["tiny_ragged"], H=4)
    lat, gamma, freqs = make_cache_write_operands(w, n, 100)
    table, num = pages([n], [10], page)
    q = torch.randn(n, 4, 192, generator=torch.Generator().manual_seed(0)).to(torch.bfloat16).to(DEV)
    kv, sc, dq = fp8(np.zeros((num, page, 576), np.uint8)), torch.zeros(num, page // 8, device=DEV), q.clone()
    call = lambda: mla.check(mla.mla_latent_cache_write_q8(kv, sc, dq, *dev, num, page, table.shape[1], 8, 1, 4, n, 100,
                                                           1e-6))
    dev = (lat.to(DEV), gamma.to(DEV), freqs.to(DEV), i32([0, n]), i32([10]), i32(table))
    call()
    torch.cuda.synchronize()
    ref = kv.clone(), sc.clone(), dq.clone()
    dq.copy_(q)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for _ in range(2):
        kv.zero_()
        sc.zero_()
        dq.copy_(q)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(kv, ref[0]) and torch.equal(sc, ref[1]) and torch.equal(dq.view(torch.int16), ref[2].view(torch.int16))

# ------------------------------------------------------------------ one key far above a long tail

def peaked(n, gap, spread, H, page=128, sb=1, sink_value=0.0, at=0, seed=0):
    """A sequence of n cached keys, one (position ``at``) `gap` nats above the
    others, which spread by `spread` nats and whose latents share a mean: with
    sink_value 0 the result is the others' alone.  Queries are 1 and +-spread in
    two rope places, so scores are exact and depend on the head's sign."""
    rng = np.random.default_rng(seed)
    d = Decode([1], [n], H, page, sb, seed)
    x = np.zeros((n + 1, 576))
    x[:, :512] = rng.standard_normal(512) + 0.25 * rng.standard_normal((n + 1, 512))
    x[:, 513] = rng.standard_normal(n + 1)
    x[at, :512] = sink_value * rng.standard_normal(512)
    x[at, 512], x[at, 513] = gap, 0.0
    d.scales[:] = 2.0 ** -5
    flat = d.codes.reshape(-1, 576)
    flat[d.rows(0, np.arange(n + 1))] = O.e4m3_encode(x / 2.0 ** -5)
    d.q[:] = 0
    d.q[..., 128] = 1.0
    d.q[..., 129] = spread * torch.where(torch.arange(H) % 2 == 0, 1.0, -1.0).to(torch.bfloat16)
    d.scale = 1.0
    return d


def far_below(H, gap, spread):
    """Share of itself by which the weight of a key may be off, `gap` nats and
    three spreads below one that stands alone in its tile and is put at 2^7.75: it
    is held to 2^-15 up to 32 heads, else to 2^-14, or 1/8 of itself and 2^-17."""
    far = np.exp(gap + 3 * spread) / 2.0 ** 7.75
    return min(1.0, 2.0 ** -15 * far if H <= 32 else min(2.0 ** -14 * far, max(1 / 8, 2.0 ** -17 * far)))


def compare_rows(out, ref, rel):
    """Every token's and head's result by itself."""
    err = np.linalg.norm(out - ref, axis=-1) / np.linalg.norm(ref, axis=-1)
    assert err.max() <= rel, (err.max(), rel)


@pytest.mark.parametrize("listed", [False, True])
@pytest.mark.parametrize("H", [4, 16, 20, 48, 64, 128])
@pytest.mark.parametrize("n,gap,spread,sink_value", [
    (9000, 10.0, 0.0, 0.0), (9000, 10.0, 0.5, 0.0), (9000, 9.5, 1.0, 1.0), (9000, 13.0, 0.5, 0.0), (30000, 12.0, 1.0, 0.0)])
def test_decode_one_key_far_above_the_others(n, gap, spread, sink_value, H, listed):
    """The others keep their share of the result, whatever the largest weight is
    (one piece, so that they share its reference).

    Per head, in the 2-norm: the output's rounding is at most 2^-8 of each value,
    sqrt(1/3) of that in the mean of 128; the weights' terms are each within 2^-8
    of the weight (where all weights are equal, all by the same share); partial
    results are fp16, 2^-11.  In the tile of the large key the other 127 of n are
    off by what far_below says."""
    d = peaked(n, gap, spread, H, sink_value=sink_value)
    lists = d.rows(0, np.arange(n + 1))[None] if listed else None
    out, lse = d.run(1, lists=lists)
    ref, ref_lse = d.reference(lists=lists)
    assert np.abs(lse - ref_lse).max() <= LSE_ABS
    compare_rows(out, ref, 2.0 ** -8 * 3 ** -0.5 + 2.0 ** -8 + 127 / n * far_below(H, gap, spread) + 2.0 ** -11)


@pytest.mark.parametrize("H", [4, 32, 64])
def test_decode_one_key_far_above_100000(H):
    d = peaked(100000, 12.0, 1.0, H)
    out, lse = d.run(1)
    ref, ref_lse = d.reference()
    assert np.abs(lse - ref_lse).max() <= LSE_ABS
    compare_rows(out, ref, 2.0 ** -8 * 3 ** -0.5 + 2.0 ** -8 + 2.0 ** -11)


@pytest.mark.parametrize("H", [4, 20, 48])
def test_decode_large_keys_come_and_go(H):
    """Large keys in every third tile, from the third on: the reference rises and
    falls many times."""
    n = 12000
    d = peaked(n, 11.0, 0.5, H, at=300)
    flat = d.codes.reshape(-1, 576)
    for p in range(600, n, 384):
        flat[d.rows(0, [p])[0]] = flat[d.rows(0, [300])[0]]
    out, lse = d.run(1)
    ref, ref_lse = d.reference()
    assert np.abs(lse - ref_lse).max() <= LSE_ABS
    # (A third of the tiles hold a large key: their weights are within 1/8 at the
    # least, 11 nats and three spreads below 2^7.)
    compare_rows(out, ref, 2.0 ** -8 * 3 ** -0.5 + 2.0 ** -8 + 2.0 ** -11 + 1 / 24)


# ------------------------------------------------------------------ rows of a very large scale

@pytest.mark.parametrize("H", [4, 9, 24, 40, 128])
def test_decode_a_row_that_is_not_seen_does_not_reach_the_result(H):
    """The second new token's row has the scale 2^120 (an infinite value's): the
    first token, in the same row tile up to 32 heads, does not see it."""
    d = Decode([2], [140], H, 128, 1)
    ref, ref_lse = d.reference()
    row = d.rows(0, [141])[0]
    d.scales.reshape(-1)[row] = 2.0 ** 120
    d.codes.reshape(-1, 576)[row, :4] = 0x7E
    out, lse = d.run(1)
    compare(out[:1], lse[:1], ref[:1], ref_lse[:1])


@pytest.mark.parametrize("listed", [False, True])
@pytest.mark.parametrize("exp", [18, 24, 60, 120])
@pytest.mark.parametrize("H", [4, 24, 40])
def test_decode_a_row_without_weight_does_not_reach_the_result(H, exp, listed):
    """A row whose scale is 2^exp times the others' 2^-6 and whose score is far
    below theirs (its rope code is the most negative one, the queries positive
    there): the result is the others', head by head (each within the bound on all
    of them, and half as much again for the heads' spread)."""
    d = Decode([1], [300], H, 128, 1, lo=-6, hi=-6)
    d.q[..., 128:130] = 4.0
    row = d.rows(0, [170])[0]
    d.scales.reshape(-1)[row] = 2.0 ** (exp - 6)
    d.codes.reshape(-1, 576)[row, :512] = O.e4m3_encode(np.random.default_rng(0).standard_normal(512))
    d.codes.reshape(-1, 576)[row, 512:] = 0
    d.codes.reshape(-1, 576)[row, 512:514] = 0xFE
    lists = d.rows(0, np.arange(301))[None] if listed else None
    out, lse = d.run(1, lists=lists)
    ref, ref_lse = d.reference(lists=lists)
    assert np.abs(lse - ref_lse).max() <= LSE_ABS
    compare_rows(out, ref, REL * 1.5)


def test_decode_whole_tiles_without_weight():
    """The first 128 scores are -infinity, the others near -200, in one piece: no
    weight may vanish for that."""
    d = Decode([1], [299], 2, 128, 1)
    rng = np.random.default_rng(0)
    d.q[:] = 0
    d.q[..., 128] = 2.0 ** 60
    d.scale = 1.0
    flat, sc = d.codes.reshape(-1, 576), d.scales.reshape(-1)
    flat[:] = O.e4m3_encode(rng.standard_normal(flat.shape))
    flat[:, 512] = O.e4m3_encode(np.array([-3.25]))[0]
    sc[:] = 2.0 ** -54
    first = d.rows(0, np.arange(128))
    flat[first, 512] = O.e4m3_encode(np.array([-448.0]))[0]
    sc[first] = 2.0 ** 100
    d.check()


@pytest.mark.parametrize("lo,hi", [(-60, -58), (97, 100)])
@pytest.mark.parametrize("H", [8, 24, 40])
def test_decode_scales_at_the_ends_of_their_range(lo, hi, H):
    """Queries divided by the largest scale, so that scores stay of order one."""
    d = Decode([1, 1], [700, 300], H, 128, 4, lo=lo, hi=hi)
    d.codes = O.e4m3_encode(np.random.default_rng(0).standard_normal(d.codes.shape))
    d.q = (d.q.float() * 2.0 ** -hi).to(torch.bfloat16)
    d.check()


@pytest.mark.parametrize("H", [8, 24, 40])
def test_decode_zero_rows_beside_others(H):
    """Half of the context, whole tiles of it, is zero rows under the smallest
    scale: they take part in the softmax, and the result is the others'."""
    d = Decode([1], [1000], H, 128, 1)
    zero = d.rows(0, np.r_[0:256, 300:310, 512:768])
    d.codes.reshape(-1, 576)[zero] = 0
    d.scales.reshape(-1)[zero] = 2.0 ** -60
    d.check(parts=1)


@pytest.mark.parametrize("H", [4, 24, 40])
def test_decode_queries_small_where_keys_are_large(H):
    """One rope place of the queries is 2^16 times the others, and zero in the
    keys; the scores come from the others alone, in places where the keys are
    large.  A query value is off by at most 2^-21 of its row's largest, 2^-5 of
    these, evenly spread: scores (of spread 1) by 2^-5 / sqrt(3), which changes a
    result by no more than sqrt(2) times that."""
    d = Decode([1], [400], H, 128, 1, lo=-3, hi=-3)
    rng = np.random.default_rng(0)
    x = rng.standard_normal(d.codes.shape)
    x[..., 512] = 0
    x[..., 513:] *= 8.0
    d.codes = O.e4m3_encode(x / 2.0 ** -3)
    d.q[:] = 0
    d.q[..., 129:] = torch.from_numpy(rng.standard_normal((1, H, 63)) * 2.0 ** -8).to(torch.bfloat16)
    d.q[..., 128] = 2.0 ** 8
    d.scale = 2.0 ** 5 / 8.0
    out, lse = d.run(1)
    ref, ref_lse = d.reference()
    assert np.abs(lse - ref_lse).max() <= 2.0 ** -5
    compare_rows(out, ref, REL + 2.0 ** -5 * (2 / 3) ** 0.5)


# ------------------------------------------------------------------ infinite, very large and very small values

def _extreme_write(lat, eps):
    """Each row of ``lat`` as a token of one sequence, a scale a slot, angles
    around the circle, queries with the same rope parts.  Returns the rows'
    codes, scales, queries' rope parts, and the definition's values in 64 bits."""
    n = lat.shape[0]
    gamma = torch.from_numpy(1.0 + 0.1 * np.random.default_rng(1).standard_normal(512)).float()
    ang = 0.3 + np.arange(n)[:, None] + np.arange(32)[None] * 0.1
    freqs = torch.from_numpy(np.stack([np.cos(ang), np.sin(ang)], -1).reshape(n, 64)).float()
    kv, sc = torch.zeros(1, n, 576, dtype=torch.uint8, device=DEV), torch.ones(1, n, device=DEV)
    q = torch.zeros(n, 1, 192, dtype=torch.bfloat16)
    q[:, 0, 128:] = lat[:, 512:]
    dq, st = q.to(DEV), status()
    mla.check(mla.mla_latent_cache_write_q8(kv, sc, dq, lat.to(DEV), gamma.to(DEV), freqs.to(DEV), i32([0, n]), i32([0]),
                                            i32([[0]]), 1, n, 1, 1, 1, 1, n, n, eps, st))
    torch.cuda.synchronize()
    assert st.item() == 0
    with np.errstate(all="ignore"):
        y = q8.new_rows(O.decode(O.codes(lat), "bf16"), gamma.numpy(), freqs.numpy(), [0, n], [0], eps)
        # (numpy's complex product turns an infinite part into NaN: the real products.)
        r, f = O.decode(O.codes(lat), "bf16")[:, 512:], freqs.double().numpy()
        y[:, 512::2] = r[:, ::2] * f[:, ::2] - r[:, 1::2] * f[:, 1::2]
        y[:, 513::2] = r[:, ::2] * f[:, 1::2] + r[:, 1::2] * f[:, ::2]
    return kv[0].cpu().numpy(), sc[0].cpu().double().numpy(), dq[:, 0, 128:].float().cpu().double().numpy(), y


def _check_codes(codes, scales, y):
    """Scales equal, NaN for NaN, +-448 for an infinite value, else as check_write."""
    for c, s, v in zip(codes, scales, y):
        assert s == q8.block_scale(float(np.nanmax(np.abs(v), initial=0.0)))
        got, pre = O.e4m3_decode(c), v / s
        assert np.array_equal(np.isnan(got), np.isnan(pre))
        inf, fin = np.isinf(pre), np.isfinite(pre)
        assert np.array_equal(got[inf], 448.0 * np.sign(pre[inf]))
        a = np.maximum(np.abs(pre[fin]), 2.0 ** -6)
        assert np.all(np.abs(got[fin] - pre[fin]) <= np.exp2(np.floor(np.log2(a)) - 4) + 2.0 ** -20 * a)


def test_write_infinite_values():
    """An infinite latent makes its row's others zero and itself NaN; infinite
    rope values, in either half of a pair, keep their signs, the queries' too."""
    lat = torch.randn(5, 576, generator=torch.Generator().manual_seed(0)).to(torch.bfloat16)
    inf = float("inf")
    lat[0, 7] = inf
    lat[1, 300], lat[1, 301] = -inf, inf
    lat[2, 513], lat[2, 520], lat[2, 575] = inf, -inf, -inf
    lat[3, 512:514] = inf                        # both halves: NaN where their products cancel
    codes, scales, q, y = _extreme_write(lat, 1e-6)
    assert np.isnan(y[0]).sum() == 1 and np.isinf(y[2]).sum() == 6
    _check_codes(codes, scales, y)
    assert np.array_equal(np.isnan(q), np.isnan(y[:, 512:])) and np.array_equal(np.isinf(q), np.isinf(y[:, 512:]))
    fin = np.isfinite(q)
    assert np.array_equal(q[np.isinf(q)], y[:, 512:][np.isinf(q)])
    assert np.all(np.abs(q[fin] - y[:, 512:][fin]) <= 2.0 ** -8 * np.abs(y[:, 512:][fin]) + 2.0 ** -20)


@pytest.mark.parametrize("size,eps", [(1e19, 1e-6), (1e22, 1e-6), (1e37, 1e-6), (1e37, 0.0), (1e-17, 0.0), (1e-22, 0.0),
                                      (1e-36, 0.0), (1e-30, 1e-35), (1e-20, 1e-6), (0.0, 1e-6)])
def test_write_latents_whose_squares_leave_the_range(size, eps):
    """The norm is that of the definition for every size that bf16 has."""
    x = torch.randn(3, 576, generator=torch.Generator().manual_seed(0), dtype=torch.float64)
    x[:, :512] *= size
    x[2, :256] = 0
    codes, scales, _, y = _extreme_write(x.to(torch.bfloat16), eps)
    _check_codes(codes, scales, y)


@pytest.mark.parametrize("H", [4, 24, 40])
@pytest.mark.parametrize("n,gap", [(100, 8.0), (100, 12.0), (500, 10.0), (500, 12.0), (500, 13.0), (2000, 14.0)])
def test_decode_one_key_far_above_a_short_context(n, gap, H):
    """The large key's tile is a good part of the context, or all of it."""
    d = peaked(n, gap, 0.25, H)
    out, lse = d.run(1)
    ref, ref_lse = d.reference()
    assert np.abs(lse - ref_lse).max() <= LSE_ABS
    compare_rows(out, ref, 2.0 ** -8 * 3 ** -0.5 + 2.0 ** -8 + min(1, 127 / n) * far_below(H, gap, 0.25) + 2.0 ** -11)
