"""GPU tests of the paged cache's bookkeeping against the plain oracle, which
they have to equal: tables, counts, lists and moved bytes are whole numbers."""
import numpy as np
import pytest
import torch

import mla_prefill_attention_plan_gb300 as mla
import oracle as O
from oracle import pages_oracle as P

pytestmark = pytest.mark.gpu
DEV = "cuda"
FILL = -7


@pytest.fixture(scope="module", autouse=True)
def _built():
    from mla_prefill_attention_plan_gb300 import build
    build.build()
    mla.load()


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(x, dtype=np.int32))).to(DEV)


def status():
    return torch.zeros(1, dtype=torch.int32, device=DEV)


def workspace(num_pages, B):
    n = mla.mla_pages_workspace_bytes(num_pages, B)
    return torch.randint(0, 256, (n,), dtype=torch.uint8, device=DEV), n     # its contents mean nothing


def state(B, page, max_pages, spare, seed, share=0.0):
    """(table, refs, lengths) of random sequences on shuffled pages; a share of
    the rows continue the row before them."""
    rng = np.random.default_rng(seed)
    lengths = rng.integers(0, page * max_pages + 1, B)
    held = -(-lengths // page)
    pool = int(held.sum()) + spare
    order = rng.permutation(pool)
    table, refs, at = np.full((B, max_pages), -1, np.int32), np.zeros(pool, np.int32), 0
    for b in range(B):
        if b and rng.random() < share:
            lengths[b], table[b] = lengths[b - 1], table[b - 1]
        else:
            table[b, :held[b]] = order[at: at + held[b]]
            at += held[b]
        refs[table[b][table[b] >= 0]] += 1
    return table, refs, lengths


def run_fork(table, refs, lengths, parents, expect=0):
    B, most = len(parents), table.shape[1]
    out, n, r, st = dev(np.full((B, most), FILL)), dev(np.full(B, FILL)), dev(refs), status()
    src = dev(table)
    mla.check(mla.mla_pages_fork(out, n, src, dev(lengths), r, dev(parents), len(refs), most, B, len(table), st))
    assert st.item() == expect and np.array_equal(src.cpu().numpy(), table)
    return out.cpu().numpy(), n.cpu().numpy(), r.cpu().numpy()


@pytest.mark.parametrize("B_src,B_dst,most", [(1, 1, 1), (1, 300, 5), (7, 13, 3), (40, 2, 300), (3, 0, 4), (64, 64, 257)])
def test_fork(B_src, B_dst, most):
    table, refs, lengths = state(B_src, 4, most, 3, B_src + most, share=0.3)
    parents = np.random.default_rng(most).integers(-1, B_src, B_dst)
    got = run_fork(table, refs, lengths, parents)
    want = P.fork(table, lengths, refs, parents)
    assert all(np.array_equal(g, w) for g, w in zip(got, (*want, refs)))


def test_fork_of_nothing_is_empty():
    got = run_fork(np.full((1, 2), -1, np.int32), np.zeros(4, np.int32), np.zeros(1, int), [-1, -1])
    assert (got[0] == -1).all() and not got[1].any() and not got[2].any()


def test_fork_reports_bad_parents_and_pages():
    table, refs = np.array([[0, 1], [2, -1]], np.int32), np.ones(3, np.int32)
    got = run_fork(table, refs, np.array([8, 3]), [1, 2, -2, 0], expect=mla.MLA_DEV_BAD_OFFSETS)
    assert got[0].tolist() == [[2, -1], [-1, -1], [-1, -1], [0, 1]] and got[1].tolist() == [3, 0, 0, 8]
    assert got[2].tolist() == [1, 1, 1]
    bad = np.array([[0, 3], [2, -5]], np.int32)
    got = run_fork(bad, refs, np.array([8, 3]), [0, 1], expect=mla.MLA_DEV_BAD_PAGE)
    assert got[0].tolist() == [[0, -1], [2, -1]]


@pytest.mark.parametrize("page,most", [(1, 40), (16, 9), (100, 700)])
@pytest.mark.parametrize("keep", ["none", "some", "same", "all"])
def test_free(page, most, keep):
    table, refs, lengths = state(9, page, most, 4, page, share=0.4)
    rng = np.random.default_rng(most)
    kept = {"none": None, "some": rng.integers(0, 2 * page * most, 9) % (page * most + 2), "same": lengths.copy(),
            "all": np.full(9, page * most)}[keep]
    if keep == "same":                          # pages reserved beyond the context go
        lengths = lengths // 2
        kept = lengths.copy()
    t, r, n, st = dev(table), dev(refs), dev(lengths), status()
    k = None if kept is None else n if keep == "same" else dev(kept)
    mla.check(mla.mla_pages_free(t, r, n, k, len(refs), page, most, 9, st))
    P.free(table, refs, lengths, kept, page)
    assert st.item() == 0 and np.array_equal(t.cpu(), table) and np.array_equal(r.cpu(), refs)
    assert np.array_equal(n.cpu(), lengths)


def test_free_reports_bad_pages():
    t, r, n, st = dev([[0, 1, 5, -3]]), dev([1, 0, 2]), dev([16]), status()
    mla.check(mla.mla_pages_free(t, r, n, None, 3, 4, 4, 1, st))
    assert st.item() == mla.MLA_DEV_BAD_PAGE and r.tolist() == [0, 0, 2] and t.tolist() == [[-1, -1, -1, -3]]


def run_reserve(table, refs, lengths, new, page, expect=0, offset=0):
    B, most = table.shape
    t, st = dev(table), status()
    r = torch.zeros(len(refs) + offset, dtype=torch.int32, device=DEV)[offset:]      # offset: not 16-byte aligned
    r.copy_(dev(refs))
    src, dst, n = dev(np.full(B + 1, FILL)), dev(np.full(B + 1, FILL)), dev([FILL])
    ws, size = workspace(len(refs), B)
    mla.check(mla.mla_pages_reserve(t, r, dev(lengths), dev(new), src, dst, n, len(refs), page, most, B, workspace=ws,
                                    workspace_bytes=size, d_status=st))
    assert st.item() == expect and src[B].item() == FILL and dst[B].item() == FILL
    k = n.item()
    assert (src[k:B] == -1).all() and (dst[k:B] == -1).all()
    return t.cpu().numpy(), r.cpu().numpy(), list(zip(src[:k].tolist(), dst[:k].tolist()))


@pytest.mark.parametrize("B,page,most,spare,share", [
    (1, 16, 4, 4, 0.0), (5, 1, 30, 200, 0.5), (9, 16, 8, 100, 0.7), (300, 4, 12, 3000, 0.8), (64, 100, 70, 5000, 0.3),
    (1300, 8, 3, 9000, 0.6), (17, 16, 8, 60000, 0.5)])
@pytest.mark.parametrize("offset", [0, 1])
def test_reserve(B, page, most, spare, share, offset):
    """Missing, shared and own pages; a table with pages reserved before; zero tokens."""
    table, refs, lengths = state(B, page, most, spare, B + page, share)
    rng = np.random.default_rng(B)
    lengths = np.where(rng.random(B) < 0.5, lengths, lengths // 2)
    new = np.where(rng.random(B) < 0.2, 0, rng.integers(0, page * most + 1, B))
    new = np.minimum(new, page * most - lengths)
    got = run_reserve(table, refs, lengths, new, page, offset=offset)
    copies = P.reserve(table, refs, lengths, new, page)
    assert copies is not None and got[2] == copies
    assert np.array_equal(got[0], table) and np.array_equal(got[1], refs)


def test_reserve_takes_the_very_last_page():
    table, refs = np.full((3, 4), -1, np.int32), np.array([1, 0] * 6, np.int32)
    got = run_reserve(table, refs, [0, 0, 0], [8, 8, 8], 4)
    assert got[0][:, :2].tolist() == [[1, 3], [5, 7], [9, 11]] and (got[1] == 1).all()
    refs[1] = 1                                  # one too few: nothing changes
    got = run_reserve(table, refs, [0, 0, 0], [8, 8, 8], 4, expect=mla.MLA_DEV_NO_PAGES)
    assert (got[0] == -1).all() and np.array_equal(got[1], refs) and got[2] == []


def test_reserve_reports_what_does_not_fit():
    table, refs = np.array([[0, -1], [1, -1]], np.int32), np.array([1, 1, 0, 0], np.int32)
    for lengths, new in (([4, 3], [1, 6]), ([4, 3], [1, (1 << 32) - 1])):
        new = np.array(new, dtype=np.int64).astype(np.uint32).view(np.int32)
        got = run_reserve(table, refs, lengths, new, 4, expect=mla.MLA_DEV_BAD_PAGE)
        assert np.array_equal(got[0], table) and np.array_equal(got[1], refs) and got[2] == []
    bad = np.array([[9, -1], [1, -1]], np.int32)
    got = run_reserve(bad, refs, [3, 3], [1, 5], 4, expect=mla.MLA_DEV_BAD_PAGE)
    assert np.array_equal(got[0], bad) and np.array_equal(got[1], refs) and got[2] == []


def test_reserve_of_no_sequences():
    n, st, r = dev([FILL]), status(), dev([1, 0, 0])
    ws, size = workspace(3, 0)
    mla.check(mla.mla_pages_reserve(r, r, r, r, r, r, n, 3, 4, 2, 0, workspace=ws, workspace_bytes=size, d_status=st))
    assert n.item() == 0 and st.item() == 0 and r.tolist() == [1, 0, 0]


@pytest.mark.parametrize("B,most,spare,share,limit", [
    (1, 1, 1, 0, 9), (4, 6, 0, 0.5, 99), (30, 20, 300, 0.5, 9999), (30, 20, 300, 0.5, 37), (200, 40, 70000, 0.2, 80000),
    (16, 8, 20, 0, 0)])
def test_compact(B, most, spare, share, limit):
    table, refs, lengths = state(B, 4, most, spare, most, share)
    t, r, st = dev(table), dev(refs), status()
    src, dst, n = dev(np.full(limit + 1, FILL)), dev(np.full(limit + 1, FILL)), dev([FILL])
    ws, size = workspace(len(refs), B)
    mla.check(mla.mla_pages_compact(t, r, src, dst, n, limit, len(refs), most, B, workspace=ws, workspace_bytes=size,
                                    d_status=st))
    moves = P.compact(table, refs, limit)
    k = n.item()
    assert st.item() == 0 and list(zip(src[:k].tolist(), dst[:k].tolist())) == moves
    assert (src[k:limit] == -1).all() and (dst[k:limit] == -1).all() and src[limit].item() == FILL
    assert np.array_equal(t.cpu(), table) and np.array_equal(r.cpu(), refs)


@pytest.mark.parametrize("size,layers,gap,dtype", [
    (1152 * 16, 3, 0, torch.uint8), (4, 2, 0, torch.uint8), (4 * 4099, 2, 4, torch.uint8), (16, 1, 0, torch.uint8),
    (16 * 1025, 5, 48, torch.uint8), (576 * 24, 2, 0, torch.uint8)])
@pytest.mark.parametrize("shift", [0, 4])
def test_copy(size, layers, gap, dtype, shift):
    """Sizes that end inside a piece, strides with a gap, 4-byte alignment only."""
    rng = np.random.default_rng(size)
    pool, most = 40, 12
    stride = pool * size + gap
    x = torch.randint(0, 256, (layers * stride + shift,), dtype=dtype, device=DEV)
    want = x.clone()
    ids = rng.permutation(pool)
    src, dst = ids[:most], ids[most: 2 * most]
    for n in (0, 7, most + 5):                    # a count past the limit copies up to it
        mla.check(mla.mla_pages_copy(x[shift:], size, layers, stride, dev(src), dev(dst), dev([n]), most, pool))
        for a in range(layers):
            p = want[shift + a * stride:][:pool * size].view(pool, size)
            p[dst[:n]] = p[src[:n]]
        assert torch.equal(x, want)


def test_copy_leaves_out_pages_that_are_none():
    x = torch.arange(8 * 4, dtype=torch.int32, device=DEV).view(8, 4)
    want, st = x.clone(), status()
    want[5] = want[1]
    mla.check(mla.mla_pages_copy(x, 16, 1, 0, dev([1, 8, 2, -1]), dev([5, 6, 8, 7]), dev([4]), 4, 8, st))
    assert st.item() == mla.MLA_DEV_BAD_PAGE and torch.equal(x, want)


@pytest.mark.parametrize("row,layers,page,longest", [
    (1152, 3, 16, 9), (576, 2, 1, 5), (4, 2, 24, 40), (256, 1, 100, 64), (4 * 300, 2, 8, 30), (16 * 300, 1, 8, 70),
    (20, 1, 16, 600)])
def test_keep_rows(row, layers, page, longest):
    rng = np.random.default_rng(row + page)
    B = 6
    lengths = rng.integers(0, 50, B)
    held = -(-(lengths + longest) // page)
    pool, most = int(held.sum()) + 2, int(held.max())
    order, at = rng.permutation(pool), 0
    table = np.full((B, most), -1, np.int32)
    for b in range(B):
        table[b, :held[b]] = order[at: at + held[b]]
        at += held[b]
    kept = [sorted(rng.choice(longest, rng.integers(0, longest + 1), replace=False)) for _ in range(B)]
    kept[0], kept[1] = [], list(range(longest))
    width = max(map(len, kept))
    x = rng.integers(0, 2 ** 31, (layers, pool * page, row // 4)).astype(np.int32)
    got, st = dev(x), status()
    pad = np.array([list(k) + [-1] * (width - len(k)) for k in kept])
    mla.check(mla.mla_cache_keep_rows(got, row, layers, pool * page * row, dev(lengths), dev(pad), width,
                                      dev([len(k) for k in kept]), dev(table), pool, page, most, B, st))
    P.keep_rows(x, lengths, kept, table, page)
    assert st.item() == 0 and np.array_equal(got.cpu().numpy(), x)


@pytest.mark.parametrize("keep,count,code", [
    ([1, 1, 2], 3, "BAD_OFFSETS"), ([2, 1, 3], 3, "BAD_OFFSETS"), ([-1, 1, 2], 3, "BAD_OFFSETS"),
    ([0, 1, 2], 4, "BAD_OFFSETS"), ([1, 2, 9], 3, "BAD_PAGE"), ([1, 2, 1 << 30], 3, "BAD_PAGE"),
    ([1, 2, 5], 3, "BAD_PAGE"), ([1, 2, 3], -1, "OK")])
def test_keep_rows_moves_a_sequence_whole_or_not_at_all(keep, count, code):
    """Positions 3 .. 8 of pages of 4, the third of which (8 .. 11) is missing; sequence 1 is good."""
    x = torch.arange(16 * 4, dtype=torch.int32, device=DEV).view(16, 4)
    want, st = x.clone(), status()
    want[4 * 3], want[4 * 3 + 1] = x[4 * 3 + 1], x[4 * 3 + 3]
    mla.check(mla.mla_cache_keep_rows(x, 16, 1, 0, dev([3, 0]), dev([keep, [1, 3, -1]]), 3, dev([count, 2]),
                                      dev([[0, 2, -1], [3, -1, -1]]), 4, 4, 3, 2, st))
    assert st.item() == getattr(mla, "MLA_DEV_" + code) and torch.equal(x, want)


def test_a_timeout_before_stops_the_calls():
    table, refs, lengths = state(5, 4, 6, 9, 1, share=0.5)
    t, r, n = dev(table), dev(refs), dev(lengths)
    st = dev([mla.MLA_DEV_TIMEOUT])
    src, dst, cnt = dev(np.full(64, FILL)), dev(np.full(64, FILL)), dev([FILL])
    out, ln = dev(np.full((5, 6), FILL)), dev(np.full(5, FILL))
    ws, size = workspace(len(refs), 5)
    x = torch.arange(len(refs) * 4, dtype=torch.int32, device=DEV)
    y = x.clone()
    mla.check(mla.mla_pages_fork(out, ln, t, n, r, dev([0] * 5), len(refs), 6, 5, 5, st))
    mla.check(mla.mla_pages_reserve(t, r, n, dev([1] * 5), src, dst, cnt, len(refs), 4, 6, 5, ws, size, st))
    mla.check(mla.mla_pages_compact(t, r, src, dst, cnt, 64, len(refs), 6, 5, ws, size, st))
    mla.check(mla.mla_pages_free(t, r, n, None, len(refs), 4, 6, 5, st))
    mla.check(mla.mla_pages_copy(x, 16, 1, 0, dev([0]), dev([1]), dev([1]), 1, len(refs), st))
    assert (out == FILL).all() and (src == FILL).all() and cnt.item() == FILL and torch.equal(x, y)
    assert np.array_equal(t.cpu(), table) and np.array_equal(r.cpu(), refs) and np.array_equal(n.cpu(), lengths)


def test_captured_and_replayed_on_another_stream():
    """Reserve and give back in a graph: every replay finds the state it left."""
    table, refs, lengths = state(40, 16, 9, 400, 5, share=0.4)
    lengths = lengths // 2
    new = np.full(40, 40)
    t, r, n, k = dev(table), dev(refs), dev(lengths), dev(new)
    src, dst, cnt, st = dev(np.zeros(40)), dev(np.zeros(40)), dev([0]), status()
    ws, size = workspace(len(refs), 40)
    g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(g, stream=s):
        mla.check(mla.mla_pages_reserve(t, r, n, k, src, dst, cnt, len(refs), 16, 9, 40, ws, size, st))
        mla.check(mla.mla_pages_free(t, r, n, n, len(refs), 16, 9, 40, st))
    for _ in range(3):
        g.replay()
        torch.cuda.synchronize()
        copies = P.reserve(table, refs, lengths, np.minimum(new, 16 * 9 - lengths), 16)
        P.free(table, refs, lengths, lengths, 16)
        assert st.item() == 0 and list(zip(src.tolist(), dst.tolist()))[:cnt.item()] == copies
        assert np.array_equal(t.cpu(), table) and np.array_equal(r.cpu(), refs)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_write_at_rotates_by_the_given_positions(dtype):
    """Slots follow the context, rotations the positions given; with the context's own positions the call is
    mla_latent_cache_write, bit for bit."""
    rng = np.random.default_rng(8)
    new, cached, page, H, L = [5, 0, 3], [13, 4, 0], 8, 3, 40
    T, held = sum(new), [-(-(a + b) // 8) for a, b in zip(new, cached)]
    table, order, at = np.full((3, max(held)), -1, np.int32), rng.permutation(sum(held)), 0
    for b, k in enumerate(held):
        table[b, :k] = order[at: at + k]
        at += k
    iro = np.concatenate([[0], np.cumsum(new)])
    lat = torch.from_numpy(rng.standard_normal((T, 576))).to(torch.bfloat16).to(DEV)
    q0 = torch.from_numpy(rng.standard_normal((T, H, 192))).to(torch.bfloat16).to(DEV)
    gamma = torch.from_numpy(1 + 0.1 * rng.standard_normal(512)).float().to(DEV)
    ang = rng.uniform(0, 6, (L, 32))
    freqs = torch.from_numpy(np.stack([np.cos(ang), np.sin(ang)], -1).reshape(L, 64)).float().to(DEV)
    kind = mla.MLA_BF16 if dtype == "bf16" else mla.MLA_E4M3
    own = np.concatenate([np.arange(c, c + n) for n, c in zip(new, cached)])
    depth = np.array([13, 14, 14, 15, 39, 0, 1, 1])

    def write(positions=None, f=freqs, expect=0):
        kv = torch.zeros(sum(held), page, 576, dtype=torch.bfloat16 if kind == mla.MLA_BF16 else torch.uint8, device=DEV)
        q, st = q0.clone(), status()
        rest = (dev(iro), dev(cached), dev(table), sum(held), page, max(held), 3, H, T, L, 1e-6, 1.0, kind, st)
        if positions is None:
            mla.check(mla.mla_latent_cache_write(kv, q, lat, gamma, f, *rest))
        else:
            mla.check(mla.mla_latent_cache_write_at(kv, q, lat, gamma, f, dev(positions), *rest))
        assert st.item() == expect
        return kv.view(torch.uint8), q.view(torch.int16)
    plain, same = write(), write(own)
    assert torch.equal(plain[0], same[0]) and torch.equal(plain[1], same[1])
    # The context position's row of a permuted table is the given position's of the table itself.
    f = freqs.clone()
    got = write(depth)
    for t in range(T):
        f[own[t]] = freqs[depth[t]]
        ref = write(f=f)
        row = table[0 if t < 5 else 2, own[t] // page], own[t] % page
        assert torch.equal(got[0].view(sum(held), page, -1)[row], ref[0].view(sum(held), page, -1)[row])
        assert torch.equal(got[1][t], ref[1][t])
    bad = depth.copy()
    bad[2] = L
    skipped = write(bad, expect=mla.MLA_DEV_BAD_OFFSETS)
    assert not skipped[0].view(sum(held), page, -1)[int(table[0, 15 // page]), 15 % page].any()
    assert torch.equal(skipped[1][2], q0.view(torch.int16)[2])


@pytest.mark.parametrize("refs,limit", [([1, 1, 1, 0, 0], 9), ([1, 0, 1, 1, 0], 0), ([0, 0, 1, 1, 1], 9)])
@pytest.mark.parametrize("bad", [5, 1 << 30, 0x7FFFFFFF])
def test_compact_reports_bad_pages(refs, limit, bad):
    """Whether pages move or not; the entry stays, what is good is done."""
    refs = np.array(refs, np.int32)
    table = np.concatenate([np.flatnonzero(refs), [-1, bad]])[None].astype(np.int32)
    t, r, st = dev(table), dev(refs), status()
    src, dst, n = dev(np.full(limit + 1, FILL)), dev(np.full(limit + 1, FILL)), dev([FILL])
    ws, size = workspace(len(refs), 1)
    mla.check(mla.mla_pages_compact(t, r, src, dst, n, limit, len(refs), 5, 1, ws, size, st))
    moves = P.compact(table, refs, limit)
    assert st.item() == mla.MLA_DEV_BAD_PAGE and n.item() == len(moves)
    assert np.array_equal(t.cpu(), table) and np.array_equal(r.cpu(), refs)


def test_calls_from_several_threads():
    """Reservations and compactions of large pools (clusters of 16), each thread on a stream and a pool of its own."""
    from concurrent.futures import ThreadPoolExecutor

    def one(i):
        table, refs, lengths = state(9, 16, 8, 40000 + i, 70 + i, share=0.5)
        lengths = lengths // 2
        new = np.full(9, 20 + i)
        new = np.minimum(new, 16 * 8 - lengths)
        with torch.cuda.stream(torch.cuda.Stream()):
            got = run_reserve(table, refs, lengths, new, 16)
            copies = P.reserve(table, refs, lengths, new, 16)
            assert got[2] == copies and np.array_equal(got[0], table) and np.array_equal(got[1], refs)
            t, r, st = dev(table), dev(refs), status()
            src, dst, n = dev(np.full(99, FILL)), dev(np.full(99, FILL)), dev([FILL])
            ws, size = workspace(len(refs), 9)
            mla.check(mla.mla_pages_compact(t, r, src, dst, n, 99, len(refs), 8, 9, ws, size, st))
            moves = P.compact(table, refs, 99)
            assert st.item() == 0 and list(zip(src.tolist(), dst.tolist()))[:n.item()] == moves
            assert np.array_equal(t.cpu(), table) and np.array_equal(r.cpu(), refs)
        return i

    with ThreadPoolExecutor(8) as threads:
        assert list(threads.map(one, range(16))) == list(range(16))


@pytest.mark.parametrize("seed", range(8))
def test_a_walk_of_all_calls(seed):
    """The pool under random calls in a row, each on what the one before left: tables, counts, lengths, lists and a
    cache of two layers are the oracle's after every one, and each sequence's rows hold the tokens of its text."""
    rng = np.random.default_rng(seed)
    B, page, most = [(6, 4, 10), (24, 16, 7), (6, 1, 30), (40, 8, 12)][seed % 4]
    pool = int(B * most * [0.4, 0.9][seed // 4]) + (40000 if seed == 5 else 0)        # (a pool that 16 CTAs look after)
    table, refs, lengths = np.full((B, most), -1, np.int32), np.zeros(pool, np.int32), np.zeros(B, np.int64)
    cache, text, word = np.zeros((2, pool * page), np.int32), [[] for _ in range(B)], 1
    t, r, n, x, st = dev(table), dev(refs), dev(lengths), dev(cache), status()
    src, dst, cnt = dev(np.zeros(pool)), dev(np.zeros(pool)), dev([0])
    ws, size = workspace(pool, B)

    def moved():
        k = cnt.item()
        return list(zip(src[:k].tolist(), dst[:k].tolist()))

    def copies(limit):
        mla.check(mla.mla_pages_copy(x, 4 * page, 2, 4 * page * pool, src, dst, cnt, limit, pool, st))

    done = set()
    for _ in range(40):
        op = ["fork", "free", "compact", "reserve", "reserve", "draft", "draft"][rng.integers(7)]
        expect = 0
        if op == "fork":
            parents = rng.integers(-1, B, B)
            t2, n2 = dev(np.zeros((B, most))), dev(np.zeros(B))
            mla.check(mla.mla_pages_fork(t2, n2, t, n, r, dev(parents), pool, most, B, B, st))
            t, n = t2, n2
            table, lengths = P.fork(table, lengths, refs, parents)
            text = [list(text[p]) if p >= 0 else [] for p in parents]
        elif op == "free":
            keep = rng.integers(0, page * most, B)
            mla.check(mla.mla_pages_free(t, r, n, dev(keep), pool, page, most, B, st))
            P.free(table, refs, lengths, keep, page)
            text = [w[:int(k)] for w, k in zip(text, lengths)]
        elif op == "compact":
            limit = int(rng.integers(0, 20))
            mla.check(mla.mla_pages_compact(t, r, src, dst, cnt, limit, pool, most, B, ws, size, st))
            copies(limit)
            moves = P.compact(table, refs, limit)
            P.copy(cache.reshape(2, pool, page), moves)
            assert moved() == moves
        else:
            new = np.minimum(rng.integers(0, 9, B), page * most - lengths)
            mla.check(mla.mla_pages_reserve(t, r, n, dev(new), src, dst, cnt, pool, page, most, B, ws, size, st))
            copies(B)
            moves = P.reserve(table, refs, lengths, new, page)
            if moves is None:
                expect, op = mla.MLA_DEV_NO_PAGES, "refused"
                assert cnt.item() == 0
            else:
                P.copy(cache.reshape(2, pool, page), moves)
                assert moved() == moves
                # New tokens are written behind each sequence; of drafts, some are kept and what was reserved for the
                # others goes back.
                kept = []
                for b in range(B):
                    words = np.arange(word, word + new[b])
                    word += int(new[b])
                    at = lengths[b] + np.arange(new[b])
                    cache[:, table[b, at // page] * page + at % page] = [words, -words]
                    keeps = sorted(rng.choice(new[b], rng.integers(0, new[b] + 1), replace=False)) if op == "draft" else range(new[b])
                    kept.append(list(keeps))
                    text[b] += [int(words[k]) for k in keeps]
                x.copy_(dev(cache))
                counts = np.array([len(k) for k in kept])
                if op == "draft":
                    pad = np.full((B, 9), -1)
                    for b, k in enumerate(kept):
                        pad[b, :len(k)] = k
                    mla.check(mla.mla_cache_keep_rows(x, 4, 2, 4 * page * pool, n, dev(pad), 9, dev(counts), t, pool, page,
                                                      most, B, st))
                    P.keep_rows(cache, lengths, kept, table, page)
                n += dev(counts)
                lengths = lengths + counts
                if op == "draft":
                    mla.check(mla.mla_pages_free(t, r, n, n, pool, page, most, B, st))
                    P.free(table, refs, lengths, lengths, page)
        done.add(op)
        assert st.item() == expect
        st.zero_()
        assert np.array_equal(t.cpu(), table) and np.array_equal(r.cpu(), refs) and np.array_equal(n.cpu(), lengths)
        assert np.array_equal(x.cpu(), cache)
        for b in range(B):
            at = np.arange(len(text[b]))
            rows = table[b, at // page] * page + at % page
            assert cache[0, rows].tolist() == text[b] and (cache[1, rows] == -cache[0, rows]).all()
    assert {"fork", "free", "compact", "reserve", "draft"} <= done
