"""Attention over the paged cache where it is easily wrong: infinite values that some rows see, lengths beyond the table
under a window, and references that move inside a key tile.  Against the 64-bit plain form of paged_ref."""
import math

import numpy as np
import pytest
import torch

from paged_ref import attend, attend_tol
from test_gpu_paged_attn import ATTN_P, DECODE_P, DT, Case, np64, rand

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mr():
    from cross_model_attention_mr_b200 import mr as m
    assert torch.cuda.is_available() and m.LIB.mr_device_supported() == 1
    return m


# ---------------------------------------------------------------------------------------------- infinite values
INFINITE = [(2, 1), (16, 2), (12, 1), (40, 2), (5, 5)]  # H_q, H_kv: groups of 2, 8, 12, 20 and 1 heads


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("Hq,Hk", INFINITE)
@pytest.mark.parametrize("d", [64, 128])
def test_decode_gives_infinities_that_are_seen(mr, dt, Hq, Hk, d):
    """A row's weights are positive, so an infinite value gives an infinity of its sign whatever its weight's rounding, and
    two of opposite signs NaN; every other column stays as it was."""
    c = Case(mr, [1, 1, 1], [900, 40, 70], Hq, Hk, 16, d, dt, seed=21)
    cache, table, lens, q = c.args()
    want, wl = mr.paged_decode(cache, table, lens, q, return_lse=True, ws=c.ws)
    c.check(want, wl, p_eps=DECODE_P[dt])
    put = [(0, 3, 5, math.inf), (0, 600, 9, -math.inf), (0, 899, d - 1, math.inf), (1, 0, 0, -math.inf),
           (1, 39, 17, math.inf), (2, 11, 30, math.inf), (2, 64, 30, -math.inf)]
    for s, row, col, x in put:
        c.v[c.table[s, row // 16], :, row % 16, col] = x
    got, gl = mr.paged_decode(cache, table, lens, q, return_lse=True, ws=c.ws)
    assert torch.equal(gl, wl)
    for s, _, col, x in put[:5]:
        assert bool((got[:, s, col] == x).all()), (s, col, got[:, s, col].tolist())
    assert bool(torch.isnan(got[:, 2, 30]).all())
    for s, _, col, _ in put:
        got[:, s, col] = want[:, s, col]
    assert torch.equal(got, want)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("new", [6, 60])  # a token each, and in tiles
def test_attn_gives_infinities_to_the_rows_that_see_them(mr, dt, new):
    c = Case(mr, [new], [300 + new], 8, 2, 16, 64, dt, seed=22)
    cache, table, lens, q = c.args()
    want, wl = mr.paged_attn(cache, table, lens, q, c.cu, window=50, return_lse=True, ws=c.ws)
    rows = [(302, 7, math.inf), (299, 40, -math.inf), (270, 63, math.inf)]
    for row, col, x in rows:
        c.v[c.table[0, row // 16], :, row % 16, col] = x
    got, gl = mr.paged_attn(cache, table, lens, q, c.cu, window=50, return_lse=True, ws=c.ws)
    pos = np.arange(300, 300 + new)
    for row, col, x in rows:
        seen = torch.from_numpy((row <= pos) & (row > pos - 50)).cuda()
        assert bool((got[:, seen, col] == x).all()) and bool(torch.isfinite(got[:, ~seen, col]).all())
        got[:, seen, col] = want[:, seen, col]
    c.check(got, gl, window=50, p_eps=(DECODE_P if new <= 8 else ATTN_P)[dt])


# ---------------------------------------------------------------------------------------------- short tables
@pytest.mark.parametrize("dt,pr", [("bf16", 16), ("bf16", 12), ("f32", 16)])
@pytest.mark.parametrize("new,held,pages", [(300, 400, 4), (300, 330, 4), (40, 600, 2), (12, 600, 2), (600, 600, 1)])
@pytest.mark.parametrize("window,sinks", [(1, 0), (10, 0), (200, 0), (10, 3)])
def test_rows_behind_a_short_table_see_nothing(mr, dt, pr, new, held, pages, window, sinks):
    """A length beyond the table: rows whose whole window lies behind it are written as rows that see nothing."""
    Hq, Hk, d = 4, 2, 64
    c = Case(mr, [new, 30], [held, 30], Hq, Hk, pr, d, dt, seed=23)
    cache, table, lens, q = c.args()
    table = table[:, :max(pages, -(-30 // pr))].contiguous()
    cap = table.shape[1] * pr
    O = torch.full_like(q, 5.0)
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    mr.paged_attn(cache, table, lens, q, c.cu, window=window, sinks=sinks, out=O, lse=lse, ws=c.ws)
    assert c.ws.sync_status() == mr.MR_ERR_DEVICE_CHECK
    scale = float(np.float32(1 / math.sqrt(d)))
    pos = np.concatenate([np.arange(held - new, held), np.arange(30)])
    seq = np.repeat([0, 1], [new, 30])
    O, lse, Q = np64(O), np64(lse), np64(q)
    eps = torch.finfo(DT[dt]).eps
    few = new + 30 <= (16 if dt == "bf16" else 8)
    for i, (s, p) in enumerate(zip(seq, pos)):
        j = np.arange(min(p + 1, cap))
        j = j[(j > p - window) | (j < sinks)]
        if len(j) == 0:
            assert np.all(O[:, i] == 0) and np.all(lse[:, i] == -np.inf), (i, p)
            continue
        pages_, rows = c.table.numpy()[s, j // pr], j % pr
        for h in range(Hq):
            K, V = c.clean_k[pages_, h // 2, rows], c.clean_v[pages_, h // 2, rows]
            x = scale * (K @ Q[h, i])
            w = np.exp(x - x.max())
            want, wl = w @ V / w.sum(), x.max() + np.log(w.sum())
            A, S = w @ np.abs(V) / w.sum(), scale * (np.abs(K) @ np.abs(Q[h, i])).max()
            tol, ltol = attend_tol(want, np.float64(wl), A, np.float64(S), d, len(j), eps, ATTN_P[dt])
            assert np.all(np.abs(O[h, i] - want) <= tol) and abs(lse[h, i] - wl) <= ltol, (i, p, h)


# ---------------------------------------------------------------------------------------------- moving references
def test_attn_rounds_probabilities_once(mr):
    """The second half of the first key tile holds scores 0 and -e, the first half one of s > 8 (in base 2): the reference
    moves after the second half's probabilities were made.  63 equal ones carry the output's only values, so a second
    rounding of them would show: rounded twice, 172 of these shifts would put some row beyond half a step of the
    probabilities and half a step of the output."""
    shifts, es = 8 + np.arange(1, 256) / 32, np.arange(1, 512) / 256
    new = 510
    d, past = 64, 128
    e = es[:new]
    for at in range(0, len(shifts), 8):
        Hq = min(8, len(shifts) - at)
        c = Case(mr, [new], [past + new], Hq, 1, 16, d, "bf16", seed=24)
        c.q.zero_()
        for x, y in ((c.k, c.clean_k), (c.v, c.clean_v)):
            live = torch.isfinite(x)
            x.masked_fill_(live, 0.0)
            y[:] = 0.0

        def put(t, clean, row, col, x):
            t[c.table[0, row // 16], 0, row % 16, col] = x
            clean[int(c.table[0, row // 16]), 0, row % 16, col] = x
        for h in range(Hq):
            s = shifts[at + h]
            c.q[h, :new, 0] = math.floor(s)
            c.q[h, :new, 1] = s - math.floor(s)
        c.q[:, :new, 2] = torch.from_numpy(np.floor(e)).bfloat16().cuda()
        c.q[:, :new, 3] = torch.from_numpy(e - np.floor(e)).bfloat16().cuda()
        put(c.k, c.clean_k, 5, 0, 1.0)
        put(c.k, c.clean_k, 5, 1, 1.0)
        for row in range(65, 128):
            put(c.k, c.clean_k, row, 2, -1.0)
            put(c.k, c.clean_k, row, 3, -1.0)
            put(c.v, c.clean_v, row, 7, 1.0)
        assert np.array_equal(np64(c.q)[0, :new, 2] + np64(c.q)[0, :new, 3], e)
        O, lse = mr.paged_attn(*c.args(), c.cu, scale=math.log(2.0), window=1, sinks=128, return_lse=True, ws=c.ws)
        # (scores are sums of two products of small fractions: exact, but for the scale; the bound's terms for them are
        # far below the rounding's)
        Q, scale = np64(c.q)[:, :new], float(np.float32(math.log(2.0)))
        top, low = scale * (Q[..., 0] + Q[..., 1]), -scale * (Q[..., 2] + Q[..., 3])
        # 63 + 1 keys at 0 in the first tile and the row's own, one at `top`, 63 at `low`
        total = 65 + np.exp(top) + 63 * np.exp(low)
        want = 63 * np.exp(low) / total
        tol, ltol = attend_tol(want[..., None], np.log(total), want[..., None], top, d, 129, torch.finfo(torch.bfloat16).eps,
                               2.0 ** -8)
        err = np.abs(np64(O)[:, :new, 7] - want)
        assert np.all(err <= tol[..., 0]), float((err / tol[..., 0]).max())
        assert np.all(np.abs(np64(lse)[:, :new] - np.log(total)) <= ltol)
        assert c.ws.sync_status() == mr.MR_OK


# ---------------------------------------------------------------------------------------------- more rows than there are
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_append_with_an_upper_bound_of_the_rows(mr, dt):
    """total_q may be an upper bound: tensors that end with the last sequence's rows are enough.  (Theirs lie in front of a
    larger allocation here, so that nothing else is in reach of rows behind them.)"""
    import ctypes
    T, most, Hq, Hk, d, pr = 37, 5000, 4, 2, 64, 16
    each = Hq + 2 * Hk
    x = torch.full((most, each, d), math.nan, dtype=DT[dt], device="cuda")
    x[:T] = rand((T, each, d), dt, 25)
    out = torch.full((most, Hq, d), 5.0, dtype=DT[dt], device="cuda")
    lens = torch.tensor([20, 60], dtype=torch.int32).cuda()
    cu = torch.tensor([0, 12, T], dtype=torch.int32).cuda()
    table = torch.arange(8, dtype=torch.int32).view(2, 4).cuda()
    a, b = (mr.KVCache(torch.full((8, Hk, pr, d), 9.0, dtype=DT[dt], device="cuda"),
                       torch.full((8, Hk, pr, d), -9.0, dtype=DT[dt], device="cuda")) for _ in range(2))
    r, ws = mr.Rope(d), mr.Workspace(256)
    esize = x.element_size()
    rows = lambda t, head, heads: mr.Rows(t.data_ptr() + head * d * esize, d, heads * d)
    seqs = mr.KvSeqs(table.data_ptr(), lens.data_ptr(), 4, 2)
    ref = ctypes.byref
    st = mr.LIB.mr_kv_append(ref(a.c), ref(seqs), ref(r.c), ref(rows(x, 0, each)), ref(rows(out, 0, Hq)), Hq,
                             ref(rows(x, Hq, each)), ref(rows(x, Hq + Hk, each)), cu.data_ptr(), most, ws.ptr, ws.nbytes,
                             torch.cuda.current_stream().cuda_stream)
    assert st == mr.MR_OK and ws.sync_status() == mr.MR_OK
    q, k, v = (t.transpose(0, 1) for t in x[:T].split([Hq, Hk, Hk], 1))
    want = mr.kv_append(b, table, lens, k, v, cu_q=cu, rope=r, Q=q)
    assert torch.equal(out[:T].transpose(0, 1), want) and bool((out[T:] == 5.0).all())
    assert torch.equal(a.k, b.k) and torch.equal(a.v, b.v)


# ---------------------------------------------------------------------------------------------- rejected rows
def test_rejected_rows_behind_a_window_that_has_moved_on(mr):
    """Drafted rows are appended, attended to and partly rejected, under a window that gives pages up; the tables go to the
    calls as the pool has them, with -1 for pages that were given up, so a page that is needed after all would show."""
    from test_gpu_paged_serving import Server

    class Plain(Server):
        def tables(self, seqs):
            t, n = self.pool.tables(seqs)
            return torch.from_numpy(t).cuda(), torch.from_numpy(n).cuda()

    s = Plain(mr, 14, 16, 8, 2, 64, seed=26)
    window, sinks = 40, 20
    a = s.pool.open()
    s.append([a], [100])
    refused = freed = 0
    rng = np.random.default_rng(5)
    for _ in range(30):
        freed += s.pool.slide(a, window, sinks)
        held = s.pool.rows(a)
        q, table, lens, cu = s.append([a], [6])
        O, lse = mr.paged_attn(s.cache, table, lens, q, cu, window=window, sinks=sinks, return_lse=True, ws=s.ws)
        s.check(O, lse, q, [a], [6], window, sinks, 2.0 ** -16)
        with pytest.raises(mr.MRError):
            s.pool.truncate(a, held - 16)      # a page that the next query would see is gone
        refused += 1
        keep = held + int(rng.integers(0, 7))
        s.pool.truncate(a, keep)
        s.told[a] = tuple(x[:, :keep] for x in s.told[a])
        s.decode([a], window, sinks)
    b = s.pool.fork(a, s.pool.rows(a))
    s.told[b] = s.told[a]
    s.decode([a, b], window, sinks)
    assert refused == 30 and freed >= 5 and -1 in s.pool.tables([a])[0]


# ---------------------------------------------------------------------------------------------- no workspace given
def test_status_of_calls_without_a_workspace(mr):
    import threading
    c = Case(mr, [1, 20], [40, 20], 2, 1, 16, 64, "bf16", seed=27)
    cache, table, lens, q = c.args()
    bad = table.clone()
    bad[0, 1] = 10 ** 6
    k, v = rand((1, 2, 64), "bf16", 1), rand((1, 2, 64), "bf16", 2)
    two = q[:, :2].contiguous()
    pairs = torch.tensor([[0, 1], [2, 1]], dtype=torch.int32).cuda()
    calls = [lambda t, **kw: mr.paged_decode(cache, t, lens, two, **kw),
             lambda t, **kw: mr.paged_attn(cache, t, lens, q, c.cu, **kw),
             lambda t, **kw: mr.kv_append(cache, t, lens - 10, k, v, **kw),
             lambda t, **kw: mr.pages_copy([cache.k], pairs if t is bad else pairs[:1], **kw)]
    st = torch.cuda.Stream()
    for call in calls:
        for kw in ({}, {"stream": st}):
            torch.cuda.synchronize()
            call(bad, **kw)
            assert mr.last_status() == mr.MR_ERR_DEVICE_CHECK
            with pytest.raises((ValueError, TypeError, mr.MRError)):
                mr.paged_decode(cache, bad, lens, two, window=-1)        # a refused call has no status
            call(table, ws=c.ws)                                         # nor is one asked for with a workspace of its own
            assert mr.last_status() == mr.MR_ERR_DEVICE_CHECK
            torch.cuda.synchronize()
            call(table, **kw)
            assert mr.last_status() == mr.MR_OK
    calls[0](bad)
    seen = []

    def other():
        with pytest.raises(ValueError):
            mr.last_status()
        calls[0](table)
        seen.append(mr.last_status())
    th = threading.Thread(target=other)
    th.start()
    th.join()
    assert seen == [mr.MR_OK] and mr.last_status() == mr.MR_ERR_DEVICE_CHECK


# ---------------------------------------------------------------------------------------------- tokens or tiles
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("spread", ["one each", "all in one", "some"])
def test_few_rows_however_they_are_spread(mr, dt, spread):
    """Batches whose rows' way through the library depends on the lengths on the device (pages are shared between the
    sequences, so that they can be long)."""
    n, pr, d, Hq, Hk, long = 96, 64, 128, 4, 2, 7000
    new = {"one each": [1] * n, "all in one": [0] * 40 + [n] + [0] * (n - 41), "some": [2, 0, 0, 0, 5, 1] * 16}[spread]
    held = [long if i % 3 == 1 else 65 + 7 * i for i in range(n)]
    pages = -(-long // pr)
    k, v = rand((pages, Hk, pr, d), dt, 31), rand((pages, Hk, pr, d), dt, 32)
    cache = mr.KVCache(k, v)
    # (wide tables: the host's bound is the table, not the lengths)
    table = torch.zeros((n, 4 * pages), dtype=torch.int32)
    table[:, :pages] = torch.stack([torch.randperm(pages, generator=torch.Generator().manual_seed(i)) for i in range(n)])
    lens = torch.tensor(held, dtype=torch.int32)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32).cuda()
    q = rand((Hq, sum(new), d), dt, 33)
    ws = mr.Workspace(mr.paged_workspace_bytes(cache, Hq, n))
    O, lse = mr.paged_attn(cache, table.cuda(), lens.cuda(), q, cu, return_lse=True, ws=ws)
    assert ws.sync_status() == mr.MR_OK
    want, wl, A, S = attend(np64(q), np64(k), np64(v), table.numpy(), held, new, float(np.float32(1 / math.sqrt(d))))
    tol, ltol = attend_tol(want, wl, A, S, d, long, torch.finfo(DT[dt]).eps, ATTN_P[dt])
    assert np.all(np.abs(np64(O) - want) <= tol) and np.all(np.abs(np64(lse) - wl) <= ltol)


def test_how_rows_are_spread_decides(mr):
    """With the test hook the tensor-core kernel's tiles run into their time limit, so the status tells which way a call
    took: rows of their own where each sequence has one, tiles where one sequence has them all, also when a captured call
    meets other lengths and offsets."""
    n, pr, Hk, d, long = 64, 128, 4, 128, 20000
    cache = mr.KVCache(*(rand((-(-long // pr), Hk, pr, d), "bf16", 34 + i) for i in range(2)))
    table = torch.arange(-(-long // pr), dtype=torch.int32).expand(n, -1).contiguous().cuda()
    lens = torch.full((n,), long, dtype=torch.int32).cuda()
    offsets = lambda new: torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32).cuda()
    each, one = offsets([1] * n), offsets([0] * 7 + [n] + [0] * (n - 8))
    q = rand((8, n, d), "bf16", 36)
    ws = mr.Workspace(mr.paged_workspace_bytes(cache, 8, n))
    plain = {}
    for name, cu in (("each", each), ("one", one)):
        plain[name] = mr.paged_attn(cache, table, lens, q, cu, ws=ws)
        assert ws.sync_status() == mr.MR_OK
    assert torch.equal(plain["each"], mr.paged_decode(cache, table, lens, q))
    cu, out = each.clone(), torch.zeros_like(q)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mr.paged_attn(cache, table, lens, q, cu, out=out, ws=ws)
    for name, to in (("one", one), ("each", each), ("one", one)):
        cu.copy_(to)
        g.replay()
        assert ws.sync_status() == mr.MR_OK and torch.equal(out, plain[name])
    assert mr.LIB.mr_debug_set(1_000_000, 1) == mr.MR_OK
    try:
        for to, want in ((each, mr.MR_OK), (one, mr.MR_ERR_TIMEOUT)):
            mr.paged_attn(cache, table, lens, q, to, ws=ws)
            assert ws.sync_status() == want
        lens.fill_(200)                              # little is read again: rows of their own either way
        mr.paged_attn(cache, table, lens, q, one, ws=ws)
        assert ws.sync_status() == mr.MR_OK
        # a short table is recorded whichever way is taken
        lens.fill_(long + 5000)
        mr.paged_attn(cache, table, lens, q, each, ws=ws)
        assert ws.sync_status() == mr.MR_ERR_DEVICE_CHECK
    finally:
        assert mr.LIB.mr_debug_set(0, 0) == mr.MR_OK


# ---------------------------------------------------------------------------------------------- many pairs, bf16 gradients
def test_page_copies_of_more_pairs_than_threads(mr):
    """Conflicts between pairs that the same thread of a block looks at, one round after the other."""
    n, most = 4000, 1500
    pool = torch.arange(n * 64, dtype=torch.float32, device="cuda").view(n, 1, 1, 64).contiguous()
    order = torch.randperm(n, generator=torch.Generator().manual_seed(3)).to(torch.int32)
    pairs = torch.stack([order[:most], order[most: 2 * most]], 1)
    ws = mr.Workspace(mr.pages_copy_workspace_bytes())
    old = pool.clone()
    mr.pages_copy([pool], pairs.cuda(), ws=ws)
    assert ws.sync_status() == mr.MR_OK
    want = old.clone()
    want[pairs[:, 1].long()] = old[pairs[:, 0].long()]
    assert torch.equal(pool, want)
    # far apart in the list: a destination named twice (the first counts), sources that others write, a swap, pages that
    # do not exist, and a page with itself, which counts for nothing
    bad = pairs.clone()
    bad[1400, 1] = bad[3, 1]                     # 1400 is skipped
    bad[700, 0] = bad[1301, 1]                   # 700 is skipped
    bad[20] = torch.tensor([int(bad[1290, 1]), int(bad[1290, 0])])  # 20 and 1290 would swap: both are skipped
    bad[900, 0], bad[901, 1] = n, -1             # 900 and 901 are skipped
    bad[1450, 0] = bad[1450, 1]
    pool.copy_(old)
    mr.pages_copy([pool], bad.cuda(), ws=ws)
    assert ws.sync_status() == mr.MR_ERR_DEVICE_CHECK
    want = old.clone()
    keep = [i for i in range(most) if i not in (1400, 700, 20, 1290, 900, 901, 1450)]
    want[bad[keep, 1].long()] = old[bad[keep, 0].long()]
    assert torch.equal(pool, want)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("scaling", ["none", "ramp"])
def test_adjoint_of_the_rotation_in_bf16(mr, interleaved, scaling):
    """The formula in 64 bits, and differences of the forward call: the rotation is linear, so a difference over a whole
    unit has no other error than the forward's rounding."""
    from paged_ref import inv_freq
    from test_gpu_paged_rope import check_rotated
    H, T, d, rot = 3, 50, 128, 96
    kw = dict(scaling=scaling, factor=4.0 if scaling == "ramp" else 1.0)
    g = rand((H, T, d), "bf16", 41)
    pos = torch.randint(0, 100000, (T,), generator=torch.Generator().manual_seed(42), dtype=torch.int32)
    r = mr.Rope(d, rot_dim=rot, interleaved=interleaved, orig_len=4096, mscale=1.125, **kw)
    gx = mr.rope(r, g, pos.cuda(), adjoint=True)
    check_rotated(gx, g, pos.numpy(), inv_freq(rot, **kw), "bf16", interleaved, 1.125, -1)
    step = torch.zeros((d, T, d), dtype=torch.bfloat16, device="cuda")
    step[torch.arange(d), :, torch.arange(d)] = 1.0      # head e: a unit of element e in every row
    diff = np64(mr.rope(r, step, pos.cuda()))            # [e][row][element]
    for h in range(H):
        want = np.einsum("etc,tc->te", diff, np64(g)[h])
        # two elements of a column are not zero, each off by half a step (2^-8 of at most 1.125) and 2^-21 for the
        # rotation; gx itself is rounded once
        tol = (2.0 ** -8 + 2.0 ** -20) * 1.125 * 2 * np.abs(np64(g)[h]).max(1, keepdims=True) + 2.0 ** -8 * np.abs(want)
        assert np.all(np.abs(want - np64(gx)[h]) <= tol)


# ---------------------------------------------------------------------------------------------- the queries' own place
@pytest.mark.parametrize("dt,pr", [("bf16", 16), ("bf16", 12), ("f32", 16)])
@pytest.mark.parametrize("new,held", [([1, 1, 1], [9000, 40, 3]), ([200, 3, 90], [3000, 3, 500]), ([5, 2], [700, 2])])
def test_outputs_in_the_queries_place(mr, dt, pr, new, held):
    c = Case(mr, new, held, 8, 2, pr, 128, dt, seed=43)
    cache, table, lens, q = c.args()
    want = mr.paged_attn(cache, table, lens, q, c.cu, ws=c.ws)
    got = q.clone()
    mr.paged_attn(cache, table, lens, got, c.cu, out=got, ws=c.ws)
    assert torch.equal(got, want)
    if max(new) == 1:
        want = mr.paged_decode(cache, table, lens, q, ws=c.ws)
        got = q.clone()
        mr.paged_decode(cache, table, lens, got, out=got, ws=c.ws)
        assert torch.equal(got, want)
