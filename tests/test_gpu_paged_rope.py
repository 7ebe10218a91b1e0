"""Rotary positions, appending to the paged cache, and page copies on the GPU, against 64-bit plain forms."""
import numpy as np
import pytest
import torch

from paged_ref import inv_freq, rotate, rotate_tol

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def mr():
    from cross_model_attention_mr_b200 import mr as m
    assert torch.cuda.is_available() and m.LIB.mr_device_supported() == 1
    return m


def rand(shape, dt, seed):
    g = torch.Generator(device="cpu")
    g.manual_seed(seed)
    return torch.randn(shape, generator=g).to(DT[dt]).cuda()


def np64(t):
    return t.detach().cpu().double().numpy()


def check_rotated(got, x, pos, freq, dt, interleaved=False, mscale=1.0, sign=1):
    y = rotate(np64(x), pos, freq, interleaved, mscale, sign)
    tol = rotate_tol(np64(x), y, 2 * len(freq), torch.finfo(DT[dt]).eps, interleaved, mscale)
    err = np.abs(np64(got) - y)
    assert np.all(err <= tol), float((err / np.maximum(tol, 1e-300)).max())
    rest = np64(x)[..., 2 * len(freq):]
    assert np.array_equal(np64(got)[..., 2 * len(freq):], rest)  # unrotated elements are copied


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("H,T,d,rot", [(1, 1, 64, 64), (3, 1, 128, 128), (5, 33, 128, 64), (2, 300, 64, 16),
                                       (3, 7, 8, 2), (2, 9, 96, 90), (1, 5, 256, 256), (33, 650, 64, 32)])
def test_rope_against_64_bits(mr, dt, interleaved, H, T, d, rot):
    x = rand((H, T, d), dt, 1)
    pos = torch.randint(0, 70000, (T,), generator=torch.Generator().manual_seed(2), dtype=torch.int32)
    r = mr.Rope(d, rot_dim=rot, interleaved=interleaved, mscale=1.25)
    got = mr.rope(r, x, pos.cuda())
    check_rotated(got, x, pos.numpy(), inv_freq(rot), dt, interleaved, 1.25)


@pytest.mark.parametrize("scaling,factor", [("linear", 4.0), ("base", 8.0), ("ramp", 4.0)])
def test_rope_far_positions_and_scaling(mr, scaling, factor):
    pos = torch.tensor([0, 1, 2 ** 20 + 1, 2 ** 31 - 1, -5, -2 ** 31, 131071], dtype=torch.int32)
    x = rand((2, 7, 128), "f32", 3)
    r = mr.Rope(128, scaling=scaling, factor=factor, orig_len=4096)
    got = mr.rope(r, x, pos.cuda())
    check_rotated(got, x, pos.numpy(), inv_freq(128, scaling=scaling, factor=factor), "f32")


def test_rope_adjoint_is_the_gradient(mr):
    """<rope(x), g> == <x, adjoint(g)>, the adjoint equals the formula, and it equals differences of the
    forward call (which is linear, so a difference over a whole unit is exact up to rounding)."""
    x, g = rand((2, 40, 64), "f32", 4), rand((2, 40, 64), "f32", 5)
    pos = torch.arange(100, 140, dtype=torch.int32)
    r = mr.Rope(64, rot_dim=48, interleaved=True, mscale=0.7)
    y, gx = mr.rope(r, x, pos.cuda()), mr.rope(r, g, pos.cuda(), adjoint=True)
    check_rotated(gx, g, pos.numpy(), inv_freq(48), "f32", True, 0.7, -1)
    a, b = float((np64(y) * np64(g)).sum()), float((np64(x) * np64(gx)).sum())
    # each element of y and gx is within 2^-21 (|x_a| + |x_b|): summed over 5120 elements against |g| or |x|
    bound = 2.0 ** -21 * 2 * float(np.abs(np64(x)).sum() + np.abs(np64(g)).sum()) * 5
    assert abs(a - b) <= bound
    for e in (0, 1, 47, 60):
        step = torch.zeros_like(x)
        step[1, 17, e] = 1.0
        d = np64(mr.rope(r, step, pos.cuda()))
        assert abs((d * np64(g)).sum() - np64(gx)[1, 17, e]) <= 2.0 ** -19 * (np.abs(np64(g)[1, 17]).max() + 1)


def test_rope_strides_in_place_and_alignment(mr):
    pos = torch.arange(50, dtype=torch.int32).cuda()
    r = mr.Rope(64)
    base = rand((50, 6, 64), "bf16", 6)
    want = mr.rope(r, base.transpose(0, 1).contiguous(), pos)
    got = mr.rope(r, base.transpose(0, 1), pos)                       # [rows][H][d] storage
    assert torch.equal(got, want)
    out = torch.empty_like(base).transpose(0, 1)
    assert torch.equal(mr.rope(r, base.transpose(0, 1), pos, out=out), want)
    odd = torch.empty(6 * 50 * 67 + 3, dtype=torch.bfloat16, device="cuda").fill_(7.0)
    view = odd[3:].view(6, 50, 67)[..., :64]                          # odd strides, 2-byte alignment
    view.copy_(base.transpose(0, 1))
    got = mr.rope(r, view, pos)
    assert torch.equal(got, want)
    mr.rope(r, view, pos, out=view)
    assert torch.equal(view, want)
    assert bool((odd[3:].view(6, 50, 67)[..., 64:] == 7.0).all()) and bool((odd[:3] == 7.0).all())
    one = rand((1, 50, 64), "bf16", 8)
    many = mr.rope(r, one.expand(4, 50, 64), pos)                     # one head broadcast: stride 0
    assert torch.equal(many, mr.rope(r, one, pos).expand(4, 50, 64))
    assert mr.rope(r, base.transpose(0, 1)[:, :0], pos[:0]).shape == (6, 0, 64)


# ---------------------------------------------------------------------------------------------- append
def make_cache(mr, n_pages, H, pr, d, dt, fill=9.0):
    c = mr.KVCache.empty(n_pages, H, pr, d, DT[dt])
    c.k.fill_(fill)
    c.v.fill_(-fill)
    return c


APPENDS = [  # new rows and rows held of each sequence, H_q, H_kv, page_rows, d
    ([1], [1], 1, 1, 16, 64), ([1, 1, 1], [1, 17, 64], 8, 2, 16, 128), ([5, 0, 33, 1], [5, 3, 70, 200], 4, 4, 64, 64),
    ([100, 31], [131, 31], 7, 1, 7, 128), ([700], [900], 28, 4, 128, 128), ([3, 2], [2, 2], 2, 1, 16, 64),
]


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("case", range(len(APPENDS)))
@pytest.mark.parametrize("turned", [True, False])
def test_append_against_64_bits(mr, dt, case, turned):
    new, held, Hq, Hk, pr, d = APPENDS[case]
    n, T = len(new), sum(new)
    per = max(max(-(-h // pr) for h in held), 1) + 1
    table = torch.randperm(n * per, generator=torch.Generator().manual_seed(case)).to(torch.int32).view(n, per)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32)
    behind = 3                                       # rows of Q, K, V behind the last sequence
    q, k, v = rand((Hq, T + behind, d), dt, 1), rand((Hk, T + behind, d), dt, 2), rand((Hk, T + behind, d), dt, 3)
    c = make_cache(mr, n * per + 2, Hk, pr, d, dt)
    r = mr.Rope(d, rot_dim=d // 2, interleaved=bool(case % 2)) if turned else None
    q_out = torch.full_like(q, 5.0)
    ws = mr.Workspace(mr.paged_workspace_bytes(c, Hq, n))
    got = mr.kv_append(c, table.cuda(), torch.tensor(held, dtype=torch.int32).cuda(), k, v, cu_q=cu.cuda(), rope=r, Q=q,
                       q_out=q_out, ws=ws)
    assert got is q_out and ws.sync_status() == mr.MR_OK
    assert bool((q_out[:, T:] == 5.0).all())
    want_k, want_v = np.full(c.k.shape, 9.0), np.full(c.v.shape, -9.0)
    pos = np.concatenate([np.arange(h - m, h) for m, h in zip(new, held)])
    seq = np.concatenate([np.full(m, s) for s, m in enumerate(new)]).astype(int)
    freq = inv_freq(d // 2)
    kr = rotate(np64(k)[:, :T], pos, freq, bool(case % 2)) if turned else np64(k)[:, :T]
    tol = np.zeros(c.k.shape)
    ktol = rotate_tol(np64(k)[:, :T], kr, d // 2, torch.finfo(DT[dt]).eps, bool(case % 2)) if turned else np.zeros(kr.shape)
    for t in range(T):
        if pos[t] < 0:                               # a row in front of the sequence's start
            assert bool((q_out[:, t] == 0).all())
            continue
        page, row = int(table[seq[t], pos[t] // pr]), pos[t] % pr
        want_k[page, :, row], want_v[page, :, row] = kr[:, t], np64(v)[:, t]
        tol[page, :, row] = ktol[:, t]
    assert np.all(np.abs(np64(c.k) - want_k) <= tol)     # rows that nothing was written to are exact
    assert np.array_equal(np64(c.v), want_v)
    live = np.nonzero(pos >= 0)[0]
    if turned:
        check_rotated(q_out[:, live], q[:, live], pos[live], freq, dt, bool(case % 2))
    else:
        assert torch.equal(q_out[:, live], q[:, live])


def test_append_one_row_each_strided_and_without_queries(mr):
    """The decoding form: no offsets, projections laid out [rows][heads][d] in one buffer."""
    n, Hq, Hk, d, pr = 6, 8, 2, 128, 16
    qkv = rand((n, Hq + 2 * Hk, d), "bf16", 1)
    q, k, v = (x.transpose(0, 1) for x in qkv.split([Hq, Hk, Hk], 1))
    lens = torch.tensor([1, 16, 17, 33, 2, 48], dtype=torch.int32).cuda()
    table = torch.arange(n * 3, dtype=torch.int32).view(n, 3).cuda()
    r = mr.Rope(d)
    a, b = make_cache(mr, n * 3, Hk, pr, d, "bf16"), make_cache(mr, n * 3, Hk, pr, d, "bf16")
    qo = mr.kv_append(a, table, lens, k, v, rope=r, Q=q)
    cu = torch.arange(n + 1, dtype=torch.int32).cuda()
    mr.kv_append(b, table, lens, k.contiguous(), v.contiguous(), cu_q=cu, rope=r)
    assert torch.equal(a.k, b.k) and torch.equal(a.v, b.v)
    assert torch.equal(qo, mr.rope(r, q, lens - 1))
    mr.kv_append(a, table, lens, k, v, rope=r, Q=q, q_out=q)          # the queries in place
    assert torch.equal(q, qo)


def test_append_reports_what_it_cannot_store(mr):
    Hk, d, pr = 2, 64, 16
    k, v = rand((Hk, 3, d), "bf16", 1), rand((Hk, 3, d), "bf16", 2)
    for bad, lens in (([[0, 8], [1, 2], [3, 4]], [17, 1, 1]), ([[0, -1], [1, 2], [3, 4]], [32, 1, 1]),
                      ([[0, 5], [1, 2], [3, 4]], [33, 1, 1])):
        c = make_cache(mr, 8, Hk, pr, d, "bf16")
        ws = mr.Workspace(mr.paged_workspace_bytes(c, Hk, 3))
        table = torch.tensor(bad, dtype=torch.int32).cuda()
        mr.kv_append(c, table, torch.tensor(lens, dtype=torch.int32).cuda(), k, v, ws=ws)
        assert ws.sync_status() == mr.MR_ERR_DEVICE_CHECK
        want = torch.full_like(c.k, 9.0)
        want[1, :, 0], want[3, :, 0] = k[:, 1], k[:, 2]               # the good rows are there, nothing else is
        assert torch.equal(c.k, want)
        mr.kv_append(c, torch.tensor([[0, 5], [1, 2], [3, 4]], dtype=torch.int32).cuda(),
                     torch.tensor([1, 1, 1], dtype=torch.int32).cuda(), k, v, ws=ws)
        assert ws.sync_status() == mr.MR_OK                            # the status is the last call's


def test_append_many_sequences(mr):
    """More sequences than one round of the search covers, many of them without new rows."""
    n, Hk, d, pr = 1500, 1, 64, 16
    rng = np.random.default_rng(3)
    new = rng.integers(0, 4, n)
    new[:40] = 0
    held = new + rng.integers(0, 10, n)
    T = int(new.sum())
    cu = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32).cuda()
    k, v = rand((Hk, T, d), "f32", 1), rand((Hk, T, d), "f32", 2)
    c = make_cache(mr, n, Hk, pr, d, "f32")
    table = torch.arange(n, dtype=torch.int32).view(n, 1).cuda()
    mr.kv_append(c, table, torch.tensor(held, dtype=torch.int32).cuda(), k, v, cu_q=cu)
    want = torch.full_like(c.k, 9.0)
    seq = torch.tensor(np.repeat(np.arange(n), new)).cuda()
    pos = torch.tensor(np.concatenate([np.arange(h - m, h) for m, h in zip(new, held)])).cuda()
    want[seq, :, pos] = k.transpose(0, 1)
    assert torch.equal(c.k, want)


# ---------------------------------------------------------------------------------------------- page copies
@pytest.mark.parametrize("shape,dt", [((40, 1, 16, 64), "bf16"), ((40, 3, 7, 64), "f32"), ((20, 8, 128, 128), "bf16"),
                                      ((300, 1, 1, 64), "f32")])
def test_pages_copy(mr, shape, dt):
    pools = [rand(shape, dt, i) for i in range(3)]
    order = torch.randperm(shape[0], generator=torch.Generator().manual_seed(1)).to(torch.int32)
    h = shape[0] // 2
    src = order[:h].clone()
    src[1] = src[0]                                  # one source, two destinations
    pairs = torch.stack([src, order[h: 2 * h]], 1)
    pairs = torch.cat([pairs, torch.tensor([[int(order[2]), int(order[2])]], dtype=torch.int32)])  # onto itself
    ws = mr.Workspace(mr.pages_copy_workspace_bytes())
    want = [p.clone() for p in pools]
    for w in want:
        w[pairs[:, 1].long()] = w[pairs[:, 0].long()]
    mr.pages_copy(pools, pairs.cuda(), ws=ws)
    assert ws.sync_status() == mr.MR_OK
    assert all(torch.equal(p, w) for p, w in zip(pools, want))
    mr.pages_copy(pools, pairs[:0].cuda(), ws=ws)    # no pairs
    assert ws.sync_status() == mr.MR_OK


def test_pages_copy_skips_conflicts(mr):
    pool = rand((16, 1, 16, 64), "f32", 1)
    old = pool.clone()
    pairs = [[0, 8], [8, 9], [1, 10], [2, 10], [3, 16], [-1, 11], [4, 12], [4, 13], [5, 5], [5, 14], [6, 15], [15, 6]]
    ws = mr.Workspace(mr.pages_copy_workspace_bytes())
    mr.pages_copy([pool], torch.tensor(pairs, dtype=torch.int32).cuda(), ws=ws)
    assert ws.sync_status() == mr.MR_ERR_DEVICE_CHECK
    want = old.clone()
    # 8 is written, so it is not a source; 10 takes its first pair; 5 with itself counts for nothing; 6 and 15 would
    # swap: both are skipped
    for a, b in ((0, 8), (1, 10), (4, 12), (4, 13), (5, 14)):
        want[b] = old[a]
    assert torch.equal(pool, want)


def test_many_pools_in_one_call(mr):
    pools = list(rand((300, 6, 1, 1, 64), "bf16", 1).unbind(0))
    old = [p.clone() for p in pools]
    mr.pages_copy(pools, torch.tensor([[0, 5], [1, 3]], dtype=torch.int32).cuda())
    for p, o in zip(pools, old):
        o[5], o[3] = o[0].clone(), o[1].clone()
        assert torch.equal(p, o)


# ---------------------------------------------------------------------------------------------- streams, graphs
def test_streams_and_graphs(mr):
    c = make_cache(mr, 12, 2, 16, 64, "bf16")
    table = torch.arange(12, dtype=torch.int32).view(4, 3).cuda()
    lens = torch.tensor([1, 20, 33, 48], dtype=torch.int32).cuda()
    q, k, v = rand((4, 4, 64), "bf16", 1), rand((2, 4, 64), "bf16", 2), rand((2, 4, 64), "bf16", 3)
    r = mr.Rope(64)
    ws = mr.Workspace(mr.paged_workspace_bytes(c, 4, 4))
    qo = torch.zeros_like(q)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        mr.kv_append(c, table, lens, k, v, rope=r, Q=q, q_out=qo, ws=ws)
    st.synchronize()
    want_k, want_q = c.k.clone(), qo.clone()
    c.k.fill_(9.0)
    qo.zero_()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mr.kv_append(c, table, lens, k, v, rope=r, Q=q, q_out=qo, ws=ws)
        mr.pages_copy([c.k], table[:1, :2].contiguous(), ws=ws)
    g.replay()
    torch.cuda.synchronize()
    want_k[1] = want_k[0]
    assert torch.equal(c.k, want_k) and torch.equal(qo, want_q)
    lens += 1                                        # new lengths reach the captured call
    lens[3] = 2
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(qo, mr.rope(r, q, lens - 1))
    assert ws.sync_status() == mr.MR_OK
