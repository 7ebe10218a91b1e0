"""Attention of new rows over the paged cache on the GPU, against a 64-bit plain form."""
import math

import numpy as np
import pytest
import torch

from paged_ref import attend, attend_tol

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
# half a step of the probabilities in the second product: two bf16 parts (2^-8 of 2^-8), or fp32
DECODE_P = {"bf16": 2.0 ** -16, "f32": 0.0}
# one bf16 part, or fp32
ATTN_P = {"bf16": 2.0 ** -8, "f32": 0.0}


@pytest.fixture(scope="module")
def mr():
    from cross_model_attention_mr_b200 import mr as m
    assert torch.cuda.is_available() and m.LIB.mr_device_supported() == 1
    return m


def rand(shape, dt, seed, scale=1.0):
    g = torch.Generator(device="cpu")
    g.manual_seed(seed)
    return (scale * torch.randn(shape, generator=g)).to(DT[dt]).cuda()


def np64(t):
    return t.detach().cpu().double().numpy()


class Case:
    """A cache with shuffled pages whose rows that no sequence holds are NaN, and the new rows' queries."""

    def __init__(self, mr, new, held, Hq, Hk, pr, d, dt, seed=0, spread=1.0, behind=0):
        n = len(new)
        self.new, self.held, self.dt, self.d = list(new), list(held), dt, d
        self.per = max(max(-(-h // pr) for h in held), 1) + 1
        order = torch.randperm(n * self.per + 1, generator=torch.Generator().manual_seed(seed)).to(torch.int32)
        self.table = order[: n * self.per].view(n, self.per).contiguous()
        self.lens = torch.tensor(held, dtype=torch.int32)
        shape = (n * self.per + 1, Hk, pr, d)
        self.k, self.v = rand(shape, dt, seed + 1), rand(shape, dt, seed + 2)
        live = torch.zeros(shape[0], pr, dtype=torch.bool)
        for s, h in enumerate(held):
            for j in range(max(h, 0)):
                live[self.table[s, j // pr], j % pr] = True
        dead = (~live).cuda()[:, None, :, None]
        self.clean_k, self.clean_v = np64(self.k), np64(self.v)
        self.k.masked_fill_(dead, math.nan)
        self.v.masked_fill_(dead, math.inf)
        self.cache = mr.KVCache(self.k, self.v)
        self.T = sum(new)
        self.q = rand((Hq, self.T + behind, d), dt, seed + 3, spread)
        self.cu = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32).cuda()
        self.ws = mr.Workspace(mr.paged_workspace_bytes(self.cache, Hq, n))
        self.mr = mr

    def args(self):
        return self.cache, self.table.cuda(), self.lens.cuda(), self.q

    def hide(self, window, sinks):
        """What no new row sees becomes NaN as well."""
        for s, (n, h) in enumerate(zip(self.new, self.held)):
            lo = max(h - max(n, 1) - window + 1, 0) if window else 0
            for j in range(min(sinks, lo) if window else 0, lo):
                page, row = self.table[s, j // self.k.shape[2]], j % self.k.shape[2]
                self.k[page, :, row] = math.nan
                self.v[page, :, row] = math.nan

    def check(self, O, lse, scale=None, window=0, sinks=0, p_eps=0.0):
        scale = 1.0 / math.sqrt(self.d) if scale is None else scale
        scale = float(np.float32(scale))
        want, wl, A, S = attend(np64(self.q)[:, : self.T], self.clean_k, self.clean_v, self.table.numpy(),
                                self.lens.numpy(), self.new, scale, window, sinks)
        tol, ltol = attend_tol(want, wl, A, S, self.d, max(self.held), torch.finfo(DT[self.dt]).eps, p_eps)
        err = np.abs(np64(O)[:, : self.T] - want)
        assert np.all(err <= tol), (float((err / np.maximum(tol, 1e-300)).max()), np.argwhere(~(err <= tol))[:4].tolist())
        got = np64(lse)[:, : self.T]
        full = np.isfinite(wl)
        assert np.array_equal(got[~full], wl[~full])
        off = np.abs(got[full] - wl[full])
        assert np.all(off <= ltol[full]), float((off / ltol[full]).max())
        assert self.ws.sync_status() == self.mr.MR_OK


# rows held of each sequence, H_q, H_kv, page_rows, d
DECODES = [
    ([1], 1, 1, 16, 64), ([0], 2, 1, 16, 128), ([5, 0, 17, 64, 65, 0], 4, 2, 16, 64), ([130, 1], 7, 1, 7, 128),
    ([63, 64, 65, 200], 28, 4, 64, 128), ([300], 40, 2, 32, 128), ([90, 33], 34, 2, 128, 64), ([2000], 1, 1, 16, 128),
    ([1, 700, 2], 64, 8, 128, 128), ([257], 33, 1, 1, 64), ([15] * 40, 5, 5, 16, 64), ([-3, 20], 8, 1, 16, 64),
]


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("case", range(len(DECODES)))
def test_decode_against_64_bits(mr, dt, case):
    held, Hq, Hk, pr, d = DECODES[case]
    c = Case(mr, [1] * len(held), held, Hq, Hk, pr, d, dt, seed=case)
    O, lse = mr.paged_decode(*c.args(), return_lse=True, ws=c.ws)
    c.check(O, lse, p_eps=DECODE_P[dt])
    again, lse2 = mr.paged_decode(*c.args(), return_lse=True, ws=c.ws)
    assert torch.equal(O, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 3), (40, 0), (64, 16), (100, 200), (5000, 16), (0, 16), (17, 1000)])
def test_decode_window_and_sinks(mr, dt, window, sinks):
    c = Case(mr, [1] * 4, [300, 1, 18, 129], 8, 2, 16, 64, dt, seed=3)
    c.hide(window, sinks)
    O, lse = mr.paged_decode(*c.args(), window=window, sinks=sinks, return_lse=True, ws=c.ws)
    c.check(O, lse, window=window, sinks=sinks, p_eps=DECODE_P[dt])


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("scale,spread", [(0.0, 1.0), (-0.3, 1.0), (2.0, 8.0)])
def test_decode_scales(mr, dt, scale, spread):
    c = Case(mr, [1, 1], [500, 77], 6, 2, 32, 128, dt, seed=4, spread=spread)
    O, lse = mr.paged_decode(*c.args(), scale=scale, return_lse=True, ws=c.ws)
    c.check(O, lse, scale=scale, p_eps=DECODE_P[dt])


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_decode_long_and_ragged(mr, dt):
    """Units that begin and end inside a CTA's share, and units that many CTAs share."""
    held = [9000, 1, 64, 0, 4097, 130, 12345, 5]
    c = Case(mr, [1] * len(held), held, 8, 4, 64, 128, dt, seed=5)
    O, lse = mr.paged_decode(*c.args(), return_lse=True, ws=c.ws)
    c.check(O, lse, p_eps=DECODE_P[dt])


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_decode_strides_and_alignment(mr, dt):
    c = Case(mr, [1] * 3, [50, 3, 120], 6, 2, 16, 64, dt, seed=6)
    cache, table, lens, q = c.args()
    want, wl = mr.paged_decode(cache, table, lens, q, return_lse=True)
    buf = torch.full((3 * 6 * 67 + 1,), 5.0, dtype=q.dtype, device="cuda")
    out = buf[1:].view(3, 6, 67).transpose(0, 1)[..., :64]      # [rows][heads][67] storage, odd offset
    qv = torch.empty_like(buf)[1:].view(3, 6, 67).transpose(0, 1)[..., :64]
    qv.copy_(q)
    mr.paged_decode(cache, table, lens, qv, out=out, ws=c.ws)
    assert torch.equal(out, want)
    assert bool((buf[1:].view(3, 6, 67)[..., 64:] == 5.0).all()) and float(buf[0]) == 5.0
    one = q[:1].expand(6, 3, 64)                                 # one query row for every head
    a = mr.paged_decode(cache, table, lens, one)
    assert torch.equal(a, mr.paged_decode(cache, table, lens, one.contiguous()))


def test_decode_infinite_and_nan_values_that_are_seen(mr):
    """What a visible row holds does reach the result, as in the formula, and only its sequence's."""
    c = Case(mr, [1, 1], [40, 40], 2, 1, 16, 64, "f32", seed=7)
    cache, table, lens, q = c.args()
    want = mr.paged_decode(cache, table, lens, q)
    c.v[c.table[0, 1], 0, 3, 5] = math.nan
    got = mr.paged_decode(cache, table, lens, q)
    assert bool(torch.isnan(got[:, 0, 5]).all())
    got[:, 0, 5] = want[:, 0, 5]
    assert torch.equal(got, want)


def test_decode_reports_bad_pages_and_short_tables(mr):
    c = Case(mr, [1, 1], [40, 20], 2, 1, 16, 64, "bf16", seed=8)
    cache, table, lens, q = c.args()
    want = mr.paged_decode(cache, table, lens, q, ws=c.ws)
    for bad in (-1, 10 ** 6):
        t = table.clone()
        t[0, 1] = bad
        got = mr.paged_decode(cache, t, lens, q, ws=c.ws)
        assert c.ws.sync_status() == mr.MR_ERR_DEVICE_CHECK
        assert torch.equal(got[:, 1], want[:, 1]) and bool(torch.isfinite(got).all())
    t = table.clone()
    t[:, 3:] = 10 ** 6                                           # behind the last row: not used
    assert torch.equal(mr.paged_decode(cache, t, lens, q, ws=c.ws), want) and c.ws.sync_status() == mr.MR_OK
    short = table[:, :2].contiguous()
    mr.paged_decode(cache, short, lens, q, ws=c.ws)
    assert c.ws.sync_status() == mr.MR_ERR_DEVICE_CHECK


def test_decode_on_a_stream_and_in_a_graph(mr):
    c = Case(mr, [1] * 3, [50, 3, 900], 8, 2, 16, 128, "bf16", seed=9)
    cache, table, lens, q = c.args()
    want, wl = mr.paged_decode(cache, table, lens, q, return_lse=True, ws=c.ws)
    out, lse = torch.zeros_like(want), torch.zeros_like(wl)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        mr.paged_decode(cache, table, lens, q, out=out, lse=lse, ws=c.ws)
    st.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, wl)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mr.paged_decode(cache, table, lens, q, out=out, lse=lse, ws=c.ws)
    for n in (50, 20, 1):
        lens[0] = n
        out.zero_()
        g.replay()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, mr.paged_decode(cache, table, lens, q))


# ---------------------------------------------------------------------------------------------- chunks of new rows
# new rows and rows held of each sequence, H_q, H_kv, page_rows, d
CHUNKS = [
    ([1], [1], 1, 1, 16, 64), ([3, 0, 5], [3, 9, 200], 4, 2, 16, 128), ([70, 1, 200], [70, 333, 230], 8, 2, 64, 128),
    ([33], [300], 7, 1, 7, 64), ([130, 129], [130, 700], 5, 5, 32, 64), ([257], [400], 28, 4, 128, 128),
    ([20, 20], [15, 20], 2, 1, 16, 64), ([5, 3], [0, -4], 2, 2, 16, 128), ([100], [1000], 40, 1, 48, 128),
    ([2], [3000], 3, 1, 16, 64), ([1, 1, 1], [513, 1, 64], 66, 2, 8, 64), ([300], [300], 1, 1, 1, 128),
    ([384], [512], 1, 1, 128, 128), ([9] * 20, [40 + i for i in range(20)], 8, 4, 16, 64),
]


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("case", range(len(CHUNKS)))
def test_attn_against_64_bits(mr, dt, case):
    new, held, Hq, Hk, pr, d = CHUNKS[case]
    c = Case(mr, new, held, Hq, Hk, pr, d, dt, seed=case, behind=3)
    cache, table, lens, q = c.args()
    O = torch.full_like(q, 5.0)
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    mr.paged_attn(cache, table, lens, q, c.cu, out=O, lse=lse, ws=c.ws)
    c.check(O, lse, p_eps=ATTN_P[dt])
    assert bool((O[:, c.T:] == 5.0).all()) and bool((lse[:, c.T:] == 7.0).all())
    again, lse2 = mr.paged_attn(cache, table, lens, q, c.cu, return_lse=True, ws=c.ws)
    assert torch.equal(O[:, : c.T], again[:, : c.T]) and torch.equal(lse[:, : c.T], lse2[:, : c.T])


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("pr", [16, 12])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 3), (40, 0), (64, 16), (100, 200), (5000, 16), (0, 16), (130, 129),
                                          (17, 1000), (2 ** 31 - 1, 2 ** 31 - 1)])
def test_attn_window_and_sinks(mr, dt, pr, window, sinks):
    c = Case(mr, [300, 1, 18, 150], [300, 400, 700, 129], 8, 2, pr, 64, dt, seed=3)
    c.hide(window, sinks)
    O, lse = mr.paged_attn(*c.args(), c.cu, window=window, sinks=sinks, return_lse=True, ws=c.ws)
    c.check(O, lse, window=window, sinks=sinks, p_eps=ATTN_P[dt])


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("scale,spread", [(0.0, 1.0), (-0.3, 1.0), (2.0, 8.0)])
def test_attn_scales(mr, dt, d, scale, spread):
    c = Case(mr, [70, 90], [500, 90], 6, 2, 32, d, dt, seed=4, spread=spread)
    O, lse = mr.paged_attn(*c.args(), c.cu, scale=scale, return_lse=True, ws=c.ws)
    c.check(O, lse, scale=scale, p_eps=ATTN_P[dt])


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_attn_growing_logits(mr, dt):
    """Scores that keep passing the running maximum, so that what was summed has to be scaled again and again."""
    c = Case(mr, [40], [900], 2, 1, 16, 128, dt, seed=5)
    ramp = (torch.arange(900, dtype=torch.float32) / 60).to(DT[dt]).cuda()
    c.q[:, :, 0] = 4.0
    for j in range(900):
        c.k[c.table[0, j // 16], 0, j % 16, 0] = ramp[j]
        c.clean_k[int(c.table[0, j // 16]), 0, j % 16, 0] = float(ramp[j])
    O, lse = mr.paged_attn(*c.args(), c.cu, scale=2.0, return_lse=True, ws=c.ws)
    c.check(O, lse, scale=2.0, p_eps=ATTN_P[dt])


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
def test_attn_many_units_and_parts(mr, dt, d):
    c = Case(mr, [700, 1, 90, 0, 350], [700, 2500, 1400, 30, 3600], 4, 2, 64, d, dt, seed=6)
    O, lse = mr.paged_attn(*c.args(), c.cu, window=1000, sinks=20, return_lse=True, ws=c.ws)
    c.check(O, lse, window=1000, sinks=20, p_eps=ATTN_P[dt])


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("most", [2, 5])
def test_attn_many_sequences(mr, dt, most):
    """More runs of new rows than a CTA has threads, some without rows, some that hold nothing (most 2: fewer rows than
    sequences)."""
    rng = np.random.default_rng(2)
    new = rng.integers(0, most, 1300)
    held = np.maximum(new + rng.integers(-1, 40, 1300), 0)
    new[:5], held[700:705] = 0, 0
    c = Case(mr, new.tolist(), held.tolist(), 2, 1, 16, 64, dt, seed=16)
    O, lse = mr.paged_attn(*c.args(), c.cu, window=20, sinks=2, return_lse=True, ws=c.ws)
    c.check(O, lse, window=20, sinks=2, p_eps=ATTN_P[dt])


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("new,held,p", [([7], [7], DECODE_P), ([4, 0, 3], [2, 5, 600], DECODE_P),
                                        # 41 rows (one behind the last) of 40 sequences: worked on in tiles, P is one part
                                        ([1] * 40, list(range(40)), ATTN_P),
                                        ([1] * 40 + [0], list(range(40)) + [3], DECODE_P), ([8], [5000], DECODE_P)])
def test_attn_of_few_rows(mr, dt, new, held, p):
    """Rows that are worked on one by one, each with its own end and window."""
    c = Case(mr, new, held, 12, 3, 16, 128, dt, seed=19, behind=1)
    for window, sinks in ((0, 0), (5, 0), (30, 7)):
        O, lse = mr.paged_attn(*c.args(), c.cu, window=window, sinks=sinks, return_lse=True, ws=c.ws)
        c.check(O, lse, window=window, sinks=sinks, p_eps=p[dt])


def test_two_calls_at_once(mr):
    """Two streams, a workspace each."""
    a = Case(mr, [200, 1500], [700, 1500], 8, 2, 16, 128, "bf16", seed=17)
    b = Case(mr, [1] * 6, [9000, 1, 300, 4000, 64, 20], 8, 2, 64, 128, "bf16", seed=18)
    x, y = a.args(), b.args()
    wa, wb = mr.paged_attn(*x, a.cu, window=400, ws=a.ws), mr.paged_decode(*y, ws=b.ws)
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for _ in range(8):
        got.append((mr.paged_attn(*x, a.cu, window=400, ws=a.ws, stream=s), mr.paged_decode(*y, ws=b.ws, stream=t)))
    torch.cuda.synchronize()
    assert all(torch.equal(g, wa) and torch.equal(h, wb) for g, h in got)
    assert a.ws.sync_status() == mr.MR_OK and b.ws.sync_status() == mr.MR_OK


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("what", ["k", "v"])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_attn_rows_that_only_some_see(mr, dt, what, bad):
    """A value that is not finite, in a row that is the future of some new rows and outside the window of others, reaches
    the rows that see it and no other."""
    c = Case(mr, [200, 60], [260, 60], 4, 2, 16, 128, dt, seed=7)
    cache, table, lens, q = c.args()
    want, wl = mr.paged_attn(cache, table, lens, q, c.cu, window=64, sinks=4, return_lse=True)
    row = 130                                              # new rows 70 .. 133 of sequence 0 see it
    getattr(c, what)[c.table[0, row // 16], 1, row % 16, 11] = bad
    got, gl = mr.paged_attn(cache, table, lens, q, c.cu, window=64, sinks=4, return_lse=True, ws=c.ws)
    seen = torch.zeros(4, 260, dtype=torch.bool, device="cuda")
    seen[2:, 70: 134] = True
    # rows that are computed another way once such a value is found may differ by roundings: half a step of the
    # probabilities and of the output each
    tol = (torch.finfo(DT[dt]).eps + 2.0 ** -18) * c.v.float().nan_to_num(0, 0, 0).abs().max()
    assert bool(((got - want)[~seen].abs() <= tol).all())
    assert bool(((gl - wl)[~seen].abs() <= 1e-5).all())
    if what == "v":
        assert bool(((gl - wl).abs() <= 1e-5).all())
        rest = torch.ones(128, dtype=torch.bool)
        rest[11] = False
        assert bool(((got - want)[seen][:, rest].abs() <= tol).all())
        assert bool((~torch.isfinite(got[seen][:, 11])).all())
    elif math.isnan(bad):
        assert bool(torch.isnan(got[seen]).all()) and bool(torch.isnan(gl[seen]).all())
    else:                                                  # scores of +inf (NaN) and -inf (nothing: like hidden)
        up = seen & (q[:, :, 11] > 0)
        assert bool(torch.isnan(got[up]).all()) and bool(torch.isfinite(got[seen & (q[:, :, 11] < 0)]).all())


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("scale", [0.2, -0.2])
def test_attn_values_that_only_some_see_in_split_units(mr, dt, scale):
    """The same where many CTAs share a unit, with either sign of the scale: what is finite stays right, rows that see the
    infinite value get it (its own weight's sign), the others do not."""
    c = Case(mr, [64], [5000], 2, 1, 16, 128, dt, seed=15)
    cache, table, lens, q = c.args()
    want, wl = mr.paged_attn(cache, table, lens, q, c.cu, scale=scale, return_lse=True, ws=c.ws)
    c.check(want, wl, scale=scale, p_eps=ATTN_P[dt])
    for row, col in ((4990, 3), (4950, 127), (4999, 64)):
        c.v[c.table[0, row // 16], 0, row % 16, col] = math.inf
    got, gl = mr.paged_attn(cache, table, lens, q, c.cu, scale=scale, return_lse=True, ws=c.ws)
    assert torch.equal(gl, wl)
    for row, col in ((4990, 3), (4950, 127), (4999, 64)):
        i = row - 4936                                     # the first new row that sees it
        assert bool((got[:, i:, col] == math.inf).all()) and bool(torch.isfinite(got[:, :i, col]).all())
        got[:, i:, col] = want[:, i:, col]
    assert torch.equal(got, want)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_attn_strides_and_alignment(mr, dt):
    c = Case(mr, [40, 3], [50, 120], 6, 2, 16, 64, dt, seed=8)
    cache, table, lens, q = c.args()
    want, _, A, S = attend(np64(q), c.clean_k, c.clean_v, c.table.numpy(), c.lens.numpy(), c.new, 0.125)
    tol = attend_tol(want, _, A, S, 64, 120, torch.finfo(DT[dt]).eps, ATTN_P[dt])[0]
    for width, off in ((64, 0), (72, 8), (67, 1)):               # [rows][heads][width] storage
        buf = torch.full((43 * 6 * width + off,), 5.0, dtype=q.dtype, device="cuda")
        out = buf[off:].view(43, 6, width).transpose(0, 1)[..., :64]
        qv = torch.empty_like(buf)[off:].view(43, 6, width).transpose(0, 1)[..., :64]
        qv.copy_(q)
        mr.paged_attn(cache, table, lens, qv, c.cu, out=out, ws=c.ws)
        assert np.all(np.abs(np64(out) - want) <= tol)
        assert bool((buf[off:].view(43, 6, width)[..., 64:] == 5.0).all()) and bool((buf[:off] == 5.0).all())
    one = q[:1].expand(6, 43, 64)                                 # one head's queries for all of them
    got = mr.paged_attn(cache, table, lens, one, c.cu)
    ref = mr.paged_attn(cache, table, lens, one.contiguous(), c.cu)
    assert np.all(np.abs(np64(got) - np64(ref)) <= 2 * tol.max())


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_attn_of_one_row_is_decode(mr, dt):
    c = Case(mr, [1] * 4, [300, 1, 64, 129], 8, 2, 16, 128, dt, seed=9)
    O, lse = mr.paged_attn(*c.args(), c.cu, window=100, sinks=5, return_lse=True, ws=c.ws)
    P, lse2 = mr.paged_decode(*c.args(), window=100, sinks=5, return_lse=True, ws=c.ws)
    c.check(O, lse, window=100, sinks=5, p_eps=ATTN_P[dt])
    c.check(P, lse2, window=100, sinks=5, p_eps=DECODE_P[dt])


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_attn_reports_bad_pages_and_short_tables(mr, dt):
    c = Case(mr, [30, 20], [40, 20], 2, 1, 16, 64, dt, seed=10)
    cache, table, lens, q = c.args()
    want = mr.paged_attn(cache, table, lens, q, c.cu, ws=c.ws)
    for bad in (-1, 10 ** 6):
        t = table.clone()
        t[0, 1] = bad
        got = mr.paged_attn(cache, t, lens, q, c.cu, ws=c.ws)
        assert c.ws.sync_status() == mr.MR_ERR_DEVICE_CHECK
        assert torch.equal(got[:, 30:], want[:, 30:]) and bool(torch.isfinite(got).all())
    t = table.clone()
    t[0, 3:] = 10 ** 6
    t[1, 2:] = -7
    assert torch.equal(mr.paged_attn(cache, t, lens, q, c.cu, ws=c.ws), want) and c.ws.sync_status() == mr.MR_OK
    mr.paged_attn(cache, table[:, :2].contiguous(), lens, q, c.cu, ws=c.ws)
    assert c.ws.sync_status() == mr.MR_ERR_DEVICE_CHECK


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_attn_no_rows(mr, dt):
    c = Case(mr, [0, 0], [40, 20], 2, 1, 16, 64, dt, seed=11, behind=2)
    cache, table, lens, q = c.args()
    out = torch.full_like(q, 5.0)
    mr.paged_attn(cache, table, lens, q, c.cu, out=out, ws=c.ws)
    assert bool((out == 5.0).all()) and c.ws.sync_status() == mr.MR_OK
    assert mr.paged_attn(cache, table, lens, q[:, :0], c.cu).shape == (2, 0, 64)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_attn_on_a_stream_and_in_a_graph(mr, dt):
    c = Case(mr, [50, 3, 200], [50, 80, 900], 8, 2, 16, 128, dt, seed=12)
    cache, table, lens, q = c.args()
    want, wl = mr.paged_attn(cache, table, lens, q, c.cu, return_lse=True, ws=c.ws)
    out, lse = torch.zeros_like(want), torch.zeros_like(wl)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        mr.paged_attn(cache, table, lens, q, c.cu, out=out, lse=lse, ws=c.ws)
    st.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, wl)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mr.paged_attn(cache, table, lens, q, c.cu, out=out, lse=lse, ws=c.ws)
    for n in (900, 500, 210):
        lens[2] = n
        out.zero_()
        g.replay()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, mr.paged_attn(cache, table, lens, q, c.cu))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_rows_that_see_one_key_give_its_value(mr, dt):
    """softmax of one score is 1: nothing is left to round."""
    c = Case(mr, [90, 1], [130, 1], 8, 2, 16, 128, dt, seed=14)
    cache, table, lens, q = c.args()
    O, lse = mr.paged_attn(cache, table, lens, q, c.cu, window=1, return_lse=True, ws=c.ws)
    pos = np.concatenate([np.arange(40, 130), [0]])
    seq = np.array([0] * 90 + [1])
    v = c.v[c.table[seq, pos // 16].long(), :, pos % 16].transpose(0, 1).repeat_interleave(4, 0)
    assert torch.equal(O, v)
    one = mr.paged_decode(cache, table, lens, q[:, :2].contiguous(), window=1, ws=c.ws)
    assert torch.equal(one, v[:, [89, 90]])


# ---------------------------------------------------------------------------------------------- pools beyond 2^32 bytes
def test_pages_far_into_a_large_pool(mr):
    """Rows whose byte offsets pass 32 bits (a pool of 5.2 GB for keys and one for values): appended, read and copied."""
    n_pages, pr, d = 160000, 128, 128
    cache = mr.KVCache.empty(n_pages, 1, pr, d)
    table = torch.tensor([[n_pages - 1, 5, n_pages - 3], [131073, n_pages - 7, 131072]], dtype=torch.int32).cuda()
    lens = torch.tensor([300, 257], dtype=torch.int32).cuda()
    cu = torch.tensor([0, 300, 557], dtype=torch.int32).cuda()
    q, k, v = rand((4, 557, d), "bf16", 1), rand((1, 557, d), "bf16", 2), rand((1, 557, d), "bf16", 3)
    ws = mr.Workspace(mr.paged_workspace_bytes(cache, 4, 2))
    mr.kv_append(cache, table, lens, k, v, cu_q=cu, ws=ws)
    assert ws.sync_status() == mr.MR_OK
    small = mr.KVCache.empty(6, 1, pr, d)
    near = torch.arange(6, dtype=torch.int32).view(2, 3).cuda()
    mr.kv_append(small, near, lens, k, v, cu_q=cu, ws=ws)
    assert torch.equal(cache.k[table.view(-1)[:2].long()], small.k[:2])
    want = mr.paged_attn(small, near, lens, q, cu, ws=ws)
    assert torch.equal(mr.paged_attn(cache, table, lens, q, cu, ws=ws), want) and ws.sync_status() == mr.MR_OK
    one = q[:, [299, 556]].contiguous()
    assert torch.equal(mr.paged_decode(cache, table, lens, one), mr.paged_decode(small, near, lens, one))
    mr.pages_copy([cache.k, cache.v], torch.tensor([[n_pages - 1, 140000]], dtype=torch.int32).cuda(), ws=ws)
    assert torch.equal(cache.v[140000], small.v[0]) and ws.sync_status() == mr.MR_OK


# ---------------------------------------------------------------------------------------------- streams that are given
@pytest.mark.parametrize("handle", [False, True])
def test_a_given_stream_without_a_workspace(mr, handle):
    """Outputs and workspaces made inside a call belong to its stream: nothing on the current one can reuse them while
    the call runs."""
    c = Case(mr, [50, 3, 200], [50, 80, 900], 8, 2, 16, 128, "bf16", seed=13)
    cache, table, lens, q = c.args()
    want = mr.paged_attn(cache, table, lens, q, c.cu)
    one = mr.paged_decode(cache, table, lens, q[:, :3].contiguous())
    r = mr.Rope(128)
    pos = torch.arange(c.T, dtype=torch.int32, device="cuda")
    turned = mr.rope(r, q, pos)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    arg = st.cuda_stream if handle else st
    torch.cuda.synchronize()
    got = [mr.paged_attn(cache, table, lens, q, c.cu, stream=arg), mr.paged_decode(cache, table, lens, q[:, :3], stream=arg),
           mr.rope(r, q, pos, stream=arg)]
    junk = [torch.full((1 << 22,), math.nan, device="cuda") for _ in range(8)]
    st.synchronize()
    for g, w in zip(got, (want, one, turned)):
        assert torch.equal(g, w)
    del junk
    assert torch.cuda.current_stream() == torch.cuda.default_stream()
    assert torch.equal(mr.rope(r, q, pos, stream=0), turned)
