"""Attention of new rows over the paged cache on the GPU, against a 64-bit plain form."""
import math

import numpy as np
import pytest
import torch

from paged_ref import attend, attend_tol

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
# half a step of the probabilities in the second product: two bf16 parts (2^-9 of 2^-9), or fp32
DECODE_P = {"bf16": 2.0 ** -17, "f32": 0.0}


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
