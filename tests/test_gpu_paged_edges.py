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
