"""A receiver's requests from end to end: a reused prefix, suffixes computed exactly, decoding token by token, forks that
share pages, a sliding window that frees them, and a pool that is compacted while requests are under way."""
import math
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from cross_model_attention_mr_b200.workloads import config, draw_layers, shrink

from paged_ref import attend, attend_tol, inv_freq, rotate, rotate_tol
from parity import dev, p32

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
EPS = torch.finfo(torch.bfloat16).eps


@pytest.fixture(scope="module")
def mr():
    from cross_model_attention_mr_b200 import mr as m
    assert torch.cuda.is_available()
    return m


def np64(t):
    return t.detach().cpu().double().numpy()


class Server:
    """One layer of a receiver: its cache, its pages, and the projections of new tokens drawn at random."""

    def __init__(self, mr, n_pages, pr, Hq, Hk, d, seed):
        self.mr, self.Hq, self.Hk, self.d, self.pr = mr, Hq, Hk, d, pr
        self.cache = mr.KVCache.empty(n_pages, Hk, pr, d)
        self.cache.k.fill_(math.nan)                       # pages that nothing was written to
        self.cache.v.fill_(math.nan)
        self.pool = mr.PagePool(n_pages, pr)
        self.rope = mr.Rope(d)
        self.ws = mr.Workspace(mr.paged_workspace_bytes(self.cache, Hq, 8))
        self.gen = torch.Generator(device="cpu").manual_seed(seed)
        self.told = {}                                     # sequence -> its rows' (rotated K, V), in 64 bits

    def draw(self, heads, n):
        return torch.randn((heads, n, self.d), generator=self.gen).bfloat16().cuda()

    def copy(self, pairs):
        if len(pairs):
            p = torch.tensor(np.asarray(pairs, np.int32).reshape(-1, 2)).cuda()
            self.mr.pages_copy([self.cache.k, self.cache.v], p, ws=self.ws)
            assert self.ws.sync_status() == self.mr.MR_OK

    def tables(self, seqs):
        t, n = self.pool.tables(seqs)
        return torch.from_numpy(np.maximum(t, 0)).cuda(), torch.from_numpy(n).cuda()

    def append(self, seqs, new, V=None):
        """New rows of each sequence; returns their rotated queries."""
        for s, n in zip(seqs, new):
            self.copy(self.pool.extend(s, n))
        T = sum(new)
        q, k = self.draw(self.Hq, T), self.draw(self.Hk, T)
        v = self.draw(self.Hk, T) if V is None else V
        table, lens = self.tables(seqs)
        cu = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32).cuda()
        one = all(n == 1 for n in new)
        qr = self.mr.kv_append(self.cache, table, lens, k, v, cu_q=None if one else cu, rope=self.rope, Q=q, ws=self.ws)
        assert self.ws.sync_status() == self.mr.MR_OK
        t = 0
        for s, n, h in zip(seqs, new, lens.tolist()):
            pos = np.arange(h - n, h)
            want = rotate(np64(k)[:, t: t + n], pos, inv_freq(self.d))
            tol = rotate_tol(np64(k)[:, t: t + n], want, self.d, EPS)
            pages, rows = table[list(seqs).index(s)].cpu().numpy()[pos // self.pr], pos % self.pr
            held = np64(self.cache.k)[pages, :, rows].transpose(1, 0, 2)
            assert np.all(np.abs(held - want) <= tol)
            old = self.told.get(s, (np.zeros((self.Hk, 0, self.d)),) * 2)
            self.told[s] = (np.concatenate([old[0], held], 1), np.concatenate([old[1], np64(v)[:, t: t + n]], 1))
            t += n
        return qr, table, lens, cu

    def check(self, O, lse, q, seqs, new, window=0, sinks=0, p_eps=0.0):
        """Against what the sequences were told, laid out plainly, one page each."""
        held = [self.told[s][0].shape[1] for s in seqs]
        most = max(held)
        k, v = (np.zeros((len(seqs), self.Hk, most, self.d)) for _ in range(2))
        for i, s in enumerate(seqs):
            k[i, :, : held[i]], v[i, :, : held[i]] = self.told[s]
        scale = float(np.float32(1 / math.sqrt(self.d)))
        want, wl, A, S = attend(np64(q), k, v, np.arange(len(seqs))[:, None], held, new, scale, window, sinks)
        tol, ltol = attend_tol(want, wl, A, S, self.d, most, EPS, p_eps)
        assert np.all(np.abs(np64(O) - want) <= tol)
        assert np.all(np.abs(np64(lse) - wl) <= ltol)
        assert self.ws.sync_status() == self.mr.MR_OK

    def decode(self, seqs, window=0, sinks=0):
        q, table, lens, _ = self.append(seqs, [1] * len(seqs))
        O, lse = self.mr.paged_decode(self.cache, table, lens, q, window=window, sinks=sinks, return_lse=True, ws=self.ws)
        self.check(O, lse, q, seqs, [1] * len(seqs), window, sinks, 2.0 ** -16)
        return q, O


def test_reuse_suffix_decode_fork_and_compact(mr):
    spec = shrink(config(5), L=512, H_s=4, H_r=4)
    lay = draw_layers(spec)[0]
    m = mr.compress(dev(lay.Q, "bf16"), dev(lay.K, "bf16"), p32(spec.p), spec.block, bias=mr.Bias.from_spec(lay.bias),
                    scale=spec.scale)
    W = torch.from_numpy(lay.W).cuda()
    s = Server(mr, 40, 64, 4, 2, 128, seed=1)
    # the prefix: keys and values in the cache, outputs from the sender's maps, read straight from the cache's pages
    a = s.pool.open()
    V = s.draw(2, spec.L)
    _, table, _, _ = s.append([a], [spec.L], V=V)
    got = mr.retrieve(m, W, s.cache.v, v_group=2, v_pages=table, page_rows=64, n_req=1)
    want = mr.retrieve(m, W, V.contiguous(), v_group=2)
    assert torch.equal(got, want)
    # two requests behind it; their suffixes are computed exactly
    b = s.pool.fork(a, spec.L)
    s.told[b] = s.told[a]
    assert s.pool.stats()["shared"] == 8
    new = [70, 41]
    q, table, lens, cu = s.append([a, b], new)
    O, lse = mr.paged_attn(s.cache, table, lens, q, cu, return_lse=True, ws=s.ws)
    s.check(O, lse, q, [a, b], new, p_eps=2.0 ** -8)
    # decoding; a third request forks off in the middle of a page
    for _ in range(3):
        s.decode([a, b])
    c = s.pool.fork(b, 540)
    s.told[c] = tuple(x[:, :540] for x in s.told[b])
    for _ in range(3):
        s.decode([c, a, b])
    # one ends, the pages in use move to the front, the others go on as if nothing had happened
    s.pool.close(a)
    table, lens = s.tables([c, b])
    q = s.draw(4, 2)
    before = mr.paged_decode(s.cache, table, lens, q)
    used = s.pool.stats()["pages"] - s.pool.stats()["free"]
    s.copy(s.pool.compact())
    table, lens = s.tables([c, b])
    assert int(table.max()) < used
    assert torch.equal(mr.paged_decode(s.cache, table, lens, q), before)
    s.decode([b, c])


def test_sliding_window_frees_pages_while_decoding(mr):
    """A pool too small for what the request has seen: pages that leave the window are handed out again."""
    s = Server(mr, 12, 16, 8, 2, 64, seed=2)
    a = s.pool.open()
    window, sinks = 60, 20
    q, table, lens, cu = s.append([a], [150])
    O, lse = mr.paged_attn(s.cache, table, lens, q, cu, window=window, sinks=sinks, return_lse=True, ws=s.ws)
    s.check(O, lse, q, [a], [150], window, sinks, 2.0 ** -8)
    freed = 0
    for _ in range(100):
        freed += s.pool.slide(a, window, sinks)
        s.decode([a], window, sinks)
    assert freed >= 7 and s.pool.rows(a) == 250


def test_a_decoding_step_as_one_graph(mr):
    """Append and decode captured once and replayed with new lengths and projections."""
    s = Server(mr, 24, 16, 4, 2, 128, seed=3)
    seqs = [s.pool.open() for _ in range(3)]
    s.append(seqs, [20, 5, 33])
    for q in seqs:
        s.pool.extend(q, 8)                                # room for the steps ahead
    table, _ = s.tables(seqs)
    lens = torch.tensor([20, 5, 33], dtype=torch.int32).cuda()
    q, k, v = (torch.zeros((h, 3, 128), dtype=torch.bfloat16, device="cuda") for h in (4, 2, 2))
    out, qr, lse = torch.empty_like(q), torch.empty_like(q), torch.empty((4, 3), device="cuda")

    def step():
        lens.add_(1)
        mr.kv_append(s.cache, table, lens, k, v, rope=s.rope, Q=q, q_out=qr, ws=s.ws)
        mr.paged_decode(s.cache, table, lens, qr, out=out, lse=lse, ws=s.ws)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        step()                                             # warm-up
    st.synchronize()
    lens.sub_(1)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for _ in range(6):
        for x in (q, k, v):
            x.copy_(s.draw(x.shape[0], 3))
        g.replay()
        torch.cuda.synchronize()
        for i, sq in enumerate(seqs):
            h = int(lens[i])
            page, row = int(table[i, (h - 1) // 16]), (h - 1) % 16
            k1, v1 = np64(s.cache.k)[page, :, row], np64(s.cache.v)[page, :, row]
            assert np.array_equal(v1, np64(v)[:, i])
            s.told[sq] = tuple(np.concatenate([o, n[:, None]], 1) for o, n in zip(s.told[sq], (k1, v1)))
        s.check(out, lse, qr, seqs, [1] * 3, p_eps=2.0 ** -16)


def test_attn_wait_runs_out_then_next_call_is_clean(mr):
    """With the test hook the first tile's softmax keeps its first P back: the MMA warp's wait runs out after 1 ms, the
    call records it, drains and returns, and the next call on the same workspace is right."""
    s = Server(mr, 24, 64, 2, 1, 128, seed=4)
    a = s.pool.open()
    q, table, lens, cu = s.append([a], [200])
    want, wl = mr.paged_attn(s.cache, table, lens, q, cu, return_lse=True, ws=s.ws)
    s.check(want, wl, q, [a], [200], p_eps=2.0 ** -8)
    assert mr.LIB.mr_debug_set(1_000_000, 1) == mr.MR_OK
    try:
        mr.paged_attn(s.cache, table, lens, q, cu, ws=s.ws)
        st = s.ws.sync_status()
        off = s.ws.ptr - s.ws.buf.data_ptr()
        detail = int(s.ws.buf[off + 4: off + 8].view(torch.int32).item())
    finally:
        assert mr.LIB.mr_debug_set(0, 0) == mr.MR_OK
    assert st == mr.MR_ERR_TIMEOUT and detail == 0xA16
    O, lse = mr.paged_attn(s.cache, table, lens, q, cu, return_lse=True, ws=s.ws)
    assert s.ws.sync_status() == mr.MR_OK and torch.equal(O, want) and torch.equal(lse, wl)


def test_attention_under_the_checked_build():
    if os.environ.get("MR_LIBRARY") == "checked":
        pytest.skip("already the bounds-checked build")
    env = dict(os.environ, MR_LIBRARY="checked")
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-p", "no:cacheprovider", "tests/test_gpu_paged_attn.py",
                        "-k", "(attn_against or attn_window or rows_that_only or many_units or strides) and bf16"],
                       cwd=ROOT, env=env, capture_output=True, text=True, timeout=900)
    tail = "\n".join((r.stdout + r.stderr).splitlines()[-25:])
    assert r.returncode == 0, tail
    assert " passed" in r.stdout and "failed" not in r.stdout, tail
