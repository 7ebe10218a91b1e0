"""The paged cache's host side, without a GPU: the rotation's frequencies, the refusals of every entry point
(nothing is launched by a refused call), and the page pool against a plain model of it."""
import ctypes
import random

import numpy as np
import pytest

from paged_ref import inv_freq


@pytest.fixture(scope="module")
def mr():
    from cross_model_attention_mr_b200 import mr as m
    return m


# ------------------------------------------------------------------------------------------------ rope table
@pytest.mark.parametrize("rot", [2, 16, 64, 128, 250])
@pytest.mark.parametrize("scaling,factor", [("none", 1.0), ("linear", 4.0), ("base", 8.0), ("ramp", 4.0)])
def test_frequencies_are_exact_fractions_of_a_turn(mr, rot, scaling, factor):
    if scaling == "base" and rot < 4:
        pytest.skip("rot_dim - 2 divides")
    r = mr.Rope(256, rot_dim=rot, scaling=scaling, factor=factor, orig_len=4096)
    f = inv_freq(rot, scaling=scaling, factor=factor)
    turns = f / (2 * np.longdouble(np.pi) + np.longdouble(2.4492935982947064e-16))
    got = np.array([r.c.turn[i] for i in range(rot // 2)], dtype=np.uint64).astype(np.longdouble) / np.longdouble(2) ** 64
    # both sides are in 64-bit-mantissa arithmetic; pow loses a few units in the last place, more for the
    # long exponents of "base" (|log2 b| * rot): 2^-58 relative
    assert np.all(np.abs(got - turns) <= turns * 2.0 ** -58 + 2.0 ** -64)
    assert all(r.c.turn[i] == 0 for i in range(rot // 2, 128))


def test_given_frequencies_and_their_sign(mr):
    r = mr.Rope(64, rot_dim=8, inv_freq=[1.0, -1.0, 0.0, 0.25])
    assert (r.c.turn[0] + r.c.turn[1]) % 2 ** 64 == 0 and r.c.turn[2] == 0
    assert abs(r.c.turn[3] * 4 - r.c.turn[0]) <= 4


@pytest.mark.parametrize("kw", [dict(d=0), dict(d=60), dict(d=264), dict(d=64, rot_dim=0), dict(d=64, rot_dim=66),
                                dict(d=64, rot_dim=7), dict(d=64, base=1.0), dict(d=64, base=float("nan")),
                                dict(d=64, factor=2.0), dict(d=64, scaling="linear", factor=0.0),
                                dict(d=64, rot_dim=2, scaling="base", factor=2.0),
                                dict(d=64, scaling="ramp", factor=2.0, orig_len=0),
                                dict(d=64, scaling="ramp", factor=2.0, orig_len=10, beta_slow=3.0, beta_fast=3.0),
                                dict(d=64, mscale=float("inf")), dict(d=64, mscale=1e300),
                                dict(d=64, rot_dim=4, inv_freq=[1.0, 6.3]),
                                dict(d=64, rot_dim=4, inv_freq=[1.0, float("nan")])])
def test_rope_refusals(mr, kw):
    with pytest.raises(mr.MRError) as e:
        mr.Rope(**kw)
    assert e.value.code == mr.MR_ERR_INVALID_ARG


def test_rope_python_refusals(mr):
    with pytest.raises(ValueError):
        mr.Rope(64, scaling="unknown")
    with pytest.raises(ValueError):
        mr.Rope(64, rot_dim=8, inv_freq=[1.0])


# ------------------------------------------------------------------------------------------------ C refusals
FAKE = 0x10000  # never dereferenced: every call here must fail validation first


def _cache(mr, **kw):
    a = dict(k=FAKE, v=FAKE, dt=mr.MR_BF16, H_kv=2, page_rows=16, d=64, n_pages=10)
    a.update(kw)
    return mr.KvCache(*[a[n] for n, _ in mr.KvCache._fields_])


def _seqs(mr, **kw):
    a = dict(table=FAKE, kv_len=FAKE, pages_per_seq=4, n_seq=3)
    a.update(kw)
    return mr.KvSeqs(*[a[n] for n, _ in mr.KvSeqs._fields_])


BAD_CACHES = [(dict(k=None), 1), (dict(v=FAKE + 8), 1), (dict(dt=2), 2), (dict(H_kv=0), 1), (dict(page_rows=0), 1),
              (dict(n_pages=0), 1), (dict(d=96), 2), (dict(n_pages=2 ** 26), 2), (dict(n_pages=2 ** 62), 2)]
BAD_SEQS = [dict(table=None), dict(kv_len=None), dict(pages_per_seq=0), dict(n_seq=0)]


def test_rope_apply_refuses(mr):
    r = mr.Rope(64)
    x = mr.Rows(FAKE, 640, 64)

    def call(rope=r.c, X=x, Y=x, dt=0, H=4, n=10, pos=FAKE):
        return mr.LIB.mr_rope_apply(ctypes.byref(rope) if rope else None, ctypes.byref(X) if X else None,
                                    ctypes.byref(Y) if Y else None, dt, H, n, pos, 0, None)
    assert call(rope=None) == call(X=None) == call(Y=None) == call(pos=None) == mr.MR_ERR_INVALID_ARG
    assert call(H=0) == call(n=-1) == mr.MR_ERR_INVALID_ARG
    assert call(dt=2) == call(H=5000) == mr.MR_ERR_UNSUPPORTED
    assert call(X=mr.Rows(FAKE, -640, 64)) == mr.MR_ERR_INVALID_ARG
    assert call(X=mr.Rows(FAKE + 1, 640, 64)) == mr.MR_ERR_INVALID_ARG
    assert call(Y=mr.Rows(FAKE, 64, 64)) == mr.MR_ERR_INVALID_ARG          # output heads and rows overlap
    assert call(Y=mr.Rows(FAKE * 2, 630, 64)) == mr.MR_ERR_INVALID_ARG     # the last row runs into the next head
    assert call(Y=mr.Rows(FAKE, 64, 256)) == mr.MR_ERR_INVALID_ARG         # in place with other strides
    bad = mr.RopeTable.from_buffer_copy(r.c)
    bad.rot_dim = 66
    assert call(rope=bad) == mr.MR_ERR_INVALID_ARG
    assert call(n=0, pos=None) == mr.MR_OK                                 # nothing to do


def test_append_refuses(mr):
    r = mr.Rope(64)
    x = mr.Rows(FAKE, 640, 64)
    n_ws = mr.LIB.mr_paged_workspace_bytes(ctypes.byref(_cache(mr)), 4, 3)
    assert n_ws >= 256

    def call(c=None, s=None, rope=r.c, Q=x, Qo=x, Hq=4, K=x, V=x, cu=FAKE, total=10, ws=FAKE, wsb=n_ws):
        ref = lambda o: ctypes.byref(o) if o is not None else None
        return mr.LIB.mr_kv_append(ref(c or _cache(mr)), ref(s or _seqs(mr)), ref(rope), ref(Q), ref(Qo), Hq, ref(K),
                                   ref(V), cu, total, ws, wsb, None)
    for kw, code in BAD_CACHES:
        assert call(c=_cache(mr, **kw)) == code, kw
    for kw in BAD_SEQS:
        assert call(s=_seqs(mr, **kw)) == mr.MR_ERR_INVALID_ARG, kw
    for kw in (dict(ws=None), dict(wsb=16), dict(total=-1), dict(cu=None), dict(K=None), dict(V=None), dict(Q=None),
               dict(Qo=None), dict(Hq=0), dict(rope=mr.Rope(128).c), dict(K=mr.Rows(None, 640, 64)),
               dict(Qo=mr.Rows(FAKE, 64, 64))):
        assert call(**kw) == mr.MR_ERR_INVALID_ARG, kw
    assert call(Hq=5000) == mr.MR_ERR_UNSUPPORTED


def test_decode_refuses(mr):
    x = mr.Rows(FAKE, 192, 64)
    n_ws = mr.LIB.mr_paged_workspace_bytes(ctypes.byref(_cache(mr)), 4, 3)

    def call(c=None, s=None, Q=x, Hq=4, scale=0.125, window=0, sinks=0, O=x, ws=FAKE, wsb=n_ws):
        ref = lambda o: ctypes.byref(o) if o is not None else None
        return mr.LIB.mr_paged_decode(ref(c or _cache(mr)), ref(s or _seqs(mr)), ref(Q), Hq, scale, window, sinks, ref(O),
                                      None, ws, wsb, None)
    for kw, code in BAD_CACHES:
        assert call(c=_cache(mr, **kw)) == code, kw
    for kw in BAD_SEQS:
        assert call(s=_seqs(mr, **kw)) == mr.MR_ERR_INVALID_ARG, kw
    for kw in (dict(ws=None), dict(ws=FAKE + 8), dict(wsb=n_ws - 1), dict(Q=None), dict(O=None), dict(Hq=0), dict(Hq=5),
               dict(scale=float("nan")), dict(scale=float("inf")), dict(window=-1), dict(sinks=-1),
               dict(Q=mr.Rows(FAKE, -192, 64)), dict(Q=mr.Rows(FAKE + 1, 192, 64)), dict(O=mr.Rows(FAKE, 64, 64)),
               dict(O=mr.Rows(FAKE, 0, 64))):
        assert call(**kw) == mr.MR_ERR_INVALID_ARG, kw
    assert call(Hq=2048) == mr.MR_ERR_UNSUPPORTED


def test_attn_refuses(mr):
    x = mr.Rows(FAKE, 640, 64)
    n_ws = mr.LIB.mr_paged_workspace_bytes(ctypes.byref(_cache(mr)), 4, 3)

    def call(c=None, s=None, Q=x, Hq=4, cu=FAKE, total=10, scale=0.125, window=0, sinks=0, O=x, ws=FAKE, wsb=n_ws):
        ref = lambda o: ctypes.byref(o) if o is not None else None
        return mr.LIB.mr_paged_attn(ref(c or _cache(mr)), ref(s or _seqs(mr)), ref(Q), Hq, cu, total, scale, window, sinks,
                                    ref(O), None, ws, wsb, None)
    for kw, code in BAD_CACHES:
        assert call(c=_cache(mr, **kw)) == code, kw
    for kw in BAD_SEQS:
        assert call(s=_seqs(mr, **kw)) == mr.MR_ERR_INVALID_ARG, kw
    for kw in (dict(ws=None), dict(ws=FAKE + 8), dict(wsb=n_ws - 1), dict(Q=None), dict(O=None), dict(Hq=0), dict(Hq=5),
               dict(scale=float("nan")), dict(scale=float("-inf")), dict(window=-1), dict(sinks=-1), dict(cu=None),
               dict(total=-1), dict(Q=mr.Rows(FAKE, -640, 64)), dict(Q=mr.Rows(FAKE + 1, 640, 64)),
               dict(O=mr.Rows(FAKE, 64, 64)), dict(O=mr.Rows(FAKE, 0, 64)), dict(O=mr.Rows(FAKE, 630, 64))):
        assert call(**kw) == mr.MR_ERR_INVALID_ARG, kw
    assert call(Hq=2048) == mr.MR_ERR_UNSUPPORTED


def test_workspace_sizes(mr):
    n = lambda Hq=4, n_seq=3, **kw: mr.LIB.mr_paged_workspace_bytes(ctypes.byref(_cache(mr, **kw)), Hq, n_seq)
    assert n() >= 256 and n(d=96) == 0 and n(Hq=5) == 0 and n(Hq=0) == 0 and n(n_seq=0) == 0
    assert mr.LIB.mr_paged_workspace_bytes(None, 4, 3) == 0
    assert mr.pages_copy_workspace_bytes() >= 256


def test_pages_copy_refuses(mr):
    def call(pools=(FAKE, FAKE * 2), n_pools=2, page=1024, n_pages=8, pairs=FAKE, n=3, ws=FAKE, wsb=256):
        arr = (ctypes.c_void_p * len(pools))(*pools) if pools is not None else None
        return mr.LIB.mr_pages_copy(arr, n_pools, page, n_pages, pairs, n, ws, wsb, None)
    for kw in (dict(pools=None), dict(n_pools=0), dict(page=0), dict(page=24), dict(n_pages=0), dict(pairs=None), dict(n=-1),
               dict(ws=None), dict(wsb=16), dict(pools=(FAKE, None)), dict(pools=(FAKE, FAKE + 8))):
        assert call(**kw) == mr.MR_ERR_INVALID_ARG, kw
    assert call(n_pages=2 ** 31) == mr.MR_ERR_UNSUPPORTED


def test_python_refuses_what_is_not_on_a_gpu(mr):
    import torch
    x, pos = torch.zeros(2, 3, 64), torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError):
        mr.rope(mr.Rope(64), x, pos)
    with pytest.raises(ValueError):
        mr.KVCache(x[None], x[None])
    with pytest.raises(ValueError):
        mr.pages_copy([], pos.view(-1, 1))
    with pytest.raises(ValueError):
        mr.pages_copy([x], pos.view(-1, 1))


# ------------------------------------------------------------------------------------------------ page pool
def test_pool_extend_fork_and_copy_on_write(mr):
    pp = mr.PagePool(8, 16)
    a = pp.open()
    assert pp.extend(a, 0) == [] and pp.extend(a, 40) == []
    t, n = pp.tables([a], 5)
    assert t.tolist() == [[0, 1, 2, -1, -1]] and n.tolist() == [40]
    b = pp.fork(a, 40)
    c = pp.fork(a, 32)                       # ends with a whole page: nothing of it is written later
    assert pp.stats() == dict(pages=8, free=5, sequences=3, shared=3)
    assert pp.extend(b, 1) == [(2, 3)]       # the partly filled page is shared: b gets its own
    assert pp.extend(a, 1) == []             # and a is alone with the old one
    assert pp.extend(c, 1) == []
    assert pp.tables([a, b, c])[0].tolist() == [[0, 1, 2], [0, 1, 3], [0, 1, 4]]
    pp.close(a)
    assert pp.stats()["free"] == 4
    with pytest.raises(mr.MRError):
        pp.extend(a, 1)


def test_pool_refuses_and_changes_nothing(mr):
    assert not mr.LIB.mr_pp_create(0, 16) and not mr.LIB.mr_pp_create(4, 0)
    pp = mr.PagePool(3, 16)
    a = pp.open()
    pp.extend(a, 40)
    b = pp.fork(a, 40)
    before = pp.tables([a, b])[0].tolist(), pp.stats()
    for f in (lambda: pp.extend(b, 1),                     # no page left for its own copy
              lambda: pp.extend(a, 9)):
        with pytest.raises(mr.MRError) as e:
            f()
        assert e.value.code == mr.MR_ERR_CAPACITY
    for f in (lambda: pp.fork(a, 41), lambda: pp.fork(99, 0), lambda: pp.truncate(a, 41), lambda: pp.extend(a, -1),
              lambda: pp.extend(a, 2 ** 31 - 1), lambda: pp.slide(a, 0), lambda: pp.slide(a, 4, -1), lambda: pp.close(-1)):
        with pytest.raises(mr.MRError) as e:
            f()
        assert e.value.code == mr.MR_ERR_INVALID_ARG
    assert (pp.tables([a, b])[0].tolist(), pp.stats()) == before
    assert mr.LIB.mr_pp_open(None) < 0 and mr.LIB.mr_pp_compact(pp.h, None, 1) < 0


def test_pool_slide_keeps_what_the_next_query_sees(mr):
    pp = mr.PagePool(16, 16)
    a = pp.open()
    pp.extend(a, 100)                        # rows 0 .. 99 on 7 pages
    # the next query (position 100, window 40) sees rows 61 .. 100, and rows 0 .. 19
    assert pp.slide(a, 40, 20) == 1
    assert pp.tables([a])[0].tolist() == [[0, 1, -1, 3, 4, 5, 6]]
    assert pp.slide(a, 40, 20) == 0
    with pytest.raises(mr.MRError):
        pp.truncate(a, 40)                   # row 39 is gone
    with pytest.raises(mr.MRError):
        pp.fork(a, 48)
    pp.truncate(a, 32)
    assert pp.tables([a])[0].tolist() == [[0, 1]]
    b = pp.open()
    pp.extend(b, 32)
    assert pp.slide(b, 1) == 2 and pp.extend(b, 1) == []   # window 1: nothing held is seen again


def test_pool_against_a_model(mr):
    rng = random.Random(7)
    n_pages, pr = 24, 4
    pp = mr.PagePool(n_pages, pr)
    model = {}                               # id -> list of row contents
    store = {}                               # page -> row contents, moved by the pairs

    def check():
        ids = sorted(model)
        refs = {}
        for s in ids:
            t, n = pp.tables([s])
            assert n[0] == len(model[s])
            pages = t[0][: -(-len(model[s]) // pr)].tolist()
            for p in pages:
                refs[p] = refs.get(p, 0) + 1
            got = [store[(pages[j // pr], j % pr)] for j in range(len(model[s]))]
            assert got == model[s]
        st = pp.stats()
        assert st["free"] == n_pages - len(refs) and st["sequences"] == len(ids)
        assert st["shared"] == sum(r > 1 for r in refs.values())

    tick = 0
    for _ in range(3000):
        op = rng.choice(("open", "extend", "extend", "extend", "fork", "truncate", "close", "compact"))
        s = rng.choice(sorted(model)) if model else None
        if op == "open" and len(model) < 6:
            model[pp.open()] = []
        elif op == "extend" and s is not None:
            n = rng.randrange(0, 9)
            try:
                pairs = pp.extend(s, n)
            except mr.MRError as e:
                assert e.code == mr.MR_ERR_CAPACITY
                check()
                continue
            for a, b in pairs:
                for r in range(pr):
                    if (a, r) in store:
                        store[(b, r)] = store[(a, r)]
            t = pp.tables([s])[0][0]
            for _ in range(n):
                j = len(model[s])
                store[(int(t[j // pr]), j % pr)] = tick
                model[s].append(tick)
                tick += 1
        elif op == "fork" and s is not None and len(model) < 6:
            n = rng.randrange(0, len(model[s]) + 1)
            model[pp.fork(s, n)] = model[s][:n]
        elif op == "truncate" and s is not None:
            n = rng.randrange(0, len(model[s]) + 1)
            pp.truncate(s, n)
            del model[s][n:]
        elif op == "close" and s is not None:
            pp.close(s)
            del model[s]
        elif op == "compact":
            most = rng.choice((1, 2, n_pages))
            pairs = pp.compact(most).tolist()
            assert len(pairs) <= most
            assert not {a for a, _ in pairs} & {b for _, b in pairs}
            old = dict(store)
            for a, b in pairs:
                for r in range(pr):
                    if (a, r) in old:
                        store[(b, r)] = old[(a, r)]
            if most == n_pages and model:
                used = n_pages - pp.stats()["free"]
                tables = [p for s in model for p in pp.tables([s])[0][0].tolist() if p >= 0]
                assert not tables or max(tables) < used
        check()
