"""Cutting and forking sequences whose window has moved on: the page pool refuses what a later query could not be answered
from.  Host only."""
import random

import numpy as np
import pytest


@pytest.fixture(scope="module")
def mr():
    from cross_model_attention_mr_b200 import mr as m
    return m


def seen(rows, window, sinks):
    """Held rows that a query at position `rows` sees."""
    j = np.arange(rows)
    return j[(j > rows - window) | (j < sinks)] if window else j


def test_rejecting_rows_after_a_slide(mr):
    pp = mr.PagePool(16, 16)
    a = pp.open()
    pp.extend(a, 100)
    assert pp.slide(a, 40) == 3              # rows 0 .. 47: the next query sees rows 61 .. 100
    for rows in (70, 80, 86, 49):            # the next query would see row 47 or an earlier one
        for f in (pp.truncate, pp.fork):
            with pytest.raises(mr.MRError) as e:
                f(a, rows)
            assert e.value.code == mr.MR_ERR_INVALID_ARG
    assert pp.tables([a])[0].tolist() == [[-1, -1, -1, 3, 4, 5, 6]] and pp.rows(a) == 100
    b = pp.fork(a, 87)                       # rows 48 .. 86
    c = pp.fork(a, 100)
    pp.truncate(a, 87)
    assert pp.tables([a, b, c])[0].tolist() == [[-1, -1, -1, 3, 4, 5, -1], [-1, -1, -1, 3, 4, 5, -1],
                                               [-1, -1, -1, 3, 4, 5, 6]]
    with pytest.raises(mr.MRError):
        pp.truncate(b, 86)                   # a fork knows the slide, too
    pp.truncate(b, 0)
    assert pp.extend(b, 40) == [] and (pp.tables([b])[0] >= 0).all()
    pp.truncate(b, 20)                       # nothing of what it holds now was given up


def test_sinks_and_later_slides(mr):
    pp = mr.PagePool(32, 4)
    a = pp.open()
    pp.extend(a, 60)
    pp.slide(a, 10, 6)                       # pages 0 and 1 stay; rows 8 .. 47 go
    assert pp.tables([a])[0][0].tolist() == [0, 1] + [-1] * 10 + [12, 13, 14]
    with pytest.raises(mr.MRError):
        pp.truncate(a, 56)                   # sees row 47
    b = pp.fork(a, 57)
    pp.slide(b, 4, 30)                       # more sinks than were kept: rows 8 .. 29 are not there
    with pytest.raises(mr.MRError):
        pp.truncate(b, 55)
    pp.slide(b, 4, 6)
    pp.truncate(b, 55)
    c = pp.fork(a, 60)
    pp.slide(c, 1, 0)                        # window 1: nothing held is seen again
    with pytest.raises(mr.MRError):
        pp.truncate(c, 59)                   # but new rows continue in the last row's page
    pp.truncate(c, 60)


def test_slides_against_a_model(mr):
    rng = random.Random(11)
    n_pages, pr = 60, 4
    pp = mr.PagePool(n_pages, pr)
    model = {}                               # id -> [rows, window, sinks]

    def pages(s):
        t, n = pp.tables([s])
        assert n[0] == model[s][0]
        return t[0]

    refused = cut = 0
    for _ in range(4000):
        op = rng.choice(("open", "extend", "extend", "extend", "slide", "slide", "truncate", "truncate", "fork", "close"))
        s = rng.choice(sorted(model)) if model else None
        if op == "open" and len(model) < 5:
            model[pp.open()] = [0, 0, 0]
        elif s is None:
            continue
        elif op == "extend":
            n = rng.randrange(0, 14)
            try:
                pp.extend(s, n)
            except mr.MRError as e:
                assert e.code == mr.MR_ERR_CAPACITY
                continue
            model[s][0] += n
        elif op == "slide":
            # a window and sinks of the sequence, as a model has them
            if not model[s][1]:
                model[s][1:] = [rng.randrange(1, 30), rng.choice((0, 0, 3, 9))]
            pp.slide(s, *model[s][1:])
        elif op in ("truncate", "fork") and (op == "truncate" or len(model) < 5):
            rows, window, sinks = model[s]
            n = rng.randrange(0, rows + 1)
            t = pages(s)
            gone = any(t[j // pr] < 0 for j in seen(n, window, sinks)) or (0 < n and t[(n - 1) // pr] < 0)
            if n < rows and gone:
                with pytest.raises(mr.MRError):
                    getattr(pp, op)(s, n)
                refused += 1
            elif op == "truncate":
                pp.truncate(s, n)
                model[s][0] = n
                cut += n < rows
            else:
                model[pp.fork(s, n)] = [n, window, sinks]
        elif op == "close":
            pp.close(s)
            del model[s]
        for q in model:
            t = pages(q)
            assert all(t[j // pr] >= 0 for j in seen(*model[q]))
    assert refused > 50 and cut > 50
