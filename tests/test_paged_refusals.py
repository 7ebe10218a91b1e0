"""Addresses that the paged cache's kernels could not read or write in whole elements, and scales that they could not work
with, are refused on the host, before anything is launched.  No GPU is needed: a refused call touches no device."""
import ctypes

import pytest

FAKE = 0x10000  # never dereferenced: every call here must fail validation first


@pytest.fixture(scope="module")
def mr():
    from cross_model_attention_mr_b200 import mr as m
    return m


def _ref(o):
    return ctypes.byref(o) if o is not None else None


def _calls(mr):
    """Each entry point as a function of the addresses that it takes beside the tensors."""
    cache = mr.KvCache(FAKE, FAKE, mr.MR_BF16, 2, 16, 64, 10)
    x = mr.Rows(FAKE, 640, 64)
    rope = mr.Rope(64)
    n_ws = mr.LIB.mr_paged_workspace_bytes(ctypes.byref(cache), 4, 3)

    def append(table=FAKE, kv_len=FAKE, cu=FAKE, ws=FAKE):
        return mr.LIB.mr_kv_append(_ref(cache), _ref(mr.KvSeqs(table, kv_len, 4, 3)), _ref(rope.c), _ref(x), _ref(x), 4,
                                   _ref(x), _ref(x), cu, 10, ws, n_ws, None)

    def decode(table=FAKE, kv_len=FAKE, lse=None, ws=FAKE, scale=0.125):
        return mr.LIB.mr_paged_decode(_ref(cache), _ref(mr.KvSeqs(table, kv_len, 4, 3)), _ref(x), 4, scale, 0, 0, _ref(x),
                                      lse, ws, n_ws, None)

    def attn(table=FAKE, kv_len=FAKE, cu=FAKE, lse=None, ws=FAKE, scale=0.125):
        return mr.LIB.mr_paged_attn(_ref(cache), _ref(mr.KvSeqs(table, kv_len, 4, 3)), _ref(x), 4, cu, 10, scale, 0, 0,
                                    _ref(x), lse, ws, n_ws, None)

    def copy(pairs=FAKE, ws=FAKE):
        return mr.LIB.mr_pages_copy((ctypes.c_void_p * 1)(FAKE), 1, 1024, 8, pairs, 3, ws, 256, None)

    def rotate(pos=FAKE):
        return mr.LIB.mr_rope_apply(_ref(rope.c), _ref(x), _ref(mr.Rows(2 * FAKE, 640, 64)), 0, 4, 10, pos, 0, None)
    return {"append": append, "decode": decode, "attn": attn, "copy": copy, "rotate": rotate}


@pytest.mark.parametrize("name,what", [("append", "ws"), ("decode", "ws"), ("attn", "ws"), ("copy", "ws"),
                                       ("append", "table"), ("append", "kv_len"), ("append", "cu"), ("decode", "table"),
                                       ("decode", "kv_len"), ("decode", "lse"), ("attn", "table"), ("attn", "kv_len"),
                                       ("attn", "cu"), ("attn", "lse"), ("copy", "pairs"), ("rotate", "pos")])
def test_misaligned_addresses_are_refused(mr, name, what):
    call = _calls(mr)[name]
    for off in (1, 2, 3) + ((4, 8, 12) if what == "ws" else ()):
        assert call(**{what: FAKE + off}) == mr.MR_ERR_INVALID_ARG, off


@pytest.mark.parametrize("name", ["decode", "attn"])
@pytest.mark.parametrize("scale", [3e38, -3e38, 2.4e38])
def test_scales_that_overflow_in_base_2_are_refused(mr, name, scale):
    """They would make products of infinity and 0 of every score that is 0."""
    assert _calls(mr)[name](scale=scale) == mr.MR_ERR_INVALID_ARG
