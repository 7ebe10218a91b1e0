"""What the paged-cache operators cost: their cases, their plain forms and their definitions in 64 bits.

The five operators are the ones a receiver model needs around the reuse of a prefix: rotary positions
(``rope``), rotation and appending of new rows to a paged key-value cache (``append``), attention of one
new token per sequence over that cache (``decode``), attention of a chunk of new rows over it with an
optional sliding window and first rows that stay visible (``attn``), and copying pages (``pages``).

A pool is [page][kv head][row][d].  Sequence s holds ``kv_len[s]`` rows after its new rows are appended;
its row j is row j % page_rows of page table[s][j // page_rows].  The i-th of its n new rows has
position p = kv_len[s] - n + i and sees row j when 0 <= j <= p and (window == 0, j > p - window or
j < sinks).
"""
import math

import torch

own = False

# head counts that this repository's workloads have on either side, and the divisors used as groups
_HEADS = (4, 8, 28, 32, 40, 64)
_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_SIZE = {"bf16": 2, "f32": 4}


# ---------------------------------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------------------------------
def _rope_case(**kw):
    return dict(dict(op="rope", H=32, T=4096, d=128, rot=128, dt="bf16", interleaved=False, scaling="none", factor=1.0,
                     adjoint=False, far=0), **kw)


def _append_case(**kw):
    return dict(dict(op="append", Hq=32, group=4, n_seq=16, rows_min=1, rows_max=1, len_min=4096, len_max=6144, d=128,
                     rot=128, dt="bf16", interleaved=False, scaling="none", factor=1.0, page_rows=64), **kw)


def _decode_case(**kw):
    return dict(dict(op="decode", Hq=32, group=4, n_seq=16, len_min=4608, len_max=6144, d=128, dt="bf16", page_rows=64,
                     window=0, sinks=0), **kw)


def _attn_case(**kw):
    return dict(dict(op="attn", Hq=32, group=4, n_seq=4, rows_min=512, rows_max=2048, past=4096, d=128, dt="bf16",
                     page_rows=64, window=0, sinks=0), **kw)


def _pages_case(**kw):
    return dict(dict(op="pages", n_pages=512, moved=64, layers=1, H=8, page_rows=64, d=128, dt="bf16"), **kw)


def listed():
    return [
        # the gradient with respect to the unrotated queries of a 4096-token prompt
        _rope_case(name="rope_adjoint_4096", adjoint=True),
        # half of the head rotated in neighbouring pairs, single precision, a short toy prompt
        _rope_case(name="rope_part_f32_500", H=4, T=500, d=64, rot=32, dt="f32", interleaved=True),
        # one decoding step of 16 requests that share a 4096-token prefix
        _append_case(name="append_step_16"),
        # a whole 8192-token prompt behind nothing, frequencies stretched for a long context
        _append_case(name="append_prompt_8192", n_seq=1, rows_min=8192, rows_max=8192, len_min=8192, len_max=8192,
                     Hq=28, group=7, scaling="ramp", factor=4.0),
        # one request of the toy workload in single precision: the time of a call that does little
        _decode_case(name="decode_f32_512", Hq=4, group=1, n_seq=1, len_min=512, len_max=512, d=64, dt="f32"),
        # 16 requests behind a shared prefix of 4096 tokens, suffixes of 512 to 2048
        _decode_case(name="decode_ragged_16"),
        # 8 long conversations, 64 receiver heads in groups of 8
        _decode_case(name="decode_8x32768", Hq=64, group=8, n_seq=8, len_min=32768, len_max=32768, page_rows=128),
        # the toy workload's prompt beside two shorter ones in single precision, its sink and window as a mask
        _attn_case(name="attn_f32_toy", Hq=4, group=1, n_seq=3, rows_min=77, rows_max=512, past=0, d=64, dt="f32",
                   window=128, sinks=16),
        # the rows that four requests compute themselves behind a reused prefix of 4096 tokens
        _attn_case(name="attn_suffix_4"),
        # a long prompt under a sliding window with 16 first tokens kept
        _attn_case(name="attn_window_16384", Hq=8, group=4, n_seq=1, rows_min=16384, rows_max=16384, past=0, window=4096,
                   sinks=16, page_rows=128),
        # the last, partly filled page of each of 16 forked requests, one layer
        _pages_case(name="pages_fork_16", moved=16),
        # a pool of four layers compacted: a quarter of its pages move to the front
        _pages_case(name="pages_compact_1024", n_pages=2048, moved=512, layers=4),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _heads(rng, most=64):
    h = rng.choice([x for x in _HEADS if x <= most])
    return h, rng.choice([g for g in (1, 2, 4, 5, 7, 8) if h % g == 0])


def draw(rng):
    op = rng.choice(("rope", "append", "decode", "attn", "pages"))
    dt = rng.choice(("bf16", "bf16", "f32"))
    d = rng.choice((64, 128))
    rot = rng.choice((d, d, d // 2, d // 4))
    turn = dict(interleaved=rng.random() < 0.5, scaling=rng.choice(("none", "linear", "base", "ramp")))
    turn["factor"] = 1.0 if turn["scaling"] == "none" else rng.choice((2.0, 4.0, 8.0))
    page_rows = rng.choice((16, 32, 64, 128))
    if op == "rope":
        h, _ = _heads(rng)
        return _rope_case(H=h, T=_log(rng, 1, 4096), d=d, rot=rot, dt=dt, adjoint=rng.random() < 0.5,
                          far=rng.choice((0, 100000)), **turn)
    if op == "append":
        h, g = _heads(rng)
        n = _log(rng, 1, 32)
        most = 2 ** 17 // (n * h // g)  # rows of a sequence that keep the pools below 128 MB each
        rows = 1 if rng.random() < 0.4 else _log(rng, 2, min(4096, most))
        return _append_case(Hq=h, group=g, n_seq=n, rows_min=max(1, rows // 2), rows_max=rows, len_min=rows,
                            len_max=rows + _log(rng, 1, min(2048, most)), d=d, rot=rot, dt=dt, page_rows=page_rows, **turn)
    if op == "decode":
        h, g = _heads(rng)
        n = _log(rng, 1, 64)
        longest = _log(rng, 1, min(32768, 2 ** 21 * g // (n * h * _SIZE[dt])))  # pools below 512 MB
        win = rng.random() < 0.4
        return _decode_case(Hq=h, group=g, n_seq=n, len_min=max(1, longest // 3), len_max=longest, d=d, dt=dt,
                            page_rows=page_rows, window=_log(rng, 1, 4096) if win else 0,
                            sinks=rng.choice((0, 4, 16)) if win else 0)
    if op == "attn":
        h, g = _heads(rng, 40)
        n = _log(rng, 1, 8)
        rows = _log(rng, 1, 4096)
        past = rng.choice((0, _log(rng, 1, 4096)))
        while n * h * rows * (rows + past) > 2 ** 29:
            rows = rows // 2 + 1
            past = past // 2
        win = rng.random() < 0.6
        return _attn_case(Hq=h, group=g, n_seq=n, rows_min=max(1, rows // 3), rows_max=rows, past=past, d=d, dt=dt,
                          page_rows=page_rows, window=_log(rng, 1, 4096) if win else 0,
                          sinks=rng.choice((0, 4, 16, 200)) if win else 0)
    layers, h = rng.choice((1, 2, 4)), rng.choice((1, 2, 4, 8))
    n_pages = _log(rng, 8, min(4096, 2 ** 30 // (layers * h * page_rows * d * _SIZE[dt])))  # pools below 2 GB together
    return _pages_case(n_pages=n_pages, moved=_log(rng, 1, n_pages // 4), layers=layers, H=h, page_rows=page_rows, d=d,
                       dt=dt)


# ---------------------------------------------------------------------------------------------------
# Sizes that follow from a case (lengths are drawn from the case alone, so that work() knows them)
# ---------------------------------------------------------------------------------------------------
def _spread(n, lo, hi):
    """n lengths between lo and hi, both of them among these, in an order that is not sorted."""
    if n == 1:
        return [hi]
    return [lo + (hi - lo) * ((7 * i + n - 1) % n if math.gcd(7, n) == 1 else i) // (n - 1) for i in range(n)]


def _lens(c):
    """(new rows, rows held after them) of each sequence."""
    if c["op"] == "decode":
        held = _spread(c["n_seq"], c["len_min"], c["len_max"])
        return [1] * c["n_seq"], held
    new = _spread(c["n_seq"], c["rows_min"], c["rows_max"])
    if c["op"] == "attn":
        return new, [n + c["past"] for n in new]
    return new, _spread(c["n_seq"], c["len_min"], c["len_max"])


def _seen(new, held, window, sinks):
    """(pairs of a new row and a row it sees, rows that any of them sees) of one sequence."""
    pairs = 0
    for p in range(held - new, held):
        lo = 0 if window == 0 else max(0, p - window + 1)
        pairs += p + 1 - lo + min(sinks, lo)
    lo = 0 if window == 0 else max(0, held - new - window + 1)
    return pairs, held - lo + min(sinks, lo)


def work(c):
    if c["op"] == "pages":
        page = c["H"] * c["page_rows"] * c["d"] * _SIZE[c["dt"]]
        return {"bytes": 2.0 * c["moved"] * 2 * c["layers"] * page + 8.0 * c["moved"], "flops": 0.0}
    e, d = _SIZE[c["dt"]], c["d"]
    if c["op"] == "rope":
        return {"bytes": 2.0 * c["H"] * c["T"] * d * e + 4.0 * c["T"], "flops": 3.0 * c["H"] * c["T"] * c["rot"]}
    new, held = _lens(c)
    Hq, Hk, T = c["Hq"], c["Hq"] // c["group"], sum(new)
    if c["op"] == "append":
        return {"bytes": 2.0 * (Hq + 2 * Hk) * T * d * e + 8.0 * c["n_seq"], "flops": 3.0 * (Hq + Hk) * T * c["rot"]}
    seen = [_seen(n, h, c["window"], c["sinks"]) for n, h in zip(new, held)]
    rows = sum(r for _, r in seen)
    pages = sum(-(-h // c["page_rows"]) for h in held)
    return {"bytes": 2.0 * Hk * rows * d * e + 2.0 * Hq * T * d * e + 4.0 * Hq * T + 4.0 * pages,
            "flops": 4.0 * Hq * sum(p for p, _ in seen) * d}


# ---------------------------------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------------------------------
def _normal(gen, shape, dt):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(dt)


def _inputs(c, seed):
    """The tensors of one call, from the seed alone."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed) * 1000003 + 17)
    dt, d = _DT[c["dt"]], c["d"]
    s = {"c": c}
    if c["op"] == "rope":
        s["x"] = _normal(gen, (c["H"], c["T"], d), dt)
        s["pos"] = torch.arange(c["T"], dtype=torch.int32, device="cuda") + c["far"]
        return s
    if c["op"] == "pages":
        shape = (c["n_pages"], c["H"], c["page_rows"], d)
        s["pools"] = [_normal(gen, shape, dt) for _ in range(2 * c["layers"])]
        order = torch.randperm(c["n_pages"], generator=gen, device="cuda").to(torch.int32)
        s["pairs"] = torch.stack([order[: c["moved"]], order[c["moved"]: 2 * c["moved"]]], 1).contiguous()
        return s
    new, held = _lens(c)
    Hq, Hk, n, pr = c["Hq"], c["Hq"] // c["group"], c["n_seq"], c["page_rows"]
    per = max(-(-h // pr) for h in held)
    s["T"], s["most_new"], s["most_held"] = sum(new), max(new), max(held)
    # every sequence has pages of its own, handed out in no order
    s["table"] = torch.randperm(n * per, generator=gen, device="cuda").to(torch.int32).reshape(n, per).contiguous()
    s["kv_len"] = torch.tensor(held, dtype=torch.int32, device="cuda")
    s["cu"] = torch.tensor([0] + [sum(new[: i + 1]) for i in range(n)], dtype=torch.int32, device="cuda")
    s["k"], s["v"] = (_normal(gen, (n * per, Hk, pr, d), dt) for _ in range(2))
    s["q"] = _normal(gen, (Hq, s["T"], d), dt)
    if c["op"] == "append":
        s["k_new"], s["v_new"] = (_normal(gen, (Hk, s["T"], d), dt) for _ in range(2))
    return s


def prepare(c, seed):
    s = _inputs(c, seed)
    if c["op"] in ("rope", "append"):
        s["inv_freq"], s["mscale"] = _inv_freq(c)
    if own:
        from cross_model_attention_mr_b200 import mr
        s["mr"] = mr
        if c["op"] in ("rope", "append"):
            s["rope"] = mr.Rope(c["d"], rot_dim=c["rot"], base=10000.0, interleaved=c["interleaved"],
                                scaling=c["scaling"], factor=c["factor"], orig_len=4096, mscale=s["mscale"])
        if c["op"] == "pages":
            s["ws"] = mr.Workspace(mr.pages_copy_workspace_bytes())
        elif c["op"] != "rope":
            s["cache"] = mr.KVCache(s["k"], s["v"])
            s["ws"] = mr.Workspace(mr.paged_workspace_bytes(s["cache"], c["Hq"], c["n_seq"]))
    return s


# ---------------------------------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------------------------------
def run(s):
    c = s["c"]
    if own:
        mr = s["mr"]
        if c["op"] == "rope":
            return mr.rope(s["rope"], s["x"], s["pos"], adjoint=c["adjoint"])
        if c["op"] == "append":
            q = mr.kv_append(s["cache"], s["table"], s["kv_len"], s["k_new"], s["v_new"], cu_q=s["cu"], rope=s["rope"],
                             Q=s["q"], ws=s["ws"])
            return [q, s["k"], s["v"]]
        if c["op"] == "decode":
            return mr.paged_decode(s["cache"], s["table"], s["kv_len"], s["q"], window=c["window"], sinks=c["sinks"],
                                   return_lse=True, ws=s["ws"])
        if c["op"] == "attn":
            return mr.paged_attn(s["cache"], s["table"], s["kv_len"], s["q"], s["cu"], window=c["window"],
                                 sinks=c["sinks"], return_lse=True, ws=s["ws"])
        mr.pages_copy(s["pools"], s["pairs"], ws=s["ws"])
        return s["pools"]
    if c["op"] == "rope":
        return _plain_rope(s, s["x"], s["pos"], -1.0 if c["adjoint"] else 1.0).to(s["x"].dtype)
    if c["op"] == "append":
        return _plain_append(s)
    if c["op"] == "decode":
        return _plain_decode(s)
    if c["op"] == "attn":
        return _plain_attn(s)
    src, dst = s["pairs"][:, 0].long(), s["pairs"][:, 1].long()
    for p in s["pools"]:
        p[dst] = p[src]
    return s["pools"]


# ---------------------------------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------------------------------
def _inv_freq(c):
    """Angles per position of the rotated pairs (in 64 bits), and the factor on rotated values."""
    r = c["rot"]
    base = 10000.0
    if c["scaling"] == "base":
        base *= c["factor"] ** (r / (r - 2))
    f = base ** (-torch.arange(0, r, 2, dtype=torch.float64, device="cuda") / r)
    if c["scaling"] == "linear":
        f = f / c["factor"]
    if c["scaling"] == "ramp":
        turns = 4096 * f / (2 * math.pi)                     # over the length the model was trained on
        keep = ((turns - 1.0) / (32.0 - 1.0)).clamp(0.0, 1.0)  # 1: left alone, 0: stretched by the factor
        f = f * keep + f / c["factor"] * (1 - keep)
    return f, 0.1 * math.log(c["factor"]) + 1.0 if c["scaling"] == "ramp" else 1.0


def _plain_rope(s, x, pos, sign):
    """x [H][T][d] rotated by sign * pos * f, in 32 bits (angles in 64)."""
    c, r = s["c"], s["c"]["rot"]
    angle = pos.double()[:, None] * s["inv_freq"]
    cos, sin = (angle.cos() * s["mscale"]).float(), (angle.sin() * (sign * s["mscale"])).float()
    x = x.float()
    if c["interleaved"]:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., : r // 2], x[..., r // 2: r]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([y, x[..., r:]], -1)


def _places(s):
    """Of each new row: its sequence, its number among that sequence's new rows, and its position."""
    t = torch.arange(s["T"], device="cuda", dtype=torch.int32)
    seq = (t[:, None] >= s["cu"][None, 1:]).sum(1)
    i = t - s["cu"][seq]
    return seq, i.long(), (s["kv_len"][seq] - s["cu"][seq + 1] + t).long()


def _plain_append(s):
    seq, _, pos = _places(s)
    pr = s["c"]["page_rows"]
    page, row = s["table"][seq, pos // pr].long(), pos % pr
    s["k"][page, :, row] = _plain_rope(s, s["k_new"], pos, 1.0).to(s["k"].dtype).transpose(0, 1)
    s["v"][page, :, row] = s["v_new"].transpose(0, 1)
    return [_plain_rope(s, s["q"], pos, 1.0).to(s["q"].dtype), s["k"], s["v"]]


def _rows(s, pool):
    """[n_seq][kv heads][rows][d] of a pool in 32 bits, page by page."""
    n, per = s["table"].shape
    got = pool[s["table"].long()].transpose(1, 2)
    return got.reshape(n, pool.shape[1], per * pool.shape[2], pool.shape[3])[:, :, : s["most_held"]].float()


def _softmax_product(x, v):
    """softmax(x) v over the last axis and its log normaliser; a row of -inf gives zeros and -inf."""
    top = x.amax(-1, keepdim=True)
    x = x.sub_(top.masked_fill(top == -math.inf, 0.0)).exp_()
    total = x.sum(-1, keepdim=True)
    out = x @ v
    return out / total.masked_fill(total == 0, 1.0), (top + total.log()).squeeze(-1)


def _plain_decode(s):
    c = s["c"]
    n, Hk, G, d = c["n_seq"], c["Hq"] // c["group"], c["group"], c["d"]
    k, v = _rows(s, s["k"]), _rows(s, s["v"])
    q = s["q"].float().reshape(Hk, G, n, d).permute(2, 0, 1, 3)
    x = q @ k.transpose(-1, -2) * (1.0 / math.sqrt(d))
    j = torch.arange(k.shape[2], device="cuda")
    p = (s["kv_len"] - 1)[:, None]
    hidden = j > p
    if c["window"]:
        hidden = hidden | ((j <= p - c["window"]) & (j >= c["sinks"]))
    out, lse = _softmax_product(x.masked_fill_(hidden[:, None, None, :], -math.inf), v)
    return (out.permute(1, 2, 0, 3).reshape(c["Hq"], n, d).to(s["q"].dtype),
            lse.permute(1, 2, 0).reshape(c["Hq"], n))


def _plain_attn(s):
    c = s["c"]
    n, Hk, G, d = c["n_seq"], c["Hq"] // c["group"], c["group"], c["d"]
    k, v = _rows(s, s["k"]), _rows(s, s["v"])
    seq, i, pos = _places(s)
    q = torch.zeros((n, c["Hq"], s["most_new"], d), device="cuda")  # the new rows, padded to the most of any sequence
    q[seq, :, i] = s["q"].float().transpose(0, 1)
    p = torch.full((n, s["most_new"]), -1, device="cuda", dtype=torch.long)
    p[seq, i] = pos
    x = q.reshape(n, Hk, G * s["most_new"], d) @ k.transpose(-1, -2) * (1.0 / math.sqrt(d))
    x = x.reshape(n, Hk, G, s["most_new"], -1)
    j, p = torch.arange(k.shape[2], device="cuda"), p[:, :, None]
    hidden = j > p
    if c["window"]:
        hidden = hidden | ((j <= p - c["window"]) & (j >= c["sinks"]))
    out, lse = _softmax_product(x.masked_fill_(hidden[:, None, None], -math.inf), v[:, :, None])
    out, lse = out.reshape(n, c["Hq"], -1, d), lse.reshape(n, c["Hq"], -1)
    return out[seq, :, i].transpose(0, 1).to(s["q"].dtype).contiguous(), lse[seq, :, i].transpose(0, 1).contiguous()


# ---------------------------------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------------------------------
def _exact_turn(c, x, pos, sign):
    """Rotation as a product of complex numbers, one per pair."""
    r = c["rot"]
    i = torch.arange(r // 2, dtype=torch.float64, device="cuda")
    factor = c["factor"]
    theta = torch.exp(-2.0 * i / r * math.log(10000.0))
    m = 1.0
    if c["scaling"] == "linear":
        theta = theta / factor
    elif c["scaling"] == "base":
        theta = torch.exp(-2.0 * i / r * (math.log(10000.0) + r / (r - 2) * math.log(factor)))
    elif c["scaling"] == "ramp":
        wave = 2.0 * math.pi / theta
        g = torch.clamp((4096.0 / wave - 1.0) / 31.0, min=0.0, max=1.0)
        theta = (1.0 - g) * theta / factor + g * theta
        m = 1.0 + 0.1 * math.log(factor)
    x = x.double()
    head = x[..., :r]
    if c["interleaved"]:
        z = torch.complex(head[..., 0::2].contiguous(), head[..., 1::2].contiguous())
    else:
        z = torch.complex(head[..., : r // 2].contiguous(), head[..., r // 2:].contiguous())
    z = z * torch.polar(torch.full_like(theta, m).expand(len(pos), -1).contiguous(), sign * torch.outer(pos.double(), theta))
    out = x.clone()
    if c["interleaved"]:
        out[..., 0:r:2], out[..., 1:r:2] = z.real, z.imag
    else:
        out[..., : r // 2], out[..., r // 2: r] = z.real, z.imag
    return out


def exact(c, seed):
    s = _inputs(c, seed)
    if c["op"] == "pages":
        for a, b in s["pairs"].tolist():  # copies: nothing is computed
            for pool in s["pools"]:
                pool[b].copy_(pool[a])
        return s["pools"]
    if c["op"] == "rope":
        return _exact_turn(c, s["x"], s["pos"], -1.0 if c["adjoint"] else 1.0)
    new, held = _lens(c)
    pr, d, G = c["page_rows"], c["d"], c["group"]
    table = s["table"].cpu().tolist()
    if c["op"] == "append":
        pos = torch.cat([torch.arange(h - n, h, device="cuda") for n, h in zip(new, held)])
        q, kr = _exact_turn(c, s["q"], pos, 1.0), _exact_turn(c, s["k_new"], pos, 1.0)
        k, v = s["k"].double(), s["v"].double()
        t = 0
        for b, (n, h) in enumerate(zip(new, held)):
            p = h - n
            while p < h:  # one page at a time
                m = min(h - p, pr - p % pr)
                page = table[b][p // pr]
                k[page, :, p % pr: p % pr + m] = kr[:, t: t + m]
                v[page, :, p % pr: p % pr + m] = s["v_new"][:, t: t + m].double()
                p, t = p + m, t + m
        return [q, k, v]
    O = torch.empty((c["Hq"], s["T"], d), dtype=torch.float64, device="cuda")
    lse = torch.empty((c["Hq"], s["T"]), dtype=torch.float64, device="cuda")
    t = 0
    for b, (n, h) in enumerate(zip(new, held)):
        pages = s["table"][b, : -(-h // pr)].long()
        K, V = (x[pages].double().permute(1, 0, 2, 3).flatten(1, 2)[:, :h] for x in (s["k"], s["v"]))
        for a in range(0, n, 1024):
            m = min(1024, n - a)
            p = torch.arange(h - n + a, h - n + a + m, device="cuda")[:, None]
            j = torch.arange(h, device="cuda")[None, :]
            ok = (j <= p) & ((j > p - c["window"]) | (j < c["sinks"]) if c["window"] else torch.ones_like(j > p))
            for r in range(c["Hq"]):
                x = s["q"][r, t + a: t + a + m].double() @ K[r // G].T / math.sqrt(d)
                x = torch.where(ok, x, torch.full_like(x, -math.inf))
                lse[r, t + a: t + a + m] = torch.logsumexp(x, -1)
                O[r, t + a: t + a + m] = torch.softmax(x, -1) @ V[r // G]
        t += n
    return O, lse
