"""Timed cases of the operators that serve new tokens over a paged cache of keys and values.

Four operators, which a layer runs one after another when it answers:

* ``append``: the RMS norm of the new query and key heads and the position
  rotation, as a prompt's, with K and V written into their pages on the way;
  16-bit pages, or 4-bit ones (a token's row of a head: bf16 ``low`` and
  ``step`` and a code of 0 .. 15 an entry, ``low + step * code``);
* ``read``: rows of the cache back as K and V tensors;
* ``attn``: attention of the new tokens over a 16-bit cache, causal, with an
  optional window and first tokens that stay visible behind it (sinks);
* ``attn`` with ``bits`` 4: the same over a 4-bit cache.

``run`` computes a case in its plain form (elementary torch operations in
fp32, rounded once at the end), or, with ``own``, through this package's
operators. ``exact`` computes it from the definition in fp64.
"""

import math

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
_EPS = 1e-6
_BASE = 10000.0
_TINY = 2.0 ** -60  # a smaller step is stored as 0


# ---------------------------------------------------------------- cases

def _append(name, B, M, H, G, D, dtype, bits, page, rot, interleaved, fused, pad, first=0):
    """``first``: position of a sequence's first token (decoding, M = 1: each
    sequence at a place of its own up to it); ``fused``: q, k and v are slices
    of one [B, M, H + 2G, D] projection; ``pad``: shorter sequences end in
    padding tokens."""
    case = {"op": "append", "B": B, "M": M, "H": H, "G": G, "D": D, "dtype": dtype, "bits": bits,
            "page": page, "rot": rot, "interleaved": interleaved, "fused": fused, "pad": pad,
            "first": first}
    return case if name is None else dict(case, name=name)


def _read(name, B, M, G, D, dtype, bits, page):
    """The first tokens of each sequence, M of the longest one."""
    case = {"op": "read", "B": B, "M": M, "G": G, "D": D, "dtype": dtype, "bits": bits,
            "page": page}
    return case if name is None else dict(case, name=name)


def _attn(name, B, M, H, G, D, dtype, bits, page, length, ragged, left=-1, sinks=0):
    """M new tokens at the end of every sequence; ``length`` tokens in the
    longest, the others (``ragged``) shorter; pages that a window has left
    behind are given back, and their entries of the table are -1."""
    case = {"op": "attn", "B": B, "M": M, "H": H, "G": G, "D": D, "dtype": dtype, "bits": bits,
            "page": page, "length": length, "ragged": ragged, "left": left, "sinks": sinks}
    return case if name is None else dict(case, name=name)


def listed():
    return [
        # one sequence's next token, far into its context: latency
        _append("append_token", 1, 1, 64, 8, 128, "bf16", 16, 64, 128, False, True, False, first=65535),
        # a decoding batch, each sequence at a position of its own, 4-bit pages
        _append("append_decode_q4", 48, 1, 32, 4, 128, "bf16", 4, 64, 128, False, True, False, first=8191),
        # a padded batch of prompts: odd length, half of each head rotated, pairs side by side
        _append("append_padded_q4", 3, 777, 16, 2, 64, "f16", 4, 16, 32, True, False, True),
        # a long prompt
        _append("append_16k", 1, 16384, 64, 8, 128, "bf16", 16, 64, 128, False, True, False),
        # cached tokens of a short batch back as tensors, to go on from
        _read("read_short", 3, 777, 2, 64, "f16", 16, 16),
        # a long 4-bit context back as tensors
        _read("read_64k_q4", 1, 65536, 8, 128, "bf16", 4, 64),
        # the next token of one long sequence: work split over its length
        _attn("attn_token_64k", 1, 1, 64, 8, 128, "bf16", 16, 64, 65536, False),
        # a decoding batch under a window with four first tokens, most pages given back
        _attn("attn_decode_w1024", 48, 1, 32, 4, 128, "bf16", 16, 64, 20000, True, left=1024, sinks=4),
        # drafted tokens checked in one call: small heads, odd lengths, small pages
        _attn("attn_draft", 16, 5, 16, 2, 64, "f16", 16, 16, 2047, True),
        # one short sequence over a 4-bit cache: latency
        _attn("attn_q4_short", 1, 1, 8, 2, 64, "f16", 4, 16, 300, False),
        # a full decoding batch over a 4-bit cache, ragged lengths
        _attn("attn_q4_batch", 64, 1, 64, 8, 128, "bf16", 4, 64, 16384, True),
        # a piece of a prompt over a windowed 4-bit cache
        _attn("attn_q4_chunk", 2, 65, 32, 4, 128, "bf16", 4, 32, 9000, True, left=4096, sinks=16),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "append", "read", "attn", "attn", "attn"])
    dtype = rng.choice(["bf16", "bf16", "f16"])
    bits = rng.choice([16, 4])
    D = rng.choice([64, 128])
    G = rng.choice([1, 2, 4, 8])
    H = G * rng.choice([1, 2, 3, 4, 7, 8, 16] if op == "attn" else [1, 2, 3, 4, 8])
    H = min(H, 64)
    H -= H % G
    page = rng.choice([16, 32, 64, 128])
    if op == "append":
        rows = _log(rng, 1, 16384)  # tokens in all
        B = rng.randint(1, 48) if rows < 64 else rng.randint(1, 3)
        M = max(1, rows // B)
        return _append(None, B, M, H, G, D, dtype, bits, page, rng.choice([D, D, D // 2]),
                       rng.random() < 0.3, rng.random() < 0.7, M > 1 and rng.random() < 0.3,
                       first=rng.choice([0, rng.randint(0, 20000)]))
    if op == "read":
        B = rng.randint(1, 4)
        return _read(None, B, _log(rng, 1, 65536 // B), G, D, dtype, bits, page)
    left, sinks = rng.choice([(-1, 0), (-1, 0), (_log(rng, 16, 4096), 0),
                              (_log(rng, 16, 4096), rng.randint(1, 40))])
    if rng.random() < 0.6:  # decoding, or a few drafted tokens
        B, M = _log(rng, 1, 64), rng.choice([1, 1, 1, 2, 4, 7])
        return _attn(None, B, M, H, G, D, dtype, bits, page,
                     max(M, _log(rng, 10, min(65536, 400000 // B))), rng.random() < 0.7, left, sinks)
    M = _log(rng, 9, 200)
    B = rng.randint(1, 3)
    return _attn(None, B, M, H, G, D, dtype, bits, page, M + _log(rng, 1, 9000), rng.random() < 0.5,
                 left, sinks)


# ---------------------------------------------------------------- inputs

def _normal(g, shape, dtype, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def _quantise(x, wide=torch.float32):
    """Codes, step and low (bf16 values) of every row of the 16-bit x."""
    xf = x.to(wide)
    low = xf.amin(-1, keepdim=True).to(torch.bfloat16).to(wide)
    # (a tensor of 15s: divided by a number, the GPU multiplies by its reciprocal)
    step = ((xf.amax(-1, keepdim=True) - low) / torch.full_like(low, 15.0)).to(torch.bfloat16).to(wide)
    live = step >= _TINY
    code = torch.where(live, ((xf - low) / torch.where(live, step, 1.0)).round().clamp(0, 15), 0.0)
    return code, torch.where(live, step, 0.0), low


def _pack(x):
    """4-bit form of x [..., D]: bytes [..., D/2] (even entries in the low
    four bits) and bf16 (step, low) [..., 2]."""
    code, step, low = _quantise(x)
    code = code.to(torch.uint8)
    return code[..., 0::2] | (code[..., 1::2] << 4), torch.cat((step, low), -1).to(torch.bfloat16)


def _unpack(codes, scale, wide=torch.float32):
    code = torch.stack((codes & 15, codes >> 4), -1).flatten(-2)
    return scale[..., 1:].to(wide) + scale[..., :1].to(wide) * code.to(wide)


def _pages(g, count, case):
    """A cache of `count` pages that holds something everywhere."""
    G, D, page, dt = case["G"], case["D"], case["page"], _DTYPES[case["dtype"]]
    k, v = (_normal(g, (count, page, G, D), dt) for _ in range(2))
    if case["bits"] == 16:
        return {"k": k, "v": v, "k_scale": None, "v_scale": None}
    (kc, ks), (vc, vs) = _pack(k), _pack(v)  # a scale per (page, head, token)
    return {"k": kc, "v": vc, "k_scale": ks.transpose(1, 2).contiguous(),
            "v_scale": vs.transpose(1, 2).contiguous()}


def _table(g, B, tokens, page):
    """Page table of B sequences of up to `tokens`: pages in random order."""
    cols = -(-tokens // page)
    ids = torch.randperm(B * cols + 3, generator=g, device="cuda")[:B * cols]
    return ids.view(B, cols).to(torch.int32), B * cols + 3


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    B, M, G, D, page = (case[x] for x in ("B", "M", "G", "D", "page"))
    dt = _DTYPES[case["dtype"]]
    if case["op"] == "append":
        H, length = case["H"], case["first"] + M
        if case["fused"]:
            x = _normal(g, (B, M, H + 2 * G, D), dt, 1.5)
            q, k, v = x[:, :, :H], x[:, :, H:H + G], x[:, :, H + G:]
        else:
            q, k, v = (_normal(g, (B, M, n, D), dt, 1.5) for n in (H, G, G))
        wq, wk = (_normal(g, (D,), torch.float32, 0.2) + 1.0 for _ in range(2))
        pos = torch.arange(M, device="cuda").expand(B, M) + case["first"]
        if case["first"] and M == 1:  # decoding: every sequence at its own length
            pos = torch.randint(0, length, (B, 1), generator=g, device="cuda")
            pos[0] = case["first"]
        if case["pad"]:  # sequence b ends after ends[b] tokens; the first one is whole
            ends = torch.randint(1, M + 1, (B, 1), generator=g, device="cuda")
            ends[0] = M
            pos = torch.where(torch.arange(M, device="cuda") < ends, pos, -1)
        half = case["rot"] // 2
        freq = _BASE ** (-torch.arange(half, dtype=torch.float64, device="cuda") / half)
        ang = torch.arange(length, dtype=torch.float64, device="cuda")[:, None] * freq
        table, count = _table(g, B, length, page)
        return {"case": case, "q": q, "k": k, "v": v, "wq": wq, "wk": wk, "cos": ang.cos().float(),
                "sin": ang.sin().float(), "pos": pos.to(torch.int32).contiguous(), "table": table,
                "cache": _pages(g, count, case)}
    if case["op"] == "read":
        table, count = _table(g, B, M, page)
        ends = torch.randint(1, M + 1, (B, 1), generator=g, device="cuda")
        ends[0] = M
        at = torch.arange(M, device="cuda")
        return {"case": case, "pos": torch.where(at < ends, at, -1).to(torch.int32).contiguous(),
                "table": table, "cache": _pages(g, count, case)}
    length = case["length"]
    table, count = _table(g, B, length, page)
    lens = torch.full((B, 1), length, device="cuda")
    if case["ragged"]:
        lens[1:] = torch.randint(M, length + 1, (B - 1, 1), generator=g, device="cuda")
    pos = lens - M + torch.arange(M, device="cuda")
    first = torch.arange(table.shape[1], device="cuda") * page  # of every page
    table = torch.where(first < lens, table, -1)
    if case["left"] >= 0:
        gone = (first + page <= pos[:, :1] - case["left"]) & (first >= case["sinks"])
        table = torch.where(gone, -1, table)
    return {"case": case, "q": _normal(g, (B, M, case["H"], D), dt),
            "pos": pos.to(torch.int32).contiguous(), "table": table.to(torch.int32).contiguous(),
            "cache": _pages(g, count, case)}


# ---------------------------------------------------------------- plain form

def _slots(s, at):
    """Flat cache rows of the positions `at` [B, n]; -1 where there is none."""
    page = s["case"]["page"]
    col = (at // page).clamp(0, s["table"].shape[1] - 1)
    ids = torch.gather(s["table"].long(), 1, col)
    return torch.where((at >= 0) & (ids >= 0), ids * page + at % page, -1)


def _rows(s, name, slot, wide=torch.float32):
    """Cache rows [B, n, G, D] at the given slots, as `wide` numbers."""
    c, page = s["cache"], s["case"]["page"]
    at = slot.clamp(min=0)
    data = c[name].flatten(0, 1)[at]
    if c["k_scale"] is None:
        return data.to(wide)
    return _unpack(data, c[name + "_scale"][at // page, :, at % page], wide)


def _turn(x, cos, sin, interleaved):
    """Rotate the first 2 * cos.shape[-1] entries of every head."""
    half = cos.shape[-1]
    rot, rest = x[..., :2 * half], x[..., 2 * half:]
    if interleaved:
        a, b = rot[..., 0::2], rot[..., 1::2]
        rot = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = rot[..., :half], rot[..., half:]
        rot = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((rot, rest), -1)


def _norm_turn(x, w, cos, sin, interleaved):
    xf = x.float()
    n = xf * torch.rsqrt(xf.square().mean(-1, keepdim=True) + _EPS) * w
    return _turn(n, cos, sin, interleaved).to(x.dtype)


def _plain_append(s):
    case, c, pos = s["case"], s["cache"], s["pos"].long()
    page, live = case["page"], pos >= 0
    at = pos.clamp(min=0)
    turn = (s["cos"][at][:, :, None], s["sin"][at][:, :, None], case["interleaved"])
    q = _norm_turn(s["q"], s["wq"], *turn) * live[..., None, None]
    k = _norm_turn(s["k"], s["wk"], *turn)
    slot = _slots(s, pos)[live]
    for name, x in (("k", k[live]), ("v", s["v"][live])):
        if case["bits"] == 16:
            c[name].flatten(0, 1).index_copy_(0, slot, x)
        else:
            codes, scale = _pack(x)
            c[name].flatten(0, 1).index_copy_(0, slot, codes)
            c[name + "_scale"][slot // page, :, slot % page] = scale
    return q


def _plain_attn(s):
    case = s["case"]
    B, M, H, G, D = (case[x] for x in ("B", "M", "H", "G", "D"))
    left, sinks = case["left"], case["sinks"]
    pos = s["pos"].long()
    if left < 0:
        at = torch.arange(case["length"], device="cuda").expand(B, -1)
    else:  # the first tokens, then what the windows of a sequence's queries touch
        lo = (pos.amin(1, keepdim=True) - left).clamp(min=sinks)
        at = torch.cat((torch.arange(sinks, device="cuda").expand(B, -1),
                        lo + torch.arange(left + M, device="cuda")), 1)
    slot = _slots(s, at)
    see = (at[:, None] <= pos[:, :, None]) & (slot >= 0)[:, None]
    if left >= 0:
        see &= (at[:, None] >= pos[:, :, None] - left) | (at < sinks)[:, None]
    k, v = (_rows(s, n, slot).permute(0, 2, 1, 3) for n in ("k", "v"))
    q = s["q"].float().view(B, M, G, H // G, D).permute(0, 2, 1, 3, 4).reshape(B, G, -1, D)
    x = (q @ k.transpose(-1, -2) / math.sqrt(D)).view(B, G, M, H // G, -1)
    x = x.masked_fill_(~see[:, None, :, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    e = (x - top).exp_()
    total = e.sum(-1, keepdim=True)
    o = (e.view(B, G, -1, e.shape[-1]) @ v).view(B, G, M, H // G, D) / total
    lse = (top + total.log())[..., 0]
    return (o.permute(0, 2, 1, 3, 4).reshape(B, M, H, D).to(s["q"].dtype),
            lse.permute(0, 1, 3, 2).reshape(B, H, M))


def run(state):
    case, c = state["case"], state["cache"]
    dt = _DTYPES[case["dtype"]]
    if own:
        import nsa_block_selection_gb300 as nsa

        cache = nsa.KvCache(c["k"], c["v"], c["k_scale"], c["v_scale"])
        where = (cache, state["table"], state["pos"])
        if case["op"] == "attn":
            o, lse = nsa.paged_attn(state["q"], *where, window=(case["left"], 0),
                                    sinks=case["sinks"])
            return {"o": o, "lse": lse}
        if case["op"] == "read":
            k, v = nsa.kv_read(*where, dtype=dt)
            return {"k": k, "v": v}
        q = nsa.kv_append(state["q"], state["k"], state["v"], *where, state["wq"], state["wk"],
                          state["cos"], state["sin"], eps=_EPS, interleaved=case["interleaved"])
        if case["bits"] == 16:
            return {"q": q, "k": c["k"], "v": c["v"]}
        k, v = nsa.kv_read(*where, dtype=dt)  # the codes as the values that they stand for
        return {"q": q, "k": k, "v": v}
    if case["op"] == "attn":
        o, lse = _plain_attn(state)
        return {"o": o, "lse": lse}
    out = {}
    if case["op"] == "append":
        out["q"] = _plain_append(state)
        if case["bits"] == 16:
            return {**out, "k": c["k"], "v": c["v"]}
    slot = _slots(state, state["pos"].long())
    live = (slot >= 0)[..., None, None]
    return {**out, "k": (_rows(state, "k", slot) * live).to(dt),
            "v": (_rows(state, "v", slot) * live).to(dt)}


# ---------------------------------------------------------------- work

def _visible(case):
    """(keys that a sequence's queries touch, visible pairs of a head) of the
    whole batch, lengths halfway down the range where they are ragged."""
    B, M, n = case["B"], case["M"], case["length"]
    mean = n if B == 1 or not case["ragged"] else (n + (B - 1) * (n + M) / 2) / B
    span = mean if case["left"] < 0 else min(mean, case["left"] + M + case["sinks"])
    row = mean - (M - 1) / 2 if case["left"] < 0 else min(mean, case["left"] + 1 + case["sinks"])
    return B * span, B * M * row


def work(case):
    B, M, G, D = (case[x] for x in ("B", "M", "G", "D"))
    row = 2 * D if case["bits"] == 16 else D // 2 + 4  # bytes of a cached row
    tokens = B * M
    if case["op"] == "append":
        x = tokens * (case["H"] + G) * D
        tables = tokens * (8 + case["rot"] * 4)
        back = 0 if case["bits"] == 16 else 2 * tokens * G * (row + 2 * D)
        return {"bytes": x * 2 + tokens * (case["H"] + G) * D * 2 + 2 * tokens * G * row + tables + back,
                "flops": 10 * x}
    if case["op"] == "read":
        tokens = M if B == 1 else int(M + (B - 1) * (M + 1) / 2)
        return {"bytes": 2 * tokens * G * row + 2 * B * M * G * D * 2 + B * M * 8,
                "flops": 2 * tokens * G * D}
    keys, pairs = _visible(case)
    return {"bytes": 2 * keys * G * row + tokens * case["H"] * (4 * D + 4),
            "flops": 4 * D * case["H"] * pairs}


# ---------------------------------------------------------------- 64 bits

def _exact_turn(x, w, s):
    """Every pair of entries as a complex number: a turn is a product."""
    case = s["case"]
    half, D = case["rot"] // 2, case["D"]
    x = x.double()
    y = x / ((x * x).sum(-1, keepdim=True) / D + _EPS).sqrt() * w.double()
    one = torch.arange(half, device="cuda") * (2 if case["interleaved"] else 1)
    two = one + (1 if case["interleaved"] else half)
    unit = torch.complex(s["cos"].double(), s["sin"].double())[s["pos"].long().clamp(min=0)][:, :, None]
    z = torch.complex(y[..., one], y[..., two]) * unit
    y[..., one], y[..., two] = z.real, z.imag
    return y


def _exact_rows(s, name, b, at):
    """Rows [n, G, D] of the tokens `at` of sequence b, from their pages."""
    c, page = s["cache"], s["case"]["page"]
    ids, off = s["table"][b].long()[at // page], at % page
    data = c[name][ids, off]
    if s["case"]["bits"] == 16:
        return data.double()
    step, low = c[name + "_scale"][ids, :, off].double().unbind(-1)
    y = torch.empty(*data.shape[:-1], s["case"]["D"], dtype=torch.float64, device="cuda")
    y[..., 0::2], y[..., 1::2] = (data % 16).double(), torch.div(data, 16, rounding_mode="floor").double()
    return y * step[..., None] + low[..., None]


def _exact_append(s):
    case, page = s["case"], s["case"]["page"]
    live = s["pos"] >= 0
    out = {"q": _exact_turn(s["q"], s["wq"], s) * live[..., None, None]}
    k = _exact_turn(s["k"], s["wk"], s)
    for name, x in (("k", k), ("v", s["v"].double())):
        if case["bits"] == 4:  # what is stored is the 16-bit row's 4-bit form
            code, step, low = _quantise(x.to(_DTYPES[case["dtype"]]), torch.float64)
            out[name] = (low + step * code) * live[..., None, None]
            continue
        out[name] = s["cache"][name].double()
        for b in range(case["B"]):
            at = s["pos"][b][live[b]].long()
            out[name][s["table"][b].long()[at // page], at % page] = x[b][live[b]]
    return out


def exact(case, seed):
    s = prepare(case, seed)
    B, M, G, D = (case[x] for x in ("B", "M", "G", "D"))
    if case["op"] == "append":
        return _exact_append(s)
    if case["op"] == "read":
        out = {n: torch.zeros(B, M, G, D, dtype=torch.float64, device="cuda") for n in ("k", "v")}
        for b in range(B):
            n = int((s["pos"][b] >= 0).sum())
            for name in out:
                out[name][b, :n] = _exact_rows(s, name, b, torch.arange(n, device="cuda"))
        return out
    H, hpg = case["H"], case["H"] // G
    o = torch.zeros(B, M, H, D, dtype=torch.float64, device="cuda")
    lse = torch.full((B, H, M), -math.inf, dtype=torch.float64, device="cuda")
    for b in range(B):
        last = int(s["pos"][b, -1])
        at = torch.arange(last + 1, device="cuda")
        if case["left"] >= 0:
            at = at[(at < case["sinks"]) | (at >= int(s["pos"][b, 0]) - case["left"])]
        k, v = _exact_rows(s, "k", b, at), _exact_rows(s, "v", b, at)
        for m0 in range(0, M, 16):
            p = s["pos"][b, m0:m0 + 16].long()[:, None]
            hidden = at > p
            if case["left"] >= 0:
                hidden |= (at < p - case["left"]) & (at >= case["sinks"])
            for h in range(H):
                t = s["q"][b, m0:m0 + 16, h].double() @ k[:, h // hpg].T / math.sqrt(D)
                t[hidden] = -math.inf
                lse[b, h, m0:m0 + 16] = torch.logsumexp(t, -1)
                o[b, m0:m0 + 16, h] = torch.softmax(t, -1) @ v[:, h // hpg]
    return {"o": o, "lse": lse}
