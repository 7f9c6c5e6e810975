"""Timed cases of the attention layer's training and decoding operators.

Two families, which a layer runs next to one another:

* ``norm_rope`` / ``norm_rope_bwd``: the RMS norm of every query and key head
  and the position rotation in one pass over the projections' outputs, and
  its gradients (of the heads and of the two norm weights);
* ``swa_bwd``: dQ, dK and dV of the sliding-window (or dense) grouped-query
  attention forward, from its inputs, O, LSE and dO.

``run`` computes a case in its plain form (elementary torch operations in
fp32, rounded once at the end), or, with ``own``, through this package's
operators. ``exact`` computes it from the definition in fp64.
"""

import math

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_EPS = 1e-6
_BASE = 10000.0


# ---------------------------------------------------------------- cases

def _norm_rope(name, B, M, H, G, D, dtype, rot, interleaved, fused, pad, grad=None, first=0):
    """``fused``: q and k are slices of one [B, M, H + 2G, D] projection;
    ``pad``: the batch's shorter sequences end in padding tokens;
    ``first``: position of the first token; ``grad``: type of the incoming
    gradients (None: the forward)."""
    case = {"op": "norm_rope" if grad is None else "norm_rope_bwd", "B": B, "M": M, "H": H, "G": G,
            "D": D, "dtype": dtype, "rot": rot, "interleaved": interleaved, "fused": fused,
            "pad": pad, "first": first}
    if grad is not None:
        case["grad"] = grad
    if name:
        case["name"] = name
    return case


def _swa_bwd(name, B, M, N, H, G, D, left, right, dtype):
    case = {"op": "swa_bwd", "B": B, "M": M, "N": N, "H": H, "G": G, "D": D, "left": left,
            "right": right, "dtype": dtype}
    if name:
        case["name"] = name
    return case


def listed():
    return [
        # one sequence decoding one token far into its context: latency
        _norm_rope("norm_rope_token", 1, 1, 64, 8, 128, "bf16", 128, False, True, False, first=65535),
        # a decoding batch, each sequence at a position of its own
        _norm_rope("norm_rope_decode", 48, 1, 32, 4, 128, "bf16", 128, False, True, False, first=8191),
        # a small padded batch: odd length, half of each head rotated, pairs side by side
        _norm_rope("norm_rope_padded", 3, 777, 16, 2, 64, "f16", 32, True, False, True),
        # the prefill of a long sequence
        _norm_rope("norm_rope_64k", 1, 65536, 64, 8, 128, "bf16", 128, False, True, False),
        # a short training sequence with small heads
        _norm_rope("norm_rope_bwd_short", 1, 700, 8, 2, 64, "f16", 64, False, False, False, grad="f16"),
        # training behind the selection attention, whose gradients are fp32
        _norm_rope("norm_rope_bwd_f32", 2, 4095, 32, 4, 128, "bf16", 64, False, True, True, grad="f32"),
        # long-context training behind the sliding-window attention
        _norm_rope("norm_rope_bwd_32k", 1, 32768, 64, 8, 128, "bf16", 128, False, True, False, grad="bf16"),
        # a single short sequence, one KV head: latency
        _swa_bwd("swa_bwd_short", 1, 130, 130, 4, 1, 64, 64, 0, "bf16"),
        # an ordinary small batch of odd length
        _swa_bwd("swa_bwd_1000", 2, 1000, 1000, 8, 2, 128, 256, 0, "f16"),
        # bidirectional, other queries than keys, small heads
        _swa_bwd("swa_bwd_dense_d64", 2, 1500, 2048, 16, 16, 64, -1, -1, "bf16"),
        # the sliding-window branch of a native-sparse layer at its usual window
        _swa_bwd("swa_bwd_8k_w512", 1, 8192, 8192, 64, 8, 128, 512, 0, "bf16"),
        # long-context training with a wide window
        _swa_bwd("swa_bwd_16k_w4096", 1, 16384, 16384, 64, 8, 128, 4096, 0, "bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_rope", "norm_rope_bwd", "swa_bwd"])
    dtype = rng.choice(["bf16", "bf16", "f16"])
    D = rng.choice([64, 128])
    G = rng.choice([1, 2, 4, 8])
    H = G * rng.choice([1, 2, 3, 4, 8])
    if op != "swa_bwd":
        fwd = op == "norm_rope"
        rows = _log(rng, 1, 65536) if fwd else _log(rng, 64, 32768)  # tokens in all
        B = rng.randint(1, 48) if fwd and rows < 64 else rng.randint(1, 3)
        M = max(1, rows // B)
        return _norm_rope(None, B, M, H, G, D, dtype, rng.choice([D, D, D // 2]),
                          rng.random() < 0.3, rng.random() < 0.7, M > 1 and rng.random() < 0.3,
                          grad=None if fwd else rng.choice([dtype, "f32"]),
                          first=rng.choice([0, rng.randint(0, 65000)]))
    left, right = rng.choice([(_log(rng, 16, 2048), 0), (_log(rng, 16, 2048), 0), (-1, 0), (-1, -1),
                              (rng.randint(0, 300), rng.randint(0, 300))])
    M = _log(rng, 65, 8192) if left >= 0 else _log(rng, 65, 4096)
    B = rng.randint(1, 2) if M < 4096 else 1
    N = M if rng.random() < 0.8 else max(1, int(M * rng.uniform(0.7, 1.4)))
    return _swa_bwd(None, B, M, N, H, G, D, left, right, dtype)


# ---------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _normal(g, shape, dtype, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def _window(case, rows, keys):
    """Which of `keys` each query of `rows` sees."""
    i, j = rows[:, None], keys[None, :]
    see = torch.ones(rows.numel(), keys.numel(), dtype=torch.bool, device=rows.device)
    if case["left"] >= 0:
        see &= j >= i - case["left"]
    if case["right"] >= 0:
        see &= j <= i + case["right"]
    return see


def _span(case, i0, i1):
    """The keys that the queries i0 .. i1 - 1 can see, as a half-open range."""
    lo = 0 if case["left"] < 0 else min(case["N"], max(0, i0 - case["left"]))
    hi = case["N"] if case["right"] < 0 else max(lo, min(case["N"], i1 + case["right"]))
    return lo, hi


def _block(case):
    """Queries at a time: no more than a window's keys (so that few entries
    of a score matrix are hidden ones), under 2^29 entries a matrix."""
    per = case["B"] * case["H"]
    wide = case["M"]
    if case["left"] >= 0 and case["right"] >= 0:
        wide = max(512, case["left"] + case["right"])
    for rows in (case["M"], 4096, 2048, 1024, 512, 256):
        if rows <= min(case["M"], wide):
            lo, hi = _span(case, case["M"] - rows, case["M"])
            if per * rows * max(1, hi - lo) <= 2 ** 29:
                return rows
    return 256


def _heads(x, G):
    """[B, M, H, D] as fp32 [B, G, (H / G) M, D]: the query heads of a KV head
    one after the other, so that one product serves them all."""
    B, M, H, D = x.shape
    return x.float().view(B, M, G, H // G, D).permute(0, 2, 3, 1, 4).reshape(B, G, H // G * M, D)


def _forward(case, q, k, v):
    """O (rounded once) and LSE, as the layer's forward left them."""
    B, M, H, G, D = (case[x] for x in ("B", "M", "H", "G", "D"))
    hpg, step = H // G, _block(case)
    out, lse = torch.zeros_like(q), torch.full((B, H, M), -math.inf, device="cuda")
    kf, vf = k.float().permute(0, 2, 1, 3), v.float().permute(0, 2, 1, 3)
    for i0 in range(0, M, step):
        i1 = min(M, i0 + step)
        lo, hi = _span(case, i0, i1)
        if hi == lo:
            continue
        see = _window(case, torch.arange(i0, i1, device="cuda"), torch.arange(lo, hi, device="cuda"))
        s = _heads(q[:, i0:i1], G) @ kf[:, :, lo:hi].transpose(-1, -2)
        s = (s / math.sqrt(D)).view(B, G, hpg, i1 - i0, hi - lo).masked_fill_(~see, -math.inf)
        m = s.amax(-1, keepdim=True).clamp_(min=-1e30)
        e = (s - m).exp_()
        total = e.sum(-1, keepdim=True)
        o = (e.view(B, G, -1, hi - lo) @ vf[:, :, lo:hi]).view(B, G, hpg, i1 - i0, D)
        o = o / total.clamp(min=1e-30)
        out[:, i0:i1] = o.permute(0, 3, 1, 2, 4).reshape(B, i1 - i0, H, D).to(q.dtype)
        lse[:, :, i0:i1] = (m + total.log())[..., 0].view(B, H, i1 - i0)
    return out, lse


def prepare(case, seed):
    g = _gen(seed)
    B, M, H, G, D = (case[x] for x in ("B", "M", "H", "G", "D"))
    dt = _DTYPES[case["dtype"]]
    if case["op"] == "swa_bwd":
        q = _normal(g, (B, M, H, D), dt)
        k, v = (_normal(g, (B, case["N"], G, D), dt) for _ in range(2))
        o, lse = _forward(case, q, k, v)
        return {"case": case, "q": q, "k": k, "v": v, "o": o, "lse": lse,
                "do": _normal(g, (B, M, H, D), dt, 0.1)}
    if case["fused"]:  # one projection's output; the values' slice is not this operator's
        x = _normal(g, (B, M, H + 2 * G, D), dt, 1.5)
        q, k = x[:, :, :H], x[:, :, H:H + G]
    else:
        q, k = _normal(g, (B, M, H, D), dt, 1.5), _normal(g, (B, M, G, D), dt, 1.5)
    wq, wk = (_normal(g, (D,), torch.float32, 0.2) + 1.0 for _ in range(2))
    length = case["first"] + M
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
    state = {"case": case, "q": q, "k": k, "wq": wq, "wk": wk, "pos": pos.to(torch.int32).contiguous(),
             "cos": ang.cos().float(), "sin": ang.sin().float()}
    if case["op"] == "norm_rope_bwd":
        gt = _DTYPES[case["grad"]]
        state["dq"], state["dk"] = _normal(g, (B, M, H, D), gt, 0.1), _normal(g, (B, M, G, D), gt, 0.1)
    return state


# ---------------------------------------------------------------- plain form

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


def _angles(s):
    at = s["pos"].clamp(min=0).long()
    return s["cos"][at][:, :, None], s["sin"][at][:, :, None], (s["pos"] >= 0)[:, :, None, None]


def _norm_turn(x, w, cos, sin, live, interleaved):
    xf = x.float()
    n = xf * torch.rsqrt(xf.square().mean(-1, keepdim=True) + _EPS) * w
    return (_turn(n, cos, sin, interleaved) * live).to(x.dtype)


def _norm_turn_bwd(x, w, dy, cos, sin, live, interleaved):
    xf, g = x.float(), _turn(dy.float() * live, cos, -sin, interleaved)
    r = torch.rsqrt(xf.square().mean(-1, keepdim=True) + _EPS)
    xhat, gw = xf * r, g * w
    dx = r * (gw - xhat * (gw * xhat).mean(-1, keepdim=True))
    return dx.to(x.dtype), (g * xhat).sum((0, 1, 2), dtype=torch.float64).float()


def _plain_swa_bwd(s):
    case = s["case"]
    B, M, H, G, D = (case[x] for x in ("B", "M", "H", "G", "D"))
    hpg, step, scale = H // G, _block(case), 1.0 / math.sqrt(D)
    kf, vf = s["k"].float().permute(0, 2, 1, 3), s["v"].float().permute(0, 2, 1, 3)
    dk, dv, dq = torch.zeros_like(kf), torch.zeros_like(vf), torch.zeros_like(s["q"])
    for i0 in range(0, M, step):
        i1 = min(M, i0 + step)
        lo, hi = _span(case, i0, i1)
        if hi == lo:
            continue
        see = _window(case, torch.arange(i0, i1, device="cuda"), torch.arange(lo, hi, device="cuda"))
        q, do, o = (_heads(s[x][:, i0:i1], G) for x in ("q", "do", "o"))
        lse = s["lse"][:, :, i0:i1].reshape(B, G, hpg, i1 - i0, 1)
        p = (q @ kf[:, :, lo:hi].transpose(-1, -2)).mul_(scale).view(B, G, hpg, i1 - i0, hi - lo)
        p = p.sub_(lse).exp_().masked_fill_(~see, 0.0).view(B, G, -1, hi - lo)
        dv[:, :, lo:hi] += p.transpose(-1, -2) @ do
        ds = (do @ vf[:, :, lo:hi].transpose(-1, -2)).sub_((do * o).sum(-1, keepdim=True)).mul_(p)
        ds = ds.mul_(scale)
        dk[:, :, lo:hi] += ds.transpose(-1, -2) @ q
        d = (ds @ kf[:, :, lo:hi]).view(B, G, hpg, i1 - i0, D)
        dq[:, i0:i1] = d.permute(0, 3, 1, 2, 4).reshape(B, i1 - i0, H, D).to(dq.dtype)
    dt = s["q"].dtype
    return dq, dk.permute(0, 2, 1, 3).to(dt).contiguous(), dv.permute(0, 2, 1, 3).to(dt).contiguous()


def run(state):
    case = state["case"]
    if own:
        import nsa_block_selection_gb300 as nsa

        if case["op"] == "swa_bwd":
            dq, dk, dv = nsa.swa_bwd(state["q"], state["k"], state["v"], state["o"], state["lse"],
                                     state["do"], window=(case["left"], case["right"]))
            return {"dq": dq, "dk": dk, "dv": dv}
        rope = {"positions": state["pos"], "eps": _EPS, "interleaved": case["interleaved"]}
        if case["op"] == "norm_rope":
            q, k = nsa.qk_norm_rope(state["q"], state["k"], state["wq"], state["wk"], state["cos"],
                                    state["sin"], **rope)
            return {"q": q, "k": k}
        dq, dk, dwq, dwk = nsa.qk_norm_rope_bwd(state["q"], state["k"], state["dq"], state["dk"],
                                                state["wq"], state["wk"], state["cos"],
                                                state["sin"], **rope)
        return {"dq": dq, "dk": dk, "dwq": dwq, "dwk": dwk}
    if case["op"] == "swa_bwd":
        dq, dk, dv = _plain_swa_bwd(state)
        return {"dq": dq, "dk": dk, "dv": dv}
    turn = (*_angles(state), case["interleaved"])
    if case["op"] == "norm_rope":
        return {"q": _norm_turn(state["q"], state["wq"], *turn),
                "k": _norm_turn(state["k"], state["wk"], *turn)}
    dq, dwq = _norm_turn_bwd(state["q"], state["wq"], state["dq"], *turn)
    dk, dwk = _norm_turn_bwd(state["k"], state["wk"], state["dk"], *turn)
    return {"dq": dq, "dk": dk, "dwq": dwq, "dwk": dwk}


# ---------------------------------------------------------------- work

def _pairs(case):
    """Visible (query, key) pairs of one head."""
    M, N, left, right = case["M"], case["N"], case["left"], case["right"]
    i = torch.arange(M)
    lo = torch.zeros_like(i) if left < 0 else (i - left).clamp(min=0)
    hi = torch.full_like(i, N - 1) if right < 0 else (i + right).clamp(max=N - 1)
    return int((hi - lo + 1).clamp(min=0).sum())


def work(case):
    B, M, H, G, D = (case[x] for x in ("B", "M", "H", "G", "D"))
    if case["op"] == "swa_bwd":
        # Q, O, dO read and dQ written; K, V read and dK, dV written; LSE.
        # Five products of 2 D operations for every visible pair.
        return {"bytes": B * (4 * M * H * D * 2 + 4 * case["N"] * G * D * 2 + M * H * 4),
                "flops": 10 * D * B * H * _pairs(case)}
    x = B * M * (H + G) * D
    tables = B * M * (4 + case["rot"] * 4) if B * M < case["first"] + M else \
        B * M * 4 + (case["first"] + M) * case["rot"] * 4
    if case["op"] == "norm_rope":
        return {"bytes": 2 * x * 2 + tables + 2 * D * 4, "flops": 10 * x}
    return {"bytes": x * (2 + 2 + (4 if case["grad"] == "f32" else 2)) + tables + 4 * D * 4,
            "flops": 20 * x}


# ---------------------------------------------------------------- 64 bits

def _exact_rope(state):
    """Every pair of entries as a complex number: a turn is a product."""
    case = state["case"]
    half, D = case["rot"] // 2, case["D"]
    first = torch.arange(half, device="cuda") * (2 if case["interleaved"] else 1)
    second = first + (1 if case["interleaved"] else half)
    pos = state["pos"].long()
    unit = torch.complex(state["cos"].double(), state["sin"].double())[pos.clamp(min=0)].unsqueeze(2)
    live = (pos >= 0).double()[..., None, None]

    def turned(x, back):
        z = torch.complex(x[..., first], x[..., second]) * (unit.conj() if back else unit)
        y = x.clone()
        y[..., first], y[..., second] = z.real, z.imag
        return y * live

    res = {}
    for n in ("q", "k"):
        x, w = state[n].double(), state["w" + n].double()
        rms = ((x * x).sum(-1, keepdim=True) / D + _EPS).sqrt()
        if case["op"] == "norm_rope":
            res[n] = turned(x / rms * w, False)
            continue
        g = turned(state["d" + n].double(), True)
        u = x / rms
        res["dw" + n] = torch.einsum("bmhd,bmhd->d", g, u)
        g = g * w
        res["d" + n] = (g - u * torch.einsum("bmhd,bmhd->bmh", g, u)[..., None] / D) / rms
    return res


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] != "swa_bwd":
        return _exact_rope(s)
    B, M, N, H, G, D = (case[x] for x in ("B", "M", "N", "H", "G", "D"))
    if 10 * D * B * H * _pairs(case) > 6e12:
        return None
    hpg, scale = H // G, 1.0 / math.sqrt(D)
    dq = torch.zeros(B, M, H, D, dtype=torch.float64, device="cuda")
    dk, dv = (torch.zeros(B, N, G, D, dtype=torch.float64, device="cuda") for _ in range(2))
    rows = 512
    for b in range(B):
        for g in range(G):
            k, v = s["k"][b, :, g].double(), s["v"][b, :, g].double()
            for h in range(g * hpg, (g + 1) * hpg):
                for i0 in range(0, M, rows):
                    i1 = min(M, i0 + rows)
                    lo, hi = _span(case, i0, i1)
                    if lo == hi:
                        continue
                    q, do, o = (s[x][b, i0:i1, h].double() for x in ("q", "do", "o"))
                    i = torch.arange(i0, i1, device="cuda")[:, None]
                    j = torch.arange(lo, hi, device="cuda")[None]
                    hidden = (j < i - case["left"]) if case["left"] >= 0 else (j < 0)
                    if case["right"] >= 0:
                        hidden = hidden | (j > i + case["right"])
                    t = torch.einsum("id,jd->ij", q, k[lo:hi]) * scale
                    p = torch.exp(t - s["lse"][b, h, i0:i1].double()[:, None])
                    p = torch.where(hidden, torch.zeros_like(p), p)
                    dp = torch.einsum("id,jd->ij", do, v[lo:hi])
                    ds = p * (dp - torch.einsum("id,id->i", do, o)[:, None])
                    dq[b, i0:i1, h] = ds @ k[lo:hi] * scale
                    dk[b, lo:hi, g] += ds.T @ q * scale
                    dv[b, lo:hi, g] += p.T @ do
    return {"dq": dq, "dk": dk, "dv": dv}
