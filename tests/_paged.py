"""Shared helpers of the paged-cache tests: problems, the cache's rows as the
oracle sees them, and the bounds of the attention's error.

Bounds of paged_attn, per element, from the unit roundoff u of the stored type,
u_p of p's (2^-8 bf16, 2^-11 fp16; fp16 over a 4-bit cache) and e = 2^-24:

* a score is a sum of D products in fp32 (taken as D + 16 roundings of 2 e of
  the largest partial sum: the tensor cores may truncate), so it is off by at
  most d = (D + 16) 2 e scale |q|.|k|; over 4 bits |k| is 15 step + |low| an
  entry. p = e^(x - r) is then off by d + 2^-20 (ex2 and the scaling) of
  itself, and O, numerator and sum, by 2 (d + 2^-20) sum p |v|;
* p rounded for the product: u_p sum p |v|; over 4 bits only step code is under
  it, at most 16 / 15 of |v| + |low| + ...: 2 u_p (sum p |v| + sum p |low|);
  fp16 p below 2^-14 is off by 2^-25 of the reference each, and l is at least 1
  (over 4 bits at least 1 / the largest step): n 2^-25 max |v| (16 step);
* the store: u |O|;
* LSE: d + 2^-20 (1 + |LSE|).
"""

import numpy as np

import oracle.paged as P

E = 2.0 ** -24
U = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}
TINY = {"bf16": 2.0 ** -134, "f16": 2.0 ** -25}


def dt(name):
    import torch

    return {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}[name]


def np64(t):
    return t.detach().double().cpu().numpy()


def pack(x):
    """The 4-bit form of x (numpy [..., D]) as torch tensors on the GPU:
    codes uint8 [..., D/2], scales bf16 [..., 2]."""
    import torch

    code, step, low = P.quantise(x)
    code = code.astype(np.uint8)
    return (torch.from_numpy(code[..., 0::2] | (code[..., 1::2] << 4)).cuda(),
            torch.from_numpy(np.concatenate([step, low], -1)).cuda().bfloat16())


def make_cache(g, pages, page, G, D, dtype, bits, layout="plain", fill=None, std=1.0):
    """A cache that holds random rows (or `fill`) everywhere."""
    import torch

    from nsa_block_selection_gb300 import KvCache

    def rows():
        x = torch.randn((pages, page, G, D), generator=g, device="cuda") * std
        return x.to(dt(dtype)) if fill is None else torch.full_like(x, fill).to(dt(dtype))

    k, v = rows(), rows()
    if bits == 4:
        (kc, ks), (vc, vs) = pack(np64(k)), pack(np64(v))
        return KvCache(kc, vc, ks.transpose(1, 2).contiguous(), vs.transpose(1, 2).contiguous())
    if layout == "joint":  # one tensor that holds both
        both = torch.stack((k, v), 1)
        k, v = both[:, 0], both[:, 1]
    elif layout == "heads":  # a page's rows of a head one after the other
        k, v = (x.transpose(1, 2).contiguous().transpose(1, 2) for x in (k, v))
    return KvCache(k, v)


def rows_of(cache, name):
    """Every row of the cache as float64 [pages, page_size, G, D]; over 4 bits
    also |low| and step of each."""
    x = getattr(cache, name)
    if cache.bits == 16:
        return np64(x), None, None
    c = x.cpu().numpy()
    s = np64(getattr(cache, name + "_scale")).transpose(0, 2, 1, 3)
    codes = np.stack([c & 15, c >> 4], -1).reshape(*c.shape[:-1], -1)
    return s[..., 1:] + s[..., :1] * codes, np.abs(s[..., 1:]), s[..., :1]


def sequence_rows(all_rows, table_row, page, N):
    """[N, G, D] of a sequence's positions, and which of them it has."""
    pages = all_rows.shape[0]
    out = np.zeros((N,) + all_rows.shape[2:])
    present = np.zeros(N, bool)
    for j in range(N):
        at = P.place(table_row, j, page, pages)
        if at is not None:
            present[j] = True
            out[j] = all_rows[at]
    return out, present


def check_attn(q, cache, table, pos, left, sinks, scale, o, lse, dtype):
    """O and LSE against the oracle, every element."""
    qn, tn = np64(q), table.cpu().numpy()
    B, M, H, D = qn.shape
    pn = np.broadcast_to(pos.cpu().numpy(), (B, M))
    sc = scale if scale else 1 / np.sqrt(D)
    on, ln = np64(o), None if lse is None else np64(lse)
    page, hpg = cache.page_size, H // cache.kv_heads
    k, klow, kstep = rows_of(cache, "k")
    v, vlow, vstep = rows_of(cache, "v")
    u, up = U[dtype], U["f16" if cache.bits == 4 else dtype]
    for b in range(B):
        N = max(0, min(int(pn[b].max()) + 1, tn.shape[1] * page))
        kb, present = sequence_rows(k, tn[b], page, N)
        vb, _ = sequence_rows(v, tn[b], page, N)
        want, wl, mag, seen = P.attend(qn[b], kb, vb, present, pn[b], left, sinks, sc)
        size, vtop = np.abs(kb), np.abs(vb).max(initial=0.0)
        extra = 0.0
        if cache.bits == 4:
            low = sequence_rows(np.broadcast_to(klow, k.shape), tn[b], page, N)[0]
            step = sequence_rows(np.broadcast_to(kstep, k.shape), tn[b], page, N)[0]
            size = low + 15 * step
            low = sequence_rows(np.broadcast_to(vlow, v.shape), tn[b], page, N)[0]
            step = sequence_rows(np.broadcast_to(vstep, v.shape), tn[b], page, N)[0]
            vtop = 16 * step.max(initial=0.0)
            _, _, extra, _ = P.attend(qn[b], kb, low, present, pn[b], left, sinks, sc)
            mag = mag + extra
        for h in range(H):
            big = size[present, h // hpg].max(0, initial=0.0) if N > 0 else np.zeros(D)
            d = (D + 16) * 2 * E * sc * (np.abs(qn[b, :, h]) @ big)  # [M]
            bound = (2 * (d[:, None] + 2.0 ** -20) + (2 if cache.bits == 4 else 1) * up) * mag[:, h] \
                + u * np.abs(want[:, h]) + TINY[dtype]
            if dtype == "f16" or cache.bits == 4:
                bound = bound + (seen * 2.0 ** -25 * vtop)[:, None]
            empty = seen == 0
            bound[empty] = 0
            err = np.abs(on[b, :, h] - want[:, h])
            assert np.isfinite(on[b, :, h]).all(), f"O of sequence {b}, head {h}: not finite"
            assert (err <= bound).all(), (f"O of sequence {b}, head {h}: "
                                          f"{(err / np.maximum(bound, 1e-300)).max():.2f} x bound")
            if ln is None:
                continue
            assert (ln[b, h][empty] == -np.inf).all(), "LSE of a query without keys"
            le = np.abs(ln[b, h][~empty] - wl[h][~empty])
            lb = (d + 2.0 ** -20 * (1 + np.abs(wl[h])))[~empty]
            assert (le <= lb).all(), (f"LSE of sequence {b}, head {h}: "
                                      f"{(le / np.maximum(lb, 1e-300)).max():.2f} x bound")
