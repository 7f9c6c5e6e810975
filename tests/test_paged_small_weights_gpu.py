"""Many keys that each have little of the weight beside one that has most of it.

Where p is rounded to fp16 the largest p of a row is 2^7 or more, so that a key keeps
its part down to 2^-32 of the largest: a p' below 2^-14 is off by 2^-25 at most, 2^-32
of the reference. (512 keys: one CTA's, whose warps each have a reference of their
own; so a quarter or a half of the keys are beside the one.) The bound is that of _paged.py with this in place of its 2^-25:
(2 (d + 2^-20) + u_p) sum p |v| + u |O| + n 2^-32 max |v|. bf16 has fp32's range."""

import numpy as np
import pytest

import oracle.paged as P
from _paged import E, TINY, U, dt, make_cache, np64
from _parity import poisoned

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("M", [1, 2, 20])
@pytest.mark.parametrize("down", [20, 24, 26, 28])
def test_one_key_with_most_of_the_weight(down, M, dtype):
    import torch

    from nsa_block_selection_gb300 import _lib, paged_attn

    g = torch.Generator(device="cuda").manual_seed(down + M)
    n, page, H, D = 512, 64, 8, 64
    cache = make_cache(g, n // page, page, 1, D, dtype, 16)
    cache.k.mul_(0.02)
    cache.v.mul_(10.0).add_(100.0)  # the others' values; the one key's are zeros
    q = torch.rand((1, M, H, D), generator=g, device="cuda")
    q = (q / q.sum(-1, keepdim=True) * D).to(dt(dtype))  # (entries that sum to D, nearly)
    cache.k[0, 5], cache.v[0, 5] = down * np.log(2.0) / np.sqrt(D), 0.0
    table = torch.arange(n // page, device="cuda").view(1, -1).int()
    pos = torch.arange(n - M, n, device="cuda").view(1, M).int()
    o, lse = poisoned(q.shape, q.dtype), poisoned((1, H, M), torch.float32)
    paged_attn(q, cache, table, pos, out=o, lse=lse)
    torch.cuda.synchronize()
    assert _lib.sync_status() == 0
    kk, vv = (np64(x).reshape(n, 1, D) for x in (cache.k, cache.v))
    qn = np64(q)[0]
    want, wl, mag, seen = P.attend(qn, kk, vv, np.ones(n, bool), pos.cpu().numpy()[0], -1, 0, 1 / np.sqrt(D))
    d = (D + 16) * 2 * E / np.sqrt(D) * (np.abs(qn) @ np.abs(kk).max(0)[0])  # [M, H]
    bound = (2 * (d[..., None] + 2.0 ** -20) + U[dtype]) * mag + U[dtype] * np.abs(want) + TINY[dtype]
    if dtype == "f16":
        bound += (seen * 2.0 ** -32)[:, None, None] * np.abs(vv).max()
    err = np.abs(np64(o)[0] - want)
    assert (err <= bound).all(), f"{(err / bound).max():.2f} x bound"
    assert (np.abs(np64(lse)[0] - wl) <= d.T + 2.0 ** -20 * (1 + np.abs(wl))).all()
