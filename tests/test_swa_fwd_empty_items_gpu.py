"""nsa_swa_fwd where a CTA's work items follow one another without keys: tiles of
128 queries past the last key's window, many to a CTA, between others that have
keys. Such an item takes no time, so a head's next O tile is ready while the
last one may still be on its way out of shared memory."""

import pytest

import oracle.swa as W

pytestmark = pytest.mark.gpu


def _problem(B, M, N, H, G, D, dtype, seed):
    import torch

    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda").to(dtype)  # noqa: E731
    return rand(B, M, H, D), rand(B, N, G, D), rand(B, N, G, D)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("H,G", [(2, 1), (8, 2), (3, 1)])
@pytest.mark.parametrize("M,N,window", [(1300, 100, (5, 5)), (2074, 2, (0, 0)), (700, 300, (3, 130))])
def test_items_with_and_without_keys(M, N, window, H, G, D):
    """A batch whose items fill the SMs several times over, against every
    sequence on its own, whose items have an SM each."""
    import torch

    from nsa_block_selection_gb300 import _lib, swa_fwd

    B = 96
    q, k, v = _problem(B, M, N, H, G, D, torch.bfloat16, 51)
    want = [swa_fwd(q[b:b + 1], k[b:b + 1], v[b:b + 1], window=window) for b in range(B)]
    o = torch.cat([x[0] for x in want])
    lse = torch.cat([x[1] for x in want])
    for _ in range(10):
        out = torch.full_like(q, float("nan"))
        got, l2 = swa_fwd(q, k, v, window=window, out=out)
        assert torch.equal(got, o) and torch.equal(l2, lse)
    torch.cuda.synchronize()
    assert _lib.sync_status() == 0
    assert (o[:, N + window[0]:] == 0).all() and torch.isneginf(lse[:, :, N + window[0]:]).all()
    n = [x[:1].double().cpu().numpy() for x in (q, k, v)]
    rows = [(0, i, g) for i in range(0, min(M, N + window[0]), 7) for g in range(G)]
    ref, _ = W.swa_rows(*n, rows, *window)
    hpg = H // G
    for (b, i, g), r in zip(rows, ref):
        err = abs(o[b, i, g * hpg:(g + 1) * hpg].double().cpu().numpy() - r).max()
        # P and O are rounded to bf16, half a step 2^-8 each, relative to |v| < 6
        assert err <= 2 * 2.0 ** -8 * 6
