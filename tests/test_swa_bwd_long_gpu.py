"""nsa_swa_bwd where one item (128 queries of a head, or 128 keys) takes longer
than the 1 s that a single device wait is given: every wait that spans an item
has to allow for its steps.

All but the first and the last 64 rows of the long side are zeros, so every sum
over it has 128 terms that are not, and is checked against the definition
in float64.
"""

import pytest

pytestmark = pytest.mark.gpu

U = 2.0 ** -8  # bf16


def _sparse(rows, heads, seed):
    """bf16 [1, rows, heads, 64], zeros but for the first and last 64 rows, and
    those rows."""
    import torch

    x = torch.zeros(1, rows, heads, 64, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(seed)
    ends = torch.cat((torch.arange(64), torch.arange(rows - 64, rows))).cuda()
    x[:, ends] = torch.randn(1, 128, heads, 64, generator=g, device="cuda").bfloat16()
    return x, ends


def _room(gib):
    import torch

    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < gib << 30:
        pytest.skip(f"needs {gib} GiB of free device memory")


@pytest.fixture(autouse=True)
def _give_back():
    import torch

    yield
    torch.cuda.empty_cache()


def _terms(q, k, v, o, do, lse):
    """p, dS and what fp32 errors of dS are relative to, of all pairs of rows."""
    import torch

    p = torch.exp(q @ k.T / 8.0 - lse)
    delta = (do * o).sum(-1, keepdim=True)
    wide = p * (do.abs() @ v.abs().T + (do * o).abs().sum(-1, keepdim=True))
    return p, p * (do @ v.T - delta), wide


# relative errors of p: the fp32 score (64 products, under 2^-17 of |q|.|k| / 8 < 64)
# and 2^-20 beside it; of dP and delta under 2^-15 together
EP, ED = 64 * 2.0 ** -17 + 2.0 ** -20, 2.0 ** -15


def test_a_query_tile_of_four_million_steps():
    import torch

    from nsa_block_selection_gb300 import _lib, swa_bwd

    _room(120)
    H, M, N, lse = 152, 128, 2 ** 28, 4.0  # one item for each SM, uncut: 1.7 s
    k, ends = _sparse(N, 1, 1)
    g = torch.Generator(device="cuda").manual_seed(2)
    q, o, do = (torch.randn(1, M, H, 64, generator=g, device="cuda").bfloat16() for _ in range(3))
    dq, dk, dv = swa_bwd(q, k, k, o, torch.full((1, H, M), lse, device="cuda"), do)
    torch.cuda.synchronize()
    assert _lib.sync_status() == 0
    assert torch.isfinite(dq).all()
    kd = k[0, ends, 0].double()
    del k
    for h in (0, 77, 151):
        qh, oh, dh = (x[0, :, h].double() for x in (q, o, do))
        _, ds, wide = _terms(qh, kd, kd, oh, dh, lse)
        want = ds @ kd / 8.0
        bound = U * (ds.abs() @ kd.abs() / 8.0 + want.abs()) + (EP + ED) * wide @ kd.abs() / 8.0
        assert ((dq[0, :, h].double() - want).abs() <= bound).all(), h
    # a key of zeros in the middle: p = exp(-lse) for all, dV = p sum dO
    pairs = do[0].double().reshape(-1, 64)
    p = torch.exp(torch.tensor(-lse, dtype=torch.float64, device="cuda"))
    bound = (2 * U + EP + 2.0 ** -11) * p * pairs.abs().sum(0)
    assert ((dv[0, N // 2, 0].double() - p * pairs.sum(0)).abs() <= bound).all()
    assert torch.isfinite(dk[0, ends]).all() and torch.isfinite(dk[0, N // 2]).all()


def test_a_key_tile_of_three_million_steps():
    import torch

    from nsa_block_selection_gb300 import _lib, swa_bwd

    _room(70)
    M, N, lse = 3 * 2 ** 26, 152 * 128, 4.0  # one item for each SM, uncut: 1.8 s
    q, ends = _sparse(M, 1, 3)
    g = torch.Generator(device="cuda").manual_seed(4)
    k, v = (torch.randn(1, N, 1, 64, generator=g, device="cuda").bfloat16() for _ in range(2))
    dq, dk, dv = swa_bwd(q, k, v, q, torch.full((1, 1, M), lse, device="cuda"), q)
    torch.cuda.synchronize()
    assert _lib.sync_status() == 0
    qd, kd, vd = q[0, ends, 0].double(), k[0, :, 0].double(), v[0, :, 0].double()
    del q
    p, ds, wide = _terms(qd, kd, vd, qd, qd, lse)
    want = ds.T @ qd / 8.0
    bound = U * (ds.abs().T @ qd.abs() / 8.0 + want.abs()) + (EP + ED) * wide.T @ qd.abs() / 8.0
    assert ((dk[0, :, 0].double() - want).abs() <= bound).all()
    want = p.T @ qd
    bound = U * want.abs() + (U + EP + U * U) * p.T @ qd.abs()
    assert ((dv[0, :, 0].double() - want).abs() <= bound).all()
    # rows without a gradient have none
    assert (dq[0, M // 2 - 1000:M // 2 + 1000] == 0).all()
    assert torch.isfinite(dq[0, ends]).all()
