"""Arguments of the paged-cache calls at the ends of what is allowed."""

import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bits", [16, 4])
def test_keys_of_one_sequence_for_a_whole_batch(bits):
    """K and V that repeat one sequence's rows, without queries."""
    import torch

    from nsa_block_selection_gb300 import kv_append, kv_cache, kv_read

    g = torch.Generator(device="cuda").manual_seed(1)
    k, v = (torch.randn((1, 40, 2, 64), generator=g, device="cuda").bfloat16() for _ in range(2))
    caches = [kv_cache(9, 16, 2, 64, bits=bits) for _ in range(2)]
    table = torch.randperm(9, generator=g, device="cuda").view(3, 3).int()
    assert kv_append(None, k.expand(3, -1, -1, -1), v.expand(3, -1, -1, -1), caches[0], table) is None
    kv_append(None, k.repeat(3, 1, 1, 1), v.repeat(3, 1, 1, 1), caches[1], table)
    pos = torch.arange(40, device="cuda", dtype=torch.int32)
    for x, y in zip(*(kv_read(c, table, pos) for c in caches)):
        assert torch.equal(x, y) and not (x == 0).all()
