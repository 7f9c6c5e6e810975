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


def test_missing_tables_and_positions_are_named():
    import torch

    from nsa_block_selection_gb300 import kv_append, kv_cache, kv_read, paged_attn

    cache = kv_cache(4, 16, 2, 64)
    table = torch.zeros((1, 4), dtype=torch.int32, device="cuda")
    pos = torch.zeros((1, 1), dtype=torch.int32, device="cuda")
    q, k = (torch.zeros((1, 1, n, 64), device="cuda").bfloat16() for n in (4, 2))
    for call in (lambda: kv_read(cache, table, None), lambda: paged_attn(q, cache, table, None),
                 lambda: kv_read(cache, table, pos[0, 0]), lambda: kv_read(cache, table, pos[:, :, None])):
        with pytest.raises(ValueError, match="positions"):
            call()
    for call in (lambda: kv_read(cache, None, pos), lambda: paged_attn(q, cache, None, pos),
                 lambda: kv_append(q, k, k, cache, None, pos), lambda: kv_read(cache, table[0], pos),
                 lambda: kv_read(cache, table[0, 0], pos), lambda: paged_attn(q, cache, table[0, 0], pos)):
        with pytest.raises(ValueError, match="page_table"):
            call()
    for x in kv_read(cache, table, pos[:, :0]):
        assert x.shape == (1, 0, 2, 64)


def test_queries_that_repeat_rows_are_refused_by_name():
    import torch

    from nsa_block_selection_gb300 import kv_cache, paged_attn

    cache = kv_cache(4, 16, 2, 64)
    table = torch.zeros((2, 4), dtype=torch.int32, device="cuda")
    pos = torch.zeros((2, 2), dtype=torch.int32, device="cuda")
    for shape in ((1, 2, 4, 64), (2, 1, 4, 64), (2, 2, 1, 64)):
        q = torch.zeros(shape, device="cuda").bfloat16().expand(2, 2, 4, 64)
        with pytest.raises(ValueError, match="repeat"):
            paged_attn(q, cache, table, pos)
    # (the stride of a dimension of one is never used)
    q = torch.zeros(256, device="cuda").bfloat16().as_strided((1, 1, 2, 64), (0, 0, 128, 1))
    assert paged_attn(q, cache, table[:1], pos[:1, :1].contiguous())[0].shape == q.shape
