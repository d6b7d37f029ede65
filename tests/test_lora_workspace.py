"""gwa_lora_workspace_bytes, without a GPU."""
import pytest


@pytest.fixture(scope="module")
def size():
    import group_wise_affine_gb300 as gwa
    gwa.build()
    lib = gwa.load()

    def bytes_of(M, K=5120, sections=1, rank=64):
        n = lib.gwa_lora_workspace_bytes(gwa._Lora(a=1 << 20, b=1 << 20, N=sections * 64, K=K, sections=sections, rank=rank,
                                                   adapters=3), M)
        assert n and not gwa.last_error()
        return n
    return bytes_of


@pytest.mark.parametrize("K,sections,rank", [(32, 1, 8), (5120, 1, 64), (13824, 2, 24), (1 << 20, 8, 128)])
def test_more_tokens_never_need_less(size, K, sections, rank):
    """A workspace made for the largest step serves every smaller one."""
    need = [size(M, K, sections, rank) for M in range(1, 20000)]
    assert all(a <= b for a, b in zip(need, need[1:]))


def test_more_of_anything_never_needs_less(size):
    for M in (1, 256, 257, 5000, 8192, 8193, 50000):
        assert size(M, K=5120) <= size(M, K=5152) <= size(M, K=40960)
        assert size(M, sections=1) < size(M, sections=2) < size(M, sections=8)
        ranks = [size(M, rank=r) for r in range(8, 129, 8)]
        assert all(a < b for a, b in zip(ranks, ranks[1:]))
