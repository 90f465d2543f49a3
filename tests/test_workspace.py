"""lora_workspace_bytes, on a machine without a GPU: a record laid out like the table stands in for one
(test_layer_checks.py)."""
import ctypes

import pytest

import heterogeneous_adapters_sgmv_b200 as L
from tests.test_layer_checks import P, table

TOKENS = (list(range(0, 70)) + list(range(496, 530)) + [777, 1023, 1024, 1025, 1279, 1280, 2047, 2048, 2049, 4096, 8192,
                                                        100000, 2 ** 31 - 1])


def need(t, T):
    return L._load().lora_workspace_bytes(ctypes.addressof(t), T)


@pytest.mark.parametrize("h", [8, 1024, 2040, 2048, 4096, 14336])
@pytest.mark.parametrize("rank", [1, 16, 60, 64, 128])
def test_workspace_grows_with_the_batch(h, rank):
    """An engine keeps one workspace, sized for its largest batch, for every smaller one."""
    t = table(h=h, max_rank=rank, min_rank=rank, d_tmaps_pfA=P if rank % 8 == 0 and rank <= 64 else None)
    sizes = [need(t, T) for T in TOKENS]
    assert all(s > 0 and s % 256 == 0 for s in sizes)
    assert sizes == sorted(sizes)


def plain(T, n, ldv, tcgen05):
    """What the calls without a layer need: the intermediate (fp32, or hi and lo of 64 columns), sorted
    tokens, segment bounds and adapters, and one block of counters, each rounded up to 256 bytes."""
    up = lambda b: (b + 255) // 256 * 256
    return (up(max(T * ldv * 4, T * 256 if tcgen05 else 0)) + up(4 * T) + up(4 * (n + 1)) + up(4 * n) + 256)


@pytest.mark.parametrize("T", [0, 1, 64, 300, 512, 513, 1024, 2048, 5000])
def test_workspace_grows_only_where_the_layer_call_needs_it(T):
    """fp32 tables have no layer call; large batches keep its intermediate in one part, where that of the other
    calls lies."""
    assert need(table(h=4096, dtype=L.LORA_F32, d_tmaps_pfA=None), T) == plain(T, 4, 16, False)
    for h, rank, tcgen05 in ((4096, 16, True), (4096, 64, True), (4096, 128, False), (256, 128, False)):
        got = need(table(h=h, max_rank=rank, d_tmaps_pfA=P if tcgen05 else None), T)
        rows = T if h < 2048 else max(T, 4 * min(T, 512))
        assert got == max(plain(T, 4, rank, tcgen05), (rows * rank * 4 + 255) // 256 * 256)
