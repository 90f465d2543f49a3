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
