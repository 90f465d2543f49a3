"""GPU tests of forms of the layer calls that the sizes in test_gpu_layer.py do not reach, with that file's
layer, 64-bit reference and tolerances."""
import pytest
import torch

import heterogeneous_adapters_sgmv_b200 as L
from tests.test_gpu_layer import Layer

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    assert torch.cuda.is_available()
    L._load()


def test_bgmv_layer_with_the_workspace_of_a_larger_batch():
    """The scaled intermediate has more parts in smaller batches; one workspace serves all."""
    big = Layer(1024, 2048, 136, (16, 40), seed=41)
    assert big.table.workspace_bytes(512) <= big.ws.numel()
    for T in (512, 130, 1):
        m = Layer(T, 2048, 136, (16, 40), seed=42, act="silu")
        ids = m.ids()
        big.ws.fill_(255)
        m.check(m.bgmv(ids, ws=big.ws), ids, "%d tokens" % T)
