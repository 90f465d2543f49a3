"""The largest batches of the layer calls, on a machine without a GPU (the stand-in table of
test_layer_checks.py)."""
import pytest
import torch

import heterogeneous_adapters_sgmv_b200 as L
from tests.test_layer_checks import OK, bgmv, sgmv, table

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="the stand-in table must not reach a device")


@pytest.mark.parametrize("call", [bgmv, sgmv])
def test_layer_batches_end_where_the_row_arithmetic_does(call):
    """Rows are counted in 32 bits, tiles and windows of them rounded up: from 2^31 - 256 on that would wrap, in
    the shrink's loop over windows without end."""
    far = dict(t=table(h=8, o=8), x=1 << 40, ldx=8, ldw=8, y=1 << 44, ldy=8, ws=1 << 46, ws_bytes=1 << 45)
    assert call(T=L.LORA_MAX_LAYER_TOKENS, **far) == OK
    for T in (L.LORA_MAX_LAYER_TOKENS + 1, 2 ** 31 - 256, 2 ** 31 - 1):
        assert call(T=T, **far) == L.LORA_ERR_UNSUPPORTED


def test_no_ids_no_more_tokens():
    far = dict(t=table(h=8, o=8), ids=None, x=1 << 40, ldx=8, ldw=8, y=1 << 44, ldy=8)
    assert bgmv(T=2 ** 31 - 1, **far) == L.LORA_ERR_UNSUPPORTED and bgmv(T=1 << 30, **far) == OK
