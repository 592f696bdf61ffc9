"""CPU tests of what the block binding refuses before it looks at a tensor."""

import pytest
import torch

moe = pytest.importorskip("mixture_experts_grouped_moe_amd")


@pytest.mark.parametrize("quant", ["fp8", "MXFP8", "", 1, True])
def test_unknown_quant(quant):
    with pytest.raises(ValueError, match="quant must be"):
        moe.moe_rmsnorm(torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(64), quant=quant)


@pytest.mark.parametrize("adapter", [(), (1, 2), (1, 2, None, 3), torch.zeros(3), "abc"])
def test_adapters_that_are_not_three(adapter):
    x, ids, w = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)
    m = torch.zeros(8, 64, 64)
    with pytest.raises(ValueError, match="adapter must be"):
        moe.moe_w4a16_layer(x, ids, w, m, m, m, m, adapter=adapter)
    with pytest.raises(ValueError, match="adapter must be"):
        moe.moe_relu2_layer(x, ids, w, m, m, adapter=adapter)
