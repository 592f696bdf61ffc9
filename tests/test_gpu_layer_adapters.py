"""GPU tests of the layers' adapters beside the token dimension's padding: the
real rows' bits are those of the unpadded call, whatever the padding holds."""

import pytest
import torch

import synth
from block_helpers import normal
from helpers import need_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


# decode; token counts whose bucket takes another way through the adapters
# (another number of launches; of parts that the sum over the inner width is
# added from)
@pytest.mark.parametrize("T,inner,R", [(17, 192, 16), (27, 512, 8), (145, 192, 16), (145, 512, 64), (3950, 512, 16),
                                       (3950, 512, 40)])
def test_padded_layer_with_an_adapter(T, inner, R):
    import mixture_experts_grouped_moe_amd as moe
    Tr = moe.moe_bucket_round_up(T)
    assert Tr > T
    d = synth.config3(Tr, seed=T, bias=True, device="cuda", E=8, H=64, I=inner)
    a, b = normal((8, R, inner), 2, "a", std=inner ** -0.5), normal((8, 64, R), 2, "b", std=0.3)
    scale = torch.rand(8, generator=synth.gen(2, "s")).cuda()
    weights = (d["w1"], d["s1"], d["w2"], d["s2"])
    kw = dict(b1=d["b1"], b2=d["b2"], num_tokens=T)
    x, ids, w = (d[t] for t in ("x", "ids", "topk_w"))
    plain = moe.moe_w4a16_layer(x, ids, w, *weights, **kw)
    y = moe.moe_w4a16_layer(x, ids, w, *weights, **kw, adapter=(a, b, scale))
    assert y.shape == (T, 64) and not torch.equal(y, plain)
    exact = moe.moe_w4a16_layer(x[:T].contiguous(), ids[:T].contiguous(), w[:T].contiguous(), *weights, b1=d["b1"],
                                b2=d["b2"], adapter=(a, b, scale))
    assert torch.equal(y, exact)
    for k in range(3):
        x[T:] = normal((Tr - T, 64), 30 + k, "pad", std=50.0) if k < 2 else float("nan")
        ids[T:] = torch.randint(0, 8, tuple(ids[T:].shape), generator=synth.gen(k, "i"), dtype=torch.int32).cuda()
        assert torch.equal(moe.moe_w4a16_layer(x, ids, w, *weights, **kw, pad_token_dim=True), plain)
        padded = moe.moe_w4a16_layer(x, ids, w, *weights, **kw, pad_token_dim=True, adapter=(a, b, scale))
        off = (padded.view(torch.int16) != y.view(torch.int16)).sum().item()
        assert off == 0, f"{off} of {y.numel()} elements"
