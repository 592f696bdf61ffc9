"""GPU test of moe_lora over a block list that one launch does not hold."""

import pytest
import torch

from helpers import need_gpu
from test_gpu_lora import Case

pytestmark = pytest.mark.gpu


def test_list_of_more_blocks_than_one_launch_holds():
    """2^21 blocks and more, nearly all without a group; those that have one lie
    at the front, across the border between two launches and at the end."""
    need_gpu()
    import mixture_experts_grouped_moe_amd as moe
    case = Case(90, 3, 24, 136, 264, 1, 8, seed=4)
    c, h, *_ = case.run()
    ids, groups, post = case.routing
    blocks, used = (1 << 21) + 50, int(post) // 8
    at = torch.cat([torch.arange(2), (1 << 21) - 3 + torch.arange(used - 4), blocks - 2 + torch.arange(2)]).cuda()
    assert used > 8 and int(at[-3]) > 1 << 21
    long_ids = torch.full((blocks, 8), case.S, dtype=torch.int32, device="cuda")
    long_groups = torch.full((blocks,), -1, dtype=torch.int32, device="cuda")
    long_ids[at], long_groups[at] = ids.reshape(-1, 8)[:used], groups[:used]
    out = case.c.clone()
    _, h2 = moe.moe_lora(out, case.x, case.a, case.b, (long_ids.reshape(-1), long_groups, post), case.scale, keep_h=True)
    case.check(out, h2, case.c)
    on = (case.ids >= 0).cuda()
    assert torch.equal(h2[on], h[on]) and torch.equal(out[on], c[on])
