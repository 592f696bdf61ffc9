"""GPU tests of the number of slots that moe_lora and moe_lora_backward take
from a block list, beside buffers of more rows and of fewer."""

import pytest
import torch

from helpers import need_gpu
from test_gpu_lora import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


def _moe():
    import mixture_experts_grouped_moe_amd as moe
    return moe


def longer(t, rows):
    """t with further rows behind it, of ones."""
    return torch.cat([t, torch.ones((rows, *t.shape[1:]), dtype=t.dtype, device=t.device)])


def same(u, v):
    assert torch.equal(u.nan_to_num(1.0), v.nan_to_num(1.0))


# few slots, many (`up`, joined parts, segments of several blocks); the padding
# places hold S, a row of the longer buffers
@pytest.mark.parametrize("S,G,R,bm,div", [(20, 3, 16, 16, 1), (20, 3, 64, 16, 1), (2000, 3, 24, 64, 2), (3000, 2, 8, 16, 1)])
@pytest.mark.parametrize("more", [2, 700])
def test_rows_behind_the_slots(S, G, R, bm, div, more):
    moe = _moe()
    case = Case(S, G, R, 520, 264, div, bm, seed=S + R)
    c, h, dx, da, db = case.run()
    assert case.routing.num_slots == S
    x, big, dy, dx2 = (longer(t, more) for t in (case.x, case.c, case.dy, case.dx))
    args = x, case.a, case.b, case.routing
    out, h2 = moe.moe_lora(big, *args, scale=case.scale, row_div=div, keep_h=True)
    assert out is big and h2.shape == h.shape
    same(big[:S], c)
    assert (big[S:] == 1).all()          # left as they were
    on = (case.ids >= 0).cuda()
    assert torch.equal(h2[on], h[on])
    for k in range(2):
        da2, db2 = moe.moe_lora_backward(dy, *args, h, scale=case.scale, row_div=div, dx=dx2)
        assert torch.equal(da2, da) and torch.equal(db2, db)
        if k == 0:
            same(dx2[:S], dx)
        assert (dx2[S:] == 1).all()
    # a list of one's own, its slots said by the caller
    own = tuple(case.routing)
    again = longer(case.c, more)
    moe.moe_lora(again, x, case.a, case.b, own, scale=case.scale, row_div=div, num_slots=S)
    same(again[:S], c)
    assert (again[S:] == 1).all()
    da2, db2 = moe.moe_lora_backward(dy, x, case.a, case.b, own, h, scale=case.scale, row_div=div, num_slots=S)
    assert torch.equal(da2, da) and torch.equal(db2, db)


def test_fewer_slots_than_the_list_has():
    """Slots from num_slots, or from the rows of c, on are skipped."""
    moe = _moe()
    case = Case(60, 3, 16, 64, 48, 1, 16, seed=2, free=0.0)
    whole, h = moe.moe_lora(case.c.clone(), *case.args(), scale=case.scale, keep_h=True)
    part = moe.moe_lora(case.c.clone(), *case.args(), scale=case.scale, num_slots=37)
    assert torch.equal(part[:37], whole[:37]) and torch.equal(part[37:], case.c[37:])
    short = moe.moe_lora(case.c[:37].clone(), *case.args(), scale=case.scale)
    assert torch.equal(short, whole[:37])
    dx = case.dx.clone()
    da, db = moe.moe_lora_backward(case.dy, *case.args(), h[:37].contiguous(), scale=case.scale, dx=dx, num_slots=37)
    less = Case(60, 3, 16, 64, 48, 1, 16, seed=2, free=0.0)
    less.ids[37:] = -1
    less.check_grad(dx, da, db, h, case.dx)
    assert torch.equal(dx[37:], case.dx[37:])


def test_numbers_of_slots_that_are_refused():
    moe = _moe()
    case = Case(20, 3, 16, 64, 48, 1, 16, seed=1)
    c, dy = longer(case.c, 9), longer(case.dy, 9)
    h = torch.zeros((29, 16), device="cuda")
    for call in (lambda n: moe.moe_lora(c, longer(case.x, 9), case.a, case.b, case.routing, num_slots=n),
                 lambda n: moe.moe_lora_backward(dy, longer(case.x, 9), case.a, case.b, case.routing, h[:n], num_slots=n)):
        for n in (-1, 21, 29, 30):
            with pytest.raises(ValueError, match="num_slots"):
                call(n)
    assert torch.equal(c[20:], torch.ones_like(c[20:]))


def test_align_says_what_it_was_made_for():
    moe = _moe()
    ids = torch.zeros((9, 2), dtype=torch.int32, device="cuda")
    routing = moe.moe_align(ids, 4, 16)
    assert isinstance(routing, tuple) and routing.num_slots == 18 and len(routing) == 3
    out = tuple(torch.empty_like(t) for t in routing)
    again = moe.moe_align(ids, 4, 16, num_tokens=5, out=out)
    assert again.num_slots == 10 and all(a is b for a, b in zip(again, out))


def test_align_into_an_earlier_routing():
    """A list aligned again for fewer slots into the same Routing: its padding holds the new number."""
    moe = _moe()
    case = Case(60, 3, 16, 64, 48, 1, 16, seed=2, free=0.0)
    ids = case.ids[:, None].contiguous().cuda()
    routing = moe.moe_align(ids, 3, 16)
    assert moe.moe_align(ids, 3, 16, num_tokens=37, out=routing) is routing and routing.num_slots == 37
    c = case.c.clone()
    moe.moe_lora(c, case.x, case.a, case.b, routing, case.scale)
    want = moe.moe_lora(case.c[:37].clone(), case.x[:37], case.a, case.b, moe.moe_align(ids[:37], 3, 16), case.scale)
    # (the longer list may split K otherwise: two sums of K + R + 4 = 84 roundings of
    # magnitudes below 32 in all, 2^-12, and a half step of bf16 each)
    d = (c[:37].float() - want.float()).abs()
    assert (d <= 2.0 ** -7 * want.float().abs() + 2.0 ** -12).all()
    assert torch.equal(c[37:], case.c[37:])
