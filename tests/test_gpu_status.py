"""One device status word shared by several calls: what it holds in the end, and that an
earlier call's report does not reach into a later call's results."""
import pytest
import torch

import ntk_rope_flashattn_b200 as lcx

pytestmark = pytest.mark.gpu


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def randn(seed, *shape):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").bfloat16()


def out_of_pages(status):
    cache = lcx.PagedCache(2, 4, 1, 64, 2, 4)
    lcx.pages_extend(cache, ints([0]), ints([9]), status=status)


@pytest.mark.parametrize("first", ["pages", "timeout"])
def test_a_timeout_outlasts_other_reports(first):
    """LCX_ERR_TIMEOUT (o and lse undefined) stays in the word whatever else is reported
    before or behind it."""
    rope = lcx.RopeParams("plain", 128)
    plan = lcx.VarlenPlan([300, 40])
    q, k, v = (randn(i, 340, h, 128) for i, h in ((1, 4), (2, 2), (3, 2)))
    status = ints([0])
    calls = [lambda: out_of_pages(status),
             lambda: lcx.attn_varlen(q, k, v, plan, rope, status=status, watchdog_ms=50,
                                     _test_stall=True)]
    for c in calls if first == "pages" else calls[::-1]:
        c()
    assert int(status) == lcx.LCX_ERR_TIMEOUT
