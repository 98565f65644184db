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


@pytest.mark.parametrize("code", ["LCX_ERR_INVALID_ARG", "LCX_ERR_NO_PAGES"])
@pytest.mark.parametrize("L,Lq,splits", [(700, 700, 0), (700, 1, 0), (700, 1, 4)])
def test_attn_fwd_runs_with_another_calls_report(code, L, Lq, splits):
    """attn_fwd gives up early on a timeout only: a page call's report in the word leaves
    its results, and the word, alone."""
    rope = lcx.RopeParams("plain", 128)
    q, k, v = randn(1, 1, 8, Lq, 128), randn(2, 1, 2, L, 128), randn(3, 1, 2, L, 128)
    kw = dict(num_splits=splits) if splits else {}
    want, wl = lcx.attn_fwd(q, k, v, rope, q_offset=L - Lq, return_lse=True, **kw)
    status = ints([getattr(lcx, code)])
    out = torch.full_like(want, 7.0)
    o, lse = lcx.attn_fwd(q, k, v, rope, q_offset=L - Lq, return_lse=True, status=status, out=out,
                          **kw)
    assert torch.equal(o, want) and torch.equal(lse, wl)
    assert int(status) == getattr(lcx, code)
