"""The page cache's bookkeeping on the GPU against a plain simulation of the
definitions in lcx.h: every integer equal, page data moved exactly."""
import random

import pytest
import torch

import ntk_rope_flashattn_b200 as lcx
from serving_plain import PlainPages

pytestmark = pytest.mark.gpu


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def word():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def make(P, ps, S, MP, H=2, D=64, layers=2, dtype=torch.bfloat16, nhd=False):
    pools = {}
    if nhd:     # [page][slot][head], with room between heads: rows, not one dense run
        for f in ("k_pages", "v_pages"):
            pools[f] = torch.zeros((layers, P, ps, H + 1, D), dtype=dtype,
                                   device="cuda")[:, :, :, :H]
    c = lcx.PagedCache(P, ps, H, D, S, MP, num_layers=layers, dtype=dtype, **pools)
    g = torch.Generator(device="cuda").manual_seed(P + ps)
    for t in (c.k_pages, c.v_pages):
        t.copy_(torch.randn(t.shape, generator=g, device="cuda").to(dtype))
    return c, PlainPages(P, ps, S, MP)


def moved(cache, before, model):
    """The pools hold `before` with the model's page copies applied."""
    for t, b in zip((cache.k_pages, cache.v_pages), before):
        want = b.clone()
        for a, d in model.copies:
            want[:, d] = b[:, a]
        assert torch.equal(t, want)


def pools(c):
    return c.k_pages.clone(), c.v_pages.clone()


@pytest.mark.parametrize("P,ps,S,MP,nhd,dtype", [
    (50, 4, 9, 14, False, torch.bfloat16), (7, 1, 5, 9, False, torch.bfloat16),
    (300, 16, 20, 40, True, torch.float32), (5000, 2, 12, 900, False, torch.bfloat16),
])
def test_random_calls_equal_the_simulation(P, ps, S, MP, nhd, dtype):
    cache, model = make(P, ps, S, MP, nhd=nhd, dtype=dtype)
    rng = random.Random(P)
    status = word()
    for step in range(60):
        op = rng.randrange(6)
        n = rng.randrange(1, S + 2)
        ids = [rng.randrange(-1, S) for _ in range(n)]
        if step % 7 == 3:
            ids[0] = S                                   # out of range
        before = pools(cache)
        model.copies = []
        if op <= 2:
            cnt = [rng.randrange(0, max(2, P * ps // (2 * S))) for _ in ids]
            want = model.extend(ids, cnt)
            assert lcx.pages_extend(cache, ints(ids), ints(cnt), status=status).tolist() == want
        elif op == 3:
            src = [rng.randrange(-1, S) for _ in ids]
            model.fork(src, ids)
            lcx.pages_fork(cache, ints(src), ints(ids), status=status)
        elif op == 4:
            model.release(ids[:2])
            lcx.pages_free(cache, ints(ids[:2]), status=status)
        else:
            model.compact()
            lcx.pages_compact(cache, status=status)
        model.equal(cache)
        moved(cache, before, model)
        assert int(status) == model.status


def test_extend_one_token_and_page_borders():
    cache, model = make(10, 4, 3, 4)
    ids = ints([2, -1, 0])
    for _ in range(9):
        assert lcx.pages_extend(cache, ids).tolist() == model.extend([2, -1, 0], [1, 1, 1])
        model.equal(cache)


def test_extend_skips_what_does_not_fit():
    cache, model = make(5, 4, 6, 4)
    status = word()
    ids, cnt = [0, 1, 2, 3, 0, 4], [8, 9, 1, 0, 1, 17]
    want = model.extend(ids, cnt)
    got = lcx.pages_extend(cache, ints(ids), ints(cnt), status=status)
    # 2 + 3 pages fit; entry 2 finds none; 3 needs none; 0 came before; 17 > 4 * 4
    assert got.tolist() == want == [0, 0, -1, 0, -1, -1]
    assert int(status) == lcx.LCX_ERR_NO_PAGES
    model.equal(cache)


@pytest.mark.parametrize("n", [1024])
def test_extend_many_entries(n):
    cache, model = make(3000, 2, 1100, 6, H=1, layers=1)
    rng = random.Random(5)
    ids = rng.sample(range(1100), n)
    cnt = [rng.randrange(0, 12) for _ in ids]
    assert lcx.pages_extend(cache, ints(ids), ints(cnt)).tolist() == model.extend(ids, cnt)
    model.equal(cache)
    lcx.pages_free(cache, ints(ids))
    model.release(ids)
    model.equal(cache)


def test_fork_same_source_twice_and_refused_targets():
    cache, model = make(40, 4, 8, 6)
    status = word()
    model.extend([0, 1, 2], [10, 8, 3])
    lcx.pages_extend(cache, ints([0, 1, 2]), ints([10, 8, 3]))
    before = pools(cache)
    # 0 twice (partial page copied twice), 1 (full pages only), onto a taken
    # sequence, twice onto one target, an empty source, a target that is a source
    src, dst = [0, 0, 1, 0, 2, 7, 3], [3, 4, 5, 1, 3, 6, 7]
    model.fork(src, dst)
    lcx.pages_fork(cache, ints(src), ints(dst), status=status)
    model.equal(cache)
    moved(cache, before, model)
    assert len(model.copies) == 2 and int(status) == lcx.LCX_ERR_INVALID_ARG
    assert cache.seq_lens.tolist()[7] == 0       # 3 was empty before the call


def test_fork_without_free_pages():
    cache, model = make(4, 4, 6, 4)
    status = word()
    for m in (model.extend([0, 1], [6, 5]), lcx.pages_extend(cache, ints([0, 1]), ints([6, 5]))):
        pass
    model.fork([0, 1], [2, 3])
    lcx.pages_fork(cache, ints([0, 1]), ints([2, 3]), status=status)
    model.equal(cache)
    assert int(status) == lcx.LCX_ERR_NO_PAGES and cache.seq_lens.tolist()[2:4] == [0, 0]


@pytest.mark.parametrize("nhd,H,D,ps,dtype", [
    (False, 3, 64, 8, torch.bfloat16), (True, 3, 128, 8, torch.float32),
    (False, 1, 64, 1, torch.bfloat16), (False, 8, 128, 64, torch.bfloat16),
])
def test_copy_pages(nhd, H, D, ps, dtype):
    cache, model = make(30, ps, 2, 2, H=H, D=D, dtype=dtype, nhd=nhd, layers=3)
    status = word()
    before, meta = pools(cache), cache.meta.clone()
    src, dst = [1, 1, 5, -1, 9, 3, 30, 20], [2, 4, 6, 7, 9, 2, 8, 5]
    lcx.pages_copy(cache, ints(src), ints(dst), status=status)
    # 9 -> 9 is left alone; 3 -> 2 repeats a target, 30 is no page, 5 is a source
    model.copies = [(1, 2), (1, 4), (5, 6)]
    moved(cache, before, model)
    assert torch.equal(cache.meta, meta) and int(status) == lcx.LCX_ERR_INVALID_ARG


def test_calls_replay_from_a_graph():
    """A beam step (drop, fork, grow) captured once and replayed follows the state."""
    cache, model = make(60, 4, 8, 8)
    model.extend([0, 1], [9, 6])
    lcx.pages_extend(cache, ints([0, 1]), ints([9, 6]))
    kids, par = ints([2, 3, 4]), ints([0, 1, 0])
    start = torch.empty(3, dtype=torch.int32, device="cuda")

    def step():
        lcx.pages_free(cache, kids)
        lcx.pages_fork(cache, par, kids)
        lcx.pages_extend(cache, kids, start=start)

    meta = cache.meta.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    cache.meta.copy_(meta)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    cache.meta.copy_(meta)
    for _ in range(3):
        graph.replay()
        model.release([2, 3, 4])
        model.fork([0, 1, 0], [2, 3, 4])
        assert start.tolist() == model.extend([2, 3, 4], [1, 1, 1])
        model.equal(cache)
