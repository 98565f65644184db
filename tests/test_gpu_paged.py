"""paged_append and paged_decode on the GPU against their plain 64-bit forms
(bounds: serving_plain)."""
import dataclasses
import random

import pytest
import torch

import ntk_rope_flashattn_b200 as lcx
from serving_plain import U_OUT, attend, check, rotate

pytestmark = pytest.mark.gpu


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def word():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def randn(seed, *shape, dtype=torch.bfloat16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def cache_of(lens, ps=16, H=2, D=128, dtype=torch.bfloat16, layers=1, extra=3, seed=0, nhd=False,
             fill=float("nan")):
    """A cache whose pools hold NaN wherever no token is, sequences of these lengths
    in shuffled pages filled with N(0, 1) keys and values."""
    mp = max(max(-(-x // ps) for x in lens), 1) + 1
    P = sum(-(-x // ps) for x in lens) + extra
    shape = (layers, P, ps, H, D)
    kw = {}
    for f in ("k_pages", "v_pages"):
        t = torch.full(shape if nhd else (layers, P, H, ps, D), fill, dtype=dtype, device="cuda")
        kw[f] = t if nhd else t.transpose(2, 3)
    c = lcx.PagedCache(P, ps, H, D, len(lens), mp, num_layers=layers, dtype=dtype, **kw)
    order = list(range(P))
    random.Random(seed).shuffle(order)
    c.free_pages.copy_(ints(order))
    lcx.pages_extend(c, ints(list(range(len(lens)))), ints(lens))
    rows = []
    for s, n in enumerate(lens):
        k, v = randn(seed + 2 * s, n, H, D, dtype=dtype), randn(seed + 2 * s + 1, n, H, D, dtype=dtype)
        pos = torch.arange(n, device="cuda")
        pg, sl = c.block_table[s].long()[pos // ps], pos % ps
        for x in range(layers):
            c.k_pages[x, pg, sl] = k
            c.v_pages[x, pg, sl] = v
        rows.append((k.double().cpu(), v.double().cpu()))
    return c, rows


def plain_decode(q, rows, lens, ids, rope, window=0, sinks=0, scale=None, prerotated=False):
    q = q.double().cpu()
    scale = q.shape[-1] ** -0.5 if scale is None else scale
    parts = []
    for e, s in enumerate(ids):
        n = lens[s] if s >= 0 else 0
        k, v = (x[:n] for x in rows[s]) if s >= 0 else (torch.zeros(0, 1, q.shape[-1]).double(),) * 2
        if s < 0:
            k = v = torch.zeros(0, rows[0][0].shape[1], q.shape[-1]).double()
        pos = torch.tensor([n - 1])
        qe = q[e:e + 1] if prerotated else rotate(q[e:e + 1], pos, rope)
        parts.append(attend(qe, k, v, pos, True, window, sinks, scale))
    return (torch.cat([p[0] for p in parts]), torch.cat([p[1] for p in parts], 1).T,
            torch.cat([p[2] for p in parts]), torch.cat([p[3] for p in parts], 1).T)


def arithmetic(dtype, G, n):
    """(u_s, u_p) of paged_decode for G query heads per kv head and n keys.  fp32
    sums of D = 128 products and of n weights, cut instead of rounded by the tensor
    core (2^-23 a step); operands in two parts of bf16 (2^-16), of tf32 (2^-21 for
    each factor of a product), weights in one bf16 part for 16-bit pools and G > 8."""
    acc, accp = 128 * 2.0 ** -23, n * 2.0 ** -23 + 2.0 ** -20
    if dtype == torch.float32:
        return 2.0 ** -20 + acc, 2.0 ** -20 + accp
    return 2.0 ** -16 + acc, (2.0 ** -16 if G <= 8 else 2.0 ** -8) + accp


def check_decode(o, lse, want, dtype, G, n, label=""):
    wo, wl, wm, wp = want
    u_s, u_p = arithmetic(dtype, G, n)
    check(o, lse.T, (wo, wl.T, wm, wp.T), u_s, u_p, label)


CASES = [
    # lens, ps, Hq, H, D, dtype, window, sinks, kind
    ([1], 16, 2, 2, 64, "bf16", 0, 0, {}),
    ([17, 1, 0, 300, 16], 16, 8, 2, 128, "bf16", 0, 0, {}),
    ([1000, 63, 64, 65, 129], 8, 8, 1, 64, "bf16", 0, 0, {}),
    ([700, 2], 1, 5, 1, 128, "bf16", 0, 0, {}),
    ([2500, 31], 128, 12, 1, 128, "bf16", 0, 0, {}),            # 12 heads a group
    ([900, 40, 333], 32, 48, 2, 64, "bf16", 0, 0, {}),          # 24 heads a group
    ([5000, 77], 64, 6, 2, 128, "bf16", 100, 4, {}),
    ([5000, 10, 200], 16, 4, 4, 64, "bf16", 1, 0, {}),
    ([3000, 60], 16, 16, 2, 128, "bf16", 64, 130, dict(nhd=True)),
    ([555, 1, 0, 64], 16, 8, 2, 128, "f32", 0, 0, {}),
    ([1234, 9], 32, 5, 1, 64, "f32", 0, 0, dict(nhd=True)),
    ([700, 33], 8, 24, 2, 128, "f32", 50, 3, {}),
    ([4097], 1024, 32, 2, 64, "f32", 0, 0, {}),
]


@pytest.mark.parametrize("lens,ps,Hq,H,D,dt,window,sinks,kw", CASES)
@pytest.mark.parametrize("mode", ["yarn"])
def test_decode(lens, ps, Hq, H, D, dt, window, sinks, kw, mode):
    dtype = {"bf16": torch.bfloat16, "f32": torch.float32}[dt]
    rope = lcx.RopeParams(mode, D, scale=4.0, original_max_pos=1024, base=500000.0)
    c, rows = cache_of(lens, ps, H, D, dtype, seed=len(lens) + ps, **kw)
    ids = list(range(len(lens))) + [-1, 0]
    q = randn(99, len(ids), Hq, D, dtype=dtype)
    status = word()
    o, lse = lcx.paged_decode(c, q, ints(ids), rope, window=window, sinks=sinks, return_lse=True,
                              status=status)
    want = plain_decode(q, rows, lens, ids, rope, window, sinks)
    check_decode(o, lse, want, dtype, Hq // H, max(lens), "decode %s" % lens)
    assert int(status) == 0
    # deterministic: a second call gives the same bits
    o2, lse2 = lcx.paged_decode(c, q, ints(ids), rope, window=window, sinks=sinks, return_lse=True)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("pairing", ["half", "interleaved"])
@pytest.mark.parametrize("mode", ["none", "plain", "pi", "ntk", "dynamic_ntk"])
def test_decode_modes_and_prerotated(mode, pairing):
    rope = lcx.RopeParams(mode, 64, scale=2.0, original_max_pos=100, pairing=pairing, seq_len=400)
    lens = [77, 400]
    c, rows = cache_of(lens, 16, 2, 64, torch.float32)
    q = randn(5, 2, 6, 64, dtype=torch.float32)
    o, lse = lcx.paged_decode(c, q, ints([0, 1]), rope, return_lse=True)
    check_decode(o, lse, plain_decode(q, rows, lens, [0, 1], rope), torch.float32, 3, 400, mode)
    o, lse = lcx.paged_decode(c, q, ints([1, 0]), rope, return_lse=True, prerotated=True,
                              softmax_scale=0.3)
    check_decode(o, lse, plain_decode(q, rows, lens, [1, 0], rope, scale=0.3, prerotated=True),
                 torch.float32, 3, 400, "prerotated")


def test_factor_tables_through_append_and_decode():
    """Per-pair factors (host tables, built anew for every call): the long table beyond
    the training length, the short one within it."""
    import numpy as np
    f, short = np.linspace(1.0, 7.0, 32), np.linspace(1.0, 1.5, 32)
    for seq_len in (100, 3000):
        rope = lcx.RopeParams("factors", 64, original_max_pos=1000, factors=f, factors_short=short,
                              seq_len=seq_len)
        lens = [40]
        c, rows = cache_of(lens, 16, 2, 64, torch.float32)
        k, v, q = (randn(i, 1, h, 64, dtype=torch.float32) for i, h in ((1, 2), (2, 2), (3, 4)))
        start = lcx.pages_extend(c, ints([0]))
        lcx.paged_append(c, k, v, ints([0]), start, rope)
        kr = rotate(k.cpu(), torch.tensor([40]), rope)
        rows = [(torch.cat([rows[0][0], kr]), torch.cat([rows[0][1], v.double().cpu()]))]
        o, lse = lcx.paged_decode(c, q, ints([0]), rope, return_lse=True)
        check_decode(o, lse, plain_decode(q, rows, [41], [0], rope), torch.float32, 2, 41)


def test_decode_strided_tensors_and_layers():
    lens = [150, 20]
    rope = lcx.RopeParams("plain", 128)
    c, rows = cache_of(lens, 16, 2, 128, layers=3)
    c.k_pages[0], c.k_pages[2] = float("nan"), float("nan")   # only layer 1 is read
    big = randn(3, 2, 3, 8, 128)
    q = big[:, 1]
    out = torch.full((2, 10, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    lcx.paged_decode(c, q, ints([1, 0]), rope, layer=1, out=out[:, 1:9])
    o, lse = lcx.paged_decode(c, q.contiguous(), ints([1, 0]), rope, layer=1, return_lse=True)
    assert torch.equal(out[:, 1:9], o)
    assert (out[:, 0] == 7).all() and (out[:, 9] == 7).all()
    check_decode(o, lse, plain_decode(q, rows, lens, [1, 0], rope), torch.bfloat16, 4, 150)


def test_decode_hidden_values_are_never_read():
    """NaN and infinity in keys and values that the window hides, in free slots of
    the last page and in other sequences' pages change nothing; in a visible key
    they reach the output."""
    lens = [500, 90]
    rope = lcx.RopeParams("plain", 64)
    for dtype in (torch.bfloat16, torch.float32):
        c, rows = cache_of(lens, 16, 2, 64, dtype)
        q = randn(8, 2, 8, 64, dtype=dtype)
        a = lcx.paged_decode(c, q, ints([0, 1]), rope, window=37, sinks=3)
        for j, bad in ((10, float("nan")), (3, float("inf")), (462, -float("inf")), (400, float("nan"))):
            pg, sl = int(c.block_table[0, j // 16]), j % 16
            c.k_pages[0, pg, sl] = bad
            c.v_pages[0, pg, sl] = bad
        b = lcx.paged_decode(c, q, ints([0, 1]), rope, window=37, sinks=3)
        assert torch.equal(a, b) and torch.isfinite(a.float()).all()
        pg, sl = int(c.block_table[0, 470 // 16]), 470 % 16
        c.v_pages[0, pg, sl, 1, 5] = float("nan")
        b = lcx.paged_decode(c, q, ints([0, 1]), rope, window=37, sinks=3)
        assert torch.isnan(b[0, 4:, 5].float()).all()
        assert torch.equal(a[1], b[1]) and torch.equal(a[0, :4], b[0, :4])
        c.v_pages[0, pg, sl, 1, 5] = float("inf")
        c.v_pages[0, pg, sl, 1, 6] = -float("inf")
        b = lcx.paged_decode(c, q, ints([0, 1]), rope, window=37, sinks=3)
        assert (b[0, 4:, 5] == float("inf")).all() and (b[0, 4:, 6] == -float("inf")).all()
        assert torch.equal(a[0, 4:, :5], b[0, 4:, :5]) and torch.equal(a[0, 4:, 7:], b[0, 4:, 7:])
        c.k_pages[0, pg, sl, 0, 3] = float("nan")
        b = lcx.paged_decode(c, q, ints([0, 1]), rope, window=37, sinks=3)
        assert torch.isnan(b[0, :4].float()).all()


def test_decode_bad_numbers_are_hidden_and_reported():
    lens = [70, 40, 50]
    rope = lcx.RopeParams("plain", 64)
    c, rows = cache_of(lens, 16, 2, 64)
    q = randn(8, 4, 4, 64)
    good = lcx.paged_decode(c, q, ints([0, 1, 2, 1]), rope)
    status = word()
    b = lcx.paged_decode(c, q, ints([0, 1, 3, 1]), rope, status=status)       # sequence 3 of 3
    assert int(status) == lcx.LCX_ERR_INVALID_ARG
    assert torch.equal(b[[0, 1, 3]], good[[0, 1, 3]]) and (b[2] == 0).all()
    status.zero_()
    c.block_table[0, 1] = c.num_pages                      # no such page: keys 16..31 hidden
    b, lse = lcx.paged_decode(c, q, ints([0, 1, 2, 1]), rope, status=status, return_lse=True)
    assert int(status) == lcx.LCX_ERR_INVALID_ARG and torch.equal(b[1:], good[1:])
    k, v = rows[0]
    keep = [j for j in range(70) if not 16 <= j < 32]
    qe = rotate(q[:1].double().cpu(), torch.tensor([69]), rope)
    want = attend(qe, k[keep], v[keep], torch.tensor([69]), True, 0, 0, 64 ** -0.5)
    check(b[:1], lse[:1].T, want, *arithmetic(torch.bfloat16, 2, 70))
    status.zero_()
    c.seq_lens[1] = 10 ** 6                                # beyond the table: cut there
    c.block_table[1] = -1
    b, lse = lcx.paged_decode(c, q, ints([0, 1, 2, 1]), rope, status=status, return_lse=True)
    assert int(status) == lcx.LCX_ERR_INVALID_ARG
    assert (b[1] == 0).all() and torch.isinf(lse[1]).all() and torch.equal(b[2], good[2])


@pytest.mark.parametrize("n", [129, 300])
def test_decode_many_entries(n):
    """More entries than threads, the same sequences named over and over, padded
    entries among them: every row as in a call of its own."""
    lens = [70, 1, 0, 333, 16]
    rope = lcx.RopeParams("plain", 64)
    c, _ = cache_of(lens, 16, 2, 64, torch.float32)
    ids = [(7 * i) % 6 - 1 for i in range(n)]
    q = randn(8, n, 4, 64, dtype=torch.float32)
    o, lse = lcx.paged_decode(c, q, ints(ids), rope, return_lse=True)
    for lo in range(0, n, 97):
        a, b = lcx.paged_decode(c, q[lo:lo + 97], ints(ids[lo:lo + 97]), rope, return_lse=True)
        # other cuts of the lists: equal up to fp32 rounding of the joined parts
        assert (o[lo:lo + 97] - a).abs().max() <= 1e-5
        fin = torch.isfinite(b)
        assert torch.equal(torch.isfinite(lse[lo:lo + 97]), fin)
        assert (lse[lo:lo + 97][fin] - b[fin]).abs().max() <= 1e-5
    pad = torch.tensor([i < 0 or lens[i] == 0 for i in ids], device="cuda")
    assert (o[pad] == 0).all() and (lse[pad] == -float("inf")).all()


def test_decode_one_sequence_over_every_cta():
    """One long sequence with one kv head: every CTA holds a part of one segment."""
    lens = [70001]
    rope = lcx.RopeParams("plain", 64)
    for dtype in (torch.bfloat16, torch.float32):
        c, rows = cache_of(lens, 64, 1, 64, dtype)
        q = randn(2, 1, 3, 64, dtype=dtype)
        o, lse = lcx.paged_decode(c, q, ints([0]), rope, return_lse=True)
        check_decode(o, lse, plain_decode(q, rows, lens, [0], rope), dtype, 3, 70001)


def test_decode_on_another_stream_with_its_own_workspace():
    lens = [3000, 100]
    rope = lcx.RopeParams("plain", 128)
    c, _ = cache_of(lens, 16, 2, 128)
    q = randn(4, 2, 8, 128)
    want = lcx.paged_decode(c, q, ints([0, 1]), rope)
    ws = torch.empty(max(lcx.paged_decode_workspace_bytes(c, 2, 8), 256), dtype=torch.uint8,
                     device="cuda").fill_(255)
    ids = ints([0, 1])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = lcx.paged_decode(c, q, ids, rope, workspace=ws)
    s.synchronize()
    assert torch.equal(got, want)


# ------------------------------------------------------------------ append
@pytest.mark.parametrize("pairing", ["half", "interleaved"])
@pytest.mark.parametrize("D,H,Hq,ps,dt,nhd", [(64, 1, 3, 8, "bf16", False),
                                              (128, 8, 32, 16, "bf16", True),
                                              (64, 4, 4, 1, "f32", False),
                                              (128, 2, 10, 64, "f32", True)])
def test_append_rotates_and_places(D, H, Hq, ps, dt, nhd, pairing):
    """Keys land in their pages rotated (within one rounding of the 64-bit rotation,
    and equal to the packed copy), values as they are, and nothing else is touched."""
    dtype = {"bf16": torch.bfloat16, "f32": torch.float32}[dt]
    rope = lcx.RopeParams("yarn", D, scale=8.0, original_max_pos=512, pairing=pairing)
    old, new = [30, 0, 7, 511], [1, 40, 0, 130]
    c, rows = cache_of(old, ps, H, D, dtype, layers=2, extra=400, nhd=nhd, fill=3.0)
    ids = [3, 1, -1, 2, 0]
    cnt = [new[3], new[1], 5, new[2], new[0]]
    # the table of cache_of has no room for 511 + 130 tokens beyond one page: grow it
    big = lcx.PagedCache(c.num_pages, ps, H, D, 4, 700, num_layers=2, dtype=dtype,
                         k_pages=c.k_pages, v_pages=c.v_pages)
    big.block_table.fill_(-1)
    big.block_table[:, :c.max_pages_per_seq] = c.block_table
    for f in ("seq_lens", "ref_counts", "free_pages", "n_free"):
        getattr(big, f).copy_(getattr(c, f))
    c = big
    start = lcx.pages_extend(c, ints(ids), ints(cnt))
    assert start.tolist() == [511, 0, -1, 7, 30]
    cu = [0]
    for x in cnt:
        cu.append(cu[-1] + x)
    T = cu[-1] + 2                                      # rows behind the last entry
    k, v, q = (randn(i, T, h, D, dtype=dtype) for i, h in ((1, H), (2, H), (3, Hq)))
    q_out, k_out = torch.full_like(q, 9.0), torch.full_like(k, 9.0)
    kp, vp = c.k_pages.clone(), c.v_pages.clone()
    lcx.paged_append(c, k, v, ints(ids), start, rope, layer=1, cu_new=ints(cu), q=q, q_out=q_out,
                     k_out=k_out)
    wq, wk = torch.full_like(q, 9.0), torch.full_like(k, 9.0)
    for i, s in enumerate(ids):
        if s < 0 or cnt[i] == 0:
            continue
        r = slice(cu[i], cu[i + 1])
        p0 = int(start[i])
        pos = torch.arange(p0, p0 + cnt[i], device="cuda")
        for x, w, got in ((q, wq, q_out), (k, wk, k_out)):
            exact = rotate(x[r].cpu(), pos.cpu(), rope)
            # one output rounding; the angle, its cos/sin and mscale within 2^-22 each,
            # times the pair's length (at most sqrt(2) max|x| mscale)
            tol = U_OUT[dtype] * exact.abs() + 8 * 2.0 ** -22 * float(x.abs().max())
            assert ((got[r].double().cpu() - exact).abs() <= tol).all()
            w[r] = got[r]
        pg, sl = c.block_table[s].long()[pos // ps], pos % ps
        kp[1, pg, sl], vp[1, pg, sl] = wk[r], v[r]
    assert torch.equal(c.k_pages, kp) and torch.equal(c.v_pages, vp)
    assert torch.equal(q_out, wq) and torch.equal(k_out, wk)
    # in place, into the other layer
    k2, q2 = k.clone(), q.clone()
    lcx.paged_append(c, k2, v, ints(ids), start, rope, cu_new=ints(cu), q=q2, q_out=q2, k_out=k2)
    wq[wq == 9.0], wk[wk == 9.0] = q[wq == 9.0], k[wk == 9.0]
    assert torch.equal(q2, wq) and torch.equal(k2, wk)


def test_append_far_positions():
    """Angles stay exact near position 10^6 (the plain form in 64 bits)."""
    rope = lcx.RopeParams("plain", 64)
    c = lcx.PagedCache(4, 1024, 1, 64, 1, 2 ** 20, dtype=torch.float32)
    n = 10 ** 6
    c.seq_lens[0] = n + 3
    c.block_table[0, n // 1024] = 2
    k = randn(1, 3, 1, 64, dtype=torch.float32)
    lcx.paged_append(c, k, k, ints([0]), ints([n]), rope, cu_new=ints([0, 3]))
    want = rotate(k.cpu(), torch.arange(n, n + 3), rope)
    got = c.k_pages[0, 2, n % 1024:n % 1024 + 3].double().cpu()
    # one rounding of the angle (|phi| <= pi: 2^-23), of cos/sin and two products
    assert (got - want).abs().max() <= 8 * 2.0 ** -22 * float(k.abs().max())


def test_append_refuses_unreserved_positions():
    c, _ = cache_of([5, 5], 4, 1, 64, fill=1.0)
    rope = lcx.RopeParams("plain", 64)
    status = word()
    kp, vp = c.k_pages.clone(), c.v_pages.clone()
    k = randn(0, 4, 1, 64)
    # beyond the length, no such sequence, a negative start, a bad page
    lcx.paged_append(c, k, k, ints([0, 2, 1, -1]), ints([5, 0, -1, 0]), rope, status=status)
    assert torch.equal(c.k_pages, kp) and torch.equal(c.v_pages, vp)
    assert int(status) == lcx.LCX_ERR_INVALID_ARG
    c.block_table[1, 1] = c.num_pages + 7
    status.zero_()
    lcx.paged_append(c, k[:1], k[:1], ints([1]), ints([4]), rope, status=status)
    assert torch.equal(c.k_pages, kp) and int(status) == lcx.LCX_ERR_INVALID_ARG


# ------------------------------------------------------------------ together
def test_a_run_of_them_together():
    """Prompts through packed prefill and append, decode steps, a fork, an end and a
    compaction: decode agrees with attn_fwd over the same tokens."""
    D, H, Hq, ps = 128, 2, 8, 16
    rope = lcx.RopeParams("yarn", D, scale=4.0, original_max_pos=256)
    lens = [40, 129, 7]
    c = lcx.PagedCache(64, ps, H, D, 6, 20)
    plan = lcx.VarlenPlan(lens)
    T = sum(lens)
    q, k, v = (randn(i, T, h, D) for i, h in ((1, Hq), (2, H), (3, H)))
    ids = ints([0, 1, 2])
    start = lcx.pages_extend(c, ids, ints(lens))
    k_out = torch.empty_like(k)
    q_out = lcx.paged_append(c, k, v, ids, start, rope, cu_new=plan.cu_q, q=q, k_out=k_out)
    o = lcx.attn_varlen(q, k, v, plan, rope)
    o2 = lcx.attn_varlen(q_out, k_out, v, plan, rope, prerotated=True)
    hist = []
    a = 0
    for s, n in enumerate(lens):
        r = slice(a, a + n)
        a += n
        x = [t[r].transpose(0, 1)[None] for t in (q, k, v)]
        w = lcx.attn_fwd(*x, rope)[0].transpose(0, 1)
        for got in (o[r], o2[r]):       # two bf16 paths: each within 2e-2 of exact
            assert (got.float() - w.float()).abs().max() <= 4e-2
        hist.append([x[1], x[2]])

    def step(entries, seed, swap=False):
        n = len(entries)
        qs, ks, vs = (randn(seed + i, n, h, D) for i, h in ((1, Hq), (2, H), (3, H)))
        e = ints(entries)
        st = lcx.pages_extend(c, e)
        lcx.paged_append(c, ks, vs, e, st, rope)
        got = lcx.paged_decode(c, qs, e, rope)
        for i, s in enumerate(entries):
            hist[s] = [torch.cat([hist[s][0], ks[i][None, :, None]], 2),
                       torch.cat([hist[s][1], vs[i][None, :, None]], 2)]
            L = hist[s][0].shape[2]
            w = lcx.attn_fwd(qs[i][None, :, None], hist[s][0], hist[s][1], rope, q_offset=L - 1)
            assert (got[i].float() - w[0, :, 0].float()).abs().max() <= 4e-2
        return qs, e, got

    for i in range(12):
        step([0, 1, 2], 100 + 10 * i)
    lcx.pages_fork(c, ints([1, 1]), ints([4, 5]))
    hist += [None, list(hist[1]), list(hist[1])]
    step([4, 0, 5, 1], 400)
    lcx.pages_free(c, ints([1, 2]))
    qs, e, got = step([5, 0, 4], 500)
    lcx.pages_compact(c)
    assert torch.equal(lcx.paged_decode(c, qs, e, rope), got)
    used = int((c.ref_counts > 0).sum())
    assert (c.ref_counts[:used] > 0).all() and int(c.n_free) == c.num_pages - used
    step([4, 5, 0], 600)


def test_decode_step_replays_from_a_graph():
    """extend + append + decode captured once; two graphs with workspaces of their
    own, replayed in turn, equal eager steps on a twin cache."""
    D, H, Hq = 64, 2, 4
    rope = lcx.RopeParams("plain", D)
    lens = [100, 3, 0]
    (a, _), (b, _) = cache_of(lens, 16, H, D, extra=30), cache_of(lens, 16, H, D, extra=30)
    ids = ints([0, 1, 2])
    q, k, v = (randn(i, 3, h, D) for i, h in ((1, Hq), (2, H), (3, H)))
    need = max(lcx.paged_decode_workspace_bytes(a, 3, Hq), 256)

    def step(c, ws):
        st = lcx.pages_extend(c, ids)
        lcx.paged_append(c, k, v, ids, st, rope)
        return lcx.paged_decode(c, q, ids, rope, workspace=ws)

    meta = a.meta.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step(a, None)
    torch.cuda.current_stream().wait_stream(s)
    a.meta.copy_(meta)
    graphs = []
    for _ in range(2):
        ws = torch.empty(need, dtype=torch.uint8, device="cuda")
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            o = step(a, ws)
        graphs.append((g, o, ws))
    a.meta.copy_(meta)
    for i in range(6):
        for t in (q, k, v):
            t.copy_(randn(i + t.shape[1], *t.shape))
        g, o, _ = graphs[i % 2]
        g.replay()
        want = step(b, None)
        assert torch.equal(o, want)
        assert torch.equal(a.seq_lens, b.seq_lens)


def test_a_cache_keeps_its_buffers():
    """The calls hold the buffers' addresses: a cache refuses other ones."""
    cache = lcx.PagedCache(4, 16, 2, 64, 2, 2)
    for name in ("k_pages", "block_table", "page_size"):
        with pytest.raises(AttributeError):
            setattr(cache, name, getattr(lcx.PagedCache(4, 16, 2, 64, 2, 2), name)
                    if name != "page_size" else 32)
    cache.seq_lens += 0          # in place
    cache.reset()


@pytest.mark.parametrize("captured", [False, True])
def test_calls_behind_copies_and_fills(captured):
    """Every call's first kernel is a programmatic dependent of what lies before it in the
    stream: copies from the host, fills and small kernels are seen, in a stream and in
    a captured graph."""
    rope = lcx.RopeParams("plain", 64)
    n, L = 8, 600
    cache = lcx.PagedCache(n * 40, 16, 2, 64, n, 40)
    dev = torch.device("cuda")
    ids = torch.zeros(n, dtype=torch.int32, device=dev)
    host_ids = torch.arange(n, dtype=torch.int32).pin_memory()
    cu = torch.arange(0, n * L + 1, L, dtype=torch.int32, device=dev)
    new = torch.full((n,), L, dtype=torch.int32, device=dev)
    start = torch.empty_like(ids)
    g = torch.Generator().manual_seed(5)
    hk, hv, hq = (torch.randn((m, h, 64), generator=g).bfloat16().pin_memory()
                  for m, h in ((n * L, 2), (n * L, 2), (n, 4)))
    k, v, q, o = (torch.zeros(t.shape, dtype=torch.bfloat16, device=dev) for t in (hk, hv, hq, hq))
    qp = torch.zeros((n * L, 4, 64), dtype=torch.bfloat16, device=dev)
    op = torch.empty_like(qp)
    plan = lcx.VarlenPlan([L] * n)
    ws = torch.empty(lcx.paged_decode_workspace_bytes(cache, n, 4), dtype=torch.uint8, device=dev)
    wp = torch.empty(lcx.varlen_workspace_bytes(plan, 2, 64, k.dtype), dtype=torch.uint8, device=dev)
    status = torch.ones(1, dtype=torch.int32, device=dev)

    def step():
        status.zero_()
        ids.copy_(host_ids, non_blocking=True)
        lcx.pages_extend(cache, ids, new, start=start, status=status)
        k.copy_(hk, non_blocking=True)
        v.copy_(hv, non_blocking=True)
        lcx.paged_append(cache, k, v, ids, start, rope, cu_new=cu, status=status)
        q.copy_(hq, non_blocking=True)
        lcx.paged_decode(cache, q, ids, rope, out=o, workspace=ws, status=status)
        qp[L - 1::L].copy_(q)
        lcx.attn_varlen(qp, k, v, plan, rope, out=op, workspace=wp, status=status)
        k.zero_()
        v.zero_()
        lcx.pages_free(cache, ids, status=status)
        ids.zero_()
        q.zero_()

    if captured:
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            step()
        torch.cuda.current_stream().wait_stream(s)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
    for _ in range(3):
        o.zero_()
        op.zero_()
        graph.replay() if captured else step()
        assert int(status) == 0 and int(cache.n_free) == n * 40
        pos = torch.arange(L)
        for i in range(n):
            kk, vv = hk[i * L:(i + 1) * L], hv[i * L:(i + 1) * L]
            # the cache holds the rotated keys rounded to bf16; the library's max-abs tolerance
            kr = rotate(kk, pos, rope).bfloat16().double()
            qr = rotate(hq[i:i + 1], pos[-1:], rope)
            want = attend(qr, kr, vv.double(), pos[-1:], True, 0, 0, 0.125)[0]
            assert (o[i].double().cpu() - want[0]).abs().max() <= 2e-2
            assert (op[(i + 1) * L - 1].double().cpu() - want[0]).abs().max() <= 2e-2


@pytest.mark.parametrize("Hq", [4, 24])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_decode_key_at_minus_infinity_weighs_nothing(dt, Hq):
    """A logit of -inf (an infinite cached key) has the weight 0, as in attn_varlen."""
    dtype = {"bf16": torch.bfloat16, "f32": torch.float32}[dt]
    rope = lcx.RopeParams("plain", 64)
    c, rows = cache_of([300], 16, 2, 64, dtype)
    q = randn(1, 1, Hq, 64, dtype=dtype)
    q[:, :, 3] = q[:, :, 3].abs() + 0.5
    for j in (7, 250):
        c.k_pages[0, int(c.block_table[0, j // 16]), j % 16, :, 3] = -float("inf")
    keep = [j for j in range(300) if j not in (7, 250)]
    o, lse = lcx.paged_decode(c, q, ints([0]), rope, prerotated=True, return_lse=True)
    rows = [tuple(x[keep] for x in rows[0])]
    want = plain_decode(q, rows, [298], [0], rope, prerotated=True)
    check_decode(o, lse, want, dtype, Hq // 2, 300)


def counted(lens, ps, H, D, dtype, unit):
    """A cache whose keys count for the same (q = 0) and whose values say which run of
    `unit` keys they belong to: column (j // unit) mod D is 1, the others 0.  With it,
    per sequence, how often each column's 1 occurs."""
    c, _ = cache_of(lens, ps, H, D, dtype)
    counts = []
    for s, n in enumerate(lens):
        pos = torch.arange(n, device="cuda")
        col = (pos // unit) % D
        pg, sl = c.block_table[s].long()[pos // ps], pos % ps
        c.v_pages[0, pg, sl] = torch.eye(D, device="cuda", dtype=dtype)[col][:, None]
        counts.append(torch.bincount(col.cpu(), minlength=D).double())
    return c, counts


@pytest.mark.parametrize("lens,H,Hq,D", [
    ([70001], 1, 3, 64), ([70001], 1, 12, 64), ([70001], 1, 2, 128),
    ([30000, 5, 0, 12345, 64, 8191], 2, 8, 128), ([9000] * 7 + [1], 3, 60, 64),
    ([200000], 1, 20, 128), ([257] * 40, 4, 4, 64)])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_decode_joins_every_key_once(lens, H, Hq, D, dt):
    """Equal weights: lse is the logarithm of the number of keys and o the share of every
    run of 48 keys.  A lost or doubled part, block or tile (8 keys and more of a run)
    moves both far beyond the rounding: the weights are 1, all sums are whole numbers
    below 2^24, so o carries 1/z, a product and the output's rounding, lse a logarithm
    and a product."""
    dtype = {"bf16": torch.bfloat16, "f32": torch.float32}[dt]
    c, counts = counted(lens, 64, H, D, dtype, 48)
    q = torch.zeros((len(lens), Hq, D), dtype=dtype, device="cuda")
    o, lse = lcx.paged_decode(c, q, ints(list(range(len(lens)))), lcx.RopeParams("plain", D),
                              return_lse=True)
    for s, n in enumerate(lens):
        if n == 0:
            assert (o[s] == 0).all() and (lse[s] == -float("inf")).all()
            continue
        want = counts[s] / n
        assert ((o[s].double().cpu() - want).abs() <= (U_OUT[dtype] + 2.0 ** -22) * want).all()
        wl = float(torch.log(torch.tensor(n).double()))
        assert (lse[s].double().cpu() - wl).abs().max() <= 2.0 ** -21 * (1 + wl)


@pytest.mark.parametrize("Hq", [3, 12])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_decode_long_sequence_within_its_chained_sums(Hq, dt):
    """A sequence over every CTA against the 64-bit form, the sums bounded by what the
    kernel chains: a warp's quarter of a stretch (two CTAs an SM share the keys, in blocks
    of at most 128), four warps, and the parts, which lanes of a warp add (10 and 5
    steps).  Half a CTA's keys missing would move lse by 1.7e-3, beyond its bound."""
    dtype = {"bf16": torch.bfloat16, "f32": torch.float32}[dt]
    n, D = 70001, 64
    rope = lcx.RopeParams("plain", D)
    c, rows = cache_of([n], 64, 1, D, dtype)
    q = (0.5 * randn(2, 1, Hq, D, dtype=torch.float32)).to(dtype)
    o, lse = lcx.paged_decode(c, q, ints([0]), rope, return_lse=True)
    ctas = 2 * torch.cuda.get_device_properties(0).multi_processor_count
    chain = (n // ctas + 2 * 128) // 4 + 4 + 15
    wo, wl, wm, wp = plain_decode(q, rows, [n], [0], rope)
    check_decode(o, lse, (wo, wl, wm, wp), dtype, Hq, chain)
    u_s, u_p = arithmetic(dtype, Hq, chain)
    if Hq > 8 and dtype == torch.bfloat16:
        u_p -= 2.0 ** -8                   # lse sums the weights before their rounding
    bound = u_s * wp + 2.0 ** -22 * (1 + wl.abs()) + u_p
    assert float(bound.max()) <= 1e-3
    assert ((lse.double().cpu() - wl).abs() <= bound).all()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_pages_far_apart_in_memory(dt):
    """Pages more than 2^32 bytes and 2^31 elements apart: append, decode, fork, page copy
    and compaction equal the same calls on a dense cache."""
    dtype = {"bf16": torch.bfloat16, "f32": torch.float32}[dt]
    P, ps, H, D = 6, 4, 2, 64
    stride = (1 << 29) + 64
    rope = lcx.RopeParams("plain", D)
    big = [torch.empty(5 * stride + ps * H * D, dtype=dtype, device="cuda") for _ in range(2)]
    far = [t.as_strided((1, P, ps, H, D), (0, stride, H * D, D, 1)) for t in big]
    assert 5 * stride > 2 ** 31 and 5 * stride * big[0].element_size() > 2 ** 32
    a = lcx.PagedCache(P, ps, H, D, 3, 6, dtype=dtype, k_pages=far[0], v_pages=far[1])
    b = lcx.PagedCache(P, ps, H, D, 3, 6, dtype=dtype)
    k, v = randn(1, 10, H, D, dtype=dtype), randn(2, 10, H, D, dtype=dtype)
    q = randn(3, 3, 4, D, dtype=dtype)
    for c in (a, b):
        c.k_pages.zero_()
        c.v_pages.zero_()
    got = []
    for c in (a, b):
        ids = ints([0, 1])
        c.free_pages.copy_(ints([4, 3, 1, 5, 0, 2]))    # sequence 0 takes 5 and 0, 1 takes 2
        start = lcx.pages_extend(c, ids, ints([7, 3]))
        lcx.paged_append(c, k, v, ids, start, rope, cu_new=ints([0, 7, 10]))
        lcx.pages_fork(c, ints([0]), ints([2]))
        one = lcx.paged_decode(c, q, ints([0, 1, 2]), rope)
        lcx.pages_free(c, ints([1]))
        lcx.pages_compact(c)                            # 5 -> 2
        assert c.block_table[0, :2].tolist() == [2, 0]
        two = lcx.paged_decode(c, q, ints([0, 1, 2]), rope)
        lcx.pages_copy(c, ints([0]), ints([5]))
        got.append((one, two, c.meta.clone(), c.k_pages.clone(), c.v_pages.clone()))
    for x, y in zip(*got):
        assert torch.equal(x, y)
    assert torch.equal(got[0][0][[0, 2]], got[0][1][[0, 2]])


@pytest.mark.parametrize("Hq", [8, 24])
def test_decode_in_place(Hq):
    """out = q: a query is read before its row is written, whole or joined."""
    lens = [3000, 40, 0, 700]
    rope = lcx.RopeParams("plain", 128)
    c, _ = cache_of(lens, 16, 2, 128)
    q = randn(4, 4, Hq, 128)
    want = lcx.paged_decode(c, q, ints([0, 1, 2, 3]), rope)
    assert torch.equal(lcx.paged_decode(c, q, ints([0, 1, 2, 3]), rope, out=q), want)
    assert torch.equal(q, want)
