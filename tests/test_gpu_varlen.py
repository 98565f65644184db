"""attn_varlen on the GPU against the plain 64-bit form (bounds: serving_plain)
and, for bf16, the library's own tolerance (max-abs 2e-2, mean-abs 2e-3)."""
import pytest
import torch

import ntk_rope_flashattn_b200 as lcx
from serving_plain import attend, check, rotate

pytestmark = pytest.mark.gpu


def randn(seed, *shape, dtype=torch.bfloat16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def plain(q, k, v, lq, lk, rope, causal=True, window=0, sinks=0, scale=None, prerotated=False):
    q, k, v = (x.double().cpu() for x in (q, k, v))
    scale = q.shape[-1] ** -0.5 if scale is None else scale
    parts, a, b = [], 0, 0
    for nq, nk in zip(lq, lk):
        qp = torch.arange(nq) + (nk - nq)
        qs, ks = q[a:a + nq], k[b:b + nk]
        if not prerotated:
            qs, ks = rotate(qs, qp, rope), rotate(ks, torch.arange(nk), rope)
        parts.append(attend(qs, ks, v[b:b + nk], qp, causal, window, sinks, scale))
        a, b = a + nq, b + nk
    return (torch.cat([p[0] for p in parts]), torch.cat([p[1] for p in parts], 1),
            torch.cat([p[2] for p in parts]), torch.cat([p[3] for p in parts], 1))


def arithmetic(dtype, n):
    """(u_s, u_p): bf16 inputs: q' and k' rounded to fp16 (2^-11 each), their products'
    sums cut by the tensor core, the weights rounded to bf16 (their sum is not); fp32
    cuts each factor into two tf32 parts (2^-21 each, 2^-20 for the product left out:
    2^-19, within acc for the logits and 2 u_p for the values) and rounds q', k' to fp32."""
    acc = 128 * 2.0 ** -23 + 2.0 ** -18
    if dtype == torch.bfloat16:
        return 2.0 ** -10 + 2.0 ** -20 + acc, 2.0 ** -8 + n * 2.0 ** -23 + 2.0 ** -20
    return 2.0 ** -22 + acc, n * 2.0 ** -24 + 2.0 ** -20


def compare(o, lse, want, dtype, n, label=""):
    check(o, lse, want, *arithmetic(dtype, n), label)
    if dtype == torch.bfloat16:
        err = (o.double().cpu() - want[0]).abs()
        half = torch.where(want[0].abs() >= 4, torch.exp2(torch.floor(torch.log2(
            want[0].abs().clamp(min=1e-30))) - 8), torch.zeros(()).double())
        assert float((err - half).max()) <= 2e-2 and float(err.mean()) <= 2e-3


LENS = [
    ([1], None), ([5, 1, 0, 3], None), ([128, 127, 129], None), ([64, 300, 1, 0, 257], None),
    ([1, 2, 130], [400, 131, 130]), ([10, 200, 0], [3, 200, 9]), ([600], [1000]),
]


@pytest.mark.parametrize("lq,lk", LENS)
@pytest.mark.parametrize("Hq,H,D,dt", [(2, 2, 64, "bf16"), (8, 2, 128, "bf16"),
                                       (3, 1, 128, "bf16"), (10, 2, 64, "bf16"),
                                       (4, 2, 64, "f32"), (3, 1, 128, "f32")])
def test_packed_lengths(lq, lk, Hq, H, D, dt):
    dtype = {"bf16": torch.bfloat16, "f32": torch.float32}[dt]
    lk = lq if lk is None else lk
    rope = lcx.RopeParams("yarn", D, scale=4.0, original_max_pos=64)
    q, k, v = (randn(i, n, h, D, dtype=dtype)
               for i, n, h in ((1, sum(lq), Hq), (2, sum(lk), H), (3, sum(lk), H)))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    o, lse = lcx.attn_varlen(q, k, v, lcx.VarlenPlan(lq, lk), rope, return_lse=True, status=status)
    assert int(status) == 0
    compare(o, lse, plain(q, k, v, lq, lk, rope), dtype, max(lk), "%s" % lq)
    o2, lse2 = lcx.attn_varlen(q, k, v, lcx.VarlenPlan(lq, lk), rope, return_lse=True)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("window,sinks", [(1, 0), (7, 0), (130, 3), (200, 150), (1000, 4)])
@pytest.mark.parametrize("Hq,H,D,dt", [(4, 2, 64, "bf16"), (3, 1, 128, "bf16"), (2, 1, 64, "f32")])
def test_window_and_sinks(window, sinks, Hq, H, D, dt):
    dtype = {"bf16": torch.bfloat16, "f32": torch.float32}[dt]
    lq, lk = [513, 40, 90], [513, 40, 700]
    rope = lcx.RopeParams("plain", D)
    q, k, v = (randn(i, n, h, D, dtype=dtype)
               for i, n, h in ((1, sum(lq), Hq), (2, sum(lk), H), (3, sum(lk), H)))
    o, lse = lcx.attn_varlen(q, k, v, lcx.VarlenPlan(lq, lk), rope, window=window, sinks=sinks,
                             return_lse=True)
    compare(o, lse, plain(q, k, v, lq, lk, rope, True, window, sinks), dtype, 700)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("mode,pairing", [("none", "half"), ("plain", "interleaved"),
                                          ("ntk", "half"), ("dynamic_ntk", "half"),
                                          ("pi", "interleaved")])
def test_modes_not_causal_prerotated(mode, pairing, dt):
    dtype = {"bf16": torch.bfloat16, "f32": torch.float32}[dt]
    lq, lk = [100, 3, 140], [100, 250, 20]
    # dynamic NTK takes the plan's longest key length
    import dataclasses
    rope = lcx.RopeParams(mode, 128, scale=2.0, original_max_pos=50, pairing=pairing)
    fixed = dataclasses.replace(rope, seq_len=250)
    q, k, v = (randn(i, n, h, 128, dtype=dtype) for i, n, h in ((1, 243, 4), (2, 370, 2), (3, 370, 2)))
    plan = lcx.VarlenPlan(lq, lk)
    o, lse = lcx.attn_varlen(q, k, v, plan, rope, causal=False, return_lse=True, softmax_scale=0.05)
    compare(o, lse, plain(q, k, v, lq, lk, fixed, causal=False, scale=0.05), dtype, 250, mode)
    o, lse = lcx.attn_varlen(q, k, v, plan, rope, prerotated=True, return_lse=True)
    compare(o, lse, plain(q, k, v, lq, lk, fixed, prerotated=True), dtype, 250, "prerotated")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_strides_and_rows_behind_the_last_sequence(dt):
    """q, k, v cut out of one fused projection, outputs into a larger tensor; rows
    behind the last sequence are left as they were."""
    dtype = {"bf16": torch.bfloat16, "f32": torch.float32}[dt]
    lq = [90, 131]
    T = sum(lq) + 37
    qkv = randn(0, T, 8, 64, dtype=dtype)
    qkv[sum(lq):] = float("nan")
    q, k, v = qkv[:, :4], qkv[:, 4:6], qkv[:, 6:]
    rope = lcx.RopeParams("plain", 64)
    out = torch.full((T, 6, 64), 5.0, dtype=dtype, device="cuda")
    lse = torch.full((4, T), 5.0, device="cuda")
    lcx.attn_varlen(q, k, v, lcx.VarlenPlan(lq), rope, out=out[:, 1:5], lse=lse)
    n = sum(lq)
    compare(out[:n, 1:5], lse[:, :n], plain(q[:n], k[:n], v[:n], lq, lq, rope), dtype, 131)
    assert (out[n:] == 5).all() and (lse[:, n:] == 5).all()
    assert (out[:, 0] == 5).all() and (out[:, 5] == 5).all()
    o = lcx.attn_varlen(q, k, v, lcx.VarlenPlan(lq), rope)
    assert (o[n:] == 0).all() and torch.equal(o[:n], out[:n, 1:5])


@pytest.mark.parametrize("Hq,H,D,dt", [(4, 2, 64, "bf16"), (8, 2, 128, "bf16"),
                                       (3, 1, 128, "bf16"), (2, 1, 128, "f32")])
def test_hidden_nan_and_infinity(Hq, H, D, dt):
    """NaN and infinity in other sequences, later tokens and tokens behind the window
    leave a query alone bit for bit; where they are visible they show."""
    dtype = {"bf16": torch.bfloat16, "f32": torch.float32}[dt]
    lens = [200, 330]
    rope = lcx.RopeParams("plain", D)
    q, k, v = (randn(i, 530, h, D, dtype=dtype) for i, h in ((1, Hq), (2, H), (3, H)))
    plan = lcx.VarlenPlan(lens)
    for window, sinks in ((0, 0), (50, 2)):
        a, la = lcx.attn_varlen(q, k, v, plan, rope, window=window, sinks=sinks, return_lse=True)
        k2, v2 = k.clone(), v.clone()
        # token 150 of the first, 100 of the second sequence
        k2[150], v2[300] = float("nan"), float("inf")
        v2[150, 0, :7] = float("nan")
        b, lb = lcx.attn_varlen(q, k2, v2, plan, rope, window=window, sinks=sinks, return_lse=True)
        sees = torch.zeros(530, dtype=torch.bool, device="cuda")
        for first, n, t in ((0, 200, 150), (200, 330, 100)):
            last = n if window == 0 else min(n, t + window)
            sees[first + t:first + last] = True
        assert torch.equal(a[~sees], b[~sees]) and torch.equal(la[:, ~sees], lb[:, ~sees])
        assert not torch.isfinite(b[sees].float()).any()
        assert torch.isnan(b[150:200 if window == 0 else 200].float()).all()
        assert (b[200:][sees[200:]] == float("inf")).all()
        assert torch.equal(la[:, 200:], lb[:, 200:])     # values do not enter the lse


MANY = [(37 * i * i + 11 * i) % 330 for i in range(48)] + [1, 0, 128, 256, 257, 511]


@pytest.mark.parametrize("window,sinks", [(0, 0), (60, 0), (200, 70)])
@pytest.mark.parametrize("Hq,H,D", [(8, 2, 128), (8, 2, 64), (9, 3, 128), (10, 2, 64), (6, 6, 64)])
def test_many_sequences(Hq, H, D, window, sinks):
    """Enough row blocks for two query tiles a CTA: two heads of an even group, two row
    blocks of an odd one, precise blocks among them, chunks with keys before them."""
    lk = [n + (7 * i) % 90 if i % 3 == 0 else n for i, n in enumerate(MANY)]
    rope = lcx.RopeParams("yarn", D, scale=4.0, original_max_pos=64)
    q, k, v = (randn(i, n, h, D) for i, n, h in ((1, sum(MANY), Hq), (2, sum(lk), H),
                                                 (3, sum(lk), H)))
    o, lse = lcx.attn_varlen(q, k, v, lcx.VarlenPlan(MANY, lk), rope, window=window, sinks=sinks,
                             return_lse=True)
    compare(o, lse, plain(q, k, v, MANY, lk, rope, True, window, sinks), torch.bfloat16, 511)
    o2 = lcx.attn_varlen(q, k, v, lcx.VarlenPlan(MANY, lk), rope, window=window, sinks=sinks)
    assert torch.equal(o, o2)


@pytest.mark.parametrize("Hq,H,D", [(8, 2, 128), (9, 3, 64)])
def test_many_sequences_hidden_values_and_scaled_keys(Hq, H, D):
    """With two query tiles a CTA: a NaN and an infinite value in one late token of every
    sequence, and keys far outside fp16's range."""
    rope = lcx.RopeParams("plain", D)
    plan = lcx.VarlenPlan(MANY)
    T = sum(MANY)
    q, k, v = (randn(i, T, h, D) for i, h in ((1, Hq), (2, H), (3, H)))
    a, la = lcx.attn_varlen(q, k, v, plan, rope, return_lse=True)
    v2, sees = v.clone(), torch.zeros(T, dtype=torch.bool, device="cuda")
    at = 0
    for i, n in enumerate(MANY):
        if n > 1:
            t = at + (3 * n) // 4
            v2[t, i % H, 3] = float("nan")
            v2[t, i % H, 5] = float("inf")
            sees[t:at + n] = True
        at += n
    b, lb = lcx.attn_varlen(q, k, v2, plan, rope, return_lse=True)
    hit = ~torch.isfinite(b.float())
    assert torch.equal(la, lb) and not hit[~sees].any()
    assert torch.equal(a[~hit], b[~hit])
    assert not hit[:, :, [c for c in range(D) if c not in (3, 5)]].any()
    G, at = Hq // H, 0
    for i, n in enumerate(MANY):
        if n > 1:
            t, h = at + (3 * n) // 4, slice((i % H) * G, (i % H) * G + G)
            assert torch.isnan(b[t:at + n, h, 3].float()).all()
            assert (b[t:at + n, h, 5] == float("inf")).all()
            assert int(hit[at:at + n].sum()) == 2 * G * (at + n - t)
        at += n
    ks, qs = k.clone(), (q.float() * 2.0 ** -20).bfloat16()
    ks[::50] = (k[::50].float() * 2.0 ** 20).bfloat16()
    o, lse = lcx.attn_varlen(qs, ks, v, plan, rope, return_lse=True)
    compare(o, lse, plain(qs, ks, v, MANY, MANY, rope), torch.bfloat16, 511)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_one_token_and_one_head_of_any_stride(dt):
    """Strides of sizes of one are never taken."""
    dtype = {"bf16": torch.bfloat16, "f32": torch.float32}[dt]
    rope = lcx.RopeParams("plain", 64)
    q, k, v = (randn(i, 1, h, 64, dtype=dtype) for i, h in ((1, 4), (2, 1), (3, 1)))
    k, v = (t.as_strided(t.shape, (0, 0, 1)) for t in (k, v))
    o, lse = lcx.attn_varlen(q, k, v, lcx.VarlenPlan([1]), rope, return_lse=True)
    compare(o, lse, plain(q, k, v, [1], [1], rope), dtype, 1)


def test_expanded_heads_fp32():
    """One kv head expanded to all: read as it stands (fp32)."""
    rope = lcx.RopeParams("plain", 64)
    lens = [70, 30]
    q, k, v = (randn(i, 100, h, 64, dtype=torch.float32) for i, h in ((1, 4), (2, 1), (3, 1)))
    plan = lcx.VarlenPlan(lens)
    a = lcx.attn_varlen(q, k, v, plan, rope)
    b = lcx.attn_varlen(q, k.expand(-1, 4, -1), v.expand(-1, 4, -1), plan, rope)
    assert torch.equal(a, b)


@pytest.mark.parametrize("D", [64, 128])
def test_fp32_values_not_finite(D):
    """fp32: a NaN and an infinite value in two columns reach the queries that see
    them in those columns, over several key tiles, and nothing else."""
    rope = lcx.RopeParams("plain", D)
    q, k, v = (randn(i, 300, h, D, dtype=torch.float32) for i, h in ((1, 4), (2, 2), (3, 2)))
    plan = lcx.VarlenPlan([40, 260])
    for window in (0, 100):
        a = lcx.attn_varlen(q, k, v, plan, rope, window=window)
        v2 = v.clone()
        v2[140, 1, 7] = float("nan")         # token 100 of the second sequence
        v2[140, 0, D - 1] = -float("inf")
        b = lcx.attn_varlen(q, k, v2, plan, rope, window=window)
        last = 300 if window == 0 else 140 + window
        hit = torch.zeros_like(a, dtype=torch.bool)
        hit[140:last, 2:, 7] = True
        hit[140:last, :2, D - 1] = True
        assert torch.isnan(b[140:last, 2:, 7]).all()
        assert (b[140:last, :2, D - 1] == -float("inf")).all()
        assert torch.equal(a[~hit], b[~hit])


def test_nan_value_of_one_column():
    """A NaN in one column of one visible value reaches that column of the queries
    that see it, and nothing else."""
    rope = lcx.RopeParams("plain", 128)
    q, k, v = (randn(i, 300, h, 128) for i, h in ((1, 4), (2, 2), (3, 2)))
    plan = lcx.VarlenPlan([300])
    a = lcx.attn_varlen(q, k, v, plan, rope)
    v2 = v.clone()
    v2[140, 1, 77] = float("nan")
    b = lcx.attn_varlen(q, k, v2, plan, rope)
    hit = torch.zeros_like(a, dtype=torch.bool)
    hit[140:, 2:, 77] = True
    assert torch.isnan(b[hit].float()).all() and torch.equal(a[~hit], b[~hit])


def test_long_rows_against_attn_fwd():
    """Many key tiles: the packed call agrees with attn_fwd per sequence."""
    rope = lcx.RopeParams("yarn", 128, scale=4.0, original_max_pos=2048)
    lens = [4000, 1300]
    q, k, v = (randn(i, 5300, h, 128) for i, h in ((1, 8), (2, 2), (3, 2)))
    o, lse = lcx.attn_varlen(q, k, v, lcx.VarlenPlan(lens), rope, return_lse=True)
    a = 0
    for n in lens:
        x = [t[a:a + n].transpose(0, 1)[None] for t in (q, k, v)]
        w, wl = lcx.attn_fwd(*x, rope, return_lse=True)
        assert (o[a:a + n].float() - w[0].transpose(0, 1).float()).abs().max() <= 4e-2
        assert (lse[:, a:a + n] - wl[0]).abs().max() <= 2e-2
        a += n


def test_replays_from_a_graph_and_other_streams():
    rope = lcx.RopeParams("plain", 64)
    plan = lcx.VarlenPlan([77, 200])
    q, k, v = (randn(i, 277, h, 64) for i, h in ((1, 4), (2, 2), (3, 2)))
    out = torch.empty_like(q)
    ws = torch.empty(lcx.varlen_workspace_bytes(plan, 2, 64, k.dtype), dtype=torch.uint8,
                     device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        lcx.attn_varlen(q, k, v, plan, rope, workspace=ws, out=out)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(out, lcx.attn_varlen(q, k, v, plan, rope))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lcx.attn_varlen(q, k, v, plan, rope, workspace=ws, out=out)
    for i in range(3):
        for t in (q, k, v):
            t.copy_(randn(10 * i + t.shape[1], *t.shape))
        g.replay()
        assert torch.equal(out, lcx.attn_varlen(q, k, v, plan, rope))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_calls_at_once_on_two_streams(dt):
    """One plan, one set of keys, two streams, a workspace for each call in flight."""
    dtype = {"bf16": torch.bfloat16, "f32": torch.float32}[dt]
    rope = lcx.RopeParams("plain", 64)
    plan = lcx.VarlenPlan([300, 7, 450])
    k, v = (randn(i, 757, 2, 64, dtype=dtype) for i in (2, 3))
    qs = [randn(10 + i, 757, 4, 64, dtype=dtype) for i in range(2)]
    want = [lcx.attn_varlen(q, k, v, plan, rope) for q in qs]
    need = lcx.varlen_workspace_bytes(plan, 2, 64, dtype)
    ws = [torch.empty(need, dtype=torch.uint8, device="cuda") for _ in qs]
    outs = [[torch.empty_like(q) for _ in range(8)] for q in qs]
    streams = [torch.cuda.Stream() for _ in qs]
    torch.cuda.synchronize()
    for r in range(8):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                lcx.attn_varlen(qs[i], k, v, plan, rope, workspace=ws[i], out=outs[i][r])
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(o, want[i]) for o in outs[i])


def test_a_plan_that_is_not_the_tensors_is_refused():
    rope = lcx.RopeParams("plain", 64)
    q, k = randn(0, 10, 2, 64), randn(1, 10, 2, 64)
    with pytest.raises(lcx.LcxError):
        lcx.attn_varlen(q, k, k, lcx.VarlenPlan([11]), rope)
    with pytest.raises(ValueError):
        lcx.attn_varlen(q, k, k, lcx.VarlenPlan([10], device="cpu"), rope)


def test_expired_waits_report_timeout_and_context_survives():
    """With no copies issued every wait runs out: the kernel ends on its own, reports
    LCX_ERR_TIMEOUT and leaves the context usable."""
    rope = lcx.RopeParams("plain", 128)
    plan = lcx.VarlenPlan([300, 40])
    q, k, v = (randn(i, 340, h, 128) for i, h in ((1, 4), (2, 2), (3, 2)))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    lcx.attn_varlen(q, k, v, plan, rope, status=status, watchdog_ms=50, _test_stall=True)
    torch.cuda.synchronize()
    assert int(status) == lcx.LCX_ERR_TIMEOUT
    status.zero_()
    o, lse = lcx.attn_varlen(q, k, v, plan, rope, status=status, return_lse=True)
    assert int(status) == 0
    compare(o, lse, plain(q, k, v, [300, 40], [300, 40], rope), torch.bfloat16, 300)


@pytest.mark.parametrize("Hq,H", [(2, 1), (3, 1)])
def test_values_far_outside_fp16(Hq, H):
    """Rows of q and k of any bf16 magnitude: rows beyond fp16's range are scaled, the
    others keep their bits of precision."""
    rope = lcx.RopeParams("plain", 64)
    lens = [150, 400]
    plan = lcx.VarlenPlan(lens)
    q, k, v = (randn(i, 550, h, 64) for i, h in ((1, Hq), (2, H), (3, H)))
    # queries down as far as their keys are up, so the logits stay of ordinary size
    qs, ks = q.clone(), k.clone()
    ks[:150] = (k[:150].float() * 2.0 ** 30).bfloat16()
    qs[:150] = (q[:150].float() * 2.0 ** -30).bfloat16()
    ks[150:] = (k[150:].float() * 2.0 ** -25).bfloat16()
    qs[150:] = (q[150:].float() * 2.0 ** 25).bfloat16()
    o, lse = lcx.attn_varlen(qs, ks, v, plan, rope, return_lse=True)
    compare(o, lse, plain(qs, ks, v, lens, lens, rope), torch.bfloat16, 400)
    # one key row in a hundred far up, met by queries far down
    ks, qs = k.clone(), (q.float() * 2.0 ** -20).bfloat16()
    ks[::100] = (k[::100].float() * 2.0 ** 20).bfloat16()
    o, lse = lcx.attn_varlen(qs, ks, v, plan, rope, return_lse=True)
    compare(o, lse, plain(qs, ks, v, lens, lens, rope), torch.bfloat16, 400)


def test_lse_of_short_rows_is_precise():
    """fp16 operands, in two parts where a row sees few keys: lse stays within 3e-5
    of exact for rows of 1 to 127 keys (u_s = 2^-21 for two parts of both factors;
    E < 20 for N(0, 1) inputs at D = 128) and windows below 128 keys."""
    rope = lcx.RopeParams("plain", 128)
    lens = [1, 2, 60, 127, 300]
    n = sum(lens)
    plan = lcx.VarlenPlan(lens)
    q, k, v = (randn(i, n, h, 128) for i, h in ((1, 4), (2, 2), (3, 2)))
    o, lse = lcx.attn_varlen(q, k, v, plan, rope, return_lse=True)
    w = plain(q, k, v, lens, lens, rope)
    short = torch.cat([torch.arange(x) < 127 for x in lens])
    assert ((lse.double().cpu() - w[1]).abs()[:, short]).max() <= 3e-5
    o, lse = lcx.attn_varlen(q, k, v, plan, rope, window=9, sinks=1, return_lse=True)
    w = plain(q, k, v, lens, lens, rope, True, 9, 1)
    assert (lse.double().cpu() - w[1]).abs().max() <= 3e-5


# Pair frequencies above 1 (context shrunk: scale or factors below 1): angles many turns
# a token, which keys and queries must reduce alike.
FAST = [("pi", dict(scale=0.01)), ("factors", 1e-3), ("factors", 1e-6)]


@pytest.mark.parametrize("pairing", ["half", "interleaved"])
@pytest.mark.parametrize("lens,Hq,H,D", [([60, 127, 300], 4, 2, 128), ([60, 127, 300], 3, 1, 64),
                                         ([300] * 10, 32, 2, 64), ([300] * 10, 30, 2, 128)])
@pytest.mark.parametrize("mode,kw", FAST)
def test_frequencies_above_one(mode, kw, lens, Hq, H, D, pairing):
    """Angles of up to 10^8 rad: within the bounds of any other, and lse of short rows
    within 3e-5 (the angles add 2^-22 rad a pair to the bound derived below)."""
    if mode == "factors":
        kw = dict(factors=[kw] * (D // 2))
    rope = lcx.RopeParams(mode, D, original_max_pos=64, pairing=pairing, **kw)
    n = sum(lens)
    q, k, v = (randn(i, n, h, D) for i, h in ((1, Hq), (2, H), (3, H)))
    o, lse = lcx.attn_varlen(q, k, v, lcx.VarlenPlan(lens), rope, return_lse=True)
    want = plain(q, k, v, lens, lens, rope)
    compare(o, lse, want, torch.bfloat16, max(lens), mode)
    short = torch.cat([torch.arange(x) < 127 for x in lens])
    assert ((lse.double().cpu() - want[1]).abs()[:, short]).max() <= 3e-5


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_rows_of_a_foreign_plan_are_left_out_and_reported(dt):
    """A device plan whose second sequence ends behind the tensors: its rows stay as they
    were, the status word says so, the first sequence's are right."""
    dtype = {"bf16": torch.bfloat16, "f32": torch.float32}[dt]
    rope = lcx.RopeParams("plain", 64)
    lens = [100, 101]
    plan, other = lcx.VarlenPlan(lens), lcx.VarlenPlan([100, 128])
    plan.plan.copy_(other.plan)
    q, k, v = (randn(i, 201, h, 64, dtype=dtype) for i, h in ((1, 4), (2, 2), (3, 2)))
    out, lse = torch.full_like(q, 5.0), torch.full((4, 201), 5.0, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    lcx.attn_varlen(q, k, v, plan, rope, out=out, lse=lse, status=status)
    assert int(status) == lcx.LCX_ERR_INVALID_ARG
    assert (out[100:] == 5).all() and (lse[:, 100:] == 5).all()
    compare(out[:100], lse[:, :100], plain(q[:100], k[:100], v[:100], [100], [100], rope), dtype,
            100)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_a_visible_key_at_minus_infinity_weighs_nothing(dt):
    """A logit of -inf (an infinite key, given rotated) has the weight 0, a logit of
    +inf makes the row NaN."""
    dtype = {"bf16": torch.bfloat16, "f32": torch.float32}[dt]
    rope = lcx.RopeParams("plain", 64)
    n = 150
    q, k, v = (randn(i, n, h, 64, dtype=dtype) for i, h in ((1, 4), (2, 2), (3, 2)))
    q[:, :, 3] = q[:, :, 3].abs() + 0.5
    k[[7, 90], :, 3] = -float("inf")
    keep = [j for j in range(n) if j not in (7, 90)]
    o, lse = lcx.attn_varlen(q, k, v, lcx.VarlenPlan([n]), rope, causal=False, prerotated=True,
                             return_lse=True)
    want = plain(q, k[keep], v[keep], [n], [n - 2], rope, causal=False, prerotated=True)
    compare(o, lse, want, dtype, n)
    k[20, 1, 3] = float("inf")
    o2, lse2 = lcx.attn_varlen(q, k, v, lcx.VarlenPlan([n]), rope, causal=False, prerotated=True,
                               return_lse=True)
    assert torch.equal(o2[:, :2], o[:, :2]) and torch.equal(lse2[:2], lse[:2])
    assert torch.isnan(o2[:, 2:].float()).all() and torch.isnan(lse2[2:]).all()


@pytest.mark.parametrize("Hq,H,D", [(4, 2, 128), (3, 1, 64)])
@pytest.mark.parametrize("up,down", [(500.0, 1.0), (8000.0, 2.0 ** -8), (2000.0, 2.0 ** -13)])
def test_rows_with_outlier_channels(Hq, H, D, up, down):
    """Rows of q and k with a few channels far above the others, not the same ones, so the
    logits come from the products of both sizes.  Bound: besides fp16's relative
    rounding, values below 2^-14 (after a row's scaling by a power of two, which makes its
    largest value at least 2^-6) keep an absolute one of 2^-25; a logit moves by c
    (|q'|_1 + |k'|_1) 2^-25 for it, in units of rows whose largest value is below 2^14."""
    rope = lcx.RopeParams("plain", D)
    lens = [130, 300, 7]
    n = sum(lens)
    q, k, v = (randn(i, n, h, D, dtype=torch.float32) for i, h in ((1, Hq), (2, H), (3, H)))
    q, k = q * down, k * down
    q[:, :, [3, D // 2 + 9]] *= up / down / 8
    k[:, :, [5, D - 2]] *= up / down
    q, k, v = (x.bfloat16() for x in (q, k, v))
    o, lse = lcx.attn_varlen(q, k, v, lcx.VarlenPlan(lens), rope, return_lse=True)
    w = plain(q, k, v, lens, lens, rope)
    u_s, u_p = arithmetic(torch.bfloat16, 300)
    # |q'|_1 <= sqrt(2) |q|_1, and scaled rows' floors are 2^-25 of the row's power of two
    def floor(x):
        mx = (2.0 ** 0.5) * x.float().abs().amax(-1)
        return torch.exp2(torch.floor(torch.log2(torch.clamp(mx / 2.0 ** 14, min=1.0))) - 24)
    f = max(float(floor(q).max()), float(floor(k).max()))
    one = 2.0 ** 0.5 * max(float(x.float().abs().sum(-1).max()) for x in (q, k))
    extra = D ** -0.5 * 2 * one * f
    check(o, lse, (w[0], w[1], w[2], w[3] + extra / u_s), u_s, u_p, "outliers %g %g" % (up, down))


@pytest.mark.parametrize("Hq,H,D", [(4, 2, 128), (3, 1, 64)])
@pytest.mark.parametrize("e", [60, 115, 122, -122])
def test_queries_and_keys_at_opposite_ends_of_the_exponents(e, Hq, H, D):
    """Rows of q about 2^-e, rows of k about 2^e: ordinary logits."""
    rope = lcx.RopeParams("plain", D)
    lens = [200, 333]
    q, k, v = (randn(i, 533, h, D) for i, h in ((1, Hq), (2, H), (3, H)))
    q, k = (q.double() * 2.0 ** -e).bfloat16(), (k.double() * 2.0 ** e).bfloat16()
    o, lse = lcx.attn_varlen(q, k, v, lcx.VarlenPlan(lens), rope, return_lse=True)
    compare(o, lse, plain(q, k, v, lens, lens, rope), torch.bfloat16, 333)


# Packed keys beyond 80 MiB take the CTA order by kv head (heads of 128, groups of two and
# more): two heads a CTA, two row blocks a CTA (odd groups), one tile a CTA (few row blocks).
LONG = [([4000, 1300], [4000, 1300], 8, 2, 128, "bf16"),
        ([200, 3, 300], [9000, 6000, 6001], 64, 8, 128, "bf16"),
        ([200, 3, 300], [9000, 6000, 6001], 40, 8, 128, "bf16"),
        ([40, 130], [15000, 6001], 16, 8, 128, "bf16"),
        ([70, 300], [36000, 6001], 8, 8, 64, "bf16"),
        ([33, 130], [5000, 1000], 4, 2, 128, "f32"),
        ([33, 130], [5000, 1000], 3, 1, 64, "f32")]


@pytest.mark.parametrize("lq,lk,Hq,H,D,dt", LONG)
@pytest.mark.parametrize("window,sinks", [(0, 0), (2500, 200)])
def test_long_rows_see_every_key_once(lq, lk, Hq, H, D, dt, window, sinks):
    """Equal weights (q = 0) and values that say which run of 48 keys, of which sequence
    and kv head, they belong to: o is the share of every run, lse the logarithm of the
    number of keys.  A lost, doubled or foreign tile moves both far beyond the rounding:
    the weights are 1 (or a power of two), all sums whole numbers below 2^24, so o
    carries 1/z, a product and the output's rounding, lse a logarithm and a product."""
    dtype = {"bf16": torch.bfloat16, "f32": torch.float32}[dt]
    rope = lcx.RopeParams("plain", D)
    q = torch.zeros((sum(lq), Hq, D), dtype=dtype, device="cuda")
    k = randn(2, sum(lk), H, D, dtype=dtype)
    v = torch.zeros_like(k)
    eye = torch.eye(D, dtype=dtype, device="cuda")
    at, cols = 0, []
    for s, n in enumerate(lk):
        cols.append([(torch.arange(n, device="cuda") // 48 + 5 * s + 11 * g) % D for g in range(H)])
        for g in range(H):
            v[at:at + n, g] = eye[cols[s][g]]
        at += n
    o, lse = lcx.attn_varlen(q, k, v, lcx.VarlenPlan(lq, lk), rope, window=window, sinks=sinks,
                             return_lse=True)
    at = 0
    for s, (n, m) in enumerate(zip(lq, lk)):
        pos, key = torch.arange(n, device="cuda") + (m - n), torch.arange(m, device="cuda")
        keep = key[None, :] <= pos[:, None]
        if window:
            keep &= (pos[:, None] - key[None, :] < window) | (key[None, :] < sinks)
        z = keep.sum(1).double()
        for g in range(H):
            want = (keep.double() @ eye[cols[s][g]].double()) / z[:, None]
            r = slice(g * (Hq // H), (g + 1) * (Hq // H))
            err = (o[at:at + n, r].double() - want[:, None]).abs()
            u = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24
            assert (err <= (u + 2.0 ** -22) * want[:, None]).all()
        wl = torch.log(z)
        assert ((lse[:, at:at + n].double() - wl).abs() <= 2.0 ** -21 * (1 + wl)).all()
        at += n


@pytest.mark.parametrize("lq,lk,Hq,H,D,dt", LONG)
def test_long_rows_find_their_key(lq, lk, Hq, H, D, dt):
    """Every query looks for one key anywhere in its past (q' = 3 k' there, a logit of
    some 3 sqrt(D) among N(0, 9) ones), so o is nearly that key's value: within the bounds
    of the 64-bit form, on every eleventh row."""
    dtype = {"bf16": torch.bfloat16, "f32": torch.float32}[dt]
    rope = lcx.RopeParams("plain", D)
    k, v = (randn(i, sum(lk), H, D, dtype=dtype) for i in (2, 3))
    g = torch.Generator().manual_seed(7)
    q = torch.empty((sum(lq), Hq, D), dtype=dtype, device="cuda")
    rows, a, b = [], 0, 0
    kc = k.double().cpu()
    for n, m in zip(lq, lk):
        pos = torch.arange(n) + (m - n)
        for h in range(Hq):
            t = (torch.rand(n, generator=g) * (pos + 1)).long()
            # R(p) q = 3 R(t) k
            x = rotate(kc[b + t, h // (Hq // H)][:, None], t - pos, rope)
            q[a:a + n, h] = (3 * x[:, 0]).to(dtype).cuda()
        rows.append((torch.arange(0, n, 11), a, b, n, m))
        a, b = a + n, b + m
    o, lse = lcx.attn_varlen(q, k, v, lcx.VarlenPlan(lq, lk), rope, return_lse=True)
    for r, a, b, n, m in rows:
        pos = r + (m - n)
        qs = rotate(q[a + r.cuda()].cpu(), pos, rope)
        ks = rotate(k[b:b + m].cpu(), torch.arange(m), rope)
        want = attend(qs, ks, v[b:b + m].double().cpu(), pos, True, 0, 0, D ** -0.5)
        assert float(want[0].abs().mean()) > 0.5
        check(o[a + r.cuda()], lse[:, a + r.cuda()], want, *arithmetic(dtype, m), "%d of %d" % (n, m))


@pytest.mark.parametrize("Hq,H,D", [(16, 8, 128), (32, 16, 64)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (4000, 300)])
def test_long_prompts_see_every_key_once(Hq, H, D, window, sinks):
    """Prompts of 123 MiB of keys and values (with heads of 128 in the CTA order by kv
    head): equal weights over values that say which run of 240 keys, of which sequence and
    kv head, they belong to, on rows all over the prompts (bounds:
    test_long_rows_see_every_key_once)."""
    lens = [17000, 14500]
    rope = lcx.RopeParams("plain", D)
    q = torch.zeros((sum(lens), Hq, D), dtype=torch.bfloat16, device="cuda")
    k = randn(2, sum(lens), H, D)
    eye = torch.eye(D, dtype=torch.bfloat16, device="cuda")
    cols = [[(torch.arange(n, device="cuda") // 240 + 5 * s + 11 * g) % D for g in range(H)]
            for s, n in enumerate(lens)]
    v = torch.stack([torch.cat([eye[cols[s][g]] for s in range(2)]) for g in range(H)], 1)
    o, lse = lcx.attn_varlen(q, k, v, lcx.VarlenPlan(lens), rope, window=window, sinks=sinks,
                             return_lse=True)
    at = 0
    for s, n in enumerate(lens):
        pos = torch.cat([torch.arange(0, n, 37), torch.arange(n - 200, n)]).cuda()
        key = torch.arange(n, device="cuda")
        keep = key[None, :] <= pos[:, None]
        if window:
            keep &= (pos[:, None] - key[None, :] < window) | (key[None, :] < sinks)
        z, keep = keep.sum(1).double(), keep.double()
        for g in range(H):
            want = (keep @ eye[cols[s][g]].double()) / z[:, None]
            got = o[at + pos, g * (Hq // H):(g + 1) * (Hq // H)].double()
            assert ((got - want[:, None]).abs() <= (2.0 ** -8 + 2.0 ** -22) * want[:, None]).all()
        wl = torch.log(z)
        assert ((lse[:, at + pos].double() - wl).abs() <= 2.0 ** -21 * (1 + wl)).all()
        at += n


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_rows_far_apart_in_memory(dt):
    """Tokens 2^24 bytes apart and more, in all more than 2^31 elements: equal to the packed call."""
    dtype = {"bf16": torch.bfloat16, "f32": torch.float32}[dt]
    lens, D = [150, 130], 64
    T, stride = 280, (1 << 23) + 64
    rope = lcx.RopeParams("plain", D)
    plan = lcx.VarlenPlan(lens)
    q, k, v = (randn(i, T, h, D, dtype=dtype) for i, h in ((1, 4), (2, 2), (3, 2)))
    want, wl = lcx.attn_varlen(q, k, v, plan, rope, return_lse=True)
    big = torch.empty((T - 1) * stride + 12 * D, dtype=dtype, device="cuda")
    assert big.numel() > 2 ** 31
    at, far = 0, []
    for t in (q, k, v, want):
        x = big.as_strided(t.shape, (stride, D, 1), at)
        x.copy_(t)
        far.append(x)
        at += t.shape[1] * D
    far[3].fill_(7)
    o, lse = lcx.attn_varlen(*far[:3], plan, rope, return_lse=True, out=far[3])
    assert torch.equal(o, want) and torch.equal(lse, wl)


@pytest.mark.parametrize("lens", [[300, 7, 129], [64] * 40])
@pytest.mark.parametrize("Hq,H,dt", [(8, 2, "bf16"), (9, 3, "bf16"), (4, 2, "f32")])
def test_output_over_the_queries(lens, Hq, H, dt):
    """out = q (o does not overlap k or v, but may take q's place)."""
    dtype = {"bf16": torch.bfloat16, "f32": torch.float32}[dt]
    rope = lcx.RopeParams("plain", 64)
    plan, T = lcx.VarlenPlan(lens), sum(lens)
    q, k, v = (randn(i, T, h, 64, dtype=dtype) for i, h in ((1, Hq), (2, H), (3, H)))
    want = lcx.attn_varlen(q, k, v, plan, rope)
    for prerotated in (False, True):
        x = q.clone()
        w = lcx.attn_varlen(x, k, v, plan, rope, prerotated=prerotated)
        assert torch.equal(lcx.attn_varlen(x, k, v, plan, rope, prerotated=prerotated, out=x), w)
        assert prerotated or torch.equal(x, want)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_queries_without_any_key(dt):
    """No sequence has a key: o = 0, lse = -inf, causal or not."""
    dtype = {"bf16": torch.bfloat16, "f32": torch.float32}[dt]
    rope = lcx.RopeParams("plain", 64)
    q, k = randn(1, 140, 4, 64, dtype=dtype), randn(2, 0, 2, 64, dtype=dtype)
    for causal in (True, False):
        o, lse = lcx.attn_varlen(q, k, k, lcx.VarlenPlan([130, 0, 10], [0, 0, 0]), rope,
                                 causal=causal, return_lse=True)
        assert (o == 0).all() and (lse == -float("inf")).all()
