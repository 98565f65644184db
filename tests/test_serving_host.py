"""CPU checks of the paged-cache and packed-prompt calls: struct layouts, the
host-made plan, and malformed arguments refused before any device work."""
import ctypes
import os
import random
import subprocess

import numpy as np
import pytest
import torch

import ntk_rope_flashattn_b200 as lcx
from ntk_rope_flashattn_b200 import build as lcx_build
from ntk_rope_flashattn_b200 import paged, varlen

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BAD, UNS = lcx.LCX_ERR_INVALID_ARG, lcx.LCX_ERR_UNSUPPORTED
F = 0x10000000       # a fake, aligned device address: never followed


@pytest.fixture(scope="module")
def lib():
    lcx_build.build()
    return lcx.load()


STRUCTS = {"lcx_paged_cache": paged._Cache, "lcx_paged_append_args": paged._AppendArgs,
           "lcx_paged_decode_args": paged._DecodeArgs, "lcx_varlen_info": varlen._Info,
           "lcx_varlen_args": varlen._VarlenArgs}


def test_struct_layouts_match_the_header(tmp_path):
    lines = ["#include <stdio.h>", "#include <stddef.h>", '#include "lcx.h"', "int main(void) {"]
    for name, T in STRUCTS.items():
        lines.append('printf("%s %%zu\\n", sizeof(%s));' % (name, name))
        for f, _ in T._fields_:
            lines.append('printf("%s.%s %%zu\\n", offsetof(%s, %s));' % (name, f, name, f))
    src = tmp_path / "layout.c"
    src.write_text("\n".join(lines + ["return 0; }"]))
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-std=c99", "-I", os.path.join(ROOT, "include"), str(src), "-o",
                    str(exe)], check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout
    for line in out.splitlines():
        key, val = line.rsplit(" ", 1)
        name, _, field = key.partition(".")
        T = STRUCTS[name]
        assert (getattr(T, field).offset if field else ctypes.sizeof(T)) == int(val), key


def test_status_word_code_has_a_name(lib):
    assert lib.lcx_status_string(lcx.LCX_ERR_NO_PAGES).decode() != "unknown status"


# ------------------------------------------------------------------ plan
@pytest.mark.parametrize("lq,lk", [
    ([], []), ([0], [0]), ([1], [1]), ([128, 129, 0, 255, 256, 257], None),
    ([3, 700, 1], [500, 700, 2]), ([5], [2]), ([4, 4], [0, 9]),
])
def test_plan_covers_every_row_once(lq, lk):
    plan = lcx.VarlenPlan(lq, lk, device="cpu")
    lk = lq if lk is None else lk
    n = len(lq)
    assert (plan.total_q, plan.total_k) == (sum(lq), sum(lk))
    assert plan.cu_q.tolist() == [sum(lq[:i]) for i in range(n + 1)]
    assert plan.cu_k.tolist() == [sum(lk[:i]) for i in range(n + 1)]
    base = (8 + 2 * (n + 1) + 7) // 8 * 8
    for which, rows in ((0, 128), (1, 256)):
        m = int(plan.info.n_units[which])
        u = plan.plan[base:base + 8 * m].view(m, 8).tolist() if m else []
        base += 8 * m
        seen, weight = set(), None
        for q0, r, k0, nk, pos0, *pad in u:
            s = max(i for i in range(n) if plan.cu_q[i] <= q0 and lq[i] > 0)
            assert 1 <= r <= rows and q0 + r <= plan.cu_q[s + 1]
            assert (k0, nk) == (int(plan.cu_k[s]), lk[s]) and pad == [0, 0, 0]
            assert pos0 == lk[s] - lq[s] + q0 - int(plan.cu_q[s])
            assert not seen & set(range(q0, q0 + r))
            seen |= set(range(q0, q0 + r))
            w = min(nk, pos0 + r)
            assert weight is None or w <= weight      # heaviest first
            weight = w
        assert seen == set(range(sum(lq)))


@pytest.mark.parametrize("lens", [[1.5], [2.0, 3.0], ["4"], [True], [1 << 40]])
def test_plan_takes_whole_numbers(lens):
    with pytest.raises(ValueError):
        lcx.VarlenPlan(lens, device="cpu")


def test_plan_of_arrays():
    """Lists, arrays and host tensors of any integer type make the same plan."""
    a = lcx.VarlenPlan([5, 0, 300], device="cpu").plan
    for x in (np.array([5, 0, 300], np.uint16), torch.tensor([5, 0, 300]), (5, 0, 300)):
        assert torch.equal(lcx.VarlenPlan(x, device="cpu").plan, a)
    assert lcx.VarlenPlan([], device="cpu").total_q == 0


def test_plan_refusals(lib):
    with pytest.raises(ValueError):
        lcx.VarlenPlan([-1], device="cpu")
    with pytest.raises(ValueError):
        lcx.VarlenPlan([1, 2], [3], device="cpu")
    with pytest.raises(ValueError):
        lcx.VarlenPlan([1 << 30, 1 << 30], device="cpu")
    a = np.array([5], np.int32)
    info = varlen._Info()
    buf = np.zeros(64, np.int32)
    p = a.ctypes.data
    assert lib.lcx_varlen_plan(p, p, 1, buf.ctypes.data, 8, ctypes.byref(info)) == BAD
    assert lib.lcx_varlen_plan(None, p, 1, buf.ctypes.data, 64, ctypes.byref(info)) == BAD
    assert lib.lcx_varlen_plan(p, p, 1, None, 64, ctypes.byref(info)) == BAD
    assert lib.lcx_varlen_plan_ints(p, p, -1) == -1


# ------------------------------------------------------------------ refusals
def rope(D=128, **kw):
    return lcx.RopeParams(kw.pop("mode", "plain"), D, **kw)


def cache_args(**kw):
    c = paged._Cache()
    for f in ("k_pages", "v_pages", "block_table", "seq_lens", "ref_counts", "free_pages",
              "n_free", "scratch"):
        setattr(c, f, F)
    c.dtype, c.page_size = 0, 16
    c.num_layers, c.num_pages, c.Hkv, c.D, c.max_seqs, c.max_pages = 2, 10, 4, 128, 3, 5
    c.k_strides = c.v_strides = (ctypes.c_int64 * 5)(10 * 4 * 16 * 128, 4 * 16 * 128, 128,
                                                     16 * 128, 1)
    for k, x in kw.items():
        setattr(c, k, (ctypes.c_int64 * 5)(*x) if k.endswith("strides") else x)
    return c


@pytest.mark.parametrize("kw,expect", [
    (dict(dtype=3), BAD), (dict(num_pages=0), BAD), (dict(num_pages=1 << 21), UNS),
    (dict(D=96), UNS), (dict(page_size=0), UNS), (dict(page_size=24), UNS),
    (dict(page_size=2048), UNS), (dict(max_seqs=0), BAD), (dict(max_pages=1 << 28), UNS),
    (dict(k_pages=0), BAD), (dict(scratch=0), BAD), (dict(v_pages=F + 8), UNS),
    (dict(k_strides=[1, 8192, 128, 2048, 2]), UNS), (dict(k_strides=[81920, 0, 128, 2048, 1]), UNS),
    (dict(v_strides=[81920, 8192, 132, 2048, 1]), UNS),
    (dict(v_strides=[81920, -8192, 128, 2048, 1]), UNS),
])
def test_cache_checks_in_every_call(lib, kw, expect):
    c = ctypes.byref(cache_args(**kw))
    assert lib.lcx_pages_extend(c, F, F, 2, F, None, None) == expect
    assert lib.lcx_pages_fork(c, F, F, 2, None, None) == expect
    assert lib.lcx_pages_free(c, F, 2, None, None) == expect
    assert lib.lcx_pages_compact(c, None, None) == expect
    assert lib.lcx_pages_copy(c, F, F, 2, None, None) == expect
    assert lib.lcx_paged_append(c, ctypes.byref(append_args()), None) == expect
    assert lib.lcx_paged_decode(c, ctypes.byref(decode_args()), F, 1 << 40, None) == expect
    assert lib.lcx_last_error().decode()


def test_page_call_checks(lib):
    c = ctypes.byref(cache_args())
    assert lib.lcx_pages_extend(c, F, F, -1, F, None, None) == BAD
    assert lib.lcx_pages_extend(c, 0, F, 2, F, None, None) == BAD
    assert lib.lcx_pages_extend(c, F, F, 2, 0, None, None) == BAD
    assert lib.lcx_pages_extend(c, F, F, 1025, F, None, None) == UNS
    assert lib.lcx_pages_fork(c, F, 0, 2, None, None) == BAD
    assert lib.lcx_pages_free(c, 0, 2, None, None) == BAD
    assert lib.lcx_pages_copy(c, 0, F, 2, None, None) == BAD
    for call in (lambda: lib.lcx_pages_extend(c, 0, 0, 0, 0, None, None),
                 lambda: lib.lcx_pages_fork(c, 0, 0, 0, None, None),
                 lambda: lib.lcx_pages_free(c, 0, 0, None, None),
                 lambda: lib.lcx_pages_copy(c, 0, 0, 0, None, None)):
        assert call() == lcx.LCX_OK                 # nothing to do
    assert lib.lcx_pages_compact(None, None, None) == BAD
    assert lib.lcx_paged_scratch_ints(0) == -1
    assert lib.lcx_paged_scratch_ints(10) > 0


def append_args(**kw):
    a = paged._AppendArgs()
    a.k = a.v = a.seq_ids = a.start = F
    a.n = a.T = 3
    for f in ("k_strides", "v_strides", "k_out_strides"):
        setattr(a, f, (ctypes.c_int64 * 3)(4 * 128, 128, 1))
    for f in ("q_strides", "q_out_strides"):
        setattr(a, f, (ctypes.c_int64 * 3)(8 * 128, 128, 1))
    a.rope = rope()._c()
    for k, x in kw.items():
        if k == "rope":
            a.rope = x._c()
        else:
            setattr(a, k, (ctypes.c_int64 * 3)(*x) if k.endswith("strides") else x)
    return a


@pytest.mark.parametrize("kw,expect", [
    (dict(layer=2), BAD), (dict(layer=-1), BAD), (dict(T=4), BAD), (dict(n=-1), BAD),
    (dict(q=F), BAD), (dict(q_out=F), BAD), (dict(q=F, q_out=F, Hq=0), BAD),
    (dict(k=0), BAD), (dict(v=F + 8), UNS), (dict(seq_ids=0), BAD), (dict(start=0), BAD),
    (dict(rope=rope(64)), UNS), (dict(rope=rope(mode="dynamic_ntk")), BAD),
    (dict(k_strides=[4 * 128, 128, 2]), UNS), (dict(v_strides=[4 * 128, 100, 1]), UNS),
    (dict(k_strides=[-512, 128, 1]), UNS), (dict(k_out=F, k_out_strides=[1024, 128, 1]), BAD),
    (dict(T=1 << 31, cu_new=F), UNS),
])
def test_append_refusals(lib, kw, expect):
    assert lib.lcx_paged_append(ctypes.byref(cache_args()), ctypes.byref(append_args(**kw)),
                                None) == expect
    assert lib.lcx_last_error().decode()


def decode_args(**kw):
    a = paged._DecodeArgs()
    a.q = a.o = a.seq_ids = F
    a.n, a.Hq = 3, 8
    a.q_strides = a.o_strides = (ctypes.c_int64 * 3)(8 * 128, 128, 1)
    a.rope = rope()._c()
    for k, x in kw.items():
        if k == "rope":
            a.rope = x._c()
        else:
            setattr(a, k, (ctypes.c_int64 * 3)(*x) if k.endswith("strides") else x)
    return a


@pytest.mark.parametrize("kw,expect", [
    (dict(Hq=6), BAD), (dict(Hq=0), BAD), (dict(n=-1), BAD), (dict(layer=2), BAD),
    (dict(window=-1), BAD), (dict(sinks=-1), BAD), (dict(softmax_scale=float("nan")), BAD),
    (dict(softmax_scale=-1.0), BAD), (dict(flags=2), BAD), (dict(q=0), BAD), (dict(o=F + 4), UNS),
    (dict(seq_ids=0), BAD), (dict(rope=rope(64)), UNS), (dict(rope=rope(mode="dynamic_ntk")), BAD),
    (dict(q_strides=[1024, 129, 1]), UNS), (dict(o_strides=[1024, 128, 2]), UNS),
])
def test_decode_refusals(lib, kw, expect):
    assert lib.lcx_paged_decode(ctypes.byref(cache_args()), ctypes.byref(decode_args(**kw)), F,
                                1 << 40, None) == expect
    assert lib.lcx_last_error().decode()


def test_decode_workspace(lib):
    f = lib.lcx_paged_decode_workspace_bytes
    for bad in ((-1, 8, 4, 128), (1, 6, 4, 128), (1, 8, 4, 96), (1, 8, 0, 128),
                (1 << 21, 8, 4, 128)):
        assert f(*bad) == -1
    need = f(3, 8, 4, 128)
    assert need >= 0
    if need > 0:
        c = ctypes.byref(cache_args())
        a = ctypes.byref(decode_args())
        assert lib.lcx_paged_decode(c, a, F, need - 1, None) == BAD
        assert lib.lcx_paged_decode(c, a, F + 16, need, None) == BAD
        assert lib.lcx_paged_decode(c, a, None, need, None) == BAD


def varlen_args(**kw):
    a = varlen._VarlenArgs()
    a.q = a.k = a.v = a.o = a.plan = a.workspace = F
    a.workspace_bytes = 1 << 30
    a.info = lcx.VarlenPlan([100, 28], device="cpu").info
    a.causal, a.Tq, a.Tk, a.Hq, a.Hkv, a.D = 1, 128, 128, 8, 4, 128
    a.q_strides = a.o_strides = (ctypes.c_int64 * 3)(8 * 128, 128, 1)
    a.k_strides = a.v_strides = (ctypes.c_int64 * 3)(4 * 128, 128, 1)
    a.rope = rope()._c()
    for k, x in kw.items():
        if k == "rope":
            a.rope = x._c()
        else:
            setattr(a, k, (ctypes.c_int64 * 3)(*x) if k.endswith("strides") else x)
    return a


@pytest.mark.parametrize("kw,expect", [
    (dict(dtype=2), BAD), (dict(D=96, rope=rope(96)), UNS), (dict(Hkv=3), BAD), (dict(Hq=0), BAD),
    (dict(Tq=127), BAD), (dict(Tk=100), BAD), (dict(causal=2), BAD), (dict(window=-1), BAD),
    (dict(causal=0, window=5), UNS), (dict(flags=2), BAD), (dict(reserved0=1), BAD),
    (dict(watchdog_ms=60001), BAD), (dict(softmax_scale=float("inf")), BAD), (dict(plan=0), BAD),
    (dict(plan=F + 4), BAD), (dict(q=F + 2), UNS), (dict(v=0), BAD), (dict(o=0), BAD),
    (dict(workspace=0), BAD), (dict(workspace_bytes=1000), BAD), (dict(workspace=F + 16), BAD), (dict(rope=rope(64)), UNS),
    (dict(q_strides=[1024, 128, 2]), UNS), (dict(k_strides=[512, 100, 1]), UNS),
])
def test_varlen_refusals(lib, kw, expect):
    assert lib.lcx_attn_varlen(ctypes.byref(varlen_args(**kw)), None) == expect
    assert lib.lcx_last_error().decode()


def test_varlen_without_rows_is_a_noop(lib):
    a = varlen_args(info=lcx.VarlenPlan([0, 0], device="cpu").info, q=0, k=0, v=0, o=0, plan=0)
    assert lib.lcx_attn_varlen(ctypes.byref(a), None) == lcx.LCX_OK


@pytest.mark.parametrize("bad", [[0, 128, 1], [8 * 128, 0, 1]])
def test_expanded_outputs_are_refused(lib, bad):
    """Tokens or heads that share memory: outputs of every call, and what the bf16
    packed call reads through tensor maps."""
    c = ctypes.byref(cache_args())
    for a in (append_args(q=F, q_out=F + (1 << 20), Hq=8, q_out_strides=bad),
              append_args(k_out=F + (1 << 20), k_out_strides=bad)):
        assert lib.lcx_paged_append(c, ctypes.byref(a), None) == UNS
    a = decode_args(o_strides=bad)
    assert lib.lcx_paged_decode(c, ctypes.byref(a), F, 1 << 40, None) == UNS
    for name in ("o", "q", "k", "v"):
        a = varlen_args(**{name + "_strides": bad})
        assert lib.lcx_attn_varlen(ctypes.byref(a), None) == UNS
    a = varlen_args(dtype=1, o_strides=bad)
    assert lib.lcx_attn_varlen(ctypes.byref(a), None) == UNS
    assert b"stride 0" in lib.lcx_last_error()


def test_rope_struct_follows_the_fields():
    """One struct per set of values; the parameters stay plain data."""
    import copy
    import pickle
    r = rope(mode="yarn", scale=4.0)
    a, packed = paged._rope_c(r)
    assert bytes(a) == packed == bytes(r._c()) and paged._rope_c(r)[0] is a
    assert pickle.loads(pickle.dumps(r)) == r == copy.deepcopy(r)
    r.scale = 8.0
    assert paged._rope_c(r)[1] == bytes(r._c()) != packed
    f = rope(mode="factors", factors=np.ones(64))
    assert paged._rope_c(f)[0] is not paged._rope_c(f)[0]


def test_packed_structs_are_the_declared_ones():
    r = rope(mode="yarn", scale=4.0)._c()
    s = (ctypes.c_int64 * 3)(11, 12, 13)
    want = paged._DecodeArgs(1, 2, None, 4, None, 6, 7, 8, s, s, r, 9, 10, 0.5, 1)
    assert paged._pack_decode(1, 2, 0, 4, 0, 6, 7, 8, *s, *s, bytes(r), 9, 10, 0.5, 1) == bytes(want)
    want = paged._AppendArgs(1, 2, 3, 4, None, 6, 7, 8, 9, 10, 11, 12, 13, s, s, s, s, s, r)
    got = paged._pack_append(1, 2, 3, 4, 0, 6, 7, 8, 9, 10, 11, 12, 13, *s, *s, *s, *s, *s, bytes(r))
    assert got == bytes(want)
    info = lcx.VarlenPlan([3, 5], device="cpu").info
    want = varlen._VarlenArgs(1, 2, 3, 4, 5, 6, 7, 8, 9, info, 0, 1, 12, 13, 14, 15, 16, s, s, s, s,
                              r, 17, 18, 0.25, 1, 20, 0)
    got = varlen._pack_args(1, 2, 3, 4, 5, 6, 7, 8, 9, bytes(info), 0, 1, 12, 13, 14, 15, 16, *s, *s,
                            *s, *s, bytes(r), 17, 18, 0.25, 1, 20, 0)
    assert got == bytes(want)


def test_binding_refuses_host_tensors():
    q = torch.zeros((4, 2, 64))
    plan = lcx.VarlenPlan([4], device="cpu")
    with pytest.raises(ValueError, match="CUDA"):
        lcx.attn_varlen(q, q, q, plan, rope(64))
    with pytest.raises(ValueError, match="CUDA"):
        lcx.PagedCache(4, 16, 2, 64, 2, 2, device="cpu")


def test_plain_pages_hold_their_invariants():
    """The plain bookkeeping the GPU tests compare with: every page is free or
    counted once per holder, and partial pages have one holder."""
    import serving_plain as sp
    rng = random.Random(3)
    m = sp.PlainPages(40, 4, 8, 12)
    for _ in range(300):
        op = rng.randrange(4)
        ids = [rng.randrange(-1, 8) for _ in range(rng.randrange(1, 5))]
        if op == 0:
            m.extend(ids, [rng.randrange(0, 9) for _ in ids])
        elif op == 1:
            m.fork([rng.randrange(8) for _ in ids], ids)
        elif op == 2:
            m.release(ids[:1])
        else:
            m.compact()
        held = [0] * 40
        for s in range(8):
            pages = [p for p in m.table[s] if p >= 0]
            assert len(pages) == -(-m.lens[s] // 4) == len(set(pages))
            for p in pages:
                held[p] += 1
            if m.lens[s] % 4:
                assert m.ref[pages[-1]] == 1
        assert held == m.ref
        assert sorted(m.free) == [p for p in range(40) if m.ref[p] == 0]


def test_decode_refuses_more_blocks_than_an_int_counts(lib):
    """2^20 entries of up to 65503 fp32 keys, D 128: blocks of 32 keys, 2047 of them; a
    window and sinks that begin inside a block add up to two more, and the blocks of all
    entries are counted in 32 bits."""
    c = cache_args(dtype=1, D=128, Hkv=1, page_size=1, max_pages=65503, num_pages=1 << 20)
    a = decode_args(n=1 << 20, Hq=1, window=65472, sinks=31)
    need = lib.lcx_paged_decode_workspace_bytes(1 << 20, 1, 1, 128)
    assert lib.lcx_paged_decode(ctypes.byref(c), ctypes.byref(a), F, need, None) == UNS
