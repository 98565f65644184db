"""Timed cases of the paged-cache and packed-prompt operators, with their plain forms.

Four operators of a serving loop around the RoPE attention library:

  prefill  attention over packed prompts of different lengths (``attn_varlen``)
  append   rotate new keys (and queries), write keys and values into cache pages
           (``paged_append``)
  decode   attention of one new token per sequence over the paged cache
           (``paged_decode``)
  pages    free + fork of sequences, and compaction (``pages_free``,
           ``pages_fork``, ``pages_compact``)

``run`` computes a pass in elementary torch operations while ``own`` is false and
calls the library while it is true.  RoPE here is plain (theta_i = b^(-2i/D), pair
(i, i + D/2)).
"""
import math
import random

import torch

own = False

BASE = 500000.0


def listed():
    return [
        # one chat turn of a small model: a few hundred cached tokens, latency counts
        dict(name="decode_one_short", op="decode", B=1, lo=300, hi=300, Hq=8, Hkv=2, D=64,
             page=16, dtype="bf16", window=0, sinks=0, lens_seed=1),
        # a continuous-batching step: 32 users of ragged lengths, 32/8 heads
        dict(name="decode_batch", op="decode", B=32, lo=400, hi=9000, Hq=32, Hkv=8, D=128,
             page=16, dtype="bf16", window=0, sinks=0, lens_seed=2),
        # long context: a few users near the 128K limit beside shorter ones
        dict(name="decode_long", op="decode", B=4, lo=60000, hi=131072, Hq=32, Hkv=8, D=128,
             page=64, dtype="bf16", window=0, sinks=0, lens_seed=3),
        # sliding window with sinks over a long fp32 cache, odd group of 5
        dict(name="decode_window_f32", op="decode", B=24, lo=3000, hi=65000, Hq=20, Hkv=4, D=128,
             page=32, dtype="f32", window=4096, sinks=4, lens_seed=4),
        # three short prompts of a small model
        dict(name="prefill_short", op="prefill", n=3, lo=17, hi=250, Hq=8, Hkv=2, D=64,
             dtype="bf16", window=0, sinks=0, prefix=0, lens_seed=5),
        # an ordinary admission batch: mixed prompts, 32/8 heads
        dict(name="prefill_batch", op="prefill", n=12, lo=200, hi=4100, Hq=32, Hkv=8, D=128,
             dtype="bf16", window=0, sinks=0, prefix=0, lens_seed=6),
        # long documents: chunks of new tokens against keys kept from earlier chunks
        dict(name="prefill_long", op="prefill", n=2, lo=9000, hi=14000, Hq=32, Hkv=8, D=128,
             dtype="bf16", window=0, sinks=0, prefix=6000, lens_seed=7),
        # window and sinks, odd head group, fp32 operands
        dict(name="prefill_window_f32", op="prefill", n=5, lo=100, hi=1500, Hq=6, Hkv=2, D=64,
             dtype="f32", window=333, sinks=4, prefix=0, lens_seed=8),
        # the append of one decode step: 64 users, one token each, queries rotated too
        dict(name="append_step", op="append", n=64, lo=1, hi=1, Hq=32, Hkv=8, D=128, page=16,
             dtype="bf16", lens_seed=9),
        # the append behind a prefill: whole prompts into their pages
        dict(name="append_prompts", op="append", n=12, lo=300, hi=4100, Hq=32, Hkv=8, D=128,
             page=64, dtype="bf16", lens_seed=10),
        # a beam step over 4 layers: 8 parents, children dropped and forked again
        dict(name="pages_fork", op="fork", n=32, parents=8, lo=500, hi=5000, layers=16, Hkv=8,
             D=128, page=64, dtype="bf16", lens_seed=11),
        # a fragmented pool moved together before it is shrunk
        dict(name="pages_compact", op="compact", n=40, lo=100, hi=900, layers=8, Hkv=8, D=128,
             page=32, dtype="bf16", lens_seed=12),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["decode", "decode", "decode", "prefill", "prefill", "prefill", "append",
                     "fork", "compact"])
    dt = rng.choice(["bf16", "bf16", "bf16", "f32"])
    D = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    seed = rng.randrange(1 << 30)
    page = rng.choice([8, 16, 32, 64, 128])
    if op == "decode":
        G = rng.choice([1, 2, 3, 4, 5, 6, 7, 8, 12, 16])
        B = _log_int(rng, 1, 64)
        # K and V of all sequences stay below 1.5 GB
        per_key = 2 * Hkv * D * (2 if dt == "bf16" else 4)
        hi = min(131072, int(1.5e9 / (per_key * B)))
        hi = _log_int(rng, 1, hi)
        win = rng.choice([0, 0, _log_int(rng, 1, 8192)])
        return dict(op=op, B=B, lo=_log_int(rng, 1, hi), hi=hi, Hq=G * Hkv, Hkv=Hkv, D=D,
                    page=page, dtype=dt, window=win,
                    sinks=rng.choice([0, 4, 130]) if win else 0, lens_seed=seed)
    if op == "prefill":
        G = rng.choice([1, 2, 3, 4, 7, 8])
        n = _log_int(rng, 1, 16)
        hi = _log_int(rng, 1, 4000 if dt == "bf16" else 1500)
        win = rng.choice([0, 0, _log_int(rng, 1, 4096)])
        return dict(op=op, n=n, lo=_log_int(rng, 1, hi), hi=hi, Hq=min(32, G * Hkv) // Hkv * Hkv,
                    Hkv=Hkv, D=D, dtype=dt, window=win, sinks=rng.choice([0, 4]) if win else 0,
                    prefix=rng.choice([0, 0, _log_int(rng, 1, 2000)]), lens_seed=seed)
    if op == "append":
        hi = _log_int(rng, 1, 3000)
        return dict(op=op, n=_log_int(rng, 1, 64 if hi < 500 else 12), lo=_log_int(rng, 1, hi),
                    hi=hi, Hq=Hkv * rng.choice([1, 4, 5]), Hkv=Hkv, D=D, page=page, dtype=dt,
                    lens_seed=seed)
    hi = _log_int(rng, 10, 1500)
    c = dict(op=op, n=_log_int(rng, 2, 40), lo=_log_int(rng, 1, hi), hi=hi,
             layers=rng.choice([1, 2, 5, 8]), Hkv=Hkv, D=D, page=page, dtype=dt, lens_seed=seed)
    if op == "fork":
        c["parents"] = _log_int(rng, 1, c["n"])
    return c


# ------------------------------------------------------------------ sizes
def _lengths(case):
    """The case's sequence lengths, spread over the logarithm of [lo, hi]."""
    rng = random.Random(case["lens_seed"])
    n = case["B"] if case["op"] == "decode" else case.get("parents", case["n"])
    return [_log_int(rng, case["lo"], case["hi"]) for _ in range(n)]


def _prefixes(case):
    """Keys before each prompt's first query (chunks of a longer prompt)."""
    rng = random.Random(case["lens_seed"] + 1)
    return [rng.randrange(case["prefix"] + 1) for _ in range(case["n"])]


def _visible(p, nk, window, sinks):
    """Keys a query at position p sees."""
    if window <= 0 or p < window:
        return p + 1
    return window + min(sinks, p + 1 - window)


def _es(case):
    return 2 if case["dtype"] == "bf16" else 4


def _dt(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _max_pages(case, lens):
    return max((x + case["page"] - 1) // case["page"] for x in lens) + 1


def work(case):
    es, lens = _es(case), _lengths(case)
    if case["op"] == "decode":
        vis = sum(_visible(n - 1, n, case["window"], case["sinks"]) for n in lens)
        return {"bytes": vis * 2 * case["Hkv"] * case["D"] * es
                + case["B"] * case["Hq"] * (2 * case["D"] * es + 4),
                "flops": 4 * vis * case["Hq"] * case["D"]}
    if case["op"] == "prefill":
        pre = _prefixes(case)
        pairs = 0
        for n, x in zip(lens, pre):
            pairs += sum(_visible(x + i, x + n, case["window"], case["sinks"]) for i in range(n))
        tq, tk = sum(lens), sum(lens) + sum(pre)
        return {"bytes": es * case["D"] * (2 * tq * case["Hq"] + 2 * tk * case["Hkv"])
                + 4 * tq * case["Hq"],
                "flops": 4 * pairs * case["Hq"] * case["D"]}
    if case["op"] == "append":
        t = sum(lens)
        # k, v and q read; rotated k twice (pages and packed), v and rotated q written
        return {"bytes": t * case["D"] * es * (5 * case["Hkv"] + 2 * case["Hq"]),
                "flops": 3 * t * case["D"] * (case["Hkv"] + case["Hq"])}
    page_bytes = 2 * case["layers"] * case["page"] * case["Hkv"] * case["D"] * es
    if case["op"] == "fork":
        copied = sum(lens[i % len(lens)] % case["page"] > 0 for i in range(case["n"]))
        tables = 4 * case["n"] * _max_pages(case, lens) * 3
        return {"bytes": 2 * copied * page_bytes + tables, "flops": 0}
    moved = len(_fragments(case)[1])
    return {"bytes": 2 * moved * page_bytes + 4 * 4 * _fragments(case)[0], "flops": 0}


def _fragments(case):
    """A pool after sequences came and went: (pages in the pool, ids of the used
    pages that lie beyond the used count)."""
    lens = _lengths(case)
    need = sum((x + case["page"] - 1) // case["page"] for x in lens)
    total = 2 * need + 3
    used = sorted(random.Random(case["lens_seed"] + 2).sample(range(total), need))
    return total, [u for u in used if u >= need]


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(_dt(case))

    lens = _lengths(case)
    st = {"case": case}
    if case["op"] == "prefill":
        pre = _prefixes(case)
        nk = [a + b for a, b in zip(lens, pre)]
        st["lens_q"], st["lens_k"] = lens, nk
        st["q"] = normal(sum(lens), case["Hq"], case["D"])
        st["k"] = normal(sum(nk), case["Hkv"], case["D"])
        st["v"] = normal(sum(nk), case["Hkv"], case["D"])
        if own:
            lcx = _lcx()
            st["plan"] = lcx.VarlenPlan(lens, nk, device="cuda")
            st["rope"] = _rope(case)
        return st

    page = case["page"]
    layers = case.get("layers", 1)
    if case["op"] == "append":
        hist = random.Random(case["lens_seed"] + 3)
        start = [hist.randrange(2000) for _ in lens]
        full = [a + b for a, b in zip(start, lens)]
    else:
        start, full = None, lens
    mp = _max_pages(case, full)
    npg = [(x + page - 1) // page for x in full]
    if case["op"] == "compact":
        total, _ = _fragments(case)
        used = sorted(random.Random(case["lens_seed"] + 2).sample(range(total), sum(npg)))
        order = torch.randperm(sum(npg), generator=g, device="cuda").tolist()
        ids = [used[i] for i in order]
    elif case["op"] == "fork":
        total = sum(npg) + case["n"] + 5
        ids = torch.randperm(total, generator=g, device="cuda").tolist()[:sum(npg)]
    else:
        total = sum(npg) + 1
        ids = torch.randperm(total, generator=g, device="cuda").tolist()[:sum(npg)]
    seqs = len(full) + (case["n"] if case["op"] == "fork" else 0)
    # pools [layer, page, slot, head, D]; each head's slots of a page lie together
    shape = (layers, total, case["Hkv"], page, case["D"])
    st["k_pages"] = normal(*shape).transpose(2, 3)
    st["v_pages"] = normal(*shape).transpose(2, 3)
    table = torch.full((seqs, mp), -1, dtype=torch.int32)
    ref = torch.zeros(total, dtype=torch.int32)
    at = 0
    for s, c in enumerate(npg):
        table[s, :c] = torch.tensor(ids[at:at + c], dtype=torch.int32)
        at += c
    ref[torch.tensor(ids, dtype=torch.long)] = 1
    free = [p for p in range(total - 1, -1, -1) if ref[p] == 0]
    lens_t = torch.zeros(seqs, dtype=torch.int32)
    lens_t[:len(full)] = torch.tensor(full, dtype=torch.int32)
    free_t = torch.full((total,), -1, dtype=torch.int32)
    free_t[:len(free)] = torch.tensor(free, dtype=torch.int32)
    # the bookkeeping in one int32 tensor, as a cache keeps it
    st["meta"] = torch.cat([table.reshape(-1), lens_t, ref, free_t,
                            torch.tensor([len(free)], dtype=torch.int32)]).cuda()
    st["sizes"] = (seqs, mp, total)
    if case["op"] == "decode":
        st["q"] = normal(case["B"], case["Hq"], case["D"])
        st["ids"] = torch.arange(case["B"], dtype=torch.int32, device="cuda")
    elif case["op"] == "append":
        t = sum(lens)
        st["q"] = normal(t, case["Hq"], case["D"])
        st["k"], st["v"] = normal(t, case["Hkv"], case["D"]), normal(t, case["Hkv"], case["D"])
        st["q_out"], st["k_out"] = torch.empty_like(st["q"]), torch.empty_like(st["k"])
        st["ids"] = torch.arange(len(lens), dtype=torch.int32, device="cuda")
        st["start"] = torch.tensor(start, dtype=torch.int32, device="cuda")
        cu = [0]
        for x in lens:
            cu.append(cu[-1] + x)
        st["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
        st["t"] = t
    elif case["op"] == "fork":
        n, par = case["n"], len(lens)
        st["src"] = (torch.arange(n, dtype=torch.int32) % par).cuda()
        st["dst"] = (torch.arange(n, dtype=torch.int32) + par).cuda()
    else:
        st["meta0"] = st["meta"].clone()
    if own:
        lcx = _lcx()
        st["cache"] = lcx.PagedCache(total, page, case["Hkv"], case["D"], seqs, mp,
                                     num_layers=layers, dtype=_dt(case), device="cuda",
                                     k_pages=st["k_pages"], v_pages=st["v_pages"])
        st["cache"].meta.copy_(st["meta"])
        st["meta"] = st["cache"].meta
        st["rope"] = _rope(case)
    return st


def _lcx():
    import ntk_rope_flashattn_b200 as lcx
    return lcx


def _rope(case):
    return _lcx().RopeParams("plain", head_dim=case["D"], base=BASE)


def _views(st):
    """(block table, lengths, reference counts, free stack, free count) of the bookkeeping."""
    seqs, mp, total = st["sizes"]
    m = st["meta"]
    a = seqs * mp
    return (m[:a].view(seqs, mp), m[a:a + seqs], m[a + seqs:a + seqs + total],
            m[a + seqs + total:a + seqs + 2 * total], m[a + seqs + 2 * total:])


# ------------------------------------------------------------------ one pass
def run(st):
    return _run_own(st) if own else _run_plain(st)


def _run_own(st):
    lcx, case = _lcx(), st["case"]
    if case["op"] == "prefill":
        return lcx.attn_varlen(st["q"], st["k"], st["v"], st["plan"], st["rope"],
                               window=case["window"], sinks=case["sinks"], return_lse=True)
    cache = st["cache"]
    if case["op"] == "decode":
        return lcx.paged_decode(cache, st["q"], st["ids"], st["rope"], window=case["window"],
                                sinks=case["sinks"], return_lse=True)
    if case["op"] == "append":
        lcx.paged_append(cache, st["k"], st["v"], st["ids"], st["start"], st["rope"],
                         cu_new=st["cu"], q=st["q"], q_out=st["q_out"], k_out=st["k_out"])
        return st["k_pages"], st["v_pages"], st["q_out"], st["k_out"]
    if case["op"] == "fork":
        lcx.pages_free(cache, st["dst"])
        lcx.pages_fork(cache, st["src"], st["dst"])
    else:
        st["meta"].copy_(st["meta0"])
        lcx.pages_compact(cache)
    return (st["k_pages"], st["v_pages"]) + _views(st)


def _angles(pos, D):
    """cos and sin of pos * theta_i, [T, D/2]: angles and their sines in 64 bits."""
    i = torch.arange(D // 2, device=pos.device, dtype=torch.float64)
    ang = pos.to(torch.float64)[:, None] * (BASE ** (-2.0 * i / D))[None, :]
    return torch.cos(ang).float(), torch.sin(ang).float()


def _rotate(x, pos):
    """x [T, H, D] in fp32 rotated by the positions pos [T]."""
    c, s = _angles(pos, x.shape[-1])
    c, s = c[:, None, :], s[:, None, :]
    a, b = x.float().chunk(2, dim=-1)
    return torch.cat([a * c - b * s, a * s + b * c], dim=-1)


def _keep(qpos, kpos, window, sinks):
    keep = kpos[None, :] <= qpos[:, None]
    if window > 0:
        keep = keep & ((qpos[:, None] - kpos[None, :] < window) | (kpos[None, :] < sinks))
    return keep


def _plain_prefill(st):
    case = st["case"]
    D, G = case["D"], case["Hq"] // case["Hkv"]
    out = torch.empty_like(st["q"])
    lse = torch.empty(case["Hq"], st["q"].shape[0], device="cuda")
    q0 = k0 = 0
    for nq, nk in zip(st["lens_q"], st["lens_k"]):
        kp = torch.arange(nk, device="cuda")
        k = _rotate(st["k"][k0:k0 + nk], kp).transpose(0, 1)            # [Hkv, nk, D]
        v = st["v"][k0:k0 + nk].float().transpose(0, 1)
        step = max(64, (1 << 28) // (nk * case["Hq"]))                  # scores below 1 GB
        for i0 in range(0, nq, step):
            i1 = min(nq, i0 + step)
            qp = torch.arange(i0, i1, device="cuda") + (nk - nq)
            q = _rotate(st["q"][q0 + i0:q0 + i1], qp)                   # [n, Hq, D]
            q = q.view(i1 - i0, case["Hkv"], G, D).permute(1, 2, 0, 3)  # [Hkv, G, n, D]
            kx = min(nk, i1 + nk - nq)                                  # keys anyone here sees
            s = (q.reshape(case["Hkv"], -1, D) @ k[:, :kx].transpose(1, 2)) / math.sqrt(D)
            s = s.view(case["Hkv"], G, i1 - i0, kx)
            s.masked_fill_(~_keep(qp, kp[:kx], case["window"], case["sinks"]), -math.inf)
            m = s.amax(dim=-1, keepdim=True)
            p = s.sub_(m).exp_()
            z = p.sum(dim=-1, keepdim=True)
            o = (p.view(case["Hkv"], -1, kx) @ v[:, :kx]).view(case["Hkv"], G, i1 - i0, D) / z
            out[q0 + i0:q0 + i1] = o.permute(2, 0, 1, 3).reshape(i1 - i0, case["Hq"], D)
            lse[:, q0 + i0:q0 + i1] = (m + z.log()).view(case["Hq"], i1 - i0)
        q0, k0 = q0 + nq, k0 + nk
    return out, lse


def _plain_decode(st):
    case = st["case"]
    D, Hkv, G, page = case["D"], case["Hkv"], case["Hq"] // case["Hkv"], case["page"]
    table, lens, _, _, _ = _views(st)
    q = _rotate(st["q"], lens[:case["B"]] - 1)
    out = torch.empty_like(st["q"])
    lse = torch.empty(case["B"], case["Hq"], device="cuda")
    for b, n in enumerate(_lengths(case)):
        pos = torch.arange(n, device="cuda")
        if case["window"] > 0:
            pos = pos[(pos >= n - case["window"]) | (pos < case["sinks"])]
        pg, slot = table[b].long()[pos // page], pos % page
        k = st["k_pages"][0, pg, slot].float().transpose(0, 1)          # [Hkv, n, D]
        v = st["v_pages"][0, pg, slot].float().transpose(0, 1)
        s = (q[b].view(Hkv, G, D) @ k.transpose(1, 2)) / math.sqrt(D)
        m = s.amax(dim=-1, keepdim=True)
        p = (s - m).exp()
        z = p.sum(dim=-1, keepdim=True)
        out[b] = ((p @ v) / z).view(Hkv * G, D)
        lse[b] = (m + z.log()).view(Hkv * G)
    return out, lse


def _token_places(st):
    """(entry, position) of each packed new token."""
    lens = (st["cu"][1:] - st["cu"][:-1]).long()
    ent = torch.repeat_interleave(torch.arange(lens.numel(), device="cuda"), lens,
                                  output_size=st["t"])
    pos = torch.arange(st["t"], device="cuda") - st["cu"].long()[ent] + st["start"].long()[ent]
    return ent, pos


def _plain_append(st):
    case = st["case"]
    ent, pos = _token_places(st)
    table = _views(st)[0]
    pg, slot = table[st["ids"].long()[ent], pos // case["page"]].long(), pos % case["page"]
    k = _rotate(st["k"], pos).to(_dt(case))
    st["k_pages"][0, pg, slot] = k
    st["v_pages"][0, pg, slot] = st["v"]
    st["k_out"].copy_(k)
    st["q_out"].copy_(_rotate(st["q"], pos))
    return st["k_pages"], st["v_pages"], st["q_out"], st["k_out"]


def _plain_fork(st):
    """Drop the children, then fork them from their parents again: full pages are
    shared, a partial last page is copied to a page from the free stack."""
    page, (seqs, mp, total) = st["case"]["page"], st["sizes"]
    table, lens, ref, free, n_free = _views(st)
    src, dst = st["src"].long(), st["dst"].long()
    # free: freed pages return to the stack in ascending order
    rows = table[dst].long()
    held = torch.zeros(total + 1, dtype=torch.int32, device="cuda")
    held.index_add_(0, torch.where(rows >= 0, rows, total).reshape(-1),
                    torch.ones(rows.numel(), dtype=torch.int32, device="cuda"))
    ref -= held[:total]
    gone = (held[:total] > 0) & (ref == 0)
    stack = torch.cat([free, free.new_full((1,), -1)])
    at = torch.where(gone, n_free + torch.cumsum(gone, 0) - 1, total)
    stack.scatter_(0, at.long(), torch.arange(total, dtype=torch.int32, device="cuda"))
    n = n_free + gone.sum()
    # fork
    ln = lens[src]
    part = ln % page > 0
    full = (ln // page).long()
    j = torch.arange(mp, device="cuda")[None, :]
    new_rows = torch.where(j < full[:, None] + part[:, None], table[src], -1)
    shared = torch.where(j < full[:, None], table[src].long(), total)
    ref_x = torch.cat([ref, ref.new_zeros(1)])
    ref_x.index_add_(0, shared.reshape(-1),
                     torch.ones(shared.numel(), dtype=torch.int32, device="cuda"))
    need = part.sum()
    take = (n - need + torch.cumsum(part, 0) - 1).clamp(min=0).long()
    page_new = stack[take].long()
    w = torch.nonzero(part)[:, 0]
    old = new_rows[w, full[w]].long()
    new_rows[w, full[w]] = page_new[w].int()
    ref_x[page_new[w]] = 1
    st["k_pages"][:, page_new[w]] = st["k_pages"][:, old]
    st["v_pages"][:, page_new[w]] = st["v_pages"][:, old]
    table[dst] = new_rows
    lens[dst] = ln
    ref.copy_(ref_x[:total])
    n = n - need
    i = torch.arange(total, device="cuda")
    free.copy_(torch.where(i < n, stack[:total], -1))
    n_free.copy_(n)


def _plain_compact(st):
    """Used pages beyond the used count move to the holes below it, in order."""
    seqs, mp, total = st["sizes"]
    st["meta"].copy_(st["meta0"])
    table, lens, ref, free, n_free = _views(st)
    used = ref > 0
    u = used.sum()
    i = torch.arange(total, device="cuda")
    movers = torch.nonzero(used & (i >= u))[:, 0]
    holes = torch.nonzero(~used & (i < u))[:, 0]
    to = i.clone()
    to[movers] = holes
    st["k_pages"][:, holes] = st["k_pages"][:, movers]
    st["v_pages"][:, holes] = st["v_pages"][:, movers]
    table.copy_(torch.where(table >= 0, to[table.clamp(min=0).long()].int(), -1))
    ref[holes] = ref[movers]
    ref[movers] = 0
    free.copy_(torch.where(i < total - u, total - 1 - i, -1))
    n_free.copy_(total - u)


def _run_plain(st):
    op = st["case"]["op"]
    if op == "prefill":
        return _plain_prefill(st)
    if op == "decode":
        return _plain_decode(st)
    if op == "append":
        return _plain_append(st)
    _plain_fork(st) if op == "fork" else _plain_compact(st)
    return (st["k_pages"], st["v_pages"]) + _views(st)


# ------------------------------------------------------------------ 64 bits
def _turn64(x, pos):
    """Rotation as a complex product in 64 bits: (a + ib) e^(i pos theta)."""
    h = x.shape[-1] // 2
    th = torch.tensor([BASE ** (-i / h) for i in range(h)], dtype=torch.float64, device=x.device)
    w = torch.polar(torch.ones(len(pos), h, dtype=torch.float64, device=x.device),
                    pos.double().unsqueeze(1) * th)
    z = torch.complex(x[..., :h].double(), x[..., h:].double()) * w.unsqueeze(1)
    return torch.cat([z.real, z.imag], -1)


def exact(case, seed):
    if case["op"] in ("fork", "compact"):
        return None     # page moves: nothing is computed
    if case["op"] == "prefill" and work(case)["flops"] > 3e12:
        return None
    st = prepare(case, seed)
    if case["op"] == "append":
        ent, pos = _token_places(st)
        kp, vp = st["k_pages"].double(), st["v_pages"].double()
        k = _turn64(st["k"], pos)
        table = _views(st)[0].tolist()
        at = list(zip(ent.tolist(), pos.tolist()))
        pages = torch.tensor([table[e][p // case["page"]] for e, p in at], device="cuda")
        slots = torch.tensor([p % case["page"] for _, p in at], device="cuda")
        kp[0].index_put_((pages, slots), k)
        vp[0].index_put_((pages, slots), st["v"].double())
        return kp, vp, _turn64(st["q"], pos), k
    G, D = case["Hq"] // case["Hkv"], case["D"]
    o = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    if case["op"] == "prefill":
        lse = torch.zeros(case["Hq"], o.shape[0], dtype=torch.float64, device="cuda")
        q0 = k0 = 0
        for nq, nk in zip(st["lens_q"], st["lens_k"]):
            kp = torch.arange(nk, device="cuda")
            qp = kp[nk - nq:]
            q, k = _turn64(st["q"][q0:q0 + nq], qp), _turn64(st["k"][k0:k0 + nk], kp)
            keep = _keep(qp, kp, case["window"], case["sinks"])
            for h in range(case["Hq"]):
                x = torch.where(keep, q[:, h] @ k[:, h // G].T / D ** 0.5, -math.inf)
                lse[h, q0:q0 + nq] = torch.logsumexp(x, 1)
                o[q0:q0 + nq, h] = torch.softmax(x, 1) @ st["v"][k0:k0 + nk, h // G].double()
            q0, k0 = q0 + nq, k0 + nk
        return o, lse
    lse = torch.zeros(o.shape[:2], dtype=torch.float64, device="cuda")
    table = _views(st)[0].tolist()
    for b, n in enumerate(_lengths(case)):
        pages = torch.tensor(table[b][:(n + case["page"] - 1) // case["page"]], device="cuda")
        pos = torch.arange(n, device="cuda")
        seen = (pos > n - 1 - case["window"]) | (pos < case["sinks"]) if case["window"] else pos >= 0
        q = _turn64(st["q"][b:b + 1], pos[-1:])[0]
        for h in range(case["Hkv"]):
            k = st["k_pages"][0, :, :, h][pages].reshape(-1, D)[:n][seen].double()
            v = st["v_pages"][0, :, :, h][pages].reshape(-1, D)[:n][seen].double()
            x = q[h * G:(h + 1) * G] @ k.T / D ** 0.5
            lse[b, h * G:(h + 1) * G] = torch.logsumexp(x, 1)
            o[b, h * G:(h + 1) * G] = torch.softmax(x, 1) @ v
    return o, lse
