"""Plain 64-bit forms of the paged-cache and packed-prompt operators, for the
tests, with error bounds derived from the arithmetic that the calls document.

Bound of an attention output.  Let every product q'_d k'_d of a logit carry a
relative error u_s, so the logit moves by at most E = u_s c sum_d |q'_d k'_d|
(E_max the largest of a row), and every weight another relative error u_p.  The
normalised weights then move by a factor within exp(+-2 E_max) (1 +- 2 u_p), so
|o - o_ref| <= (expm1(2 E_max) + 2 u_p) sum_j p_j |v_j|, plus u_o |o_ref| for the
rounding of the output, and lse by E_max + u_p.  u = eps / 2 of the type an
operand is rounded to:
  bf16 operand 2^-8 (two rounded operands: 2^-7 with the second-order term in
  the slack below), two bf16 parts 2^-16, two tf32 parts 2^-22, fp32 2^-24; an fp32
  sum of n terms adds n 2^-24.
"""
import math

import torch

U_OUT = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def table64(rope):
    """(theta'_i, mscale) in 64 bits."""
    import oracle
    t, ms = oracle.rope_theta_ext(rope.mode, rope.head_dim, rope.base, rope.scale,
                                  rope.original_max_pos, rope.alpha, rope.beta,
                                  seq_len=rope.seq_len, factors=rope.factors,
                                  factors_short=rope.factors_short)
    return torch.from_numpy(t).double(), float(ms)


def rotate(x, pos, rope, scaled=True):
    """x [T, H, D] double rotated at positions pos [T] (times mscale when scaled)."""
    th, ms = table64(rope)
    if rope.mode == "none":
        return x.double().clone()
    ang = pos.double()[:, None] * th[None, :]
    c, s = torch.cos(ang)[:, None, :], torch.sin(ang)[:, None, :]
    x = x.double()
    y = torch.empty_like(x)
    if rope.pairing == "half":
        h = x.shape[-1] // 2
        a, b = x[..., :h], x[..., h:]
        y[..., :h], y[..., h:] = a * c - b * s, a * s + b * c
    else:
        a, b = x[..., 0::2], x[..., 1::2]
        y[..., 0::2], y[..., 1::2] = a * c - b * s, a * s + b * c
    return y * (ms if scaled else 1.0)


def attend(q, k, v, qpos, causal, window, sinks, scale):
    """q [n, Hq, D], k, v [m, Hkv, D] (rotated, double) -> o, lse [Hq, n], the mix
    sum p|v| [n, Hq, D] and the row's largest sum of |products| [Hq, n]."""
    n, Hq, D = q.shape
    m, Hkv = k.shape[0], k.shape[1]
    G = Hq // Hkv
    o, mix = torch.zeros_like(q), torch.zeros_like(q)
    lse = torch.full((Hq, n), -math.inf, dtype=torch.float64)
    prod = torch.zeros((Hq, n), dtype=torch.float64)
    if m == 0 or n == 0:
        return o, lse, mix, prod
    kpos = torch.arange(m)
    keep = torch.ones((n, m), dtype=torch.bool)
    if causal:
        keep = kpos[None, :] <= qpos[:, None]
    if window > 0:
        keep = keep & ((qpos[:, None] - kpos[None, :] < window) | (kpos[None, :] < sinks))
    for h in range(Hq):
        kk, vv = k[:, h // G], v[:, h // G]
        s = torch.where(keep, scale * (q[:, h] @ kk.T), torch.tensor(-math.inf).double())
        some = keep.any(1)
        mx = torch.where(some, s.max(1).values, torch.zeros(n).double())
        p = torch.where(keep, torch.exp(s - mx[:, None]), torch.zeros(()).double())
        z = p.sum(1)
        zz = torch.where(some, z, torch.ones(n).double())
        o[:, h] = (p @ vv) / zz[:, None]
        mix[:, h] = (p @ vv.abs()) / zz[:, None]
        lse[h] = torch.where(some, mx + torch.log(zz), torch.tensor(-math.inf).double())
        prod[h] = torch.where(keep, scale * (q[:, h].abs() @ kk.abs().T),
                              torch.zeros(()).double()).max(1).values
    return o, lse, mix, prod


def bounds(o, lse, mix, prod, u_s, u_p, u_o):
    """(bound of o, bound of lse) of attend()'s results."""
    E = u_s * prod + 2.0 ** -22 * (1.0 + lse.abs().nan_to_num(posinf=0.0, neginf=0.0))
    w = torch.expm1(2 * E) + 2 * u_p
    return w.T[:, :, None] * mix + u_o * o.abs() + 1e-30, E + u_p + 1e-30


def check(got_o, got_lse, want, u_s, u_p, label=""):
    o, lse, mix, prod = want
    bo, bl = bounds(o, lse, mix, prod, u_s, u_p, U_OUT[got_o.dtype])
    err = (got_o.double().cpu() - o).abs()
    print("[serving] %s: o max %.3g, of its bound at most %.2f" % (
        label, float(err.max()) if err.numel() else 0.0,
        float((err / bo).max()) if err.numel() else 0.0))
    assert torch.isfinite(got_o.float()).all()
    assert (err <= bo).all(), "o: %.3g beyond its bound" % float((err - bo).max())
    gl = got_lse.double().cpu()
    none = torch.isinf(lse)
    assert torch.equal(torch.isinf(gl) & (gl < 0), none)
    if (~none).any():
        assert ((gl - lse).abs()[~none] <= bl[~none]).all(), "lse"


class PlainPages:
    """The bookkeeping of a page cache in plain Python, as lcx.h defines it."""

    def __init__(self, P, ps, S, MP):
        self.P, self.ps, self.S, self.MP = P, ps, S, MP
        self.table = [[-1] * MP for _ in range(S)]
        self.lens = [0] * S
        self.ref = [0] * P
        self.free = list(range(P - 1, -1, -1))
        self.status = 0
        self.copies = []            # (src page, dst page) of the last call

    def _flag(self, code):
        self.status = max(self.status, code)

    def _pages(self, n):
        return -(-n // self.ps)

    def extend(self, ids, counts):
        avail, total, plan, start = len(self.free), 0, [], []
        for i, s in enumerate(ids):
            st = -1
            if s >= 0:
                if s >= self.S or counts[i] < 0 or s in ids[:i] or \
                        self.lens[s] + counts[i] > self.MP * self.ps:
                    self._flag(1)
                else:
                    need = self._pages(self.lens[s] + counts[i]) - self._pages(self.lens[s])
                    total += need
                    if need == 0 or total <= avail:
                        plan.append((s, counts[i], need))
                        st = self.lens[s]
                    else:
                        self._flag(5)
            start.append(st)
        taken = sum(p[2] for p in plan)
        block = self.free[len(self.free) - taken:]
        self.free = self.free[:len(self.free) - taken]
        for s, c, need in plan:
            at = self._pages(self.lens[s])
            for k in range(need):
                page, block = block[0], block[1:]
                self.table[s][at + k] = page
                self.ref[page] = 1
            self.lens[s] += c
        return start

    def fork(self, src, dst):
        lens, avail, need, plan = list(self.lens), len(self.free), 0, []
        self.copies = []
        for i, (a, b) in enumerate(zip(src, dst)):
            if a < 0 or b < 0:
                continue
            if a >= self.S or b >= self.S or lens[b] != 0 or b in dst[:i]:
                self._flag(1)
                continue
            part = lens[a] % self.ps > 0
            need += part
            if part and need > avail:
                self._flag(5)
                continue
            plan.append((a, b, part))
        taken = sum(p[2] for p in plan)
        block = self.free[len(self.free) - taken:]
        self.free = self.free[:len(self.free) - taken]
        rows = [list(r) for r in self.table]
        for a, b, part in plan:
            full = lens[a] // self.ps
            for j in range(full):
                self.table[b][j] = rows[a][j]
                self.ref[rows[a][j]] += 1
            if part:
                page, block = block[0], block[1:]
                self.table[b][full] = page
                self.ref[page] = 1
                self.copies.append((rows[a][full], page))
            self.lens[b] = lens[a]

    def release(self, ids):
        gone = []
        for i, s in enumerate(ids):
            if s < 0:
                continue
            if s >= self.S or s in ids[:i]:
                self._flag(1)
                continue
            for j, page in enumerate(self.table[s]):
                if page >= 0:
                    self.ref[page] -= 1
                    if self.ref[page] == 0:
                        gone.append(page)
                    self.table[s][j] = -1
            self.lens[s] = 0
        self.free += sorted(gone)

    def compact(self):
        used = [p for p in range(self.P) if self.ref[p] > 0]
        U = len(used)
        movers = [p for p in used if p >= U]
        holes = [p for p in range(U) if self.ref[p] == 0]
        to = dict(zip(movers, holes))
        self.copies = list(to.items())
        self.table = [[to.get(p, p) for p in r] for r in self.table]
        for a, b in to.items():
            self.ref[b], self.ref[a] = self.ref[a], 0
        self.free = list(range(self.P - 1, U - 1, -1))

    def equal(self, cache):
        free = self.free + [-1] * (self.P - len(self.free))
        assert cache.block_table.tolist() == self.table
        assert cache.seq_lens.tolist() == self.lens
        assert cache.ref_counts.tolist() == self.ref
        assert cache.n_free.tolist() == [len(self.free)]
        assert cache.free_pages.tolist() == free
