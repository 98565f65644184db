"""Attention over packed prompts of different lengths: ``VarlenPlan`` and
``attn_varlen`` (see ``lcx_attn_varlen`` in ``include/lcx.h``).

    plan = lcx.VarlenPlan([512, 17, 2048])                # host lengths, once per batch
    o = lcx.attn_varlen(q, k, v, plan, rope)              # q [T, Hq, D], k/v [T, Hkv, D]
"""
import ctypes

import numpy as np

from . import RopeParams, _check, _dtype_code, _RopeParams, load
from .paged import _call_on, _on_device, _packer, _raw, _rope_c

LCX_VARLEN_PREROTATED = 1
LCX_VARLEN_TEST_STALL = 0x80000000

_P, _I64, _I32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32


class _Info(ctypes.Structure):
    _fields_ = [("n_seqs", _I64), ("total_q", _I64), ("total_k", _I64), ("max_k", _I64),
                ("n_units", _I64 * 2), ("ints", _I64)]


class _VarlenArgs(ctypes.Structure):
    _fields_ = [("q", _P), ("k", _P), ("v", _P), ("o", _P), ("lse", _P), ("plan", _P),
                ("workspace", _P), ("workspace_bytes", _I64), ("dev_status", _P), ("info", _Info),
                ("dtype", _I32), ("causal", _I32), ("Tq", _I64), ("Tk", _I64), ("Hq", _I64),
                ("Hkv", _I64), ("D", _I64), ("q_strides", _I64 * 3), ("k_strides", _I64 * 3),
                ("v_strides", _I64 * 3), ("o_strides", _I64 * 3), ("rope", _RopeParams),
                ("window", _I64), ("sinks", _I64), ("softmax_scale", ctypes.c_float),
                ("flags", ctypes.c_uint32), ("watchdog_ms", _I32), ("reserved0", _I32)]


_pack_args = _packer(_VarlenArgs)


def _declare(lib):
    lib.lcx_varlen_plan_ints.argtypes = [_P, _P, _I64]
    lib.lcx_varlen_plan_ints.restype = _I64
    lib.lcx_varlen_plan.argtypes = [_P, _P, _I64, _P, _I64, ctypes.POINTER(_Info)]
    lib.lcx_varlen_plan.restype = ctypes.c_int
    lib.lcx_varlen_workspace_bytes.argtypes = [ctypes.POINTER(_Info), _I64, _I64, _I32]
    lib.lcx_varlen_workspace_bytes.restype = _I64
    lib.lcx_attn_varlen.argtypes = [ctypes.POINTER(_VarlenArgs), _P]
    lib.lcx_attn_varlen.restype = ctypes.c_int


class VarlenPlan:
    """The work layout of packed sequences (``lcx_varlen_plan``): ``seqlens_q[s]``
    query rows and ``seqlens_k[s]`` key rows each (the same when not given), host
    integers.  One plan serves every layer of a batch; it does not change."""

    def __init__(self, seqlens_q, seqlens_k=None, device="cuda"):
        import torch
        device = torch.device(device)
        if device.type == "cuda" and device.index is None:
            device = torch.device("cuda", torch.cuda.current_device())
        lens = []
        for x in (seqlens_q, seqlens_q if seqlens_k is None else seqlens_k):
            if isinstance(x, torch.Tensor) and x.is_cuda:
                raise ValueError("sequence lengths are host integers (got a CUDA tensor)")
            a = np.asarray(x).reshape(-1)
            if a.size and (a.dtype.kind not in "iu" or a.min() < 0 or a.max() > 2 ** 30):
                raise ValueError("sequence lengths must be integers in [0, 2^30]")
            lens.append(np.ascontiguousarray(a, np.int32))
        if lens[0].size != lens[1].size:
            raise ValueError("seqlens_q and seqlens_k must have the same length")
        n, pq, pk = lens[0].size, lens[0].ctypes.data, lens[1].ctypes.data
        ints = int(load().lcx_varlen_plan_ints(pq, pk, n))
        if ints < 0:
            raise ValueError("sequence lengths sum to more than 2^30")
        host = torch.zeros(ints, dtype=torch.int32)
        self.info = _Info()
        _check(load().lcx_varlen_plan(pq, pk, n, host.data_ptr(), ints, ctypes.byref(self.info)))
        self._info_bytes = bytes(self.info)
        self.device = device
        self.plan = host.to(device)
        self.total_q, self.total_k = int(self.info.total_q), int(self.info.total_k)
        self._workspace_bytes = {}

    @property
    def cu_q(self):
        """int32 [n + 1] device tensor: first packed query row of each sequence."""
        n = int(self.info.n_seqs)
        return self.plan[8:8 + n + 1]

    @property
    def cu_k(self):
        """int32 [n + 1] device tensor: first packed key row of each sequence."""
        n = int(self.info.n_seqs)
        return self.plan[9 + n:9 + n + n + 1]


def varlen_workspace_bytes(plan: VarlenPlan, kv_heads: int, head_dim: int, dtype) -> int:
    """Workspace bytes of ``attn_varlen`` (lcx_varlen_workspace_bytes)."""
    need = plan._workspace_bytes.get((kv_heads, head_dim, dtype))
    if need is None:
        import torch
        code = {torch.bfloat16: 0, torch.float32: 1}.get(dtype, -1)
        need = int(load().lcx_varlen_workspace_bytes(ctypes.byref(plan.info), int(kv_heads),
                                                     int(head_dim), code))
        if need < 0:
            raise ValueError("attn_varlen: %s kv heads, head_dim %s, %s are not supported" %
                             (kv_heads, head_dim, dtype))
        plan._workspace_bytes[(kv_heads, head_dim, dtype)] = need
    return need


def attn_varlen(q, k, v, plan: VarlenPlan, rope: RopeParams, causal: bool = True, window: int = 0,
                sinks: int = 0, softmax_scale: float = 0.0, return_lse: bool = False,
                prerotated: bool = False, out=None, lse=None, workspace=None, status=None,
                watchdog_ms: int = 0, _test_stall: bool = False):
    """Fused RoPE + causal attention over the plan's packed sequences.

    q [Tq, Hq, D], k/v [Tk, Hkv, D] CUDA tensors (bf16 or fp32, last dim
    contiguous) holding the sequences one behind the other; query i of a sequence
    sits at position len_k - len_q + i, key j at j.  Returns o [Tq, Hq, D] (and
    lse [Hq, Tq] fp32 if asked); rows behind the last sequence are left as they
    were (zero when the call allocates o and lse itself).  ``prerotated``: q and k
    are already rotated
    (``paged_append``'s q_out and k_out); otherwise the keys are rotated once into
    ``workspace`` (uint8, 256-byte aligned, ``varlen_workspace_bytes``; allocated when
    not given; calls in flight at the same time, replayed graphs among them, must not
    share one).  A query without a visible key gets
    o = 0 and lse = -inf.  ``out`` does not overlap k or v.  ``status`` and ``watchdog_ms`` as for ``attn_fwd``."""
    import torch
    dev = q.get_device()
    if q.dim() != 3 or k.dim() != 3 or v.dim() != 3 or dev < 0:
        raise ValueError("q, k, v must be 3-D CUDA tensors [tokens, heads, D]")
    Tq, Hq, D = q.shape
    Tk, Hkv, Dk = k.shape
    if Dk != D or v.shape != k.shape:
        raise ValueError("shape mismatch: q %s k %s v %s" % (q.shape, k.shape, v.shape))
    if not (q.dtype == k.dtype == v.dtype):
        raise ValueError("q, k, v must share a dtype")
    _on_device(dev, k=k, v=v, out=out, lse=lse, workspace=workspace, status=status,
               plan=plan.plan)
    alloc = q.new_empty if plan.total_q == Tq else q.new_zeros
    o = out if out is not None else alloc((Tq, Hq, D))
    if o.shape != q.shape or o.dtype != q.dtype:
        raise ValueError("out must be shaped like q")
    if return_lse and lse is None:
        lse = alloc((Hq, Tq), dtype=torch.float32)
    if lse is not None and (lse.shape != (Hq, Tq) or lse.dtype != torch.float32 or
                            not lse.is_contiguous()):
        raise ValueError("lse must be contiguous fp32 [%d, %d]" % (Hq, Tq))
    if status is not None and (status.dtype != torch.int32 or status.numel() < 1):
        raise ValueError("status must be an int32 tensor")
    if workspace is None and not prerotated and rope.mode != "none":
        workspace = k.new_empty(max(varlen_workspace_bytes(plan, Hkv, D, k.dtype), 1),
                                dtype=torch.uint8)
    ws, size = (0, 0) if workspace is None else (workspace.data_ptr(), workspace.nbytes)
    owner, rope_c = _rope_c(rope)      # (alive during the call: it owns factor tables)
    a = _pack_args(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(),
        0 if lse is None else lse.data_ptr(), plan.plan.data_ptr(), ws, size,
        0 if status is None else status.data_ptr(), plan._info_bytes, _dtype_code(q),
        1 if causal else 0, Tq, Tk, Hq, Hkv, D, *q.stride(), *k.stride(), *v.stride(),
        *o.stride(), rope_c, int(window), int(sinks), float(softmax_scale),
        (LCX_VARLEN_PREROTATED if prerotated else 0) |
        (LCX_VARLEN_TEST_STALL if _test_stall else 0), int(watchdog_ms), 0)
    _call_on(dev, _raw("lcx_attn_varlen", 1), a)
    return (o, lse) if return_lse else o
