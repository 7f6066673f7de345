"""Between the packed projections: norms of queries and keys with their rotation, and windowed attention.

The tensors are PyTorch views ``[n_tokens, n_heads, head_dim]`` of packed rows: columns of a
shared-input pack's output as they are (``Y[:, :4096].view(N, 32, 128)``), or tensors of their own.
Arguments are checked here for what the C ABI cannot see (types, shapes, devices); the arithmetic is
in the library's kernels.  Outputs that are not given are allocated; with ``stream`` (a
``torch.cuda.Stream``) everything runs, and is allocated, on that stream, otherwise on the current one.
"""
from __future__ import annotations

import contextlib
import itertools

import torch
from torch.autograd.function import once_differentiable

from . import _mlora as M
from .layer import _DT


def _refuse(where: str, text: str, status: int = M.MLORA_ERR_INVALID):
    raise M.MloraError(status, where, text)


def _launch_device(stream) -> int:
    """Index of the device that a call's kernels run on: the stream's, or the current one."""
    return torch._C._cuda_getDevice() if stream is None else stream.device.index


def _heads(t, where: str, name: str, n: int, h: int, d: int, dt, dev: int) -> M.mlora_heads:
    """The C descriptor of a [n, h, d] tensor on device ``dev``."""
    if t.dtype is not dt or t.get_device() != dev:
        _refuse(where, f"{name} must be a {dt} tensor on GPU {dev}, got {t.dtype} on {t.device}")
    if t.shape != (n, h, d):
        _refuse(where, f"{name} must be of shape {(n, h, d)}, got {tuple(t.shape)}")
    s = t.stride()
    if s[2] != 1 and d > 1:
        _refuse(where, f"{name}: the elements of a head vector must be contiguous")
    return M.mlora_heads(t.data_ptr(), s[0], s[1])


def _output(t, device, where: str, name: str, n: int, h: int, d: int, dt, dev: int):
    """An output: the caller's, or a new one where that is None; and its C descriptor."""
    if t is not None:
        return t, _heads(t, where, name, n, h, d, dt, dev)
    t = torch.empty((n, h, d), dtype=dt, device=device)
    return t, M.mlora_heads(t.data_ptr(), h * d, d)


def _vector(t, where: str, name: str, shape, dt, dev: int) -> int:
    if t.dtype is not dt or t.get_device() != dev or t.shape != shape or not t.is_contiguous():
        _refuse(where, f"{name} must be a contiguous {dt} tensor of shape {tuple(shape)} on GPU {dev}, "
                       f"got {t.dtype} {tuple(t.shape)} on {t.device}")
    return t.data_ptr()


def _int32(where: str, name: str, v) -> int:
    """A size for a 32-bit field of the C ABI, where a larger one would wrap around."""
    v = int(v)
    if not -2**31 <= v < 2**31:
        _refuse(where, f"{name} = {v} does not fit in 32 bits")
    return v


def _gradient(t):
    """A gradient as autograd hands it over, laid out for the kernels: it may be a slice of a larger one, at any
    element, or broadcast."""
    t = t.contiguous()
    return t if t.data_ptr() % 16 == 0 else t.clone()


class _on:
    """Run a call's allocations on the stream that its kernels use, of device ``dev``."""

    def __init__(self, stream, dev):
        self.ctx = None if stream is None else torch.cuda.stream(stream)
        self.dev = dev

    def __enter__(self):
        if self.ctx is not None:
            self.ctx.__enter__()
        # (torch.cuda.current_stream().cuda_stream, without the two objects on the way: 0.3 microseconds for 3)
        return torch._C._cuda_getCurrentRawStream(self.dev)

    def __exit__(self, *exc):
        if self.ctx is not None:
            self.ctx.__exit__(*exc)


# ------------------------------------------------------------------ norms with rotation

def _rope_problem(where, q, k, wq, wk, cos, sin, positions, eps, interleaved, dev):
    if q.dim() != 3 or k.dim() != 3:
        _refuse(where, "q and k must be [n_tokens, n_heads, head_dim]")
    n, hq, d = q.shape
    hk, dt = k.shape[1], q.dtype
    if dt is torch.bfloat16:
        code = M.MLORA_BF16
    elif dt is torch.float32:
        code = M.MLORA_F32
    else:
        _refuse(where, f"q and k are bf16 or fp32, not {dt}", M.MLORA_ERR_UNSUPPORTED)
    if cos.dim() != 2:
        _refuse(where, "cos and sin must be [positions, rot_dim / 2]")
    rows, half = cos.shape
    if hq | hk | d | half | rows >= 2**30:      # 32-bit fields, where a larger size would wrap around
        _refuse(where, f"a size of {(hq, hk, d, rows, half)} is out of range")
    p = M.mlora_rope_problem(n, hq, hk, d, 2 * half, rows, code, M.MLORA_ROPE_INTERLEAVED if interleaved else 0, eps)
    f32 = torch.float32
    tables = (_vector(wq, where, "wq", (d,), f32, dev), _vector(wk, where, "wk", (d,), f32, dev),
              _vector(cos, where, "cos", (rows, half), f32, dev), _vector(sin, where, "sin", (rows, half), f32, dev),
              _vector(positions, where, "positions", (n,), torch.int32, dev))
    return p, (n, hq, d, dt, dev), (n, hk, d, dt, dev), tables


def qk_norm_rope(q, k, wq, wk, cos, sin, positions, *, eps=1e-6, interleaved=False, q_out=None, k_out=None,
                 stream=None):
    """Root-mean-square norm of every query and key head vector, times ``wq`` / ``wk`` (fp32
    [head_dim]), and the rotation of its first ``2 * cos.shape[1]`` elements by the angles that
    ``cos`` / ``sin`` (fp32 [positions, rot_dim / 2]) hold for the token's position (int32
    [n_tokens]).  Returns (q_out, k_out)."""
    where = "qk_norm_rope"
    dev = _launch_device(stream)
    p, sq, sk, tables = _rope_problem(where, q, k, wq, wk, cos, sin, positions, eps, interleaved, dev)
    hq, hk = _heads(q, where, "q", *sq), _heads(k, where, "k", *sk)
    with _on(stream, dev) as s:
        q_out, oq = _output(q_out, q.device, where, "q_out", *sq)
        k_out, ok = _output(k_out, q.device, where, "k_out", *sk)
        M.mlora_qk_norm_rope(p, hq, hk, *tables, oq, ok, s)
    return q_out, k_out


def qk_norm_rope_backward(dq_out, dk_out, q, k, wq, wk, cos, sin, positions, *, eps=1e-6, interleaved=False, dq=None,
                          dk=None, weight_grads=True, stream=None):
    """Gradients of :func:`qk_norm_rope` from those of its outputs and from its inputs.  Returns
    (dq, dk, dwq, dwk); the weights' gradients are None with ``weight_grads=False`` (frozen norms)."""
    where = "qk_norm_rope_backward"
    dev = _launch_device(stream)
    p, sq, sk, tables = _rope_problem(where, q, k, wq, wk, cos, sin, positions, eps, interleaved, dev)
    args = (_heads(dq_out, where, "dq_out", *sq), _heads(dk_out, where, "dk_out", *sk), _heads(q, where, "q", *sq),
            _heads(k, where, "k", *sk))
    with _on(stream, dev) as s:
        dq, oq = _output(dq, q.device, where, "dq", *sq)
        dk, ok = _output(dk, q.device, where, "dk", *sk)
        dwq = dwk = ws = None
        if weight_grads:
            dwq = torch.empty(sq[2], dtype=torch.float32, device=q.device)
            dwk = torch.empty(sq[2], dtype=torch.float32, device=q.device)
            ws = torch.empty(M.mlora_qk_norm_rope_workspace(p), dtype=torch.uint8, device=q.device)
        M.mlora_qk_norm_rope_backward(p, *args, *tables, oq, ok,
                                      *(None if t is None else t.data_ptr() for t in (dwq, dwk, ws)), s)
    return dq, dk, dwq, dwk


class _NormRopeFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, wq, wk, cos, sin, positions, eps, interleaved):
        ctx.save_for_backward(q, k, wq, wk, cos, sin, positions)
        ctx.opt = dict(eps=eps, interleaved=interleaved)
        return qk_norm_rope(q, k, wq, wk, cos, sin, positions, **ctx.opt)

    @staticmethod
    @once_differentiable
    def backward(ctx, dq_out, dk_out):
        need = ctx.needs_input_grad[2] or ctx.needs_input_grad[3]
        dq, dk, dwq, dwk = qk_norm_rope_backward(_gradient(dq_out), _gradient(dk_out), *ctx.saved_tensors,
                                                 weight_grads=need, **ctx.opt)
        return dq, dk, dwq, dwk, None, None, None, None, None


class QKNormRope(torch.nn.Module):
    """:func:`qk_norm_rope` as a module: fp32 weights ``wq`` / ``wk`` and the tables of the rotation
    with frequencies ``base ** (-2 i / rot_dim)``; ``mod(q, k, positions)`` is differentiable."""

    def __init__(self, head_dim, max_pos, rot_dim=None, base=10000.0, eps=1e-6, interleaved=False, device="cuda"):
        super().__init__()
        rot_dim = head_dim if rot_dim is None else rot_dim
        self.eps, self.interleaved = eps, interleaved
        self.wq = torch.nn.Parameter(torch.ones(head_dim, device=device))
        self.wk = torch.nn.Parameter(torch.ones(head_dim, device=device))
        freq = float(base) ** (-torch.arange(rot_dim // 2, dtype=torch.float64) * 2.0 / rot_dim)
        ang = torch.arange(max_pos, dtype=torch.float64)[:, None] * freq
        self.register_buffer("cos", ang.cos().float().to(device), persistent=False)
        self.register_buffer("sin", ang.sin().float().to(device), persistent=False)

    def forward(self, q, k, positions):
        return _NormRopeFn.apply(q, k, self.wq, self.wk, self.cos, self.sin, positions, self.eps, self.interleaved)


# ------------------------------------------------------------------ attention

class WindowAttention:
    """Causal attention within each sequence of a pack: token i sees the ``window`` tokens up to
    itself and the sequence's first ``n_sink`` tokens.

    ``lens`` are the sequences' lengths, ``starts`` their first rows (default: one behind the other)
    and ``n_tokens`` the rows of the pack (default: up to the last sequence's end); rows of no
    sequence get zero outputs and gradients.  The plan is built once; :meth:`forward` keeps the
    softmax statistics in ``self.saved``, so each forward is followed by its own :meth:`backward`
    before the next one, on one stream.  Calling the object is differentiable and keeps the
    statistics with the graph instead."""

    def __init__(self, lens, n_q_heads, n_kv_heads, head_dim, window, n_sink=0, scale=None, dtype="bf16", starts=None,
                 n_tokens=None, device="cuda", flags=0):
        if dtype not in ("bf16", "f32"):
            _refuse("WindowAttention", f"queries, keys and values are bf16 or f32, not {dtype}", M.MLORA_ERR_UNSUPPORTED)
        here = "WindowAttention"
        lens = [_int32(here, "a sequence's length", n) for n in lens]
        if starts is None:
            starts = list(itertools.accumulate(lens, initial=0))[:len(lens)]
        starts = [int(s) for s in starts]
        if len(starts) != len(lens):
            _refuse("WindowAttention", "starts and lens differ in length")
        if n_tokens is None:
            n_tokens = max((s + n for s, n in zip(starts, lens)), default=0)
        code, self.tdtype = _DT[dtype]
        host = flags & M.MLORA_PLAN_HOST_ONLY
        self.device = torch.device(device)
        if not host:      # the plan's tables go where the tensors are
            if self.device.type != "cuda":
                _refuse("WindowAttention", f"the device must be a GPU, not {device}")
            dev = torch.cuda.current_device() if self.device.index is None else self.device.index
            self.device = torch.device("cuda", dev)
        self.n = int(n_tokens)
        self.hq, self.hk = _int32(here, "n_q_heads", n_q_heads), _int32(here, "n_kv_heads", n_kv_heads)
        self.d = _int32(here, "head_dim", head_dim)
        self.scale = self.d ** -0.5 if scale is None else float(scale)
        self.plan = None
        # (a window or a number of first tokens beyond every length is no different from a smaller one)
        window, n_sink = (_int32(here, *x) for x in (("window", min(int(window), 2**31 - 1)),
                                                     ("n_sink", min(int(n_sink), 2**31 - 1))))
        p = M.mlora_attention_problem(self.n, self.hq, self.hk, self.d, window, n_sink, code, self.scale, flags)
        with contextlib.nullcontext() if host else torch.cuda.device(self.device):
            self.plan = M.mlora_attention_plan(p, starts, lens)
        self.saved_elems = max(4, M.mlora_attention_kept_elems(self.plan))
        self.work_elems = M.mlora_attention_workspace_elems(self.plan)
        self.saved = None if host else self._new_saved()
        self.dev = self.device.index or 0
        self.qs, self.ks = ((self.n, h, self.d, self.tdtype, self.dev) for h in (self.hq, self.hk))

    def _new_saved(self):
        return torch.empty(self.saved_elems, dtype=torch.float32, device=self.device)

    def _saved_ptr(self, t, where):
        """The statistics' buffer: the object's own, or the caller's, of ``saved_elems`` floats."""
        if t is None:
            return None if self.saved is None else self.saved.data_ptr()
        if not (t.dtype is torch.float32 and t.device == self.device and t.is_contiguous()
                and t.numel() >= self.saved_elems):
            _refuse(where, f"saved must be a contiguous fp32 tensor of {self.saved_elems} elements on {self.device}")
        return t.data_ptr()

    def forward(self, q, k, v, out=None, stream=None, saved=None):
        """Outputs [n_tokens, n_q_heads, head_dim].  ``saved`` (fp32, ``saved_elems`` elements) takes the
        statistics instead of ``self.saved``; the backward is given the same buffer."""
        w = "WindowAttention.forward"
        a = (_heads(q, w, "q", *self.qs), _heads(k, w, "k", *self.ks), _heads(v, w, "v", *self.ks))
        with _on(stream, self.dev) as s:
            out, o = _output(out, self.device, w, "out", *self.qs)
            M.mlora_attention_forward(self.plan, *a, o, self._saved_ptr(saved, w), s)
        return out

    def backward(self, q, k, v, out, dout, dq=None, dk=None, dv=None, stream=None, saved=None):
        """(dq, dk, dv) from the forward's inputs and output and the output's gradient."""
        w = "WindowAttention.backward"
        a = (_heads(q, w, "q", *self.qs), _heads(k, w, "k", *self.ks), _heads(v, w, "v", *self.ks),
             _heads(out, w, "out", *self.qs), _heads(dout, w, "dout", *self.qs))
        with _on(stream, self.dev) as s:
            dq, oq = _output(dq, self.device, w, "dq", *self.qs)
            dk, ok = _output(dk, self.device, w, "dk", *self.ks)
            dv, ov = _output(dv, self.device, w, "dv", *self.ks)
            # scratch for the sums of long pieces, handed back with the call
            work = torch.empty(self.work_elems, dtype=torch.float32, device=self.device) if self.work_elems else None
            M.mlora_attention_backward_ws(self.plan, *a, self._saved_ptr(saved, w),
                                          None if work is None else work.data_ptr(), oq, ok, ov, s)
        return dq, dk, dv

    def __call__(self, q, k, v):
        return _AttentionFn.apply(q, k, v, self)

    def sync_status(self, stream=None) -> int:
        with _on(stream, self.dev) as s:
            return M.mlora_attention_sync_status(self.plan, s)

    def close(self):
        if getattr(self, "plan", None):
            M.mlora_attention_plan_destroy(self.plan)
            self.plan = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class _AttentionFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, attn):
        saved = attn._new_saved()
        out = attn.forward(q, k, v, saved=saved)
        ctx.save_for_backward(q, k, v, out, saved)
        ctx.attn = attn
        return out

    @staticmethod
    @once_differentiable
    def backward(ctx, dout):
        q, k, v, out, saved = ctx.saved_tensors
        return (*ctx.attn.backward(q, k, v, out, _gradient(dout), saved=saved), None)
