"""The operators of one training step put together: packed q/k/v projections, norms and rotation of queries and
keys, windowed attention over each job's samples, the packed output projection, a packed head and the distillation
loss, forward and backward, with AdamW on every job's adapters.

It is the example of how the calls fit: queries, keys and values are read where the q/k/v pack wrote them, and their
gradients are written where its backward reads them, without a copy in between.  Everything runs, and is allocated, on
the current stream."""
from __future__ import annotations

import torch

from .attention import WindowAttention, _launch_device, _refuse, qk_norm_rope, qk_norm_rope_backward
from .distill import distill_loss
from .layer import PackedLoRA


class DistilledAttention:
    """``samples[j]``: the lengths of job j's samples, packed one behind the other; ``ranks`` / ``scales``: one
    per job, of all its adapters.  The frozen bf16 weights ``Wqkv`` [(hq + 2 hk) d, d_model], ``Wo`` [d_model, hq d]
    and ``Wh`` [vocab, d_model] are held as given.  Adapters start without effect (A drawn from ``seed``, B zero);
    ``wq`` / ``wk`` are the norms' weights, frozen unless the caller uses their gradients ``dwq`` / ``dwk``."""

    def __init__(self, Wqkv, Wo, Wh, n_q_heads, n_kv_heads, head_dim, samples, ranks, scales, window, n_sink=0,
                 base=10000.0, eps=1e-6, seed=0):
        self.Wqkv, self.Wo, self.Wh = Wqkv, Wo, Wh
        self.hq, self.hk, self.d, self.eps = n_q_heads, n_kv_heads, head_dim, eps
        dev, d_model, vocab = Wqkv.device, Wqkv.shape[1], Wh.shape[0]
        if any(w.get_device() != _launch_device(None) for w in (Wqkv, Wo, Wh)):
            _refuse("DistilledAttention", "the weights must be on the current GPU, where the packs' plans are built")
        tokens = [sum(s) for s in samples]
        lens = [n for s in samples for n in s]
        widths = [n_q_heads * head_dim, n_kv_heads * head_dim, n_kv_heads * head_dim]
        per = lambda x: [[v] * 3 for v in x]
        self.qkv = PackedLoRA(d_model, sum(widths), per(ranks), tokens, per(scales), "bf16", dev, groups=widths)
        self.out = PackedLoRA(widths[0], d_model, ranks, tokens, scales, "bf16", dev)
        self.head = PackedLoRA(d_model, vocab, ranks, tokens, scales, "bf16", dev)
        self.packs = (self.qkv, self.out, self.head)
        g = torch.Generator(device=dev).manual_seed(seed)
        for p in self.packs:
            for a in p.At:
                a.normal_(0.0, a.shape[1] ** -0.5, generator=g)
        self.attention = WindowAttention(lens, n_q_heads, n_kv_heads, head_dim, window, n_sink=n_sink, device=dev)
        self.wq, self.wk = torch.ones(head_dim, device=dev), torch.ones(head_dim, device=dev)
        self.dwq = self.dwk = None
        freq = float(base) ** (-torch.arange(head_dim // 2, dtype=torch.float64) * 2.0 / head_dim)
        ang = torch.arange(max(lens), dtype=torch.float64)[:, None] * freq
        self.cos, self.sin = ang.cos().float().to(dev), ang.sin().float().to(dev)
        self.positions = torch.cat([torch.arange(n, dtype=torch.int32) for n in lens]).to(dev)
        self.t = 0

    def _split(self, Y):
        """Queries, keys and values as columns of the pack's rows."""
        a, b, n = self.hq * self.d, (self.hq + self.hk) * self.d, Y.shape[0]
        return Y[:, :a].view(n, self.hq, self.d), Y[:, a:b].view(n, self.hk, self.d), Y[:, b:].view(n, self.hk, self.d)

    def forward(self, X):
        """Logits [n_tokens, vocab] of the packed rows X."""
        self.X, self.Y = X, self.qkv.forward(X, self.Wqkv)
        q, k, v = self._split(self.Y)
        self.qr, self.kr = qk_norm_rope(q, k, self.wq, self.wk, self.cos, self.sin, self.positions, eps=self.eps)
        self.o = self.attention.forward(self.qr, self.kr, v)
        self.mid = self.out.forward(self.o.view(len(X), -1), self.Wo)
        return self.head.forward(self.mid, self.Wh)

    def backward(self, dlogits):
        """Gradient at X; the adapters' are left in the packs' dAt / dBt, the norms' in dwq / dwk."""
        n = len(dlogits)
        dmid = self.head.backward(self.mid, self.Wh, dlogits)
        do = self.out.backward(self.o.view(n, -1), self.Wo, dmid).view(n, self.hq, self.d)
        q, k, v = self._split(self.Y)
        dY = torch.empty_like(self.Y)
        dq, dk, dv = self._split(dY)
        gq, gk, _ = self.attention.backward(self.qr, self.kr, v, self.o, do, dv=dv)
        _, _, self.dwq, self.dwk = qk_norm_rope_backward(gq, gk, q, k, self.wq, self.wk, self.cos, self.sin,
                                                         self.positions, eps=self.eps, dq=dq, dk=dk)
        return self.qkv.backward(self.X, self.Wqkv, dY)

    def step(self, X, ids, teacher, weight=None, temperature=1.0, lr=1e-3, betas=(0.9, 0.999), eps=1e-8,
             weight_decay=0.0):
        """One training step; returns (loss of every token, gradient at X).  Nothing in it waits for the device: should a
        wait inside a kernel give up (a device that does not answer; never in ordinary work), the distillation's shows as
        NaN in the loss and so in the adapters, the others' in :meth:`sync_status`, for which a caller that keeps
        checkpoints asks before writing one."""
        loss, dlogits = distill_loss(self.forward(X), ids, teacher, weight, temperature=temperature)
        dX = self.backward(dlogits)
        self.t += 1
        for p in self.packs:
            p.adamw(lr, betas[0], betas[1], eps, weight_decay, self.t)
        return loss, dX

    def sync_status(self) -> int:
        """Wait for the current stream; ``MLORA_ERR_TIMEOUT`` if a wait in the packs' or the attention's kernels has
        given up since the last call, otherwise ``MLORA_OK``."""
        return max(p.sync_status() for p in (*self.packs, self.attention))

    def close(self):
        for p in (*self.packs, self.attention):
            p.close()
