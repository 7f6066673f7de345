"""Checks of arguments that need no GPU."""
from types import SimpleNamespace

import pytest
import torch

from adapter_gemm_packed_gb300 import _mlora as M
from adapter_gemm_packed_gb300 import attention as A


@pytest.fixture(scope="module", autouse=True)
def built():
    from adapter_gemm_packed_gb300 import build
    build.build()


def _on_gpu(index, shape=(6, 2, 64), dtype=torch.bfloat16):
    """What the checks look at of a tensor, said to lie on GPU `index` (-1: the host)."""
    t = torch.zeros(shape, dtype=dtype)
    return SimpleNamespace(dtype=dtype, shape=t.shape, device=f"cuda:{index}", stride=t.stride, data_ptr=lambda: 4096,
                           get_device=lambda: index, is_contiguous=t.is_contiguous, dim=t.dim)


def _refused(call, status=M.MLORA_ERR_INVALID):
    with pytest.raises(M.MloraError) as e:
        call()
    assert e.value.status == status


def test_tensors_of_another_device_are_refused():
    heads = lambda t, dev: A._heads(t, "here", "q", 6, 2, 64, torch.bfloat16, dev)
    assert heads(_on_gpu(1), 1).data == 4096
    for got, want in ((1, 0), (0, 1), (-1, 0)):
        _refused(lambda: heads(_on_gpu(got), want))
        _refused(lambda: A._output(_on_gpu(got), None, "here", "q_out", 6, 2, 64, torch.bfloat16, want))
        _refused(lambda: A._vector(_on_gpu(got, (6,), torch.int32), "here", "positions", (6,), torch.int32, want))
    assert A._vector(_on_gpu(1, (6,), torch.int32), "here", "positions", (6,), torch.int32, 1) == 4096


def test_calls_check_against_the_device_they_launch_on(monkeypatch):
    """The stream's device where a stream is given, otherwise the current one; nothing is launched."""
    from adapter_gemm_packed_gb300.distill import distill_loss
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    other = SimpleNamespace(device=torch.device("cuda", 1))
    assert A._launch_device(None) == 0 and A._launch_device(other) == 1
    table = [_on_gpu(0, s, torch.float32) for s in ((64,), (64,), (9, 32), (9, 32))]
    pos = _on_gpu(0, (6,), torch.int32)
    q = _on_gpu(0)
    _refused(lambda: A.qk_norm_rope(q, _on_gpu(1), *table, pos))
    _refused(lambda: A.qk_norm_rope(q, q, *table, _on_gpu(1, (6,), torch.int32)))
    _refused(lambda: A.qk_norm_rope(q, q, *table, pos, stream=other))
    _refused(lambda: A.qk_norm_rope_backward(q, _on_gpu(1), q, q, *table, pos))
    z, ids, teacher = _on_gpu(0, (6, 100)), _on_gpu(0, (6, 3), torch.int32), _on_gpu(0, (6, 3), torch.float32)
    _refused(lambda: distill_loss(_on_gpu(1, (6, 100)), ids, teacher))
    _refused(lambda: distill_loss(z, ids, _on_gpu(1, (6, 3), torch.float32)))
    _refused(lambda: distill_loss(z, ids, teacher, stream=other))


def test_attention_takes_tensors_of_its_plans_device():
    attn = A.WindowAttention([6], 2, 2, 64, 4, device="cuda:1", flags=M.MLORA_PLAN_HOST_ONLY)
    ok, bad = _on_gpu(1), _on_gpu(0)
    for args in ((bad, ok, ok), (ok, bad, ok), (ok, ok, bad)):
        _refused(lambda: attn.forward(*args))
        _refused(lambda: attn.backward(*args, ok, ok))
    _refused(lambda: attn.backward(ok, ok, ok, ok, bad))
    _refused(lambda: A.WindowAttention([6], 2, 2, 64, 4, device="cpu"))
    attn.close()


def _twice(fn, x, *args):
    """A second derivative through a function whose first is the library's: an error, not a constant's."""
    y = fn.apply(*args)
    y = y[0] if isinstance(y, tuple) else y
    (g,) = torch.autograd.grad(y.square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        g.sum().backward()


def test_second_derivatives_are_refused(monkeypatch):
    from adapter_gemm_packed_gb300 import layer as L
    x = lambda *s: torch.randn(s, requires_grad=True)
    attn = SimpleNamespace(_new_saved=lambda: torch.zeros(4), forward=lambda q, k, v, saved: q + k + v,
                           backward=lambda q, k, v, o, do, saved: (do * o, do * o, do * o))
    q, k, v = x(3, 2, 8), x(3, 2, 8), x(3, 2, 8)
    _twice(A._AttentionFn, q, q, k, v, attn)
    monkeypatch.setattr(A, "qk_norm_rope", lambda q, k, *t, **kw: (2 * q, 2 * k))
    monkeypatch.setattr(A, "qk_norm_rope_backward",
                        lambda dq, dk, q, k, *t, weight_grads, **kw: (2 * dq * q, 2 * dk * k, None, None))
    w = torch.ones(8)
    _twice(A._NormRopeFn, q, q, k, w, w, w, w, w, 1e-6, False)
    layer = SimpleNamespace(forward=lambda X, W: X @ W, backward=lambda X, W, dY: dY @ W.T * X)
    X = x(3, 4)
    _twice(L._PackedLoRAFn, X, X, layer, torch.ones(4, 5))


WRAP = 2**32


@pytest.mark.parametrize("kw", [dict(lens=[WRAP + 6]), dict(n_q_heads=WRAP + 2), dict(n_kv_heads=WRAP + 2),
                                dict(head_dim=WRAP + 64), dict(window=-WRAP + 4), dict(n_sink=-WRAP)])
def test_sizes_that_32_bits_do_not_hold_are_refused(kw):
    """They would come around to ordinary ones."""
    args = dict(lens=[6], n_q_heads=2, n_kv_heads=2, head_dim=64, window=4, n_tokens=6, flags=M.MLORA_PLAN_HOST_ONLY)
    A.WindowAttention(**args).close()
    A.WindowAttention(**{**args, "window": 2**40, "n_sink": 2**40}).close()
    _refused(lambda: A.WindowAttention(**{**args, **kw}))


def test_a_vocabulary_that_32_bits_do_not_hold_is_refused(monkeypatch):
    from adapter_gemm_packed_gb300.distill import distill_loss
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    z = _on_gpu(0, (1, 100))
    z.shape, z.stride = torch.Size((1, WRAP + 100)), lambda *i: 1
    _refused(lambda: distill_loss(z, _on_gpu(0, (1, 3), torch.int32), _on_gpu(0, (1, 3), torch.float32)))
    p = M.mlora_distill_problem(1, 2**31 - 200, 3, M.MLORA_BF16, 1.0, 2**31, 2**31)
    _refused(lambda: M.mlora_distill_loss(p, 16, 16, 16, None, 16, 16, None), M.MLORA_ERR_UNSUPPORTED)


def test_norm_sizes_that_32_bits_do_not_hold_are_refused(monkeypatch):
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    w, half = _on_gpu(0, (64,), torch.float32), _on_gpu(0, (9, 32), torch.float32)
    long = _on_gpu(0, (9, 32), torch.float32)
    long.shape = torch.Size((WRAP + 9, 32))
    q, many, pos = _on_gpu(0), _on_gpu(0), _on_gpu(0, (6,), torch.int32)
    many.shape = torch.Size((6, WRAP + 2, 64))
    _refused(lambda: A.qk_norm_rope(q, q, w, w, long, long, pos))
    _refused(lambda: A.qk_norm_rope(many, q, w, w, half, half, pos))
    _refused(lambda: A.qk_norm_rope(q, many, w, w, half, half, pos))


def test_unknown_flags_are_refused():
    ptr, w = M.mlora_heads(4096, 128, 64), 4096
    call = lambda f: M.mlora_qk_norm_rope(M.mlora_rope_problem(4, 2, 2, 64, 64, 16, M.MLORA_BF16, f, 1e-6), ptr, None, w, w, w,
                                          w, w, ptr, ptr, None)
    with pytest.raises(M.MloraError, match="unknown flag"):
        call(2)
    with pytest.raises(M.MloraError, match="k: null"):
        call(M.MLORA_ROPE_INTERLEAVED)
    p = M.mlora_distill_problem(1, 200, 3, M.MLORA_BF16, 1.0, 200, 200, 1 << 20)
    with pytest.raises(M.MloraError, match="unknown flag"):
        M.mlora_distill_loss(p, 16, 16, 16, None, 16, 16, None)
