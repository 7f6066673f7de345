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
        _refused(lambda: A._output(_on_gpu(got), "here", "q_out", 6, 2, 64, torch.bfloat16, want))
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
