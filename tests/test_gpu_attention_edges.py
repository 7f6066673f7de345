"""Rows, sizes and arguments at which the attention and the norms can go wrong (needs a GB300)."""
import pytest
import torch

from adapter_gemm_packed_gb300 import _mlora as M
import op_reference as R

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from adapter_gemm_packed_gb300 import build
    build.build()


def _draw(shape, seed, dt, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(dt).cuda()


# ------------------------------------------------------------------ rows that see one key

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("hq,hk,d", [(4, 2, 64), (3, 3, 128), (8, 1, 72)])
@pytest.mark.parametrize("lens,window,sinks", [([1] * 20, 1, 0), ([1] * 5, 40, 3), ([300, 1, 65, 129], 1, 0),
                                               ([200, 1, 64, 3], 50, 0), ([130, 1, 2], 1, 2), ([1, 400, 1], 10**6, 5)])
def test_gradients_of_rows_that_see_one_key_are_zero(lens, window, sinks, hq, hk, d, dtype):
    """The softmax of one score is 1 whatever the score: dq of such a row is zero, and dk of a key that only such rows
    see; exactly, at scores of any size.  Values and outputs pass through: dv is the rows' sum, the output v."""
    from adapter_gemm_packed_gb300.attention import WindowAttention
    attn = WindowAttention(lens, hq, hk, d, window, n_sink=sinks, dtype=dtype)
    q, k, v, do = (_draw((attn.n, h, d), i, DT[dtype], 3.0) for i, h in enumerate((hq, hk, hk, hq)))
    o = attn.forward(q, k, v)
    dq, dk, dv = attn.backward(q, k, v, o, do)
    alone_q, alone_k, at = [], [], 0
    for n in lens:
        rows = list(range(at, at + n))
        alone_q += rows if window == 1 and sinks == 0 else rows[:1]
        alone_k += rows if window == 1 and sinks == 0 or n == 1 else []
        at += n
    assert (dq[alone_q] == 0).all()
    assert (dk[alone_k] == 0).all()
    assert torch.equal(o[alone_k], v[alone_k].repeat_interleave(hq // hk, 1))
    terms = do[alone_k].double().view(-1, hk, hq // hk, d)
    want = terms.sum(2)      # one rounding, and fp32 sums of a few terms
    assert ((dv[alone_k].double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -18 * terms.abs().sum(2)).all()
    others = [r for r in range(attn.n) if r not in set(alone_q)]
    assert all((dq[r] != 0).any() for r in others)
    assert attn.sync_status() == M.MLORA_OK
    attn.close()
