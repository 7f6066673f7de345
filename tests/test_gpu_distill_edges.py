"""The distillation loss where something goes wrong or its arguments are unusual (needs a GB300)."""
import pytest
import torch

from adapter_gemm_packed_gb300 import _mlora as M

pytestmark = pytest.mark.gpu
DT = {"bf16": (M.MLORA_BF16, torch.bfloat16), "f32": (M.MLORA_F32, torch.float32)}


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from adapter_gemm_packed_gb300 import build
    build.build()


def _case(n, v, k, dtype):
    g = torch.Generator(device="cuda").manual_seed(n + v)
    draw = lambda *s: torch.randn(s, generator=g, device="cuda")
    return (draw(n, v).to(DT[dtype][1]), torch.randint(0, v, (n, k), generator=g, device="cuda", dtype=torch.int32),
            draw(n, k), torch.ones(n, device="cuda"))


def _call(case, dtype, flags, shift=0, grad=True):
    z, ids, teacher, weight = case
    n, v = z.shape
    loss = torch.full((n,), 7.0, device="cuda")
    buf = torch.full((n * v + 8,), 7.0, dtype=z.dtype, device="cuda")[shift:shift + n * v]
    p = M.mlora_distill_problem(n, v, ids.shape[1], DT[dtype][0], 1.0, v, v, flags)
    M.mlora_distill_loss(p, z.data_ptr(), ids.data_ptr(), teacher.data_ptr(), weight.data_ptr(), loss.data_ptr(),
                         buf.data_ptr() if grad else None, torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    return loss, buf.view(n, v)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("v,shift,grad", [(4096, 0, True), (4096, 1, True), (70000, 0, True), (3001, 0, True), (4096, 0, False)])
def test_a_wait_that_gives_up(v, shift, grad, dtype):
    """Every block arms its third slot and copies nothing into it; its waits run out after a millisecond.  Its rows from there
    on (rows of 4096 take one slot) get a loss and a gradient of NaN in every element, rows without weight among them;
    those before are what they are without that, and so is the next call."""
    blocks = 2 * torch.cuda.get_device_properties(0).multi_processor_count
    n = 5 * blocks
    case = _case(n, v, 5, dtype)
    case[3][4 * blocks::7] = 0
    want = _call(case, dtype, 0, shift, grad)
    lost = torch.arange(n, device="cuda") >= (2 * blocks if v < 5000 else 0)
    got = _call(case, dtype, M.MLORA_DEBUG_SHORT_TIMEOUT | M.MLORA_DEBUG_DROP_COPY, shift, grad)
    assert want[0].isfinite().all() and want[1].isfinite().all()
    assert got[0][lost].isnan().all() and torch.equal(got[0][~lost], want[0][~lost])
    if grad:
        assert got[1][lost].isnan().all()
    assert torch.equal(got[1][~lost], want[1][~lost])
    again = _call(case, dtype, 0, shift, grad)
    assert torch.equal(again[0], want[0]) and torch.equal(again[1], want[1])
