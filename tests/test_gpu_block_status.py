"""What a training step says of waits inside its kernels (needs a GB300)."""
import pytest
import torch

from adapter_gemm_packed_gb300 import _mlora as M

pytestmark = pytest.mark.gpu


def test_status_of_a_step():
    """After ordinary steps all is well, and a pack's or the attention's report is handed on."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from adapter_gemm_packed_gb300 import build
    from adapter_gemm_packed_gb300.block import DistilledAttention
    build.build()
    g = torch.Generator(device="cuda").manual_seed(1)
    draw = lambda *s: (torch.randn(s, generator=g, device="cuda") * 0.1).bfloat16()
    b = DistilledAttention(draw(256, 128), draw(128, 128), draw(500, 128).narrow(0, 0, 496).contiguous(), 4, 2, 32,
                           [[40, 9], [30]], [8, 4], [1.0, 1.0], 20, 1)
    ids = torch.randint(0, 496, (79, 3), generator=g, device="cuda", dtype=torch.int32)
    for _ in range(2):
        loss, dx = b.step(draw(79, 128), ids, torch.randn((79, 3), generator=g, device="cuda"))
    assert b.sync_status() == M.MLORA_OK and loss.isfinite().all() and dx.isfinite().all()
    for part in (b.head, b.attention):
        part.sync_status, kept = (lambda stream=None: M.MLORA_ERR_TIMEOUT), part.sync_status
        assert b.sync_status() == M.MLORA_ERR_TIMEOUT
        part.sync_status = kept
    assert b.sync_status() == M.MLORA_OK
    b.close()
