"""Qi21Runner over the 4-bit prefix cache on the GPU: whole images with eviction at
sizes where the workspace grows, and buffers on several streams."""
import pytest
import torch

from qi21_synth import configs as C

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from prefix_kv_cached_b200 import build
    build.build()
    from prefix_kv_cached_b200 import binding
    return binding


@pytest.fixture(scope="module")
def mid(B):
    """The mid workload in bf16 with device-drawn weights."""
    from prefix_kv_cached_b200.runner import Qi21Runner
    w = C.make_workload("mid")
    return Qi21Runner(w, B.QI21_DTYPE_BF16, weights=C.device_weights(w, torch.bfloat16, "cuda"))


def _inputs(r, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    sh = r.shape
    return (torch.randn(r.Bn, r.P, sh.d_model, device="cuda", generator=gen),
            torch.randn(r.Bn, r.N, sh.latent_ch, device="cuda", generator=gen))


def test_image_goes_on_after_an_eviction_that_needs_more_workspace(B, mid):
    """512 rows kept to 333 at 8 x 256 target rows: the step over fewer rows needs a
    larger workspace than the one before."""
    need = [B.qi21_kv4_step_workspace_bytes(mid.cfg, mid.Bn, p, mid.N) for p in (mid.P, 333)]
    assert need[1] > need[0]
    pre, x0 = _inputs(mid)
    x = mid.denoise_kv4(pre, x0, mid.w.sigmas[:4], keep=333, n_protected=256)
    B.check("device", B.qi21_check_device_error(mid.kv4_ws, mid.kv4_ws.numel(), mid.stream))
    assert mid.kv4.n_prefix == 333 and mid.kv4_ws.numel() >= need[1] and x.isfinite().all()
