"""Qi21Runner over the 4-bit prefix cache on the GPU: whole images with eviction at
sizes where the workspace grows, and buffers on several streams."""
import pytest
import torch

from qi21_synth import configs as C
from tests import _kv4

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


WAIT = 400_000_000          # cycles that a stream is held up for: some 0.2 s


def _quantised(r, pre):
    r.set_prefix_row()
    r.prefix_extract(pre)
    r.quantise_prefix()
    r.set_target_row(r.w.sigmas[0])


def test_eviction_on_another_stream_keeps_what_it_reads(B, mid):
    """The buffers that an eviction drops belong to the stream they were allocated on.
    While the eviction waits on another one, that stream's next allocations must not
    be given their memory."""
    r, keep = mid, 100
    pre, x0 = _inputs(r, 1)
    v = torch.empty_like(x0)
    _quantised(r, pre)
    r.cached_step_kv4(x0, v, accumulate=True)
    torch.cuda.synchronize()
    old = [(t.data_ptr(), t.numel() * t.element_size()) for t in (r.kv4_buf, r.kv4_scores)]
    L, H, Dh = r.cfg.n_layers, r.cfg.n_heads, r.cfg.head_dim
    vals = _kv4.read_values(r.kv4_buf, L, r.Bn, H, r.P, Dh)
    rows = _kv4.evict(r.kv4_scores.cpu().numpy(), None, keep, 7)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(WAIT)
        kept = r.evict_prefix(keep, 7)
    taken = [torch.full((n,), 0x7F, dtype=torch.uint8, device="cuda") for _, n in old for _ in range(2)]
    assert not side.query()                               # the eviction has not run yet
    for t in taken:
        assert all(t.data_ptr() + t.numel() <= p or p + n <= t.data_ptr() for p, n in old)
    torch.cuda.synchronize()
    assert (kept.cpu().numpy() == rows).all()
    got = _kv4.read_values(r.kv4_buf, L, r.Bn, H, keep, Dh)
    for l, b, h in ((0, 0, 0), (L - 1, r.Bn - 1, H - 1), (3, 5, 7)):
        assert (got[l, :, b, h] == vals[l, :, b, h][:, rows[l, b, h]]).all()


def test_requantising_under_a_step_on_another_stream(B, mid):
    """quantise_prefix replaces the 4-bit cache and its workspace; a step on another
    stream that still reads the ones before gives what it gives alone."""
    r = mid
    pre, x0 = _inputs(r, 2)
    want, v = torch.empty_like(x0), torch.empty_like(x0)
    _quantised(r, pre)
    r.cached_step_kv4(x0, want)
    torch.cuda.synchronize()
    old = [(t.data_ptr(), t.numel()) for t in (r.kv4_buf, r.kv4_ws)]
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(WAIT)
        r.cached_step_kv4(x0, v)
    r.quantise_prefix()
    taken = [torch.full((n,), 0x7F, dtype=torch.uint8, device="cuda") for _, n in old for _ in range(2)]
    assert not side.query()
    for t in [r.kv4_buf, r.kv4_ws] + taken:
        assert all(t.data_ptr() + t.numel() <= p or p + n <= t.data_ptr() for p, n in old)
    torch.cuda.synchronize()
    # bf16: the GEMMs add their last partial tiles in no fixed order
    assert (v - want).norm() < 1e-2 * want.norm()


@pytest.fixture(scope="module")
def small(B):
    """Three requests of the small64 workload in float32, whose steps give the same bits every time."""
    import dataclasses
    from prefix_kv_cached_b200.runner import Qi21Runner
    w = dataclasses.replace(C.make_workload("small64"), batch=3)
    return Qi21Runner(w, B.QI21_DTYPE_F32, host_weights=C.host_weights(w, "float32"))


@pytest.mark.parametrize("shared", [False, True])
def test_release_frees_the_extracted_cache_and_its_workspace(B, small, shared):
    """The steps, the eviction and the modulation rows go on without them, to the same
    bits, and the next image extracts into new ones."""
    from prefix_kv_cached_b200.runner import Qi21Runner
    r = Qi21Runner(small.w, B.QI21_DTYPE_F32, share_weights_with=small, shared_prefix=shared)
    pre, x0 = _inputs(r, 3)
    pre = pre[:1].contiguous() if shared else pre
    ordinary = r.denoise(pre, x0, r.w.sigmas[:3])
    want = r.denoise_kv4(pre, x0, r.w.sigmas[:4], keep=30, n_protected=7)
    held = r.cache_buf.numel() + r.ws.numel()
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    got = r.denoise_kv4(pre, x0, r.w.sigmas[:4], keep=30, n_protected=7, release=True)
    torch.cuda.synchronize()
    assert before - torch.cuda.memory_allocated() >= held - 4 * got.numel() - 1024      # `got` is new
    assert torch.equal(got, want)
    with pytest.raises(ValueError, match="released"):
        r.cached_step(x0, torch.empty_like(x0))
    assert torch.equal(r.denoise_kv4(pre, x0, r.w.sigmas[:4], keep=30, n_protected=7, release=True), want)
    assert torch.equal(r.denoise(pre, x0, r.w.sigmas[:3]), ordinary)                    # extracted anew
    r.check_device()


def test_release_under_a_step_on_another_stream(B, small):
    """An ordinary step on another stream still reads the extracted cache when it is
    released: its memory stays out of use until the step is done."""
    from prefix_kv_cached_b200.runner import Qi21Runner
    r = Qi21Runner(small.w, B.QI21_DTYPE_F32, share_weights_with=small)
    pre, x0 = _inputs(r, 4)
    want, v = torch.empty_like(x0), torch.empty_like(x0)
    _quantised(r, pre)
    r.cached_step(x0, want)
    torch.cuda.synchronize()
    old = [(t.data_ptr(), t.numel()) for t in (r.cache_buf, r.ws)]
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(WAIT)
        r.cached_step(x0, v)
    r.quantise_prefix(release=True)
    taken = [torch.full((n,), 0x7F, dtype=torch.uint8, device="cuda") for _, n in old]
    assert not side.query()
    for t in taken:
        assert all(t.data_ptr() + t.numel() <= p or p + n <= t.data_ptr() for p, n in old)
    torch.cuda.synchronize()
    assert torch.equal(v, want)


def test_captured_steps_add_to_the_weights_of_the_one_before(B, small):
    """A captured step adds its weights at every replay; the step that would make the
    weights, and so clear them at every replay, is refused in a capture."""
    from prefix_kv_cached_b200.runner import Qi21Runner
    r = Qi21Runner(small.w, B.QI21_DTYPE_F32, share_weights_with=small)
    pre, x0 = _inputs(r, 5)
    v = torch.empty_like(x0)
    _quantised(r, pre)
    r.cached_step_kv4(x0, v)                               # sets kernel attributes
    torch.cuda.synchronize()

    def capture(g):
        with torch.cuda.graph(g, capture_error_mode="thread_local"):
            v.zero_()
            r.cached_step_kv4(x0, v, accumulate=True)

    with pytest.raises(ValueError, match="capture"):
        capture(torch.cuda.CUDAGraph())
    assert r.kv4_scores is None
    r.cached_step_kv4(x0, v, accumulate=True)
    one = r.kv4_scores.clone()
    g = torch.cuda.CUDAGraph()
    capture(g)
    g.replay()
    g.replay()
    torch.cuda.synchronize()
    # three float32 sums, each off by 2^-24 of it at most, against three times the first
    assert ((r.kv4_scores - 3 * one).abs() <= 3 * 2.0 ** -23 * one).all() and (one > 0).any()
    del g
