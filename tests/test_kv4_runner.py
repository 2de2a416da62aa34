"""What Qi21Runner does on the host around the 4-bit cache's calls: the buffers it
holds, without a GPU. The library's launches are replaced; its size queries and
argument checks are the real ones."""
import pytest
import torch

from qi21_synth import configs as C

H32 = C.ModelShape(4096, 32, 128, 1, 8192, 64, 256)
H16 = C.ModelShape(1024, 16, 64, 1, 2048, 64, 256)


@pytest.fixture
def B(monkeypatch):
    from prefix_kv_cached_b200 import build
    build.build()
    from prefix_kv_cached_b200 import binding, runner

    def extracted(cache4):
        cache4.state = binding.QI21_CACHE_EXTRACTED
        return binding.QI21_OK

    monkeypatch.setattr(binding, "qi21_kv4_quantize", lambda cfg, src, dst, stream=0: extracted(dst))
    monkeypatch.setattr(binding, "qi21_kv4_evict",
                        lambda cfg, src, scores, keep, prot, dst, kept, stream=0: extracted(dst))
    monkeypatch.setattr(runner.Qi21Runner, "stream", 0)
    return binding


def _runner(B, shape, batch, P, N, shared=False):
    """A runner as its constructor leaves it, without weights or a GPU."""
    from prefix_kv_cached_b200.runner import Qi21Runner, make_config
    r = object.__new__(Qi21Runner)
    r.device, r.cfg = torch.device("cpu"), make_config(shape, B.QI21_DTYPE_BF16)
    r.Bn, r.P, r.N, r.shared_prefix = batch, P, N, shared
    r.kv4 = r.kv4_buf = r.kv4_scores = r.kv4_ws = None
    r._allocate()
    return r


def _evict(r, keep):
    k = r.kv4
    r.kv4_scores = torch.zeros(k.n_layers, k.batch, k.n_heads, k.n_prefix)
    r.evict_prefix(keep)


# the first three, the fourth's queries and the last one's partial results grow as the prefix shrinks
@pytest.mark.parametrize("shape,batch,P,N,keeps", [
    (H32, 1, 8192, 1024, (4096,)), (H32, 1, 6400, 1024, (4800, 1000, 1)), (H32, 1, 12000, 1100, (6000,)),
    (H16, 4, 1159, 512, (565, 3)), (C.MID, 8, 512, 256, (511, 333, 256, 100, 1)), (H16, 1, 4096, 4096, (2048,)),
    (C.SMALL, 2, 198, 300, (99, 1)), (H32, 1, 4608, 4096, (4607, 2304, 1))])
@pytest.mark.parametrize("shared", [False, True])
def test_workspace_holds_the_step_after_every_eviction(B, shape, batch, P, N, keeps, shared):
    r = _runner(B, shape, batch, P, N, shared)
    r.quantise_prefix()
    assert r.kv4_ws.numel() >= B.qi21_kv4_step_workspace_bytes(r.cfg, batch, P, N)
    for keep in keeps:
        _evict(r, keep)
        assert r.kv4.n_prefix == keep
        assert r.kv4_ws.numel() >= B.qi21_kv4_step_workspace_bytes(r.cfg, batch, keep, N), keep


def test_calls_without_a_4_bit_prefix_are_refused(B):
    """The constructor's runner (its buffers are not needed here) has no 4-bit prefix."""
    from prefix_kv_cached_b200 import runner
    w = C.make_workload("small64")
    r = runner.Qi21Runner(w, B.QI21_DTYPE_F32, device="cpu", host_weights=C.host_weights(w, "float32"))
    x = torch.zeros(r.Bn, r.N, r.shape.latent_ch)
    with pytest.raises(ValueError, match="quantise_prefix"):
        r.cached_step_kv4(x, x)
    with pytest.raises(ValueError):
        r.evict_prefix(3)


def test_a_refused_quantisation_or_eviction_keeps_the_cache_before_it(B, monkeypatch):
    r = _runner(B, C.SMALL, 2, 198, 300)
    r.kv4 = r.kv4_buf = r.kv4_scores = r.kv4_ws = None
    with monkeypatch.context() as m:
        m.setattr(B, "qi21_kv4_quantize", lambda *a: B.QI21_ERR_CACHE_STATE)
        with pytest.raises(B.Qi21Error):
            r.quantise_prefix()
    assert r.kv4 is None and r.kv4_buf is None
    r.quantise_prefix()
    k = r.kv4
    r.kv4_scores = torch.zeros(k.n_layers, k.batch, k.n_heads, k.n_prefix)
    before = (r.kv4, r.kv4_buf, r.kv4_scores, r.kv4_ws)
    with monkeypatch.context() as m:
        m.setattr(B, "qi21_kv4_quantize", lambda *a: B.QI21_ERR_CACHE_STATE)      # a failed extract, say
        m.setattr(B, "qi21_kv4_evict", lambda *a: B.QI21_ERR_SHAPE)               # more protected than kept
        for call in (r.quantise_prefix, lambda: r.evict_prefix(5, 6)):
            with pytest.raises(B.Qi21Error):
                call()
            assert all(a is b for a, b in zip(before, (r.kv4, r.kv4_buf, r.kv4_scores, r.kv4_ws)))


@pytest.mark.parametrize("shared", [False, True])
def test_release_gives_the_extracted_cache_back(B, shared):
    r = _runner(B, C.SMALL, 2, 198, 300, shared)
    size = r.cache_buf.numel()
    r.quantise_prefix()
    assert r.cache_buf is not None and r.ws is not None              # kept unless asked
    old = r.cache
    old.state = B.QI21_CACHE_EXTRACTED
    r.quantise_prefix(release=True)
    assert r.cache_buf is None and r.ws is None
    assert old.state == B.QI21_CACHE_EMPTY and not old.base          # no address of freed memory is left
    x = torch.zeros(1)
    for call in (lambda: r.cached_step(x, x), r.cache_kv, r.quantise_prefix):
        with pytest.raises(ValueError, match="released"):
            call()
    _evict(r, 50)                                                    # the 4-bit cache goes on
    assert r.kv4.n_prefix == 50
    # the workspace of the modulation is part of every step's
    assert r.kv4_ws.numel() >= B.qi21_workspace_bytes(r.cfg, 1, 0, 1)
    r._extracting()                                                  # as every call does that fills the cache
    assert r.cache_buf.numel() == size and r.ws.numel() == r.ws_bytes and r.cache.state == B.QI21_CACHE_EMPTY


def test_check_device_reads_what_the_4_bit_steps_reported(B, monkeypatch):
    """The error word at a workspace's start: of both workspaces, and of those that a
    quantisation, an eviction or a release has dropped."""
    def check(ws, ws_bytes, stream=0):
        found = ws[0].item()
        ws[0] = 0
        return B.QI21_ERR_DEVICE_TIMEOUT if found else B.QI21_OK

    monkeypatch.setattr(B, "qi21_check_device_error", check)
    r = _runner(B, C.MID, 8, 512, 256)
    r.check_device()
    r.quantise_prefix()
    for drop in (lambda: None, r.quantise_prefix, lambda: _evict(r, 333), lambda: r.quantise_prefix(release=True)):
        r.check_device()
        r.kv4_ws[0] = 1
        drop()
        with pytest.raises(B.Qi21Error):
            r.check_device()
    r._extracting()
    for drop in (lambda: None, lambda: r.quantise_prefix(release=True)):
        r.check_device()
        r.ws[0] = 1
        drop()
        with pytest.raises(B.Qi21Error):
            r.check_device()


def test_a_copy_of_the_prefix_is_paid_for_where_it_is_faster(B):
    """The attention over a long prefix in the 4-bit cache's own workspace up to 2048
    rows; the bf16 copy of the layer (twice 33792 rows of 4096) only above."""
    cfg, copy = _runner(B, H32, 1, 1, 1).cfg, 2 * 33792 * 4096 * 2
    assert B.qi21_kv4_workspace_bytes(cfg, 1, 2048, 33792, 2048) < copy // 10
    assert copy < B.qi21_kv4_workspace_bytes(cfg, 1, 4096, 33792, 4096) < copy + (1 << 20)
