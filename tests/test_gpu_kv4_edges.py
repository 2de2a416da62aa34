"""Edges of the 4-bit prefix cache and of the caches it is read from and written to:
memory that the caller never cleared, scores that are not finite, lengths."""
import dataclasses

import numpy as np
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


@pytest.fixture
def mode(request, B):
    """(dtype, torch dtype); switches the kernel family for the test."""
    B.qi21_set_tensor_cores(0 if request.param == "bf16_cuda_cores" else 1)
    yield (B.QI21_DTYPE_F32, torch.float32) if request.param == "f32" else (B.QI21_DTYPE_BF16, torch.bfloat16)
    B.qi21_set_tensor_cores(1)


def _np(t):
    return t.double().cpu().numpy()


def _rel(a, b):
    return float((a.double() - b.double()).norm() / b.double().norm())


# ------------------------------------------------------------------ memory that nobody cleared

@pytest.mark.parametrize("mode", ["f32", "bf16", "bf16_cuda_cores"], indirect=True)
@pytest.mark.parametrize("name", ["small64", "small"])
def test_shared_prefix_rows_behind_the_prefix_are_never_read(B, mode, name):
    """A shared-prefix cache in memory full of NaNs, filled by an extract and by the way
    back from 4 bits: rows [P, Pp) keep their NaNs, and the step gives what it gives in
    cleared memory (P 130 or 198: the last key tile of the prefix ends behind them)."""
    dtype, tdt = mode
    from prefix_kv_cached_b200.runner import Qi21Runner
    w = dataclasses.replace(C.make_workload(name), batch=2)
    r = Qi21Runner(w, dtype, host_weights=C.host_weights(w, "float32" if tdt == torch.float32 else "bfloat16"),
                   shared_prefix=True)
    assert r.P % 128
    pre = torch.randn(1, r.P, r.shape.d_model, device="cuda")
    x0 = torch.randn(2, r.N, r.shape.latent_ch, device="cuda")
    v, want = torch.empty_like(x0), torch.empty_like(x0)
    r.set_prefix_row()
    r.set_target_row(w.sigmas[0])

    def pads():
        return [t[:, r.P:-(-r.P // 128) * 128] for t in r.cache_kv()]

    def steps(fill):
        r.cache_buf.fill_(fill)
        r.prefix_extract(pre)
        r.cached_step(x0, v)
        a = v.clone()
        r.quantise_prefix()
        r.cache_buf.fill_(fill)
        B.check("dequantize", B.qi21_kv4_dequantize(r.cfg, r.kv4, r.cache, r.stream))
        r.cached_step(x0, v)
        return a, v.clone()

    want = steps(0)
    got = steps(0xFF)
    assert all(t.isnan().all() for t in pads())
    for a, b in zip(got, want):
        assert a.isfinite().all()
        # float32 steps give the same bits; bf16 ones agree to the order of the GEMMs' last sums
        assert torch.equal(a, b) if tdt == torch.float32 else _rel(a, b) < 1e-2
    # a request that is not finite leaves the others as they are
    x0[1] = float("nan")
    r.cached_step(x0, v)
    assert v[1].isnan().all() and (torch.equal(v[0], want[1][0]) if tdt == torch.float32 else
                                   _rel(v[0], want[1][0]) < 1e-2)


# ------------------------------------------------------------------ lengths

def _cfg(B, dtype, H, Dh, L=1):
    return B.qi21_config(H * Dh, H, Dh, L, 2 * H * Dh, 64, 256, dtype, 0, 1e-6, 1e-6)


def _stream():
    return torch.cuda.current_stream().cuda_stream


def test_the_way_back_of_lengths_is_no_extracted_cache(B):
    """The ordinary step attends to all n_prefix rows of every item; a cache in which
    the rows behind the lengths were never written is refused until the caller says
    that it is whole."""
    cfg = _cfg(B, B.QI21_DTYPE_BF16, 4, 64)
    src = torch.randn(1, 2, 2, 30 + 1, 256, device="cuda").bfloat16()
    cache = B.qi21_kv_cache_init(src, cfg, 2, 30, 1)
    cache.state = B.QI21_CACHE_EXTRACTED
    back = torch.zeros_like(src)
    for lens, state in ((None, B.QI21_CACHE_EXTRACTED), ([30, 11, 0, 0], B.QI21_CACHE_EMPTY)):
        lt = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
        buf = torch.zeros(B.qi21_kv4_cache_bytes(cfg, 2, 30), dtype=torch.uint8, device="cuda")
        k4 = B.qi21_kv4_cache_init(buf, cfg, 2, 30, lt)
        assert B.qi21_kv4_quantize(cfg, cache, k4, _stream()) == B.QI21_OK
        cb = B.qi21_kv_cache_init(back, cfg, 2, 30, 1)
        assert B.qi21_kv4_dequantize(cfg, k4, cb, _stream()) == B.QI21_OK
        assert cb.state == state
        again = B.qi21_kv4_cache_init(torch.zeros_like(buf), cfg, 2, 30, lt)
        if lens is not None:
            assert B.qi21_kv4_quantize(cfg, cb, again, _stream()) == B.QI21_ERR_CACHE_STATE
    torch.cuda.synchronize()


# ------------------------------------------------------------------ scores that are not finite

@pytest.mark.parametrize("mode", ["f32", "bf16", "bf16_cuda_cores"], indirect=True)
@pytest.mark.parametrize("H,Dh,N,P,T", [(2, 128, 1, 300, 140), (4, 64, 12, 300, 140), (2, 128, 60, 300, 140),
                                        (4, 64, 200, 300, 140), (32, 128, 1025, 300, 140), (16, 64, 1200, 130, 129)])
def test_an_infinite_score_makes_its_rows_nan(B, mode, H, Dh, N, P, T):
    """One tail key after the other with an infinity in a head's last dim. A row whose
    score there is +inf has the weight inf / inf: NaN, in the result and the log-sum-exp,
    wherever the key lies in its tile; one whose score is -inf stays finite."""
    dtype, tdt = mode
    cfg = _cfg(B, dtype, H, Dh)
    gen = torch.Generator(device="cuda").manual_seed(N)
    src = torch.randn(1, 2, 1, P + 1, H * Dh, device="cuda", generator=gen).to(tdt)
    cache = B.qi21_kv_cache_init(src, cfg, 1, P, 1)
    cache.state = B.QI21_CACHE_EXTRACTED
    buf = torch.zeros(B.qi21_kv4_cache_bytes(cfg, 1, P), dtype=torch.uint8, device="cuda")
    k4 = B.qi21_kv4_cache_init(buf, cfg, 1, P)
    B.check("quantize", B.qi21_kv4_quantize(cfg, cache, k4, _stream()))
    q, kt, vt = (torch.randn(1, n, H * Dh, device="cuda", generator=gen).to(tdt) for n in (N, T, T))
    q = torch.where(q == 0, torch.ones_like(q), q)                     # 0 * inf would be another NaN
    n = B.qi21_kv4_workspace_bytes(cfg, 1, N, P, T)
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    out, lse = torch.empty_like(q), torch.empty(H, 1, N, device="cuda")

    def run():
        B.check("a", B.qi21_kv4_attention(cfg, k4, 0, q, 1, N, kt, vt, T, out, lse, ws, n, _stream()))
        return out.view(N, H, Dh), lse[:, 0].T

    for key in (0, 5, 13, 14, 15, 31, 47, 64, 111, 126, 127, T - 1):
        h = key % H
        row = kt[0, key, h * Dh:(h + 1) * Dh].clone()
        kt[0, key, h * Dh:(h + 1) * Dh - 1] = 0                        # the score is q's last dim times it
        kt[0, key, h * Dh + Dh - 1] = float("inf")
        up = q[0, :, h * Dh + Dh - 1] > 0
        o, l = run()
        want = torch.zeros(N, H, dtype=torch.bool, device="cuda")
        want[up, h] = True
        assert torch.equal(o.isnan().all(-1), want) and torch.equal(o.isnan().any(-1), want), key
        assert torch.equal(l.isnan(), want), key
        assert not o.isinf().any() and not l.isinf().any()
        kt[0, key, h * Dh:(h + 1) * Dh] = row
    o, l = run()
    assert o.isfinite().all() and l.isfinite().all()


def test_long_prefix_around_the_rows_from_which_it_is_copied(B):
    """2048 and 2049 rows over a prefix whose copy does not stay in L2 (16 heads of 64,
    P 25000) take different kernels, fused and over the copy; each within the rounding
    of weights and result of 64 bits on sampled rows."""
    H, Dh, P, T = 16, 64, 25000, 40
    cfg = _cfg(B, B.QI21_DTYPE_BF16, H, Dh)
    gen = torch.Generator(device="cuda").manual_seed(8)
    src = torch.randn(1, 2, 1, P + 1, H * Dh, device="cuda", generator=gen).bfloat16()
    cache = B.qi21_kv_cache_init(src, cfg, 1, P, 1)
    cache.state = B.QI21_CACHE_EXTRACTED
    buf = torch.zeros(B.qi21_kv4_cache_bytes(cfg, 1, P), dtype=torch.uint8, device="cuda")
    k4 = B.qi21_kv4_cache_init(buf, cfg, 1, P)
    B.check("quantize", B.qi21_kv4_quantize(cfg, cache, k4, _stream()))
    B.check("back", B.qi21_kv4_dequantize(cfg, k4, cache, _stream()))
    k, v = (src[0, i, 0, :P].double().view(P, H, Dh) for i in range(2))
    kt, vt = (torch.randn(1, T, H * Dh, device="cuda", generator=gen).bfloat16() for _ in range(2))
    k, v = (torch.cat((a, t[0].double().view(T, H, Dh))) for a, t in ((k, kt), (v, vt)))
    sizes = []
    for N in (2048, 2049):
        q = torch.randn(1, N, H * Dh, device="cuda", generator=gen).bfloat16()
        sizes.append(B.qi21_kv4_workspace_bytes(cfg, 1, N, P, T))
        ws = torch.zeros(sizes[-1], dtype=torch.uint8, device="cuda")
        out, lse = torch.empty_like(q), torch.empty(H, 1, N, device="cuda")
        B.check("a", B.qi21_kv4_attention(cfg, k4, 0, q, 1, N, kt, vt, T, out, lse, ws, sizes[-1], _stream()))
        B.check("device", B.qi21_check_device_error(ws, sizes[-1], _stream()))
        for i in (0, 127, 128, 1000, N - 1):
            x = torch.einsum("hd,jhd->hj", q[0, i].double().view(H, Dh), k) / Dh ** 0.5
            w = x.softmax(-1)
            o, mag = torch.einsum("hj,jhd->hd", w, v), torch.einsum("hj,jhd->hd", w, v.abs())
            got = out[0, i].double().view(H, Dh)
            # weights and result in bf16, half a step of 2^-8 each; fp32 sums 2e-5
            assert ((got - o).abs() <= 2.0 ** -8 * (mag + o.abs()) + 2e-5 * mag).all()
            assert (lse[:, 0, i] - x.logsumexp(-1)).abs().max() <= 2e-5
    assert sizes[1] - sizes[0] > 2 * P * H * Dh            # the copy, less the partial results


# ------------------------------------------------------------------ after a wait that failed

def test_a_failed_wait_leaves_its_copies_time_to_land(B):
    """The bounded wait of the self test (2 ms) gives up and returns a millisecond later,
    in which copies into the block's shared memory can land, and no later."""
    ws = torch.zeros(4096, dtype=torch.uint8, device="cuda")
    B.check("warm", B.qi21_selftest_wait_timeout(ws, ws.numel(), 1000, _stream()))
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    torch.cuda.synchronize()
    a.record()
    B.check("selftest", B.qi21_selftest_wait_timeout(ws, ws.numel(), 2_000_000, _stream()))
    b.record()
    torch.cuda.synchronize()
    assert 2.9 < a.elapsed_time(b) < 50
    assert B.qi21_check_device_error(ws, ws.numel(), _stream()) == B.QI21_ERR_DEVICE_TIMEOUT
