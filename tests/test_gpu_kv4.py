"""The 4-bit prefix cache on the GPU against 64 bits (tests/_kv4.py).

Tolerances.
* The format: values are compared exactly (equal bits of every value).
* Attention. fp32: a score is a sum of Dh products in fp32, off by about
  sqrt(Dh) 2^-24 of |q||k|/sqrt(Dh) (at most 17 here, so some 1e-5 absolute at
  worst and 2e-6 typically); a weight is off by as much relative to itself, and
  so is a mean of values: 2e-5 of sum_j p_j |v_j|. bf16 adds the rounding of a
  weight (2^-8 of it at most) and of the result (2^-8 of it): together at most
  2^-8 (sum_j p_j |v_j| + |o|), element by element; over a tensor both are spread
  evenly, at most 2^-8 / sqrt(3) each, below 2^-8 in the 2-norm.
* lse: absolute, the error of a score and of a sum of exponentials: 2e-5.
* scores: the 2-norm of weights that are each off by 1e-5 of themselves at most.
"""
from types import SimpleNamespace

import numpy as np
import pytest
import torch

from oracle import qi21_oracle as O
from qi21_synth import configs as C
from tests import _kv4
from tests._harness import BF16_TOL, F32_TOL, max_rel, oracle_model, rel_l2

pytestmark = pytest.mark.gpu
HALF = 2.0 ** -8            # half a step of bf16, relative to the value
FP32_REL = 2e-5
LSE_ABS = 2e-5
MODES = ("f32", "bf16", "bf16_cuda_cores")


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


def _cfg(B, dtype, H, Dh, L=1):
    return B.qi21_config(H * Dh, H, Dh, L, 2 * H * Dh, 64, 256, dtype, 0, 1e-6, 1e-6)


def _stream():
    return torch.cuda.current_stream().cuda_stream


def _np(t):
    return t.double().cpu().numpy()


def _lens_t(lens):
    if lens is None:
        return None
    t = torch.zeros(max(4, len(lens)), dtype=torch.int32, device="cuda")
    t[: len(lens)] = torch.tensor(lens, dtype=torch.int32)
    return t


# ------------------------------------------------------------------ the format

@pytest.mark.parametrize("mode,H,Dh,L,Bn,P,N", [
    ("f32", 2, 128, 2, 2, 198, 3), ("f32", 8, 32, 1, 1, 5, 1), ("f32", 4, 96, 1, 2, 131, 2),
    ("bf16", 4, 64, 3, 2, 129, 5), ("bf16", 2, 128, 1, 1, 1, 1), ("bf16", 32, 128, 1, 1, 260, 4),
    ("bf16_cuda_cores", 16, 64, 1, 3, 64, 1)], indirect=["mode"])
def test_quantise_and_back(B, mode, H, Dh, L, Bn, P, N):
    """Every value equals the format's definition; the way back gives it exactly;
    target rows and padding rows are not touched."""
    dtype, tdt = mode
    cfg = _cfg(B, dtype, H, Dh, L)
    rng = np.random.default_rng(P + Dh)
    x = rng.standard_normal((L, 2, Bn, P + N, H, Dh)) * np.exp(2 * rng.standard_normal((L, 2, Bn, P + N, H, 1)))
    x[0, 0, 0, 0, 0, :32] = 0.0                                        # an empty group
    x[0, 0, 0, 0, 0, 32 % Dh] = 1e-30
    x[0, 1, 0, 0, H - 1, :16] = 2.0 ** -7 * np.arange(-8, 8)           # ties: s = 2^-7 would put halves on integers
    x[0, 1, 0, 0, H - 1, 16:32] = 2.0 ** -8 * np.arange(-14, 2) + 0.0
    x[0, 1, Bn - 1, P - 1, 0, :32] = 2.0 ** -6 * (np.arange(32) % 8 - 3.5)
    src = torch.from_numpy(x).to(tdt).cuda()
    cache = B.qi21_kv_cache_init(src, cfg, Bn, P, N)
    cache.state = B.QI21_CACHE_EXTRACTED
    buf = torch.full((B.qi21_kv4_cache_bytes(cfg, Bn, P),), 0x5A, dtype=torch.uint8, device="cuda")
    k4 = B.qi21_kv4_cache_init(buf, cfg, Bn, P)
    assert B.qi21_kv4_quantize(cfg, cache, k4, _stream()) == B.QI21_OK
    assert k4.state == B.QI21_CACHE_EXTRACTED
    stored = _np(src)[:, :, :, :P].transpose(0, 1, 2, 4, 3, 5)         # [L][2][B][H][P][Dh]
    want = _kv4.values(*_kv4.quantise(stored))
    got = _kv4.read_values(buf, L, Bn, H, P, Dh)
    assert np.array_equal(got, want)
    codes, scales = _kv4.buffer_views(buf, L, Bn, H, P, Dh)
    assert (codes[..., P:, :] == 0x5A).all() and (scales.view(torch.uint8)[..., P:, :] == 0x5A).all()
    back = torch.full((L, 2, Bn, P + N, H, Dh), 7.0, dtype=tdt, device="cuda")
    cb = B.qi21_kv_cache_init(back, cfg, Bn, P, N)
    assert B.qi21_kv4_dequantize(cfg, k4, cb, _stream()) == B.QI21_OK
    assert cb.state == B.QI21_CACHE_EXTRACTED
    assert np.array_equal(_np(back)[:, :, :, :P], want.transpose(0, 1, 2, 4, 3, 5))
    assert (back[:, :, :, P:] == 7.0).all()


def test_quantise_near_ties_and_extremes(B):
    """float32 quotients a few units in the last place from the middle of two
    integers, denormal and huge groups, and groups that are not finite."""
    cfg = _cfg(B, B.QI21_DTYPE_F32, 2, 128)
    rng = np.random.default_rng(5)
    P = 64
    x = np.zeros((1, 2, 1, P + 1, 2, 128))
    for r in range(P):
        s = _kv4.SCALES[rng.integers(800, 3000)]
        near = ((rng.integers(-7, 7, 256) + 0.5) * s).astype(np.float32)
        for _ in range(r % 4):
            near = np.nextafter(near, np.float32(np.inf if r % 8 < 4 else -np.inf))
        near[::32] = 7 * s
        x[0, 0, 0, r] = near.reshape(2, 128)
    x[0, 1, 0, 0, 0] = 1e-40 * rng.standard_normal(128)
    x[0, 1, 0, 1, 0] = 3e38 * np.sign(rng.standard_normal(128))
    x[0, 1, 0, 2, 0] = 1e37 * rng.standard_normal(128).clip(-3, 3)
    src = torch.from_numpy(x).float().cuda()
    src[0, 1, 0, 3, 0, 5] = float("nan")
    src[0, 1, 0, 4, 1, 40] = float("-inf")
    cache = B.qi21_kv_cache_init(src, cfg, 1, P, 1)
    cache.state = B.QI21_CACHE_EXTRACTED
    buf = torch.zeros(B.qi21_kv4_cache_bytes(cfg, 1, P), dtype=torch.uint8, device="cuda")
    k4 = B.qi21_kv4_cache_init(buf, cfg, 1, P)
    assert B.qi21_kv4_quantize(cfg, cache, k4, _stream()) == B.QI21_OK
    got = _kv4.read_values(buf, 1, 1, 2, P, 128)[0, :, 0]              # [2][H][P][Dh]
    stored = _np(src)[0, :, 0, :P].transpose(0, 2, 1, 3)
    bad = ~np.isfinite(stored).reshape(2, 2, P, 4, 32).all(-1)
    assert bad.sum() == 2
    want = _kv4.values(*_kv4.quantise(np.where(np.isfinite(stored), stored, 0.0)))
    isnan = np.isnan(got).reshape(2, 2, P, 4, 32)
    assert np.array_equal(isnan.all(-1), bad) and np.array_equal(isnan.any(-1), bad)
    keep = ~np.repeat(bad, 32, -1)
    assert np.array_equal(got[keep], want[keep])


def test_quantise_lengths_and_shared_layout(B):
    """Rows behind an item's length are left as they are, both ways; a shared-prefix
    cache has one item."""
    cfg = _cfg(B, B.QI21_DTYPE_BF16, 4, 64, 2)
    P, lens = 70, [70, 0, 33]
    src = torch.randn(2, 2, 3, P + 2, 256, device="cuda").bfloat16()
    cache = B.qi21_kv_cache_init(src, cfg, 3, P, 2)
    cache.state = B.QI21_CACHE_EXTRACTED
    buf = torch.full((B.qi21_kv4_cache_bytes(cfg, 3, P),), 0x33, dtype=torch.uint8, device="cuda")
    lt = _lens_t(lens)
    k4 = B.qi21_kv4_cache_init(buf, cfg, 3, P, lt)
    assert B.qi21_kv4_quantize(cfg, cache, k4, _stream()) == B.QI21_OK
    codes, scales = _kv4.buffer_views(buf, 2, 3, 4, P, 64)
    want = _kv4.values(*_kv4.quantise(_np(src)[:, :, :, :P].reshape(2, 2, 3, P, 4, 64).transpose(0, 1, 2, 4, 3, 5)))
    got = _kv4.read_values(buf, 2, 3, 4, P, 64)
    for b, n in enumerate(lens):
        assert np.array_equal(got[:, :, b, :, :n], want[:, :, b, :, :n])
        assert (codes[:, :, b, :, n:] == 0x33).all()
        assert (scales.view(torch.uint8)[:, :, b, :, n:] == 0x33).all()
    back = torch.full((2, 2, 3, P + 1, 256), 7.0, dtype=torch.bfloat16, device="cuda")
    cb = B.qi21_kv_cache_init(back, cfg, 3, P, 1)
    assert B.qi21_kv4_dequantize(cfg, k4, cb, _stream()) == B.QI21_OK
    for b, n in enumerate(lens):
        assert np.array_equal(_np(back)[:, :, b, :n].reshape(2, 2, n, 4, 64),
                              want[:, :, b, :, :n].transpose(0, 1, 3, 2, 4))
        assert (back[:, :, b, n:] == 7.0).all()
    # shared: [L][2][Pp + B N][d]
    Pp = 128
    src = torch.randn(2, 2, Pp + 3 * 5, 256, device="cuda").bfloat16()
    cache = B.qi21_kv_cache_init_shared(src, cfg, 3, P, 5)
    cache.state = B.QI21_CACHE_EXTRACTED
    buf = torch.zeros(B.qi21_kv4_cache_bytes(cfg, 1, P), dtype=torch.uint8, device="cuda")
    k4 = B.qi21_kv4_cache_init(buf, cfg, 1, P)
    assert B.qi21_kv4_quantize(cfg, cache, k4, _stream()) == B.QI21_OK
    want = _kv4.values(*_kv4.quantise(_np(src)[:, :, :P].reshape(2, 2, P, 4, 64).transpose(0, 1, 3, 2, 4)))
    assert np.array_equal(_kv4.read_values(buf, 2, 1, 4, P, 64)[:, :, 0], want)
    back = torch.full_like(src, 7.0)
    cb = B.qi21_kv_cache_init_shared(back, cfg, 3, P, 5)
    assert B.qi21_kv4_dequantize(cfg, k4, cb, _stream()) == B.QI21_OK
    assert np.array_equal(_np(back)[:, :, :P].reshape(2, 2, P, 4, 64), want.transpose(0, 1, 3, 2, 4))
    assert (back[:, :, P:] == 7.0).all()


# ------------------------------------------------------------------ attention

# H, Dh, items in the cache, requests, P, N, T, lengths
ATT = [
    (4, 64, 1, 1, 1, 1, 0, None), (2, 128, 1, 1, 1, 1, 1, None), (2, 128, 2, 2, 198, 300, 300, None),
    (4, 64, 2, 2, 130, 130, 7, None), (16, 64, 1, 1, 77, 1, 1, None), (2, 128, 1, 1, 5000, 1, 3, None),
    (4, 64, 1, 1, 4000, 8, 0, None), (2, 128, 3, 3, 700, 16, 16, [700, 0, 129]), (2, 128, 2, 2, 300, 9, 0, [0, 1]),
    (4, 64, 3, 3, 257, 40, 65, [128, 257, 0]), (2, 128, 1, 3, 260, 33, 20, None), (4, 64, 1, 4, 513, 1, 2, [500]),
    (2, 128, 1, 1, 128, 256, 128, None), (2, 128, 1, 1, 127, 257, 129, None), (8, 128, 1, 1, 1100, 64, 640, None),
    (4, 64, 2, 2, 383, 128, 0, [382, 3]), (2, 128, 1, 1, 40, 17, 1000, None), (2, 128, 2, 2, 100, 520, 30, [-5, 1000]),
    (32, 128, 1, 1, 640, 24, 5, None), (4, 64, 5, 5, 90, 2, 300, [0, 0, 90, 1, 64]),
    (16, 64, 5, 5, 200, 1030, 50, [200, 0, 130, 1, 77]), (32, 128, 1, 3, 140, 1024, 0, None),
    (16, 64, 5, 5, 130, 1024, 0, [0, 130, 2, 128, 129]), (32, 128, 2, 2, 257, 1153, 300, None),
]


def _run_attention(B, cfg, k4, q, kt, vt, lse=True, layer=0):
    Bn, N, H = q.shape[0], q.shape[1], cfg.n_heads
    T = 0 if kt is None else kt.shape[1]
    n = B.qi21_kv4_workspace_bytes(cfg, Bn, N, k4.n_prefix, T)
    ws = torch.full((n + 1024,), 0x5C, dtype=torch.uint8, device="cuda")
    ws[:64] = 0                                             # the error words
    out = torch.full_like(q, float("nan"))
    ls = torch.full((H, Bn, N), float("nan"), device="cuda") if lse else None
    B.check("attention", B.qi21_kv4_attention(cfg, k4, layer, q, Bn, N, kt, vt, T, out, ls, ws, n, _stream()))
    B.check("device", B.qi21_check_device_error(ws, n, _stream()))
    assert (ws[n:] == 0x5C).all()
    return out, ls


def _check_attention(q, vals, kt, vt, lens, H, Dh, out, lse, bf16):
    """vals [2][cache items][H][P][Dh] of one layer."""
    Bn, N = q.shape[:2]
    qn, on = _np(q).reshape(Bn, N, H, Dh), _np(out).reshape(Bn, N, H, Dh)
    ktn = None if kt is None else _np(kt).reshape(Bn, -1, H, Dh)
    vtn = None if vt is None else _np(vt).reshape(Bn, -1, H, Dh)
    want = np.zeros_like(on)
    for b in range(Bn):
        cb = min(b, vals.shape[1] - 1)
        P = vals.shape[3]
        n = P if lens is None else min(max(lens[cb], 0), P)
        for h in range(H):
            k, v = vals[0, cb, h, :n], vals[1, cb, h, :n]
            if ktn is not None:
                k, v = np.concatenate((k, ktn[b, :, h])), np.concatenate((v, vtn[b, :, h]))
            o, mag, ls, _ = _kv4.attention(qn[b, :, h], k, v)
            want[b, :, h] = o
            tol = FP32_REL * mag + 1e-30
            if bf16:
                tol = tol + HALF * (mag + np.abs(o)) * (1 + 1e-4)
            assert (np.abs(on[b, :, h] - o) <= tol).all(), (b, h, np.abs(on[b, :, h] - o).max())
            if lse is not None:
                l = _np(lse)[h, b]
                if len(k):
                    assert np.abs(l - ls).max() <= LSE_ABS, (b, h, np.abs(l - ls).max())
                else:
                    assert (l == -np.inf).all()
    if np.abs(want).max() > 0:
        assert rel_l2(on, want) < (HALF if bf16 else FP32_REL)


@pytest.mark.parametrize("mode", MODES, indirect=True)
@pytest.mark.parametrize("case", range(len(ATT)))
def test_attention(B, mode, case):
    """Rows that do not exist hold NaN scales (and an item may have none at all)."""
    dtype, tdt = mode
    H, Dh, Cb, Bn, P, N, T, lens = ATT[case]
    cfg = _cfg(B, dtype, H, Dh)
    rng = np.random.default_rng(case)
    buf, vals = _kv4.make_buffer(rng, B, cfg, Cb, P, None if lens is None else [min(max(n, 0), P) for n in lens])
    lt = _lens_t(lens)
    k4 = B.qi21_kv4_cache_init(buf, cfg, Cb, P, lt)
    k4.state = B.QI21_CACHE_EXTRACTED
    draw = lambda n, s: torch.from_numpy(rng.standard_normal((Bn, n, H * Dh)) * s).to(tdt).cuda()  # noqa: E731
    q = draw(N, 1.5)
    kt, vt = (draw(T, 1.0), draw(T, 1.0)) if T else (None, None)
    out, lse = _run_attention(B, cfg, k4, q, kt, vt)
    _check_attention(q, vals[0], kt, vt, lens, H, Dh, out, lse, dtype == B.QI21_DTYPE_BF16)
    again, none = _run_attention(B, cfg, k4, q, kt, vt, lse=False)      # the lse is optional; same bits
    assert none is None and torch.equal(again, out)


@pytest.mark.parametrize("mode", MODES, indirect=True)
@pytest.mark.parametrize("N", [1, 12, 200])
def test_attention_scores_of_very_different_size(B, mode, N):
    """One key far above the others late in the row (the running maximum has to
    move), and scores so low that every other weight vanishes."""
    dtype, tdt = mode
    cfg = _cfg(B, dtype, 2, 128, 2)
    rng = np.random.default_rng(N)
    buf, vals = _kv4.make_buffer(rng, B, cfg, 1, 900)
    k4 = B.qi21_kv4_cache_init(buf, cfg, 1, 900)
    k4.state = B.QI21_CACHE_EXTRACTED
    qn = rng.standard_normal((1, N, 256)) * np.exp(rng.standard_normal((1, N, 1)))
    qn[0, :, :128] += 6 * vals[1, 0, 0, 0, 850]                # layer 1: towards key 850 of head 0
    q = torch.from_numpy(qn).to(tdt).cuda()
    kt = torch.from_numpy(rng.standard_normal((1, 140, 256))).to(tdt).cuda()
    vt = torch.from_numpy(rng.standard_normal((1, 140, 256))).to(tdt).cuda()
    kt[0, 139] *= 8
    out, lse = _run_attention(B, cfg, k4, q, kt, vt, layer=1)
    qs = _np(q).reshape(N, 2, 128)
    for h in range(2):
        k = np.concatenate((vals[1, 0, 0, h], _np(kt)[0].reshape(140, 2, 128)[:, h]))
        v = np.concatenate((vals[1, 1, 0, h], _np(vt)[0].reshape(140, 2, 128)[:, h]))
        o, mag, ls, _ = _kv4.attention(qs[:, h], k, v)
        # scores of some hundreds: fp32 sums are off by sqrt(Dh) 2^-24 of |q||k| / sqrt(Dh)
        big = np.linalg.norm(qs[:, h], axis=1).max() * np.linalg.norm(k, axis=1).max()
        ds = 4 * 2.0 ** -24 * big
        tol = (FP32_REL + 2 * ds) * mag + (HALF * (mag + np.abs(o)) if dtype == B.QI21_DTYPE_BF16 else 0)
        assert (np.abs(_np(out).reshape(N, 2, 128)[:, h] - o) <= tol).all()
        assert np.abs(_np(lse)[h, 0] - ls).max() <= LSE_ABS + ds


def test_workspace_of_a_shared_and_of_an_own_prefix(B):
    """Sizes at which five items of their own and one shared by five take different
    kernels: the queried workspace holds either (the bytes behind it stay), and both
    give the same results to the rounding of weights and results."""
    H, Dh, Bn, P, N = 16, 64, 5, 6000, 1100
    cfg = _cfg(B, B.QI21_DTYPE_BF16, H, Dh)
    rng = np.random.default_rng(1)
    one, _ = _kv4.make_buffer(rng, B, cfg, 1, P)
    many = torch.zeros(B.qi21_kv4_cache_bytes(cfg, Bn, P), dtype=torch.uint8, device="cuda")
    for dst, src in zip(_kv4.buffer_views(many, 1, Bn, H, P, Dh), _kv4.buffer_views(one, 1, 1, H, P, Dh)):
        dst.copy_(src.expand_as(dst))
    q = torch.randn(Bn, N, H * Dh, device="cuda").bfloat16()
    n = B.qi21_kv4_workspace_bytes(cfg, Bn, N, P, 0)
    ws = torch.full((n + 4096,), 0x5C, dtype=torch.uint8, device="cuda")
    ws[:64] = 0
    outs = []
    for buf, items in ((one, 1), (many, Bn)):
        k4 = B.qi21_kv4_cache_init(buf, cfg, items, P)
        k4.state = B.QI21_CACHE_EXTRACTED
        out, lse = torch.empty_like(q), torch.empty(H, Bn, N, device="cuda")
        sc = torch.empty(items, H, P, device="cuda")
        B.check("a", B.qi21_kv4_attention(cfg, k4, 0, q, Bn, N, None, None, 0, out, lse, ws, n, _stream()))
        B.check("s", B.qi21_kv4_scores(cfg, k4, 0, q, Bn, N, lse, None, sc, ws, n, _stream()))
        B.check("d", B.qi21_check_device_error(ws, n, _stream()))
        outs.append((out, lse, sc.sum(0)))
    assert (ws[n:] == 0x5C).all()
    a, b = outs
    assert rel_l2(_np(a[0]), _np(b[0])) < 2 * HALF and rel_l2(_np(a[1]), _np(b[1])) < 1e-5
    assert rel_l2(_np(a[2]), _np(b[2])) < 3e-5


@pytest.mark.parametrize("mode", ["f32", "bf16_cuda_cores"], indirect=True)
@pytest.mark.parametrize("H,Dh,P,N,T,lens", [(8, 32, 131, 45, 20, None), (8, 96, 70, 33, 0, [70, 9]),
                                             (8, 32, 3, 1, 1, [0, 3]), (8, 96, 400, 2, 65, None)])
def test_attention_scores_and_eviction_at_other_head_dims(B, mode, H, Dh, P, N, T, lens):
    """head_dim 32 and 96, which the CUDA-core family covers."""
    dtype, tdt = mode
    cfg = _cfg(B, dtype, H, Dh)
    rng = np.random.default_rng(Dh + P)
    buf, vals = _kv4.make_buffer(rng, B, cfg, 2, P, lens)
    lt = _lens_t(lens)
    k4 = B.qi21_kv4_cache_init(buf, cfg, 2, P, lt)
    k4.state = B.QI21_CACHE_EXTRACTED
    draw = lambda n, s: torch.from_numpy(rng.standard_normal((2, n, H * Dh)) * s).to(tdt).cuda()  # noqa: E731
    q, kt, vt = draw(N, 1.5), draw(T, 1.0) if T else None, draw(T, 1.0) if T else None
    out, lse = _run_attention(B, cfg, k4, q, kt, vt)
    _check_attention(q, vals[0], kt, vt, lens, H, Dh, out, lse, dtype == B.QI21_DTYPE_BF16)
    n = B.qi21_kv4_workspace_bytes(cfg, 2, N, P, 0)
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    sc = torch.empty(2, H, P, device="cuda")
    B.check("scores", B.qi21_kv4_scores(cfg, k4, 0, q, 2, N, lse, None, sc, ws, n, _stream()))
    qn = _np(q).reshape(2, N, H, Dh)
    want = np.zeros((2, H, P))
    for b in range(2):
        m = P if lens is None else lens[b]
        for h in range(H):
            x = qn[b, :, h] @ vals[0, 0, b, h, :m].T / np.sqrt(Dh)
            want[b, h, :m] = np.exp(x - _np(lse)[h, b][:, None]).sum(0)
    assert rel_l2(_np(sc), want) < 1e-5
    keep = max(1, P // 3)
    small = torch.full((B.qi21_kv4_cache_bytes(cfg, 2, keep),), 0x77, dtype=torch.uint8, device="cuda")
    lo = None if lens is None else torch.zeros(4, dtype=torch.int32, device="cuda")
    s4 = B.qi21_kv4_cache_init(small, cfg, 2, keep, lo)
    kept = torch.zeros(1, 2, H, keep, dtype=torch.int32, device="cuda")
    assert B.qi21_kv4_evict(cfg, k4, sc, keep, 0, s4, kept, _stream()) == B.QI21_OK
    rows = _kv4.evict(sc.cpu().numpy()[None], lens, keep, 0)
    assert np.array_equal(kept.cpu().numpy(), rows)
    got = _kv4.read_values(small, 1, 2, H, keep, Dh)
    for b in range(2):
        m = keep if lens is None else min(keep, lens[b])
        for h in range(H):
            assert np.array_equal(got[0, :, b, h, :m], vals[0, :, b, h][:, rows[0, b, h, :m]])


@pytest.mark.parametrize("mode", MODES, indirect=True)
@pytest.mark.parametrize("N,Bn,P", [(1, 1, 700), (9, 1, 700), (60, 1, 700), (200, 1, 900), (1030, 5, 130)])
def test_nan_reaches_exactly_its_results(B, mode, N, Bn, P):
    """A group that is not finite makes NaNs of the results it is part of: a key of a
    head the whole head (of its item), a value its 32 dims; a NaN query its row. And
    an infinite key in a row that does not exist nothing at all."""
    dtype, tdt = mode
    H, Dh = 16, 64
    cfg = _cfg(B, dtype, H, Dh)
    rng = np.random.default_rng(N)
    lens = [P - 3] * Bn
    buf, _ = _kv4.make_buffer(rng, B, cfg, Bn, P, lens, fill=0x7F)
    codes, scales = _kv4.buffer_views(buf, 1, Bn, H, P, Dh)
    scales[0, 0, 0, 2, P - 9, 1] = float("nan")              # key: head 2 of item 0
    scales[0, 1, 0, 5, 77, 0] = float("nan")                 # value: dims 0..31 of head 5
    lt = _lens_t(lens)
    k4 = B.qi21_kv4_cache_init(buf, cfg, Bn, P, lt)
    k4.state = B.QI21_CACHE_EXTRACTED
    q = torch.randn(Bn, N, H * Dh, device="cuda").to(tdt)
    q[-1, N - 1, 9 * Dh] = float("nan")                      # query: last row of head 9, last item
    kt, vt = (torch.randn(Bn, 40, H * Dh, device="cuda").to(tdt) for _ in range(2))
    out, lse = _run_attention(B, cfg, k4, q, kt, vt)
    want = torch.zeros(Bn, N, H, Dh, dtype=torch.bool, device="cuda")
    want[0, :, 2] = True
    want[0, :, 5, :32] = True
    want[-1, N - 1, 9] = True
    assert torch.equal(out.isnan().view(Bn, N, H, Dh), want)
    wl = torch.zeros(H, Bn, N, dtype=torch.bool, device="cuda")
    wl[2, 0] = True
    wl[9, -1, N - 1] = True
    assert torch.equal(lse.isnan(), wl)
    assert not out.isinf().any() and not lse.isinf().any()
    # the weights: NaN for the head that has a NaN query (or lse), elsewhere finite
    n = B.qi21_kv4_workspace_bytes(cfg, Bn, N, P, 0)
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    sc = torch.empty(Bn, H, P, device="cuda")
    B.check("scores", B.qi21_kv4_scores(cfg, k4, 0, q, Bn, N, lse, None, sc, ws, n, _stream()))
    ws_want = torch.zeros(Bn, H, P, dtype=torch.bool, device="cuda")
    ws_want[0, 2, : P - 3] = True
    ws_want[-1, 9, : P - 3] = True
    assert torch.equal(sc.isnan(), ws_want)


# ------------------------------------------------------------------ scores

SC = [
    (4, 64, 1, 1, 1, 1, None), (2, 128, 2, 2, 198, 300, None), (4, 64, 2, 2, 130, 130, [100, 0]),
    (2, 128, 1, 3, 260, 33, None), (4, 64, 1, 1, 3000, 1, None), (16, 64, 1, 1, 129, 700, None),
    (2, 128, 1, 1, 128, 128, None), (2, 128, 1, 1, 100, 2000, [99]), (8, 128, 1, 2, 513, 9, None),
    (4, 64, 3, 3, 77, 257, [77, 1, 0]),
]


@pytest.mark.parametrize("mode", MODES, indirect=True)
@pytest.mark.parametrize("case", range(len(SC)))
def test_scores(B, mode, case):
    dtype, tdt = mode
    H, Dh, Cb, Bn, P, N, lens = SC[case]
    cfg = _cfg(B, dtype, H, Dh)
    rng = np.random.default_rng(100 + case)
    buf, vals = _kv4.make_buffer(rng, B, cfg, Cb, P, lens)
    lt = _lens_t(lens)
    k4 = B.qi21_kv4_cache_init(buf, cfg, Cb, P, lt)
    k4.state = B.QI21_CACHE_EXTRACTED
    q = torch.from_numpy(rng.standard_normal((Bn, N, H * Dh)) * 1.5).to(tdt).cuda()
    qn = _np(q).reshape(Bn, N, H, Dh)
    lse = np.zeros((H, Bn, N), np.float32)
    want = np.zeros((Cb, H, P))
    for b in range(Bn):
        cb = min(b, Cb - 1)
        n = P if lens is None else lens[cb]
        for h in range(H):
            k = vals[0, 0, cb, h, :n]
            ls = _kv4.attention(qn[b, :, h], k, k)[2]
            lse[h, b] = np.where(np.isfinite(ls), ls + np.log1p(rng.random(N)), -np.inf)   # a tail's share on top
            if n and b % 2 == 0:
                lse[h, b, N // 2] = -np.inf                     # a query without keys adds nothing
            x = qn[b, :, h] @ k.T / np.sqrt(Dh)
            want[cb, h, :n] += np.where(np.isfinite(lse[h, b])[:, None], np.exp(x - lse[h, b][:, None]), 0).sum(0)
    before = np.abs(rng.standard_normal((Cb, H, P))).astype(np.float32)
    lse_t, before_t = torch.from_numpy(lse).cuda(), torch.from_numpy(before).cuda()
    nws = B.qi21_kv4_workspace_bytes(cfg, Bn, N, P, 0)
    ws = torch.zeros(nws, dtype=torch.uint8, device="cuda")

    def call(si, so):
        B.check("scores", B.qi21_kv4_scores(cfg, k4, 0, q, Bn, N, lse_t, si, so, ws, nws, _stream()))
        B.check("device", B.qi21_check_device_error(ws, nws, _stream()))
        return so

    guard = torch.full((Cb * H * P + 8,), -1.0, device="cuda")
    got = call(None, guard)[: Cb * H * P].view(Cb, H, P)
    assert (guard[Cb * H * P:] == -1.0).all()
    if np.abs(want).max() > 0:
        assert rel_l2(_np(got), want) < 1e-5
    for b in range(Cb):
        assert (got[b, :, (P if lens is None else lens[b]):] == 0).all()
    after = call(before_t, torch.empty_like(before_t))
    assert rel_l2(_np(after), want + before) < 1e-5
    inplace = call(before_t, before_t)
    assert torch.equal(inplace, after)                          # and a second call gives the same bits
    for b in range(Cb):
        n = P if lens is None else lens[b]
        assert np.array_equal(_np(after)[b, :, n:], before[b, :, n:].astype(np.float64))


def test_scores_add_up_to_the_queries(B):
    """With the lse that the attention writes, a query's weights sum to 1: over
    prefix rows and no tail the scores of a head sum to the number of queries
    (fp32 sums of N weights; lse off by 2e-5 at most)."""
    cfg = _cfg(B, B.QI21_DTYPE_BF16, 4, 64)
    rng = np.random.default_rng(9)
    buf, _ = _kv4.make_buffer(rng, B, cfg, 2, 333)
    k4 = B.qi21_kv4_cache_init(buf, cfg, 2, 333)
    k4.state = B.QI21_CACHE_EXTRACTED
    q = torch.randn(2, 500, 256, device="cuda").bfloat16()
    _, lse = _run_attention(B, cfg, k4, q, None, None)
    n = B.qi21_kv4_workspace_bytes(cfg, 2, 500, 333, 0)
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    sc = torch.empty(2, 4, 333, device="cuda")
    B.check("scores", B.qi21_kv4_scores(cfg, k4, 0, q, 2, 500, lse, None, sc, ws, n, _stream()))
    total = sc.double().sum(-1)
    assert (total - 500).abs().max() < 500 * 3e-5


# ------------------------------------------------------------------ eviction

@pytest.mark.parametrize("H,Dh,L,Bn,P,keep,prot,lens", [
    (2, 128, 2, 2, 198, 77, 10, None), (4, 64, 1, 1, 1, 1, 0, None), (4, 64, 3, 2, 600, 600, 5, None),
    (16, 64, 1, 3, 513, 1, 0, None), (2, 128, 1, 1, 5000, 2501, 2501, None), (8, 128, 2, 1, 1024, 512, 100, None),
    (4, 64, 2, 3, 130, 60, 7, [130, 20, 0]), (2, 128, 1, 2, 40, 40, 3, [39, 40])])
def test_evict(B, H, Dh, L, Bn, P, keep, prot, lens):
    """The rows kept are those of a stable sort (ties, infinities, NaNs and -0
    among the scores), and the smaller cache holds exactly their bytes."""
    cfg = _cfg(B, B.QI21_DTYPE_BF16, H, Dh, L)
    rng = np.random.default_rng(P + keep)
    buf, vals = _kv4.make_buffer(rng, B, cfg, Bn, P, lens)
    lt = _lens_t(lens)
    k4 = B.qi21_kv4_cache_init(buf, cfg, Bn, P, lt)
    k4.state = B.QI21_CACHE_EXTRACTED
    sc = np.round(np.exp(2 * rng.standard_normal((L, Bn, H, P))) * 16).astype(np.float32) / 16
    if P > 30:
        sc[0, 0, 0, ::7] = np.nan
        sc[0, 0, 0, 1::9] = np.inf
        sc[0, 0, 0, 2::9] = -np.inf
        sc[0, 0, 1, :] = 0.0
        sc[0, 0, 1, ::3] = -0.0
        sc[-1, -1, -1, :] = 2.5
    out = torch.full((B.qi21_kv4_cache_bytes(cfg, Bn, keep),), 0x77, dtype=torch.uint8, device="cuda")
    lens_out = None if lens is None else torch.full((4,), -1, dtype=torch.int32, device="cuda")
    small = B.qi21_kv4_cache_init(out, cfg, Bn, keep, lens_out)
    kept = torch.full((L, Bn, H, keep), 99, dtype=torch.int32, device="cuda")
    sct = torch.from_numpy(sc).cuda()
    assert B.qi21_kv4_evict(cfg, k4, sct, keep, prot, small, kept, _stream()) == B.QI21_OK
    assert small.state == B.QI21_CACHE_EXTRACTED
    want = _kv4.evict(sc, lens, keep, prot)
    assert np.array_equal(kept.cpu().numpy(), want)
    got = _kv4.read_values(out, L, Bn, H, keep, Dh)
    codes, _ = _kv4.buffer_views(out, L, Bn, H, keep, Dh)
    for b in range(Bn):
        n = keep if lens is None else min(keep, lens[b])
        for l in range(L):
            for h in range(H):
                for which in range(2):
                    assert np.array_equal(got[l, which, b, h, :n], vals[l, which, b, h][want[l, b, h, :n]])
        assert (codes[:, :, b, :, n:] == 0x77).all()
    if lens is not None:
        assert lens_out[:Bn].tolist() == [min(keep, n) for n in lens]


@pytest.mark.parametrize("L,Bn,H,Dh,P,keep,prot,ragged", [
    (5, 1, 32, 64, 8300, 4100, 7, False), (3, 2, 32, 128, 2049, 1, 0, True), (10, 1, 16, 64, 300, 299, 299, False),
    (1, 1, 4, 64, 20000, 9999, 100, False), (4, 3, 16, 64, 1500, 800, 20, True), (2, 3, 32, 64, 512, 512, 0, True)])
def test_evict_many_heads_and_long_prefixes(B, L, Bn, H, Dh, P, keep, prot, ragged):
    """Either form of the eviction (one kernel, or selection and copy), prefixes that one
    block reads in pieces, against a stable sort; the copied bytes, and no others."""
    cfg = _cfg(B, B.QI21_DTYPE_BF16, H, Dh, L)
    gen = torch.Generator(device="cuda").manual_seed(P)
    buf = torch.randint(0, 256, (B.qi21_kv4_cache_bytes(cfg, Bn, P),), dtype=torch.uint8, device="cuda", generator=gen)
    lens = torch.randint(0, P + 1, (4,), dtype=torch.int32, device="cuda", generator=gen) if ragged else None
    k4 = B.qi21_kv4_cache_init(buf, cfg, Bn, P, lens)
    k4.state = B.QI21_CACHE_EXTRACTED
    sc = torch.randn(L, Bn, H, P, device="cuda", generator=gen).mul(3).round()          # ties everywhere
    out = torch.full((B.qi21_kv4_cache_bytes(cfg, Bn, keep),), 0x77, dtype=torch.uint8, device="cuda")
    lens_out = torch.zeros(4, dtype=torch.int32, device="cuda")
    small = B.qi21_kv4_cache_init(out, cfg, Bn, keep, lens_out)
    kept = torch.full((L, Bn, H, keep), 7, dtype=torch.int32, device="cuda")
    assert B.qi21_kv4_evict(cfg, k4, sc, keep, prot, small, kept, _stream()) == B.QI21_OK
    c0, s0 = _kv4.buffer_views(buf, L, Bn, H, P, Dh)
    c1, s1 = _kv4.buffer_views(out, L, Bn, H, keep, Dh)
    s0, s1 = s0.view(torch.int16), s1.view(torch.int16)
    for b in range(Bn):
        n = int(lens[b]) if ragged else P
        m = min(keep, n)
        rank = sc[:, b, :, :n].clone()
        rank[..., : min(prot, n)] = float("inf")
        want = torch.sort(rank, dim=-1, descending=True, stable=True).indices[..., :m].sort(-1).values
        assert torch.equal(kept[:, b, :, :m].long(), want) and (kept[:, b, :, m:] == -1).all()
        assert int(lens_out[b]) == m
        at = want[:, None, :, :, None].expand(L, 2, H, m, 1)
        assert torch.equal(c1[:, :, b, :, :m], c0[:, :, b].gather(3, at.expand(-1, -1, -1, -1, Dh // 2)))
        assert torch.equal(s1[:, :, b, :, :m], s0[:, :, b].gather(3, at.expand(-1, -1, -1, -1, Dh // 32)))
        assert (c1[:, :, b, :, m:] == 0x77).all() and (s1[:, :, b, :, m:] == 0x7777).all()


# ------------------------------------------------------------------ the cached step over the 4-bit prefix

def _inputs(w):
    pre = torch.from_numpy(C.host_prefix_hidden(w).astype(np.float32)).cuda()
    return pre, torch.from_numpy(C.host_noise(w).astype(np.float32)).cuda()


def _oracle_step(model, seq, ck, cv, x, sigma):
    """The oracle's cached step over any prefix rows ck, cv [L][rows][H][Dh]: the
    target rows see all of them and all target keys."""
    n = ck.shape[1]
    s = SimpleNamespace(P=n, N=seq.N, coords=np.concatenate((np.zeros((n, 3), seq.coords.dtype), seq.coords[seq.P:])),
                        allowed=np.ones((n + seq.N, n + seq.N), bool))
    mt, sf = O.modulation(1000.0 * sigma, model.wts, model.n_chunks)
    return O.cached_step(model, s, ck, cv, x, mt, sf)


@pytest.mark.parametrize("mode,name", [("f32", "small"), ("f32", "small64"), ("bf16", "small"), ("bf16", "small64"),
                                       ("bf16", "small_t1"), ("bf16_cuda_cores", "small")], indirect=["mode"])
def test_cached_step_kv4_evict_and_go_on(B, mode, name):
    """Extract, quantise, a step with its attention weights, evict, another step: each
    step against the oracle on the very prefix values that the 4-bit cache holds, the
    weights against the oracle's, the rows kept against the weights."""
    dtype, tdt = mode
    from prefix_kv_cached_b200.runner import Qi21Runner
    w = C.make_workload(name)
    model, wts = oracle_model(w, "float32" if dtype == B.QI21_DTYPE_F32 else "bfloat16")
    seq = O.make_sequence(w.segments)
    metric, tol = (max_rel, F32_TOL) if dtype == B.QI21_DTYPE_F32 else (rel_l2, BF16_TOL)
    r = Qi21Runner(w, dtype, host_weights=wts)
    pre, x0 = _inputs(w)
    L, H, Dh = w.shape.n_layers, w.shape.n_heads, w.shape.head_dim
    r.set_prefix_row()
    r.prefix_extract(pre)
    r.quantise_prefix()
    vals = _kv4.read_values(r.kv4_buf, L, r.Bn, H, r.P, Dh)
    K, V = r.cache_kv()
    rows = torch.stack((K, V), 1)[:, :, :, : r.P].permute(0, 1, 2, 4, 3, 5)
    assert np.array_equal(vals, _kv4.values(*_kv4.quantise(_np(rows))))
    x, v = x0.clone(), torch.empty_like(x0)
    r.set_target_row(w.sigmas[0])
    r.cached_step_kv4(x, v, accumulate=True)
    B.check("device", B.qi21_check_device_error(r.kv4_ws, r.kv4_ws.numel(), r.stream))
    sc = _np(r.kv4_scores)
    assert sc.shape == (L, r.Bn, H, r.P)
    keep, prot = r.P // 2 + 1, 9
    kept = r.evict_prefix(keep, prot).cpu().numpy()
    assert np.array_equal(kept, _kv4.evict(sc.astype(np.float32), None, keep, prot))
    small = _kv4.read_values(r.kv4_buf, L, r.Bn, H, keep, Dh)
    v2 = torch.empty_like(v)
    r.set_target_row(w.sigmas[1])
    r.cached_step_kv4(x, v2)
    B.check("device", B.qi21_check_device_error(r.kv4_ws, r.kv4_ws.numel(), r.stream))
    for b in range(r.Bn):
        ck, cv = (vals[:, i, b].transpose(0, 2, 1, 3) for i in range(2))
        vo, tk, _ = _oracle_step(model, seq, ck, cv, _np(x)[b], w.sigmas[0])
        assert metric(_np(v)[b], vo) < tol, b
        # weights of layer 0: the oracle's queries (target rows of layer 0 depend on nothing before it)
        total = sc[:, b].sum(-1)
        assert (total > 0).all() and (total < r.N * (1 + 1e-4)).all()
        ek, ev = (small[:, i, b].transpose(0, 2, 1, 3) for i in range(2))
        vo2, _, _ = _oracle_step(model, seq, ek, ev, _np(x)[b], w.sigmas[1])
        assert metric(_np(v2)[b], vo2) < tol, b


@pytest.mark.parametrize("mode", ["f32", "bf16"], indirect=True)
def test_denoise_kv4_shared_prefix_and_lengths(B, mode):
    """Three requests over one shared prefix: the same as each request with a cache
    of its own. Same kernels, other grouping of the keys: fp32 noise, or that of
    bf16 weights, through a few steps."""
    dtype, tdt = mode
    import dataclasses
    from prefix_kv_cached_b200.runner import Qi21Runner
    w = dataclasses.replace(C.make_workload("small64"), batch=3)
    _, wts = oracle_model(w, "float32" if dtype == B.QI21_DTYPE_F32 else "bfloat16")
    pre1 = torch.from_numpy(C.host_prefix_hidden(dataclasses.replace(w, batch=1)).astype(np.float32)).cuda()
    _, x0 = _inputs(w)
    r = Qi21Runner(w, dtype, host_weights=wts, shared_prefix=True)
    a = r.denoise_kv4(pre1, x0, w.sigmas[:4])
    s = Qi21Runner(w, dtype, share_weights_with=r)
    b = s.denoise_kv4(pre1.repeat(3, 1, 1), x0, w.sigmas[:4])
    tol = 1e-5 if dtype == B.QI21_DTYPE_F32 else 1e-2
    assert rel_l2(_np(a), _np(b)) < tol
    # the shared cache's weights are the sum over the requests
    r.set_target_row(w.sigmas[0])
    v = torch.empty_like(x0)
    r.set_prefix_row()
    r.prefix_extract(pre1)
    r.quantise_prefix()
    s.prefix_extract(pre1.repeat(3, 1, 1), mod_prefix=r.mod_prefix)
    s.quantise_prefix()
    s.set_target_row(w.sigmas[0])
    r.cached_step_kv4(x0, v, accumulate=True)
    s.cached_step_kv4(x0, v, accumulate=True)
    assert rel_l2(_np(r.kv4_scores)[:, 0], _np(s.kv4_scores).sum(1)) < (1e-5 if dtype == B.QI21_DTYPE_F32 else 1e-2)


def _same(a, b, dtype, B):
    """float32 steps give the same bits; in bf16 the block's GEMMs add the partial
    tiles of their last wave into the residual stream in no fixed order, so two
    steps agree to bf16 roundings."""
    return torch.equal(a, b) if dtype == B.QI21_DTYPE_F32 else rel_l2(_np(a), _np(b)) < 1e-2


def test_runs_with_eviction_are_reproducible(B):
    """A whole image with the prefix halved after the first step, twice: the same bits.
    An image over the 4-bit prefix is nearer to the ordinary one than an image with a
    single prefix row is."""
    from prefix_kv_cached_b200.runner import Qi21Runner
    w = C.make_workload("small")
    _, wts = oracle_model(w, "float32")
    r = Qi21Runner(w, B.QI21_DTYPE_F32, host_weights=wts)
    pre, x0 = _inputs(w)
    a = r.denoise_kv4(pre, x0, keep=99, n_protected=20)
    b = r.denoise_kv4(pre, x0, keep=99, n_protected=20)
    assert torch.equal(a, b) and r.kv4.n_prefix == 99
    full, four = r.denoise(pre, x0), r.denoise_kv4(pre, x0)
    one = r.denoise_kv4(pre, x0, keep=1)
    near, far = rel_l2(_np(four), _np(full)), rel_l2(_np(one), _np(full))
    assert near < far
    with pytest.raises(ValueError):
        r.evict_prefix(1)


@pytest.mark.parametrize("mode", ["f32", "bf16"], indirect=True)
def test_captured_step_and_two_streams(B, mode):
    """Steps captured into a graph replay to the same bits, with another prefix and
    latent in the same buffers too; two streams with a workspace each do not disturb
    one another."""
    from prefix_kv_cached_b200.runner import Qi21Runner
    w = C.make_workload("small64")
    dtype, _ = mode
    _, wts = oracle_model(w, "float32" if dtype == B.QI21_DTYPE_F32 else "bfloat16")
    pre, x0 = _inputs(w)
    r = Qi21Runner(w, dtype, host_weights=wts)
    r.set_prefix_row()
    r.prefix_extract(pre)
    r.quantise_prefix()
    r.set_target_row(w.sigmas[2])
    x, v = x0.clone(), torch.empty_like(x0)
    r.cached_step_kv4(x, v, accumulate=True)
    first, sc1 = v.clone(), r.kv4_scores.clone()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        with torch.cuda.graph(g, stream=s, capture_error_mode="thread_local"):
            r.kv4_scores.zero_()
            r.cached_step_kv4(x, v, accumulate=True)
    torch.cuda.current_stream().wait_stream(s)
    v.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert _same(v, first, dtype, B) and _same(r.kv4_scores, sc1, dtype, B)
    r.prefix_extract(pre * 0.5)
    B.check("q", B.qi21_kv4_quantize(r.cfg, r.cache, r.kv4, r.stream))
    x.copy_(x0.flip(0))
    g.replay()
    torch.cuda.synchronize()
    got = v.clone()
    r.cached_step_kv4(x, v)
    torch.cuda.synchronize()
    assert _same(got, v, dtype, B)
    del g
    # two streams at once
    t = Qi21Runner(w, dtype, share_weights_with=r)
    t.prefix_extract(pre, mod_prefix=r.mod_prefix)
    t.quantise_prefix()
    t.set_target_row(w.sigmas[2])
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    outs = {}
    for it in range(4):
        for st, run, name in ((s1, r, "a"), (s2, t, "b")):
            with torch.cuda.stream(st):
                o = torch.empty_like(x0)
                run.cached_step_kv4(x0, o)
                outs[name, it] = o
    torch.cuda.synchronize()
    for it in range(4):
        assert _same(outs["a", it], outs["a", 0], dtype, B) and _same(outs["b", it], first, dtype, B)


def test_operators_captured_and_on_two_streams(B):
    """Attention and scores alone give the same bits every time: eager, replayed, and
    with another call running beside them."""
    cfg = _cfg(B, B.QI21_DTYPE_BF16, 4, 64)
    rng = np.random.default_rng(4)
    jobs = []
    for Bn, P, N, T in ((1, 2000, 5, 3), (2, 300, 200, 100)):
        buf, _ = _kv4.make_buffer(rng, B, cfg, Bn, P)
        k4 = B.qi21_kv4_cache_init(buf, cfg, Bn, P)
        k4.state = B.QI21_CACHE_EXTRACTED
        t = {k: torch.randn(Bn, n, 256, device="cuda").bfloat16() for k, n in (("q", N), ("k", T), ("v", T))}
        n = B.qi21_kv4_workspace_bytes(cfg, Bn, N, P, T)
        t.update(buf=buf, ws=torch.zeros(n, dtype=torch.uint8, device="cuda"), out=torch.empty_like(t["q"]),
                 lse=torch.empty(4, Bn, N, device="cuda"), sc=torch.empty(Bn, 4, P, device="cuda"))

        def call(t=t, k4=k4, Bn=Bn, N=N, T=T, n=n):
            B.check("a", B.qi21_kv4_attention(cfg, k4, 0, t["q"], Bn, N, t["k"], t["v"], T, t["out"], t["lse"], t["ws"],
                                              n, _stream()))
            B.check("s", B.qi21_kv4_scores(cfg, k4, 0, t["q"], Bn, N, t["lse"], None, t["sc"], t["ws"], n, _stream()))
            return [t[k].clone() for k in ("out", "lse", "sc")]

        jobs.append((call, t, call()))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for _ in range(10):
        for (call, _, _), st in zip(jobs, streams):
            with torch.cuda.stream(st):
                got.append(call())
    torch.cuda.synchronize()
    for i, outs in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(outs, jobs[i % 2][2]))
    graphs = []
    for call, t, _ in jobs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, capture_error_mode="thread_local"):
            call()
        graphs.append(g)
    for (_, t, want), g in zip(jobs, graphs):
        for k in ("out", "lse", "sc"):
            t[k].zero_()
        g.replay()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(t[k], b) for k, b in zip(("out", "lse", "sc"), want))
    del graphs


def test_dequantised_cache_runs_the_ordinary_step(B):
    """The values written back into a bf16 cache give the ordinary cached step the
    same prefix: both steps agree to the rounding of the weights."""
    from prefix_kv_cached_b200.runner import Qi21Runner
    w = C.make_workload("small")
    _, wts = oracle_model(w, "bfloat16")
    pre, x0 = _inputs(w)
    r = Qi21Runner(w, B.QI21_DTYPE_BF16, host_weights=wts)
    r.set_prefix_row()
    r.prefix_extract(pre)
    r.quantise_prefix()
    r.set_target_row(w.sigmas[0])
    a, b = torch.empty_like(x0), torch.empty_like(x0)
    r.cached_step_kv4(x0, a)
    B.check("dequantize", B.qi21_kv4_dequantize(r.cfg, r.kv4, r.cache, r.stream))
    r.cached_step(x0, b)
    assert rel_l2(_np(a), _np(b)) < 1e-2


def test_long_prefix_offsets_beyond_32_bits(B):
    """A layer whose first row lies beyond 2^32 bytes of codes."""
    cfg = _cfg(B, B.QI21_DTYPE_BF16, 32, 128, 32)
    P = 33000
    Pp = _kv4.pad(P)
    buf = torch.zeros(B.qi21_kv4_cache_bytes(cfg, 1, P), dtype=torch.uint8, device="cuda")
    assert buf.numel() > 2 ** 32
    rng = np.random.default_rng(0)
    x = rng.standard_normal((2, 1, 32, P, 128)).astype(np.float32)
    one = _cfg(B, B.QI21_DTYPE_BF16, 32, 128, 1)
    src = torch.from_numpy(x.transpose(0, 1, 3, 2, 4).copy()).view(1, 2, 1, P, 4096)
    src = torch.cat((src, torch.zeros(1, 2, 1, 1, 4096)), 3).bfloat16().cuda()
    cache = B.qi21_kv_cache_init(src, one, 1, P, 1)
    cache.state = B.QI21_CACHE_EXTRACTED
    b1 = torch.zeros(B.qi21_kv4_cache_bytes(one, 1, P), dtype=torch.uint8, device="cuda")
    k1 = B.qi21_kv4_cache_init(b1, one, 1, P)
    assert B.qi21_kv4_quantize(one, cache, k1, _stream()) == B.QI21_OK
    nc, ns = 2 * 32 * Pp * 64, 2 * 32 * Pp * 8
    buf[31 * nc: 32 * nc] = b1[:nc]
    buf[32 * nc + 31 * ns:] = b1[nc:]
    k32 = B.qi21_kv4_cache_init(buf, cfg, 1, P)
    k32.state = B.QI21_CACHE_EXTRACTED
    for N in (2, 150):
        q = torch.randn(1, N, 4096, device="cuda").bfloat16()
        a, la = _run_attention(B, one, k1, q, None, None)
        b, lb = _run_attention(B, cfg, k32, q, None, None, layer=31)
        assert torch.equal(a, b) and torch.equal(la, lb)
    sc = torch.rand(32, 1, 32, P, device="cuda")
    keep = 700
    out = torch.zeros(B.qi21_kv4_cache_bytes(cfg, 1, keep), dtype=torch.uint8, device="cuda")
    small = B.qi21_kv4_cache_init(out, cfg, 1, keep)
    kept = torch.zeros(32, 1, 32, keep, dtype=torch.int32, device="cuda")
    assert B.qi21_kv4_evict(cfg, k32, sc, keep, 0, small, kept, _stream()) == B.QI21_OK
    want = torch.topk(sc[31, 0, 5], keep).indices.sort().values
    assert torch.equal(kept[31, 0, 5].long(), want)
    codes, _ = _kv4.buffer_views(out, 32, 1, 32, keep, 128)
    c1, _ = _kv4.buffer_views(b1, 1, 1, 32, P, 128)
    assert torch.equal(codes[31, 1, 0, 5, :keep], c1[0, 1, 0, 5][want])
