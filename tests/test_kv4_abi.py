"""The 4-bit prefix cache without a GPU: sizes, the format's exactness in bf16,
and the calls that are refused before anything is enqueued."""
import numpy as np
import pytest

from qi21_synth import configs as C
from tests import _kv4

FAKE = 0x100000          # aligned, never dereferenced on these paths


@pytest.fixture(scope="module")
def B():
    from prefix_kv_cached_b200 import build
    build.build()
    from prefix_kv_cached_b200 import binding
    return binding


def _cfg(B, dtype=0, shape=C.SMALL):
    from prefix_kv_cached_b200.runner import make_config
    return make_config(shape, dtype)


def test_values_of_the_format_are_exact_in_bf16():
    """(nibble - 8) times a 5-bit significand has at most 8 bits, and 7 s bounds the group."""
    import torch
    k = np.arange(-7, 8)[:, None] * _kv4.SCALES[None]
    assert (torch.from_numpy(k).to(torch.bfloat16).double().numpy() == k).all()
    rng = np.random.default_rng(3)
    x = rng.standard_normal((500, 64)) * np.exp(rng.standard_normal((500, 1)) * 5)
    c, s = _kv4.quantise(x)
    err = np.abs(_kv4.values(c, s) - x).reshape(500, 2, 32)
    assert (err <= s[..., None] / 2).all()
    a = np.abs(x).reshape(500, 2, 32).max(-1)
    assert (7 * s >= a).all() and (7 * s <= a * (1 + 1 / 16)).all()


def test_sizes_and_init(B):
    cfg = _cfg(B)
    for P, Bn in ((1, 1), (128, 3), (129, 2)):
        rows = cfg.n_layers * 2 * Bn * cfg.n_heads * _kv4.pad(P)
        assert B.qi21_kv4_cache_bytes(cfg, Bn, P) == rows * 64 + rows * 8
    assert B.qi21_kv4_cache_bytes(cfg, 1, 0) == 0 and B.qi21_kv4_cache_bytes(cfg, 0, 1) == 0
    c = B.qi21_kv4_cache_init(FAKE, cfg, 2, 130, FAKE)
    assert (c.batch, c.n_prefix, c.n_heads, c.head_dim, c.state) == (2, 130, 2, 128, B.QI21_CACHE_EMPTY)
    toy = _cfg(B, shape=C.TOY)            # head_dim 4: no group of 32
    assert B.qi21_kv4_cache_bytes(toy, 1, 8) == 0 and B.qi21_kv4_workspace_bytes(toy, 1, 1, 8, 0) == 0
    for bad, status in (((FAKE + 8, cfg, 1, 8), B.QI21_ERR_INVALID_ARG), ((FAKE, cfg, 0, 8), B.QI21_ERR_SHAPE),
                        ((FAKE, cfg, 1, 0), B.QI21_ERR_SHAPE), ((FAKE, toy, 1, 8), B.QI21_ERR_UNSUPPORTED),
                        ((FAKE, cfg, 1, 8, FAKE + 4), B.QI21_ERR_INVALID_ARG)):
        with pytest.raises(B.Qi21Error) as e:
            B.qi21_kv4_cache_init(*bad)
        assert e.value.status == status
    assert B.qi21_kv4_workspace_bytes(cfg, 1, 1, 8, -1) == 0
    assert B.qi21_kv4_step_workspace_bytes(cfg, 1, 8, 4) > B.qi21_kv4_workspace_bytes(cfg, 1, 4, 8, 4) > 0


def test_quantise_refusals(B):
    cfg = _cfg(B)
    src = B.qi21_kv_cache_init(FAKE, cfg, 2, 8, 4)
    dst = B.qi21_kv4_cache_init(FAKE, cfg, 2, 8)
    assert B.qi21_kv4_quantize(cfg, src, dst) == B.QI21_ERR_CACHE_STATE          # not extracted
    assert B.qi21_kv4_dequantize(cfg, dst, src) == B.QI21_ERR_CACHE_STATE
    src.state = dst.state = B.QI21_CACHE_EXTRACTED
    for other in (B.qi21_kv4_cache_init(FAKE, cfg, 1, 8), B.qi21_kv4_cache_init(FAKE, cfg, 2, 9)):
        other.state = B.QI21_CACHE_EXTRACTED
        assert B.qi21_kv4_quantize(cfg, src, other) == B.QI21_ERR_CACHE_STATE
        assert B.qi21_kv4_dequantize(cfg, other, src) == B.QI21_ERR_CACHE_STATE
    assert B.qi21_kv4_quantize(_cfg(B, B.QI21_DTYPE_BF16), src, dst) == B.QI21_ERR_CACHE_STATE    # src is float32
    shared = B.qi21_kv_cache_init_shared(FAKE, cfg, 2, 8, 4)
    shared.state = B.QI21_CACHE_EXTRACTED
    assert B.qi21_kv4_quantize(cfg, shared, dst) == B.QI21_ERR_CACHE_STATE       # a shared prefix has one item
    toy = _cfg(B, shape=C.TOY)
    assert B.qi21_kv4_quantize(toy, src, dst) == B.QI21_ERR_UNSUPPORTED
    dst.prefix_len = FAKE + 4
    assert B.qi21_kv4_quantize(cfg, src, dst) == B.QI21_ERR_INVALID_ARG
    dst.prefix_len = None
    dst.base = FAKE + 8
    assert B.qi21_kv4_quantize(cfg, src, dst) == B.QI21_ERR_INVALID_ARG


def test_attention_and_scores_refusals(B):
    cfg = _cfg(B)
    k4 = B.qi21_kv4_cache_init(FAKE, cfg, 2, 8)
    n = B.qi21_kv4_workspace_bytes(cfg, 2, 5, 8, 3)

    def att(layer=0, q=FAKE, batch=2, n_q=5, kt=FAKE, vt=FAKE, nt=3, out=FAKE, lse=FAKE, ws=FAKE, wsb=n, c=cfg, k=k4):
        return B.qi21_kv4_attention(c, k, layer, q, batch, n_q, kt, vt, nt, out, lse, ws, wsb)

    def sc(layer=0, q=FAKE, batch=2, n_q=5, lse=FAKE, si=FAKE, so=FAKE, ws=FAKE, wsb=n, c=cfg, k=k4):
        return B.qi21_kv4_scores(c, k, layer, q, batch, n_q, lse, si, so, ws, wsb)

    assert att() == sc() == B.QI21_ERR_CACHE_STATE                               # nothing in it yet
    k4.state = B.QI21_CACHE_EXTRACTED
    for kw in (dict(layer=-1), dict(layer=cfg.n_layers), dict(q=FAKE + 4), dict(lse=FAKE + 4), dict(ws=0)):
        assert att(**kw) == B.QI21_ERR_INVALID_ARG and sc(**kw) == B.QI21_ERR_INVALID_ARG
    for kw in (dict(kt=0), dict(vt=FAKE + 8), dict(out=0)):
        assert att(**kw) == B.QI21_ERR_INVALID_ARG
    for kw in (dict(lse=0), dict(si=FAKE + 4), dict(so=0)):
        assert sc(**kw) == B.QI21_ERR_INVALID_ARG
    for kw in (dict(batch=0), dict(n_q=0)):
        assert att(**kw) == B.QI21_ERR_SHAPE and sc(**kw) == B.QI21_ERR_SHAPE
    assert att(nt=-1) == B.QI21_ERR_SHAPE
    assert att(batch=3) == sc(batch=3) == B.QI21_ERR_CACHE_STATE                 # two items, three requests
    assert att(wsb=n - 1) == B.QI21_ERR_WORKSPACE_TOO_SMALL
    assert sc(wsb=64) == B.QI21_ERR_WORKSPACE_TOO_SMALL
    assert att(c=_cfg(B, shape=C.SMALL64)) == B.QI21_ERR_CACHE_STATE             # another model's cache
    one = B.qi21_kv4_cache_init(FAKE, cfg, 1, 8)
    one.state = B.QI21_CACHE_EXTRACTED
    assert att(k=one, batch=2 ** 20, n_q=2 ** 12) == B.QI21_ERR_SHAPE            # rows beyond 32 bits
    assert B.qi21_kv4_attention(cfg, k4, 0, FAKE, 2, 5, 0, 0, 0, FAKE, 0, FAKE, 0) == B.QI21_ERR_WORKSPACE_TOO_SMALL


def test_evict_refusals(B):
    cfg = _cfg(B)
    src = B.qi21_kv4_cache_init(FAKE, cfg, 2, 200)
    far = FAKE + B.qi21_kv4_cache_bytes(cfg, 2, 200)
    dst = B.qi21_kv4_cache_init(far, cfg, 2, 50)

    def ev(scores=FAKE, keep=50, prot=10, s=src, d=dst, kept=FAKE):
        return B.qi21_kv4_evict(cfg, s, scores, keep, prot, d, kept)

    assert ev() == B.QI21_ERR_CACHE_STATE
    src.state = B.QI21_CACHE_EXTRACTED
    assert ev(keep=0) == ev(keep=201) == ev(prot=51) == ev(prot=-1) == B.QI21_ERR_SHAPE
    assert ev(keep=49) == B.QI21_ERR_CACHE_STATE                                 # dst holds 50 rows
    assert ev(d=B.qi21_kv4_cache_init(far, cfg, 1, 50)) == B.QI21_ERR_CACHE_STATE
    assert ev(scores=FAKE + 4) == ev(kept=0) == B.QI21_ERR_INVALID_ARG
    for base in (FAKE, far - 16, FAKE - B.qi21_kv4_cache_bytes(cfg, 2, 50) + 16):     # overlapping buffers
        assert ev(d=B.qi21_kv4_cache_init(base, cfg, 2, 50)) == B.QI21_ERR_INVALID_ARG
    src.prefix_len = FAKE
    assert ev() == B.QI21_ERR_INVALID_ARG                                        # lengths need a place to go
    assert ev(d=B.qi21_kv4_cache_init(far, cfg, 2, 50, FAKE)) == B.QI21_ERR_INVALID_ARG    # and one of their own


def test_step_refusals(B):
    cfg = _cfg(B)
    w = B.qi21_weights(*([FAKE] * 15))
    k4 = B.qi21_kv4_cache_init(FAKE, cfg, 2, 8)
    n = B.qi21_kv4_step_workspace_bytes(cfg, 2, 8, 4)

    def step(batch=2, x=FAKE, scores=0, wsb=n, weights=w):
        return B.qi21_cached_step_kv4(cfg, weights, k4, batch, 4, x, FAKE, FAKE, FAKE, FAKE, scores, FAKE, wsb)

    assert step() == B.QI21_ERR_CACHE_STATE
    k4.state = B.QI21_CACHE_EXTRACTED
    assert step(x=FAKE + 4) == step(scores=FAKE + 4) == B.QI21_ERR_INVALID_ARG
    assert step(weights=B.qi21_weights(*([0] * 15))) == B.QI21_ERR_INVALID_ARG
    assert step(batch=4) == B.QI21_ERR_CACHE_STATE
    assert step(wsb=n - 1) == B.QI21_ERR_WORKSPACE_TOO_SMALL
