"""Buffers of one 4-bit cache call that overlap, refused on the host before anything
is enqueued."""
import pytest

from qi21_synth import configs as C

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


@pytest.mark.parametrize("src_len,dst_len", [(0, 0), (0, 16), (16, 0), (0, 32), (32, 0)])
def test_evict_lengths_that_overlap(B, src_len, dst_len):
    """Nine items' lengths are 36 bytes: arrays 16 or 32 bytes apart share some."""
    cfg = _cfg(B)
    far = FAKE + B.qi21_kv4_cache_bytes(cfg, 9, 200)
    src = B.qi21_kv4_cache_init(FAKE, cfg, 9, 200, FAKE + src_len)
    dst = B.qi21_kv4_cache_init(far, cfg, 9, 50, FAKE + dst_len)
    src.state = B.QI21_CACHE_EXTRACTED
    assert B.qi21_kv4_evict(cfg, src, FAKE, 50, 0, dst, FAKE) == B.QI21_ERR_INVALID_ARG


@pytest.mark.parametrize("shared", [False, True])
def test_quantise_and_the_way_back_in_place(B, shared):
    """A 4-bit cache inside the cache it is made from, at its start, or across one end."""
    cfg = _cfg(B)
    base = FAKE + (1 << 30)
    init, size = ((B.qi21_kv_cache_init_shared, B.qi21_kv_cache_bytes_shared) if shared else
                  (B.qi21_kv_cache_init, B.qi21_kv_cache_bytes))
    src = init(base, cfg, 2, 200, 300)
    n, n4 = size(cfg, 2, 200, 300), B.qi21_kv4_cache_bytes(cfg, 1 if shared else 2, 200)
    assert n > n4
    for at in (base, base + 16, base + n - 16, base - n4 + 16):
        k4 = B.qi21_kv4_cache_init(at, cfg, 1 if shared else 2, 200)
        src.state = k4.state = B.QI21_CACHE_EXTRACTED
        assert B.qi21_kv4_quantize(cfg, src, k4) == B.QI21_ERR_INVALID_ARG
        assert B.qi21_kv4_dequantize(cfg, k4, src) == B.QI21_ERR_INVALID_ARG
        assert src.state == k4.state == B.QI21_CACHE_EXTRACTED          # nothing has happened
