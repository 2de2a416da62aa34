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
