"""The attention weights that cached steps over a 4-bit prefix accumulate, against the
oracle's own attention of every layer, item and head; and steps, weights and eviction
over items of different lengths.

Tolerances. The step's tensors are within eps of the oracle's (F32_TOL as the largest
error, BF16_TOL in the 2-norm). Rows of q and k have norm sqrt(Dh), so eps in q moves a
score by eps sqrt(Dh) if it all points along k, and by eps if it points nowhere in
particular; a weight has the error of its score and of its log-sum-exp.
* F32: twice the worst case, 2 sqrt(128) 1e-4 = 2.3e-3, in the 2-norm of a head's rows.
* BF16: two errors of 2e-2 in no particular direction, sqrt(2) 2e-2 a weight; twice
  that, 5.7e-2, in the same norm.
"""
import dataclasses
from types import SimpleNamespace
from unittest import mock

import numpy as np
import pytest
import torch

from oracle import qi21_oracle as O
from qi21_synth import configs as C
from tests import _kv4
from tests._harness import BF16_TOL, F32_TOL, max_rel, oracle_model, rel_l2

pytestmark = pytest.mark.gpu
W_TOL = {"f32": 2.3e-3, "bf16": 5.7e-2, "bf16_cuda_cores": 5.7e-2}


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
    """(mode, dtype); switches the kernel family for the test."""
    B.qi21_set_tensor_cores(0 if request.param == "bf16_cuda_cores" else 1)
    yield request.param, B.QI21_DTYPE_F32 if request.param == "f32" else B.QI21_DTYPE_BF16
    B.qi21_set_tensor_cores(1)


def _np(t):
    return t.double().cpu().numpy()


def _oracle_step(model, seq, ck, cv, x, sigma):
    """The oracle's cached step over any prefix rows ck, cv [L][rows][H][Dh]: v, and the
    weight that each row has in every layer and head, summed over the target rows
    [L][H][rows]."""
    n, weights = ck.shape[1], []
    attention = O.masked_softmax_attention

    def recorded(q, k, v, allowed):
        x = q @ np.swapaxes(k, -1, -2) / np.sqrt(q.shape[-1])
        e = np.exp(x - x.max(-1, keepdims=True))
        weights.append((e / e.sum(-1, keepdims=True))[..., :n].sum(1))
        return attention(q, k, v, allowed)

    s = SimpleNamespace(P=n, N=seq.N, coords=np.concatenate((np.zeros((n, 3), seq.coords.dtype), seq.coords[seq.P:])),
                        allowed=np.ones((n + seq.N, n + seq.N), bool))
    mt, sf = O.modulation(1000.0 * sigma, model.wts, model.n_chunks)
    with mock.patch.object(O, "masked_softmax_attention", recorded):
        v, _, _ = O.cached_step(model, s, ck, cv, x, mt, sf)
    return v, np.stack(weights)


def _setup(B, name, batch, which, dtype):
    from prefix_kv_cached_b200.runner import Qi21Runner
    w = dataclasses.replace(C.make_workload(name), batch=batch)
    model, wts = oracle_model(w, "float32" if which == "f32" else "bfloat16")
    r = Qi21Runner(w, dtype, host_weights=wts)
    pre, x = (torch.from_numpy(f(w).astype(np.float32)).cuda() for f in (C.host_prefix_hidden, C.host_noise))
    r.set_prefix_row()
    r.prefix_extract(pre)
    r.quantise_prefix()
    return r, w, model, O.make_sequence(w.segments), x


def _far(a, b):
    """Largest relative 2-norm over the (layer, head) rows of two [L][H][rows]."""
    return max(rel_l2(a[l, h], b[l, h]) for l in range(a.shape[0]) for h in range(a.shape[1]))


@pytest.mark.parametrize("mode", ["f32", "bf16", "bf16_cuda_cores"], indirect=True)
@pytest.mark.parametrize("name", ["small", "small64"])
def test_weights_of_a_step_are_the_oracles(B, mode, name):
    """Of each layer, item and head by itself, after one step and after a second one on
    top. Mistaken layers, heads, items or rows, planted on the oracle's side, are far
    beyond the tolerance."""
    which, dtype = mode
    r, w, model, seq, x = _setup(B, name, 2, which, dtype)
    L, H, Dh = w.shape.n_layers, w.shape.n_heads, w.shape.head_dim
    vals = _kv4.read_values(r.kv4_buf, L, r.Bn, H, r.P, Dh)
    v, tol, want = torch.empty_like(x), W_TOL[which], np.zeros((2, L, H, r.P))
    for sigma in w.sigmas[:2]:
        r.set_target_row(sigma)
        r.cached_step_kv4(x, v, accumulate=True)
        B.check("device", B.qi21_check_device_error(r.kv4_ws, r.kv4_ws.numel(), r.stream))
        for b in range(2):
            ck, cv = (vals[:, i, b].transpose(0, 2, 1, 3) for i in range(2))
            vo, wt = _oracle_step(model, seq, ck, cv, _np(x)[b], sigma)
            want[b] += wt
            metric, vt = (max_rel, F32_TOL) if which == "f32" else (rel_l2, BF16_TOL)
            assert metric(_np(v)[b], vo) < vt
            assert _far(_np(r.kv4_scores)[:, b], want[b]) < tol, (sigma, b)
    for wrong in (want[:, ::-1], want[:, :, ::-1], want[::-1], np.roll(want, 1, 3), want * 2):
        assert max(_far(wrong[b], want[b]) for b in range(2)) > 3 * tol


@pytest.mark.parametrize("mode", ["f32", "bf16", "bf16_cuda_cores"], indirect=True)
@pytest.mark.parametrize("name", ["small", "small64"])
def test_steps_and_eviction_over_items_of_different_lengths(B, mode, name):
    """A whole prefix, none at all, and a third of one: a step with its weights, an
    eviction, a step on what it has kept with the lengths that it wrote. Each item
    against the oracle on its own rows; rows that do not exist hold NaN scales."""
    which, dtype = mode
    r, w, model, seq, x = _setup(B, name, 3, which, dtype)
    L, H, Dh, P = w.shape.n_layers, w.shape.n_heads, w.shape.head_dim, r.P
    lens, keep, prot = [P, 0, P // 3], P // 2, 5
    vals = _kv4.read_values(r.kv4_buf, L, 3, H, P, Dh)
    codes, scales = _kv4.buffer_views(r.kv4_buf, L, 3, H, P, Dh)
    for b, n in enumerate(lens):
        codes[:, :, b, :, n:] = 0xFF
        scales[:, :, b, :, n:] = float("nan")
    lt = torch.tensor(lens + [0], dtype=torch.int32, device="cuda")
    r.kv4.prefix_len = lt.data_ptr()
    metric, vt = (max_rel, F32_TOL) if which == "f32" else (rel_l2, BF16_TOL)
    v = torch.empty_like(x)
    r.set_target_row(w.sigmas[0])
    r.cached_step_kv4(x, v, accumulate=True)
    B.check("device", B.qi21_check_device_error(r.kv4_ws, r.kv4_ws.numel(), r.stream))
    sc = r.kv4_scores
    for b, n in enumerate(lens):
        ck, cv = (vals[:, i, b, :, :n].transpose(0, 2, 1, 3) for i in range(2))
        vo, wt = _oracle_step(model, seq, ck, cv, _np(x)[b], w.sigmas[0])
        assert metric(_np(v)[b], vo) < vt, b
        if n:
            assert _far(_np(sc)[:, b, :, :n], wt) < W_TOL[which], b
        assert (sc[:, b, :, n:] == 0).all()
    buf = torch.full((B.qi21_kv4_cache_bytes(r.cfg, 3, keep),), 0xFF, dtype=torch.uint8, device="cuda")
    lo = torch.full((4,), -7, dtype=torch.int32, device="cuda")
    small = B.qi21_kv4_cache_init(buf, r.cfg, 3, keep, lo)
    kept = torch.empty(L, 3, H, keep, dtype=torch.int32, device="cuda")
    B.check("evict", B.qi21_kv4_evict(r.cfg, r.kv4, sc, keep, prot, small, kept, r.stream))
    rows = kept.cpu().numpy()
    assert np.array_equal(rows, _kv4.evict(sc.cpu().numpy(), lens, keep, prot))
    have = [min(keep, n) for n in lens]
    assert lo.tolist() == have + [-7]
    n_ws = B.qi21_kv4_step_workspace_bytes(r.cfg, 3, keep, r.N)
    ws = torch.zeros(n_ws, dtype=torch.uint8, device="cuda")
    r.set_target_row(w.sigmas[1])
    B.check("step", B.qi21_cached_step_kv4(r.cfg, r.wstruct, small, 3, r.N, x, r.cos_sin_target, r.mod_target,
                                           r.scale_final, v, None, ws, n_ws, r.stream))
    B.check("device", B.qi21_check_device_error(ws, n_ws, r.stream))
    for b, n in enumerate(have):
        # head h of layer l reads the rows that it has kept
        ck, cv = (np.stack([np.stack([vals[l, i, b, h][rows[l, b, h, :n]] for h in range(H)], 1) for l in range(L)])
                  for i in range(2))
        vo, _ = _oracle_step(model, seq, ck, cv, _np(x)[b], w.sigmas[1])
        assert metric(_np(v)[b], vo) < vt, b
