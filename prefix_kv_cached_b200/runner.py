"""Device-side driver of one model instance over the C ABI.

Owns the torch-allocated device buffers (K/V cache, workspace, metadata
tables, modulation rows) and calls the library's entry points; it computes
nothing itself. The caller supplies the weights, either as host arrays (copied
to the device once) or as device tensors it already holds, and a description
of the model and the sequence: an object with ``shape`` (the fields of
``qi21_config`` plus ``rope``: "axial" or "lab"), ``segments`` (kind, n_text | h,
w), ``batch``, ``n_prefix`` and ``n_target``.
"""
from __future__ import annotations

from typing import Dict, Optional

import numpy as np
import torch

from . import binding as B

_TORCH_DTYPE = {B.QI21_DTYPE_F32: torch.float32, B.QI21_DTYPE_BF16: torch.bfloat16}

# qi21_weights field order
WEIGHT_NAMES = ("w_img_in", "w_out", "w_t1", "w_t2", "w_mod", "w_fin", "w_q", "w_k", "w_v", "w_o", "w_gate",
                "w_up", "w_down", "q_norm", "k_norm")
NORM_WEIGHTS = ("q_norm", "k_norm")      # float32 in both storage modes


def make_config(shape, dtype: int) -> B.qi21_config:
    return B.qi21_config(shape.d_model, shape.n_heads, shape.head_dim, shape.n_layers, shape.mlp_hidden,
                         shape.latent_ch, shape.time_dim, dtype, shape.use_shift, shape.ln_eps, shape.qk_eps)


class Qi21Runner:
    def __init__(self, workload, dtype: int = B.QI21_DTYPE_F32, device: str = "cuda",
                 host_weights: Optional[Dict[str, np.ndarray]] = None,
                 weights: Optional[Dict[str, torch.Tensor]] = None, frame_mode: int = 0,
                 shared_prefix: bool = False, share_weights_with: Optional["Qi21Runner"] = None):
        """Weights: exactly one of host_weights (arrays holding the stored values,
        copied to the device in the storage dtype), weights (device tensors in the
        storage dtype, norm weights float32) or share_weights_with (another
        runner's device weights). shared_prefix: the batch items are requests
        sharing one prefix (one extract from prefix_hidden [1][P][d], every
        request's attention reading the one copy)."""
        if sum(x is not None for x in (host_weights, weights, share_weights_with)) != 1:
            raise ValueError("give exactly one of host_weights, weights, share_weights_with")
        self.w = workload
        self.shape = workload.shape
        self.dtype = dtype
        self.tdtype = _TORCH_DTYPE[dtype]
        self.device = torch.device(device)
        if self.device.type == "cuda" and self.device.index is None:
            self.device = torch.device("cuda", torch.cuda.current_device())
        self.cfg = make_config(self.shape, dtype)
        sh = self.shape
        self.meta = B.qi21_build_metadata(list(workload.segments), frame_mode)
        self.S, self.P, self.N = self.meta["S"], self.meta["P"], self.meta["N"]
        assert (self.P, self.N) == (workload.n_prefix, workload.n_target)
        self.Bn = workload.batch
        omega = B.qi21_rope_omega_lab() if sh.rope == "lab" else B.qi21_rope_omega_axial(sh.head_dim)
        cs = B.qi21_rope_table(sh.head_dim, self.meta["coords"], omega)
        self.cos_sin_all = torch.from_numpy(cs).to(self.device)
        self.cos_sin_prefix = self.cos_sin_all[: self.P].contiguous()
        self.cos_sin_target = self.cos_sin_all[self.P:].contiguous()
        lim = torch.from_numpy(self.meta["kv_limit"].astype(np.int32)).to(self.device)
        self.kv_limit_all = lim
        self.kv_limit_prefix = lim[: self.P].contiguous()
        self.weights: Dict[str, torch.Tensor] = {}
        self.shared_prefix = shared_prefix
        for name in WEIGHT_NAMES:
            sdt = torch.float32 if name in NORM_WEIGHTS else self.tdtype
            if share_weights_with is not None:
                t = share_weights_with.weights[name]
            elif weights is not None:
                t = weights[name]
            else:
                t = torch.from_numpy(np.ascontiguousarray(host_weights[name])).to(device=self.device, dtype=sdt)
            if t.dtype != sdt or t.device != self.device or not t.is_contiguous():
                raise ValueError(f"weight {name}: expected a contiguous {sdt} tensor on {self.device}")
            self.weights[name] = t
        self.wstruct = B.qi21_weights(*[self.weights[n].data_ptr() for n in WEIGHT_NAMES])
        self._allocate()
        nch = 6 if sh.use_shift else 4
        self.mod_prefix = torch.zeros(nch * sh.d_model, dtype=torch.float32, device=self.device)
        self.mod_target = torch.zeros_like(self.mod_prefix)
        self.scale_final = torch.zeros(sh.d_model, dtype=torch.float32, device=self.device)
        self._sf0 = torch.zeros_like(self.scale_final)
        # the 4-bit prefix cache (quantise_prefix)
        self.kv4: Optional[B.qi21_kv4_cache] = None
        self.kv4_buf: Optional[torch.Tensor] = None
        self.kv4_scores: Optional[torch.Tensor] = None
        self.kv4_ws: Optional[torch.Tensor] = None

    def _allocate(self):
        """The K/V cache, empty, and the workspace."""
        if self.shared_prefix:
            kvb = B.qi21_kv_cache_bytes_shared(self.cfg, self.Bn, self.P, self.N)
            self.cache_buf = torch.zeros(kvb, dtype=torch.uint8, device=self.device)
            self.cache = B.qi21_kv_cache_init_shared(self.cache_buf, self.cfg, self.Bn, self.P, self.N)
        else:
            kvb = B.qi21_kv_cache_bytes(self.cfg, self.Bn, self.P, self.N)
            self.cache_buf = torch.zeros(kvb, dtype=torch.uint8, device=self.device)
            self.cache = B.qi21_kv_cache_init(self.cache_buf, self.cfg, self.Bn, self.P, self.N)
        self.ws_bytes = B.qi21_workspace_bytes(self.cfg, self.Bn, self.P, self.N)
        self.ws = torch.zeros(self.ws_bytes, dtype=torch.uint8, device=self.device)

    @property
    def stream(self) -> int:
        return torch.cuda.current_stream(self.device).cuda_stream

    def _in_use(self, *buffers: Optional[torch.Tensor]):
        """The current stream has work on these buffers. A later call, on whatever
        stream, may drop them; the allocator must not give their memory to the stream
        they were allocated on before this work is done."""
        if self.device.type == "cuda":
            s = torch.cuda.current_stream(self.device)
            for t in buffers:
                if t is not None:
                    t.record_stream(s)

    def _extracting(self):
        """Before a call that needs the cache and the workspace, whatever the cache holds."""
        if self.ws is None:
            self._allocate()
        self._in_use(self.cache_buf, self.ws)

    def _extracted(self):
        """Before a call that reads the extracted cache."""
        if self.ws is None:
            raise ValueError("the extracted cache was released; this needs a prefix_extract before it")
        self._in_use(self.cache_buf, self.ws)

    def _any_ws(self) -> torch.Tensor:
        """The workspace, or once it is released that of the 4-bit steps (the calls of a
        step use one after the other)."""
        ws = self.kv4_ws if self.ws is None else self.ws
        self._in_use(ws)
        return ws

    # ------------------------------------------------------------------ calls
    def modulation(self, t: float, mod_row: torch.Tensor, scale_final: torch.Tensor):
        ws = self._any_ws()
        B.check("qi21_modulation", B.qi21_modulation(self.cfg, self.wstruct, t, mod_row, scale_final, ws,
                                                     ws.numel(), self.stream))

    def set_prefix_row(self):
        """Prefix modulation row at t = 0 (3B page: prefix tokens read t = 0)."""
        self.modulation(0.0, self.mod_prefix, self._sf0)

    def set_target_row(self, sigma: float):
        """Target modulation row and final scale at noise level sigma (the library
        forms t = QI21_T_PER_SIGMA * sigma)."""
        ws = self._any_ws()
        B.check("qi21_modulation_sigma", B.qi21_modulation_sigma(self.cfg, self.wstruct, float(sigma),
                                                                 self.mod_target, self.scale_final, ws,
                                                                 ws.numel(), self.stream))

    def prefix_extract(self, prefix_hidden: torch.Tensor, mod_prefix: Optional[torch.Tensor] = None):
        self._extracting()
        B.check("qi21_prefix_extract", B.qi21_prefix_extract(
            self.cfg, self.wstruct, self.cache, prefix_hidden, self.cos_sin_prefix, self.kv_limit_prefix,
            self.mod_prefix if mod_prefix is None else mod_prefix, self.ws, self.ws_bytes, self.stream))

    def cached_step(self, x: torch.Tensor, v_out: torch.Tensor):
        self._extracted()
        B.check("qi21_cached_step", B.qi21_cached_step(
            self.cfg, self.wstruct, self.cache, x, self.cos_sin_target, self.mod_target, self.scale_final, v_out,
            self.ws, self.ws_bytes, self.stream))

    def full_recompute(self, prefix_hidden: torch.Tensor, x: torch.Tensor, v_out: torch.Tensor,
                       mod_prefix: Optional[torch.Tensor] = None):
        self._extracting()
        B.check("qi21_full_recompute_step", B.qi21_full_recompute_step(
            self.cfg, self.wstruct, self.Bn, self.P, self.N, prefix_hidden, x, self.cos_sin_all, self.kv_limit_all,
            self.mod_prefix if mod_prefix is None else mod_prefix, self.mod_target, self.scale_final, v_out,
            self.ws, self.ws_bytes, self.stream))

    def euler(self, x: torch.Tensor, v: torch.Tensor, s0: float, s1: float, x_out: torch.Tensor):
        B.check("qi21_euler_update", B.qi21_euler_update(x, v, s0, s1, x_out, x.numel(), self.stream))

    # ------------------------------------------------------------------ 4-bit prefix cache

    def quantise_prefix(self, release: bool = False):
        """Hold the extracted prefix in 4 bits from here on (for cached_step_kv4), in new
        buffers: a step captured over the ones before must not be replayed any more. The
        extracted cache and its workspace are kept for the next extract, or, with
        release, given back to the allocator: the 4-bit steps do without them, the next
        prefix_extract allocates them again, and a graph of capture_image made before
        must not be replayed any more."""
        self._extracted()
        nb = 1 if self.shared_prefix else self.Bn
        buf = torch.empty(B.qi21_kv4_cache_bytes(self.cfg, nb, self.P), dtype=torch.uint8, device=self.device)
        cache4 = B.qi21_kv4_cache_init(buf, self.cfg, nb, self.P)
        ws = self._kv4_workspace(self.P)
        B.check("qi21_kv4_quantize", B.qi21_kv4_quantize(self.cfg, self.cache, cache4, self.stream))
        self.kv4, self.kv4_buf, self.kv4_scores, self.kv4_ws = cache4, buf, None, ws
        if release:
            self._carry_error(self.ws, ws)
            self.cache.state, self.cache.base = B.QI21_CACHE_EMPTY, None
            self.cache_buf = self.ws = None

    def _kv4_workspace(self, n_prefix: int) -> torch.Tensor:
        """A workspace of the 4-bit steps, to take the place of the present one."""
        ws = torch.zeros(B.qi21_kv4_step_workspace_bytes(self.cfg, self.Bn, n_prefix, self.N), dtype=torch.uint8,
                         device=self.device)
        self._carry_error(self.kv4_ws, ws)
        return ws

    def _carry_error(self, old: Optional[torch.Tensor], new: torch.Tensor):
        """A workspace begins with the device error word that check_device reads; what a
        kernel reported in one that is dropped goes into the next."""
        if old is not None:
            self._in_use(old)
            new[:4].bitwise_or_(old[:4])

    def cached_step_kv4(self, x: torch.Tensor, v_out: torch.Tensor, accumulate: bool = False):
        """The cached step over the 4-bit prefix. accumulate: add every layer's
        attention weights of this step to kv4_scores [L][items][H][rows]; the first such
        step since quantise_prefix or evict_prefix makes them and cannot be captured."""
        if self.kv4 is None:
            raise ValueError("cached_step_kv4 needs a quantise_prefix before it")
        if accumulate and self.kv4_scores is None:
            # captured, the zeros would be written again at every replay
            if self.device.type == "cuda" and torch.cuda.is_current_stream_capturing():
                raise ValueError("capture a cached_step_kv4 with accumulate=True after one that was not captured")
            k = self.kv4
            self.kv4_scores = torch.zeros(k.n_layers, k.batch, k.n_heads, k.n_prefix, dtype=torch.float32,
                                          device=self.device)
        self._in_use(self.kv4_buf, self.kv4_ws, self.kv4_scores)
        B.check("qi21_cached_step_kv4", B.qi21_cached_step_kv4(
            self.cfg, self.wstruct, self.kv4, self.Bn, self.N, x, self.cos_sin_target, self.mod_target,
            self.scale_final, v_out, self.kv4_scores if accumulate else None, self.kv4_ws, self.kv4_ws.numel(),
            self.stream))

    def evict_prefix(self, keep: int, n_protected: int = 0) -> torch.Tensor:
        """Shrink the 4-bit prefix to the `keep` rows of every head that the steps
        with accumulate=True attended to most (the first n_protected rows stay in
        any case). Returns the rows kept, int32 [L][items][H][keep]; the weights
        start again at zero. The smaller prefix is in new buffers: a step captured before
        must not be replayed any more."""
        if self.kv4_scores is None:
            raise ValueError("evict_prefix needs a cached_step_kv4 with accumulate=True before it")
        k = self.kv4
        buf = torch.empty(B.qi21_kv4_cache_bytes(self.cfg, k.batch, keep), dtype=torch.uint8, device=self.device)
        small = B.qi21_kv4_cache_init(buf, self.cfg, k.batch, keep)
        # fewer rows can need more workspace: other splits of the work, other kernels
        need = B.qi21_kv4_step_workspace_bytes(self.cfg, self.Bn, keep, self.N)
        ws = self.kv4_ws if self.kv4_ws.numel() >= need else self._kv4_workspace(keep)
        kept = torch.empty(k.n_layers, k.batch, k.n_heads, keep, dtype=torch.int32, device=self.device)
        self._in_use(self.kv4_buf, self.kv4_ws, self.kv4_scores)
        B.check("qi21_kv4_evict", B.qi21_kv4_evict(self.cfg, k, self.kv4_scores, keep, n_protected, small, kept,
                                                   self.stream))
        self.kv4, self.kv4_buf, self.kv4_scores = small, buf, None
        self.kv4_ws = ws
        return kept

    def denoise_kv4(self, prefix_hidden: torch.Tensor, x0: torch.Tensor, sigmas=None, keep: Optional[int] = None,
                    n_protected: int = 0, release: bool = False):
        """denoise() with the prefix held in 4 bits; keep: after the first step, go
        on with the `keep` prefix rows of every head that it attended to most; release:
        as in quantise_prefix."""
        sigmas = self.w.sigmas if sigmas is None else sigmas
        self.set_prefix_row()
        self.prefix_extract(prefix_hidden)
        self.quantise_prefix(release)
        x = x0.clone()
        v = torch.empty_like(x)
        for k in range(len(sigmas) - 1):
            self.set_target_row(sigmas[k])
            self.cached_step_kv4(x, v, accumulate=keep is not None and k == 0)
            if keep is not None and k == 0:
                self.evict_prefix(keep, n_protected)
            self.euler(x, v, sigmas[k], sigmas[k + 1], x)
        return x

    # ------------------------------------------------------------------ whole image

    def denoise_image(self, prefix_hidden: torch.Tensor, x: torch.Tensor, sigmas_dev: torch.Tensor,
                      v: Optional[torch.Tensor] = None) -> torch.Tensor:
        """One call of qi21_denoise_image: extract, then len(sigmas_dev) - 1 cached
        steps with Euler, all enqueued on the current stream; x is updated in
        place (x_0 in, final latent out). sigmas_dev: float64 device tensor."""
        assert sigmas_dev.dtype == torch.float64 and sigmas_dev.is_cuda and sigmas_dev.numel() >= 2
        v = torch.empty_like(x) if v is None else v
        self._extracting()
        B.check("qi21_denoise_image", B.qi21_denoise_image(
            self.cfg, self.wstruct, self.cache, prefix_hidden, self.cos_sin_prefix, self.kv_limit_prefix,
            self.cos_sin_target, sigmas_dev, sigmas_dev.numel() - 1, B.QI21_T_PER_SIGMA, x, v, self.mod_prefix,
            self.mod_target, self.scale_final, self.ws, self.ws_bytes, self.stream))
        return x

    def capture_image(self, prefix_hidden: torch.Tensor, x: torch.Tensor, sigmas_dev: torch.Tensor):
        """Capture the whole-image call into a CUDA graph (after one eager call
        that sets kernel attributes). Replaying the returned graph re-runs the
        image on the current contents of prefix_hidden, x and sigmas_dev."""
        v = torch.empty_like(x)
        x_warm = x.clone()
        self.denoise_image(prefix_hidden, x_warm, sigmas_dev, v)
        torch.cuda.synchronize(self.device)
        g = torch.cuda.CUDAGraph()
        s = torch.cuda.Stream(self.device)
        s.wait_stream(torch.cuda.current_stream(self.device))
        with torch.cuda.stream(s):
            with torch.cuda.graph(g, stream=s, capture_error_mode="thread_local"):
                self.denoise_image(prefix_hidden, x, sigmas_dev, v)
        torch.cuda.current_stream(self.device).wait_stream(s)
        return g

    def check_device(self):
        for ws in (self.ws, self.kv4_ws):
            if ws is not None:
                self._in_use(ws)
                B.check("qi21_check_device_error", B.qi21_check_device_error(ws, ws.numel(), self.stream))

    def cache_kv(self):
        """Views of the cache as K, V [L][B][P+N][H][Dh] (for tests); with a shared
        prefix, [L][Pp + B*N][H][Dh] (prefix rows [0, P), request b at Pp + b*N)."""
        self._extracted()
        sh = self.shape
        if self.shared_prefix:
            pp = -(-self.P // 128) * 128
            t = self.cache_buf.view(self.tdtype).view(sh.n_layers, 2, pp + self.Bn * self.N, sh.n_heads,
                                                      sh.head_dim)
            return t[:, 0], t[:, 1]
        t = self.cache_buf.view(self.tdtype).view(sh.n_layers, 2, self.Bn, self.P + self.N, sh.n_heads,
                                                  sh.head_dim)
        return t[:, 0], t[:, 1]

    def denoise(self, prefix_hidden: torch.Tensor, x0: torch.Tensor, sigmas=None):
        """Whole image: t = 0 prefix row, extract once, then cached steps + Euler."""
        sigmas = self.w.sigmas if sigmas is None else sigmas
        self.set_prefix_row()
        self.prefix_extract(prefix_hidden)
        x = x0.clone()
        v = torch.empty_like(x)
        for k in range(len(sigmas) - 1):
            self.set_target_row(sigmas[k])
            self.cached_step(x, v)
            self.euler(x, v, sigmas[k], sigmas[k + 1], x)
        return x
