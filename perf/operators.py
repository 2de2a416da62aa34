"""Cases of the 4-bit prefix-cache operators: quantising a prefix K/V cache to
4 bits (and back), attention over it, the accumulated attention weight of its
rows, and eviction by that weight. Plain forms in elementary torch operations,
the same results in 64 bits, and the calls a user's program makes.

The cache format: groups of 32 consecutive dims of a head share a scale s, the
smallest number with a 5-bit significand for which 7 s >= max|x|, held as
bfloat16; an element is the nearest integer to x / s (ties to even), -7 .. 7,
plus 8, in 4 bits (dim 2i in the low half of a byte, 2i + 1 in the high half).
Buffer: codes [L][2][B][H][Pp][Dh/2], then scales [L][2][B][H][Pp][Dh/32],
Pp = P rounded up to 128 rows.
"""
import math

import torch

own = False

GROUP = 32
ROW_PAD = 128
LN2 = math.log(2.0)


# ---------------------------------------------------------------- the cases

def _case(name, op, dtype, B, H, Dh, P, **more):
    return {"name": name, "op": op, "dtype": dtype, "B": B, "H": H, "Dh": Dh, "P": P, **more}


def listed():
    return [
        # the prefix caches of a batch of eight mid-size requests, all eight layers, right after the extract
        _case("quantize_mid", "quantize", "bf16", 8, 16, 64, 512, L=8, N=256),
        # one full-width layer with two large reference images and a long text
        _case("quantize_large", "quantize", "bf16", 1, 32, 128, 33792, L=1, N=1),
        # one query row over a short prefix (a 1x1 target): the smallest call, latency
        _case("attention_one_row_short", "attention", "bf16", 1, 16, 64, 77, N=1, T=1, ragged=False),
        # one query row over the longest prefix: the cache has to be read once
        _case("attention_one_row_long", "attention", "bf16", 1, 32, 128, 33792, N=1, T=1, ragged=False),
        # a few rows each of four requests whose prefixes have different lengths
        _case("attention_few_rows_ragged", "attention", "bf16", 4, 32, 128, 4608, N=16, T=16, ragged=True),
        # one layer of the mid-size batched step
        _case("attention_mid", "attention", "bf16", 8, 16, 64, 512, N=256, T=256, ragged=False),
        # one layer of the full-width cached step
        _case("attention_full", "attention", "bf16", 1, 32, 128, 4608, N=4096, T=4096, ragged=False),
        # the float32 mode at the size of the parity tests (odd lengths)
        _case("attention_f32", "attention", "f32", 2, 2, 128, 198, N=300, T=300, ragged=False),
        # which prefix rows the target attends to: one layer of the mid-size batch
        _case("scores_mid", "scores", "bf16", 8, 16, 64, 512, N=256),
        # the same for one full-width layer
        _case("scores_full", "scores", "bf16", 1, 32, 128, 4608, N=4096),
        # all layers of the mid-size batch down to an odd number of rows, the text rows kept
        _case("evict_mid", "evict", "bf16", 8, 16, 64, 512, L=8, keep=333, protected=256),
        # eight full-width layers down to half the rows
        _case("evict_full", "evict", "bf16", 1, 32, 128, 4608, L=8, keep=2304, protected=512),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    most = {}
    for c in listed():
        w = work(c)
        for k in w:
            most[c["op"], k] = max(most.get((c["op"], k), 0), w[k])
    while True:
        op = rng.choice(("quantize", "attention", "attention", "scores", "evict"))
        H, Dh = rng.choice(((16, 64), (4, 64), (32, 128), (8, 128), (2, 128)))
        dtype = "f32" if rng.random() < 0.15 else "bf16"
        B, P = _log_int(rng, 1, 8), _log_int(rng, 1, 33792)
        if op == "quantize":
            c = _case("", op, dtype, B, H, Dh, P, L=_log_int(rng, 1, 32), N=_log_int(rng, 1, 4096))
        elif op == "attention":
            c = _case("", op, dtype, B, H, Dh, P, N=_log_int(rng, 1, 8192), T=_log_int(rng, 1, 8193) - 1,
                      ragged=rng.random() < 0.4)
        elif op == "scores":
            c = _case("", op, dtype, B, H, Dh, P, N=_log_int(rng, 1, 8192))
        else:
            keep = _log_int(rng, 1, P)
            c = _case("", op, dtype, B, H, Dh, P, L=_log_int(rng, 1, 32), keep=keep,
                      protected=rng.randint(0, keep))
        del c["name"]
        w, share = work(c), 0.05 if dtype == "f32" else 1.0
        scratch = B * H * c.get("N", 0) * (P + c.get("T", 0))
        if all(w[k] <= share * most[op, k] for k in w) and scratch <= 1.2e9:
            return c


def work(case):
    B, H, Dh, P = case["B"], case["H"], case["Dh"], case["P"]
    d, eb = H * Dh, 4 if case["dtype"] == "f32" else 2
    q4 = 0.5 + 2.0 / GROUP                   # bytes of an element held in 4 bits
    if case.get("ragged") and B > 1:         # lengths are drawn evenly from 0 .. P, and one of the B is 0
        P = P / 2 * (B - 1) / B
    if case["op"] == "quantize":             # rows read, cache written, and the values it stands for
        e = case["L"] * 2 * B * P * d
        return {"bytes": e * (eb + q4 + eb), "flops": 4 * e}
    if case["op"] == "attention":
        n, t = case["N"], case["T"]
        byt = B * (2 * P * d * q4 + 2 * n * d * eb + 2 * t * d * eb + 4 * n * H)
        return {"bytes": byt, "flops": 4 * B * n * (P + t) * d}
    if case["op"] == "scores":
        n = case["N"]
        return {"bytes": B * (P * d * q4 + n * d * eb + 4 * n * H + 8 * H * P), "flops": 2 * B * n * P * d}
    lbh, keep = case["L"] * B * H, case["keep"]
    return {"bytes": lbh * (4 * P + 4 * keep + 2 * keep * Dh * (2 * q4 + eb)), "flops": lbh * P}


# ---------------------------------------------------------------- inputs

def _torch_dtype(case):
    return torch.float32 if case["dtype"] == "f32" else torch.bfloat16


def _normal(gen, shape, std=1.0):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).mul_(std)


def _pad(P):
    return (P + ROW_PAD - 1) // ROW_PAD * ROW_PAD


def _random_cache4(gen, L, B, H, P, Dh):
    """Buffer, codes and scales of a quantised cache of normal K and V (unit rms, as after QK-RMSNorm)."""
    pp = _pad(P)
    rows = L * 2 * B * H * pp
    buf = torch.empty(rows * (Dh // 2) + rows * (Dh // GROUP) * 2, dtype=torch.uint8, device="cuda")
    codes = buf[: rows * (Dh // 2)].view(L, 2, B, H, pp, Dh // 2)
    scales = buf[rows * (Dh // 2):].view(torch.bfloat16).view(L, 2, B, H, pp, Dh // GROUP)
    for l in range(L):
        x = _normal(gen, (2, B, H, pp, Dh // GROUP, GROUP))
        m, e = torch.frexp(x.abs().amax(-1) / 7)
        s = torch.ldexp((m * 32).ceil(), e - 5)
        c = (torch.round(x / s[..., None]).clamp_(-7, 7) + 8).to(torch.uint8).view(2, B, H, pp, Dh // 2, 2)
        codes[l] = c[..., 0] | (c[..., 1] << 4)
        scales[l] = s.to(torch.bfloat16)
    return buf, codes, scales


def _user_config(B_, case, L):
    d = case["H"] * case["Dh"]
    return B_.qi21_config(d, case["H"], case["Dh"], L, 2 * d, 64, 256,
                          B_.QI21_DTYPE_F32 if case["dtype"] == "f32" else B_.QI21_DTYPE_BF16, 0, 1e-6, 1e-6)


def _user_cache4(B_, s, buf, P, prefix_len=None):
    c = B_.qi21_kv4_cache_init(buf, s["cfg"], s["B"], P, prefix_len)
    c.state = B_.QI21_CACHE_EXTRACTED
    return c


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    B, H, Dh, P = case["B"], case["H"], case["Dh"], case["P"]
    d, dt = H * Dh, _torch_dtype(case)
    s = dict(case)
    if case["op"] == "quantize":
        L, rows = case["L"], P + case["N"]
        s["src"] = _normal(gen, (L, 2, B, rows, d)).to(dt)      # the extracted cache, target rows included
    else:
        L = case.get("L", 1)
        s["buf"], s["codes"], s["scales"] = _random_cache4(gen, L, B, H, P, Dh)
    s["len"] = None
    if case.get("ragged"):                                      # prefixes of different lengths, one of them empty
        lens = torch.randint(0, P + 1, (B,), generator=gen, device="cuda", dtype=torch.int32)
        lens[B // 2] = 0 if B > 1 else P
        s["len"] = lens
    if case["op"] in ("attention", "scores"):
        s["q"] = _normal(gen, (B, case["N"], d), 1.5).to(dt)
    if case["op"] == "attention":
        s["k_tail"] = _normal(gen, (B, case["T"], d)).to(dt)
        s["v_tail"] = _normal(gen, (B, case["T"], d)).to(dt)
    if case["op"] == "scores":
        # log-sum-exp over the prefix and as much again over the target keys; weights of earlier steps
        k = _values(s["codes"][0, 0, :, :, :P], s["scales"][0, 0, :, :, :P])
        q = s["q"].float().view(B, -1, H, Dh).transpose(1, 2)
        lse = torch.stack([torch.logsumexp(q[:, h] @ k[:, h].transpose(1, 2) / math.sqrt(Dh), -1) for h in range(H)])
        s["lse"] = (lse + LN2).reshape(H, -1).contiguous()
        s["before"] = _normal(gen, (B, H, P)).abs()
    if case["op"] == "evict":
        # accumulated weights: a few rows take most of it; quantised so that ties occur
        s["scores"] = torch.round(_normal(gen, (L, B, H, P), 2.0).exp() * 1024) / 1024
    if own:
        from prefix_kv_cached_b200 import binding as B_
        s["lib"], s["cfg"] = B_, _user_config(B_, case, L)
        if case["op"] == "quantize":
            s["cache"] = B_.qi21_kv_cache_init(s["src"], s["cfg"], B, P, case["N"])
            s["cache"].state = B_.QI21_CACHE_EXTRACTED
            s["buf"] = torch.empty(B_.qi21_kv4_cache_bytes(s["cfg"], B, P), dtype=torch.uint8, device="cuda")
            s["cache4"] = _user_cache4(B_, s, s["buf"], P)
            s["back"] = torch.empty((L, 2, B, P + 1, d), dtype=dt, device="cuda")
            s["cache_back"] = B_.qi21_kv_cache_init(s["back"], s["cfg"], B, P, 1)
        else:
            s["cache4"] = _user_cache4(B_, s, s["buf"], P, s["len"])
        if case["op"] in ("attention", "scores"):
            n = B_.qi21_kv4_workspace_bytes(s["cfg"], B, case["N"], P, case.get("T", 0))
            s["ws"] = torch.zeros(n, dtype=torch.uint8, device="cuda")
        if case["op"] == "attention":
            s["out"] = torch.empty_like(s["q"])
            s["lse_out"] = torch.empty((H, B, case["N"]), dtype=torch.float32, device="cuda")
        if case["op"] == "scores":
            s["after"] = torch.empty_like(s["before"])
        if case["op"] == "evict":
            keep = case["keep"]
            s["kept"] = torch.empty((L, B, H, keep), dtype=torch.int32, device="cuda")
            s["buf2"] = torch.empty(B_.qi21_kv4_cache_bytes(s["cfg"], B, keep), dtype=torch.uint8, device="cuda")
            s["cache4_out"] = _user_cache4(B_, s, s["buf2"], keep)
            s["back"] = torch.empty((L, 2, B, keep + 1, d), dtype=dt, device="cuda")
            s["cache_back"] = B_.qi21_kv_cache_init(s["back"], s["cfg"], B, keep, 1)
    return s


# ---------------------------------------------------------------- the framework's calls

def _run_own(s):
    lib, cfg = s["lib"], s["cfg"]
    stream = torch.cuda.current_stream().cuda_stream
    if s["op"] == "quantize":
        lib.check("qi21_kv4_quantize", lib.qi21_kv4_quantize(cfg, s["cache"], s["cache4"], stream))
        lib.check("qi21_kv4_dequantize", lib.qi21_kv4_dequantize(cfg, s["cache4"], s["cache_back"], stream))
        return s["back"][:, :, :, : s["P"]]
    if s["op"] == "attention":
        lib.check("qi21_kv4_attention", lib.qi21_kv4_attention(
            cfg, s["cache4"], 0, s["q"], s["B"], s["N"], s["k_tail"], s["v_tail"], s["T"], s["out"], s["lse_out"],
            s["ws"], s["ws"].numel(), stream))
        return s["out"], s["lse_out"]
    if s["op"] == "scores":
        lib.check("qi21_kv4_scores", lib.qi21_kv4_scores(
            cfg, s["cache4"], 0, s["q"], s["B"], s["N"], s["lse"], s["before"], s["after"], s["ws"],
            s["ws"].numel(), stream))
        return s["after"]
    lib.check("qi21_kv4_evict", lib.qi21_kv4_evict(cfg, s["cache4"], s["scores"], s["keep"], s["protected"],
                                                   s["cache4_out"], s["kept"], stream))
    lib.check("qi21_kv4_dequantize", lib.qi21_kv4_dequantize(cfg, s["cache4_out"], s["cache_back"], stream))
    return s["kept"], s["back"][:, :, :, : s["keep"]]


# ---------------------------------------------------------------- plain forms

def _values(codes, scales):
    """The float32 values that codes and scales stand for, [..., rows, Dh]."""
    n = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).float() - 8
    return (n.unflatten(-1, (-1, GROUP)) * scales.float()[..., None]).flatten(-2)


def _plain_quantize(s):
    # 64 bits: a quotient next to the border between two integers must not move across it
    x = s["src"][:, :, :, : s["P"]].double().unflatten(-1, (-1, GROUP))
    m, e = torch.frexp(x.abs().amax(-1, keepdim=True) / 7)
    scale = torch.ldexp((m * 32).ceil(), e - 5)
    scale = torch.where(scale > 0, scale.clamp(2.0 ** -126, 2.0 ** 122), scale)
    n = torch.round(x / scale).clamp(-7, 7).nan_to_num(0.0)
    return (n * scale).flatten(-2).to(s["src"].dtype)


def _prefix_mask(s):
    """[B][1][1][P]: true on the rows of a prefix's own length."""
    rows = torch.arange(s["P"], device="cuda")
    return (rows < s["len"][:, None])[:, None, None, :]


def _plain_attention(s):
    B, H, Dh, P, dt = s["B"], s["H"], s["Dh"], s["P"], s["q"].dtype
    heads = lambda t: t.float().view(B, -1, H, Dh).transpose(1, 2)  # noqa: E731
    k = torch.cat((_values(s["codes"][0, 0, :, :, :P], s["scales"][0, 0, :, :, :P]), heads(s["k_tail"])), 2)
    v = torch.cat((_values(s["codes"][0, 1, :, :, :P], s["scales"][0, 1, :, :, :P]), heads(s["v_tail"])), 2)
    x = heads(s["q"]) @ k.transpose(2, 3) / math.sqrt(Dh)
    if s["len"] is not None:
        x[..., :P].masked_fill_(~_prefix_mask(s), -math.inf)
    m = x.amax(-1, keepdim=True).clamp_min(-1e30)              # a row without keys: every weight 0
    p = (x - m).exp()
    del x
    total = p.sum(-1, keepdim=True)
    out = (p @ v) / total.clamp_min(1e-30)
    lse = (m + total.log()).squeeze(-1)
    return out.transpose(1, 2).reshape(B, -1, H * Dh).to(dt), lse.transpose(0, 1).contiguous()


def _plain_scores(s):
    B, H, Dh, P = s["B"], s["H"], s["Dh"], s["P"]
    k = _values(s["codes"][0, 0, :, :, :P], s["scales"][0, 0, :, :, :P])
    x = s["q"].float().view(B, -1, H, Dh).transpose(1, 2) @ k.transpose(2, 3) / math.sqrt(Dh)
    return s["before"] + (x - s["lse"].view(H, B, -1).transpose(0, 1)[..., None]).exp().sum(2)


def _plain_evict(s):
    keep, L, B, H, Dh = s["keep"], s["L"], s["B"], s["H"], s["Dh"]
    rank = s["scores"].clone()
    rank[..., : s["protected"]] = math.inf
    kept = torch.sort(rank, dim=-1, descending=True, stable=True).indices[..., :keep].sort(-1).values
    at = kept[:, None, ..., None].expand(L, 2, B, H, keep, 1)
    codes = s["codes"].gather(4, at.expand(-1, -1, -1, -1, -1, Dh // 2))
    scales = s["scales"].gather(4, at.expand(-1, -1, -1, -1, -1, Dh // GROUP))
    val = _values(codes, scales).transpose(3, 4).reshape(L, 2, B, keep, H * Dh)
    return kept.to(torch.int32), val.to(_torch_dtype(s))


def run(state):
    if own:
        return _run_own(state)
    plain = {"quantize": _plain_quantize, "attention": _plain_attention, "scores": _plain_scores,
             "evict": _plain_evict}
    return plain[state["op"]](state)


# ---------------------------------------------------------------- 64 bits, from the definitions

def _exact_values(s, which, b, h, rows, l=0):
    c = s["codes"][l, which, b, h, :rows].long()
    out = torch.empty(rows, s["Dh"], dtype=torch.float64, device="cuda")
    out[:, 0::2] = (c % 16 - 8).double()
    out[:, 1::2] = (c // 16 - 8).double()
    for g in range(s["Dh"] // GROUP):
        out[:, g * GROUP:(g + 1) * GROUP] *= s["scales"][l, which, b, h, :rows, g:g + 1].double()
    return out


def exact(case, seed):
    s = prepare(case, seed)
    B, H, Dh, P = s["B"], s["H"], s["Dh"], s["P"]
    if s["op"] == "quantize":
        # the scales to choose from, in a table: 16 .. 31 times a power of two, smallest first
        table = torch.tensor([m * 2.0 ** e for e in range(-130, 119) for m in range(16, 32)], dtype=torch.float64,
                             device="cuda")
        table = table[: int(torch.searchsorted(table, torch.tensor(2.0 ** 122, dtype=torch.float64, device="cuda"))) + 1]
        out = torch.empty((s["L"], 2, B, P, H * Dh), dtype=torch.float64, device="cuda")
        for l in range(s["L"]):
            x = s["src"][l, :, :, :P].double().reshape(-1, GROUP)
            top = x.abs().max(1).values
            scale = table[torch.searchsorted(7 * table, top).clamp_max(len(table) - 1)][:, None]
            low = (x / scale).floor()
            over = x - low * scale - (low + 1) * scale + x          # > 0: nearer to low + 1
            up = (over > 0) | ((over == 0) & (low % 2 != 0))
            out[l] = ((low + up) * scale).view(2, B, P, H * Dh)
        return out
    if s["op"] == "attention":
        n, t = s["N"], s["T"]
        out = torch.zeros((B, n, H * Dh), dtype=torch.float64, device="cuda")
        lse = torch.full((H, B, n), -math.inf, dtype=torch.float64, device="cuda")
        lens = [P] * B if s["len"] is None else s["len"].tolist()
        for b in range(B):
            for h in range(H):
                cols = slice(h * Dh, (h + 1) * Dh)
                k = torch.cat((_exact_values(s, 0, b, h, lens[b]), s["k_tail"][b, :, cols].double()))
                v = torch.cat((_exact_values(s, 1, b, h, lens[b]), s["v_tail"][b, :, cols].double()))
                if len(k):
                    x = torch.einsum("id,jd->ij", s["q"][b, :, cols].double(), k) * Dh ** -0.5
                    lse[h, b] = torch.logsumexp(x, 1)
                    out[b, :, cols] = torch.softmax(x, 1) @ v
        return out, lse
    if s["op"] == "scores":
        out = s["before"].double()
        for b in range(B):
            for h in range(H):
                q = s["q"][b, :, h * Dh:(h + 1) * Dh].double()
                x = torch.einsum("jd,id->ji", _exact_values(s, 0, b, h, P), q) * Dh ** -0.5
                out[b, h] += torch.exp(x - s["lse"].view(H, B, -1)[h, b].double()).sum(1)
        return out
    keep = s["keep"]
    score = s["scores"].double()
    score[..., : s["protected"]] = math.inf
    val = torch.empty((s["L"], 2, B, keep, H * Dh), dtype=torch.float64, device="cuda")
    for l in range(s["L"]):
        for b in range(B):
            for h in range(H):
                order = torch.argsort(-score[l, b, h], stable=True)[:keep].sort().values
                for which in range(2):
                    val[l, which, b, :, h * Dh:(h + 1) * Dh] = _exact_values(s, which, b, h, P, l)[order]
    return None, val
