"""The 4-bit prefix cache in 64 bits, for the tests: the format written from its
definition, the buffer's layout, and the operators over it."""
import math

import numpy as np
import torch

GROUP = 32
# every scale the format has, smallest first: 16 .. 31 times a power of two in [2^-126, 2^122]
SCALES = np.array([m * 2.0 ** e for e in range(-130, 118) for m in range(16, 32)] + [2.0 ** 122])


def quantise(x):
    """x [..., Dh] float64 -> (codes k + 8 uint8 [..., Dh], scales float64 [..., Dh/32])."""
    g = np.asarray(x, np.float64).reshape(*x.shape[:-1], -1, GROUP)
    a = np.abs(g).max(-1)
    s = np.where(a > 0, SCALES[np.minimum(np.searchsorted(7 * SCALES, a), len(SCALES) - 1)], 0.0)
    k = np.clip(np.rint(np.divide(g, s[..., None], out=np.zeros_like(g), where=s[..., None] > 0)), -7, 7)
    return (k + 8).astype(np.uint8).reshape(x.shape), s


def values(codes, scales):
    k = codes.astype(np.float64).reshape(*codes.shape[:-1], -1, GROUP) - 8
    return (k * scales[..., None]).reshape(codes.shape)


def pad(P):
    return -(-P // 128) * 128


def buffer_views(buf, L, B, H, P, Dh):
    """Views of a cache buffer (uint8 tensor): codes [L][2][B][H][Pp][Dh/2], scales [L][2][B][H][Pp][Dh/32]."""
    n = L * 2 * B * H * pad(P)
    codes = buf[: n * (Dh // 2)].view(L, 2, B, H, pad(P), Dh // 2)
    scales = buf[n * (Dh // 2): n * (Dh // 2) + n * (Dh // GROUP) * 2].view(torch.bfloat16)
    return codes, scales.view(L, 2, B, H, pad(P), Dh // GROUP)


def read_values(buf, L, B, H, P, Dh):
    """What a buffer holds, float64 [L][2][B][H][P][Dh]."""
    codes, scales = buffer_views(buf.cpu(), L, B, H, P, Dh)
    c = codes[..., :P, :].numpy()
    n = np.stack((c & 15, c >> 4), -1).reshape(*c.shape[:-1], Dh)
    return values(n, scales[..., :P, :].double().numpy())


def make_buffer(rng, B_, cfg, B, P, lens=None, fill=0xFF, std=1.0):
    """A device buffer with normal K and V in 4 bits; rows that do not exist hold
    `fill` bytes (0xFF: the scales there are NaN). Returns (buf, values [L][2][B][H][P][Dh])."""
    L, H, Dh = cfg.n_layers, cfg.n_heads, cfg.head_dim
    x = rng.standard_normal((L, 2, B, H, P, Dh)) * std
    k, s = quantise(x)
    buf = torch.full((B_.qi21_kv4_cache_bytes(cfg, B, P),), fill, dtype=torch.uint8)
    codes, scales = buffer_views(buf, L, B, H, P, Dh)
    packed = torch.from_numpy(k[..., 0::2] | (k[..., 1::2] << 4))
    sc = torch.from_numpy(s).to(torch.bfloat16)
    for b in range(B):
        n = P if lens is None else lens[b]
        codes[:, :, b, :, :n] = packed[:, :, b, :, :n]
        scales[:, :, b, :, :n] = sc[:, :, b, :, :n]
    return buf.cuda(), values(k, s)


def attention(q, k, v):
    """q [n][Dh], k, v [m][Dh] float64 -> out [n][Dh], sum_j p_j |v_j| [n][Dh], lse [n], weights [n][m]."""
    if k.shape[0] == 0:
        z = np.zeros_like(q)
        return z, z, np.full(q.shape[0], -np.inf), np.zeros((q.shape[0], 0))
    x = q @ k.T / math.sqrt(q.shape[1])
    m = x.max(1, keepdims=True)
    e = np.exp(x - m)
    t = e.sum(1, keepdims=True)
    p = e / t
    return p @ v, p @ np.abs(v), (m + np.log(t))[:, 0], p


def evict(scores, lens, keep, protected):
    """scores [L][B][H][P] float32 -> kept int32 [L][B][H][keep], -1 behind an item's rows."""
    L, B, H, P = scores.shape
    out = np.full((L, B, H, keep), -1, np.int32)
    for l in range(L):
        for b in range(B):
            n = P if lens is None else min(max(lens[b], 0), P)
            for h in range(H):
                s = scores[l, b, h, :n].astype(np.float64)
                rank = sorted(range(n), key=lambda j: (j >= protected, bool(np.isnan(s[j])),
                                                       0.0 if np.isnan(s[j]) else -s[j], j))
                rows = sorted(rank[:keep])
                out[l, b, h, : len(rows)] = rows
    return out
