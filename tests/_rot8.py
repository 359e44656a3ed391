"""Plain fp64 numpy forms of the rotary positions, the 8-bit blocks and the
attention over them, for the tests; nothing here is shared with the library."""
import math

import numpy as np
import torch

BLK = 128


def f64(t):
    return t.detach().to("cpu").to(torch.float64).numpy()


def positions(T, H, W, axes, origin=(0, 0, 0), pos=None, B=1):
    """[B, N, axes] integer positions."""
    N = T * H * W
    if pos is not None:
        p = np.moveaxis(np.asarray(pos, dtype=np.int64), 0, -1)
    elif axes == 3:
        t, h, w = np.meshgrid(np.arange(T), np.arange(H), np.arange(W), indexing="ij")
        p = np.stack([t, h, w], -1).reshape(1, N, 3)
    else:
        p = np.arange(N).reshape(1, N, 1)
    return np.broadcast_to(p + np.asarray(origin[:axes], dtype=np.int64), (B, N, axes))


def rotate(x, freqs, pairs, layout, p, amp=1.0, inverse=False):
    """x [B, N, Hh, D] turned: angles from exact integer positions, reduced in
    extended precision."""
    x = np.asarray(x, dtype=np.float64)
    y = x.copy()
    P = sum(pairs)
    axis = np.repeat(np.arange(len(pairs)), pairs)
    turn = np.asarray(freqs, dtype=np.longdouble) / (2 * np.arccos(np.longdouble(-1)))
    ang = p[..., axis].astype(np.longdouble) * turn
    ang = ((ang - np.floor(ang)) * (2 * np.arccos(np.longdouble(-1)))).astype(np.float64)
    c = np.cos(ang)[:, :, None] * amp
    s = np.sin(ang)[:, :, None] * (-amp if inverse else amp)
    if layout == "half":
        a, b = x[..., :P], x[..., P:2 * P]
        y[..., :P], y[..., P:2 * P] = a * c - b * s, a * s + b * c
    else:
        a, b = x[..., 0:2 * P:2], x[..., 1:2 * P:2]
        y[..., 0:2 * P:2], y[..., 1:2 * P:2] = a * c - b * s, a * s + b * c
    return y


def to_blocks(x, perm):
    """[B, N, Hh, D] -> [B, Hh, nb, 128, D] at the slots of perm, pads zero."""
    B, N, Hh, D = x.shape
    nb = -(-N // BLK)
    out = np.zeros((B, Hh, nb * BLK, D), dtype=x.dtype)
    out[:, :, np.asarray(perm)] = np.moveaxis(x, 1, 2)
    return out.reshape(B, Hh, nb, BLK, D)


def attend(q, k, v, scale):
    """q [R, D] over all keys: (o, lse, |weights| @ |v|)."""
    s = q @ k.T * scale
    m = s.max(-1, keepdims=True)
    e = np.exp(s - m)
    l = e.sum(-1, keepdims=True)
    w = e / l
    return w @ v, (m + np.log(l))[:, 0], w @ np.abs(v)


def gather(cache, b, h, blocks):
    """Dequantised fp64 keys and values of a KVCache8's blocks, valid rows only."""
    ks, vs = [], []
    for n in blocks:
        r = int(cache.block_valid[n])
        ks.append(f64(cache.k[b, h, n, :r].float()) * float(cache.k_scale[b, h, n]))
        vs.append(f64(cache.v[b, h, n, :r].float()) * float(cache.v_scale[b, h, n]))
    return np.concatenate(ks), np.concatenate(vs)


# Tolerances, from the roundings the kernels make.
#   bf16 result: half a step, 2^-8 relative.
#   turned values: cos and sin within 2^-22 of 1 and two fp32 products: 2^-20
#   of |x| + |y|.
#   attention weights: f16, half a step 2^-11; their exponents reach 64 in
#   fp32, an error of 2^-18 each in up to four roundings: 2^-15 relative.
BF16 = 2.0 ** -8
TURN = 2.0 ** -20
WEIGHT = 2.0 ** -11 + 2.0 ** -14


def check_attn(o, lse, ref_o, ref_lse, ref_abs):
    o, lse = f64(o), f64(lse)
    assert np.isfinite(o).all() and np.isfinite(lse).all()
    tol = BF16 * np.abs(ref_o) + WEIGHT * (1 + BF16) * ref_abs + 1e-30
    assert (np.abs(o - ref_o) <= tol).all(), float((np.abs(o - ref_o) / tol).max())
    # The exponents' fp32 roundings (the query scale, the fused scales, the
    # reference), each half a step of the largest exponent, and 2^-16 for the sum.
    ltol = 2.0 ** -16 + 2.0 ** -20 * np.abs(ref_lse)
    assert (np.abs(lse - ref_lse) <= ltol).all(), float((np.abs(lse - ref_lse) / ltol).max())


def fill_cache(bsa, B, Hh, D, blocks, valid, seed, v_scale_spread=1.0, k_gain=1.0, pad=None,
               device="cuda"):
    """A KVCache8 filled with random codes and scales, ``valid`` rows per block;
    pad rows hold the code ``pad`` (None: zero)."""
    gen = torch.Generator(device=device).manual_seed(seed)
    cache = bsa.KVCache8(B, Hh, D, blocks, device=device)
    for name in ("k", "v"):
        x = torch.randn((B, Hh, blocks, BLK, D), generator=gen, device=device) * 100.0
        getattr(cache, name).copy_(x.clamp(-448, 448).to(torch.float8_e4m3fn))
    valid = torch.as_tensor(valid, dtype=torch.int32, device=device)
    cache.block_valid.copy_(valid)
    dead = (torch.arange(BLK, device=device) >= valid[:, None])[None, None, :, :, None]
    for name in ("k", "v"):
        raw = getattr(cache, name).view(torch.uint8)
        raw.masked_fill_(dead, 0 if pad is None else pad)
    cache.k_scale.copy_(torch.exp(0.3 * torch.randn((B, Hh, blocks), generator=gen,
                                                    device=device)) * 0.01 * k_gain)
    cache.v_scale.copy_(torch.exp(v_scale_spread * torch.randn(
        (B, Hh, blocks), generator=gen, device=device)) * 0.01)
    cache.n_blocks = blocks
    return cache


def sm(D):
    return 1.0 / math.sqrt(D)
