"""GPU: the 8-bit cache at the edges of what its calls accept - logits far from
zero, scales at their bounds, query elements far below their row's largest -
against the fp64 forms (tests/_rot8.py) or values known by construction."""
import numpy as np
import pytest
import torch

import block_sparse_kv_bsa_b200 as bsa
from tests import _rot8 as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
LN2 = 0.6931471805599453


def codes(x):
    """Values that e4m3 holds exactly, as codes."""
    c = x.to(torch.float8_e4m3fn)
    assert torch.equal(c.float(), x.float())
    return c


def both_forms(q, cache, n_tok, **kw):
    """Each of the two attentions over every block in use: O and LSE [B, Hq, rows(, D)]."""
    B, Hq, R, D = q.shape
    n = cache.n_blocks
    idx = torch.arange(n, dtype=torch.int32, device=DEV).expand(B, cache.Hh, R // 128, n)
    cnt = torch.full((B, cache.Hh, R // 128), n, dtype=torch.int32, device=DEV)
    out = [bsa.bsa_kv8_attn(q, cache, idx.contiguous(), cnt, **kw)]
    for k in n_tok:
        o, lse = bsa.bsa_kv8_attn_decode(q[:, :, :k].transpose(1, 2).contiguous(), cache, **kw)
        out.append((o.transpose(1, 2), lse.transpose(1, 2)))
    bsa.raise_on_device_error(DEV)
    return out


@pytest.mark.parametrize("D", [64, 128])
def test_far_logits_keep_weights_finite(D):
    # Logits (in log2 units) of 2^22 to 2^28 whose block maxima lie a few steps
    # of fp32 apart, in every order, so that a maximum 16 above the running
    # reference comes up hundreds of times.  All values are 1: whatever the
    # weights are, O is 1.
    bases, blocks = [2.0 ** e for e in range(22, 29)], 24
    Hh = len(bases)
    cache = bsa.KVCache8(1, Hh, D, blocks, device=DEV)
    k = torch.zeros((1, Hh, blocks, 128, D), device=DEV)
    k[..., 0] = 256.0
    step = np.random.default_rng(3).integers(0, 17, size=blocks)
    k[..., 1] = torch.from_numpy(step).to(DEV).float().view(1, 1, blocks, 1)
    cache.k.copy_(codes(k))
    cache.v.copy_(codes(torch.ones_like(k)))
    cache.block_valid.fill_(128)
    cache.n_blocks = blocks
    q = torch.zeros((1, Hh, 128, D), device=DEV)
    for h, base in enumerate(bases):
        q[0, h, :, 0] = base / 256.0
    q[..., 1] = 4.0 * (1 + torch.arange(128, device=DEV) % 16)
    q = q.to(torch.bfloat16)
    for o, lse in both_forms(q, cache, (1, 8, 16, 40), sm_scale=LN2):
        assert torch.isfinite(o.float()).all() and torch.isfinite(lse).all()
        # Each weight is rounded to f16, the sum that divides them is not.
        assert (np.abs(ref.f64(o) - 1) <= ref.BF16 + ref.WEIGHT * (1 + ref.BF16)).all()
        want = np.asarray(bases)[None, :, None] * LN2
        # Up to 4 * 16 * 16 above the base, the sum of the weights, and fp32 steps.
        err = ref.f64(lse) - want
        assert (err >= -2.0 ** -20 * want).all() and (err <= 1024 + 2.0 ** -20 * want).all()


def test_huge_and_tiny_query_rows_stay_finite():
    # The rows whose logits fp32 cannot resolve: no accuracy is asked of them, but
    # O is still an average of the values.
    for spread, gain, qs in [(4.0, 1.0, 1.0), (1.0, 8.0, 4.0), (6.0, 2.0, 30.0)]:
        cache = ref.fill_cache(bsa, 1, 2, 128, 13, [128] * 12 + [5], 21, v_scale_spread=spread,
                               k_gain=gain)
        g = torch.Generator(device=DEV).manual_seed(22)
        q = (torch.randn((1, 2, 128, 128), generator=g, device=DEV) * qs).to(torch.bfloat16)
        scale = 2.0 ** (torch.arange(128, device=DEV) % 48).float()
        q = (q.float() * scale[:, None]).to(torch.bfloat16)
        for o, lse in both_forms(q, cache, (8, 40)):
            assert torch.isfinite(lse).all()
            for h in range(2):
                _, vals = ref.gather(cache, 0, h, range(13))
                top = np.abs(vals).max(0) * (1 + ref.BF16 + ref.WEIGHT) + 1e-30
                assert (np.abs(ref.f64(o[0, h])) <= top).all()


# ---------------------------------------------------------------------------
# Value scales
# ---------------------------------------------------------------------------

V_SCALE_MIN = 2.0 ** -80


def flat_cache(blocks, D=64):
    """Zero keys (every weight is the same), values of one to three, scales of one."""
    cache = bsa.KVCache8(1, 1, D, blocks, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(5)
    cache.v.copy_(codes(torch.randint(1, 4, cache.v.shape, generator=g, device=DEV).float()))
    cache.block_valid.fill_(128)
    cache.n_blocks = blocks
    return cache


def test_smallest_value_scale_over_a_long_route():
    # The row sum, weights over the value scale, at the scale's bound: 301
    # thousand keys of the same weight.
    cache = flat_cache(2352)
    cache.v_scale.fill_(V_SCALE_MIN)
    vals = ref.f64(cache.v[0, 0].float()).reshape(-1, 64) * V_SCALE_MIN
    q = torch.ones((1, 1, 128, 64), dtype=torch.bfloat16, device=DEV)
    for o, lse in both_forms(q, cache, (1, 12)):
        assert (np.abs(ref.f64(lse) - np.log(2352 * 128)) <= 2.0 ** -16 + 2.0 ** -20 * 13).all()
        want = vals.mean(0)
        # The weights are equal powers of two: only the result is rounded, and the
        # fp32 sums of 301 thousand terms.
        assert (np.abs(ref.f64(o) - want) <= (ref.BF16 + 2.0 ** -9) * want).all()


@pytest.mark.parametrize("scale", [2.0 ** -81, 2.0 ** -105, 1e-45, 0.0, -1.0, float("inf")])
def test_value_scales_outside_their_bounds_are_reported(scale):
    # They count as 1, whatever they are.
    cache = flat_cache(40)
    q = torch.ones((1, 1, 128, 64), dtype=torch.bfloat16, device=DEV)
    want = both_forms(q, cache, (1,))
    cache.v_scale[0, 0, 7] = scale
    idx = torch.arange(40, dtype=torch.int32, device=DEV).view(1, 1, 1, 40)
    cnt = torch.full((1, 1, 1), 40, dtype=torch.int32, device=DEV)
    got = bsa.bsa_kv8_attn(q, cache, idx, cnt)
    assert bsa.bsa_check_device_error(DEV) == (6, 6)
    assert torch.equal(got[0], want[0][0]) and torch.equal(got[1], want[0][1])
    got = bsa.bsa_kv8_attn_decode(q[:, :, :1].transpose(1, 2).contiguous(), cache)
    assert bsa.bsa_check_device_error(DEV) == (6, 6)
    assert torch.equal(got[0], want[1][0].transpose(1, 2))
    # A key scale has no such bound, as long as it is positive and finite.
    cache.v_scale.fill_(1.0)
    cache.k_scale.fill_(scale if 0.0 < scale < float("inf") else 2.0 ** -126)
    for x, y in zip(both_forms(q, cache, (1,)), want):
        assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])


@pytest.mark.parametrize("spread", [0, 10, 20, 21, 30, 40, 64, 100])
@pytest.mark.parametrize("big_first", [False, True])
def test_value_scales_far_apart(spread, big_first):
    # Blocks whose values are 2^spread times those of the others, with weights
    # alike; in half of the columns the large blocks' values are zero, so the small
    # ones' are seen there.
    blocks, low = 6, V_SCALE_MIN if spread == 100 else 2.0 ** -9
    cache = ref.fill_cache(bsa, 1, 1, 64, blocks, [128, 128, 50, 128, 128, 9], 31, k_gain=0.5)
    big = torch.arange(blocks, device=DEV) % 2 == (0 if big_first else 1)
    cache.v_scale.copy_(torch.where(big, low * 2.0 ** spread, low).view(1, 1, blocks))
    cache.v.view(torch.uint8)[:, :, big, :, 32:] = 0
    g = torch.Generator(device=DEV).manual_seed(32)
    q = torch.randn((1, 1, 128, 64), generator=g, device=DEV).to(torch.bfloat16)
    keys, vals = ref.gather(cache, 0, 0, range(blocks))
    s = ref.f64(q[0, 0]) @ keys.T * ref.sm(64)
    w = np.exp(s - s.max(-1, keepdims=True))
    w /= w.sum(-1, keepdims=True)
    v = np.concatenate([np.full(n, float(cache.v_scale[0, 0, j]))
                        for j, n in enumerate(cache.block_valid.tolist())])
    top = (w * v).max(-1, keepdims=True)                 # largest weight * scale of a row
    want, lse_want, ra = ref.attend(ref.f64(q[0, 0]), keys, vals, ref.sm(64))
    # A weight * scale is off by WEIGHT of itself or by 2^-32 of the row's largest,
    # which every code is multiplied with.
    flush = 2.0 ** -32 * top * np.abs(vals / v[:, None]).sum(0)
    for o, lse in both_forms(q, cache, (1, 12)):
        n = o.shape[2]
        tol = (ref.BF16 * np.abs(want) + ref.WEIGHT * (1 + ref.BF16) * ra + flush)[:n]
        assert (np.abs(ref.f64(o[0, 0]) - want[:n]) <= tol).all()
        ltol = 2.0 ** -16 + 2.0 ** -20 * (np.abs(lse_want) + spread)
        assert (np.abs(ref.f64(lse[0, 0]) - lse_want[:n]) <= ltol[:n]).all()


# ---------------------------------------------------------------------------
# Repeats
# ---------------------------------------------------------------------------

def test_attn8_repeats_its_bits_over_many_tiles():
    # 12 million tiles of long routes over a cache larger than L2: a tile read
    # before it is whole, or overwritten while it is read, shows as a changed bit
    # even where that happens once in two million tiles (six expected).
    Hh, D, nqb, blocks, n = 24, 128, 49, 2352, 113
    cache = ref.fill_cache(bsa, 1, Hh, D, blocks, [128] * (blocks - 1) + [96], 55)
    g = torch.Generator(device=DEV).manual_seed(56)
    q = (torch.randn((1, Hh, nqb * 128, D), generator=g, device=DEV) * 3).to(torch.bfloat16)
    idx = torch.rand((1, Hh, nqb, blocks), generator=g, device=DEV).topk(n).indices
    idx = idx.to(torch.int32).contiguous()
    cnt = torch.full((1, Hh, nqb), n, dtype=torch.int32, device=DEV)
    want = bsa.bsa_kv8_attn(q, cache, idx, cnt)
    got = [torch.empty_like(t) for t in want]
    for _ in range(91):
        bsa.bsa_kv8_attn(q, cache, idx, cnt, o=got[0], lse=got[1])
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    # The ring of the few-token form: 56 thousand tiles a call.
    for n_tok in (1, 12):
        qt = q[:, :, :n_tok].transpose(1, 2).contiguous()
        want = bsa.bsa_kv8_attn_decode(qt, cache)
        for _ in range(50):
            got = bsa.bsa_kv8_attn_decode(qt, cache)
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    bsa.raise_on_device_error(DEV)


# ---------------------------------------------------------------------------
# Query elements far below their row's largest
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("D", [64, 128])
def test_query_elements_are_exact_down_to_2_to_the_minus_13(D):
    # Row r holds 1 and 2^-e (1 + r / 128); one key of code 448 sees the latter
    # alone, so the LSE is that element as the products saw it, times 448.
    cache = bsa.KVCache8(1, 1, D, 1, device=DEV)
    k = torch.zeros((1, 1, 1, 128, D), device=DEV)
    k[..., 0, 1] = 448.0
    cache.k.copy_(codes(k))
    cache.block_valid.fill_(1)
    cache.n_blocks = 1
    mant = 1 + torch.arange(128, device=DEV).float() / 128
    for e in range(1, 18):
        q = torch.zeros((1, 1, 128, D), device=DEV)
        q[..., 0] = 1.0
        q[0, 0, :, 1] = mant * 2.0 ** -e
        forms = both_forms(q.to(torch.bfloat16), cache, (8, 128), sm_scale=2.0 ** e)
        want = 448.0 * ref.f64(mant)
        for i, (_, lse) in enumerate(forms):
            n = lse.shape[2]
            err = np.abs(ref.f64(lse[0, 0]) - want[:n])
            tol = 2.0 ** -16 + 2.0 ** -20 * want[:n]
            # Past 2^-13 the block form may be off by 2^-21 of the row's largest; the
            # few-token form holds 2^-28.
            assert (err <= tol + (448.0 * 2.0 ** (e - 21) if e > 13 and i == 0 else 0.0)).all(), e
            if e == 14 and i == 0:
                assert (err > tol).any()   # so 2^-13 is the bound, not a loose one
