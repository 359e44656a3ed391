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
