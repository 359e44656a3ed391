"""GPU: the 8-bit cache - its append, the attention of query blocks and of a
few query tokens over it - against the fp64 forms (tests/_rot8.py), and a run
of them together."""
import numpy as np
import pytest
import torch

import block_sparse_kv_bsa_b200 as bsa
from tests import _rot8 as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
FLOOR = 2.0 ** -64


def tokens(B, N, Hh, D, seed, scale=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn((B, N, Hh, D), generator=g, device=DEV)
    x += torch.randn((1, 1, Hh, D), generator=g, device=DEV) * 0.5
    return (x * scale).to(torch.bfloat16)


def make(pairs, layout):
    freqs = np.concatenate([10000.0 ** (-np.arange(p) / max(p, 1)) for p in pairs])
    return freqs, bsa.Rope.from_frequencies(freqs, pairs, layout=layout, device=DEV)


# ---------------------------------------------------------------------------
# Append
# ---------------------------------------------------------------------------

def check_codes(codes, scale, r):
    """codes [B, Hh, nb, 128, D], scale [B, Hh, nb] against the fp64 rows r."""
    amax = np.maximum(np.abs(r).max((3, 4)), FLOOR)
    s = ref.f64(scale)
    # The largest row value carries the turn's fp32 error (none without a
    # turn), the division one rounding.
    assert (np.abs(s - amax / 448) <= (2.0 ** -19 + 2.0 ** -23) * amax / 448).all()
    got = ref.f64(codes.float()) * s[..., None, None]
    # Half an e4m3 step (2^-4 relative, or half the subnormal quantum 2^-9 of
    # the scale), the turn's error, and the same relative error of the scale.
    step = np.maximum(2.0 ** -4 * np.abs(r), 2.0 ** -10 * s[..., None, None])
    tol = step * (1 + 2.0 ** -16) + 2.0 ** -18 * amax[..., None, None]
    assert (np.abs(got - r) <= tol).all(), float((np.abs(got - r) / tol).max())


APPENDS = [((1, 1, 1), 1, 64, None, "half"), ((2, 8, 16), 2, 64, None, "half"),
           ((1, 13, 17), 3, 128, (22, 21, 21), "half"),
           ((1, 13, 17), 3, 128, (24, 20, 20), "half"),
           ((1, 13, 17), 3, 128, (22, 21, 21), "interleaved"),
           ((3, 11, 7), 5, 64, (3, 2, 2), "interleaved"), ((3, 11, 7), 5, 64, (4, 2, 2), "half"),
           ((129, 1, 1), 9, 64, (32,), "half"), ((127, 1, 1), 4, 128, (61,), "interleaved"),
           ((4, 16, 32), 12, 128, (64, 0, 0), "half")]


@pytest.mark.parametrize("grid,Hh,D,pairs,layout", APPENDS)
def test_append8(grid, Hh, D, pairs, layout):
    T, H, W = grid
    B, N, nb, base = 2, T * H * W, bsa.n_blocks_for(T, H, W), 2
    k, v = tokens(B, N, Hh, D, 1), tokens(B, N, Hh, D, 2, 3.0)
    k[:, :, 0] *= 2.0 ** -30  # heads of very different magnitude
    cache = bsa.KVCache8(B, Hh, D, base + nb + 1, device=DEV, pooled_keys=True)
    cache.n_blocks = base
    for t in (cache.k, cache.v):
        t.view(torch.uint8).fill_(0x31)
    for t in (cache.k_scale, cache.v_scale, cache.kmean):
        t.fill_(7.0)
    cache.block_valid.fill_(99)
    rope = freqs = None
    if pairs is not None:
        freqs, rope = make(pairs, layout)
    assert bsa.bsa_kv8_append(cache, k, v, T, H, W, rope=rope, origin=(188, 0, 0)) == base
    assert cache.n_blocks == base + nb
    bsa.raise_on_device_error(DEV)
    perm = bsa.bsa_gilbert_perm(T, H, W)
    r = ref.f64(k)
    if rope is not None:
        r = ref.rotate(r, freqs, pairs, layout,
                       ref.positions(T, H, W, len(pairs), (188, 0, 0), B=B))
    r = ref.to_blocks(r, perm)
    rv = ref.to_blocks(ref.f64(v), perm)
    new = slice(base, base + nb)
    check_codes(cache.k[:, :, new], cache.k_scale[:, :, new], r)
    check_codes(cache.v[:, :, new], cache.v_scale[:, :, new], rv)
    valid = [min(128, N - 128 * j) for j in range(nb)]
    assert cache.block_valid.tolist() == [99] * base + valid + [99]
    for j, n in enumerate(valid):
        assert not cache.k[:, :, base + j, n:].view(torch.uint8).any()
        assert not cache.v[:, :, base + j, n:].view(torch.uint8).any()
        mean = r[:, :, j, :n].mean(2)
        # 128 fp32 additions and the turn: 2^-17 of the largest row value.
        tol = 2.0 ** -17 * np.abs(r[:, :, j]).max((2, 3))[..., None]
        assert (np.abs(ref.f64(cache.kmean[:, :, base + j]) - mean) <= tol).all()
    # The blocks around are as they were.
    for i in list(range(base)) + [base + nb]:
        for t in (cache.k, cache.v):
            assert (t[:, :, i].view(torch.uint8) == 0x31).all()
        for t in (cache.k_scale, cache.v_scale, cache.kmean):
            assert (t[:, :, i] == 7.0).all()


def test_append8_special_values():
    B, N, Hh, D = 1, 256, 2, 64
    k = tokens(B, N, Hh, D, 3)
    v = tokens(B, N, Hh, D, 4)
    k[:, :128, 0] = 0.0                     # a block of zeros
    v[:, 128:, 1] = 0.0
    k[0, 200, 0, 3] = float("inf")
    k[0, 201, 0, 4] = float("-inf")
    v[0, 5, 0, 6] = float("nan")
    v[0, :128, 1] *= 1e-30                  # below the floor of the scale
    cache = bsa.KVCache8(B, Hh, D, 2, device=DEV)
    perm = torch.arange(N, dtype=torch.int32, device=DEV)
    bsa.bsa_kv8_append(cache, k, v, N, 1, 1, perm=perm)
    assert float(cache.k_scale[0, 0, 0]) == np.float32(FLOOR) / np.float32(448)
    assert not cache.k[0, 0, 0].view(torch.uint8).any()
    assert float(cache.v_scale[0, 1, 0]) == np.float32(FLOOR) / np.float32(448)
    codes = cache.k[0, 0, 1].float()
    assert codes[200 - 128, 3] == 448 and codes[201 - 128, 4] == -448
    finite = ref.f64(k[0, 128:, 0])
    finite[~np.isfinite(finite)] = 0
    assert float(cache.k_scale[0, 0, 1]) == pytest.approx(np.abs(finite).max() / 448, rel=1e-6)
    vc = cache.v[0, 0, 0].float()
    assert torch.isnan(vc[5, 6]) and int(torch.isnan(vc).sum()) == 1
    assert torch.isfinite(cache.v_scale).all()
    bsa.raise_on_device_error(DEV)


def test_append8_refusals_and_bad_tables():
    k = tokens(1, 130, 2, 64, 5)
    cache = bsa.KVCache8(1, 2, 64, 1, device=DEV)
    with pytest.raises(bsa.BsaError):
        bsa.bsa_kv8_append(cache, k, k, 130, 1, 1)
    assert cache.n_blocks == 0
    with pytest.raises(TypeError):
        bsa.bsa_kv8_append(bsa.KVCache(1, 2, 64, 4, device=DEV), k, k, 130, 1, 1)
    with pytest.raises(ValueError):
        bsa.bsa_kv8_append(cache, k[:, :100], k[:, :100], 130, 1, 1)
    cache = bsa.KVCache8(1, 2, 64, 2, device=DEV)
    perm = torch.arange(130, dtype=torch.int32, device=DEV)
    perm[3] = 130
    bsa.bsa_kv8_append(cache, k, k, 130, 1, 1, perm=perm)
    assert bsa.bsa_check_device_error(DEV) == (6, 4)


# ---------------------------------------------------------------------------
# Attention of query blocks
# ---------------------------------------------------------------------------

def random_route(B, Hh, nqb, blocks, counts, max_sel, seed):
    rng = np.random.default_rng(seed)
    idx = np.full((B, Hh, nqb, max_sel), -1, dtype=np.int32)
    cnt = np.zeros((B, Hh, nqb), dtype=np.int32)
    for i, at in enumerate(np.ndindex(B, Hh, nqb)):
        n = counts[i % len(counts)]
        idx[at][:n] = rng.permutation(blocks)[:n]
        cnt[at] = n
    return torch.from_numpy(idx).to(DEV), torch.from_numpy(cnt).to(DEV)


def check_blocks(q, cache, idx, cnt, o, lse, q_valid, scale):
    B, Hq, R, D = q.shape
    G = Hq // cache.Hh
    for b in range(B):
        for h in range(Hq):
            for j in range(R // 128):
                n = int(cnt[b, h // G, j])
                qv = 128 if q_valid is None else int(q_valid[j])
                rows = slice(j * 128, j * 128 + (qv if n else 0))
                rest = slice(rows.stop, j * 128 + 128)
                assert not o[b, h, rest].any() and torch.isneginf(lse[b, h, rest]).all()
                if rows.stop == rows.start:
                    continue
                keys, vals = ref.gather(cache, b, h // G, idx[b, h // G, j, :n].tolist())
                want = ref.attend(ref.f64(q[b, h, rows]), keys, vals, scale)
                ref.check_attn(o[b, h, rows], lse[b, h, rows], *want)


@pytest.mark.parametrize("B,Hh,G,D,nqb,blocks,counts", [
    (1, 1, 1, 64, 1, 1, [1]), (1, 2, 1, 64, 2, 5, [1, 2, 3, 5]), (2, 3, 2, 128, 3, 9, [9, 0, 4, 1]),
    (1, 2, 3, 64, 2, 7, [7, 6]), (1, 1, 5, 128, 1, 12, [12]), (2, 1, 1, 128, 4, 17, [2, 3, 16, 17]),
    (1, 1, 1, 128, 2, 40, [39, 40]), (1, 1, 2, 64, 3, 131, [131, 64, 97])])
def test_attn8(B, Hh, G, D, nqb, blocks, counts):
    rng = np.random.default_rng(7)
    valid = rng.integers(1, 129, size=blocks)
    valid[::2] = 128
    cache = ref.fill_cache(bsa, B, Hh, D, blocks, valid, 11)
    g = torch.Generator(device=DEV).manual_seed(12)
    q = (torch.randn((B, Hh * G, nqb * 128, D), generator=g, device=DEV) * 2).to(torch.bfloat16)
    idx, cnt = random_route(B, Hh, nqb, blocks, counts, max(counts) + 1, 13)
    q_valid = torch.full((nqb,), 128, dtype=torch.int32, device=DEV)
    q_valid[-1] = 77
    for qv in (None, q_valid):
        o, lse = bsa.bsa_kv8_attn(q, cache, idx, cnt, q_valid=qv)
        bsa.raise_on_device_error(DEV)
        check_blocks(q, cache, idx, cnt, o, lse, qv, ref.sm(D))


def test_attn8_negative_and_zero_scale():
    cache = ref.fill_cache(bsa, 1, 1, 64, 3, [128, 128, 50], 15)
    q = tokens(1, 1, 128, 64, 16).contiguous()
    idx = torch.arange(3, dtype=torch.int32, device=DEV).view(1, 1, 1, 3)
    cnt = torch.full((1, 1, 1), 3, dtype=torch.int32, device=DEV)
    keys, vals = ref.gather(cache, 0, 0, range(3))
    for scale in (-0.2, 0.0):
        o, lse = bsa.bsa_kv8_attn(q, cache, idx, cnt, sm_scale=scale)
        od, ld = bsa.bsa_kv8_attn_decode(q[:, :, :4].transpose(1, 2).contiguous(), cache,
                                         sm_scale=scale)
        want = ref.attend(ref.f64(q[0, 0]), keys, vals, scale)
        ref.check_attn(o[0, 0], lse[0, 0], *want)
        ref.check_attn(od[0, :, 0], ld[0, :, 0], *(x[:4] for x in want))


def test_calls_on_two_streams_at_once():
    # Two decodes and two appends in flight together, each with what it needs of
    # its own, give what they give alone.
    caches = [ref.fill_cache(bsa, 1, 4, 128, 60, [128] * 60, 17 + i) for i in range(2)]
    qs = [tokens(1, 1, 4, 128, 27 + i) for i in range(2)]
    ks = [tokens(1, 500, 4, 128, 37 + i) for i in range(2)]
    _, rope = make((64,), "half")

    def work(i):
        o, lse = bsa.bsa_kv8_attn_decode(qs[i], caches[i])
        c = bsa.KVCache8(1, 4, 128, 4, device=DEV)
        bsa.bsa_kv8_append(c, ks[i], ks[i], 500, 1, 1, rope=rope, origin=(i, 0, 0))
        return o, lse, c.k.view(torch.uint8), c.k_scale, c.v.view(torch.uint8)

    want = [work(0), work(1)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        got = []
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got.append(work(i))
        torch.cuda.synchronize()
        for x, y in zip(got[0] + got[1], want[0] + want[1]):
            assert torch.equal(x, y)
    bsa.raise_on_device_error(DEV)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("spread,gain,qs", [(4.0, 1.0, 1.0), (1.0, 8.0, 4.0), (0.5, 1e-3, 1.0),
                                            (6.0, 2.0, 30.0)])
def test_attn8_scales_and_sharp_rows(D, spread, gain, qs):
    # Value scales that differ by large factors from block to block, and
    # logits from almost flat to far apart.
    cache = ref.fill_cache(bsa, 1, 2, D, 13, [128] * 12 + [5], 21, v_scale_spread=spread,
                           k_gain=gain)
    g = torch.Generator(device=DEV).manual_seed(22)
    q = (torch.randn((1, 2, 128, D), generator=g, device=DEV) * qs).to(torch.bfloat16)
    q[0, 0, 3] = 0.0                          # a flat row
    q[0, 0, 4] *= 2.0 ** -100                 # tiny and huge query rows
    q[0, 1, 5] = (q[0, 1, 5].float() * 2.0 ** 40).to(torch.bfloat16)
    q[0, 1, 6, 7] = 3000.0                    # one element far above the others
    idx = torch.arange(13, dtype=torch.int32, device=DEV).expand(1, 2, 1, 13).contiguous()
    cnt = torch.full((1, 2, 1), 13, dtype=torch.int32, device=DEV)
    o, lse = bsa.bsa_kv8_attn(q, cache, idx, cnt)
    od, ld = bsa.bsa_kv8_attn_decode(q[:, :, :8].transpose(1, 2).contiguous(), cache)
    bsa.raise_on_device_error(DEV)
    for h in range(2):
        keys, vals = ref.gather(cache, 0, h, range(13))
        s = ref.f64(q[0, h]) @ keys.T * ref.sm(D)
        # fp32 exponents resolve 2^-24 of the logit: rows whose logits reach
        # thousands keep only that, which the tolerances below allow for.
        big = np.abs(s).max(-1)
        ro, rl, ra = ref.attend(ref.f64(q[0, h]), keys, vals, ref.sm(D))
        for got_o, got_l, n in ((o[0, h], lse[0, h], 128), (od[0, :, h], ld[0, :, h], 8)):
            soft = 2.0 ** -20 * big[:n, None]     # relative error of a weight
            tol = ref.BF16 * np.abs(ro[:n]) + (ref.WEIGHT + 2 * soft) * 1.01 * ra[:n] + 1e-30
            ok = soft[:, 0] < 0.25
            assert (np.abs(ref.f64(got_o) - ro[:n]) <= tol)[ok].all()
            assert (np.abs(ref.f64(got_l) - rl[:n]) <= 2.0 ** -16 + 2.0 ** -20 * (
                np.abs(rl[:n]) + big[:n])).all()


def test_attn8_ignores_what_pad_rows_hold():
    # NaN codes past the valid rows must not reach any result.
    valid = [128, 1, 17, 127, 64]
    q = tokens(1, 2, 128, 128, 31).contiguous()
    idx = torch.arange(5, dtype=torch.int32, device=DEV).view(1, 1, 1, 5).expand(1, 2, 1, 5)
    idx = idx.contiguous()
    cnt = torch.full((1, 2, 1), 5, dtype=torch.int32, device=DEV)
    got = []
    for pad in (None, 0x7f):
        cache = ref.fill_cache(bsa, 1, 2, 128, 5, valid, 32, pad=pad)
        got.append(bsa.bsa_kv8_attn(q, cache, idx, cnt)
                   + bsa.bsa_kv8_attn_decode(q[:, :, :3].transpose(1, 2).contiguous(), cache))
    for x, y in zip(*got):
        assert torch.isfinite(x.float()).all() and torch.equal(x, y)


def test_attn8_special_queries_stay_in_their_rows():
    cache = ref.fill_cache(bsa, 1, 1, 64, 3, [128, 128, 9], 41)
    q = tokens(1, 1, 128, 64, 42).contiguous()
    idx = torch.arange(3, dtype=torch.int32, device=DEV).view(1, 1, 1, 3)
    cnt = torch.full((1, 1, 1), 3, dtype=torch.int32, device=DEV)
    o, lse = bsa.bsa_kv8_attn(q, cache, idx, cnt)
    q2 = q.clone()
    q2[0, 0, 9, 3] = float("nan")
    q2[0, 0, 70, 5] = float("inf")
    o2, lse2 = bsa.bsa_kv8_attn(q2, cache, idx, cnt)
    keep = torch.ones(128, dtype=torch.bool, device=DEV)
    keep[[9, 70]] = False
    assert torch.equal(o[0, 0, keep], o2[0, 0, keep])
    assert torch.equal(lse[0, 0, keep], lse2[0, 0, keep])


def test_attn8_order_of_the_route_and_repeats():
    # The order of the blocks changes only roundings; running twice, nothing.
    cache = ref.fill_cache(bsa, 1, 1, 128, 9, [128] * 8 + [100], 51)
    q = tokens(1, 1, 128, 128, 52).contiguous()
    fwd = torch.arange(9, dtype=torch.int32, device=DEV).view(1, 1, 1, 9).contiguous()
    cnt = torch.full((1, 1, 1), 9, dtype=torch.int32, device=DEV)
    a = bsa.bsa_kv8_attn(q, cache, fwd, cnt)
    b = bsa.bsa_kv8_attn(q, cache, fwd.flip(-1).contiguous(), cnt)
    c = bsa.bsa_kv8_attn(q, cache, fwd, cnt)
    keys, vals = ref.gather(cache, 0, 0, range(9))
    want = ref.attend(ref.f64(q[0, 0]), keys, vals, ref.sm(128))
    for o, lse in (a, b):
        ref.check_attn(o[0, 0], lse[0, 0], *want)
    assert torch.equal(a[0], c[0]) and torch.equal(a[1], c[1])


def test_attn8_gives_the_same_bits_every_time():
    # 640 query blocks over several waves of CTAs, 60 times: a tile read
    # before it is whole, or overwritten while it is read, shows as a changed bit.
    B, Hh, D, nqb, blocks, n = 1, 16, 128, 40, 200, 25
    cache = ref.fill_cache(bsa, B, Hh, D, blocks, [128] * 199 + [31], 55)
    g = torch.Generator(device=DEV).manual_seed(56)
    q = (torch.randn((B, Hh, nqb * 128, D), generator=g, device=DEV) * 3).to(torch.bfloat16)
    idx, cnt = random_route(B, Hh, nqb, blocks, [n], n, 57)
    want = None
    for _ in range(60):
        got = bsa.bsa_kv8_attn(q, cache, idx, cnt)
        if want is None:
            want = got
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    for n_tok in (1, 12):
        qt = q[:, :, :n_tok].transpose(1, 2).contiguous()
        want = bsa.bsa_kv8_attn_decode(qt, cache)
        for _ in range(30):
            got = bsa.bsa_kv8_attn_decode(qt, cache)
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("what,code", [("index", 1), ("count", 2), ("valid", 3), ("scale", 6),
                                       ("nan", 6)])
def test_attn8_reports_what_only_the_device_sees(what, code):
    cache = ref.fill_cache(bsa, 1, 1, 64, 4, [128] * 4, 61)
    q = tokens(1, 1, 128, 64, 62).contiguous()
    idx = torch.arange(4, dtype=torch.int32, device=DEV).view(1, 1, 1, 4).contiguous()
    cnt = torch.full((1, 1, 1), 4, dtype=torch.int32, device=DEV)
    if what == "index":
        idx[0, 0, 0, 2] = 4
    elif what == "count":
        cnt[0, 0, 0] = 5
    elif what == "valid":
        cache.block_valid[1] = 129
    elif what == "scale":
        cache.k_scale[0, 0, 3] = 0.0
    else:
        cache.v_scale[0, 0, 3] = float("nan")
    o, lse = bsa.bsa_kv8_attn(q, cache, idx, cnt)
    assert bsa.bsa_check_device_error(DEV) == (6, code)
    assert torch.isfinite(o.float()).all() and torch.isfinite(lse).all()
    qt = q[:, :, :2].transpose(1, 2).contiguous()
    bsa.bsa_kv8_attn_decode(qt, cache, idx[:, :, 0].contiguous(), cnt[:, :, 0].contiguous())
    assert bsa.bsa_check_device_error(DEV) == (6, code)


# ---------------------------------------------------------------------------
# A few query tokens
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("B,Hh,G,D,n_tok,blocks,tail", [
    (1, 1, 1, 64, 1, 1, 1), (1, 2, 1, 64, 1, 10, 128), (2, 3, 4, 128, 1, 33, 77),
    (1, 2, 5, 128, 3, 9, 15), (1, 1, 8, 64, 16, 20, 128), (3, 1, 1, 128, 1, 300, 31),
    (1, 2, 1, 64, 17, 5, 16), (1, 40, 1, 128, 2, 18, 17), (1, 1, 8, 128, 1, 150, 100),
    (1, 2, 8, 64, 1, 4, 1), (1, 1, 16, 128, 1, 3, 127), (2, 1, 9, 128, 1, 30, 2),
    (2, 90, 1, 64, 1, 41, 65), (7, 90, 2, 64, 1, 33, 128)])
def test_decode8(B, Hh, G, D, n_tok, blocks, tail):
    valid = [128] * blocks
    valid[-1] = tail
    cache = ref.fill_cache(bsa, B, Hh, D, blocks, valid, 71)
    g = torch.Generator(device=DEV).manual_seed(72)
    q = (torch.randn((B, n_tok, Hh * G, D), generator=g, device=DEV) * 2).to(torch.bfloat16)
    rng = np.random.default_rng(73)
    n = min(blocks, 7)
    idx = np.stack([rng.permutation(blocks)[:n] for _ in range(B * Hh)]).reshape(B, Hh, n)
    cnt = rng.integers(0, n + 1, size=(B, Hh)).astype(np.int32)
    cnt[0, 0] = n
    idx_t = torch.from_numpy(idx.astype(np.int32)).to(DEV)
    cnt_t = torch.from_numpy(cnt).to(DEV)
    whole = bsa.bsa_kv8_attn_decode(q, cache)
    routed = bsa.bsa_kv8_attn_decode(q, cache, idx_t, cnt_t)
    bsa.raise_on_device_error(DEV)
    for (o, lse), lists in ((whole, None), (routed, (idx, cnt))):
        for b in range(B):
            for h in range(Hh):
                sel = range(blocks) if lists is None else idx[b, h, :cnt[b, h]]
                at = (b, slice(None), slice(h * G, h * G + G))
                if len(sel) == 0:
                    assert not o[at].any() and torch.isneginf(lse[at]).all()
                    continue
                keys, vals = ref.gather(cache, b, h, sel)
                qf = ref.f64(q[at]).reshape(-1, D)
                want = ref.attend(qf, keys, vals, ref.sm(D))
                ref.check_attn(o[at].reshape(-1, D), lse[at].reshape(-1), *want)


def test_decode8_empty_cache_and_refusals():
    cache = bsa.KVCache8(1, 2, 64, 4, device=DEV)
    q = tokens(1, 1, 4, 64, 81)
    o, lse = bsa.bsa_kv8_attn_decode(q, cache)
    assert not o.any() and torch.isneginf(lse).all()
    with pytest.raises(ValueError):
        bsa.bsa_kv8_attn_decode(tokens(1, 1, 3, 64, 82), cache)
    with pytest.raises(bsa.BsaError):
        bsa.bsa_kv8_attn_decode(tokens(1, 65, 4, 64, 83), cache)
    cache.n_blocks = 4
    cache.block_valid.fill_(128)
    with pytest.raises(bsa.BsaError):
        bsa.bsa_kv8_attn_decode(q, cache, workspace=torch.empty(256, dtype=torch.uint8,
                                                                device=DEV)[:0])
    with pytest.raises(ValueError):
        bsa.bsa_kv8_attn_decode(q, cache, idx=torch.zeros((1, 2, 1), dtype=torch.int32,
                                                          device=DEV))


def test_decode8_equals_the_block_form():
    # The same queries through both forms, each within its tolerance of fp64.
    cache = ref.fill_cache(bsa, 1, 2, 128, 21, [128] * 20 + [40], 91)
    q = tokens(1, 5, 6, 128, 92)
    od, ld = bsa.bsa_kv8_attn_decode(q, cache)
    q_blk = torch.zeros((1, 6, 128, 128), dtype=torch.bfloat16, device=DEV)
    q_blk[:, :, :5] = q.transpose(1, 2)
    idx = torch.arange(21, dtype=torch.int32, device=DEV).expand(1, 2, 1, 21).contiguous()
    cnt = torch.full((1, 2, 1), 21, dtype=torch.int32, device=DEV)
    o, lse = bsa.bsa_kv8_attn(q_blk, cache, idx, cnt,
                              q_valid=torch.tensor([5], dtype=torch.int32, device=DEV))
    for h in range(6):
        keys, vals = ref.gather(cache, 0, h // 3, range(21))
        want = ref.attend(ref.f64(q[0, :, h]), keys, vals, ref.sm(128))
        ref.check_attn(od[0, :, h], ld[0, :, h], *want)
        ref.check_attn(o[0, h, :5], lse[0, h, :5], *want)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n_tok,blocks", [(3, 1), (3, 40), (9, 40)])
def test_decode8_special_queries_stay_in_their_rows(D, n_tok, blocks):
    # A softmax over logits that are NaN or infinite has no value: NaN, as in the
    # block form, and nothing of it in the rows beside it.
    cache = ref.fill_cache(bsa, 1, 1, D, blocks, [128] * (blocks - 1) + [50], 95)
    q = tokens(1, n_tok, 2, D, 96)
    o, lse = bsa.bsa_kv8_attn_decode(q, cache)
    q2 = q.clone()
    q2[0, 0, 1, 3] = float("nan")
    q2[0, 1, 0, 7] = float("-inf")
    q2[0, 2] = float("inf")
    o2, lse2 = bsa.bsa_kv8_attn_decode(q2, cache)
    odd = torch.zeros((n_tok, 2), dtype=torch.bool, device=DEV)
    odd[0, 1] = odd[1, 0] = odd[2, 0] = odd[2, 1] = True
    assert torch.equal(o[0][~odd], o2[0][~odd]) and torch.equal(lse[0][~odd], lse2[0][~odd])
    assert torch.isnan(o2[0][odd]).all() and torch.isnan(lse2[0][odd]).all()
    q_blk = torch.zeros((1, 2, 128, D), dtype=torch.bfloat16, device=DEV)
    q_blk[:, :, :n_tok] = q2.transpose(1, 2)
    idx = torch.arange(blocks, dtype=torch.int32, device=DEV).view(1, 1, 1, blocks)
    cnt = torch.full((1, 1, 1), blocks, dtype=torch.int32, device=DEV)
    ob, lb = bsa.bsa_kv8_attn(q_blk, cache, idx, cnt)
    odd = odd.T
    assert torch.isnan(ob[0, :, :n_tok][odd]).all() and torch.isnan(lb[0, :, :n_tok][odd]).all()


# ---------------------------------------------------------------------------
# Together
# ---------------------------------------------------------------------------

def test_route_calls_take_the_8bit_cache():
    # They read the pooled keys alone: the same routes as from a bf16 cache with
    # the same pooled keys.  The calls that would read bf16 keys refuse it.
    B, Hh, D, hist, own = 2, 3, 128, 70, 2
    valid = [128] * (hist + own - 1) + [77]
    c8 = ref.fill_cache(bsa, B, Hh, D, hist + own, valid, 101)
    g = torch.Generator(device=DEV).manual_seed(102)
    kmean = torch.randn((B, Hh, hist + own, D), generator=g, device=DEV)
    c8 = bsa.KVCache8.from_tensors(c8.k, c8.k_scale, c8.v, c8.v_scale, c8.block_valid, hist + own,
                                   kmean)
    c16 = bsa.KVCache(B, Hh, D, hist + own, device=DEV, pooled_keys=True)
    c16.block_valid.copy_(c8.block_valid)
    c16.kmean.copy_(kmean)
    c16.n_blocks = hist + own
    q = torch.randn((B, Hh, own * 128, D), generator=g, device=DEV).to(torch.bfloat16)
    qm = torch.randn((B, Hh, own, D), generator=g, device=DEV)
    prior = torch.rand((B, own, hist), generator=g, device=DEV)
    for call in (lambda c: bsa.bsa_route(q, c, hist, hist, own, 9, g=prior),
                 lambda c: bsa.bsa_route_qmean(qm, c, hist, hist, own, 9, g=prior),
                 lambda c: bsa.bsa_route_velox(q, c, hist, hist, own, g=prior, k_cov=9, k_unc=20),
                 lambda c: bsa.bsa_route_velox(None, c, hist, hist, own, g=prior, k_cov=9,
                                               k_unc=20, q_mean=qm)):
        (i8, n8), (i16, n16) = call(c8), call(c16)
        bsa.raise_on_device_error(DEV)
        assert torch.equal(n8, n16)
        live = torch.arange(i8.shape[-1], device=DEV) < n8[..., None]
        assert torch.equal(i8[live], i16[live])
    idx, cnt = bsa.bsa_route_qmean(qm, c8, hist, hist, own, 9)
    k = tokens(B, 256, Hh, D, 103)
    bare = bsa.KVCache8.from_tensors(c8.k, c8.k_scale, c8.v, c8.v_scale, c8.block_valid,
                                     hist + own)
    for call in (lambda: bsa.bsa_attn(q, c8, idx, cnt),
                 lambda: bsa.bsa_kv_append(c8, k, k, 1, 16, 16),
                 lambda: bsa.bsa_kv_pool_means(c8),
                 lambda: bsa.bsa_route_qmean(qm, bare, hist, hist, own, 9)):
        with pytest.raises((bsa.BsaError, ValueError, TypeError)):
            call()
    for call in (lambda: bsa.bsa_kv8_attn(q, c16, idx, cnt),
                 lambda: bsa.bsa_kv8_attn_decode(q[:, :, :1].transpose(1, 2).contiguous(), c16),
                 lambda: bsa.bsa_kv8_append(c16, k, k, 1, 16, 16)):
        with pytest.raises(TypeError):
            call()


def test_offsets_past_32_bits():
    # The last blocks of a cache of more than 2^32 bytes a tensor give the bits of
    # a small cache with the same blocks.
    Hh, D, T, H, W, big = 2, 128, 1, 16, 20, 135000
    N, nb = T * H * W, 3
    k, v = tokens(1, N, Hh, D, 111), tokens(1, N, Hh, D, 112)
    q, qd = tokens(1, 128, Hh, D, 113), tokens(1, 12, Hh, D, 114)
    q = q.transpose(1, 2).contiguous()
    _, rope = make((22, 21, 21), "half")
    got = []
    for blocks in (nb, big):
        cache = bsa.KVCache8(1, Hh, D, blocks, device=DEV, pooled_keys=True)
        first = cache.n_blocks = blocks - nb
        assert bsa.bsa_kv8_append(cache, k, v, T, H, W, rope=rope) == first
        idx = torch.arange(first, blocks, dtype=torch.int32, device=DEV).expand(1, Hh, 1, nb)
        idx = idx.contiguous()
        cnt = torch.full((1, Hh, 1), nb, dtype=torch.int32, device=DEV)
        out = bsa.bsa_kv8_attn(q, cache, idx, cnt)
        out += bsa.bsa_kv8_attn_decode(qd, cache, idx[:, :, 0].contiguous(),
                                       cnt[:, :, 0].contiguous())
        bsa.raise_on_device_error(DEV)
        got.append(out + tuple(t[:, :, first:].view(torch.uint8).clone() for t in
                               (cache.k, cache.v, cache.k_scale, cache.v_scale, cache.kmean)))
        del cache
    for x, y in zip(*got):
        assert torch.equal(x, y)
    assert torch.isfinite(got[0][0].float()).all()


def run_step(state):
    """One rollout step on the 8-bit cache: append, Q to blocks with means, route
    from the pooled keys, attention, O to tokens, then a few decode tokens."""
    T, H, W = state["grid"]
    cache, rope = state["cache"], state["rope"]
    cache.n_blocks = state["own"]
    own = bsa.bsa_kv8_append(cache, state["k"], state["v"], T, H, W, rope=rope,
                             origin=state["origin"])
    q_blk, q_mean = bsa.bsa_tokens_to_blocks_rope(state["q"], T, H, W, rope,
                                                  origin=state["origin"], want_mean=True)
    nb = bsa.n_blocks_for(T, H, W)
    idx, cnt = bsa.bsa_route_qmean(q_mean, cache, own, own, nb, 3)
    o, lse = bsa.bsa_kv8_attn(q_blk, cache, idx, cnt, q_valid=cache.block_valid[own:own + nb])
    o_tok = bsa.bsa_blocks_to_tokens(o, T, H, W)
    qd = bsa.bsa_rope(state["qd"], state["qd"].shape[1], 1, 1, state["rope1"], origin=(77, 0, 0))
    od, ld = bsa.bsa_kv8_attn_decode(qd, cache)
    return dict(q_blk=q_blk, idx=idx, cnt=cnt, o=o, lse=lse, o_tok=o_tok, qd=qd, od=od, ld=ld)


def step_state(seed=0):
    T, H, W = 2, 9, 11
    B, Hh, D, nb, chunks = 1, 3, 128, 2, 4
    cache = bsa.KVCache8(B, Hh, D, nb * chunks, device=DEV, pooled_keys=True)
    _, rope = make((22, 21, 21), "interleaved")
    _, rope1 = make((64,), "interleaved")
    N = T * H * W
    for c in range(chunks - 1):
        bsa.bsa_kv8_append(cache, tokens(B, N, Hh, D, 100 + c), tokens(B, N, Hh, D, 200 + c), T, H,
                           W, rope=rope, origin=(c * T, 0, 0))
    return dict(grid=(T, H, W), cache=cache, rope=rope, rope1=rope1, own=cache.n_blocks,
                origin=((chunks - 1) * T, 0, 0), k=tokens(B, N, Hh, D, 300 + seed),
                v=tokens(B, N, Hh, D, 400 + seed), q=tokens(B, N, Hh, D, 500 + seed),
                qd=tokens(B, 2, Hh, D, 600 + seed))


def test_a_step_on_the_8bit_cache():
    st = step_state()
    r = run_step(st)
    bsa.raise_on_device_error(DEV)
    T, H, W = st["grid"]
    cache, nb = st["cache"], 2
    qv = cache.block_valid[st["own"]:st["own"] + nb]
    # The route: top 3 of the pooled scores of the turned, unrounded keys.
    freqs = np.concatenate([10000.0 ** (-np.arange(p) / p) for p in (22, 21, 21)])
    perm = bsa.bsa_gilbert_perm(T, H, W)
    means = []
    for c in range(3):
        k = ref.rotate(ref.f64(tokens(1, T * H * W, 3, 128, 100 + c)), freqs, (22, 21, 21),
                       "interleaved", ref.positions(T, H, W, 3, (c * T, 0, 0)))
        kb = ref.to_blocks(k, perm)
        means += [kb[0, :, j, :n].mean(1) for j, n in enumerate(qv.tolist())]
    means = np.stack(means, 1)                                   # [Hh, 6, D]
    q = ref.f64(r["q_blk"]).reshape(1, 3, nb, 128, 128)
    for h in range(3):
        for j in range(nb):
            s = means[h] @ q[0, h, j, :int(qv[j])].mean(0) * ref.sm(128)
            got = r["idx"][0, h, j, :3].tolist()
            worst = min(s[got])
            others = [s[n] for n in range(6) if n not in got]
            assert worst >= max(others) - 1e-4 * np.abs(s).max()
            assert r["idx"][0, h, j, 3:5].tolist() == [6, 7] and int(r["cnt"][0, h, j]) == 5
    check_blocks(r["q_blk"], cache, r["idx"], r["cnt"], r["o"], r["lse"], qv, ref.sm(128))
    assert torch.equal(r["o_tok"], bsa.bsa_blocks_to_tokens(r["o"], T, H, W))
    for h in range(3):
        keys, vals = ref.gather(cache, 0, h, range(8))
        want = ref.attend(ref.f64(r["qd"][0, :, h]), keys, vals, ref.sm(128))
        ref.check_attn(r["od"][0, :, h], r["ld"][0, :, h], *want)


def test_a_step_captured_and_on_another_stream():
    st = step_state()
    want = {n: t.clone() for n, t in run_step(st).items()}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = run_step(st)
        graph = torch.cuda.CUDAGraph()
        side.synchronize()
        with torch.cuda.graph(graph, stream=side):
            held = run_step(st)
    torch.cuda.synchronize()
    for n, t in want.items():
        assert torch.equal(t, got[n]), n
    # Replayed on other inputs: the eager results of those inputs.
    other = step_state(seed=1)
    for n in ("k", "v", "q", "qd"):
        st[n].copy_(other[n])
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    for n, t in run_step(other).items():
        assert torch.equal(t, held[n]), n
    bsa.raise_on_device_error(DEV)
