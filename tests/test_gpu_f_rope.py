"""GPU: rotary positions on tokens, their gradient, and the rotated moves into
blocks, against the fp64 form (tests/_rot8.py)."""
import numpy as np
import pytest
import torch

import block_sparse_kv_bsa_b200 as bsa
from tests import _rot8 as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"


def tokens(B, N, Hh, D, seed, scale=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return (torch.randn((B, N, Hh, D), generator=g, device=DEV) * scale).to(torch.bfloat16)


def make(pairs, layout, amp=1.0):
    freqs = np.concatenate([10000.0 ** (-np.arange(p) / max(p, 1)) for p in pairs])
    return freqs, bsa.Rope.from_frequencies(freqs, pairs, layout=layout, amplitude=amp, device=DEV)


def close(y, want, x, amp=1.0):
    """Half a bf16 step of the result plus the fp32 error of the turn."""
    big = np.abs(x).max(-1, keepdims=True)
    tol = ref.BF16 * np.abs(want) + ref.TURN * 2 * abs(amp) * big + 1e-38
    err = np.abs(ref.f64(y) - want)
    assert (err <= tol).all(), float((err / tol).max())


# (grid, Hh, D, pairs): whole heads, parts of a head, pair counts that are no
# multiple of 8 (nor of 4), one pair, one token, odd sizes.
CASES = [((1, 1, 1), 1, 64, (32,)), ((1, 1, 1), 24, 128, (22, 21, 21)),
         ((2, 3, 5), 3, 128, (22, 21, 21)), ((257, 1, 1), 2, 64, (32,)),
         ((63, 1, 1), 5, 128, (16,)), ((33, 1, 1), 3, 64, (1,)), ((5, 7, 3), 2, 64, (3, 2, 2)),
         ((4, 9, 11), 7, 128, (40, 0, 24)), ((3, 30, 52), 4, 64, (8, 8, 8)),
         ((129, 1, 1), 2, 128, (61,)), ((31, 1, 1), 1, 128, (64,))]


@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("grid,Hh,D,pairs", CASES)
def test_rope_tokens(grid, Hh, D, pairs, layout):
    T, H, W = grid
    N = T * H * W
    x = tokens(2, N, Hh, D, 1)
    freqs, rope = make(pairs, layout, amp=1.25)
    origin = (188, -3, 7) if len(pairs) == 3 else (1 << 20, 0, 0)
    y = bsa.bsa_rope(x, T, H, W, rope, origin=origin)
    p = ref.positions(T, H, W, len(pairs), origin, B=2)
    want = ref.rotate(ref.f64(x), freqs, pairs, layout, p, 1.25)
    close(y, want, ref.f64(x), 1.25)
    # Past the turned pairs the bits pass unchanged.
    assert torch.equal(y[..., 2 * sum(pairs):], x[..., 2 * sum(pairs):])
    # In place, and twice: the same bits.
    z = x.clone()
    assert bsa.bsa_rope(z, T, H, W, rope, origin=origin, out=z) is z
    assert torch.equal(z, y)


@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("far", [0, 1 << 20, (1 << 31) - 300, -(1 << 31)])
def test_rope_given_positions(layout, far):
    B, N, Hh, D, pairs = 2, 201, 3, 64, (11, 6, 7)
    rng = np.random.default_rng(5)
    pos = (far + rng.integers(0, 299, size=(3, B, N))).astype(np.int32)
    x = tokens(B, N, Hh, D, 2)
    freqs, rope = make(pairs, layout)
    y = bsa.bsa_rope(x, N, 1, 1, rope, pos=torch.from_numpy(pos).to(DEV))
    want = ref.rotate(ref.f64(x), freqs, pairs, layout,
                      ref.positions(N, 1, 1, 3, pos=pos, B=B))
    close(y, want, ref.f64(x))


def test_rope_origin_is_added_to_given_positions_past_32_bits():
    N, D, pairs = 5, 64, (32,)
    pos = torch.full((1, 1, N), (1 << 31) - 1, dtype=torch.int32, device=DEV)
    x = tokens(1, N, 1, D, 3)
    freqs, rope = make(pairs, "half")
    y = bsa.bsa_rope(x, N, 1, 1, rope, pos=pos, origin=((1 << 31) - 1, 0, 0))
    p = np.full((1, N, 1), 2 * ((1 << 31) - 1), dtype=np.int64)
    close(y, ref.rotate(ref.f64(x), freqs, pairs, "half", p), ref.f64(x))


def test_rope_leaves_other_rows_and_special_values():
    # NaN and infinities stay in their own pair; the passing elements keep theirs.
    x = tokens(1, 40, 2, 64, 4)
    x[0, 3, 0, 5] = float("nan")
    x[0, 3, 0, 40] = float("inf")
    freqs, rope = make((16,), "interleaved")
    y = bsa.bsa_rope(x, 40, 1, 1, rope)
    bad = ~torch.isfinite(y)
    want = torch.zeros_like(bad)
    want[0, 3, 0, 4:6] = True
    want[0, 3, 0, 40] = True
    assert torch.equal(bad, want)
    assert y[0, 3, 0, 40] == float("inf")


@pytest.mark.parametrize("layout,pairs,D", [("interleaved", (9,), 64), ("half", (16,), 64),
                                            ("half", (5, 3, 2), 64), ("half", (24, 20, 20), 128)])
def test_rope_gradient(layout, pairs, D):
    T, H, W = (5, 4, 3) if len(pairs) == 3 else (60, 1, 1)
    N, amp = T * H * W, 0.75
    x, dy = tokens(1, N, 2, D, 6), tokens(1, N, 2, D, 7)
    freqs, rope = make(pairs, layout, amp)
    dx = bsa.bsa_rope(dy, T, H, W, rope, origin=(9, 0, 0), inverse=True)
    p = ref.positions(T, H, W, len(pairs), (9, 0, 0))
    # The formula: the transpose of the turn.
    close(dx, ref.rotate(ref.f64(dy), freqs, pairs, layout, p, amp, inverse=True), ref.f64(dy),
          amp)
    # Differences of the loss sum(dy * rope(x)) in fp64.
    f = lambda z: float((ref.f64(dy) * ref.rotate(z, freqs, pairs, layout, p, amp)).sum())  # noqa: E731
    z = ref.f64(x)
    for at in [(0, 0, 0, 0), (0, 17, 1, 1), (0, 59, 0, D - 1), (0, 31, 1, sum(pairs)),
               (0, 44, 1, 2 * sum(pairs) - 1)]:
        h = 2.0 ** -10
        up, dn = z.copy(), z.copy()
        up[at] += h
        dn[at] -= h
        num = (f(up) - f(dn)) / (2 * h)
        # The loss is linear: the difference errs by fp64 rounding of ~1e3 / h.
        assert abs(float(dx[at]) - num) <= ref.BF16 * abs(num) + 1e-4


MOVES = [((1, 1, 1), 1, 64, (8,)), ((2, 8, 16), 2, 64, (12, 10, 10)), ((1, 13, 17), 3, 128, (22, 21, 21)),
         ((4, 16, 32), 12, 128, (22, 21, 21)), ((3, 11, 7), 5, 64, (5, 4, 4)),
         ((1, 127, 1), 2, 128, (16, 8, 8)), ((129, 1, 1), 9, 64, (32,))]


@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("grid,Hh,D,pairs", MOVES)
def test_moves_equal_rope_then_move(grid, Hh, D, pairs, layout):
    # The fused moves give the bits of the two calls they replace.
    T, H, W = grid
    N, nb = T * H * W, bsa.n_blocks_for(T, H, W)
    x, v = tokens(2, N, Hh, D, 8), tokens(2, N, Hh, D, 9)
    _, rope = make(pairs, layout)
    y = bsa.bsa_rope(x, T, H, W, rope, origin=(12, 0, 0))
    blk, mean = bsa.bsa_tokens_to_blocks_rope(x, T, H, W, rope, origin=(12, 0, 0), want_mean=True)
    want, want_mean = bsa.bsa_tokens_to_blocks_mean(y, T, H, W)
    assert torch.equal(blk, want) and torch.equal(mean, want_mean)
    a = bsa.KVCache(2, Hh, D, 3 + nb, device=DEV, pooled_keys=True)
    b = bsa.KVCache(2, Hh, D, 3 + nb, device=DEV, pooled_keys=True)
    for c in (a, b):
        c.n_blocks = 2
        c.k.fill_(3.0)
        c.v.fill_(5.0)
        c.kmean.fill_(7.0)
    assert bsa.bsa_kv_append_rope(a, x, v, T, H, W, rope, origin=(12, 0, 0)) == 2
    bsa.bsa_kv_append(b, y, v, T, H, W)
    assert a.n_blocks == b.n_blocks == 2 + nb
    for name in ("k", "v", "kmean", "block_valid"):
        assert torch.equal(getattr(a, name), getattr(b, name)), name
    bsa.raise_on_device_error(DEV)


def test_moves_with_a_given_table_and_beyond_the_table_limit():
    N, Hh, D = 300, 2, 64
    x = tokens(1, N, Hh, D, 10)
    freqs, rope = make((32,), "half")
    perm = torch.randperm(N, generator=torch.Generator().manual_seed(3)).to(torch.int32)
    blk = bsa.bsa_tokens_to_blocks_rope(x, N, 1, 1, rope, perm=perm.to(DEV))
    y = bsa.bsa_rope(x, N, 1, 1, rope)
    assert np.array_equal(ref.f64(blk).reshape(1, Hh, 3, 128, D),
                          ref.to_blocks(ref.f64(y), perm.numpy()))
    n = (1 << 14) + 1
    x = tokens(1, n, 1, D, 11)
    blk = bsa.bsa_tokens_to_blocks_rope(x, n, 1, 1, rope)
    want = bsa.bsa_tokens_to_blocks(bsa.bsa_rope(x, n, 1, 1, rope), n, 1, 1)
    assert torch.equal(blk, want)
    with pytest.raises(bsa.BsaError):
        bsa.bsa_tokens_to_blocks_rope(x, n, 1, 1, rope, perm=torch.arange(
            n, dtype=torch.int32, device=DEV))
    bsa.raise_on_device_error(DEV)


def test_moves_report_a_table_that_is_no_permutation():
    x = tokens(1, 130, 1, 64, 12)
    _, rope = make((32,), "half")
    for value in (-1, 130, 0):
        perm = torch.arange(130, dtype=torch.int32, device=DEV)
        perm[7] = value
        bsa.bsa_tokens_to_blocks_rope(x, 130, 1, 1, rope, perm=perm)
        assert bsa.bsa_check_device_error(DEV) == (6, 4)


def test_wrappers_refuse():
    x = tokens(1, 6, 2, 64, 13)
    _, rope = make((32,), "half")
    _, wide = make((64,), "half")
    with pytest.raises(ValueError):
        bsa.bsa_rope(x, 7, 1, 1, rope)
    with pytest.raises(ValueError):
        bsa.bsa_rope(x.transpose(1, 2), 2, 1, 1, rope)
    with pytest.raises(TypeError):
        bsa.bsa_rope(x.float(), 6, 1, 1, rope)
    with pytest.raises(TypeError):
        bsa.bsa_rope(x, 6, 1, 1, None)
    with pytest.raises(bsa.BsaError):
        bsa.bsa_rope(x, 6, 1, 1, wide)
    with pytest.raises(ValueError):
        bsa.bsa_rope(x, 6, 1, 1, rope, pos=torch.zeros((1, 6), dtype=torch.int32, device=DEV))
    with pytest.raises(ValueError):
        bsa.bsa_rope(x, 6, 1, 1, rope, origin=(1 << 31, 0, 0))
    with pytest.raises(ValueError):
        bsa.Rope.from_frequencies([1.0], (2,), device=DEV)
    cache = bsa.KVCache(1, 2, 64, 1, device=DEV)
    bsa.bsa_kv_append_rope(cache, x, x, 6, 1, 1, rope)
    with pytest.raises(bsa.BsaError):
        bsa.bsa_kv_append_rope(cache, x, x, 6, 1, 1, rope)
    assert cache.n_blocks == 1


def test_offsets_past_32_bits():
    # Tensors of more than 2^31 elements: the last tokens, batch entries and blocks
    # give the bits of a call on those alone.
    g = torch.Generator(device=DEV).manual_seed(61)
    _, rope = make((64,), "half")
    N, Hh, D, last = (1 << 20) + 5, 17, 128, 6
    x = torch.randn((1, N, Hh, D), generator=g, device=DEV, dtype=torch.bfloat16)
    part = x[:, -last:].contiguous()
    want = bsa.bsa_rope(part, last, 1, 1, rope, origin=(N - last, 0, 0))
    bsa.bsa_rope(x, N, 1, 1, rope, out=x)
    assert torch.equal(x[:, -last:], want)
    del x
    _, rope = make((22, 21, 21), "interleaved")
    B, T, H, W, Hh = 9, 8, 32, 64, 120
    x = torch.randn((B, T * H * W, Hh, D), generator=g, device=DEV, dtype=torch.bfloat16)
    blk = bsa.bsa_tokens_to_blocks_rope(x, T, H, W, rope)
    part = bsa.bsa_tokens_to_blocks_rope(x[B - 1:], T, H, W, rope)
    assert torch.equal(blk[B - 1:], part)
    bsa.raise_on_device_error(DEV)


def test_batches_up_to_the_stated_limit():
    # 65535 batch entries: the last ones give the bits of a call on those alone.
    B, N, D, last = 65535, 3, 64, 2
    x, v = tokens(B, N, 1, D, 71), tokens(B, N, 1, D, 72)
    _, rope = make((16, 8, 8), "half")
    part, vpart = x[-last:].contiguous(), v[-last:].contiguous()
    y = bsa.bsa_rope(x, 1, 1, N, rope, origin=(5, 0, 0))
    assert torch.equal(y[-last:], bsa.bsa_rope(part, 1, 1, N, rope, origin=(5, 0, 0)))
    blk, mean = bsa.bsa_tokens_to_blocks_rope(x, 1, 1, N, rope, want_mean=True)
    want = bsa.bsa_tokens_to_blocks_rope(part, 1, 1, N, rope, want_mean=True)
    assert torch.equal(blk[-last:], want[0]) and torch.equal(mean[-last:], want[1])
    del blk, mean
    for kind, append in ((bsa.KVCache, bsa.bsa_kv_append_rope), (bsa.KVCache8, bsa.bsa_kv8_append)):
        whole = kind(B, 1, D, 1, device=DEV, pooled_keys=True)
        few = kind(last, 1, D, 1, device=DEV, pooled_keys=True)
        append(whole, x, v, 1, 1, N, rope)
        append(few, part, vpart, 1, 1, N, rope)
        for name in ("k", "v", "kmean"):
            a, b = (getattr(c, name).view(torch.uint8) for c in (whole, few))
            assert torch.equal(a[-last:], b), name
        del whole, few
    bsa.raise_on_device_error(DEV)
