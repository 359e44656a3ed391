"""Host side of the rotary positions and the 8-bit cache (no GPU): frequencies,
phase tables, and the calls' refusals."""
import ctypes
import math

import numpy as np
import pytest
import torch

import block_sparse_kv_bsa_b200 as bsa

INVALID, SHAPE, CAPACITY, UNSUPPORTED = 1, 2, 3, 4
A16 = 1 << 20  # an aligned, never dereferenced address


def test_frequencies_plain_linear_and_base():
    f, amp = bsa.bsa_rope_frequencies(32, base=10000.0)
    assert amp == 1.0
    np.testing.assert_allclose(f, 10000.0 ** (-np.arange(32) / 32), rtol=1e-14)
    g, _ = bsa.bsa_rope_frequencies(32, scaling="linear", factor=8.0)
    np.testing.assert_allclose(g, f / 8.0, rtol=1e-14)
    h, _ = bsa.bsa_rope_frequencies(32, scaling="base", factor=8.0)
    assert h[0] == 1.0
    np.testing.assert_allclose(h[-1], f[-1] / 8.0, rtol=1e-12)
    one, _ = bsa.bsa_rope_frequencies(1, scaling="base", factor=8.0)
    assert one[0] == 1.0


def test_frequencies_by_parts():
    n, base, factor, length, fast, slow = 64, 10000.0, 16.0, 4096.0, 32.0, 1.0
    f, amp = bsa.bsa_rope_frequencies(n, base, "by_parts", factor, length, fast, slow)
    assert amp == pytest.approx(0.1 * math.log(factor) + 1.0, rel=1e-15)
    plain = base ** (-np.arange(n) / n)
    turns = length * plain / (2 * math.pi)
    np.testing.assert_allclose(f[turns >= fast], plain[turns >= fast], rtol=1e-13)
    np.testing.assert_allclose(f[turns <= slow], plain[turns <= slow] / factor, rtol=1e-13)
    mid = (turns > slow) & (turns < fast)
    assert mid.any() and ((f[mid] < plain[mid]) & (f[mid] > plain[mid] / factor)).all()


@pytest.mark.parametrize("kw", [dict(n_pairs=0), dict(n_pairs=4, base=0.0),
                                dict(n_pairs=4, scaling="linear", factor=0.0),
                                dict(n_pairs=4, scaling="linear", factor=math.inf),
                                dict(n_pairs=4, scaling="by_parts", factor=2.0,
                                     original_length=0.0),
                                dict(n_pairs=4, scaling="by_parts", factor=2.0,
                                     original_length=10.0, beta_fast=1.0, beta_slow=1.0)])
def test_frequencies_refuse(kw):
    with pytest.raises(bsa.BsaError):
        bsa.bsa_rope_frequencies(**kw)


def test_phases_are_fractions_of_a_turn():
    freqs = np.array([1.0, 1e-4, 2 * math.pi, 0.0, -1.0, 123.456, 1e-12])
    got = bsa.bsa_rope_phases(freqs)
    turn = freqs.astype(np.longdouble) / (2 * np.arccos(np.longdouble(-1)))
    want = turn - np.floor(turn)
    have = got.astype(np.uint64).astype(np.longdouble) / np.longdouble(2.0) ** 64
    # The quotient is rounded to 64 bits; a whole turn may fall on either end.
    d = np.abs(have - want)
    assert np.minimum(d, 1 - d).max() <= 2.0 ** -56
    # Phases add: the phase of a far position is exact in 64-bit arithmetic.
    p = 1_000_003
    prod = (got.astype(object) * p) % (1 << 64)
    ref = (want * p) - np.floor(want * p)
    d = np.abs(np.array([np.longdouble(int(x)) / np.longdouble(2.0) ** 64 for x in prod]) - ref)
    assert np.minimum(d, 1 - d).max() <= 2.0 ** -34


def test_phases_refuse():
    with pytest.raises(bsa.BsaError):
        bsa.bsa_rope_phases([1.0, math.nan])
    with pytest.raises(bsa.BsaError):
        bsa.bsa_rope_phases([])


def rope(**kw):
    d = bsa.CRope(A16, (ctypes.c_int32 * 3)(16, 8, 8), 3, 0, 0, 1.0, None,
                  (ctypes.c_int32 * 3)(0, 0, 0))
    for name, v in kw.items():
        setattr(d, name, (ctypes.c_int32 * 3)(*v) if name in ("n_pairs", "origin") else v)
    return d


@pytest.mark.parametrize("kw,status", [
    (dict(phase=None), INVALID), (dict(phase=A16 + 4), INVALID), (dict(pos=A16 + 2), INVALID),
    (dict(n_axes=2), INVALID), (dict(n_axes=1), INVALID), (dict(layout=2), INVALID),
    (dict(n_pairs=(0, 0, 0)), INVALID), (dict(n_pairs=(16, -1, 8)), INVALID),
    (dict(amplitude=math.nan), INVALID), (dict(n_pairs=(32, 1, 0)), SHAPE)])
def test_rope_refuses_descriptors(kw, status):
    lib = bsa.lib()
    d = rope(**kw)
    assert lib.bsa_rope(A16, A16, 1, 2, 64, 1, 1, 1, ctypes.byref(d), None) == status
    assert lib.bsa_tokens_to_blocks_rope(A16, A16, None, 1, 2, 64, 1, 1, 1, A16, ctypes.byref(d),
                                         None, None) == status


@pytest.mark.parametrize("args,status", [
    ((None, A16, 1, 2, 64, 1, 1, 1), INVALID), ((A16, None, 1, 2, 64, 1, 1, 1), INVALID),
    ((A16 + 2, A16, 1, 2, 64, 1, 1, 1), INVALID), ((A16, A16, 0, 2, 64, 1, 1, 1), INVALID),
    ((A16, A16, 1, 2, 96, 1, 1, 1), UNSUPPORTED), ((A16, A16, 1, 2, 64, 0, 1, 1), INVALID),
    ((A16, A16, 1, 2, 64, 1 << 20, 1 << 10, 1 << 10), SHAPE),
    ((A16, A16, 1 << 20, 2, 64, 1, 1, 1), SHAPE), ((A16, A16, 1, 1 << 20, 64, 1, 1, 1), SHAPE)])
def test_rope_refuses_sizes(args, status):
    d = rope()
    assert bsa.lib().bsa_rope(*args, ctypes.byref(d), None) == status
    assert bsa.lib().bsa_rope(*args, None, None) in (status, INVALID)


def cache8(**kw):
    c = bsa.CCache8(A16, A16, A16, A16, A16, 1, 2, 64, 10, 4, None)
    for name, v in kw.items():
        setattr(c, name, v)
    return c


@pytest.mark.parametrize("kw,status", [
    (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(k_scale=None), INVALID),
    (dict(v_scale=None), INVALID), (dict(block_valid=None), INVALID), (dict(k=A16 + 8), INVALID),
    (dict(B=0), INVALID), (dict(D=32), UNSUPPORTED), (dict(n_blocks=11), INVALID),
    (dict(n_blocks=-1), INVALID)])
def test_8bit_calls_refuse_caches(kw, status):
    lib = bsa.lib()
    c = ctypes.byref(cache8(**kw))
    assert lib.bsa_kv8_append(c, A16, A16, 1, 1, 1, None, None, None, None) == status
    assert lib.bsa_kv8_attn(A16, c, 2, None, A16, A16, 1, 4, 0.1, A16, A16, None, None) == status
    assert lib.bsa_kv8_attn_decode(A16, c, 2, 1, None, None, 0, 0.1, A16, A16, A16, 1 << 30, None,
                                   None) == status


def test_8bit_append_refuses_sizes():
    lib = bsa.lib()
    c = cache8()
    call = lambda *a: lib.bsa_kv8_append(ctypes.byref(c), *a, None, None)  # noqa: E731
    assert call(None, A16, 1, 1, 1, None, None) == INVALID
    assert call(A16, A16 + 2, 1, 1, 1, None, None) == INVALID
    assert call(A16, A16, 7, 1, 128, None, None) == CAPACITY
    assert call(A16, A16, 1, 1, (1 << 14) + 1, A16, None) == UNSUPPORTED
    assert c.n_blocks == 4


def test_8bit_attention_refuses_sizes():
    lib = bsa.lib()
    c = cache8()
    at = ctypes.byref(c)
    call = lambda q, Hq, idx, n, ms, s: lib.bsa_kv8_attn(  # noqa: E731
        q, at, Hq, None, idx, A16, n, ms, s, A16, A16, None, None)
    assert call(None, 2, A16, 1, 4, 0.1) == INVALID
    assert call(A16, 2, None, 1, 4, 0.1) == INVALID
    assert call(A16, 3, A16, 1, 4, 0.1) == SHAPE
    assert call(A16, 2, A16, 0, 4, 0.1) == INVALID
    assert call(A16, 2, A16, 1, 0, 0.1) == INVALID
    assert call(A16, 2, A16, 1, 4, math.nan) == INVALID
    assert call(A16, 2, A16, 1 << 24, 4, 0.1) == SHAPE
    dec = lambda Hq, n, idx, cnt, ms, ws, size: lib.bsa_kv8_attn_decode(  # noqa: E731
        A16, at, Hq, n, idx, cnt, ms, 0.1, A16, A16, ws, size, None, None)
    assert dec(3, 1, None, None, 0, A16, 1 << 30) == SHAPE
    assert dec(2, 0, None, None, 0, A16, 1 << 30) == INVALID
    assert dec(2, 129, None, None, 0, A16, 1 << 30) == UNSUPPORTED
    assert dec(2, 1, A16, None, 4, A16, 1 << 30) == INVALID
    assert dec(2, 1, A16, A16, 0, A16, 1 << 30) == INVALID
    assert dec(2, 1, None, None, 0, A16 + 16, 1 << 30) == INVALID
    need = bsa.bsa_kv8_attn_decode_workspace_size(1, 2, 2, 64, 1, 4)
    assert need > 0
    assert dec(2, 1, None, None, 0, A16, need - 1) == CAPACITY
    assert dec(2, 1, None, None, 0, None, 1 << 30) == CAPACITY


def test_decode_workspace_covers_every_smaller_route():
    # A workspace sized for a larger n_sel is enough for fewer blocks at the
    # sizes a program meets: it is sized once and the cache grows into it.
    for B, Hq, Hh, n in ((1, 24, 24, 1), (1, 2, 2, 1), (4, 40, 8, 3), (1, 1, 1, 100)):
        sizes = [bsa.bsa_kv8_attn_decode_workspace_size(B, Hq, Hh, 128, n, s)
                 for s in list(range(0, 40)) + [113, 288, 2352, 2353, 100000]]
        assert sizes == sorted(sizes) and sizes[0] == 0
    with pytest.raises(bsa.BsaError):
        bsa.bsa_kv8_attn_decode_workspace_size(1, 3, 2, 128, 1, 10)
    with pytest.raises(bsa.BsaError):
        bsa.bsa_kv8_attn_decode_workspace_size(1, 2, 2, 96, 1, 10)


def test_rope_handle_refuses_fractions():
    # Positions and counts are whole numbers: a fraction is refused, not cut off.
    handle = bsa.Rope((4, 2, 2), device="cpu")
    for origin in ((0.5, 0, 0), (0, -1.25, 0), (0, 0, np.float32(3.9)), ("1", 0, 0)):
        with pytest.raises(TypeError):
            handle.c_struct(1, 8, None, origin)
    got = handle.c_struct(1, 8, None, (np.int64(-7), 5.0, 188))
    assert list(got.origin) == [-7, 5, 188]
    with pytest.raises(ValueError):
        handle.c_struct(1, 8, None, (0, 1 << 31, 0))
    with pytest.raises(TypeError):
        bsa.Rope((4.5, 2, 2), device="cpu")
    with pytest.raises(TypeError):
        bsa.Rope.from_frequencies([1.0, 0.5], (2.9,), device="cpu")
    with pytest.raises(TypeError):
        bsa.bsa_rope_frequencies(2.5)
    x = torch.zeros((1, 5, 2, 64), dtype=torch.bfloat16)
    for call in (bsa.bsa_rope, bsa.bsa_tokens_to_blocks_rope):
        with pytest.raises(TypeError, match="whole"):
            call(x, 2.5, 2, 1, handle)


@pytest.mark.parametrize("B,Hh,T,status", [(65536, 1, 1, SHAPE), (1, 65536, 1, SHAPE),
                                           (65535, 65535, 1, SHAPE),
                                           (40000, 4, 1 << 24, SHAPE)])
def test_rotated_calls_refuse_sizes_past_their_limits(B, Hh, T, status):
    lib, d = bsa.lib(), rope()
    at = ctypes.byref(d)
    assert lib.bsa_rope(A16, A16, B, Hh, 64, T, 1, 1, at, None) == status
    assert lib.bsa_tokens_to_blocks_rope(A16, A16, None, B, Hh, 64, T, 1, 1, None, at, None,
                                         None) == status
    c = cache8(B=B, Hh=Hh)
    assert lib.bsa_kv8_append(ctypes.byref(c), A16, A16, T, 1, 1, None, at, None, None) == status
