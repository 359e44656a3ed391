"""Workloads of the rotary-position and 8-bit KV cache operators.

Each case is one call as a program makes it between two steps of a rollout:
rotary positions on a chunk's tokens (or their gradient), the rotation fused
into the move to 128-token blocks, the append into a cache held in e4m3 with
one scale per block and head, and attention over that cache by a chunk of
query blocks or by a few query tokens.

`run` computes the plain form with elementary torch operations in fp32
(angles in fp64), or, where `own` is true, calls the library.  `exact` is the
same result from the definition in fp64.
"""
import math

import torch

own = False

BLK = 128
E4M3_MAX = 448.0
AMAX_FLOOR = 2.0 ** -64
DEV = "cuda"


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # One token of a stream gets its positions: the smallest call, all latency.
        dict(name="rope_one_token", op="rope", B=1, T=1, H=1, W=1, Hh=24, D=128,
             pairs_t=22, pairs_h=21, pairs_w=21, layout="half", inverse=False, far=188,
             scaled=False),
        # The gradient through the positions of a long packed text sequence: one axis, part of
        # the head, scaled frequencies, explicit far positions.
        dict(name="rope_gradient_long", op="rope", B=1, T=40001, H=1, W=1, Hh=24, D=64,
             pairs_t=24, pairs_h=0, pairs_w=0, layout="interleaved", inverse=True, far=1 << 20,
             scaled=True),
        # A 2048-token query chunk rotated on its way to block order.
        dict(name="query_blocks", op="blocks", B=1, T=4, H=16, W=32, Hh=12, D=128,
             pairs_t=22, pairs_h=21, pairs_w=21, layout="interleaved", far=188),
        # A 7800-token chunk (61 blocks, the last one ragged) appended to the bf16 cache.
        dict(name="append_rope", op="append", B=1, T=5, H=30, W=52, Hh=24, D=128,
             pairs_t=22, pairs_h=21, pairs_w=21, layout="half", far=40, base=143),
        # The smallest chunk into the 8-bit cache.
        dict(name="append8_tiny", op="append8", B=1, T=2, H=8, W=16, Hh=2, D=64,
             pairs_t=0, pairs_h=0, pairs_w=0, layout="half", far=0, base=8, pooled=False),
        # Chunk 48 of a rollout into the 8-bit cache: rotated keys, pooled keys.
        dict(name="append8_chunk", op="append8", B=1, T=4, H=30, W=52, Hh=24, D=128,
             pairs_t=22, pairs_h=21, pairs_w=21, layout="interleaved", far=188, base=98,
             pooled=True),
        # Two query blocks over five blocks each.
        dict(name="attn8_tiny", op="attn8", B=1, T=2, H=8, W=16, Hk=2, G=1, D=64, hist=4, top_k=3),
        # The last chunk of a 48-chunk rollout: 49 query blocks, 113 of 2352 blocks each.
        dict(name="attn8_chunk48", op="attn8", B=1, T=4, H=30, W=52, Hk=24, G=1, D=128, hist=47,
             top_k=64),
        # Grouped heads: 40 query heads on 8 cache heads, batch 2.
        dict(name="attn8_grouped", op="attn8", B=2, T=4, H=32, W=32, Hk=8, G=5, D=128, hist=8,
             top_k=32),
        # One token over a ten-block cache: latency.
        dict(name="decode_tiny", op="decode", B=1, n_tok=1, Hk=2, G=1, D=64, blocks=10, top_k=0,
             tail=128),
        # One token over the whole cache of a 48-chunk rollout (301 thousand tokens).
        dict(name="decode_long", op="decode", B=1, n_tok=1, Hk=24, G=1, D=128, blocks=2352,
             top_k=0, tail=96),
        # A few tokens of four streams with grouped heads over routed blocks.
        dict(name="decode_grouped", op="decode", B=4, n_tok=3, Hk=8, G=5, D=128, blocks=288,
             top_k=64, tail=77),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _grid(rng, lo, hi):
    """A latent grid of about lo..hi tokens, odd extents among them."""
    n = _log_int(rng, lo, hi)
    T = rng.randint(1, 6)
    H = max(1, int(math.sqrt(n / T / rng.uniform(1.0, 2.5))))
    W = max(1, n // (T * H))
    while T * H * W > hi:
        W = max(1, W - 1)
        if W == 1 and T * H * W > hi:
            H -= 1
    return T, H, W


def _pairs(rng, D):
    """Pairs rotated by the (t, h, w) positions, the whole head or part of it."""
    P = rng.choice([D // 2, D // 2, D // 4, rng.randint(3, D // 2)])
    h = rng.randint(1, max(1, P // 3))
    return P - 2 * h, h, h


def draw(rng):
    op = rng.choice(["rope", "blocks", "append", "append8", "attn8", "decode"])
    D = rng.choice([64, 128, 128])
    layout = rng.choice(["half", "interleaved"])
    if op == "rope":
        Hh = rng.choice([1, 2, 5, 8, 12, 24, 40])
        limit = (40001 * 24 * 64) // (Hh * D)
        far = rng.choice([0, 188, 1 << 20])
        inverse = rng.random() < 0.5
        if rng.random() < 0.5:
            n = _log_int(rng, 1, min(limit, 65000))
            P = rng.choice([D // 2, D // 4, rng.randint(1, D // 2)])
            return dict(op=op, B=1, T=n, H=1, W=1, Hh=Hh, D=D, pairs_t=P, pairs_h=0, pairs_w=0,
                        layout=layout, inverse=inverse, far=far, scaled=rng.random() < 0.5)
        T, H, W = _grid(rng, 1, min(limit, 16384))
        t, h, w = _pairs(rng, D)
        return dict(op=op, B=1, T=T, H=H, W=W, Hh=Hh, D=D, pairs_t=t, pairs_h=h, pairs_w=w,
                    layout=layout, inverse=inverse, far=far, scaled=False)
    if op in ("blocks", "append", "append8"):
        Hh = rng.choice([1, 2, 3, 8, 12, 24, 40])
        T, H, W = _grid(rng, 100, min(16384, 7800 * 24 * 128 // (Hh * D)))
        t, h, w = _pairs(rng, D)
        case = dict(op=op, B=1, T=T, H=H, W=W, Hh=Hh, D=D, pairs_t=t, pairs_h=h, pairs_w=w,
                    layout=layout, far=rng.choice([0, 40, 188]))
        if op != "blocks":
            case["base"] = rng.choice([0, 7, 143])
        if op == "append8":
            case["pooled"] = rng.random() < 0.5
            if rng.random() < 0.3:
                case.update(pairs_t=0, pairs_h=0, pairs_w=0)
        return case
    if op == "attn8":
        Hk, G = rng.choice([(2, 1), (12, 1), (24, 1), (8, 3), (4, 5), (3, 2)])
        T, H, W = _grid(rng, 100, 6240)
        nb = -(-T * H * W // BLK)
        hist = rng.randint(1, max(1, min(47, 2300 // nb)))
        top_k = _log_int(rng, 1, 64)
        return dict(op=op, B=1, T=T, H=H, W=W, Hk=Hk, G=G, D=D, hist=hist, top_k=top_k)
    Hk, G = rng.choice([(1, 1), (2, 1), (24, 1), (8, 5), (4, 8), (8, 3)])
    B = rng.choice([1, 1, 2, 4])
    blocks = _log_int(rng, 2, max(3, 2352 * 24 * 128 // (B * Hk * D) // 2))
    blocks = min(blocks, 4000)
    return dict(op="decode", B=B, n_tok=rng.choice([1, 1, 2, 3, 5]), Hk=Hk, G=G, D=D,
                blocks=blocks, top_k=rng.choice([0, 0, max(1, blocks // 4)]),
                tail=rng.randint(1, BLK))


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _packed(case):
    """Whether the case gives every token's position: sequences on one axis."""
    return case["op"] == "rope" and case["T"] > 1 and not case["pairs_h"] and not case["pairs_w"]


def _frequencies(case):
    """Radians per position of every pair (fp64), section by section, and the amplitude."""
    out, amp = [], 1.0
    for n in (case["pairs_t"], case["pairs_h"], case["pairs_w"]):
        out += [10000.0 ** (-i / n) for i in range(n)]
    if case.get("scaled"):
        # Scaled by parts for a context 16 times the original 65536: pairs that turn often keep
        # their frequency, those that turn less than once are interpolated, with a ramp between.
        factor, length, fast, slow = 16.0, 65536.0, 32.0, 1.0
        for i, f in enumerate(out):
            keep = min(1.0, max(0.0, (length * f / (2 * math.pi) - slow) / (fast - slow)))
            out[i] = f * keep + f / factor * (1.0 - keep)
        amp = 0.1 * math.log(factor) + 1.0
    return out, amp


def _rope_handle(case, freqs, amp):
    import block_sparse_kv_bsa_b200 as bsa
    n = case["pairs_t"], case["pairs_h"], case["pairs_w"]
    pairs = n if n[1] or n[2] else n[:1]
    return bsa.Rope.from_frequencies(freqs, pairs, layout=case["layout"], amplitude=amp, device=DEV)


def _tile_perm(T, H, W):
    """Slot of every raster token when tiles of 8 x 16 cells are stored one after another."""
    i = torch.arange(T * H * W, device=DEV)
    t, h, w = i // (H * W), i // W % H, i % W
    order = (((t * (H // 8 + 1) + h // 8) * (W // 16 + 1) + w // 16) * 8 + h % 8) * 16 + w % 16
    perm = torch.empty_like(i)
    perm[order.argsort()] = i
    return perm.to(torch.int32)


def _tokens(case, heads, gen, offset=0.5):
    """Activations: N(0, 1) plus an offset per head and channel, as projections have."""
    n = case["T"] * case["H"] * case["W"]
    x = torch.randn((case["B"], n, heads, case["D"]), generator=gen, device=DEV)
    x += torch.randn((1, 1, heads, case["D"]), generator=gen, device=DEV) * offset
    return x.to(torch.bfloat16)


def _cache8(B, Hk, D, blocks, valid, gen):
    """A filled 8-bit cache: N(0, 1) plus block offsets, V of a magnitude that varies by block."""
    shape = (B, Hk, blocks, BLK, D)
    rows = torch.arange(BLK, device=DEV).view(1, 1, 1, BLK, 1) < valid.view(1, 1, -1, 1, 1)
    out = []
    for kind in ("k", "v"):
        x = torch.randn(shape, generator=gen, device=DEV)
        x += torch.randn((B, Hk, blocks, 1, D), generator=gen, device=DEV) * 0.5
        if kind == "v":
            x *= torch.exp(0.5 * torch.randn((B, Hk, blocks, 1, 1), generator=gen, device=DEV))
        x *= rows
        amax = x.abs().amax(dim=(3, 4))
        x *= (E4M3_MAX / amax)[..., None, None]
        out += [x.to(torch.float8_e4m3fn), amax / E4M3_MAX]
        del x
    return out


def _handle8(st):
    import block_sparse_kv_bsa_b200 as bsa
    return bsa.KVCache8.from_tensors(st["k8"], st["k_scale"], st["v8"], st["v_scale"],
                                     st["valid"], st["n_blocks"])


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    op, st = case["op"], dict(case=case)
    if op in ("rope", "blocks", "append", "append8"):
        B, D, Hh = case["B"], case["D"], case["Hh"]
        n = case["T"] * case["H"] * case["W"]
        freqs, st["amp"] = _frequencies(case)
        st["freqs"] = torch.tensor(freqs, dtype=torch.float64, device=DEV)
        st["x"] = _tokens(case, Hh, gen)
        if op != "rope":
            st["perm"] = _tile_perm(case["T"], case["H"], case["W"])
        if op in ("append", "append8"):
            st["v"] = _tokens(case, Hh, gen)
        if _packed(case):
            # Packed sequences: positions restart at random places, from a far origin on.
            starts = torch.rand((B, n), generator=gen, device=DEV) < 3.0 / n
            idx = torch.arange(n, device=DEV).expand(B, n)
            first = torch.where(starts, idx, 0).cummax(dim=1).values
            st["pos"] = (idx - first + case["far"]).to(torch.int32).view(1, B, n).contiguous()
        if op == "blocks":
            nb = -(-n // BLK)
            st["out"] = torch.empty((B, Hh, nb * BLK, D), dtype=torch.bfloat16, device=DEV)
        elif op == "rope":
            st["out"] = torch.empty_like(st["x"])
        else:
            nb = -(-n // BLK)
            total = case["base"] + nb
            shape = (B, Hh, total, BLK, D)
            kind = torch.bfloat16 if op == "append" else torch.float8_e4m3fn
            st["k"] = torch.zeros(shape, dtype=kind, device=DEV)
            st["cv"] = torch.zeros(shape, dtype=kind, device=DEV)
            st["valid"] = torch.full((total,), BLK, dtype=torch.int32, device=DEV)
            if op == "append8":
                st["k_scale"] = torch.ones((B, Hh, total), device=DEV)
                st["v_scale"] = torch.ones((B, Hh, total), device=DEV)
                st["kmean"] = (torch.zeros((B, Hh, total, D), device=DEV) if case["pooled"]
                               else None)
        if own:
            import block_sparse_kv_bsa_b200 as bsa
            st["rope"] = _rope_handle(case, freqs, st["amp"]) if freqs else None
            if op == "append":
                cache = bsa.KVCache(B, Hh, D, 1, device=DEV)
                cache.k, cache.v, cache.block_valid = st["k"], st["cv"], st["valid"]
                cache.max_blocks = st["k"].shape[2]
                st["cache"] = cache
            elif op == "append8":
                st["cache"] = bsa.KVCache8.from_tensors(st["k"], st["k_scale"], st["cv"],
                                                        st["v_scale"], st["valid"], case["base"],
                                                        kmean=st["kmean"])
        return st
    B, Hk, G, D = case["B"], case["Hk"], case["G"], case["D"]
    st["sm_scale"] = 1.0 / math.sqrt(D)
    if op == "attn8":
        n = case["T"] * case["H"] * case["W"]
        nb = -(-n // BLK)
        blocks = (case["hist"] + 1) * nb
        tail = n - (nb - 1) * BLK
        valid = torch.full((case["hist"] + 1, nb), BLK, dtype=torch.int32, device=DEV)
        valid[:, -1] = tail
        st["valid"] = valid.reshape(-1).contiguous()
        n_hist = blocks - nb
        # Sharper heads among flatter ones.
        sharp = torch.linspace(1.0, 3.0, Hk * G, device=DEV).view(1, -1, 1, 1)
        q = torch.randn((B, Hk * G, nb * BLK, D), generator=gen, device=DEV) * sharp
        row = torch.arange(nb * BLK, device=DEV).view(1, 1, -1, 1)
        st["q"] = (q * (row < n)).to(torch.bfloat16)
        st["q_valid"] = st["valid"][-nb:].contiguous()
        K = min(case["top_k"], n_hist)
        liked = torch.randn((B, Hk, 1, n_hist), generator=gen, device=DEV)
        score = torch.randn((B, Hk, nb, n_hist), generator=gen, device=DEV) + liked
        top = score.topk(K, dim=-1).indices.sort(dim=-1).values
        mine = torch.arange(n_hist, blocks, device=DEV).expand(B, Hk, nb, nb)
        st["idx"] = torch.cat([top, mine], dim=-1).to(torch.int32).contiguous()
        st["cnt"] = torch.full((B, Hk, nb), K + nb, dtype=torch.int32, device=DEV)
        st["o"] = torch.empty_like(st["q"])
        st["lse"] = torch.empty((B, Hk * G, nb * BLK), device=DEV)
    else:
        blocks = case["blocks"]
        st["valid"] = torch.full((blocks,), BLK, dtype=torch.int32, device=DEV)
        st["valid"][-1] = case["tail"]
        sharp = torch.linspace(1.0, 3.0, Hk * G, device=DEV).view(1, 1, -1, 1)
        q = torch.randn((B, case["n_tok"], Hk * G, D), generator=gen, device=DEV) * sharp
        st["q"] = q.to(torch.bfloat16)
        st["idx"] = st["cnt"] = None
        if case["top_k"]:
            K = min(case["top_k"], blocks)
            score = torch.randn((B, Hk, blocks), generator=gen, device=DEV)
            st["idx"] = score.topk(K, dim=-1).indices.sort(dim=-1).values.to(torch.int32)
            st["idx"] = st["idx"].contiguous()
            st["cnt"] = torch.full((B, Hk), K, dtype=torch.int32, device=DEV)
        st["o"] = torch.empty_like(st["q"])
        st["lse"] = torch.empty((B, case["n_tok"], Hk * G), device=DEV)
    st["n_blocks"] = blocks
    st["k8"], st["k_scale"], st["v8"], st["v_scale"] = _cache8(B, Hk, D, blocks, st["valid"], gen)
    if own:
        st["cache"] = _handle8(st)
        if op == "decode":
            import block_sparse_kv_bsa_b200 as bsa
            n_sel = blocks if st["idx"] is None else st["idx"].shape[-1]
            size = bsa.bsa_kv8_attn_decode_workspace_size(B, Hk * G, Hk, D, case["n_tok"], n_sel)
            st["workspace"] = torch.empty(max(size, 256), dtype=torch.uint8, device=DEV)
    return st


# ---------------------------------------------------------------------------
# Plain form
# ---------------------------------------------------------------------------

def _positions(st, dtype):
    """Position of every token for every pair: [B or 1, N, pairs]."""
    case = st["case"]
    T, H, W = case["T"], case["H"], case["W"]
    n = T * H * W
    counts = torch.tensor([case["pairs_t"], case["pairs_h"], case["pairs_w"]], device=DEV)
    if "pos" in st:
        return st["pos"][0].to(dtype)[..., None].expand(-1, -1, int(case["pairs_t"]))
    i = torch.arange(n, device=DEV)
    if case["pairs_h"] == 0 and case["pairs_w"] == 0:
        axes = torch.stack([i + case["far"], i, i], dim=-1)
    else:
        axes = torch.stack([i // (H * W) + case["far"], i // W % H, i % W], dim=-1)
    axis = torch.repeat_interleave(torch.arange(3, device=DEV), counts)
    return axes[None, :, axis].to(dtype)


def _rotate(st, x, inverse=False):
    """Rotated tokens in fp32, angles in fp64."""
    case = st["case"]
    P = st["freqs"].numel()
    x = x.float()
    if P == 0:
        return x
    angle = _positions(st, torch.float64) * st["freqs"]
    cos = (angle.cos() * st["amp"]).float()[:, :, None]
    sin = (angle.sin() * st["amp"]).float()[:, :, None]
    if inverse:
        sin = -sin
    if case["layout"] == "half":
        a, b, rest = x[..., :P], x[..., P:2 * P], x[..., 2 * P:]
        return torch.cat([a * cos - b * sin, a * sin + b * cos, rest], dim=-1)
    a, b, rest = x[..., 0:2 * P:2], x[..., 1:2 * P:2], x[..., 2 * P:]
    turned = torch.stack([a * cos - b * sin, a * sin + b * cos], dim=-1).flatten(-2)
    return torch.cat([turned, rest], dim=-1)


def _to_blocks(st, x):
    """[B, N, Hh, D] -> [B, Hh, nb, 128, D] at the slots of the table, pad rows zero."""
    B, n, Hh, D = x.shape
    nb = -(-n // BLK)
    out = x.new_zeros((B, Hh, nb * BLK, D))
    out[:, :, st["perm"].long()] = x.transpose(1, 2)
    return out.view(B, Hh, nb, BLK, D)


def _quantise(r):
    amax = r.abs().amax(dim=(3, 4)).clamp_min(AMAX_FLOOR)
    codes = (r * (E4M3_MAX / amax)[..., None, None]).to(torch.float8_e4m3fn)
    return codes, amax / E4M3_MAX


def _append_valid(case, n):
    nb = -(-n // BLK)
    valid = torch.full((nb,), BLK, dtype=torch.int32, device=DEV)
    valid[-1:] = n - (nb - 1) * BLK
    return valid


def _attend(q, k, v, live, scale):
    """q [R, D] over keys k, v [S, D] of which `live` count: o and lse."""
    s = (q @ k.transpose(-1, -2)) * scale
    s = s.masked_fill(~live, float("-inf"))
    m = s.amax(dim=-1, keepdim=True)
    p = (s - m).exp()
    total = p.sum(dim=-1, keepdim=True)
    return (p @ v) / total, (m + total.log()).squeeze(-1)


def _gather(st, b, h, sel):
    """Dequantised keys and values (fp32) of the blocks `sel` [..., n] of cache head (b, h)."""
    D = st["case"]["D"]
    shape = sel.shape[:-1] + (sel.shape[-1] * BLK, D)
    k = st["k8"][b, h].view(torch.uint8)[sel].view(torch.float8_e4m3fn).float()
    v = st["v8"][b, h].view(torch.uint8)[sel].view(torch.float8_e4m3fn).float()
    k = k * st["k_scale"][b, h][sel][..., None, None]
    v = v * st["v_scale"][b, h][sel][..., None, None]
    live = torch.arange(BLK, device=DEV) < st["valid"][sel][..., None]
    return k.reshape(shape), v.reshape(shape), live.flatten(-2)


def _plain_attn8(st):
    case, G = st["case"], st["case"]["G"]
    B, Hq, R, D = st["q"].shape
    nb = R // BLK
    o, lse = st["o"], st["lse"]
    for b in range(B):
        for h in range(case["Hk"]):
            k, v, live = _gather(st, b, h, st["idx"][b, h].long())
            mine = slice(h * G, h * G + G)
            q = st["q"][b, mine].float().view(G, nb, BLK, D)
            x, l = _attend(q, k, v, live[:, None], st["sm_scale"])
            dead = torch.arange(BLK, device=DEV) >= st["q_valid"][:, None]
            o[b, mine] = x.masked_fill(dead[..., None], 0.0).reshape(G, R, D)
            lse[b, mine] = l.masked_fill(dead, float("-inf")).reshape(G, R)
    return {"o": o, "lse": lse}


def _plain_decode(st):
    case, G = st["case"], st["case"]["G"]
    o, lse = st["o"], st["lse"]
    for b in range(case["B"]):
        for h in range(case["Hk"]):
            sel = (torch.arange(case["blocks"], device=DEV) if st["idx"] is None
                   else st["idx"][b, h].long())
            k, v, live = _gather(st, b, h, sel)
            q = st["q"][b, :, h * G:h * G + G].float()
            o[b, :, h * G:h * G + G], lse[b, :, h * G:h * G + G] = _attend(
                q, k, v, live, st["sm_scale"])
    return {"o": o, "lse": lse}


def _plain(st):
    case, op = st["case"], st["case"]["op"]
    if op == "rope":
        st["out"].copy_(_rotate(st, st["x"], case["inverse"]))
        return {"y": st["out"]}
    if op == "blocks":
        st["out"].copy_(_to_blocks(st, _rotate(st, st["x"])).view_as(st["out"]))
        return {"blocks": st["out"]}
    if op == "append":
        base = case["base"]
        st["k"][:, :, base:] = _to_blocks(st, _rotate(st, st["x"])).to(torch.bfloat16)
        st["cv"][:, :, base:] = _to_blocks(st, st["v"])
        st["valid"][base:] = _append_valid(case, st["x"].shape[1])
        return {"k": st["k"][:, :, base:], "v": st["cv"][:, :, base:], "valid": st["valid"]}
    if op == "append8":
        base = case["base"]
        valid = _append_valid(case, st["x"].shape[1])
        r = _to_blocks(st, _rotate(st, st["x"]))
        st["k"][:, :, base:], st["k_scale"][:, :, base:] = _quantise(r)
        if st["kmean"] is not None:
            st["kmean"][:, :, base:] = r.sum(dim=3) / valid.view(1, 1, -1, 1)
        v = _to_blocks(st, st["v"]).float()
        st["cv"][:, :, base:], st["v_scale"][:, :, base:] = _quantise(v)
        st["valid"][base:] = valid
        return _append8_outputs(st)
    if op == "attn8":
        return _plain_attn8(st)
    return _plain_decode(st)


def _append8_outputs(st):
    base = st["case"]["base"]
    out = {"k": st["k"][:, :, base:], "k_scale": st["k_scale"][:, :, base:],
           "v": st["cv"][:, :, base:], "v_scale": st["v_scale"][:, :, base:],
           "valid": st["valid"]}
    if st["kmean"] is not None:
        out["kmean"] = st["kmean"][:, :, base:]
    return out


def run(st):
    if not own:
        return _plain(st)
    import block_sparse_kv_bsa_b200 as bsa
    case = st["case"]
    op = case["op"]
    if op in ("attn8", "decode"):
        if op == "attn8":
            bsa.bsa_kv8_attn(st["q"], st["cache"], st["idx"], st["cnt"], q_valid=st["q_valid"],
                             sm_scale=st["sm_scale"], o=st["o"], lse=st["lse"])
        else:
            bsa.bsa_kv8_attn_decode(st["q"], st["cache"], idx=st["idx"], cnt=st["cnt"],
                                    sm_scale=st["sm_scale"], o=st["o"], lse=st["lse"],
                                    workspace=st["workspace"])
        return {"o": st["o"], "lse": st["lse"]}
    T, H, W = case["T"], case["H"], case["W"]
    origin = (case["far"], 0, 0)
    if op == "rope":
        if "pos" in st:
            origin = (0, 0, 0)
        bsa.bsa_rope(st["x"], T, H, W, st["rope"], pos=st.get("pos"), origin=origin,
                     inverse=case["inverse"], out=st["out"])
        return {"y": st["out"]}
    if op == "blocks":
        bsa.bsa_tokens_to_blocks_rope(st["x"], T, H, W, st["rope"], origin=origin, out=st["out"],
                                      perm=st["perm"])
        return {"blocks": st["out"]}
    base = case["base"]
    st["cache"].n_blocks = base
    if op == "append":
        bsa.bsa_kv_append_rope(st["cache"], st["x"], st["v"], T, H, W, st["rope"], origin=origin,
                               perm=st["perm"])
        return {"k": st["k"][:, :, base:], "v": st["cv"][:, :, base:], "valid": st["valid"]}
    bsa.bsa_kv8_append(st["cache"], st["x"], st["v"], T, H, W, rope=st["rope"], origin=origin,
                       perm=st["perm"])
    return _append8_outputs(st)


# ---------------------------------------------------------------------------
# The same results from the definition, in fp64
# ---------------------------------------------------------------------------

def _exact_rotated(st, case, x, sign):
    """x [B, N, Hh, D] rotated through complex products."""
    z = x.to(torch.float64)
    P = int(st["freqs"].shape[0])
    if P == 0:
        return z
    B, n, Hh, D = z.shape
    w = torch.arange(n, device=DEV, dtype=torch.int64)
    if "pos" in st:
        where = [st["pos"][0].to(torch.int64)] * 3
    elif case["pairs_h"] + case["pairs_w"] == 0:
        where = [(w + case["far"])[None]] * 3
    else:
        plane = case["H"] * case["W"]
        where = [(torch.div(w, plane, rounding_mode="floor") + case["far"])[None],
                 torch.div(w % plane, case["W"], rounding_mode="floor")[None],
                 (w % case["W"])[None]]
    turns, at = [], 0
    for p, count in zip(where, (case["pairs_t"], case["pairs_h"], case["pairs_w"])):
        turns.append(p.to(torch.float64)[..., None] * st["freqs"][at:at + count])
        at += count
    turn = torch.polar(torch.full_like(torch.cat(turns, -1), st["amp"]),
                       sign * torch.cat(turns, -1))
    out = z.clone()
    if case["layout"] == "half":
        first, second = slice(0, P), slice(P, 2 * P)
    else:
        first, second = slice(0, 2 * P, 2), slice(1, 2 * P, 2)
    pair = torch.complex(z[..., first], z[..., second]) * turn[:, :, None]
    out[..., first] = pair.real
    out[..., second] = pair.imag
    return out


def _exact_blocks(st, z):
    B, n, Hh, D = z.shape
    nb = (n + BLK - 1) // BLK
    order = torch.argsort(st["perm"])
    rows = torch.zeros((B, nb * BLK, Hh, D), dtype=torch.float64, device=DEV)
    rows[:, :n] = z[:, order]
    return rows.permute(0, 2, 1, 3).reshape(B, Hh, nb, BLK, D)


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "rope":
        return {"y": _exact_rotated(st, case, st["x"], -1.0 if case["inverse"] else 1.0)}
    if op == "blocks":
        r = _exact_blocks(st, _exact_rotated(st, case, st["x"], 1.0))
        return {"blocks": r.reshape(st["out"].shape)}
    if op in ("append", "append8"):
        r = _exact_blocks(st, _exact_rotated(st, case, st["x"], 1.0))
        v = _exact_blocks(st, st["v"].to(torch.float64))
        if op == "append":
            return {"k": r, "v": v, "valid": None}
        out = {}
        for name, x in (("k", r), ("v", v)):
            top = x.flatten(3).abs().max(dim=-1).values.clamp(min=AMAX_FLOOR)
            out[name] = x / top[..., None, None] * E4M3_MAX
            out[name + "_scale"] = top / E4M3_MAX
        out["valid"] = None
        if st["kmean"] is not None:
            n = case["T"] * case["H"] * case["W"]
            rows = [min(BLK, n - BLK * j) for j in range(r.shape[2])]
            count = torch.tensor(rows, dtype=torch.float64, device=DEV)
            out["kmean"] = r.sum(dim=3) / count[:, None]
        return {name: out[name] for name in _append8_outputs(st)}
    # Attention: every query row against the keys of its blocks, through log-sum-exp.
    G, D = case["G"], case["D"]
    o = torch.zeros(st["o"].shape, dtype=torch.float64, device=DEV)
    lse = torch.full(st["lse"].shape, -math.inf, dtype=torch.float64, device=DEV)
    for b in range(case["B"]):
        for h in range(case["Hk"]):
            kf = st["k8"][b, h].to(torch.float64) * st["k_scale"][b, h].double()[:, None, None]
            vf = st["v8"][b, h].to(torch.float64) * st["v_scale"][b, h].double()[:, None, None]
            ok = torch.arange(BLK, device=DEV)[None] < st["valid"][:, None]
            lists = ([torch.arange(case["blocks"], device=DEV)] if op == "decode" and
                     st["idx"] is None else
                     list(st["idx"][b, h].long().reshape(-1, st["idx"].shape[-1])))
            for j, sel in enumerate(lists):
                at = ok[sel].reshape(-1)
                keys = kf[sel].reshape(-1, D)[at]
                vals = vf[sel].reshape(-1, D)[at]
                for g in range(G):
                    head = h * G + g
                    if op == "decode":
                        to = (b, slice(None), head)
                    else:
                        first = j * BLK
                        to = (b, head, slice(first, first + int(st["q_valid"][j])))
                    z = st["q"][to].double() @ keys.T * st["sm_scale"]
                    whole = torch.logsumexp(z, dim=-1)
                    lse[to] = whole
                    o[to] = torch.exp(z - whole[:, None]) @ vals
    return {"o": o, "lse": lse}


# ---------------------------------------------------------------------------
# Work that no implementation can do without
# ---------------------------------------------------------------------------

def work(case):
    op, D = case["op"], case["D"]
    if op in ("rope", "blocks", "append", "append8"):
        n = case["T"] * case["H"] * case["W"]
        nb = -(-n // BLK)
        P = case["pairs_t"] + case["pairs_h"] + case["pairs_w"]
        elems = case["B"] * n * case["Hh"] * D
        slots = case["B"] * nb * BLK * case["Hh"] * D
        flops = 6 * case["B"] * n * case["Hh"] * P
        if op == "rope":
            return {"bytes": 4 * elems + (4 * case["B"] * n if _packed(case) else 0),
                    "flops": flops}
        if op == "blocks":
            return {"bytes": 2 * elems + 2 * slots, "flops": flops}
        if op == "append":
            return {"bytes": 4 * elems + 4 * slots + 4 * nb, "flops": flops}
        means = 4 * case["B"] * nb * case["Hh"] * D if case["pooled"] else 0
        scales = 8 * case["B"] * nb * case["Hh"]
        return {"bytes": 4 * elems + 2 * slots + means + scales + 4 * nb,
                "flops": flops + 4 * elems}
    B, Hk, G = case["B"], case["Hk"], case["G"]
    if op == "attn8":
        n = case["T"] * case["H"] * case["W"]
        nb = -(-n // BLK)
        hist = case["hist"] * nb
        sel = min(case["top_k"], hist) + nb
        read = min(hist, nb * min(case["top_k"], hist)) + nb
        q = B * Hk * G * nb * BLK
        return {"bytes": 4 * q * D + 4 * q + B * Hk * read * (2 * BLK * D + 8)
                + 4 * B * Hk * nb * (sel + 1),
                "flops": 4 * B * Hk * G * nb * BLK * sel * BLK * D}
    sel = min(case["top_k"], case["blocks"]) if case["top_k"] else case["blocks"]
    q = B * case["n_tok"] * Hk * G
    return {"bytes": 4 * q * D + 4 * q + B * Hk * sel * (2 * BLK * D + 8),
            "flops": 4 * q * sel * BLK * D}
