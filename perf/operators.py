"""Timed cases of the operators for continuing a clip from a history kept in pages:

  rotary       rotary positions of Q and K (nabla_rotary), forward and adjoint;
  append       new keys and values into a paged cache, keys rotated on the way
               (nabla_cache_append);
  prefix_attn  attention of a batch over one shared prefix and each sequence's own tail
               (nabla_prefix_attn), optionally merged with a partial result.

``run`` computes an operator in plain torch operations (32-bit arithmetic, angles in 64
bits), or, with ``own`` set, through the package's entry points.  ``exact`` computes it in 64
bits from its definition.
"""

from __future__ import annotations

import math
import random

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ---------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------
def _rotary(name, B, S, Hq, Hk, D, dim, style, axes, grid, dtype, out, scaling="none",
            positions=False, strided=False, reorder=False, adjoint=False):
    return dict(name=name, op="rotary", B=B, S=S, Hq=Hq, Hk=Hk, D=D, dim=dim, style=style, axes=axes,
                T=grid[0], Hg=grid[1], W=grid[2], dtype=dtype, out=out, scaling=scaling,
                positions=positions, strided=strided, reorder=reorder, adjoint=adjoint)


def _append(name, B, S, Hq, Hkv, D, dim, style, axes, Hg, W, page, past, ragged, dtype, pos0):
    return dict(name=name, op="append", B=B, S=S, Hq=Hq, Hkv=Hkv, D=D, dim=dim, style=style, axes=axes,
                Hg=Hg, W=W, page=page, past=past, ragged=ragged, dtype=dtype, pos0=pos0, lens_seed=3)


def _attn(name, B, Hq, Hkv, D, Sq, P, tail, page, causal, ragged, part, dtype):
    return dict(name=name, op="prefix_attn", B=B, Hq=Hq, Hkv=Hkv, D=D, Sq=Sq, P=P, tail=tail, page=page,
                causal=causal, ragged=ragged, part=part, dtype=dtype, lens_seed=5)


def listed():
    return [
        # one new token of each of 8 sequences at far positions: the smallest call, pure latency
        _rotary("rotary token", 8, 1, 32, 8, 128, 128, "half", 1, (1, 1, 1), "bf16", "bf16",
                scaling="linear", positions=True),
        # Q and K of the 720p-like latent, all heads, rotated into the block order the mask and
        # the attention read: the largest call of the path
        _rotary("rotary latent", 1, 80640, 40, 40, 128, 128, "interleaved", 3, (21, 48, 80), "bf16",
                "bf16", reorder=True),
        # the training step's f32 dQ and dK in block order back to bf16 gradients in the natural order
        _rotary("rotary gradient", 2, 19712, 24, 24, 128, 128, "interleaved", 3, (11, 32, 56), "f32",
                "bf16", reorder=True, adjoint=True),
        # the leading part of each head, odd length, the [B, S, H, D] views of a projection, grouped
        # heads, frequencies scaled by parts for a longer context
        _rotary("rotary partial", 3, 4097, 20, 4, 128, 96, "half", 1, (1, 1, 1), "f16", "f16",
                scaling="parts", strided=True),
        # a decoding step of 64 sequences: Q rotated, K rotated and stored, V stored
        _append("append token", 64, 1, 32, 8, 128, 128, "half", 1, 1, 1, 64, 2000, False, "bf16", 8192),
        # four finished latent frames of 24 heads added to the history
        _append("append frames", 1, 7168, 0, 24, 128, 128, "interleaved", 3, 32, 56, 64, 14336, False,
                "bf16", 0),
        # a padded batch of prompts of uneven length, small pages, half of the head rotated
        _append("append ragged", 16, 333, 16, 4, 64, 32, "half", 1, 1, 1, 16, 100, True, "f16", 1000),
        # one token for each of 4 sequences over a short prefix: pure latency
        _attn("attn token short", 4, 16, 4, 128, 1, 1000, 150, 16, False, False, False, "bf16"),
        # a decoding step of 32 sequences over a long shared prefix with uneven tails: the cache's bytes
        _attn("attn token long", 32, 32, 8, 128, 1, 32768, 1500, 64, False, False, False, "bf16"),
        # a few drafted tokens checked at once, causal among themselves
        _attn("attn drafted", 12, 24, 24, 64, 5, 4099, 300, 32, True, False, False, "f16"),
        # a padded batch of prompts behind a shared one, causal, odd lengths
        _attn("attn prompts", 5, 16, 4, 128, 1501, 5003, 1700, 128, True, True, False, "f16"),
        # two continuations of four latent frames each against a history of eight frames, merged with
        # the sparse attention inside the new frames: arithmetic
        _attn("attn frames", 2, 24, 24, 128, 7168, 14336, 0, 64, False, False, True, "bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("rotary", "append", "prefix_attn", "prefix_attn"))
    D = rng.choice((64, 128))
    dtype = rng.choice(("bf16", "f16"))
    style = rng.choice(("interleaved", "half"))
    page = rng.choice((16, 32, 64, 128, 256))
    if op == "rotary":
        grid = rng.random() < 0.5
        B, Hk = rng.randint(1, 4), rng.randint(1, 12)
        Hq = Hk * rng.choice((1, 2, 4))
        if grid:
            T, Hg, W = rng.randint(1, 12), 8 * rng.randint(1, 6), 8 * rng.randint(1, 8)
            S, dim = T * Hg * W, D
        else:
            T = Hg = W = 1
            S, dim = _log(rng, 1, 16384), 2 * rng.randint(1, D // 2)
        c = _rotary("", B, S, Hq, Hk, D, dim, style, 3 if grid else 1, (T, Hg, W),
                    rng.choice((dtype, "f32")), dtype, scaling=rng.choice(("none", "linear", "ntk", "parts")),
                    positions=not grid and rng.random() < 0.5, strided=rng.random() < 0.4,
                    reorder=grid and rng.random() < 0.5, adjoint=rng.random() < 0.4)
    elif op == "append":
        B, Hkv = _log(rng, 1, 64), rng.randint(1, 16)
        S = _log(rng, 1, max(2, 60000 // (B * Hkv)))
        grid = rng.random() < 0.3
        Hg, W = (rng.randint(2, 40), rng.randint(2, 40)) if grid else (1, 1)
        dim = D if grid else 2 * rng.randint(1, D // 2)
        c = _append("", B, S, Hkv * rng.choice((0, 1, 4)), Hkv, D, dim, style, 3 if grid else 1, Hg, W, page,
                    _log(rng, 1, 3000), rng.random() < 0.5, dtype, _log(rng, 1, 1 << 20))
        c["lens_seed"] = rng.randint(1, 1 << 20)
    else:
        Hkv, G = rng.randint(1, 12), rng.choice((1, 1, 2, 3, 4, 8))
        B, Sq = _log(rng, 1, 32), rng.choice((1, 1, _log(rng, 2, 4096)))
        P, tail = _log(rng, 1, 40000), rng.choice((0, Sq + _log(rng, 1, 2000), Sq + _log(rng, 1, 2000)))
        while B * Hkv * G * Sq * (P + tail) > 4e9:   # below the largest listed case
            if B > 1 and rng.random() < 0.5:
                B -= B // 2
            else:
                P = P - P // 2
        while B * Hkv * tail > 500000:
            B = B // 2
        causal = tail > 0 and rng.random() < 0.5
        c = _attn("", B, Hkv * G, Hkv, D, Sq, P, tail, page, causal, Sq > 1 and rng.random() < 0.5,
                  rng.random() < 0.25, dtype)
        c["lens_seed"] = rng.randint(1, 1 << 20)
    del c["name"]
    return c


# ---------------------------------------------------------------------------------------
# what a case stands for: lengths, frequencies, bytes and operations
# ---------------------------------------------------------------------------------------
def _axis_dims(c):
    """Rotated elements of the three latent axes (t takes what h and w leave)."""
    s = c["dim"] // 3 // 2 * 2
    return (c["dim"] - 2 * s, s, s) if c["axes"] == 3 else (c["dim"], 0, 0)


def _frequencies(c):
    """(64-bit frequencies of the pairs, magnitude factor): base 10000, scaled for a context 8 times
    longer than 4096 where the case asks for it."""
    f, factor, base = [], 8.0, 10000.0
    scaling = c.get("scaling", "none")
    for d in _axis_dims(c):
        b = base * factor ** (d / (d - 2)) if scaling == "ntk" and d > 2 else base
        e = [b ** (-2.0 * j / d) for j in range(d // 2)]
        if scaling == "linear":
            e = [x / factor for x in e]
        if scaling == "parts":     # fast pairs kept, slow ones interpolated, a ramp between
            at = [d * math.log(4096 / (r * 2 * math.pi)) / (2 * math.log(base)) for r in (32.0, 1.0)]
            lo, hi = max(math.floor(at[0]), 0), min(math.ceil(at[1]), d - 1)
            ramp = [min(max((j - lo) / max(hi - lo, 1e-3), 0.0), 1.0) for j in range(d // 2)]
            e = [x * (1 - r) + x / factor * r for x, r in zip(e, ramp)]
        f += e
    return f, 0.1 * math.log(factor) + 1.0 if scaling == "parts" else 1.0


def _append_lens(c):
    r = random.Random(c["lens_seed"])
    past = [r.randint(0, c["past"]) for _ in range(c["B"])]
    new = [r.randint(0, c["S"]) if c["ragged"] else c["S"] for _ in range(c["B"])]
    return past, new


def _attn_lens(c):
    r = random.Random(c["lens_seed"])
    n = [r.randint(0, c["Sq"]) if c["ragged"] else c["Sq"] for _ in range(c["B"])]
    tails = [k + r.randint(0, c["tail"] - c["Sq"]) if c["tail"] else 0 for k in n]
    return n, tails


def _size(name):
    return 4 if name == "f32" else 2


def work(case):
    c = case
    if c["op"] == "rotary":
        n = c["B"] * c["S"] * (c["Hq"] + c["Hk"]) * c["D"]
        return {"bytes": n * (_size(c["dtype"]) + _size(c["out"])), "flops": 3 * n * c["dim"] // c["D"]}
    if c["op"] == "append":
        n = sum(_append_lens(c)[1]) * c["D"]
        rot = n + (c["B"] * c["S"] * c["D"] - n if c["Hq"] else 0)
        return {"bytes": 4 * (2 * n * c["Hkv"] + rot * c["Hq"]), "flops": 3 * n * (c["Hkv"] + c["Hq"])}
    n, tails = _attn_lens(c)
    keys = 0
    for k, t in zip(n, tails):
        total = c["P"] + t
        keys += k * total - (k * (k - 1) // 2 if c["causal"] else 0)
    rows = sum(n) * c["Hq"]
    kv = 4 * c["D"] * c["Hkv"] * (c["P"] + sum(tails))
    io = rows * (4 * c["D"] + 4) + (rows * (4 * c["D"] + 4) if c["part"] else 0)
    return {"bytes": kv + io, "flops": 4 * c["D"] * c["Hq"] * keys}


# ---------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------
def _normal(gen, shape, dtype, std=1.0):
    x = torch.empty(shape, dtype=dtype, device=DEV)
    x.normal_(0.0, std, generator=gen)
    return x


def _heads(gen, c, H, dtype):
    if H == 0:
        return None
    if c.get("strided"):
        return _normal(gen, (c["B"], c["S"], H, c["D"]), dtype, 1.5).transpose(1, 2)
    return _normal(gen, (c["B"], H, c["S"], c["D"]), dtype, 1.5)


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _pages(gen, want, spare):
    """Lists of page numbers, shuffled over a pool with a few spare pages."""
    order = torch.randperm(sum(want) + spare, generator=gen, device=DEV).to(torch.int32)
    return order, order.numel()


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    s = {"case": c}
    if c["op"] in ("rotary", "append"):
        f, m = _frequencies(c)
        s["inv_freq"] = torch.tensor(f, dtype=torch.float64, device=DEV)
        s["magnitude"] = m
        s["axis"] = torch.tensor([a for a, d in enumerate(_axis_dims(c)) for _ in range(d // 2)], device=DEV)
    if c["op"] == "rotary":
        s["q"] = _heads(gen, c, c["Hq"], DTYPES[c["dtype"]])
        s["k"] = _heads(gen, c, c["Hk"], DTYPES[c["dtype"]])
        if c["positions"]:
            at = torch.randint(0, 1 << 20, (c["B"], 1), generator=gen, device=DEV)
            s["positions"] = (at + torch.arange(c["S"], device=DEV)).to(torch.int32)
        return s
    dtype = DTYPES[c["dtype"]]
    page = c["page"]
    if c["op"] == "append":
        past, new = _append_lens(c)
        s["k"], s["v"] = _heads(gen, c, c["Hkv"], dtype), _heads(gen, c, c["Hkv"], dtype)
        s["q"] = _heads(gen, c, c["Hq"], dtype)
        s["start"], s["counts"] = _ints(past), _ints(new) if c["ragged"] else None
        per = -(-max(p + n for p, n in zip(past, new)) // page)
        order, n_pages = _pages(gen, [max(per, 1)] * c["B"], 3)
        s["table"] = order[:c["B"] * max(per, 1)].reshape(c["B"], -1).contiguous()
    else:
        n, tails = _attn_lens(c)
        np_ = -(-c["P"] // page)
        per = -(-max(c["tail"], 0) // page)
        order, n_pages = _pages(gen, [np_, per * c["B"]], 3)
        s["q"] = _normal(gen, (c["B"], c["Hq"], c["Sq"], c["D"]), dtype, 1.5)
        s["prefix"] = order[:np_].contiguous()
        s["tail_pages"] = order[np_:np_ + per * c["B"]].reshape(c["B"], per).contiguous() if per else None
        s["tail_len"] = _ints(tails) if per else None
        s["q_len"] = _ints(n) if c["ragged"] else None
        s["scale"] = 1.0 / math.sqrt(c["D"])
        shape = (c["B"], c["Hq"], c["Sq"])
        if c["part"]:
            s["part_o"] = _normal(gen, shape + (c["D"],), torch.float32, 0.1)
            s["part_lse"] = _normal(gen, shape, torch.float32) + math.log(c["P"])
        # a padded batch's rows behind a sequence's queries stay as they are
        s["o"] = torch.zeros(shape + (c["D"],), dtype=dtype, device=DEV)
        s["lse"] = torch.zeros(shape, dtype=torch.float32, device=DEV)
    s["k_cache"] = _normal(gen, (n_pages, c["Hkv"], page, c["D"]), dtype)
    s["v_cache"] = _normal(gen, (n_pages, c["Hkv"], page, c["D"]), dtype)
    return s


# ---------------------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------------------
def _grid_positions(n, Hg, W):
    return torch.stack((n // (Hg * W), n // W % Hg, n % W), -1)


def _cos_sin(c, s, pos):
    """cos and sin [..., pairs] of positions [..., axes], the angle in 64 bits."""
    angle = pos.double()[..., s["axis"]] * s["inv_freq"]
    m = s["magnitude"]
    return (angle.cos() * m).float(), (angle.sin() * m).float()


def _rotate(c, x, cos, sin):
    """x [B, H, S, D] with cos, sin [B or 1, S, pairs]."""
    cos, sin = cos.unsqueeze(1), sin.unsqueeze(1)
    f, h = x.float(), c["dim"] // 2
    if c["style"] == "half":
        a, b = f[..., :h], f[..., h:2 * h]
        y = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    else:
        a, b = f[..., 0:2 * h:2], f[..., 1:2 * h:2]
        y = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    return torch.cat((y, f[..., 2 * h:]), -1)


def _to_blocks(c, x):
    """[B, H, S, D] natural order -> 8 x 8 patches of a frame as runs of 64 tokens."""
    B, H, S, D = x.shape
    y = x.reshape(B, H, c["T"], c["Hg"] // 8, 8, c["W"] // 8, 8, D).transpose(4, 5)
    return y.reshape(B, H, S, D)


def _from_blocks(c, x):
    B, H, S, D = x.shape
    y = x.reshape(B, H, c["T"], c["Hg"] // 8, c["W"] // 8, 8, 8, D).transpose(4, 5)
    return y.reshape(B, H, S, D)


def _plain_rotary(s):
    c = s["case"]
    n = torch.arange(c["S"], device=DEV)
    if c["positions"]:
        pos = s["positions"].unsqueeze(-1)
    else:
        pos = (_grid_positions(n, c["Hg"], c["W"]) if c["axes"] == 3 else n.unsqueeze(-1)).unsqueeze(0)
    cos, sin = _cos_sin(c, s, pos)
    out = []
    for x in (s["q"], s["k"]):
        if c["adjoint"]:
            x = _from_blocks(c, x) if c["reorder"] else x
            y = _rotate(c, x, cos, -sin)
        else:
            y = _rotate(c, x, cos, sin)
            y = _to_blocks(c, y) if c["reorder"] else y
        out.append(y.to(DTYPES[c["out"]]))
    return tuple(out)


def _plain_append(s):
    c = s["case"]
    at = s["start"].long().unsqueeze(1) + torch.arange(c["S"], device=DEV)        # [B, S]
    n = at + c["pos0"]
    pos = _grid_positions(n, c["Hg"], c["W"]) if c["axes"] == 3 else n.unsqueeze(-1)
    cos, sin = _cos_sin(c, s, pos)
    dtype = DTYPES[c["dtype"]]
    k = _rotate(c, s["k"], cos, sin).to(dtype).transpose(1, 2)                     # [B, S, H, D]
    v = s["v"].transpose(1, 2)
    page = torch.gather(s["table"].long(), 1, (at // c["page"]).clamp(max=s["table"].shape[1] - 1))
    slot = at % c["page"]
    if s["counts"] is not None:
        keep = torch.arange(c["S"], device=DEV) < s["counts"].unsqueeze(1)
        k, v, page, slot = k[keep], v[keep], page[keep], slot[keep]
    s["k_cache"][page, :, slot] = k
    s["v_cache"][page, :, slot] = v
    if s["q"] is None:
        return s["k_cache"], s["v_cache"]
    return s["k_cache"], s["v_cache"], _rotate(c, s["q"], cos, sin).to(dtype)


def _read_pages(cache, pages):
    """[..., n] page numbers -> f32 [..., H, n * page, D]."""
    x = cache[pages.long()].transpose(-4, -3)
    return x.flatten(-3, -2).float()


def _plain_attn(s):
    c = s["case"]
    B, Hq, Hkv, D, Sq, P = (c[k] for k in ("B", "Hq", "Hkv", "D", "Sq", "P"))
    G, R = Hq // Hkv, Hq // Hkv * Sq
    q = (s["q"].float() * s["scale"]).reshape(B, Hkv, R, D)
    i = torch.arange(Sq, device=DEV)
    n = s["q_len"].long() if s["q_len"] is not None else torch.full((B,), Sq, device=DEV)
    tl = s["tail_len"].long() if s["tail_len"] is not None else torch.zeros(B, dtype=torch.long, device=DEV)
    if c["causal"]:
        seen = (P + tl - n).unsqueeze(1) + i + 1                                   # [B, Sq] visible keys
    else:
        seen = (P + tl).unsqueeze(1).expand(B, Sq)
    seen = seen.repeat(1, G).reshape(B, 1, R, 1)
    kp, vp = (_read_pages(s[x], s["prefix"])[:, :P] for x in ("k_cache", "v_cache"))    # [Hkv, P, D]
    rows = q.transpose(0, 1).reshape(Hkv, B * R, D)
    sp = (rows @ kp.transpose(1, 2)).reshape(Hkv, B, R, P).transpose(0, 1)
    if c["causal"] and c["tail"] < Sq:
        sp = torch.where(torch.arange(P, device=DEV) < seen, sp, -math.inf)
    top = sp.amax(-1, keepdim=True)
    if c["tail"]:
        kt, vt = (_read_pages(s[x], s["tail_pages"]) for x in ("k_cache", "v_cache"))   # [B, Hkv, L, D]
        L = kt.shape[2]
        j = torch.arange(L, device=DEV)
        st = torch.where((j + P < seen) & (j < tl.reshape(B, 1, 1, 1)), q @ kt.transpose(2, 3), -math.inf)
        top = torch.maximum(top, st.amax(-1, keepdim=True))
    top = top.clamp(min=-1e30)
    ep = torch.exp(sp - top)
    total = ep.sum(-1, keepdim=True)
    o = (ep.transpose(0, 1).reshape(Hkv, B * R, P) @ vp).reshape(Hkv, B, R, D).transpose(0, 1)
    if c["tail"]:
        et = torch.exp(st - top)
        total = total + et.sum(-1, keepdim=True)
        o = o + et @ vt
    o = (o / total.clamp(min=1e-37)).reshape(B, Hq, Sq, D)
    lse = (top + total.log()).reshape(B, Hq, Sq)
    if c["part"]:
        both = torch.logaddexp(lse, s["part_lse"])
        o = o * (lse - both).exp().unsqueeze(-1) + s["part_o"] * (s["part_lse"] - both).exp().unsqueeze(-1)
        lse = both
    if s["q_len"] is not None:
        keep = (i < n.unsqueeze(1)).unsqueeze(1)
        o = torch.where(keep.unsqueeze(-1), o, s["o"].float())
        lse = torch.where(keep, lse, s["lse"])
    return o.to(s["q"].dtype), lse


def run(state):
    s, c = state, state["case"]
    if not own:
        return {"rotary": _plain_rotary, "append": _plain_append, "prefix_attn": _plain_attn}[c["op"]](s)
    import adaptive_block_sparse_b200 as m
    if c["op"] == "prefix_attn":
        return m.nabla_prefix_attn(s["q"], s["k_cache"], s["v_cache"], s["prefix"], c["P"],
                                   tail_pages=s["tail_pages"], tail_len=s["tail_len"], q_len=s["q_len"],
                                   causal=c["causal"], scale=s["scale"], part_o=s.get("part_o"),
                                   part_lse=s.get("part_lse"), o=s["o"], lse=s["lse"])
    rope = m.Rope(s["inv_freq"], style=m.NABLA_ROPE_HALF if c["style"] == "half" else m.NABLA_ROPE_INTERLEAVED,
                  axis_dims=_axis_dims(c) if c["axes"] == 3 else None, magnitude=s["magnitude"])
    if c["op"] == "rotary":
        nat = m.NABLA_LAYOUT_NATURAL
        blocks = m.NABLA_LAYOUT_REORDERED if c["reorder"] else nat
        return m.nabla_rotary(s["q"], s["k"], rope, grid=(c["T"], c["Hg"], c["W"]) if c["axes"] == 3 else None,
                              positions=s.get("positions"), adjoint=c["adjoint"], out_dtype=DTYPES[c["out"]],
                              src_layout=blocks if c["adjoint"] else nat,
                              dst_layout=nat if c["adjoint"] else blocks)
    q = m.nabla_cache_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["table"], s["start"], rope=rope,
                             frame=(c["Hg"], c["W"]), pos0=c["pos0"], counts=s["counts"], q=s["q"])
    return (s["k_cache"], s["v_cache"]) if q is None else (s["k_cache"], s["v_cache"], q)


# ---------------------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------------------
def _exact_rotate(c, s, x, pos):
    """Pairs as complex numbers times m e^(i angle); x [B, H, S, D], pos [B or 1, S, axes]."""
    h, y = c["dim"] // 2, x.double()
    first = 0
    for a, d in enumerate(_axis_dims(c)[:c["axes"]]):
        p = torch.arange(first, first + d // 2, device=x.device)
        first += d // 2
        i0, i1 = (p, p + h) if c["style"] == "half" else (2 * p, 2 * p + 1)
        turn = pos[..., a].double().unsqueeze(-1) * s["inv_freq"][p]
        z = torch.polar(torch.full_like(turn, s["magnitude"]), -turn if c.get("adjoint") else turn).unsqueeze(1)
        w = torch.complex(y[..., i0], y[..., i1]) * z
        y[..., i0], y[..., i1] = w.real, w.imag
    return y


def _block_order(c):
    """Natural index of every token of the block order."""
    n = torch.arange(c["T"] * c["Hg"] * c["W"], device=DEV).reshape(c["T"], c["Hg"], c["W"])
    n = n.unfold(1, 8, 8).unfold(2, 8, 8)      # [T, Hg/8, W/8, 8, 8]
    return n.reshape(-1)


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "rotary":
        n = torch.arange(c["S"], device=DEV)
        pos = (torch.stack((n // (c["Hg"] * c["W"]), n // c["W"] % c["Hg"], n % c["W"]), -1)
               if c["axes"] == 3 else n.unsqueeze(-1)).unsqueeze(0)
        if c["positions"]:
            pos = s["positions"].unsqueeze(-1)
        order = _block_order(c) if c["reorder"] else n
        out = []
        for x in (s.pop("q"), s.pop("k")):
            if c["adjoint"]:
                y = torch.empty_like(x)
                y[:, :, order] = x
                out.append(_exact_rotate(c, s, y, pos))
            else:
                out.append(_exact_rotate(c, s, x, pos)[:, :, order])
        return tuple(out)
    if c["op"] == "append":
        past, new = _append_lens(c)
        kc, vc = s["k_cache"].double(), s["v_cache"].double()
        at = torch.stack([torch.arange(p, p + c["S"], device=DEV) for p in past])
        n = at + c["pos0"]
        pos = (torch.stack((n // (c["Hg"] * c["W"]), n // c["W"] % c["Hg"], n % c["W"]), -1)
               if c["axes"] == 3 else n.unsqueeze(-1))
        k = _exact_rotate(c, s, s["k"], pos)
        for b in range(c["B"]):
            pg, sl = s["table"][b].long()[at[b, :new[b]] // c["page"]], at[b, :new[b]] % c["page"]
            kc[pg, :, sl] = k[b].transpose(0, 1)[:new[b]]
            vc[pg, :, sl] = s["v"][b].transpose(0, 1)[:new[b]].double()
        return (kc, vc) if s["q"] is None else (kc, vc, _exact_rotate(c, s, s["q"], pos))
    n, tails = _attn_lens(c)
    P, G, page = c["P"], c["Hq"] // c["Hkv"], c["page"]
    o, lse = s["o"].double(), s["lse"].double()
    for h in range(c["Hkv"]):
        def keys(cache, pages, count):
            return s[cache][pages.long(), h].reshape(-1, c["D"])[:count].double()
        kp, vp = (keys(x, s["prefix"], P) for x in ("k_cache", "v_cache"))
        for b in range(c["B"]):
            if n[b] == 0:
                continue
            k, v = kp, vp
            if tails[b]:
                t = s["tail_pages"][b, :-(-tails[b] // page)]
                k, v = torch.cat((k, keys("k_cache", t, tails[b]))), torch.cat((v, keys("v_cache", t, tails[b])))
            for g in range(G):
                hq = h * G + g
                logits = (s["q"][b, hq, :n[b]].double() @ k.T).mul_(s["scale"])
                if c["causal"]:
                    hidden = torch.ones(logits.shape, dtype=torch.bool, device=DEV).triu_(P + tails[b] - n[b] + 1)
                    logits.masked_fill_(hidden, -math.inf)
                e = torch.logsumexp(logits, -1)
                r = logits.sub_(e.unsqueeze(-1)).exp_() @ v
                if c["part"]:
                    pe = s["part_lse"][b, hq, :n[b]].double()
                    both = torch.logsumexp(torch.stack((e, pe)), 0)
                    r = r * (e - both).exp().unsqueeze(-1)
                    r += s["part_o"][b, hq, :n[b]].double() * (pe - both).exp().unsqueeze(-1)
                    e = both
                o[b, hq, :n[b]], lse[b, hq, :n[b]] = r, e
    return o, lse
