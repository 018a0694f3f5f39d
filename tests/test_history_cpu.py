"""Rotary positions and the paged cache on the host: the oracle against closed forms, the
frequencies, and the C entry points' refusals (nothing reaches a GPU)."""
import ctypes
import math

import numpy as np
import pytest
import torch

from oracle import history as H


@pytest.fixture(scope="module")
def nb():
    from adaptive_block_sparse_b200 import build as b
    b.build()
    import adaptive_block_sparse_b200 as m
    m.load_library()
    return m


def test_oracle_rotary_is_a_rotation():
    rng = np.random.default_rng(0)
    x = rng.normal(size=(1, 2, 5, 64))
    f, _ = H.rotary_freqs(64)
    pos = H.grid_positions(5, 1, 1, 1, first=9)[None]
    for inter in (True, False):
        y = H.rotary(x, pos, f, inter)
        np.testing.assert_allclose((y ** 2).sum(-1), (x ** 2).sum(-1), rtol=1e-12)
        np.testing.assert_allclose(H.rotary(y, pos, f, inter, adjoint=True), x, atol=1e-12)
        # logits depend on the distance of positions alone
        a = H.rotary(x[:, :, :1], pos[:, :1], f, inter)[0, 0, 0] @ H.rotary(x[:, 1:, 1:2], pos[:, :1] + 3, f, inter)[0, 0, 0]
        b = H.rotary(x[:, :, :1], pos[:, :1] + 50, f, inter)[0, 0, 0] @ H.rotary(x[:, 1:, 1:2], pos[:, :1] + 53, f, inter)[0, 0, 0]
        assert abs(a - b) < 1e-10
    # one pair, a quarter turn
    y = H.rotary(np.array([[[[3.0, 4.0]]]]), np.array([[[1]]]), np.array([math.pi / 2]), True)
    np.testing.assert_allclose(y, [[[[-4.0, 3.0]]]], atol=1e-12)


def test_oracle_append_and_positions():
    assert H.grid_positions(3, 4, 5, 3, first=19).tolist() == [[0, 3, 4], [1, 0, 0], [1, 0, 1]]
    c = H.append(np.zeros((3, 1, 2, 1)), np.arange(1.0, 4.0).reshape(1, 1, 3, 1), [[2, 0]], [1], [3])
    assert c.reshape(3, 2).tolist() == [[2, 3], [0, 0], [0, 1]]


@pytest.mark.parametrize("scaling", ["plain", "linear", "base", "parts"])
@pytest.mark.parametrize("dim", [2, 4, 42, 44, 64, 96, 128])
def test_frequencies(nb, scaling, dim):
    code = {"plain": nb.NABLA_ROPE_PLAIN, "linear": nb.NABLA_ROPE_LINEAR, "base": nb.NABLA_ROPE_BASE,
            "parts": nb.NABLA_ROPE_PARTS}[scaling]
    got, mag = nb.nabla_rotary_freqs(dim, 10000.0, code, 8.0, 4096)
    want, wmag = H.rotary_freqs(dim, 10000.0, scaling, 8.0, 4096)
    np.testing.assert_allclose(got, want, rtol=1e-13)
    assert mag == pytest.approx(wmag, rel=1e-15)
    assert got[0] == (0.125 if scaling == "linear" else 1.0)
    # the slowest pair ends divided by the factor (base: by design at the last pair)
    if scaling in ("base", "parts", "linear") and dim >= 42:
        assert got[-1] == pytest.approx(10000.0 ** (-(dim - 2) / dim) / 8, rel=1e-12)


def test_frequencies_refuse(nb):
    bad = [dict(dim=3), dict(dim=0), dict(base=1.0), dict(base=math.nan), dict(factor=0.5), dict(scaling=4),
           dict(scaling=-1), dict(scaling=nb.NABLA_ROPE_PARTS, trained_len=0.0)]
    for kw in bad:
        with pytest.raises(nb.NablaError) as e:
            nb.nabla_rotary_freqs(**{"dim": 64, **kw})
        assert e.value.status == nb.NABLA_ERR_INVALID_ARG


A, B2, C3, D4 = 0x10000000, 0x20000000, 0x30000000, 0x40000000    # fake, aligned, never dereferenced


def _view(nb, ptr, Hh=2, dtype=0, S=32, D=64, **kw):
    d = dict(ptr=ptr, dtype=dtype, H=Hh, stride_b=Hh * S * D, stride_h=S * D, stride_s=D)
    d.update(kw)
    return nb._Heads(*[d[k] for k in ("ptr", "dtype", "H", "stride_b", "stride_h", "stride_s")])


def _rope(nb, style=0, dim=64, axes=1, dims=(64, 0, 0), mag=1.0, freq=0x5000):
    return nb._Rope(style, dim, axes, *dims, mag, freq)


def test_rotary_refuses(nb):
    lib = nb.load_library()
    INV, UNS = nb.NABLA_ERR_INVALID_ARG, nb.NABLA_ERR_UNSUPPORTED

    def call(qs=None, qd=None, ks=nb._Heads(), kd=nb._Heads(), B=1, grid=(2, 16, 1), D=64, rope=None,
             pos=None, sl=1, dl=1, adj=0):
        return lib.nabla_rotary(qs or _view(nb, A), qd or _view(nb, B2), ks, kd, B, nb._Grid(*grid), D,
                                rope or _rope(nb), nb._Grid(0, 0, 0), pos, sl, dl, adj, None)
    assert call(B=0) == INV and call(grid=(0, 1, 1)) == INV and call(D=96) == UNS
    assert call(rope=_rope(nb, style=2)) == INV and call(rope=_rope(nb, dim=66)) == INV
    assert call(rope=_rope(nb, dim=7)) == INV and call(rope=_rope(nb, dim=0)) == INV
    assert call(rope=_rope(nb, axes=2)) == INV and call(rope=_rope(nb, axes=3, dims=(20, 20, 20))) == INV
    assert call(rope=_rope(nb, axes=3, dims=(21, 21, 22))) == INV
    assert call(rope=_rope(nb, freq=None)) == INV and call(rope=_rope(nb, freq=0x5004)) == INV
    assert call(rope=_rope(nb, mag=math.nan)) == INV
    assert call(adj=2) == INV and call(sl=2) == INV and call(dl=-1) == INV
    assert call(dl=0) == INV                                           # 16 x 1 is no grid of 8 x 8 patches
    assert call(grid=(1 << 20, 1 << 12, 1)) == UNS                     # 2^32 tokens
    assert call(pos=0x10002) == INV
    assert call(qs=nb._Heads(), qd=nb._Heads()) == INV                 # nothing to do
    assert call(qd=nb._Heads()) == INV and call(qs=_view(nb, A + 8)) == INV
    assert call(qs=_view(nb, A, stride_s=68)) == INV                   # rows not 16-byte aligned
    assert call(qs=_view(nb, A, stride_s=-64)) == INV
    assert call(qd=_view(nb, B2, stride_h=0)) == INV                   # a destination written twice
    assert call(qd=_view(nb, B2, Hh=3)) == INV and call(qs=_view(nb, A, Hh=0)) == INV
    assert call(qs=_view(nb, A, dtype=7)) == INV and call(qd=_view(nb, B2, dtype=2)) == INV   # bf16 -> fp16
    assert call(qd=_view(nb, A)) == INV                                # in place
    assert call(qd=_view(nb, A + 64 * 64)) == INV                      # overlap
    assert call(ks=_view(nb, C3, dtype=1), kd=_view(nb, D4)) == INV    # Q and K of different dtypes
    assert call(ks=_view(nb, C3), kd=_view(nb, A)) == INV              # K's output over Q's input
    assert call(ks=_view(nb, C3), kd=_view(nb, B2)) == INV             # one output for both


def test_append_refuses(nb):
    lib = nb.load_library()
    INV, UNS = nb.NABLA_ERR_INVALID_ARG, nb.NABLA_ERR_UNSUPPORTED

    def cache(k=C3, v=D4, n=4, Hh=2, page=16, D=64, dtype=0):
        return nb._Cache(k, v, n, Hh, page, D, dtype)

    def call(k=None, v=None, qs=nb._Heads(), qd=nb._Heads(), B=1, S=32, c=None, table=0x1000, width=4,
             start=0x2000, counts=None, rope=None, frame=(0, 1, 1), pos0=0, pos=None, status=None):
        return lib.nabla_cache_append(k or _view(nb, A), v or _view(nb, B2), qs, qd, B, S, c or cache(), table,
                                      width, start, counts, ctypes.byref(rope) if rope else None,
                                      nb._Grid(*frame), pos0, pos, status, None)
    assert call(B=0) == INV and call(S=0) == INV
    assert call(c=cache(page=24)) == UNS and call(c=cache(page=8)) == UNS and call(c=cache(page=8192)) == UNS
    assert call(c=cache(D=96)) == UNS and call(c=cache(n=0)) == INV and call(c=cache(dtype=1)) == INV
    assert call(c=cache(k=None)) == INV and call(c=cache(v=D4 + 8)) == INV
    assert call(c=cache(v=C3)) == INV                                  # one pool over the other
    assert call(table=None) == INV and call(width=0) == INV and call(start=None) == INV
    assert call(table=0x1002) == INV and call(counts=0x1001) == INV and call(status=0x1002) == INV
    assert call(c=cache(page=4096), width=1 << 20) == UNS
    assert call(pos0=-1) == INV
    assert call(k=_view(nb, A, Hh=3)) == INV and call(v=_view(nb, B2, dtype=2)) == INV
    assert call(k=_view(nb, C3)) == INV                                # a source inside the pool
    assert call(rope=_rope(nb, dim=68)) == INV
    assert call(rope=_rope(nb, axes=3, dims=(20, 20, 24)), frame=(0, 0, 4)) == INV
    q = _view(nb, 0x50000000, Hh=4)
    qd = _view(nb, 0x60000000, Hh=4)
    assert call(qs=q, qd=qd) == INV                                    # Q without a rope
    assert call(qs=q, qd=q, rope=_rope(nb)) == INV                     # in place
    assert call(qs=q, qd=_view(nb, A, Hh=4), rope=_rope(nb)) == INV    # over K
    assert call(qs=q, rope=_rope(nb)) == INV


def test_binding_refuses(nb):
    x = torch.zeros(1, 2, 4, 64)
    freq = torch.ones(32, dtype=torch.float64)
    with pytest.raises(ValueError):
        nb.Rope(freq.float())
    with pytest.raises(ValueError):
        nb.Rope.build(64, "cpu", axis_dims=(20, 20, 20))
    rope = nb.Rope(freq)
    with pytest.raises(ValueError, match="CUDA"):
        nb.nabla_rotary(x, None, rope)
    with pytest.raises(ValueError):
        nb.nabla_rotary(None, None, rope)
    with pytest.raises(TypeError):
        nb.nabla_rotary([1.0], None, rope)
    with pytest.raises(ValueError, match="CUDA"):
        nb.nabla_cache_append(x, x, x, x, freq, freq)
    with pytest.raises(ValueError, match="CUDA"):
        nb.nabla_prefix_attn(x, x, x, None, 0)


def test_oracle_prefix_attention():
    """Against torch's attention over gathered keys, a merge against the union, and empty rows."""
    rng = np.random.default_rng(3)
    B, Hq, Hkv, Sq, D, page, P, tails = 2, 4, 2, 3, 64, 16, 21, [5, 17]
    kc, vc = rng.normal(size=(2, 8, Hkv, page, D))
    q = rng.normal(size=(B, Hq, Sq, D))
    prefix, table = [6, 1], [[0, 2], [4, 5]]
    for causal in (False, True):
        o, lse = H.prefix_attention(q, kc, vc, prefix, P, table, tails, [Sq] * B, causal, 0.125)
        for b in range(B):
            pages = [(prefix[j // page], j % page) for j in range(P)] + [(table[b][j // page], j % page) for j in range(tails[b])]
            k = np.stack([kc[p, :, s] for p, s in pages], 1).repeat(Hq // Hkv, 0)
            v = np.stack([vc[p, :, s] for p, s in pages], 1).repeat(Hq // Hkv, 0)
            n = len(pages)
            mask = torch.ones(Sq, n, dtype=torch.bool).tril(n - Sq) if causal else None
            ref = torch.nn.functional.scaled_dot_product_attention(
                torch.tensor(q[b]), torch.tensor(k), torch.tensor(v), attn_mask=mask, scale=0.125)
            np.testing.assert_allclose(o[b], ref.numpy(), atol=1e-12)
    # prefix alone merged with tails alone = both
    both, bl = H.prefix_attention(q, kc, vc, prefix, P, table, tails, [Sq] * B, False, 0.125)
    po, pl = H.prefix_attention(q, kc, vc, [], 0, table, tails, [Sq] * B, False, 0.125)
    o, lse = H.prefix_attention(q, kc, vc, prefix, P, table, [0, 0], [Sq] * B, False, 0.125, po, pl)
    np.testing.assert_allclose(o, both, atol=1e-12)
    np.testing.assert_allclose(lse, bl, atol=1e-12)
    o, lse = H.prefix_attention(q, kc, vc, [], 0, table, [1, 0], [3, 2], True, 0.125)
    assert np.isneginf(lse[0, :, :2]).all() and (o[0, :, :2] == 0).all() and np.isfinite(lse[0, :, 2]).all()
    assert np.isneginf(lse[1, :, :2]).all() and np.isnan(o[1, :, 2]).all()


def test_prefix_attn_refuses(nb):
    lib = nb.load_library()
    INV, UNS, WS = nb.NABLA_ERR_INVALID_ARG, nb.NABLA_ERR_UNSUPPORTED, nb.NABLA_ERR_WORKSPACE
    need = lib.nabla_prefix_workspace_bytes(1, 4, 2, 32, 64)
    assert need > 256
    for bad in ((0, 4, 2, 32, 64), (1, 3, 2, 32, 64), (1, 4, 0, 32, 64), (1, 4, 2, 0, 64), (1, 4, 2, 32, 96),
                (1 << 20, 4, 2, 1 << 20, 64)):
        assert lib.nabla_prefix_workspace_bytes(*bad) == 0
    Q, K, V, O, L, W = (0x10000000 * i for i in range(1, 7))

    def call(q=None, B=1, Sq=32, cache=None, pages=0x1000, P=20, tail=0x2000, width=4, tlen=0x3000, qlen=None, causal=0,
             scale=0.125, part=nb._Heads(), plse=None, o=None, lse=L, ws=W, wsb=need):
        return lib.nabla_prefix_attn(q or _view(nb, Q, Hh=4), B, Sq, cache or nb._Cache(K, V, 4, 2, 16, 64, 0), pages,
                                     P, tail, width, tlen, qlen, causal, scale, part, plse,
                                     o or _view(nb, O, Hh=4), lse, ws, wsb, None)
    # sizes, dtypes, views
    assert call(B=0) == INV and call(Sq=0) == INV
    assert call(q=_view(nb, Q, Hh=3), o=_view(nb, O, Hh=3)) == INV          # 3 heads on 2 key heads
    assert call(q=_view(nb, Q, Hh=4, dtype=2)) == INV                        # fp16 on a bf16 cache
    assert call(o=_view(nb, O, Hh=2)) == INV and call(o=_view(nb, O, Hh=4, dtype=2)) == INV
    assert call(q=_view(nb, Q + 8, Hh=4)) == INV and call(o=_view(nb, O, Hh=4, stride_s=0)) == INV
    assert call(cache=nb._Cache(K, V, 4, 2, 48, 64, 0)) == UNS and call(cache=nb._Cache(K, V, 4, 2, 16, 32, 0)) == UNS
    assert call(cache=nb._Cache(K, V, 4, 2, 16, 64, 1)) == INV and call(cache=nb._Cache(None, V, 4, 2, 16, 64, 0)) == INV
    # prefix and tails
    assert call(P=-1) == INV and call(pages=None) == INV and call(pages=0x1002) == INV
    assert call(tlen=None) == INV and call(width=0) == INV and call(tail=None) == INV
    assert call(qlen=0x3001) == INV and call(causal=2) == INV
    assert call(P=2147483647) == UNS and call(width=1 << 28) == UNS
    for scale in (0.0, -1.0, math.nan, math.inf):
        assert call(scale=scale) == INV
    # the merged part
    part = _view(nb, 0x70000000, Hh=4, dtype=1)
    assert call(part=part) == INV and call(plse=0x71000000) == INV           # one without the other
    assert call(part=_view(nb, 0x70000000, Hh=4, dtype=2), plse=0x71000000) == INV
    assert call(part=_view(nb, 0x70000000, Hh=2, dtype=1), plse=0x71000000) == INV
    assert call(part=_view(nb, O, Hh=4, dtype=1), plse=0x71000000) == INV    # over o, but not o itself
    assert call(part=part, plse=O) == INV and call(part=part, plse=L + 4) == INV
    # outputs over inputs
    assert call(o=_view(nb, Q, Hh=4)) == INV and call(o=_view(nb, K, Hh=4)) == INV
    assert call(lse=O) == INV and call(lse=Q) == INV and call(lse=V) == INV
    assert call(lse=L + 2) == INV
    # workspace
    assert call(ws=None) == WS and call(wsb=need - 1) == WS and call(ws=W + 16) == WS
