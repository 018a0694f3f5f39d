"""Rotary positions and the paged cache on the GPU, against the fp64 oracle.

Tolerances.  A rotated value is y = m (x0 c - x1 s).  The f32 factors are off by at most
2^-25 pi (the reduced angle's rounding) + 2 * 2^-23 (sincospif, 2 steps) + 2^-24 (times m),
under 4.0e-7; two products and a sum add 3 * 2^-24 = 1.8e-7: together 6e-7 m (|x0| + |x1|).
Storing y rounds by at most half a step, eps / 2 |y| (or half the smallest subnormal).
"""
import math

import numpy as np
import pytest
import torch

from oracle import history as H
from parity_lib import nbl

pytestmark = pytest.mark.gpu
DEV = "cuda"
F32_ERR = 6e-7


def to64(t):
    return t.detach().cpu().double().numpy()


def rnd(shape, dtype, seed, std=1.5):
    g = torch.Generator(device="cpu").manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(dtype).to(DEV)


def assert_rotated(got, x, ref, dtype, m):
    """`got` against the oracle's `ref`, x the unrotated input in the order of ref."""
    big = m * 2 * np.abs(x).max(axis=-1, keepdims=True)
    tiny = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134, torch.float32: 2.0 ** -150}[dtype]
    tol = torch.finfo(dtype).eps / 2 * np.abs(ref) + F32_ERR * big * (1 + torch.finfo(dtype).eps) + tiny
    err = np.abs(to64(got) - ref)
    assert np.isfinite(to64(got)).all()
    assert (err <= tol).all(), f"worst {np.max(err / tol):.3f} of the tolerance"


def block_order(T, Hg, W):
    n = np.arange(T * Hg * W).reshape(T, Hg // 8, 8, W // 8, 8)
    return n.transpose(0, 1, 3, 2, 4).reshape(-1)


# (B, S, Hq, Hk, D, dim, interleaved, src dtype, dst dtype, strided, adjoint)
PLAIN = [
    (1, 1, 1, 1, 64, 64, True, torch.bfloat16, torch.bfloat16, False, False),
    (8, 1, 32, 8, 128, 128, False, torch.bfloat16, torch.bfloat16, False, False),
    (2, 37, 5, 1, 128, 96, False, torch.float16, torch.float16, True, False),
    (3, 129, 6, 2, 64, 2, True, torch.float16, torch.float32, True, True),
    (2, 50, 3, 3, 128, 6, False, torch.bfloat16, torch.float32, False, False),
    (1, 300, 7, 7, 128, 126, False, torch.float32, torch.bfloat16, True, True),
    (2, 65, 4, 2, 64, 62, True, torch.float32, torch.float16, False, False),
    (1, 77, 3, 1, 64, 64, False, torch.float32, torch.float32, True, False),
    (1, 4097, 2, 1, 128, 34, False, torch.float16, torch.float16, False, True),
    (2, 70, 3, 2, 128, 76, False, torch.float32, torch.bfloat16, True, False),
    (2, 70, 13, 2, 128, 10, False, torch.bfloat16, torch.bfloat16, True, False),
    (2, 70, 3, 12, 64, 50, False, torch.float16, torch.float16, True, True),
    (2, 70, 3, 2, 64, 56, False, torch.bfloat16, torch.bfloat16, False, False),
    (1, 900, 40, 40, 128, 128, True, torch.bfloat16, torch.bfloat16, True, False),
]


@pytest.mark.parametrize("B,S,Hq,Hk,D,dim,inter,sd,dd,strided,adjoint", PLAIN)
@pytest.mark.parametrize("far", [False, True])
def test_rotary_sequence(B, S, Hq, Hk, D, dim, inter, sd, dd, strided, adjoint, far):
    m = nbl()
    f, mag = H.rotary_freqs(dim, 10000.0, "parts" if far else "plain", 8.0, 4096)
    style = m.NABLA_ROPE_INTERLEAVED if inter else m.NABLA_ROPE_HALF
    rope = m.Rope.build(dim, DEV, style, scaling=m.NABLA_ROPE_PARTS if far else m.NABLA_ROPE_PLAIN,
                        factor=8.0, trained_len=4096)
    np.testing.assert_allclose(to64(rope.inv_freq), f, rtol=1e-14)
    mag32 = float(np.float32(mag))
    if strided:
        q, k = (rnd((B, S, h, D), sd, 3 + h).transpose(1, 2) for h in (Hq, Hk))
    else:
        q, k = (rnd((B, h, S, D), sd, 5 + h) for h in (Hq, Hk))
    pos = H.grid_positions(S, 1, 1, 1)[None]
    positions = None
    if far:
        pos = pos + np.arange(B)[:, None, None] * 100003 + 1000000
        positions = torch.tensor(pos[..., 0], dtype=torch.int32, device=DEV)
    qo, ko = m.nabla_rotary(q, k, rope, positions=positions, out_dtype=dd, adjoint=adjoint)
    torch.cuda.synchronize()
    for x, y in ((q, qo), (k, ko)):
        ref = H.rotary(to64(x), pos, f, inter, None, mag32, adjoint)
        assert_rotated(y, to64(x), ref, dd, max(mag, 1.0))
        # channels behind the rotated part are the input's, rounded once
        assert torch.equal(y[..., dim:], x[..., dim:].to(dd))


@pytest.mark.parametrize("inter", [True, False])
@pytest.mark.parametrize("src_blocks,dst_blocks", [(False, True), (True, False), (False, False), (True, True)])
def test_rotary_latent_grid(inter, src_blocks, dst_blocks):
    m = nbl()
    B, Hh, T, Hg, W, D = 2, 3, 3, 16, 24, 128
    dims = (44, 42, 42)
    S = T * Hg * W
    f = np.concatenate([H.rotary_freqs(d)[0] for d in dims])
    rope = m.Rope.build(D, DEV, m.NABLA_ROPE_INTERLEAVED if inter else m.NABLA_ROPE_HALF, dims)
    q = rnd((B, Hh, S, D), torch.bfloat16, 1)
    pos = H.grid_positions(S, Hg, W, 3)[None] + np.array([7, 0, 100])
    order = block_order(T, Hg, W)
    nat, blk = m.NABLA_LAYOUT_NATURAL, m.NABLA_LAYOUT_REORDERED
    qo, ko = m.nabla_rotary(q, None, rope, grid=(T, Hg, W), origin=(7, 0, 100),
                            src_layout=blk if src_blocks else nat, dst_layout=blk if dst_blocks else nat)
    assert ko is None
    x = to64(q)
    if src_blocks:
        y = np.empty_like(x)
        y[:, :, order] = x
        x = y
    ref = H.rotary(x, pos, f, inter, dims)
    if dst_blocks:
        x, ref = x[:, :, order], ref[:, :, order]
    assert_rotated(qo, x, ref, torch.bfloat16, 1.0)
    # explicit positions on three axes give the same bits
    p3 = torch.tensor(np.broadcast_to(pos, (B, S, 3)).copy(), dtype=torch.int32, device=DEV)
    q2, _ = m.nabla_rotary(q, None, rope, grid=(T, Hg, W), positions=p3,
                           src_layout=blk if src_blocks else nat, dst_layout=blk if dst_blocks else nat)
    assert torch.equal(q2, qo)


def test_rotary_adjoint_is_the_gradient():
    """<dy, R x> = <R^T dy, x>, and against differences of the forward map."""
    m = nbl()
    B, Hh, S, D, dim = 1, 2, 9, 64, 40
    rope = m.Rope.build(dim, DEV, m.NABLA_ROPE_HALF, scaling=m.NABLA_ROPE_PARTS, factor=4.0, trained_len=64)
    x, dy = rnd((B, Hh, S, D), torch.float32, 1), rnd((B, Hh, S, D), torch.float32, 2)
    y, _ = m.nabla_rotary(x, None, rope)
    dx, _ = m.nabla_rotary(dy, None, rope, adjoint=True)
    lhs, rhs = (to64(dy) * to64(y)).sum(), (to64(dx) * to64(x)).sum()
    # every term is off by at most 2 |x| |dy| F32_ERR m
    bound = 4 * F32_ERR * 1.2 * np.abs(to64(dy)).max() * np.abs(to64(x)).max() * x.numel()
    assert abs(lhs - rhs) <= bound
    # the map is linear, so a difference over a step of 1 is its derivative
    for idx in ((0, 0, 3, 5), (0, 1, 8, 25), (0, 1, 8, 50)):
        x2 = x.clone()
        x2[idx] += 1.0
        y2, _ = m.nabla_rotary(x2, None, rope)
        diff = (to64(dy) * (to64(y2) - to64(y))).sum()
        # x + 1 is off by 2^-24 (|x| + 1), each of the two y by F32_ERR * 2 max|x| m
        tol = 2 * np.abs(to64(dy)).max() * 2.4 * 2 * F32_ERR * (np.abs(to64(x)).max() + 1) * 2
        assert abs(diff - to64(dx)[idx]) <= tol


def test_rotary_keeps_infinities_of_unrotated_channels_apart():
    m = nbl()
    rope = m.Rope.build(32, DEV, m.NABLA_ROPE_INTERLEAVED)
    for style in (m.NABLA_ROPE_INTERLEAVED, m.NABLA_ROPE_HALF):
        rope = m.Rope(rope.inv_freq, style)
        x = rnd((1, 2, 5, 64), torch.bfloat16, 3)
        x[..., 32:] = math.inf
        y, _ = m.nabla_rotary(x, None, rope)
        assert torch.isfinite(y[..., :32]).all() and torch.equal(y[..., 32:], x[..., 32:])


def test_rotary_fused_projection_views_streams_and_graph():
    """Q and K as views of one [B, S, 3, H, D] projection, outputs in a given buffer, on a side
    stream and replayed from a graph."""
    m = nbl()
    B, S, Hh, D = 2, 33, 4, 128
    rope = m.Rope.build(D, DEV, m.NABLA_ROPE_HALF)
    qkv = rnd((B, S, 3, Hh, D), torch.bfloat16, 9)
    q, k = (qkv[:, :, i].transpose(1, 2) for i in (0, 1))
    want = m.nabla_rotary(q, k, rope)
    out = torch.full((B, S, 2, Hh, D), 7.0, dtype=torch.bfloat16, device=DEV)
    # interleaved outputs: their address ranges meet, their elements do not
    qo, ko = (out[:, :, i].transpose(1, 2) for i in (0, 1))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    m.nabla_rotary(q, k, rope, q_out=qo, k_out=ko, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(qo, want[0]) and torch.equal(ko, want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.nabla_rotary(q, k, rope, q_out=qo, k_out=ko)
    qkv.mul_(2)
    graph.replay()
    again = m.nabla_rotary(q, k, rope)
    assert torch.equal(qo, again[0]) and torch.equal(ko, again[1])


# (B, S, Hkv, Hq, D, dim, interleaved, axes, page, dtype, ragged)
APPEND = [
    (1, 1, 1, 0, 64, 64, True, 1, 16, torch.bfloat16, False),
    (64, 1, 8, 32, 128, 128, False, 1, 64, torch.bfloat16, False),
    (3, 77, 2, 6, 128, 126, False, 3, 32, torch.float16, True),
    (4, 300, 3, 3, 64, 18, True, 1, 16, torch.float16, True),
    (2, 200, 5, 0, 128, 128, True, 3, 256, torch.bfloat16, False),
    (2, 40, 7, 5, 128, 6, False, 1, 16, torch.bfloat16, True),
    (2, 40, 7, 0, 64, 62, False, 1, 16, torch.bfloat16, True),
    (3, 33, 9, 2, 128, 108, False, 1, 32, torch.float16, True),
    (2, 21, 5, 3, 64, 40, False, 1, 32, torch.float16, False),
    (5, 9, 1, 4, 64, 64, False, 1, 4096, torch.bfloat16, True),
]


@pytest.mark.parametrize("B,S,Hkv,Hq,D,dim,inter,axes,page,dtype,ragged", APPEND)
def test_cache_append(B, S, Hkv, Hq, D, dim, inter, axes, page, dtype, ragged):
    m = nbl()
    rng = np.random.default_rng(B * 1000 + S)
    dims = None if axes == 1 else (dim - 2 * (dim // 3 // 2 * 2), dim // 3 // 2 * 2, dim // 3 // 2 * 2)
    f = np.concatenate([H.rotary_freqs(d)[0] for d in (dims or (dim,))])
    rope = m.Rope.build(dim, DEV, m.NABLA_ROPE_INTERLEAVED if inter else m.NABLA_ROPE_HALF, dims)
    start = rng.integers(0, 3 * page + 5, B)
    counts = rng.integers(0, S + 1, B) if ragged else np.full(B, S)
    width = int(-(-(start.max() + S) // page)) + 1
    n_pages = B * width + 2
    table = rng.permutation(n_pages)[:B * width].reshape(B, width)
    kc, vc = rnd((n_pages, Hkv, page, D), dtype, 1), rnd((n_pages, Hkv, page, D), dtype, 2)
    k = rnd((B, S, Hkv, D), dtype, 3).transpose(1, 2)
    v = rnd((B, Hkv, S, D), dtype, 4)
    q = rnd((B, Hq, S, D), dtype, 5) if Hq else None
    kc0, vc0 = kc.clone(), vc.clone()
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    status = torch.zeros(64, dtype=torch.int32, device=DEV)
    frame, pos0 = (5, 7), 123456
    qo = m.nabla_cache_append(k, v, kc, vc, ints(table), ints(start), rope=rope, frame=frame, pos0=pos0,
                              counts=ints(counts) if ragged else None, q=q, status=status)
    assert m.nabla_read_device_status(status) == 0
    pos = np.stack([H.grid_positions(S, *frame, axes, first=pos0 + s0) for s0 in start])
    assert torch.equal(vc, torch.tensor(H.append(to64(vc0), to64(v), table, start, counts)).to(dtype).to(DEV))
    kr = H.rotary(to64(k), pos, f, inter, dims)
    ref = H.append(to64(kc0), kr, table, start, counts)
    x = H.append(to64(kc0), to64(k), table, start, counts)
    touched = H.append(np.zeros_like(x), np.ones_like(kr), table, start, counts) > 0
    assert np.array_equal(to64(kc)[~touched], to64(kc0)[~touched])
    assert_rotated(kc, x, ref, dtype, 1.0)
    if Hq:
        assert_rotated(qo, to64(q), H.rotary(to64(q), pos, f, inter, dims), dtype, 1.0)
    # given positions, and no rotation at all
    kc2, vc2 = kc0.clone(), vc0.clone()
    m.nabla_cache_append(k, v, kc2, vc2, ints(table), ints(start), rope=rope, positions=ints(pos),
                         counts=ints(counts) if ragged else None)
    assert torch.equal(kc2, kc) and torch.equal(vc2, vc)
    m.nabla_cache_append(k, v, kc2, vc2, ints(table), ints(start), counts=ints(counts) if ragged else None)
    assert torch.equal(kc2, torch.tensor(H.append(to64(kc0), to64(k), table, start, counts)).to(dtype).to(DEV))


def test_cache_append_skips_bad_pages_and_lengths():
    m = nbl()
    B, S, Hkv, D, page = 4, 20, 2, 64, 16
    kc = torch.zeros((6, Hkv, page, D), dtype=torch.bfloat16, device=DEV)
    vc = torch.zeros_like(kc)
    k, v = rnd((B, Hkv, S, D), torch.bfloat16, 1), rnd((B, Hkv, S, D), torch.bfloat16, 2)
    table = torch.tensor([[0, 1], [2, 6], [-1, 3], [4, 5]], dtype=torch.int32, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    start = torch.tensor([0, 0, 0, 0], dtype=torch.int32, device=DEV)
    m.nabla_cache_append(k, v, kc, vc, table, start, status=status)
    assert m.nabla_read_device_status(status) == m.DEVICE_BAD_PAGE
    assert m.nabla_read_device_status(status) == 0              # cleared by the read
    for page_id, b, first in ((0, 0, 0), (1, 0, 16), (2, 1, 0), (3, 2, 16), (4, 3, 0), (5, 3, 16)):
        n = min(16, S - first)
        assert torch.equal(vc[page_id, :, :n], v[b, :, first:first + n])
        assert torch.equal(kc[page_id, :, :n], k[b, :, first:first + n])
    # a start below 0 and tokens beyond the table: skipped and reported, the rest is stored
    vc.zero_()
    table = torch.tensor([[0, 1], [2, 3], [4, 5], [4, 5]], dtype=torch.int32, device=DEV)
    start = torch.tensor([-3, 25, 0, 0], dtype=torch.int32, device=DEV)
    counts = torch.tensor([20, 20, 20, 0], dtype=torch.int32, device=DEV)
    m.nabla_cache_append(k, v, kc, vc, table, start, counts=counts, status=status)
    assert m.nabla_read_device_status(status) == m.DEVICE_BAD_LENGTH
    assert torch.equal(vc[0, :, :16], v[0, :, 3:19]) and torch.equal(vc[1, :, :1], v[0, :, 19:])
    assert torch.equal(vc[3, :, 9:], v[1, :, :7]) and not vc[2].any()
    assert torch.equal(vc[4], v[2, :, :16]) and torch.equal(vc[5, :, :4], v[2, :, 16:])


@pytest.mark.parametrize("with_q", [False, True])
@pytest.mark.parametrize("dim", [64, 10])
def test_cache_append_reports_counts_outside_the_batch(dim, with_q):
    """counts below 0 or beyond S: reported, the former appends nothing and the latter S tokens."""
    m = nbl()
    B, S, Hkv, Hq, D, page = 4, 20, 2, 3, 64, 16
    rope = m.Rope.build(dim, DEV, m.NABLA_ROPE_HALF)         # 10: turned in shared memory
    k, v, q = (rnd((B, h, S, D), torch.bfloat16, i) for i, h in enumerate((Hkv, Hkv, Hq)))
    q = q if with_q else None
    table = torch.arange(12, dtype=torch.int32, device=DEV).reshape(B, 3)
    start = torch.tensor([3, 0, 5, 28], dtype=torch.int32, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)

    def append(counts, word=status):
        pools = [torch.full((12, Hkv, page, D), 9.0, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
        n = None if counts is None else torch.tensor(counts, dtype=torch.int32, device=DEV)
        qo = m.nabla_cache_append(k, v, *pools, table, start, rope=rope, counts=n, q=q, status=word)
        return pools, qo
    want, wq = append([7, 0, S, S])
    assert m.nabla_read_device_status(status) == 0
    for counts in ([7, -1, S, S], [7, 0, S + 1, S], [7, 0, S, 1 << 30], [7, -(1 << 31), (1 << 31) - 1, S]):
        got, gq = append(counts)
        assert m.nabla_read_device_status(status) == m.DEVICE_BAD_LENGTH, counts
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert gq is None if q is None else torch.equal(gq, wq)
        assert all(torch.equal(a, b) for a, b in zip(append(counts, None)[0], want))     # without a word
    assert m.nabla_read_device_status(status) == 0
    # an earlier error stays: the first one wins
    append([7, S + 1, S, S])
    table[0, 0] = 12
    append([7, 0, S, S])
    assert m.nabla_read_device_status(status) == m.DEVICE_BAD_LENGTH
    append([0, -5, 0, 0])
    assert m.nabla_read_device_status(status) == m.DEVICE_BAD_LENGTH


def test_binding_refuses():
    """What the C side cannot see; nothing is launched."""
    m = nbl()

    def ints(x):
        return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)
    rope, rope3 = m.Rope.build(64, DEV), m.Rope.build(64, DEV, axis_dims=(32, 16, 16))
    q = rnd((2, 4, 24, 64), torch.bfloat16, 1)
    k = rnd((2, 2, 24, 64), torch.bfloat16, 2)

    def rotary(q=q, k=k, rope=rope, **kw):
        m.nabla_rotary(q, k, rope, **kw)
    for kw in (dict(q=None, k=None), dict(q=q[0]), dict(k=k[:, :, :5]), dict(k=k[:1]), dict(k=k.cpu()),
               dict(q=q.transpose(2, 3)), dict(q=q[..., ::2], k=None), dict(rope=m.Rope.build(64, "cpu")),
               dict(rope=rope3, grid=(2, 3, 5)), dict(grid=(24,)), dict(q_out=q[:, :1].clone()[..., :32]),
               dict(k=None, k_out=k.clone()), dict(positions=ints(np.zeros((2, 23, 1)))),
               dict(positions=torch.zeros(2, 24, 1, device=DEV)), dict(rope=rope3, positions=ints(np.zeros((2, 24))))):
        with pytest.raises(ValueError):
            rotary(**kw)
    for kw in (dict(q="q"), dict(rope=3.0), dict(q=q.double()), dict(out_dtype=2)):
        with pytest.raises((TypeError, AttributeError)):
            rotary(**kw)
    for kw in (dict(q_out=q), dict(k=k.half()), dict(q_out=q.half()), dict(q_out=torch.empty_like(q[:, :2])),
               dict(q=k, q_out=(x := torch.empty_like(k)), k_out=x)):
        with pytest.raises(m.NablaError):
            rotary(**kw)

    kc = torch.zeros((6, 2, 16, 64), dtype=torch.bfloat16, device=DEV)
    vc = torch.zeros_like(kc)
    table, start = ints([[0, 1], [2, 3]]), ints([0, 0])

    def append(k=k, v=k, kc=kc, vc=vc, table=table, start=start, **kw):
        m.nabla_cache_append(k, v, kc, vc, table, start, **kw)
    for kw in (dict(v=k[:1]), dict(v=k[:, :, :23]), dict(kc=kc.cpu()), dict(vc=vc[:5]), dict(kc=kc[:, :, ::2], vc=vc[:, :, ::2]),
               dict(table=table[0]), dict(table=table.long()), dict(start=start[:1]), dict(counts=ints([1])),
               dict(positions=ints(np.zeros((2, 24, 1)))), dict(q_out=q.clone(), rope=rope),
               dict(status=torch.zeros(1, dtype=torch.int16, device=DEV)), dict(k=k[..., :32], v=k[..., :32])):
        with pytest.raises(ValueError):
            append(**kw)
    for kw in (dict(k=k[:, :1], v=k[:, :1]), dict(k=k.half(), v=k.half()), dict(vc=kc), dict(q=q), dict(pos0=-1),
               dict(rope=rope3, frame=(0, 0, 4))):
        with pytest.raises(m.NablaError):
            append(**kw)
    assert not kc.any() and not vc.any()


def test_cache_append_past_two_to_the_31_elements():
    """Pages whose element offset does not fit 32 bits."""
    m = nbl()
    Hkv, page, D = 8, 256, 128
    n_pages = (1 << 31) // (Hkv * page * D) + 3
    kc = torch.zeros((n_pages, Hkv, page, D), dtype=torch.bfloat16, device=DEV)
    vc = torch.zeros_like(kc)
    k, v = rnd((1, Hkv, 300, D), torch.bfloat16, 1), rnd((1, Hkv, 300, D), torch.bfloat16, 2)
    table = torch.tensor([[n_pages - 1, n_pages - 2]], dtype=torch.int32, device=DEV)
    start = torch.zeros(1, dtype=torch.int32, device=DEV)
    m.nabla_cache_append(k, v, kc, vc, table, start)
    assert torch.equal(kc[n_pages - 1], k[0, :, :256]) and torch.equal(vc[n_pages - 2, :, :44], v[0, :, 256:])
    assert not kc[:n_pages - 2].any() and not vc[n_pages - 2, :, 44:].any()
