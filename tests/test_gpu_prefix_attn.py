"""Attention over a shared prefix and own tails (nabla_prefix_attn) against the fp64 oracle.

Tolerances, with A = sum_j softmax_j |v_j| per output element, n keys, eps the 16-bit type's:
  * weights enter the second product rounded to 16 bits: eps / 2 A (fp16 weights below
    2^-14 of the scale are rounded absolutely: n 2^-32 max|v|);
  * a score is a sum of D products, accumulated in f32 and at worst truncated at each step:
    dS = scale D 2^-23 max_j sum|q k|, which changes a normalised weight by at most 2 dS;
  * the second product accumulates 16 keys at a time: (n / 16 + 16) 2^-23 A;
  * exponent argument and ex2 (2^-22), joins of parts: under 1e-5 A;
  * the stored value: eps_o / 2 |O|.
LSE: dS + n 2^-24 (sum of weights) + 1e-5 + 2^-22 |LSE|.
"""
import math

import numpy as np
import pytest
import torch

from oracle import history as H
from parity_lib import nbl

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def to64(t):
    return t.detach().cpu().double().numpy()


def ints(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


class Problem:
    """Inputs of one call: shuffled pages, every cache slot that is no token's NaN."""

    def __init__(self, B, Hq, Hkv, D, Sq, P, tails, page, causal=False, q_len=None, part=None, dtype=BF, seed=0,
                 q_std=1.0, width_extra=1):
        g = torch.Generator().manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.__dict__.update(B=B, Hq=Hq, Hkv=Hkv, D=D, Sq=Sq, P=P, page=page, causal=causal, dtype=dtype)
        self.scale = 1.0 / math.sqrt(D)
        n_pre = -(-P // page)
        width = (max(-(-t // page) for t in tails) + width_extra) if tails is not None else 0
        n_pages = n_pre + B * width + 2
        order = rng.permutation(n_pages)
        self.prefix = order[:n_pre]
        self.tails = tails
        self.table = order[n_pre:n_pre + B * width].reshape(B, width) if tails is not None else None
        used = torch.zeros(n_pages, page, dtype=torch.bool)
        for j in range(P):
            used[self.prefix[j // page], j % page] = True
        for b in range(B if tails is not None else 0):
            for j in range(tails[b]):
                used[self.table[b][j // page], j % page] = True
        self.caches = []
        for _ in range(2):
            c = torch.randn((n_pages, Hkv, page, D), generator=g).to(dtype)
            c[~used.unsqueeze(1).expand(-1, Hkv, -1)] = math.nan
            self.caches.append(c.to(DEV))
        if self.table is not None:          # entries behind a tail's last page are never read
            for b in range(B):
                self.table[b, -(-tails[b] // page):] = -7
        self.q = (torch.randn((B, Hq, Sq, D), generator=g) * q_std).to(dtype).to(DEV)
        self.q_len = q_len
        self.part_o = self.part_lse = None
        if part is not None:
            self.part_o = torch.randn((B, Hq, Sq, D), generator=g).to(part).to(DEV)
            self.part_lse = (torch.randn((B, Hq, Sq), generator=g) * 2 + 3).to(DEV)
            self.part_lse[:, :, ::3] = -math.inf
            self.part_o[:, :, ::3] = math.nan

    def args(self):
        t = self.tails is not None
        return dict(prefix_pages=ints(self.prefix) if self.P else None, prefix_len=self.P,
                    tail_pages=ints(self.table) if t else None, tail_len=ints(self.tails) if t else None,
                    q_len=None if self.q_len is None else ints(self.q_len), causal=self.causal,
                    part_o=self.part_o, part_lse=self.part_lse)

    def run(self, **kw):
        m = nbl()
        need = m.nabla_prefix_workspace_bytes(self.B, self.Hq, self.Hkv, self.Sq, self.D)
        room = torch.full((need + 4096,), 0x5A, dtype=torch.uint8, device=DEV)
        ws = room[:need]
        lse = torch.full((self.B, self.Hq, self.Sq), 77.0, dtype=F32, device=DEV)
        o = torch.full((self.B, self.Hq, self.Sq, self.D), 55.0, dtype=kw.pop("o_dtype", self.dtype), device=DEV)
        a = {**self.args(), "o": o, "lse": lse, "workspace": ws, **kw}
        q = a.pop("q", self.q)
        m.nabla_prefix_attn(q, *self.caches, **a)
        torch.cuda.synchronize()
        assert m.nabla_read_device_status(ws) == 0
        assert (room[need:] == 0x5A).all()
        return a["o"], a["lse"]

    def oracle(self, absolute=False):
        kc, vc = (np.nan_to_num(to64(c)) for c in self.caches)
        n = [self.Sq] * self.B if self.q_len is None else self.q_len
        t = [0] * self.B if self.tails is None else self.tails
        po = None if self.part_o is None else np.nan_to_num(to64(self.part_o))
        return H.prefix_attention(to64(self.q), kc, np.abs(vc) if absolute else vc, self.prefix, self.P, self.table,
                                  t, n, self.causal, self.scale, np.abs(po) if absolute and po is not None else po,
                                  None if po is None else to64(self.part_lse))

    def check(self, o, lse):
        ref, rl = self.oracle()
        A, _ = self.oracle(absolute=True)
        keys = self.P + (max(self.tails) if self.tails is not None else 0)
        kmax = np.abs(np.nan_to_num(to64(self.caches[0]))).max()
        dS = self.scale * self.D * 2.0 ** -23 * np.abs(to64(self.q)).sum(-1, keepdims=True).max() * kmax
        eps = torch.finfo(self.dtype).eps
        live = ~np.isnan(rl)
        got, gl = to64(o), to64(lse)
        # rows that do not exist are left as they were
        assert (got[~live] == 55.0).all() and (gl[~live] == 77.0).all()
        tol = (eps / 2 + 2 * dS + (keys / 16 + 16) * 2.0 ** -23 + 1e-5) * A * 1.01
        tol = tol + torch.finfo(o.dtype).eps / 2 * np.abs(ref) + keys * 2.0 ** -32 * 6 + 2.0 ** -24
        err = np.abs(got - ref)
        assert np.isfinite(got[live]).all()
        assert (err[live] <= tol[live]).all(), f"O: worst {np.max(err[live] / tol[live]):.3f} of the tolerance"
        none = live & np.isneginf(rl)
        assert (got[none] == 0).all() and np.isneginf(gl[none]).all()
        some = live & ~none
        ltol = dS + keys * 2.0 ** -24 + 1e-5 + 2.0 ** -22 * np.abs(rl[some])
        assert (np.abs(gl[some] - rl[some]) <= ltol).all(), "LSE"


CASES = {
    # few rows: the batch's rows share the prefix, tails are parts of their own
    "one": dict(B=1, Hq=1, Hkv=1, D=64, Sq=1, P=1, tails=None, page=16),
    "token": dict(B=4, Hq=8, Hkv=2, D=128, Sq=1, P=300, tails=[0, 1, 129, 300], page=16),
    "token f16": dict(B=3, Hq=6, Hkv=2, D=64, Sq=1, P=1000, tails=[5, 64, 200], page=64, dtype=F16),
    "no tails": dict(B=5, Hq=3, Hkv=3, D=128, Sq=2, P=257, tails=None, page=32),
    "no prefix": dict(B=3, Hq=4, Hkv=4, D=64, Sq=3, P=0, tails=[1, 0, 400], page=128),
    "nothing": dict(B=2, Hq=2, Hkv=1, D=128, Sq=3, P=0, tails=None, page=64),
    "tile edges": dict(B=2, Hq=2, Hkv=2, D=128, Sq=1, P=128, tails=[128, 256], page=128),
    "big pages": dict(B=2, Hq=4, Hkv=1, D=64, Sq=5, P=5000, tails=[700, 4097], page=4096, dtype=F16),
    "drafted": dict(B=6, Hq=4, Hkv=4, D=64, Sq=5, P=200, tails=[5, 6, 130, 140, 9, 260], page=32, causal=True),
    "causal empty rows": dict(B=2, Hq=2, Hkv=2, D=64, Sq=6, P=0, tails=[3, 0], page=16, causal=True),
    "causal into the prefix": dict(B=2, Hq=2, Hkv=2, D=128, Sq=9, P=131, tails=[3, 0], page=16, causal=True),
    "many rows": dict(B=30, Hq=12, Hkv=2, D=128, Sq=3, P=700, tails=list(range(0, 300, 10)), page=64),
    "few rows wide": dict(B=3, Hq=12, Hkv=2, D=128, Sq=3, P=700, tails=[0, 31, 300], page=16),
    "wide tails": dict(B=5, Hq=6, Hkv=2, D=64, Sq=11, P=260, tails=[11, 12, 0, 130, 300], page=64, causal=True,
                       q_len=[11, 5, 0, 11, 3], dtype=F16),
    "wide prefix alone": dict(B=33, Hq=1, Hkv=1, D=128, Sq=1, P=1111, tails=None, page=32),
    "alternate slots": dict(B=2, Hq=2, Hkv=2, D=64, Sq=70, P=900, tails=[70, 333], page=32, causal=True),
    "dual tails": dict(B=3, Hq=10, Hkv=2, D=128, Sq=40, P=300, tails=[400, 0, 77], page=64, q_len=[40, 0, 33]),
    "ragged causal": dict(B=4, Hq=4, Hkv=2, D=128, Sq=60, P=100, tails=[90, 60, 0, 17], page=16, causal=True,
                          q_len=[60, 1, 0, 17], dtype=F16),
    "part": dict(B=3, Hq=4, Hkv=2, D=128, Sq=7, P=200, tails=[0, 50, 300], page=64, part=F32),
    "part bf16": dict(B=2, Hq=2, Hkv=2, D=64, Sq=5, P=0, tails=[0, 20], page=16, part=BF),
    "more rows than join blocks": dict(B=31, Hq=16, Hkv=2, D=64, Sq=21, P=33, tails=[(5 * i) % 48 for i in range(31)], page=32,
                                       part=F32, dtype=F16, q_len=[21 - i % 3 for i in range(31)]),
    # 128 to 255 rows a sequence: items of their own over a short prefix, parts over a long one
    "half a tile": dict(B=3, Hq=4, Hkv=2, D=128, Sq=64, P=200, tails=[64, 300, 70], page=32, causal=True, part=F32),
    "half a tile f16": dict(B=4, Hq=5, Hkv=1, D=64, Sq=31, P=130, tails=[0, 31, 40, 129], page=16, dtype=F16, q_len=[31, 0, 30, 31]),
    "half a tile long": dict(B=3, Hq=4, Hkv=2, D=128, Sq=64, P=4000, tails=[64, 300, 70], page=32, causal=True, part=F32),
    "half a tile alone": dict(B=2, Hq=3, Hkv=3, D=128, Sq=255, P=2100, tails=None, page=128),
    # few-row items alone, more tiles than CTAs
    "many tails": dict(B=40, Hq=16, Hkv=8, D=64, Sq=1, P=0, tails=[(11 * i) % 301 for i in range(40)], page=16),
    "long and short tail": dict(B=2, Hq=4, Hkv=2, D=128, Sq=2, P=77, tails=[15000, 5], page=64, causal=True, dtype=F16),
    # long and few-row items on one kernel's CTAs: fewer and more long items than CTAs, short prefixes
    "shared CTAs": dict(B=20, Hq=60, Hkv=60, D=64, Sq=1, P=700, tails=[3 * i for i in range(20)], page=16),
    "shared CTAs many": dict(B=20, Hq=160, Hkv=160, D=64, Sq=1, P=200, tails=[i % 9 for i in range(20)], page=16, dtype=F16),
    "shared CTAs one tile": dict(B=18, Hq=3, Hkv=1, D=128, Sq=5, P=1, tails=[200 * (i % 3) + 5 for i in range(18)], page=32,
                                 causal=True),
    "shared CTAs long tail": dict(B=17, Hq=1, Hkv=1, D=128, Sq=1, P=130, tails=[0] * 16 + [20000], page=256),
    # many rows of a sequence: prefix and tail in one walk
    "chunk": dict(B=2, Hq=2, Hkv=2, D=128, Sq=300, P=1000, tails=None, page=64),
    "chunk f16": dict(B=1, Hq=3, Hkv=1, D=64, Sq=400, P=333, tails=[500], page=32, dtype=F16),
    "chunk causal": dict(B=2, Hq=4, Hkv=2, D=128, Sq=420, P=130, tails=[420, 611], page=128, causal=True),
    "chunk ragged": dict(B=3, Hq=2, Hkv=2, D=64, Sq=600, P=77, tails=[600, 5, 0], page=16, causal=True,
                         q_len=[511, 5, 0]),
    "chunk empty rows": dict(B=1, Hq=1, Hkv=1, D=64, Sq=700, P=0, tails=[100], page=64, causal=True),
    "chunk nothing": dict(B=1, Hq=2, Hkv=2, D=128, Sq=260, P=0, tails=None, page=64),
    "chunk part": dict(B=2, Hq=2, Hkv=1, D=128, Sq=150, P=513, tails=[10, 0], page=64, part=F32),
    "chunk part f16": dict(B=1, Hq=2, Hkv=2, D=64, Sq=300, P=513, tails=None, page=256, part=F16, dtype=F16),
    # more items than CTAs: whole rounds, then a split remainder
    "rounds": dict(B=2, Hq=40, Hkv=40, D=128, Sq=513, P=300, tails=None, page=64),
    "many sequences": dict(B=300, Hq=2, Hkv=2, D=64, Sq=1, P=40, tails=[(7 * i) % 50 for i in range(300)], page=16),
    "group of 16": dict(B=2, Hq=32, Hkv=2, D=128, Sq=1, P=333, tails=[129, 1], page=32, dtype=F16),
    "group of 17": dict(B=2, Hq=17, Hkv=1, D=64, Sq=1, P=333, tails=[129, 0], page=32),
    "uneven items": dict(B=4, Hq=40, Hkv=40, D=64, Sq=300, P=130, tails=[300, 7, 0, 290], page=64,
                         q_len=[300, 7, 0, 260]),
    "rounds causal": dict(B=3, Hq=18, Hkv=9, D=64, Sq=700, P=60, tails=[700, 350, 720], page=16, causal=True,
                          q_len=[700, 300, 650], part=BF),
}


@pytest.mark.parametrize("name", list(CASES))
def test_prefix_attention(name):
    pr = Problem(**CASES[name], seed=len(name))
    pr.check(*pr.run())


@pytest.mark.parametrize("name", ["token", "part", "chunk part", "chunk causal"])
def test_f32_output_strides_and_in_place_merge(name):
    pr = Problem(**CASES[name], seed=3)
    base, bl = pr.run()
    o32, l32 = pr.run(o_dtype=F32)
    pr.check(o32, l32)
    assert torch.equal(o32.to(pr.dtype), base) and torch.equal(l32, bl)
    # q and o as [B, S, H, D] memory
    qs = pr.q.transpose(1, 2).contiguous().transpose(1, 2)
    os_ = torch.full((pr.B, pr.Sq, pr.Hq, pr.D), 55.0, dtype=pr.dtype, device=DEV).transpose(1, 2)
    o2, l2 = pr.run(q=qs, o=os_)
    assert torch.equal(o2, base) and torch.equal(l2, bl)
    if pr.part_o is not None and pr.part_o.dtype == F32:
        po, pl = pr.part_o.clone(), pr.part_lse.clone()
        o3, l3 = pr.run(o=po, lse=pl, part_o=po, part_lse=pl)
        assert torch.equal(o3, o32) and torch.equal(l3, l32)


@pytest.mark.parametrize("name", ["token", "many rows", "dual tails", "chunk causal", "rounds"])
def test_repeated_calls_give_the_same_bits(name):
    pr = Problem(**CASES[name], seed=4)
    a = pr.run()
    for _ in range(3):
        b = pr.run()
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("name", ["token", "drafted", "causal into the prefix"])
def test_a_wider_page_table_cuts_the_work_another_way(name):
    """Small calls of few rows take a CTA for every tile that the table can hold, wider ones runs: other
    parts, the same result within the tolerance, and each width repeats its own bits."""
    for extra in (0, 2000):
        pr = Problem(**{**CASES[name], "width_extra": extra}, seed=18)
        a, b = pr.run(), pr.run()
        pr.check(*a)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("dtype", [BF, F16])
def test_peaked_and_large_scores(dtype):
    """Maxima that grow along the keys, by far more than one rescale's step, and rows that one key
    dominates."""
    pr = Problem(B=2, Hq=2, Hkv=2, D=64, Sq=3, P=900, tails=[300, 10], page=32, dtype=dtype, seed=7, q_std=6.0)
    k = pr.caches[0]
    for j in range(pr.P):       # scores grow along the prefix
        k[pr.prefix[j // 32], :, j % 32] *= 0.2 + 2.0 * j / pr.P
    pr.check(*pr.run())


def test_infinities_and_nans_of_visible_scores_stay_in_their_rows():
    pr = Problem(B=2, Hq=2, Hkv=2, D=64, Sq=2, P=300, tails=[40, 200], page=16, seed=8)
    base, bl = pr.run()
    q = pr.q.clone()
    q[0, 0, 1, 3] = math.nan
    q[1, 1, 0, 0] = math.inf
    o, l = pr.run(q=q)
    assert torch.isnan(o[0, 0, 1]).all() and torch.isnan(l[0, 0, 1])
    assert torch.isnan(o[1, 1, 0]).all() and torch.isnan(l[1, 1, 0])
    keep = torch.ones_like(l, dtype=torch.bool)
    keep[0, 0, 1] = keep[1, 1, 0] = False
    assert torch.equal(o[keep], base[keep]) and torch.equal(l[keep], bl[keep])


@pytest.mark.parametrize("name", ["one row", "wide", "chunk"])
def test_a_nan_key_reaches_every_row_that_sees_it(name):
    """A NaN score at each place of a tile, one head each: no path of the exponential drops it."""
    B, Hq, Sq = {"one row": (1, 32, 1), "wide": (1, 32, 40), "chunk": (1, 32, 300)}[name]
    pr = Problem(B=B, Hq=Hq, Hkv=32, D=64, Sq=Sq, P=384, tails=None, page=64, seed=10)
    base, bl = pr.run()
    k = pr.caches[0]
    for h in range(0, 32, 2):          # even heads; the others keep their results
        for j0 in (128, 192):
            j = j0 + 32 * (h & 3) // 2 + h // 2 + 16 * (j0 == 192)
            k[pr.prefix[j // 64], h, j % 64, 5] = math.nan if j0 == 128 else -math.inf
    o, l = pr.run()
    assert torch.isnan(o[:, 0::2]).all() and torch.isnan(l[:, 0::2]).all()
    assert torch.equal(o[:, 1::2], base[:, 1::2]) and torch.equal(l[:, 1::2], bl[:, 1::2])


@pytest.mark.parametrize("Sq", [5, 33, 300])
def test_keys_that_no_query_sees_may_hold_anything(Sq):
    """Causal, one query of each sequence: the keys behind it are masked."""
    pr = Problem(B=2, Hq=2, Hkv=2, D=64, Sq=Sq, P=100, tails=[Sq, Sq + 40], page=16, causal=True, seed=13)
    base, bl = pr.run()
    for b in range(2):
        j = pr.tails[b] - 1                     # the last query's own key: no other row sees it
        pr.caches[0][pr.table[b][j // 16], :, j % 16] = math.nan
    o, l = pr.run()
    assert torch.equal(o[:, :, :-1], base[:, :, :-1]) and torch.equal(l[:, :, :-1], bl[:, :, :-1])
    assert torch.isnan(o[:, :, -1]).all() and torch.isnan(l[:, :, -1]).all()


PADDED = {
    "few rows": dict(B=3, Hq=4, Hkv=2, D=64, Sq=5, P=300, tails=[5, 140, 9], page=16, q_len=[5, 1, 0], causal=True),
    "batch of rows": dict(B=6, Hq=6, Hkv=2, D=128, Sq=11, P=700, tails=None, page=32, q_len=[11, 5, 0, 11, 3, 1]),
    "alternate slots": dict(B=2, Hq=2, Hkv=2, D=64, Sq=70, P=900, tails=[300, 333], page=32, q_len=[70, 33], dtype=F16),
    "dual tails": dict(B=3, Hq=10, Hkv=2, D=128, Sq=40, P=300, tails=[400, 0, 300], page=64, q_len=[40, 0, 21]),
    "chunk": dict(B=2, Hq=2, Hkv=2, D=128, Sq=500, P=1000, tails=[300, 0], page=64, q_len=[500, 277]),
    "chunk causal": dict(B=3, Hq=2, Hkv=2, D=64, Sq=600, P=520, tails=[600, 45, 0], page=16, causal=True,
                         q_len=[511, 45, 0], dtype=F16),
}


@pytest.mark.parametrize("name", list(PADDED))
@pytest.mark.parametrize("fill", [math.nan, -math.inf, 3e4])
def test_queries_behind_a_sequences_own_may_hold_anything(name, fill):
    """The same bits whatever a padded batch holds behind q_len, and those rows are left alone."""
    pr = Problem(**PADDED[name], seed=17)
    for b, n in enumerate(pr.q_len):
        pr.q[b, :, n:] = 0.0
    base, bl = pr.run()
    pr.check(base, bl)
    for b, n in enumerate(pr.q_len):
        pr.q[b, :, n:] = fill
    o, l = pr.run()
    assert torch.equal(o, base) and torch.equal(l, bl)


@pytest.mark.parametrize("name", ["dual tails", "chunk", "chunk causal"])
def test_bad_pages_leave_the_other_sequences_alone(name):
    m = nbl()
    pr = Problem(**CASES[name], seed=14)
    base, bl = pr.run()
    a = pr.args()
    ws = torch.empty(m.nabla_prefix_workspace_bytes(pr.B, pr.Hq, pr.Hkv, pr.Sq, pr.D), dtype=torch.uint8, device=DEV)
    if pr.table is not None:
        table = pr.table.copy()
        table[0, 0] = pr.caches[0].shape[0] + 5
        o = torch.full_like(base, 55.0)
        m.nabla_prefix_attn(pr.q, *pr.caches, **{**a, "tail_pages": ints(table)}, o=o, workspace=ws)
        assert m.nabla_read_device_status(ws) == m.DEVICE_BAD_PAGE
        assert torch.equal(o[1:], base[1:])
    pages = pr.prefix.copy()
    pages[1] = -2
    m.nabla_prefix_attn(pr.q, *pr.caches, **{**a, "prefix_pages": ints(pages)}, workspace=ws)
    assert m.nabla_read_device_status(ws) == m.DEVICE_BAD_PAGE
    o, l = pr.run()
    assert torch.equal(o, base) and torch.equal(l, bl)


def test_binding_refuses():
    """What the C side cannot see; nothing is launched."""
    m = nbl()
    pr = Problem(**CASES["token"], seed=15)
    k, v = pr.caches
    a = pr.args()

    def call(q=pr.q, k=k, v=v, **kw):
        m.nabla_prefix_attn(q, k, v, **{**a, **kw})
    wrong = [dict(q=pr.q[0]), dict(q=pr.q.cpu()), dict(k=k.cpu()), dict(k=k[:, :, ::2]), dict(v=v[:-1]), dict(v=v.half()),
             dict(q=pr.q[..., :64]), dict(q=pr.q.transpose(2, 3)), dict(prefix_pages=a["prefix_pages"].long()),
             dict(prefix_pages=a["prefix_pages"][:2]), dict(tail_pages=a["tail_pages"][:2]),
             dict(tail_pages=a["tail_pages"][0]), dict(tail_len=a["tail_len"][:3]), dict(tail_len=a["tail_len"].cpu()),
             dict(q_len=ints([1, 1])), dict(o=pr.q[:, :, :, :64].clone()), dict(lse=torch.zeros(4, 8, 2, device=DEV)),
             dict(lse=torch.zeros(4, 8, 1, device=DEV, dtype=F16)), dict(workspace=torch.zeros(64, device=DEV)),
             dict(part_o=pr.q.clone(), part_lse=torch.zeros(4, 8, device=DEV))]
    for kw in wrong:
        with pytest.raises(ValueError):
            call(**kw)
    for kw in (dict(q=pr.q.double()), dict(q=[1.0]), dict(o_dtype="f32")):
        with pytest.raises(TypeError):
            call(**kw)
    for kw in (dict(q=pr.q.half()), dict(tail_len=None), dict(prefix_pages=None), dict(scale=-1.0), dict(o=pr.q),
               dict(part_o=pr.q.clone())):
        with pytest.raises(m.NablaError):
            call(**kw)
    with pytest.raises(m.NablaError):
        call(workspace=torch.zeros(256, dtype=torch.uint8, device=DEV))


def test_bad_pages_and_lengths_are_reported():
    m = nbl()
    pr = Problem(**CASES["token"], seed=9)
    base, bl = pr.run()

    def status(**kw):
        ws = torch.empty(m.nabla_prefix_workspace_bytes(pr.B, pr.Hq, pr.Hkv, pr.Sq, pr.D), dtype=torch.uint8, device=DEV)
        o, lse = torch.empty_like(pr.q), torch.empty(pr.B, pr.Hq, pr.Sq, device=DEV)
        m.nabla_prefix_attn(pr.q, *pr.caches, **{**pr.args(), **kw}, o=o, lse=lse, workspace=ws)
        return m.nabla_read_device_status(ws), o, lse
    assert status()[0] == 0
    table = pr.table.copy()
    table[2, 0] = pr.caches[0].shape[0]
    code, o, _ = status(tail_pages=ints(table))
    assert code == m.DEVICE_BAD_PAGE
    for b in (0, 1, 3):                             # the other sequences are not concerned
        assert torch.equal(o[b], base[b])
    table[2, 0] = -1
    assert status(tail_pages=ints(table))[0] == m.DEVICE_BAD_PAGE
    assert status(prefix_pages=ints(np.full_like(pr.prefix, 1 << 30)))[0] == m.DEVICE_BAD_PAGE
    code, o, lse = status(tail_len=ints([-5, 1, 129, 300]))   # as a length of 0
    assert code == m.DEVICE_BAD_LENGTH and torch.equal(o, base) and torch.equal(lse, bl)
    full = ints(np.where(pr.table < 0, 0, pr.table))
    assert status(tail_len=ints([0, 1, 129, 1 << 30]), tail_pages=full)[0] == m.DEVICE_BAD_LENGTH
    assert status(q_len=ints([1, 1, 2, 1]))[0] == m.DEVICE_BAD_LENGTH
    assert status(q_len=ints([1, -1, 1, 1]))[0] == m.DEVICE_BAD_LENGTH


@pytest.mark.parametrize("warp", [0, 1, 2, 3])
@pytest.mark.parametrize("name", ["token", "many tails"])
def test_a_bad_page_of_any_warp_is_reported(name, warp):
    """Items of few rows, a CTA a tile and in runs: a warp reads every fourth group of 16 keys, here
    a page.  The one bad page is some warp's, the workspace holds what an earlier call left."""
    m = nbl()
    pr = Problem(**CASES[name], seed=16)
    b = int(np.argmax(pr.tails))
    assert pr.page == 16 and pr.tails[b] > 64
    need = m.nabla_prefix_workspace_bytes(pr.B, pr.Hq, pr.Hkv, pr.Sq, pr.D)
    base = pr.run()[0]
    table = pr.table.copy()
    table[b, warp] = pr.caches[0].shape[0]
    bad = {**pr.args(), "tail_pages": ints(table)}
    for left in (0x00, 0x5A, 0xFF) * 10:
        ws = torch.full((need,), left, dtype=torch.uint8, device=DEV)
        o, _ = m.nabla_prefix_attn(pr.q, *pr.caches, **bad, workspace=ws)
        assert m.nabla_read_device_status(ws) == m.DEVICE_BAD_PAGE
        others = [i for i in range(pr.B) if i != b]
        assert torch.equal(o[others], base[others])
        ws.fill_(left)
        m.nabla_prefix_attn(pr.q, *pr.caches, **pr.args(), workspace=ws)
        assert m.nabla_read_device_status(ws) == 0


def test_graph_follows_the_lengths_and_side_streams():
    """A captured call replayed with other lengths, and two calls at once with workspaces of their
    own."""
    m = nbl()
    pr = Problem(B=3, Hq=4, Hkv=2, D=128, Sq=1, P=300, tails=[10, 200, 400], page=16, seed=11)
    a = pr.args()
    o, lse = torch.empty_like(pr.q), torch.empty(3, 4, 1, device=DEV)
    ws = torch.empty(m.nabla_prefix_workspace_bytes(3, 4, 2, 1, 128), dtype=torch.uint8, device=DEV)
    m.nabla_prefix_attn(pr.q, *pr.caches, **a, o=o, lse=lse, workspace=ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.nabla_prefix_attn(pr.q, *pr.caches, **a, o=o, lse=lse, workspace=ws)
    for tails in ([10, 200, 400], [1, 0, 399], [9, 150, 16]):
        a["tail_len"].copy_(ints(tails))
        graph.replay()
        want, wl = m.nabla_prefix_attn(pr.q, *pr.caches, **a, lse=torch.empty_like(lse))
        assert torch.equal(o, want) and torch.equal(lse, wl)
        assert m.nabla_read_device_status(ws) == 0
    big = Problem(**CASES["chunk"], seed=12)
    bo, _ = big.run()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for s in (s1, s2):
        s.wait_stream(torch.cuda.current_stream())
    outs = []
    for _ in range(4):
        outs.append((m.nabla_prefix_attn(big.q, *big.caches, **big.args(), stream=s1)[0],
                     m.nabla_prefix_attn(pr.q, *pr.caches, **a, stream=s2)[0]))
    torch.cuda.synchronize()
    for x, y in outs:
        assert torch.equal(x, bo) and torch.equal(y, want)


def test_pages_past_two_to_the_31_elements():
    m = nbl()
    Hkv, page, D = 8, 256, 128
    n_pages = (1 << 31) // (Hkv * page * D) + 3
    kc = torch.zeros((n_pages, Hkv, page, D), dtype=BF, device=DEV)
    vc = torch.zeros_like(kc)
    g = torch.Generator(device=DEV).manual_seed(1)
    for i in (n_pages - 1, n_pages - 2, 0, 1):
        kc[i].normal_(generator=g)
        vc[i].normal_(generator=g)
    q = torch.randn((2, 8, 1, D), generator=g, device=DEV).to(BF)
    o1, _ = m.nabla_prefix_attn(q, kc, vc, ints([n_pages - 1, n_pages - 2]), 400)
    small_k, small_v = kc[[n_pages - 2, n_pages - 1]].contiguous(), vc[[n_pages - 2, n_pages - 1]].contiguous()
    o2, _ = m.nabla_prefix_attn(q, small_k, small_v, ints([1, 0]), 400)
    assert torch.equal(o1, o2)


def test_continuing_a_clip():
    """The operators together, as a user chains them: rotated Q and K of new frames, sparse
    attention inside them, attention to the history in the cache merged into it, and the new
    frames appended; against dense attention over the history and the kept blocks."""
    import oracle
    m = nbl()
    B, Hh, T, Hg, W, D, hist = 2, 2, 2, 16, 16, 64, 3
    S, frame, page = T * Hg * W, Hg * W, 64
    P = hist * frame
    sh = m.Shape(B, Hh, T, Hg, W, D)
    rope = m.Rope.build(D, DEV, m.NABLA_ROPE_INTERLEAVED, (24, 20, 20))
    g = torch.Generator().manual_seed(5)
    rnd = lambda *s: torch.randn(s, generator=g).to(BF).to(DEV)  # noqa: E731
    nat = m.NABLA_LAYOUT_NATURAL
    n_pages = P // page + 4
    kc = torch.full((n_pages, Hh, page, D), math.nan, dtype=BF, device=DEV)
    vc = torch.full_like(kc, math.nan)
    pages = ints(np.random.default_rng(1).permutation(n_pages)[:P // page])
    hk, hv = rnd(1, Hh, P, D), rnd(1, Hh, P, D)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    m.nabla_cache_append(hk, hv, kc, vc, pages.reshape(1, -1), ints([0]), rope=rope, frame=(Hg, W), status=status)
    assert m.nabla_read_device_status(status) == 0
    q, k, v = rnd(B, Hh, S, D), rnd(B, Hh, S, D), rnd(B, Hh, S, D)
    qr, kr = m.nabla_rotary(q, k, rope, grid=(T, Hg, W), origin=(hist, 0, 0))
    bits, *_ = m.nabla_build_mask(qr, kr, sh, 0.6, layout=nat)
    lse = torch.empty(B, Hh, S, dtype=F32, device=DEV)
    o, lse = m.nabla_attn_fwd(qr, kr, v, bits, sh, o_dtype=m.NABLA_F32, lse=lse, layout=nat)
    out, ol = m.nabla_prefix_attn(qr, kc, vc, pages, P, part_o=o, part_lse=lse, lse=torch.empty_like(lse))
    # the oracle: every key of the history, and the chunk's kept blocks (block order)
    perm = oracle.fractal_permutation(T, Hg, W, 8)
    mask = oracle.unpack_mask_bits(bits.cpu().numpy().view(np.uint32), sh.nb)
    f = np.concatenate([H.rotary_freqs(d)[0] for d in (24, 20, 20)])
    hkr = H.rotary(to64(hk), H.grid_positions(P, Hg, W, 3)[None], f, True, (24, 20, 20))
    hkr = torch.tensor(hkr).to(BF).double().numpy()[0]         # stored in bf16
    block = np.empty(S, dtype=np.int64)                         # block of every natural token
    order = np.array([((t * (Hg // 8) + h // 8) * (W // 8) + w // 8) for t in range(T) for h in range(Hg) for w in range(W)])
    block[:] = order
    assert len(perm) == S
    for b in range(B):
        for h in range(Hh):
            keys = np.concatenate((hkr[h], to64(kr)[b, h]))
            vals = np.concatenate((to64(hv)[0, h], to64(v)[b, h]))
            s = to64(qr)[b, h] @ keys.T / math.sqrt(D)
            keep = np.concatenate((np.ones((S, P), dtype=bool), mask[b, h][block][:, block]), 1)
            s = np.where(keep, s, -np.inf)
            e = np.exp(s - s.max(1, keepdims=True))
            pr = e / e.sum(1, keepdims=True)
            ref, A = pr @ vals, pr @ np.abs(vals)
            # two bf16 roundings of weights at worst, the output's, and f32 sums
            tol = (2.0 ** -8 * 1.1 + 1e-3) * A + 2.0 ** -8 * np.abs(ref)
            assert (np.abs(to64(out)[b, h] - ref) <= tol).all()
            rl = s.max(1) + np.log(e.sum(1))
            # the sparse forward sums its weights after rounding them: 2^-8 at worst
            assert (np.abs(to64(ol)[b, h] - rl) <= 2.0 ** -8 * 1.1).all()
