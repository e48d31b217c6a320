"""Scores that are not finite in the shared-prefix decode: a NaN or +inf score
makes its row NaN (output and lse), as softmax of it is; a score of -inf is a
weight of 0; every other row keeps its bits.  A row all of whose scores are
-inf is one without visible keys: O = 0, lse = -inf.  And scores near the ends
of fp32's range under a scale that brings them back.

Error bound of the finite rows that meet a -inf score: that of
test_gpu_shared.py, over the keys whose scores are finite.
"""
from __future__ import annotations

import math

import pytest

from test_gpu_shared import Batch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def cuda():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from tiled_attention_17_b200 import binding
    binding.load()
    return torch, binding


def expect(torch, b, scale=None):
    """Definition in 64 bits: (o, tolerance, lse, tolerance); NaN where a score is NaN or +inf."""
    scale = b.d ** -0.5 if scale is None else scale
    G = b.Hq // b.Hkv
    o = torch.zeros(b.S, b.Hq, b.d, dtype=torch.float64)
    tol, lse = torch.zeros_like(o), torch.full((b.S, b.Hq), -math.inf, dtype=torch.float64)
    lse_tol = torch.zeros_like(lse)
    for s in range(b.S):
        ks, vs = [], []
        for src, lo, hi in b.parts(s):
            t = torch.arange(lo, hi)
            pg = b.table[src, t // b.ps].long()
            ks.append(b.k[pg, :, t % b.ps])
            vs.append(b.v[pg, :, t % b.ps])
        k, v = torch.cat(ks).double(), torch.cat(vs).double()
        if not len(k):
            continue
        q = b.q[s].double().view(b.Hkv, G, b.d)
        score = scale * torch.einsum("hgd,thd->hgt", q, k)
        size = scale * torch.einsum("hgd,thd->hgt", q.abs(), k.abs())
        D = (torch.where(torch.isfinite(score), size, torch.zeros_like(size)).amax(-1) * b.d * 2.0 ** -24 + 2.0 ** -20)[..., None]
        none = torch.isneginf(score).all(-1, keepdim=True)
        p = torch.where(none, torch.zeros_like(score), torch.softmax(score, -1))
        val = torch.einsum("hgt,thd->hgd", p, v)
        o[s] = val.reshape(b.Hq, b.d)
        tol[s] = (torch.einsum("hgt,thd->hgd", p, v.abs()) * (2.0 ** -8 + 4 * D + 2.0 ** -15) + val.abs() * 2.0 ** -8).reshape(b.Hq, b.d)
        bad = torch.isnan(p).any(-1)
        row = torch.logsumexp(score, -1)
        lse[s] = torch.where(bad, torch.full_like(row, math.nan), row).reshape(-1)
        lse_tol[s] = (2 * D[..., 0] + 2.0 ** -18).reshape(-1)
    return o, tol, lse, lse_tol


def compare(torch, got, want, clean, touched, what):
    """touched [S, Hq]: rows that meet the planted value; the others keep the clean run's bits."""
    o, lse, flags = got
    ow, tol, lw, ltol = want
    assert flags == 0, (what, flags)
    same = ~touched.cuda()
    assert torch.equal(o[same].view(torch.int16), clean[0][same].view(torch.int16)), f"{what}: another row's output changed"
    assert torch.equal(lse[same], clean[1][same]), f"{what}: another row's lse changed"
    o, lse = o.double().cpu(), lse.double().cpu()
    nan = torch.isnan(lw)
    assert torch.equal(torch.isnan(lse), nan), f"{what}: lse is NaN in other rows than expected"
    assert torch.equal(torch.isnan(o), nan[..., None].expand_as(o)), f"{what}: output is NaN in other rows than expected"
    assert torch.equal(torch.isneginf(lse), torch.isneginf(lw)), what
    seen = ~nan & ~torch.isneginf(lw)
    assert bool(((o - ow).abs() <= tol)[~nan].all()), f"{what}: output beyond the bound"
    assert bool(((lse - lw).abs() <= ltol)[seen].all()), f"{what}: lse beyond the bound"


LAYOUTS = [
    # groups, Hq, Hkv, d, page: prefixes of one and of two row tiles, own keys of one to several steps
    ([(600, [70, 3, 300, 0]), (200, [40, 9])], 8, 2, 128, 16),
    ([(600, [70, 3, 300, 0]), (200, [40, 9])], 8, 1, 64, 8),
    ([(700, [20] * 40 + [150, 260]), (None, [513])], 8, 2, 128, 32),
    ([(700, [20] * 20 + [150, 260]), (None, [513])], 16, 2, 64, 64),
    ([(257, [130, 1])], 2, 2, 128, 16),
]


@pytest.mark.parametrize("groups,Hq,Hkv,d,ps", LAYOUTS)
@pytest.mark.parametrize("value", ["nan", "inf", "-inf"])
@pytest.mark.parametrize("where", ["prefix", "own"])
def test_one_key(cuda, groups, Hq, Hkv, d, ps, value, where):
    # one element of one key: NaN scores in every row that meets it, or (infinite) +inf and -inf by the query's sign
    torch, binding = cuda
    b = Batch(torch, groups, Hq, Hkv, d, ps, seed=Hq + d + ps)
    assert bool((b.q != 0).all())
    clean = b.run(torch, binding)
    s = 0 if where == "prefix" else max(range(b.S), key=lambda i: int(b.lens[i]) - b.start[i])
    cut = b.start[s]
    for t in ([0, 5, cut // 2, cut - 1] if where == "prefix" else [cut, (cut + int(b.lens[s])) // 2, int(b.lens[s]) - 1]):
        src = b.leader[s] if where == "prefix" else s
        page, row, head, column = int(b.table[src, t // ps]), t % ps, Hkv - 1, d // 2 + 3
        kept = b.k[page, head, row, column].clone()
        b.k[page, head, row, column] = float(value)
        touched = torch.zeros(b.S, Hq, dtype=torch.bool)
        who = [i for i in range(b.S) if b.leader[i] == b.leader[s] and b.start[i] == cut] if where == "prefix" else [s]
        touched[who, head * (Hq // Hkv):] = True
        want = expect(torch, b)
        assert value != "nan" or torch.equal(torch.isnan(want[2]), touched)
        compare(torch, b.run(torch, binding), want, clean, touched, f"{value} in {where} key {t}")
        b.k[page, head, row, column] = kept


@pytest.mark.parametrize("groups,Hq,Hkv,d,ps", LAYOUTS)
def test_overflowing_score(cuda, groups, Hq, Hkv, d, ps):
    # finite queries and keys whose product passes the range of fp32
    torch, binding = cuda
    b = Batch(torch, groups, Hq, Hkv, d, ps, seed=Hq + d + ps + 1)
    clean = b.run(torch, binding)
    page, row = int(b.table[0, 100 // ps]), 100 % ps
    b.k[page, 0, row] = torch.where(b.q[0, 0] > 0, 3e38, -3e38).to(torch.bfloat16)   # the first row's score overflows
    touched = torch.zeros(b.S, Hq, dtype=torch.bool)
    touched[[i for i in range(b.S) if b.leader[i] == 0 and b.start[i] == b.start[0]], :Hq // Hkv] = True
    o, lse, flags = b.run(torch, binding)
    assert flags == 0 and bool(torch.isnan(o[0, 0]).all()) and bool(torch.isnan(lse[0, 0]))
    same = ~touched.cuda()
    assert torch.equal(o[same].view(torch.int16), clean[0][same].view(torch.int16)) and torch.equal(lse[same], clean[1][same])


@pytest.mark.parametrize("groups,Hq,Hkv,d,ps", LAYOUTS)
@pytest.mark.parametrize("value", ["nan", "inf"])
def test_one_query(cuda, groups, Hq, Hkv, d, ps, value):
    torch, binding = cuda
    b = Batch(torch, groups, Hq, Hkv, d, ps, seed=Hq + d + ps + 2)
    clean = b.run(torch, binding)
    b.q[1, Hq - 1, 7] = float(value)   # inf: scores of both signs, so +inf among them
    touched = torch.zeros(b.S, Hq, dtype=torch.bool)
    touched[1, Hq - 1] = True
    want = expect(torch, b)
    assert torch.equal(torch.isnan(want[2]), touched)
    compare(torch, b.run(torch, binding), want, clean, touched, f"{value} in a query")


def test_one_value(cuda):
    # a NaN in V reaches its column of the rows that meet it, and their lse not at all
    torch, binding = cuda
    for groups, Hq, Hkv, d, ps in LAYOUTS:
        b = Batch(torch, groups, Hq, Hkv, d, ps, seed=Hq + d + ps + 3)
        clean = b.run(torch, binding)
        b.v[int(b.table[0, 200 // ps]), 0, 200 % ps, 11] = float("nan")
        o, lse, flags = b.run(torch, binding)
        nan = torch.zeros(b.S, Hq, d, dtype=torch.bool)
        nan[[i for i in range(b.S) if b.leader[i] == 0 and b.start[i] == b.start[0]], :Hq // Hkv, 11] = True
        nan = nan.cuda()
        assert flags == 0 and torch.equal(lse, clean[1]) and torch.equal(torch.isnan(o), nan)
        assert torch.equal(o[~nan].view(torch.int16), clean[0][~nan].view(torch.int16))


def test_all_scores_minus_infinity(cuda):
    # infinite keys throughout: rows whose query is negative there see no key at all, the others are NaN
    torch, binding = cuda
    for Hq, Hkv, d, ps in ((8, 2, 128, 16), (8, 1, 64, 8)):
        b = Batch(torch, [(140, [3, 0]), (None, [9])], Hq, Hkv, d, ps, seed=d)
        clean = b.run(torch, binding)
        b.k[..., 5] = math.inf
        touched = torch.ones(b.S, Hq, dtype=torch.bool)
        want = expect(torch, b)
        assert bool(torch.isnan(want[2]).any()) and bool(torch.isneginf(want[2]).any())
        compare(torch, b.run(torch, binding), want, clean, touched, "all keys")


@pytest.mark.parametrize("Hq,Hkv,d,ps", [(8, 2, 128, 16), (8, 1, 64, 8)])
def test_small_scales_and_large_scores(cuda, Hq, Hkv, d, ps):
    # the scale may be far below the smallest difference of scores: 0 weighs all keys alike however large they are,
    # and a tiny one is applied as it is
    torch, binding = cuda
    b = Batch(torch, [(300, [40, 2, 90]), (None, [33])], Hq, Hkv, d, ps, seed=d + 1)
    b.q, b.k = b.q * 2.0 ** 50, b.k * 2.0 ** 50
    for scale in (0.0, d ** -0.5 * 2.0 ** -100, d ** -0.5 * 2.0 ** -103):
        want = expect(torch, b, scale)
        assert bool(torch.isfinite(want[2]).all())
        nothing = torch.ones(b.S, Hq, dtype=torch.bool)
        got = b.run(torch, binding, scale)
        compare(torch, got, want, got, nothing, f"scale {scale}")
