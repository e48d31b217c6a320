"""Paged decode over shared prefixes (attn_paged_decode_shared) on the GPU,
against the definition in 64 bits: softmax over the prefix read through the
group's first block-table row, then the sequence's own tokens.

Error bound.  A score is a sum of d exact products in fp32, off by at most
d 2^-24 of scale sum |q_i k_i| (with d = 128: 2^-17), and so, up to a few
2^-22 of the exponential, is the log of its weight: call that D.  Weights over
the prefix are rounded to bf16 (2^-8 of each, at most) before the product with
V; sums are fp32.  So lse is within 2 D + 2^-18, and an output element within
(2^-8 + 4 D + 2^-15) sum_j p_j |v_j| plus its own rounding to bf16, 2^-8 of
its value.
"""
from __future__ import annotations

import math

import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def cuda():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from tiled_attention_17_b200 import binding
    binding.load()
    return torch, binding


class Batch:
    """Sequences in groups.  groups: [(prefix length, [own tokens of each sequence])]; a negative number is a
    sequence of that (absolute) length that is shorter than the prefix and has its own copy of its tokens;
    a group with prefix None holds sequences outside every group (only first or last)."""

    def __init__(self, torch, groups, Hq, Hkv, d, ps, seed, poison=True, q_scale=1.0):
        g = torch.Generator().manual_seed(seed)
        self.Hq, self.Hkv, self.d, self.ps = Hq, Hkv, d, ps
        rows, lens, self.offsets, self.prefix, self.start, self.leader = [], [], [], [], [], []
        at = 0

        def take(n):
            nonlocal at
            at += n
            return list(range(at - n, at))

        pages = lambda n: -(-n // ps)   # noqa: E731
        for plen, own in groups:
            first = len(rows)
            if plen is not None:
                self.offsets.append(first)
                self.prefix.append(plen)
            p = plen or 0
            lead = take(pages(p))
            for i, n in enumerate(own):
                if n < 0:
                    rows.append(lead if i == 0 else take(pages(-n)))   # the first row lists the prefix whatever its length
                    lens.append(-n)
                    self.start.append(0)
                else:
                    # pages wholly inside the prefix are shared, the rest are its own
                    keep = p // ps
                    rows.append((lead if i == 0 else lead[:keep] + take(pages(p) - keep)) + take(pages(p + n) - pages(p)))
                    lens.append(p + n)
                    self.start.append(p)
                self.leader.append(first)
            if plen is not None:
                last = len(rows)
        self.offsets.append(last if self.offsets else 0)
        self.P = at + 2
        perm = torch.randperm(self.P, generator=g)
        width = max([len(r) for r in rows] + [1]) + 1
        self.table = torch.full((len(rows), width), -1, dtype=torch.int32)
        for s, r in enumerate(rows):
            if r:
                self.table[s, :len(r)] = perm[torch.tensor(r)].to(torch.int32)
        self.lens = torch.tensor(lens, dtype=torch.int32)
        self.S = len(rows)
        self.q = (q_scale * torch.randn(self.S, Hq, d, generator=g)).to(torch.bfloat16)
        fill = float("nan") if poison else 0.0
        self.k = torch.full((self.P, Hkv, ps, d), fill, dtype=torch.bfloat16)
        self.v = torch.full((self.P, Hkv, ps, d), float("inf") if poison else 0.0, dtype=torch.bfloat16)
        # only rows that some sequence reads get numbers; all others keep the poison
        for s in range(self.S):
            for src, lo, hi in self.parts(s):
                if hi > lo:
                    t = torch.arange(lo, hi)
                    pg = self.table[src, t // ps].long()
                    for c in (self.k, self.v):
                        c[pg, :, t % ps] = torch.randn(hi - lo, Hkv, d, generator=g).to(torch.bfloat16)
        for gi, plen in enumerate(self.prefix):   # the whole prefix, if only short sequences read less of it
            if plen and self.offsets[gi + 1] > self.offsets[gi]:
                t = torch.arange(plen)
                pg = self.table[self.offsets[gi], t // ps].long()
                for c in (self.k, self.v):
                    c[pg, :, t % ps] = torch.randn(plen, Hkv, d, generator=g).to(torch.bfloat16)
        self.max_own = max([0] + [n - s for n, s in zip(lens, self.start)])

    def parts(self, s):
        """(block-table row, first token, end) runs of sequence s."""
        n, cut = int(self.lens[s]), self.start[s]
        return [(self.leader[s], 0, cut), (s, cut, n)]

    def run(self, torch, binding, scale=None, stream=None, workspace=None, **over):
        dev = lambda x: x.cuda() if torch.is_tensor(x) else torch.tensor(x, dtype=torch.int32).cuda()   # noqa: E731
        get = lambda name, default: over.get(name, default)   # noqa: E731
        args = [dev(self.q), dev(self.k), dev(self.v), dev(get("table", self.table)), dev(get("lens", self.lens)),
                dev(get("offsets", self.offsets)), dev(get("prefix", self.prefix))]
        max_own = get("max_own", self.max_own)
        if workspace is None:
            need = binding.attn_paged_decode_shared_workspace_size(self.S, len(self.prefix), self.Hq, self.Hkv, self.d)
            workspace = torch.full((need,), 255, dtype=torch.uint8, device="cuda")   # NaN wherever it is not written
        torch.cuda.synchronize()
        o, lse, ws = binding.paged_decode_shared(*args, max_own_len=max_own, scale=scale, workspace=workspace,
                                                 stream=stream)
        torch.cuda.synchronize()
        return o, lse, binding.attn_paged_decode_check(ws)[1]

    def expect(self, torch, scale=None):
        scale = self.d ** -0.5 if scale is None else scale
        G = self.Hq // self.Hkv
        o = torch.zeros(self.S, self.Hq, self.d, dtype=torch.float64)
        tol = torch.zeros_like(o)
        lse = torch.full((self.S, self.Hq), -math.inf, dtype=torch.float64)
        lse_tol = torch.zeros_like(lse)
        for s in range(self.S):
            ks, vs = [], []
            for src, lo, hi in self.parts(s):
                t = torch.arange(lo, hi)
                pg = self.table[src, t // self.ps].long()
                ks.append(self.k[pg, :, t % self.ps])
                vs.append(self.v[pg, :, t % self.ps])
            k, v = torch.cat(ks).double(), torch.cat(vs).double()
            if not len(k):
                continue
            q = self.q[s].double().view(self.Hkv, G, self.d)
            score = scale * torch.einsum("hgd,thd->hgt", q, k)
            size = scale * torch.einsum("hgd,thd->hgt", q.abs(), k.abs()).amax(-1)
            D = (size * self.d * 2.0 ** -24 + 2.0 ** -20)[..., None]
            p = torch.softmax(score, -1)
            val = torch.einsum("hgt,thd->hgd", p, v)
            o[s] = val.reshape(self.Hq, self.d)
            spread = torch.einsum("hgt,thd->hgd", p, v.abs())
            tol[s] = (spread * (2.0 ** -8 + 4 * D + 2.0 ** -15) + val.abs() * 2.0 ** -8).reshape(self.Hq, self.d)
            lse[s] = torch.logsumexp(score, -1).reshape(-1)
            lse_tol[s] = (2 * D[..., 0] + 2.0 ** -18).reshape(-1)
        return o, tol, lse, lse_tol


def check(torch, got, want, what):
    o, lse, flags = got
    ow, tol, lw, ltol = want
    assert flags == 0, (what, flags)
    o, lse = o.double().cpu(), lse.double().cpu()
    assert bool(torch.isfinite(o).all()), what
    over = ((o - ow).abs() - tol).max().item()
    assert over <= 0, f"{what}: output {over:.3e} beyond the bound"
    empty = torch.isneginf(lw)
    assert torch.equal(torch.isneginf(lse), empty), what
    over = torch.where(empty, torch.zeros_like(lw), (lse - lw).abs() - ltol).max().item()
    assert over <= 0, f"{what}: lse {over:.3e} beyond the bound"


CASES = [
    # groups, Hq, Hkv, d, page
    ([(1, [1])], 1, 1, 64, 8),
    ([(128, [5, 9, 1])], 4, 1, 128, 16),
    ([(129, [3, 64, 65, 200])], 8, 2, 128, 16),               # a last tile of one key
    ([(127, [1] * 33)], 8, 1, 64, 32),                        # 264 rows: two blocks, the second nearly empty
    ([(300, [2] * 17)], 16, 2, 64, 64),                       # groups of 8 heads: 136 rows, two row tiles
    ([(515, [33, 1, 7, 20, 2, 30, 15, 8])], 8, 2, 64, 8),
    ([(1000, [70] * 5), (40, [300, 1]), (0, [20, 90]), (700, [1])], 4, 2, 128, 8),
    ([(None, [10, 400]), (256, [17, 18]), (None, [77])], 4, 4, 128, 32),   # sequences outside every group
    ([(200, [-150, 30, -3, 0, -0, 64])], 4, 1, 128, 16),      # short ones, one with no token of its own
    ([(500, []), (64, [0, 0]), (90, [])], 2, 1, 128, 64),     # empty groups; only prefix tokens
    ([(2000, [1] * 3)], 2, 2, 64, 16),
    ([(37, [1 + i % 9 for i in range(300)])], 1, 1, 128, 16), # 300 rows of one head
    ([(4100, [130] * 4)], 16, 8, 128, 64),
    ([(6000, [40] * 70)], 4, 1, 128, 16),                     # 280 rows, split over every SM
    ([(17 + i, [i % 4 + 1] * (i % 3)) for i in range(90)], 4, 2, 64, 8),   # many small groups, some empty
]


@pytest.mark.parametrize("groups,Hq,Hkv,d,ps", CASES)
def test_shared_parity(cuda, groups, Hq, Hkv, d, ps):
    torch, binding = cuda
    b = Batch(torch, groups, Hq, Hkv, d, ps, seed=d + ps + len(groups))
    check(torch, b.run(torch, binding), b.expect(torch), f"{groups} {Hq}/{Hkv} d{d} p{ps}")


@pytest.mark.parametrize("G", [1, 2, 4, 8])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("ps", [8, 16, 32, 64])
def test_shared_shapes(cuda, G, d, ps):
    # every head layout and page size; the prefix ends inside a tile and a page
    torch, binding = cuda
    b = Batch(torch, [(333, [1, 50, 129, 0, 12]), (70, [200, 3])], 2 * G, 2, d, ps, seed=G + d + ps)
    check(torch, b.run(torch, binding), b.expect(torch), f"G{G} d{d} p{ps}")


def test_shared_scales_and_sharp_scores(cuda):
    torch, binding = cuda
    b = Batch(torch, [(300, [40, 2, 90])], 4, 1, 128, 16, seed=5, q_scale=6.0)
    for scale in (0.0, 0.02, 1.0):
        check(torch, b.run(torch, binding, scale), b.expect(torch, scale), f"scale {scale}")


def test_shared_without_groups_or_own_tokens(cuda):
    torch, binding = cuda
    b = Batch(torch, [(None, [40, 0, 300])], 4, 1, 128, 16, seed=6)
    check(torch, b.run(torch, binding), b.expect(torch), "no groups")
    b = Batch(torch, [(160, [0, 0, 0])], 4, 1, 128, 16, seed=7)
    assert b.max_own == 0
    check(torch, b.run(torch, binding), b.expect(torch), "no own tokens")


def test_shared_equals_paged_decode(cuda):
    # the same batch through the ordinary decode: its tables hold every token
    torch, binding = cuda
    b = Batch(torch, [(512, [64, 9, 200]), (96, [1, 2])], 8, 2, 128, 16, seed=9, poison=False)
    o, lse, flags = b.run(torch, binding)
    ref_o, ref_lse, _ = binding.paged_decode(b.q.cuda(), b.k.cuda(), b.v.cuda(), b.table.cuda(), b.lens.cuda())
    ow, tol, lw, ltol = b.expect(torch)
    assert bool(((o - ref_o).double().cpu().abs() <= 2 * tol).all())
    assert bool(((lse - ref_lse).double().cpu().abs() <= 2 * ltol).all())


def test_shared_repeats_bit_for_bit(cuda):
    torch, binding = cuda
    b = Batch(torch, [(3000, [100] * 40), (77, [600, 5])], 8, 2, 128, 16, seed=10)
    o, lse, _ = b.run(torch, binding)
    for _ in range(3):
        o2, lse2, _ = b.run(torch, binding)
        assert torch.equal(o.view(torch.int16), o2.view(torch.int16)) and torch.equal(lse, lse2)


@pytest.mark.parametrize("G,d", [(4, 128), (8, 64), (1, 128), (2, 64)])
def test_shared_many_short_segments(cuda, G, d):
    # hundreds of sequences with one or two tiles of their own behind a prefix cut over every SM: row tiles that run
    # far apart, partials of one and of two steps, the same bits every time
    torch, binding = cuda
    own = [(37 * i) % 260 for i in range(200)]
    b = Batch(torch, [(1500, own[:150]), (90, own[150:])], 4 * G, 4, d, 16, seed=G + d)
    first = b.run(torch, binding)
    check(torch, first, b.expect(torch), f"G{G} d{d}")
    for _ in range(20):
        o, lse, flags = b.run(torch, binding)
        assert flags == 0 and torch.equal(o.view(torch.int16), first[0].view(torch.int16)) and torch.equal(lse, first[1])


@pytest.mark.parametrize("G,d", [(4, 128), (8, 64)])
@pytest.mark.parametrize("groups", [[(2000, [1 + (53 * i) % 700 for i in range(64)])],   # narrow prefixes, then own keys
                                    [(130, [300] * 3), (900, [(91 * i) % 400 for i in range(90)]), (0, [513] * 7)]])
def test_shared_beside_other_copies(cuda, G, d, groups):
    # another stream keeps the memory busy, so K and V tiles arrive late and out of step: nothing may depend on it
    torch, binding = cuda
    b = Batch(torch, groups, 4 * G, 4, d, 16, seed=G * d)
    first = b.run(torch, binding)
    check(torch, first, b.expect(torch), f"G{G} d{d}")
    args = [x.cuda() for x in (b.q, b.k, b.v, b.table, b.lens)] + [
        torch.tensor(x, dtype=torch.int32).cuda() for x in (b.offsets, b.prefix)]
    need = binding.attn_paged_decode_shared_workspace_size(b.S, len(b.prefix), b.Hq, b.Hkv, b.d)
    workspaces = [torch.empty(need, dtype=torch.uint8, device="cuda") for _ in range(4)]
    src, dst = (torch.empty(1 << 28, dtype=torch.uint8, device="cuda") for _ in range(2))
    side = torch.cuda.Stream()
    for i in range(40):
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            dst.copy_(src)
            dst[i::64].copy_(src[i::64])   # scattered
            dst.copy_(src)
        got = [binding.paged_decode_shared(*args, max_own_len=b.max_own, workspace=w) for w in workspaces]
        for o, lse, ws in got:
            assert binding.attn_paged_decode_check(ws)[1] == 0
            assert torch.equal(o.view(torch.int16), first[0].view(torch.int16)) and torch.equal(lse, first[1])
    torch.cuda.synchronize()


def test_shared_large_batches(cuda):
    # thousands of sequences in more than a thousand groups (the plan's windows and searches), whose tables hold
    # whole prefixes: the ordinary decode gives the same result on the same pages
    torch, binding = cuda
    S, ps, Hq, Hkv, d = 6000, 16, 2, 1, 64
    sizes = [(i * 7) % 11 for i in range(1200)]           # some empty
    g = torch.Generator().manual_seed(3)
    pages = torch.randint(0, 5000, (S, 12), generator=g, dtype=torch.int32)
    lens = torch.randint(1, 12 * ps + 1, (S,), generator=g, dtype=torch.int32)
    lens[::97] = 0
    offsets, prefix = [5], []
    for i, n in enumerate(sizes):
        offsets.append(min(offsets[-1] + n, S))
        prefix.append(ps * (i % 9))
        pages[offsets[-2]:offsets[-1], :i % 9] = pages[offsets[-2]:offsets[-2] + 1, :i % 9].clone()
    q = torch.randn(S, Hq, d, generator=g).to(torch.bfloat16).cuda()
    kc, vc = (torch.randn(5000, Hkv, ps, d, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    i32 = lambda x: torch.as_tensor(x, dtype=torch.int32).cuda()   # noqa: E731
    o, lse, ws = binding.paged_decode_shared(q, kc, vc, i32(pages), i32(lens), i32(offsets), i32(prefix))
    ref, ref_lse, _ = binding.paged_decode(q, kc, vc, i32(pages), i32(lens))
    assert binding.attn_paged_decode_check(ws) == (0, 0)
    assert torch.equal(torch.isneginf(lse), torch.isneginf(ref_lse))
    seen = ~torch.isneginf(ref_lse)
    assert (lse - ref_lse)[seen].abs().max().item() <= 1e-3
    # both are within the parity bar of the definition
    assert (o - ref).float().norm().item() <= 1e-2 * ref.float().norm().item()
    assert (o - ref).float().abs().max().item() <= 4e-2


def test_shared_flags_bad_inputs(cuda):
    torch, binding = cuda
    b = Batch(torch, [(100, [20, 30]), (64, [5])], 4, 1, 64, 16, seed=11, poison=False)
    for bad in (-1, b.P, 2 ** 31 - 1, -2 ** 31):
        table = b.table.clone()
        table[0, 1] = bad
        assert b.run(torch, binding, table=table)[2] & binding.TA_DEV_BAD_BLOCK_TABLE
    cap = b.table.shape[1] * b.ps
    for prefix in ([-1, 64], [100, cap + 1], [2 ** 31 - 1, -2 ** 31]):
        o, _, flags = b.run(torch, binding, prefix=prefix, max_own=cap)
        assert flags & binding.TA_DEV_BAD_SEQ_LEN and bool(torch.isfinite(o).all())
    for offsets in ([0, 3, 2], [-1, 2, 3], [0, 2, 9], [2, 1, 0], [-2 ** 31, 2 ** 31 - 1, 0]):
        # no prefix is shared: every sequence reads its own row, which here holds the same tokens or page 0
        o, _, flags = b.run(torch, binding, offsets=offsets, max_own=cap)
        assert flags & binding.TA_DEV_BAD_SEQ_LEN and bool(torch.isfinite(o).all())
    lens = b.lens.clone()
    lens[1] = cap + 5
    assert b.run(torch, binding, lens=lens, max_own=cap)[2] & binding.TA_DEV_BAD_SEQ_LEN
    # more own tokens than announced: cut there
    o, lse, flags = b.run(torch, binding, max_own=20)
    assert flags == binding.TA_DEV_BAD_SEQ_LEN
    cut = b.lens.clone()
    cut[1] = 120
    o2, lse2, flags2 = b.run(torch, binding, lens=cut, max_own=20)
    assert flags2 == 0 and torch.equal(o, o2) and torch.equal(lse, lse2)


def test_shared_graph_streams_and_workspaces(cuda):
    torch, binding = cuda
    b = Batch(torch, [(700, [33, 60, 4, 90]), (130, [9, 9])], 8, 2, 128, 16, seed=13, poison=False)
    want = b.run(torch, binding)
    dev = lambda x: x.cuda() if torch.is_tensor(x) else torch.tensor(x, dtype=torch.int32).cuda()   # noqa: E731
    args = [dev(x) for x in (b.q, b.k, b.v, b.table, b.lens, b.offsets, b.prefix)]
    # two calls at once on two streams, each with its own workspace
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    outs = []
    for _ in range(4):
        for st in (s1, s2.cuda_stream):
            outs.append(binding.paged_decode_shared(*args, max_own_len=b.max_own, stream=st))
    torch.cuda.synchronize()
    for o, lse, _ in outs:
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    # captured and replayed with other lengths and groups
    o, lse = torch.zeros_like(args[0]), torch.zeros(b.S, b.Hq, device="cuda")
    ws = torch.empty_like(outs[0][2])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        binding.paged_decode_shared(*args, max_own_len=b.max_own, workspace=ws, out=o, lse=lse)
    lens = b.lens.clone()
    lens[0] -= 20
    lens[3] = 0
    for lens_now, prefix in ((b.lens, b.prefix), (lens, [640, 130]), (b.lens, b.prefix)):
        args[4].copy_(lens_now)
        args[6].copy_(dev(prefix))
        ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        ref = b.run(torch, binding, lens=lens_now, prefix=prefix)
        assert torch.equal(o, ref[0]) and torch.equal(lse, ref[1])


def test_shared_refusals(cuda):
    torch, binding = cuda
    b = Batch(torch, [(16, [1, 2])], 4, 1, 64, 16, seed=1, poison=False)
    dev = lambda x: x.cuda() if torch.is_tensor(x) else torch.tensor(x, dtype=torch.int32).cuda()   # noqa: E731
    args = [dev(x) for x in (b.q, b.k, b.v, b.table, b.lens, b.offsets, b.prefix)]
    for i, bad in ((0, args[0].float()), (3, args[3].long()), (4, args[4][:1]), (5, args[5][:1]), (6, args[6].cpu()),
                   (1, args[1].transpose(1, 2))):
        with pytest.raises(ValueError):
            binding.paged_decode_shared(*args[:i], bad, *args[i + 1:])
    for over in (dict(out=args[0].float()), dict(out=args[0][:1]), dict(lse=torch.empty(1, 4, device="cuda")),
                 dict(lse=torch.empty(2, 4, dtype=torch.bfloat16, device="cuda")),
                 dict(workspace=torch.empty(1 << 26, dtype=torch.uint8))):
        with pytest.raises(ValueError):
            binding.paged_decode_shared(*args, **over)
    with pytest.raises(binding.TiledAttnError):
        binding.paged_decode_shared(*args, workspace=torch.empty(1024, dtype=torch.uint8, device="cuda"))
    with pytest.raises(binding.TiledAttnError):
        binding.paged_decode_shared(*args, max_own_len=10 ** 6)
    with pytest.raises(binding.TiledAttnError):
        binding.paged_decode_shared(*args, scale=-1.0)
