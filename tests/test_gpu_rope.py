"""Rotary positions (attn_rope) and the paged append (attn_paged_append) on the
GPU, against the definition in 64 bits.

Error bound of one rotated element.  The fraction of a turn is exact in fp64 up
to 2^-51 of the angle; as an angle of at most pi it is rounded twice to fp32
(2^-24 each: under 2^-21.4 radians together); the hardware's sine and cosine are
within 2^-21.1 on that range; the amplitude's product, the two products and the
sum round in fp32 (2^-24 each).  Together under 2^-19.9, taken as 2^-19.5, of
amp (|a| + |b|), plus 2^-51 |angle| amp (|a| + |b|).  Then one rounding to
bf16, at most 2^-8 of the value.  Copied elements are equal bit for bit.
"""
from __future__ import annotations

import numpy as np
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


def turned(torch, x, pos, inv_freq, interleaved, amp, sign=1.0):
    """(value, bound) of the definition for x [..., tokens, d] (fp64, CPU) at pos [..., tokens]."""
    x = x.double()
    r = 2 * inv_freq.numel()
    angle = pos.double()[..., None] * inv_freq
    i = torch.arange(r // 2)
    ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + r // 2)
    a, b = x[..., ia], x[..., ib]
    c, s = torch.cos(angle), sign * torch.sin(angle)
    y, tol = x.clone(), torch.zeros_like(x)
    y[..., ia], y[..., ib] = amp * (a * c - b * s), amp * (a * s + b * c)
    t = abs(amp) * (a.abs() + b.abs()) * (2.0 ** -19.5 + 2.0 ** -51 * angle.abs())
    tol[..., ia] = t + y[..., ia].abs() * 2.0 ** -8
    tol[..., ib] = t + y[..., ib].abs() * 2.0 ** -8
    return y, tol


def check(got, want, tol, what):
    err = (got.double().cpu() - want).abs()
    worst = (err - tol).max().item() if err.numel() else 0.0
    assert worst <= 0, f"{what}: {worst:.3e} beyond the bound"


def normal(torch, *shape, seed=0):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g).to(torch.bfloat16)


def freqs(torch, r, scaling=None):
    from tiled_attention_17_b200 import rope
    return rope.frequencies(r, scaling=scaling, device="cpu")


ROPE_CASES = [
    # B, H, N, d, rotary, interleaved, positions
    (1, 1, 1, 64, 64, False, "none"),
    (1, 1, 1, 128, 16, True, "one"),
    (2, 3, 5, 128, 128, False, "each"),
    (1, 7, 33, 64, 32, True, "one"),
    (3, 5, 129, 128, 48, False, "far"),
    (2, 8, 257, 128, 64, True, "each"),
    (1, 64, 70, 64, 16, False, "negative"),
    (4, 1, 1021, 128, 112, True, "far"),
    (2, 13, 511, 64, 48, False, "none"),
    (1, 40, 2050, 128, 128, True, "one"),
    (2, 3, 9, 128, 0, False, "none"),
]


def positions_of(torch, kind, B, N, seed):
    g = torch.Generator().manual_seed(seed)
    if kind == "none":
        return None, torch.arange(N).expand(B, N)
    if kind == "one":
        p = torch.randint(0, 100000, (N,), generator=g, dtype=torch.int32)
        return p, p.expand(B, N)
    if kind == "far":
        p = torch.randint(2 ** 31 - 2 ** 20, 2 ** 31 - 1, (B, N), generator=g, dtype=torch.int32)
    elif kind == "negative":
        p = torch.randint(-5000, 5000, (B, N), generator=g, dtype=torch.int32)
    else:
        p = torch.randint(0, 300000, (B, N), generator=g, dtype=torch.int32)
    return p, p


@pytest.mark.parametrize("B,H,N,d,r,interleaved,kind", ROPE_CASES)
@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("layout", ["heads", "fused"])
def test_rope_parity(cuda, B, H, N, d, r, interleaved, kind, inverse, layout):
    torch, binding = cuda
    x = normal(torch, B, N, H + 2, d, seed=N + d + r)
    inv, amp = freqs(torch, r, {"type": "yarn", "factor": 4.0, "trained_length": 512}) if r > 2 else (None, 1.0)
    p_dev, p = positions_of(torch, kind, B, N, seed=N)
    view = x.cuda()[:, :, 1:H + 1].transpose(1, 2)
    if layout == "heads":
        view = view.contiguous()
    f = binding.rope_backward if inverse else binding.rope
    got = f(view, None if inv is None else inv.cuda(), None if p_dev is None else p_dev.cuda(), interleaved=interleaved,
            amplitude=amp)
    assert got.is_contiguous() and got.shape == (B, H, N, d)
    xs = x[:, :, 1:H + 1].transpose(1, 2)
    if r == 0:
        assert torch.equal(got.cpu().view(torch.int16), xs.contiguous().view(torch.int16))
        return
    want, tol = turned(torch, xs, p[:, None], inv, interleaved, amp, -1.0 if inverse else 1.0)
    check(got, want, tol, (B, H, N, d, r))
    assert torch.equal(got.cpu()[..., r:].view(torch.int16), xs[..., r:].contiguous().view(torch.int16))


def test_rope_writes_only_its_rows_and_runs_in_place(cuda):
    torch, binding = cuda
    x = normal(torch, 2, 31, 6, 128, seed=4).cuda()
    inv, _ = freqs(torch, 64)
    inv = inv.cuda()
    out = torch.full((2, 31, 9, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    heads = x[:, :, :6].transpose(1, 2)
    binding.rope(heads, inv, out=out[:, :, 2:8].transpose(1, 2))
    assert bool((out[:, :, :2] == 7).all()) and bool((out[:, :, 8:] == 7).all())
    want = binding.rope(heads, inv)
    assert torch.equal(out[:, :, 2:8].transpose(1, 2), want)
    same = x.clone()
    binding.rope(same.transpose(1, 2), inv, out=same.transpose(1, 2))
    assert torch.equal(same.transpose(1, 2), want)


def test_rope_copies_what_it_does_not_turn(cuda):
    torch, binding = cuda
    x = normal(torch, 1, 4, 8, 128, seed=5)
    x[..., 64:] = torch.tensor([float("nan"), float("inf"), -float("inf"), -0.0] * 16)
    got = binding.rope(x.cuda(), freqs(torch, 64)[0].cuda(), amplitude=1.5)
    assert torch.equal(got.cpu()[..., 64:].view(torch.int16), x[..., 64:].view(torch.int16))
    assert bool(torch.isfinite(got[..., :64]).all())


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_gradient(cuda, interleaved):
    # L = sum(g * rope(x)): the formula's gradient by autograd in 64 bits, and
    # central differences of L (linear in x: exact up to rounding)
    torch, binding = cuda
    B, H, N, d, r, amp = 2, 3, 17, 64, 48, 1.25
    x, g = normal(torch, B, H, N, d, seed=1), normal(torch, B, H, N, d, seed=2)
    inv, _ = freqs(torch, r)
    pos = torch.randint(0, 5000, (B, N), generator=torch.Generator().manual_seed(3), dtype=torch.int32)
    dx = binding.rope_backward(g.cuda(), inv.cuda(), pos.cuda(), interleaved=interleaved, amplitude=amp).cpu().double()
    xr = x.double().requires_grad_(True)
    i = torch.arange(r // 2)
    ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + r // 2)
    angle = pos.double()[:, None, :, None] * inv

    def forward(z):
        y = torch.zeros_like(z) + z
        a, b = z[..., ia], z[..., ib]
        y = y.index_copy(-1, ia, amp * (a * torch.cos(angle) - b * torch.sin(angle)))
        return y.index_copy(-1, ib, amp * (a * torch.sin(angle) + b * torch.cos(angle)))

    (forward(xr) * g.double()).sum().backward()
    _, tol = turned(torch, g, pos[:, None], inv, interleaved, amp, -1.0)
    check(dx, xr.grad, tol, "formula")
    v = torch.randn(B, H, N, d, dtype=torch.float64, generator=torch.Generator().manual_seed(9))
    loss = lambda z: (forward(z) * g.double()).sum()   # noqa: E731
    diff = (loss(x.double() + v) - loss(x.double() - v)) / 2
    # every element of dx may be off by its own tolerance
    assert abs((dx * v).sum() - diff) <= (tol * v.abs()).sum() + 1e-9 * abs(diff)


def test_rope_graph_and_stream(cuda):
    torch, binding = cuda
    x = normal(torch, 1, 5, 300, 128, seed=6).cuda()
    inv = freqs(torch, 128)[0].cuda()
    want = binding.rope(x, inv)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for s in (side, side.cuda_stream):
        got = binding.rope(x, inv, stream=s)
        side.synchronize()
        assert torch.equal(got, want)
    out = torch.zeros_like(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        binding.rope(x, inv, out=out)
    x.copy_(x.flip(2))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, binding.rope(x, inv))


def test_rope_refusals(cuda):
    torch, binding = cuda
    x = torch.zeros(1, 2, 4, 64, dtype=torch.bfloat16, device="cuda")
    inv = torch.ones(32, dtype=torch.float64, device="cuda")
    with pytest.raises(ValueError):
        binding.rope(x.float(), inv)
    with pytest.raises(ValueError):
        binding.rope(x[0], inv)
    with pytest.raises(ValueError):
        binding.rope(x, inv.float())
    with pytest.raises(ValueError):
        binding.rope(x, inv, torch.arange(4, device="cuda"))               # int64
    with pytest.raises(ValueError):
        binding.rope(x, inv, torch.arange(5, device="cuda", dtype=torch.int32))
    with pytest.raises(ValueError):
        binding.rope(x, inv, out=torch.empty(1, 2, 4, 128, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(binding.TiledAttnError):
        binding.rope(x, torch.ones(20, dtype=torch.float64, device="cuda"))   # rotary_dim 40
    with pytest.raises(binding.TiledAttnError):
        binding.rope(x, inv, out=x.view(1, 4, 2, 64).transpose(1, 2))         # in place with other strides


# ---------------------------------------------------------------------------
# Paged append
# ---------------------------------------------------------------------------

class Batch:
    """A ragged batch of new tokens and a cache with room for them."""

    def __init__(self, torch, new, lens, Hq, Hkv, d, ps, r, seed, before=0, behind=0, extra_table=2):
        g = torch.Generator().manual_seed(seed)
        S = len(new)
        pages = [-(-n // ps) for n in lens]
        P = sum(pages) + 3
        perm = torch.randperm(P, generator=g)
        self.table = torch.full((S, max(pages + [1]) + extra_table), -1, dtype=torch.int32)
        at = 0
        for s, n in enumerate(pages):
            self.table[s, :n] = perm[at:at + n]
            at += n
        self.new, self.lens, self.ps, self.r = new, lens, ps, r
        self.cu = torch.tensor([before + sum(new[:i]) for i in range(S + 1)], dtype=torch.int32)
        self.seq_lens = torch.tensor(lens, dtype=torch.int32)
        T = before + sum(new) + behind
        qkv = torch.randn(T, Hq + 2 * Hkv, d, generator=g).to(torch.bfloat16)
        self.qkv, self.Hq, self.Hkv, self.d, self.T = qkv, Hq, Hkv, d, T
        self.kc = torch.randn(P, Hkv, ps, d, generator=g).to(torch.bfloat16)
        self.vc = torch.randn(P, Hkv, ps, d, generator=g).to(torch.bfloat16)

    def split(self, t):
        Hq, Hkv = self.Hq, self.Hkv
        return t[:, :Hq], t[:, Hq:Hq + Hkv], t[:, Hq + Hkv:]

    def run(self, torch, binding, inv, amp=1.0, interleaved=False, positions=None, use_cu=True, with_q=True,
            table=None, seq_lens=None, cu=None):
        dev = lambda t: None if t is None else t.cuda()   # noqa: E731
        q, k, v = self.split(self.qkv.cuda())
        q_out = torch.full((self.T, self.Hq, self.d), 5.0, dtype=torch.bfloat16, device="cuda") if with_q else None
        kc, vc = self.kc.cuda(), self.vc.cuda()
        binding.ta_device_status(True)
        got = binding.paged_append(k, v, kc, vc, dev(self.table if table is None else table),
                                   dev(self.seq_lens if seq_lens is None else seq_lens),
                                   cu_seqlens=dev(self.cu if cu is None else cu) if use_cu else None,
                                   q=q if with_q else None, q_out=q_out, inv_freq=dev(inv), positions=dev(positions),
                                   interleaved=interleaved, amplitude=amp)
        torch.cuda.synchronize()
        flags = binding.ta_device_status(True)[1]
        return (got.cpu() if with_q else None), kc.cpu(), vc.cpu(), flags

    def tokens(self):
        """(row, sequence, slot) of every new token."""
        at = int(self.cu[0])
        for s, n in enumerate(self.new):
            for i in range(n):
                yield at, s, self.lens[s] - n + i
                at += 1

    def expect(self, torch, inv, amp, interleaved, positions=None, skip=(), skip_page=()):
        q, k, v = self.split(self.qkv)
        q_want = torch.full((self.T, self.Hq, self.d), 5.0, dtype=torch.float64)
        kc, vc = self.kc.double(), self.vc.clone()
        q_tol, k_tol = torch.zeros_like(q_want), torch.zeros_like(kc)
        rows = [x for x in self.tokens() if x[0] not in skip]
        if rows:
            row, seq, slot = (torch.tensor(x) for x in zip(*rows))
            pos = slot if positions is None else positions[row].long()
            page, off = self.table[seq, slot // self.ps].long(), slot % self.ps
            keep = torch.tensor([x[0] not in skip_page for x in rows])
            if inv is None:
                q_want[row] = q[row].double()
                kc[page[keep], :, off[keep]] = k[row][keep].double()
            else:
                y, t = turned(torch, q[row].transpose(0, 1), pos, inv, interleaved, amp)
                q_want[row], q_tol[row] = y.transpose(0, 1), t.transpose(0, 1)
                y, t = turned(torch, k[row].transpose(0, 1), pos, inv, interleaved, amp)
                kc[page[keep], :, off[keep]] = y.transpose(0, 1)[keep]
                k_tol[page[keep], :, off[keep]] = t.transpose(0, 1)[keep]
            vc[page[keep], :, off[keep]] = v[row][keep]
        return q_want, q_tol, kc, k_tol, vc


def check_batch(torch, b, got, want, with_q=True):
    q, kc, vc, _ = got
    q_want, q_tol, k_want, k_tol, v_want = want
    if with_q:
        check(q, q_want, q_tol, "q")       # a tolerance of 0 where nothing may be written
    check(kc, k_want, k_tol, "k cache")    # every other slot of the cache stays as it was
    assert torch.equal(vc.view(torch.int16), v_want.view(torch.int16))


APPEND_CASES = [
    # new tokens, lengths after, Hq, Hkv, d, page, rotary, interleaved, rows before, rows behind
    ([1], [1], 1, 1, 64, 8, 64, False, 0, 0),
    ([7, 0, 1, 40], [7, 90, 64, 101], 4, 2, 128, 16, 128, False, 0, 0),
    ([3, 65, 128, 0, 0, 2], [3, 65, 300, 0, 17, 1000], 8, 1, 64, 8, 32, True, 0, 9),
    ([16, 16], [16, 32], 2, 2, 128, 16, 64, False, 4, 3),              # exactly whole pages
    ([250, 1], [250, 64], 16, 4, 128, 64, 48, True, 1, 40),
    ([1] * 40, list(range(1, 41)), 8, 8, 64, 32, 16, False, 0, 1),
    ([0, 0], [5, 0], 2, 1, 128, 8, 128, False, 2, 3),                  # rows, but none belongs to a sequence
]


@pytest.mark.parametrize("new,lens,Hq,Hkv,d,ps,r,interleaved,before,behind", APPEND_CASES)
def test_append_parity(cuda, new, lens, Hq, Hkv, d, ps, r, interleaved, before, behind):
    torch, binding = cuda
    b = Batch(torch, new, lens, Hq, Hkv, d, ps, r, seed=sum(lens) + ps, before=before, behind=behind)
    inv, amp = freqs(torch, r, {"type": "wavelength", "factor": 8.0, "trained_length": 256})
    for with_q in (True, False):
        got = b.run(torch, binding, inv, 1.125, interleaved, with_q=with_q)
        assert got[3] == 0
        check_batch(torch, b, got, b.expect(torch, inv, 1.125, interleaved), with_q)


def test_append_without_rotation_and_with_positions(cuda):
    torch, binding = cuda
    b = Batch(torch, [5, 30], [50, 30], 4, 2, 128, 16, 0, seed=8)
    got = b.run(torch, binding, None)
    check_batch(torch, b, got, b.expect(torch, None, 1.0, False))
    inv, _ = freqs(torch, 64)
    pos = torch.randint(-100, 2 ** 30, (35,), dtype=torch.int32, generator=torch.Generator().manual_seed(2))
    got = b.run(torch, binding, inv, positions=pos)
    check_batch(torch, b, got, b.expect(torch, inv, 1.0, False, positions=pos))


@pytest.mark.parametrize("S", [1, 64, 300])
def test_append_one_token_each(cuda, S):
    # cu_seqlens None; length 0 marks an empty place of the batch
    torch, binding = cuda
    lens = [(i * 37) % 200 for i in range(S)]
    new = [1 if n else 0 for n in lens]
    b = Batch(torch, [1] * S, lens, 4, 2, 64, 16, 64, seed=S)
    inv, _ = freqs(torch, 64)
    got = b.run(torch, binding, inv, use_cu=False)
    assert got[3] == 0
    check_batch(torch, b, got, b.expect(torch, inv, 1.0, False, skip={i for i in range(S) if not new[i]}))


@pytest.mark.parametrize("S", [1023, 1024, 1025, 2500, 4096])
def test_append_many_sequences(cuda, S):
    # more sequence ends than the staged table holds; empty sequences among them
    torch, binding = cuda
    new = [(i * 7919) % 5 if i % 3 else 0 for i in range(S)]
    lens = [n + (i * 31) % 20 for i, n in enumerate(new)]
    b = Batch(torch, new, lens, 1, 1, 64, 8, 16, seed=S, before=3, behind=2, extra_table=0)
    inv, _ = freqs(torch, 16)
    got = b.run(torch, binding, inv)
    assert got[3] == 0
    check_batch(torch, b, got, b.expect(torch, inv, 1.0, False))


def test_append_flags_bad_tables_and_lengths(cuda):
    torch, binding = cuda
    b = Batch(torch, [4, 6, 3], [20, 38, 3], 2, 1, 64, 16, 64, seed=3)
    inv, _ = freqs(torch, 64)
    P = b.kc.shape[0]
    rows = list(b.tokens())
    for bad in (-1, P, 2 ** 31 - 1, -2 ** 31):
        table = b.table.clone()
        table[1, 2] = bad   # slots 32..37 of sequence 1: its six new tokens
        got = b.run(torch, binding, inv, table=table)
        assert got[3] == binding.TA_DEV_BAD_BLOCK_TABLE
        lost = {row for row, s, slot in rows if s == 1}
        check_batch(torch, b, got, b.expect(torch, inv, 1.0, False, skip_page=lost))
    cap = b.table.shape[1] * 16
    for bad in (-5, 5, cap + 1, 2 ** 31 - 1, -2 ** 31):   # below the new tokens, or past the table
        seq_lens = b.seq_lens.clone()
        seq_lens[1] = bad
        got = b.run(torch, binding, inv, seq_lens=seq_lens)
        assert got[3] == binding.TA_DEV_BAD_SEQ_LEN
        check_batch(torch, b, got, b.expect(torch, inv, 1.0, False, skip={row for row, s, _ in rows if s == 1}))
    cu = b.cu.clone()
    cu[3] = b.T + 9   # runs past the rows: the last sequence's tokens write nothing
    got = b.run(torch, binding, inv, cu=cu)
    assert got[3] == binding.TA_DEV_BAD_SEQ_LEN
    check_batch(torch, b, got, b.expect(torch, inv, 1.0, False, skip={r for r, s, _ in rows if s == 2}))


def test_append_in_place_queries_graph_and_stream(cuda):
    torch, binding = cuda
    b = Batch(torch, [9, 20], [40, 20], 4, 2, 128, 16, 128, seed=12)
    inv, _ = freqs(torch, 128)
    want = b.run(torch, binding, inv)
    q, k, v = (x.contiguous().cuda() for x in b.split(b.qkv))
    kc, vc = b.kc.cuda(), b.vc.cuda()
    table, lens, cu, f = b.table.cuda(), b.seq_lens.cuda(), b.cu.cuda(), inv.cuda()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = binding.paged_append(k, v, kc, vc, table, lens, cu, q=q, q_out=q, inv_freq=f, stream=side)
    side.synchronize()
    assert got is q and torch.equal(q.cpu(), want[0]) and torch.equal(kc.cpu(), want[1])
    # captured: the replay reads the lengths and rows of its own time
    q, k, v = (x.contiguous().cuda() for x in b.split(b.qkv))
    kc, vc = b.kc.cuda(), b.vc.cuda()
    out = torch.full_like(q, 5.0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        binding.paged_append(k, v, kc, vc, table, lens, cu, q=q, q_out=out, inv_freq=f)
    kc.copy_(b.kc)
    lens.copy_(torch.tensor([30, 20], dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    b.lens = [30, 20]
    b.seq_lens = torch.tensor(b.lens, dtype=torch.int32)
    check_batch(torch, b, (out.cpu(), kc.cpu(), vc.cpu(), 0), b.expect(torch, inv, 1.0, False))


def test_append_refusals(cuda):
    torch, binding = cuda
    b = Batch(torch, [2], [2], 2, 1, 64, 8, 64, seed=1)
    q, k, v = b.split(b.qkv.cuda())
    kc, vc, table, lens, cu = b.kc.cuda(), b.vc.cuda(), b.table.cuda(), b.seq_lens.cuda(), b.cu.cuda()
    for call in (lambda: binding.paged_append(k, v, kc, vc, table.long(), lens, cu),
                 lambda: binding.paged_append(k, v, kc, vc[:, :, :4], table, lens, cu),
                 lambda: binding.paged_append(k, v, kc, vc, table, lens, cu[:1]),
                 lambda: binding.paged_append(k, v[:1], kc, vc, table, lens, cu),
                 lambda: binding.paged_append(k, v, kc.float(), vc, table, lens, cu),
                 lambda: binding.paged_append(k, v, kc, vc, table, lens, cu, q=q, q_out=torch.empty_like(q[:, :, :32])),
                 lambda: binding.paged_append(k, v, kc, vc, table, lens.cpu(), cu)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(binding.TiledAttnError):
        binding.paged_append(k, v, kc, vc, table, lens)   # two rows, one sequence, no offsets
