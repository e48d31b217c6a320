"""The position, cache and shared-prefix calls run together as they are used: a
serving step (append with rotation, then each of the attention calls over the
pages) and a training step (rotation, attention, its backward, the rotation's
backward), against the definition in 64 bits from the unrotated inputs.

Error bounds.  A rotated query or key carries one rounding to bf16 (2^-8 of the
element at most), so a score is off by at most 2 x 2^-8 scale sum |q_i k_i|
beyond the attention's own error, and a weight relatively by twice that (its
own score's and the normaliser's).  Those roundings of d elements and N keys are
independent; the tests take the attention's parity bar (relative L2 5e-3 and, for
gradients, 5e-3) and add the rounding's root-mean-square share: 2^-9 of each
element and at most three products deep, 3 x 2^-9 = 6e-3.
"""
from __future__ import annotations

import math

import pytest

pytestmark = pytest.mark.gpu
REL = 5e-3 + 3 * 2.0 ** -9


@pytest.fixture(scope="module")
def cuda():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from tiled_attention_17_b200 import binding
    binding.load()
    return torch, binding


def rel(torch, got, want):
    return ((got.double().cpu() - want).norm() / want.norm()).item()


def turn(torch, x, pos, inv, interleaved, amp):
    """[..., tokens, d] in 64 bits (differentiable)."""
    r = 2 * inv.numel()
    i = torch.arange(r // 2)
    ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + r // 2)
    angle = pos.double()[:, None] * inv
    c, s = amp * torch.cos(angle), amp * torch.sin(angle)
    a, b = x[..., ia], x[..., ib]
    return x.index_copy(-1, ia, a * c - b * s).index_copy(-1, ib, a * s + b * c)


def attend(torch, q, k, v, scale):
    """q [Hq, n, d] at the end of k, v [Hkv, N, d]: bottom-right causal attention."""
    G = q.shape[0] // k.shape[0]
    s = scale * q @ k.repeat_interleave(G, 0).transpose(1, 2)
    n, N = s.shape[1:]
    s = s.masked_fill(torch.arange(N)[None] > torch.arange(n)[:, None] + N - n, -math.inf)
    return torch.softmax(s, -1) @ v.repeat_interleave(G, 0)


@pytest.mark.parametrize("interleaved,d,rotary", [(False, 128, 128), (True, 64, 32)])
def test_serving_run(cuda, interleaved, d, rotary):
    # a shared prefix enters the cache once, then each sequence's prompt, then two decode steps
    torch, binding = cuda
    from tiled_attention_17_b200 import rope
    Hq, Hkv, ps, shared, prompts = 8, 2, 16, 208, [40, 1, 97, 16]
    S, steps = len(prompts), 2
    inv, amp = rope.frequencies(rotary, scaling={"type": "yarn", "factor": 4.0, "trained_length": 128})
    inv64 = inv.cpu()
    g = torch.Generator().manual_seed(d)
    tokens = [torch.randn(shared + n + steps, Hq + 2 * Hkv, d, generator=g).to(torch.bfloat16) for n in prompts]
    for t in tokens[1:]:
        t[:shared] = tokens[0][:shared]
    scale = d ** -0.5
    width = -(-(shared + max(prompts) + steps) // ps)
    keep = shared // ps
    P = keep + S * (width - keep) + 1
    perm = torch.randperm(P, generator=g).to(torch.int32)
    table = torch.full((S, width), -1, dtype=torch.int32)
    for s in range(S):
        table[s, :keep] = perm[:keep]
        table[s, keep:] = perm[keep + s * (width - keep):keep + (s + 1) * (width - keep)]
    table = table.cuda()
    kc = torch.zeros(P, Hkv, ps, d, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")   # noqa: E731

    def split(x):
        return x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]

    def append(rows, lens, cu):
        q, k, v = split(rows.cuda())
        return binding.paged_append(k, v, kc, vc, table, lens, cu, q=q, inv_freq=inv, interleaved=interleaved,
                                    amplitude=amp)

    def want(s, lo, hi):
        x = tokens[s][:hi].double()
        q, k, v = (y.transpose(0, 1) for y in split(x))
        pos = torch.arange(hi)
        q, k = (turn(torch, y, pos, inv64, interleaved, amp) for y in (q, k))
        return attend(torch, q[:, lo:], k, v, scale).transpose(0, 1)

    # the shared prefix, as the first sequence's tokens (the others bring none)
    cu = i32([0] + [shared] * S)
    lens = i32([shared] + [0] * (S - 1))
    q = append(tokens[0][:shared], lens, cu)
    o, _ = binding.paged_prefill(q, kc, vc, table, cu, lens, shared, True)
    assert rel(torch, o, want(0, 0, shared)) <= REL
    # every sequence's own prompt
    ends = [shared + n for n in prompts]
    offs = [sum(prompts[:i]) for i in range(S + 1)]
    cu, lens = i32(offs), i32(ends)
    q = append(torch.cat([t[shared:e] for t, e in zip(tokens, ends)]), lens, cu)
    o, _ = binding.paged_prefill(q, kc, vc, table, cu, lens, max(prompts), True)
    assert rel(torch, o, torch.cat([want(s, shared, ends[s]) for s in range(S)])) <= REL
    # decode steps: one token each, through the shared prefix and through the ordinary call
    groups, prefix = i32([0, S]), i32([shared])
    ws = None
    for step in range(steps):
        lens = i32([e + step + 1 for e in ends])
        q = append(torch.stack([t[e + step] for t, e in zip(tokens, ends)]), lens, None)
        o, lse, ws = binding.paged_decode_shared(q, kc, vc, table, lens, groups, prefix,
                                                 max_own_len=max(prompts) + steps, workspace=ws)
        assert binding.attn_paged_decode_check(ws) == (0, 0)
        ref = torch.cat([want(s, ends[s] + step, ends[s] + step + 1) for s in range(S)])
        assert rel(torch, o, ref) <= REL
        plain, plain_lse, _ = binding.paged_decode(q, kc, vc, table, lens)
        assert rel(torch, plain, ref) <= REL
        assert (lse - plain_lse).abs().max().item() <= 1e-3
    assert binding.ta_device_status(True) == (0, 0)


def test_training_run(cuda):
    # heads of a fused projection -> rotation -> causal attention -> gradients back into the fused rows
    torch, binding = cuda
    from tiled_attention_17_b200 import rope
    B, N, Hq, Hkv, d, rotary = 2, 150, 4, 2, 64, 48
    inv, amp = rope.frequencies(rotary, scaling={"type": "linear", "factor": 2.0})
    inv64 = inv.cpu()
    g = torch.Generator().manual_seed(5)
    qkv = torch.randn(B, N, Hq + 2 * Hkv, d, generator=g).to(torch.bfloat16)
    dout = torch.randn(B, Hq, N, d, generator=g).to(torch.bfloat16)
    rows = qkv.cuda()
    q = binding.rope(rows[:, :, :Hq].transpose(1, 2), inv, amplitude=amp)
    k = binding.rope(rows[:, :, Hq:Hq + Hkv].transpose(1, 2), inv, amplitude=amp)
    v = binding.rope(rows[:, :, Hq + Hkv:].transpose(1, 2), None)   # only laid out head by head
    o, lse = binding.attention(q, k, v, True)
    dq, dk, dv = binding.attention_backward(q, k, v, o, lse, dout.cuda(), True)
    grad = torch.empty_like(rows)
    heads = grad.transpose(1, 2)
    binding.rope_backward(dq, inv, amplitude=amp, out=heads[:, :Hq])
    binding.rope_backward(dk, inv, amplitude=amp, out=heads[:, Hq:Hq + Hkv])
    binding.rope_backward(dv, None, out=heads[:, Hq + Hkv:])
    x = qkv.double().requires_grad_(True)
    pos = torch.arange(N)

    def forward(x):
        out = []
        for b in range(B):
            h = x[b].transpose(0, 1)
            qr = turn(torch, h[:Hq], pos, inv64, False, amp)
            kr = turn(torch, h[Hq:Hq + Hkv], pos, inv64, False, amp)
            out.append(attend(torch, qr, kr, h[Hq + Hkv:], d ** -0.5))
        return torch.stack(out)

    ref = forward(x)
    assert rel(torch, o, ref.detach()) <= REL
    (ref * dout.double()).sum().backward()
    for part in (slice(0, Hq), slice(Hq, Hq + Hkv), slice(Hq + Hkv, None)):
        assert rel(torch, grad[:, :, part], x.grad[:, :, part]) <= REL
    # and against differences of the loss along a direction
    step = torch.randn(x.shape, generator=g, dtype=torch.float64)
    step /= step.norm()
    with torch.no_grad():
        eps = 1e-4
        diff = ((forward(x + eps * step) - forward(x - eps * step)) * dout.double()).sum() / (2 * eps)
    got = (grad.double().cpu() * step).sum()
    # |<grad error, step>| <= |grad error| |step|
    assert abs(got - diff) <= REL * x.grad.norm() + 1e-6 * abs(diff)
