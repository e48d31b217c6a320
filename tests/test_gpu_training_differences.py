"""The gradients of the training run - rotation, causal attention, its backward,
the rotation's backward into the fused rows - against central differences of
the loss, along directions in which the loss moves: the 64-bit gradient of the
query, key and value rows, each by itself.

Along the unit vector of a part's gradient the derivative is that gradient's
norm |g|.  The kernels' gradient e off by |e| <= REL |g| (the bound of
test_gpu_position_cache_run.py) is off by at most as much along it, so the
tolerance is REL = 1.1% of the value compared: a missing gradient, a flipped sign
or one of a few per cent too much is seen.  The differences themselves, of step
1e-4 along a unit vector in 64 bits, are good to well under 1e-6 of it.
"""
from __future__ import annotations

import pytest

from test_gpu_position_cache_run import REL, attend, turn

pytestmark = pytest.mark.gpu

B, N, HQ, HKV, D, ROTARY = 2, 150, 4, 2, 64, 48
PARTS = {"q": slice(0, HQ), "k": slice(HQ, HQ + HKV), "v": slice(HQ + HKV, None)}


def reference(torch, qkv, dout, inv, amp):
    """(loss of fused rows, its gradient) in 64 bits."""
    pos = torch.arange(N)

    def loss(x):
        total = 0.0
        for b in range(B):
            h = x[b].transpose(0, 1)
            q, k = (turn(torch, h[PARTS[p]], pos, inv, False, amp) for p in "qk")
            total = total + (attend(torch, q, k, h[PARTS["v"]], D ** -0.5) * dout[b].double()).sum()
        return total

    x = qkv.double().requires_grad_(True)
    loss(x).backward()
    return loss, x.grad


def check_along_gradients(torch, grad, loss, x, want):
    for part in PARTS.values():
        step = torch.zeros_like(want)
        step[:, :, part] = want[:, :, part] / want[:, :, part].norm()
        with torch.no_grad():
            eps = 1e-4
            diff = (loss(x + eps * step) - loss(x - eps * step)) / (2 * eps)
        tol = REL * want[:, :, part].norm()
        assert tol < 0.02 * abs(diff)   # a wrong gradient cannot hide in it
        assert abs((grad * step).sum() - diff) <= tol + 1e-6 * abs(diff)


def inputs(torch):
    from tiled_attention_17_b200 import rope
    inv, amp = rope.frequencies(ROTARY, scaling={"type": "linear", "factor": 2.0}, device="cpu")
    g = torch.Generator().manual_seed(5)
    qkv = torch.randn(B, N, HQ + 2 * HKV, D, generator=g).to(torch.bfloat16)
    dout = torch.randn(B, HQ, N, D, generator=g).to(torch.bfloat16)
    return qkv, dout, inv, amp


def test_training_gradients_along_themselves():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from tiled_attention_17_b200 import binding
    qkv, dout, inv, amp = inputs(torch)
    rows, freq = qkv.cuda(), inv.cuda()
    q, k = (binding.rope(rows[:, :, PARTS[p]].transpose(1, 2), freq, amplitude=amp) for p in "qk")
    v = binding.rope(rows[:, :, PARTS["v"]].transpose(1, 2), None)
    o, lse = binding.attention(q, k, v, True)
    grads = binding.attention_backward(q, k, v, o, lse, dout.cuda(), True)
    grad = torch.empty_like(rows)
    for (name, part), dx in zip(PARTS.items(), grads):
        binding.rope_backward(dx, None if name == "v" else freq, amplitude=amp, out=grad.transpose(1, 2)[:, part])
    loss, want = reference(torch, qkv, dout, inv, amp)
    check_along_gradients(torch, grad.double().cpu(), loss, qkv.double(), want)
