"""Offsets and lengths out of range in the paged append (attn_paged_append):
they are flagged wherever they stand, whether or not a token leads to them; a
sequence with bad ones gets no tokens, and nothing else is touched."""
from __future__ import annotations

import pytest

from test_gpu_rope import Batch, check_batch, freqs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def cuda():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from tiled_attention_17_b200 import binding
    binding.load()
    return torch, binding


def append(torch, binding, cu, lens, T, seed=0, Hq=2, Hkv=1, d=64, ps=8, seq_lens=None):
    """The batch as its cache and table say (lens), the call with offsets cu and lengths seq_lens."""
    b = Batch(torch, [1] * len(lens), lens, Hq, Hkv, d, ps, 64, seed=seed, behind=T - len(lens))
    assert b.T == T
    inv, _ = freqs(torch, 64)
    as_tensor = lambda x: torch.tensor(x, dtype=torch.int32)   # noqa: E731
    got = b.run(torch, binding, inv, cu=as_tensor(cu), seq_lens=as_tensor(lens if seq_lens is None else seq_lens))
    b.cu = as_tensor(cu)
    return b, inv, got


def claimed(b, cu, ok):
    """(rows, slots) that the sequences in `ok` claim: all that a call may write."""
    rows, slots = set(), set()
    for s in ok:
        for t in range(cu[s], cu[s + 1]):
            slot = b.lens[s] - cu[s + 1] + t
            rows.add(t)
            slots.add((int(b.table[s, slot // b.ps]), slot % b.ps))
    return rows, slots


@pytest.mark.parametrize("cu,lens,T,ok", [
    ([0, 5, 3, 8], [9, 7, 12], 8, [0, 2]),       # decreasing between two sequences that are in order
    ([0, 4, 20], [9, 30], 4, [0]),               # past the rows, and no row leads there
    ([0, 4, 20, 20], [9, 30, 5], 4, [0]),
    ([0, 4, 2, 4], [6, 6, 6], 4, [0, 2]),        # a sequence of minus two tokens
    ([-2, 3, 5], [9, 9], 5, [1]),                # from before the rows
    ([-3, -1, 2], [9, 9], 4, []),
    ([4, 9], [9], 4, []),                        # begins where the rows end
    ([7, 9, 9], [9, 3], 4, []),                  # all of it past the rows
    ([2 ** 31 - 1, -2 ** 31, 2], [9, 9], 4, []),
])
def test_bad_offsets_are_flagged_wherever_they_stand(cuda, cu, lens, T, ok):
    torch, binding = cuda
    b, _, (q, kc, vc, flags) = append(torch, binding, cu, lens, T)
    assert flags == binding.TA_DEV_BAD_SEQ_LEN
    rows, slots = claimed(b, cu, ok)
    for t in range(T):
        if t not in rows:
            assert bool((q[t] == 5).all()), t   # the fill
    for now, before in ((kc, b.kc), (vc, b.vc)):
        changed = {tuple(x) for x in (now != before).any(-1).any(1).nonzero().tolist()}
        assert changed <= slots, changed - slots


@pytest.mark.parametrize("S", [300, 1024, 1025, 5000])
@pytest.mark.parametrize("at", [0.0, 0.4, 1.0])
def test_one_bad_offset_among_many(cuda, S, at):
    # one sequence of minus one token (at the end: one that ends past the rows), between ends that are in order; T rows
    # that need several blocks, and more sequences than the staged table holds
    torch, binding = cuda
    lens = [3 + i % 5 for i in range(S)]
    cu = list(range(S + 1))
    s = min(int(at * S), S - 1)
    if s == S - 1:
        cu[S] += 1
    else:
        cu[s + 1] = cu[s] - 1 if s else -1
    _, _, (_, _, _, flags) = append(torch, binding, cu, lens, S)
    assert flags == binding.TA_DEV_BAD_SEQ_LEN
    cu = list(range(S + 1))
    b, inv, got = append(torch, binding, cu, lens, S)
    assert got[3] == 0
    check_batch(torch, b, got, b.expect(torch, inv, 1.0, False))


def test_a_sequence_past_the_rows_leaves_the_others_alone(cuda):
    torch, binding = cuda
    b, inv, got = append(torch, binding, [0, 1, 2, 30], [9, 4, 60], 3)
    assert got[3] == binding.TA_DEV_BAD_SEQ_LEN
    check_batch(torch, b, got, b.expect(torch, inv, 1.0, False, skip={2}))


@pytest.mark.parametrize("bad", [-1, 1 << 20, 2 ** 31 - 1, -2 ** 31])
@pytest.mark.parametrize("where", [0, 1, 3])
def test_bad_lengths_of_sequences_without_tokens_are_flagged(cuda, bad, where):
    torch, binding = cuda
    cu, lens = [0, 0, 0, 3, 3], [4, 8, 9, 2]
    b = Batch(torch, [0, 0, 3, 0], lens, 2, 1, 64, 8, 64, seed=7)
    inv, _ = freqs(torch, 64)
    seq_lens = b.seq_lens.clone()
    seq_lens[where] = bad
    got = b.run(torch, binding, inv, seq_lens=seq_lens)
    assert got[3] == binding.TA_DEV_BAD_SEQ_LEN
    check_batch(torch, b, got, b.expect(torch, inv, 1.0, False))
    got = b.run(torch, binding, inv)
    assert got[3] == 0


@pytest.mark.parametrize("s", [0, 12345, 18943, 18944, 19999])
def test_more_sequences_than_one_round_of_blocks_looks_at(cuda, s):
    # 148 blocks of 128 threads take a sequence each at a time
    torch, binding = cuda
    S = 20000
    cu, lens = [0] * (S + 1), [1] * S
    for bad in (False, True):
        if bad:
            lens[s] = -1
        table = torch.zeros(S, 1, dtype=torch.int32, device="cuda")
        kc, vc = (torch.zeros(1, 1, 8, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        k = torch.ones(3, 1, 64, dtype=torch.bfloat16, device="cuda")
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")   # noqa: E731
        binding.ta_device_status(True)
        binding.paged_append(k, k, kc, vc, table, i32(lens), i32(cu))
        torch.cuda.synchronize()
        assert binding.ta_device_status(True)[1] == (binding.TA_DEV_BAD_SEQ_LEN if bad else 0)
        assert not bool(kc.any()) and not bool(vc.any())
