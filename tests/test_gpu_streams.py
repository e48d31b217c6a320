"""The stream argument of the calls that allocate on it: a torch stream, a
stream's handle, and 0, the handle of the default stream."""
from __future__ import annotations

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


def test_handles(cuda):
    torch, binding = cuda
    device, side = torch.device("cuda", 0), torch.cuda.Stream(0)
    for stream, handle in ((0, 0), (side.cuda_stream, side.cuda_stream), (side, side.cuda_stream),
                           (torch.cuda.default_stream(0), 0)):
        with torch.cuda.stream(torch.cuda.Stream(0)):
            with binding._scope(device, stream):
                assert torch.cuda.current_stream(0).cuda_stream == handle


@pytest.mark.parametrize("call", ["rope", "append", "shared"])
def test_default_stream_by_its_handle(cuda, call):
    # the input is written late on the default stream, another stream is current: a call on handle 0 waits for the write
    torch, binding = cuda
    x = torch.zeros(1, 2, 16, 64, dtype=torch.bfloat16, device="cuda")
    kc, vc = (torch.ones(3, 2, 8, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")   # noqa: E731
    table, lens, offsets, prefix = i32([[0, 1]]), i32([9]), i32([0, 1]), i32([8])
    run = {"rope": lambda s: binding.rope(x, None, stream=s),
           "append": lambda s: binding.paged_append(x[0, :, :1].transpose(0, 1), x[0, :, :1].transpose(0, 1), kc, vc, table, lens,
                                                    q=x[0, :, 1:2].transpose(0, 1), stream=s),
           "shared": lambda s: binding.paged_decode_shared(x[0, :, :1].transpose(0, 1).contiguous(), kc, vc, table, lens, offsets,
                                                           prefix, stream=s)[0]}[call]
    run(0)   # the first launches are over before the clock below starts
    side = torch.cuda.Stream()
    written = vc if call == "shared" else x
    for value in (3.0, 7.0):
        torch.cuda.synchronize()
        torch.cuda._sleep(20_000_000)   # cycles: some 10 ms
        written.fill_(value)
        with torch.cuda.stream(side):
            if call == "shared":
                q = torch.ones(1, 2, 64, dtype=torch.bfloat16, device="cuda")
                side.synchronize()
                got = binding.paged_decode_shared(q, kc, vc, table, lens, offsets, prefix, stream=0)[0]
            else:
                got = run(0)
        torch.cuda.synchronize()
        assert bool((got == value).all()), (call, value)
