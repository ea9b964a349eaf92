"""quantize_rows allocates what it is not given on the stream it runs on: memory
that another stream still uses is not handed out, and what the caller drops
is not handed out elsewhere while the call still writes it."""

import pytest
import torch

import mixture_experts_layer_62_b200 as moe

pytestmark = pytest.mark.gpu
DEV = "cuda"
SHAPE = (1000, 4096)


@pytest.mark.parametrize("as_handle", [False, True])
def test_results_do_not_share_memory_that_another_stream_still_uses(as_handle):
    x = torch.randn(SHAPE, device=DEV).to(torch.bfloat16)
    want = moe.quantize_rows(x)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    stream = side.cuda_stream if as_handle else side
    for _ in range(5):
        # work of the current stream, still waiting when its tensors are dropped
        held = [torch.empty(SHAPE, dtype=torch.int8, device=DEV), torch.empty(SHAPE[0], device=DEV)]
        torch.cuda._sleep(20_000_000)
        for t in held:
            t.fill_(99)
        del held, t
        q, s = moe.quantize_rows(x, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(q, want[0]) and torch.equal(s, want[1])
        del q, s


def test_dropped_results_are_not_handed_out_while_they_are_written():
    x = torch.randn(SHAPE, device=DEV).to(torch.bfloat16)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)
        out = moe.quantize_rows(x, stream=side)
        del out
        got = [torch.full(SHAPE, 5, dtype=torch.int8, device=DEV), torch.full((SHAPE[0],), 5.0, device=DEV)]
        torch.cuda.synchronize()
        assert all((t == 5).all() for t in got)
        del got


def test_given_outputs_and_the_default_stream():
    x = torch.randn((30, 256), device=DEV).to(torch.bfloat16)
    want = moe.quantize_rows(x)
    q, s = torch.empty_like(want[0]), torch.empty_like(want[1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for stream in (side, side.cuda_stream, 0, torch.cuda.current_stream()):
        for give in (dict(q=q), dict(scale=s), dict(q=q, scale=s)):
            q.zero_(), s.zero_()
            torch.cuda.synchronize()
            out = moe.quantize_rows(x, stream=stream, **give)
            torch.cuda.synchronize()
            assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
            assert all(out[("q", "scale").index(n)] is t for n, t in give.items())
