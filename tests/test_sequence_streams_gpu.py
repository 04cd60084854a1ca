"""Sequence operators on a stream of their own, behind work of that stream that writes their
inputs: until it has run the inputs are NaN, so a launch anywhere else shows."""
import pytest
import torch

import seq_ref as R
import sparse_memory_linear_scoring_b200 as sdm

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def _operators(dtype):
    """name -> (inputs that are read or updated, function of a stream)"""
    g = torch.Generator(device="cuda").manual_seed(0)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").to(dtype)  # noqa: E731
    x, w, dyc, cs = r(2, 4, 300, 64), r(4, 64, 4), r(2, 4, 300, 64), r(2, 4, 3, 64)
    Bm, Cm, dy = r(2, 2, 300, 64), r(2, 2, 300, 64), r(2, 4, 300, 64)
    dt, A, S = torch.rand(2, 4, 300, generator=g, device="cuda"), -torch.rand(4, generator=g, device="cuda"), r(2, 4, 64, 64).float()
    q, k, v, do = r(2, 8, 700, 64), r(2, 2, 700, 64), r(2, 2, 700, 64), r(2, 8, 700, 64)
    kc = R.pool(k, 64)
    idx = R.select(q, kc, 5, 64, 700)
    o, lse = sdm.block_forward(q, k, v, idx, return_lse=True)
    first = lambda t: t[:, :, :1]  # noqa: E731
    return {
        "conv": ([x, cs], lambda s: [sdm.conv_forward(x, w, state=cs, stream=s), cs]),
        "conv_grad": ([x, dyc], lambda s: list(sdm.conv_backward(x, w, dyc, stream=s).values())),
        "scan": ([x, dt, Bm, Cm, S], lambda s: [sdm.ssm_forward(x, dt, A, Bm, Cm, S, stream=s), S]),
        "step": ([x, dt, Bm, Cm, S], lambda s: [sdm.ssm_step(first(x), first(dt), A, first(Bm), first(Cm), S, stream=s), S]),
        "scan_grad": ([x, dt, Bm, Cm, S, dy], lambda s: list(sdm.ssm_backward(x, dt, A, Bm, Cm, S, dy, S, stream=s).values())),
        "pool": ([k], lambda s: [sdm.block_pool(k, stream=s)]),
        "select": ([q, kc], lambda s: [sdm.block_select(q, kc, n_sel=5, stream=s)]),
        "attend": ([q, k, v], lambda s: list(sdm.block_forward(q, k, v, idx, return_lse=True, stream=s))),
        "attend_token": ([q, k, v], lambda s: [sdm.block_forward(q[:, :, -1:], k, v, idx[:, :, -1:].contiguous(), stream=s)]),
        "attend_grad": ([q, k, v, o, do], lambda s: list(sdm.block_backward(q, k, v, idx, o, lse, do, stream=s).values())),
    }


@pytest.mark.parametrize("dtype", [BF, F32])
def test_behind_work_of_its_stream(dtype):
    ops = _operators(dtype)
    side = torch.cuda.Stream()
    for name, (inputs, call) in ops.items():
        keep = [t.clone() for t in inputs]
        want = [t.clone() for t in call(None)]
        call(side)  # its allocations are made before the inputs are spoilt
        for t in inputs:
            t.fill_(float("nan"))
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)  # about 10 ms
            for t, s in zip(inputs, keep):
                t.copy_(s)
        got = call(side)
        side.synchronize()
        for a, b in zip(want, got):
            assert torch.equal(a, b), name
        for t, s in zip(inputs, keep):
            t.copy_(s)
        torch.cuda.synchronize()


def test_behind_an_event_of_another_stream():
    """The current stream waits for an event of the stream that writes the inputs."""
    ops = _operators(BF)
    other = torch.cuda.Stream()
    for name, (inputs, call) in ops.items():
        keep = [t.clone() for t in inputs]
        want = [t.clone() for t in call(None)]
        for t in inputs:
            t.fill_(float("nan"))
        torch.cuda.synchronize()
        with torch.cuda.stream(other):
            torch.cuda._sleep(20_000_000)
            for t, s in zip(inputs, keep):
                t.copy_(s)
            done = other.record_event()
        torch.cuda.current_stream().wait_event(done)
        got = call(None)
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert torch.equal(a, b), name
        for t, s in zip(inputs, keep):
            t.copy_(s)
