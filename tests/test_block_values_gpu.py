"""Block-selected attention where its values are unusual: infinities and NaN in queries and
incoming gradients, channels of very different sizes, keys that share a large component."""
import pytest
import torch

import seq_ref as R
import sparse_memory_linear_scoring_b200 as sdm
from test_block_gpu import _k, _make

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("value", [NAN, INF])
@pytest.mark.parametrize("name", ["q", "do"])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d,block,Tq,Tk", [(64, 64, 200, 200), (64, 32, 20, 200), (128, 128, 200, 200),
                                          (32, 64, 300, 333), (64, 128, 900, 900), (128, 32, 150, 150)])
def test_queries_stay_out_of_later_keys(d, block, Tq, Tk, dtype, name, value):
    """A query or an incoming gradient that is not finite reaches dK and dV of the keys that
    the query sees and leaves the others', those behind it in its own block among them."""
    q, k, v, g = _make(1, 4, 2, Tq, Tk, d, dtype)
    idx = R.select(q, R.pool(k, block), 3, block, Tk)
    do = torch.randn(q.shape, generator=g, device="cuda").to(dtype)
    o, lse = sdm.block_forward(q, k, v, idx, block=block, return_lse=True)
    good = sdm.block_backward(q, k, v, idx, o, lse, do, block=block)
    seen = torch.zeros(2, Tk, dtype=torch.bool, device="cuda")
    c = R.counts(idx, block, Tk, R.positions(1, Tq, Tk, None, q.device))[0] > 0
    for h, t in ((1, Tq // 2), (2, Tq - 18), (0, 3)):
        (q if name == "q" else do)[0, h, t, 5] = value
        seen[h // 2] |= c[h // 2, t]
    assert not seen[0, Tk - Tq + Tq // 2 + 1:].all() and seen.any(1).all()
    o, lse = sdm.block_forward(q, k, v, idx, block=block, return_lse=True)
    got = sdm.block_backward(q, k, v, idx, o, lse, do, block=block)
    for n in ("k", "v"):
        for gr in range(2):
            a, b, s = got[n][0, gr], good[n][0, gr], seen[gr]
            assert torch.equal(a[~s], b[~s]), "d%s of group %d" % (n, gr)
            if name == "do" and n == "v":  # one column of dO
                assert torch.equal(a[:, :5], b[:, :5]) and torch.equal(a[:, 6:], b[:, 6:])
                assert not torch.isfinite(a[s, 5]).any()
            elif value != value or name == "do":
                assert not torch.isfinite(a[s]).any()


@pytest.mark.parametrize("Tq", [1, 20, 1500])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d,block", [(64, 64), (128, 32), (32, 128)])
def test_channels_of_different_sizes(d, block, dtype, Tq):
    """Values, and keys for dQ, whose channels differ by up to 2^23: each channel of the
    result is as exact as its own terms allow."""
    q, k, v, g = _make(2, 12, 2, Tq, 1777, d, dtype, "token")
    size = 2.0 ** -(torch.arange(d, device="cuda") % 24).float()
    v.copy_((v.float() * size).to(dtype))
    k.copy_((k.float() * size).to(dtype))
    idx = R.select(q, R.pool(k, block), 24, block, 1777)
    do = torch.randn(q.shape, generator=g, device="cuda").to(dtype)
    ref = R.block_attention(q, k, v, idx, block, 1.0, None, do)
    o, lse = sdm.block_forward(q, k, v, idx, block=block, scale=1.0, return_lse=True)
    R.close(o, ref["o"], _k(dtype, d, ref) * ref["o_mag"], "o")
    out = sdm.block_backward(q, k, v, idx, o, lse, do, block=block, scale=1.0)
    # as the other gradients: scores twice, one rounding of P or dS, one of o in do.o
    k1 = 4 * d * R.ADD * float(ref["smag"].max()) + 2.0 ** -18 + (300 + 24 * 8) * R.ADD
    if dtype == BF:
        k1 += 2 * 2.0 ** -8 * 1.02
    R.close(out["q"], ref["q"], k1 * ref["q_mag"], "dq")


def _norm(a, b):
    return float((a.double() - b).norm() / b.norm())


@pytest.mark.parametrize("H,G,Tq,Tk,d,block,layout", [
    (8, 2, 1, 600, 64, 64, "dense"), (8, 8, 20, 600, 64, 64, "token"), (4, 2, 300, 600, 128, 32, "odd"),
    (8, 2, 600, 600, 64, 64, "token"), (12, 2, 900, 900, 128, 64, "token"), (6, 3, 500, 500, 32, 128, "dense")])
def test_keys_with_a_common_part(H, G, Tq, Tk, d, block, layout):
    """A row of dS sums to zero, so what a query's keys share drops out of dQ.  Keys 8 units
    off centre: the result's rounding makes 0.0017 of the norm; what is left of dS behind its
    two parts, 2^-17, of do.o behind its correction, 2^-4 of 0.0022, and of the parts, 2^-12,
    enters eight times as large: below 0.004.  One part of dS or no correction: about 0.02."""
    q, k, v, g = _make(2, H, G, Tq, Tk, d, BF, layout)
    k += 8 * torch.sign(torch.randn(d, generator=g, device="cuda")).to(BF)
    q *= 0.25
    idx = R.select(q, R.pool(k, block), 6, block, Tk)
    do = torch.randn(q.shape, generator=g, device="cuda").to(BF)
    ref = R.block_attention(q, k, v, idx, block, d ** -0.5, None, do)
    o, lse = sdm.block_forward(q, k, v, idx, block=block, return_lse=True)
    out = sdm.block_backward(q, k, v, idx, o, lse, do, block=block)
    assert _norm(out["q"], ref["q"]) <= 0.004


@pytest.mark.parametrize("H,G,Tq,Tk,d,block", [
    (8, 2, 1, 600, 64, 64), (8, 8, 20, 600, 64, 64), (8, 2, 600, 600, 64, 64), (12, 2, 900, 900, 128, 64),
    (6, 3, 500, 500, 32, 128)])
def test_norms(H, G, Tq, Tk, d, block):
    """bf16 results and gradients: 0.00165 of the norm is the rounding of a result with
    evenly spread mantissas; one more rounding of an operand adds its square at most once."""
    q, k, v, g = _make(2, H, G, Tq, Tk, d, BF, "token")
    idx = R.select(q, R.pool(k, block), 6, block, Tk)
    do = torch.randn(q.shape, generator=g, device="cuda").to(BF)
    ref = R.block_attention(q, k, v, idx, block, d ** -0.5, None, do)
    o, lse = sdm.block_forward(q, k, v, idx, block=block, return_lse=True)
    out = sdm.block_backward(q, k, v, idx, o, lse, do, block=block)
    for n, a in (("o", o), *out.items()):
        assert _norm(a, ref[n]) <= 2 ** 0.5 * 0.00165 * 1.05, n
