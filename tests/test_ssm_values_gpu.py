"""The selective scan where its inputs hold infinities or NaN: what does not depend on such
a value keeps its own result; what does is not finite either.  float64 walk step by step as
the reference."""
import pytest
import torch

import seq_ref as R
import sparse_memory_linear_scoring_b200 as sdm
from test_ssm_gpu import _k, _k_state, _mag, _make

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
NAN, INF = float("nan"), float("inf")

# one or several chunks a segment, one or several segments, tensor cores and CUDA cores
SHAPES = [
    # B, H, G, T, P, N, dtype, layout
    (1, 2, 1, 150, 64, 64, BF, "token"), (1, 2, 2, 150, 128, 128, BF, "token"),
    (1, 2, 1, 150, 64, 128, BF, "dense"), (1, 2, 1, 150, 128, 64, BF, "token"),
    (1, 2, 1, 150, 32, 16, BF, "token"), (1, 2, 1, 150, 64, 64, BF, "odd"),
    (1, 2, 1, 150, 16, 32, F32, "token"), (1, 24, 2, 800, 64, 128, BF, "token"),
    (1, 24, 2, 800, 128, 64, BF, "token"), (20, 16, 1, 150, 64, 64, BF, "token"),
]


def _poke(a, name, at, value):
    """One element of one step; every head of its group reads those of Bm and Cm."""
    t = a[name]
    if name == "dt":
        t[0, 0, at] = value
    else:
        t[0, 0, at, 11] = value


@pytest.mark.parametrize("at,value", [(5, NAN), (70, INF), (111, NAN), (128, -INF)])
@pytest.mark.parametrize("name", ["x", "Bm", "Cm", "dt"])
@pytest.mark.parametrize("B,H,G,T,P,N,dtype,layout", SHAPES)
def test_later_values_stay_out(B, H, G, T, P, N, dtype, layout, name, at, value):
    a, _ = _make(B, H, G, T, P, N, dtype, layout)
    if name == "dt":
        value = NAN
    ym, Sm, _ = R.ssm(**_mag(a))
    _poke(a, name, at, value)
    y, ST, _ = R.ssm(**a)
    S = a["S"].clone()
    got = sdm.ssm_forward(a["x"], a["dt"], a["A"], a["Bm"], a["Cm"], S, a["D"])
    for g, r, bound, what in ((got, y, _k(dtype, T, P, N) * ym, "y"), (S, ST, _k_state(T) * Sm, "S")):
        fin = torch.isfinite(r)
        assert torch.equal(torch.isfinite(g), fin), "%s: finite in different places" % what
        z = torch.zeros((), device="cuda")
        R.close(torch.where(fin, g, z.to(g.dtype)), torch.where(fin, r, z.double()), bound, what)
    if T <= 150:  # no decay that reaches 0: an infinity stays one in the state
        R.close(S, ST, _k_state(T) * Sm, "S")


def _grads(a, dy, dS):
    return sdm.ssm_backward(a["x"], a["dt"], a["A"], a["Bm"], a["Cm"], a["S"], dy, dS, D=a["D"])


@pytest.mark.parametrize("at,value", [(5, NAN), (70, INF), (111, NAN), (128, -INF)])
@pytest.mark.parametrize("name", ["x", "Bm", "Cm", "dy"])
@pytest.mark.parametrize("B,H,G,T,P,N,dtype,layout", SHAPES[:7])
def test_gradients_stay_apart(B, H, G, T, P, N, dtype, layout, name, at, value):
    a, g = _make(B, H, G, T, P, N, dtype, layout)
    dy = torch.randn(B, T, H, P, generator=g, device="cuda").to(dtype).transpose(1, 2)
    dS = torch.randn(B, H, P, N, generator=g, device="cuda") * 0.3
    args = [a[n] for n in ("x", "dt", "A", "Bm", "Cm", "S")]
    mag = R.ssm_grads(*args, dy, dS, a["D"], magnitude=True)
    _poke({**a, "dy": dy}, name, at, value)
    ref = R.ssm_grads(*args, dy, dS, a["D"])
    out = _grads(a, dy, dS)
    k16 = _k(dtype, T, P, N) + P * R.ADD
    k32 = (64 + 2 * max(P, N) + T / 32 + 16) * R.ADD + 2.0 ** -17
    # dt's gradient is a running sum over a chunk of at most 64 steps that may be taken from
    # either end: the terms of both count
    mag["dt"] = 2 * torch.nn.functional.max_pool1d(mag["dt"].float().flatten(0, 1)[None], 129, 1, 64)[0].view_as(mag["dt"]).double()
    for n in ("x", "Bm", "Cm", "dt", "S0"):
        fin = torch.isfinite(ref[n])
        assert torch.equal(torch.isfinite(out[n]), fin), "d%s: finite in different places" % n
        z = torch.zeros((), device="cuda")
        R.close(torch.where(fin, out[n], z.to(out[n].dtype)), torch.where(fin, ref[n], z.double()),
                (k16 if n in ("x", "Bm", "Cm") else k32) * mag[n], "d" + n)


def test_step_decay_is_exact():
    """exp(dt A) of one step for decays down to e^-80: expf's 2 units in the last place and
    two roundings, 2^-21 of the state, however large |dt A| is."""
    H = 512
    dt = torch.linspace(0.01, 9.99, H, device="cuda").view(1, H, 1)
    A = -torch.full((H,), 8.0, device="cuda") + torch.linspace(0, 0.1, H, device="cuda")
    S = torch.linspace(1, 2, 256, device="cuda").view(1, 1, 16, 16).repeat(1, H, 1, 1)
    z = torch.zeros(1, H, 1, 16, device="cuda")
    want = S.double() * torch.exp(dt.double() * A.double()[None, :, None])[..., None]
    sdm.ssm_step(z, dt, A, z, z, S)
    assert float(((S.double() - want) / want).abs().max()) <= 2.0 ** -21


@pytest.mark.parametrize("B,H,G,T,P,N", [(2, 8, 2, 64, 64, 64), (2, 8, 2, 500, 64, 64), (2, 4, 4, 500, 128, 128),
                                         (2, 4, 1, 500, 64, 128), (24, 12, 1, 200, 128, 64)])
def test_norms(B, H, G, T, P, N):
    """bf16 results and gradients: 0.00165 of the norm is the rounding of a result with
    evenly spread mantissas; y and dx have one more rounding of an operand in each term,
    which adds its square at most once.  One part of the weights in dB and dC would make
    0.0027 in a short call."""
    a, g = _make(B, H, G, T, P, N, BF)
    dy = torch.randn(B, T, H, P, generator=g, device="cuda").to(BF).transpose(1, 2)
    dS = torch.randn(B, H, P, N, generator=g, device="cuda") * 0.1
    S = a["S"].clone()
    y = sdm.ssm_forward(a["x"], a["dt"], a["A"], a["Bm"], a["Cm"], S, a["D"])
    out = _grads(a, dy, dS)
    ry, _, _ = R.ssm(**a)
    ref = R.ssm_grads(a["x"], a["dt"], a["A"], a["Bm"], a["Cm"], a["S"], dy, dS, a["D"])
    for n, got, want in [("y", y, ry)] + [(n, out[n], ref[n]) for n in ("x", "Bm", "Cm")]:
        assert float((got.double() - want).norm() / want.norm()) <= 2 ** 0.5 * 0.00165 * 1.05, n
