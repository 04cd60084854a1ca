"""ssm_forward / ssm_step / ssm_backward against the float64 walk: state widths, both
types, groups, lengths from one step over several segments, padded batches, decays
from none to complete, carried states."""
import math

import pytest
import torch

import seq_ref as R
import sparse_memory_linear_scoring_b200 as sdm

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def _make(B, H, G, T, P, N, dtype, layout="token", decay="usual", seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    off = 1 if layout == "odd" else 0
    xbc = rn(B, T, H * P + 2 * G * N + off).to(dtype)[..., off:]
    x = xbc[..., :H * P].unflatten(-1, (H, P)).transpose(1, 2)
    Bm = xbc[..., H * P:H * P + G * N].unflatten(-1, (G, N)).transpose(1, 2)
    Cm = xbc[..., H * P + G * N:].unflatten(-1, (G, N)).transpose(1, 2)
    if layout == "dense":
        x, Bm, Cm = x.contiguous(), Bm.contiguous(), Cm.contiguous()
    u = torch.rand(B, T, H, generator=g, device="cuda")
    if decay == "usual":
        dt, A = torch.exp(u * 4.6 - 6.9), -torch.exp(torch.rand(H, generator=g, device="cuda") * 2.8)
    elif decay == "none":
        dt, A = u * 0.1, torch.zeros(H, device="cuda")
    elif decay == "strong":   # a chunk's decay far below the smallest float
        dt, A = u * 2.0, -torch.full((H,), 100.0, device="cuda")
    else:                     # steps that write nothing
        dt, A = torch.where(u < 0.5, torch.zeros_like(u), u), -torch.ones(H, device="cuda")
    D = rn(H)
    return dict(x=x, dt=dt.transpose(1, 2), A=A, Bm=Bm, Cm=Cm, S=rn(B, H, P, N) * 0.5, D=D), g


def _mag(a):
    return {n: (t if n in ("dt", "A") else t.abs()) for n, t in a.items()}


def _k(dtype, T, P, N):
    """Roundings of a term: bf16 operands of the products in y (weights and the state, one
    each), float32 sums over a chunk and the state's width, one more an earlier chunk."""
    n = 64 + N + T / 32 + 8
    # exp2 and the decay differences: 2^-21 each, a few of them
    return (2.0 ** -8 * 1.02 if dtype == BF else 0.0) + n * R.ADD + 2.0 ** -20


def _k_state(T):
    return (64 + T / 32 + 8) * R.ADD + 2.0 ** -20


SHAPES = [
    # B, H, G, T, P, N, dtype, layout, decay
    (1, 1, 1, 1, 64, 64, BF, "token", "usual"), (2, 4, 2, 63, 64, 64, BF, "token", "usual"),
    (1, 2, 1, 64, 64, 128, BF, "dense", "usual"), (1, 2, 2, 65, 128, 64, BF, "token", "usual"),
    (2, 2, 1, 130, 128, 128, BF, "token", "usual"), (1, 3, 3, 200, 32, 16, BF, "token", "usual"),
    (1, 2, 1, 100, 16, 128, BF, "odd", "usual"), (1, 2, 1, 300, 64, 64, BF, "odd", "usual"),
    (1, 2, 1, 700, 64, 64, BF, "token", "none"), (1, 2, 1, 300, 64, 64, BF, "token", "strong"),
    (1, 2, 1, 300, 64, 128, BF, "token", "gaps"), (1, 6, 2, 90, 16, 32, F32, "token", "usual"),
    (1, 2, 1, 333, 128, 128, F32, "token", "usual"), (2, 2, 1, 33, 64, 16, F32, "odd", "usual"),
    (1, 2, 1, 200, 32, 64, F32, "dense", "strong"), (1, 2, 1, 200, 32, 64, F32, "dense", "none"),
    (1, 1, 1, 1500, 64, 64, BF, "token", "usual"), (1, 1, 1, 1100, 32, 32, F32, "token", "usual"),
]


@pytest.mark.parametrize("B,H,G,T,P,N,dtype,layout,decay", SHAPES)
def test_forward(B, H, G, T, P, N, dtype, layout, decay):
    a, _ = _make(B, H, G, T, P, N, dtype, layout, decay)
    y, ST, _ = R.ssm(**a)
    ym, Sm, _ = R.ssm(**_mag(a))
    S = a["S"].clone()
    got = sdm.ssm_forward(a["x"], a["dt"], a["A"], a["Bm"], a["Cm"], S, a["D"])
    assert got.dtype == dtype and got.shape == a["x"].shape
    R.close(got, y, _k(dtype, T, P, N) * ym, "y")
    R.close(S, ST, _k_state(T) * Sm, "S")
    # without D
    S2 = a["S"].clone()
    got = sdm.ssm_forward(a["x"], a["dt"], a["A"], a["Bm"], a["Cm"], S2)
    a["D"] = torch.zeros_like(a["D"])
    R.close(got, R.ssm(**a)[0], _k(dtype, T, P, N) * R.ssm(**_mag(a))[0], "y without D")
    assert torch.equal(S, S2)


@pytest.mark.parametrize("dtype,P,N", [(BF, 64, 64), (BF, 32, 16), (F32, 16, 32)])
def test_padded_batch(dtype, P, N):
    B, H, G, T = 5, 2, 1, 700
    a, _ = _make(B, H, G, T, P, N, dtype)
    n = [700, 0, 1, 64, 399]
    for i, l in enumerate(n):
        for t in ("x", "Bm", "Cm", "dt"):
            a[t][i, :, l:] = float("nan")
    S = a["S"].clone()
    y = sdm.ssm_forward(a["x"], a["dt"], a["A"], a["Bm"], a["Cm"], S, a["D"],
                        lengths=torch.tensor(n, dtype=torch.int32, device="cuda"))
    for i, l in enumerate(n):
        assert (y[i, :, l:] == 0).all()
        if l == 0:
            assert torch.equal(S[i], a["S"][i])
            continue
        one = {t: (v[i:i + 1, :, :l] if v.dim() >= 3 and t != "S" else v) for t, v in a.items()}
        one["S"] = a["S"][i:i + 1]
        ry, rS, _ = R.ssm(**one)
        my, mS, _ = R.ssm(**_mag(one))
        R.close(y[i:i + 1, :, :l], ry, _k(dtype, T, P, N) * my, "y %d" % i)
        R.close(S[i:i + 1], rS, _k_state(T) * mS, "S %d" % i)


@pytest.mark.parametrize("B,H,G,T,P,N,dtype,layout,decay", [
    (3, 4, 2, 1, 64, 64, BF, "token", "usual"), (1, 2, 1, 3, 128, 128, BF, "odd", "usual"),
    (2, 3, 1, 5, 16, 16, BF, "token", "gaps"), (1, 2, 2, 1, 32, 32, F32, "token", "strong"),
    (2, 2, 1, 7, 16, 128, F32, "odd", "usual"), (1, 1, 1, 2, 128, 16, F32, "dense", "none"),
])
def test_step(B, H, G, T, P, N, dtype, layout, decay):
    a, _ = _make(B, H, G, T, P, N, dtype, layout, decay)
    y, ST, _ = R.ssm(**a)
    ym, Sm, _ = R.ssm(**_mag(a))
    S = a["S"].clone()
    got = sdm.ssm_step(a["x"], a["dt"], a["A"], a["Bm"], a["Cm"], S, a["D"])
    k = (N + 2 * T + 8) * R.ADD + 2.0 ** -20
    # exp(dt A) from the rounded product: |dt A| 2^-24
    k += float((a["dt"].max() * a["A"].abs().max())) * 2.0 ** -23 if decay != "strong" else 2.0 ** -16
    R.close(got, y, k * ym, "y")
    R.close(S, ST, k * Sm, "S")


def test_prompt_then_tokens():
    a, _ = _make(1, 2, 1, 150, 64, 64, BF)
    y, ST, _ = R.ssm(**a)
    ym, Sm, _ = R.ssm(**_mag(a))
    S = a["S"].clone()
    cut = lambda n, i, j: a[n][:, :, i:j]  # noqa: E731
    out = [sdm.ssm_forward(cut("x", 0, 140), cut("dt", 0, 140), a["A"], cut("Bm", 0, 140), cut("Cm", 0, 140), S, a["D"])]
    for t in range(140, 150):
        out.append(sdm.ssm_step(*(cut(n, t, t + 1) for n in ("x", "dt")), a["A"],
                                *(cut(n, t, t + 1) for n in ("Bm", "Cm")), S, a["D"]))
    R.close(torch.cat(out, 2), y, _k(BF, 150, 64, 64) * ym, "y")
    R.close(S, ST, (_k_state(150) + 2.0 ** -19) * Sm, "S")


@pytest.mark.parametrize("B,H,G,T,P,N,dtype,layout,decay", SHAPES)
def test_backward(B, H, G, T, P, N, dtype, layout, decay):
    a, g = _make(B, H, G, T, P, N, dtype, layout, decay)
    dy = torch.randn(B, T, H, P, generator=g, device="cuda").to(dtype).transpose(1, 2)
    dS = torch.randn(B, H, P, N, generator=g, device="cuda") * 0.3
    ref = R.ssm_grads(a["x"], a["dt"], a["A"], a["Bm"], a["Cm"], a["S"], dy, dS, a["D"])
    mag = R.ssm_grads(a["x"], a["dt"], a["A"], a["Bm"], a["Cm"], a["S"], dy, dS, a["D"], magnitude=True)
    out = sdm.ssm_backward(a["x"], a["dt"], a["A"], a["Bm"], a["Cm"], a["S"], dy, dS, D=a["D"])
    k16 = _k(dtype, T, P, N) + P * R.ADD
    # what stays in float32: products of exact inputs, the states as bf16 parts that leave
    # less than 2^-17 of them
    k32 = (64 + 2 * max(P, N) + T / 32 + 16) * R.ADD + 2.0 ** -17
    for n in ("x", "Bm", "Cm"):
        assert out[n].dtype == dtype
        R.close(out[n], ref[n], k16 * mag[n], "d" + n)
    for n in ("dt", "S0"):
        R.close(out[n], ref[n], k32 * mag[n], "d" + n)
    many = (B * T / 64 + 64) * R.ADD
    for n in ("A", "D"):
        R.close(out[n], ref[n], (k32 + many) * (mag[n] if n == "A" else
                (a["x"].double() * dy.double()).abs().sum((0, 2, 3))), "d" + n)


def test_backward_defaults():
    a, g = _make(1, 2, 1, 100, 64, 64, BF)
    dy = torch.randn(1, 2, 100, 64, generator=g, device="cuda").to(BF)
    z = torch.zeros_like(a["S"])
    args = [a[n] for n in ("x", "dt", "A", "Bm", "Cm")]
    p = sdm.ssm_backward(*args, None, dy)
    q = sdm.ssm_backward(*args, z, dy, z, D=torch.zeros_like(a["D"]))
    assert "D" not in p and "D" in q
    for n in p:
        assert torch.equal(p[n], q[n]), n


def test_backward_is_the_slope():
    """Central differences of the kernel's own forward in float32."""
    a, g = _make(1, 2, 1, 40, 16, 16, F32)
    dy = torch.randn(1, 2, 40, 16, generator=g, device="cuda")
    dS = torch.randn(1, 2, 16, 16, generator=g, device="cuda")
    out = sdm.ssm_backward(a["x"], a["dt"], a["A"], a["Bm"], a["Cm"], a["S"], dy, dS, D=a["D"])

    def f(c):
        S = c["S"].clone()
        y = sdm.ssm_forward(c["x"], c["dt"], c["A"], c["Bm"], c["Cm"], S, c["D"])
        return float((y.double() * dy.double()).sum() + (S.double() * dS.double()).sum())

    for n, m, h in (("x", "x", 1e-2), ("dt", "dt", 1e-4), ("A", "A", 1e-2), ("Bm", "Bm", 1e-2),
                    ("Cm", "Cm", 1e-2), ("S", "S0", 1e-2), ("D", "D", 1e-2)):
        v = torch.randn(a[n].shape, generator=g, device="cuda")
        slope = (f({**a, n: a[n] + h * v}) - f({**a, n: a[n] - h * v})) / (2 * h)
        got = float((out[m].double() * v.double()).sum())
        size = float(out[m].double().norm() * v.double().norm())
        # the forward is linear in all but dt and A; float32 noise of f over 2h
        assert abs(slope - got) <= 2e-3 * size, (n, slope, got)


def test_equal_calls_give_equal_bits():
    a, g = _make(2, 4, 1, 1000, 64, 64, BF)
    dy = torch.randn(2, 4, 1000, 64, generator=g, device="cuda").to(BF)
    args = [a[n] for n in ("x", "dt", "A", "Bm", "Cm")]
    runs = []
    for _ in range(2):
        S = a["S"].clone()
        y = sdm.ssm_forward(*args, S, a["D"])
        runs.append(dict(sdm.ssm_backward(*args, a["S"], dy, a["S"], D=a["D"]), y=y, S_T=S))
    for n in runs[0]:
        assert torch.equal(runs[0][n], runs[1][n]), n


def test_many_heads_take_one_segment():
    """Enough heads to fill the card: the single-pass walk."""
    a, _ = _make(20, 16, 1, 300, 64, 64, BF)
    y, ST, _ = R.ssm(**a)
    ym, Sm, _ = R.ssm(**_mag(a))
    S = a["S"].clone()
    R.close(sdm.ssm_forward(a["x"], a["dt"], a["A"], a["Bm"], a["Cm"], S, a["D"]), y,
            _k(BF, 300, 64, 64) * ym, "y")
    R.close(S, ST, _k_state(300) * Sm, "S")
