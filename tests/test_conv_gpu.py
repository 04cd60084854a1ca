"""conv_forward / conv_backward against the float64 form: every filter length, both
types, dense and sliced layouts, aligned and not, carried states, padded batches,
lengths from one to several tiles."""
import pytest
import torch

import seq_ref as R
import sparse_memory_linear_scoring_b200 as sdm

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def _rn(gen, *shape, dtype=F32, sd=1.0):
    return (torch.randn(*shape, generator=gen, device="cuda") * sd).to(dtype)


def _make(B, H, T, d, K, dtype, layout, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    if layout == "dense":
        x = _rn(g, B, H, T, d, dtype=dtype)
    elif layout == "token":  # a slice of a wider token-major projection, 16-byte aligned
        x = _rn(g, B, T, H * d + 16, dtype=dtype)[..., 8:8 + H * d].view(B, T, H, d).transpose(1, 2)
    else:                    # a slice at an odd element
        x = _rn(g, B, T, H * d + 3, dtype=dtype)[..., 1:1 + H * d].view(B, T, H, d).transpose(1, 2)
    w = _rn(g, H, d, K, dtype=dtype, sd=K ** -0.5)
    b = _rn(g, H, d, dtype=dtype, sd=0.3)
    st = _rn(g, B, H, K - 1, d, dtype=dtype)
    return g, x, w, b, st


def _bound(x, w, b, st, silu):
    """p: K + 1 float32 additions.  silu has slope at most 1.1, and __expf (2^-21 and a
    half step of p log2 e in the exponent) moves it by at most (2^-21 + |p| 2^-23) |y|."""
    mag, _, _ = R.conv(x.abs(), w.abs(), None if b is None else b.abs(), None if st is None else st.abs(), False)
    y, p, _ = R.conv(x, w, b, st, silu)
    k = (w.shape[-1] + 2) * R.ADD
    if not silu:
        return y, k * mag
    return y, 1.1 * k * mag + (2.0 ** -20 + p.abs() * 2.0 ** -22) * y.abs()


CASES = [
    # B, H, T, d, K, dtype, layout, silu
    (2, 3, 1, 64, 4, BF, "dense", True), (2, 3, 2, 64, 4, BF, "token", True),
    (1, 1, 3, 40, 4, BF, "dense", True), (2, 2, 100, 24, 4, BF, "odd", True),
    (1, 2, 33, 7, 3, BF, "dense", False), (3, 1, 257, 640, 4, BF, "token", True),
    (2, 2, 70, 16, 2, BF, "dense", True), (1, 2, 65, 8, 8, BF, "dense", True),
    (1, 3, 31, 12, 5, F32, "dense", True), (2, 2, 130, 20, 4, F32, "token", True),
    (1, 2, 90, 5, 4, F32, "odd", True), (1, 1, 5, 4, 7, F32, "dense", False),
    (1, 1, 4, 4, 6, F32, "dense", True), (1, 4, 5000, 32, 4, BF, "token", True),
]


@pytest.mark.parametrize("B,H,T,d,K,dtype,layout,silu", CASES)
@pytest.mark.parametrize("full", [True, False])
def test_forward(B, H, T, d, K, dtype, layout, silu, full):
    _, x, w, b, st = _make(B, H, T, d, K, dtype, layout)
    if not full:
        b = st = None
    ref, bound = _bound(x, w, b, st, silu)
    s = None if st is None else st.clone()
    y = sdm.conv_forward(x, w, b, s, silu=silu)
    R.close(y, ref, bound, "y")
    if s is not None:
        assert torch.equal(s, torch.cat([st, x], 2)[:, :, T:])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("layout", ["token", "odd"])
def test_padded_batch(dtype, layout):
    B, H, T, d, K = 5, 2, 77, 24, 4
    _, x, w, b, st = _make(B, H, T, d, K, dtype, layout)
    n = [77, 0, 1, 2, 40]
    for i, l in enumerate(n):
        x[i, :, l:] = float("nan")
    s = st.clone()
    y = sdm.conv_forward(x, w, b, s, lengths=torch.tensor(n, dtype=torch.int32, device="cuda"))
    for i, l in enumerate(n):
        assert (y[i, :, l:] == 0).all()
        assert torch.equal(s[i], torch.cat([st[i], x[i, :, :l]], 1)[:, l:])
        if l:
            ref, bound = _bound(x[i:i + 1, :, :l], w, b, st[i:i + 1], True)
            R.close(y[i:i + 1, :, :l], ref, bound, "row %d" % i)
    # values outside [0, T] are clamped
    s2 = st.clone()
    sdm.conv_forward(x, w, b, s2, lengths=torch.tensor([999, -3, 1, 2, 40], dtype=torch.int32, device="cuda"))
    assert torch.equal(s2, s)


def test_tokens_equal_prompt():
    _, x, w, b, st = _make(2, 2, 9, 16, 4, BF, "token")
    s1, s2 = st.clone(), st.clone()
    y = sdm.conv_forward(x, w, b, s1)
    one = torch.cat([sdm.conv_forward(x[:, :, t:t + 1], w, b, s2) for t in range(9)], 2)
    assert torch.equal(y, one) and torch.equal(s1, s2)


@pytest.mark.parametrize("B,H,T,d,K,dtype,layout,silu", CASES)
@pytest.mark.parametrize("full", [True, False])
def test_backward(B, H, T, d, K, dtype, layout, silu, full):
    g, x, w, b, st = _make(B, H, T, d, K, dtype, layout)
    dy = _rn(g, B, T, H, d, dtype=dtype).transpose(1, 2)
    ds = _rn(g, B, H, K - 1, d)
    if not full:
        b = st = ds = None

    def grads(x, w, b, st, dy, ds, magnitude):
        y, p, past = R.conv(x, w, b, st, False)
        sg = torch.sigmoid(p)
        dp = dy.double() * (sg * (1 + p * (1 - sg)) if silu else 1.0)
        if magnitude:
            x, w, past, dp = x.abs(), w.abs(), past.abs(), dp.abs()
            ds = None if ds is None else ds.abs()
        dpast, dw = torch.zeros_like(past), torch.zeros_like(w.double())
        for i in range(K):
            dpast[:, :, i:i + T] += dp * w.double()[None, :, None, :, i]
            dw[..., i] = (dp * past[:, :, i:i + T]).sum((0, 2))
        if ds is not None:
            dpast[:, :, T:] += ds.double()
        return dpast, dw, dp.sum((0, 2)), dp, p

    dpast, dw, db, _, p = grads(x, w, b, st, dy, ds, False)
    mpast, mw, mb, mdp, _ = grads(x, w, b, st, dy, ds, True)
    # dp = dy silu'(p), |silu''| <= 1/2: its error is half of p's on dy, and a few steps of
    # its own; sums of B T terms in order within a tile, then over tiles
    pm = R.conv(x.abs(), w.abs(), None if b is None else b.abs(), None if st is None else st.abs(), False)[0]
    e = (K + 2) * R.ADD * pm * 0.5 * dy.double().abs() + (2.0 ** -19 + p.abs() * 2.0 ** -21) * (dy.double().abs() * 1.1) \
        if silu else 0 * mdp
    ew, epast = torch.zeros_like(mw), torch.zeros_like(mpast)
    past = torch.cat([x.new_zeros(B, H, K - 1, d) if st is None else st, x], 2).double().abs()
    for i in range(K):
        epast[:, :, i:i + T] += e * w.double().abs()[None, :, None, :, i]
        ew[..., i] = (e * past[:, :, i:i + T]).sum((0, 2))
    out = sdm.conv_backward(x, w, dy, b, st, ds, silu=silu)
    n_add = 96 + B * T // 64
    R.close(out["x"], dpast[:, :, K - 1:], epast[:, :, K - 1:] + (K + 2) * R.ADD * mpast[:, :, K - 1:], "dx")
    R.close(out["w"], dw, ew + n_add * R.ADD * mw, "dw")
    if full:
        R.close(out["bias"], db, e.sum((0, 2)) + n_add * R.ADD * mb, "dbias")
        R.close(out["state"], dpast[:, :, :K - 1], epast[:, :, :K - 1] + (K + 2) * R.ADD * mpast[:, :, :K - 1], "dstate")
    else:
        assert "bias" not in out and "state" not in out


def test_backward_is_the_slope():
    """Central differences of the kernel's own forward, float32, along one direction."""
    g, x, w, b, st = _make(1, 2, 37, 8, 4, F32, "dense")
    dy = _rn(g, 1, 2, 37, 8)
    out = sdm.conv_backward(x, w, dy, b, st)
    for name, t in (("x", x), ("w", w), ("bias", b), ("state", st)):
        v = _rn(g, *t.shape)
        h = 1e-2

        def f(sign):
            args = {"x": x, "w": w, "bias": b, "state": st, name: t + sign * h * v}
            y = sdm.conv_forward(args["x"], args["w"], args["bias"], args["state"].clone())
            return float((y.double() * dy.double()).sum())

        slope = (f(1) - f(-1)) / (2 * h)
        got = float((out[name].double() * v.double()).sum())
        # third derivatives of silu are below 1: h^2 / 6 of sum |dy| |dp|^3 is far under 1e-3
        # of the norms; float32 differences add 2^-24 |f| / h
        size = float(out[name].double().norm() * v.double().norm())
        assert abs(slope - got) <= 2e-3 * size + 1e-3, (name, slope, got)


def test_equal_calls_give_equal_bits():
    g, x, w, b, st = _make(2, 2, 3000, 32, 4, BF, "token")
    dy = _rn(g, 2, 2, 3000, 32, dtype=BF)
    a, c = (sdm.conv_backward(x, w, dy, b, st) for _ in range(2))
    for n in a:
        assert torch.equal(a[n], c[n]), n
