"""Padded batches through layers and in training: each row as by itself."""
import pytest
import torch

import seq_ref as R
import sparse_memory_linear_scoring_b200 as sdm

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
LENS = [300, 1, 129, 64, 2]


def _rn(g, *s):
    return torch.randn(*s, generator=g, device="cuda")


def _live(n, T):
    return torch.arange(T, device="cuda")[None] < torch.tensor(n, device="cuda")[:, None]


@pytest.mark.parametrize("dtype", [BF, F32])
def test_convolution_then_block_attention(dtype):
    """Prompts of different lengths, padded behind, without lengths for the attention: lists,
    results and gradients of the live queries are those of each prompt alone."""
    B, T, H, G, d, block, n_sel = len(LENS), 300, 4, 2, 64, 32, 3
    g = torch.Generator(device="cuda").manual_seed(1)
    C = (H + 2 * G) * d
    xbc = _rn(g, B, 1, T, C).to(dtype)
    live = _live(LENS, T)
    xbc = torch.where(live[:, None, :, None], xbc, torch.full_like(xbc, float("nan")))
    w = (_rn(g, 1, C, 4) * 0.5).to(dtype)
    y = sdm.conv_forward(xbc, w, lengths=torch.tensor(LENS, dtype=torch.int32, device="cuda"))[:, 0]
    q = y[..., :H * d].view(B, T, H, d).transpose(1, 2)
    k = y[..., H * d:(H + G) * d].view(B, T, G, d).transpose(1, 2)
    v = y[..., (H + G) * d:].view(B, T, G, d).transpose(1, 2)
    idx = sdm.block_select(q, sdm.block_pool(k, block=block), n_sel=n_sel, block=block)
    o, lse = sdm.block_forward(q, k, v, idx, block=block, return_lse=True)
    do = (_rn(g, B, H, T, d) * live[:, None, :, None]).to(dtype)
    out = sdm.block_backward(q, k, v, idx, o, lse, do, block=block)
    for b, n in enumerate(LENS):
        one = [t[b:b + 1, :, :n] for t in (q, k, v)]
        i1 = R.select(one[0], R.pool(one[1], block), n_sel, block, n)
        assert torch.equal(idx[b:b + 1, :, :n], i1)
        ref = R.block_attention(*one, i1, block, d ** -0.5, None, do[b:b + 1, :, :n])
        f = 2 * d * R.ADD * ref["smag"][..., None] + 2.0 ** -20 + 300 * R.ADD
        r = 2.0 ** -8 * 1.02 if dtype == BF else 0.0
        R.close(o[b:b + 1, :, :n], ref["o"], (f + r) * ref["o_mag"], "o")
        # scores twice, sums of up to 300 queries' rows; one rounding of P or dS, one of o
        k1 = 2 * float(f.max()) + 2.0 ** -18 + 600 * R.ADD + 2 * r
        for m in ("q", "k", "v"):
            R.close(out[m][b:b + 1, :, :n], ref[m], k1 * ref[m + "_mag"], "d" + m)
            assert (out[m][b, :, n:] == 0).all()


@pytest.mark.parametrize("dtype,P,N", [(BF, 64, 64), (BF, 128, 128), (F32, 32, 16)])
def test_scan_in_training(dtype, P, N):
    """dt = 0 and dy = 0 behind each row's length: the gradients, that of the state left
    among them, are those of each row alone."""
    B, T, H, G = len(LENS), 300, 4, 2
    g = torch.Generator(device="cuda").manual_seed(2)
    x, Bm, Cm = (_rn(g, B, h, T, w).to(dtype) for h, w in ((H, P), (G, N), (G, N)))
    live = _live(LENS, T)[:, None]
    dt = torch.rand(B, H, T, generator=g, device="cuda") * 0.1
    A, D, S0, dS = -_rn(g, H).abs() * 4, _rn(g, H), _rn(g, B, H, P, N), _rn(g, B, H, P, N)
    dy = (_rn(g, B, H, T, P) * live[..., None]).to(dtype)
    dt0 = dt * live
    S = S0.clone()
    sdm.ssm_forward(x, dt0, A, Bm, Cm, S, D)
    out = sdm.ssm_backward(x, dt0, A, Bm, Cm, S0, dy, dS, D=D)
    k16 = (2.0 ** -8 * 1.02 if dtype == BF else 0.0) + (64 + N + P + T / 32 + 8) * R.ADD + 2.0 ** -20
    k32 = (64 + 2 * max(P, N) + T / 32 + 16) * R.ADD + 2.0 ** -17
    dA = dA_mag = 0
    for b, n in enumerate(LENS):
        one = [t[b:b + 1, :, :n] for t in (x, dt)] + [A] + [t[b:b + 1, :, :n] for t in (Bm, Cm)] + [S0[b:b + 1]]
        rest = (dy[b:b + 1, :, :n], dS[b:b + 1], D)
        ref, mag = R.ssm_grads(*one, *rest), R.ssm_grads(*one, *rest, magnitude=True)
        _, ST, _ = R.ssm(*one)
        _, Sm, _ = R.ssm(*[t.abs() if i not in (1, 2) else t for i, t in enumerate(one)])
        R.close(S[b:b + 1], ST, ((64 + T / 32 + 8) * R.ADD + 2.0 ** -20) * Sm, "S")
        for m in ("x", "Bm", "Cm"):
            R.close(out[m][b:b + 1, :, :n], ref[m], k16 * mag[m], "d" + m)
        R.close(out["dt"][b:b + 1, :, :n], ref["dt"], k32 * mag["dt"], "ddt")
        R.close(out["S0"][b:b + 1], ref["S0"], k32 * mag["S0"], "dS0")
        dA, dA_mag = dA + ref["A"], dA_mag + mag["A"]
    R.close(out["A"], dA, (k32 + (B * T / 64 + 64) * R.ADD) * dA_mag, "dA")


@pytest.mark.parametrize("dtype", [BF, F32])
def test_convolution_in_training(dtype):
    """dy = 0 behind each row's length, and the gradient of the state left added where its
    inputs are: in dx, and in the first state's for rows shorter than the filter."""
    B, T, H, d, K = len(LENS), 300, 2, 24, 4
    g = torch.Generator(device="cuda").manual_seed(3)
    x, w, b = _rn(g, B, H, T, d).to(dtype), (_rn(g, H, d, K) * 0.5).to(dtype), _rn(g, H, d).to(dtype)
    st, ds = _rn(g, B, H, K - 1, d).to(dtype), _rn(g, B, H, K - 1, d)
    dy = (_rn(g, B, H, T, d) * _live(LENS, T)[:, None, :, None]).to(dtype)
    out = sdm.conv_backward(x, w, dy, b, st)
    dx, dst = out["x"].float(), out["state"].clone()
    leaves = [t.double().requires_grad_() for t in (w, b)]
    dw = db = 0
    for i, n in enumerate(LENS):
        past = torch.cat([dst[i], dx[i, :, :n]], 1)
        past[:, n:] += ds[i]
        xi, si = x[i:i + 1, :, :n].double().requires_grad_(), st[i:i + 1].double().requires_grad_()
        y, _, p = R.conv(xi, leaves[0], leaves[1], si)
        loss = (y * dy[i:i + 1, :, :n].double()).sum() + (p[:, :, n:] * ds[i:i + 1].double()).sum()
        r = torch.autograd.grad(loss, [xi, si] + leaves)
        want = torch.cat([r[1], r[0]], 2)[0]
        # dx was rounded to its type before the state's part came: half a step of the larger,
        # and sums of 4 terms of order 10 in float32
        R.close(past, want, R.U[dtype] * (want.abs() + 2 * 8) * 1.01 + 64 * R.ADD * 10, "row %d" % i)
        dw, db = dw + r[2], db + r[3]
    for got, ref in ((out["w"], dw), (out["bias"], db)):
        assert float((got.double() - ref).norm() / ref.norm()) <= 2.0 ** -15
