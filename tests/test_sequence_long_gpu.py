"""The loops that long calls of the sequence operators run in: several chunks a segment of
the scan, several groups of rows a tile of the convolution, lists from more than one tile
of block means, plans over many blocks and queries.  The host's rules are repeated here to
make sure that the sizes reach them."""
import math

import pytest
import torch

import seq_ref as R
import sparse_memory_linear_scoring_b200 as sdm
import test_conv_gpu
from test_ssm_gpu import _k, _k_state, _mag, _make

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


# ---------------------------------------------------------------- scan
def _segments(B, H, T, P, tensor):
    """Chunks a segment and segments of a head's walk."""
    nch = -(-T // (64 if tensor else 32))
    walks = B * H * (-(-P // 64) if tensor else 1)
    n = 296 // walks
    while n > 1 and n * n > 64 * nch:
        n -= 1
    n = max(1, min(n, nch))
    cps = -(-nch // n)
    return cps, -(-nch // cps)


@pytest.mark.parametrize("padded", [False, True])
@pytest.mark.parametrize("B,H,G,T,P,N,dtype,layout,several", [
    (4, 12, 2, 1500, 128, 128, BF, "token", True), (4, 12, 2, 1500, 64, 128, BF, "dense", True),
    (4, 12, 1, 1500, 64, 64, BF, "token", True), (4, 12, 3, 1500, 128, 64, BF, "token", True),
    (4, 24, 2, 700, 64, 64, BF, "odd", True), (4, 24, 1, 700, 32, 16, F32, "token", True),
    (4, 75, 1, 330, 64, 128, BF, "token", False), (4, 40, 1, 330, 128, 128, BF, "token", False),
    (4, 75, 1, 200, 16, 32, F32, "token", False)])
def test_scan_of_several_chunks(B, H, G, T, P, N, dtype, layout, several, padded):
    tensor = dtype == BF and layout != "odd" and min(P, N) >= 64
    cps, nseg = _segments(B, H, T, P, tensor)
    assert cps >= 3 and (nseg >= 2) == several
    a, _ = _make(B, H, G, T, P, N, dtype, layout)
    Q = 64 if tensor else 32
    n = [T, cps * Q + Q + 5 if several else Q + 5, 0, Q // 2] if padded else [T] * B
    live = torch.arange(T, device="cuda")[None] < torch.tensor(n, device="cuda")[:, None]
    ref = {**a, "dt": torch.where(live[:, None], a["dt"], 0.0)}
    for m in ("x", "Bm", "Cm"):
        ref[m] = torch.where(live[:, None, :, None], a[m], torch.zeros_like(a[m]))
    y, ST, _ = R.ssm(**ref)
    ym, Sm, _ = R.ssm(**_mag(ref))
    for m in ("x", "Bm", "Cm", "dt"):
        for b in range(B):
            a[m][b, :, n[b]:] = float("nan")
    S = a["S"].clone()
    lengths = torch.tensor(n, dtype=torch.int32, device="cuda") if padded else None
    got = sdm.ssm_forward(a["x"], a["dt"], a["A"], a["Bm"], a["Cm"], S, a["D"], lengths=lengths)
    y = torch.where(live[:, None, :, None], y, torch.zeros_like(y))
    R.close(got, y, _k(dtype, T, P, N) * ym, "y")
    R.close(S, ST, _k_state(T) * Sm, "S")


# ---------------------------------------------------------------- convolution
def _tile(rows, T, lo, hi, sub):
    tt = hi
    while tt > lo and rows * -(-T // (tt * sub)) * sub < 148 * 768:
        tt //= 2
    return tt


@pytest.mark.parametrize("T,d,dtype,layout", [(12001, 1280, BF, "token"), (12001, 1280, F32, "token"),
                                             (24100, 1280, BF, "dense"), (9001, 1283, BF, "odd")])
def test_convolution_of_several_groups(T, d, dtype, layout):
    one = layout == "odd"  # a channel a thread
    fwd = _tile(d if one else d // 4, T, 8, 32, 1)
    bwd = _tile(d // 4 if dtype == BF else d // 2, T, 8, 64, 4)
    assert fwd // 8 >= 2 and (bwd - 3) // 4 >= 2
    test_conv_gpu.test_forward(1, 1, T, d, 4, dtype, layout, True, True)
    test_conv_gpu.test_backward(1, 1, T, d, 4, dtype, layout, True, True)


def test_convolution_of_several_groups_padded():
    B, T, d, K = 2, 9000, 1280, 4
    assert _tile(B * d // 4, T, 8, 32, 1) >= 32
    _, x, w, b, st = test_conv_gpu._make(B, 1, T, d, K, BF, "token")
    n = [T, 4711]
    x[1, :, n[1]:] = float("nan")
    s = st.clone()
    y = sdm.conv_forward(x, w, b, s, lengths=torch.tensor(n, dtype=torch.int32, device="cuda"))
    for i, l in enumerate(n):
        ref, bound = test_conv_gpu._bound(x[i:i + 1, :, :l], w, b, st[i:i + 1], True)
        R.close(y[i:i + 1, :, :l], ref, bound, "row %d" % i)
        assert (y[i, :, l:] == 0).all() and torch.equal(s[i], x[i, :, l - K + 1:l])


# ---------------------------------------------------------------- selection
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n_sel", [1, 2, 16, 64])
@pytest.mark.parametrize("Tk,block,d", [(9000, 32, 64), (140000, 32, 32), (300000, 64, 128)])
def test_single_token_lists_of_long_caches(Tk, block, d, n_sel, dtype):
    """More blocks than one tile of 128: the kept list meets every later tile."""
    g = torch.Generator(device="cuda").manual_seed(Tk + n_sel)
    B, H, G = 4, 6, 2
    q = torch.randn(B, H, 1, d, generator=g, device="cuda").to(dtype)
    kc = torch.randn(B, G, Tk // block, d, generator=g, device="cuda").to(dtype)
    kc[1, :, ::7] = kc[1, :, 3:4]                                # ties over all tiles
    kc[2] *= torch.linspace(0.1, 2, kc.shape[2], device="cuda").to(dtype)[None, :, None]  # better ones come late
    n = torch.tensor([Tk, Tk - 77, 200 * block + 1, 1], dtype=torch.int32, device="cuda")
    for lengths in (None, n):
        idx = sdm.block_select(q, kc, n_sel=n_sel, block=block, Tk=Tk, lengths=lengths)
        assert torch.equal(idx, R.select(q, kc, n_sel, block, Tk, lengths))


# ---------------------------------------------------------------- plans
def _gathered(q, k, v, idx, block, scale, do):
    """o and the gradients over gathered keys in float64, with the sums of magnitudes; the
    lists hold distinct blocks."""
    B, H, Tq, d = q.shape
    G, Tk = k.shape[1:3]
    r = H // G
    out = {n: torch.zeros(t.shape, dtype=torch.float64, device="cuda")
           for m, t in (("o", q), ("q", q), ("k", k), ("v", v)) for n in (m, m + "_mag")}
    smag = 0.0
    pos = Tk - Tq + torch.arange(Tq, device="cuda")
    for b in range(B):
        for g in range(G):
            for t0 in range(0, Tq, 4096):
                t1, h = min(Tq, t0 + 4096), slice(g * r, (g + 1) * r)
                i = idx[b, g, t0:t1].long()
                key = (i[..., None] * block + torch.arange(block, device="cuda")).flatten(1)
                ok = (key >= 0) & (key <= pos[t0:t1, None]) & (i >= 0).repeat_interleave(block, 1)
                key = key.clamp(0, Tk - 1)
                Q, K, V, D = q[b, h, t0:t1].double(), k[b, g].double()[key], v[b, g].double()[key], do[b, h, t0:t1].double()
                e = lambda s, x, y: torch.einsum(s, x, y)  # noqa: E731
                smag = max(smag, float((e("rtd,tkd->rtk", Q.abs(), K.abs()) * ok).max()) * scale)
                P = torch.softmax((e("rtd,tkd->rtk", Q, K) * scale).masked_fill(~ok, -math.inf), -1).nan_to_num(0.0)
                o = e("rtk,tkd->rtd", P, V)
                dS = P * (e("rtd,tkd->rtk", D, V) - (D * o).sum(-1, keepdim=True)) * scale
                om = e("rtk,tkd->rtd", P, V.abs())
                mS = P * (e("rtd,tkd->rtk", D.abs(), V.abs()) + (D.abs() * om).sum(-1, keepdim=True)) * scale
                out["o"][b, h, t0:t1], out["o_mag"][b, h, t0:t1] = o, om
                out["q"][b, h, t0:t1], out["q_mag"][b, h, t0:t1] = e("rtk,tkd->rtd", dS, K), e("rtk,tkd->rtd", mS, K.abs())
                for n, x in (("k", e("rtk,rtd->tkd", dS, Q)), ("k_mag", e("rtk,rtd->tkd", mS, Q.abs())),
                             ("v", e("rtk,rtd->tkd", P, D)), ("v_mag", e("rtk,rtd->tkd", P, D.abs()))):
                    out[n][b, g].index_add_(0, key.flatten(), x.reshape(-1, d))
    return out, smag


@pytest.mark.parametrize("H,G,Tq,Tk,d,block,n_sel,dtype", [
    (2, 1, 300, 40000, 64, 32, 16, BF),       # more than 1024 blocks: the running totals of the offsets
    (2, 2, 40, 40000, 32, 32, 8, F32),
    (1, 1, 700, 140000, 32, 32, 64, BF),      # fewer warps a segment
    (1, 1, 64, 49152 * 32, 32, 32, 64, BF),   # the most blocks: one warp a segment
    (1, 1, 700, 49152 * 32, 32, 32, 64, BF),
    (1, 1, 40000, 40000, 32, 128, 2, BF),     # segments of more than 128 queries
])
def test_plans_of_long_calls(H, G, Tq, Tk, d, block, n_sel, dtype):
    g = torch.Generator(device="cuda").manual_seed(Tk)
    q, k, v, do = (torch.randn(1, h, n, d, generator=g, device="cuda").to(dtype)
                   for h, n in ((H, Tq), (G, Tk), (G, Tk), (H, Tq)))
    # the own block, then others before it: the first ones, the last ones and some between
    cur = ((Tk - Tq + torch.arange(Tq, device="cuda")) // block)[None, None, :, None]
    step = torch.randint(1, 1 + max(1, (Tk - Tq) // block // n_sel), (1, G, Tq, n_sel - 1), generator=g, device="cuda")
    idx = torch.cat([cur.expand(1, G, -1, -1), cur - torch.cumsum(step, -1)], -1)
    idx[..., 1::3] = torch.where(torch.arange(Tq, device="cuda")[:, None] % 2 == 0, idx[..., 1::3], -1)
    idx = torch.where(idx < 0, -1, idx).int().contiguous()
    ref, smag = _gathered(q, k, v, idx, block, d ** -0.5, do)
    o, lse = sdm.block_forward(q, k, v, idx, block=block, return_lse=True)
    out = sdm.block_backward(q, k, v, idx, o, lse, do, block=block)
    r = 2.0 ** -8 * 1.02 if dtype == BF else 0.0
    # scores of d additions, sums of at most 8192 listed keys in parts; backward: scores twice
    # and, a key, up to 64 R Tq / 8 additions in order
    f = 2 * d * R.ADD * smag + 2.0 ** -20 + 300 * R.ADD
    R.close(o, ref["o"], (f + r) * ref["o_mag"], "o")
    k1 = 2 * f + 2.0 ** -18 + (300 + min(Tq, 4000) * 8) * R.ADD + 2 * r
    for n in ("q", "k", "v"):
        R.close(out[n], ref[n], k1 * ref[n + "_mag"], "d" + n)
