"""block_pool / block_select / block_forward / block_backward against the float64 form:
head groups, block sizes, lists of every kind, chunked prompts, padded caches, values
that no query may see."""
import math

import pytest
import torch

import seq_ref as R
import sparse_memory_linear_scoring_b200 as sdm

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def _make(B, H, G, Tq, Tk, d, dtype, layout="dense", seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def t(h, n):
        if layout == "dense":
            return torch.randn(B, h, n, d, generator=g, device="cuda").to(dtype)
        off = 1 if layout == "odd" else 8
        x = torch.randn(B, n, h * d + 16, generator=g, device="cuda").to(dtype)
        return x[..., off:off + h * d].unflatten(-1, (h, d)).transpose(1, 2)

    return t(H, Tq), t(G, Tk), t(G, Tk), g


def _k(dtype, d, ref):
    """Weights: scores err by d additions of |q||k| scale (smag) and exp by 2^-21, and are
    rounded to bf16 once for the second product; sums of up to 8192 listed keys in parts."""
    n = 2 * d * R.ADD * ref["smag"][..., None] + 2.0 ** -20 + 300 * R.ADD
    return n + (2.0 ** -8 * 1.02 if dtype == BF else 0.0)


def _check_forward(q, k, v, idx, block, dtype, scale=None, lengths=None):
    d = q.shape[3]
    sc = d ** -0.5 if scale is None else scale
    ref = R.block_attention(q, k, v, idx, block, sc, lengths)
    o, lse = sdm.block_forward(q, k, v, idx, block=block, scale=scale, lengths=lengths, return_lse=True)
    R.close(o, ref["o"], _k(dtype, d, ref) * ref["o_mag"], "o")
    R.close(lse, ref["lse"], 2 * d * R.ADD * ref["smag"] + 2.0 ** -18, "lse")
    return o, lse


SHAPES = [
    # B, H, G, Tq, Tk, d, block, n_sel, dtype, layout
    (1, 1, 1, 1, 1, 64, 64, 1, BF, "dense"), (2, 4, 2, 70, 70, 64, 64, 2, BF, "token"),
    (1, 8, 2, 300, 300, 128, 64, 4, BF, "token"), (1, 6, 6, 257, 257, 64, 32, 5, BF, "dense"),
    (2, 16, 1, 130, 130, 64, 64, 3, BF, "token"), (1, 4, 2, 33, 1000, 128, 128, 4, BF, "token"),
    (1, 9, 1, 65, 400, 32, 32, 16, BF, "odd"), (1, 4, 2, 900, 900, 64, 128, 6, BF, "dense"),
    (1, 2, 1, 100, 100, 64, 64, 64, BF, "dense"), (1, 4, 4, 77, 333, 64, 32, 8, F32, "dense"),
    (2, 6, 2, 200, 200, 128, 64, 3, F32, "token"), (1, 10, 1, 50, 50, 32, 32, 2, F32, "odd"),
    (1, 2, 2, 1, 500, 128, 128, 4, F32, "dense"), (3, 4, 1, 2, 777, 64, 64, 5, BF, "dense"),
]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,G,T,d,block,layout", [
    (1, 1, 64, 64, 64, "dense"), (2, 3, 1000, 128, 64, "token"), (1, 2, 333, 32, 32, "odd"),
    (1, 1, 300, 64, 128, "dense"), (1, 1, 63, 64, 64, "dense")])
def test_pool(B, G, T, d, block, layout, dtype):
    _, k, _, _ = _make(B, G, G, 1, T, d, dtype, layout)
    kc = sdm.block_pool(k, block=block)
    ref = R.pool(k, block)
    assert kc.shape == ref.shape and kc.dtype == dtype
    assert torch.equal(kc, ref)  # the float64 sum is exact but for float32's last bits of 64
    # a growing cache: the blocks already there stay as they are
    n = T // block
    big = torch.full((B, G, n + 2, d), 7.0, dtype=dtype, device="cuda")
    sdm.block_pool(k, big, block=block, first=n // 2)
    assert torch.equal(big[:, :, n // 2:n], ref[:, :, n // 2:])
    assert (big[:, :, :n // 2] == 7).all() and (big[:, :, n:] == 7).all()


@pytest.mark.parametrize("B,H,G,Tq,Tk,d,block,n_sel,dtype,layout", SHAPES)
def test_select(B, H, G, Tq, Tk, d, block, n_sel, dtype, layout):
    q, k, _, _ = _make(B, H, G, Tq, Tk, d, dtype, layout)
    kc = sdm.block_pool(k, block=block)
    idx = sdm.block_select(q, kc, n_sel=n_sel, block=block, Tk=Tk)
    assert torch.equal(idx, R.select(q, kc, n_sel, block, Tk))


def test_select_long_and_ragged():
    q, k, _, _ = _make(3, 4, 2, 40, 9000, 64, BF)
    kc = sdm.block_pool(k, block=32)
    n = torch.tensor([9000, 25, 4111], dtype=torch.int32, device="cuda")
    idx = sdm.block_select(q, kc, n_sel=33, block=32, Tk=9000, lengths=n)
    assert torch.equal(idx, R.select(q, kc, 33, 32, 9000, n))
    assert (idx[1, :, :15] == -1).all()  # queries before the row's first key


@pytest.mark.parametrize("d,block,n_sel,Tk", [(128, 32, 64, 9000), (64, 64, 16, 3000), (32, 32, 5, 5000)])
def test_select_near_ties(d, block, n_sel, Tk):
    """Scores that differ by less than float32 sums do, equal ones, large and tiny ones."""
    q, k, _, g = _make(1, 8, 2, 300, Tk, d, BF)
    kc = sdm.block_pool(k, block=block)
    n = kc.shape[2]
    kc[:, :, 1::3] = kc[:, :, 0:-1:3][:, :, :kc[:, :, 1::3].shape[2]]     # equal pairs
    kc[:, :, 2::3, 0] = kc[:, :, 2::3, 0] * 1.0078125                     # one step of one element
    q[:, :, 100:150] *= 2.0 ** 60
    q[:, :, 150:200] *= 2.0 ** -100
    q[:, 1:4, 200:250] = -q[:, :1, 200:250] * 0.99609375                  # heads that cancel
    kc[:, 1, n // 2] *= 1000                                              # one long mean
    idx = sdm.block_select(q, kc, n_sel=n_sel, block=block, Tk=Tk)
    assert torch.equal(idx, R.select(q, kc, n_sel, block, Tk))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_select_ties_and_non_finite(dtype):
    q, k, _, _ = _make(1, 2, 1, 600, 600, 64, dtype)
    kc = sdm.block_pool(k, block=32)
    kc[:, :, 3] = kc[:, :, 1]
    kc[:, :, 9] = kc[:, :, 1]
    kc[:, :, 5] = float("nan")
    kc[:, :, 6] = 0
    q[:, :, 500] = 0                      # all scores equal
    q[0, 0, 550, 0] = float("inf")
    idx = sdm.block_select(q, kc, n_sel=8, block=32)
    assert torch.equal(idx, R.select(q, kc, 8, 32, 600))
    assert idx[0, 0, 500].tolist() == [15, 0, 1, 2, 3, 4, 6, 7]


@pytest.mark.parametrize("B,H,G,Tq,Tk,d,block,n_sel,dtype,layout", SHAPES)
def test_forward(B, H, G, Tq, Tk, d, block, n_sel, dtype, layout):
    q, k, v, _ = _make(B, H, G, Tq, Tk, d, dtype, layout)
    idx = R.select(q, R.pool(k, block), n_sel, block, Tk)
    _check_forward(q, k, v, idx, block, dtype)
    _check_forward(q, k, v, idx, block, dtype, scale=-0.3)


def _wild(B, G, Tq, nb, n_sel, g):
    """Lists as a caller may give them: any order, repeats, later blocks, no blocks."""
    idx = torch.randint(-3, nb + 3, (B, G, Tq, n_sel), generator=g, device="cuda", dtype=torch.int32)
    idx[:, :, ::5] = -1                  # rows without a key
    idx[:, :, 1::7] = idx[:, :, 1::7, :1]  # one block throughout
    idx[:, :, 3] = 2 ** 31 - 1
    idx[:, :, 2] = -2 ** 31
    return idx


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("H,G,d,block,Tq,Tk", [(4, 2, 64, 64, 200, 500), (3, 3, 128, 32, 150, 150),
                                              (2, 1, 32, 128, 300, 301)])
def test_any_lists(dtype, H, G, d, block, Tq, Tk):
    q, k, v, g = _make(2, H, G, Tq, Tk, d, dtype, "token")
    idx = _wild(2, G, Tq, -(-Tk // block), 6, g)
    o, lse = _check_forward(q, k, v, idx, block, dtype)
    assert (o[:, :, 0] == 0).all() and (lse[:, :, 0] == -math.inf).all()
    _check_backward(q, k, v, idx, block, dtype, g)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_unseen_keys_may_hold_anything(dtype):
    q, k, v, g = _make(3, 4, 2, 64, 700, 64, dtype)
    n = [700, 30, 389]
    for b, l in enumerate(n):
        k[b, :, l:] = float("nan")
        v[b, :, l:] = float("inf")
    k[0, :, 64:128] = float("inf")       # a block that no list names
    v[0, :, 64:128] = float("nan")
    lengths = torch.tensor(n, dtype=torch.int32, device="cuda")
    idx = R.select(q, R.pool(k, 64).nan_to_num(0, 0, 0), 4, 64, 700, lengths)
    idx[0] = torch.where(idx[0] == 1, torch.full_like(idx[0], -1), idx[0])
    o, lse = _check_forward(q, k, v, idx, 64, dtype, lengths=lengths)
    assert (o[1, :, :34] == 0).all() and (lse[1, :, :34] == -math.inf).all()
    d = torch.full_like(lengths, 5)
    d[0] = -4
    d[2] = 10 ** 6
    # clamped to [0, Tk]; a row of length 0 has no key at all
    o2, _ = _check_forward(torch.nan_to_num(q), torch.nan_to_num(k, 0, 0, 0), torch.nan_to_num(v, 0, 0, 0),
                           idx, 64, dtype, lengths=d)
    assert (o2[0] == 0).all()
    g_ = _check_backward(q, k, v, idx, 64, dtype, g, lengths)
    for b, l in enumerate(n):
        assert (g_["k"][b, :, l:] == 0).all() and (g_["v"][b, :, l:] == 0).all()
    assert (g_["k"][0, :, 64:128] == 0).all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("block,Tq", [(64, 200), (32, 20), (128, 200)])
def test_later_values_stay_out(dtype, block, Tq):
    """Infinite and NaN keys and values behind a query, in a block that it lists, leave it
    as it is; the queries that see them do get them."""
    q, k, v, _ = _make(1, 4, 2, Tq, 200, 64, dtype)
    idx = R.select(q, R.pool(k, block), 3, block, 200)
    ref = R.block_attention(q, k, v, idx, block, 0.125)
    first = 200 - Tq
    v[:, 0, 185] = float("inf")
    v[:, 0, 190, :5] = float("nan")
    k[:, 1, 195] = float("nan")
    o = sdm.block_forward(q, k, v, idx, block=block)
    for h, end in ((0, 185), (1, 185), (2, 195), (3, 195)):
        n = end - first
        one = {x: ref[x][:, h:h + 1, :n] for x in ("o", "o_mag", "smag")}
        R.close(o[:, h:h + 1, :n], one["o"], _k(dtype, 64, one) * one["o_mag"], "head %d" % h)
    lists = (idx[0, 0] == 185 // block).any(-1)  # the queries of group 0 that list the keys' block
    mid, end = o[:, :2, 185 - first:190 - first], o[0, :2, 190 - first:][:, lists[190 - first:]]
    assert lists[185 - first:190 - first].all() and (mid == math.inf).all()
    assert end[..., :5].isnan().all() and (end[..., 5:] == math.inf).all()
    assert o[:, 2:, 195 - first:].isnan().all()


def _check_backward(q, k, v, idx, block, dtype, g, lengths=None, scale=None):
    d = q.shape[3]
    sc = d ** -0.5 if scale is None else scale
    d_o = torch.randn(q.shape, generator=g, device="cuda").to(dtype)
    ref = R.block_attention(q, k, v, idx, block, sc, lengths, d_o)
    o, lse = sdm.block_forward(q, k, v, idx, block=block, scale=scale, lengths=lengths, return_lse=True)
    out = sdm.block_backward(q, k, v, idx, o, lse, d_o, block=block, scale=scale, lengths=lengths)
    # P and its products: the scores' error twice (own and lse), one rounding of P or ds to
    # bf16 for the product, one of o in do.o; up to 64 R Tq / 8 additions a key, in order
    smag = float(ref["smag"].max())
    k1 = 4 * d * R.ADD * smag + 2.0 ** -18 + (300 + idx.shape[2] * 8) * R.ADD
    if dtype == BF:
        k1 += 2 * 2.0 ** -8 * 1.02
    for n in ("q", "k", "v"):
        assert out[n].dtype == dtype and out[n].shape == {"q": q, "k": k, "v": v}[n].shape
        R.close(out[n], ref[n], k1 * ref[n + "_mag"], "d" + n)
    return out


@pytest.mark.parametrize("B,H,G,Tq,Tk,d,block,n_sel,dtype,layout", SHAPES)
def test_backward(B, H, G, Tq, Tk, d, block, n_sel, dtype, layout):
    q, k, v, g = _make(B, H, G, Tq, Tk, d, dtype, layout)
    idx = R.select(q, R.pool(k, block), n_sel, block, Tk)
    _check_backward(q, k, v, idx, block, dtype, g)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("block,Tq", [(64, 200), (32, 20), (128, 200)])
def test_backward_later_keys_stay_out(dtype, block, Tq):
    """Infinite and NaN keys and values behind a query leave its gradient as it is."""
    q, k, v, g = _make(1, 4, 2, Tq, 200, 64, dtype)
    idx = R.select(q, R.pool(k, block), 3, block, 200)
    d_o = torch.randn(q.shape, generator=g, device="cuda").to(dtype)
    o, lse = sdm.block_forward(q, k, v, idx, block=block, return_lse=True)
    good = sdm.block_backward(q, k, v, idx, o, lse, d_o, block=block)
    k[:, 0, 195, :5], k[:, 1, 193], v[:, :, 196] = float("inf"), float("nan"), float("nan")
    o, lse = sdm.block_forward(q, k, v, idx, block=block, return_lse=True)
    got = sdm.block_backward(q, k, v, idx, o, lse, d_o, block=block)
    assert torch.equal(got["q"][:, :, :Tq - 7], good["q"][:, :, :Tq - 7])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_small_values(dtype):
    """Values and their gradients near the bottom of the type's range."""
    q, k, v, g = _make(1, 4, 2, 150, 150, 64, dtype)
    idx = R.select(q, R.pool(k, 64), 3, 64, 150)
    v = (v.float() * 2.0 ** -124).to(dtype)
    o = sdm.block_forward(q, k, v, idx)
    ref = R.block_attention(q, k, v, idx, 64, 0.125)
    R.close(o, ref["o"], _k(dtype, 64, ref) * ref["o_mag"], "o")


@pytest.mark.parametrize("Tq", [1, 150, 700])
def test_scale_zero(Tq):
    """Equal weights over the listed keys."""
    q, k, v, g = _make(2, 16, 4, Tq, 700, 128, BF)
    idx = R.select(q, R.pool(k, 64), 9, 64, 700)
    _check_forward(q, k, v, idx, 64, BF, scale=0.0)


@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("block", [32, 64, 128])
def test_tiles(d, block):
    """Enough listed keys for the block-by-block kernels at every width and block, items
    of several row tiles, blocks that some queries see in part, long and short rows."""
    q, k, v, g = _make(2, 12, 2, 1500, 1777, d, BF, "token")
    n = torch.tensor([1777, 1201], dtype=torch.int32, device="cuda")
    idx = R.select(q, R.pool(k, block), 24, block, 1777, n)
    v[0, 0, 800], v[0, 0, 1000, 3], v[1, 1, 7, 1] = float("inf"), float("nan"), float("-inf")
    ref = R.block_attention(q, k, v, idx, block, 0.3, n)
    o, lse = sdm.block_forward(q, k, v, idx, block=block, scale=0.3, lengths=n, return_lse=True)
    # float64 products spread a NaN or infinity to every query of the group: compare the
    # groups without one, and the others where their lists leave those keys out
    for b, h0 in ((0, 6), (1, 0)):
        one = {x: ref[x][b:b + 1, h0:h0 + 6] for x in ("o", "o_mag", "smag")}
        R.close(o[b:b + 1, h0:h0 + 6], one["o"], _k(BF, d, one) * one["o_mag"], "o %d" % b)
    clean = v.clone()
    clean[0, 0, 800] = clean[0, 0, 1000, 3] = clean[1, 1, 7, 1] = 0
    ref = R.block_attention(q, k, clean, idx, block, 0.3, n)
    R.close(lse, ref["lse"], 2 * d * R.ADD * ref["smag"] + 2.0 ** -18, "lse")
    pos = R.positions(2, 1500, 1777, n, q.device)
    c = R.counts(idx, block, 1777, pos)
    out = torch.where((c[0, 0, :, 800] + c[0, 0, :, 1000] > 0)[None, :, None], ref["o"][0, :6], o[0, :6].double())
    one = {x: ref[x][0, :6] for x in ("o", "o_mag", "smag")}
    R.close(out.to(BF), one["o"], (_k(BF, d, one) + 2.0 ** -8) * one["o_mag"], "o of rows without such keys")
    inf, nan = c[0, 0, :, 800] > 0, c[0, 0, :, 1000] > 0
    got = o[0, :6]
    assert (got[:, inf & ~nan] == math.inf).all() and got[:, nan, 3].isnan().all()
    assert torch.equal(o[1, 6:, :, 1] == -math.inf, (c[1, 1, :, 7] > 0)[None].expand(6, -1))


def test_many_passes():
    """Lists so long that queries are taken in passes, with repeated entries."""
    q, k, v, g = _make(8, 64, 4, 300, 300, 128, BF)
    idx = torch.randint(-1, 4, (8, 4, 300, 64), generator=g, device="cuda", dtype=torch.int32)
    _check_forward(q, k, v, idx, 128, BF)
    _check_backward(q, k, v, idx, 128, BF, g)


def test_backward_is_the_slope():
    q, k, v, g = _make(1, 4, 2, 90, 90, 32, F32)
    idx = R.select(q, R.pool(k, 32), 2, 32, 90)
    d_o = torch.randn(q.shape, generator=g, device="cuda")
    o, lse = sdm.block_forward(q, k, v, idx, block=32, return_lse=True)
    out = sdm.block_backward(q, k, v, idx, o, lse, d_o, block=32)
    for n, t in (("q", q), ("k", k), ("v", v)):
        w = torch.randn(t.shape, generator=g, device="cuda")
        h = 1e-2

        def f(s):
            a = {"q": q, "k": k, "v": v, n: t + s * h * w}
            return float((sdm.block_forward(a["q"], a["k"], a["v"], idx, block=32).double() * d_o.double()).sum())

        slope, got = (f(1) - f(-1)) / (2 * h), float((out[n].double() * w.double()).sum())
        size = float(out[n].double().norm() * w.double().norm())
        assert abs(slope - got) <= 5e-3 * size, (n, slope, got)


@pytest.mark.parametrize("H,G", [(4, 4), (16, 2)])
def test_single_tokens_equal_prompt(H, G):
    """A cache read one query at a time against the prompt's rows."""
    q, k, v, _ = _make(2, H, G, 200, 200, 64, BF)
    kc = sdm.block_pool(k, block=32)
    idx = sdm.block_select(q, kc, n_sel=4, block=32)
    ref = R.block_attention(q, k, v, idx, 32, 0.125)
    for t in (0, 31, 32, 150, 199):
        n = torch.full((2,), t + 1, dtype=torch.int32, device="cuda")
        q1 = q[:, :, t:t + 1]
        i1 = sdm.block_select(q1, kc, n_sel=4, block=32, Tk=200, lengths=n)
        assert torch.equal(i1, idx[:, :, t:t + 1])
        o = sdm.block_forward(q1, k, v, i1, block=32, lengths=n)
        one = {x: ref[x][:, :, t:t + 1] for x in ("smag", "o_mag", "o")}
        R.close(o, one["o"], _k(BF, 64, one) * one["o_mag"], "o at %d" % t)


def test_equal_calls_give_equal_bits():
    q, k, v, g = _make(1, 8, 2, 2000, 2000, 64, BF)
    idx = sdm.block_select(q, sdm.block_pool(k), n_sel=8)
    d_o = torch.randn(q.shape, generator=g, device="cuda").to(BF)
    runs = []
    for _ in range(2):
        o, lse = sdm.block_forward(q, k, v, idx, return_lse=True)
        runs.append(dict(sdm.block_backward(q, k, v, idx, o, lse, d_o), o=o, lse=lse))
    for n in runs[0]:
        assert torch.equal(runs[0][n], runs[1][n]), n
