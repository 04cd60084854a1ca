"""The sequence operators together, as a model layer uses them, and the calls around them:
other streams, captured graphs, shared workspaces, refusals on the GPU's tensors, offsets
past 32 bits."""
import math

import pytest
import torch

import seq_ref as R
import sparse_memory_linear_scoring_b200 as sdm

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def _gen(seed=0):
    return torch.Generator(device="cuda").manual_seed(seed)


def _layer(B, T, H, G, P, N, dtype, seed=0):
    """A token-major projection, the filters and the scan's parameters of one layer."""
    g = _gen(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    C = H * P + 2 * G * N
    return dict(xbc=r(B, T, C).to(dtype), w=(r(1, C, 4) * 0.5).to(dtype), b=(r(1, C) * 0.1).to(dtype),
                dt=torch.nn.functional.softplus(r(B, T, H) - 3), A=-torch.exp(r(H).abs()), D=r(H) * 0.1 + 1)


def _split(y, H, G, P, N):
    """[B, 1, T, C] from the convolution: x, Bm, Cm as views."""
    B, _, T, _ = y.shape
    f = y[:, 0]
    return (f[..., :H * P].view(B, T, H, P).transpose(1, 2),
            f[..., H * P:H * P + G * N].view(B, T, G, N).transpose(1, 2),
            f[..., H * P + G * N:].view(B, T, G, N).transpose(1, 2))


def _run(p, H, G, P, N, conv_state, S, lo=0, hi=None, step=False):
    hi = p["xbc"].shape[1] if hi is None else hi
    y = sdm.conv_forward(p["xbc"][:, lo:hi].unsqueeze(1), p["w"], p["b"], conv_state)
    x, Bm, Cm = _split(y, H, G, P, N)
    dt = p["dt"][:, lo:hi].transpose(1, 2)
    if step:
        return sdm.ssm_step(x, dt, p["A"], Bm, Cm, S, p["D"])
    return sdm.ssm_forward(x, dt, p["A"], Bm, Cm, S, p["D"])


@pytest.mark.parametrize("dtype,P,N", [(BF, 64, 64), (F32, 32, 16), (BF, 128, 128)])
def test_convolution_then_scan(dtype, P, N):
    """A prompt in two pieces, then single tokens, against the whole in float64."""
    B, T, H, G = 2, 210, 4, 2
    p = _layer(B, T, H, G, P, N, dtype)
    cs = torch.zeros(B, 1, 3, H * P + 2 * G * N, dtype=dtype, device="cuda")
    S = torch.zeros(B, H, P, N, device="cuda")
    out = [_run(p, H, G, P, N, cs, S, 0, 130), _run(p, H, G, P, N, cs, S, 130, 200)]
    out += [_run(p, H, G, P, N, cs, S, t, t + 1, step=True) for t in range(200, T)]
    y = torch.cat(out, 2)
    assert torch.equal(cs[:, 0], p["xbc"][:, -3:])
    # the convolution's result is rounded to its type once: the scan starts from that
    yc = R.conv(p["xbc"].unsqueeze(1), p["w"], p["b"], None)[0].to(dtype)
    x, Bm, Cm = _split(yc, H, G, P, N)
    ref, ST, _ = R.ssm(x, p["dt"].transpose(1, 2), p["A"], Bm, Cm, torch.zeros_like(S), p["D"])
    mag, Sm, _ = R.ssm(x.abs(), p["dt"].transpose(1, 2), p["A"], Bm.abs(), Cm.abs(), torch.zeros_like(S), p["D"].abs())
    # a bf16 result of the convolution may fall on the other side of a rounding: one step,
    # 2 * 2^-8 of an operand, in each of the three factors
    k = (6 * 2.0 ** -8 + 2.0 ** -8) if dtype == BF else 2.0 ** -16
    R.close(y, ref, k * mag, "y")
    R.close(S, ST, k * Sm, "S")


def test_gradient_through_both():
    """Chained backward passes in float32 against float64's automatic ones."""
    B, T, H, G, P, N = 2, 150, 4, 2, 32, 16
    p = _layer(B, T, H, G, P, N, F32)
    g = _gen(1)
    dy = torch.randn(B, H, T, P, generator=g, device="cuda")
    xbc = p["xbc"].unsqueeze(1)
    y = sdm.conv_forward(xbc, p["w"], p["b"])
    x, Bm, Cm = _split(y, H, G, P, N)
    dt = p["dt"].transpose(1, 2)
    gs = sdm.ssm_backward(x, dt, p["A"], Bm, Cm, None, dy, D=p["D"])
    dyc = torch.cat([gs[n].transpose(1, 2).reshape(B, T, -1) for n in ("x", "Bm", "Cm")], -1)
    gc = sdm.conv_backward(xbc, p["w"], dyc.unsqueeze(1), p["b"])
    leaf = {n: v.double().requires_grad_() for n, v in p.items()}
    yc = R.conv(leaf["xbc"].unsqueeze(1), leaf["w"], leaf["b"], None)[0]
    x, Bm, Cm = _split(yc, H, G, P, N)
    S = torch.zeros(B, H, P, N, dtype=torch.float64, device="cuda")
    out, _, _ = R.ssm(x, leaf["dt"].transpose(1, 2), leaf["A"], Bm, Cm, S, leaf["D"])
    ref = dict(zip(leaf, torch.autograd.grad(out, list(leaf.values()), dy.double())))
    got = dict(xbc=gc["x"][:, 0], w=gc["w"], b=gc["bias"], dt=gs["dt"].transpose(1, 2), A=gs["A"], D=gs["D"])
    for n in got:
        # float32 sums of at most 300 terms twice over, 2^-15 of their magnitudes, and
        # magnitudes at most about 30 times the results' norm
        e = float((got[n].double() - ref[n]).norm() / ref[n].norm())
        assert e <= 30 * 2.0 ** -15, (n, e)


def _attention(q, k, v, kc, block, n_sel, lengths=None):
    idx = sdm.block_select(q, kc, n_sel=n_sel, block=block, Tk=k.shape[2], lengths=lengths)
    return idx, sdm.block_forward(q, k, v, idx, block=block, lengths=lengths)


def test_convolution_then_block_attention():
    """Queries, keys and values from one convolved projection; the cache is then read by
    padded single tokens whose means grow block by block."""
    B, T, H, G, d, block, n_sel = 2, 300, 8, 2, 64, 32, 4
    g = _gen(3)
    C = (H + 2 * G) * d
    xbc = torch.randn(B, 1, T, C, generator=g, device="cuda").to(BF)
    w = (torch.randn(1, C, 4, generator=g, device="cuda") * 0.5).to(BF)
    y = sdm.conv_forward(xbc, w, silu=False)[:, 0]
    q = y[..., :H * d].view(B, T, H, d).transpose(1, 2)
    k = y[..., H * d:(H + G) * d].view(B, T, G, d).transpose(1, 2)
    v = y[..., (H + G) * d:].view(B, T, G, d).transpose(1, 2)
    kc = sdm.block_pool(k, block=block)
    idx, o = _attention(q, k, v, kc, block, n_sel)
    assert torch.equal(kc, R.pool(k, block)) and torch.equal(idx, R.select(q, kc, n_sel, block, T))
    ref = R.block_attention(q, k, v, idx, block, d ** -0.5)
    bound = (2 * d * R.ADD * ref["smag"][..., None] + 2.0 ** -20 + 300 * R.ADD + 2.0 ** -8 * 1.02) * ref["o_mag"]
    R.close(o, ref["o"], bound, "o")
    grown = torch.zeros_like(kc)
    for t in range(0, T, 23):
        n = torch.tensor([t + 1, max(t - 40, 0) + 1], dtype=torch.int32, device="cuda")
        sdm.block_pool(k[:, :, :t + 1], grown, block=block, first=0)
        q1 = torch.stack([q[0, :, t:t + 1], q[1, :, n[1] - 1:n[1]]])
        i1, o1 = _attention(q1, k, v, grown, block, n_sel, n)
        for b, at in ((0, t), (1, int(n[1]) - 1)):
            assert torch.equal(i1[b, :, 0], idx[b, :, at])
            R.close(o1[b, :, 0], ref["o"][b, :, at], bound[b, :, at], "token %d" % at)


# ---------------------------------------------------------------- streams and graphs
def _calls(dtype=BF):
    """Every operator on its own inputs: name -> (function of a stream, clone of results)."""
    p = _layer(2, 300, 4, 2, 64, 64, dtype, seed=5)
    g = _gen(6)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").to(dtype)  # noqa: E731
    xbc = p["xbc"].unsqueeze(1)
    x, Bm, Cm = _split(xbc, 4, 2, 64, 64)
    dt, S0 = p["dt"].transpose(1, 2), torch.randn(2, 4, 64, 64, generator=g, device="cuda")
    q, k, v = r(2, 8, 700, 64), r(2, 2, 700, 64), r(2, 2, 700, 64)
    do = r(2, 8, 700, 64)
    kc = R.pool(k, 64)
    idx = R.select(q, kc, 5, 64, 700)
    dyc, dys = r(*xbc.shape), r(*x.shape)
    o, lse = sdm.block_forward(q, k, v, idx, return_lse=True)
    S, S1 = S0.clone(), S0.clone()

    def scan(stream):
        S.copy_(S0)
        return [sdm.ssm_forward(x, dt, p["A"], Bm, Cm, S, p["D"], stream=stream), S]

    def step(stream):
        S1.copy_(S0)
        return [sdm.ssm_step(x[:, :, :1], dt[:, :, :1], p["A"], Bm[:, :, :1], Cm[:, :, :1], S1, p["D"], stream=stream), S1]

    return dict(
        conv=lambda s: [sdm.conv_forward(xbc, p["w"], p["b"], stream=s)],
        conv_grad=lambda s: list(sdm.conv_backward(xbc, p["w"], dyc, p["b"], stream=s).values()),
        scan=scan, step=step,
        scan_grad=lambda s: list(sdm.ssm_backward(x, dt, p["A"], Bm, Cm, S0, dys, S0, D=p["D"], stream=s).values()),
        pool=lambda s: [sdm.block_pool(k, stream=s)],
        select=lambda s: [sdm.block_select(q, kc, n_sel=5, stream=s)],
        attend=lambda s: [sdm.block_forward(q, k, v, idx, stream=s)],
        attend_step=lambda s: [sdm.block_forward(q[:, :, -1:], k, v, idx[:, :, -1:].contiguous(), stream=s)],
        attend_grad=lambda s: list(sdm.block_backward(q, k, v, idx, o, lse, do, stream=s).values()))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_other_streams(dtype):
    """A call on a stream of its own, behind work that it has to wait for by an event, and
    two of them side by side."""
    calls = _calls(dtype)
    want = {n: [t.clone() for t in f(None)] for n, f in calls.items()}
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    for n, f in calls.items():
        if n in ("scan", "step"):
            continue  # their inputs are restored on the current stream: below
        ga, gb = f(a), f(b)
        torch.cuda.synchronize()
        for x, y, z in zip(want[n], ga, gb):
            assert torch.equal(x, y) and torch.equal(x, z), n
    for n in ("scan", "step"):
        with torch.cuda.stream(a):
            got = [t.clone() for t in calls[n](None)]
        torch.cuda.synchronize()
        for x, y in zip(want[n], got):
            assert torch.equal(x, y), n


@pytest.mark.parametrize("dtype", [BF, F32])
def test_captured_and_replayed(dtype):
    """Each operator captured into a graph and replayed twice."""
    calls = _calls(dtype)
    for n, f in calls.items():
        want = [t.clone() for t in f(None)]
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = f(None)
        for _ in range(2):
            for t in out:
                t.zero_() if t.dtype != torch.int32 else t.fill_(-5)
            graph.replay()
            torch.cuda.synchronize()
            for x, y in zip(want, out):
                assert torch.equal(x, y), n


def test_replay_reads_new_inputs_and_lengths():
    """A captured selection and attention follows its buffers: queries, cache, lengths."""
    g = _gen(8)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").to(BF)  # noqa: E731
    q, k, v = r(3, 8, 1, 64), r(3, 2, 640, 64), r(3, 2, 640, 64)
    n = torch.tensor([640, 100, 1], dtype=torch.int32, device="cuda")
    kc = sdm.block_pool(k)
    for _ in range(2):
        _attention(q, k, v, kc, 64, 4, n)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sdm.block_pool(k, kc)
        idx, o = _attention(q, k, v, kc, 64, 4, n)
    for lens in ([640, 100, 1], [65, 0, 639]):
        q.copy_(r(3, 8, 1, 64))
        k.copy_(r(3, 2, 640, 64))
        n.copy_(torch.tensor(lens, dtype=torch.int32))
        graph.replay()
        want_idx = R.select(q, R.pool(k, 64), 4, 64, 640, n)
        assert torch.equal(idx, want_idx)
        ref = R.block_attention(q, k, v, want_idx, 64, 0.125, n)
        R.close(o, ref["o"], (2.0 ** -8 * 1.02 + 2.0 ** -12) * ref["o_mag"], "o")


def test_graphs_that_share_a_workspace():
    """Two captured graphs with one workspace, replayed in turn on one stream."""
    g = _gen(9)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").to(BF)  # noqa: E731
    sets, outs, graphs, want = [], [], [], []
    ws = torch.empty(256 << 20, dtype=torch.uint8, device="cuda")
    for T in (2000, 1300):
        q, k, v = r(1, 32, T, 64), r(1, 4, T, 64), r(1, 4, T, 64)
        idx = R.select(q, R.pool(k, 64), 16, 64, T)
        sets.append((q, k, v, idx))
        want.append(sdm.block_forward(q, k, v, idx).clone())
    torch.cuda.synchronize()
    for q, k, v, idx in sets:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append(sdm.block_forward(q, k, v, idx, workspace=ws))
        graphs.append(gr)
    for i in (0, 1, 1, 0):
        graphs[i].replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[i], want[i])


# ---------------------------------------------------------------- refusals
def test_refusals_on_gpu_tensors():
    g = _gen(11)
    x = torch.randn(2, 4, 50, 64, generator=g, device="cuda").to(BF)
    w = torch.randn(4, 64, 4, generator=g, device="cuda").to(BF)
    with pytest.raises(ValueError, match="dense"):
        sdm.conv_forward(x.transpose(2, 3).contiguous().transpose(2, 3), w)
    with pytest.raises(ValueError, match="contiguous"):
        sdm.conv_forward(x, w.transpose(0, 1).contiguous().transpose(0, 1))
    with pytest.raises(ValueError, match="overlaps"):
        sdm.conv_forward(x, w, y=x)
    st = torch.zeros(2, 4, 3, 64, device="cuda", dtype=BF)
    with pytest.raises(ValueError, match="overlap"):
        sdm.conv_forward(x, w, state=st, y=x.new_zeros(2, 4, 1, 64).expand(2, 4, 50, 64))
    with pytest.raises(ValueError, match="one device|CUDA"):
        sdm.conv_forward(x, w.cpu())
    with pytest.raises(sdm.SDMError) as e:
        sdm.conv_forward(x, torch.randn(4, 64, 9, device="cuda").to(BF))
    assert e.value.code == 5
    dt, A = torch.rand(2, 4, 50, device="cuda"), -torch.rand(4, device="cuda")
    S = torch.zeros(2, 4, 64, 64, device="cuda")
    with pytest.raises(sdm.SDMError) as e:
        sdm.ssm_forward(x, dt, A, x, x, S, workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))
    assert e.value.code == 4
    with pytest.raises(ValueError, match="contiguous"):
        sdm.ssm_forward(x, dt, A, x, x, S.transpose(2, 3))
    with pytest.raises(sdm.SDMError) as e:
        sdm.ssm_backward(x[:, :, :0], dt[:, :, :0], A, x[:, :, :0], x[:, :, :0], None, x[:, :, :0])
    assert e.value.code == 2
    kc = sdm.block_pool(x, block=32)
    with pytest.raises(sdm.SDMError) as e:
        sdm.block_select(x, kc, n_sel=65, block=32)
    assert e.value.code == 5
    with pytest.raises(sdm.SDMError) as e:
        sdm.block_select(x, kc[:, :, :0], n_sel=2, block=32)
    assert e.value.code == 2
    idx = sdm.block_select(x, kc, n_sel=2, block=32)
    with pytest.raises(ValueError, match="overlaps"):
        sdm.block_forward(x, x, x, idx, block=32, o=x)
    with pytest.raises(sdm.SDMError) as e:
        sdm.block_forward(x, x, x, idx, block=32, scale=float("nan"))
    assert e.value.code == 2
    # nothing to do is not an error
    e0 = x[:, :, :0]
    assert sdm.conv_forward(e0, w).shape == e0.shape
    assert sdm.ssm_forward(e0, dt[:, :, :0], A, e0, e0, S).shape == e0.shape and (S == 0).all()
    i0 = sdm.block_select(e0, kc, n_sel=2, block=32, Tk=50)
    assert i0.shape == (2, 4, 0, 2) and sdm.block_forward(e0, x, x, i0, block=32).shape == e0.shape


def test_offsets_past_32_bits():
    """Keys whose rows lie 2 MB apart, 8.6 GB in all."""
    Tk, d, block = 4100, 64, 32
    store = torch.zeros(Tk << 20, dtype=BF, device="cuda")
    g = _gen(13)
    k0, v0 = (torch.randn(1, 1, Tk, d, generator=g, device="cuda").to(BF) for _ in range(2))
    k = store.as_strided((1, 1, Tk, d), (Tk << 20, Tk << 20, 1 << 20, 1))
    v = store.as_strided((1, 1, Tk, d), (Tk << 20, Tk << 20, 1 << 20, 1), 4096)
    k.copy_(k0)
    v.copy_(v0)
    q = torch.randn(1, 16, Tk, d, generator=g, device="cuda").to(BF)
    kc = sdm.block_pool(k, block=block)
    assert torch.equal(kc, sdm.block_pool(k0, block=block))
    n_sel = 64
    idx = sdm.block_select(q, kc, n_sel=n_sel, block=block)
    do = torch.randn(q.shape, generator=g, device="cuda").to(BF)
    for n in (1, Tk):  # a single token; enough queries for the tiles
        qn, i_n = q[:, :, -n:], idx[:, :, -n:].contiguous()
        o, lse = sdm.block_forward(qn, k, v, i_n, block=block, return_lse=True)
        o0, lse0 = sdm.block_forward(qn, k0, v0, i_n, block=block, return_lse=True)
        assert torch.equal(o, o0) and torch.equal(lse, lse0)
        a = sdm.block_backward(qn, k, v, i_n, o, lse, do[:, :, -n:], block=block)
        b = sdm.block_backward(qn, k0, v0, i_n, o, lse, do[:, :, -n:], block=block)
        for t in a:
            assert torch.equal(a[t], b[t]), t


def test_one_index_many_times():
    """The same block listed twice counts twice, in the result and in the gradient."""
    g = _gen(14)
    for T in (40, 700):
        q, k, v = (torch.randn(1, h, T, 64, generator=g, device="cuda").to(BF) for h in (16, 2, 2))
        idx = torch.zeros(1, 2, T, 33, dtype=torch.int32, device="cuda")
        do = torch.randn(q.shape, generator=g, device="cuda").to(BF)
        ref = R.block_attention(q, k, v, idx, 32, 0.125, None, do)
        o, lse = sdm.block_forward(q, k, v, idx, block=32, return_lse=True)
        R.close(o, ref["o"], (2.0 ** -8 * 1.02 + 2.0 ** -12) * ref["o_mag"], "o")
        out = sdm.block_backward(q, k, v, idx, o, lse, do, block=32)
        # two roundings of a weight and one of o in do.o, float32 sums of 33 * 8 * T terms
        for n in ("q", "k", "v"):
            R.close(out[n], ref[n], (2 * 2.0 ** -8 * 1.02 + 2.0 ** -10) * ref[n + "_mag"], "d" + n)
        assert math.isfinite(float(lse.sum()))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_calls_back_to_back(dtype):
    """Calls that follow one another without a pause, with torch's own kernels between
    them that write their inputs and overwrite their results' sources, give the bits that
    the same calls give with the device idle before each one."""
    B, T, H, G, P, N = 2, 96, 4, 2, 64, 64
    p = _layer(B, T, H, G, P, N, dtype)
    g = _gen(7)
    q = torch.randn(B, T, H, P, generator=g, device="cuda").to(dtype).transpose(1, 2)
    do = torch.randn(B, T, H, P, generator=g, device="cuda").to(dtype).transpose(1, 2)

    def chain(wait):
        out = []
        cs = torch.zeros(B, 1, 3, H * P + 2 * G * N, dtype=dtype, device="cuda")
        S = torch.zeros(B, H, P, N, device="cuda")
        xbc = p["xbc"].clone()
        for i in range(12):
            wait()
            y = sdm.conv_forward(xbc.unsqueeze(1), p["w"], p["b"], cs)
            wait()
            x, Bm, Cm = _split(y, H, G, P, N)
            dt = p["dt"].transpose(1, 2)
            o = sdm.ssm_forward(x, dt, p["A"], Bm, Cm, S, p["D"])
            wait()
            k, v = Bm, Cm
            kc = sdm.block_pool(k, block=32)
            wait()
            idx = sdm.block_select(q, kc, n_sel=2, block=32)
            wait()
            a, lse = sdm.block_forward(q, k, v, idx, block=32, return_lse=True)
            wait()
            grads = sdm.block_backward(q, k, v, idx, a, lse, do, block=32)
            wait()
            out += [t.clone() for t in (o, S, idx, a, *grads.values())]
            for t in (y, kc, a, lse):  # torch's kernels right behind the readers
                t.fill_(float("nan"))
            xbc.mul_(0.5).add_(p["xbc"], alpha=1.0 / (i + 2))
        torch.cuda.synchronize()
        return out

    for s, t in zip(chain(torch.cuda.synchronize), chain(lambda: None)):
        assert torch.equal(s, t)
        assert torch.isfinite(s.float()).all()
