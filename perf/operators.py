"""What the sequence operators are measured on: short causal convolution, selective
state space scan, and sparse attention over selected blocks, each in a plain form
(elementary torch operations) and through the package's entry points."""
import math

import numpy as np
import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # decoding: one token for each of 64 sequences, 16 heads of 64 channels (the high-batch workload)
        dict(name="conv_step_b64", op="conv", mode="step", B=64, T=1, H=16, d=64, K=4, dtype="bf16", ragged=False),
        # a padded batch of prompts, token-major projection of 8 heads and one B/C group
        dict(name="conv_prompt_ragged", op="conv", mode="prompt", B=4, T=2048, H=1, d=640, K=4, dtype="bf16", ragged=True),
        # training on long sequences: forward and backward, 8 heads of 128 and one group of B and C
        dict(name="conv_train_long", op="conv", mode="train", B=1, T=65536, H=1, d=1280, K=4, dtype="bf16", ragged=False),
        # decoding: one token for each of 64 sequences, 16 heads, state 64 x 64
        dict(name="ssm_step_b64", op="ssm", mode="step", B=64, H=16, G=1, T=1, P=64, N=64, dtype="bf16", ragged=False),
        # a prompt at the pages-scale workload's heads and length, few heads and a long axis
        dict(name="ssm_prompt_pages", op="ssm", mode="prompt", B=2, H=4, G=1, T=8192, P=64, N=64, dtype="bf16", ragged=False),
        # the long-context workload's length and widths
        dict(name="ssm_prompt_long", op="ssm", mode="prompt", B=1, H=8, G=1, T=65536, P=128, N=128, dtype="bf16", ragged=False),
        # a training step of the "small" workload, forward and backward, two B/C groups
        dict(name="ssm_train_small", op="ssm", mode="train", B=4, H=8, G=2, T=2048, P=64, N=64, dtype="bf16", ragged=False),
        # training in float32, odd length and narrow widths
        dict(name="ssm_train_f32_odd", op="ssm", mode="train", B=1, H=3, G=1, T=777, P=32, N=16, dtype="f32", ragged=False),
        # decoding against caches of different lengths
        dict(name="block_step_b64", op="block", mode="step", B=64, H=16, G=4, Tq=1, Tk=4096, d=64, block=64, n_sel=16, dtype="bf16", ragged=True),
        # a whole prompt, 16 heads on 4 key heads
        dict(name="block_prompt_pages", op="block", mode="prompt", B=2, H=16, G=4, Tq=8192, Tk=8192, d=128, block=64, n_sel=16, dtype="bf16", ragged=False),
        # a training step, forward and backward
        dict(name="block_train_small", op="block", mode="train", B=4, H=8, G=2, Tq=2048, Tk=2048, d=64, block=64, n_sel=8, dtype="bf16", ragged=False),
        # a prompt's later chunk in float32, odd lengths, one head per key head, small blocks
        dict(name="block_chunk_f32_odd", op="block", mode="prompt", B=1, H=4, G=4, Tq=333, Tk=2777, d=64, block=32, n_sel=8, dtype="f32", ragged=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["conv", "ssm", "block"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "conv":
        mode = rng.choice(["step", "prompt", "train"])
        H, d = rng.choice([(16, 64), (8, 128), (1, _log(rng, 40, 1280)), (1, 8 * _log(rng, 8, 160))])
        B = _log(rng, 1, 128) if mode == "step" else rng.randint(1, 4)
        T = 1 if mode == "step" else _log(rng, 2, 16384)
        return dict(op=op, mode=mode, B=B, T=T, H=H, d=d, K=rng.choice([2, 3, 4, 4]), dtype=dtype,
                    ragged=mode == "prompt" and rng.random() < 0.5)
    if op == "ssm":
        mode = rng.choice(["step", "prompt", "train"])
        G = rng.choice([1, 1, 2])
        H = G * rng.randint(1, 6)
        B = _log(rng, 1, 64) if mode == "step" else rng.randint(1, 3)
        T = rng.choice([1, 1, 3]) if mode == "step" else _log(rng, 5, 8192 if mode == "prompt" else 4096)
        return dict(op=op, mode=mode, B=B, H=H, G=G, T=T, P=rng.choice([32, 64, 64, 128]), N=rng.choice([16, 64, 128, 128]),
                    dtype=dtype, ragged=mode == "prompt" and rng.random() < 0.5)
    mode = rng.choice(["step", "prompt", "train"])
    G = rng.choice([1, 2, 4])
    H = G * rng.choice([1, 2, 4, 7])
    block = rng.choice([32, 64, 64, 128])
    d = rng.choice([32, 64, 128])
    B = _log(rng, 1, 64) if mode == "step" else rng.randint(1, 2)
    Tk = _log(rng, 50, 8192) if mode == "step" else _log(rng, 50, 4096)
    Tq = 1 if mode == "step" else Tk if mode == "train" or rng.random() < 0.5 else max(2, Tk // rng.randint(2, 9))
    return dict(op=op, mode=mode, B=B, H=H, G=G, Tq=Tq, Tk=Tk, d=d, block=block, n_sel=rng.choice([2, 5, 8, 16]), dtype=dtype,
                ragged=mode == "step" and rng.random() < 0.5)


# ---------------------------------------------------------------- inputs
def _lengths(c, T, gen):
    """Lengths of a padded batch, from a tenth of T to all of it."""
    n = torch.randint(max(1, T // 10), T + 1, (c["B"],), device="cuda", generator=gen, dtype=torch.int32)
    n[0] = T
    return n


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    dt = _DT[c["dtype"]]

    def rn(*shape, sd=1.0):
        return (torch.randn(*shape, device="cuda", generator=gen) * sd).to(dt)

    def r32(*shape, sd=1.0):
        return torch.randn(*shape, device="cuda", generator=gen) * sd

    s = {"c": c}
    B, H = c["B"], c["H"]
    if c["op"] == "conv":
        T, d, K = c["T"], c["d"], c["K"]
        # token-major, as a projection writes it; the operator sees [B, H, T, d]
        s["x"] = rn(B, T, H, d).transpose(1, 2)
        s["w"] = rn(H, d, K, sd=K ** -0.5)
        s["bias"] = rn(H, d, sd=0.1)
        s["lengths"] = _lengths(c, T, gen) if c["ragged"] else None
        if c["mode"] == "train":
            s["dy"] = rn(B, T, H, d).transpose(1, 2)
        else:
            s["state"] = rn(B, H, K - 1, d)
        return s
    if c["op"] == "ssm":
        T, P, N, G = c["T"], c["P"], c["N"], c["G"]
        # x, B and C are slices of one token-major projection
        xbc = rn(B, T, H * P + 2 * G * N)
        s["x"] = xbc[..., :H * P].view(B, T, H, P).transpose(1, 2)
        s["Bm"] = xbc[..., H * P:H * P + G * N].view(B, T, G, N).transpose(1, 2)
        s["Cm"] = xbc[..., H * P + G * N:].view(B, T, G, N).transpose(1, 2)
        # decays as such layers are initialised: dt log-uniform in [0.001, 0.1], A in [-16, -1]
        u = torch.rand(B, T, H, device="cuda", generator=gen)
        s["dt"] = torch.exp(u * math.log(100.0) + math.log(0.001)).transpose(1, 2)
        s["A"] = -torch.exp(torch.rand(H, device="cuda", generator=gen) * math.log(16.0))
        s["D"] = r32(H) * 0.1 + 1.0
        s["S"] = r32(B, H, P, N, sd=0.5)
        s["lengths"] = _lengths(c, T, gen) if c["ragged"] else None
        if c["mode"] == "train":
            s["dy"] = rn(B, T, H, P).transpose(1, 2)
            s["dS"] = r32(B, H, P, N, sd=0.1)
        return s
    Tq, Tk, d, G, bs = c["Tq"], c["Tk"], c["d"], c["G"], c["block"]
    nb = -(-Tk // bs)
    # keys drift from block to block, and queries look for some block's direction
    topic = r32(B, G, nb, d, sd=0.8)
    k = r32(B, G, Tk, d, sd=0.7) + topic.repeat_interleave(bs, 2)[:, :, :Tk]
    pick = torch.randint(0, nb, (B, G, Tq), device="cuda", generator=gen)
    want = torch.gather(topic, 2, pick[..., None].expand(-1, -1, -1, d)).repeat_interleave(H // G, 1)
    s["q"] = (r32(B, H, Tq, d, sd=0.8) + want).to(dt)
    s["k"] = k.to(dt)
    s["v"] = rn(B, G, Tk, d)
    s["lengths"] = _lengths(c, Tk, gen) if c["ragged"] else None
    if c["mode"] == "train":
        s["do"] = rn(B, H, Tq, d)
    if c["mode"] == "step":  # block means are kept beside the cache
        s["kc"] = _pool(s["k"], bs)
    return s


# ---------------------------------------------------------------- plain forms
def _silu(x):
    return x / (1 + torch.exp(-x))


def _conv(x, w, bias, state):
    """Pre-activation and padded input in float32; state: the K - 1 inputs before x."""
    K = w.shape[-1]
    xp = torch.cat([state, x], 2)
    return (xp.unfold(2, K, 1) * w[:, None]).sum(-1) + bias[:, None], xp


def _run_conv(s):
    c = s["c"]
    x, K = s["x"], c["K"]
    if c["mode"] == "train":
        with torch.enable_grad():
            x, w, b = (t.detach().float().requires_grad_() for t in (s["x"], s["w"], s["bias"]))
            p, _ = _conv(x, w, b, torch.zeros_like(x[:, :, :1]).expand(-1, -1, K - 1, -1))
            y = _silu(p)
            dx, dw, db = torch.autograd.grad(y, (x, w, b), s["dy"].float())
        return y.detach().to(s["x"].dtype), dx.to(s["x"].dtype), dw, db
    p, xp = _conv(x.float(), s["w"].float(), s["bias"].float(), s["state"].float())
    y = _silu(p)
    T = x.shape[2]
    if s["lengths"] is None:
        new = xp[:, :, T:]
    else:
        n = s["lengths"].long()
        y = torch.where(torch.arange(T, device="cuda")[None, None, :, None] < n[:, None, None, None], y, torch.zeros_like(y))
        at = n[:, None, None, None] + torch.arange(K - 1, device="cuda")[None, None, :, None]
        new = torch.gather(xp, 2, at.expand(-1, xp.shape[1], -1, xp.shape[3]))
    s["state"].copy_(new)
    return y.to(x.dtype), s["state"]


def _ssm(x, dt, A, Bm, Cm, S, D):
    """The scan over chunks of 64 steps, decays in float64: y and the last state."""
    B, H, T, P = x.shape
    G, N = Bm.shape[1], Bm.shape[-1]
    Q = 64
    n = -(-T // Q)
    pad = n * Q - T

    def chunks(t):
        t = torch.cat([t, t.new_zeros(*t.shape[:2], pad, *t.shape[3:])], 2) if pad else t
        return t.reshape(*t.shape[:2], n, Q, *t.shape[3:])

    xc, dc = chunks(x), chunks(dt)
    Bc, Cc = (chunks(t).repeat_interleave(H // G, 1) for t in (Bm, Cm))
    la = dc.double() * A.double()[None, :, None, None]
    g = torch.cumsum(la, -1)
    low = torch.ones(Q, Q, dtype=torch.bool, device=x.device).tril()
    neg = torch.tensor(-math.inf, dtype=torch.float64, device=x.device)
    W = torch.exp(torch.where(low, g[..., :, None] - g[..., None, :], neg)).float()
    M = (Cc @ Bc.transpose(-1, -2)) * W * dc[..., None, :]
    local = (xc * (torch.exp(g[..., -1:] - g).float() * dc)[..., None]).transpose(-1, -2) @ Bc
    # states between chunks: every earlier chunk's part decayed to the chunk's start
    e = torch.cat([torch.zeros_like(g[:, :, :1, 0]), torch.cumsum(g[..., -1], -1)], -1)
    below = torch.ones(n + 1, n + 1, dtype=torch.bool, device=x.device).tril()
    E = torch.exp(torch.where(below, e[..., :, None] - e[..., None, :], neg)).float()
    parts = torch.cat([S[:, :, None], local], 2).reshape(B, H, n + 1, P * N)
    states = (E @ parts).reshape(B, H, n + 1, P, N)
    y = M @ xc + torch.exp(g).float()[..., None] * (Cc @ states[:, :, :-1].transpose(-1, -2))
    y = (y + D[None, :, None, None, None] * xc).reshape(B, H, n * Q, P)[:, :, :T]
    return y, states[:, :, -1]


def _run_ssm(s):
    c = s["c"]
    dt = s["x"].dtype
    if c["mode"] == "train":
        with torch.enable_grad():
            a = [s[n].detach().float().requires_grad_() for n in ("x", "dt", "A", "Bm", "Cm", "S", "D")]
            y, S = _ssm(*a)
            g = torch.autograd.grad((y, S), a, (s["dy"].float(), s["dS"]))
        return [y.detach().to(dt), S.detach()] + [t.to(dt) if n in ("x", "Bm", "Cm") else t
                                                 for n, t in zip(("x", "dt", "A", "Bm", "Cm", "S", "D"), g)]
    x, d = s["x"].float(), s["dt"]
    if s["lengths"] is not None:
        live = torch.arange(c["T"], device="cuda")[None, None, :] < s["lengths"][:, None, None]
        d = torch.where(live, d, torch.zeros_like(d))
    y, S = _ssm(x, d, s["A"], s["Bm"].float(), s["Cm"].float(), s["S"], s["D"])
    if s["lengths"] is not None:
        y = torch.where(live[..., None], y, torch.zeros_like(y))
    if c["mode"] == "step":
        s["S"].copy_(S)
        S = s["S"]
    return y.to(dt), S


def _pool(k, bs):
    """Means of the complete blocks, summed in float64 and rounded once."""
    B, G, T, d = k.shape
    n = T // bs
    return k[:, :, :n * bs].double().reshape(B, G, n, bs, d).mean(3).to(k.dtype)


def _positions(c, lengths):
    """Position of every query: the last Tq of the keys."""
    n = torch.full((c["B"],), c["Tk"], device="cuda") if lengths is None else lengths.long()
    return n[:, None] - c["Tq"] + torch.arange(c["Tq"], device="cuda")


def _select(c, q, kc, lengths):
    """Current block, then the best earlier ones by summed score (float64, ties to the lowest index), -1 behind."""
    B, G, n = c["B"], c["G"], kc.shape[2]
    pos = _positions(c, lengths)
    cur = torch.div(pos, c["block"], rounding_mode="floor")
    qs = q.double().reshape(B, G, c["H"] // G, c["Tq"], c["d"]).sum(2)
    sc = qs @ kc.double().transpose(-1, -2)
    at = torch.arange(n, device="cuda")
    sc = torch.where((at < cur[..., None])[:, None], sc, torch.full_like(sc, -math.inf))
    top, idx = torch.sort(sc, dim=-1, descending=True, stable=True)
    m = min(c["n_sel"] - 1, n)
    idx = torch.where(top[..., :m] > -math.inf, idx[..., :m], torch.full_like(idx[..., :m], -1))
    cur = torch.where(pos >= 0, cur, torch.full_like(cur, -1))[:, None, :, None].expand(-1, G, -1, -1)
    out = torch.cat([cur, idx, idx.new_full((B, G, c["Tq"], c["n_sel"] - 1 - m), -1)], -1)
    return out.to(torch.int32)


def _attend(c, q, k, v, idx, lengths):
    """Softmax over the keys of the listed blocks up to the query's position: dense scores under a mask."""
    B, G, Tk, bs = c["B"], c["G"], c["Tk"], c["block"]
    nb = -(-Tk // bs)
    sel = torch.zeros(B, G, c["Tq"], nb + 1, dtype=torch.bool, device="cuda")
    i = idx.long()
    sel.scatter_(-1, torch.where(i < 0, torch.full_like(i, nb), i), True)
    ok = sel[..., :nb].repeat_interleave(bs, -1)[..., :Tk]
    ok = ok & (torch.arange(Tk, device="cuda") <= _positions(c, lengths)[:, None, :, None])
    qg = q.reshape(B, G, c["H"] // G, c["Tq"], c["d"])
    sc = (qg @ k[:, :, None].transpose(-1, -2)) * c["d"] ** -0.5
    sc = torch.where(ok[:, :, None], sc, torch.full((), -math.inf, device="cuda"))
    m = sc.detach().amax(-1, keepdim=True)
    p = torch.exp(sc - torch.where(m == -math.inf, torch.zeros_like(m), m))
    o = (p @ v[:, :, None]) / p.sum(-1, keepdim=True).clamp_min(1e-30)
    return o.reshape(B, c["H"], c["Tq"], c["d"])


def _run_block(s):
    c = s["c"]
    kc = s["kc"] if c["mode"] == "step" else _pool(s["k"], c["block"])
    idx = _select(c, s["q"], kc, s["lengths"])
    dt = s["q"].dtype
    if c["mode"] == "train":
        with torch.enable_grad():
            a = [s[n].detach().float().requires_grad_() for n in ("q", "k", "v")]
            o = _attend(c, *a, idx, s["lengths"])
            g = torch.autograd.grad(o, a, s["do"].float())
        return [idx, o.detach().to(dt)] + [t.to(dt) for t in g]
    return idx, _attend(c, s["q"].float(), s["k"].float(), s["v"].float(), idx, s["lengths"]).to(dt)


# ---------------------------------------------------------------- the package's entry points
def _own(s):
    import sparse_memory_linear_scoring_b200 as sdm
    c = s["c"]
    if c["op"] == "conv":
        if c["mode"] == "train":
            y = sdm.conv_forward(s["x"], s["w"], s["bias"])
            g = sdm.conv_backward(s["x"], s["w"], s["dy"], s["bias"])
            return y, g["x"], g["w"], g["bias"]
        return sdm.conv_forward(s["x"], s["w"], s["bias"], s["state"], lengths=s["lengths"]), s["state"]
    if c["op"] == "ssm":
        args = [s[n] for n in ("x", "dt", "A", "Bm", "Cm")]
        if c["mode"] == "step":
            return sdm.ssm_step(*args, s["S"], s["D"]), s["S"]
        S = s["S"].clone()
        y = sdm.ssm_forward(*args, S, s["D"], lengths=s["lengths"])
        if c["mode"] == "prompt":
            return y, S
        g = sdm.ssm_backward(*args, s["S"], s["dy"], s["dS"], D=s["D"])
        return [y, S] + [g[n] for n in ("x", "dt", "A", "Bm", "Cm", "S0", "D")]
    kc = s["kc"] if c["mode"] == "step" else sdm.block_pool(s["k"], block=c["block"])
    idx = sdm.block_select(s["q"], kc, n_sel=c["n_sel"], block=c["block"], Tk=c["Tk"], lengths=s["lengths"])
    if c["mode"] == "train":
        o, lse = sdm.block_forward(s["q"], s["k"], s["v"], idx, block=c["block"], return_lse=True)
        g = sdm.block_backward(s["q"], s["k"], s["v"], idx, o, lse, s["do"], block=c["block"])
        return [idx, o, g["q"], g["k"], g["v"]]
    return idx, sdm.block_forward(s["q"], s["k"], s["v"], idx, block=c["block"], lengths=s["lengths"])


def run(state):
    if own:
        return _own(state)
    return {"conv": _run_conv, "ssm": _run_ssm, "block": _run_block}[state["c"]["op"]](state)


# ---------------------------------------------------------------- what cannot be left out
def work(case):
    c = case
    e = 2 if c["dtype"] == "bf16" else 4
    B, H = c["B"], c["H"]
    if c["op"] == "conv":
        n, ch, K = B * c["T"] * H * c["d"], H * c["d"], c["K"]
        if c["mode"] == "train":  # x and dy in, y and dx out
            return {"bytes": 4 * n * e + ch * (K + 1) * (e + 4), "flops": n * (6 * K + 20)}
        return {"bytes": 2 * n * e + 2 * B * ch * (K - 1) * e + ch * (K + 1) * e, "flops": n * (2 * K + 5)}
    if c["op"] == "ssm":
        P, N = c["P"], c["N"]
        th, tg, st = B * H * c["T"], B * c["G"] * c["T"], B * H * P * N * 4
        if c["mode"] == "train":  # x, dy, B, C, dt, S, dS in; y, dx, dB, dC, ddt, S, dS0 out
            return {"bytes": th * (4 * P * e + 8) + tg * 4 * N * e + 4 * st, "flops": th * 16 * P * N}
        return {"bytes": th * (2 * P * e + 4) + tg * 2 * N * e + 2 * st, "flops": th * 5 * P * N}
    Tq, Tk, d, bs, G = c["Tq"], c["Tk"], c["d"], c["block"], c["G"]
    pos = np.arange(Tk - Tq, Tk, dtype=np.int64)
    cur = pos // bs
    keys = np.minimum(cur, c["n_sel"] - 1) * bs + pos % bs + 1
    mean = 0.55 if c["ragged"] else 1.0  # ragged lengths are uniform from a tenth to all
    rows, cand = B * H * float(keys.sum()) * (mean if c["mode"] == "step" else 1.0), B * G * float(cur.sum()) * mean
    seen = min(float(Tk) * mean, float(keys.sum()))  # keys that some query lists
    kv = B * G * (seen if c["mode"] == "step" else Tk) * d * e
    means = cand if c["mode"] == "step" else B * G * (Tk // bs)
    byt = 2 * B * H * Tq * d * e + 2 * kv + means * d * e + B * G * Tq * c["n_sel"] * 4
    if c["mode"] == "train":
        return {"bytes": byt + 2 * B * H * Tq * d * e + 2 * kv, "flops": 14 * d * rows + 2 * d * cand}
    return {"bytes": byt, "flops": 4 * d * rows + 2 * d * cand}


# ---------------------------------------------------------------- from the definitions, in float64
def exact(case, seed):
    def exact_conv(s):
        c = s["c"]
        B, T, H, d, K = (c[n] for n in ("B", "T", "H", "d", "K"))
        x, w, b = s["x"].double(), s["w"].double(), s["bias"].double()
        st = s["state"].double() if c["mode"] != "train" else x.new_zeros(B, H, K - 1, d)
        past = torch.cat([st, x], 2)
        p = b[None, :, None].expand(B, H, T, d).clone()
        for i in range(K):
            p += past[:, :, i:i + T] * w[None, :, None, :, i]
        sg = torch.sigmoid(p)
        y = p * sg
        if c["mode"] == "train":
            dp = s["dy"].double() * (sg + y * (1 - sg))
            dx = torch.zeros_like(past)
            dw = torch.zeros_like(w)
            for i in range(K):
                dx[:, :, i:i + T] += dp * w[None, :, None, :, i]
                dw[..., i] = (dp * past[:, :, i:i + T]).sum((0, 2))
            return y, dx[:, :, K - 1:], dw, dp.sum((0, 2))
        if s["lengths"] is None:
            return y, past[:, :, T:]
        new = torch.empty_like(st)
        for i, n in enumerate(s["lengths"].tolist()):
            y[i, :, n:] = 0
            new[i] = past[i, :, n:n + K - 1]
        return y, new

    def exact_ssm(s):
        """Step by step. Training: the states of the forward walk are kept, and the walk back reads them."""
        c = s["c"]
        B, H, G, T, P, N = (c[n] for n in ("B", "H", "G", "T", "P", "N"))
        x, dt, A, D, S = (s[n].double() for n in ("x", "dt", "A", "D", "S"))
        Bm, Cm = s["Bm"].double(), s["Cm"].double()
        if s["lengths"] is not None:
            live = torch.arange(T, device="cuda")[None, :] < s["lengths"][:, None]
            dt = dt * live[:, None]
        a = torch.exp(dt * A[None, :, None])
        u = x * dt[..., None]
        Bh, Ch = Bm.repeat_interleave(H // G, 1), Cm.repeat_interleave(H // G, 1)
        y = torch.empty_like(x)
        keep = x.new_empty(T, B, H, P, N) if c["mode"] == "train" else None
        S = S.clone()
        for t in range(T):
            S.mul_(a[:, :, t, None, None]).addcmul_(u[:, :, t, :, None], Bh[:, :, t, None, :])
            y[:, :, t] = (S @ Ch[:, :, t, :, None])[..., 0]
            if keep is not None:
                keep[t] = S
        y += D[None, :, None, None] * x
        if s["lengths"] is not None:
            y = y * live[:, None, :, None]
        if c["mode"] != "train":
            return y, S
        dy, R = s["dy"].double(), s["dS"].double().clone()
        du, dBh, dCh = torch.empty_like(x), torch.empty_like(Bh), torch.empty_like(Ch)
        la = torch.empty_like(dt)
        S0 = s["S"].double()
        for t in range(T - 1, -1, -1):
            R.addcmul_(dy[:, :, t, :, None], Ch[:, :, t, None, :])
            prev = keep[t - 1] if t else S0
            du[:, :, t] = (R @ Bh[:, :, t, :, None])[..., 0]
            dBh[:, :, t] = (u[:, :, t, None, :] @ R)[..., 0, :]
            dCh[:, :, t] = (dy[:, :, t, None, :] @ keep[t])[..., 0, :]
            R.mul_(a[:, :, t, None, None])
            la[:, :, t] = (R * prev).sum((-1, -2))
        dx = du * dt[..., None] + dy * D[None, :, None, None]
        ddt = (du * x).sum(-1) + la * A[None, :, None]
        fold = lambda t: t.reshape(B, G, H // G, T, N).sum(2)  # noqa: E731
        return [y, S, dx, ddt, (la * dt).sum((0, 2)), fold(dBh), fold(dCh), R, (dy * x).sum((0, 2, 3))]

    def exact_block(s):
        """Query by query in tiles, over gathered keys."""
        c = s["c"]
        B, H, G, Tq, Tk, d, bs, n_sel = (c[n] for n in ("B", "H", "G", "Tq", "Tk", "d", "block", "n_sel"))
        r, train = H // G, c["mode"] == "train"
        kc = s["kc"].double() if "kc" in s else None
        if kc is None:
            n = Tk // bs
            kc = (s["k"][:, :, :n * bs].double().reshape(B, G, n, bs, d).sum(3) / bs).to(s["k"].dtype).double()
        o = torch.zeros(B, H, Tq, d, dtype=torch.float64, device="cuda")
        dq, dk, dv = torch.zeros_like(o), *(torch.zeros(B, G, Tk, d, dtype=torch.float64, device="cuda") for _ in range(2))
        lens = [Tk] * B if s["lengths"] is None else s["lengths"].tolist()
        tile = max(1, min(Tq, (1 << 26) // (n_sel * bs * d)))
        for b in range(B):
            for g in range(G):
                K, V, means = s["k"][b, g].double(), s["v"][b, g].double(), kc[b, g]
                for t0 in range(0, Tq, tile):
                    t1 = min(Tq, t0 + tile)
                    q = s["q"][b, g * r:(g + 1) * r, t0:t1].double()
                    p = lens[b] - Tq + torch.arange(t0, t1, device="cuda")
                    cur = torch.div(p, bs, rounding_mode="floor")
                    sc = torch.einsum("rtd,nd->tn", q, means)
                    sc[torch.arange(means.shape[0], device="cuda") >= cur[:, None]] = -math.inf
                    m = min(n_sel - 1, means.shape[0])
                    val, at = torch.topk(sc, m, -1)
                    blocks = torch.cat([cur[:, None], torch.where(val > -math.inf, at, torch.full_like(at, -1))], -1)
                    key = (blocks[..., None] * bs + torch.arange(bs, device="cuda")).flatten(1)
                    good = (key >= 0) & (key <= p[:, None]) & (blocks >= 0).repeat_interleave(bs, 1)
                    key = key.clamp(0, Tk - 1)
                    Kg, Vg = K[key], V[key]
                    sm = torch.einsum("rtd,tkd->rtk", q, Kg) / math.sqrt(d)
                    sm = sm.masked_fill(~good, -math.inf)
                    w = torch.softmax(sm, -1).nan_to_num(0.0)
                    out = torch.einsum("rtk,tkd->rtd", w, Vg)
                    o[b, g * r:(g + 1) * r, t0:t1] = out
                    if train:
                        do = s["do"][b, g * r:(g + 1) * r, t0:t1].double()
                        dw = torch.einsum("rtd,tkd->rtk", do, Vg)
                        ds = w * (dw - (do * out).sum(-1, keepdim=True)) / math.sqrt(d)
                        dq[b, g * r:(g + 1) * r, t0:t1] = torch.einsum("rtk,tkd->rtd", ds, Kg)
                        flat = key.flatten()
                        dk[b, g].index_add_(0, flat, torch.einsum("rtk,rtd->tkd", ds, q).reshape(-1, d))
                        dv[b, g].index_add_(0, flat, torch.einsum("rtk,rtd->tkd", w, do).reshape(-1, d))
        return [None, o, dq, dk, dv] if train else (None, o)

    c = case
    if c["op"] == "ssm" and c["mode"] == "train" and c["T"] * c["B"] * c["H"] * c["P"] * c["N"] * 8 > 24e9:
        return None  # the kept states would not fit
    s = prepare(case, seed)
    return {"conv": exact_conv, "ssm": exact_ssm, "block": exact_block}[c["op"]](s)
