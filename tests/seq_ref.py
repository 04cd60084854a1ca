"""Plain float64 forms of the sequence operators (torch, any device) and the error
bounds the GPU tests hold the kernels to.

Every bound is k * (the same sums over absolute values) plus one rounding of the
result to its type, half a step: finfo(t).eps / 2 relative.  k counts the roundings a
term meets: operands rounded to bf16 for the tensor cores (2^-8 each) and n float32
additions (2^-23 each: tensor-core sums may truncate)."""
import math

import torch

U = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
ADD = 2.0 ** -23


def close(got, ref, bound, what):
    """|got - ref| <= half a step of got's type + bound, elementwise; equal non-finites."""
    g, r = got.double(), ref.double()
    fin = torch.isfinite(r)
    assert torch.equal(torch.isfinite(g), fin), "%s: finite in different places" % what
    assert torch.equal(g[~fin & ~r.isnan()], r[~fin & ~r.isnan()]), what
    # the smallest normal of either type: below it a step is absolute (and may be flushed)
    lim = U[got.dtype] * r.abs() + bound + 2.0 ** -126
    bad = fin & ((g - r).abs() > lim)
    if bad.any():
        i = tuple(torch.nonzero(bad)[0].tolist())
        raise AssertionError("%s: %d of %d out, first at %s: got %r, ref %r, allowed %r" % (
            what, int(bad.sum()), bad.numel(), i, float(g[i]), float(r[i]),
            float(lim.expand_as(r)[i])))


# ---------------------------------------------------------------- convolution
def conv(x, w, b, state, silu=True):
    x, w = x.double(), w.double()
    K = w.shape[-1]
    st = x.new_zeros(*x.shape[:2], K - 1, x.shape[3]) if state is None else state.double()
    past = torch.cat([st, x], 2)
    p = torch.zeros_like(x) if b is None else b.double()[None, :, None].expand_as(x).clone()
    for i in range(K):
        p = p + past[:, :, i:i + x.shape[2]] * w[None, :, None, :, i]
    return (p * torch.sigmoid(p) if silu else p), p, past


# ---------------------------------------------------------------- scan
def ssm(x, dt, A, Bm, Cm, S, D=None):
    """(y, S_T, [S_1 .. S_T]) step by step."""
    x, dt, A, Bm, Cm, S = (t.double() for t in (x, dt, A, Bm, Cm, S))
    r = x.shape[1] // Bm.shape[1]
    Bh, Ch = Bm.repeat_interleave(r, 1), Cm.repeat_interleave(r, 1)
    a = torch.exp(dt * A[None, :, None])
    ys, keep = [], []
    for t in range(x.shape[2]):
        S = a[:, :, t, None, None] * S + (dt[:, :, t, None] * x[:, :, t])[..., None] * Bh[:, :, t, None]
        ys.append((S * Ch[:, :, t, None]).sum(-1))
        keep.append(S)
    y = torch.stack(ys, 2)
    if D is not None:
        y = y + D.double()[None, :, None, None] * x
    return y, S, keep


def ssm_grads(x, dt, A, Bm, Cm, S0, dy, dST, D, magnitude=False):
    """Gradients by the reverse walk.  With magnitude, every term enters with its size
    (absolute inputs, differences added): the sums the error bounds are made of."""
    A = A.double()
    if magnitude:
        x, Bm, Cm, S0, dy, dST = (t.double().abs() for t in (x, Bm, Cm, S0, dy, dST))
        D = None if D is None else D.abs()
    x, dt, Bm, Cm, S0, dy, R = (t.double() for t in (x, dt, Bm, Cm, S0, dy, dST))
    B, H, T, P = x.shape
    G, N = Bm.shape[1], Bm.shape[3]
    _, _, keep = ssm(x, dt, A, Bm, Cm, S0)
    Bh, Ch = Bm.repeat_interleave(H // G, 1), Cm.repeat_interleave(H // G, 1)
    a = torch.exp(dt * A[None, :, None])
    du, dB, dC = torch.zeros_like(x), torch.zeros_like(Bh), torch.zeros_like(Ch)
    q, yd, E = torch.zeros_like(dt), torch.zeros_like(dt), torch.zeros_like(dt)
    for t in range(T - 1, -1, -1):
        E[:, :, t] = (R * keep[t]).sum((-1, -2))  # what arrives from later steps
        R = R + dy[:, :, t, :, None] * Ch[:, :, t, None]
        prev = keep[t - 1] if t else S0
        du[:, :, t] = (R * Bh[:, :, t, None]).sum(-1)
        dB[:, :, t] = (R * (dt[:, :, t, None] * x[:, :, t])[..., None]).sum(-2)
        dC[:, :, t] = (keep[t] * dy[:, :, t, :, None]).sum(-2)
        yd[:, :, t] = (dC[:, :, t] * Ch[:, :, t]).sum(-1)
        R = a[:, :, t, None, None] * R
        q[:, :, t] = (R * prev).sum((-1, -2))
    xu = (x * du).sum(-1)
    if magnitude:
        # a kernel may reach q_t from the end of its chunk (at most 64 steps on), adding up
        # what lies between: every term of that sum counts
        step = yd + dt * xu
        tot = torch.cumsum(torch.cat([step, step.new_zeros(B, H, 64)], 2), 2)
        run = tot[:, :, 63:63 + T] - tot[:, :, :T] + step
        pad = torch.cat([E, E.new_zeros(B, H, 63)], 2).unfold(2, 64, 1).amax(-1)
        q, A = run + pad, A.abs()
    dx = dt[..., None] * du
    if D is not None:
        dx = dx + D.double()[None, :, None, None] * dy
    fold = lambda t: t.reshape(B, G, H // G, T, N).sum(2)  # noqa: E731
    return dict(x=dx, dt=xu + A[None, :, None] * q, A=(dt * q).sum((0, 2)), Bm=fold(dB), Cm=fold(dC),
                S0=R, D=(x * dy).sum((0, 2, 3)))


# ---------------------------------------------------------------- block attention
def positions(B, Tq, Tk, lengths, device):
    n = torch.full((B,), Tk, device=device) if lengths is None else lengths.long().clamp(0, Tk)
    return n[:, None] - Tq + torch.arange(Tq, device=device)


def pool(k, block):
    B, G, T, d = k.shape
    n = T // block
    return (k[:, :, :n * block].double().reshape(B, G, n, block, d).sum(3) / block).float().to(k.dtype)


def select(q, kc, n_sel, block, Tk, lengths=None):
    B, H, Tq, d = q.shape
    G, n = kc.shape[1], kc.shape[2]
    pos = positions(B, Tq, Tk, lengths, q.device)
    cur = torch.div(pos, block, rounding_mode="floor")
    s = q.double().reshape(B, G, H // G, Tq, d).sum(2) @ kc.double().transpose(-1, -2)
    s = torch.where(s.isnan(), torch.full_like(s, -math.inf), s)
    s = s.masked_fill((torch.arange(n, device=q.device) >= cur[..., None])[:, None], -math.inf)
    val, at = torch.sort(s, dim=-1, descending=True, stable=True)
    out = torch.full((B, G, Tq, n_sel), -1, dtype=torch.int32, device=q.device)
    out[..., 0] = torch.where(pos >= 0, cur, torch.full_like(cur, -1))[:, None]
    m = min(n_sel - 1, n)
    out[..., 1:1 + m] = torch.where(val[..., :m] > -math.inf, at[..., :m], torch.full_like(at[..., :m], -1))
    return out


def counts(idx, block, Tk, pos):
    """How often each key is listed for each query and lies at or before it."""
    B, G, Tq, _ = idx.shape
    nb = -(-Tk // block)
    i = idx.long()
    i = torch.where((i < 0) | (i >= nb), torch.full_like(i, nb), i)
    c = torch.zeros(B, G, Tq, nb + 1, dtype=torch.float64, device=idx.device)
    c.scatter_add_(-1, i, torch.ones_like(i, dtype=torch.float64))
    c = c[..., :nb].repeat_interleave(block, -1)[..., :Tk]
    return c * (torch.arange(Tk, device=idx.device) <= pos[:, None, :, None])


def block_attention(q, k, v, idx, block, scale, lengths=None, d_o=None):
    """o, lse, and with d_o the gradients; the sums of magnitudes beside each.  Keys no
    query lists take no part, whatever they hold."""
    B, H, Tq, d = q.shape
    G, Tk = k.shape[1], k.shape[2]
    r = H // G
    pos = positions(B, Tq, Tk, lengths, q.device)
    c = counts(idx, block, Tk, pos)
    used = c.sum(2) > 0
    qd = q.double().reshape(B, G, r, Tq, d)
    kd = torch.where(used[..., None], k.double(), torch.zeros((), dtype=torch.float64, device=q.device))[:, :, None]
    vd = torch.where(used[..., None], v.double(), torch.zeros((), dtype=torch.float64, device=q.device))[:, :, None]
    on = (c > 0)[:, :, None]
    s = (qd @ kd.transpose(-1, -2)) * scale
    smag = ((qd.abs() @ kd.abs().transpose(-1, -2)) * abs(scale)).masked_fill(~on, 0).amax(-1, keepdim=True)
    s = s.masked_fill(~on, -math.inf)
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    e = torch.exp(s - m) * c[:, :, None]
    l = e.sum(-1, keepdim=True)
    P = e / torch.where(l == 0, torch.ones_like(l), l)
    o = P @ vd
    lse = torch.where(l == 0, torch.full_like(l, -math.inf), m + torch.log(l))
    out = dict(o=o.reshape(B, H, Tq, d), lse=lse.reshape(B, H, Tq), smag=smag.reshape(B, H, Tq),
               o_mag=(P @ vd.abs()).reshape(B, H, Tq, d))
    if d_o is not None:
        g = d_o.double().reshape(B, G, r, Tq, d)
        dP = g @ vd.transpose(-1, -2)
        dlt = (g * o).sum(-1, keepdim=True)
        dS = P * (dP - dlt) * scale
        mS = P * (g.abs() @ vd.abs().transpose(-1, -2) + (g.abs() * (P @ vd.abs())).sum(-1, keepdim=True)) * abs(scale)
        out.update(q=(dS @ kd).reshape(B, H, Tq, d), k=(dS.transpose(-1, -2) @ qd).sum(2),
                   v=(P.transpose(-1, -2) @ g).sum(2),
                   q_mag=(mS @ kd.abs()).reshape(B, H, Tq, d),
                   k_mag=(mS.transpose(-1, -2) @ qd.abs()).sum(2),
                   v_mag=(P.transpose(-1, -2) @ g.abs()).sum(2))
    return out
