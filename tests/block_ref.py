"""The attention-block operators in float64, from their definitions, each with a
bound on the error of a float32 computation of it.

Every bound counts roundings: U = 2^-24 is half a float32 step, `half(t)` half a
step of the stored type (bf16 2^-8, fp16 2^-11, fp32 2^-24).  A sum of n float32
terms in any order is off by at most n U times the sum of their magnitudes; the
magnitudes are computed here, in float64, beside the values.
"""
import math

import torch

U = 2.0 ** -24
# float32's smallest normal value.  2^x is 0 or a subnormal for x < -126, off by less than
# this; a weight of 1e-59 is therefore 0 in float32, whatever the kernel does.
UNDER = 2.0 ** -126


def half(dtype):
    return torch.finfo(dtype).eps / 2


def tiny(dtype):
    """Half of the smallest step of the type (results below its normal range)."""
    f = torch.finfo(dtype)
    return f.tiny * f.eps / 2 if dtype != torch.float32 else UNDER


def check(got, ref, bound, label):
    """|got - ref| <= bound + half a step of ref in got's type, element by element."""
    assert got.shape == ref.shape, f"{label}: shape {tuple(got.shape)} vs {tuple(ref.shape)}"
    assert torch.isfinite(got.float()).all(), f"{label}: non-finite values"
    ref = ref.double().cpu()
    err = (got.double().cpu() - ref).abs()
    lim = bound.double().cpu() + half(got.dtype) * (ref.abs() + bound.double().cpu()) + tiny(got.dtype)
    worst = (err - lim).max() if err.numel() else torch.tensor(-1.0)
    assert worst <= 0, (f"{label}: |got - ref| exceeds its bound by {float(worst):.3e} "
                        f"(largest error {float(err.max()):.3e}, "
                        f"{float((err / lim).max()):.2f} of the bound)")


# ---------------------------------------------------------------- rotary positions

def rope(x, pos, freqs, pairs, interleaved, inverse=False, grad_out=None):
    """(out, bound), or with grad_out ((grad_x, bound), (grad_pos, bound))."""
    x, pos, f = x.double().cpu(), pos.double().cpu(), freqs.double().cpu()
    axis = torch.repeat_interleave(torch.arange(len(pairs)), torch.tensor(pairs))
    th = (pos[..., axis] * f)[:, :, None] * (-1.0 if inverse else 1.0)
    R = f.numel()

    def split(t):
        if interleaved:
            return t[..., 0:2 * R:2], t[..., 1:2 * R:2], t[..., 2 * R:]
        return t[..., :R], t[..., R:2 * R], t[..., 2 * R:]

    def join(a, b, rest):
        both = torch.stack([a, b], -1).flatten(-2) if interleaved else torch.cat([a, b], -1)
        return torch.cat([both, rest], -1)

    def turn(t, th):
        a, b, rest = split(t)
        out = join(a * th.cos() - b * th.sin(), a * th.sin() + b * th.cos(), rest)
        # the angle is within 2^-25 of a turn (2 pi 2^-26 rad of rounding), sine and cosine
        # within two steps, then two products and a sum: 12 roundings cover them
        mag = torch.hypot(a, b)
        return out, 12 * U * join(mag, mag, torch.zeros_like(rest))

    if grad_out is None:
        return turn(x, th)
    g = grad_out.double().cpu()
    ga, gb, _ = split(g)
    oa, ob, _ = split(turn(x, th)[0])
    N = x.shape[0]
    shared = pos.shape[0] == 1 and N > 1
    term = f * (gb * oa - ga * ob) * (-1.0 if inverse else 1.0)
    mag = f.abs() * (torch.hypot(ga, gb) * torch.hypot(oa, ob))
    dims = (0, 2) if shared else (2,)
    per = term.sum(dims, keepdim=True)[:, :, 0]
    pmag = mag.sum(dims, keepdim=True)[:, :, 0]
    A = len(pairs)
    gp = torch.zeros(per.shape[0], x.shape[1], A, dtype=torch.float64).index_add(2, axis, per)
    pm = torch.zeros_like(gp).index_add(2, axis, pmag)
    terms = x.shape[2] * max(max(pairs), 1) * (N if shared else 1)
    return turn(g, -th), (gp, (terms + 24) * U * pm)


# ------------------------------------------------------------ differential attention

def visible(N, Lq, Lk, mask, lengths, causal):
    j = torch.arange(Lk)
    n = torch.full((N,), Lk) if lengths is None else lengths.cpu().long().clamp(0, Lk)
    see = (j < n[:, None])[:, None, :].expand(N, Lq, Lk).clone()
    if causal:
        see &= j <= torch.arange(Lq)[:, None] + (n[:, None, None] - Lq)
    if mask is not None:
        see &= ~mask.cpu().bool()[:, None, :]
    return see                                        # [N, Lq, Lk]


def attn(q, k, v, lam, mask=None, lengths=None, causal=False, scale=None, grad_out=None):
    """Dict name -> (value, bound): out, maps, lse and, with grad_out, q, k, v, lam."""
    dt = q.dtype
    N, Lq, M, _, D = q.shape
    Lk, Mk, Dv = v.shape[1:]
    G = M // Mk
    scale = D ** -0.5 if scale is None else scale
    see = visible(N, Lq, Lk, mask, lengths, causal)[:, None, None, None]
    kept = see.any(dim=-2)[:, 0, 0, 0]                # [N, Lk]: keys some token sees
    f64 = (lambda t: t.double().cpu())
    q, k, v, lam = f64(q), f64(k), f64(v), f64(lam)
    k = k.where(kept[:, :, None, None, None], torch.zeros(()).double())
    v = v.where(kept[:, :, None, None], torch.zeros(()).double())
    Q = q.view(N, Lq, Mk, G, 2, D).permute(0, 2, 3, 4, 1, 5)       # [N,Mk,G,2,Lq,D]
    K = k.permute(0, 2, 3, 1, 4)[:, :, None]                       # [N,Mk,1,2,Lk,D]
    V = v.permute(0, 2, 1, 3)[:, :, None]                          # [N,Mk,1,Lk,Dv]
    l = lam.view(Mk, G, 1, 1)
    s = (Q @ K.transpose(-1, -2) * scale).masked_fill(~see, -math.inf)
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - top.clamp_min(-1e300))
    tot = p.sum(-1, keepdim=True)
    p = p / tot.clamp_min(1e-300)
    # a score's error: D products and the scale, then the exponential's argument is a
    # difference of two such scores in base 2, itself rounded (|score| log2 e U each)
    mag = (Q.abs() @ K.abs().transpose(-1, -2) * abs(scale)).masked_fill(~see, 0.0)
    ds = (D + 6) * U * mag.amax(-1, keepdim=True)                  # [N,Mk,G,2,Lq,1]
    rel = 2 * ds + (Lk + 24) * U                                   # of a normalised weight
    up = half(dt) if dt != torch.float32 else 0.0                  # weights rounded for the product
    under = UNDER * see                                            # weights that vanish in float32
    rp = rel + up
    heads = (lambda t: t.permute(0, 3, 1, 2, 4).reshape(N, Lq, M, -1))
    O = p.unbind(3)
    o0, o1 = O[0] @ V, O[1] @ V
    a0, a1 = O[0] @ V.abs(), O[1] @ V.abs()
    lost = under[:, :, :, 0].double() @ V.abs()
    b0 = (rp[:, :, :, 0] + (Lk + 8) * U) * a0 + lost
    b1 = (rp[:, :, :, 1] + (Lk + 8) * U) * a1 + lost
    out, bout = o0 - l * o1, b0 + l.abs() * b1 + 4 * U * (a0 + l.abs() * a1)
    lse = ((top + torch.log(tot)) * math.log2(math.e))[..., 0]     # [N,Mk,G,2,Lq]
    lse = torch.where(tot[..., 0] > 0, lse, torch.full_like(lse, math.inf)).reshape(N, M, 2, Lq)
    blse = ((2 * ds[..., 0] + (Lk + 24) * U) * 1.5).reshape(N, M, 2, Lq) + 4 * U * lse.abs()
    r = {"out": (heads(out), heads(bout)), "maps": (torch.stack([heads(o0), heads(o1)], 3), torch.stack([heads(b0), heads(b1)], 3)), "lse": (lse, blse)}
    if grad_out is None:
        return r
    g = f64(grad_out).view(N, Lq, Mk, G, Dv).permute(0, 2, 3, 1, 4)
    dp, mdp = g @ V.transpose(-1, -2), g.abs() @ V.abs().transpose(-1, -2)
    e = torch.stack([(g * o0).sum(-1), (g * o1).sum(-1)], 3)[..., None]          # [N,Mk,G,2,Lq,1]
    s1, s0 = b1 + 2 * U * o1.abs(), b0 + 2 * U * o0.abs()       # the saved outputs are float32
    be = torch.stack([(g.abs() * s0).sum(-1), (g.abs() * s1).sum(-1)], 3)[..., None]
    be = be + (Dv + 8) * U * torch.stack([(g.abs() * o0.abs()).sum(-1),
                                          (g.abs() * o1.abs()).sum(-1)], 3)[..., None]
    sign = torch.stack([torch.ones_like(l), -l], 2)                              # [Mk,G,2,1,1]
    x = dp[:, :, :, None] - e
    t = sign * p * x
    bx = (Dv + 4) * U * mdp[:, :, :, None] + be + 2 * U * (dp[:, :, :, None].abs() + e.abs())
    # weights from the saved lse carry twice the score's error; in 16 bits a score gradient is
    # rounded to the type, fp16 ones scaled so that the largest they could be is 2^14 or more
    bt = sign.abs() * p * (bx * (1 + 2 * rel) + (2 * rel + 4 * U) * x.abs()) + up * t.abs()
    bt = bt + under * sign.abs() * x.abs() + under
    if dt == torch.float16:
        most = 2 * (g.norm(dim=-1).max() if g.numel() else torch.tensor(0.0).double()) * (
            V.norm(dim=-1).max() if V.numel() else torch.tensor(0.0).double()) * (1 + lam.abs().max())
        bt = bt + (2.0 ** -25 * 2.0 ** -14 * most) * see
    both = O[0] - l * O[1]
    bboth = (2 * rel[:, :, :, 0] * O[0] + l.abs() * 2 * rel[:, :, :, 1] * O[1]
             + (up + 2 * U) * (O[0] + l.abs() * O[1]) + under[:, :, :, 0] * (1 + l.abs())) + (2.0 ** -25 * see[:, :, :, 0] if dt == torch.float16 else 0.0)
    rows = Lq * G + 8
    gq = scale * (t @ K)
    bq = abs(scale) * ((bt + (Lk + 8) * U * t.abs()) @ K.abs())
    T = (lambda z: z.transpose(-1, -2))
    gk = scale * (T(t) @ Q).sum(2)
    bk = abs(scale) * (T(bt + rows * U * t.abs()) @ Q.abs()).sum(2)
    gv = (T(both) @ g).sum(2)
    bv = (T(bboth + rows * U * both.abs()) @ g.abs()).sum(2)
    gl = -e[:, :, :, 1].sum(dim=(0, 3, 4)).view(M)
    bl = (be[:, :, :, 1] + (N * Lq + 8) * U * (g.abs() * a1).sum(-1, keepdim=True)).sum(dim=(0, 3, 4)).view(M)
    back = (lambda z: z.permute(0, 4, 1, 2, 3, 5).reshape(N, Lq, M, 2, D))
    keys = (lambda z: z.permute(0, 3, 1, 2, 4))
    r.update(q=(back(gq), back(bq)), k=(keys(gk), keys(bk)),
             v=(gv.permute(0, 2, 1, 3), bv.permute(0, 2, 1, 3)), lam=(gl, bl))
    return r


# ------------------------------------------------------------------- residual joins

def _norm(t, rms, eps):
    """Normalised rows, reciprocal spread, and the error of a normalised value: the
    sums run over at most 8 values, 5 shuffles and 32 warps (48 roundings); a mean
    error of 48 U mean|t| shifts every value by that over the spread."""
    m = t.mean(-1, keepdim=True)
    c = t if rms else t - m
    r = (c.square().mean(-1, keepdim=True) + eps).rsqrt()
    n = c * r
    shift = torch.zeros_like(m) if rms else 48 * U * t.abs().mean(-1, keepdim=True) * r
    return n, r, 64 * U * n.abs() + shift * (1 + n.abs())


def join(x, y, f, norm="layer", post=True, pre=True, eps=1e-6):
    """{"z": (value, bound), "h": (value, bound)}; f: the factors by name, None where absent."""
    rms = norm == "rms"
    d = {k: None if t is None else t.double().cpu() for k, t in f.items()}
    one = torch.ones((), dtype=torch.float64)
    x, y = x.double().cpu(), y.double().cpu()
    fac = (one if d.get("scale") is None else d["scale"]) * (
        one if d.get("gate") is None else d["gate"][:, None])
    n1, _, b1 = _norm(y, rms, eps) if post else (y, None, torch.zeros_like(y))
    w = one if d.get("post_weight") is None else d["post_weight"]
    b = 0 * one if d.get("post_bias") is None else d["post_bias"]
    u, bu = n1 * w + b, b1 * w.abs() + 4 * U * ((n1 * w).abs() + b.abs())
    z, bz = x + fac * u, fac.abs() * bu + 4 * U * (x.abs() + (fac * u).abs())
    r = {"z": (z, bz)}
    if pre:
        n2, r2, b2 = _norm(z, rms, eps)
        w = one if d.get("pre_weight") is None else d["pre_weight"]
        b = 0 * one if d.get("pre_bias") is None else d["pre_bias"]
        # z's own error moves the statistics too
        b2 = b2 + r2 * (bz + (1 + n2.abs()) * bz.mean(-1, keepdim=True) +
                        n2.abs() * (bz * n2.abs()).mean(-1, keepdim=True))
        r["h"] = (n2 * w + b, b2 * w.abs() + 4 * U * ((n2 * w).abs() + b.abs()))
    return r


def join_grad(y, z, gz, gh, f, norm="layer", post=True, pre=True, eps=1e-6):
    """Gradients by name with bounds, from y and the stored z."""
    rms = norm == "rms"
    d = {k: None if t is None else t.double().cpu() for k, t in f.items()}
    one = torch.ones((), dtype=torch.float64)
    get = (lambda k, other: other * one if d.get(k) is None else d[k])
    y, z, g = y.double().cpu(), z.double().cpu(), gz.double().cpu()
    scale = get("scale", 1.0)
    gate = one if d.get("gate") is None else d["gate"][:, None]
    mean = (lambda t: t.mean(-1, keepdim=True))

    def back(v, bv, n, r, bn):
        m1, m2 = (0 * mean(v) if rms else mean(v)), mean(v * n)
        val = r * (v - m1 - n * m2)
        mm = mean(v.abs())
        mn = mean((v * n).abs())
        err = r * (bv + mean(bv) + n.abs() * mean(bv * n.abs() + v.abs() * bn) + bn * m2.abs()
                   + 64 * U * (mm + n.abs() * mn))
        rel = mean(bn * n.abs()) + 64 * U        # of the reciprocal spread
        return val, err + rel * r * (v.abs() + mm + n.abs() * mn)

    res = {}
    bg = torch.zeros_like(g)
    if pre:
        n2, r2, b2 = _norm(z, rms, eps)
        h = gh.double().cpu()
        v = h * get("pre_weight", 1.0)
        val, err = back(v, 2 * U * v.abs(), n2, r2, b2)
        g, bg = g + val, err + 2 * U * (g.abs() + val.abs())
        rows = h.shape[0] * h.shape[1] + 64
        res["pre_weight"] = ((h * n2).sum((0, 1)),
                             (h.abs() * b2 + rows * U * (h * n2).abs()).sum((0, 1)))
        res["pre_bias"] = (h.sum((0, 1)), rows * U * h.abs().sum((0, 1)))
    res["x"] = (g, bg)
    n1, r1, b1 = _norm(y, rms, eps) if post else (y, None, torch.zeros_like(y))
    w, b = get("post_weight", 1.0), get("post_bias", 0.0)
    rows = g.shape[0] * g.shape[1] + 64
    # the factors' gradients come from the column sums of g n1 and of g
    A, B = (g * n1), g
    bA = bg * n1.abs() + g.abs() * b1 + rows * U * A.abs()
    bB = bg + rows * U * g.abs()
    t = (w * A + b * B).sum(1)
    bt = (w.abs() * (bA + 4 * U * A.abs()) + b.abs() * (bB + 4 * U * B.abs())).sum(1)
    gt = torch.ones_like(t) if d.get("gate") is None else d["gate"]
    res["gate"] = (scale * t, scale.abs() * bt + 4 * U * (scale * t).abs())
    res["scale"] = ((gt * t).sum(0), (gt.abs() * bt * (1 + rows * U)).sum(0))
    gs = gt * scale
    res["post_weight"] = ((gs * A.sum(1)).sum(0), (gs.abs() * bA.sum(1)).sum(0) * (1 + 8 * U) +
                          rows * U * (gs.abs() * A.abs().sum(1)).sum(0))
    res["post_bias"] = ((gs * B.sum(1)).sum(0), (gs.abs() * bB.sum(1)).sum(0) * (1 + 8 * U) +
                        rows * U * (gs.abs() * B.abs().sum(1)).sum(0))
    gu, bgu = g * scale * gate, (scale * gate).abs() * bg + 4 * U * (g * scale * gate).abs()
    if post:
        res["y"] = back(gu * w, bgu * w.abs() + 2 * U * (gu * w).abs(), n1, r1, b1)
    else:
        res["y"] = (gu, bgu)
    return res
