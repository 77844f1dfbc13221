"""The attention-block operators that surround the deformable samplers, as measured cases.

Three operators, each forward and backward:

  axial_rope     rotary positions over one to four axes (row and column of a
                 feature map's cell, frame of a video, index in a sequence)
  diff_attn      differential attention, the difference of two softmax maps
                 with a learned weight per head; grouped key / value heads, key
                 padding masks, per-image key counts, causal order
  norm_residual  the join of two blocks: the norm after a block, its per-image
                 gate and its learned residual scale, the addition to the
                 residual stream, and the norm before the next block

`run` computes a case in its plain form (elementary torch operations in float32,
float64 for the angles) when `own` is false, and with this package's calls when
it is true.  `exact` computes the same outputs in float64 from the definitions.
"""
import math

import torch

own = False

DEV = "cuda"
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # one new token a sequence, 16 sequences: the step of a serving loop
        {"name": "rope_step_bf16", "op": "rope", "dtype": "bf16", "N": 16, "T": 1, "H": 1, "W": 1, "M": 16,
         "D": 64, "axes": 3, "rotated": 32, "interleaved": False, "grad": False, "far": True},
        # queries of a deformable encoder: every cell of a 100 x 150 map, 8 heads of 32
        {"name": "rope_map_f32", "op": "rope", "dtype": "f32", "N": 2, "T": 1, "H": 100, "W": 150, "M": 8,
         "D": 32, "axes": 2, "rotated": 16, "interleaved": True, "grad": False, "far": False},
        # video tokens in training: gradients of the tokens and of the positions
        {"name": "rope_video_grad_bf16", "op": "rope", "dtype": "bf16", "N": 2, "T": 8, "H": 37, "W": 41, "M": 16,
         "D": 64, "axes": 3, "rotated": 32, "interleaved": False, "grad": True, "far": False},
        # one new token a sequence over caches that are half to wholly full
        {"name": "attn_step_bf16", "op": "attn", "dtype": "bf16", "N": 16, "Lq": 1, "Lk": 8192, "M": 16, "Mk": 4,
         "D": 64, "Dv": 128, "causal": True, "lengths": True, "grid_w": 0, "train": False},
        # self-attention of a detection decoder's 300 object queries
        {"name": "attn_queries_f16", "op": "attn", "dtype": "f16", "N": 2, "Lq": 300, "Lk": 300, "M": 4, "Mk": 4,
         "D": 32, "Dv": 64, "causal": False, "lengths": False, "grid_w": 0, "train": False},
        # a long prompt
        {"name": "attn_prompt_bf16", "op": "attn", "dtype": "bf16", "N": 1, "Lq": 8192, "Lk": 8192, "M": 16,
         "Mk": 4, "D": 64, "Dv": 128, "causal": True, "lengths": False, "grid_w": 0, "train": False},
        # float32 attention over the cells of a 25 x 38 map, padded images
        {"name": "attn_map_f32", "op": "attn", "dtype": "f32", "N": 2, "Lq": 950, "Lk": 950, "M": 8, "Mk": 8,
         "D": 32, "Dv": 32, "causal": False, "lengths": False, "grid_w": 38, "train": False},
        # a training step of a sequence model: forward and every gradient
        {"name": "attn_train_bf16", "op": "attn", "dtype": "bf16", "N": 2, "Lq": 4096, "Lk": 4096, "M": 8, "Mk": 4,
         "D": 64, "Dv": 128, "causal": True, "lengths": False, "grid_w": 0, "train": True},
        # a training step over a 50 x 75 map, padded images, odd length
        {"name": "attn_train_map_f16", "op": "attn", "dtype": "f16", "N": 2, "Lq": 3750, "Lk": 3750, "M": 4, "Mk": 4,
         "D": 32, "Dv": 64, "causal": False, "lengths": False, "grid_w": 75, "train": True},
        # the joins of a serving step, 16 sequences of one token
        {"name": "norm_step_f16", "op": "norm", "dtype": "f16", "N": 16, "L": 1, "C": 1024, "rms": True,
         "bias": False, "gate": False, "post": True, "pre": True, "grad": False},
        # the first stage of a convolutional backbone: 64 images of 56 x 56 x 64, layer norms and layer scale
        {"name": "norm_stage_f16", "op": "norm", "dtype": "f16", "N": 64, "L": 3136, "C": 64, "rms": False,
         "bias": True, "gate": False, "post": True, "pre": True, "grad": False},
        # a training step of a block of 1024 channels, gated per image
        {"name": "norm_train_bf16", "op": "norm", "dtype": "bf16", "N": 8, "L": 4096, "C": 1024, "rms": True,
         "bias": False, "gate": True, "post": True, "pre": True, "grad": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "attn", "attn", "norm"])
    dtype = rng.choice(["f32", "f16", "bf16", "bf16"])
    if op == "rope":
        D = rng.choice([16, 32, 64, 80, 128])
        axes = rng.randint(1, 3)
        T = rng.randint(1, 8) if axes == 3 else 1
        return {"op": op, "dtype": dtype, "N": rng.randint(1, 4), "T": T, "H": 1 if axes == 1 else _log(rng, 1, 40),
                "W": _log(rng, 1, 90), "M": rng.randint(1, 16), "D": D, "axes": axes,
                "rotated": D // 2 - rng.choice([0, 0, 4]), "interleaved": rng.random() < 0.5,
                "grad": rng.random() < 0.5, "far": axes == 1}
    if op == "norm":
        C = rng.choice([rng.randint(4, 130) * 8, _log(rng, 16, 4096)])
        return {"op": op, "dtype": dtype, "N": rng.randint(1, 8), "L": _log(rng, 1, 2500), "C": C,
                "rms": rng.random() < 0.5, "bias": rng.random() < 0.5, "gate": rng.random() < 0.5,
                "post": rng.random() < 0.8, "pre": rng.random() < 0.8, "grad": rng.random() < 0.5}
    D, Dv = rng.choice([(32, 32), (32, 64), (64, 64), (64, 128), (64, 128), (128, 128)])
    Mk = rng.choice([1, 2, 4])
    step = rng.random() < 0.3
    train = not step and rng.random() < 0.5
    if train and D == 128:
        D, Dv = 64, 128
    big = 700 if dtype == "f32" else 2500
    c = {"op": op, "dtype": dtype, "N": rng.randint(1, 3), "M": Mk * rng.choice([1, 2, 4]), "Mk": Mk, "D": D,
         "Dv": Dv, "causal": rng.random() < 0.5, "lengths": False, "grid_w": 0, "train": train}
    if step:
        c.update(Lq=rng.randint(1, 4), Lk=_log(rng, 5, 12000), causal=True, lengths=rng.random() < 0.7)
    elif rng.random() < 0.4:
        w = _log(rng, 4, 48)
        c.update(Lk=w * _log(rng, 4, big // w), grid_w=w, causal=False)
        c.update(Lq=c["Lk"])
    else:
        c.update(Lk=_log(rng, 30, big))
        c.update(Lq=c["Lk"] if rng.random() < 0.6 else _log(rng, 30, big))
        c.update(causal=c["causal"] and c["Lq"] <= c["Lk"])
    return c


# ------------------------------------------------------------------ the inputs

def _pairs(c):
    """Rotated channel pairs of each axis: even shares, the rest to the last axes."""
    r, a = c["rotated"], c["axes"]
    return [r // a + (1 if i >= a - r % a else 0) for i in range(a)]


def _valid(c):
    """Cells that are no padding, per image: image n keeps 1, 7/8, 3/4, 1, ... of its rows and columns."""
    h, w = c["Lk"] // c["grid_w"], c["grid_w"]
    return [(max(1, math.ceil(h * (8 - n % 3) / 8)), max(1, math.ceil(w * (8 - (n + n // 3) % 3) / 8)))
            for n in range(c["N"])]


def _key_counts(c):
    """Valid keys of each sequence: from half of the cache to all of it."""
    if not c["lengths"]:
        return [c["Lk"]] * c["N"]
    lo = max(c["Lq"], c["Lk"] // 2)
    return [lo + (c["Lk"] - lo) * (n + 1) // c["N"] for n in range(c["N"])]


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV).manual_seed(int(seed))
    dt = DT[c["dtype"]]

    def normal(*shape, std=1.0, mean=0.0, dtype=dt):
        return (torch.randn(shape, generator=g, device=DEV) * std + mean).to(dtype)

    s = {"case": c}
    if c["op"] == "rope":
        T, H, W = c["T"], c["H"], c["W"]
        L = T * H * W
        s["x"] = normal(c["N"], L, c["M"], c["D"])
        cell = torch.arange(L, device=DEV)
        grid = torch.stack([cell // (H * W), cell // W % H, cell % W], dim=-1).float()
        # cell centres, each image's map at its own place
        place = torch.randint(0, 100000 if c["far"] else 32, (c["N"], 1, c["axes"]), generator=g, device=DEV)
        s["pos"] = (grid[:, 3 - c["axes"]:] + 0.5 + place).contiguous()
        base = 10000.0 if c["far"] else 100.0
        s["freqs"] = torch.cat([base ** (-torch.arange(p, device=DEV, dtype=torch.float32) / max(p, 1))
                                for p in _pairs(c)])
        if c["grad"]:
            s["grad_out"] = normal(c["N"], L, c["M"], c["D"])
    elif c["op"] == "attn":
        N, M, Mk, Lq, Lk, D, Dv = (c[k] for k in ("N", "M", "Mk", "Lq", "Lk", "D", "Dv"))
        s["q"] = normal(N, Lq, M, 2, D, std=1.5)
        s["k"] = normal(N, Lk, Mk, 2, D)
        s["v"] = normal(N, Lk, Mk, Dv)
        s["lam"] = normal(M, std=0.1, mean=0.7)
        s["mask"] = s["lengths"] = None
        if c["grid_w"]:
            at = torch.arange(Lk, device=DEV)
            valid = torch.tensor(_valid(c), device=DEV)
            s["mask"] = (at // c["grid_w"] >= valid[:, :1]) | (at % c["grid_w"] >= valid[:, 1:])
        if c["lengths"]:
            at = torch.randperm(N, generator=g, device=DEV)
            s["lengths"] = torch.tensor(_key_counts(c), device=DEV, dtype=torch.int32)[at].contiguous()
        if c["train"]:
            s["grad_out"] = normal(N, Lq, M, Dv)
    else:
        N, L, C = c["N"], c["L"], c["C"]
        s["x"] = normal(N, L, C, std=2.0, mean=0.1)
        s["y"] = normal(N, L, C, std=1.5, mean=-0.2)
        s["scale"] = normal(C, std=0.1, mean=0.5)
        s["gate"] = normal(N, C, std=0.3, mean=0.8) if c["gate"] else None
        for k in ("post", "pre"):
            s[k + "_weight"] = normal(C, std=0.2, mean=1.0) if c[k] else None
            s[k + "_bias"] = normal(C, std=0.2) if c[k] and c["bias"] else None
        if c["grad"]:
            s["grad_z"] = normal(N, L, C)
            s["grad_h"] = normal(N, L, C) if c["pre"] else None
    return s


# ------------------------------------------------------------- one pass

def run(state):
    s, c = state, state["case"]
    if c["op"] == "rope":
        return _own_rope(s, c) if own else _plain_rope(s, c)
    if c["op"] == "attn":
        return _own_attn(s, c) if own else _plain_attn(s, c)
    return _own_norm(s, c) if own else _plain_norm(s, c)


def _own_rope(s, c):
    import deformable_attention_sampling_b200 as dcnb
    if c["grad"]:
        return dcnb.axial_rope_grad(s["x"], s["pos"], s["freqs"], _pairs(c), s["grad_out"],
                                    interleaved=c["interleaved"])
    return dcnb.axial_rope(s["x"], s["pos"], s["freqs"], _pairs(c), interleaved=c["interleaved"])


def _own_attn(s, c):
    import deformable_attention_sampling_b200 as dcnb
    kw = {"mask": s["mask"], "lengths": s["lengths"], "causal": c["causal"]}
    if not c["train"]:
        return dcnb.diff_attn(s["q"], s["k"], s["v"], s["lam"], **kw)
    out, saved = dcnb.diff_attn(s["q"], s["k"], s["v"], s["lam"], save=True, **kw)
    return (out,) + dcnb.diff_attn_grad(s["q"], s["k"], s["v"], s["lam"], out, saved, s["grad_out"], **kw)


def _own_norm(s, c):
    import deformable_attention_sampling_b200 as dcnb
    kw = {k: s[k] for k in ("scale", "gate", "post_weight", "post_bias", "pre_weight", "pre_bias")}
    kw.update(norm="rms" if c["rms"] else "layer", post=c["post"], pre=c["pre"], eps=1e-6)
    z, h = dcnb.norm_residual(s["x"], s["y"], **kw)
    if not c["grad"]:
        return z, h
    return (z, h) + dcnb.norm_residual_grad(s["y"], z, s["grad_z"], s["grad_h"], **kw)


# ----------------------------------------------------------- the plain forms

def _plain_rope(s, c):
    x, R = s["x"].float(), c["rotated"]
    axis = torch.repeat_interleave(torch.arange(c["axes"], device=DEV), torch.tensor(_pairs(c), device=DEV))
    turn = s["pos"].double()[..., axis] * s["freqs"].double()      # [N, L, R]
    cos, sin = turn.cos().float()[:, :, None], turn.sin().float()[:, :, None]

    def split(t):
        if c["interleaved"]:
            return t[..., 0:2 * R:2], t[..., 1:2 * R:2], t[..., 2 * R:]
        return t[..., :R], t[..., R:2 * R], t[..., 2 * R:]

    def join(a, b, rest):
        both = torch.stack([a, b], dim=-1).flatten(-2) if c["interleaved"] else torch.cat([a, b], dim=-1)
        return torch.cat([both, rest], dim=-1).to(s["x"].dtype)

    a, b, rest = split(x)
    oa, ob = a * cos - b * sin, a * sin + b * cos
    if not c["grad"]:
        return join(oa, ob, rest)
    ga, gb, grest = split(s["grad_out"].float())
    per_pair = (gb * oa - ga * ob).double().sum(dim=2) * s["freqs"].double()
    grad_pos = torch.zeros(s["pos"].shape, device=DEV, dtype=torch.float64).index_add(2, axis, per_pair).float()
    return join(ga * cos + gb * sin, gb * cos - ga * sin, grest), grad_pos


def _hidden(s, c):
    """True where query i may not see key j, broadcast to [N, 1, 1, 1, Lq, Lk]."""
    j = torch.arange(c["Lk"], device=DEV)
    count = s["lengths"].long() if s["lengths"] is not None else torch.full((c["N"],), c["Lk"], device=DEV)
    count = count[:, None, None]
    hide = j >= count
    if c["causal"]:
        hide = hide | (j > torch.arange(c["Lq"], device=DEV)[:, None] + count - c["Lq"])
    if s["mask"] is not None:
        hide = hide | s["mask"][:, None, :]
    return hide[:, None, None, None]


def _plain_attn(s, c):
    N, M, Mk, Lq, Lk, D, Dv = (c[k] for k in ("N", "M", "Mk", "Lq", "Lk", "D", "Dv"))
    G, dt = M // Mk, s["q"].dtype
    q = s["q"].float().view(N, Lq, Mk, G, 2, D).permute(0, 2, 3, 4, 1, 5)      # [N, Mk, G, 2, Lq, D]
    k = s["k"].float().permute(0, 2, 3, 1, 4)[:, :, None]                      # [N, Mk, 1, 2, Lk, D]
    v = s["v"].float().permute(0, 2, 1, 3)[:, :, None]                         # [N, Mk, 1, Lk, Dv]
    lam = s["lam"].float().view(Mk, G, 1, 1)
    scale = D ** -0.5
    hide = _hidden(s, c)
    score = (torch.matmul(q, k.transpose(-1, -2)) * scale).masked_fill(hide, -math.inf)
    top = score.amax(dim=-1, keepdim=True).clamp_min(-1e30)
    p = torch.exp(score - top)
    del score
    p = p / p.sum(dim=-1, keepdim=True).clamp_min(1e-30)                       # [N, Mk, G, 2, Lq, Lk]
    gone = hide.all(dim=-2).view(N, 1, 1, Lk, 1)                               # keys that no query sees
    v = v.masked_fill(gone, 0.0)
    both = p[:, :, :, 0] - lam * p[:, :, :, 1]
    out = torch.matmul(both, v)
    heads = (lambda t: t.permute(0, 3, 1, 2, 4).reshape(N, Lq, M, Dv).to(dt))
    if not c["train"]:
        return heads(out)
    go = s["grad_out"].float().view(N, Lq, Mk, G, Dv).permute(0, 2, 3, 1, 4)
    gv = torch.matmul(both.transpose(-1, -2), go).sum(dim=2)                   # [N, Mk, Lk, Dv]
    del both
    gp = torch.matmul(go, v.transpose(-1, -2))[:, :, :, None]                  # [N, Mk, G, 1, Lq, Lk]
    along = (p * gp).sum(dim=-1, keepdim=True)                                 # [N, Mk, G, 2, Lq, 1]
    sign = torch.stack([torch.ones_like(lam), -lam], dim=2)                    # [Mk, G, 2, 1, 1]
    glam = -along[:, :, :, 1].sum(dim=(0, 3, 4)).view(M)
    gs = p.mul_(gp - along).mul_(sign * scale)
    gq = torch.matmul(gs, k).permute(0, 4, 1, 2, 3, 5).reshape(N, Lq, M, 2, D)
    gk = torch.matmul(gs.transpose(-1, -2), q).sum(dim=2).permute(0, 3, 1, 2, 4)
    return heads(out), gq.to(dt), gk.contiguous().to(dt), gv.permute(0, 2, 1, 3).contiguous().to(dt), glam.to(dt)


def _normed(t, rms, eps=1e-6):
    """The normalised rows and the reciprocal of their spread."""
    if not rms:
        t = t - t.mean(dim=-1, keepdim=True)
    r = torch.rsqrt(t.square().mean(dim=-1, keepdim=True) + eps)
    return t * r, r


def _norm_back(g, n, r, rms):
    """Gradient of a row's values from that of its normalised values `n`."""
    g = g if rms else g - g.mean(dim=-1, keepdim=True)
    return r * (g - n * (g * n).mean(dim=-1, keepdim=True))


def _affine(n, w, b):
    n = n * w.float()
    return n if b is None else n + b.float()


def _plain_norm(s, c):
    dt, rms = s["y"].dtype, c["rms"]
    y = s["y"].float()
    scale = s["scale"].float()
    gate = s["gate"].float()[:, None] if c["gate"] else torch.ones(1, 1, 1, device=DEV)
    n1, r1 = _normed(y, rms) if c["post"] else (y, None)
    u = _affine(n1, s["post_weight"], s["post_bias"]) if c["post"] else y
    z = s["x"].float() + scale * gate * u
    n2, r2 = _normed(z, rms) if c["pre"] else (None, None)
    h = _affine(n2, s["pre_weight"], s["pre_bias"]).to(dt) if c["pre"] else None
    if not c["grad"]:
        return z.to(dt), h
    g, gpw, gpb, gqw, gqb = s["grad_z"].float(), None, None, None, None
    if c["pre"]:
        gh = s["grad_h"].float()
        gqw = (gh * n2).sum(dim=(0, 1)).to(dt)
        gqb = gh.sum(dim=(0, 1)).to(dt) if c["bias"] else None
        g = g + _norm_back(gh * s["pre_weight"].float(), n2, r2, rms)
    gu = g * scale * gate
    gscale = (g * gate * u).sum(dim=(0, 1)).to(dt)
    ggate = (g * scale * u).sum(dim=1).to(dt) if c["gate"] else None
    gy = gu
    if c["post"]:
        gpw = (gu * n1).sum(dim=(0, 1)).to(dt)
        gpb = gu.sum(dim=(0, 1)).to(dt) if c["bias"] else None
        gy = _norm_back(gu * s["post_weight"].float(), n1, r1, rms)
    return z.to(dt), h, g.to(dt), gy.to(dt), gscale, ggate, gpw, gpb, gqw, gqb


# ------------------------------------------------------------------- the work

def _visible(c):
    """(query, key) pairs that a head looks at, over the batch, and the keys that are read."""
    if c["grid_w"]:
        keys = [a * b for a, b in _valid(c)]
        return sum(c["Lq"] * n for n in keys), sum(keys)
    counts = _key_counts(c)
    if not c["causal"]:
        return sum(c["Lq"] * n for n in counts), sum(counts)
    return sum(sum(max(0, min(n, i + 1 + n - c["Lq"])) for i in range(c["Lq"])) for n in counts), sum(counts)


def work(case):
    c = case
    es = DT[c["dtype"]].itemsize
    if c["op"] == "rope":
        tokens = c["N"] * c["T"] * c["H"] * c["W"]
        per = c["M"] * c["D"] * es * (3 if c["grad"] else 2) + c["axes"] * 4 * (2 if c["grad"] else 1)
        return {"bytes": tokens * per, "flops": tokens * c["M"] * c["rotated"] * (16 if c["grad"] else 6)}
    if c["op"] == "attn":
        pairs, keys = _visible(c)
        q, o = c["N"] * c["Lq"] * c["M"] * 2 * c["D"], c["N"] * c["Lq"] * c["M"] * c["Dv"]
        kv = keys * c["Mk"] * (2 * c["D"] + c["Dv"])
        flops = pairs * c["M"] * (4 * c["D"] + 4 * c["Dv"])
        if c["train"]:
            # q, k, v, grad_out in, out and the gradients out; one product each for the
            # scores (2), the maps' gradient, the values, the queries (2) and the keys (2)
            return {"bytes": (2 * q + 2 * kv + 2 * o) * es,
                    "flops": flops + pairs * c["M"] * (12 * c["D"] + 4 * c["Dv"])}
        return {"bytes": (q + kv + o) * es, "flops": flops}
    t = c["N"] * c["L"] * c["C"]
    moved = t * (3 + c["pre"]) + (t * (3 + c["pre"]) if c["grad"] else 0)
    return {"bytes": moved * es, "flops": t * (14 if not c["grad"] else 44)}


# --------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    """Outputs from the definitions in float64; gradients by differentiating those."""
    c, s = case, prepare(case, seed)
    up = {k: t.double() for k, t in s.items() if torch.is_tensor(t) and t.is_floating_point()}
    if c["op"] == "rope":
        pos = up["pos"].requires_grad_(c["grad"])
        x = up["x"].requires_grad_(c["grad"])
        turns, at = [], 0
        for a, p in enumerate(_pairs(c)):
            turns.append(pos[:, :, a:a + 1] * up["freqs"][at:at + p])
            at += p
        spin = torch.polar(torch.ones((), device=DEV, dtype=torch.float64), torch.cat(turns, -1))[:, :, None]
        R = c["rotated"]
        if c["interleaved"]:
            z = torch.view_as_complex(x[..., :2 * R].unflatten(-1, (R, 2)).contiguous()) * spin
            turned = torch.view_as_real(z).flatten(-2)
        else:
            z = torch.complex(x[..., :R].contiguous(), x[..., R:2 * R].contiguous()) * spin
            turned = torch.cat([z.real, z.imag], -1)
        out = torch.cat([turned, x[..., 2 * R:]], -1)
        return torch.autograd.grad(out, (x, pos), up["grad_out"]) if c["grad"] else out
    if c["op"] == "attn":
        N, M, Mk, Lq, Lk = (c[k] for k in ("N", "M", "Mk", "Lq", "Lk"))
        counts = [Lk] * N if s["lengths"] is None else s["lengths"].tolist()
        outs, grads = [], {"q": [], "k": [], "v": [], "lam": torch.zeros(M, device=DEV, dtype=torch.float64)}
        for n in range(N):          # image by image and head by head: the maps are large
            seen = torch.zeros(Lq, Lk, dtype=torch.bool, device=DEV)
            seen[:, :counts[n]] = True
            if c["causal"]:
                seen = seen.tril(counts[n] - Lq)
            if s["mask"] is not None:
                seen &= ~s["mask"][n]
            heads, gq = [], []
            gk, gv = torch.zeros_like(up["k"][n]), torch.zeros_like(up["v"][n])
            for m in range(M):
                a = m // (M // Mk)
                ins = [up["q"][n, :, m], up["k"][n, :, a], up["v"][n, :, a], up["lam"][m]]
                ins = [t.clone().requires_grad_(c["train"]) for t in ins]
                qm, km, vm, lm = ins
                maps = []
                for i in (0, 1):
                    sc = (qm[:, i] @ km[:, i].T / math.sqrt(c["D"])).where(seen, -math.inf)
                    maps.append(torch.softmax(sc, -1).where(seen.any(-1, keepdim=True), 0.0))
                o = (maps[0] - lm * maps[1]) @ vm
                heads.append(o.detach())
                if c["train"]:
                    r = torch.autograd.grad(o, ins, up["grad_out"][n, :, m])
                    gq.append(r[0])
                    gk[:, a] += r[1]
                    gv[:, a] += r[2]
                    grads["lam"][m] += r[3]
                del maps, o
            outs.append(torch.stack(heads, 1))
            if c["train"]:
                grads["q"].append(torch.stack(gq, 1))
                grads["k"].append(gk)
                grads["v"].append(gv)
        out = torch.stack(outs)
        if not c["train"]:
            return out
        return (out,) + tuple(torch.stack(grads[k]) for k in ("q", "k", "v")) + (grads["lam"],)
    names = [k for k in ("x", "y", "scale", "gate", "post_weight", "post_bias", "pre_weight", "pre_bias") if k in up]
    for k in names:
        up[k].requires_grad_(c["grad"])

    def norm(t, w, b):
        if c["rms"]:
            r = t / (t.pow(2).mean(-1, keepdim=True) + 1e-6).sqrt() * w
            return r if b is None else r + b
        return torch.nn.functional.layer_norm(t, t.shape[-1:], w, b, 1e-6)

    u = norm(up["y"], up["post_weight"], up.get("post_bias")) if c["post"] else up["y"]
    z = up["x"] + up["scale"] * u * (up["gate"].unsqueeze(1) if c["gate"] else 1.0)
    h = norm(z, up["pre_weight"], up.get("pre_bias")) if c["pre"] else None
    if not c["grad"]:
        return z, h
    aim = (z * up["grad_z"]).sum() + ((h * up["grad_h"]).sum() if c["pre"] else 0.0)
    got = dict(zip(names, torch.autograd.grad(aim, [up[k] for k in names])))
    order = ("x", "y", "scale", "gate", "post_weight", "post_bias", "pre_weight", "pre_bias")
    return (z, h) + tuple(got.get(k) for k in order)
