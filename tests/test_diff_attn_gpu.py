"""diff_attn and diff_attn_grad against the float64 definition, with bounds that
count roundings (tests/block_ref.py)."""
import math

import pytest
import torch

import deformable_attention_sampling_b200 as dcnb
from tests import block_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(autouse=True)
def no_wait_ran_out():
    yield
    torch.cuda.synchronize()
    assert dcnb.dcn_device_flags(reset=True) == 0


def inputs(N, Lq, Lk, M, Mk, D, Dv, dtype, seed=0):
    g = torch.Generator().manual_seed(seed)
    n = (lambda *s, std=1.0, mean=0.0: (torch.randn(s, generator=g) * std + mean).to(dtype).to(DEV))
    return (n(N, Lq, M, 2, D, std=1.5), n(N, Lk, Mk, 2, D), n(N, Lk, Mk, Dv),
            n(M, std=0.1, mean=0.7), n(N, Lq, M, Dv))


def run_and_check(q, k, v, lam, go, grad=True, **kw):
    out, saved = dcnb.diff_attn(q, k, v, lam, save=True, **kw)
    r = ref.attn(q, k, v, lam, grad_out=go if grad else None, **kw)
    ref.check(out, *r["out"], "out")
    ref.check(saved[0], *r["maps"], "maps")
    want, bound = r["lse"]
    got = saved[1].double().cpu()
    empty = torch.isinf(want)
    assert torch.equal(torch.isinf(got), empty)
    assert ((got - want).abs()[~empty] <= bound[~empty]).all(), "lse"
    assert torch.equal(out, dcnb.diff_attn(q, k, v, lam, **kw))
    if not grad:
        return out, saved, r
    grads = dcnb.diff_attn_grad(q, k, v, lam, out, saved, go, **kw)
    again = dcnb.diff_attn_grad(q, k, v, lam, out, saved, go, **kw)
    for name, got, twice in zip(("q", "k", "v", "lam"), grads, again):
        ref.check(got, *r[name], "grad_" + name)
        assert torch.equal(got, twice), f"grad_{name} differs between equal calls"
    return out, saved, r


SHAPES = [  # N, Lq, Lk, M, Mk, D, Dv
    (1, 1, 1, 1, 1, 1, 1),
    (2, 3, 5, 2, 1, 8, 8),
    (1, 17, 33, 6, 2, 20, 12),
    (2, 64, 64, 4, 4, 32, 64),
    (1, 130, 200, 4, 2, 64, 128),
    (1, 129, 257, 3, 3, 64, 64),
    (2, 100, 100, 6, 2, 32, 32),
    (1, 65, 190, 2, 1, 128, 128),
    (1, 40, 300, 2, 2, 96, 80),
    (1, 33, 70, 2, 1, 128, 256),
    (1, 40, 65, 2, 1, 16, 200),
    (1, 257, 513, 2, 1, 48, 48),
]


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("causal", [False, True])
def test_shapes(shape, dt, causal):
    run_and_check(*inputs(*shape, DT[dt]), causal=causal)


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("Lq,Lk,M,Mk,D,Dv", [
    (1, 1, 4, 1, 64, 128), (1, 700, 16, 4, 64, 128), (1, 1025, 8, 8, 32, 32),
    (4, 1500, 4, 1, 64, 64), (2, 333, 3, 1, 128, 128), (3, 900, 32, 2, 64, 64),
    (1, 640, 5, 1, 40, 24), (1, 2000, 2, 2, 128, 256)])
def test_steps_with_lengths(Lq, Lk, M, Mk, D, Dv, dt):
    """New tokens over caches of uneven fill, empty and shorter than the tokens among them."""
    N = 5
    q, k, v, lam, go = inputs(N, Lq, Lk, M, Mk, D, Dv, DT[dt], 1)
    lengths = torch.tensor([Lk, 0, 1, max(1, Lk // 2), Lk + 9], dtype=torch.int32, device=DEV)
    n = lengths.clamp(max=Lk).tolist()
    for i in range(N):                     # what lies behind a sequence is not read
        k[i, n[i]:] = math.nan
        v[i, n[i]:] = math.inf
    out, _, r = run_and_check(q, k, v, lam, go, causal=True, lengths=lengths)
    assert not out[1].any()
    run_and_check(q, k, v, lam, go, causal=False, lengths=lengths)


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("N,Lq,Lk,M,Mk,D,Dv", [(1, 40, 700, 2, 1, 64, 256), (1, 20, 1500, 1, 1, 128, 128),
                                               (2, 17, 900, 2, 2, 32, 64), (1, 130, 3000, 1, 1, 64, 64)])
def test_few_tiles_over_many_keys(N, Lq, Lk, M, Mk, D, Dv, dt):
    """Few query tiles: the keys are split, and some splits of a short image are empty."""
    q, k, v, lam, go = inputs(N, Lq, Lk, M, Mk, D, Dv, DT[dt], 11)
    run_and_check(q, k, v, lam, go)
    lengths = torch.tensor([Lk // 3, 60][:N], dtype=torch.int32, device=DEV)
    run_and_check(q, k, v, lam, go, lengths=lengths, causal=True)


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("Lq,Lk,M,Mk,D,Dv", [(70, 150, 4, 2, 32, 64), (200, 300, 2, 1, 64, 128),
                                             (1, 260, 4, 4, 64, 64), (20, 40, 2, 2, 12, 20)])
def test_masks(Lq, Lk, M, Mk, D, Dv, dt):
    """Scattered masks, a masked image, masked tiles; masked keys hold NaN and infinities."""
    N = 4
    q, k, v, lam, go = inputs(N, Lq, Lk, M, Mk, D, Dv, DT[dt], 2)
    g = torch.Generator().manual_seed(7)
    mask = torch.rand(N, Lk, generator=g) < 0.3
    mask[1] = True                          # nothing visible
    mask[2] = True
    mask[2, Lk - 1] = False                 # one key
    mask[3, :Lk // 2] = True                # whole tiles
    mask = mask.to(DEV)
    k.masked_fill_(mask[:, :, None, None, None], math.nan)
    v.masked_fill_(mask[:, :, None, None], -math.inf)
    out, _, _ = run_and_check(q, k, v, lam, go, mask=mask)
    assert not out[1].any()
    run_and_check(q, k, v, lam, go, mask=mask.to(torch.uint8) * 4, causal=True,
                  lengths=torch.tensor([Lk, Lk, Lk, Lk - 3], dtype=torch.int32, device=DEV))


@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
def test_strided_inputs(dt):
    """q, k, v as slices of one projection; images and tokens apart."""
    N, L, M, D, Dv = 2, 140, 2, 64, 64
    g = torch.Generator().manual_seed(3)
    wide = torch.randn(N, L + 5, M * (4 * D + Dv) + 8, generator=g).to(DT[dt]).to(DEV)
    flat = wide[:, 2:2 + L]
    q = flat[:, :, :2 * M * D].unflatten(2, (M, 2, D))
    k = flat[:, :, 2 * M * D:4 * M * D].unflatten(2, (M, 2, D))
    v = flat[:, :, 4 * M * D:4 * M * D + M * Dv].unflatten(2, (M, Dv))
    assert not q.is_contiguous()
    lam = torch.tensor([0.4, -0.9], device=DEV).to(DT[dt])
    go = torch.randn(N, L, M, Dv, generator=g).to(DT[dt]).to(DEV)
    run_and_check(q, k, v, lam, go, causal=True)
    # a storage that starts 2 bytes off the 16-byte grid
    off = torch.empty(k.numel() + 1, dtype=k.dtype, device=DEV)[1:].view(k.shape)
    off.copy_(k)
    run_and_check(q, off, v, lam, go, causal=True)


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("Lq", [1, 150])
def test_offsets_past_32_bits(dt, Lq):
    """A cache whose tokens lie 2^27 elements apart: 24 of them pass 2^31 elements."""
    N, Lk, M, D, Dv = 1, 24, 2, 64, 64
    q, k, v, lam, go = inputs(N, Lq, Lk, M, M, D, Dv, DT[dt], 4)
    far = torch.empty(Lk << 27, dtype=DT[dt], device=DEV)
    kf = far.as_strided(k.shape, (0, 1 << 27, 2 * D, D, 1))
    kf.copy_(k)
    vf = far[4096:].as_strided(v.shape, (0, 1 << 27, Dv, 1))
    vf.copy_(v)
    out, saved = dcnb.diff_attn(q, kf, vf, lam, save=True)
    want, wsaved = dcnb.diff_attn(q, k, v, lam, save=True)
    assert torch.equal(out, want) and torch.equal(saved[1], wsaved[1])
    for a, b in zip(dcnb.diff_attn_grad(q, kf, vf, lam, out, saved, go),
                    dcnb.diff_attn_grad(q, k, v, lam, out, saved, go)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("D,Dv", [(64, 64), (32, 128)])
def test_large_and_uneven_scores(dt, D, Dv):
    """Rows whose maximum keeps growing along the keys, and scores of a few hundred."""
    N, L, M = 1, 400, 2
    q, k, v, lam, go = inputs(N, L, L, M, M, D, Dv, DT[dt], 5)
    grow = torch.linspace(0.02, 6.0, L, device=DEV).to(DT[dt])
    run_and_check(q, k * grow[None, :, None, None, None], v, lam, go)
    run_and_check(q * 8, k * grow.flip(0)[None, :, None, None, None], v, lam, go, causal=True)


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("size", [1e-4, 30.0])
def test_small_and_large_gradients(dt, size):
    """Incoming gradients far from 1 (a loss's mean, or its scale in 16-bit training)."""
    q, k, v, lam, go = inputs(2, 150, 170, 2, 1, 64, 64, DT[dt], 6)
    run_and_check(q, k, v * 4, lam, (go.float() * size).to(DT[dt]))


@pytest.mark.parametrize("dt", list(DT))
def test_scale_and_repeated_use(dt):
    q, k, v, lam, go = inputs(2, 33, 40, 4, 2, 64, 64, DT[dt], 8)
    run_and_check(q, k, v, lam, go, scale=0.3)
    run_and_check(q, k, v, lam * 0, go, scale=-0.05)
    run_and_check(q, k, v, lam, go, scale=0.0)


def test_empty_calls():
    for N, Lq, Lk in ((0, 3, 4), (2, 0, 4), (2, 3, 0), (0, 0, 0)):
        q, k, v, lam, go = inputs(N, Lq, Lk, 4, 2, 64, 64, torch.float16)
        out, saved = dcnb.diff_attn(q, k, v, lam, save=True)
        assert not out.any()
        for g, t in zip(dcnb.diff_attn_grad(q, k, v, lam, out, saved, go), (q, k, v, lam)):
            assert g.shape == t.shape and not g.any()


def test_other_streams_and_graphs():
    """Calls on a side stream and captured into two graphs that run side by side."""
    shape = (2, 150, 700, 4, 2, 64, 128)
    q, k, v, lam, go = inputs(*shape, torch.bfloat16, 9)
    q1 = q[:, :1].contiguous()

    def step():
        out, saved = dcnb.diff_attn(q, k, v, lam, causal=True, save=True)
        one = dcnb.diff_attn(q1, k, v, lam, causal=True)
        return (out, one) + dcnb.diff_attn_grad(q, k, v, lam, out, saved, go, causal=True)

    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    # the stream as an argument, an object or a handle: launch and scratch go there
    for stream in (side, side.cuda_stream):
        side.wait_stream(torch.cuda.current_stream())
        out, saved = dcnb.diff_attn(q, k, v, lam, causal=True, save=True, stream=stream)
        got = (out, dcnb.diff_attn(q1, k, v, lam, causal=True, stream=stream)) + dcnb.diff_attn_grad(
            q, k, v, lam, out, saved, go, causal=True, stream=stream)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step())
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(3):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for o in outs:
        assert all(torch.equal(a, b) for a, b in zip(o, want))


def test_gradient_against_differences():
    """float32, central differences of the float64 definition in random directions."""
    q, k, v, lam, go = inputs(1, 9, 11, 4, 2, 8, 12, torch.float32, 10)
    mask = (torch.arange(11, device=DEV) % 4 == 3)[None]
    kw = dict(causal=True, mask=mask)
    out, saved = dcnb.diff_attn(q, k, v, lam, save=True, **kw)
    grads = dcnb.diff_attn_grad(q, k, v, lam, out, saved, go, **kw)
    at = [t.double().cpu() for t in (q, k, v, lam)]
    g = torch.Generator().manual_seed(3)
    h = 1e-4
    for i, got in enumerate(grads):
        d = torch.randn(at[i].shape, generator=g).double()

        def value(step):
            m = list(at)
            m[i] = m[i] + step * d
            return float((ref.attn(*m, **kw)["out"][0] * go.double().cpu()).sum())

        slope = (value(h) - value(-h)) / (2 * h)
        mag = float((got.double().cpu() * d).abs().sum())
        assert abs(float((got.double().cpu() * d).sum()) - slope) <= 1e-5 * mag + 1e-5


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_a_block_of_the_operators(dt):
    """Rotary positions, differential attention and the normed join, as one
    block uses them, forward and backward, against the float64 chain."""
    N, H, W, M, D = 2, 6, 9, 4, 16
    L, C, Dv, pairs = H * W, 4 * 2 * 16, 32, (4, 4)
    g = torch.Generator().manual_seed(12)
    n = (lambda *s, std=1.0, mean=0.0: (torch.randn(s, generator=g) * std + mean).to(DT[dt]).to(DEV))
    x, q, k, v = n(N, L, C), n(N, L, M, 2, D), n(N, L, M, 2, D), n(N, L, M, Dv)
    lam, scale = n(M, std=0.1, mean=0.6), n(C, std=0.1, mean=0.5)
    w1, w2 = n(C, std=0.2, mean=1.0), n(C, std=0.2, mean=1.0)
    gz, gh = n(N, L, C), n(N, L, C)
    cell = torch.arange(L, device=DEV)
    pos = torch.stack([cell // W + 0.5, cell % W + 0.5], -1).float()[None]
    freqs = (100.0 ** (-torch.arange(4, device=DEV) / 4.0)).repeat(2).float()
    mask = (cell % W >= W - 2)[None].repeat(N, 1)
    mask[0] = False

    qr = dcnb.axial_rope(q.view(N, L, 2 * M, D), pos, freqs, pairs).view(q.shape)
    kr = dcnb.axial_rope(k.view(N, L, 2 * M, D), pos, freqs, pairs).view(k.shape)
    y, saved = dcnb.diff_attn(qr, kr, v, lam, mask=mask, save=True)
    kw = dict(scale=scale, post_weight=w1, pre_weight=w2, norm="rms")
    z, h = dcnb.norm_residual(x, y.view(N, L, C), **kw)
    back = dcnb.norm_residual_grad(y.view(N, L, C), z, gz, gh, **kw)
    gy = back[1].view(y.shape)
    gq, gk, gv, glam = dcnb.diff_attn_grad(qr, kr, v, lam, y, saved, gy, mask=mask)
    gq, gpq = dcnb.axial_rope_grad(q.view(N, L, 2 * M, D), pos, freqs, pairs, gq.view(N, L, 2 * M, D))
    gk, gpk = dcnb.axial_rope_grad(k.view(N, L, 2 * M, D), pos, freqs, pairs, gk.view(N, L, 2 * M, D))

    # the same chain, each link from the framework's previous output
    ref.check(qr.view(N, L, 2 * M, D), *ref.rope(q.view(N, L, 2 * M, D), pos, freqs, pairs, False), "q")
    r = ref.attn(qr, kr, v, lam, mask=mask, grad_out=gy)
    ref.check(y, *r["out"], "attention")
    f = {"scale": scale, "post_weight": w1, "pre_weight": w2}
    j = ref.join(x, y.view(N, L, C), f, norm="rms")
    ref.check(z, *j["z"], "z")
    ref.check(h, *j["h"], "h")
    ref.check(gv, *r["v"], "grad_v")
    ref.check(glam, *r["lam"], "grad_lam")
    b = ref.join_grad(y.view(N, L, C), z, gz, gh, f, norm="rms")
    ref.check(back[0], *b["x"], "grad_x")
    ref.check(gy.view(N, L, C), *b["y"], "grad_y")
    # gradient of the positions through both rotations: one shared row of positions
    assert gpq.shape == pos.shape and gpk.shape == pos.shape
    if dt == "f32":
        X = [t.double().cpu().requires_grad_() for t in (q, k, pos)]

        def turn(t):
            th = (X[2][..., [0] * 4 + [1] * 4] * freqs.double().cpu())[:, :, None, None]
            a, b = t[..., :8], t[..., 8:]
            return torch.cat([a * th.cos() - b * th.sin(), a * th.sin() + b * th.cos()], -1)

        s = torch.einsum("nimsd,njmsd->nmsij", turn(X[0]), turn(X[1])) * D ** -0.5
        p = s.masked_fill(mask.cpu()[:, None, None, None], -math.inf).softmax(-1)
        o = torch.einsum("nmij,njmv->nimv", p[:, :, 0] - lam.double().cpu()[:, None, None] * p[:, :, 1],
                         v.double().cpu()).reshape(N, L, C)
        rms = (lambda t: t * (t.square().mean(-1, keepdim=True) + 1e-6).rsqrt())
        zz = x.double().cpu() + scale.double().cpu() * rms(o) * w1.double().cpu()
        ((zz * gz.double().cpu()).sum() + (rms(zz) * w2.double().cpu() * gh.double().cpu()).sum()).backward()
        # float32 links: each gradient carries the roundings of some hundreds of terms
        for got, want in ((gq.view(q.shape), X[0].grad), (gk.view(k.shape), X[1].grad),
                          (gpq + gpk, X[2].grad)):
            assert (got.double().cpu() - want).abs().max() <= 2e-5 * want.abs().max()
