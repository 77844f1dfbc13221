"""axial_rope and norm_residual, forward and gradient, against their float64
definitions with rounding-count bounds (tests/block_ref.py)."""
import pytest
import torch

import deformable_attention_sampling_b200 as dcnb
from tests import block_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def normal(g, *shape, dtype=torch.float32, std=1.0, mean=0.0):
    return (torch.randn(shape, generator=g) * std + mean).to(dtype).to(DEV)


def rope_inputs(N, L, M, D, pairs, dtype, seed, shared=False, far=False):
    g = torch.Generator().manual_seed(seed)
    A, R = len(pairs), sum(pairs)
    pos = torch.rand((1 if shared else N, L, A), generator=g) * (1e5 if far else 200.0) - 20.0
    freqs = torch.rand(R, generator=g) * 1.2 + 1e-4
    return (normal(g, N, L, M, D, dtype=dtype), pos.to(DEV), freqs.to(DEV),
            normal(g, N, L, M, D, dtype=dtype))


ROPE = [  # N, L, M, D, pairs, interleaved, shared pos
    (1, 1, 1, 2, (1,), True, False),
    (2, 3, 5, 6, (1, 2), False, False),
    (1, 7, 3, 64, (10, 11, 11), False, False),
    (3, 37, 8, 32, (8, 8), True, True),
    (2, 50, 16, 80, (20, 16), True, False),
    (2, 9, 1, 128, (31, 0, 33), False, True),
    (1, 5, 2, 33, (3, 4, 5, 2), True, False),
    (1, 4, 3, 40, (0,), False, False),          # nothing turns: channels pass
    (1, 300, 4, 512, (256,), False, False),
    (2, 11, 7, 20, (5, 5), False, True),
]


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("case", ROPE)
def test_axial_rope(case, dt):
    N, L, M, D, pairs, inter, shared = case
    x, pos, freqs, go = rope_inputs(N, L, M, D, pairs, DT[dt], 3, shared, far=D == 64)
    for inverse in (False, True):
        out = dcnb.axial_rope(x, pos, freqs, pairs, interleaved=inter, inverse=inverse)
        ref.check(out, *ref.rope(x, pos, freqs, pairs, inter, inverse), "out")
        gx, gp = dcnb.axial_rope_grad(x, pos, freqs, pairs, go, interleaved=inter, inverse=inverse)
        rx, rp = ref.rope(x, pos, freqs, pairs, inter, inverse, go)
        ref.check(gx, *rx, "grad_x")
        ref.check(gp, *rp, "grad_pos")
        only, none = dcnb.axial_rope_grad(x, pos, freqs, pairs, go, interleaved=inter,
                                          inverse=inverse, need_pos=False)
        assert none is None and torch.equal(only, gx)
    assert torch.equal(out, dcnb.axial_rope(x, pos, freqs, pairs, interleaved=inter, inverse=True))


def test_axial_rope_strides_in_place_and_ends():
    """A slice of a projection's output (strided tokens), in place, and memory
    behind the last token left as it was."""
    N, L, M, D, pairs = 2, 13, 4, 48, (12, 12)
    x, pos, freqs, _ = rope_inputs(N, L, M, D, pairs, torch.bfloat16, 5)
    wide = torch.randn(N, L, 3, M, D, device=DEV).bfloat16()
    for i in range(3):
        view = wide[:, :, i]
        got = dcnb.axial_rope(view, pos, freqs, pairs)
        assert torch.equal(got, dcnb.axial_rope(view.contiguous(), pos, freqs, pairs))
    buf = torch.full((N * L * M * D + 64,), 7.0, device=DEV, dtype=torch.bfloat16)
    y = buf[:N * L * M * D].view(N, L, M, D)
    y.copy_(x)
    want = dcnb.axial_rope(x, pos, freqs, pairs)
    assert dcnb.axial_rope(y, pos, freqs, pairs, out=y) is y
    assert torch.equal(y, want) and bool((buf[-64:] == 7.0).all())
    # odd start of the storage: element-wise accesses
    odd = torch.randn(N * L * M * D + 1, device=DEV).bfloat16()[1:].view(N, L, M, D)
    assert torch.equal(dcnb.axial_rope(odd, pos, freqs, pairs),
                       dcnb.axial_rope(odd.clone(), pos, freqs, pairs))


def test_axial_rope_turn_and_back_and_empty():
    N, L, M, D, pairs = 1, 20, 2, 32, (16,)
    x, pos, freqs, _ = rope_inputs(N, L, M, D, pairs, torch.float32, 9, far=True)
    there = dcnb.axial_rope(x, pos, freqs, pairs)
    back = dcnb.axial_rope(there, pos, freqs, pairs, inverse=True)
    assert (back - x).abs().max() <= 48 * ref.U * x.abs().max()
    e = torch.empty(0, L, M, D, device=DEV)
    assert dcnb.axial_rope(e, pos, freqs, pairs).shape == (0, L, M, D)
    gx, gp = dcnb.axial_rope_grad(e, pos, freqs, pairs, e)
    assert gx.numel() == 0 and gp.shape == pos.shape and not gp.any()
    z = torch.empty(2, 0, M, D, device=DEV)
    assert dcnb.axial_rope(z, pos[:, :0], freqs, pairs).numel() == 0


JOIN = [  # N, L, C
    (1, 1, 1), (2, 3, 7), (3, 5, 8), (2, 33, 64), (1, 100, 100), (4, 7, 257), (2, 65, 1024),
    (16, 1, 1024), (1, 3, 4096), (2, 2, 8192), (1, 5, 2049), (40, 3, 96), (1, 700, 72),
]


def join_inputs(N, L, C, dtype, seed, gate, bias, post, pre, offset=0.0):
    g = torch.Generator().manual_seed(seed)
    f = {"scale": normal(g, C, dtype=dtype, std=0.3, mean=0.5),
         "gate": normal(g, N, C, dtype=dtype, std=0.3, mean=0.8) if gate else None}
    for k, on in (("post", post), ("pre", pre)):
        f[k + "_weight"] = normal(g, C, dtype=dtype, std=0.2, mean=1.0) if on else None
        f[k + "_bias"] = normal(g, C, dtype=dtype, std=0.2) if on and bias else None
    rows = [normal(g, N, L, C, dtype=dtype, std=s, mean=m)
            for s, m in ((2.0, 0.1), (1.5, -0.2 + offset), (1.0, 0.0), (1.0, 0.0))]
    return rows, f


NAMES = ("x", "y", "scale", "gate", "post_weight", "post_bias", "pre_weight", "pre_bias")


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("shape", JOIN)
@pytest.mark.parametrize("norm,gate,bias,post,pre", [
    ("layer", False, True, True, True), ("rms", True, False, True, True),
    ("layer", True, True, False, True), ("rms", False, False, True, False),
    ("rms", True, False, False, False)])
def test_norm_residual(shape, dt, norm, gate, bias, post, pre):
    (x, y, gz, gh), f = join_inputs(*shape, DT[dt], 11, gate, bias, post, pre)
    kw = dict(norm=norm, post=post, pre=pre, eps=1e-5)
    z, h = dcnb.norm_residual(x, y, **f, **kw)
    r = ref.join(x, y, f, **kw)
    ref.check(z, *r["z"], "z")
    assert (h is None) == (not pre)
    if pre:
        ref.check(h, *r["h"], "h")
    grads = dcnb.norm_residual_grad(y, z, gz, gh if pre else None, **f, **kw)
    again = dcnb.norm_residual_grad(y, z, gz, gh if pre else None, **f, **kw)
    r = ref.join_grad(y, z, gz, gh, f, **kw)
    for name, got, twice in zip(NAMES, grads, again):
        if name not in ("x", "y") and f[name] is None:
            assert got is None
            continue
        ref.check(got, *r[name], "grad_" + name)
        assert torch.equal(got, twice), f"grad_{name} differs between equal calls"


def test_norm_residual_without_factors_and_with_a_large_mean():
    (x, y, gz, gh), _ = join_inputs(2, 9, 72, torch.float32, 13, False, False, True, True,
                                    offset=300.0)
    none = {k: None for k in NAMES[2:]}
    z, h = dcnb.norm_residual(x, y)
    r = ref.join(x, y, none)
    ref.check(z, *r["z"], "z")
    ref.check(h, *r["h"], "h")
    grads = dcnb.norm_residual_grad(y, z, gz, gh)
    r = ref.join_grad(y, z, gz, gh, none)
    ref.check(grads[0], *r["x"], "grad_x")
    ref.check(grads[1], *r["y"], "grad_y")
    assert grads[2:] == (None,) * 6


def test_norm_residual_in_place_misaligned_and_empty():
    (x, y, gz, gh), f = join_inputs(3, 5, 40, torch.float16, 17, True, True, True, True)
    z, h = dcnb.norm_residual(x, y, **f)
    mine = x.clone()
    z2, h2 = dcnb.norm_residual(mine, y, **f, out=mine)
    assert z2 is mine and torch.equal(z2, z) and torch.equal(h2, h)
    odd = torch.empty(y.numel() + 1, device=DEV, dtype=y.dtype)[1:].view(y.shape)
    odd.copy_(y)
    z3, h3 = dcnb.norm_residual(x, odd, **f)
    r = ref.join(x, y, f)
    ref.check(z3, *r["z"], "z")
    ref.check(h3, *r["h"], "h")
    a = dcnb.norm_residual_grad(odd, z, gz, gh, **f)
    rg = ref.join_grad(y, z, gz, gh, f)
    for name, got in zip(NAMES, a):
        ref.check(got, *rg[name], "grad_" + name)
    e = torch.empty(3, 0, 40, device=DEV, dtype=torch.float16)
    z, h = dcnb.norm_residual(e, e, **f)
    assert z.numel() == 0 and h.numel() == 0
    for got in dcnb.norm_residual_grad(e, e, e, e, **f)[2:]:
        assert not got.any()


def test_norm_residual_gradient_against_differences():
    """float32, central differences of the float64 definition in random directions."""
    (x, y, gz, gh), f = join_inputs(2, 3, 24, torch.float32, 19, True, True, True, True)
    z, _ = dcnb.norm_residual(x, y, **f)
    grads = dict(zip(NAMES, dcnb.norm_residual_grad(y, z, gz, gh, **f)))
    at = {"x": x, "y": y, **f}
    g = torch.Generator().manual_seed(1)

    def value(name, step):
        m = {k: t.double().cpu() for k, t in at.items()}
        m[name] = m[name] + step
        r = ref.join(m["x"], m["y"], {k: m[k] for k in f})
        return float((r["z"][0] * gz.double().cpu()).sum() + (r["h"][0] * gh.double().cpu()).sum())

    for name, t in at.items():
        d = torch.randn(t.shape, generator=g).double()
        h = 1e-4
        slope = (value(name, h * d) - value(name, -h * d)) / (2 * h)
        # float32 gradients summed over at most 144 terms; the difference itself is good to h^2
        mag = float((grads[name].double().cpu() * d).abs().sum())
        assert abs(float((grads[name].double().cpu() * d).sum()) - slope) <= 1e-5 * mag + 1e-4, name


def test_axial_rope_gradient_of_positions_against_differences():
    x, pos, freqs, go = rope_inputs(2, 6, 3, 24, (5, 7), torch.float32, 23)
    _, gp = dcnb.axial_rope_grad(x, pos, freqs, (5, 7), go)
    d = torch.randn(pos.shape, generator=torch.Generator().manual_seed(2)).double()
    h = 1e-5

    def value(s):
        out, _ = ref.rope(x, pos.double().cpu() + s * d, freqs, (5, 7), False)
        return float((out * go.double().cpu()).sum())

    slope = (value(h) - value(-h)) / (2 * h)
    mag = float((gp.double().cpu() * d).abs().sum())
    assert abs(float((gp.double().cpu() * d).sum()) - slope) <= 1e-5 * mag + 1e-5


def test_a_stream_as_an_argument():
    x, pos, freqs, go = rope_inputs(2, 6, 3, 24, (5, 7), torch.bfloat16, 29)
    (a, b, gz, gh), f = join_inputs(2, 7, 48, torch.bfloat16, 31, True, True, True, True)

    def step(**kw):
        z, h = dcnb.norm_residual(a, b, **f, **kw)
        return ((dcnb.axial_rope(x, pos, freqs, (5, 7), **kw), z, h) +
                dcnb.axial_rope_grad(x, pos, freqs, (5, 7), go, **kw) +
                dcnb.norm_residual_grad(b, z, gz, gh, **f, **kw))

    want = step()
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        side.wait_stream(torch.cuda.current_stream())
        got = step(stream=stream)
        torch.cuda.synchronize()
        assert all(torch.equal(g, w) for g, w in zip(got, want))


def test_more_axes_than_tasks():
    """One pair a token and four axes: the position gradients need as many lanes."""
    x, pos, freqs, go = rope_inputs(3, 5, 1, 2, (0, 1, 0, 0), torch.float32, 33)
    gx, gp = dcnb.axial_rope_grad(x, pos, freqs, (0, 1, 0, 0), go)
    rx, rp = ref.rope(x, pos, freqs, (0, 1, 0, 0), False, False, go)
    ref.check(gx, *rx, "grad_x")
    ref.check(gp, *rp, "grad_pos")
