"""diff_attn calls that share a batch between very different images, heads or
tokens, and layouts other than [image][token]; against the float64 definition."""
import pytest
import torch

import deformable_attention_sampling_b200 as dcnb
from tests import block_ref as ref
from tests.test_diff_attn_gpu import DT, inputs, no_wait_ran_out, run_and_check  # noqa: F401

pytestmark = pytest.mark.gpu


def grads_of(q, k, v, lam, go, **kw):
    out, saved = dcnb.diff_attn(q, k, v, lam, save=True, **kw)
    return dcnb.diff_attn_grad(q, k, v, lam, out, saved, go, **kw)


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("causal", [False, True])
def test_small_gradients_beside_large_ones_of_other_images_and_heads(dt, causal):
    """Image 0 has large incoming gradients and small values, image 1 the reverse, and
    so have the key / value heads of image 2: no image and no group of heads may lose
    digits to another's magnitude.  Each is held to the bound of its own inputs."""
    N, L, M, Mk, D, Dv = 3, 150, 4, 2, 64, 64
    q, k, v, lam, go = inputs(N, L, L, M, Mk, D, Dv, DT[dt], 21)
    big, small = 4000.0, 1.0 / 1024
    go[0], v[0] = go[0] * big, v[0] * small
    go[1], v[1] = go[1] * small, v[1] * big
    go[2, :, :2], v[2, :, 0] = go[2, :, :2] * big, v[2, :, 0] * small
    go[2, :, 2:], v[2, :, 1] = go[2, :, 2:] * small, v[2, :, 1] * big
    gq, gk, gv, _ = grads_of(q, k, v, lam, go, causal=causal)
    for n in range(N):
        for a in range(Mk):
            h, one = slice(2 * a, 2 * a + 2), slice(n, n + 1)
            r = ref.attn(q[one, :, h], k[one, :, a:a + 1], v[one, :, a:a + 1], lam[h],
                         causal=causal, grad_out=go[one, :, h])
            where = f" of image {n}, head {a}"
            ref.check(gq[one, :, h], *r["q"], "grad_q" + where)
            ref.check(gk[one, :, a:a + 1], *r["k"], "grad_k" + where)
            ref.check(gv[one, :, a:a + 1], *r["v"], "grad_v" + where)


@pytest.mark.parametrize("dt", list(DT))
def test_small_gradients_beside_large_ones_of_other_tokens(dt):
    """grad_q of a token is held to the bound of its own incoming gradient."""
    q, k, v, lam, go = inputs(1, 140, 130, 2, 2, 64, 64, DT[dt], 22)
    go[:, ::2] *= 4000.0
    go[:, 1::2] *= 1.0 / 4096
    gq = grads_of(q, k, v, lam, go)[0]
    for i in range(0, 140, 9):
        at = slice(i, i + 1)
        r = ref.attn(q[:, at], k, v, lam, grad_out=go[:, at])
        ref.check(gq[:, at], *r["q"], f"grad_q of token {i}")


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("Lq,D,Dv", [(1, 64, 128), (150, 64, 128), (70, 32, 32), (40, 128, 128)])
def test_token_first_and_broadcast_inputs(dt, Lq, D, Dv):
    """q, k, v stored [token][image] (an image's stride is below a token's), and keys
    and values that all images share (stride 0)."""
    N, Lk, M, Mk = 3, 200, 4, 2
    q, k, v, lam, go = inputs(N, Lq, Lk, M, Mk, D, Dv, DT[dt], 23)
    kw = dict(causal=True)

    def token_first(t):
        return t.transpose(0, 1).contiguous().transpose(0, 1)

    run_and_check(token_first(q), token_first(k), token_first(v), lam, go, **kw)
    run_and_check(q, k[:1].expand(k.shape), v[:1].expand(v.shape), lam, go, **kw)


def test_gradients_without_the_output():
    """The gradient needs what was saved, not `out`: a caller may let it go."""
    q, k, v, lam, go = inputs(2, 40, 50, 4, 2, 64, 64, torch.bfloat16, 24)
    out, saved = dcnb.diff_attn(q, k, v, lam, save=True)
    for a, b in zip(dcnb.diff_attn_grad(q, k, v, lam, None, saved, go),
                    dcnb.diff_attn_grad(q, k, v, lam, out, saved, go)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("shape,causal", [((1, 400, 400, 2, 1, 64, 64), True),
                                          ((2, 300, 500, 2, 2, 32, 64), False)])
def test_grad_q_is_rounded_once(shape, causal, dt):
    """Root mean square error of grad_q against that of rounding the float64 result once,
    which is 1.  Score gradients rounded to the type before their product would add an
    error of the same size for every term: sqrt(2) and more.  What is left beside the last
    rounding is the row sums' share (weights rounded in the forward pass; their errors
    average over the keys, a quarter of a rounding): sqrt(1 + 1/16) = 1.03."""
    q, k, v, lam, go = inputs(*shape, DT[dt], 25)
    want = ref.attn(q, k, v, lam, causal=causal, grad_out=go)["q"][0]
    got = grads_of(q, k, v, lam, go, causal=causal)[0].double().cpu()
    once = want.to(DT[dt]).double()
    assert (got - want).norm() <= 1.25 * (once - want).norm()


@pytest.mark.parametrize("Lq,Lk,M,Mk", [(2048, 128, 8, 1), (40, 8192, 2, 2)])
def test_long_float32_sums_of_gradients(Lq, Lk, M, Mk):
    """Root mean square errors of float32 gradients that sum many terms (grad_k and grad_v
    2048 tokens of 8 heads, grad_q 8192 keys).  A float32 addition's rounding error is
    2.6e-8 of the sum on average, so n additions one after another of terms with random
    signs are off by 2.6e-8 sqrt(n / 2): 2.4e-6 for 16384 terms, 1.7e-6 for 8192.  Sums of
    64 first, then of those, are off by 2.6e-8 (sqrt(32) + sqrt(n / 128)), at most 4.4e-7;
    the terms themselves (a dot product of 32, an exponential) by 6e-7.  Together 7.5e-7."""
    q, k, v, lam, go = inputs(1, Lq, Lk, M, Mk, 32, 32, torch.float32, 26)
    r = ref.attn(q, k, v, lam, grad_out=go)
    got = dict(zip("qkv", grads_of(q, k, v, lam, go)))
    for name in ("kv" if Lq > Lk else "q"):
        want = r[name][0]
        off = (got[name].double().cpu() - want).norm() / want.norm()
        assert off <= 1e-6, f"grad_{name}: {float(off):.2e}"


def test_long_float32_sums_of_values():
    """The maps' outputs over 8192 keys in one go (enough heads that the keys are not split):
    1.7e-6 for additions one after another, 4.4e-7 in tiles, the weights' own 6e-7."""
    q, k, v, lam, _ = inputs(1, 4, 8192, 160, 160, 8, 8, torch.float32, 27)
    assert dcnb.diff_attn_forward_workspace_size(1, 4, 8192, 160, 160, 8, 8, 0) == 0
    _, (maps, _) = dcnb.diff_attn(q, k, v, lam, save=True)
    want = ref.attn(q, k, v, lam)["maps"][0]
    off = (maps.double().cpu() - want).norm() / want.norm()
    assert off <= 1e-6, f"{float(off):.2e}"
