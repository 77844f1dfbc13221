"""norm_residual over rows that blocks share unevenly: teams without a row in a
block's last step, and blocks that take several steps; against the float64
definitions of tests/block_ref.py."""
import pytest
import torch

import deformable_attention_sampling_b200 as dcnb
from tests import block_ref as ref
from tests.test_rope_norm_gpu import DT, NAMES, join_inputs

pytestmark = pytest.mark.gpu


def run_and_check(shape, dtype, norm, gate, bias, eps):
    (x, y, gz, gh), f = join_inputs(*shape, dtype, 41, gate, bias, True, True)
    kw = dict(norm=norm, eps=eps)
    z, h = dcnb.norm_residual(x, y, **f, **kw)
    r = ref.join(x, y, f, **kw)
    ref.check(z, *r["z"], "z")
    ref.check(h, *r["h"], "h")
    grads = dcnb.norm_residual_grad(y, z, gz, gh, **f, **kw)
    r = ref.join_grad(y, z, gz, gh, f, **kw)
    for name, got in zip(NAMES, grads):
        if name in ("x", "y") or f[name] is not None:
            ref.check(got, *r[name], "grad_" + name)


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("norm", ["layer", "rms"])
@pytest.mark.parametrize("N,L,C,gate", [(1, 131, 1024, False), (3, 5, 40, True), (1, 3, 40, False),
                                        (2, 333, 64, True)])
@pytest.mark.parametrize("eps", [0.0, 1e-50])
def test_no_eps(N, L, C, gate, norm, dt, eps):
    """eps = 0 (or 0 in float32): a team without a row must not add 0 / 0 to the sums."""
    run_and_check((N, L, C), DT[dt], norm, gate, True, eps)


@pytest.mark.parametrize("dt,norm,bias", [("f32", "layer", True), ("bf16", "rms", False)])
@pytest.mark.parametrize("N,L,C,gate", [(1, 2501, 1024, False), (3, 1203, 1000, True),
                                        (1, 1001, 4096, False), (2, 388, 8192, True),
                                        (1, 20011, 64, False)])
def test_several_steps_a_block(N, L, C, gate, dt, norm, bias):
    """Blocks walk several rows and end in a step that not every team takes part in:
    prefetched rows, the second row of a team, column sums over steps."""
    run_and_check((N, L, C), DT[dt], norm, gate, bias, 1e-5)
