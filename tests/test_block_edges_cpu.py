"""Refusals of the attention-block operators at the edges of their arguments,
without a GPU: an empty side, a stream or a workspace of another device."""
import pytest

import deformable_attention_sampling_b200 as dcnb
from tests.test_block_abi_cpu import ALIGN, BAD, P, attn, lib  # noqa: F401


@pytest.mark.parametrize("change,status", [
    (dict(k=None), BAD), (dict(v=None), BAD), (dict(k=P[1] + 1), ALIGN), (dict(v=P[2] + 1), ALIGN)])
def test_gradients_of_no_tokens_need_the_keys(lib, change, status):  # noqa: F811
    """The key kernel runs for keys without tokens (it writes zeros) and reads k and v."""
    before = dcnb.dcn_launch_count()
    assert attn(lib, True, Lq=0, **change) == status
    assert dcnb.dcn_launch_count() == before
