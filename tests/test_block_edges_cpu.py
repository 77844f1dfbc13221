"""Refusals of the attention-block operators at the edges of their arguments,
without a GPU: an empty side, a stream or a workspace of another device."""
import pytest
import torch

import deformable_attention_sampling_b200 as dcnb
from deformable_attention_sampling_b200 import _binding
from tests.test_block_abi_cpu import ALIGN, BAD, P, attn, lib  # noqa: F401


@pytest.mark.parametrize("change,status", [
    (dict(k=None), BAD), (dict(v=None), BAD), (dict(k=P[1] + 1), ALIGN), (dict(v=P[2] + 1), ALIGN)])
def test_gradients_of_no_tokens_need_the_keys(lib, change, status):  # noqa: F811
    """The key kernel runs for keys without tokens (it writes zeros) and reads k and v."""
    before = dcnb.dcn_launch_count()
    assert attn(lib, True, Lq=0, **change) == status
    assert dcnb.dcn_launch_count() == before


class _OnDevice:
    """Stands for a tensor of GPU `index`, as far as the checks look at it."""

    def __init__(self, index, nbytes=64):
        self.device, self.nbytes = torch.device("cuda", index), nbytes
        self.is_cuda, self.get_device = True, lambda: index

    def is_contiguous(self):
        return True

    def numel(self):
        return self.nbytes

    def element_size(self):
        return 1


class _Stream:
    def __init__(self, index):
        self.device, self.cuda_stream = torch.device("cuda", index), 0


def test_a_stream_of_another_device_is_refused(monkeypatch):
    """Its launch would run there on this device's addresses."""
    entered = []
    monkeypatch.setattr(torch.cuda, "Stream", _Stream)
    monkeypatch.setattr(torch.cuda, "stream", entered.append)
    _binding._scope(_OnDevice(0), _Stream(0))
    assert len(entered) == 1
    with pytest.raises(ValueError):
        _binding._scope(_OnDevice(0), _Stream(1))
    assert len(entered) == 1


def test_a_workspace_of_another_device_is_refused():
    device = torch.device("cuda", 0)
    assert _binding._workspace(64, device, _OnDevice(0))[1] == 64
    with pytest.raises(ValueError):
        _binding._workspace(64, device, _OnDevice(1))


def test_join_gradient_blocks_of_long_rows(lib):  # noqa: F811
    """A block of 512 threads (up to 4096 channels) or of 1024 (up to 8192) fills a
    multiprocessor by its registers: both lengths have one partial row of each."""
    def blocks(C):
        return dcnb.norm_residual_backward_workspace_size(1, 100000, C, 0, 2) // (16 * C)

    assert blocks(8192) == blocks(4096) and blocks(1024) == 2 * blocks(4096)
