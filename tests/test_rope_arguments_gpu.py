"""Norm and rotation on arguments that are laid out, or typed, in other ways than usual."""
import pytest
import torch

import exact_io_aware_27_gb300 as fa
from tests.test_rope_gpu import _inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _built():
    fa.build()
    yield
    assert fa.fa_get_device_status() == 0


def test_a_gradient_off_its_alignment():
    """A contiguous gradient that starts between two 16-byte boundaries."""
    q, k, pos, table, wq, wk, dq, dk = _inputs(33, 4, 2, 64, 64, 96)
    x, y = q.clone().requires_grad_(), k.clone().requires_grad_()
    out = fa.qk_norm_rope(x, y, pos, table, wq, wk)
    off = []
    for g in (dq, dk):
        flat = torch.empty(g.numel() + 1, dtype=torch.bfloat16, device="cuda")
        off.append(flat[1:].view(g.shape).copy_(g))
        assert off[-1].is_contiguous() and off[-1].data_ptr() % 16 != 0
    got = torch.autograd.grad(out, (x, y), off)
    want = fa.fa_qk_norm_rope_backward(dq, dk, q, k, pos, table, wq, wk)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_an_argument_without_a_truth_value():
    q, k, pos, table, wq, wk, dq, dk = _inputs(5, 4, 2, 64, 64, 97)
    with pytest.raises(RuntimeError):
        fa.fa_qk_norm_rope(q, k, pos, table, wq, wk, interleaved=torch.zeros(2))
