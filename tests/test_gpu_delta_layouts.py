"""delta_rule on tensors that lie where the kernels cannot read them in place: copied, as documented."""
import pytest
import torch

from gated_linear_recurrence_b200 import delta_rule
from tests.test_gpu_delta import draw, ins

pytestmark = pytest.mark.gpu


def shifted(t):
    """The same values, contiguous, one element off an allocation's start (as pieces of a flat buffer are)."""
    flat = torch.empty(t.numel() + 1, dtype=t.dtype, device=t.device)
    out = flat[1:].view(t.shape)
    out.copy_(t)
    assert out.is_contiguous() and out.data_ptr() % 16
    return out


@pytest.mark.parametrize("dt,n", [("bf16", 70), ("f16", 5), ("f32", 70), ("f32", 200)])
def test_contiguous_tensors_off_16_bytes(cuda_device, dt, n):
    x, S0, dS = draw(dt, 2, n, 2, 64, seed=1)

    def grads(move):
        leaves = [move(t).requires_grad_() for t in (*ins(x), S0)]
        y, S = delta_rule(*leaves[:5], S_init=leaves[5])
        return (y, S, *torch.autograd.grad((y, S), leaves, (move(x["dy"]), move(dS))))

    for got, want in zip(grads(shifted), grads(torch.clone)):
        assert torch.equal(got, want)


def test_gradients_from_a_flat_buffer(cuda_device):
    """Gradients that reach y as pieces of one concatenated tensor."""
    x, S0, _ = draw("bf16", 1, 40, 2, 32, seed=2)
    leaves = [t.requires_grad_() for t in ins(x)]
    y, S = delta_rule(*leaves, S_init=S0)
    flat = torch.cat([torch.ones(3, device="cuda"), y.float().flatten(), S.flatten()])
    w = torch.randn(flat.numel(), device="cuda")
    got = torch.autograd.grad((flat * w).sum(), leaves)
    y, S = delta_rule(*leaves, S_init=S0)
    dy, dS = w[3:3 + y.numel()].view(y.shape).to(y.dtype), w[3 + y.numel():].view(S.shape).clone()
    for g, want in zip(got, torch.autograd.grad((y, S), leaves, (dy, dS))):
        assert torch.equal(g, want)
