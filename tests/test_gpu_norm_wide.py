"""The layer norm of wide rows in number, and its gradients inside a block, against float64."""
import pytest
import torch

from gated_linear_recurrence_b200 import ESA, GatedDelta, PreNorm, layer_norm
from tests.test_gpu_norm import check, draw

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt,wdt", [("f32", "f32"), ("f16", "f16"), ("bf16", "f32")])
@pytest.mark.parametrize("rows,N", [(300, 8200), (170, 8193), (299, 12000), (151, 16383), (400, 16384)])
def test_many_wide_rows(cuda_device, dt, wdt, rows, N):
    """More rows than blocks on the device at once, widths up to the widest, on 16 bytes and off."""
    check(*draw(dt, wdt, rows, N, seed=N, residual=rows % 2 == 0))


@pytest.mark.parametrize("make", [lambda: ESA(64, 2, device="cuda", dtype=torch.float16),
                                  lambda: GatedDelta(64, 2, device="cuda", dtype=torch.bfloat16)])
@pytest.mark.parametrize("norm_dtype", [None, torch.float32])
def test_weight_and_bias_gradients_in_a_block(cuda_device, make, norm_dtype):
    """The block's norm gets the gradient that its mixer returns: dweight = sum dn n, dbias = sum dn, from that."""
    torch.manual_seed(0)
    block = PreNorm(make(), norm_dtype=norm_dtype)
    with torch.no_grad():
        block.weight.add_(0.2 * torch.randn_like(block.weight))
        block.bias.add_(0.1 * torch.randn_like(block.bias))
    dt = block.mixer.W_O.weight.dtype
    x, res = (torch.randn(2, 70, 64, device="cuda").to(dt) for _ in range(2))
    seen = []

    def look(_, args):
        args[0].retain_grad()
        seen.append(args[0])

    block.mixer.register_forward_pre_hook(look)
    y, h = block(x, res)
    torch.autograd.backward([y], [torch.randn_like(y)])
    dn = seen[0].grad.double().reshape(-1, 64)
    hd = h.detach().double().reshape(-1, 64)
    n = (hd - hd.mean(-1, keepdim=True)) / torch.sqrt(hd.var(-1, unbiased=False, keepdim=True) + block.eps)
    half = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}[block.weight.dtype]
    for got, terms in ((block.weight.grad, dn * n), (block.bias.grad, dn)):
        want = terms.sum(0)
        # n passes some 40 float32 roundings, the sum of 140 rows at most 72 more in a chain
        bound = half * want.abs() + 112 * 2.0 ** -24 * terms.abs().sum(0)
        assert bool(((got.double() - want).abs() <= bound).all())
    assert float(block.weight.grad.abs().max()) > 0


def test_a_number_is_no_row(cuda_device):
    x = torch.tensor(1.0, device="cuda")
    with pytest.raises(TypeError):
        layer_norm(x)
    with pytest.raises(TypeError):
        layer_norm(torch.zeros(3, device="cuda"), residual=x)
