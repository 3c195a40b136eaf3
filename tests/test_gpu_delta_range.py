"""The gated delta rule in chunks at the ends of float32's range: factors whose products leave it, values far apart.

The bounds are test_gpu_delta's: half a step of the output's type, 20 float32 roundings a token, and for 16-bit
outputs three float16 roundings of intermediates.
"""
import pytest
import torch

from tests._delta_reference import delta_reference
from tests.test_gpu_delta import check, draw, ins, run

pytestmark = pytest.mark.gpu

T = 200
HALF_P = 3 * 2.0 ** -11
# each way the work is spread over the device: warps and blocks of the chains by heads and D
SPREADS = [(32, 2), (64, 2), (64, 80), (128, 2), (128, 40), (128, 80)]


def two_heads(x, S0, dS, out):
    """The first two heads of the inputs and results, and their reference."""
    D = x["q"].shape[-1]
    xs = {n: t[:, :, :2] for n, t in x.items()}
    got = {n: t[:, :2] if n in ("S", "dS0") else t[:, :, :2] for n, t in out.items() if t is not None}
    S0, dS = (None if t is None else t[:, :2] for t in (S0, dS))
    return xs, got, delta_reference(*ins(xs), D ** -0.5, S0, xs["dy"], dS)


@pytest.mark.parametrize("D,H", SPREADS)
@pytest.mark.parametrize("dt,which,factor", [("bf16", "q", 1e-8), ("bf16", "k", 1e-8), ("bf16", "q", 1e8), ("f16", "q", 1e-3),
                                             ("f16", "k", 1e-3)])
def test_queries_and_keys_of_different_size(cuda_device, dt, which, factor, D, H):
    """dq has the queries' gradient through dP K: its unit is not the one in which dP^T Q joins dk."""
    x, S0, dS = draw(dt, 1, T, H, D, seed=3)
    x[which] = (x[which].float() * factor).to(x[which].dtype)
    if factor > 1:   # gradients of the size of dy times q
        x["dy"] = (x["dy"].float() / factor).to(x["dy"].dtype)
    xs, got, ref = two_heads(x, S0, dS, run(x, S0, dS, D ** -0.5))
    check(xs, got, ref, T, D, half_p=HALF_P)


@pytest.mark.parametrize("D,H", SPREADS)
@pytest.mark.parametrize("state", [False, True])
@pytest.mark.parametrize("where", ["start", "middle", "end", "all"])
def test_closed_write_gates(cuda_device, where, state, D, H):
    """Chunks in which nothing is written (padding, b = -inf: beta = e^-80), from a state of zeros and from another:
    what the chunk writes is 2^-115 of what it reads."""
    x, S0, dS = draw("bf16", 1, T, H, D, seed=3, state=state)
    x["b"][:, {"start": slice(0, 64), "middle": slice(64, 128), "end": slice(128, T), "all": slice(0, T)}[where]] = float("-inf")
    xs, got, ref = two_heads(x, S0, dS, run(x, S0, dS, D ** -0.5))
    if where == "all":
        # the reference's clamp passes no gradient; the kernel's is u.du with |u| <= e^-80 (|v| + |S k|) < 1e-33, |du| < 1e2
        assert float(got["db"].abs().max()) < 1e-31
        got["db"] = None
    check(xs, got, ref, T, D, half_p=HALF_P)


@pytest.mark.parametrize("D,H", SPREADS)
@pytest.mark.parametrize("which", ["v", "dy"])
def test_tiny_values(cuda_device, which, D, H):
    x, _, _ = draw("bf16", 1, T, H, D, seed=4, state=False)
    x[which] = (x[which].float() * 1e-30).to(x[which].dtype)
    xs, got, ref = two_heads(x, None, None, run(x, None, None, D ** -0.5))
    check(xs, got, ref, T, D, half_p=HALF_P)
