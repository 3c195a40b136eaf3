"""The gradient of the gated delta rule's forget gate, relative to its own size.

da_t is (1 - alpha_t) times a sum of terms that each have the factor alpha_t: where the gate forgets it is small beside
q.dq and v.dv, and must keep its digits all the same.  Bounds: half a step of the type, and for 16-bit results three
float16 roundings of intermediates, as for the other gradients.  float32 results are the difference of sums whose
terms are 1 / alpha_t times as large, each off by what dq and dv are off by (two sweeps of 20 roundings a token).
"""
import math

import pytest
import torch

from tests._delta_reference import HALF, PER_TOKEN, assert_within, delta_reference
from tests.test_gpu_delta import draw, ins, run
from tests.test_gpu_delta_range import SPREADS, two_heads

T = 200
HALF_P = 3 * 2.0 ** -11


def check_da(got, ref, mean):
    extra = HALF_P if got.dtype != torch.float32 else 2 * PER_TOKEN * T ** 0.5 * max(1.0, math.exp(-mean))
    assert_within("da", got, ref, extra, extra)


def gates(x, mean):
    x["a"] = (mean + 0.5 * (x["a"].float() - x["a"].float().mean())).to(x["a"].dtype)


@pytest.mark.parametrize("mean", [30, 3, 0, -2, -4, -6, -30])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_the_bound_rejects(dt, mean):
    """The check passes the rounded gradient and nothing that is off by a twentieth (float32: below -4 its own
    cancellation may be as large)."""
    g = torch.Generator().manual_seed(1)
    r = lambda *s: torch.randn(*s, generator=g)   # noqa: E731
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)   # noqa: E731
    x = {"q": unit(r(1, 80, 2, 32)), "k": unit(r(1, 80, 2, 32)), "v": r(1, 80, 2, 32), "a": r(1, 80, 2), "b": r(1, 80, 2)}
    gates(x, mean)
    ref = delta_reference(*ins(x), 32 ** -0.5, 0.3 * r(1, 2, 32, 32), r(1, 80, 2, 32), 0.1 * r(1, 2, 32, 32))["da"]
    check_da(ref.to(dt), ref, mean)
    if dt == torch.float32 and mean < -4:
        return
    for wrong in (torch.zeros_like(ref), -ref, 0.95 * ref, 1.05 * ref, ref + 0.05 * ref.norm() / ref.numel() ** 0.5):
        with pytest.raises(AssertionError):
            check_da(wrong.to(dt), ref, mean)


@pytest.mark.gpu
@pytest.mark.parametrize("D,H", SPREADS)
@pytest.mark.parametrize("state", [True, False])
@pytest.mark.parametrize("dt,mean", [("bf16", m) for m in (30, 3, 0, -2, -4, -6, -30)] + [("f16", m) for m in (3, 0, -2, -4)]
                         + [("f32", m) for m in (3, 0, -4)])
def test_gate_gradient(cuda_device, dt, mean, state, D, H):
    x, S0, dS = draw(dt, 1, T, H, D, seed=7, state=state)
    gates(x, mean)
    _, got, ref = two_heads(x, S0, dS, run(x, S0, dS, D ** -0.5))
    check_da(got["da"], ref["da"], mean)


@pytest.mark.gpu
@pytest.mark.parametrize("D,H", SPREADS)
def test_gate_gradient_around_a_reset(cuda_device, D, H):
    """Gates that keep nearly all with one that forgets nearly all inside a chunk, at its first token and at its last:
    a reset's own gradient is as small as its alpha, its neighbours' are not."""
    x, S0, dS = draw("bf16", 1, T, H, D, seed=8)
    x["a"].fill_(6.0)
    resets = [20, 64, 100, 127, 199]
    x["a"][:, resets] = -12.0
    _, got, ref = two_heads(x, S0, dS, run(x, S0, dS, D ** -0.5))
    check_da(got["da"], ref["da"], 0)
    check_da(got["da"][:, resets], ref["da"][:, resets], 0)


@pytest.mark.gpu
@pytest.mark.parametrize("n", [1, 15, 16, 17, 33, 48, 63, 64, 65])
def test_gate_gradient_of_short_sequences(cuda_device, n):
    """Every number of whole and partial blocks of 16 tokens; one token more or less in the chunk."""
    x, S0, dS = draw("bf16", 2, n, 2, 64, seed=n)
    gates(x, -3)
    if n < 2:
        x["a"].fill_(-3.0)
    ref = delta_reference(*ins(x), 0.125, S0, x["dy"], dS)
    check_da(run(x, S0, dS, 0.125)["da"], ref["da"], -3)


@pytest.mark.gpu
@pytest.mark.parametrize("D,H", [(32, 2), (64, 2), (64, 65), (128, 2), (128, 17)])
@pytest.mark.parametrize("n", [1, 17, 64, 65, 200, 333])
@pytest.mark.parametrize("mean", [30, 3, 0, -4, -9, -30])
def test_gate_gradient_in_float32(cuda_device, mean, n, D, H):
    """Token sweeps, from end to end and chunk by chunk.  Where every gate keeps a quarter the terms are at most four times
    as large as their sum, else none is larger than the sum's own: the bound of two sweeps, four times."""
    x, S0, dS = draw("f32", 1, n, H, D, seed=n)
    if n > 1:
        gates(x, mean)
    xs, got, ref = two_heads(x, S0, dS, run(x, S0, dS, D ** -0.5))
    # autograd's 1 - sigmoid(a) in float64 is off by 2^-53 e^a of itself, 0.1% at 30: the same factor without the difference
    a = xs["a"].cpu().double()
    want = ref["da"] / (1.0 - torch.sigmoid(a)) / (1.0 + torch.exp(a))
    extra = 4 * 2 * PER_TOKEN * n ** 0.5
    assert_within("da", got["da"], want, extra, extra)


@pytest.mark.gpu
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("n", [5, 7, 200])
def test_gate_gradient_of_one_gate_that_forgets(cuda_device, n, dt):
    """Chunks with one such gate and chunks without; a short 16-bit sequence goes token by token too."""
    x, S0, dS = draw(dt, 1, n, 2, 64, seed=n)
    x["a"].fill_(5.0)
    x["a"][:, [3, n - 1]] = -8.0
    ref = delta_reference(*ins(x), 0.125, S0, x["dy"], dS)["da"]
    da = run(x, S0, dS, 0.125)["da"]
    extra = 4 * 2 * PER_TOKEN * n ** 0.5 if dt == "f32" or n < 8 else HALF_P
    assert_within("da", da, ref, extra, extra)
    assert_within("da of the gates that forget", da[:, [3, n - 1]], ref[:, [3, n - 1]], extra, extra)


@pytest.mark.gpu
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_gate_gradient_of_strided_rows(cuda_device, dt):
    n, H, D = 5 if dt == "bf16" else 70, 2, 64
    x, S0, dS = draw(dt, 2, n, H, D, seed=12)
    gates(x, -4)
    want = run(x, S0, dS, 0.125)["da"]
    P = torch.zeros(2, n, 3 * H * D + 16, dtype=x["q"].dtype, device="cuda")
    q, k, v = (P[..., i * H * D:(i + 1) * H * D].unflatten(-1, (H, D)) for i in range(3))
    a, b = P[..., 3 * H * D + 1:3 * H * D + 1 + H], P[..., 3 * H * D + 5:3 * H * D + 5 + H]
    for dst, name in zip((q, k, v, a, b), "qkvab"):
        dst.copy_(x[name])
    assert torch.equal(run(dict(q=q, k=k, v=v, a=a, b=b, dy=x["dy"]), S0, dS, 0.125)["da"], want)
