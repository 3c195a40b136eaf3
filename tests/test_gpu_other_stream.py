"""The delta rule's and the norm's calls on a stream that is not the current one."""
import pytest
import torch

from gated_linear_recurrence_b200 import esa_delta_bwd, esa_delta_fwd, esa_delta_step, esa_norm_bwd, esa_norm_fwd
from gated_linear_recurrence_b200.esa import load_library
from tests.test_gpu_delta import draw, ins

pytestmark = pytest.mark.gpu


def busy(stream):
    """Some 20 ms of waiting in front of what is put on the stream next."""
    with torch.cuda.stream(stream):
        torch.cuda._sleep(40_000_000)


def fill_behind(sizes):
    """Allocate and fill on the current stream, as a program that goes on does."""
    return [torch.full((n,), 171, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(3)]


def untouched(fills):
    return all(bool((t == 171).all()) for t in fills)


@pytest.mark.parametrize("rows,N,dt", [(300, 512, torch.bfloat16), (64, 129, torch.float32), (5, 8192, torch.float16)])
def test_norm_backward_keeps_its_workspace(cuda_device, rows, N, dt):
    """The sums' workspace belongs to the call's stream: the current stream's next allocations are not given it."""
    x, w, dy = (torch.randn(s, device="cuda").to(dt) for s in ((rows, N), (N,), (rows, N)))
    y, h, stats = esa_norm_fwd(x, w, w)
    want = esa_norm_bwd(dy, h, w, stats)
    code = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}[dt]
    size = load_library().esa_norm_workspace_size(rows, N, code, code)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    busy(s)
    got = esa_norm_bwd(dy, h, w, stats, stream=s)
    fills = fill_behind([size])
    torch.cuda.synchronize()
    assert untouched(fills)
    for g, t in zip(got, want):
        assert torch.equal(g, t)


@pytest.mark.parametrize("dt,T", [("bf16", 100), ("f32", 200), ("f32", 20)])
@pytest.mark.parametrize("keep", [False, True])
def test_delta_calls(cuda_device, dt, T, keep):
    x, S0, dS = draw(dt, 1, T, 2, 64, seed=3)
    y0, S, ws0 = esa_delta_fwd(*ins(x), S_init=S0, keep=keep)
    want = esa_delta_bwd(*ins(x), x["dy"], ws0, S_init=S0, dS_final=dS) if keep else ()
    size = ws0.numel()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    busy(s)
    y, S1, ws = esa_delta_fwd(*ins(x), S_init=S0, keep=keep, stream=s)
    got = esa_delta_bwd(*ins(x), x["dy"], ws, S_init=S0, dS_final=dS, stream=s) if keep else ()
    del ws
    fills = fill_behind([size])
    torch.cuda.synchronize()
    assert untouched(fills)
    for g, t in zip((y, S1, *got), (y0, S, *want)):
        assert torch.equal(g, t)


def test_step_and_norm_forward(cuda_device):
    x, S0, _ = draw("bf16", 3, 1, 2, 64, seed=4)
    tok = [t[:, 0].contiguous() for t in ins(x)]
    want_S, S = S0.clone(), S0.clone()
    want = esa_delta_step(*tok, want_S)
    h = torch.randn(100, 96, device="cuda")
    want_n = esa_norm_fwd(h, residual=h)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    busy(s)
    y = esa_delta_step(*tok, S, stream=s)
    n = esa_norm_fwd(h, residual=h, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(y, want) and torch.equal(S, want_S)
    assert all(torch.equal(a, b) for a, b in zip(n, want_n))
