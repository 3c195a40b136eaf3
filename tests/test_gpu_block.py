"""The delta rule and the layer norm together on the GPU: the autograd
functions, and stacks of pre-norm blocks with GatedDelta and ESA mixers, whole
sequences, training and token by token.

Bounds.  A float32 projection of 128 channels is a chain of at most 128
roundings, 128 * 2^-24 of the largest value; a block has a handful of such
stages (norm, projections, recurrence, output), two blocks and their backward
some 20: 20 * 128 * 2^-24 = 1.5e-4 of the largest value.  In bfloat16 a stage
rounds by half a step, 2^-8, independently: 40 stages add sqrt(40) 2^-8 = 2.5e-2
in the 2-norm, and the norms of queries and keys pass on at most twice that.
"""
import pytest
import torch

from gated_linear_recurrence_b200 import (ESA, GatedDelta, PreNorm, delta_rule, esa_delta_step, esa_norm_fwd,
                                          layer_norm)
from tests._delta_reference import HALF, assert_within, delta_reference, norm_reference
from tests.test_block_host import _loop

pytestmark = pytest.mark.gpu


def stack(dtype, C=128, H=2, n=2, norm_dtype=None, seed=3):
    torch.manual_seed(seed)
    blocks = torch.nn.ModuleList(PreNorm(GatedDelta(C, H, bias=True), norm_dtype=norm_dtype) for _ in range(n))
    with torch.no_grad():
        for b in blocks:
            b.weight.add_(0.1 * torch.randn(C))
            b.bias.add_(0.1 * torch.randn(C))
            b.mixer.W_G.bias.add_(torch.tensor([3.0] * H + [0.0] * H))
    for b in blocks:
        b.mixer.to("cuda", dtype)
        b.to("cuda")
        if norm_dtype is None:
            b.to(dtype)
    return blocks


def run(blocks, x):
    res = None
    for b in blocks:
        x, res = b(x, res)
    return x + res


def test_stack_matches_float64(cuda_device):
    blocks = stack(torch.float32)
    x = torch.randn(2, 70, 128, device="cuda", requires_grad=True)
    g = torch.randn(2, 70, 128, device="cuda")
    out = run(blocks, x)
    leaves = [x, *blocks.parameters()]
    grads = torch.autograd.grad((out * g).sum(), leaves)
    ref_blocks = stack(torch.float32).cpu().double()
    x64 = x.detach().cpu().double().requires_grad_(True)
    y, res = x64, None
    for b in ref_blocks:
        y, res, _ = _loop(b, y, res, torch.zeros(2, 2, 64, 64, dtype=torch.float64))
    ref = y + res
    ref_grads = torch.autograd.grad((ref * g.cpu().double()).sum(), [x64, *ref_blocks.parameters()])
    assert_within("out", out, ref.detach(), 1.5e-4, 1.5e-4)
    names = ["x"] + [n for n, _ in blocks.named_parameters()]
    for n, a, b in zip(names, grads, ref_grads):
        # a weight's gradient sums 140 tokens' terms, which may cancel: the terms' size is the largest entry's at least
        assert_within(n, a, b, 1.5e-4, 1.5e-4)


@pytest.mark.parametrize("norm_dtype", [None, torch.float32])
def test_bf16_stack_near_float32(cuda_device, norm_dtype):
    blocks = stack(torch.bfloat16, norm_dtype=norm_dtype)
    wide = stack(torch.float32)
    wide.load_state_dict({n: t.float() for n, t in blocks.state_dict().items()})
    x = torch.randn(3, 200, 128, device="cuda").bfloat16()
    g = torch.randn(3, 200, 128, device="cuda").bfloat16()
    xs = [x.clone().requires_grad_(True), x.float().requires_grad_(True)]
    outs = [run(blocks, xs[0]), run(wide, xs[1])]
    rel = lambda a, b: float((a.float() - b.float()).norm() / b.float().norm())   # noqa: E731
    assert rel(*outs) < 5e-2
    ga = torch.autograd.grad((outs[0].float() * g.float()).sum(), [xs[0], *blocks.parameters()])
    gb = torch.autograd.grad((outs[1] * g.float()).sum(), [xs[1], *wide.parameters()])
    assert all(a.dtype == p.dtype for a, p in zip(ga, [xs[0], *blocks.parameters()]))
    assert rel(ga[0], gb[0]) < 5e-2
    num = sum(float((a.float() - b).norm()) ** 2 for a, b in zip(ga, gb))
    den = sum(float(b.norm()) ** 2 for b in gb)
    assert (num / den) ** 0.5 < 5e-2


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("C,H", [(128, 1), (128, 2), (96, 3)])
def test_prompt_then_tokens(cuda_device, dtype, C, H):
    blocks = stack(dtype, C, H)
    x = torch.randn(3, 75, C, device="cuda", dtype=dtype)
    with torch.no_grad():
        want = run(blocks, x)
        y, res, states = x[:, :70], None, []
        for b in blocks:
            y, res, S = b(y, res, return_state=True)
            states.append(S)
        got = [y + res]
        for t in range(70, 75):
            y, res = x[:, t], None
            for b, S in zip(blocks, states):
                y, res = b.step(y, res, S)
            got.append((y + res)[:, None])
    got = torch.cat(got, 1)
    tol = 1.5e-4 if dtype == torch.float32 else 5e-2
    assert float((got.float() - want.float()).norm()) <= tol * float(want.float().norm())


def test_decoding_in_a_graph(cuda_device):
    blocks = stack(torch.bfloat16)
    x = torch.randn(5, 4, 128, device="cuda", dtype=torch.bfloat16)

    def token(xt, states):
        y, res = xt, None
        for b, S in zip(blocks, states):
            y, res = b.step(y, res, S)
        return y + res

    states = [b.init_state(4) for b in blocks]
    want = [token(xt, states).clone() for xt in x]
    states = [b.init_state(4) for b in blocks]
    buf = x[0].clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        token(buf, [t.clone() for t in states])
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = token(buf, states)
    for t in states:
        t.zero_()
    for xt, w in zip(x, want):
        buf.copy_(xt)
        graph.replay()
        assert torch.equal(out, w)


def test_training_step_in_a_graph(cuda_device):
    """Forward and backward of the stack captured and replayed on new inputs."""
    blocks = stack(torch.bfloat16)
    leaves = list(blocks.parameters())
    g = torch.randn(2, 100, 128, device="cuda", dtype=torch.bfloat16)
    xs = [torch.randn(2, 100, 128, device="cuda", dtype=torch.bfloat16) for _ in range(2)]
    step = lambda x: torch.autograd.grad(run(blocks, x), leaves, g)   # noqa: E731
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        want = [step(x) for x in xs]
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    buf = xs[0].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(buf)
    for x, w in zip(xs, want):
        buf.copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, w):
            torch.testing.assert_close(a, b, rtol=0, atol=2 ** -8 * float(b.abs().max()))   # library GEMMs may split differently


@pytest.mark.parametrize("mode", ["controlled", "direct"])
def test_esa_mixer(cuda_device, mode):
    torch.manual_seed(4)
    block = PreNorm(ESA(64, 2, mode=mode, device="cuda", dtype=torch.float16), norm_dtype=torch.float32)
    x, r = (torch.randn(2, 40, 64, device="cuda").half().requires_grad_(True) for _ in range(2))
    y, h, E = block(x, r, return_state=True)
    n, h2, _ = esa_norm_fwd(x.detach(), block.weight.detach(), block.bias.detach(), residual=r.detach())
    assert torch.equal(h, h2)
    y2, E2 = block.mixer(n, return_state=True)
    assert torch.equal(y, y2) and torch.equal(E, E2)
    gx, gr, gw, gb = torch.autograd.grad((y.float().sum() + (h.float() * 0.5).sum()), [x, r, block.weight, block.bias])
    assert torch.equal(gx, gr) and gw.dtype == torch.float32 and all(torch.isfinite(t).all() for t in (gx, gw, gb))
    St = block.init_state(2)
    for t in range(40):
        yt, ht = block.step(x.detach()[:, t], r.detach()[:, t], St)
    # a sequence in chunks against token by token: the state is float32, y is rounded to float16
    assert torch.equal(ht, h[:, -1])
    assert_within("y", yt, y[:, -1].detach().cpu().double(), 8 * HALF[torch.float16], 8 * HALF[torch.float16])


@pytest.mark.parametrize("dtype,T", [(torch.float32, 40), (torch.bfloat16, 150)])
def test_delta_rule_gradients_and_views(cuda_device, dtype, T):
    """Column blocks read in place, transposed views copied, gradients of both outputs, twice through one graph."""
    B, H, D = 2, 3, 64
    torch.manual_seed(6)
    qk = torch.randn(B, T, 2, H, D, device="cuda") / 8
    base = {"qk": qk, "v": torch.randn(B, H, T, D, device="cuda"), "g": torch.randn(B, T, 2, H, device="cuda") + 1,
            "S": torch.randn(B, H, D, D, device="cuda")}
    base = {n: (t if n == "S" else t.to(dtype)).requires_grad_(True) for n, t in base.items()}
    q, k = base["qk"].unbind(2)
    a, b = base["g"].unbind(2)
    y, S = delta_rule(q, k, base["v"].transpose(1, 2), a, b, S_init=base["S"])
    gy, gS = torch.randn_like(y), torch.randn_like(S)
    leaves = list(base.values())
    first = torch.autograd.grad([y, S], leaves, [gy, gS], retain_graph=True)
    again = torch.autograd.grad([y, S], leaves, [gy, gS])
    assert all(torch.equal(s, t) for s, t in zip(first, again))
    ref = delta_reference(q, k, base["v"].transpose(1, 2), a, b, D ** -0.5, base["S"], gy, gS)
    want = [torch.stack([ref["dq"], ref["dk"]], 2), ref["dv"].transpose(1, 2), torch.stack([ref["da"], ref["db"]], 2),
            ref["dS0"]]
    tol = 2e-5 if dtype == torch.float32 else 2 * HALF[dtype]
    for n, got, w in zip(base, first, want):
        assert got.shape == base[n].shape and got.dtype == base[n].dtype
        assert float((got.cpu().double() - w).norm()) <= tol * float(w.norm()), n
    # a gradient broadcast over everything (the sum's) and one that is missing
    q2 = base["qk"].detach()[:, :, 0].clone().requires_grad_(True)
    y, S = delta_rule(q2, k.detach(), base["v"].detach().transpose(1, 2), a.detach(), b.detach())
    d1, = torch.autograd.grad(y.sum(), q2, retain_graph=True)
    d2, = torch.autograd.grad(y, q2, torch.ones_like(y), retain_graph=True)
    assert torch.equal(d1, d2)
    d3, = torch.autograd.grad(S.sum(), q2)
    assert float(d3.abs().max()) == 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_delta_rule_copies_rows_off_16_bytes(cuda_device, dtype):
    torch.manual_seed(7)
    B, T, H, D = 2, 40, 2, 32
    P = torch.randn(B, T, 3 * H * D + 1, device="cuda", dtype=dtype) / 6       # an odd row stride
    q, k, v = (P[..., i * H * D:(i + 1) * H * D].unflatten(-1, (H, D)) for i in range(3))
    flat = torch.randn(B * T * H * D + 1, device="cuda", dtype=dtype)
    g = torch.randn(B, T, H, device="cuda", dtype=dtype)
    want = delta_rule(q.contiguous(), k.contiguous(), v.contiguous(), g, g)
    assert all(torch.equal(x, y) for x, y in zip(delta_rule(q, k, v, g, g), want))
    off = flat[1:].view(B, T, H, D)                                             # contiguous, one element off
    want = delta_rule(q.contiguous(), k.contiguous(), off.clone(), g, g)
    assert all(torch.equal(x, y) for x, y in zip(delta_rule(q, k, off, g, g), want))


@pytest.mark.parametrize("dtype,D,H", [(torch.float32, 32, 2), (torch.bfloat16, 64, 2), (torch.bfloat16, 128, 40)])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_a_gradient_that_is_not_finite_shows(cuda_device, dtype, D, H, value):
    """It reaches its head's gradients of all earlier tokens, no other head, and none behind its chunk of 64."""
    torch.manual_seed(12)
    B, T = 2, 200
    r = lambda *s: torch.randn(*s, device="cuda").to(dtype)   # noqa: E731
    x = [r(B, T, H, D) / 8, r(B, T, H, D) / 16, r(B, T, H, D), r(B, T, H) + 3, r(B, T, H)]
    x = [t.requires_grad_(True) for t in x]
    y, _ = delta_rule(*x)
    dy = r(B, T, H, D)
    dy[1, 70, 1, 5] = value
    grads = torch.autograd.grad(y, x, dy)
    for name, g in zip("qkvab", grads):
        bad = ~g.float().isfinite().reshape(B, T, H, -1).all(-1)
        if name != "q":
            assert bool(bad[1, :71, 1].all()), name
        else:
            assert bool(bad[1, 70, 1]), name
        assert not bad[1, 128:].any() and not bad[0].any() and not bad[1, :, 0].any(), name


def test_against_differences(cuda_device):
    """The gradients along a random direction against central differences of the float32 forward.

    With step s the difference is off by s^2 |third derivative| / 6 and by the forward's rounding over s: s = 2^-7 makes both
    about 1e-4 of the derivative's size, which the sum of the terms' sizes bounds."""
    B, T, H, D = 1, 90, 2, 32
    torch.manual_seed(8)
    r = lambda *s: torch.randn(*s, device="cuda")   # noqa: E731
    ins = [r(B, T, H, D) / 6, r(B, T, H, D) / 6, r(B, T, H, D), r(B, T, H) + 2, r(B, T, H), r(B, H, D, D) / 4]
    w, c, gy, gS = 1 + r(D) / 5, r(D) / 5, r(B, T, H, D), r(B, H, D, D) / 4

    def f(q, k, v, a, b, S0, w, c):
        y, S = delta_rule(q, k, v, a, b, S_init=S0)
        z, h = layer_norm(y, w, c, residual=v)
        return (z.double() * gy).sum() + (h.double() * gy).sum() + (S.double() * gS).sum()

    leaves = [t.clone().requires_grad_(True) for t in (*ins, w, c)]
    grads = torch.autograd.grad(f(*leaves), leaves)
    s = 2.0 ** -7
    for i, (t, g) in enumerate(zip(leaves, grads)):
        d = torch.randn_like(t)
        d = d / d.norm() * t.norm() / 4
        with torch.no_grad():
            up, dn = ([u.detach() + (sg * s * d if j == i else 0) for j, u in enumerate(leaves)] for sg in (1, -1))
            diff = float(f(*up) - f(*dn)) / (2 * s)
        size = float(g.norm() * d.norm())
        assert abs(diff - float((g.double() * d.double()).sum())) <= 1e-3 * size, i


def test_layer_norm_function(cuda_device):
    torch.manual_seed(9)
    x = torch.randn(4, 9, 2, 50, device="cuda")
    view = x[:, :, 0].requires_grad_(True)          # evenly spaced rows, read in place
    flipped = x.transpose(0, 1)[..., ::2]           # copied
    w = torch.randn(50, device="cuda", requires_grad=True)
    g = torch.randn(4, 9, 50, device="cuda")
    y = layer_norm(view, w)
    dx, dw = torch.autograd.grad(y, [view, w], g)
    ref = norm_reference(view.reshape(-1, 50), w, None, 1e-5, None, g.reshape(-1, 50))
    assert_within("y", y.reshape(-1, 50), ref["y"], 100 * HALF[torch.float32], 100 * HALF[torch.float32])
    assert_within("dx", dx.reshape(-1, 50), ref["dx"], 100 * HALF[torch.float32], 100 * HALF[torch.float32])
    assert_within("dw", dw, ref["dweight"], 100 * HALF[torch.float32], 100 * HALF[torch.float32])
    z = layer_norm(flipped)
    assert torch.equal(z, layer_norm(flipped.contiguous()))
    # only the stream's gradient, only the bias's, and neither input
    res = torch.randn_like(view).requires_grad_(True)
    y, h = layer_norm(view, w, residual=res)
    dr, = torch.autograd.grad(h, res, g, retain_graph=True)
    assert torch.equal(dr, g)
    c = torch.zeros(50, device="cuda", requires_grad=True)
    dc, = torch.autograd.grad(layer_norm(view.detach(), None, c), c, g)
    assert_within("dc", dc, g.cpu().double().sum((0, 1)), 100 * HALF[torch.float32], 100 * HALF[torch.float32])
    # gradients of two inputs that are one result do not share memory once they accumulate
    u, r = view.detach().clone().requires_grad_(True), res.detach().clone().requires_grad_(True)
    y, h = layer_norm(u, w, residual=r)
    (y * g).sum().backward()
    before = r.grad.clone()
    u.grad.zero_()
    assert torch.equal(r.grad, before)


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_step_reads_views_in_place(cuda_device, dt):
    torch.manual_seed(11)
    B, H, D = 5, 3, 64
    qk = (torch.randn(B, 2, H, D, device="cuda") / 8).to(dt)
    g = torch.randn(B, 2, H, device="cuda").to(dt)
    vv = torch.randn(B, 4, H, D, device="cuda").to(dt)
    S = torch.randn(B, H, D, D, device="cuda")
    S2 = S.clone()
    q, k = qk.unbind(1)
    a, b = g.unbind(1)
    y = esa_delta_step(q, k, vv[:, 2], a, b, S)
    assert torch.equal(y, esa_delta_step(*(t.contiguous() for t in (q, k, vv[:, 2], a, b)), S2))
    assert torch.equal(S, S2)
    with pytest.raises(ValueError):
        esa_delta_step(q, k.contiguous(), vv[:, 2], a, b, S)        # two strides
    with pytest.raises(ValueError):
        esa_delta_step(qk[:, 0, :1].expand(B, H, D), k, vv[:, 2], a, b, S)
    with pytest.raises(ValueError):
        esa_delta_step(q, k, vv[:, 2], a[:1].expand(B, H), b[:1].expand(B, H), S)
