"""Host logic of the delta rule's and the layer norm's autograd functions and
of the layers on top of them, on the CPU: the library calls are replaced by
the float64 definitions (test doubles that take the same arguments), so the
plumbing -- layouts, which gradient goes where, states, the step -- is checked
without a GPU, against autograd through a per-token loop of the whole block.
"""
import pytest
import torch

from gated_linear_recurrence_b200 import GatedDelta, PreNorm, delta, delta_rule, layer_norm, norm
from tests._delta_reference import delta_reference


def _delta_fwd(q, k, v, a, b, scale=None, S_init=None, keep=True, want_S_final=True, **_):
    r = delta_reference(q, k, v, a, b, q.shape[-1] ** -0.5 if scale is None else scale, S_init)
    return r["y"].to(q.dtype), (r["S"].to(q.dtype) if want_S_final else None), torch.ones(1) if keep else None


def _delta_bwd(q, k, v, a, b, dy, ws, scale=None, S_init=None, dS_final=None, want_dS_init=True, **_):
    assert ws is not None
    with torch.enable_grad():
        r = delta_reference(q, k, v, a, b, q.shape[-1] ** -0.5 if scale is None else scale, S_init, dy, dS_final)
    return (*(r["d" + n].to(q.dtype) for n in ("q", "k", "v", "a", "b")), r["dS0"].to(q.dtype) if want_dS_init else None)


def _delta_step(q, k, v, a, b, S, scale=None, **_):
    y, S1, _ = _delta_fwd(*(t[:, None] for t in (q, k, v, a, b)), scale=scale, S_init=S)
    S.copy_(S1)
    return y[:, 0]


def _norm_fwd(x, weight=None, bias=None, eps=1e-5, residual=None, want_stats=True, **_):
    h = x if residual is None else x + residual
    mean, var = h.mean(-1, keepdim=True), h.var(-1, unbiased=False, keepdim=True)
    rstd = (var + eps).rsqrt()
    n = (h - mean) * rstd
    y = n * (1 if weight is None else weight) + (0 if bias is None else bias)
    return y, h, torch.stack([mean.reshape(-1), rstd.reshape(-1)], 1) if want_stats else None


def _norm_bwd(dy, h, weight, stats, dh=None, want_dweight=True, want_dbias=True, wdtype=None, **_):
    mean, rstd = (s.reshape(*h.shape[:-1], 1) for s in stats.unbind(1))
    n, g = (h - mean) * rstd, dy * (1 if weight is None else weight)
    dx = rstd * (g - g.mean(-1, keepdim=True) - n * (g * n).mean(-1, keepdim=True)) + (0 if dh is None else dh)
    over = tuple(range(h.dim() - 1))
    return dx, (dy * n).sum(over) if want_dweight else None, dy.sum(over) if want_dbias else None


@pytest.fixture
def doubles(monkeypatch):
    monkeypatch.setattr(delta, "esa_delta_fwd", _delta_fwd)
    monkeypatch.setattr(delta, "esa_delta_bwd", _delta_bwd)
    monkeypatch.setattr(delta, "esa_delta_step", _delta_step)
    monkeypatch.setattr(norm, "esa_norm_fwd", _norm_fwd)
    monkeypatch.setattr(norm, "esa_norm_bwd", _norm_bwd)
    monkeypatch.setattr(norm, "_rows", lambda *a, **k: None)


def _loop(block, x, residual, S):
    """The block per token with plain operations."""
    h = x if residual is None else x + residual
    n = torch.nn.functional.layer_norm(h, (h.shape[-1],), block.weight, block.bias, block.eps)
    m = block.mixer
    B, T, C = x.shape
    H, D = m.head, m.head_dim
    qk = torch.nn.functional.layer_norm(m.W_QK(n).reshape(B, T, 2, H, D), (D,), eps=m.eps) * D ** -0.5
    q, k = qk[:, :, 0], qk[:, :, 1]
    v = m.W_V(n).reshape(B, T, H, D)
    g = torch.sigmoid(m.W_G(n)).reshape(B, T, 2, H)
    ys = []
    for t in range(T):
        S = g[:, t, 0, :, None, None] * S
        u = g[:, t, 1, :, None] * (v[:, t] - torch.einsum("bhij,bhi->bhj", S, k[:, t]))
        S = S + k[:, t, :, :, None] * u[:, :, None]
        ys.append(torch.einsum("bhij,bhi->bhj", S, q[:, t]))
    return m.W_O(torch.stack(ys, 1).reshape(B, T, C)), h, S


@pytest.mark.parametrize("bias,residual", [(True, True), (False, False)])
def test_block_gradients(doubles, bias, residual):
    torch.manual_seed(1)
    B, T, C, H = 2, 5, 64, 2
    block = PreNorm(GatedDelta(C, H, bias=bias, dtype=torch.float64))
    with torch.no_grad():
        block.weight.add_(0.1 * torch.randn(C))
        block.bias.add_(0.1 * torch.randn(C))
    r = lambda *s: torch.randn(*s, dtype=torch.float64, requires_grad=True)   # noqa: E731
    x, res, S0 = r(B, T, C), r(B, T, C) if residual else None, r(B, H, 32, 32)
    leaves = [x, S0, *block.parameters()] + ([res] if residual else [])
    gy, gh, gS = (torch.randn_like(t) for t in (x, x, S0))
    loss = lambda y, h, S: (y * gy).sum() + (h * gh).sum() + (S * gS).sum()   # noqa: E731
    got = block(x, res, state=S0, return_state=True)
    want = _loop(block, x, res, S0)
    for g, w in zip(got, want):
        torch.testing.assert_close(g, w, rtol=1e-9, atol=1e-9)
    for g, w in zip(torch.autograd.grad(loss(*got), leaves), torch.autograd.grad(loss(*want), leaves)):
        torch.testing.assert_close(g, w, rtol=1e-8, atol=1e-8)


def test_steps_and_prefill(doubles):
    torch.manual_seed(2)
    block = PreNorm(GatedDelta(64, 1, dtype=torch.float64))
    x = torch.randn(3, 4, 64, dtype=torch.float64)
    with torch.no_grad():
        y, h, S = block(x, x, state=block.init_state(3).double(), return_state=True)
    St = block.init_state(3).double()
    for t in range(4):
        yt, ht = block.step(x[:, t], x[:, t], St)
        torch.testing.assert_close(yt, y[:, t])
        assert torch.equal(ht, h[:, t])
    torch.testing.assert_close(St, S)
    n = layer_norm(h, block.weight, block.bias)
    out, S2 = block.mixer.prefill(n)
    torch.testing.assert_close(S2, S)
    assert not out.requires_grad


def test_what_is_kept(doubles):
    """Only a call with a gradient to come keeps a workspace; an unused output has a zero gradient."""
    seen = []
    real = delta.esa_delta_fwd
    delta.esa_delta_fwd = lambda *a, **k: (seen.append(k["keep"]), real(*a, **k))[1]
    try:
        z, g = torch.randn(1, 3, 1, 32), torch.randn(1, 3, 1)
        q = z.clone().requires_grad_(True)
        with torch.no_grad():
            delta_rule(q, z, z, g, g)
        delta_rule(z, z, z, g, g)
        y, S = delta_rule(q, z, z, g, g)
        assert seen == [False, False, True]
        assert torch.autograd.grad(S.sum(), q, retain_graph=True)[0].abs().sum() == 0
        assert torch.autograd.grad(y.sum(), q)[0].abs().sum() > 0
    finally:
        delta.esa_delta_fwd = real


def test_gradient_of_a_gradient_is_refused(doubles):
    x = torch.randn(2, 8, requires_grad=True)
    g, = torch.autograd.grad(layer_norm(x).sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):
        g.sum().backward()


def test_layer_shapes_refused():
    with pytest.raises(ValueError):
        GatedDelta(96, 4)       # heads of 24
    with pytest.raises(ValueError):
        GatedDelta(100, 3)
    layer = GatedDelta(64, 2)
    with pytest.raises(ValueError):
        layer(torch.zeros(1, 2, 32))
    with pytest.raises(ValueError):
        layer.step(torch.zeros(1, 32), layer.init_state(1))
    with pytest.raises(TypeError):
        layer_norm(torch.zeros(2, 8))            # no CPU path
    with pytest.raises(TypeError):
        layer(torch.zeros(1, 2, 64))
    assert "unit" not in layer.state_dict()
