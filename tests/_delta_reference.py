"""The gated delta rule and the layer norm from their definitions, in float64
on the CPU, one token (one row) at a time, with torch's autograd for the
gradients; and the error bounds that the GPU results are held to.

Bounds.  A kernel rounds an output once to its type: at most
``finfo(type).eps / 2`` of the value.  Before that its arithmetic is float32.
In the delta rule a token's dot products have chains of D / 16 packed
multiply-adds, one addition of the pair and three of the shuffle tree (12 for
D = 128), and the update has 4 more roundings, so a token adds at most
``20 * 2^-24`` of the largest magnitude it handles; with |k| <= 1 and
alpha <= 1 the recurrence does not amplify, so T tokens add at most T times
that (worst case, element by element) and sqrt(T) times that in the 2-norm
(independent roundings).  A gradient goes through two such sweeps.
"""
import torch

HALF = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
PER_TOKEN = 20 * 2.0 ** -24


def delta_reference(q, k, v, a, b, scale, S0, dy=None, dS=None):
    """Inputs any dtype / device -> dict of float64 CPU tensors (y, S and, with dy, the gradients)."""
    names = ("q", "k", "v", "a", "b")
    x = [t.detach().cpu().double() for t in (q, k, v, a, b)]
    B, T, H, D = x[0].shape
    S0 = torch.zeros(B, H, D, D, dtype=torch.float64) if S0 is None else S0.detach().cpu().double()
    leaves = [t.clone().requires_grad_(dy is not None) for t in (*x, S0)]
    q, k, v, a, b, S = leaves
    alpha, beta = torch.sigmoid(a.clamp(min=-80.0)), torch.sigmoid(b.clamp(min=-80.0))
    y = []
    for t in range(T):
        S = alpha[:, t, :, None, None] * S
        u = beta[:, t, :, None] * (v[:, t] - torch.einsum("bhij,bhi->bhj", S, k[:, t]))
        S = S + k[:, t, :, :, None] * u[:, :, None, :]
        y.append(scale * torch.einsum("bhij,bhi->bhj", S, q[:, t]))
    y = torch.stack(y, 1) if T else torch.zeros_like(v)
    out = {"y": y.detach(), "S": S.detach()}
    if dy is not None:
        loss = (y * dy.detach().cpu().double()).sum()
        if dS is not None:
            loss = loss + (S * dS.detach().cpu().double()).sum()
        grads = torch.autograd.grad(loss, leaves, allow_unused=True)
        for n, g, leaf in zip((*names, "S0"), grads, leaves):
            out["d" + n] = torch.zeros_like(leaf) if g is None else g
    return out


def norm_reference(x, w, c, eps, residual=None, dy=None, dh=None):
    """float64 CPU layer norm: dict y, h, mean, rstd (and dx, dweight, dbias with dy)."""
    N = x.shape[-1]
    h = x.detach().cpu()
    if residual is not None:
        h = (h.float() + residual.detach().cpu().float()).to(x.dtype)   # the stream is stored in its type
    h = h.double().requires_grad_(dy is not None)
    w = torch.ones(N).double() if w is None else w.detach().cpu().double()
    c = torch.zeros(N).double() if c is None else c.detach().cpu().double()
    w.requires_grad_(dy is not None)
    c.requires_grad_(dy is not None)
    mean = h.mean(-1, keepdim=True)
    rstd = 1.0 / torch.sqrt(((h - mean) ** 2).mean(-1, keepdim=True) + eps)
    y = (h - mean) * rstd * w + c
    out = {"y": y.detach(), "h": h.detach(), "mean": mean.detach()[..., 0], "rstd": rstd.detach()[..., 0]}
    if dy is not None:
        loss = (y * dy.detach().cpu().double()).sum()
        if dh is not None:
            loss = loss + (h * dh.detach().cpu().double()).sum()
        out["dx"], out["dweight"], out["dbias"] = torch.autograd.grad(loss, (h, w, c))
    return out


def assert_within(name, got, ref, absolute, norm_rel):
    """|got - ref| <= half a step of got's type + `absolute` max|ref| for every element, and the 2-norm of the
    difference within half a step + `norm_rel` of the reference's."""
    half = HALF[got.dtype]
    g = got.detach().cpu().double()
    assert g.shape == ref.shape, (name, g.shape, ref.shape)
    if g.numel() == 0:
        return
    assert torch.isfinite(g).all(), f"{name}: non-finite"
    err, top = (g - ref).abs(), float(ref.abs().max())
    tiny = torch.finfo(got.dtype).tiny * half * 2   # a subnormal result is off by half a subnormal step
    over = err - (half * (ref.abs() + absolute * top) + absolute * top + tiny)
    assert float(over.max()) <= 0, f"{name}: off by {float(err.max()):.3e} (largest value {top:.3e})"
    n = float(ref.norm())
    if n > 0:
        rel = float((g - ref).norm()) / n
        assert rel <= half + norm_rel + tiny * g.numel() ** 0.5 / n, f"{name}: 2-norm off by {rel:.3e}"
