"""The float64 references of the delta rule and the layer norm, pinned on the
CPU: closed forms, and their gradients against central differences."""
import torch

from tests._delta_reference import delta_reference, norm_reference


def _inputs(B=2, T=5, H=2, D=4, seed=0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)   # noqa: E731
    k = r(B, T, H, D)
    return dict(q=r(B, T, H, D), k=k / k.norm(dim=-1, keepdim=True), v=r(B, T, H, D), a=r(B, T, H), b=r(B, T, H),
                scale=0.5, S0=r(B, H, D, D)), r(B, T, H, D), r(B, H, D, D)


def test_orthogonal_keys_are_a_table():
    """alpha = beta = 1 (logits +80) and one-hot keys: the state's row i is the value last written with key i."""
    D = 4
    k = torch.eye(D).reshape(1, D, 1, D)
    k = torch.cat([k, k[:, :1]], 1)   # key 0 is written twice
    v = torch.arange(5.0 * D).reshape(1, 5, 1, D)
    big = torch.full((1, 5, 1), 80.0)
    out = delta_reference(k, k, v, big, big, 1.0, None)
    want = v[0, :, 0].double().clone()
    assert torch.allclose(out["S"][0, 0], torch.cat([want[4:5], want[1:4]]), atol=1e-12)
    assert torch.allclose(out["y"][0, :, 0], want, atol=1e-12)


def test_zero_write_strength_only_forgets():
    x, _, _ = _inputs()
    x["b"] = torch.full_like(x["b"], -80.0)
    out = delta_reference(**x)
    decay = torch.sigmoid(x["a"]).prod(1)
    assert torch.allclose(out["S"], decay[..., None, None] * x["S0"], atol=1e-12)


def test_gradients_against_differences():
    x, dy, dS = _inputs()

    def loss(z):
        o = delta_reference(**z)
        return float((o["y"] * dy).sum() + (o["S"] * dS).sum())

    ref = delta_reference(**x, dy=dy, dS=dS)
    e = 1e-6
    for n in ("q", "k", "v", "a", "b", "S0"):
        g = torch.Generator().manual_seed(3)
        d = torch.randn(x[n].shape, generator=g, dtype=torch.float64)
        num = (loss({**x, n: x[n] + e * d}) - loss({**x, n: x[n] - e * d})) / (2 * e)
        assert abs(num - float((ref["d" + n] * d).sum())) <= 1e-7 * (1 + abs(num)), n


def test_norm_gradients_against_differences():
    g = torch.Generator().manual_seed(0)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)   # noqa: E731
    x, w, c, dy, dh = r(5, 7), r(7), r(7), r(5, 7), r(5, 7)

    def loss(x, w, c):
        o = norm_reference(x, w, c, 1e-5)
        return float((o["y"] * dy).sum() + (o["h"] * dh).sum())

    ref = norm_reference(x, w, c, 1e-5, dy=dy, dh=dh)
    e = 1e-6
    for i, n in enumerate(("dx", "dweight", "dbias")):
        base = [x, w, c]
        d = r(*base[i].shape)
        up, dn = list(base), list(base)
        up[i], dn[i] = base[i] + e * d, base[i] - e * d
        num = (loss(*up) - loss(*dn)) / (2 * e)
        assert abs(num - float((ref[n] * d).sum())) <= 1e-7 * (1 + abs(num)), n
