"""The layer norm on the GPU against the float64 definition.

Bounds.  Outputs are rounded once (half a step).  Before that: the mean and
the variance are float32 sums in which an element passes at most N / (TPR)
additions of its thread and 10 of the tree, 26 roundings for the widest rows;
n and y add 4.  So y is off by at most 40 * 2^-24 of the largest |y| and of
the mean's share |mean| rstd |w|; dx likewise through two more row sums; the
column sums add rows / 1024 + 64 terms in a chain.
"""
import pytest
import torch

from gated_linear_recurrence_b200 import EsaError, esa_norm_bwd, esa_norm_fwd
from tests._delta_reference import assert_within, norm_reference

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
E = 2.0 ** -24


def draw(dt, wdt, rows, N, seed=0, residual=True, mean=0.3):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)   # noqa: E731
    x = (r(rows, N) + mean * r(rows, 1)).to(DT[dt]).cuda()
    res = r(rows, N).to(DT[dt]).cuda() if residual else None
    w, c = (1 + 0.2 * r(N)).to(DT[wdt]).cuda(), (0.1 * r(N)).to(DT[wdt]).cuda()
    return x, res, w, c, r(rows, N).to(DT[dt]).cuda(), (r(rows, N).to(DT[dt]).cuda() if residual else None)


def check(x, res, w, c, dy, dh, eps=1e-5):
    y, h, stats = esa_norm_fwd(x, w, c, eps=eps, residual=res)
    dx, dw, dc = esa_norm_bwd(dy, h, w, stats, dh=dh)
    ref = norm_reference(x, w, c, eps, res, dy, dh)
    rows, N = x.shape
    assert torch.equal(h.cpu().double(), ref["h"])
    share = float((ref["mean"].abs() * ref["rstd"]).max()) if rows else 0.0
    grow = 1 + share + float(ref["y"].abs().max()) if rows else 1.0
    assert_within("y", y, ref["y"], 40 * E * grow, 40 * E * grow)
    assert_within("mean", stats[:, 0], ref["mean"], 40 * E * max(1.0, float(ref["h"].abs().max()) / max(1e-30, float(ref["mean"].abs().max()))), 1.0)
    assert_within("rstd", stats[:, 1], ref["rstd"], 40 * E * (1 + share), 40 * E * (1 + share))
    assert_within("dx", dx, ref["dx"], 80 * E * grow, 80 * E * grow)
    chain = (64 + rows / 256) * E
    # a column sum can cancel: its error goes by the sum of the terms' sizes
    n = (ref["h"] - ref["mean"][:, None]) * ref["rstd"][:, None]
    for name, got, terms in (("dweight", dw, dy.cpu().double() * n), ("dbias", dc, dy.cpu().double())):
        big = terms.abs().sum(0)
        half = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}[got.dtype]
        off = (got.cpu().double() - ref[name]).abs()
        assert bool((off <= half * ref[name].abs() + (chain + 40 * E * grow) * big + 1e-30).all()), name


@pytest.mark.parametrize("dt,wdt", [("f32", "f32"), ("f16", "f16"), ("bf16", "bf16"), ("f16", "f32"), ("bf16", "f32")])
@pytest.mark.parametrize("rows,N", [(1, 1), (3, 2), (5, 7), (4, 8), (9, 31), (130, 32), (17, 64), (33, 100), (64, 128),
                                    (7, 129), (19, 255), (40, 256), (3, 512), (11, 1000), (5, 1024), (6, 1026),
                                    (3, 2047), (4, 4096), (2, 5001), (3, 8192), (2, 8200), (2, 12345), (2, 16384)])
def test_forward_and_backward(cuda_device, dt, wdt, rows, N):
    check(*draw(dt, wdt, rows, N, seed=N, residual=N % 2 == 0))


@pytest.mark.parametrize("rows,N", [(20000, 128), (3001, 257), (1500, 2048)])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_many_rows(cuda_device, dt, rows, N):
    check(*draw(dt, "f32", rows, N, seed=rows))


def test_far_mean(cuda_device):
    """Rows far from zero keep their variance: the sum of squared differences, not of squares."""
    check(*draw("f32", "f32", 8, 512, seed=1, residual=False, mean=1000.0))


def test_constant_rows(cuda_device):
    x = torch.full((4, 96), 2.5, device="cuda")
    y, h, stats = esa_norm_fwd(x, None, None, eps=1e-5)
    assert not y.any() and bool((stats[:, 1] == torch.tensor(1e-5).rsqrt().item()).all() or
                                ((stats[:, 1] - 1e-5 ** -0.5).abs() <= 1e-4).all())
    dx, dw, db = esa_norm_bwd(torch.ones_like(x), h, None, stats)
    assert not dx.any() and not dw.any() and bool((db == 4).all())


def test_nan_and_infinity_stay_in_their_row(cuda_device):
    x, _, w, c, dy, _ = draw("bf16", "f32", 6, 128, seed=3, residual=False)
    clean, h, stats = esa_norm_fwd(x, w, c)
    cdx, _, _ = esa_norm_bwd(dy, h, w, stats, want_dweight=False, want_dbias=False)
    x2 = x.clone()
    x2[2, 5] = float("nan")
    x2[4, 7] = float("inf")
    y, h, stats = esa_norm_fwd(x2, w, c)
    dx, _, _ = esa_norm_bwd(dy, h, w, stats, want_dweight=False, want_dbias=False)
    ok = [0, 1, 3, 5]
    assert torch.equal(y[ok], clean[ok]) and torch.equal(dx[ok], cdx[ok])
    assert bool(y[2].isnan().all()) and bool(y[4].isnan().all())


def test_strided_rows_and_in_place(cuda_device):
    x, res, w, c, dy, dh = draw("f16", "f16", 12, 64, seed=4)
    y0, h0, s0 = esa_norm_fwd(x, w, c, residual=res)
    g0 = esa_norm_bwd(dy, h0, w, s0, dh=dh)
    for step in (72, 65):   # rows that start on 16 bytes, and rows that do not
        wide = [torch.zeros(3, 4, step, dtype=torch.float16, device="cuda")[..., :64] for _ in range(4)]
        for v, t in zip(wide, (x, res, dy, dh)):
            v.copy_(t.view(3, 4, 64))
        y, h, s = esa_norm_fwd(wide[0], w, c, residual=wide[1])
        assert torch.equal(y.view(12, 64), y0) and torch.equal(h.view(12, 64), h0)
        g = esa_norm_bwd(wide[2], h, w, s, dh=wide[3])
        for a, b in zip(g, g0):
            assert torch.allclose(a.reshape(b.shape).float(), b.float(), rtol=2.0 ** -10, atol=1e-4)
    # the stream updated in place, and dx over dh
    r = res.clone()
    y, h, s = esa_norm_fwd(x, w, c, residual=r, h=r)
    assert torch.equal(y, y0) and torch.equal(r, h0)
    d = dh.clone()
    dx, _, _ = esa_norm_bwd(dy, r, w, s, dh=d, dx=d)
    assert torch.equal(d, g0[0])


@pytest.mark.parametrize("dt", ["f32", "f16"])
@pytest.mark.parametrize("rows,N", [(1, 1), (2, 3), (19, 5), (9, 131), (37, 300), (13, 511), (5, 1001), (700, 1501),
                                    (3, 4095), (4, 5001), (3, 8191), (2, 12345), (2, 16383)])
@pytest.mark.parametrize("alike", [False, True])
def test_any_alignment_and_nothing_written_outside(cuda_device, dt, rows, N, alike):
    """Every tensor at its own distance from a 16-byte boundary, or all at the same, inside a buffer whose other
    elements stay as they were and, as they are not a number, show if they are used."""
    x, res, w, c, dy, dh = draw(dt, dt, rows, N, seed=N)
    room = 64

    def at(t, shift):
        buf = torch.full((2 * room + t.numel(),), float("nan"), dtype=t.dtype, device="cuda")
        view = buf[room // 2 + (1 if alike else shift):][:t.numel()].view(t.shape)
        view.copy_(t)
        return buf, view

    outside = lambda buf, view: buf.isnan().sum() - view.isnan().sum() == 2 * room   # noqa: E731
    plain = esa_norm_fwd(x, w, c, residual=res)
    grads = esa_norm_bwd(dy, plain[1], w, plain[2], dh=dh)
    bufs = {n: at(t, s) for n, t, s in (("x", x, 1), ("res", res, 3), ("w", w, 1), ("c", c, 2), ("dy", dy, 5), ("dh", dh, 2),
                                        ("y", torch.zeros_like(x), 7), ("h", torch.zeros_like(x), 6),
                                        ("dx", torch.zeros_like(x), 1), ("dw", torch.zeros_like(w), 3),
                                        ("dc", torch.zeros_like(w), 5))}
    v = {n: t for n, (_, t) in bufs.items()}
    y, h, st = esa_norm_fwd(v["x"], v["w"], v["c"], residual=v["res"], y=v["y"], h=v["h"])
    dx, dw, dc = esa_norm_bwd(v["dy"], h, v["w"], st, dh=v["dh"], dx=v["dx"], dweight=v["dw"], dbias=v["dc"])
    assert torch.equal(h, plain[1])
    ref = norm_reference(x, w, c, 1e-5, res, dy, dh)
    tol = 100 * E * (1 + float(ref["y"].abs().max()))
    assert_within("y", y, ref["y"], tol, tol)
    assert_within("dx", dx, ref["dx"], tol, tol)
    for a, b in zip((dw, dc), grads[1:]):   # two orders of one sum, each a float32 chain, then a rounding each
        size = (dy.float().abs() * (1 + ref["y"].abs().max())).sum(0)
        step = torch.finfo(a.dtype).eps
        assert bool(((a.float() - b.float()).abs() <= step * b.float().abs() + 200 * E * size).all())
    for buf, view in bufs.values():
        assert outside(buf, view)
    # rows apart from one another, which lets each row start elsewhere
    ld = N + (8 if alike else 3)
    wide = [torch.full((rows, ld), float("nan"), dtype=x.dtype, device="cuda")[:, :N] for _ in range(4)]
    for u, t in zip(wide, (x, res, dy, dh)):
        u.copy_(t)
    y, h, st = esa_norm_fwd(wide[0], w, c, residual=wide[1])
    assert torch.equal(h, plain[1])
    assert_within("y", y, ref["y"], tol, tol)
    assert_within("dx", esa_norm_bwd(wide[2], h, w, st, dh=wide[3])[0], ref["dx"], tol, tol)


def test_no_rows(cuda_device):
    x = torch.empty(0, 32, device="cuda")
    y, h, s = esa_norm_fwd(x, torch.ones(32, device="cuda"), None)
    dx, dw, db = esa_norm_bwd(x, h, torch.ones(32, device="cuda"), s)
    assert dx.shape == x.shape and not dw.any() and not db.any()


def test_same_sums_every_time_and_in_a_graph(cuda_device):
    x, res, w, c, dy, dh = draw("bf16", "f32", 5000, 320, seed=6)
    y, h, s = esa_norm_fwd(x, w, c, residual=res)
    want = esa_norm_bwd(dy, h, w, s, dh=dh)
    for _ in range(3):
        for a, b in zip(esa_norm_bwd(dy, h, w, s, dh=dh), want):
            assert torch.equal(a, b)
    st, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(st):
        torch.cuda.synchronize()
        with torch.cuda.graph(g, stream=st):
            y2, h2, s2 = esa_norm_fwd(x, w, c, residual=res)
            got = esa_norm_bwd(dy, h2, w, s2, dh=dh)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(y2, y)
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_refusals(cuda_device):
    x, res, w, c, dy, dh = draw("f16", "f16", 4, 32, seed=7)
    with pytest.raises(TypeError):
        esa_norm_fwd(x, w.to(torch.bfloat16), c)
    with pytest.raises(TypeError):
        esa_norm_fwd(x, w.float(), c)
    with pytest.raises(ValueError):
        esa_norm_fwd(x, w[:16], c)
    with pytest.raises(ValueError):
        esa_norm_fwd(x, w, c, residual=res[:2])
    with pytest.raises(ValueError):
        esa_norm_fwd(x.t(), None, None)
    with pytest.raises(ValueError):
        esa_norm_fwd(x[:, :1].expand(4, 32), w, c)
    with pytest.raises(ValueError):
        esa_norm_fwd(x, w, c, h=x.clone())
    with pytest.raises(EsaError):
        esa_norm_fwd(x, w, c, eps=-1.0)
    with pytest.raises(EsaError):
        esa_norm_fwd(torch.zeros(2, 16385, device="cuda"))
    y, h, s = esa_norm_fwd(x, w, c)
    with pytest.raises(ValueError):
        esa_norm_bwd(dy, h, w, s[:2])
    with pytest.raises(EsaError):
        esa_norm_bwd(dy, h, w, s, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
