"""The gated delta rule on the GPU against the float64 definition."""
import pytest
import torch

from gated_linear_recurrence_b200 import (EsaError, PreparedDeltaStep, esa_delta_bwd, esa_delta_fwd, esa_delta_step,
                                          esa_delta_workspace_size)
from tests._delta_reference import HALF, PER_TOKEN, assert_within, delta_reference

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
NAMES = ("q", "k", "v", "a", "b")


def draw(dt, B, T, H, D, seed=0, a_mean=3.0, state=True):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)   # noqa: E731
    unit = lambda x: x / x.norm(dim=-1, keepdim=True).clamp(min=1e-30)   # noqa: E731
    x = {"q": unit(r(B, T, H, D)), "k": unit(r(B, T, H, D)) * 0.99, "v": r(B, T, H, D), "a": r(B, T, H) + a_mean,
         "b": r(B, T, H), "dy": r(B, T, H, D)}
    x = {n: t.to(DT[dt]).cuda() for n, t in x.items()}
    S0 = 0.3 * r(B, H, D, D).cuda() if state else None
    dS = 0.1 * r(B, H, D, D).cuda() if state else None
    return x, S0, dS


def ins(x):
    return [x[n] for n in NAMES]


def check(x, out, ref, T, D, gradients=True, half_p=0.0):
    """`half_p`: further roundings of intermediates, in the 2-norm and per element of the largest value."""
    a, n = PER_TOKEN * max(T, 1), PER_TOKEN * max(T, 1) ** 0.5
    for name in ("y", "S"):
        if out.get(name) is not None:
            extra = half_p if out[name].dtype != torch.float32 else 0.0
            assert_within(name, out[name], ref[name], a + extra, n + extra)
    if gradients:
        for name in ("dq", "dk", "dv", "db", "dS0"):
            if out.get(name) is not None:
                extra = half_p if out[name].dtype != torch.float32 else 0.0
                assert_within(name, out[name], ref[name], 2 * a + extra, 2 * n + extra)
        # da is (1 - alpha) times a sum of q.dq - v.dv over the later tokens, which cancel where alpha is small: its
        # error goes by the terms' sizes, each off by what dq and dv are off by before their rounding
        terms = (x["q"].cpu().double() * ref["dq"]).sum(-1).abs() + (x["v"].cpu().double() * ref["dv"]).sum(-1).abs()
        top = float(terms.max()) + float(ref["da"].abs().max())
        extra = half_p if out["da"].dtype != torch.float32 else 0.0
        off = (out["da"].cpu().double() - ref["da"]).abs()
        half = HALF[out["da"].dtype]
        assert torch.isfinite(off).all() and bool((off <= half * ref["da"].abs() + (2 * a + extra) * top + 1e-30).all()), \
            f"da: off by {float(off.max()):.3e} of {top:.3e}"


def run(x, S0, dS, scale, **kw):
    y, S, ws = esa_delta_fwd(*ins(x), scale=scale, S_init=S0, **kw)
    dq, dk, dv, da, db, dS0 = esa_delta_bwd(*ins(x), x["dy"], ws, scale=scale, S_init=S0, dS_final=dS,
                                            want_dS_init=S0 is not None)
    return dict(y=y, S=S, dq=dq, dk=dk, dv=dv, da=da, db=db, dS0=dS0)


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("B,T,H", [(1, 1, 1), (2, 2, 3), (1, 15, 2), (2, 16, 1), (1, 17, 2), (2, 63, 2), (1, 64, 1),
                                   (1, 65, 2), (2, 131, 3)])
def test_forward_and_backward(cuda_device, dt, D, B, T, H):
    x, S0, dS = draw(dt, B, T, H, D, seed=T)
    out = run(x, S0, dS, D ** -0.5)
    # 16-bit outputs of the chunked kernels: three 16-bit roundings of intermediates, of half a float16 step each
    check(x, out, delta_reference(*ins(x), D ** -0.5, S0, x["dy"], dS), T, D, half_p=3 * 2.0 ** -11)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_without_states(cuda_device, dt):
    x, _, _ = draw(dt, 2, 70, 2, 64, seed=5, state=False)
    out = run(x, None, None, 1.0)
    check(x, out, delta_reference(*ins(x), 1.0, None, x["dy"], None), 70, 64, half_p=3 * 2.0 ** -11)


@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("T", [1, 90])
def test_inference_call_and_many_heads(cuda_device, D, T):
    """Enough heads for whole-head blocks; keep=False; no final state wanted."""
    x, S0, _ = draw("f16", 4, T, 80, D, seed=9)
    y, S, ws = esa_delta_fwd(*ins(x), S_init=S0, keep=False, want_S_final=False)
    assert S is None
    full = run(x, S0, None, None)
    assert torch.equal(y, full["y"])
    pick = slice(1, 2)
    ref = delta_reference(*(t[pick, :, :4] for t in ins(x)), D ** -0.5, S0[pick, :4])
    check(x, {"y": y[pick, :, :4], "S": full["S"][pick, :4]}, ref, T, D, gradients=False, half_p=3 * 2.0 ** -11)


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("T", [7, 8, 31, 32])
def test_short_sequences(cuda_device, dt, D, T):
    """Around the lengths from which chunks are used, with and without a backward to come."""
    x, S0, dS = draw(dt, 2, T, 3, D, seed=T + D)
    ref = delta_reference(*ins(x), D ** -0.5, S0, x["dy"], dS)
    check(x, run(x, S0, dS, None), ref, T, D, half_p=3 * 2.0 ** -11)
    y, S, _ = esa_delta_fwd(*ins(x), S_init=S0, keep=False)
    check(x, {"y": y, "S": S}, ref, T, D, gradients=False, half_p=3 * 2.0 ** -11)


@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("B,T,H,state", [(1, 191, 2, True), (1, 192, 2, True), (2, 333, 3, False), (1, 1100, 1, True)])
def test_long_float32_sequences(cuda_device, D, B, T, H, state):
    """Around the length from which the states between chunks come first; strided inputs, without what the backward
    needs, and a final state over the initial one as well."""
    x, S0, dS = draw("f32", B, T, H, D, seed=T, state=state)
    ref = delta_reference(*ins(x), D ** -0.5, S0, x["dy"], dS)
    check(x, run(x, S0, dS, None), ref, T, D)
    P = torch.zeros(B, T, 3 * H * D + 4, device="cuda")
    for i, n in enumerate("qkv"):
        P[..., i * H * D:(i + 1) * H * D] = x[n].flatten(2)
    q, k, v = (P[..., i * H * D:(i + 1) * H * D].unflatten(-1, (H, D)) for i in range(3))
    over = None if S0 is None else S0.clone()
    y, S, _ = esa_delta_fwd(q, k, v, x["a"], x["b"], S_init=over, S_final=over, keep=False)
    check(x, {"y": y, "S": S}, ref, T, D, gradients=False)


@pytest.mark.parametrize("which", ["forget", "reset_inside"])
def test_long_float32_gates(cuda_device, which):
    x, S0, dS = draw("f32", 1, 260, 2, 64, seed=21)
    if which == "forget":
        x["a"].fill_(-100.0)
    else:
        x["a"].fill_(8.0)
        x["a"][:, 77] = -90.0
        x["a"][:, 200:202] = float("-inf")
    ref = delta_reference(*ins(x), 0.125, S0, x["dy"], dS)
    check(x, run(x, S0, dS, None), ref, 260, 64)


@pytest.mark.parametrize("D,H", [(32, 64), (32, 65), (64, 64), (64, 65), (128, 16), (128, 17)])
def test_long_float32_every_spread_of_heads(cuda_device, D, H):
    x, S0, dS = draw("f32", 1, 200, H, D, seed=H)
    out = run(x, S0, dS, None)
    for h in (0, H - 1):
        one = {n: t[:, :, h:h + 1] for n, t in x.items()}
        ref = delta_reference(*ins(one), D ** -0.5, S0[:, h:h + 1], one["dy"], dS[:, h:h + 1])
        check(one, {n: t[:, h:h + 1] if n in ("S", "dS0") else t[:, :, h:h + 1] for n, t in out.items()}, ref, 200, D)


@pytest.mark.parametrize("what", ["v", "k", "q", "S"])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_long_float32_values_that_are_not_finite(cuda_device, what, value):
    """From their token on, in their value channel (v, S), their head (k) or their token (q) only."""
    D, T = 32, 300
    x, S0, _ = draw("f32", 2, T, 2, D, seed=23)
    clean, _, _ = esa_delta_fwd(*ins(x), S_init=S0)
    if what == "S":
        S0[1, 1, 3, 5] = value
    else:
        x[what][1, 100, 1, 5] = value
    y, S, _ = esa_delta_fwd(*ins(x), S_init=S0)
    same = torch.ones_like(y, dtype=torch.bool)
    if what == "q":
        same[1, 100, 1] = False
    elif what == "k":
        same[1, 100:, 1] = False
    else:
        same[1, 100 if what == "v" else 0:, 1, 5] = False
    assert torch.equal(y[same], clean[same])
    assert not torch.isfinite(y[~same]).all()
    if what == "k":
        assert not torch.isfinite(S[1, 1]).any()


@pytest.mark.parametrize("D", [32, 64, 128])
def test_steps_equal_the_sequence(cuda_device, D):
    T = 21
    x, S0, _ = draw("f32", 3, T, 2, D, seed=2)
    y, S, _ = esa_delta_fwd(*ins(x), S_init=S0)
    St = S0.clone()
    ys = []
    for t in range(T):
        ys.append(esa_delta_step(*(z[:, t].contiguous() for z in ins(x)), St))
    # the same recurrence, summed in another order
    assert_within("y", torch.stack(ys, 1), y.double().cpu(), 2 * PER_TOKEN * T, 2 * PER_TOKEN * T ** 0.5)
    assert_within("S", St, S.double().cpu(), 2 * PER_TOKEN * T, 2 * PER_TOKEN * T ** 0.5)


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("B,H,D", [(1, 1, 32), (3, 5, 32), (1, 8, 64), (2, 3, 64), (1, 2, 128), (40, 4, 128)])
def test_one_token(cuda_device, dt, B, H, D):
    x, S0, _ = draw(dt, B, 1, H, D, seed=B + D)
    S = S0.clone()
    y = esa_delta_step(*(z[:, 0].contiguous() for z in ins(x)), S, scale=0.7)
    ref = delta_reference(*ins(x), 0.7, S0)
    assert_within("y", y, ref["y"][:, 0], PER_TOKEN, PER_TOKEN)
    assert_within("S", S, ref["S"], PER_TOKEN, PER_TOKEN)


def test_prepared_step_and_graph(cuda_device):
    x, S0, _ = draw("bf16", 2, 3, 4, 64, seed=4)
    toks = [[z[:, t].contiguous() for z in ins(x)] for t in range(3)]
    want_S, want = S0.clone(), []
    for t in range(3):
        want.append(esa_delta_step(*toks[t], want_S).clone())
    buf = [z.clone() for z in toks[0]]
    S = S0.clone()
    step = PreparedDeltaStep(*buf, S)
    for t in range(3):
        for z, w in zip(buf, toks[t]):
            z.copy_(w)
        assert torch.equal(step(), want[t])
    assert torch.equal(S, want_S)
    S.copy_(S0)
    st = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(st):
        step = PreparedDeltaStep(*buf, S)
        torch.cuda.synchronize()
        with torch.cuda.graph(g, stream=st):
            y = step()
    S.copy_(S0)
    for t in range(3):
        for z, w in zip(buf, toks[t]):
            z.copy_(w)
        g.replay()
        assert torch.equal(y, want[t])
    assert torch.equal(S, want_S)


@pytest.mark.parametrize("T", [5, 130])
@pytest.mark.parametrize("D", [32, 64, 128])
def test_split_sequence(cuda_device, T, D):
    """Two calls with the state handed over equal one call."""
    x, S0, _ = draw("f32", 2, T, 2, D, seed=6)
    y, S, _ = esa_delta_fwd(*ins(x), S_init=S0)
    c = T // 3
    y1, S1, _ = esa_delta_fwd(*(z[:, :c].contiguous() for z in ins(x)), S_init=S0)
    y2, S2, _ = esa_delta_fwd(*(z[:, c:].contiguous() for z in ins(x)), S_init=S1)
    assert_within("y", torch.cat([y1, y2], 1), y.double().cpu(), 2 * PER_TOKEN * T, 2 * PER_TOKEN * T ** 0.5)
    assert_within("S", S2, S.double().cpu(), 2 * PER_TOKEN * T, 2 * PER_TOKEN * T ** 0.5)


@pytest.mark.parametrize("dt,D,H,T", [("f32", 32, 2, 40), ("bf16", 128, 2, 150), ("bf16", 128, 40, 150), ("f16", 64, 90, 70),
                                      ("bf16", 64, 3, 5)])
def test_final_state_over_the_initial_one(cuda_device, dt, D, H, T):
    x, S0, _ = draw(dt, 2, T, H, D, seed=17)
    y, S, _ = esa_delta_fwd(*ins(x), S_init=S0)
    y2, S2, _ = esa_delta_fwd(*ins(x), S_init=S0, S_final=S0)
    assert S2 is S0 and torch.equal(S, S0) and torch.equal(y, y2)


def test_strided_rows_and_outputs_given(cuda_device):
    B, T, H, D = 2, 77, 2, 64
    C = H * D
    x, S0, dS = draw("bf16", B, T, H, D, seed=8)
    P = torch.full((B, T, 3 * C + 8 + 16), 7.0, dtype=torch.bfloat16, device="cuda")
    q, k, v = (P[..., i * C:(i + 1) * C].view(B, T, H, D) for i in range(3))
    a, b = P[..., 3 * C + 1:3 * C + 1 + H], P[..., 3 * C + 5:3 * C + 5 + H]
    for dst, n in zip((q, k, v, a, b), NAMES):
        dst.copy_(x[n])
    base = run(x, S0, dS, 0.3)
    y = torch.empty(B, T, H, D, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(esa_delta_workspace_size(B, T, H, D, torch.bfloat16), dtype=torch.uint8, device="cuda")
    y2, S, ws2 = esa_delta_fwd(q, k, v, a, b, scale=0.3, S_init=S0, y=y, workspace=ws)
    assert y2 is y and ws2 is ws and torch.equal(y, base["y"]) and torch.equal(S, base["S"])
    g = esa_delta_bwd(q, k, v, a, b, x["dy"], ws, scale=0.3, S_init=S0, dS_final=dS)
    for n, t in zip(("dq", "dk", "dv", "da", "db", "dS0"), g):
        assert torch.equal(t, base[n]), n
    # the column blocks' neighbours are read only
    assert bool((P[..., 3 * C:3 * C + 1] == 7).all()) and bool((P[..., 3 * C + 8:] == 7).all())


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("which", ["forget", "keep", "no_write", "overwrite", "reset_inside", "far_below", "infinite"])
def test_gate_extremes(cuda_device, which, D):
    B, T, H = 1, 150, 2
    x, S0, dS = draw("bf16", B, T, H, D, seed=11)
    if which == "forget":
        x["a"].fill_(-30.0)
    elif which == "keep":
        x["a"].fill_(30.0)
    elif which == "no_write":
        x["b"].fill_(-30.0)
    elif which == "overwrite":
        x["b"].fill_(30.0)
    elif which == "reset_inside":
        x["a"].fill_(6.0)
        x["a"][:, 40] = -60.0
        x["a"][:, 100] = -1000.0
    elif which == "far_below":
        x["a"].fill_(-1.0e4)
        x["b"][:, ::2] = -1.0e4
    else:
        x["a"][:, 20] = float("-inf")
        x["a"][:, 30:] = float("inf")
        x["b"][:, 60:] = float("inf")
    out = run(x, S0, dS, D ** -0.5)
    check(x, out, delta_reference(*ins(x), D ** -0.5, S0, x["dy"], dS), T, D, half_p=3 * 2.0 ** -11)


@pytest.mark.parametrize("scale_v,scale_k", [(1.0e3, 1.0), (1.0e-4, 1.0), (1.0, 1.0e-3), (1.0, 0.0), (0.0, 1.0)])
@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_sizes_of_values(cuda_device, dt, scale_v, scale_k):
    B, T, H, D = 1, 140, 2, 128
    x, _, _ = draw(dt, B, T, H, D, seed=12)
    x["v"] = x["v"] * scale_v
    x["k"] = x["k"] * scale_k
    out = run(x, None, None, D ** -0.5)
    ref = delta_reference(*ins(x), D ** -0.5, None, x["dy"], None)
    check(x, out, ref, T, D, half_p=3 * 2.0 ** -11)


def test_repeated_key(cuda_device):
    """The same key at every token: the chunk matrix is as far from the identity as it gets."""
    B, T, H, D = 1, 200, 1, 128
    x, S0, dS = draw("bf16", B, T, H, D, seed=13, a_mean=8.0)
    x["k"].copy_(x["k"][:, :1].expand_as(x["k"]))
    x["b"].fill_(4.0)
    out = run(x, S0, dS, D ** -0.5)
    check(x, out, delta_reference(*ins(x), D ** -0.5, S0, x["dy"], dS), T, D, half_p=3 * 2.0 ** -11)


def test_no_tokens_and_no_batch(cuda_device):
    S0 = torch.randn(2, 3, 32, 32, device="cuda")
    z = torch.empty(2, 0, 3, 32, device="cuda")
    g = torch.empty(2, 0, 3, device="cuda")
    y, S, ws = esa_delta_fwd(z, z, z, g, g, S_init=S0)
    assert y.shape == z.shape and torch.equal(S, S0)
    _, S, _ = esa_delta_fwd(z, z, z, g, g)
    assert not S.any()
    *_, dS0 = esa_delta_bwd(z, z, z, g, g, z, ws, S_init=S0, dS_final=S0)
    assert torch.equal(dS0, S0)
    z, g = torch.empty(0, 4, 3, 32, device="cuda"), torch.empty(0, 4, 3, device="cuda")
    y, S, ws = esa_delta_fwd(z, z, z, g, g)
    assert y.numel() == 0 and S.numel() == 0


@pytest.mark.parametrize("dt,D", [("bf16", 64), ("f16", 128), ("f32", 32)])
def test_same_results_every_time_and_two_streams(cuda_device, dt, D):
    x, S0, dS = draw(dt, 2, 200, 4, D, seed=14)
    x2, S02, dS2 = draw(dt, 2, 200, 4, D, seed=15)
    first, second = run(x, S0, dS, 0.1), run(x2, S02, dS2, 0.1)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        with torch.cuda.stream(s1):
            a = run(x, S0, dS, 0.1)
        with torch.cuda.stream(s2):
            b = run(x2, S02, dS2, 0.1)
        torch.cuda.synchronize()
        for n in first:
            assert torch.equal(a[n], first[n]) and torch.equal(b[n], second[n]), n


@pytest.mark.parametrize("dt,T,D", [("bf16", 129, 64), ("bf16", 129, 128), ("f32", 70, 64), ("f32", 260, 32), ("f32", 260, 128)])
def test_graph_of_forward_and_backward(cuda_device, dt, T, D):
    x, S0, dS = draw(dt, 1, T, 2, D, seed=16)
    want = run(x, S0, dS, 0.2)
    st = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(st):
        run(x, S0, dS, 0.2)
        torch.cuda.synchronize()
        with torch.cuda.graph(g, stream=st):
            out = run(x, S0, dS, 0.2)
    for t in out.values():
        t.zero_()
    g.replay()
    torch.cuda.synchronize()
    for n in want:
        assert torch.equal(out[n], want[n]), n


@pytest.mark.parametrize("dt,T,H,D", [("f16", 67, 2, 128), ("f32", 67, 2, 64), ("f32", 200, 2, 128), ("f32", 257, 3, 32),
                                      ("bf16", 67, 40, 64), ("bf16", 9, 3, 32), ("f16", 5, 2, 64)])
def test_nothing_written_outside(cuda_device, dt, T, H, D):
    """Canary rows around every output stay as they were."""
    B = 1
    x, S0, dS = draw(dt, B, T, H, D, seed=17)

    def guarded(shape, dtype):
        n = 1
        for s in shape:
            n *= s
        flat = torch.full((n + 512,), 3.0, dtype=dtype, device="cuda")
        return flat, flat[256:256 + n].view(shape)

    h, f = DT[dt], torch.float32
    bufs = {n: guarded(s, t) for n, s, t in (("y", (B, T, H, D), h), ("S", (B, H, D, D), f), ("dq", (B, T, H, D), h),
                                             ("dk", (B, T, H, D), h), ("dv", (B, T, H, D), h), ("da", (B, T, H), h),
                                             ("db", (B, T, H), h), ("dS0", (B, H, D, D), f))}
    need = esa_delta_workspace_size(B, T, H, D, DT[dt])
    wflat = torch.full((need + 512,), 171, dtype=torch.uint8, device="cuda")
    ws = wflat[256:256 + need]
    out = {n: t[1] for n, t in bufs.items()}
    esa_delta_fwd(*ins(x), S_init=S0, y=out["y"], S_final=out["S"], workspace=ws)
    esa_delta_bwd(*ins(x), x["dy"], ws, S_init=S0, dS_final=dS, dq=out["dq"], dk=out["dk"], dv=out["dv"],
                  da=out["da"], db=out["db"], dS_init=out["dS0"])
    torch.cuda.synchronize()
    for n, (flat, _) in bufs.items():
        assert bool((flat[:256] == 3).all()) and bool((flat[-256:] == 3).all()), n
    assert bool((wflat[:256] == 171).all()) and bool((wflat[-256:] == 171).all())
    check(x, out, delta_reference(*ins(x), D ** -0.5, S0, x["dy"], dS), T, D, half_p=3 * 2.0 ** -11)


def test_refusals(cuda_device):
    x, S0, _ = draw("bf16", 1, 8, 2, 64, seed=18)
    q, k, v, a, b = ins(x)
    with pytest.raises(ValueError):
        esa_delta_fwd(q, k[:, :4], v, a, b)
    with pytest.raises(ValueError):
        esa_delta_fwd(q, k.float(), v, a, b)
    with pytest.raises(ValueError):
        esa_delta_fwd(q, k, v, a[..., :1], b)
    with pytest.raises(ValueError):
        esa_delta_fwd(q.transpose(1, 2).contiguous().transpose(1, 2), k, v, a, b)
    with pytest.raises(ValueError):
        esa_delta_fwd(q, k, v, a, b, S_init=S0.half())
    with pytest.raises(ValueError):
        esa_delta_fwd(q, k, v, a, b, y=torch.empty_like(q).float())
    with pytest.raises(TypeError):
        esa_delta_fwd(*(t.to(torch.float8_e4m3fn) for t in (q, k, v, a, b)))
    with pytest.raises(ValueError):
        esa_delta_fwd(*(t[..., :16].contiguous() for t in (q, k, v)), a, b)
    with pytest.raises(EsaError):
        esa_delta_fwd(q, k, v, a, b, scale=float("nan"))
    with pytest.raises(EsaError):
        esa_delta_fwd(q, k, v, a, b, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        esa_delta_bwd(q, k, v, a, b, x["dy"], None)
    with pytest.raises(EsaError):   # rows that do not start on 16 bytes
        wide = torch.zeros(1, 8, 2 * 64 + 4, dtype=torch.bfloat16, device="cuda")
        w = wide[..., :128].view(1, 8, 2, 64)
        esa_delta_fwd(w, w, v, a, b)


@pytest.mark.parametrize("dt,D,H", [("bf16", 128, 2), ("f16", 64, 2), ("bf16", 32, 2), ("f32", 64, 2), ("bf16", 128, 40),
                                    ("f16", 128, 80), ("bf16", 64, 80)])
@pytest.mark.parametrize("what", ["v_nan", "v_inf", "k_nan", "q_nan", "S_nan"])
def test_values_that_are_not_finite_stay_where_they_belong(cuda_device, dt, D, H, what):
    """A value channel is poisoned from its token on, a key poisons its head from its token on, a query its token
    alone; earlier tokens, other channels and other heads keep their results."""
    T = 150
    x, S0, _ = draw(dt, 1, T, H, D, seed=20)
    bad = float("inf") if what == "v_inf" else float("nan")
    if what[0] == "S":
        S0[0, 1, 3, 5] = bad
    else:
        x[what[0]][0, 70, 1, 5] = bad
    y, S, _ = esa_delta_fwd(*ins(x), S_init=S0)
    ref = delta_reference(*(t[:, :, :3] for t in ins(x)), D ** -0.5, S0[:, :3])
    got = {"y": y[:, :, :3].cpu(), "S": S[:, :3].cpu()}
    for n in ("y", "S"):
        fine = torch.isfinite(ref[n])
        assert torch.equal(torch.isfinite(got[n]), fine), n
        extra = 3 * 2.0 ** -11 if n == "y" and dt != "f32" else 0.0
        assert_within(n, torch.where(fine, got[n], torch.zeros_like(got[n])), torch.where(fine, ref[n], 0.0),
                      PER_TOKEN * T + extra, PER_TOKEN * T ** 0.5 + extra)


@pytest.mark.parametrize("D,H", [(128, 18), (128, 19), (128, 37), (128, 38), (128, 75), (64, 37), (64, 38), (32, 150)])
def test_every_spread_of_heads(cuda_device, D, H):
    """The head counts at which the work is spread differently over the device; two heads of each are checked."""
    T = 100
    x, S0, dS = draw("bf16", 1, T, H, D, seed=H)
    out = run(x, S0, dS, D ** -0.5)
    pick = [0, H - 1]
    cut = {n: (t[:, pick] if n in ("S", "dS0") else t[:, :, pick]) for n, t in out.items()}
    xs = {n: t[:, :, pick] for n, t in x.items()}
    check(xs, cut, delta_reference(*ins(xs), D ** -0.5, S0[:, pick], xs["dy"], dS[:, pick]), T, D, half_p=3 * 2.0 ** -11)
