"""The gated delta rule in chunks at the ends of float32's range: factors whose products leave it, values far apart.

The bounds are test_gpu_delta's: half a step of the output's type, 20 float32 roundings a token, and for 16-bit
outputs three float16 roundings of intermediates.
"""
import pytest
import torch

from gated_linear_recurrence_b200 import esa_delta_bwd, esa_delta_fwd, esa_delta_step
from tests._delta_reference import PER_TOKEN, assert_within, delta_reference
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
@pytest.mark.parametrize("size", [1e-30, 1e-36])
def test_tiny_values(cuda_device, size, which, D, H):
    """Values down to 2^6 of the smallest normal number."""
    x, _, _ = draw("bf16", 1, T, H, D, seed=4, state=False)
    x[which] = (x[which].float() * size).to(x[which].dtype)
    xs, got, ref = two_heads(x, None, None, run(x, None, None, D ** -0.5))
    if size == 1e-30:
        check(xs, got, ref, T, D, half_p=HALF_P)
        return
    # At 1e-36 the factor of a prediction, about the state over 2^20, is a subnormal number of 12 bits or more; and
    # subnormal bfloat16 results are whole multiples of 2^-133: at most 2^-8 of a value of 2^-126, values being 2^-119.
    for n, t in got.items():
        extra = 2.0 ** -11 + 2.0 ** -9 + (HALF_P if n != "S" else 0.0)
        assert_within(n, t, ref[n], extra, extra)


@pytest.mark.parametrize("D,H", SPREADS)
@pytest.mark.parametrize("dt,which", [("bf16", "v"), ("bf16", "dy"), ("f16", "v"), ("f16", "dy"), ("bf16", "S")])
def test_value_channels_do_not_mix(cuda_device, dt, which, D, H):
    """One value channel 10^9 (float16: 10^7) times its neighbours: each channel is held to its own largest value."""
    x, S0, dS = draw(dt, 1, T, H, D, seed=5)
    factor = 1e7 if dt == "f16" else 1e9
    if which == "S":
        S0[..., 5] *= factor
        dS[..., 5] *= factor
    else:
        S0 = dS = None
        x[which] = (x[which].float() * 1e-3).to(x[which].dtype)
        x[which][..., 5] *= factor
    xs, got, ref = two_heads(x, S0, dS, run(x, S0, dS, D ** -0.5))
    a, n = PER_TOKEN * T, PER_TOKEN * T ** 0.5
    for name, k in (("y", 1), ("S", 1), ("dv", 2)) + ((("dS0", 2),) if which == "S" else ()):
        extra = HALF_P if got[name].dtype != torch.float32 else 0.0
        for c in (0, 4, 5, 6, 15, 16, D - 1):
            assert_within(f"{name}[..., {c}]", got[name][..., c], ref[name][..., c], k * a + extra, k * n + extra)


@pytest.mark.parametrize("D,H", SPREADS)
@pytest.mark.parametrize("value", [float("inf"), float("nan")])
def test_states_that_are_not_finite(cuda_device, value, D, H):
    """An entry of S_init reaches y and S_final of its value channel alone, one of dS_final dv of its channel alone; the
    gradients that sum over the channels are lost in its head alone."""
    x, S0, dS = draw("bf16", 1, T, H, D, seed=6)
    clean = run(x, S0, dS, D ** -0.5)
    own = torch.zeros(1, 1, H, D, dtype=torch.bool, device="cuda")
    own[0, 0, 1, 5] = True
    S1, dS1 = S0.clone(), dS.clone()
    S1[0, 1, 3, 5] = value
    dS1[0, 1, 3, 5] = value
    bad = run(x, S1, dS, D ** -0.5)
    y_own, S_own = own.expand_as(clean["y"]), own.transpose(1, 2).expand_as(clean["S"])
    assert torch.equal(bad["y"][~y_own], clean["y"][~y_own]) and not torch.isfinite(bad["y"][y_own]).any()
    assert torch.equal(bad["S"][~S_own], clean["S"][~S_own]) and not torch.isfinite(bad["S"][S_own]).any()
    for n in ("dq", "dk", "da"):
        assert not torch.isfinite(bad[n][0, :64, 1]).any(), n
        assert torch.equal(bad[n][:, :, 0], clean[n][:, :, 0]), n
    bad = run(x, S0, dS1, D ** -0.5)
    assert torch.equal(bad["dv"][~y_own], clean["dv"][~y_own]) and not torch.isfinite(bad["dv"][y_own]).any()
    assert torch.equal(bad["dS0"][~S_own], clean["dS0"][~S_own]) and not torch.isfinite(bad["dS0"][S_own]).any()
    for n in ("dk", "da", "db"):
        assert not torch.isfinite(bad[n][0, :192, 1]).any(), n
        assert torch.equal(bad[n][:, :, 0], clean[n][:, :, 0]), n


@pytest.mark.parametrize("dt,D,H", [("bf16", *s) for s in SPREADS] + [("f16", 64, 2), ("f32", 32, 2), ("f32", 64, 80)])
@pytest.mark.parametrize("value", [float("inf"), float("nan")])
@pytest.mark.parametrize("what", ["q", "k"])
def test_gradients_of_keys_and_queries_that_are_not_finite(cuda_device, what, value, dt, D, H):
    """All earlier tokens of the head have a share of such a key's or query's gradient; other heads have none."""
    x, S0, dS = draw(dt, 1, T, H, D, seed=9)
    clean = run(x, S0, dS, D ** -0.5)
    x[what][0, 150, 1, 3] = value
    bad = run(x, S0, dS, D ** -0.5)
    for n in ("dk", "dv", "da", "db"):
        assert not torch.isfinite(bad[n][0, :150, 1]).any(), n
    assert not torch.isfinite(bad["dS0"][0, 1]).any()
    other = [h for h in range(H) if h != 1]
    for n in ("y", "dq", "dk", "dv", "da", "db"):
        assert torch.equal(bad[n][:, :, other], clean[n][:, :, other]), n
    assert torch.equal(bad["dq"][0, :128, 1], clean["dq"][0, :128, 1])   # of earlier chunks: S dy of the past alone


@pytest.mark.parametrize("dt,T,D,H", [("bf16", T, D, H) for T in (20, 200) for D, H in SPREADS]
                         + [("f16", 200, 64, 2), ("bf16", 5, 64, 2), ("f32", 5, 64, 2), ("f32", 150, 32, 80), ("f32", 333, 32, 2),
                            ("f32", 333, 128, 2)])
@pytest.mark.parametrize("what", ["a", "b"])
@pytest.mark.parametrize("at", [2, 3, -1])
def test_gates_that_are_nan(cuda_device, at, what, dt, T, D, H):
    """A NaN logit makes its head NaN from its token on (and is not a gate of e^-80), in y, S and the gradients."""
    x, S0, dS = draw(dt, 1, T, H, D, seed=10)
    clean = run(x, S0, dS, D ** -0.5)
    at = at % T
    x[what][0, at, 1] = float("nan")
    bad = run(x, S0, dS, D ** -0.5)
    y, S, _ = esa_delta_fwd(*ins(x), S_init=S0, keep=False)
    for out in (bad["y"], y):
        assert not torch.isfinite(out[0, at:, 1]).any() and torch.isfinite(out[0, :at, 1]).all()
    assert torch.equal(bad["y"][0, :at, 1], clean["y"][0, :at, 1])
    assert not torch.isfinite(bad["S"][0, 1]).any() and not torch.isfinite(S[0, 1]).any()
    for n in ("dk", "dv", "da", "db"):
        assert not torch.isfinite(bad[n][0, :at, 1]).any(), n
    assert not torch.isfinite(bad["dS0"][0, 1]).any()
    other = [h for h in range(H) if h != 1]
    for n in ("y", "dq", "dk", "dv", "da", "db"):
        assert torch.equal(bad[n][:, :, other], clean[n][:, :, other]), n


@pytest.mark.parametrize("what", ["a", "b"])
@pytest.mark.parametrize("D", [32, 64, 128])
def test_one_token_with_a_gate_that_is_nan(cuda_device, D, what):
    x, S0, _ = draw("bf16", 2, 1, 3, D, seed=11)
    tok = {n: t[:, 0].contiguous() for n, t in x.items()}
    want_S = S0.clone()
    want = esa_delta_step(*ins(tok), want_S)
    tok[what][1, 2] = float("nan")
    S = S0.clone()
    y = esa_delta_step(*ins(tok), S)
    assert not torch.isfinite(y[1, 2]).any() and not torch.isfinite(S[1, 2]).any()
    y[1, 2], S[1, 2] = want[1, 2], want_S[1, 2]
    assert torch.equal(y, want) and torch.equal(S, want_S)


@pytest.mark.parametrize("D,H", SPREADS)
@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_value_channels_of_zeros(cuda_device, dt, D, H):
    """Channels that are zero throughout beside small ones: zeros times any scale."""
    x, _, _ = draw(dt, 1, T, H, D, seed=13, state=False)
    x["v"] = (x["v"].float() * 1e-4).to(x["v"].dtype)
    x["v"][..., 3] = 0
    x["v"][..., 16:32] = 0
    x["dy"] = (x["dy"].float() * 1e-3).to(x["dy"].dtype)
    x["dy"][..., 5] = 0
    xs, got, ref = two_heads(x, None, None, run(x, None, None, 1.0))
    for n in ("y", "S"):
        assert not got[n][..., [3, *range(16, 32)]].any()
    assert not got["dv"][..., 5].any()
    ref = delta_reference(*ins(xs), 1.0, None, xs["dy"], None)
    # da is some 1e-7: in float16 a whole multiple of 2^-24, off by 2^-25, which assert_within counts
    assert_within("da", got["da"], ref["da"], HALF_P, HALF_P)
    check(xs, got | {"da": ref["da"].float()}, ref, T, D, half_p=HALF_P)


FAR = {   # factors of the inputs; closed: no token writes; steep: gates of about e^-10
    "dy_far_below_its_share_of_dk": (dict(dy=2e-24, k=7e-17, S=0), False, False),
    "closed_and_large_dy": (dict(q=2e-8, dy=8e5, scale=4e4, k=4e-5, S=0), True, False),
    "steep_and_tiny_scale": (dict(S=6e-19, scale=3e-18, k=5e-18), False, True),
    "tiny_dy_and_scale_and_large_v": (dict(q=1e-4, v=1e17, dy=7e-26, scale=4e-23, S=0), False, False),
    "closed_and_large_states": (dict(q=3e-10, v=7e-11, S=9e15, dS=1e22), True, False),
    "tiny_keys_and_scale": (dict(scale=2e-12, k=1e-29), False, False),
    "tiny_scale": (dict(scale=1e-25), False, False),
    "tiny_keys_queries_and_dS": (dict(q=9e-30, v=6, k=2e-23, dS=4e-29), False, False),
}


@pytest.mark.parametrize("D,H", SPREADS)
@pytest.mark.parametrize("n", [8, 64, 130])
@pytest.mark.parametrize("which", FAR)
def test_factors_far_apart(cuda_device, which, n, D, H):
    """Inputs of sizes so different that products of two of their scales are outside float32: no infinity, and every
    gradient within the bounds of its largest value."""
    fac, closed, steep = FAR[which]
    x, S0, dS = draw("bf16", 1, n, H, D, seed=n, state=fac.get("S") != 0)
    for m in ("q", "k", "v", "dy"):
        x[m] = (x[m].float() * fac.get(m, 1)).to(x[m].dtype)
    if S0 is not None:
        S0, dS = S0 * fac.get("S", 1), dS * fac.get("dS", 1)
    if closed:
        x["b"].fill_(float("-inf"))
    if steep:
        x["a"] = x["a"] - 13
    scale = D ** -0.5 * fac.get("scale", 1)
    out = run(x, S0, dS, scale)
    xs, got, _ = two_heads(x, S0, dS, out)
    ref = delta_reference(*ins(xs), scale, None if S0 is None else S0[:, :2], xs["dy"], None if dS is None else dS[:, :2])
    for name, t in got.items():
        r = ref[name]
        # da = (1 - alpha) f with f of about <dS, S>: 1e22 x 0.1 x 9e15 x 0.3 x 128 = 3.5e38, past float32's 3.4e38
        if name == "da" and float((r * (1 + torch.exp(xs["a"].cpu().double()))).abs().max()) > 8e37:
            continue
        assert torch.isfinite(t).all(), name
        # Steep gates leave db to the last token alone: db = (1 - beta) sum_c du_c u_c is off by 2^-11 sum_c |du_c u_c|,
        # which is any multiple of one token's |db| (of a tensor's largest, a small one).
        if steep and name == "db":
            continue
        if float(r.abs().max()) > 1e-33:   # else of some few digits itself
            extra = HALF_P if t.dtype != torch.float32 else 2 * PER_TOKEN * n
            assert_within(name, t, r, extra, extra)


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("D,lengths", [(32, (15, 16, 39, 40)), (64, (11, 12, 39, 40)), (128, (7, 8, 23, 24))])
def test_lengths_around_the_chunks_use(cuda_device, D, lengths, dt):
    for n in lengths:
        x, S0, dS = draw(dt, 2, n, 3, D, seed=n)
        ref = delta_reference(*ins(x), D ** -0.5, S0, x["dy"], dS)
        check(x, run(x, S0, dS, None), ref, n, D, half_p=HALF_P)
        y, S, _ = esa_delta_fwd(*ins(x), S_init=S0, keep=False)
        check(x, {"y": y, "S": S}, ref, n, D, gradients=False, half_p=HALF_P)


@pytest.mark.parametrize("dt,D,H", [("bf16", *s) for s in SPREADS] + [("f32", 64, 2), ("f32", 32, 80)])
@pytest.mark.parametrize("scale", [0.0, -0.3, 1e-40])
def test_scales_of_zero_and_below(cuda_device, scale, dt, D, H):
    x, S0, dS = draw(dt, 1, T, H, D, seed=14)
    out = run(x, S0, dS, scale)
    xs, got, _ = two_heads(x, S0, dS, out)
    if scale == 1e-40:   # below float32's normal range: zero
        scale = 0.0
    ref = delta_reference(*ins(xs), scale, S0[:, :2], xs["dy"], dS[:, :2])
    if scale == 0.0:
        assert not got["y"].any() and not got["dq"].any()
    check(xs, got, ref, T, D, half_p=HALF_P)


@pytest.mark.parametrize("dt,D,H,n", [("bf16", 128, 2, 150), ("bf16", 64, 80, 70), ("bf16", 32, 2, 9), ("f32", 64, 2, 40),
                                      ("f32", 64, 2, 300)])
def test_state_gradient_over_the_final_one(cuda_device, dt, D, H, n):
    x, S0, dS = draw(dt, 1, n, H, D, seed=15)
    _, _, ws = esa_delta_fwd(*ins(x), S_init=S0)
    want = esa_delta_bwd(*ins(x), x["dy"], ws, S_init=S0, dS_final=dS)
    got = esa_delta_bwd(*ins(x), x["dy"], ws, S_init=S0, dS_final=dS, dS_init=dS)   # the workspace is read again
    assert got[5] is dS
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("D,H", SPREADS)
@pytest.mark.parametrize("n", [64, 300])
def test_float16_results_near_their_rounding(cuda_device, n, D, H):
    """Of each product's operands one is rounded to float16, S or dS, so a gradient's error is at most sqrt(2) times that
    of its own rounding in the 2-norm.  (Not da's: its sum's parts, <dS, S> and those of earlier and later tokens, are each
    off by so much of their own size and may cancel; it is held in test_delta_gate_gradient.)"""
    x, S0, dS = draw("f16", 1, n, H, D, seed=16, a_mean=4.0)
    xs, got, ref = two_heads(x, S0, dS, run(x, S0, dS, D ** -0.5))
    for name, times in (("y", 1.1), ("dv", 1.1), ("dq", 1.5), ("dk", 1.5), ("db", 1.5)):
        r = ref[name]
        own = float((r.half().double() - r).norm())
        off = float((got[name].cpu().double() - r).norm())
        assert off <= times * own, f"{name}: {off / float(r.norm()):.2e}, rounding {own / float(r.norm()):.2e}"


@pytest.mark.parametrize("dt,D,H", [("bf16", *s) for s in SPREADS] + [("f16", 128, 2), ("f32", 64, 2), ("f32", 32, 80)])
@pytest.mark.parametrize("what", ["k", "v", "a", "b", "S"])
def test_later_gradients_of_entries_that_are_not_finite(cuda_device, what, dt, D, H):
    """What makes the state NaN makes all later gradients that read it NaN; other heads keep theirs."""
    x, S0, dS = draw(dt, 1, T, H, D, seed=17)
    clean = run(x, S0, dS, D ** -0.5)
    if what == "S":
        S0[0, 1, 3, 5] = float("nan")
    elif what in "ab":
        x[what][0, 70, 1] = float("nan")
    else:
        x[what][0, 70, 1, 5] = float("nan")
    bad = run(x, S0, dS, D ** -0.5)
    for n in ("dq", "dk", "da", "db"):
        assert not torch.isfinite(bad[n][0, 70:, 1]).any(), n
    other = [h for h in range(H) if h != 1]
    for n in ("y", "dq", "dk", "dv", "da", "db"):
        assert torch.equal(bad[n][:, :, other], clean[n][:, :, other]), n
