"""What the gated delta rule and the layer norm are measured on.

Two operators of a pre-norm recurrent block:

* the gated delta rule, the matrix-state recurrence of a head (whole sequences,
  training, and one token at a time), with S [D, D] (rows: key channels,
  columns: value channels), alpha_t = sigmoid(a_t), beta_t = sigmoid(b_t):

      u_t = beta_t (v_t - alpha_t S_{t-1}^T k_t)
      S_t = alpha_t S_{t-1} + k_t u_t^T
      y_t = scale S_t^T q_t,          scale = D^(-1/2)

* layer norm over the last axis with the residual addition before it,
  h = x + residual (in the tensors' type), y = (h - mean) rstd w + c, and its
  backward with the gradients of the weight and the bias.

``own`` chooses between plain torch operations and the library's calls.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
OUT_OF_RANGE = -80.0   # gate logits are clamped here, as in every gate of the library
CHUNK = 64             # tokens per block of the plain form


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def _delta(name, op, dtype, B, T, H, D, state=True):
    return {"name": name, "op": op, "dtype": dtype, "B": B, "T": T, "H": H, "D": D, "state": state}


def _norm(name, op, dtype, wdtype, rows, N, residual=True):
    return {"name": name, "op": op, "dtype": dtype, "wdtype": wdtype, "rows": rows, "N": N, "residual": residual}


def listed():
    return [
        # one interactive stream generating a token: latency only
        _delta("step_b1_h8_d64", "step", "bf16", 1, 1, 8, 64),
        # a serving batch generating a token: the state's traffic
        _delta("step_b64_h8_d128", "step", "f16", 64, 1, 8, 128),
        # a prompt of odd length that continues a state
        _delta("prefill_t1777_d128", "fwd", "bf16", 1, 1777, 8, 128),
        # two long documents: few heads, a long time axis
        _delta("prefill_t32768_d128", "fwd", "f16", 2, 32768, 8, 128, False),
        # training at the batch and heads of the bf16 workload of the scan benchmark, a slice of its length
        _delta("train_b64_t1024_h8_d64", "train", "bf16", 64, 1024, 8, 64, False),
        # training with wide heads: the largest case
        _delta("train_b8_t2048_h16_d128", "train", "bf16", 8, 2048, 16, 128),
        # float32 training at the small workload's heads, ragged length
        _delta("train_f32_t333_d32", "train", "f32", 2, 333, 4, 32),
        # the norm of one generated token per stream
        _norm("norm_64x512", "norm_fwd", "f16", "f16", 64, 512),
        # the norm of a prompt batch at 128 channels
        _norm("norm_262144x128", "norm_fwd", "f16", "f16", 262144, 128),
        # a training step's norm at 512 channels, float32 master weights
        _norm("norm_train_65536x512", "norm_train", "bf16", "f32", 65536, 512),
        # wide float32 rows of odd width
        _norm("norm_train_4099x5001", "norm_train", "f32", "f32", 4099, 5001, False),
    ]


def _log_uniform(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("step", "fwd", "train", "norm_fwd", "norm_train"))
    if op in ("norm_fwd", "norm_train"):
        dtype = rng.choice(("f32", "f16", "bf16"))
        N = _log_uniform(rng, 8, 8192)
        rows = _log_uniform(rng, 1, max(1, min(262144, 33_000_000 // N)))
        return {"op": op, "dtype": dtype, "wdtype": rng.choice((dtype, "f32")), "rows": rows, "N": N,
                "residual": rng.random() < 0.5}
    D = rng.choice((32, 64, 128))
    dtype = rng.choice(("f16", "bf16", "bf16", "f32"))
    H = _log_uniform(rng, 1, 16)
    if op == "step":
        B, T = _log_uniform(rng, 1, 64), 1
    else:
        T = _log_uniform(rng, 1, 8192)
        most = 200_000 // (T * H) if dtype != "f32" else 20_000 // (T * H)
        B = _log_uniform(rng, 1, max(1, min(64, most)))
    return {"op": op, "dtype": dtype, "B": B, "T": T, "H": H, "D": D, "state": rng.random() < 0.5}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def randn(*shape):
        return torch.randn(*shape, device="cuda", generator=g)

    s = {"op": case["op"], "dtype": dt}
    if case["op"].startswith("norm"):
        rows, N, wdt = case["rows"], case["N"], DTYPES[case["wdtype"]]
        # a residual stream has rows of different size and a mean of its own
        s["x"] = (randn(rows, N) * (0.5 + randn(rows, 1).abs()) + 0.3 * randn(rows, 1)).to(dt)
        s["residual"] = randn(rows, N).to(dt) if case["residual"] else None
        s["weight"] = (1.0 + 0.2 * randn(N)).to(wdt)
        s["bias"] = (0.1 * randn(N)).to(wdt)
        s["eps"] = 1e-5
        if case["op"] == "norm_train":
            s["dy"] = randn(rows, N).to(dt)
            # the gradient that reaches h through the residual stream itself
            s["dh"] = randn(rows, N).to(dt) if case["residual"] else None
        return s
    B, T, H, D = case["B"], case["T"], case["H"], case["D"]
    lead = (B, H) if case["op"] == "step" else (B, T, H)

    def unit(*shape):
        x = randn(*shape)
        return (x / x.norm(dim=-1, keepdim=True)).to(dt)

    s["q"], s["k"], s["v"] = unit(*lead, D), unit(*lead, D), randn(*lead, D).to(dt)
    s["a"], s["b"] = (4.0 + randn(*lead)).to(dt), randn(*lead).to(dt)   # long memory, as the long-context workload
    s["scale"] = D ** -0.5
    if case["op"] == "step":
        s["S"] = 0.3 * randn(B, H, D, D)
        return s
    s["S_init"] = 0.3 * randn(B, H, D, D) if case["state"] else None
    if case["op"] == "train":
        s["dy"] = randn(B, T, H, D).to(dt)
        s["dS_final"] = 0.1 * randn(B, H, D, D) if case["state"] else None
    return s


# ---------------------------------------------------------------------------
# Plain forms: elementary torch operations in float32 (float64 where a sum of
# logarithms is exponentiated and for the inverse of a chunk's matrix)
# ---------------------------------------------------------------------------
def _plain_delta(q, k, v, a, b, scale, S):
    """q, k, v [B, T, H, D], a, b [B, T, H] float32, S [B, H, D, D] float32 -> y, S_T.  Chunks of CHUNK tokens:
    with G the running sum of log alpha in a chunk and M_ij = beta_i exp(G_i - G_j) k_i.k_j (j < i),
    (1 + M) U = beta (V - exp(G) K S),  Y = scale (exp(G) Q S + (exp(G_i - G_j) q_i.k_j)_{j<=i} U),
    S' = exp(G_last) S + (exp(G_last - G) K)^T U."""
    B, T, H, D = q.shape
    n = -(-T // CHUNK)
    pad = n * CHUNK - T

    def chunks(x):   # [n, B, H, CHUNK, ...]; the padded tokens write nothing and forget nothing
        x = torch.cat([x, x.new_zeros(B, pad, *x.shape[2:])], 1) if pad else x
        x = x.reshape(B, n, CHUNK, *x.shape[2:])
        return x.permute(1, 0, 3, 2, *range(4, x.dim()))

    g = -torch.log1p(torch.exp(-a.clamp(min=OUT_OF_RANGE).double()))
    beta = 1.0 / (1.0 + torch.exp(-b.clamp(min=OUT_OF_RANGE)))
    q, k, v, g, beta = chunks(q), chunks(k), chunks(v), chunks(g), chunks(beta)
    G = g.cumsum(-1)
    low = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=q.device).tril()
    decay = torch.exp((G[..., :, None] - G[..., None, :]).masked_fill(~low, -math.inf)).float()
    M = (beta[..., None] * decay * (k @ k.transpose(-1, -2))).tril(-1)
    inv = torch.eye(CHUNK, dtype=torch.float64, device=q.device) - M.double()
    P = M.double()
    for _ in range(int(math.log2(CHUNK)) - 1):   # (1 + M)^-1 = (1 - M)(1 + M^2)(1 + M^4)...: M^CHUNK = 0
        P = P @ P
        inv = inv + inv @ P
    inv = inv.float()
    A = decay * (q @ k.transpose(-1, -2))
    into, last, out = torch.exp(G).float(), torch.exp(G[..., -1]).float(), torch.exp(G[..., -1:] - G).float()
    y = []
    for i in range(n):   # the recurrence itself, CHUNK tokens at a time
        U = inv[i] @ (beta[i][..., None] * (v[i] - into[i][..., None] * (k[i] @ S)))
        y.append(scale * (into[i][..., None] * (q[i] @ S) + A[i] @ U))
        S = last[i][..., None, None] * S + (out[i][..., None] * k[i]).transpose(-1, -2) @ U
    y = torch.stack(y).permute(1, 0, 3, 2, 4).reshape(B, n * CHUNK, H, D)[:, :T]
    return y, S


def _plain_step(s):
    q, k, v, a, b, S = (s[n].float() for n in ("q", "k", "v", "a", "b", "S"))
    alpha = 1.0 / (1.0 + torch.exp(-a.clamp(min=OUT_OF_RANGE)))[..., None]
    beta = 1.0 / (1.0 + torch.exp(-b.clamp(min=OUT_OF_RANGE)))[..., None]
    S = alpha[..., None] * S
    u = beta * (v - (S * k[..., None]).sum(-2))
    S = S + k[..., None] * u[..., None, :]
    y = s["scale"] * (S * q[..., None]).sum(-2)
    s["S"].copy_(S)
    return {"y": y.to(s["dtype"]), "S": s["S"]}


def _plain_norm(s):
    x, dt, wdt = s["x"], s["dtype"], s["weight"].dtype
    h = x if s["residual"] is None else (x.float() + s["residual"].float()).to(dt)
    w, c = s["weight"].float(), s["bias"].float()
    hf = h.float()
    mean = hf.mean(-1, keepdim=True)
    d = hf - mean
    rstd = torch.rsqrt((d * d).mean(-1, keepdim=True) + s["eps"])
    n = d * rstd
    out = {"y": (n * w + c).to(dt)}
    if s["residual"] is not None:
        out["h"] = h
    if s["op"] == "norm_train":
        dy = s["dy"].float()
        dn = dy * w
        dx = rstd * (dn - dn.mean(-1, keepdim=True) - n * (dn * n).mean(-1, keepdim=True))
        if s["dh"] is not None:
            dx = dx + s["dh"].float()
        out.update(dx=dx.to(dt), dweight=(dy * n).sum(0).to(wdt), dbias=dy.sum(0).to(wdt))
    return out


def _plain(s):
    if s["op"] == "step":
        return _plain_step(s)
    if s["op"].startswith("norm"):
        return _plain_norm(s)
    dt = s["dtype"]
    names = ("q", "k", "v", "a", "b")
    x = [s[n].float() for n in names]
    B, T, H, D = x[0].shape
    S0 = x[0].new_zeros(B, H, D, D) if s["S_init"] is None else s["S_init"]
    if s["op"] == "fwd":
        y, S = _plain_delta(*x, s["scale"], S0)
        return {"y": y.to(dt), "S": S}
    leaves = [t.detach().requires_grad_() for t in (*x, S0)]
    with torch.enable_grad():
        y, S = _plain_delta(*leaves[:5], s["scale"], leaves[5])
        outs, grads = [y], [s["dy"].float()]
        if s["dS_final"] is not None:
            outs.append(S)
            grads.append(s["dS_final"])
        dx = torch.autograd.grad(outs, leaves, grads)
    out = {"y": y.detach().to(dt), "S": S.detach()}
    out.update({"d" + n: g.to(dt) for n, g in zip(names, dx)})
    if s["S_init"] is not None:
        out["dS_init"] = dx[5]
    return out


# ---------------------------------------------------------------------------
# The library's calls
# ---------------------------------------------------------------------------
def _own(s):
    import gated_linear_recurrence_b200 as glr

    if s["op"] == "step":
        y = glr.esa_delta_step(s["q"], s["k"], s["v"], s["a"], s["b"], s["S"], scale=s["scale"])
        return {"y": y, "S": s["S"]}
    if s["op"].startswith("norm"):
        train = s["op"] == "norm_train"
        y, h, stats = glr.esa_norm_fwd(s["x"], s["weight"], s["bias"], eps=s["eps"], residual=s["residual"],
                                       want_stats=train)
        out = {"y": y}
        if s["residual"] is not None:
            out["h"] = h
        if train:
            dx, dw, db = glr.esa_norm_bwd(s["dy"], h, s["weight"], stats, dh=s["dh"], want_dbias=True)
            out.update(dx=dx, dweight=dw, dbias=db)
        return out
    x = [s[n] for n in ("q", "k", "v", "a", "b")]
    if s["op"] == "fwd":
        y, S, _ = glr.esa_delta_fwd(*x, scale=s["scale"], S_init=s["S_init"], keep=False)
        return {"y": y, "S": S}
    y, S, ws = glr.esa_delta_fwd(*x, scale=s["scale"], S_init=s["S_init"])
    *dx, dS = glr.esa_delta_bwd(*x, s["dy"], ws, scale=s["scale"], S_init=s["S_init"], dS_final=s["dS_final"],
                                want_dS_init=s["S_init"] is not None)
    out = {"y": y, "S": S}
    out.update({"d" + n: g for n, g in zip(("q", "k", "v", "a", "b"), dx)})
    if s["S_init"] is not None:
        out["dS_init"] = dS
    return out


def run(state):
    if own:
        return _own(state)
    with torch.no_grad():
        return _plain(state)


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    e = 4 if case["dtype"] == "f32" else 2
    if case["op"].startswith("norm"):
        n, ew = case["rows"] * case["N"], 4 if case["wdtype"] == "f32" else 2
        res = 1 if case["residual"] else 0
        tensors, flops = 2 + 2 * res, 8 + res        # x, y (residual, h)
        if case["op"] == "norm_train":
            tensors, flops = tensors + 2 + res, flops + 14   # dy, dx (dh); h is still at hand
        return {"bytes": n * e * tensors + case["N"] * ew * (2 if case["op"] == "norm_fwd" else 4),
                "flops": n * flops}
    n = case["B"] * case["T"] * case["H"]
    D = case["D"]
    state = case["B"] * case["H"] * D * D * 4
    if case["op"] == "step":
        return {"bytes": n * (4 * D + 2) * e + 2 * state, "flops": n * 7 * D * D}
    had = 1 if case["state"] else 0
    if case["op"] == "fwd":
        return {"bytes": n * (4 * D + 2) * e + (1 + had) * state, "flops": n * 7 * D * D}
    return {"bytes": n * (8 * D + 4) * e + (1 + 3 * had) * state, "flops": n * 23 * D * D}


# ---------------------------------------------------------------------------
# The definitions, token by token, in float64
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].startswith("norm"):
        return _exact_norm(s)
    q, k, v, a, b = (s[n].double() for n in ("q", "k", "v", "a", "b"))
    scale = s["scale"]
    alpha, beta = torch.sigmoid(a.clamp(min=-80.0)), torch.sigmoid(b.clamp(min=-80.0))
    if case["op"] == "step":
        S = alpha[..., None, None] * s["S"].double()
        u = beta[..., None] * (v - torch.einsum("bhij,bhi->bhj", S, k))
        S = S + torch.einsum("bhi,bhj->bhij", k, u)
        return {"y": scale * torch.einsum("bhij,bhi->bhj", S, q), "S": S}
    B, T, H, D = q.shape
    train = case["op"] == "train"
    q, k, v = (x.permute(1, 0, 2, 3).reshape(T, B * H, 1, D) for x in (q, k, v))
    alpha, beta = (x.permute(1, 0, 2).reshape(T, B * H, 1, 1) for x in (alpha, beta))
    S0 = (q.new_zeros(B * H, D, D) if s["S_init"] is None else s["S_init"].double().reshape(B * H, D, D))

    def back(x):   # [T, BH, 1, d] -> [B, T, H, d]
        return x.reshape(T, B, H, x.shape[-1]).permute(1, 0, 2, 3)

    S = S0.clone()
    y, u = torch.empty_like(v), torch.empty_like(v)
    for t in range(T):
        S *= alpha[t]
        u[t] = beta[t] * (v[t] - k[t] @ S)
        S.baddbmm_(k[t].transpose(1, 2), u[t])
        y[t] = q[t] @ S
    y *= scale
    out = {"y": back(y), "S": S.reshape(B, H, D, D).clone()}
    if not train:
        return out
    dy = s["dy"].double().permute(1, 0, 2, 3).reshape(T, B * H, 1, D)
    dS = torch.zeros_like(S) if s["dS_final"] is None else s["dS_final"].double().reshape(B * H, D, D).clone()
    end = (dS * S).sum((1, 2)).reshape(B * H, 1, 1)
    du, dk, dq = torch.empty_like(v), torch.empty_like(v), torch.empty_like(v)
    for t in range(T - 1, -1, -1):
        dS.baddbmm_(q[t].transpose(1, 2), dy[t], alpha=scale)
        du[t] = k[t] @ dS
        dk[t] = u[t] @ dS.transpose(1, 2)
        dS.baddbmm_(k[t].transpose(1, 2), du[t] * -beta[t])
        dS *= alpha[t]
    S = S0.clone()
    for t in range(T):
        S *= alpha[t]
        dk[t] -= beta[t] * (du[t] @ S.transpose(1, 2))
        S.baddbmm_(k[t].transpose(1, 2), u[t])
        dq[t] = dy[t] @ S.transpose(1, 2)
    dq *= scale
    # <dS_t, S_t> = alpha_t d/dalpha_t + beta_t v_t.du_t, and <dS_t, S_t> = y_t.dy_t + alpha_{t+1} d/dalpha_{t+1}
    gain = (y * dy).sum(-1, keepdim=True) - beta * (v * du).sum(-1, keepdim=True)
    dlog = gain.flip(0).cumsum(0).flip(0) + end
    da = dlog * (1.0 - alpha)
    db = (du * u).sum(-1, keepdim=True) * (1.0 - beta)
    out.update(dq=back(dq), dk=back(dk), dv=back(beta * du), da=back(da)[..., 0], db=back(db)[..., 0])
    if s["S_init"] is not None:
        out["dS_init"] = dS.reshape(B, H, D, D)
    return out


def _exact_norm(s):
    x = s["x"].double()
    h = x if s["residual"] is None else (x + s["residual"].double()).to(s["dtype"]).double()
    w = s["weight"].double()
    N = x.shape[-1]
    mean = h.sum(-1, keepdim=True) / N
    var = ((h - mean) ** 2).sum(-1, keepdim=True) / N
    n = (h - mean) / torch.sqrt(var + s["eps"])
    out = {"y": n * w + s["bias"].double()}
    if s["residual"] is not None:
        out["h"] = x + s["residual"].double()
    if s["op"] == "norm_train":
        dy = s["dy"].double()
        g = dy * w
        dx = (g - g.sum(-1, keepdim=True) / N - n * (g * n).sum(-1, keepdim=True) / N) / torch.sqrt(var + s["eps"])
        if s["dh"] is not None:
            dx = dx + s["dh"].double()
        out.update(dx=dx, dweight=(dy * n).sum(0), dbias=dy.sum(0))
    return out
