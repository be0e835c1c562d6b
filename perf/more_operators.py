"""The operators of a selective state space block -- the short causal
convolution, the selective scan and the layer norm with its residual stream --
as measurable cases.

``run`` computes a case either through this package's entry points (``own``
true) or in a plain form of elementary torch operations in 32 bits; ``exact``
computes the same outputs from the definitions in 64 bits.

Convolution, per sequence and channel, with the rows before a sequence from
its state (K - 1 rows, zero without one):

    u_t = bias + sum_j w[j] x_{t - (K - 1) + j},  out = u or silu(u)

Selective scan, per sequence, channel c and state n, D_t = softplus(delta_t + delta_bias):

    h_t[n] = exp(D_t A[n]) h_{t-1}[n] + D_t B_t[n] x_t
    out_t = (sum_n C_t[n] h_t[n] + skip x_t) silu(z_t)

B and C are shared by the channels of a group; A is negative.

Layer norm, per token, r' = x + r (r optional):

    out = (r' - mean) / sqrt(var + eps) w + b
"""
import math
import random

import torch

own = False

DEVICE = "cuda"
MOST_SEQS = 64
EPS = 1e-5


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def listed():
    def conv(name, **kw):
        base = dict(name=name, op="conv", dtype="bf16", tokens=1, seqs=1, width=2048, taps=4, act="silu", bias=True,
                    ragged=False, states=False, fused=False, lens=1)
        return dict(base, **kw)

    def scan(name, **kw):
        base = dict(name=name, op="select", dtype="bf16", tokens=1, seqs=1, width=2048, state=16, groups=1, gate=True,
                    skip=True, ragged=False, states=False, fused=False, lens=1)
        return dict(base, **kw)

    def norm(name, **kw):
        base = dict(name=name, op="layer_norm", dtype="bf16", tokens=1, width=2048, residual=True, bias=True)
        return dict(base, **kw)

    return [
        # one user's prompt in front of a reply: latency
        conv("conv_prompt", tokens=500, width=1024, states=True),
        # training step of a layer: 8 x 4096 tokens, the input a slice of the block's projection
        conv("conv_train", op="conv_train", tokens=32768, seqs=8, fused=True),
        # full precision, odd lengths, empty sequences, a width that is no multiple of 64, three taps
        conv("conv_train_ragged", op="conv_train", dtype="f32", tokens=3001, seqs=9, width=1000, taps=3, act="none",
             ragged=True, states=True, lens=5),
        # 256 streams answering at once
        conv("conv_step", op="conv_step", tokens=256, fused=True),
        # one user's prompt in front of a reply: latency
        scan("select_prompt", tokens=500, width=1024, states=True, fused=True),
        # long documents of uneven length, continued from stored states
        scan("select_varlen", tokens=24001, seqs=16, ragged=True, states=True, lens=3),
        # training step of a layer: 8 x 4096 tokens
        scan("select_train", op="select_train", tokens=32768, seqs=8, fused=True),
        # training on a small ragged batch in full precision, B and C of two groups, no gate
        scan("select_train_ragged", op="select_train", dtype="f32", tokens=1501, seqs=5, width=528, state=8, groups=2,
             gate=False, ragged=True, states=True, lens=7),
        # 256 streams answering at once
        scan("select_step", op="select_step", tokens=256, fused=True),
        # in front of a block while decoding a few streams
        norm("norm_step", tokens=4),
        # in front of a block: 4 x 4096 tokens, the residual stream summed and normed
        norm("norm_block", tokens=16384, width=2304),
        # its gradient in a training step
        norm("norm_grad", op="layer_norm_grad", tokens=16384),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["conv", "conv_train", "conv_step", "select", "select", "select_train", "select_train", "select_step",
                     "layer_norm", "layer_norm_grad"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    limit = 24_000_000 if dtype == "f32" else 48_000_000  # elements of one token tensor
    width = 8 * _log(rng, 8, 512)
    case = dict(op=op, dtype=dtype, width=width)
    if op in ("layer_norm", "layer_norm_grad"):
        case.update(tokens=_log(rng, 1, min(65536, limit // width)), residual=rng.random() < 0.6, bias=rng.random() < 0.7)
        return case
    if op == "conv_step" or op == "select_step":
        tokens = _log(rng, 1, 512)
    elif op.startswith("conv"):
        tokens = _log(rng, 1, min(65536, limit // width))
    else:
        state, groups = rng.choice([8, 16, 16, 32, 64]), rng.choice([1, 1, 2, 4])
        width = width // (8 * groups) * 8 * groups or 8 * groups
        most = (500_000_000 if dtype == "f32" else 1_000_000_000) // (width * state)
        tokens = _log(rng, 1, min(32768, most))
        case.update(width=width, state=state, groups=groups)
    if op == "select_step":
        state, groups = rng.choice([8, 16, 16, 32, 64]), rng.choice([1, 1, 2, 4])
        case.update(width=width // (8 * groups) * 8 * groups or 8 * groups, state=state, groups=groups)
    seqs = 1 if rng.random() < 0.4 else _log(rng, 2, MOST_SEQS)
    case.update(tokens=tokens, seqs=seqs, ragged=seqs > 1, states=rng.random() < 0.6, fused=rng.random() < 0.5,
                lens=rng.randrange(1 << 20))
    if op.startswith("conv"):
        case.update(taps=rng.choice([2, 3, 4, 4]), act=rng.choice(["none", "silu"]), bias=rng.random() < 0.6)
    else:
        case.update(gate=rng.random() < 0.6, skip=rng.random() < 0.7)
    return case


def _lengths(case):
    """The sequences' lengths: even, or cut at random places (some sequences empty)."""
    t, s = case["tokens"], case["seqs"]
    if not case["ragged"]:
        return [t * (i + 1) // s - t * i // s for i in range(s)]
    r = random.Random(case["lens"])
    cuts = sorted(r.randrange(t + 1) for _ in range(s - 1))
    if s > 3:
        cuts[1] = cuts[0]  # an empty sequence
    return [b - a for a, b in zip([0] + cuts, cuts + [t])]


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
class _Plan(dict):
    """What a program keeps of an operator's settings; the package's own form of it is made at its first call."""


def prepare(case, seed):
    g = torch.Generator(device=DEVICE).manual_seed(seed)
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    f32 = torch.float32
    T, W, op = case["tokens"], case["width"], case["op"]

    def normal(*shape, std=1.0, mean=0.0, dtype=dt):
        return (torch.randn(*shape, generator=g, device=DEVICE) * std + mean).to(dtype)

    st = {"case": case, "dt": dt}
    if op in ("layer_norm", "layer_norm_grad"):
        # a residual stream: a few units, some channels far from zero
        st["x"] = (normal(T, W, std=2.0, dtype=f32) + normal(W, std=1.5, dtype=f32)).to(dt)
        st["r"] = normal(T, W, std=0.7) if case["residual"] and op == "layer_norm" else None
        st["w"] = normal(W, std=0.1, mean=1.0, dtype=f32)
        st["b"] = normal(W, std=0.1, dtype=f32) if case["bias"] else None
        if op == "layer_norm_grad":
            st["d_out"] = normal(T, W, std=0.1)
            st["d_r"] = normal(T, W, std=0.1) if case["residual"] else None
        st["cfg"] = _Plan(width=W, eps=EPS, dtype=case["dtype"])
        return st

    lens = _lengths(case)
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    S = len(lens)
    step = op.endswith("step")
    if not step:
        st["cu"] = torch.tensor(cu, dtype=torch.int32, device=DEVICE)
    rows = T if step else S  # sequences
    states = step or case["states"]
    if op.startswith("conv"):
        K = case["taps"]
        # the projection of the block's normed input; fused: beside the gate
        st["x"] = normal(T, 2 * W)[:, :W] if case["fused"] else normal(T, W)
        st["w"] = normal(W, K, std=K ** -0.5, dtype=f32)
        st["bias"] = normal(W, std=0.1, dtype=f32) if case["bias"] else None
        st["state"] = normal(rows, K - 1, W) if states else None
        if op == "conv_train":
            st["d_out"] = normal(T, W)
            st["d_final"] = normal(S, K - 1, W) if states else None
        st["cfg"] = _Plan(width=W, taps=K, act=case["act"], dtype=case["dtype"])
        return st
    N, G = case["state"], case["groups"]
    u = normal(T, W, dtype=f32)
    st["x"] = (u / (1 + torch.exp(-u))).to(dt)  # behind the convolution's SiLU
    # steps from 0.001 to 0.1: the bias is the inverse softplus of them, the projection moves them by some factor
    dt0 = torch.exp(torch.rand(W, generator=g, device=DEVICE) * math.log(100.0) + math.log(0.001))
    st["delta_bias"] = dt0 + torch.log(-torch.expm1(-dt0))
    st["delta"] = normal(T, W, std=0.7)
    # decays around 1, 2, ..., N, as such models start and a little on
    n = torch.arange(1, N + 1, device=DEVICE, dtype=f32)
    st["A"] = -torch.exp(torch.log(n) + normal(W, N, std=0.1, dtype=f32))
    if case["fused"]:  # B, C and the gate are slices of projections' rows
        bc = normal(T, 2 * G * N + 64)
        st["B"] = bc[:, 64:64 + G * N].unflatten(1, (G, N))
        st["C"] = bc[:, 64 + G * N:].unflatten(1, (G, N))
        st["z"] = normal(T, 2 * W)[:, W:] if case["gate"] else None
    else:
        st["B"], st["C"] = normal(T, G, N), normal(T, G, N)
        st["z"] = normal(T, W) if case["gate"] else None
    st["skip"] = normal(W, std=0.1, mean=1.0, dtype=f32) if case["skip"] else None
    st["state"] = normal(rows, W, N, std=0.3, dtype=f32) if states else None
    if op == "select_train":
        st["d_out"] = normal(T, W)
        st["d_final"] = normal(S, W, N, std=0.3, dtype=f32) if states else None
    st["cfg"] = _Plan(width=W, state=N, groups=G, dtype=case["dtype"])
    return st


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------
def run(st):
    op = st["case"]["op"]
    if own:
        return _run_own(st, op)
    if op == "layer_norm":
        return _plain_norm(st)
    if op == "layer_norm_grad":
        return _plain_norm_grad(st)
    if op == "conv_step":
        return _plain_conv_step(st)
    if op == "select_step":
        return _plain_select_step(st)
    return _plain_conv(st) if op.startswith("conv") else _plain_select(st)


def _run_own(st, op):
    from sparse_state_linear_router_gb300 import binding
    cfg = st["cfg"].get("own")
    if cfg is None:
        make = (binding.make_layer_norm_config if op.startswith("layer") else
                binding.make_conv_config if op.startswith("conv") else binding.make_selective_config)
        cfg = make(**st["cfg"])
        st["cfg"]["own"] = cfg
    if op == "layer_norm":
        r = binding.layer_norm(cfg, st["x"], st["w"], st["b"], residual=st["r"])
        return {"out": r["out"], "residual": r["residual_out"]}
    if op == "layer_norm_grad":
        b = binding.layer_norm_backward(cfg, st["x"], st["w"], st["d_out"], d_residual_out=st["d_r"],
                                        want_d_bias=st["b"] is not None)
        return {"dx": b["dx"], "d_w": b["d_weight"], "d_b": b["d_bias"]}
    if op == "conv_step":
        r = binding.conv_step(cfg, st["state"], st["x"], st["w"], bias=st["bias"])
        return {"out": r["out"], "state": st["state"]}
    if op == "select_step":
        r = binding.selective_step(cfg, st["state"], st["x"], st["delta"], st["A"], st["B"], st["C"],
                                   delta_bias=st["delta_bias"], skip=st["skip"], gate=st["z"])
        return {"out": r["out"], "state": st["state"]}
    if op.startswith("conv"):
        r = binding.conv_forward(cfg, st["x"], st["w"], st["cu"], bias=st["bias"], initial_state=st["state"])
        out = {"out": r["out"], "final": r["final_state"]}
        if op == "conv_train":
            b = binding.conv_backward(cfg, st["x"], st["w"], st["cu"], st["d_out"], bias=st["bias"],
                                      initial_state=st["state"], d_final_state=st["d_final"],
                                      want_d_initial_state=st["state"] is not None)
            out.update(dx=b["dx"], d_w=b["d_weight"], d_bias=b["d_bias"], d_init=b["d_initial_state"])
        return out
    args = (st["x"], st["delta"], st["A"], st["B"], st["C"], st["cu"])
    kw = dict(delta_bias=st["delta_bias"], skip=st["skip"], gate=st["z"], initial_state=st["state"])
    r = binding.selective_forward(cfg, *args, want_checkpoints=op == "select_train", **kw)
    out = {"out": r["out"], "final": r["final_state"]}
    if op == "select_train":
        b = binding.selective_backward(cfg, *args, r["checkpoints"], st["d_out"], d_final_state=st["d_final"],
                                       want_d_initial_state=st["state"] is not None, **kw)
        out.update(dx=b["dx"], d_delta=b["d_delta"], d_A=b["d_A"], d_B=b["d_B"], d_C=b["d_C"],
                   d_delta_bias=b["d_delta_bias"], d_skip=b["d_skip"], d_z=b["d_gate"], d_init=b["d_initial_state"])
    return out


# ---------------------------------------------------------------------------
# Plain forms (32 bits)
# ---------------------------------------------------------------------------
def _silu(u):
    """silu(u) and its derivative."""
    s = 1 / (1 + torch.exp(-u))
    return u * s, s * (1 + u * (1 - s))


def _softplus(u):
    """log(1 + exp(u)) and its derivative."""
    e = torch.exp(-u.abs())
    return u.clamp(min=0) + torch.log1p(e), torch.where(u > 0, 1 / (1 + e), e / (1 + e))


def _plain_norm(st):
    dt = st["dt"]
    r = st["x"].float()
    if st["r"] is not None:
        r = r + st["r"].float()
    d = r - r.mean(1, keepdim=True)
    out = d * (1 / torch.sqrt((d * d).mean(1, keepdim=True) + EPS)) * st["w"]
    if st["b"] is not None:
        out = out + st["b"]
    return {"out": out.to(dt), "residual": r.to(dt) if st["r"] is not None else None}


def _plain_norm_grad(st):
    r, dy = st["x"].float(), st["d_out"].float()
    d = r - r.mean(1, keepdim=True)
    rstd = 1 / torch.sqrt((d * d).mean(1, keepdim=True) + EPS)
    hat = d * rstd
    p = dy * st["w"]
    dx = rstd * (p - p.mean(1, keepdim=True) - hat * (p * hat).mean(1, keepdim=True))
    if st["d_r"] is not None:
        dx = dx + st["d_r"].float()
    return {"dx": dx.to(st["dt"]), "d_w": (dy * hat).sum(0), "d_b": dy.sum(0) if st["b"] is not None else None}


def _plain_conv_step(st):
    case, x, state = st["case"], st["x"].float(), st["state"].float()
    rows = torch.cat([state, x.unsqueeze(1)], 1)  # [B, K, W]
    u = (rows * st["w"].t()).sum(1)
    if st["bias"] is not None:
        u = u + st["bias"]
    if case["act"] == "silu":
        u = _silu(u)[0]
    st["state"].copy_(rows[:, 1:])
    return {"out": u.to(st["dt"]), "state": st["state"]}


def _token_rows(cu, T):
    """The sequence of each token, and its place in it."""
    t = torch.arange(T, device=cu.device)
    seq = (t.unsqueeze(1) >= cu[1:-1].unsqueeze(0)).sum(1) if len(cu) > 2 else torch.zeros_like(t)
    return seq, t - cu[seq]


def _plain_conv(st):
    case, dt, K = st["case"], st["dt"], st["case"]["taps"]
    x, cu, w = st["x"].float(), st["cu"].long(), st["w"]
    T, W = x.shape
    S = len(cu) - 1
    init = torch.zeros(S, K - 1, W, device=x.device) if st["state"] is None else st["state"].float()
    ext = torch.cat([init.reshape(S * (K - 1), W), x])  # the states' rows, then the tokens
    seq, pos = _token_rows(cu, T)
    taps = []  # taps[j][t]: the row that tap j of token t reads
    for j in range(K):
        back = K - 1 - j
        taps.append(torch.where(pos >= back, S * (K - 1) + torch.arange(T, device=x.device) - back,
                                seq * (K - 1) + pos + j))
    u = sum(ext[taps[j]] * w[:, j] for j in range(K))
    if st["bias"] is not None:
        u = u + st["bias"]
    out, slope = _silu(u) if case["act"] == "silu" else (u, None)
    # the state behind a sequence: its last K - 1 rows, the initial state's among them where it is shorter
    lens = cu[1:] - cu[:-1]
    i = torch.arange(K - 1, device=x.device)
    at = lens.unsqueeze(1) + i - (K - 1)  # [S, K - 1], negative: a row of the initial state
    last = torch.where(at >= 0, S * (K - 1) + cu[:-1].unsqueeze(1) + at,
                       torch.arange(S, device=x.device).unsqueeze(1) * (K - 1) + at + K - 1)
    got = {"out": out.to(dt), "final": ext[last].to(dt)}
    if case["op"] == "conv":
        return got
    du = st["d_out"].float()
    if slope is not None:
        du = du * slope
    d_ext = torch.zeros_like(ext)
    for j in range(K):  # no row comes twice within a tap
        d_ext[taps[j]] = d_ext[taps[j]] + du * w[:, j]
    if st["d_final"] is not None:
        d_ext[last.flatten()] = d_ext[last.flatten()] + st["d_final"].float().reshape(-1, W)
    got["dx"] = d_ext[S * (K - 1):].to(dt)
    got["d_w"] = torch.stack([(du * ext[taps[j]]).sum(0) for j in range(K)], 1)
    got["d_bias"] = du.sum(0) if st["bias"] is not None else None
    got["d_init"] = d_ext[:S * (K - 1)].view(S, K - 1, W).to(dt) if st["state"] is not None else None
    return got


def _channels(v, W):
    """[rows, G, N] -> [rows, W, N]: each group's rows for its channels."""
    return v.float().repeat_interleave(W // v.shape[1], 1)


def _plain_select_step(st):
    x, W = st["x"].float(), st["case"]["width"]
    d, _ = _softplus(st["delta"].float() + st["delta_bias"])
    h = torch.exp(d.unsqueeze(2) * st["A"]) * st["state"] + (d * x).unsqueeze(2) * _channels(st["B"], W)
    y = (h * _channels(st["C"], W)).sum(2)
    if st["skip"] is not None:
        y = y + st["skip"] * x
    if st["z"] is not None:
        y = y * _silu(st["z"].float())[0]
    st["state"].copy_(h)
    return {"out": y.to(st["dt"]), "state": st["state"]}


def _doubling(a, b, longest):
    """All h_t = a_t h_{t-1} + b_t of the rows, by doublings of the composed steps up to the longest sequence."""
    n = 1
    while n < longest:
        b = torch.cat([b[:n], a[n:] * b[:-n] + b[n:]])
        if 2 * n < longest:
            a = torch.cat([a[:n], a[n:] * a[:-n]])
        n *= 2
    return b


def _plain_select(st):
    case, dt = st["case"], st["dt"]
    x, cu, A = st["x"].float(), st["cu"].long(), st["A"]
    T, W = x.shape
    N, G = case["state"], case["groups"]
    longest = max(_lengths(case))
    d, d_slope = _softplus(st["delta"].float() + st["delta_bias"])
    B, C = _channels(st["B"], W), _channels(st["C"], W)
    a = torch.exp(d.unsqueeze(2) * A)  # [T, W, N]
    full = cu[1:] > cu[:-1]  # sequences with tokens
    first, last = cu[:-1][full], cu[1:][full] - 1
    carry = a.clone()
    carry[first] = 0
    b = (d * x).unsqueeze(2) * B
    init = st["state"]
    if init is not None:
        b[first] += a[first] * init[full]
    h = _doubling(carry, b, longest)
    del b
    y = (h * C).sum(2)
    if st["skip"] is not None:
        y = y + st["skip"] * x
    gate = d_gate = None
    if st["z"] is not None:
        gate, d_gate = _silu(st["z"].float())
    final = torch.zeros(len(cu) - 1, W, N, device=x.device) if init is None else init.clone()
    final[full] = h[last]
    got = {"out": (y if gate is None else y * gate).to(dt), "final": final}
    if case["op"] == "select":
        return got
    dy = st["d_out"].float()
    got["d_z"] = None
    if gate is not None:
        got["d_z"] = (dy * y * d_gate).to(dt)
        dy = dy * gate
    # reverse: g_t = C_t dy_t + a_{t+1} g_{t+1}
    e = dy.unsqueeze(2) * C
    if st["d_final"] is not None:
        e[last] += st["d_final"][full]
    after = torch.cat([carry[1:], torch.zeros_like(carry[:1])])
    del carry
    g = _doubling(after.flip(0), e.flip(0), longest).flip(0)
    del after, e

    def group_sum(v):  # [T, W, N] -> [T, G, N]
        return v.view(T, G, W // G, N).sum(2).to(dt)

    got["d_C"] = group_sum(dy.unsqueeze(2) * h)
    before = torch.cat([torch.zeros_like(h[:1]), h[:-1]])
    del h
    before[first] = 0 if init is None else init[full]
    got["d_init"] = None
    if init is not None:
        d_init = torch.zeros_like(init) if st["d_final"] is None else st["d_final"].clone()
        d_init[full] = a[first] * g[first]
        got["d_init"] = d_init
    got["d_B"] = group_sum(g * (d * x).unsqueeze(2))
    Bg = (g * B).sum(2)
    gah = g * a * before
    del g, a, before
    got["d_A"] = (gah * d.unsqueeze(2)).sum(0)
    dx = d * Bg
    got["d_skip"] = None
    if st["skip"] is not None:
        dx = dx + st["skip"] * dy
        got["d_skip"] = (dy * x).sum(0)
    got["dx"] = dx.to(dt)
    dd = (x * Bg + (gah * A).sum(2)) * d_slope
    got["d_delta"] = dd.to(dt)
    got["d_delta_bias"] = dd.sum(0)
    return got


# ---------------------------------------------------------------------------
# Least work
# ---------------------------------------------------------------------------
def work(case):
    T, W, e, op = case["tokens"], case["width"], 2 if case["dtype"] == "bf16" else 4, case["op"]
    n = T * W
    if op in ("layer_norm", "layer_norm_grad"):
        vectors = (1 + case["bias"]) * 4 * W
        if op == "layer_norm":
            return {"bytes": (2 + 2 * case["residual"]) * n * e + vectors, "flops": 10 * n}
        return {"bytes": (3 + case["residual"]) * n * e + 4 * W + vectors, "flops": 20 * n}
    S = case["seqs"]
    if op.startswith("conv"):
        K = case["taps"]
        weights = 4 * W * (K + case["bias"])
        if op == "conv_step":
            return {"bytes": 2 * n * e * K + weights, "flops": (2 * K + 6) * n}
        state = S * (K - 1) * W * e
        size = 2 * n * e + weights + state * (1 + case["states"]) + 4 * (S + 1)
        flops = (2 * K + 6) * n
        if op == "conv_train":
            size += 2 * n * e + weights + 2 * state * case["states"]
            flops += (6 * K + 12) * n
        return {"bytes": size, "flops": flops}
    N, G = case["state"], case["groups"]
    weights = 4 * W * (N + 1 + case["skip"])
    tokens = (3 + case["gate"]) * n * e + 2 * T * G * N * e
    if op == "select_step":
        return {"bytes": tokens + weights + 8 * n * N, "flops": 7 * n * N}
    state = S * W * N * 4
    size = tokens + weights + state * (1 + case["states"]) + 4 * (S + 1)
    flops = 7 * n * N
    if op == "select_train":  # d_out in; gradients of the inputs, the weights and the states out
        size += (3 + case["gate"]) * n * e + 2 * T * G * N * e + weights + 2 * state * case["states"]
        flops += 20 * n * N
    return {"bytes": size, "flops": flops}


# ---------------------------------------------------------------------------
# 64 bits, from the definitions
# ---------------------------------------------------------------------------
def exact(case, seed):
    st = prepare(case, seed)
    st = {k: v.double() if torch.is_tensor(v) and v.is_floating_point() else v for k, v in st.items()}
    op = case["op"]
    if op.startswith("layer"):
        return _exact_norm(case, st)
    if op.startswith("conv"):
        return _exact_conv(case, st)
    return _exact_select(case, st)


def _exact_norm(case, st):
    """The definition; its gradients by automatic differentiation."""
    v = {k: st[k].clone().requires_grad_(True) for k in ("x", "w", "b") if st[k] is not None}
    r = v["x"] if st["r"] is None else v["x"] + st["r"]
    var, mean = torch.var_mean(r, 1, correction=0, keepdim=True)
    out = (r - mean) / (var + EPS).sqrt() * v["w"]
    if "b" in v:
        out = out + v["b"]
    if case["op"] == "layer_norm":
        return {"out": out.detach(), "residual": None if st["r"] is None else r.detach()}
    got = dict(zip(v, torch.autograd.grad(out, list(v.values()), st["d_out"])))
    dx = got["x"] if st["d_r"] is None else got["x"] + st["d_r"]
    return {"dx": dx, "d_w": got["w"], "d_b": got.get("b")}


def _exact_conv(case, st):
    """Sequence by sequence, the state's rows in front; gradients by automatic differentiation."""
    K, W, step = case["taps"], case["width"], case["op"] == "conv_step"
    names = [k for k in ("x", "w", "bias", "state") if st[k] is not None]
    grad = case["op"] == "conv_train"
    v = {k: st[k].clone().requires_grad_(grad) for k in names}

    def act(u):
        return u * torch.sigmoid(u) if case["act"] == "silu" else u

    if step:
        rows = torch.cat([v["state"], v["x"][:, None]], 1)
        u = torch.einsum("bkw,wk->bw", rows, v["w"])
        return {"out": act(u + v["bias"] if "bias" in v else u), "state": rows[:, 1:]}
    outs, finals = [], []
    at = 0
    for b, n in enumerate(_lengths(case)):
        rows = v["state"][b] if "state" in v else torch.zeros(K - 1, W, dtype=torch.float64, device=DEVICE)
        rows = torch.cat([rows, v["x"][at:at + n]])
        u = (rows.unfold(0, K, 1)[:n] * v["w"]).sum(2) if n else rows[:0]
        outs.append(act(u + v["bias"] if "bias" in v else u))
        finals.append(rows[n:])
        at += n
    out, final = torch.cat(outs), torch.stack(finals)
    got = {"out": out.detach(), "final": final.detach()}
    if not grad:
        return got
    outputs, grads = [out], [st["d_out"]]
    if st["d_final"] is not None:
        outputs, grads = outputs + [final], grads + [st["d_final"]]
    d = dict(zip(names, torch.autograd.grad(outputs, [v[k] for k in names], grads)))
    got.update(dx=d["x"], d_w=d["w"], d_bias=d.get("bias"), d_init=d.get("state"))
    return got


def _exact_select(case, st):
    """Token by token, all sequences side by side; the gradients by the adjoint recurrence."""
    W, N, G, op = case["width"], case["state"], case["groups"], case["op"]
    x, A = st["x"], st["A"]
    T, dev = x.shape[0], x.device
    raw = st["delta"] + st["delta_bias"]
    d = torch.logaddexp(raw, torch.zeros_like(raw))
    per = torch.arange(W, device=dev) // (W // G)  # the group of a channel
    skip = torch.zeros(W, dtype=torch.float64, device=dev) if st["skip"] is None else st["skip"]
    s = None if st["z"] is None else torch.sigmoid(st["z"])
    if op == "select_step":
        h = torch.exp(d[:, :, None] * A) * st["state"] + (d * x)[:, :, None] * st["B"][:, per]
        y = torch.einsum("twn,twn->tw", h, st["C"][:, per]) + skip * x
        return {"out": y if s is None else y * st["z"] * s, "state": h}
    lens, cu = _lengths(case), st["cu"].tolist()
    S = len(lens)
    if max(lens) > (80000 if op == "select" else 40000):
        return None
    order = sorted(range(S), key=lambda i: -lens[i])  # longest first: the running ones stay in front
    back = torch.tensor(order, device=dev)
    at = torch.tensor([cu[i] for i in order], device=dev)
    h = torch.zeros(S, W, N, dtype=torch.float64, device=dev) if st["state"] is None else st["state"][back].clone()
    train = op == "select_train"
    before = torch.empty(T, W, N, dtype=torch.float64, device=dev) if train else None
    y = torch.empty_like(x)
    live, alive = [], S
    for t in range(max(lens)):
        while alive and lens[order[alive - 1]] <= t:
            alive -= 1
        live.append(alive)
        rows = at[:alive] + t
        if train:
            before[rows] = h[:alive]
        dd = d[rows]
        h[:alive] = torch.exp(dd[:, :, None] * A) * h[:alive] + (dd * x[rows])[:, :, None] * st["B"][rows][:, per]
        y[rows] = (h[:alive] * st["C"][rows][:, per]).sum(2)
    y += skip * x
    final = torch.empty_like(h)
    final[back] = h
    got = {"out": y if s is None else y * st["z"] * s, "final": final}
    if not train:
        return got
    dy, got["d_z"] = st["d_out"], None
    if s is not None:
        got["d_z"] = dy * y * (s + st["z"] * s * (1 - s))
        dy = dy * st["z"] * s
    e = torch.zeros_like(h) if st["d_final"] is None else st["d_final"][back].clone()
    Bg, Agah = torch.empty_like(x), torch.empty_like(x)
    dA = torch.zeros_like(A)
    dB, dC = torch.empty_like(st["B"]), torch.empty_like(st["C"])
    for t in reversed(range(max(lens))):
        k = live[t]
        rows = at[:k] + t
        Bt, Ct = st["B"][rows][:, per], st["C"][rows][:, per]
        dd, h0 = d[rows], before[rows]
        a = torch.exp(dd[:, :, None] * A)
        du = (dd * x[rows])[:, :, None]
        g = e[:k] + dy[rows][:, :, None] * Ct
        dC[rows] = (dy[rows][:, :, None] * (a * h0 + du * Bt)).view(k, G, W // G, N).sum(2)
        dB[rows] = (g * du).view(k, G, W // G, N).sum(2)
        Bg[rows] = (g * Bt).sum(2)
        e[:k] = g * a
        w = e[:k] * h0
        Agah[rows] = (w * A).sum(2)
        dA += (w * dd[:, :, None]).sum(0)
    got["d_C"], got["d_B"], got["d_A"] = dC, dB, dA
    got["dx"] = d * Bg + skip * dy
    got["d_skip"] = None if st["skip"] is None else (dy * x).sum(0)
    dd = (x * Bg + Agah) * torch.sigmoid(raw)
    got["d_delta"], got["d_delta_bias"] = dd, dd.sum(0)
    got["d_init"] = None
    if st["state"] is not None:
        got["d_init"] = torch.empty_like(e)
        got["d_init"][back] = e
    return got
