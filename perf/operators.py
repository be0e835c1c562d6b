"""The operators beside the SSE layer -- the gated linear recurrence (scan) and
the norms around a block -- as measurable cases.

``run`` computes a case either through this package's entry points (``own``
true) or in a plain form of elementary torch operations in 32 bits; ``exact``
computes the same outputs from the definitions in 64 bits.

Scan, per sequence and channel, with a_t = exp(log_gate_t), log_gate_t <= 0:

    h_t = a_t h_{t-1} + s(a_t) x_t        s = 1, 1 - a, or sqrt(1 - a^2)

Block norm, per token (RMS(u; w) = u * rsqrt(mean(u^2) + eps) * w):

    r' = residual_scale * r + branch_scale * c * act(z) * RMS_group(o; w_after)
    x' = RMS_row(r'; w_before)

with every part but one of o and r optional.
"""
import random

import torch

own = False

MOST_SEQS = 64


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def listed():
    def scan(name, **kw):
        base = dict(name=name, op="scan", dtype="bf16", scale="plain", tokens=1, seqs=1, width=2048, ragged=False,
                    states=False, fused=False, lens=1)
        return dict(base, **kw)

    def norm(name, **kw):
        base = dict(name=name, op="norm", dtype="bf16", tokens=1, width=2048, group=0, gate="none", after=True,
                    channel=False, residual=True, before=True, fused=False)
        return dict(base, **kw)

    return [
        # one user's prompt in front of a reply: latency
        scan("scan_prompt", scale="unit", tokens=500, width=1024, states=True),
        # long documents of uneven length, continued from stored states
        scan("scan_varlen", scale="unit", tokens=72001, seqs=16, ragged=True, states=True, lens=3),
        # full precision, odd lengths, empty sequences, a width that is no multiple of 64
        scan("scan_ragged_f32", dtype="f32", scale="complement", tokens=3001, seqs=9, width=1000, ragged=True,
             states=True, lens=5),
        # training step of a layer: 8 x 4096 tokens, 16 heads of 128
        scan("scan_train_layer", op="scan_train", tokens=32768, seqs=8),
        # training on a small ragged batch in full precision
        scan("scan_train_ragged", op="scan_train", dtype="f32", scale="unit", tokens=1501, seqs=5, width=520,
             ragged=True, states=True, lens=7),
        # one stream answering, token by token
        scan("step_one", op="step", scale="unit", tokens=1),
        # 256 streams answering at once, inputs sliced from one projection
        scan("step_batch", op="step", scale="unit", tokens=256, fused=True),
        # between two blocks while decoding a few streams
        norm("norm_step", tokens=4, channel=True),
        # a layer's read-out of 8 x 4096 tokens: per-head norm and gate, gate sliced from a projection
        norm("norm_heads", tokens=32768, group=128, gate="silu", residual=False, before=False, fused=True),
        # between two blocks: norm after, channel scale, residual, norm before
        norm("norm_between", tokens=16384, width=2304, channel=True),
        # its gradient in a training step, the block's output normed by heads and gated
        norm("norm_grad_layer", op="norm_grad", tokens=16384, group=128, gate="silu"),
        # full precision, odd sizes
        norm("norm_grad_odd", op="norm_grad", dtype="f32", tokens=1009, width=1000, gate="sigmoid", channel=True),
    ]


def _log(rng, lo, hi):
    import math
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["scan", "scan", "scan_train", "step", "norm", "norm", "norm_grad"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    limit = 24_000_000 if dtype == "f32" else 48_000_000  # elements of one token tensor
    width = 8 * _log(rng, 8, 512)
    if op == "step":
        tokens = _log(rng, 1, 512)
    else:
        tokens = _log(rng, 1, min(65536, limit // width))
    if op in ("scan", "scan_train", "step"):
        seqs = 1 if rng.random() < 0.4 else _log(rng, 2, MOST_SEQS)
        return dict(op=op, dtype=dtype, scale=rng.choice(["plain", "complement", "unit"]), tokens=tokens, seqs=seqs,
                    width=width, ragged=seqs > 1, states=rng.random() < 0.6, fused=rng.random() < 0.5,
                    lens=rng.randrange(1 << 20))
    residual = rng.random() < 0.7
    group = 0
    if rng.random() < 0.5:
        group = rng.choice([32, 64, 128])
        width = max(group, width // group * group)
        tokens = max(1, min(tokens, limit // width))
    return dict(op=op, dtype=dtype, tokens=tokens, width=width, group=group,
                gate=rng.choice(["none", "silu", "sigmoid", "linear"]), after=group > 0 or rng.random() < 0.7,
                channel=rng.random() < 0.5, residual=residual, before=rng.random() < 0.7, fused=rng.random() < 0.5)


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
def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    T, W = case["tokens"], case["width"]

    def normal(*shape, std=1.0, mean=0.0, dtype=dt):
        return (torch.randn(*shape, generator=g, device="cuda") * std + mean).to(dtype)

    st = {"case": case, "dt": dt}
    if case["op"] in ("scan", "scan_train", "step"):
        # log-gates as the layer's front end makes them: logsigmoid(N(0, 1)) / 16
        def log_gate():
            return torch.nn.functional.logsigmoid(torch.randn(T, W, generator=g, device="cuda")) / 16

        if case["fused"]:  # both are slices of one projection's rows
            both = torch.empty(T, 2 * W, device="cuda", dtype=dt)
            both[:, :W] = normal(T, W)
            both[:, W:] = log_gate().to(dt)
            st["x"], st["log_gate"] = both[:, :W], both[:, W:]
        else:
            st["x"], st["log_gate"] = normal(T, W), log_gate().to(dt)
        if case["op"] == "step":
            st["state"] = normal(T, W, dtype=torch.float32)
            st["out"] = torch.empty(T, W, device="cuda", dtype=dt)
        else:
            lens = _lengths(case)
            cu = [0]
            for n in lens:
                cu.append(cu[-1] + n)
            st["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
            S = len(lens)
            st["init"] = normal(S, W, dtype=torch.float32) if case["states"] else None
            if case["op"] == "scan_train":
                st["d_out"] = normal(T, W)
                st["d_final"] = normal(S, W, dtype=torch.float32) if case["states"] else None
        st["cfg"] = _scan_config(case)
        return st
    st["o"] = normal(T, W, std=0.7)
    st["z"] = None
    if case["gate"] != "none":
        if case["fused"]:
            st["z"] = normal(T, 3 * W)[:, 2 * W:]
        else:
            st["z"] = normal(T, W)
    st["r"] = normal(T, W, std=2.0) if case["residual"] else None
    f32 = torch.float32
    st["w_after"] = normal(W, std=0.1, mean=1.0, dtype=f32) if case["after"] else None
    st["channel"] = normal(W, std=0.05, mean=0.5, dtype=f32) if case["channel"] else None
    st["w_before"] = normal(W, std=0.1, mean=1.0, dtype=f32) if case["before"] else None
    if case["op"] == "norm_grad":
        st["r_out"] = normal(T, W, std=2.1)  # the stored residual stream
        st["d_r_out"] = normal(T, W, std=0.1)
        st["d_next"] = normal(T, W, std=0.1) if case["before"] else None
    st["cfg"] = _norm_config(case)
    return st


EPS, RESIDUAL_SCALE, BRANCH_SCALE = 1e-6, 0.9, 1.1


class _Plan(dict):
    """What a program keeps of an operator's settings; the package's own form of it is made at its first call."""


def _scan_config(case):
    return _Plan(width=case["width"], input_scale=case["scale"], dtype=case["dtype"])


def _norm_config(case):
    return _Plan(width=case["width"], group=case["group"], gate=case["gate"], eps=EPS,
                 residual_scale=RESIDUAL_SCALE, branch_scale=BRANCH_SCALE, dtype=case["dtype"])


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------
def run(st):
    if own:
        return _run_own(st)
    op = st["case"]["op"]
    if op == "step":
        return _plain_step(st)
    if op == "norm":
        return _plain_norm(st)
    if op == "norm_grad":
        return _plain_norm_grad(st)
    return _plain_scan(st)


def _run_own(st):
    from sparse_state_linear_router_gb300 import binding
    op, case = st["case"]["op"], st["case"]
    cfg = st["cfg"].get("own")
    if cfg is None:
        make = binding.make_scan_config if op in ("scan", "scan_train", "step") else binding.make_norm_config
        cfg = make(**st["cfg"])
        st["cfg"]["own"] = cfg
    if op == "step":
        binding.scan_step(cfg, st["state"], st["x"], st["log_gate"], out=st["out"])
        return {"out": st["out"], "state": st["state"]}
    if op == "scan":
        r = binding.scan_forward(cfg, st["x"], st["log_gate"], st["cu"], initial_state=st["init"])
        return {"out": r["out"], "final": r["final_state"]}
    if op == "scan_train":
        r = binding.scan_forward(cfg, st["x"], st["log_gate"], st["cu"], initial_state=st["init"],
                                 want_checkpoints=True)
        b = binding.scan_backward(cfg, st["x"], st["log_gate"], st["cu"], r["checkpoints"], st["d_out"],
                                  initial_state=st["init"], d_final_state=st["d_final"],
                                  want_d_initial_state=case["states"])
        return {"out": r["out"], "final": r["final_state"], "dx": b["dx"], "d_log_gate": b["d_log_gate"],
                "d_init": b["d_initial_state"]}
    if op == "norm":
        r = binding.block_norm(cfg, st["o"], gate=st["z"], residual=st["r"], w_after=st["w_after"],
                               channel_scale=st["channel"], w_before=st["w_before"])
        return {"residual": r["residual_out"], "next": r["next_in"]}
    b = binding.block_norm_backward(cfg, st["d_r_out"], st["o"], gate=st["z"], w_after=st["w_after"],
                                    channel_scale=st["channel"], w_before=st["w_before"], residual_out=st["r_out"],
                                    d_next_in=st["d_next"], want_d_residual=case["residual"])
    return {"d_o": b["d_block_out"], "d_z": b["d_gate"], "d_r": b["d_residual"], "d_w_after": b["d_w_after"],
            "d_channel": b["d_channel_scale"], "d_w_before": b["d_w_before"]}


# ---------------------------------------------------------------------------
# Plain forms (32 bits)
# ---------------------------------------------------------------------------
def _decay_and_scale(la, mode):
    """a = exp(la), s(a), and ds/dla."""
    a = torch.exp(la)
    if mode == "plain":
        return a, None, None
    if mode == "complement":
        return a, -torch.expm1(la), -a
    s = torch.sqrt(-torch.expm1(2 * la))
    return a, s, torch.where(s > 0, -a * a / s, torch.zeros_like(s))


def _scan_doubling(a, b):
    """All h_t = a_t h_{t-1} + b_t of the rows, by log2(T) doublings of the composed steps."""
    n = 1
    while n < a.shape[0]:
        b = torch.cat([b[:n], a[n:] * b[:-n] + b[n:]])
        a = torch.cat([a[:n], a[n:] * a[:-n]])
        n *= 2
    return b


def _plain_step(st):
    x, la = st["x"].float(), st["log_gate"].float()
    a, s, _ = _decay_and_scale(la, st["case"]["scale"])
    h = a * st["state"] + (x if s is None else s * x)
    st["state"].copy_(h)
    st["out"].copy_(h)
    return {"out": st["out"], "state": st["state"]}


def _plain_scan(st):
    case, dt = st["case"], st["dt"]
    x, la, cu = st["x"].float(), st["log_gate"].float(), st["cu"].long()
    T, W = x.shape
    a, s, ds = _decay_and_scale(la, case["scale"])
    b = x if s is None else s * x
    init = st["init"]
    full = cu[1:] > cu[:-1]                      # sequences with tokens
    first, last = cu[:-1][full], cu[1:][full] - 1
    carry = a.clone()
    carry[first] = 0
    if init is not None:
        b = b.clone()
        b[first] += a[first] * init[full]
    h = _scan_doubling(carry, b)
    final = torch.zeros(len(cu) - 1, W, device=x.device) if init is None else init.clone()
    final[full] = h[last]
    out = {"out": h.to(dt), "final": final}
    if case["op"] == "scan":
        return out
    # reverse: dh_t = d_out_t + a_{t+1} dh_{t+1}
    dy = st["d_out"].float()
    if st["d_final"] is not None:
        dy = dy.clone()
        dy[last] += st["d_final"][full]
    after = torch.cat([carry[1:], torch.zeros_like(carry[:1])])
    dh = _scan_doubling(after.flip(0), dy.flip(0)).flip(0)
    h_before = torch.cat([torch.zeros_like(h[:1]), h[:-1]])
    h_before[first] = 0 if init is None else init[full]
    out["dx"] = (dh if s is None else s * dh).to(dt)
    d_la = a * h_before
    if ds is not None:
        d_la = d_la + ds * x
    out["d_log_gate"] = (dh * d_la).to(dt)
    out["d_init"] = None
    if init is not None:
        d_init = torch.zeros_like(init) if st["d_final"] is None else st["d_final"].clone()
        d_init[full] = a[first] * dh[first]
        out["d_init"] = d_init
    return out


def _act(z, kind):
    """act(z) and its derivative."""
    if kind == "linear":
        return z, torch.ones_like(z)
    sg = 1 / (1 + torch.exp(-z))
    if kind == "sigmoid":
        return sg, sg * (1 - sg)
    return z * sg, sg * (1 + z * (1 - sg))


def _normed(u, group):
    """u / sqrt(mean(u^2) + eps) over groups of columns, and the factor."""
    v = u.view(u.shape[0], -1, group) if group else u.unsqueeze(1)
    rstd = 1 / torch.sqrt((v * v).mean(-1, keepdim=True) + EPS)
    return (v * rstd).view_as(u), rstd


def _plain_norm(st):
    case, dt = st["case"], st["dt"]
    u = st["o"].float()
    if case["after"]:
        u = _normed(u, case["group"])[0] * st["w_after"]
    if st["z"] is not None:
        u = u * _act(st["z"].float(), case["gate"])[0]
    if st["channel"] is not None:
        u = u * st["channel"]
    r = BRANCH_SCALE * u
    if st["r"] is not None:
        r = r + RESIDUAL_SCALE * st["r"].float()
    nxt = None
    if case["before"]:
        nxt = (_normed(r, 0)[0] * st["w_before"]).to(dt)
    return {"residual": r.to(dt), "next": nxt}


def _norm_pull(d_hat, hat, rstd, group):
    """The gradient through hat = u * rstd."""
    n = hat.shape[0]
    d, h = (v.view(n, -1, group) if group else v.unsqueeze(1) for v in (d_hat, hat))
    return (rstd * (d - h * (d * h).mean(-1, keepdim=True))).view_as(hat)


def _plain_norm_grad(st):
    case, dt = st["case"], st["dt"]
    out = {"d_z": None, "d_r": None, "d_w_after": None, "d_channel": None, "d_w_before": None}
    d = st["d_r_out"].float()
    if case["before"]:
        hat, rstd = _normed(st["r_out"].float(), 0)
        dn = st["d_next"].float()
        out["d_w_before"] = (dn * hat).sum(0)
        d = d + _norm_pull(dn * st["w_before"], hat, rstd, 0)
    if case["residual"]:
        out["d_r"] = (RESIDUAL_SCALE * d).to(dt)
    d = BRANCH_SCALE * d
    u = st["o"].float()
    if case["after"]:
        hat, rstd = _normed(u, case["group"])
    else:
        hat = u
    plain = d * hat
    if st["z"] is not None:
        act, d_act = _act(st["z"].float(), case["gate"])
        d_z = plain * d_act
        if case["after"]:
            d_z = d_z * st["w_after"]
        if st["channel"] is not None:
            d_z = d_z * st["channel"]
        out["d_z"] = d_z.to(dt)
        plain, d = plain * act, d * act
    if st["channel"] is not None:
        out["d_channel"] = (plain * st["w_after"] if case["after"] else plain).sum(0)
        plain, d = plain * st["channel"], d * st["channel"]
    if case["after"]:
        out["d_w_after"] = plain.sum(0)
        d = _norm_pull(d * st["w_after"], hat, rstd, case["group"])
    out["d_o"] = d.to(dt)
    return out


# ---------------------------------------------------------------------------
# Least work
# ---------------------------------------------------------------------------
def work(case):
    T, W, e = case["tokens"], case["width"], 2 if case["dtype"] == "bf16" else 4
    n, op = T * W, case["op"]
    if op == "step":
        return {"bytes": n * (3 * e + 8), "flops": 8 * n}
    if op in ("scan", "scan_train"):
        S, states = case["seqs"], case["seqs"] * W * 4
        size = 3 * n * e + states + 4 * (S + 1) + (states if case["states"] else 0)
        flops = 8 * n
        if op == "scan_train":  # d_out in, two gradients out, the states' gradients
            size += 3 * n * e + (2 * states if case["states"] else 0)
            flops += 12 * n
        return {"bytes": size, "flops": flops}
    vectors = sum(bool(case[k]) for k in ("after", "channel", "before")) * 4 * W
    gate = case["gate"] != "none"
    if op == "norm":
        tensors = 2 + gate + case["residual"] + case["before"]
        return {"bytes": tensors * n * e + vectors, "flops": 16 * n}
    tensors = 3 + 2 * gate + case["residual"] + 2 * case["before"]
    return {"bytes": tensors * n * e + 2 * vectors, "flops": 40 * n}


# ---------------------------------------------------------------------------
# 64 bits, from the definitions
# ---------------------------------------------------------------------------
def exact(case, seed):
    st = prepare(case, seed)
    st = {k: v.double() if torch.is_tensor(v) and v.is_floating_point() else v for k, v in st.items()}
    if case["op"] in ("norm", "norm_grad"):
        return _exact_norm(case, st)
    if case["op"] == "step":
        a = st["log_gate"].exp()
        h = a * st["state"] + _exact_scale(st["log_gate"], case["scale"]) * st["x"]
        return {"out": h, "state": h}
    return _exact_scan(case, st)


def _exact_scale(la, mode):
    if mode == "plain":
        return torch.ones_like(la)
    return -torch.expm1(la) if mode == "complement" else (-torch.expm1(2 * la)).sqrt()


def _exact_scan(case, st):
    """Token by token, all sequences side by side; the gradients by the adjoint recurrence."""
    lens = _lengths(case)
    cu = st["cu"].tolist()
    dev, W, S = st["x"].device, case["width"], len(lens)
    x, la = st["x"], st["log_gate"]
    s = _exact_scale(la, case["scale"])
    h = torch.zeros(S, W, dtype=torch.float64, device=dev) if st["init"] is None else st["init"].clone()
    h0 = h.clone()
    order = sorted(range(S), key=lambda i: -lens[i])  # longest first: the running ones stay in front
    at = torch.tensor([cu[i] for i in order], device=dev)
    back = torch.tensor(order, device=dev)
    h = h[back]
    a, b = la.exp(), s * x
    out, before = torch.empty_like(x), torch.empty_like(x)
    longest, alive = max(lens), S
    live = []
    for t in range(longest):
        while alive and lens[order[alive - 1]] <= t:
            alive -= 1
        live.append(alive)
        rows = at[:alive] + t
        before[rows] = h[:alive]
        h[:alive] = a[rows] * h[:alive] + b[rows]
        out[rows] = h[:alive]
    final = torch.empty_like(h)
    final[back] = h
    got = {"out": out, "final": final}
    if case["op"] == "scan":
        return got
    e = torch.zeros_like(h0) if st["d_final"] is None else st["d_final"].clone()
    e = e[back]  # what reaches h_t from later steps
    dh = torch.empty_like(x)
    for t in reversed(range(longest)):
        k = live[t]
        rows = at[:k] + t
        d = st["d_out"][rows] + e[:k]
        dh[rows] = d
        e[:k] = a[rows] * d
    got["dx"] = s * dh
    slope = {"plain": 0.0 * a, "complement": -a}.get(case["scale"])
    if slope is None:
        slope = -(2 * la).exp() / s
    got["d_log_gate"] = dh * (a * before + slope * x)
    got["d_init"] = None
    if case["states"]:
        got["d_init"] = torch.empty_like(e)
        got["d_init"][back] = e
    return got


def _exact_norm(case, st):
    """The definition, and its gradients by automatic differentiation."""
    names = ["o", "z", "r", "w_after", "channel", "w_before"]
    grad = case["op"] == "norm_grad"
    v = {k: st[k].clone().requires_grad_(grad) if st[k] is not None else None for k in names}

    def rms(u, w, group):
        g = u.reshape(u.shape[0], -1, group or u.shape[1])
        return (g / (g.square().mean(2, keepdim=True) + EPS).sqrt()).reshape(u.shape) * w

    u = v["o"] if v["w_after"] is None else rms(v["o"], v["w_after"], case["group"])
    if v["z"] is not None:
        z = v["z"]
        u = u * {"silu": lambda: z * torch.sigmoid(z), "sigmoid": lambda: torch.sigmoid(z), "linear": lambda: z}[case["gate"]]()
    if v["channel"] is not None:
        u = u * v["channel"]
    r = BRANCH_SCALE * u
    if v["r"] is not None:
        r = r + RESIDUAL_SCALE * v["r"]
    if not grad:
        return {"residual": r, "next": None if v["w_before"] is None else rms(r, v["w_before"], 0)}
    d = st["d_r_out"]
    d_w_before = None
    if v["w_before"] is not None:  # the gradient is taken at the stored residual stream
        at = st["r_out"].clone().requires_grad_(True)
        pulled, d_w_before = torch.autograd.grad(rms(at, v["w_before"], 0), [at, v["w_before"]], st["d_next"])
        d = d + pulled
    wanted = [k for k in names[:5] if v[k] is not None]
    got = dict(zip(wanted, torch.autograd.grad(r, [v[k] for k in wanted], d)))
    return {"d_o": got["o"], "d_z": got.get("z"), "d_r": got.get("r"), "d_w_after": got.get("w_after"),
            "d_channel": got.get("channel"), "d_w_before": d_w_before}
