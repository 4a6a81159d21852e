"""What the token-wise fast-weight operators and the layer norm beside them are measured on.

Five operators: the gated delta rule over whole sequences (`delta`), its backward pass (`delta_grad`), its step of one
token for each row of a serving batch (`step`), layer norm (`norm`) and its backward pass with the reduction of the
weight's and the bias's gradient (`norm_grad`).

The gated delta rule, for each value head with its state S [dk, dv] (kept transposed, W [dv, dk]), S_0 = W_init^T or 0:
    e_t = v_t - exp(g_t) S_{t-1}^T k_t,   S_t = exp(g_t) S_{t-1} + beta_t k_t e_t^T,   o_t = scale S_t^T q_t.
Layer norm, for each row x of width d:
    y = (x - mean(x)) / sqrt(mean((x - mean(x))^2) + eps) * weight + bias.
"""
import math

import torch

own = False

CHUNK = 64  # tokens taken together in the plain form of the gated delta rule
EPS = 1e-5
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
LARGEST = 65536 * 32 * 128 * 128  # tokens x value heads x state size of the largest listed sequence


def listed():
    return [
        # a prompt of 64K tokens for one user, heads cut out of a token-major projection, two value heads to a key head
        {"name": "delta_64k", "op": "delta", "dtype": "bf16", "seqs": "65536", "k_heads": 16, "v_heads": 32, "k_dim": 128,
         "v_dim": 128, "batch": 1, "packed": False, "resumed": False, "layout": "token", "behind": 0},
        # a serving batch of prompts packed one behind the other, each resumed from its state: a long one, ordinary
        # ones, a single token, an empty one, and rows behind the last sequence that belong to nobody
        {"name": "delta_packed", "op": "delta", "dtype": "bf16",
         "seqs": "6007 1 0 517 2048 64 63 1000 4096 129 31 2500", "k_heads": 8, "v_heads": 16, "k_dim": 128, "v_dim": 128,
         "batch": 1, "packed": True, "resumed": True, "layout": "token", "behind": 45},
        # a short fp32 sequence on narrow heads: what a check of a model runs, where latency counts
        {"name": "delta_short_f32", "op": "delta", "dtype": "f32", "seqs": "100", "k_heads": 4, "v_heads": 4, "k_dim": 64,
         "v_dim": 72, "batch": 2, "packed": False, "resumed": False, "layout": "head", "behind": 0},
        # one training step's rows, two value heads to a key head
        {"name": "delta_grad_4x4k", "op": "delta_grad", "dtype": "bf16", "seqs": "4096", "k_heads": 8, "v_heads": 16,
         "k_dim": 128, "v_dim": 128, "batch": 4, "packed": False, "resumed": False, "layout": "token", "behind": 0},
        # a fine-tuning step in fp32: a packed row of documents of odd lengths carried on from earlier states
        {"name": "delta_grad_docs_f32", "op": "delta_grad", "dtype": "f32", "seqs": "777 1 300 64 35", "k_heads": 2,
         "v_heads": 4, "k_dim": 96, "v_dim": 80, "batch": 1, "packed": True, "resumed": True, "layout": "head", "behind": 3},
        # one user's next token
        {"name": "step_1", "op": "step", "dtype": "bf16", "rows": 1, "pool": 4, "padding": 0, "k_heads": 16, "v_heads": 32,
         "k_dim": 128, "v_dim": 128},
        # a full serving batch: rows in any order over a pool of states
        {"name": "step_256", "op": "step", "dtype": "bf16", "rows": 256, "pool": 320, "padding": 0, "k_heads": 16,
         "v_heads": 32, "k_dim": 128, "v_dim": 128},
        # a captured fp32 batch padded to its size, odd heads
        {"name": "step_33_f32", "op": "step", "dtype": "f32", "rows": 33, "pool": 40, "padding": 5, "k_heads": 5,
         "v_heads": 5, "k_dim": 96, "v_dim": 80},
        # the hidden states that one 128K call of the In-Place layer takes
        {"name": "norm_128k", "op": "norm", "dtype": "bf16", "rows": 131072, "dim": 2560, "bias": True},
        # a few tokens of an odd width
        {"name": "norm_7_f32", "op": "norm", "dtype": "f32", "rows": 7, "dim": 1001, "bias": True},
        # training rows of the In-Place layer's width
        {"name": "norm_grad_32k", "op": "norm_grad", "dtype": "bf16", "rows": 32768, "dim": 2560, "bias": True},
        # the norm of each head's output: short rows, many of them
        {"name": "norm_grad_heads", "op": "norm_grad", "dtype": "bf16", "rows": 524288, "dim": 128, "bias": False},
    ]


def _log_uniform(rng, low, high):
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["delta", "delta", "delta_grad", "delta_grad", "step", "step", "norm", "norm_grad"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op in ("norm", "norm_grad"):
        dim = rng.choice([_log_uniform(rng, 8, 8192), 8 * _log_uniform(rng, 8, 1024), rng.choice([128, 1024, 2560, 4096])])
        most = (131072 if op == "norm" else 32768) * 2560 // (dim * (1 if dtype == "bf16" else 2))
        rows = _log_uniform(rng, 1, min(1 << 19, most))
        return {"op": op, "dtype": dtype, "rows": rows, "dim": dim, "bias": rng.random() < 0.5}
    k_heads, shared = rng.choice([1, 2, 3, 4, 8, 16]), rng.choice([1, 1, 2, 2, 4])
    k_dim = rng.choice([128, 128, 64, 8 * rng.randint(2, 32)])
    v_dim = rng.choice([k_dim, 128, 8 * rng.randint(2, 32)])
    v_heads = k_heads * shared
    size = v_heads * k_dim * v_dim
    heads = {"k_heads": k_heads, "v_heads": v_heads, "k_dim": k_dim, "v_dim": v_dim}
    if op == "step":
        rows = _log_uniform(rng, 1, max(1, min(512, 256 * 32 * 128 * 128 // size)))
        return {"op": op, "dtype": dtype, "rows": rows, "pool": rows + rng.randint(0, rows),
                "padding": rng.randint(0, rows // 4), **heads}
    # fp32 and the backward pass cost more for a token: fewer tokens
    most = LARGEST // size // (1 if op == "delta" else 8) // (1 if dtype == "bf16" else 8)
    total = _log_uniform(rng, 1, max(1, min(65536 if op == "delta" else 16384, most)))
    packed = rng.random() < 0.5
    case = {"op": op, "dtype": dtype, "batch": 1, "packed": packed, "resumed": rng.random() < 0.5,
            "layout": rng.choice(["token", "head"]), "behind": rng.randint(0, 70) if packed else 0, **heads}
    if packed:
        cuts = sorted(rng.randint(0, total) for _ in range(rng.randint(0, 15)))
        case["seqs"] = " ".join(str(b - a) for a, b in zip([0] + cuts, cuts + [total]))
    else:
        case["batch"] = min(total, rng.choice([1, 1, 2, 3, 5]))
        case["seqs"] = str(total // case["batch"])
    return case


# ------------------------------------------------------------------------------------------------------------ inputs


def _unit(x):
    return x / x.square().sum(-1, keepdim=True).sqrt()


def _gates(gen, heads, shape):
    """Log decays -a softplus(N(0, 1) + c), a in 1..16 and softplus(c) in 0.001..0.1 for each head, and rates in (0, 1)."""
    a = torch.empty(heads, device="cuda").uniform_(1, 16, generator=gen)
    c = torch.empty(heads, device="cuda").uniform_(math.log(1e-3), math.log(1e-1), generator=gen).exp().expm1().log()
    x = torch.randn(*shape, heads, device="cuda", generator=gen) + c
    g = -a * torch.log1p(torch.exp(x))
    return g, torch.sigmoid(torch.randn(*shape, heads, device="cuda", generator=gen))


def prepare(case, seed):
    gen = torch.Generator("cuda")
    gen.manual_seed(seed)
    dt = TYPES[case["dtype"]]
    normal = lambda *s: torch.randn(*s, device="cuda", generator=gen)  # noqa: E731
    s = {"case": case}
    if case["op"] in ("norm", "norm_grad"):
        rows, d = case["rows"], case["dim"]
        x = normal(rows, d)
        s["x"] = x.mul_(0.5 + 2 * torch.rand(rows, 1, device="cuda", generator=gen)).add_(normal(rows, 1)).to(dt)
        s["weight"] = (1 + 0.2 * normal(d)).to(dt)
        s["bias"] = (0.2 * normal(d)).to(dt) if case["bias"] else None
        if case["op"] == "norm_grad":
            s["dY"] = normal(rows, d).to(dt)
            # what the forward pass has left for it
            xf = s["x"].float()
            s["mean"] = xf.mean(-1)
            s["rstd"] = ((xf - s["mean"][:, None]).square_().mean(-1) + EPS).rsqrt_()
        return s
    Hk, Hv, dk, dv = (case[n] for n in ("k_heads", "v_heads", "k_dim", "v_dim"))
    s["scale"] = dk ** -0.5
    if case["op"] == "step":
        R, pool = case["rows"], case["pool"]
        s["q"], s["k"] = (_unit(normal(R, Hk, dk)).to(dt) for _ in range(2))
        s["v"] = normal(R, Hv, dv).to(dt)
        s["g"], s["beta"] = _gates(gen, Hv, (R,))
        s["W"] = 0.3 * normal(pool, Hv, dv, dk)
        slots = torch.randperm(pool, device="cuda", generator=gen)[:R].to(torch.int32)
        slots[R - case["padding"]:] = -1
        s["slots"] = slots
        s["live"] = R - case["padding"]
        return s
    lens = [int(n) for n in case["seqs"].split()]
    B, n = case["batch"], sum(lens) + case["behind"]
    swap = (lambda x: x.transpose(1, 2)) if case["layout"] == "token" else (lambda x: x.transpose(1, 2).contiguous())
    s["q"], s["k"] = (swap(_unit(normal(B, n, Hk, dk)).to(dt)) for _ in range(2))
    s["v"] = swap(normal(B, n, Hv, dv).to(dt))
    s["g"], s["beta"] = (swap(x) for x in _gates(gen, Hv, (B, n)))
    s["lens"] = lens
    rows = len(lens) if case["packed"] else B
    s["starts"] = torch.tensor([0] + lens, device="cuda").cumsum(0).to(torch.int32) if case["packed"] else None
    s["W_init"] = 0.3 * normal(rows, Hv, dv, dk) if case["resumed"] else None
    # outputs are the caller's: rows behind the last sequence stay as they are
    s["O"] = torch.zeros_like(s["v"])
    if case["op"] == "delta_grad":
        s["dO"] = swap(normal(B, n, Hv, dv).to(dt))
        s["dW_final"] = 0.1 * normal(rows, Hv, dv, dk) if case["resumed"] else None
        s["grads"] = [torch.zeros_like(s[n], dtype=dt) for n in ("q", "k", "v", "g", "beta")]
    return s


# ------------------------------------------------------------------------------------------------- the operators, plain


def _delta_sequence(q, k, v, g, beta, scale, S):
    """The gated delta rule over one length of rows [B, H, n, .] in 32 bits, CHUNK tokens at a time, from S [B, H, dk, dv]:
    O and the last state. Within a chunk with b the running sum of g, L = strictly lower (k_i . k_j exp(b_i - b_j)):
    U = (I + beta L)^-1 beta (V - exp(b) K S), and the state moves on by K^T exp(b_last - b) U."""
    B, H, n, dk = q.shape
    m = -(-n // CHUNK)
    pad = lambda x: torch.nn.functional.pad(x, (0, 0, 0, m * CHUNK - n)).reshape(B, H, m, CHUNK, x.shape[-1])  # noqa: E731
    q, k, v, beta = pad(q), pad(k), pad(v), pad(beta[..., None])
    b = pad(g[..., None].double()).cumsum(-2)  # in 64 bits: differences of sums that grow
    seen = torch.ones(CHUNK, CHUNK, device=q.device).tril().bool()
    D = torch.where(seen, b - b.mT, -math.inf).exp().float()
    rest, last, b = (b[..., -1:, :] - b).exp().float(), b[..., -1:, :].exp().float(), b.exp().float()
    kT = k.mT.contiguous()
    P = scale * (q @ kT) * D
    N = -beta * (k @ kT) * D.tril(-1)
    # (I - N)^-1 = (I + N)(I + N^2)(I + N^4)..., N^CHUNK = 0
    T = torch.eye(CHUNK, device=q.device) + N
    for _ in range(CHUNK.bit_length() - 2):
        N = N @ N
        T = T + T @ N
    O = []
    for c in range(m):
        U = T[:, :, c] @ (beta[:, :, c] * (v[:, :, c] - b[:, :, c] * (k[:, :, c] @ S)))
        O.append(scale * b[:, :, c] * (q[:, :, c] @ S) + P[:, :, c] @ U)
        S = last[:, :, c] * S + kT[:, :, c] @ (rest[:, :, c] * U)
    return (torch.cat(O, 2)[:, :, :n] if O else v.flatten(2, 3)), S


def _delta_plain(s, q, k, v, g, beta, W_init):
    """O for the tokens of sequences and every sequence's last state W, from 32-bit inputs."""
    case = s["case"]
    q, k = (x.repeat_interleave(case["v_heads"] // case["k_heads"], 1) for x in (q, k))
    rows = len(s["lens"]) if case["packed"] else case["batch"]
    S = v.new_zeros(rows, v.shape[1], q.shape[3], v.shape[3]) if W_init is None else W_init.mT
    if not case["packed"]:
        O, S = _delta_sequence(q, k, v, g, beta, s["scale"], S)
        return O, S.mT
    O, W, at = [], [], 0
    for i, n in enumerate(s["lens"]):
        part = [x[:, :, at:at + n] for x in (q, k, v, g, beta)]
        o, last = _delta_sequence(*part, s["scale"], S[i:i + 1])
        O.append(o)
        W.append(last.mT)
        at += n
    return torch.cat(O, 2), torch.cat(W)


def _wide(s, names):
    return [None if s[n] is None else s[n].float() for n in names]


def _run_plain(s):
    case = s["case"]
    dt = TYPES[case["dtype"]]
    if case["op"] == "delta":
        O, W = _delta_plain(s, *_wide(s, ("q", "k", "v", "g", "beta", "W_init")))
        s["O"][:, :, :O.shape[2]] = O.to(dt)
        return {"O": s["O"], "W_final": W.contiguous()}
    if case["op"] == "delta_grad":
        args = [None if x is None else x.detach().requires_grad_() for x in _wide(s, ("q", "k", "v", "g", "beta", "W_init"))]
        with torch.enable_grad():
            O, W = _delta_plain(s, *args)
            loss = (O * s["dO"][:, :, :O.shape[2]].float()).sum()
            if s["dW_final"] is not None:
                loss = loss + (W * s["dW_final"]).sum()
        d = torch.autograd.grad(loss, [x for x in args if x is not None])
        for out, x in zip(s["grads"], d):
            out.copy_(x)
        return {**dict(zip(("dq", "dk", "dv", "dg", "dbeta"), s["grads"])), **({"dW_init": d[5]} if len(d) > 5 else {})}
    if case["op"] == "step":
        live, shared = s["live"], case["v_heads"] // case["k_heads"]
        q, k, v, g, beta = (x[:live] for x in _wide(s, ("q", "k", "v", "g", "beta")))
        q, k = (x.repeat_interleave(shared, 1)[:, :, None] for x in (q, k))
        at = s["slots"][:live].long()
        W = s["W"][at] * g.exp()[..., None, None]
        W = W + (beta[..., None] * (v - (W * k).sum(-1)))[..., None] * k
        s["W"][at] = W
        O = torch.zeros_like(s["v"])
        O[:live] = (s["scale"] * (W * q).sum(-1)).to(dt)
        return {"O": O, "W": s["W"]}
    x, w = s["x"].float(), s["weight"].float()
    if case["op"] == "norm":
        x = x - x.mean(-1, keepdim=True)
        y = x * (x.square().mean(-1, keepdim=True) + EPS).rsqrt() * w
        return {"Y": (y if s["bias"] is None else y + s["bias"].float()).to(dt)}
    dY, rstd = s["dY"].float(), s["rstd"][:, None]
    h = (x - s["mean"][:, None]) * rstd
    a = dY * w
    dx = rstd * (a - a.mean(-1, keepdim=True) - h * (a * h).mean(-1, keepdim=True))
    # long sums: in 64 bits
    return {"dx": dx.to(dt), "dweight": (dY * h).sum(0, dtype=torch.float64).float(),
            "dbias": dY.sum(0, dtype=torch.float64).float() if case["bias"] else None}


def run(state):
    if not own:
        return _run_plain(state)
    import chunk_wise_weight_amd as cw

    s, op = state, state["case"]["op"]
    if op == "delta":
        O, W = cw.ttt_gated_delta(s["q"], s["k"], s["v"], s["g"], s["beta"], scale=s["scale"], W_init=s["W_init"],
                                  seq_starts=s["starts"], O=s["O"])
        return {"O": O, "W_final": W}
    if op == "delta_grad":
        dq, dk, dv, dg, dbeta = s["grads"]
        d = cw.ttt_gated_delta_backward(s["q"], s["k"], s["v"], s["g"], s["beta"], s["dO"], dW_final=s["dW_final"],
                                        scale=s["scale"], W_init=s["W_init"], seq_starts=s["starts"], dq=dq, dk=dk, dv=dv,
                                        dg=dg, dbeta=dbeta)
        return {n: x for n, x in zip(("dq", "dk", "dv", "dg", "dbeta", "dW_init"), d) if x is not None}
    if op == "step":
        O = cw.ttt_gated_delta_step(s["q"], s["k"], s["v"], s["g"], s["beta"], s["W"], slots=s["slots"], scale=s["scale"])
        return {"O": O, "W": s["W"]}
    if op == "norm":
        return {"Y": cw.ttt_layer_norm(s["x"], s["weight"], s["bias"], eps=EPS)[0]}
    dx, dweight, dbias = cw.ttt_layer_norm_backward(s["x"], s["weight"], s["dY"], s["mean"], s["rstd"],
                                                    bias=state["case"]["bias"])
    return {"dx": dx, "dweight": dweight, "dbias": dbias}


# --------------------------------------------------------------------------------------------------------- work, exact


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] in ("norm", "norm_grad"):
        rows, d = case["rows"], case["dim"]
        if case["op"] == "norm":
            return {"bytes": 2 * rows * d * e + (2 if case["bias"] else 1) * d * e, "flops": 8 * rows * d}
        return {"bytes": 3 * rows * d * e + 8 * rows + d * e + (8 if case["bias"] else 4) * d, "flops": 13 * rows * d}
    Hk, Hv, dk, dv = (case[n] for n in ("k_heads", "v_heads", "k_dim", "v_dim"))
    state = Hv * dk * dv
    if case["op"] == "step":
        live = case["rows"] - case["padding"]
        return {"bytes": case["rows"] * (Hv * dv * e + 4) + live * ((2 * Hk * dk + Hv * dv) * e + 8 * Hv + 8 * state),
                "flops": 7 * live * state}
    lens = [int(n) for n in case["seqs"].split()]
    n = sum(lens) * case["batch"]
    rows = len(lens) if case["packed"] else case["batch"]
    gates = 8 * n * Hv
    if case["op"] == "delta":
        return {"bytes": n * 2 * (Hk * dk + Hv * dv) * e + gates + 4 * rows * state * (2 if case["resumed"] else 1),
                "flops": 6 * n * state}
    # the states again (4 of the 6), then each of the six products that touch a state or its gradient, and their product
    states = 4 * rows * state * (3 if case["resumed"] else 0)
    return {"bytes": n * (4 * Hk * dk + 3 * Hv * dv + 2 * Hv) * e + gates + states, "flops": 18 * n * state}


def _tokens(s, grad):
    """The recurrence itself, token by token in 64 bits, states as W [B, H, dv, dk]; with `grad` its reverse too."""
    case, scale = s["case"], s["scale"]
    shared = case["v_heads"] // case["k_heads"]
    q, k, v, a, beta = (s[n].double() for n in ("q", "k", "v", "g", "beta"))
    a = a.exp()
    O = torch.zeros_like(v)
    dv, da, dbeta = (torch.zeros_like(x) for x in (v, a, beta))
    dO = s["dO"].double() if grad else None
    q, k = (x.unsqueeze(2).expand(-1, -1, shared, -1, -1).flatten(1, 2) for x in (q, k))
    dq, dk = torch.zeros_like(q), torch.zeros_like(k)
    lens = s["lens"]
    rows = len(lens) if case["packed"] else case["batch"]
    first = v.new_zeros(rows, v.shape[1], v.shape[3], q.shape[3]) if s["W_init"] is None else s["W_init"].double()
    finals, dfirst, at = [], [], 0
    for i, n in enumerate(lens):
        W = (first[i:i + 1] if case["packed"] else first).clone()

        def one(W, t):
            A = W * a[:, :, t, None, None]
            e = v[:, :, t] - (A * k[:, :, t, None]).sum(-1)
            return A, e, A + (beta[:, :, t, None] * e)[..., None] * k[:, :, t, None]

        kept = []
        for t in range(at, at + n):
            if grad and (t - at) % 64 == 0:
                kept.append(W)
            W = one(W, t)[2]
            if not grad:
                O[:, :, t] = scale * (W * q[:, :, t, None]).sum(-1)
        finals.append(W)
        if grad:
            dW = torch.zeros_like(first) if s["dW_final"] is None else s["dW_final"].double()
            dW = (dW[i:i + 1] if case["packed"] else dW).clone()
            for c in range(len(kept) - 1, -1, -1):
                steps, W = [], kept[c]
                for t in range(at + 64 * c, at + min(n, 64 * c + 64)):
                    A, e, new = one(W, t)
                    steps.append((t, W, A, e, new))
                    W = new
                for t, old, A, e, new in reversed(steps):
                    o = dO[:, :, t, :, None]
                    dq[:, :, t] = scale * (new * o).sum(-2)
                    dW = dW + scale * o * q[:, :, t, None]
                    du = (dW * k[:, :, t, None]).sum(-1)
                    de = beta[:, :, t, None] * du
                    dbeta[:, :, t] = (du * e).sum(-1)
                    dv[:, :, t] = de
                    dA = dW - de[..., None] * k[:, :, t, None]
                    dk[:, :, t] = (dW * (beta[:, :, t, None] * e)[..., None]).sum(-2) - (A * de[..., None]).sum(-2)
                    da[:, :, t] = (old * dA).sum((-1, -2))
                    dW = a[:, :, t, None, None] * dA
            dfirst.append(dW)
        at += n
    if not grad:
        return {"O": O, "W_final": torch.cat(finals)}
    dq, dk = (x.unflatten(1, (-1, shared)).sum(2) for x in (dq, dk))
    return {"dq": dq, "dk": dk, "dv": dv, "dg": da * a, "dbeta": dbeta,
            **({"dW_init": torch.cat(dfirst)} if s["W_init"] is not None else {})}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("delta", "delta_grad"):
        tokens = sum(int(n) for n in case["seqs"].split())
        if tokens * (1 if case["op"] == "delta" else 8) > 70000:
            return None  # about 20 seconds
        return _tokens(s, case["op"] == "delta_grad")
    if case["op"] == "step":
        q, k, v, g, beta, W = (s[n].double() for n in ("q", "k", "v", "g", "beta", "W"))
        O = torch.zeros_like(v)
        for r, slot in enumerate(s["slots"].tolist()):
            if slot < 0:
                continue
            for h in range(case["v_heads"]):
                j = h // (case["v_heads"] // case["k_heads"])
                M = W[slot, h] * torch.exp(g[r, h])
                M = M + torch.outer(beta[r, h] * (v[r, h] - M.mv(k[r, j])), k[r, j])
                W[slot, h] = M
                O[r, h] = s["scale"] * M.mv(q[r, j])
        return {"O": O, "W": W}
    x, w = s["x"].double(), s["weight"].double()
    var, mean = torch.var_mean(x, -1, correction=0, keepdim=True)
    if case["op"] == "norm":
        bias = s["bias"].double() if case["bias"] else torch.zeros_like(w)
        return {"Y": torch.addcmul(bias, (x - mean) / torch.sqrt(var + EPS), w)}
    # from the statistics that the forward pass left, as the operator's definition takes them
    r = s["rstd"].double()[:, None]
    h = (x - s["mean"].double()[:, None]) * r
    dY = s["dY"].double()
    a = dY * w
    d = a.shape[1]
    dx = r * (a - a.sum(-1, keepdim=True) / d - h * ((a * h).sum(-1, keepdim=True) / d))
    return {"dx": dx, "dweight": (dY * h).sum(0), "dbias": dY.sum(0) if case["bias"] else None}
