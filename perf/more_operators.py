"""What the selective state space scan, its short convolution and the root-mean-square norm are measured on.

Five operators: the selective scan over whole sequences (`scan`), its backward pass (`scan_grad`), its step of one token
for each row of a serving batch (`step`); the short causal convolution in front of it, forward, backward and for single
tokens (`conv`); and the root-mean-square norm of the sum with the residual, in 8 bits too, with its backward (`norm`).

The scan, for each head with its state S [P, N], S_0 = S_init or 0, B and C shared by the heads of a group:
    r_t = softplus(dt_t + dt_bias) or dt_t,   S_t = exp(A r_t) S_{t-1} + r_t x_t B_t^T,   o_t = S_t C_t + D x_t.
The convolution, for each channel with K taps w, earlier rows from x_init or 0:
    y_t = silu(bias + sum_j w_j x_{t-K+1+j}).
The norm, for each row: h = x + residual, rounded to their type, y = h / sqrt(mean(h^2) + eps) * weight; in 8 bits (e4m3)
y / scale with scale = max |y| / 448 over a row or over groups of its columns.
"""
import math

import torch

own = False

CHUNK = 64  # tokens taken together in the plain form of the scan
EPS = 1e-5
E4M3_MAX = 448.0
TINY = 2.0 ** -126  # the least scale
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SCAN_MOST = 65536 * 64 * 64 * 128  # tokens x heads x state size of the largest listed sequence
GRAD_MOST = 4 * 4096 * 32 * 64 * 128
CONV_MOST = 65536 * 6144
NORM_MOST = 131072 * 2560


def listed():
    return [
        # a prompt of 64K tokens for one user: x, B and C cut out of the convolution's token-major output
        {"name": "scan_64k", "op": "scan", "dtype": "bf16", "seqs": "65536", "heads": 64, "groups": 8, "head_dim": 64,
         "state": 128, "batch": 1, "packed": False, "resumed": False, "layout": "token", "behind": 0, "skip": True,
         "softplus": True},
        # a serving batch of prompts packed one behind the other, each resumed from its state: long and ordinary ones, a
        # single token, an empty one, and rows behind the last sequence that belong to nobody
        {"name": "scan_packed", "op": "scan", "dtype": "bf16", "seqs": "6007 1 0 517 2048 64 63 1000 4096 129 31 2500",
         "heads": 32, "groups": 1, "head_dim": 64, "state": 128, "batch": 1, "packed": True, "resumed": True,
         "layout": "token", "behind": 45, "skip": True, "softplus": True},
        # a short fp32 sequence on odd heads: what a check of a model runs, where latency counts
        {"name": "scan_short_f32", "op": "scan", "dtype": "f32", "seqs": "100", "heads": 4, "groups": 2, "head_dim": 72,
         "state": 16, "batch": 2, "packed": False, "resumed": False, "layout": "head", "behind": 0, "skip": False,
         "softplus": False},
        # one training step's rows
        {"name": "scan_grad_4x4k", "op": "scan_grad", "dtype": "bf16", "seqs": "4096", "heads": 32, "groups": 4,
         "head_dim": 64, "state": 128, "batch": 4, "packed": False, "resumed": False, "layout": "token", "behind": 0,
         "skip": True, "softplus": True},
        # a fine-tuning step in fp32: a packed row of documents of odd lengths carried on from earlier states
        {"name": "scan_grad_docs_f32", "op": "scan_grad", "dtype": "f32", "seqs": "777 1 300 64 35", "heads": 4,
         "groups": 2, "head_dim": 80, "state": 64, "batch": 1, "packed": True, "resumed": True, "layout": "head",
         "behind": 3, "skip": True, "softplus": False},
        # one user's next token
        {"name": "step_1", "op": "step", "dtype": "bf16", "rows": 1, "pool": 4, "padding": 0, "heads": 64, "groups": 8,
         "head_dim": 64, "state": 128, "skip": True, "softplus": True},
        # a full serving batch, padded to its size: rows in any order over a pool of states
        {"name": "step_256", "op": "step", "dtype": "bf16", "rows": 256, "pool": 320, "padding": 7, "heads": 64,
         "groups": 8, "head_dim": 64, "state": 128, "skip": True, "softplus": True},
        # the convolution in front of the prompt's scan: channels of x, B and C
        {"name": "conv_64k", "op": "conv", "pass": "forward", "dtype": "bf16", "seqs": "65536", "batch": 1, "packed": False,
         "resumed": False, "behind": 0, "dim": 6144, "taps": 4, "bias": True, "silu": True},
        # its backward on packed documents of odd lengths, carried on from earlier rows
        {"name": "conv_grad_docs", "op": "conv", "pass": "backward", "dtype": "bf16",
         "seqs": "6007 1 0 517 2 2048 64 63 1000 4096 129 31 2500", "batch": 1, "packed": True, "resumed": True, "behind": 45,
         "dim": 2304, "taps": 4, "bias": True, "silu": True},
        # the serving batch's next tokens
        {"name": "conv_step_256", "op": "conv", "pass": "step", "dtype": "bf16", "rows": 256, "pool": 320, "padding": 7,
         "dim": 6144, "taps": 4, "bias": True, "silu": True},
        # the hidden states that one 128K call of the In-Place layer takes, added to the residual stream and given out in 8
        # bits with a scale for every 128 columns
        {"name": "norm_128k_e4m3", "op": "norm", "pass": "forward", "dtype": "bf16", "rows": 131072, "dim": 2560,
         "residual": True, "bits8": True, "group": 128},
        # the backward of a few thousand fp32 rows of an odd width, with the residual stream's own gradient
        {"name": "norm_grad_f32", "op": "norm", "pass": "backward", "dtype": "f32", "rows": 4099, "dim": 1001,
         "residual": True, "bits8": False, "group": 0},
    ]


def _log_uniform(rng, low, high):
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def _draw_seqs(rng, total, packed):
    if packed:
        cuts = sorted(rng.randint(0, total) for _ in range(rng.randint(0, 15)))
        return 1, " ".join(str(b - a) for a, b in zip([0] + cuts, cuts + [total]))
    batch = min(total, rng.choice([1, 1, 2, 3, 5]))
    return batch, str(total // batch)


def draw(rng):
    op = rng.choice(["scan", "scan", "scan_grad", "scan_grad", "step", "conv", "conv", "norm", "norm"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    wide = 1 if dtype == "bf16" else 2
    case = {"op": op, "dtype": dtype}
    if op == "norm":
        case["pass"] = rng.choice(["forward", "forward", "backward"])
        dim = rng.choice([_log_uniform(rng, 8, 8192), 8 * _log_uniform(rng, 8, 1024), rng.choice([128, 1024, 2560, 4096])])
        most = NORM_MOST // (dim * wide * (1 if case["pass"] == "forward" else 2))
        bits8 = case["pass"] == "forward" and rng.random() < 0.5
        return {**case, "rows": _log_uniform(rng, 1, min(1 << 19, most)), "dim": dim, "residual": rng.random() < 0.7,
                "bits8": bits8, "group": rng.choice([0, 32, 64, 128]) if bits8 else 0}
    if op == "conv":
        case.update(dim=rng.choice([_log_uniform(rng, 8, 8192), 8 * _log_uniform(rng, 8, 1024)]),
                    taps=rng.choice([4, 4, rng.randint(2, 8)]), bias=rng.random() < 0.7, silu=rng.random() < 0.7)
        case["pass"] = rng.choice(["forward", "backward", "step"])
        if case["pass"] == "step":
            rows = _log_uniform(rng, 1, 512)
            return {**case, "rows": rows, "pool": rows + rng.randint(0, rows), "padding": rng.randint(0, rows // 4)}
        packed = rng.random() < 0.5
        most = CONV_MOST // (case["dim"] * wide * (1 if case["pass"] == "forward" else 4))
        batch, seqs = _draw_seqs(rng, _log_uniform(rng, 1, min(1 << 18, most)), packed)
        return {**case, "batch": batch, "seqs": seqs, "packed": packed, "resumed": rng.random() < 0.5,
                "behind": rng.randint(0, 70) if packed else 0}
    groups, shared = rng.choice([1, 1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 8, 16])
    head_dim = rng.choice([64, 64, 128, 8 * rng.randint(1, 32)])
    state = rng.choice([128, 128, 64, 16, 8 * rng.randint(1, 32)])
    heads = groups * shared
    size = heads * head_dim * state
    case.update(heads=heads, groups=groups, head_dim=head_dim, state=state, skip=rng.random() < 0.7,
                softplus=rng.random() < 0.6)
    if op == "step":
        rows = _log_uniform(rng, 1, max(1, min(512, 256 * 64 * 64 * 128 // size)))
        return {**case, "rows": rows, "pool": rows + rng.randint(0, rows), "padding": rng.randint(0, rows // 4)}
    # fp32 costs more for a token: fewer tokens
    most = (SCAN_MOST if op == "scan" else GRAD_MOST) // size // (1 if dtype == "bf16" else 8)
    packed = rng.random() < 0.5
    batch, seqs = _draw_seqs(rng, _log_uniform(rng, 1, max(1, min(65536 if op == "scan" else 16384, most))), packed)
    return {**case, "batch": batch, "packed": packed, "resumed": rng.random() < 0.5,
            "layout": rng.choice(["token", "head"]), "behind": rng.randint(0, 70) if packed else 0, "seqs": seqs}


# ------------------------------------------------------------------------------------------------------------ inputs


def _slots(case, gen):
    slots = torch.randperm(case["pool"], device="cuda", generator=gen)[:case["rows"]].to(torch.int32)
    slots[case["rows"] - case["padding"]:] = -1
    return slots


def _sequences(case, s):
    """Lengths and packed starts into `s`; the number of sequences."""
    s["lens"] = lens = [int(n) for n in case["seqs"].split()]
    s["starts"] = torch.tensor([0] + lens, device="cuda").cumsum(0).to(torch.int32) if case["packed"] else None
    return len(lens) if case["packed"] else case["batch"]


def _prepare_norm(case, s, normal, dt):
    rows, d = case["rows"], case["dim"]
    s["x"] = normal(rows, d).to(dt)
    s["residual"] = normal(rows, d).mul_(3.0).to(dt) if case["residual"] else None
    s["weight"] = (1 + 0.2 * normal(d)).to(dt)
    if case["pass"] == "backward":
        # what the forward pass has left for it, and the gradient that comes down the residual stream
        s["H"] = s["x"] if s["residual"] is None else (s["x"].float() + s["residual"].float()).to(dt)
        s["rstd"] = (s["H"].float().square().mean(-1) + EPS).rsqrt_()
        s["dY"] = normal(rows, d).to(dt)
        s["dH"] = normal(rows, d).to(dt) if case["residual"] else None


def _prepare_conv(case, s, normal, gen, dt):
    d, K = case["dim"], case["taps"]
    s["w"] = (normal(d, K) * K ** -0.5).to(dt)
    s["bias"] = (0.2 * normal(d)).to(dt) if case["bias"] else None
    if case["pass"] == "step":
        s["x"] = normal(case["rows"], d).to(dt)
        s["halo"] = normal(case["pool"], K - 1, d).to(dt)
        s["slots"] = _slots(case, gen)
        s["live"] = case["rows"] - case["padding"]
        return
    rows = _sequences(case, s)
    n = sum(s["lens"]) + case["behind"]
    s["x"] = normal(case["batch"], n, d).to(dt)
    s["x_init"] = normal(rows, K - 1, d).to(dt) if case["resumed"] else None
    # outputs are the caller's: rows behind the last sequence stay as they are
    s["out"] = torch.zeros_like(s["x"])
    if case["pass"] == "backward":
        s["dY"] = normal(case["batch"], n, d).to(dt)
        s["dx_final"] = normal(rows, K - 1, d).to(dt) if case["resumed"] else None


def prepare(case, seed):
    gen = torch.Generator("cuda")
    gen.manual_seed(seed)
    dt = TYPES[case["dtype"]]
    normal = lambda *z: torch.randn(*z, device="cuda", generator=gen)  # noqa: E731
    uniform = lambda a, b, *z: torch.empty(*z, device="cuda").uniform_(a, b, generator=gen)  # noqa: E731
    s = {"case": case}
    if case["op"] == "norm":
        _prepare_norm(case, s, normal, dt)
        return s
    if case["op"] == "conv":
        _prepare_conv(case, s, normal, gen, dt)
        return s
    H, G, P, N = (case[n] for n in ("heads", "groups", "head_dim", "state"))
    # rates of 0.001 to 0.1 about which the projection's values vary, decays A of -1 to -16
    s["A"] = -uniform(1, 16, H)
    middle = uniform(math.log(1e-3), math.log(1e-1), H).exp()
    s["dt_bias"] = middle.expm1().log() if case["softplus"] else None
    rates = (lambda *z: normal(*z, H)) if case["softplus"] else (lambda *z: middle * normal(*z, H).mul_(0.5).exp_())
    s["D"] = 1 + 0.2 * normal(H) if case["skip"] else None
    if case["op"] == "step":
        R = case["rows"]
        s["x"] = normal(R, H, P).to(dt)
        s["B"], s["C"] = (normal(R, G, N).to(dt) for _ in range(2))
        s["dt"] = rates(R)
        s["S"] = 0.3 * normal(case["pool"], H, P, N)
        s["slots"] = _slots(case, gen)
        s["live"] = R - case["padding"]
        return s
    rows = _sequences(case, s)
    b, n = case["batch"], sum(s["lens"]) + case["behind"]
    # token-major, one row of x, B and C behind one another for each token, as the convolution gives them out
    xbc = normal(b, n, H * P + 2 * G * N).to(dt)
    parts = [t.unflatten(-1, z).transpose(1, 2)
             for t, z in zip(xbc.split([H * P, G * N, G * N], -1), ((H, P), (G, N), (G, N)))]
    s["x"], s["B"], s["C"] = parts if case["layout"] == "token" else [t.contiguous() for t in parts]
    s["dt"] = rates(b, n).transpose(1, 2)
    s["S_init"] = 0.3 * normal(rows, H, P, N) if case["resumed"] else None
    s["O"] = torch.zeros(b, n, H, P, dtype=dt, device="cuda").transpose(1, 2)
    if case["op"] == "scan_grad":
        s["dO"] = normal(b, n, H, P).to(dt).transpose(1, 2)
        s["dS_final"] = 0.1 * normal(rows, H, P, N) if case["resumed"] else None
        s["grads"] = [torch.zeros_like(s[n]) for n in ("x", "dt", "B", "C")]
    return s


# ------------------------------------------------------------------------------------------------- the operators, plain


def _softplus(x):
    return x.clamp(min=0) + torch.log1p(torch.exp(-x.abs()))


def _silu(x):
    return x / (1 + torch.exp(-x))


def _chunks(s):
    """Tokens in chunks that lie within one sequence: each place's token (0 where it has none), whether it has one, and of
    each chunk the sequence that it begins and that it ends, or -1."""
    token, begins, ends, at = [], [], [], 0
    for i, n in enumerate(s["lens"]):
        m = -(-n // CHUNK)
        place = torch.arange(m * CHUNK)
        token.append(torch.where(place < n, place + at, -1))
        begins += [i if c == 0 else -1 for c in range(m)]
        ends += [i if c == m - 1 else -1 for c in range(m)]
        at += n
    token = torch.cat(token).cuda()
    return token.clamp(min=0), token >= 0, begins, ends


def _scan_plain(s, x, dt, A, B, C, D, dt_bias, S_init):
    """O for the tokens of sequences and every sequence's last state, from 32-bit inputs, CHUNK tokens at a time: with b the
    running sum of A r in a chunk, O = (C B^T exp(b_i - b_j)) r x + exp(b) C S + D x, and S moves on by the chunk's
    (r x exp(b_last - b))^T B."""
    case = s["case"]
    shared = case["heads"] // case["groups"]
    token, there, begins, ends = _chunks(s)
    m, rows = len(begins), len(s["lens"]) if case["packed"] else case["batch"]
    r = dt if dt_bias is None else dt + dt_bias[:, None]
    r = _softplus(r) if case["softplus"] else r
    cut = lambda t: torch.where(there[:, None], t[:, :, token], 0).unflatten(2, (m, CHUNK))  # noqa: E731
    skip = 0 if D is None else cut(D[:, None, None] * x)
    u, B, C = cut(r[..., None] * x), cut(B), cut(C)
    b = cut((A[:, None].double() * r)[..., None]).cumsum(-2)  # in 64 bits: differences of sums that grow
    seen = torch.ones(CHUNK, CHUNK, device=x.device).tril().bool()
    decay = torch.where(seen, b - b.mT, -math.inf).exp().float()
    G = (C @ B.mT).repeat_interleave(shared, 1)
    B, C = B.repeat_interleave(shared, 1), C.repeat_interleave(shared, 1)
    O = (G * decay) @ u + skip
    added = (u * (b[..., -1:, :] - b).exp().float()).mT @ B
    last, b = b[..., -1:, :].exp().float(), b.exp().float()
    zero = x.new_zeros(rows, case["heads"], x.shape[3], B.shape[-1]) if S_init is None else S_init
    before, final, S = [], [zero[i:i + 1] for i in range(len(s["lens"]))] if case["packed"] else [zero], zero
    for c in range(m):
        if begins[c] >= 0:
            S = final[begins[c]]
        before.append(S)
        S = last[:, :, c] * S + added[:, :, c]
        if ends[c] >= 0:
            final[ends[c]] = S
    if m:
        O = O + b * (C @ torch.stack(before, 2).mT)
    O = O.flatten(2, 3)[:, :, there]
    return O, torch.cat(final)


def _wide(s, names):
    return [None if s.get(n) is None else s[n].float() for n in names]


def _step_plain(s, dt):
    case, live = s["case"], s["live"]
    x, rate, B, C = (t[:live] for t in _wide(s, ("x", "dt", "B", "C")))
    B, C = (t.repeat_interleave(case["heads"] // case["groups"], 1)[:, :, None] for t in (B, C))
    rate = rate if s["dt_bias"] is None else rate + s["dt_bias"]
    rate = (_softplus(rate) if case["softplus"] else rate)[..., None]
    at = s["slots"][:live].long()
    S = s["S"][at] * (s["A"][:, None] * rate).exp()[..., None] + (rate * x)[..., None] * B
    s["S"][at] = S
    O = torch.zeros_like(s["x"])
    o = (S * C).sum(-1)
    O[:live] = (o if s["D"] is None else o + s["D"][:, None] * x).to(dt)
    return {"O": O, "S": s["S"]}


def _conv_line(s, x, x_init):
    """The rows of every sequence behind its K - 1 earlier ones, sequences one after the other: the line [batch, rows, d],
    and where its tokens, the earlier rows and each sequence's last K - 1 rows lie in it."""
    case, back, lens = s["case"], s["case"]["taps"] - 1, s["lens"]
    count = len(lens) if case["packed"] else case["batch"]
    if x_init is None:
        x_init = x.new_zeros(count, back, x.shape[2])
    if case["packed"]:
        line = torch.cat([t for pair in zip(x_init, x[0, :sum(lens)].split(lens)) for t in pair])[None]
    else:
        line = torch.cat([x_init, x], 1)
    ends = torch.tensor(lens).cumsum(0) + back * torch.arange(1, len(lens) + 1)
    n = torch.tensor(lens)
    tokens = torch.arange(sum(lens)) + torch.repeat_interleave(back * torch.arange(1, len(lens) + 1), n)
    earlier = ((ends - n)[:, None] - back + torch.arange(back)).flatten()
    last = (ends[:, None] - back + torch.arange(back)).flatten()
    return line, tokens.cuda(), earlier.cuda(), last.cuda()


def _taps_plain(s, line, w, bias):
    """The taps' sums for the line's rows from the K-th on."""
    K = s["case"]["taps"]
    z = sum(w[:, j] * line[:, j:line.shape[1] - K + 1 + j] for j in range(K))
    return z if bias is None else z + bias


def _run_conv_plain(s, dt):
    case, K = s["case"], s["case"]["taps"]
    w, bias = _wide(s, ("w", "bias"))
    if case["pass"] == "step":
        live = s["live"]
        at = s["slots"][:live].long()
        line = torch.cat([s["halo"][at], s["x"][:live, None]], 1)
        z = (line.float() * w.mT).sum(1)
        z = z if bias is None else z + bias
        Y = torch.zeros_like(s["x"])
        Y[:live] = (_silu(z) if case["silu"] else z).to(dt)
        s["halo"][at] = line[:, 1:]
        return {"Y": Y, "halo": s["halo"]}
    line, tokens, earlier, last = _conv_line(s, *_wide(s, ("x", "x_init")))
    z = _taps_plain(s, line, w, bias)
    n = sum(s["lens"])
    halo = (len(s["lens"]) if case["packed"] else case["batch"], K - 1, case["dim"])
    if case["pass"] == "forward":
        s["out"][:, :n] = (_silu(z) if case["silu"] else z).to(dt)[:, tokens - (K - 1)]
        return {"Y": s["out"], "x_final": line[:, last].reshape(halo).to(dt)}
    dz = torch.zeros_like(z)
    dz[:, tokens - (K - 1)] = s["dY"][:, :n].float()
    if case["silu"]:
        p = 1 / (1 + torch.exp(-z))
        dz = dz * p * (1 + z * (1 - p))
    dline = torch.zeros_like(line)
    if s["dx_final"] is not None:
        # short sequences' last rows are among their earlier ones, each place once
        dline[:, last] += s["dx_final"].float().reshape(line.shape[0], -1, case["dim"])
    dw = []
    for j in range(K):
        part = slice(j, line.shape[1] - K + 1 + j)
        dline[:, part] += w[:, j] * dz
        dw.append((dz * line[:, part]).sum((0, 1), dtype=torch.float64))  # long sums: in 64 bits
    s["out"][:, :n] = dline[:, tokens].to(dt)
    out = {"dx": s["out"], "dw": torch.stack(dw, -1).float()}
    if case["bias"]:
        out["dbias"] = dz.sum((0, 1), dtype=torch.float64).float()
    if case["resumed"]:
        out["dx_init"] = dline[:, earlier].reshape(halo).to(dt)
    return out


def _run_norm_plain(s, dt):
    case = s["case"]
    w = s["weight"].float()
    if case["pass"] == "backward":
        h, dY, rstd = s["H"].float(), s["dY"].float(), s["rstd"][:, None]
        n, a = h * rstd, dY * w
        dx = rstd * (a - n * (a * n).mean(-1, keepdim=True))
        dx = dx if s["dH"] is None else dx + s["dH"].float()
        return {"dx": dx.to(dt), "dweight": (dY * n).sum(0, dtype=torch.float64).float()}
    H = s["x"] if s["residual"] is None else (s["x"].float() + s["residual"].float()).to(dt)
    h = H.float()
    y = h * (h.square().mean(-1, keepdim=True) + EPS).rsqrt() * w
    out = {} if s["residual"] is None else {"H": H}
    if not case["bits8"]:
        return {**out, "Y": y.to(dt)}
    d, group = case["dim"], case["group"] or case["dim"]
    parts = torch.nn.functional.pad(y, (0, -d % group)).unflatten(-1, (-1, group))
    scale = (parts.abs().amax(-1) / E4M3_MAX).clamp(min=TINY)
    q = (parts / scale[..., None]).flatten(1)[:, :d]
    return {**out, "Y": q.to(torch.float8_e4m3fn), "scale": scale}


def _run_plain(s):
    case = s["case"]
    dt = TYPES[case["dtype"]]
    if case["op"] == "norm":
        return _run_norm_plain(s, dt)
    if case["op"] == "conv":
        return _run_conv_plain(s, dt)
    if case["op"] == "step":
        return _step_plain(s, dt)
    names = ("x", "dt", "A", "B", "C", "D", "dt_bias", "S_init")
    args = _wide(s, names)
    if case["op"] == "scan":
        O, S = _scan_plain(s, *args)
        s["O"][:, :, :O.shape[2]] = O.to(dt)
        return {"O": s["O"], "S_final": S}
    args = [None if t is None else t.detach().requires_grad_() for t in args]
    with torch.enable_grad():
        O, S = _scan_plain(s, *args)
        loss = (O * s["dO"][:, :, :O.shape[2]].float()).sum()
        if s["dS_final"] is not None:
            loss = loss + (S * s["dS_final"]).sum()
    d = torch.autograd.grad(loss, [t for t in args if t is not None])
    d = dict(zip([n for n, t in zip(names, args) if t is not None], d))
    for out, n in zip(s["grads"], ("x", "dt", "B", "C")):
        out.copy_(d[n])
    return {**dict(zip(("dx", "ddt", "dB", "dC"), s["grads"])),
            **{"d" + n: d[n] for n in ("A", "D", "dt_bias", "S_init") if n in d}}


def run(state):
    if not own:
        return _run_plain(state)
    import chunk_wise_weight_amd as cw

    s, case = state, state["case"]
    op = case["op"]
    if op == "norm":
        if case["pass"] == "backward":
            dx, dweight = cw.ttt_rms_norm_backward(s["H"], s["weight"], s["dY"], s["rstd"], dH=s["dH"])
            return {"dx": dx, "dweight": dweight}
        Y, H, _, scale = cw.ttt_rms_norm(s["x"], s["weight"], s["residual"], eps=EPS,
                                         out_dtype=torch.float8_e4m3fn if case["bits8"] else None, group=case["group"] or None)
        return {**({"H": H} if case["residual"] else {}), "Y": Y, **({"scale": scale} if case["bits8"] else {})}
    if op == "conv":
        if case["pass"] == "step":
            Y = cw.ttt_short_conv_step(s["x"], s["w"], s["halo"], s["bias"], silu=case["silu"], slots=s["slots"])
            return {"Y": Y, "halo": s["halo"]}
        if case["pass"] == "forward":
            Y, final = cw.ttt_short_conv(s["x"], s["w"], s["bias"], silu=case["silu"], x_init=s["x_init"],
                                         seq_starts=s["starts"], Y=s["out"])
            return {"Y": Y, "x_final": final}
        dx, dw, dbias, dx_init = cw.ttt_short_conv_backward(
            s["x"], s["w"], s["dY"], s["bias"], silu=case["silu"], x_init=s["x_init"], seq_starts=s["starts"],
            dx_final=s["dx_final"], dx=s["out"])
        return {"dx": dx, "dw": dw, **({"dbias": dbias} if case["bias"] else {}),
                **({"dx_init": dx_init} if case["resumed"] else {})}
    args = [s[n] for n in ("x", "dt", "A", "B", "C")]
    more = {"D": s["D"], "dt_bias": s["dt_bias"], "softplus": case["softplus"]}
    if op == "step":
        return {"O": cw.ttt_selective_scan_step(*args, s["S"], slots=s["slots"], **more), "S": s["S"]}
    more.update(S_init=s["S_init"], seq_starts=s["starts"])
    if op == "scan":
        O, S = cw.ttt_selective_scan(*args, O=s["O"], **more)
        return {"O": O, "S_final": S}
    dx, ddt, dB, dC = s["grads"]
    d = cw.ttt_selective_scan_backward(*args, s["dO"], dS_final=s["dS_final"], dx=dx, ddt=ddt, dB=dB, dC=dC, **more)
    names = ("dx", "ddt", "dA", "dB", "dC", "dD", "ddt_bias", "dS_init")
    d = dict(zip(names, d))
    return {n: d[n] for n in ("dx", "ddt", "dB", "dC", "dA", "dD", "ddt_bias", "dS_init") if d[n] is not None}


# --------------------------------------------------------------------------------------------------------- work, exact


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "norm":
        rows, d, more = case["rows"], case["dim"], case["residual"]
        if case["pass"] == "backward":  # h, dY, perhaps the residual stream's gradient; dx, dweight
            return {"bytes": rows * d * e * (4 if more else 3) + 4 * rows + d * (e + 4), "flops": 9 * rows * d}
        out = rows * d + 4 * rows * -(-d // (case["group"] or d)) if case["bits8"] else rows * d * e
        return {"bytes": rows * d * e * (3 if more else 1) + out + d * e, "flops": 5 * rows * d}
    if case["op"] == "conv":
        d, K = case["dim"], case["taps"]
        taps = d * (K + (1 if case["bias"] else 0))
        if case["pass"] == "step":
            R, live = case["rows"], case["rows"] - case["padding"]
            return {"bytes": (R * d + live * d * (2 * (K - 1) + 1) + taps) * e + 4 * R, "flops": live * d * (2 * K + 4)}
        lens = [int(n) for n in case["seqs"].split()]
        n = sum(lens) * case["batch"]
        halo = (len(lens) if case["packed"] else case["batch"]) * (K - 1) * d * e
        if case["pass"] == "forward":
            return {"bytes": 2 * n * d * e + halo * (2 if case["resumed"] else 1) + taps * e, "flops": n * d * (2 * K + 4)}
        return {"bytes": 3 * n * d * e + (3 * halo if case["resumed"] else 0) + taps * (e + 4), "flops": n * d * (6 * K + 8)}
    H, G, P, N = (case[n] for n in ("heads", "groups", "head_dim", "state"))
    size = H * P * N
    token = (H * P + 2 * G * N) * e + 4 * H
    if case["op"] == "step":
        live = case["rows"] - case["padding"]
        return {"bytes": case["rows"] * (H * P * e + 4) + live * (token + 8 * size), "flops": 6 * live * size}
    lens = [int(n) for n in case["seqs"].split()]
    n = sum(lens) * case["batch"]
    states = 4 * (len(lens) if case["packed"] else case["batch"]) * size
    if case["op"] == "scan":
        return {"bytes": n * (token + H * P * e) + states * (2 if case["resumed"] else 1), "flops": 5 * n * size}
    # the states again, then the gradients' recurrence and the products of it with x, B and C
    return {"bytes": n * (2 * token + H * P * e) + (3 * states if case["resumed"] else 0), "flops": 13 * n * size}


def _tokens(s, grad):
    """The scan's recurrence itself, token by token in 64 bits; with `grad` its reverse too."""
    case = s["case"]
    shared, soft = case["heads"] // case["groups"], case["softplus"]
    x, raw, A, B, C = (s[n].double() for n in ("x", "dt", "A", "B", "C"))
    D = torch.zeros_like(A) if s["D"] is None else s["D"].double()
    raw = raw if s["dt_bias"] is None else raw + s["dt_bias"].double()[:, None]
    # log(1 + exp(raw)), from the side on which exp stays small
    r = torch.where(raw > 0, raw + torch.log1p(torch.exp(-raw)), torch.log1p(torch.exp(raw))) if soft else raw
    a = torch.exp(A[:, None] * r)
    B, C = (t.unsqueeze(2).expand(-1, -1, shared, -1, -1).flatten(1, 2) for t in (B, C))
    O = torch.zeros_like(x)
    dx, dB, dC, dr, da = (torch.zeros_like(t) for t in (x, B, C, r, a))
    dO = s["dO"].double() if grad else None
    lens = s["lens"]
    rows = len(lens) if case["packed"] else case["batch"]
    first = x.new_zeros(rows, x.shape[1], x.shape[3], B.shape[3]) if s["S_init"] is None else s["S_init"].double()
    finals, dfirst, dD, at = [], [], torch.zeros_like(D), 0
    for i, n in enumerate(lens):
        S = (first[i:i + 1] if case["packed"] else first).clone()

        def one(S, t):
            return S * a[:, :, t, None, None] + (r[:, :, t, None] * x[:, :, t])[..., None] * B[:, :, t, None]

        kept = []
        for t in range(at, at + n):
            if grad and (t - at) % 64 == 0:
                kept.append(S)
            S = one(S, t)
            if not grad:
                O[:, :, t] = (S @ C[:, :, t, :, None])[..., 0] + D[:, None] * x[:, :, t]
        finals.append(S)
        if grad:
            dS = torch.zeros_like(first) if s["dS_final"] is None else s["dS_final"].double()
            dS = (dS[i:i + 1] if case["packed"] else dS).clone()
            for c in range(len(kept) - 1, -1, -1):
                steps, S = [], kept[c]
                for t in range(at + 64 * c, at + min(n, 64 * c + 64)):
                    new = one(S, t)
                    steps.append((t, S, new))
                    S = new
                for t, old, new in reversed(steps):
                    o = dO[:, :, t]
                    dC[:, :, t] = (new * o[..., None]).sum(-2)
                    dS = dS + o[..., None] * C[:, :, t, None]
                    du = (dS * B[:, :, t, None]).sum(-1)
                    dB[:, :, t] = (dS * (r[:, :, t, None] * x[:, :, t])[..., None]).sum(-2)
                    dx[:, :, t] = r[:, :, t, None] * du + D[:, None] * o
                    dr[:, :, t] = (du * x[:, :, t]).sum(-1)
                    da[:, :, t] = (dS * old).sum((-1, -2))
                    dD += (o * x[:, :, t]).sum((0, 2))
                    dS = a[:, :, t, None, None] * dS
            dfirst.append(dS)
        at += n
    if not grad:
        return {"O": O, "S_final": torch.cat(finals)}
    dlog = da * a
    dr = dr + dlog * A[:, None]
    draw_ = dr * torch.sigmoid(raw) if soft else dr
    dB, dC = (t.unflatten(1, (-1, shared)).sum(2) for t in (dB, dC))
    out = {"dx": dx, "ddt": draw_, "dB": dB, "dC": dC, "dA": (dlog * r).sum((0, 2))}
    if s["D"] is not None:
        out["dD"] = dD
    if s["dt_bias"] is not None:
        out["ddt_bias"] = draw_.sum((0, 2))
    if s["S_init"] is not None:
        out["dS_init"] = torch.cat(dfirst)
    return out


def _exact_conv(s):
    case, K = s["case"], s["case"]["taps"]
    w = s["w"].double()
    bias = torch.zeros_like(w[:, 0]) if s["bias"] is None else s["bias"].double()

    def act(z):
        return z * torch.sigmoid(z) if case["silu"] else z

    if case["pass"] == "step":
        Y, halo = torch.zeros_like(s["x"], dtype=torch.float64), s["halo"].double()
        for row, slot in enumerate(s["slots"].tolist()):
            if slot >= 0:
                line = torch.cat([halo[slot], s["x"][row:row + 1].double()])
                Y[row] = act(bias + torch.einsum("kd,dk->d", line, w))
                halo[slot] = line[1:]
        return {"Y": Y, "halo": halo}
    x, lens = s["x"].double(), s["lens"]
    grad = case["pass"] == "backward"
    out, dw, dbias = torch.zeros_like(x), torch.zeros_like(w), torch.zeros_like(bias)
    edges, at = [], 0
    for i, n in enumerate(lens):
        mine = slice(i, i + 1) if case["packed"] else slice(None)
        count = 1 if case["packed"] else case["batch"]
        old = x.new_zeros(count, K - 1, x.shape[2]) if s["x_init"] is None else s["x_init"][mine].double()
        line = torch.cat([old, x[:, at:at + n]], 1)
        z = bias.expand(count, n, -1).clone()
        for j in range(K):
            z += line[:, j:j + n] * w[:, j]
        if not grad:
            out[:, at:at + n] = act(z)
            edges.append(line[:, n:])
        else:
            g = s["dY"][:, at:at + n].double()
            if case["silu"]:
                p = torch.sigmoid(z)
                g = g * (p + z * p * (1 - p))
            dline = torch.zeros_like(line)
            if s["dx_final"] is not None:
                dline[:, n:] += s["dx_final"][mine].double()
            for j in range(K):
                dline[:, j:j + n] += g * w[:, j]
                dw[:, j] += (g * line[:, j:j + n]).sum((0, 1))
            dbias += g.sum((0, 1))
            out[:, at:at + n] = dline[:, K - 1:]
            edges.append(dline[:, :K - 1])
        at += n
    if not grad:
        return {"Y": out, "x_final": torch.cat(edges)}
    return {"dx": out, "dw": dw, **({"dbias": dbias} if case["bias"] else {}),
            **({"dx_init": torch.cat(edges)} if case["resumed"] else {})}


def _exact_norm(s):
    case, d = s["case"], s["case"]["dim"]
    w = s["weight"].double()
    if case["pass"] == "backward":
        # from the inverse root that the forward pass left, as the operator's definition takes it
        h, r, dY = s["H"].double(), s["rstd"].double()[:, None], s["dY"].double()
        a = dY * w
        dx = r * a - h * r ** 3 * ((a * h).sum(-1, keepdim=True) / d)
        return {"dx": dx if s["dH"] is None else dx + s["dH"].double(), "dweight": (dY * h * r).sum(0)}
    H = s["x"].double() if s["residual"] is None else s["x"].double() + s["residual"].double()
    h = H.to(s["x"].dtype).double()  # the norm is of the sum as it is kept
    y = h / torch.sqrt((h * h).sum(-1, keepdim=True) / d + EPS) * w
    out = {} if s["residual"] is None else {"H": H}
    if not case["bits8"]:
        return {**out, "Y": y}
    # the scaled values before their rounding to 8 bits
    group = case["group"] or d
    scale = torch.stack([p.abs().amax(-1) for p in y.split(group, -1)], -1) / E4M3_MAX
    scale = torch.clamp(scale, min=TINY)
    return {**out, "Y": y / scale.repeat_interleave(group, -1)[:, :d], "scale": scale}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        return _exact_norm(s)
    if case["op"] == "conv":
        return _exact_conv(s)
    if case["op"] == "step":
        x, raw, A, B, C, S = (s[n].double() for n in ("x", "dt", "A", "B", "C", "S"))
        D = torch.zeros_like(A) if s["D"] is None else s["D"].double()
        raw = raw if s["dt_bias"] is None else raw + s["dt_bias"].double()
        r = torch.where(raw > 0, raw + torch.log1p(torch.exp(-raw)), torch.log1p(torch.exp(raw))) if case["softplus"] else raw
        O, shared = torch.zeros_like(x), case["heads"] // case["groups"]
        for row, slot in enumerate(s["slots"].tolist()):
            if slot < 0:
                continue
            b, c = (t[row].repeat_interleave(shared, 0) for t in (B, C))
            S[slot] = S[slot] * torch.exp(A * r[row])[:, None, None] + torch.einsum("h,hp,hn->hpn", r[row], x[row], b)
            O[row] = torch.einsum("hpn,hn->hp", S[slot], c) + D[:, None] * x[row]
        return {"O": O, "S": S}
    tokens = sum(int(n) for n in case["seqs"].split())
    if tokens * (1 if case["op"] == "scan" else 8) > 70000:
        return None  # about 20 seconds
    return _tokens(s, case["op"] == "scan_grad")
