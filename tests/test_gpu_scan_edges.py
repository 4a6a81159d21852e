"""The state-space layer's operators (RMS norm, short convolution, selective scan) run together, captured, on several
streams at once, at large offsets and sizes.

Where a call is compared with another call of the same operator the bits have to be the same: rows, channels, sequences
and heads are worked out alike wherever they lie.  The layer as a whole, in fp32: a stage's output is off by at most 320 *
2^-24 relative (a sum of at most 256 + 64 terms), the stages behind it multiply a relative error by at most 4 (a norm
divides by a row's own length, SiLU's slope is at most 1.1, the scan is linear in x, B and C, at most their product), and
there are 4 stages one behind the other: 4 * 4 * 320 * 2^-24 = 3.1e-4.  A gradient passes them forward and back: twice that.
"""
import numpy as np
import pytest
import torch

import chunk_wise_weight_amd as cw
from oracle import scan as osc
from tests.test_gpu_scan import f64, make, rel

pytestmark = pytest.mark.gpu

DTYPES = [torch.float32, torch.bfloat16]
TOL_LAYER = 16 * 320 * 2.0 ** -24


class Layer:
    """h, y = norm(x + residual); x, B, C = conv(y W_in); o = scan; norm(o) W_out."""

    def __init__(self, d=96, H=4, G=2, P=24, N=16, K=4, seed=1):
        gen = torch.Generator().manual_seed(seed)
        r = lambda *s: torch.randn(*s, generator=gen)
        self.sizes = d, H, G, P, N, K
        width = H * P + 2 * G * N
        self.w1, self.w2 = 1 + 0.2 * r(d), 1 + 0.2 * r(H * P)
        self.W_in, self.W_dt = r(d, width) * d ** -0.5, r(d, H) * d ** -0.5
        self.cw, self.cb = r(width, K) * K ** -0.5, 0.2 * r(width)
        self.A, self.D, self.bias = -(0.05 + 3 * torch.rand(H, generator=gen) ** 2), r(H), r(H) - 1
        self.gpu = {k: v.cuda() for k, v in vars(self).items() if isinstance(v, torch.Tensor)}

    def split(self, z):
        d, H, G, P, N, K = self.sizes
        x, B, C = z.split([H * P, G * N, G * N], -1)
        heads = lambda t, h: t.unflatten(-1, (h, -1)).transpose(-3, -2)
        return heads(x, H), heads(B, G), heads(C, G)

    def prompt(self, x, res):
        g = self.gpu
        y, h, rstd, _ = cw.ttt_rms_norm(x, g["w1"], residual=res)
        z = y @ g["W_in"]
        dt = (y @ g["W_dt"]).transpose(1, 2)
        xbc, halo = cw.ttt_short_conv(z, g["cw"], g["cb"])
        xs, B, C = self.split(xbc)
        O, S = cw.ttt_selective_scan(xs, dt, g["A"], B, C, D=g["D"], dt_bias=g["bias"], softplus=True)
        o = O.transpose(1, 2).flatten(2)
        out, _, rstd2, _ = cw.ttt_rms_norm(o, g["w2"])
        return out, (halo, S), (y, h, rstd, z, dt, xs, B, C, o, rstd2)

    def token(self, x, res, state, slots):
        g, (d, H, G, P, N, K) = self.gpu, self.sizes
        halo, S = state
        y, h, _, _ = cw.ttt_rms_norm(x, g["w1"], residual=res)
        xbc = cw.ttt_short_conv_step(y @ g["W_in"], g["cw"], halo, g["cb"], slots=slots)
        xs, B, C = xbc.split([H * P, G * N, G * N], -1)
        o = cw.ttt_selective_scan_step(xs.unflatten(-1, (H, P)).contiguous(), y @ g["W_dt"], g["A"],
                                       B.unflatten(-1, (G, N)).contiguous(), C.unflatten(-1, (G, N)).contiguous(), S,
                                       D=g["D"], dt_bias=g["bias"], softplus=True, slots=slots)
        return cw.ttt_rms_norm(o.flatten(1), g["w2"])[0]

    def backward(self, x, kept, dout):
        """dx (and the residual's) and the weights' gradients of the layer."""
        g = self.gpu
        y, h, rstd, z, dt, xs, B, C, o, rstd2 = kept
        do, dw2 = cw.ttt_rms_norm_backward(o, g["w2"], dout, rstd2)
        dO = do.unflatten(-1, (self.sizes[1], -1)).transpose(1, 2)
        dxbc = torch.empty_like(z)
        dxs, dB, dC = self.split(dxbc)
        _, ddt, dA, _, _, dD, dbias, _ = cw.ttt_selective_scan_backward(
            xs, dt, g["A"], B, C, dO, D=g["D"], dt_bias=g["bias"], softplus=True, dx=dxs, dB=dB, dC=dC)
        dz, dcw, dcb, _ = cw.ttt_short_conv_backward(z, g["cw"], dxbc, g["cb"])
        ddt = ddt.transpose(1, 2)
        dy = dz @ g["W_in"].T + ddt @ g["W_dt"].T
        dx, dw1 = cw.ttt_rms_norm_backward(h, g["w1"], dy.contiguous(), rstd, dH=None)
        return dict(x=dx, w1=dw1, w2=dw2, cw=dcw, cb=dcb, A=dA, D=dD, bias=dbias)

    def plain(self, x, res, p):
        """The formulas token by token, of one sequence, in fp64 with autograd."""
        d, H, G, P, N, K = self.sizes
        norm = lambda v, w: v * (v.square().mean(-1, keepdim=True) + 1e-5).rsqrt() * w
        y = norm(x + res, p["w1"])
        z, dt = y @ self.W_in.double(), y @ self.W_dt.double()
        r = torch.nn.functional.softplus(dt + p["bias"])
        zp = torch.cat([z.new_zeros(K - 1, z.shape[1]), z])
        xbc = torch.nn.functional.silu(sum(zp[j:j + len(z)] * p["cw"][:, j] for j in range(K)) + p["cb"])
        xs, B, C = self.split(xbc)
        B, C = B.repeat_interleave(H // G, 0), C.repeat_interleave(H // G, 0)
        S, out = z.new_zeros(H, P, N), []
        for t in range(len(x)):
            S = (p["A"] * r[t]).exp()[:, None, None] * S + r[t][:, None, None] * xs[:, t, :, None] * B[:, t, None, :]
            out.append((S * C[:, t, None, :]).sum(-1) + p["D"][:, None] * xs[:, t])
        return norm(torch.stack(out).flatten(1), p["w2"])


def inputs(n, B=2, d=96, seed=3):
    gen = torch.Generator().manual_seed(seed)
    return torch.randn(B, n, d, generator=gen), torch.randn(B, n, d, generator=gen)


def test_a_prompt_then_tokens():
    layer, (n, more) = Layer(), (100, 7)
    x, res = inputs(n + more)
    out, state, _ = layer.prompt(x[:, :n].contiguous().cuda(), res[:, :n].contiguous().cuda())
    p = {k: getattr(layer, k).double() for k in ("w1", "w2", "cw", "cb", "A", "D", "bias")}
    want = torch.stack([layer.plain(x[b].double(), res[b].double(), p) for b in range(2)])
    print("prompt", rel(out, want[:, :n].numpy()), flush=True)
    assert rel(out, want[:, :n].numpy()) <= TOL_LAYER
    # into pools of 5 states each, in another order, and a padding row
    slots = torch.tensor([3, -1, 0], dtype=torch.int32, device="cuda")
    pools = [torch.randn(5, *t.shape[1:], device="cuda", generator=torch.Generator("cuda").manual_seed(1)) for t in state]
    for pool, t in zip(pools, state):
        pool[[3, 0]] = t
    kept = [pool[[1, 2, 4]].clone() for pool in pools]
    for t in range(n, n + more):
        rows = lambda v: torch.stack([v[0, t], torch.ones_like(v[0, t]), v[1, t]]).cuda()
        o = layer.token(rows(x), rows(res), pools, slots)
        assert rel(o[[0, 2]], want[:, t].numpy()) <= TOL_LAYER, t
        assert (o[1] == 0).all()
    assert all(torch.equal(pool[[1, 2, 4]], k) for pool, k in zip(pools, kept))
    # the same state as that of the longer prompt
    _, long, _ = layer.prompt(x.cuda(), res.cuda())
    assert all(rel(pool[[3, 0]], f64(t)) <= TOL_LAYER for pool, t in zip(pools, long))


def test_the_layer_gradients():
    layer = Layer()
    x, res = inputs(90)
    dout = torch.randn(2, 90, 96, generator=torch.Generator().manual_seed(4))
    out, _, kept = layer.prompt(x.cuda(), res.cuda())
    got = layer.backward(x.cuda(), kept, dout.cuda())
    p = {k: getattr(layer, k).double().requires_grad_() for k in ("w1", "w2", "cw", "cb", "A", "D", "bias")}
    xd = x.double().requires_grad_()
    loss = sum((layer.plain(xd[b], res[b].double(), p) * dout[b].double()).sum() for b in range(2))
    loss.backward()
    for k, t in {**p, "x": xd}.items():
        print("d" + k, rel(got[k], t.grad.numpy()), flush=True)
        assert rel(got[k], t.grad.numpy()) <= 2 * TOL_LAYER, k
    # and against a difference along a direction: 1e-6 is balanced between its square (1e-12) and fp64's 2e-16 / 1e-6
    u, eps = torch.randn(x.shape, generator=torch.Generator().manual_seed(5), dtype=torch.float64), 1e-6
    with torch.no_grad():
        q = {k: v.detach() for k, v in p.items()}
        at = lambda e: sum((layer.plain(x[b].double() + e * u[b], res[b].double(), q) * dout[b].double()).sum() for b in range(2))
        diff = float(at(eps) - at(-eps)) / (2 * eps)
    along = float((got["x"].double().cpu() * u).sum())
    scale = float(got["x"].double().norm().cpu() * u.norm())
    assert abs(along - diff) <= 2 * TOL_LAYER * scale


def calls(kind, dtype, seed=0):
    """A call of one entry point, and the tensors that it changes in place."""
    gen = torch.Generator("cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, device="cuda", generator=gen)
    if kind.startswith("scan"):
        n = 1300
        *args, D, bias = make(1, 4, 2, n, 64, 64, dtype, seed=seed)
        more = dict(D=D, dt_bias=bias, softplus=True)
        if "step" in kind:
            S, slots = r(9, 4, 64, 64), torch.tensor([4, 0, -1, 7, 4], dtype=torch.int32, device="cuda")
            x, dt, A, B, C = args
            row = lambda t: t[0].transpose(0, 1)[:5].contiguous()
            a = (row(x), row(dt), A, row(B), row(C))
            return lambda: (cw.ttt_selective_scan_step(*a, S, slots=slots, **more),), [S]
        if "packed" in kind:
            more["seq_starts"] = torch.tensor([0, 700, 700, 701, 1300], dtype=torch.int32, device="cuda")
        more["S_init"] = r(4 if "packed" in kind else 1, 4, 64, 64)
        if "backward" in kind:
            dO, dS = r(*args[0].shape).to(dtype), r(*more["S_init"].shape)
            return lambda: cw.ttt_selective_scan_backward(*args, dO, dS_final=dS, **more), []
        return lambda: cw.ttt_selective_scan(*args, **more), []
    if kind.startswith("conv"):
        d, K = 200, 4
        w, b = r(d, K).to(dtype), r(d).to(dtype)
        if "step" in kind:
            halo, slots = r(9, K - 1, d).to(dtype), torch.tensor([4, 0, -1, 7, 4], dtype=torch.int32, device="cuda")
            x = r(5, d).to(dtype)
            return lambda: (cw.ttt_short_conv_step(x, w, halo, b, slots=slots),), [halo]
        x, x0, dY = r(2, 333, d).to(dtype), r(2, K - 1, d).to(dtype), r(2, 333, d).to(dtype)
        if "backward" in kind:
            return lambda: cw.ttt_short_conv_backward(x, w, dY, b, x_init=x0, dx_final=x0), []
        return lambda: cw.ttt_short_conv(x, w, b, x_init=x0), []
    x, res, w = r(77, 1000).to(dtype), r(77, 1000).to(dtype), r(1000).to(dtype)
    if "backward" in kind:
        rstd = r(77).abs()
        return lambda: cw.ttt_rms_norm_backward(x, w, res, rstd, dH=res), []
    if "8" in kind:
        return lambda: cw.ttt_rms_norm(x, w, residual=res, out_dtype=torch.float8_e4m3fn, group=64), []
    return lambda: cw.ttt_rms_norm(x, w, residual=res)[:3], []


KINDS = ["scan", "scan_packed", "scan_backward", "scan_packed_backward", "scan_step", "conv", "conv_backward", "conv_step",
         "rms", "rms8", "rms_backward"]


def bits(t):
    return t.contiguous().view(torch.uint8)


def same(a, b):
    return all((s is None and t is None) or torch.equal(bits(s), bits(t)) for s, t in zip(a, b, strict=True))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("kind", KINDS)
def test_replays_match_eager(kind, dtype):
    print("graph", kind, dtype, flush=True)
    call, changed = calls(kind, dtype)
    start = [t.clone() for t in changed]

    def reset():
        for t, s in zip(changed, start):
            t.copy_(s)
        torch.cuda.synchronize()

    eager = [*(t.clone() if t is not None else None for t in call()), *(t.clone() for t in changed)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    reset()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    for r in range(3):
        reset()
        for t in out:
            if t is not None:
                bits(t).fill_(255) if t.is_contiguous() else t.fill_(float("nan"))
        again = call()
        torch.cuda.synchronize()
        assert same([*again, *changed], eager), r
        reset()
        graph.replay()
        torch.cuda.synchronize()
        assert same([*out, *changed], eager), r


@pytest.mark.parametrize("kind", KINDS)
def test_two_streams_at_once(kind):
    """Calls on their own tensors on two streams, several of each under way: the bits of each alone."""
    print("streams", kind, flush=True)
    both = [calls(kind, torch.bfloat16, seed) for seed in (1, 2)]
    alone = []
    for call, changed in both:
        start = [t.clone() for t in changed]
        alone.append([*call(), *(t.clone() for t in changed)])
        for t, s in zip(changed, start):
            t.copy_(s)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in both]
    out = [None, None]
    for turn in range(1 if both[0][1] else 4):
        for i, ((call, _), s) in enumerate(zip(both, streams)):
            with torch.cuda.stream(s):
                out[i] = call()
    torch.cuda.synchronize()
    for (_, changed), got, want in zip(both, out, alone):
        assert same([*got, *changed], want)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("starts", [[-5, 40, 30, 900, 20, 2000], [2000, 1000, 0, -1], [0, 130, 131, 64, 700]])
def test_starts_outside_the_row_do_not_lead_out_of_it(starts, dtype):
    """Starts of any values: what lies outside the row is neither read (it is not finite) nor written."""
    print("starts", starts, dtype, flush=True)
    n, H, G, P, N = 700, 2, 1, 64, 64
    *args, D, bias = make(1, H, G, n + 128, P, N, dtype)
    for t in (args[0], args[1], args[3], args[4]):
        t[:, :, :64] = t[:, :, n + 64:] = float("nan")
    view = lambda t: t[:, :, 64:n + 64]
    x, dt, A, B, C = (view(t) if t.dim() > 1 else t for t in args)
    st = torch.tensor(starts, dtype=torch.int32, device="cuda")
    num = len(starts) - 1
    whole = torch.full_like(args[0], 3.0)
    _, S = cw.ttt_selective_scan(x, dt, A, B, C, D=D, dt_bias=bias, softplus=True, seq_starts=st, O=view(whole))
    assert (whole[:, :, :64] == 3).all() and (whole[:, :, n + 64:] == 3).all()
    assert S.shape[0] == num and torch.isfinite(S).all() and torch.isfinite(view(whole)).all()
    full = [torch.full_like(t, 3.0) for t in args]
    dx, ddt, _, dB, dC = (view(t) if t.dim() > 1 else t for t in full)
    cw.ttt_selective_scan_backward(x, dt, A, B, C, torch.ones_like(x), D=D, dt_bias=bias, softplus=True, seq_starts=st, dx=dx,
                                   ddt=ddt, dB=dB, dC=dC)
    for t in (full[0], full[1], full[3], full[4]):
        assert (t[:, :, :64] == 3).all() and (t[:, :, n + 64:] == 3).all()


@pytest.mark.parametrize("dtype", DTYPES)
def test_what_is_not_finite_stays_in_its_sequence_and_head(dtype):
    n, H, G, P, N = 900, 4, 2, 64, 64
    *args, D, bias = make(1, H, G, n, P, N, dtype)
    starts = torch.tensor([0, 290, 610, n], dtype=torch.int32, device="cuda")
    dO = torch.randn(args[0].shape, device="cuda").to(dtype)
    more = dict(D=D, dt_bias=bias, softplus=True, seq_starts=starts)
    O, S = cw.ttt_selective_scan(*args, **more)
    grads = cw.ttt_selective_scan_backward(*args, dO, **more)
    for value in (float("nan"), float("inf")):
        x = args[0].clone()
        x[0, 1, 400] = value                               # head 1 of group 0, sequence 1
        O2, S2 = cw.ttt_selective_scan(x, *args[1:], **more)
        g2 = cw.ttt_selective_scan_backward(x, *args[1:], dO, **more)
        assert not torch.isfinite(O2[0, 1, 400]).all()
        O2[0, 1, 290:610], S2[1, 1] = O[0, 1, 290:610], S[1, 1]
        assert torch.equal(O2, O) and torch.equal(S2, S)
        for i, heads in ((0, [0, 1]), (1, [0, 1]), (3, [0]), (4, [0])):      # dx, ddt, dB, dC
            for h in heads:
                g2[i][0, h, 290:610] = grads[i][0, h, 290:610]
            assert torch.equal(g2[i], grads[i]), i


def test_offsets_past_32_bits():
    """Elements past 2^31 and bytes past 2^32: the bits of the same rows in small tensors."""
    gen = torch.Generator("cuda").manual_seed(1)
    r = lambda *s: torch.randn(*s, device="cuda", generator=gen)
    # a pool of 150,000 states of 32 KB
    S = torch.empty(150_000, 1, 64, 128, device="cuda")
    slots = torch.tensor([149_999, 0, 140_001], dtype=torch.int32, device="cuda")
    few = r(3, 1, 64, 128)
    S[slots.long()] = few
    x, dt, A, B, C = r(3, 1, 64), r(3, 1).abs(), -r(1).abs(), r(3, 1, 128), r(3, 1, 128)
    O = cw.ttt_selective_scan_step(x, dt, A, B, C, S, slots=slots)
    O2 = cw.ttt_selective_scan_step(x, dt, A, B, C, few)
    assert torch.equal(O, O2) and torch.equal(S[slots.long()], few)
    del S
    # sequences and heads 2^31 and more elements apart
    *args, D, bias = make(2, 2, 1, 300, 64, 128, torch.bfloat16, layout="head")
    x = args[0]
    big = torch.empty((1 << 32) + (1 << 21), dtype=torch.bfloat16, device="cuda")
    far = big.as_strided(x.shape, ((1 << 31) + 64, 1 << 30, 64, 1))
    far.copy_(x)
    out = torch.empty_like(big)
    Of = out.as_strided(x.shape, far.stride())
    more = dict(D=D, dt_bias=bias, softplus=True)
    want, Sw = cw.ttt_selective_scan(x, *args[1:], **more)
    _, Sf = cw.ttt_selective_scan(far, *args[1:], O=Of, **more)
    assert torch.equal(Of, want) and torch.equal(Sf, Sw)
    dO = torch.randn(x.shape, device="cuda").to(x.dtype)
    w = cw.ttt_selective_scan_backward(x, *args[1:], dO, **more)
    g = cw.ttt_selective_scan_backward(far, *args[1:], dO, dx=Of, **more)
    assert all(torch.equal(a, b) for a, b in zip(g, w) if a is not None)
    # rows of a convolution 2^31 elements apart
    t = r(2, 2, 256).to(torch.bfloat16)
    cwt = r(256, 4).to(torch.bfloat16)
    far, Yf = (b.as_strided(t.shape, (512, (1 << 31), 1)) for b in (big, out))
    far.copy_(t)
    want, last = cw.ttt_short_conv(t, cwt)
    _, lf = cw.ttt_short_conv(far, cwt, Y=Yf)
    assert torch.equal(Yf, want) and torch.equal(lf, last)
    # the last rows of a norm past 2^32 elements
    d = 4096
    x = big[:(1 << 32) + (1 << 18)].view(-1, d)
    x.zero_()
    x[-70:] = r(70, d).to(x.dtype)
    Y, _, rstd, _ = cw.ttt_rms_norm(x, Y=out[:x.numel()].view(-1, d))
    want = cw.ttt_rms_norm(x[-70:].contiguous())
    assert torch.equal(Y[-70:], want[0]) and torch.equal(rstd[-70:], want[2])


@pytest.mark.parametrize("dtype", DTYPES)
def test_large_calls_are_their_pieces(dtype):
    """Operands of more than 256 MiB pass by the caches: the bits of calls on pieces that do not."""
    gen = torch.Generator("cuda").manual_seed(1)
    r = lambda *s: torch.randn(*s, device="cuda", generator=gen)
    wide = 2 if dtype == torch.float32 else 1
    print("large", dtype, flush=True)
    rows, d = 40_000 // wide, 1536
    x, res, w = r(rows, d).to(dtype), r(rows, d).to(dtype), r(d).to(dtype)
    for more in (dict(), dict(out_dtype=torch.float8_e4m3fn, group=128), dict(out_dtype=torch.float8_e4m3fn)):
        got = cw.ttt_rms_norm(x, w, residual=res, **more)
        for part in range(4):
            cut = slice(part * rows // 4, (part + 1) * rows // 4)
            want = cw.ttt_rms_norm(x[cut], w, residual=res[cut], **more)
            assert same([t[cut] if t is not None else None for t in got], want)
    n, d = 50_000 // wide, 1600
    x, w = r(1, n, d).to(dtype), r(d, 4).to(dtype)
    Y, last = cw.ttt_short_conv(x, w)
    for c in range(0, d, 400):
        y2, l2 = cw.ttt_short_conv(x[:, :, c:c + 400], w[c:c + 400].contiguous())
        assert torch.equal(Y[:, :, c:c + 400], y2) and torch.equal(last[:, :, c:c + 400], l2)
    R, H = 300, 32
    x, B, C = r(R, H, 64).to(dtype), r(R, 2, 128).to(dtype), r(R, 2, 128).to(dtype)
    dt, A, S = r(R, H).abs(), -r(H).abs(), r(R, H, 64, 128)
    S2 = S.clone()
    O = cw.ttt_selective_scan_step(x, dt, A, B, C, S)
    for c in range(0, R, 100):
        k = slice(c, c + 100)
        assert torch.equal(O[k], cw.ttt_selective_scan_step(x[k], dt[k], A, B[k], C[k], S2[k]))
    assert torch.equal(S, S2)


@pytest.mark.parametrize("kind", ["scan_packed_backward", "conv_backward", "rms_backward", "scan_packed"])
def test_the_same_bits_at_every_call(kind):
    call, _ = calls(kind, torch.bfloat16)
    first = call()
    for _ in range(3):
        assert same(call(), first)


def test_one_tap():
    """K = 1 has no earlier rows: y = silu(w x + b), its state has no rows."""
    gen = torch.Generator("cuda").manual_seed(1)
    x, w, b = (torch.randn(*s, device="cuda", generator=gen) for s in ((2, 50, 72), (72, 1), (72,)))
    Y, last = cw.ttt_short_conv(x, w, b)
    want = np.stack([osc.short_conv(f64(x[i]), f64(w), f64(b))[0] for i in range(2)])
    assert last.shape == (2, 0, 72) and rel(Y, want) <= 8 * 2.0 ** -24     # a product, a sum and SiLU's few operations
    halo = torch.empty(4, 0, 72, device="cuda")
    assert torch.equal(cw.ttt_short_conv_step(x[0, :4].contiguous(), w, halo, b), Y[0, :4])
    dx, dw, db, _ = cw.ttt_short_conv_backward(x, w, torch.ones_like(x), b)
    assert dx.shape == x.shape and torch.isfinite(dx).all() and dw.shape == w.shape and db.shape == b.shape


@pytest.mark.parametrize("dtype", DTYPES)
def test_no_tokens_and_no_rows(dtype):
    """Zero tokens leave the states as they were (or zero) and give zero sums; zero rows and sequences give empty tensors."""
    H, G, P, N = 2, 1, 24, 16
    print("empty", dtype, flush=True)
    for B, n in ((3, 0), (0, 5), (0, 0)):
        *args, D, bias = make(B, H, G, n, P, N, dtype)
        S0 = torch.randn(B, H, P, N, device="cuda")
        more = dict(D=D, dt_bias=bias, softplus=True, S_init=S0)
        O, S = cw.ttt_selective_scan(*args, **more)
        assert O.shape == (B, H, n, P) and torch.equal(S, S0)
        assert (cw.ttt_selective_scan(*args)[1] == 0).all()
        dS = torch.randn_like(S0)
        dx, ddt, dA, dB, dC, dD, db, dS0 = cw.ttt_selective_scan_backward(*args, torch.empty_like(args[0]), dS_final=dS, **more)
        assert dx.shape == (B, H, n, P) and torch.equal(dS0, dS)
        assert not dA.any() and not dD.any() and not db.any()
        x, w, b = torch.empty(B, n, 40, dtype=dtype, device="cuda"), torch.randn(40, 4).to(dtype).cuda(), torch.randn(40).to(dtype).cuda()
        x0 = torch.randn(B, 3, 40).to(dtype).cuda()
        Y, last = cw.ttt_short_conv(x, w, b, x_init=x0)
        dx, dw, db, dx0 = cw.ttt_short_conv_backward(x, w, x, b, x_init=x0, dx_final=x0)
        assert Y.shape == x.shape and dx.shape == x.shape and torch.equal(last, x0) and torch.equal(dx0, x0)
        assert not dw.any() and not db.any()
    e = lambda *s: torch.empty(*s, dtype=dtype, device="cuda")
    f = lambda *s: torch.empty(*s, device="cuda")
    assert cw.ttt_selective_scan_step(e(0, H, P), f(0, H), f(H), e(0, G, N), e(0, G, N), f(3, H, P, N)).shape == (0, H, P)
    assert cw.ttt_short_conv_step(e(0, 40), e(40, 4), e(3, 3, 40)).shape == (0, 40)
    assert cw.ttt_rms_norm(e(0, 40), residual=e(0, 40))[0].shape == (0, 40)
    dx, dw = cw.ttt_rms_norm_backward(e(0, 40), e(40), e(0, 40), f(0))
    assert dx.shape == (0, 40) and not dw.any()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("H,G,P,N", [(1, 1, 1000, 16), (2, 1, 264, 200), (1, 1, 4096, 8), (9, 1, 8, 8), (40, 2, 16, 24)])
def test_wide_narrow_and_many_heads(H, G, P, N, dtype):
    """Heads over several workgroups, and groups of more heads than a workgroup has, against the oracle; the bounds of
    the scan's tests (2^-8 and 2^-13 of bf16 outputs; 320 * 2^-24 of fp32 ones) with 4 times the fp32 bound in the backward
    pass, which has two such products one behind the other and their sums over heads."""
    n = 150
    print("heads", H, G, P, N, dtype, flush=True)
    *args, D, bias = make(1, H, G, n, P, N, dtype, layout="token")
    dO = torch.randn(args[0].shape, generator=torch.Generator().manual_seed(3)).to(dtype).cuda()
    more = dict(D=D, dt_bias=bias, softplus=True)
    O, S = cw.ttt_selective_scan(*args, **more)
    ref = [f64(t[0]) if t.dim() > 1 else f64(t) for t in args]
    Or, Sr = osc.selective_scan(*ref, f64(D), f64(bias), True)
    fp32 = 320 * 2.0 ** -24
    out = fp32 if dtype == torch.float32 else 2.0 ** -8 + 2.0 ** -13
    assert rel(O[0], Or) <= out and rel(S[0], Sr) <= fp32
    got = cw.ttt_selective_scan_backward(*args, dO, **more)
    want = osc.selective_scan_backward(*ref, f64(dO[0]), f64(D), f64(bias), True)
    for t, k in zip(got, ("dx", "ddt", "dA", "dB", "dC", "dD", "ddt_bias")):
        v = t[0] if t.dim() > 1 else t
        print(" ", k, rel(v, want[k]), flush=True)
        assert rel(v, want[k]) <= (4 * fp32 if t.dtype == torch.float32 else out), k


@pytest.mark.parametrize("dtype", DTYPES)
def test_many_short_sequences_are_a_batch(dtype):
    """2000 packed sequences of 3 tokens give the bits of a batch of them."""
    num, n, H, G, P, N = 2000, 3, 2, 1, 64, 32
    *args, D, bias = make(num, H, G, n, P, N, dtype)
    dO = torch.randn(num, H, n, P, generator=torch.Generator().manual_seed(3)).to(dtype).cuda()
    more = dict(D=D, dt_bias=bias, softplus=True)
    flat = lambda t: t.transpose(1, 2).flatten(0, 1)[None].transpose(1, 2).contiguous()
    starts = torch.arange(0, num * n + 1, n, dtype=torch.int32, device="cuda")
    pack = [flat(t) if t.dim() > 1 else t for t in args]
    O, S = cw.ttt_selective_scan(*args, **more)
    Op, Sp = cw.ttt_selective_scan(*pack, **more, seq_starts=starts)
    assert torch.equal(flat(O), Op) and torch.equal(S, Sp)
    g = cw.ttt_selective_scan_backward(*args, dO, **more)
    p = cw.ttt_selective_scan_backward(*pack, flat(dO), **more, seq_starts=starts)
    for i in (0, 1, 3, 4):
        assert torch.equal(flat(g[i]), p[i]), i
    # (sums over all tokens: fp64 of the chunks' fp32 parts, in another order)
    for i in (2, 5, 6):
        assert rel(p[i], f64(g[i])) <= 4 * 2.0 ** -24, i
