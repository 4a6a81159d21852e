"""The selective scan (whole sequences, token step) on the GPU against the oracle's token-by-token recurrence in fp64.

Tolerances (relative Frobenius norm).  A rounding to bf16 is off by at most half a step, 2^-8 of the value; fp32 by 2^-24.
  state   fp32 sums of the 64 tokens of a chunk, each as at most 3 parts, then one decay a chunk whose errors decay with
          the state: (3 * 64 + 128) * 2^-24 = 1.9e-5, fp32 and bf16 inputs alike.
  fp32 O  sums of at most N + 64 <= 320 terms: 320 * 2^-24 = 1.9e-5.
  bf16 O  its own rounding, 2^-8; the state and the decayed products before it are pairs of bf16 values, 2^-16 of terms
          whose norm is at most 8 times the sum's in these random inputs: 2^-13.
  step    fp32 sums of N <= 256 terms: 256 * 2^-24 = 1.5e-5; bf16 O adds its rounding.
"""
import numpy as np
import pytest
import torch

import chunk_wise_weight_amd as cw
from oracle import scan as osc

pytestmark = pytest.mark.gpu

TOL_S = 320 * 2.0 ** -24
TOL_O = {torch.bfloat16: 2.0 ** -8 + 2.0 ** -13, torch.float32: 320 * 2.0 ** -24}
TOL_STEP = {torch.bfloat16: 2.0 ** -8 + 256 * 2.0 ** -24, torch.float32: 256 * 2.0 ** -24}
DTYPES = [torch.float32, torch.bfloat16]


def rel(a, b):
    a = a.double().cpu().numpy() if isinstance(a, torch.Tensor) else a
    n = np.linalg.norm(b)
    return float(np.linalg.norm(a - b) / n) if n else float(np.abs(a).max(initial=0.0))


def f64(x):
    return None if x is None else x.double().cpu().numpy()


def make(B, H, G, n, P, N, dtype, layout="token", seed=0):
    """x, dt, A, B, C on the GPU, heads cut out of one token-major tensor or contiguous, and D, dt_bias."""
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen)
    xbc = r(B, n, H * P + 2 * G * N).to(dtype).cuda()
    parts = [t.unflatten(-1, s).transpose(1, 2) for t, s in
             zip(xbc.split([H * P, G * N, G * N], -1), ((H, P), (G, N), (G, N)))]
    if layout == "head":
        parts = [t.contiguous() for t in parts]
    dt = (r(B, n, H).cuda()).transpose(1, 2)
    A = -(0.05 + 3 * torch.rand(H, generator=gen) ** 2).cuda()
    return parts[0], dt, A, parts[1], parts[2], r(H).cuda(), (r(H) - 1).cuda()


def oracle(b, args, D=None, bias=None, softplus=False, S0=None, cut=slice(None)):
    x, dt, A, B, C = args
    return osc.selective_scan(f64(x[b][:, cut]), f64(dt[b][:, cut]), f64(A), f64(B[b][:, cut]), f64(C[b][:, cut]), f64(D),
                              f64(bias), softplus, f64(S0))


CASES = [  # B, H, G, n, P, N, layout: every variant of heads and widths, one segment and several
    (1, 1, 1, 1, 64, 16, "head"),
    (2, 4, 2, 63, 64, 72, "token"),
    (1, 2, 2, 64, 128, 128, "head"),
    (1, 3, 1, 200, 16, 8, "token"),
    (1, 4, 2, 130, 96, 80, "head"),
    (1, 2, 1, 257, 40, 256, "token"),
    (3, 1, 1, 65, 24, 8, "token"),
    (1, 2, 1, 700, 136, 128, "token"),
    (1, 3, 3, 150, 200, 200, "head"),
    (1, 8, 1, 1100, 32, 64, "token"),
    (1, 5, 1, 600, 64, 128, "token"),
    (2, 6, 2, 330, 8, 128, "head"),
    (1, 7, 1, 300, 32, 136, "token"),
]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("start", [False, True])
def test_sequence(case, dtype, start):
    B, H, G, n, P, N, layout = case
    print("scan", case, dtype, start, flush=True)
    *args, D, bias = make(B, H, G, n, P, N, dtype, layout)
    S0 = torch.randn(B, H, P, N, generator=torch.Generator().manual_seed(5)).mul(0.3).cuda() if start else None
    more = dict(D=D, dt_bias=bias, softplus=True) if start else dict(softplus=True)
    O, S = cw.ttt_selective_scan(*args, S_init=S0, **more)
    assert O.stride() == torch.empty_like(args[0]).stride() and O.dtype == dtype and S.dtype == torch.float32
    for b in range(B):
        Or, Sr = oracle(b, args, more.get("D"), more.get("dt_bias"), True, S0[b] if start else None)
        print("  rel err", rel(O[b], Or), rel(S[b], Sr), flush=True)
        assert rel(O[b], Or) <= TOL_O[dtype]
        assert rel(S[b], Sr) <= TOL_S


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("lens", [[70, 0, 1, 64, 129], [0, 0], [3], [64, 64, 64], [1] * 9, [0, 700, 0], [300, 257, 0, 256, 513], []])
def test_packed_sequences(dtype, lens):
    """Sequences of any lengths in one row.  What lies in front of the first and behind the last is not read (NaN) and
    stays as it was."""
    H, G, P, N, front, behind = 2, 1, 48, 64, 5, 37
    n = front + sum(lens) + behind
    print("scan packed", lens, dtype, flush=True)
    *args, D, bias = make(1, H, G, n, P, N, dtype, seed=len(lens))
    for t in (args[0], args[1], args[3], args[4]):
        t[:, :, :front] = float("nan")
        t[:, :, n - behind:] = float("nan")
    starts = torch.tensor([front] + lens).cumsum(0).to(torch.int32).cuda()
    S0 = torch.randn(len(lens), H, P, N, generator=torch.Generator().manual_seed(6)).cuda()
    O = torch.full_like(args[0], 7.0)
    _, S = cw.ttt_selective_scan(*args, D=D, dt_bias=bias, softplus=True, S_init=S0, seq_starts=starts, O=O)
    assert (O[:, :, :front] == 7).all() and (O[:, :, n - behind:] == 7).all()
    at = front
    for i, m in enumerate(lens):
        Or, Sr = oracle(0, args, D, bias, True, S0[i], slice(at, at + m))
        assert rel(O[0, :, at:at + m], Or) <= TOL_O[dtype], (i, m)
        assert rel(S[i], Sr) <= TOL_S, (i, m)
        if m == 0:
            assert torch.equal(S[i], S0[i])
        at += m


@pytest.mark.parametrize("dtype", DTYPES)
def test_rates_without_softplus_idle_tokens_and_emptied_states(dtype):
    """A rate of zero leaves the state as it is; a log decay far below -104 empties it, also what is not finite in it;
    decays that differ by much inside a chunk keep the digits of their differences."""
    x, dt, A, B, C, D, _ = make(1, 2, 1, 600, 64, 64, dtype, "head", seed=9)
    dt = dt.abs() * 0.3
    dt[:, :, 20:30] = 0.0
    dt[:, :, 64:70] = 0.0
    dt[:, :, 100:130] = 0.0
    dt[:, 1, 140:170] = 20.0
    dt[:, :, 300] = 1e6
    dt[:, 0, 17] = 1e6
    S0 = torch.full((1, 2, 64, 64), float("inf"), device="cuda")
    dt[:, :, 0] = 1e6
    A[:] = torch.tensor([-1.0, -2.0])
    args = (x, dt, A, B, C)
    O, S = cw.ttt_selective_scan(*args, D=D, S_init=S0)
    Or, Sr = oracle(0, args, D, None, False, torch.zeros(2, 64, 64))
    assert rel(O[0, :, 1:], Or[:, 1:]) <= TOL_O[dtype] and rel(S[0], Sr) <= TOL_S
    # nothing before it reaches what follows
    x2 = x.clone()
    x2[:, :, :300] += 100.0
    O2, S2 = cw.ttt_selective_scan(x2, *args[1:], D=D)
    assert torch.equal(O2[:, :, 300:], O[:, :, 300:]) and torch.equal(S2, S)


@pytest.mark.parametrize("dtype", DTYPES)
def test_resumed_calls_go_on(dtype):
    *args, D, bias = make(2, 2, 1, 900, 64, 128, dtype)
    cut = lambda a, b: [args[0][:, :, a:b], args[1][:, :, a:b], args[2], args[3][:, :, a:b], args[4][:, :, a:b]]
    kw = dict(D=D, dt_bias=bias, softplus=True)
    O, S = cw.ttt_selective_scan(*args, **kw)
    Sa, parts = None, []
    for a, b in ((0, 130), (130, 131), (131, 600), (600, 900)):
        o, Sa = cw.ttt_selective_scan(*cut(a, b), S_init=Sa, **kw)
        parts.append(o)
    for b in range(2):
        Or, Sr = oracle(b, args, D, bias, True)
        assert rel(torch.cat(parts, 2)[b], Or) <= TOL_O[dtype] and rel(Sa[b], Sr) <= 2 * TOL_S


@pytest.mark.parametrize("dtype", DTYPES)
def test_prompt_then_tokens_is_the_sequence(dtype):
    """A prompt through the scan, then token after token through the step, in a pool of states."""
    *args, D, bias = make(2, 4, 2, 200, 64, 128, dtype)
    kw = dict(D=D, dt_bias=bias, softplus=True)
    x, dt, A, B, C = args
    O, S = cw.ttt_selective_scan(x[:, :, :190], dt[:, :, :190], A, B[:, :, :190], C[:, :, :190], **kw)
    pool = torch.randn(5, 4, 64, 128, device="cuda")
    slots = torch.tensor([3, 1], dtype=torch.int32, device="cuda")
    pool[slots.long()] = S
    for t in range(190, 200):
        o = cw.ttt_selective_scan_step(*(v[:, :, t].contiguous() if v.dim() > 1 else v for v in args), pool, slots=slots, **kw)
        for b in range(2):
            Or, Sr = oracle(b, args, D, bias, True, cut=slice(0, t + 1))
            assert rel(o[b], Or[:, t]) <= TOL_O[dtype] + TOL_STEP[torch.float32]
    for b in range(2):
        assert rel(pool[slots[b]], Sr) <= 2 * TOL_S if b == 1 else True


@pytest.mark.parametrize("dtype", DTYPES)
def test_any_strides(dtype):
    """Groups repeated by zero strides, gates and tokens of any strides, outputs inside a wider tensor."""
    x, dt, A, B, C, D, bias = make(2, 4, 4, 150, 64, 32, dtype, "head")
    B1, C1 = B[:, :1].expand(2, 4, 150, 32), C[:1].expand(2, 4, 150, 32)
    dtw = torch.zeros(4, 150, 2, 3, device="cuda")[..., 1].permute(2, 0, 1).copy_(dt)
    O = torch.zeros(2, 150, 4, 128, dtype=dtype, device="cuda")[..., 64:].transpose(1, 2)
    out, S = cw.ttt_selective_scan(x, dtw, A, B1, C1, D=D, O=O)
    ref = cw.ttt_selective_scan(x, dt.contiguous(), A, B1.contiguous(), C1.contiguous(), D=D)
    assert out is O and torch.equal(O, ref[0]) and torch.equal(S, ref[1])


STEPS = [(1, 2, 4, 2, 64, 128), (9, 12, 3, 1, 72, 16), (5, 5, 2, 2, 8, 256), (33, 40, 4, 1, 40, 64), (3, 4, 1, 1, 136, 8),
         (7, 9, 6, 2, 16, 32), (4, 4, 2, 1, 256, 200)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("case", STEPS)
def test_step(case, dtype):
    R, pool, H, G, P, N = case
    print("scan step", case, dtype, flush=True)
    *args, D, bias = make(1, H, G, R, P, N, dtype, seed=4)
    x, dt, A, B, C = (v[0].transpose(0, 1).contiguous() if v.dim() > 1 else v for v in args)
    S0 = torch.randn(pool, H, P, N, generator=torch.Generator().manual_seed(2)).cuda()
    slots = torch.randperm(pool, generator=torch.Generator().manual_seed(1))[:R].to(torch.int32).cuda()
    if R > 2:
        slots[1], slots[-1] = -1, pool
    for named, kw in ((True, dict(D=D, dt_bias=bias, softplus=True)), (False, {})):
        S = S0.clone()
        O = cw.ttt_selective_scan_step(x, dt, A, B, C, S, slots=slots if named else None, **kw)
        want = f64(S0)
        for r in range(R):
            s = int(slots[r]) if named else r
            if not 0 <= s < pool:
                assert (O[r] == 0).all()
                continue
            one = [f64(v[r])[:, None] if v.dim() > 1 else f64(v) for v in (x, dt, A, B, C)]
            Or, Sr = osc.selective_scan(*one, f64(kw.get("D")), f64(kw.get("dt_bias")), kw.get("softplus", False), want[s])
            assert rel(O[r], Or[:, 0]) <= TOL_STEP[dtype]
            want[s] = Sr
        assert rel(S, want) <= TOL_STEP[torch.float32]
        untouched = sorted(set(range(pool)) - {int(s) for s in (slots if named else range(R))})
        assert torch.equal(S[untouched], S0[untouched])


@pytest.mark.parametrize("dtype", DTYPES)
def test_step_rows_of_one_slot_go_in_row_order(dtype):
    *args, D, bias = make(1, 2, 1, 700, 32, 64, dtype, seed=8)
    x, dt, A, B, C = (v[0].transpose(0, 1).contiguous() if v.dim() > 1 else v for v in args)
    slots = torch.randint(0, 3, (700,), generator=torch.Generator().manual_seed(3)).to(torch.int32).cuda()
    slots[::50] = -1
    S = torch.zeros(3, 2, 32, 64, device="cuda")
    O = cw.ttt_selective_scan_step(x, dt, A, B, C, S, D=D, dt_bias=bias, softplus=True, slots=slots)
    for s in range(3):
        mine = (slots == s).nonzero()[:, 0]
        Or, Sr = osc.selective_scan(*(f64(v[mine].transpose(0, 1)) if v.dim() > 1 else f64(v) for v in (x, dt, A, B, C)),
                                    f64(D), f64(bias), True)
        assert rel(O[mine].transpose(0, 1), Or) <= TOL_STEP[dtype] + TOL_S and rel(S[s], Sr) <= TOL_S
    assert (O[::50] == 0).all()


def test_a_step_that_empties_a_state():
    *args, D, bias = make(1, 2, 1, 2, 16, 16, torch.float32)
    x, dt, A, B, C = (v[0].transpose(0, 1).contiguous() if v.dim() > 1 else v for v in args)
    dt[:] = 1e6
    S = torch.full((2, 2, 16, 16), float("nan"), device="cuda")
    O = cw.ttt_selective_scan_step(x, dt, A, B, C, S)
    assert torch.isfinite(O).all() and torch.isfinite(S).all()


def test_refusals():
    x, dt, A, B, C, D, bias = make(2, 4, 2, 50, 64, 32, torch.bfloat16, "head")
    good = dict(x=x, dt=dt, A=A, B=B, C=C)
    for bad in (dict(dt=dt.bfloat16()), dict(A=A[:2]), dict(B=B.float()), dict(C=C[:, :, :20]), dict(D=D.bfloat16()),
                dict(dt_bias=bias[:1]), dict(x=x.transpose(2, 3)), dict(x=x.cpu()), dict(S_init=torch.zeros(2, 4, 64, 16, device="cuda")),
                dict(seq_starts=torch.zeros(3, dtype=torch.int32, device="cuda")), dict(O=x[:, :1].expand(2, 4, 50, 64)),
                dict(workspace=torch.empty(0, device="cuda"), x=torch.cat([x] * 20, 2), dt=torch.cat([dt] * 20, 2),
                     B=torch.cat([B] * 20, 2), C=torch.cat([C] * 20, 2))):
        with pytest.raises((ValueError, TypeError)):
            cw.ttt_selective_scan(**{**good, **bad})
    for bad in (dict(B=B[:, :1].expand(2, 3, 50, 32), C=C[:, :1].expand(2, 3, 50, 32)),
                dict(B=torch.zeros(2, 2, 50, 264, device="cuda", dtype=torch.bfloat16),
                     C=torch.zeros(2, 2, 50, 264, device="cuda", dtype=torch.bfloat16))):
        with pytest.raises(cw.TTTError):
            cw.ttt_selective_scan(**{**good, **bad})
    S = torch.zeros(1, 4, 64, 32, device="cuda")
    one = dict(x=x[:, :, 0].contiguous(), dt=dt[:, :, 0].contiguous(), A=A, B=B[:, :, 0].contiguous(), C=C[:, :, 0].contiguous())
    with pytest.raises(cw.TTTError):
        cw.ttt_selective_scan_step(**one, S=S)               # more rows than states
    with pytest.raises(ValueError):
        cw.ttt_selective_scan_step(**{**one, "x": x[:, :, 0]}, S=S)
