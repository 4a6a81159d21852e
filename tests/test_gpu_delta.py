"""The gated delta rule on the GPU against the oracle's token-by-token recurrence in fp64.

Tolerances (relative Frobenius norm).  A rounding to bf16 is off by at most half a step, 2^-8 of the value; fp32 by
2^-24.
  bf16 O        four roundings to bf16 lie between the inputs and O (the state, P, the errors, O itself), independent,
                each of relative norm <= 2^-8: sqrt(4) 2^-8.
  bf16 W_final  operands are pairs of bf16 values, off by 2^-16 at most: the state, the residual, T, the products of
                two low parts left out, and the scaled errors, each chunk: sqrt(5) 2^-16, taken twice for the chunks
                that follow one another (what a chunk adds decays and is corrected by later ones).
  fp32          sums of at most dk + 64 <= 320 terms in fp32, 320 * 2^-24 = 1.9e-5.
  step          fp32 sums of dk <= 256 terms: 256 * 2^-24 = 1.5e-5; bf16 O adds one rounding, 2^-8.
"""
import numpy as np
import pytest
import torch

import chunk_wise_weight_amd as cw
from oracle import delta as od

pytestmark = pytest.mark.gpu

TOL_O = {torch.bfloat16: 2 * 2.0 ** -8, torch.float32: 320 * 2.0 ** -24}
TOL_W = {torch.bfloat16: 2 * 5 ** 0.5 * 2.0 ** -16, torch.float32: 320 * 2.0 ** -24}
TOL_STEP = {torch.bfloat16: 2.0 ** -8 + 256 * 2.0 ** -24, torch.float32: 256 * 2.0 ** -24}
DTYPES = [torch.float32, torch.bfloat16]


def rel(a, b):
    a = a.double().cpu().numpy() if isinstance(a, torch.Tensor) else a
    n = np.linalg.norm(b)
    return float(np.linalg.norm(a - b) / n) if n else float(np.abs(a).max(initial=0.0))


def f64(x):
    return None if x is None else x.double().cpu().numpy()


def make(B, Hk, Hv, n, dk, dv, dtype, layout="token", seed=0):
    """q, k (unit), v, g, beta on the GPU, heads cut out of token-major tensors or contiguous."""
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen)
    swap = (lambda t: t.cuda().transpose(1, 2)) if layout == "token" else (lambda t: t.cuda().transpose(1, 2).contiguous())
    q, k = (torch.nn.functional.normalize(r(B, n, Hk, dk), dim=-1).to(dtype) for _ in range(2))
    v = r(B, n, Hv, dv).to(dtype)
    g = -torch.rand(B, n, Hv, generator=gen) ** 3 * 2
    beta = torch.sigmoid(r(B, n, Hv))
    return [swap(t) for t in (q, k, v, g, beta)]


CASES = [  # B, Hk, Hv, n, dk, dv, layout
    (1, 1, 1, 1, 64, 16, "head"),
    (2, 2, 4, 63, 64, 72, "token"),
    (1, 2, 2, 64, 128, 128, "head"),
    (1, 1, 3, 200, 16, 8, "token"),
    (1, 2, 4, 130, 96, 80, "head"),
    (1, 1, 2, 257, 256, 40, "token"),
    (3, 1, 1, 65, 8, 24, "token"),
    (1, 1, 2, 700, 128, 136, "token"),
    (1, 3, 3, 150, 200, 200, "head"),
]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("start", [False, True])
def test_sequence(case, dtype, start):
    B, Hk, Hv, n, dk, dv, layout = case
    print("delta", case, dtype, start, flush=True)
    q, k, v, g, beta = make(B, Hk, Hv, n, dk, dv, dtype, layout)
    W0 = torch.randn(B, Hv, dv, dk, generator=torch.Generator().manual_seed(5)).mul(0.3).cuda() if start else None
    O, W = cw.ttt_gated_delta(q, k, v, g, beta, scale=0.4, W_init=W0)
    assert O.stride() == v.stride() and O.dtype == dtype and W.dtype == torch.float32
    for b in range(B):
        Or, Wr = od.delta_rule(*(f64(t[b]) for t in (q, k, v, g, beta)), 0.4, f64(W0[b]) if start else None)
        print("  rel err", rel(O[b], Or), rel(W[b], Wr), flush=True)
        assert rel(O[b], Or) <= TOL_O[dtype]
        assert rel(W[b], Wr) <= TOL_W[dtype]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("lens", [[70, 0, 1, 64, 129], [0, 0], [3], [64, 64, 64], [1] * 9, [0, 200, 0]])
def test_packed_sequences(dtype, lens):
    """Sequences of any lengths in one row.  What lies in front of the first and behind the last is not read (NaN) and
    stays as it was."""
    Hk, Hv, dk, dv, front, behind = 1, 2, 64, 48, 5, 37
    n = front + sum(lens) + behind
    q, k, v, g, beta = make(1, Hk, Hv, n, dk, dv, dtype, seed=len(lens))
    for t in (q, k, v, g, beta):
        t[:, :, :front] = float("nan")
        t[:, :, n - behind:] = float("nan")
    starts = torch.tensor([front] + lens).cumsum(0).to(torch.int32).cuda()
    W0 = torch.randn(len(lens), Hv, dv, dk, generator=torch.Generator().manual_seed(6)).cuda()
    O = torch.full_like(v, 7.0)
    _, W = cw.ttt_gated_delta(q, k, v, g, beta, W_init=W0, seq_starts=starts, O=O)
    assert (O[:, :, :front] == 7).all() and (O[:, :, n - behind:] == 7).all()
    at = front
    for i, m in enumerate(lens):
        part = [f64(t[0, :, at:at + m]) for t in (q, k, v, g, beta)]
        Or, Wr = od.delta_rule(*part, dk ** -0.5, f64(W0[i]))
        assert rel(O[0, :, at:at + m], Or) <= TOL_O[dtype], (i, m)
        assert rel(W[i], Wr) <= TOL_W[dtype], (i, m)
        if m == 0:
            assert torch.equal(W[i], W0[i])
        at += m


@pytest.mark.parametrize("dtype", DTYPES)
def test_packed_equals_rows_bit_for_bit(dtype):
    """A sequence's results do not depend on where it lies or on its neighbours."""
    q, k, v, g, beta = make(3, 2, 4, 100, 128, 64, dtype, "head")
    O, W = cw.ttt_gated_delta(q, k, v, g, beta)
    flat = [t.transpose(0, 1).reshape(1, t.shape[1], 300, *t.shape[3:]).contiguous() for t in (q, k, v, g, beta)]
    Op, Wp = cw.ttt_gated_delta(*flat, seq_starts=torch.tensor([0, 100, 200, 300], dtype=torch.int32, device="cuda"))
    assert torch.equal(Wp, W)
    assert torch.equal(Op.reshape(4, 3, 100, 64).transpose(0, 1), O)


@pytest.mark.parametrize("dtype", DTYPES)
def test_resets_strong_decays_and_idle_tokens(dtype):
    """g = -inf empties the state (a document boundary), very strong and zero decays, beta = 0 and beta = 2; decays
    that differ by much inside a chunk keep the digits of their differences."""
    q, k, v, g, beta = make(1, 1, 2, 200, 64, 64, dtype, "head", seed=9)
    g[:, :, 17] = float("-inf")
    g[:, :, 64] = float("-inf")
    g[:, :, 90:95] = -150.0
    g[:, :, 100:130] = 0.0
    g[:, 1, 140:] = -40.0
    g[:, 1, 180] = float("-inf")
    beta[:, :, 20:30] = 0.0
    beta[:, :, 110] = 2.0
    O, W = cw.ttt_gated_delta(q, k, v, g, beta)
    Or, Wr = od.delta_rule(*(f64(t[0]) for t in (q, k, v, g, beta)), 64 ** -0.5)
    assert rel(O[0], Or) <= TOL_O[dtype] and rel(W[0], Wr) <= TOL_W[dtype]
    # nothing before the reset reaches what follows it
    v2 = v.clone()
    v2[:, :, :64] += 100.0
    O2, _ = cw.ttt_gated_delta(q, k, v2, g, beta)
    assert torch.equal(O2[:, :, 64:], O[:, :, 64:])


@pytest.mark.parametrize("dtype", DTYPES)
def test_two_calls_equal_one(dtype):
    q, k, v, g, beta = make(2, 1, 2, 256, 64, 64, dtype, "head")
    O, W = cw.ttt_gated_delta(q, k, v, g, beta)
    first = [t[:, :, :128] for t in (q, k, v, g, beta)]
    Oa, Wa = cw.ttt_gated_delta(*first)
    Ob, Wb = cw.ttt_gated_delta(*(t[:, :, 128:] for t in (q, k, v, g, beta)), W_init=Wa)
    assert torch.equal(torch.cat([Oa, Ob], 2), O) and torch.equal(Wb, W)


def test_strides_of_a_joint_projection_and_repeated_inputs():
    """q, k and v as slices of one token-major projection; one query row repeated with stride 0."""
    B, n, Hk, Hv, d = 2, 90, 2, 4, 64
    x = torch.randn(B, n, (2 * Hk + Hv) * d, generator=torch.Generator().manual_seed(3)).bfloat16().cuda() * 0.1
    cut = lambda a, H: x[..., a * d:(a + H) * d].unflatten(-1, (H, d)).transpose(1, 2)
    q, k, v = cut(0, Hk), cut(Hk, Hk), cut(2 * Hk, Hv)
    g, beta = -torch.rand(B, n, Hv, device="cuda").transpose(1, 2), torch.rand(B, n, Hv, device="cuda").transpose(1, 2)
    O, W = cw.ttt_gated_delta(q, k, v, g, beta)
    Oc, Wc = cw.ttt_gated_delta(*(t.contiguous() for t in (q, k, v, g, beta)))
    assert torch.equal(O, Oc) and torch.equal(W, Wc)
    one = q[:, :, :1].expand(-1, -1, n, -1)
    assert torch.equal(cw.ttt_gated_delta(one, k, v, g, beta)[0],
                       cw.ttt_gated_delta(one.contiguous(), k, v, g, beta)[0])


def test_empty():
    for B, n in ((0, 5), (2, 0), (0, 0)):
        q, k, v, g, beta = make(B, 1, 2, n, 64, 64, torch.bfloat16, "head")
        W0 = torch.randn(B, 2, 64, 64, device="cuda")
        O, W = cw.ttt_gated_delta(q, k, v, g, beta, W_init=W0)
        assert O.shape == (B, 2, n, 64) and torch.equal(W, W0)
        assert not cw.ttt_gated_delta(q, k, v, g, beta)[1].any()
    q, k, v, g, beta = make(1, 1, 2, 10, 64, 64, torch.bfloat16, "head")
    O, W = cw.ttt_gated_delta(q, k, v, g, beta, seq_starts=torch.zeros(1, dtype=torch.int32, device="cuda"))
    assert W.shape[0] == 0


# ---------------------------------------------------------------------------------------------- step


def make_step(R, P, Hk, Hv, dk, dv, dtype, seed=0):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen)
    q, k = (torch.nn.functional.normalize(r(R, Hk, dk), dim=-1).to(dtype).cuda() for _ in range(2))
    v = r(R, Hv, dv).to(dtype).cuda()
    g, beta = -torch.rand(R, Hv, generator=gen).cuda(), torch.rand(R, Hv, generator=gen).cuda()
    return q, k, v, g, beta, r(P, Hv, dv, dk).cuda()


def step_reference(q, k, v, g, beta, W, slots, scale):
    W = f64(W)
    O = np.zeros(tuple(v.shape))
    for r, s in enumerate(slots):
        if 0 <= s < W.shape[0]:
            o, W[s] = od.delta_rule(*(f64(t[r])[:, None] for t in (q, k, v)), *(f64(t[r])[:, None] for t in (g, beta)),
                                    scale, W[s])
            O[r] = o[:, 0]
    return O, W


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("case", [
    (1, 1, 1, 1, 64, 16, [0]),
    (3, 5, 2, 4, 128, 128, [4, 0, 2]),
    (4, 4, 5, 5, 96, 80, None),
    (5, 3, 1, 2, 256, 40, [-1, 2, 3, 0, 1 << 30]),          # padding rows, and a slot behind the pool
    (7, 3, 1, 3, 8, 24, [1, 0, 1, -1, 1, 0, 2]),            # rows of one state: in row order
    (140, 2, 1, 1, 64, 8, [i % 2 for i in range(140)]),     # the same, over more rows than a wave has lanes
])
def test_step(case, dtype):
    R, P, Hk, Hv, dk, dv, slots = case
    print("step", case[:6], dtype, flush=True)
    q, k, v, g, beta, W = make_step(R, P, Hk, Hv, dk, dv, dtype)
    Or, Wr = step_reference(q, k, v, g, beta, W, list(range(R)) if slots is None else slots, dk ** -0.5)
    untouched = [i for i in range(P) if slots is not None and i not in slots]
    before = W.clone()
    O = torch.full_like(v, float("nan"))
    cw.ttt_gated_delta_step(q, k, v, g, beta, W, O=O,
                            slots=None if slots is None else torch.tensor(slots, dtype=torch.int32, device="cuda"))
    assert rel(O, Or) <= TOL_STEP[dtype]
    assert rel(W, Wr) <= TOL_STEP[torch.float32]
    assert torch.equal(W[untouched], before[untouched])
    for r, s in enumerate(slots or []):
        if not 0 <= s < P:
            assert not O[r].any()


@pytest.mark.parametrize("dtype", DTYPES)
def test_step_goes_on_from_a_sequence(dtype):
    """A prompt with ttt_gated_delta, then tokens with the step on its W_final: as the whole sequence at once."""
    B, Hk, Hv, n, dk, dv = 3, 2, 4, 70, 128, 128
    q, k, v, g, beta = make(B, Hk, Hv, n + 4, dk, dv, dtype)
    O, W = cw.ttt_gated_delta(q, k, v, g, beta)
    _, pool = cw.ttt_gated_delta(*(t[:, :, :n] for t in (q, k, v, g, beta)))
    for t in range(n, n + 4):
        o = cw.ttt_gated_delta_step(*(x[:, :, t].contiguous() for x in (q, k, v, g, beta)), pool)
        assert rel(o, f64(O[:, :, t])) <= TOL_O[dtype] + TOL_STEP[dtype]
    assert rel(pool, f64(W)) <= 2 * TOL_W[dtype]


# ---------------------------------------------------------------------------------------------- refusals, streams


def test_refusals():
    q, k, v, g, beta = make(2, 1, 2, 40, 64, 64, torch.bfloat16, "head")
    W0 = torch.zeros(2, 2, 64, 64, device="cuda")
    one = torch.tensor([0, 40], dtype=torch.int32, device="cuda")
    bad = [
        (TypeError, dict(k=k.float())), (TypeError, dict(g=g.bfloat16())), (ValueError, dict(v=v[:, :, :39])),
        (ValueError, dict(W_init=W0[:1])), (ValueError, dict(seq_starts=one)),         # two rows
        (TypeError, dict(seq_starts=one.long())), (ValueError, dict(q=q.transpose(2, 3).contiguous().transpose(2, 3))),
        (ValueError, dict(k=k.cpu())), (ValueError, dict(O=v[:, :1].expand(-1, 2, -1, -1))),
        (ValueError, dict(workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))),
        (cw.TTTError, dict(scale=float("nan"))),
    ]
    for err, change in bad:
        args = dict(q=q, k=k, v=v, g=g, beta=beta) | change
        with pytest.raises(err):
            cw.ttt_gated_delta(**args)
    with pytest.raises(cw.TTTError):                                  # 3 value heads on 2 key heads
        cw.ttt_gated_delta(*make(1, 2, 3, 8, 64, 64, torch.bfloat16))
    with pytest.raises((cw.TTTError, ValueError)):                    # k_dim 12
        cw.ttt_gated_delta(*make(1, 1, 1, 8, 12, 64, torch.float32))
    q, k, v, g, beta, W = make_step(3, 2, 1, 1, 64, 64, torch.bfloat16)
    with pytest.raises(cw.TTTError):                                  # rows without slots need as many states
        cw.ttt_gated_delta_step(q, k, v, g, beta, W)
    with pytest.raises(TypeError):
        cw.ttt_gated_delta_step(q, k, v, g, beta, W, slots=torch.zeros(3, dtype=torch.int64, device="cuda"))


def test_captured_replays_equal_the_eager_calls():
    q, k, v, g, beta = make(2, 1, 2, 200, 128, 64, torch.bfloat16)
    starts = torch.tensor([0, 150, 400], dtype=torch.int32, device="cuda")
    flat = [t.transpose(0, 1).reshape(1, t.shape[1], 400, *t.shape[3:]).contiguous() for t in (q, k, v, g, beta)]
    O = torch.empty_like(flat[2])
    sq, sk, sv, sg, sb, pool = make_step(4, 4, 1, 2, 128, 64, torch.bfloat16)
    slots = torch.tensor([3, -1, 0, 2], dtype=torch.int32, device="cuda")
    call = lambda: (cw.ttt_gated_delta(*flat, seq_starts=starts, O=O)[1],
                    cw.ttt_gated_delta_step(sq, sk, sv, sg, sb, pool, slots=slots))
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        W, o = call()
    first = pool.clone()
    for i in range(3):
        starts[1] = 150 + 20 * i                   # lengths are read on the device: a replay takes the new ones
        flat[2].add_(0.5)
        pool.copy_(first)
        O.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (O, W, o, pool)]
        pool.copy_(first)
        O.zero_()
        We, oe = call()
        torch.cuda.synchronize()
        for a, b in zip(got, (O, We, oe, pool)):
            assert torch.equal(a, b)


def test_other_stream_and_two_calls_at_once():
    args = make(1, 2, 4, 600, 128, 128, torch.bfloat16)
    other = make(1, 2, 4, 600, 128, 128, torch.bfloat16, seed=1)
    ref, ref2 = cw.ttt_gated_delta(*args), cw.ttt_gated_delta(*other)
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        with torch.cuda.stream(a):
            x = cw.ttt_gated_delta(*args)
        with torch.cuda.stream(b):
            y = cw.ttt_gated_delta(*other)
        torch.cuda.synchronize()
        assert all(torch.equal(s, t) for s, t in zip(x + y, ref + ref2))


def test_starts_outside_the_row_are_taken_as_its_ends():
    q, k, v, g, beta = make(1, 1, 2, 100, 64, 64, torch.bfloat16)
    starts = lambda *s: torch.tensor(s, dtype=torch.int32, device="cuda")
    O, W = cw.ttt_gated_delta(q, k, v, g, beta, seq_starts=starts(0, 40, 100, 100))
    O2, W2 = cw.ttt_gated_delta(q, k, v, g, beta, seq_starts=starts(-5, 40, 1000, 1 << 30))
    assert torch.equal(O, O2) and torch.equal(W, W2)


def test_offsets_past_32_bits():
    """Rows further apart than 2^31 elements, and a state of the pool further in than that."""
    n, far = 70, (1 << 31) + 4096
    base = torch.zeros(far + 64 * n, dtype=torch.bfloat16, device="cuda")
    near = make(2, 1, 1, n, 64, 64, torch.bfloat16, "head", seed=8)
    views = []
    for t in near[:3]:                              # one tensor after the other at the same far places
        view = base.as_strided((2, 1, n, 64), (far, n * 64, 64, 1))
        view.copy_(t)
        args = [view if x is t else x for x in near]
        O, W = cw.ttt_gated_delta(*args)
        ref = cw.ttt_gated_delta(*near)
        assert torch.equal(O, ref[0]) and torch.equal(W, ref[1])
        views.append(view)
    out = views[0]
    out.zero_()
    cw.ttt_gated_delta(*near, O=out)
    assert torch.equal(out, cw.ttt_gated_delta(*near)[0])
    dO = torch.randn_like(near[2])
    d = cw.ttt_gated_delta_backward(*near, dO)
    d2 = cw.ttt_gated_delta_backward(*near, dO, dk=out)
    assert all(torch.equal(a, b) for a, b in zip(d[:5], d2[:5]))
    del base, views, view, out, args, d2
    q, k, v, g, beta, W = make_step(2, 2, 1, 32, 128, 128, torch.bfloat16)
    P = 4100                                        # 4100 x 32 x 128 x 128 > 2^31
    pool = torch.empty(P, 32, 128, 128, device="cuda")
    pool[[P - 1, 0]] = W
    o = cw.ttt_gated_delta_step(q, k, v, g, beta, pool, slots=torch.tensor([P - 1, 0], dtype=torch.int32, device="cuda"))
    assert torch.equal(o, cw.ttt_gated_delta_step(q, k, v, g, beta, W)) and torch.equal(pool[[P - 1, 0]], W)
