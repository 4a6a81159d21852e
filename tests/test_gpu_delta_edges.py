"""The gated delta rule, forward and step, at the edges of what it takes.  Tolerances are those of test_gpu_delta."""
import pytest
import torch

import chunk_wise_weight_amd as cw
from oracle import delta as od
from test_gpu_delta import DTYPES, TOL_O, TOL_STEP, TOL_W, f64, make, make_step, rel, step_reference

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n", [64, 128, 257])
def test_no_sequences(dtype, n):
    """A single start, the first entry of a longer tensor whose next one is the row's length: no token belongs to a
    sequence, none is read, every row of O stays as it is."""
    args = make(1, 1, 2, n, 64, 64, dtype, "head")
    for t in args:
        t.fill_(float("nan"))
    starts = torch.tensor([0, n], dtype=torch.int32, device="cuda")[:1]
    O = torch.full_like(args[2], 7.0)
    _, W = cw.ttt_gated_delta(*args, seq_starts=starts, O=O)
    torch.cuda.synchronize()
    assert W.shape == (0, 2, 64, 64) and (O == 7).all()


# Batches whose walks fill the chip, for which the state waves make O themselves: B, Hk, Hv, n, dk, dv, layout
FULL = [(8, 8, 32, 130, 128, 128, "token"), (8, 16, 32, 130, 64, 128, "head"), (8, 8, 32, 65, 128, 136, "token"),
        (20, 4, 32, 129, 64, 48, "head"), (6, 16, 64, 191, 96, 112, "token"), (40, 32, 32, 1, 64, 64, "token"),
        (9, 32, 32, 200, 40, 64, "token")]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("case", FULL)
def test_batches_that_fill_the_chip(case, dtype):
    """Against the oracle (some rows and heads), and bit for bit against rows on their own, whose walks do not fill it."""
    B, Hk, Hv, n, dk, dv, layout = case
    print("full", case, dtype, flush=True)
    args = make(B, Hk, Hv, n, dk, dv, dtype, layout, seed=31)
    W0 = torch.randn(B, Hv, dv, dk, generator=torch.Generator().manual_seed(32)).mul(0.3).cuda()
    O, W = cw.ttt_gated_delta(*args, W_init=W0)
    group = Hv // Hk
    for b, kh in ((0, 0), (B // 2, Hk - 1), (B - 1, Hk // 2)):
        v = slice(kh * group, (kh + 1) * group)
        one = [t[b, kh:kh + 1] for t in args[:2]] + [t[b, v] for t in args[2:]]
        Or, Wr = od.delta_rule(*(f64(t) for t in one), dk ** -0.5, f64(W0[b, v]))
        assert rel(O[b, v], Or) <= TOL_O[dtype] and rel(W[b, v], Wr) <= TOL_W[dtype]
        Oa, Wa = cw.ttt_gated_delta(*(t[None] for t in one), W_init=W0[b:b + 1, v].contiguous())
        assert torch.equal(Oa[0], O[b, v]) and torch.equal(Wa[0], W[b, v])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("dk", [64, 128])
def test_many_packed_sequences(dk, dtype):
    """Enough packed sequences to fill the chip, of 0 to 200 tokens, with NaN around them."""
    Hk, Hv, dv, front, behind = 8, 16, 128, 3, 70
    lens = [(i * 37) % 201 for i in range(90)]
    n = front + sum(lens) + behind
    args = make(1, Hk, Hv, n, dk, dv, dtype, seed=33)
    for t in args:
        t[:, :, :front] = float("nan")
        t[:, :, n - behind:] = float("nan")
    starts = torch.tensor([front] + lens).cumsum(0).to(torch.int32)
    W0 = torch.randn(len(lens), Hv, dv, dk, generator=torch.Generator().manual_seed(34)).mul(0.3).cuda()
    O = torch.full_like(args[2], 7.0)
    _, W = cw.ttt_gated_delta(*args, W_init=W0, seq_starts=starts.cuda(), O=O)
    assert (O[:, :, :front] == 7).all() and (O[:, :, n - behind:] == 7).all() and not O.isnan().any()
    for i in (0, 1, 11, 38, 89):
        at = slice(int(starts[i]), int(starts[i + 1]))
        Oa, Wa = cw.ttt_gated_delta(*(t[:, :, at] for t in args), W_init=W0[i:i + 1])
        assert torch.equal(Oa, O[:, :, at]) and torch.equal(Wa[0], W[i])
        h, kh = (i * 5) % Hv, (i * 5) % Hv // 2
        part = [f64(t[0, kh:kh + 1, at]) for t in args[:2]] + [f64(t[0, h:h + 1, at]) for t in args[2:]]
        Or, Wr = od.delta_rule(*part, dk ** -0.5, f64(W0[i, h:h + 1]))
        assert rel(O[0, h:h + 1, at], Or) <= TOL_O[dtype] and rel(W[i, h:h + 1], Wr) <= TOL_W[dtype], i


@pytest.mark.parametrize("dtype", DTYPES)
def test_reset_at_the_first_token_clears_any_state(dtype):
    """Fresh sequences among resumed ones: g = -inf at the first token, and a state that was never written (NaN, inf).
    An empty sequence has no such token and keeps its state."""
    lens, Hk, Hv, dk, dv = [70, 0, 1, 130], 1, 2, 64, 48
    args = make(1, Hk, Hv, sum(lens), dk, dv, dtype, seed=51)
    starts = torch.tensor([0] + lens).cumsum(0).to(torch.int32)
    W0 = torch.randn(4, Hv, dv, dk, generator=torch.Generator().manual_seed(52)).cuda()
    zero = W0.clone()
    for i in (0, 2):
        args[3][:, :, int(starts[i])] = float("-inf")
        W0[i], zero[i] = float("nan"), 0.0
        W0[i, :, ::2] = float("inf")
    O, W = cw.ttt_gated_delta(*args, W_init=W0, seq_starts=starts.cuda())
    Or, Wr = cw.ttt_gated_delta(*args, W_init=zero, seq_starts=starts.cuda())
    assert torch.equal(O, Or) and torch.equal(W, Wr) and not O.isnan().any() and torch.equal(W[1], W0[1])
    q, k, v, g, beta, pool = make_step(3, 3, Hk, Hv, dk, dv, dtype)
    g[1] = float("-inf")
    clean = pool.clone()
    pool[1], clean[1] = float("nan"), 0.0
    pool[1, 0] = float("-inf")
    o, c = (cw.ttt_gated_delta_step(q, k, v, g, beta, w) for w in (pool, clean))
    assert torch.equal(o, c) and torch.equal(pool, clean) and not o.isnan().any()


@pytest.mark.parametrize("dtype", DTYPES)
def test_values_that_are_not_finite_stay_in_their_sequence_and_heads(dtype):
    lens, Hk, Hv = [70, 64, 100, 5], 2, 4
    args = make(1, Hk, Hv, sum(lens), 64, 64, dtype, seed=53)
    starts = torch.tensor([0] + lens).cumsum(0).to(torch.int32)
    ref = cw.ttt_gated_delta(*args, seq_starts=starts.cuda())
    at, same = 75, [i for i in range(4) if i != 1]
    inside = torch.zeros(sum(lens), dtype=torch.bool, device="cuda")
    inside[int(starts[1]):int(starts[2])] = True
    for t, heads in ((0, [0, 1]), (1, [0, 1]), (2, [1]), (3, [1]), (4, [1])):      # q and k: both heads that read them
        bad = [x.clone() for x in args]
        bad[t][:, heads[0] if t > 1 else 0, at] = float("nan")
        O, W = cw.ttt_gated_delta(*bad, seq_starts=starts.cuda())
        others = [h for h in range(Hv) if h not in heads]
        assert torch.equal(O[:, others], ref[0][:, others]) and torch.equal(W[:, others], ref[1][:, others])
        assert torch.equal(O[:, :, ~inside], ref[0][:, :, ~inside]) and torch.equal(W[same], ref[1][same])
        assert O[:, heads, at].isnan().any()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("R,P", [(511, 300), (512, 512), (513, 2), (1600, 700), (3000, 2000)])
def test_step_of_many_rows(R, P, dtype):
    """Rows of one state near and far from each other, at the ends of the blocks that are looked through, and padding."""
    gen = torch.Generator().manual_seed(R)
    slots = torch.randint(-1, P, (R,), generator=gen).to(torch.int32)
    for i in (0, 1, 63, 64, 255, 256, 510, 511, 512, 513, 1023, 1024, 1535, 1536, 2559, R - 1):
        if i < R:
            slots[i] = 1
    q, k, v, g, beta, W = make_step(R, P, 1, 1, 16, 8, dtype, seed=R)
    Or, Wr = step_reference(q, k, v, g, beta, W, slots.tolist(), 0.25)
    O = cw.ttt_gated_delta_step(q, k, v, g, beta, W, slots=slots.cuda(), scale=0.25)
    assert rel(O, Or) <= TOL_STEP[dtype] and not O[slots.cuda() < 0].any()
    # a state's roundings of its rows one after the other: 2^-24 times dk a row, which later rows' decays and
    # corrections shrink; the longest run here is R / 2 rows (513 rows on 2 states), whose decays are e^-0.5 on average:
    # less than 3 rows' roundings remain
    assert rel(W, Wr) <= 3 * TOL_STEP[torch.float32]


@pytest.mark.parametrize("full", [False, True])
@pytest.mark.parametrize("Hk,Hv,n,dk,dv", [(2, 4, 300, 128, 128), (1, 3, 200, 64, 72), (2, 2, 130, 96, 80), (1, 2, 700, 128, 136)])
def test_outputs_are_off_by_their_own_rounding(Hk, Hv, n, dk, dv, full):
    """With heads of up to 128, what O is made of is off by no more than the state (test_gpu_delta: c = 2 sqrt(5) 2^-16 of
    its norm), so O is the oracle's rounded to bf16 but where that little moves a value past the middle between two bf16
    numbers: with a share e / u of the values, e the error and u <= 2^-7 of the value a step, which moves them by u.  The
    squares of those moves add up to sum(e u) <= c 2^-7 of O's squares: sqrt(c 2^-7), 7.3e-4, of its norm.  `full`: as a
    row of a batch whose state waves make O themselves."""
    B = -(-520 // Hv) if full else 1
    args = make(B, Hk, Hv, n, dk, dv, torch.bfloat16, seed=71)
    W0 = torch.randn(B, Hv, dv, dk, generator=torch.Generator().manual_seed(72)).mul(0.3).cuda()
    O, _ = cw.ttt_gated_delta(*args, W_init=W0)
    Or, _ = od.delta_rule(*(f64(t[0]) for t in args), dk ** -0.5, f64(W0[0]))
    err = rel(O[0], f64(torch.from_numpy(Or).bfloat16()))
    print("from the rounded oracle", err, flush=True)
    assert err <= (TOL_W[torch.bfloat16] * 2.0 ** -7) ** 0.5
