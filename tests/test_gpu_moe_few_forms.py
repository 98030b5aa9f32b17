"""The few-token experts through every form that a call can take: one and two tiles of tokens, whole and ragged steps and
several spans of a contraction, up to 64, 256 and 1024 experts, few and many slots.

Whole numbers. With operands of small whole numbers the first product is exact in any order, so its bf16 rounding and the
MXFP8 of h are the oracle's byte for byte, and an expert's output keeps the product's bound 2^-20 sum |h w| before its
share p of the sum, which is within 2^-21 (an exponential of a few ulp, a sum and a division). So
    |y - sum p (h W^T)| <= 2^-7 |y| + 2^-19 sum p sum |h w|."""
import numpy as np
import pytest
import torch

import mxfp8_precision_numerics_amd as mxq
import oracle
from gpu_util import DEV, need_gpu, say
from mxfp8_precision_numerics_amd import workloads
from test_gpu_moe_few import _choice, _mx, _near, _operands, _reference, _values

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,E,k,D,F", [
    (16, 24, 2, 4128, 96),       # one tile of tokens, three spans with a rest
    (13, 24, 2, 6144, 64),       # the same in whole steps, the second product a quarter of a step
    (3, 64, 8, 4096, 2112),      # a slot per (token, rank); both products over two spans
    (50, 24, 1, 4128, 2112),     # two tiles of tokens
    (64, 20, 2, 2048, 2048),     # the same, one span each
    (40, 200, 2, 2080, 96),      # more than 64 experts
    (17, 300, 1, 96, 4160),      # more than 256
    (2, 8, 4, 4128, 2112),       # few slots: two waves a slot in the second product
    (3, 70, 5, 2080, 96),        # few slots, more than 64 experts, most waves with one slot
    (12, 3, 3, 96, 160),         # few slots, a slot per expert: every wave's rows hold the same tokens
])
def test_whole_numbers_in_every_form(T, E, k, D, F):
    need_gpu()
    say("few-token experts, whole numbers", T, E, k, D, F)
    rng = np.random.default_rng(T + D)
    whole = lambda *s: torch.from_numpy(rng.integers(-2, 3, s).astype(np.float32)).to(torch.bfloat16).to(DEV)  # noqa: E731
    x, up, down = _mx(whole(T, D)), _mx(whole(E, 2 * F, D)), _mx(whole(E, D, F))
    logits = workloads.normal_f32((T, E), 1.0, 53, T, DEV)
    y = mxq.moe_mx_few_tokens(*x, logits, k, *up, *down)
    torch.cuda.synchronize()
    got, xv = y.double().cpu().numpy(), _values(*x)
    lg = logits.cpu().numpy().astype(np.float64)
    want, room = np.zeros((T, D)), np.zeros((T, D))
    chosen = _choice(lg, k)
    for e in sorted({e for c in chosen for e in c}):
        tok = [t for t in range(T) if e in chosen[t]]
        c = oracle.bf16_from_f32((xv[tok] @ _values(up[0][e], up[1][e]).T).astype(np.float32))
        q, s, _ = oracle.swiglu_mx_quantize(c)
        h = oracle.fp8_value(q, oracle.E4M3) * np.repeat(np.ldexp(1.0, s.astype(np.int64) - 127), 32, axis=1)
        w = _values(down[0][e], down[1][e])
        for i, t in enumerate(tok):
            l = lg[t][chosen[t]]
            p = np.exp(lg[t][e] - l.max()) / np.exp(l - l.max()).sum()
            want[t] += p * (w @ h[i])
            room[t] += p * (np.abs(w) @ np.abs(h[i]))
    assert np.all(np.abs(got - want) <= 2.0 ** -7 * np.abs(want) + 2.0 ** -19 * room)


@pytest.mark.parametrize("T,E,k,D,F", [(3, 64, 8, 2048, 1024), (6, 256, 8, 1056, 544), (16, 64, 8, 2048, 1024),
                                       (20, 200, 6, 544, 1056), (40, 24, 3, 2048, 512)])
def test_a_token_does_not_depend_on_its_place_in_the_batch(T, E, k, D, F):
    """With more than 16 slots: the batch in another order gives the same rows in that order, byte for byte."""
    need_gpu()
    say("few-token experts, order of the batch", T, E, k, D, F)
    x, up, down = (_mx(workloads.normal_bf16(s, v, 53, 300 + i, DEV)) for i, (s, v) in enumerate(
        [((T, D), 1.0), ((E, 2 * F, D), 0.02), ((E, D, F), 0.02)]))
    logits = workloads.normal_f32((T, E), 1.5, 53, 310, DEV)
    y = mxq.moe_mx_few_tokens(*x, logits, k, *up, *down)
    for order in (torch.arange(T).flip(0), torch.arange(T).roll(1), torch.from_numpy(np.random.default_rng(T).permutation(T))):
        o = order.to(DEV)
        z = mxq.moe_mx_few_tokens(x[0][o].contiguous(), x[1][o].contiguous(), logits[o].contiguous(), k, *up, *down)
        torch.cuda.synchronize()
        assert torch.equal(z.view(torch.int16), y[o].contiguous().view(torch.int16))


@pytest.mark.parametrize("T,E,k,D,F", [(2, 24, 8, 512, 256), (2, 17, 8, 2048, 1024), (5, 18, 3, 544, 96), (8, 20, 2, 256, 1056),
                                       (4, 16, 4, 512, 256)])
def test_place_in_the_batch_with_few_slots(T, E, k, D, F):
    """The same with at most 16 slots; all tokens ask for much the same experts, in different orders."""
    need_gpu()
    say("few-token experts, order of the batch, few slots", T, E, k, D, F)
    x, up, down = (_mx(workloads.normal_bf16(s, v, 53, 320 + i, DEV)) for i, (s, v) in enumerate(
        [((T, D), 1.0), ((E, 2 * F, D), 0.02), ((E, D, F), 0.02)]))
    for rep in range(8):
        logits = workloads.normal_f32((T, E), 0.5, 53, 330 + rep, DEV)
        logits[:, : k + 1] += 4.0
        y = mxq.moe_mx_few_tokens(*x, logits, k, *up, *down)
        for o in (torch.arange(T, device=DEV).flip(0), torch.arange(T, device=DEV).roll(1)):
            z = mxq.moe_mx_few_tokens(x[0][o].contiguous(), x[1][o].contiguous(), logits[o].contiguous(), k, *up, *down)
            torch.cuda.synchronize()
            assert torch.equal(z.view(torch.int16), y[o].contiguous().view(torch.int16)), rep


@pytest.mark.parametrize("T,E,k,D,F,normalize", [
    (1, 128, 8, 2048, 1024, True), (1, 256, 8, 544, 160, False), (2, 256, 8, 512, 96, True), (16, 200, 1, 544, 256, True),
    (16, 200, 1, 512, 96, False),                                  # up to 16 slots, 65 to 256 experts
    (1, 520, 4, 544, 96, True), (2, 1024, 8, 96, 160, False),      # up to 16 slots, more
    (4, 130, 8, 512, 256, True), (12, 256, 3, 544, 96, False),     # streaming, one tile, 65 to 256 experts
    (20, 300, 4, 512, 128, True), (33, 1000, 3, 96, 96, False), (64, 260, 2, 288, 64, True),   # two tiles, more than 256
    (6, 600, 7, 512, 64, True),
])
def test_many_experts(T, E, k, D, F, normalize):
    """The tolerance of test_gpu_moe_few.py, against its plain form."""
    need_gpu()
    say("few-token experts, many experts", T, E, k, D, F, normalize)
    x, up, down, logits = _operands(T, E, D, F, 30 + k)
    y = mxq.moe_mx_few_tokens(*x, logits, k, *up, *down, normalize=normalize)
    torch.cuda.synchronize()
    _near(y, _reference(x, up, down, logits, k, normalize), F)


@pytest.mark.parametrize("T,E,k", [(3, 64, 8), (20, 16, 4), (2, 100, 5), (7, 90, 6), (5, 12, 12), (2, 300, 3)])
@pytest.mark.parametrize("normalize", [True, False])
def test_masks_over_chosen_and_all_logits(T, E, k, normalize):
    """Masks that leave fewer than k experts or none, the lowest finite logit, ties, a NaN and a +inf, with the weights taken
    over the chosen logits and over all of them."""
    need_gpu()
    say("few-token experts, masks", T, E, k, normalize)
    D, F = 160, 96
    x, up, down, _ = _operands(T, E, D, F, 40)
    inf, low = float("inf"), torch.finfo(torch.float32).min
    logits = workloads.normal_f32((T, E), 1.5, 53, 78, DEV)
    kinds = {"few left": lambda l: (l[0].fill_(-inf), l[0, E - 1:].fill_(0.5), l[1, : E - 2].fill_(-inf)),
             "none left": lambda l: (l[0].fill_(-inf), l[T - 1].fill_(-inf)),
             "nobody": lambda l: l.fill_(-inf),
             "lowest": lambda l: (l[0].fill_(low), l[1, 1:].fill_(low)),
             "mask and lowest": lambda l: (l[0].fill_(-inf), l[0, 3:5].fill_(low)),
             "ties": lambda l: (l.fill_(1.0), l[1, ::2].fill_(2.0)),
             "far apart": lambda l: (l[0].fill_(-3e38), l[0, 2:3].fill_(3e38)),
             "nan": lambda l: l[1, E // 2:E // 2 + 1].fill_(float("nan")),
             "inf": lambda l: (l[0, :1].fill_(inf), l[1, E - 1:].fill_(-inf))}
    for kind, change in kinds.items():
        l = logits.clone()
        change(l)
        y = mxq.moe_mx_few_tokens(*x, l, k, *up, *down, normalize=normalize)
        torch.cuda.synchronize()
        say(kind)
        with np.errstate(invalid="ignore"):
            want = _reference(x, up, down, l, k, normalize)
        _near(y, want, F)
        for t, c in enumerate(_choice(l.cpu().numpy(), k)):
            assert c != [] or bool((y[t] == 0).all())


@pytest.mark.parametrize("T,E,k", [(2, 8, 2), (12, 8, 2), (16, 24, 2), (40, 24, 3), (2, 100, 4)])
def test_nan_and_infinite_operands_stay_where_they_are(T, E, k):
    """A NaN or an infinity in a token's x makes that token's row NaN; a NaN in an up weight, the rows of the tokens that chose
    its expert; one in a down weight, its column of those rows. Every other value keeps its bytes."""
    need_gpu()
    say("few-token experts, NaN", T, E, k)
    D, F = 288, 96
    x, up, down, logits = _operands(T, E, D, F, 50)
    clean = mxq.moe_mx_few_tokens(*x, logits, k, *up, *down)
    chosen = _choice(logits.cpu().numpy(), k)
    e, victim = chosen[0][k - 1], T // 2
    near_e = torch.tensor([e in c for c in chosen], device=DEV)

    def planted(pair, at, value):
        q, s = pair[0].clone(), pair[1].clone()
        v = torch.zeros((1, 32), dtype=torch.bfloat16, device=DEV)
        v[0, at[-1] % 32] = value
        m = mxq.mx_quantize(v, colwise=False)
        b = at[-1] // 32
        q[at[:-1]][32 * b:32 * b + 32] = m.q_row[0]
        s[at[:-1]][b] = m.s_row[0, 0]
        return q, s

    nan, rows = float("nan"), torch.arange(T, device=DEV)
    for name, args, bad in (
            ("x nan", (planted(x, (victim, 37), nan), up, down), (rows == victim)[:, None].expand(T, D)),
            ("x inf", (planted(x, (victim, 280), float("inf")), up, down), (rows == victim)[:, None].expand(T, D)),
            ("up gate nan", (x, planted(up, (e, 5, 287), nan), down), near_e[:, None].expand(T, D)),
            ("up nan", (x, planted(up, (e, F + 70, 0), nan), down), near_e[:, None].expand(T, D)),
            ("down nan", (x, up, planted(down, (e, 133, 95), nan)),
             near_e[:, None] & (torch.arange(D, device=DEV) == 133)[None])):
        say(name)
        y = mxq.moe_mx_few_tokens(*args[0], logits, k, *args[1], *args[2])
        torch.cuda.synchronize()
        assert torch.equal(torch.isnan(y), bad)
        assert torch.equal(y[~bad].view(torch.int16), clean[~bad].view(torch.int16))
