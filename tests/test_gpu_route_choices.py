"""Choices of the routing that hang on how its keys and its groups' keys are made, ids against the 64-bit oracle.

Every row is checked in batches of three lengths, which reach the kernel's three ways of dealing lanes to tokens."""
import numpy as np
import pytest

import moe_expert_load_ultraep_amd as U
import oracle.layer_oracle as Y
from test_gpu_layer import ctx_of, dev, host, logits_of, weight_slack

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
DEV = "cuda"
BATCHES = (24, 6000, 40000)
INF, NAN = np.inf, np.nan


def check(x, k, bf16=False, bias=None, batches=BATCHES, **kw):
    """The rows x again and again to the batch's length; the oracle's ids of each."""
    l, v = logits_of(x, bf16)
    b = None if bias is None else np.asarray(bias, dtype=np.float32)
    idx_kw = dict(groups=kw.get("groups", 1), topk_groups=kw.get("topk_groups", 1), group_top=kw.get("group_top", 1))
    score, renorm = kw.get("score", 0), kw.get("renormalize", True)
    want, want_w = Y.route(v, k, bool(score), b, renorm=renorm, **idx_kw)
    slack = weight_slack(v, want, score, renorm)[:, None] * want_w + 2.0 ** -120
    for tokens in batches:
        times = -(-tokens // len(v))
        many = l.repeat(times, 1)[:tokens].contiguous()
        idx = torch.full((tokens, k), -77, dtype=torch.int32, device=DEV)
        w = torch.full((tokens, k), -7.0, device=DEV)
        U.ultraep_route(ctx_of(l.shape[1]), many, k, idx, w, bias=None if b is None else dev(b), **kw)
        got, rows = host(idx), np.arange(tokens) % len(v)
        wrong = (got != want[rows]).any(axis=1)
        assert not wrong.any(), (tokens, int(wrong.sum()), v[rows[wrong][0]].tolist(), got[wrong][0].tolist(), want[rows[wrong][0]].tolist())
        assert (np.abs(host(w) - want_w[rows]) <= slack[rows]).all()
    return want


# ---------------------------------------------------------------- bf16 logits, sums of two scores

def test_two_scores_of_negative_bf16_logits_by_hand():
    """sigmoid(0.5) + sigmoid(-20) = 0.62246 against sigmoid(0) + sigmoid(-1.96875) = 0.62253."""
    x = np.array([[0.5, -20.0, 0.0, -1.96875]])
    assert check(x, 1, bf16=True, score=1, groups=2, topk_groups=1, group_top=2).tolist() == [[2]]


@pytest.mark.parametrize("E,groups,taken", [(16, 8, 2), (60, 10, 8), (128, 8, 4), (160, 8, 3), (256, 8, 4), (512, 16, 5)])
@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("mean", [-3.0, 0.0])
def test_two_scores_of_bf16_logits(E, groups, taken, score, mean):
    rng = np.random.default_rng(E)
    check(rng.standard_normal((400, E)) + mean, min(8, E), bf16=True, score=score, groups=groups, topk_groups=taken, group_top=2)


# ---------------------------------------------------------------- groups with one expert left beside groups with more

def alone(rng, E, groups, rows=400):
    """Rows in which some groups keep one expert, some two and some all, the others none."""
    per = E // groups
    x = rng.standard_normal((rows, E)) * 1.3
    keep = rng.choice([0, 1, 1, 2, per], size=(rows, groups))
    place = np.argsort(rng.random((rows, groups, per)), axis=2)
    gone = (place >= keep[:, :, None]).reshape(rows, E)
    return np.where(gone, rng.choice([-INF, NAN], size=(rows, E)), x)


def test_a_group_with_one_expert_left_by_hand():
    """0.9003 alone against 0.4013 twice: less the smallest bias, -0.3, once and twice."""
    x = np.array([[2.2, -INF, -INF, -INF] + [-0.4] * 4 + [-0.6] * 4 + [-5.0] * 4])
    bias = np.zeros(16)
    bias[12] = -0.3
    assert check(x, 2, bias=bias, score=1, groups=4, topk_groups=1, group_top=2).tolist() == [[0, -1]]


@pytest.mark.parametrize("E,groups,taken", [(16, 4, 1), (16, 8, 3), (60, 10, 4), (64, 16, 5), (128, 8, 4), (160, 8, 3), (256, 8, 4), (512, 16, 5)])
@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("shift", [0.0, 1.0, -1.0, 40.0, -300.0])
def test_groups_with_one_expert_left(E, groups, taken, score, shift):
    rng = np.random.default_rng(E + groups)
    bias = shift + rng.standard_normal(E) * 0.1
    how = dict(score=score, groups=groups, topk_groups=taken, group_top=2)
    for bf16 in (False, True):
        check(alone(rng, E, groups), 4, bf16=bf16, bias=bias, **how)
    # by the bias: the first group keeps one expert, the second none, the third two
    per = E // groups
    if per > 2:
        bias[1:per], bias[per:2 * per], bias[2 * per + 2:3 * per] = -INF, NAN, -INF
    else:
        bias[1], bias[2:4] = -INF, NAN
    check(rng.standard_normal((400, E)) * 1.3, 4, bias=bias, **how)


# ---------------------------------------------------------------- fp32 logits more than 16 below the row's largest

def test_a_second_score_far_below_the_largest_logit_by_hand():
    """Sums of two scores: 0.99995 and 0.99995 + 0.0015; 1 and 2^-7.2 each but for a far smaller term."""
    x = np.array([[10.0, -100.0, 9.9, -6.5]])
    assert check(x, 1, score=1, groups=2, topk_groups=1, group_top=2).tolist() == [[2]]
    x = np.array([[10.0, 0.0, 5.0, -100.0, 5.0, -6.5, 0.0, 0.0]])
    assert check(x, 2, score=0, groups=4, topk_groups=2, group_top=2).tolist() == [[0, 4]]


@pytest.mark.parametrize("E,groups,taken", [(8, 4, 2), (16, 4, 1), (64, 16, 5), (96, 6, 2), (128, 8, 4), (160, 8, 3), (256, 8, 4), (512, 16, 5)])
@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("top", [1, 2])
@pytest.mark.parametrize("spread,mean", [(20.0, 0.0), (20.0, -30.0), (60.0, 10.0), (6.0, 0.0)])
def test_logits_of_a_wide_spread(E, groups, taken, score, top, spread, mean):
    """Some groups have the same best, and seconds that lie far below or are masked."""
    rng = np.random.default_rng(E + groups)
    x = rng.standard_normal((300, E)) * spread + mean
    per = E // groups
    for t in range(0, 300, 2):
        a, b = rng.choice(groups, 2, replace=False)
        best = x[t].max() - rng.choice([0.0, 3.0, 8.0, 15.0, 20.0])
        x[t, a * per:(a + 1) * per] = best - 16 - rng.random(per) * 20
        x[t, b * per:(b + 1) * per] = best - 16 - rng.random(per) * 20
        x[t, a * per] = best
        x[t, b * per + per - 1] = best - rng.choice([0.0, 1e-6, 1e-4])
        if t % 8 == 0:
            x[t, b * per:(b + 1) * per - 1] = rng.choice([-INF, NAN])
    check(x, min(4, E), score=score, groups=groups, topk_groups=taken, group_top=top)


# ---------------------------------------------------------------- large biases

@pytest.mark.parametrize("size", [700.0, -5e3, 6e4, 1e6, -1e7, 1e10, -3e30])
@pytest.mark.parametrize("E,groups,taken,top", [(32, 1, 1, 1), (60, 4, 2, 2), (128, 8, 4, 1), (160, 8, 3, 2), (256, 8, 4, 2), (400, 8, 3, 2)])
@pytest.mark.parametrize("score", [0, 1])
def test_biases_that_are_large(E, groups, taken, top, score, size):
    """Scores plus bias tie in 64 bits, or nearly so: the lower id, and the lower group, go first there."""
    rng = np.random.default_rng(E)
    x = rng.standard_normal((200, E)) * rng.choice([1.0, 12.0], size=(200, 1))
    x[::5] = np.round(x[::5])
    how = dict(score=score, groups=groups, topk_groups=taken, group_top=top)
    for bias in (np.full(E, size), size + rng.integers(0, 4, E) * max(1.0, abs(size) * 2.0 ** -22), size + rng.standard_normal(E) * 50,
                 np.where(rng.random(E) < 0.2, size, rng.standard_normal(E) * 0.05)):
        check(x, min(8, E), bias=bias, **how)


# ---------------------------------------------------------------- sums of two scores that differ by one rounding

def test_two_scores_that_differ_by_less_than_the_sum_of_exponentials_shows():
    """Not normalised, 1 + e^-37 and 1 + e^-47 both round to 1; over the sum, 2 + e^-22.75, the first is the larger."""
    x = np.array([[0.0, -47.0, 0.0, -37.0, -22.75, -100.0]])
    for bf16 in (False, True):
        assert check(x, 1, bf16=bf16, score=0, groups=3, topk_groups=1, group_top=2).tolist() == [[2]]
    x = np.array([[0.0, -40.0, 0.0, -40.0, -22.75, -100.0]])   # the same: the lower group
    for bf16 in (False, True):
        assert check(x, 1, bf16=bf16, score=0, groups=3, topk_groups=1, group_top=2).tolist() == [[0]]


@pytest.mark.parametrize("E,groups,taken", [(16, 4, 1), (128, 8, 4), (160, 8, 3), (512, 16, 5)])
def test_two_scores_of_equal_pairs(E, groups, taken):
    """Pairs of the same two logits, and of one alone, in several groups: the lower group; a coarse grid of values."""
    rng = np.random.default_rng(E)
    x = np.round(rng.standard_normal((300, E)) * 3) / 2
    per = E // groups
    for t in range(0, 300, 3):
        best = x[t].max() + 1.0
        for g in rng.choice(groups, taken + 1, replace=False):
            x[t, g * per:g * per + 2] = rng.permutation([best, best - 0.5]) if t % 2 else [best, -INF]
            if not t % 2:
                x[t, g * per + 1:(g + 1) * per] = -INF
    for bf16 in (False, True):
        for score in (0, 1):
            check(x, 4, bf16=bf16, score=score, groups=groups, topk_groups=taken, group_top=2)


# ---------------------------------------------------------------- every width, list and way of dealing lanes

@pytest.mark.parametrize("E,groups,taken", [(20, 5, 3), (32, 4, 2), (64, 8, 3), (128, 8, 4), (144, 9, 4), (160, 8, 3), (250, 5, 2), (256, 8, 4), (384, 12, 5),
                                            (512, 16, 7)])
@pytest.mark.parametrize("k", [3, 8, 12])
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("score", [0, 1])
def test_widths_and_lists(E, groups, taken, k, bf16, score):
    rng = np.random.default_rng(E + k)
    for spread in (1.3, 25.0):
        x = rng.standard_normal((70, E)) * spread
        x[rng.random((70, E)) < 0.1] = -INF
        for bias in (None, rng.standard_normal(E) * 0.05):
            check(x, k, bf16=bf16, bias=bias, score=score, renormalize=spread < 2)
            for top in (1, 2):
                check(x, k, bf16=bf16, bias=bias, score=score, groups=groups, topk_groups=taken, group_top=top, renormalize=spread > 2)
