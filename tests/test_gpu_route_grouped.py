"""moe_route_grouped against a plain implementation in 64 bits: ids equal,
weights within a few roundings of fp32.

Weight tolerance, 16 half steps of fp32 (2^-20): the scores themselves may be
computed in fp32, where exp is off by at most 2 steps (4 half steps), 1 + e and
the quotient by one half step each, the sum of at most 32 scores by 5 (a tree)
and the division and the scale by one each: 13 in all; a softmax's sum over E
adds what its own terms are off by, which its weights divide out."""
import numpy as np
import pytest
import torch

from streamed_quantized_expert_b200 import build, ops, synth
from tests import _ref64 as ref

pytestmark = pytest.mark.gpu
TOL = 16 * ref.U32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    ops.lib()


def dev(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()


def run(logits, k, cfg, bias=None, L=0.0, table=None, ns=0, sw=None, guard=2, stream=None):
    T, E = logits.shape
    d = ops.desc(E, k, 64, 32, 32, 4)
    ids = torch.full((T + guard, k + ns), -7, dtype=torch.int32, device="cuda")
    w = torch.full((T + guard, k + ns), -7.0, device="cuda")
    lg, b, tb, s = dev(logits), dev(bias), dev(table), dev(sw)
    torch.cuda.synchronize()
    ops.moe_route_grouped(lg, T, d, cfg, b, L, tb, ns, s, ids, w, stream)
    torch.cuda.synchronize()
    ids, w = ids.cpu().numpy(), w.cpu().numpy()
    assert (ids[T:] == -7).all() and (w[T:] == -7).all()  # rows behind the last token stay as they were
    return ids[:T], w[:T]


def check(logits, k, score, bias=None, G=1, top=1, gtop=1, renorm=True, scale=1.0, L=0.0, table=None):
    cfg = ops.route_config(score, G, top, gtop, renorm, scale)
    ids, w = run(logits, k, cfg, bias, L, table)
    rid, rw, _ = ref.route(logits, k, score == "sigmoid", bias, G, top, gtop, renorm, scale, L, table)
    assert np.array_equal(ids, rid)
    assert np.all(np.abs(w - rw) <= TOL * np.abs(rw) + 1e-38)
    return ids, w


SHAPES = [  # T, E, k, G, top, gtop
    (1, 1, 1, 1, 1, 1), (3, 2, 2, 2, 1, 1), (1, 8, 2, 1, 1, 1), (5, 31, 7, 1, 1, 1), (7, 33, 32, 1, 1, 1),
    (64, 64, 6, 8, 3, 2), (65, 96, 4, 3, 2, 1), (33, 160, 6, 8, 3, 1), (130, 256, 8, 8, 4, 2),
    (17, 384, 8, 1, 1, 1), (9, 512, 10, 16, 5, 2), (257, 512, 10, 1, 1, 1), (5, 1000, 16, 8, 2, 2),
    (3, 1024, 32, 32, 9, 2), (40, 60, 30, 20, 10, 2), (11, 32, 1, 32, 1, 1),
]


@pytest.mark.parametrize("T,E,k,G,top,gtop", SHAPES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_against_64_bits(T, E, k, G, top, gtop, score):
    if k > top * (E // G):
        k = top * (E // G)
    r = np.random.default_rng(E * 7 + T)
    for step, (bias, renorm, scale, L) in enumerate([(False, True, 1.0, 0.0), (True, True, 2.5, 0.0),
                                                     (True, False, 1.0, 0.125), (False, False, 0.5, 0.125)]):
        logits = synth.router_logits(3, step, T, E)
        b = (0.1 * r.standard_normal(E)).astype(np.float32) if bias else None
        table = np.where(r.random(E) < 0.4, r.integers(0, 50, E), -1).astype(np.int32)
        check(logits, k, score, b, G, top, gtop, renorm, scale, L, table)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_ties(score):
    """Equal logits go to the lower expert; equal group sums to the lower group."""
    E, k = 64, 8
    logits = np.zeros((4, E), np.float32)
    logits[1] = np.round(synth.router_logits(1, 0, 1, E)[0] * 2) / 2
    logits[2, ::2] = 1.0
    logits[3] = -np.arange(E, dtype=np.float32) // 16
    check(logits, k, score)
    check(logits, k, score, np.zeros(E, np.float32), 8, 4, 2)
    check(logits, k, score, np.full(E, 0.25, np.float32), 8, 4, 1)


def test_scores_one_part_in_2_to_the_30_apart():
    """Differences far below fp32's step decide: sigmoid(l) + b with sums that
    round to the same fp32 number, for many pairs."""
    E = 64
    r = np.random.default_rng(0)
    logits = np.full((50, E), -20.0, np.float32)
    bias = np.zeros(E, np.float32)
    bias[:32] = 1.0
    for t in range(50):  # scores below 2^-28 next to a bias of 1
        logits[t, :32] = (-21.0 + 0.25 * r.standard_normal(32)).astype(np.float32)
    ids, _ = check(logits, 16, "sigmoid", bias)
    assert not np.array_equal(ids[0], np.arange(16))


def test_saturated_scores_go_by_the_logit():
    """sigmoid(40 + x) is 1 in 64 bits: the larger logit is still first."""
    logits = np.linspace(60.0, 40.0, 32, dtype=np.float32)[None, ::-1].copy()
    ids, _ = run(logits, 4, ops.route_config("sigmoid"))
    assert ids[0].tolist() == [31, 30, 29, 28]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_experts_that_are_off(score):
    E, k = 32, 4
    r = np.random.default_rng(5)
    logits = r.standard_normal((8, E)).astype(np.float32)
    logits[0, :28] = -np.inf                       # exactly k left
    logits[1, :30] = -np.inf                       # fewer than k: off experts fill up with weight 0
    logits[2] = -np.inf                            # none left
    logits[3, 3] = np.nan                          # a NaN is off
    logits[4] = np.nan
    logits[5, ::2] = np.finfo(np.float32).min      # the type's lowest value is a number
    logits[6] = np.finfo(np.float32).min
    bias = np.linspace(2.0, 3.0, E).astype(np.float32)  # larger than any score
    for b in (None, bias):
        for G, top, gtop in ((1, 1, 1), (4, 2, 1)):
            ids, w = check(logits, k, score, b, G, top, gtop)
            assert all(len(set(x)) == k for x in ids.tolist())
            assert ids.min() >= 0 and ids.max() < E and np.isfinite(w).all()
            assert (w[2] == 0).all() and (w[4] == 0).all()
    ids, w = check(logits, k, score, bias, L=0.5, table=np.arange(E, dtype=np.int32) - 16)


def test_infinite_logits_give_distinct_valid_ids():
    logits = np.zeros((3, 40), np.float32)
    logits[0, 5] = np.inf
    logits[1, :] = np.inf
    logits[2, 7], logits[2, 8] = np.inf, np.nan
    for score in ("softmax", "sigmoid"):
        ids, _ = run(logits, 8, ops.route_config(score), np.zeros(40, np.float32))
        assert all(len(set(x)) == 8 and 0 <= min(x) and max(x) < 40 for x in ids.tolist())


@pytest.mark.parametrize("ns", [1, 8])
def test_shared_experts_follow(ns):
    T, E, k = 5, 64, 6
    logits = synth.router_logits(2, 0, T, E)
    cfg = ops.route_config("sigmoid", 8, 4, 2, True, 2.5)
    sw = np.linspace(0.1, 0.9, T).astype(np.float32)
    for g in (None, sw):
        ids, w = run(logits, k, cfg, None, ns=ns, sw=g)
        rid, rw, _ = ref.route(logits, k, True, None, 8, 4, 2, True, 2.5)
        assert np.array_equal(ids[:, :k], rid) and np.all(np.abs(w[:, :k] - rw) <= TOL * rw)
        assert np.array_equal(ids[:, k:], np.tile(np.arange(E, E + ns), (T, 1)))
        assert np.array_equal(w[:, k:], np.tile((np.ones(T, np.float32) if g is None else sw)[:, None], (1, ns)))


def test_softmax_without_bias_equals_moe_route():
    """The plain softmax router chooses as moe_route does."""
    T, E, k = 70, 512, 10
    logits = synth.router_logits(9, 0, T, E)
    ids, w = run(logits, k, ops.route_config("softmax"))
    d = ops.desc(E, k, 64, 32, 32, 4)
    i2, w2 = torch.empty((T, k), dtype=torch.int32, device="cuda"), torch.empty((T, k), device="cuda")
    ops.moe_route(dev(logits), T, d, 0.0, None, i2, w2)
    torch.cuda.synchronize()
    assert np.array_equal(ids, i2.cpu().numpy())
    assert np.max(np.abs(w - w2.cpu().numpy())) <= 1e-6


def test_another_stream_and_a_replayed_graph():
    T, E, k = 12, 256, 8
    cfg = ops.route_config("sigmoid", 8, 4, 2)
    bias = (0.1 * np.random.default_rng(1).standard_normal(E)).astype(np.float32)
    side = torch.cuda.Stream()
    ids, _ = run(synth.router_logits(4, 0, T, E), k, cfg, bias, stream=side)
    assert np.array_equal(ids, ref.route(synth.router_logits(4, 0, T, E), k, True, bias, 8, 4, 2)[0])
    d = ops.desc(E, k, 64, 32, 32, 4)
    lg, b = torch.zeros((T, E), device="cuda"), dev(bias)
    ids, w = torch.zeros((T, k), dtype=torch.int32, device="cuda"), torch.zeros((T, k), device="cuda")
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=side):
        ops.moe_route_grouped(lg, T, d, cfg, b, 0.0, None, 0, None, ids, w, side)
    for layer in range(3):
        logits = synth.router_logits(4, layer, T, E)
        lg.copy_(dev(logits))
        g.replay()
        torch.cuda.synchronize()
        assert np.array_equal(ids.cpu().numpy(), ref.route(logits, k, True, bias, 8, 4, 2)[0])


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,k,G,top,gtop", [(32, 8, 1, 1, 1), (100, 20, 1, 1, 1), (256, 8, 8, 3, 2), (512, 31, 1, 1, 1),
                                            (512, 32, 4, 2, 2), (1024, 16, 32, 7, 1)])
@pytest.mark.parametrize("L", [0.0, 0.125])
def test_choices_below_fp32(score, E, k, G, top, gtop, L):
    """A bias that takes every token-0 score to 1 up to its own rounding (some
    2^-25): experts and groups are told apart by what fp32 does not hold.  The
    other tokens have some such pairs or none."""
    r = np.random.default_rng(E + k)
    T = 9
    logits = r.standard_normal((T, E)).astype(np.float32)
    l64 = logits[0].astype(np.float64)
    s = 1 / (1 + np.exp(-l64)) if score == "sigmoid" else np.exp(l64 - l64.max()) / np.exp(l64 - l64.max()).sum()
    bias = (1.0 - s).astype(np.float32)
    logits[1, :E // 2] = logits[0, :E // 2]                    # half of the pairs (the softmax's sum is another)
    logits[2] = logits[0][::-1]
    logits[3] = np.nextafter(logits[0], np.float32(9))
    logits[4] = np.float32(0.5)
    table = np.where(r.random(E) < 0.5, r.integers(0, 9, E), -1).astype(np.int32)
    check(logits, k, score, bias, G, top, gtop, True, 1.0, L, table)
    # pairs of equal experts at the border of the choice
    bias[1::2] = bias[::2]
    logits[:, 1::2] = logits[:, ::2]
    check(logits, k, score, bias, G, top, gtop, False, 1.0, L, np.repeat(table[::2], 2)[:E])


@pytest.mark.parametrize("lmax", [1e3, 1e5, 3e38])
def test_large_logits(lmax):
    r = np.random.default_rng(2)
    logits = (lmax * r.uniform(-1, 1, (6, 96))).astype(np.float32)
    for score in ("softmax", "sigmoid"):
        for bias in (None, (0.1 * r.standard_normal(96)).astype(np.float32)):
            for renorm in (True, False):
                check(logits, 5, score, bias, 8, 4, 2, renorm)


def test_logits_at_an_odd_address():
    """Rows that start 4-byte aligned only."""
    T, E, k = 7, 256, 8
    logits = synth.router_logits(8, 0, T, E)
    buf = torch.zeros(T * E + 3, device="cuda")
    buf[3:] = dev(logits).reshape(-1)
    d = ops.desc(E, k, 64, 32, 32, 4)
    ids, w = torch.zeros((T, k), dtype=torch.int32, device="cuda"), torch.zeros((T, k), device="cuda")
    ops.moe_route_grouped(buf[3:], T, d, ops.route_config("sigmoid", 8, 4, 2), None, 0.0, None, 0, None, ids, w)
    torch.cuda.synchronize()
    assert np.array_equal(ids.cpu().numpy(), ref.route(logits, k, True, None, 8, 4, 2)[0])


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,E,k,G,top,gtop", [(40, 64, 24, 1, 1, 1), (17, 512, 32, 1, 1, 1), (33, 128, 30, 8, 4, 2)])
def test_weights_far_below_the_largest(score, renorm, T, E, k, G, top, gtop):
    """A weight keeps its own relative precision: exp(l - max) of a difference
    of a hundred, where an exponent rounded once is off by |x| half steps."""
    logits = 30.0 * synth.router_logits(5, 0, T, E)
    check(logits, k, score, None, G, top, gtop, renorm)
    check(logits - 80.0, k, score, None, G, top, gtop, renorm)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_renormalised_scores_below_fp32(score):
    """A bias that chooses experts whose scores are far below fp32's range:
    they are still renormalised to their sum."""
    E, k = 64, 4
    r = np.random.default_rng(4)
    logits = (synth.router_logits(6, 0, 9, E) - 120.0).astype(np.float32)
    logits[:, :8] = r.uniform(20, 30, (9, 8))
    b = np.where(np.arange(E) < 8, -10.0, 0.0).astype(np.float32)
    b[20:24] = 10.0
    ids, w = check(logits, k, score, b)
    assert (np.sort(ids, axis=1) == np.arange(20, 24)).all() and np.abs(w.sum(axis=1) - 1).max() <= 8 * ref.U32


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("T,E,k,G,top,gtop", [(200, 4, 1, 4, 1, 1), (200, 8, 6, 1, 1, 1), (60, 64, 24, 8, 4, 2),
                                              (60, 256, 32, 1, 1, 1), (40, 48, 32, 1, 1, 1)])
def test_full_substitution_ties_the_lowest_with_the_highest(score, bias, T, E, k, G, top, gtop):
    """L = 1 lifts the lowest score to the highest exactly: the larger logit goes first."""
    r = np.random.default_rng(E)
    b = (0.1 * r.standard_normal(E)).astype(np.float32) if bias else None
    for step, logits in enumerate([synth.router_logits(8, 0, T, E), np.round(synth.router_logits(8, 1, T, E) * 4) / 4]):
        table = np.where(r.random(E) < 0.5, r.integers(0, 50, E), -1).astype(np.int32)
        check(logits.astype(np.float32), k, score, b, G, top, gtop, True, 1.0, 1.0, table)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,k,twins", [(31, 5, 2), (64, 9, 2), (256, 8, 4), (512, 20, 3)])
def test_a_third_expert_behind_twins_at_the_last_place(score, E, k, twins):
    """The last place falls between experts alike in logit and bias, and one that
    differs in both comes within a few steps of fp32 of them: it is compared too."""
    r = np.random.default_rng(E + k)
    T, sig = 96, score == "sigmoid"
    logits = r.uniform(-4, -2, (T, E)).astype(np.float32)
    b = np.zeros(E, np.float32)
    logits[:, :k - 1] = r.uniform(3, 4, (T, k - 1))
    b[:k - 1] = 1.0
    pair, third = np.arange(k - 1, k - 1 + twins), E - 1
    logits[:, pair] = r.uniform(-1, 1, (T, 1))
    b[pair], b[third] = 0.5, 0.5 - 2.0**-9
    for _ in range(30):  # the logit that makes the third's score theirs, then some steps off it
        s = ref.route(logits, k, sig, None)[2]
        want = s[:, pair[0]] + np.float64(b[pair[0]]) - np.float64(b[third])
        if sig:
            logits[:, third] = np.log(want / (1 - want))
        else:
            rest = np.delete(np.exp(logits.astype(np.float64)), third, axis=1).sum(axis=1)
            logits[:, third] = np.log(want * rest / (1 - want))
    steps = np.arange(T) % 9 - 4
    l3 = logits[:, third]
    logits[:, third] = l3 + steps * np.spacing(np.abs(l3)) * np.sign(np.abs(l3))
    assert np.isfinite(logits).all()
    ids, _ = check(logits, k, score, b)
    assert 0 < (ids == third).any(axis=1).sum() < T  # both sides are met


@pytest.mark.parametrize("E,k", [(31, 10), (40, 12), (64, 20)])
def test_full_substitution_with_equal_lowest_scores(E, k):
    r = np.random.default_rng(k)
    for step in range(4):
        logits = (np.round(synth.router_logits(9, step, 340, E) * 4) / 4).astype(np.float32)
        check(logits, k, "softmax", None, 1, 1, 1, False, 2.5, 1.0,
              np.where(r.random(E) < k / E, r.integers(0, 50, E), -1).astype(np.int32))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,k,G,top", [(48, 29, 16, 10), (64, 28, 32, 20), (128, 8, 16, 5), (256, 8, 32, 9)])
def test_groups_equal_over_the_reals(score, E, k, G, top):
    """Few distinct logits: groups' sums are often equal over the reals because
    the same scores, lifts or biases are paired otherwise; the lower group is kept."""
    r = np.random.default_rng(E)
    logits = (np.round(synth.router_logits(10, 0, 300, E) * 2) / 2).astype(np.float32)
    table = np.where(r.random(E) < 0.4, r.integers(0, 50, E), -1).astype(np.int32)
    b = (np.round(r.standard_normal(E)) / 8).astype(np.float32)
    check(logits, k, score, None, G, top, 2, True, 1.0, 0.125, table)
    check(logits, k, score, b, G, top, 2, True, 1.0, 0.0, table)
