"""GPU parity of moe_route_scored where its quick decisions are nearest to going wrong.

A wave that meets one row it is not sure of decides all of its rows in 64 bits,
so the rows here are launched one by one, or with rows of their own kind only:
each takes the path that it takes by itself.  Choices are compared with the
fp64 oracle (equal); the bounds of the weights are those of
tests/test_gpu_route_scored.py.
"""
import numpy as np
import pytest

from oracle import scored_fp8 as S
from tests.gpu_util import need_gpu
from tests.test_gpu_route_scored import _logits, _run, _weight_bound

pytestmark = pytest.mark.gpu


def _compare(x, bias, k, sigmoid, groups, renorm, dev):
    _, idx, w = _run(x, bias, k, sigmoid, *groups, renorm, 1.0, dev)
    ri, rw = S.route_scored(x, bias, k, sigmoid, *groups, renorm)
    assert np.array_equal(idx.cpu().numpy(), ri), (idx.cpu().numpy()[:4], ri[:4])
    got = w.cpu().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(rw))
    ok = ~np.isnan(rw)
    bound = np.broadcast_to(_weight_bound(x, sigmoid, renorm, k), rw.shape)
    # below 2^-126 an fp32 weight has fewer bits, or is flushed to 0
    assert (np.abs(got - rw)[ok] <= (bound * rw)[ok] + 2.0 ** -126).all()


@pytest.mark.parametrize("sigmoid", [True, False], ids=["sigmoid", "softmax"])
@pytest.mark.parametrize("size", [2, 5])
@pytest.mark.parametrize("big", [1.0, 64.0, 1e4, 1e7, 2e38])
def test_group_sums_of_large_biases_of_both_signs(big, size, sigmoid):
    """A group's two best choices almost cancel (2e38: overflow in 32 bits): the sum's error is that of its addends."""
    dev = need_gpu()
    T, G, k = 96, 8, 3
    r = np.random.Generator(np.random.PCG64(int(np.log2(big)) + size))
    x = (1.0 + r.standard_normal((T, G * size)) * 1e-3).astype(np.float32)
    bias = np.full((G, size), -np.float32(3e38), np.float32)
    if big < 1e38:
        bias[:, 0], bias[:, 1] = big, -big
        bias[::3] = 0                                          # groups without cancellation among them
        bias[::3, 2:] = -np.float32(3e38)
    else:
        bias[:, 0], bias[:, 1] = big, big * np.linspace(0.9, 1.0, G)
    perm = r.permutation(size)
    for t0 in (0, 48):
        _compare(x[t0:t0 + 48], bias[:, perm].reshape(-1).copy(), k, sigmoid, (G, 4, 2), True, dev)
    for t in range(8):
        _compare(x[t:t + 1], bias.reshape(-1), k, sigmoid, (G, 3, 2), False, dev)


@pytest.mark.parametrize("sigmoid", [True, False], ids=["sigmoid", "softmax"])
def test_group_sums_next_to_a_group_of_large_addends(sigmoid):
    """The error of one group's sum decides about another whose own is small."""
    dev = need_gpu()
    G, k = 8, 2
    r = np.random.Generator(np.random.PCG64(9))
    x = (r.standard_normal((64, G * 2)) * 0.5).astype(np.float32)
    s = S.scores(x, sigmoid).reshape(64, G, 2)
    for keep in (1, 4, 7):
        for t in range(64):
            bias = np.zeros((G, 2), np.float32)
            g = int(r.integers(0, G))
            sums = np.sort(np.delete(s[t].sum(1), g))
            near = sums[int(r.integers(0, G - 1))]            # the large group's sum lands next to another's
            lift = np.float32(near - s[t, g].sum())
            bias[g, 0], bias[g, 1] = 512.0 + lift, -512.0
            _compare(x[t:t + 1], bias.reshape(-1), k, sigmoid, (G, keep, 2), True, dev)


ROWS = ["masked", "lowest", "three left", "five left", "half masked", "saturated", "small scores", "two NaN", "all NaN",
        "tiny scores", "one infinite", "group left", "all infinite", "infinite in the last group"]


def _special(name, E, x):
    low = np.finfo(np.float32).min
    if name == "masked":
        x[:] = -np.inf
    elif name == "lowest":
        x[:] = low
    elif name == "three left":
        x[3:] = -np.inf
    elif name == "five left":
        x[5:] = low
    elif name == "half masked":
        x[::2] = -np.inf
    elif name == "saturated":
        x[:] = np.linspace(30, 90, E)
    elif name == "small scores":
        x[:] = np.linspace(-90, -30, E)
    elif name == "two NaN":
        x[[1, 9]] = np.nan
    elif name == "all NaN":
        x[:] = np.nan
    elif name == "tiny scores":
        x[:] = np.linspace(-300, -200, E)
    elif name == "one infinite":
        x[6] = np.inf
    elif name == "group left":
        x[:3 * E // 4] = -np.inf
    elif name == "all infinite":
        x[:] = np.inf
    else:
        x[E - 1] = np.inf
    return x


@pytest.mark.parametrize("sigmoid", [True, False], ids=["sigmoid", "softmax"])
@pytest.mark.parametrize("groups", [(1, 1, 1), (4, 2, 2), (4, 2, 1), (4, 1, 2)],
                         ids=["whole", "groups-top2", "groups-top1", "one-group"])
@pytest.mark.parametrize("biased", [True, False], ids=["bias", "plain"])
@pytest.mark.parametrize("name", ROWS)
def test_special_rows_by_themselves(name, biased, groups, sigmoid):
    """Each row alone, and behind rows that the quick path is sure of."""
    dev = need_gpu()
    for E, k in ((16, 4), (64, 3)):
        x, r = _logits(9, E, 2 + E)
        bias = (r.standard_normal(E) * 0.1).astype(np.float32) if biased else None
        row = _special(name, E, x[1].copy())
        for renorm in (True, False):
            _compare(row[None], bias, k, sigmoid, groups, renorm, dev)
            y = x[1:].copy()
            y[5] = row
            _compare(y, bias, k, sigmoid, groups, renorm, dev)


# E, k, n_group, topk_group, group_top: with more than 2048 tokens a lane holds up to 8 experts and a token 8 to 64 lanes
MANY = [(64, 4, 1, 1, 1), (128, 8, 1, 1, 1), (256, 8, 8, 4, 2), (256, 6, 8, 3, 1), (160, 6, 8, 3, 2), (24, 2, 3, 1, 2),
        (512, 10, 1, 1, 1), (1020, 9, 17, 5, 2), (37, 32, 1, 1, 1)]


@pytest.mark.parametrize("sigmoid", [True, False], ids=["sigmoid", "softmax"])
@pytest.mark.parametrize("biased", [True, False], ids=["bias", "plain"])
@pytest.mark.parametrize("case", MANY, ids=["E%d-k%d-g%d-%d-top%d" % c for c in MANY])
def test_more_than_2048_tokens(case, biased, sigmoid):
    """The same rows as in launches of fewer, special ones among them, over the last block's end."""
    dev = need_gpu()
    E, k, ng, tg, gt = case
    T = 2049 + E % 7
    x, r = _logits(T, E, 7 * E + k)
    for i, name in enumerate(ROWS):
        if E > 9:
            x[100 * i + 3] = _special(name, E, x[100 * i + 3].copy())
    x[1600:1700] = (1 + r.standard_normal((100, E)) * 3e-3).astype(np.float32)
    bias = (r.standard_normal(E) * (0.1 if E % 8 else 64.0)).astype(np.float32) if biased else None
    for renorm in (True, False):
        _compare(x, bias, k, sigmoid, (ng, tg, gt), renorm, dev)
