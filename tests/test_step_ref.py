"""The 64-bit forms of tests/step_ref.py against closed forms and worked cases."""
import numpy as np
import pytest
import torch

from tests import step_ref as ref


def test_e4m3_table_is_torchs():
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(np.isnan(t), np.isnan(ref.TABLE))
    assert np.array_equal(t[~np.isnan(t)], ref.TABLE[~np.isnan(t)])


def test_nearest_is_nearest_and_ties_are_even():
    held = [b for b in range(127) if (4 * ref.TABLE[b]).is_integer()]
    grid = ref.TABLE[held]
    assert np.array_equal(grid[:17], np.arange(17) / 4) and len(held) == 17 + 8 * 6 + 6
    assert np.array_equal(ref.nearest_e4m3(grid), held)
    mid = (grid[:-1] + grid[1:]) / 2
    got = ref.nearest_e4m3(mid)
    n = np.array([grid[1 + i] / (grid[1 + i] - grid[i]) for i in range(len(mid))])
    even = np.where(n % 2 == 0, held[1:], held[:-1])        # the even multiple of the step
    assert np.array_equal(got, even)
    assert np.array_equal(ref.nearest_e4m3(np.nextafter(mid, 0)), held[:-1])
    assert np.array_equal(ref.nearest_e4m3(np.nextafter(mid, 1e9)), held[1:])
    assert ref.nearest_e4m3(np.array([1e30]))[0] == 126


def test_block_scale_and_order():
    v = np.zeros((1, 544))
    v[0, 0], v[0, 40], v[0, 130], v[0, 512] = 1.0, 300.0, 2.0 ** -130, np.inf
    code, e = ref.encode8(v)
    assert list(e[0, [0, 1, 4, 16]]) == [119, 127, 0, 255] and e[0, 2] == 0
    assert ref.decode8(code, e)[0, 0] == 1.0 and ref.decode8(code, e)[0, 40] == 288.0 + 0
    rows = ref.scale_rows(e)
    assert rows.shape == (1, 32)
    # block 1 of group 0, block 0 of group 1, the first block of the second 512
    assert rows[0, 4] == 127 and rows[0, 1] == 0 and rows[0, 16] == 255 and rows[0, 31] == 127


def test_route_by_hand():
    l = np.array([[0.0, 1.0, 1.0, -np.inf]])
    e, s = ref.route(l, 3, renorm=False)
    assert list(e[0]) == [1, 2, 0]
    assert np.allclose(s[0], np.exp([1, 1, 0]) / (2 * np.e + 1))
    e, s = ref.route(l, 4)
    assert list(e[0]) == [1, 2, 0, -1] and s[0, 3] == 0 and np.isclose(s.sum(), 1)
    # two groups: the first has the largest, the second the larger sum of two
    l = np.array([[3.0, -3.0, 2.0, 2.0]])
    assert ref.route(l, 1, "sigmoid", groups=2, kept=1, terms=1)[0][0, 0] == 0
    assert ref.route(l, 1, "sigmoid", groups=2, kept=1, terms=2)[0][0, 0] == 2
    # the bias chooses, the score counts
    e, s = ref.route(l, 1, "sigmoid", bias=np.array([0, 1.0, 0, 0]), renorm=False)
    assert e[0, 0] == 1 and np.isclose(s[0, 0], 1 / (1 + np.exp(3.0)))


@pytest.mark.parametrize("with_probs", [False, True])
def test_verified_tokens_follow_the_targets_distribution(with_probs):
    """Whatever the drafter draws from, the first token out is distributed as the
    target's: 40000 sequences, every frequency within six standard deviations."""
    rng = np.random.default_rng(5)
    n, V = 40000, 5
    target, guess = rng.normal(size=V), rng.dirichlet(np.ones(V))
    p = np.exp(target) / np.exp(target).sum()
    drafts = rng.choice(V, size=(n, 1), p=guess) if with_probs else np.full((n, 1), 2)
    q = np.broadcast_to(guess, (n, 1, V)) if with_probs else None
    logits = np.broadcast_to(target, (n, 2, V))
    tokens, _ = ref.verify(logits, drafts, rng.random((n, 2)), q)
    f = np.bincount(tokens[:, 0], minlength=V) / n
    assert np.all(np.abs(f - p) <= 6 * np.sqrt(p * (1 - p) / n))
