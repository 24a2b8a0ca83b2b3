"""Token log-probabilities of rows in which a grammar or a filter leaves few tokens (GPU).

Where fewer than top_k logits are above the mask, the rest of the top is masked tokens, lowest ids first: ids and
-inf are compared exactly, values at the bounds of test_logprobs_gpu.  Rows run one to a warp, one to a CTA and one
to a cluster of CTAs, by their number and length."""
import numpy as np
import pytest

import synth
from _packed import U32, store
from test_logprobs_gpu import _check, _reference, _run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lb():
    import decoder_block_gb300 as m
    m.load()
    return m


# (rows, vocabulary): a warp per row, a CTA per row, clusters of two to eight CTAs per row
SHAPES = [(6000, 700), (3, 4000), (5, 7999), (2, 16500), (3, 33001), (2, 128256)]
LEFT = [(1, 2), (1, 32), (3, 5), (12, 20), (16, 32), (31, 32), (32, 32), (40, 20)]


def _rows(tag, T, V, left, mask):
    """`left` logits of each row at random places, `mask` elsewhere; targets in turn allowed and masked."""
    rng = np.random.default_rng(tag)
    x = np.full((T, V), mask, np.float32)
    at = np.argsort(rng.random((T, V)), axis=1)[:, :left + 1]
    x[np.arange(T)[:, None], at[:, :left]] = rng.normal(0, 2.5, (T, left))
    return x, np.where(np.arange(T) % 2 == 0, at[:, 0], at[:, left])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,V", SHAPES)
@pytest.mark.parametrize("left,k", LEFT)
def test_few_tokens_left(lb, dtype, T, V, left, k):
    x, y = _rows(left * 64 + k, T, V, left, -np.inf)
    _check(lb, store(x, dtype), V, V, y, k)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,V", SHAPES)
@pytest.mark.parametrize("left,k", [(1, 2), (3, 5), (16, 32)])
def test_few_tokens_left_above_the_lowest_value(lb, dtype, T, V, left, k):
    """A mask of the type's lowest finite value: such logits count, at weight 0 and at their own distance."""
    lowest = np.finfo(np.float32).min if dtype == "f32" else -(2.0 - 2.0 ** -7) * 2.0 ** 127
    x, y = _rows(left * 64 + k + 7, T, V, left, lowest)
    bits = store(x, dtype)
    y = np.where(np.arange(T) % 2 == 0, y, -1)
    lp, ent, ids, top, status = _run(lb, bits, V, V, y, k)
    x = synth.as_f64(bits)
    rids = np.argsort(-x, axis=-1, kind="stable")[:, :k]
    x[x <= lowest] = -np.inf  # e^(lowest - m) is 0 in 64 bits too
    rlp, rent, _, ez, au = _reference(x, k)
    tol = ez + 4 * U32 * (np.abs(np.where(np.isfinite(rlp), rlp, 0.0)).max(-1) + 32.0)
    want = np.where(y >= 0, rlp[np.arange(T), np.maximum(y, 0)], 0.0)
    assert np.all(np.abs(lp - want) <= tol)
    assert np.all(np.abs(ent - rent) <= 2 * ez * (1 + au) + 4 * U32 * (np.abs(rent) + 32.0))
    assert np.array_equal(ids, rids)
    tt = np.take_along_axis(rlp, rids, axis=1)
    masked = np.isinf(tt)
    assert np.all(np.abs(top[masked] / lowest - 1.0) <= 4 * U32)  # two subtractions far below its last bit
    assert np.all(np.abs(top - np.where(masked, top, tt)) <= tol[:, None])
    assert status == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [4000, 33001, 128256])
@pytest.mark.parametrize("where", ["front", "end", "together"])
def test_few_tokens_left_in_one_place(lb, dtype, V, where):
    """All that is left lies in one CTA's part of the row, or in the logits behind its last whole vector."""
    x = np.full((3, V), -np.inf, np.float32)
    for t, n in enumerate((2, 3, 11)):
        first = {"front": 0, "end": V - n, "together": V // 2 + 5}[where]
        x[t, first:first + n] = np.linspace(-1.0, 1.0, n) * (1 if t % 2 else -1)
    for k in (4, 20):
        _check(lb, store(x, dtype), V, V, np.array([V - 1, 0, V // 2 + 5]), k)
