"""Paged attention of query rows that hold NaN or infinities (GPU).

By the formula such a row's scores hold NaN, or an infinity that the softmax subtracts from itself: where the row sees
a key its output is NaN, on every way through the kernels, and no other row or head is touched by it.  A row that sees
no key is zeros whatever it holds."""
import numpy as np
import pytest

import synth
from _helpers import to_dev, to_f64, torch
from _packed import Problem, run_decode, run_packed, store

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lb():
    import decoder_block_gb300 as m
    m.load()
    return m


def _spoil(p, rows):
    """NaN, +inf and -inf in one component, and a whole row of NaN, at rows x heads; the spoilt places."""
    q = synth.as_f64(p.q)
    spoilt = np.zeros((p.T, p.H), dtype=bool)
    kinds = [lambda r: r.__setitem__(3, np.nan), lambda r: r.__setitem__(0, np.inf),
             lambda r: r.__setitem__(p.D - 1, -np.inf), lambda r: r.__setitem__(slice(None), np.nan)]
    for n, row in enumerate(rows):
        head = (n * 5 + 1) % p.H
        kinds[n % 4](q[row, head])
        spoilt[row, head] = True
    return store(q.astype(np.float32), p.dtype), spoilt


def _check(lb, p, run, rows, max_kv, what):
    sees = np.concatenate([np.arange(L - n, L) >= 0 for n, L in zip(p.q_lens, p.kv_lens)] + [np.zeros(p.pad, bool)])
    q, spoilt = _spoil(p, rows)
    d = p.device(lb)
    d.q = to_dev(q)
    run(lb, p, d, max_kv=max_kv)
    torch().cuda.synchronize()
    got = to_f64(d.o)
    nan = spoilt & sees[:, None]
    assert np.all(np.isnan(got[nan])), f"{what}: finite values for a query that is not"
    ref, bound = p.attention()  # of the rows as they were
    bound[spoilt & ~sees[:, None]] = 0.0
    keep = np.isnan(bound)
    assert np.all(got[keep & ~nan[..., None]] == 7.0)
    rest = ~keep & ~nan[..., None]
    assert np.all(np.abs(got - ref)[rest] <= bound[rest]), f"{what}: another row was touched"
    assert int(d.status[0]) == 0


HEADS = [("bf16", 8, 2, 128), ("bf16", 9, 3, 64), ("bf16", 20, 1, 32), ("f32", 6, 2, 64), ("f32", 4, 2, 16)]


@pytest.mark.parametrize("dtype,H,G,D", HEADS)
@pytest.mark.parametrize("name,kv_lens,max_kv", [
    ("one_part", [300, 17, 1, 128, 64, 90], None),                        # clusters, or unsplit fp32
    ("clusters", [1700, 900, 1, 129, 0], None),
    ("many_whole", [150 + 3 * (i % 40) for i in range(160)], None),       # more sequences than clusters
    ("cut_by_every_cta", [3000, 5, 700, 2222, 0, 64], 1 << 18),
    ("cut_by_the_plan", [3000, 5, 700, 2222, 0] + [40] * 35, 1 << 18),
])
def test_decode(lb, dtype, H, G, D, name, kv_lens, max_kv):
    p = Problem(f"nf/{name}{dtype}{D}", dtype, H, G, D, 32, [1] * len(kv_lens), kv_lens)
    # rows of empty sequences have no position (kv_len - 1 < 0): they stay zeros
    rows = [0, 1, 2, 3, 4, len(kv_lens) - 1]
    _check(lb, p, run_decode, rows, max_kv, name)


@pytest.mark.parametrize("dtype,H,G,D", HEADS)
@pytest.mark.parametrize("name,q_lens,kv_lens,max_kv", [
    ("direct", [5, 40, 130], [5, 200, 130], None),
    ("planned", [5, 40, 130], [5, 200, 130], 1 << 18),
    ("few_rows_many_keys", [2, 3, 1], [9000, 3333, 1], None),
    ("see_nothing", [20, 9], [12, 0], None),
    ("see_nothing_in_parts", [200, 9, 4], [170, 0, 6000], None),
])
def test_packed(lb, dtype, H, G, D, name, q_lens, kv_lens, max_kv):
    p = Problem(f"nfp/{name}{dtype}{D}", dtype, H, G, D, 16, q_lens, kv_lens, pad=2)
    n = int(p.offsets[-1])
    rows = [0, 1, n // 3, n // 2, n - 2, n - 1]
    _check(lb, p, run_packed, rows, max_kv, name)
