"""Attention over 4-bit pages on the ways that test_kv4_gpu.py does not come by (GPU): many sequences, offsets and pages
out of range in each kernel, waits that run out, calls on two streams at once."""
import numpy as np
import pytest

from _helpers import to_f64, torch
from _kv4 import Kv4Problem, run_decode, run_packed

pytestmark = pytest.mark.gpu

FAR = 1 << 18  # a bound on the lengths that makes few of the tiles that there could be


@pytest.fixture(scope="module")
def lb():
    import decoder_block_gb300 as m
    m.load()
    yield m
    m.check(m.llama_op_set_wait_budget(0))


@pytest.mark.parametrize("H,G,D", [(32, 8, 128), (12, 2, 64), (6, 3, 16)])
@pytest.mark.parametrize("name,q_lens,kv_lens,max_kv", [
    ("few_rows_some_see_nothing", [3, 2, 4, 1], [1, 0, 900, 450], None),
    ("no_row_sees_a_key", [3, 2], [0, 0], 1000),
    ("one_long_among_few", [1, 70, 2, 1, 1, 1, 3, 1, 1, 1], [700, 800, 30, 5, 900, 64, 63, 1, 2000, 33], None),
    ("one_query_tile_in_pieces", [20, 20, 20], [3000, 500, 5000], FAR),
    ("one_query_tile", [20] * 24, [30 + 14 * i for i in range(24)], None),
    ("rows_of_many_items", [40, 9], [1500, 700], None),
    ("many_of_few_keys", [1 + i % 5 for i in range(120)], [5 + (37 * i) % 300 for i in range(120)], None),
    ("few_of_few_keys", [1 + i % 5 for i in range(7)], [5 + (37 * i) % 300 for i in range(7)], None),
])
def test_packed(lb, H, G, D, name, q_lens, kv_lens, max_kv):
    p = Kv4Problem(f"pp/{name}{D}", "bf16", H, G, D, 32, q_lens, kv_lens, pad=2)
    d = run_packed(lb, p, max_kv=max_kv)
    torch().cuda.synchronize()
    p.check(to_f64(d.o), name)
    assert int(d.status[0]) == 0


@pytest.mark.parametrize("n", [1000, 4096])
def test_decode_of_many_sequences(lb, n):
    rng = np.random.default_rng(n)
    lens = [int(x) for x in rng.integers(0, 70, n)]
    lens[n // 2] = 900
    p = Kv4Problem(f"many{n}", "bf16", 4, 2, 16, 16, [1] * n, lens)
    for max_kv in (None, 1 << 16):
        d = run_decode(lb, p, max_kv=max_kv)
        torch().cuda.synchronize()
        p.check(to_f64(d.o), f"{n} {max_kv}")


@pytest.mark.parametrize("H,G,D", [(32, 8, 128), (18, 6, 64), (12, 6, 16)])
@pytest.mark.parametrize("longest", [1024, 1025, 2048, 2049])
def test_decode_either_side_of_the_forms_limits(lb, H, G, D, longest):
    for n in (2, 16):  # items for few SMs, and for most of them
        lens = [longest - 97 * i if 97 * i < longest else 0 for i in range(n)]
        p = Kv4Problem(f"lim{longest}{n}{D}", "bf16", H, G, D, 64, [1] * n, lens)
        d = run_decode(lb, p)
        torch().cuda.synchronize()
        p.check(to_f64(d.o), f"{n} {longest}")


def test_packed_of_many_sequences(lb):
    n = 4096
    lens = [5 + i % 40 for i in range(n)]
    lens[17] = 700
    p = Kv4Problem("manyp", "bf16", 2, 1, 16, 16, [1 + i % 2 for i in range(n)], lens)
    d = run_packed(lb, p)
    torch().cuda.synchronize()
    p.check(to_f64(d.o))


@pytest.mark.parametrize("max_kv", [None, 1000, FAR])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_offsets_out_of_range_leave_the_others_alone(lb, dtype, max_kv):
    t = torch()
    p = Kv4Problem("off", dtype, 8, 2, 64, 16, [3, 2, 4, 5], [50, 40, 70, 33])
    ref, bound = p.attention()
    for bad, keep in (([0, 3, 900, 9, 14], [0, 3]), ([-2, 3, 5, 9, 14], [1, 2, 3]), ([0, 3, 1, 9, 14], [0, 3])):
        d = p.device(lb)
        d.offsets.copy_(t.tensor(bad, dtype=t.int32))
        run_packed(lb, p, d, max_kv=max_kv)
        t.cuda.synchronize()
        assert int(d.status[0]) == lb.LLAMA_ERR_RANGE
        got = to_f64(d.o)
        for i in keep:
            if bad[i:i + 2] != p.offsets[i:i + 2].tolist():
                continue
            rows = slice(p.offsets[i], p.offsets[i + 1])
            if bad == [0, 3, 1, 9, 14] and i == 0:
                continue  # a sequence that overlaps it may have written its rows
            assert np.all(np.abs(got - ref)[rows] <= bound[rows]), (bad, i)
        assert np.all(np.isfinite(got))


@pytest.mark.parametrize("run", [run_packed, run_decode])
@pytest.mark.parametrize("page", [16, 32, 64, 256])
@pytest.mark.parametrize("D", [128, 64, 32, 16])
def test_bad_pages_are_zeros(lb, run, page, D):
    """Ids out of range at a tile's first, later and last page, over every page size and way."""
    t = torch()
    for max_kv in (None, FAR):
        p = Kv4Problem(f"bp{page}{D}", "bf16", 4, 2, D, page, [1] * 3, [700, 300, 3 * page + 1])
        for i, which in enumerate(([0, 2], [1], [3])):
            for j in which:
                if j * page < p.kv_lens[i]:
                    p.table[i, j] = (-1, p.n_pages, 0x7fffffff)[(i + j) % 3]
        d = p.device(lb)
        run(lb, p, d, max_kv=max_kv)
        t.cuda.synchronize()
        assert int(d.status[0]) == lb.LLAMA_ERR_RANGE
        for name in "kv":
            x = getattr(p, name)
            setattr(p, name, np.concatenate([x, np.zeros((1,) + x.shape[1:], x.dtype)]))
        p.table[(p.table < 0) | (p.table >= p.n_pages)] = p.n_pages
        p.check(to_f64(d.o), f"{page} {D} {max_kv}")


def test_two_streams_at_once(lb):
    t = torch()
    for run in (run_packed, run_decode):
        ps = [Kv4Problem(f"st{i}", "bf16", 8, 2, 128, 64, [1] * 12, [400 + 150 * j + i for j in range(12)]) for i in range(2)]
        ds = [p.device(lb) for p in ps]
        streams = [t.cuda.Stream(), t.cuda.Stream()]
        t.cuda.synchronize()
        for _ in range(5):
            for p, d, s in zip(ps, ds, streams):
                with t.cuda.stream(s):
                    run(lb, p, d, s, max_kv=FAR)
        t.cuda.synchronize()
        for p, d in zip(ps, ds):
            p.check(to_f64(d.o))


WAITS = [  # calls of many tiles: the kernel of few rows has no waits
    ("two_tiles", 32, 8, 128, 64, [700, 1, 333, 200], [900, 700, 1333, 327], None),
    ("two_tiles_d64", 32, 8, 64, 16, [700, 1, 333, 200], [900, 700, 1333, 327], None),
    ("two_tiles_d16", 16, 8, 16, 16, [1400, 600], [2900, 1700], None),
    ("direct", 8, 2, 128, 16, [40, 90], [200, 300], None),
    ("one_tile", 32, 8, 128, 32, [20, 20, 20], [3000, 500, 5000], FAR),
]


@pytest.mark.parametrize("name,H,G,D,page,q_lens,kv_lens,max_kv", WAITS, ids=[w[0] for w in WAITS])
def test_waits_that_run_out_are_reported_and_the_next_call_is_right(lb, name, H, G, D, page, q_lens, kv_lens, max_kv):
    t = torch()
    p = Kv4Problem(f"to/{name}", "bf16", H, G, D, page, q_lens, kv_lens)
    d = p.device(lb)
    reported = 0
    for budget in (1, 300, 1000, 2000, 4000, 8000, 1, 1):
        lb.check(lb.llama_op_set_wait_budget(budget))
        try:
            run_packed(lb, p, d, max_kv=max_kv)
        finally:
            lb.check(lb.llama_op_set_wait_budget(0))
        t.cuda.synchronize()  # raises if the kernel faulted: it may not
        status = int(d.status[0])
        assert status in (lb.LLAMA_OK, lb.LLAMA_ERR_DEVICE_TIMEOUT)
        reported += status == lb.LLAMA_ERR_DEVICE_TIMEOUT
        d.status.zero_()
        d.o.fill_(7.0)
        run_packed(lb, p, d, max_kv=max_kv)
        t.cuda.synchronize()
        assert int(d.status[0]) == 0
    p.check(to_f64(d.o), name)
    assert reported > 0, "no wait ran out: nothing was tested"
