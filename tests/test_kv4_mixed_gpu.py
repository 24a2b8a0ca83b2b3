"""Batches over 4-bit pages that mix sequences of few and of many rows (GPU).

With few rows on average a batch goes to the kernel for them; where one sequence could bring so many that they would
take long there, sequences of more than 48 rows a KV head go to the tensor core kernel of prompts and the others stay.
The bound on the lengths given here lets short batches take that way."""
import numpy as np
import pytest

from _helpers import to_f64, torch
from _kv4 import Kv4Problem, run_packed

pytestmark = pytest.mark.gpu

FAR = 1 << 20


@pytest.fixture(scope="module")
def lb():
    import decoder_block_gb300 as m
    m.load()
    yield m
    m.check(m.llama_op_set_wait_budget(0))


def launches(lb, call):
    before = lb.llama_kernel_launch_count()
    call()
    torch().cuda.synchronize()
    return lb.llama_kernel_launch_count() - before


HEADS = [(32, 8, 128), (8, 2, 64), (9, 3, 64), (6, 2, 32), (4, 4, 16)]


def cases(r):
    """(name, q_lens, kv_lens); r: heads of a group."""
    many = 48 // r + 1  # the least tokens that are not few
    one = [17 + 23 * i for i in range(40)]
    return [
        ("one_prompt", [1] * 20 + [180] + [1] * 19, one[:20] + [700] + one[20:39]),
        ("prompts_and_drafts", [many + 100, 1, 0, 3, many, 2] + [1] * 50, [500, 1, 9, 300, many, 0] + [40 + 9 * i for i in range(50)]),
        ("either_side", [many - 1, many] + [1] * 60, [400, 400] + [5 + i for i in range(60)]),
        ("some_see_nothing", [many + 60, many + 9, 2, 5, 1] + [1] * 40, [many + 3, 0, 1, 0, 0] + [33] * 40),
        ("the_others_are_empty", [0] * 40 + [200] + [0] * 40, [3] * 40 + [260] + [0] * 40),
    ]


@pytest.mark.parametrize("H,G,D", HEADS)
@pytest.mark.parametrize("which", range(5))
def test_mixed(lb, H, G, D, which):
    name, q_lens, kv_lens = cases(H // G)[which]
    p = Kv4Problem(f"mix/{name}{D}{H}", "bf16", H, G, D, (16, 32, 64, 128, 256)[which], q_lens, kv_lens, pad=3)
    d = p.device(lb)
    n = launches(lb, lambda: run_packed(lb, p, d, max_kv=FAR))
    p.check(to_f64(d.o), name)
    assert int(d.status[0]) == 0
    first = d.o.clone()
    for _ in range(3):
        d.o.fill_(7.0)
        run_packed(lb, p, d, max_kv=FAR)
        assert torch().equal(d.o, first), "the same call twice"
    few = sum(q_lens) - len(q_lens) + 1 <= 48 // (H // G)
    assert n == (2 if few else 5)


def test_batches_that_one_sequence_cannot_hold_up_take_one_kernel(lb):
    """Drafts of many sequences under a bound near their lengths: two launches, as for single tokens."""
    p = Kv4Problem("nomix", "bf16", 8, 2, 64, 32, [5] * 24, [100 + 20 * i for i in range(24)])
    assert launches(lb, lambda: run_packed(lb, p)) == 2
    p = Kv4Problem("nomix1", "bf16", 8, 2, 64, 32, [1] * 24, [100 + 20 * i for i in range(24)])
    assert launches(lb, lambda: run_packed(lb, p, max_kv=FAR)) == 2


def test_graph_replays_follow_the_rows_from_one_kernel_to_the_other(lb):
    t = torch()
    H, G, D, n, T = 8, 2, 64, 40, 140
    kv = [200 + 11 * i for i in range(n)]
    splits = [[1] * 39 + [101], [101] + [1] * 39, [3] * 20 + [4] * 20, [50, 0, 40] + [1] * 24 + [2] * 13, [0] * 39 + [140]]
    ps = [Kv4Problem(f"mg{i}", "bf16", H, G, D, 32, q, kv) for i, q in enumerate(splits)]
    d = ps[0].device(lb)
    d.batch = lb.make_packed_batch(d.offsets, d.kv_lens, T, FAR)
    need = lb.llama_op_attention_packed_kv4_workspace_bytes(d.code, d.batch, H, G, D)
    ws = t.full((need,), 0x5A, dtype=t.uint8, device="cuda")
    side = t.cuda.Stream()
    run_packed(lb, ps[0], d, side, ws, FAR)
    t.cuda.synchronize()
    g = t.cuda.CUDAGraph()
    with t.cuda.graph(g, stream=side):
        run_packed(lb, ps[0], d, side, ws, FAR)
    for p in ps:
        assert p.T == T and p.n_pages == ps[0].n_pages
        e = p.device(lb)
        for to, x in ((d.q, e.q), (d.k, e.k), (d.v, e.v), (d.table, e.table), (d.offsets, e.offsets), (d.kv_lens, e.kv_lens)):
            to.copy_(x)
        d.o.fill_(7.0)
        ws.random_(0, 256)
        g.replay()
        t.cuda.synchronize()
        p.check(to_f64(d.o), str(p.q_lens))
        assert int(d.status[0]) == 0


def test_bad_pages_offsets_and_lengths(lb):
    t = torch()
    q_lens, kv_lens = [1] * 30 + [150, 2], [40 + 7 * i for i in range(30)] + [400, 90]
    p = Kv4Problem("mbad", "bf16", 8, 2, 64, 16, q_lens, kv_lens)
    p.table[30, 3], p.table[5, 1], p.table[31, 0] = -1, p.n_pages, 0x7fffffff
    d = p.device(lb)
    d.kv_lens[7] = -3
    run_packed(lb, p, d, max_kv=FAR)
    t.cuda.synchronize()
    assert int(d.status[0]) == lb.LLAMA_ERR_RANGE
    for name in "kv":
        x = getattr(p, name)
        setattr(p, name, np.concatenate([x, np.zeros((1,) + x.shape[1:], x.dtype)]))
    p.table[(p.table < 0) | (p.table >= p.n_pages)] = p.n_pages
    p.kv_lens[7] = 0
    p.check(to_f64(d.o), "pages")
    # the long sequence's offsets out of range: the others are as they were, and nothing of its rows is written
    p = Kv4Problem("moff", "bf16", 8, 2, 64, 16, q_lens, kv_lens)
    ref, bound = p.attention()
    d = p.device(lb)
    d.offsets[31:] = p.T + 1
    run_packed(lb, p, d, max_kv=FAR)
    t.cuda.synchronize()
    assert int(d.status[0]) == lb.LLAMA_ERR_RANGE
    got = to_f64(d.o)
    assert np.all(np.abs(got - ref)[:30] <= bound[:30]) and np.all(got[30:] == 7.0)
    for bad in ([0, 200, 30] + list(range(31, 61)), [5] * 20 + [0] * 13):
        d = p.device(lb)
        d.offsets.copy_(t.tensor(bad[:33], dtype=t.int32))
        run_packed(lb, p, d, max_kv=FAR)
        t.cuda.synchronize()
        assert int(d.status[0]) == lb.LLAMA_ERR_RANGE and np.all(np.isfinite(to_f64(d.o)))


def test_waits_that_run_out_are_reported_and_the_next_call_is_right(lb):
    t = torch()
    p = Kv4Problem("mto", "bf16", 32, 8, 128, 64, [1] * 64 + [300], [30 + 5 * i for i in range(64)] + [900])
    d = p.device(lb)
    reported = 0
    for budget in (1, 300, 1000, 2000, 4000, 8000, 1, 1):
        lb.check(lb.llama_op_set_wait_budget(budget))
        try:
            run_packed(lb, p, d, max_kv=FAR)
        finally:
            lb.check(lb.llama_op_set_wait_budget(0))
        t.cuda.synchronize()  # raises if the kernel faulted: it may not
        status = int(d.status[0])
        assert status in (lb.LLAMA_OK, lb.LLAMA_ERR_DEVICE_TIMEOUT)
        reported += status == lb.LLAMA_ERR_DEVICE_TIMEOUT
        d.status.zero_()
        d.o.fill_(7.0)
        run_packed(lb, p, d, max_kv=FAR)
        t.cuda.synchronize()
        assert int(d.status[0]) == 0
    p.check(to_f64(d.o), "after")
    assert reported > 0, "no wait ran out: nothing was tested"
