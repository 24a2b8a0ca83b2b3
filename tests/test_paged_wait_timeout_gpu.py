"""Bounded waits of the packed and paged-decode attention kernels, made to run out (GPU).

With a budget of a few cycles the first waits that are not satisfied at once give up, at places that vary with the
budget: between the copies of a stage, between a product and its softmax, between items.  The kernels report it, leave
nothing of theirs in flight, and the next call with the default budget matches the 64-bit results.  Nothing here faults
or traps."""
import pytest

from _helpers import to_f64, torch
from _packed import Problem, run_decode, run_packed

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lb():
    import decoder_block_gb300 as m
    m.load()
    yield m
    m.check(m.llama_op_set_wait_budget(0))


PACKED = ([700, 1, 333, 200], [900, 700, 1333, 327])
CASES = [
    ("packed_small_pages", run_packed, 32, 8, 128, 16, *PACKED, None),     # four loading warps
    ("packed_small_pages_d64", run_packed, 32, 8, 64, 16, *PACKED, None),  # three S buffers
    ("packed", run_packed, 32, 8, 128, 64, *PACKED, None),
    ("packed_d64", run_packed, 32, 8, 64, 128, *PACKED, None),
    ("packed_direct", run_packed, 8, 2, 128, 16, [40, 90], [900, 300], None),
    ("packed_in_pieces", run_packed, 8, 2, 128, 32, [2, 70], [9000, 3333], None),
    ("decode_whole", run_decode, 32, 8, 128, 16, [1] * 40, [100 + 30 * i for i in range(40)], None),
    ("decode_clusters", run_decode, 8, 2, 128, 32, [1] * 5, [4000, 900, 1, 129, 0], None),
    ("decode_clusters_d64", run_decode, 9, 3, 64, 16, [1] * 5, [4000, 900, 1, 129, 0], None),
    ("decode_cut_by_every_cta", run_decode, 32, 8, 128, 16, [1] * 5, [9000, 5, 700, 2222, 64], 1 << 17),
    ("decode_cut_by_the_plan", run_decode, 32, 8, 64, 64, [1] * 40, [9000, 5, 700, 2222] + [300] * 36, 1 << 17),
]


@pytest.mark.parametrize("name,run,H,G,D,page,q_lens,kv_lens,max_kv", CASES, ids=[c[0] for c in CASES])
def test_waits_that_run_out_are_reported_and_the_next_call_is_right(lb, name, run, H, G, D, page, q_lens, kv_lens,
                                                                    max_kv):
    t = torch()
    p = Problem(f"to/{name}", "bf16", H, G, D, page, q_lens, kv_lens)
    d = p.device(lb)
    reported = 0
    for budget in (1, 300, 1000, 2000, 4000, 8000, 1, 1):
        lb.check(lb.llama_op_set_wait_budget(budget))
        try:
            run(lb, p, d, max_kv=max_kv)
        finally:
            lb.check(lb.llama_op_set_wait_budget(0))
        t.cuda.synchronize()  # raises if the kernel faulted: it may not
        status = int(d.status[0])
        assert status in (lb.LLAMA_OK, lb.LLAMA_ERR_DEVICE_TIMEOUT)
        reported += status == lb.LLAMA_ERR_DEVICE_TIMEOUT
        d.status.zero_()
        d.o.fill_(7.0)
        run(lb, p, d, max_kv=max_kv)
        t.cuda.synchronize()
        assert int(d.status[0]) == 0
    p.check(to_f64(d.o), name)
    assert reported > 0, "no wait ran out: nothing was tested"
