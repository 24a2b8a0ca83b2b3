"""Arrays that are read or written element by element may start at any element (GPU): slices of longer arrays, a status
word inside a struct, logits rows from the middle of a batch with an odd vocabulary.  The results are those of the
same data in arrays of its own, bit for bit."""
import numpy as np
import pytest

import synth
from _helpers import make_cfg, to_dev, torch
from _packed import Problem, run_decode, run_packed, store
from test_logprobs_gpu import _run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lb():
    import decoder_block_gb300 as m
    m.load()
    return m


def _moved(x, n):
    """A copy of x that starts n elements into an array of its own."""
    pool = torch().zeros(x.numel() + n, dtype=x.dtype, device="cuda")
    pool[n:].copy_(x.reshape(-1))
    return pool[n:].view(x.shape)


@pytest.mark.parametrize("dtype,H,G,D", [("bf16", 8, 2, 128), ("f32", 4, 2, 32)])
@pytest.mark.parametrize("n", [1, 2, 3])
def test_offsets_lengths_pages_and_status(lb, dtype, H, G, D, n):
    t = torch()
    p = Problem(f"align/{dtype}{D}", dtype, H, G, D, 16, [1] * 3, [300, 17, 2000], pad=1)
    table = t.empty((2000, D // 2, 2), dtype=t.float32, device="cuda")
    lb.check(lb.llama_op_rope_table(table, 2000, D, 1e4))
    qkv = to_dev(store(synth.normal(0, f"align/{D}", (p.T, (H + 2 * G) * D)), dtype))
    results = []
    for shift in (0, n):
        d = p.device(lb)
        d.table, d.offsets, d.kv_lens, d.status = (_moved(x, shift) for x in (d.table, d.offsets, d.kv_lens, d.status))
        assert (d.kv_lens.data_ptr() % 16 == 0) == (shift == 0)
        d.kv, d.batch = lb.make_paged_kv_cache(d.k, d.v, d.table), lb.make_packed_batch(d.offsets, d.kv_lens, p.T, 2000)
        out = []
        for run in (run_packed, run_decode):
            run(lb, p, d)
            out.append(d.o.clone())
        lb.check(lb.llama_op_rope_kv_write_paged(d.code, qkv, d.o, d.kv, d.batch, table, 2000, H, G, D, 0, d.status))
        t.cuda.synchronize()
        assert int(d.status[0]) == 0
        results.append(out + [d.o.clone(), d.kall.view(t.uint8), d.vall.view(t.uint8)])
    for a, b in zip(*results):
        assert t.equal(a, b)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,V", [(3, 1001), (2, 33333), (5000, 701)])
def test_logprobs_of_rows_from_the_middle(lb, dtype, T, V):
    t = torch()
    bits = store(synth.normal(0, f"mid/{V}", (T + 3, V), std=2.5), dtype)
    y = synth.uniform_int(0, f"mid/y{V}", (T + 3,), V)
    k = 5
    whole = _run(lb, bits, V, V, y, k)
    x = to_dev(bits)
    code = lb.LLAMA_BF16 if dtype == "bf16" else lb.LLAMA_F32
    for n in (1, 2, 3):
        targets = to_dev(y)[n:]
        lp, ent, top = (t.zeros(T + 3, device="cuda")[n:], t.zeros(T + 3, device="cuda")[n:],
                        t.zeros(n + T * k, device="cuda")[n:])
        ids, status = t.zeros(n + T * k, dtype=t.int32, device="cuda")[n:], t.zeros(4, dtype=t.int32, device="cuda")[n:]
        lb.check(lb.llama_op_token_logprobs(code, x[n:], V, targets, T, V, lp, ent, k, ids, top, status))
        t.cuda.synchronize()
        # the order of a row's sums follows from where its 16-byte vectors start: the same row, the same bits
        assert np.array_equal(lp.cpu().numpy()[:T], whole[0][n:n + T])
        assert np.array_equal(ent.cpu().numpy()[:T], whole[1][n:n + T])
        assert np.array_equal(ids.cpu().numpy().reshape(T, k), whole[2][n:n + T])
        assert np.array_equal(top.cpu().numpy().reshape(T, k), whole[3][n:n + T])
        assert int(status[0]) == 0


def test_stack_score_of_sliced_arrays(lb):
    t = torch()
    shape = synth.SHAPES["tiny_f32"]
    vocab, S, k = 301, 7, 3
    w = {n: to_dev(v) for n, v in synth.block_weights(shape).items()}
    embed, head = (to_dev(synth.normal(0, n, (vocab, shape["d_model"]), std=0.3)) for n in ("embed", "lm_head"))
    norm = to_dev(synth.normal(0, "final_norm", (shape["d_model"],), std=0.1, mean=1.0))
    st, stk = lb.llama_stack_create(make_cfg(shape, 16), 1, vocab, embed, [lb.make_weights(w)], norm, head, S)
    lb.check(st, "llama_stack_create")
    try:
        caches = [to_dev(c) for c in synth.kv_cache(shape, max_batch=1, max_seq_len=16)]
        kvs = [lb.make_kv_cache(*caches, 1, 16)]
        tokens, y = to_dev(synth.uniform_int(0, "tokens", (S,), vocab)), to_dev(synth.uniform_int(0, "y", (S,), vocab))
        got = []
        for n in (0, 1):
            logits = t.empty((S, vocab), device="cuda")
            lp, ent, top = (_moved(t.zeros(m, device="cuda"), n) for m in (S, S, S * k))
            ids = _moved(t.zeros(S * k, dtype=t.int32, device="cuda"), n)
            lb.check(lb.llama_stack_score(stk, tokens, 1, S, 0, kvs, _moved(y, n), logits, lp, ent, k, ids, top,
                                          t.cuda.current_stream()))
            t.cuda.synchronize()
            assert lb.llama_stack_device_status(stk) == lb.LLAMA_OK
            got.append([a.clone() for a in (lp, ent, top, ids)])
        for a, b in zip(*got):
            assert t.equal(a, b)
    finally:
        lb.llama_stack_destroy(stk)
