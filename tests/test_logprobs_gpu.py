"""Token log-probabilities, entropy and top alternatives against 64-bit results (GPU).

Bounds: ln p = (x - m) - ln Z.  Z is an fp32 sum of V positive terms in which no
addend meets more than V / 128 + 64 others one after another, of exponentials
good to 2^-20 relative (their arguments are rounded to 2^-24 |x - m|): relative
error e_z = (V / 128 + 64) 2^-24 + 2^-20 + 2^-24 max|x - m|, which is the
absolute error of ln Z.  The subtractions round to 2^-24 of their results.  The
entropy ln Z - U / Z adds the error of U = sum e (x - m), e_z relative to
sum |e (x - m)|, once more e_z for the quotient."""
import numpy as np
import pytest

import synth
from _helpers import make_cfg, to_dev, to_f64, torch
from _packed import store

pytestmark = pytest.mark.gpu
U32 = 2.0 ** -24


@pytest.fixture(scope="module")
def lb():
    import decoder_block_gb300 as m
    m.load()
    return m


def _reference(x, k):
    m = x.max(-1, keepdims=True)
    e = np.exp(x - m)
    z = e.sum(-1, keepdims=True)
    lp = (x - m) - np.log(z)
    terms = np.where(e > 0, e * np.where(e > 0, x - m, 0.0), 0.0)
    ent = np.log(z[:, 0]) - terms.sum(-1) / z[:, 0]
    ids = np.argsort(-x, axis=-1, kind="stable")[:, :k]
    span = np.where(np.isfinite(x), m - x, 0.0).max(-1)
    ez = (x.shape[1] / 128 + 64) * U32 + 2.0 ** -20 + U32 * span
    return lp, ent, ids, ez, np.abs(terms).sum(-1) / z[:, 0]


def _run(lb, bits, V, stride, targets, k, want_entropy=True):
    t = torch()
    T = bits.shape[0]
    x = to_dev(bits)
    code = lb.LLAMA_BF16 if bits.dtype == np.uint16 else lb.LLAMA_F32
    y = None if targets is None else to_dev(np.asarray(targets, dtype=np.int32))
    lp = None if targets is None else t.full((T,), 3.0, device="cuda")
    ent = t.full((T,), 3.0, device="cuda") if want_entropy else None
    ids = t.full((T, max(k, 1)), -7, dtype=t.int32, device="cuda")
    top = t.full((T, max(k, 1)), 3.0, device="cuda")
    status = t.zeros(4, dtype=t.int32, device="cuda")
    lb.check(lb.llama_op_token_logprobs(code, x, stride, y, T, V, lp, ent, k, ids if k else None, top if k else None,
                                        status, t.cuda.current_stream()))
    t.cuda.synchronize()
    f = lambda a: None if a is None else to_f64(a)
    return f(lp), f(ent), ids.cpu().numpy()[:, :k], f(top)[:, :k], int(status[0])


def _check(lb, bits, V, stride, targets, k):
    lp, ent, ids, top, status = _run(lb, bits, V, stride, targets, k)
    x = synth.as_f64(bits)[:, :V]
    rlp, rent, rids, ez, au = _reference(x, k)
    tol = ez[:, None] * 1.01 + 4 * U32 * (np.abs(np.where(np.isfinite(rlp), rlp, 0.0)) + 32.0)
    rows = np.arange(len(x))
    y = np.asarray(targets)
    ok = y >= 0
    want = np.where(ok, rlp[rows, np.maximum(y, 0)], 0.0)
    fin = np.isfinite(want)
    assert np.array_equal(lp[~fin], want[~fin])
    with np.errstate(invalid="ignore"):
        err = np.abs(lp - want)
    assert np.all(err[fin] <= tol[rows, np.maximum(y, 0)][fin])
    assert np.all(np.abs(ent - rent) <= 2 * ez * (1 + au) + 4 * U32 * (np.abs(rent) + 32.0))
    assert np.array_equal(ids, rids)
    tt = np.take_along_axis(rlp, rids, axis=1)
    fin = np.isfinite(tt)
    assert np.array_equal(top[~fin], tt[~fin])
    with np.errstate(invalid="ignore"):
        err = np.abs(top - tt)
    assert np.all(err[fin] <= np.take_along_axis(tol, rids, axis=1)[fin])
    assert status == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,V,stride,k", [(1, 1, 1, 1), (3, 2, 2, 2), (2, 33, 40, 32), (5, 257, 257, 5),
                                          (64, 1000, 1024, 20), (7, 49152, 49152, 1), (3, 128256, 128256, 20),
                                          (1, 128255, 128320, 5), (2, 50257, 50257, 32), (700, 4099, 4099, 3),
                                          (4, 151936, 151936, 0), (20, 32001, 32001, 10)])
def test_token_logprobs(lb, dtype, T, V, stride, k):
    x = synth.normal(0, f"lp/{T}{V}", (T, stride), std=2.5)
    x[:, V:] = np.nan
    x[0, V // 2] = 14.0
    bits = store(x, dtype)
    y = synth.uniform_int(0, f"lp/y{T}{V}", (T,), V)
    y[T // 2] = -1 if T > 1 else y[0]
    _check(lb, bits, V, stride, y, k)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["rising", "falling", "equal", "few_values", "spike", "masked", "huge", "tiny_range"])
def test_token_logprobs_orders_and_masks(lb, dtype, kind):
    T, V, k = 3, 20011, 32
    i = np.arange(V, dtype=np.float32)[None].repeat(T, 0)
    noise = synth.normal(0, f"lpo/{kind}", (T, V))
    x = {"rising": i / 700.0, "falling": -i / 700.0, "equal": np.full((T, V), -3.25, np.float32),
         "few_values": np.floor(noise * 1.5), "spike": noise * 0.1 + (i == 17777) * 60.0,
         "masked": np.where(i % 997 == 5, noise, -np.inf), "huge": noise * 1e4,
         "tiny_range": 1.0 + noise * 1e-3}[kind].astype(np.float32)
    y = np.array([5, V - 1, 17777])
    _check(lb, store(x, dtype), V, V, y, k)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,V,k", [(4900, 261, 32), (1300, 3001, 8), (640, 4100, 1), (2500, 8197, 4), (40, 9000, 20),
                                   (76, 33000, 3), (152, 8300, 2)])
@pytest.mark.parametrize("kind", ["rising", "few_values", "masked", "noise"])
def test_token_logprobs_many_rows(lb, dtype, T, V, k, kind):
    i = np.arange(V, dtype=np.float32)[None].repeat(T, 0)
    noise = synth.normal(0, f"lpm/{T}{V}", (T, V))
    x = {"rising": i / 70.0, "few_values": np.floor(noise * 1.5), "masked": np.where(i % 7 == 5, noise, -np.inf),
         "noise": noise * 2.5}[kind].astype(np.float32)
    y = synth.uniform_int(0, f"lpm/y{T}{V}", (T,), V)
    _check(lb, store(x, dtype), V, V, y, k)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [40, 9000])
def test_token_logprobs_without_a_distribution(lb, dtype, V):
    x = synth.normal(0, f"lpn{V}", (4, V))
    x[0] = -np.inf
    x[1, V // 3] = np.nan
    x[2, V // 2] = np.inf
    x[3] = np.nan
    x[3, 7] = -np.inf
    lp, ent, ids, top, status = _run(lb, store(x, dtype), V, V, [2, 2, 2, 7], 3)
    assert lp[0] == -np.inf and ent[0] == 0.0 and np.array_equal(ids[0], [0, 1, 2]) and np.all(top[0] == -np.inf)
    assert np.all(np.isnan(lp[1:])) and np.all(np.isnan(ent[1:])) and np.all(np.isnan(top[1:]))
    bits = synth.as_f64(store(x, dtype))
    assert np.array_equal(ids[1], np.argsort(-np.where(np.isnan(bits[1]), -np.inf, bits[1]), kind="stable")[:3])
    assert ids[2][0] == V // 2
    assert np.array_equal(ids[3], [7, -1, -1])
    assert status == 0


def test_token_logprobs_targets_and_optional_outputs(lb):
    V = 300
    x = synth.normal(0, "lpt", (4, V))
    lp, ent, _, _, status = _run(lb, x, V, V, [-1, V, 5, -2], 0)
    rlp, rent, _, _, _ = _reference(x.astype(np.float64), 0)
    assert lp[0] == 0.0 and np.isnan(lp[1]) and np.isnan(lp[3]) and abs(lp[2] - rlp[2, 5]) < 1e-5
    assert np.allclose(ent, rent, atol=1e-5) and status == lb.LLAMA_ERR_RANGE
    lp, ent, ids, top, status = _run(lb, x, V, V, None, 4, want_entropy=False)
    assert lp is None and ent is None and np.array_equal(ids, _reference(x.astype(np.float64), 4)[2]) and status == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_token_logprobs_rows_more_than_four_gigabytes_apart(lb, dtype):
    t = torch()
    V, k, stride = 3001, 7, (1 << 30) + 5  # rows 2^30 elements apart, none of them aligned alike
    x = store(synth.normal(0, "lpfar", (4, V), std=2.5), dtype)
    pool = t.empty(3 * stride + V, dtype=t.float32 if dtype == "f32" else t.bfloat16, device="cuda")
    t.as_strided(pool, (4, V), (stride, 1)).copy_(to_dev(x))
    y = to_dev(np.array([0, 5, V - 1, 1000], np.int32))
    out = [t.empty(4, device="cuda"), t.empty(4, device="cuda"), t.empty((4, k), dtype=t.int32, device="cuda"),
           t.empty((4, k), device="cuda")]
    lb.check(lb.llama_op_token_logprobs(lb.LLAMA_F32 if dtype == "f32" else lb.LLAMA_BF16, pool, stride, y, 4, V, out[0],
                                        out[1], k, out[2], out[3], None, t.cuda.current_stream()))
    t.cuda.synchronize()
    lp, ent, ids, _, _ = _reference(synth.as_f64(x), k)
    assert np.allclose(to_f64(out[0]), lp[np.arange(4), [0, 5, V - 1, 1000]], atol=1e-5)
    assert np.allclose(to_f64(out[1]), ent, atol=1e-5)
    assert np.array_equal(out[2].cpu().numpy(), ids)


def test_token_logprobs_repeat_and_capture(lb):
    t = torch()
    T, V, k = 37, 30011, 8
    x = to_dev(synth.normal(0, "lpg", (T, V)))
    y = to_dev(synth.uniform_int(0, "lpgy", (T,), V))
    outs = [t.empty(T, device="cuda"), t.empty(T, device="cuda"), t.empty((T, k), dtype=t.int32, device="cuda"),
            t.empty((T, k), device="cuda")]

    def call():
        lb.check(lb.llama_op_token_logprobs(lb.LLAMA_F32, x, V, y, T, V, outs[0], outs[1], k, outs[2], outs[3], None,
                                            t.cuda.current_stream()))

    call()
    t.cuda.synchronize()
    first = [o.clone() for o in outs]
    graph = t.cuda.CUDAGraph()
    with t.cuda.graph(graph):
        call()
    for _ in range(3):
        for o in outs:
            o.zero_()
        graph.replay()
        t.cuda.synchronize()
        assert all(t.equal(a, b) for a, b in zip(first, outs))
    x2 = synth.normal(0, "lpg2", (T, V))
    x.copy_(to_dev(x2))
    graph.replay()
    t.cuda.synchronize()
    assert np.array_equal(outs[2].cpu().numpy(), _reference(x2.astype(np.float64), k)[2])


@pytest.mark.parametrize("S", [1, 12])
def test_stack_score(lb, S):
    """llama_stack_score: the stack's own logits, scored."""
    t = torch()
    shape = synth.SHAPES["tiny_f32"]
    vocab, B, L, k = 501, 2, 16, 5
    layers = [synth.block_weights(shape, layer=i) for i in range(2)]
    wd = [{n: to_dev(v) for n, v in w.items()} for w in layers]
    embed, head = (to_dev(synth.normal(0, n, (vocab, shape["d_model"]), std=0.3)) for n in ("embed", "lm_head"))
    norm = to_dev(synth.normal(0, "final_norm", (shape["d_model"],), std=0.1, mean=1.0))
    st, stk = lb.llama_stack_create(make_cfg(shape, L), 2, vocab, embed, [lb.make_weights(w) for w in wd], norm, head,
                                    B * S)
    lb.check(st, "llama_stack_create")
    try:
        caches = [[to_dev(c) for c in synth.kv_cache(shape, max_batch=B, max_seq_len=L, layer=i)] for i in range(2)]
        kvs = [lb.make_kv_cache(a, b, B, L) for a, b in caches]
        tok = synth.uniform_int(0, "tokens", (B, S), vocab)
        y = np.concatenate([tok[:, 1:], np.full((B, 1), -1, np.int32)], axis=1)
        y[0, 0] = 3
        tokens, targets = to_dev(tok), to_dev(y)
        logits, plain = (t.empty((B, S, vocab), device="cuda") for _ in range(2))
        lp, ent = t.empty((B, S), device="cuda"), t.empty((B, S), device="cuda")
        ids, top = t.empty((B, S, k), dtype=t.int32, device="cuda"), t.empty((B, S, k), device="cuda")
        lb.check(lb.llama_stack_forward(stk, tokens, B, S, 0, kvs, plain, t.cuda.current_stream()))
        n0 = lb.llama_kernel_launch_count()
        lb.check(lb.llama_stack_score(stk, tokens, B, S, 0, kvs, targets, logits, lp, ent, k, ids, top,
                                      t.cuda.current_stream()))
        assert lb.llama_kernel_launch_count() > n0
        t.cuda.synchronize()
        assert lb.llama_stack_device_status(stk) == lb.LLAMA_OK
        assert t.equal(plain, logits)
        x = to_f64(logits).reshape(B * S, vocab)
        rlp, rent, rids, ez, _ = _reference(x, k)
        want = np.where(y.reshape(-1) >= 0, rlp[np.arange(B * S), np.maximum(y.reshape(-1), 0)], 0.0)
        assert np.all(np.abs(to_f64(lp).reshape(-1) - want) <= ez + 4 * U32 * 64)
        assert np.allclose(to_f64(ent).reshape(-1), rent, atol=1e-5)
        assert np.array_equal(ids.cpu().numpy().reshape(-1, k), rids)
        assert np.allclose(to_f64(top).reshape(-1, k), np.take_along_axis(rlp, rids, 1), atol=1e-5)
        targets[0, 0] = vocab
        lb.check(lb.llama_stack_score(stk, tokens, B, S, 0, kvs, targets, logits, lp, None, 0, None, None,
                                      t.cuda.current_stream()))
        assert lb.llama_stack_device_status(stk) == lb.LLAMA_ERR_RANGE
        assert bool(t.isnan(lp[0, 0]))
        assert lb.llama_stack_score(stk, tokens, B, S, 0, kvs, None, logits, lp) == lb.LLAMA_ERR_INVALID_ARG
        assert lb.llama_stack_score(stk, tokens, B, S, 0, kvs, targets, logits, lp, None, 33, ids, top) \
            == lb.LLAMA_ERR_UNSUPPORTED
    finally:
        lb.llama_stack_destroy(stk)
