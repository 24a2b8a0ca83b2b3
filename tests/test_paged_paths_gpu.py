"""Paged operators at sizes that choose other ways through the kernels: many rows per CTA of the page write, sequence
look-ups of two and three rounds, 16-row pages dealt out over many items, fp32 over many sequences (GPU)."""
import numpy as np
import pytest

import oracle
import synth
from _helpers import to_dev, to_f64, to_host_bits, torch
from _packed import U32, U_BF16, Problem, run_decode, run_packed, store

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lb():
    import decoder_block_gb300 as m
    m.load()
    return m


def _split(rng, total, n):
    """n lengths, empty ones among them, that add up to total."""
    cuts = np.sort(rng.integers(0, total + 1, n - 1))
    return np.diff(np.concatenate([[0], cuts, [total]])).astype(int)


# tokens: one, two and four rows per CTA (with 152 SMs from 1216 and 2432 on), the last CTA full and not
@pytest.mark.parametrize("layout", ["interleaved", "halves"])
@pytest.mark.parametrize("dtype,H,G,D,page", [("bf16", 9, 3, 64, 16), ("bf16", 4, 1, 128, 64), ("f32", 3, 1, 32, 128),
                                              ("bf16", 2, 2, 16, 32)])
@pytest.mark.parametrize("tokens,n,pad", [(1215, 3, 0), (1217, 40, 2), (2435, 33, 0), (2430, 1100, 7), (5000, 4096, 5),
                                          (4864, 1, 0)])
def test_rope_kv_write_of_many_rows(lb, layout, dtype, H, G, D, page, tokens, n, pad):
    t = torch()
    rng = np.random.default_rng(tokens + n)
    q_lens = _split(rng, tokens, n) if n > 1 else np.array([tokens])
    kv_lens = q_lens + rng.integers(0, 30, n)
    p = Problem(f"many/{layout}{dtype}{D}{tokens}", dtype, H, G, D, page, q_lens.tolist(), kv_lens.tolist(), pad=pad,
                rubbish=False)
    d = p.device(lb)
    qkv = store(synth.normal(0, f"many/qkv{dtype}{H}{D}{tokens}", (p.T, (H + 2 * G) * D)), dtype)
    max_seq, theta = int(kv_lens.max()), 1e4
    table = t.empty((max_seq, D // 2, 2), dtype=t.float32, device="cuda")
    lb.check(lb.llama_op_rope_table(table, max_seq, D, theta))
    lay = lb.LLAMA_ROPE_HALVES if layout == "halves" else lb.LLAMA_ROPE_INTERLEAVED
    before_k, before_v = to_host_bits(d.kall).copy(), to_host_bits(d.vall).copy()
    lb.check(lb.llama_op_rope_kv_write_paged(d.code, to_dev(qkv), d.o, d.kv, d.batch, table, max_seq, H, G, D, lay,
                                             d.status, t.cuda.current_stream()))
    t.cuda.synchronize()
    assert int(d.status[0]) == 0
    seq = np.repeat(np.arange(n), q_lens)
    pos = kv_lens[seq] - (p.offsets[seq + 1] - np.arange(tokens))
    x = synth.as_f64(qkv[:tokens]).reshape(tokens, H + 2 * G, D)
    rot = oracle.rope(x[None, :, :H + G], pos, theta, layout)[0]
    half = np.abs(x[:, :H + G])
    # two products of a rounded cos / sin and their sum, then the store
    tol = (U_BF16 if dtype == "bf16" else U32) * 1.01 * np.abs(rot) + 4 * U32 * (half + half.max(-1, keepdims=True))
    got_q = to_f64(d.o)
    assert np.all(np.abs(got_q[:tokens] - rot[:, :H]) <= tol[:, :H])
    assert np.all(got_q[tokens:] == 7.0)
    where, slot = p.table[seq, pos // page], pos % page
    got_k, got_v = to_host_bits(d.kall), to_host_bits(d.vall)
    assert np.all(np.abs(synth.as_f64(got_k[where, 0, :, slot]) - rot[:, H:]) <= tol[:, H:])
    assert np.array_equal(got_v[where, 0, :, slot], qkv[:tokens].reshape(tokens, -1, D)[:, H + G:])
    same = np.ones(before_k.shape, dtype=bool)
    same[where, 0, :, slot] = False
    assert np.array_equal(got_k[same], before_k[same]) and np.array_equal(got_v[same], before_v[same])


# several items per CTA, 16-row pages at both head widths; 300 sequences beside a long one
@pytest.mark.parametrize("H,G,D,q_lens,kv_lens", [
    (64, 8, 128, [700, 1, 333, 0, 64, 200], [700, 900, 1333, 40, 64, 327]),
    (64, 8, 64, [700, 1, 333, 0, 64, 200], [700, 900, 1333, 40, 64, 327]),
    (32, 4, 128, [1] * 300 + [90], [1 + 7 * (i % 50) for i in range(300)] + [3000]),
    (16, 8, 64, [3] * 300 + [40], [3 + 7 * (i % 50) for i in range(300)] + [3000]),
])
def test_packed_attention_of_many_items_over_small_pages(lb, H, G, D, q_lens, kv_lens):
    p = Problem(f"items/{H}{D}{len(q_lens)}", "bf16", H, G, D, 16, q_lens, kv_lens, pad=3)
    for max_kv in (None, 1 << 17):
        d = run_packed(lb, p, max_kv=max_kv)
        torch().cuda.synchronize()
        p.check(to_f64(d.o), f"bound {max_kv}")
        assert int(d.status[0]) == 0


@pytest.mark.parametrize("H,G,D", [(4, 2, 64), (3, 1, 16), (10, 1, 128)])
@pytest.mark.parametrize("n", [41, 300, 1100])
def test_fp32_over_many_sequences(lb, n, H, G, D):
    rng = np.random.default_rng(n + D)
    q = rng.integers(0, 3, n)
    kv = q + rng.integers(0, 40, n)
    q[n // 2], kv[n // 2], kv[n - 1] = 1, 900, max(1, q[n - 1])
    p = Problem(f"f32many/{n}{D}", "f32", H, G, D, 16, q.tolist(), kv.tolist(), pad=2)
    for max_kv in (None, 1 << 16):
        d = run_packed(lb, p, max_kv=max_kv)
        torch().cuda.synchronize()
        p.check(to_f64(d.o), f"packed, bound {max_kv}")
        assert int(d.status[0]) == 0
    p = Problem(f"f32many/d{n}{D}", "f32", H, G, D, 16, [1] * n, np.maximum(kv, 1).tolist())
    for max_kv in (None, 1 << 16):
        d = run_decode(lb, p, max_kv=max_kv)
        torch().cuda.synchronize()
        p.check(to_f64(d.o), f"decode, bound {max_kv}")
        assert int(d.status[0]) == 0
