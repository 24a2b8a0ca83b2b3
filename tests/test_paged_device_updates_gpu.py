"""Lengths, offsets and page ids that the kernels directly in front of the paged operators write (GPU)."""
import numpy as np
import pytest

import synth
from _helpers import to_dev, to_host_bits, torch
from _packed import Problem, store

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lb():
    import decoder_block_gb300 as m
    m.load()
    return m


@pytest.mark.parametrize("dtype,H,G,D", [("bf16", 8, 2, 128), ("bf16", 9, 3, 64), ("f32", 4, 2, 32)])
@pytest.mark.parametrize("n,max_kv", [(3, 700), (40, 700), (3, 1 << 17), (40, 1 << 17)])
def test_lengths_offsets_and_pages_changed_by_the_kernel_in_front(lb, dtype, H, G, D, n, max_kv):
    """A captured step whose own first kernels move the lengths on, shift the rows and give out pages, replayed without
    a stop in between; every replay's results are kept on the device and checked afterwards."""
    t = torch()
    page, steps, pad = 16, 6, 2
    start = [(37 * i + 5) % 400 + 1 for i in range(n)]
    p = Problem(f"front/{dtype}{D}{n}", dtype, H, G, D, page, [1] * n, [s + steps for s in start], pad=pad,
                rubbish=False)
    p.table[p.table == 0x7fffffff] = 0
    d = p.device(lb)
    T = n + pad
    qkv = to_dev(store(synth.normal(0, f"front/qkv{D}{n}", (steps, T, (H + 2 * G) * D)), dtype))
    table = t.empty((500, D // 2, 2), dtype=t.float32, device="cuda")
    lb.check(lb.llama_op_rope_table(table, 500, D, 1e4))
    k0, v0 = d.kall.clone(), d.vall.clone()
    lens = t.zeros(n, dtype=t.int32, device="cuda")
    offsets, ids = t.zeros(n + 1, dtype=t.int32, device="cuda"), t.zeros_like(d.table)
    at = t.zeros(1, dtype=t.int64, device="cuda")
    first = to_dev(np.array(start, np.int32))
    base = to_dev(np.arange(n + 1, dtype=np.int32))
    rows = t.empty((T, (H + 2 * G) * D), dtype=d.q.dtype, device="cuda")
    q, o1, o2 = (t.empty((T, H, D), dtype=d.q.dtype, device="cuda") for _ in range(3))
    kept = [t.zeros((steps, T, H, D), dtype=d.q.dtype, device="cuda") for _ in range(3)]
    kv = lb.make_paged_kv_cache(d.k, d.v, ids)
    batch = lb.make_packed_batch(offsets, lens, T, max_kv)
    need = max(16, lb.llama_op_attention_paged_decode_workspace_bytes(d.code, n, max_kv, H, G, D),
               lb.llama_op_attention_packed_workspace_bytes(d.code, batch, H, G, D))
    ws = t.empty(need, dtype=t.uint8, device="cuda")

    def step():
        s = t.cuda.current_stream()
        rows.copy_(qkv.index_select(0, at)[0])
        t.add(base, (at % (pad + 1)).to(t.int32), out=offsets)  # the rows start at 0, 1, 2, 0, ...
        t.add(first, (at + 1).to(t.int32), out=lens)
        t.sub(d.table, 0, out=ids)
        lb.check(lb.llama_op_rope_kv_write_paged(d.code, rows, q, kv, batch, table, 500, H, G, D, 0, d.status, s))
        lb.check(lb.llama_op_attention_packed(d.code, q, kv, batch, o1, H, G, D, ws, need, d.status, s))
        for a, b in zip(kept, (q, o1)):
            a.index_copy_(0, at, b[None])
        # decode takes row i for sequence i: the rows moved to the front, then moved away again behind it
        q.copy_(t.gather(q, 0, (t.arange(T, device="cuda") + at % (pad + 1)).clamp(max=T - 1)[:, None, None].expand_as(q)))
        lb.check(lb.llama_op_attention_paged_decode(d.code, q, kv, lens, n, max_kv, o2, H, G, D, ws, need, d.status, s))
        kept[2].index_copy_(0, at, o2[None])
        ids.fill_(-1)
        lens.fill_(-1)
        offsets.fill_(-1)
        at.add_(1)

    side = t.cuda.Stream()
    side.wait_stream(t.cuda.current_stream())
    with t.cuda.stream(side):
        step()  # kernels are set up outside of the capture
    t.cuda.current_stream().wait_stream(side)
    t.cuda.synchronize()
    graph = t.cuda.CUDAGraph()
    with t.cuda.graph(graph):
        step()
    at.zero_()
    d.kall.copy_(k0)
    d.vall.copy_(v0)
    t.cuda.synchronize()
    for _ in range(steps):
        graph.replay()
    t.cuda.synchronize()
    assert int(d.status[0]) == 0
    p.k, p.v = to_host_bits(d.kall), to_host_bits(d.vall)
    qs, packed, decoded = (to_host_bits(a) for a in kept)
    for i in range(steps):
        shift = i % (pad + 1)
        p.kv_lens = [s + i + 1 for s in start]
        p.q = np.concatenate([qs[i][shift:shift + n], qs[i][:pad]])
        ref, bound = p.attention()
        for what, got in (("packed", packed[i][shift:shift + n]), ("decode", decoded[i][:n])):
            err = np.abs(synth.as_f64(got) - ref[:n])
            assert np.all(err <= bound[:n]), f"{what}, replay {i}"
