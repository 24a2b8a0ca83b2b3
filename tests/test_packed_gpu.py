"""Packed batches over a paged cache: RoPE + paged write, packed prompt attention
and paged decode attention against plain 64-bit results (GPU)."""
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


def _finish(d):
    torch().cuda.synchronize()
    return to_f64(d.o), int(d.status[0])


# ------------------------------------------------------ packed attention ---

LENS = [
    ("one_token", [1], [1]),
    ("one_tile", [128], [128]),
    ("tile_plus_one", [129], [129]),
    ("odd_lengths", [1, 130, 17, 63], [1, 130, 17, 63]),
    ("prefixes", [5, 1, 64, 40], [133, 257, 64, 295]),
    ("empty_sequences", [0, 33, 0, 0, 7, 0], [40, 33, 0, 128, 300, 0]),
    ("rows_that_see_nothing", [20, 9, 140], [12, 0, 135]),
    ("longer", [700, 3, 391], [700, 1500, 1024]),
    ("few_rows_many_keys", [2, 70], [9000, 3333]),
]
HEADS = [
    ("bf16", 32, 8, 128), ("bf16", 9, 3, 64), ("bf16", 4, 4, 128), ("bf16", 10, 2, 64), ("bf16", 16, 1, 128),
    ("bf16", 40, 1, 64), ("bf16", 7, 1, 128), ("bf16", 150, 1, 64), ("bf16", 4, 2, 32), ("bf16", 6, 2, 16), ("f32", 4, 2, 16),
    ("f32", 6, 2, 32), ("f32", 9, 3, 64), ("f32", 8, 2, 128),
]


@pytest.mark.parametrize("name,q_lens,kv_lens", LENS, ids=[c[0] for c in LENS])
@pytest.mark.parametrize("dtype,H,G,D", HEADS)
def test_packed_attention(lb, name, q_lens, kv_lens, dtype, H, G, D):
    page = {"one_token": 16, "one_tile": 128, "tile_plus_one": 64, "odd_lengths": 16, "prefixes": 32,
            "empty_sequences": 256, "rows_that_see_nothing": 64, "longer": 32, "few_rows_many_keys": 128}[name]
    p = Problem(f"pk/{name}/{dtype}{H}{G}{D}", dtype, H, G, D, page, q_lens, kv_lens, pad=3)
    d = run_packed(lb, p)
    got, status = _finish(d)
    p.check(got, name)
    assert status == 0


@pytest.mark.parametrize("name,q_lens,kv_lens", LENS, ids=[c[0] for c in LENS])
@pytest.mark.parametrize("dtype,H,G,D", HEADS)
def test_packed_attention_under_a_loose_bound(lb, name, q_lens, kv_lens, dtype, H, G, D):
    """A server that captures one graph for all lengths gives its longest: the work is then dealt out on the device."""
    p = Problem(f"pkl/{name}/{dtype}{H}{G}{D}", dtype, H, G, D, 32, q_lens, kv_lens, pad=2)
    got, status = _finish(run_packed(lb, p, max_kv=1 << 18))
    p.check(got, name)
    assert status == 0


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("bf16", 64), ("f32", 64)])
def test_packed_attention_every_page_size(lb, page, dtype, D):
    p = Problem(f"pkp/{page}{dtype}{D}", dtype, 6, 2, D, page, [70, 1, 300], [471, 777, 300], interleave=True)
    got, status = _finish(run_packed(lb, p))
    p.check(got, f"page {page}")
    assert status == 0


def test_packed_attention_shared_prefix_pages(lb):
    p = Problem("pk/shared", "bf16", 8, 2, 128, 64, [30, 50, 1], [222, 242, 193], shared_prefix=3, rubbish=False)
    got, status = _finish(run_packed(lb, p))
    p.check(got, "shared prefix")
    assert status == 0


@pytest.mark.parametrize("n", [33, 300, 4096])
def test_packed_attention_many_sequences(lb, n):
    rng = np.random.default_rng(n)
    q = rng.integers(0, 4, n)
    kv = q + rng.integers(0, 40, n)
    p = Problem(f"pk/many{n}", "bf16", 2, 1, 64, 16, q.tolist(), kv.tolist(), pad=2)
    got, status = _finish(run_packed(lb, p))
    p.check(got, f"{n} sequences")
    assert status == 0


def test_packed_attention_scores_that_keep_growing(lb):
    # every key's score is above the last one's: the running maximum rises all along the row
    p = Problem("pk/grow", "bf16", 4, 1, 128, 64, [200, 5], [1000, 700])
    k = synth.as_f64(p.k)
    ramp = np.zeros((p.n_pages, 1, 1, p.page, 1))
    for i, L in enumerate(p.kv_lens):
        for pos in range(L):
            ramp[p.table[i, pos // p.page], 0, 0, pos % p.page] = 1.0 + pos / 40.0
    p.k = synth.f32_to_bf16_bits((k * ramp).astype(np.float32))
    got, status = _finish(run_packed(lb, p))
    p.check(got, "growing scores")
    assert status == 0


def test_packed_attention_looser_length_bound_and_dirty_workspace(lb):
    p = Problem("pk/loose", "bf16", 8, 2, 128, 32, [90, 257, 1], [90, 600, 333], pad=1)
    p.table = np.concatenate([p.table, np.full((3, 60), -5, np.int32)], axis=1)
    d = run_packed(lb, p)
    a, _ = _finish(d)
    p.check(a, "tight bound")
    d2 = run_packed(lb, p, max_kv=2400)
    b, status = _finish(d2)
    p.check(b, "loose bound")
    assert status == 0


# ------------------------------------------------------ decode attention ---

DECODE_LENS = [
    ("one", [1]), ("empty", [0, 0]), ("short", [300, 17, 1, 128, 0, 64, 511]), ("chunk_edges", [512, 513, 1024, 255, 256, 257]),
    ("long_one", [9001]), ("ragged", [2049, 0, 5, 4096, 127, 1300, 640]),
]


@pytest.mark.parametrize("name,kv_lens", DECODE_LENS, ids=[c[0] for c in DECODE_LENS])
@pytest.mark.parametrize("dtype,H,G,D", HEADS)
def test_paged_decode(lb, name, kv_lens, dtype, H, G, D):
    page = {"one": 16, "empty": 32, "short": 16, "chunk_edges": 64, "long_one": 32, "ragged": 128}[name]
    p = Problem(f"dec/{name}/{dtype}{H}{G}{D}", dtype, H, G, D, page, [1 if L else 1 for L in kv_lens], kv_lens)
    got, status = _finish(run_decode(lb, p))
    p.check(got, name)
    assert status == 0


@pytest.mark.parametrize("name,kv_lens", DECODE_LENS, ids=[c[0] for c in DECODE_LENS])
@pytest.mark.parametrize("dtype,H,G,D", HEADS)
def test_paged_decode_under_a_loose_bound(lb, name, kv_lens, dtype, H, G, D):
    """A server that captures one graph for all lengths gives its longest: the split is then found on the device."""
    p = Problem(f"decl/{name}/{dtype}{H}{G}{D}", dtype, H, G, D, 64, [1] * len(kv_lens), kv_lens)
    got, status = _finish(run_decode(lb, p, max_kv=1 << 20))
    p.check(got, name)
    assert status == 0


@pytest.mark.parametrize("dtype,H,G,D", [("bf16", 8, 2, 128), ("bf16", 3, 1, 64), ("bf16", 20, 1, 32)])
@pytest.mark.parametrize("n", [31, 32, 33, 64, 1500])
def test_paged_decode_many_sequences_under_a_loose_bound(lb, n, dtype, H, G, D):
    kv = np.random.default_rng(n + D).integers(0, 60, n)
    kv[:3], kv[n - 1] = [2100, 0, 1290], 900
    p = Problem(f"decl/many{n}{D}", dtype, H, G, D, 16, [1] * n, kv.tolist())
    got, status = _finish(run_decode(lb, p, max_kv=1 << 17))
    p.check(got, f"{n} sequences")
    assert status == 0


@pytest.mark.parametrize("n,most", [(16, 1024), (15, 2100), (40, 2050), (80, 1500), (170, 1537)])
def test_paged_decode_more_clusters_than_run_at_once(lb, n, most):
    kv = np.random.default_rng(n).integers(1, most + 1, n)
    kv[0] = most
    p = Problem(f"dec/room{n}", "bf16", 3, 1, 64, 64, [1] * n, kv.tolist())
    got, status = _finish(run_decode(lb, p))
    p.check(got, f"{n} sequences of up to {most}")
    assert status == 0


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("bf16", 64), ("f32", 64)])
def test_paged_decode_every_page_size(lb, page, dtype, D):
    p = Problem(f"decp/{page}{dtype}{D}", dtype, 6, 2, D, page, [1, 1, 1], [471, 1777, 300], interleave=True)
    got, status = _finish(run_decode(lb, p, max_kv=1777 + 15))
    p.check(got, f"page {page}")
    assert status == 0


@pytest.mark.parametrize("n", [65, 1000, 4096])
def test_paged_decode_many_sequences(lb, n):
    kv = np.random.default_rng(n).integers(0, 50, n)
    kv[n // 2] = 700
    p = Problem(f"dec/many{n}", "bf16", 2, 1, 64, 16, [1] * n, kv.tolist())
    got, status = _finish(run_decode(lb, p))
    p.check(got, f"{n} sequences")
    assert status == 0


def test_paged_decode_is_the_last_row_of_packed(lb):
    p = Problem("dec/same", "bf16", 32, 8, 128, 64, [1] * 4, [1000, 37, 2048, 513])
    a, _ = _finish(run_decode(lb, p))
    b, _ = _finish(run_packed(lb, p))
    _, bound = p.attention()
    assert np.all(np.abs(a - b) <= 2 * bound)


@pytest.mark.parametrize("dtype,H,G,D", [("bf16", 32, 8, 128), ("bf16", 9, 3, 64), ("f32", 4, 2, 16)])
def test_runs_repeat_bit_for_bit_on_a_dirty_workspace(lb, dtype, H, G, D):
    t = torch()
    p = Problem(f"rep/{dtype}{D}", dtype, H, G, D, 32, [1] * 5, [3000, 1, 700, 2222, 64])
    w = t.full((64 << 20,), 0x7F, dtype=t.uint8, device="cuda")  # larger than asked for: fine
    first = to_host_bits(run_decode(lb, p, workspace=w).o)
    packed = to_host_bits(run_packed(lb, p, workspace=w).o)
    for _ in range(3):
        assert np.array_equal(first, to_host_bits(run_decode(lb, p, workspace=w).o))
        assert np.array_equal(packed, to_host_bits(run_packed(lb, p, workspace=w).o))


# --------------------------------------------- bad lengths, offsets, ids ---

def test_bad_lengths_count_as_zero(lb):
    p = Problem("bad/len", "bf16", 4, 2, 128, 16, [1, 1, 1, 1], [40, 33, 20, 25])
    d = p.device(lb)
    d.kv_lens[1] = -3
    d.kv_lens[2] = 41  # above max_kv_len = 40
    run_decode(lb, p, d)
    got, status = _finish(d)
    assert status == lb.LLAMA_ERR_RANGE
    assert np.all(got[1:3] == 0.0)
    p.kv_lens[1] = p.kv_lens[2] = 0
    p.check(got, "decode, bad lengths")
    d.o.fill_(7.0)
    d.status.zero_()
    run_packed(lb, p, d)
    got, status = _finish(d)
    assert status == lb.LLAMA_ERR_RANGE
    p.check(got, "packed, bad lengths")


@pytest.mark.parametrize("n", [4, 40])
def test_bad_lengths_count_as_zero_under_a_loose_bound(lb, n):
    p = Problem(f"bad/lenl{n}", "bf16", 4, 2, 64, 16, [1] * n, [40, 33, 700, 25] * (n // 4))
    d = p.device(lb)
    bound = 1 << 17
    d.kv_lens[1] = -(1 << 31)
    d.kv_lens[n - 1] = bound + 1
    d.kv_lens[n - 4] = p.table.shape[1] * 16 + 1  # more than the pages of a row hold
    p.kv_lens[1] = p.kv_lens[n - 1] = p.kv_lens[n - 4] = 0
    for run in (run_decode, run_packed):
        d.o.fill_(7.0)
        d.status.zero_()
        run(lb, p, d, max_kv=bound)
        got, status = _finish(d)
        assert status == lb.LLAMA_ERR_RANGE
        p.check(got, run.__name__)


@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("bf16", 64), ("f32", 32)])
@pytest.mark.parametrize("bad_id", [-1, 1 << 20, -(1 << 31)])
def test_bad_page_ids_read_as_zeros(lb, dtype, D, bad_id):
    p = Problem(f"bad/id{dtype}{D}", dtype, 4, 2, D, 16, [1, 1, 1], [400, 33, 90])
    d = p.device(lb)
    where = int(p.table[0, 3])
    d.table[0, 3] = bad_id
    p.k[where], p.v[where] = 0, 0  # the page as it has to read
    run_decode(lb, p, d)
    got, status = _finish(d)
    assert status == lb.LLAMA_ERR_RANGE
    p.check(got, "decode, bad page id")
    d.o.fill_(7.0)
    d.status.zero_()
    run_packed(lb, p, d)
    got, status = _finish(d)
    assert status == lb.LLAMA_ERR_RANGE
    p.check(got, "packed, bad page id")


def test_bad_offsets_leave_the_sequence_out(lb):
    p = Problem("bad/off", "bf16", 4, 2, 64, 16, [8, 8, 8, 8], [20, 30, 8, 41])
    d = p.device(lb)
    d.offsets[2] = 3  # sequence 1 ends before it starts; sequence 2 then covers rows 3 .. 24
    run_packed(lb, p, d)
    got, status = _finish(d)
    assert status == lb.LLAMA_ERR_RANGE
    assert np.all(np.isfinite(got))
    d.offsets.copy_(to_dev(p.offsets))
    d.offsets[4] = 33  # behind the last row
    d.o.fill_(7.0)
    d.status.zero_()
    run_packed(lb, p, d)
    got, status = _finish(d)
    assert status == lb.LLAMA_ERR_RANGE
    assert np.all(got[24:] == 7.0)
    ref, bound = p.attention()
    assert np.all(np.abs(got[:24] - ref[:24]) <= bound[:24])


@pytest.mark.parametrize("dtype,H,G,D", [("bf16", 40, 1, 64), ("bf16", 4, 2, 128), ("f32", 4, 2, 32)])
def test_offsets_that_descend_stay_in_bounds(lb, dtype, H, G, D):
    """Every other sequence claims all rows: more blocks than the plan has room for, and nothing behind it written."""
    p = Problem("bad/desc", dtype, H, G, D, 16, [60] * 40, [1500] * 40)
    d = p.device(lb)
    n = len(p.kv_lens)
    d.offsets.copy_(to_dev(np.asarray([0 if i % 2 == 0 else p.T for i in range(n + 1)], dtype=np.int32)))
    need = lb.llama_op_attention_packed_workspace_bytes(d.code, d.batch, H, G, D)
    ws = torch().full((need + 4096,), 0xA5, dtype=torch().uint8, device="cuda")
    lb.check(lb.llama_op_attention_packed(d.code, d.q, d.kv, d.batch, d.o, H, G, D, ws, need, d.status))
    got, status = _finish(d)
    assert status == lb.LLAMA_ERR_RANGE
    assert bool((ws[need:] == 0xA5).all())
    d.offsets.copy_(to_dev(p.offsets))  # and the next call is right
    d.status.zero_()
    run_packed(lb, p, d)
    got, status = _finish(d)
    assert status == 0
    p.check(got, "after the bad call")


@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("f32", 32)])
def test_bound_of_no_keys(lb, dtype, D):
    p = Problem("bound0", dtype, 4, 2, D, 16, [3, 0, 2], [0, 0, 0])
    for run in (run_packed, run_decode):
        d = run(lb, p)
        got, status = _finish(d)
        assert status == 0
        assert np.all((got if run is run_packed else got[:3]) == 0.0)


# ----------------------------------------------------- RoPE + page write ---

@pytest.mark.parametrize("layout", ["interleaved", "halves"])
@pytest.mark.parametrize("dtype,H,G,D,page", [("bf16", 32, 8, 128, 64), ("bf16", 9, 3, 64, 16), ("f32", 4, 2, 16, 16),
                                              ("f32", 5, 1, 128, 256), ("bf16", 3, 3, 32, 32), ("bf16", 2, 1, 16, 16)])
def test_rope_kv_write_paged(lb, layout, dtype, H, G, D, page):
    t = torch()
    q_lens, kv_lens = [37, 1, 0, 70, 1, 5], [37, 300, 12, 111, 1, 2]  # the last one: 3 tokens before position 0
    p = Problem(f"wr/{layout}{dtype}{H}{G}{D}", dtype, H, G, D, page, q_lens, kv_lens, pad=4, interleave=True)
    d = p.device(lb)
    qkv = store(synth.normal(0, f"wr/qkv{dtype}{H}{G}{D}", (p.T, (H + 2 * G) * D)), dtype)
    max_seq, theta = 300, 1e4
    table = t.empty((max_seq, D // 2, 2), dtype=t.float32, device="cuda")
    lb.check(lb.llama_op_rope_table(table, max_seq, D, theta))
    lay = lb.LLAMA_ROPE_HALVES if layout == "halves" else lb.LLAMA_ROPE_INTERLEAVED
    before_k, before_v = to_host_bits(d.kall).copy(), to_host_bits(d.vall).copy()
    lb.check(lb.llama_op_rope_kv_write_paged(d.code, to_dev(qkv), d.o, d.kv, d.batch, table, max_seq, H, G, D, lay,
                                             d.status, t.cuda.current_stream()))
    t.cuda.synchronize()
    got_q, got_k, got_v = to_f64(d.o), to_host_bits(d.kall), to_host_bits(d.vall)
    x = synth.as_f64(qkv).reshape(p.T, H + 2 * G, D)
    u = U_BF16 if dtype == "bf16" else U32
    as64 = synth.as_f64
    seen = np.zeros(before_k.shape, dtype=bool)
    for i, (n, L) in enumerate(zip(q_lens, kv_lens)):
        for j in range(n):
            row, pos = int(p.offsets[i]) + j, L - n + j
            if pos < 0:
                assert np.all(got_q[row] == 0.0)
                continue
            rot = oracle.rope(x[row][None, None, :H + G], np.array([pos]), theta, layout)[0, 0]
            half = np.abs(x[row, :H + G])
            # two products of a rounded cos / sin and their sum, then the store
            slack = 4 * U32 * (half + half.max(axis=-1, keepdims=True))
            assert np.all(np.abs(got_q[row] - rot[:H]) <= u * 1.01 * np.abs(rot[:H]) + slack[:H])
            page_id, slot = p.table[i, pos // page], pos % page
            assert np.all(np.abs(as64(got_k[page_id, 0, :, slot]) - rot[H:]) <= u * 1.01 * np.abs(rot[H:]) + slack[H:])
            assert np.array_equal(got_v[page_id, 0, :, slot], qkv[row].reshape(-1, D)[H + G:])
            seen[page_id, 0, :, slot] = True
    assert int(d.status[0]) == lb.LLAMA_ERR_RANGE  # the tokens before position 0
    same = lambda a, b: np.array_equal(a.view(np.uint8 if a.dtype != np.uint16 else np.uint16),
                                       b.view(np.uint8 if b.dtype != np.uint16 else np.uint16))
    assert same(got_k[~seen], before_k[~seen]) and same(got_v[~seen], before_v[~seen])
    assert np.all(got_q[p.offsets[-1]:] == 7.0)


def test_rope_kv_write_paged_bad_ids_and_positions(lb):
    t = torch()
    H, G, D = 4, 2, 64
    p = Problem("wr/bad", "bf16", H, G, D, 16, [40, 20], [40, 60], rubbish=False)
    d = p.device(lb)
    qkv = to_dev(store(synth.normal(0, "wr/badqkv", (p.T, (H + 2 * G) * D)), "bf16"))
    table = t.empty((50, D // 2, 2), dtype=t.float32, device="cuda")
    lb.check(lb.llama_op_rope_table(table, 50, D, 1e4))
    before = d.kall.clone()
    lost = int(p.table[0, 1])
    d.table[0, 1] = p.n_pages  # positions 16 .. 31 of sequence 0
    lb.check(lb.llama_op_rope_kv_write_paged(d.code, qkv, d.o, d.kv, d.batch, table, 50, H, G, D, 0, d.status))
    t.cuda.synchronize()
    assert int(d.status[0]) == lb.LLAMA_ERR_RANGE
    assert t.equal(d.kall[lost], before[lost])
    assert not t.equal(d.kall[int(p.table[0, 0])], before[int(p.table[0, 0])])
    assert bool((d.o[:40] != 0).any(-1).all())      # q does not need the page
    assert bool((d.o[50:] == 0).all())              # positions 50 .. 59 are past the table
    tail = int(p.table[1, 3])                       # positions 48 .. 59 of sequence 1
    assert not t.equal(d.kall[tail, 0, :, :2], before[tail, 0, :, :2])
    assert t.equal(d.kall[tail, 0, :, 2:], before[tail, 0, :, 2:])


# -------------------------------------------------------- used together ---

def _serve(lb, layout, dtype, H, G, D, page, steps, prompt_lens, chunk):
    """Prompts in chunks, then decode steps, each written and attended through the pages; against the oracle's
    rope and attention over a plain contiguous history.  Returns the largest error over its bound."""
    t = torch()
    n = len(prompt_lens)
    total = [L + steps for L in prompt_lens]
    max_seq = max(total)
    p = Problem(f"serve/{layout}{dtype}{D}", dtype, H, G, D, page, [1] * n, total)
    d = p.device(lb)
    code = d.code
    lay = lb.LLAMA_ROPE_HALVES if layout == "halves" else lb.LLAMA_ROPE_INTERLEAVED
    table = t.empty((max_seq, D // 2, 2), dtype=t.float32, device="cuda")
    lb.check(lb.llama_op_rope_table(table, max_seq, D, 1e4))
    x = [store(synth.normal(0, f"serve/x{i}", (L, (H + 2 * G) * D)), dtype) for i, L in enumerate(total)]
    done = [0] * n
    outs = [[] for _ in range(n)]

    def step(counts, decode):
        rows = np.concatenate([x[i][done[i]:done[i] + c] for i, c in enumerate(counts)])
        off = to_dev(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32))
        lens = to_dev(np.array([a + c for a, c in zip(done, counts)], dtype=np.int32))
        T = len(rows)
        b = lb.make_packed_batch(off, lens, T, max_seq)
        q = t.empty((T, H, D), dtype=d.q.dtype, device="cuda")
        o = t.empty_like(q)
        stream = t.cuda.current_stream()
        lb.check(lb.llama_op_rope_kv_write_paged(code, to_dev(rows), q, d.kv, b, table, max_seq, H, G, D, lay,
                                                 d.status, stream))
        if decode:
            need = lb.llama_op_attention_paged_decode_workspace_bytes(code, n, max_seq, H, G, D)
            ws = t.empty(max(need, 16), dtype=t.uint8, device="cuda")
            lb.check(lb.llama_op_attention_paged_decode(code, q, d.kv, lens, n, max_seq, o, H, G, D, ws, ws.numel(),
                                                        d.status, stream))
        else:
            need = lb.llama_op_attention_packed_workspace_bytes(code, b, H, G, D)
            ws = t.empty(max(need, 16), dtype=t.uint8, device="cuda")
            lb.check(lb.llama_op_attention_packed(code, q, d.kv, b, o, H, G, D, ws, ws.numel(), d.status, stream))
        t.cuda.synchronize()
        o = to_f64(o)
        at = 0
        for i, c in enumerate(counts):
            outs[i].append(o[at:at + c])
            at += c
            done[i] += c

    while any(a < b for a, b in zip(done, prompt_lens)):
        step([min(chunk, b - a) for a, b in zip(done, prompt_lens)], False)
    for _ in range(steps):
        step([1] * n, True)
    assert int(d.status[0]) == 0
    worst = 0.0
    for i in range(n):
        xi = synth.as_f64(x[i]).reshape(total[i], H + 2 * G, D)
        rot = oracle.rope(xi[None, :, :H + G], np.arange(total[i]), 1e4, layout)[0]
        kc, vc = rot[None, :, H:].transpose(0, 2, 1, 3), xi[None, :, H + G:].transpose(0, 2, 1, 3)
        ref = oracle.gqa_attention(rot[None, :, :H], kc, vc, 0)[0]
        got = np.concatenate(outs[i])
        err = np.linalg.norm(got - ref) / np.linalg.norm(ref)
        worst = max(worst, float(err))
    return worst


@pytest.mark.parametrize("layout,dtype,H,G,D,page", [("interleaved", "bf16", 32, 8, 128, 64),
                                                     ("halves", "bf16", 9, 3, 64, 16),
                                                     ("interleaved", "f32", 4, 2, 16, 16)])
def test_prompt_in_chunks_then_decode(lb, layout, dtype, H, G, D, page):
    # the framework's parity bars: relative Frobenius 5e-3 (bf16), 1e-4 (fp32)
    err = _serve(lb, layout, dtype, H, G, D, page, steps=5, prompt_lens=[150, 1, 333, 64], chunk=128)
    assert err <= (5e-3 if dtype == "bf16" else 1e-4), err


def test_captured_step_follows_the_lengths(lb):
    """One graph of write + decode, replayed while the conversation grows."""
    t = torch()
    H, G, D, page, n, most = 8, 2, 128, 32, 3, 700
    start = [5, 300, 690]
    p = Problem("graph", "bf16", H, G, D, page, [1] * n, [most] * n, rubbish=False)
    d = p.device(lb)
    table = t.empty((most, D // 2, 2), dtype=t.float32, device="cuda")
    lb.check(lb.llama_op_rope_table(table, most, D, 1e4))
    qkv = to_dev(store(synth.normal(0, "graph/qkv", (n, (H + 2 * G) * D)), "bf16"))
    q = t.empty((n, H, D), dtype=t.bfloat16, device="cuda")
    lens = to_dev(np.array(start, dtype=np.int32))
    batch = lb.make_packed_batch(d.offsets, lens, n, most)
    ws = t.empty(max(16, lb.llama_op_attention_paged_decode_workspace_bytes(d.code, n, most, H, G, D)),
                 dtype=t.uint8, device="cuda")
    ws2 = t.empty(max(16, lb.llama_op_attention_packed_workspace_bytes(d.code, batch, H, G, D)), dtype=t.uint8,
                  device="cuda")
    o2 = t.empty_like(q)

    def step():
        s = t.cuda.current_stream()
        lb.check(lb.llama_op_rope_kv_write_paged(d.code, qkv, q, d.kv, batch, table, most, H, G, D, 0, d.status, s))
        lb.check(lb.llama_op_attention_paged_decode(d.code, q, d.kv, lens, n, most, d.o, H, G, D, ws, ws.numel(),
                                                    d.status, s))
        lb.check(lb.llama_op_attention_packed(d.code, q, d.kv, batch, o2, H, G, D, ws2, ws2.numel(), d.status, s))

    k0, v0 = d.kall.clone(), d.vall.clone()
    graph = t.cuda.CUDAGraph()
    side = t.cuda.Stream()
    side.wait_stream(t.cuda.current_stream())
    with t.cuda.stream(side):
        step()  # kernels are set up outside of the capture
    t.cuda.current_stream().wait_stream(side)
    with t.cuda.graph(graph):
        step()
    d.kall.copy_(k0)
    d.vall.copy_(v0)
    for grow in range(4):
        lens.copy_(to_dev(np.array([a + grow for a in start], dtype=np.int32)))
        graph.replay()
        t.cuda.synchronize()
        p.kv_lens = [a + grow for a in start]
        p.q, p.k, p.v = to_host_bits(q), to_host_bits(d.kall), to_host_bits(d.vall)
        p.check(to_f64(d.o), f"decode, replay {grow}")
        p.check(to_f64(o2), f"packed, replay {grow}")
    assert int(d.status[0]) == 0


def test_two_streams_with_their_own_workspaces(lb):
    t = torch()
    a = Problem("str/a", "bf16", 32, 8, 128, 64, [1] * 6, [3000, 10, 2000, 600, 4000, 1])
    b = Problem("str/b", "bf16", 9, 3, 64, 16, [200, 40], [800, 1040])
    da, db = a.device(lb), b.device(lb)
    wa, wb = (t.empty(32 << 20, dtype=t.uint8, device="cuda") for _ in range(2))
    t.cuda.synchronize()
    s1, s2 = t.cuda.Stream(), t.cuda.Stream()
    for _ in range(20):
        run_decode(lb, a, da, stream=s1, workspace=wa)
        run_packed(lb, b, db, stream=s2, workspace=wb)
    t.cuda.synchronize()
    a.check(to_f64(da.o), "stream 1")
    b.check(to_f64(db.o), "stream 2")


# ------------------------------------------------- far offsets, long keys ---

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_pages_more_than_four_gigabytes_apart(lb, dtype):
    """Page offsets past 2^32 bytes and 2^31 elements (a pool whose pages lie far apart)."""
    t = torch()
    H, G, D, page = 4, 2, 64, 16
    p = Problem(f"far/{dtype}", dtype, H, G, D, page, [20, 1], [20, 40], spare=0, rubbish=False)
    d = p.device(lb)
    stride = (3 << 29) // (1 if dtype == "bf16" else 2)  # elements; 5 pages
    pools = []
    for src in (d.k, d.v):
        pool = t.empty((p.n_pages - 1) * stride + G * page * D, dtype=src.dtype, device="cuda")
        view = t.as_strided(pool, (p.n_pages, G, page, D), (stride, page * D, D, 1))
        view.copy_(src)
        pools.append(view)
    assert (p.n_pages - 1) * stride * pools[0].element_size() > 1 << 32
    d.kv = lb.make_paged_kv_cache(pools[0], pools[1], d.table)
    run_packed(lb, p, d)
    got, status = _finish(d)
    p.check(got, "packed")
    # decode: one row per sequence, the first rows of q
    q = Problem(f"far/{dtype}", dtype, H, G, D, page, [1, 1], [20, 40], spare=0, rubbish=False)
    q.table, q.k, q.v, q.n_pages = p.table, p.k, p.v, p.n_pages
    q.q = p.q[:2]
    d.o.fill_(7.0)
    lens = to_dev(np.array([20, 40], np.int32))
    need = lb.llama_op_attention_paged_decode_workspace_bytes(d.code, 2, 40, H, G, D)
    ws = t.empty(max(16, need), dtype=t.uint8, device="cuda")
    lb.check(lb.llama_op_attention_paged_decode(d.code, d.q, d.kv, lens, 2, 40, d.o, H, G, D, ws, ws.numel(), d.status))
    t.cuda.synchronize()
    q.check(to_f64(d.o)[:2], "decode")
    # write: the same pages as in a dense pool
    qkv = to_dev(store(synth.normal(0, "far/qkv", (p.T, (H + 2 * G) * D)), dtype))
    table = t.empty((64, D // 2, 2), dtype=t.float32, device="cuda")
    lb.check(lb.llama_op_rope_table(table, 64, D, 1e4))
    dense = [d.k.clone(), d.v.clone()]
    for k, v in (pools, dense):
        lb.check(lb.llama_op_rope_kv_write_paged(d.code, qkv, d.o, lb.make_paged_kv_cache(k, v, d.table), d.batch,
                                                 table, 64, H, G, D, 0, d.status))
    t.cuda.synchronize()
    assert not t.equal(dense[0], d.k)
    assert t.equal(pools[0], dense[0]) and t.equal(pools[1], dense[1])
    assert int(d.status[0]) == 0 and status == 0


def test_packed_attention_very_long_keys(lb):
    p = Problem("pk/150k", "bf16", 4, 1, 64, 256, [3, 40, 1], [150001, 200, 140000], rubbish=False)
    got, status = _finish(run_packed(lb, p))
    p.check(got, "150001 keys")
    assert status == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_paged_decode_very_long_keys(lb, dtype):
    p = Problem(f"dec/150k{dtype}", dtype, 4, 1, 64, 128, [1, 1], [150001, 77], rubbish=False)
    got, status = _finish(run_decode(lb, p))
    p.check(got, "150001 keys")
    assert status == 0


def test_packed_attention_more_blocks_than_the_planner_keeps(lb):
    """128 heads per KV head make a block of every two positions: 6000 blocks.  An item does not
    depend on its company, so the batch has to equal its two halves bit for bit."""
    t = torch()
    n, H, D, page = 2000, 128, 64, 16
    p = Problem("pk/blocks", "bf16", H, 1, D, page, [5] * n, [9] * n, rubbish=False)
    d = p.device(lb)
    d.batch = lb.make_packed_batch(d.offsets, d.kv_lens, p.T, 2000)  # a bound that rules out no split
    run_packed(lb, p, d, max_kv=2000)
    t.cuda.synchronize()
    whole = d.o.clone()
    assert int(d.status[0]) == 0
    d.o.zero_()
    for a, b in ((0, n // 2), (n // 2, n)):
        rows = slice(int(p.offsets[a]), int(p.offsets[b]))
        q, o = d.q[rows].contiguous(), t.zeros_like(d.o[rows])
        off, lens = (d.offsets[a:b + 1] - d.offsets[a]).contiguous(), d.kv_lens[a:b].clone()
        batch = lb.make_packed_batch(off, lens, q.shape[0], 2000)
        kv = lb.make_paged_kv_cache(d.k, d.v, d.table[a:b].clone())
        ws = t.empty(lb.llama_op_attention_packed_workspace_bytes(d.code, batch, H, 1, D), dtype=t.uint8,
                     device="cuda")
        lb.check(lb.llama_op_attention_packed(d.code, q, kv, batch, o, H, 1, D, ws, ws.numel(), d.status))
        d.o[rows] = o
    t.cuda.synchronize()
    assert t.equal(whole, d.o)
    assert bool(t.isfinite(whole.float()).all())


def test_two_graphs_share_a_workspace(lb):
    t = torch()
    a = Problem("share/a", "bf16", 32, 8, 128, 64, [1] * 7, [3000, 10, 2000, 600, 4000, 1, 2500])
    b = Problem("share/b", "bf16", 8, 2, 128, 32, [300, 2, 1], [1300, 5000, 700])
    c = Problem("share/c", "f32", 8, 2, 64, 32, [30, 2, 1], [1300, 900, 700])
    da, db, dc = a.device(lb), b.device(lb), c.device(lb)
    need = [lb.llama_op_attention_paged_decode_workspace_bytes(da.code, 7, a.max_kv, 32, 8, 128),
            lb.llama_op_attention_packed_workspace_bytes(db.code, db.batch, 8, 2, 128),
            lb.llama_op_attention_packed_workspace_bytes(dc.code, dc.batch, 8, 2, 64)]
    assert min(need) > 0
    ws = t.empty(max(need), dtype=t.uint8, device="cuda")
    graphs = []
    for run, p, d in ((run_decode, a, da), (run_packed, b, db), (run_packed, c, dc)):
        run(lb, p, d, workspace=ws)
        t.cuda.synchronize()
        g = t.cuda.CUDAGraph()
        with t.cuda.graph(g):
            run(lb, p, d, workspace=ws)
        graphs.append(g)
    for d in (da, db, dc):
        d.o.fill_(7.0)
    for _ in range(5):
        for g in graphs:
            g.replay()
    t.cuda.synchronize()
    for p, d in ((a, da), (b, db), (c, dc)):
        p.check(to_f64(d.o), "shared workspace")
        assert int(d.status[0]) == 0


def test_workspace_too_small_is_refused(lb):
    t = torch()
    p = Problem("ws", "bf16", 32, 8, 128, 64, [40, 1], [3000, 2000])
    d = p.device(lb)
    need = lb.llama_op_attention_packed_workspace_bytes(d.code, d.batch, 32, 8, 128)
    ws = t.empty(need, dtype=t.uint8, device="cuda")
    assert lb.llama_op_attention_packed(d.code, d.q, d.kv, d.batch, d.o, 32, 8, 128, ws, need - 1, d.status) \
        == lb.LLAMA_ERR_RANGE
    assert lb.llama_op_attention_packed(d.code, d.q, d.kv, d.batch, d.o, 32, 8, 128, None, need, d.status) \
        == lb.LLAMA_ERR_INVALID_ARG
    # 40 sequences of up to 3000 keys: too many for clusters, so planned
    need = lb.llama_op_attention_paged_decode_workspace_bytes(d.code, 40, 3000, 32, 8, 128)
    assert need > 0
    lens = t.ones(40, dtype=t.int32, device="cuda")
    q = t.zeros((40, 32, 128), dtype=t.bfloat16, device="cuda")
    tab = t.zeros((40, 47), dtype=t.int32, device="cuda")
    kv = lb.make_paged_kv_cache(d.k, d.v, tab)
    assert lb.llama_op_attention_paged_decode(d.code, q, kv, lens, 40, 3000, q, 32, 8, 128, ws, need - 1) \
        == lb.LLAMA_ERR_RANGE
    t.cuda.synchronize()
    assert bool((d.o == 7.0).all())
