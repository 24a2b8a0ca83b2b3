"""The 4-bit cache on the GPU: writing, reading, attention over it."""
import numpy as np
import pytest

import synth
from _helpers import to_dev, to_f64, to_host_bits, torch
from _kv4 import F32, Kv4Problem, blocks, pack, quantise, run_decode, run_packed, unpack, values
from _packed import hash_tag, store

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lb():
    import decoder_block_gb300 as m
    m.load()
    return m


def _table(n, D, theta=1e4):
    ang = np.arange(n)[:, None] * theta ** (-2.0 * np.arange(D // 2) / D)
    return np.stack([np.cos(ang), np.sin(ang)], -1).astype(F32)


def _rotate(x, cs, halves):
    """fp32 [T][heads][D] turned by cs [T][D / 2][2], each operation rounded to fp32."""
    D = x.shape[-1]
    c, s = cs[:, None, :, 0], cs[:, None, :, 1]
    a, b = (x[..., :D // 2], x[..., D // 2:]) if halves else (x[..., 0::2], x[..., 1::2])
    p, q = a * c - b * s, a * s + b * c
    if halves:
        return np.concatenate([p, q], -1)
    return np.stack([p, q], -1).reshape(x.shape)


class WriteCase:
    def __init__(self, tag, dtype, H, G, D, page, q_lens, kv_lens, halves, pad=0, size=1.0):
        self.p = p = Kv4Problem(tag, dtype, H, G, D, page, q_lens, kv_lens, pad=pad)
        self.dtype, self.halves = dtype, halves
        qkv = synth.normal(0, tag + "/qkv", (p.T, (H + 2 * G) * D)) * F32(size)
        self.set(qkv)
        self.table = _table(max(max(kv_lens), 1) + 3, D)

    def set(self, qkv):
        p = self.p
        self.qkv = store(qkv.astype(F32), self.dtype)
        self.x = synth.as_f64(self.qkv).astype(F32).reshape(p.T, p.H + 2 * p.G, p.D)

    def expected(self):
        """q_out (fp32, 7 where untouched) and the two pools."""
        p = self.p
        q = np.full((p.T, p.H, p.D), 7.0, F32)
        pools = [x.copy() for x in p.pools]
        for i, (n, L) in enumerate(zip(p.q_lens, p.kv_lens)):
            rows = np.arange(p.offsets[i], p.offsets[i + 1])
            pos = L - n + np.arange(n)
            ok = pos >= 0
            q[rows[~ok]] = 0.0
            rows, pos = rows[ok], pos[ok]
            if not len(rows):
                continue
            with np.errstate(invalid="ignore", over="ignore"):
                rot = _rotate(self.x[rows, :p.H + p.G], self.table[pos], self.halves)
            q[rows] = rot[:, :p.H]
            for pool, new in zip(pools, (rot[:, p.H:], self.x[rows, p.H + p.G:])):
                codes, byte = unpack(pool, p.page, p.D)
                c, b = quantise(new)
                at = p.table[i, pos // p.page]
                codes[at, :, pos % p.page] = c
                byte = byte.copy()
                byte[at, :, pos % p.page] = b
                pool[:] = np.concatenate([pack(codes).reshape(*pool.shape[:2], -1), byte.reshape(*pool.shape[:2], -1)], -1)
        return q, pools

    def run(self, lb, d=None):
        t = torch()
        p = self.p
        d = d or p.device(lb)
        d.q_out = t.full((p.T, p.H, p.D), 7.0, dtype=d.q.dtype, device="cuda")
        lb.check(lb.llama_op_rope_kv4_write_paged(d.code, to_dev(self.qkv), d.q_out, d.kv, d.batch, to_dev(self.table),
                                                  len(self.table), p.H, p.G, p.D, 1 if self.halves else 0, d.status,
                                                  t.cuda.current_stream()))
        t.cuda.synchronize()
        return d

    def check(self, d):
        q, pools = self.expected()
        want = store(q, self.dtype)
        assert np.array_equal(to_host_bits(d.q_out).view(want.dtype), want)
        for name, got, pool in zip("kv", (d.k, d.v), pools):
            bad = np.nonzero(got.cpu().numpy() != pool)
            assert not len(bad[0]), f"{name}: {len(bad[0])} bytes differ, first {[int(b[0]) for b in bad]}"


SHAPES = [("bf16", 32, 8, 128, 64), ("bf16", 9, 3, 64, 16), ("bf16", 4, 4, 32, 32), ("bf16", 6, 2, 16, 16),
          ("f32", 4, 2, 128, 256), ("f32", 5, 5, 64, 128), ("f32", 8, 2, 32, 16), ("f32", 4, 1, 16, 64)]


@pytest.mark.parametrize("halves", [False, True])
@pytest.mark.parametrize("dtype,H,G,D,page", SHAPES)
@pytest.mark.parametrize("q_lens,kv_lens,pad", [([1], [1], 0), ([1, 0, 17, 40], [130, 5, 17, 300], 3),
                                                ([700, 1000], [700, 1100], 1)])
def test_write(lb, dtype, H, G, D, page, halves, q_lens, kv_lens, pad):
    c = WriteCase(f"w{dtype}{D}{len(q_lens)}", dtype, H, G, D, page, q_lens, kv_lens, halves, pad)
    d = c.run(lb)
    c.check(d)
    assert int(d.status[0]) == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("size", [1e-30, 1e-6, 3e-3, 50.0, 4000.0])
def test_write_sizes(lb, dtype, size):
    c = WriteCase("sizes", dtype, 2, 2, 64, 16, [33], [40], False, size=size)
    d = c.run(lb)
    c.check(d)
    assert int(d.status[0]) == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind,code", [("nan", 1), ("inf", 1), ("huge", 1), ("most", 0), ("zero", 0)])
def test_write_values_that_do_not_fit(lb, dtype, kind, code):
    c = WriteCase("odd", dtype, 2, 2, 32, 16, [9], [9], True)
    x = c.x.copy()
    v = x[:, 4:]  # the values: not rotated
    v[2, 1, 5] = dict(nan=np.nan, inf=-np.inf, huge=30000.0, most=26880.0, zero=0.0)[kind]
    if kind == "nan":
        v[3, 0, 16:32] = np.nan
    if kind == "zero":
        v[4] = 0.0
    c.set(x.reshape(9, -1))
    d = c.run(lb)
    c.check(d)
    assert int(d.status[0]) == (lb.LLAMA_ERR_RANGE if code else 0)


def test_write_positions_and_pages_out_of_range(lb):
    t = torch()
    c = WriteCase("range", "bf16", 2, 1, 64, 16, [5, 4, 3], [3, 40, 3], False)
    c.table = _table(38, 64)  # positions 38 and 39 of the second sequence are behind it
    p = c.p
    p.table[2, 0] = -1
    d = c.run(lb)
    got = to_f64(d.q_out)
    assert np.all(got[:2] == 0) and np.all(got[7:9] == 0)  # before the sequence's start, behind the table
    assert np.all(np.abs(got[[2, 3, 4, 5, 6, 9, 10, 11]]).max((1, 2)) > 0)
    assert int(d.status[0]) == lb.LLAMA_ERR_RANGE
    changed = (d.k.cpu().numpy() != p.pools[0]).any((1, 2))
    allowed = {int(p.table[0, 0]), int(p.table[1, 2])}
    assert set(np.nonzero(changed)[0].tolist()) <= allowed
    t.cuda.synchronize()


@pytest.mark.parametrize("halves", [False, True])
@pytest.mark.parametrize("dtype,H,G,D,page", [("bf16", 4, 2, 128, 16), ("bf16", 2, 1, 64, 32), ("f32", 3, 3, 16, 16)])
def test_write_stores_the_rows_in_range_and_no_other_byte(lb, dtype, H, G, D, page, halves):
    """Rows before their sequence's start, positions behind the table, page ids out of range at a first and at a later
    page, beside rows that are fine, some of them in the same sequences: both pools byte for byte, q_out bit for bit."""
    c = WriteCase(f"wr{dtype}{D}", dtype, H, G, D, page, [5, 4, 3, 2 * page + 3, page + 9, 2],
                  [3, 40, 3, 3 * page, 3 * page - 5, 1], halves, pad=2)
    p, limit = c.p, 3 * page - 2
    c.table = _table(limit, D)     # the fourth sequence's last two positions are behind it
    p.table[2, 0] = -1
    p.table[3, 1] = p.n_pages      # the middle page: rows before and behind it are stored
    p.table[4, 2] = 0x7fffffff
    q, pools = np.full((p.T, H, D), 7.0, F32), [x.copy() for x in p.pools]
    stored = 0
    for i, (n, L) in enumerate(zip(p.q_lens, p.kv_lens)):
        for t in range(n):
            row, pos = p.offsets[i] + t, L - n + t
            if not 0 <= pos < limit:
                q[row] = 0.0
                continue
            rot = _rotate(c.x[row:row + 1, :H + G], c.table[pos:pos + 1], halves)[0]
            q[row] = rot[:H]
            at = int(p.table[i, pos // page])
            if not 0 <= at < p.n_pages:
                continue
            stored += 1
            for pool, new in zip(pools, (rot[H:], c.x[row, H + G:])):
                codes, byte = quantise(new)
                block, s = pool[at], pos % page
                block[:, s * D // 2:(s + 1) * D // 2] = pack(codes)
                block[:, page * D // 2:].reshape(G, page, D // 16)[:, s] = byte
    assert page < stored < int(p.offsets[-1]) - 8
    d = c.run(lb)
    for name, got, want in zip("kv", (d.k, d.v), pools):
        bad = np.nonzero(got.cpu().numpy() != want)
        assert not len(bad[0]), f"{name}: {len(bad[0])} bytes differ, first {[int(b[0]) for b in bad]}"
    want = store(q, dtype)
    assert np.array_equal(to_host_bits(d.q_out).view(want.dtype), want)
    assert int(d.status[0]) == lb.LLAMA_ERR_RANGE


@pytest.mark.parametrize("dtype,H,G,D,page", SHAPES)
@pytest.mark.parametrize("q_lens,kv_lens,pad", [([300, 0, 17], [300, 9, 17], 5), ([4, 30], [100, 20], 0), ([1], [77], 2),
                                                ([900, 800], [900, 2000], 0)])
def test_read(lb, dtype, H, G, D, page, q_lens, kv_lens, pad):
    t = torch()
    p = Kv4Problem(f"r{dtype}{D}", dtype, H, G, D, page, q_lens, kv_lens, pad=pad)
    d = p.device(lb)
    out = [t.full((p.T, G, D), 7.0, dtype=d.q.dtype, device="cuda") for _ in "kv"]
    lb.check(lb.llama_op_kv4_read_paged(d.code, d.kv, d.batch, out[0], out[1], G, D, d.status, t.cuda.current_stream()))
    only = t.full((p.T, G, D), 7.0, dtype=d.q.dtype, device="cuda")
    lb.check(lb.llama_op_kv4_read_paged(d.code, d.kv, d.batch, None, only, G, D, d.status, t.cuda.current_stream()))
    t.cuda.synchronize()
    for got, pool in zip(out, (p.k, p.v)):
        want = np.full((p.T, G, D), 7.0)
        for i, (n, L) in enumerate(zip(q_lens, kv_lens)):
            rows = np.zeros((n, G, D))
            have = min(n, L)
            if have:
                rows[n - have:] = p.rows(i, pool).transpose(1, 0, 2)[L - have:]
            want[p.offsets[i]:p.offsets[i + 1]] = rows
        assert np.array_equal(to_f64(got), want)
    assert t.equal(only, out[1])
    assert int(d.status[0]) == 0


def test_read_bad_page(lb):
    t = torch()
    p = Kv4Problem("rb", "bf16", 2, 2, 64, 16, [40], [40])
    p.table[0, 1] = p.n_pages
    d = p.device(lb)
    out = [t.full((40, 2, 64), 7.0, dtype=t.bfloat16, device="cuda") for _ in "kv"]
    lb.check(lb.llama_op_kv4_read_paged(d.code, d.kv, d.batch, out[0], out[1], 2, 64, d.status, t.cuda.current_stream()))
    t.cuda.synchronize()
    assert float(out[0][16:32].abs().max()) == 0 and float(out[0][32:].abs().max()) > 0
    assert int(d.status[0]) == lb.LLAMA_ERR_RANGE


HEADS = [("bf16", 8, 2, 128), ("bf16", 9, 3, 64), ("bf16", 20, 1, 32), ("bf16", 4, 2, 16), ("bf16", 12, 1, 128),
         ("bf16", 8, 8, 64), ("bf16", 34, 2, 128), ("f32", 6, 2, 64), ("f32", 4, 2, 16), ("f32", 8, 1, 128)]


@pytest.mark.parametrize("dtype,H,G,D", HEADS)
@pytest.mark.parametrize("name,kv_lens,max_kv", [
    ("one", [1], None),
    ("short", [300, 17, 1, 0, 128, 31, 32, 33], None),
    ("direct", [2000, 900, 1, 129, 0, 2048], None),
    ("planned", [3000, 5, 700, 2222, 0, 64], 1 << 18),
    ("planned_many", [150 + 37 * (i % 40) for i in range(70)], 1 << 18),
    ("planned_one", [5001], None),
    ("planned_none", [0, 0, 0], 1 << 18),
])
def test_decode(lb, dtype, H, G, D, name, kv_lens, max_kv):
    page = {"one": 16, "short": 16, "direct": 256, "planned": 32, "planned_many": 64, "planned_one": 128}.get(name, 16)
    p = Kv4Problem(f"d/{name}{dtype}{D}{H}", dtype, H, G, D, page, [1] * len(kv_lens), kv_lens)
    d = run_decode(lb, p, max_kv=max_kv)
    torch().cuda.synchronize()
    p.check(to_f64(d.o), name)
    assert int(d.status[0]) == 0


@pytest.mark.parametrize("dtype,H,G,D", HEADS)
@pytest.mark.parametrize("name,q_lens,kv_lens,max_kv", [
    ("one", [1], [1], None),
    ("direct", [5, 40, 130], [5, 200, 130], None),
    ("planned", [5, 40, 0, 130], [5, 200, 9, 130], 1 << 18),
    ("few_rows_many_keys", [2, 3, 1], [9000, 3333, 1], None),
    ("drafts", [5] * 20, [130 + 61 * i for i in range(20)], None),
    ("see_nothing", [20, 9], [12, 0], None),
    ("prompt", [600], [600], None),
])
def test_packed(lb, dtype, H, G, D, name, q_lens, kv_lens, max_kv):
    page = {"one": 16, "direct": 32, "planned": 16, "few_rows_many_keys": 64, "drafts": 128, "prompt": 256}.get(name, 16)
    p = Kv4Problem(f"p/{name}{dtype}{D}{H}", dtype, H, G, D, page, q_lens, kv_lens, pad=3)
    d = run_packed(lb, p, max_kv=max_kv)
    torch().cuda.synchronize()
    p.check(to_f64(d.o), name)
    assert int(d.status[0]) == 0


@pytest.mark.parametrize("H,G,D,page", [(4, 1, 128, 32), (3, 1, 64, 16)])
def test_long_caches(lb, H, G, D, page):
    """One token and a few drafts behind more than 100000 keys, beside a short sequence, and a prompt of 3000 rows."""
    for q_lens, kv_lens in (([1, 1], [100003, 40]), ([3, 1], [100003, 40]), ([3001], [3100])):
        p = Kv4Problem(f"long{D}{len(q_lens)}{q_lens[0]}", "bf16", H, G, D, page, q_lens, kv_lens)
        runs = [run_packed] + ([run_decode] if max(q_lens) == 1 else [])
        for run in runs:
            d = run(lb, p)
            torch().cuda.synchronize()
            p.check(to_f64(d.o), str(q_lens))
            assert int(d.status[0]) == 0


@pytest.mark.parametrize("run", [run_packed, run_decode])
@pytest.mark.parametrize("dtype,H,G,D", HEADS[:4] + HEADS[7:9])
@pytest.mark.parametrize("max_kv", [None, 1 << 18])
def test_query_rows_that_are_not_finite(lb, run, dtype, H, G, D, max_kv):
    kv_lens = [700, 90, 1, 0, 1300]
    p = Kv4Problem(f"nf{dtype}{D}", dtype, H, G, D, 32, [1] * 5, kv_lens)
    ref, bound = p.attention()
    q = synth.as_f64(p.q)
    spoilt = np.zeros((p.T, H), bool)
    for row, (col, v) in enumerate([(3, np.nan), (0, np.inf), (D - 1, -np.inf), (2, np.nan), (1, np.inf)]):
        q[row, (row * 5 + 1) % H, col] = v
        spoilt[row, (row * 5 + 1) % H] = True
    p.q = store(q.astype(F32), dtype)
    d = run(lb, p, max_kv=max_kv)
    torch().cuda.synchronize()
    got = to_f64(d.o)
    sees = np.array(kv_lens)[:, None] > 0
    assert np.all(np.isnan(got[spoilt & sees]))
    assert np.all(got[3] == 0)
    rest = ~spoilt & sees
    assert np.all(np.abs(got - ref)[rest] <= bound[rest])


def test_large_scores_and_values(lb):
    """Keys and values near the top of the range: one key takes all the weight, or many do.  Scores are 10^6 apart here,
    so that weights fall below 2^-126, fp32's smallest normal number, and are 0: each may take 2^-126 max|v| off an
    output beside the bound of the others."""
    for D, H, G in ((128, 8, 2), (64, 4, 4)):
        for run in (run_packed, run_decode):
            p = Kv4Problem(f"big{D}", "bf16", H, G, D, 16, [1, 1], [600, 200], size=5000.0)
            ref, bound = p.attention()
            got = to_f64(run(lb, p).o)
            slack = max(p.kv_lens) * 2.0 ** -126 * np.abs(p.v[np.isfinite(p.v)]).max()
            assert np.all(np.abs(got - ref) <= bound + slack)


@pytest.mark.parametrize("run", [run_packed, run_decode])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_bad_lengths_and_pages(lb, run, dtype):
    p = Kv4Problem("bad", dtype, 4, 2, 64, 16, [1] * 4, [100, 40, 70, 33])
    p.table[1, 1] = -5
    d = p.device(lb)
    lens = p.kv_lens
    d.kv_lens.copy_(torch().tensor([100, 40, 1 << 30, -3], dtype=torch().int32))
    run(lb, p, d)
    torch().cuda.synchronize()
    assert int(d.status[0]) == lb.LLAMA_ERR_RANGE
    got = to_f64(d.o)
    assert np.all(got[2:] == 0) and np.all(np.isfinite(got))
    page = int(p.table[1, 0])
    for pool in (p.k, p.v):  # the bad page reads as zeros
        zero = np.zeros((1,) + pool.shape[1:], pool.dtype)
        pool_with = np.concatenate([pool, zero])
        setattr(p, "k" if pool is p.k else "v", pool_with)
    p.table[1, 1] = p.n_pages
    p.kv_lens = [100, 40, 0, 0]
    assert page >= 0 and lens is not p.kv_lens
    ref, bound = p.attention()
    assert np.all(np.abs(got - ref)[:2] <= bound[:2])


def test_pages_of_several_layers_and_shared_ones(lb):
    """Pages of k and v side by side, and a prefix that every sequence reads."""
    t = torch()
    for run in (run_packed, run_decode):
        for D in (128, 16):
            p = Kv4Problem(f"il{D}", "bf16", 4, 2, D, 16, [1] * 3, [200, 90, 60], shared_prefix=3)
            d = p.device(lb)
            both = t.stack([d.k, d.v, t.full_like(d.k, 255)], dim=1).contiguous()
            d.both = both
            d.kv = lb.make_paged_kv4_cache(both[:, 0], both[:, 1], d.table, 16)
            run(lb, p, d)
            t.cuda.synchronize()
            p.check(to_f64(d.o))


def test_graphs_replay_with_other_lengths_and_share_a_workspace(lb):
    t = torch()
    longs = [[3000, 700, 64], [2, 2999, 1500]]
    for run, need in ((run_packed, lambda d, p: lb.llama_op_attention_packed_kv4_workspace_bytes(d.code, d.batch, p.H, p.G, p.D)),
                      (run_decode, lambda d, p: lb.llama_op_attention_paged_decode_kv4_workspace_bytes(d.code, 3, 8192, p.H, p.G, p.D))):
        ps = [Kv4Problem(f"g{i}", "bf16", 8, 2, 128, 32, [1] * 3, [3000, 2999, 1500]) for i in range(2)]
        ds = [p.device(lb) for p in ps]
        for p, d in zip(ps, ds):
            d.batch = lb.make_packed_batch(d.offsets, d.kv_lens, p.T, 8192)
        ws = t.full((max(need(d, p) for p, d in zip(ps, ds)) + 16,), 0x5A, dtype=t.uint8, device="cuda")
        side = t.cuda.Stream()
        graphs = []
        for p, d in zip(ps, ds):
            side.wait_stream(t.cuda.current_stream())
            with t.cuda.stream(side):
                run(lb, p, d, side, ws, 8192)
            t.cuda.synchronize()
            g = t.cuda.CUDAGraph()
            with t.cuda.graph(g, stream=side):
                run(lb, p, d, side, ws, 8192)
            graphs.append(g)
        for lens in longs:
            for p, d in zip(ps, ds):
                d.kv_lens.copy_(t.tensor(lens, dtype=t.int32))
                d.o.fill_(7.0)
            ws.random_(0, 256)
            t.cuda.synchronize()
            for g in graphs:
                g.replay()
            t.cuda.synchronize()
            for p, d in zip(ps, ds):
                p.kv_lens = lens
                p.check(to_f64(d.o), str(lens))


def test_results_repeat_bit_for_bit(lb):
    t = torch()
    for run in (run_packed, run_decode):
        p = Kv4Problem("rep", "bf16", 8, 2, 128, 64, [1] * 40, [100 + 91 * i for i in range(40)])
        first = run(lb, p, max_kv=1 << 16).o
        for _ in range(3):
            assert t.equal(run(lb, p, max_kv=1 << 16).o, first)


@pytest.mark.parametrize("run", [run_packed, run_decode])
@pytest.mark.parametrize("D", [128, 64, 16])
def test_weights_are_rounded_to_fp16(lb, run, D):
    """Closer than weights of 8 bits allow: with rounding errors of at most 2^-11 of each weight (and what fp32 adds, as
    in _packed) instead of 2^-8, next to the rounding of the output.  Values of one sign and near one another, so that
    nothing hides behind large ones."""
    p = Kv4Problem(f"fp16{D}", "bf16", 4, 2, D, 32, [1] * 3, [900, 2500, 60])
    ref, bound = p.attention()
    got = to_f64(run(lb, p, max_kv=1 << 16).o)
    o = np.abs(ref)
    rel = (bound - 2.0 ** -8 * 1.01 * o) / 1.01  # of sum w |v|: the statistics' share and 2^-8
    weights = np.zeros_like(ref)
    r = p.H // p.G
    for i, L in enumerate(p.kv_lens):
        k, v = p.rows(i, p.k), p.rows(i, p.v)
        for h in range(p.H):
            s = synth.as_f64(p.q)[i, h] @ k[h // r].T / np.sqrt(D)
            w = np.exp(s - s.max())
            weights[i, h] = (w / w.sum()) @ np.abs(v[h // r])
    tight = rel - weights * (2.0 ** -8 - 2.0 ** -11 - 3000 * 2.0 ** -32)
    assert np.all(tight > 0) and np.all(np.abs(got - ref) <= tight * 1.01 + 2.0 ** -8 * 1.01 * o)


def test_far_pages(lb):
    """Pages whose bytes lie past 2^32 from the pool's start."""
    t = torch()
    p = Kv4Problem("far", "bf16", 4, 2, 128, 16, [1, 1], [100, 60])
    d = p.device(lb)
    block = d.k.shape[1] * d.k.shape[2]
    stride = (5 << 30) // p.n_pages // 16 * 16
    far = t.zeros(stride * (p.n_pages - 1) + block, dtype=t.uint8, device="cuda")
    k = far.as_strided((p.n_pages, d.k.shape[1], d.k.shape[2]), (stride, d.k.shape[2], 1))
    k.copy_(d.k)
    v = far[block:].as_strided((p.n_pages - 1,) + tuple(d.k.shape[1:]), (stride, d.k.shape[2], 1))
    v.copy_(d.v[:-1])
    used = int(p.table[p.table < p.n_pages].max())
    if used == p.n_pages - 1:  # the last page's values have no room behind it: swap it for a spare one
        spare = next(i for i in range(p.n_pages) if i not in set(p.table[p.table < p.n_pages].tolist()))
        for x in (p.k, p.v):
            x[[spare, used]] = x[[used, spare]]
        for x in (d.k, d.v):
            x[[spare, used]] = x[[used, spare]]
        p.table[p.table == used] = spare
        d.table.copy_(to_dev(p.table))
        k.copy_(d.k)
        v.copy_(d.v[:-1])
    d.kv = lb.llama_paged_kv_cache(k.data_ptr(), v.data_ptr(), d.table.data_ptr(), p.n_pages - 1, 16, p.table.shape[1],
                                   p.table.shape[1], stride)
    for run in (run_packed, run_decode):
        d.o.fill_(7.0)
        run(lb, p, d)
        t.cuda.synchronize()
        p.check(to_f64(d.o))
    out = [t.zeros((2, 2, 128), dtype=t.bfloat16, device="cuda") for _ in "kv"]
    lb.check(lb.llama_op_kv4_read_paged(d.code, d.kv, d.batch, out[0], out[1], 2, 128, d.status, t.cuda.current_stream()))
    t.cuda.synchronize()
    for got, pool in zip(out, (p.k, p.v)):
        want = np.stack([p.rows(i, pool)[:, -1] for i in range(2)])
        assert np.array_equal(to_f64(got), want)


def test_blocks_helper_agrees_with_values():
    x = synth.normal(1, "blocks", (2, 16, 32))
    codes, byte = unpack(blocks(x), 16, 32)
    c, b = quantise(x)
    assert np.array_equal(codes, c) and np.array_equal(byte, b) and np.isfinite(values(c, b)).all()
    assert hash_tag("x") > 0
