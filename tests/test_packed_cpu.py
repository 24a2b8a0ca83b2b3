"""Refusals of the packed / paged operators and of the token log-probabilities:
arguments are checked on the host before anything touches a GPU."""
import ctypes
import os

import pytest


@pytest.fixture(scope="module")
def lb():
    import decoder_block_gb300 as m
    if not os.path.exists(m.LIB_PATH):
        from decoder_block_gb300 import build
        build.build()
    m.load()
    return m


HOST = (ctypes.c_char * 4096)()
ADDR = (ctypes.addressof(HOST) + 15) & ~15


def _kv(lb, **f):
    base = dict(k=ADDR, v=ADDR, page_table=ADDR, n_pages=8, page_size=16, max_pages=4, table_stride=4, page_stride=0)
    base.update(f)
    return lb.llama_paged_kv_cache(**base)


def _batch(lb, **f):
    base = dict(q_offsets=ADDR, kv_lens=ADDR, n_seqs=2, n_tokens=10, max_kv_len=64)
    base.update(f)
    return lb.llama_packed_batch(**base)


def _all(lb, kv, batch, H=4, G=2, D=64, dtype=None):
    """The three packed / paged calls with the same cache, batch and heads."""
    dtype = lb.LLAMA_BF16 if dtype is None else dtype
    return [
        lb.llama_op_rope_kv_write_paged(dtype, ADDR, ADDR, kv, batch, ADDR, 64, H, G, D),
        lb.llama_op_attention_packed(dtype, ADDR, kv, batch, ADDR, H, G, D),
        lb.llama_op_attention_paged_decode(dtype, ADDR, kv, ADDR, batch.n_seqs, batch.max_kv_len, ADDR, H, G, D),
    ]


@pytest.mark.parametrize("kv,expected", [
    (dict(n_pages=0), "LLAMA_ERR_INVALID_ARG"), (dict(page_size=0), "LLAMA_ERR_INVALID_ARG"),
    (dict(max_pages=0), "LLAMA_ERR_INVALID_ARG"), (dict(table_stride=3), "LLAMA_ERR_INVALID_ARG"),
    (dict(page_size=8), "LLAMA_ERR_UNSUPPORTED"), (dict(page_size=48), "LLAMA_ERR_UNSUPPORTED"),
    (dict(page_size=512), "LLAMA_ERR_UNSUPPORTED"), (dict(page_stride=-1), "LLAMA_ERR_INVALID_ARG"),
    (dict(page_stride=2 * 16 * 64 - 8), "LLAMA_ERR_INVALID_ARG"), (dict(page_stride=2 * 16 * 64 + 4), "LLAMA_ERR_ALIGN"),
    (dict(page_stride=1 << 45), "LLAMA_ERR_UNSUPPORTED"),
    (dict(), "LLAMA_ERR_INVALID_ARG"),  # host memory
])
def test_cache_refusals(lb, kv, expected):
    assert _all(lb, _kv(lb, **kv), _batch(lb)) == [getattr(lb, expected)] * 3


@pytest.mark.parametrize("batch,expected", [
    (dict(n_seqs=-1), "LLAMA_ERR_INVALID_ARG"), (dict(max_kv_len=-1), "LLAMA_ERR_INVALID_ARG"),
    (dict(n_seqs=4097), "LLAMA_ERR_UNSUPPORTED"), (dict(n_seqs=0), "LLAMA_OK"),
    (dict(max_kv_len=8388481), "LLAMA_ERR_UNSUPPORTED"), (dict(max_kv_len=8388480), "LLAMA_ERR_INVALID_ARG"),
])
def test_batch_refusals(lb, batch, expected):
    assert _all(lb, _kv(lb), _batch(lb, **batch)) == [getattr(lb, expected)] * 3


@pytest.mark.parametrize("heads,expected", [
    (dict(H=0), "LLAMA_ERR_INVALID_ARG"), (dict(G=0), "LLAMA_ERR_INVALID_ARG"), (dict(D=0), "LLAMA_ERR_INVALID_ARG"),
    (dict(H=5), "LLAMA_ERR_SHAPE"), (dict(D=96), "LLAMA_ERR_UNSUPPORTED"), (dict(D=256), "LLAMA_ERR_UNSUPPORTED"),
    (dict(dtype=2), "LLAMA_ERR_INVALID_ARG"), (dict(H=65536, G=1, D=16), "LLAMA_ERR_UNSUPPORTED"),
    (dict(H=65535, G=1, D=16), "LLAMA_ERR_INVALID_ARG"),  # host memory
])
def test_head_refusals(lb, heads, expected):
    assert _all(lb, _kv(lb), _batch(lb), **heads) == [getattr(lb, expected)] * 3


def test_more_rows_than_the_kernels_count(lb):
    kv, bf = _kv(lb), lb.LLAMA_BF16
    for n, expected in ((lb.LLAMA_PACKED_MAX_ROWS // 4, lb.LLAMA_ERR_INVALID_ARG),  # host memory
                        (lb.LLAMA_PACKED_MAX_ROWS // 4 + 1, lb.LLAMA_ERR_UNSUPPORTED)):
        b = _batch(lb, n_tokens=n)
        assert lb.llama_op_attention_packed(bf, ADDR, kv, b, ADDR, 4, 2, 64) == expected
        assert lb.llama_op_rope_kv_write_paged(bf, ADDR, ADDR, kv, b, ADDR, 64, 4, 2, 64) == expected
        assert (lb.llama_op_attention_packed_workspace_bytes(bf, b, 4, 2, 64) > 0) == (
            expected == lb.LLAMA_ERR_INVALID_ARG)


def test_struct_builders_refuse_what_the_structs_cannot_say(lb):
    torch = pytest.importorskip("torch")
    pool = torch.zeros(4, 2, 2, 16, 32)
    table, lens = torch.zeros(3, 5, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    kv = lb.make_paged_kv_cache(pool[:, 0], pool[:, 1], table[:, :4])
    assert (kv.n_pages, kv.page_size, kv.max_pages, kv.table_stride, kv.page_stride) == (4, 16, 4, 5, 2 * 2 * 16 * 32)
    for k, v, t in [(pool[:, 0], pool[:, 1].contiguous(), table), (pool[:, 0], pool[:, 1], table.long()),
                    (pool[:, 0].transpose(1, 2), pool[:, 1].transpose(1, 2), table),
                    (pool[:, 0], pool[:, 1].bfloat16(), table), (pool[:, 0], pool[:2, 1], table),
                    (pool[:, 0], pool[:, 1], table[:, ::2])]:
        with pytest.raises(ValueError):
            lb.make_paged_kv_cache(k, v, t)
    offsets = torch.zeros(4, dtype=torch.int32)
    assert lb.make_packed_batch(offsets, lens, 9, 7).n_seqs == 3
    for o, n in [(offsets.long(), lens), (offsets, lens.long()), (offsets[:3], lens), (offsets.float(), lens)]:
        with pytest.raises(ValueError):
            lb.make_packed_batch(o, n, 9, 7)


def test_no_tokens_is_no_work(lb):
    kv, b = _kv(lb, k=None, v=None, page_table=None), _batch(lb, n_tokens=0, q_offsets=None, kv_lens=None)
    assert lb.llama_op_rope_kv_write_paged(lb.LLAMA_BF16, None, None, kv, b, None, 64, 4, 2, 64) == lb.LLAMA_OK
    assert lb.llama_op_attention_packed(lb.LLAMA_BF16, None, kv, b, None, 4, 2, 64) == lb.LLAMA_OK
    assert lb.llama_op_attention_paged_decode(lb.LLAMA_F32, None, kv, None, 0, 64, None, 4, 2, 64) == lb.LLAMA_OK
    assert lb.llama_op_token_logprobs(lb.LLAMA_F32, None, 10, None, 0, 10, None) == lb.LLAMA_OK


def test_alignment_and_null_pointers(lb):
    b = _batch(lb)
    assert _all(lb, _kv(lb, k=ADDR + 8), b) == [lb.LLAMA_ERR_INVALID_ARG] * 3  # q is host memory: met first
    bf = lb.LLAMA_BF16
    assert lb.llama_op_attention_packed(bf, ADDR + 4, _kv(lb), b, ADDR, 4, 2, 64) == lb.LLAMA_ERR_ALIGN
    assert lb.llama_op_attention_packed(bf, None, _kv(lb), b, ADDR, 4, 2, 64) == lb.LLAMA_ERR_INVALID_ARG
    assert lb.llama_op_attention_paged_decode(bf, ADDR + 2, _kv(lb), ADDR, 2, 64, ADDR, 4, 2, 64) == lb.LLAMA_ERR_ALIGN
    assert lb.llama_op_rope_kv_write_paged(bf, ADDR + 4, ADDR, _kv(lb), b, ADDR, 64, 4, 2, 64) == lb.LLAMA_ERR_ALIGN
    assert lb.llama_op_rope_kv_write_paged(bf, ADDR, ADDR, _kv(lb), b, ADDR, 0, 4, 2, 64) == lb.LLAMA_ERR_INVALID_ARG
    assert lb.llama_op_rope_kv_write_paged(bf, ADDR, ADDR, _kv(lb), b, ADDR, 64, 4, 2, 64, 2) \
        == lb.LLAMA_ERR_INVALID_ARG


def test_workspace_sizes(lb):
    assert lb.llama_op_attention_paged_decode_workspace_bytes(lb.LLAMA_BF16, 4, 8192, 5, 2, 64) == 0  # refused heads
    assert lb.llama_op_attention_paged_decode_workspace_bytes(lb.LLAMA_BF16, 0, 8192, 4, 2, 64) == 0
    assert lb.llama_op_attention_paged_decode_workspace_bytes(lb.LLAMA_BF16, 4, -1, 4, 2, 64) == 0
    assert lb.llama_op_attention_paged_decode_workspace_bytes(lb.LLAMA_BF16, 4097, 64, 4, 2, 64) == 0
    assert lb.llama_op_attention_packed_workspace_bytes(lb.LLAMA_BF16, _batch(lb, n_seqs=-1), 4, 2, 64) == 0
    assert lb.llama_op_attention_packed_workspace_bytes(lb.LLAMA_BF16, _batch(lb), 4, 3, 64) == 0
    for dtype in (lb.LLAMA_F32, lb.LLAMA_BF16):
        for D in (16, 32, 64, 128):
            # a few megabytes hold the parts of one long sequence, and sizes do not depend on the call's data
            n = lb.llama_op_attention_paged_decode_workspace_bytes(dtype, 1, 1 << 20, 32, 8, D)
            assert 0 < n < 64 << 20


@pytest.mark.parametrize("args,expected", [
    (dict(V=0), "LLAMA_ERR_INVALID_ARG"), (dict(T=-1), "LLAMA_ERR_INVALID_ARG"), (dict(stride=9), "LLAMA_ERR_INVALID_ARG"),
    (dict(k=-1), "LLAMA_ERR_INVALID_ARG"), (dict(k=11), "LLAMA_ERR_RANGE"), (dict(V=100, stride=100, k=33), "LLAMA_ERR_UNSUPPORTED"),
    (dict(dtype=2), "LLAMA_ERR_INVALID_ARG"), (dict(targets=None), "LLAMA_ERR_INVALID_ARG"),
    (dict(logprobs=None), "LLAMA_ERR_INVALID_ARG"), (dict(logits=ADDR + 2), "LLAMA_ERR_ALIGN"),
    (dict(logits=None), "LLAMA_ERR_INVALID_ARG"), (dict(), "LLAMA_ERR_INVALID_ARG"),  # host memory
])
def test_logprobs_refusals(lb, args, expected):
    a = dict(dtype=lb.LLAMA_F32, logits=ADDR, stride=10, targets=ADDR, T=2, V=10, logprobs=ADDR, k=0)
    a.update(args)
    assert lb.llama_op_token_logprobs(a["dtype"], a["logits"], a["stride"], a["targets"], a["T"], a["V"], a["logprobs"],
                                      None, a["k"], ADDR, ADDR) == getattr(lb, expected)


def test_stack_score_refuses_a_null_handle(lb):
    assert lb.llama_stack_score(None, ADDR, 1, 1, 0, [], ADDR, ADDR, ADDR) == lb.LLAMA_ERR_INVALID_ARG
