"""Host-side checks of the packed / paged operators beside those of test_packed_cpu.py."""
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


def test_wait_budget_setter(lb):
    assert lb.llama_op_set_wait_budget(-1) == lb.LLAMA_ERR_INVALID_ARG
    assert lb.llama_op_set_wait_budget(1000) == lb.LLAMA_OK
    assert lb.llama_op_set_wait_budget(0) == lb.LLAMA_OK


def _batch(lb, n_seqs, n_tokens, max_kv):
    return lb.llama_packed_batch(q_offsets=None, kv_lens=None, n_seqs=n_seqs, n_tokens=n_tokens, max_kv_len=max_kv)


@pytest.mark.parametrize("G,n_tokens,n_seqs,max_kv", [
    (8, 8192, 4, 1024),      # no sequence is long enough for an item to be split
    (8, 100000, 300, 1000),
    (512, 4096, 2, 8192),    # more KV heads than there are SMs: nor does any item outlast the rest
    (2048, 300, 1, 1 << 20),
])
def test_packed_workspace_holds_no_parts_that_cannot_be(lb, G, n_tokens, n_seqs, max_kv):
    for r, D in ((1, 128), (4, 64)):
        blocks = n_tokens // (2 * (128 // r)) + n_seqs
        n = lb.llama_op_attention_packed_workspace_bytes(lb.LLAMA_BF16, _batch(lb, n_seqs, n_tokens, max_kv), G * r, G, D)
        assert 32 * blocks < n < 32 * blocks + (64 << 10), (r, D)


def test_elements_have_to_be_aligned(lb):
    host = (ctypes.c_char * 4096)()
    at = (ctypes.addressof(host) + 15) & ~15
    for dtype, off, expected in ((lb.LLAMA_F32, 2, lb.LLAMA_ERR_ALIGN), (lb.LLAMA_BF16, 1, lb.LLAMA_ERR_ALIGN),
                                 (lb.LLAMA_F32, 4, lb.LLAMA_ERR_INVALID_ARG),   # host memory, met next
                                 (lb.LLAMA_BF16, 2, lb.LLAMA_ERR_INVALID_ARG)):
        assert lb.llama_op_token_logprobs(dtype, at + off, 10, at, 2, 10, at) == expected


def test_fp32_parts_follow_the_sms_of_the_device(lb):
    torch = pytest.importorskip("torch")
    sms = torch.cuda.get_device_properties(0).multi_processor_count if torch.cuda.is_available() else 1
    kv, H, G, D = 1 << 20, 8, 4, 64
    for n_seqs in (1, 3, 40, 1000):
        want = -(-16 * sms // (n_seqs * G))  # parts that make 16 CTAs per SM
        chunk = -(-(-(-kv // want)) // 64) * 64
        parts = -(-kv // chunk)
        assert lb.llama_op_attention_paged_decode_workspace_bytes(lb.LLAMA_F32, n_seqs, kv, H, G, D) == (
            n_seqs * H * parts * (D + 2) * 4 if parts > 1 else 0)
