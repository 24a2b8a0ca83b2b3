"""Host-side checks of the packed / paged operators beside those of test_packed_cpu.py."""
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
