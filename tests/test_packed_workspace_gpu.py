"""What packed attention reserves for split items, and calls at the border of splitting (GPU)."""
import pytest

from _helpers import to_f64, torch
from _packed import Problem, run_packed

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lb():
    import decoder_block_gb300 as m
    m.load()
    return m


@pytest.mark.parametrize("H,G", [(152, 152), (160, 160), (154, 77), (310, 155), (304, 152)])
@pytest.mark.parametrize("q_lens,kv_lens", [([2, 1], [2500, 40]), ([130], [1300])])
def test_packed_attention_of_many_kv_heads(lb, H, G, q_lens, kv_lens):
    p = Problem(f"heads/{H}{G}{len(q_lens)}", "bf16", H, G, 64, 64, q_lens, kv_lens, pad=1)
    for max_kv in (None, 1 << 17):
        d = run_packed(lb, p, max_kv=max_kv)
        torch().cuda.synchronize()
        p.check(to_f64(d.o), f"bound {max_kv}")
        assert int(d.status[0]) == 0


def test_workspace_holds_parts_only_where_items_can_be_split(lb):
    def need(n_tokens, n_seqs, max_kv, H, G, D=128):
        b = lb.llama_packed_batch(q_offsets=None, kv_lens=None, n_seqs=n_seqs, n_tokens=n_tokens, max_kv_len=max_kv)
        return lb.llama_op_attention_packed_workspace_bytes(lb.LLAMA_BF16, b, H, G, D)

    sms = torch().cuda.get_device_properties(0).multi_processor_count
    part = 8 * 130 * 32 * 4  # of one piece and KV head, D = 128
    entries = 32 * (8192 // 64 + 4)
    assert need(8192, 4, 1024, 32, 8) < entries + 1024
    assert 2 * sms // 8 * 8 * part <= need(8192, 4, 1025, 32, 8) <= 2 * sms * part + 2 * entries + (32 << 10)
    assert need(4096, 2, 1 << 20, sms, sms) < 1 << 20
    assert need(4096, 2, 1 << 20, sms - 1, sms - 1) > 2 * (sms - 1) * part
