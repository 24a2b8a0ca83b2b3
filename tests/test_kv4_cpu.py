"""The 4-bit cache without a GPU: what a block stands for, sizes and refusals on the host."""
import ctypes
import os

import numpy as np
import pytest

import _kv4


@pytest.fixture(scope="module")
def lb():
    import decoder_block_gb300 as m
    if not os.path.exists(m.LIB_PATH):
        from decoder_block_gb300 import build
        build.build()
    m.load()
    return m


def test_blocks_round_to_half_a_scale():
    rng = np.random.default_rng(3)
    x = (rng.standard_normal((400, 64)) * np.exp(rng.uniform(-9, 9, (400, 1)))).astype(np.float32)
    x[5] = 0
    x[6, 3] = 26880
    codes, byte = _kv4.quantise(x)
    assert codes.min() >= 1 and codes.max() <= 15
    s = np.repeat(_kv4.SCALES[byte], 16, -1)
    # x / s is rounded to fp32 (2^-24 of at most 7) before it is rounded to a code
    assert np.all(np.abs(_kv4.values(codes, byte) - x) <= s * (0.5 + 7 * 2.0 ** -24))
    a = np.abs(x.astype(np.float64)).reshape(400, 4, 16).max(-1)
    assert np.all(7 * _kv4.SCALES[byte] >= a * (1 - 2.0 ** -23))
    smaller = 7 * _kv4.SCALES[np.maximum(byte.astype(int) - 1, 0)]
    assert np.all((smaller < a) | (byte == 0))
    assert np.all(_kv4.values(codes, byte)[5] == 0)


def test_what_four_bits_lose_of_normal_values():
    """The RMS error of the format relative to the values' own, and of fp4 (0, 0.5, 1, 1.5, 2, 3, 4, 6) in the same blocks
    with exact scales and with this format's.  The ratio's square is a mean over 65536 blocks, whose own squared errors
    are spread by half of their mean or less: 0.5 / 256 = 0.2 %, 0.1 % of the root; four times that is allowed."""
    x = np.random.default_rng(9).standard_normal((8192, 128)).astype(np.float32)
    b = x.reshape(-1, 16).astype(np.float64)
    most = np.abs(b).max(-1, keepdims=True)
    fp4 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])

    def loss(y):
        return np.sqrt(((y.reshape(b.shape) - b) ** 2).sum() / (b ** 2).sum())

    def held(s):
        return np.sign(b) * s * fp4[np.abs(np.abs(b / s)[..., None] - fp4).argmin(-1)]

    coarse = _kv4.SCALES[np.searchsorted(_kv4.SCALES, most / 6)]
    for got, want in ((loss(_kv4.values(*_kv4.quantise(x))), 0.0929), (loss(held(most / 6)), 0.0942),
                      (loss(held(coarse)), 0.1004)):
        assert abs(got / want - 1) < 0.004, (got, want)


def test_pack_and_unpack_are_inverse():
    rng = np.random.default_rng(4)
    for page, D in ((16, 16), (32, 128), (256, 64)):
        codes = rng.integers(0, 16, (3, page, D))
        byte = rng.integers(0, 256, (3, page, D // 16)).astype(np.uint8)
        pool = np.concatenate([_kv4.pack(codes).reshape(3, -1), byte.reshape(3, -1)], -1)
        assert pool.shape[1] == _kv4.block_bytes(page, D)
        c, b = _kv4.unpack(pool, page, D)
        assert np.array_equal(c, codes) and np.array_equal(b, byte)


def test_every_value_is_a_bf16():
    v = (np.arange(16)[:, None] - 8) * _kv4.SCALES[None]
    assert np.all((v.astype(np.float32).view(np.uint32) & 0xffff) == 0) and np.array_equal(v.astype(np.float32), v)


def test_block_bytes(lb):
    for page in (16, 32, 64, 128, 256):
        for D in (16, 32, 64, 128):
            assert lb.llama_kv4_block_bytes(page, D) == _kv4.block_bytes(page, D)
            assert lb.llama_kv4_block_bytes(page, D) % 16 == 0
    for page, D in ((8, 64), (512, 64), (64, 96), (64, 8), (0, 64), (64, 0), (-16, 64), (64, 256)):
        assert lb.llama_kv4_block_bytes(page, D) == 0


def _cache(lb, at=None, n_pages=4, page=16, max_pages=2, table_stride=2, page_stride=0):
    return lb.llama_paged_kv_cache(at, at, at, n_pages, page, max_pages, table_stride, page_stride)


def _batch(lb, at=None, n_seqs=1, n_tokens=2, max_kv=16):
    return lb.llama_packed_batch(at, at, n_seqs, n_tokens, max_kv)


def _calls(lb, dtype, kv, batch, at, H, G, D, table_max=16, layout=0):
    return [lb.llama_op_rope_kv4_write_paged(dtype, at, at, kv, batch, at, table_max, H, G, D, layout),
            lb.llama_op_kv4_read_paged(dtype, kv, batch, at, at, G, D),
            lb.llama_op_attention_packed_kv4(dtype, at, kv, batch, at, H, G, D, at, 1 << 40),
            lb.llama_op_attention_paged_decode_kv4(dtype, at, kv, at, batch.n_seqs, batch.max_kv_len, at, H, G, D, at, 1 << 40)]


@pytest.fixture(scope="module")
def host():
    buf = (ctypes.c_char * 8192)()
    host.keep = buf
    return (ctypes.addressof(buf) + 255) & ~255


def test_refusals(lb, host):
    bf = lb.LLAMA_BF16
    ok_kv, ok_b = _cache(lb, host), _batch(lb, host)
    inv, shape, align, uns = lb.LLAMA_ERR_INVALID_ARG, lb.LLAMA_ERR_SHAPE, lb.LLAMA_ERR_ALIGN, lb.LLAMA_ERR_UNSUPPORTED
    # host memory is no device memory: the last check of a call that is otherwise right
    assert _calls(lb, bf, ok_kv, ok_b, host, 4, 2, 64) == [inv] * 4
    assert _calls(lb, 7, ok_kv, ok_b, host, 4, 2, 64) == [inv] * 4
    assert _calls(lb, bf, ok_kv, ok_b, host, 5, 2, 64)[0] == shape
    assert _calls(lb, bf, ok_kv, ok_b, host, 5, 2, 64)[2:] == [shape] * 2
    assert _calls(lb, bf, ok_kv, ok_b, host, 4, 2, 96) == [uns] * 4
    assert _calls(lb, bf, ok_kv, ok_b, host, 0, 0, 64) == [inv] * 4
    assert _calls(lb, bf, _cache(lb, host, page=48), ok_b, host, 4, 2, 64) == [uns] * 4
    assert _calls(lb, bf, _cache(lb, host, n_pages=0), ok_b, host, 4, 2, 64) == [inv] * 4
    assert _calls(lb, bf, _cache(lb, host, max_pages=3), ok_b, host, 4, 2, 64) == [inv] * 4  # table_stride < max_pages
    dense = 2 * _kv4.block_bytes(16, 64)
    assert _calls(lb, bf, _cache(lb, host, page_stride=dense - 16), ok_b, host, 4, 2, 64) == [inv] * 4
    assert _calls(lb, bf, _cache(lb, host, page_stride=dense + 8), ok_b, host, 4, 2, 64) == [align] * 4
    assert _calls(lb, bf, _cache(lb, host, page_stride=1 << 39), ok_b, host, 4, 2, 64) == [uns] * 4
    assert _calls(lb, bf, _cache(lb, host, page_stride=1 << 32), ok_b, host, 4, 2, 64) == [uns] * 4
    assert _calls(lb, bf, ok_kv, _batch(lb, host, n_seqs=-1), host, 4, 2, 64) == [inv] * 4
    assert _calls(lb, bf, ok_kv, _batch(lb, host, n_seqs=4097), host, 4, 2, 64) == [uns] * 4
    assert _calls(lb, bf, ok_kv, _batch(lb, host, max_kv=lb.LLAMA_PACKED_MAX_KV + 1), host, 4, 2, 64) == [uns] * 4
    assert _calls(lb, bf, ok_kv, ok_b, host + 8, 4, 2, 64) == [align] * 4
    assert _calls(lb, bf, ok_kv, ok_b, host, 4, 2, 64, layout=2)[0] == inv
    assert _calls(lb, bf, ok_kv, ok_b, host, 4, 2, 64, table_max=0)[0] == inv
    # more tiles than a kernel counts
    for n, heads in ((1 << 23, 65535), (1 << 24, 1)):
        many = (bf, host, ok_kv, host, 4096, n, host, heads, heads, 64, host, 1 << 40)
        assert lb.llama_op_attention_paged_decode_kv4(*many) == uns
        assert lb.llama_op_attention_paged_decode_kv4_workspace_bytes(bf, 4096, n, heads, heads, 64) == 0
    # nothing to do: nothing is looked at
    assert _calls(lb, bf, _cache(lb), _batch(lb, n_seqs=0), None, 4, 2, 64) == [lb.LLAMA_OK] * 4
    assert _calls(lb, bf, _cache(lb), _batch(lb, n_tokens=0), None, 4, 2, 64)[:3] == [lb.LLAMA_OK] * 3
    assert lb.llama_op_kv4_read_paged(bf, ok_kv, ok_b, None, None, 2, 64) == lb.LLAMA_OK


def test_workspaces(lb):
    for dtype in (lb.LLAMA_BF16, lb.LLAMA_F32):
        for args in ((0, 100, 4, 2, 64), (-1, 100, 4, 2, 64), (1, -1, 4, 2, 64), (1, 100, 4, 3, 64), (1, 100, 4, 2, 48),
                     (4097, 100, 4, 2, 64)):
            assert lb.llama_op_attention_paged_decode_kv4_workspace_bytes(dtype, *args) == 0
        assert lb.llama_op_attention_paged_decode_kv4_workspace_bytes(dtype, 1, 1 << 20, 32, 8, 128) > 0
        assert lb.llama_op_attention_packed_kv4_workspace_bytes(dtype, _batch(lb, n_tokens=0), 4, 2, 64) == 0
    assert lb.llama_op_attention_paged_decode_kv4_workspace_bytes(7, 1, 1 << 20, 4, 2, 64) == 0


def test_builders(lb):
    torch = pytest.importorskip("torch")
    k = torch.zeros((3, 2, _kv4.block_bytes(16, 64)), dtype=torch.uint8)
    table = torch.zeros((1, 2), dtype=torch.int32)
    kv = lb.make_paged_kv4_cache(k, k, table, 16)
    assert (kv.n_pages, kv.page_size, kv.max_pages, kv.page_stride) == (3, 16, 2, k[0].numel())
    both = torch.zeros((3, 2, 2, _kv4.block_bytes(16, 64)), dtype=torch.uint8)  # pages of k and v interleaved
    assert lb.make_paged_kv4_cache(both[:, 0], both[:, 1], table, 16).page_stride == both[0].numel()
    for bad in (lambda: lb.make_paged_kv4_cache(k, k, table, 48), lambda: lb.make_paged_kv4_cache(k, k[:2], table, 16),
                lambda: lb.make_paged_kv4_cache(k[..., ::2], k[..., ::2], table, 16),
                lambda: lb.make_paged_kv4_cache(k.float(), k.float(), table, 16),
                lambda: lb.make_paged_kv4_cache(k, k, table.long(), 16),
                lambda: lb.make_paged_kv4_cache(k[:, :, :-16], k[:, :, :-16], table, 16)):
        with pytest.raises(ValueError):
            bad()


def _drafts(lb, at, n_seqs=2, n_rows=4, max_drafts=3, uniforms=True, noise=True, noise_stride=1000, temps=None):
    return lb.llama_draft_batch(at, at, temps, at if uniforms else None, at if noise else None, noise_stride, n_seqs,
                                n_rows, max_drafts)


def test_verify_refusals(lb, host):
    inv, align, uns = lb.LLAMA_ERR_INVALID_ARG, lb.LLAMA_ERR_ALIGN, lb.LLAMA_ERR_UNSUPPORTED

    def call(b, dtype=lb.LLAMA_F32, target=host, ts=1000, draft=host, ss=3000, step=1000, V=1000, out=host, ws=host,
             ws_bytes=1 << 30):
        return lb.llama_op_verify_drafts(dtype, target, ts, draft, ss, step, V, b, out, out, None, ws, ws_bytes)

    assert call(_drafts(lb, host)) == inv                         # host memory, met last
    assert call(_drafts(lb, host), dtype=2) == inv
    assert call(_drafts(lb, host), V=0) == inv
    assert call(_drafts(lb, host), ts=999) == inv
    assert call(_drafts(lb, host), ss=-1) == inv and call(_drafts(lb, host), step=-1) == inv
    assert call(_drafts(lb, host, noise_stride=999)) == inv
    assert call(_drafts(lb, host, uniforms=False)) == inv and call(_drafts(lb, host, noise=False)) == inv
    assert call(_drafts(lb, host, n_seqs=-1)) == inv and call(_drafts(lb, host, max_drafts=-1)) == inv
    assert call(_drafts(lb, host, n_seqs=4097)) == uns
    assert call(_drafts(lb, host, max_drafts=lb.LLAMA_MAX_DRAFTS + 1)) == uns
    assert call(_drafts(lb, host, n_rows=4096 * 65 + 1)) == uns
    assert call(_drafts(lb, host), target=host + 2) == align
    assert call(_drafts(lb, host), dtype=lb.LLAMA_BF16, target=host + 1) == align
    assert call(_drafts(lb, host, n_seqs=0)) == lb.LLAMA_OK
    assert lb.llama_op_verify_drafts_workspace_bytes(_drafts(lb, host, n_rows=0), 1000) == 0
    assert lb.llama_op_verify_drafts_workspace_bytes(_drafts(lb, host), 0) == 0
    assert lb.llama_op_verify_drafts_workspace_bytes(_drafts(lb, host), 1000) == 4 * 2 * 16
    assert lb.llama_op_verify_drafts_workspace_bytes(_drafts(lb, host, n_rows=1), 1 << 30) <= 2 * 32 * 16


def test_draft_builder(lb):
    torch = pytest.importorskip("torch")
    off, tok = torch.zeros(3, dtype=torch.int32), torch.zeros(5, dtype=torch.int32)
    uni, noise = torch.zeros((2, 3)), torch.zeros((2, 64))
    b = lb.make_draft_batch(off, tok, 5, 3, None, uni, noise[:, :60])
    assert (b.n_seqs, b.n_rows, b.max_drafts, b.noise_stride) == (2, 5, 3, 64) and b.temperatures is None
    for bad in (lambda: lb.make_draft_batch(off.long(), tok, 5, 3), lambda: lb.make_draft_batch(off, tok, 6, 3),
                lambda: lb.make_draft_batch(off, tok, 5, 3, None, uni[:, :2], noise),
                lambda: lb.make_draft_batch(off, tok, 5, 3, None, uni, noise.double()),
                lambda: lb.make_draft_batch(off, tok, 5, 3, torch.zeros(3), uni, noise)):
        with pytest.raises(ValueError):
            bad()
