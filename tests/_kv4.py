"""Problems over a cache held in 4 bits: the blocks written out in numpy, and attention problems over such pages.

A block's values are exact bf16 numbers, so the plain results and error bounds of _packed.Problem hold as they are for
the values that the pages stand for."""
from __future__ import annotations

import numpy as np

import synth
from _helpers import to_dev, torch
from _packed import Device, Problem, hash_tag, store

F32 = np.float32
SCALES = np.array([2.0 ** (b // 8 - 20) * (1 + (b % 8) / 8) for b in range(256)])
_SHIFT = np.array([4 * (e // 2) + 16 * (e % 2) for e in range(8)])


def block_bytes(page, D):
    return page * (D // 2 + D // 16)


def quantise(x):
    """(codes [..., D], scale bytes [..., D / 16]) of fp32 [..., D], finite or not."""
    x = np.asarray(x, F32)
    b = x.reshape(*x.shape[:-1], -1, 16)
    a = np.where(np.isnan(b), F32(0), np.abs(b)).max(-1)
    byte = np.minimum(np.searchsorted(SCALES, (a / F32(7)).astype(np.float64)), 255)
    with np.errstate(invalid="ignore", over="ignore"):
        n = np.clip(np.rint(b / SCALES[byte].astype(F32)[..., None]), -7, 7)
    n = np.where(np.isnan(b), 0, n)
    return (n + 8).astype(np.int64).reshape(x.shape), byte.astype(np.uint8)


def values(codes, byte):
    """fp64 [..., D]."""
    n = (codes - 8).reshape(*codes.shape[:-1], -1, 16)
    return (n * SCALES[byte][..., None]).reshape(codes.shape)


def pack(codes):
    """Bytes [..., D / 2] of codes [..., D]."""
    w = (codes.reshape(*codes.shape[:-1], -1, 8).astype(np.uint64) << _SHIFT.astype(np.uint64)).sum(-1).astype("<u4")
    return w.view(np.uint8).reshape(*codes.shape[:-1], -1)


def blocks(x):
    """Pool bytes [..., page * (D / 2 + D / 16)] of fp32 rows [..., page, D]."""
    codes, byte = quantise(x)
    lead = x.shape[:-2]
    return np.concatenate([pack(codes).reshape(*lead, -1), byte.reshape(*lead, -1)], -1)


def unpack(pool, page, D):
    """(codes [..., page, D], scale bytes [..., page, D / 16]) of pool bytes."""
    at = page * D // 2
    w = np.ascontiguousarray(pool[..., :at]).view("<u4").reshape(*pool.shape[:-1], page, D // 8, 1)
    codes = ((w >> _SHIFT.astype(np.uint32)) & 15).astype(np.int64).reshape(*pool.shape[:-1], page, D)
    return codes, pool[..., at:].reshape(*pool.shape[:-1], page, D // 16)


class Kv4Problem(Problem):
    """A packed batch over 4-bit pages; rows that nothing may read hold the largest values there are."""

    def __init__(self, tag, dtype, H, G, D, page, q_lens, kv_lens, pad=0, spare=2, shared_prefix=0, size=1.0):
        super().__init__(tag, "f32", H, G, D, page, q_lens, kv_lens, pad=pad, spare=spare, shared_prefix=shared_prefix)
        self.dtype = dtype
        self.q = store(self.q, dtype)
        rng = np.random.default_rng(hash_tag(tag) + 1)
        self.pools = []
        for which in "kv":
            x = getattr(self, which) * F32(size)
            dead = np.isnan(x)
            codes, byte = quantise(np.where(dead, F32(0), x))
            codes[dead] = rng.choice([0, 15], size=int(dead.sum()))
            byte[dead.reshape(*byte.shape, 16)[..., 0]] = 255
            lead = x.shape[:-2]
            pool = np.concatenate([pack(codes).reshape(*lead, -1), byte.reshape(*lead, -1)], -1)
            self.pools.append(np.ascontiguousarray(pool[:, 0]))
            setattr(self, which, values(codes, byte).astype(F32))

    def device(self, lb):
        t = torch()
        d = Device()
        d.code = lb.LLAMA_BF16 if self.dtype == "bf16" else lb.LLAMA_F32
        d.k, d.v = (to_dev(x) for x in self.pools)
        d.table = to_dev(self.table)
        d.offsets, d.kv_lens = to_dev(self.offsets), to_dev(np.asarray(self.kv_lens, dtype=np.int32))
        d.q = to_dev(self.q)
        d.o = t.full((self.T, self.H, self.D), 7.0, dtype=d.q.dtype, device="cuda")
        d.status = t.zeros(4, dtype=t.int32, device="cuda")
        d.kv = lb.make_paged_kv4_cache(d.k, d.v, d.table, self.page)
        d.batch = lb.make_packed_batch(d.offsets, d.kv_lens, self.T, self.max_kv)
        return d


def run_packed(lb, p, d=None, stream=None, workspace=None, max_kv=None):
    t = torch()
    d = d or p.device(lb)
    if max_kv is not None:
        d.batch = lb.make_packed_batch(d.offsets, d.kv_lens, p.T, max_kv)
    need = lb.llama_op_attention_packed_kv4_workspace_bytes(d.code, d.batch, p.H, p.G, p.D)
    ws = workspace if workspace is not None else t.full((max(need, 16),), 0xA5, dtype=t.uint8, device="cuda")
    lb.check(lb.llama_op_attention_packed_kv4(d.code, d.q, d.kv, d.batch, d.o, p.H, p.G, p.D, ws, ws.numel(), d.status,
                                              stream or t.cuda.current_stream()), "llama_op_attention_packed_kv4")
    return d


def run_decode(lb, p, d=None, stream=None, workspace=None, max_kv=None):
    t = torch()
    d = d or p.device(lb)
    n, m = len(p.kv_lens), p.max_kv if max_kv is None else max_kv
    need = lb.llama_op_attention_paged_decode_kv4_workspace_bytes(d.code, n, m, p.H, p.G, p.D)
    ws = workspace if workspace is not None else t.full((max(need, 16),), 0xA5, dtype=t.uint8, device="cuda")
    lb.check(lb.llama_op_attention_paged_decode_kv4(d.code, d.q, d.kv, d.kv_lens, n, m, d.o, p.H, p.G, p.D, ws,
                                                    ws.numel(), d.status, stream or t.cuda.current_stream()),
             "llama_op_attention_paged_decode_kv4")
    return d
