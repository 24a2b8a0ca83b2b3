"""Problems over a paged cache, their plain 64-bit results and error bounds.

The plain results come from the oracle's equations written out per sequence and
head in fp64 (numpy); nothing here uses the library but the struct builders.

Error bounds (unit roundoff of a type: half its epsilon).  With A = sum_j w_j |v_j|
(w the exact softmax weights), an attention output that a kernel computes in
fp32 differs from the exact one by at most
    A (2 e_s + 2 (n + 64) 2^-24 + 2^-18)  (+ u_bf16 A where the weights are rounded to bf16)
and by u |o| from the rounding of the output:
  * e_s bounds a score's error: (D + 8) 2^-24 times the largest sum_d |q_d k_d| / sqrt(D), the standard bound of a
    D-term fp32 dot product and its scaling.  It changes a weight by e^(e_s), numerator and denominator: 2 e_s.
  * 2 (n + 64) 2^-24: two fp32 sums over n keys.
  * 2^-18: the exponentials (a few 2^-22 relative, on arguments whose own rounding is below 64 * 2^-24 = 2^-18 / 1).
"""
from __future__ import annotations

import math

import numpy as np

import synth
from _helpers import to_dev, torch

U32 = 2.0 ** -24
U_BF16 = 2.0 ** -8


def store(a32, dtype):
    return a32 if dtype == "f32" else synth.f32_to_bf16_bits(a32)


class Problem:
    """A packed batch over a page pool with random page order and rubbish wherever nothing may be read."""

    def __init__(self, tag, dtype, H, G, D, page, q_lens, kv_lens, pad=0, spare=2, interleave=False, rubbish=True,
                 shared_prefix=0):
        self.dtype, self.H, self.G, self.D, self.page = dtype, H, G, D, page
        self.q_lens, self.kv_lens, self.pad = list(q_lens), list(kv_lens), pad
        n = len(q_lens)
        self.offsets = np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int32)
        self.T = int(self.offsets[-1]) + pad
        rng = np.random.default_rng(abs(hash_tag(tag)) % (1 << 32))
        counts = [(L + page - 1) // page for L in kv_lens]
        keep = min([shared_prefix] + counts) if shared_prefix else 0  # pages that every sequence reads from the first
        total = sum(counts) + spare
        order = rng.permutation(total).astype(np.int32)
        width = max(max(counts), 1) + 1
        self.table = np.full((n, width), 0x7fffffff if rubbish else 0, dtype=np.int32)
        at = 0
        for i, c in enumerate(counts):
            self.table[i, :c] = order[at:at + c]
            at += c
            if i and keep:
                self.table[i, :keep] = self.table[0, :keep]
        self.n_pages = total
        planes = 2 if interleave else 1
        shape = (total, planes, G, page, D)
        pools = []
        for which in "kv":
            a = synth.normal(0, f"{tag}/{which}", shape)
            pools.append(a)
        self.q = store(synth.normal(0, f"{tag}/q", (self.T, H, D)), dtype)
        if rubbish:
            live = np.zeros((total, page), dtype=bool)
            for i, L in enumerate(kv_lens):
                for p in range(L):
                    live[self.table[i, p // page], p % page] = True
            for a in pools:
                a[~live[:, None, None, :].repeat(planes, 1).repeat(G, 2)] = np.nan
            if pad:
                self.q[self.offsets[-1]:] = store(np.full((pad, H, D), np.nan, np.float32), dtype)
        self.k, self.v = (store(a, dtype) for a in pools)
        self.max_kv = max(max(kv_lens), 0)

    def device(self, lb):
        t = torch()
        d = Device()
        d.code = lb.LLAMA_BF16 if self.dtype == "bf16" else lb.LLAMA_F32
        d.kall, d.vall = to_dev(self.k), to_dev(self.v)
        d.k, d.v = d.kall[:, 0], d.vall[:, 0]
        d.table = to_dev(self.table)
        d.offsets, d.kv_lens = to_dev(self.offsets), to_dev(np.asarray(self.kv_lens, dtype=np.int32))
        d.q = to_dev(self.q)
        d.o = t.full((self.T, self.H, self.D), 7.0, dtype=d.q.dtype, device="cuda")
        d.status = t.zeros(4, dtype=t.int32, device="cuda")
        d.kv = lb.make_paged_kv_cache(d.k, d.v, d.table)
        d.batch = lb.make_packed_batch(d.offsets, d.kv_lens, self.T, self.max_kv)
        return d

    def rows(self, i, pool):
        """[G][L][D] fp64 of sequence i."""
        L = self.kv_lens[i]
        x = synth.as_f64(pool[self.table[i, :(L + self.page - 1) // self.page], 0])
        return x.transpose(1, 0, 2, 3).reshape(self.G, -1, self.D)[:, :L]

    def attention(self):
        """(o, bound) fp64 [T][H][D]; NaN bound where a row must stay as it was."""
        o = np.zeros((self.T, self.H, self.D))
        bound = np.full(o.shape, np.nan)
        r = self.H // self.G
        u_out = U_BF16 if self.dtype == "bf16" else U32
        q = synth.as_f64(self.q)
        for i, (n, L) in enumerate(zip(self.q_lens, self.kv_lens)):
            if n == 0:
                continue
            k, v = self.rows(i, self.k), self.rows(i, self.v)
            rows = slice(self.offsets[i], self.offsets[i + 1])
            pos = np.arange(L - n, L)
            see = pos >= 0
            for h in range(self.H):
                g = h // r
                bound[rows, h] = 0.0
                if L == 0 or not see.any():
                    continue
                qh = q[rows, h][see]
                s = qh @ k[g].T / math.sqrt(self.D)
                s[np.arange(L)[None, :] > pos[see][:, None]] = -np.inf
                w = np.exp(s - s.max(-1, keepdims=True))
                w /= w.sum(-1, keepdims=True)
                e_s = (self.D + 8) * U32 * (np.abs(qh) @ np.abs(k[g]).T).max() / math.sqrt(self.D)
                rel = 2 * e_s + 2 * (L + 64) * U32 + 2.0 ** -18 + (U_BF16 if self.dtype == "bf16" else 0.0)
                at = np.arange(rows.start, rows.stop)[see]
                o[at, h] = w @ v[g]
                bound[at, h] = (w @ np.abs(v[g])) * rel * 1.01 + u_out * np.abs(o[at, h]) * 1.01
        return o, bound

    def check(self, got, what=""):
        ref, bound = self.attention()
        keep = np.isnan(bound)
        assert np.all(got[keep] == 7.0), f"{what}: rows outside the sequences were written"
        err = np.abs(got - ref)
        err[keep] = 0.0
        bad = ~(err <= np.where(keep, 0.0, bound))
        if bad.any():
            t, h, d = (int(a[0]) for a in np.nonzero(bad))
            raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} outside the bound; first at token {t} head "
                                 f"{h} column {d}: got {got[t, h, d]}, exact {ref[t, h, d]}, bound {bound[t, h, d]}")


class Device:
    pass


def hash_tag(tag: str) -> int:
    h = 2166136261
    for c in tag.encode():
        h = (h ^ c) * 16777619 % (1 << 32)
    return h


def run_packed(lb, p: Problem, d=None, stream=None, workspace=None, max_kv=None):
    t = torch()
    d = d or p.device(lb)
    if max_kv is not None:
        d.batch = lb.make_packed_batch(d.offsets, d.kv_lens, p.T, max_kv)
    need = lb.llama_op_attention_packed_workspace_bytes(d.code, d.batch, p.H, p.G, p.D)
    ws = workspace if workspace is not None else t.full((max(need, 16),), 0xA5, dtype=t.uint8, device="cuda")
    lb.check(lb.llama_op_attention_packed(d.code, d.q, d.kv, d.batch, d.o, p.H, p.G, p.D, ws, ws.numel(), d.status,
                                          stream or t.cuda.current_stream()), "llama_op_attention_packed")
    return d


def run_decode(lb, p: Problem, d=None, stream=None, workspace=None, max_kv=None):
    t = torch()
    d = d or p.device(lb)
    n, m = len(p.kv_lens), p.max_kv if max_kv is None else max_kv
    need = lb.llama_op_attention_paged_decode_workspace_bytes(d.code, n, m, p.H, p.G, p.D)
    ws = workspace if workspace is not None else t.full((max(need, 16),), 0xA5, dtype=t.uint8, device="cuda")
    lb.check(lb.llama_op_attention_paged_decode(d.code, d.q, d.kv, d.kv_lens, n, m, d.o, p.H, p.G, p.D, ws, ws.numel(),
                                                d.status, stream or t.cuda.current_stream()),
             "llama_op_attention_paged_decode")
    return d
