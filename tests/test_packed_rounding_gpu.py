"""Packed attention rounds a softmax weight to bf16 once, also where the running maximum rises inside a key tile (GPU).

95 keys share one weight w, a later key of the same tile scores a little more than 2^8 times theirs and first of all
raises the maximum; it and the first key have values of 0.  So o = c W with W = 95 w / l.  Rounding w once moves that by
u = 2^-8 of itself at most, fp32 sums and exponentials by the slack below, and the store rounds to the nearest bf16:
o lies between the bf16 neighbours of c W (1 - u - slack) and c W (1 + u + slack).  Weights rounded, scaled by the raise
and rounded again move it by up to 2 u, which the columns' different c show."""
import numpy as np
import pytest

import synth
from _helpers import to_f64, torch
from _packed import U32, U_BF16, Problem, run_packed

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lb():
    import decoder_block_gb300 as m
    m.load()
    return m


def _bf16(x):
    return synth.as_f64(synth.f32_to_bf16_bits(np.asarray(x, dtype=np.float32)))


def _three(x):
    """x as a sum of three bf16 numbers, to 24 bits."""
    hi = _bf16(x)
    mid = _bf16(x - hi)
    return hi, mid, _bf16(x - hi - mid)


@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("base", [0.0, 0.3, -5.85])
# scores (in powers of two) of the 95 keys below the first one's and of the last above it: both roundings, w's and the
# scaled w's, go up by nearly half a step
@pytest.mark.parametrize("below,above", [(0.950125313283208, 8.038471867966992), (0.95, 8.038)])
def test_one_rounding_of_the_weights(lb, page, D, base, below, above):
    keys = 97
    p = Problem("round", "bf16", 1, 1, D, page, [1], [keys], rubbish=False)
    score = np.full(keys, base - below)
    score[0], score[96] = base, base + above
    q = np.zeros((1, 1, D))
    q[0, 0, :3] = 1.0
    parts = _three(score * np.sqrt(D) * np.log(2.0))
    k, v = np.zeros((p.n_pages, 1, 1, page, D)), np.zeros((p.n_pages, 1, 1, page, D))
    c = 1.0 + np.arange(D) / 128.0
    for j in range(keys):
        at = (p.table[0, j // page], 0, 0, j % page)
        for i in range(3):
            k[at + (i,)] = parts[i][j]
        if 1 <= j < 96:
            v[at] = c
    p.q, p.k, p.v = (synth.f32_to_bf16_bits(a.astype(np.float32)) for a in (q, k, v))
    got = {}
    for max_kv in (None, 1 << 17):
        d = run_packed(lb, p, max_kv=max_kv)
        torch().cuda.synchronize()
        got[max_kv] = to_f64(d.o)[0, 0]
    s = synth.as_f64(p.q)[0, 0] @ p.rows(0, p.k)[0].T / np.sqrt(D)
    w = np.exp(s - s.max())
    o = (w / w.sum()) @ p.rows(0, p.v)[0]
    e_s = (D + 8) * U32 * np.abs(s).max()
    slack = 2 * e_s + 2 * (keys + 64) * U32 + 2.0 ** -18
    lo, hi = _bf16(o * (1 - U_BF16 - slack)), _bf16(o * (1 + U_BF16 + slack))
    for max_kv, o in got.items():
        bad = (o < lo) | (o > hi)
        assert not bad.any(), (max_kv, int(bad.sum()), o[bad][:3], lo[bad][:3], hi[bad][:3])
