"""Verification of drafted tokens (GPU) against the definition in 64 bits.

Decisions: u < p / q is taken where the two differ by more than 1e-5 relative (sums of V fp32 exponentials whose
arguments are off by at most 2^-22 times 40: 1e-5), and a race is won by more than 1e-5 relative; the inputs here are
checked to keep that distance.  Log-probabilities: 1e-5 absolute on the same grounds, and half a step of fp32."""
import numpy as np
import pytest

import synth
from _helpers import to_dev, torch
from _packed import store

pytestmark = pytest.mark.gpu

CLEAR = 1e-5


@pytest.fixture(scope="module")
def lb():
    import decoder_block_gb300 as m
    m.load()
    return m


class Drafts:
    def __init__(self, tag, dtype, V, drafts, temps=None, model=True, stride=None, max_drafts=None, pad=0, steps_first=False,
                 greedy=False):
        """drafts: drafts of each sequence, -1 for an empty slot."""
        rng = np.random.default_rng(sum(map(ord, tag)) + V)
        self.dtype, self.V, self.drafts = dtype, V, drafts
        n = len(drafts)
        self.n = n
        self.most = max(max(drafts), 0) if max_drafts is None else max_drafts
        self.offsets = np.concatenate([[0], np.cumsum([d + 1 for d in drafts])]).astype(np.int32)
        self.rows = int(self.offsets[-1]) + pad
        stride = stride or V
        self.target = rng.standard_normal((self.rows, stride)).astype(np.float32) * 2.5
        for r in range(self.rows):
            self.target[r, rng.integers(0, V, 3)] += 9
        if V > 20:
            self.target[:, rng.integers(0, V, 3)] = -np.inf
        self.draft = rng.standard_normal((n, max(self.most, 1), stride)).astype(np.float32) * 0.7
        for i, d in enumerate(drafts):
            for j in range(d):
                self.draft[i, j] += self.target[self.offsets[i] + j]
        self.tokens = rng.integers(0, V, self.rows).astype(np.int32)
        self.temps = None if temps is None else np.array([temps[i % len(temps)] for i in range(n)], np.float32)
        self.target[:, V:] = np.nan
        self.draft[..., V:] = np.nan
        self.target, self.draft = (store(x, dtype) for x in (self.target, self.draft))
        x64 = synth.as_f64(self.draft)[..., :V]
        for i, d in enumerate(drafts):
            for j in range(d):
                t = self.temp(i) or 1.0
                z = x64[i, j] / t if model else synth.as_f64(self.target)[self.offsets[i] + j, :V]
                self.tokens[self.offsets[i] + 1 + j] = np.argmax(z - np.log(rng.exponential(size=V) + 1e-30))
        self.model = model
        self.uniforms = rng.random((n, max(self.most, 1))).astype(np.float32)
        self.noise = (rng.exponential(size=(n, V)) + 1e-20).astype(np.float32)
        self.steps_first = steps_first
        self.greedy = greedy

    def temp(self, i):
        return 1.0 if self.temps is None else float(self.temps[i])

    def expected(self):
        """out, accepted, logprobs; asserts that every decision is clear."""
        out = np.full((self.n, self.most + 1), -1)
        acc, logp = np.zeros(self.n, int), np.zeros((self.n, self.most + 1))
        target, draft = synth.as_f64(self.target)[:, :self.V], synth.as_f64(self.draft)[..., :self.V]

        def log_softmax(x):
            with np.errstate(invalid="ignore", divide="ignore"):
                if not np.any(x > -np.inf) or np.any(np.isnan(x)) or np.any(x == np.inf):
                    return None
                y = x - x.max()
                return y - np.log(np.exp(y).sum())

        for i, d in enumerate(self.drafts):
            if d < 0:
                continue
            greedy = self.greedy or self.temp(i) == 0
            t = 1.0 if greedy else self.temp(i)
            for j in range(d + 1):
                row = target[self.offsets[i] + j]
                lp = log_softmax(row / t)
                if lp is None:
                    break
                x = self.tokens[self.offsets[i] + 1 + j] if j < d else -1
                lq = log_softmax(draft[i, j] / t) if j < d and self.model else None
                keep = False
                if j < d and 0 <= x < self.V:
                    if greedy:
                        keep = int(np.argmax(row)) == x
                    else:
                        with np.errstate(invalid="ignore"):
                            ratio = np.exp(lp[x] - (lq[x] if lq is not None else 0.0))
                        u = float(self.uniforms[i, j])
                        assert not abs(u - ratio) < CLEAR * ratio, "too close to call"
                        keep = u < ratio
                if keep:
                    out[i, j], logp[i, j] = x, lp[x]
                    acc[i] = j + 1
                    continue
                if greedy:
                    x = int(np.argmax(row))
                else:
                    p = np.exp(lp)
                    w = p.copy()
                    if j < d and lq is not None:
                        w = np.maximum(p - np.exp(lq), 0)
                    elif j < d and 0 <= x < self.V:
                        w[x] = 0
                    if not np.any(w > 0):
                        w = p
                    e = self.noise[i].astype(np.float64)
                    with np.errstate(invalid="ignore", divide="ignore"):
                        score = np.where(e > 0, w / e, 0.0)
                    x = int(np.argmax(score))
                    second = np.partition(score, -2)[-2] if self.V > 1 else 0
                    if score[x] > 0:
                        # what p - q loses to cancellation counts too
                        slack = CLEAR * (1 + p[x] / w[x])
                        assert second <= score[x] * (1 - slack), "too close to call"
                    else:
                        x = -1
                if x >= 0:
                    out[i, j], logp[i, j] = x, lp[x]
                break
        return out, acc, logp

    def run(self, lb, ws=None, stream=None):
        t = torch()
        d = self.d = type("D", (), {})()
        d.target = to_dev(self.target)
        draft = self.draft.transpose(1, 0, 2) if self.steps_first else self.draft
        d.draft = to_dev(np.ascontiguousarray(draft)) if self.model else None
        stride = self.target.shape[1]
        ss, step = (stride, self.n * stride) if self.steps_first else (max(self.most, 1) * stride, stride)
        d.offsets, d.tokens = to_dev(self.offsets), to_dev(self.tokens)
        d.temps = None if self.temps is None else to_dev(self.temps)
        d.uniforms = to_dev(self.uniforms[:, :self.most]) if self.most else None
        d.noise = None if self.greedy else to_dev(self.noise)
        d.batch = lb.make_draft_batch(d.offsets, d.tokens, self.rows, self.most, d.temps,
                                      None if self.greedy else d.uniforms, d.noise)
        d.code = lb.LLAMA_BF16 if self.dtype == "bf16" else lb.LLAMA_F32
        d.out = t.full((self.n, self.most + 1), 99, dtype=t.int32, device="cuda")
        d.acc = t.full((self.n,), 99, dtype=t.int32, device="cuda")
        d.logp = t.full((self.n, self.most + 1), 99.0, device="cuda")
        d.status = t.zeros(1, dtype=t.int32, device="cuda")
        need = lb.llama_op_verify_drafts_workspace_bytes(d.batch, self.V)
        d.ws = ws if ws is not None else t.full((max(need, 16),), 0xA5, dtype=t.uint8, device="cuda")
        d.call = lambda s: lb.check(lb.llama_op_verify_drafts(
            d.code, d.target, stride, d.draft, ss, step, self.V, d.batch, d.out, d.acc, d.logp, d.ws, d.ws.numel(),
            d.status, s))
        d.call(stream or t.cuda.current_stream())
        t.cuda.synchronize()
        return d

    def check(self, d, status=0):
        out, acc, logp = self.expected()
        assert np.array_equal(d.acc.cpu().numpy(), acc), (d.acc.cpu().numpy().tolist(), acc.tolist())
        assert np.array_equal(d.out.cpu().numpy(), out)
        got = d.logp.cpu().numpy().astype(np.float64)
        assert np.all(np.abs(got - logp) <= 1e-5 + np.abs(logp) * 2.0 ** -24)
        assert int(d.status[0]) == status


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("model", [True, False])
@pytest.mark.parametrize("V,stride", [(1, 1), (7, 9), (1000, 1000), (1001, 1001), (4099, 4160), (50257, 50257), (128256, 128256)])
def test_sizes(lb, dtype, model, V, stride):
    c = Drafts(f"s{dtype}", dtype, V, [3, 0, 1, 4], [0.7, 1.0, 0.0, 1.3], model=model, stride=stride)
    c.check(c.run(lb))


@pytest.mark.parametrize("n,V", [(1, 128256), (1, 300), (40, 9001), (300, 520), (3, 33000)])
@pytest.mark.parametrize("most", [0, 1, 8])
def test_batches(lb, n, V, most):
    rng = np.random.default_rng(n)
    c = Drafts("b", "f32", V, [int(rng.integers(0, most + 1)) for _ in range(n)], [1.0, 0.5], max_drafts=most, pad=2)
    c.check(c.run(lb))


def test_most_drafts_and_sequences(lb):
    c = Drafts("most", "bf16", 257, [64, 0, 63], None)
    c.check(c.run(lb))
    c = Drafts("seqs", "f32", 65, [1] * 4096, [1.0, 0.0])
    c.check(c.run(lb))


@pytest.mark.parametrize("greedy", [True, False])
def test_greedy(lb, greedy):
    c = Drafts("g", "bf16", 3000, [4, 2, 0], [0.0], greedy=greedy)
    # equal maxima, and drafts that follow the lowest of them for a while
    x = synth.as_f64(c.target)
    x[0, [17, 900]] = 50.0
    x[1, [2999, 3 - 1]] = 60.0
    c.target = store(x.astype(np.float32), "bf16")
    c.tokens[1:4] = [17, 2, 5]
    c.check(c.run(lb))
    assert c.d.out.cpu().numpy()[0, :2].tolist() == [17, 2]


def test_steps_first_and_empty_slots(lb):
    c = Drafts("e", "f32", 700, [2, -1, 3, 0, -1, 1], [0.9], steps_first=True, max_drafts=5, pad=4)
    c.check(c.run(lb))


def test_equal_distributions_keep_everything(lb):
    c = Drafts("same", "f32", 5000, [4, 4, 4], [1.0])
    for i, d in enumerate(c.drafts):
        for j in range(d):
            c.draft[i, j] = c.target[c.offsets[i] + j]
    c.uniforms[:] = np.float32(1 - 2.0 ** -23)
    d = c.run(lb)
    assert d.acc.cpu().numpy().tolist() == [4, 4, 4]
    assert int(d.out.min()) >= 0


def test_a_certain_refusal(lb):
    """p[x] = 0: refused whatever u; q[x] = 0: kept; nothing of p - q left: drawn from p."""
    c = Drafts("c", "f32", 64, [1, 1, 1], [1.0])
    c.uniforms[:] = 0.0
    for i in range(3):
        r = c.offsets[i]
        c.tokens[r + 1] = 11
        c.target[r] = np.linspace(-3, 3, 64)
        c.draft[i, 0] = np.linspace(3, -3, 64)
    c.target[c.offsets[0], 11] = -np.inf
    c.draft[1, 0, 11] = -np.inf
    # both put everything on one token, which the draft is not: p = q there, and 0 for the draft
    c.target[c.offsets[2]] = -np.inf
    c.target[c.offsets[2], 40] = 1.0
    c.draft[2, 0] = -np.inf
    c.draft[2, 0, 40] = 5.0
    d = c.run(lb)
    c.check(d)
    assert d.acc.cpu().numpy().tolist() == [0, 1, 0] and int(d.out[2, 0]) == 40


def test_rows_without_probabilities(lb):
    c = Drafts("n", "f32", 5000, [2, 2, 2, 2], [1.0, 0.0])
    c.target[c.offsets[0] + 1, 77] = np.nan
    c.target[c.offsets[1], 4999] = np.inf
    c.target[c.offsets[2] + 2] = -np.inf
    c.draft[3, 0, 5] = np.nan       # greedy: not looked at
    c.draft[0, 0, 9] = np.inf       # counts as a certain draft
    c.check(c.run(lb))


def test_noise_that_is_not_above_zero_is_never_drawn(lb):
    c = Drafts("z", "f32", 200, [0, 0, 0], None)
    best = [int(np.argmax(synth.as_f64(c.target)[r, :200] - np.log(c.noise[r]))) for r in range(3)]
    for r, bad in enumerate((0.0, -1.0, np.nan)):
        c.noise[r, best[r]] = bad
    c.check(c.run(lb))
    c.noise[:] = 0.0
    d = c.run(lb)
    assert d.out.cpu().numpy().ravel().tolist() == [-1, -1, -1]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [64, 40001])  # a CTA a sequence, a cluster a sequence
@pytest.mark.parametrize("model", [True, False])
def test_a_residual_whose_ids_have_no_noise_draws_nothing(lb, model, V, dtype):
    """max(p - q, 0) is above 0 at ids that may not be drawn, and 0 elsewhere: no token, and not one from p, which
    has weight at the refused draft and at every id that the draft's q covers."""
    c = Drafts("rn", dtype, V, [1, 1, 1, 2], [1.0], model=model)
    x = 6
    high = np.arange(V) % 2 == 1   # p > q there
    for i in range(c.n):
        for j in range(c.drafts[i]):
            c.target[c.offsets[i] + j] = store(np.where(high, 1.0, -1.0).astype(np.float32), dtype)
            c.draft[i, j] = store(np.where(high, -1.0, 1.0).astype(np.float32), dtype)
            c.tokens[c.offsets[i] + 1 + j] = x
    c.uniforms[:] = 0.9            # p[x] / q[x] = e^-2
    left = high if model else np.arange(V) != x
    for i, bad in enumerate((0.0, -1.0, np.nan)):
        c.noise[i, left] = bad
    c.noise[3, left] = 0.0
    c.noise[3, V - 3 if (V - 3) % 2 else V - 4] = 2.0  # one that may be drawn
    d = c.run(lb)
    c.check(d)
    assert d.out[:3].max() == -1 and int(d.out[3, 0]) >= V - 4


@pytest.mark.parametrize("V", [64, 40001])
def test_an_empty_residual_is_drawn_from_p(lb, V):
    """The other side: p <= q at every id and q has more there, so that p - q is 0 and the token comes from p, among the
    ids whose noise lets it."""
    c = Drafts("er", "f32", V, [1, 1, 1], [1.0])
    c.uniforms[:] = 0.5
    for i in range(3):
        r = c.offsets[i]
        c.tokens[r + 1] = 11
        c.target[r] = -np.inf
        c.draft[i, 0] = -np.inf
        c.target[r, [40, V - 2]] = 1.0     # p = q = 1 / 2 at both; the draft, 11, has neither
        c.draft[i, 0, [40, V - 2]] = 5.0
    c.noise[:, 40], c.noise[:, V - 2] = [1.0, 2.0, 0.0], [2.0, 1.0, 0.0]
    d = c.run(lb)
    c.check(d)
    assert d.out[:, 0].tolist() == [40, V - 2, -1]


def test_bad_inputs_are_reported(lb):
    c = Drafts("bad", "f32", 300, [2, 2, 1], [1.0])
    c.tokens[1] = 300
    c.tokens[5] = -7
    c.check(c.run(lb), lb.LLAMA_ERR_RANGE)
    for temp in (-1.0, np.inf, np.nan):
        c = Drafts("bt", "f32", 300, [2, 1], [1.0])
        c.temps[0] = temp
        d = c.run(lb)
        assert d.out[0].tolist() == [-1, -1, -1] and int(d.acc[0]) == 0 and float(d.logp[0].abs().max()) == 0
        assert int(d.status[0]) == lb.LLAMA_ERR_RANGE and int(d.out[1, 0]) >= 0
    c = Drafts("bo", "f32", 300, [1, 1, 2], [1.0])
    c.offsets = np.array([0, 9, 4, 7], np.int32)  # the first ends behind the rows, the second descends
    d = c.run(lb)
    assert d.out[0].tolist() == [-1, -1, -1] and d.out[1].tolist() == [-1, -1, -1]
    assert int(d.status[0]) == lb.LLAMA_ERR_RANGE
    for greedy in (True, False):  # rows that no part of the sums has seen
        c = Drafts("bo2", "f32", 5000, [2, 2, 2], [1.0], greedy=greedy)
        c.offsets = np.array([0, 3, 1, 4], np.int32)
        d = c.run(lb, ws=torch().randint(0, 256, (1 << 16,), dtype=torch().uint8, device="cuda"))
        assert int(d.status[0]) == lb.LLAMA_ERR_RANGE
        assert d.out[1].tolist() == [-1, -1, -1]
        assert int(d.out.max()) < 5000 and int(d.out.min()) >= -1


def test_any_alignment(lb):
    """Rows, noise and results that begin at any element."""
    t = torch()
    for dtype in ("f32", "bf16"):
        c = Drafts("al", dtype, 5003, [2, 1], [0.8], stride=5005)
        d = c.run(lb)
        want = [x.clone() for x in (d.out, d.acc, d.logp)]
        for off in (1, 3):
            def moved(x):
                flat = t.zeros(x.numel() + off, dtype=x.dtype, device="cuda")
                flat[off:] = x.reshape(-1)
                d.keep = getattr(d, "keep", []) + [flat]
                return flat[off:].view(x.shape)
            d.target, d.draft = moved(d.target), moved(d.draft)
            d.batch = lb.make_draft_batch(moved(d.offsets), moved(d.tokens), c.rows, c.most, moved(d.temps),
                                          moved(d.uniforms), moved(d.noise))
            d.out, d.acc, d.logp = (moved(x.fill_(99)) for x in (d.out, d.acc, d.logp))
            d.call(t.cuda.current_stream())
            t.cuda.synchronize()
            assert all(t.equal(a, b) for a, b in zip(want[:2], (d.out, d.acc)))
            assert float((want[2] - d.logp).abs().max()) < 1e-5


def test_graph_replays_read_the_inputs_of_then(lb):
    t = torch()
    a, b = (Drafts(f"gr{i}", "f32", 6000, [3, 1, 2], [1.0, 0.6]) for i in range(2))
    d = a.run(lb)
    side = t.cuda.Stream()
    g = t.cuda.CUDAGraph()
    with t.cuda.graph(g, stream=side):
        d.call(side)
    g.replay()
    t.cuda.synchronize()
    a.check(d)
    d.target.copy_(to_dev(b.target))
    d.draft.copy_(to_dev(b.draft))
    d.tokens.copy_(to_dev(b.tokens))
    d.uniforms.copy_(to_dev(b.uniforms))
    d.noise.copy_(to_dev(b.noise))
    d.ws.random_(0, 256)
    g.replay()
    t.cuda.synchronize()
    b.check(d)


def test_tokens_follow_the_target(lb):
    """What comes out at a sequence's first place is distributed as p, whatever the draft's q: chi-squared over 8 tokens
    and 4096 sequences of one row's logits (the 1e-6 quantile of 7 degrees of freedom is 40.5)."""
    V, n = 8, 4096
    c = Drafts("chi", "f32", V, [1] * n, [1.0])
    c.target[:] = np.array([0.3, -1, 0.8, 0, -0.4, 1.2, -2, 0.1], np.float32)
    c.draft[:] = np.array([-1, 1, 0, 0.5, -0.4, -1.2, 1, 0.1], np.float32)
    rng = np.random.default_rng(8)
    q = np.exp(c.draft[0, 0].astype(np.float64))
    c.tokens[1::2] = rng.choice(V, n, p=q / q.sum())
    first = c.run(lb).out[:, 0].cpu().numpy()
    p = np.exp(c.target[0].astype(np.float64))
    p /= p.sum()
    seen = np.bincount(first, minlength=V)
    assert ((seen - n * p) ** 2 / (n * p)).sum() < 40.5


def _follows(p, seen):
    """Chi-squared over 8 tokens: the 1e-6 quantile of 7 degrees of freedom is 40.5."""
    p = np.exp(p.astype(np.float64))
    p /= p.sum()
    n = len(seen)
    count = np.bincount(seen, minlength=8)
    return ((count - n * p) ** 2 / (n * p)).sum() < 40.5


def test_tokens_follow_the_target_where_drafts_are_certain(lb):
    """Looked-up drafts, one token for every sequence: what comes out at the first place is distributed as p."""
    V, n = 8, 4096
    c = Drafts("chc", "f32", V, [1] * n, [1.0], model=False)
    c.target[:] = np.array([0.3, -1, 0.8, 0, -0.4, 1.2, -2, 0.1], np.float32)
    for x in (5, 6):
        c.tokens[1::2] = x
        assert _follows(c.target[0], c.run(lb).out[:, 0].cpu().numpy())


def test_the_token_behind_kept_drafts_follows_the_target(lb):
    """Drafts that are all kept (u = 0): the token behind is distributed as p of the last row, at the temperature."""
    V, n = 8, 4096
    for model in (True, False):
        c = Drafts("chb", "f32", V, [1] * n, [0.5], model=model)
        c.target[1::2] = np.array([0.3, -1, 0.8, 0, -0.4, 0.7, -0.5, 0.1], np.float32)
        c.tokens[1::2] = c.tokens[1::2] % V
        c.target[0::2], c.draft[:] = 0.0, 0.0
        c.uniforms[:] = 0.0
        d = c.run(lb)
        assert d.acc.cpu().numpy().min() == 1
        assert _follows(2 * c.target[1], d.out[:, 1].cpu().numpy())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("size,temp", [(0.2, 1.0), (2.5, 1.0), (2.5, 0.1), (2.5, 3.0)])
def test_decisions_near_the_ratio(lb, dtype, size, temp):
    """u within a few 1e-5 of p / q on both sides of it, over a wide vocabulary, flat and steep."""
    V, n = 128256, 16
    c = Drafts("near", dtype, V, [1] * n, [temp])
    rng = np.random.default_rng(5)
    row = (rng.standard_normal(V) * size).astype(np.float32)
    c.target[:] = store(row, dtype)
    c.draft[:] = store(row + (rng.standard_normal(V) * 0.2 * size * temp).astype(np.float32), dtype)
    p, q = (np.exp((y - y.max()) / temp) for y in (synth.as_f64(c.target)[0], synth.as_f64(c.draft)[0, 0]))
    ratio = (p / p.sum()) / (q / q.sum())
    at = np.flatnonzero((ratio > 0.3) & (ratio < 0.9) & (p > 0))
    off = np.concatenate([np.linspace(-4e-5, -1.1e-5, n // 2), np.linspace(1.1e-5, 4e-5, n // 2)])
    for i in range(n):
        x = at[(i * 977) % len(at)]
        c.tokens[c.offsets[i] + 1] = x
        c.uniforms[i, 0] = ratio[x] * (1 + off[i])
    d = c.run(lb)
    assert d.acc.cpu().numpy().tolist() == [1] * (n // 2) + [0] * (n // 2)
    c.check(d)


@pytest.mark.parametrize("V,temp", [(4099, 0.3), (128256, 0.1), (128256, 0.7), (200003, 0.9)])
def test_decisions_on_certain_drafts_near_p(lb, V, temp):
    """Half of the probability on the draft and the rest flat: every weight of the rest has the same rounded argument,
    so that their errors add up."""
    n = 8
    c = Drafts("near2", "f32", V, [1] * n, [temp], model=False)
    temp, x = float(np.float32(temp)), 77
    c.target[:] = 0.0
    c.target[:, x] = np.float32(temp * np.log(V - 1) * 1.01)
    c.tokens[1::2] = x
    y = synth.as_f64(c.target)[0] / temp
    p = 1 / np.exp(y - y.max()).sum()
    c.uniforms[:, 0] = p * (1 + np.concatenate([np.linspace(-4e-5, -1.1e-5, n // 2), np.linspace(1.1e-5, 4e-5, n // 2)]))
    d = c.run(lb)
    assert d.acc.cpu().numpy().tolist() == [1] * (n // 2) + [0] * (n // 2)
    c.check(d)


def test_a_speculative_step(lb):
    """Write, attention over the 4-bit pages, logits, verification, one after another on one stream: greedy drafts that
    the step itself would choose are all kept, and a wrong one ends them."""
    from _kv4 import Kv4Problem
    t = torch()
    H, G, D, V = 8, 2, 64, 1024
    p = Kv4Problem("spec", "bf16", H, G, D, 16, [4, 3, 1], [200, 77, 31])
    d = p.device(lb)
    T = p.T
    qkv = to_dev(store(synth.normal(0, "spec/qkv", (T, (H + 2 * G) * D)), "bf16"))
    head = to_dev(store(synth.normal(0, "spec/head", (V, H * D)), "bf16"))
    rope = t.empty((256, D // 2, 2), device="cuda")
    st = t.cuda.Stream()
    st.wait_stream(t.cuda.current_stream())
    q_out, logits = t.empty_like(d.q), t.empty((T, V), device="cuda")
    need = lb.llama_op_attention_packed_kv4_workspace_bytes(d.code, d.batch, H, G, D)
    ws = t.empty(max(need, 16), dtype=t.uint8, device="cuda")
    tokens = t.zeros(T, dtype=t.int32, device="cuda")
    out, acc = t.empty((3, 4), dtype=t.int32, device="cuda"), t.empty(3, dtype=t.int32, device="cuda")
    batch = lb.make_draft_batch(d.offsets, tokens, T, 3)
    vws = t.empty(lb.llama_op_verify_drafts_workspace_bytes(batch, V), dtype=t.uint8, device="cuda")

    def step():
        lb.check(lb.llama_op_rope_kv4_write_paged(d.code, qkv, q_out, d.kv, d.batch, rope, 256, H, G, D, 0, d.status, st))
        lb.check(lb.llama_op_attention_packed_kv4(d.code, q_out, d.kv, d.batch, d.o, H, G, D, ws, ws.numel(), d.status, st))
        lb.check(lb.llama_op_linear(d.code, d.o, head, None, logits, T, V, H * D, lb.EPI_F32OUT, st))
        lb.check(lb.llama_op_verify_drafts(lb.LLAMA_F32, logits, V, None, 0, 0, V, batch, out, acc, None, vws,
                                           vws.numel(), d.status, st))

    lb.check(lb.llama_op_rope_table(rope, 256, D, 1e4, None, st))
    step()
    t.cuda.synchronize()
    best = logits.argmax(-1).to(t.int32)
    tokens[1:4] = best[0:3]
    tokens[5], tokens[6] = best[4], (best[5] + 1) % V
    t.cuda.synchronize()
    step()
    t.cuda.synchronize()
    assert acc.tolist() == [3, 1, 0] and int(d.status[0]) == 0
    assert out[0].tolist() == best[0:4].tolist()
    assert out[1].tolist() == best[4:6].tolist() + [-1, -1]
    assert out[2].tolist() == [int(best[7]), -1, -1, -1]
    # the attention of that step is the plain one over the pages as they now are
    from _kv4 import unpack, values
    from _helpers import to_f64, to_host_bits
    p.k, p.v = (values(*unpack(x.cpu().numpy(), 16, D)).astype(np.float32)[:, None] for x in (d.k, d.v))
    p.q = to_host_bits(q_out)
    p.check(to_f64(d.o))
