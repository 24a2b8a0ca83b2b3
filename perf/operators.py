"""Cases, inputs and plain forms of the operators that serve a batch of sequences of different lengths.

Four operators of include/llama_ops.h are measured here:

  write    llama_op_rope_kv_write_paged     RoPE on packed tokens, keys and values stored into cache pages
  packed   llama_op_attention_packed        causal grouped-query attention of packed prompts over the pages
  decode   llama_op_attention_paged_decode  one new token per sequence over the pages
  logprobs llama_op_token_logprobs          log-probabilities of given tokens, entropy, top alternatives

`own` False: elementary torch operations in 32 bits.  `own` True: the library's entry points.
"""
import math

import torch

own = False

_DEV = "cuda"
_THETA = 500000.0


# ------------------------------------------------------------------ cases ---

def listed():
    return [
        # A whole 8192-token prompt of the 8B-shaped block: the largest prompt pass.
        _packed("packed_8b_s8192", "bf16", 32, 8, 128, 64, "8192", "0", 0),
        # One scheduler step of a server under load: fresh prompts, prompts continued over a cached prefix (prefix
        # reuse, chunked prompts), a lone token riding along, an empty slot, and padding up to a fixed token count.
        _packed("packed_8b_ragged", "bf16", 32, 8, 128, 16, "2048,1,777,0,1301,64,3001,129,512,40",
                "0,2900,0,0,1024,5003,0,127,2000,0", 23),
        # Short chat turns on the 135M-shaped model (9 heads on 3): a few microseconds of work.
        _packed("packed_135m_short", "bf16", 9, 3, 64, 16, "31,7,120,1,64,18,55,90", "0,0,0,33,0,200,0,0", 0),
        # The fp32 configuration over a few hundred tokens.
        _packed("packed_tiny_f32", "f32", 4, 2, 16, 16, "200,33,1,150", "0,7,300,0", 0),
        # A decode step of 64 users of the 8B-shaped block, each at a different point of its conversation.
        _decode("decode_8b_b64", "bf16", 32, 8, 128, 64, ",".join(str(4096 - 61 * ((i * 29) % 64)) for i in range(64))),
        # One user with a very long document in the cache: work exists only along the cache's length.
        _decode("decode_8b_b1_long", "bf16", 32, 8, 128, 32, "120001"),
        # A few short conversations on the 135M-shaped model: pure latency.
        _decode("decode_135m_b8", "bf16", 9, 3, 64, 16, "300,17,1,128,1000,64,0,511"),
        # Rotating and storing a whole prompt of the 8B-shaped block.
        _write("write_8b_prompt", "bf16", 32, 8, 128, 64, "6001,2100,91", "0,1000,4000", "interleaved", 0),
        # The same for one decode step of 24 users of the 135M-shaped model.
        _write("write_135m_step", "bf16", 9, 3, 64, 16, ",".join(["1"] * 24),
               ",".join(str((i * 37) % 1000) for i in range(24)), "halves", 8),
        # Scoring a 2048-token prompt of the 8B-shaped stack, with the 20 likeliest alternatives.
        _logprobs("logprobs_8b_prompt", "f32", 2048, 128256, 128256, 20),
        # One decode step of 64 users with bf16 logits in rows padded to a multiple of 64 beyond an odd vocabulary.
        _logprobs("logprobs_step_b64", "bf16", 64, 128255, 128320, 5),
        # One user of the 135M-shaped stack: latency.
        _logprobs("logprobs_135m_b1", "f32", 1, 49152, 49152, 1),
    ]


def _packed(name, dtype, H, G, D, page, q_lens, prefixes, pad):
    return dict(name=name, op="packed", dtype=dtype, H=H, G=G, D=D, page=page, q_lens=q_lens, prefixes=prefixes,
                pad=pad)


def _decode(name, dtype, H, G, D, page, kv_lens):
    return dict(name=name, op="decode", dtype=dtype, H=H, G=G, D=D, page=page, kv_lens=kv_lens)


def _write(name, dtype, H, G, D, page, q_lens, prefixes, layout, pad):
    return dict(name=name, op="write", dtype=dtype, H=H, G=G, D=D, page=page, q_lens=q_lens, prefixes=prefixes,
                layout=layout, pad=pad)


def _logprobs(name, dtype, T, V, stride, top):
    return dict(name=name, op="logprobs", dtype=dtype, T=T, V=V, stride=stride, top=top)


def _ints(text):
    return [int(v) for v in text.split(",")]


def _log_int(rng, lo, hi):
    """A whole number in [lo, hi], its logarithm spread evenly."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.999)))))))


def _draw_heads(rng):
    """(dtype, H, G, D): mostly bf16 with the tensor-core head widths, the small widths and fp32 among them."""
    dtype = "f32" if rng.random() < 0.2 else "bf16"
    D = rng.choice([64, 128]) if rng.random() < 0.8 else rng.choice([16, 32])
    G = rng.choice([1, 2, 3, 4, 8])
    r = rng.choice([1, 2, 3, 4, 5, 6, 7, 8, 12, 16] if G <= 4 else [1, 2, 3, 4, 5, 8])
    return dtype, G * r, G, D


def draw(rng):
    op = rng.choice(["packed", "packed", "packed", "decode", "decode", "write", "logprobs", "logprobs"])
    page = rng.choice([16, 32, 64, 128, 256])
    if op == "logprobs":
        V = _log_int(rng, 1000, 160000)
        T = _log_int(rng, 1, max(1, min(4096, 260_000_000 // V)))
        stride = V if rng.random() < 0.5 else (V + 63) // 64 * 64
        return _logprobs("", rng.choice(["f32", "bf16"]), T, V, stride, rng.choice([0, 1, 5, 20, 32]))
    dtype, H, G, D = _draw_heads(rng)
    small = dtype == "f32" or D < 64
    n = _log_int(rng, 1, 48)
    if op == "decode":
        longest = _log_int(rng, 16, 200_000 if n <= 4 else 8192)
        if small:
            longest = min(longest, 8192)
        longest = min(longest, max(16, 480_000_000 // (n * 2 * G * D * (4 if dtype == "f32" else 2))))
        lens = [longest if i == 0 else rng.randint(0, longest) for i in range(n)]
        return _decode("", dtype, H, G, D, page, ",".join(map(str, lens)))
    longest = _log_int(rng, 1, 700 if small else 6000)
    q_lens = [longest if i == 0 else _log_int(rng, 1, longest) for i in range(n)]
    prefixes = [0 if rng.random() < 0.6 else rng.randint(1, 4000) for _ in range(n)]
    budget = 700 if small else (8192 if op == "write" else 6000)  # query tokens of one pass
    total = 0
    for i in range(n):
        q_lens[i] = min(q_lens[i], max(0, budget - total))
        total += q_lens[i]
    while sum(q * (p + q) for q, p in zip(q_lens, prefixes)) * 4 * D * H > 500_000_000_000:
        q_lens, prefixes = [(q + 1) // 2 for q in q_lens], [p // 2 for p in prefixes]
    pad = rng.choice([0, 0, 5, 64])
    args = ("", dtype, H, G, D, page, ",".join(map(str, q_lens)), ",".join(map(str, prefixes)))
    if op == "write":
        return _write(*args, rng.choice(["interleaved", "halves"]), pad)
    return _packed(*args, pad)


# ----------------------------------------------------------------- inputs ---

def _torch_dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _normal(gen, shape, dtype, std=1.0):
    out = torch.empty(shape, dtype=dtype, device=_DEV)
    flat = out.view(-1)
    step = 1 << 27
    for i in range(0, flat.numel(), step):
        n = min(step, flat.numel() - i)
        flat[i:i + n] = torch.randn(n, device=_DEV, generator=gen) * std
    return out


def _pages_of(lens, page):
    return [(n + page - 1) // page for n in lens]


def _cache(gen, case, kv_lens, dtype):
    """A page pool with a few spare pages, in an order that a server's allocator leaves behind."""
    counts = _pages_of(kv_lens, case["page"])
    n_pages = sum(counts) + 3
    order = torch.randperm(n_pages, device=_DEV, generator=gen).to(torch.int32)
    width = max(max(counts), 1)
    table = torch.zeros((len(kv_lens), width), dtype=torch.int32, device=_DEV)
    at = 0
    for i, c in enumerate(counts):
        table[i, :c] = order[at:at + c]
        at += c
    shape = (n_pages, case["G"], case["page"], case["D"])
    return _normal(gen, shape, dtype), _normal(gen, shape, dtype), table


def _batch(case):
    q_lens, prefixes = _ints(case["q_lens"]), _ints(case["prefixes"])
    kv_lens = [a + b for a, b in zip(q_lens, prefixes)]
    offsets = [0]
    for n in q_lens:
        offsets.append(offsets[-1] + n)
    return q_lens, kv_lens, offsets


def _rope_table(max_seq, D):
    f = _THETA ** (-2.0 * torch.arange(D // 2, dtype=torch.float64, device=_DEV) / D)
    ang = torch.arange(max_seq, dtype=torch.float64, device=_DEV)[:, None] * f
    return torch.stack([ang.cos(), ang.sin()], dim=-1).float().contiguous()


def prepare(case, seed):
    gen = torch.Generator(device=_DEV)
    gen.manual_seed(seed)
    dtype = _torch_dtype(case)
    st = dict(case=case)
    if case["op"] == "logprobs":
        T, V, stride = case["T"], case["V"], case["stride"]
        logits = _normal(gen, (T, stride), dtype, std=2.5)
        logits[:, V:] = float("nan")  # the padding of a row is never a logit
        likely = torch.randint(0, V, (T, 4), device=_DEV, generator=gen)
        boost = 8.0 + 8.0 * torch.rand((T, 4), device=_DEV, generator=gen)
        logits.scatter_(1, likely, boost.to(dtype))
        banned = torch.randint(0, V, (7,), device=_DEV, generator=gen)  # tokens a server never lets through
        logits[:, banned] = float("-inf")
        anywhere = torch.randint(0, V, (T,), device=_DEV, generator=gen)
        pick = torch.rand((T,), device=_DEV, generator=gen) < 0.7
        targets = torch.where(pick, likely[:, 0], anywhere).to(torch.int32)
        k = case["top"]
        st.update(logits=logits, targets=targets, logp=torch.zeros(T, device=_DEV), entropy=torch.zeros(T, device=_DEV),
                  top_ids=torch.zeros((T, k), dtype=torch.int32, device=_DEV) if k else None,
                  top_logp=torch.zeros((T, k), device=_DEV) if k else None)
        return st
    H, G, D = case["H"], case["G"], case["D"]
    if case["op"] == "decode":
        kv_lens = _ints(case["kv_lens"])
        k, v, table = _cache(gen, case, kv_lens, dtype)
        n = len(kv_lens)
        st.update(q=_normal(gen, (n, H, D), dtype), k=k, v=v, table=table,
                  kv_lens=torch.tensor(kv_lens, dtype=torch.int32, device=_DEV), max_kv=max(kv_lens),
                  o=torch.zeros((n, H, D), dtype=dtype, device=_DEV))
    else:
        q_lens, kv_lens, offsets = _batch(case)
        k, v, table = _cache(gen, case, kv_lens, dtype)
        T = offsets[-1] + case["pad"]
        st.update(k=k, v=v, table=table, T=T, offsets=torch.tensor(offsets, dtype=torch.int32, device=_DEV),
                  kv_lens=torch.tensor(kv_lens, dtype=torch.int32, device=_DEV), max_kv=max(kv_lens))
        if case["op"] == "packed":
            st.update(q=_normal(gen, (T, H, D), dtype), o=torch.zeros((T, H, D), dtype=dtype, device=_DEV))
        else:
            st.update(qkv=_normal(gen, (T, (H + 2 * G) * D), dtype), rope=_rope_table(max(kv_lens), D),
                      q_out=torch.zeros((T, H, D), dtype=dtype, device=_DEV))
    if own:
        _prepare_own(case, st)
    return st


def _prepare_own(case, st):
    """What a program keeps between calls: the structs, and a workspace as large as the call asks for."""
    import decoder_block_gb300 as lb
    code = lb.LLAMA_BF16 if case["dtype"] == "bf16" else lb.LLAMA_F32
    st["code"] = code
    st["kv"] = lb.make_paged_kv_cache(st["k"], st["v"], st["table"])
    need = 0
    if case["op"] == "decode":
        need = lb.llama_op_attention_paged_decode_workspace_bytes(code, len(st["kv_lens"]), st["max_kv"], case["H"],
                                                                  case["G"], case["D"])
    else:
        st["batch"] = lb.make_packed_batch(st["offsets"], st["kv_lens"], st["T"], st["max_kv"])
        if case["op"] == "packed":
            need = lb.llama_op_attention_packed_workspace_bytes(code, st["batch"], case["H"], case["G"], case["D"])
    st["ws"] = torch.empty(max(need, 16), dtype=torch.uint8, device=_DEV)


# -------------------------------------------------------------------- run ---

def run(st):
    return _run_own(st) if own else _PLAIN[st["case"]["op"]](st)


def _run_own(st):
    import decoder_block_gb300 as lb
    c = st["case"]
    stream = torch.cuda.current_stream()
    if c["op"] == "packed":
        lb.check(lb.llama_op_attention_packed(st["code"], st["q"], st["kv"], st["batch"], st["o"], c["H"], c["G"],
                                              c["D"], st["ws"], st["ws"].numel(), None, stream))
        return st["o"]
    if c["op"] == "decode":
        lb.check(lb.llama_op_attention_paged_decode(st["code"], st["q"], st["kv"], st["kv_lens"], len(st["kv_lens"]),
                                                    st["max_kv"], st["o"], c["H"], c["G"], c["D"], st["ws"],
                                                    st["ws"].numel(), None, stream))
        return st["o"]
    if c["op"] == "write":
        layout = lb.LLAMA_ROPE_HALVES if c["layout"] == "halves" else lb.LLAMA_ROPE_INTERLEAVED
        lb.check(lb.llama_op_rope_kv_write_paged(st["code"], st["qkv"], st["q_out"], st["kv"], st["batch"], st["rope"],
                                                 st["rope"].shape[0], c["H"], c["G"], c["D"], layout, None, stream))
        return st["q_out"], st["k"], st["v"]
    code = lb.LLAMA_BF16 if c["dtype"] == "bf16" else lb.LLAMA_F32
    lb.check(lb.llama_op_token_logprobs(code, st["logits"], c["stride"], st["targets"], c["T"], c["V"], st["logp"],
                                        st["entropy"], c["top"], st["top_ids"], st["top_logp"], None, stream))
    return _logprob_outputs(st["logp"], st["entropy"], st["top_ids"], st["top_logp"])


def _logprob_outputs(logp, entropy, ids, top):
    return (logp, entropy) if ids is None else (logp, entropy, ids, top)


def _gather(pool, pages, L):
    """[G][L][D] fp32 of one sequence's pages."""
    x = pool[pages.long()]                      # [n][G][page][D]
    return x.permute(1, 0, 2, 3).reshape(pool.shape[1], -1, pool.shape[3])[:, :L].float()


def _plain_packed(st):
    c = st["case"]
    H, G, D = c["H"], c["G"], c["D"]
    q_lens, kv_lens, offsets = _batch(c)
    counts = _pages_of(kv_lens, c["page"])
    o = st["o"]
    for i, (n, L) in enumerate(zip(q_lens, kv_lens)):
        if n == 0:
            continue
        k, v = _gather(st["k"], st["table"][i, :counts[i]], L), _gather(st["v"], st["table"][i, :counts[i]], L)
        keys = torch.arange(L, device=_DEV)
        for s0 in range(0, n, 1024):
            s1 = min(n, s0 + 1024)
            last = L - n + s1
            q = st["q"][offsets[i] + s0:offsets[i] + s1].float().permute(1, 0, 2).reshape(G, -1, D)
            s = torch.matmul(q, k[:, :last].transpose(1, 2)) * (1.0 / math.sqrt(D))
            s = s.view(H, s1 - s0, last)
            pos = torch.arange(L - n + s0, L - n + s1, device=_DEV)
            s.masked_fill_(keys[:last] > pos[:, None], float("-inf"))
            p = torch.exp(s - s.amax(-1, keepdim=True))
            p = p / p.sum(-1, keepdim=True)
            r = torch.matmul(p.view(G, -1, last), v[:, :last]).view(H, s1 - s0, D)
            o[offsets[i] + s0:offsets[i] + s1] = r.permute(1, 0, 2).to(o.dtype)
    return o


def _plain_decode(st):
    c = st["case"]
    H, G, D = c["H"], c["G"], c["D"]
    lens, table, o = st["kv_lens"], st["table"], st["o"]
    n, L = len(lens), table.shape[1] * c["page"]
    keys = torch.arange(L, device=_DEV)
    step = max(1, (1 << 29) // (G * L * D))
    for b0 in range(0, n, step):
        b1 = min(n, b0 + step)
        idx = table[b0:b1].long()
        k = st["k"][idx].permute(0, 2, 1, 3, 4).reshape(b1 - b0, G, L, D).float()
        q = st["q"][b0:b1].float().view(b1 - b0, G, H // G, D)
        s = torch.matmul(q, k.transpose(2, 3)) * (1.0 / math.sqrt(D))
        visible = keys[None, :] < lens[b0:b1, None].long()
        s = torch.where(visible[:, None, None, :], s, torch.full_like(s, -3.0e38))
        p = torch.exp(s - s.amax(-1, keepdim=True)) * visible[:, None, None, :]
        z = p.sum(-1, keepdim=True)
        p = p / torch.where(z > 0, z, torch.ones_like(z))
        v = st["v"][idx].permute(0, 2, 1, 3, 4).reshape(b1 - b0, G, L, D).float()
        o[b0:b1] = torch.matmul(p, v).view(b1 - b0, H, D).to(o.dtype)
    return o


def _plain_write(st):
    c = st["case"]
    H, G, D, page = c["H"], c["G"], c["D"], c["page"]
    n_tok = int(_batch(c)[2][-1])
    if n_tok == 0:
        return st["q_out"], st["k"], st["v"]
    tok = torch.arange(n_tok, device=_DEV)
    off = st["offsets"].long()
    seq = torch.searchsorted(off[1:], tok, right=True)
    pos = st["kv_lens"].long()[seq] - (off[seq + 1] - tok)
    cs = st["rope"][pos]                         # [T][D/2][2]
    cos, sin = cs[..., 0][:, None], cs[..., 1][:, None]
    x = st["qkv"][:n_tok].float().view(n_tok, H + 2 * G, D)
    qk = x[:, :H + G]
    if c["layout"] == "halves":
        a, b = qk[..., :D // 2], qk[..., D // 2:]
        rot = torch.cat([a * cos - b * sin, a * sin + b * cos], dim=-1)
    else:
        a, b = qk[..., 0::2], qk[..., 1::2]
        rot = torch.stack([a * cos - b * sin, a * sin + b * cos], dim=-1).reshape(qk.shape)
    dtype = st["qkv"].dtype
    st["q_out"][:n_tok] = rot[:, :H].to(dtype)
    where = st["table"].long()[seq, pos // page]
    st["k"][where, :, pos % page] = rot[:, H:].to(dtype)
    st["v"][where, :, pos % page] = x[:, H + G:].to(dtype)
    return st["q_out"], st["k"], st["v"]


def _plain_logprobs(st):
    c = st["case"]
    T, V, k = c["T"], c["V"], c["top"]
    x = st["logits"][:, :V].float()
    m = x.amax(-1, keepdim=True)
    e = torch.exp(x - m)
    z = e.sum(-1)
    log_z = torch.log(z) + m[:, 0]
    st["logp"].copy_(torch.gather(x, 1, st["targets"].long()[:, None])[:, 0] - log_z)
    st["entropy"].copy_(log_z - torch.where(e > 0, e * x, torch.zeros_like(x)).sum(-1) / z)
    if k:
        ids = torch.arange(V, device=_DEV, dtype=torch.int32)
        taken = torch.zeros_like(x, dtype=torch.bool)
        for j in range(k):  # the largest left, the lowest id among equals
            left = torch.where(taken, torch.full_like(x, float("-inf")), x)
            best = left.amax(-1, keepdim=True)
            at = torch.where((left == best) & ~taken, ids, torch.full_like(ids, V)).amin(-1)
            st["top_ids"][:, j] = at
            st["top_logp"][:, j] = best[:, 0] - log_z
            taken.scatter_(1, at.long()[:, None], True)
    return _logprob_outputs(st["logp"], st["entropy"], st["top_ids"], st["top_logp"])


_PLAIN = dict(packed=_plain_packed, decode=_plain_decode, write=_plain_write, logprobs=_plain_logprobs)


# ------------------------------------------------------------------- work ---

def work(case):
    """The bytes and operations that no implementation can do without."""
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "logprobs":
        T, V, k = case["T"], case["V"], case["top"]
        return dict(bytes=T * V * e + T * 12 + T * k * 8, flops=6 * T * V)
    H, G, D = case["H"], case["G"], case["D"]
    if case["op"] == "decode":
        lens = _ints(case["kv_lens"])
        entries = sum(_pages_of(lens, case["page"])) + len(lens)
        return dict(bytes=sum(lens) * 2 * G * D * e + 2 * len(lens) * H * D * e + 4 * entries,
                    flops=4 * D * H * sum(lens))
    q_lens, kv_lens, offsets = _batch(case)
    T = offsets[-1]
    tables = 4 * (sum(_pages_of(kv_lens, case["page"])) + 2 * len(q_lens) + 1)
    if case["op"] == "write":
        rows = set()
        for n, L in zip(q_lens, kv_lens):
            rows.update(range(L - n, L))
        return dict(bytes=2 * T * (H + 2 * G) * D * e + len(rows) * D * 4 + tables, flops=3 * T * (H + G) * D)
    pairs = sum(n * (L - n) + n * (n + 1) // 2 for n, L in zip(q_lens, kv_lens))
    seen = sum(L for n, L in zip(q_lens, kv_lens) if n)
    return dict(bytes=2 * T * H * D * e + seen * 2 * G * D * e + tables, flops=4 * D * H * pairs)


# ------------------------------------------------------------------ exact ---

def exact(case, seed):
    """The definitions in 64 bits, sequence by sequence and head by head."""
    st = prepare(case, seed)
    f64 = torch.float64
    if case["op"] == "logprobs":
        T, V, k = case["T"], case["V"], case["top"]
        logp, ent = torch.empty(T, dtype=f64, device=_DEV), torch.empty(T, dtype=f64, device=_DEV)
        ids = torch.empty((T, k), dtype=torch.int32, device=_DEV)
        top = torch.empty((T, k), dtype=f64, device=_DEV)
        for t0 in range(0, T, 256):
            x = st["logits"][t0:t0 + 256, :V].to(f64)
            lsm = x - torch.logsumexp(x, -1, keepdim=True)
            logp[t0:t0 + 256] = lsm.gather(1, st["targets"][t0:t0 + 256].long()[:, None])[:, 0]
            p = lsm.exp()
            ent[t0:t0 + 256] = -(p * lsm.clamp_min(-1e300)).sum(-1)
            if k:
                val, idx = torch.sort(lsm, dim=-1, descending=True, stable=True)
                idx = torch.sort(x, dim=-1, descending=True, stable=True).indices
                ids[t0:t0 + 256] = idx[:, :k].to(torch.int32)
                top[t0:t0 + 256] = val[:, :k]
        return (logp, ent) if not k else (logp, ent, ids, top)
    H, G, D, page = case["H"], case["G"], case["D"], case["page"]
    r = H // G
    if case["op"] == "write":
        q_out = st["q_out"].to(f64)
        k, v = st["k"].to(f64), st["v"].to(f64)
        q_lens, kv_lens, offsets = _batch(case)
        for i, (n, L) in enumerate(zip(q_lens, kv_lens)):
            if n == 0:
                continue
            pos = torch.arange(L - n, L, device=_DEV)
            freq = torch.tensor([_THETA ** (-2.0 * j / D) for j in range(D // 2)], dtype=f64, device=_DEV)
            turn = torch.polar(torch.ones((n, D // 2), dtype=f64, device=_DEV), pos.to(f64)[:, None] * freq)
            x = st["qkv"][offsets[i]:offsets[i] + n].to(f64).view(n, H + 2 * G, D)

            def rotate(u):
                if case["layout"] == "halves":
                    z = torch.complex(u[..., :D // 2].contiguous(), u[..., D // 2:].contiguous()) * turn[:, None]
                    return torch.cat([z.real, z.imag], dim=-1)
                z = torch.view_as_complex(u.reshape(n, -1, D // 2, 2).contiguous()) * turn[:, None]
                return torch.view_as_real(z).reshape(u.shape)

            q_out[offsets[i]:offsets[i] + n] = rotate(x[:, :H])
            where = st["table"][i].long()[pos // page]
            k[where, :, pos % page] = rotate(x[:, H:H + G])
            v[where, :, pos % page] = x[:, H + G:]
        return q_out, k, v
    if case["op"] == "decode":
        kv_lens = _ints(case["kv_lens"])
        q_lens, offsets = [1] * len(kv_lens), list(range(len(kv_lens) + 1))
    else:
        q_lens, kv_lens, offsets = _batch(case)
    o = torch.zeros(st["o"].shape, dtype=f64, device=_DEV)
    for i, (n, L) in enumerate(zip(q_lens, kv_lens)):
        if n == 0 or L == 0:
            continue
        pages = st["table"][i, :(L + page - 1) // page].long()
        for g in range(G):
            k = st["k"][pages, g].reshape(-1, D)[:L].to(f64)
            v = st["v"][pages, g].reshape(-1, D)[:L].to(f64)
            for s0 in range(0, n, 2048):
                s1 = min(n, s0 + 2048)
                end = L - n + s1
                future = torch.ones((s1 - s0, end), dtype=torch.bool, device=_DEV).triu(L - n + s0 + 1)
                for h in range(g * r, (g + 1) * r):
                    q = st["q"][offsets[i] + s0:offsets[i] + s1, h].to(f64)
                    logit = (q @ k[:end].T) / math.sqrt(D)
                    w = torch.softmax(logit.masked_fill(future, -math.inf), dim=-1)
                    o[offsets[i] + s0:offsets[i] + s1, h] = w @ v[:end]
    return o
