"""Cases, inputs and plain forms of the operators that serve drafted tokens from a cache held in 4 bits.

Five operators of include/llama_ops.h are measured here:

  write    llama_op_rope_kv4_write_paged       RoPE on packed tokens, keys and values stored into 4-bit cache pages;
           the new tokens' values are then read back as the pages hold them (llama_op_kv4_read_paged)
  read     llama_op_kv4_read_paged             keys and values of whole sequences back from their 4-bit pages
  packed   llama_op_attention_packed_kv4       causal grouped-query attention of packed tokens over the 4-bit pages
  decode   llama_op_attention_paged_decode_kv4 one new token per sequence over the 4-bit pages
  verify   llama_op_verify_drafts              drafted tokens kept or replaced, by the target's probabilities

`own` False: elementary torch operations in 32 bits (64 where a decision is taken).  `own` True: the library's entry
points.

A page holds, for each KV head, page_size rows of D / 2 bytes of codes and behind them page_size rows of D / 16 scale
bytes.  Eight elements of a row are four bytes: the low half of the 32-bit word holds the elements 0, 2, 4, 6 and the
high half 1, 3, 5, 7, four bits each, the lowest first.  A code n stands for (n - 8) * scale; a scale byte b, one for
16 elements, for 2^(b / 8 - 20) (1 + (b % 8) / 8), b / 8 rounded down.  A block is stored with the smallest scale that
is at least a seventh of its largest magnitude, and each value with the nearest code.
"""
import math

import torch

own = False

_DEV = "cuda"
_THETA = 500000.0


# ------------------------------------------------------------------ cases ---

def listed():
    lens64 = [4096 - 61 * ((i * 29) % 64) for i in range(64)]
    return [
        # Rotating and storing a whole prompt of the 8B-shaped block, three sequences of it at different points.
        _write("write_8b_prompt", "bf16", 32, 8, 128, 64, "6001,2100,91", "0,1000,4000", "interleaved", 0),
        # The same for one decode step of 24 users of the 135M-shaped model.
        _write("write_135m_step", "bf16", 9, 3, 64, 16, ",".join(["1"] * 24),
               ",".join(str((i * 37) % 1000) for i in range(24)), "halves", 8),
        # Long prefixes of the 8B-shaped block leave the 4-bit cache (moved to another server, or kept in bf16).
        _read("read_8b_prefixes", "bf16", 8, 128, 64, "30001,9000,777"),
        # A few short conversations of the 135M-shaped model, in fp32.
        _read("read_135m_f32", "f32", 3, 64, 16, "300,17,1,128"),
        # A whole 8192-token prompt of the 8B-shaped block: the largest pass.
        _packed("packed_8b_s8192", "bf16", 32, 8, 128, 64, "8192", "0", 0),
        # Verifying four drafted tokens for each of 64 users of the 8B-shaped block: five rows a sequence over its cache.
        _packed("packed_8b_drafts", "bf16", 32, 8, 128, 64, ",".join(["5"] * 64), ",".join(map(str, lens64)), 0),
        # The fp32 configuration over a few hundred tokens, padding rows behind them.
        _packed("packed_tiny_f32", "f32", 4, 2, 16, 16, "200,33,1,150", "0,7,300,0", 5),
        # A decode step of 64 users of the 8B-shaped block, each at a different point of its conversation.
        _decode("decode_8b_b64", "bf16", 32, 8, 128, 64, ",".join(map(str, lens64))),
        # One user with a very long document in the cache: work exists only along the cache's length.
        _decode("decode_8b_b1_long", "bf16", 32, 8, 128, 32, "120001"),
        # A few short conversations on the 135M-shaped model: pure latency.
        _decode("decode_135m_b8", "bf16", 9, 3, 64, 16, "300,17,1,128,1000,64,0,511"),
        # Four drafts for each of 64 users of the 8B-shaped stack, every fourth of them decoding greedily.
        _verify("verify_8b_b64", "f32", 128256, 128256, ",".join(["4"] * 64), "0,0.7,1,0.9", True),
        # Two users of the 135M-shaped stack, their drafts looked up in the prompt (no draft model): latency.
        _verify("verify_135m_lookup", "f32", 49152, 49152, "3,2", "1", False),
    ]


def _packed(name, dtype, H, G, D, page, q_lens, prefixes, pad):
    return dict(name=name, op="packed", dtype=dtype, H=H, G=G, D=D, page=page, q_lens=q_lens, prefixes=prefixes,
                pad=pad)


def _decode(name, dtype, H, G, D, page, kv_lens):
    return dict(name=name, op="decode", dtype=dtype, H=H, G=G, D=D, page=page, kv_lens=kv_lens)


def _write(name, dtype, H, G, D, page, q_lens, prefixes, layout, pad):
    return dict(name=name, op="write", dtype=dtype, H=H, G=G, D=D, page=page, q_lens=q_lens, prefixes=prefixes,
                layout=layout, pad=pad)


def _read(name, dtype, G, D, page, kv_lens):
    return dict(name=name, op="read", dtype=dtype, G=G, D=D, page=page, q_lens=kv_lens,
                prefixes=",".join("0" for _ in kv_lens.split(",")), pad=0)


def _verify(name, dtype, V, stride, drafts, temperatures, draft_model):
    return dict(name=name, op="verify", dtype=dtype, V=V, stride=stride, drafts=drafts, temperatures=temperatures,
                draft_model=draft_model)


def _ints(text):
    return [int(v) for v in text.split(",")]


def _log_int(rng, lo, hi):
    """A whole number in [lo, hi], its logarithm spread evenly."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.999)))))))


def _draw_heads(rng):
    """(dtype, H, G, D): mostly bf16 with head widths of 64 and 128, the small widths and fp32 among them."""
    dtype = "f32" if rng.random() < 0.2 else "bf16"
    D = rng.choice([64, 128]) if rng.random() < 0.8 else rng.choice([16, 32])
    G = rng.choice([1, 2, 3, 4, 8])
    r = rng.choice([1, 2, 3, 4, 5, 6, 7, 8, 12, 16] if G <= 4 else [1, 2, 3, 4, 5, 8])
    return dtype, G * r, G, D


def draw(rng):
    op = rng.choice(["packed", "packed", "drafts", "decode", "decode", "write", "read", "verify", "verify"])
    page = rng.choice([16, 32, 64, 128, 256])
    if op == "verify":
        V = _log_int(rng, 1000, 160000)
        n = _log_int(rng, 1, max(1, min(256, 7_000_000 // V)))
        most = rng.choice([1, 3, 4, 5, 8])
        drafts = [most if i == 0 else rng.randint(0, most) for i in range(n)]
        stride = V if rng.random() < 0.5 else (V + 63) // 64 * 64
        temps = rng.choice(["1", "0", "0.8", "0,1,0.6,1.3", "0.5,1"])
        return _verify("", rng.choice(["f32", "bf16"]), V, stride, ",".join(map(str, drafts)), temps,
                       rng.random() < 0.75)
    dtype, H, G, D = _draw_heads(rng)
    small = dtype == "f32" or D < 64
    n = _log_int(rng, 1, 48)
    if op == "read":
        longest = _log_int(rng, 16, 30000)
        longest = min(longest, max(16, 40_000_000 // (n * G * D)))
        return _read("", dtype, G, D, page, ",".join(str(longest if i == 0 else rng.randint(0, longest)) for i in range(n)))
    if op in ("decode", "drafts"):
        longest = _log_int(rng, 16, 200_000 if n <= 4 and op == "decode" else 8192)
        if small:
            longest = min(longest, 8192 if op == "decode" else 1024)
        longest = min(longest, max(16, 240_000_000 // (n * 2 * G * D)))
        lens = [longest if i == 0 else rng.randint(0, longest) for i in range(n)]
        if op == "decode":
            return _decode("", dtype, H, G, D, page, ",".join(map(str, lens)))
        most = rng.choice([2, 3, 5, 6, 9])  # the last confirmed token and its drafts
        q_lens = [most if i == 0 else rng.randint(1, most) for i in range(n)]
        return _packed("", dtype, H, G, D, page, ",".join(map(str, q_lens)), ",".join(map(str, lens)), 0)
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


# ----------------------------------------------------------- 4-bit blocks ---

_AT = [0, 4, 1, 5, 2, 6, 3, 7]      # where element e of eight lies among the nibbles of its word
_ELEMENT = [0, 2, 4, 6, 1, 3, 5, 7]  # the element that a word's nibble holds


def _scale_of(byte):
    """fp32 scales of scale bytes: the byte is the exponent (from -20) and three bits of mantissa."""
    return ((byte.to(torch.int32) + ((127 - 20) << 3)) << 20).view(torch.float32)


def _quantise(x):
    """(codes, scale bytes) of fp32 [..., D]: codes uint8 [..., D / 2], scales uint8 [..., D / 16]."""
    D = x.shape[-1]
    b = x.reshape(*x.shape[:-1], D // 16, 16)
    most = b.abs().amax(-1)
    least = most / torch.full_like(most, 7.0)  # (a number in its place would be multiplied by as 1/7, rounded)
    byte = (((least.view(torch.int32) + 0xFFFFF) >> 20) - ((127 - 20) << 3)).clamp(0, 255)
    n = torch.round(b / _scale_of(byte)[..., None]).clamp(-7, 7).to(torch.int32) + 8
    n = n.reshape(*x.shape[:-1], D // 8, 8)[..., _ELEMENT].reshape(*x.shape[:-1], D // 2, 2)
    return (n[..., 0] | n[..., 1] << 4).to(torch.uint8), byte.to(torch.uint8)


def _values(codes, scales):
    """fp32 [..., D] that codes [..., D / 2] and scale bytes [..., D / 16] stand for."""
    D = codes.shape[-1] * 2
    n = torch.stack([codes & 15, codes >> 4], dim=-1).reshape(*codes.shape[:-1], D // 8, 8)[..., _AT]
    v = n.reshape(*codes.shape[:-1], D // 16, 16).float() - 8.0
    return (v * _scale_of(scales)[..., None]).reshape(*codes.shape[:-1], D)


def _split_pool(pool, page, D):
    """Views of a pool uint8 [n][G][page * (D / 2 + D / 16)]: codes [n][G][page][D / 2], scales [n][G][page][D / 16]."""
    n, G, _ = pool.shape
    at = page * D // 2
    return pool[..., :at].unflatten(-1, (page, D // 2)), pool[..., at:].unflatten(-1, (page, D // 16))


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


def _pool(gen, n_pages, G, page, D):
    """Pages of keys or values as a model leaves them: some columns of a head an order larger than the rest."""
    pool = torch.empty((n_pages, G, page * (D // 2 + D // 16)), dtype=torch.uint8, device=_DEV)
    codes, scales = _split_pool(pool, page, D)
    size = torch.exp(0.8 * torch.randn((G, 1, D), device=_DEV, generator=gen))
    step = max(1, (1 << 26) // (G * page * D))
    for i in range(0, n_pages, step):
        n = min(step, n_pages - i)
        x = torch.randn((n, G, page, D), device=_DEV, generator=gen) * size
        codes[i:i + n], scales[i:i + n] = _quantise(x)
    return pool


def _cache(gen, case, kv_lens):
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
    args = (gen, n_pages, case["G"], case["page"], case["D"])
    return _pool(*args), _pool(*args), table


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


def _verify_state(gen, case):
    """Target and draft logits that agree as a good draft model's do, drafts drawn from the draft's distribution."""
    dtype, V, stride, drafts = _torch_dtype(case), case["V"], case["stride"], _ints(case["drafts"])
    n, most = len(drafts), max(max(drafts), 1)
    offsets = [0]
    for d in drafts:
        offsets.append(offsets[-1] + d + 1)
    rows, n_drafts = offsets[-1], sum(drafts)
    target = _normal(gen, (rows, stride), dtype, std=2.5)
    likely = torch.randint(0, V, (rows, 4), device=_DEV, generator=gen)
    boost = 9.0 + 7.0 * torch.rand((rows, 4), device=_DEV, generator=gen)
    target.scatter_(1, likely, boost.to(dtype))
    banned = torch.randint(0, V, (7,), device=_DEV, generator=gen)  # tokens a server never lets through
    target[:, banned] = float("-inf")
    off = torch.tensor(offsets, dtype=torch.int64, device=_DEV)
    row = torch.arange(rows, device=_DEV)
    seq = torch.searchsorted(off[1:], row, right=True)
    has_draft = row + 1 < off[seq + 1]
    drow = row[has_draft]
    dseq = seq[drow]
    step = drow - off[dseq]
    draft = _normal(gen, (n, most, stride), dtype, std=0.7)  # a step of the draft model for all of its sequences each
    draft[dseq, step] += target[drow]
    temps = [float(t) for t in case["temperatures"].split(",")]
    temps = torch.tensor([temps[i % len(temps)] for i in range(n)], device=_DEV)
    tokens = torch.randint(0, V, (rows,), device=_DEV, generator=gen, dtype=torch.int32)
    if n_drafts:
        z = draft[dseq, step, :V].float() / temps[dseq].clamp_min(0.05)[:, None]
        noise = torch.empty((n_drafts, V), device=_DEV).exponential_(generator=gen)
        picked = (z - torch.log(noise)).argmax(-1)
        if not case["draft_model"]:  # looked up: the likeliest token most of the time
            picked = torch.where(torch.rand(n_drafts, device=_DEV, generator=gen) < 0.7,
                                 target[drow, :V].float().argmax(-1), picked)
        tokens[drow + 1] = picked.to(torch.int32)
    target[:, V:] = float("nan")  # the padding of a row is never a logit
    draft[..., V:] = float("nan")
    # fp32 uniforms of 24 bits, and exponential variates above 0
    uniforms = torch.rand((n, most), device=_DEV, generator=gen)
    noise = torch.empty((n, V), device=_DEV).exponential_(generator=gen).clamp_min(1e-30)
    return dict(target=target, draft=draft if case["draft_model"] else None, tokens=tokens, temps=temps,
                uniforms=uniforms, noise=noise, offsets=off.to(torch.int32), most=most, n_drafts=n_drafts,
                out=torch.zeros((n, most + 1), dtype=torch.int32, device=_DEV),
                accepted=torch.zeros(n, dtype=torch.int32, device=_DEV),
                logp=torch.zeros((n, most + 1), device=_DEV))


def prepare(case, seed):
    gen = torch.Generator(device=_DEV)
    gen.manual_seed(seed)
    dtype = _torch_dtype(case)
    st = dict(case=case)
    if case["op"] == "verify":
        st.update(_verify_state(gen, case))
    elif case["op"] == "decode":
        H, D = case["H"], case["D"]
        kv_lens = _ints(case["kv_lens"])
        k, v, table = _cache(gen, case, kv_lens)
        n = len(kv_lens)
        st.update(q=_normal(gen, (n, H, D), dtype), k=k, v=v, table=table,
                  kv_lens=torch.tensor(kv_lens, dtype=torch.int32, device=_DEV), max_kv=max(kv_lens),
                  o=torch.zeros((n, H, D), dtype=dtype, device=_DEV))
    else:
        G, D = case["G"], case["D"]
        q_lens, kv_lens, offsets = _batch(case)
        k, v, table = _cache(gen, case, kv_lens)
        T = offsets[-1] + case["pad"]
        st.update(k=k, v=v, table=table, T=T, offsets=torch.tensor(offsets, dtype=torch.int32, device=_DEV),
                  kv_lens=torch.tensor(kv_lens, dtype=torch.int32, device=_DEV), max_kv=max(kv_lens))
        if case["op"] in ("write", "read"):
            st.update(k_out=torch.zeros((T, G, D), dtype=dtype, device=_DEV),
                      v_out=torch.zeros((T, G, D), dtype=dtype, device=_DEV))
        if case["op"] == "packed":
            H = case["H"]
            st.update(q=_normal(gen, (T, H, D), dtype), o=torch.zeros((T, H, D), dtype=dtype, device=_DEV))
        if case["op"] == "write":
            H = case["H"]
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
    need = 0
    if case["op"] == "verify":
        st["batch"] = lb.make_draft_batch(st["offsets"], st["tokens"], st["target"].shape[0], st["most"], st["temps"],
                                          st["uniforms"], st["noise"])
        need = lb.llama_op_verify_drafts_workspace_bytes(st["batch"], case["V"])
    else:
        st["kv"] = lb.make_paged_kv4_cache(st["k"], st["v"], st["table"], case["page"])
        if case["op"] == "decode":
            need = lb.llama_op_attention_paged_decode_kv4_workspace_bytes(code, len(st["kv_lens"]), st["max_kv"],
                                                                          case["H"], case["G"], case["D"])
        else:
            st["batch"] = lb.make_packed_batch(st["offsets"], st["kv_lens"], st["T"], st["max_kv"])
            if case["op"] == "packed":
                need = lb.llama_op_attention_packed_kv4_workspace_bytes(code, st["batch"], case["H"], case["G"],
                                                                        case["D"])
    st["ws"] = torch.empty(max(need, 16), dtype=torch.uint8, device=_DEV)


# -------------------------------------------------------------------- run ---

def run(st):
    return _run_own(st) if own else _PLAIN[st["case"]["op"]](st)


def _run_own(st):
    import decoder_block_gb300 as lb
    c = st["case"]
    stream = torch.cuda.current_stream()
    if c["op"] == "packed":
        lb.check(lb.llama_op_attention_packed_kv4(st["code"], st["q"], st["kv"], st["batch"], st["o"], c["H"], c["G"],
                                                  c["D"], st["ws"], st["ws"].numel(), None, stream))
        return st["o"]
    if c["op"] == "decode":
        lb.check(lb.llama_op_attention_paged_decode_kv4(st["code"], st["q"], st["kv"], st["kv_lens"],
                                                        len(st["kv_lens"]), st["max_kv"], st["o"], c["H"], c["G"],
                                                        c["D"], st["ws"], st["ws"].numel(), None, stream))
        return st["o"]
    if c["op"] == "verify":
        lb.check(lb.llama_op_verify_drafts(st["code"], st["target"], c["stride"], st["draft"], st["most"] * c["stride"],
                                           c["stride"], c["V"], st["batch"], st["out"], st["accepted"], st["logp"],
                                           st["ws"], st["ws"].numel(), None, stream))
        return st["out"], st["accepted"], st["logp"]
    if c["op"] == "write":
        layout = lb.LLAMA_ROPE_HALVES if c["layout"] == "halves" else lb.LLAMA_ROPE_INTERLEAVED
        lb.check(lb.llama_op_rope_kv4_write_paged(st["code"], st["qkv"], st["q_out"], st["kv"], st["batch"], st["rope"],
                                                  st["rope"].shape[0], c["H"], c["G"], c["D"], layout, None, stream))
    lb.check(lb.llama_op_kv4_read_paged(st["code"], st["kv"], st["batch"], st["k_out"], st["v_out"], c["G"], c["D"],
                                        None, stream))
    return (st["q_out"], st["k_out"], st["v_out"]) if c["op"] == "write" else (st["k_out"], st["v_out"])


def _gather(pool, pages, L, page, D):
    """[G][L][D] fp32 of one sequence's pages."""
    codes, scales = _split_pool(pool[pages.long()], page, D)
    x = _values(codes, scales)                  # [n][G][page][D]
    return x.permute(1, 0, 2, 3).reshape(pool.shape[1], -1, D)[:, :L]


def _plain_packed(st):
    c = st["case"]
    H, G, D, page = c["H"], c["G"], c["D"], c["page"]
    q_lens, kv_lens, offsets = _batch(c)
    counts = _pages_of(kv_lens, page)
    o = st["o"]
    for i, (n, L) in enumerate(zip(q_lens, kv_lens)):
        if n == 0:
            continue
        k = _gather(st["k"], st["table"][i, :counts[i]], L, page, D)
        v = _gather(st["v"], st["table"][i, :counts[i]], L, page, D)
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
    H, G, D, page = c["H"], c["G"], c["D"], c["page"]
    lens, table, o = st["kv_lens"], st["table"], st["o"]
    n, L = len(lens), table.shape[1] * page
    keys = torch.arange(L, device=_DEV)
    step = max(1, (1 << 29) // (G * L * D))

    def rows(pool, b0, b1):
        codes, scales = _split_pool(pool[table[b0:b1].reshape(-1).long()], page, D)
        x = _values(codes, scales).view(b1 - b0, -1, G, page, D)
        return x.permute(0, 2, 1, 3, 4).reshape(b1 - b0, G, L, D)

    for b0 in range(0, n, step):
        b1 = min(n, b0 + step)
        q = st["q"][b0:b1].float().view(b1 - b0, G, H // G, D)
        s = torch.matmul(q, rows(st["k"], b0, b1).transpose(2, 3)) * (1.0 / math.sqrt(D))
        visible = keys[None, :] < lens[b0:b1, None].long()
        s = torch.where(visible[:, None, None, :], s, torch.full_like(s, -3.0e38))
        p = torch.exp(s - s.amax(-1, keepdim=True)) * visible[:, None, None, :]
        z = p.sum(-1, keepdim=True)
        p = p / torch.where(z > 0, z, torch.ones_like(z))
        o[b0:b1] = torch.matmul(p, rows(st["v"], b0, b1)).view(b1 - b0, H, D).to(o.dtype)
    return o


def _where(st, n_tok):
    """Page and row of each token's position, and the position."""
    tok = torch.arange(n_tok, device=_DEV)
    off = st["offsets"].long()
    seq = torch.searchsorted(off[1:], tok, right=True)
    pos = st["kv_lens"].long()[seq] - (off[seq + 1] - tok)
    page = st["case"]["page"]
    return st["table"].long()[seq, pos // page], pos % page, pos


def _plain_read(st):
    c = st["case"]
    n_tok = int(_batch(c)[2][-1])
    if n_tok:
        page, slot, _ = _where(st, n_tok)
        for out, pool in (("k_out", st["k"]), ("v_out", st["v"])):
            codes, scales = _split_pool(pool, c["page"], c["D"])
            st[out][:n_tok] = _values(codes[page, :, slot], scales[page, :, slot]).to(st[out].dtype)
    return st["k_out"], st["v_out"]


def _plain_write(st):
    c = st["case"]
    H, G, D = c["H"], c["G"], c["D"]
    n_tok = int(_batch(c)[2][-1])
    if n_tok:
        page, slot, pos = _where(st, n_tok)
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
        st["q_out"][:n_tok] = rot[:, :H].to(st["qkv"].dtype)
        for pool, new in ((st["k"], rot[:, H:]), (st["v"], x[:, H + G:])):
            codes, scales = _split_pool(pool, c["page"], D)
            codes[page, :, slot], scales[page, :, slot] = _quantise(new)
    return (st["q_out"],) + _plain_read(st)


def _first(x, best):
    """The lowest index of each row's entries that equal `best`."""
    ids = torch.arange(x.shape[1], device=_DEV, dtype=torch.int32)
    return torch.where(x == best, ids, torch.full_like(ids, x.shape[1])).amin(-1)


def _plain_verify(st):
    c = st["case"]
    V, most, n_drafts = c["V"], st["most"], st["n_drafts"]
    off = st["offsets"].long()
    n, rows = off.shape[0] - 1, st["target"].shape[0]
    row = torch.arange(rows, device=_DEV)
    seq = torch.searchsorted(off[1:], row, right=True)
    greedy = st["temps"] == 0
    temp = torch.where(greedy, torch.ones_like(st["temps"]), st["temps"])

    def softmax_parts(logits, temps):
        x = logits[:, :V].float()
        m = x.amax(-1, keepdim=True)
        e = torch.exp((x - m) / temps[:, None])
        return x, m[:, 0], e, e.sum(-1, dtype=torch.float64)

    x, m, e, z = softmax_parts(st["target"], temp[seq])
    best = _first(x, m[:, None])
    keep = torch.zeros((n, most + 1), dtype=torch.bool, device=_DEV)
    if n_drafts:
        drow = row[row + 1 < off[seq + 1]]
        dseq = seq[drow]
        step = drow - off[dseq]
        drafted = st["tokens"][drow + 1].long()

        def log_p(x, m, z, at, t):
            return (x.gather(1, at[:, None])[:, 0].double() - m.double()) / t.double() - z.log()

        ratio = log_p(x[drow], m[drow], z[drow], drafted, temp[dseq])
        if st["draft"] is not None:
            xd, md, ed, zd = softmax_parts(st["draft"][dseq, step], temp[dseq])
            ratio = ratio - log_p(xd, md, zd, drafted, temp[dseq])
        ok = torch.where(greedy[dseq], best[drow].long() == drafted, st["uniforms"][dseq, step].double() < ratio.exp())
        keep[dseq, step] = ok
    accepted = keep.long().cumprod(-1).sum(-1)
    last = off[:-1] + accepted                   # the row that the next token is drawn from
    p = e[last] / z[last, None].float()
    w = p
    if n_drafts:
        refused = last + 1 < off[1:]             # a draft was not kept: what it would have been drawn from goes
        d = (last - torch.arange(n, device=_DEV)).clamp_max(n_drafts - 1)  # its place among all drafts
        if st["draft"] is not None:
            q = ed[d] / zd[d, None].float()
        else:
            q = torch.zeros_like(p).scatter_(1, drafted[d][:, None], 2.0)
        w = torch.where(refused[:, None], (p - q).clamp_min(0.0), p)
        w = torch.where((w > 0).any(-1, keepdim=True), w, p)
    score = w / st["noise"]
    drawn = torch.where(greedy, best[last], _first(score, score.amax(-1, keepdim=True)))
    slot = torch.arange(most + 1, device=_DEV)
    at = (off[:-1, None] + 1 + slot).clamp_max(rows - 1)
    out = torch.where(slot < accepted[:, None], st["tokens"][at], torch.full_like(st["out"], -1))
    out.scatter_(1, accepted[:, None], drawn[:, None].to(torch.int32))
    here = (off[:-1, None] + slot).clamp_max(rows - 1)
    lp = (x[here, out.long().clamp_min(0)] - m[here]) / temp[:, None] - z.log()[here].float()
    st["out"].copy_(out)
    st["accepted"].copy_(accepted)
    st["logp"].copy_(torch.where(out >= 0, lp, torch.zeros_like(lp)))
    return st["out"], st["accepted"], st["logp"]


_PLAIN = dict(packed=_plain_packed, decode=_plain_decode, write=_plain_write, read=_plain_read, verify=_plain_verify)


# ------------------------------------------------------------------- work ---

def work(case):
    """The bytes and operations that no implementation can do without."""
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "verify":
        V, drafts = case["V"], _ints(case["drafts"])
        temps = [float(t) for t in case["temperatures"].split(",")]
        n, rows = len(drafts), sum(drafts) + len(drafts)
        drawn = sum(temps[i % len(temps)] > 0 for i in range(n))
        read = rows
        if case["draft_model"]:
            read += sum(d for i, d in enumerate(drafts) if temps[i % len(temps)] > 0)
        return dict(bytes=read * V * e + drawn * V * 4 + rows * 12 + n * (max(max(drafts), 1) + 1) * 8,
                    flops=4 * read * V + 4 * drawn * V)
    G, D = case["G"], case["D"]
    held = D // 2 + D // 16  # bytes of a head's row
    if case["op"] == "decode":
        H, lens = case["H"], _ints(case["kv_lens"])
        entries = sum(_pages_of(lens, case["page"])) + len(lens)
        return dict(bytes=sum(lens) * 2 * G * held + 2 * len(lens) * H * D * e + 4 * entries,
                    flops=4 * D * H * sum(lens))
    q_lens, kv_lens, offsets = _batch(case)
    T = offsets[-1]
    tables = 4 * (sum(_pages_of(kv_lens, case["page"])) + 2 * len(q_lens) + 1)
    if case["op"] == "read":
        return dict(bytes=T * 2 * G * (held + D * e) + tables, flops=2 * T * 2 * G * D)
    H = case["H"]
    if case["op"] == "write":  # and the read that follows it
        rows = set()
        for n, L in zip(q_lens, kv_lens):
            rows.update(range(L - n, L))
        return dict(bytes=T * (2 * H + 2 * G) * D * e + T * 2 * G * held + len(rows) * D * 4 + tables
                    + T * 2 * G * (held + D * e), flops=3 * T * (H + G) * D + 5 * T * 2 * G * D)
    pairs = sum(n * (L - n) + n * (n + 1) // 2 for n, L in zip(q_lens, kv_lens))
    seen = sum(L for n, L in zip(q_lens, kv_lens) if n)
    return dict(bytes=2 * T * H * D * e + seen * 2 * G * held + tables, flops=4 * D * H * pairs)


# ------------------------------------------------------------------ exact ---

def _exact_rows(st, which, i, L, g=slice(None)):
    """[L][G][D] fp64 that sequence i's pages hold, nibble by nibble."""
    c = st["case"]
    page, D = c["page"], c["D"]
    pool = st[which][st["table"][i, :(L + page - 1) // page].long()][:, g].to(torch.int64)
    n = pool.shape[0]
    word = pool[..., :page * D // 2].reshape(n, -1, page, D // 8, 4)
    word = word[..., 0] + (word[..., 1] << 8) + (word[..., 2] << 16) + (word[..., 3] << 24)
    shift = torch.tensor([4 * (e // 2) + 16 * (e % 2) for e in range(8)], device=_DEV)
    code = ((word[..., None] >> shift) & 15).reshape(n, -1, page, D // 16, 16)
    byte = pool[..., page * D // 2:].reshape(n, -1, page, D // 16, 1)
    scale = torch.exp2((byte // 8 - 20).double()) * (1.0 + (byte % 8).double() / 8.0)
    x = ((code - 8).double() * scale).reshape(n, -1, page, D)
    return x.transpose(1, 2).reshape(n * page, -1, D)[:L]


def _exact_held(x):
    """What fp64 [..., D] stands for once it is held in 4 bits."""
    b = x.reshape(*x.shape[:-1], -1, 16)
    steps = torch.arange(256, device=_DEV, dtype=torch.float64)
    scales = torch.exp2(torch.floor(steps / 8) - 20) * (1 + (steps % 8) / 8)
    at = torch.searchsorted(scales, (b.abs().amax(-1) / 7).contiguous()).clamp_max(255)
    s = scales[at][..., None]
    return (torch.round(b / s).clamp(-7, 7) * s).reshape(x.shape)


def _exact_verify(case, st):
    V, f64 = case["V"], torch.float64
    off, drafts = st["offsets"].tolist(), _ints(case["drafts"])
    out, acc = torch.full_like(st["out"], -1), torch.zeros_like(st["accepted"])
    logp = torch.zeros_like(st["logp"], dtype=f64)
    tokens, uniforms, temps = st["tokens"].tolist(), st["uniforms"].tolist(), st["temps"].double().tolist()
    for i, n in enumerate(drafts):
        t = temps[i] or 1.0
        x = st["target"][off[i]:off[i + 1], :V].to(f64)
        lp = torch.log_softmax(x / t, -1)
        lq = torch.log_softmax(st["draft"][i, :n, :V].to(f64) / t, -1) if case["draft_model"] else None
        top = torch.sort(x, dim=-1, descending=True, stable=True).indices[:, 0].tolist()
        j = 0
        while j < n:
            tok = tokens[off[i] + 1 + j]
            if temps[i] == 0:
                kept = top[j] == tok
            else:
                q = float(lq[j, tok]) if lq is not None else 0.0
                kept = uniforms[i][j] < math.exp(float(lp[j, tok]) - q)
            if not kept:
                break
            out[i, j] = tok
            logp[i, j] = lp[j, tok]
            j += 1
        acc[i] = j
        if temps[i] == 0:
            tok = top[j]
        else:
            w = lp[j].exp()
            if j < n and lq is not None:
                w = (w - lq[j].exp()).clamp_min(0)
            elif j < n:
                w[tokens[off[i] + 1 + j]] = 0
            score = w / st["noise"][i].to(f64)
            tok = int(torch.sort(score, descending=True, stable=True).indices[0])
        out[i, j] = tok
        logp[i, j] = lp[j, tok]
    return out, acc, logp


def exact(case, seed):
    """The definitions in 64 bits, sequence by sequence and head by head."""
    st = prepare(case, seed)
    f64 = torch.float64
    if case["op"] == "verify":
        return _exact_verify(case, st)
    G, D = case["G"], case["D"]
    if case["op"] == "decode":
        kv_lens = _ints(case["kv_lens"])
        q_lens, offsets = [1] * len(kv_lens), list(range(len(kv_lens) + 1))
    else:
        q_lens, kv_lens, offsets = _batch(case)
    if case["op"] in ("write", "read"):
        k, v = st["k_out"].to(f64), st["v_out"].to(f64)
        q_out = st["q_out"].to(f64) if case["op"] == "write" else None
        for i, (n, L) in enumerate(zip(q_lens, kv_lens)):
            if n == 0:
                continue
            at = slice(offsets[i], offsets[i] + n)
            if case["op"] == "read":
                k[at], v[at] = _exact_rows(st, "k", i, L)[L - n:], _exact_rows(st, "v", i, L)[L - n:]
                continue
            H = case["H"]
            turn = torch.view_as_complex(st["rope"][L - n:L].to(f64))[:, None]  # the table is an input
            x = st["qkv"][at].to(f64).view(n, H + 2 * G, D)

            def rotate(u):
                if case["layout"] == "halves":
                    z = torch.complex(u[..., :D // 2].contiguous(), u[..., D // 2:].contiguous()) * turn
                    return torch.cat([z.real, z.imag], dim=-1)
                z = torch.view_as_complex(u.reshape(n, -1, D // 2, 2).contiguous()) * turn
                return torch.view_as_real(z).reshape(u.shape)

            q_out[at] = rotate(x[:, :H])
            k[at] = _exact_held(rotate(x[:, H:H + G]))
            v[at] = _exact_held(x[:, H + G:])
        return (q_out, k, v) if case["op"] == "write" else (k, v)
    r = case["H"] // G
    o = torch.zeros(st["o"].shape, dtype=f64, device=_DEV)
    for i, (n, L) in enumerate(zip(q_lens, kv_lens)):
        if n == 0 or L == 0:
            continue
        for g in range(G):
            k = _exact_rows(st, "k", i, L, slice(g, g + 1))[:, 0]
            v = _exact_rows(st, "v", i, L, slice(g, g + 1))[:, 0]
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
