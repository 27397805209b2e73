"""Cases, plain forms and exact values of the decoder-block operators that stand next
to the MoE path: int4 group-64 projections, the quantised KV cache (written, read
back) and decode attention over it for sequences that share a prefix.

Sizes follow this repository's configurations (d = 2048 and 1536, 64 and 256
sequences, a 3,100-token prompt, prompts of up to 8192 tokens) or are generic
(64/128/256-wide heads, vocabulary-sized outputs).
"""
import math

import torch

own = False

GROUP = 64


# ------------------------------------------------------------------ cases ----
def listed():
    return [
        # one token through a d x d projection: launch latency counts
        dict(name="q4_one_token_square", op="q4", B=1, n_in=2048, n_out=2048),
        # one token through a vocabulary-sized output projection of odd size
        dict(name="q4_one_token_vocabulary", op="q4", B=1, n_in=2048, n_out=65537),
        # a few sequences decoded together, fused query/key/value projection
        dict(name="q4_seven_tokens", op="q4", B=7, n_in=2048, n_out=5120),
        # the 64-sequence batch, a wide projection
        dict(name="q4_64_tokens", op="q4", B=64, n_in=1536, n_out=6144),
        # one decode step's keys and values of 64 sequences, cut from a fused projection
        dict(name="kv_step_64", op="kv", bits=4, Hkv=8, D=128, page=64, B=64, lo=1, hi=1, at=300, fused=True),
        # three prompts written at once, 8-bit codes
        dict(name="kv_prompts_8192", op="kv", bits=8, Hkv=8, D=128, page=64, B=3, lo=1000, hi=4800, at=0, fused=False),
        # short ragged pieces read back, small heads
        dict(name="read_ragged", op="read", bits=8, Hkv=4, D=64, page=16, B=13, lo=0, hi=70, at=0),
        # a long context read back in whole
        dict(name="read_long", op="read", bits=4, Hkv=8, D=128, page=64, B=2, lo=30001, hi=33000, at=17),
        # one sequence, no shared prefix, wide heads: latency of a short context
        dict(name="attn_one_sequence", op="attn", bits=8, Hq=16, Hkv=2, D=256, page=64, B=1, lo=777, hi=777, prefix=0,
             fused=True),
        # 64 sequences behind the 3,100-token prompt, ragged own contexts
        dict(name="attn_64_prompt_3100", op="attn", bits=4, Hq=32, Hkv=8, D=128, page=64, B=64, lo=0, hi=512,
             prefix=3100, fused=True),
        # 256 sequences behind a prompt of 8191 tokens
        dict(name="attn_256_prompt_8191", op="attn", bits=4, Hq=16, Hkv=2, D=128, page=64, B=256, lo=1, hi=1024,
             prefix=8191, fused=False),
        # four long contexts that share nothing
        dict(name="attn_long", op="attn", bits=4, Hq=32, Hkv=8, D=128, page=128, B=4, lo=100003, hi=131072, prefix=0,
             fused=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["q4", "q4", "kv", "read", "attn", "attn"])
    if op == "q4":
        n_in = GROUP * _log(rng, 8, 64)
        B = _log(rng, 1, 256)
        return dict(op=op, B=B, n_in=n_in, n_out=_log(rng, 100, min(65537, 600_000_000 // (n_in * B))))
    bits, D = rng.choice([4, 8]), rng.choice([64, 128, 256])
    Hkv, page = rng.choice([1, 2, 3, 4, 8]), 16 * rng.choice([1, 2, 3, 4, 8])
    if op == "kv":
        B = _log(rng, 1, 64)
        hi = _log(rng, 1, max(2, 8192 // B))
        return dict(op=op, bits=bits, Hkv=Hkv, D=D, page=page, B=B, lo=rng.randint(0, 1), hi=hi, at=rng.randint(0, 500),
                    fused=rng.random() < 0.5)
    if op == "read":
        B = _log(rng, 1, 64)
        hi = _log(rng, 2, max(3, 30000 // B))
        return dict(op=op, bits=bits, Hkv=Hkv, D=D, page=page, B=B, lo=rng.randint(0, 1), hi=hi, at=rng.randint(0, 100))
    B = _log(rng, 1, 256)
    Hq = Hkv * rng.choice([1, 2, 4, 5, 8, 16])
    prefix = rng.choice([0, _log(rng, 1, min(8192, max(2, 17_000_000_000 // (4 * B * Hq * D))))])
    hi = _log(rng, 1, max(2, min(65536, 1_800_000_000 // (Hkv * D * bits * B))))
    return dict(op=op, bits=bits, Hq=Hq, Hkv=Hkv, D=D, page=page, B=B, lo=min(hi, rng.randint(0, 1)), hi=hi,
                prefix=prefix, fused=rng.random() < 0.5)


def _counts(case):
    """Tokens of each sequence: spread over [lo, hi], both ends among them."""
    B, lo, hi = case["B"], case["lo"], case["hi"]
    if B == 1:
        return [hi]
    spread = [lo + int((hi - lo) * ((i * 0.6180339887498949) % 1.0)) for i in range(B)]
    spread[B // 2] = hi
    spread[0] = lo
    return spread


def _token_bytes(case):
    return 2 * case["Hkv"] * (case["D"] * case["bits"] // 8 + case["D"] // GROUP * 4)


def work(case):
    if case["op"] == "q4":
        B, n_in, n_out = case["B"], case["n_in"], case["n_out"]
        return dict(bytes=n_out * n_in // 2 + n_out * (n_in // GROUP) * 4 + 2 * B * (n_in + n_out),
                    flops=2 * B * n_in * n_out)
    T = sum(_counts(case))
    values = T * case["Hkv"] * case["D"] * 2
    if case["op"] == "kv":      # K and V in, the pages' bytes and the values they stand for out
        return dict(bytes=2 * 2 * values + T * _token_bytes(case), flops=12 * values)
    if case["op"] == "read":
        return dict(bytes=2 * values + T * _token_bytes(case), flops=2 * values)
    rows = case["B"] * case["Hq"] * case["D"]
    return dict(bytes=(case["prefix"] + T) * _token_bytes(case) + 2 * 2 * rows,
                flops=4 * case["Hq"] * case["D"] * (case["B"] * case["prefix"] + T))


# ----------------------------------------------------- the cache's pages ----
# A page holds [kv head][strip of 16 tokens]; a strip K codes, K (s, b), V codes,
# V (s, b).  The 16-byte pieces of a token's codes are stored exclusive-ored with
# a number that goes by the token's row in the strip.
def _row_bytes(bits, D):
    return D * bits // 8


def _strip_bytes(bits, D):
    return 2 * 16 * (_row_bytes(bits, D) + D // GROUP * 4)


def _turn(bits, D, device):
    """[16, pieces]: the stored place of each 16-byte piece of a token's codes."""
    R = _row_bytes(bits, D)
    row = torch.arange(16, device=device)
    x = row % 8 if R >= 128 else (row * R // 128) % (R // 16)
    return torch.arange(R // 16, device=device)[None, :] ^ x[:, None]


def _quantise(x, bits, wide):
    """Codes (uint8), s and b (fp16) of x [..., D]; `wide` is the type of the arithmetic."""
    top = 2 ** bits - 1
    g = x.unflatten(-1, (-1, GROUP)).to(wide)
    mn, mx = g.amin(-1), g.amax(-1)
    s = ((mx - mn).float() / top).half()
    d = torch.where(s == 0, torch.ones_like(s), s).to(wide)
    q = torch.round((g - mn[..., None]) / d[..., None]).clamp(0, top)
    q = torch.where((s == 0)[..., None], torch.zeros_like(q), q)
    return q.to(torch.uint8).flatten(-2), s, mn.half()


def _row_image(codes, s, b, bits):
    """Stored bytes of tokens: codes [..., D] -> [..., R], (s, b) -> [..., D/64 * 4]."""
    if bits == 4:
        codes = codes[..., 0::2] | (codes[..., 1::2] << 4)
    return codes, torch.stack([s, b], -1).flatten(-2).contiguous().view(torch.uint8)


def _random_pages(case, n_pages, gen, device):
    """A filled pool [n_pages, page bytes]: every token's K and V drawn and quantised."""
    bits, D, H = case["bits"], case["D"], case["Hkv"]
    S = case["page"] // 16
    per = _strip_bytes(bits, D)
    out = torch.empty(n_pages * H * S, per, dtype=torch.uint8, device=device)
    turn = _turn(bits, D, device)
    half = per // 2
    R = _row_bytes(bits, D)
    gain = torch.exp(0.4 * torch.randn(2, D, generator=gen, device=device))
    step = max(1, (1 << 26) // (16 * D))
    for at in range(0, out.shape[0], step):
        n = min(step, out.shape[0] - at)
        for kv in range(2):
            x = (torch.randn(n, 16, D, generator=gen, device=device) * gain[kv]).half()
            codes, sb = _row_image(*_quantise(x, bits, torch.float32), bits)
            codes = codes.unflatten(-1, (-1, 16))
            stored = torch.empty_like(codes).scatter_(2, turn[None, :, :, None].expand_as(codes), codes)
            out[at:at + n, kv * half:kv * half + 16 * R] = stored.flatten(1)
            out[at:at + n, kv * half + 16 * R:(kv + 1) * half] = sb.flatten(1)
    return out.view(n_pages, -1)


def _unpack(strips, bits, D, wide):
    """Values [n, 2, 16, D] of strips [n, strip bytes], in type `wide`."""
    R, half = _row_bytes(bits, D), _strip_bytes(bits, D) // 2
    turn = _turn(bits, D, strips.device)
    both = strips.view(-1, 2, half)
    codes = both[..., :16 * R].unflatten(-1, (16, R // 16, 16))
    codes = codes.gather(3, turn[None, None, :, :, None].expand_as(codes)).flatten(-2)
    if bits == 4:
        codes = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)
    sb = both[..., 16 * R:].contiguous().view(torch.float16).view(-1, 2, 16, D // GROUP, 2).to(wide)
    return (codes.unflatten(-1, (-1, GROUP)).to(wide) * sb[..., 0:1] + sb[..., 1:2]).flatten(-2)


def _pages_values(pages, ids, case, wide):
    """K, V [len(ids) * page, Hkv, D] of whole pages, in the order of ids."""
    H, D, S = case["Hkv"], case["D"], case["page"] // 16
    strips = pages[ids.flatten().long()].view(-1, _strip_bytes(case["bits"], D))
    v = _unpack(strips, case["bits"], D, wide).view(-1, H, S, 2, 16, D)
    v = v.permute(3, 0, 2, 4, 1, 5).reshape(2, -1, H, D)
    return v[0], v[1]


# ---------------------------------------------------------------- prepare ----
def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(1000003 * seed + 17)
    st = dict(case=case)
    if case["op"] == "q4":
        B, n_in, n_out = case["B"], case["n_in"], case["n_out"]
        q = torch.randint(0, 256, (n_out * n_in // 2,), dtype=torch.uint8, device=dev, generator=gen)
        st["q"] = q.view(torch.int32).view(1, n_out, n_in // 8)
        u = torch.rand(1, n_out, n_in // GROUP, device=dev, generator=gen)
        st["s"] = ((u + 0.5) / (8.0 * math.sqrt(n_in))).half()
        z = torch.randint(0, 16, st["s"].shape, device=dev, generator=gen)
        st["b"] = (-(st["s"].float() * z)).half()
        st["x"] = torch.randn(B, n_in, device=dev, generator=gen).half()
        if own:
            from int4_routed_expert_prerouter_gb300 import binding
            st["packed"] = binding.pack_q4_rows((st["q"], st["s"], st["b"]))
        return st
    counts, B, page, H, D = _counts(case), case["B"], case["page"], case["Hkv"], case["D"]
    at = case.get("at", 0)
    need = [max(1, -(-(at + n) // page)) for n in counts]
    W = max(need)
    n_prefix = -(-case.get("prefix", 0) // page)
    n_pages = sum(need) + n_prefix + 1
    order = torch.randperm(n_pages, generator=gen, device=dev).to(torch.int32)
    first = torch.tensor([0] + need, device=dev).cumsum(0)[:-1]
    col = torch.arange(W, device=dev)[None, :]
    st["table"] = torch.where(col < torch.tensor(need, device=dev)[:, None],
                              order[(first[:, None] + col).clamp(max=n_pages - 1)], -1).to(torch.int32)
    st["prefix"] = order[sum(need):sum(need) + n_prefix].contiguous()
    if case["op"] == "kv":
        S = page // 16
        st["pages"] = torch.zeros(n_pages, H * S * _strip_bytes(case["bits"], D), dtype=torch.uint8, device=dev)
    else:
        st["pages"] = _random_pages(case, n_pages, gen, dev)
    st["lens"] = torch.tensor(counts, dtype=torch.int32, device=dev)
    st["start"] = torch.full((B,), at, dtype=torch.int32, device=dev)
    st["cu"] = torch.tensor([0] + counts, device=dev).cumsum(0).to(torch.int32)
    T = sum(counts)
    st["T"] = T
    if case["op"] == "kv":
        if case["fused"]:       # rows of a fused query/key/value projection
            wide = torch.randn(T, 4 * H * D, device=dev, generator=gen).half()
            st["k"] = wide[:, 2 * H * D:3 * H * D].unflatten(1, (H, D))
            st["v"] = wide[:, 3 * H * D:].unflatten(1, (H, D))
        else:
            st["k"], st["v"] = torch.randn(2, T, H, D, device=dev, generator=gen).half()
    if case["op"] == "attn":
        Hq = case["Hq"]
        if case["fused"]:
            wide = torch.randn(B, (Hq + 2 * H) * D, device=dev, generator=gen).half()
            st["query"] = wide[:, :Hq * D].unflatten(1, (Hq, D))
        else:
            st["query"] = torch.randn(B, Hq, D, device=dev, generator=gen).half()
    if own:
        from int4_routed_expert_prerouter_gb300 import binding
        st["cache"] = binding.KVCache(n_pages, page, H, D, case["bits"], pages=st["pages"])
    return st


# -------------------------------------------------------------------- run ----
def run(st):
    case = st["case"]
    if own:
        from int4_routed_expert_prerouter_gb300 import binding
        if case["op"] == "q4":
            return binding.q4_linear(st["packed"], case["n_out"], st["x"])
        if case["op"] == "kv":
            binding.kv_append(st["cache"], st["k"], st["v"], st["table"], st["start"], st["cu"])
            return binding.kv_read(st["cache"], st["table"], st["start"], st["cu"], st["T"])
        if case["op"] == "read":
            return binding.kv_read(st["cache"], st["table"], st["start"], st["cu"], st["T"])
        return binding.attn_decode(st["cache"], st["query"], st["table"], st["lens"], st["prefix"], case["prefix"])
    if case["op"] == "q4":
        return _q4(st, torch.float32).half()
    if case["op"] == "kv":
        _append(st)
    if case["op"] in ("kv", "read"):
        k, v = _read(st, torch.float32)
        return k.half(), v.half()
    return _attention(st, torch.float32).half()


def _q4(st, wide):
    sh = torch.arange(0, 32, 4, device=st["q"].device, dtype=torch.int32)
    q = (st["q"][0, :, :, None] >> sh) & 15
    w = q.flatten(1).unflatten(1, (-1, GROUP)).to(wide) * st["s"][0, ..., None].to(wide) + st["b"][0, ..., None].to(wide)
    return st["x"].to(wide) @ w.flatten(1).T


def _rows(st):
    """Sequence and position of every row of the call."""
    T = st["T"]
    r = torch.arange(T, device=st["cu"].device)
    b = torch.searchsorted(st["cu"].long(), r, right=True) - 1
    return b, st["start"].long()[b] + r - st["cu"].long()[b]


def _places(st):
    """Byte offsets in the pool of the strips' starts, [T, Hkv], and rows in them, [T]."""
    case = st["case"]
    b, pos = _rows(st)
    page = st["table"].long()[b, pos // case["page"]]
    per = _strip_bytes(case["bits"], case["D"])
    S = case["page"] // 16
    head = torch.arange(case["Hkv"], device=pos.device)
    strip = (page[:, None] * case["Hkv"] + head[None, :]) * S + (pos % case["page"] // 16)[:, None]
    return strip * per, pos % 16


def _append(st):
    case = st["case"]
    bits, D = case["bits"], case["D"]
    R, half = _row_bytes(bits, D), _strip_bytes(bits, D) // 2
    base, row = _places(st)
    turn = _turn(bits, D, base.device)[row]
    flat = st["pages"].view(-1)
    piece = torch.arange(16, device=base.device)
    sbs = torch.arange(D // GROUP * 4, device=base.device)

    def put(x, off):
        codes, sb = _row_image(*_quantise(x, bits, torch.float64), bits)     # in 64 bits: codes next to a border
        at = base[:, :, None, None] + off + (row * R)[:, None, None, None] + turn[:, None, :, None] * 16 + piece
        flat[at.flatten(2)] = codes
        flat[base[:, :, None] + off + 16 * R + (row * (D // GROUP * 4))[:, None, None] + sbs] = sb

    put(st["k"], 0)
    put(st["v"], half)


def _read(st, wide):
    case = st["case"]
    bits, D = case["bits"], case["D"]
    base, row = _places(st)
    strips = st["pages"].view(-1, _strip_bytes(bits, D))[base.flatten() // _strip_bytes(bits, D)]
    # the token's own row of its strip
    R, half = _row_bytes(bits, D), _strip_bytes(bits, D) // 2
    both = strips.view(*base.shape, 2, half)
    codes = both[..., :16 * R].unflatten(-1, (16, R // 16, 16))
    t = torch.arange(base.shape[0], device=base.device)
    codes = codes[t, :, :, row]                                  # [T, Hkv, 2, pieces, 16]
    turn = _turn(bits, D, base.device)[row]
    codes = codes.gather(3, turn[:, None, None, :, None].expand_as(codes)).flatten(-2)
    if bits == 4:
        codes = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)
    sb = both[..., 16 * R:].unflatten(-1, (16, D // GROUP * 4))[t, :, :, row].contiguous().view(torch.float16)
    sb = sb.unflatten(-1, (-1, 2)).to(wide)
    x = (codes.unflatten(-1, (-1, GROUP)).to(wide) * sb[..., 0:1] + sb[..., 1:2]).flatten(-2)
    return x[:, :, 0], x[:, :, 1]


def _attention(st, wide):
    case = st["case"]
    B, Hq, H, D, P = case["B"], case["Hq"], case["Hkv"], case["D"], case["prefix"]
    q = st["query"].to(wide).unflatten(1, (H, Hq // H))                            # [B, H, G, D]
    W = st["table"].shape[1] * case["page"]
    k, v = (x.view(B, W, H, D) for x in _pages_values(st["pages"], st["table"].clamp(min=0), case, wide))
    score = torch.matmul(q, k.permute(0, 2, 3, 1))                                 # [B, H, G, W]
    seen = torch.arange(W, device=q.device)[None, :] < st["lens"][:, None]
    score = score.masked_fill(~seen[:, None, None, :], -math.inf)
    if P:
        pk, pv = (x[:P] for x in _pages_values(st["pages"], st["prefix"], case, wide))
        rows = q.permute(1, 0, 2, 3).flatten(1, 2)                                 # [H, B G, D]
        ps = torch.matmul(rows, pk.permute(1, 2, 0)).unflatten(1, (B, -1)).transpose(0, 1)
        score = torch.cat([ps, score], -1)
    score = score / math.sqrt(D)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(torch.isinf(top), torch.zeros_like(top), top))
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p[..., P:], v.permute(0, 2, 1, 3))
    if P:
        o = o + torch.matmul(p[..., :P].transpose(0, 1).flatten(1, 2), pv.transpose(0, 1)).unflatten(1, (B, -1)).transpose(0, 1)
    return torch.where(total > 0, o / torch.where(total > 0, total, torch.ones_like(total)), torch.zeros_like(o)).flatten(1, 2)


# ------------------------------------------------------------------ exact ----
def exact(case, seed):
    """What run() returns, in 64 bits, sequence by sequence from the definitions."""
    st = prepare(case, seed)
    f8 = torch.float64
    if case["op"] == "q4":
        out = []
        for rows in torch.arange(case["n_out"], device=st["q"].device).split(8192):
            words = st["q"][0, rows]
            w = torch.stack([(words >> (4 * i)) & 15 for i in range(8)], -1).reshape(len(rows), -1, GROUP).to(f8)
            w = w * st["s"][0, rows].to(f8)[..., None] + st["b"][0, rows].to(f8)[..., None]
            out.append(st["x"].to(f8) @ w.reshape(len(rows), -1).T)
        return torch.cat(out, 1)
    if case["op"] == "kv":
        both = []
        for x in (st["k"], st["v"]):
            g = x.to(f8).reshape(st["T"], case["Hkv"], -1, GROUP)
            low, high = g.min(-1, keepdim=True).values, g.max(-1, keepdim=True).values
            top = float(2 ** case["bits"] - 1)
            s = ((high - low) / top).half().to(f8)
            q = torch.round((g - low) / s).nan_to_num(0.0).clamp(0.0, top)
            both.append((low + s * q).reshape(x.shape))
        return tuple(both)
    counts = _counts(case)
    values = []
    for b, n in enumerate(counts):
        pages = -(-(case.get("at", 0) + n) // case["page"])
        k, v = _pages_values(st["pages"], st["table"][b, :pages], case, f8)
        values.append((k[case.get("at", 0):][:n], v[case.get("at", 0):][:n]))
    if case["op"] == "read":
        return tuple(torch.cat(x) for x in zip(*values))
    prefix = _pages_values(st["pages"], st["prefix"], case, f8) if case["prefix"] else None
    G = case["Hq"] // case["Hkv"]
    out = torch.zeros(case["B"], case["Hq"], case["D"], dtype=f8, device=st["query"].device)
    for b in range(case["B"]):
        k, v = values[b]
        if prefix is not None:
            k, v = torch.cat([prefix[0][:case["prefix"]], k]), torch.cat([prefix[1][:case["prefix"]], v])
        if not k.shape[0]:
            continue
        for h in range(case["Hkv"]):
            w = torch.softmax(st["query"][b, h * G:(h + 1) * G].to(f8) @ k[:, h].T / case["D"] ** 0.5, -1)
            out[b, h * G:(h + 1) * G] = w @ v[:, h]
    return out
