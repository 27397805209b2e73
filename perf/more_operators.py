"""Cases, plain forms and exact values of the operators that take a prompt and drafted
tokens through a decoder block: rotary positions, attention over packed prompts, attention of
trees of drafted tokens over the quantised KV cache, and moves of that cache's rows and pages.

Sizes follow this repository's configurations (64 and 256 sequences, a 3,100-token
prompt, 64/128/256-wide heads, contexts of up to 131,072 tokens) or are generic.
"""
import math
import random

import torch

own = False

GROUP = 64


# ------------------------------------------------------------------ cases ----
def listed():
    return [
        # one decode step of 64 sequences, queries and keys cut from the fused projection: latency counts
        dict(name="rope_step_64", op="rope", layout="half", Hq=32, Hkv=8, D=128, rot=128, scaling="plain", B=64, lo=1, hi=1,
             at=131000, fused=True, back=False),
        # three prompts written at once, part of the head turned, scaled for long contexts
        dict(name="rope_prompts_8192", op="rope", layout="interleaved", Hq=32, Hkv=8, D=128, rot=64, scaling="ramp", B=3,
             lo=1000, hi=4800, at=0, fused=True, back=False),
        # one short prompt with wide heads: latency
        dict(name="prompt_one_short", op="prompt", Hq=16, Hkv=2, D=256, B=1, lo=131, hi=131, ctx=0, fused=True),
        # 64 prompts of 1 to 1,024 tokens packed together
        dict(name="prompt_ragged_64", op="prompt", Hq=32, Hkv=8, D=128, B=64, lo=1, hi=1024, ctx=0, fused=True),
        # the next 509 tokens of a prompt whose first 32,003 have been read back from the cache
        dict(name="prompt_next_part", op="prompt", Hq=32, Hkv=8, D=128, B=1, lo=509, hi=509, ctx=32003, fused=False),
        # one long prompt in whole
        dict(name="prompt_long", op="prompt", Hq=32, Hkv=8, D=128, B=1, lo=16384, hi=16384, ctx=0, fused=False),
        # one sequence, a small tree, wide heads: latency of a short context
        dict(name="tree_one_sequence", op="tree", bits=8, Hq=16, Hkv=2, D=256, page=64, B=1, lo=777, hi=777, drafts=12,
             chain=False),
        # 64 sequences with trees of up to 16 drafted tokens
        dict(name="tree_64", op="tree", bits=4, Hq=32, Hkv=8, D=128, page=64, B=64, lo=500, hi=4000, drafts=16, chain=False),
        # four long contexts, trees of up to 48 drafted tokens
        dict(name="tree_long", op="tree", bits=4, Hq=32, Hkv=8, D=128, page=128, B=4, lo=100003, hi=131072, drafts=48,
             chain=False),
        # the accepted ones of 64 sequences' drafted tokens moved to the end of the context
        dict(name="compact_accepted_64", op="compact", bits=4, Hkv=8, D=128, page=64, B=64, n=16, keep=6, at=900),
        # a quarter of long contexts kept
        dict(name="compact_contexts", op="compact", bits=8, Hkv=8, D=128, page=64, B=7, n=8191, keep=2047, at=33),
        # the pages of a prompt copied for eight continuations
        dict(name="fork_pages", op="fork", bits=4, Hkv=8, D=128, page=64, pages=1000, copies=8),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "prompt", "prompt", "tree", "tree", "compact", "fork"])
    D = rng.choice([64, 128, 256])
    Hkv = rng.choice([1, 2, 3, 4, 8])
    Hq = Hkv * rng.choice([1, 2, 4, 5, 8])
    if op == "rope":
        B = _log(rng, 1, 64)
        T = _log(rng, 1, 8192 * 40 * 128 // ((Hq + Hkv) * D))
        return dict(op=op, layout=rng.choice(["half", "interleaved"]), Hq=Hq, Hkv=Hkv, D=D, rot=rng.choice([D, D, D // 2, D // 4, D - 6]),
                    scaling=rng.choice(["plain", "linear", "base", "ramp", "bands"]), B=B, lo=rng.randint(0, 1),
                    hi=max(1, T // B), at=_log(rng, 1, 500000), fused=rng.random() < 0.5, back=rng.random() < 0.25)
    if op == "prompt":
        B = _log(rng, 1, 64)
        most = min(8192, int(math.sqrt(0.4e12 / (B * Hq * D))), 4_000_000 // (B * 8))
        hi = _log(rng, 1, max(2, most))
        ctx = rng.choice([0, 0, _log(rng, 1, max(2, min(32768, int(0.2e12 / (B * hi * Hq * D)), 400_000 // B)))])
        return dict(op=op, Hq=Hq, Hkv=Hkv, D=D, B=B, lo=min(hi, rng.randint(0, 1)), hi=hi, ctx=ctx, fused=rng.random() < 0.5 and not ctx)
    bits, page = rng.choice([4, 8]), 16 * rng.choice([1, 2, 3, 4, 8])
    if op == "tree":
        B = _log(rng, 1, 64)
        drafts = _log(rng, 1, 100)
        hi = _log(rng, 1, max(2, min(65536, 1_500_000_000 // (Hkv * D * bits * B), 10 ** 11 // (B * drafts * Hq * D))))
        return dict(op=op, bits=bits, Hq=Hq, Hkv=Hkv, D=D, page=page, B=B, lo=min(hi, rng.randint(0, 1)), hi=hi, drafts=drafts,
                    chain=rng.random() < 0.25)
    if op == "compact":
        B = _log(rng, 1, 64)
        n = _log(rng, 2, max(3, min(8192, 60000 * 1024 // (B * Hkv * D))))
        return dict(op=op, bits=bits, Hkv=Hkv, D=D, page=page, B=B, n=n, keep=rng.randint(0, n // 2), at=rng.randint(0, 500))
    copies = rng.choice([1, 2, 8])
    return dict(op=op, bits=bits, Hkv=Hkv, D=D, page=page, pages=_log(rng, 1, 600_000_000 // (copies * Hkv * D * page)), copies=copies)


def _counts(case):
    """Tokens of each sequence: spread over [lo, hi], both ends among them."""
    B, lo, hi = case["B"], case["lo"], case["hi"]
    if B == 1:
        return [hi]
    spread = [lo + int((hi - lo) * ((i * 0.6180339887498949) % 1.0)) for i in range(B)]
    spread[B // 2] = hi
    spread[0] = lo
    return spread


def _drafts(case):
    """Drafted tokens of each sequence: from none (where there are several) to case["drafts"]."""
    B, n = case["B"], case["drafts"]
    return [n if b == 0 else (b * 7 + n) % (n + 1) if b % 5 == 0 else max(1, n - b % 4) for b in range(B)]


def _kept(case):
    """Kept rows of each sequence."""
    return [case["keep"] if b == 0 else case["keep"] * (b % 4) // 3 for b in range(case["B"])]


def _token_bytes(case):
    return 2 * case["Hkv"] * (case["D"] * case["bits"] // 8 + case["D"] // GROUP * 4)


def work(case):
    if case["op"] == "rope":
        values = sum(_counts(case)) * (case["Hq"] + case["Hkv"]) * case["D"]
        return dict(bytes=2 * 2 * values, flops=3 * values)
    if case["op"] == "prompt":
        n = _counts(case)
        keys = sum(x + case["ctx"] for x in n)
        seen = sum(x * case["ctx"] + x * (x + 1) // 2 for x in n)
        return dict(bytes=2 * case["D"] * (2 * sum(n) * case["Hq"] + 2 * keys * case["Hkv"]), flops=4 * case["Hq"] * case["D"] * seen)
    if case["op"] == "tree":
        n, d = _counts(case), _drafts(case)
        seen = sum(x * y + y * (y + 1) // 2 for x, y in zip(n, d))
        tokens = sum(x + y for x, y in zip(n, d) if y)
        return dict(bytes=tokens * _token_bytes(case) + 2 * 2 * sum(d) * case["Hq"] * case["D"], flops=4 * case["Hq"] * case["D"] * seen)
    if case["op"] == "compact":
        return dict(bytes=2 * sum(_kept(case)) * _token_bytes(case), flops=0)
    # each page of the prompt read once, each copy written once
    return dict(bytes=(1 + case["copies"]) * case["pages"] * case["page"] * _token_bytes(case), flops=0)


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


def _random_pages(case, n_pages, gen, device):
    """A filled pool [n_pages, page bytes]: every token's K and V drawn and quantised."""
    bits, D, H = case["bits"], case["D"], case["Hkv"]
    per, R, top = _strip_bytes(bits, D), _row_bytes(bits, D), 2 ** bits - 1
    half = per // 2
    out = torch.empty(n_pages * H * (case["page"] // 16), per, dtype=torch.uint8, device=device)
    turn = _turn(bits, D, device)
    gain = torch.exp(0.4 * torch.randn(2, D, generator=gen, device=device))
    step = max(1, (1 << 26) // (16 * D))
    for at in range(0, out.shape[0], step):
        n = min(step, out.shape[0] - at)
        for kv in range(2):
            x = (torch.randn(n, 16, D, generator=gen, device=device) * gain[kv]).half()
            g = x.unflatten(-1, (-1, GROUP)).float()
            mn, mx = g.amin(-1), g.amax(-1)
            s = ((mx - mn) / top).half()
            codes = torch.round((g - mn[..., None]) / s.float()[..., None]).clamp(0, top).to(torch.uint8).flatten(-2)
            if bits == 4:
                codes = codes[..., 0::2] | (codes[..., 1::2] << 4)
            sb = torch.stack([s, mn.half()], -1).flatten(-2).contiguous().view(torch.uint8)
            codes = codes.unflatten(-1, (-1, 16))
            stored = torch.empty_like(codes).scatter_(2, turn[None, :, :, None].expand_as(codes), codes)
            out[at:at + n, kv * half:kv * half + 16 * R] = stored.flatten(1)
            out[at:at + n, kv * half + 16 * R:(kv + 1) * half] = sb.flatten(1)
    return out.view(n_pages, -1)


def _pages_values(pages, ids, case, wide):
    """K, V [len(ids) * page, Hkv, D] of whole pages, in the order of ids, in type `wide`."""
    bits, H, D, S = case["bits"], case["Hkv"], case["D"], case["page"] // 16
    R, half = _row_bytes(bits, D), _strip_bytes(bits, D) // 2
    strips = pages[ids.flatten().long()].view(-1, 2, half)
    turn = _turn(bits, D, pages.device)
    codes = strips[..., :16 * R].unflatten(-1, (16, R // 16, 16))
    codes = codes.gather(3, turn[None, None, :, :, None].expand_as(codes)).flatten(-2)
    if bits == 4:
        codes = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)
    sb = strips[..., 16 * R:].contiguous().view(torch.float16).view(-1, 2, 16, D // GROUP, 2).to(wide)
    v = (codes.unflatten(-1, (-1, GROUP)).to(wide) * sb[..., 0:1] + sb[..., 1:2]).flatten(-2)
    v = v.view(-1, H, S, 2, 16, D).permute(3, 0, 2, 4, 1, 5).reshape(2, -1, H, D)
    return v[0], v[1]


# --------------------------------------------------------------- rotation ----
BASE, TRAINED, FACTOR = 500000.0, 8192.0, 16.0


def _angles_per_position(case):
    """Angle per position of each pair (fp64, on the host) and the factor on the result."""
    r, kind = case["rot"], case["scaling"]
    base = BASE * FACTOR ** (r / (r - 2)) if kind == "base" else BASE
    f = [base ** (-2.0 * i / r) for i in range(r // 2)]
    if kind == "linear":
        return [x / FACTOR for x in f], 1.0
    if kind == "ramp":
        # pairs that turn less than once over the trained length are slowed down, those that turn more than 32 times stay
        lo, hi = (r * math.log(TRAINED / (t * 2 * math.pi)) / (2 * math.log(BASE)) for t in (32.0, 1.0))
        lo, hi = max(math.floor(lo), 0), min(math.ceil(hi), r - 1)
        keep = [1.0 - min(max((i - lo) / max(hi - lo, 0.001), 0.0), 1.0) for i in range(r // 2)]
        return [x * k + x / FACTOR * (1 - k) for x, k in zip(f, keep)], 0.1 * math.log(FACTOR) + 1.0
    if kind == "bands":
        # by wavelength: below trained / 4 as it is, above trained slowed down, smooth between
        keep = [min(max((TRAINED * x / (2 * math.pi) - 1.0) / (4.0 - 1.0), 0.0), 1.0) for x in f]
        return [x * k + x / FACTOR * (1 - k) for x, k in zip(f, keep)], 1.0
    return f, 1.0


def _pairs(x, case):
    """The two halves of the turned pairs, [.., rot / 2] each, as views."""
    r = case["rot"]
    return (x[..., :r // 2], x[..., r // 2:r]) if case["layout"] == "half" else (x[..., 0:r:2], x[..., 1:r:2])


def _positions(st):
    r = torch.arange(st["T"], device=st["cu"].device)
    b = torch.searchsorted(st["cu"].long(), r, right=True) - 1
    return st["start"].long()[b] + r - st["cu"].long()[b]


def _rope(x, st, wide):
    case = st["case"]
    f, m = _angles_per_position(case)
    angle = _positions(st).double()[:, None] * torch.tensor(f, dtype=torch.float64, device=x.device)   # far positions: 64 bits
    c, s = (a.to(wide)[:, None, :] for a in (torch.cos(angle) * m, torch.sin(angle) * m))
    if case["back"]:
        s = -s
    y = x.to(wide)
    a, b = _pairs(y, case)
    u, v = a * c - b * s, a * s + b * c
    y = y.clone()
    a, b = _pairs(y, case)
    a.copy_(u)
    b.copy_(v)
    return y


# ---------------------------------------------------------------- prepare ----
def _cu(counts, dev):
    return torch.tensor([0] + list(counts), device=dev).cumsum(0).to(torch.int32)


def _tree_words(case, seed, dev):
    """[rows, words] int32: bit j of a row is set where it sees the j-th drafted token of its own
    sequence, that is, for itself and its ancestors in a random tree."""
    rng = random.Random(seed)
    n = _drafts(case)
    words = -(-max(n) // 32)
    rows = []
    for x in n:
        mine = []
        for j in range(x):
            parent = rng.randint(max(0, j - 5), j) - 1          # -1: a root of its own
            mine.append((mine[parent] if parent >= 0 else 0) | 1 << j)
        rows += mine
    flat = [((m >> 32 * w) & 0xFFFFFFFF) for m in rows for w in range(words)]
    return torch.tensor([w - (1 << 32) if w >> 31 else w for w in flat], dtype=torch.int32).view(len(rows), words).to(dev)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(1000003 * seed + 29)
    st = dict(case=case)
    H, D = case["Hkv"], case["D"]

    def rows(n, *heads):
        """fp16 rows [n, h, D] for each h of heads, cut from one wide projection where the case says so."""
        if case.get("fused"):
            wide = torch.randn(n, sum(heads) * D, device=dev, generator=gen).half()
            return [x.unflatten(1, (-1, D)) for x in wide.split([h * D for h in heads], 1)]
        return [torch.randn(n, h, D, device=dev, generator=gen).half() for h in heads]

    if case["op"] == "rope":
        counts = _counts(case)
        st["T"], st["cu"] = sum(counts), _cu(counts, dev)
        st["start"] = torch.randint(0, case["at"] + 1, (case["B"],), device=dev, generator=gen).to(torch.int32)
        st["q"], st["k"], _ = rows(st["T"], case["Hq"], H, H)
        if own:
            from int4_routed_expert_prerouter_gb300 import binding
            extra = {} if case["scaling"] == "plain" else dict(factor=FACTOR)
            if case["scaling"] == "ramp":
                extra.update(trained_len=TRAINED, low=1.0, high=32.0)
            if case["scaling"] == "bands":
                extra.update(trained_len=TRAINED, low=1.0, high=4.0)
            st["plan"] = binding.RopePlan(D, case["rot"], base=BASE, layout=case["layout"], scaling=case["scaling"], device=dev, **extra)
        return st
    if case["op"] == "prompt":
        counts = _counts(case)
        st["cu"] = _cu(counts, dev)
        st["cu_keys"] = _cu([n + case["ctx"] for n in counts], dev) if case["ctx"] else None
        if case["ctx"]:
            st["q"], = rows(sum(counts), case["Hq"])
            st["k"], st["v"] = rows(sum(counts) + case["B"] * case["ctx"], H, H)
        else:
            st["q"], st["k"], st["v"] = rows(sum(counts), case["Hq"], H, H)
        return st
    page = case["page"]
    if case["op"] == "fork":
        n, copies = case["pages"], case["copies"]
        n_pages = n * (1 + copies)
        order = torch.randperm(n_pages, generator=gen, device=dev).to(torch.int32)
        st["src"] = order[:n].repeat(copies).contiguous()
        st["dst"] = order[n:].contiguous()
    else:
        if case["op"] == "tree":
            counts, more = _counts(case), _drafts(case)
        else:
            counts, more = [case["at"]] * case["B"], [case["n"]] * case["B"]
        need = [max(1, -(-(a + b) // page)) for a, b in zip(counts, more)]
        n_pages, W = sum(need) + 1, max(need)
        order = torch.randperm(n_pages, generator=gen, device=dev).to(torch.int32)
        first = torch.tensor([0] + need, device=dev).cumsum(0)[:-1]
        col = torch.arange(W, device=dev)[None, :]
        st["table"] = torch.where(col < torch.tensor(need, device=dev)[:, None],
                                  order[(first[:, None] + col).clamp(max=n_pages - 1)], -1).to(torch.int32)
        st["lens"] = torch.tensor(counts, dtype=torch.int32, device=dev)
        if case["op"] == "tree":
            st["cu"] = _cu(more, dev)
            st["q"], = rows(sum(more), case["Hq"])
            st["mask"] = None if case["chain"] else _tree_words(case, seed, dev)
        else:
            kept = _kept(case)
            st["cu"] = _cu(kept, dev)
            rng = random.Random(seed)
            src = []
            for m in kept:      # the first ones stay where they are, the others come from behind all kept places
                stay = rng.randint(0, m // 2)
                src += list(range(stay)) + sorted(rng.sample(range(m, case["n"]), m - stay))
            st["src"] = (torch.tensor(src, dtype=torch.int64, device=dev) + case["at"]).to(torch.int32)
    st["pages"] = _random_pages(case, n_pages, gen, dev)
    if own:
        from int4_routed_expert_prerouter_gb300 import binding
        st["cache"] = binding.KVCache(n_pages, page, H, D, case["bits"], pages=st["pages"])
    return st


# -------------------------------------------------------------------- run ----
def run(st):
    case = st["case"]
    if own:
        from int4_routed_expert_prerouter_gb300 import binding
        if case["op"] == "rope":
            return binding.rope(st["plan"], st["q"], st["k"], st["start"], st["cu"], backward=case["back"])
        if case["op"] == "prompt":
            return binding.attn_prompt(st["q"], st["k"], st["v"], st["cu"], st["cu_keys"])
        if case["op"] == "tree":
            return binding.attn_tree(st["cache"], st["q"], st["table"], st["lens"], st["cu"], st["mask"])
        if case["op"] == "compact":
            binding.kv_compact(st["cache"], st["table"], st["lens"], st["src"], st["cu"])
        else:
            binding.kv_copy_pages(st["cache"], st["src"], st["dst"])
        return st["pages"]          # moved bytes as they are: nothing is computed from them
    if case["op"] == "rope":
        return tuple(_rope(x, st, torch.float32).half() for x in (st["q"], st["k"]))
    if case["op"] == "prompt":
        return _prompt(st)
    if case["op"] == "tree":
        return _tree(st)
    if case["op"] == "compact":
        _compact(st)
    else:
        st["pages"][st["dst"].long()] = st["pages"][st["src"].long()]
    return st["pages"]


def _attend(q, k, v, seen):
    """q [n, Hq, D], k, v [m, Hkv, D] in 32 bits, seen [n, m] truth values -> [n, Hq, D]; rows that see
    nothing give zeros.  A few heads at a time, so that the scores stay within a few GB."""
    n, Hq, D = q.shape
    m, H, _ = k.shape
    G = Hq // H
    out = torch.zeros_like(q)
    step = max(1, (1 << 29) // max(1, G * n * m))
    for h in range(0, H, step):
        hs = slice(h, min(H, h + step))
        qs = q[:, hs.start * G:hs.stop * G].unflatten(1, (-1, G)).permute(1, 2, 0, 3).flatten(1, 2)     # [h, G n, D]
        s = torch.matmul(qs, k[:, hs].permute(1, 2, 0)).unflatten(1, (G, n)) / math.sqrt(D)
        s = s.masked_fill(~seen, -math.inf)
        top = s.amax(-1, keepdim=True)
        p = torch.exp(s - torch.where(torch.isinf(top), torch.zeros_like(top), top))
        total = p.sum(-1, keepdim=True)
        o = torch.matmul(p.flatten(1, 2), v[:, hs].transpose(0, 1)).unflatten(1, (G, n))
        o = torch.where(total > 0, o / torch.where(total > 0, total, torch.ones_like(total)), torch.zeros_like(o))
        out[:, hs.start * G:hs.stop * G] = o.permute(2, 0, 1, 3).flatten(1, 2)
    return out


def _prompt(st):
    case, out = st["case"], torch.zeros_like(st["q"], memory_format=torch.contiguous_format)
    r = kk = 0
    for n in _counts(case):
        m = n + case["ctx"]
        if n:
            q, k, v = (x.float() for x in (st["q"][r:r + n], st["k"][kk:kk + m], st["v"][kk:kk + m]))
            seen = torch.arange(m, device=q.device)[None, :] <= torch.arange(n, device=q.device)[:, None] + case["ctx"]
            out[r:r + n] = _attend(q, k, v, seen).half()
        r, kk = r + n, kk + m
    return out


def _seen_by_drafts(st, r, x, n):
    """[x, n + x]: the context and those drafted tokens that the rows r .. r + x - 1 see."""
    dev = st["q"].device
    if st["mask"] is None:
        tree = torch.ones(x, x, dtype=torch.bool, device=dev).tril()
    else:
        j = torch.arange(x, device=dev)
        tree = (st["mask"][r:r + x][:, j // 32] >> (j % 32).to(torch.int32)) & 1 != 0
    return torch.cat([torch.ones(x, n, dtype=torch.bool, device=dev), tree], 1)


def _tree(st):
    case, out = st["case"], torch.zeros_like(st["q"])
    r = 0
    for b, (n, x) in enumerate(zip(_counts(case), _drafts(case))):
        if x:
            k, v = _pages_values(st["pages"], st["table"][b, :-(-(n + x) // case["page"])], case, torch.float32)
            out[r:r + x] = _attend(st["q"][r:r + x].float(), k[:n + x], v[:n + x], _seen_by_drafts(st, r, x, n)).half()
        r += x
    return out


def _compact(st):
    """Codes and (s, b) pairs of the kept rows, gathered, then put at their new places."""
    case = st["case"]
    bits, D, H, page = case["bits"], case["D"], case["Hkv"], case["page"]
    R, half, per, S = _row_bytes(bits, D), _strip_bytes(bits, D) // 2, _strip_bytes(bits, D), page // 16
    T = st["src"].shape[0]
    if not T:
        return
    dev = st["src"].device
    r = torch.arange(T, device=dev)
    b = torch.searchsorted(st["cu"].long(), r, right=True) - 1
    dst = st["lens"].long()[b] + r - st["cu"].long()[b]
    head = torch.arange(H, device=dev)
    turn = _turn(bits, D, dev)

    def places(pos):
        """Byte numbers of the rows' codes and pairs, [T, H, 2, R + pairs]."""
        strip = (st["table"].long()[b, pos // page][:, None] * H + head) * S + (pos % page // 16)[:, None]
        row = pos % 16
        codes = (row * R)[:, None, None] + turn[row][:, :, None] * 16 + torch.arange(16, device=dev)
        pairs = 16 * R + (row * (D // GROUP * 4))[:, None] + torch.arange(D // GROUP * 4, device=dev)
        inner = torch.cat([codes.flatten(1), pairs], 1)
        return (strip * per)[:, :, None, None] + torch.arange(2, device=dev)[:, None] * half + inner[:, None, None, :]

    flat = st["pages"].view(-1)
    flat[places(dst)] = flat[places(st["src"].long())]


# ------------------------------------------------------------------ exact ----
def exact(case, seed):
    """What run() returns, in 64 bits, row block by row block from the definitions."""
    if case["op"] in ("compact", "fork"):
        return None                 # moved, not computed
    st = prepare(case, seed)
    f8 = torch.float64
    if case["op"] == "rope":
        both = []
        f, m = _angles_per_position(case)
        for x in (st["q"], st["k"]):
            turns = _positions(st).to(f8)[:, None] * torch.tensor(f, dtype=f8, device=x.device)
            z = torch.polar(torch.full_like(turns, m), -turns if case["back"] else turns)[:, None, :]
            a, b = _pairs(x.to(f8), case)
            z = z * torch.complex(a.contiguous(), b.contiguous())
            y = x.to(f8).clone()
            a, b = _pairs(y, case)
            a.copy_(z.real)
            b.copy_(z.imag)
            both.append(y)
        return tuple(both)
    counts = _counts(case)
    rows = _drafts(case) if case["op"] == "tree" else counts
    G = case["Hq"] // case["Hkv"]
    out = torch.zeros(st["q"].shape, dtype=f8, device=st["q"].device)
    r = kk = 0
    for b, (n, x) in enumerate(zip(counts, rows)):
        if case["op"] == "tree":
            ctx, m = n, n + x
            k, v = _pages_values(st["pages"], st["table"][b, :max(1, -(-m // case["page"]))], case, f8)
        else:
            ctx, m = case["ctx"], n + case["ctx"]
            k, v = st["k"][kk:kk + m].to(f8), st["v"][kk:kk + m].to(f8)
            kk += m
        hidden = ~_seen_by_drafts(st, r, x, ctx) if case["op"] == "tree" else None
        for at in range(0, x, 2048):
            to = min(x, at + 2048)
            last = m if case["op"] == "tree" else ctx + to
            mask = hidden[at:to] if hidden is not None else \
                torch.ones(to - at, last, dtype=torch.bool, device=out.device).triu(ctx + at + 1)
            for h in range(case["Hq"]):
                w = st["q"][r + at:r + to, h].to(f8) @ k[:last, h // G].T / case["D"] ** 0.5
                w = torch.softmax(w.masked_fill(mask, -math.inf), -1)
                out[r + at:r + to, h] = w @ v[:last, h // G]
        r += x
    return out
