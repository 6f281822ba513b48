"""What is measured of the operators around a paged e4m3 cache with a scale for
each block of 16 tokens and head: their plain forms in elementary torch
operations, the library's calls, and the cases.

* append, write: one token per request, or chunks of prompts, with rotary
  positions, into blocks whose scales follow their largest value.
* decode: attention of one query token per request.
* chunk: attention of several query tokens per request at the end of its
  context, or over all of an encoder's states (cross attention).
"""
import math
import random

import torch

own = False

D = 128
TILE = 16
LOW, HIGH = -50, 30  # exponents of a block's scale


# ------------------------------------------------------------------- cases
def listed():
    return [
        # one request's next token: a latency
        dict(name="append_b1", kind="append", B=1, Hq=64, Hkv=8, ps=16, rot=128, interleaved=False, pos=8190),
        # a full decode batch, interleaved pairs on half of the head, far positions
        dict(name="append_b64", kind="append", B=64, Hq=64, Hkv=8, ps=64, rot=64, interleaved=True, pos=131071),
        # a prefill batch of prompts from their start
        dict(name="write_16k", kind="write", B=4, tokens=16384, Hq=64, Hkv=8, ps=16, rot=128, interleaved=False, pos=0),
        # ragged chunks of long prompts, five query heads to a kv head
        dict(name="write_chunks", kind="write", B=7, tokens=2011, Hq=40, Hkv=8, ps=64, rot=96, interleaved=True, pos=100000),
        # a few short conversations: the smallest decode batch
        dict(name="decode_b4_512", kind="decode", B=4, Hq=64, Hkv=8, ps=16, ctx=512, ragged=False),
        # the benchmark's batch and context
        dict(name="decode_b32_8k", kind="decode", B=32, Hq=64, Hkv=8, ps=16, ctx=8192, ragged=False),
        # contexts of all lengths, wide pages
        dict(name="decode_b61_ragged", kind="decode", B=61, Hq=40, Hkv=8, ps=64, ctx=16001, ragged=True),
        # a few very long documents
        dict(name="decode_b4_128k", kind="decode", B=4, Hq=64, Hkv=8, ps=64, ctx=131072, ragged=False),
        # drafted tokens of a batch checked in one pass
        dict(name="chunk_verify_b16", kind="chunk", causal=True, B=16, tokens=80, Hq=64, Hkv=8, ps=16, pos=2048),
        # a whole prompt
        dict(name="chunk_prompt_8k", kind="chunk", causal=True, B=1, tokens=8192, Hq=64, Hkv=8, ps=16, pos=0),
        # ragged chunks behind long contexts
        dict(name="chunk_ragged_b5", kind="chunk", causal=True, B=5, tokens=1999, Hq=40, Hkv=8, ps=64, pos=16000),
        # a decoder's tokens over an encoder's states, one query head to a kv head
        dict(name="chunk_cross_b8", kind="chunk", causal=False, B=8, tokens=1031, Hq=16, Hkv=16, ps=32, pos=1500),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["append", "write", "decode", "decode", "chunk", "chunk", "chunk"])
    ps = rng.choice([16, 16, 32, 64, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    Hq = Hkv * rng.choice([1, 4, 5, 7, 8])
    if kind == "decode":
        B = _log_int(rng, 1, 64)
        return dict(kind=kind, B=B, Hq=Hq, Hkv=Hkv, ps=ps, ctx=_log_int(rng, 1, min(32768, 400000 // B)),
                    ragged=rng.random() < 0.6)
    if kind == "chunk":
        B = _log_int(rng, 1, 16)
        return dict(kind=kind, causal=rng.random() < 0.7, B=B, tokens=_log_int(rng, B, 4096), Hq=Hq, Hkv=Hkv, ps=ps,
                    pos=_log_int(rng, 1, 8192))
    rot, inter = rng.choice([32, 64, 96, 128]), rng.random() < 0.5
    if kind == "append":
        return dict(kind=kind, B=_log_int(rng, 1, 256), Hq=Hq, Hkv=Hkv, ps=ps, rot=rot, interleaved=inter,
                    pos=_log_int(rng, 1, 131071))
    B = _log_int(rng, 1, 16)
    return dict(kind=kind, B=B, tokens=_log_int(rng, 4 * B, 8192), Hq=Hq, Hkv=Hkv, ps=ps, rot=rot,
                interleaved=inter, pos=_log_int(rng, 1, 100000))


# ------------------------------------------------ shapes that a case stands for
def _pages(tokens, ps):
    return -(-tokens // ps)


def _chunks(c):
    """(tokens of each request's chunk, tokens before it; cross attention: the encoder's states)"""
    B, T = c["B"], c["tokens"]
    cut = [T * r * (r + 2) // (B * (B + 2)) for r in range(B + 1)]
    n = [b - a for a, b in zip(cut, cut[1:])]
    if c["kind"] == "write":
        return n, [c["pos"] * (r + 1) // B for r in range(B)]
    return n, [c["pos"] - (1009 * r) % (c["pos"] // 2 + 1) for r in range(B)]


def _lengths(c):
    """Context of each request, the new tokens among them."""
    B = c["B"]
    if c["kind"] == "append":
        return [max(1, c["pos"] + 1 - (1009 * r) % (c["pos"] + 1)) for r in range(B)]
    if c["kind"] == "decode":
        return [max(1, c["ctx"] - (9973 * r) % c["ctx"]) if c["ragged"] else c["ctx"] for r in range(B)]
    n, before = _chunks(c)
    return [a + b for a, b in zip(n, before)] if c["kind"] == "write" or c["causal"] else before


def work(c):
    lens = _lengths(c)
    if c["kind"] in ("append", "write"):
        T = c["B"] if c["kind"] == "append" else c["tokens"]
        scales = 2 * c["Hkv"] * (T if c["kind"] == "append" else T // TILE)
        return {"bytes": T * D * (4 * c["Hq"] + 6 * c["Hkv"]) + scales, "flops": 3 * T * (c["Hq"] + c["Hkv"]) * c["rot"]}
    kv = sum(lens) * c["Hkv"] * 2 * D + sum(-(-x // TILE) for x in lens) * c["Hkv"] * 2
    if c["kind"] == "decode":
        return {"bytes": kv + c["B"] * c["Hq"] * (6 * D + 4), "flops": 4 * D * c["Hq"] * sum(lens)}
    n, before = _chunks(c)
    seen = sum(a * b + a * (a + 1) // 2 if c["causal"] else a * b for a, b in zip(n, before))
    return {"bytes": kv + c["tokens"] * c["Hq"] * (4 * D + 4), "flops": 4 * D * c["Hq"] * seen}


# ----------------------------------------------------------------- preparing
def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _freqs(c):
    """Inverse frequencies of a long context: base 500000, the slow half of them stretched eightfold."""
    f = [500000.0 ** (-2.0 * i / c["rot"]) / (8.0 if i >= c["rot"] // 4 else 1.0) for i in range(c["rot"] // 2)]
    return torch.tensor(f, dtype=torch.float32, device="cuda")


def _cache(g, num_pages, Hkv, tpp):
    """Codes and scales of blocks whose values have a standard deviation between a half and two."""
    codes = (torch.randn(num_pages * Hkv * tpp * 2 * TILE * D, device="cuda", generator=g, dtype=torch.bfloat16) * 100)
    codes = codes.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    scales = torch.randint(127 - 8, 127 - 5, (num_pages * Hkv * tpp * 2,), device="cuda", generator=g).to(torch.uint8)
    return codes, scales


def prepare(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = random.Random(seed)
    s = dict(c)
    B, Hkv, ps = c["B"], c["Hkv"], c["ps"]
    lens = _lengths(c)
    n, first = [1] * B, [x - 1 for x in lens]
    if c["kind"] in ("chunk", "write"):
        n, first = _chunks(c)
        s["cu"] = _ints([sum(n[:r]) for r in range(B + 1)])
        s["most"] = max(n)
    if c["kind"] in ("append", "write"):
        # only the pages that get tokens exist in the pool; earlier ones are not looked at
        spans = [(f // ps, _pages(x, ps)) for f, x in zip(first, lens)]
    else:
        spans = [(0, _pages(x, ps)) for x in lens]
    maxp = _pages(max(lens), ps) + 1
    num_pages = sum(b - a for a, b in spans) + 3
    ids = list(range(num_pages))
    rnd.shuffle(ids)
    table = torch.full((B, maxp), -1, dtype=torch.int32)
    for r, (a, b) in enumerate(spans):
        table[r, a:b] = torch.tensor([ids.pop() for _ in range(b - a)], dtype=torch.int32)
    T = sum(n)
    s["pool"], s["scales"] = _cache(g, num_pages, Hkv, ps // TILE)
    s.update(num_pages=num_pages, table=table.cuda(), lens=_ints(lens), T=T, longest=max(lens),
             q=torch.randn(T, c["Hq"], D, device="cuda", generator=g).to(torch.bfloat16))
    if c["kind"] in ("append", "write"):
        s.update(first=_ints(first), freqs=_freqs(c), rot_scale=1.1,
                 k=torch.randn(T, Hkv, D, device="cuda", generator=g).to(torch.bfloat16),
                 v=torch.randn(T, Hkv, D, device="cuda", generator=g).to(torch.bfloat16),
                 q_out=torch.empty(T, c["Hq"], D, device="cuda", dtype=torch.bfloat16))
    else:
        s.update(sm_scale=D ** -0.5, lse=torch.empty(T, c["Hq"], device="cuda"),
                 out=torch.empty(T, c["Hq"], D, device="cuda",
                                 dtype=torch.float32 if c["kind"] == "decode" else torch.bfloat16))
    return s


# --------------------------------------------------------------- plain forms
def _blocks(s):
    """Codes as [pages][Hkv][tiles][2][16 D] and scales as [pages][Hkv][tiles][2]."""
    shape = (s["num_pages"], s["Hkv"], s["ps"] // TILE, 2)
    return s["pool"].view(torch.float8_e4m3fn).view(*shape, TILE * D), s["scales"].view(shape)


def _contexts(s):
    """K and V of each request in 32 bits, [B, Hkv, tokens, D]; what lies behind a context is 0."""
    codes, scales = _blocks(s)
    at = s["table"].clamp(min=0).long()
    x = codes[at].float() * torch.exp2(scales[at].float() - 127).unsqueeze(-1)
    B, p, h, t = x.shape[:4]
    k = x[..., 0, :].reshape(B, p, h, t, TILE, D).movedim(1, 2).reshape(B, h, -1, D)
    v = x[..., 1, :].reshape(B, p, h, t, D, TILE).transpose(-1, -2).movedim(1, 2).reshape(B, h, -1, D)
    k, v = k[:, :, :s["longest"]], v[:, :, :s["longest"]]
    there = torch.arange(s["longest"], device=v.device) < s["lens"].view(B, 1)
    return k, torch.where(there.view(B, 1, -1, 1), v, 0.0)


def _plain_attend(s):
    """q [B, n, Hq, D] over the contexts: query i of request r sees limit[r, i] tokens."""
    B, Hkv = s["B"], s["Hkv"]
    G = s["Hq"] // Hkv
    k, v = _contexts(s)
    if s["kind"] == "decode":
        q, limit = s["q"].float().unsqueeze(1), s["lens"].view(B, 1)
    else:
        i = torch.arange(s["most"], device=k.device)
        n = (s["cu"][1:] - s["cu"][:-1]).view(B, 1)
        rows = (s["cu"][:-1].view(B, 1) + i).clamp(max=s["T"] - 1)
        q = s["q"][rows].float()
        limit = s["lens"].view(B, 1) - n + 1 + i if s["causal"] else s["lens"].view(B, 1).expand(B, s["most"])
    N = q.shape[1]
    q = q.view(B, N, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, N * G, D)
    x = torch.matmul(q, k.transpose(-1, -2)).mul_(s["sm_scale"])
    hidden = torch.arange(k.shape[2], device=k.device) >= limit.repeat_interleave(G, 1).unsqueeze(-1)
    x.masked_fill_(hidden.unsqueeze(1), -math.inf)
    m = x.amax(-1, keepdim=True).clamp_(min=torch.finfo(torch.float32).min)
    p = torch.exp_(x.sub_(m))
    z = p.sum(-1, keepdim=True)
    out = torch.matmul(p, v) / torch.where(z > 0, z, 1.0)
    out = out.view(B, Hkv, N, G, D).permute(0, 2, 1, 3, 4).reshape(B, N, -1, D)
    lse = (m + torch.log(z)).view(B, Hkv, N, G).permute(0, 2, 1, 3).reshape(B, N, -1)
    if s["kind"] == "decode":
        return {"out": out[:, 0], "lse": lse[:, 0]}
    mine = i < n
    return {"out": out[mine].to(torch.bfloat16), "lse": lse[mine]}


def _rotated(s, x, pos):
    """x [tokens][heads][D] in 32 bits with its first `rot` values rotated; angles in 64 bits."""
    rot = s["rot"]
    angle = pos.double().view(-1, 1, 1) * s["freqs"].double()
    cos, sin = (torch.cos(angle) * s["rot_scale"]).float(), (torch.sin(angle) * s["rot_scale"]).float()
    x = x.float()
    if s["interleaved"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((y, x[..., rot:]), -1)


def _exponent(top):
    """The least e with top <= 448 * 2^e, within the scales' range."""
    m, x = torch.frexp(top)
    return torch.where(top > 0, x - 9 + (m > 0.875), LOW).clamp(LOW, HIGH)


def _plain_write(s):
    if s["kind"] == "append":
        r, pos = torch.arange(s["B"], device="cuda"), (s["lens"] - 1).long()
    else:
        t = torch.arange(s["tokens"], device="cuda")
        r = torch.searchsorted(s["cu"], t.to(torch.int32), right=True) - 1
        pos = t - s["cu"][r] + s["first"][r]
    P, Hkv, tpp = s["num_pages"], s["Hkv"], s["ps"] // TILE
    tile = s["table"][r, pos // s["ps"]].long() * tpp + pos % s["ps"] // TILE  # of the pool
    slot = pos % TILE
    kv = torch.stack((_rotated(s, s["k"], pos), s["v"].float()), 2)  # [tokens, Hkv, 2, D]
    # exponents: of the blocks' new values, and of the old ones where a block holds some
    need = _exponent(kv.abs().amax(-1)).view(-1, Hkv * 2)
    most = torch.full((P * tpp, Hkv * 2), LOW, dtype=need.dtype, device="cuda")
    most.scatter_reduce_(0, tile.view(-1, 1).expand_as(need), need, "amax")
    start = torch.full((P * tpp,), TILE, dtype=slot.dtype, device="cuda").scatter_reduce_(0, tile, slot, "amin")
    touched, most = (start < TILE).view(P, 1, tpp, 1), most.view(P, tpp, Hkv, 2).movedim(1, 2)
    start = start.view(P, 1, tpp, 1)
    codes, scales = _blocks(s)
    old = scales.int() - 127
    e = torch.where(touched, torch.where(start > 0, torch.maximum(old, most), most), old)
    # codes before the new tokens: the same values under the new scale
    x = torch.exp2((old - e).float()).unsqueeze(-1) * codes.float()
    at = torch.arange(TILE * D, device="cuda")
    token = torch.stack((at // D, at % TILE))  # of a K block, and of a V block
    codes.copy_(torch.where((token < start.unsqueeze(-1)) & touched.unsqueeze(-1), x, codes.float()).to(torch.float8_e4m3fn))
    scales.copy_((e + 127).to(torch.uint8))
    # the new tokens
    page, tile = tile // tpp, tile % tpp
    y = (kv * torch.exp2(-e.float())[page, :, tile].unsqueeze(-1)).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    blocks = s["pool"].view(P, Hkv, tpp, 2, TILE * D)
    blocks[..., 0, :].view(P, Hkv, tpp, TILE, D)[page, :, tile, slot] = y[:, :, 0]
    blocks[..., 1, :].view(P, Hkv, tpp, D, TILE)[page, :, tile, :, slot] = y[:, :, 1]
    s["q_out"] = _rotated(s, s["q"], pos).to(torch.bfloat16)


# --------------------------------------------------------------------- a pass
def run(s):
    kind = s["kind"]
    geo = dict(Hkv=s["Hkv"], page_size=s["ps"], num_pages=s["num_pages"])
    if kind in ("append", "write"):
        if own:
            import fp8_paged_kv_gb300 as fpk
            rope = dict(rot_dim=s["rot"], interleaved=s["interleaved"], rot_scale=s["rot_scale"], **geo)
            if kind == "append":
                fpk.fpk_rope_append_fp8_block(s["q"], s["k"], s["v"], s["freqs"], s["q_out"], s["pool"], s["scales"],
                                              s["table"], s["lens"], **rope)
            else:
                fpk.fpk_rope_prefill_fp8_block(s["q"], s["k"], s["v"], s["cu"], s["first"], s["freqs"], s["q_out"],
                                               s["pool"], s["scales"], s["table"], **rope)
        else:
            _plain_write(s)
        return {"q": s["q_out"], "codes": s["pool"].view(torch.float8_e4m3fn),
                "scales": s["scales"].view(torch.float8_e8m0fnu)}
    if not own:
        return _plain_attend(s)
    import fp8_paged_kv_gb300 as fpk
    if kind == "decode":
        if "ws" not in s:  # a workspace that the program keeps
            s["ws"] = torch.zeros(fpk.fpk_decode_workspace_bytes(s["B"], s["Hq"], s["Hkv"]), dtype=torch.uint8, device="cuda")
        fpk.fpk_paged_decode_attn_fp8_block(s["q"], s["pool"], s["scales"], s["table"], s["lens"], None, s["out"], s["lse"],
                                            s["ws"], sm_scale=s["sm_scale"], **geo)
    else:
        if "ws" not in s:
            s["ws"] = torch.zeros(fpk.fpk_prefill_workspace_bytes(s["B"], s["T"], s["Hq"], s["Hkv"]), dtype=torch.uint8, device="cuda")
        fpk.fpk_paged_prefill_attn_fp8_block(s["q"], s["cu"], s["pool"], s["scales"], s["table"], s["lens"], None, s["out"],
                                             s["lse"], s["ws"], causal=s["causal"], sm_scale=s["sm_scale"], **geo)
    return {"out": s["out"], "lse": s["lse"]}


# ------------------------------------------------------- the definition, 64 bits
def _exact_rope(c, s):
    n, first = ([1] * c["B"], [x - 1 for x in _lengths(c)]) if c["kind"] == "append" else _chunks(c)
    pos = [f + i for k, f in zip(n, first) for i in range(k)]
    turn = torch.tensor(pos, dtype=torch.float64, device="cuda").view(-1, 1) * s["freqs"].double()
    unit = s["rot_scale"] * torch.polar(torch.ones_like(turn), turn).unsqueeze(1)
    x, rot = s["q"].double(), c["rot"]
    if c["interleaved"]:
        z = torch.complex(x[..., 0:rot:2].contiguous(), x[..., 1:rot:2].contiguous()) * unit
        x[..., 0:rot:2], x[..., 1:rot:2] = z.real, z.imag
    else:
        z = torch.complex(x[..., :rot // 2].contiguous(), x[..., rot // 2:rot].contiguous()) * unit
        x[..., :rot // 2], x[..., rot // 2:rot] = z.real, z.imag
    return {"q": x, "codes": None, "scales": None}  # rounded codes, and their powers of two


def exact(c, seed):
    s = prepare(c, seed)
    if c["kind"] in ("append", "write"):
        return _exact_rope(c, s)
    Hkv, G, lens = c["Hkv"], c["Hq"] // c["Hkv"], _lengths(c)
    n = [1] * c["B"] if c["kind"] == "decode" else _chunks(c)[0]
    codes, scales = _blocks(s)
    scale = torch.pow(2.0, scales.double() - 127)
    out = torch.zeros(sum(n), Hkv, G, D, dtype=torch.float64, device="cuda")
    lse = torch.full((sum(n), Hkv, G), -math.inf, dtype=torch.float64, device="cuda")
    q = s["q"].double().view(-1, Hkv, G, D)
    row = 0
    for r, L in enumerate(lens):
        ids = s["table"][r, :_pages(L, c["ps"])].long()
        for h in range(Hkv if n[r] else 0):
            x = codes[ids, h].double() * scale[ids, h].unsqueeze(-1)
            k = x[:, :, 0].reshape(-1, D)[:L]
            v = x[:, :, 1].reshape(-1, D, TILE).transpose(1, 2).reshape(-1, D)[:L]
            for a in range(0, n[r], 2048):  # some query tokens at a time
                b = min(n[r], a + 2048)
                e = (q[row + a:row + b, h].reshape(-1, D) @ k.T).mul_(s["sm_scale"]).view(b - a, G, L)
                if c.get("causal"):
                    last = L - n[r] + torch.arange(a, b, device="cuda")
                    e.masked_fill_((torch.arange(L, device="cuda") > last.view(-1, 1)).unsqueeze(1), -math.inf)
                z = torch.logsumexp(e, -1)
                lse[row + a:row + b, h] = z
                out[row + a:row + b, h] = torch.exp_(e.sub_(z.unsqueeze(-1))) @ v
        row += n[r]
    return {"out": out.view(sum(n), -1, D), "lse": lse.view(sum(n), -1)}
