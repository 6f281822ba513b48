"""What is measured of three operators around the paged KV cache: their plain
forms in elementary torch operations, the library's calls, and the cases.

* prefix: decode attention of a batch whose requests share long prefixes.
* fork, compact: requests forked from one another, and pages moved to the
  front of the pool, with tables and tags kept right.
* rope: rotary positions for queries and keys, the keys written to the cache
  with the values (one token per request, or whole chunks of prompts).
"""
import math
import random

import torch

own = False

D = 128
TILE = 16
NAN_FREE_SCALE = 0.02  # a per-tensor scale of N(0, 1) keys and values: 5 sigma lands at 250 of 448


# ------------------------------------------------------------------- cases
def listed():
    return [
        # a few samples of a short prompt: the smallest calls, latency counts
        dict(name="prefix_fp8_b4_512", kind="prefix", fp8=True, B=4, Hq=64, Hkv=8, ps=16, groups=1, prefix=512, suffix=64),
        # the benchmark's batch and context, one prompt for all, answers of up to 512 tokens
        dict(name="prefix_fp8_b32_8k", kind="prefix", fp8=True, B=32, Hq=64, Hkv=8, ps=16, groups=1, prefix=8192, suffix=512),
        # several system prompts of uneven length, five query heads to a kv head, the bf16 cache
        dict(name="prefix_bf16_b61_groups", kind="prefix", fp8=False, B=61, Hq=40, Hkv=8, ps=64, groups=5, prefix=9001, suffix=700),
        # a large evaluation batch over one long document
        dict(name="prefix_fp8_b128_32k", kind="prefix", fp8=True, B=128, Hq=64, Hkv=8, ps=64, groups=1, prefix=32768, suffix=512),
        # four samples of one request, one layer: a fork's latency
        dict(name="fork_fp8_n4_l1", kind="fork", fp8=True, n=4, L=1000, Hkv=8, ps=16, layers=1),
        # 64 samples of one request through 32 layers, wide pages
        dict(name="fork_bf16_n64_l32", kind="fork", fp8=False, n=64, L=8219, Hkv=8, ps=64, layers=32),
        # a few pages, one layer
        dict(name="compact_fp8_m64_l1", kind="compact", fp8=True, moves=64, B=32, max_pages=512, Hkv=8, ps=16, layers=1),
        # a pool shrunk by a quarter, eight layers at once
        dict(name="compact_fp8_m4001_l8", kind="compact", fp8=True, moves=4001, B=64, max_pages=256, Hkv=8, ps=16, layers=8),
        # one request's next token
        dict(name="rope_append_fp8_b1", kind="append", fp8=True, B=1, Hq=64, Hkv=8, ps=16, rot=128, interleaved=False, pos=8191),
        # a full decode batch, interleaved pairs on half of the head, far positions
        dict(name="rope_append_bf16_b64", kind="append", fp8=False, B=64, Hq=64, Hkv=8, ps=64, rot=64, interleaved=True, pos=131071),
        # a prefill batch of prompts from their start
        dict(name="rope_prefill_fp8_16k", kind="prefill", fp8=True, B=4, tokens=16384, Hq=64, Hkv=8, ps=16, rot=128, interleaved=False, pos=0),
        # ragged chunks of long prompts, interleaved pairs on part of the head
        dict(name="rope_prefill_bf16_chunks", kind="prefill", fp8=False, B=7, tokens=2011, Hq=40, Hkv=8, ps=64, rot=96, interleaved=True, pos=100000),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["prefix", "prefix", "prefix", "fork", "compact", "append", "prefill"])
    fp8 = rng.random() < 0.6
    ps = rng.choice([16, 16, 32, 64, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    Hq = Hkv * rng.choice([1, 4, 5, 7, 8])
    if kind == "prefix":
        B = _log_int(rng, 2, 128)
        return dict(kind=kind, fp8=fp8, B=B, Hq=Hq, Hkv=Hkv, ps=ps, groups=rng.randint(1, min(B, 4)),
                    prefix=_log_int(rng, 64, 16384), suffix=_log_int(rng, 1, 1024))
    if kind == "fork":
        return dict(kind=kind, fp8=fp8, n=_log_int(rng, 1, 48), L=_log_int(rng, 1, 8192), Hkv=Hkv, ps=ps,
                    layers=_log_int(rng, 1, 24))
    if kind == "compact":
        layers = _log_int(rng, 1, 8)
        return dict(kind=kind, fp8=fp8, moves=_log_int(rng, 1, 16384 // (ps * layers)), B=_log_int(rng, 1, 64),
                    max_pages=_log_int(rng, 16, 512), Hkv=Hkv, ps=ps, layers=layers)
    rot, inter = rng.choice([32, 64, 96, 128]), rng.random() < 0.5
    if kind == "append":
        return dict(kind=kind, fp8=fp8, B=_log_int(rng, 1, 256), Hq=Hq, Hkv=Hkv, ps=ps, rot=rot, interleaved=inter,
                    pos=_log_int(rng, 1, 131071))
    B = _log_int(rng, 1, 16)
    return dict(kind=kind, fp8=fp8, B=B, tokens=_log_int(rng, 4 * B, 8192), Hq=Hq, Hkv=Hkv, ps=ps, rot=rot,
                interleaved=inter, pos=_log_int(rng, 1, 100000))


# ------------------------------------------------ shapes that a case stands for
def _pages(tokens, ps):
    return -(-tokens // ps)


def _prefix_shape(c):
    """(first request of each group and B, prefix of each group, context of each request)"""
    n, B = c["groups"], c["B"]
    starts = [B * g * (g + 1) // (n * (n + 1)) for g in range(n + 1)]
    pre = [max(1, c["prefix"] - g * (c["prefix"] // (n + 1))) for g in range(n)]
    shared = [p // c["ps"] * c["ps"] for p in pre]  # whole pages are shared
    lens = [0] * B
    for g in range(n):
        for r in range(starts[g], starts[g + 1]):
            lens[r] = pre[g] + 1 + (131 * r) % c["suffix"]
    return starts, pre, shared, lens


def _prefill_shape(c):
    """(tokens of each request's chunk, position of its first token)"""
    B, T = c["B"], c["tokens"]
    cut = [T * r * (r + 2) // (B * (B + 2)) for r in range(B + 1)]
    return [b - a for a, b in zip(cut, cut[1:])], [c["pos"] * (r + 1) // B for r in range(B)]


def work(c):
    el = 1 if c["fp8"] else 2
    if c["kind"] == "prefix":
        starts, _, shared, lens = _prefix_shape(c)
        kv = sum(shared) + sum(lens) - sum(s * (b - a) for s, a, b in zip(shared, starts, starts[1:]))
        return {"bytes": kv * c["Hkv"] * 2 * D * el + c["B"] * c["Hq"] * (4 * D + 4), "flops": 4 * D * c["Hq"] * sum(lens)}
    if c["kind"] == "fork":
        tiles = -(-(c["L"] % c["ps"]) // TILE)
        # one parent: its page in use is read once, and written n times
        return {"bytes": (1 + c["n"]) * c["layers"] * c["Hkv"] * tiles * 2 * TILE * D * el + 8 * (1 + c["n"]) * _pages(c["L"], c["ps"])}
    if c["kind"] == "compact":
        return {"bytes": 2 * c["moves"] * c["layers"] * c["Hkv"] * c["ps"] * 2 * D * el + 8 * c["B"] * c["max_pages"]}
    T = c["B"] if c["kind"] == "append" else c["tokens"]
    return {"bytes": T * D * (4 * c["Hq"] + c["Hkv"] * 2 * (2 + el)), "flops": 3 * T * (c["Hq"] + c["Hkv"]) * c["rot"]}


# ----------------------------------------------------------------- preparing
def _pool(g, fp8, *shape):
    x = torch.randn(*shape, device="cuda", generator=g, dtype=torch.bfloat16)
    return (x / NAN_FREE_SCALE).to(torch.float8_e4m3fn).view(torch.uint8) if fp8 else x


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _freqs(c):
    """Inverse frequencies of a long context: base 500000, the slow half of them stretched eightfold."""
    f = [500000.0 ** (-2.0 * i / c["rot"]) / (8.0 if i >= c["rot"] // 4 else 1.0) for i in range(c["rot"] // 2)]
    return torch.tensor(f, dtype=torch.float32, device="cuda")


def prepare(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = random.Random(seed)
    s = dict(c)
    Hkv, ps, el = c["Hkv"], c["ps"], 1 if c["fp8"] else 2
    s["k_scale"] = torch.tensor([NAN_FREE_SCALE], device="cuda")
    s["v_scale"] = torch.tensor([NAN_FREE_SCALE * 1.25], device="cuda")
    if c["kind"] == "prefix":
        starts, pre, shared, lens = _prefix_shape(c)
        maxp = _pages(max(lens), ps) + 1
        need = sum(sh // ps for sh in shared) + sum(_pages(x, ps) for x in lens)
        num_pages = need + 7
        ids = list(range(num_pages))
        rnd.shuffle(ids)
        table = torch.full((c["B"], maxp), -1, dtype=torch.int32)
        for i, sh in enumerate(shared):
            head = [ids.pop() for _ in range(sh // ps)]
            for r in range(starts[i], starts[i + 1]):
                row = head + [ids.pop() for _ in range(_pages(lens[r], ps) - len(head))]
                table[r, :len(row)] = torch.tensor(row, dtype=torch.int32)
        s.update(num_pages=num_pages, table=table.cuda(), lens=_ints(lens), starts=_ints(starts), pre=_ints(pre),
                 pool=_pool(g, c["fp8"], num_pages * Hkv * ps * 2 * D),
                 q=torch.randn(c["B"], c["Hq"], D, device="cuda", generator=g).to(torch.bfloat16),
                 out=torch.empty(c["B"], c["Hq"], D, device="cuda", dtype=torch.bfloat16),
                 lse=torch.empty(c["B"], c["Hq"], device="cuda"), sm_scale=D ** -0.5)
        return s
    if c["kind"] == "fork":
        # row 0 is the parent, rows 1..n its children to be
        pages = _pages(c["L"], ps)
        num_pages = pages + c["n"] + 5
        ids = list(range(num_pages))
        rnd.shuffle(ids)
        table = torch.full((c["n"] + 1, pages + 3), -1, dtype=torch.int32)
        table[0, :pages] = torch.tensor(ids[:pages], dtype=torch.int32)
        live = torch.randint(0, 1 << 30, (num_pages,), device="cuda", generator=g, dtype=torch.int32)
        s["table"] = table.cuda()
        s["tags"] = torch.where(s["table"] >= 0, live[s["table"].clamp(min=0).long()], 0)
        s.update(num_pages=num_pages, live=live, lens=_ints([c["L"]] + [0] * c["n"]), parent=_ints([0] * c["n"]),
                 child=_ints(list(range(1, c["n"] + 1))), fresh=_ints(ids[pages:pages + c["n"]]),
                 abort=torch.zeros(c["n"] + 1, dtype=torch.uint8, device="cuda"),
                 pool=_pool(g, c["fp8"], c["layers"], num_pages * Hkv * ps * 2 * D))
        return s
    if c["kind"] == "compact":
        # the moved pages lie behind a pool of four times as many; the rows hold moved and unmoved ones
        m = c["moves"]
        num_pages = 4 * m
        front, back = list(range(3 * m)), list(range(3 * m, 4 * m))
        rnd.shuffle(front)
        dst, keep = front[:m], front[m:]
        live = torch.randint(0, 1 << 30, (num_pages,), device="cuda", generator=g, dtype=torch.int32)
        held = back + keep
        rnd.shuffle(held)
        n = c["B"] * c["max_pages"]
        table = torch.tensor((held * (n // len(held) + 1))[:n], dtype=torch.int32).view(c["B"], c["max_pages"]).cuda()
        lens = [max(1, c["max_pages"] * ps - (977 * r) % (c["max_pages"] * ps)) for r in range(c["B"])]
        s.update(num_pages=num_pages, live=live, table=table, tags=live[table.long()], lens=_ints(lens),
                 there=(_ints(back), _ints(dst)), turn=0, pool=_pool(g, c["fp8"], c["layers"], num_pages * Hkv * ps * 2 * D))
        order = sorted(range(m), key=lambda i: dst[i])  # the way back, again in the order of the pages moved
        s["back"] = (_ints([dst[i] for i in order]), _ints([back[i] for i in order]))
        return s
    if c["kind"] == "append":
        lens = [max(1, c["pos"] + 1 - (1009 * r) % (c["pos"] + 1)) for r in range(c["B"])]
        T = c["B"]
    else:
        n, first = _prefill_shape(c)
        lens = [a + b for a, b in zip(n, first)]
        T = c["tokens"]
        s["cu"] = _ints([sum(n[:r]) for r in range(c["B"] + 1)])
        s["first"] = _ints(first)
    # only the pages that get tokens exist in the pool; earlier ones are not looked at
    maxp = _pages(max(lens), ps)
    table = torch.full((c["B"], maxp), -1, dtype=torch.int32)
    spans = [(first[r] // ps if c["kind"] == "prefill" else (lens[r] - 1) // ps, _pages(lens[r], ps)) for r in range(c["B"])]
    num_pages = sum(b - a for a, b in spans) + 3
    ids = list(range(num_pages))
    rnd.shuffle(ids)
    for r, (a, b) in enumerate(spans):
        table[r, a:b] = torch.tensor([ids.pop() for _ in range(b - a)], dtype=torch.int32)
    s.update(num_pages=num_pages, table=table.cuda(), lens=_ints(lens), freqs=_freqs(c), rot_scale=1.1,
             q=torch.randn(T, c["Hq"], D, device="cuda", generator=g).to(torch.bfloat16),
             k=torch.randn(T, Hkv, D, device="cuda", generator=g).to(torch.bfloat16),
             v=torch.randn(T, Hkv, D, device="cuda", generator=g).to(torch.bfloat16),
             q_out=torch.empty(T, c["Hq"], D, device="cuda", dtype=torch.bfloat16),
             pool=torch.zeros(num_pages * Hkv * ps * 2 * D * el, device="cuda", dtype=torch.uint8))
    if not c["fp8"]:
        s["pool"] = s["pool"].view(torch.bfloat16)
    return s


# --------------------------------------------------------------- plain forms
def _dense(s, x):
    """Values [..., pages, Hkv, tiles, 2, 16 * D] as K and V in 32 bits, [..., Hkv, tokens, D]."""
    if s["fp8"]:
        x = x.view(torch.float8_e4m3fn)
    lead, (p, h, t) = x.shape[:-5], x.shape[-5:-2]
    k = x[..., 0, :].float().reshape(*lead, p, h, t, TILE, D).movedim(-5, -4)
    v = x[..., 1, :].float().reshape(*lead, p, h, t, D, TILE).transpose(-1, -2).movedim(-5, -4)
    k, v = (y.reshape(*lead, h, p * t * TILE, D) for y in (k, v))
    return (k * s["k_scale"], v * s["v_scale"]) if s["fp8"] else (k, v)


def _plain_prefix(s):
    Hkv, B = s["Hkv"], s["B"]
    pages = s["pool"].view(s["num_pages"], Hkv, s["ps"] // TILE, 2, TILE * D)
    k, v = _dense(s, pages[s["table"].clamp(min=0).long()])
    q = s["q"].float().view(B, Hkv, s["Hq"] // Hkv, D)
    x = torch.matmul(q, k.transpose(-1, -2)) * s["sm_scale"]
    x = x.masked_fill(torch.arange(x.shape[-1], device=x.device) >= s["lens"].view(B, 1, 1, 1), -math.inf)
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - m)
    z = p.sum(-1, keepdim=True)
    out = torch.matmul(p, v) / z
    return {"out": out.reshape(B, -1, D).to(torch.bfloat16), "lse": (m + torch.log(z)).view(B, -1)}


def _tiled(s):
    return s["pool"].view(s["layers"], s["num_pages"], s["Hkv"], s["ps"] // TILE, 2 * TILE * D)


def _plain_fork(s):
    ps, table, tags = s["ps"], s["table"], s["tags"]
    parent, child, fresh = s["parent"].long(), s["child"].long(), s["fresh"].long()
    L = s["lens"][parent]
    at = (L // ps).long()  # the place of the page that is not full
    own_page = L % ps != 0
    cols = torch.arange(table.shape[1], device=table.device)
    held = cols < -(-L // ps).view(-1, 1)
    mine = own_page.view(-1, 1) & (cols == at.view(-1, 1))
    s["live"].index_add_(0, fresh, own_page.to(torch.int32))
    table[child] = torch.where(mine, s["fresh"].view(-1, 1), torch.where(held, table[parent], -1))
    tags[child] = torch.where(mine, s["live"][fresh].view(-1, 1), torch.where(held, tags[parent], 0))
    s["lens"][child] = L
    src = table[parent].gather(1, at.clamp(max=table.shape[1] - 1).view(-1, 1)).view(-1).clamp(min=0).long()
    pool = _tiled(s)
    used = torch.arange(ps // TILE, device=L.device) < -(-(L % ps) // TILE).view(-1, 1)
    pool[:, fresh] = torch.where(used.view(1, -1, 1, ps // TILE, 1), pool[:, src], pool[:, fresh])


def _plain_compact(s, src, dst):
    table, tags, live = s["table"], s["tags"], s["live"]
    to = torch.arange(s["num_pages"], dtype=torch.int32, device=live.device)
    to[src.long()] = dst
    held = torch.arange(table.shape[1], device=live.device) < -(-s["lens"] // s["ps"]).view(-1, 1)
    moved = held & (to[table.long()] != table) & (tags == live[table.long()])
    live[dst.long()] += 1
    table.copy_(torch.where(moved, to[table.long()], table))
    tags.copy_(torch.where(moved, live[table.long()], tags))
    pool = _tiled(s)
    pool[:, dst.long()] = pool[:, src.long()]


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


def _places(s):
    """Request and position of each token."""
    if s["kind"] == "append":
        return torch.arange(s["B"], device="cuda"), (s["lens"] - 1).long()
    t = torch.arange(s["tokens"], device="cuda")
    r = torch.searchsorted(s["cu"], t.to(torch.int32), right=True) - 1
    return r, t - s["cu"][r] + s["first"][r]


def _plain_rope(s):
    r, pos = _places(s)
    page = s["table"][r, pos // s["ps"]].long()
    tile, row = pos % s["ps"] // TILE, pos % TILE
    k, v = _rotated(s, s["k"], pos), s["v"].float()
    if s["fp8"]:
        k, v = ((x / sc).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
                for x, sc in ((k, s["k_scale"]), (v, s["v_scale"])))
    else:
        k, v = k.to(torch.bfloat16), v.to(torch.bfloat16)
    blocks = s["pool"].view(s["num_pages"], s["Hkv"], s["ps"] // TILE, 2, TILE * D)
    blocks[..., 0, :].view(s["num_pages"], s["Hkv"], s["ps"] // TILE, TILE, D)[page, :, tile, row] = k
    blocks[..., 1, :].view(s["num_pages"], s["Hkv"], s["ps"] // TILE, D, TILE)[page, :, tile, :, row] = v
    s["q_out"] = _rotated(s, s["q"], pos).to(torch.bfloat16)


# --------------------------------------------------------------------- a pass
def run(s):
    kind, fp8 = s["kind"], s["fp8"]
    geo = dict(Hkv=s["Hkv"], page_size=s["ps"], num_pages=s["num_pages"])
    scales = (s["k_scale"], s["v_scale"]) if fp8 else ()
    if kind == "prefix":
        if not own:
            return _plain_prefix(s)
        import fp8_paged_kv_gb300 as fpk
        if "ws" not in s:  # a workspace that the program keeps
            s["ws"] = torch.zeros(fpk.fpk_prefix_workspace_bytes(s["B"], s["Hq"], s["Hkv"]), dtype=torch.uint8, device="cuda")
        attn = fpk.fpk_paged_decode_attn_fp8_prefix if fp8 else fpk.fpk_paged_decode_attn_bf16_prefix
        attn(s["q"], s["pool"], *scales, s["table"], s["lens"], None, s["starts"], s["pre"], s["out"], s["lse"], s["ws"],
             sm_scale=s["sm_scale"], **geo)
        return {"out": s["out"], "lse": s["lse"]}
    if kind == "fork":
        if own:
            import fp8_paged_kv_gb300 as fpk
            fpk.fpk_kv_fork(s["pool"], s["table"], s["tags"], s["lens"], s["live"], s["abort"], s["parent"], s["child"],
                            s["fresh"], layers=s["layers"], D=D, **geo)
        else:
            _plain_fork(s)
        return {"pool": s["pool"] if fp8 else s["pool"].view(torch.int16), "table": s["table"], "tags": s["tags"],
                "lens": s["lens"], "live": s["live"], "abort": s["abort"]}
    if kind == "compact":
        src, dst = s["back"] if s["turn"] else s["there"]
        s["turn"] ^= 1
        if own:
            import fp8_paged_kv_gb300 as fpk
            fpk.fpk_kv_compact(s["pool"], s["table"], s["tags"], s["lens"], s["live"], src, dst, layers=s["layers"], D=D, **geo)
        else:
            _plain_compact(s, src, dst)
        return {"pool": s["pool"] if fp8 else s["pool"].view(torch.int16), "table": s["table"], "tags": s["tags"], "live": s["live"]}
    if own:
        import fp8_paged_kv_gb300 as fpk
        rope = dict(rot_dim=s["rot"], interleaved=s["interleaved"], rot_scale=s["rot_scale"], **geo)
        if kind == "append":
            call = fpk.fpk_rope_append_fp8 if fp8 else fpk.fpk_rope_append_bf16
            call(s["q"], s["k"], s["v"], s["freqs"], s["q_out"], s["pool"], *scales, s["table"], s["lens"], **rope)
        else:
            call = fpk.fpk_rope_prefill_fp8 if fp8 else fpk.fpk_rope_prefill_bf16
            call(s["q"], s["k"], s["v"], s["cu"], s["first"], s["freqs"], s["q_out"], s["pool"], *scales, s["table"], **rope)
    else:
        _plain_rope(s)
    return {"q": s["q_out"], "pool": s["pool"].view(torch.float8_e4m3fn) if fp8 else s["pool"]}


# ------------------------------------------------------- the definition, 64 bits
def exact(c, seed):
    if c["kind"] in ("fork", "compact"):
        return None  # copies and whole numbers
    s = prepare(c, seed)
    Hkv, ps = c["Hkv"], c["ps"]
    if c["kind"] == "prefix":
        G = c["Hq"] // Hkv
        pages = s["pool"].view(s["num_pages"], Hkv, ps // TILE, 2, TILE * D)

        def tokens(ids, h):
            x = pages[ids, h]
            x = (x.view(torch.float8_e4m3fn) if c["fp8"] else x).double()
            k = x[:, :, 0].reshape(-1, D)
            v = x[:, :, 1].reshape(-1, ps // TILE, D, TILE).transpose(2, 3).reshape(-1, D)
            return (k * s["k_scale"].double(), v * s["v_scale"].double()) if c["fp8"] else (k, v)

        starts, _, shared, lens = _prefix_shape(c)
        out = torch.empty(c["B"], Hkv, G, D, dtype=torch.float64, device="cuda")
        lse = torch.empty(c["B"], Hkv, G, dtype=torch.float64, device="cuda")
        q = s["q"].double().view(c["B"], Hkv, G, D)
        for i, n in enumerate(shared):
            rows = range(starts[i], starts[i + 1])
            for h in range(Hkv if rows else 0):
                kp, vp = tokens(s["table"][rows[0], :n // ps].long(), h)
                for r in rows:
                    ks, vs = tokens(s["table"][r, n // ps:_pages(lens[r], ps)].long(), h)
                    x = torch.cat((q[r, h] @ kp.T, q[r, h] @ ks[:lens[r] - n].T), 1) * s["sm_scale"]
                    lse[r, h] = torch.logsumexp(x, 1)
                    p = torch.exp(x - lse[r, h].unsqueeze(1))
                    out[r, h] = p[:, :n] @ vp + p[:, n:] @ vs[:lens[r] - n]
        return {"out": out.view(c["B"], -1, D), "lse": lse.view(c["B"], -1)}
    if c["kind"] == "append":
        pos = [int(x) - 1 for x in s["lens"].tolist()]
    else:
        n, first = _prefill_shape(c)
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
    return {"q": x, "pool": None}  # the pool holds rounded codes
