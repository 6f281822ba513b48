"""64-bit reference of attention over caches with block scales on the GPU, for every row of a call."""
import math

import numpy as np
import torch

from block_helpers import D, TILE, context


def check_rows(s, got, *, causal, sm, dead=(), weight=2.0 ** -11, floor=2.0 ** -25):
    """Every row of a call (s: a scene of test_gpu_block_attention, got: (out, lse)) within that file's bounds.

    causal None: decode.  weight, floor: what a softmax weight may be off by, relative to it, and to the largest weight
    times V's scale.
    Returns the largest share of its bound that a result uses."""
    G, worst = s["Hq"] // s["Hkv"], 0.0
    up = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731
    q, out, lse = s["q"].cuda().double(), up(got[0]), up(got[1])
    for r, n in enumerate(s["counts"]):
        L, a = int(s["lens"][r]), int(s["cu"][r])
        o, l_ = out[a:a + n], lse[a:a + n]
        if r in dead or L <= 0:
            assert torch.all(o == 0) and torch.all(l_ == -torch.inf), f"dead request {r}"
            continue
        limit = torch.arange(n, device="cuda") + (L - n + 1) if causal else torch.full((n,), L, device="cuda")
        limit = limit.clamp(min=0).repeat_interleave(G)
        none = limit == 0
        for h in range(s["Hkv"] if n else 0):
            k, v, ev = (up(x) for x in context(s["pool"], s["scales"], s["table"][r], L, h, s["ps"]))
            x = q[a:a + n, h * G:(h + 1) * G].reshape(-1, D)
            oh, lh = o[:, h * G:(h + 1) * G].reshape(-1, D), l_[:, h * G:(h + 1) * G].reshape(-1)
            assert torch.all(oh[none] == 0) and torch.all(lh[none] == -torch.inf), f"request {r}, head {h}: rows that see nothing"
            hidden = torch.arange(L, device="cuda") >= limit.unsqueeze(1)
            e = (x @ k.T * sm).masked_fill(hidden, -torch.inf)
            z = torch.logsumexp(e, 1)
            p = torch.exp(e - torch.where(none, 0.0, z).unsqueeze(1))
            ref, size = p @ v, p @ v.abs()
            unit = (p * torch.exp2(ev.double())).amax(1)
            d = 2.0 ** -17 * (x.abs() @ k.abs().T * abs(sm)).masked_fill(hidden, 0.0).amax(1) + 2.0 ** -20
            if causal is not None:
                d = d + 2.0 ** -17 * abs(sm) * x.abs().amax(1) * k.abs().sum(1).amax()
            w = (2 * d + 2.0 ** -20 + L * 2.0 ** -24 + weight).unsqueeze(1) * size
            w = w + (448.0 * L * floor * unit).unsqueeze(1) + (0.0 if causal is None else 2.0 ** -8) * ref.abs() + 1e-30
            share = ((oh - ref).abs() / w)[~none]
            assert torch.all(share <= 1), f"request {r}, head {h}: {int((share > 1).sum())} of {share.numel()}, worst {share.max():.2f} of its bound"
            le = ((lh - z).abs() / (d + L * 2.0 ** -24 + 2.0 ** -20 + 2.0 ** -23 * z.abs()))[~none]
            assert torch.all(le <= 1), f"request {r}, head {h}: lse"
            worst = max(worst, float(share.max()) if share.numel() else 0.0)
    return worst


def blocks(s, tensor, kv):
    """K (kv 0) or V (kv 1) of a scene as [pages][heads][tiles][16 tokens][D]: a view that writes through."""
    x = tensor[..., kv, :]
    return x.reshape(*x.shape[:-1], TILE, D) if kv == 0 else np.swapaxes(x.reshape(*x.shape[:-1], D, TILE), -1, -2)


def codes(x):
    return torch.tensor(x).to(torch.float8_e4m3fn).view(torch.uint8).item()


def cancelling(s):
    """Tokens in turn of weight 1 and p, of values x and -y with x / y near p: what is left is the error of p, which
    lies 0.15 of an f16 step above a value halfway between two.  Returns the scale of the scores."""
    x, y, p, key = 11.0, 13.0, 3465.3 / 4096, 8.0
    s["scales"][...] = 127
    k, v = blocks(s, s["pool"], 0), blocks(s, s["pool"], 1)
    k[...] = 0
    k[..., 1::2, 0] = codes(-key)
    for i in range(4):
        v[..., 0::2, i::4], v[..., 1::2, i::4] = codes(x * 2.0 ** (i - 2)), codes(-y * 2.0 ** (i - 2))
    s["q"].zero_()
    s["q"][..., 0] = 1.0
    return -math.log(p) / key


def outlier_block(s, far):
    """The second tile of each request has values in one dim alone, under a V scale 2^far as large as the others'."""
    v = blocks(s, s["pool"], 1)
    v &= 0x7F  # (what is left where values do not cancel)
    for r in range(len(s["counts"])):
        page, tile = s["table"][r, TILE // s["ps"]], TILE % s["ps"] // TILE
        v[page, :, tile] = 0
        v[page, :, tile, :, 5] = codes(448.0)
        s["scales"][page, :, tile, 1] += far


def sink(s, far):
    """Each request's first token has a weight 2^far as large as every other's, and no value.  Returns the scale of the
    scores."""
    k, v = blocks(s, s["pool"], 0), blocks(s, s["pool"], 1)
    v &= 0x7F
    k[...] = 0
    for r in range(len(s["counts"])):
        page = s["table"][r, 0]
        k[page, :, 0, 0, 0] = codes(8.0)
        s["scales"][page, :, 0, 0] = 127
        v[page, :, 0, 0] = 0
    s["q"].zero_()
    s["q"][..., 0] = 1.0
    return far * math.log(2) / 8.0
