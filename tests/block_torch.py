"""64-bit reference of attention over caches with block scales on the GPU, for every row of a call."""
import numpy as np
import torch

from block_helpers import D, context


def check_rows(s, got, *, causal, sm, dead=(), weight=2.0 ** -11, floor=2.0 ** -25):
    """Every row of a call (s: a scene of test_gpu_block_attention, got: (out, lse)) within that file's bounds.

    weight, floor: what a softmax weight may be off by, relative to it, and to the largest weight times V's scale.
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
            d = d + 2.0 ** -17 * abs(sm) * x.abs().amax(1) * k.abs().sum(1).amax()
            w = (2 * d + 2.0 ** -20 + L * 2.0 ** -24 + weight).unsqueeze(1) * size
            w = w + (448.0 * L * floor * unit).unsqueeze(1) + 2.0 ** -8 * ref.abs() + 1e-30
            share = ((oh - ref).abs() / w)[~none]
            assert torch.all(share <= 1), f"request {r}, head {h}: {int((share > 1).sum())} of {share.numel()}, worst {share.max():.2f} of its bound"
            le = ((lh - z).abs() / (d + L * 2.0 ** -24 + 2.0 ** -20 + 2.0 ** -23 * z.abs()))[~none]
            assert torch.all(le <= 1), f"request {r}, head {h}: lse"
            worst = max(worst, float(share.max()) if share.numel() else 0.0)
    return worst
