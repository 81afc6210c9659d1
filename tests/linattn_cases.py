"""Inputs of linear attention's gradients with a decay for each token, and the cases whose decays'
gradient is checked by linattn_spread."""
import torch

SPREAD = [
    # dtype, b, L, G, H, dk, dv, first and last states, lengths
    ("bf16", 1, 64, 2, 2, 64, 64, True, None),
    ("bf16", 1, 65, 1, 2, 64, 64, True, None),
    ("bf16", 2, 257, 2, 6, 72, 200, True, None),
    ("bf16", 1, 300, 4, 4, 128, 128, False, None),
    ("bf16", 1, 150, 2, 2, 256, 256, True, None),
    ("bf16", 1, 1100, 1, 2, 128, 128, True, None),         # segments
    ("bf16", 4, 900, 1, 2, 72, 136, True, [900, 0, 65, 320]),
    ("fp32", 2, 17, 2, 2, 24, 16, True, None),
    ("fp32", 1, 257, 1, 3, 72, 200, True, None),
    ("fp32", 1, 150, 1, 2, 256, 256, True, None),
    ("fp32", 3, 600, 1, 2, 64, 48, False, [1, 600, 449]),
]


def inputs(case, dev, seed=0, rate=0.3):
    dtype, b, L, G, H, dk, dv, state, _ = case
    gen = torch.Generator().manual_seed(seed)
    td = {"fp32": torch.float32, "bf16": torch.bfloat16}[dtype]
    rnd = lambda *s: torch.randn(*s, generator=gen)
    d = dict(do=rnd(b, L, H, dv), q=rnd(b, L, G, dk), k=rnd(b, L, G, dk), v=rnd(b, L, H, dv),
             g=-rate * torch.rand(b, L, H, generator=gen) ** 3)
    d = {n: t.to(td).to(dev) for n, t in d.items()}
    for n in ("h0", "dhT"):
        d[n] = rnd(b, H, dv, dk).to(dev) if state else None
    return d


# One chunk, where nothing but the output's own rounding is as coarse as bf16: its own pairs, reads of
# a large first state, writes that a large last state's gradient reads.
ONE_CHUNK = ("inside", "read", "written")


def one_chunk(part, dev, seed):
    d = inputs(("bf16", 8, 64, 2, 4, 64, 64, True, None), dev, seed)
    d["h0"] = 32 * d["h0"] if part == "read" else None
    d["dhT"] = 32 * d["dhT"] if part == "written" else None
    return d
