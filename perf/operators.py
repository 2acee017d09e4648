"""Cases of the 4-bit key/value cache: writing it, attending over it, weighing a prompt's keys and evicting slots.

A cache row (one token of one cache head, d = 64 or 128 channels) is d/2 bytes of signed 4-bit codes and d/32 bf16
scales, one per group of 32 consecutive channels: value = code * scale, code in [-7, 7].  Byte u*(d/16) + 2*g + h
(u < 8, g < d/32, h < 2) holds channel 32*g + 4*u + 2*h in its low nibble and the next channel in its high nibble.
"""
import math

import torch

own = False

GROUP = 32


# ------------------------------------------------------------------ the format, in elementary operations
def _pack(code):
    """codes [..., d] (whole numbers in [-7, 7]) -> packed bytes [..., d/2]."""
    d = code.shape[-1]
    c = (code.to(torch.int16) & 15).reshape(*code.shape[:-1], d // 32, 8, 2, 2).transpose(-4, -3)
    return (c[..., 0] | (c[..., 1] << 4)).to(torch.uint8).reshape(*code.shape[:-1], d // 2)


def _unpack(b):
    """packed bytes [..., d/2] -> codes [..., d] as float32."""
    d = 2 * b.shape[-1]
    c = b.reshape(*b.shape[:-1], 8, d // 32, 2)
    c = torch.stack((c & 15, c >> 4), dim=-1).transpose(-4, -3).reshape(*b.shape[:-1], d)
    return ((c ^ 8).to(torch.int8) - 8).to(torch.float32)


def _quantize(x):
    """bf16 [..., d] -> (codes [..., d] float32, scales [..., d/32] bf16)."""
    g = x.to(torch.float32).reshape(*x.shape[:-1], -1, GROUP)
    s = (g.abs().amax(dim=-1) / 7.0).to(torch.bfloat16)
    f = s.to(torch.float32)[..., None]
    c = torch.where(f > 0, torch.round(g / f).clamp(-7, 7), torch.zeros_like(g))
    return c.reshape(x.shape), s


def _values(codes, scales):
    """packed codes and scales -> float32 values [..., d]."""
    c = _unpack(codes)
    v = c.reshape(*c.shape[:-1], -1, GROUP) * scales.to(torch.float32)[..., None]
    return v.reshape(c.shape)


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one short conversation, lone request: latency
        {"name": "decode-short", "op": "decode", "B": 1, "Hq": 8, "Hkv": 2, "N": 333, "d": 64, "weights": False, "ragged": False},
        # the decode workload's batch with 4 query heads per cache head: throughput serving
        {"name": "decode-batch", "op": "decode", "B": 64, "Hq": 32, "Hkv": 8, "N": 8192, "d": 128, "weights": False, "ragged": False},
        # requests of different lengths, 8 heads per cache head, weights kept for eviction
        {"name": "decode-ragged-weights", "op": "decode", "B": 16, "Hq": 32, "Hkv": 4, "N": 16384, "d": 128, "weights": True, "ragged": True},
        # one long document, weights kept: few rows, a long axis
        {"name": "decode-long-weights", "op": "decode", "B": 1, "Hq": 32, "Hkv": 8, "N": 131072, "d": 128, "weights": True, "ragged": False},
        # one new token for each sequence of a batch
        {"name": "append-token", "op": "append", "B": 64, "Hkv": 8, "n": 1, "d": 128, "ragged": False},
        # a prompt's keys and values at once
        {"name": "append-prompt", "op": "append", "B": 4, "Hkv": 16, "n": 4096, "d": 128, "ragged": False},
        # chunks of different lengths, smaller heads
        {"name": "append-chunks", "op": "append", "B": 7, "Hkv": 3, "n": 1001, "d": 64, "ragged": True},
        # the last queries of a long prompt decide which of its keys stay
        {"name": "weigh-window", "op": "weigh", "B": 4, "Hq": 32, "Hkv": 8, "Nq": 32, "Nkv": 16384, "d": 128, "causal": True, "padded": False},
        # every query of a prompt (the prefill workload's length)
        {"name": "weigh-prompt", "op": "weigh", "B": 1, "Hq": 32, "Hkv": 8, "Nq": 4096, "Nkv": 4096, "d": 128, "causal": True, "padded": False},
        # a padded batch of odd length, 3 heads per cache head
        {"name": "weigh-padded", "op": "weigh", "B": 3, "Hq": 6, "Hkv": 2, "Nq": 1500, "Nkv": 1500, "d": 64, "causal": True, "padded": True},
        # a lone request over its budget
        {"name": "evict-short", "op": "evict", "B": 1, "Hkv": 2, "L": 700, "n_keep": 512, "n_recent": 64, "d": 64, "ragged": False},
        # a batch of long prompts cut to half
        {"name": "evict-long", "op": "evict", "B": 16, "Hkv": 8, "L": 32768, "n_keep": 16384, "n_recent": 256, "d": 128, "ragged": True},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("decode", "decode", "append", "weigh", "evict"))
    d = rng.choice((64, 128))
    Hkv = rng.choice((1, 2, 3, 4, 8))
    if op == "decode":
        G = rng.choice((1, 2, 3, 4, 5, 6, 7, 8, 16))
        B = _log(rng, 1, 64)
        most = min(131072, 64 * 8 * 8192 * 128 // (B * Hkv * d), 64 * 32 * 8192 * 2 // (B * Hkv * G))
        return {"op": op, "B": B, "Hq": Hkv * G, "Hkv": Hkv, "N": _log(rng, 1, most), "d": d,
                "weights": rng.random() < 0.5, "ragged": rng.random() < 0.5}
    if op == "append":
        B = _log(rng, 1, 64)
        return {"op": op, "B": B, "Hkv": Hkv, "n": _log(rng, 1, min(8192, 4 * 16 * 4096 // (B * Hkv))), "d": d,
                "ragged": rng.random() < 0.5}
    if op == "weigh":
        G = rng.choice((1, 2, 3, 4, 8))
        B = _log(rng, 1, 4)
        Nkv = _log(rng, 1, 16384)
        Nq = _log(rng, 1, max(1, min(Nkv, 32 * 4096 * 4096 // (B * Hkv * G * Nkv))))
        return {"op": op, "B": B, "Hq": Hkv * G, "Hkv": Hkv, "Nq": Nq, "Nkv": Nkv, "d": d,
                "causal": rng.random() < 0.8, "padded": rng.random() < 0.3}
    B = _log(rng, 1, 16)
    L = _log(rng, 2, 32768)
    n_keep = rng.randint(1, L)
    return {"op": op, "B": B, "Hkv": Hkv, "L": L, "n_keep": n_keep, "n_recent": rng.randint(0, min(n_keep, 256)), "d": d,
            "ragged": rng.random() < 0.5}


def _lengths(case, seed, most):
    """Live slots of each sequence: all `most`, or from about an eighth to all."""
    B = case["B"]
    if not (case.get("ragged") or case.get("padded")):
        return [most] * B
    g = torch.Generator().manual_seed(seed * 7919 + 13)
    lens = torch.randint(max(1, most // 8), most + 1, (B,), generator=g).tolist()
    lens[0] = most
    return lens


def _capacity(n):
    return (n + 15) // 16 * 16 + 16


def work(case):
    d = case["d"]
    row = 2 * (d // 2 + d // 16)  # codes and scales of one key and one value row
    if case["op"] == "decode":
        n = sum(_lengths(case, 1, case["N"]))
        by = case["Hkv"] * n * (row + (8 if case["weights"] else 0)) + case["B"] * case["Hq"] * (4 * d + 4)
        return {"bytes": by, "flops": 4.0 * case["Hq"] * n * d}
    if case["op"] == "append":
        n = sum(_lengths(case, 1, case["n"])) * case["Hkv"]
        return {"bytes": n * (4 * d + row + 8) + case["B"] * case["Hkv"] * case["n"] * 4 * d, "flops": 4.0 * n * d}
    if case["op"] == "weigh":
        lens = _lengths(case, 1, case["Nkv"])
        off = case["Nkv"] - case["Nq"]
        pairs = 0
        for n in lens:
            q = max(0, n - off)
            pairs += sum(range(off + 1, off + q + 1)) if case["causal"] else q * n
        by = case["B"] * (2 * d * (case["Hq"] * case["Nq"] + case["Hkv"] * case["Nkv"]) + 4 * case["Hq"] * case["Nq"] + 4 * case["Hkv"] * case["Nkv"])
        return {"bytes": by, "flops": 2.0 * case["Hq"] * pairs * d}
    lens = _lengths(case, 1, case["L"])
    n_keep = case["n_keep"]
    live = case["Hkv"] * sum(lens)
    kept = case["Hkv"] * sum(min(n, n_keep) for n in lens)
    moved = case["Hkv"] * sum((n - n_keep) * n_keep // n for n in lens if n > n_keep)  # expected, weights in random order
    return {"bytes": 8 * live + 12 * kept + 2 * row * moved, "flops": 8.0 * live}


# ------------------------------------------------------------------ what a program has in hand
def _normal(shape, gen, gain=None):
    x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)
    return (x if gain is None else x * gain).to(torch.bfloat16)


def _gain(Hkv, d, gen):
    """Keys have channels of different size."""
    return torch.exp(0.5 * torch.randn((Hkv, 1, d), generator=gen, device="cuda"))


def _cache(B, Hkv, cap, d, gen):
    """A cache whose every slot holds a quantised row (those behind the live ones hold older rows)."""
    kg, st = _gain(Hkv, d, gen), {}
    for name, gain in (("k", kg), ("v", None)):
        codes = torch.empty((B, Hkv, cap, d // 2), dtype=torch.uint8, device="cuda")
        scales = torch.empty((B, Hkv, cap, d // 32), dtype=torch.bfloat16, device="cuda")
        for b in range(B):
            c, s = _quantize(_normal((Hkv, cap, d), gen, gain))
            codes[b], scales[b] = _pack(c), s
        st[name + "c"], st[name + "s"] = codes, scales
    return st


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    B, d, op = case["B"], case["d"], case["op"]
    s = {"case": case}
    if op == "decode":
        Hq, Hkv, N = case["Hq"], case["Hkv"], case["N"]
        cap = _capacity(N)
        lens = _lengths(case, 1, N)
        s |= _cache(B, Hkv, cap, d, gen)
        s["q"] = _normal((B, Hq, 1, d), gen, 1.5)
        s["seqlens"] = _ints(lens)
        s["weights"] = torch.rand((B, Hkv, cap), generator=gen, device="cuda") if case["weights"] else None
        s["o"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty((B, Hq, 1), dtype=torch.float32, device="cuda")
        s["scale"] = d ** -0.5
        if own:
            import tiled_attention_24_b200 as ta
            s["splits"] = ta.attn_decode_kv4_splits(B, Hq, Hkv, cap, d)
            s["ws"] = torch.empty(ta.attn_decode_kv4_workspace_bytes(B, Hq, Hkv, cap, d, s["splits"], case["weights"]),
                                  dtype=torch.uint8, device="cuda")
    elif op == "append":
        Hkv, n = case["Hkv"], case["n"]
        cap = _capacity(n + 100)
        lens = _lengths(case, 1, n)
        s |= {"kc": torch.zeros((B, Hkv, cap, d // 2), dtype=torch.uint8, device="cuda"),
              "vc": torch.zeros((B, Hkv, cap, d // 2), dtype=torch.uint8, device="cuda"),
              "ks": torch.zeros((B, Hkv, cap, d // 32), dtype=torch.bfloat16, device="cuda"),
              "vs": torch.zeros((B, Hkv, cap, d // 32), dtype=torch.bfloat16, device="cuda"),
              "weights": torch.rand((B, Hkv, cap), generator=gen, device="cuda"),
              "positions": torch.full((B, Hkv, cap), -1, dtype=torch.int32, device="cuda"),
              "k": _normal((B, Hkv, n, d), gen, _gain(Hkv, d, gen)), "v": _normal((B, Hkv, n, d), gen),
              "starts": torch.randint(0, 101, (B,), generator=gen, device="cuda", dtype=torch.int32),
              "counts": _ints(lens)}
        s["next_pos"] = s["starts"] + 1000
        s["k_out"], s["v_out"] = torch.empty_like(s["k"]), torch.empty_like(s["v"])
    elif op == "weigh":
        Hq, Hkv, Nq, Nkv = case["Hq"], case["Hkv"], case["Nq"], case["Nkv"]
        lens = _lengths(case, 1, Nkv)
        s["q"] = _normal((B, Hq, Nq, d), gen, 1.5)
        s["k"] = _normal((B, Hkv, Nkv, d), gen, _gain(Hkv, d, gen))
        s["scale"] = d ** -0.5
        s["seqlens"] = _ints(lens) if case["padded"] else None
        s["lse"] = torch.empty((B, Hq, Nq), dtype=torch.float32, device="cuda")
        for b in range(B):  # as the forward of the prompt left it
            for h in range(Hq):
                x = s["q"][b, h].float() @ s["k"][b, h // (Hq // Hkv)].float().T * s["scale"]
                if case["causal"]:
                    x.masked_fill_(~_visible(Nq, Nkv), -math.inf)
                s["lse"][b, h] = torch.logsumexp(x, dim=-1)
        s["weights"] = torch.empty((B, Hkv, Nkv), dtype=torch.float32, device="cuda")
        if own:
            import tiled_attention_24_b200 as ta
            s["ws"] = torch.empty(max(16, ta.attn_key_weights_workspace_bytes(B, Hq, Hkv, Nq, Nkv, d)), dtype=torch.uint8, device="cuda")
    else:
        Hkv, L = case["Hkv"], case["L"]
        cap = _capacity(L)
        lens = _lengths(case, 1, L)
        s |= _cache(B, Hkv, cap, d, gen)
        # accumulated weights: a few large ones, many small
        s["weights"] = torch.randn((B, Hkv, cap), generator=gen, device="cuda").mul_(2.0).exp_()
        # slots were filled and reused in another order than the tokens'
        s["positions"] = torch.argsort(torch.rand((B, Hkv, cap), generator=gen, device="cuda"), dim=-1).to(torch.int32)
        s["seqlens"], s["next_pos"] = _ints(lens), _ints([cap] * B)
        s["weights_out"] = torch.zeros_like(s["weights"])
        s["positions_out"] = torch.full_like(s["positions"], -1)
        s["kept"] = torch.empty((B, Hkv, case["n_keep"]), dtype=torch.int32, device="cuda")
        if own:
            import tiled_attention_24_b200 as ta
            s["ws"] = torch.empty(ta.attn_kv4_evict_workspace_bytes(B, Hkv, cap, case["n_keep"]), dtype=torch.uint8, device="cuda")
    return s


def _visible(Nq, Nkv):
    i = torch.arange(Nq, device="cuda")[:, None] + (Nkv - Nq)
    return torch.arange(Nkv, device="cuda")[None, :] <= i


# ------------------------------------------------------------------ one pass
def run(s):
    return {"decode": _decode, "append": _append, "weigh": _weigh, "evict": _evict}[s["case"]["op"]](s)


def _decode(s):
    if own:
        import tiled_attention_24_b200 as ta
        ta.attn_decode_kv4(s["q"], s["kc"], s["ks"], s["vc"], s["vs"], s["o"], s["lse"], s["seqlens"], s["scale"],
                           s["splits"], s["ws"], s["weights"])
        return {"o": s["o"], "lse": s["lse"], "weights": s["weights"]}
    B, Hq, _, d = s["q"].shape
    Hkv, cap = s["kc"].shape[1:3]
    live = torch.arange(cap, device="cuda")[None, :] < s["seqlens"][:, None]
    live = live[:, None, None, :]
    x = torch.matmul(s["q"].float().reshape(B, Hkv, Hq // Hkv, d), _values(s["kc"], s["ks"]).transpose(-1, -2))
    x = torch.where(live, x * s["scale"], torch.full_like(x, -math.inf))
    m = x.amax(dim=-1, keepdim=True)
    p = torch.exp(x - m)
    l = p.sum(dim=-1, keepdim=True)
    p = p / l
    o = torch.matmul(p, _values(s["vc"], s["vs"])).reshape(B, Hq, 1, d).to(torch.bfloat16)
    lse = (m + torch.log(l)).reshape(B, Hq, 1)
    if s["weights"] is not None:
        s["weights"].add_(p.sum(dim=2))
    return {"o": o, "lse": lse, "weights": s["weights"]}


def _append(s):
    if own:
        import tiled_attention_24_b200 as ta
        ta.attn_kv4_append(s["k"], s["v"], s["kc"], s["ks"], s["vc"], s["vs"], s["starts"], s["counts"], s["weights"],
                           s["positions"], s["next_pos"])
        ta.attn_kv4_read(s["kc"], s["ks"], s["k_out"], s["starts"])
        ta.attn_kv4_read(s["vc"], s["vs"], s["v_out"], s["starts"])
        return {"k": s["k_out"], "v": s["v_out"], "weights": s["weights"], "positions": s["positions"]}
    B, Hkv, n, d = s["k"].shape
    i = torch.arange(n, device="cuda")[None, :]
    slot = (s["starts"][:, None] + i).long()
    fresh = (i < s["counts"][:, None])[:, None, :, None]
    at = slot[:, None, :, None].expand(B, Hkv, n, 1)
    out = {}
    for x, codes, scales in (("k", "kc", "ks"), ("v", "vc", "vs")):
        c, f = _quantize(s[x])
        rows = at.expand(B, Hkv, n, d // 2)
        s[codes].scatter_(2, rows, torch.where(fresh, _pack(c), s[codes].gather(2, rows)))
        rows = at.expand(B, Hkv, n, d // 32)
        s[scales].scatter_(2, rows, torch.where(fresh, f, s[scales].gather(2, rows)))
        out[x] = _values(s[codes].gather(2, at.expand(B, Hkv, n, d // 2)), s[scales].gather(2, rows)).to(torch.bfloat16)
    at, fresh = at[..., 0], fresh[..., 0]
    w = s["weights"].gather(2, at)
    s["weights"].scatter_(2, at, torch.where(fresh, torch.zeros_like(w), w))
    pos = (s["next_pos"][:, None] + i).to(torch.int32)[:, None, :].expand(B, Hkv, n)
    s["positions"].scatter_(2, at, torch.where(fresh, pos, s["positions"].gather(2, at)))
    return {**out, "weights": s["weights"], "positions": s["positions"]}


def _weigh(s):
    c = s["case"]
    if own:
        import tiled_attention_24_b200 as ta
        ta.attn_key_weights(s["q"], s["k"], s["lse"], s["weights"], c["causal"], s["scale"], s["ws"], seqlens=s["seqlens"])
        return s["weights"]
    B, Hq, Nq, d = s["q"].shape
    Hkv, Nkv = s["k"].shape[1:3]
    G = Hq // Hkv
    x = torch.matmul(s["q"].float().reshape(B, Hkv, G * Nq, d), s["k"].float().transpose(-1, -2)).mul_(s["scale"])
    x = x.reshape(B, Hkv, G, Nq, Nkv).sub_(s["lse"].reshape(B, Hkv, G, Nq, 1)).exp_()
    if c["causal"]:
        x.masked_fill_(~_visible(Nq, Nkv), 0.0)
    if s["seqlens"] is not None:
        n = s["seqlens"][:, None, None, None, None]
        i = torch.arange(Nq, device="cuda")[:, None] + (Nkv - Nq)
        x.masked_fill_((i >= n) | (torch.arange(Nkv, device="cuda") >= n), 0.0)
    return x.sum(dim=3).sum(dim=2)


def _evict(s):
    c = s["case"]
    if own:
        import tiled_attention_24_b200 as ta
        ta.attn_kv4_evict(s["kc"], s["ks"], s["vc"], s["vs"], s["weights"], s["positions"], s["seqlens"], s["next_pos"],
                          s["weights_out"], s["positions_out"], s["kept"], c["n_recent"], s["ws"])
    else:
        B, Hkv, cap = s["weights"].shape
        n_keep = c["n_keep"]
        n = s["seqlens"][:, None, None]
        slot = torch.arange(cap, device="cuda").expand(B, Hkv, cap)
        live = slot < n
        w = torch.where(s["weights"].isnan(), torch.full_like(s["weights"], -math.inf), s["weights"])
        w = torch.where(s["positions"] >= s["next_pos"][:, None, None] - c["n_recent"], torch.full_like(w, math.inf), w)
        order = torch.sort(w.masked_fill(~live, -math.inf), dim=-1, descending=True, stable=True).indices
        # a dead slot never comes before a live one
        order = order.gather(2, torch.sort((~live.gather(2, order)).to(torch.int8), dim=-1, stable=True).indices)
        keep = torch.zeros_like(live).scatter_(2, order[..., :n_keep], True) & live
        hole = (slot < n_keep) & live & ~keep
        rank = (hole.long().cumsum(dim=-1) - 1).clamp_(min=0)
        source = torch.sort((~(keep & (slot >= n_keep))).to(torch.int8), dim=-1, stable=True).indices
        kept = torch.where(hole, source.gather(2, rank), slot)[..., :n_keep]
        front = live[..., :n_keep]
        for x in ("kc", "ks", "vc", "vs"):
            w = s[x].shape[-1]
            s[x][:, :, :n_keep] = s[x].gather(2, kept[..., None].expand(B, Hkv, n_keep, w))
        s["weights_out"][..., :n_keep] = torch.where(front, s["weights"].gather(2, kept), s["weights_out"][..., :n_keep])
        s["positions_out"][..., :n_keep] = torch.where(front, s["positions"].gather(2, kept), s["positions_out"][..., :n_keep])
        s["kept"].copy_(torch.where(front, kept, torch.full_like(kept, -1)))
    # the rows are moved, never computed with: their bytes are compared as the whole numbers they are
    return {"kept": s["kept"], "weights": s["weights_out"], "positions": s["positions_out"], "kc": s["kc"], "vc": s["vc"],
            "ks": s["ks"].view(torch.int16), "vs": s["vs"].view(torch.int16)}


# ------------------------------------------------------------------ the definition in 64 bits
def _row64(codes, scales):
    """float64 values of packed rows, channel by channel from the format's description."""
    d = 2 * codes.shape[-1]
    ch = torch.arange(d, device=codes.device)
    byte = (ch % 32) // 4 * (d // 16) + 2 * (ch // 32) + ch % 4 // 2
    nib = (codes[..., byte].to(torch.int64) >> (4 * (ch % 2))) % 16
    return (nib - 16 * (nib >= 8)).double() * scales.double()[..., ch // 32]


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "decode":
        B, Hq, Hkv, N = case["B"], case["Hq"], case["Hkv"], case["N"]
        G = Hq // Hkv
        o, lse = s["q"].double() * 0, s["lse"].double()
        w = None if s["weights"] is None else s["weights"].double()
        for b, n in enumerate(s["seqlens"].tolist()):
            for h in range(Hkv):
                k, v = _row64(s["kc"][b, h, :n], s["ks"][b, h, :n]), _row64(s["vc"][b, h, :n], s["vs"][b, h, :n])
                x = s["q"][b, h * G:(h + 1) * G, 0].double() @ k.T * case["d"] ** -0.5
                z = torch.logsumexp(x, dim=1)
                p = torch.exp(x - z[:, None])
                o[b, h * G:(h + 1) * G, 0], lse[b, h * G:(h + 1) * G, 0] = p @ v, z
                if w is not None:
                    w[b, h, :n] += p.sum(dim=0)
        return {"o": o, "lse": lse, "weights": w}
    if op == "append":
        out = {"weights": s["weights"].double(), "positions": None}
        for b, (at, n) in enumerate(zip(s["starts"].tolist(), s["counts"].tolist())):
            out["weights"][b, :, at:at + n] = 0
        for x in ("k", "v"):
            g = s[x].double().unflatten(-1, (-1, 32))
            f = (g.abs().amax(dim=-1, keepdim=True) / 7).bfloat16().double()
            y = (torch.where(f > 0, torch.round(g / f), 0 * g).clamp(-7, 7) * f).flatten(-2)
            out[x] = y * (torch.arange(case["n"], device="cuda") < s["counts"][:, None])[:, None, :, None]
        return out
    if op == "weigh":
        B, Hq, Hkv, Nq, Nkv = (case[x] for x in ("B", "Hq", "Hkv", "Nq", "Nkv"))
        w = torch.zeros((B, Hkv, Nkv), dtype=torch.float64, device="cuda")
        lens = [Nkv] * B if s["seqlens"] is None else s["seqlens"].tolist()
        for b in range(B):
            rows = max(0, lens[b] - (Nkv - Nq))
            for h in range(Hq):
                q, k = s["q"][b, h, :rows].double(), s["k"][b, h // (Hq // Hkv), :lens[b]].double()
                p = torch.exp(q @ k.T * case["d"] ** -0.5 - s["lse"][b, h, :rows, None].double())
                w[b, h // (Hq // Hkv), :lens[b]] += (torch.tril(p, Nkv - Nq) if case["causal"] else p).sum(dim=0)
        return w
    return None
