"""The serving operators of the library as measured cases: sliding-window prefill attention with
visible first tokens, and the 4-bit paged KV cache (append and read back, single-token attention
that can accumulate attention weight, eviction by that weight).

``run`` computes a case with plain torch operations in 32 bits, or, where ``own`` is set, with the
library's calls.  ``exact`` computes the same from the definitions in 64 bits.

The cache format both forms work on: a pool [n_pages, Hkv, d / 64 * 4608] of bytes; each (page,
KV head) holds 64 slots.  A slot's key (value) is cut into groups of 64 channels; a group is 32
bytes of codes (word w, nibble j: channel 8 w + j) and a bf16 pair (s, m), and stands for s * n + m.
In the bytes of a (page, head): key codes [d / 64][64 slots][32], value codes alike, key pairs
[d / 64][64 slots][2], value pairs alike."""
import math
import random

import torch

own = False

PAGE, GROUP = 64, 64


# ---------------------------------------------------------------------------------------- cases


def listed():
    llama = {"Hq": 32, "Hkv": 8, "d": 128}
    return [
        # a handful of short prompts, packed: the smallest prefill, where latency counts
        {"name": "window, short prompts", "op": "window", "B": 6, "min_len": 1, "max_len": 700, "mix": 1,
         "Hq": 8, "Hkv": 2, "d": 64, "window": 256, "sinks": 4},
        # one long prompt of a Llama-3.1-8B shaped layer
        {"name": "window, 32K prompt", "op": "window", "B": 1, "min_len": 32768, "max_len": 32768, "mix": 2,
         **llama, "window": 2048, "sinks": 4},
        # a ragged batch of prompts, a tile of first tokens kept visible
        {"name": "window, ragged batch", "op": "window", "B": 17, "min_len": 200, "max_len": 9001, "mix": 3,
         **llama, "window": 1024, "sinks": 128},
        # a wide window and many first tokens (a system prompt that stays visible), odd sizes
        {"name": "window, wide", "op": "window", "B": 1, "min_len": 15001, "max_len": 15001, "mix": 4,
         "Hq": 16, "Hkv": 16, "d": 128, "window": 8191, "sinks": 1000},
        # one decode step of a batch: one token per sequence is written
        {"name": "append, decode step", "op": "append", "B": 64, "min_len": 1, "max_len": 1, "mix": 5, "start": 4000,
         **llama, "weights": True},
        # prompts (or prefill chunks) written behind what the cache already holds
        {"name": "append, prompts", "op": "append", "B": 5, "min_len": 900, "max_len": 16000, "mix": 6, "start": 777,
         **llama, "weights": True},
        # one chat, one token: the smallest decode
        {"name": "decode, one chat", "op": "decode", "B": 1, "min_len": 700, "max_len": 700, "mix": 7,
         **llama, "window": 0, "sinks": 0, "weights": False},
        # a serving batch with ragged lengths, attention weights accumulated for eviction
        {"name": "decode, batch + weights", "op": "decode", "B": 64, "min_len": 100, "max_len": 8191, "mix": 8,
         **llama, "window": 0, "sinks": 0, "weights": True},
        # few long contexts: the cache's bandwidth
        {"name": "decode, 4 x 128K", "op": "decode", "B": 4, "min_len": 120000, "max_len": 131072, "mix": 9,
         **llama, "window": 0, "sinks": 0, "weights": False},
        # sliding-window layer in decode, one query head per KV head, head dim 64
        {"name": "decode, window", "op": "decode", "B": 16, "min_len": 3000, "max_len": 30000, "mix": 10,
         "Hq": 16, "Hkv": 16, "d": 64, "window": 4096, "sinks": 64, "weights": False},
        # a batch at its budget: every so many steps the cache goes back to 4096 slots
        {"name": "evict, steady state", "op": "evict", "B": 32, "min_len": 4200, "max_len": 4352, "mix": 11,
         **llama, "keep": 4096, "sinks": 4, "recent": 512},
        # a long prompt's cache cut to its heavy hitters right after prefill
        {"name": "evict, after prefill", "op": "evict", "B": 2, "min_len": 100001, "max_len": 131072, "mix": 12,
         **llama, "keep": 8192, "sinks": 16, "recent": 1024},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["window", "append", "decode", "evict"])
    Hkv = rng.choice([1, 2, 4, 8])
    c = {"op": op, "Hq": Hkv * rng.choice([1, 2, 3, 4, 7, 8] if Hkv <= 4 else [1, 2, 4]), "Hkv": Hkv,
         "d": rng.choice([64, 128]), "mix": rng.randrange(1 << 20)}
    if op == "window":
        top = _log_int(rng, 8, 15000)
        c |= {"B": _log_int(rng, 1, max(1, min(16, 60000 // top))), "max_len": top, "min_len": _log_int(rng, 1, top),
              "window": _log_int(rng, 1, 4096), "sinks": rng.choice([0, 1, 4, _log_int(rng, 1, 500)])}
    elif op == "append":
        top = _log_int(rng, 1, 10000)
        c |= {"B": _log_int(rng, 1, max(1, min(128, 40000 // top))), "max_len": top, "min_len": _log_int(rng, 1, top),
              "start": _log_int(rng, 1, 5000), "weights": rng.random() < 0.5}
    elif op == "decode":
        top = _log_int(rng, 10, 120000)
        window = rng.choice([0, _log_int(rng, 1, 5000)])
        c |= {"B": _log_int(rng, 1, max(1, min(128, 400000 // top))), "max_len": top, "min_len": _log_int(rng, 1, top),
              "window": window, "sinks": rng.choice([0, 4, 100]) if window else 0, "weights": rng.random() < 0.5}
    else:
        top = _log_int(rng, 64, 120000)
        keep = _log_int(rng, 16, top)
        recent = _log_int(rng, 1, max(1, keep // 2))
        c |= {"B": _log_int(rng, 1, max(1, min(64, 200000 // top))), "max_len": top, "min_len": _log_int(rng, 1, top),
              "keep": keep, "sinks": rng.choice([0, 1, 4, 7]), "recent": recent}
    return c


def _lengths(c):
    """The case's own lengths: the first is the longest, one of a batch the shortest."""
    rng = random.Random(c["mix"])
    n = [rng.randint(c["min_len"], c["max_len"]) for _ in range(c["B"])]
    n[0] = c["max_len"]
    if c["B"] > 1:
        n[rng.randrange(1, c["B"])] = c["min_len"]
    return n


def _starts(c):
    rng = random.Random(c["mix"] + 1)
    return [rng.randint(0, c["start"]) for _ in range(c["B"])]


def _window_pairs(n, window, sinks):
    """Query-key pairs of one sequence: key j of query i where j <= i and (i - j < window or j < sinks)."""
    w, s = min(window, n), min(sinks, n)
    near = w * (w + 1) // 2 + (n - w) * w
    first = sum(min(s, i + 1 - w) for i in range(w, min(n, w + s))) + max(0, n - w - s) * s
    return near + first


# -------------------------------------------------------------------------------------- prepare


def _words(n):
    """[..., 64] codes 0..15 -> [..., 8] words."""
    n = n.to(torch.int64).unflatten(-1, (8, 8)) << (4 * torch.arange(8, device=n.device))
    n = n.sum(-1)
    return torch.where(n >= 1 << 31, n - (1 << 32), n).to(torch.int32)


def _nibbles(w):
    """[..., 8] words -> [..., 64] codes."""
    return ((w.unsqueeze(-1) >> (4 * torch.arange(8, dtype=torch.int32, device=w.device))) & 15).flatten(-2)


def _parts(pool):
    """Views of a pool: key codes, value codes [pages, Hkv, d / 64, 64, 8] int32 and key, value pairs
    [pages, Hkv, d / 64, 64, 2] bf16."""
    g = pool.shape[2] // 4608
    w, h = pool.view(torch.int32), pool.view(torch.bfloat16)
    c, p = g * PAGE * 8, g * PAGE * 2
    return (w[..., :c].unflatten(-1, (g, PAGE, 8)), w[..., c:2 * c].unflatten(-1, (g, PAGE, 8)),
            h[..., 4 * c:4 * c + p].unflatten(-1, (g, PAGE, 2)), h[..., 4 * c + p:].unflatten(-1, (g, PAGE, 2)))


def _quantize(x):
    """[..., 64] bf16 -> codes [..., 64] and pairs [..., 2] (bf16)."""
    x = x.float()
    lo, hi = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
    s = ((hi.double() - lo.double()) / 15).float().bfloat16()
    step = torch.where(s == 0, torch.ones_like(s), s).double()  # 64 bits: quotients next to a half
    n = ((x.double() - lo.double()) / step).round().clamp(0, 15)
    n = torch.where(s == 0, torch.zeros_like(n), n)
    return n, torch.cat([s, lo.bfloat16()], -1)


def _filled_pool(c, pages, gen):
    """A pool as appends leave it: quantised keys and values."""
    d, Hkv = c["d"], c["Hkv"]
    pool = torch.empty((pages, Hkv, d // 64 * 4608), dtype=torch.uint8, device="cuda")
    kc, vc, kp, vp = _parts(pool)
    step = max(1, (1 << 25) // (Hkv * d * PAGE))
    for a in range(0, pages, step):
        b = min(pages, a + step)
        for codes, pairs in ((kc, kp), (vc, vp)):
            x = torch.randn((b - a, Hkv, d // 64, PAGE, GROUP), device="cuda", generator=gen)
            lo, hi = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
            s = ((hi - lo) / 15).bfloat16()
            codes[a:b] = _words(((x - lo) / s.float()).round().clamp(0, 15))
            pairs[a:b] = torch.cat([s, lo.bfloat16()], -1)
    return pool


def _tables(slots, gen):
    """Pages in random order: the page table for these many slots per sequence, and the pages in all."""
    need = [-(-n // PAGE) for n in slots]
    width, total = max(1, max(need)), max(1, sum(need))
    order = torch.randperm(total, device="cuda", generator=gen).to(torch.int32)
    table = torch.full((len(slots), width), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table, total


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator("cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, device="cuda", generator=gen).bfloat16()

    n, B, Hq, Hkv, d = _lengths(c), c["B"], c["Hq"], c["Hkv"], c["d"]
    cu = _ints([0] + [sum(n[:i + 1]) for i in range(B)])
    s = {"case": c, "n": n, "max": max(n), "cu": cu, "lens": _ints(n)}
    s["ws"] = torch.empty(_workspace_bytes(c, n), dtype=torch.uint8, device="cuda")
    if c["op"] == "window":
        s |= {"Q": normal(sum(n), Hq, d), "K": normal(sum(n), Hkv, d), "V": normal(sum(n), Hkv, d),
              "O": torch.empty((sum(n), Hq, d), dtype=torch.bfloat16, device="cuda"),
              "lse": torch.empty((Hq, sum(n)), device="cuda")}
    elif c["op"] == "append":
        start = _starts(c)
        end = [a + b for a, b in zip(start, n)]
        table, pages = _tables(end, gen)
        s |= {"K": normal(sum(n), Hkv, d), "V": normal(sum(n), Hkv, d), "table": table, "start": _ints(start),
              "lens": _ints(end), "seen": _ints([e + 100 for e in end]),
              "pool": torch.zeros((pages, Hkv, d // 64 * 4608), dtype=torch.uint8, device="cuda"),
              "K_read": torch.empty((sum(n), Hkv, d), dtype=torch.bfloat16, device="cuda"),
              "V_read": torch.empty((sum(n), Hkv, d), dtype=torch.bfloat16, device="cuda"),
              "acc": torch.zeros((B, Hkv, max(end)), device="cuda"),
              "pos": torch.zeros((B, Hkv, max(end)), dtype=torch.int32, device="cuda"),
              "A_v": torch.rand((Hq, sum(n)), device="cuda", generator=gen).square() * 8 if c["weights"] else None}
    elif c["op"] == "decode":
        table, pages = _tables(n, gen)
        s |= {"Q": normal(B, Hq, d), "pool": _filled_pool(c, pages, gen), "table": table,
              "O": torch.empty((B, Hq, d), dtype=torch.bfloat16, device="cuda"),
              "lse": torch.empty((Hq, B), device="cuda")}
        if c["weights"]:
            s["acc"] = torch.rand((B, Hkv, max(n)), device="cuda", generator=gen)
            s["acc_out"] = torch.zeros((B, Hkv, max(n)), device="cuda")
    else:
        table, pages = _tables(n, gen)
        # accumulated weights are heavy-tailed; positions are what earlier evictions left: increasing gaps
        acc = torch.exp(2 * torch.randn((B, Hkv, max(n)), device="cuda", generator=gen))
        gaps = torch.randint(1, 4, (B, Hkv, max(n)), device="cuda", generator=gen)
        pos = gaps.cumsum(-1).sub_(gaps[..., :1]).to(torch.int32)
        last = torch.gather(pos, 2, (s["lens"].long() - 1)[:, None, None].expand(B, Hkv, 1))
        s |= {"acc": acc, "pos": pos, "seen": last.amax((1, 2)).to(torch.int32) + 1, "table": table,
              "pool": _filled_pool(c, pages, gen), "lens_out": torch.zeros_like(s["lens"]),
              "acc_out": torch.zeros((B, Hkv, c["keep"]), device="cuda"),
              "pos_out": torch.zeros((B, Hkv, c["keep"]), dtype=torch.int32, device="cuda")}
    return s


def _workspace_bytes(c, n):
    """A workspace that is large enough for any of the calls, as a program sizes it once: scores of
    every slot (one float per query head and slot) and 64 MiB for the rest."""
    slots = c["B"] * (-(-max(n) // PAGE)) * PAGE
    return (64 << 20) + (4 * slots * (c["Hq"] + 16 * c["Hkv"]) if c["op"] in ("decode", "evict") else 0)


# ---------------------------------------------------------------------------------- plain forms


def _softmax_sum(scores, values, eq):
    """Rows of scores (-inf where masked; overwritten) -> weighted sum of values, log-sum-exp, weights."""
    m = scores.amax(-1, keepdim=True)
    p = scores.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    p = p.div_(l)
    return torch.einsum(eq, p, values), (m + torch.log(l)).squeeze(-1), p


def _plain_window(s):
    c, dev = s["case"], s["Q"].device
    B, Hq, Hkv, d, N = c["B"], c["Hq"], c["Hkv"], c["d"], s["max"]
    G, R = Hq // Hkv, min(256, N)
    blocks, W, S = -(-N // R), min(c["window"], N), min(c["sinks"], N)
    row = torch.arange(blocks * R, device=dev).view(blocks, R)
    near = torch.arange(1 - W, R, device=dev) + R * torch.arange(blocks, device=dev)[:, None]
    key = torch.cat([torch.arange(S, device=dev).expand(blocks, S), near], 1)  # [blocks, S + W + R - 1]
    i, j = row[:, :, None], key[:, None, :]
    first = torch.arange(key.shape[1], device=dev) < S
    seen = (j <= i) & torch.where(first, i - j >= W, (j >= 0) & (i - j < W))
    last = s["Q"].shape[0] - 1
    cu = s["cu"].long()
    at_q = (cu[:-1, None, None] + row).clamp(0, last)  # [B, blocks, R]
    at_k = (cu[:-1, None, None] + key).clamp(0, last)
    q = s["Q"][at_q].float().unflatten(3, (Hkv, G))
    k, v = s["K"][at_k].float(), s["V"][at_k].float()
    scores = torch.einsum("bnrhgd,bnchd->bnhgrc", q, k) / math.sqrt(d)
    scores = scores.masked_fill_(~seen[:, None, None], -math.inf)
    o, lse, _ = _softmax_sum(scores, v, "bnhgrc,bnchd->bnrhgd")
    live = row.flatten() < s["lens"][:, None]  # [B, blocks * R]
    o = o.reshape(B, blocks * R, Hq, d)[live].bfloat16()
    return {"O": o, "lse": lse.permute(0, 1, 4, 2, 3).reshape(B, blocks * R, Hq)[live].t().contiguous()}


def _token_places(s):
    """Sequence, and place among its new tokens, of every packed token."""
    t = torch.arange(s["K"].shape[0], device="cuda")
    b = torch.searchsorted(s["cu"][1:].long(), t, right=True)
    return b, t - s["cu"].long()[b]


def _plain_append(s):
    c = s["case"]
    Hq, Hkv, d = c["Hq"], c["Hkv"], c["d"]
    kc, vc, kp, vp = _parts(s["pool"])
    b, i = _token_places(s)
    slot = s["start"].long()[b] + i
    page = s["table"].long()[b, slot // PAGE]
    read = []
    for x, codes, pairs in ((s["K"], kc, kp), (s["V"], vc, vp)):
        n, pair = _quantize(x.unflatten(2, (d // 64, GROUP)))
        codes[page, :, :, slot % PAGE] = _words(n)
        pairs[page, :, :, slot % PAGE] = pair
        p = pairs[page, :, :, slot % PAGE].float()
        read.append((_nibbles(codes[page, :, :, slot % PAGE]) * p[..., :1] + p[..., 1:]).bfloat16().flatten(2))
    w = s["A_v"].unflatten(0, (Hkv, Hq // Hkv)).sum(1).t() if s["A_v"] is not None else 0.0
    s["acc"][b, :, slot] = w
    s["pos"][b, :, slot] = (s["seen"].long()[b] - (s["cu"][1:] - s["cu"][:-1]).long()[b] + i).to(torch.int32)[:, None]
    return {"K": read[0], "V": read[1], "acc": s["acc"], "pos": s["pos"]}


def _plain_decode(s):
    c = s["case"]
    B, Hq, Hkv, d, N = c["B"], c["Hq"], c["Hkv"], c["d"], s["max"]
    G = Hq // Hkv
    kc, vc, kp, vp = _parts(s["pool"])
    at = s["table"].long().clamp(min=0)

    def values(codes, pairs):  # [B, pages, Hkv, groups, 64, 64] -> [B, Hkv, slots, d]
        p = pairs[at].float()
        x = _nibbles(codes[at]) * p[..., :1] + p[..., 1:]
        return x.permute(0, 2, 1, 4, 3, 5).reshape(B, Hkv, -1, d)

    t = torch.arange(at.shape[1] * PAGE, device=at.device)
    n = s["lens"][:, None]
    seen = t < n
    if c["window"]:
        seen = seen & ((t >= n - c["window"]) | (t < c["sinks"]))
    q = s["Q"].float().view(B, Hkv, G, d)
    scores = torch.einsum("bhgd,bhtd->bhgt", q, values(kc, kp)) / math.sqrt(d)
    scores = scores.masked_fill_(~seen[:, None, None], -math.inf)
    # slots behind a sequence's last belong to nobody: their values do not count
    o, lse, p = _softmax_sum(scores, values(vc, vp), "bhgt,bhtd->bhgd")
    out = {"O": o.reshape(B, Hq, d).bfloat16(), "lse": lse.reshape(B, Hq).t().contiguous()}
    if c["weights"]:
        live = (t[:N] < n)[:, None]
        out["acc"] = torch.where(live, s["acc"] + p.sum(2)[..., :N], torch.zeros_like(s["acc"]))
    return out


def _plain_evict(s):
    c = s["case"]
    keep, N = c["keep"], s["max"]
    t = torch.arange(N, device="cuda")
    n = s["lens"][:, None, None]
    kept_n = torch.clamp(s["lens"], max=keep)
    fixed = (s["pos"] < c["sinks"]) | (s["pos"] >= s["seen"][:, None, None] - c["recent"])
    key = torch.where(fixed, torch.full_like(s["acc"], math.inf), s["acc"])
    key = torch.where(t < n, key, torch.full_like(key, -math.inf))
    order = torch.sort(key, dim=-1, descending=True, stable=True).indices
    kept = torch.zeros_like(key, dtype=torch.bool)
    kept.scatter_(2, order, (t < kept_n[:, None, None]).expand_as(key))
    k = kept_n[:, None, None]
    hole = ((t < k) & ~kept).nonzero()  # row by row, ascending: the i-th hole takes the i-th kept slot behind k
    tail = ((t >= k) & kept).nonzero()
    source = t.expand_as(key).clone()
    source[hole[:, 0], hole[:, 1], hole[:, 2]] = tail[:, 2]
    b, h, dst, src = hole[:, 0], hole[:, 1], hole[:, 2], tail[:, 2]
    table = s["table"].long()
    to, of = table[b, dst // PAGE], table[b, src // PAGE]
    for x in _parts(s["pool"]):
        x[to, h, :, dst % PAGE] = x[of, h, :, src % PAGE]
    live, source = (t < k)[..., :keep], source[..., :keep]
    out = {"lens": kept_n, "pool": s["pool"]}
    for name, x in (("acc", s["acc"]), ("pos", s["pos"])):
        y = torch.zeros_like(s[name + "_out"])
        y[..., :source.shape[2]] = torch.where(live, torch.gather(x, 2, source), torch.zeros_like(x[..., :source.shape[2]]))
        out[name] = y
    return out


# ------------------------------------------------------------------------------------------ run


def _own(s):
    import sparse_attention_long_head_b200 as vs
    c = s["case"]
    if c["op"] == "window":
        vs.vs_window_attn_fwd_varlen(s["Q"], s["K"], s["V"], s["cu"], s["max"], c["window"], c["sinks"], s["O"],
                                     s["lse"], s["ws"])
        return {"O": s["O"], "lse": s["lse"]}
    if c["op"] == "append":
        vs.vs_kv4_append(s["K"], s["V"], s["cu"], s["max"], s["pool"], s["table"], s["lens"], s["ws"],
                         n_tokens=s["seen"], A_v=s["A_v"], acc=s["acc"], pos=s["pos"])
        vs.vs_kv4_read(s["pool"], s["table"], s["lens"], s["start"], s["cu"], s["max"], s["K_read"], s["V_read"],
                       s["ws"])
        return {"K": s["K_read"], "V": s["V_read"], "acc": s["acc"], "pos": s["pos"]}
    if c["op"] == "decode":
        vs.vs_kv4_decode_attn_fwd(s["Q"], s["pool"], s["table"], s["lens"], s["max"], s["O"], s["lse"], s["ws"],
                                  window=c["window"], sinks=c["sinks"], acc_in=s.get("acc"),
                                  acc_out=s.get("acc_out"))
        out = {"O": s["O"], "lse": s["lse"]}
        return out | {"acc": s["acc_out"]} if c["weights"] else out
    vs.vs_kv4_evict(s["pool"], s["table"], s["lens"], s["seen"], s["max"], s["acc"], s["pos"], c["keep"], c["sinks"],
                    c["recent"], s["lens_out"], s["acc_out"], s["pos_out"], s["ws"])
    return {"lens": s["lens_out"], "pool": s["pool"], "acc": s["acc_out"], "pos": s["pos_out"]}


def run(s):
    if own:
        return _own(s)
    return {"window": _plain_window, "append": _plain_append, "decode": _plain_decode, "evict": _plain_evict}[
        s["case"]["op"]](s)


# ----------------------------------------------------------------------------------------- work


def work(case):
    c, n = case, _lengths(case)
    Hq, Hkv, d, total = c["Hq"], c["Hkv"], c["d"], sum(_lengths(case))
    slot = Hkv * (d // 64) * 72  # bytes of one slot's key and value, all heads
    if c["op"] == "window":
        pairs = sum(_window_pairs(x, c["window"], c["sinks"]) for x in n)
        return {"bytes": total * (4 * Hq * d + 4 * Hkv * d + 4 * Hq), "flops": 4 * pairs * Hq * d}
    if c["op"] == "append":  # written, and read back
        aux = 8 * Hkv + (4 * Hq if c["weights"] else 0)
        return {"bytes": total * (8 * Hkv * d + 2 * slot + aux), "flops": total * Hkv * d * 8}
    if c["op"] == "decode":
        seen = sum(min(x, c["window"] + min(c["sinks"], max(0, x - c["window"]))) if c["window"] else x for x in n)
        return {"bytes": seen * slot + c["B"] * Hq * (4 * d + 4) + (8 * total * Hkv if c["weights"] else 0),
                "flops": 4 * seen * Hq * d}
    kept = [min(x, c["keep"]) for x in n]
    moved = sum(k * (1 - k / x) for x, k in zip(n, kept))
    return {"bytes": 8 * Hkv * (total + sum(kept)) + 2 * moved * slot, "flops": 4 * Hkv * total}


# ---------------------------------------------------------------------------------------- exact


def _exact_window(s):
    c = s["case"]
    G = c["Hq"] // c["Hkv"]
    o = torch.empty(s["Q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.empty(s["lse"].shape, dtype=torch.float64, device="cuda")
    at = 0
    for n in s["n"]:
        for h in range(c["Hkv"]):
            k, v = s["K"][at:at + n, h].double(), s["V"][at:at + n, h].double()
            for r in range(0, n, 1024):
                i = torch.arange(r, min(n, r + 1024), device="cuda")
                lo = max(0, r - c["window"] + 1)
                cols = torch.arange(lo, int(i[-1]) + 1, device="cuda")
                cols = torch.cat([torch.arange(min(c["sinks"], lo), device="cuda"), cols])
                ok = (cols <= i[:, None]) & ((i[:, None] - cols < c["window"]) | (cols < c["sinks"]))
                q = s["Q"][at + r:at + r + len(i), h * G:(h + 1) * G].double()
                z = torch.einsum("rgd,cd->grc", q, k[cols]) * c["d"] ** -0.5
                z = torch.where(ok, z, torch.tensor(-math.inf, dtype=torch.float64, device="cuda"))
                lse[h * G:(h + 1) * G, at + r:at + r + len(i)] = torch.logsumexp(z, -1)
                o[at + r:at + r + len(i), h * G:(h + 1) * G] = torch.einsum("grc,cd->rgd", torch.softmax(z, -1), v[cols])
        at += n
    return {"O": o, "lse": lse}


def _exact_append(s):
    c = s["case"]
    out = {"pos": None}
    for name in ("K", "V"):
        x = s[name].double().reshape(-1, GROUP)
        lo, hi = x.min(1, keepdim=True).values, x.max(1, keepdim=True).values
        scale = ((hi - lo) / 15).float().bfloat16().double()
        n = torch.clamp(torch.round((x - lo) / torch.where(scale > 0, scale, 1.0)), 0, 15) * (scale > 0)
        out[name] = (n * scale + lo).reshape(s[name].shape)
    acc = torch.zeros(s["acc"].shape, dtype=torch.float64, device="cuda")
    if s["A_v"] is not None:
        cu, start = s["cu"].tolist(), s["start"].tolist()
        for b in range(c["B"]):
            w = s["A_v"][:, cu[b]:cu[b + 1]].double().view(c["Hkv"], -1, cu[b + 1] - cu[b]).sum(1)
            acc[b, :, start[b]:start[b] + w.shape[1]] = w
    return out | {"acc": acc}


def _exact_cache(s, b, h, n):
    """Keys and values of the first n slots of one sequence and head, in 64 bits, from the bytes."""
    c = s["case"]
    g = c["d"] // 64
    raw = s["pool"][s["table"][b, :-(-n // PAGE)].long(), h]  # [pages, bytes]
    found = []
    for part in (0, 1):
        codes = raw[:, part * g * 2048:(part + 1) * g * 2048].reshape(-1, g, PAGE, 32)
        at = 2 * g * 2048 + part * g * 256
        pairs = raw[:, at:at + g * 256].contiguous().view(torch.bfloat16).reshape(-1, g, PAGE, 2).double()
        n16 = torch.stack([codes & 15, codes >> 4], -1).reshape(-1, g, PAGE, GROUP).double()
        x = n16 * pairs[..., 0:1] + pairs[..., 1:2]
        found.append(x.transpose(1, 2).reshape(-1, c["d"])[:n])
    return found


def _exact_decode(s):
    c = s["case"]
    G = c["Hq"] // c["Hkv"]
    o = torch.zeros(s["O"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["lse"].shape, dtype=torch.float64, device="cuda")
    acc = torch.zeros(s["acc"].shape, dtype=torch.float64, device="cuda") if c["weights"] else None
    for b, n in enumerate(s["n"]):
        at = torch.arange(n, device="cuda")
        if c["window"]:
            at = at[(at >= n - c["window"]) | (at < c["sinks"])]
        for h in range(c["Hkv"]):
            k, v = _exact_cache(s, b, h, n)
            z = s["Q"][b, h * G:(h + 1) * G].double() @ k[at].t() * c["d"] ** -0.5
            p = torch.softmax(z, -1)
            lse[h * G:(h + 1) * G, b] = torch.logsumexp(z, -1)
            o[b, h * G:(h + 1) * G] = p @ v[at]
            if acc is not None:
                acc[b, h, :n] = s["acc"][b, h, :n].double()
                acc[b, h, at] += p.sum(0)
    return {"O": o, "lse": lse} | ({"acc": acc} if c["weights"] else {})


def _exact_evict(s):
    c = s["case"]
    acc_out = torch.zeros(s["acc_out"].shape, dtype=torch.float64)
    for b, n in enumerate(s["n"]):
        k, seen = min(n, c["keep"]), int(s["seen"][b])
        for h in range(c["Hkv"]):
            acc, pos = s["acc"][b, h, :n].double().cpu(), s["pos"][b, h, :n].cpu()
            fixed = (pos < c["sinks"]) | (pos >= seen - c["recent"])
            rank = sorted(range(n), key=lambda t, f=fixed.tolist(), a=acc.tolist(): (not f[t], 0.0 if f[t] else -a[t], t))
            stay = set(rank[:k])
            later = sorted(t for t in stay if t >= k)
            at = [t if t in stay else None for t in range(k)]
            for t in range(k):
                if at[t] is None:
                    at[t] = later.pop(0)
            acc_out[b, h, :k] = acc[at]
    return {"lens": None, "pool": None, "pos": None, "acc": acc_out}


def exact(case, seed):
    s = prepare(case, seed)
    n, slow = _lengths(case), case["B"] * case["Hkv"]
    if case["op"] == "evict" and sum(n) * case["Hkv"] > 3_000_000:
        return None
    if case["op"] in ("window", "decode") and slow > 4096:
        return None
    return {"window": _exact_window, "append": _exact_append, "decode": _exact_decode, "evict": _exact_evict}[
        case["op"]](s)
