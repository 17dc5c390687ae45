"""The paged-cache operators as measured cases: rotary positions with the quantized append into a paged
K/V cache, attention of a ragged chunk of new tokens (or single tokens) over it, the attention weight each
cached token has gathered, and the eviction that keeps the heaviest tokens.

``run`` computes a case in plain torch where ``own`` is false, and by the package's entry points where it
is true.  Cache codes are int8, or E4M3 bytes (returned as float8_e4m3fn, the values they stand for).
"""
from __future__ import annotations

import random

import torch

own = False

HEAD_MODES = ("int8_per_head", "fp8_per_head")  # one calibrated scale per head
MODES = ("int8_per_head", "fp8_per_token", "int8_per_token", "fp8_per_head")


def listed():
    """The cases, four operators."""
    return [
        # a serving step: 16 sequences add one token each (the smallest call, launch latency)
        dict(name="append_step", op="append", mode="int8_per_head", layout="BNSD", B=16, Hq=32, Hkv=8, D=128, page=64,
             q=1, kv=2048, ragged=1, rd=128, inter=False, fused=True, pad=0, far=8192),
        # five prompts' chunks, ragged, half of each head rotated in interleaved pairs, padded rows behind
        dict(name="append_chunks", op="append", mode="fp8_per_token", layout="BSND", B=5, Hq=40, Hkv=40, D=128, page=16,
             q=1333, kv=4001, ragged=2, rd=64, inter=True, fused=True, pad=37, far=8192),
        # two long prompts at once, positions far out
        dict(name="append_prompts", op="append", mode="int8_per_token", layout="BNSD", B=2, Hq=32, Hkv=8, D=128, page=128,
             q=16384, kv=32768, ragged=0, rd=128, inter=False, fused=False, pad=0, far=131072),
        # one user's next token over a short history
        dict(name="attend_single", op="attend", mode="int8_per_head", layout="BNSD", B=1, Hq=32, Hkv=8, D=128, page=64,
             q=1, kv=1000, ragged=0, causal=True, pad=0),
        # a decode batch over long ragged histories: bound by the cache's bytes
        dict(name="attend_batch", op="attend", mode="int8_per_head", layout="BNSD", B=16, Hq=32, Hkv=8, D=128, page=64,
             q=1, kv=32768, ragged=3, causal=True, pad=0),
        # one very long history
        dict(name="attend_far", op="attend", mode="fp8_per_token", layout="BSND", B=1, Hq=32, Hkv=8, D=128, page=64,
             q=1, kv=131071, ragged=0, causal=True, pad=0),
        # a few drafted tokens per sequence verified at once, an odd group of query heads, head_dim 64
        dict(name="attend_drafts", op="attend", mode="fp8_per_head", layout="BNSD", B=8, Hq=24, Hkv=8, D=64, page=32,
             q=6, kv=8000, ragged=4, causal=True, pad=3),
        # prompts' chunks behind long histories: bound by the matrix products
        dict(name="attend_chunk", op="attend", mode="fp8_per_token", layout="BNSD", B=2, Hq=32, Hkv=8, D=128, page=64,
             q=1500, kv=32768, ragged=5, causal=True, pad=0),
        # the weight that one decoded token gives each cached token
        dict(name="weigh_step", op="weigh", mode="int8_per_head", layout="BNSD", B=16, Hq=32, Hkv=8, D=128, page=64,
             q=1, kv=16384, ragged=6, causal=True, pad=0),
        # the weight that a prompt's last tokens give it (the window an eviction goes by)
        dict(name="weigh_window", op="weigh", mode="fp8_per_token", layout="BNSD", B=2, Hq=32, Hkv=8, D=128, page=64,
             q=64, kv=32768, ragged=7, causal=True, pad=0),
        # one short sequence cut to a quarter
        dict(name="evict_single", op="evict", mode="int8_per_head", layout="BNSD", B=1, Hkv=8, D=128, page=64, kv=2000,
             ragged=0, budget=512, sink=4, recent=64),
        # a batch of long sequences cut to 4096 tokens per head
        dict(name="evict_batch", op="evict", mode="fp8_per_token", layout="BNSD", B=8, Hkv=8, D=128, page=64, kv=32768,
             ragged=8, budget=4096, sink=4, recent=256),
    ]


def draw(rng):
    """One more case of the listed ones' ranges."""
    spread = lambda lo, hi: int(round(lo * (hi / lo) ** rng.random()))
    op = rng.choice(("append", "attend", "weigh", "evict"))
    c = dict(op=op, mode=rng.choice(MODES), layout=rng.choice(("BNSD", "BSND")), D=rng.choice((64, 128, 128)),
             page=rng.choice((16, 32, 64, 128)), ragged=rng.randrange(1000), Hkv=rng.choice((1, 2, 4, 8, 8, 40)))
    if op == "evict":
        c["B"] = spread(1, 16)
        c["kv"] = spread(64, max(64, min(32768, 2_000_000 // (c["B"] * c["Hkv"]))))
        c["sink"], c["recent"] = rng.choice((0, 1, 4)), spread(1, 300)
        c["budget"] = max(c["sink"] + c["recent"], spread(16, 4096))
        return c
    group = rng.choice((1, 2, 3, 4, 4, 5, 8))
    c["Hq"] = c["Hkv"] * (1 if c["Hkv"] == 40 else group)
    c["pad"] = rng.choice((0, 0, 1, 5))
    if op == "append":
        c["B"] = spread(1, 64)
        c["q"] = spread(1, max(1, min(8192, 16384 // c["B"])))
        c["kv"] = c["q"] + spread(1, 1024)
        c["rd"] = rng.choice((c["D"], c["D"], c["D"] // 2, 32))
        c["inter"], c["fused"], c["far"] = rng.random() < 0.5, rng.random() < 0.5, rng.choice((16384, 131072))
        return c
    c["causal"] = rng.random() < 0.8
    kind = rng.choice(("step", "drafts", "chunk"))
    c["q"] = 1 if kind == "step" else spread(2, 16) if kind == "drafts" else spread(17, 1500)
    c["B"] = spread(1, 32 if kind == "step" else 8 if kind == "drafts" else 2)
    if op == "weigh":
        c["q"] = min(c["q"], 64)
    rows = c["B"] * c["Hq"] * c["q"]
    most = max(64, min(131072 if c["B"] == 1 else 32768, 2_000_000_000 // rows, 4_000_000 // (c["B"] * c["Hkv"])))
    c["kv"] = max(c["q"], spread(64, most)) if c["causal"] else spread(64, most)
    return c


def _lengths(c):
    """Each sequence's new tokens and its cached tokens (new ones included): fixed by the case."""
    r = random.Random(c["ragged"])
    cut = (lambda n: n) if not c["ragged"] else (lambda n: max(1, int(n * (0.4 + 0.6 * r.random()))))
    qs = [c.get("q", 0) if c.get("q", 0) < 2 or b == 0 else cut(c["q"]) for b in range(c["B"])]
    kvs = [c["kv"] if b == 0 else max(cut(c["kv"]), qs[b] if c.get("causal", True) else 1) for b in range(c["B"])]
    return qs, kvs


def _e4m3(x):
    return x.clamp(-448.0, 448.0).to(torch.float8_e4m3fn)


def _rope_table(n, rd):
    """cos | sin of position * 10000^(-2 i / rd), by 64 bits."""
    inv = 10000.0 ** (-torch.arange(0, rd, 2, dtype=torch.float64, device="cuda") / rd)
    ang = torch.arange(n, dtype=torch.float64, device="cuda")[:, None] * inv[None]
    return torch.cat((ang.cos(), ang.sin()), 1).float()


def prepare(case, seed):
    c = case
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    rand = lambda *s: torch.randn(s, generator=g, device=dev)
    B, H, D, page = c["B"], c["Hkv"], c["D"], c["page"]
    qs, kvs = _lengths(c)
    s = dict(c=c)
    # pages in no order, a few more than the sequences hold; entries past a sequence's end name no page
    need = [-(-n // page) for n in kvs]
    pages, wide = sum(need) + 3, max(need)
    order = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
    held = torch.tensor(need, device=dev)
    at = torch.arange(wide, device=dev)
    starts = held.cumsum(0) - held
    s["table"] = torch.where(at[None] < held[:, None], order[(starts[:, None] + at[None]).clamp(max=pages - 1)],
                             torch.full((), -1, dtype=torch.int32, device=dev)).contiguous()
    s["lens"] = torch.tensor(kvs, dtype=torch.int32, device=dev)
    shape = (pages, H, page, D) if c["layout"] == "BNSD" else (pages, page, H, D)
    fp8, qmax = c["mode"].startswith("fp8"), 448.0 if c["mode"].startswith("fp8") else 127.0
    for n in ("k", "v"):
        x = rand(*shape) * (qmax / 4.5)
        s[n + "c"] = _e4m3(x).view(torch.uint8) if fp8 else x.round().clamp(-128, 127).to(torch.int8)
        per = (H,) if c["mode"] in HEAD_MODES else (pages, H, page)
        s[n + "s"] = (4.5 / qmax) * (0.8 + 0.4 * torch.rand(per, generator=g, device=dev))
    if c["op"] == "evict":
        # gathered weights: heavy-tailed, as attention leaves them
        s["scores"] = torch.where(at.new_tensor(range(wide * page))[None, None] < s["lens"][:, None, None],
                                  (1.5 * rand(B, H, wide * page)).exp(), torch.zeros((), device=dev))
        s["scores_out"] = torch.zeros_like(s["scores"])
        return s
    T = sum(qs)
    s["cu"] = torch.tensor([0] + [sum(qs[: b + 1]) for b in range(B)], dtype=torch.int32, device=dev)
    s["max_q"] = max(qs)
    Hq = c["Hq"]
    rows = T + c["pad"]
    if c["op"] == "append":
        if c["fused"]:  # the columns of one projection's output
            x = rand(rows, (Hq + 2 * H) * D).to(torch.bfloat16).view(rows, Hq + 2 * H, D)
            s["q"], s["k"], s["v"] = x[:, :Hq], x[:, Hq:Hq + H], x[:, Hq + H:]
        else:
            s["q"], s["k"], s["v"] = (rand(rows, h, D).to(torch.bfloat16) for h in (Hq, H, H))
        s["cos_sin"] = _rope_table(c["far"], c["rd"])
        # the tokens' positions: the last ones of a text that ends near the table's end
        b = torch.searchsorted(s["cu"][1:].contiguous(), torch.arange(rows, device=dev, dtype=torch.int32),
                               right=True).clamp(max=B - 1)
        s["pos"] = (c["far"] - 1 - 3 * b + torch.arange(rows, device=dev) - s["cu"][1:][b].long()).clamp(0, c["far"] - 1).to(
            torch.int32)
        s["amax"] = tuple(4.2 + 0.4 * torch.rand(H, generator=g, device=dev) for _ in range(2))
        s["out"] = torch.zeros(rows, Hq, D, dtype=torch.bfloat16, device=dev)
        return s
    s["q"] = (1.5 * rand(rows, Hq, D)).to(torch.bfloat16)
    if c["op"] == "attend":
        s["out"] = torch.zeros(rows, Hq, D, dtype=torch.bfloat16, device=dev)
        s["lse"] = torch.zeros(rows, Hq, dtype=torch.float32, device=dev)
    else:
        s["lse"] = torch.zeros(rows, Hq, dtype=torch.float32, device=dev)
        s["lse"][:T] = _weights(s)[1]
        # what earlier tokens have given: a few times what these will
        s["acc"] = torch.rand(B, H, wide * page, generator=g, device=dev) * (4.0 * s["max_q"] * (Hq // H) / max(kvs))
    return s


# ------------------------------------------------------------------ plain forms


def _cached(s, n, dtype=torch.float32):
    """The sequences' cached values [B, H, S, D], S the table's width in tokens; zero where no token is."""
    c = s["c"]
    B, H, D = c["B"], c["Hkv"], c["D"]
    t = s["table"].clamp(min=0).long()
    x = s[n + "c"][t]
    if c["mode"].startswith("fp8"):
        x = x.view(torch.float8_e4m3fn)
    x = x.to(dtype)
    x = (x.permute(0, 2, 1, 3, 4) if c["layout"] == "BNSD" else x.permute(0, 3, 1, 2, 4)).reshape(B, H, -1, D)
    sc = s[n + "s"].to(dtype)
    sc = sc[None, :, None, None] if c["mode"] in HEAD_MODES else sc[t].permute(0, 2, 1, 3).reshape(B, H, -1)[..., None]
    live = torch.arange(x.shape[2], device=x.device)[None] < s["lens"][:, None]
    return torch.where(live[:, None, :, None], x * sc, x.new_zeros(()))


def _rows(s):
    """Which sequence each new token belongs to, and which of its new tokens it is."""
    T = sum(_lengths(s["c"])[0])
    t = torch.arange(T, device="cuda")
    b = torch.searchsorted(s["cu"][1:].long().contiguous(), t, right=True)
    return t, b, t - s["cu"].long()[b]


def _scores(s):
    """Scaled scores [B, Hkv, max_q * group, S], minus infinity where a key is not visible, and the padded
    rows' visibility."""
    c = s["c"]
    B, H, D, Q = c["B"], c["Hkv"], c["D"], s["max_q"]
    G = c["Hq"] // H
    n = s["cu"][1:] - s["cu"][:-1]
    i = torch.arange(Q, device="cuda")
    at = (s["cu"][:-1, None] + i[None]).clamp(max=s["q"].shape[0] - 1).long()
    q = s["q"][at].float().view(B, Q, H, G, D).permute(0, 2, 1, 3, 4).reshape(B, H, Q * G, D)
    x = torch.matmul(q, _cached(s, "k").transpose(2, 3)).mul_(D ** -0.5).view(B, H, Q, G, -1)
    j = torch.arange(x.shape[-1], device="cuda")
    end = s["lens"][:, None] + (torch.zeros_like(i)[None] if not c["causal"] else i[None] + 1 - n[:, None])
    end = torch.where(i[None] < n[:, None], torch.minimum(end, s["lens"][:, None]), torch.zeros_like(end))
    x.masked_fill_((j[None, None] >= end[:, :, None])[:, None, :, None], float("-inf"))
    return x


def _softmax(x):
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == float("-inf"), torch.zeros_like(m), m)
    x = x.sub_(m).exp_()
    l = x.sum(-1, keepdim=True)
    return x, m, l


def _weights(s):
    """Unnormalised softmax [B, H, Q, G, S] and, per new token, the rows' log-sum-exp [T, Hq]; row sums."""
    p, m, l = _softmax(_scores(s))
    _, b, i = _rows(s)
    lse = (m + l.log())[..., 0].permute(0, 2, 1, 3)[b, i].reshape(-1, s["c"]["Hq"])
    return p, lse, l


def _attend(s):
    c = s["c"]
    p, lse, l = _weights(s)
    t, b, i = _rows(s)
    B, H, Q, G, S = p.shape
    o = torch.matmul(p.view(B, H, Q * G, S), _cached(s, "v")).view(B, H, Q, G, -1)
    o = torch.where(l > 0, o / l, torch.zeros_like(o)).permute(0, 2, 1, 3, 4)[b, i].reshape(len(t), c["Hq"], c["D"])
    s["out"][: len(t)] = o.to(torch.bfloat16)
    s["lse"][: len(t)] = lse
    return [s["out"], s["lse"]]


def _weigh(s):
    c = s["c"]
    x = _scores(s)
    B, H, Q, G, S = x.shape
    at = (s["cu"][:-1, None] + torch.arange(Q, device="cuda")[None]).clamp(max=s["q"].shape[0] - 1).long()
    lse = s["lse"][at].view(B, Q, H, G).permute(0, 2, 1, 3)[..., None]
    p = torch.where(lse > float("-inf"), x.sub_(lse).exp_(), x.new_zeros(()))
    s["acc"] += p.sum((2, 3))
    return [s["acc"]]


def _turn(x, cs, inter, rd):
    """x [T, H, D] with its first rd elements rotated by the tokens' (cos | sin) rows."""
    cos, sin = (v[:, None] for v in cs.chunk(2, -1))
    r = x[..., :rd]
    a, b = (r[..., 0::2], r[..., 1::2]) if inter else r.chunk(2, -1)
    u, w = a * cos - b * sin, b * cos + a * sin
    r = torch.stack((u, w), -1).flatten(-2) if inter else torch.cat((u, w), -1)
    return torch.cat((r, x[..., rd:]), -1)


def _append(s):
    c = s["c"]
    H, page = c["Hkv"], c["page"]
    fp8, qmax = c["mode"].startswith("fp8"), 448.0 if c["mode"].startswith("fp8") else 127.0
    t, b, i = _rows(s)
    T = len(t)
    cs = s["cos_sin"][s["pos"][:T].long()]
    s["out"][:T] = _turn(s["q"][:T].float(), cs, c["inter"], c["rd"]).to(torch.bfloat16)
    k = _turn(s["k"][:T].float(), cs, c["inter"], c["rd"]).to(torch.bfloat16).float()
    n = (s["lens"].long() - (s["cu"][1:] - s["cu"][:-1]))[b] + i
    pg, o = s["table"][b, n // page].long(), n % page
    for x, name, am in ((k, "k", s["amax"][0]), (s["v"][:T].float(), "v", s["amax"][1])):
        # divisors as tensors: a division, not a product with the reciprocal
        top = torch.full((), qmax, device=x.device)
        if c["mode"] in HEAD_MODES:
            sc = am / top
            s[name + "s"].copy_(sc)
            sc = sc[None, :, None]
        else:
            sc = (x.abs().amax(-1) / top)
            s[name + "s"][pg, :, o] = sc
            sc = sc[..., None]
        y = torch.where(sc > 0, x / sc, torch.zeros_like(x))
        y = _e4m3(y).view(torch.uint8) if fp8 else y.round().clamp(-128, 127).to(torch.int8)
        if c["layout"] == "BNSD":
            s[name + "c"][pg, :, o] = y
        else:
            s[name + "c"][pg, o] = y
    return [s["out"]] + _cache_out(s)


def _cache_out(s):
    codes = [s["kc"], s["vc"]]
    if s["c"]["mode"].startswith("fp8"):
        codes = [x.view(torch.float8_e4m3fn) for x in codes]
    return codes + [s["ks"], s["vs"]]


def _evict(s):
    c = s["c"]
    B, H, page, budget = c["B"], c["Hkv"], c["page"], c["budget"]
    x, n = s["scores"], s["lens"].long()
    cap = x.shape[-1]
    j = torch.arange(cap, device=x.device)
    kind = torch.where(j[None] >= n[:, None], 2, 1)
    kind = torch.where((kind == 1) & ((j[None] < c["sink"]) | (j[None] >= (n - c["recent"])[:, None])), 0, kind)
    kind = kind[:, None].expand(B, H, cap)
    order = torch.argsort(x, dim=-1, descending=True, stable=True)
    order = order.gather(-1, torch.argsort(kind.gather(-1, order), dim=-1, stable=True))
    r = torch.arange(budget, device=x.device)
    new = n.clamp(max=budget)
    if cap < budget:
        order = torch.cat((order, order.new_full((B, H, budget - cap), cap)), -1)
    kept = torch.where(r[None, None] < new[:, None, None], order[..., :budget], cap).sort(-1).values
    live = kept < cap
    src = kept.clamp(max=cap - 1)
    got = torch.where(live, x.gather(-1, src), x.new_zeros(()))
    s["scores_out"].zero_()
    s["scores_out"][..., : min(budget, cap)] = got[..., : min(budget, cap)]
    # rows moved to the front: all read before any is written
    b, h, d = (v.expand(B, H, budget)[live] for v in (torch.arange(B, device=x.device)[:, None, None],
                                                      torch.arange(H, device=x.device)[None, :, None], r[None, None]))
    f = src[live]
    pf, of, pd, od = s["table"][b, f // page].long(), f % page, s["table"][b, d // page].long(), d % page
    for name in ("k", "v"):
        if c["layout"] == "BNSD":
            s[name + "c"][pd, h, od] = s[name + "c"][pf, h, of]
        else:
            s[name + "c"][pd, od, h] = s[name + "c"][pf, of, h]
        if c["mode"] not in HEAD_MODES:
            s[name + "s"][pd, h, od] = s[name + "s"][pf, h, of]
    return [torch.where(live, kept, -1).to(torch.int32), new.to(torch.int32), s["scores_out"]] + _cache_out(s)


def run(state):
    s = state
    c = s["c"]
    if own:
        return _own(s)
    return {"append": _append, "attend": _attend, "weigh": _weigh, "evict": _evict}[c["op"]](s)


def _own(s):
    import quantized_attention_amax_b200 as faq

    c = s["c"]
    cache = faq.PagedCache(s["kc"], s["vc"], s["ks"], s["vs"], c["mode"], c["layout"])
    batch = faq.PagedBatch(s["table"], s["lens"], s.get("cu"), s.get("max_q", 0))
    if c["op"] == "append":
        faq.rope_append(s["q"], s["k"], s["v"], cache, batch, s["cos_sin"], s["pos"], interleaved=c["inter"],
                        amax=s["amax"] if c["mode"] in HEAD_MODES else None, out=s["out"])
        return [s["out"]] + _cache_out(s)
    if c["op"] == "attend":
        faq.paged_attention(s["q"], cache, batch, causal=c["causal"], out=s["out"], lse=s["lse"])
        return [s["out"], s["lse"]]
    if c["op"] == "weigh":
        faq.paged_weights(s["q"], s["lse"], cache, batch, s["acc"], causal=c["causal"])
        return [s["acc"]]
    kept, new = faq.paged_evict(cache, batch, s["scores"], c["budget"], c["sink"], c["recent"], scores_out=s["scores_out"])
    return [kept, new, s["scores_out"]] + _cache_out(s)


# ------------------------------------------------------------------ work and the exact values


def work(case):
    c = case
    qs, kvs = _lengths(c)
    H, D, T = c["Hkv"], c["D"], sum(qs)
    token = D + (0 if c["mode"] in HEAD_MODES else 4)  # a cached row's codes and its scale
    if c["op"] == "append":
        b = T * (2 * (2 * c["Hq"] + 2 * H) * D + 2 * H * token + 4 * c["rd"])
        return {"bytes": b, "flops": T * (c["Hq"] + H) * 3 * c["rd"]}
    if c["op"] == "evict":
        kept = sum(min(n, c["budget"]) for n in kvs)
        moved = sum(min(n, c["budget"]) for n in kvs if n > c["budget"])
        return {"bytes": H * (4 * sum(kvs) + 4 * kept + 4 * kept + 4 * moved * token), "flops": 0}
    pairs = 0
    for n, m in zip(qs, kvs):
        pairs += sum(max(0, min(m, i + 1 + m - n)) for i in range(n)) if c["causal"] else n * m
    if c["op"] == "attend":
        return {"bytes": 2 * H * sum(kvs) * token + T * c["Hq"] * (4 * D + 4), "flops": 4 * D * c["Hq"] * pairs}
    return {"bytes": H * sum(kvs) * (token + 8) + T * c["Hq"] * (2 * D + 4), "flops": 2 * D * c["Hq"] * pairs}


def exact(case, seed):
    """The definitions in 64 bits; None in the place of codes and indices."""
    c = case
    s = prepare(c, seed)
    qs, kvs = _lengths(c)
    H, D, page = c["Hkv"], c["D"], c["page"]
    f64 = torch.float64
    if c["op"] == "evict":
        return None
    if c["op"] == "append":
        T = sum(qs)
        cs = s["cos_sin"][s["pos"][:T].long()].to(f64)
        half = c["rd"] // 2
        cos, sin = cs[:, None, :half], cs[:, None, half:]

        def turned(x):
            y = x.to(f64).clone()
            i = torch.arange(half, device=x.device)
            a, b = (2 * i, 2 * i + 1) if c["inter"] else (i, i + half)
            xa, xb = y[..., a].clone(), y[..., b].clone()
            y[..., a], y[..., b] = xa * cos - xb * sin, xa * sin + xb * cos
            return y

        out = s["out"].to(f64)
        out[:T] = turned(s["q"][:T])
        k, v = turned(s["k"][:T]).to(torch.bfloat16).to(f64), s["v"][:T].to(f64)
        top = 448.0 if c["mode"].startswith("fp8") else 127.0
        if c["mode"] in HEAD_MODES:
            return [out, None, None, s["amax"][0].to(f64) / top, s["amax"][1].to(f64) / top]
        ks, vs = s["ks"].to(f64), s["vs"].to(f64)
        t = 0
        for b, (n, m) in enumerate(zip(qs, kvs)):
            at = torch.arange(m - n, m, device="cuda")
            pg = s["table"][b].long()[at // page]
            ks[pg, :, at % page] = k[t:t + n].abs().amax(-1) / top
            vs[pg, :, at % page] = v[t:t + n].abs().amax(-1) / top
            t += n
        return [out, None, None, ks, vs]
    G = c["Hq"] // H
    t = 0
    out = s["out"].to(f64) if c["op"] == "attend" else None
    lse = s["lse"].to(f64)
    acc = s["acc"].to(f64) if c["op"] == "weigh" else None
    for b, (n, m) in enumerate(zip(qs, kvs)):
        at = torch.arange(m, device="cuda")
        pg, o = s["table"][b].long()[at // page], at % page
        end = torch.arange(n, device="cuda") + 1 + m - n if c["causal"] else torch.full((n,), m, device="cuda")
        hide = at[None] >= end[:, None]

        def head(name, h):
            x = s[name + "c"][pg, h, o] if c["layout"] == "BNSD" else s[name + "c"][pg, o, h]
            x = (x.view(torch.float8_e4m3fn) if c["mode"].startswith("fp8") else x).to(f64)
            w = s[name + "s"].to(f64)
            return x * (w[h] if c["mode"] in HEAD_MODES else w[pg, h, o][:, None])

        for h in range(H):
            k, v = head("k", h), head("v", h) if c["op"] == "attend" else None
            for r in range(h * G, h * G + G):
                x = (s["q"][t:t + n, r].to(f64) @ k.T) / D ** 0.5
                x = x.masked_fill(hide, float("-inf"))
                if c["op"] == "attend":
                    z = torch.logsumexp(x, -1)
                    p = torch.where(z[:, None] > float("-inf"), (x - z[:, None]).exp(), 0.0)
                    out[t:t + n, r], lse[t:t + n, r] = p @ v, z
                else:
                    z = lse[t:t + n, r]
                    acc[b, h, :m] += torch.where(z[:, None] > float("-inf"), (x - z[:, None]).exp(), 0.0).sum(0)
        t += n
    return [out, lse] if c["op"] == "attend" else [acc]
