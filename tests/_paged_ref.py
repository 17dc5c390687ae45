"""Plain 64-bit forms of the paged-cache operators for the tests (CPU torch; no code of the package).

A paged cache here is a dict of CPU tensors: kc, vc (codes), ks, vs (scales), mode, layout, page."""
import torch

PER_HEAD = ("int8_per_head", "fp8_per_head")
MODES = ("int8_per_head", "fp8_per_head", "int8_per_token", "fp8_per_token")


def e4m3(x):
    return x.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)


def values(cache, name):
    c = cache[name + "c"]
    return (c.view(torch.float8_e4m3fn).to(torch.float32) if cache["mode"].startswith("fp8") else c).to(torch.float64)


def slots(cache, table_row, js):
    page = cache["page"]
    return table_row[js // page].long(), js % page


def head_rows(cache, name, h, pg, o):
    """Dequantized rows [n, D] of slots (pg, o) of kv head h."""
    x = values(cache, name)
    x = x[pg, h, o] if cache["layout"] == "BNSD" else x[pg, o, h]
    s = cache[name + "s"].to(torch.float64)
    return x * (s[h] if cache["mode"] in PER_HEAD else s[pg, h, o][:, None])


def make_cache(mode, layout, pages, H, page, D, seed, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    qmax = 448.0 if mode.startswith("fp8") else 127.0
    shp = (pages, H, page, D) if layout == "BNSD" else (pages, page, H, D)
    c = dict(mode=mode, layout=layout, page=page, H=H, D=D)
    for n in "kv":
        x = torch.randn(shp, generator=g) * (qmax / 4.5)
        c[n + "c"] = e4m3(x) if mode.startswith("fp8") else x.round().clamp(-128, 127).to(torch.int8)
        s = (H,) if mode in PER_HEAD else (pages, H, page)
        c[n + "s"] = (4.5 / qmax) * (spread * torch.randn(s, generator=g)).exp()
    return c


def make_table(lens, page, seed, spare=2):
    """A table whose sequences' pages lie in no order; entries past a sequence's end are -1."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-n // page) for n in lens]
    pages = sum(need) + spare
    order = torch.randperm(pages, generator=g).to(torch.int32)
    table = torch.full((len(lens), max(need + [1])), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table, pages


def visible(n, m, causal):
    """[m, n] bool: does new token i see cached key j."""
    i, j = torch.arange(m)[:, None], torch.arange(n)[None]
    return (j <= n - m + i) if causal else torch.ones(m, n, dtype=torch.bool)


def scores(q, k, scale):
    """Scaled scores and, per score, sum_d |q_d k_d| scale (for error bounds)."""
    q, k = q.to(torch.float64), k.to(torch.float64)
    return q @ k.T * scale, q.abs() @ k.abs().T * scale


def attend(q, cache, table, lens, qlens, causal, scale=None):
    """q [T, Hq, D] bf16 -> per (token, head): out, lse, the error bound of each.  Rows of no sequence
    are absent (NaN bound -> not compared)."""
    T, Hq, D = q.shape
    H = cache["H"]
    G = Hq // H
    scale = D ** -0.5 if scale is None else scale
    out, lse = torch.zeros(T, Hq, D, dtype=torch.float64), torch.full((T, Hq), -torch.inf, dtype=torch.float64)
    tol, ltol = torch.zeros_like(out), torch.zeros_like(lse)
    t = 0
    for b, (n, m) in enumerate(zip(lens, qlens)):
        if m and n:
            js = torch.arange(n)
            pg, o = slots(cache, table[b], js)
            see = visible(n, m, causal)
            for h in range(H):
                k, v = head_rows(cache, "k", h, pg, o), head_rows(cache, "v", h, pg, o)
                sv = cache["vs"].to(torch.float64)
                sv = sv[h].expand(n) if cache["mode"] in PER_HEAD else sv[pg, h, o]
                code = v.abs() / sv[:, None]
                for r in range(h * G, h * G + G):
                    x, ax = scores(q[t:t + m, r], k, scale)
                    x = x.masked_fill(~see, -torch.inf)
                    z = torch.logsumexp(x, -1)
                    some = z > -torch.inf
                    p = torch.where(some[:, None], (x - z[:, None]).exp(), 0.0)
                    out[t:t + m, r], lse[t:t + m, r] = p @ v, z
                    # a score is a sum of D fp32 products (D + 8 roundings of 2^-24 of sum |q_d k_d|), then
                    # scaled and shifted in the exponent: 4 roundings of 2^-24 of |x| + |max| each
                    xe = torch.where(see, ax * (D + 8) * 2.0 ** -24 + x.abs().nan_to_num(posinf=0.0) * 2.0 ** -21, 0.0)
                    big = xe.amax(-1) + 2.0 ** -20
                    # a factor w_j = p_j s_v(j) enters the product with at least 11 bits (half a step 2^-11: fp16,
                    # or three E4M3 digits of 4 bits), but no finer than a fixed step below the row's largest
                    # w: fp16 of w 2^14 has steps 2^-24 / 2^14, three E4M3 digits of 256 w have a last step of
                    # 2^-9 / 256 / 256 = 2^-25 (half: 2^-26), 24-bit integers 2^-24 (half: 2^-25, and 2^-24 where w = 1
                    # is held as 1 - 2^-24): at most 2^-24 of the largest, times the key's code.
                    # bf16 output: half a step 2^-8.
                    pe = p * (2.0 ** -11 + 2.0 * big[:, None])
                    top = (p * sv).amax(-1, keepdim=True) * 2.0 ** -24
                    tol[t:t + m, r] = out[t:t + m, r].abs() * 2.0 ** -8 + (1 + 2.0 ** -7) * (
                        pe @ v.abs() + top * (see.to(torch.float64) @ code)) + 1e-30
                    ltol[t:t + m, r] = 2 * big + z.abs().nan_to_num(posinf=0.0) * 2.0 ** -22
        t += m
    return out, lse, tol, ltol


def weigh(q, lse, cache, table, lens, qlens, causal, stride, scale=None):
    """The new weights [B, H, stride] and their error bounds; lse fp32 [T, Hq] as given."""
    T, Hq, D = q.shape
    H = cache["H"]
    G = Hq // H
    scale = D ** -0.5 if scale is None else scale
    w = torch.zeros(len(lens), H, stride, dtype=torch.float64)
    tol = torch.zeros_like(w)
    t = 0
    for b, (n, m) in enumerate(zip(lens, qlens)):
        if m and n:
            pg, o = slots(cache, table[b], torch.arange(n))
            see = visible(n, m, causal)
            for h in range(H):
                k = head_rows(cache, "k", h, pg, o)
                for r in range(h * G, h * G + G):
                    x, ax = scores(q[t:t + m, r], k, scale)
                    z = lse[t:t + m, r].to(torch.float64)
                    some = (z > -torch.inf)[:, None] & see
                    p = torch.where(some, (x - z[:, None]).exp(), 0.0)
                    e = ax * (D + 8) * 2.0 ** -24 + (x.abs() + z.abs()[:, None].nan_to_num(posinf=0.0)) * 2.0 ** -22 + 2.0 ** -21
                    w[b, h, :n] += p.sum(0)
                    tol[b, h, :n] += (p * 2 * e).sum(0)
        t += m
    rows = max(list(qlens) + [1]) * G
    return w, tol + w * rows * 2.0 ** -24 + 1e-30


def evict(cache, table, lens, sc, budget, sink, recent):
    """kept [B, H, budget] (-1 past the end), new lengths, moved scores; the cache's tensors change."""
    B, H, stride = sc.shape
    kept = torch.full((B, H, budget), -1, dtype=torch.int32)
    so = torch.zeros_like(sc)
    new = torch.tensor([min(n, budget) for n in lens], dtype=torch.int32)
    for b, n in enumerate(lens):
        for h in range(H):
            if n <= budget:
                idx = list(range(n))
            else:
                mid = range(sink, n - recent)
                val = sc[b, h].tolist()
                order = sorted(mid, key=lambda j: (val[j] != val[j], -val[j] if val[j] == val[j] else 0.0, j))
                idx = sorted(list(range(sink)) + order[: budget - sink - recent] + list(range(n - recent, n)))
            k = len(idx)
            f = torch.tensor(idx, dtype=torch.long)
            kept[b, h, :k] = f.to(torch.int32)
            so[b, h, :k] = sc[b, h, f]
            if n <= budget or not k:
                continue
            (pf, of), (pd, od) = slots(cache, table[b], f), slots(cache, table[b], torch.arange(k))
            for name in "kv":
                c = cache[name + "c"]
                if cache["layout"] == "BNSD":
                    c[pd, h, od] = c[pf, h, of].clone()
                else:
                    c[pd, od, h] = c[pf, of, h].clone()
                if cache["mode"] not in PER_HEAD:
                    s = cache[name + "s"]
                    s[pd, h, od] = s[pf, h, of].clone()
    return kept, new, so


def turn(x, cs, inter):
    """x [T, H, D] bf16 rotated by fp32 rows cs [T, rd], every product and sum rounded to fp32, then bf16."""
    rd = cs.shape[1]
    y = x.to(torch.float32).clone()
    i = torch.arange(rd // 2)
    a, b = (2 * i, 2 * i + 1) if inter else (i, i + rd // 2)
    c, s = cs[:, None, : rd // 2], cs[:, None, rd // 2:]
    xa, xb = y[..., a].clone(), y[..., b].clone()
    y[..., a], y[..., b] = xa * c - xb * s, xb * c + xa * s
    return y.to(torch.bfloat16)
