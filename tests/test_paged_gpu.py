"""GPU tests of the paged-cache operators against their 64-bit forms (tests/_paged_ref.py): every mode,
both layouts, ragged batches, lengths of zero and one, pages that end inside a tile, rows that see no
key, NaN in places no row sees, padded rows, strided inputs, CUDA graphs, streams and bad device data."""
import numpy as np
import pytest
import torch

import _paged_ref as ref
import workloads as wl
from _gpu import faq_module

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def faq():
    return faq_module()


def to_gpu(faq, c):
    return faq.PagedCache(c["kc"].cuda(), c["vc"].cuda(), c["ks"].cuda(), c["vs"].cuda(), c["mode"], c["layout"])


def batch_of(faq, table, lens, qlens=None, max_q=0):
    cu = None
    if qlens is not None:
        cu = torch.tensor([0] + list(np.cumsum(qlens)), dtype=torch.int32).cuda()
    return faq.PagedBatch(table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), cu, max_q)


def bf16(shape, seed, gain=1.0):
    return (torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * gain).to(torch.bfloat16)


def poison(c, table, lens):
    """NaN codes and scales in every slot that no sequence holds."""
    live = torch.zeros((c["kc"].shape[0], c["page"]), dtype=torch.bool)
    for b, n in enumerate(lens):
        js = torch.arange(n)
        live[table[b, js // c["page"]].long(), js % c["page"]] = True
    for n in "kv":
        codes = c[n + "c"] if c["layout"] == "BNSD" else c[n + "c"].transpose(1, 2)
        if c["mode"].startswith("fp8"):
            codes.masked_fill_(~live[:, None, :, None], 0x7F)
        if c["mode"] not in ref.PER_HEAD:
            c[n + "s"].masked_fill_(~live[:, None], float("nan"))


def assert_within(got, want, tol, what):
    got = got.double().cpu()
    inf = torch.isinf(want)
    assert torch.equal(torch.isinf(got), inf) and torch.equal(got[inf], want[inf]), what
    over = ((got - want).abs() - tol)[~inf]
    assert not torch.isnan(over).any() and (over.numel() == 0 or over.max() <= 0), \
        f"{what}: {int((over > 0).sum())} of {over.numel()} outside, by {float(over.max()):.3g}"


# lens, qlens, Hq, Hkv, D, page: lengths of zero and one, more new tokens than cached ones (rows that see
# nothing), odd groups, query rows past one block, tiles and pages that end early
SHAPES = [
    ((1,), (1,), 4, 1, 128, 16),
    ((0, 5, 1), (1, 1, 1), 8, 2, 128, 16),
    ((300, 17, 256, 1000), (1, 1, 1, 1), 16, 4, 128, 64),
    ((257, 31, 64), (1, 0, 3), 6, 2, 64, 32),
    ((2, 700), (5, 9), 6, 2, 128, 128),
    ((513, 90), (40, 90), 4, 4, 64, 16),
    ((400,), (150,), 10, 2, 128, 1024),
    ((129, 1, 640), (1, 1, 17), 34, 2, 128, 64),
    ((1500, 1100), (260, 1), 8, 1, 128, 64),
    ((700, 130, 16), (1, 1, 1), 5, 1, 128, 16),
    ((90, 33), (2, 1), 3, 1, 64, 16),
]


@pytest.mark.parametrize("shape", range(len(SHAPES)))
@pytest.mark.parametrize("mode", ref.MODES)
@pytest.mark.parametrize("layout,causal", [("BNSD", True), ("BSND", True), ("BSND", False)])
def test_attention(faq, shape, mode, layout, causal):
    lens, qlens, Hq, Hkv, D, page = SHAPES[shape]
    table, pages = ref.make_table(lens, page, 3 * shape)
    c = ref.make_cache(mode, layout, pages, Hkv, page, D, 7 + shape, spread=0.5)
    poison(c, table, lens)
    T, pad = sum(qlens), 2
    q = bf16((T + pad, Hq, D), 11 + shape, 1.5)
    want, lse, tol, ltol = ref.attend(q[:T], c, table, lens, qlens, causal)
    gc, gb = to_gpu(faq, c), batch_of(faq, table, lens, qlens)
    out = torch.full((T + pad, Hq, D), 7.0, dtype=torch.bfloat16).cuda()
    z = torch.full((T + pad, Hq), 7.0).cuda()
    faq.paged_attention(q.cuda(), gc, gb, causal=causal, out=out, lse=z)
    faq.check_device_status()
    assert_within(out[:T], want, tol, "out")
    assert_within(z[:T], lse, ltol, "lse")
    assert (out[T:] == 7.0).all() and (z[T:] == 7.0).all()  # rows of no sequence
    again = faq.paged_attention(q.cuda(), gc, gb, causal=causal, out=torch.full_like(out, 7.0))
    assert torch.equal(again.view(torch.int16), out.view(torch.int16))


def test_attention_scale_bound_and_strided_rows(faq):
    """A given softmax scale, max_q given, and q as columns of a wider matrix."""
    lens, qlens = (200, 75), (20, 3)
    table, pages = ref.make_table(lens, 32, 1)
    c = ref.make_cache("int8_per_token", "BNSD", pages, 2, 32, 64, 2, spread=0.5)
    x = bf16((23, 12, 64), 3)
    q = x[:, 2:8]
    want, lse, tol, ltol = ref.attend(q, c, table, lens, qlens, True, 0.3)
    out, z = faq.paged_attention(x.cuda()[:, 2:8], to_gpu(faq, c), batch_of(faq, table, lens, qlens, 20),
                                 softmax_scale=0.3, return_lse=True)
    faq.check_device_status()
    assert_within(out, want, tol, "out")
    assert_within(z, lse, ltol, "lse")


@pytest.mark.parametrize("mode", ref.MODES)
@pytest.mark.parametrize("rows", [1, 40])
def test_attention_long_and_sharp(faq, mode, rows):
    """Long histories over many runs; scores far apart, V scales over nine orders of magnitude."""
    lens, qlens = (20011, 4097), (rows, 1)
    table, pages = ref.make_table(lens, 64, 5)
    c = ref.make_cache(mode, "BNSD", pages, 2, 64, 128, 6, spread=0.2)
    if mode not in ref.PER_HEAD:
        c["vs"] *= 10.0 ** torch.randint(-6, 4, c["vs"].shape, generator=torch.Generator().manual_seed(1)).float()
    q = bf16((rows + 1, 8, 128), 8, 8.0)
    want, lse, tol, ltol = ref.attend(q, c, table, lens, qlens, True)
    out, z = faq.paged_attention(q.cuda(), to_gpu(faq, c), batch_of(faq, table, lens, qlens), return_lse=True)
    faq.check_device_status()
    assert_within(out, want, tol, "out")
    assert_within(z, lse, ltol, "lse")


@pytest.mark.parametrize("gain", [1e-30, 1e30])
def test_attention_query_range(faq, gain):
    """Queries whose values lie outside fp16's range: scores vanish, or one key takes all."""
    lens, qlens = (150,), (4,)
    table, pages = ref.make_table(lens, 16, 2)
    c = ref.make_cache("fp8_per_head", "BNSD", pages, 2, 16, 64, 3)
    q = bf16((4, 4, 64), 4, gain)
    want, lse, tol, ltol = ref.attend(q, c, table, lens, qlens, True)
    out, z = faq.paged_attention(q.cuda(), to_gpu(faq, c), batch_of(faq, table, lens, qlens), return_lse=True)
    faq.check_device_status()
    if gain > 1:  # scores of 1e30: the largest wins by more than its rounding
        assert_within(out, want, want.abs() * 2.0 ** -7 + 1e-6 * want.abs().max(), "out")
        assert ((z.cpu().double() - lse).abs() <= lse.abs() * 1e-5).all()
    else:
        assert_within(out, want, tol, "out")
        assert_within(z, lse, ltol, "lse")


def test_nan_in_a_visible_row_shows_and_in_a_hidden_one_does_not(faq):
    """Per-token modes: a NaN scale (what the append leaves for a row with NaN) reaches the rows that see the
    token and no others."""
    for mode in ("int8_per_token", "fp8_per_token"):
        for rows in (3, 70):
            n = 200
            lens, qlens = (n,), (rows,)
            table, pages = ref.make_table(lens, 16, 2)
            c = ref.make_cache(mode, "BNSD", pages, 1, 16, 128, 3)
            q = bf16((rows, 2, 128), 4)
            want, _, tol, _ = ref.attend(q, c, table, lens, qlens, True)
            bad = n - 1  # seen by the last new token only
            pg, o = int(table[0, bad // 16]), bad % 16
            c["vs"][pg, 0, o] = float("nan")
            out = faq.paged_attention(q.cuda(), to_gpu(faq, c), batch_of(faq, table, lens, qlens))
            faq.check_device_status()
            assert torch.isnan(out[-1]).all()
            assert_within(out[:-1], want[:-1], tol[:-1], mode)


def test_attention_pages_past_32_bits(faq):
    """Codes more than 2^31 bytes into the pool."""
    H, page, D = 8, 128, 128
    pages = (1 << 31) // (H * page * D) + 40
    lens, qlens = (500, 300), (1, 30)
    need = [4, 3]
    table = torch.full((2, 4), -1, dtype=torch.int32)
    ids = [pages - 1, 3, pages - 9, pages - 20, pages - 2, 0, pages - 30]
    table[0], table[1, :3] = torch.tensor(ids[:4], dtype=torch.int32), torch.tensor(ids[4:], dtype=torch.int32)
    small_table = torch.full((2, 4), -1, dtype=torch.int32)
    small_table[0], small_table[1, :3] = torch.arange(4, dtype=torch.int32), torch.arange(4, 7, dtype=torch.int32)
    c = ref.make_cache("int8_per_token", "BNSD", sum(need), H, page, D, 4)
    q = bf16((31, 16, D), 5)
    want, lse, tol, ltol = ref.attend(q, c, small_table, lens, qlens, True)
    big = faq.empty_paged_cache(pages, H, page, D, "int8_per_token")
    at = torch.tensor(ids).cuda()
    for n, t in (("kc", big.k_codes), ("vc", big.v_codes), ("ks", big.k_scales), ("vs", big.v_scales)):
        t[at] = c[n].cuda()
    gb = batch_of(faq, table, lens, qlens)
    out, z = faq.paged_attention(q.cuda(), big, gb, return_lse=True)
    faq.check_device_status()
    assert_within(out, want, tol, "out")
    w, wtol = ref.weigh(q, z.cpu(), c, small_table, lens, qlens, True, 512)
    acc = faq.paged_weights(q.cuda(), z, big, gb, torch.zeros(2, H, 512).cuda())
    assert_within(acc, w, wtol, "weights")
    sc = torch.rand(2, H, 512, generator=torch.Generator().manual_seed(6))
    kept, new, _ = ref.evict(c, small_table, lens, sc, 100, 1, 5)
    gk, gn = faq.paged_evict(big, gb, sc.cuda(), 100, 1, 5)
    faq.check_device_status()
    assert torch.equal(gk.cpu(), kept) and torch.equal(gn.cpu(), new)
    for n, t in (("kc", big.k_codes), ("vc", big.v_codes), ("ks", big.k_scales), ("vs", big.v_scales)):
        assert torch.equal(t[at].cpu(), c[n]), n


@pytest.mark.parametrize("shape", range(len(SHAPES)))
@pytest.mark.parametrize("mode", ref.MODES)
@pytest.mark.parametrize("layout,causal", [("BNSD", True), ("BSND", False)])
def test_weights(faq, shape, mode, layout, causal):
    lens, qlens, Hq, Hkv, D, page = SHAPES[shape]
    table, pages = ref.make_table(lens, page, 3 * shape)
    c = ref.make_cache(mode, layout, pages, Hkv, page, D, 7 + shape, spread=0.5)
    T, pad = sum(qlens), 3
    q = bf16((T + pad, Hq, D), 11 + shape, 1.5)
    _, lse, _, _ = ref.attend(q[:T], c, table, lens, qlens, causal)
    poison(c, table, lens)
    lse32 = torch.cat((lse.float(), torch.zeros(pad, Hq)))
    stride = max(lens) + 5
    w, tol = ref.weigh(q[:T], lse32[:T], c, table, lens, qlens, causal, stride)
    g = torch.Generator().manual_seed(1)
    acc0 = torch.rand(len(lens), Hkv, stride, generator=g)
    gc, gb = to_gpu(faq, c), batch_of(faq, table, lens, qlens)
    live = torch.arange(stride)[None] < torch.tensor(lens)[:, None]
    for add in (True, False):
        acc = acc0.clone().cuda()
        got = faq.paged_weights(q.cuda(), lse32.cuda(), gc, gb, acc, causal=causal, accumulate=add)
        faq.check_device_status()
        # without accumulate a sequence with no new tokens gets zeros; with it, it keeps what it had
        want = torch.where(live[:, None], w + (acc0.double() if add else 0.0), acc0.double())
        assert_within(got, want, tol + (want.abs() * 2.0 ** -24 if add else 0.0), f"add {add}")
        # past the lengths nothing is written
        assert torch.equal(got.cpu().masked_select(~live[:, None].expand_as(want)),
                           acc0.masked_select(~live[:, None].expand_as(want)))


def test_weights_sum_to_the_rows(faq):
    """Every row's probabilities sum to one: a head's weights sum to its visible rows."""
    lens, qlens = (900, 33), (50, 33)
    table, pages = ref.make_table(lens, 64, 1)
    c = ref.make_cache("fp8_per_token", "BNSD", pages, 2, 64, 128, 2)
    q = bf16((83, 6, 128), 3)
    gc, gb = to_gpu(faq, c), batch_of(faq, table, lens, qlens)
    _, lse = faq.paged_attention(q.cuda(), gc, gb, return_lse=True)
    acc = faq.paged_weights(q.cuda(), lse, gc, gb, torch.zeros(2, 2, 900).cuda())
    faq.check_device_status()
    want = torch.tensor([[50.0 * 3] * 2, [33.0 * 3] * 2], dtype=torch.float64)
    assert ((acc.double().sum(-1).cpu() - want).abs() <= want * 1e-5).all()


EVICTIONS = [  # lens, Hkv, D, page, budget, sink, recent
    ((1,), 1, 64, 16, 1, 0, 0),
    ((0, 40, 7), 2, 128, 16, 7, 0, 7),
    ((300, 64, 65), 2, 128, 64, 64, 4, 10),
    ((1000, 513), 3, 64, 32, 200, 0, 1),
    ((5000,), 1, 128, 64, 4999, 1, 100),
    ((2600, 2000, 1), 8, 128, 128, 513, 4, 0),
    ((45000,), 1, 64, 64, 6000, 3, 30),
    ((100, 90), 20, 64, 16, 33, 33, 0),
]


@pytest.mark.parametrize("case", range(len(EVICTIONS)))
@pytest.mark.parametrize("mode", ref.MODES)
@pytest.mark.parametrize("layout", ["BNSD", "BSND"])
@pytest.mark.parametrize("kind", ["spread", "ties"])
def test_evict(faq, case, mode, layout, kind):
    lens, Hkv, D, page, budget, sink, recent = EVICTIONS[case]
    table, pages = ref.make_table(lens, page, case)
    c = ref.make_cache(mode, layout, pages, Hkv, page, D, 3 + case)
    g = torch.Generator().manual_seed(case)
    stride = max(lens) + 3
    sc = torch.randn(len(lens), Hkv, stride, generator=g)
    if kind == "ties":  # few values, both zeros, infinities, NaN
        vals = torch.tensor([0.0, -0.0, 1.0, 1.0, -2.0, float("inf"), float("-inf"), float("nan")])
        sc = vals[torch.randint(0, 8, sc.shape, generator=g)]
    gc, gb = to_gpu(faq, c), batch_of(faq, table, lens)
    kept, new, so = ref.evict(c, table, lens, sc, budget, sink, recent)
    out = torch.full_like(sc, 9.0).cuda()
    gk, gn = faq.paged_evict(gc, gb, sc.cuda(), budget, sink, recent, scores_out=out)
    faq.check_device_status()
    assert torch.equal(gk.cpu(), kept)
    assert torch.equal(gn.cpu(), new)
    assert torch.equal(out.cpu().view(torch.int32), so.view(torch.int32))
    for n, t in (("kc", gc.k_codes), ("vc", gc.v_codes), ("ks", gc.k_scales), ("vs", gc.v_scales)):
        assert torch.equal(t.cpu(), c[n]), n  # moved rows, and every other row as it was


APPENDS = [  # qlens, lens before, Hq, Hkv, D, page, rotary_dim, interleaved
    ((1,), (0,), 1, 1, 64, 16, 64, False),
    ((1, 1, 1), (0, 15, 16), 8, 2, 128, 16, 128, False),
    ((3, 0, 20, 1), (5, 9, 0, 62), 6, 2, 128, 64, 64, True),
    ((70, 5), (30, 1), 10, 5, 64, 32, 32, True),
    ((33,), (100,), 4, 4, 128, 128, 16, False),
    ((9, 2), (7, 0), 3, 1, 128, 16, 0, False),
    ((300, 211), (11, 0), 32, 8, 128, 64, 128, True),
]


@pytest.mark.parametrize("case", range(len(APPENDS)))
@pytest.mark.parametrize("mode", ref.MODES)
@pytest.mark.parametrize("layout", ["BNSD", "BSND"])
def test_append(faq, orc, case, mode, layout):
    qlens, before, Hq, Hkv, D, page, rd, inter = APPENDS[case]
    lens = [a + b for a, b in zip(before, qlens)]
    table, pages = ref.make_table(lens, page, case)
    c = ref.make_cache(mode, layout, pages, Hkv, page, D, case)
    T, pad = sum(qlens), 2
    x = bf16((T + pad, Hq + 2 * Hkv, D), 5 + case)
    x[0, :, 3] *= 30.0  # an outlier, past the static range too
    x[0, Hq] = 0.0      # an all-zero key
    seq = torch.cat([torch.arange(n) + p for n, p in zip(qlens, before)])
    pos = None if case % 2 else torch.cat((seq * 7 + 1000, torch.full((pad,), -5))).to(torch.int32)
    cs = faq.rope_table(8192, rd) if rd else None
    amax = (torch.rand(Hkv, generator=torch.Generator().manual_seed(1)) + 3.0, torch.full((Hkv,), 3.5))
    gc, gb = to_gpu(faq, c), batch_of(faq, table, lens, qlens)
    gx = x.cuda()
    out = torch.full((T + pad, Hq, D), 7.0, dtype=torch.bfloat16).cuda()
    faq.rope_append(gx[:, :Hq], gx[:, Hq:Hq + Hkv], gx[:, Hq + Hkv:], gc, gb, cs, None if pos is None else pos.cuda(),
                    interleaved=inter, amax=[a.cuda() for a in amax] if mode in ref.PER_HEAD else None, out=out)
    faq.check_device_status()
    p = seq if pos is None else pos[:T].long()
    q, k, v = x[:T, :Hq], x[:T, Hq:Hq + Hkv], x[:T, Hq + Hkv:]
    if rd:
        rows = cs.cpu()[p]
        q, k = ref.turn(q, rows, inter), ref.turn(k, rows, inter)
    assert torch.equal(out[:T].cpu().view(torch.int16), q.contiguous().view(torch.int16))
    assert (out[T:] == 7.0).all()
    # the oracle's codes and scales of the rotated rows
    t = 0
    for name, y, am in (("k", k, amax[0]), ("v", v, amax[1])):
        bits = wl.bf16_bits(y[None])  # [1, T, H, D]: BSND
        if mode in ref.PER_HEAD:
            codes, sc = getattr(orc, "quantize_" + mode)(bits, am.numpy(), "BSND")
            c[name + "s"] = torch.from_numpy(sc)
        else:
            codes, sc = getattr(orc, "quantize_" + mode)(bits, "BSND")
        codes = torch.from_numpy(codes)[0]
        t = 0
        for b, (n, m) in enumerate(zip(lens, qlens)):
            pg, o = ref.slots(c, table[b], torch.arange(n - m, n))
            if layout == "BNSD":
                c[name + "c"][pg, :, o] = codes[t:t + m]
            else:
                c[name + "c"][pg, o] = codes[t:t + m]
            if mode not in ref.PER_HEAD:
                c[name + "s"][pg, :, o] = torch.from_numpy(sc)[0, :, t:t + m].T
            t += m
    for n, g in (("kc", gc.k_codes), ("vc", gc.v_codes), ("ks", gc.k_scales), ("vs", gc.v_scales)):
        assert torch.equal(g.cpu(), c[n]), n  # the new rows, and every other slot as it was


def test_append_in_place_and_without_q(faq):
    lens, qlens = (40,), (40,)
    table, pages = ref.make_table(lens, 16, 0)
    c = ref.make_cache("int8_per_token", "BNSD", pages, 2, 16, 128, 1)
    x = bf16((40, 8, 128), 2)
    cs = faq.rope_table(64, 128)
    outs = []
    for how in ("out", "in place", "no q"):
        gc, gb, gx = to_gpu(faq, c), batch_of(faq, table, lens, qlens), x.cuda()
        q, k, v = gx[:, :4], gx[:, 4:6], gx[:, 6:]
        o = faq.rope_append(None if how == "no q" else q, k, v, gc, gb, cs, out=q if how == "in place" else None)
        faq.check_device_status()
        outs.append((None if o is None else o.clone(), gc.k_codes, gc.v_codes, gc.k_scales, gc.v_scales))
        assert torch.equal(gx[:, 4:].cpu(), x[:, 4:])
    assert torch.equal(outs[0][0], outs[1][0]) and outs[2][0] is None
    for a, b in zip(outs[0][1:], outs[1][1:]):
        assert torch.equal(a, b)
    for a, b in zip(outs[0][1:], outs[2][1:]):
        assert torch.equal(a, b)


def test_append_nan_and_infinity(faq):
    """A NaN in a row of a per-token mode: NaN scale, zero codes.  Infinities give an infinite scale."""
    for mode in ("int8_per_token", "fp8_per_token"):
        table, pages = ref.make_table((3,), 16, 0)
        gc = to_gpu(faq, ref.make_cache(mode, "BNSD", pages, 1, 16, 64, 1))
        x = bf16((3, 1, 64), 2)
        x[1, 0, 5], x[2, 0, 7] = float("nan"), float("inf")
        faq.rope_append(None, x.cuda(), x.cuda(), gc, batch_of(faq, table, (3,), (3,)))
        faq.check_device_status()
        pg = int(table[0, 0])
        for s, codes in ((gc.k_scales, gc.k_codes), (gc.v_scales, gc.v_codes)):
            s = s[pg, 0, :3].cpu()
            assert torch.isfinite(s[0]) and torch.isnan(s[1]) and torch.isinf(s[2])
            # finite / infinity: zeros of either sign (E4M3 has both)
            zero = codes[pg, 0, 2].cpu()[torch.arange(64) != 7] & (0x7F if mode.startswith("fp8") else -1)
            assert (codes[pg, 0, 1] == 0).all() and (zero == 0).all()


@pytest.mark.parametrize("scaling", [None, {"type": "linear", "factor": 4.0}, {"type": "ntk", "factor": 8.0},
                                     {"type": "yarn", "factor": 8.0, "original": 4096},
                                     {"type": "bands", "factor": 8.0, "original": 8192}])
def test_table(faq, scaling):
    n, rd = 131072, 64
    t = faq.rope_table(n, rd, 10000.0, scaling).cpu()
    f, m = faq.rope_frequencies(rd, 10000.0, scaling)
    ang = torch.arange(n, dtype=torch.float64)[:, None] * torch.tensor(f, dtype=torch.float64)[None]
    want = torch.cat((ang.cos(), ang.sin()), 1) * m
    # one rounding of a 64-bit value (itself a few 2^-53 off, times angles up to 2^17)
    assert ((t.double() - want).abs() <= want.abs() * 2.0 ** -24 + 2.0 ** -33).all()


def test_bad_device_data_is_reported_and_skipped(faq):
    """Pages, lengths, offsets and positions out of range: an error in the status word, other sequences'
    results as ever, nothing written outside."""
    lens, qlens = (100, 60, 30), (2, 2, 2)
    table, pages = ref.make_table(lens, 16, 1)
    c = ref.make_cache("int8_per_token", "BNSD", pages, 2, 16, 64, 2)
    q = bf16((6, 4, 64), 3)
    good, lse, tol, _ = ref.attend(q, c, table, lens, qlens, True)
    sc = torch.rand(3, 2, 112)

    def expect_bounds(fn, *a, **kw):
        r = fn(*a, **kw)
        with pytest.raises(faq.FaqError) as e:
            faq.check_device_status()
        assert e.value.status == 8
        faq.check_device_status()  # cleared
        return r

    for page in (-1, pages, 2 ** 31 - 1, -2 ** 31):
        bad = table.clone()
        bad[1, 2] = page
        gc, gb = to_gpu(faq, c), batch_of(faq, bad, lens, qlens)
        out = expect_bounds(faq.paged_attention, q.cuda(), gc, gb)
        keep = [0, 1, 4, 5]
        assert_within(out[keep], good[keep], tol[keep], "other sequences")
        expect_bounds(faq.paged_weights, q.cuda(), lse.float().cuda(), gc, gb, torch.zeros(3, 2, 112).cuda())
        expect_bounds(faq.paged_evict, gc, gb, sc.cuda(), 50)  # at least 6 of the bad page's 16 tokens stay
        bad = table.clone()
        bad[1, 3] = page
        gc = to_gpu(faq, c)
        expect_bounds(faq.rope_append, None, q[:, :2].contiguous().cuda(), q[:, 2:].contiguous().cuda(), gc,
                      batch_of(faq, bad, lens, qlens))
    for bad in ((100, -1, 30), (100, 16 * table.shape[1] + 1, 30), (100, 2 ** 31 - 1, 30)):
        gc, gb = to_gpu(faq, c), batch_of(faq, table, bad, qlens)
        out = expect_bounds(faq.paged_attention, q.cuda(), gc, gb)
        keep = [0, 1, 4, 5]
        assert_within(out[keep], good[keep], tol[keep], "other sequences")
        expect_bounds(faq.paged_weights, q.cuda(), lse.float().cuda(), gc, gb, torch.zeros(3, 2, 112).cuda())
        expect_bounds(faq.paged_evict, gc, gb, sc.cuda(), 10)
        expect_bounds(faq.rope_append, None, q[:, :2].contiguous().cuda(), q[:, 2:].contiguous().cuda(), gc, gb)
    gc = to_gpu(faq, c)
    # scores and accumulators shorter than a sequence
    expect_bounds(faq.paged_weights, q.cuda(), lse.float().cuda(), gc, batch_of(faq, table, lens, qlens),
                  torch.zeros(3, 2, 99).cuda())
    expect_bounds(faq.paged_evict, gc, batch_of(faq, table, lens), torch.rand(3, 2, 99).cuda(), 10)
    # offsets: past the rows, falling, or more than max_q tokens
    for cu in ((0, 2, 4, 7), (0, 5, 4, 6), (-1, 2, 4, 6)):
        gb = faq.PagedBatch(table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(),
                            torch.tensor(cu, dtype=torch.int32).cuda())
        expect_bounds(faq.paged_attention, q.cuda(), gc, gb)
    expect_bounds(faq.paged_attention, q.cuda(), gc, batch_of(faq, table, lens, qlens, 1))
    # positions outside the table, and more new tokens than cached ones
    k = q[:, :2].contiguous().cuda()
    for p in (-1, 50, 2 ** 31 - 1):
        pos = torch.tensor([3, 4, p, 5, 6, 7], dtype=torch.int32).cuda()
        expect_bounds(faq.rope_append, None, k, k, gc, batch_of(faq, table, lens, qlens), faq.rope_table(50, 64), pos)
    expect_bounds(faq.rope_append, None, k, k, gc, batch_of(faq, table, (100, 1, 30), qlens))


def test_graph_replay_with_other_lengths_and_a_second_stream(faq):
    """A captured step follows the lengths, pages and rows in its buffers; two graphs with their own
    workspaces on two streams do not disturb each other."""
    caches, state = [], []
    for k in range(2):
        lens = (400, 300 + 100 * k)
        table, pages = ref.make_table((600, 600), 16, k)
        c = ref.make_cache("fp8_per_token", "BNSD", pages, 2, 16, 128, 20 + k)
        caches.append(c)
        gb = batch_of(faq, table, lens)
        q = torch.zeros(2, 8, 128, dtype=torch.bfloat16).cuda()
        kv = torch.zeros(2, 2, 128, dtype=torch.bfloat16).cuda()
        gc = to_gpu(faq, c)
        ws = torch.empty(faq.paged_attention_workspace_size(q, gc, gb), dtype=torch.uint8).cuda()
        out, lse, rot = torch.empty_like(q), torch.empty(2, 8).cuda(), torch.empty_like(q)
        acc = torch.zeros(2, 2, 600).cuda()
        cs = faq.rope_table(700, 128)
        stream = torch.cuda.Stream()

        def step(gc=gc, gb=gb, q=q, kv=kv, ws=ws, out=out, lse=lse, rot=rot, acc=acc, cs=cs):
            faq.rope_append(q, kv, kv, gc, gb, cs, out=rot)
            faq.paged_attention(rot, gc, gb, out=out, lse=lse, workspace=ws)
            faq.paged_weights(rot, lse, gc, gb, acc, accumulate=False)

        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            step()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=stream):
                step()
        state.append((table, gb, gc, q, kv, rot, out, lse, acc, cs, stream, graph))
    torch.cuda.synchronize()
    faq.check_device_status()
    for turn, lens in enumerate([(1, 600), (599, 17)]):
        for k, (table, gb, gc, q, kv, rot, out, lse, acc, cs, stream, graph) in enumerate(state):
            gc.k_codes.copy_(caches[k]["kc"])
            gc.v_codes.copy_(caches[k]["vc"])
            gc.k_scales.copy_(caches[k]["ks"])
            gc.v_scales.copy_(caches[k]["vs"])
            gb.seq_lens.copy_(torch.tensor(lens, dtype=torch.int32))
            q.copy_(bf16((2, 8, 128), 100 * turn + k))
            kv.copy_(bf16((2, 2, 128), 100 * turn + k + 50))
            acc.zero_()
        torch.cuda.synchronize()
        for s in state:
            with torch.cuda.stream(s[-2]):
                s[-1].replay()
        torch.cuda.synchronize()
        faq.check_device_status()
        for k, (table, gb, gc, q, kv, rot, out, lse, acc, cs, stream, graph) in enumerate(state):
            now = dict(caches[k], kc=gc.k_codes.cpu(), vc=gc.v_codes.cpu(), ks=gc.k_scales.cpu(), vs=gc.v_scales.cpu())
            p = torch.tensor(lens) - 1
            assert torch.equal(rot.cpu(), ref.turn(q.cpu(), cs.cpu()[p], False))
            want, z, tol, ltol = ref.attend(rot.cpu(), now, table, lens, (1, 1), True)
            assert_within(out, want, tol, "out")
            assert_within(lse, z, ltol, "lse")
            w, wtol = ref.weigh(rot.cpu(), lse.cpu(), now, table, lens, (1, 1), True, 600)
            assert_within(acc, w, wtol, "weights")


@pytest.mark.parametrize("mode", ref.MODES)
def test_serving_run(faq, orc, mode):
    """Prompt in two chunks, weights, eviction, then single tokens behind the kept ones: each step's
    output against the 64-bit form on the cache as the operators left it, and the codes against the
    oracle's."""
    H, Hq, D, page = 2, 6, 64, 16
    prompt, budget = (150, 61), 48
    table, pages = ref.make_table((160, 160), page, 4)
    c = ref.make_cache(mode, "BNSD", pages, H, page, D, 5)
    gc = to_gpu(faq, c)
    cs = faq.rope_table(256, 32)
    amax = [torch.full((H,), 4.0).cuda()] * 2 if mode in ref.PER_HEAD else None
    acc = torch.zeros(2, H, 160).cuda()
    lens, true = [0, 0], [0, 0]

    def step(qlens, seed, evict_after=False):
        T = sum(qlens)
        x = bf16((T, Hq + 2 * H, D), seed).cuda()
        for b in range(2):
            lens[b] += qlens[b]
            true[b] += qlens[b]
        pos = torch.cat([torch.arange(true[b] - qlens[b], true[b]) for b in range(2)]).to(torch.int32)
        gb = batch_of(faq, table, lens, qlens, max(qlens))
        before = [t.clone() for t in (gc.k_codes, gc.v_codes)]
        q = faq.rope_append(x[:, :Hq], x[:, Hq:Hq + H], x[:, Hq + H:], gc, gb, cs, pos.cuda(), amax=amax)
        out, lse = faq.paged_attention(q, gc, gb, return_lse=True)
        faq.paged_weights(q, lse, gc, gb, acc)
        faq.check_device_status()
        assert torch.equal(q.cpu(), ref.turn(x[:, :Hq].cpu(), cs.cpu()[pos.long()], False))
        now = dict(c, kc=gc.k_codes.cpu(), vc=gc.v_codes.cpu(), ks=gc.k_scales.cpu(), vs=gc.v_scales.cpu())
        changed = (before[0] != gc.k_codes).any(-1).sum() if mode != "x" else 0
        assert changed <= T * H  # only the new tokens' slots
        want, z, tol, ltol = ref.attend(q.cpu(), now, table, lens, qlens, True)
        assert_within(out, want, tol, "out")
        assert_within(lse, z, ltol, "lse")
        return gb, now

    step((100, 61), 1)
    gb, now = step((50, 0), 2)
    kept, new, so = ref.evict(now, table, lens, acc.cpu(), budget, 2, 8)
    acc2 = torch.empty_like(acc)
    gk, gn = faq.paged_evict(gc, gb, acc, budget, 2, 8, scores_out=acc2)
    faq.check_device_status()
    assert torch.equal(gk.cpu(), kept) and torch.equal(gn.cpu(), new) and torch.equal(acc2.cpu(), so)
    assert torch.equal(gc.k_codes.cpu(), now["kc"]) and torch.equal(gc.v_codes.cpu(), now["vc"])
    acc.copy_(acc2)
    lens[:] = gn.tolist()
    for k in range(4):
        step((1, 1), 10 + k)


def test_tensors_of_another_kind_are_refused(faq):
    c = faq.empty_paged_cache(4, 2, 16, 64, "int8_per_token")
    b = faq.PagedBatch(torch.zeros(1, 2, dtype=torch.int32).cuda(), torch.ones(1, dtype=torch.int32).cuda())
    q = torch.zeros(1, 4, 64, dtype=torch.bfloat16).cuda()
    for bad in (q.float(), q.cpu(), q[0], q.transpose(1, 2).contiguous().transpose(1, 2)):
        with pytest.raises(ValueError):
            faq.paged_attention(bad, c, b)
    with pytest.raises(ValueError):
        faq.paged_attention(q, c, b, out=torch.zeros(1, 4, 32, dtype=torch.bfloat16).cuda())
    with pytest.raises(ValueError):
        faq.paged_weights(q, torch.zeros(1, 3).cuda(), c, b, torch.zeros(1, 2, 32).cuda())
    with pytest.raises(ValueError):
        faq.paged_weights(q, torch.zeros(1, 4).cuda(), c, b, torch.zeros(1, 3, 32).cuda())
    with pytest.raises(ValueError):
        faq.paged_evict(c, b, torch.zeros(1, 2, 32).cuda(), 0)
    with pytest.raises(ValueError):
        faq.PagedBatch(torch.zeros(1, 2, dtype=torch.int64).cuda(), torch.ones(1, dtype=torch.int32).cuda())
    with pytest.raises(faq.FaqError) as e:
        faq.paged_evict(c, b, torch.zeros(1, 2, 32).cuda(), 4, 3, 2)
    assert e.value.status == 1
    with pytest.raises(faq.FaqError) as e:
        need = faq.paged_attention_workspace_size(q, c, b)
        faq.paged_attention(q, c, b, workspace=torch.empty(need + 1, dtype=torch.uint8).cuda()[1:])
    assert e.value.status == 7


def test_weights_of_no_new_token_are_zero(faq):
    """A call whose batch holds no new token at all still sets the weights when it does not accumulate."""
    for mode in ("int8_per_head", "fp8_per_token"):
        table, pages = ref.make_table((40, 0, 129), 16, 5)
        c = ref.make_cache(mode, "BNSD", pages, 2, 16, 64, 3)
        gc = to_gpu(faq, c)
        gb = faq.PagedBatch(table.cuda(), torch.tensor((40, 0, 129), dtype=torch.int32).cuda(),
                            torch.zeros(4, dtype=torch.int32).cuda())
        q, lse = torch.zeros(0, 4, 64, dtype=torch.bfloat16).cuda(), torch.zeros(0, 4).cuda()
        for add in (True, False):
            acc = torch.full((3, 2, 140), 5.0).cuda()
            faq.paged_weights(q, lse, gc, gb, acc, accumulate=add)
            faq.check_device_status()
            want = torch.full((3, 2, 140), 5.0)
            if not add:
                want[0, :, :40], want[2, :, :129] = 0.0, 0.0
            assert torch.equal(acc.cpu(), want)


def test_empty_scores_of_empty_sequences(faq):
    c = faq.empty_paged_cache(4, 2, 16, 64, "int8_per_token")
    b = faq.PagedBatch(torch.zeros(3, 0, dtype=torch.int32).cuda(), torch.zeros(3, dtype=torch.int32).cuda())
    none = torch.zeros(3, 2, 0).cuda()
    kept, new = faq.paged_evict(c, b, none, 4, scores_out=torch.zeros_like(none))
    q, lse = torch.zeros(3, 4, 64, dtype=torch.bfloat16).cuda(), torch.zeros(3, 4).cuda()
    out, z = faq.paged_attention(q, c, b, return_lse=True)
    faq.paged_weights(q, z, c, b, none, accumulate=False)
    faq.check_device_status()
    assert (kept == -1).all() and (new == 0).all()
    assert (out == 0).all() and torch.isneginf(z).all()


def test_descriptors_stay_with_their_tensors_and_device(faq, monkeypatch):
    import dataclasses

    import quantized_attention_amax_b200.paged as paged
    c = faq.empty_paged_cache(4, 2, 16, 64, "int8_per_token")
    b = faq.PagedBatch(torch.zeros(1, 2, dtype=torch.int32).cuda(), torch.ones(1, dtype=torch.int32).cuda())
    q = torch.zeros(1, 4, 64, dtype=torch.bfloat16).cuda()
    with pytest.raises(dataclasses.FrozenInstanceError):
        b.seq_lens = torch.zeros(1, dtype=torch.int32).cuda()
    with pytest.raises(dataclasses.FrozenInstanceError):
        c.k_codes = c.v_codes
    need = faq.paged_attention_workspace_size(q, c, b)
    with pytest.raises(ValueError):
        faq.paged_attention(q, c, b, workspace=torch.empty(need, dtype=torch.uint8))
    with pytest.raises(ValueError):
        faq.paged_attention(q, c, b, workspace=torch.empty(2 * need, dtype=torch.uint8).cuda()[::2])
    scores = torch.zeros(1, 2, 32).cuda()
    for kw in (dict(budget=2 ** 32 + 4), dict(budget=2 ** 30 + 1), dict(budget=8, sink=2 ** 32), dict(budget=8, recent=2 ** 32)):
        with pytest.raises(ValueError):
            faq.paged_evict(c, b, scores, **kw)
    with pytest.raises(ValueError):
        faq.PagedBatch(b.page_table, b.seq_lens, None, 2 ** 32)
    # with another device current, no call takes them (the check comes before any launch)
    there = torch.cuda.current_device() + 1
    monkeypatch.setattr(paged, "_current_device", lambda: there)
    for use in (c.c, b.c):
        with pytest.raises(ValueError):
            use()


@pytest.mark.parametrize("mode", ["fp8_per_head", "int8_per_token"])
def test_chunk_attention_repeats_bit_for_bit(faq, mode):
    """Many blocks of few key tiles, whose conversion runs ahead of the products: each of 40 calls gives the same
    bits.  V's element d is 1 for the tokens of the d-th 16, so that with equal weights (q = 0) a row's element d is the
    share of them that it sees: a tile read late would show as a share that is off."""
    n, H, D, page = 1500, 8, 128, 64
    lens, qlens = (n, 1200), (n, 1100)
    table, pages = ref.make_table(lens, page, 2)
    c = ref.make_cache(mode, "BNSD", pages, H, page, D, 4, spread=0.5)
    for x in ("kc", "vc"):
        c[x].zero_()
        for b, m in enumerate(lens):
            for j in range(m):
                c[x][int(table[b, j // page]), :, j % page, j // 16] = 0x38 if mode.startswith("fp8") else 1
    c["ks"].fill_(1.0), c["vs"].fill_(1.0)
    gc, gb = to_gpu(faq, c), batch_of(faq, table, lens, qlens)
    q = torch.zeros(sum(qlens), 4 * H, D, dtype=torch.bfloat16).cuda()
    first, lse = faq.paged_attention(q, gc, gb, return_lse=True)
    i = torch.cat([torch.arange(b - a, b) + 1 for a, b in zip(qlens, lens)]).double()  # keys a row sees
    d = torch.arange(D).double() * 16
    want = ((i[:, None] - d).clamp(0, 16) / i[:, None])[:, None].expand(-1, 4 * H, D)
    # fp16 shares are 2^7 exactly and sums of them exact in fp32: what rounds is the quotient, and bf16
    assert_within(first, want, want * (2.0 ** -8 + 2.0 ** -21), "shares")
    for _ in range(40):
        out, z = faq.paged_attention(q, gc, gb, return_lse=True)
        assert torch.equal(out.view(torch.int16), first.view(torch.int16)) and torch.equal(z, lse)
    faq.check_device_status()


def test_chunks_over_empty_sequences(faq):
    """Blocks that see no key at all, many in a row, among blocks that do: zeros and -inf, and the others right."""
    lens, qlens = (0, 0, 0, 300, 0, 0, 0, 0, 0, 0, 20, 0), (40, 300, 33, 200, 64, 17, 90, 40, 129, 300, 20, 70)
    table, pages = ref.make_table(lens, 16, 9)
    c = ref.make_cache("int8_per_token", "BNSD", pages, 2, 16, 128, 21, spread=0.5)
    q = bf16((sum(qlens), 4, 128), 22, 1.5)
    for causal in (False, True):
        want, lse, tol, ltol = ref.attend(q, c, table, lens, qlens, causal)
        out, z = faq.paged_attention(q.cuda(), to_gpu(faq, c), batch_of(faq, table, lens, qlens), causal=causal, return_lse=True)
        faq.check_device_status()
        assert_within(out, want, tol, "out")
        assert_within(z, lse, ltol, "lse")
