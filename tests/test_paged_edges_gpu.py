"""GPU tests of the paged-cache operators at their edges: values that are no numbers, histories cut between
CTAs, and weights far below a row's largest, against the 64-bit forms of tests/_paged_ref.py."""
import math

import pytest
import torch

import _paged_ref as ref
from _gpu import faq_module
from test_paged_gpu import assert_within, batch_of, bf16, to_gpu

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def faq():
    return faq_module()


def slot(table, page, j, b=0):
    return int(table[b, j // page]), j % page


def put(c, name, pg, h, o, value):
    """Codes of one row (an int for all of them, or (dim, code))."""
    x = c[name + "c"]
    row = x[pg, h, o] if c["layout"] == "BNSD" else x[pg, o, h]
    if isinstance(value, tuple):
        row[value[0]] = value[1]
    else:
        row.fill_(value)


def attend(faq, q, c, table, lens, qlens, causal=True, **kw):
    out, lse = faq.paged_attention(q.cuda(), to_gpu(faq, c), batch_of(faq, table, lens, qlens), causal=causal,
                                   return_lse=True, **kw)
    faq.check_device_status()
    return out.cpu(), lse.cpu()


def expect_rows(got, want, nan_rows):
    """(out, lse) within the bounds outside nan_rows [T, Hq], NaN in them."""
    (out, lse), (o, z, tol, ltol) = got, want
    assert torch.isnan(out[nan_rows]).all() and torch.isnan(lse[nan_rows]).all()
    assert_within(out[~nan_rows], o[~nan_rows], tol[~nan_rows], "out")
    assert_within(lse[~nan_rows], z[~nan_rows], ltol[~nan_rows], "lse")


# one query row and several for the kernel of few rows, then blocks of up to 128 rows and of more
ROWS = [1, 3, 20, 70]


@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("mode", ["fp8_per_head", "int8_per_token", "fp8_per_token"])  # (an int8 code is never NaN)
@pytest.mark.parametrize("n", [129, 385])
def test_a_nan_key_alone_in_its_tile(faq, rows, mode, n):
    """The last token's K is NaN (its scale, or an E4M3 code) and stands alone in the last tile, which a CTA of its own
    takes: the row that sees it is NaN, output and LSE, although that piece has no score that is a number."""
    lens, qlens = (n,), (rows,)
    table, pages = ref.make_table(lens, 16, 2)
    c = ref.make_cache(mode, "BNSD", pages, 1, 16, 128, 3, spread=0.5)
    q = bf16((rows, 2, 128), 4)
    want = ref.attend(q, c, table, lens, qlens, True)
    pg, o = slot(table, 16, n - 1)
    if mode in ref.PER_HEAD:
        put(c, "k", pg, 0, o, (7, 0x7F))
    else:
        c["ks"][pg, 0, o] = NAN
    bad = torch.zeros(rows, 2, dtype=torch.bool)
    bad[-1] = True
    expect_rows(attend(faq, q, c, table, lens, qlens), want, bad)


@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("mode", ref.MODES)
@pytest.mark.parametrize("value", [NAN, INF])
def test_a_query_that_is_no_number_over_a_cut_history(faq, rows, mode, value):
    """One head's query of one token holds a NaN or an infinity: its row is NaN, over one tile and over many pieces."""
    for n in (100, 5000):
        lens, qlens = (n,), (rows,)
        table, pages = ref.make_table(lens, 64, 2)
        c = ref.make_cache(mode, "BNSD", pages, 2, 64, 64, 3, spread=0.5)
        q = bf16((rows, 4, 64), 4)
        want = ref.attend(q, c, table, lens, qlens, True)
        q[rows // 2, 1, 9] = value
        bad = torch.zeros(rows, 4, dtype=torch.bool)
        bad[rows // 2, 1] = True
        expect_rows(attend(faq, q, c, table, lens, qlens), want, bad)


@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("mode", ref.PER_HEAD)
def test_a_nan_head_scale_over_a_cut_history(faq, rows, mode):
    n = 5000
    lens, qlens = (n,), (rows,)
    table, pages = ref.make_table(lens, 64, 2)
    c = ref.make_cache(mode, "BSND", pages, 2, 64, 128, 3, spread=0.5)
    q = bf16((rows, 4, 128), 4)
    want = ref.attend(q, c, table, lens, qlens, True)
    c["ks"][1] = NAN
    bad = torch.zeros(rows, 4, dtype=torch.bool)
    bad[:, 2:] = True
    expect_rows(attend(faq, q, c, table, lens, qlens), want, bad)


@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("mode", ["fp8_per_head", "fp8_per_token"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n", [300, 5000])
def test_a_nan_value_code_reaches_its_element(faq, rows, mode, D, n):
    """A NaN E4M3 code of V makes that element of the rows that see its token NaN, wherever the token lies: in a tile
    that every row sees whole, or in one that some do not.  The rows' other elements, their LSE and the other rows
    are as without it."""
    lens, qlens = (n, 40), (rows, 1)
    table, pages = ref.make_table(lens, 16, 2)
    c = ref.make_cache(mode, "BNSD", pages, 1, 16, D, 3, spread=0.5)
    q = bf16((rows + 1, 2, D), 4)
    out, lse, tol, ltol = ref.attend(q, c, table, lens, qlens, True)
    nan = torch.zeros(rows + 1, 2, D, dtype=torch.bool)
    i = torch.arange(rows)
    for j, d in ((5, 3), (n - 1, 0), (n - 1, 40), (n - rows, D - 1), (n - 1 - rows // 2, 17), (n - 1, 17), (n // 2, 33)):
        pg, o = slot(table, 16, j)
        put(c, "v", pg, 0, o, (d, 0x7F if j & 1 else 0xFF))
        nan[:rows, :, d] |= (n - rows + i >= j)[:, None]
    pg, o = slot(table, 16, 39, 1)
    put(c, "v", pg, 0, o, (11, 0x7F))
    nan[rows, :, 11] = True
    got, z = attend(faq, q, c, table, lens, qlens)
    assert torch.equal(torch.isnan(got), nan)
    assert_within(got[~nan], out[~nan], tol[~nan], "out")
    assert_within(z, lse, ltol, "lse")


@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("mode", ["int8_per_token", "fp8_per_token"])
@pytest.mark.parametrize("value", [NAN, INF])
@pytest.mark.parametrize("n", [129, 2000])
def test_a_value_scale_that_is_no_number(faq, rows, mode, value, n):
    """The rows that see the token are NaN; their LSE, which V has no part in, is as without it."""
    for j in (n - 1, n - 1 - rows // 2, 3):
        lens, qlens = (n, 20), (rows, 2)
        table, pages = ref.make_table(lens, 16, 2)
        c = ref.make_cache(mode, "BSND", pages, 1, 16, 128, 3, spread=0.5)
        q = bf16((rows + 2, 2, 128), 4)
        out, lse, tol, ltol = ref.attend(q, c, table, lens, qlens, True)
        pg, o = slot(table, 16, j)
        c["vs"][pg, 0, o] = value
        nan = torch.zeros(rows + 2, 2, dtype=torch.bool)
        nan[:rows] = (n - rows + torch.arange(rows) >= j)[:, None]
        got, z = attend(faq, q, c, table, lens, qlens)
        assert torch.isnan(got[nan]).all()
        assert_within(got[~nan], out[~nan], tol[~nan], "out")
        assert_within(z, lse, ltol, "lse")


@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("mode", ref.MODES)
@pytest.mark.parametrize("value", [NAN, INF])
def test_scales_of_a_head_that_are_no_numbers(faq, rows, mode, value):
    """K scales: the rows that see such a token are NaN, output and LSE, whatever its scores' signs.  V scales: the output.
    Rows that see no key stay zero and -inf."""
    lens, qlens = (2000, 1, 0), (rows, rows + 2, rows)
    table, pages = ref.make_table(lens, 16, 2)
    T = sum(qlens)
    q = bf16((T, 4, 64), 4)
    q[:, 2:] = q[:, 2:].abs()
    see = torch.zeros(T, 4, dtype=torch.bool)
    see[:rows] = True
    see[2 * rows + 1] = True  # the second sequence's one token is seen by its last row
    for which in ("ks", "vs"):
        c = ref.make_cache(mode, "BNSD", pages, 2, 16, 64, 3, spread=0.5)
        if which == "ks":  # every score of head 1's rows below zero
            k = c["kc"][:, 1]
            c["kc"][:, 1] = k | 0x80 if mode.startswith("fp8") else -(k.abs().clamp(1, 127))
        out, lse, tol, ltol = ref.attend(q, c, table, lens, qlens, True)
        if mode in ref.PER_HEAD:
            c[which][1] = value
        else:
            c[which][:, 1] = value
        got, z = attend(faq, q, c, table, lens, qlens)
        hit = see.clone()
        hit[:, :2] = False
        assert torch.isnan(got[hit]).all()
        assert_within(got[~hit], out[~hit], tol[~hit], "out")
        if which == "ks":
            assert torch.isnan(z[hit]).all()
            assert_within(z[~hit], lse[~hit], ltol[~hit], "lse")
        else:
            assert_within(z, lse, ltol, "lse")


def sink_and_tail(mode, n, D):
    """One sequence of n tokens: the first one's scores lie 17.5 (natural) above the others', which are equal; its V is zero,
    theirs lie in [1, 1.98].  (cache, table, softmax scale for queries of ones)"""
    page = 128
    table, pages = ref.make_table((n,), page, 1)
    c = ref.make_cache(mode, "BNSD", pages, 1, page, D, 2)
    c["kc"].zero_()
    v = torch.randint(50, 100, c["vc"].shape, generator=torch.Generator().manual_seed(3))
    c["vc"] = ref.e4m3(v.float()) if mode.startswith("fp8") else v.to(torch.int8)
    c["ks"].fill_(0.01), c["vs"].fill_(0.02)
    pg, o = slot(table, page, 0)
    put(c, "k", pg, 0, o, int(ref.e4m3(torch.tensor(64.0))) if mode.startswith("fp8") else 64)
    put(c, "v", pg, 0, o, 0)
    return c, table, 17.5 / (D * 64 * 0.01)


@pytest.mark.parametrize("group", [1, 8, 16])
@pytest.mark.parametrize("mode", ref.MODES)
@pytest.mark.parametrize("D", [64, 128])
def test_a_flat_tail_under_one_large_weight(faq, group, mode, D):
    """The first token takes nearly all of the weight and has a zero V; the others, each 2^-25 of it, are all of the output.
    Many sequences read the same pages, so that a CTA's run of keys is long."""
    n, B = 16384, 300
    c, table1, scale = sink_and_tail(mode, n, D)
    q = torch.ones(B, group, D, dtype=torch.bfloat16)
    table, lens = table1.expand(B, -1).contiguous(), (n,) * B
    want, lse, _, ltol = ref.attend(q[:1], c, table1, (n,), (1,), True, scale)
    out, z = attend(faq, q, c, table, lens, (1,) * B, softmax_scale=scale)
    # The tokens of the first token's tile (127) are held against it: each is off by at most 2^-24 of the largest weight
    # (1 to nine digits), times its value (at most 104 * 0.02: 99 as E4M3).  The others are held against their own
    # tile's largest: 2^-11 of each (and the scores' roundings, below 2^-18), and bf16's half step 2^-8.
    tol = want.abs() * (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -18) + 127 * 2.0 ** -24 * 104 * 0.02
    assert (tol < 0.05 * want.abs()).all()  # the bound says something
    assert_within(out, want.expand(B, -1, -1), tol.expand(B, -1, -1), "out")
    assert_within(z, lse.expand(B, -1), ltol.expand(B, -1), "lse")


@pytest.mark.parametrize("rows", [20, 200])
@pytest.mark.parametrize("mode", ref.MODES)
def test_a_flat_tail_under_one_large_weight_of_a_chunk(faq, rows, mode):
    """As above for more rows: weights are fp16 of 2^7 of the row's largest, whose steps end at 2^-24: each is off by at most
    2^-32 of the largest."""
    n, D = 16384, 128
    c, table, scale = sink_and_tail(mode, n, D)
    q = torch.ones(rows, 2, D, dtype=torch.bfloat16)
    want, lse, _, ltol = ref.attend(q[:1], c, table, (n,), (1,), False, scale)
    out, z = attend(faq, q, c, table, (n,), (rows,), causal=False, softmax_scale=scale)
    tol = want.abs() * (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -18) + n * 2.0 ** -32 * 104 * 0.02
    assert (tol < 0.05 * want.abs()).all()
    assert_within(out, want.expand(rows, -1, -1), tol.expand(rows, -1, -1), "out")
    assert_within(z, lse.expand(rows, -1), ltol.expand(rows, -1), "lse")


@pytest.mark.parametrize("rows", [1, 3])
@pytest.mark.parametrize("mode", ref.MODES)
def test_tiles_far_apart(faq, rows, mode):
    """Keys' scores that step up and down by hundreds from tile to tile: a tile far below the largest adds nothing and
    disturbs nothing, in either order."""
    n, page, D, B = 8192, 128, 64, 40
    for kind in ("up", "down", "saw"):
        table1, pages = ref.make_table((n,), page, 1)
        c = ref.make_cache(mode, "BNSD", pages, 1, page, D, 5)
        c["kc"].zero_()
        c["ks"].fill_(1.0)
        tiles = n // page
        level = {"up": list(range(tiles)), "down": list(range(tiles))[::-1], "saw": [(t * 37) % tiles for t in range(tiles)]}[kind]
        for t, x in enumerate(level):
            put_code = int(ref.e4m3(torch.tensor(float(x)))) if mode.startswith("fp8") else x
            pgs = int(table1[0, t])
            c["kc"][pgs, 0, :, 0] = put_code
        q = torch.zeros(B * rows, 2, D, dtype=torch.bfloat16)
        q[..., 0] = 1.0
        table = table1.expand(B, -1).contiguous()
        want, lse, tol, ltol = ref.attend(q[:rows], c, table1, (n,), (rows,), True, 100.0)
        out, z = attend(faq, q, c, table, (n,) * B, (rows,) * B, softmax_scale=100.0)
        assert_within(out, want.repeat(B, 1, 1), tol.repeat(B, 1, 1), kind)
        assert_within(z, lse.repeat(B, 1), ltol.repeat(B, 1), kind)


@pytest.mark.parametrize("qlen,Hq", [(1, 1), (1, 3), (2, 8), (30, 8)])
@pytest.mark.parametrize("mode", ref.MODES)
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("out_by", [-INF, NAN, INF])
def test_rows_without_a_finite_lse_give_nothing(faq, qlen, Hq, mode, causal, out_by):
    """A row that the caller takes out by its LSE, or whose attention was NaN, adds nothing to any key, also where its query
    or a key is no number, in tiles that every row sees whole too.  The other rows' weights are as ever."""
    n = 700
    lens, qlens = (n,), (qlen,)
    table, pages = ref.make_table(lens, 32, 2)
    c = ref.make_cache(mode, "BNSD", pages, 1, 32, 128, 3, spread=0.5)
    q = bf16((qlen, Hq, 128), 4)
    _, lse, _, _ = ref.attend(q, c, table, lens, qlens, causal)
    lse = lse.float()
    off = torch.zeros(qlen, Hq, dtype=torch.bool)
    off[qlen // 2, Hq // 2] = True
    ref_lse = torch.where(off, -INF, lse)
    w, tol = ref.weigh(q, ref_lse, c, table, lens, qlens, causal, n)
    lse[off] = out_by
    for value in (1.0, NAN, INF):
        bad_q = q.clone()
        bad_q[off] = bad_q[off] * value
        acc = torch.full((1, 1, n), 3.0).cuda()
        faq.paged_weights(bad_q.cuda(), lse.cuda(), to_gpu(faq, c), batch_of(faq, table, lens, qlens), acc, causal=causal)
        faq.check_device_status()
        assert_within(acc, w + 3.0, tol + (w + 3.0) * 2.0 ** -24, "weights")
    # every row taken out, a key whose K is NaN: nothing is added anywhere
    pg, o = slot(table, 32, 40)
    if mode.startswith("fp8"):
        put(c, "k", pg, 0, o, (3, 0x7F))
    elif mode not in ref.PER_HEAD:
        c["ks"][pg, 0, o] = NAN
    else:
        c["ks"][0] = INF
    acc = torch.full((1, 1, n), 3.0).cuda()
    faq.paged_weights(q.cuda(), torch.full_like(lse, out_by).cuda(), to_gpu(faq, c), batch_of(faq, table, lens, qlens), acc,
                      causal=causal)
    faq.check_device_status()
    assert (acc == 3.0).all()


def test_an_append_with_offsets_that_fall(faq):
    """Offsets that fall, and a bad length of a sequence without new tokens: reported by the append too, although no row leads
    to those sequences, and the rows of the others are theirs."""
    table, pages = ref.make_table((100, 60, 30), 16, 1)
    k = bf16((6, 2, 64), 3).cuda()
    for cu, lens in (((0, 2, 1, 1), (100, 60, 30)), ((0, 2, 2, 4), (100, -5, 30)), ((0, 2, 2, 4), (100, 2 ** 30, 30))):
        c = ref.make_cache("int8_per_token", "BNSD", pages, 2, 16, 64, 2)
        gc, want = to_gpu(faq, c), to_gpu(faq, c)
        gb = faq.PagedBatch(table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), torch.tensor(cu, dtype=torch.int32).cuda())
        faq.rope_append(None, k, k, gc, gb)
        with pytest.raises(faq.FaqError) as e:
            faq.check_device_status()
        assert e.value.status == 8
        fine = (0, 2, 2, 2 + max(0, cu[3] - cu[2]))
        faq.rope_append(None, k, k, want, batch_of(faq, table, (100, 60, 30), [fine[i + 1] - fine[i] for i in range(3)]))
        faq.check_device_status()
        for a, b in ((gc.k_codes, want.k_codes), (gc.v_codes, want.v_codes), (gc.k_scales, want.k_scales), (gc.v_scales, want.v_scales)):
            assert torch.equal(a, b)
