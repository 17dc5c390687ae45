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
