"""Paged-cache entry points on the host (no GPU): refusals before any launch, workspace sizes, and the
rotation frequencies' scaling rules."""
import ctypes
import math

import pytest

by = ctypes.byref
OK, INVALID, UNSUPPORTED, NO_CALIBRATION, WORKSPACE = 0, 1, 2, 3, 7


@pytest.fixture(scope="module")
def N():
    from quantized_attention_amax_b200 import build
    build.build()
    from quantized_attention_amax_b200 import _native
    _native.lib()
    return _native


def cache(N, mode=1, pages=4, H=2, page=64, D=128, layout=0, k=0x10000, v=0x20000, ks=0x30000, vs=0x40000):
    return N.FaPagedCache(k, v, ks, vs, mode, pages, H, page, D, layout)


def batch(N, B=2, wide=2, cu=0x50000, table=0x60000, lens=0x70000, max_q=0):
    return N.FaPagedBatch(table, lens, cu, B, wide, max_q)


def rows(N, T=5, H=4, D=128, stride=None, data=0x80000):
    return N.FaRows(data, T, H, D, H * D if stride is None else stride)


BAD_CACHES = [(dict(mode=0), UNSUPPORTED), (dict(mode=3), UNSUPPORTED), (dict(mode=4), UNSUPPORTED),
              (dict(mode=7), UNSUPPORTED), (dict(mode=9), UNSUPPORTED), (dict(H=0), INVALID), (dict(pages=0), INVALID), (dict(pages=-1), INVALID),
              (dict(D=96), UNSUPPORTED), (dict(page=8), UNSUPPORTED), (dict(page=48), UNSUPPORTED),
              (dict(page=2048), UNSUPPORTED), (dict(layout=2), INVALID), (dict(k=0x10008), INVALID),
              (dict(v=None), INVALID), (dict(ks=None), INVALID), (dict(vs=0x40002), INVALID),
              (dict(H=1 << 20, page=1024), UNSUPPORTED)]
BAD_BATCHES = [(dict(B=-1), INVALID), (dict(wide=-1), INVALID), (dict(max_q=-1), INVALID), (dict(table=None), INVALID),
               (dict(lens=None), INVALID), (dict(lens=0x70002), INVALID), (dict(cu=0x50001), INVALID),
               (dict(cu=None), INVALID),  # T != B
               (dict(wide=1 << 28), UNSUPPORTED)]
BAD_ROWS = [(dict(T=-1), INVALID), (dict(H=0), INVALID), (dict(D=64), INVALID), (dict(stride=8), INVALID),
            (dict(stride=517), INVALID), (dict(data=None), INVALID), (dict(data=0x80008), INVALID)]


@pytest.mark.parametrize("bad,st", BAD_CACHES)
def test_bad_caches(N, bad, st):
    L, c, b, q = N.lib(), cache(N, **bad), batch(N), rows(N, H=4 if bad.get("H", 2) == 2 else max(1, bad["H"]))
    kv = rows(N, H=max(1, c.H))
    assert L.fa_paged_attention(by(q), by(c), by(b), 1, 0.0, 0x90000, None, 0xA0000, 1 << 40, None) == st
    assert L.fa_paged_weights(by(q), 0x90000, by(c), by(b), 1, 0.0, 0xA0000, 128, 1, None) == st
    assert L.fa_rope_append(None, by(kv), by(kv), by(c), by(b), None, 0, 0, None, 0, 0x90000, 0x90000, None, None) == st
    assert L.fa_paged_evict(by(c), by(b), 0x90000, 128, 8, 0, 0, 0xA0000, 0xB0000, None, None) == st
    assert L.fa_paged_attention_workspace_size(by(q), by(c), by(b)) == 0


@pytest.mark.parametrize("bad,st", BAD_BATCHES)
def test_bad_batches(N, bad, st):
    L, c, b, q, kv = N.lib(), cache(N), batch(N, **bad), rows(N), rows(N, H=2)
    assert L.fa_paged_attention(by(q), by(c), by(b), 1, 0.0, 0x90000, None, 0xA0000, 1 << 40, None) == st
    assert L.fa_paged_weights(by(q), 0x90000, by(c), by(b), 1, 0.0, 0xA0000, 128, 1, None) == st
    assert L.fa_rope_append(None, by(kv), by(kv), by(c), by(b), None, 0, 0, None, 0, 0x90000, 0x90000, None, None) == st
    if "cu" not in bad:
        assert L.fa_paged_evict(by(c), by(b), 0x90000, 128, 8, 0, 0, 0xA0000, 0xB0000, None, None) == st


@pytest.mark.parametrize("bad,st", BAD_ROWS)
def test_bad_rows(N, bad, st):
    L, c, b, q = N.lib(), cache(N), batch(N), rows(N, **bad)
    kv = rows(N, H=2)
    assert L.fa_paged_attention(by(q), by(c), by(b), 1, 0.0, 0x90000, None, 0xA0000, 1 << 40, None) == st
    assert L.fa_paged_weights(by(q), 0x90000, by(c), by(b), 1, 0.0, 0xA0000, 128, 1, None) == st
    args = (by(c), by(b), None, 0, 0, None, 0, 0x90000, 0x90000)
    assert L.fa_rope_append(by(q), by(kv), by(kv), *args, by(rows(N)), None) == st
    assert L.fa_rope_append(by(rows(N)), by(kv), by(kv), *args, by(q), None) == st
    bkv = rows(N, **{**dict(H=2), **bad})
    assert L.fa_rope_append(None, by(bkv), by(kv), *args, None, None) == st
    assert L.fa_rope_append(None, by(kv), by(bkv), *args, None, None) == st


def test_null_descriptors(N):
    L, c, b, q, kv = N.lib(), cache(N), batch(N), rows(N), rows(N, H=2)
    for a in ((None, by(c), by(b)), (by(q), None, by(b)), (by(q), by(c), None)):
        assert L.fa_paged_attention(*a, 1, 0.0, 0x90000, None, 0xA0000, 1 << 40, None) == INVALID
        assert L.fa_paged_attention_workspace_size(*a) == 0
    assert L.fa_rope_append(None, None, by(kv), by(c), by(b), None, 0, 0, None, 0, 0x90000, 0x90000, None, None) == INVALID
    assert L.fa_rope_append(None, by(kv), None, by(c), by(b), None, 0, 0, None, 0, 0x90000, 0x90000, None, None) == INVALID


def test_attention_refusals(N):
    L, c, b, q = N.lib(), cache(N), batch(N), rows(N)
    need = L.fa_paged_attention_workspace_size(by(q), by(c), by(b))
    assert need > 0
    run = lambda out=0x90000, lse=None, ws=0xA0000, n=need, qq=q: L.fa_paged_attention(
        by(qq), by(c), by(b), 1, 0.0, out, lse, ws, n, None)
    assert run(out=None) == INVALID and run(out=0x90008) == INVALID and run(lse=0x90001) == INVALID
    assert run(ws=None) == WORKSPACE and run(n=need - 1) == WORKSPACE and run(ws=0xA0080) == WORKSPACE
    assert run(qq=rows(N, H=3)) == INVALID  # 3 query heads over 2
    # nothing to do: no launch, whatever the buffers
    assert run(out=None, ws=None, n=0, qq=rows(N, T=0, data=None)) == OK
    b0 = batch(N, B=0, table=None, lens=None)
    assert L.fa_paged_attention(by(q), by(c), by(b0), 1, 0.0, None, None, None, 0, None) == OK


def test_weights_refusals(N):
    L, c, b, q = N.lib(), cache(N), batch(N), rows(N)
    run = lambda lse=0x90000, acc=0xA0000, stride=128: L.fa_paged_weights(by(q), lse, by(c), by(b), 1, 0.0, acc, stride, 1,
                                                                         None)
    assert run(lse=None) == INVALID and run(lse=0x90002) == INVALID
    assert run(acc=None) == INVALID and run(acc=0xA0001) == INVALID and run(stride=-1) == INVALID


def test_append_refusals(N):
    L, c, b = N.lib(), cache(N), batch(N)
    kv, q = rows(N, H=2), rows(N)

    def run(q=None, k=kv, v=kv, cs=None, npos=0, rd=0, pos=None, ak=0x90000, av=0x90000, qo=None, c=c):
        r = lambda x: None if x is None else by(x)
        return L.fa_rope_append(r(q), r(k), r(v), by(c), by(b), cs, npos, rd, pos, 0, ak, av, r(qo), None)

    assert run(ak=None) == NO_CALIBRATION and run(av=None) == NO_CALIBRATION
    assert run(k=rows(N, H=4)) == INVALID and run(v=rows(N, H=2, T=4)) == INVALID
    assert run(q=q) == INVALID and run(qo=q) == INVALID  # one without the other
    assert run(q=q, qo=rows(N, T=4)) == INVALID and run(q=q, qo=rows(N, H=2)) == INVALID
    assert run(q=q, qo=rows(N, stride=1024)) == INVALID  # in place at another stride
    for rd in (-16, 8, 24, 144):
        assert run(cs=0x90000, npos=8, rd=rd) == INVALID
    assert run(rd=64) == INVALID and run(cs=0x90008, npos=8, rd=64) == INVALID and run(cs=0x90000, npos=-1, rd=64) == INVALID
    assert run(pos=0x90002) == INVALID
    assert run(k=rows(N, H=2, T=0, data=None), v=rows(N, H=2, T=0, data=None)) == OK


def test_table_refusals(N):
    L = N.lib()
    f = (ctypes.c_double * 64)()
    assert L.fa_rope_table(0x90000, -1, 64, f, 1.0, None) == INVALID
    for rd in (0, -2, 3, 130):
        assert L.fa_rope_table(0x90000, 8, rd, f, 1.0, None) == INVALID
    assert L.fa_rope_table(None, 8, 64, f, 1.0, None) == INVALID and L.fa_rope_table(0x90000, 8, 64, None, 1.0, None) == INVALID
    assert L.fa_rope_table(None, 0, 64, f, 1.0, None) == OK


def test_evict_refusals(N):
    L, c, b = N.lib(), cache(N), batch(N, cu=None)
    run = lambda sc=0x90000, stride=128, budget=8, sink=0, recent=0, kept=0xA0000, new=0xB0000, so=None: L.fa_paged_evict(
        by(c), by(b), sc, stride, budget, sink, recent, kept, new, so, None)
    assert run(budget=0) == INVALID and run(sink=-1) == INVALID and run(recent=-1) == INVALID
    assert run(sink=5, recent=4) == INVALID and run(stride=-1) == INVALID
    assert run(sink=2 ** 31 - 1, recent=2 ** 31 - 1, budget=2 ** 31 - 1) == INVALID
    assert run(sc=None) == INVALID and run(kept=None) == INVALID and run(new=None) == INVALID
    assert run(so=0x90000) == INVALID and run(so=0xC0001) == INVALID


def test_frequencies():
    import quantized_attention_amax_b200 as faq
    f, m = faq.rope_frequencies(8, 10000.0)
    assert m == 1.0 and f == [10000.0 ** (-2 * i / 8) for i in range(4)]
    g, m = faq.rope_frequencies(8, 10000.0, {"type": "linear", "factor": 4.0})
    assert m == 1.0 and g == [x / 4.0 for x in f]
    g, m = faq.rope_frequencies(8, 10000.0, {"type": "ntk", "factor": 4.0})
    assert m == 1.0 and g[0] == 1.0 and g[3] == pytest.approx(f[3] / 4.0, rel=1e-12)
    # yarn: pairs that turn often stay, pairs that hardly turn slow by the factor, between them a blend
    g, m = faq.rope_frequencies(128, 10000.0, {"type": "yarn", "factor": 8.0, "original": 4096})
    f, _ = faq.rope_frequencies(128)
    turns = [4096 * x / (2 * math.pi) for x in f]
    assert m == pytest.approx(0.1 * math.log(8.0) + 1.0)
    for x, y, n in zip(f, g, turns):
        if n > 40:
            assert y == x
        if n < 0.9:
            assert y == pytest.approx(x / 8.0, rel=1e-12)
        assert x / 8.0 * (1 - 1e-12) <= y <= x
    assert all(a > b for a, b in zip(g, g[1:]))
    # bands: by wavelength
    g, m = faq.rope_frequencies(128, 500000.0, {"type": "bands", "factor": 8.0, "original": 8192})
    f, _ = faq.rope_frequencies(128, 500000.0)
    for x, y in zip(f, g):
        wave = 2 * math.pi / x
        want = x if wave < 8192 / 4 else x / 8 if wave > 8192 else (
            lambda s: (1 - s) * x / 8 + s * x)((8192 / wave - 1) / 3)
        assert y == pytest.approx(want, rel=1e-12)
    for bad in (dict(rotary_dim=7), dict(rotary_dim=8, scaling={"type": "other", "factor": 2.0}),
                dict(rotary_dim=8, scaling={"type": "linear", "factor": 0.0}),
                dict(rotary_dim=2, scaling={"type": "ntk", "factor": 2.0})):
        with pytest.raises(ValueError):
            faq.rope_frequencies(**bad)


def test_binding_refuses_what_the_boundary_cannot_see():
    import torch
    import quantized_attention_amax_b200 as faq
    z = torch.zeros(4, 2, 16, 64, dtype=torch.int8)
    with pytest.raises(ValueError):  # a CPU tensor
        faq.PagedCache(z, z, torch.zeros(2), torch.zeros(2), "int8_per_head")
    with pytest.raises(ValueError):
        faq.PagedCache(z, z, torch.zeros(2), torch.zeros(2), "mxfp8")
    with pytest.raises(ValueError):
        faq.PagedCache(z, z, torch.zeros(2), torch.zeros(2), "int8_per_head", "SBND")
    with pytest.raises(ValueError):
        faq.empty_paged_cache(4, 2, 16, 64, "float", device="cpu")
    with pytest.raises(ValueError):
        faq.PagedBatch(torch.zeros(2, dtype=torch.int32), torch.zeros(2, dtype=torch.int32))


def test_sizes_of_weights_and_eviction(N):
    """No new token with accumulate=0 is work (zeros are written), so its buffers are checked; a budget past
    2^30 is refused; score rows of no token need no buffer (the refusal is then that of the kept list)."""
    L, c = N.lib(), cache(N)
    b = batch(N)
    none = rows(N, T=0, H=8)
    run = lambda acc=0x90000, stride=128, add=0: L.fa_paged_weights(by(none), None, by(c), by(b), 1, 0.0, acc, stride, add, None)
    assert run(acc=None) == INVALID and run(acc=0x90002) == INVALID
    assert run(acc=None, add=1) == OK
    b = batch(N, cu=None)
    assert L.fa_paged_evict(by(c), by(b), 0x90000, 128, 2 ** 30 + 1, 0, 0, 0xA0000, 0xB0000, None, None) == UNSUPPORTED
    assert L.fa_paged_evict(by(c), by(b), None, 0, 8, 0, 0, None, 0xB0000, None, None) == INVALID
