"""GPU tests of what the paged-cache operators leave in memory: a serving run whose caches are built on the host step by
step (the 64-bit forms' rotation, the oracle's codes and scales), and calls on bad device data, which must change
nothing but what their good sequences own."""
import ctypes

import pytest
import torch

import _paged_ref as ref
import workloads as wl
from _gpu import faq_module
from test_paged_gpu import assert_within, batch_of, bf16, to_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def faq():
    return faq_module()


def append_on_host(orc, c, table, lens, qlens, k, v, amax, written=None):
    """Quantize the new rows k (rotated) and v [T, H, D] into the host cache c by the oracle.  written: [T] bool, the
    tokens that are (None: all)."""
    for name, y, am in (("k", k, amax[0]), ("v", v, amax[1])):
        bits = wl.bf16_bits(y[None])
        if c["mode"] in ref.PER_HEAD:
            codes, sc = getattr(orc, "quantize_" + c["mode"])(bits, am.numpy(), "BSND")
            c[name + "s"] = torch.from_numpy(sc)
        else:
            codes, sc = getattr(orc, "quantize_" + c["mode"])(bits, "BSND")
        codes, sc = torch.from_numpy(codes)[0], torch.from_numpy(sc)
        t = 0
        for b, (n, m) in enumerate(zip(lens, qlens)):
            for i in range(m):
                if written is not None and not written[t + i]:
                    continue
                j = n - m + i
                pg, o = int(table[b, j // c["page"]]), j % c["page"]
                if c["layout"] == "BNSD":
                    c[name + "c"][pg, :, o] = codes[t + i]
                else:
                    c[name + "c"][pg, o] = codes[t + i]
                if c["mode"] not in ref.PER_HEAD:
                    c[name + "s"][pg, :, o] = sc[0, :, t + i]
            t += m


def assert_cache(gc, c):
    for n, t in (("kc", gc.k_codes), ("vc", gc.v_codes), ("ks", gc.k_scales), ("vs", gc.v_scales)):
        assert torch.equal(t.cpu(), c[n]), n  # every slot of every page


@pytest.mark.parametrize("mode", ref.MODES)
@pytest.mark.parametrize("layout", ["BNSD", "BSND"])
def test_serving_run_against_a_cache_made_on_the_host(faq, orc, mode, layout):
    """Prompts in chunks, drafts, weights, eviction, single tokens behind the kept ones.  After every call the four tensors
    of the cache are the host's bit for bit; attention and weights are compared with the 64-bit forms on the
    host's cache."""
    H, Hq, D, page = 2, 6, 64, 16
    budget, room = 48, 208
    table, pages = ref.make_table((room, room, room), page, 4)
    c = ref.make_cache(mode, layout, pages, H, page, D, 5)
    gc = to_gpu(faq, c)
    cs = faq.rope_table(512, 32)
    amax = [torch.full((H,), 4.0), torch.full((H,), 3.5)]
    acc = torch.zeros(3, H, room).cuda()
    lens, true = [0, 0, 0], [0, 0, 0]

    def step(qlens, seed):
        T = sum(qlens)
        x = bf16((T + 1, Hq + 2 * H, D), seed)
        for b in range(3):
            lens[b] += qlens[b]
            true[b] += qlens[b]
        pos = torch.cat([torch.arange(true[b] - qlens[b], true[b]) for b in range(3)] + [torch.tensor([0])]).to(torch.int32)
        gb, gx = batch_of(faq, table, lens, qlens, max(qlens)), x.cuda()
        out = torch.full((T + 1, Hq, D), 7.0, dtype=torch.bfloat16).cuda()
        faq.rope_append(gx[:, :Hq], gx[:, Hq:Hq + H], gx[:, Hq + H:], gc, gb, cs, pos.cuda(),
                        amax=[a.cuda() for a in amax] if mode in ref.PER_HEAD else None, out=out)
        faq.check_device_status()
        rows = cs.cpu()[pos[:T].long()]
        q, k = ref.turn(x[:T, :Hq], rows, False), ref.turn(x[:T, Hq:Hq + H], rows, False)
        append_on_host(orc, c, table, lens, qlens, k, x[:T, Hq + H:], amax)
        assert torch.equal(out[:T].cpu().view(torch.int16), q.view(torch.int16)) and (out[T:] == 7.0).all()
        assert_cache(gc, c)
        before = acc.cpu()
        got, lse = faq.paged_attention(out, gc, gb, return_lse=True)
        faq.paged_weights(out, lse, gc, gb, acc)
        faq.check_device_status()
        assert_cache(gc, c)
        want, z, tol, ltol = ref.attend(q, c, table, lens, qlens, True)
        assert_within(got[:T], want, tol, "out")
        assert_within(lse[:T], z, ltol, "lse")
        w, wtol = ref.weigh(q, lse[:T].cpu(), c, table, lens, qlens, True, room)
        w = w + before.double()
        assert_within(acc, w, wtol + w.abs() * 2.0 ** -24, "weights")
        return gb

    step((100, 61, 1), 1)
    step((50, 0, 30), 2)
    gb = step((6, 3, 0), 3)
    kept, new, so = ref.evict(c, table, lens, acc.cpu(), budget, 2, 8)
    acc2 = torch.empty_like(acc)
    gk, gn = faq.paged_evict(gc, gb, acc, budget, 2, 8, scores_out=acc2)
    faq.check_device_status()
    assert torch.equal(gk.cpu(), kept) and torch.equal(gn.cpu(), new) and torch.equal(acc2.cpu(), so)
    assert_cache(gc, c)
    acc.copy_(acc2)
    lens[:] = gn.tolist()
    for k in range(3):
        step((1, 1, 1), 10 + k)


class Guarded:
    """A tensor between two bands that must stay as they are."""

    def __init__(self, shape, dtype, fill):
        n = 1
        for s in shape:
            n *= s
        self.band = 4096
        self.all = torch.full((n + 2 * self.band,), fill, dtype=dtype).cuda()
        self.t = self.all[self.band:self.band + n].view(shape)
        self.fill = fill

    def check(self):
        assert (self.all[:self.band] == self.fill).all() and (self.all[-self.band:] == self.fill).all()


def reported(faq):
    with pytest.raises(faq.FaqError) as e:
        faq.check_device_status()
    assert e.value.status == 8
    faq.check_device_status()


LENS, QLENS = (100, 60, 30), (2, 2, 2)


def bad_setups(table, pages):
    """(what, table, lens, cu, sequences that stay good)"""
    for page in (-1, pages, 2 ** 31 - 1, -2 ** 31):
        t = table.clone()
        t[1, 3] = page  # tokens 48 to 63 of sequence 1
        yield f"page {page}", t, LENS, (0, 2, 4, 6), (0, 2)
    for n in (-1, 16 * table.shape[1] + 1, 2 ** 31 - 1):
        yield f"length {n}", table, (100, n, 30), (0, 2, 4, 6), (0, 2)
    yield "cu past the rows", table, LENS, (0, 2, 4, 9), (0, 1)
    yield "cu falls", table, LENS, (0, 2, 1, 1), (0, 2)
    yield "cu below zero", table, LENS, (-1, 2, 4, 6), (1, 2)


@pytest.mark.parametrize("mode", ref.MODES)
@pytest.mark.parametrize("layout", ["BNSD", "BSND"])
def test_bad_device_data_changes_nothing_else(faq, orc, mode, layout):
    H, Hq, D, page = 2, 4, 64, 16
    table, pages = ref.make_table(LENS, page, 1)
    clean = ref.make_cache(mode, layout, pages, H, page, D, 2)
    q, kv = bf16((6, Hq, D), 3), bf16((6, 2 * H, D), 4)
    amax = [torch.full((H,), 4.0), torch.full((H,), 3.5)]
    from quantized_attention_amax_b200 import _native as N
    by = ctypes.byref
    for what, tab, lens, cu, good in bad_setups(table, pages):
        gb = faq.PagedBatch(tab.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), torch.tensor(cu, dtype=torch.int32).cuda())
        m = [cu[b + 1] - cu[b] for b in range(3)]
        rows = torch.cat([torch.arange(cu[b], cu[b + 1]) for b in good])
        # attention and weights: the good sequences' rows, nothing outside the buffers, the cache as it was
        gc = to_gpu(faq, clean)
        out, lse = Guarded((6, Hq, D), torch.bfloat16, 7.0), Guarded((6, Hq), torch.float32, 7.0)
        faq.paged_attention(q.cuda(), gc, gb, out=out.t, lse=lse.t)
        reported(faq)
        out.check(), lse.check()
        assert_cache(gc, clean)
        for b in good:
            r = slice(cu[b], cu[b + 1])
            want, z, tol, ltol = ref.attend(q[r], clean, table[b:b + 1], LENS[b:b + 1], (m[b],), True)
            assert_within(out.t[r], want, tol, what)
            assert_within(lse.t[r], z, ltol, what)
        lse_in = torch.zeros(6, Hq)
        for b in good:
            r = slice(cu[b], cu[b + 1])
            lse_in[r] = lse.t[r].cpu()
        acc = Guarded((3, H, 112), torch.float32, 5.0)
        faq.paged_weights(q.cuda(), lse_in.cuda(), gc, gb, acc.t)
        reported(faq)
        acc.check()
        assert_cache(gc, clean)
        for b in good:
            r = slice(cu[b], cu[b + 1])
            w, wtol = ref.weigh(q[r], lse_in[r], clean, table[b:b + 1], LENS[b:b + 1], (m[b],), True, 112)
            w = w + 5.0
            assert_within(acc.t[b:b + 1], w, wtol + w * 2.0 ** -24, what)
            assert (acc.t[b, :, LENS[b]:] == 5.0).all()
        # the append: the good sequences' tokens and nothing else (a bad page's tokens are left out; both of sequence 1's are)
        gc, c = to_gpu(faq, clean), {n: x.clone() if torch.is_tensor(x) else x for n, x in clean.items()}
        faq.rope_append(None, kv[:, :H].contiguous().cuda(), kv[:, H:].contiguous().cuda(), gc, gb,
                        amax=[a.cuda() for a in amax] if mode in ref.PER_HEAD else None)
        reported(faq)
        sel = torch.cat([kv[cu[b]:cu[b + 1]] for b in good])
        append_on_host(orc, c, table[list(good)], [LENS[b] for b in good], [m[b] for b in good], sel[:, :H], sel[:, H:], amax)
        if mode in ref.PER_HEAD:
            assert torch.equal(gc.k_scales.cpu(), c["ks"]) and torch.equal(gc.v_scales.cpu(), c["vs"])
        assert_cache(gc, c)
        # the eviction (it does not read cu): the good sequences' slots as they should be, no slot of a page that no
        # sequence has, nothing outside the lists
        if what.startswith("cu"):
            continue
        sc = torch.rand(3, H, 112, generator=torch.Generator().manual_seed(6))
        gc, c = to_gpu(faq, clean), {n: x.clone() if torch.is_tensor(x) else x for n, x in clean.items()}
        kept, new, so = Guarded((3, H, 20), torch.int32, -9), Guarded((3,), torch.int32, -9), Guarded((3, H, 112), torch.float32, 9.0)
        st = N.lib().fa_paged_evict(by(gc.c()), by(gb.c()), sc.cuda().data_ptr(), 112, 20, 2, 18, kept.t.data_ptr(), new.t.data_ptr(),
                                    so.t.data_ptr(), torch.cuda.current_stream().cuda_stream)
        assert st == 0
        torch.cuda.synchronize()
        reported(faq)
        kept.check(), new.check(), so.check()
        for b in good:
            k, n, s = ref.evict(c, table[b:b + 1], LENS[b:b + 1], sc[b:b + 1], 20, 2, 18)
            assert torch.equal(kept.t[b:b + 1].cpu(), k) and torch.equal(new.t[b:b + 1].cpu(), n)
            assert torch.equal(so.t[b:b + 1].cpu(), s)
        own = torch.zeros(pages, dtype=torch.bool)
        own[table[1][table[1] >= 0].long()] = True  # pages of the bad sequence: not compared
        for n, t in (("kc", gc.k_codes), ("vc", gc.v_codes), ("ks", gc.k_scales), ("vs", gc.v_scales)):
            t = t.cpu()
            assert torch.equal(t, c[n]) if t.dim() == 1 else torch.equal(t[~own], c[n][~own]), (what, n)


def test_bad_positions_leave_their_tokens_out(faq, orc):
    H, D, page = 2, 64, 16
    table, pages = ref.make_table(LENS, page, 1)
    k, v, q = bf16((6, H, D), 3), bf16((6, H, D), 4), bf16((6, 4, D), 5)
    cs = faq.rope_table(50, 64)
    for p in (-1, 50, 2 ** 31 - 1):
        c = ref.make_cache("fp8_per_token", "BNSD", pages, H, page, D, 2)
        gc, gb = to_gpu(faq, c), batch_of(faq, table, LENS, QLENS)
        pos = torch.tensor([3, 4, p, 5, 6, 7], dtype=torch.int32)
        out = Guarded((6, 4, D), torch.bfloat16, 7.0)
        faq.rope_append(q.cuda(), k.cuda(), v.cuda(), gc, gb, cs, pos.cuda(), out=out.t)
        reported(faq)
        out.check()
        written = torch.tensor([True, True, False, True, True, True])
        rows = cs.cpu()[torch.where(written, pos, 0).long()]
        append_on_host(orc, c, table, LENS, QLENS, ref.turn(k, rows, False), v, (None, None), written)
        assert_cache(gc, c)
        assert torch.equal(out.t.cpu()[written], ref.turn(q, rows, False)[written]) and (out.t[2] == 7.0).all()
