"""Outputs of the paged-cache operators that lie on what the kernels still read are refused before any launch; columns of
one matrix side by side are not.  Rows are compared byte by byte with what the host's arithmetic decides.  (What must
pass is stopped by a later refusal, so that no call here launches anything on made-up addresses.)"""
import ctypes
import random

import pytest

from test_paged_cpu import N, batch, cache, rows  # noqa: F401  (N is a fixture)

by = ctypes.byref
INVALID, NO_CALIBRATION, WORKSPACE = 1, 3, 7
BASE = 0x1000000


def granules(data, T, H, D, stride):
    """The 16-byte pieces that rows hold."""
    return {(data + 2 * t * stride + b) // 16 for t in range(T) for b in range(0, 2 * H * D, 16)}


def crossing(a, b):
    return max(min(a), min(b)) <= min(max(a), max(b))


def test_rotated_rows_against_what_is_read(N):
    L, c, b = N.lib(), cache(N, H=1, D=64), batch(N)
    rng = random.Random(1)
    seen = set()
    for _ in range(4000):
        T, Hq = rng.choice((1, 2, 3, 5)), rng.choice((1, 2))
        strides = [rng.choice((h * 64, h * 64 + 8, 256, 320)) for h in (Hq, 1, 1, Hq)]
        if rng.random() < 0.6:
            strides = [max(strides)] * 4
        at = [BASE + 16 * rng.randrange(0, 200) for _ in range(4)]
        if rng.random() < 0.3:
            at[3], strides[3] = at[0], strides[0]  # in place
        hs = (Hq, 1, 1, Hq)
        q, k, v, o = (N.FaRows(a, T, h, 64, s) for a, h, s in zip(at, hs, strides))
        sets = [granules(a, T, h, 64, s) for a, h, s in zip(at, hs, strides)]
        bad = False
        for i in range(3):
            if i == 0 and at[0] == at[3]:
                bad |= strides[0] != strides[3]
                continue
            same = strides[i] == strides[3] or T == 1
            bad |= bool(sets[i] & sets[3]) if same else crossing(sets[i], sets[3])
        got = L.fa_rope_append(by(q), by(k), by(v), by(c), by(b) if T == 5 else by(batch(N, B=T)), None, 0, 0, None, 0, None, None,
                               by(o), None)
        assert got == (INVALID if bad else NO_CALIBRATION), (at, strides, T, Hq)
        seen.add((bad, at[0] == at[3], T == 1))
    assert len(seen) >= 7


def test_attention_outputs_against_the_queries(N):
    L, c = N.lib(), cache(N, H=1, D=64)
    rng = random.Random(2)
    seen = set()
    for _ in range(4000):
        T, H = rng.choice((1, 2, 3, 5)), rng.choice((1, 2))
        stride = rng.choice((H * 64, H * 64 + 8, 512, 2048))
        q = N.FaRows(BASE, T, H, 64, stride)
        out = BASE + 16 * rng.randrange(-100, 1000)
        lse = rng.choice((None, BASE + 16 * rng.randrange(-100, 1000)))
        sq, so = granules(BASE, T, H, 64, stride), granules(out, 1, T * H, 64, 0)
        sl = set() if lse is None else {(lse + x) // 16 for x in range(0, 4 * T * H, 4)}
        bad = bool(sq & so or sq & sl or so & sl)
        got = L.fa_paged_attention(by(q), by(c), by(batch(N, B=T)), 1, 0.0, out, lse, None, 0, None)
        assert got == (INVALID if bad else WORKSPACE), (T, H, stride, out - BASE, lse)
        seen.add((bad, T == 1))
    assert len(seen) == 4
    # the workspace
    at = 0x40000000
    q, b = rows(N, T=2, H=2, data=at), batch(N, B=2)
    need = L.fa_paged_attention_workspace_size(by(q), by(cache(N)), by(b))
    assert 0 < need < at // 2
    up = lambda x: (x + 255) // 256 * 256
    for out, lse, ws in ((2 * at, None, 2 * at), (2 * at + need - 256, None, 2 * at), (0x90000, 2 * at + 256, 2 * at),
                         (0x90000, None, at + 256), (0x90000, None, up(at - need) + 256)):
        assert L.fa_paged_attention(by(q), by(cache(N)), by(b), 1, 0.0, out, lse, ws, need, None) == INVALID


def test_weights_and_eviction_outputs(N):
    L, c, b, q = N.lib(), cache(N), batch(N), rows(N)
    n = 2 * 2 * 128 * 4  # of acc and scores: B 2, heads 2, stride 128
    for acc in (0x80000, 0x80000 + 5 * 4 * 128 * 2 - 4, 0x80000 - n + 4, 0x90000, 0x90000 + 5 * 4 * 4 - 4):
        assert L.fa_paged_weights(by(q), 0x90000, by(c), by(b), 1, 0.0, acc, 128, 1, None) == INVALID
    b = batch(N, cu=None)
    run = lambda kept=0xA0000, new=0xB0000, so=None: L.fa_paged_evict(by(c), by(b), 0x90000, 128, 8, 0, 0, kept, new, so, None)
    for so in (0x90000, 0x90000 + n - 4, 0x90000 - n + 4, 0x60000, 0x70000, 0xA0000, 0xB0004):
        assert run(so=so) == INVALID
    for kept in (0x90004, 0x60000 + 12, 0x70004, 0xB0000):
        assert run(kept=kept) == INVALID
    for new in (0x70000, 0x70004, 0x60008, 0x90000 + n - 4, 0xA0000 + 2 * 2 * 8 * 4 - 4):  # (seq_lens itself among them)
        assert run(new=new) == INVALID
