"""Rotary positions, the paged KV cache and attention over a shared prefix:
host arithmetic, and refusals before any device work (no GPU)."""
import ctypes
import math

import numpy as np
import pytest
import torch

from fp8_w8a8_dynamic_b200 import build as B
from fp8_w8a8_dynamic_b200 import mfp8

F = 1 << 20  # a 16-byte-aligned non-null address; never dereferenced
OK, ARG, ALIGN, SHAPE, WS = (mfp8.OK, mfp8.ERR_INVALID_ARG, mfp8.ERR_MISALIGNED, mfp8.ERR_UNSUPPORTED_SHAPE,
                             mfp8.ERR_WORKSPACE)


@pytest.fixture(scope="module", autouse=True)
def lib():
    B.build()
    return mfp8.lib()


def freqs(*a, **kw):
    t, m = mfp8.rope_frequencies(*a, device="cpu", **kw)
    return t.numpy(), m


def test_frequencies_plain_linear_ntk():
    i = np.arange(32, dtype=np.float64)
    base = 10000.0 ** (-2 * i / 64)
    t, m = freqs(64, 10000.0)
    assert m == 1.0 and np.array_equal(t, base.astype(np.float32)) and t.dtype == np.float32
    t, m = freqs(64, 10000.0, mfp8.ROPE_SCALE_LINEAR, 4.0)
    assert m == 1.0 and np.allclose(t, base / 4, rtol=2.0 ** -23, atol=0)
    t, m = freqs(64, 10000.0, mfp8.ROPE_SCALE_NTK, 4.0)
    # the fastest pair keeps its frequency, the slowest is divided by the factor
    assert m == 1.0 and t[0] == 1.0 and math.isclose(t[31], base[31] / 4, rel_tol=2.0 ** -22)
    assert (np.diff(t) < 0).all()


def test_frequencies_yarn():
    n, theta, L, f, fast, slow = 128, 5e6, 32768, 8.0, 32.0, 1.0
    base = theta ** (-2 * np.arange(64) / n)
    t, m = freqs(n, theta, mfp8.ROPE_SCALE_YARN, f, L, fast, slow)
    assert math.isclose(m, 0.1 * math.log(f) + 1)
    turns = L * base / (2 * math.pi)
    kept, cut = turns > fast * 1.3, turns < slow / 1.3
    assert kept.any() and cut.any()
    assert np.allclose(t[kept], base[kept], rtol=2.0 ** -22, atol=0)
    assert np.allclose(t[cut], base[cut] / f, rtol=2.0 ** -22, atol=0)
    ratio = t / base
    assert (np.diff(ratio) <= 1e-6).all() and (ratio <= 1 + 1e-6).all() and (ratio >= 1 / f - 1e-6).all()
    # the ramp runs over whole pairs: linear in the pair's number between its ends
    mid = ratio[(ratio < 0.999) & (ratio > 1 / f + 0.001)]
    assert len(mid) > 2 and np.allclose(np.diff(mid, 2), 0, atol=1e-6)
    assert freqs(n, theta, mfp8.ROPE_SCALE_YARN, 1.0, L)[1] == 1.0


def test_frequencies_refused():
    out = (ctypes.c_float * 128)()
    p = ctypes.addressof(out)

    def call(rot=64, theta=1e4, scaling=0, factor=1.0, L=0, fast=32.0, slow=1.0, table=p):
        return mfp8.mfp8_rope_frequencies(rot, theta, scaling, factor, L, fast, slow, table, None)

    assert call() == OK and call(rot=256) == OK
    assert [call(rot=r) for r in (0, -16, 24, 272)] == [SHAPE] * 4
    assert [call(theta=t) for t in (1.0, 0.0, -5.0, math.inf, math.nan)] == [ARG] * 5
    assert [call(scaling=s) for s in (-1, 4)] == [ARG] * 2
    assert [call(scaling=1, factor=f) for f in (0.5, math.nan, math.inf)] == [ARG] * 3
    assert call(table=None) == ARG
    assert call(scaling=3, factor=2.0, L=4096) == OK
    assert [call(scaling=3, factor=2.0, L=l) for l in (0, -1)] == [ARG] * 2
    assert call(scaling=3, factor=2.0, L=4096, fast=1.0, slow=1.0) == ARG
    assert call(scaling=3, factor=2.0, L=4096, slow=0.0) == ARG
    with pytest.raises(mfp8.Mfp8Error):
        mfp8.rope_frequencies(20, 1e4, device="cpu")


def test_rope_refused():
    base = dict(X=F, ldx=1024, T=4, H=8, D=128, pos=2 * F, n=1, axis=None, freq=3 * F, rot=128, layout=0, ms=1.0,
                Y=4 * F, ldy=1024)

    def call(**kw):
        a = {**base, **kw}
        return mfp8.mfp8_rope(*a.values())

    assert call(T=0) == OK and call(T=0, X=None, Y=None, pos=None) == OK
    assert [call(**k) for k in (dict(T=-1), dict(H=-1), dict(n=0), dict(n=5), dict(layout=2), dict(layout=-1),
                                dict(ms=math.nan), dict(ms=math.inf), dict(X=None), dict(Y=None), dict(pos=None),
                                dict(freq=None), dict(n=3), dict(ldx=-8))] == [ARG] * 14
    assert [call(**k) for k in (dict(D=0), dict(D=120), dict(D=272, ldx=4096, ldy=4096), dict(rot=8), dict(rot=144),
                                dict(rot=-16), dict(H=0), dict(ldx=1016), dict(ldx=1028), dict(ldy=1016),
                                dict(T=1 << 40), dict(H=1 << 20, ldx=1 << 27, ldy=1 << 27))] == [SHAPE] * 12
    assert [call(**k) for k in (dict(X=F + 8), dict(Y=4 * F + 2), dict(pos=2 * F + 2), dict(freq=3 * F + 1))] == [ALIGN] * 4
    assert call(Y=F + 16) == ARG                # shifted over the input
    assert call(Y=F, ldy=2048) == ARG           # in place with other strides
    assert call(Y=F + 4 * 2048 - 16) == ARG     # its last row
    assert call(Y=2 * F) == ARG and call(Y=3 * F) == ARG  # over the positions, the table
    assert call(Y=5 * F, n=2, axis=5 * F + 64) == ARG
    assert call(Y=2 * F, rot=0, T=0) == OK


def test_page_store_and_read_refused():
    base = dict(X=F, ld=1024, slot=2 * F + 8, T=4, H=8, D=128, pages=16 * F, scale=32 * F, n=4, ps=16)

    def store(**kw):
        return mfp8.mfp8_kv_page_store(*{**base, **kw}.values())

    assert store(T=0) == OK and store(T=0, X=None, slot=None) == OK
    assert [store(**k) for k in (dict(T=-1), dict(n=-1), dict(X=None), dict(slot=None), dict(pages=None),
                                 dict(scale=None), dict(D=-16))] == [ARG] * 7
    assert [store(**k) for k in (dict(H=0), dict(D=0), dict(D=24), dict(D=272), dict(ld=1016), dict(ld=1028),
                                 dict(ps=0), dict(ps=4), dict(ps=24), dict(ps=512), dict(ps=-8), dict(n=1 << 40),
                                 dict(n=2 ** 31 - 1, ps=256, H=64, ld=8192))] == [SHAPE] * 13
    assert [store(**k) for k in (dict(X=F + 2), dict(slot=2 * F + 4), dict(pages=16 * F + 8),
                                 dict(scale=32 * F + 4))] == [ALIGN] * 4
    assert store(pages=F + 16) == ARG and store(scale=F + 64) == ARG and store(scale=16 * F + 1024) == ARG
    assert store(pages=2 * F) == ARG  # over the slots

    rbase = dict(pages=16 * F, scale=32 * F, n=4, ps=16, slot=2 * F, T=4, H=8, D=128, out=F)

    def read(**kw):
        return mfp8.mfp8_kv_page_read(*{**rbase, **kw}.values())

    assert read(T=0) == OK and read(T=0, out=None, slot=None) == OK
    assert [read(**k) for k in (dict(T=-1), dict(out=None), dict(slot=None), dict(pages=None))] == [ARG] * 4
    assert [read(**k) for k in (dict(H=0), dict(D=40), dict(ps=12), dict(T=1 << 40))] == [SHAPE] * 4
    assert [read(**k) for k in (dict(out=F + 2), dict(scale=32 * F + 8), dict(slot=2 * F + 2))] == [ALIGN] * 3
    assert read(out=16 * F + 16) == ARG and read(out=32 * F) == ARG


def test_rope_kv_store_refused():
    base = dict(X=F, ld=1536, T=4, Hq=8, Hkv=2, D=128, pos=2 * F, n=1, axis=None, freq=3 * F, rot=128, layout=0,
                ms=1.0, slot=4 * F, Q=5 * F, kp=16 * F, ks=32 * F, vp=48 * F, vs=64 * F, np=4, ps=16)

    def call(**kw):
        return mfp8.mfp8_rope_kv_store(*{**base, **kw}.values())

    assert call(T=0) == OK
    assert [call(**k) for k in (dict(T=-1), dict(X=None), dict(Q=None), dict(slot=None), dict(kp=None), dict(vs=None),
                                dict(layout=3), dict(n=2), dict(ms=math.inf))] == [ARG] * 9
    assert [call(**k) for k in (dict(Hq=0), dict(Hkv=0), dict(ld=1528), dict(ld=1540), dict(ps=100), dict(rot=24),
                                dict(D=20), dict(Hq=1 << 40))] == [SHAPE] * 8
    assert [call(**k) for k in (dict(X=F + 4), dict(Q=5 * F + 8), dict(kp=16 * F + 1), dict(vs=64 * F + 4),
                                dict(slot=4 * F + 4))] == [ALIGN] * 5
    assert [call(**k) for k in (dict(Q=F), dict(vp=16 * F), dict(vs=32 * F + 16), dict(kp=5 * F),
                                dict(ks=4 * F), dict(Q=2 * F), dict(vp=3 * F))] == [ARG] * 7


BASE = dict(Q=F, ldq=1024, T=4, Hq=8, Hkv=2, D=128, qs=2 * F, kl=3 * F, B=4, mq=1, kp=16 * F, ks=32 * F, vp=48 * F,
            vs=64 * F, n=8, ps=16, pp=4 * F, P=40, pt=5 * F, ldt=2, mp=2, scale=0.1, O=6 * F, lse=None, ws=80 * F,
            wsb=1 << 30, path=0, stream=None)


def attend(**kw):
    return mfp8.lib().mfp8_prefix_attention(*{**BASE, **kw}.values())


def test_prefix_attention_refused():
    assert attend(T=0) == OK and attend(B=0) == OK
    assert [attend(**k) for k in (dict(T=-1), dict(B=-1), dict(Q=None), dict(O=None), dict(qs=None), dict(kl=None),
                                  dict(pp=None), dict(pt=None), dict(kp=None), dict(vs=None), dict(n=0), dict(P=-1),
                                  dict(scale=0.0), dict(scale=-1.0), dict(scale=math.nan),
                                  dict(scale=math.inf), dict(path=-1), dict(path=3))] == [ARG] * 18
    assert [attend(**k) for k in (dict(D=96), dict(D=256, ldq=2048), dict(Hq=7, ldq=896), dict(Hkv=0), dict(mq=0),
                                  dict(ldq=1016), dict(ldq=1028), dict(ps=20), dict(ldt=1), dict(T=1 << 21),
                                  dict(B=1 << 21), dict(P=1 << 31), dict(mp=1 << 30, ldt=1 << 30))] == [SHAPE] * 13
    assert [attend(**k) for k in (dict(Q=F + 8), dict(O=6 * F + 4), dict(kp=16 * F + 8), dict(ws=80 * F + 8),
                                  dict(qs=2 * F + 2), dict(lse=7 * F + 1), dict(pt=5 * F + 2))] == [ALIGN] * 7
    assert [attend(**k) for k in (dict(ws=None), dict(wsb=100))] == [WS] * 2
    assert [attend(**k) for k in (dict(O=F), dict(lse=6 * F), dict(O=48 * F + 64), dict(ws=32 * F), dict(lse=3 * F),
                                  dict(O=4 * F), dict(O=5 * F), dict(ws=6 * F + 16))] == [ARG] * 8


def test_prefix_attention_workspace():
    size = mfp8.mfp8_prefix_attention_workspace_bytes
    assert size(0, 4, 1, 8, 2, 128, 40, 2, 16) == 0 and size(4, 4, 1, 8, 2, 96, 40, 2, 16) == 0
    assert size(4, 4, 1, 8, 2, 128, 40, 2, 24) == 0
    # a prefix and own tokens: at least one partial output and log-sum-exp of each per row
    assert size(4, 4, 1, 8, 2, 128, 40, 2, 16) >= 2 * 4 * 8 * (128 + 1) * 4
    # one short part alone is written straight to the output
    assert size(4, 4, 1, 8, 2, 128, 0, 2, 16) == 0 and size(4, 4, 1, 8, 2, 128, 40, 0, 16) == 0
    assert size(4, 4, 1, 8, 2, 128, 0, 0, 16) == 0


def test_binding_checks_before_the_library():
    bf, i32 = torch.bfloat16, torch.int32
    x = torch.zeros(4, 8, 64, dtype=bf)
    pos = torch.zeros(4, dtype=i32)
    f = torch.zeros(32)
    pages, scale = torch.zeros(2, 8, 16, 64, dtype=torch.uint8), torch.zeros(2, 8, 16)
    slot = torch.zeros(4, dtype=torch.int64)
    bad = [lambda: mfp8.rope(x.float(), pos, f), lambda: mfp8.rope(x[:, ::2], pos, f),
           lambda: mfp8.rope(x, pos[:3], f), lambda: mfp8.rope(x, pos.long(), f), lambda: mfp8.rope(x, pos, f.double()),
           lambda: mfp8.rope(x, torch.zeros(3, 4, dtype=i32), f),
           lambda: mfp8.kv_page_store(x, slot, pages[:, :4], scale), lambda: mfp8.kv_page_store(x, slot[:3], pages, scale),
           lambda: mfp8.kv_page_store(x, slot.int(), pages, scale), lambda: mfp8.kv_page_store(x, slot, pages, scale[:1]),
           lambda: mfp8.kv_page_read(pages[0], scale, slot), lambda: mfp8.kv_page_read(pages.int(), scale, slot),
           lambda: mfp8.rope_kv_store(x.flatten(1), 8, pos, f, slot, pages, scale, pages, scale),
           lambda: mfp8.prefix_attention(x, pos, pos, None, None, 0, pages, scale, pages, scale, 1),
           lambda: mfp8.prefix_attention(x, torch.zeros(5, dtype=i32), pos, pos, None, 0, pages, scale, pages, scale, 1),
           lambda: mfp8.prefix_attention(x, torch.zeros(5, dtype=i32), pos, None, pos[:1], 17, pages, scale, pages,
                                         scale, 1)]
    for call in bad:
        with pytest.raises(ValueError):
            call()
