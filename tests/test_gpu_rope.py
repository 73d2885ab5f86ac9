"""Rotary positions and the paged FP8 KV cache on the GPU: against 64-bit
forms, the CPU oracle's quantizer and one another."""
import math

import numpy as np
import pytest
import torch

import oracle
from fp8_w8a8_dynamic_b200 import mfp8
from fp8_w8a8_dynamic_b200 import workloads as W
from helpers import bits16, f32, u8
from serving_ref import rope_ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
BOTH = (mfp8.ROPE_HALF, mfp8.ROPE_INTERLEAVED)


@pytest.fixture(autouse=True)
def status_stays_clean():
    yield
    assert mfp8.device_status() == mfp8.OK


def rows(T, H, D, seed):
    return W.make_x(T * H, D, seed=seed, stream=D, kind="rowscale", device=DEV).view(T, H, D)


def positions(T, axes, far, seed):
    g = torch.Generator().manual_seed(seed)
    p = torch.randint(-far, far, (axes, T), generator=g, dtype=torch.int32)
    p[:, 0] = 0
    p[:, -1] = far
    return (p if axes > 1 else p[0]).to(DEV)


def axis_of(rot, axes):
    return (torch.arange(rot // 2) % axes).to(torch.uint8).to(DEV) if axes > 1 else None


@pytest.mark.parametrize("layout", BOTH)
@pytest.mark.parametrize("T,H,D,rot,axes,far", [
    (1, 1, 16, 16, 1, 5), (1, 32, 128, 128, 1, 100000), (3, 5, 96, 32, 1, 2 ** 31 - 1), (7, 40, 128, 128, 3, 262144),
    (33, 3, 256, 256, 2, 1000000), (700, 8, 64, 48, 4, 32768), (2500, 2, 80, 80, 1, 8192), (1300, 1, 16, 16, 3, 999),
    (5, 300, 32, 16, 1, 77), (9, 4, 192, 176, 1, 4096)])
def test_rope_against_64_bits(T, H, D, rot, axes, far, layout):
    x = rows(T, H, D, seed=T + D)
    pos = positions(T, axes, far, seed=T)
    freq, _ = mfp8.rope_frequencies(rot, 5e6)
    axis = axis_of(rot, axes)
    y = mfp8.rope(x, pos, freq, axis=axis, layout=layout, mscale=1.25)
    ref, tol = rope_ref(x, pos, freq, axis, layout, 1.25)
    assert ((y.double() - ref).abs() <= tol).all()
    assert torch.equal(y[..., rot:], x[..., rot:])


@pytest.mark.parametrize("layout", BOTH)
def test_rope_strided_in_place_and_back(layout):
    T, Hq, Hkv, D, rot = 37, 6, 2, 64, 32
    qkv = rows(T, Hq + 2 * Hkv, D, seed=3).reshape(T, -1).contiguous()
    before = qkv.clone()
    pos = positions(T, 1, 5000, seed=4)
    freq, _ = mfp8.rope_frequencies(rot, 10000.0)
    q = qkv[:, :Hq * D].unflatten(1, (Hq, D))
    fresh = mfp8.rope(q, pos, freq, layout=layout)
    same = mfp8.rope(q.contiguous(), pos, freq, layout=layout)
    assert torch.equal(fresh, same)
    wide = torch.full((T, Hq + 3, D), 7.0, dtype=torch.bfloat16, device=DEV)
    mfp8.rope(q, pos, freq, layout=layout, out=wide[:, :Hq])
    assert torch.equal(wide[:, :Hq], fresh) and (wide[:, Hq:] == 7.0).all()
    assert torch.equal(qkv, before)
    mfp8.rope(q, pos, freq, layout=layout, out=q)  # in place, inside the packed rows
    assert torch.equal(q, fresh) and torch.equal(qkv[:, Hq * D:], before[:, Hq * D:])
    # the negated position turns back: two bf16 roundings and the rotations' own errors
    back = mfp8.rope(fresh, -pos, freq, layout=layout)
    size = before[:, :Hq * D].unflatten(1, (Hq, D)).double().abs().amax(-1, keepdim=True)
    assert ((back.double() - before[:, :Hq * D].unflatten(1, (Hq, D)).double()).abs() <= size * 2.0 ** -6).all()


def test_rope_identity_cases():
    x = rows(11, 4, 48, seed=1)
    freq, _ = mfp8.rope_frequencies(48, 100.0)
    zero = torch.zeros(11, dtype=torch.int32, device=DEV)
    assert torch.equal(mfp8.rope(x, zero, freq), x)
    none = torch.empty(0, device=DEV)
    assert torch.equal(mfp8.rope(x, zero + 9, none), x)  # rot = 0 copies
    empty = mfp8.rope(x[:0], zero[:0], freq)
    assert empty.shape == (0, 4, 48)


@pytest.mark.parametrize("scaling", [mfp8.ROPE_SCALE_LINEAR, mfp8.ROPE_SCALE_NTK, mfp8.ROPE_SCALE_YARN])
def test_rope_scaled_tables(scaling):
    freq, mscale = mfp8.rope_frequencies(64, 10000.0, scaling, 8.0, 4096)
    x = rows(50, 3, 64, seed=9)
    pos = positions(50, 1, 32768, seed=2)
    y = mfp8.rope(x, pos, freq, mscale=mscale)
    ref, tol = rope_ref(x, pos, freq, None, 0, mscale)
    assert ((y.double() - ref).abs() <= tol).all()


def pool(n_pages, H, ps, D):
    return (torch.full((n_pages, H, ps, D), 0x55, dtype=torch.uint8, device=DEV),
            torch.full((n_pages, H, ps), -3.0, device=DEV))


def some_slots(T, n_pages, ps, seed, skip=0.2):
    g = torch.Generator().manual_seed(seed)
    s = torch.randperm(n_pages * ps, generator=g)[:T]
    return torch.where(torch.rand(T, generator=g) < skip, torch.tensor(-1), s).to(DEV)


SHAPES = [(1, 8, 128, 8), (5, 1, 16, 16), (37, 3, 64, 32), (9, 4, 256, 128), (700, 8, 128, 16), (3, 2, 48, 256),
          (2001, 5, 96, 64)]


@pytest.mark.parametrize("T,H,D,ps", SHAPES)
def test_page_store_and_read(T, H, D, ps):
    n_pages = -(-T // ps) + 2
    pages, scale = pool(n_pages, H, ps, D)
    wide = rows(T, H + 2, D, seed=T + D)
    kv = wide[:, 1:1 + H]
    slot = some_slots(T, n_pages, ps, seed=T)
    mfp8.kv_page_store(kv, slot, pages, scale)
    q_ref, s_ref = oracle.kv_quantize(bits16(kv))
    codes, scales = u8(pages), f32(scale)
    want_c, want_s = np.full(codes.shape, 0x55, np.uint8), np.full(scales.shape, -3.0, np.float32)
    for t, s in enumerate(slot.tolist()):
        if s >= 0:
            want_c[s // ps, :, s % ps] = q_ref[t]
            want_s[s // ps, :, s % ps] = s_ref[t]
    assert np.array_equal(codes, want_c) and np.array_equal(scales.view(np.uint32), want_s.view(np.uint32))
    # read back, in another order, with repeats and padding
    pick = torch.cat([slot.flip(0), slot[:1], slot[:1], torch.tensor([-5], device=DEV)])
    back = mfp8.kv_page_read(pages, scale, pick)
    index = [s for s in pick.tolist()]
    d_ref = oracle.kv_dequantize(q_ref, s_ref)
    at = {s: t for t, s in enumerate(slot.tolist())}
    got = bits16(back)
    for i, s in enumerate(index):
        assert np.array_equal(got[i], d_ref[at[s]] if s >= 0 else np.zeros((H, D), np.uint16))


@pytest.mark.parametrize("layout", BOTH)
@pytest.mark.parametrize("T,Hq,Hkv,D,rot,axes,ps", [
    (1, 32, 8, 128, 128, 1, 16), (16, 32, 8, 128, 128, 3, 64), (37, 3, 3, 64, 32, 1, 8), (5, 7, 1, 256, 256, 2, 32),
    (777, 4, 2, 96, 96, 1, 128), (1500, 2, 1, 32, 16, 1, 256), (3, 200, 100, 16, 0, 1, 8)])
def test_rope_kv_store_is_its_parts(T, Hq, Hkv, D, rot, axes, ps, layout):
    n_pages = -(-T // ps) + 1
    wide = rows(T, Hq + 2 * Hkv + 1, D, seed=T + D)
    qkv = wide[:, :Hq + 2 * Hkv].flatten(1)
    qkv = wide.flatten(1)[:, :(Hq + 2 * Hkv) * D]  # a strided view of the same values
    pos = positions(T, axes, 50000, seed=T)
    freq = mfp8.rope_frequencies(rot, 5e6)[0] if rot else torch.empty(0, device=DEV)
    axis = axis_of(rot, axes)
    slot = some_slots(T, n_pages, ps, seed=T + 1)
    kp, ks = pool(n_pages, Hkv, ps, D)
    vp, vs = pool(n_pages, Hkv, ps, D)
    q = mfp8.rope_kv_store(qkv, Hq, pos, freq, slot, kp, ks, vp, vs, axis=axis, layout=layout, mscale=0.75)
    qk = mfp8.rope(wide[:, :Hq + Hkv], pos, freq, axis=axis, layout=layout, mscale=0.75)
    kp2, ks2 = pool(n_pages, Hkv, ps, D)
    vp2, vs2 = pool(n_pages, Hkv, ps, D)
    mfp8.kv_page_store(qk[:, Hq:], slot, kp2, ks2)
    mfp8.kv_page_store(wide[:, Hq + Hkv:Hq + 2 * Hkv], slot, vp2, vs2)
    for a, b in ((q, qk[:, :Hq]), (kp, kp2), (ks, ks2), (vp, vp2), (vs, vs2)):
        assert torch.equal(a, b)


def test_edge_rows_store_and_read_exactly():
    """Zero, -0, subnormal and near-max rows."""
    D = 128
    kv = torch.zeros((4, 2, D), dtype=torch.bfloat16)
    kv[0, 1] = -0.0
    kv[1, 0, 3] = 1e-40
    kv[1, 1] = torch.linspace(-3e38, 3e38, D, dtype=torch.float64).to(torch.bfloat16)
    kv[2, 0] = torch.tensor([(-1.0) ** i * 2.0 ** (i - 64) for i in range(D)]).to(torch.bfloat16)
    kv[3] = torch.randn(2, D).to(torch.bfloat16)
    kv = kv.to(DEV)
    pages, scale = pool(1, 2, 8, D)
    slot = torch.tensor([6, 0, 3, 1], device=DEV)
    mfp8.kv_page_store(kv, slot, pages, scale)
    q_ref, s_ref = oracle.kv_quantize(bits16(kv))
    assert np.array_equal(u8(pages)[0][:, slot.cpu()].swapaxes(0, 1), q_ref)
    assert np.array_equal(bits16(mfp8.kv_page_read(pages, scale, slot)), oracle.kv_dequantize(q_ref, s_ref))


def test_slots_out_of_range_are_skipped_and_reported():
    pages, scale = pool(2, 2, 8, 32)
    kv = rows(3, 2, 32, seed=1)
    slot = torch.tensor([16, 3, 2 ** 40], device=DEV)
    mfp8.kv_page_store(kv, slot, pages, scale)
    assert mfp8.device_status() == mfp8.ERR_INDEX
    assert mfp8.device_status() == mfp8.OK
    touched = (scale != -3.0).nonzero().tolist()
    assert touched == [[0, 0, 3], [0, 1, 3]]
    back = mfp8.kv_page_read(pages, scale, slot)
    assert mfp8.device_status() == mfp8.ERR_INDEX
    assert (back[0] == 0).all() and (back[2] == 0).all()
    assert torch.equal(back[1], mfp8.kv_page_read(pages, scale, slot[1:2])[0])


def test_offsets_past_32_bits():
    """A pool of more than 2^32 code bytes: the last page is reached."""
    H, ps, D = 8, 256, 128
    n_pages = 2 ** 32 // (H * ps * D) + 2
    pages = torch.zeros((n_pages, H, ps, D), dtype=torch.uint8, device=DEV)
    scale = torch.zeros((n_pages, H, ps), device=DEV)
    kv = rows(2, H, D, seed=1)
    slot = torch.tensor([n_pages * ps - 1, 5], device=DEV)
    mfp8.kv_page_store(kv, slot, pages, scale)
    q_ref, s_ref = oracle.kv_quantize(bits16(kv))
    assert np.array_equal(u8(pages[-1, :, -1]), q_ref[0]) and np.array_equal(u8(pages[0, :, 5]), q_ref[1])
    assert int((scale != 0).sum()) == 2 * H
    assert np.array_equal(bits16(mfp8.kv_page_read(pages, scale, slot)), oracle.kv_dequantize(q_ref, s_ref))


def test_other_stream_and_graph():
    T, Hq, Hkv, D, ps = 16, 4, 2, 64, 16
    freq, _ = mfp8.rope_frequencies(D, 10000.0)
    qkv = rows(T, Hq + 2 * Hkv, D, seed=5).flatten(1)
    pos = positions(T, 1, 100, seed=1)
    slot = some_slots(T, 2, ps, seed=2, skip=0.0)
    kp, ks = pool(2, Hkv, ps, D)
    vp, vs = pool(2, Hkv, ps, D)
    want = mfp8.rope_kv_store(qkv, Hq, pos, freq, slot, kp, ks, vp, vs)
    kp2, ks2 = pool(2, Hkv, ps, D)
    vp2, vs2 = pool(2, Hkv, ps, D)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = mfp8.rope_kv_store(qkv, Hq, pos, freq, slot, kp2, ks2, vp2, vs2, stream=side)
    side.synchronize()
    assert torch.equal(got, want) and torch.equal(kp, kp2) and torch.equal(vs, vs2)
    # captured, then replayed on new values in the same buffers
    out = torch.empty_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mfp8.rope_kv_store(qkv, Hq, pos, freq, slot, kp2, ks2, vp2, vs2, out=out)
        back = mfp8.kv_page_read(kp2, ks2, slot)
    new = rows(T, Hq + 2 * Hkv, D, seed=6).flatten(1)
    qkv.copy_(new)
    pos.add_(3)
    graph.replay()
    want = mfp8.rope_kv_store(new, Hq, pos, freq, slot, kp, ks, vp, vs)
    assert torch.equal(out, want) and torch.equal(kp, kp2) and torch.equal(vp, vp2)
    assert torch.equal(back, mfp8.kv_page_read(kp, ks, slot))


def test_mscale_and_math_at_far_positions():
    """At 2^31 - 1 the angle's 64-bit product still leaves 2^-22 of a turn."""
    T, D = 64, 32
    pos = (torch.arange(T, dtype=torch.int64) * 33554393 % (2 ** 31 - 1)).to(torch.int32).to(DEV)
    freq, _ = mfp8.rope_frequencies(D, 5e6)
    x = torch.ones((T, 1, D), dtype=torch.bfloat16, device=DEV)
    y = mfp8.rope(x, pos, freq).double().cpu()
    a = pos.double().cpu()[:, None] * freq.double().cpu()
    ref = torch.cat([a.cos() - a.sin(), a.cos() + a.sin()], -1)
    assert ((y[:, 0] - ref).abs() <= ref.abs() * 2.0 ** -8 + 2.0 ** -21).all()
    assert math.isfinite(float(y.sum()))
