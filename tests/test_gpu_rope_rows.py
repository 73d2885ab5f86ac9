"""Rotation and the fused store over every number of rows that a thread of the
kernel may take, whole passes and passes with places to spare."""
import pytest
import torch

from fp8_w8a8_dynamic_b200 import mfp8
from fp8_w8a8_dynamic_b200 import workloads as W
from serving_ref import rope_ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("layout", (mfp8.ROPE_HALF, mfp8.ROPE_INTERLEAVED))
@pytest.mark.parametrize("D,rot", [(128, 128), (256, 96), (96, 48)])
@pytest.mark.parametrize("rows", range(1, 11))
def test_rows_per_thread(rows, D, rot, layout):
    """128 threads take a token while there are few: 128 / (threads of a row)
    heads are one row per thread."""
    lanes = 16 if D > 128 else 8
    H = rows * (128 // lanes)
    Hkv = max(1, H // 6)
    Hq, T, ps = H - 2 * Hkv, 5, 8
    x = W.make_x(T * H, D, seed=rows, stream=D, kind="rowscale", device="cuda").view(T, H, D)
    pos = torch.tensor([0, 1, 77, 4095, 262143], dtype=torch.int32, device="cuda")
    freq, _ = mfp8.rope_frequencies(rot, 5e6)
    y = mfp8.rope(x, pos, freq, layout=layout)
    ref, tol = rope_ref(x, pos, freq, None, layout, 1.0)
    assert ((y.double() - ref).abs() <= tol).all()
    pages = [torch.zeros((2, Hkv, ps, D), dtype=torch.uint8, device="cuda") for _ in range(4)]
    scale = [torch.ones((2, Hkv, ps), device="cuda") for _ in range(4)]
    slot = torch.tensor([9, 0, -1, 7, 15], device="cuda")
    q = mfp8.rope_kv_store(x.flatten(1), Hq, pos, freq, slot, pages[0], scale[0], pages[1], scale[1], layout=layout)
    mfp8.kv_page_store(y[:, Hq:Hq + Hkv], slot, pages[2], scale[2])
    mfp8.kv_page_store(x[:, Hq + Hkv:], slot, pages[3], scale[3])
    assert torch.equal(q, y[:, :Hq])
    for k in range(2):
        assert torch.equal(pages[k], pages[2 + k]) and torch.equal(scale[k], scale[2 + k])
    assert mfp8.device_status() == mfp8.OK
