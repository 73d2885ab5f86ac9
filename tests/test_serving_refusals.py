"""Each refusal of the Python helpers for rotary positions, the paged KV cache
and attention by its own message, so that a check that went missing is not
covered by the next one (that of the device, which every tensor on the CPU
fails where there is a GPU)."""
import pytest
import torch

from fp8_w8a8_dynamic_b200 import mfp8

BF, I32 = torch.bfloat16, torch.int32


class Inputs:
    """Arguments that fit each other, on one device."""

    def __init__(self, device):
        def zeros(*shape, dtype=torch.float32):
            return torch.zeros(shape, dtype=dtype, device=device)

        self.x = zeros(4, 8, 64, dtype=BF)
        self.qkv = zeros(4, 24 * 64, dtype=BF)
        self.pos, self.pos2 = zeros(4, dtype=I32), zeros(2, 4, dtype=I32)
        self.freq, self.axis = zeros(32), zeros(32, dtype=torch.uint8)
        self.slot = torch.arange(4, device=device)
        self.pages, self.scale = zeros(2, 8, 16, 64, dtype=torch.uint8), zeros(2, 8, 16)
        self.start, self.len = torch.arange(5, dtype=I32, device=device), zeros(4, dtype=I32)
        self.table, self.prefix = zeros(4, 3, dtype=I32), zeros(2, dtype=I32)
        self.out = zeros(4, 8, 64, dtype=BF)

    def rope(self, **kw):
        a = dict(x=self.x, pos=self.pos, inv_freq=self.freq)
        return mfp8.rope(**{**a, **kw})

    def store(self, **kw):
        a = dict(kv=self.x, slot=self.slot, pages=self.pages, scale=self.scale)
        return mfp8.kv_page_store(**{**a, **kw})

    def read(self, **kw):
        a = dict(pages=self.pages, scale=self.scale, slot=self.slot)
        return mfp8.kv_page_read(**{**a, **kw})

    def both(self, **kw):
        a = dict(qkv=self.qkv, n_heads=8, pos=self.pos, inv_freq=self.freq, slot=self.slot, k_pages=self.pages,
                 k_scale=self.scale, v_pages=self.pages.clone(), v_scale=self.scale.clone())
        return mfp8.rope_kv_store(**{**a, **kw})

    def attend(self, **kw):
        a = dict(q=self.x, q_start=self.start, kv_len=self.len, page_table=self.table, prefix_pages=self.prefix,
                 prefix_len=32, k_pages=self.pages, k_scale=self.scale, v_pages=self.pages, v_scale=self.scale, max_q=1)
        return mfp8.prefix_attention(**{**a, **kw})


SHAPE_X = r"must be bf16 \[T, H, D\]"
HEAD_ROWS = r"the head rows of a token in \w+ must be contiguous"
POS, FREQ = "pos must be contiguous int32", "inv_freq must be contiguous fp32"
AXIS = "axis must be contiguous uint8"
SLOT, PER_TOKEN = "slot must be contiguous int64", "slot must have one entry per token"
PAGES, SCALE = "pages must be contiguous uint8", "scale must be contiguous fp32"
ONE_SHAPE = "k_pages and v_pages must have one shape"
QKV = "qkv must be bf16"
START, LEN = "q_start must be contiguous int32", "kv_len must be contiguous int32"
TABLE, TABLE_ROWS = r"page_table must be int32 \[B, max_pages\]", "the rows of page_table must be contiguous"
PREFIX = "prefix_pages must be contiguous int32 and cover prefix_len"
DEVICE = "tensors must be on the current CUDA device"

REFUSED = [
    ("rope", lambda i: dict(x=i.x.float()), SHAPE_X),
    ("rope", lambda i: dict(x=i.x[0]), SHAPE_X),
    ("rope", lambda i: dict(x=i.x[:, ::2]), HEAD_ROWS),
    ("rope", lambda i: dict(x=i.x.transpose(1, 2)), HEAD_ROWS),
    ("rope", lambda i: dict(pos=i.pos[:3]), POS),
    ("rope", lambda i: dict(pos=i.pos.long()), POS),
    ("rope", lambda i: dict(pos=i.pos2.t()), POS),
    ("rope", lambda i: dict(pos=i.pos2[None]), POS),
    ("rope", lambda i: dict(inv_freq=i.freq.double()), FREQ),
    ("rope", lambda i: dict(inv_freq=i.freq[::2]), FREQ),
    ("rope", lambda i: dict(inv_freq=i.freq[None]), FREQ),
    ("rope", lambda i: dict(pos=i.pos2), "several position axes need `axis`"),
    ("rope", lambda i: dict(pos=i.pos2, axis=i.axis.int()), AXIS),
    ("rope", lambda i: dict(pos=i.pos2, axis=i.axis[:16]), AXIS),
    ("store", lambda i: dict(kv=i.x.half()), SHAPE_X),
    ("store", lambda i: dict(kv=i.x[:, ::2]), HEAD_ROWS),
    ("store", lambda i: dict(pages=i.pages.int()), PAGES),
    ("store", lambda i: dict(pages=i.pages[0]), PAGES),
    ("store", lambda i: dict(pages=i.pages.transpose(1, 2)), PAGES),
    ("store", lambda i: dict(scale=i.scale[:1]), SCALE),
    ("store", lambda i: dict(scale=i.scale.double()), SCALE),
    ("store", lambda i: dict(pages=i.pages[:, :4].contiguous(), scale=i.scale[:, :4].contiguous()),
     "kv and pages must have the same heads and head size"),
    ("store", lambda i: dict(slot=i.slot[:3]), PER_TOKEN),
    ("store", lambda i: dict(slot=i.slot.int()), SLOT),
    ("store", lambda i: dict(slot=torch.zeros(8, dtype=torch.int64)[::2]), SLOT),
    ("read", lambda i: dict(pages=i.pages[0]), PAGES),
    ("read", lambda i: dict(pages=i.pages.int()), PAGES),
    ("read", lambda i: dict(scale=i.scale[..., :8]), SCALE),
    ("read", lambda i: dict(slot=i.slot.int()), SLOT),
    ("read", lambda i: dict(slot=i.slot[None]), SLOT),
    ("both", lambda i: dict(qkv=i.qkv.float()), QKV),
    ("both", lambda i: dict(qkv=i.qkv[:, :-64]), QKV),
    ("both", lambda i: dict(qkv=i.qkv[None]), QKV),
    ("both", lambda i: dict(n_heads=7), QKV),
    ("both", lambda i: dict(v_pages=i.pages[:1], v_scale=i.scale[:1]), ONE_SHAPE),
    ("both", lambda i: dict(v_scale=i.scale[:1]), SCALE),
    ("both", lambda i: dict(pos=i.pos[:2]), POS),
    ("both", lambda i: dict(slot=i.slot[:2]), PER_TOKEN),
    ("attend", lambda i: dict(q=i.x.float()), SHAPE_X),
    ("attend", lambda i: dict(q=i.x[:, ::2]), HEAD_ROWS),
    ("attend", lambda i: dict(q=i.x[..., :32].contiguous()), "q and the pages must have one head size"),
    ("attend", lambda i: dict(v_pages=i.pages[:1], v_scale=i.scale[:1]), ONE_SHAPE),
    ("attend", lambda i: dict(kv_len=i.len.long()), LEN),
    ("attend", lambda i: dict(kv_len=i.len[None]), LEN),
    ("attend", lambda i: dict(q_start=i.start[:4]), START),
    ("attend", lambda i: dict(q_start=i.start.long()), START),
    ("attend", lambda i: dict(page_table=i.table[:3]), TABLE),
    ("attend", lambda i: dict(page_table=i.table.long()), TABLE),
    ("attend", lambda i: dict(page_table=i.len), TABLE),
    ("attend", lambda i: dict(page_table=torch.zeros(3, 4, dtype=I32).t()), TABLE_ROWS),
    ("attend", lambda i: dict(prefix_len=33), PREFIX),
    ("attend", lambda i: dict(prefix_len=-1), PREFIX),
    ("attend", lambda i: dict(prefix_pages=None), PREFIX),
    ("attend", lambda i: dict(prefix_pages=i.prefix.long()), PREFIX),
    ("attend", lambda i: dict(prefix_pages=i.table[:, :2]), PREFIX),
]


@pytest.mark.parametrize("k", range(len(REFUSED)))
def test_refused_for_its_own_reason(k):
    name, change, message = REFUSED[k]
    i = Inputs("cpu")
    where = {"rope": "rope", "store": "kv_page_store", "read": "kv_page_read", "both": "rope_kv_store",
             "attend": "prefix_attention"}[name]
    with pytest.raises(ValueError, match=f"^{where}: .*{message}"):
        getattr(i, name)(**change(i))


@pytest.mark.gpu
def test_refused_on_the_device():
    """What is checked behind the device: outputs, workspace, streams; and tensors elsewhere."""
    i, host = Inputs("cuda"), Inputs("cpu")
    for name in ("rope", "store", "read", "both", "attend"):
        getattr(i, name)()  # fits as it is
        with pytest.raises(ValueError, match=DEVICE):
            getattr(host, name)()
    torch.cuda.synchronize()
    for name, change, message in [
            ("rope", dict(pos=host.pos), DEVICE), ("store", dict(slot=host.slot), DEVICE),
            ("attend", dict(page_table=host.table), DEVICE), ("read", dict(out=host.out), DEVICE),
            ("rope", dict(out=i.out[:3]), "out must have x's shape"),
            ("rope", dict(out=i.out.float()), SHAPE_X),
            ("read", dict(out=i.out.float()), "out must be contiguous bf16"),
            ("read", dict(out=i.out[:2]), "out must be contiguous bf16"),
            ("both", dict(out=i.out[:, ::2]), "out must be contiguous bf16"),
            ("both", dict(out=i.out.half()), "out must be contiguous bf16"),
            ("attend", dict(out=i.out[:3]), "out must be contiguous bf16"),
            ("attend", dict(out=i.out.transpose(0, 1)), "out must be contiguous bf16"),
            ("attend", dict(workspace=torch.zeros(1 << 20, 2, device="cuda")[:, 0]), "workspace must be contiguous")]:
        with pytest.raises(ValueError, match=message):
            getattr(i, name)(**change)
    assert mfp8.device_status() == mfp8.OK
