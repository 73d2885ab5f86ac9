"""Attention over a shared prefix where a row, a cached token or a length is
not as it should be, on the GPU against the 64-bit form."""
import copy
import math

import pytest
import torch

from fp8_w8a8_dynamic_b200 import mfp8
from serving_ref import Batch

pytestmark = pytest.mark.gpu

PATHS = (mfp8.ATTEND_ROWS, mfp8.ATTEND_TALL)
ALL_PATHS = (mfp8.ATTEND_AUTO,) + PATHS


@pytest.fixture(autouse=True)
def status_stays_clean():
    yield
    assert mfp8.device_status() == mfp8.OK


def run(b, path, **kw):
    out, lse = mfp8.prefix_attention(*b.args(), want_lse=True, path=path, **kw)
    return out, lse, b.D ** -0.5


# ------------------------------------------- a query row that is not finite --

@pytest.mark.parametrize("path", ALL_PATHS)
@pytest.mark.parametrize("D", (64, 128))
def test_one_infinite_element_makes_its_row_nan(D, path):
    """Every product with an infinity is infinite or NaN, so the softmax has no
    value, however small the keys; the other rows keep their bits."""
    b = Batch([1] * 80, [9, 700] * 40, 6000, 8, 2, D, 64, seed=31, k_gain=2.0 ** -6)
    want, want_lse, _ = run(b, path)
    bad = [(17, 3, 5, math.inf), (40, 0, D - 1, -math.inf), (41, 7, 0, math.nan), (79, 2, D // 2, math.inf)]
    keep = torch.ones(80, 8, dtype=torch.bool, device="cuda")
    for t, h, d, x in bad:
        b.q[t, h, d] = x
        keep[t, h] = False
    got, lse, _ = run(b, path)
    assert got[~keep].isnan().all() and lse[~keep].isnan().all()
    assert torch.equal(got[keep], want[keep]) and torch.equal(lse[keep], want_lse[keep])


@pytest.mark.parametrize("path", PATHS)
def test_an_infinite_row_whose_only_logit_is_minus_infinity(path):
    """It sees a token, so it is not a row that sees nothing."""
    b = Batch([1, 1], [1, 1], 0, 1, 1, 128, 8, seed=32)
    key = b.values(b.slots[1], 0)[0][0]
    d = int(key.abs().argmax())
    b.q[0, 0, d] = -math.inf if key[d] > 0 else math.inf
    out, lse, _ = run(b, path)
    assert out[0].isnan().all() and lse[0].isnan().all()
    assert out[1].isfinite().all() and lse[1].isfinite().all()


@pytest.mark.parametrize("path", PATHS)
def test_an_infinite_row_that_sees_nothing(path):
    b = Batch([1, 3], [0, 2], 0, 8, 2, 128, 16, seed=33)
    b.q[0, 1, 3] = math.inf
    b.q[1, 5, 9] = math.nan  # the first of three new tokens with two cached: before both
    out, lse, scale = run(b, path)
    b.check(out, lse, scale)
    assert (out[:2] == 0).all() and (lse[:2] == -math.inf).all()


# ------------------------------------------ more query tokens than `max_q` --

def cut_ref(b, max_q, scale):
    """(out, out bound, lse, lse bound) when query tokens past max_q of their sequence see the prefix alone."""
    c = copy.copy(b)
    c.own, c.slots = [0] * b.B, [b.slots[0]] + [b.slots[0][:0]] * b.B
    late = torch.zeros(b.T, dtype=torch.bool, device="cuda")
    for i in range(b.B):
        late[b.start[i] + max_q:b.start[i + 1]] = True
    full, alone = b.ref(scale), c.ref(scale)
    return late, [torch.where(late.view((-1,) + (1,) * (x.dim() - 1)), y, x) for x, y in zip(full, alone)]


@pytest.mark.parametrize("path", ALL_PATHS)
@pytest.mark.parametrize("n,own,P,D", [([3, 9, 2], [20, 40, 8], 0, 64), ([3, 9, 2], [700, 40, 3000], 0, 128),
                                       ([3, 9, 2], [20, 40, 8], 90, 128), ([40, 1, 300], [60, 5, 900], 3000, 64)])
def test_query_tokens_past_max_q(n, own, P, D, path):
    """They see the prefix alone, whatever the workspace holds, and are
    reported; the others are not disturbed."""
    b = Batch(n, own, P, 8, 2, D, 16, seed=P + D, first_row=2, extra_rows=1)
    max_q = 4
    b.max_q = max_q
    size = mfp8.mfp8_prefix_attention_workspace_bytes(b.T, b.B, max_q, 8, 2, D, P, b.page_table.shape[1], 16)
    outs = []
    for fill in (1.0, math.nan, -3.0e38):
        ws = torch.full((max(size, 16) // 4,), fill, device="cuda")
        out = torch.full((b.T, 8, D), 7.0, dtype=torch.bfloat16, device="cuda")
        out, lse, scale = run(b, path, workspace=ws, out=out)
        assert mfp8.device_status() == mfp8.ERR_INDEX
        outs.append((out, lse))
    late, (ref, tol, rl, lt) = cut_ref(b, max_q, scale)
    assert late.any()
    for out, lse in outs:
        assert (out[:2] == 7.0).all() and (out[-1:] == 7.0).all()
        rows = slice(b.start[0], b.start[-1])
        assert torch.equal(out[rows], outs[0][0][rows]) and torch.equal(lse[rows], outs[0][1][rows])
    o, r, t = out[rows].double(), ref[rows], tol[rows]
    assert ((o - r).abs() <= t).all()
    none = torch.isinf(rl[rows])
    assert torch.equal(none, lse[rows] == -math.inf)
    assert ((lse[rows].double() - rl[rows]).abs()[~none] <= lt[rows][~none]).all()
    assert (o[none] == 0).all() and bool(none.any()) == (P == 0)


# ------------------------------------------------------ a prefix and no table --

@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("B", (3, 200))
def test_lengths_without_a_page_table_are_checked(B, path):
    """Starts past the last token or decreasing, own tokens without a table,
    and more query tokens than max_q are reported where nothing but the prefix
    is read; the rows they do not concern keep their bits."""
    b = Batch([1] * B, [0] * B, 70, 8, 2, 64, 16, seed=B)
    want, want_lse, scale = run(b, path)
    b.check(want, want_lse, scale)
    assert mfp8.device_status() == mfp8.OK
    start, none = b.q_start.clone(), b.kv_len.clone()
    for where, at, value in (("q_start", B, B + 5), ("q_start", 0, -1), ("q_start", 1, 0), ("q_start", B - 1, 0), ("q_start", B - 2, B),
                             ("kv_len", B - 1, 1), ("kv_len", 0, -4)):
        getattr(b, where)[at] = value
        out, lse, _ = run(b, path)
        assert mfp8.device_status() == mfp8.ERR_INDEX, (where, at, value)
        assert torch.equal(out, want) and torch.equal(lse, want_lse)
        b.q_start.copy_(start)
        b.kv_len.copy_(none)


# --------------------------------------- cached tokens that are not finite --

SPOILT = {  # n, own, P, D, [(sequence or -1 for the prefix, token)]
    "in the middle of a prompt": ([40, 3], [60, 20], 100, 128, [(0, 47)]),
    "a prompt's last token": ([40, 3], [60, 20], 0, 64, [(0, 59)]),
    "two in a long prompt": ([300], [900], 0, 128, [(0, 700), (0, 893)]),
    "in a short prompt and a long one": ([300, 20, 70], [700, 20, 300], 555, 64, [(1, 11), (2, 299), (0, 410)]),
    "before the prompt": ([30, 30], [200, 40], 0, 128, [(0, 3)]),
    "a decode step": ([1] * 5, [50, 700, 3, 9, 1], 20, 128, [(1, 655), (4, 0)]),
    "in the prefix": ([1, 4], [50, 9], 300, 64, [(-1, 131)]),
}


@pytest.mark.parametrize("path", ALL_PATHS)
@pytest.mark.parametrize("what", (math.inf, -math.inf, math.nan))
@pytest.mark.parametrize("side", ("value", "key"))
@pytest.mark.parametrize("name", SPOILT)
def test_cached_tokens_that_are_not_finite(name, side, what, path):
    """A value row that holds an infinity or NaN makes NaN the outputs of the
    rows that see it and of no others, those of its tile and page among them;
    the log-sum-exps, which have no values in them, stay.  A key row makes
    both NaN."""
    n, own, P, D, spots = SPOILT[name]
    Hq, Hkv, ps, head = 8, 2, 16, 1
    b = Batch(n, own, P, Hq, Hkv, D, ps, seed=len(name))
    pages, scale = (b.v_pages, b.v_scale) if side == "value" else (b.k_pages, b.k_scale)
    slots = torch.stack([b.slots[1 + q][t] for q, t in spots]).cuda()
    x = torch.randn((len(spots), Hkv, D), generator=torch.Generator("cuda").manual_seed(1), device="cuda").bfloat16()
    mfp8.kv_page_store(x, slots, pages, scale)
    ref, tol, rl, lt = b.ref(D ** -0.5)
    x[:, head, 7] = what
    mfp8.kv_page_store(x, slots, pages, scale)  # the other heads' bytes stay as they were
    out, lse, _ = run(b, path)
    sees = torch.zeros(b.T, Hq, dtype=torch.bool, device="cuda")
    for q, t in spots:
        for s in range(b.B) if q < 0 else [q]:
            first = 0 if q < 0 else max(0, t - (own[s] - n[s]))
            sees[b.start[s] + first:b.start[s + 1], head * Hq // Hkv:(head + 1) * Hq // Hkv] = True
    assert sees.any()
    assert out[sees].isnan().all()
    assert ((out.double() - ref).abs() <= tol)[~sees].all()
    fine = ~sees if side == "key" else torch.ones_like(sees)
    assert ((lse.double() - rl).abs() <= lt)[fine].all() and lse[~fine].isnan().all()


@pytest.mark.parametrize("path", PATHS)
def test_a_value_that_is_not_finite_under_no_weight(path):
    """A token whose weight is far below the smallest number still counts: 0 NaN is NaN, whatever slot it is in."""
    b = Batch([1, 1], [3000, 3000], 3000, 8, 2, 128, 16, seed=41)
    q = torch.zeros_like(b.q)
    q[..., 0] = 100.0
    b.q = q
    k = torch.zeros((1, 2, 128), dtype=torch.bfloat16, device="cuda")
    for s, t, z in ((0, 5, 100.0), (1, 2000, -100.0), (2, 2000, -100.0)):
        k[..., 0] = z
        mfp8.kv_page_store(k, b.slots[s][t:t + 1].cuda(), b.k_pages, b.k_scale)
    out, lse, _ = run(b, path)
    assert out.isfinite().all() and lse.isfinite().all()
    at = b.slots[1][2000]
    b.v_scale[at // 16, 0, at % 16] = math.nan
    out, lse2, _ = run(b, path)
    assert out[0, :4].isnan().all() and out[0, 4:].isfinite().all() and out[1].isfinite().all()
    assert torch.equal(lse2, lse)


# ------------------------------------------------------ decode steps in a row --

@pytest.mark.parametrize("update", ("before the store", "after the store"))
@pytest.mark.parametrize("P,Hq", [(6000, 8), (1500, 32)])  # own tokens in 8-row and in 16-row tiles beside a tall prefix
def test_decode_steps_in_a_row(P, Hq, update):
    """Steps of rope_kv_store and prefix_attention whose two kernels run beside
    each other: each step writes new tokens next to cached ones, lengthens the
    sequences and gives some a new page right before the attention that needs
    them.  The bits of the same steps with a synchronisation after every call,
    eager and replayed, and the last step against 64 bits."""
    Hkv, D, ps, steps = 2, 128, 64, 6
    own = [9, 61, 62, 700] * 20
    B = len(own)
    b = Batch([1] * B, own, P, Hq, Hkv, D, ps, seed=P, spare_pages=2 * B, max_pages=12)
    free = sorted(set(range(b.k_pages.shape[0])) - set(b.prefix_pages.tolist())
                  - set(b.page_table[b.page_table >= 0].tolist()))
    tables, slots, table = [], [], b.page_table.clone()
    for s in range(steps):
        rows = []
        for i, l in enumerate(own):
            at = l + s
            if int(table[i, at // ps]) < 0:
                table[i, at // ps] = free.pop()
            rows.append(int(table[i, at // ps]) * ps + at % ps)
        tables.append(table.clone())
        slots.append(torch.tensor(rows, device="cuda"))
    lens = [torch.tensor(own, dtype=torch.int32, device="cuda") + s + 1 for s in range(steps)]
    pos = [(P + x - 1).contiguous() for x in lens]
    qkv = [torch.randn((B, (Hq + 2 * Hkv) * D), device="cuda", generator=torch.Generator("cuda").manual_seed(s)).bfloat16()
           for s in range(steps)]
    freq, _ = mfp8.rope_frequencies(D, 5e6)
    start = [x.clone() for x in (b.k_pages, b.k_scale, b.v_pages, b.v_scale, b.page_table, b.kv_len)]
    outs = [torch.zeros((B, Hq, D), dtype=torch.bfloat16, device="cuda") for _ in range(steps)]
    size = mfp8.mfp8_prefix_attention_workspace_bytes(B, B, 1, Hq, Hkv, D, P, 12, ps)
    ws = torch.zeros((size,), dtype=torch.uint8, device="cuda")

    def decode(state, outs, ws, between):
        kp, ks, vp, vs, table, kv_len = state
        for s in range(steps):
            if update == "before the store":
                table.copy_(tables[s])
                kv_len.add_(1)
                between()
            q = mfp8.rope_kv_store(qkv[s], Hq, pos[s], freq, slots[s], kp, ks, vp, vs)
            between()
            if update == "after the store":
                table.copy_(tables[s])
                kv_len.add_(1)
                between()
            mfp8.prefix_attention(q, b.q_start, kv_len, table, b.prefix_pages, P, kp, ks, vp, vs, 1, out=outs[s],
                                  workspace=ws)
            between()
        return q

    def apart():
        state = [x.clone() for x in start]
        ys = [torch.zeros_like(x) for x in outs]
        q = decode(state, ys, torch.zeros_like(ws), torch.cuda.synchronize)
        return q, ys, state

    def same(state, ys, want):
        assert all(torch.equal(x, y) for x, y in zip(ys, want[1]))
        assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(state, want[2]))

    want = apart()
    live = [x.clone() for x in start]
    decode(live, outs, ws, lambda: None)
    same(live, outs, want)

    last = copy.copy(b)
    last.q = want[0]
    last.k_pages, last.k_scale, last.v_pages, last.v_scale, last.page_table, last.kv_len = want[2]
    last.own = [l + steps for l in own]
    last.slots = [b.slots[0]] + [torch.cat([sl, torch.stack([x[i] for x in slots]).cpu()])
                                 for i, sl in enumerate(b.slots[1:])]
    last.check(outs[-1], None, D ** -0.5)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        decode(live, outs, ws, lambda: None)
    for k in range(4):
        for x in qkv:
            x.mul_(-0.5 if k % 2 else -2.0)
        want = apart()
        for x, y in zip(live, start):
            x.copy_(y)
        ws.fill_(255)
        graph.replay()
        same(live, outs, want)


# ----------------------------------------------------------- what is written --

@pytest.mark.parametrize("path", ALL_PATHS)
@pytest.mark.parametrize("max_q", (2, 9))  # cuts the prompt of 9, or fits
@pytest.mark.parametrize("P,own", [(0, [20, 40, 8]), (90, [20, 40, 8]), (3000, [700, 40, 3000]), (700, [0, 0, 0])])
def test_nothing_else_is_written(P, own, max_q, path):
    """Outputs, log-sum-exps and workspace between guards: rows outside the
    batch and everything around the buffers keep their bytes."""
    D, Hq, Hkv, ps = 128, 8, 2, 16
    b = Batch([3, 9, 2], own, P, Hq, Hkv, D, ps, seed=P, first_row=2, extra_rows=3)
    table = b.page_table if b.page_table.shape[1] else None
    pages = 0 if table is None else table.shape[1]
    need = mfp8.mfp8_prefix_attention_workspace_bytes(b.T, b.B, max_q, Hq, Hkv, D, P, pages, ps)
    sizes = (b.T * Hq * D * 2, b.T * Hq * 4, need)
    bufs = [torch.full((n + 8192,), 0xa5, dtype=torch.uint8, device="cuda") for n in sizes]
    q = b.q.contiguous()
    status = mfp8.mfp8_prefix_attention(
        q.data_ptr(), Hq * D, b.T, Hq, Hkv, D, b.q_start.data_ptr(), b.kv_len.data_ptr(), b.B, max_q,
        b.k_pages.data_ptr(), b.k_scale.data_ptr(), b.v_pages.data_ptr(), b.v_scale.data_ptr(), b.k_pages.shape[0], ps,
        b.prefix_pages.data_ptr() if P else None, P, None if table is None else table.data_ptr(), pages, pages, 0.1,
        bufs[0].data_ptr() + 4096, bufs[1].data_ptr() + 4096, bufs[2].data_ptr() + 4096, need, path)
    assert status == mfp8.OK
    assert mfp8.device_status() == (mfp8.ERR_INDEX if max_q == 2 else mfp8.OK)
    for x, n in zip(bufs, sizes):
        assert (x[:4096] == 0xa5).all() and (x[4096 + n:] == 0xa5).all()
    for x, row in zip(bufs[:2], (Hq * D * 2, Hq * 4)):
        rows = x[4096:4096 + b.T * row].view(b.T, row)
        assert (rows[:2] == 0xa5).all() and (rows[-3:] == 0xa5).all()
        assert not (rows[2:-3] == 0xa5).all(-1).any()
    if max_q == 9:
        b.check(bufs[0][4096:4096 + sizes[0]].view(torch.bfloat16).view(b.T, Hq, D),
                bufs[1][4096:4096 + sizes[1]].view(torch.float32).view(b.T, Hq), 0.1)
