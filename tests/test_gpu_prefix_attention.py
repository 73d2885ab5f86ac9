"""Attention over a shared prefix on the GPU against its 64-bit form."""
import math

import pytest
import torch

from fp8_w8a8_dynamic_b200 import mfp8
from serving_ref import Batch

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def status_stays_clean():
    yield
    assert mfp8.device_status() == mfp8.OK


def run(b, scale=None, **kw):
    scale = scale or b.D ** -0.5
    out, lse = mfp8.prefix_attention(*b.args(), scale=scale, want_lse=True, **kw)
    return out, lse, scale


#        n, own, P, Hq, Hkv, D, ps
CASES = {
    "one token": ([1], [1], 0, 1, 1, 128, 8),
    "one token of prefix": ([1], [0], 1, 4, 1, 64, 8),
    "nothing to see": ([1, 1], [0, 0], 0, 4, 2, 128, 16),
    "some see nothing": ([1, 1, 1], [0, 5, 0], 0, 8, 2, 128, 16),
    "decode": ([1] * 4, [1, 16, 17, 130], 300, 32, 8, 128, 16),
    "decode narrow heads": ([1] * 5, [3, 64, 65, 0, 200], 129, 12, 4, 64, 32),
    "decode mha": ([1] * 3, [31, 32, 33], 95, 6, 6, 128, 8),
    "decode mqa 16": ([1] * 3, [7, 300, 1], 64, 16, 1, 128, 64),
    "group of 7": ([1] * 9, [5] * 9, 500, 14, 2, 128, 256),
    "many query rows per head": ([1] * 70, [9] * 70, 260, 8, 2, 64, 16),
    "no prefix": ([1] * 6, [1, 2, 255, 256, 257, 700], 0, 8, 2, 128, 64),
    "prefix alone": ([1] * 6, [0] * 6, 777, 8, 2, 128, 64),
    "prompts": ([5, 1, 0, 37, 128], [9, 1, 0, 37, 130], 100, 8, 2, 128, 16),
    "prompts without prefix": ([17, 33], [17, 50], 0, 4, 4, 64, 8),
    "more new tokens than cached": ([6, 3], [2, 0], 0, 4, 2, 128, 8),
    "more new tokens than cached, behind a prefix": ([6, 3], [2, 0], 20, 4, 2, 64, 8),
    "one long sequence": ([1], [9000], 0, 32, 8, 128, 64),
    "long prefix": ([1, 1], [70, 1], 20001, 8, 2, 128, 128),
    "tall prompt": ([300], [300], 555, 4, 1, 128, 32),
    "group of 64": ([1, 2], [40, 50], 333, 64, 1, 128, 16),
}


PATHS = (mfp8.ATTEND_ROWS, mfp8.ATTEND_TALL)


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("name", CASES)
def test_against_64_bits(name, path):
    b = Batch(*CASES[name], seed=len(name))
    out, lse, scale = run(b, path=path)
    b.check(out, lse, scale, name)
    plain = mfp8.prefix_attention(*b.args(), path=path)
    assert torch.equal(plain, out)  # the same bits again, without lse and with the default scale


def test_the_choice_by_size():
    """Sizes on both sides of the border, each part's kernel its own: a large
    batch's prefix with few own tokens, long prompts, and a small batch."""
    for n, own, P in (([1] * 150, [9] * 150, 1500), ([400, 1, 333], [700, 5, 333], 900), ([1] * 3, [30] * 3, 800)):
        b = Batch(n, own, P, 16, 4, 128, 32, seed=P)
        out, lse, scale = run(b)
        b.check(out, lse, scale, str(P))


def test_strided_queries_rows_outside_and_workspace_contents():
    b = Batch([1, 3, 2], [20, 40, 2], 90, 8, 4, 128, 16, seed=3, extra_rows=4, first_row=2, ldq_extra=8 * 24)
    assert not b.q.is_contiguous()
    nbytes = mfp8.mfp8_prefix_attention_workspace_bytes(b.T, b.B, b.max_q, 8, 4, 128, 90, b.page_table.shape[1], 16)
    out = torch.full((b.T, 8, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.full((nbytes,), 0xff, dtype=torch.uint8, device="cuda")  # NaNs
    got, lse, scale = run(b, out=out, workspace=ws)
    assert got is out
    b.check(out, lse, scale)
    assert (out[:2] == 7.0).all() and (out[-4:] == 7.0).all()


def test_wide_table_strided_rows_and_longer_max_q():
    b = Batch([1, 2], [33, 70], 50, 8, 2, 64, 8, seed=4, max_pages=40)
    wide = torch.full((2, 64), -1, dtype=torch.int32, device="cuda")
    wide[:, :40] = b.page_table
    b.page_table = wide[:, :40]
    b.max_q = 9
    out, lse, scale = run(b)
    b.check(out, lse, scale)


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("k_gain,scale", [(30.0, 0.3), (1e-3, 1.0), (1.0, 1e-6), (8.0, 2.0)])
def test_peaked_and_flat_rows(k_gain, scale, path):
    b = Batch([1, 1, 4], [100, 3, 80], 700, 8, 2, 128, 16, seed=5, k_gain=k_gain)
    out, lse, _ = run(b, scale, path=path)
    b.check(out, lse, scale)


@pytest.mark.parametrize("path", PATHS)
def test_value_scales_far_apart_and_zero_rows(path):
    b = Batch([1, 2], [60, 40], 400, 8, 2, 128, 16, seed=6, v_spread=4.0)
    for sl in b.slots:  # rows of zeros take FLT_MIN as their scale
        z = sl[::5].cuda()
        b.v_pages[z // 16, :, z % 16] = 0
        b.v_scale[z // 16, :, z % 16] = 2.0 ** -126
        z = sl[1::7].cuda()
        b.k_pages[z // 16, :, z % 16] = 0
        b.k_scale[z // 16, :, z % 16] = 2.0 ** -126
    out, lse, scale = run(b, path=path)
    b.check(out, lse, scale)


@pytest.mark.parametrize("path", PATHS)
def test_all_values_zero_or_tiny(path):
    b = Batch([1, 1], [9, 30], 40, 4, 2, 64, 8, seed=7)
    for sl in b.slots:
        s = sl.cuda()
        b.v_scale[s // 8, :, s % 8] *= 2.0 ** -80
    out, lse, scale = run(b, path=path)
    b.check(out, lse, scale)
    b.v_pages.zero_()
    out, lse, scale = run(b, path=path)
    assert (out == 0).all()


@pytest.mark.parametrize("path", PATHS)
def test_query_magnitudes(path):
    b = Batch([1, 1, 1, 1], [9, 30, 2, 44], 120, 4, 2, 128, 8, seed=8)
    b.q[0] *= 2.0 ** -100
    b.q[1] = 0
    b.q[2, :, 5] = 3.0e4  # one element far above the others
    b.q[3] *= 2.0 ** -20
    out, lse, scale = run(b, path=path)
    b.check(out, lse, scale)


@pytest.mark.parametrize("path", PATHS)
def test_offsets_past_32_bits(path):
    H, ps, D = 8, 256, 128
    b = Batch([1, 1], [300, 30], 700, 16, H, D, ps, seed=9, wide_pool=2 ** 32 // (H * ps * D) + 9)
    out, lse, scale = run(b, path=path)
    b.check(out, lse, scale)


def test_other_stream():
    b = Batch([1] * 4, [5, 50, 70, 9], 300, 8, 2, 128, 16, seed=10)
    want, lse, scale = run(b)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got, lse2, _ = run(b, stream=side)
    side.synchronize()
    assert torch.equal(got, want) and torch.equal(lse, lse2)


@pytest.mark.parametrize("path", PATHS)
def test_graph_replayed_with_new_lengths_and_a_shared_workspace(path):
    """Two captured graphs share a workspace and are replayed in turn; a replay
    follows lengths and pages that changed since the capture."""
    b = Batch([1] * 4, [40, 64, 1, 17], 300, 8, 2, 128, 16, seed=11, max_pages=8)
    c = Batch([1] * 3, [70, 3, 100], 200, 8, 2, 128, 16, seed=12, max_pages=8)
    size = [mfp8.mfp8_prefix_attention_workspace_bytes(x.T, x.B, 1, 8, 2, 128, x.P, 8, 16) for x in (b, c)]
    ws = torch.empty((max(size),), dtype=torch.uint8, device="cuda")
    got = []
    for x in (b, c):
        run(x, workspace=ws, path=path)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out, lse, scale = run(x, workspace=ws, path=path)
        got.append((graph, out, lse))
    for _ in range(2):
        for graph, _, _ in got:
            graph.replay()
    b.check(got[0][1], got[0][2], scale)
    c.check(got[1][1], got[1][2], scale)
    # shorter and empty sequences in the same buffers
    b.own = [33, 0, 1, 16]
    b.slots = [b.slots[0]] + [s[:l] for s, l in zip(b.slots[1:], b.own)]
    b.kv_len.copy_(torch.tensor(b.own, dtype=torch.int32))
    got[0][0].replay()
    b.check(got[0][1], got[0][2], scale)


@pytest.mark.parametrize("n,own,P,Hq", [
    ([1] * 80, [9, 700] * 40, 6000, 8),  # tall prefix, own tokens in 8-row tiles beside it
    ([1] * 80, [9, 700] * 40, 1500, 32),  # ... in 16-row tiles
    ([400, 1, 200], [700, 5, 200], 24, 8),  # tall own tokens, the prefix beside them
])
def test_layers_in_a_row_with_both_kernels(n, own, P, Hq):
    """Calls whose two kernels run beside each other, each reading the output
    of the one before and all with one workspace: the bits of the same calls
    with a synchronisation and fresh memory between them, eager and replayed."""
    b = Batch(n, own, P, Hq, 2, 128, 64, seed=P)
    size = mfp8.mfp8_prefix_attention_workspace_bytes(b.T, b.B, b.max_q, Hq, 2, 128, P, b.page_table.shape[1], 64)
    ws = torch.zeros((size,), dtype=torch.uint8, device="cuda")
    rest = b.args()[1:]
    first = b.args()[0].contiguous()
    bufs = [torch.zeros_like(first) for _ in range(6)]

    def layers(x):
        for y in bufs:
            mfp8.prefix_attention(x, *rest, workspace=ws, out=y)
            x = y

    def separate(x):
        ys = []
        for _ in bufs:
            x = mfp8.prefix_attention(x, *rest, out=torch.zeros_like(first))
            torch.cuda.synchronize()
            ys.append(x)
        return ys

    out, lse, scale = run(b)
    b.check(out, lse, scale)
    want = separate(first)
    layers(first)
    assert all(torch.equal(x, y) for x, y in zip(bufs, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layers(first)
    for k in range(3):
        first.mul_(-0.5)
        want = separate(first)
        ws.fill_(255)
        graph.replay()
        assert all(torch.equal(x, y) for x, y in zip(bufs, want)), k


def test_two_streams_at_once_with_both_kernels():
    batches = [Batch([1] * 80, [9, 700] * 40, 6000, 8, 2, 128, 64, seed=21),
               Batch([1] * 70, [300, 40] * 35, 3000, 16, 4, 64, 32, seed=22)]
    want = [run(b)[0] for b in batches]
    for b, w in zip(batches, want):
        b.check(*run(b))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in batches]
    got = [[], []]
    for _ in range(6):
        for i, s in enumerate(streams):
            got[i].append(run(batches[i], stream=s)[0])
    torch.cuda.synchronize()
    for w, outs in zip(want, got):
        assert all(torch.equal(w, o) for o in outs)


@pytest.mark.parametrize("path", (mfp8.ATTEND_AUTO,) + PATHS)
def test_a_row_with_nan_leaves_the_others_alone(path):
    def run(x):
        return mfp8.prefix_attention(*x.args(), want_lse=True, path=path) + (x.D ** -0.5,)

    b = Batch([1] * 80, [9, 700] * 40, 6000, 8, 2, 128, 64, seed=23)
    want, _, _ = run(b)
    b.q[17].fill_(math.nan)
    b.q[40, 3] = math.inf
    got, lse, _ = run(b)
    assert got[17].isnan().all() and got[40, 3].isnan().all() and lse[17].isnan().all()
    keep = torch.ones(80, 8, dtype=torch.bool, device="cuda")
    keep[17] = False
    keep[40, 3] = False
    assert torch.equal(got[keep], want[keep])


@pytest.mark.parametrize("path", PATHS)
def test_lengths_and_pages_out_of_range_are_cut_and_reported(path):
    def run(x):
        return mfp8.prefix_attention(*x.args(), want_lse=True, path=path) + (x.D ** -0.5,)

    b = Batch([1, 1], [20, 20], 64, 4, 2, 64, 16, seed=13)
    want, lse, scale = run(b)
    table = b.page_table.clone()
    b.page_table[0, 1] = 10 ** 6
    out, _, _ = run(b)
    assert mfp8.device_status() == mfp8.ERR_INDEX
    assert torch.equal(out[1], want[1])
    b.page_table.copy_(table)
    b.prefix_pages[2] = -1
    run(b)
    assert mfp8.device_status() == mfp8.ERR_INDEX
    b = Batch([1, 1], [20, 32], 64, 4, 2, 64, 16, seed=13)
    want, _, _ = run(b)
    b.kv_len[1] = 1000  # the table holds 32 tokens
    out, _, _ = run(b)
    assert mfp8.device_status() == mfp8.ERR_INDEX
    assert torch.equal(out, want)
    b.kv_len[1] = 32
    b.q_start[2] = 7  # past the last token
    out, _, _ = run(b)
    assert mfp8.device_status() == mfp8.ERR_INDEX
    assert torch.equal(out, want)


def test_the_layer_between_the_projections():
    """qkv_proj -> rope_kv_store -> prefix_attention -> o_proj over two decode
    steps behind a stored prefix, against the same chain of its parts."""
    Hq, Hkv, D, ps, hidden, B, P = 8, 2, 64, 16, 256, 3, 40
    g = torch.Generator(device="cuda").manual_seed(1)

    def rnd(*shape, std=1.0):
        return (torch.randn(shape, generator=g, device="cuda") * std).to(torch.bfloat16)

    wqkv = mfp8.quantize_weight(rnd((Hq + 2 * Hkv) * D, hidden, std=0.1))
    wo = mfp8.quantize_weight(rnd(hidden, Hq * D, std=0.1))
    freq, _ = mfp8.rope_frequencies(D, 10000.0)
    n_pages = 3 + 2 * B
    kp = torch.zeros((n_pages, Hkv, ps, D), dtype=torch.uint8, device="cuda")
    vp, ks = torch.zeros_like(kp), torch.ones((n_pages, Hkv, ps), device="cuda")
    vs = torch.ones_like(ks)
    prefix_pages = torch.tensor([4, 0, 8], dtype=torch.int32, device="cuda")
    table = torch.tensor([[1, 2], [3, 5], [6, 7]], dtype=torch.int32, device="cuda")

    def step(x, pos, slot, q_start, kv_len, prefix_len):
        qkv = mfp8.linear(x, *wqkv)
        q = mfp8.rope_kv_store(qkv, Hq, pos, freq, slot, kp, ks, vp, vs)
        o = mfp8.prefix_attention(q, q_start, kv_len, table, prefix_pages, prefix_len, kp, ks, vp, vs, max_q=1)
        return qkv, q, o, mfp8.linear(o.flatten(1), *wo)

    def i32(v):
        return torch.tensor(v, dtype=torch.int32, device="cuda")

    # the prefix itself: stored as one prompt
    x = rnd(P, hidden)
    t = torch.arange(P, device="cuda")
    slot = prefix_pages.long()[t // ps] * ps + t % ps
    mfp8.rope_kv_store(mfp8.linear(x, *wqkv), Hq, t.int(), freq, slot, kp, ks, vp, vs)
    pk, pv = mfp8.kv_page_read(kp, ks, slot), mfp8.kv_page_read(vp, vs, slot)
    own_k, own_v = [], []
    for s in range(18):
        x = rnd(B, hidden)
        slot = table.long()[:, s // ps] * ps + s % ps
        pos = i32([P + s] * B)
        qkv, q, o, y = step(x, pos, slot, i32(list(range(B + 1))), i32([s + 1] * B), P)
        assert torch.equal(q, mfp8.rope(qkv.view(B, -1, D)[:, :Hq], pos, freq))
        own_k.append(mfp8.kv_page_read(kp, ks, slot))
        own_v.append(mfp8.kv_page_read(vp, vs, slot))
        assert torch.equal(y, mfp8.linear(o.flatten(1), *wo))
        # read back to bf16 the cache is off by 2^-8 relative per element: a logit by 2^-8 sum |q k|, and so a
        # weight by twice that; a value by 2^-8; the output's rounding 2^-8
        for b in range(B):
            k = torch.cat([pk] + [v[b:b + 1] for v in own_k]).double()
            v = torch.cat([pv] + [v[b:b + 1] for v in own_v]).double()
            qb = q[b].double().view(Hkv, Hq // Hkv, D)
            z = torch.einsum("hgd,thd->hgt", qb, k) / math.sqrt(D)
            a = torch.einsum("hgd,thd->hgt", qb.abs(), k.abs()).amax(-1) / math.sqrt(D)
            p = torch.softmax(z, -1)
            ref = torch.einsum("hgt,thd->hgd", p, v)
            size = torch.einsum("hgt,thd->hgd", p, v.abs())
            tol = ref.abs() * 2.0 ** -8 + size * (2.0 ** -8 + 2.0 ** -11 + 2 * a[..., None] * (2.0 ** -8 + 2.0 ** -15))
            assert ((o[b].double().view_as(ref) - ref).abs() <= tol).all()
