"""The operators between qkv_proj and o_proj: rotary positions, the paged FP8
e4m3 KV cache (written, read back) and attention for a batch that shares a
prefix.  Each is given in its plain form (elementary torch operations) and as
the framework's call; cases, inputs, least work and 64-bit values are below.

Shapes follow the language model the library serves (32 query and 8 KV heads
of 128) and generic ones beside it."""
import math
import random

import torch

own = False

FLT_MIN = 2.0 ** -126


# ------------------------------------------------------------------ cases --

def listed():
    return [
        # one decode step of 8 sequences: the query heads alone
        dict(name="rope decode", op="rope", T=8, H=32, D=128, rot=128, layout="half", axes=1, factor=1.0,
             far=32768, strided=True),
        # a long prefill with three position axes (frame, row, column), rotated straight out of the packed qkv
        dict(name="rope prefill 3 axes", op="rope", T=16384, H=32, D=128, rot=128, layout="half", axes=3,
             factor=1.0, far=262144, strided=True),
        # odd length, a quarter of a narrower head, interleaved pairs, frequencies stretched 8-fold for long contexts
        dict(name="rope partial interleaved", op="rope", T=5003, H=20, D=96, rot=32, layout="interleaved", axes=1,
             factor=8.0, far=1000000, strided=False),
        # one decode step of 16 sequences: rotate, quantize, write into the pages
        dict(name="store decode", op="store", T=16, Hq=32, Hkv=8, D=128, rot=128, layout="half", axes=1, ps=16,
             far=32768, skip=0.0),
        # a prefill chunk behind qkv_proj
        dict(name="store prefill", op="store", T=16384, Hq=32, Hkv=8, D=128, rot=128, layout="half", axes=3, ps=64,
             far=262144, skip=0.0),
        # a padded batch of odd length, as many KV heads as query heads, narrow heads
        dict(name="store padded mha", op="store", T=1999, Hq=12, Hkv=12, D=64, rot=32, layout="interleaved", axes=1,
             ps=32, far=4096, skip=0.2),
        # a layer's keys of a long context gathered back to bf16
        dict(name="read long", op="read", T=65536, H=8, D=128, ps=64),
        # the same for a short one
        dict(name="read short", op="read", T=333, H=8, D=128, ps=16),
        # decode of 4 sequences behind a system prompt
        dict(name="attend small batch", op="attend", B=4, qlo=1, qhi=1, Hq=32, Hkv=8, D=128, ps=16, prefix=1000,
             lo=1, hi=200),
        # decode of 64 sequences behind a long document
        dict(name="attend decode 64", op="attend", B=64, qlo=1, qhi=1, Hq=32, Hkv=8, D=128, ps=64, prefix=32768,
             lo=16, hi=1024),
        # decode of 256 sequences with long answers of their own
        dict(name="attend decode 256", op="attend", B=256, qlo=1, qhi=1, Hq=32, Hkv=8, D=128, ps=64, prefix=8192,
             lo=128, hi=4096),
        # user prompts appended to a shared document: many query tokens per sequence, ragged
        dict(name="attend prompts", op="attend", B=7, qlo=1, qhi=700, Hq=32, Hkv=8, D=128, ps=32, prefix=10007,
             lo=0, hi=900),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "store", "read", "attend", "attend"])
    if op == "rope":
        D = rng.choice([64, 96, 128, 192, 256])
        rot = rng.choice([r for r in range(16, D + 1, 16)])
        H = rng.choice([1, 5, 8, 20, 32, 40])
        return dict(op=op, T=min(_log(rng, 1, 16384), 16384 * 32 * 128 // (H * D)), H=H, D=D, rot=rot,
                    layout=rng.choice(["half", "interleaved"]), axes=rng.choice([1, 1, 2, 3]),
                    factor=rng.choice([1.0, 4.0, 8.0]), far=_log(rng, 1000, 1000000), strided=rng.random() < 0.5)
    if op == "store":
        D = rng.choice([64, 96, 128, 256])
        Hkv = rng.choice([1, 2, 4, 8])
        Hq = Hkv * rng.choice([1, 2, 3, 4, 8])
        T = min(_log(rng, 1, 16384), 16384 * 48 * 128 // ((Hq + 2 * Hkv) * D))
        return dict(op=op, T=T, Hq=Hq, Hkv=Hkv, D=D, rot=rng.choice([r for r in range(16, D + 1, 16)]),
                    layout=rng.choice(["half", "interleaved"]), axes=rng.choice([1, 1, 3]),
                    ps=rng.choice([8, 16, 32, 64, 128]), far=_log(rng, 1000, 262144),
                    skip=rng.choice([0.0, 0.0, 0.1]))
    if op == "read":
        D = rng.choice([64, 96, 128, 256])
        H = rng.choice([1, 2, 4, 8, 16])
        return dict(op=op, T=min(_log(rng, 1, 65536), 65536 * 8 * 128 // (H * D)), H=H, D=D,
                    ps=rng.choice([8, 16, 32, 64, 128, 256]))
    Hkv, G = rng.choice([(8, 4), (8, 4), (4, 8), (8, 1), (2, 7), (1, 16)])
    D = rng.choice([128, 128, 64])
    prompts = rng.random() < 0.3
    B = _log(rng, 1, 12 if prompts else 200)
    qhi = _log(rng, 2, 300) if prompts else 1
    return dict(op=op, B=B, qlo=1, qhi=qhi, Hq=Hkv * G, Hkv=Hkv, D=D, ps=rng.choice([8, 16, 32, 64, 128, 256]),
                prefix=_log(rng, 1, 10000 if prompts else 32768) if rng.random() < 0.9 else 0, lo=rng.choice([0, 1, 50]),
                hi=_log(rng, 60, 2000))


def _lens(case):
    """(new query tokens, own cached tokens) of each sequence, from the case alone."""
    r = random.Random(case["B"] * 1000003 + case["hi"] * 101 + case["qhi"])
    n = [r.randint(case["qlo"], case["qhi"]) for _ in range(case["B"])]
    # the new tokens are in the cache already, behind what was there (lo .. hi tokens)
    own_len = [r.randint(case["lo"], case["hi"]) + k - case["qlo"] for k in n]
    return n, own_len


# ----------------------------------------------------------------- inputs --

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 7919 + 17)
    return g


def _acts(shape, g):
    """Activations as qkv_proj writes them: unit normal with rare outliers, rows of unequal size."""
    x = torch.randn(shape, generator=g, device="cuda")
    x *= torch.exp(torch.rand(shape[:-1] + (1,), generator=g, device="cuda") * 2.0 - 1.0)
    x = torch.where(torch.rand(shape, generator=g, device="cuda") < 0.001, x * 20.0, x)
    return x.to(torch.bfloat16)


def _table(rot, factor, axes):
    """Frequencies theta^(-2i/rot) / factor, and the axis that each follows (interleaved over the axes)."""
    i = torch.arange(rot // 2, device="cuda", dtype=torch.float64)
    freq = (5e6 ** (-2.0 * i / rot) / factor).to(torch.float32)
    axis = (torch.arange(rot // 2, device="cuda") % axes).to(torch.uint8) if axes > 1 else None
    return freq, axis


def _quantized(x):
    """fp32 rows -> e4m3 codes (as bytes) and fp32 scales."""
    s = (x.abs().amax(-1) / 448.0).clamp_min(FLT_MIN)
    return (x / s[..., None]).to(torch.float8_e4m3fn).view(torch.uint8), s


def prepare(case, seed):
    def positions(T, axes, far, g):
        """Increasing token positions somewhere in a context of `far`; further axes are coordinates within a frame."""
        start = int(torch.randint(0, max(1, far - T), (1,), generator=g, device="cuda"))
        pos = (torch.arange(T, device="cuda") + start)[None].repeat(axes, 1)
        for a in range(1, axes):
            pos[a] = start + torch.randint(0, 64, (T,), generator=g, device="cuda")
        return pos.to(torch.int32) if axes > 1 else pos[0].to(torch.int32)

    def pool(n_pages, H, ps, D, g, spread):
        """Pages of a cache in use: codes [n_pages, H, ps, D], scales [n_pages, H, ps]."""
        codes = torch.empty((n_pages, H, ps, D), dtype=torch.uint8, device="cuda")
        scale = torch.empty((n_pages, H, ps), dtype=torch.float32, device="cuda")
        step = max(1, (1 << 26) // (H * ps * D))
        for at in range(0, n_pages, step):
            to = min(n_pages, at + step)
            x = torch.randn((to - at, H, ps, D), generator=g, device="cuda")
            x *= torch.exp(torch.randn((to - at, H, ps, 1), generator=g, device="cuda") * spread)
            codes[at:to], scale[at:to] = _quantized(x)
        return codes, scale

    g = _gen(seed)
    op = case["op"]
    s = dict(case)
    if op == "rope":
        T, H, D = case["T"], case["H"], case["D"]
        wide = _acts((T, (H + 2 * (H // 4 + 1)) if case["strided"] else H, D), g)
        s["x"] = wide[:, :H]  # the query columns of the packed projection
        s["pos"] = positions(T, case["axes"], case["far"], g)
        s["freq"], s["axis"] = _table(case["rot"], case["factor"], case["axes"])
        s["mscale"] = 1.0 if case["factor"] == 1.0 else 0.1 * math.log(case["factor"]) + 1.0
    elif op == "store":
        T, Hq, Hkv, D, ps = (case[k] for k in ("T", "Hq", "Hkv", "D", "ps"))
        s["qkv"] = _acts((T, Hq + 2 * Hkv, D), g).view(T, (Hq + 2 * Hkv) * D)
        s["pos"] = positions(T, case["axes"], case["far"], g)
        s["freq"], s["axis"] = _table(case["rot"], 1.0, case["axes"])
        n_pages = -(-T // ps) + 3
        # tokens lie page by page, the pages in any order; some rows are padding
        page = torch.randperm(n_pages, generator=g, device="cuda")
        t = torch.arange(T, device="cuda")
        slot = page[t // ps] * ps + t % ps
        drop = torch.rand(T, generator=g, device="cuda") < case["skip"]
        s["slot"] = torch.where(drop, -1, slot)
        for name in ("k", "v"):
            s[name + "_pages"] = torch.zeros((n_pages, Hkv, ps, D), dtype=torch.uint8, device="cuda")
            s[name + "_scale"] = torch.ones((n_pages, Hkv, ps), dtype=torch.float32, device="cuda")
    elif op == "read":
        T, H, D, ps = (case[k] for k in ("T", "H", "D", "ps"))
        n_pages = -(-T // ps) + 3
        s["pages"], s["scale"] = pool(n_pages, H, ps, D, g, 0.7)
        page = torch.randperm(n_pages, generator=g, device="cuda")
        t = torch.arange(T, device="cuda")
        s["slot"] = page[t // ps] * ps + t % ps
    else:
        B, Hq, Hkv, D, ps, P = (case[k] for k in ("B", "Hq", "Hkv", "D", "ps", "prefix"))
        n, own_len = _lens(case)
        most = max(1, -(-max(own_len) // ps))
        n_prefix = -(-P // ps)
        n_pages = n_prefix + B * most + 5
        s["k_pages"], s["k_scale"] = pool(n_pages, Hkv, ps, D, g, 0.3)
        s["v_pages"], s["v_scale"] = pool(n_pages, Hkv, ps, D, g, 0.7)
        order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
        s["prefix_pages"] = order[:n_prefix].contiguous()
        s["page_table"] = order[n_prefix:n_prefix + B * most].view(B, most).contiguous()
        T = sum(n)
        s["q"] = (torch.randn((T, Hq, D), generator=g, device="cuda") * 1.5).to(torch.bfloat16)
        start = [0]
        for k in n:
            start.append(start[-1] + k)
        s["q_start"] = torch.tensor(start, dtype=torch.int32, device="cuda")
        s["kv_len"] = torch.tensor(own_len, dtype=torch.int32, device="cuda")
        s["max_q"], s["max_len"], s["softmax_scale"] = max(n), max(own_len), 1.0 / math.sqrt(D)
        # where token t of the batch sits: its sequence, and its place among that sequence's new tokens
        s["of"] = torch.repeat_interleave(torch.arange(B, device="cuda"), torch.tensor(n, device="cuda"))
        s["at"] = torch.arange(T, device="cuda") - s["q_start"].long()[s["of"]]
    return s


# ------------------------------------------------------------ plain forms --

def _plain_cos_sin(pos, freq, axis, mscale):
    """fp32 cosines and sines [T, rot/2]; the angles in 64 bits, which far positions need."""
    p = pos.double()
    p = p[axis.long()].t() if axis is not None else p[:, None]
    a = p * freq.double()
    return (a.cos() * mscale).float(), (a.sin() * mscale).float()


def _plain_rope(x, pos, freq, axis, layout, mscale):
    """x [T, H, D] bf16 -> rotated bf16."""
    rot = 2 * freq.numel()
    c, s = (v[:, None] for v in _plain_cos_sin(pos, freq, axis, mscale))
    xf = x.float()
    y = xf.clone()
    if layout == "half":
        a, b = xf[..., :rot // 2], xf[..., rot // 2:rot]
        y[..., :rot // 2] = a * c - b * s
        y[..., rot // 2:rot] = b * c + a * s
    else:
        a, b = xf[..., 0:rot:2], xf[..., 1:rot:2]
        y[..., 0:rot:2] = a * c - b * s
        y[..., 1:rot:2] = b * c + a * s
    return y.to(torch.bfloat16)


def _plain_store(x, slot, pages, scale):
    """bf16 rows [T, H, D] into their slots, quantized; rows with a negative slot are left out."""
    ps = pages.shape[2]
    live = slot >= 0
    x, slot = x[live], slot[live]
    codes, s = _quantized(x.float())
    pages[slot // ps, :, slot % ps] = codes
    scale[slot // ps, :, slot % ps] = s


def _plain_values(pages, scale):
    return pages.view(torch.float8_e4m3fn).float() * scale[..., None]


def _plain_gather(pages, scale, table):
    """fp32 values [..., tokens, H, D] of the pages in `table` [..., n]."""
    v = _plain_values(pages[table], scale[table])  # [..., n, H, ps, D]
    v = v.transpose(-3, -2)
    return v.reshape(table.shape[:-1] + (table.shape[-1] * v.shape[-3],) + v.shape[-2:])


def _plain_attend(s):
    Hq, Hkv, D, P, B = s["Hq"], s["Hkv"], s["D"], s["prefix"], s["B"]
    G, n, L = Hq // Hkv, s["max_q"], max(s["max_len"], 1)
    T = s["q"].shape[0]
    of, at = s["of"], s["at"]
    # queries [Hkv, T, G, D]
    q = (s["q"].float() * s["softmax_scale"]).view(T, Hkv, G, D).transpose(0, 1)
    neg = torch.tensor(-math.inf, device="cuda")
    # the shared prefix, once for every query
    pk = _plain_gather(s["k_pages"], s["k_scale"], s["prefix_pages"].long())[:P].transpose(0, 1)
    pv = _plain_gather(s["v_pages"], s["v_scale"], s["prefix_pages"].long())[:P].transpose(0, 1)
    sp = torch.matmul(q.reshape(Hkv, T * G, D), pk.transpose(1, 2)).view(Hkv, T, G, P)
    # each sequence's own tokens, padded to the longest
    ok = _plain_gather(s["k_pages"], s["k_scale"], s["page_table"].long())[:, :L].permute(0, 2, 3, 1)
    ov = _plain_gather(s["v_pages"], s["v_scale"], s["page_table"].long())[:, :L].permute(0, 2, 1, 3)
    padded = torch.zeros((B, n, Hkv, G, D), device="cuda")
    padded[of, at] = q.transpose(0, 1)
    so = torch.matmul(padded.permute(0, 2, 1, 3, 4).reshape(B, Hkv, n * G, D), ok).view(B, Hkv, n, G, L)
    count = s["q_start"].long().diff()
    limit = s["kv_len"].long()[:, None] - count[:, None] + torch.arange(n, device="cuda")[None] + 1
    seen = torch.arange(L, device="cuda")[None, None] < limit[..., None]  # [B, n, L]
    so = torch.where(seen[:, None, :, None], so, neg)
    mp = sp.amax(-1) if P else torch.full((Hkv, T, G), -math.inf, device="cuda")
    mo = so.amax(-1).permute(0, 2, 1, 3)[of, at].transpose(0, 1)
    m = torch.maximum(mp, mo)
    fine = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    ep = torch.exp(sp - fine[..., None])
    padded_m = torch.zeros((B, n, Hkv, G), device="cuda")
    padded_m[of, at] = fine.transpose(0, 1)
    eo = torch.exp(so - padded_m.permute(0, 2, 1, 3)[..., None])
    total = ep.sum(-1) + eo.sum(-1).permute(0, 2, 1, 3)[of, at].transpose(0, 1)
    out = torch.matmul(ep.view(Hkv, T * G, P), pv).view(Hkv, T, G, D)
    oo = torch.matmul(eo.view(B, Hkv, n * G, L), ov).view(B, Hkv, n, G, D)
    out = out + oo.permute(0, 2, 1, 3, 4)[of, at].transpose(0, 1)
    empty = total == 0
    out = out / torch.where(empty, torch.ones_like(total), total)[..., None]
    lse = torch.where(empty, neg, fine + torch.log(total))
    return (out.transpose(0, 1).reshape(T, Hq, D).to(torch.bfloat16),
            lse.transpose(0, 1).reshape(T, Hq).contiguous())


def run(state):
    s = state
    op = s["op"]
    if own:
        from fp8_w8a8_dynamic_b200 import mfp8
        layout = mfp8.ROPE_HALF if s.get("layout") == "half" else mfp8.ROPE_INTERLEAVED
        if op == "rope":
            return mfp8.rope(s["x"], s["pos"], s["freq"], axis=s["axis"], layout=layout, mscale=s["mscale"])
        if op == "store":
            q = mfp8.rope_kv_store(s["qkv"], s["Hq"], s["pos"], s["freq"], s["slot"], s["k_pages"], s["k_scale"],
                                   s["v_pages"], s["v_scale"], axis=s["axis"], layout=layout)
            return [q, s["k_pages"].view(torch.float8_e4m3fn), s["k_scale"],
                    s["v_pages"].view(torch.float8_e4m3fn), s["v_scale"]]
        if op == "read":
            return mfp8.kv_page_read(s["pages"], s["scale"], s["slot"])
        return mfp8.prefix_attention(s["q"], s["q_start"], s["kv_len"], s["page_table"], s["prefix_pages"],
                                     s["prefix"], s["k_pages"], s["k_scale"], s["v_pages"], s["v_scale"],
                                     max_q=s["max_q"], scale=s["softmax_scale"], want_lse=True)
    if op == "rope":
        return _plain_rope(s["x"], s["pos"], s["freq"], s["axis"], s["layout"], s["mscale"])
    if op == "store":
        T, Hq, Hkv, D = s["T"], s["Hq"], s["Hkv"], s["D"]
        x = s["qkv"].view(T, Hq + 2 * Hkv, D)
        r = _plain_rope(x[:, :Hq + Hkv], s["pos"], s["freq"], s["axis"], s["layout"], 1.0)
        _plain_store(r[:, Hq:], s["slot"], s["k_pages"], s["k_scale"])
        _plain_store(x[:, Hq + Hkv:], s["slot"], s["v_pages"], s["v_scale"])
        return [r[:, :Hq].contiguous(), s["k_pages"].view(torch.float8_e4m3fn), s["k_scale"],
                s["v_pages"].view(torch.float8_e4m3fn), s["v_scale"]]
    if op == "read":
        ps, slot = s["ps"], s["slot"]
        page, at = slot // ps, slot % ps
        return _plain_values(s["pages"][page, :, at], s["scale"][page, :, at]).to(torch.bfloat16)
    return _plain_attend(s)


# -------------------------------------------------------------- least work --

def work(case):
    op = case["op"]
    if op == "rope":
        n = case["T"] * case["H"] * case["D"]
        return {"bytes": 4 * n + 4 * case["T"] * case["axes"] + 2 * case["rot"],
                "flops": 6.0 * case["T"] * case["H"] * case["rot"] // 2}
    if op == "store":
        T, Hq, Hkv, D = (case[k] for k in ("T", "Hq", "Hkv", "D"))
        return {"bytes": T * (2 * (Hq + 2 * Hkv) * D + 2 * Hq * D + 2 * Hkv * (D + 4) + 4 * case["axes"] + 8),
                "flops": 3.0 * T * (Hq + Hkv) * case["rot"] + 4.0 * T * Hkv * D}
    if op == "read":
        T, H, D = case["T"], case["H"], case["D"]
        return {"bytes": T * H * (3 * D + 4) + 8 * T, "flops": float(T * H * D)}
    n, own_len = _lens(case)
    T, Hq, Hkv, D = sum(n), case["Hq"], case["Hkv"], case["D"]
    kv = case["prefix"] + sum(own_len)
    pairs = T * case["prefix"] + sum(sum(max(0, l - k + j + 1) for j in range(k)) for k, l in zip(n, own_len))
    return {"bytes": kv * Hkv * 2 * (D + 4) + T * Hq * (4 * D + 4), "flops": 4.0 * D * Hq * pairs}


# ----------------------------------------------------------- 64-bit values --

def exact(case, seed):
    def rotated(x, pos, freq, axis, layout, mscale):
        T, H, D = x.shape
        rot = 2 * freq.numel()
        y = x.double().clone()
        for i in range(rot // 2):
            p = pos if pos.dim() == 1 else pos[int(axis[i])]
            a = p.double() * float(freq[i])
            c, s = (mscale * torch.cos(a))[:, None], (mscale * torch.sin(a))[:, None]
            u, w = (i, i + rot // 2) if layout == "half" else (2 * i, 2 * i + 1)
            y[:, :, u] = x[:, :, u].double() * c - x[:, :, w].double() * s
            y[:, :, w] = x[:, :, w].double() * c + x[:, :, u].double() * s
        return y

    def e4m3_grid():
        """The value of each of the 256 codes, from the format: 4 exponent bits (bias 7), 3 mantissa bits."""
        v = []
        for b in range(256):
            e, m = (b >> 3) & 15, b & 7
            x = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
            v.append((-x if b & 128 else x) if b & 127 != 127 else math.nan)
        return torch.tensor(v, dtype=torch.float64, device="cuda")

    s = prepare(case, seed)
    op = case["op"]
    if op == "rope":
        return rotated(s["x"], s["pos"], s["freq"], s["axis"], s["layout"], s["mscale"])
    if op == "store":
        # the codes are those of rows rounded to bf16: the queries and the scales have 64-bit values of their own
        T, Hq, Hkv, D, ps = (case[k] for k in ("T", "Hq", "Hkv", "D", "ps"))
        x = s["qkv"].view(T, Hq + 2 * Hkv, D)
        r = rotated(x[:, :Hq + Hkv], s["pos"], s["freq"], s["axis"], s["layout"], 1.0)
        live = s["slot"] >= 0
        page, at = s["slot"][live] // ps, s["slot"][live] % ps
        scales = []
        for rows in (r[live, Hq:], x[live, Hq + Hkv:].double()):
            sc = torch.ones(s["k_scale"].shape, dtype=torch.float64, device="cuda")
            sc[page, :, at] = (rows.to(torch.bfloat16).double().abs().amax(-1) / 448.0).clamp_min(FLT_MIN)
            scales.append(sc)
        return [r[:, :Hq], None, scales[0], None, scales[1]]
    grid = e4m3_grid()
    if op == "read":
        out = torch.empty((case["T"], case["H"], case["D"]), dtype=torch.float64, device="cuda")
        page, at = s["slot"] // case["ps"], s["slot"] % case["ps"]
        for h in range(case["H"]):
            out[:, h] = grid[s["pages"][page, h, at].long()] * s["scale"][page, h, at].double()[:, None]
        return out
    Hq, Hkv, D, P, ps = (case[k] for k in ("Hq", "Hkv", "D", "prefix", "ps"))
    n, own_len = _lens(case)
    if 4.0 * Hq * D * (sum(n) * P + sum(k * l for k, l in zip(n, own_len))) > 4e12:
        return None
    G, T = Hq // Hkv, sum(n)
    out = torch.zeros((T, Hq, D), dtype=torch.float64, device="cuda")
    lse = torch.full((T, Hq), -math.inf, dtype=torch.float64, device="cuda")

    def tokens(pages, scale, table, h, count):
        t = table.long()
        v = grid[pages[t, h].long()] * scale[t, h].double()[..., None]
        return v.reshape(-1, D)[:count]

    for h in range(Hkv):
        pk = tokens(s["k_pages"], s["k_scale"], s["prefix_pages"], h, P)
        pv = tokens(s["v_pages"], s["v_scale"], s["prefix_pages"], h, P)
        at = 0
        for b in range(case["B"]):
            k, l = n[b], own_len[b]
            keys = torch.cat([pk, tokens(s["k_pages"], s["k_scale"], s["page_table"][b], h, l)])
            vals = torch.cat([pv, tokens(s["v_pages"], s["v_scale"], s["page_table"][b], h, l)])
            q = s["q"][at:at + k, h * G:(h + 1) * G].double().reshape(k * G, D)
            z = (q @ keys.t() * s["softmax_scale"]).view(k, G, P + l)
            j = torch.arange(P + l, device="cuda")[None]
            i = torch.arange(k, device="cuda")[:, None]
            z = z.masked_fill((j >= P + l - k + i + 1)[:, None] & (j >= P)[:, None], -math.inf)
            w = torch.logsumexp(z, -1)
            p = torch.where(torch.isinf(w)[..., None], torch.zeros_like(z), torch.exp(z - w[..., None]))
            out[at:at + k, h * G:(h + 1) * G] = p @ vals
            lse[at:at + k, h * G:(h + 1) * G] = w
            at += k
    return [out, lse]
