"""Plain 64-bit forms of rotary positions and of attention over the paged FP8
cache, the bounds their kernels are held to, and inputs for both."""
import math

import torch

import oracle


def e4m3_table(device):
    return torch.from_numpy(oracle.e4m3_decode(torch.arange(256, dtype=torch.uint8).numpy())).to(device)


# ------------------------------------------------------------------- rope --

def rope_ref(x, pos, inv_freq, axis, layout, mscale):
    """(y, bound) in fp64: the rotated rows and how far a kernel may be off.

    Bound: bf16 rounding of the result, 2^-8 |y|; before it, cosine and sine
    rounded to fp32 and off by an ulp of the 64-bit function (2^-24 + 2^-50),
    the products (2^-24) and the sum (2^-24 |y|): at most 4 * 2^-24 of
    |x1| + |x2| times mscale; and half of bf16's smallest step."""
    x = x.double()
    rot = 2 * inv_freq.numel()
    p = pos.double()[axis.long().clamp(max=pos.shape[0] - 1)].t() if pos.dim() == 2 else pos.double()[:, None]
    a = (p * inv_freq.double())[:, None]
    c, s = a.cos() * mscale, a.sin() * mscale
    if layout == 0:
        i1 = torch.arange(rot // 2, device=x.device)
        i2 = i1 + rot // 2
    else:
        i1 = torch.arange(0, rot, 2, device=x.device)
        i2 = i1 + 1
    y, b = x.clone(), torch.zeros_like(x)
    y[..., i1] = x[..., i1] * c - x[..., i2] * s
    y[..., i2] = x[..., i2] * c + x[..., i1] * s
    size = (x[..., i1].abs() + x[..., i2].abs()) * abs(mscale)
    b[..., i1] = b[..., i2] = size * 2.0 ** -22
    b[..., :rot] += y[..., :rot].abs() * 2.0 ** -8 + 2.0 ** -134
    return y, b


# -------------------------------------------------------------- attention --

def quantized(x):
    """fp32 rows -> (codes uint8, scales fp32), by the oracle's rule in torch's own arithmetic."""
    s = (x.abs().amax(-1) / 448.0).clamp_min(2.0 ** -126)
    return (x / s[..., None]).to(torch.float8_e4m3fn).view(torch.uint8), s


class Batch:
    """A batch over a paged cache: n[b] query tokens and own[b] cached tokens
    per sequence, a prefix of P tokens, its pages scattered over the pool.
    Every place that no token occupies holds NaN codes and NaN scales."""

    def __init__(self, n, own, P, Hq, Hkv, D, ps, seed=0, device="cuda", extra_rows=0, first_row=0, spare_pages=3,
                 max_pages=None, k_gain=1.0, v_spread=0.7, ldq_extra=0, wide_pool=None):
        g = torch.Generator(device=device)
        g.manual_seed(seed)
        self.n, self.own, self.P, self.Hq, self.Hkv, self.D, self.ps = n, own, P, Hq, Hkv, D, ps
        B = len(n)
        self.B = B
        need = [-(-l // ps) for l in own]
        most = max(need + [0]) if max_pages is None else max_pages
        n_prefix = -(-P // ps)
        n_pages = n_prefix + sum(need) + spare_pages
        pool = wide_pool or n_pages
        where = torch.randperm(n_pages, generator=g, device=device).cpu().tolist()
        where = [w + pool - n_pages for w in where]
        self.k_pages = torch.full((pool, Hkv, ps, D), 0xff, dtype=torch.uint8, device=device)
        self.v_pages = torch.full((pool, Hkv, ps, D), 0x7f, dtype=torch.uint8, device=device)
        self.k_scale = torch.full((pool, Hkv, ps), math.nan, device=device)
        self.v_scale = torch.full((pool, Hkv, ps), math.nan, device=device)
        self.prefix_pages = torch.tensor(where[:n_prefix], dtype=torch.int32, device=device)
        table = torch.full((B, most), -7, dtype=torch.int32)  # entries past the end are never read
        at = n_prefix
        self.slots = [self._slots(where[:n_prefix], P)]
        for b in range(B):
            table[b, :need[b]] = torch.tensor(where[at:at + need[b]], dtype=torch.int32)
            self.slots.append(self._slots(where[at:at + need[b]], own[b]))
            at += need[b]
        self.page_table = table.to(device)
        self.kv = []
        for sl in self.slots:
            k = torch.randn((len(sl), Hkv, D), generator=g, device=device) * k_gain
            v = torch.randn((len(sl), Hkv, D), generator=g, device=device)
            v = v * torch.exp(torch.randn((len(sl), Hkv, 1), generator=g, device=device) * v_spread)
            self.put(sl, k, v)
        T = sum(n) + extra_rows + first_row
        self.T = T
        wide = torch.randn((T, Hq * D + ldq_extra), generator=g, device=device).to(torch.bfloat16)
        self.q = wide[:, :Hq * D].unflatten(1, (Hq, D))
        start = [first_row]
        for k in n:
            start.append(start[-1] + k)
        self.start = start
        self.q_start = torch.tensor(start, dtype=torch.int32, device=device)
        self.kv_len = torch.tensor(own, dtype=torch.int32, device=device)
        self.max_q = max(n + [1])

    def _slots(self, pages, count):
        return torch.tensor([pages[t // self.ps] * self.ps + t % self.ps for t in range(count)], dtype=torch.int64)

    def put(self, slots, k, v):
        if len(slots) == 0:
            return
        sl = slots.to(k.device)
        for x, pages, scale in ((k, self.k_pages, self.k_scale), (v, self.v_pages, self.v_scale)):
            codes, s = quantized(x.float())
            pages[sl // self.ps, :, sl % self.ps] = codes
            scale[sl // self.ps, :, sl % self.ps] = s

    def values(self, slots, h):
        tab = e4m3_table(self.k_pages.device)
        sl = slots.to(self.k_pages.device)
        out = []
        for pages, scale in ((self.k_pages, self.k_scale), (self.v_pages, self.v_scale)):
            out.append(tab[pages[sl // self.ps, h, sl % self.ps].long()]
                       * scale[sl // self.ps, h, sl % self.ps].double()[:, None])
        return out

    def args(self):
        return (self.q, self.q_start, self.kv_len, self.page_table if self.page_table.shape[1] else None,
                self.prefix_pages if self.P else None, self.P, self.k_pages, self.k_scale, self.v_pages, self.v_scale,
                self.max_q)

    def ref(self, scale):
        """(out, out bound, lse, lse bound) in fp64; rows outside the batch are NaN.

        With A the largest sum_d scale |q_d k_d| of a row's tokens and C the
        same with q's largest element in every place: a logit is a sum of D
        products in fp32 on the tensor cores, each addition off by at most
        2^-23 of the terms' sum (truncated), D <= 128: 2^-16 A; q itself is
        held to 2^-17 of its row's largest element (two e4m3 terms, half of
        the smallest step 2^-9 against a largest element of at least 224: 2^-17.8): 2^-17 C.  Scaling and
        exponential add 2^-22 relative and 2^-22 of the logit.  That error dz
        moves a weight by dz and the sum by dz, so a probability by 2 dz.  The
        weight, the value scale and the scaled value are each rounded to f16
        (or the weight times the value scale once): 3 * 2^-11.  The fp32 sums
        over N tokens, 16 to an addition, are off by (N / 16 + 32) 2^-22 of
        the sum of magnitudes; and the output is rounded to bf16: 2^-8."""
        dev = self.q.device
        G = self.Hq // self.Hkv
        out = torch.full((self.T, self.Hq, self.D), math.nan, dtype=torch.float64, device=dev)
        tol, lse = out.clone(), out[..., 0].clone()
        ltol = lse.clone()
        for h in range(self.Hkv):
            pk, pv = self.values(self.slots[0], h)
            for b in range(self.B):
                n, l = self.n[b], self.own[b]
                if n == 0:
                    continue
                ok, ov = self.values(self.slots[1 + b], h)
                k, v = torch.cat([pk, ok]), torch.cat([pv, ov])
                N = k.shape[0]
                r = slice(self.start[b], self.start[b] + n)
                q = self.q[r, h * G:(h + 1) * G].double().reshape(n * G, self.D)
                j = torch.arange(N, device=dev)[None]
                i = torch.arange(n, device=dev).repeat_interleave(G)[:, None]
                seen = (j < self.P) | (j < self.P + l - n + i + 1)
                z = torch.where(seen, q @ k.t() * scale, torch.tensor(-math.inf, dtype=torch.float64, device=dev))
                a = torch.where(seen, q.abs() @ k.abs().t() * scale, 0.0)
                c = torch.where(seen, q.abs().amax(-1, keepdim=True) * k.abs().sum(-1)[None] * scale, 0.0)
                none = ~seen.any(-1)
                w = torch.logsumexp(z, -1) if N else torch.full((n * G,), -math.inf, dtype=torch.float64, device=dev)
                p = torch.where(seen, torch.exp(z - torch.where(none, 0.0, w)[:, None]), 0.0)
                o = p @ v
                if N:
                    dz = (a * 2.0 ** -16 + c * 2.0 ** -17 + a * 2.0 ** -22).amax(-1) + 2.0 ** -21
                else:
                    dz = torch.zeros(n * G, dtype=torch.float64, device=dev)
                rel = 3 * 2.0 ** -11 + 2 * dz + (N / 16 + 32) * 2.0 ** -22
                t = o.abs() * 2.0 ** -8 + rel[:, None] * (p @ v.abs())
                shape = (n, G, self.D)
                out[r, h * G:(h + 1) * G] = o.view(shape)
                tol[r, h * G:(h + 1) * G] = t.view(shape)
                lse[r, h * G:(h + 1) * G] = w.view(n, G)
                ltol[r, h * G:(h + 1) * G] = (dz + 2.0 ** -22 * w.abs().nan_to_num(posinf=0.0)).view(n, G)
        return out, tol, lse, ltol

    def check(self, out, lse, scale, what=""):
        ref, tol, rl, lt = self.ref(scale)
        rows = slice(self.start[0], self.start[-1])
        o, r, t = out[rows].double(), ref[rows], tol[rows]
        assert torch.isfinite(o).all(), f"{what}: not finite"
        bad = (o - r).abs() > t
        assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} outputs off, worst "
                               f"{float(((o - r).abs() / t.clamp_min(1e-300)).max()):.2f} times the bound, first at "
                               f"{bad.nonzero()[0].tolist()}")
        if lse is not None:
            a, b, lt = lse[rows].double(), rl[rows], lt[rows]
            none = torch.isinf(b)
            assert torch.equal(none, torch.isinf(a)) and (a[none] < 0).all(), f"{what}: rows that see nothing"
            bad = (a - b).abs()[~none] > lt[~none]
            assert not bad.any(), f"{what}: {int(bad.sum())} log-sum-exps off"
            assert (o[none] == 0).all(), f"{what}: rows that see nothing are zero"
