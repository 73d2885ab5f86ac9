"""Run rotation, cache store, attention and read-back of one batch a few
times, for profilers.

    python -m fp8_w8a8_dynamic_b200.run_serving --B 64 --new 1 --own 1024 --prefix 32768 --reps 2

Builds nothing (the library must be built).  B sequences with `new` query
tokens each share a prefix of `prefix` cached tokens and have own / 8 to own
cached tokens of their own (the new ones among them).  Makes `reps` rounds of
rope_kv_store, prefix_attention and kv_page_read (of the prefix) on the
current stream, synchronises, checks the device status word and prints one
line.  A profiler such as Nsight Compute captures the kernels of those calls
by name.
"""
import argparse


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--B", type=int, default=64)
    ap.add_argument("--new", type=int, default=1)
    ap.add_argument("--own", type=int, default=1024)
    ap.add_argument("--prefix", type=int, default=32768)
    ap.add_argument("--Hq", type=int, default=32)
    ap.add_argument("--Hkv", type=int, default=8)
    ap.add_argument("--D", type=int, default=128)
    ap.add_argument("--page", type=int, default=64)
    ap.add_argument("--reps", type=int, default=2)
    ap.add_argument("--seed", type=int, default=1)
    args = ap.parse_args()

    import torch
    from fp8_w8a8_dynamic_b200 import mfp8

    dev = torch.device("cuda", 0)
    torch.cuda.set_device(dev)
    B, ps, T = args.B, args.page, args.B * args.new
    gen = torch.Generator(device=dev).manual_seed(args.seed)
    own = torch.linspace(max(args.own // 8, args.new), args.own, B).round().int()
    per, shared = -(-args.own // ps), -(-args.prefix // ps)
    pages = torch.randperm(B * per + shared, generator=gen, device=dev).int()
    table, prefix_pages = pages[:B * per].view(B, per), pages[B * per:].contiguous()

    def pool():
        codes = torch.randint(0, 256, (pages.numel(), args.Hkv, ps, args.D), generator=gen, device=dev).byte()
        codes[codes & 127 == 127] = 0  # no NaN codes
        return codes, torch.rand(codes.shape[:3], generator=gen, device=dev).mul_(0.01)

    k_pages, k_scale = pool()
    v_pages, v_scale = pool()
    qkv = torch.randn(T, (args.Hq + 2 * args.Hkv) * args.D, generator=gen, device=dev).bfloat16()
    place = (own[:, None] - args.new + torch.arange(args.new)).to(dev)  # of each new token among its own
    slot = (torch.gather(table, 1, place // ps) * ps + place % ps).long().view(-1)
    pos = (args.prefix + place).int().view(-1)
    q_start = torch.arange(B + 1, dtype=torch.int32, device=dev) * args.new
    kv_len = own.to(dev)
    freq, _ = mfp8.rope_frequencies(args.D, 5e6, device=dev)
    at = torch.arange(args.prefix, device=dev)
    prefix_slot = prefix_pages[at // ps].long() * ps + at % ps
    for _ in range(args.reps):
        q = mfp8.rope_kv_store(qkv, args.Hq, pos, freq, slot, k_pages, k_scale, v_pages, v_scale)
        out = mfp8.prefix_attention(q, q_start, kv_len, table, prefix_pages, args.prefix, k_pages, k_scale, v_pages,
                                    v_scale, args.new)
        mfp8.kv_page_read(k_pages, k_scale, prefix_slot)
    torch.cuda.synchronize()
    st = mfp8.device_status()
    if st != mfp8.OK:
        raise mfp8.Mfp8Error(st, "run_serving")
    print(f"run_serving B={B} new={args.new} own={args.own} prefix={args.prefix} reps={args.reps}: ok, "
          f"out {tuple(out.shape)}")


if __name__ == "__main__":
    main()
