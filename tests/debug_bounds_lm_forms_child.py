"""Runs in a child process with M3_LIBRARY=debug (the bounds-checked build): the
norm, the head's loss and the 4-bit products in the forms that only larger calls
take; the device status word must stay 0.  Prints "ALL OK"."""
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

from selective_state_space_exp_b200 import m3  # noqa: E402

assert m3.LIB_PATH.endswith("libm3_debug.so"), m3.LIB_PATH


def status_ok(what):
    st = m3.m3_stream_status()
    print(f"{what}: status {st}", flush=True)
    assert st == 0, (what, st)


def main():
    g = torch.Generator(device="cuda").manual_seed(2)

    def randn(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    # several splits of a sample (statistics, join, result; sums, means, dx, partial rows);
    # one block a tile that is not the whole form; groups in pieces with splits
    for dt in (torch.bfloat16, torch.float32):
        for B, L, G, cg in ((2, 3000, 2, 24), (300, 80, 16, 64), (2, 400, 1, 4100), (3, 1001, 6, 85)):
            x, z, dy = (randn(B, L, G * cg).to(dt) for _ in range(3))
            for act in ("none", "silu", "gate"):
                zz = z if act == "gate" else None
                y, m, r = m3.m3_group_norm_fwd(x, G, z=zz, act=act, scope="sequence")
                m3.m3_group_norm_bwd(x, G, m, r, dy, z=zz, act=act, scope="sequence")
            T = B * L
            cu = torch.tensor([1, 1, T // 3, T - 1], dtype=torch.int32, device="cuda")
            x, dy = x.view(T, -1), dy.view(T, -1)
            y, m, r = m3.m3_group_norm_fwd_varlen(cu, x, G)
            m3.m3_group_norm_bwd_varlen(cu, x, G, m, r, dy)
            status_ok(f"norm {dt} {B} x {L} x {G} x {cg}")
        for T, G, cg in ((5000, 6, 8), (3000, 1, 600), (700, 3, 4096)):  # single positions, many rows
            x, dy = randn(T, G * cg).to(dt), randn(T, G * cg).to(dt)
            y, m, r = m3.m3_group_norm_fwd(x, G)
            m3.m3_group_norm_bwd(x, G, m, r, dy)
            status_ok(f"norm {dt} {T} x {G} x {cg}")
    # pairs of CTAs; three pieces of the vocabulary, added up; a split dW; a split dh
    for M, V, K in ((260, 9000, 64), (20000, 15000, 16), (2000, 120, 64), (40, 9000, 1040)):
        h, W = randn(M, K).bfloat16(), randn(V, K).bfloat16() / 8
        t = torch.randint(0, V, (M,), generator=g, device="cuda")
        t[::5] = -100
        loss, lse = m3.m3_linear_xent_fwd(h, W, t)
        m3.m3_linear_xent_bwd(h, W, t, lse, torch.ones_like(lse))
        status_ok(f"xent {M} x {V} x {K}")
    # tiles of 128 tokens; token values read again for each slice; split inputs
    for M, N, K, G in ((65, 4800, 256, 128), (130, 3300, 384, 64), (3, 2, 33280, 64), (16, 7, 33280, 128), (40, 129, 4096, 32)):
        W = randn(N, K)
        for sym in (False, True):
            q = m3.m3_w4_quantize(W, G, symmetric=sym)
            for dt in (torch.bfloat16, torch.float32):
                m3.m3_linear_w4(randn(M, K).bfloat16(), *q, out_dtype=dt)
        status_ok(f"w4 {M} x {N} x {K} group {G}")
    print("ALL OK")


if __name__ == "__main__":
    main()
