"""Runs in a child process with M3_LIBRARY=debug (the bounds-checked build): the
norm, the head's loss and the 4-bit products in every form they have, on small
ragged sizes; the device status word must stay 0.  Prints "ALL OK"."""
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
    g = torch.Generator(device="cuda").manual_seed(1)

    def randn(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    for dt in (torch.bfloat16, torch.float32):
        for T, G, cg in ((5, 3, 7), (70, 4, 64), (9, 1, 1200), (3, 1, 9000)):
            x, z, dy = (randn(T, G * cg).to(dt) for _ in range(3))
            for act in ("none", "silu", "gate"):
                zz = z if act == "gate" else None
                for scope in ("token", "sequence"):
                    v = [None if a is None else (a if scope == "token" else a[None]) for a in (x, zz, dy)]
                    y, m, r = m3.m3_group_norm_fwd(v[0], G, z=v[1], act=act, scope=scope)
                    m3.m3_group_norm_bwd(v[0], G, m, r, v[2], z=v[1], act=act, scope=scope)
            cu = torch.tensor([1, 1, T - 1], dtype=torch.int32, device="cuda")
            y, m, r = m3.m3_group_norm_fwd_varlen(cu, x, G)
            m3.m3_group_norm_bwd_varlen(cu, x, G, m, r, dy)
            status_ok(f"norm {dt} {T} x {G} x {cg}")
    for M, V, K in ((1, 1, 8), (130, 300, 72), (700, 90, 64), (9, 5000, 128)):
        h, W = randn(M, K).bfloat16(), randn(V, K).bfloat16() / 8
        t = torch.randint(0, V, (M,), generator=g, device="cuda")
        loss, lse = m3.m3_linear_xent_fwd(h, W, t)
        m3.m3_linear_xent_bwd(h, W, t, lse, torch.ones_like(lse))
        status_ok(f"xent {M} x {V} x {K}")
    for M, N, K, G in ((1, 3, 32, 32), (7, 50, 640, 128), (16, 33, 96, 32), (20, 130, 320, 64), (70, 200, 2048, 128),
                       (130, 17, 512, 32)):
        W = randn(N, K)
        for sym in (False, True):
            q = m3.m3_w4_quantize(W, G, symmetric=sym)
            for dt in (torch.bfloat16, torch.float32):
                m3.m3_linear_w4(randn(M, K).bfloat16(), *q, out_dtype=dt)
        status_ok(f"w4 {M} x {N} x {K} group {G}")
    print("ALL OK")


if __name__ == "__main__":
    main()
