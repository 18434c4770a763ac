"""Host-side checks of the decode-step operators: refusals, size queries, frequency tables and the packed argument
structs.  No call here reaches a launch."""
import math
import struct

import numpy as np
import pytest
import torch

from _step_ops import fixed60, verify_ref
from mixture_experts_ffn_moe_gb300 import build, gbmoe

P = 4096  # never dereferenced
# moe_rope_args_t and moe_tree_attention_args_t, as the C compiler lays them out
ROPE_ARGS = struct.Struct("@9if2i3P3P3P6q5q3q")
TREE_ARGS = struct.Struct("@9ifq3P3PPP4q6q")


@pytest.fixture(scope="module")
def lib():
    build.build()
    return gbmoe.load()


ROPE = dict(dtype=0, tokens=4, dim=128, rot=128, off=0, inter=0, inv=0, hq=4, hk=2, scale=1.0, page=0, pages=0, pos=P,
            freq=P, slots=0, q=P, k=P, v=0, qo=P, ko=P, vc=0)


def rope(lib, **kw):
    d = {**ROPE, **kw}
    strides = d.pop("strides", [512, 128, 256, 128, 256, 128, 512, 128, 0, 256, 128, 0, 0, 0])
    return lib.moe_rope(ROPE_ARGS.pack(*d.values(), *strides), None)


def test_rope_refusals(lib):
    assert lib.moe_rope(None, None) == 1
    assert rope(lib, tokens=0) == 0
    assert rope(lib, hq=0, hk=0) == 0
    assert rope(lib, dtype=3) == 1
    assert rope(lib, tokens=-1) == 1
    assert rope(lib, rot=127) == 1
    assert rope(lib, rot=0) == 1
    assert rope(lib, rot=64, off=65) == 1
    assert rope(lib, rot=64, off=-2) == 1
    assert rope(lib, rot=6, off=3, inter=1) == 1
    assert rope(lib, dim=2048) == 2
    assert rope(lib, pos=0) == 1
    assert rope(lib, freq=0) == 1
    assert rope(lib, q=0) == 1
    assert rope(lib, ko=0) == 1
    assert rope(lib, slots=P) == 1                              # a cache of no pages
    assert rope(lib, slots=P, page=16, pages=4) == 1            # no values
    assert rope(lib, slots=P, page=1 << 20, pages=1 << 20, v=P, vc=P) == 2
    assert rope(lib, q=P + 1) == 1
    assert rope(lib, q=P + 2, inter=1) == 1                     # half a pair
    assert b"moe_rope" in lib.moe_last_error()


def linear(lib, dtype=0, x=P, xs=256, w=P, s=P, M=4, N=64, K=256, group=128, gated=0, y=P, ys=64, ws=None, size=0):
    return lib.moe_linear_int4(dtype, x, xs, w, s, M, N, K, group, gated, y, ys, ws, size, None)


def test_linear_refusals(lib):
    assert linear(lib, M=0) == 0
    assert linear(lib, dtype=2) == 1
    assert linear(lib, M=-1) == 1
    assert linear(lib, N=0) == 1
    assert linear(lib, group=16) == 2
    assert linear(lib, K=192, group=128) == 1
    assert linear(lib, gated=2) == 1
    assert linear(lib, M=1 << 21) == 2
    assert linear(lib, x=None) == 1
    assert linear(lib, xs=255) == 1
    assert linear(lib, ys=63) == 1
    assert linear(lib, x=P + 2) == 1
    assert linear(lib, xs=260) == 1
    assert linear(lib, w=P + 4) == 1
    assert linear(lib, y=P + 1) == 1
    size = gbmoe.moe_linear_int4_workspace_size
    assert size(17, 64, 256, 128) > 0 and size(16, 64, 256, 128) == 0 and size(9, 64, 7168, 128) > 0
    assert size(1, 64, 1 << 16, 32) > 0 and size(17, 64, 200, 128) == 0 and size(0, 64, 256, 128) == 0
    assert size(64, 64, 256, 128, True) > 0


TREE = dict(dtype=0, nodes=8, batch=2, hq=4, hk=2, dim=128, page=16, pages=10, width=4, scale=0.1, tld=4, q=P, k=P, v=P,
            table=P, ctx=P, offs=P, mask=P, out=P)


def tree(lib, ws=P, size=1 << 40, **kw):
    d = {**TREE, **kw}
    strides = d.pop("strides", [512, 128, 512, 128, 4096, 256, 128, 4096, 256, 128])
    return lib.moe_tree_attention(TREE_ARGS.pack(*d.values(), *strides), ws, size, None)


def test_tree_refusals(lib):
    assert lib.moe_tree_attention(None, P, 1, None) == 1
    assert tree(lib, nodes=0) == 0
    assert tree(lib, batch=0) == 0
    assert tree(lib, dtype=2) == 1
    assert tree(lib, hq=5) == 1
    assert tree(lib, dim=96) == 2
    assert tree(lib, batch=2000) == 2
    assert tree(lib, page=0) == 1
    assert tree(lib, page=1 << 20, width=1 << 20) == 2
    assert tree(lib, scale=math.inf) == 1
    assert tree(lib, scale=math.nan) == 1
    assert tree(lib, q=0) == 1
    assert tree(lib, offs=0) == 1
    assert tree(lib, q=P + 8) == 1
    assert tree(lib, out=P + 4) == 1
    assert tree(lib, strides=[512, 128, 512, 128, 4096, 255, 128, 4096, 256, 128]) == 1
    assert tree(lib, strides=[512, 128, 510, 128, 4096, 256, 128, 4096, 256, 128]) == 1


def test_tree_workspace(lib):
    size = gbmoe.moe_tree_attention_workspace_size
    assert size(8, 2, 4, 2, 128) > 0
    assert size(8, 0, 4, 2, 128) == 0 and size(8, 2000, 4, 2, 128) == 0 and size(8, 2, 4, 3, 128) == 0
    assert size(8, 2, 4, 2, 96) == 0 and size(-1, 2, 4, 2, 128) == 0
    assert lib.moe_read_tree_status(None, None, None) == 1


def verify(lib, t=P, ts=100, d=None, ds=0, tok=P, par=None, offs=P, coins=P, last=P, B=2, N=4, V=100, mx=4, out=P, path=P,
           acc=P):
    return lib.moe_verify_draft(t, ts, d, ds, tok, par, offs, coins, last, B, N, V, mx, out, path, acc, None)


def test_verify_refusals(lib):
    assert verify(lib, B=0) == 0
    assert verify(lib, B=-1) == 1
    assert verify(lib, V=0) == 1
    assert verify(lib, mx=65) == 2
    assert verify(lib, V=1 << 25, ts=1 << 25) == 2
    assert verify(lib, t=None) == 1
    assert verify(lib, acc=None) == 1
    assert verify(lib, d=P, ds=100, par=P) == 1                 # draft probabilities need a chain
    assert verify(lib, ts=99) == 1
    assert verify(lib, d=P, ds=99) == 1


def test_bindings_refuse_cpu_tensors_and_wrong_types():
    x = torch.zeros(2, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        gbmoe.moe_linear_int4(x, torch.zeros(4, 64, dtype=torch.uint8), torch.zeros(4, 1))
    with pytest.raises(ValueError):
        gbmoe.moe_rope(x.view(2, 1, 128), None, torch.zeros(2, dtype=torch.int32), torch.zeros(64, dtype=torch.float64))
    with pytest.raises(ValueError):
        gbmoe.moe_tree_attention(x.view(2, 1, 128), x, x, x, x, x)
    with pytest.raises(ValueError):
        gbmoe.moe_verify_draft(x.float(), x, x, x, x, 1)


def test_frequencies():
    f, s = gbmoe.rope_frequencies(8, 10000.0, device="cpu")
    assert np.allclose(f.numpy(), [1.0, 0.1, 0.01, 0.001], rtol=1e-15) and s == 1.0
    g, s = gbmoe.rope_frequencies(8, 10000.0, "linear", 4.0, device="cpu")
    assert np.allclose(g.numpy(), f.numpy() / 4, rtol=1e-15) and s == 1.0
    g, _ = gbmoe.rope_frequencies(8, 10000.0, "ntk", 4.0, device="cpu")
    assert g[0] == 1.0 and abs(g[-1] / (f[-1] / 4) - 1) < 1e-12       # the slowest pair is stretched by the factor
    g, s = gbmoe.rope_frequencies(128, 10000.0, "yarn", 40.0, 4096, device="cpu")
    f, _ = gbmoe.rope_frequencies(128, 10000.0, device="cpu")
    turns = 4096 * f / (2 * math.pi)
    assert torch.allclose(g[turns > 40], f[turns > 40]) and torch.allclose(g[turns < 0.8], f[turns < 0.8] / 40)
    assert ((g <= f) & (g >= f / 40)).all() and abs(s - (0.1 * math.log(40) + 1)) < 1e-15
    for bad in (dict(rot_dim=7), dict(rot_dim=0), dict(rot_dim=8, base=1.0), dict(rot_dim=8, factor=0.0),
                dict(rot_dim=8, scaling="yarn"), dict(rot_dim=8, scaling="other"), dict(rot_dim=2, scaling="ntk")):
        with pytest.raises(ValueError):
            gbmoe.rope_frequencies(device="cpu", **bad)


def test_argument_structs_have_the_compilers_size(tmp_path):
    import subprocess
    src = tmp_path / "s.c"
    src.write_text('#include <stdio.h>\n#include "gbmoe.h"\nint main(void) { printf("%zu %zu\\n", sizeof(moe_rope_args_t), '
                   'sizeof(moe_tree_attention_args_t)); return 0; }\n')
    subprocess.run(["gcc", "-I", build.INCLUDE, str(src), "-o", str(tmp_path / "s")], check=True)
    sizes = subprocess.run([str(tmp_path / "s")], capture_output=True, text=True, check=True).stdout.split()
    assert [int(v) for v in sizes] == [ROPE_ARGS.size, TREE_ARGS.size]


def test_the_reference_sampler_draws_from_the_target():
    """The oracle itself: over a grid of coins, what a one-node draft yields is distributed as the target row."""
    V = 6
    p = torch.tensor([0.05, 0.3, 0.15, 0.25, 0.2, 0.05])
    q = torch.tensor([0.3, 0.1, 0.2, 0.1, 0.25, 0.05])
    steps = 64
    for draft in (q[None], None):
        hist = np.zeros(V)
        for x in range(V):
            weight = float(q[x]) if draft is not None else 1.0
            for i in range(steps):
                coins = torch.tensor([(i + 0.5) / steps, 0.5])
                for j in range(steps):
                    last = torch.tensor([(j + 0.5) / steps])
                    out, _, acc = verify_ref(torch.stack([p, p]), [x], [0, 1], coins, last, 1, None, draft)
                    hist[out[0, 0]] += weight / steps / steps
            if draft is None:
                break
        assert np.abs(hist / hist.sum() - p.numpy()).max() < 2.0 / steps


def test_fixed_point_reference():
    for p in (0.0, 1.0, 0.5, 2.0 ** -24, 0.1, 1e-9, 1e-20, 3e-17, 2.0, -1.0, float("nan")):
        v = np.float32(p)
        exact = 0.0 if not v > 0 else min(float(v), 1.0)
        assert abs(fixed60([v])[0] - exact * 2.0 ** 60) <= 0.5
