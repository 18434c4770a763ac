"""GPU tests of the head norms, the E4M3 cache, attention over it and sampling at the ends of what they take."""
import math

import pytest
import torch

from _more_ops import norm_ref, rounded
from mixture_experts_ffn_moe_gb300 import build, gbmoe
from test_gpu_more_ops import BF, F32, I32, close, gen

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()
    return gbmoe.load()


# ------------------------------------------------------------------ norms of heads
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("dt,D", [(F32, 128), (BF, 128), (F32, 64), (BF, 1024), (F32, 22), (BF, 22)])
def test_norm_rope_of_heads_near_the_largest_numbers(dt, D, inter):
    """Heads of nothing but (nearly) the type's largest number, whose scaled squares must not leave fp32's range either, with small
    elements beside them; heads whose sum of squares has just left it."""
    big = float(torch.finfo(dt).max)
    x = torch.randn(8, 2, D, generator=gen(D)).to(dt)
    sign = torch.where(torch.rand(5, D, generator=gen(1)) < 0.5, -1.0, 1.0)
    x[0, 0], x[1, 0], x[2, 0] = (sign[0] * big).to(dt), big, (sign[2] * 2.0 ** 125).to(dt)
    x[3, 0] = (sign[3] * 1.01 * 2.0 ** 64 / math.sqrt(D)).to(dt)
    x[4, 0] = (sign[4] * big).to(dt)
    x[4, 0, D // 2:] = (x[4, 1, D // 2:].float() * 2.0 ** 66).to(dt)
    w = (1 + 0.2 * torch.randn(D, generator=gen(2))).to(dt)
    pos = torch.arange(8, dtype=I32) * 5
    f, _ = gbmoe.rope_frequencies(D - 2)
    got, _ = gbmoe.moe_qk_norm_rope(x.cuda(), None, pos.cuda(), f, w.cuda(), None, 1e-6, interleaved=inter)
    y, err = norm_ref(x, w, 1e-6, pos, f.cpu(), 1.0, inter, 0)
    close(got, y, rounded(y, err, dt))


def test_norm_rope_of_as_many_heads_as_it_takes():
    """2^31 - 1 heads of one element: as many pieces of work as an int counts, the last CTA not full."""
    T, many = 2 ** 31 - 1, 2053
    f = torch.empty(0, dtype=torch.float64).cuda()
    w = torch.tensor([1.5], dtype=BF).cuda()
    x = (torch.randn(many, 1, 1, generator=gen(4)) * 1e-3).to(BF).cuda()
    want, _ = gbmoe.moe_qk_norm_rope(x, None, torch.zeros(many, dtype=I32).cuda(), f, w, None, 1e-6)
    q = x.repeat(T // many + 1, 1, 1)[:T]
    gbmoe.moe_qk_norm_rope(q, None, torch.zeros(T, dtype=I32, device="cuda"), f, w, None, 1e-6, q_out=q)
    whole = T // many * many
    assert (q[:whole].view(-1, many) == want.view(1, many)).all() and torch.equal(q[whole:], want[:T - whole])
