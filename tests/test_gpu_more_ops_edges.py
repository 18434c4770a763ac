"""GPU tests of the head norms, the E4M3 cache, attention over it and sampling at the ends of what they take."""
import math

import pytest
import torch

from _more_ops import norm_ref, quantised, rounded
from mixture_experts_ffn_moe_gb300 import build, gbmoe
from test_gpu_more_ops import BF, F32, FP, I32, attend, close, gen, make_cache, make_q, ref_of

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


# ------------------------------------------------------------------ attention over the cache
def with_zero_values(lens, counts, D, page, seed, zeros, scale, sink):
    """A cache of one KV head whose values have the size 448 * scale, but for the slots `zeros`, which hold zeros as the append writes
    them (scale 1); with `sink` these take 2^13 times the others' share."""
    side, table = make_cache(lens, counts, 1, D, page, seed, spread=0.0)
    (kc, ks), (vc, vs) = side
    base = torch.randn(D, generator=gen(seed))
    for b, n in enumerate(lens):
        for s in range(n + counts[b]):
            at = (int(table[b, s // page]), s % page, 0)
            strong = sink and zeros(s)
            key = base / (base @ base) * (13.0 * math.log(2.0) * D ** 0.5) if strong else 0.05 * torch.randn(D, generator=gen(s))
            c, x = quantised(key[None])
            kc[at], ks[at] = c[0], x[0]
            vs[at] = scale
            if zeros(s):
                vc[at], vs[at] = 0, 1.0
    return base, side, table


@pytest.mark.parametrize("where,scale", [("sink", 2.0 ** -12), ("all over", 2.0 ** -29), ("all over", 2.0 ** -36), ("run", 2.0 ** -29)])
@pytest.mark.parametrize("hq,counts", [(4, [1, 1]), (8, [2, 1]), (16, [2, 2]), (16, [8, 9]), (16, [20, 18])])
@pytest.mark.parametrize("dt,D,page", [(BF, 128, 16), (FP, 64, 5)])
def test_fp8_attention_over_slots_of_zero_values(dt, D, page, hq, counts, where, scale):
    """Slots of zero values (scale 1) add nothing and take no bits from the others, much smaller than that: the bound is that of a
    cache where these slots have a tiny scale, which is the same cache."""
    lens = [130, 37]
    zeros = {"sink": lambda s: s == 3, "all over": lambda s: s % 5 == 3, "run": lambda s: s < 20 or 40 < s < 100}[where]
    base, side, table = with_zero_values(lens, counts, D, page, 60 + D, zeros, scale, where == "sink")
    q = (base + 0.05 * torch.randn(sum(counts), hq, D, generator=gen(9))).to(dt)
    (kc, ks), (vc, vs) = side
    low = torch.where((vc & 127).amax(-1) == 0, torch.full_like(vs, 2.0 ** -40), vs)
    ref, bound = ref_of(q, ((kc, ks), (vc, low)), table, lens, counts, None, D ** -0.5)
    got = attend(q, side, table, lens, counts, None)
    close(got, ref, bound)
    assert (ref.abs().amax(-1) > 0).all()


@pytest.mark.parametrize("hq,counts", [(4, [1, 1]), (16, [20, 18])])
def test_fp8_attention_over_nothing_but_zero_values(hq, counts):
    """All of a sequence's values are zero, or only those that a row sees first: zeros, no NaN."""
    lens, D, page = [300, 37], 64, 16
    _, side, table = with_zero_values(lens, counts, D, page, 61, lambda s: s < 290, 1.0, False)
    q = make_q(counts, hq, D, BF, 61)
    ref, bound = ref_of(q, side, table, lens, counts, None, D ** -0.5)
    got = attend(q, side, table, lens, counts, None)
    close(got, ref, bound)
    assert (got[counts[0]:] == 0).all() and (got[:counts[0]] != 0).any()


# ------------------------------------------------------------------ sampling
@pytest.mark.parametrize("V,top_k", [(14, None), (200, 100), (3000, 2049), (20000, None), (60000, 30000)])
def test_min_p_of_one_keeps_the_largest_logit_alone(V, top_k):
    """Logits that differ by less than weights can tell: 1 and above leave the ones that are equal to the largest, in any of the
    kernel's ways to cut."""
    logits = 1.0 + torch.arange(V).flip(0).repeat(5, 1) % 7 * -2.0 ** -23
    logits[1] *= 1e-30
    logits[2, V // 2:] = -3.0
    logits[3] = torch.randn(V, generator=gen(V)) * 1e-9
    logits[4, ::3] = -1.0
    more = {} if top_k is None else {"top_k": torch.full((5,), top_k, dtype=I32).cuda()}
    temperature = torch.full((5,), 30.0).cuda()
    for min_p in (1.0, 7.0):
        for top_p in (None, torch.full((5,), 0.9).cuda()):
            p = gbmoe.moe_filter_probs(logits.cuda(), temperature, more.get("top_k"), top_p, torch.full((5,), min_p).cuda()).cpu()
            tokens = gbmoe.moe_sample(logits.cuda(), torch.full((5,), 0.999).cuda(), temperature, more.get("top_k"), top_p,
                                      torch.full((5,), min_p).cuda()).cpu()
            for i in range(5):
                best = (logits[i] == logits[i].max()).nonzero()[:, 0]
                kept = (p[i] > 0).nonzero()[:, 0]
                assert 0 < len(kept) <= len(best) and torch.equal(kept, best[:len(kept)]) and int(tokens[i]) == int(kept[-1] if len(kept) < 1000 else tokens[i])
                assert len(kept) == len(best) or top_p is not None or top_k is not None and top_k < len(best)
                assert int(tokens[i]) in kept and (p[i, kept] - 1 / len(kept)).abs().max() <= 2.0 ** -22


# ------------------------------------------------------------------ devices
@pytest.mark.skipif(torch.cuda.device_count() < 2, reason="needs two GPUs")
def test_calls_run_on_their_tensors_device():
    """Every call of a decode step, with tensors on a device that is not the current one."""
    g = gen(70)
    D, page, V = 64, 16, 500
    x = torch.randn(2, 6, D, generator=g).to(BF)
    pos, slots, offs = torch.tensor([0, 3], dtype=I32), torch.tensor([0, 19], dtype=I32), torch.arange(3, dtype=I32)
    w, s = torch.randint(0, 256, (32, D // 2), generator=g, dtype=torch.uint8), torch.rand(32, 2, generator=g)
    cache, scale = torch.randn(4, page, 2, D, generator=g), torch.rand(4, page, 2, generator=g) + 0.1
    logits, coins = torch.randn(4, V, generator=g), torch.rand(4, generator=g)

    def calls(dev):
        d = [t.to(dev) for t in (x, pos, slots, offs, w, s, cache.to(BF), cache.to(BF), cache.to(torch.float8_e4m3fn),
                                 cache.to(torch.float8_e4m3fn), scale, scale, logits, coins)]
        f, table = gbmoe.rope_frequencies(D, device=dev)[0], torch.tensor([[0], [1]], dtype=I32, device=dev)
        q, k, v = d[0][:, :2], d[0][:, 2:4], d[0][:, 4:]
        probs = gbmoe.moe_filter_probs(d[12])
        return [*gbmoe.moe_rope(q, k, d[1], f), gbmoe.moe_rope_append(q, k, v, d[1], f, d[2], d[6], d[7]),
                gbmoe.moe_linear_int4(q[:, 0], d[4], d[5]), gbmoe.moe_tree_attention(q, d[6], d[7], table, d[1], d[3]),
                *gbmoe.moe_verify_draft(probs, d[2], d[3], d[13], d[13][:2], 1), *gbmoe.moe_qk_norm_rope(q, k, d[1], f),
                gbmoe.moe_qk_norm_rope_append(q, k, v, d[1], f, d[2], d[8], d[9], None, None, d[10], d[11]),
                gbmoe.moe_tree_attention_fp8(q, d[8], d[9], d[10], d[11], table, d[1], d[3]),
                *gbmoe.moe_cache_read(d[8], d[9], d[10], d[11], d[2]), gbmoe.moe_sample(d[12], d[13]), probs]

    with torch.cuda.device(0):
        here, there = calls("cuda:0"), calls("cuda:1")
        torch.cuda.synchronize(1)
        assert torch.cuda.current_device() == 0
    for a, b in zip(here, there):
        assert b.device.index == 1 and torch.equal(a.float().cpu(), b.float().cpu())
