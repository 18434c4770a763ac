"""GPU parity of the decode-step operators against their plain 64-bit forms, within bounds derived from the number
formats and the lengths of the sums (tests/_step_ops.py); draft verification is exact."""
import numpy as np
import pytest
import torch

from _step_ops import ancestors, int4_values, linear_ref, mask_tensor, rope_ref, tree_ref, verify_ref
from mixture_experts_ffn_moe_gb300 import build, gbmoe

pytestmark = pytest.mark.gpu

BF, FP, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()
    return gbmoe.load()


def gen(seed):
    return torch.Generator().manual_seed(seed)


def close(got, ref, bound, what=""):
    got = got.double().cpu()
    bad = ~((got - ref).abs() <= bound)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} outside, worst {(got - ref).abs().max():.3e}, "
                           f"first at {bad.nonzero()[0].tolist()}")


# ------------------------------------------------------------------ rotary positions
@pytest.mark.parametrize("T,hq,hk,D,rot,off,inter,inv,dt,far", [
    (1, 1, 1, 64, 64, 0, False, False, BF, 10),
    (33, 8, 2, 128, 128, 0, False, False, BF, 1 << 20),
    (33, 8, 2, 128, 128, 0, True, False, BF, 1 << 20),
    (5, 3, 1, 192, 64, 128, False, True, FP, 32768),
    (5, 3, 1, 192, 64, 128, True, True, F32, 2 ** 31 - 1),
    (700, 7, 1, 80, 32, 8, False, False, FP, 4096),
    (9, 2, 2, 21, 6, 3, False, False, BF, 100),        # odd head: single elements
    (9, 2, 2, 22, 6, 4, True, False, F32, 100),
    (9, 2, 0, 20, 4, 16, True, False, FP, 100),
    (2000, 5, 1, 64, 2, 0, False, False, F32, 100000),
    (3, 1, 1, 1024, 1024, 0, False, False, BF, 100000),
])
def test_rope(T, hq, hk, D, rot, off, inter, inv, dt, far):
    g = gen(T + D)
    q, k = torch.randn(T, hq, D, generator=g).to(dt), torch.randn(T, hk, D, generator=g).to(dt)
    pos = torch.randint(-3, far, (T,), generator=g, dtype=torch.int64).to(torch.int32)
    f, scale = gbmoe.rope_frequencies(rot, 10000.0, "yarn", 4.0, 4096)
    qo, ko = gbmoe.moe_rope(q.cuda(), k.cuda() if hk else None, pos.cuda(), f, scale, inter, inv, off)
    close(qo, *rope_ref(q, pos, f.cpu(), scale, inter, inv, off), "q")
    if hk:
        close(ko, *rope_ref(k, pos, f.cpu(), scale, inter, inv, off), "k")


def test_rope_in_place_on_a_strided_projection():
    g = gen(1)
    T, hq, hk, D = 37, 4, 2, 64
    row = torch.randn(T, (hq + 2 * hk) * D + 8, generator=g).to(BF)  # a padded row: strides are not the shape's
    pos = torch.arange(T, dtype=torch.int32) * 1001
    f, _ = gbmoe.rope_frequencies(D)
    d = row.cuda()
    view = d[:, :(hq + 2 * hk) * D].view(T, hq + 2 * hk, D)
    q, k = view[:, :hq], view[:, hq:hq + hk]
    gbmoe.moe_rope(q, k, pos.cuda(), f, q_out=q, k_out=k)
    src = row[:, :(hq + 2 * hk) * D].view(T, hq + 2 * hk, D)
    close(q, *rope_ref(src[:, :hq], pos, f.cpu(), 1.0, False, False, 0))
    close(k, *rope_ref(src[:, hq:hq + hk], pos, f.cpu(), 1.0, False, False, 0))
    assert torch.equal(d.cpu()[:, (hq + hk) * D:], row[:, (hq + hk) * D:])  # v and the padding are untouched


@pytest.mark.parametrize("dt,D,rot,inter,page,heads_first", [
    (BF, 128, 128, False, 16, False), (FP, 64, 32, True, 24, True), (F32, 80, 32, False, 1, False),
    (BF, 21, 6, False, 7, True)])
def test_rope_append(dt, D, rot, inter, page, heads_first):
    g = gen(D)
    T, hq, hk = 45, 4, 2
    qkv = torch.randn(T, hq + 2 * hk, D, generator=g).to(dt)
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
    pages = -(-T // page) + 2
    shape = (pages, hk, page, D) if heads_first else (pages, page, hk, D)
    kc, vc = torch.full(shape, 7.0, dtype=dt), torch.full(shape, 9.0, dtype=dt)
    slots = torch.randperm(pages * page, generator=g)[:T].to(torch.int32)
    slots[::5] = -1
    slots[3] = pages * page  # just past the cache: skipped as well
    pos = torch.randint(0, 100000, (T,), generator=g).to(torch.int32)
    f, scale = gbmoe.rope_frequencies(rot, 1e6, "linear", 2.0)
    order = (0, 2, 1, 3) if heads_first else (0, 1, 2, 3)
    kd, vd = kc.cuda().permute(order), vc.cuda().permute(order)
    d = qkv.cuda()
    qo = gbmoe.moe_rope_append(d[:, :hq], d[:, hq:hq + hk], d[:, hq + hk:], pos.cuda(), f, slots.cuda(), kd, vd,
                               scale, inter)
    close(qo, *rope_ref(q, pos, f.cpu(), scale, inter, False, 0))
    kr, kb = rope_ref(k, pos, f.cpu(), scale, inter, False, 0)
    want_k, bound = kc.permute(order).double().clone(), torch.zeros(kc.permute(order).shape, dtype=torch.float64)
    want_v = vc.permute(order).clone()
    for t, s in enumerate(slots.tolist()):
        if 0 <= s < pages * page:
            want_k[s // page, s % page], bound[s // page, s % page] = kr[t], kb[t]
            want_v[s // page, s % page] = v[t]
    close(kd, want_k, bound, "keys")
    assert torch.equal(vd.cpu(), want_v)


def test_rope_turns_back():
    g = gen(4)
    q = torch.randn(50, 4, 64, generator=g).cuda()
    pos = torch.randint(0, 1000000, (50,), generator=g).to(torch.int32).cuda()
    f, _ = gbmoe.rope_frequencies(64)
    there, _ = gbmoe.moe_rope(q, None, pos, f)
    back, _ = gbmoe.moe_rope(there, None, pos, f, inverse=True)
    # two turns, each off by 2^-20 of the pair
    assert (back - q).abs().max() <= 2.0 ** -18 * q.abs().max()


def test_rope_is_its_own_gradient_direction():
    """The gradient of sum(w * rope(x)) is the inverse turn of w: against differences of the 64-bit form."""
    g = gen(5)
    x, w = torch.randn(3, 1, 8, generator=g, dtype=torch.float64), torch.randn(3, 1, 8, generator=g, dtype=torch.float64)
    pos = torch.tensor([0, 5, 70000], dtype=torch.int32)
    f, _ = gbmoe.rope_frequencies(8)
    grad, _ = gbmoe.moe_rope(w.float().cuda(), None, pos.cuda(), f, inverse=True)
    num = torch.zeros_like(x)
    for i in range(x.numel()):
        d = torch.zeros_like(x)
        d.view(-1)[i] = 0.5
        num.view(-1)[i] = ((rope_ref(x.float() * 0 + d.float(), pos, f.cpu(), 1.0, False, False, 0)[0]
                            - rope_ref(-d.float(), pos, f.cpu(), 1.0, False, False, 0)[0]) * w).sum()
    assert (grad.double().cpu() - num).abs().max() <= 2.0 ** -19 * w.abs().max() * 2


# ------------------------------------------------------------------ 4-bit linear
@pytest.mark.parametrize("M,N,K,group,gated,dt", [
    (1, 1, 128, 128, False, BF), (1, 16, 32, 32, False, FP), (2, 17, 64, 64, False, BF), (3, 15, 64, 32, True, BF),
    (8, 100, 1024, 128, False, BF), (9, 33, 2048 + 128, 128, True, FP), (16, 64, 4000, 32, False, FP),
    (17, 47, 1088, 64, False, BF), (33, 130, 512, 128, True, BF), (64, 31, 7168, 128, False, BF),
    (65, 40, 96, 32, True, FP), (100, 5, 192, 64, False, FP), (1, 300, 18432, 128, False, BF),
    (5, 9, 12320, 32, True, BF)])
def test_linear_int4(M, N, K, group, gated, dt):
    g = gen(M * 7 + K)
    rows = N * (2 if gated else 1)
    x = torch.randn(M, K, generator=g).to(dt)
    w = torch.randint(0, 256, (rows, K // 2), generator=g, dtype=torch.uint8)
    s = (0.5 + torch.rand(rows, K // group, generator=g)) * 0.05
    y = gbmoe.moe_linear_int4(x.cuda(), w.cuda(), s.cuda(), gated)
    close(y, *linear_ref(x, w, s, gated))
    assert torch.equal(y, gbmoe.moe_linear_int4(x.cuda(), w.cuda(), s.cuda(), gated))


@pytest.mark.parametrize("M", [1, 8, 9, 16])
@pytest.mark.parametrize("N,K,group", [(2100, 544, 32), (2431, 192, 64), (4865, 128, 128), (9729, 128, 128), (40, 5504, 64)])
def test_linear_int4_tiles_of_16_and_32_rows(M, N, K, group):
    """Widths around the ones where the tile changes, a warp's share of K from a part of a block to many."""
    g = gen(M + N)
    x = torch.randn(M, K, generator=g).to(BF)
    w = torch.randint(0, 256, (N, K // 2), generator=g, dtype=torch.uint8)
    s = (0.5 + torch.rand(N, K // group, generator=g)) * 0.05
    close(gbmoe.moe_linear_int4(x.cuda(), w.cuda(), s.cuda()), *linear_ref(x, w, s, False))


def test_linear_int4_every_code_and_wide_ranges():
    """All 16 codes at every place of a word, scales from 2^-30 to 2^20 and activations from 1e-30 to 1e30."""
    g = gen(2)
    N, K = 48, 256
    w = ((torch.arange(N)[:, None] * 7 + torch.arange(K // 2)[None] * 11) % 256).to(torch.uint8)
    s = torch.exp2(torch.randint(-30, 21, (N, 2), generator=g).float())
    x = (torch.randn(4, K, generator=g) * torch.tensor([1e-30, 1.0, 1e4, 1e25])[:, None]).to(BF)
    close(gbmoe.moe_linear_int4(x.cuda(), w.cuda(), s.cuda()), *linear_ref(x, w, s, False))


@pytest.mark.parametrize("dt,M,K", [(BF, 3, 512), (FP, 12, 512), (BF, 40, 8192)])
def test_linear_int4_infinities_and_sums_near_overflow(dt, M, K):
    """An infinite activation gives infinities of the code's sign; sums of x past the type's range do no harm."""
    g = gen(6)
    N, K = 40, K
    x = torch.randn(M, K, generator=g).to(dt)
    x[0] = torch.finfo(dt).max / 64 if dt == FP else 1e35
    x[1, 7] = float("inf")
    w = torch.randint(0, 256, (N, K // 2), generator=g, dtype=torch.uint8)
    w[:, 3] = torch.where((w[:, 3] >> 4) == 0, w[:, 3] + 16, w[:, 3])  # column 7 has no zero codes
    s = (0.5 + torch.rand(N, K // 128, generator=g)) * 1e-3
    y = gbmoe.moe_linear_int4(x.cuda(), w.cuda(), s.cuda())
    ref, bound = linear_ref(x, w, s, False)
    keep = [m for m in range(M) if m != 1]
    close(y[keep], ref[keep], bound[keep])
    q7 = int4_values(w)[:, 7]
    assert (y[1].float().cpu() == torch.where(q7 > 0, float("inf"), float("-inf"))).all()


def test_linear_int4_strided_rows_and_nonfinite_rows_stay_apart():
    g = gen(3)
    x = torch.randn(4, 512 + 64, generator=g).to(BF)
    x[2, :512] = float("nan")
    w = torch.randint(0, 256, (40, 256), generator=g, dtype=torch.uint8)
    s = torch.rand(40, 4, generator=g)
    out = torch.full((4, 48), 3.0, dtype=BF, device="cuda")
    gbmoe.moe_linear_int4(x.cuda()[:, :512], w.cuda(), s.cuda(), out=out[:, :40])
    ref, bound = linear_ref(x[:, :512], w, s, False)
    keep = [0, 1, 3]
    close(out[keep][:, :40], ref[keep], bound[keep])
    assert out[2, :40].isnan().all() and (out[:, 40:] == 3.0).all()


# ------------------------------------------------------------------ tree attention
def make_tree(ctx, counts, hq, hk, D, page, dt, seed, masks="tree", heads_first=False, fill=float("nan")):
    """A paged cache whose unused slots hold `fill`, tables with -1 past the end."""
    g, r = gen(seed), np.random.default_rng(seed)
    N = sum(counts)
    need = [-(-(c + n) // page) for c, n in zip(ctx, counts)]
    pool = sum(need) + 3
    shape = (pool, hk, page, D) if heads_first else (pool, page, hk, D)
    order = (0, 2, 1, 3) if heads_first else (0, 1, 2, 3)
    kc, vc = torch.full(shape, fill, dtype=dt).permute(order), torch.full(shape, fill, dtype=dt).permute(order)
    table = np.full((len(ctx), max(max(need), 1)), -1, dtype=np.int32)
    free, at = r.permutation(pool), 0
    for b, p in enumerate(need):
        table[b, :p] = free[at:at + p]
        at += p
        for s in range(ctx[b] + counts[b]):
            kc[table[b, s // page], s % page] = torch.randn(hk, D, generator=g).to(dt)
            vc[table[b, s // page], s % page] = torch.randn(hk, D, generator=g).to(dt)
    q = torch.randn(N, hq, D, generator=g).to(dt)
    if masks == "tree":
        masks = [m for n in counts for m in ancestors([int(r.integers(-1, j)) if j else -1 for j in range(n)])]
    elif masks == "random":
        masks = [int(r.integers(0, 2 ** 63)) * 2 + int(r.integers(0, 2)) for _ in range(N)]
    offs = [0] + [int(x) for x in np.cumsum(counts)]
    return q, kc, vc, table, ctx, offs, masks


def run_tree(q, kc, vc, table, ctx, offs, masks, scale=None, workspace=None):
    return gbmoe.moe_tree_attention(q.cuda(), _dev(kc), _dev(vc), torch.from_numpy(table).cuda(),
                                    torch.tensor(ctx, dtype=torch.int32).cuda(),
                                    torch.tensor(offs, dtype=torch.int32).cuda(),
                                    None if masks is None else mask_tensor(masks).cuda(), scale=scale,
                                    workspace=workspace)


def _dev(c):
    """On the GPU with the same strides."""
    d = torch.empty_strided(c.shape, c.stride(), dtype=c.dtype, device="cuda")
    d.copy_(c)
    return d


@pytest.mark.parametrize("ctx,counts,hq,hk,D,page,dt,masks,hf", [
    ([0], [1], 1, 1, 128, 16, BF, None, False),
    ([1], [1], 2, 1, 64, 16, FP, None, False),
    ([37], [5], 8, 2, 128, 16, BF, "tree", False),
    ([0, 15, 16, 17, 63, 64, 65], [1, 2, 3, 1, 5, 4, 8], 4, 2, 128, 16, BF, "tree", False),
    ([0, 15, 16, 17, 63, 64, 65], [1, 2, 3, 1, 5, 4, 8], 4, 2, 64, 1, FP, "tree", True),
    ([1000, 3], [64, 64], 10, 2, 128, 48, BF, "tree", False),
    ([200, 0, 129], [33, 7, 64], 16, 1, 64, 3, BF, "random", True),
    ([5000], [4], 16, 2, 128, 64, BF, None, False),
    ([2500, 130, 1], [16, 24, 2], 5, 1, 128, 256, FP, "tree", False),
    ([700] * 40, [3] * 40, 4, 4, 64, 32, BF, None, False),
    ([12000, 1], [2, 1], 8, 8, 128, 128, FP, "random", False),
    # wide trees: one and two products of 128 rows, several row tiles, ragged ones, tiles of 128 slots and their edges
    ([0], [33], 1, 1, 128, 16, BF, "tree", False),
    ([127], [1], 64, 1, 64, 16, BF, None, False),
    ([126, 128, 129, 0, 300], [64, 60, 63, 1, 50], 4, 1, 128, 16, FP, "random", True),
    ([5000, 0, 40, 250], [64, 64, 2, 33], 32, 2, 128, 7, BF, "tree", False),
    ([3000], [64], 48, 2, 64, 64, FP, "tree", False),
    ([257] * 9, [20] * 9, 12, 3, 64, 1, BF, "tree", False),
    ([20000], [40], 8, 1, 128, 256, BF, None, False),
])
def test_tree_attention(ctx, counts, hq, hk, D, page, dt, masks, hf):
    case = make_tree(ctx, counts, hq, hk, D, page, dt, 11 + len(ctx) + D, masks, hf)
    ws = torch.empty(gbmoe.moe_tree_attention_workspace_size(sum(counts), len(ctx), hq, hk, D), dtype=torch.uint8,
                     device="cuda")
    got = run_tree(*case, workspace=ws)
    close(got, *tree_ref(*case, D ** -0.5))
    assert gbmoe.moe_read_tree_status(ws) == (0, 0, 0)
    assert torch.equal(got, run_tree(*case))  # the same bits on another workspace


@pytest.mark.parametrize("B,hq,n", [(33, 4, 3), (1024, 2, 2), (65, 64, 9)])
def test_tree_attention_of_many_sequences_some_of_them_empty(B, hq, n):
    """Cut units whose sequences stand anywhere among many, between ones without nodes."""
    r = np.random.default_rng(B)
    counts = [0 if r.random() < 0.4 else int(r.integers(1, n + 1)) for _ in range(B)]
    ctx = [int(r.integers(0, 90)) for _ in range(B)]
    for b in (1, B // 2, B - 1):
        ctx[b], counts[b] = 3000, n
    case = make_tree(ctx, counts, hq, 2, 64, 16, BF, B)
    ws = torch.empty(gbmoe.moe_tree_attention_workspace_size(sum(counts), B, hq, 2, 64), dtype=torch.uint8, device="cuda")
    close(run_tree(*case, workspace=ws), *tree_ref(*case, 64 ** -0.5))
    assert gbmoe.moe_read_tree_status(ws) == (0, 0, 0)


def test_tree_rows_that_see_nothing_and_empty_sequences():
    case = list(make_tree([0, 40, 0], [3, 0, 2], 4, 2, 64, 16, BF, 3, "tree"))
    case[6] = [0, 0b010, 0b111, 0, 0b10]
    got = run_tree(*case)
    close(got, *tree_ref(*case, 64 ** -0.5))
    assert (got[0] == 0).all() and (got[3] == 0).all()


@pytest.mark.parametrize("hq", [4, 64])
@pytest.mark.parametrize("dt,value", [(BF, float("nan")), (BF, float("inf")), (FP, float("-inf"))])
def test_tree_hidden_slots_do_not_leak(dt, value, hq):
    """Node 1 holds infinities and NaN; nodes that do not see it are as without, those that see it get them."""
    ctx, counts, D, page, half = [70], [5], 128, 16, hq // 2
    case = list(make_tree(ctx, counts, hq, 2, D, page, dt, 5, "tree"))
    case[6] = ancestors([-1, -1, 0, 1, 2])
    q, kc, vc, table = case[:4]
    slot = 71
    vc[table[0, slot // page], slot % page, :, ::3] = value
    kc[table[0, slot // page], slot % page, 1] = value
    got = run_tree(*case).double().cpu()
    ref, bound = tree_ref(*case, D ** -0.5)
    for j in (0, 2, 4):
        close(got[j], ref[j], bound[j])
    for j in (1, 3):
        assert not got[j, :half, ::3].isfinite().any()  # first KV head: keys are finite, the value's elements are not
        close(got[j, :half, 1::3], ref[j, :half, 1::3], bound[j, :half, 1::3])
        close(got[j, :half, 2::3], ref[j, :half, 2::3], bound[j, :half, 2::3])


@pytest.mark.parametrize("hq", [4, 32])
def test_tree_attention_large_scores_and_scale(hq):
    case = make_tree([300], [6], hq, 1, 128, 16, BF, 9, "tree")
    q = case[0] * 30
    close(run_tree(q, *case[1:], scale=0.5), *tree_ref(q, *case[1:], 0.5))
    close(run_tree(q, *case[1:], scale=-0.01), *tree_ref(q, *case[1:], -0.01))


def test_tree_attention_over_offsets_past_32_bits():
    """Pages 2^31 elements apart: element offsets need 64 bits."""
    case = list(make_tree([40], [3], 2, 1, 64, 16, BF, 21, "tree"))
    far = (1 << 31) + 64
    big = torch.empty(2 * far + 4096, dtype=BF, device="cuda")
    k, v = (big[o:].as_strided((3, 16, 1, 64), (far, 64, 64, 1)) for o in (0, 2048))
    order = case[3][0, :3].tolist()
    k.copy_(case[1][order])
    v.copy_(case[2][order])
    got = gbmoe.moe_tree_attention(case[0].cuda(), k, v, torch.tensor([[0, 1, 2]], dtype=torch.int32).cuda(),
                                   torch.tensor([40], dtype=torch.int32).cuda(),
                                   torch.tensor([0, 3], dtype=torch.int32).cuda(), mask_tensor(case[6]).cuda())
    close(got, *tree_ref(*case, 64 ** -0.5))


def test_tree_attention_strided_tensors():
    case = list(make_tree([90, 20], [4, 4], 4, 2, 64, 16, FP, 8, "tree"))
    wide = torch.zeros(8, 9, 64, dtype=FP, device="cuda")  # q is a part of a projection's rows
    wide[:, 1:5] = case[0].cuda()
    out = torch.zeros(8, 6, 72, dtype=FP, device="cuda")
    table = torch.full((2, 9), 10 ** 6, dtype=torch.int32, device="cuda")
    table[:, :case[3].shape[1]] = torch.from_numpy(case[3]).cuda()
    gbmoe.moe_tree_attention(wide[:, 1:5], _dev(case[1]), _dev(case[2]), table[:, :case[3].shape[1]],
                             torch.tensor(case[4], dtype=torch.int32).cuda(),
                             torch.tensor(case[5], dtype=torch.int32).cuda(), mask_tensor(case[6]).cuda(),
                             out=out[:, 1:5, :64])
    close(out[:, 1:5, :64], *tree_ref(*case, 64 ** -0.5))
    assert (out[:, 0] == 0).all() and (out[:, 5] == 0).all() and (out[:, :, 64:] == 0).all()


@pytest.mark.parametrize("hq", [2, 64])
def test_tree_attention_reports_and_leaves_out_bad_pages(hq):
    case = list(make_tree([100, 30], [2, 2], hq, 1, 64, 16, BF, 13, "tree"))
    case[3][0, 2] = 9999
    case[3][1, 0] = -5
    ws = torch.empty(gbmoe.moe_tree_attention_workspace_size(4, 2, hq, 1, 64), dtype=torch.uint8, device="cuda")
    close(run_tree(*case, workspace=ws), *tree_ref(*case, 64 ** -0.5))
    seqs, pages, st = gbmoe.moe_read_tree_status(ws)
    assert seqs == 0 and pages >= 32 and st == 6


@pytest.mark.parametrize("hq", [2, 64])
def test_tree_attention_bad_lengths_are_counted(hq):
    case = list(make_tree([100, 30], [2, 2], hq, 1, 64, 16, BF, 14, "tree"))
    ws = torch.empty(gbmoe.moe_tree_attention_workspace_size(4, 2, hq, 1, 64), dtype=torch.uint8, device="cuda")
    good = run_tree(*case, workspace=ws)
    case[4] = [100, 10 ** 9]  # longer than its table: shortened
    got = run_tree(*case, workspace=ws)
    assert gbmoe.moe_read_tree_status(ws)[0] == 1
    assert torch.equal(got[:2], good[:2])
    case[4], case[5] = [100, 30], [0, 2, 900]  # offsets past the nodes: left out
    got = run_tree(*case, workspace=ws)
    assert gbmoe.moe_read_tree_status(ws)[0] == 1
    assert torch.equal(got[:2], good[:2])


@pytest.mark.parametrize("hq", [4, 40])
def test_tree_attention_in_a_graph_serves_other_lengths(hq):
    long, short = make_tree([300], [6], hq, 2, 64, 16, BF, 15, "tree"), make_tree([20], [6], hq, 2, 64, 16, BF, 16, "tree")
    table = torch.full((1, 20), -1, dtype=torch.int32, device="cuda")
    ctx, offs = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.tensor([0, 6], dtype=torch.int32, device="cuda")
    q, mask = torch.zeros(6, hq, 64, dtype=BF, device="cuda"), torch.zeros(6, dtype=torch.int64, device="cuda")
    kc, vc = (torch.zeros(30, 16, 2, 64, dtype=BF, device="cuda") for _ in range(2))
    out = torch.zeros_like(q)
    ws = torch.empty(gbmoe.moe_tree_attention_workspace_size(6, 1, hq, 2, 64), dtype=torch.uint8, device="cuda")

    def load(case):
        q.copy_(case[0])
        kc[:case[1].shape[0]].copy_(case[1])
        vc[:case[2].shape[0]].copy_(case[2])
        table.fill_(-1)
        table[:, :case[3].shape[1]].copy_(torch.from_numpy(case[3]))
        ctx.copy_(torch.tensor(case[4], dtype=torch.int32))
        mask.copy_(mask_tensor(case[6]))

    def call():
        gbmoe.moe_tree_attention(q, kc, vc, table, ctx, offs, mask, out=out, workspace=ws)

    load(long)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for case in (long, short, long):
        load(case)
        graph.replay()
        torch.cuda.synchronize()
        close(out, *tree_ref(*case, 64 ** -0.5))


# ------------------------------------------------------------------ draft verification
def probs(rows, V, seed, sharp=3.0):
    return torch.softmax(torch.randn(rows, V, generator=gen(seed)) * sharp, -1)


def check_verify(target, tokens, offs, coins, last, max_nodes, parents=None, draft=None):
    i32 = torch.int32
    got = gbmoe.moe_verify_draft(target.cuda(), torch.tensor(tokens, dtype=i32).cuda(), torch.tensor(offs, dtype=i32).cuda(),
                                 coins.cuda(), last.cuda(), max_nodes,
                                 None if parents is None else torch.tensor(parents, dtype=i32).cuda(),
                                 None if draft is None else draft.cuda())
    want = verify_ref(target, tokens, offs, coins, last, max_nodes, parents, draft)
    for g, w, name in zip(got, want, ("tokens", "path", "accepted")):
        assert np.array_equal(g.cpu().numpy(), w), (name, g.cpu().numpy(), w)
    return want


@pytest.mark.parametrize("B,n,V", [(1, 1, 2), (3, 5, 33), (4, 7, 1000), (40, 3, 2049), (2, 31, 32003), (700, 1, 64)])
def test_verify_chain(B, n, V):
    g = gen(V)
    r = np.random.default_rng(V)
    counts = [n] + [int(r.integers(0, n + 1)) for _ in range(B - 1)]
    N, offs = sum(counts), [0] + [int(x) for x in np.cumsum(counts)]
    target = probs(N + B, V, V)
    draft = torch.zeros(N, V)
    tokens = []
    for b in range(B):
        for j in range(counts[b]):
            d = target[offs[b] + b + j] * (0.2 + torch.rand(V, generator=g))
            draft[offs[b] + j] = d / d.sum()
            tokens.append(int(torch.multinomial(draft[offs[b] + j], 1, generator=g)))
    want = check_verify(target, tokens, offs, torch.rand(N + B, generator=g), torch.rand(B, generator=g), n, None, draft)
    assert B < 3 or (want[2] > 0).any()


@pytest.mark.parametrize("B,n,V,seed", [(1, 1, 5, 0), (3, 8, 40, 1), (2, 64, 700, 2), (30, 16, 3001, 3), (1, 24, 50001, 4)])
def test_verify_tree(B, n, V, seed):
    g, r = gen(seed), np.random.default_rng(seed)
    target = probs(B * (n + 1), V, seed, 4.0)
    parents, tokens = [], []
    for b in range(B):
        up = [int(r.integers(-1, max(j // 3, 1) + 0)) if j else -1 for j in range(n)]
        for j in range(n):
            rank = sum(up[i] == up[j] for i in range(j))
            row = target[b * (n + 1) + up[j] + 1]
            tokens.append(int(torch.topk(row, min(V, rank + 1)).indices[-1]) if r.random() < 0.8 else int(r.integers(0, V)))
        parents += up
    offs = list(range(0, B * n + 1, n))
    check_verify(target, tokens, offs, torch.rand(B * (n + 1), generator=g), torch.rand(B, generator=g), n, parents)


def test_verify_edges():
    V = 300
    target = probs(4, V, 7)
    coins, last = torch.zeros(4), torch.tensor([0.0])
    top = [int(i) for i in target.argmax(-1)]
    assert check_verify(target, top[:3], [0, 3], coins, last, 3)[2][0] == 3                # coin 0: all kept
    check_verify(target, top[:3], [0, 3], torch.full((4,), 1 - 2.0 ** -24), torch.tensor([1 - 2.0 ** -24]), 3)
    check_verify(target, [5, 5, 5], [0, 3], coins + 0.9, last + 0.5, 3, [-1, -1, -1])       # the same candidate three times
    assert check_verify(target[:1], [], [0, 0], coins[:1], last + 0.3, 0)[2][0] == 0        # no nodes: a plain sample
    hot = torch.zeros(2, V)
    hot[:, 9] = 1.0
    check_verify(hot, [9], [0, 1], coins[:2] + 0.5, last + 0.7, 1)                          # kept
    check_verify(hot, [8], [0, 1], coins[:2] + 0.5, last + 0.7, 1)                          # refused
    draft = torch.zeros(1, V)
    draft[0, 9] = 1.0
    check_verify(hot * 0.5, [9], [0, 1], coins[:2] + 0.9, last + 0.7, 1, None, draft)       # the residual is empty
    tiny = torch.full((2, V), 1e-30)
    assert check_verify(tiny, [3], [0, 1], coins[:2] + 0.5, last + 0.5, 1)[2][0] == -1      # no weight at all
    odd = probs(2, V, 8)
    odd[1, :50] = float("nan")
    odd[1, 50:60] = -1.0
    check_verify(odd, [int(odd[0].argmax())], [0, 1], coins[:2], last + 0.4, 1)


def test_verify_refuses_bad_sequences_alone():
    V, i32 = 100, torch.int32
    target = probs(9, V, 9)

    def call(tokens, offs, parents):
        return gbmoe.moe_verify_draft(target.cuda(), torch.tensor(tokens, dtype=i32).cuda(),
                                      torch.tensor(offs, dtype=i32).cuda(), torch.full((9,), 0.5).cuda(),
                                      torch.full((3,), 0.5).cuda(), 4, torch.tensor(parents, dtype=i32).cuda())

    out, path, acc = call([1, 2, 3, 4, 5, 6], [0, 2, 4, 6], [-1, 0, -1, 0, -1, 0])
    for tokens, offs, parents in (([1, 2, 3, V, 5, 6], [0, 2, 4, 6], [-1, 0, -1, 0, -1, 0]),
                                  ([1, 2, -1, 4, 5, 6], [0, 2, 4, 6], [-1, 0, -1, 0, -1, 0]),
                                  ([1, 2, 3, 4, 5, 6], [0, 2, 4, 6], [-1, 0, -1, 1, -1, 0]),
                                  ([1, 2, 3, 4, 5, 6], [0, 2, 4, 6], [-1, 0, -2, 0, -1, 0])):
        o, p, a = call(tokens, offs, parents)
        assert a[1] == -1 and (o[1] == -1).all() and (p[1] == -1).all()
        assert torch.equal(o[[0, 2]], out[[0, 2]]) and torch.equal(a[[0, 2]], acc[[0, 2]])
    assert call([1, 2, 3, 4, 5, 6], [0, 2, 1, 6], [-1, 0, -1, 0, -1, 0])[2].tolist()[1:] == [-1, -1]
    assert call([1, 2, 3, 4, 5, 6], [0, 2, 4, 7], [-1, 0, -1, 0, -1, 0])[2].tolist()[2] == -1


# ------------------------------------------------------------------ streams
def test_operators_follow_the_current_stream():
    s = torch.cuda.Stream()
    g = gen(30)
    x = torch.randn(2, 512, generator=g).to(BF)
    w = torch.randint(0, 256, (64, 256), generator=g, dtype=torch.uint8)
    sc = torch.rand(64, 4, generator=g)
    xd, wd, sd = torch.zeros(2, 512, dtype=BF, device="cuda"), w.cuda(), sc.cuda()
    xp = x.pin_memory()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)
        xd.copy_(xp, non_blocking=True)
        y = gbmoe.moe_linear_int4(xd, wd, sd)
    s.synchronize()
    close(y, *linear_ref(x, w, sc, False))


# ------------------------------------------------------------------ the binding's refusals
def test_bindings_refuse_wrong_tensors():
    x, w = torch.zeros(2, 256, dtype=BF, device="cuda"), torch.zeros(8, 128, dtype=torch.uint8, device="cuda")
    s = torch.zeros(8, 2, device="cuda")
    for bad in (lambda: gbmoe.moe_linear_int4(x.float(), w, s), lambda: gbmoe.moe_linear_int4(x, w[:, :64], s),
                lambda: gbmoe.moe_linear_int4(x, w, s.cpu()), lambda: gbmoe.moe_linear_int4(x, w, s[:7]),
                lambda: gbmoe.moe_linear_int4(x.T, w, s), lambda: gbmoe.moe_linear_int4(x, w[:7], s[:7], True),
                lambda: gbmoe.moe_linear_int4(x, w, s, out=torch.zeros(2, 9, dtype=BF, device="cuda")),
                lambda: gbmoe.moe_linear_int4(x, w, None)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(gbmoe.MoEError) as e:  # a group size of 8
        gbmoe.moe_linear_int4(x, w, torch.zeros(8, 32, device="cuda"))
    assert e.value.status == 2 and "group" in str(e.value)
    with pytest.raises(gbmoe.MoEError) as e:  # a workspace that is too small
        gbmoe.moe_linear_int4(torch.zeros(20, 256, dtype=BF, device="cuda"), w, s,
                              workspace=torch.zeros(256, dtype=torch.uint8, device="cuda"))
    assert e.value.status == 3
    q, pos = torch.zeros(3, 2, 64, dtype=BF, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda")
    f, _ = gbmoe.rope_frequencies(64)
    for bad in (lambda: gbmoe.moe_rope(q, None, pos.long(), f), lambda: gbmoe.moe_rope(q, None, pos[:2], f),
                lambda: gbmoe.moe_rope(q, None, pos, f.float()), lambda: gbmoe.moe_rope(q, q[:, :, :32], pos, f),
                lambda: gbmoe.moe_rope(q.transpose(1, 2), None, pos, f), lambda: gbmoe.moe_rope(q[0], None, pos, f)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(gbmoe.MoEError):  # a turning part wider than the head
        gbmoe.moe_rope(q[..., :32], None, pos, f)
    cache = torch.zeros(4, 16, 1, 64, dtype=BF, device="cuda")
    table, one = torch.zeros(1, 4, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    offs = torch.tensor([0, 3], dtype=torch.int32, device="cuda")
    for bad in (lambda: gbmoe.moe_tree_attention(q, cache.half(), cache, table, one, offs),
                lambda: gbmoe.moe_tree_attention(q, cache, cache[:3], table, one, offs),
                lambda: gbmoe.moe_tree_attention(q, cache, cache, table.long(), one, offs),
                lambda: gbmoe.moe_tree_attention(q, cache, cache, table, one, offs[:1]),
                lambda: gbmoe.moe_tree_attention(q, cache, cache, table, one, offs, pos)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(gbmoe.MoEError):  # 2 query heads cannot share 3 KV heads
        gbmoe.moe_tree_attention(q, torch.zeros(4, 16, 3, 64, dtype=BF, device="cuda"),
                                 torch.zeros(4, 16, 3, 64, dtype=BF, device="cuda"), table, one, offs)


def test_empty_calls_return_empty_results():
    f, _ = gbmoe.rope_frequencies(64)
    z = torch.zeros(0, dtype=torch.int32, device="cuda")
    q, k = gbmoe.moe_rope(torch.zeros(0, 2, 64, dtype=BF, device="cuda"), None, z, f)
    assert q.shape == (0, 2, 64) and k is None
    w, s = torch.zeros(8, 128, dtype=torch.uint8, device="cuda"), torch.zeros(8, 2, device="cuda")
    assert gbmoe.moe_linear_int4(torch.zeros(0, 256, dtype=FP, device="cuda"), w, s).shape == (0, 8)
    cache = torch.zeros(4, 16, 1, 64, dtype=BF, device="cuda")
    out = gbmoe.moe_tree_attention(torch.zeros(0, 2, 64, dtype=BF, device="cuda"), cache, cache, z.view(0, 4), z,
                                   torch.zeros(1, dtype=torch.int32, device="cuda"))
    assert out.shape == (0, 2, 64)
    out, path, acc = gbmoe.moe_verify_draft(torch.zeros(0, 9, device="cuda"), z, torch.zeros(1, dtype=torch.int32, device="cuda"),
                                            z.float(), z.float(), 3)
    assert out.shape == (0, 4) and path.shape == (0, 3) and acc.shape == (0,)
