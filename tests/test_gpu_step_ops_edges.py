"""GPU tests of the decode-step operators where inputs are unusual but valid, or wrong in a way that a call has to
notice: broadcast and padded rows, probabilities outside [0, 1], weights far below a row's largest, bad offsets."""
import numpy as np
import pytest
import torch

from _step_ops import HALF, TINY, int4_values, mask_tensor, rope_ref, tree_ref, verify_ref
from mixture_experts_ffn_moe_gb300 import build, gbmoe
from test_gpu_step_ops import _dev, close, make_tree

pytestmark = pytest.mark.gpu

BF, FP, F32, I32 = torch.bfloat16, torch.float16, torch.float32, torch.int32


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()
    return gbmoe.load()


def gen(seed):
    return torch.Generator().manual_seed(seed)


# ------------------------------------------------------------------ draft verification
def probs(rows, V, seed, sharp=3.0):
    return torch.softmax(torch.randn(rows, V, generator=gen(seed)) * sharp, -1)


def verify(target, tokens, offs, coins, last, max_nodes, parents=None, draft=None):
    return gbmoe.moe_verify_draft(target, torch.tensor(tokens, dtype=I32).cuda(), torch.tensor(offs, dtype=I32).cuda(),
                                  coins.cuda(), last.cuda(), max_nodes,
                                  None if parents is None else torch.tensor(parents, dtype=I32).cuda(), draft)


def same(got, want):
    for g, w, name in zip(got, want, ("tokens", "path", "accepted")):
        assert np.array_equal(g.cpu().numpy(), np.asarray(w)), (name, g.cpu().numpy(), w)


@pytest.mark.parametrize("B,n,V", [(12, 5, 40000), (40, 3, 9001), (300, 2, 5000)])
def test_verify_in_clusters_with_refused_sequences_among_them(B, n, V):
    """Clusters of 8, 4 and 1 CTAs, replayed from a graph: kept and refused sequences, rows without weight and rows that
    are no probabilities leave their barriers alike, and every replay gives the same."""
    g = gen(B)
    target = probs(B * (n + 1), V, B)
    target[5 * (n + 1):6 * (n + 1)] = 0.0                 # no weight
    target[7 * (n + 1):8 * (n + 1)] = 0.5                 # sums far above 1
    tokens = target.view(B, n + 1, V)[:, :n].argmax(-1)
    tokens[3, 1] = V                                      # no such token
    coins, last = torch.rand(B * (n + 1), generator=g), torch.rand(B, generator=g)
    offs = list(range(0, B * n + 1, n))
    keep = [b for b in range(B) if b not in (3, 5, 7)]
    rows = torch.cat([torch.arange(b * (n + 1), (b + 1) * (n + 1)) for b in keep])
    want = verify_ref(target[rows], tokens[keep].flatten().tolist(), offs[:len(keep) + 1], coins[rows], last[keep], n)
    args = (target.cuda(), tokens.to(I32).flatten().cuda(), torch.tensor(offs, dtype=I32).cuda(), coins.cuda(), last.cuda(), n)
    gbmoe.moe_verify_draft(*args)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        results = [gbmoe.moe_verify_draft(*args) for _ in range(4)]
    for _ in range(20):
        graph.replay()
    torch.cuda.synchronize()
    for got in results:
        same([t[keep] for t in got], want)
        assert got[2][[3, 5, 7]].tolist() == [-1, -1, -1] and (got[0][[3, 5, 7]] == -1).all()


@pytest.mark.parametrize("V,pad", [(64, 4), (64, 3), (33, 7)])
def test_verify_reads_padded_rows(V, pad):
    g, offs = gen(V + pad), [0, 3, 5]
    target, draft = probs(7, V, 1), probs(5, V, 2)
    tokens = [int(row.argmax()) for row in draft]
    coins, last = torch.rand(7, generator=g), torch.rand(2, generator=g)
    wide_t, wide_d = torch.full((7, V + pad), 9.0, device="cuda"), torch.full((5, V + pad), 9.0, device="cuda")
    wide_t[:, :V], wide_d[:, :V] = target.cuda(), draft.cuda()
    same(verify(wide_t[:, :V], tokens, offs, coins, last, 3, None, wide_d[:, :V]),
         verify_ref(target, tokens, offs, coins, last, 3, None, draft))


@pytest.mark.parametrize("stride", [0, 1, 32, 63])
def test_verify_refuses_rows_that_overlap(stride):
    """A broadcast row (stride 0) or rows less than a vocabulary apart.  (The storage behind each view is as large as
    rows a vocabulary apart would be, so that no reading of the strides leaves it.)"""
    V, coins, last = 64, torch.full((4,), 0.5), torch.full((1,), 0.5)
    rows = probs(4, V, 3).cuda()
    view = rows.as_strided((4, V), (stride, 1))
    with pytest.raises(gbmoe.MoEError, match="row stride") as e:
        verify(view, [1, 2, 3], [0, 3], coins, last, 3)
    assert e.value.status == 1
    with pytest.raises(gbmoe.MoEError, match="row stride") as e:
        verify(rows, [1, 2, 3], [0, 3], coins, last, 3, None, view[:3])
    assert e.value.status == 1


def test_verify_takes_a_single_row_of_any_stride():
    V = 64
    target, draft = probs(2, V, 4), probs(1, V, 5)
    coins, last = torch.tensor([0.9, 0.3]), torch.tensor([0.4])
    one = draft.cuda().as_strided((1, V), (0, 1))
    same(verify(target.cuda(), [7], [0, 1], coins, last, 1, None, one),
         verify_ref(target, [7], [0, 1], coins, last, 1, None, draft))
    row = target[:1].cuda().as_strided((1, V), (1, 1))
    same(verify(row, [], [0, 0], coins[:1], last, 0), verify_ref(target[:1], [], [0, 0], coins[:1], last, 0))


# ------------------------------------------------------------------ tree attention
@pytest.mark.parametrize("hq,nodes,page", [(2, 3, 16), (2, 3, 5), (8, 6, 16), (8, 6, 5), (32, 8, 16), (32, 8, 5)])
@pytest.mark.parametrize("dt,D", [(FP, 128), (FP, 64), (BF, 128)])
def test_tree_attention_weights_far_below_a_rows_largest(hq, nodes, page, dt, D):
    """Every 16th slot outweighs the others by about 2^25 and has a value of zero: what the result is made of are the small
    weights, which have to reach the product with V with their bits."""
    (q, kc, vc, table, ctx, offs, masks), r = make_tree([300], [nodes], hq, 1, D, page, dt, 41, None), gen(42)
    L = 300 + nodes
    base = torch.randn(D, generator=r)
    q = (base + 0.05 * torch.randn(nodes, hq, D, generator=r)).to(dt)
    top = base / (base @ base) * (25.0 * np.log(2.0) * D ** 0.5)
    for s in range(L):
        at = (table[0, s // page], s % page)
        kc[at] = (top if s % 16 == 5 else 0.02 * torch.randn(D, generator=r)).to(dt)
        vc[at] = (torch.zeros(D) if s % 16 == 5 else 4000.0 * (0.5 + torch.rand(D, generator=r))).to(dt)
    ref, bound = tree_ref(q, kc, vc, table, ctx, offs, masks, D ** -0.5)
    if dt == FP:
        # P stands with 2^7 on top of a row's reference, which is at most its largest score: half a subnormal step of
        # 2^-25 is 2^-32 of the largest weight, a slot; the sinks (one in 16 slots) carry the sum
        sinks = sum(s % 16 == 5 for s in range(300))
        bound = bound + L * 6000.0 * 2.0 ** -32 * 4 / sinks  # (their scores differ by less than 2 powers of two)
    got = gbmoe.moe_tree_attention(q.cuda(), _dev(kc), _dev(vc), torch.from_numpy(table).cuda(), torch.tensor(ctx, dtype=I32).cuda(),
                                   torch.tensor(offs, dtype=I32).cuda())
    assert (ref > 8 * bound).all()
    close(got, ref, bound)


def test_verify_counts_probabilities_outside_0_and_1_alike_everywhere():
    """At the drafted token: NaN and negative values count as 0 and values above 1 as 1, in the test of acceptance as
    in the sample."""
    V, odd = 40, [float("nan"), -0.5, 0.0, 0.3, 2.0, 3.0]
    pairs = [(p, q) for p in odd for q in odd]
    B = len(pairs)
    target, draft = probs(2 * B, V, 11), probs(B, V, 12)
    tokens = [(7 * b) % V for b in range(B)]
    for b, (p, q) in enumerate(pairs):
        target[2 * b, tokens[b]] = p
        draft[b, tokens[b]] = q
    last = torch.rand(B, generator=gen(13))
    for coin in (0.0, 0.7):
        coins = torch.full((2 * B,), coin)
        plain = [x.nan_to_num(nan=0.0).clamp(0.0, 1.0) for x in (target, draft)]
        want = verify_ref(plain[0], tokens, list(range(B + 1)), coins, last, 1, None, plain[1])
        assert 0 < want[2].sum() < B
        same(verify(target.cuda(), tokens, list(range(B + 1)), coins, last, 1, None, draft.cuda()), want)


def test_verify_children_past_the_end_of_the_shares_are_never_kept():
    """Shares that add up to 16 and more (a root row that is no distribution): only what lies in [0, 1) can hold a coin."""
    V, n = 100, 40
    target = probs(n + 1, V, 14)
    for value, coin, kept in ((1.0, 0.25, 0), (0.9, 0.95, 1), (0.4, 0.9, 2)):
        target[0] = 0.0
        target[0, :n] = value
        coins, last = torch.full((n + 1,), coin), torch.tensor([0.6])
        want = verify_ref(target, list(range(n)), [0, n], coins, last, n, [-1] * n)
        assert want[2][0] == 1 and want[1][0, 0] == kept
        same(verify(target.cuda(), list(range(n)), [0, n], coins, last, n, [-1] * n), want)


@pytest.mark.parametrize("hq", [4, 64])
@pytest.mark.parametrize("before", [0, 40])
def test_tree_attention_joins_sequences_beside_bad_offsets(hq, before):
    """Cut units of good sequences are joined whatever the offsets of the others are; rows of bad ones stay as they are."""
    ctx, counts = [10] * before + [4000, 20, 4000], [1] * before + [4, 4, 4]
    q, kc, vc, table, ctx, offs, masks = make_tree(ctx, counts, hq, 2, 64, 16, BF, 31)
    ref, bound = tree_ref(q, kc, vc, table, ctx, offs, masks, 64 ** -0.5)
    b = before + 2                                       # a sequence more, between the last two: [.., o + 4, -5, o + 8, ..]
    table = np.insert(table, b, table[before], 0)
    ctx, offs = ctx[:b] + [50] + ctx[b:], offs[:b] + [-5] + offs[b:]
    N = q.shape[0]
    out = torch.full(q.shape, 7.0, dtype=BF, device="cuda")
    ws = torch.empty(gbmoe.moe_tree_attention_workspace_size(N, len(ctx), hq, 2, 64), dtype=torch.uint8, device="cuda")
    gbmoe.moe_tree_attention(q.cuda(), _dev(kc), _dev(vc), torch.from_numpy(table).cuda(), torch.tensor(ctx, dtype=I32).cuda(),
                             torch.tensor(offs, dtype=I32).cuda(), mask_tensor(masks).cuda(), out=out, workspace=ws)
    good = [i for i in range(N) if not before + 4 <= i < before + 8]
    close(out[good], ref[good], bound[good])
    assert (out[before + 4:before + 8] == 7.0).all()
    assert gbmoe.moe_read_tree_status(ws)[0] == 2


# ------------------------------------------------------------------ rotary positions
@pytest.mark.parametrize("inter", [False, True])
def test_rope_of_unit_vectors_is_right_to_the_last_bits(inter):
    """Sines and cosines themselves, of any size: an angle keeps its bits near every quarter of a turn and near zero."""
    f = torch.tensor([2.0 ** -40, 1e-9, 3e-7, 1e-4, 0.37, 1.0, np.pi / 2, np.pi / 2 + 1e-6, 1.5, 100.25, np.pi, 2 * np.pi,
                      np.pi / 4, np.nextafter(np.pi / 4, 0.0), np.nextafter(np.pi / 4, 1.0)], dtype=torch.float64)
    half, pos = len(f), torch.tensor([0, 1, 2, 3, 7, -1, -1000, 4096, 99991, 1 << 20, 2 ** 31 - 1], dtype=I32)
    x = torch.zeros(len(pos), 2, 2 * half)
    first = slice(0, 2 * half, 2) if inter else slice(0, half)
    second = slice(1, 2 * half, 2) if inter else slice(half, 2 * half)
    x[:, 0, first] = 1.0                                  # (cos, sin)
    x[:, 1, second] = 1.0                                 # (-sin, cos)
    got = gbmoe.moe_rope(x.cuda(), None, pos.cuda(), f.cuda(), interleaved=inter)[0].double().cpu()
    ref, _ = rope_ref(x, pos, f, 1.0, inter, False, 0)
    # the angle as a 64-bit fraction of a turn: 2^-52 of it (the frequency's conversion) and 2^-62 a position; then the
    # rest to a quarter turn as fp32 (two roundings of 2^-24 of it), sine and cosine (a unit of the last place, 2^-23);
    # the scale, the product with 1 and the sum with 0 are exact
    phase = (pos.double().abs()[:, None] * (f * 2.0 ** -52 + 2.0 ** -62)).repeat(1, 2) if not inter else \
        (pos.double().abs()[:, None] * (f * 2.0 ** -52 + 2.0 ** -62)).repeat_interleave(2, 1)
    close(got, ref, ref.abs() * 4 * 2.0 ** -24 + phase[:, None])


# ------------------------------------------------------------------ 4-bit linear
@pytest.mark.parametrize("M,N,K,group", [(1, 40, 512, 128), (8, 33, 256, 32), (16, 64, 1024, 64), (40, 70, 640, 128), (33, 40, 320, 64), (64, 40, 96, 32)])
@pytest.mark.parametrize("dt", [BF, FP])
def test_linear_int4_with_activations_that_stand_out(M, N, K, group, dt):
    """A column of every block is 2^12 times the others and meets codes of zero and others: the bound follows what the kernels
    compute, sums of x (q + 8) less 8 sums of x, both in fp32."""
    g = gen(M + K)
    x = torch.randn(M, K, generator=g).to(dt)
    x[:, 5::128] = (4096.0 * (1.0 + torch.rand(M, (K + 122) // 128, generator=g))).to(dt)
    w = torch.randint(0, 256, (N, K // 2), generator=g, dtype=torch.uint8)
    w[: N // 2, 2::64] &= 15                              # column 5 is a high nibble: zero for the first rows
    s = (0.5 + torch.rand(N, K // group, generator=g)) * 0.05
    q, sc = int4_values(w), s.double().repeat_interleave(group, 1)
    xd = x.double()
    ref = xd @ (q * sc).T
    # products are exact; x (q + 8) and 8 x in at most K / 16 steps each, off by 2^-22 (the steps may truncate) of the
    # absolute sums; x itself by 2^-35 of its block's largest
    err = (xd.abs() @ ((q + 8 + 8) * sc).T) * (16 + K / 128) * 2.0 ** -22
    top = xd.abs().amax(1, keepdim=True) @ (q.abs() * sc).sum(1)[None] * 2.0 ** -35
    close(gbmoe.moe_linear_int4(x.cuda(), w.cuda(), s.cuda()), ref, err + top + ref.abs() * HALF[dt] + TINY[dt])
