"""GPU parity of the head norms and of attention over an E4M3 cache where a warp or a CTA works through many rounds, tiles and
pieces: prompts, long sequences.  The references are computed in 64 bits on the GPU."""
import numpy as np
import pytest
import torch

from _more_ops import EPS24, e4m3, quantised, rounded
from _step_ops import HALF, TINY, mask_tensor
from mixture_experts_ffn_moe_gb300 import build, gbmoe
from test_gpu_more_ops import BF, F32, FP, I32, U8, tree_masks

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()
    return gbmoe.load()


def rng(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def near(got, ref, bound, what=""):
    bad = ~((got.double() - ref).abs() <= bound)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} outside, first at {bad.nonzero()[0].tolist()}"


# ------------------------------------------------------------------ norms of heads
def norms_and_turns(x, weight, pos, f, inter, offset):
    """norm_ref of tests/_more_ops.py, with eps 1e-6 and a scale of 1, on the GPU."""
    d, dim = x.double(), x.shape[-1]
    d = d / torch.sqrt(d.square().mean(-1, keepdim=True) + 1e-6) * weight.double()
    rel = (max(32, dim / 32) / 2 + 3 + 2 + 4 + 4 + 2) * EPS24
    ang = pos.cpu().numpy().astype(np.longdouble)[:, None] * f.cpu().numpy().astype(np.longdouble)
    ang = np.fmod(ang, 2 * np.longdouble("3.14159265358979323846264338327950288"))
    c, s = (torch.from_numpy(t.astype(np.float64)).cuda()[:, None] for t in (np.cos(ang), np.sin(ang)))
    rot = 2 * len(f)
    if inter:
        i0, i1 = slice(offset, offset + rot, 2), slice(offset + 1, offset + rot, 2)
    else:
        i0, i1 = slice(offset, offset + rot // 2), slice(offset + rot // 2, offset + rot)
    y, err = d.clone(), d.abs() * rel
    a, b = d[..., i0], d[..., i1]
    y[..., i0], y[..., i1] = a * c - b * s, b * c + a * s
    slack = (a.abs() + b.abs()) * (2.0 ** -20 + rel)
    err[..., i0], err[..., i1] = slack, slack
    return y, err


PROMPTS = [
    # tokens, q heads, k heads, D, rot, offset, interleaved, type: 4 and more rounds a warp
    (4096, 64, 4, 128, 128, 0, False, BF),
    (8001, 7, 3, 128, 64, 32, False, FP),        # heads that do not fill their rounds, q, k and v in one piece
    (8001, 5, 1, 64, 64, 0, True, F32),
    (5001, 9, 3, 22, 6, 4, True, BF),            # pairs of elements, more than one head a warp
    (4001, 5, 2, 21, 6, 3, False, FP),           # single elements
    (6001, 3, 1, 1024, 512, 0, False, F32),      # more than one vector a lane
]


def prompt(T, hq, hk, D, rot, off, inter, dt):
    """A projection's rows on the GPU, weights, positions, frequencies; a warp gets several rounds of heads."""
    vec = 16 // dt.itemsize
    vec = vec if D % vec == 0 and rot // 2 % vec == 0 and off % vec == 0 else 2 if inter else 1
    units = D // vec if inter else (D - rot // 2) // vec
    step = 32 // min(32, 1 << (units - 1).bit_length())   # heads of a round
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert T * (-(-hq // step) + -(-hk // step)) >= 3 * 48 * sms
    g = rng(T + D)
    qkv = (torch.randn(T, hq + 2 * hk, D, generator=g, device="cuda") * 3).to(dt)
    w = [(1 + 0.5 * torch.randn(D, generator=g, device="cuda")).to(dt) for _ in "qk"]
    pos = torch.randint(0, 100000, (T,), generator=g, device="cuda").to(I32)
    f, _ = gbmoe.rope_frequencies(rot)
    return qkv, w, pos, f


@pytest.mark.parametrize("T,hq,hk,D,rot,off,inter,dt", PROMPTS)
def test_norm_rope_of_a_prompt_in_place(T, hq, hk, D, rot, off, inter, dt):
    qkv, w, pos, f = prompt(T, hq, hk, D, rot, off, inter, dt)
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
    want = [norms_and_turns(x, wt, pos, f, inter, off) for x, wt in ((q, w[0]), (k, w[1]))]
    old = v.clone()
    apart = gbmoe.moe_qk_norm_rope(q, k, pos, f, *w, interleaved=inter, offset=off)
    gbmoe.moe_qk_norm_rope(q, k, pos, f, *w, interleaved=inter, offset=off, q_out=q, k_out=k)
    for got, other, (y, err), what in zip((q, k), apart, want, "qk"):
        near(got, y, rounded(y, err, dt), what)
        assert torch.equal(got, other)
    assert torch.equal(v, old)


@pytest.mark.parametrize("codes", [False, True])
@pytest.mark.parametrize("T,hq,hk,D,rot,off,inter,dt", PROMPTS)
def test_norm_rope_append_of_a_prompt(T, hq, hk, D, rot, off, inter, dt, codes):
    qkv, w, pos, f = prompt(T, hq, hk, D, rot, off, inter, dt)
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
    page = 24
    pages = -(-T // page) + 3
    slots = torch.randperm(pages * page, generator=rng(1), device="cuda")[:T].to(I32)
    slots[::7] = -1
    slots[5] = pages * page
    kept = (slots >= 0) & (slots < pages * page)
    at = slots[kept].long()
    kind = U8 if codes else dt
    kc, vc = (torch.full((pages, page, hk, D), 7, dtype=kind, device="cuda") for _ in "kv")
    ks, vs = (torch.full((pages, page, hk), 5.0, device="cuda") for _ in "kv")
    more = {"k_scale": ks, "v_scale": vs} if codes else {}
    qo = gbmoe.moe_qk_norm_rope_append(q, k, v, pos, f, slots, kc, vc, *w, interleaved=inter, offset=off, **more)
    y, err = norms_and_turns(q, w[0], pos, f, inter, off)
    near(qo, y, rounded(y, err, dt), "q")
    y, err = (t[kept] for t in norms_and_turns(k, w[1], pos, f, inter, off))
    kf, vf, ksf, vsf = kc.view(-1, hk, D), vc.view(-1, hk, D), ks.view(-1, hk), vs.view(-1, hk)
    if codes:
        top, i = y.abs().max(-1)
        e = err.gather(2, i[..., None])[..., 0] + err.amax(-1)
        assert ((ksf[at].double() * 448 - top).abs() <= e + top * 2.0 ** -23).all()
        # half a step of E4M3 (2^-4 of the value, 2^-10 of the scale below 2^-6) and what y was off before
        half = torch.maximum(y.abs() * 2.0 ** -4, ksf[at].double()[..., None] * 2.0 ** -10)
        near(e4m3(kf[at]) * ksf[at].double()[..., None], y, (half + 2 * err) * (1 + 2.0 ** -20), "key codes")
        code, scale = (t.cuda() for t in quantised(v[kept].float().cpu()))  # (on the GPU torch multiplies by 1 / 448)
        assert torch.equal(vf[at] & 127, code & 127) and torch.equal(vsf[at], scale)  # (a code of 0 may keep its sign)
    else:
        near(kf[at], y, rounded(y, err, dt), "keys")
        assert torch.equal(vf[at], v[kept])
    rest = torch.ones(pages * page, dtype=torch.bool, device="cuda")
    rest[at] = False
    assert (kf[rest] == 7).all() and (vf[rest] == 7).all() and (ksf[rest] == 5.0).all() and (vsf[rest] == 5.0).all()


# ------------------------------------------------------------------ attention over codes
def long_cache(lens, counts, hk, D, page, heads_first, shape, seed):
    """Codes and scales on the GPU whose scores and value scales grow along every sequence ("up"), or fall, so that a row's reference
    moves often, or stands from the start; block table."""
    need = [-(-(n + c) // page) for n, c in zip(lens, counts)]
    pool = sum(need) + 3
    order = np.random.default_rng(seed).permutation(pool)
    table = np.full((len(lens), max(need)), -1, dtype=np.int32)
    size = torch.zeros(pool, page)
    at = 0
    for b, p in enumerate(need):
        table[b, :p] = order[at:at + p]
        along = torch.linspace(0, 1, p * page).view(p, page)
        size[torch.from_numpy(order[at:at + p])] = along if shape == "up" else 1 - along
        at += p
    size = size.cuda()[..., None]
    g, side = rng(seed), []
    for name in "kv":
        # keys: scores of a size from 0.05 to 6; values: sizes from 2^-10 to 2^10
        amount = 0.05 + 6 * size if name == "k" else torch.exp2(20 * size - 10)
        amount = amount * torch.exp2(torch.randint(-1, 2, (pool, page, hk), generator=g, device="cuda").float())
        codes = torch.empty(pool, page, hk, D, dtype=U8, device="cuda")
        scale = torch.empty(pool, page, hk, device="cuda")
        for h in range(hk):
            x = torch.randn(pool, page, D, generator=g, device="cuda") * amount[:, :, h, None]
            codes[:, :, h], scale[:, :, h] = quantised(x)
        if heads_first:
            codes, scale = codes.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3), scale.permute(0, 2, 1).contiguous().permute(0, 2, 1)
        side.append((codes, scale))
    return side, torch.from_numpy(table).cuda()


def long_ref(q, side, table, lens, counts, masks):
    """fp8_tree_ref of tests/_more_ops.py, sequence by sequence and head by head on the GPU."""
    (kc, ks), (vc, vs) = side
    page, hk, (N, hq, D) = kc.shape[1], kc.shape[2], q.shape
    g, scale = hq // hk, q.shape[2] ** -0.5
    out, bound = (torch.zeros(N, hq, D, dtype=torch.float64, device="cuda") for _ in range(2))
    lo = 0
    for b, (n, c) in enumerate(zip(lens, counts)):
        slots = torch.arange(n + c, device="cuda")
        pg, at = table[b].long()[slots // page], slots % page
        hide = torch.zeros(c, n + c, dtype=torch.bool)
        for j in range(c):
            m = masks[lo + j] if masks is not None else (2 << j) - 1
            hide[j, n:] = torch.tensor([not (m >> i) & 1 for i in range(c)])
        hide = hide.cuda()[:, None]
        for h in range(hk):
            k = e4m3(kc[pg, at, h]) * ks[pg, at, h].double()[:, None]
            vscale, code = vs[pg, at, h].double(), e4m3(vc[pg, at, h])
            v, all_codes = code * vscale[:, None], code.abs().sum(0)
            for j in range(0, c, 8):
                x = q[lo + j:lo + min(j + 8, c), h * g:(h + 1) * g].double()
                hidden = hide[j:j + 8]
                p = torch.softmax((x @ k.T * scale).masked_fill_(hidden, -torch.inf), -1)
                ds = ((x.abs() @ k.abs().T) * scale * (D / 16 + 6) * 2.0 ** -22).masked_fill_(hidden, 0.0).amax(-1, keepdim=True) + 66 * 2.0 ** -22
                o, av = p @ v, p @ v.abs()
                small = (p * vscale).amax(-1, keepdim=True) * 2.0 ** -32 * all_codes
                rows = slice(lo + j, lo + min(j + 8, c))
                out[rows, h * g:(h + 1) * g] = o
                bound[rows, h * g:(h + 1) * g] = ((2.0 ** -11 + 3 * ds + 2.0 ** -18) * av * 1.01 + small + o.abs() * HALF[q.dtype] + TINY[q.dtype])
        lo += c
    return out, bound


def places_a_cta(ws, batch):
    """Of the line of tiles, from the workspace: the header (482 words), then the places of the sequences and this."""
    return int(ws[2048:2048 + 8 * (batch + 2)].view(torch.int64)[batch + 1])


def check_long(lens, counts, hq, hk, D, page, dt, heads_first, shape, masked, least):
    seed = sum(lens) + D + page
    side, table = long_cache(lens, counts, hk, D, page, heads_first, shape, seed)
    q = torch.randn(sum(counts), hq, D, generator=rng(seed + 1), device="cuda").to(dt)
    masks = tree_masks(counts, seed) if masked else None
    (kc, ks), (vc, vs) = side
    offs = torch.tensor([0] + list(np.cumsum(counts)), dtype=I32).cuda()
    ws = torch.full((gbmoe.moe_tree_attention_fp8_workspace_size(len(q), len(lens), hq, hk, D),), 255, dtype=U8, device="cuda")
    got = gbmoe.moe_tree_attention_fp8(q, kc, vc, ks, vs, table, torch.tensor(lens, dtype=I32).cuda(), offs,
                                       None if masks is None else mask_tensor(masks).cuda(), workspace=ws)
    assert gbmoe.moe_read_tree_status(ws) == (0, 0, 0)
    assert places_a_cta(ws, len(lens)) >= least
    ref, bound = long_ref(q, side, table, lens, counts, masks)
    near(got, ref, bound)
    again = gbmoe.moe_tree_attention_fp8(q, kc, vc, ks, vs, table, torch.tensor(lens, dtype=I32).cuda(), offs,
                                         None if masks is None else mask_tensor(masks).cuda())
    assert torch.equal(got, again)


@pytest.mark.parametrize("shape", ["up", "down"])
@pytest.mark.parametrize("lens,counts,hq,hk,D,page,dt,heads_first,masked", [
    ([110000, 50001, 7000], [1, 1, 1], 32, 8, 128, 16, BF, False, False),           # 8 rows
    ([200000, 120003, 9000], [4, 3, 4], 16, 4, 128, 48, FP, False, True),           # 16 rows, pages of three runs
    ([300000, 130001, 20000], [16, 8, 8], 8, 2, 128, 5, BF, False, True),           # 32 rows, two row tiles, odd pages
    ([200000, 130007, 5000], [1, 1, 1], 16, 4, 64, 24, FP, False, False),           # two KV heads side by side, odd pages
    ([400000, 250001, 20000], [4, 4, 4], 8, 2, 64, 16, BF, True, False),            # one of them, heads first
    ([300000, 140001, 6000], [8, 8, 8], 8, 2, 64, 32, FP, False, True)])            # two, 32 rows
def test_fp8_attention_of_long_sequences(lens, counts, hq, hk, D, page, dt, heads_first, masked, shape):
    """A CTA walks over more than 40 tiles: stages in turn, pages looked up 32 tiles at once, references that move, several pieces."""
    check_long(lens, counts, hq, hk, D, page, dt, heads_first, shape, masked, 44)


@pytest.mark.parametrize("shape", ["up", "down"])
@pytest.mark.parametrize("lens,counts,hq,hk,D,page,dt,heads_first", [
    ([60000, 300, 50001, 1, 17, 200, 9000], [32, 27, 30, 20, 30, 28, 32], 16, 2, 128, 16, BF, False),   # up to 256 rows
    ([90000, 300, 70001, 10, 9000], [16, 12, 16, 16, 15], 16, 2, 64, 5, FP, False),                     # one half, odd pages
    ([80000, 70001, 500, 90], [64, 60, 50, 64], 8, 1, 64, 24, BF, True),                                # two CTAs side by side
    ([50000, 30001, 700], [64, 64, 61], 16, 1, 128, 64, FP, False)])                                    # four
def test_fp8_attention_of_wide_trees_over_long_sequences(lens, counts, hq, hk, D, page, dt, heads_first, shape):
    """More than 8 tiles a CTA in the tcgen05 kernel: stages, parities and scales in turn, moved references, several pieces."""
    check_long(lens, counts, hq, hk, D, page, dt, heads_first, shape, True, 13)
