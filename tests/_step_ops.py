"""Plain 64-bit forms of the decode-step operators (rotary positions, 4-bit linear, tree attention, draft
verification), each with the error bound that its arithmetic allows."""
import math

import numpy as np
import torch

HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}  # half a step
TINY = {torch.bfloat16: 1e-38, torch.float16: 2.0 ** -25, torch.float32: 1e-38}  # half a step of subnormals


def rope_ref(x, positions, inv_freq, scale, interleaved, inverse, offset):
    """x [T, H, D] -> (turned, bound).  Angles in long double (64 significant bits on x86, 113 on Arm)."""
    rot = 2 * len(inv_freq)
    ang = positions.numpy().astype(np.longdouble)[:, None] * inv_freq.numpy().astype(np.longdouble)
    ang = np.fmod(ang, 2 * np.longdouble("3.14159265358979323846264338327950288"))
    c = torch.from_numpy(np.cos(ang).astype(np.float64))[:, None] * scale
    s = torch.from_numpy(np.sin(ang).astype(np.float64))[:, None] * scale * (-1 if inverse else 1)
    d = x.double()
    if interleaved:
        i0, i1 = slice(offset, offset + rot, 2), slice(offset + 1, offset + rot, 2)
    else:
        i0, i1 = slice(offset, offset + rot // 2), slice(offset + rot // 2, offset + rot)
    y, bound = d.clone(), torch.zeros_like(d)
    a, b = d[..., i0], d[..., i1]
    y[..., i0], y[..., i1] = a * c - b * s, b * c + a * s
    # cos and sin off by at most 2^-21 (an angle rounded to 2^-24 of a half turn, pi * 2^-24, and a few units of
    # fp32), two products and a sum in fp32
    slack = (a.abs() + b.abs()) * abs(scale) * 2.0 ** -20
    bound[..., i0], bound[..., i1] = slack, slack
    turned = torch.zeros_like(d, dtype=torch.bool)
    turned[..., offset:offset + rot] = True
    bound = torch.where(turned, bound + y.abs() * HALF[x.dtype] + TINY[x.dtype], bound)
    return y, bound


def int4_values(w):
    b = w.to(torch.int16)
    lo, hi = b & 15, b >> 4
    q = torch.stack([lo, hi], -1).flatten(1)
    return torch.where(q > 7, q - 16, q).double()


def linear_ref(x, w, w_scale, gated):
    """x [M, K] -> (y, bound).  A product is exact; the fp32 sums take K / 16 tensor-core steps at most, each off by
    at most 2^-22 of the absolute sum (two units: the steps may truncate)."""
    K = x.shape[1]
    wd = int4_values(w) * w_scale.double().repeat_interleave(K // w_scale.shape[1], 1)
    xd = x.double()
    y = xd @ wd.T
    err = (xd.abs() @ wd.abs().T) * (16 + K / 128) * 2.0 ** -22
    if gated:
        g, u = y.chunk(2, -1)
        eg, eu = err.chunk(2, -1)
        sil = g * torch.sigmoid(g)
        y = sil * u
        # |silu'| <= 1.1; the fast exponential and quotient are good to 2^-19
        err = 1.1 * eg * (u.abs() + eu) + sil.abs() * eu + y.abs() * 2.0 ** -19
    return y, err + y.abs() * HALF[x.dtype] + TINY[x.dtype]


def tree_ref(q, k_cache, v_cache, table, ctx, offs, masks, scale):
    """-> (out, bound) on float64; masks: list of python ints (None: chains)."""
    N, hq, D = q.shape
    page, hk = k_cache.shape[1], k_cache.shape[2]
    g = hq // hk
    out, bound = torch.zeros(N, hq, D, dtype=torch.float64), torch.zeros(N, hq, D, dtype=torch.float64)
    half = HALF[q.dtype]
    for b in range(len(ctx)):
        lo, hi = offs[b], offs[b + 1]
        for j in range(lo, hi):
            m = masks[j] if masks is not None else (2 << (j - lo)) - 1
            slots = list(range(ctx[b])) + [ctx[b] + i for i in range(hi - lo) if (m >> i) & 1]
            slots = [s for s in slots if 0 <= table[b][s // page] < k_cache.shape[0]]
            if not slots:
                continue
            pg = torch.tensor([table[b][s // page] for s in slots])
            at = torch.tensor([s % page for s in slots])
            for h in range(hk):
                kk, vv = k_cache[pg, at, h].double(), v_cache[pg, at, h].double()
                qq = q[j, h * g:(h + 1) * g].double()
                s = qq @ kk.T * scale
                p = torch.softmax(s, -1)
                o, av = p @ vv, p @ vv.abs()
                # scores: D / 16 tensor-core steps and the scaling in fp32; exp off by 2 ds and 2^-20; P rounded to
                # the type of V; the joins of partial sums in fp32; the output rounded once
                ds = ((qq.abs() @ kk.abs().T) * abs(scale) * (D / 16 + 4) * 2.0 ** -22).amax(-1, keepdim=True)
                out[j, h * g:(h + 1) * g] = o
                bound[j, h * g:(h + 1) * g] = (half + 2 * ds + 2.0 ** -18) * av * 1.01 + o.abs() * half + TINY[q.dtype]
    return out, bound


def fixed60(p):
    """p * 2^60 rounded to nearest even, for float32 p clamped to [0, 1]; python ints."""
    p = np.nan_to_num(np.asarray(p, dtype=np.float32), nan=0.0, posinf=1.0, neginf=0.0)
    p = np.clip(p, 0.0, 1.0)
    m, e = np.frexp(p.astype(np.float64))
    mant = (m * 2.0 ** 24).astype(np.int64)  # exact: 24 bits
    out = []
    for a, s in zip(mant.tolist(), (e.astype(np.int64) - 24 + 60).tolist()):
        if s >= 0:
            out.append(a << s)
        else:
            half, v = 1 << (-s - 1), a >> -s
            rest = a - (v << -s)
            out.append(v + (rest > half or (rest == half and v & 1)))
    return out


def verify_ref(target, tokens, offs, coins, last, max_nodes, parents=None, draft=None):
    """The walk of every sequence in exact integer arithmetic."""
    target, coins, last = target.numpy(), coins.numpy().astype(np.float64), last.numpy()
    B = len(last)
    out, path, acc = np.full((B, max_nodes + 1), -1), np.full((B, max_nodes), -1), np.zeros(B, dtype=np.int64)
    for b in range(B):
        lo, n = offs[b], offs[b + 1] - offs[b]
        up = [int(parents[lo + j]) if parents is not None else j - 1 for j in range(n)]
        tok = [int(tokens[lo + j]) for j in range(n)]
        node, kept = -1, []
        while True:
            row = target[lo + b + node + 1]
            coin = float(coins[lo + b + node + 1])
            kids = [j for j in range(n) if up[j] == node]
            found, w = None, fixed60(row)
            if draft is not None:
                if kids:
                    j = kids[0]
                    if coin * float(draft[lo + j][tok[j]]) < float(row[tok[j]]):
                        found = j
                    else:
                        w = [max(a - c, 0) for a, c in zip(w, fixed60(draft[lo + j].numpy()))]
            else:
                share, seen, coin60 = 0, set(), int(math.floor(coin * 2.0 ** 60))  # exact: 24 bits
                for j in kids:
                    if tok[j] in seen:
                        continue
                    seen.add(tok[j])
                    p = fixed60(row[tok[j]:tok[j] + 1])[0]
                    if share <= coin60 < share + p:
                        found = j
                        break
                    share += p
                if found is None:
                    w = [0 if x in seen else v for x, v in enumerate(w)]
            if found is None:
                break
            kept.append(found)
            node = found
        if sum(w) == 0:
            w = fixed60(row)
        total = sum(w)
        if total == 0:
            acc[b] = -1
            continue
        u = float(last[b])
        u64 = int(math.floor(u * 2.0 ** 64))  # exact: u has 24 significant bits
        level, run, x = (u64 * total) >> 64, 0, 0
        for x, v in enumerate(w):
            run += v
            if run > level:
                break
        acc[b] = len(kept)
        out[b, :len(kept)] = [tok[j] for j in kept]
        out[b, len(kept)] = x
        path[b, :len(kept)] = kept
    return out, path, acc


def ancestors(parents):
    masks = []
    for j, p in enumerate(parents):
        masks.append((1 << j) | (masks[p] if p >= 0 else 0))
    return masks


def mask_tensor(masks):
    return torch.from_numpy(np.array(masks, dtype=np.uint64).view(np.int64))
