"""Plain 64-bit forms of the speculative-step operators (numpy), for the tests."""
import math

import numpy as np
import torch

BF16, F32 = torch.bfloat16, torch.float32
HALF_STEP = {BF16: 2.0 ** -8, F32: 2.0 ** -24}  # the most that one rounding is off, relative


def np64(t):
    return t.detach().cpu().double().numpy()


def rope(x, pos, inv_freq, interleaved, mscale, backward=False):
    """Rotated x [T, H, d] and, per element, the sum of the magnitudes that met in it."""
    x, w = np64(x), np.asarray(inv_freq, dtype=np.float64)
    half = len(w)
    t = np.asarray(pos, dtype=np.float64)[:, None] * w
    c, s = mscale * np.cos(t)[:, None], mscale * np.sin(t)[:, None] * (-1 if backward else 1)
    ia = np.arange(half) * 2 if interleaved else np.arange(half)
    ib = ia + 1 if interleaved else ia + half
    y, mag = x.copy(), np.abs(x)
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, a * s + b * c
    mag[..., ia] = mag[..., ib] = abs(mscale) * (np.abs(a) + np.abs(b))
    return y, mag


def ancestors(parent):
    """[m, m] truth values: node i sees node j."""
    m = len(parent)
    sees = np.zeros((m, m), dtype=bool)
    for i in range(m):
        sees[i, i] = True
        if i:
            sees[i] |= sees[parent[i]]
    return sees


def attn(q, k, v, k_pages, v_pages, table, ctx, cu, parent, scale):
    """o, lse, and per output the bound's ingredients: sum p |v|, and the largest scale * sum |q||k| of a row."""
    q, k, v, table = np64(q), np64(k), np64(v), table.cpu().numpy()
    kp, vp = np64(k_pages), np64(v_pages)
    T, Hq, dk = q.shape
    Hkv, dv, G = v.shape[1], v.shape[2], q.shape[1] // v.shape[1]
    page = kp.shape[1]
    o, lse = np.zeros((T, Hq, dv)), np.zeros((T, Hq))
    weight, reach = np.zeros((T, Hq, dv)), np.zeros((T, Hq))
    for n in range(len(ctx)):
        a, b = int(cu[n]), int(cu[n + 1])
        if a == b:
            continue
        at = np.arange(int(ctx[n]))
        keys = np.concatenate([kp[table[n, at // page], at % page], k[a:b]])
        vals = np.concatenate([vp[table[n, at // page], at % page], v[a:b]])
        up = list(range(-1, b - a - 1)) if parent is None else parent[a:b].cpu().tolist()
        mask = np.concatenate([np.ones((b - a, len(at)), dtype=bool), ancestors(up)], 1)
        for h in range(Hq):
            kk, vv = keys[:, h // G], vals[:, h // G]
            s = np.where(mask, scale * (q[a:b, h] @ kk.T), -np.inf)
            top = s.max(1, keepdims=True)
            e = np.exp(s - top)
            l = e.sum(1, keepdims=True)
            o[a:b, h] = (e / l) @ vv
            weight[a:b, h] = (e / l) @ np.abs(vv)
            lse[a:b, h] = (top + np.log(l))[:, 0]
            reach[a:b, h] = (abs(scale) * (np.abs(q[a:b, h]) @ np.abs(kk).T)).max(1)
    return o, lse, weight, reach


def attn_bounds(dtype, dk, longest, o, lse, weight, reach):
    """Elementwise bounds of o and lse.  A score is a sum of dk products in fp32 (dk roundings of at most its
    magnitudes, plus the scaling and the exponential's argument and own error, 8 in all, of their size); a weight is then off
    by the relative amount of that difference, twice (numerator and sum), and the sums over the keys round `longest` times
    more; bf16 weights are rounded once more, and the result once."""
    f = HALF_STEP[F32]
    score = (dk + 8) * f * (reach + 8) + 8 * f
    rel = 2 * score + (longest + 64) * f + (HALF_STEP[BF16] if dtype == BF16 else 0.0)
    return (np.abs(o) + weight * rel[..., None]) * HALF_STEP[dtype] + weight * rel[..., None], \
        score + (longest + 64) * f + 4 * f * np.abs(lse)


def verify(tokens, cu, parent, target, draft, u_accept, u_sample):
    """cu_accept, rows, next_token by the definition, the residual normalised after every refusal."""
    p_all, q_all = np64(target), None if draft is None else np64(draft)
    u, us, tok = np64(u_accept), np64(u_sample), tokens.cpu().tolist()
    counts, kept, nxt = [0], [], []
    for n in range(len(cu) - 1):
        a, b = int(cu[n]), int(cu[n + 1])
        if a == b:
            nxt.append(-1)
            counts.append(len(kept))
            continue
        up = list(range(-1, b - a - 1)) if parent is None else parent[a:b].cpu().tolist()
        cur = 0
        kept.append(a)
        while True:
            p = np.nan_to_num(p_all[a + cur], nan=0.0)
            r, found = p.copy(), None
            for c in [i for i in range(1, b - a) if up[i] == cur]:
                x = tok[a + c]
                if u[a + c] * (1.0 if draft is None else q_all[a + cur, x]) < r[x]:
                    found = c
                    break
                if draft is None:
                    rest = 1.0 - r[x]
                    r[x] = 0.0
                else:
                    r = np.maximum(r - q_all[a + cur], 0.0)
                    rest = r.sum()
                if rest > 0:
                    r = r / rest
            if found is None:
                break
            cur = found
            kept.append(a + cur)
        w = r if r.sum() > 0 else p
        below = np.cumsum(w)
        nxt.append(int(np.argmax(below > us[n] * below[-1])) if below[-1] > 0 else -1)
        counts.append(len(kept))
    rows = np.full(len(tok), -1)
    rows[:len(kept)] = kept
    return np.array(counts), rows, np.array(nxt)


# ---- inputs ---------------------------------------------------------------------------------------------------------


def random_parents(lengths, rng):
    out = []
    for m in lengths:
        i = np.arange(m)
        out.append(np.where(i == 0, -1, np.minimum((i * rng.random(m) ** 1.5).astype(np.int64), i - 1)))
    return torch.tensor(np.concatenate(out) if out else [], dtype=torch.int32)


def offsets(lengths):
    return torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32)


def paged(lengths, page, Hkv, dk, dv, dtype, seed, spare=2, fill=float("nan")):
    """Pools whose rows beyond the lengths hold `fill`, and a shuffled block table (unused entries far out of range)."""
    rng, gen = np.random.default_rng(seed), torch.Generator().manual_seed(seed)
    per = [-(-int(n) // page) for n in lengths]
    total, width = sum(per) + spare, max(per + [1])
    order, table, at = rng.permutation(total), np.full((len(per), width), 1 << 30), 0
    kp, vp = (torch.full((total, page, Hkv, d), fill).to(dtype) for d in (dk, dv))
    for n, c in enumerate(per):
        table[n, :c] = order[at:at + c]
        at += c
        i = np.arange(int(lengths[n]))
        kp[table[n, i // page], i % page] = torch.randn(len(i), Hkv, dk, generator=gen).to(dtype)
        vp[table[n, i // page], i % page] = torch.randn(len(i), Hkv, dv, generator=gen).to(dtype)
    return kp, vp, torch.tensor(table, dtype=torch.int32)
