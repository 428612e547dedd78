"""Cases for the operators of one speculative step of a softmax-attention layer beside KDA layers: rotary positions,
attention of a drafted tree over a paged cache, verification of the drafted tokens, and the append of accepted tokens.

``own`` False: the operators in plain torch operations; True: the library's calls.  A case's ``op`` names the operator."""
import math

import numpy as np
import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # the rollout's verify step: 128 sequences of 4 drafted tokens, positions anywhere in a 128K context
        {"name": "rope_step", "op": "rope", "T": 512, "Hq": 32, "Hk": 8, "d": 128, "rot": 128, "dtype": "bf16",
         "interleaved": False, "scaling": "yarn", "max_pos": 131072, "bwd": False},
        # prefill of four 4096-token sequences (q and k of one layer)
        {"name": "rope_prefill", "op": "rope", "T": 16384, "Hq": 32, "Hk": 8, "d": 128, "rot": 128, "dtype": "bf16",
         "interleaved": False, "scaling": "none", "max_pos": 4096, "bwd": False},
        # training in fp32, 64-wide heads, half of each head rotated, interleaved pairs: the gradient
        {"name": "rope_grad", "op": "rope", "T": 8191, "Hq": 32, "Hk": 32, "d": 64, "rot": 32, "dtype": "f32",
         "interleaved": True, "scaling": "linear", "max_pos": 32768, "bwd": True},
        # one user, one token: the latency of a decode step
        {"name": "attn_one", "op": "attn", "N": 1, "nodes": 1, "ctx": 1025, "ragged": False, "Hq": 32, "Hkv": 8, "dk": 128,
         "dv": 128, "page": 16, "dtype": "bf16", "tree": False},
        # the rollout's verify step: 128 sequences, a chain of 4 tokens each, about 2048 tokens of context
        {"name": "attn_rollout", "op": "attn", "N": 128, "nodes": 4, "ctx": 4096, "ragged": True, "Hq": 32, "Hkv": 8,
         "dk": 128, "dv": 128, "page": 64, "dtype": "bf16", "tree": False},
        # a few long-context users with wide draft trees
        {"name": "attn_long", "op": "attn", "N": 4, "nodes": 33, "ctx": 131072, "ragged": False, "Hq": 32, "Hkv": 4,
         "dk": 128, "dv": 128, "page": 128, "dtype": "bf16", "tree": True},
        # fp32, 64-wide heads, ragged trees and contexts, pages of 24 rows
        {"name": "attn_f32", "op": "attn", "N": 7, "nodes": 13, "ctx": 4099, "ragged": True, "Hq": 12, "Hkv": 4, "dk": 64,
         "dv": 64, "page": 24, "dtype": "f32", "tree": True},
        # one user, a small draft tree
        {"name": "verify_one", "op": "verify", "N": 1, "nodes": 6, "V": 32001, "ragged": False, "tree": True,
         "draft": True, "dtype": "f32"},
        # the rollout: 128 chains of 3 drafts after the last token, a large vocabulary
        {"name": "verify_rollout", "op": "verify", "N": 128, "nodes": 4, "V": 131072, "ragged": False, "tree": False,
         "draft": True, "dtype": "f32"},
        # deterministic drafts (no draft probabilities), wide trees, an odd vocabulary, bf16 probabilities
        {"name": "verify_tree", "op": "verify", "N": 24, "nodes": 32, "V": 100003, "ragged": True, "tree": True,
         "draft": False, "dtype": "bf16"},
        # the rollout's accepted tokens (1 to 4 of each 4) into the cache
        {"name": "append_accepted", "op": "append", "N": 128, "count": 4, "ctx": 2048, "Hkv": 8, "dk": 128, "dv": 128,
         "page": 64, "dtype": "bf16", "picked": True},
        # the prompt's keys and values into the cache
        {"name": "append_prefill", "op": "append", "N": 16, "count": 2048, "ctx": 500, "Hkv": 8, "dk": 128, "dv": 128,
         "page": 16, "dtype": "bf16", "picked": False},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "attn", "verify", "append"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "rope":
        d = rng.choice([64, 128])
        Hk = rng.randint(1, 16)
        Hq = Hk * rng.randint(1, 8)
        return {"op": op, "T": _log(rng, 1, max(1, min(16384, 2 ** 26 // (Hq * d)))), "Hq": Hq, "Hk": Hk, "d": d,
                "rot": 2 * rng.randint(1, d // 2), "dtype": dtype, "interleaved": rng.random() < 0.5,
                "scaling": rng.choice(["none", "linear", "ntk", "yarn"]), "max_pos": _log(rng, 16, 1 << 20),
                "bwd": rng.random() < 0.5}
    if op == "attn":
        N, nodes, Hkv = _log(rng, 1, 128), rng.choice([1, rng.randint(1, 8), rng.randint(1, 64)]), rng.randint(1, 8)
        G, dk, dv = rng.randint(1, 8), rng.choice([64, 128]), rng.choice([64, 128])
        # at most the long case's query rows times keys, and its cache
        most = min(2 ** 26 * 2 // (N * nodes * Hkv * G), 2 ** 19 * 4 // (N * Hkv))
        return {"op": op, "N": N, "nodes": nodes, "ctx": _log(rng, 1, max(1, min(131072, most))),
                "ragged": rng.random() < 0.7, "Hq": Hkv * G, "Hkv": Hkv, "dk": dk, "dv": dv,
                "page": rng.choice([8, 16, 24, 64, 128, 100]), "dtype": dtype, "tree": rng.random() < 0.6}
    if op == "verify":
        N, V = _log(rng, 1, 128), _log(rng, 1000, 160001)
        return {"op": op, "N": N, "nodes": max(1, min(rng.choice([1, rng.randint(2, 8), rng.randint(2, 64)]),
                                                      2 ** 26 // (N * V))),
                "V": V, "ragged": rng.random() < 0.5, "tree": rng.random() < 0.6, "draft": rng.random() < 0.6,
                "dtype": rng.choice(["f32", "f32", "bf16"])}
    N, Hkv = _log(rng, 1, 128), rng.randint(1, 16)
    dk, dv = rng.choice([64, 128]), rng.choice([64, 128])
    picked = rng.random() < 0.5
    count = rng.randint(1, 64) if picked else _log(rng, 1, max(1, 2 ** 24 // (N * Hkv * 256)))
    return {"op": op, "N": N, "count": count, "ctx": _log(rng, 1, max(1, 2 ** 18 // (N * Hkv))), "Hkv": Hkv, "dk": dk,
            "dv": dv, "page": rng.choice([8, 16, 24, 64, 128, 100]), "dtype": dtype, "picked": picked}


# ---- inputs -------------------------------------------------------------------------------------------------------


def _inv_freq(rot, scaling, factor=8.0, base=10000.0, original=4096):
    """Frequencies of the pairs (radians per position) and the factor on the rotated values."""
    j = np.arange(0, rot, 2, dtype=np.float64)
    w, m = base ** (-j / rot), 1.0
    if scaling == "linear":
        w = w / factor
    elif scaling == "ntk" and rot > 2:
        w = (base * factor ** (rot / (rot - 2))) ** (-j / rot)
    elif scaling == "yarn":
        turn = lambda n: rot * math.log(original / (n * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
        lo, hi = max(math.floor(turn(32)), 0), min(math.ceil(turn(1)), rot - 1)
        ramp = np.clip((j / 2 - lo) / max(hi - lo, 1e-3), 0, 1)
        w, m = w / factor * ramp + w * (1 - ramp), 0.1 * math.log(factor) + 1
    return w, m


def _lengths(n, most, ragged, least=1, order=0):
    """Lengths spread evenly over [least, most], mixed: the same for every seed, so that the outputs keep their shapes."""
    return np.random.default_rng(order).permutation(np.linspace(most, least, n).round().astype(np.int64)) if ragged else np.full(n, most)


def _cu(lengths):
    return torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32).cuda()


def _parents(lengths, tree, rng):
    """Each node's parent in its own sequence (-1: the root, node 0): chains, or trees that branch near the root."""
    out = []
    for n in lengths:
        i = np.arange(n)
        out.append(np.where(i == 0, -1, np.minimum((i * rng.random(n) ** 1.5).astype(np.int64), i - 1)) if tree else i - 1)
    return torch.tensor(np.concatenate(out), dtype=torch.int32).cuda()


def _cache(case, lengths, gen, rng):
    """Pages in random order, as a server that has run for a while has them."""
    per = -(-np.asarray(lengths) // case["page"])
    width, total = int(per.max()), int(per.sum())
    order, table, at = rng.permutation(total + 3), np.zeros((len(per), width), dtype=np.int64), 0
    for n, p in enumerate(per):
        table[n, :p] = order[at:at + p]
        at += p
    make = lambda d: torch.randn(total + 3, case["page"], case["Hkv"], d, generator=gen, device="cuda",  # noqa: E731
                                 dtype=_DT[case["dtype"]])
    return make(case["dk"]), make(case["dv"]), torch.tensor(table, dtype=torch.int32).cuda()


def prepare(case, seed):
    gen, rng = torch.Generator("cuda").manual_seed(seed), np.random.default_rng(seed)
    rand = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    dt = _DT[case["dtype"]]
    s = {"case": case}
    if case["op"] == "rope":
        w, s["mscale"] = _inv_freq(case["rot"], case["scaling"])
        s["inv_freq"] = torch.tensor(w).cuda()
        s["q"], s["k"] = (rand(case["T"], case[h], case["d"]).to(dt) for h in ("Hq", "Hk"))
        s["positions"] = torch.randint(0, case["max_pos"], (case["T"],), generator=gen, device="cuda", dtype=torch.int32)
    elif case["op"] == "attn":
        m, ctx = (_lengths(case["N"], case[key], case["ragged"], order=i) for i, key in enumerate(("nodes", "ctx")))
        T = int(m.sum())
        s["cu"], s["parent"] = _cu(m), _parents(m, case["tree"], rng) if case["tree"] else None
        s["ctx_len"] = torch.tensor(ctx, dtype=torch.int32).cuda()
        s["k_pages"], s["v_pages"], s["table"] = _cache(case, ctx, gen, rng)
        s["q"] = (2 * rand(T, case["Hq"], case["dk"])).to(dt)  # sharper than independent keys would give
        s["k"], s["v"] = rand(T, case["Hkv"], case["dk"]).to(dt), rand(T, case["Hkv"], case["dv"]).to(dt)
    elif case["op"] == "verify":
        m = _lengths(case["N"], case["nodes"], case["ragged"])
        T, V = int(m.sum()), case["V"]
        s["cu"], parent = _cu(m), _parents(m, case["tree"], rng)
        s["parent"] = parent if case["tree"] else None
        logits = 2.5 * rand(T, V)
        s["target"] = torch.softmax(logits, -1).to(dt)
        draft = torch.softmax(logits + rand(T, V), -1)
        first = torch.repeat_interleave(s["cu"][:-1].long(), torch.tensor(m).cuda())
        s["tokens"] = torch.multinomial(draft[first + parent.long().clamp(min=0)], 1, generator=gen)[:, 0].int()
        s["draft"] = draft.to(dt) if case["draft"] else None
        s["u_accept"] = torch.rand(T, generator=gen, device="cuda")
        s["u_sample"] = torch.rand(case["N"], generator=gen, device="cuda")
    else:
        new = _lengths(case["N"], case["count"], True)
        ctx = _lengths(case["N"], case["ctx"], True, least=0, order=1)
        s["cu"], s["ctx_len"] = _cu(new), torch.tensor(ctx, dtype=torch.int32).cuda()
        s["k_pages"], s["v_pages"], s["table"] = _cache(case, ctx + new, gen, rng)
        T = int(new.sum())
        src = case["N"] * case["count"] if case["picked"] else T
        s["k"], s["v"] = rand(src, case["Hkv"], case["dk"]).to(dt), rand(src, case["Hkv"], case["dv"]).to(dt)
        picks = [n * case["count"] + np.sort(rng.permutation(case["count"])[:c]) for n, c in enumerate(new)]
        s["rows"] = torch.tensor(np.concatenate(picks), dtype=torch.int32).cuda() if case["picked"] else None
    return s


# ---- one pass -----------------------------------------------------------------------------------------------------


def run(s):
    case = s["case"]
    if own:
        import gated_linear_attention_chunk_gb300 as kda
        if case["op"] == "rope":
            call = kda.kda_rope_bwd if case["bwd"] else kda.kda_rope
            return call(s["q"], s["k"], s["positions"], s["inv_freq"], interleaved=case["interleaved"], mscale=s["mscale"])
        if case["op"] == "attn":
            return kda.kda_tree_attn(s["q"], s["k"], s["v"], s["k_pages"], s["v_pages"], s["table"], s["ctx_len"], s["cu"],
                                     parent=s["parent"], scale=case["dk"] ** -0.5, max_nodes=case["nodes"])
        if case["op"] == "verify":
            return kda.kda_draft_verify(s["tokens"], s["cu"], s["target"], s["u_accept"], s["u_sample"],
                                        parent=s["parent"], draft_probs=s["draft"])
        new_len = kda.kda_cache_append(s["k"], s["v"], s["k_pages"], s["v_pages"], s["table"], s["ctx_len"], s["cu"],
                                       rows=s["rows"])
        return new_len, s["k_pages"], s["v_pages"]
    return {"rope": _plain_rope, "attn": _plain_attn, "verify": _plain_verify, "append": _plain_append}[case["op"]](s)


def _plain_rope(s):
    case, half = s["case"], s["case"]["rot"] // 2
    angle = (s["positions"].double()[:, None] * s["inv_freq"]) * (-1.0 if case["bwd"] else 1.0)
    cos, sin = ((s["mscale"] * f(angle)).float()[:, None, :] for f in (torch.cos, torch.sin))

    def turn(x):
        y = x.float()
        a, b = (y[..., 0:2 * half:2], y[..., 1:2 * half:2]) if case["interleaved"] else (y[..., :half], y[..., half:2 * half])
        pair = (a * cos - b * sin, a * sin + b * cos)
        turned = torch.stack(pair, -1).flatten(-2) if case["interleaved"] else torch.cat(pair, -1)
        return torch.cat((turned, y[..., 2 * half:]), -1).to(x.dtype)

    return turn(s["q"]), turn(s["k"])


def _nodes(cu, most, T):
    """Rows [N, most] of each sequence's nodes in the packed arrays, which of them exist, and each row's sequence."""
    i = torch.arange(most, device="cuda")
    there = i < (cu[1:] - cu[:-1])[:, None]
    rows = (cu[:-1, None] + i).clamp(max=T - 1).long()
    return rows, there, torch.searchsorted(cu, torch.arange(T, device="cuda", dtype=torch.int32), right=True) - 1


def _plain_attn(s):
    case, G = s["case"], s["case"]["Hq"] // s["case"]["Hkv"]
    N, M, T, Hkv = case["N"], case["nodes"], s["q"].shape[0], case["Hkv"]
    rows, there, seq = _nodes(s["cu"], M, T)
    i = torch.arange(M, device="cuda")
    up = i.expand(N, M) - 1 if s["parent"] is None else s["parent"][rows].long()
    step = torch.eye(M, device="cuda", dtype=torch.float64) + (up[:, :, None] == i)
    sees = (torch.linalg.matrix_power(step, M) > 0) & there[:, None, :]
    q = s["q"][rows].float().view(N, M, Hkv, G, case["dk"])
    whole = lambda pages, new: torch.cat((pages[s["table"].long()].flatten(1, 2), new[rows]), 1).float()  # noqa: E731
    keys, values = whole(s["k_pages"], s["k"]), whole(s["v_pages"], s["v"])
    L = keys.shape[1] - M
    live = torch.arange(L, device="cuda") < s["ctx_len"][:, None]
    mask = torch.cat((live[:, None, :].expand(N, M, L), sees), 2)
    values = values * torch.cat((live, there), 1)[:, :, None, None]
    score = torch.einsum("nmhgd,nlhd->nhgml", q, keys) * case["dk"] ** -0.5
    score = score.masked_fill(~mask[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True).clamp(min=-1e30)
    e = torch.exp(score - top)
    total = e.sum(-1, keepdim=True)
    o = torch.einsum("nhgml,nlhd->nmhgd", e / total, values).reshape(N, M, case["Hq"], case["dv"])
    lse = (top + torch.log(total))[..., 0].permute(0, 3, 1, 2).reshape(N, M, case["Hq"])
    at = torch.arange(T, device="cuda") - s["cu"][seq]
    return o[seq, at].to(s["q"].dtype), lse[seq, at]


def _plain_verify(s):
    """Node by node: each decision rests on the one before.  In 64 bits, since a decision next to a border has to stand."""
    case, N, M, T = s["case"], s["case"]["N"], s["case"]["nodes"], s["tokens"].shape[0]
    rows, there, seq = _nodes(s["cu"], M, T)
    up = torch.arange(M, device="cuda").expand(N, M) - 1 if s["parent"] is None else s["parent"][rows].long()
    n = torch.arange(N, device="cuda")
    cur = torch.zeros(N, dtype=torch.long, device="cuda")
    passed = torch.zeros(N, M, dtype=torch.bool, device="cuda")
    passed[:, 0] = True
    p = s["target"][rows[:, 0]].double()
    q = s["draft"][rows[:, 0]].double() if case["draft"] else None
    r, mass = p, torch.ones(N, dtype=torch.float64, device="cuda")
    for i in range(1, M):
        x, u = s["tokens"][rows[:, i]].long(), s["u_accept"][rows[:, i]].double()
        tried = there[:, i] & (up[:, i] == cur)
        weight = q[n, x] if case["draft"] else 1.0
        yes = tried & (u * weight * mass < r[n, x])
        no = tried & ~yes
        if case["draft"]:
            left = (r - mass[:, None] * q).clamp(min=0)
            after = left.sum(1)
        else:
            left, after = r.clone(), mass - r[n, x]
            left[n, x] = 0
        r, mass = torch.where(no[:, None], left, r), torch.where(no, after, mass)
        passed[:, i] = yes
        cur = torch.where(yes, i, cur)
        p = torch.where(yes[:, None], s["target"][rows[:, i]].double(), p)
        q = torch.where(yes[:, None], s["draft"][rows[:, i]].double(), q) if case["draft"] else None
        r, mass = torch.where(yes[:, None], p, r), torch.where(yes, 1.0, mass)
    r = torch.where(r.sum(1, keepdim=True) > 0, r, p)
    below = torch.cumsum(r, 1)
    token = (below > s["u_sample"].double()[:, None] * below[:, -1:]).int().argmax(1)
    cu_accept = torch.cat((torch.zeros(1, dtype=torch.long, device="cuda"), passed.sum(1).cumsum(0))).int()
    kept = passed[seq, torch.arange(T, device="cuda") - s["cu"][seq]]
    order = torch.sort(kept.logical_not().int(), stable=True).indices
    packed = torch.where(torch.arange(T, device="cuda") < cu_accept[-1], order, -1).int()
    return cu_accept, packed, token.int()


def _plain_append(s):
    case, T = s["case"], s["k"].shape[0] if s["rows"] is None else s["rows"].shape[0]
    j = torch.arange(T, device="cuda", dtype=torch.int32)
    seq = torch.searchsorted(s["cu"], j, right=True) - 1
    at = s["ctx_len"][seq] + j - s["cu"][seq]
    page, slot = s["table"][seq, (at // case["page"]).long()].long(), (at % case["page"]).long()
    src = j.long() if s["rows"] is None else s["rows"].long()
    s["k_pages"][page, slot] = s["k"][src]
    s["v_pages"][page, slot] = s["v"][src]
    return s["ctx_len"] + (s["cu"][1:] - s["cu"][:-1]), s["k_pages"], s["v_pages"]


# ---- what a pass cannot do without --------------------------------------------------------------------------------


def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    half = 0.5 if case.get("ragged") else 1.0  # lengths uniform up to the largest
    if case["op"] == "rope":
        heads = case["T"] * (case["Hq"] + case["Hk"])
        return {"bytes": 2 * es * heads * case["d"] + 4 * case["T"], "flops": 3 * heads * case["rot"]}
    if case["op"] == "attn":
        N, width = case["N"], case["dk"] + case["dv"]
        nodes, ctx = half * case["nodes"], half * case["ctx"]
        return {"bytes": N * es * (case["Hkv"] * (ctx + nodes) + nodes * case["Hq"]) * width + 4 * N * ctx / case["page"],
                "flops": 2 * N * nodes * (ctx + nodes / 2) * case["Hq"] * width}
    if case["op"] == "verify":  # each sequence ends with one sampling pass over a row
        per = 2 if case["draft"] else 1
        return {"bytes": case["N"] * (es * case["V"] * per + 16 * half * case["nodes"]), "flops": 2 * per * case["N"] * case["V"]}
    new = case["N"] * (case["count"] + 1) / 2
    return {"bytes": 2 * es * new * case["Hkv"] * (case["dk"] + case["dv"]), "flops": 0}


# ---- the definitions in 64 bits ------------------------------------------------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": _exact_rope, "attn": _exact_attn, "verify": _exact_verify, "append": _exact_append}[case["op"]](case, s)


def _exact_rope(case, s):
    """A rotated pair is a complex number times exp(i t); the gradient takes the conjugate."""
    t = s["positions"].double().outer(s["inv_freq"])
    unit = torch.polar(torch.full_like(t, s["mscale"]), -t if case["bwd"] else t)[:, None]
    done = []
    for x in (s["q"], s["k"]):
        y = x.double()
        z = y[..., :case["rot"]].unflatten(-1, (-1, 2) if case["interleaved"] else (2, -1))
        z = (z if case["interleaved"] else z.transpose(-1, -2)).contiguous()
        z = torch.view_as_real(torch.view_as_complex(z) * unit)
        y[..., :case["rot"]] = (z if case["interleaved"] else z.transpose(-1, -2)).flatten(-2)
        done.append(y)
    return tuple(done)


def _exact_attn(case, s):
    """Sequence by sequence, head by head, the visible keys of each node gathered by walking up to the root."""
    cu, ctx = s["cu"].tolist(), s["ctx_len"].tolist()
    G, T = case["Hq"] // case["Hkv"], s["q"].shape[0]
    o = torch.empty(T, case["Hq"], case["dv"], dtype=torch.float64, device="cuda")
    lse = torch.empty(T, case["Hq"], dtype=torch.float64, device="cuda")
    for n in range(case["N"]):
        a, b = cu[n], cu[n + 1]
        up = list(range(-1, b - a - 1)) if s["parent"] is None else s["parent"][a:b].tolist()
        bias = torch.full((b - a, ctx[n] + b - a), -math.inf, dtype=torch.float64)
        bias[:, :ctx[n]] = 0
        for i in range(b - a):
            j = i
            while j >= 0:
                bias[i, ctx[n] + j] = 0
                j = up[j]
        pos = torch.arange(ctx[n], device="cuda")
        page, slot = s["table"][n].long()[pos // case["page"]], pos % case["page"]
        bias = bias.cuda()
        for h in range(case["Hkv"]):
            k = torch.cat((s["k_pages"][page, slot, h], s["k"][a:b, h])).double()
            v = torch.cat((s["v_pages"][page, slot, h], s["v"][a:b, h])).double()
            for g in range(h * G, (h + 1) * G):
                z = s["q"][a:b, g].double() @ k.T / math.sqrt(case["dk"]) + bias
                lse[a:b, g] = torch.logsumexp(z, 1)
                o[a:b, g] = torch.exp(z - lse[a:b, g, None]) @ v
    return o, lse


def _exact_verify(case, s):
    """The walk of each sequence by its definition, the residual normalised after every refusal."""
    cu, tokens = s["cu"].tolist(), s["tokens"].tolist()
    u, us = s["u_accept"].double().tolist(), s["u_sample"].double().tolist()
    counts, kept, nxt = [0], [], []
    for n in range(case["N"]):
        a, b = cu[n], cu[n + 1]
        up = list(range(-1, b - a - 1)) if s["parent"] is None else s["parent"][a:b].tolist()
        cur, path = 0, [a]
        while True:
            p = s["target"][a + cur].double().cpu().numpy()
            q = s["draft"][a + cur].double().cpu().numpy() if case["draft"] else None
            left, found = p.copy(), None
            for c in (i for i in range(1, b - a) if up[i] == cur):
                x = tokens[a + c]
                if u[a + c] * (q[x] if case["draft"] else 1.0) < left[x]:
                    found = c
                    break
                if case["draft"]:
                    left = np.maximum(left - q, 0.0)
                    rest = left.sum()
                else:
                    rest = 1.0 - left[x]
                    left[x] = 0.0
                left = left / rest if rest > 0 else left
            if found is None:
                break
            cur = found
            path.append(a + cur)
        weights = left if left.sum() > 0 else p
        below = np.cumsum(weights)
        nxt.append(int(np.argmax(below > us[n] * below[-1])))
        kept += path
        counts.append(len(kept))
    packed = np.full(len(tokens), -1)
    packed[:len(kept)] = kept
    return tuple(torch.tensor(np.asarray(z), dtype=torch.int32) for z in (counts, packed, nxt))


def _exact_append(case, s):
    cu, ctx = s["cu"].tolist(), s["ctx_len"].tolist()
    out = [s["k_pages"].cpu().double(), s["v_pages"].cpu().double()]
    table, new = s["table"].cpu(), [s["k"].cpu().double(), s["v"].cpu().double()]
    rows = torch.arange(cu[-1]) if s["rows"] is None else s["rows"].long().cpu()
    for n in range(case["N"]):
        at = torch.arange(cu[n + 1] - cu[n]) + ctx[n]
        page, slot = table[n].long()[at // case["page"]], at % case["page"]
        for pages, x in zip(out, new):
            pages[page, slot] = x[rows[cu[n]:cu[n + 1]]]
    return torch.tensor([c + cu[n + 1] - cu[n] for n, c in enumerate(ctx)], dtype=torch.int32), *out
