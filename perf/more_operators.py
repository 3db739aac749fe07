"""Benchmark cases of rotary positions and of the paged 16-bit KV cache: rotating queries and keys (and their gradients),
appending rotated rows to the cache, attention of drafted trees over it, and keeping a tree's accepted nodes.  `run`
computes each case with elementary torch operations in fp32 (angles in fp64), or, where `own` is true, with the package's
kernels; `exact` computes the same in fp64 from the definitions.

The cache: a pool of pages, bf16 [pages, 2, Hkv, page_size, D], K in front of V.  Position p of the sequence in slot s
lives in page table[s, p // page_size] at row p % page_size; lens counts the positions of each slot.  The call's
sequences are packed: cu holds their prefix offsets, and the rows of a call are the last positions of their sequences.

A drafted tree lists its nodes parents first: the likeliest chain, then the side branches.  Node i sees the whole prefix,
its ancestors and itself: bit j % 32 of mask[i, j // 32] stands for node j.  Its position is the prefix length plus its
depth.
"""
import functools
import math
import random

import torch

own = False

DEV = "cuda"


# ----------------------------------------------------------------------------------------------------------- cases

def listed():
    return [
        # a decode step of 16 requests: q and k of one layer, where latency counts
        dict(name="rope_step", op="rope", T=16, Hq=32, Hkv=8, D=128, R=128, start=0, inter=False, kind="packed",
             dtype="bf16", scaling="none"),
        # the repository's packed batch of 8 prompts (39235 tokens), read out of the fused projection's rows, with the
        # frequencies of a context stretched by 8
        dict(name="rope_prompts", op="rope", T=39235, Hq=32, Hkv=8, D=128, R=128, start=0, inter=False, kind="packed",
             dtype="bf16", scaling="parts"),
        # the repository's (192, 128) heads at 16384 tokens: the last 64 of 192 dimensions turn, in neighbouring pairs;
        # the projection's [B, L, H, D] becomes the attention's [B, H, L, D] on the way
        dict(name="rope_part", op="rope", T=16384, Hq=16, Hkv=16, D=192, R=64, start=128, inter=True, kind="dense",
             dtype="bf16", scaling="none"),
        # the training step of the packed batch: fp32 gradients of q and k as the attention's backward gives them, turned
        # back and handed on in bf16
        dict(name="rope_grad", op="rope", T=39235, Hq=32, Hkv=8, D=128, R=128, start=0, inter=False, kind="packed",
             dtype="grad", scaling="none"),
        # the cache write of a drafting server: trees of up to 8 nodes for 64 requests, small heads, small pages
        dict(name="append_drafts", op="append", n=64, Hq=16, Hkv=4, D=64, P=16, new_lo=1, new_hi=8, old_hi=4096, R=64,
             start=0, inter=True, scaling="none", tree=True),
        # the cache write of a packed batch of 8 prompts of 512 to 8192 tokens
        dict(name="append_prompts", op="append", n=8, Hq=32, Hkv=8, D=128, P=64, new_lo=512, new_hi=8192, old_hi=0,
             R=128, start=0, inter=False, scaling="parts", tree=False),
        # one chat request early in its answer: a single token over a short cache, where latency counts
        dict(name="attn_one_short", op="attn", B=1, Hq=32, Hkv=8, D=128, P=64, lo=777, hi=777, new_lo=1, new_hi=1,
             tree=False),
        # a drafting server's step: 32 requests of very different ages, a tree of 1 to 24 nodes each
        dict(name="attn_ragged", op="attn", B=32, Hq=16, Hkv=4, D=64, P=16, lo=1, hi=8192, new_lo=1, new_hi=24,
             tree=True),
        # the repository's decode workload (B = 8, 32 x 8 heads, 32768 keys) with trees of 64 nodes
        dict(name="attn_long", op="attn", B=8, Hq=32, Hkv=8, D=128, P=64, lo=32768, hi=32768, new_lo=64, new_hi=64,
             tree=True),
        # the next 2048 tokens of two long prompts that are worked off in chunks
        dict(name="attn_chunk", op="attn", B=2, Hq=32, Hkv=8, D=128, P=128, lo=18432, hi=18432, new_lo=2048,
             new_hi=2048, tree=False),
        # accepted drafts of a few requests in a small model
        dict(name="keep_small", op="keep", layers=4, n=5, Hkv=2, D=64, P=16, draft=12, depth=4, old_hi=200),
        # accepted drafts of 64 requests in 32 layers of a server's pool
        dict(name="keep_layers", op="keep", layers=32, n=64, Hkv=8, D=128, P=16, draft=64, depth=7, old_hi=300),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "rope", "append", "append", "attn", "attn", "attn", "keep"])
    D, P, Hkv = rng.choice([64, 128]), rng.choice([16, 32, 64, 128, 256]), rng.choice([1, 2, 3, 4, 8])
    group = rng.choice([1, 2, 4, 5, 8])
    scaling = rng.choice(["none", "linear", "base", "parts"])
    if op == "rope":
        D = rng.choice([64, 128, 192])
        R = rng.choice([D, D, D // 2, 32])
        start = rng.choice([0, D - R])
        return dict(op=op, T=_log(rng, 1, 20000), Hq=Hkv * group, Hkv=Hkv, D=D, R=R, start=start,
                    inter=rng.random() < 0.5, kind=rng.choice(["packed", "dense"]),
                    dtype=rng.choice(["bf16", "bf16", "grad", "fp32"]), scaling=scaling)
    if op == "append":
        n, tree = _log(rng, 1, 64), rng.random() < 0.5
        R = rng.choice([D, D, D // 2])
        return dict(op=op, n=n, Hq=Hkv * group, Hkv=Hkv, D=D, P=P, new_lo=rng.choice([0, 1]),
                    new_hi=_log(rng, 1, 64 if tree else max(2, 20000 // n)), old_hi=_log(rng, 1, 4000), R=R,
                    start=rng.choice([0, D - R]), inter=rng.random() < 0.5, scaling=scaling, tree=tree)
    if op == "attn":
        B = _log(rng, 1, 128)
        hi = _log(rng, 1, max(2, min(65536, (1 << 21) // (B * Hkv))))
        tree = rng.random() < 0.6
        new_hi = min(hi, _log(rng, 1, 96) if tree else rng.choice([1, _log(rng, 1, 1024)]))
        return dict(op=op, B=B, Hq=Hkv * group, Hkv=Hkv, D=D, P=P, lo=rng.choice([0, 1, hi // 3, hi]), hi=hi,
                    new_lo=rng.choice([0, 1, new_hi]), new_hi=new_hi, tree=tree)
    return dict(op=op, layers=_log(rng, 1, 32), n=_log(rng, 1, 48), Hkv=Hkv, D=D, P=P, draft=_log(rng, 1, 64),
                depth=rng.randint(1, 10), old_hi=_log(rng, 1, 600))


# Structure (lengths, trees, accepted paths) follows from the case alone; values follow from the seed.

def _tree(n, depth, rng):
    """Parents of a tree of n nodes: a chain of min(n, depth), then side branches no deeper than it."""
    chain = min(n, depth)
    parents, deep = [], []
    for i in range(n):
        if i < chain:
            parents.append(i - 1)
        else:
            parents.append(rng.choice([j for j in range(-1, i) if j < 0 or deep[j] < chain - 1]))
        deep.append(0 if parents[i] < 0 else deep[parents[i]] + 1)
    return parents, deep


def _lengths(case):
    """(positions in the cache, new ones among them, trees) of each sequence; the longest always among them."""
    if case["op"] == "append":
        n = case["n"]
        rng = random.Random(case["n"] + 77 * case["new_hi"])
        new = [case["new_lo"] if rng.random() < 0.05 else _log(rng, max(1, case["new_lo"]), case["new_hi"])
               for _ in range(n)]
        new[rng.randrange(n)] = case["new_hi"]
        lens = [m + rng.randint(0, case["old_hi"]) for m in new]
    elif case["op"] == "attn":
        n, lo, hi = case["B"], case["lo"], case["hi"]
        rng = random.Random(1000 * n + hi)
        lens = [lo if lo == hi or rng.random() < 0.05 else max(lo, _log(rng, max(lo, 1), hi)) for _ in range(n)]
        lens[rng.randrange(n)] = hi
        new = []
        for a in lens:
            m = case["new_lo"] if rng.random() < 0.05 else _log(rng, max(1, case["new_lo"]), case["new_hi"])
            new.append(min(a, case["new_hi"] if a == hi else m))
    else:
        n = case["n"]
        rng = random.Random(n + 13 * case["draft"])
        new = [case["draft"]] * n
        lens = [case["draft"] + rng.randint(0, case["old_hi"]) for _ in range(n)]
    trees = [_tree(m, case.get("depth") or 1 + m // 4, rng) for m in new] if case.get("tree", case["op"] == "keep") else None
    return lens, new, trees


def _paths(case):
    """Accepted nodes of each sequence of a keep case: the way to a node, or nothing.  Side nodes have indices of at
    least the longest path's length, so that a pass finds the rows of the next one as it found its own."""
    lens, new, trees = _lengths(case)
    rng = random.Random(5 + case["n"])
    got = []
    for parents, _ in trees:
        path, i = [], rng.randrange(-1 if rng.random() < 0.1 else 0, len(parents))
        while i >= 0:
            path.append(i)
            i = parents[i]
        got.append(path[::-1])
    return got


# ---------------------------------------------------------------------------------------------------------- inputs

def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _prefix(counts):
    at = [0]
    for c in counts:
        at.append(at[-1] + c)
    return _ints(at)


def _frequencies(case):
    """Radians per position of each pair (fp64), and the rotated pairs' length factor, for a context stretched by 8
    from 8192: all slower, a larger base, or the slow ones only (turning less than once in the old context) with a ramp
    to the fast ones (32 times)."""
    R, factor, old = case["R"], 8.0, 8192
    c = torch.arange(0, R, 2, dtype=torch.float64) / R
    w, m = 500000.0 ** -c, 1.0
    if case["scaling"] == "linear":
        w = w / factor
    elif case["scaling"] == "base":
        w = (500000.0 * factor ** (R / max(R - 2, 1))) ** -c
    elif case["scaling"] == "parts":
        turns = old * w / (2 * math.pi)
        keep = ((turns - 1) / (32 - 1)).clamp(0, 1)
        w = w * keep + w / factor * (1 - keep)
        m = 0.1 * math.log(factor) + 1.0
    return w, m


def _plan(st, case):
    w, m = _frequencies(case)
    if own:
        import exact_attention_07_gb300 as fa
        st["rope"] = fa.rope_plan(inv_freq=w, mscale=m, start=case["start"], interleaved=case["inter"], device=DEV)
    st["w"], st["m"] = w.to(DEV), m


def _bits(trees):
    """mask int32 [total, words] of the trees' nodes."""
    words = max(1, max(-(-len(p) // 32) for p, _ in trees))
    rows = []
    for parents, _ in trees:
        seen = []
        for i, p in enumerate(parents):
            seen.append((seen[p] if p >= 0 else 0) | 1 << i)
        for s in seen:
            w = [s >> 32 * j & 0xffffffff for j in range(words)]
            rows.append([x - (1 << 32) if x >> 31 else x for x in w])
    return torch.tensor(rows, dtype=torch.int32, device=DEV).view(-1, words)


def _cache(st, lens, case, gen, layers=None):
    """A pool whose sequences own pages in random order."""
    P = case["P"]
    need = [-(-a // P) for a in lens]
    total = sum(need) + 3
    order = torch.randperm(total, generator=gen, device=DEV).to(torch.int32)
    table = torch.full((len(lens), max(1, max(need))), -1, dtype=torch.int32, device=DEV)
    at = 0
    for i, c in enumerate(need):
        table[i, :c] = order[at:at + c]
        at += c
    shape = (total, 2, case["Hkv"], P, case["D"])
    st["pool"] = torch.empty(shape if layers is None else (layers, *shape), dtype=torch.bfloat16, device=DEV)
    for part in st["pool"].view(-1, *shape[-3:]).split(max(1, (1 << 26) // math.prod(shape[-3:]))):
        part.copy_(torch.randn(part.shape, generator=gen, device=DEV))
    if layers is None:  # keys have a few louder dimensions
        loud = 1 + 3 * (torch.rand(case["Hkv"], 1, case["D"], generator=gen, device=DEV) < 0.03).to(torch.bfloat16)
        st["pool"][:, 0] *= loud
    st["table"], st["lens"] = table, _ints(lens)


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    op, H, D = case["op"], case["Hkv"], case["D"]
    st = dict(case=case)

    def rand(*shape):
        return torch.randn(*shape, generator=gen, device=DEV)

    if op == "rope":
        T, Hq = case["T"], case["Hq"]
        _plan(st, case)
        if case["dtype"] == "bf16":  # q, k and v lie side by side in the projection's rows
            x = rand(T, Hq + 2 * H, D).bfloat16()
            q, k = x[:, :Hq], x[:, Hq:Hq + H]
        else:
            q, k = rand(T, Hq, D), rand(T, H, D)
        if case["kind"] == "dense":
            B = 2 if T % 2 == 0 and case.get("name") is None else 1
            q, k = (t.unflatten(0, (B, -1)).transpose(1, 2) for t in (q, k))
            first = torch.randint(0, 1 << 17, (B, 1), generator=gen, device=DEV)
            st["pos"] = (first + torch.arange(T // B, device=DEV)).to(torch.int32)
        else:
            st["pos"] = torch.randint(0, 1 << 17, (T,), generator=gen, device=DEV, dtype=torch.int32)
        st["q"], st["k"] = q, k
        return st
    lens, new, trees = _lengths(case)
    total = sum(new)
    st["cu"], st["total"] = _prefix(new), total
    if trees is not None:
        st["mask"] = _bits(trees)
    if op == "keep":
        _cache(st, lens, case, gen, layers=case["layers"])
        paths = _paths(case)
        st["counts"] = _ints([len(p) for p in paths])
        st["keep"] = _ints([x for p in paths for x in p + [-1] * (case["draft"] - len(p))])
        return st
    _cache(st, lens, case, gen)
    if op == "append":
        _plan(st, case)
        x = rand(total, case["Hq"] + 2 * H, D).bfloat16()
        st["q"], st["k"], st["v"] = x.split([case["Hq"], H, H], 1)
        st["pos"] = _ints([a - m + d for a, m, t in zip(lens, new, trees) for d in t[1]]) if trees else None
    else:
        st["q"] = rand(total, case["Hq"], D).bfloat16()
        st["new"], st["old"] = new, [a - m for a, m in zip(lens, new)]
    return st


# ------------------------------------------------------------------------------------------------------ plain forms

def _turn(x, cos, sin, case, m):
    """x [..., D] in fp32 with its pairs turned; cos, sin broadcast over [..., R / 2]."""
    R, s = case["R"], case["start"]
    y = x.clone()
    part = x[..., s:s + R]
    if case["inter"]:
        a, b = part[..., 0::2], part[..., 1::2]
    else:
        a, b = part[..., :R // 2], part[..., R // 2:]
    ya, yb = m * (a * cos - b * sin), m * (a * sin + b * cos)
    y[..., s:s + R] = torch.stack((ya, yb), -1).flatten(-2) if case["inter"] else torch.cat((ya, yb), -1)
    return y


def _plain_rope(st):
    c = st["case"]
    back = c["dtype"] == "grad"
    theta = st["pos"].double().unsqueeze(-1) * st["w"]
    cos, sin = theta.cos().float(), (-theta if back else theta).sin().float()
    axis = 1 if c["kind"] == "dense" else -2
    cos, sin = cos.unsqueeze(axis), sin.unsqueeze(axis)
    dt = torch.float32 if c["dtype"] == "fp32" else torch.bfloat16
    return [_turn(st[n].float(), cos, sin, c, st["m"]).to(dt).contiguous() for n in ("q", "k")]


def _new_rows(st):
    """(slot, position) of each row of a call."""
    cu, lens = st["cu"].long(), st["lens"].long()
    t = torch.arange(st["total"], device=DEV)
    s = torch.searchsorted(cu, t, right=True) - 1
    return s, lens[s] - cu[s + 1] + t


def _plain_append(st):
    c = st["case"]
    s, p = _new_rows(st)
    pos = p if st["pos"] is None else st["pos"]
    theta = pos.double().view(-1, 1, 1) * st["w"]
    cos, sin = theta.cos().float(), theta.sin().float()
    page, row = st["table"][s, p // c["P"]].long(), p % c["P"]
    st["pool"][page, 0, :, row] = _turn(st["k"].float(), cos, sin, c, st["m"]).bfloat16()
    st["pool"][page, 1, :, row] = st["v"]
    return [st["pool"], _turn(st["q"].float(), cos, sin, c, st["m"]).bfloat16()]


def _visible(st, s, i0, n):
    """Which of sequence s's n new positions each of its rows sees: truth values [n, n]."""
    j = torch.arange(n, device=DEV)
    if not st["case"]["tree"]:
        return j <= j.unsqueeze(1)
    return (st["mask"][i0:i0 + n][:, j // 32] >> j % 32 & 1).bool()


def _plain_attn(st):
    c, q = st["case"], st["q"]
    T, Hq, D = q.shape
    H, P = c["Hkv"], c["P"]
    o = torch.empty(T, Hq, D, dtype=torch.bfloat16, device=DEV)
    lse = torch.empty(Hq, T, dtype=torch.float32, device=DEV)
    i0 = 0
    for s, (old, n) in enumerate(zip(st["old"], st["new"])):
        if n == 0:
            continue
        a = old + n
        pages = st["table"][s, :-(-a // P)].long()
        seen = _visible(st, s, i0, n).repeat_interleave(Hq // H, 0)
        heads = max(1, min(H, (1 << 30) // (n * (Hq // H) * a)))
        for h in range(0, H, heads):
            kv = st["pool"][pages, :, h:h + heads].float()  # [pages, 2, heads, P, D]
            k, v = (kv[:, w].transpose(0, 1).flatten(1, 2)[:, :a] for w in (0, 1))
            g = k.shape[0]
            x = q[i0:i0 + n].float().view(n, H, -1, D)[:, h:h + g].permute(1, 0, 2, 3).reshape(g, -1, D)
            z = (x @ k.transpose(1, 2)) * (1.0 / math.sqrt(D))
            z[:, :, old:].masked_fill_(~seen, -math.inf)
            top = z.amax(-1, keepdim=True)
            e = torch.exp(z - top)
            total = e.sum(-1, keepdim=True)
            y = ((e @ v) / total).view(g, n, -1, D).permute(1, 0, 2, 3).flatten(1, 2)
            cols = slice(h * (Hq // H), (h + g) * (Hq // H))
            o[i0:i0 + n, cols] = y.bfloat16()
            lse[cols, i0:i0 + n] = (top + total.log()).view(g, n, -1).transpose(1, 2).flatten(0, 1)
        i0 += n
    return [o, lse]


def _plain_keep(st):
    c, cu = st["case"], st["cu"].long()
    j = torch.arange(c["draft"], device=DEV)
    took = j < st["counts"].unsqueeze(1)
    src = st["keep"].view(-1, c["draft"])
    s, j = took.nonzero(as_tuple=True)
    base = st["lens"].long()[s] - c["draft"]
    a, b = base + src[s, j], base + j
    pool, P = st["pool"], c["P"]
    rows = pool[:, st["table"][s, a // P].long(), :, :, a % P]
    pool[:, st["table"][s, b // P].long(), :, :, b % P] = rows
    return [pool, (st["counts"] - (cu[1:] - cu[:-1])).to(torch.int32)]


# -------------------------------------------------------------------------------------------------- the package's calls

def _own(st):
    import exact_attention_07_gb300 as fa
    c = st["case"]
    if c["op"] == "rope":
        if c["dtype"] == "grad":
            return list(fa.fa_rope_bwd(st["q"], st["k"], st["rope"], positions=st["pos"], dtype=torch.bfloat16))
        return list(fa.fa_rope(st["q"], st["k"], st["rope"], positions=st["pos"]))
    if c["op"] == "append":
        q = fa.fa_kv16_append(st["k"], st["v"], st["cu"], st["pool"], st["table"], st["lens"], rope=st["rope"],
                              positions=st["pos"], q=st["q"])
        return [st["pool"], q]
    if c["op"] == "attn":
        o, lse = fa.fa_fwd_kv16(st["q"], st["cu"], st["pool"], st["table"], st["lens"], mask=st.get("mask"),
                                causal=not c["tree"])
        return [o, lse]
    back = fa.fa_kv16_keep(st["keep"], st["counts"], st["cu"], st["pool"], st["table"], st["lens"])
    return [st["pool"], back]


def run(state):
    if own:
        return _own(state)
    return {"rope": _plain_rope, "append": _plain_append, "attn": _plain_attn, "keep": _plain_keep}[state["case"]["op"]](state)


# ------------------------------------------------------------------------------------------------------ exact values

def _exact_turn(x, theta, case, m):
    """x in fp64 with its pairs, as complex numbers, times m exp(i theta); theta broadcasts over [..., R / 2]."""
    R, s = case["R"], case["start"]
    y = x.double().clone(memory_format=torch.contiguous_format)
    lo = torch.arange(R // 2, device=DEV)
    first = s + (2 * lo if case["inter"] else lo)
    second = first + (1 if case["inter"] else R // 2)
    z = torch.complex(y[..., first], y[..., second]) * torch.polar(torch.full_like(theta, m), theta)
    y[..., first], y[..., second] = z.real, z.imag
    return y


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "rope":
        theta = st["pos"].double()[..., None] * (st["w"] if case["dtype"] != "grad" else -st["w"])
        theta = theta[:, None] if case["kind"] == "dense" else theta[..., None, :]
        return [_exact_turn(st[n], theta, case, st["m"]) for n in ("q", "k")]
    if op == "append":
        pool = st["pool"].double()
        lens, new, _ = _lengths(case)
        slots = [i for i, m in enumerate(new) for _ in range(m)]
        places = [a - m + j for a, m in zip(lens, new) for j in range(m)]
        page = st["table"].cpu()[slots, [p // case["P"] for p in places]].long().to(DEV) if places else None
        row = torch.tensor([p % case["P"] for p in places], device=DEV)
        pos = torch.tensor(places, device=DEV) if st["pos"] is None else st["pos"]
        theta = (pos.double()[:, None] * st["w"])[:, None]
        if places:
            pool[page, 0, :, row] = _exact_turn(st["k"], theta, case, st["m"])
            pool[page, 1, :, row] = st["v"].double()
        return [pool, _exact_turn(st["q"], theta, case, st["m"])]
    if op == "attn":
        return _exact_attn(st)
    pool = st["pool"].double() if st["pool"].numel() < 1 << 32 else st["pool"].clone()
    lens, new, _ = _lengths(case)
    table = st["table"].tolist()
    P = case["P"]
    for s, path in enumerate(_paths(case)):
        for j, i in enumerate(path):
            a, b = lens[s] - new[s] + i, lens[s] - new[s] + j
            if a != b:
                pool[:, table[s][b // P], :, :, b % P] = pool[:, table[s][a // P], :, :, a % P]
    return [pool, _ints([len(p) - m for p, m in zip(_paths(case), new)])]


def _exact_attn(st):
    c = st["case"]
    lens, new, trees = _lengths(c)
    T, Hq, D = st["q"].shape
    G, P = Hq // c["Hkv"], c["P"]
    o = torch.zeros(T, Hq, D, dtype=torch.float64, device=DEV)
    lse = torch.full((Hq, T), -math.inf, dtype=torch.float64, device=DEV)
    at = 0
    for s, (a, n) in enumerate(zip(lens, new)):
        if n == 0:
            continue
        bias = torch.zeros(n, a, dtype=torch.float64, device=DEV)
        if trees is None:
            bias[:, a - n:] = torch.full((n, n), -math.inf, dtype=torch.float64, device=DEV).triu(1)
        else:
            own_keys = torch.full((n, n), -math.inf, dtype=torch.float64)
            for i, p in enumerate(trees[s][0]):
                if p >= 0:
                    own_keys[i] = own_keys[p]
                own_keys[i, i] = 0.0
            bias[:, a - n:] = own_keys.to(DEV)
        index = torch.arange(a, device=DEV)
        page = st["table"][s].long()[index // P]
        for h in range(c["Hkv"]):
            k = st["pool"][page, 0, h, index % P].double()
            v = st["pool"][page, 1, h, index % P].double()
            for g in range(G):
                z = torch.addmm(bias, st["q"][at:at + n, h * G + g].double(), k.T, alpha=D ** -0.5)
                top = torch.logsumexp(z, 1)
                lse[h * G + g, at:at + n] = top
                o[at:at + n, h * G + g] = torch.exp(z - top[:, None]) @ v
        at += n
    return [o, lse]


# -------------------------------------------------------------------------------------------------------------- work

@functools.lru_cache(maxsize=64)
def _work(items):
    case = dict(items)
    op, H, D = case["op"], case["Hkv"], case["D"]
    if op == "rope":
        n = case["T"] * (case["Hq"] + H)
        size = {"bf16": 4, "grad": 6, "fp32": 8}[case["dtype"]]
        return {"bytes": n * D * size + 4 * case["T"], "flops": 3 * n * case["R"]}
    lens, new, trees = _lengths(case)
    if op == "append":
        rows = sum(new) * (case["Hq"] + 2 * H)
        return {"bytes": rows * D * 4 + 8 * len(new), "flops": 3 * sum(new) * (case["Hq"] + H) * case["R"]}
    if op == "attn":
        live = [(a, m) for a, m in zip(lens, new) if m]
        pairs = sum((a - m) * m for a, m in live)
        pairs += sum(d + 1 for t in trees for d in t[1]) if trees else sum(m * (m + 1) // 2 for _, m in live)
        q = sum(new) * case["Hq"]
        return {"bytes": 4 * D * H * sum(a for a, _ in live) + q * (4 * D + 4) + (8 * sum(new) if trees else 0),
                "flops": 4 * D * case["Hq"] * pairs}
    moved = sum(i != j for p in _paths(case) for j, i in enumerate(p))
    return {"bytes": moved * case["layers"] * 2 * H * D * 4 + 8 * len(new), "flops": 0}


def work(case):
    return dict(_work(tuple(sorted((k, v) for k, v in case.items() if k != "name"))))
