"""Benchmark cases of the paged 4-bit KV cache (kv4): attention over it, quantising append, dequantising read and the
page operations.  `run` computes each case with elementary torch operations in fp32, or, where `own` is true, with the
package's kernels; `exact` computes the floating outputs in fp64 from the definitions.

The cache: a pool of pages, uint8 [pages, Hkv, page_size / 16, 18 D].  The last axis is one unit, 16 consecutive
positions of one KV head:

    K codes   8 D bytes  [16 keys][D / 2]               low nibble = even dimension
    V codes   8 D bytes  [2 halves][D / 16][4 pairs][16] low nibble = even key of the pair of keys
    K scales    D bytes  [16 keys][D / 16]              e4m3
    V scales    D bytes  [D / 16][16 keys]              e4m3

Codes are e2m1 (0, 0.5, 1, 1.5, 2, 3, 4, 6 and a sign bit); a value is code * scale of its 16 dimensions * scale of its
KV head.  Position p of the sequence in slot s lives in page table[s, p // page_size].  A page used by several
sequences has that many references and is full.
"""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"
SECTION = {"kc": 0, "vc": 8, "ks": 16, "vs": 17}  # byte offsets of a unit's sections, in units of D


# ----------------------------------------------------------------------------------------------------------- cases

def listed():
    return [
        # one chat request early in its answer: a single token over a short cache, where latency counts
        dict(name="attn_one_short", op="attn", B=1, Hq=32, Hkv=8, D=128, Lq=1, P=64, lo=777, hi=777, causal=True,
             scaled=False),
        # a decode step of a running server: 32 requests of very different ages, single-key ones among them
        dict(name="attn_ragged", op="attn", B=32, Hq=32, Hkv=8, D=128, Lq=1, P=64, lo=1, hi=8192, causal=True,
             scaled=True),
        # the repository's decode workload (B = 8, 32 x 8 heads, 32768 keys) over the 4-bit cache
        dict(name="attn_long", op="attn", B=8, Hq=32, Hkv=8, D=128, Lq=1, P=64, lo=32768, hi=32768, causal=False,
             scaled=False),
        # checking 3 drafted tokens and one more (speculative decoding), small heads, small pages, 16 rows per KV head
        dict(name="attn_draft", op="attn", B=6, Hq=16, Hkv=4, D=64, Lq=4, P=16, lo=900, hi=9001, causal=True,
             scaled=True),
        # the cache write of a decode step: one new token for each of 64 requests
        dict(name="append_step", op="append", n=64, Hkv=8, D=128, P=64, new_lo=1, new_hi=1, old_hi=4096, scaled=False),
        # the cache write of a packed batch of 8 prompts of 512 to 8192 tokens
        dict(name="append_prompts", op="append", n=8, Hkv=8, D=128, P=64, new_lo=512, new_hi=8192, old_hi=0,
             scaled=True),
        # a short shared prefix read back for the prompt that follows it
        dict(name="read_prefix", op="read", n=2, Hkv=4, D=64, P=16, lo=37, hi=1001, scaled=True),
        # long cached documents read back for prompt attention
        dict(name="read_documents", op="read", n=4, Hkv=8, D=128, P=128, lo=9000, hi=32768, scaled=False),
        # a beam-search step on one layer's pool: 2 parents, 7 children
        dict(name="fork_beams", op="fork", layers=1, n=2, kids=7, Hkv=2, D=64, P=16, lo=20, hi=300, spare=8),
        # 64 samples of 4 prompts: the last pages of 32 layers are copied for each
        dict(name="fork_samples", op="fork", layers=32, n=4, kids=64, Hkv=8, D=128, P=64, lo=1000, hi=4000, spare=64),
        # a small pool where the requests of one half leave and come anew, then those of the other half
        dict(name="turnover_small", op="turnover", layers=1, n=5, Hkv=2, D=64, P=16, lo=1, hi=200, spare=6),
        # the same in 16 layers of a server's pool, compacted twice
        dict(name="turnover_layers", op="turnover", layers=16, n=12, Hkv=8, D=128, P=64, lo=500, hi=4000, spare=64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "append", "append", "read", "fork", "turnover"])
    D, P, Hkv = rng.choice([64, 128]), rng.choice([16, 32, 64, 128, 256]), rng.choice([1, 2, 3, 4, 8])
    scaled = rng.random() < 0.5
    if op == "attn":
        B = _log(rng, 1, 128)
        hi = _log(rng, 1, max(2, min(32768, (1 << 21) // (B * Hkv))))
        Lq = rng.choice([1, 1, 1, 2, 3, 5])
        return dict(op=op, B=B, Hq=Hkv * rng.choice([1, 2, 4, 5, 8, 12]), Hkv=Hkv, D=D, Lq=Lq, P=P,
                    lo=rng.choice([0, 1, hi // 3, hi]), hi=hi, causal=rng.random() < 0.7, scaled=scaled)
    if op == "append":
        n = _log(rng, 1, 64)
        top = max(1, 32000 // n) if rng.random() < 0.5 else 2
        return dict(op=op, n=n, Hkv=Hkv, D=D, P=P, new_lo=rng.choice([0, 1]), new_hi=_log(rng, 1, top) + 1,
                    old_hi=_log(rng, 1, 2000), scaled=scaled)
    if op == "read":
        n = _log(rng, 1, 32)
        hi = _log(rng, 2, 64000 // n)
        return dict(op=op, n=n, Hkv=Hkv, D=D, P=P, lo=rng.randint(0, hi), hi=hi, scaled=scaled)
    if op == "fork":
        n = rng.randint(1, 6)
        hi = _log(rng, 2, 2000)
        return dict(op=op, layers=_log(rng, 1, 16), n=n, kids=_log(rng, 1, 48), Hkv=Hkv, D=D, P=P,
                    lo=rng.randint(1, hi), hi=hi, spare=rng.randint(0, 40))
    hi = _log(rng, 2, 2000)
    return dict(op=op, layers=_log(rng, 1, 12), n=rng.randint(1, 10), Hkv=Hkv, D=D, P=P, lo=rng.randint(1, hi), hi=hi,
                spare=rng.randint(0, 40))


def _lengths(case):
    """The case's sequence lengths: spread over their logarithm from lo to hi, the longest always among them."""
    n = case["B"] if case["op"] == "attn" else 2 * case["n"] if case["op"] == "turnover" else case["n"]
    lo, hi = case["lo"], case["hi"]
    rng = random.Random(1000 * n + hi)
    if case["op"] == "turnover":  # the two halves hold the same lengths in another order
        half = [_log(rng, lo, hi) for _ in range(case["n"])]
        return half + half[::-1]
    got = [lo if lo == hi or rng.random() < 0.05 else max(lo, _log(rng, max(lo, 1), hi)) for _ in range(n)]
    got[rng.randrange(n)] = hi
    return got


def _append_lengths(case):
    """(tokens in the cache before, new tokens) of each sequence."""
    rng = random.Random(case["n"] + 77 * case["new_hi"])
    old = [rng.randint(0, case["old_hi"]) for _ in range(case["n"])]
    new = [case["new_lo"] if rng.random() < 0.05 else _log(rng, max(1, case["new_lo"]), case["new_hi"])
           for _ in range(case["n"])]
    new[rng.randrange(case["n"])] = case["new_hi"]
    return old, new


def _pages(n, P):
    return -(-n // P)


# ---------------------------------------------------------------------------------------------------------- inputs

def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _scattered(lens, P, gen, width=None, spare=3):
    """A table whose sequences own pages in random order; (table, number of pages)."""
    need = [_pages(x, P) for x in lens]
    total = sum(need) + spare
    order = torch.randperm(total, generator=gen, device=DEV).to(torch.int32)
    table = torch.full((len(lens), width or max(1, max(need))), -1, dtype=torch.int32, device=DEV)
    at = 0
    for i, c in enumerate(need):
        table[i, :c] = order[at:at + c]
        at += c
    return table, total


def _packed_prefix(counts):
    return _ints([0] + list(np.cumsum(counts)))


def _levels(x):
    """e2m1 codes (0..15) of values, ties to even, saturating."""
    a = x.abs()
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75).to(torch.uint8) + (a > 1.25).to(torch.uint8)
            + (a >= 1.75).to(torch.uint8) + (a > 2.5).to(torch.uint8) + (a >= 3.5).to(torch.uint8)
            + (a > 5.0).to(torch.uint8))
    return code + 8 * torch.signbit(x).to(torch.uint8)


def _quantise(x, g):
    """Codes and e4m3 scales of rows x [..., D]; g: the head scales, or None.  In 64 bits: a value on the border
    between two codes goes by the last bit of the quotient."""
    x = x.double() if g is None else x.double() / g.double()
    xg = x.unflatten(-1, (-1, 16))
    six = torch.full((1,), 6.0, dtype=torch.float64, device=DEV)  # a tensor: a quotient, not a product with 1 / 6
    s8 = (xg.abs().amax(-1) / six).clamp(max=448.0).to(torch.float8_e4m3fn)
    s = s8.double().unsqueeze(-1)
    codes = _levels(torch.where(s > 0, xg / s, torch.zeros_like(xg)))
    return codes.flatten(-2), s8.view(torch.uint8)


def _fill(pool, D, gen):
    """Random contents for a whole pool: rows of N(0, 1) with a few louder dimensions, quantised."""
    pages, H, U = pool.shape[:3]
    loud = 1 + 4 * (torch.rand(H, 1, D, generator=gen, device=DEV) < 0.03).float()
    step = max(1, (1 << 25) // (H * U * 16 * D))
    for a in range(0, pages, step):
        part = pool[a:a + step]
        n = part.shape[0]
        for which in ("k", "v"):
            x = torch.randn(n, H, U * 16, D, generator=gen, device=DEV) * (loud if which == "k" else 1.0)
            codes, s = _quantise(x, None)
            codes, s = codes.view(n, H, U, 16, D), s.view(n, H, U, 16, D // 16)
            if which == "k":
                part[..., :8 * D] = (codes[..., 0::2] | codes[..., 1::2] << 4).flatten(3)
                part[..., 16 * D:17 * D] = s.flatten(3)
            else:
                pair = codes[..., 0::2, :] | codes[..., 1::2, :] << 4  # [.., 8 pairs, D]
                pair = pair.view(n, H, U, 2, 4, D // 16, 16).transpose(4, 5)
                part[..., 8 * D:16 * D] = pair.flatten(3)
                part[..., 17 * D:] = s.transpose(-1, -2).flatten(3)


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    op, H, D, P = case["op"], case["Hkv"], case["D"], case["P"]
    st = dict(case=case)
    if case.get("scaled"):
        st["k_scale"] = 0.5 + torch.rand(H, generator=gen, device=DEV)
        st["v_scale"] = 0.5 + torch.rand(H, generator=gen, device=DEV)
    else:
        st["k_scale"] = st["v_scale"] = None
    if op in ("attn", "read"):
        lens = _lengths(case)
        st["table"], pages = _scattered(lens, P, gen)
        st["pool"] = torch.zeros(pages, H, P // 16, 18 * D, dtype=torch.uint8, device=DEV)
        _fill(st["pool"], D, gen)
        st["lens"] = _ints(lens)
        if op == "attn":
            st["q"] = torch.randn(case["B"], case["Hq"], case["Lq"], D, generator=gen, device=DEV).bfloat16()
        else:
            st["cu"], st["total"] = _packed_prefix(lens), sum(lens)
    elif op == "append":
        old, new = _append_lengths(case)
        lens = [a + b for a, b in zip(old, new)]
        st["table"], pages = _scattered(lens, P, gen)
        st["pool"] = torch.zeros(pages, H, P // 16, 18 * D, dtype=torch.uint8, device=DEV)
        st["lens"], st["cu"], st["total"] = _ints(lens), _packed_prefix(new), sum(new)
        loud = 1 + 4 * (torch.rand(H, D, generator=gen, device=DEV) < 0.03).float()
        st["k"] = (torch.randn(st["total"], H, D, generator=gen, device=DEV) * loud).bfloat16()
        st["v"] = torch.randn(st["total"], H, D, generator=gen, device=DEV).bfloat16()
    else:
        lens = _lengths(case)
        need = [_pages(x, P) for x in lens]
        if op == "fork":
            pages = sum(need) + case["kids"] + case["spare"]
            used = torch.randperm(pages, generator=gen, device=DEV)[:sum(need)].to(torch.int32)
            slots, width = case["n"] + case["kids"], max(need) + 1
            st["parents"] = torch.randint(0, case["n"], (case["kids"],), generator=gen, device=DEV).to(torch.int32)
            st["children"] = torch.arange(case["n"], slots, device=DEV).to(torch.int32)
        else:
            # the first half's pages lie in front of the second half's
            pages = sum(need) + case["spare"]
            used = torch.arange(sum(need), device=DEV).to(torch.int32)
            slots, width = 2 * case["n"], max(need)
            st["halves"] = [torch.arange(case["n"] * h, case["n"] * (h + 1), device=DEV).to(torch.int32) for h in (0, 1)]
            st["new"] = [_ints(lens[:case["n"]]), _ints(lens[case["n"]:])]
        table = torch.full((slots, width), -1, dtype=torch.int32, device=DEV)
        at = 0
        for i, c in enumerate(need):
            table[i, :c] = used[at:at + c]
            at += c
        st["table"] = table
        st["lens"] = _ints(lens + [0] * (slots - len(lens)))
        st["refs"] = torch.zeros(pages, dtype=torch.int32, device=DEV)
        st["refs"][used.long()] = 1
        st["pool"] = torch.randint(0, 256, (case["layers"], pages, H, P // 16, 18 * D), generator=gen, device=DEV,
                                   dtype=torch.uint8)
    return st


# ------------------------------------------------------------------------------------------------------ plain forms

def _value(code):
    """e2m1 codes to fp32."""
    c = code.int()
    e, f = (c >> 1) & 3, (c & 1).float()
    mag = torch.where(e == 0, 0.5 * f, (1.0 + 0.5 * f) * (2.0 ** (e - 1).float()))
    return torch.where(c >= 8, -mag, mag)


def _unit_values(u, D):
    """K and V of units u [..., 18 D] in fp32, without the head scales: two tensors [..., 16, D]."""
    kc = u[..., :8 * D].unflatten(-1, (16, D // 2))
    k = torch.stack((_value(kc & 15), _value(kc >> 4)), -1).flatten(-2)
    ks = u[..., 16 * D:17 * D].contiguous().view(torch.float8_e4m3fn).float().unflatten(-1, (16, D // 16))
    vc = u[..., 8 * D:16 * D].unflatten(-1, (2, D // 16, 4, 16)).transpose(-2, -3)  # [.., half, pair, group, 16]
    v = torch.stack((_value(vc & 15), _value(vc >> 4)), -3)  # [.., half, pair, parity, group, 16]
    v = v.flatten(-2).flatten(-4, -2)
    vs = u[..., 17 * D:].contiguous().view(torch.float8_e4m3fn).float().unflatten(-1, (D // 16, 16)).transpose(-1, -2)
    return k * ks.repeat_interleave(16, -1), v * vs.repeat_interleave(16, -1)


def _plain_attn(st):
    c, q = st["case"], st["q"]
    B, Hq, Lq, D = q.shape
    H, P, G = c["Hkv"], c["P"], Hq // c["Hkv"]
    units = st["pool"][st["table"].clamp(min=0).long()]  # [B, W, H, U, 18 D]
    k, v = _unit_values(units.transpose(1, 2), D)  # [B, H, W, U, 16, D]
    k, v = k.flatten(2, 4), v.flatten(2, 4)
    if st["k_scale"] is not None:
        k, v = k * st["k_scale"].view(1, H, 1, 1), v * st["v_scale"].view(1, H, 1, 1)
    lens = st["lens"].view(B, 1, 1, 1)
    key = torch.arange(k.shape[2], device=DEV).view(1, 1, 1, -1)
    seen = key < lens
    if c["causal"]:
        seen = seen & (key <= torch.arange(Lq, device=DEV).repeat(G).view(1, 1, -1, 1) + lens - Lq)
    v = torch.where((key < lens).transpose(2, 3), v, torch.zeros_like(v))
    s = torch.matmul(q.float().view(B, H, G * Lq, D), k.transpose(2, 3)) * (1.0 / math.sqrt(D))
    s = torch.where(seen, s, torch.full_like(s, -math.inf))
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = torch.exp(s - m)
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / torch.where(total > 0, total, torch.ones_like(total))
    return o.view(B, Hq, Lq, D), (m + torch.log(total)).view(B, Hq, Lq)


def _rows(st):
    """(page, position within the page) of each packed row: rows of sequence s are its last positions."""
    cu, P = st["cu"].long(), st["case"]["P"]
    row = torch.arange(st["total"], device=DEV)
    s = torch.searchsorted(cu, row, right=True) - 1
    pos = st["lens"].long()[s] - cu[s + 1] + row
    return st["table"].long()[s, pos // P], pos % P


def _addresses(st):
    """Byte addresses in the flat pool of each row's K codes, V codes, K scales and V scales: [rows, H, ...]."""
    D, H, U = st["case"]["D"], st["case"]["Hkv"], st["case"]["P"] // 16
    page, at = _rows(st)
    h = torch.arange(H, device=DEV)
    unit = ((page.view(-1, 1) * H + h) * U + (at // 16).view(-1, 1)) * (18 * D)
    key = (at % 16).view(-1, 1, 1)
    unit, d, g = unit.unsqueeze(-1), torch.arange(D, device=DEV), torch.arange(D // 16, device=DEV)
    kc = unit + key * (D // 2) + torch.arange(D // 2, device=DEV)
    vc = unit + 8 * D + key // 8 * (4 * D) + d // 16 * 64 + key % 8 // 2 * 16 + d % 16
    ks = unit + 16 * D + key * (D // 16) + g
    vs = unit + 17 * D + g * 16 + key
    return kc, vc, ks, vs, (at % 2 == 1).view(-1, 1, 1)


def _plain_append(st):
    H = st["case"]["Hkv"]
    flat = st["pool"].view(-1)
    kc, vc, ks, vs, odd = _addresses(st)
    gk, gv = ((None, None) if st["k_scale"] is None else (st["k_scale"].view(1, H, 1), st["v_scale"].view(1, H, 1)))
    codes, s = _quantise(st["k"], gk)
    flat[kc] = codes[..., 0::2] | codes[..., 1::2] << 4
    flat[ks] = s
    codes, s = _quantise(st["v"], gv)
    flat[vs] = s
    for high in (False, True):  # the two keys of a pair share their bytes: first the even ones, then the odd ones
        rows = (odd == high).flatten()
        a, new = vc[rows], codes[rows]
        flat[a] = (flat[a] & 15) | new << 4 if high else (flat[a] & 240) | new


def _plain_read(st):
    H, flat = st["case"]["Hkv"], st["pool"].view(-1)
    kc, vc, ks, vs, odd = _addresses(st)
    b = flat[kc]
    k = torch.stack((_value(b & 15), _value(b >> 4)), -1).flatten(-2)
    b = flat[vc]
    v = _value(torch.where(odd, b >> 4, b & 15))
    k = k * flat[ks].view(torch.float8_e4m3fn).float().repeat_interleave(16, -1)
    v = v * flat[vs].view(torch.float8_e4m3fn).float().repeat_interleave(16, -1)
    if st["k_scale"] is not None:
        k, v = k * st["k_scale"].view(1, H, 1), v * st["v_scale"].view(1, H, 1)
    return k.bfloat16(), v.bfloat16()


def _owned(st, slots):
    """Which entries of the slots' table rows are pages in use."""
    P = st["case"]["P"]
    return torch.arange(st["table"].shape[1], device=DEV) < ((st["lens"][slots] + P - 1) // P).unsqueeze(1)


def _plain_release(st, slots):
    slots = slots.long()
    pages = st["table"][slots][_owned(st, slots)].long()
    st["refs"].index_add_(0, pages, torch.full_like(pages, -1, dtype=torch.int32))
    st["table"][slots] = -1
    st["lens"][slots] = 0


def _plain_fork(st):
    P, par, kid = st["case"]["P"], st["parents"].long(), st["children"].long()
    table, refs, pool = st["table"], st["refs"], st["pool"]
    full, rest = st["lens"][par].long() // P, st["lens"][par].long() % P
    col = torch.arange(table.shape[1], device=DEV)
    shared = col < full.unsqueeze(1)
    table[kid] = torch.where(shared, table[par], torch.full_like(table[par], -1))
    pages = table[par][shared].long()
    refs.index_add_(0, pages, torch.ones_like(pages, dtype=torch.int32))
    st["lens"][kid] = st["lens"][par]
    some = rest > 0
    fresh = torch.nonzero(refs == 0).flatten()
    left = fresh.numel() - some.sum()
    dst = fresh[(torch.cumsum(some, 0) - 1)[some]]
    src = table[par[some], full[some]].long()
    table[kid[some], full[some]] = dst.int()
    refs[dst] = 1
    keep = torch.arange(P // 16, device=DEV) * 16 < rest[some].unsqueeze(1)  # units that hold rows
    i, u = torch.nonzero(keep, as_tuple=True)
    pool[:, dst[i], :, u] = pool[:, src[i], :, u]
    return torch.stack((left.int(), torch.zeros_like(left).int()))


def _plain_compact(st):
    refs, pool, table = st["refs"], st["pool"], st["table"]
    live = refs > 0
    index = torch.arange(refs.numel(), device=DEV)
    front = index < live.sum()
    src, dst = index[live & ~front], index[~live & front]
    pool[:, dst] = pool[:, src]
    refs[dst] = refs[src]
    refs[src] = 0
    to = index.clone()
    to[src] = dst
    owned = _owned(st, torch.arange(table.shape[0], device=DEV))
    table[owned] = to[table[owned].long()].int()


def _plain_reserve(st, slots, new):
    P, slots = st["case"]["P"], slots.long()
    before = (st["lens"][slots] + P - 1) // P
    st["lens"][slots] += new
    after = (st["lens"][slots] + P - 1) // P
    col = torch.arange(st["table"].shape[1], device=DEV)
    wanted = (col >= before.unsqueeze(1)) & (col < after.unsqueeze(1))
    fresh = torch.nonzero(st["refs"] == 0).flatten()
    need = wanted.sum()
    rows = st["table"][slots]
    rows[wanted] = fresh[:need].int()
    st["table"][slots] = rows
    st["refs"][fresh[:need]] = 1
    return torch.stack(((fresh.numel() - need).int(), torch.zeros_like(need).int()))


# ------------------------------------------------------------------------------------------------------------- run

def run(st):
    c, op = st["case"], st["case"]["op"]
    if own:
        import exact_attention_07_gb300 as fa
    heads = dict(k_scale=st["k_scale"], v_scale=st["v_scale"])
    if op == "attn":
        if own:
            return fa.fa_fwd_kv4(st["q"], st["pool"], st["table"], st["lens"], causal=c["causal"], **heads)
        return _plain_attn(st)
    if op == "append":  # a chunk enters the cache, and what the cache now holds of it is read back for its attention
        if own:
            fa.fa_kv4_append(st["k"], st["v"], st["cu"], st["pool"], st["table"], st["lens"], **heads)
            return fa.fa_kv4_read(st["cu"], st["total"], st["pool"], st["table"], st["lens"], **heads)
        _plain_append(st)
        return _plain_read(st)
    if op == "read":
        if own:
            return fa.fa_kv4_read(st["cu"], st["total"], st["pool"], st["table"], st["lens"], **heads)
        return _plain_read(st)
    pages = (st["pool"], st["table"], st["lens"], st["refs"])
    if op == "fork":  # the children of the last step leave, those of the next one share their parents' pages
        if own:
            fa.fa_kv4_release(st["children"], st["table"], st["lens"], st["refs"], c["P"])
            info = fa.fa_kv4_fork(st["parents"], st["children"], *pages)
        else:
            _plain_release(st, st["children"])
            info = _plain_fork(st)
        return info, st["table"], st["lens"], st["refs"], st["pool"].view(torch.int32)
    infos = []
    for half, new in zip(st["halves"], st["new"]):  # a half leaves, the rest moves to the front, new requests come
        if own:
            fa.fa_kv4_release(half, st["table"], st["lens"], st["refs"], c["P"])
            fa.fa_kv4_compact(*pages)
            infos.append(fa.fa_kv4_reserve(new, st["table"], st["lens"], st["refs"], c["P"], seq_ids=half))
        else:
            _plain_release(st, half)
            _plain_compact(st)
            infos.append(_plain_reserve(st, half, new))
    return infos, st["table"], st["lens"], st["refs"], st["pool"].view(torch.int32)


# ------------------------------------------------------------------------------------------------------------ work

def work(case):
    op, H, D, P = case["op"], case["Hkv"], case["D"], case["P"]
    row = H * 18 * D / 16  # the cache's bytes of one position
    if op == "attn":
        keys, rows = sum(_lengths(case)), case["B"] * case["Hq"] * case["Lq"]
        return {"bytes": keys * row + rows * (2 * D + 4 * D + 4) + 4 * case["B"] + 4 * keys / P,
                "flops": 4.0 * D * keys * case["Hq"] * case["Lq"]}
    if op == "append":
        return {"bytes": sum(_append_lengths(case)[1]) * (2 * row + 2 * H * 4 * D), "flops": 0}
    if op == "read":
        return {"bytes": sum(_lengths(case)) * (row + H * 4 * D), "flops": 0}
    lens = _lengths(case)
    pages = sum(_pages(x, P) for x in lens)
    if op == "fork":  # on average over the parents that a child may have
        units = sum(_pages(x % P, 16) for x in lens) / case["n"] * case["kids"]
        table = 4.0 * case["kids"] * sum(_pages(x, P) for x in lens) / case["n"]
        return {"bytes": 2 * case["layers"] * units * H * 18 * D + 5 * table, "flops": 0}
    # each half's pages move once; its table entries and references are read and written
    return {"bytes": 2 * case["layers"] * pages * P * row + 32.0 * pages, "flops": 0}


# ----------------------------------------------------------------------------------------------------------- exact

def _exact_tables():
    """The value of every byte as an e4m3 number, and of every nibble as an e2m1 number, in fp64."""
    e4m3 = []
    for b in range(256):
        e, f = b >> 3 & 15, b & 7
        x = math.nan if b & 127 == 127 else math.ldexp(f, -9) if e == 0 else math.ldexp(8 + f, e - 10)
        e4m3.append(-x if b >= 128 else x)
    e2m1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
    e2m1 += [-x for x in e2m1]
    return (torch.tensor(e4m3, dtype=torch.float64, device=DEV), torch.tensor(e2m1, dtype=torch.float64, device=DEV))


def _exact_cache(st, slot, count):
    """K and V [H, count, D] in fp64 of one sequence's first `count` positions."""
    D, P, H = st["case"]["D"], st["case"]["P"], st["case"]["Hkv"]
    e4m3, e2m1 = _exact_tables()
    u = st["pool"][st["table"][slot, :_pages(count, P)].long()].transpose(0, 1).reshape(H, -1, 18 * D).int()
    out = []
    for which in ("kc", "vc"):
        a = SECTION[which] * D
        codes = torch.empty(H, u.shape[1], 16, D, dtype=torch.float64, device=DEV)
        byte = u[..., a:a + 8 * D]
        if which == "kc":
            byte = byte.reshape(H, -1, 16, D // 2)
            codes[..., 0::2], codes[..., 1::2] = e2m1[byte % 16], e2m1[byte // 16]
            scale = e4m3[u[..., 16 * D:17 * D].reshape(H, -1, 16, D // 16)]
        else:
            byte = byte.reshape(H, -1, 2, D // 16, 4, 16).permute(0, 1, 2, 4, 3, 5).reshape(H, -1, 8, D)
            codes[:, :, 0::2], codes[:, :, 1::2] = e2m1[byte % 16], e2m1[byte // 16]
            scale = e4m3[u[..., 17 * D:].reshape(H, -1, D // 16, 16)].transpose(2, 3)
        x = (codes.view(H, -1, 16, D // 16, 16) * scale.unsqueeze(-1)).reshape(H, -1, D)[:, :count]
        g = st["k_scale" if which == "kc" else "v_scale"]
        out.append(x if g is None else x * g.double().view(H, 1, 1))
    return out


def _exact_quantised(x, g):
    """What the cache holds of bf16 rows x [T, H, D], in fp64."""
    x = x.double() if g is None else x.double() / g.double().view(1, -1, 1)
    x = x.unflatten(-1, (-1, 16))
    a = (x.abs().amax(-1, keepdim=True) / torch.full((1,), 6.0, dtype=torch.float64, device=DEV)).clamp(max=448.0)
    two = torch.tensor([2.0 ** k for k in range(-9, 10)], dtype=torch.float64, device=DEV)  # a power may be rounded
    step = two[(torch.frexp(a)[1] - 1).clamp(min=-6) - 3 + 9]  # spacing of e4m3 there
    s = torch.round(a / step) * step
    y = torch.where(s > 0, x / torch.where(s > 0, s, torch.ones_like(s)), torch.zeros_like(x)).clamp(-6.0, 6.0)
    step = two[(torch.frexp(y)[1] - 1).clamp(min=0) - 1 + 9]  # spacing of e2m1 there
    x = (torch.round(y / step) * step * s).flatten(-2)
    return x if g is None else x * g.double().view(1, -1, 1)


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "append":
        return _exact_quantised(st["k"], st["k_scale"]), _exact_quantised(st["v"], st["v_scale"])
    if op == "read":
        parts = [_exact_cache(st, s, n) for s, n in enumerate(_lengths(case))]
        return tuple(torch.cat([p[i] for p in parts], 1).transpose(0, 1).contiguous() for i in (0, 1))
    if op == "attn":
        B, Hq, Lq, D = st["q"].shape
        o = torch.zeros(B, Hq, Lq, D, dtype=torch.float64, device=DEV)
        lse = torch.full((B, Hq, Lq), -math.inf, dtype=torch.float64, device=DEV)
        for b, n in enumerate(_lengths(case)):
            if n == 0:
                continue
            k, v = _exact_cache(st, b, n)
            for h in range(Hq):
                s = st["q"][b, h].double() @ k[h // (Hq // case["Hkv"])].T / math.sqrt(D)
                if case["causal"]:
                    s[torch.arange(n, device=DEV) > torch.arange(Lq, device=DEV).view(-1, 1) + (n - Lq)] = -math.inf
                lse[b, h] = torch.logsumexp(s, -1)
                w = torch.exp(s - lse[b, h].unsqueeze(1).clamp(min=-1e300))
                o[b, h] = w @ v[h // (Hq // case["Hkv"])]
        return o, lse
    return None  # the page operations move whole numbers and bytes
