"""GPU tests of the paged bf16 KV cache against its fp64 oracle (oracle/kv16.py).

Rows that are copied are compared bit for bit; turned rows and attention are held to bounds derived from the
arithmetic (``turn_tolerance``, ``attention_tolerance``), not to a measured error.  What a call must not look at holds
NaN in these caches: pages of nobody, positions behind a sequence's end, table entries behind its last page (-7).
"""
import math
import threading

import numpy as np
import pytest
import torch

import exact_attention_07_gb300 as fa
from oracle import kv16

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    fa.load_library()


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def f64(t):
    return t.detach().double().cpu().numpy()


def prefix(counts):
    return np.concatenate([[0], np.cumsum(counts)])


def cache(lens, H, D, P, seed, spare=2, loud=1.0, slots=None, layers=None):
    """A pool with normal rows at the used positions and NaN elsewhere, pages in random order.  Returns (pool, table,
    lens) on the device; slot s holds lens[s] positions."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-n // P) for n in lens]
    N = max(1, sum(need) + spare)
    order = torch.randperm(N, generator=g).to(torch.int32)
    table = torch.full((len(lens), max(1, max(need)) + 1), -7, dtype=torch.int32)
    L = layers or 1
    pool = torch.full((L, N, 2, H, P, D), math.nan, dtype=torch.bfloat16)
    at = 0
    for s, n in enumerate(lens):
        table[s, :need[s]] = order[at:at + need[s]]
        at += need[s]
        for i in range(need[s]):
            m = min(P, n - i * P)
            x = torch.randn(L, 2, H, m, D, generator=g)
            x[:, 0, ..., :3] *= loud
            pool[:, table[s, i], :, :, :m] = x.bfloat16()
    pool = pool if layers else pool[0]
    return pool.to(DEV), table.to(DEV), i32(lens)


def tree(n, rng):
    return [int(rng.integers(-1, i)) if rng.random() < 0.7 else i - 1 for i in range(n)]


def check_attention(q, o, lse, cu, pool, table, slots, lens, scale, own, what=""):
    """Every sequence against the oracle; own[s]: [n, n] truth values."""
    pool64, tab = f64(pool), table.cpu().numpy()
    for s, slot in enumerate(slots):
        a, b = cu[s], cu[s + 1]
        if a == b:
            continue
        k, v = kv16.rows(pool64, tab, slot, lens[slot])
        q64 = f64(q[a:b])
        ro, rl, mag = kv16.attention(q64, k, v, scale, own[s])
        go, gl = f64(o[a:b]), f64(lse[:, a:b])
        assert np.array_equal(np.isneginf(rl), np.isneginf(gl)), f"{what}: empty rows of sequence {s}"
        empty = np.isneginf(rl).T
        assert not go[empty].any(), f"{what}: O of empty rows"
        to, tl = kv16.attention_tolerance(q64, np.nan_to_num(k), scale, ro, rl, mag)
        err = np.abs(go - ro)
        assert (err <= to).all(), f"{what}: O of sequence {s}: {err.max()}, bound {to[err > to].max()}, at {np.argwhere(~(err <= to))[0]}"
        fin = np.isfinite(rl)
        if fin.any():
            assert np.abs(gl[fin] - rl[fin]).max() <= tl, f"{what}: LSE of sequence {s}: {np.abs(gl[fin] - rl[fin]).max()} > {tl}"


def visible(mode, n, parents=None):
    if mode == "tree":
        return kv16.ancestors(parents)
    return np.tril(np.ones((n, n), bool)) if mode == "causal" else np.ones((n, n), bool)


def run_attention(lens, new, Hq, H, D, P, mode, seed=0, loud=1.0, scale=None, q=None, **kw):
    rng = np.random.default_rng(seed)
    pool, table, tl = cache(lens, H, D, P, seed, loud=loud)
    cu = prefix(new)
    T = int(cu[-1])
    if q is None:
        q = torch.randn(T, Hq, D, generator=torch.Generator().manual_seed(seed + 1)).bfloat16().to(DEV)
    parents = [tree(n, rng) for n in new]
    mask = None
    if mode == "tree":
        mask = fa.draft_mask([p for t in parents for p in t], cu.tolist())[0].to(DEV)
    o, lse = fa.fa_fwd_kv16(q, i32(cu), pool, table, tl, mask=mask, causal=mode == "causal", softmax_scale=scale, **kw)
    assert fa.fa_last_launch_count() == 2
    fa.fa_check()
    assert o.dtype is torch.bfloat16 and o.shape == q.shape and lse.shape == (Hq, T)
    check_attention(q, o, lse, cu, pool, table, range(len(lens)), lens, scale or D ** -0.5,
                    [visible(mode, n, p) for n, p in zip(new, parents)], mode)


ATTENTION = [  # lens, new, Hq, Hkv, D, page, mode
    ([1], [1], 1, 1, 64, 16, "causal"), ([1], [1], 4, 1, 128, 256, "tree"), ([777], [1], 32, 8, 128, 64, "causal"),
    ([128], [1], 2, 1, 128, 16, "full"), ([129, 127, 1, 255], [1, 1, 1, 2], 4, 2, 64, 32, "causal"),
    ([40, 0, 300, 5], [3, 0, 7, 5], 6, 2, 128, 16, "tree"), ([90, 33], [33, 33], 5, 1, 64, 16, "tree"),
    ([500, 70], [70, 70], 8, 1, 128, 64, "tree"), ([1000], [300], 4, 4, 128, 128, "causal"),
    ([300], [300], 2, 1, 64, 256, "causal"), ([260, 17], [65, 17], 12, 1, 128, 32, "full"),
    ([600], [3], 128, 1, 64, 64, "tree"), ([130, 700], [2, 2], 127, 1, 128, 16, "causal"),
    ([20000], [1], 8, 2, 128, 64, "causal"), ([9000, 5, 6000], [20, 5, 1], 8, 2, 64, 16, "tree"),
    ([2500], [129], 2, 2, 64, 128, "tree")]


@pytest.mark.parametrize("lens,new,Hq,H,D,P,mode", ATTENTION)
def test_attention(lens, new, Hq, H, D, P, mode):
    run_attention(lens, new, Hq, H, D, P, mode, seed=sum(lens) + D)


@pytest.mark.parametrize("B,mode", [(130, "causal"), (1000, "tree")])
def test_attention_of_many_sequences(B, mode):
    rng = np.random.default_rng(B)
    new = rng.integers(0, 4, B)
    lens = [int(n + rng.integers(0, 60)) for n in new]
    run_attention(lens, new.tolist(), 2, 1, 64, 16, mode, seed=B)


@pytest.mark.parametrize("D,mode,top", [(128, "tree", 40), (64, "causal", 24), (128, "full", 1), (64, "tree", 6),
                                        (64, "full", 40), (128, "causal", 70)])
def test_attention_of_mixed_sequences(D, mode, top):
    """Blocks whose shares mix items of one and two tiles of rows, short ones and long ones, alone and cut."""
    rng = np.random.default_rng(D + top)
    B = 330
    new = rng.integers(0, top + 1, B)
    lens = [int(n + rng.choice([0, rng.integers(0, 130), rng.integers(0, 700), rng.integers(900, 2500)], p=[.1, .5, .3, .1]))
            for n in new]
    run_attention(lens, new.tolist(), 8, 1, D, 32, mode, seed=D + top)


def test_a_call_gives_the_same_bits_every_time():
    """Many items of a few tiles, the last of them partly masked: V of a tile must not be looked over while the stage
    still waits for an earlier one."""
    rng = np.random.default_rng(12)
    B, H, P = 150, 8, 16
    lens = [int(n) for n in rng.integers(385, 520, B)]
    pool, table, tl = cache(lens, H, 128, P, 12)
    q = torch.randn(B, 4 * H, 128, generator=torch.Generator().manual_seed(13)).bfloat16().to(DEV)
    cu = i32(range(B + 1))
    first = fa.fa_fwd_kv16(q, cu, pool, table, tl, causal=True)
    other = torch.zeros((), dtype=torch.bool, device=DEV)
    for _ in range(1500):
        o, lse = fa.fa_fwd_kv16(q, cu, pool, table, tl, causal=True)
        other |= (o != first[0]).any() | (lse != first[1]).any()
    fa.fa_check()
    assert not other.item()
    check_attention(q, *first, range(B + 1), pool, table, range(B), lens, 128 ** -0.5, [visible("causal", 1)] * B)


def test_attention_of_thousands_of_sequences():
    """More sequences in every block's share than it looks ahead."""
    rng = np.random.default_rng(9)
    new = (rng.random(8000) < 0.9).astype(int)
    run_attention([int(n + rng.integers(0, 4)) for n in new], new.tolist(), 1, 1, 64, 16, "causal", seed=9)


def test_pools_beyond_32_bits():
    """Rows whose element offsets in the pool pass 2^32: append, attention and keep (in the second of two layers)."""
    H, Hq, D, P = 8, 8, 128, 256
    per = 2 * H * P * D
    pages = (1 << 32) // per + 3
    pool = torch.empty(2, pages, 2, H, P, D, dtype=torch.bfloat16, device=DEV)
    one = pool[1]
    table, lens = i32([[pages - 1, pages - 2, -7]]), i32([300])
    g = torch.Generator().manual_seed(3)
    q, k, v = (torch.randn(300, h, D, generator=g).bfloat16().to(DEV) for h in (Hq, H, H))
    for layer in pool:
        fa.fa_kv16_append(k, v, i32([0, 300]), layer, table, lens)
    o, lse = fa.fa_fwd_kv16(q[-5:], i32([0, 5]), one, table, lens, causal=True)
    fa.fa_check()
    ro, rl, mag = kv16.attention(f64(q[-5:]), f64(k), f64(v), D ** -0.5, visible("causal", 5))
    to, tl = kv16.attention_tolerance(f64(q[-5:]), f64(k), D ** -0.5, ro, rl, mag)
    assert (np.abs(f64(o) - ro) <= to).all() and np.abs(f64(lse) - rl).max() <= tl
    fa.fa_kv16_keep(i32([1, 3, 4, 0, 0]), i32([3]), i32([0, 5]), pool, table, lens)
    fa.fa_check()
    for layer in pool:
        got = torch.cat([layer[pages - 1, :, :, :], layer[pages - 2, :, :, :44]], 2)[:, :, 295:300]
        want = torch.stack([k[[296, 298, 299, 298, 299]], v[[296, 298, 299, 298, 299]]]).transpose(1, 2)
        assert torch.equal(got, want)


@pytest.mark.parametrize("mode", ["causal", "tree"])
def test_attention_with_sharp_scores(mode):
    """Scores of tens: rows that one key dominates, references that move many times."""
    run_attention([3000, 200], [9, 9], 8, 2, 128, 64, mode, seed=3, loud=12.0, scale=0.3)


@pytest.mark.parametrize("order", ["fused", "heads first", "one"])
def test_attention_of_strided_queries(order):
    T, Hq, H, D = 6, 4, 2, 128
    g = torch.Generator().manual_seed(8)
    if order == "fused":
        q = torch.randn(T, Hq + 2 * H, D, generator=g).bfloat16().to(DEV)[:, :Hq]
    elif order == "heads first":
        q = torch.randn(Hq, T, D, generator=g).bfloat16().to(DEV).transpose(0, 1)
    else:
        T = 1
        q = torch.randn(3, Hq + 2, D, generator=g).bfloat16().to(DEV)[1:2, 1:1 + Hq]
    run_attention([50], [T], Hq, H, D, 16, "causal", q=q)


def test_rows_that_see_nothing_and_masked_rows_of_anything():
    """A tree whose nodes see an arbitrary set, some none at all, with NaN and infinities in K and V of nodes that
    nobody or only some see; the rest of the word in the mask is set and means nothing."""
    H, Hq, D, P, n = 1, 3, 128, 16, 40
    lens, new = [n, n + 200], [n, n]
    pool, table, tl = cache(lens, H, D, P, 21)
    rng = np.random.default_rng(5)
    own = [rng.random((n, n)) < 0.3 for _ in new]
    own[0][7] = own[0][30] = False  # no prefix either: nothing to see
    own[1][7] = False
    for s in (0, 1):
        own[s][:, 11] = False  # node 11: seen by nobody
        own[s][:, 12] = False
        own[s][3, 12] = True   # node 12: by row 3 only
    tab = table.cpu().numpy()
    for s, slot in enumerate((0, 1)):
        for node, kv, val in ((11, 0, math.nan), (11, 1, math.nan), (12, 1, math.inf)):
            p = lens[s] - n + node
            pool[int(tab[slot, p // P]), kv, 0, p % P, 5:9] = val
    words = 3  # more than needed
    bits = np.zeros((2 * n, 32 * words), bool)
    for s in (0, 1):
        bits[s * n:(s + 1) * n, :n] = own[s]
        bits[s * n:(s + 1) * n, n:] = True
    mask = torch.from_numpy(np.packbits(bits, axis=1, bitorder="little").copy().view(np.int32)).to(DEV)
    q = torch.randn(2 * n, Hq, D, generator=torch.Generator().manual_seed(1)).bfloat16().to(DEV)
    cu = prefix(new)
    o, lse = fa.fa_fwd_kv16(q, i32(cu), pool, table, tl, mask=mask)
    fa.fa_check()
    got = f64(o)
    for s in (0, 1):
        hit = got[s * n + 3]
        assert np.isposinf(hit[:, 5:9]).all() and np.isfinite(hit[:, :5]).all() and np.isfinite(hit[:, 9:]).all()
    rest = np.isfinite(got)
    rest[[3, n + 3]] = True
    assert rest.all()
    clean = pool.clone()
    for s, slot in enumerate((0, 1)):
        for node in (11, 12):
            p = lens[s] - n + node
            clean[int(tab[slot, p // P]), 1, 0, p % P, 5:9] = 0.0
            if node == 11:
                clean[int(tab[slot, p // P]), 0, 0, p % P, 5:9] = 0.0
    pool64 = f64(clean)  # with finite values, the infinity a 0: its rows' other dimensions and all other rows
    for s in (0, 1):
        k, v = kv16.rows(pool64, tab, s, lens[s])
        q64 = f64(q[s * n:(s + 1) * n])
        ro, rl, mag = kv16.attention(q64, k, v, D ** -0.5, own[s])
        to, tl_ = kv16.attention_tolerance(q64, k, D ** -0.5, ro, rl, mag)
        go, gl = got[s * n:(s + 1) * n].copy(), f64(lse[:, s * n:(s + 1) * n])
        go[3, :, 5:9] = ro[3, :, 5:9]
        assert (np.abs(go - ro) <= to).all()
        assert np.array_equal(np.isneginf(rl), np.isneginf(gl)) and not go[np.isneginf(rl).T].any()
        fin = np.isfinite(rl)
        assert np.abs(gl[fin] - rl[fin]).max() <= tl_


@pytest.mark.parametrize("n,mode", [(150, "causal"), (150, "tree"), (5, "causal")])
def test_infinite_values_reach_the_rows_that_see_them(n, mode):
    """A value of +inf at one of the call's positions: +inf for the rows behind it, nothing for those in front."""
    H, Hq, D, P, L = 1, 4, 64, 32, 400
    pool, table, tl = cache([L], H, D, P, 4)
    at = n // 2
    p = L - n + at
    pool[int(table[0, p // P]), 1, 0, p % P, 33] = math.inf
    q = torch.randn(n, Hq, D, generator=torch.Generator().manual_seed(1)).bfloat16().to(DEV)
    mask = fa.draft_mask(list(range(-1, n - 1)), [0, n])[0].to(DEV) if mode == "tree" else None
    o, _ = fa.fa_fwd_kv16(q, i32([0, n]), pool, table, tl, mask=mask, causal=mode == "causal")
    fa.fa_check()
    bad = ~torch.isfinite(o)
    assert torch.isposinf(o[at:, :, 33]).all()
    bad[at:, :, 33] = False
    assert not bad.any()


def test_rows_behind_the_last_sequence_and_padded_batches():
    H, Hq, D, P = 2, 4, 64, 16
    lens = [50, 0, 70]
    pool, table, tl = cache(lens, H, D, P, 31)
    ids, new = [2, 1, 0, 1, 1], [4, 0, 2, 0, 0]
    cu = prefix(new)
    T = int(cu[-1]) + 3
    q = torch.randn(T, Hq, D, generator=torch.Generator().manual_seed(1)).bfloat16().to(DEV)
    out = torch.full((T, Hq, D), 7.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((Hq, T), 7.0, device=DEV)
    o, l = fa.fa_fwd_kv16(q, i32(cu), pool, table, tl, causal=True, seq_ids=i32(ids), out=out, lse=lse)
    fa.fa_check()
    assert o is out and l is lse and (out[-3:] == 7).all() and (lse[:, -3:] == 7).all()
    check_attention(q, out, lse, cu, pool, table, ids, lens, D ** -0.5, [visible("causal", n) for n in new])
    before = pool.clone()
    k = torch.randn(2, T, H, D, generator=torch.Generator().manual_seed(2)).bfloat16().to(DEV)
    y = torch.full_like(q, 7.0)
    got = fa.fa_kv16_append(k[0], k[1], i32(cu), pool, table, tl, seq_ids=i32(ids), rope=fa.rope_plan(D), q=q, q_out=y)
    fa.fa_check()
    assert got is y and (y[-3:] == 7).all() and not (y[:-3] == 7).all(-1).any()
    changed = (pool.view(torch.int16) != before.view(torch.int16)).any(-1).sum().item()
    assert changed <= 2 * H * sum(new)


# ------------------------------------------------------------------ append

APPEND = [  # lens, new, Hq, Hkv, D, page, R, start, interleaved, positions
    ([1], [1], 1, 1, 64, 16, 64, 0, False, False), ([40, 0, 300, 5], [3, 0, 7, 5], 4, 2, 128, 16, 128, 0, False, False),
    ([65, 64, 63], [2, 1, 17], 6, 3, 64, 64, 32, 16, True, True), ([700], [700], 2, 1, 128, 256, 64, 64, False, True),
    ([5000, 3000], [4100, 13], 4, 4, 128, 32, 128, 0, True, False)]


@pytest.mark.parametrize("lens,new,Hq,H,D,P,R,start,inter,given", APPEND)
def test_append(lens, new, Hq, H, D, P, R, start, inter, given):
    pool, table, tl = cache(lens, H, D, P, sum(lens))
    before = pool.clone()
    cu = prefix(new)
    T = int(cu[-1])
    g = torch.Generator().manual_seed(T)
    x = torch.randn(T, Hq + 2 * H, D, generator=g).bfloat16().to(DEV)
    q, k, v = x.split([Hq, H, H], 1)
    w = [10000.0 ** (-2 * c / R) for c in range(R // 2)]
    rope = fa.rope_plan(R, start=start, interleaved=inter, mscale=0.75)
    at = np.concatenate([np.arange(a - n, a) for a, n in zip(lens, new)]).astype(np.int64)
    pos = np.random.default_rng(T).integers(0, 1 << 20, T) if given else at
    y = fa.fa_kv16_append(k, v, i32(cu), pool, table, tl, rope=rope, positions=i32(pos) if given else None, q=q)
    assert fa.fa_last_launch_count() == 1
    fa.fa_check()
    tab = table.cpu().numpy()
    slot = np.repeat(np.arange(len(new)), new)
    page, row = torch.from_numpy(tab[slot, at // P]).long(), torch.from_numpy(at % P)
    got_k, got_v = pool[page, 0, :, row], pool[page, 1, :, row]
    assert torch.equal(got_v, v)
    for a, b, what in ((got_k, k, "k"), (y, q, "q")):
        want = kv16.turn(f64(b), pos, w, 0.75, start, inter)
        tol = kv16.turn_tolerance(f64(b), want, 1.0, R // 2, True)
        assert (np.abs(f64(a) - want) <= tol).all(), what
    before[page, :, :, row] = pool[page, :, :, row]
    assert torch.equal(before.view(torch.int16), pool.view(torch.int16)), "other positions"


def test_append_without_rope_and_in_place():
    pool, table, tl = cache([20], 2, 64, 16, 1)
    k, v = torch.randn(2, 3, 2, 64, generator=torch.Generator().manual_seed(1)).bfloat16().to(DEV)
    assert fa.fa_kv16_append(k, v, i32([0, 3]), pool, table, tl) is None
    fa.fa_check()
    tab = table.cpu()[0].long()
    p = torch.tensor([17, 18, 19])
    assert torch.equal(pool[tab[p // 16], 0, :, p % 16], k) and torch.equal(pool[tab[p // 16], 1, :, p % 16], v)
    rope = fa.rope_plan(64)
    q = torch.randn(3, 4, 64, generator=torch.Generator().manual_seed(2)).bfloat16().to(DEV)
    want = fa.fa_kv16_append(k, v, i32([0, 3]), pool, table, tl, rope=rope, q=q)
    assert fa.fa_kv16_append(k, v, i32([0, 3]), pool, table, tl, rope=rope, q=q, q_out=q) is q
    assert torch.equal(q, want)


# ------------------------------------------------------------------ keep

def test_keep():
    lens, n, P, H, D, layers = [60, 23, 300, 40, 100], [12, 5, 260, 3, 0], 16, 2, 64, 3
    paths = [[0, 3, 11], [], list(range(0, 260, 1)), [2], []]
    paths[2] = [i for i in range(260) if i % 7 != 3]  # long lists, in several rounds
    pool, table, tl = cache(lens, H, D, P, 9, layers=layers)
    want = pool.clone()
    tab = table.cpu().numpy()
    for s, path in enumerate(paths):
        base = lens[s] - n[s]
        old = [pool[:, int(tab[s, (base + i) // P]), :, :, (base + i) % P].clone() for i in path]
        for j, x in enumerate(old):
            want[:, int(tab[s, (base + j) // P]), :, :, (base + j) % P] = x
    cu = prefix(n)
    keep = np.full(int(cu[-1]), -5, np.int32)
    for s, path in enumerate(paths):
        keep[cu[s]:cu[s] + len(path)] = path
    back = fa.fa_kv16_keep(i32(keep), i32([len(p) for p in paths]), i32(cu), pool, table, tl)
    assert fa.fa_last_launch_count() == 1
    fa.fa_check()
    assert torch.equal(pool.view(torch.int16), want.view(torch.int16))
    assert back.tolist() == [len(p) - m for p, m in zip(paths, n)]


@pytest.mark.parametrize("keep,count", [([0, 0, 1], 3), ([1, 0, 2], 2), ([0, 4, 5], 2), ([-1, 1, 2], 1), ([0, 1, 2], 5),
                                        ([0, 1, 2], -1)])
def test_keep_refuses_lists_that_are_none(keep, count):
    pool, table, tl = cache([30, 30], 1, 64, 16, 2)
    before = pool.clone()
    back = fa.fa_kv16_keep(i32([2, 0, 0, 0] + keep + [9]), i32([1, count]), i32([0, 4, 8]), pool, table, tl)
    with pytest.raises(fa.FAError, match="invalid"):
        fa.fa_check()
    assert back.tolist() == [-3, 0]
    tab = table.cpu()
    assert torch.equal(pool[tab[1, :2].long()].view(torch.int16), before[tab[1, :2].long()].view(torch.int16))


# ------------------------------------------------------------------ together

@pytest.mark.parametrize("D,P", [(64, 16), (128, 64)])
def test_drafting_loop(D, P):
    """Three rounds of drafting: reserve, append the trees, attend, keep a path, give the rest back.  What the cache
    holds then equals one built from the accepted rows alone, and attention over it agrees with the oracle."""
    H, Hq, B = 2, 4, 3
    rng = np.random.default_rng(D)
    pages = 64
    pool = fa.kv16_pool(pages, H, P, D)
    table = torch.zeros(B, 16, dtype=torch.int32, device=DEV)
    lens, refs = i32([0] * B), i32([0] * pages)
    rope, w = fa.rope_plan(D), [10000.0 ** (-2 * c / D) for c in range(D // 2)]
    g = torch.Generator().manual_seed(D)
    held = [np.zeros((0, 2, H, D)) for _ in range(B)]
    new = [37, 5, 21]  # prompts
    for turn in range(4):
        parents = [list(range(-1, n - 1)) if turn == 0 else tree(n, rng) for n in new]
        cu = prefix(new)
        mask, depth = fa.draft_mask([p for t in parents for p in t], cu.tolist())
        before = lens.cpu().numpy()
        assert fa.fa_kv4_reserve(i32(new), table, lens, refs, P)[1].item() == 0
        x = torch.randn(int(cu[-1]), Hq + 2 * H, D, generator=g).bfloat16().to(DEV)
        q, k, v = x.split([Hq, H, H], 1)
        pos = np.repeat(before, new) + depth.numpy()
        q = fa.fa_kv16_append(k, v, i32(cu), pool, table, lens, rope=rope, positions=i32(pos), q=q)
        o, lse = fa.fa_fwd_kv16(q, i32(cu), pool, table, lens, mask=mask.to(DEV))
        fa.fa_check()
        now = lens.tolist()
        check_attention(q, o, lse, cu, pool, table, range(B), now, D ** -0.5, [kv16.ancestors(t) for t in parents])
        paths = []
        for s, t in enumerate(parents):
            path, i = [], new[s] - 1 if turn == 0 else int(rng.integers(-1, new[s]))
            while i >= 0:
                path.insert(0, i)
                i = t[i]
            paths.append(path)
            kk, vv = kv16.rows(f64(pool), table.cpu().numpy(), s, now[s])
            held[s] = np.concatenate([held[s], np.stack([kk, vv], 1)[now[s] - new[s] + np.array(path, int)]])
        keep = np.zeros(int(cu[-1]), np.int32)
        for s, path in enumerate(paths):
            keep[cu[s]:cu[s] + len(path)] = path
        back = fa.fa_kv16_keep(i32(keep), i32([len(p) for p in paths]), i32(cu), pool, table, lens)
        assert fa.fa_kv4_reserve(back, table, lens, refs, P)[1].item() == 0
        fa.fa_check()
        for s in range(B):
            assert lens[s].item() == len(held[s])
            kk, vv = kv16.rows(f64(pool), table.cpu().numpy(), s, len(held[s]))
            assert np.array_equal(np.stack([kk, vv], 1), held[s])
        new = rng.integers(1, 40, B).tolist()
    fa.fa_kv4_release(i32(range(B)), table, lens, refs, P)
    assert refs.sum().item() == 0


def test_chunked_prompt_equals_the_packed_forward():
    """A prompt in chunks through the cache against fa_fwd_varlen on the whole of it: both within their bounds of the
    same values (O here rounded to bf16, 2^-8; P in bf16 on both sides)."""
    H, Hq, D, P, L = 2, 4, 128, 64, 700
    g = torch.Generator().manual_seed(1)
    q, k, v = (torch.randn(L, h, D, generator=g).bfloat16().to(DEV) for h in (Hq, H, H))
    pool, table = fa.kv16_pool(12, H, P, D), torch.zeros(1, 12, dtype=torch.int32, device=DEV)
    lens, refs = i32([0]), i32([0] * 12)
    got = []
    for a, b in ((0, 300), (300, 301), (301, 700)):
        fa.fa_kv4_reserve(i32([b - a]), table, lens, refs, P)
        fa.fa_kv16_append(k[a:b], v[a:b], i32([0, b - a]), pool, table, lens)
        got.append(fa.fa_fwd_kv16(q[a:b], i32([0, b - a]), pool, table, lens, causal=True))
    fa.fa_check()
    cu = i32([0, L])
    o, lse = fa.fa_fwd_varlen(q, k, v, cu, cu, L, L, causal=True)
    assert (torch.cat([x[0] for x in got]).float() - o).abs().max() <= 4 * 2.0 ** -8 * v.abs().max()
    assert (torch.cat([x[1] for x in got], 1) - lse).abs().max() <= 1e-4


# ------------------------------------------------------------------ errors, streams, graphs

def latched(fn):
    fn()
    with pytest.raises(fa.FAError, match="invalid"):
        fa.fa_check()


def test_bad_lengths_slots_pages_and_offsets_are_latched():
    H, D, P = 1, 64, 16
    pool, table, tl = cache([40, 20], H, D, P, 1)
    rope = fa.rope_plan(D)
    q = torch.randn(4, 2, D, generator=torch.Generator().manual_seed(1)).bfloat16().to(DEV)
    k = q[:, :1].contiguous()
    before = pool.clone()

    def both(cu=(0, 2, 4), t=table, l=tl, ids=None, mask=None):
        cu, ids = i32(cu), None if ids is None else i32(ids)
        latched(lambda: fa.fa_fwd_kv16(q, cu, pool, t, l, causal=mask is None, seq_ids=ids, mask=mask))
        if mask is None:
            latched(lambda: fa.fa_kv16_append(k, k, cu, pool, t, l, seq_ids=ids, rope=rope))
            latched(lambda: fa.fa_kv16_keep(i32([1, 0, 1, 0]), i32([1, 1]), cu, pool, t, l, seq_ids=ids))

    both(l=i32([40, 1]))            # fewer positions than rows
    both(l=i32([-1, 20]))
    both(l=i32([1 << 20, 20]))      # more than the table holds
    both(cu=(0, 3, 2))
    both(cu=(1, 2, 4))
    both(cu=(0, 2, 5))
    both(ids=[0, 2])
    both(ids=[-1, 0])
    bad = table.clone()
    bad[1, 1] = pool.shape[0]
    both(t=bad)
    bad[1, 1] = -1
    both(t=bad)
    latched(lambda: fa.fa_kv16_append(k, k, i32([0, 2, 4]), pool, table, tl, seq_ids=i32([1, 1]), rope=rope))
    long = torch.zeros(40, 2, D, dtype=torch.bfloat16, device=DEV)
    latched(lambda: fa.fa_fwd_kv16(long, i32([0, 40, 40]), pool, table, tl,
                                   mask=torch.zeros(40, 1, dtype=torch.int32, device=DEV)))
    assert pool.shape == before.shape


def test_a_lost_copy_ends_the_kernel():
    pool, table, tl = cache([300], 1, 128, 64, 1)
    q = torch.randn(1, 1, 128, generator=torch.Generator().manual_seed(1)).bfloat16().to(DEV)
    fa.load_library().fa_test_inject_fault(1)
    fa.fa_fwd_kv16(q, i32([0, 1]), pool, table, tl, causal=True)
    with pytest.raises(fa.FAError) as e:
        fa.fa_check()
    assert e.value.status == fa.FA_ERR_TIMEOUT
    run_attention([300], [1], 1, 1, 128, 64, "causal")


@pytest.mark.parametrize("lens,new,Hq,D", [([3000, 40], [40, 3], 8, 64), ([3000, 40], [40, 3], 8, 128), ([700], [1], 4, 64)])
def test_a_lost_copy_ends_a_long_call(lens, new, Hq, D):
    pool, table, tl = cache(lens, 1, D, 16, 1)
    q = torch.randn(sum(new), Hq, D, generator=torch.Generator().manual_seed(1)).bfloat16().to(DEV)
    fa.load_library().fa_test_inject_fault(1)
    fa.fa_fwd_kv16(q, i32(prefix(new)), pool, table, tl, causal=True)
    with pytest.raises(fa.FAError) as e:
        fa.fa_check()
    assert e.value.status == fa.FA_ERR_TIMEOUT
    run_attention(lens, new, Hq, 1, D, 16, "causal")


def test_two_graphs_replayed_with_other_lengths():
    """Two captured steps with workspaces of their own, replayed in turn and at once on two streams."""
    H, Hq, D, P = 2, 8, 128, 32
    steps, alive = [], []
    for seed, lens in ((1, [2000, 31]), (2, [400, 3000])):
        pool, table, tl = cache(lens, H, D, P, seed)
        q = torch.randn(4, Hq, D, generator=torch.Generator().manual_seed(seed)).bfloat16().to(DEV)
        cu = i32([0, 2, 4])
        out, lse = torch.empty_like(q), torch.empty(Hq, 4, device=DEV)
        ws = torch.empty(fa.kv16_workspace(4, Hq, H, D), dtype=torch.uint8, device=DEV)
        fa.fa_fwd_kv16(q, cu, pool, table, tl, causal=True, out=out, lse=lse, workspace=ws)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            fa.fa_fwd_kv16(q, cu, pool, table, tl, causal=True, out=out, lse=lse, workspace=ws)
        steps.append((graph, q, pool, table, tl, lens, out, lse))
        alive.append((cu, ws))  # the graphs use them
    streams = [torch.cuda.Stream() for _ in steps]
    for shorter in (0, 5, 40):
        for _, _, _, _, tl, lens, out, _ in steps:
            tl.copy_(i32([max(2, n - shorter) for n in lens]))
            out.fill_(9.0)
        torch.cuda.synchronize()
        for s, st in zip(streams, steps):
            with torch.cuda.stream(s):
                st[0].replay()
        torch.cuda.synchronize()
        fa.fa_check()
        for _, q, pool, table, tl, _, out, lse in steps:
            check_attention(q, out, lse, [0, 2, 4], pool, table, (0, 1), tl.tolist(), D ** -0.5, [visible("causal", 2)] * 2)


def test_other_streams_and_threads():
    pool, table, tl = cache([900, 77], 2, 64, 16, 5)
    q = torch.randn(6, 4, 64, generator=torch.Generator().manual_seed(5)).bfloat16().to(DEV)
    cu = i32([0, 3, 6])
    want = fa.fa_fwd_kv16(q, cu, pool, table, tl, causal=True)
    torch.cuda.synchronize()
    got = [None] * 4

    def work(i):
        s = torch.cuda.Stream()
        for _ in range(20):
            got[i] = fa.fa_fwd_kv16(q, cu, pool, table, tl, causal=True, stream=s if i % 2 else s.cuda_stream)
        s.synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    fa.fa_check()
    for o, lse in got:  # the same shares of the same work: the same bits
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


def test_no_rows():
    pool, table, tl = cache([9], 1, 64, 16, 5)
    q = torch.empty(0, 2, 64, dtype=torch.bfloat16, device=DEV)
    k = torch.empty(0, 1, 64, dtype=torch.bfloat16, device=DEV)
    o, lse = fa.fa_fwd_kv16(q, i32([0, 0]), pool, table, tl)
    assert o.shape == q.shape and lse.shape == (2, 0) and fa.fa_last_launch_count() == 0
    y = fa.fa_kv16_append(k, k, i32([0, 0]), pool, table, tl, rope=fa.rope_plan(64), q=q)
    assert y.shape == q.shape and fa.fa_last_launch_count() == 0
    back = fa.fa_kv16_keep(i32([]), i32([0]), i32([0, 0]), pool, table, tl)
    fa.fa_check()
    assert back.tolist() == [0]


# cu, slots, lens: a sequence that is not sound and has no token in front of the call's end
UNSOUND = [((0, 4, 9), None, None), ((0, 4, 2), None, None), ((0, 4, 4), [0, 2], None), ((0, 4, 4), [0, -1], None),
           ((0, 4, 4), None, [40, -1]), ((0, 4, 4), [0, 1], [40, 1 << 20])]


@pytest.mark.parametrize("call", ["append", "attention", "keep"])
@pytest.mark.parametrize("cu,ids,lens", UNSOUND)
def test_sequences_without_tokens_are_checked(cu, ids, lens, call):
    D = 64
    pool, table, tl = cache([40, 20], 1, D, 16, 1)
    q = torch.randn(4, 2, D, generator=torch.Generator().manual_seed(1)).bfloat16().to(DEV)
    k = q[:, :1].contiguous()
    tl, cu, ids = tl if lens is None else i32(lens), i32(cu), None if ids is None else i32(ids)
    if call == "append":
        latched(lambda: fa.fa_kv16_append(k, k, cu, pool, table, tl, seq_ids=ids, rope=fa.rope_plan(D), q=q))
    elif call == "attention":
        latched(lambda: fa.fa_fwd_kv16(q, cu, pool, table, tl, causal=True, seq_ids=ids))
    else:
        latched(lambda: fa.fa_kv16_keep(i32([0, 1, 0, 0]), i32([2, 0]), cu, pool, table, tl, seq_ids=ids))


@pytest.mark.parametrize("at", [0, 127, 128, 2999, 25000])
@pytest.mark.parametrize("named", [False, True])
def test_append_checks_every_sequence_of_a_large_batch(at, named):
    """One slot of a batch of empty ones has a length that is none; the rows of the others are written."""
    B, D, P = 25001, 64, 16
    pool, table, tl = cache([9] + [0] * (B - 1), 1, D, P, 2)
    lens = tl.clone()
    first = 1 if at == 0 else 0  # the sequence with the rows
    if at == 0:
        table, lens = table.roll(1, 0), lens.roll(1)
    lens[at] = -3
    cu = torch.full((B + 1,), 5, dtype=torch.int32, device=DEV)
    cu[:first + 1] = 0
    k, v = torch.randn(2, 5, 1, D, generator=torch.Generator().manual_seed(3)).bfloat16().to(DEV)
    ids = torch.arange(B, dtype=torch.int32, device=DEV) if named else None
    latched(lambda: fa.fa_kv16_append(k, v, cu, pool, table, lens, seq_ids=ids))
    got = pool[int(table[first, 0]), :, 0, 4:9]
    assert torch.equal(got[0], k[:, 0]) and torch.equal(got[1], v[:, 0])
    lens[at] = 0
    fa.fa_kv16_append(k, v, cu, pool, table, lens, seq_ids=ids)
    fa.fa_check()


@pytest.mark.parametrize("B", [32, 33, 64, 65, 1024, 1025, 4000])
@pytest.mark.parametrize("empty", ["some", "first", "middle", "last", "most"])
@pytest.mark.parametrize("named", [False, True])
def test_append_to_many_sequences(B, empty, named):
    """A token's sequence among many, with runs of empty ones: rows of k, v bit for bit, q turned at its index in the
    cache, all else untouched (rows behind the last sequence too)."""
    rng = np.random.default_rng(B + 7 * len(empty) + named)
    new = rng.integers(0, 4, B)
    third = B // 3
    if empty == "first":
        new[:2 * third] = 0
    elif empty == "middle":
        new[third:2 * third] = 0
    elif empty == "last":
        new[third:] = 0
    elif empty == "most":
        new[rng.random(B) < 0.95] = 0
    new[rng.integers(third)] = 40  # more rows than a block has tokens
    slots = rng.permutation(B) if named else np.arange(B)
    old = rng.integers(0, 30, B)
    lens = np.zeros(B, int)
    lens[slots] = old + new
    H, Hq, D, P, behind = 1, 2, 64, 16, 3
    pool, table, tl = cache(lens.tolist(), H, D, P, B)
    cu = prefix(new)
    T = int(cu[-1])
    x = torch.randn(T + behind, Hq + 2 * H, D, generator=torch.Generator().manual_seed(B)).bfloat16().to(DEV)
    q, k, v = x.split([Hq, H, H], 1)
    at = np.concatenate([np.arange(a, a + n) for a, n in zip(old, new)])
    slot = np.repeat(slots, new)
    page, row = torch.from_numpy(table.cpu().numpy()[slot, at // P]).long(), torch.from_numpy(at % P)
    want = pool.clone()
    y = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device=DEV)
    ids = i32(slots) if named else None
    fa.fa_kv16_append(k, v, i32(cu), pool, table, tl, seq_ids=ids)
    fa.fa_check()
    want[page, 0, :, row], want[page, 1, :, row] = k[:T], v[:T]
    assert torch.equal(pool.view(torch.int16), want.view(torch.int16))
    rope, w = fa.rope_plan(D), [10000.0 ** (-2 * c / D) for c in range(D // 2)]
    fa.fa_kv16_append(k, v, i32(cu), pool, table, tl, seq_ids=ids, rope=rope, q=q, q_out=y)
    fa.fa_check()
    assert (y[T:] == 7).all()
    for got, src in ((y[:T], q[:T]), (pool[page, 0, :, row], k[:T])):
        turned = kv16.turn(f64(src), at, w)
        assert (np.abs(f64(got) - turned) <= kv16.turn_tolerance(f64(src), turned, 1.0, D // 2, True)).all()
    want[page, 0, :, row] = pool[page, 0, :, row]
    assert torch.equal(pool.view(torch.int16), want.view(torch.int16))


def test_append_of_a_padded_batch_writes_the_rows():
    """Sequences of a batch padded with an empty slot, named out of order: each row at its place, bit for bit."""
    H, D, P, lens = 2, 64, 16, [50, 0, 70]
    pool, table, tl = cache(lens, H, D, P, 31)
    ids, new = [2, 1, 0, 1, 1], [4, 0, 2, 0, 0]
    k, v = torch.randn(2, 9, H, D, generator=torch.Generator().manual_seed(2)).bfloat16().to(DEV)
    want = pool.clone()
    tab = table.cpu()
    for s, first, n in ((2, 0, 4), (0, 4, 2)):
        p = torch.arange(lens[s] - n, lens[s])
        want[tab[s, p // P].long(), 0, :, p % P], want[tab[s, p // P].long(), 1, :, p % P] = k[first:first + n], v[first:first + n]
    fa.fa_kv16_append(k, v, i32(prefix(new)), pool, table, tl, seq_ids=i32(ids))
    fa.fa_check()
    assert torch.equal(pool.view(torch.int16), want.view(torch.int16))


def test_keep_refuses_counts_as_its_output():
    """512 columns and more take several blocks a sequence, which all read counts.  Beside it is well."""
    lens, n, layers = [60, 40], [5, 3], 9
    pool, table, tl = cache(lens, 4, 64, 16, 9, layers=layers)
    assert layers * 2 * 4 * 8 > 512
    ints = i32([1, 2, 0, 0])
    counts, beside = ints[:2], ints[2:]
    before = pool.clone()
    with pytest.raises(fa.FAError, match="invalid"):
        fa.fa_kv16_keep(i32([1, 0, 0, 0, 0, 0, 2, 0]), counts, i32(prefix(n)), pool, table, tl, new_tokens=counts)
    fa.fa_check()
    assert torch.equal(pool.view(torch.int16), before.view(torch.int16)) and ints.tolist() == [1, 2, 0, 0]
    back = fa.fa_kv16_keep(i32([1, 0, 0, 0, 0, 0, 2, 0]), counts, i32(prefix(n)), pool, table, tl, new_tokens=beside)
    fa.fa_check()
    assert back is beside and ints.tolist() == [1, 2, -4, -1]
    for s, moves in enumerate(([(0, 1)], [(1, 2)])):
        for to, of in moves:
            p, o = lens[s] - n[s] + to, lens[s] - n[s] + of
            before[:, int(table[s, p // 16]), :, :, p % 16] = before[:, int(table[s, o // 16]), :, :, o % 16].clone()
    assert torch.equal(pool.view(torch.int16), before.view(torch.int16))
