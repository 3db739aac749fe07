"""GPU tests of the paged 4-bit KV cache against its fp64 oracle (oracle/kv4.py).

Append and the page operations are compared byte for byte, read to the
rounded bf16 value.  Attention is held to a bound derived from its arithmetic
(``attention_bounds``), not to a measured error.
"""
import math

import numpy as np
import pytest
import torch

import exact_attention_07_gb300 as fa
import oracle
from oracle import kv4

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    fa.load_library()


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def bf16(x):
    return torch.tensor(np.asarray(x), dtype=torch.float32).bfloat16()


def f64(t):
    return t.detach().double().cpu().numpy()


def same_bytes(got, want, what):
    at = np.argwhere(got != want)
    assert not len(at), f"{what}: {len(at)} bytes differ: " + ", ".join(
        f"{tuple(map(int, a))} is {got[tuple(a)]:#x}, not {want[tuple(a)]:#x}" for a in at[:8])


def random_cache(rng, lens, H, D, P, spare=2, width=None, loud=1.0, layers=None):
    """A pool whose used positions hold quantised normal rows and whose other bytes are 0xff (NaN scales), pages in
    random order.  Returns (pool, table) as numpy."""
    need = [-(-n // P) for n in lens]
    N = max(1, sum(need) + spare)
    order = rng.permutation(N)
    width = width or max(1, max(need)) + 1
    table = np.full((len(lens), width), -7, np.int32)  # entries behind the last page are never looked at
    pool = np.full((N, H, P // 16, 18 * D), 255, np.uint8)
    at = 0
    for s, n in enumerate(lens):
        table[s, :need[s]] = order[at:at + need[s]]
        at += need[s]
        if n == 0:
            continue
        k, v = rng.standard_normal((2, n, H, D))
        k[..., :3] *= loud
        (kc, ks), (vc, vs) = kv4.quantise(k, np.ones(H)), kv4.quantise(v, np.ones(H))
        pos = np.arange(n)
        page, u, key = table[s][pos // P], pos % P // 16, pos % 16
        d, g = np.arange(D), np.arange(D // 16)
        for h in range(H):
            pool[page[:, None], h, u[:, None], key[:, None] * (D // 2) + d[:D // 2]] = kc[:, h, 0::2] | kc[:, h, 1::2] << 4
            pool[page[:, None], h, u[:, None], 16 * D + key[:, None] * (D // 16) + g] = ks[:, h]
            pool[page[:, None], h, u[:, None], 17 * D + g * 16 + key[:, None]] = vs[:, h]
            a = 8 * D + key[:, None] // 8 * 4 * D + d // 16 * 64 + key[:, None] % 8 // 2 * 16 + d % 16
            for odd in (0, 1):
                r = np.nonzero(key % 2 == odd)[0][:, None]
                at_ = (page[r], h, u[r], a[r[:, 0]])
                pool[at_] = (pool[at_] & 15 | vc[r[:, 0], h] << 4) if odd else (pool[at_] & 240 | vc[r[:, 0], h])
    return pool, table


def attention_bounds(q, k, v, scale, lse):
    """Bounds on |O - O_ref| and |LSE - LSE_ref| of one KV head's rows from the kernel's arithmetic.

    Codes times scales are exact; q is exact up to 2^-25 of its row's maximum.  A score sums D products in fp32 in
    some order: its error is below D 2^-23 sum|q||k| scale even if each addition truncates, and the exponent's
    argument, at most 2^7 in magnitude in log2 units above the underflow, loses 2^-23 * 2^7 more where scores are that
    far apart.  2^x is good to 2^-21, a sum of L terms in fp32 to L 2^-24 at worst (pairwise or chunked in practice;
    the worst is used), P as two fp16 numbers to 2^-21."""
    qk = (np.abs(q).reshape(-1, q.shape[-1]) @ np.abs(k).reshape(-1, k.shape[-1]).T).max() * scale
    spread = min(2.0 ** 7, 4 * np.abs(qk) + 1)
    ds = q.shape[-1] * 2.0 ** -23 * qk + spread * 2.0 ** -23
    rel = 2 * ds + k.shape[-2] * 2.0 ** -23 + 2.0 ** -19
    fin = np.isfinite(lse)
    return 2 * rel * np.abs(v).max(), rel + 2.0 ** -22 * (np.abs(lse[fin]).max() if fin.any() else 0)


def check_attention(q, o, lse, pool, table, slots, lens, ks, vs, scale, causal, what):
    """Every sequence of a batch against the oracle."""
    B, Hq, Lq, D = q.shape
    for b, s in enumerate(slots):
        k, v = kv4.rows(pool, table, s, lens[s], ks, vs)
        ro, rl = kv4.attention(f64(q[b]), k, v, scale, causal)
        go, gl = f64(o[b]), f64(lse[b])
        assert np.array_equal(np.isneginf(rl), np.isneginf(gl)), f"{what}: empty rows of sequence {b}"
        assert not go[np.isneginf(rl)].any(), f"{what}: O of empty rows"
        if lens[s] == 0:
            continue
        to, tl = attention_bounds(f64(q[b]), k, v, scale, rl)
        fin = np.isfinite(rl)
        assert np.abs(go - ro).max() <= to, f"{what}: O of sequence {b}: {np.abs(go - ro).max()} > {to}"
        if fin.any():
            assert np.abs(gl[fin] - rl[fin]).max() <= tl, f"{what}: LSE of sequence {b}"


def run_attention(q, *args, **kw):
    """fa_fwd_kv4 with guard bands around O and LSE."""
    n, m, G = q.numel(), q.numel() // q.shape[-1], 1024
    ob = torch.full((n + 2 * G,), 777.0, device=DEV)
    lb = torch.full((m + 2 * G,), 777.0, device=DEV)
    o, lse = ob[G:G + n].view(q.shape), lb[G:G + m].view(q.shape[:3])
    fa.fa_fwd_kv4(q, *args, out=o, lse=lse, **kw)
    fa.fa_check()
    for x in (ob, lb):
        assert (x[:G] == 777).all() and (x[-G:] == 777).all(), "guard band written"
    return o, lse


ATTN = [
    # Hq, Hkv, Lq, D, page_size, lengths, causal, head scales, multiplier of q
    (32, 8, 1, 128, 64, [1, 2, 15, 16, 17, 63, 64, 65, 700], True, False, 1.0),
    (8, 8, 1, 128, 16, [0, 1, 33, 500], False, True, 1.0),          # one row per KV head, an empty sequence
    (4, 1, 1, 64, 32, [31, 32, 129, 1000], True, True, 1.0),
    (8, 2, 4, 64, 16, [1, 3, 4, 5, 400, 777], True, False, 1.0),    # 16 rows; rows before the first key
    (5, 1, 1, 128, 128, [127, 128, 300], False, False, 1.0),        # 5 rows
    (6, 2, 2, 128, 256, [255, 257, 1000], True, True, 3.0),         # 6 rows, pages of 256
    (8, 1, 1, 128, 64, [640], False, False, 20.0),                  # 8 rows, very sharp softmax
    (9, 1, 1, 64, 64, [333, 5], True, False, 1.0),                  # 9 rows
    (24, 2, 5, 128, 64, [4, 5, 6, 900], True, True, 1.0),           # 60 rows
    (64, 1, 1, 64, 16, [1, 1234], True, False, 1.0),                # 64 rows
    (16, 1, 2, 128, 32, [50, 2000], False, False, 1.0),             # 32 rows, no mask
    (2, 1, 16, 64, 64, [8, 100], True, False, 1.0),                 # Lq above the length: empty rows
    (32, 8, 1, 128, 64, [4000] * 3 + [1] * 40, True, False, 1.0),   # many short sequences beside long ones
]


@pytest.mark.parametrize("Hq,Hkv,Lq,D,P,lens,causal,scaled,qm", ATTN)
def test_attention_matches_the_oracle(Hq, Hkv, Lq, D, P, lens, causal, scaled, qm):
    rng = np.random.default_rng(len(lens) + Hq + Lq + D + P)
    pool, table = random_cache(rng, lens, Hkv, D, P, loud=4.0)
    ks, vs = (rng.random((2, Hkv)) + 0.5 if scaled else np.ones((2, Hkv))).astype(np.float32)
    q = bf16(rng.standard_normal((len(lens), Hq, Lq, D)) * qm).to(DEV)
    heads = dict(k_scale=torch.tensor(ks, device=DEV), v_scale=torch.tensor(vs, device=DEV)) if scaled else {}
    dev = (torch.tensor(pool, device=DEV), i32(table), i32(lens))
    o, lse = run_attention(q, *dev, causal=causal, **heads)
    check_attention(q, o, lse, pool, table, range(len(lens)), lens, ks.astype(float), vs.astype(float),
                    1 / math.sqrt(D), causal, "attention")
    o2, lse2 = run_attention(q, *dev, causal=causal, **heads)
    assert torch.equal(o, o2) and torch.equal(lse, lse2), "two runs differ"


def test_attention_over_slots_named_in_any_order_and_twice():
    rng = np.random.default_rng(3)
    lens = [70, 0, 300, 16, 5]
    pool, table = random_cache(rng, lens, 2, 64, 16)
    slots = [4, 2, 2, 0, 1, 3, 4]
    q = bf16(rng.standard_normal((len(slots), 4, 2, 64))).to(DEV)
    o, lse = run_attention(q, torch.tensor(pool, device=DEV), i32(table), i32(lens), causal=True, softmax_scale=0.2,
                           seq_ids=i32(slots))
    check_attention(q, o, lse, pool, table, slots, lens, np.ones(2), np.ones(2), 0.2, True, "slots")


def test_nan_in_keys_that_a_row_may_not_see_does_not_reach_it():
    """NaN scales in the last three positions: rows that may not see them are as without them, the others are NaN
    where the definition says so."""
    rng = np.random.default_rng(4)
    Hq, D, P, L, Lq = 4, 128, 64, 200, 4
    pool, table = random_cache(rng, [L], 2, D, P)
    for which in ("v", "k"):
        bad = pool.copy()
        for pos in (197, 198, 199):
            unit = bad[table[0, pos // P], :, pos % P // 16]
            if which == "v":
                unit[:, 17 * D + 3 * 16 + pos % 16] = 0x7f  # dimensions 48 .. 63
            else:
                unit[:, 16 * D + pos % 16 * (D // 16) + 2] = 0xff
        q = bf16(rng.standard_normal((1, Hq, Lq, D))).to(DEV)
        o, lse = run_attention(q, torch.tensor(bad, device=DEV), i32(table), i32([L]), causal=True)
        k, v = kv4.rows(bad, table, 0, L, np.ones(2), np.ones(2))
        ro, rl = kv4.attention(f64(q[0]), k, v, 1 / math.sqrt(D), True)
        go, gl = f64(o[0]), f64(lse[0])
        assert np.array_equal(np.isnan(ro), np.isnan(go)) and np.array_equal(np.isnan(rl), np.isnan(gl)), which
        fin = ~np.isnan(ro)
        assert fin[:, 0].all()  # the first query sees none of the three
        assert np.abs(go[fin] - ro[fin]).max() < 1e-4  # well above attention_bounds at 200 keys (2e-5)


def test_infinite_and_nan_queries_stay_in_their_rows():
    rng = np.random.default_rng(5)
    pool, table = random_cache(rng, [150], 1, 64, 32)
    x = rng.standard_normal((1, 6, 1, 64))
    x[0, 1, 0, 5], x[0, 4, 0, 0] = np.nan, np.inf
    q = bf16(x).to(DEV)
    o, lse = run_attention(q, torch.tensor(pool, device=DEV), i32(table), i32([150]))
    clean = bf16(np.where(np.isfinite(x), x, 0)).to(DEV)
    o2, lse2 = run_attention(clean, torch.tensor(pool, device=DEV), i32(table), i32([150]))
    for h in range(6):
        if h in (1, 4):
            assert torch.isnan(o[0, h]).all() and torch.isnan(lse[0, h]).all()
        else:
            assert torch.equal(o[0, h], o2[0, h]) and torch.equal(lse[0, h], lse2[0, h])


def test_queries_of_every_magnitude():
    """The kernel holds q as fp16 with a power of two per row: rows far apart in size, and large and small numbers in
    one row, keep their meaning."""
    rng = np.random.default_rng(6)
    pool, table = random_cache(rng, [300], 1, 64, 64)
    x = rng.standard_normal((1, 8, 1, 64))
    scale = np.float32(0.125)
    for h, m in enumerate([1e-30, 1e-8, 1e-3, 1, 8, 0, 1e-3, 1]):
        x[0, h] *= m
    x[0, 6, 0, :4] *= 1e4
    x[0, 7, 0, 10:] *= 1e-5
    q = bf16(x).to(DEV)
    o, lse = run_attention(q, torch.tensor(pool, device=DEV), i32(table), i32([300]), softmax_scale=float(scale))
    check_attention(q, o, lse, pool, table, [0], [300], np.ones(1), np.ones(1), float(scale), False, "magnitudes")


@pytest.mark.parametrize("Hq,Lq,D", [(4, 1, 128), (8, 1, 64), (16, 1, 128), (8, 2, 64), (40, 1, 128), (16, 2, 64)])
def test_small_elements_of_a_query_beside_large_ones(Hq, Lq, D):
    """Rows whose first elements, which meet keys of 0 there, are 2^16 or 2^24 times the others: the scores are those of
    the others.  Where the row's largest magnitude is below 2^27, elements from 2^-6 on are exact and those below, one
    or two of 112, are off by 2^-14 at most: against keys of normal numbers 2^-14 sqrt(1.4 / 3) / sqrt(128) < 2^-17 of
    a weight in the mean.  fp32 adds 2^-18 (as in the test of the mean error)."""
    rng = np.random.default_rng(60 + Hq + Lq + D)
    H, P, lens = 4 if Hq == 4 else 2, 64, [300, 41, 777]
    pool, table = random_cache(rng, lens, H, D, P)
    pool[..., :8 * D].reshape(*pool.shape[:3], 16, D // 2)[..., :8] = 0  # K codes of the dimensions 0 .. 15
    x = rng.standard_normal((len(lens), Hq, Lq, D))
    x[..., :16] *= 2.0 ** 16
    x[:, ::2, :, :16] *= 2.0 ** 8
    q = bf16(x).to(DEV)
    o, lse = run_attention(q, torch.tensor(pool, device=DEV), i32(table), i32(lens), causal=True)
    for b, n in enumerate(lens):
        ro, rl = kv4.attention(f64(q[b]), *kv4.rows(pool, table, b, n, np.ones(H), np.ones(H)), 1 / math.sqrt(D), True)
        err = math.sqrt(np.square(f64(o[b]) - ro).mean() / np.square(ro).mean())
        assert err < 2.0 ** -17 + 2.0 ** -18, (b, err)
        assert np.abs(f64(lse[b]) - rl).max() < 2.0 ** -15


@pytest.mark.parametrize("scale,head,mult", [(2.0 ** -30, 2.0 ** -64, 2.0 ** -100), (2.0 ** 60, 2.0 ** 64, 2.0 ** 100)])
def test_factors_beyond_the_range_of_fp32_leave_masked_keys_out(scale, head, mult):
    """softmax_scale, a head scale and a row's power of two whose product underflows (all scores are 0) or overflows
    (against keys that are 0, so that all scores are 0 again): each row's mean of the values that it sees."""
    rng = np.random.default_rng(21)
    Hq, Lq, D, P, L = 2, 3, 64, 32, 75
    pool, table = random_cache(rng, [L], 1, D, P)
    if mult > 1:
        used = table[0, :-(-L // P)]
        pool[used, :, :, :8 * D] = 0
        pool[used, :, :, 16 * D:17 * D] = 0
    q = bf16(rng.standard_normal((1, Hq, Lq, D)) * mult).to(DEV)
    o, lse = run_attention(q, torch.tensor(pool, device=DEV), i32(table), i32([L]), causal=True, softmax_scale=scale,
                           k_scale=torch.tensor([head], dtype=torch.float32, device=DEV))
    check_attention(q, o, lse, pool, table, [0], [L], np.array([head]), np.ones(1), scale, True, "factors")


@pytest.mark.parametrize("Hq,Lq,D", [(16, 1, 128), (28, 1, 128), (16, 3, 128), (8, 1, 64), (16, 2, 64), (80, 1, 64)])
@pytest.mark.parametrize("B", [1024, 3])
def test_keys_far_below_a_heavy_one_keep_their_weight(Hq, Lq, D, B):
    """The first key weighs e^2 to e^20 times as much as each other one and its value is 0, so O is what the others
    carry.  All keys of a row but the first have one score, so a rounding of P does not average out.  With 1024
    sequences a warp takes a whole one, with 3 they are cut.

    P is good to 2^-22, or to 2^-41 of the heaviest key.  Scores are single products here: the factor of the scores has
    three roundings and the exponent's argument, up to 20 / ln 2 + 5, one, together 35 * 2^-22 * ln 2 = 5.8e-6 of a
    weight; 2^x and the division are good to 2^-22 each; all values have one sign, so 25 tiles, two steps of a product
    and 8 warps lose at most 25 * 2^-24 + 2 * 2^-23 + 8 * 2^-24 = 2.2e-6 of their sum.  Together below 2^-16."""
    rng = np.random.default_rng(40 + Hq + Lq + D)
    H, P, L = 4, 64, 777
    need = -(-L // P)
    pool, row = np.zeros((need, H, P // 16, 18 * D), np.uint8), list(range(need))
    k, v = rng.standard_normal((2, L, H, D))
    k[..., :16], v = 0, np.abs(v)
    k[0, :, 0], v[0] = 6, 0
    one = np.ones(H)
    kv4.append(pool, [row], [L], [0], [L], k, v, one, one)
    lens = [int(x) for x in rng.integers(2, L + 1, B)] if B > 3 else [2, 600, L]
    scale = 1 / math.sqrt(D)
    x = np.zeros((B, Hq, Lq, D))
    x[..., 0] = rng.uniform(2, 20, (B, Hq, Lq)) / (6 * scale)
    q = bf16(x).to(DEV)
    gap = f64(q)[..., 0] * 6 * scale
    o, lse = run_attention(q, torch.tensor(pool, device=DEV), i32([row] * B), i32(lens))
    go, gl = f64(o), f64(lse)
    for b in range(0, B, 37) if B > 3 else range(B):
        ro, rl = kv4.attention(f64(q[b]), *kv4.rows(pool, [row], 0, lens[b], one, one), scale, False)
        bound = 2.0 ** -16 + 2.0 ** -41 * np.exp(gap[b])
        assert (np.abs(go[b] - ro) <= ro * bound[..., None]).all(), (b, lens[b], np.abs(go[b] - ro).max())
        assert (np.abs(gl[b] - rl) <= 2.0 ** -16 + 2.0 ** -22 * np.abs(rl)).all()


@pytest.mark.parametrize("Hq,Lq,D", [(16, 1, 128), (28, 1, 128), (16, 3, 128), (8, 1, 64), (16, 2, 64), (80, 1, 64)])
@pytest.mark.parametrize("B,L", [(3, 4000), (40, 300)])
def test_attention_is_as_good_as_fp32(Hq, Lq, D, B, L):
    """The error's root mean square, against O's.  A score of normal rows is a sum of D products, in D / 16 steps that
    each lose up to 2^-23 of a partial sum of magnitude 4 at most: below D / 16 * 2^-21 = 3.8e-6 of a weight if all
    went one way.  They do not, and the errors of P (2^-22), 2^x (2^-22) and of the sums stay below what that leaves:
    2^-18.  P as a single fp16 number is at 1.9e-4."""
    rng = np.random.default_rng(50 + Hq + Lq + D)
    H, lens = 4, [L - b for b in range(B)]
    pool, table = random_cache(rng, lens, H, D, 64)
    q = bf16(rng.standard_normal((B, Hq, Lq, D))).to(DEV)
    o, lse = run_attention(q, torch.tensor(pool, device=DEV), i32(table), i32(lens), causal=True)
    go, gl = f64(o), f64(lse)
    for b in range(0, B, 13):
        ro, rl = kv4.attention(f64(q[b]), *kv4.rows(pool, table, b, lens[b], np.ones(H), np.ones(H)), 1 / math.sqrt(D), True)
        err = math.sqrt(np.square(go[b] - ro).mean() / np.square(ro).mean())
        assert err < 2.0 ** -18, (b, err)
        assert np.abs(gl[b] - rl).max() < 2.0 ** -17


def test_long_cache_with_offsets_beyond_32_bits():
    H, D, P = 2, 128, 256
    page_bytes = H * P // 16 * 18 * D
    N = 6 * (1 << 30) // page_bytes
    pool = torch.zeros(N, H, P // 16, 18 * D, dtype=torch.uint8, device=DEV)
    rng = np.random.default_rng(7)
    small, table = random_cache(rng, [1000], H, D, P, spare=0)
    high = N - 1 - np.arange(small.shape[0])
    pool[torch.tensor(high, device=DEV)] = torch.tensor(small, device=DEV)
    where = table.copy()
    where[0, :4] = high[table[0, :4]]
    q = bf16(rng.standard_normal((1, 8, 1, D))).to(DEV)
    o, lse = run_attention(q, pool, i32(where), i32([1000]))
    check_attention(q, o, lse, small, table, [0], [1000], np.ones(H), np.ones(H), 1 / math.sqrt(D), False, "high pages")
    k, v = fa.fa_kv4_read(i32([0, 1000]), 1000, pool, i32(where), i32([1000]))
    rk, _ = kv4.rows(small, table, 0, 1000, np.ones(H), np.ones(H))
    assert np.array_equal(f64(k).transpose(1, 0, 2), rk)
    new = bf16(rng.standard_normal((2, 7, H, D))).to(DEV)
    fa.fa_kv4_append(new[0], new[1], i32([0, 7]), pool, i32(where), i32([1000]))
    kv4.append(small, table, [1000], [0], [7], f64(new[0]), f64(new[1]), np.ones(H), np.ones(H))
    assert torch.equal(pool[torch.tensor(high, device=DEV)], torch.tensor(small, device=DEV))
    # a move between pages 4 GB apart
    refs = torch.zeros(N, dtype=torch.int32, device=DEV)
    refs[torch.tensor(high, device=DEV)] = 1
    t, n = i32(where), i32([1000])
    info = fa.fa_kv4_compact(pool, t, n, refs)
    fa.fa_check()
    assert info.tolist() == [N - 4, 0] and sorted(t[0, :4].tolist()) == [0, 1, 2, 3] and refs[:4].tolist() == [1] * 4
    o2, lse2 = run_attention(q, pool, t, n)
    check_attention(q, o2, lse2, small, table, [0], [1000], np.ones(H), np.ones(H), 1 / math.sqrt(D), False, "moved")


# ------------------------------------------------------------------ append and read

ROWS = [
    # H, D, page_size, lengths before, new tokens, head scales
    (8, 128, 64, [0, 1, 62, 63, 64, 100], [1] * 6, False),            # a decode step, odd and even positions
    (2, 64, 16, [0, 3, 15, 40], [40, 13, 2, 0], True),                # pages that end inside, none at all
    (3, 128, 32, [7], [200], True),
    (1, 64, 256, [255, 0], [3, 300], False),
    (4, 128, 128, [5] * 9, [2, 1, 3, 0, 0, 1, 2, 5, 130], False),
]


@pytest.mark.parametrize("H,D,P,old,new,scaled", ROWS)
@pytest.mark.parametrize("named", [False, True])
def test_append_and_read_match_the_oracle(H, D, P, old, new, scaled, named):
    rng = np.random.default_rng(D + P + len(old))
    n = len(old)
    slots = list(rng.permutation(n + 2)[:n]) if named else list(range(n))
    lens = np.full(n + 2, 9)
    lens[slots] = [a + b for a, b in zip(old, new)]
    pool, table = random_cache(rng, list(lens), H, D, P)
    T = sum(new)
    x = rng.standard_normal((2, T + 3, H, D)) * np.exp(rng.standard_normal((2, T + 3, H, 1)) * 3)
    x[:, ::3, :, 16:32] = np.round(x[:, ::3, :, 16:32] * 4) / 4     # values on the borders between codes
    x[0, 0, 0, 20], x[1, T - 1, H - 1, 40] = np.nan, -np.inf
    x[0, T // 2, 0, :16] = 0.0
    x[1, T // 3, 0, :16] *= 1e-12                                    # below the smallest scale
    x[0, T // 3, 0, 32:48] *= 1e12                                   # above the largest
    k, v = bf16(x[0]).to(DEV), bf16(x[1]).to(DEV)
    ks, vs = (rng.random((2, H)) + 0.5 if scaled else np.ones((2, H))).astype(np.float32)
    if scaled:
        ks[0], vs[0] = 2.0 ** -3, 2.0 ** 5  # powers of two: borders stay borders
    heads = dict(k_scale=torch.tensor(ks, device=DEV), v_scale=torch.tensor(vs, device=DEV)) if scaled else {}
    cu = np.concatenate([[0], np.cumsum(new)])
    ids = dict(seq_ids=i32(slots)) if named else {}
    dev = (torch.tensor(pool, device=DEV), i32(table), i32(lens))
    fa.fa_kv4_append(k, v, i32(cu), *dev, **ids, **heads)  # three rows behind the last sequence are not the call's
    assert fa.fa_last_launch_count() == 1
    fa.fa_check()
    kv4.append(pool, table, list(lens), slots, new, f64(k[:T]), f64(v[:T]), ks.astype(float), vs.astype(float))
    got = dev[0].cpu().numpy()
    if scaled:
        # a quotient by a scale that is no power of two is rounded once more before its border is looked at: a code
        # next to it in at most 1 of 10000 bytes (a border within 2^-22 of a value is hit with a chance of about 2^-20)
        assert (got != pool).mean() < 1e-4
    else:
        same_bytes(got, pool, "append")
    dev[0].copy_(torch.tensor(pool))
    out = [torch.full((T + 2, H, D), 3.0, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    fa.fa_kv4_read(i32(cu), T + 2, *dev, **ids, **heads, k_out=out[0], v_out=out[1])
    fa.fa_check()
    assert (out[0][T:] == 3).all() and (out[1][T:] == 3).all(), "rows behind the last sequence"
    row = 0
    for s, c in zip(slots, new):
        for g, r in zip(out, kv4.rows(pool, table, s, lens[s], ks.astype(float), vs.astype(float))):
            want = r[:, lens[s] - c:].transpose(1, 0, 2)
            have = f64(g[row:row + c])
            assert np.array_equal(np.isnan(want), np.isnan(have))
            fin = ~np.isnan(want)
            # one rounding to bf16, and one to fp32 where the head scale is no power of two
            assert (np.abs(have[fin] - want[fin]) <= np.abs(want[fin]) * (2.0 ** -8 + 2.0 ** -23)).all()
            if not scaled:
                assert np.array_equal(have[fin], want[fin])
        row += c


@pytest.mark.parametrize("D,P", [(64, 16), (128, 64)])
def test_append_under_head_scales_rounds_to_the_nearest(D, P):
    """Head 0 has a power of two for its scale: its bytes are the oracle's, as are all that the call does not own.
    Elsewhere 6 g and s g (g the head's scale, s the group's) are rounded to fp32 before a quotient by them, which is
    rounded itself: two relative errors of 2^-24 each.  A scale or code may so be the other neighbour where the
    quotient lies within 2^-22 of the border between two, and nowhere else."""
    rng = np.random.default_rng(70 + D)
    H, old, new, slots = 5, [3, 0, 40, 17], [60, 33, 1, 14], [3, 0, 4, 1]
    heads = {"k": np.array([0.25, 1.1, 0.7001, 3e-5, 7.3e6], np.float32), "v": np.array([8, 0.9, 1.37, 1.3e4, 2e-7], np.float32)}
    lens = [16] * 5
    for i, s in enumerate(slots):
        lens[s] = old[i] + new[i]
    pool, table = random_cache(rng, lens, H, D, P)
    T = sum(new)
    x = {n: f64(bf16(rng.standard_normal((T, H, D)) * np.exp(rng.standard_normal((T, H, 1)) * 2) * heads[n][:, None]))
         for n in "kv"}
    dev = (torch.tensor(pool, device=DEV), i32(table), i32(lens))
    fa.fa_kv4_append(bf16(x["k"]).to(DEV), bf16(x["v"]).to(DEV), i32(np.concatenate([[0], np.cumsum(new)])), *dev,
                     seq_ids=i32(slots), k_scale=torch.tensor(heads["k"], device=DEV),
                     v_scale=torch.tensor(heads["v"], device=DEV))
    fa.fa_check()
    want, got = pool.copy(), dev[0].cpu().numpy()
    g = {n: heads[n].astype(float) for n in "kv"}
    kv4.append(want, table, lens, slots, new, x["k"], x["v"], g["k"], g["v"])
    kc, ks = kv4.quantise(x["k"], g["k"])
    vc, vs = kv4.quantise(x["v"], g["v"])
    d, grp = np.arange(D), np.arange(D // 16)
    row = 0
    for i, s in enumerate(slots):
        for pos in range(old[i], lens[s]):
            for h in range(1, H):
                unit, key = got[table[s][pos // P], h, pos % P // 16], pos % 16
                k = unit[key * (D // 2):(key + 1) * (D // 2)]
                v = unit[8 * D + key // 8 * 4 * D + d // 16 * 64 + key % 8 // 2 * 16 + d % 16]
                have = {"k": (np.stack([k & 15, k >> 4], 1).reshape(D), unit[16 * D + key * (D // 16) + grp]),
                        "v": (v >> 4 if key % 2 else v & 15, unit[17 * D + grp * 16 + key])}
                for n, (codes, scales) in have.items():
                    y = np.abs(x[n][row, h]).reshape(D // 16, 16) / g[n][h]
                    top = y.max(1) / 6
                    off = np.abs(top[:, None] - kv4.E4M3)
                    assert (off[grp, scales] <= off.min(1) + 2.0 ** -22 * top).all(), (n, pos, h)
                    e = kv4.E4M3[scales][:, None]
                    z = np.where(e > 0, y / np.where(e > 0, e, 1), 0).reshape(D)  # a scale of 0: codes of 0
                    off = np.abs(z[:, None] - kv4.E2M1)
                    assert (off[d, codes & 7] <= off.min(1) + 2.0 ** -22 * z).all(), (n, pos, h)
                    assert ((codes >> 3) == ((x[n][row, h] < 0) & (e > 0).repeat(16))).all(), (n, pos, h)
                kv4.write_row(unit, key, D, kc[row, h], ks[row, h], vc[row, h], vs[row, h])
            row += 1
    same_bytes(got, want, "append")


def test_rows_at_addresses_that_are_not_32_byte_aligned():
    rng = np.random.default_rng(13)
    H, D, P = 2, 64, 16
    pool, table = random_cache(rng, [40], H, D, P)
    dev = (torch.tensor(pool, device=DEV), i32(table), i32([40]))
    kv = [torch.zeros(8 + 20 * H * D, dtype=torch.bfloat16, device=DEV)[8:].view(20, H, D) for _ in range(4)]
    for t in kv[:2]:
        t.copy_(bf16(rng.standard_normal(t.shape)))
    assert kv[0].data_ptr() % 32 == 16
    fa.fa_kv4_append(kv[0], kv[1], i32([0, 20]), *dev)
    kv4.append(pool, table, [40], [0], [20], f64(kv[0]), f64(kv[1]), np.ones(H), np.ones(H))
    same_bytes(dev[0].cpu().numpy(), pool, "append")
    fa.fa_kv4_read(i32([0, 20]), 20, *dev, k_out=kv[2], v_out=kv[3])
    for got, want in zip(kv[2:], kv4.rows(pool, table, 0, 40, np.ones(H), np.ones(H))):
        assert np.array_equal(f64(got), want[:, 20:].transpose(1, 0, 2))
    fa.fa_check()


@pytest.mark.parametrize("D", [64, 128])
def test_append_of_rows_of_every_magnitude(D):
    """Groups from the smallest to the largest bf16 numbers under the smallest and largest head scales: what is above
    6 * 448 of them takes the largest scale and codes.  Scales are powers of two, so every byte is the oracle's."""
    rng = np.random.default_rng(20 + D)
    H, P, T = 4, 32, 90
    heads = np.array([2.0 ** -64, 2.0 ** -3, 1.0, 2.0 ** 64], np.float32)
    pool, table = random_cache(rng, [T + 5], H, D, P)
    x = rng.standard_normal((2, T, H, D // 16, 16)) * 10.0 ** rng.uniform(-38, 37.9, (2, T, H, D // 16, 1))
    x[:, :6] = np.sign(x[:, :6]) * 10.0 ** rng.uniform(36, 38.5, (2, 6, H, D // 16, 16))
    k, v = (bf16(t.reshape(T, H, D)).to(DEV) for t in x)
    assert k.isfinite().all() and v.isfinite().all()
    scales = torch.tensor(heads, device=DEV)
    dev = (torch.tensor(pool, device=DEV), i32(table), i32([T + 5]))
    fa.fa_kv4_append(k, v, i32([0, T]), *dev, k_scale=scales, v_scale=scales)
    fa.fa_check()
    kv4.append(pool, table, [T + 5], [0], [T], f64(k), f64(v), heads.astype(float), heads.astype(float))
    same_bytes(dev[0].cpu().numpy(), pool, "append")


def test_no_rows_at_all():
    pool, table, lens = fa.kv4_pool(2, 1, 16, 64), i32([[0], [1]]), i32([3, 0])
    none = torch.zeros(0, 1, 64, dtype=torch.bfloat16, device=DEV)
    fa.fa_kv4_append(none, none, i32([0, 0, 0]), pool, table, lens)
    assert fa.fa_last_launch_count() == 0 and not pool.any()
    k, v = fa.fa_kv4_read(i32([0, 0, 0]), 0, pool, table, lens)
    assert k.shape == (0, 1, 64) and v.shape == (0, 1, 64)


# ------------------------------------------------------------------ pages

def _page_state(m, pool):
    return torch.tensor(pool, device=DEV), i32(m.table), i32(m.lens), i32(m.refs)


def _same_state(m, pool, dev, what):
    assert dev[1].tolist() == m.table, f"{what}: table"
    assert dev[2].tolist() == m.lens, f"{what}: lengths"
    assert dev[3].tolist() == m.refs, f"{what}: references"
    same_bytes(dev[0].cpu().numpy(), pool, what)


@pytest.mark.parametrize("N,slots,width,P,H,D,layers,seed", [
    (24, 6, 5, 16, 2, 64, 1, 0), (400, 9, 40, 16, 1, 64, 3, 1), (131, 40, 6, 64, 2, 128, 2, 2),
    (5000, 300, 40, 32, 1, 64, 1, 3), (7, 3, 2, 256, 1, 64, 2, 4)])
def test_page_operations_follow_the_sequential_model(N, slots, width, P, H, D, layers, seed):
    rng = np.random.default_rng(seed)
    m = kv4.Pages(N, slots, width, P)
    pool = rng.integers(0, 256, (layers, N, H, P // 16, 18 * D), dtype=np.uint8)
    dev = _page_state(m, pool)
    done = {}
    for step in range(40):
        empty = [s for s in range(slots) if m.lens[s] == 0]
        held = [s for s in range(slots) if m.lens[s]]
        op = rng.choice(["reserve", "reserve", "fork", "release", "compact"])
        if op == "reserve":
            ids = [int(s) for s in rng.permutation(slots)[:rng.integers(1, slots + 1)]]
            new = [int(min(P * width - m.lens[s], rng.integers(0, 2 * P))) for s in ids]
            want = m.reserve(ids, new)
            got = fa.fa_kv4_reserve(i32(new), *dev[1:], P, seq_ids=i32(ids))
        elif op == "fork" and empty and held:
            kids = [int(s) for s in rng.permutation(empty)[:rng.integers(1, len(empty) + 1)]]
            parents = [int(rng.choice(held)) for _ in kids]
            want = m.fork(parents, kids, pool)
            got = fa.fa_kv4_fork(i32(parents), i32(kids), *dev)
        elif op == "release" and held:
            ids = [int(s) for s in rng.choice(slots, rng.integers(1, max(2, slots // 2)))]  # some twice, some empty
            m.release(ids)
            fa.fa_kv4_release(i32(ids), *dev[1:], P)
            want = got = None
        else:
            op = "compact"
            want = m.compact(pool)
            got = fa.fa_kv4_compact(*dev)
        fa.fa_check()
        if want is not None:
            assert tuple(got.tolist()) == want, (step, op)
        done[op, want and want[1] > 0] = 1
        _same_state(m, pool, dev, f"step {step}, {op}")
    assert {k[0] for k in done} == {"reserve", "fork", "release", "compact"}


def test_positions_taken_back():
    """Drafted tokens are rejected: pages behind the new end are dropped, a page that others use is left alone."""
    rng = np.random.default_rng(18)
    P = 16
    m = kv4.Pages(40, 6, 6, P)
    pool = rng.integers(0, 256, (1, 40, 1, 1, 18 * 64), dtype=np.uint8)
    dev = _page_state(m, pool)

    def both(ids, new):
        want = m.reserve(ids, new)
        assert tuple(fa.fa_kv4_reserve(i32(new), *dev[1:], P, seq_ids=i32(ids)).tolist()) == want
        if want[1] < 0:
            with pytest.raises(fa.FAError, match="invalid argument"):
                fa.fa_check()
        fa.fa_check()
        _same_state(m, pool, dev, (ids, new))
        return want[1]

    assert both([0, 1], [50, 32]) == 0
    fa.fa_kv4_fork(i32([0, 1]), i32([2, 3]), *dev)
    m.fork([0, 1], [2, 3], pool)
    assert both([0, 2, 4], [-1, 30, 5]) == 0        # within its own last page, growth beside it
    assert both([0], [-2]) == -1                    # 47: a page shared with slot 2
    assert both([0, 2], [-1, -32]) == 0             # 48 and 48: on the edge of shared pages
    assert both([0, 2], [-16, -16]) == 0            # whole shared pages: a reference less each
    assert both([3, 3, 0, 5], [-32, 0, 7, 0]) == 0  # nothing left of slot 3
    assert both([1, 1], [-1, -1]) == -1             # a slot twice
    assert both([1], [-1]) == 0                     # its page is its own again
    for _ in range(60):
        ids = [int(x) for x in rng.permutation(6)[:rng.integers(1, 7)]]
        both(ids, [int(max(-m.lens[s], min(96 - m.lens[s], rng.integers(-40, 41)))) for s in ids])


def test_reserve_and_release_of_more_sequences_than_fit_in_shared_memory():
    rng = np.random.default_rng(17)
    S, P = 5000, 16
    m = kv4.Pages(9000, S, 3, P)
    dev = _page_state(m, np.zeros((1, 1, 1, 1, 18 * 64), np.uint8))
    for n in (2048, 2049, 5000, 3000):
        ids = [int(x) for x in rng.permutation(S)[:n]]
        new = [int(x) for x in rng.integers(0, 17, n)]
        want = m.reserve(ids, new)  # the last ones are refused: beyond the table's rows
        assert tuple(fa.fa_kv4_reserve(i32(new), *dev[1:], P, seq_ids=i32(ids)).tolist()) == want
        if want[1] < 0:
            with pytest.raises(fa.FAError, match="invalid argument"):
                fa.fa_check()
        out = [int(x) for x in rng.permutation(S)[:n // 3]]
        fa.fa_kv4_release(i32(out), *dev[1:], P)
        m.release(out)
        fa.fa_check()
        assert dev[1].tolist() == m.table and dev[2].tolist() == m.lens and dev[3].tolist() == m.refs
    empty = [s for s in range(S) if m.lens[s] == 0]
    held = [s for s in range(S) if m.lens[s]]
    kids = empty[:2049]
    parents = [int(x) for x in rng.choice(held, len(kids))]
    pool = rng.integers(0, 256, (1, 9000, 1, 1, 18 * 64), dtype=np.uint8)
    dpool = torch.tensor(pool, device=DEV)
    assert len(kids) == 2049
    assert tuple(fa.fa_kv4_fork(i32(parents), i32(kids), dpool, *dev[1:]).tolist()) == m.fork(parents, kids, pool)
    fa.fa_check()
    _same_state(m, pool, (dpool, *dev[1:]), "fork of many")


def test_page_operations_refuse_and_change_nothing():
    P = 16
    m = kv4.Pages(12, 6, 4, P)
    assert m.reserve([0, 1], [40, 16]) == (8, 0)
    pool = np.random.default_rng(0).integers(0, 256, (1, 12, 1, 1, 18 * 64), dtype=np.uint8)
    dev = _page_state(m, pool)

    def bad(fn, *args, latched=True, info=-1, **kw):
        got = fn(*args, **kw)
        if latched:
            with pytest.raises(fa.FAError, match="invalid argument"):
                fa.fa_check()
        fa.fa_check()
        if got is not None:
            assert got.tolist() == [8, info]
        _same_state(m, pool, dev, fn.__name__)

    reserve = lambda ids, new, **kw: bad(fa.fa_kv4_reserve, i32(new), *dev[1:], P, seq_ids=i32(ids), **kw)  # noqa: E731
    fork = lambda a, b, **kw: bad(fa.fa_kv4_fork, i32(a), i32(b), *dev, **kw)  # noqa: E731
    reserve([0, 0], [1, 1])                     # a slot twice
    reserve([6], [1])
    reserve([-1], [1])
    reserve([2], [-1])                          # more than it has
    reserve([0], [-41])
    reserve([2], [65])                          # beyond the table row
    reserve([2, 3, 4], [64, 64, 64], latched=False, info=4)
    reserve([2, 3], [2 ** 31 - 1, 2 ** 31 - 1])
    fork([0, 0], [2, 2])                        # a child twice
    fork([0], [1])                              # a child in use
    fork([2, 0], [3, 2])                        # a child that is a parent
    fork([0], [6])
    fork([-1], [2])
    bad(fa.fa_kv4_release, i32([6, -1]), *dev[1:], P)
    dev[2][5] = 65                              # a length beyond the table
    m.lens[5] = 65
    bad(fa.fa_kv4_compact, *dev)
    fork([5], [2])
    reserve([5], [0])
    bad(fa.fa_kv4_release, i32([5]), *dev[1:], P)
    dev[2][5] = m.lens[5] = 0
    fork([0, 0, 0, 0, 0], [2, 3, 4, 5, 5])
    m.refs[4:] = [1] * 8
    dev[3].copy_(i32(m.refs))
    got = fa.fa_kv4_fork(i32([0]), i32([2]), *dev)  # no page left for the copy of the last one
    fa.fa_check()
    assert got.tolist() == [0, 1]
    _same_state(m, pool, dev, "fork without pages")


def test_bad_slots_lengths_and_pages_are_latched_and_never_followed():
    rng = np.random.default_rng(8)
    lens = [100, 50]
    pool, table = random_cache(rng, lens, 2, 64, 16)
    dpool = torch.tensor(pool, device=DEV)
    q = bf16(rng.standard_normal((2, 4, 1, 64))).to(DEV)
    kv = bf16(rng.standard_normal((2, 3, 2, 64))).to(DEV)
    cu = i32([0, 1, 3])

    def latched(table, lens, ids=None, cu=cu):
        t, n = i32(table), i32(lens)
        before = dpool.clone()
        for call in (lambda: fa.fa_fwd_kv4(q, dpool, t, n, causal=True, seq_ids=ids),
                     lambda: fa.fa_kv4_read(cu, 3, dpool, t, n, seq_ids=ids),
                     lambda: fa.fa_kv4_append(kv[0], kv[1], cu, dpool, t, n, seq_ids=ids)):
            call()
            with pytest.raises(fa.FAError, match="invalid argument"):
                fa.fa_check()
            fa.fa_check()
        dpool.copy_(before)

    for page in (-1, dpool.shape[0], 2 ** 31 - 1):
        t = table.copy()
        t[1, 3] = page                          # the page of the last positions of sequence 1
        latched(t, lens)
    latched(table, [100, -1])
    latched(table, [100, 16 * table.shape[1] + 1])
    latched(table, lens, ids=i32([0, 2]))
    latched(table, lens, ids=i32([-1, 1]))
    t, n = i32(table), i32(lens)
    for bad in ([0, 2, 1], [1, 2, 3], [0, 1, 4], [0, -1, 3]):
        for fn in (lambda: fa.fa_kv4_append(kv[0], kv[1], i32(bad), dpool, t, n),
                   lambda: fa.fa_kv4_read(i32(bad), 3, dpool, t, n)):
            fn()
            with pytest.raises(fa.FAError, match="invalid argument"):
                fa.fa_check()
    fa.fa_kv4_append(kv[0], kv[1], cu, dpool, t, n, seq_ids=i32([1, 1]))  # one sequence twice
    with pytest.raises(fa.FAError, match="invalid argument"):
        fa.fa_check()
    fa.fa_kv4_read(i32([0, 51]), 51, dpool, t[1:], n[1:])  # more rows than the sequence has
    with pytest.raises(fa.FAError, match="invalid argument"):
        fa.fa_check()
    run_attention(q, dpool, t, n)


def test_binding_refuses_wrong_tensors():
    pool, table, lens = fa.kv4_pool(4, 2, 16, 64), i32([[0, 1], [2, 3]]), i32([3, 4])
    q = torch.zeros(2, 4, 1, 64, dtype=torch.bfloat16, device=DEV)
    kv = torch.zeros(2, 2, 64, dtype=torch.bfloat16, device=DEV)
    refs = torch.ones(4, dtype=torch.int32, device=DEV)
    for err, call in [
        (TypeError, lambda: fa.fa_fwd_kv4(q.half(), pool, table, lens)),
        (TypeError, lambda: fa.fa_fwd_kv4(None, pool, table, lens)),
        (TypeError, lambda: fa.fa_fwd_kv4(q, None, table, lens)),
        (TypeError, lambda: fa.fa_fwd_kv4(q, pool, [[0, 1], [2, 3]], lens)),
        (TypeError, lambda: fa.fa_fwd_kv4(q, pool, table, 3)),
        (TypeError, lambda: fa.fa_kv4_append(kv, kv, [0, 1, 2], pool, table, lens)),
        (TypeError, lambda: fa.fa_kv4_compact(pool, table, lens, None)),
        (TypeError, lambda: fa.fa_kv4_compact(None, table, lens, refs)),
        (TypeError, lambda: fa.fa_kv4_release([0], table, lens, refs, 16)),
        (ValueError, lambda: fa.fa_fwd_kv4(q[:, :, 0], pool, table, lens)),
        (ValueError, lambda: fa.fa_fwd_kv4(q.repeat(1, 1, 2, 1)[:, :, ::2], pool, table, lens)),  # not contiguous
        (ValueError, lambda: fa.fa_fwd_kv4(q.repeat(2, 1, 1, 1), pool, table, lens)),  # more sequences than slots
        (ValueError, lambda: fa.fa_fwd_kv4(torch.cat([q, q], -1), pool, table, lens)),
        (ValueError, lambda: fa.fa_fwd_kv4(q, pool[..., :100].contiguous(), table, lens)),
        (TypeError, lambda: fa.fa_fwd_kv4(q, pool, table.long(), lens)),
        (ValueError, lambda: fa.fa_fwd_kv4(q, pool, table, lens[:1])),
        (ValueError, lambda: fa.fa_fwd_kv4(q, pool, table, lens, seq_ids=i32([0]))),
        (ValueError, lambda: fa.fa_fwd_kv4(q, pool, table, lens, k_scale=torch.ones(3, device=DEV))),
        (ValueError, lambda: fa.fa_fwd_kv4(q, pool, table, lens.cpu())),
        (ValueError, lambda: fa.fa_fwd_kv4(q, pool, table, lens, out=torch.zeros(2, 4, 2, 64, device=DEV))),
        (fa.FAError, lambda: fa.fa_fwd_kv4(q.repeat(1, 33, 1, 1), pool, table, lens)),  # 66 rows per KV head
        (ValueError, lambda: fa.fa_kv4_append(kv, kv[:1], i32([0, 1, 2]), pool, table, lens)),
        (ValueError, lambda: fa.fa_kv4_append(kv, kv, i32([0]), pool, table, lens)),
        (ValueError, lambda: fa.fa_kv4_read(i32([0, 2]), 2, pool, table, lens, k_out=kv.cpu())),
        (ValueError, lambda: fa.fa_kv4_read(i32([0, 2]), 3, pool, table, lens, k_out=kv)),
        (ValueError, lambda: fa.fa_kv4_fork(i32([0]), i32([0, 1]), pool, table, lens, refs)),
        (ValueError, lambda: fa.fa_kv4_fork(i32([0]), i32([1]), pool, table, lens, refs[:3])),
        (fa.FAError, lambda: fa.fa_kv4_release(i32([]), table, lens, refs, 16)),
        (fa.FAError, lambda: fa.fa_kv4_reserve(i32([1]), table, lens, refs, 48)),
    ]:
        with pytest.raises(err):
            call()


# ------------------------------------------------------------------ together

def test_a_served_batch_from_prompt_to_beams():
    """Prompts enter the cache, are forked, decode a few tokens, some leave, the pool is compacted and decoding goes
    on; each step's attention against the oracle on what the cache must hold by then, and a cached prefix read back
    for the packed prompt forward."""
    rng = np.random.default_rng(9)
    Hq, H, D, P, N = 8, 2, 128, 16, 60
    m = kv4.Pages(N, 6, 12, P)
    pool = np.zeros((N, H, P // 16, 18 * D), np.uint8)
    dev = [torch.zeros(N, H, P // 16, 18 * D, dtype=torch.uint8, device=DEV), i32(m.table), i32(m.lens), i32(m.refs)]
    one = np.ones(H)

    def extend(ids, new):
        assert fa.fa_kv4_reserve(i32(new), *dev[1:], P, seq_ids=i32(ids)).tolist() == list(m.reserve(ids, new))
        k, v = bf16(rng.standard_normal((2, sum(new), H, D))).to(DEV)
        cu = np.concatenate([[0], np.cumsum(new)])
        fa.fa_kv4_append(k, v, i32(cu), *dev[:3], seq_ids=i32(ids))
        kv4.append(pool, m.table, m.lens, ids, new, f64(k), f64(v), one, one)

    def decode(ids, Lq):
        extend(ids, [Lq] * len(ids))
        q = bf16(rng.standard_normal((len(ids), Hq, Lq, D))).to(DEV)
        o, lse = run_attention(q, *dev[:3], causal=True, seq_ids=i32(ids))
        check_attention(q, o, lse, pool, m.table, ids, m.lens, one, one, 1 / math.sqrt(D), True, "served")
        same_bytes(dev[0].cpu().numpy(), pool, "served")
        assert dev[1].tolist() == m.table

    extend([0, 1], [100, 37])
    # prompt attention over what the cache holds, packed
    cu = i32([0, 100, 137])
    k, v = fa.fa_kv4_read(cu, 137, *dev[:3])
    q = bf16(rng.standard_normal((137, Hq, D)))
    o, lse = fa.fa_fwd_varlen(q.to(DEV), k, v, cu, cu, 100, 100, causal=True)
    fa.fa_check()
    ro, rl = oracle.attention_varlen(q, k.cpu(), v.cpu(), cu.cpu().numpy(), cu.cpu().numpy(), scale=1 / math.sqrt(D),
                                     causal=True)
    assert np.abs(f64(o) - ro).max() < 1e-2 and np.abs(f64(lse) - rl).max() < 1e-3
    assert fa.fa_kv4_fork(i32([0, 0, 1]), i32([2, 3, 4]), *dev).tolist() == list(m.fork([0, 0, 1], [2, 3, 4], pool[None]))
    decode([0, 1, 2, 3, 4], 1)
    decode([4, 3, 2], 3)
    fa.fa_kv4_release(i32([0, 3]), *dev[1:], P)
    m.release([0, 3])
    assert fa.fa_kv4_compact(*dev).tolist() == list(m.compact(pool[None]))
    decode([1, 2, 4], 1)
    fa.fa_kv4_fork(i32([2]), i32([0]), *dev)
    m.fork([2], [0], pool[None])
    decode([0, 2], 2)
    fa.fa_check()


def test_padded_batch_names_an_empty_slot_again_and_again():
    rng = np.random.default_rng(15)
    H, D, P = 2, 64, 16
    m = kv4.Pages(20, 4, 4, P)
    m.reserve([0, 2], [20, 31])
    pool = np.full((20, H, 1, 18 * D), 255, np.uint8)
    k, v = rng.standard_normal((2, 51, H, D))
    kv4.append(pool, m.table, m.lens, [0, 2], [20, 31], k, v, np.ones(H), np.ones(H))
    dev = _page_state(m, pool)
    ids, new = [2, 3, 0, 3, 3, 0], [1, 0, 2, 0, 0, 0]
    assert fa.fa_kv4_reserve(i32(new), *dev[1:], P, seq_ids=i32(ids)).tolist() == list(m.reserve(ids, new))
    k, v = bf16(rng.standard_normal((2, 3, H, D))).to(DEV)
    fa.fa_kv4_append(k, v, i32([0, 1, 1, 3, 3, 3, 3]), *dev[:3], seq_ids=i32(ids))
    kv4.append(pool, m.table, m.lens, ids, new, f64(k), f64(v), np.ones(H), np.ones(H))
    fa.fa_check()
    _same_state(m, pool, dev, "padded")
    q = bf16(rng.standard_normal((6, 4, 1, D))).to(DEV)
    o, lse = run_attention(q, *dev[:3], causal=True, seq_ids=i32(ids))
    check_attention(q, o, lse, pool, m.table, ids, m.lens, np.ones(H), np.ones(H), 1 / math.sqrt(D), True, "padded")
    fa.fa_kv4_release(i32([3, 2, 3, 2]), *dev[1:], P)
    m.release([3, 2, 3, 2])
    fa.fa_check()
    _same_state(m, pool, dev, "released")


def test_two_graphs_replayed_at_once():
    rng = np.random.default_rng(16)
    lens = [2500, 0, 400]
    pool, table = random_cache(rng, lens, 2, 128, 32)
    dev = (torch.tensor(pool, device=DEV), i32(table), i32(lens))
    qs = [bf16(rng.standard_normal((3, 8, 1, 128))).to(DEV) for _ in range(2)]
    want = [fa.fa_fwd_kv4(q, *dev, causal=True) for q in qs]
    torch.cuda.synchronize()
    graphs, got, streams = [], [], [torch.cuda.Stream() for _ in range(2)]
    for q in qs:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            got.append(fa.fa_fwd_kv4(q, *dev, causal=True))
    for _ in range(20):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert torch.equal(g[0], w[0]) and torch.equal(g[1], w[1])


def test_too_small_a_workspace_is_refused():
    lib = fa.load_library()
    pool, table, lens = fa.kv4_pool(4, 2, 16, 64), i32([[0, 1], [2, 3]]), i32([3, 4])
    q, o = torch.zeros(2, 4, 1, 64, dtype=torch.bfloat16, device=DEV), torch.zeros(2, 4, 1, 64, device=DEV)
    c = fa._kv4(pool, table, lens, None, None, None, 2)[0]
    need = fa.kv4_workspace(2, 4, 2, 1, 64)
    ws = torch.zeros(need, dtype=torch.uint8, device=DEV)
    for ptr, n in ((ws.data_ptr(), need - 1), (None, need), (ws.data_ptr() + 8, need)):
        assert lib.fa_fwd_kv4(q.data_ptr(), o.data_ptr(), o.data_ptr(), 2, 4, 1, 0, 0.1, c, ptr, n,
                              None) == fa.FA_ERR_INVALID_ARG


def test_a_workspace_that_covers_less_memory_than_it_has_elements_is_refused():
    pool, table, lens, refs = fa.kv4_pool(4, 2, 16, 64), i32([[0, 1], [2, 3]]), i32([3, 4]), i32([1, 0, 1, 0])
    q = torch.zeros(2, 4, 1, 64, dtype=torch.bfloat16, device=DEV)
    wide = torch.zeros(1, dtype=torch.uint8, device=DEV).expand(fa.kv4_workspace(2, 4, 2, 1, 64))
    with pytest.raises(ValueError, match="contiguous"):
        fa.fa_fwd_kv4(q, pool, table, lens, workspace=wide)
    with pytest.raises(ValueError, match="contiguous"):
        fa.fa_kv4_compact(pool, table, lens, refs, workspace=wide)


def test_captured_decode_step_follows_the_cache():
    """reserve, append and attention captured once and replayed: each replay is one more token."""
    rng = np.random.default_rng(10)
    Hq, H, D, P, B = 8, 2, 64, 16, 3
    m = kv4.Pages(40, B, 8, P)
    m.reserve([0, 1, 2], [30, 1, 63])
    pool = np.full((40, H, 1, 18 * D), 255, np.uint8)
    dev = _page_state(m, pool)
    k, v = rng.standard_normal((2, 94, H, D))
    kv4.append(pool, m.table, m.lens, [0, 1, 2], [30, 1, 63], k, v, np.ones(H), np.ones(H))
    dev[0].copy_(torch.tensor(pool))
    q, kn, vn = (torch.zeros(B, h, 1, D, dtype=torch.bfloat16, device=DEV) for h in (Hq, H, H))
    one, cu = torch.ones(B, dtype=torch.int32, device=DEV), i32(range(B + 1))
    ws = [torch.empty(n, dtype=torch.uint8, device=DEV) for n in (fa.kv4_pages_workspace(40, B),
                                                                  max(1, fa.kv4_workspace(B, Hq, H, 1, D)))]
    out, lse, info = torch.empty(B, Hq, 1, D, device=DEV), torch.empty(B, Hq, 1, device=DEV), i32([0, 0])

    def step():
        fa.fa_kv4_reserve(one, *dev[1:], P, info=info, workspace=ws[0])
        fa.fa_kv4_append(kn.view(B, H, D), vn.view(B, H, D), cu, *dev[:3])
        fa.fa_fwd_kv4(q, *dev[:3], causal=True, out=out, lse=lse, workspace=ws[1])

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()  # one step without the graph: it is the first token
    side.synchronize()
    m.reserve([0, 1, 2], [1, 1, 1])
    kv4.append(pool, m.table, m.lens, [0, 1, 2], [1, 1, 1], f64(kn)[:, :, 0], f64(vn)[:, :, 0], np.ones(H), np.ones(H))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(20):
        for t in (q, kn, vn):
            t.copy_(bf16(rng.standard_normal(t.shape)))
        graph.replay()
        m.reserve([0, 1, 2], [1, 1, 1])
        kv4.append(pool, m.table, m.lens, [0, 1, 2], [1, 1, 1], f64(kn)[:, :, 0], f64(vn)[:, :, 0], np.ones(H),
                   np.ones(H))
        check_attention(q, out, lse, pool, m.table, range(B), m.lens, np.ones(H), np.ones(H), 1 / math.sqrt(D), True,
                        "replay")
    same_bytes(dev[0].cpu().numpy(), pool, "replays")
    assert dev[2].tolist() == m.lens and info[1] == 0
    fa.fa_check()


def test_calls_of_several_threads_at_once():
    """Threads that share a stream, whose launches may interleave, and one with its own."""
    import threading
    rng = np.random.default_rng(14)
    lens = [3000, 10, 700]
    pool, table = random_cache(rng, lens, 2, 64, 64)
    dev = (torch.tensor(pool, device=DEV), i32(table), i32(lens))
    qs = [bf16(rng.standard_normal((3, 8, 1, 64))).to(DEV) for _ in range(4)]
    want = [fa.fa_fwd_kv4(q, *dev, causal=True) for q in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.current_stream()] * 3 + [torch.cuda.Stream()]
    got = [[] for _ in qs]

    def work(i):
        with torch.cuda.stream(streams[i]):
            for _ in range(50):
                got[i].append(fa.fa_fwd_kv4(qs[i], *dev, causal=True))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert len(g) == 50 and all(torch.equal(o, w[0]) and torch.equal(lse, w[1]) for o, lse in g)


def test_a_load_that_never_arrives_ends_the_call_with_a_timeout():
    rng = np.random.default_rng(12)
    pool, table = random_cache(rng, [500, 40], 2, 64, 32)
    dev = (torch.tensor(pool, device=DEV), i32(table), i32([500, 40]))
    q = bf16(rng.standard_normal((2, 4, 1, 64))).to(DEV)
    fa.load_library().fa_test_inject_fault(1)
    fa.fa_fwd_kv4(q, *dev)
    with pytest.raises(fa.FAError) as e:
        fa.fa_check()
    assert e.value.status == fa.FA_ERR_TIMEOUT
    o, lse = run_attention(q, *dev)
    check_attention(q, o, lse, pool, table, [0, 1], [500, 40], np.ones(2), np.ones(2), 0.125, False, "after a timeout")


@pytest.mark.parametrize("Hq,Hkv,Lq,D", [(8, 2, 1, 128), (7, 1, 1, 128), (16, 1, 1, 128), (10, 1, 4, 64), (16, 2, 1, 64)])
def test_a_timeout_ends_all_warps_of_every_form(Hq, Hkv, Lq, D):
    """Warps that wait on different tiles of long sequences, beside short ones of a warp each: some lanes see the time
    limit and some the flag of another warp, and the block leaves as one."""
    rng = np.random.default_rng(30 + Hq + D)
    lens = [9000, 4000] + [60] * 30
    pool, table = random_cache(rng, lens, Hkv, D, 64)
    dev = (torch.tensor(pool, device=DEV), i32(table), i32(lens))
    q = bf16(rng.standard_normal((len(lens), Hq, Lq, D))).to(DEV)
    want = run_attention(q, *dev, causal=True)
    fa.load_library().fa_test_inject_fault(1)
    fa.fa_fwd_kv4(q, *dev, causal=True)
    with pytest.raises(fa.FAError) as e:
        fa.fa_check()
    assert e.value.status == fa.FA_ERR_TIMEOUT
    got = run_attention(q, *dev, causal=True)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_two_calls_at_once_on_two_streams():
    rng = np.random.default_rng(11)
    lens = [2000, 3, 700]
    pool, table = random_cache(rng, lens, 2, 128, 64)
    dev = (torch.tensor(pool, device=DEV), i32(table), i32(lens))
    qs = [bf16(rng.standard_normal((3, 8, 1, 128))).to(DEV) for _ in range(2)]
    want = [fa.fa_fwd_kv4(q, *dev, causal=True) for q in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(10):
        for q, s in zip(qs, streams):
            with torch.cuda.stream(s):
                got.append(fa.fa_fwd_kv4(q, *dev, causal=True))
    torch.cuda.synchronize()
    for i, (o, lse) in enumerate(got):
        assert torch.equal(o, want[i % 2][0]) and torch.equal(lse, want[i % 2][1])
    out, lse = torch.empty_like(want[0][0]), torch.empty_like(want[0][1])
    torch.cuda.synchronize()
    fa.fa_fwd_kv4(qs[0], *dev, causal=True, out=out, lse=lse, stream=streams[0])  # on a stream that is not current
    streams[0].synchronize()
    assert torch.equal(out, want[0][0])
    for stream in (streams[1], streams[1].cuda_stream, 0):  # all that the call allocates is that stream's
        o, lse = fa.fa_fwd_kv4(qs[1], *dev, causal=True, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(o, want[1][0]) and torch.equal(lse, want[1][1])
        k, v = fa.fa_kv4_read(i32([0, 5, 5, 9]), 9, *dev, stream=stream)
        torch.cuda.synchronize()
        rk, rv = kv4.rows(pool, table, 2, 700, np.ones(2), np.ones(2))
        assert np.array_equal(f64(k[5:]).transpose(1, 0, 2), rk[:, -4:])
    refs = torch.zeros(pool.shape[0], dtype=torch.int32, device=DEV)
    refs[torch.tensor(np.concatenate([table[s, :-(-n // 64)] for s, n in enumerate(lens)]), device=DEV).long()] = 1
    fa.fa_kv4_release(i32([1]), dev[1], dev[2], refs, 64, stream=streams[0])
    info = fa.fa_kv4_reserve(i32([70]), dev[1], dev[2], refs, 64, seq_ids=i32([1]), stream=streams[0])
    streams[0].synchronize()
    assert dev[2].tolist() == [2000, 70, 700] and info.tolist() == [int((refs == 0).sum()), 0]
    fa.fa_check()
