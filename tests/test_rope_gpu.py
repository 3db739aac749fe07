"""GPU tests of rotary positions against the fp64 oracle (oracle/kv16.py)."""
import math

import numpy as np
import pytest
import torch

import exact_attention_07_gb300 as fa
from oracle import kv16

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    fa.load_library()


def f64(t):
    return t.detach().double().cpu().numpy()


def freqs(R, base=500000.0):
    return [base ** (-2 * c / R) for c in range(R // 2)]


def check(got, x, pos, w, rope, back=False, what=""):
    """got [T, H, D] against the oracle for inputs x [T, H, D]."""
    a = f64(x)
    want = kv16.turn(a, pos, w, rope.mscale, rope.start, rope.interleaved, back)
    tol = kv16.turn_tolerance(a, want, max(1.0, rope.mscale), len(w), got.dtype is BF)
    err = np.abs(f64(got) - want)
    assert (err <= tol).all(), f"{what}: {err.max()} at {np.argwhere(err > tol)[0]}"
    rest = np.ones(a.shape[-1], bool)
    rest[rope.start:rope.start + rope.rot_dim] = False
    assert torch.equal(got[..., torch.from_numpy(rest)], x.to(got.dtype)[..., torch.from_numpy(rest)]), "copied dimensions"


CASES = [  # T, Hq, Hk, D, R, start, interleaved, in, out
    (1, 1, 1, 64, 64, 0, False, BF, BF), (1, 32, 8, 128, 128, 0, False, BF, BF), (16, 32, 8, 128, 128, 0, True, BF, BF),
    (3, 5, 3, 192, 64, 128, True, BF, BF), (7, 2, 1, 192, 64, 128, False, F32, BF), (5, 4, 4, 128, 64, 32, False, BF, BF),
    (257, 6, 2, 64, 32, 16, True, F32, F32), (4096, 3, 1, 128, 128, 0, False, F32, BF), (999, 1, 0, 16, 16, 0, True, F32, F32),
    (33, 2, 2, 512, 512, 0, False, BF, BF), (12289, 9, 1, 128, 96, 16, True, BF, BF), (20000, 4, 2, 80, 48, 32, False, F32, F32)]


@pytest.mark.parametrize("T,Hq,Hk,D,R,start,inter,src,dst", CASES)
@pytest.mark.parametrize("back", [False, True])
def test_packed_rows(T, Hq, Hk, D, R, start, inter, src, dst, back):
    g = torch.Generator().manual_seed(T + D)
    q, k = (torch.randn(T, h, D, generator=g).to(src).to(DEV) for h in (Hq, Hk))
    pos = torch.randint(0, 1 << 20, (T,), generator=g, dtype=torch.int32)
    pos[0] = (1 << 31) - 1  # as far as positions go
    if T > 2:
        pos[1], pos[2] = -(1 << 31), 0
    w = freqs(R)
    rope = fa.rope_plan(inv_freq=w, start=start, interleaved=inter, mscale=1.25)
    fn = fa.fa_rope_bwd if back else fa.fa_rope
    yq, yk = fn(q, k if Hk else None, rope, pos.to(DEV), dtype=dst)
    assert fa.fa_last_launch_count() == 1
    fa.fa_check()
    assert yq.dtype is dst and yq.is_contiguous() and (yk is None) == (Hk == 0)
    check(yq, q, pos.numpy(), w, rope, back, "q")
    if Hk:
        check(yk, k, pos.numpy(), w, rope, back, "k")


def test_dense_views_of_a_projection():
    """[B, H, L, D] views of [B, L, (H + 2 Hkv) D] rows become contiguous; positions per batch, shared, or counted."""
    B, H, Hkv, L, D = 3, 4, 2, 37, 128
    g = torch.Generator().manual_seed(1)
    x = torch.randn(B, L, H + 2 * Hkv, D, generator=g).bfloat16().to(DEV)
    q, k = x[:, :, :H].transpose(1, 2), x[:, :, H:H + Hkv].transpose(1, 2)
    rope, w = fa.rope_plan(D, base=10000.0), freqs(D, 10000.0)
    each = torch.randint(0, 1 << 16, (B, L), generator=g, dtype=torch.int32)
    for pos, want in ((each.to(DEV), each), (each[1].to(DEV), each[1].expand(B, L)), (None, torch.arange(L).expand(B, L))):
        yq, yk = fa.fa_rope(q, k, rope, pos)
        for y, a in ((yq, q), (yk, k)):
            assert y.is_contiguous() and y.shape == a.shape
            for b in range(B):
                check(y[b].transpose(0, 1), a[b].transpose(0, 1), want[b].numpy(), w, rope)


def test_in_place_and_broadcast_inputs():
    T, H, D = 50, 3, 128
    rope, w = fa.rope_plan(64, base=10000.0, start=64), freqs(64, 10000.0)
    x = torch.randn(T, 2 * H, D, generator=torch.Generator().manual_seed(2)).bfloat16().to(DEV)
    keep = x.clone()
    q = x[:, :H]
    got, _ = fa.fa_rope(q, None, rope, q_out=q)
    assert got is q and torch.equal(x[:, H:], keep[:, H:])
    check(q, keep[:, :H], np.arange(T), w, rope)
    one = keep[:1, :1].expand(T, H, D)  # strides of 0
    y, _ = fa.fa_rope(one, None, rope)
    check(y, one, np.arange(T), w, rope)
    with pytest.raises(fa.FAError):
        fa.fa_rope(one, None, rope, q_out=one)  # rows that coincide


def test_not_a_number_stays_in_its_pair():
    x = torch.ones(2, 1, 64, device=DEV)
    x[0, 0, 5], x[1, 0, 40] = math.nan, math.inf
    y, _ = fa.fa_rope(x, None, fa.rope_plan(64))
    bad = (~torch.isfinite(y)).nonzero().tolist()
    assert bad == [[0, 0, 5], [0, 0, 37], [1, 0, 8], [1, 0, 40]]


def test_backward_is_the_gradient():
    """<g, turn(x + e d) - turn(x - e d)> / 2e = <turn_back(g), d>: turning is linear, so any e will do.  fp32 terms
    are good to 2^-21 each (turn_tolerance), and 2 T H D of them meet."""
    T, H, D = 13, 2, 64
    g = torch.Generator().manual_seed(3)
    x, d, up = (torch.randn(T, H, D, generator=g).to(DEV) for _ in range(3))
    rope = fa.rope_plan(D, base=100.0, scaling="parts", factor=4.0, original_length=64)
    a, b = (fa.fa_rope(x + s * d, None, rope)[0].double() for s in (0.5, -0.5))
    dx = fa.fa_rope_bwd(up, None, rope)[0].double()
    terms = up.double().abs().sum() * 8 * 2.0 ** -20
    assert abs(((a - b) * up.double()).sum() - (dx * d.double()).sum()) <= terms


def test_turned_back_is_unturned():
    x = torch.randn(100, 4, 128, generator=torch.Generator().manual_seed(4)).to(DEV)
    rope = fa.rope_plan(128)
    pos = torch.arange(100, dtype=torch.int32, device=DEV) * 9973
    y = fa.fa_rope_bwd(fa.fa_rope(x, None, rope, pos)[0], None, rope, pos)[0]
    assert (y - x).abs().max() <= 2 * 2 * 2.0 ** -21 * 2 * x.abs().max()


def test_feeds_attention_and_takes_its_gradients():
    """Turned q and k through the dense forward and backward: the scores depend on distances only, and the gradients
    come back through fa_rope_bwd as those of the unturned inputs (fp64 autograd)."""
    B, Hq, Hkv, L, D = 1, 2, 1, 96, 64
    g = torch.Generator().manual_seed(5)
    q, k, v, do = (torch.randn(B, h, L, D, generator=g).bfloat16().to(DEV) for h in (Hq, Hkv, Hkv, Hq))
    rope = fa.rope_plan(D)
    pos = torch.arange(L, dtype=torch.int32, device=DEV)
    outs = []
    for shift in (0, 1000):
        tq, tk = fa.fa_rope(q, k, rope, pos + shift)
        o, lse = fa.fa_fwd(tq, tk, v, causal=True)
        dq, dk, dv = fa.fa_bwd(tq, tk, v, o, lse, do, causal=True)
        outs.append((o, *fa.fa_rope_bwd(dq, dk, rope, pos + shift), dv))
    q64, k64, v64 = (t.double().cpu().requires_grad_() for t in (q, k, v))
    w = torch.tensor(freqs(D, 10000.0), dtype=torch.float64)
    th = torch.arange(L).double()[:, None] * w

    def turned(x):
        a, b = x[..., :D // 2], x[..., D // 2:]
        return torch.cat((a * th.cos() - b * th.sin(), a * th.sin() + b * th.cos()), -1)

    s = turned(q64) @ turned(k64).transpose(-1, -2) / math.sqrt(D)
    s = s.masked_fill(torch.ones(L, L, dtype=torch.bool).triu(1), -math.inf)
    (s.softmax(-1) @ v64 * do.double().cpu()).sum().backward()
    # q and k are rounded to bf16 behind the turn (2^-8 each), the kernels' own bound is 1e-2 of unit inputs' outputs
    for got in outs:
        for y, ref in zip(got[1:], (q64.grad, k64.grad, v64.grad)):
            rel = (y.double().cpu() - ref).norm() / ref.norm()
            assert rel <= 4 * 2.0 ** -8, rel


def test_streams_and_graph():
    T, H, D = 40, 4, 128
    x = torch.randn(T, H, D, generator=torch.Generator().manual_seed(6)).bfloat16().to(DEV)
    pos = torch.arange(T, dtype=torch.int32, device=DEV)
    rope, w = fa.rope_plan(D), freqs(D, 10000.0)
    want, _ = fa.fa_rope(x, None, rope, pos)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got, _ = fa.fa_rope(x, None, rope, pos, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(got, want)
    y = torch.empty_like(x)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fa.fa_rope(x, None, rope, pos, q_out=y)
    pos += 7
    x.mul_(2)
    graph.replay()
    torch.cuda.synchronize()
    check(y, x, pos.cpu().numpy(), w, rope)


def test_no_rows():
    rope = fa.rope_plan(64)
    q = torch.empty(0, 3, 64, dtype=BF, device=DEV)
    y, z = fa.fa_rope(q, q, rope)
    assert y.shape == z.shape == q.shape and fa.fa_last_launch_count() == 0
