"""Refusals of the rotary calls and of the 16-bit cache's, and their host helpers, that need no GPU."""
import ctypes
import math

import numpy as np
import pytest
import torch

import exact_attention_07_gb300 as fa
from oracle import kv16

INV, UNS = fa.FA_ERR_INVALID_ARG, fa.FA_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    from exact_attention_07_gb300 import _build
    _build.build()
    return fa.load_library()


def cache(**over):
    a = dict(pool=16, table=16, seq_lens=16, seq_ids=None, num_pages=4, num_slots=3, table_width=2, page_size=64, Hkv=2,
             D=128)
    a.update(over)
    return ctypes.byref(fa._KV16(*a.values()))


def rows(**over):
    a = dict(x=16, y=32, x_batch=0, x_token=256, x_head=128, y_batch=0, y_token=256, y_head=128, heads=2)
    a.update(over)
    return ctypes.byref(fa._RotaryRows(*a.values()))


def rope(**over):
    a = dict(freqs=16, rot_dim=128, start=0, interleaved=0, mscale=1.0)
    a.update(over)
    return ctypes.byref(fa._Rope(*a.values()))


BAD_CACHE = [(dict(pool=None), INV), (dict(table=None), INV), (dict(seq_lens=None), INV), (dict(pool=24), INV),
             (dict(table=18), INV), (dict(seq_ids=2), INV), (dict(num_pages=0), INV), (dict(num_slots=0), INV),
             (dict(num_slots=65537), INV), (dict(table_width=0), INV), (dict(table_width=1 << 25), INV),
             (dict(Hkv=0), INV), (dict(D=96), UNS), (dict(D=0), INV), (dict(page_size=48), UNS), (dict(page_size=8), UNS),
             (dict(page_size=512), UNS), (dict(num_slots=1), INV), (dict(num_pages=1 << 29, Hkv=2), INV)]


@pytest.mark.parametrize("over,status", BAD_CACHE)
def test_cache_descriptions_are_refused(lib, over, status):
    H, D = over.get("Hkv", 2), over.get("D", 128)
    assert lib.fa_kv16_append(None, rows(), rows(), 16, 2, 4, cache(**over), rope(), None, None) == status
    assert lib.fa_kv16_keep(16, 16, 16, 2, 4, 1, 16, cache(**over), None) == status
    if H and D in (64, 128):
        assert lib.fa_fwd_kv16(16, 512, 128, 16, 16, 16, 2, 4, 4, None, 0, 1, 0.1, cache(**over), 16, 1 << 40, None) == status
    assert lib.fa_last_launch_count() == 0


def test_append_calls_are_refused(lib):
    def call(q=None, k=rows(), v=rows(), cu=16, n=2, total=4, c=cache(), r=rope(), pos=None):
        return lib.fa_kv16_append(q, k, v, cu, n, total, c, r, pos, None)

    assert call(c=None) == INV and call(k=None) == INV and call(v=None) == INV and call(cu=None) == INV
    assert call(cu=18) == INV and call(pos=18) == INV and call(n=0) == INV and call(total=-1) == INV
    assert call(total=(1 << 30) + 1) == INV
    assert call(k=rows(heads=1)) == INV and call(v=rows(heads=3)) == INV        # not the cache's heads
    assert call(k=rows(x=None)) == INV and call(k=rows(x=24)) == INV and call(v=rows(x_token=12)) == INV
    assert call(q=rows(), r=None) == INV                                        # q without a rotation
    assert call(q=rows(y=None)) == INV and call(q=rows(y_token=0)) == INV and call(q=rows(heads=0)) == INV
    assert call(q=rows(y=16, y_token=512)) == INV                               # in place with other strides
    assert call(r=rope(rot_dim=0)) == INV and call(r=rope(rot_dim=256)) == INV and call(r=rope(start=64)) == INV
    assert call(r=rope(rot_dim=24)) == UNS and call(r=rope(rot_dim=64, start=8)) == UNS
    assert call(r=rope(freqs=None)) == INV and call(r=rope(freqs=20)) == INV
    for m in (0.0, -1.0, math.nan, math.inf):
        assert call(r=rope(mscale=m)) == INV


def test_rope_calls_are_refused(lib):
    def call(q=rows(), k=None, B=1, T=4, D=128, src=0, dst=0, r=rope(), pos=None, fn=lib.fa_rope):
        return fn(q, k, B, T, D, src, dst, r, pos, 0, None)

    for fn in (lib.fa_rope, lib.fa_rope_bwd):
        assert call(q=None, fn=fn) == INV and call(r=None, fn=fn) == INV
        assert call(D=120, fn=fn) == UNS and call(D=528, fn=fn) == UNS and call(D=0, fn=fn) == INV
        assert call(dst=1, fn=fn) == UNS                                         # bf16 rows do not become fp32
        assert call(B=-1, fn=fn) == INV and call(T=-1, fn=fn) == INV and call(pos=2, fn=fn) == INV
        assert call(q=rows(x_head=100), fn=fn) == INV and call(q=rows(y_head=0), fn=fn) == INV
        assert call(q=rows(y=16), src=1, fn=fn) == INV                           # fp32 to bf16 in place
        assert call(k=rows(x=8), fn=fn) == INV
        assert call(B=1 << 16, T=1 << 15, fn=fn) == INV
        assert call(T=0, fn=fn) == 0 and call(B=0, fn=fn) == 0                   # no rows: nothing to do
    assert call(q=rows(x_token=3, y_token=3), T=1) not in (INV, 0)               # of one token any stride will do (no device here)


def test_attention_calls_are_refused(lib):
    def call(q=16, qt=512, qh=128, o=16, lse=16, cu=16, n=2, total=4, Hq=4, mask=None, words=0, causal=1, scale=0.1, ws=16,
             **over):
        return lib.fa_fwd_kv16(q, qt, qh, o, lse, cu, n, total, Hq, mask, words, causal, scale, cache(**over), ws, 1 << 40, None)

    assert lib.fa_fwd_kv16(16, 512, 128, 16, 16, 16, 2, 4, 4, None, 0, 1, 0.1, None, 16, 1 << 40, None) == INV
    assert call(cu=None) == INV and call(cu=17) == INV and call(n=0) == INV and call(total=-1) == INV
    assert call(Hq=3) == INV and call(Hq=0) == INV and call(Hq=258) == UNS and call(total=(1 << 30) + 1) == INV
    assert call(scale=0.0) == INV and call(scale=-1.0) == INV and call(scale=float("nan")) == INV
    assert call(mask=16, words=1, causal=1) == INV and call(mask=16, words=0, causal=0) == INV
    assert call(mask=18, words=1, causal=0) == INV
    n = ctypes.c_size_t()
    assert lib.fa_fwd_kv16_workspace(4, 4, 2, 128, None) == INV
    assert lib.fa_fwd_kv16_workspace(4, 4, 3, 128, ctypes.byref(n)) == INV
    assert lib.fa_fwd_kv16_workspace(4, 4, 2, 32, ctypes.byref(n)) == UNS
    assert lib.fa_fwd_kv16_workspace(4, 512, 2, 64, ctypes.byref(n)) == UNS


def test_keep_calls_are_refused(lib):
    def call(keep=16, counts=16, cu=16, n=2, total=4, layers=1, new=16):
        return lib.fa_kv16_keep(keep, counts, cu, n, total, layers, new, cache(), None)

    assert call(keep=None) == INV and call(counts=None) == INV and call(cu=None) == INV and call(new=None) == INV
    assert call(keep=18) == INV and call(new=2) == INV and call(n=0) == INV and call(total=-1) == INV
    assert call(layers=0) == INV and call(layers=1 << 28) == INV


def test_tensors_are_refused_before_the_library():
    """Wrong types, shapes, devices: with CPU tensors every call stops at its checks."""
    bf = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    plan = fa.rope_plan(64, device="cpu")
    with pytest.raises(TypeError):
        fa.fa_rope([1], None, plan)
    with pytest.raises(TypeError):
        fa.fa_rope(bf.half(), None, plan)
    with pytest.raises(ValueError):
        fa.fa_rope(bf[0], None, plan)
    with pytest.raises(ValueError, match="CUDA"):
        fa.fa_rope(bf, None, plan)
    pool, table, lens = torch.zeros(2, 2, 1, 16, 64), torch.zeros(1, 2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    cu = torch.tensor([0, 4], dtype=torch.int32)
    for call in (lambda p: fa.fa_fwd_kv16(bf, cu, p, table, lens), lambda p: fa.fa_kv16_append(bf, bf, cu, p, table, lens),
                 lambda p: fa.fa_kv16_keep(cu, lens, cu, p, table, lens)):
        with pytest.raises(ValueError):
            call(pool.bfloat16())
        with pytest.raises((TypeError, ValueError)):
            call(pool)
        with pytest.raises(TypeError):
            call(None)


def test_pools():
    assert fa.kv16_pool(3, 2, 32, 64, device="cpu").shape == (3, 2, 2, 32, 64)
    assert fa.kv16_pool(3, 2, 32, 128, layers=4, device="cpu").shape == (4, 3, 2, 2, 32, 128)
    for P, D in ((8, 64), (48, 64), (512, 64), (16, 96)):
        with pytest.raises(ValueError):
            fa.kv16_pool(3, 2, P, D, device="cpu")


def turns(plan):
    """The plan's turns per position as fp64."""
    return np.array([(x % 2 ** 64) / 2.0 ** 64 for x in plan.freqs.tolist()])


@pytest.mark.parametrize("scaling", [None, "linear", "base", "parts"])
def test_plans_hold_the_frequencies(scaling):
    R, base, f, old = 64, 10000.0, 8.0, 4096
    c = np.arange(R // 2)
    w, m = base ** (-2 * c / R), 1.0
    if scaling == "linear":
        w = w / f
    elif scaling == "base":
        w = (base * f ** (R / (R - 2))) ** (-2 * c / R)
    elif scaling == "parts":
        n = old * w / (2 * np.pi)
        a = np.clip((n - 1) / 31, 0, 1)
        w, m = w * a + w / f * (1 - a), 0.1 * math.log(f) + 1
        assert a[0] == 1 and a[-1] == 0
    plan = fa.rope_plan(R, base=base, scaling=scaling, factor=f, original_length=old if scaling == "parts" else None,
                        device="cpu")
    assert np.allclose(turns(plan) * 2 * np.pi, w, rtol=1e-13, atol=0)  # a handful of fp64 steps
    assert plan.mscale == m and (plan.rot_dim, plan.start, plan.end, plan.interleaved) == (R, 0, R, False)
    other = fa.rope_plan(inv_freq=torch.tensor(w), start=16, interleaved=True, mscale=2.0, device="cpu")
    assert np.allclose(turns(other) * 2 * np.pi, w, rtol=1e-13, atol=0) and other.mscale == 2.0 and other.end == 80


def test_plans_are_exact_at_far_positions():
    """Position times frequency modulo 2^64 against the product in exact numbers (oracle): 2^-64 of a turn a position."""
    w = [1.0, 0.3, 3e-5, 0.0, -0.25, 7.0, 1e-9, 123.456]
    plan = fa.rope_plan(inv_freq=w, device="cpu")
    pos = [0, 1, -1, 2 ** 31 - 1, -2 ** 31, 123456789]
    want = kv16.angles(pos, w) / (2 * np.pi)
    for i, p in enumerate(pos):
        for c, f in enumerate(plan.freqs.tolist()):
            got = (p * f % 2 ** 64) / 2.0 ** 64
            d = abs(got - want[i, c])
            assert min(d, 1 - d) <= abs(p) * 2.0 ** -64 + 2.0 ** -52


@pytest.mark.parametrize("bad", [dict(), dict(rot_dim=24), dict(rot_dim=-16), dict(rot_dim=32, base=0.0),
                                 dict(rot_dim=32, factor=-1.0), dict(rot_dim=32, scaling="none"),
                                 dict(rot_dim=32, scaling="parts", factor=2.0), dict(inv_freq=[1.0] * 7),
                                 dict(inv_freq=[]), dict(inv_freq=[math.nan] * 8), dict(inv_freq=[1.0] * 8, factor=2.0),
                                 dict(inv_freq=[1.0] * 8, rot_dim=32), dict(rot_dim=32, mscale=0.0),
                                 dict(rot_dim=32, mscale=math.inf), dict(rot_dim=32, start=8), dict(rot_dim=32, start=-16)])
def test_plans_are_refused(bad):
    with pytest.raises(ValueError):
        fa.rope_plan(device="cpu", **bad)


def test_draft_masks():
    rng = np.random.default_rng(3)
    sizes = [0, 1, 70, 33, 0, 5]
    parents = [[int(rng.integers(-1, i)) if i else -1 for i in range(n)] for n in sizes]
    cu = np.concatenate([[0], np.cumsum(sizes)]).tolist()
    mask, depth = fa.draft_mask([p for t in parents for p in t], cu)
    assert mask.shape == (cu[-1], 3) and mask.dtype == depth.dtype == torch.int32
    for s, t in enumerate(parents):
        see = kv16.ancestors(t)
        bits = np.unpackbits(mask[cu[s]:cu[s + 1]].numpy().view(np.uint8), axis=1, bitorder="little")
        assert np.array_equal(bits[:, :len(t)], see) and not bits[:, len(t):].any()
        assert np.array_equal(depth[cu[s]:cu[s + 1]].numpy(), see.sum(1) - 1)
    empty, none = fa.draft_mask([], [0, 0])
    assert empty.shape == (0, 1) and none.shape == (0,)
    for p, c in (([0], [0, 1]), ([-2], [0, 1]), ([-1, 1], [0, 2]), ([-1], [0, 2]), ([-1], [1, 1]), ([-1], [0]),
                 ([-1, -1], [0, 2, 1])):
        with pytest.raises(ValueError):
            fa.draft_mask(p, c)


def test_oracle_turns_pairs():
    """Against a rotation matrix written out, and its transpose for the gradient."""
    rng = np.random.default_rng(1)
    x, w, m = rng.standard_normal((5, 2, 12)), [0.7, 0.01], 1.3
    pos = [0, 3, -5, 1000, 7]
    for inter in (False, True):
        for i, p in enumerate(pos):
            M = np.eye(12)
            for c, f in enumerate(w):
                a, b = (4 + 2 * c, 5 + 2 * c) if inter else (4 + c, 6 + c)
                M[a, a] = M[b, b] = m * np.cos(p * f)
                M[a, b], M[b, a] = -m * np.sin(p * f), m * np.sin(p * f)
            assert np.allclose(kv16.turn(x, pos, w, m, 4, inter)[i], x[i] @ M.T, atol=1e-12)
            assert np.allclose(kv16.turn(x, pos, w, m, 4, inter, back=True)[i], x[i] @ M, atol=1e-12)


def test_oracle_attends_what_rows_see():
    rng = np.random.default_rng(2)
    q, k, v = rng.standard_normal((3, 4, 8)), rng.standard_normal((7, 2, 8)), rng.standard_normal((7, 2, 8))
    own = np.array([[1, 0, 0], [1, 1, 0], [0, 0, 0]], bool)
    v[6], k[6] = np.nan, np.inf  # the last position: seen by nobody
    o, lse, mag = kv16.attention(q, k, v, 0.5, own)
    for i in range(3):
        keys = [0, 1, 2, 3] + [4 + j for j in range(3) if own[i, j]]
        for h in range(4):
            s = 0.5 * k[keys, h // 2] @ q[i, h]
            p = np.exp(s) / np.exp(s).sum()
            assert np.allclose(o[i, h], p @ v[keys, h // 2]) and np.isclose(lse[h, i], np.log(np.exp(s).sum()))
    o, lse, _ = kv16.attention(q, k[4:], v[4:], 0.5, np.zeros((3, 3), bool))
    assert not o.any() and np.isneginf(lse).all()


# Where the call's inputs begin: keep [4], counts [2], cu_seqlens [3], slots [2], lengths [3], table [3][2], 4 bytes each
KEEP_INPUTS = dict(keep=(0x1000, 4), counts=(0x2000, 2), cu=(0x3000, 3), seq_ids=(0x4000, 2), seq_lens=(0x5000, 3),
                   table=(0x6000, 6))


@pytest.mark.parametrize("name", KEEP_INPUTS)
def test_keep_refuses_new_tokens_over_its_inputs(lib, name):
    """One block of a sequence writes its new_tokens while others may not have read the inputs yet."""
    at, n = KEEP_INPUTS[name]
    a = {k: v[0] for k, v in KEEP_INPUTS.items()}

    c = cache(seq_ids=a["seq_ids"], seq_lens=a["seq_lens"], table=a["table"], num_slots=3, table_width=2)
    for new in (at, at + 4, at - 4, at + 4 * (n - 1)):
        assert lib.fa_kv16_keep(a["keep"], a["counts"], a["cu"], 2, 4, 1, new, c, None) == INV


def test_early_ways_out_of_the_attention_leave_nothing_to_join():
    """The second kernel runs whatever becomes of the first and takes its blocks' parts from the workspace, which can
    hold anything: a block that returns before it has said that there are none says so on its way out.  No launch gets
    there (the address that the branch looks at is always aligned), so the source is what can be looked at."""
    import os
    import re

    path = os.path.join(os.path.dirname(fa.__file__), "csrc", "fa_kv16_attn.cu")
    with open(path) as f:
        text = f.read()
    head = text[text.index("fa_kv16_attn_kernel(const"):]
    head = head[:head.index("__syncthreads()")]
    exits = [m.start() for m in re.finditer(r"\breturn;", head)]
    assert len(exits) == 1
    for at in exits:
        depth, begin = 0, at  # the branch that returns: back to the brace that opens it
        while depth >= 0:
            begin -= 1
            depth += {"}": 1, "{": -1}.get(head[begin], 0)
        assert "join[blockIdx.x].parts = 0;" in head[begin:at]


def held(plan):
    """What a call hands to the library: address of the frequencies, dimensions, start, order, factor."""
    p = fa._Rope.from_buffer_copy(plan.packed)
    return p.freqs, p.rot_dim, p.start, p.interleaved, p.mscale


@pytest.mark.parametrize("way", ["copy", "deepcopy", "pickle", "module"])
def test_copies_of_plans_hold_frequencies_of_their_own(way):
    """A copied plan must not hand over the address of the original's frequencies, which may be gone by then."""
    import copy
    import pickle

    plan = fa.rope_plan(32, base=500.0, start=16, interleaved=True, mscale=0.5, device="cpu")
    if way == "module":
        m = torch.nn.Linear(1, 1)
        m.rope = plan
        other = copy.deepcopy(m).rope
    else:
        other = pickle.loads(pickle.dumps(plan)) if way == "pickle" else getattr(copy, way)(plan)
    assert torch.equal(other.freqs, plan.freqs) and (other.freqs is plan.freqs) == (way == "copy")
    assert held(other) == (other.freqs.data_ptr(), 32, 16, 1, 0.5)
    assert (other.end, other.device, other.interleaved) == (48, -1, True)


def test_plans_stay_as_they_are():
    """The library gets what a plan was made with: a changed attribute would say otherwise."""
    plan = fa.rope_plan(32, device="cpu")
    for name, value in (("mscale", 2.0), ("start", 16), ("interleaved", True), ("freqs", plan.freqs + 1), ("rot_dim", 16)):
        with pytest.raises(AttributeError):
            setattr(plan, name, value)
        with pytest.raises(AttributeError):
            delattr(plan, name)
    assert held(plan) == (plan.freqs.data_ptr(), 32, 0, 0, 1.0)


@pytest.mark.parametrize("bad", [dict(freqs=[1] * 8), dict(freqs=torch.zeros(8)), dict(freqs=torch.zeros(8, dtype=torch.int32)),
                                 dict(freqs=torch.zeros(0, dtype=torch.int64)), dict(freqs=torch.zeros(12, dtype=torch.int64)),
                                 dict(freqs=torch.zeros(2, 8, dtype=torch.int64)),
                                 dict(freqs=torch.zeros(16, dtype=torch.int64)[::2]), dict(start=8), dict(start=-16),
                                 dict(mscale=0.0), dict(mscale=math.nan), dict(mscale=math.inf)])
def test_plans_of_other_frequencies_are_refused(bad):
    """The kernels read rot_dim / 2 numbers of 64 bits where the plan says that they are."""
    args = dict(freqs=torch.zeros(8, dtype=torch.int64), start=0, interleaved=False, mscale=1.0)
    assert held(fa.RopePlan(**args))[1:] == (16, 0, 0, 1.0)
    with pytest.raises((TypeError, ValueError)):
        fa.RopePlan(**{**args, **bad})


def test_rows_written_are_no_other_rows(lib):
    """One block turns q in place while another reads it as k, or both write the same rows."""
    x, y, z = 0x1000, 0x2000, 0x3000
    for fn in (lib.fa_rope, lib.fa_rope_bwd):
        for q, k in (((x, x), (x, y)), ((x, y), (y, z)), ((x, y), (y, y)), ((x, y), (z, x)), ((x, y), (z, y)), ((x, x), (x, x))):
            assert fn(rows(x=q[0], y=q[1]), rows(x=k[0], y=k[1]), 1, 4, 128, 0, 0, rope(), None, 0, None) == INV
    for k, v in ((y, z), (z, y), (y, y)):
        assert lib.fa_kv16_append(rows(x=x, y=y), rows(x=k), rows(x=v), 16, 2, 4, cache(), rope(), None, None) == INV


@pytest.mark.parametrize("gpu", [False, True])
def test_calls_that_would_launch_on_nothing_stay_off_a_gpu(gpu, monkeypatch, request):
    """test_rope_calls_are_refused makes one call that is sound but for its made-up addresses: it ends for want of a
    device, and with one it would read them."""
    class Item:
        def __init__(self, name):
            self.name, self.marks = name, []

        def add_marker(self, mark):
            self.marks.append(mark.name)

    conftest = [p for p in request.config.pluginmanager.get_plugins() if hasattr(p, "NEEDS_NO_GPU")]
    monkeypatch.setattr(torch.cuda, "is_available", lambda: gpu)
    items = [Item("test_rope_calls_are_refused"), Item("test_keep_calls_are_refused")]
    assert conftest, "no list of such tests"
    conftest[0].pytest_collection_modifyitems(items)
    assert [i.marks for i in items] == [["skip"] if gpu else [], []]
