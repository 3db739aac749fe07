"""Refusals of the 4-bit cache's entry points that need no GPU."""
import ctypes

import pytest
import torch

import exact_attention_07_gb300 as fa

INV, UNS = fa.FA_ERR_INVALID_ARG, fa.FA_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    from exact_attention_07_gb300 import _build
    _build.build()
    return fa.load_library()


def cache(**over):
    a = dict(pool=16, table=16, seq_lens=16, seq_ids=None, k_scale=None, v_scale=None, num_pages=4, num_slots=3,
             table_width=2, page_size=64, Hkv=2, D=128)
    a.update(over)
    return fa._KV4(*a.values())


def pages(**over):
    a = dict(pool=16, table=16, seq_lens=16, refs=16, num_pages=4, num_slots=3, table_width=2, page_size=64, Hkv=2,
             D=128, num_layers=1)
    a.update(over)
    return fa._KV4Pages(*a.values())


BAD_CACHE = [(dict(pool=None), INV), (dict(table=None), INV), (dict(seq_lens=None), INV), (dict(pool=24), INV),
             (dict(table=18), INV), (dict(seq_ids=2), INV), (dict(k_scale=6), INV), (dict(v_scale=1), INV),
             (dict(num_pages=0), INV), (dict(num_slots=0), INV), (dict(num_slots=65537), INV),
             (dict(table_width=0), INV), (dict(table_width=1 << 25), INV), (dict(Hkv=0), INV), (dict(D=96), UNS),
             (dict(D=0), INV), (dict(page_size=48), UNS), (dict(page_size=8), UNS), (dict(page_size=512), UNS),
             (dict(num_slots=1), INV)]  # two sequences in one slot's place


@pytest.mark.parametrize("over,status", BAD_CACHE)
def test_cache_descriptions_are_refused(lib, over, status):
    c = cache(**over)
    for fn in (lib.fa_kv4_append, lib.fa_kv4_read):
        assert fn(16, 16, 16, 2, 4, ctypes.byref(c), None) == status
    assert lib.fa_fwd_kv4(16, 16, 16, 2, 4, 1, 0, 0.1, ctypes.byref(c), 16, 1 << 40, None) == status
    assert lib.fa_last_launch_count() == 0


def test_row_calls_are_refused(lib):
    c = ctypes.byref(cache())
    for fn in (lib.fa_kv4_append, lib.fa_kv4_read):
        assert fn(16, 16, 16, 2, 4, None, None) == INV
        assert fn(None, 16, 16, 2, 4, c, None) == INV
        assert fn(16, 8, 16, 2, 4, c, None) == INV        # 16-byte alignment
        assert fn(16, 16, None, 2, 4, c, None) == INV
        assert fn(16, 16, 18, 2, 4, c, None) == INV
        assert fn(16, 16, 16, 0, 4, c, None) == INV
        assert fn(16, 16, 16, 2, -1, c, None) == INV


def test_attention_calls_are_refused(lib):
    def call(q=16, o=16, lse=16, B=2, Hq=4, Lq=1, scale=0.1, **over):
        return lib.fa_fwd_kv4(q, o, lse, B, Hq, Lq, 0, scale, ctypes.byref(cache(**over)), 16, 1 << 40, None)

    assert call(q=None) == INV and call(o=None) == INV and call(lse=24) == INV
    assert call(B=0) == INV and call(Lq=0) == INV and call(Hq=3) == INV
    assert call(scale=0.0) == INV and call(scale=float("nan")) == INV
    assert call(Hq=2, Lq=65) == UNS and call(Hq=130, Hkv=2) == UNS
    n = ctypes.c_size_t()
    assert lib.fa_fwd_kv4_workspace(1, 4, 2, 1, 128, None) == INV
    assert lib.fa_fwd_kv4_workspace(1, 4, 3, 1, 128, ctypes.byref(n)) == INV
    assert lib.fa_fwd_kv4_workspace(1, 4, 2, 1, 32, ctypes.byref(n)) == UNS


BAD_PAGES = [(dict(table=None), INV), (dict(seq_lens=None), INV), (dict(refs=None), INV), (dict(refs=20), INV),
             (dict(num_pages=0), INV), (dict(num_slots=70000), INV), (dict(page_size=20), UNS), (dict(D=32), UNS)]


@pytest.mark.parametrize("over,status", BAD_PAGES)
def test_page_descriptions_are_refused(lib, over, status):
    p = ctypes.byref(pages(**over))
    big = 1 << 40
    assert lib.fa_kv4_reserve(None, 16, 2, p, 16, 16, big, None) == status
    assert lib.fa_kv4_fork(16, 16, 2, p, 16, 16, big, None) == status
    assert lib.fa_kv4_release(16, 2, p, None) == status
    assert lib.fa_kv4_compact(p, 16, 16, big, None) == status


def test_page_calls_are_refused(lib):
    p, big = ctypes.byref(pages()), 1 << 40
    assert lib.fa_kv4_reserve(None, None, 2, p, 16, 16, big, None) == INV
    assert lib.fa_kv4_reserve(None, 16, 0, p, 16, 16, big, None) == INV
    assert lib.fa_kv4_reserve(None, 16, 2, p, None, 16, big, None) == INV
    n = fa.KV4_SEQS_WITHOUT_WORKSPACE + 1
    assert lib.fa_kv4_reserve(16, 16, n, p, 16, None, big, None) == INV    # up to 2048 sequences it needs none
    assert lib.fa_kv4_reserve(16, 16, n, p, 16, 16, 8, None) == INV        # workspace too small
    assert lib.fa_kv4_fork(16, 16, n, p, 16, None, big, None) == INV
    assert lib.fa_kv4_compact(p, 16, None, big, None) == INV
    assert lib.fa_kv4_fork(None, 16, 2, p, 16, 16, big, None) == INV
    assert lib.fa_kv4_fork(16, None, 2, p, 16, 16, big, None) == INV
    assert lib.fa_kv4_fork(16, 16, 65537, p, 16, 16, big, None) == INV
    nopool = ctypes.byref(pages(pool=None))
    assert lib.fa_kv4_fork(16, 16, 2, nopool, 16, 16, big, None) == INV
    assert lib.fa_kv4_compact(nopool, 16, 16, big, None) == INV
    assert lib.fa_kv4_compact(ctypes.byref(pages(num_layers=0)), 16, 16, big, None) == INV
    assert lib.fa_kv4_release(None, 2, p, None) == INV and lib.fa_kv4_release(16, 0, p, None) == INV
    n = ctypes.c_size_t()
    assert lib.fa_kv4_pages_workspace(0, 1, ctypes.byref(n)) == INV
    assert lib.fa_kv4_pages_workspace(4, -1, ctypes.byref(n)) == INV
    assert lib.fa_kv4_pages_workspace(1000, 10, ctypes.byref(n)) == fa.FA_OK and n.value >= 4 * (2 * 1000 + 10)


def test_binding_checks_shapes_before_the_library():
    with pytest.raises(ValueError, match="page_size"):
        fa.kv4_pool(4, 2, 48, 64, device="cpu")
    pool = fa.kv4_pool(4, 2, 32, 64, layers=3, device="cpu")
    assert pool.shape == (3, 4, 2, 2, 18 * 64) and not pool.any()
    i32 = torch.int32
    with pytest.raises(ValueError, match="CUDA tensor"):
        fa.fa_fwd_kv4(torch.zeros(1, 2, 1, 64, dtype=torch.bfloat16), pool[0], torch.zeros(1, 2, dtype=i32),
                      torch.zeros(1, dtype=i32))
