"""Refusals of the 4-bit cache's entry points that need no GPU."""
import contextlib
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


class FakeStream:
    def __init__(self, device, handle):
        self.device, self.cuda_stream = torch.device("cuda", device), handle


class OnCuda1(torch.Tensor):
    """A host tensor that says it is on cuda:1 and keeps the streams it is recorded on."""
    is_cuda, device = True, torch.device("cuda", 1)

    def get_device(self):
        return 1

    def record_stream(self, stream):
        self.__dict__.setdefault("recorded", []).append(stream.cuda_stream)


@pytest.fixture
def two_gpus(monkeypatch):
    """Two devices of the CUDA runtime's host side, cuda:0 current, and a library that keeps (call, device, stream)."""
    now, current, calls = [0], {0: FakeStream(0, 100), 1: FakeStream(1, 200)}, []

    @contextlib.contextmanager
    def device(index):
        before, now[0] = now[0], torch.device("cuda", index).index if isinstance(index, int) else index.index
        yield
        now[0] = before

    @contextlib.contextmanager
    def stream(s):
        before, current[s.device.index] = current[s.device.index], s
        with device(s.device):
            yield
        current[s.device.index] = before

    def index_of(device):
        return now[0] if device is None else torch.device("cuda", device).index if isinstance(device, int) else device.index

    class Library:
        def __getattr__(self, name):
            return lambda *args: calls.append((name, now[0], args[-1])) or fa.FA_OK

    monkeypatch.setattr(torch.cuda, "Stream", FakeStream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: FakeStream(index_of(device), handle))
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: FakeStream(index_of(device), 0))
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: current[index_of(device)])
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: now[0])
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: current[index].cuda_stream)
    monkeypatch.setattr(fa, "_lib", Library())
    monkeypatch.setattr(fa, "_attn_workspace", lambda *args: 64)
    monkeypatch.setattr(fa, "kv4_pages_workspace", lambda *args: 64)
    return calls


def kv4_calls():
    """Every call that takes a stream, on tensors of cuda:1, and the workspace it is given (or None)."""
    def there(*shape, dtype=torch.int32):
        return torch.zeros(shape, dtype=dtype).as_subclass(OnCuda1)

    pool, table, lens, refs = there(4, 2, 1, 18 * 64, dtype=torch.uint8), there(2, 2), there(2), there(4)
    q, kv, cu = there(2, 4, 1, 64, dtype=torch.bfloat16), there(3, 2, 64, dtype=torch.bfloat16), there(3)
    o, lse, info = there(2, 4, 1, 64, dtype=torch.float32), there(2, 4, 1, dtype=torch.float32), there(2)
    ws = [there(64, dtype=torch.uint8) for _ in range(4)]
    return [
        ("fa_kv4_append", lambda s: fa.fa_kv4_append(kv, kv, cu, pool, table, lens, stream=s), None),
        ("fa_kv4_read", lambda s: fa.fa_kv4_read(cu, 3, pool, table, lens, k_out=kv, v_out=kv, stream=s), None),
        ("fa_fwd_kv4", lambda s: fa.fa_fwd_kv4(q, pool, table, lens, out=o, lse=lse, workspace=ws[0], stream=s), ws[0]),
        ("fa_kv4_reserve", lambda s: fa.fa_kv4_reserve(lens, table, lens, refs, 16, info=info, workspace=ws[1], stream=s),
         ws[1]),
        ("fa_kv4_fork", lambda s: fa.fa_kv4_fork(lens, lens, pool, table, lens, refs, info=info, workspace=ws[2], stream=s),
         ws[2]),
        ("fa_kv4_release", lambda s: fa.fa_kv4_release(lens, table, lens, refs, 16, stream=s), None),
        ("fa_kv4_compact", lambda s: fa.fa_kv4_compact(pool, table, lens, refs, info=info, workspace=ws[3], stream=s), ws[3]),
    ]


def test_a_stream_is_one_of_the_tensors_device(two_gpus):
    for name, call, _ in kv4_calls():
        for stream, handle in ((7, 7), (0, 0), (FakeStream(1, 55), 55), (None, 200)):
            two_gpus.clear()
            call(stream)
            assert two_gpus == [(name, 1, handle)]
        two_gpus.clear()
        with pytest.raises(ValueError, match="stream"):
            call(FakeStream(0, 66))
        assert two_gpus == []


def test_a_callers_workspace_is_kept_until_its_stream_is_done(two_gpus):
    for name, call, ws in kv4_calls():
        call(FakeStream(1, 55))
        call(None)  # on the current stream, whose order protects it
        assert ws is None or ws.recorded == [55], name
