"""The Python side of the paged calls on the CPU: whose memory they hand to the library, and
on which stream they take it.  No kernel runs."""
import contextlib
import copy
import pickle

import pytest
import torch

import canvas_denoising_denoise_b200 as dg
from canvas_denoising_denoise_b200 import _lib


def tensors(n_pages):
    pages = torch.zeros((n_pages, 2, 16, 64), dtype=torch.uint8)
    exps = torch.zeros((n_pages, 2), dtype=torch.uint8)
    return pages, pages.clone(), exps, exps.clone()


@pytest.mark.parametrize("name", ["k_pages", "v_pages", "k_exp", "v_exp"])
def test_a_caches_tensors_cannot_be_exchanged(name):
    """The calls hand over memory that the constructor has checked: no other tensor takes its place."""
    cache = dg.PagedCache(*tensors(4))
    with pytest.raises(AttributeError):
        setattr(cache, name, getattr(cache, name).clone())


@pytest.mark.parametrize("at", range(4))
def test_a_caches_pointers_follow_its_tensors(at):
    parts = tensors(4)
    cache = dg.PagedCache(*parts)
    assert cache.pointers == tuple(t.data_ptr() for t in parts)
    parts[at].set_(torch.zeros_like(parts[at]).clone())
    assert cache.pointers == tuple(t.data_ptr() for t in parts)
    parts[at].resize_(1 << 20)
    with pytest.raises(ValueError):
        cache.pointers


@pytest.mark.parametrize("how", [copy.deepcopy, lambda c: pickle.loads(pickle.dumps(c))])
def test_a_copied_cache_has_its_own_memory(how):
    cache = dg.PagedCache(*tensors(4))
    cache.k_pages.fill_(3)
    other = how(cache)
    own = tuple(t.data_ptr() for t in (other.k_pages, other.v_pages, other.k_exp, other.v_exp))
    assert other.pointers == own and not set(own) & set(cache.pointers)
    assert other.n_pages == 4 and torch.equal(other.k_pages, cache.k_pages)


class Library:
    """Answers as the library does to a workspace that is too small for `need` bytes."""

    def __init__(self, need, log):
        self.need, self.log = need, log

    def dg_paged_attn_workspace_bytes(self, *sizes):
        return self.need

    def dg_paged_attn_e4m3(self, *args):
        pointer, size = args[-3:-1]
        self.log.append(("call", size))
        return 4 if not pointer or size < self.need else 0


def test_a_workspace_grows_on_the_calls_stream(monkeypatch):
    """Its memory belongs to the stream that the kernels run on, and the memory that it replaces is
    kept from other use until that stream has passed it."""
    log = []

    class Stream:
        cuda_stream = 7

    class Buffer:  # the workspace's earlier memory
        def get_device(self):
            return -1

        def data_ptr(self):
            return 4096

        def numel(self):
            return 300

        def record_stream(self, stream):
            log.append(("keep for", stream))

    @contextlib.contextmanager
    def on(stream):
        log.append(("enter", stream))
        yield
        log.append(("leave", stream))

    class Workspace(dg.Workspace):
        def get(self, nbytes):
            log.append(("allocate", nbytes))
            return super().get(nbytes)

    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: "current")
    monkeypatch.setattr(dg, "_ptr", lambda t: t.data_ptr())
    monkeypatch.setattr(dg, "_paged_batch", lambda *a: (1, 2, 3, 1, 4, -1))
    monkeypatch.setattr(_lib, "load", lambda: Library(1000, log))
    cache = dg.PagedCache(*tensors(4))
    q = torch.zeros((1, 128), dtype=torch.bfloat16)
    side, ws = Stream(), Workspace("cpu")
    ws.buf = Buffer()

    def call():
        dg.paged_attn_e4m3(q, cache, None, None, None, 1, 64, q, n_q_heads=2, ws=ws, stream=side)

    call()
    assert ("keep for", "current") in log  # the current stream within the block: the call's
    assert [e for e in log if e[0] != "keep for"] == [
        ("call", 300), ("enter", side), ("allocate", 1000), ("leave", side), ("call", 1000)]
    assert log.index(("enter", side)) < log.index(("keep for", "current")) < log.index(("allocate", 1000))
    log.clear()
    call()  # large enough now: one call, nothing else
    assert log == [("call", 1000)]


def no_gpu(monkeypatch, library):
    """The calls' own checks and marshalling, on CPU tensors."""
    monkeypatch.setattr(dg, "_paged_batch", lambda *a: (1, 2, 3, 1, 4, -1))
    monkeypatch.setattr(dg, "_raw_stream", lambda stream, dev: 0)
    monkeypatch.setattr(_lib, "load", lambda: library)
    return dg.PagedCache(*tensors(4)), torch.zeros((3, 128), dtype=torch.bfloat16)


@pytest.mark.parametrize("grown", [False, True])
def test_a_workspace_on_another_device_is_refused(monkeypatch, grown):
    log = []
    cache, q = no_gpu(monkeypatch, Library(1000, log))

    class Elsewhere:
        def get_device(self):
            return 1

        def data_ptr(self):
            return 4096

        def numel(self):
            return 2000

    class Workspace(dg.Workspace):
        def get(self, nbytes):
            self.buf = Elsewhere()
            return self.buf

    ws = Workspace("cuda:1")
    if grown:
        ws.get(2000)
    with pytest.raises(ValueError, match="device"):
        dg.paged_attn_e4m3(q, cache, None, None, None, 1, 64, q, n_q_heads=2, ws=ws)
    assert all(size == 0 for _, size in log)  # its pointer was not handed over


class Recorder:
    def __init__(self):
        self.args = {}

    def __getattr__(self, name):
        def call(*args):
            self.args[name] = args
            return 0
        return call


@pytest.mark.parametrize("bound", [3, 64, (1 << 31) - 1, 1 << 32, (1 << 40) + 3])
def test_bounds_past_32_bits_stay_bounds(monkeypatch, bound):
    """A bound on the new rows counts up to T, one on the cached rows up to the table's positions: a
    larger one must not wrap around (to no rows, say, and a call that does nothing)."""
    library = Recorder()
    cache, q = no_gpu(monkeypatch, library)
    kv = torch.zeros((3, 128), dtype=torch.bfloat16)
    dg.kv_append_e4m3(kv, kv, cache, None, None, None, bound)
    dg.paged_attn_e4m3(q, cache, None, None, None, bound, bound, q, n_q_heads=2)
    append, attn = library.args["dg_kv_append_e4m3"], library.args["dg_paged_attn_e4m3"]
    query = library.args["dg_paged_attn_workspace_bytes"]
    positions = 4 * 16  # of the table that no_gpu stands for
    assert append[-6] == 3  # max_new
    assert attn[12:14] == (3, min(bound, positions))
    assert query[-2:] == (3, min(bound, positions))
