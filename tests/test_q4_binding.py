"""Host-only checks of the binding of the rotary, paged-append and 4-bit KV calls
(no GPU): what reaches the library is what the caller passed."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")


def _dsb():
    from session_decode_step_dsb_gb300 import dsb
    return dsb


BATCH = dict(block_table=[[0, 1], [2, 3]], n_blocks=[2, 2], window=[0, 0], new_tokens=[1, 2], seq_lens=[130, 2])
BAD = [np.array([(1 << 32) + 1, 2]), np.array([1, -(1 << 32) + 2]), np.array([1, 1 << 31], np.uint32), [1, (1 << 31)],
       np.array([1.5, 2.0]), np.array([1.0, np.nan]), np.array([1.0, np.inf]), ["1", "2"]]


@pytest.mark.parametrize("bad", BAD)
@pytest.mark.parametrize("name", list(BATCH))
def test_batches_take_only_what_int32_holds(name, bad):
    d = _dsb()
    value = [bad, bad] if name == "block_table" else bad
    with pytest.raises(ValueError, match=name):
        d.PagedBatch(**{**BATCH, name: value})


@pytest.mark.parametrize("bad", BAD)
def test_positions_and_spans_take_only_what_int32_holds(bad):
    d = _dsb()
    with pytest.raises(ValueError, match="pos must hold"):
        d.rope_rotary(torch.zeros((2, 4, 64)), None, bad, d.Rotary(), None)
    kv = d.KVQ4Pages(1 << 20, 8, 2, 64)
    kv._tensors = (torch.zeros((8, 2, 128 * 72), dtype=torch.uint8),)
    batch = d.PagedBatch(**BATCH)
    with pytest.raises(ValueError, match="first must hold"):
        d.kv_gather_q4(kv, batch, bad, [1, 1], d.DSB_F16, None)
    with pytest.raises(ValueError, match="count must hold"):
        d.kv_gather_q4(kv, batch, [0, 0], bad, d.DSB_F16, None)


@pytest.mark.parametrize("kind", [np.int8, np.uint8, np.int16, np.int64, np.uint64, np.float32, np.float64, bool, list])
def test_whole_numbers_of_any_type_arrive(kind):
    """And as a copy: the batch is not the caller's array."""
    d = _dsb()
    arrays = {k: np.array(v) for k, v in BATCH.items()}
    arrays["new_tokens"] = [1, 0] if kind is list else np.array([1, 0]).astype(kind)
    b = d.PagedBatch(**arrays)
    assert [b.c.new_tokens[i] for i in range(2)] == [1, 0] and [b.c.seq_lens[i] for i in range(2)] == [130, 2]
    own = np.array([1, 2], np.int32)
    b = d.PagedBatch(**{**BATCH, "new_tokens": own})
    own[:] = 9
    assert [b.c.new_tokens[i] for i in range(2)] == [1, 2]
    arr, at = d._host_i32(own, 2, "x")
    assert arr is own and at == own.ctypes.data
    assert d._host_i32(np.array([3, 4, 5, 6])[::2], 2, "x")[0].tolist() == [3, 5]


def test_what_a_call_makes_belongs_to_its_stream(monkeypatch):
    """The handle 0 is the default stream's; other handles are wrapped, streams
    taken as they are."""
    import contextlib
    d, entered = _dsb(), []

    class Stream:
        def __init__(self, name):
            self.name = name

    @contextlib.contextmanager
    def on(stream):
        entered.append(stream.name)
        yield

    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device: Stream(("handle", handle, device)))
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device: Stream(("default", device)))
    monkeypatch.setattr(torch.cuda, "stream", on)
    for stream in (0, 77, Stream("given"), None):
        assert d._empty_on(stream, (2, 3), torch.float32, "cpu").shape == (2, 3)
    assert entered == [("default", "cpu"), ("handle", 77, "cpu"), "given"]


def _lib():
    import os
    from session_decode_step_dsb_gb300 import build
    d = _dsb()
    if not os.path.exists(d.LIB_PATH):
        build.build()
    return d, d.lib()


def test_memory_that_a_call_reads_and_writes_is_apart():
    """Before any device work.  The workspace is a stand-in that belongs to no device:
    a call that passed these checks would be refused for that."""
    import ctypes
    d, lib = _lib()
    ws, rot, b = ctypes.create_string_buffer(b"\xff" * 4096), d.Rotary(), d.PagedBatch(**BATCH)
    hq, hkv, D, n, pages, mb = 4, 2, 64, 3, 8, 1 << 20
    width, pool = (hq + 2 * hkv) * D * 4, pages * hkv * 128 * (D + 8)
    pool16 = pages * hkv * 128 * D * 2

    def said(st):
        assert st == d.DSB_ERR_INVALID_ARG
        return lib.dsb_last_error().decode()

    def append(k, v, qkv, stride=width // 4, qn=None, kn=None):
        if v is None:
            kv, fn = d.KVQ4Pages(k, pages, hkv, D), lib.dsb_kv_append_q4
        else:
            kv, fn = d.KVPages(k, v, 0, pages, hkv, D), lib.dsb_kv_append_paged
        return said(fn(qkv, stride, hq, ctypes.byref(kv), b.ref, rot.ref, qn, kn, 1e-6, ws, None))

    for v in (mb, mb + pool16 - 16, mb - pool16 + 16):
        assert append(mb, v, 64 * mb) == "the pools of K and V overlap"
    for k, v, end in ((mb, None, mb + pool), (mb, 16 * mb, mb + pool16), (16 * mb, mb, mb + pool16)):
        for qkv in (mb, end - 16, mb - n * width + 16):
            assert append(k, v, qkv) == "qkv and a page pool overlap"
    rows = 64 * mb
    for w in (rows, rows + 2 * width + 16, rows + width - 16, rows - D * 4 + 16):
        assert append(mb, None, rows, qn=w) == "qkv and the weights of a norm overlap"
        assert append(mb, 16 * mb, rows, kn=w) == "qkv and the weights of a norm overlap"
    # between rows that lie far apart, at the last byte that a row leaves free
    wide = width // 4 + D
    assert append(mb, None, rows, stride=wide, qn=rows + width + 16) == "qkv and the weights of a norm overlap"
    assert lib.dsb_kv_append_q4(rows, wide, hq, ctypes.byref(d.KVQ4Pages(mb, pages, hkv, D)), b.ref, rot.ref, rows + width,
                                None, 1e-6, ws, None) != d.DSB_OK
    assert "overlap" not in lib.dsb_last_error().decode()

    kv = d.KVQ4Pages(mb, pages, hkv, D)
    out = n * hq * D * 4
    for o in (mb, mb + pool - 16, mb - out + 16):
        assert said(lib.dsb_attention_decode_q4(rows, hq * D, hq, ctypes.byref(kv), b.ref, o, ws, None)) == \
            "out overlaps the page pool"
    f, c = np.array([0, 0], np.int32), np.array([100, 2], np.int32)
    each = 102 * hkv * D * 2
    for o in (mb, mb + pool - 16, mb - each + 16):
        for k, v in ((o, rows), (rows, o)):
            assert said(lib.dsb_kv_gather_q4(ctypes.byref(kv), b.ref, f.ctypes.data, c.ctypes.data, 0, k, v, ws, None)) == \
                "k_out / v_out and the page pool overlap"


PROGRAM = r"""
#include <cstdio>
#include <cstdlib>
#include <new>
#include "dsb_host.h"
static bool none = false;
void* operator new(std::size_t n) {
  if (none) throw std::bad_alloc();
  if (void* p = std::malloc(n)) return p;
  throw std::bad_alloc();
}
void operator delete(void* p) noexcept { std::free(p); }
void operator delete(void* p, std::size_t) noexcept { std::free(p); }
int main() {
  none = true;
  dsb_status st = dsbh::fail(DSB_ERR_INVALID_ARG, "%s", "a message that is longer than a string holds without memory");
  none = false;
  std::printf("%d [%s]\n", (int)st, dsbh::g_last_error.c_str());
  st = dsbh::fail(DSB_ERR_WORKSPACE, "%s", "a message that is longer than a string holds without memory");
  std::printf("%d %zu\n", (int)st, dsbh::g_last_error.size());
}
"""


def test_an_error_without_memory_for_its_message_is_still_a_status(tmp_path):
    import os
    import shutil
    import subprocess
    from session_decode_step_dsb_gb300 import build
    cxx, cuda = shutil.which("g++"), os.path.join(os.path.dirname(os.path.dirname(build._nvcc())), "include")
    if cxx is None or not os.path.exists(os.path.join(cuda, "cuda_runtime.h")):
        pytest.skip("no host compiler or CUDA headers")
    src, exe = tmp_path / "m.cpp", tmp_path / "m"
    src.write_text(PROGRAM)
    subprocess.run([cxx, "-std=c++17", "-O1", "-I", build.INCLUDE, "-I", build.CSRC, "-I", cuda, str(src), "-o", str(exe),
                    "-lpthread"], check=True, capture_output=True)
    got = subprocess.run([str(exe)], capture_output=True, text=True)
    assert got.returncode == 0 and got.stdout.splitlines() == ["1 []", "3 59"]
