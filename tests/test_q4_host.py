"""Refusals of the rotary, paged-append and 4-bit KV entry points (no GPU):
every bad argument is named before any device work, and the binding checks
buffers before a pointer reaches the library."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest

torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = ctypes.c_void_p(1 << 20)          # never dereferenced: validation fails first
ODD = ctypes.c_void_p((1 << 20) + 4)
INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3


@pytest.fixture(scope="module")
def d():
    from session_decode_step_dsb_gb300 import build, dsb
    if not os.path.exists(dsb.LIB_PATH):
        build.build()
    dsb.lib()
    return dsb


def _pages(d, n_pages=8, heads=2, dim=64, blocks=FAKE):
    return d.KVQ4Pages(blocks, n_pages, heads, dim)


def _batch(d, **kw):
    a = dict(block_table=[[0, 1], [2, 3]], n_blocks=[2, 2], window=[0, 0], new_tokens=[1, 2], seq_lens=[130, 2])
    a.update(kw)
    return d.PagedBatch(**a)


BAD_BATCHES = [
    (dict(seq_lens=[257, 2]), "do not cover"),
    (dict(seq_lens=[130, 1]), "new_tokens"),
    (dict(seq_lens=[-1, 2]), "seq_lens"),
    (dict(new_tokens=[-1, 2]), "new_tokens"),
    (dict(block_table=[[0, 8], [2, 3]]), "block_table"),
    (dict(block_table=[[0, 1], [-1, 3]]), "block_table"),
    (dict(n_blocks=[3, 2]), "n_blocks"),
    (dict(n_blocks=[-1, 2]), "n_blocks"),
    (dict(window=[-1, 0]), "window"),
    (dict(window=[0, 256]), "ring"),                       # 256 + 2 - 1 keys in two pages
    (dict(new_tokens=[8000, 8000], seq_lens=[8000, 8000], n_blocks=[63, 63], block_table=[[0] * 63] * 2), "exceed"),
]


@pytest.mark.parametrize("change,word", BAD_BATCHES)
def test_bad_batches_are_named(d, change, word):
    lib, kv, b = d.lib(), _pages(d), _batch(d, **change)
    rot, z = d.Rotary(), np.zeros(2, np.int32)
    pz = z.ctypes.data_as(ctypes.POINTER(ctypes.c_int32))
    calls = [lambda: lib.dsb_kv_append_q4(FAKE, 512, 4, ctypes.byref(kv), b.ref, rot.ref, None, None, 0.0, FAKE, None),
             lambda: lib.dsb_attention_decode_q4(FAKE, 256, 4, ctypes.byref(kv), b.ref, FAKE, FAKE, None),
             lambda: lib.dsb_kv_gather_q4(ctypes.byref(kv), b.ref, pz, pz, 0, FAKE, FAKE, FAKE, None)]
    kp = d.KVPages(FAKE, FAKE, 0, 8, 2, 64)
    calls.append(lambda: lib.dsb_kv_append_paged(FAKE, 512, 4, ctypes.byref(kp), b.ref, rot.ref, None, None, 0.0, FAKE,
                                                 None))
    for call in calls:
        assert call() == INVALID
        assert word in lib.dsb_last_error().decode()


def test_appends_refuse_two_tokens_on_one_row(d):
    lib, kv, rot = d.lib(), _pages(d), d.Rotary()
    for b in (_batch(d, block_table=[[0, 1], [1, 3]]),                   # page 1 row 1 (key 129), rows 0..1
              _batch(d, block_table=[[0, 0], [2, 3]], new_tokens=[130, 2])):   # one page twice in a table
        assert lib.dsb_kv_append_q4(FAKE, 512, 4, ctypes.byref(kv), b.ref, rot.ref, None, None, 0.0, FAKE, None) == INVALID
        assert "two tokens" in lib.dsb_last_error().decode()


@pytest.mark.parametrize("kw", [
    dict(theta=0.0), dict(theta=float("nan")), dict(rotary_dim=3), dict(rotary_dim=66), dict(rotary_dim=-2),
    dict(scaling="linear", factor=0.5), dict(scaling="linear", factor=float("inf")),
    dict(scaling="ntk", factor=2.0, rotary_dim=2), dict(scaling="bands", factor=2.0, orig_ctx=0, low=1, high=4),
    dict(scaling="bands", factor=2.0, orig_ctx=10, low=4, high=4), dict(scaling="bands", factor=2.0, orig_ctx=10, high=4)])
def test_bad_rotations_are_refused(d, kw):
    lib, kv, b, rot = d.lib(), _pages(d), _batch(d), d.Rotary(**kw)
    pos = np.zeros(1, np.int32)
    pp = pos.ctypes.data_as(ctypes.POINTER(ctypes.c_int32))
    assert lib.dsb_rope_rotary(FAKE, 64, 1, None, 0, 0, 64, 1, pp, rot.ref, FAKE, None) == INVALID
    assert lib.dsb_kv_append_q4(FAKE, 512, 4, ctypes.byref(kv), b.ref, rot.ref, None, None, 0.0, FAKE, None) == INVALID


def test_yarn_excludes_the_other_scalings(d):
    rot = d.Rotary(scaling="linear", factor=2.0, yarn=d.Yarn(4.0, 4096))
    pos = np.zeros(1, np.int32)
    pp = pos.ctypes.data_as(ctypes.POINTER(ctypes.c_int32))
    assert d.lib().dsb_rope_rotary(FAKE, 64, 1, None, 0, 0, 64, 1, pp, rot.ref, FAKE, None) == INVALID
    with pytest.raises(ValueError, match="scaling"):
        d.Rotary(scaling="cubic")


def test_rope_rotary_refusals(d):
    lib, rot = d.lib(), d.Rotary()
    pos = np.zeros(2, np.int32)
    pp = pos.ctypes.data_as(ctypes.POINTER(ctypes.c_int32))

    def call(q=FAKE, qs=128, hq=2, k=FAKE, ks=64, hkv=1, dim=64, n=2, p=pp, ws=FAKE):
        return lib.dsb_rope_rotary(q, qs, hq, k, ks, hkv, dim, n, p, rot.ref, ws, None)

    assert call(n=-1) == INVALID and call(n=8193) == INVALID
    assert call(dim=63) == INVALID and call(dim=1026, qs=4096, ks=4096) == INVALID
    assert call(hq=0) == INVALID and call(hkv=0) == INVALID and call(k=None) == INVALID
    assert call(qs=127) == INVALID and call(ks=63) == INVALID
    assert call(q=None) == INVALID and call(q=ODD) == INVALID and call(k=ODD) == INVALID and call(p=None) == INVALID
    assert call(ws=None) == WORKSPACE
    for bad in (-1, 1 << 24):
        pos[1] = bad
        assert call() == INVALID and "pos[1]" in lib.dsb_last_error().decode()
    assert call(n=0) == 0


def test_pool_and_buffer_refusals(d):
    lib, b, rot = d.lib(), _batch(d), d.Rotary()
    for kv, want in ((_pages(d, blocks=None), INVALID), (_pages(d, blocks=ODD), INVALID), (_pages(d, n_pages=0), INVALID),
                     (_pages(d, heads=0), INVALID), (_pages(d, dim=96), UNSUPPORTED),
                     (_pages(d, n_pages=1 << 20, heads=1 << 15), UNSUPPORTED)):
        assert lib.dsb_attention_decode_q4(FAKE, 512, 4, ctypes.byref(kv), b.ref, FAKE, FAKE, None) == want
        assert lib.dsb_kv_append_q4(FAKE, 512, 4, ctypes.byref(kv), b.ref, rot.ref, None, None, 0.0, FAKE, None) == want
    kv = _pages(d)

    def attn(q=FAKE, stride=256, hq=4, out=FAKE, ws=FAKE, batch=b):
        return lib.dsb_attention_decode_q4(q, stride, hq, ctypes.byref(kv), batch.ref, out, ws, None)

    assert attn(hq=3) == INVALID and attn(hq=0) == INVALID and attn(stride=255) == INVALID and attn(stride=258) == INVALID
    assert attn(q=None) == INVALID and attn(q=ODD) == INVALID and attn(out=None) == INVALID and attn(out=ODD) == INVALID
    assert attn(ws=None) == WORKSPACE
    none = _batch(d, new_tokens=[0, 0])
    assert attn(batch=none, q=None, out=None) == 0            # no rows: nothing to do

    def app(qkv=FAKE, stride=512, hq=4, eps=0.0, qn=None, kn=None, ws=FAKE, batch=b):
        return lib.dsb_kv_append_q4(qkv, stride, hq, ctypes.byref(kv), batch.ref, rot.ref, qn, kn, eps, ws, None)

    assert app(hq=-1) == INVALID and app(stride=508) == INVALID and app(stride=514) == INVALID
    assert app(eps=-1.0) == INVALID and app(eps=float("nan")) == INVALID and app(qn=ODD) == INVALID and app(kn=ODD) == INVALID
    assert app(qkv=None) == INVALID and app(qkv=ODD) == INVALID and app(ws=None) == WORKSPACE
    assert app(batch=none, qkv=None) == 0

    def gather(first, count, dtype=0, k=FAKE, v=FAKE, ws=FAKE, batch=b):
        f, c = np.array(first, np.int32), np.array(count, np.int32)
        p = [a.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)) for a in (f, c)]
        return lib.dsb_kv_gather_q4(ctypes.byref(kv), batch.ref, p[0], p[1], dtype, k, v, ws, None)

    assert gather([0, 0], [131, 0]) == INVALID and gather([-1, 0], [1, 0]) == INVALID and gather([0, 0], [-1, 0]) == INVALID
    assert gather([0, 0], [1, 0], dtype=2) == INVALID and gather([0, 0], [1, 0], k=None) == INVALID
    assert gather([0, 0], [1, 0], v=ODD) == INVALID and gather([0, 0], [1, 0], ws=None) == WORKSPACE
    assert gather([0, 0], [0, 0], k=None, v=None) == 0
    ring = _batch(d, window=[100, 0], seq_lens=[1000, 2])
    assert gather([743, 0], [10, 0], batch=ring) == INVALID and "ring" in lib.dsb_last_error().decode()


def test_memory_shared_between_arguments_is_refused(d):
    """Before any device work: the workspace is not looked at either."""
    lib, b, rot, kv = d.lib(), _batch(d), d.Rotary(), _pages(d)
    base = 1 << 20
    ws = ctypes.create_string_buffer(4096)          # stands for a workspace: only its size is read
    pos = np.arange(3, dtype=np.int32)
    pp = pos.ctypes.data_as(ctypes.POINTER(ctypes.c_int32))

    def rope(k, qs, ks, n=3):
        st = lib.dsb_rope_rotary(base, qs, 2, k, ks, 1, 64, n, pp, rot.ref, ws, None)
        return st, lib.dsb_last_error().decode()

    for k, qs, ks in ((base, 128, 64), (base, 192, 192), (base + 4 * 64, 192, 192), (base + 4 * 160, 192, 192),
                      (base + 4 * 128, 192, 256), (base - 4 * 32, 128, 64)):
        st, why = rope(k, qs, ks)
        assert st == INVALID and "share" in why, (k - base, qs, ks)
    st, why = rope(base, 128, 64, 1)
    assert st == INVALID and "share" in why

    def gather(k, v):
        f, c = np.array([0, 0], np.int32), np.array([100, 2], np.int32)
        p = [a.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)) for a in (f, c)]
        return lib.dsb_kv_gather_q4(ctypes.byref(kv), b.ref, p[0], p[1], 0, k, v, ws, None), lib.dsb_last_error().decode()

    for v in (base, base + 102 * 2 * 64 * 2 - 16, base - 102 * 2 * 64 * 2 + 16):
        st, why = gather(base, v)
        assert st == INVALID and "overlap" in why

    def attn(out, stride=256):
        return (lib.dsb_attention_decode_q4(base, stride, 4, ctypes.byref(kv), b.ref, out, ws, None),
                lib.dsb_last_error().decode())

    for out, stride in ((base, 256), (base + 4 * 256 * 3 - 16, 256), (base - 4 * 256 * 3 + 16, 256), (base + 4 * 300, 512)):
        st, why = attn(out, stride)
        assert st == INVALID and "overlap" in why


def test_a_block_table_past_the_staging_slot_is_refused(d):
    kv = _pages(d)
    b = d.PagedBatch(np.zeros((1, 12000)), [12000], [0], [1], [12000 * 128])
    assert d.lib().dsb_attention_decode_q4(FAKE, 128, 2, ctypes.byref(kv), b.ref, FAKE, FAKE, None) == UNSUPPORTED


def test_binding_checks_buffers(d):
    with pytest.raises(ValueError, match="new_tokens has 1"):
        d.PagedBatch([[0], [1]], [1, 1], [0, 0], [1], [1, 1])
    with pytest.raises(ValueError, match="block_table"):
        d.PagedBatch([0, 1], [1], [0], [1], [1])
    with pytest.raises(ValueError, match="uint8"):
        d.kv_q4_pages(torch.zeros((2, 2, 128 * 72), dtype=torch.int8), 64)
    with pytest.raises(ValueError, match="pool must be"):
        d.kv_q4_pages(torch.zeros((2, 2, 128 * 71), dtype=torch.uint8), 64)
    kv = _pages(d)
    kv._tensors = (torch.zeros((8, 2, 128 * 72), dtype=torch.uint8),)
    b, rot = _batch(d), d.Rotary()
    with pytest.raises(ValueError, match="qkv must be 3 rows"):
        d.kv_append_q4(torch.zeros((2, 512)), 4, kv, b, rot, None)
    with pytest.raises(ValueError, match="contiguous"):
        d.kv_append_q4(torch.zeros((3, 1024))[:, ::2], 4, kv, b, rot, None)
    with pytest.raises(ValueError, match="float32"):
        d.attention_decode_q4(torch.zeros((3, 4, 64), dtype=torch.float16), kv, b, None)
    with pytest.raises(ValueError, match="q must be"):
        d.attention_decode_q4(torch.zeros((3, 4, 32)), kv, b, None)
    with pytest.raises(ValueError, match="CUDA device"):
        d.attention_decode_q4(torch.zeros((3, 4, 64)), kv, b, None)
    with pytest.raises(ValueError, match="pos has 2"):
        d.rope_rotary(torch.zeros((3, 4, 64)), None, [0, 1], rot, None)
    with pytest.raises(ValueError, match="k \\[n_tok"):
        d.rope_rotary(torch.zeros((3, 4, 64)), torch.zeros((2, 4, 64)), [0, 1, 2], rot, None)


def test_page_bytes(d):
    assert d.kv_q4_page_bytes(8, 128) == 8 * 128 * 136 and d.kv_q4_page_bytes(2, 64) == 2 * 128 * 72
    assert d.kv_q4_page_bytes(0, 64) == 0 and d.kv_q4_page_bytes(1, 80) == 0


def test_struct_layouts_match_the_header(d, tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    structs = {"dsb_rotary": d.RotaryC, "dsb_kv_q4_pages": d.KVQ4Pages, "dsb_paged_batch": d.PagedBatchC}
    lines = ["#include <stddef.h>", "#include <stdio.h>", '#include "dsb.h"', "int main(void) {"]
    for name, cls in structs.items():
        lines.append(f'  printf("{name} size %zu\\n", sizeof({name}));')
        lines += [f'  printf("{name} {f} %zu\\n", offsetof({name}, {f}));' for f, _ in cls._fields_]
    lines += [f'  printf("scaling {i} %d\\n", (int){m});' for i, m in
              enumerate(("DSB_ROPE_UNSCALED", "DSB_ROPE_LINEAR", "DSB_ROPE_NTK", "DSB_ROPE_BANDS"))]
    lines += ["  return 0;", "}"]
    src, exe = tmp_path / "l.c", tmp_path / "l"
    src.write_text("\n".join(lines))
    subprocess.run([cc, "-std=c99", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)],
                   check=True, capture_output=True)
    for line in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.splitlines():
        name, field, v = line.split()
        if name == "scaling":
            assert list(d.ROPE_SCALINGS.values())[int(field)] == int(v)
        elif field == "size":
            assert ctypes.sizeof(structs[name]) == int(v)
        else:
            assert getattr(structs[name], field).offset == int(v)
