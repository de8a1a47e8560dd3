"""Host checks of the paged KV cache's entry points (CPU only: no call here reaches a CUDA launch)."""
import ctypes
import os
import subprocess
import sys

import pytest

from bit_compressed_decode_b200 import _binding as B

INVALID, SHAPE, UNSUPPORTED, WORKSPACE = 1, 2, 3, 7
P = 0x800000                                                # aligned, never dereferenced


def cache(**o):
    kv = B.fg_paged_kv()
    for i, (name, _) in enumerate(B.fg_paged_kv._fields_[:9]):
        setattr(kv, name, 0x100000 * (i + 1))
    d = dict(num_pages=8, page_size=64, num_seqs=4, max_pages=2, num_heads=2, head_dim=128, group=64)
    for k, v in (d | o).items():
        setattr(kv, k, v)
    return kv


def append(kv=None, **o):
    d = dict(k=P, v=P + 512, ld=768, rows=4, per=1, pos=P * 3, counts=None, first=None) | o
    return B.lib().fg_paged_kv_append(ctypes.byref(kv or cache()), d["k"], d["v"], d["ld"], d["rows"], d["per"],
                                      d["pos"], d["counts"], d["first"], None)


def attend(kv=None, **o):
    d = dict(q=P, ldq=512, heads=4, out=P * 2, ldo=512, rows=4, per=1, pos=P * 3, counts=None, max_len=0, acc=0, ws=None,
             nbytes=0) | o
    return B.lib().fg_paged_attention(ctypes.byref(kv or cache()), d["q"], d["ldq"], d["heads"], d["out"], d["ldo"],
                                      d["rows"], d["per"], d["pos"], d["counts"], d["max_len"], d["acc"], d["ws"],
                                      d["nbytes"], None)


def evict(kv=None, **o):
    d = dict(lengths=P, next=P * 2, budget=32, recent=8, max_len=0, new=P * 3, wout=None, tout=None, ws=None, nbytes=0) | o
    return B.lib().fg_paged_kv_evict(ctypes.byref(kv or cache()), d["lengths"], d["next"], d["budget"], d["recent"],
                                     d["max_len"], d["new"], d["wout"], d["tout"], d["ws"], d["nbytes"], None)


BAD_CACHES = [
    (dict(num_pages=0), INVALID), (dict(max_pages=0), INVALID), (dict(num_seqs=-1), INVALID), (dict(num_heads=0), INVALID),
    (dict(page_size=0), INVALID), (dict(page_size=40), SHAPE), (dict(head_dim=96), UNSUPPORTED),
    (dict(group=32), UNSUPPORTED), (dict(head_dim=64, group=128), SHAPE), (dict(k_codes=None), INVALID),
    (dict(v_scales=None), INVALID), (dict(page_table=None), INVALID), (dict(k_codes=0x100008), INVALID),
    (dict(v_mins=0x100008), INVALID), (dict(page_table=0x100002), INVALID), (dict(weights=0x100002), INVALID),
    (dict(tokens=0x100001), INVALID), (dict(max_pages=1 << 27), SHAPE), (dict(max_pages=(1 << 24) + 1), SHAPE),
]


@pytest.mark.parametrize("change,code", BAD_CACHES, ids=[str(c) for c, _ in BAD_CACHES])
def test_bad_caches_are_refused(change, code):
    for call in (append, attend, evict):
        assert call(cache(**change)) == code


def test_sizes():
    cb, mb, tb = ctypes.c_size_t(), ctypes.c_size_t(), ctypes.c_size_t()
    f = lambda *a: B.lib().fg_paged_kv_bytes(*a, ctypes.byref(cb), ctypes.byref(mb), ctypes.byref(tb))
    assert f(10, 3, 128, 48, 0) == 0
    assert (cb.value, mb.value, tb.value) == (10 * 3 * 48 * 64, 10 * 3 * 48 * 4, 10 * 3 * 48 * 4)
    assert f(70000, 96, 256, 256, 128) == 0
    assert (cb.value, mb.value) == (70000 * 96 * 256 * 128, 70000 * 96 * 256 * 4)      # past 32 bits
    assert f(0, 3, 128, 48, 64) == INVALID and f(1, 3, 128, 24, 64) == SHAPE and f(1, 3, 80, 48, 64) == UNSUPPORTED
    assert f(1, 3, 64, 48, 128) == SHAPE and f(1, 3, 64, 48, 65) == UNSUPPORTED


def test_append_refusals():
    assert append(rows=0) == 0                                         # nothing to do
    assert append(rows=-1) == SHAPE and append(rows=5) == SHAPE and append(rows=4, per=3) == SHAPE
    assert append(per=0) == SHAPE
    assert append(k=None) == INVALID and append(v=None) == INVALID and append(pos=None) == INVALID
    assert append(k=P + 8) == INVALID and append(v=P + 2) == INVALID
    assert append(ld=255) == SHAPE and append(ld=260) == SHAPE


def test_attention_refusals():
    assert attend(rows=0) == 0
    assert attend(rows=-1) == SHAPE and attend(rows=5) == SHAPE and attend(rows=4, per=3) == SHAPE and attend(per=0) == SHAPE
    assert attend(heads=3) == SHAPE and attend(heads=0) == SHAPE and attend(heads=-2) == SHAPE
    assert attend(q=None) == INVALID and attend(out=None) == INVALID and attend(pos=None) == INVALID
    assert attend(q=P + 8) == INVALID and attend(out=P + 2) == INVALID and attend(ws=P + 4) == INVALID
    assert attend(ldq=504) == SHAPE and attend(ldo=516) == SHAPE
    assert attend(max_len=-1) == INVALID and attend(acc=2) == INVALID
    assert attend(cache(weights=None), acc=1) == INVALID               # nothing to accumulate in


def test_evict_refusals():
    assert evict(cache(num_seqs=0)) == 0
    assert evict(cache(weights=None)) == INVALID and evict(cache(tokens=None)) == INVALID
    assert evict(budget=0) == INVALID and evict(recent=-1) == INVALID and evict(recent=33) == INVALID
    assert evict(max_len=-1) == INVALID
    assert evict(lengths=None) == INVALID and evict(next=None) == INVALID and evict(new=None) == INVALID
    assert evict(wout=P + 2) == INVALID and evict(tout=P + 1) == INVALID and evict(ws=P + 8) == INVALID


def test_evict_refuses_lengths_that_are_written_while_they_are_read():
    for new in (P * 2, P * 2 + 12, P * 2 - 12, P + 4, P - 4):           # next_tokens, or part of an input
        assert evict(new=new) == INVALID
    for clear in (dict(new=P * 2 + 16), dict(new=P * 2 - 16), dict(new=P), dict(new=P, next=P)):
        assert evict(**clear, ws=P + 8) == INVALID                      # (refused for its workspace alone:)
        assert evict(kv=cache(page_size=1 << 20), **clear) == WORKSPACE # beside, or the lengths in place


def test_import_without_torch_internals():
    """A torch built without CUDA has neither name; the package imports there and its host checks answer."""
    code = """
import torch
for name in ("_cuda_getDevice", "_cuda_getCurrentRawStream"):
    if hasattr(torch._C, name):
        delattr(torch._C, name)
import bit_compressed_decode_b200 as fg
try:
    fg.PagedKVCache(4, 2, 128, 16, torch.zeros((1, 4), dtype=torch.int32))
except ValueError as e:
    assert "page_table" in str(e)
else:
    raise SystemExit("a table on the CPU was taken")
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
