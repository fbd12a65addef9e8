"""Host side of the calls around the decode step (packed prompts, shared prefixes, shared
pages): sizes, argument and shape rules, which answer before any device work.  No GPU is
needed, and no call here enqueues anything."""
import ctypes
import os
import subprocess

import pytest
import torch

import dynamic_sparse_attention_block_b200 as prr
from dynamic_sparse_attention_block_b200 import _abi, build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, SHAPE, CAPACITY = 0, 1, 2, 3
BIG = 1 << 60  # workspace bytes: not the limiting check


@pytest.fixture(scope="module")
def lib():
    build.build(verbose=False)
    return _abi.load()


def _dims(**kw):
    base = dict(B=3, Hq=8, Hkv=2, d=128, bs=64, cap_tokens=4096, K=8, P=4)
    base.update(kw)
    return _abi.Dims(**base)


def _paged(**kw):
    return _dims(pages=50, block_table=1 << 24, **kw)


def _cache(**kw):
    names = [n for n, _ in _abi.PrrCacheBuffers._fields_]
    vals = {n: (1 << 24) * (i + 20) for i, n in enumerate(names)}
    vals["block_table"] = 1 << 24
    vals.update(kw)
    return _abi.PrrCacheBuffers(*[vals[n] for n in names])


def _call(lib, fn, dims, **kw):
    """The call with plausible, never-dereferenced addresses; kw replaces arguments by name."""
    order = {
        "prr_append_prompt": ["k_rows", "v_rows", "stride", "q_begin", "rows", "seq_lens", "k_cache", "v_cache", "summ"],
        "prr_attend_prompt": ["q", "stride", "q_begin", "rows", "seq_lens", "k_cache", "v_cache", "out", "lse"],
        "prr_attend_shared": ["q", "stride", "members", "n_members", "group_begin", "shared_blocks", "n_groups", "seq_lens",
                              "k_cache", "v_cache", "out", "lse"],
        "prr_cache_reserve": ["want", "cache"], "prr_cache_fork": ["parents", "children", "n", "cache"],
        "prr_cache_release": ["seqs", "n", "cache"], "prr_cache_compact": ["cache", "remap", "n_live"],
    }[fn]
    vals = {n: (1 << 20) * (i + 1) for i, n in enumerate(order)}
    vals.update(rows=10, n=2, n_members=3, n_groups=1, ws=1 << 30, ws_bytes=BIG,
                stride=(dims.Hkv if "append" in fn else dims.Hq) * dims.d, cache=_cache())
    vals.update(kw)
    c = dims.c()
    args = [ctypes.byref(vals[n]) if isinstance(vals[n], ctypes.Structure) else vals[n] for n in order]
    return getattr(lib, fn)(ctypes.byref(c), *args, vals["ws"], vals["ws_bytes"], None)


ALL = ["prr_append_prompt", "prr_attend_prompt", "prr_attend_shared", "prr_cache_reserve", "prr_cache_fork",
       "prr_cache_release", "prr_cache_compact"]


def test_workspace_sizes(lib):
    small, large = (prr.prr_serving_workspace_bytes(_dims(), n) for n in (1, 1 << 20))
    assert 0 < small < large
    assert prr.prr_serving_workspace_bytes(_paged(), 1) >= small
    for rows in (0, -1, (1 << 30) + 1):
        assert prr.prr_serving_workspace_bytes(_dims(), rows) == 0
    assert prr.prr_serving_workspace_bytes(_dims(), 1 << 30) > 0
    assert prr.prr_serving_workspace_bytes(_dims(d=96), 1) == 0


@pytest.mark.parametrize("fn", ALL)
def test_unsupported_dims_and_small_workspaces_are_refused(lib, fn):
    dims = _paged()
    assert _call(lib, fn, _paged(d=96)) == SHAPE
    assert _call(lib, fn, _paged(Hq=18)) == SHAPE  # nine query heads to a KV head
    assert _call(lib, fn, dims, ws=None) == INVALID
    need = prr.prr_serving_workspace_bytes(dims, 10 if fn == "prr_attend_prompt" else 1)
    assert _call(lib, fn, dims, ws_bytes=need - 1) == CAPACITY


@pytest.mark.parametrize("fn,names", [
    ("prr_append_prompt", ["k_rows", "v_rows", "q_begin", "seq_lens", "k_cache", "v_cache"]),
    ("prr_attend_prompt", ["q", "q_begin", "seq_lens", "k_cache", "v_cache", "out"]),
    ("prr_attend_shared", ["q", "members", "group_begin", "shared_blocks", "seq_lens", "k_cache", "v_cache", "out"]),
    ("prr_cache_reserve", ["want", "cache"]), ("prr_cache_fork", ["parents", "children", "cache"]),
    ("prr_cache_release", ["seqs", "cache"]), ("prr_cache_compact", ["cache", "remap", "n_live"]),
])
def test_null_buffers_are_refused(lib, fn, names):
    for name in names:
        assert _call(lib, fn, _paged(), **{name: None}) == INVALID, name


@pytest.mark.parametrize("fn,names", [
    ("prr_append_prompt", ["k_rows", "v_rows", "k_cache", "v_cache", "summ"]),
    ("prr_attend_prompt", ["q", "k_cache", "v_cache", "out"]), ("prr_attend_shared", ["q", "k_cache", "v_cache", "out"]),
])
def test_misaligned_buffers_are_refused(lib, fn, names):
    for name in names:
        assert _call(lib, fn, _paged(), **{name: (1 << 26) + 2}) == INVALID, name


@pytest.mark.parametrize("fn,heads", [("prr_append_prompt", 2), ("prr_attend_prompt", 8), ("prr_attend_shared", 8)])
def test_row_strides(lib, fn, heads):
    for stride in (heads * 128 - 8, heads * 128 + 4, 0, -heads * 128):
        assert _call(lib, fn, _dims(), stride=stride) == SHAPE, stride


def test_counts_out_of_range_are_refused_and_empty_calls_do_nothing(lib):
    for fn in ("prr_append_prompt", "prr_attend_prompt"):
        assert _call(lib, fn, _dims(), rows=-1) == SHAPE and _call(lib, fn, _dims(), rows=(1 << 30) + 1) == SHAPE
        assert _call(lib, fn, _dims(), rows=0, ws=None) == OK
    assert _call(lib, "prr_attend_shared", _dims(), n_members=4) == SHAPE       # more than the batch
    assert _call(lib, "prr_attend_shared", _dims(), n_groups=4) == SHAPE        # nor more groups
    assert _call(lib, "prr_attend_shared", _dims(), n_members=-1) == SHAPE
    assert _call(lib, "prr_attend_shared", _dims(), n_groups=0, ws=None) == OK
    assert _call(lib, "prr_attend_shared", _dims(), n_members=0, n_groups=3, ws=None) == OK
    for fn in ("prr_cache_fork", "prr_cache_release"):
        assert _call(lib, fn, _paged(), n=4) == SHAPE and _call(lib, fn, _paged(), n=-1) == SHAPE
        assert _call(lib, fn, _paged(), n=0) == OK


@pytest.mark.parametrize("fn", ALL[3:])
def test_page_calls_need_a_paged_cache_and_its_table(lib, fn):
    assert _call(lib, fn, _dims()) == SHAPE
    assert _call(lib, fn, _paged(), cache=_cache(block_table=1 << 25)) == INVALID  # not the dims' table
    for name in ("block_table", "page_refs"):
        assert _call(lib, fn, _paged(), cache=_cache(**{name: None})) == INVALID, name
    for name in ("k_cache", "v_cache", "summ"):
        assert _call(lib, fn, _paged(), cache=_cache(**{name: (1 << 26) + 2})) == INVALID, name
    if fn != "prr_cache_compact":
        assert _call(lib, fn, _paged(), cache=_cache(seq_lens=None)) == INVALID
    if fn in ("prr_cache_fork", "prr_cache_compact"):
        assert _call(lib, fn, _paged(), cache=_cache(k_cache=None)) == INVALID
        assert _call(lib, fn, _paged(), cache=_cache(v_cache=None)) == INVALID


def test_cache_buffers_match_the_header_layout(tmp_path):
    lines = ['#include <stdio.h>', '#include <stddef.h>', '#include "prr.h"', 'int main(void) {',
             '  printf("size %zu\\n", sizeof(prr_cache_buffers));']
    lines += [f'  printf("{n} %zu\\n", offsetof(prr_cache_buffers, {n}));' for n, _ in _abi.PrrCacheBuffers._fields_]
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text("\n".join(lines + ["  return 0;", "}"]) + "\n")
    inc = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include")
    subprocess.run(["gcc", "-std=c99", "-I", os.path.join(ROOT, "include"), "-I", inc, str(src), "-o", str(exe)], check=True)
    out = dict(ln.split() for ln in subprocess.run([str(exe)], capture_output=True, text=True).stdout.splitlines())
    assert int(out["size"]) == ctypes.sizeof(_abi.PrrCacheBuffers)
    for name, _ in _abi.PrrCacheBuffers._fields_:
        assert int(out[name]) == getattr(_abi.PrrCacheBuffers, name).offset, name


def test_the_binding_refuses_wrong_tensors():
    d = _dims()
    ws = torch.zeros(16, dtype=torch.uint8)
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    i32 = lambda n: torch.zeros(n, dtype=torch.int32)  # noqa: E731
    with pytest.raises(ValueError):  # CPU tensors
        prr.prr_attend_prompt(d, bf(5, 8, 128), i32(4), i32(3), bf(1), bf(1), bf(5, 8, 128), None, ws)
    with pytest.raises(ValueError):  # another head count
        prr.prr_attend_prompt(d, bf(5, 4, 128), i32(4), i32(3), bf(1), bf(1), bf(5, 8, 128), None, ws)
    with pytest.raises(ValueError):  # another type
        prr.prr_append_prompt(d, torch.zeros(5, 2, 128), torch.zeros(5, 2, 128), i32(4), i32(3), bf(1), bf(1), None, ws)
    with pytest.raises(ValueError):  # rows that overlap
        prr.prr_attend_prompt(d, torch.as_strided(bf(4096), (5, 8, 128), (128, 128, 1)), i32(4), i32(3), bf(1), bf(1),
                              bf(5, 8, 128), None, ws)
    with pytest.raises(ValueError):  # one query for each sequence
        prr.prr_attend_shared(d, bf(2, 8, 128), i32(3), i32(2), i32(1), i32(3), bf(1), bf(1), bf(2, 8, 128), None, ws)
    with pytest.raises(ValueError):
        prr.prr_cache_fork(_paged(), i32(2), i32(1), _cache(), ws)
