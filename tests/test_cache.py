"""Rotary positions, the cache in pages and the tree attention on the CPU: the references
against special cases, the frequencies, and the refusals of the C entry points and the
binding (none of these needs a GPU)."""
import ctypes
import math
import os
import re

import numpy as np
import pytest
import torch

from streaming_sinkhorn_solver_gb300 import binding as fs
from tests.kv_ref import quantise, rotary64, sees, tree64


@pytest.fixture(scope="module")
def lib():
    from streaming_sinkhorn_solver_gb300.build import build
    build()
    return fs.load_library()


# --- references ---------------------------------------------------------------

@pytest.mark.parametrize("interleaved", [False, True])
def test_rotary_reference(interleaved):
    g = torch.Generator().manual_seed(0)
    x = torch.randn(2, 3, 2, 10, generator=g, dtype=torch.float64).float().bfloat16()
    w = torch.from_numpy(fs.fs_rotary_frequencies(8))
    pos = torch.tensor([[0, 1, 7], [5, 5, 100]])
    y, _ = rotary64(x, w, pos, interleaved)
    # turns keep lengths, position 0 keeps all, the rest of the head stays
    assert torch.allclose(y[..., :8].norm(dim=-1), x[..., :8].double().norm(dim=-1))
    assert torch.equal(y[0, 0], x[0, 0].double()) and torch.equal(y[..., 8:], x[..., 8:].double())
    # products of queries and keys depend on the distance alone
    a, b = x[:1, :1], x[:1, 1:2]
    dots = [float((rotary64(a, w, torch.tensor([[p]]), interleaved)[0] *
                   rotary64(b, w, torch.tensor([[p + 4]]), interleaved)[0])[..., :8].sum())
            for p in (0, 11, 1000)]
    assert max(dots) - min(dots) < 1e-9
    # the gradient: <turn(x), y> = <x, turn back(y)>, amplitude included
    up = rotary64(a, w, torch.tensor([[9]]), interleaved, 1.3)[0]
    down = rotary64(b, w, torch.tensor([[9]]), interleaved, 1.3, back=True)[0]
    assert math.isclose(float((up * b.double())[..., :8].sum()), float((down * a.double())[..., :8].sum()),
                        rel_tol=1e-12)


def test_frequencies():
    f = fs.fs_rotary_frequencies(64)
    assert f.shape == (32,) and f.dtype == np.float64 and f[0] == 1.0
    assert np.allclose(f[1:] / f[:-1], 10000.0 ** (-1 / 32))
    assert np.allclose(fs.fs_rotary_frequencies(64, factor=4.0), f / 4)
    g = fs.fs_rotary_frequencies(64, factor=8.0, trained=8192)
    turns = 8192 * f / (2 * np.pi)
    assert np.array_equal(g[turns >= 4], f[turns >= 4])
    assert np.allclose(g[turns <= 1], f[turns <= 1] / 8)
    assert np.all(np.diff(g) < 0) and np.all(g <= f) and np.all(g >= f / 8)
    for bad in (dict(rotary_dim=7), dict(rotary_dim=0), dict(rotary_dim=8, base=0.0),
                dict(rotary_dim=8, factor=0.0), dict(rotary_dim=8, trained=5, low=4.0)):
        with pytest.raises(ValueError):
            fs.fs_rotary_frequencies(**bad)


def test_quantise_reference():
    x = torch.tensor([[448.0, -3.0, 0.0, 1.0], [0.0] * 4, [math.nan, 1, 2, 3], [1, math.inf, 0, 0]])
    code, scale = quantise(x.bfloat16(), torch.float8_e4m3fn)
    assert torch.equal(code[0].float(), x[0]) and float(scale[0]) == 1.0
    assert torch.all(code[1:].float() == 0) and torch.all(torch.isnan(scale[2:]))
    code, scale = quantise(x.bfloat16(), torch.int8)
    assert code[0].tolist() == [127, -1, 0, 0]


def test_tree_reference():
    assert sees(4, [-1, 0, 0, 2]).int().tolist() == [[1, 0, 0, 0], [1, 1, 0, 0], [1, 0, 1, 0], [1, 0, 1, 1]]
    assert torch.equal(sees(5, None), torch.ones(5, 5, dtype=torch.bool).tril())
    # no chain to -1: a parent of -2, a later one, itself, and their children
    assert torch.equal(sees(5, [-1, -2, 3, 3, 1]).any(1), torch.tensor([True, False, False, False, False]))
    g = torch.Generator().manual_seed(0)
    q, k, v = (torch.randn(1, r, h, 4, generator=g).bfloat16() for r, h in ((2, 2), (5, 1), (5, 1)))
    there = torch.ones(1, 5, dtype=torch.bool)
    r = tree64(torch.zeros_like(q), k, v, there, [3], torch.tensor([-1, -1]))
    assert torch.allclose(r["out"][0, 0, 0], v[0, [0, 1, 2, 3], 0].double().mean(0))
    assert torch.allclose(r["out"][0, 1, 0], v[0, [0, 1, 2, 4], 0].double().mean(0))
    assert math.isclose(float(r["lse"][0, 0, 0]), math.log(4))
    r = tree64(q, k, v, torch.zeros_like(there), [3])
    assert torch.all(r["out"] == 0) and torch.all(r["lse"] == -math.inf)


# --- the C boundary -----------------------------------------------------------

def _header_struct(name):
    text = open(os.path.join(os.path.dirname(__file__), "..", "include", "flashsinkhorn.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    body = re.search(r"typedef struct %s \{(.*?)\} %s;" % (name, name), text, flags=re.S).group(1)
    want = []
    for decl in filter(None, (x.strip() for x in body.split(";"))):
        kind, names = re.match(r"((?:const )?\w+)\s*(.*)", decl, flags=re.S).groups()
        for field in names.split(","):
            field = field.strip()
            arr = re.match(r"(\w+)\[(\d+)\]", field)
            base = ctypes.c_void_p if field.startswith("*") else \
                {"int32_t": ctypes.c_int32, "int64_t": ctypes.c_int64, "float": ctypes.c_float}[kind]
            want.append((arr.group(1), base * int(arr.group(2))) if arr else (field.lstrip("* "), base))
    return want


@pytest.mark.parametrize("name", ["fs_rotation", "fs_cache", "fs_cache_rows", "fs_tree"])
def test_descriptions_mirror_the_header(name):
    want, got = _header_struct(name), getattr(fs, name)._fields_
    assert [n for n, _ in got] == [n for n, _ in want]
    for (_, a), (_, b) in zip(got, want):
        assert ctypes.sizeof(a) == ctypes.sizeof(b) and getattr(a, "_length_", 0) == getattr(b, "_length_", 0)


def _rotation(**over):
    r = fs.fs_rotation()
    r.dtype, r.heads, r.kv_heads, r.d, r.rotary_dim, r.batch, r.n, r.amplitude = 0, 4, 2, 64, 64, 2, 3, 1.0
    for name, heads in (("q", 4), ("k", 2), ("q_out", 4), ("k_out", 2)):
        setattr(r, name + "_stride", (ctypes.c_int64 * 3)(3 * heads * 64, heads * 64, 64))
    r.pos_stride = (ctypes.c_int64 * 2)(3, 1)
    for k, v in over.items():
        setattr(r, k, v)
    return r


@pytest.mark.parametrize("over", [
    dict(dtype=2), dict(dtype=-1), dict(heads=0), dict(heads=2 ** 20), dict(kv_heads=-1), dict(d=0),
    dict(d=5000), dict(rotary_dim=0), dict(rotary_dim=7), dict(rotary_dim=66), dict(interleaved=2),
    dict(batch=-1), dict(n=-1), dict(n=2 ** 31), dict(amplitude=float("nan")),
    dict(amplitude=float("inf")), dict(reserved=1), dict(pos_stride=(ctypes.c_int64 * 2)(-1, 1)), dict()])
def test_rotary_refuses_bad_descriptions(lib, over):
    """The last case is a good description with null tensors."""
    r = _rotation(**over)
    for fn in (lib.fs_rotary, lib.fs_rotary_grad):
        assert fn(ctypes.byref(r), *[None] * 5) == fs.FS_ERR_INVALID_ARG
        assert fs.fs_last_error()
        assert fn(None, *[None] * 5) == fs.FS_ERR_INVALID_ARG


def _cache_desc(**over):
    c = fs.fs_cache()
    c.dtype, c.kv_heads, c.d, c.page_size = 2, 2, 64, 16
    c.pages, c.batch, c.table_pages, c.table_stride = 8, 2, 4, 4
    for name in ("k", "v"):
        setattr(c, name + "_stride", (ctypes.c_int64 * 3)(2 * 16 * 64, 16 * 64, 64))
        setattr(c, name + "_scale_stride", (ctypes.c_int64 * 2)(32, 16))
    for k, v in over.items():
        setattr(c, k, v)
    return c


_BAD_CACHES = [dict(dtype=4), dict(dtype=-1), dict(kv_heads=0), dict(d=0), dict(d=12), dict(d=136),
               dict(page_size=0), dict(page_size=4), dict(page_size=24), dict(page_size=2 ** 21),
               dict(pages=-1), dict(pages=2 ** 31), dict(batch=-1), dict(batch=2 ** 31), dict(table_pages=-1),
               dict(table_pages=2 ** 28), dict(table_stride=-1), dict()]


@pytest.mark.parametrize("over", _BAD_CACHES)
def test_cache_calls_refuse_bad_caches(lib, over):
    """The last case is a good description with null tensors."""
    c = _cache_desc(**over)
    rows, tree = fs.fs_cache_rows(), fs.fs_tree()
    rows.n = 3
    tree.heads, tree.n, tree.scale = 4, 3, 0.125
    for fn in (lib.fs_cache_write, lib.fs_cache_read):
        assert fn(ctypes.byref(c), ctypes.byref(rows), None, None, None) == fs.FS_ERR_INVALID_ARG
        assert fn(None, ctypes.byref(rows), None, None, None) == fs.FS_ERR_INVALID_ARG
    assert lib.fs_tree_attention(ctypes.byref(c), ctypes.byref(tree), *[None] * 4) == fs.FS_ERR_INVALID_ARG
    assert lib.fs_tree_attention(None, ctypes.byref(tree), *[None] * 4) == fs.FS_ERR_INVALID_ARG
    assert fs.fs_last_error()


def _empty_pool(**over):
    """No pages and no table: a description whose tensors may be null."""
    return _cache_desc(pages=0, table_pages=0, **over)


@pytest.mark.parametrize("over", [dict(dtype=2), dict(dtype=3), dict(reserved=1), dict(n=-1), dict(n=2 ** 31)])
def test_cache_calls_refuse_bad_rows(lib, over):
    rows = fs.fs_cache_rows()
    for k, v in over.items():
        setattr(rows, k, v)
    for fn in (lib.fs_cache_write, lib.fs_cache_read):
        assert fn(ctypes.byref(_empty_pool()), ctypes.byref(rows), None, None, None) == fs.FS_ERR_INVALID_ARG
        assert fn(ctypes.byref(_empty_pool()), None, None, None, None) == fs.FS_ERR_INVALID_ARG


def test_a_cache_in_16_bits_takes_its_own_type(lib):
    rows, tree = fs.fs_cache_rows(), fs.fs_tree()
    rows.dtype = tree.dtype = 1
    tree.heads, tree.scale = 4, 1.0
    c = _empty_pool(dtype=0)
    assert lib.fs_cache_write(ctypes.byref(c), ctypes.byref(rows), None, None, None) == fs.FS_ERR_INVALID_ARG
    assert lib.fs_tree_attention(ctypes.byref(c), ctypes.byref(tree), *[None] * 4) == fs.FS_ERR_INVALID_ARG


@pytest.mark.parametrize("over", [
    dict(dtype=2), dict(heads=0), dict(heads=3), dict(n=-1), dict(n=257), dict(scale=0.0), dict(scale=-1.0),
    dict(scale=float("nan")), dict(scale=float("inf")), dict(reserved=1),
    dict(parents=ctypes.c_void_p(8), parents_stride=-1), dict(n=2)])
def test_tree_attention_refuses_bad_trees(lib, over):
    """The last case is a good description with null tensors."""
    tree = fs.fs_tree()
    tree.heads, tree.scale = 4, 0.125
    for k, v in over.items():
        setattr(tree, k, v)
    assert lib.fs_tree_attention(ctypes.byref(_empty_pool()), ctypes.byref(tree), *[None] * 4) == \
        fs.FS_ERR_INVALID_ARG
    assert lib.fs_tree_attention(ctypes.byref(_empty_pool()), None, *[None] * 4) == fs.FS_ERR_INVALID_ARG


# --- the binding --------------------------------------------------------------

def test_binding_refuses_other_kinds():
    q = torch.zeros(1, 2, 2, 8, dtype=torch.bfloat16)
    cache = fs.KVCache(q, q)
    for bad in (q, q.float(), np.zeros((1, 2, 2, 8), np.float16), None):
        with pytest.raises(TypeError):
            fs.fs_rotary(bad, None, None, None)
        with pytest.raises(TypeError):
            fs.fs_rotary_grad(bad, None, None, None)
        with pytest.raises(TypeError):
            fs.fs_cache_write(cache, None, None, bad, bad)
        with pytest.raises(TypeError):
            fs.fs_cache_read(fs.KVCache(bad, bad), None)
        with pytest.raises(TypeError):
            fs.fs_tree_attention(bad, cache, None, None)
    with pytest.raises(TypeError):
        fs.fs_cache_new(1, 1, 16, 64, torch.float32, device="cpu")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float8_e4m3fn, torch.int8])
@pytest.mark.parametrize("d", [64, 72])
def test_new_caches(dtype, d):
    c = fs.fs_cache_new(3, 2, 16, d, dtype, device="cpu")
    assert c.k.shape == c.v.shape == (3, 2, 16, d) and c.k.dtype == dtype and c.k.stride(3) == 1
    assert c.k.stride(2) * c.k.element_size() % 16 == 0
    assert c.k.data_ptr() != c.v.data_ptr()
    if c.k.element_size() == 1:
        assert c.k_scale.shape == (3, 2, 16) and c.k_scale.dtype == torch.float32
    else:
        assert c.k_scale is None and c.v_scale is None
