"""Cross attention on the CPU: the 64-bit reference against differences and
special cases, the bucket map, and the refusals of the C entry points and the
binding (none of these needs a GPU)."""
import ctypes
import math

import numpy as np
import pytest
import torch

from streaming_sinkhorn_solver_gb300 import binding as fs
from tests.attention_ref import attention64


@pytest.fixture(scope="module")
def lib():
    from streaming_sinkhorn_solver_gb300.build import build
    build()
    return fs.load_library()


def _case(seed=0, B=2, n=3, m=5, H=4, G=2, d=3):
    g = torch.Generator().manual_seed(seed)

    def r(*s):
        return torch.randn(*s, generator=g, dtype=torch.float64)

    c = dict(q=r(B, n, H, d), k=r(B, m, G, d), v=r(B, m, G, d), scale=0.7,
             kv_len=torch.tensor([m, 2]), key_mask=torch.tensor([[1, 0, 1, 1, 1], [1, 1, 1, 1, 1]]),
             bias=r(H, 4), buckets=torch.from_numpy(fs.fs_relative_buckets(4, 3)),
             q_pos=torch.tensor([1, 0]))
    return c, r(B, n, H, d)


@pytest.mark.parametrize("name", ["q", "k", "v", "bias"])
@pytest.mark.parametrize("shared", [False, True])
def test_reference_gradients_match_differences(name, shared):
    c, dout = _case()
    if shared:
        c["bias"] = c["bias"][:1]
    r = attention64(**c, dout=dout)
    g = torch.Generator().manual_seed(1)
    direction = torch.randn(c[name].shape, generator=g, dtype=torch.float64)
    h = 1e-5
    up, down = dict(c), dict(c)
    up[name], down[name] = c[name] + h * direction, c[name] - h * direction
    got = float(((attention64(**up)["out"] - attention64(**down)["out"]) * dout).sum() / (2 * h))
    want = float((r["d" + name] * direction).sum())
    # central differences of a function with third derivatives of order 10: 10 h^2, and
    # 64-bit rounding 1e-16 / h
    assert abs(got - want) <= 1e-8 * (1 + abs(want))


def test_reference_special_cases():
    # equal scores average the counted values; a lone key is returned; no key: 0 and -inf
    q = torch.zeros(3, 2, 2, 4, dtype=torch.float64)
    k = torch.randn(3, 6, 1, 4, dtype=torch.float64)
    v = torch.randn(3, 6, 1, 4, dtype=torch.float64)
    r = attention64(q, k, v, 1.0, kv_len=torch.tensor([6, 1, 0]))
    assert torch.allclose(r["out"][0, 1, 1], v[0, :, 0].mean(0))
    assert torch.equal(r["out"][1, 0, 0], v[1, 0, 0])
    assert torch.all(r["out"][2] == 0) and torch.all(r["lse"][2] == -math.inf)
    assert math.isclose(float(r["lse"][0, 0, 0]), math.log(6))


@pytest.mark.parametrize("nb,far", [(4, 3), (8, 16), (32, 128), (64, 1000), (6, 40)])
def test_relative_buckets(nb, far):
    b = fs.fs_relative_buckets(nb, far)
    assert b.dtype == np.int32 and b.shape == (2 * far + 1,)
    half, near = nb // 2, nb // 4
    # single distances next to the query, every bucket in order, the last at max_distance
    for a in range(min(near, far) + 1):
        assert b[far - a] == a
    assert list(b[far + 1:]) == [half + x for x in b[:far][::-1]]
    assert np.all(np.diff(b[:far + 1]) <= 0) and b[0] == half - 1
    one = fs.fs_relative_buckets(nb, far, bidirectional=False)
    assert np.all(one[far:] == 0) and one[0] == nb - 1
    assert np.all(np.diff(one[:far + 1]) <= 0)


def test_relative_buckets_are_exact_at_their_boundaries():
    # near 8, wide 8, far 128: boundaries at 8 * 16^(s/8) = 8 * 2^(s/2); the even ones
    # are whole numbers, which belong to the upper bucket
    b = fs.fs_relative_buckets(32, 128)[128::-1]
    for s, edge in ((0, 8), (2, 16), (4, 32), (6, 64)):
        assert b[edge] == 8 + s and b[edge - 1] == 8 + s - 1
    with pytest.raises(ValueError):
        fs.fs_relative_buckets(5, 16)
    with pytest.raises(ValueError):
        fs.fs_relative_buckets(32, 8)


def _desc(**over):
    at = fs.fs_attention()
    at.dtype, at.heads, at.kv_heads, at.d = 0, 4, 2, 64
    at.batch, at.n, at.m, at.scale = 2, 3, 5, 0.125
    for name, heads, tokens in (("q", 4, 3), ("out", 4, 3), ("dout", 4, 3), ("dq", 4, 3),
                                ("k", 2, 5), ("v", 2, 5), ("dk", 2, 5), ("dv", 2, 5)):
        setattr(at, name + "_stride", (ctypes.c_int64 * 3)(tokens * heads * 64, heads * 64, 64))
    for k, v in over.items():
        setattr(at, k, v)
    return at


@pytest.mark.parametrize("over", [
    dict(dtype=2), dict(dtype=-1), dict(heads=0), dict(kv_heads=0), dict(kv_heads=3), dict(d=0),
    dict(d=129), dict(batch=-1), dict(n=-1), dict(m=-1), dict(m=2 ** 31), dict(scale=0.0),
    dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")), dict(reserved=1),
    dict(n_buckets=-1), dict(n_buckets=1025), dict(n_buckets=8), dict()])
def test_entry_points_refuse_bad_descriptions(lib, over):
    """The last case is a good description with null tensors."""
    at = _desc(**over)
    assert lib.fs_cross_attention(ctypes.byref(at), *[None] * 6) == fs.FS_ERR_INVALID_ARG
    assert fs.fs_last_error()
    assert lib.fs_cross_attention_grad(ctypes.byref(at), *[None] * 11) == fs.FS_ERR_INVALID_ARG
    assert fs.fs_last_error()


def test_entry_points_refuse_a_null_description(lib):
    assert lib.fs_cross_attention(None, *[None] * 6) == fs.FS_ERR_INVALID_ARG
    assert lib.fs_cross_attention_grad(None, *[None] * 11) == fs.FS_ERR_INVALID_ARG


def test_description_mirrors_the_header():
    import os
    import re
    text = open(os.path.join(os.path.dirname(__file__), "..", "include", "flashsinkhorn.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    body = re.search(r"typedef struct fs_attention \{(.*?)\} fs_attention;", text, flags=re.S).group(1)
    want = []
    for decl in filter(None, (x.strip() for x in body.split(";"))):
        kind, names = re.match(r"(const [\w]+ ?\*|\w+)\s*(.*)", decl, flags=re.S).groups()
        for name in names.split(","):
            arr = re.match(r"(\w+)\[(\d+)\]", name.strip())
            base = {"int32_t": ctypes.c_int32, "int64_t": ctypes.c_int64,
                    "float": ctypes.c_float}.get(kind, ctypes.c_void_p)
            want.append((arr.group(1), base * int(arr.group(2))) if arr else (name.strip(), base))
    got = fs.fs_attention._fields_
    assert [n for n, _ in got] == [n for n, _ in want]
    for (_, a), (_, b) in zip(got, want):
        assert ctypes.sizeof(a) == ctypes.sizeof(b) and getattr(a, "_length_", 0) == getattr(b, "_length_", 0)


def test_binding_refuses_cpu_and_float32_tensors():
    q = torch.zeros(1, 2, 2, 8, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        fs.fs_cross_attention(q, q, q)
    with pytest.raises(TypeError):
        fs.fs_cross_attention(q.float(), q.float(), q.float())
