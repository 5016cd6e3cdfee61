"""The test of whether two strided tensors share memory, against all their addresses; and the calls that refuse such outputs."""
import ctypes
import os
import random
import subprocess

import pytest

from numerics_tcgen05_tmem_gb300 import binding, build
from tests import test_kv_weights_cpu as W
from tests import test_norm_rotate_cpu as N

G, BAD = N.G, N.BAD
lib = N.lib


@pytest.fixture(scope="module")
def overlap(tmp_path_factory):
    d = tmp_path_factory.mktemp("overlap")
    src = d / "overlap.cpp"
    src.write_text('#include "overlap.h"\nextern "C" int go(const long long* x) {\n'
                   "  fa::Pieces p[2];\n  for (int i = 0; i < 2; ++i, x += 8) {\n"
                   "    p[i] = {reinterpret_cast<const void*>(x[0]), x[1], {x[2], x[3], x[4]}, {x[5], x[6], x[7]}};\n  }\n"
                   "  return fa::pieces_overlap(p[0], p[1]);\n}\n")
    so = d / "overlap.so"
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I", build.CSRC, str(src), "-o", str(so)], check=True)
    go = ctypes.CDLL(str(so)).go
    return lambda a, b: bool(go((ctypes.c_longlong * 16)(*a, *b)))


def addresses(p, size, n, s):
    return {p + i * s[0] + j * s[1] + k * s[2] + e for i in range(n[0]) for j in range(n[1]) for k in range(n[2]) for e in range(size)}


def flat(p, size, n, s):
    return (p, size, *n, *s)


def test_against_all_addresses(overlap):
    r = random.Random(1)
    seen = set()
    for _ in range(4000):
        kind = r.randrange(3)
        size = r.randint(1, 6)
        if kind == 0:      # two views of one buffer
            n, h = [r.randint(1, 4) for _ in range(3)], r.randint(1, 8)
            s = [h * size * n[1] + r.randint(0, 9), h * size, size]
            a = (1000, size, n, s)
            m = [r.randint(1, x + 1) for x in n]
            b = (1000 + r.randint(-4, 4) * size + r.choice([0, 0, 1, -1]), size, m, s)
        else:              # anything
            a, b = ((1000 + r.randint(0, 60), r.randint(1, 6), [r.randint(1, 4) for _ in range(3)], [r.randint(0, 40) for _ in range(3)])
                    for _ in range(2))
        want = bool(addresses(*a) & addresses(*b))
        assert overlap(flat(*a), flat(*b)) == want, (a, b)
        seen.add((kind > 0, want))
    assert len(seen) == 4


def test_large_tensors_and_a_search_that_ends(overlap):
    # [8, 4096, 96 heads of 256 bytes]: queries and keys of one projection, apart by a head, a byte
    q = flat(1 << 40, 256, [8, 4096, 64], [4096 * 96 * 256, 96 * 256, 256])
    k = lambda p: flat(p, 256, [8, 4096, 16], [4096 * 96 * 256, 96 * 256, 256])
    assert not overlap(q, k((1 << 40) + 64 * 256)) and overlap(q, k((1 << 40) + 64 * 256 - 1)) and overlap(q, k((1 << 40) + 63 * 256))
    assert overlap(q, k((1 << 40) - 16 * 256)) == overlap(k((1 << 40) - 16 * 256), q)
    # strides without a common order: an answer after a bounded number of steps
    a = flat(0, 1, [100000, 100000, 100000], [1000003 * 2, 999983 * 2, 999979 * 2])
    b = flat(1, 1, [100000, 100000, 100000], [999961 * 2, 999959 * 2, 999953 * 2])
    overlap(a, b)


def test_norm_rotate_refuses_outputs_that_overlap(lib):
    # views [2, 4, 100, 64] of tokens of 12 heads: q, k, v heads of one projection, 128 bytes a head
    head = 128
    at = lambda i, base=G: N.view(base + i * head, b=12 * 100 * 64, h=64, n=12 * 64)
    far = [at(0, G + (i << 24)) for i in range(1, 7)]
    for qo in (at(1), at(-1), at(4), at(7), at(5)):             # within q's or k's heads
        assert N.forward(lib, q=at(0), k=at(4), qo=qo, ko=far[0]) == BAD and ("same strides" in binding.last_error() or "another tensor" in binding.last_error())
    assert N.forward(lib, q=at(0), k=at(4), qo=far[0], ko=at(3)) == BAD
    assert N.forward(lib, q=at(0), k=at(4), qo=at(0, 3 * G), ko=at(3, 3 * G)) == BAD   # the outputs each other
    for dx in (at(1), at(3), at(5)):
        assert N.backward(lib, q=at(0), k=at(4), dz=far[0], dzk=far[1], dx=dx, dk=far[2]) == BAD
        assert N.backward(lib, q=far[0], k=far[1], dz=at(0), dzk=at(4), dx=far[3], dk=dx) == BAD
    assert N.backward(lib, dw=(G, G + 252)) == BAD and "overlap" in binding.last_error()


def test_append_refuses_an_output_that_overlaps(lib):
    # rows of 8 + 2 + 2 heads of 64, five tokens
    row, head = 12 * 64, 128
    kw = dict(q=G, q_stride=row, k=G + 8 * head, v=G + 10 * head, stride=row)
    for out in (G + head, G - head, G + 8 * head, G + 11 * head, G + 4 * row * 2 + 10 * head, G):
        assert N.append(lib, out=out, **kw) == BAD and "q_out" in binding.last_error()


def test_evict_refuses_outputs_that_overlap(lib):
    for kw in (dict(kept=(1 << 22) + 8), dict(kept=(1 << 22) - 8), dict(kept=(1 << 21) + 4), dict(kept_len=(1 << 21) + 8), dict(kept_len=G + 4),
               dict(kept_len=G - 8), dict(kept=G - 4)):
        assert W.evict(lib, **kw) == BAD
        assert "another" in binding.last_error() or "kv_len" in binding.last_error()
