"""The host check for tensors that share bytes (csrc/overlap.h) against all pairs of bytes, and the
rotary call's refusals by it (the addresses are never touched)."""
import ctypes
import os
import random
import subprocess

import pytest

from sparse_attention_lightning_indexer_gb300 import build, ds4idx

from .test_operators_host import P, _vp

SOURCE = """
#include "overlap.h"
using namespace ds4;
static Pieces make(const int64_t* v) {
  return Pieces(reinterpret_cast<const void*>(v[0]), v[1], v[2], v[3], v[4], v[5]);
}
extern "C" int self(const int64_t* a) { return overlaps_itself(make(a)); }
extern "C" int pair(const int64_t* a, const int64_t* b) { return overlap(make(a), make(b)); }
"""


@pytest.fixture(scope="module")
def check(tmp_path_factory):
    d = tmp_path_factory.mktemp("overlap")
    src, lib = d / "overlap.cpp", d / "overlap.so"
    src.write_text(SOURCE)
    subprocess.run(["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-I", build.CSRC, str(src), "-o",
                    str(lib)], check=True)
    return ctypes.CDLL(os.fspath(lib))


def _spec(base, nt, st, nh, sh, w):
    return (ctypes.c_int64 * 6)(base, nt, st, nh, sh, w)


def _pieces(base, nt, st, nh, sh, w):
    return [range(base + t * st + h * sh, base + t * st + h * sh + w)
            for t in range(nt) for h in range(nh)]


def test_against_all_bytes(check):
    rng = random.Random(1)
    seen = {("self", 0): 0, ("self", 1): 0, ("pair", 0): 0, ("pair", 1): 0}
    for _ in range(20000):
        nt, w = rng.randint(1, 5), rng.randint(1, 4)
        st = rng.randint(-14, 14)
        a = (200 + rng.randint(-9, 9), nt, st, rng.randint(1, 5), rng.randint(-9, 14), w)
        b = (200 + rng.randint(-30, 30), nt, st if rng.random() < 0.8 else rng.randint(-14, 14),
             rng.randint(1, 5), a[4] if rng.random() < 0.5 else rng.randint(-9, 14), rng.randint(1, 4))
        used = [x for r in _pieces(*a) for x in r]
        want = int(len(set(used)) < len(used))
        assert check.self(_spec(*a)) == want, a
        seen["self", want] += 1
        other = {x for r in _pieces(*b) for x in r}
        want = int(bool(set(used) & other))
        got = check.pair(_spec(*a), _spec(*b))
        if got and not want:           # the documented refusal: interleaved spans, other strides
            assert nt > 1 and a[2] != b[2]
            assert min(used) <= max(other) and min(other) <= max(used)
        else:
            assert got == want, (a, b)
            seen["pair", want] += 1
    assert min(seen.values()) > 1000, seen


def test_large_strides_and_counts(check):
    assert check.self(_spec(1 << 40, 2 ** 31 - 1, 65536 * 512, 65536, 512, 512)) == 0
    assert check.self(_spec(1 << 40, 2 ** 31 - 1, 65536 * 512 - 1, 65536, 512, 512)) == 1
    assert check.self(_spec(1 << 40, 2 ** 31 - 1, 1 << 62, 2, 128, 128)) == 0


def _call(lib, tensors, T=4, rot=64):
    """tensors: keyword arguments of RotaryTensor, x and out in bytes from P."""
    base = dict(dtype=0, interleaved=1, n_heads=2, reserved=0, x_stride_t=256, x_stride_h=64,
                out_stride_t=256, out_stride_h=64)
    a = (ds4idx.RotaryTensor * len(tensors))()
    for k, t in enumerate(tensors):
        d = dict(base, **t)
        d["x"], d["out"] = P + d["x"], P + d["out"]
        a[k] = ds4idx.RotaryTensor(**d)
    f = (ctypes.c_uint64 * 128)()
    return lib.ds4idx_rotary(len(tensors), _vp(a), T, rot, P, _vp(f), 1.0, 0, None)


FAR = 1 << 30


@pytest.mark.parametrize("what,tensors", [
    ("heads of an out in one place", [dict(x=0, out=FAR, out_stride_h=0)]),
    ("tokens of an out in one place", [dict(x=0, out=FAR, out_stride_t=0)]),
    ("heads that overlap by one element", [dict(x=0, out=FAR, out_stride_h=63)]),
    ("tokens that overlap the last head", [dict(x=0, out=FAR, out_stride_t=127)]),
    ("an out shifted against its input", [dict(x=0, out=2)]),
    ("an out one token behind its input", [dict(x=0, out=512)]),
    ("in place with heads in another order", [dict(x=0, out=0, x_stride_t=128, out_stride_t=64,
                                                   x_stride_h=64, out_stride_h=256)]),
    ("two outs in one place", [dict(x=0, out=FAR), dict(x=0, out=FAR)]),
    ("an out over another tensor's input", [dict(x=0, out=0), dict(x=0, out=FAR)]),
    ("an out over a later tensor's input", [dict(x=0, out=FAR), dict(x=FAR, out=2 * FAR)]),
    ("an fp32 out over a bf16 input", [dict(x=FAR, out=FAR + 65536, dtype=ds4idx.F32, n_heads=1),
                                       dict(x=FAR + 65536 + 100, out=0, n_heads=1)]),
])
def test_rotary_refuses_shared_bytes(what, tensors):
    build.build()
    assert _call(ds4idx.load(), tensors) == ds4idx.ERR_INVALID_ARG, what
