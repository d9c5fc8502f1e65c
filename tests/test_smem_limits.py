"""The table of shared-memory limits (csrc/smem_limits.h) against a fake driver: whatever the number of
kernels and contexts, a limit covers each call that has asked for it and never goes down."""
import ctypes
import os
import random
import subprocess

import pytest

from image_dits_b200 import build as rf2_build

SOURCE = r"""
#include "smem_limits.h"
extern "C" {
typedef int (*Set)(unsigned long long func, unsigned long long bytes);
void* limits_new() { return new rf2::SmemLimits; }
void limits_delete(void* p) { delete static_cast<rf2::SmemLimits*>(p); }
int limits_ensure(void* p, unsigned long long func, int have_ctx, unsigned long long ctx, unsigned long long bytes, Set set)
{
    return static_cast<rf2::SmemLimits*>(p)->ensure(
        reinterpret_cast<const void*>(func), have_ctx != 0, ctx, bytes,
        [&](const void* f, size_t n) { return set(reinterpret_cast<unsigned long long>(f), n) != 0; });
}
}
"""
SET = ctypes.CFUNCTYPE(ctypes.c_int, ctypes.c_ulonglong, ctypes.c_ulonglong)


@pytest.fixture(scope="module")
def limits(tmp_path_factory):
    d = tmp_path_factory.mktemp("limits")
    src, out = d / "limits.cpp", d / "limits.so"
    src.write_text(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-shared", "-fPIC", "-I", rf2_build.CSRC, "-o", os.fspath(out), os.fspath(src)], check=True)
    L = ctypes.CDLL(os.fspath(out))
    L.limits_new.restype = ctypes.c_void_p
    L.limits_delete.argtypes = [ctypes.c_void_p]
    L.limits_ensure.argtypes = [ctypes.c_void_p, ctypes.c_ulonglong, ctypes.c_int, ctypes.c_ulonglong, ctypes.c_ulonglong, SET]
    return L


class Driver:
    """Limits per (kernel, context), and the calls that set them."""

    def __init__(self, L, refuse_above=1 << 20):
        self.L, self.table, self.attr, self.ctx, self.calls, self.refuse_above = L, L.limits_new(), {}, 0, 0, refuse_above
        self.set = SET(self._set)

    def _set(self, func, n):
        self.calls += 1
        if n > self.refuse_above:
            return 0
        assert n >= self.attr.get((func, self.ctx), 0), "a limit went down"
        self.attr[func, self.ctx] = n
        return 1

    def ask(self, func, ctx, n, known=True):
        self.ctx = ctx
        before = self.attr.get((func, ctx), 0)
        ok = self.L.limits_ensure(self.table, func, int(known), ctx, n, self.set)
        assert self.attr.get((func, ctx), 0) >= before, "a limit went down"
        assert not ok or self.attr[func, ctx] >= n
        return ok

    def __del__(self):
        self.L.limits_delete(self.table)


@pytest.mark.parametrize("kernels,contexts", [(39, 1), (39, 2), (40, 8), (200, 3)])
def test_limits_never_go_down(limits, kernels, contexts):
    d = Driver(limits)
    rng = random.Random(kernels + contexts)
    # everything at a long sequence once, then at short ones in any order
    for c in range(contexts):
        for k in range(kernels):
            assert d.ask(0x1000 + 16 * k, 64 * c + 5, 200000 + k)
    for _ in range(2000):
        assert d.ask(0x1000 + 16 * rng.randrange(kernels), 64 * rng.randrange(contexts) + 5, rng.choice([50000, 100000, 230000]))


def test_a_limit_is_set_once(limits):
    d = Driver(limits)
    for _ in range(5):
        for k in range(100):
            assert d.ask(0x1000 + 16 * k, 7, 150000)
    assert d.calls == 100


def test_unknown_context(limits):
    """Without a context's name the limit is set each time, and still never down."""
    d = Driver(limits)
    for n in (200000, 60000, 100000, 210000, 50000):
        assert d.ask(0x1000, 3, n, known=False)
    assert d.attr[0x1000, 3] == 210000 and d.calls == 5


def test_refused_limit(limits):
    """One that the driver refuses is reported, leaves the kernel as it was and does not spoil later calls."""
    d = Driver(limits, refuse_above=232448)
    assert d.ask(0x1000, 3, 100000)
    assert not d.ask(0x1000, 3, 300000)
    assert d.attr[0x1000, 3] == 100000
    assert d.ask(0x1000, 3, 120000) and d.ask(0x1000, 4, 60000)
    assert not d.ask(0x2000, 3, 300000) and d.ask(0x2000, 3, 90000)
