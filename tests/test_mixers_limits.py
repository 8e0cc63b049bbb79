"""The largest calls of the token mixers that a launch can count (its threads, in 32 bits) pass the shape checks, and the next
larger ones are refused with TL_ERR_SHAPE.  No call here reaches a launch: each lacks a pointer, which is found later."""
from __future__ import annotations

import ctypes
import os

import pytest

import quantized_gemv_gemm_amd as tl

pytestmark = pytest.mark.skipif(not os.path.exists(tl.LIB_PATH), reason="libtl.so not built")
SHAPE, NULLPTR = 2, 1


def P(n):
    return ctypes.c_void_p((n + 1) << 34)


@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("sizes,fits", [
    (dict(T=(1 << 18) - 16, H=1024), True), (dict(T=(1 << 18) - 15, H=1024), False),            # 16 tokens of a head a workgroup
    (dict(T=1 << 20, H=1, Hq=1016, D=64), True), (dict(T=1 << 20, H=1, Hq=1020, D=64), False),   # 64 rows of q, and 2^16 for k and v
    (dict(T=1 << 20, H=1, Hq=254, D=256), True), (dict(T=1 << 20, H=1, Hq=255, D=256), False)], ids=str)
def test_write(sizes, fits, norm):
    s = {**dict(Hq=0, D=64), **sizes}
    T, H, Hq, D = (s[n] for n in ("T", "H", "Hq", "D"))
    q, qo = (P(3), P(4)) if Hq else (None, None)
    far = max(H, Hq) * D
    if norm:
        got = tl.lib().tl_kv_write_norm(P(0), far, P(1), far, None, T, H, D, q, far, D, Hq, None, None, 1e-6, None, 1, None, None, 0, 0, qo,
                                        P(5), P(6), None, None, tl.TL_BF16, 4, 16, None)
    else:
        got = tl.lib().tl_kv_write(P(0), far, P(1), far, None, T, H, D, q, far, Hq, None, None, 0, 0, qo, P(5), P(6), None, None,
                                   tl.TL_BF16, 4, 16, None)
    assert got == (NULLPTR if fits else SHAPE)


@pytest.mark.parametrize("T,R,fits", [((1 << 30) - 64, 0, True), ((1 << 30) - 65, 1, True), ((1 << 30) - 64, 1, False), (1 << 30, 1, False)])
def test_conv(T, R, fits):
    got = tl.lib().tl_short_conv(None, 8, T, 8, P(1), 4, None, P(2), P(3), P(4), R, None, 0, 64, 1e-6, P(5), 4, P(6), 8, None)
    assert got == (0 if R == 0 else NULLPTR if fits else SHAPE)


@pytest.mark.parametrize("form,sizes,fits", [
    ("step", dict(R=4095, Hk=4096), True), ("step", dict(R=4096, Hk=4096), False),
    ("step", dict(R=4095, Hk=512, G=4, Dv=64), True), ("step", dict(R=4096, Hk=512, G=4, Dv=64), False),
    ("chunk", dict(R=4095, Hk=2048, Dv=128), True), ("chunk", dict(R=4096, Hk=2048, Dv=128), False),
    ("chunk", dict(R=4095, Hk=1024, Dv=144), True), ("chunk", dict(R=4096, Hk=1024, Dv=144), False),
    ("tree", dict(R=4095, Hk=2048), True), ("tree", dict(R=4096, Hk=2048), False),
    ("scan", dict(R=4095, Hk=2048, Dv=32), True), ("scan", dict(R=4096, Hk=2048, Dv=32), False),
    ("scan", dict(R=1, Hk=1, G=65535, Dv=512), True), ("scan", dict(R=1, Hk=1, G=65535, Dv=528), False),
    ("scan", dict(R=1, Hk=1, T=(1 << 30) - 65), True), ("scan", dict(R=1, Hk=1, T=1 << 30), False)], ids=str)
def test_delta(form, sizes, fits):
    s = {**dict(G=1, Dv=32, T=9), **sizes}
    T, R, Hk, G, Dv = (s[n] for n in ("T", "R", "Hk", "G", "Dv"))
    nodes, mask = dict(step=(6, None), chunk=(64, None), tree=(64, P(9)), scan=(65, None))[form]
    got = tl.lib().tl_delta_rule(None, Hk * 64, P(1), Hk * 64, P(2), Hk * G * Dv, P(3), Hk * G, P(4), Hk * G, None, None, T, Hk, G, 64, Dv,
                                 P(5), P(6), P(7), R, mask, 0.1, P(8), 1, nodes, P(10), P(11), 1 << 62, None)
    assert got == (NULLPTR if fits else SHAPE)


@pytest.mark.parametrize("sizes,fits", [
    (dict(L=4096, R=4095), True), (dict(L=4096, R=4096), False), (dict(L=48, R=2750, Hk=32, Dv=128), False),
    (dict(L=32, R=4096, Hk=31, Dv=128), True), (dict(L=32, R=4096, Hk=32, Dv=128), False),
    (dict(L=4096, R=2047, C=2048), True), (dict(L=4096, R=2048, C=2048), False), (dict(L=4096, R=2047, C=2056), False)], ids=str)
def test_commit(sizes, fits):
    s = {**dict(Hk=1, Dv=32, C=0), **sizes}
    L, R, Hk, Dv, C = (s[n] for n in ("L", "R", "Hk", "Dv", "C"))
    x, conv = (P(9), P(10)) if C else (None, None)
    got = tl.lib().tl_delta_commit(None, P(1), 9, P(2), P(3), P(4), R, 9, L, P(5), Hk * 64, 0, P(6), Hk * Dv, 0, P(7), Hk, 0, P(8), Hk, 0, None,
                                   None, Hk, 1, 64, Dv, P(11), 1, x, C, 0, C, 4, conv, None)
    assert got == (NULLPTR if fits else SHAPE)
