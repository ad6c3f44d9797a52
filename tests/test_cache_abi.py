"""The paged-cache operators on the host: the rope table against a plain calculation, struct
layouts against the C compiler's, and refusals (nothing here reaches a launch)."""
import ctypes
import math
import os
import shutil
import subprocess
from fractions import Fraction

import numpy as np
import pytest

import kv_cache_block_lowrank_gb300 as hss

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x10000  # never dereferenced: every call below fails validation first


@pytest.fixture(scope="module", autouse=True)
def lib():
    from kv_cache_block_lowrank_gb300 import _build

    _build.build()
    return hss.load()


def dims(**kw):
    d = dict(num_layers=1, num_q_heads=32, num_kv_heads=8, head_dim=128, r=32, block_size=16,
             max_blocks=2048)
    d.update(kw)
    return hss.hss_dims(*[d[k] for k in ("num_layers", "num_q_heads", "num_kv_heads", "head_dim",
                                         "r", "block_size", "max_blocks")])


def status_of(fn, *args, **kw):
    with pytest.raises(hss.HssError) as e:
        fn(*args, **kw)
    return e.value.status


def table(rot, scaling=0, base=10000.0, factor=1.0, ctx=0.0, low=0.0, high=0.0):
    out = np.zeros(max(rot // 2, 1) + 1, dtype=np.uint64)
    out[-1] = 77
    hss.hss_rope_table(hss.hss_rope(rot, scaling, base, factor, ctx, low, high),
                       out.ctypes.data)
    assert out[-1] == 77
    return [int(x) for x in out[:-1]]


def turns_of(f):
    return Fraction(f) / Fraction(2 * math.pi) % 1 * 2 ** 64


def close(got, radians):
    # double arithmetic: a few parts in 2^53 of the frequency
    for t, f in zip(got, radians):
        want = turns_of(f)
        off = abs(t - want)
        assert min(off, 2 ** 64 - off) <= 1 + Fraction(f) * 2 ** 64 / 2 ** 50, (t, float(want))


@pytest.mark.parametrize("rot", [2, 4, 32, 74, 128, 256])
def test_rope_table_frequencies(rot):
    plain = [10000.0 ** (-2 * i / rot) for i in range(rot // 2)]
    close(table(rot), plain)
    close(table(rot, hss.HSS_ROPE_SCALE_LINEAR, factor=8.0), [f / 8 for f in plain])
    close(table(rot, hss.HSS_ROPE_SCALE_LINEAR, factor=0.01), [f * 100 for f in plain])
    if rot > 2:
        b = 10000.0 * 4.0 ** (rot / (rot - 2))
        close(table(rot, hss.HSS_ROPE_SCALE_BASE, factor=4.0),
              [b ** (-2 * i / rot) for i in range(rot // 2)])
    ramp = []
    for f in plain:
        w = min(1.0, max(0.0, (8192 * f / (2 * math.pi) - 1.0) / 31.0))
        ramp.append(w * f + (1 - w) * f / 4)
    close(table(rot, hss.HSS_ROPE_SCALE_RAMP, factor=4.0, ctx=8192.0, low=1.0, high=32.0), ramp)


def test_rope_table_first_pair_is_one_radian():
    assert table(2)[0] == pytest.approx(2 ** 64 / (2 * math.pi), rel=1e-15)


@pytest.mark.parametrize("rope", [
    (0, 0, 1e4, 1.0, 0, 0, 0), (3, 0, 1e4, 1.0, 0, 0, 0), (258, 0, 1e4, 1.0, 0, 0, 0),
    (64, 9, 1e4, 1.0, 0, 0, 0), (64, 0, 0.0, 1.0, 0, 0, 0), (64, 0, math.nan, 1.0, 0, 0, 0),
    (64, 0, math.inf, 1.0, 0, 0, 0), (64, 1, 1e4, 0.0, 0, 0, 0), (64, 1, 1e4, -2.0, 0, 0, 0),
    (64, 1, 1e4, math.nan, 0, 0, 0), (2, 2, 1e4, 4.0, 0, 0, 0), (64, 3, 1e4, 4.0, 0, 1, 32),
    (64, 3, 1e4, 4.0, 8192, 32, 32), (64, 3, 1e4, 4.0, 8192, math.nan, 32)])
def test_rope_table_refusals(rope):
    out = np.zeros(128, dtype=np.uint64)
    r = hss.hss_rope(*rope)
    assert status_of(hss.hss_rope_table, r, out.ctypes.data) == hss.HSS_ERR_INVALID_ARGUMENT


def test_rope_table_null():
    assert status_of(hss.hss_rope_table, hss.hss_rope(64, 0, 1e4, 1, 0, 0, 0), None) == \
        hss.HSS_ERR_NULL_POINTER
    assert hss.load().hss_rope_table(None, FAKE) == hss.HSS_ERR_NULL_POINTER


def rope(d=None, rot=128, layout=0, turns=FAKE, magnitude=1.0, pos=FAKE, slots=FAKE, n=4,
         qs=4096, ks=1024, vs=1024, io=(FAKE,) * 7):
    call = hss.RopeTokens(d or dims(), rot, layout, turns, magnitude, pos, slots, n, qs, ks, vs)
    call(*io, stream=0)


def test_rope_tokens_refusals():
    bad = hss.HSS_ERR_INVALID_ARGUMENT
    assert status_of(rope, dims(num_q_heads=9)) == hss.HSS_ERR_INVALID_DIMS
    assert status_of(rope, dims(head_dim=96)) == hss.HSS_ERR_UNSUPPORTED_SHAPE
    for kw in ({"rot": 0}, {"rot": 7}, {"rot": 130}, {"layout": 2}, {"magnitude": math.nan},
               {"n": -1}, {"qs": 4095}, {"qs": 4100}, {"ks": 1016}, {"vs": 8}, {"vs": 2 ** 33}):
        assert status_of(rope, **kw) == bad, kw
    for kw in ({"turns": None}, {"pos": None}, {"slots": None},
               {"io": (None, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE)},
               {"io": (FAKE, None, FAKE, FAKE, FAKE, FAKE, FAKE)},
               {"io": (FAKE, FAKE, None, FAKE, FAKE, FAKE, FAKE)}):
        assert status_of(rope, **kw) == hss.HSS_ERR_NULL_POINTER, kw
    for i in range(7):
        io = [FAKE] * 7
        io[i] += 8
        assert status_of(rope, io=io) == hss.HSS_ERR_MISALIGNED, i
    assert status_of(rope, turns=FAKE + 4) == hss.HSS_ERR_MISALIGNED
    rope(n=0)
    rope(io=(FAKE, FAKE, FAKE, None, None, None, None))  # nothing asked for
    assert hss.load().hss_rope_tokens(None, *[None] * 8) == hss.HSS_ERR_NULL_POINTER


def attend(d=None, qo=FAKE, total_q=4, max_q=4, mask=None, words=0, tab=FAKE, so=FAKE, ctx=FAKE,
           S=1, total=10, scale=1.0, decay=1.0, ws=FAKE, wsb=1 << 40, io=(FAKE,) * 7):
    call = hss.AttendTree(d or dims(), qo, total_q, max_q, mask, words, tab, so, ctx, S, total,
                          scale, decay, ws, wsb)
    call(*io, stream=0)


def test_attend_tree_refusals():
    assert status_of(attend, dims(num_q_heads=9)) == hss.HSS_ERR_INVALID_DIMS
    assert status_of(attend, dims(num_q_heads=129, num_kv_heads=1)) == \
        hss.HSS_ERR_UNSUPPORTED_SHAPE
    for kw in ({"S": -1}, {"max_q": -1}, {"total_q": -1}, {"total": -1}, {"total": 2 ** 31},
               {"total_q": 5}, {"S": 0, "total_q": 0}, {"scale": math.inf}, {"decay": math.nan},
               {"words": -1}, {"mask": FAKE, "words": 0}):
        assert status_of(attend, **kw) == hss.HSS_ERR_INVALID_ARGUMENT, kw
    for kw in ({"qo": None}, {"tab": None}, {"so": None}, {"ctx": None}, {"ws": None},
               {"io": (None,) + (FAKE,) * 6}, {"io": (FAKE, None) + (FAKE,) * 5},
               {"io": (FAKE, FAKE, None) + (FAKE,) * 4},
               {"io": (FAKE, FAKE, FAKE, None) + (FAKE,) * 3}):
        assert status_of(attend, **kw) == hss.HSS_ERR_NULL_POINTER, kw
    for kw in ({"io": (FAKE + 2,) + (FAKE,) * 6}, {"mask": FAKE + 4, "words": 1},
               {"ws": FAKE + 16}, {"io": (FAKE,) * 4 + (FAKE + 2, FAKE, FAKE)}):
        assert status_of(attend, **kw) == hss.HSS_ERR_MISALIGNED, kw
    need = hss.hss_attend_tree_workspace_bytes(dims(), 1, 4, 10, True)
    assert need > 0
    assert status_of(attend, wsb=need - 1) == hss.HSS_ERR_WORKSPACE_TOO_SMALL
    attend(S=0, total_q=0, total=0)  # nothing to do
    assert hss.load().hss_attend_tree(None, *[None] * 8) == hss.HSS_ERR_NULL_POINTER


def test_attend_workspace_bytes():
    size = hss.hss_attend_tree_workspace_bytes
    assert size(dims(num_q_heads=9), 1, 1, 1, True) == 0
    assert size(dims(), -1, 1, 1, True) == 0 and size(dims(), 1, -1, 1, True) == 0
    small = size(dims(), 2, 4, 100, True)
    assert small <= size(dims(), 3, 4, 100, True) and small <= size(dims(), 2, 5, 100, True)
    assert small <= size(dims(), 2, 4, 101, True) and size(dims(), 2, 4, 100, False) <= small


def evict(**kw):
    a = dict(weights=FAKE, table=FAKE, offs=FAKE, ctx=FAKE, budgets=FAKE, S=2, total=10, bs=16,
             first=1, last=1, nt=FAKE, no=FAKE, nw=FAKE, nc=FAKE, freed=FAKE, fo=FAKE)
    a.update(kw)
    hss.hss_evict_blocks(*a.values(), stream=0)


def test_evict_refusals():
    for kw in ({"S": -1}, {"total": -1}, {"total": 2 ** 30 + 1}, {"bs": 0}, {"first": -1},
               {"last": -1}, {"S": 0}):
        assert status_of(evict, **kw) == hss.HSS_ERR_INVALID_ARGUMENT, kw
    for name in ("weights", "table", "offs", "ctx", "budgets", "nt", "no", "nw", "nc", "freed",
                 "fo"):
        assert status_of(evict, **{name: None}) == hss.HSS_ERR_NULL_POINTER, name
        assert status_of(evict, **{name: FAKE + 2}) == hss.HSS_ERR_MISALIGNED, name
    evict(S=0, total=0)


@pytest.mark.parametrize("name", ["hss_rope", "hss_rope_args", "hss_attend_args"])
def test_struct_layouts(name, tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    cls = getattr(hss, name)
    fields = [f for f, _ in cls._fields_]
    src = tmp_path / "layout.c"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "hss.h"\nint main(void) {\n'
                   f'  printf("%zu\\n", sizeof({name}));\n' +
                   "".join(f'  printf("%zu\\n", offsetof({name}, {f}));\n' for f in fields) +
                   "  return 0;\n}\n")
    exe = tmp_path / "layout"
    subprocess.run([cc, "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)],
                   check=True)
    got = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True,
                                          check=True).stdout.split()]
    assert got == [ctypes.sizeof(cls)] + [getattr(cls, f).offset for f in fields]
