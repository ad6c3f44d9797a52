"""The packed cache's and the pages' operators on the host: struct layouts against the C
compiler's, sizes, the documented layout, and refusals (nothing here reaches a launch)."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest

import kv_cache_block_lowrank_gb300 as hss
from packed_util import key_place, scale_place, tile_bytes, value_place

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


@pytest.mark.parametrize("name", ["hss_norm_rope_args", "hss_pack_args", "hss_packed_args"])
def test_structs_match_c_layout(name, tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    struct = getattr(hss, name)
    fields = [f for f, _ in struct._fields_]
    lines = [f'printf("%zu\\n", offsetof({name}, {f}));' for f in fields]
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "hss.h"\nint main(void){'
                   + "".join(lines) + f'printf("%zu\\n", sizeof({name}));return 0;}}\n')
    exe = tmp_path / "layout"
    subprocess.run([cc, "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)],
                   check=True)
    got = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True,
                                          check=True).stdout.split()]
    assert got == [getattr(struct, f).offset for f in fields] + [ctypes.sizeof(struct)]


@pytest.mark.parametrize("hd", [64, 128, 192, 256])
def test_layout_has_a_place_for_everything(hd):
    seen = set()
    owner = {}
    for t in range(16):
        for d in range(hd):
            for what, (byte, half) in (("k", key_place(t, d, hd)), ("v", value_place(t, d, hd))):
                assert 0 <= byte < 16 * hd
                assert (byte, half) not in seen
                seen.add((byte, half))
                assert owner.setdefault(byte, (what, t)) == (what, t)  # no byte holds two tokens
        for group in range(hd // 32):
            for value in (False, True):
                at = scale_place(t, group, hd, value)
                for byte in (2 * at, 2 * at + 1):
                    assert 16 * hd <= byte < tile_bytes(hd) and (byte, 0) not in seen
                    seen.add((byte, 0))
    assert len(seen) == 2 * 16 * hd + 2 * hd
    assert hss.hss_packed_page_bytes(dims(head_dim=hd, block_size=48)) == 8 * 3 * tile_bytes(hd)
    assert hss.hss_packed_page_bytes(dims(head_dim=96)) == 0


def test_workspace_sizes():
    f = hss.hss_attend_packed_workspace_bytes
    for hd in (64, 256):
        n = f(dims(head_dim=hd), 64, 16, 1 << 20, 0, 0)
        assert 0 < n < 1 << 31
        assert f(dims(head_dim=hd), 1, 1, 1, 0, 0) <= n
        assert f(dims(head_dim=hd), 0, 0, 0, 0, 0) <= n
    for bad in ((-1, 1, 1, 0, 0), (1, -1, 1, 0, 0), (1, 1, -1, 0, 0), (1, 1, 1, -1, 0),
                (1, 1, 1, 0, -1)):
        assert f(dims(), *bad) == 0
    assert f(dims(head_dim=100), 1, 1, 1, 0, 0) == 0
    assert hss.hss_fork_pages_workspace_bytes(-1, 5) == 0
    assert hss.hss_fork_pages_workspace_bytes(7, 100) > 0
    assert hss.hss_compact_pages_workspace_bytes(-1) == 0
    assert hss.hss_compact_pages_workspace_bytes(1 << 30) > 1 << 30


def norm(tokens=4, rot=128, layout=0, strides=(4096, 1024, 1024), weights=(0, 0), eps=1e-6,
         offset=0.0, q=FAKE, k=FAKE, v=FAKE, qw=FAKE, kw=FAKE, q_out=FAKE, d=None, slots=FAKE,
         turns=FAKE):
    call = hss.NormRopeTokens(d or dims(), rot, layout, turns, 1.0, FAKE, slots, tokens, *strides,
                              *weights, eps, offset)
    call(q, k, v, qw, kw, q_out, None, FAKE, FAKE, stream=0)


@pytest.mark.parametrize("kw,want", [
    (dict(eps=-1e-6), "INVALID_ARGUMENT"), (dict(eps=float("nan")), "INVALID_ARGUMENT"),
    (dict(eps=float("inf")), "INVALID_ARGUMENT"), (dict(offset=float("nan")), "INVALID_ARGUMENT"),
    (dict(weights=(120, 0)), "INVALID_ARGUMENT"), (dict(weights=(0, 132)), "INVALID_ARGUMENT"),
    (dict(weights=(-128, 0)), "INVALID_ARGUMENT"), (dict(qw=FAKE + 8), "MISALIGNED"),
    (dict(kw=FAKE + 2), "MISALIGNED"), (dict(rot=130), "INVALID_ARGUMENT"),
    (dict(rot=3), "INVALID_ARGUMENT"), (dict(layout=2), "INVALID_ARGUMENT"),
    (dict(tokens=-1), "INVALID_ARGUMENT"), (dict(strides=(4088, 1024, 1024)), "INVALID_ARGUMENT"),
    (dict(strides=(4096, 1024, 1028)), "INVALID_ARGUMENT"), (dict(q=None), "NULL_POINTER"),
    (dict(v=None), "NULL_POINTER"), (dict(slots=None), "NULL_POINTER"),
    (dict(turns=None), "NULL_POINTER"), (dict(k=FAKE + 8), "MISALIGNED"),
    (dict(d=dims(head_dim=96)), "UNSUPPORTED_SHAPE"), (dict(d=dims(num_q_heads=33)),
                                                       "INVALID_DIMS")])
def test_norm_rope_refusals(kw, want):
    assert status_of(norm, **kw) == getattr(hss, "HSS_ERR_" + want)


def pack(d=None, tokens=4, strides=(1024, 1024), slots=FAKE, k=FAKE, v=FAKE, cache=FAKE,
         back=False, status=None):
    call = hss.PackTokens(d or dims(), slots, tokens, *strides, dev_status=status)
    if back:
        call.unpack(cache, k, v, stream=0)
    else:
        call.pack(k, v, cache, stream=0)


@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("kw,want", [
    (dict(tokens=-1), "INVALID_ARGUMENT"), (dict(tokens=(1 << 30) + 1), "INVALID_ARGUMENT"),
    (dict(strides=(1016, 1024)), "INVALID_ARGUMENT"),
    (dict(strides=(1024, 1025)), "INVALID_ARGUMENT"), (dict(slots=None), "NULL_POINTER"),
    (dict(cache=None), "NULL_POINTER"), (dict(k=FAKE + 2), "MISALIGNED"),
    (dict(v=FAKE + 8), "MISALIGNED"), (dict(cache=FAKE + 8), "MISALIGNED"),
    (dict(slots=FAKE + 4), "MISALIGNED"), (dict(status=FAKE + 2), "MISALIGNED"),
    (dict(d=dims(block_size=8)), "UNSUPPORTED_SHAPE"), (dict(d=dims(max_blocks=0)),
                                                        "INVALID_DIMS")])
def test_pack_refusals(back, kw, want):
    assert status_of(pack, back=back, **kw) == getattr(hss, "HSS_ERR_" + want)


def test_pack_of_nothing_is_no_call():
    pack(tokens=0, slots=None, cache=None)
    pack(k=None, v=None, slots=None, cache=None)
    pack(back=True, tokens=0, slots=None, cache=None)


def attend(d=None, total_q=4, max_q=4, num_seqs=1, total_blocks=8, window=0, sinks=0, scale=0.1,
           q=FAKE, cache=FAKE, out=FAKE, lse=None, work=FAKE, size=None, table=FAKE, offs=FAKE,
           ctx=FAKE, q_offs=FAKE, status=None):
    d = d or dims()
    if size is None:
        size = hss.hss_attend_packed_workspace_bytes(d, max(num_seqs, 0), max(max_q, 0),
                                                     max(total_blocks, 0), max(window, 0),
                                                     max(sinks, 0))
    call = hss.AttendPacked(d, q_offs, total_q, max_q, table, offs, ctx, num_seqs, total_blocks,
                            window, sinks, scale, work, size, status)
    call(q, cache, out, lse, stream=0)


@pytest.mark.parametrize("kw,want", [
    (dict(total_q=-1), "INVALID_ARGUMENT"), (dict(max_q=-1), "INVALID_ARGUMENT"),
    (dict(num_seqs=-1), "INVALID_ARGUMENT"), (dict(total_blocks=-1), "INVALID_ARGUMENT"),
    (dict(total_blocks=1 << 31), "INVALID_ARGUMENT"), (dict(window=-1), "INVALID_ARGUMENT"),
    (dict(sinks=-1), "INVALID_ARGUMENT"), (dict(total_q=5), "INVALID_ARGUMENT"),
    (dict(num_seqs=0, total_q=0), "INVALID_ARGUMENT"),
    (dict(scale=float("nan")), "INVALID_ARGUMENT"), (dict(scale=float("inf")), "INVALID_ARGUMENT"),
    (dict(max_q=1 << 30, total_q=1 << 30, size=1 << 60), "INVALID_ARGUMENT"),
    (dict(q=None), "NULL_POINTER"), (dict(cache=None), "NULL_POINTER"),
    (dict(out=None), "NULL_POINTER"), (dict(work=None), "NULL_POINTER"),
    (dict(table=None), "NULL_POINTER"), (dict(offs=None), "NULL_POINTER"),
    (dict(ctx=None), "NULL_POINTER"), (dict(q_offs=None), "NULL_POINTER"),
    (dict(q=FAKE + 8), "MISALIGNED"), (dict(cache=FAKE + 8), "MISALIGNED"),
    (dict(out=FAKE + 8), "MISALIGNED"), (dict(lse=FAKE + 2), "MISALIGNED"),
    (dict(work=FAKE + 128), "MISALIGNED"), (dict(status=FAKE + 1), "MISALIGNED"),
    (dict(size=1000), "WORKSPACE_TOO_SMALL"),
    (dict(d=dims(num_q_heads=129, num_kv_heads=1)), "UNSUPPORTED_SHAPE")])
def test_attend_packed_refusals(kw, want):
    assert status_of(attend, **kw) == getattr(hss, "HSS_ERR_" + want)


def test_attend_of_no_rows_is_no_call():
    attend(total_q=0, q=None, cache=None, out=None, work=None, table=None)


def fork(num_seqs=2, total=8, pages=16, num_released=0, new=3, bs=16, room=32, size=None, **kw):
    p = dict(table=FAKE, offs=FAKE, refs=FAKE, released=None, parents=FAKE, lengths=FAKE,
             rooms=FAKE, new_table=FAKE, new_offs=FAKE, new_refs=FAKE, src=FAKE, dst=FAKE,
             counts=FAKE, work=FAKE)
    p.update(kw)
    if size is None:
        size = 1 << 40
    hss.hss_fork_pages(p["table"], p["offs"], num_seqs, total, p["refs"], pages, p["released"],
                       num_released, p["parents"], p["lengths"], p["rooms"], new, bs, room,
                       p["new_table"], p["new_offs"], p["new_refs"], p["src"], p["dst"],
                       p["counts"], p["work"], size, stream=0)


@pytest.mark.parametrize("kw,want", [
    (dict(num_seqs=-1), "INVALID_ARGUMENT"), (dict(num_seqs=(1 << 20) + 1), "INVALID_ARGUMENT"),
    (dict(new=-1), "INVALID_ARGUMENT"), (dict(total=-1), "INVALID_ARGUMENT"),
    (dict(pages=(1 << 30) + 1), "INVALID_ARGUMENT"), (dict(num_released=-1), "INVALID_ARGUMENT"),
    (dict(room=-1), "INVALID_ARGUMENT"), (dict(bs=0), "INVALID_ARGUMENT"),
    (dict(num_seqs=0), "INVALID_ARGUMENT"), (dict(num_released=2), "NULL_POINTER"),
    (dict(table=None), "NULL_POINTER"), (dict(offs=None), "NULL_POINTER"),
    (dict(refs=None), "NULL_POINTER"), (dict(parents=None), "NULL_POINTER"),
    (dict(lengths=None), "NULL_POINTER"), (dict(rooms=None), "NULL_POINTER"),
    (dict(new_table=None), "NULL_POINTER"), (dict(new_offs=None), "NULL_POINTER"),
    (dict(new_refs=None), "NULL_POINTER"), (dict(src=None), "NULL_POINTER"),
    (dict(dst=None), "NULL_POINTER"), (dict(counts=None), "NULL_POINTER"),
    (dict(work=None), "NULL_POINTER"), (dict(work=FAKE + 2), "MISALIGNED"),
    (dict(counts=FAKE + 1), "MISALIGNED"), (dict(refs=FAKE + 2), "MISALIGNED"),
    (dict(size=10), "WORKSPACE_TOO_SMALL")])
def test_fork_refusals(kw, want):
    assert status_of(fork, **kw) == getattr(hss, "HSS_ERR_" + want)


def compact(total=8, pages=16, room=4, size=1 << 40, **kw):
    p = dict(table=FAKE, refs=FAKE, new_table=FAKE, new_refs=FAKE, src=FAKE, dst=FAKE,
             counts=FAKE, work=FAKE)
    p.update(kw)
    hss.hss_compact_pages(p["table"], total, p["refs"], pages, room, p["new_table"],
                          p["new_refs"], p["src"], p["dst"], p["counts"], p["work"], size,
                          stream=0)


@pytest.mark.parametrize("kw,want", [
    (dict(total=-1), "INVALID_ARGUMENT"), (dict(pages=-1), "INVALID_ARGUMENT"),
    (dict(room=-1), "INVALID_ARGUMENT"), (dict(room=(1 << 30) + 1), "INVALID_ARGUMENT"),
    (dict(table=None), "NULL_POINTER"), (dict(new_table=None), "NULL_POINTER"),
    (dict(refs=None), "NULL_POINTER"), (dict(new_refs=None), "NULL_POINTER"),
    (dict(src=None), "NULL_POINTER"), (dict(dst=None), "NULL_POINTER"),
    (dict(counts=None), "NULL_POINTER"), (dict(work=None), "NULL_POINTER"),
    (dict(src=FAKE + 2), "MISALIGNED"), (dict(size=100), "WORKSPACE_TOO_SMALL")])
def test_compact_refusals(kw, want):
    assert status_of(compact, **kw) == getattr(hss, "HSS_ERR_" + want)


def copy(most=4, page=64, pages=8, layers=1, src=FAKE, dst=FAKE, count=None, a=FAKE, b=None):
    hss.hss_copy_pages(src, dst, count, most, a, b, page, pages, layers, stream=0)


@pytest.mark.parametrize("kw,want", [
    (dict(most=-1), "INVALID_ARGUMENT"), (dict(page=0), "INVALID_ARGUMENT"),
    (dict(page=24), "INVALID_ARGUMENT"), (dict(page=(1 << 30) + 16), "INVALID_ARGUMENT"),
    (dict(pages=-1), "INVALID_ARGUMENT"), (dict(layers=0), "INVALID_ARGUMENT"),
    (dict(layers=65536), "INVALID_ARGUMENT"), (dict(src=None), "NULL_POINTER"),
    (dict(dst=None), "NULL_POINTER"), (dict(a=None), "NULL_POINTER"),
    (dict(a=FAKE + 8), "MISALIGNED"), (dict(b=FAKE + 8), "MISALIGNED"),
    (dict(count=FAKE + 2), "MISALIGNED"), (dict(src=FAKE + 1), "MISALIGNED")])
def test_copy_refusals(kw, want):
    assert status_of(copy, **kw) == getattr(hss, "HSS_ERR_" + want)


def test_copy_of_nothing_is_no_call():
    copy(most=0, src=None, dst=None, a=None)


def test_quantise_reference_halfway_cases():
    """(the plain definition itself: ties to even, no code past 7, NaN for a group with one)"""
    from packed_util import quantise

    x = np.zeros(64)
    x[:4] = [7.0, 0.5, 1.5, -2.5]
    x[32] = np.inf
    codes, scales = quantise(x)
    assert scales[0] == 1.0 and list(codes[:4]) == [7, 0, 2, -2]
    assert np.isnan(scales[1]) and (codes[32:] == 0).all()
