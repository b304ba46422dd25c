"""Host side of the rotary, paged-attention and page calls (no GPU): struct layouts, refusals, frequencies."""
import ctypes
import math
import os

import numpy as np
import pytest

import dsa_sparse_mla_gb300 as hs
from dsa_sparse_mla_gb300 import build
from test_abi import ROOT, _struct_fields

STRUCTS = {"hs_rope_args": "_RopeArgs", "hs_paged_mla_args": "_PagedMlaArgs", "hs_kv_copy_args": "_CopyArgs",
           "hs_kv_fork_args": "_ForkArgs", "hs_kv_free_args": "_FreeArgs", "hs_kv_compact_args": "_CompactArgs"}


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return hs.load()


def test_structs_match_the_binding(tmp_path):
    import subprocess
    with open(os.path.join(ROOT, "include", "hs.h")) as f:
        text = f.read()
    lines = ["#include <stddef.h>", "#include <stdio.h>", '#include "hs.h"', "int main(void) {"]
    for c in STRUCTS:
        lines.append('printf("%s size %%zu\\n", sizeof(%s));' % (c, c))
        lines += ['printf("%s %s %%zu\\n", offsetof(%s, %s));' % (c, f, c, f) for f in _struct_fields(text, c)]
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text("\n".join(lines + ["return 0;", "}"]) + "\n")
    subprocess.run(["gcc", "-std=c11", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = {tuple(ln.split()[:2]): int(ln.split()[2]) for ln in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.splitlines()}
    for c, name in STRUCTS.items():
        cls = getattr(hs, name)
        assert [f[0] for f in cls._fields_] == _struct_fields(text, c)
        assert ctypes.sizeof(cls) == got[(c, "size")]
        for f in cls._fields_:
            assert getattr(cls, f[0]).offset == got[(c, f[0])], (c, f[0])


def refused(call, args, word):
    st = call(ctypes.byref(args) if args is not None else None, None)
    return st == 1 and word.encode() in hs.load().hs_last_error()


def good(cls, **kw):
    a = cls()
    for name, t in cls._fields_:
        setattr(a, name, 16 if t is ctypes.c_void_p else 1)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("change,word", [
    (dict(T=-1), "T"), (dict(H=0), "H"), (dict(rot=0), "rot"), (dict(rot=7), "rot"), (dict(rot=514), "rot"), (dict(dtype=3), "dtype"),
    (dict(scale=math.nan), "scale"), (dict(x=None), "NULL"), (dict(positions=None), "NULL"), (dict(inv_freq=None), "NULL"),
    (dict(x_stride_t=-1), "strides"), (dict(y_out=None), "y_out"), (dict(H2=0), "H2"), (dict(x=17), "aligned"), (dict(y_stride_h=-4), "strides")])
def test_rope_refuses(change, word):
    assert refused(hs.load().hs_rope, good(hs._RopeArgs, **{"rot": 64, "dtype": 0, **change}), word)


@pytest.mark.parametrize("change,word", [
    (dict(T=-1), "T"), (dict(B=0), "B"), (dict(B=4097), "B"), (dict(H=0), "H must"), (dict(H=129), "H must"), (dict(kv_tokens=-1), "kv_tokens"),
    (dict(err_flag=None), "err_flag"), (dict(q=None), "NULL"), (dict(workspace=None), "NULL"), (dict(q=8), "aligned"), (dict(out=24), "aligned"),
    (dict(R=0), "R must"), (dict(R=2 ** 31), "R must"), (dict(bt_stride=0), "bt_stride"), (dict(softmax_scale=math.inf), "softmax_scale"),
    (dict(T=2 ** 30, H=2), "T * H")])
def test_paged_mla_refuses(change, word):
    assert refused(hs.load().hs_paged_mla_fwd, good(hs._PagedMlaArgs, **change), word)


def test_page_calls_refuse():
    L = hs.load()
    for call, cls in ((L.hs_kv_copy_pages, hs._CopyArgs), (L.hs_kv_fork, hs._ForkArgs), (L.hs_kv_compact, hs._CompactArgs)):
        assert refused(call, None, "NULL")
        assert refused(call, good(cls, err_flag=None, Di=64), "err_flag")
        assert refused(call, good(cls, Di=32), "Di must")
        assert refused(call, good(cls, Di=64, pools=None), "pools")
        assert refused(call, good(cls, Di=64, k_scales=None), "k_scales")
        assert refused(call, good(cls, Di=64, L=-1), "L, Li")
        assert refused(call, good(cls, Di=64, nblk=0), "nblk")
        assert refused(call, good(cls, Di=64, src=None), "NULL")
    assert refused(L.hs_kv_copy_pages, good(hs._CopyArgs, n=-1), "n must")
    assert refused(L.hs_kv_fork, good(hs._ForkArgs, n=8193), "n must")
    assert refused(L.hs_kv_free, good(hs._FreeArgs, n=-1), "n must")
    assert refused(L.hs_kv_free, good(hs._FreeArgs, refcount=None), "NULL")
    assert refused(L.hs_kv_compact, good(hs._CompactArgs, Di=64, workspace_bytes=4), "workspace")
    assert refused(L.hs_kv_compact, good(hs._CompactArgs, Di=64, B=-1), "B")
    n = ctypes.c_uint64(0)
    assert L.hs_kv_compact_workspace_size(0, ctypes.byref(n)) == 1
    assert L.hs_kv_compact_workspace_size(1500, ctypes.byref(n)) == 0 and n.value == 4 * (1500 + 2)


def test_nothing_to_do_is_fine():
    L = hs.load()
    for call, a in ((L.hs_rope, good(hs._RopeArgs, rot=64, dtype=0, T=0)), (L.hs_paged_mla_fwd, good(hs._PagedMlaArgs, T=0)),
                    (L.hs_kv_copy_pages, good(hs._CopyArgs, n=0)), (L.hs_kv_fork, good(hs._ForkArgs, n=0)), (L.hs_kv_free, good(hs._FreeArgs, n=0))):
        assert call(ctypes.byref(a), None) == 0


def test_frequencies():
    f, s = hs.hs_rope_inv_freq(64)
    i = np.arange(32)
    np.testing.assert_allclose(f.numpy(), 10000.0 ** (-2.0 * i / 64), rtol=1e-15)
    assert s == 1.0
    g, s = hs.hs_rope_inv_freq(64, kind="linear", factor=8.0)
    np.testing.assert_allclose(g.numpy(), f.numpy() / 8.0, rtol=1e-15)
    g, s = hs.hs_rope_inv_freq(64, base=10000.0, kind="yarn", factor=16.0, original=4096)
    assert abs(s - (0.1 * math.log(16.0) + 1.0)) < 1e-6
    turns = 4096 * f.numpy() / (2 * math.pi)                        # of each pair within the original context
    assert np.all(g.numpy()[turns > 64] == f.numpy()[turns > 64])
    np.testing.assert_allclose(g.numpy()[turns < 0.5], f.numpy()[turns < 0.5] / 16.0, rtol=1e-14)
    assert np.all(np.diff(g.numpy()) < 0)
    lo, hi = [64 * math.log(4096 / (b * 2 * math.pi)) / (2 * math.log(10000.0)) for b in (32.0, 1.0)]
    ramp = np.clip((i - math.floor(lo)) / (math.ceil(hi) - math.floor(lo)), 0, 1)
    np.testing.assert_allclose(g.numpy(), f.numpy() * (ramp / 16.0 + 1 - ramp), rtol=1e-14)
    for bad in (dict(rot=5), dict(rot=64, base=1.0), dict(rot=64, kind="linear", factor=0.5), dict(rot=64, kind="other"),
                dict(rot=64, kind="yarn", factor=2.0, original=0), dict(rot=64, kind="yarn", factor=2.0, beta_fast=1.0, beta_slow=2.0)):
        with pytest.raises(hs.HSError):
            hs.hs_rope_inv_freq(**bad)


def test_plain_pages_by_hand():
    """The tests' own plain versions on a case worked by hand."""
    import plain_ops as plain
    layers = {"pool": np.zeros((0, 0, 656), np.uint8), "keys": np.zeros((0, 6, 64, 64), np.uint8), "key_scale": np.zeros((0, 6, 64), np.float32)}
    table, seq = np.array([[4, 5, -1], [-1, -1, -1], [-1, -1, -1]], np.int32), np.array([70, 0, 0], np.int32)
    ref = np.array([0, 0, 0, 0, 1, 1], np.int32)
    src, dst, short = plain.fork([0, 0], [2, 1], table, seq, ref, layers)
    assert not short and src.tolist() == [5, 5] and dst.tolist() == [0, 1]
    assert table.tolist() == [[4, 5, -1], [4, 1, -1], [4, 0, -1]] and ref.tolist() == [1, 1, 0, 0, 3, 1] and seq.tolist() == [70] * 3
    assert not plain.free([0], table, seq, ref) and ref.tolist() == [1, 1, 0, 0, 2, 0]
    s, d, k = plain.compact(table, ref, layers)
    assert k.tolist() == [3, 1] and s[0] == 4 and d[0] == 2 and table.tolist()[1:] == [[2, 1, -1], [2, 0, -1]]
    assert ref.tolist() == [1, 1, 2, 0, 0, 0]
