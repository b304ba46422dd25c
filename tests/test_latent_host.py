"""hs_kv_read, the head products and the expanded attention without a GPU: refusals of bad arguments, and the argument structures."""
import ctypes
import os
import subprocess

import pytest
import torch

import dsa_sparse_mla_gb300 as hs
import test_abi
from dsa_sparse_mla_gb300 import build

STRUCTS = {"hs_kv_read_args": "_KvReadArgs", "hs_mla_heads_args": "_MlaHeadsArgs", "hs_mla_expand_args": "_MlaExpandArgs",
           "hs_mla_expanded_args": "_MlaExpandedArgs"}


@pytest.fixture(scope="module")
def L():
    build.build()
    return hs.load()


def refused(L, call, a, word):
    st = call(ctypes.byref(a), None)
    assert st == 1 and word in L.hs_last_error(), (st, L.hs_last_error())


def read_args():
    a = hs._KvReadArgs()
    a.B, a.bt_stride, a.R, a.n, a.out_stride = 1, 1, 64, 5, 576
    a.kv_pool = a.block_table = a.out_start = a.out = a.err_flag = 16
    return a


@pytest.mark.parametrize("field,value,word", [("B", 0, b"B"), ("n", -1, b"n >="), ("n", 2 ** 31, b"n must"), ("dtype", 3, b"dtype"), ("err_flag", None, b"err_flag"),
                                              ("kv_pool", None, b"NULL"), ("block_table", None, b"NULL"), ("out_start", None, b"NULL"),
                                              ("out", None, b"NULL"), ("out", 24, b"aligned"), ("kv_pool", 8, b"aligned"), ("R", 0, b"R"),
                                              ("bt_stride", 0, b"bt_stride"), ("out_stride", 568, b"out_stride"), ("out_stride", 580, b"out_stride")])
def test_read_refuses(L, field, value, word):
    a = read_args()
    setattr(a, field, value)
    refused(L, L.hs_kv_read, a, word)


def test_read_of_nothing(L):
    a = read_args()
    a.n, a.out, a.kv_pool = 0, None, None
    assert L.hs_kv_read(ctypes.byref(a), None) == 0


def heads_args():
    a = hs._MlaHeadsArgs()
    a.T, a.H, a.Dn, a.Dv = 3, 2, 128, 128
    a.x = a.w = a.out = a.err_flag = 16
    a.x_stride_t, a.x_stride_h, a.out_stride_t, a.out_stride_h = 1024, 512, 1024, 512
    return a


@pytest.mark.parametrize("field,value,word", [("T", -1, b"T >="), ("H", 0, b"H in"), ("H", 1025, b"H in"), ("Dn", 96, b"Dn"), ("Dv", 512, b"Dv"),
                                              ("err_flag", None, b"err_flag"), ("x", None, b"NULL"), ("w", None, b"NULL"), ("out", None, b"NULL"),
                                              ("x", 8, b"aligned"), ("w", 18, b"aligned"), ("out", 4, b"aligned"), ("x_stride_t", 1025, b"strides"),
                                              ("x_stride_h", 0, b"strides"), ("out_stride_t", -1024, b"strides"), ("out_stride_h", 4, b"strides"),
                                              ("x_stride_t", 2 ** 38, b"strides")])
def test_products_refuse(L, field, value, word):
    for call in (L.hs_mla_absorb, L.hs_mla_project):
        a = heads_args()
        setattr(a, field, value)
        refused(L, call, a, word)


@pytest.mark.parametrize("field,value,word", [("N", -1, b"N >="), ("H", 0, b"H in"), ("width", 96, b"width"), ("width", 576, b"width"), ("err_flag", None, b"err_flag"),
                                              ("latent", None, b"NULL"), ("w", 8, b"aligned"), ("latent_stride", 504, b"stride"),
                                              ("latent_stride", 516, b"stride"), ("kv_stride", 504, b"stride")])
def test_expand_refuses(L, field, value, word):
    a = hs._MlaExpandArgs()
    a.N, a.H, a.width, a.latent_stride, a.kv_stride = 3, 2, 256, 512, 512
    a.latent = a.w = a.kv = a.err_flag = 16
    setattr(a, field, value)
    refused(L, L.hs_mla_expand, a, word)


def expanded_args():
    a = hs._MlaExpandedArgs()
    a.T, a.B, a.H, a.Dn, a.Dv, a.N = 3, 1, 2, 128, 128, 9
    a.q = a.kv = a.rope = a.req_start = a.kv_start = a.out = a.err_flag = a.workspace = 16
    a.q_stride_t, a.q_stride_h, a.kv_stride, a.rope_stride, a.softmax_scale = 384, 192, 512, 64, 0.1
    return a


@pytest.mark.parametrize("field,value,word", [("T", -1, b"T >="), ("B", 0, b"B in"), ("B", 4097, b"B in"), ("H", 0, b"H must"), ("Dn", 64, b"Dn and Dv"), ("Dv", 256, b"Dn and Dv"),
                                              ("err_flag", None, b"err_flag"), ("q", None, b"NULL"), ("kv", None, b"NULL"), ("rope", None, b"NULL"),
                                              ("req_start", None, b"NULL"), ("kv_start", None, b"NULL"), ("out", None, b"NULL"), ("workspace", None, b"NULL"),
                                              ("q", 8, b"aligned"), ("kv", 2, b"aligned"), ("rope", 4, b"aligned"), ("out", 8, b"aligned"), ("workspace", 4, b"aligned"),
                                              ("N", 0, b"N must"), ("N", 2 ** 31 - 100, b"N must"), ("q_stride_t", 388, b"strides"), ("rope_stride", 0, b"strides"),
                                              ("kv_stride", 504, b"kv_stride"), ("rope_stride", 56, b"rope_stride"), ("softmax_scale", float("nan"), b"finite"),
                                              ("softmax_scale", float("inf"), b"finite"), ("T", 2 ** 30, b"T * H")])
def test_expanded_refuses(L, field, value, word):
    a = expanded_args()
    setattr(a, field, value)
    refused(L, L.hs_mla_expanded_fwd, a, word)


def test_workspace_size_refuses(L):
    n = ctypes.c_uint64(0)
    for B, Dv in ((0, 128), (4097, 128), (1, 64)):
        assert L.hs_mla_expanded_workspace_size(B, Dv, ctypes.byref(n)) == 1
    assert L.hs_mla_expanded_workspace_size(1, 128, None) == 1


def test_host_tensors_are_refused():
    t = torch.zeros((2, 2, 576), dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    for call in (lambda: hs.hs_kv_read(t, i[None], i, t[0], i), lambda: hs.hs_mla_absorb(t, t, t, i), lambda: hs.hs_mla_project(t, t, t, i),
                 lambda: hs.hs_mla_expand(t[0], t, t, i), lambda: hs.hs_mla_expanded_fwd(t, t, t[0], i, i, 1.0, t, i, i)):
        with pytest.raises(hs.HSError):
            call()


def test_argument_structs(tmp_path):
    with open(os.path.join(test_abi.ROOT, "include", "hs.h")) as f:
        text = f.read()
    lines = ["#include <stddef.h>", "#include <stdio.h>", '#include "hs.h"', "int main(void) {"]
    want = []
    for cname, pyname in STRUCTS.items():
        cls = getattr(hs, pyname)
        assert [f[0] for f in cls._fields_] == test_abi._struct_fields(text, cname)
        lines.append('printf("%%zu\\n", sizeof(%s));' % cname)
        want.append(ctypes.sizeof(cls))
        for name, _ in cls._fields_:
            lines.append('printf("%%zu\\n", offsetof(%s, %s));' % (cname, name))
            want.append(getattr(cls, name).offset)
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text("\n".join(lines + ["return 0;", "}"]))
    subprocess.run(["gcc", "-std=c11", "-I", os.path.join(test_abi.ROOT, "include"), str(src), "-o", str(exe)], check=True)
    assert [int(x) for x in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()] == want
