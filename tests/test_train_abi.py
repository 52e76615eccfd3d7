"""Host side of the operators that close a training step (cross entropy of a linear head, Muon's update):
size queries and refusals.  No call here launches a kernel."""
import ctypes
import os
import shutil
import subprocess

import pytest
import torch

from latent_compressed_expert_gb300 import build, lmoe

# Fake device addresses that the host-side checks must turn down before any CUDA call: not on a
# machine with a GPU, where a check that let one through would touch them.
no_gpu = pytest.mark.skipif(torch.cuda.is_available(),
                            reason="fake-pointer host checks run on CPU-only machines")
OK, ARG, UNSUP, SMALL = (lmoe.LMOE_OK, lmoe.LMOE_ERR_INVALID_ARG, lmoe.LMOE_ERR_UNSUPPORTED,
                         lmoe.LMOE_ERR_WORKSPACE_TOO_SMALL)
BUF = {n: 0x100000 * (i + 1) for i, n in enumerate(
    ("x", "w", "target", "loss", "lse", "flag", "ws", "dloss", "dx", "dw", "grad", "out", "momentum",
     "master"))}
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    build.build()
    return lmoe.load()


def _fill(d, p, a):
    p.update(a)
    for k, v in p.items():
        setattr(d, k, v)
    return d


def _xent(**a):
    return _fill(lmoe.LinearXentDesc(), dict(
        M=8, V=300, K=64, x=BUF["x"], ldx=64, w=BUF["w"], ldw=64, target=BUF["target"],
        target_type=lmoe.I64, loss=BUF["loss"], lse=BUF["lse"], dev_flag=BUF["flag"]), a)


SIZES = [
    (dict(M=-1), ARG), (dict(V=0), ARG), (dict(K=0), ARG), (dict(target_type=lmoe.F32), ARG),
    (dict(target_type=9), ARG), (dict(K=60), UNSUP), (dict(M=(1 << 30) + 1), UNSUP),
    (dict(V=(1 << 30) + 1), UNSUP), (dict(K=(1 << 30) + 8, ldx=1 << 31, ldw=1 << 31), UNSUP),
    (dict(M=1 << 20, V=1 << 20), UNSUP),                # tiles
    (dict(ldx=56), ARG), (dict(ldw=56), ARG), (dict(ldx=68), ARG), (dict(ldw=68), ARG),
]
INPUTS = [
    (dict(x=None), ARG), (dict(w=None), ARG), (dict(target=None), ARG), (dict(dev_flag=None), ARG),
    (dict(x=BUF["x"] + 8), ARG), (dict(w=BUF["w"] + 2), ARG), (dict(target=BUF["target"] + 4), ARG),
    (dict(target=BUF["target"] + 2, target_type=lmoe.I32), ARG), (dict(lse=BUF["lse"] + 2), ARG),
    (dict(dev_flag=BUF["flag"] + 1), ARG),
]


def _forward(lib, d, ws=BUF["ws"], nb=1 << 40):
    return lib.lmoe_linear_xent_forward(ctypes.byref(d), ws, nb, None)


@no_gpu
@pytest.mark.parametrize("change,code", SIZES + INPUTS + [
    (dict(loss=None, lse=None), ARG), (dict(loss=BUF["loss"] + 2), ARG), (dict(loss=BUF["x"]), ARG),
    (dict(loss=BUF["w"]), ARG), (dict(lse=BUF["target"]), ARG), (dict(loss=BUF["lse"]), ARG),
    (dict(loss=BUF["ws"]), ARG), (dict(M=0, x=None, w=None), OK),
])
def test_xent_forward_refusals(lib, change, code):
    assert _forward(lib, _xent(**change)) == code


@no_gpu
def test_xent_forward_workspace_refusals(lib):
    q = lib.lmoe_linear_xent_workspace_bytes(ctypes.byref(_xent()))
    assert _forward(lib, _xent(), ws=None) == ARG
    assert _forward(lib, _xent(), ws=BUF["ws"] + 8) == ARG
    assert _forward(lib, _xent(), ws=BUF["x"]) == ARG
    assert _forward(lib, _xent(), nb=q - 1) == SMALL


def _backward(lib, d, **a):
    p = dict(dloss=BUF["dloss"], dx=BUF["dx"], lddx=64, dw=BUF["dw"], type=lmoe.F32, ws=BUF["ws"],
             nb=1 << 40)
    p.update(a)
    return lib.lmoe_linear_xent_backward(ctypes.byref(d), *p.values(), None)


@no_gpu
@pytest.mark.parametrize("change,code", SIZES + INPUTS + [(dict(lse=None), ARG)])
def test_xent_backward_description_refusals(lib, change, code):
    assert _backward(lib, _xent(**change)) == code


@no_gpu
@pytest.mark.parametrize("change,code", [
    (dict(dloss=None), ARG), (dict(dloss=BUF["dloss"] + 2), ARG), (dict(lddx=56), ARG),
    (dict(lddx=68), ARG), (dict(dx=BUF["dx"] + 8), ARG), (dict(dw=BUF["dw"] + 4), ARG),
    (dict(type=lmoe.E4M3), ARG), (dict(type=lmoe.I32), ARG),
    (dict(dx=BUF["x"]), ARG), (dict(dx=BUF["w"]), ARG), (dict(dw=BUF["w"]), ARG),
    (dict(dw=BUF["lse"]), ARG), (dict(dx=BUF["dloss"]), ARG), (dict(dw=BUF["dx"]), ARG),
    (dict(ws=BUF["dw"]), ARG), (dict(ws=None), ARG), (dict(ws=BUF["ws"] + 8), ARG),
    (dict(nb=1000), SMALL), (dict(dx=None, dw=None, ws=None), OK),
])
def test_xent_backward_refusals(lib, change, code):
    assert _backward(lib, _xent(), **change) == code


def test_xent_workspaces(lib):
    f = lambda **a: lib.lmoe_linear_xent_workspace_bytes(ctypes.byref(_xent(**a)))
    b = lambda **a: lib.lmoe_linear_xent_backward_workspace_bytes(ctypes.byref(_xent(**a)))
    for q in (f, b):
        assert q(M=0) == 0 and q(M=-1) == 0 and q(K=60) == 0 and q(M=1) > 0
    assert lib.lmoe_linear_xent_workspace_bytes(None) == 0
    assert lib.lmoe_linear_xent_backward_workspace_bytes(None) == 0
    # nothing of the size of the logits: sums and maxima of tiles, and one piece of their gradient
    big = dict(M=16384, V=1 << 18, K=64)
    assert f(**big) <= 16384 * ((1 << 18) // 256) * 16 + 16384 * 8
    assert b(**big) <= (256 << 20) + 16384 * 64 * 4 + 16384 * 4 + 4096
    # few rows: the sum's slices are bounded
    assert b(M=1, V=1 << 18, K=7168, ldx=7168, ldw=7168) <= 4 * (1 << 18) + 64 * 7168 * 4


@pytest.mark.parametrize("M,V,K", [(1, 1 << 28, 8), (16, 1 << 24, 8), (128, 1 << 20, 8),
                                   (128, 1 << 20, 7168), (129, 1 << 21, 64), (4096, 1 << 17, 7168),
                                   (40000, 1 << 17, 64)])
def test_xent_backward_workspace_is_what_the_header_says(lib, M, V, K):
    """d of a piece of the vocabulary in at most 256 MB, or of 4096 tokens, in as many terms as it has;
    up to 32 copies of dx in fp32 while its tiles of 128 x 256 are fewer than 152; vectors."""
    b = lib.lmoe_linear_xent_backward_workspace_bytes(ctypes.byref(_xent(M=M, V=V, K=K, ldx=K, ldw=K)))
    copies = max(1, min(32, 152 // (-(-M // 128) * -(-K // 256))))
    assert b <= max(256 << 20, 2 * M * 4096) + copies * 4 * M * K + 4 * M + 1024


def test_muon_workspace_is_what_the_header_says(lib):
    for n, r, c in ((3, 5000, 1), (3, 1, 5000), (2, 70, 129), (1, 4097, 333)):
        eight = lambda v: -(-v // 8) * 8
        side = min(r, c)
        q = lib.lmoe_muon_workspace_bytes(ctypes.byref(_muon(batch=n, rows=r, cols=c)))
        assert q <= n * (6 * r * eight(c) + 4 * side * eight(side) + 8 * eight(side)) + (1 << 16)


@no_gpu
def test_xent_without_a_description(lib):
    assert lib.lmoe_linear_xent_forward(None, None, 0, None) == ARG
    assert lib.lmoe_linear_xent_backward(None, None, None, 0, None, 0, None, 0, None) == ARG


COEFFS = (ctypes.c_float * 15)(*(3.4445, -4.7750, 2.0315) * 5)


def _muon(**a):
    c = a.pop("coeffs", COEFFS)
    return _fill(lmoe.MuonDesc(), dict(
        batch=3, rows=40, cols=24, steps=5, coeffs=None if c is None else ctypes.addressof(c), eps=1e-7,
        grad=BUF["grad"], grad_type=lmoe.F32, ldg=24, grad_stride=960, out=BUF["out"], ldo=24,
        out_stride=960, momentum=BUF["momentum"], ldm=24, momentum_stride=960, beta=0.95, nesterov=1,
        w=BUF["w"], ldw=24, w_stride=960, master=BUF["master"], ldmaster=24, master_stride=960,
        rate=0.1, weight_decay=0.1, scale=1.0, dev_flag=BUF["flag"]), a)


COMMON = [
    (dict(batch=-1), ARG), (dict(rows=-1), ARG), (dict(cols=-1), ARG), (dict(batch=65536), UNSUP),
    (dict(rows=(1 << 20) + 1), UNSUP), (dict(cols=(1 << 20) + 1), UNSUP),
    (dict(rows=1 << 17, cols=1 << 16), UNSUP),
    (dict(batch=0, grad=None), OK), (dict(rows=0, grad=None), OK), (dict(cols=0, grad=None), OK),
    (dict(steps=0), ARG), (dict(steps=65), ARG), (dict(coeffs=None), ARG), (dict(eps=0.0), ARG),
    (dict(eps=-1e-7), ARG), (dict(eps=NAN), ARG), (dict(eps=INF), ARG),
    (dict(coeffs=(ctypes.c_float * 15)(*[NAN] * 15)), ARG),
    (dict(coeffs=(ctypes.c_float * 15)(*[1.0] * 14 + [INF])), ARG),
    (dict(grad=None), ARG), (dict(grad_type=lmoe.E4M3), ARG), (dict(grad=BUF["grad"] + 2), ARG),
    (dict(grad=BUF["grad"] + 1, grad_type=lmoe.BF16), ARG), (dict(dev_flag=None), ARG),
    (dict(dev_flag=BUF["flag"] + 2), ARG), (dict(ldg=23), ARG), (dict(grad_stride=-1), ARG),
]


@no_gpu
@pytest.mark.parametrize("change,code", COMMON + [
    (dict(out=None), ARG), (dict(out=BUF["out"] + 1), ARG), (dict(ldo=23), ARG),
    (dict(out_stride=23), ARG), (dict(out=BUF["grad"]), ARG),     # over fp32
    (dict(out=BUF["grad"], grad_type=lmoe.BF16, ldo=32), ARG),
    (dict(out=BUF["grad"], grad_type=lmoe.BF16, out_stride=1000), ARG), (dict(out=BUF["ws"]), ARG),
    (dict(grad=BUF["ws"]), ARG),
])
def test_orthogonalize_refusals(lib, change, code):
    assert lib.lmoe_orthogonalize(ctypes.byref(_muon(**change)), BUF["ws"], 1 << 40, None) == code


@no_gpu
@pytest.mark.parametrize("change,code", COMMON + [
    (dict(momentum=None), ARG), (dict(w=None, master=None), ARG), (dict(beta=NAN), ARG),
    (dict(rate=INF), ARG), (dict(weight_decay=NAN), ARG), (dict(scale=-INF), ARG),
    (dict(momentum=BUF["momentum"] + 2), ARG), (dict(w=BUF["w"] + 1), ARG),
    (dict(master=BUF["master"] + 2), ARG), (dict(ldm=20), ARG), (dict(ldw=20), ARG),
    (dict(ldmaster=20), ARG), (dict(momentum_stride=0), ARG), (dict(w_stride=0), ARG),
    (dict(master_stride=8), ARG), (dict(momentum=BUF["grad"]), ARG), (dict(w=BUF["grad"]), ARG),
    (dict(master=BUF["grad"]), ARG), (dict(momentum=BUF["master"]), ARG), (dict(w=BUF["master"]), ARG),
    (dict(w=BUF["ws"]), ARG),
])
def test_update_refusals(lib, change, code):
    assert lib.lmoe_muon_update(ctypes.byref(_muon(**change)), BUF["ws"], 1 << 40, None) == code


@no_gpu
def test_muon_workspace_refusals(lib):
    d = ctypes.byref(_muon())
    q = lib.lmoe_muon_workspace_bytes(d)
    for call in (lib.lmoe_orthogonalize, lib.lmoe_muon_update):
        assert call(d, None, q, None) == ARG
        assert call(d, BUF["ws"] + 8, q, None) == ARG
        assert call(d, BUF["ws"], q - 1, None) == SMALL
        assert call(None, BUF["ws"], q, None) == ARG


def test_muon_workspace(lib):
    q = lambda **a: lib.lmoe_muon_workspace_bytes(ctypes.byref(_muon(**a)))
    assert q(batch=0) == q(rows=0) == q(cols=0) == q(batch=-1) == q(rows=(1 << 20) + 1) == 0
    assert lib.lmoe_muon_workspace_bytes(None) == 0
    # 6 bytes an element, 4 for each of the smaller side squared, and vectors
    for n, r, c in ((1, 4096, 7168), (64, 512, 3584), (64, 3584, 512)):
        side = min(r, c)
        least = n * (6 * r * c + 4 * side * side)
        assert least <= q(batch=n, rows=r, cols=c) <= least + n * 8 * side + (1 << 16)


@pytest.mark.parametrize("struct,cls", [("lmoe_linear_xent", lmoe.LinearXentDesc),
                                        ("lmoe_muon", lmoe.MuonDesc)])
def test_binding_structs_match_the_header(struct, cls, tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    fields = [n for n, _ in cls._fields_]
    body = "".join(f'  printf(" %zu", offsetof({struct}, {f}));\n' for f in fields)
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "lmoe.h"\n'
                   f'int main(void) {{\n  printf("%zu", sizeof({struct}));\n{body}'
                   '  printf(" %d %d %d", LMOE_MUON_MAX_STEPS, LMOE_I32, LMOE_I64);\n  return 0;\n}\n')
    include = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")
    subprocess.run([cc, "-I" + include, str(src), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()
    assert [int(v) for v in out] == [ctypes.sizeof(cls)] + [getattr(cls, f).offset for f in fields] + \
        [lmoe.MUON_MAX_STEPS, lmoe.I32, lmoe.I64]
