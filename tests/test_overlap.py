"""Calls whose outputs share memory with each other or, but for what the header allows, with an input are refused before
anything is launched: workgroups read and write at once.  Addresses here are made up and reach no device."""
import os
import shutil
import struct
import subprocess

import pytest

import fp8_block_scaled_05_amd as fb
from fp8_block_scaled_05_amd import build
from test_train_abi import ACT, ACT_BACK, NORM, NORM_BACK, _grads

HERE = os.path.dirname(os.path.abspath(__file__))
INVALID, NULL = 1, 0
AT = [0x1000000 * (i + 1) for i in range(12)]          # 16 MiB apart
ROWS, COLS = 64, 256


@pytest.fixture(scope="module")
def L():
    return fb.lib()


def test_shared_bytes(tmp_path):
    cc = shutil.which("g++")
    if cc is None:
        pytest.skip("g++ not found")
    exe = str(tmp_path / "overlap_check")
    r = subprocess.run([cc, "-std=c++17", "-O2", "-Wall", "-Werror", "-I", build.CSRC, os.path.join(HERE, "overlap_check.cpp"), "-o", exe],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    r = subprocess.run([exe], capture_output=True, text=True, timeout=100)
    assert r.returncode == 0, r.stdout


def _refused(call, *pairs):
    for kw in pairs:
        assert call(**kw) == INVALID and "overlaps" in fb.last_error(), (kw, fb.last_error())


def test_norm(L):
    def call(x=AT[0], res=AT[1], w=AT[2], out=AT[3], y=AT[4], q=AT[5], s=AT[6], ldo=COLS, ldy=COLS):
        return L.fp8_rmsnorm_quant(struct.pack(NORM, x, res, w, out, y, q, s, ROWS, COLS, COLS, COLS, ldo, ldy, COLS, 0, 0, 1e-6), None)

    row = 2 * COLS
    _refused(call, dict(out=AT[0] + row), dict(out=AT[1] + 16), dict(out=AT[0] - row), dict(y=AT[3]), dict(y=AT[0] + row), dict(y=AT[1] + 5 * row),
             dict(q=AT[0]), dict(q=AT[3] + 16), dict(s=AT[0] + 4), dict(s=AT[5]), dict(y=AT[2] - 16), dict(w=AT[5] + 512), dict(w=AT[6]),
             dict(out=AT[0], ldo=COLS + 8), dict(y=AT[0], ldy=2 * COLS), dict(out=AT[0], y=AT[0]))


def test_norm_gradient(L):
    need = L.fp8_rmsnorm_backward_workspace(ROWS, COLS)
    assert need > 0

    def call(dy=AT[0], h=AT[1], w=AT[2], res=AT[3], dx=AT[4], dw=AT[5], ws=AT[6], ldx=COLS):
        return L.fp8_rmsnorm_backward(struct.pack(NORM_BACK, dy, h, w, res, dx, dw, ws, need, ROWS, COLS, COLS, COLS, COLS, ldx, 0, 0, 1e-6), None)

    _refused(call, dict(dx=AT[0] + 16), dict(dx=AT[1] - 512), dict(dx=AT[3] + 1024), dict(dx=AT[2]), dict(dw=AT[2]), dict(dw=AT[0] + 512), dict(dw=AT[4]),
             dict(ws=AT[1]), dict(ws=AT[5]), dict(ws=AT[4] + 16), dict(ws=AT[2]), dict(dx=AT[1], ldx=COLS + 8))


def test_activation(L):
    def call(g=AT[0], u=AT[0] + 2 * COLS, y=AT[1], q=AT[2], s=AT[3], ldy=COLS):
        return L.fp8_swiglu_quant(struct.pack(ACT, g, u, y, q, s, ROWS, COLS, 2 * COLS, 2 * COLS, ldy, COLS, 0), None)

    _refused(call, dict(y=AT[0]), dict(y=AT[0] + 16, ldy=2 * COLS), dict(y=AT[0] + 4 * COLS, ldy=2 * COLS), dict(q=AT[0] + 16), dict(s=AT[0] + 8), dict(q=AT[1]),
             dict(s=AT[2]), dict(s=AT[1] + 512))


def test_activation_gradient(L):
    def call(dy=AT[1], g=AT[0], u=AT[0] + 2 * COLS, d=AT[2], q=AT[3], s=AT[4], ldd=2 * COLS):
        return L.fp8_swiglu_backward(struct.pack(ACT_BACK, dy, g, u, d, q, s, ROWS, COLS, COLS, 2 * COLS, 2 * COLS, ldd, 2 * COLS, 0), None)

    _refused(call, dict(d=AT[0] + 16), dict(d=AT[0] + 4 * COLS), dict(d=AT[0], ldd=2 * COLS + 8), dict(d=AT[1]), dict(d=AT[1] - 512), dict(q=AT[2]), dict(s=AT[3]),
             dict(q=AT[1] + 512), dict(s=AT[0]), dict(d=AT[0] - 512, g=AT[0] + 16))


def test_transposed_tiles(L):
    def call(x=AT[0], off=AT[1], order=AT[2], q=AT[3], s=AT[4], padded=AT[5]):
        return L.fp8_quant_grouped_t(x, 0, 300, 64, 64, off, 4, order, 300, 1, q, 768, s, 768, padded, None)

    _refused(call, dict(q=AT[0]), dict(q=AT[0] + 300 * 128 - 16), dict(s=AT[0] + 64), dict(q=AT[1] - 16), dict(s=AT[2]), dict(padded=AT[0] + 4), dict(padded=AT[3]),
             dict(padded=AT[4] + 8), dict(s=AT[3] + 64 * 768 - 4), dict(padded=AT[1] + 16), dict(padded=AT[2] + 1196))


def test_weight_gradient(L):
    def call(a=AT[0], b=AT[1], sa=AT[2], sb=AT[3], padded=AT[4], y=AT[5], lda=256):
        return L.fp8_blockscaled_grouped_wgrad(64, 32, 256, 4, padded, a, lda, sa, b, 256, sb, y, 1, 0, None)

    size = 4 * 64 * 32 * 4
    _refused(call, dict(y=AT[0]), dict(y=AT[1] + 32 * 256 - 16), dict(y=AT[2] - size + 16), dict(y=AT[3]), dict(y=AT[4] + 16), dict(a=AT[5] + size - 16))


def test_gradient_norm(L):
    grads = _grads((AT[0], 100, 1), (AT[1], 1 << 20, 0))
    need = L.fp8_grad_norm_workspace(grads, 2)
    for ws in (AT[0], AT[0] + 384, AT[1] + (1 << 21) - 16, AT[1] - need + 16 & ~15):
        assert L.fp8_grad_norm(grads, 2, AT[2], ws, need, None) == INVALID and "overlaps" in fb.last_error()
