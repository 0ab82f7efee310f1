"""Boundary checks of the training step's operators that need no GPU: exports, struct layouts, workspace sizes, and the
refusal of bad arguments with the documented status before anything reaches the HIP runtime."""
import os
import re
import shutil
import struct
import subprocess

import pytest

import fp8_block_scaled_05_amd as fb

OK, INVALID, SHAPE, ALIGN = 0, 1, 2, 3
A = 0x10000            # a fake, 16-byte aligned "device" address; never dereferenced
NULL = 0
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def L():
    return fb.lib()


def test_exports_every_declared_symbol(L):
    names = fb.header_functions("fp8bs_train.h")
    assert set(names) == {"fp8_rmsnorm_quant", "fp8_rmsnorm_backward", "fp8_rmsnorm_backward_workspace", "fp8_swiglu_quant",
                          "fp8_swiglu_backward", "fp8_quant_grouped_t", "fp8_quant_grouped_t_columns", "fp8_blockscaled_grouped_wgrad",
                          "fp8_grad_norm", "fp8_grad_norm_workspace", "fp8_grad_clip"}
    for n in names:
        assert hasattr(L, n), n
        if not n.endswith(("_workspace", "_columns")):
            assert n in fb.__all__ and callable(getattr(fb, n))


NORM = "7Q7q2qd"
NORM_BACK = "7Qq6q2qd"
ACT = "5Q7q"
ACT_BACK = "6Q8q"
GRAD = "Q2q"


def test_structs_have_the_headers_fields():
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "fp8bs_train.h")).read(), flags=re.S)
    for name, form in (("fp8bs_rmsnorm_args", NORM), ("fp8bs_rmsnorm_backward_args", NORM_BACK), ("fp8bs_swiglu_args", ACT),
                       ("fp8bs_swiglu_backward_args", ACT_BACK), ("fp8bs_grad", GRAD)):
        body = re.search(r"typedef struct %s \{(.*?)\}" % name, text, re.S).group(1)
        want = "".join("Q" if "*" in line else ("d" if line.strip().startswith("double") else "q") * (line.count(",") + 1)
                       for line in body.split(";") if line.strip())
        assert "".join(c * int(n or 1) for n, c in re.findall(r"(\d*)([Qqd])", form)) == want, name


def _norm(L, x=A, res=A, w=A, out=A, y=A, q=A, s=A, rows=4, cols=256, ldx=256, ldr=256, ldo=256, ldy=256, ldq=256, dt=0, wdt=0, eps=1e-6):
    return L.fp8_rmsnorm_quant(struct.pack(NORM, x, res, w, out, y, q, s, rows, cols, ldx, ldr, ldo, ldy, ldq, dt, wdt, eps), None)


SIZES = [(dict(rows=-1), INVALID), (dict(cols=-128), INVALID), (dict(cols=0), SHAPE), (dict(cols=200), SHAPE), (dict(cols=32896), SHAPE),
         (dict(dt=2), INVALID), (dict(wdt=2), INVALID), (dict(eps=0.0), INVALID), (dict(eps=-1e-6), INVALID), (dict(eps=NAN), INVALID),
         (dict(eps=INF), INVALID), (dict(eps=1e-45), INVALID), (dict(w=A + 8), ALIGN), (dict(rows=1 << 31), INVALID)]


def test_norm_validation(L):
    assert _norm(L, rows=0) == OK and _norm(L, rows=0, x=NULL, res=NULL, out=NULL, y=NULL, q=NULL, s=NULL) == OK
    for kw, status in SIZES + [
            (dict(x=NULL), INVALID), (dict(out=NULL), INVALID), (dict(res=NULL), INVALID), (dict(q=NULL), INVALID), (dict(s=NULL), INVALID),
            (dict(y=NULL, q=NULL, s=NULL), INVALID), (dict(ldx=128), INVALID), (dict(ldr=128), INVALID), (dict(ldo=0), INVALID),
            (dict(ldy=255), INVALID), (dict(ldq=128), INVALID), (dict(x=A + 8), ALIGN), (dict(res=A + 2), ALIGN), (dict(out=A + 4), ALIGN),
            (dict(y=A + 8), ALIGN), (dict(q=A + 1), ALIGN), (dict(s=A + 2), ALIGN), (dict(ldx=260), ALIGN), (dict(ldq=264), ALIGN),
            (dict(ldx=1 << 40), INVALID), (dict(rows=(1 << 31) - 1, ldx=1 << 30), INVALID)]:
        assert _norm(L, **kw) == status, kw
        assert "fp8_rmsnorm_quant" in fb.last_error()
    assert L.fp8_rmsnorm_quant(None, None) == INVALID


def _norm_back(L, dy=A, h=A, w=A, res=A, dx=A, dw=A, ws=NULL, wsb=0, rows=1, cols=256, ldg=256, ldh=256, ldr=256, ldx=256, dt=0, wdt=0, eps=1e-6):
    return L.fp8_rmsnorm_backward(struct.pack(NORM_BACK, dy, h, w, res, dx, dw, ws, wsb, rows, cols, ldg, ldh, ldr, ldx, dt, wdt, eps), None)


def test_norm_backward_validation(L):
    assert _norm_back(L, rows=0, dw=NULL, dy=NULL, h=NULL, dx=NULL) == OK
    for kw, status in SIZES + [
            (dict(dy=NULL), INVALID), (dict(h=NULL), INVALID), (dict(dx=NULL), INVALID), (dict(ldg=128), INVALID), (dict(ldh=128), INVALID),
            (dict(ldr=128), INVALID), (dict(ldx=128), INVALID), (dict(dy=A + 2), ALIGN), (dict(h=A + 8), ALIGN), (dict(res=A + 4), ALIGN),
            (dict(dx=A + 8), ALIGN), (dict(dw=A + 4), ALIGN), (dict(ldh=260), ALIGN), (dict(ldh=1 << 40), INVALID)]:
        assert _norm_back(L, **kw) == status, kw
        assert "fp8_rmsnorm_backward" in fb.last_error()
    need = L.fp8_rmsnorm_backward_workspace(5000, 256)
    assert need > 0 and need % 1024 == 0
    big = dict(rows=5000)
    assert _norm_back(L, **big) == INVALID and "workspace" in fb.last_error()
    assert _norm_back(L, ws=A, wsb=need - 1, **big) == INVALID and _norm_back(L, ws=A + 8, wsb=need, **big) == ALIGN
    assert L.fp8_rmsnorm_backward(None, None) == INVALID


def test_norm_workspace(L):
    f = L.fp8_rmsnorm_backward_workspace
    assert f(0, 128) == 0 and f(1, 128) == 0
    assert f(-1, 128) == -1 and f(4, 0) == -1 and f(4, 100) == -1 and f(4, 40000) == -1 and f(1 << 40, 128) == -1
    for cols in (128, 2048, 2176, 8192, 8320, 32768):
        for rows in (2, 100, 5000, 1 << 20, (1 << 31) - 1):
            assert 0 <= f(rows, cols) <= 64 << 20


def _act(L, g=A, u=A, y=A, q=A, s=A, rows=4, cols=256, ldg=256, ldu=256, ldy=256, ldq=256, dt=0):
    return L.fp8_swiglu_quant(struct.pack(ACT, g, u, y, q, s, rows, cols, ldg, ldu, ldy, ldq, dt), None)


def test_activation_validation(L):
    assert _act(L, rows=0) == OK and _act(L, cols=0) == OK
    for kw, status in [(dict(rows=-1), INVALID), (dict(cols=-128), INVALID), (dict(cols=130), SHAPE), (dict(dt=2), INVALID), (dict(g=NULL), INVALID),
                       (dict(u=NULL), INVALID), (dict(q=NULL), INVALID), (dict(s=NULL), INVALID), (dict(y=NULL, q=NULL, s=NULL), INVALID),
                       (dict(ldg=128), INVALID), (dict(ldu=128), INVALID), (dict(ldy=128), INVALID), (dict(ldq=128), INVALID), (dict(g=A + 8), ALIGN),
                       (dict(u=A + 2), ALIGN), (dict(y=A + 4), ALIGN), (dict(q=A + 8), ALIGN), (dict(s=A + 1), ALIGN), (dict(ldu=260), ALIGN),
                       (dict(rows=1 << 31), INVALID), (dict(rows=(1 << 31) - 1, cols=256), INVALID), (dict(ldg=1 << 40), INVALID)]:
        assert _act(L, **kw) == status, kw
        assert "fp8_swiglu_quant" in fb.last_error()
    assert L.fp8_swiglu_quant(None, None) == INVALID


def _act_back(L, dy=A, g=A, u=A, d=A, q=A, s=A, rows=4, cols=256, ldy=256, ldg=256, ldu=256, ldd=512, ldq=512, dt=0):
    return L.fp8_swiglu_backward(struct.pack(ACT_BACK, dy, g, u, d, q, s, rows, cols, ldy, ldg, ldu, ldd, ldq, dt), None)


def test_activation_backward_validation(L):
    assert _act_back(L, rows=0) == OK and _act_back(L, cols=0) == OK
    for kw, status in [(dict(rows=-1), INVALID), (dict(cols=130), SHAPE), (dict(dt=2), INVALID), (dict(dy=NULL), INVALID), (dict(g=NULL), INVALID),
                       (dict(u=NULL), INVALID), (dict(q=NULL), INVALID), (dict(s=NULL), INVALID), (dict(d=NULL, q=NULL, s=NULL), INVALID),
                       (dict(ldd=256), INVALID), (dict(ldq=256), INVALID), (dict(ldy=128), INVALID), (dict(dy=A + 8), ALIGN), (dict(d=A + 8), ALIGN),
                       (dict(q=A + 8), ALIGN), (dict(s=A + 2), ALIGN), (dict(ldd=516), ALIGN), (dict(ldd=1 << 40), INVALID)]:
        assert _act_back(L, **kw) == status, kw
        assert "fp8_swiglu_backward" in fb.last_error()
    assert L.fp8_swiglu_backward(None, None) == INVALID


def _tiles(L, x=A, dt=0, rows=300, cols=64, ldx=64, off=A, G=4, order=NULL, places=300, top=1, q=A, ldq=768, s=A, columns=768, padded=4 * A):
    return L.fp8_quant_grouped_t(x, dt, rows, cols, ldx, off, G, order, places, top, q, ldq, s, columns, padded, None)


def test_grouped_t_validation(L):
    for kw, status in [(dict(rows=-1), INVALID), (dict(cols=-16), INVALID), (dict(places=-1), INVALID), (dict(G=0), INVALID), (dict(G=1025), INVALID),
                       (dict(dt=2), INVALID), (dict(cols=72), SHAPE), (dict(top=0), INVALID), (dict(top=1025, order=A), INVALID), (dict(top=2), INVALID),
                       (dict(places=299), INVALID), (dict(columns=640), SHAPE), (dict(columns=800), SHAPE), (dict(columns=1 << 23, ldq=1 << 23), INVALID),
                       (dict(off=NULL), INVALID), (dict(padded=NULL), INVALID), (dict(x=NULL), INVALID), (dict(q=NULL), INVALID), (dict(s=NULL), INVALID),
                       (dict(off=A + 2), ALIGN), (dict(padded=4 * A + 1), ALIGN), (dict(order=A + 2), ALIGN), (dict(x=A + 8), ALIGN), (dict(q=A + 8), ALIGN),
                       (dict(s=A + 2), ALIGN), (dict(ldx=48), INVALID), (dict(ldx=68), ALIGN), (dict(ldq=640), INVALID), (dict(ldq=776), ALIGN),
                       (dict(ldx=1 << 40), INVALID), (dict(rows=1 << 31, places=1 << 31), INVALID), (dict(places=1 << 40, order=A), INVALID)]:
        assert _tiles(L, **kw) == status, kw
        assert "fp8_quant_grouped_t" in fb.last_error()


def test_grouped_t_refuses_tables_that_it_would_write(L):
    for kw in (dict(padded=A, off=A), dict(padded=A + 16, off=A), dict(padded=A, off=A + 16), dict(padded=A + 1196, off=2 * A, order=A, places=300, rows=400),
               dict(padded=A, off=2 * A, order=A + 16)):
        assert _tiles(L, **kw) == INVALID, kw
        assert "overlaps" in fb.last_error()


def test_grouped_t_columns(L):
    """The bound holds for every way to share the rows out, and some way reaches it."""
    f = L.fp8_quant_grouped_t_columns
    assert f(-1, 4) == -1 and f(4, 0) == -1 and f(4, 1025) == -1 and f(1 << 31, 4) == -1
    for places in (0, 1, 5, 127, 128, 129, 300, 1000):
        for G in (1, 2, 7, 64, 1024):
            short = min(places, G)                             # experts with one row, the rest to one of them
            worst = (short - 1) + -(-(places - short + 1) // 128) if places else 0
            assert worst * 128 <= f(places, G)
            assert f(places, G) % 128 == 0 and f(places, G) <= (places + 127 * short)


def _wgrad(L, N=64, K=32, columns=256, G=4, padded=A, a=A, lda=256, sa=A, b=A, ldb=256, sb=A, y=A, ydt=1, acc=0):
    return L.fp8_blockscaled_grouped_wgrad(N, K, columns, G, padded, a, lda, sa, b, ldb, sb, y, ydt, acc, None)


def test_wgrad_validation(L):
    assert _wgrad(L, N=0) == OK and _wgrad(L, K=0) == OK
    for kw, status in [(dict(N=-16), INVALID), (dict(K=-16), INVALID), (dict(columns=-128), INVALID), (dict(G=0), INVALID), (dict(G=1025), INVALID),
                       (dict(ydt=2), INVALID), (dict(acc=2), INVALID), (dict(N=24), SHAPE), (dict(K=40), SHAPE), (dict(columns=200), SHAPE),
                       (dict(padded=NULL), INVALID), (dict(y=NULL), INVALID), (dict(a=NULL), INVALID), (dict(b=NULL), INVALID), (dict(sa=NULL), INVALID),
                       (dict(sb=NULL), INVALID), (dict(padded=A + 2), ALIGN), (dict(y=A + 8), ALIGN), (dict(a=A + 8), ALIGN), (dict(b=A + 1), ALIGN),
                       (dict(sa=A + 2), ALIGN), (dict(sb=A + 1), ALIGN), (dict(lda=128), INVALID), (dict(ldb=248), INVALID), (dict(lda=264), ALIGN),
                       (dict(lda=(1 << 22) + 16), INVALID), (dict(columns=(1 << 22) + 128, lda=1 << 23, ldb=1 << 23), INVALID),
                       (dict(N=1 << 34), INVALID), (dict(N=1 << 24, K=1 << 24), INVALID)]:
        assert _wgrad(L, **kw) == status, kw
        assert "fp8_blockscaled_grouped_wgrad" in fb.last_error()


def _grads(*of):
    return b"".join(struct.pack(GRAD, *g) for g in of)


def test_grad_norm_validation(L):
    one = _grads((A, 5, 1))
    assert L.fp8_grad_norm_workspace(None, 0) == 0 and L.fp8_grad_norm_workspace(one, -1) == -1
    need = L.fp8_grad_norm_workspace(one, 1)
    assert need == 8
    assert L.fp8_grad_norm_workspace(_grads(*[(A, 100, 0)] * 1000), 1000) > need
    assert L.fp8_grad_norm_workspace(_grads(*[(A, 1 << 40, 0)] * 3), 3) <= 3 << 20
    for grads, n, status in [(None, 1, INVALID), (one, -1, INVALID), (one, 65537, INVALID), (_grads((NULL, 5, 1)), 1, INVALID), (_grads((A, -1, 1)), 1, INVALID),
                             (_grads((A, 5, 2)), 1, INVALID), (_grads((A + 2, 5, 1)), 1, ALIGN), (_grads((A + 1, 5, 0)), 1, ALIGN),
                             (_grads((A, 1 << 50, 1)), 1, INVALID), (_grads((A, 1 << 43, 1), (A, 1 << 43, 1), (A, 5, 1)), 3, INVALID)]:
        assert L.fp8_grad_norm(grads, n, A, A, 1 << 20, None) == status, (n, status)
        assert "fp8_grad_norm" in fb.last_error()
    assert L.fp8_grad_norm(one, 1, NULL, A, 8, None) == INVALID and L.fp8_grad_norm(one, 1, A + 2, A, 8, None) == ALIGN
    assert L.fp8_grad_norm(one, 1, A, NULL, 8, None) == INVALID and "workspace" in fb.last_error()
    assert L.fp8_grad_norm(one, 1, A, A, 7, None) == INVALID and L.fp8_grad_norm(one, 1, A, A + 8, 8, None) == ALIGN


def test_grad_clip_validation(L):
    one, none = _grads((A, 5, 1)), _grads((NULL, 0, 1))
    assert L.fp8_grad_clip(None, None, 0, A, 1.0, None) == OK and L.fp8_grad_clip(none, none, 1, A, 1.0, None) == OK
    for max_norm in (0.0, -1.0, NAN, INF, 1e-60, 1e60):
        assert L.fp8_grad_clip(one, None, 1, A, max_norm, None) == INVALID, max_norm
        assert "max_norm" in fb.last_error()
    assert L.fp8_grad_clip(one, None, 1, NULL, 1.0, None) == INVALID and L.fp8_grad_clip(one, None, 1, A + 2, 1.0, None) == ALIGN
    for outs in (_grads((A, 4, 1)), _grads((A, 5, 0)), _grads((NULL, 5, 1))):
        assert L.fp8_grad_clip(one, outs, 1, A, 1.0, None) == INVALID
    assert L.fp8_grad_clip(one, _grads((A + 2, 5, 1)), 1, A, 1.0, None) == ALIGN


def test_grad_clip_refuses_shared_memory(L):
    """What one workgroup writes no other may read: tensors twice, ranges that touch, outputs over other inputs, the norm."""
    def clip(grads, outs=None, norm=8 * A):
        return L.fp8_grad_clip(_grads(*grads), None if outs is None else _grads(*outs), len(grads), norm, 1.0, None)

    far = (4 * A, 100, 1)
    for grads in ([(A, 5, 1), (A, 5, 1)], [(A, 100, 1), far, (A + 396, 5, 1)], [(A, 100, 0), (A + 198, 1, 0)], [far, (A, 1 << 20, 1)]):
        assert clip(grads) == INVALID and "shares memory" in fb.last_error(), grads
    assert clip([far, (A, 5, 1)], norm=4 * A + 40) == INVALID and "shares memory" in fb.last_error()
    pair = [(A, 100, 1), (2 * A, 100, 1)]
    for outs in ([(4 * A, 100, 1), (4 * A, 100, 1)], [(2 * A, 100, 1), (A, 100, 1)], [(A + 4, 100, 1), far], [far, (4 * A + 40, 100, 1)],
                 [(A, 100, 1), (A + 396, 100, 1)]):
        assert clip(pair, outs) == INVALID and "shares memory" in fb.last_error(), outs
    assert clip(pair, [far, (5 * A, 100, 1)], norm=5 * A) == INVALID


def test_train_header_is_plain_c(tmp_path):
    cc = shutil.which("gcc")
    if cc is None:
        pytest.skip("gcc not found")
    src = tmp_path / "use.c"
    src.write_text('#include "fp8bs_train.h"\n'
                   'int main(void) { return sizeof(fp8bs_rmsnorm_args) == %d && sizeof(fp8bs_rmsnorm_backward_args) == %d &&\n'
                   '                        sizeof(fp8bs_swiglu_args) == %d && sizeof(fp8bs_swiglu_backward_args) == %d && sizeof(fp8bs_grad) == %d ? 0 : 1; }\n'
                   % tuple(struct.calcsize(f) for f in (NORM, NORM_BACK, ACT, ACT_BACK, GRAD)))
    exe = str(tmp_path / "use")
    r = subprocess.run([cc, "-std=c99", "-Wall", "-Wextra", "-Werror", "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(ROOT, "include"), "-I",
                        os.path.join(os.environ.get("ROCM_PATH", "/opt/rocm"), "include"), str(src), "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    assert subprocess.run([exe]).returncode == 0


def test_binding_refuses_what_the_library_cannot_see():
    """Shapes, types and layouts of tensors (CPU tensors: whatever is left is refused for not being on the GPU)."""
    torch = pytest.importorskip("torch")
    x, u8 = torch.zeros(4, 256), torch.zeros(4, 256, dtype=torch.uint8)
    i32 = torch.zeros(3, dtype=torch.int32)
    for call in (lambda: fb.fp8_rmsnorm_quant(x), lambda: fb.fp8_rmsnorm_backward(x, x), lambda: fb.fp8_swiglu_quant(x, x),
                 lambda: fb.fp8_swiglu_backward(x, x, x), lambda: fb.fp8_quant_grouped_t(x, i32),
                 lambda: fb.fp8_blockscaled_grouped_wgrad(i32, u8, x, u8, x), lambda: fb.fp8_grad_norm([x]), lambda: fb.fp8_grad_clip([x], x, 1.0)):
        with pytest.raises(ValueError, match="GPU"):
            call()
    for call in (lambda: fb.fp8_rmsnorm_quant(None), lambda: fb.fp8_rmsnorm_backward(x, 3), lambda: fb.fp8_swiglu_quant(x, None),
                 lambda: fb.fp8_grad_norm(x), lambda: fb.fp8_grad_norm([None]), lambda: fb.fp8_grad_clip([3], x, 1.0),
                 lambda: fb.fp8_blockscaled_grouped_wgrad(i32, u8, x, u8, x, out_dtype=torch.float16)):
        with pytest.raises(TypeError):
            call()
    with pytest.raises(ValueError, match="no gradients"):
        fb.fp8_grad_norm([])
