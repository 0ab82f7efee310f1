"""The training step's operators where an operand or a result passes 4 GiB: rows far out are those of a small call on them,
bit by bit (rows, tiles and experts do not depend on each other)."""
import pytest

from gpu_util import banner
from train_util import BF16, F32

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
fb = pytest.importorskip("fp8_block_scaled_05_amd")

ROWS, COLS = (1 << 20) + 5, 4096
FAR = [0, (1 << 19) - 1, 1 << 19, (1 << 20) - 1, 1 << 20, ROWS - 1]


def _normal(*shape, dtype=BF16, seed=0):
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(generator=torch.Generator(device="cuda").manual_seed(seed))


def _same(big, small, rows=FAR):
    for a, b in zip(big, small):
        assert torch.equal(a[rows], b)


@pytest.fixture(autouse=True)
def _give_back():
    yield
    torch.cuda.empty_cache()


def test_norm():
    banner("norm of more than 2^32 elements")
    x, residual, w = _normal(ROWS, COLS), _normal(ROWS, COLS, seed=1), _normal(COLS, dtype=F32, seed=2)
    _same(fb.fp8_rmsnorm_quant(x, w, residual=residual, with_y=True), fb.fp8_rmsnorm_quant(x[FAR], w, residual=residual[FAR], with_y=True))


def test_norm_gradient():
    """dy is zero but for one far row, so that the weight's gradient is that row's."""
    banner("norm gradient of more than 2^32 elements")
    h, dresidual, w = _normal(ROWS, COLS), _normal(ROWS, COLS, seed=1), _normal(COLS, seed=2)
    dy = torch.zeros_like(h)
    dy[ROWS - 2] = _normal(COLS, seed=3)
    rows = FAR + [ROWS - 2]
    small = fb.fp8_rmsnorm_backward(dy[rows], h[rows], w, dresidual=dresidual[rows])
    dx, dw = fb.fp8_rmsnorm_backward(dy, h, w, dresidual=dresidual)
    _same([dx], small[:1], rows)
    assert torch.equal(dw, small[1])
    assert fb.fp8_rmsnorm_backward(dy, h, w, dresidual=dresidual, dx=h)[0] is h
    _same([h], small[:1], rows)


def test_activation():
    banner("activation of 2^33 elements")
    x = _normal(ROWS, 2 * COLS)
    gate, up = x[:, :COLS], x[:, COLS:]
    _same(fb.fp8_swiglu_quant(gate, up, with_y=True), fb.fp8_swiglu_quant(gate[FAR], up[FAR], with_y=True))
    banner("activation gradient of 2^33 elements")
    dy = _normal(ROWS, COLS, seed=1)
    _same(fb.fp8_swiglu_backward(dy, gate, up, with_d=True), fb.fp8_swiglu_backward(dy[FAR], gate[FAR], up[FAR], with_d=True))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_tiles(dtype):
    places, cols = 4190000, 1040
    banner(f"transposed tiles of {places} {dtype} rows")
    x = _normal(places, cols, dtype=dtype)
    last, mid = places - 200, 128 * 20000
    off = torch.tensor([0, last, places], dtype=torch.int32, device="cuda")
    for order in (None, torch.arange(places - 1, -1, -1, dtype=torch.int32, device="cuda")):
        q, s, padded = fb.fp8_quant_grouped_t(x, off, order=order)
        at = (last + 127) // 128 * 128
        assert padded.tolist() == [0, at, at + 256] and q.numel() > 1 << 32
        for lo, hi, c in ((0, 128, 0), (mid, mid + 256, mid), (last, places, at)):
            rows = x[lo:hi] if order is None else x[order[lo:hi].long()]
            few = fb.fp8_quant_grouped_t(rows, torch.tensor([0, hi - lo], dtype=torch.int32, device="cuda"))
            n = few[0].shape[1]
            assert torch.equal(q[:, c:c + n], few[0]) and torch.equal(s[:, c // 128:(c + n) // 128], few[1]), (lo, hi)
        del q, s


def _codes(rows, columns, seed):
    """0, 1, -1 and 2: sums of their products are exact."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    some = torch.tensor([0, 0x38, 0xb8, 0x40], dtype=torch.uint8, device="cuda")
    pieces = [some[torch.randint(0, 4, (16, columns), dtype=torch.int32, device="cuda", generator=g).long()] for _ in range(min(rows // 16, 4))]
    return torch.cat([pieces[i % len(pieces)].roll(i, 0) for i in range(rows // 16)])


def _alone(padded, a, b, e, dtype=F32):
    lo, hi = padded[e], padded[e + 1]
    ones = [torch.ones(len(m), (hi - lo) // 128, device="cuda") for m in (a, b)]
    return fb.fp8_blockscaled_grouped_wgrad(torch.tensor([0, hi - lo], dtype=torch.int32, device="cuda"), a[:, lo:hi], ones[0], b[:, lo:hi], ones[1],
                                            out_dtype=dtype)[0]


def test_weight_gradient_of_long_operands():
    banner("weight gradient of operands of more than 4 GiB")
    n, k, columns = 1040, 64, 1 << 22
    padded = [0, 128, columns - 256, columns]
    a, b = _codes(n, columns, 1), _codes(k, columns, 2)
    y = fb.fp8_blockscaled_grouped_wgrad(torch.tensor(padded, dtype=torch.int32, device="cuda"), a, torch.ones(n, columns // 128, device="cuda"), b,
                                         torch.ones(k, columns // 128, device="cuda"))
    assert torch.equal(y[0], _alone(padded, a, b, 0)) and torch.equal(y[2], _alone(padded, a, b, 2))
    want = sum(a[:, c:c + (1 << 18)].view(torch.float8_e4m3fn).float() @ b[:, c:c + (1 << 18)].view(torch.float8_e4m3fn).float().T
               for c in range(0, columns, 1 << 18))
    assert torch.equal(y.sum(0), want)


@pytest.mark.parametrize("deep", [1, 2])
def test_large_weight_gradient(deep):
    """One block an expert goes to tiles of 128, two to tiles of 256."""
    banner(f"weight gradients of 8 GiB, {deep} blocks an expert")
    experts, n, k = 16, 8192, 16384
    padded = [128 * deep * i for i in range(experts + 1)]
    a, b = _codes(n, padded[-1], 3), _codes(k, padded[-1], 4)
    y = fb.fp8_blockscaled_grouped_wgrad(torch.tensor(padded, dtype=torch.int32, device="cuda"), a, torch.ones(n, experts * deep, device="cuda"), b,
                                         torch.ones(k, experts * deep, device="cuda"))
    for e in (0, 7, 8, 15):
        lo, hi = padded[e], padded[e + 1]
        want = a[:, lo:hi].view(torch.float8_e4m3fn).float() @ b[:, lo:hi].view(torch.float8_e4m3fn).float().T
        assert torch.equal(y[e], want), e
