"""Rows in 8 bits and the linear layer over them (include/flashopt_lm.h,
int8.py) against plain 64-bit forms (lm_plain.py): codes and scales exactly,
products within their few roundings, over types, odd sizes, strides and the
special rows; weights rounded from the optimizers' compressed state."""
import math

import pytest
import torch

import lm_plain as P
from compressed_adamw_state_amd import flashopt as F
from compressed_adamw_state_amd import int8 as I
from compressed_adamw_state_amd import optim as O

pytestmark = pytest.mark.gpu

TYPES = [torch.bfloat16, torch.float16, torch.float32]


def draw(rows, cols, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, cols, generator=g) * torch.exp(torch.randn(rows, 1, generator=g))
    return x.to(dtype)


def quantized(x):
    rows, cols = x.shape
    ld = F.lib().flashopt_int8_ld(cols)
    codes = torch.full((rows, ld), 99, dtype=torch.int8, device="cuda")
    scale = torch.full((rows,), 99.0, device="cuda")
    F.flashopt_quantize_rows(x, codes, scale)
    assert bool((codes[:, cols:] == 0).all())
    return codes[:, :cols].cpu(), scale.cpu()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("cols", [1, 2, 15, 127, 128, 129, 768, 1000, 4096, 4097, 14336, 33001])
def test_quantize_rows(dtype, cols):
    x = draw(7, cols, dtype, cols)
    for v in (x.cuda(), torch.cat([x, x], 1).cuda()[:, :cols], torch.cat([x[:, :1], x], 1).cuda()[:, 1:]):
        q, s = quantized(v)
        rq, rs = P.row_codes(x)
        assert torch.equal(q, rq)
        assert torch.equal(s, rs)


@pytest.mark.parametrize("dtype", TYPES)
def test_quantize_borders_and_special_rows(dtype):
    """Values on the border between two codes (ties go to the even one), rows of zeros, subnormal
    and largest rows, infinities and NaN."""
    k = torch.arange(-126, 127).float()
    x = torch.zeros(8, 256)
    x[0, :253] = k + 0.5
    x[0, 255] = 127.0                                      # q = x: half codes exactly
    x[1, :253] = (k + 0.5) * 2 ** -20
    x[1, 255] = 127.0 * 2 ** -20
    x[3] = torch.finfo(dtype).tiny * torch.linspace(-1, 1, 256)
    x[4] = torch.finfo(dtype).max * torch.linspace(-1, 1, 256)
    x[5, 17] = math.inf
    x[6, 18] = math.nan
    x[7, 3] = -5.0
    x = x.to(dtype)
    q, s = quantized(x.cuda())
    ok = [0, 1, 2, 3, 4, 7]
    rq, rs = P.row_codes(x[ok])
    assert torch.equal(q[ok], rq)
    assert torch.equal(s[ok], rs)
    for r in (5, 6):
        assert bool((q[r] == 0).all()) and math.isnan(s[r].item())


SHAPES = [(1, 1, 1), (1, 64, 128), (1, 4099, 4096), (1, 33, 33001), (2, 130, 77), (2, 40, 9000), (3, 1000, 4097), (5, 31, 1300),
          # tiles of 256 x 256 (more than blocks in the last), small tiles more than blocks
          (2600, 5200, 384), (8000, 1700, 129), (5000, 6001, 300), (3300, 3299, 130), (3300, 3300, 640),
          (7, 257, 768), (8, 70, 2050), (8, 50, 5000), (9, 100, 640), (16, 50257, 768),
          (17, 100, 300), (33, 513, 1024), (63, 640, 129), (65, 2304, 768), (100, 129, 2048), (129, 257, 640), (200, 1000, 5120),
          (256, 256, 256), (300, 700, 14336), (70, 1, 2048), (129, 130, 2176), (66, 4000, 3456), (513, 1025, 384), (1000, 2304, 768), (2049, 300, 130)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_linear(dtype, m, n, k):
    g = torch.Generator().manual_seed(m + n + k)
    x = draw(m, k, dtype, m * n + k)
    codes = torch.randint(-127, 128, (n, k), generator=g, dtype=torch.int8)
    scale = torch.rand(n, generator=g) / 1000
    w = I.Int8Weight.from_codes(codes.cuda(), scale.cuda())
    bias = torch.randn(n, generator=g).to(dtype) if (m + n) % 2 else None
    xq, xs = P.row_codes(x)
    ref, tol = P.int8_product(xq.cuda(), xs.cuda(), codes.cuda(), scale.cuda(), None if bias is None else bias.cuda(), dtype)
    wide = torch.full((m, n + 3), 9.0, dtype=dtype, device="cuda")       # rows of a wider buffer
    for xin, out in ((x.cuda(), None), (torch.cat([x[:, :1], x], 1).cuda()[:, 1:], wide[:, 1:1 + n])):
        y = I.int8_linear(xin, w, None if bias is None else bias.cuda(), out=out)
        bad = (y.double() - ref).abs() > tol
        assert not bool(bad.any()), (int(bad.sum()), (y.double() - ref).abs().max().item())
    assert bool((wide[:, 0] == 9).all()) and bool((wide[:, n + 1:] == 9).all())
    a, s = torch.empty((m, w.codes.shape[1]), dtype=torch.int8, device="cuda"), torch.empty(m, device="cuda")
    F.flashopt_quantize_rows(x.cuda(), a, s)
    out = torch.empty((m, n), dtype=dtype, device="cuda")
    F.flashopt_int8_matmul(a, s, w.codes, w.scale, k, out, None if bias is None else bias.cuda())
    assert torch.equal(out, y)                             # the product alone: the same bits


def test_largest_sum_stays_exact():
    """All codes 127 over the longest row: the sum is 127^2 * 2^17 < 2^31."""
    k = 131072
    w = I.Int8Weight.from_codes(torch.full((40, k), 127, dtype=torch.int8, device="cuda"), torch.ones(40, device="cuda"))
    for m in (1, 20, 300):
        x = torch.ones((m, k), dtype=torch.bfloat16, device="cuda")
        x[0] *= -1
        y = I.int8_linear(x.float(), w)
        s = torch.tensor(1.0) / 127
        want = 127.0 * 127 * k * s.double()
        assert (y[0].double() + want).abs().max().item() <= 4 * P.U * want
        if m > 1:
            assert (y[1:].double() - want).abs().max().item() <= 4 * P.U * want


def test_special_rows_stay_in_their_row():
    x = draw(40, 512, torch.bfloat16, 3)
    x[3, 5], x[9, 6], x[11] = math.nan, -math.inf, 0.0
    w = I.Int8Weight.from_weight(draw(300, 512, torch.bfloat16, 4).cuda())
    y = I.int8_linear(x.cuda(), w)
    assert bool(torch.isnan(y[[3, 9]]).all()) and bool((y[11] == 0).all())
    keep = [r for r in range(40) if r not in (3, 9)]
    assert bool(torch.isfinite(y[keep]).all())


def test_shapes_module_and_refusals():
    lin = torch.nn.Linear(200, 33).to("cuda", torch.bfloat16)
    mod = I.Int8Linear.from_linear(lin)
    x = draw(12, 200, torch.bfloat16, 6).cuda()
    with torch.no_grad():
        y = mod(x.view(3, 4, 200))
        assert y.shape == (3, 4, 33)
        assert torch.equal(y.view(12, 33), mod(x))
        assert torch.equal(mod(x[0]), y[0, 0])
        assert mod(x[:0]).shape == (0, 33)
        again = I.Int8Linear.from_linear(torch.nn.Linear(200, 33).to("cuda", torch.bfloat16))
        again.load_state_dict(mod.state_dict())
        assert torch.equal(again(x), y.view(12, 33))
    w = I.Int8Weight(mod.codes, mod.scale, 200)
    assert (w.dequantize() - lin.weight.float()).abs().max() <= lin.weight.float().abs().amax() / 254 * 1.001
    with pytest.raises(ValueError):
        mod(x.clone().requires_grad_())
    with pytest.raises(ValueError):
        mod(x[:, :199])
    with pytest.raises(ValueError):
        I.int8_linear(x, w, bias=torch.zeros(33, device="cuda"))          # FP32 bias, BF16 x
    with pytest.raises(ValueError):
        I.int8_linear(x, w, out=torch.empty(12, 33, device="cuda"))
    with pytest.raises(ValueError):
        I.int8_linear(x.double(), w)
    with pytest.raises(ValueError):
        I.int8_linear(x.expand(3, 12, 200)[:, 0], w)                      # rows of stride 0


@pytest.mark.parametrize("opt,kw", [(O.FlashAdamW, {}), (O.FlashSGD, {}), (O.FlashLion, {}),
                                    (O.FlashAdamW, {"compress": False}), (O.FlashSGD, {"compress": False})])
def test_export_from_state(opt, kw):
    """export_int8 gives the codes of the rebuilt FP32 master weight."""
    g = torch.Generator().manual_seed(2)
    for shape in ((5, 700), (64, 128), (3, 5, 7, 9), (1030, 33)):
        p = torch.nn.Parameter((torch.randn(shape, generator=g) * 0.02).cuda())
        o = opt([p], lr=1e-2, **kw)
        for _ in range(2):
            p.grad = torch.randn(shape, generator=g).cuda().to(torch.bfloat16)
            o.step()
        w = o.export_int8(p)
        master = torch.empty(p.numel(), device="cuda")
        F.flashopt_tensor_export(o.state[p]["flash"], master)
        q, s = P.row_codes(master.view(shape[0], -1).cpu())
        assert torch.equal(w.codes[:, :w.k].cpu(), q) and bool((w.codes[:, w.k:] == 0).all())
        assert torch.equal(w.scale.cpu(), s)


def test_captured_and_replayed():
    w = I.Int8Weight.from_weight(draw(3000, 1024, torch.bfloat16, 1).cuda())
    for m in (1, 6, 40, 300):
        x = draw(m, 1024, torch.bfloat16, 2).cuda()
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            I.int8_linear(x, w)
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            held = I.int8_linear(x, w)
        for k in range(3):
            x.copy_(draw(m, 1024, torch.bfloat16, 10 + k))
            eager = I.int8_linear(x, w)
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(held, eager)


def test_output_beside_the_input():
    """Rows of input and output by turns in one buffer; an output over its input is refused."""
    w = I.Int8Weight.from_weight(draw(96, 200, torch.bfloat16, 5).cuda())
    for m in (2, 40):
        x = draw(m, 200, torch.bfloat16, m).cuda()
        both = torch.zeros(m, 296, dtype=torch.bfloat16, device="cuda")
        both[:, :200] = x
        I.int8_linear(both[:, :200], w, out=both[:, 200:])
        assert torch.equal(both[:, 200:], I.int8_linear(x, w)) and torch.equal(both[:, :200], x)
        with pytest.raises(F.FlashoptError):
            I.int8_linear(both[:, :200], w, out=both[:, 199:295])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("m,n,k", [(20, 70000, 130), (40, 300, 14336), (64, 4096, 8193), (48, 12289, 640), (70000, 20, 130),
                                   (128, 33000, 129), (129, 25700, 130)])
def test_linear_of_few_rows_or_channels(dtype, m, n, k):
    """Up to 128 rows of a side in small tiles, more of them than blocks; few tokens cut along
    the row; just past either."""
    test_linear(dtype, m, n, k)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("m,n,k", [(1, 30, 7), (1, 30, 8), (1, 100, 8191), (1, 4200, 4095), (1, 17000, 4097), (1, 40, 8193),
                                   (2, 4200, 2047), (2, 4200, 2049), (2, 33, 4096), (3, 40, 2048), (3, 5000, 1000),
                                   (4, 4200, 1023), (4, 4200, 1025), (4, 20000, 513), (4, 31, 2049)])
def test_linear_of_few_tokens(dtype, m, n, k):
    """Tokens rounded by the product's own blocks of 4 or 8 waves, and just past what those hold."""
    test_linear(dtype, m, n, k)


def test_no_outputs():
    """A layer without output channels, with any leading dimensions."""
    w = I.Int8Weight.from_weight(torch.zeros(0, 40, device="cuda"))
    for shape in ((40,), (7, 40), (2, 3, 40), (0, 3, 40)):
        x = torch.ones(shape, device="cuda")
        assert I.int8_linear(x, w).shape == shape[:-1] + (0,)
        assert I.int8_linear(x, w, torch.empty(0, device="cuda")).shape == shape[:-1] + (0,)


def test_export_of_no_rows():
    p = torch.nn.Parameter(torch.zeros(0, 40, device="cuda"))
    q = torch.nn.Parameter(torch.ones(3, 40, device="cuda"))
    w = O.FlashAdamW([p, q], lr=1e-2).export_int8(p)
    assert (w.n, w.k) == (0, 40) and w.codes.shape == (0, 128)
