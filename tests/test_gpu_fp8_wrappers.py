"""Arguments that the block-scaled e4m3 wrappers refuse before anything runs."""
import pytest
import torch

import expert_gemm_layers_gb300 as dg
from expert_gemm_layers_gb300._lib import DGError
from test_gpu_fp8 import BF16, DEV, E4M3, E8M0, randn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def t():
    x, w = randn((6, 272), 1).to(DEV), randn((400, 272), 2).to(DEV)
    return dict(x=x, w=w, x8=dg.fp8_quantize(x), w8=dg.fp8_quantize(w, 128), g=randn((272,), 3).to(DEV),
                dy=randn((6, 400), 4).to(DEV), b=randn((400,), 5).to(DEV))


def refused(call, *errors):
    with pytest.raises(errors or (ValueError, TypeError, DGError)):
        call()


def test_quantize(t):
    x = t["x"]
    refused(lambda: dg.fp8_quantize(x.t()), ValueError)                # strides
    refused(lambda: dg.fp8_quantize(x[:, 16:]), ValueError)
    refused(lambda: dg.fp8_quantize(x.cpu()), ValueError)
    refused(lambda: dg.fp8_quantize(x.half()), TypeError)
    refused(lambda: dg.fp8_quantize(x, 64), ValueError)
    refused(lambda: dg.fp8_quantize(x.view(2, 3, 272), 128), ValueError)
    refused(lambda: dg.fp8_quantize(x[0, 0]), ValueError)              # no dimension
    refused(lambda: dg.fp8_quantize(randn((4, 24), 1).to(DEV)))        # 24 columns
    codes, scales = t["x8"]
    refused(lambda: dg.fp8_dequantize(codes, scales[:, :2].contiguous()), ValueError)
    refused(lambda: dg.fp8_dequantize(codes, scales.view(torch.uint8)), TypeError)
    refused(lambda: dg.fp8_dequantize(codes.view(torch.uint8), scales), TypeError)
    refused(lambda: dg.fp8_dequantize(codes, scales, out=t["x"][:5]), ValueError)


def test_linear(t):
    x8, w8 = t["x8"], t["w8"]
    refused(lambda: dg.fp8_linear(x8, t["w"]), TypeError)              # a weight that is not in 8 bits
    refused(lambda: dg.fp8_linear(x8, x8), ValueError)                 # activations for a weight
    refused(lambda: dg.fp8_linear(w8, w8), ValueError)                 # a weight for activations
    refused(lambda: dg.fp8_linear(x8, w8, t["b"][:-1].contiguous()), ValueError)
    refused(lambda: dg.fp8_linear(x8, w8, t["b"].float()), TypeError)
    refused(lambda: dg.fp8_linear(x8, w8, out=torch.empty((6, 399), dtype=BF16, device=DEV)), ValueError)
    refused(lambda: dg.fp8_linear(x8, w8, workspace=torch.zeros(128, dtype=torch.uint8, device=DEV)), ValueError)
    refused(lambda: dg.fp8_linear(t["x"], w8, workspace=torch.zeros(256, dtype=torch.uint8, device=DEV)), ValueError)
    refused(lambda: dg.fp8_linear(t["x"][:, :256].contiguous(), w8), ValueError)
    shared = torch.empty(6 * 272 + 6 * 400 * 2, dtype=torch.uint8, device=DEV)
    codes = shared[:6 * 272].view(E4M3).view(6, 272)
    out = shared[6 * 272 - 32:6 * 272 - 32 + 6 * 800].view(BF16).view(6, 400)
    refused(lambda: dg.fp8_linear((codes, x8[1]), w8, out=out), DGError)   # y over the codes


def test_backward(t):
    x8, w8, dy = t["x8"], t["w8"], t["dy"]
    refused(lambda: dg.fp8_linear_backward(None, w8, dy), ValueError)
    refused(lambda: dg.fp8_linear_backward(x8, None, dy), ValueError)
    refused(lambda: dg.fp8_linear_backward(x8, w8, dy[:5].contiguous()), ValueError)
    refused(lambda: dg.fp8_linear_backward(x8, w8, dy[:, :384].contiguous()), ValueError)
    refused(lambda: dg.fp8_linear_backward(x8, w8, dy.float()), TypeError)
    refused(lambda: dg.rms_norm_backward(t["x"], t["g"], t["x"][:5].contiguous()), ValueError)
    refused(lambda: dg.rms_norm_backward(t["x"], t["g"], t["x"], dh=t["x"].float()), TypeError)


def test_norm(t):
    x, g = t["x"], t["g"]
    refused(lambda: dg.rms_norm(x, g[:-1].contiguous()), ValueError)
    refused(lambda: dg.rms_norm(x, g, x[:5].contiguous()), ValueError)
    refused(lambda: dg.rms_norm(x, g.float()), TypeError)
    refused(lambda: dg.rms_norm(x, g, eps=0.0))
    refused(lambda: dg.rms_norm(x[:, :264].contiguous(), g[:264].contiguous(), fp8=True))   # no multiple of 16
    refused(lambda: dg.rms_norm(x[0, 0], g), ValueError)


def test_scales_outside_what_the_quantiser_writes():
    """Foreign scales from 2^-127 up, and NaN: the product takes what they stand for."""
    codes = torch.full((2, 128), 0x38, dtype=torch.uint8, device=DEV).view(E4M3)     # ones
    scales = torch.tensor([[0], [255]], dtype=torch.uint8, device=DEV).view(E8M0)
    w8 = (torch.full((16, 128), 0x38, dtype=torch.uint8, device=DEV).view(E4M3),
          torch.tensor([[127 + 100]], dtype=torch.uint8, device=DEV).view(E8M0))
    y = dg.fp8_linear((codes, scales), w8)
    assert (y[0].double() == 2.0 ** (-127 + 100 + 7)).all() and y[1].isnan().all()
