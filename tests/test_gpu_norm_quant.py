"""Residual addition + RMS norm + NVFP4 quantization and the dequantizer
against numpy and the C oracle's quantizer. The norm's sum is exact to 64
bits, so every output is compared bit for bit."""
import numpy as np
import pytest
import torch

import nvfp4_quantized_dense_amd as nv
import oracle
from attention_reference import bf16, e4m3, nibbles, numbers

pytestmark = pytest.mark.gpu
EPS = 1e-6


def make(seed, M, K, xt, rt, wt):
    r = np.random.RandomState(seed)

    def t(a, dt):
        return torch.from_numpy(a.astype(np.float32)).to(dt)

    x, res, w = t(r.randn(M, K), xt), t(3 * r.randn(M, K), rt), t(1 + 0.2 * r.randn(K), wt)
    if M > 2:
        x[1] = 0
        res[1] = 0  # a row of zeros
        x[2] *= 1e-4
        res[2] *= 1e-4
    return x, res, w


def plain(x, res, w, eps=EPS):
    z = x if res is None else (x.float() + res.float()).to(res.dtype)
    zd = z.double().numpy()
    rstd = (1.0 / np.sqrt((zd * zd).sum(1, keepdims=True) / zd.shape[1] + eps)).astype(np.float32)
    return z, (z.float().numpy() * rstd) * w.float().numpy()


@pytest.mark.parametrize("M,K", [(1, 16), (1, 5120), (3, 48), (5, 7168), (333, 2064), (4, 8192), (3, 33024), (700, 512)])
@pytest.mark.parametrize("xt,rt,wt", [(torch.bfloat16,) * 3, (torch.float32, torch.bfloat16, torch.float32),
                                      (torch.bfloat16, torch.float32, torch.bfloat16), (torch.float32,) * 3])
def test_static_and_per_token(M, K, xt, rt, wt):
    x, res, w = make(M + K, M, K, xt, rt, wt)
    z, y = plain(x, res, w)
    g_inv = np.float32(2688.0 / 5.0)
    oc, os_ = oracle.quantize(y, g_inv)
    xd, rd, wd = x.cuda(), res.cuda(), w.cuda()
    c, s, zo = nv.add_rmsnorm_nvfp4_quant(xd, wd, torch.tensor([g_inv], device="cuda"), residual=rd, eps=EPS)
    assert torch.equal(zo.cpu(), z) and zo.dtype == rt
    assert np.array_equal(s.cpu().numpy(), os_) and np.array_equal(c.cpu().numpy(), oc)
    oc, os_, og = oracle.quantize_per_token(y)
    c, s, zo, g = nv.add_rmsnorm_nvfp4_quant_per_token(xd, wd, residual=rd, eps=EPS, residual_out=rd)  # in place
    assert zo is rd and torch.equal(rd.cpu(), z)
    assert np.array_equal(g.cpu().numpy(), og)
    assert np.array_equal(s.cpu().numpy(), os_) and np.array_equal(c.cpu().numpy(), oc)


@pytest.mark.parametrize("xt", [torch.bfloat16, torch.float32])
def test_without_residual(xt):
    x, _, w = make(3, 9, 5120, xt, xt, torch.bfloat16)
    z, y = plain(x, None, w)
    oc, os_ = oracle.quantize(y, np.float32(500.0))
    c, s, zo = nv.add_rmsnorm_nvfp4_quant(x.cuda(), w.cuda(), torch.tensor([500.0], device="cuda"))
    assert torch.equal(zo.cpu(), x)
    assert np.array_equal(s.cpu().numpy(), os_) and np.array_equal(c.cpu().numpy(), oc)


def test_residual_out_is_x():
    x, res, w = make(4, 40, 512, torch.bfloat16, torch.bfloat16, torch.bfloat16)
    z, _ = plain(x, res, w)
    xd = x.cuda()
    nv.add_rmsnorm_nvfp4_quant(xd, w.cuda(), torch.ones(1, device="cuda"), residual=res.cuda(), residual_out=xd)
    assert torch.equal(xd.cpu(), z)


@pytest.mark.parametrize("M,K", [(1, 16), (7, 48), (130, 7168), (1, 0), (0, 32)])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_dequantize(M, K, dt):
    r = np.random.RandomState(M + K)
    codes = torch.from_numpy(r.randint(0, 256, (M, K // 2)).astype(np.uint8))
    scales = torch.from_numpy(r.randint(0, 0x7F, (M, K // 16)).astype(np.uint8))
    row_g = (r.rand(M) + 0.1).astype(np.float32)
    v = numbers(nibbles(codes.numpy()), scales.numpy(), np.float32(0.37)).astype(np.float32)
    out = nv.nvfp4_dequantize(codes.cuda(), scales.cuda(), g=torch.tensor([0.37], device="cuda"), out_dtype=dt)
    assert torch.equal(out.cpu(), torch.from_numpy(v).to(dt))
    v = numbers(nibbles(codes.numpy()), scales.numpy(), row_g[:, None]).astype(np.float32)
    out = nv.nvfp4_dequantize(codes.cuda(), scales.cuda(), row_g=torch.from_numpy(row_g).cuda(), out_dtype=dt)
    assert torch.equal(out.cpu(), torch.from_numpy(v).to(dt))


def test_dequantize_inverts_quantize_on_its_own_numbers():
    """Numbers that NVFP4 holds come back from a second pass unchanged."""
    x = torch.randn(64, 1024, device="cuda")
    g, g_inv = nv.nvfp4_calibrate(x)
    c, s = nv.nvfp4_quantize(x, g_inv)
    y = nv.nvfp4_dequantize(c, s, g=g, out_dtype=torch.float32)
    assert float((y - x).norm() / x.norm()) < 0.2  # a 2-bit mantissa: a quarter of a value at most
    assert e4m3(s.cpu().numpy()).max() == 448.0
