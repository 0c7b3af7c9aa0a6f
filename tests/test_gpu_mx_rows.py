"""GPU tests of rows in block-scaled numbers (gemm_mx_quantize, gemm_mx_dequantize): codes and values bit for bit.

A code is one rounding of an exact multiple, a value exact up to the output's rounding, so nothing is tolerated.
"""
import numpy as np
import pytest
import torch

import oracle.mx_rows as om

pytestmark = pytest.mark.gpu

F32, F16, BF16 = 0, 1, 2
DT = {F32: torch.float32, F16: torch.float16, BF16: torch.bfloat16}
E4M3, E2M1 = 0, 1
PER = {E4M3: 1, E2M1: 2}


def quantize(g, X, M, K, elem, dtype, ldx, source=None, top=1, rows_x=None, qpad=0, spad=0, shift=0):
    """Codes and scales from buffers filled with 0xA5 that start `shift` bytes into their allocation."""
    qp, sp = K // PER[elem] + qpad, K // 32 + spad
    q = torch.full((shift + M * qp + 16,), 0xA5, dtype=torch.uint8, device="cuda")
    s = torch.full((shift + M * sp + 16,), 0xA5, dtype=torch.uint8, device="cuda")
    g.gemm_mx_quantize(M, K, elem, dtype, X, ldx, q[shift:], qp * PER[elem], s[shift:], sp, source, top, rows_x)
    torch.cuda.synchronize()
    for t, p, used in ((q, qp, K // PER[elem]), (s, sp, K // 32)):
        assert (t[:shift] == 0xA5).all() and (t[shift + M * p:] == 0xA5).all()
        assert (t[shift:shift + M * p].view(M, p)[:, used:] == 0xA5).all()
    return (q[shift:shift + M * qp].view(M, qp)[:, :K // PER[elem]].cpu().numpy(),
            s[shift:shift + M * sp].view(M, sp)[:, :K // 32].cpu().numpy())


@pytest.mark.parametrize("M,K", [(1, 32), (1, 4096), (3, 96), (65, 64), (37, 2880), (130, 1056), (5, 8192), (2000, 32)])
@pytest.mark.parametrize("elem", [E4M3, E2M1])
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
def test_codes(cuda_lib, M, K, elem, dtype):
    """Normal values whose rows span the type's exponents; pitches and bases of several alignments."""
    rng = np.random.default_rng(M + K)
    lo, hi = (-6, 4) if dtype == F16 else (-36, 36)
    v = rng.standard_normal((M, K)) * 10.0 ** rng.uniform(lo, hi, (M, 1)) * 10.0 ** rng.uniform(-2, 0, (M, K))
    x = torch.from_numpy(v).to(DT[dtype])
    want = om.quantize_reference(x.double().numpy(), elem)
    for pad, xshift, qpad, spad, shift in ((0, 0, 0, 0, 0), (8, 0, 16, 16 - K // 32 % 16, 0), (3, 1, 1, 3, 1), (0, 0, 4, 0, 4)):
        buf = torch.full((xshift + M * (K + pad),), float("nan"), dtype=DT[dtype], device="cuda")
        buf[xshift:].view(M, K + pad)[:, :K] = x.cuda()
        q, s = quantize(cuda_lib, buf[xshift:], M, K, elem, dtype, K + pad, qpad=qpad, spad=spad, shift=shift)
        np.testing.assert_array_equal(s, want[1])
        np.testing.assert_array_equal(q, om.packed(want[0], elem))


@pytest.mark.parametrize("elem", [E4M3, E2M1])
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
def test_every_16_bit_value_and_ties(cuda_lib, elem, dtype):
    """Every finite 16-bit value beside each block maximum 1, 1.5, 1.999, 2^-100, ...; in fp32, every midpoint between
    representable values and its neighbours, subnormals among them."""
    if dtype == F32:
        t = om._table(elem)
        mid = ((t[1:] + t[:-1]) / 2).astype(np.float32)
        v = np.concatenate([t.astype(np.float32), mid, np.nextafter(mid, np.float32(9e9)), np.nextafter(mid, np.float32(-1))])
        v = np.concatenate([v, -v])
        v = np.resize(v, (len(v) + 30) // 31 * 31).reshape(-1, 31)
        blocks = []
        for e in (-149, -140, -127, -126, -100, 0, 60, 119):
            top = np.full((len(v), 1), 2.0 ** om.EMAX[elem])
            with np.errstate(over="ignore"):
                blocks.append((np.concatenate([top, v], 1) * 2.0 ** e).astype(np.float32))
        x = torch.from_numpy(np.concatenate(blocks))
    else:
        bits = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(DT[dtype])
        bits = bits[torch.isfinite(bits)]
        v = torch.cat([bits, bits.new_zeros(-len(bits) % 31)]).view(-1, 31)
        rows = []
        for peak in (1.0, 1.5, 1.99, 2.0 ** -14, 2.0 ** -20, 0.0, 30000.0):
            m = torch.full((len(v), 1), peak).to(DT[dtype])
            rows += [torch.cat([m, torch.where(v.abs() <= m, v, torch.zeros_like(v))], 1), torch.cat([m, v], 1)]
        x = torch.cat(rows)
    x = x.contiguous()
    want = om.quantize_reference(x.double().numpy(), elem)
    q, s = quantize(cuda_lib, x.cuda(), len(x), 32, elem, dtype, 32)
    np.testing.assert_array_equal(s, want[1])
    np.testing.assert_array_equal(q, om.packed(want[0], elem))


@pytest.mark.parametrize("elem", [E4M3, E2M1])
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
def test_zeros_infinities_and_nan(cuda_lib, elem, dtype):
    """Only the block that holds one shows it: scale NaN, elements 0; a block of zeros: scale 0."""
    x = torch.ones(4, 128)
    x[0, 5], x[1, 40], x[2, 127] = float("inf"), float("nan"), -float("inf")
    x[3, :64] = 0
    x = x.to(DT[dtype])
    q, s = quantize(cuda_lib, x.cuda(), 4, 128, elem, dtype, 128)
    want = om.quantize_reference(x.double().numpy(), elem)
    np.testing.assert_array_equal(s, want[1])
    np.testing.assert_array_equal(q, om.packed(want[0], elem))
    assert (s == 255).sum() == 3 and s[3].tolist()[:2] == [0, 0]


@pytest.mark.parametrize("elem", [E4M3, E2M1])
def test_gathered_rows(cuda_lib, elem):
    """Rows named by a source, some by none and some past X: those keep what their codes held."""
    rng = np.random.default_rng(1)
    T, top, K, M = 9, 4, 160, 40
    x = torch.from_numpy(rng.standard_normal((T, K))).bfloat16()
    src = rng.integers(0, T * top, M)
    src[[2, 7]], src[9], src[11] = -1, T * top, 2 ** 31 - 1
    q, s = quantize(cuda_lib, x.cuda(), M, K, elem, BF16, K, torch.from_numpy(src).int().cuda(), top, T)
    codes, scale = om.quantize_reference(x.double().numpy(), elem)
    live = (src >= 0) & (src < T * top)
    np.testing.assert_array_equal(q[live], om.packed(codes, elem)[src[live] // top])
    np.testing.assert_array_equal(s[live], scale[src[live] // top])
    assert (q[~live] == 0xA5).all() and (s[~live] == 0xA5).all()


@pytest.mark.parametrize("M,K", [(1, 32), (7, 96), (300, 320)])
@pytest.mark.parametrize("elem", [E4M3, E2M1])
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
def test_dequantize(cuda_lib, M, K, elem, dtype):
    """Every code and scale, E4M3's NaN and the NaN scale among them."""
    rng = np.random.default_rng(M + K)
    codes = rng.integers(0, 256 if elem == E4M3 else 16, (M, K))
    scale = rng.integers(0, 256, (M, K // 32))
    want = torch.from_numpy(om.values_of(codes, scale, elem)).float().to(DT[dtype])  # fp32 holds the values exactly
    for qpad, ypad, shift in ((0, 0, 0), (16, 8, 0), (1, 3, 1)):
        qp, sp = K // PER[elem] + qpad, K // 32 + qpad
        q, s = np.full((M, qp), 0xA5, np.uint8), np.full((M, sp), 0xA5, np.uint8)
        q[:, :K // PER[elem]], s[:, :K // 32] = om.packed(codes, elem), scale
        qd, sd = (torch.cat([torch.zeros(shift, dtype=torch.uint8), torch.from_numpy(a).flatten()]).cuda()[shift:] for a in (q, s))
        y = torch.full((M, K + ypad), 5.0, dtype=DT[dtype], device="cuda")
        cuda_lib.gemm_mx_dequantize(M, K, elem, qd, qp * PER[elem], sd, sp, dtype, y, K + ypad)
        y = y.cpu()
        assert (y[:, K:] == 5.0).all()
        got = y[:, :K].contiguous()
        nan = torch.isnan(want)
        assert torch.equal(torch.isnan(got), nan)
        assert torch.equal(got[~nan], want[~nan])


@pytest.mark.parametrize("elem", [E4M3, E2M1])
def test_round_trip(cuda_lib, elem):
    """Values that the type holds come back as they were."""
    rng = np.random.default_rng(2)
    codes = rng.integers(0, 256 if elem == E4M3 else 16, (64, 256))
    codes[codes % 128 == 127] = 3
    codes[:, ::32] = 7 if elem == E2M1 else 126  # the largest element in each block: its scale is found again
    scale = rng.integers(100, 150, (64, 8))
    x = torch.from_numpy(om.values_of(codes, scale, elem)).float().cuda()
    q, s = quantize(cuda_lib, x, 64, 256, elem, F32, 256)
    np.testing.assert_array_equal(s, scale)
    np.testing.assert_array_equal(q, om.packed(codes, elem))


def test_rows_past_2_to_the_31_elements(cuda_lib):
    """Offsets in 64 bits, both ways: the last rows of 2^31 values and more."""
    K, M = 8192, (1 << 18) + 3
    x = torch.zeros(M, K, dtype=torch.bfloat16, device="cuda")
    x[-2:] = torch.arange(2 * K, device="cuda").view(2, K).remainder(7).bfloat16()
    q = torch.empty(M, K, dtype=torch.uint8, device="cuda")
    s = torch.empty(M, K // 32, dtype=torch.uint8, device="cuda")
    cuda_lib.gemm_mx_quantize(M, K, E4M3, BF16, x, K, q, K, s, K // 32)
    y = torch.full_like(x, float("nan"))
    cuda_lib.gemm_mx_dequantize(M, K, E4M3, q, K, s, K // 32, BF16, y, K)
    assert torch.equal(y, x)  # small integers survive
