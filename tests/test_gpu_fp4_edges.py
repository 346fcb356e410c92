"""GPU checks of the products with 4-bit weights where a workgroup takes several items, at
the ends of the scales' range, and with scales that begin anywhere.

Tolerances count roundings as in the checks of the products beside them: seven of eight
neighbouring products may lose 2^-13 of the largest one, sums of fp32 2 u a term, bf16
2^-8 of a value.
"""
import os
import subprocess
import sys

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from test_gpu_block import BF, F8, GRID, U, _deq, _dev, _fp8_rows, _gen, _largest8, _randn  # noqa: E402

F32 = torch.float32


def _weights64(codes, byte):
    """The values of one group's codes [N, K/2] and scales' bytes [N, K/32]."""
    grid = torch.tensor(np.concatenate([GRID, -GRID]), device=codes.device)
    v = torch.stack([grid[(codes & 15).long()], grid[(codes >> 4).long()]], -1).view(codes.shape[0], -1)
    return v * torch.ldexp(torch.ones_like(v[:, ::32]), byte.int() - 127).repeat_interleave(32, 1)


def _offsets(counts, stride=0):
    """(offsets, first row of each group, rows in all)"""
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    first = np.arange(len(counts)) * stride if stride else off[:-1]
    return torch.from_numpy(off).to(_dev()), first, len(counts) * stride if stride else int(off[-1])


def _check(out, x, xs, codes, byte, counts, first):
    for i, (f, c) in enumerate(zip(first, counts)):
        if c == 0:
            continue
        w = _weights64(codes[i], byte[i])
        xd = _deq(x[f:f + c], xs[f:f + c])
        y, mag = xd @ w.T, xd.abs() @ w.abs().T
        tol = 7 * 2.0 ** -13 * (_largest8(xd) @ _largest8(w).T) + (16 + x.shape[1] // 128 + 8) * 2 * U * mag
        assert ((out[f:f + c].double() - y).abs() <= (tol + 2.0 ** -8 * y.abs()) * (1 + 2.0 ** -7)).all(), i


# columns streamed past rows: 64 columns of a row tile of 16 are an item, 256 or 512 workgroups share them
APART = [1, 0, 1, 1, 0, 0, 1, 1, 1, 1, 0, 1]
MIXED = [1, 0, 33, 1, 0, 17, 1, 16, 0, 2, 1]


@pytest.mark.parametrize("counts", [APART, MIXED])
@pytest.mark.parametrize("N,K", [
    (8192, 7168),     # seven waves of eight blocks, scales in whole fours
    (8192, 5248),     # six waves, an odd number of blocks (the last wave has one)
    (16384, 2048),    # four waves of four blocks, two workgroups a CU
    (16384, 640),     # two waves, four workgroups a CU
    (8192, 8192),     # eight waves of eight
    (8192, 4096),     # eight waves of four
])
@pytest.mark.parametrize("column_major", [False, True])
def test_product_fp4_streamed_over_many_items(ep, counts, N, K, column_major):
    """Two to six items a workgroup, with changes of rows and of groups among them: the sums' two buffers in LDS
    are used again and again by several waves while the next columns are already on their way."""
    dev, g = _dev(), _gen(N + K + len(counts))
    off, first, rows = _offsets(counts)
    x, xs, given = _fp8_rows(g, rows, K, column_major)
    codes = torch.randint(0, 256, (len(counts), N, K // 2), generator=g, device=dev, dtype=torch.uint8)
    byte = torch.randint(118, 128, (len(counts), N, K // 32), generator=g, device=dev, dtype=torch.uint8)
    args = (x, given, codes, byte.view(torch.float8_e8m0fnu), off)
    out = torch.full((rows, N), 7.0, dtype=BF, device=dev)
    ep.grouped_gemm_fp4(*args, expected_rows=1, column_major_scales=column_major, out=out)
    _check(out, x, xs, codes, byte, counts, first)
    for _ in range(3):        # a sum taken too early or too late would not come out the same each time
        assert torch.equal(out, ep.grouped_gemm_fp4(*args, expected_rows=1, column_major_scales=column_major))


@pytest.mark.parametrize("N,K", [(8192, 7168), (16384, 2048), (8192, 5248)])
def test_product_fp4_streamed_over_many_items_exactly(ep, N, K):
    """Where every sum is exact (products are multiples of 1/4 and at most 18, powers of two leave multiples of 1/8 and sums
    below 2^18): equal bit for bit."""
    dev, g = _dev(), _gen(N + K)
    pick = lambda values, *s: torch.tensor(values, device=dev)[torch.randint(0, len(values), s, generator=g, device=dev)]  # noqa: E731
    for counts, stride in ((APART, 0), (MIXED, 0), (MIXED, 33)):
        off, first, rows = _offsets(counts, stride)
        x, xs = pick([1.0, 1.5, 2.0, 3.0, -1.0, -1.5, -2.0, -3.0], rows, K).to(F8), pick([1.0, 2.0], rows, K // 128)
        codes = torch.randint(0, 256, (len(counts), N, K // 2), generator=g, device=dev, dtype=torch.uint8)
        byte = torch.randint(126, 128, (len(counts), N, K // 32), generator=g, device=dev, dtype=torch.uint8)
        out = ep.grouped_gemm_fp4(x, xs, codes, byte, off, group_stride=stride, expected_rows=1)
        for i, (f, c) in enumerate(zip(first, counts)):
            if c:
                want = _deq(x[f:f + c], xs[f:f + c]) @ _weights64(codes[i], byte[i]).T
                assert torch.equal(out[f:f + c], want.to(F32).to(BF)), (counts, stride, i)


# every form: streamed columns, small tiles, large tiles (two of them: split)
@pytest.mark.parametrize("expected", [1, 40, 100000])
@pytest.mark.parametrize("low,high", [(0, 1), (0, 10), (1, 30), (90, 140), (225, 237)])
@pytest.mark.parametrize("K", [256, 512, 640])
def test_product_fp4_scales_of_every_size(ep, expected, low, high, K):
    """Scales down to 2^-127 (byte 0), and up to 2^109: weights below 2^112, for which no block's sum of 128 products with up
    to 448 passes fp32's range before the rows' scales bring it back."""
    dev, g = _dev(), _gen(low + high + K)
    counts, N = [3, 0, 40, 17], 256
    off, first, rows = _offsets(counts)
    x = (_randn(g, rows, K) * 60).clamp(-448, 448).to(F8)
    # the rows' scales bring the results back to about 1; a block's sums are far above fp32's smallest normal number but
    # for the smallest scales, where a lost 2^-149 times 2^126 is 2^-23: counted below
    xs = torch.exp2(127.0 - torch.tensor(float(high - 1), device=dev).clamp(min=1.0, max=240.0)) * (0.5 + torch.rand(rows, K // 128, generator=g, device=dev))
    codes = torch.randint(0, 256, (4, N, K // 2), generator=g, device=dev, dtype=torch.uint8)
    byte = torch.randint(low, high, (4, N, K // 32), generator=g, device=dev, dtype=torch.uint8)
    out = ep.grouped_gemm_fp4(x, xs, codes, byte, off, expected_rows=expected)
    for i, (f, c) in enumerate(zip(first, counts)):
        if c == 0:
            continue
        w = _weights64(codes[i], byte[i])
        xd = _deq(x[f:f + c], xs[f:f + c])
        y, mag = xd @ w.T, xd.abs() @ w.abs().T
        # 128 products and 16 sums a block may each lose the smallest subnormal
        lost = 144 * 2.0 ** -149 * xs[f:f + c].double().sum(1, keepdim=True)
        tol = 7 * 2.0 ** -13 * (_largest8(xd) @ _largest8(w).T) + (16 + K // 128 + 8) * 2 * U * mag + lost + 2.0 ** -8 * y.abs()
        assert y.abs().max() > 1 and ((out[f:f + c].double() - y).abs() <= tol * (1 + 2.0 ** -7)).all(), i


@pytest.mark.parametrize("expected", [1, 40, 100000])
@pytest.mark.parametrize("K", [512, 1024, 4096])
@pytest.mark.parametrize("shift", [4, 8, 12])
def test_product_fp4_scales_at_any_offset(ep, expected, K, shift):
    """Scales that begin 4, 8 or 12 bytes behind a 16-byte boundary, the rows' ones too, with whole fours of blocks: the
    same bits as aligned ones (which are read four at a time)."""
    dev, g = _dev(), _gen(K + shift)
    counts, N = [3, 0, 40, 300, 17], 256
    off, first, rows = _offsets(counts)
    x, xs, _ = _fp8_rows(g, rows, K)
    codes = torch.randint(0, 256, (5, N, K // 2), generator=g, device=dev, dtype=torch.uint8)
    byte = torch.randint(118, 128, (5, N, K // 32), generator=g, device=dev, dtype=torch.uint8)

    def moved(t):
        b = torch.empty(t.numel() * t.element_size() + 32, dtype=torch.uint8, device=dev)
        b = b[shift:shift + t.numel() * t.element_size()].view(t.dtype).view(t.shape)
        assert b.data_ptr() % 16 == shift
        return b.copy_(t)

    want = ep.grouped_gemm_fp4(x, xs, codes, byte, off, expected_rows=expected)
    _check(want, x, xs, codes, byte, counts, first)
    for s, b in ((xs, moved(byte)), (moved(xs), byte), (moved(xs), moved(byte))):
        assert torch.equal(want, ep.grouped_gemm_fp4(x, s, codes, b, off, expected_rows=expected))


@pytest.mark.parametrize("shift", [4, 8, 12])
def test_product_fp4_whole_large_tiles_with_scales_at_any_offset(ep, shift):
    """The same for large tiles that are not split (70 of them)."""
    dev, g = _dev(), _gen(shift)
    counts, N, K = [700, 0, 1025], 2304, 1024
    off, first, rows = _offsets(counts)
    x, xs, _ = _fp8_rows(g, rows, K)
    codes = torch.randint(0, 256, (3, N, K // 2), generator=g, device=dev, dtype=torch.uint8)
    byte = torch.randint(118, 128, (3, N, K // 32), generator=g, device=dev, dtype=torch.uint8)
    want = ep.grouped_gemm_fp4(x, xs, codes, byte, off, expected_rows=100000)
    _check(want, x, xs, codes, byte, counts, first)
    b = torch.empty(byte.numel() + 16, dtype=torch.uint8, device=dev)[shift:shift + byte.numel()].view(byte.shape).copy_(byte)
    s = torch.empty(xs.numel() + 4, device=dev)[shift // 4:shift // 4 + xs.numel()].view(xs.shape).copy_(xs)
    assert b.data_ptr() % 16 == shift and s.data_ptr() % 16 == shift
    assert torch.equal(want, ep.grouped_gemm_fp4(x, s, codes, b, off, expected_rows=100000))


_FORMS = r"""
import torch
import combine_get_dispatch_scan_amd as ep
for K in (128, 256, 384):
    for G, N in ((27, 7680), (256, 7680)):
        x = torch.ones(G, K, device="cuda").to(torch.float8_e4m3fn)
        w, s = (torch.zeros(G, N, K // n, device="cuda", dtype=torch.uint8) for n in (2, 32))
        off = torch.arange(0, G + 1, device="cuda", dtype=torch.int32)
        ep.grouped_gemm_fp4(x, torch.ones(G, K // 128, device="cuda"), w, s, off)
        torch.cuda.synchronize()
"""


def test_form_of_short_rows(ep):
    """One row a group: one block of K is streamed (256 groups, N = 7680: 38 us, 80 from small tiles), two go by the size.
    EP_DEBUG is read once a process, hence another one."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", _FORMS], cwd=root, capture_output=True, text=True, timeout=100,
                       env=dict(os.environ, EP_DEBUG="1"))
    assert r.returncode == 0, r.stderr[-2000:]
    got = [line.split()[1] for line in r.stderr.splitlines() if line.startswith("[moe_ep] grouped")]
    assert got == ["grouped_gemm_fp4_" + n for n in ("stream", "stream", "small", "stream", "stream", "stream")]
