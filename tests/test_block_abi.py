"""CPU checks of the entry points around the expert layer: invalid arguments are refused
before any HIP call, and the binding refuses tensors the kernels cannot take."""
import ctypes

import pytest

import combine_get_dispatch_scan_amd as ep

torch = pytest.importorskip("torch")

FAKE = 1 << 20  # never dereferenced: every call below fails validation first


def _args(**kw):
    a = dict(x=FAKE, y=FAKE, weight=FAKE, y_weight=FAKE, gate=FAKE, x_ld=256, y_ld=256, num_rows=10, width=256, x_f32=0,
             norm=1, y_norm=1, weights_f32=0, gate_kind=ep.EP_GATE_TOKEN, gate_f32=1, residual_scale=1.0, y_scale=1.0,
             eps=1e-6, weight_offset=0.0)
    a.update(kw)
    return ep.ep_block_norm_t(**a)


ALONE = dict(y=None, y_weight=None, y_norm=0, gate=None, gate_kind=0)   # a norm of x alone
NORM_CASES = [
    (dict(num_rows=-1), "num_rows"), (dict(num_rows=2 ** 31 - 1), "num_rows"), (dict(width=4), "width"),
    (dict(width=257), "width"), (dict(width=32768 + 8, x_ld=1 << 20, y_ld=1 << 20), "width"), (dict(x_f32=2), "x_f32"),
    (dict(norm=-1), "norm"), (dict(y_norm=2), "y_norm"), (dict(weights_f32=3), "weights_f32"),
    (dict(gate_f32=2), "gate_f32"), (dict(gate_kind=3), "gate_kind"), (dict(gate_kind=-1), "gate_kind"),
    (dict(y=None), "need y"), (dict(ALONE, y_weight=FAKE), "need y"), (dict(ALONE, y_norm=1), "need y"),
    (dict(ALONE, gate=FAKE, gate_kind=1), "need y"), (dict(ALONE, norm=0, weight=None), "norm must be 1"),
    (dict(ALONE, residual_scale=0.5), "residual_scale 1"), (dict(norm=0), "weight needs norm"),
    (dict(gate=None), "together"), (dict(gate_kind=0), "together"), (dict(eps=0.0), "eps"), (dict(eps=-1.0), "eps"),
    (dict(eps=float("nan")), "eps"), (dict(eps=float("inf")), "eps"), (dict(eps=1e-38), "eps"),
    (dict(residual_scale=float("inf")), "finite"), (dict(y_scale=float("nan")), "finite"),
    (dict(weight_offset=float("nan")), "finite"), (dict(x_ld=248), "x_ld"), (dict(x_ld=260), "x_ld"),
    (dict(x_ld=1 << 50), "x_ld"), (dict(y_ld=0), "y_ld"), (dict(y_ld=257), "y_ld"), (dict(x=None), "x must"),
    (dict(x=FAKE + 8), "x must"), (dict(y=FAKE + 2), "16-byte"), (dict(weight=FAKE + 8), "16-byte"),
    (dict(y_weight=FAKE + 4), "16-byte"), (dict(gate=FAKE + 2), "gate must be aligned"),
    (dict(gate=FAKE + 4, gate_kind=2), "gate must be aligned"),
]


def _refused(rc, msg):
    assert rc == ep.EP_EINVAL
    assert msg in ep.ep_last_error(), ep.ep_last_error()


@pytest.mark.parametrize("kw,msg", NORM_CASES)
def test_norm_refusals(kw, msg):
    _refused(ep.ep_block_norm(_args(**kw), FAKE, FAKE, FAKE, FAKE, None), msg)
    _refused(ep.ep_block_norm_backward(_args(**kw), FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 1 << 30, None), msg)


@pytest.mark.parametrize("kw,out,msg", [
    ({}, (FAKE, FAKE, None, FAKE), "together"), ({}, (FAKE, FAKE, FAKE, None), "together"),
    ({}, (None, None, None, None), "nothing to write"), (ALONE, (FAKE, FAKE, None, None), "x_out needs y"),
    (dict(norm=0, weight=None), (FAKE, FAKE, None, None), "need norm"),
    (dict(norm=0, weight=None), (FAKE, None, FAKE, FAKE), "need norm"),
    (dict(width=200, x_ld=200), (FAKE, FAKE, FAKE, FAKE), "multiple of 128"),
    (dict(x_ld=512), (FAKE, FAKE, None, None), "dense"), ({}, (FAKE + 8, FAKE, None, None), "16-byte"),
    ({}, (FAKE, FAKE + 2, None, None), "16-byte"), ({}, (FAKE, FAKE, FAKE + 4, FAKE), "16-byte"),
    ({}, (FAKE, FAKE, FAKE, FAKE + 2), "16-byte"),
])
def test_norm_output_refusals(kw, out, msg):
    _refused(ep.ep_block_norm(_args(**kw), *out, None), msg)


@pytest.mark.parametrize("kw,a,msg", [
    (dict(norm=0, weight=None), {}, "grad_h needs norm"), (ALONE, {}, "out_y needs y"),
    (dict(weight=None), {}, "out_weight"), (dict(y_weight=None), {}, "out_y_weight"),
    (dict(gate=None, gate_kind=0), {}, "out_gate"), ({}, dict(ws=None), "workspace"),
    ({}, dict(ws=FAKE + 128), "workspace"), ({}, dict(ws_bytes=100), "too small"), ({}, dict(grad_x=FAKE + 8), "16-byte"),
    ({}, dict(grad_h=FAKE + 2), "16-byte"), ({}, dict(out_x=FAKE + 4), "16-byte"), ({}, dict(out_y=FAKE + 4), "16-byte"),
    ({}, dict(out_weight=FAKE + 2), "4-byte"), ({}, dict(out_gate=FAKE + 1), "4-byte"),
    ({}, dict(out_x=None, out_y=None, out_weight=None, out_y_weight=None, out_gate=None), "nothing to write"),
])
def test_norm_backward_refusals(kw, a, msg):
    b = dict(grad_x=FAKE, grad_h=FAKE, out_x=FAKE, out_y=FAKE, out_weight=FAKE, out_y_weight=FAKE, out_gate=FAKE, ws=FAKE,
             ws_bytes=1 << 30, stream=None)
    b.update(a)
    _refused(ep.ep_block_norm_backward(_args(**kw), **b), msg)


def test_norm_null_arguments_and_workspace():
    _refused(ep.ep_block_norm(None, FAKE, FAKE, None, None, None), "args")
    _refused(ep.ep_block_norm_backward(None, *([FAKE] * 8), 1 << 30, None), "args")
    for bad in ((-1, 256), (10, 0), (10, 12), (10, 32776), (2 ** 31 - 1, 256)):
        assert ep.ep_block_norm_workspace_bytes(*bad) == 0
    for rows in (0, 1, 7, 600, 1 << 20, 0x7FFFFF00):
        for width in (8, 1000, 7168, 32768):
            n = ep.ep_block_norm_workspace_bytes(rows, width)
            assert n % 256 == 0 and 2 * width * 4 <= n <= 512 * 2 * width * 4 + 255   # at most 512 workgroups' sums


def test_norm_struct_matches_the_header():
    """The struct's size and order as the C compiler lays them out: pointers, 64-bit, then 32-bit fields."""
    assert ctypes.sizeof(ep.ep_block_norm_t) == 5 * 8 + 2 * 8 + 8 * 4 + 4 * 4
    assert ep.ep_block_norm_t.x_ld.offset == 40 and ep.ep_block_norm_t.num_rows.offset == 56
    assert ep.ep_block_norm_t.weight_offset.offset == 100


WEIGHTS = dict(w=FAKE, w_f32=0, num_groups=4, n=256, k=128, codes=FAKE, scales=FAKE, stream=None)
BACK = dict(codes=FAKE, scales=FAKE, num_groups=4, n=256, k=128, out=FAKE, out_f32=0, stream=None)
GEMM = dict(x=FAKE, x_scales=FAKE, scale_ld=0, w=FAKE, w_scales=FAKE, group_offsets=FAKE, num_groups=4, group_stride=0,
            num_rows=100, n=256, k=128, expected_rows=0, out=FAKE, stream=None)


@pytest.mark.parametrize("name,args,kw,msg", [
    ("ep_quantize_weights_fp4", WEIGHTS, dict(n=100), "n=100"), ("ep_quantize_weights_fp4", WEIGHTS, dict(k=64), "k=64"),
    ("ep_quantize_weights_fp4", WEIGHTS, dict(num_groups=0), "num_groups"),
    ("ep_quantize_weights_fp4", WEIGHTS, dict(num_groups=1025), "num_groups"),
    ("ep_quantize_weights_fp4", WEIGHTS, dict(w_f32=2), "w_f32"), ("ep_quantize_weights_fp4", WEIGHTS, dict(w=None), "w must"),
    ("ep_quantize_weights_fp4", WEIGHTS, dict(codes=FAKE + 8), "codes must"),
    ("ep_quantize_weights_fp4", WEIGHTS, dict(scales=FAKE + 1), "scales must"),
    ("ep_quantize_weights_fp4", WEIGHTS, dict(num_groups=33, n=32768, k=32768), "2^35"),
    ("ep_dequantize_weights_fp4", BACK, dict(num_groups=1024, n=32768, k=32768), "2^35"),
    ("ep_dequantize_weights_fp4", BACK, dict(k=0), "k=0"), ("ep_dequantize_weights_fp4", BACK, dict(out_f32=-1), "out_f32"),
    ("ep_dequantize_weights_fp4", BACK, dict(out=FAKE + 2), "out must"),
    ("ep_dequantize_weights_fp4", BACK, dict(codes=None), "codes must"),
    ("ep_dequantize_weights_fp4", BACK, dict(scales=None), "scales must"),
    ("ep_grouped_gemm_fp4", GEMM, dict(n=130), "n=130"), ("ep_grouped_gemm_fp4", GEMM, dict(k=32768 + 128), "k="),
    ("ep_grouped_gemm_fp4", GEMM, dict(num_groups=0), "num_groups"),
    ("ep_grouped_gemm_fp4", GEMM, dict(group_stride=-1), "group_stride"),
    ("ep_grouped_gemm_fp4", GEMM, dict(num_rows=-1), "num_rows"),
    ("ep_grouped_gemm_fp4", GEMM, dict(num_rows=2 ** 31 - 1), "num_rows"),
    ("ep_grouped_gemm_fp4", GEMM, dict(group_offsets=FAKE + 2), "group_offsets"),
    ("ep_grouped_gemm_fp4", GEMM, dict(group_offsets=None), "group_offsets"),
    ("ep_grouped_gemm_fp4", GEMM, dict(scale_ld=50), "scale_ld"), ("ep_grouped_gemm_fp4", GEMM, dict(scale_ld=102), "scale_ld"),
    ("ep_grouped_gemm_fp4", GEMM, dict(expected_rows=-1), "expected_rows"),
    ("ep_grouped_gemm_fp4", GEMM, dict(w=FAKE + 8), "w must"), ("ep_grouped_gemm_fp4", GEMM, dict(w_scales=FAKE + 2), "w_scales"),
    ("ep_grouped_gemm_fp4", GEMM, dict(x=None), "x must"), ("ep_grouped_gemm_fp4", GEMM, dict(x_scales=None), "x_scales"),
    ("ep_grouped_gemm_fp4", GEMM, dict(out=FAKE + 2), "out must"),
])
def test_fp4_refusals(name, args, kw, msg):
    a = dict(args)
    a.update(kw)
    _refused(getattr(ep, name)(**a), msg)


def test_binding_refusals():
    bf = torch.bfloat16
    x = torch.zeros(4, 256, dtype=bf)
    w = torch.zeros(256, dtype=bf)
    with pytest.raises(ValueError, match="GPU"):
        ep.block_norm(x)
    with pytest.raises(ValueError, match="GPU"):
        ep.block_norm_backward(x, grad_h=x)
    f8, e8 = torch.float8_e4m3fn, torch.float8_e8m0fnu
    off = torch.zeros(3, dtype=torch.int32)
    x8, xs = torch.zeros(4, 256, dtype=torch.uint8).view(f8), torch.zeros(4, 2)
    w4, ws = torch.zeros(2, 128, 128, dtype=torch.uint8), torch.zeros(2, 128, 8, dtype=torch.uint8).view(e8)
    with pytest.raises(ValueError, match=r"\[G, N, K\]"):
        ep.quantize_weights_fp4(w)
    with pytest.raises(TypeError, match="bfloat16"):
        ep.quantize_weights_fp4(torch.zeros(1, 128, 128, dtype=torch.float16))
    with pytest.raises(ValueError, match="K=100"):
        ep.quantize_weights_fp4(torch.zeros(1, 128, 100))
    with pytest.raises(ValueError, match="GPU"):
        ep.quantize_weights_fp4(torch.zeros(1, 128, 128))
    with pytest.raises(ValueError, match="GPU"):
        ep.dequantize_weights_fp4(ep.Fp4Weights(w4, ws))
    with pytest.raises(ValueError, match="w_scales"):
        ep.dequantize_weights_fp4(ep.Fp4Weights(w4, ws[:1]))
    with pytest.raises(ValueError, match="GPU"):
        ep.grouped_gemm_fp4(x8, xs, w4, ws, off)
    with pytest.raises(ValueError, match="w must be"):
        ep.grouped_gemm_fp4(x8[:, :128], xs[:, :1], w4, ws, off)
    with pytest.raises(ValueError, match="x_scales"):
        ep.grouped_gemm_fp4(x8, xs.t(), w4, ws, off)
    for n in (2 ** 31, 2 ** 32, 2 ** 32 + 5):
        with pytest.raises(ValueError, match="group_stride"):
            ep.grouped_gemm_fp4(x8, xs, w4, ws, off, group_stride=n)
        with pytest.raises(ValueError, match="expected_rows"):
            ep.grouped_gemm_fp4(x8, xs, w4, ws, off, expected_rows=n)
