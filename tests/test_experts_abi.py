"""CPU checks of the expert layer's entry points: invalid arguments are refused
before any HIP call, and the binding refuses tensors the kernels cannot take."""
import pytest

import combine_get_dispatch_scan_amd as ep

torch = pytest.importorskip("torch")

FAKE = 1 << 20  # never dereferenced: every call below fails validation first


def _refused(fn, args, kw, msg):
    a = dict(args)
    a.update(kw)
    assert fn(**a) == ep.EP_EINVAL
    assert msg in ep.ep_last_error(), ep.ep_last_error()


GATE = dict(logits=FAKE, logits_bf16=0, ld=64, num_tokens=10, num_experts=64, num_topk=8, score=0, normalize=1,
            scale=1.0, balance_coef=0.0, token_mask=None, topk_idx=FAKE, topk_weights=FAKE,
            num_tokens_per_expert=FAKE, num_valid=FAKE, loss=FAKE, ws=FAKE,
            ws_bytes=ep.ep_gate_workspace_bytes(10, 64), stream=None)


@pytest.mark.parametrize("kw,msg", [
    (dict(num_tokens=-1), "invalid dims"), (dict(num_experts=0), "invalid dims"),
    (dict(num_experts=1025, ld=2000), "invalid dims"), (dict(num_topk=0), "invalid dims"),
    (dict(num_topk=17), "invalid dims"), (dict(num_experts=4, num_topk=5), "invalid dims"),
    (dict(num_tokens=1 << 28, num_topk=16), "invalid dims"), (dict(logits_bf16=2), "logits_bf16"),
    (dict(normalize=3), "normalize"), (dict(score=2), "score"), (dict(ld=63), "ld"),
    (dict(logits=None), "logits"), (dict(logits=FAKE + 2), "logits"), (dict(topk_idx=FAKE + 4), "topk_idx"),
    (dict(topk_weights=None), "topk_weights"), (dict(num_tokens_per_expert=None), "num_tokens_per_expert"),
    (dict(num_valid=FAKE + 1), "num_valid"), (dict(loss=None), "loss"), (dict(ws=FAKE + 64), "workspace"),
    (dict(ws_bytes=4), "workspace too small"),
])
def test_gate_refusals(kw, msg):
    _refused(ep.ep_gate, GATE, kw, msg)


GATE_BACK = {k: v for k, v in GATE.items() if k not in ("topk_weights", "loss", "ws", "ws_bytes")}
GATE_BACK.update(grad_weights=FAKE, grad_loss=FAKE, grad_logits=FAKE)


@pytest.mark.parametrize("kw,msg", [
    (dict(num_topk=65), "invalid dims"), (dict(score=-1), "score"), (dict(topk_idx=None), "topk_idx"),
    (dict(grad_logits=None), "grad_logits"), (dict(grad_weights=FAKE + 2), "grad_weights"),
    (dict(grad_loss=FAKE + 1), "grad_loss"), (dict(num_valid=None), "num_valid"),
])
def test_gate_backward_refusals(kw, msg):
    _refused(ep.ep_gate_backward, GATE_BACK, kw, msg)


GROUPS = dict(group_offsets=FAKE, num_groups=4, group_stride=0, num_rows=100)
GROUP_CASES = [
    (dict(num_groups=0), "num_groups"), (dict(num_groups=1025), "num_groups"),
    (dict(group_stride=-1), "group_stride"), (dict(num_rows=-1), "num_rows"),
    (dict(num_rows=2 ** 31 - 1), "num_rows"), (dict(group_offsets=FAKE + 2), "group_offsets"),
]
ROWS = dict(x=FAKE, width=256, **GROUPS, scale_ld=0, codes=FAKE, scales=FAKE, stream=None)
WEIGHTS = dict(w=FAKE, w_f32=0, num_groups=4, n=256, k=128, codes=FAKE, scales=FAKE, codes_t=FAKE, scales_t=FAKE,
               stream=None)
GEMM = dict(x=FAKE, x_scales=FAKE, scale_ld=0, w=FAKE, w_scales=FAKE, **GROUPS, n=256, k=128, expected_rows=0,
            out=FAKE, stream=None)
WGRAD = dict(grad=FAKE, x=FAKE, x_scales=FAKE, scale_ld=0, **GROUPS, n=256, k=128, out=FAKE, out_f32=0, stream=None)
SWIGLU = dict(h=FAKE, inner=256, **GROUPS, scale_ld=0, codes=FAKE, scales=FAKE, ckpt=FAKE, ckpt_scales=FAKE,
              stream=None)
SWIGLU_BACK = dict(grad_a=FAKE, ckpt=FAKE, ckpt_scales=FAKE, inner=256, **GROUPS, scale_ld=0, grad_h=FAKE,
                   codes=FAKE, scales=FAKE, stream=None)


@pytest.mark.parametrize("name,args", [("ep_quantize_rows", ROWS), ("ep_grouped_gemm_fp8", GEMM),
                                       ("ep_grouped_wgrad_fp8", WGRAD), ("ep_swiglu_fp8", SWIGLU),
                                       ("ep_swiglu_fp8_backward", SWIGLU_BACK)])
@pytest.mark.parametrize("kw,msg", GROUP_CASES + [(dict(scale_ld=50), "scale_ld"), (dict(scale_ld=102), "scale_ld")])
def test_group_refusals(name, args, kw, msg):
    _refused(getattr(ep, name), args, kw, msg)


@pytest.mark.parametrize("name,args,kw,msg", [
    ("ep_quantize_rows", ROWS, dict(width=100), "width"),
    ("ep_quantize_rows", ROWS, dict(width=32768 + 128), "width"),
    ("ep_quantize_rows", ROWS, dict(x=FAKE + 8), "x must"),
    ("ep_quantize_rows", ROWS, dict(scales=None), "scales"),
    ("ep_quantize_rows", ROWS, dict(group_offsets=None), "num_groups"),
    ("ep_quantize_rows", ROWS, dict(num_rows=(1 << 28) + 1), "2^29"),
    ("ep_quantize_weights", WEIGHTS, dict(n=100), "n=100"),
    ("ep_quantize_weights", WEIGHTS, dict(k=0), "k=0"),
    ("ep_quantize_weights", WEIGHTS, dict(num_groups=0), "num_groups"),
    ("ep_quantize_weights", WEIGHTS, dict(w_f32=2), "w_f32"),
    ("ep_quantize_weights", WEIGHTS, dict(w=None), "w must"),
    ("ep_quantize_weights", WEIGHTS, dict(codes=FAKE + 4), "codes must"),
    ("ep_quantize_weights", WEIGHTS, dict(scales_t=None), "together"),
    ("ep_grouped_gemm_fp8", GEMM, dict(n=130), "n=130"),
    ("ep_grouped_gemm_fp8", GEMM, dict(k=64), "k=64"),
    ("ep_grouped_gemm_fp8", GEMM, dict(expected_rows=-1), "expected_rows"),
    ("ep_grouped_gemm_fp8", GEMM, dict(w_scales=None), "w_scales"),
    ("ep_grouped_gemm_fp8", GEMM, dict(out=FAKE + 2), "out must"),
    ("ep_grouped_gemm_fp8", GEMM, dict(group_offsets=None), "group_offsets"),
    ("ep_grouped_wgrad_fp8", WGRAD, dict(out_f32=5), "out_f32"),
    ("ep_grouped_wgrad_fp8", WGRAD, dict(out=None), "out must"),
    ("ep_grouped_wgrad_fp8", WGRAD, dict(grad=FAKE + 4), "grad must"),
    ("ep_swiglu_fp8", SWIGLU, dict(inner=64), "inner"),
    ("ep_swiglu_fp8", SWIGLU, dict(ckpt_scales=None), "together"),
    ("ep_swiglu_fp8", SWIGLU, dict(h=None), "h must"),
    ("ep_swiglu_fp8_backward", SWIGLU_BACK, dict(grad_h=None, codes=None, scales=None), "nothing to write"),
    ("ep_swiglu_fp8_backward", SWIGLU_BACK, dict(codes=None), "together"),
    ("ep_swiglu_fp8_backward", SWIGLU_BACK, dict(ckpt=FAKE + 1), "ckpt must"),
])
def test_refusals(name, args, kw, msg):
    _refused(getattr(ep, name), args, kw, msg)


def test_gate_workspace():
    assert ep.ep_gate_workspace_bytes(-1, 8) == 0 and ep.ep_gate_workspace_bytes(8, 0) == 0
    assert ep.ep_gate_workspace_bytes(8, 1025) == 0
    for T in (0, 1, 128, 1000, 5000, 1 << 20):
        for E in (1, 60, 256, 512, 1024):
            assert ep.ep_gate_workspace_bytes(T, E) >= (2 * E + 1) * 4
    # bounded: at most 256 workgroups' sums
    assert ep.ep_gate_workspace_bytes(1 << 30, 256) == 256 * (2 * 256 + 1) * 4


def test_binding_refuses_cpu_tensors_and_wrong_shapes():
    f8 = torch.float8_e4m3fn
    off = torch.zeros(3, dtype=torch.int32)
    x, xs = torch.zeros(4, 256, dtype=torch.uint8).view(f8), torch.zeros(4, 2)
    w, ws = torch.zeros(2, 128, 256, dtype=torch.uint8).view(f8), torch.zeros(2, 1, 2)
    with pytest.raises(ValueError, match="GPU"):
        ep.gate(torch.zeros(4, 8), 2)
    with pytest.raises(TypeError, match="float32 or torch.bfloat16"):
        ep.gate(torch.zeros(4, 8, dtype=torch.float64), 2)
    with pytest.raises(ValueError, match="score"):
        ep.gate(torch.zeros(4, 8), 2, score="relu")
    with pytest.raises(ValueError, match="token_mask"):
        ep.gate(torch.zeros(4, 8), 2, token_mask=torch.zeros(3, dtype=torch.uint8))
    with pytest.raises(ValueError, match="contiguous"):
        ep.gate(torch.zeros(8, 4).t(), 2)
    with pytest.raises(ValueError, match="overlap"):
        ep.gate(torch.zeros(8).expand(4, 8), 2)
    with pytest.raises(ValueError, match="GPU"):
        ep.quantize_rows(torch.zeros(4, 256, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="multiple of 128"):
        ep.quantize_rows(torch.zeros(4, 100, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match=r"\[G, N, K\]"):
        ep.quantize_weights(torch.zeros(4, 128))
    with pytest.raises(TypeError, match="bfloat16"):
        ep.quantize_weights(torch.zeros(1, 128, 128, dtype=torch.float16))
    with pytest.raises(ValueError, match="GPU"):
        ep.grouped_gemm_fp8(x, xs, w, ws, off)
    with pytest.raises(ValueError, match="w must be"):
        ep.grouped_gemm_fp8(x, xs, w.transpose(1, 2), ws, off)
    with pytest.raises(ValueError, match="w_scales"):
        ep.grouped_gemm_fp8(x, xs, w, ws.transpose(1, 2), off)
    with pytest.raises(ValueError, match="x_scales"):
        ep.grouped_gemm_fp8(x, xs.t(), w, ws, off)
    with pytest.raises(ValueError, match="column-major"):
        ep.grouped_gemm_fp8(x, torch.zeros(2, 6), w, ws, off, column_major_scales=True)
    with pytest.raises(ValueError, match="grad must"):
        ep.grouped_wgrad_fp8(torch.zeros(3, 128, dtype=torch.bfloat16), x, xs, off)
    with pytest.raises(ValueError, match="inner"):
        ep.swiglu_fp8(torch.zeros(3, 200, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="ckpt"):
        ep.swiglu_fp8_backward(torch.zeros(3, 128, dtype=torch.bfloat16), x, xs)


def test_binding_refuses_numbers_past_32_bits():
    """The C calls take them as int: 2^32 would arrive as 0."""
    f8 = torch.float8_e4m3fn
    off = torch.zeros(3, dtype=torch.int32)
    x, xs = torch.zeros(4, 256, dtype=torch.uint8).view(f8), torch.zeros(4, 2)
    w, ws = torch.zeros(2, 128, 256, dtype=torch.uint8).view(f8), torch.zeros(2, 1, 2)
    meta = lambda *s, dt=torch.bfloat16: torch.empty(*s, dtype=dt, device="meta")  # noqa: E731
    for n in (2 ** 31, 2 ** 32, 2 ** 32 + 5):
        with pytest.raises(ValueError, match="2\\^31"):
            ep.gate(meta(n, 1), 1)
        with pytest.raises(ValueError, match="2\\^31"):
            ep.gate_backward(meta(n, 1), None)
        with pytest.raises(ValueError, match="2\\^31"):
            ep.quantize_rows(meta(n, 128))
        with pytest.raises(ValueError, match="2\\^31"):
            ep.swiglu_fp8(meta(n, 256))
        with pytest.raises(ValueError, match="group_stride"):
            ep.grouped_gemm_fp8(x, xs, w, ws, off, group_stride=n)
        with pytest.raises(ValueError, match="group_stride"):
            ep.quantize_rows(torch.zeros(4, 256, dtype=torch.bfloat16), off, group_stride=n)
        with pytest.raises(ValueError, match="expected_rows"):
            ep.grouped_gemm_fp8(x, xs, w, ws, off, expected_rows=n)
        with pytest.raises(ValueError, match="num_topk"):
            ep.gate(torch.zeros(4, 8), n)
        with pytest.raises(ValueError, match="experts"):
            ep.gate(meta(1, n), 1)
    with pytest.raises(ValueError, match="2\\^31"):
        ep.quantize_rows(meta(1, 2 ** 32 + 128))


@pytest.mark.parametrize("name,args,width", [("ep_quantize_rows", ROWS, "width"), ("ep_swiglu_fp8", SWIGLU, "inner"),
                                             ("ep_swiglu_fp8_backward", SWIGLU_BACK, "inner")])
@pytest.mark.parametrize("rows", [1 << 22, (1 << 22) - 1 + (1 << 20)])
def test_row_calls_refuse_more_than_a_launch_covers(name, args, width, rows):
    """2^29 blocks of 128 are 2^32 threads, one more than a launch can have."""
    _refused(getattr(ep, name), args, {width: 16384, "num_rows": rows}, "2^29")
