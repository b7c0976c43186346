"""Host-side checks of the block-scaled entry points (include/gbfuse_block.h):
exports, argument validation of the C ABI with addresses that are never read,
and the Python binding's operand checks.  No kernel is launched."""
import os
import re
import subprocess

import pytest
import torch

from conftest import ROOT
from test_decode_host import A, call, gbf, last   # noqa: F401


def test_block_header_and_exports(gbf):
    text = open(os.path.join(ROOT, "include", "gbfuse_block.h")).read()
    declared = set(re.findall(r"GBF_API\s+[\w\s\*]+?\b(gbfb_\w+)\s*\(", text))
    out = subprocess.run(["nm", "-D", "--defined-only", gbf.LIB_PATH], capture_output=True, text=True).stdout
    assert set(re.findall(r"\bT (gbfb_\w+)", out)) == declared == set(gbf.EXPORTED_BLOCK)


def test_add_rmsnorm_validation(gbf):
    names = lambda: [("x", A(0)), ("res", A(1)), ("out", A(2)), ("gate", None), ("mode", 0), ("weight", A(3)),  # noqa
                     ("scale", None), ("shift", None), ("q", A(4)), ("s", A(5)), ("rows", 4), ("hidden", 64),
                     ("eps", 1e-6), ("stream", None)]
    f = lambda **k: call(gbf.raw().gbfb_add_rmsnorm_fp8, names(), k)              # noqa: E731
    assert f(rows=0) == gbf.OK
    for bad in (dict(rows=-1), dict(hidden=0), dict(mode=3), dict(eps=-1.0), dict(eps=float("nan")), dict(weight=None),
                dict(mode=2), dict(mode=2, scale=A(6)), dict(x=None), dict(res=None), dict(out=None), dict(q=None),
                dict(s=None), dict(out=A(0)), dict(out=A(1, 16)), dict(q=A(1, 16)), dict(s=A(3)), dict(s=A(4, 16)),
                dict(q=A(2, 16)), dict(gate=A(2))):
        assert f(**bad) == gbf.EINVAL, bad
    for bad in (dict(hidden=72), dict(x=A(0, 8)), dict(out=A(2, 8)), dict(s=A(5, 2)), dict(weight=A(3, 8)),
                dict(gate=A(6, 8))):
        assert f(**bad) == gbf.EALIGN, bad
    assert f(hidden=32784) == gbf.EUNSUPPORTED and "32768" in last(gbf)
    assert f(rows=1 << 60) == gbf.EUNSUPPORTED


@pytest.mark.parametrize("which", ["gated", "quantize"])
def test_quantiser_validation(gbf, which):
    names = lambda: [("x", A(0)), ("q", A(1)), ("s", A(2)), ("rows", 4), ("d", 64),                            # noqa
                     ("act", 3 if which == "gated" else 1), ("stream", None)]
    fn = gbf.raw().gbfb_gated_act_fp8 if which == "gated" else gbf.raw().gbfb_quantize_fp8
    f = lambda **k: call(fn, names(), k)                                           # noqa: E731
    assert f(rows=0) == gbf.OK
    for bad in (dict(rows=-1), dict(d=0), dict(act=0 if which == "gated" else 64), dict(act=-1), dict(x=None),
                dict(q=None), dict(s=None), dict(q=A(0, 64)), dict(s=A(0, 16)), dict(s=A(1, 16))):
        assert f(**bad) == gbf.EINVAL, bad
    for bad in (dict(d=72), dict(x=A(0, 8)), dict(q=A(1, 8)), dict(s=A(2, 2))):
        assert f(**bad) == gbf.EALIGN, bad
    assert f(d=1 << 31) == gbf.EUNSUPPORTED
    if which == "quantize":
        assert f(rows=1 << 38, d=128, act=128) == gbf.EUNSUPPORTED and "128 x 128" in last(gbf)


def test_linear_validation(gbf):
    names = lambda: [("x", A(0)), ("sx", A(1)), ("w", A(2)), ("sw", A(3)), ("bias", None), ("y", A(4)),       # noqa
                     ("m", 4), ("n", 64), ("k", 256), ("act", 0), ("stream", None)]
    f = lambda **k: call(gbf.raw().gbfb_linear_fp8, names(), k)                    # noqa: E731
    assert f(m=0) == gbf.OK
    for bad in (dict(m=-1), dict(n=0), dict(k=0), dict(act=4), dict(act=-1), dict(x=None), dict(sx=None), dict(w=None),
                dict(sw=None), dict(y=None), dict(y=A(0, 16)), dict(y=A(1)), dict(y=A(2)), dict(y=A(3)),
                dict(bias=A(4, 16))):
        assert f(**bad) == gbf.EINVAL, bad
    for bad in (dict(k=136), dict(n=60), dict(m=1 << 31), dict(n=1 << 31), dict(k=1 << 31),
                dict(m=(1 << 31) - 1, n=(1 << 31) - 8)):
        assert f(**bad) == gbf.EUNSUPPORTED, bad
    for bad in (dict(x=A(0, 8)), dict(w=A(2, 8)), dict(y=A(4, 8)), dict(bias=A(5, 8)), dict(sx=A(1, 2)), dict(sw=A(3, 1))):
        assert f(**bad) == gbf.EALIGN, bad


# ------------------------------------------------------- the Python operands

bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)       # noqa: E731
u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8)          # noqa: E731
f32 = torch.zeros


def test_binding_refuses_operands(gbf):
    norm = dict(x=bf(4, 256), res_in=bf(4, 256), res_out=bf(4, 256), q_out=u8(4, 256), scales=f32(4, 2), mode=1)
    gated = dict(x=bf(4, 512), q_out=u8(4, 256), scales=f32(4, 2))
    quant = dict(x=bf(130, 144), q_out=u8(130, 144), scales=f32(130, 2))
    lin = dict(xq=u8(4, 256), x_scales=f32(4, 2), wq=u8(136, 256), w_scales=f32(2, 2), bias=None, y=bf(4, 136))
    cases = [
        (gbf.add_rmsnorm_fp8_block, norm, dict(scales=f32(4, 1)), ValueError, "scales: holds 4"),
        (gbf.add_rmsnorm_fp8_block, norm, dict(res_in=bf(4, 255)), ValueError, "res_in"),
        (gbf.add_rmsnorm_fp8_block, norm, dict(weight=bf(255)), ValueError, "weight"),
        (gbf.add_rmsnorm_fp8_block, norm, dict(ada_shift=bf(1)), ValueError, "ada_shift"),
        (gbf.add_rmsnorm_fp8_block, norm, dict(q_out=bf(4, 256)), TypeError, "q_out: expected torch.uint8"),
        (gbf.add_rmsnorm_fp8_block, norm, dict(x=bf(256, 4).t()), ValueError, "contiguous"),
        (gbf.add_rmsnorm_fp8_block, norm, dict(mode="ada"), TypeError, "mode"),
        (gbf.gated_act_fp8_block, gated, dict(x=bf(8, 256)), ValueError, "x: rows of 256"),
        (gbf.gated_act_fp8_block, gated, dict(x=bf(3, 512)), ValueError, "x: holds"),
        (gbf.gated_act_fp8_block, gated, dict(scales=f32(4, 2).bfloat16()), TypeError, "scales: expected torch.float32"),
        (gbf.quantize_fp8_block, quant, dict(scales=f32(2, 2)), ValueError, "scales: holds 4"),
        (gbf.quantize_fp8_block, quant, dict(block_rows=128), ValueError, "the call needs 4"),
        (gbf.quantize_fp8_block, quant, dict(x=f32(130, 144)), TypeError, "x: expected torch.bfloat16"),
        (gbf.quantize_fp8_block, quant, dict(block_rows=1 << 40), ValueError, "32 bits"),
        (gbf.linear_fp8_block, lin, dict(wq=u8(136, 128)), ValueError, "wq: expected"),
        (gbf.linear_fp8_block, lin, dict(wq=u8(136 * 256)), ValueError, "wq: expected"),
        (gbf.linear_fp8_block, lin, dict(x_scales=f32(4, 1)), ValueError, "x_scales"),
        (gbf.linear_fp8_block, lin, dict(w_scales=f32(136, 2)), ValueError, "w_scales"),
        (gbf.linear_fp8_block, lin, dict(bias=bf(4)), ValueError, "bias"),
        (gbf.linear_fp8_block, lin, dict(y=bf(136)), ValueError, "y: holds"),
        (gbf.linear_fp8_block, lin, dict(xq=1), TypeError, "xq: expected a torch.Tensor"),
    ]
    for fn, good, bad, error, text in cases:
        with pytest.raises(error, match=text):
            fn(**{**good, **bad})
    for fn, good in ((gbf.add_rmsnorm_fp8_block, norm), (gbf.gated_act_fp8_block, gated), (gbf.quantize_fp8_block, quant),
                     (gbf.linear_fp8_block, lin)):
        with pytest.raises(ValueError, match="CUDA device"):
            fn(**good)
        with pytest.raises(TypeError, match="missing required"):
            fn(*list(good.values())[:2])
