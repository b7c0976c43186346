"""Operands without a dimension: refused by name, as any other wrong extent."""
import pytest
import torch

from test_decode_host import gbf   # noqa: F401

bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)       # noqa: E731
u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8)          # noqa: E731


def test_operands_without_a_dimension(gbf):                                           # noqa: F811
    f32, dot = torch.zeros, ()
    for call, name in ((lambda: gbf.gated_act_fp8_block(bf(dot), u8(4, 256), f32(4, 2)), "x: rows of 0"),
                       (lambda: gbf.gated_act_fp8_block(bf(4, 512), u8(dot), f32(4, 2)), "x: rows of 512"),
                       (lambda: gbf.quantize_fp8_block(bf(dot), u8(dot), f32(dot)), "x: holds 1"),
                       (lambda: gbf.add_rmsnorm_fp8_block(*[bf(dot)] * 3, u8(dot), f32(dot), 1), "x: holds 1"),
                       (lambda: gbf.linear_fp8_block(u8(dot), f32(dot), u8(8, 16), f32(1, 1), None, bf(1, 8)), "wq: expected"),
                       (lambda: gbf.linear_fp8_block(u8(4, 16), f32(4, 1), u8(dot), f32(1, 1), None, bf(4, 8)), "wq: expected")):
        with pytest.raises(ValueError, match=name):
            call()
