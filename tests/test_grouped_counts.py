"""Sizes past 32 bits, which the C ABI cannot be given, are refused by the binding (tensors without memory, on the CPU)."""
import pytest
import torch

import moe_dispatch_expert_amd as mk

BIG = 2 ** 32 + 8   # its low 32 bits are a size that the calls take
BF, I32, I8, F32 = torch.bfloat16, torch.int32, torch.int8, torch.float32


def _t(*shape, dtype=BF):
    return torch.empty(shape, dtype=dtype, device="meta")


def _off(E):
    return _t(E + 1, dtype=I32)


CALLS = {
    "layout_tokens": lambda: mk.mk_expert_layout(_t(BIG, 2, dtype=I32), 8),
    "layout_begin": lambda: mk.mk_expert_layout(_t(4, 2, dtype=I32), 8, BIG),
    "combine_tokens": lambda: mk.mk_combine_backward(_t(BIG, 8), _t(4, 8), _t(BIG, 1, dtype=I32), _t(BIG, 1, dtype=F32)),
    "combine_rows": lambda: mk.mk_combine_backward(_t(4, 8), _t(BIG, 8), _t(4, 1, dtype=I32), _t(4, 1, dtype=F32)),
    "combine_columns": lambda: mk.mk_combine_backward(_t(4, BIG), _t(4, BIG), _t(4, 1, dtype=I32), _t(4, 1, dtype=F32)),
    "swiglu_rows": lambda: mk.mk_swiglu_backward(_t(BIG, 16), _t(BIG, 8)),
    "swiglu_columns": lambda: mk.mk_swiglu_backward(_t(4, 2 * BIG), _t(4, BIG)),
    "dgrad_rows": lambda: mk.mk_grouped_gemm_dgrad(_t(BIG, 8), _off(1), _t(1, 8, 8)),
    "wgrad_rows": lambda: mk.mk_grouped_gemm_wgrad(_t(BIG, 8), _t(BIG, 8), _off(1)),
    "wgrad_tokens": lambda: mk.mk_grouped_gemm_wgrad(_t(8, 8), _t(BIG, 8), _off(1), row_token=_t(8, dtype=I32)),
    "quant_rows": lambda: mk.mk_quant_i8(_t(BIG, 8)),
    "quant_columns": lambda: mk.mk_quant_i8(_t(2, BIG)),
    "swiglu_i8_rows": lambda: mk.mk_swiglu_i8(_t(BIG, 16)),
    "i8_rows": lambda: mk.mk_grouped_gemm_i8(_t(BIG, 16, dtype=I8), _t(BIG, dtype=F32), _off(1), _t(1, 8, 16, dtype=I8),
                                             _t(1, 8, dtype=F32)),
    "i8_gathered_rows": lambda: mk.mk_grouped_gemm_i8(_t(8, 16, dtype=I8), _t(8, dtype=F32), _off(1), _t(1, 8, 16, dtype=I8),
                                                      _t(1, 8, dtype=F32), row_token=_t(BIG, dtype=I32)),
}


@pytest.mark.parametrize("name", sorted(CALLS))
def test_sizes_past_32_bits_are_refused(name):
    with pytest.raises(ValueError, match=r"2\^31 - 1"):
        CALLS[name]()
