"""CPU checks of the workspace sizes of the products with adapters: nothing for arguments that the call rejects, a
function of the arguments alone, and room for the copy of rows that do not start at 16-byte addresses."""
import pytest
import torch

import dequant_gemm_quantize_amd as w4

GOOD = {"m": 12, "k": 4096, "n": 11008, "group_size": 128, "rank": 16, "segments": 3}
BAD = [("rank", 0), ("rank", -8), ("rank", 4), ("rank", 12), ("rank", 264), ("segments", -1), ("segments", (1 << 20) + 1),
       ("m", -1), ("m", 0), ("m", (1 << 24) + 1), ("k", 0), ("k", 4097), ("n", 0), ("n", -1), ("group_size", 48)]


@pytest.mark.parametrize("name,value", BAD)
def test_rejected_arguments_have_no_size(name, value):
    assert w4.w4a16_lora_matmul_t_workspace_size(**GOOD) > 0
    assert w4.w4a16_lora_matmul_t_workspace_size(**{**GOOD, name: value}) == 0
    if name not in ("rank", "segments"):
        args = {k: v for k, v in {**GOOD, name: value}.items() if k not in ("rank", "segments")}
        assert w4.w4a16_matmul_t_workspace_size(**args) == 0
        assert w4.w4a16_lora_matmul_workspace_size(**args) == 0


def test_rejected_types_have_no_size():
    for name in ("dy_dtype", "sz_dtype", "dx_dtype"):
        bad = torch.bfloat16 if name == "sz_dtype" else torch.float16
        assert w4.w4a16_lora_matmul_t_workspace_size(**GOOD, **{name: bad}) == 0


def test_no_segments_need_no_more_than_the_product():
    own = w4.w4a16_matmul_t_workspace_size(12, 4096, 11008, 128)
    assert w4.w4a16_lora_matmul_t_workspace_size(**{**GOOD, "segments": 0}) == own
    more = w4.w4a16_lora_matmul_t_workspace_size(**GOOD) - own
    assert more > 0 and more % (12 * 16 * 4) == 0  # whole parts of v


@pytest.mark.parametrize("m,n", [(65, 11001), (2048, 11001), (333, 4090)])
def test_rows_copied_to_aligned_ones(m, n):
    size, rows = w4.w4a16_matmul_t_workspace_size(m, 4096, n, 128), m * -(-n // 8) * 16
    sums = size - -(-rows // 128) * 128
    assert sums >= 0 and sums % (4 * m * 4096) == 0
