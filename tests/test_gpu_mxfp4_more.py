"""Further cases of the MXFP4 quantiser, dequantisers and grouped product on the GPU."""
import pytest
import torch

import sigmoid_top_routing_02_amd as moe
from helpers import dev, say
from test_gpu_mxfp4 import F8, offsets, operands, ref_product

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,N,K", [(40000, 1, 65536), (1100000, 1, 32), (1100000, 1, 96), (20000, 1024, 32),
                                   (5000, 256, 65536), (40, 1, 65536), (5, 3, 1056)])
def test_one_row_of_a_and_few_of_b(M, N, K):
    """A of one row, which every row of the product (but two outside A) names, and B of few: the tensors
    are smaller than what the kernels send for ahead.  Scales of 1: every product is a multiple of 1/4 of at
    most 36, so that sums of 65536 are binary32 numbers."""
    dev()
    say(f"  M={M} N={N} K={K}")
    aq, a_s, bq, b_s, idx = operands(M, 1, 1, N, K, N + K, low=127, high=128)
    idx[[0, M // 2]] = torch.tensor([1, -1], dtype=torch.int32, device="cuda")
    got = moe.grouped_gemm_mxfp4(aq, a_s, offsets([M]), M, bq, b_s, a_row_index=idx)
    torch.cuda.synchronize()
    row = ref_product(aq, a_s, bq, b_s, None, [1])
    zero = torch.zeros(M, dtype=torch.bool, device="cuda")
    zero[[0, M // 2]] = True
    assert (got[zero] == 0).all() and (got[~zero].to(F8) == row).all()


def test_sizes_past_the_c_abis_integers_are_refused():
    """Widths that a C int would hold modulo 2^32 (as 32, 128 or 1): refused, not taken for those."""
    dev()
    new = lambda *s, dtype=torch.uint8: torch.empty(s, dtype=dtype, device="cuda")  # noqa: E731
    wide, index = 2 ** 32, torch.zeros(1, dtype=torch.int32, device="cuda")
    bad = [
        lambda: moe.mxfp4_quant_1x32(new(1, wide + 32, dtype=torch.bfloat16)),
        lambda: moe.mxfp4_dequant_1x32(new(1, wide // 2 + 16), new(1, wide // 32 + 1)),
        lambda: moe.fp8_dequant_1x128(new(1, wide + 128), new(1, wide // 128 + 1, dtype=torch.float32)),
        lambda: moe.moe_add_rmsnorm(new(1, wide + 1, dtype=torch.bfloat16), new(wide + 1, dtype=torch.bfloat16), 1e-6),
        lambda: moe.moe_add_rmsnorm_backward(new(1, wide + 1, dtype=torch.bfloat16), new(1, wide + 1, dtype=torch.bfloat16),
                                             new(wide + 1, dtype=torch.bfloat16), new(1, dtype=torch.float32)),
        lambda: moe.grouped_gemm_mxfp4(new(1, 16), new(1, 1), offsets([1]), 1, new(1, wide + 1, 16), new(1, wide + 1, 1),
                                       a_row_index=index),
        lambda: moe.grouped_gemm_mxfp4(new(1, wide // 2 + 16), new(1, wide // 32 + 1), offsets([1]), 1,
                                       new(1, 1, wide // 2 + 16), new(1, 1, wide // 32 + 1)),
        lambda: moe.grouped_gemm_mxfp4(new(1, 16), new(1, 1), new(wide + 2, dtype=torch.int32), 1, new(wide + 1, 1, 16),
                                       new(wide + 1, 1, 1), a_row_index=index),
    ]
    taken = []
    for i, f in enumerate(bad):
        say(f"  call {i}")
        try:
            f()
            taken.append(i)
        except moe.MoEError:
            pass
        torch.cuda.synchronize()
        torch.cuda.empty_cache()
    assert not taken


def test_more_columns_than_a_few_row_launch_takes():
    """Few rows on 2^27 columns: 1.5 times 2^32 threads of the kernel that few rows take otherwise.  B repeats
    4099 rows."""
    dev()
    G, per, N, K, period = 8, 8, 2 ** 27, 32, 4099
    M = G * per
    aq, a_s, bq, b_s, _ = operands(M, M, 1, period, K, 12)
    bq, b_s = (t[0].repeat(N // period + 1, 1)[:N].expand(G, N, t.shape[2]).contiguous() for t in (bq, b_s))
    out = moe.grouped_gemm_mxfp4(aq, a_s, offsets([per] * G), M, bq, b_s, epi=moe.MOE_MX_STORE_BF16)
    torch.cuda.synchronize()
    want = ref_product(aq, a_s, bq[:1, :period], b_s[:1, :period], None, [M]).float().bfloat16()
    whole = N // period * period
    assert (out[:, :whole].view(M, -1, period) == want[:, None]).all()
    assert torch.equal(out[:, whole:], want[:, :N - whole])
