"""Rows of the feed-forward block that are as long as rows may be."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def test_copies_of_the_longest_rows(cuda):
    """x of 2^30 - 1 columns, whose rows are copied to 16 bytes, and the weights' gradients that are made
    of it.  Small integers, gates of 32: every number is exact."""
    import dense_fp32_gemm_09_gb300 as sg
    M, K = 3, 2 ** 30 - 1
    torch.cuda.empty_cache()
    whole = lambda rows, seed: torch.randint(
        -2, 3, (rows, K), dtype=torch.int8, device="cuda",
        generator=torch.Generator("cuda").manual_seed(seed)).bfloat16()
    x, wg, wu = whole(M, 1), whole(1, 2), whole(1, 3)
    of = lambda *v: torch.tensor(v, device="cuda").bfloat16()[:, None]
    dh, g, u = of(1, -2, 1), of(32, 32, 64), of(2, 1, -1)
    dx, dwg, dwu = sg.gated_ff_backward(dh, x, wg, wu, (g, u))
    dg, du = (dh.float() * u.float()), (dh.float() * g.float())
    for c in range(0, K, 2 ** 27):
        at = slice(c, min(c + 2 ** 27, K))
        assert torch.equal(dwg[:, at], (dg.t() @ x[:, at].float()).bfloat16())
        assert torch.equal(dwu[:, at], (du.t() @ x[:, at].float()).bfloat16())
        assert torch.equal(dx[:, at], (dg * wg[:, at].float() + du * wu[:, at].float()).bfloat16())
    del x, wg, wu, dx, dwg, dwu
    torch.cuda.empty_cache()
