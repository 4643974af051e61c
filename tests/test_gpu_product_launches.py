"""An 8-bit product of more workgroups than one launch takes, on an MI355X."""
import pytest
import torch

import dispatch_fp8_grouped_topk_amd as mm
from test_gpu_parts import _check_product, _codes

pytestmark = pytest.mark.gpu


def test_a_product_launched_in_parts():
    """1023 groups of one row, then one of the others: its last tiles come in the second part, 2^22 workgroups on.  137 GB
    of weights, of which three groups' are looked at."""
    M, N, K, G = 4096, 1 << 20, 128, 1024
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 160 << 30:
        pytest.skip("needs 160 GiB of free device memory")
    g = torch.Generator().manual_seed(1)
    x, x_sf = _codes(M, K, g).cuda(), torch.rand(M, 1, generator=g).add_(0.5).mul_(0.01).cuda()
    w_sf = torch.rand(G, N // 128, 1, generator=g).add_(0.5).mul_(0.001).cuda()
    w = torch.empty(G, N, K, dtype=torch.uint8, device="cuda")
    block = _codes(1 << 12, K, g).cuda()
    groups = (0, 700, G - 1)
    for i in groups:
        w[i] = block.roll(i, 0).repeat(N >> 12, 1)
    offset = torch.arange(G + 1, dtype=torch.int32, device="cuda")
    offset[G] = M
    y = torch.zeros(M, N, dtype=torch.bfloat16, device="cuda")
    mm.mega_moe_block_product(mm.ProductProblem.make(M, N, K, G), x, x_sf, w, w_sf, y, group_offset=offset)
    torch.cuda.synchronize()
    for i in groups:
        lo, hi = int(offset[i]), int(offset[i + 1])
        for nb in (0, 1, 4095, 6000, N // 128 - 1):
            cols = slice(128 * nb, 128 * nb + 128)
            _check_product(y[lo:hi, cols], x[lo:hi], x_sf[lo:hi], w[i:i + 1, cols].contiguous(), w_sf[i:i + 1, nb:nb + 1].contiguous())
    # every column of the last group: the weights repeat every 32 blocks, the scales do not; two BF16 roundings apart
    last = y[G - 1:].view(M - G + 1, N // 128, 128).float() / w_sf[G - 1].view(1, -1, 1)
    first = last[:, :32]
    for lo in range(32, N // 128, 1024):
        part = last[:, lo:lo + 1024]
        part = part[:, :part.shape[1] // 32 * 32].reshape(M - G + 1, -1, 32, 128)
        assert ((part - first[:, None]).abs() <= 2.0 ** -7 * 1.01 * first[:, None].abs()).all()
    del w, y, last
    torch.cuda.empty_cache()
