"""A workspace of qlinear_w4a16 made for a number of rows serves fewer rows too."""
import numpy as np
import pytest
import torch

from bit_gemm_block_amd import decode as D
from oracle import decode_oracle as O


@pytest.mark.parametrize("N,K", [(4096, 14336), (4096, 4096), (28672, 4096), (855, 1472), (16, 16384), (1, 64), (70000, 512)])
def test_size_does_not_shrink(N, K):
    sizes = [D.qlinear_w4a16_workspace_size(M, N, K) for M in (*range(1, 1400), 4096, 65536, 4194240)]
    assert sizes == sorted(sizes)
    assert sizes[15] == 0                        # up to 16 rows need none


@pytest.mark.gpu
@pytest.mark.parametrize("most", [64, 65, 129, 400, 3000])
def test_one_workspace_for_all_rows(most):
    print("w4a16 workspace", most, flush=True)
    N, K = 1040, 2048
    rng = np.random.default_rng(most)
    x = rng.integers(-3, 4, (most, K)).astype(np.float16)        # whole numbers: exact in any order
    q = rng.integers(-8, 8, (N, K))
    ref = (x.astype(np.float64) @ q.T).astype(np.float32)
    dev = lambda a: torch.from_numpy(a).to("cuda:0")  # noqa: E731
    w, s, xd = dev(O.tile(O.pack(q, 4))), torch.ones(N, dtype=torch.float16, device="cuda:0"), dev(x)
    size = D.qlinear_w4a16_workspace_size(most, N, K)
    own = torch.full((size + 64,), 0x5a, dtype=torch.uint8, device="cuda:0")
    for M in sorted({1, 16, 17, 32, 33, 64, 65, 128, 129, 200, most} - set(range(most + 1, 300))):
        y = D.qlinear_w4a16(xd[:M], w, s, workspace=own[:size])
        torch.cuda.synchronize()
        assert np.array_equal(y.cpu().numpy(), ref[:M]), M
    assert bool((own[size:] == 0x5a).all())
