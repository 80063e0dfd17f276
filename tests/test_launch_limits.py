"""A grid of HIP holds less than 2^32 threads along each dimension, more is refused at the
launch: the norm and feed-forward calls stay below it at every size that the header
allows (the gradient product's at what fits this GPU's memory).  CPU only."""

import pytest

from tests import launches

ROWS = 1 << 25                                          # MXQ_NORM_MAX_ROWS


def _threads(done):
    return [max(g * b for g, b in zip(t.grid, t.block)) for t in done]


@pytest.mark.parametrize("K", [32, 512, 544, 1024, 1056, 2048, 2080, 4096, 8192, 8224, 16384])
@pytest.mark.parametrize("M", [1, 2047, 2048, 1 << 22, (1 << 24) - 1, 1 << 24, ROWS - 1, ROWS])
def test_norm(K, M):
    # both copies at M x K bytes of column copy that the GPU's 288 GB hold, or the row copy alone
    columns = int(M * K <= 1 << 38)
    _, out = launches.run([f"norm {M} {K} {columns} 1", f"norm {M} {K} 0 0", f"grad {M} {K}"])
    for status, done in out:
        assert status == 0 and done
        assert all(n < 1 << 32 for n in _threads(done)), done
    # every row has its wavefront or its workgroup
    for _, done in out[:2]:
        rows = sum(t.grid[0] * (4 if t.kernel in ("k_norm_rows<1, 1>", "k_norm_rows<1, 4>") else 1)
                   for t in done if "k_norm_rows" in t.kernel)
        assert any("k_norm_dual" in t.kernel for t in done) or M <= rows < M + 4


@pytest.mark.parametrize("call", [
    f"ffn {1 << 20} 32 {1 << 20} 32 256", f"ffn 1 32 {1 << 20} {1 << 17} 1",
    f"ffn 8 32 32 {1 << 20} 256", f"ffn {1 << 20} 32 32 1 1",
    f"swiglu 256 {1 << 21} 8192 32 0 1", f"swiglu 256 {1 << 15} {1 << 20} 32 1 0", f"swiglu 1 {1 << 30} 32 32 0 0"])
def test_feed_forward(call):
    _, [(status, done)] = launches.run([call])
    assert status == 0 and done
    assert all(n < 1 << 32 for n in _threads(done)), done
    assert all(max(t.grid[1:]) <= 65535 for t in done)
