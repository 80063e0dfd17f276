"""Every kernel of the norm and feed-forward calls is launched by a GPU test that compares it
with the oracle: the tests' own shapes, through the library's launch rules.  CPU only."""

from collections import Counter

from tests import launches
from tests import test_gpu_ffn_decode as decode
from tests import test_gpu_ffn_decode_tiles as tiles
from tests import test_gpu_norm as norm
from tests import test_gpu_norm_rows as norm_rows
from tests import test_gpu_swiglu_backward as backward


def _param(test, first):
    """The values that a parametrised test takes under the names that begin with `first`."""
    return next(m.args[1] for m in test.pytestmark if m.name == "parametrize" and m.args[0].startswith(first))


def test_every_kernel_is_reached():
    calls = [f"ffn {M} {K} {F} {N} 1" for M, K, F, N in decode.DENSE + tiles.TILES]
    calls += [f"ffn {sum(c)} {K} {F} {N} {len(c)}"
              for c, K, F, N in _param(decode.test_experts, "counts") + tiles.EXPERTS]
    calls += [f"norm {M} {K} 1 1" for M, K in norm.ROWS]
    calls += [f"norm {M} {K} 0 1" for M, K in norm_rows.ROWS]
    calls += [f"grad {M} {K}" for M, K in _param(norm.test_gradient, "M,K")]
    calls += [f"swiglu {len(c)} {sum(c)} {F} {K} {accum} {windows}" for c, F, K in backward.CASES
              for accum in (0, 1) for windows in (0, 1)]
    kernels, out = launches.run(calls)
    assert all(status == 0 for status, _ in out)
    reached = Counter(t.kernel for _, done in out for t in done)
    ours = {k for k in kernels if k.startswith(("k_ffn_", "k_norm_", "k_gemm_swiglu_grad"))}
    assert len(ours) >= 25
    assert not ours - set(reached), sorted(ours - set(reached))


def test_tiles_with_experts_and_long_contractions():
    """Two and four token tiles, 4 and 16 wavefronts, dense and with offsets."""
    dense = [f"ffn {M} {K} {F} {N} 1" for M, K, F, N in tiles.TILES]
    experts = [f"ffn {sum(c)} {K} {F} {N} {len(c)}" for c, K, F, N in tiles.EXPERTS]
    for calls in (dense, experts):
        _, out = launches.run(calls)
        reached = {t.kernel for _, done in out for t in done}
        assert reached >= {f"k_ffn_down<{t}, 1, {nw}>" for t in (2, 4) for nw in (4, 16)}, sorted(reached)
        assert reached >= {"k_ffn_gate<2, 8, 2>", "k_ffn_gate<4, 8, 1>"}, sorted(reached)
