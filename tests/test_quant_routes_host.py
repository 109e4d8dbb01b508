"""The shapes of the GPU tests reach every kernel of the 8-bit products and of
the expert layer (the library's own choice, asked on the host)."""
import pytest

import block_wise_int4_matmulnbits_amd as mnb
from tests import quant_routes
from tests import test_gpu_int8 as I8
from tests import test_gpu_moe as MOE
from tests import test_gpu_moe_range as RANGE
from tests import test_gpu_quant_routes as GPU


@pytest.fixture(scope="module")
def routes(tmp_path_factory):
    return quant_routes.Routes(tmp_path_factory.mktemp("routes"))


def test_tiles_reach_their_steady_state(routes):
    """Each tile by name, with more stages than twice its ring holds, with and
    without a ragged last one."""
    chosen = routes.int8([(mnb.MNB_I8, m, K, N) for _, m, K, N in GPU.TILES])
    ragged = {t: set() for t in quant_routes.TILES}
    for (tile, m, K, N), (got, _, _, fused) in zip(GPU.TILES, chosen):
        assert got == tile and not fused, (m, K, N, got)
        stage, ring = quant_routes.TILES[tile]
        assert -(-K // stage) > 2 * ring, (tile, K)
        ragged[tile].add(K % stage != 0)
    assert all(r == {False, True} for r in ragged.values()), ragged


def test_few_rows_variants(routes):
    shapes = I8.SHAPES + GPU.ROWS
    for dtype, fused in ((mnb.MNB_I8, False), (mnb.MNB_F16, True), (mnb.MNB_BF16, True)):
        found = routes.int8([(dtype,) + s for s in shapes])
        rows = [(s, r) for s, r in zip(shapes, found) if r[0] is None and r[3] == fused]
        assert {r[2] for _, r in rows} == set(range(1, 9)), sorted({r[2] for _, r in rows})
        # Eight waves where sixteen would fit K: two and four units each.
        assert {2, 4} <= {r[2] for (_, K, _), r in rows if r[1] == 8 and K >= 2048}
        if fused:
            # More rows than waves; several waves a row; rows read again.
            assert any(m >= r[1] > 1 for (m, _, _), r in rows)
            assert any(r[1] // m > 1 and m > 1 for (m, _, _), r in rows)
            assert any(K // 8 > 8 * 64 * (r[1] // m) for (m, K, _), r in rows if m < r[1])
    assert all(r[0] is None for r in routes.int8([(mnb.MNB_F16,) + s for s in GPU.ROWS]))


def test_expert_layer_variants(routes):
    every = {"wide %s %d vec %d" % (launch, rows, vec) for launch in ("up", "down") for rows in (16, 32) for vec in (1, 4, 8)}
    for rows in (4, 8):
        every |= {"up %d vec %d %s %s" % (rows, vec, t, stage) for vec in (1, 4) for t in ("f16", "bf16")
                  for stage in ("tokens", "batch", "spans")}
        every |= {"down %d quads %d vec %d" % (rows, quads, vec) for quads in (1, 2, 4) for vec in {1, quads}}
    found = set().union(*routes.moe(MOE.CASES + RANGE.KERNELS + GPU.EXPERTS))
    assert found == every, (sorted(every - found), sorted(found - every))
