"""The shared memory of a dense product whose depth is split over the pairs of
a cluster: the chunks that the other parts send lie from its start on, and
while some warps read them others fill the boxes on their way out.  Checked
for every form (tile width, parts) that any size can reach."""
import pytest

from helpers import build_lib

SMEM = 12 * 16384                    # the pipeline stages' shared memory
CHUNK = 128 * (32 + 4) * 4           # 128 rows of 32 fp32 columns and 4 words of padding
SLOTS = [(76, 36, 24, 16), (76, 38, 25, 19), (76, 37, 24, 18), (66, 30, 20, 14), (76, 0, 0, 0)]


@pytest.fixture(scope="module")
def ops():
    build_lib()
    from grouped_gemm_top_gb300 import ops
    return ops


def forms(ops, product, slots):
    found = {}
    for m in (1, 64, 129, 256, 300, 512, 1024, 2048, 4096):
        for n in list(range(64, 2048, 64)) + list(range(2048, 16384, 512)):
            for k in (256, 512, 1000, 2048, 4096, 8192, 10752, 12288, 16384, 32768):
                p = ops.moe_selftest_dense_plan(product, m, n, k, slots)
                if p.parts > 1:
                    found.setdefault((p.tile_cols, p.parts), (p.swap_bytes, p.box_at, p.box_bytes))
    return found


@pytest.mark.parametrize("slots", SLOTS)
@pytest.mark.parametrize("product", ["FWD", "GATED", "DGRAD", "WGRAD"])
def test_boxes_lie_above_the_chunks(ops, product, slots):
    gated = product == "GATED"
    found = forms(ops, getattr(ops, "MOE_DENSE_" + product), slots)
    if slots[1]:
        assert {parts for _, parts in found} == {2, 3, 4}
    else:
        assert not found
    for (cols, parts), (swap, box_at, box) in found.items():
        units = cols // (64 if gated else 32)            # of one chunk, gated: of a gate and an up chunk
        own = -(-units // parts)
        chunks = (parts - 1) * own * (2 if gated else 1)
        assert swap == chunks * CHUNK
        # a warp's units: every second of the part's own; gate, up and h of 2 KB each, else z and y, or 4 KB of fp32
        need = -(-own // 2) * (3 * 2048 if gated else 4096)
        assert box >= need and box % 1024 == 0, (cols, parts)
        assert swap <= box_at and box_at + 8 * box <= SMEM, (cols, parts, swap, box_at)


def test_gated_256_columns_in_three_parts_is_reached(ops):
    """The form with the most chunks."""
    p = ops.moe_selftest_dense_plan(ops.MOE_DENSE_GATED, 256, 2560, 12288, SLOTS[0])
    assert (p.few_rows, p.tile_cols, p.parts) == (0, 256, 3)
    assert p.swap_bytes == 8 * CHUNK <= p.box_at


def test_refusals(ops):
    for bad in ((5, 256, 256, 256), (-1, 256, 256, 256), (0, 0, 256, 256), (0, 256, 0, 256), (0, 256, 256, 0)):
        with pytest.raises(ops.MoEError) as e:
            ops.moe_selftest_dense_plan(*bad, SLOTS[0])
        assert e.value.status == ops.MOE_ERR_INVALID_ARG, bad
    with pytest.raises(ops.MoEError) as e:
        ops.moe_selftest_dense_plan(0, 1 << 31, 256, 256, SLOTS[0])
    assert e.value.status == ops.MOE_ERR_UNSUPPORTED
    assert ops.lib.moe_selftest_dense_plan(0, 256, 256, 256, None, None) == ops.MOE_ERR_INVALID_ARG
    assert ops.moe_selftest_dense_plan(0, 4, 256, 256, SLOTS[0]).few_rows == 1


@pytest.mark.parametrize("slots", SLOTS[:4])
def test_both_gradients_and_few_rows(ops, slots):
    """One launch of both gradients in every tile width, two launches for long
    work; few rows in 1, 2, 4 and 8 parts."""
    sizes = [(m, n, k) for m in (129, 256, 1000, 4096, 8192) for n in (64, 512, 1024, 2048, 4096, 8192) for k in (64, 512, 2048, 4096)]
    widths = {ops.moe_selftest_dense_plan(ops.MOE_DENSE_BACKWARD, *s, slots).tile_cols for s in sizes}
    assert {0, 64, 128, 256} <= widths <= {0, 64, 128, 192, 224, 256}
    assert ops.moe_selftest_dense_plan(ops.MOE_DENSE_BACKWARD, 32, 512, 512, slots).few_rows == 1
    for product in (ops.MOE_DENSE_FWD, ops.MOE_DENSE_GATED, ops.MOE_DENSE_DGRAD):
        parts = {ops.moe_selftest_dense_plan(product, m, n, k, slots).few_parts for m in (1, 64) for n in (128, 4096, 65536)
                 for k in (64, 512, 1024, 4096)}
        assert parts == {1, 2, 4, 8}
