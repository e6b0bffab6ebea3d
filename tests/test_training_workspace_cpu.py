"""Workspaces of the adapters: what a call's kernels hand on, no region that none of them reaches, and none
where rows go each by themselves."""
import ternary_weight_linear_amd as tw

size = tw._lib.bl_adapter_workspace_bytes


def handed_on(M, L, R, backward):
    """Sorted rows, and h or dh as coefficients in each layout (both and by rank too, backward)."""
    rows, RP, RK = 32 * (M // 32 + min(M, L + 1)), -(-R // 16) * 16, -(-R // 32) * 32
    return rows * (4 + 4 * RP + 6 * RK + (4 * RP + 12 * RP if backward else 0))


def test_no_partial_sums_where_nothing_is_split():
    small = 1 << 20                                       # tiles, counters, alignment
    # one share of the sums over rows: no pieces of the gradients, 134 MB each
    assert size(1, 65536, 65536, 1, 256, 1) <= handed_on(1, 1, 256, True) + 16 * 32 * 256 * 4 + small
    # a workgroup has a tile's whole product: no partial sums, 268 MB
    assert size(1 << 20, 64, 64, 1, 64, 0) <= handed_on(1 << 20, 1, 64, False) + small
    assert size(1 << 20, 64, 64, 1, 64, 1) <= handed_on(1 << 20, 1, 64, True) + small + 2 * 32 * 64 * 2 * 64 * 4


def test_partial_sums_where_something_is():
    # two blocks of ranks meet, though the long axis is whole: 128 ranks of each sorted row
    assert size(1 << 20, 64, 64, 1, 128, 0) >= handed_on(1 << 20, 1, 128, False) + (1 << 20) * 128 * 4
    # an adapter's rows in 32 shares: two pieces a share of both gradients
    assert size(4096, 128, 128, 1, 16, 1) >= handed_on(4096, 1, 16, True) + 2 * 32 * 16 * 2 * 128 * 4


def test_many_rows_of_narrow_layers_are_sorted():
    """A forward pass takes a workspace where its rows are sorted: workgroups for every four ranks of every row would
    be most of its time otherwise, however few values they read."""
    for M, K, N, R in ((4000, 64, 64, 64), (4096, 128, 128, 8), (20000, 22, 19, 79), (16384, 512, 512, 8), (60000, 16, 16, 1)):
        assert size(M, K, N, 8, R, 0) > 0, (M, K, N, R)
    for M, K, N, R in ((1, 8192, 8192, 16), (64, 8192, 8192, 64), (320, 4096, 4096, 32), (48, 28672, 8192, 16), (1024, 512, 512, 8)):
        assert size(M, K, N, 8, R, 0) == 0, (M, K, N, R)
