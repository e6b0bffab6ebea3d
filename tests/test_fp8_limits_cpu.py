"""Size queries of the 8-bit floating point operators at the limits of one pass (no GPU)."""
import ternary_weight_linear_amd as tw

ws = tw._lib.bl_fp8_experts_workspace_bytes


def test_experts_run_in_passes_of_less_than_2_gib_of_codes():
    """The workspace is one pass's: 2^31 / H tokens and more run in equal passes."""
    one = ws((1 << 18), 4096, 2, 8, 4096)
    assert ws((1 << 18) + 1, 4096, 2, 8, 4096) > one
    assert ws(1 << 19, 4096, 2, 8, 4096) == one
    assert ws((1 << 19) - 1, 4096, 2, 8, 4096) > one
    assert ws(1 << 20, 4096, 1, 8, 4096) == ws(-(-(1 << 20) // 3), 4096, 1, 8, 4096)


def test_passes_of_wide_experts_keep_the_grids_in_their_limits():
    # matrices of 2 GiB and more are streamed, 2^19 slots at a time
    assert ws(1 << 15, 1 << 15, 32, 1, 1 << 15) == ws(1 << 14, 1 << 15, 32, 1, 1 << 15)
    # 2^35 hidden values at most
    assert ws(1 << 18, 128, 4, 1, 1 << 17) == ws(1 << 16, 128, 4, 1, 1 << 17)


def test_experts_workspace_holds_one_fp32_buffer():
    """Codes of x and of the hidden values, fp32 values before or after the down product (never
    both at a time), and what goes by slot or block."""
    M, H, k, E, I = 4096, 4096, 8, 64, 1024
    slots = M * k
    most = M * H + slots * I + 4 * slots * max(H, I) + M * H // 32 + slots * I // 32 + 64 * slots + (1 << 20)
    assert M * H + slots * I + 4 * slots * max(H, I) <= ws(M, H, k, E, I) <= most
