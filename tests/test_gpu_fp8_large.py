"""Calls of the 8-bit floating point operators that need more than 2^32 work-items or offsets past
32 bits: accepted sizes are computed, from the first row to the last."""
import numpy as np
import pytest
import torch

import oracle.fp8 as of
import ternary_weight_linear_amd as tw
from tests.gpu_util import DEV, host, say

pytestmark = pytest.mark.gpu


def needs(gib):
    torch.cuda.empty_cache()
    free = torch.cuda.mem_get_info()[0]
    if free < gib * 2 ** 30:
        pytest.skip(f"needs {gib} GiB of free GPU memory, has {free / 2 ** 30:.0f}")


@pytest.fixture(autouse=True)
def give_back():
    yield
    torch.cuda.empty_cache()


def test_quant_act_of_more_than_2_28_blocks():
    M, K = 1 << 20, 33008                          # 258 blocks a row
    needs(110)
    say("quant_act large", M, K)
    x = torch.zeros((M, K), dtype=torch.float16, device=DEV)
    rows = [0, 1, (1 << 19) + 3, M - 2, M - 1]
    v = np.random.default_rng(0).standard_normal((len(rows), K)).astype(np.float16)
    x[rows] = torch.from_numpy(v).to(DEV)
    q, s = tw.bl_quant_act_fp8(x)
    c, sr, _ = of.quant_act(v.astype(np.float32))
    assert np.array_equal(host(q[rows].view(torch.uint8)), c) and np.array_equal(host(s[:, rows]), sr)
    zero, floor = [2, (1 << 19) + 4, M - 3], of.quant_act(np.zeros((1, K), np.float32))[1]
    assert not host(q[zero].view(torch.uint8)).any() and np.array_equal(host(s[:, zero]), np.repeat(floor, 3, 1))


@pytest.mark.parametrize("M,E,k", [((1 << 26) + 5, 18, 17), ((1 << 28) + 5, 2, 1)])
def test_route_of_many_rows(M, E, k):
    """Rows repeat every 1000: each repetition gives what the first does."""
    needs(24)
    say("route large", M, E, k)
    some = torch.from_numpy(np.random.default_rng(1).standard_normal((1000, E)).astype(np.float16)).to(DEV)
    times = -(-M // 1000)
    logits = some.repeat(times, 1)[:M]
    w, i = tw.bl_route_experts(logits, k)
    w0, i0 = tw.bl_route_experts(some, k)
    for got, want in ((w, w0), (i, i0)):
        whole = got[: (times - 1) * 1000].view(times - 1, 1000, k)
        assert bool((whole == want).all()) and torch.equal(got[(times - 1) * 1000:], want[: M - (times - 1) * 1000])


def test_experts_of_activations_past_2_gib():
    """2^19 tokens of 4096: any 4096 of them by themselves give the same bits."""
    M, E, k, H, I = 1 << 19, 8, 2, 4096, 4096
    needs(70)
    say("experts large", M, E, k, H, I)
    g = torch.Generator(device=DEV).manual_seed(2)

    def matrices(count, rows, cols):
        both = [tw.bl_fp8_quant_weight(torch.randn(rows, cols, generator=g, device=DEV) * cols ** -0.5) for _ in range(count)]
        return torch.stack([c.view(torch.uint8) for c, _ in both]).view(torch.float8_e4m3fn), torch.stack([s for _, s in both])

    wgu, sgu = (t.view(E, 2, *t.shape[1:]) for t in matrices(2 * E, I, H))
    wd, sd = matrices(E, H, I)
    x = torch.randn(M, H, generator=g, device=DEV, dtype=torch.bfloat16)
    first = torch.randint(0, E, (M,), generator=g, device=DEV)
    index = torch.stack([first, (first + torch.randint(1, E, (M,), generator=g, device=DEV)) % E], 1).to(torch.int32)
    weight = torch.rand(M, k, generator=g, device=DEV)
    y = tw.bl_fp8_experts(x, index, weight, wgu, sgu, wd, sd)
    for at in (0, M // 2 - 2048, M - 4096):
        s = slice(at, at + 4096)
        assert torch.equal(y[s], tw.bl_fp8_experts(x[s], index[s].contiguous(), weight[s].contiguous(), wgu, sgu, wd, sd))
