"""Adapters on values of unlike size: rows and ranks far louder than those beside them, gradients near
the ends of fp32's range, matrices of 16-bit values below the normal ones.

Bounds are those of test_gpu_adapter: roundings of fp32 sums, relative to the sum of the magnitudes that
meet in a result. Where a loud row or rank is multiplied by zeros that sum is the quiet ones' alone, so
h and dh have to go whole into what they are multiplied by."""
import numpy as np
import pytest
import torch

import oracle.adapters as oa
import ternary_weight_linear_amd as tw
from tests.gpu_util import say
from tests.test_gpu_adapter import PAIRS, TYPES, Case, close, gpu, host, u

pytestmark = pytest.mark.gpu


def put(c, name, values):
    """A case's tensor replaced by values, rounded to its type."""
    t = gpu(values.astype(np.float32)).to(getattr(c, name).dtype)
    setattr(c, name, t)
    setattr(c, name + "h", host(t))


@pytest.mark.parametrize("M,K,N,L,R", [(70, 200, 136, 2, 12), (300, 520, 264, 3, 40), (130, 96, 1001, 1, 5), (700, 264, 200, 2, 100)])
@pytest.mark.parametrize("dtype,out,loud", [(d, o, l) for d, o in PAIRS for l in (24, 40, 90) if o == "fp32" or l == 24])
def test_sums_over_rows_beside_louder_rows(M, K, N, L, R, dtype, out, loud):
    """Every seventh row's h and dy are 2^loud times the others'; half of the columns of x and dy are zero in
    those rows, where da and db are the quiet rows' sums."""
    say("adapter loud rows", M, K, N, L, R, dtype, out, loud)
    c = Case(M, K, N, L, R, dtype, out, 1)
    h = c.forward()[1]
    rows = np.arange(M) % 7 == 3
    up, down = 2.0 ** (loud // 2 if out == "fp32" else 13), 2.0 ** -((loud + 1) // 2 if out == "fp32" else 11)
    put(c, "dy", c.dyh * np.where(rows, up, down)[:, None] * np.where(rows[:, None] & (np.arange(N) % 2 == 1), 0, 1))
    put(c, "x", c.xh * np.where(rows[:, None] & (np.arange(K) % 2 == 1), 0, 1))
    h = h * gpu(np.where(rows, up, down).astype(np.float32))[:, None]
    c.out = "fp32"                                                 # dx of the loud rows is beyond fp16
    c.check_backward(c.backward(h, base=None, out_dtype=torch.float32), h, np.zeros_like(c.dbaseh))


@pytest.mark.parametrize("M,K,N,L,R", [(70, 200, 136, 2, 12), (300, 520, 264, 3, 40), (700, 2056, 1104, 2, 64), (130, 96, 1001, 1, 100)])
@pytest.mark.parametrize("dtype,out", [p for p in PAIRS if p[1] == "fp32"])
def test_products_beside_louder_ranks(M, K, N, L, R, dtype, out):
    """Rank 2's values of h and dh are 2^24 times the others', and half of the columns that they are
    multiplied by are zero."""
    say("adapter loud ranks", M, K, N, L, R, dtype, out)
    c = Case(M, K, N, L, R, dtype, out, 2)
    size = np.where(np.arange(R) == 2, 2.0 ** 10, 2.0 ** -8)[:, None]      # with a or b one of them makes 2^18 ...
    odd = (np.arange(R) == 2)[:, None]
    a = c.ah * size * np.where(odd & (np.arange(K) % 2 == 1), 0, 1)
    b = c.bh * np.where(odd, 2.0 ** 6, 1.0) * np.where(odd & (np.arange(N) % 2 == 1), 0, 1)   # ... and the other 2^6
    put(c, "a", a)
    put(c, "b", b)
    y, h = c.forward(base=None)
    c.check_forward(y, h, np.zeros_like(c.baseh))
    c.check_backward(c.backward(h, base=None), h, np.zeros_like(c.dbaseh))
    put(c, "a", c.ah / size)
    put(c, "b", c.bh * size)
    c.check_backward(c.backward(h, base=None), h, np.zeros_like(c.dbaseh))


@pytest.mark.parametrize("M", [2, 90, 70000])
@pytest.mark.parametrize("size", [1e-30, 1e-20, 1e20])
@pytest.mark.parametrize("dtype", list(TYPES))
def test_gradients_of_any_size(M, size, dtype):
    say("adapter sizes", M, size, dtype)
    c = Case(M, 72, 136, 3, 9, dtype, "fp32", 3)
    y, h = c.forward()
    put(c, "dy", c.dyh * size)
    c.check_backward(c.backward(h, base=None), h, np.zeros_like(c.dbaseh))
    put(c, "dy", c.dyh / size)
    h = h * size
    c.check_backward(c.backward(h, base=None), h, np.zeros_like(c.dbaseh))


@pytest.mark.parametrize("M", [2, 90, 70000])
@pytest.mark.parametrize("least", [2.0 ** -22, 2.0 ** -18])
def test_matrices_of_subnormal_halves(M, least):
    """Values of a few and some dozens of fp16's least, 2^-24, in x and dy or in both matrices. The instruction
    that multiplies two fp16 values keeps a product of subnormal ones where those of 2^-14 lie, with
    the digits that fp32 has there, so in the bounds of h and dh they count as 2^-14."""
    say("adapter subnormal", M, least)
    count = lambda v: np.where(v != 0, np.maximum(np.abs(v), 2.0 ** -14), 0)
    for names in (("a", "b"), ("x", "dy")):
        c = Case(M, 72, 136, 3, 9, "fp16", "fp16", 4)
        for n in names:
            put(c, n, np.sign(getattr(c, n + "h")) * np.minimum(np.abs(getattr(c, n + "h")) * least * 4, 2.0 ** -14))
        y, h = c.forward(base=None, out_dtype=torch.float32)
        got = dict(zip(("dx", "da", "db"), c.backward(h, base=None, out_dtype=torch.float32)))
        none = np.zeros_like(c.baseh), np.zeros_like(c.dbaseh)
        ref, href, _, _ = oa.forward(c.xh, c.ah, c.bh, c.indexh, c.scaleh, none[0])
        _, _, mag, hmag = oa.forward(count(c.xh), count(c.ah), count(c.bh), c.indexh, c.scaleh, none[0])
        close(h, href, (c.K / 4 + 64) * u * hmag, "fp32", "h")
        close(y, ref, (c.K / 4 + c.R + 72) * u * mag + u * np.abs(ref), "fp32", "y")
        ref, _ = oa.backward(c.xh, c.ah, c.bh, c.indexh, c.scaleh, host(h), c.dyh, none[1])
        _, mag = oa.backward(count(c.xh), count(c.ah), count(c.bh), c.indexh, c.scaleh, host(h), count(c.dyh), none[1])
        for name, n in (("dx", c.N / 4 + c.R + 72), ("da", c.N / 4 + M / 4 + 136)):
            close(got[name], ref[name], n * u * mag[name] + u * np.abs(ref[name]), "fp32", name)
        # h is given, so no sum of db is one of fp16 products
        _, mag = oa.backward(c.xh, c.ah, c.bh, c.indexh, c.scaleh, host(h), c.dyh, none[1])
        close(got["db"], ref["db"], (M / 4 + 72) * u * mag["db"] + u * np.abs(ref["db"]), "fp32", "db")


@pytest.mark.parametrize("M,K,N,L,R", [(1, 65536, 32768, 1, 256), (66000, 64, 72, 1, 64), (90, 1000, 136, 3, 9), (2048, 520, 264, 64, 33), (70000, 40, 24, 700, 100)])
@pytest.mark.parametrize("dtype,out", PAIRS)
def test_nothing_is_written_outside_the_outputs_and_the_workspace(M, K, N, L, R, dtype, out):
    """Both calls with a workspace of just the size that they ask for, everything that they write between guards."""
    say("adapter guarded", M, K, N, L, R, dtype, out)
    c = Case(M, K, N, L, R, dtype, out, 5)
    code, guard, lib, size = {"fp16": 0, "bf16": 1, "fp32": 2}, 1 << 12, tw._lib, TYPES[out].itemsize
    ws = [lib.bl_adapter_workspace_bytes(M, K, N, L, R, b) for b in (0, 1)]
    sizes = [M * N * size, M * R * 4, ws[0], M * K * size, L * R * K * 4, L * R * N * 4, ws[1]]
    up = lambda n: -(-n // 256) * 256
    room = torch.full((sum(up(n) + guard for n in sizes) + guard,), 0xA5, dtype=torch.uint8, device=c.x.device)
    at, where, kept = [], guard, []
    for n in sizes:
        at.append(room.data_ptr() + where)
        kept.append(room[where - guard:where])
        kept.append(room[where + n:where + up(n)])
        where += up(n) + guard
    kept.append(room[where - guard:])
    stream = tw._stream(c.x.device)
    p = lambda t: t.data_ptr()
    assert lib.bl_adapter_forward(p(c.x), code[dtype], M, K, K, p(c.a), p(c.b), L, R, N, p(c.index), p(c.scale), p(c.base), N, at[0], code[out], N,
                                  at[1], at[2], ws[0], stream) == 0
    assert lib.bl_adapter_backward(p(c.x), code[dtype], M, K, K, p(c.a), p(c.b), L, R, N, p(c.index), p(c.scale), at[1], p(c.dy), code[out], N,
                                   p(c.dbase), K, at[3], code[out], K, at[4], at[5], 0, at[6], ws[1], stream) == 0
    torch.cuda.synchronize()
    assert all(torch.all(k == 0xA5) for k in kept)
    y, h = c.forward()
    for got, n, want in zip(at, sizes, (y, h)):
        start = got - room.data_ptr()
        assert torch.equal(room[start:start + n], want.contiguous().view(torch.uint8).flatten())
    for i, want in zip((3, 4, 5), c.backward(h)):
        start = at[i] - room.data_ptr()
        assert torch.equal(room[start:start + sizes[i]], want.contiguous().view(torch.uint8).flatten())
