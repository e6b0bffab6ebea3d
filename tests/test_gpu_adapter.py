"""GPU parity of the low-rank adapters, forward and backward, against the oracle in 64 bits.

Bounds. u = 2^-24 is half a unit of fp32. Products of two values of 16 bits are exact, others are
rounded once. A sum over D values runs in at most four chains of D / 4 additions (of which the matrix cores
round each at most once), whose results are added with those of other parts: D / 4 + 64 roundings of partial
sums that are at most the sum of magnitudes. A second sum over R or M values takes the first one's
error on and adds its own."""
import numpy as np
import pytest
import torch

import oracle.adapters as oa
import ternary_weight_linear_amd as tw
from tests.gpu_util import DEV, say

pytestmark = pytest.mark.gpu

TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
UNIT = {"fp16": 2.0 ** -11, "bf16": 2.0 ** -8, "fp32": 2.0 ** -24}     # half a step, relative
LEAST = {"fp16": 2.0 ** -25, "bf16": 2.0 ** -134, "fp32": 2.0 ** -149}
u = 2.0 ** -24
SHAPES = [(1, 1, 1, 1, 1), (1, 64, 128, 3, 16), (2, 8, 8, 1, 5), (5, 100, 36, 2, 3), (16, 4096, 1032, 6, 16), (31, 256, 130, 4, 8),
          (33, 129, 257, 3, 17), (64, 512, 384, 1, 33), (100, 72, 1000, 7, 48), (257, 640, 264, 5, 64), (300, 1001, 777, 3, 5),
          (500, 64, 96, 9, 65), (130, 200, 136, 2, 100), (70, 96, 80, 2, 256), (513, 2056, 512, 40, 12), (1100, 320, 1000, 2, 32)]
# Enough values of adapters that the rows are sorted, tiles of few and many rows among them.
SORTED = [(65600, 17, 9, 3, 2), (65536, 40, 130, 700, 5), (2100, 1001, 777, 5, 33), (900, 3000, 1544, 300, 40), (700, 2056, 1100, 2, 64),
          (450, 1032, 400, 2, 256), (3000, 520, 520, 9, 48), (4100, 640, 1000, 3, 16), (2500, 4104, 1031, 1, 10)]
PAIRS = [("fp16", "fp16"), ("fp16", "fp32"), ("bf16", "bf16"), ("bf16", "fp32"), ("fp32", "fp32")]


def values(shape, dtype, seed, size=1.0):
    """Values of the type on the GPU, and the same in 64 bits on the host."""
    t = torch.from_numpy((np.random.default_rng(seed).standard_normal(shape) * size).astype(np.float32)).to(TYPES[dtype])
    return t.to(DEV), t.double().numpy()


def gpu(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def host(t):
    return t.double().cpu().numpy()


def rows_of(M, L, seed, kind="mixed"):
    g = np.random.default_rng(seed)
    if kind == "runs":
        e = np.sort(g.integers(0, L, M))
    else:                                          # some rows without an adapter, by any number that names none
        e = g.integers(0, L, M)
        e = np.where(g.random(M) < 0.2, g.choice([-1, L, -2 ** 31, 2 ** 31 - 1, L + 7], M), e)
    return e.astype(np.int32)


def close(got, ref, bound, dtype, what):
    got = host(got)
    tol = bound + UNIT[dtype] * (np.abs(ref) + bound) + LEAST[dtype]
    bad = ~(np.abs(got - ref) <= tol)
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        raise AssertionError(f"{what}: {bad.sum()} of {bad.size} out of tolerance, first at {i}: {got[i]!r} for {ref[i]!r}, "
                             f"allowed {tol[i]:.3g}")


class Case:
    def __init__(self, M, K, N, L, R, dtype, out, seed, kind="mixed"):
        self.M, self.K, self.N, self.L, self.R, self.dtype, self.out = M, K, N, L, R, dtype, out
        self.x, self.xh = values((M, K), dtype, seed)
        self.a, self.ah = values((L, R, K), dtype, seed + 1, K ** -0.5)
        self.b, self.bh = values((L, R, N), dtype, seed + 2, R ** -0.5)
        self.base, self.baseh = values((M, N), out, seed + 3)
        self.dy, self.dyh = values((M, N), out, seed + 4)
        self.dbase, self.dbaseh = values((M, K), out, seed + 5)
        self.scaleh = np.random.default_rng(seed + 6).choice([0.25, 1.0, 2.0, -3.0], L).astype(np.float32)
        self.indexh = rows_of(M, L, seed + 7, kind)
        self.scale, self.index = gpu(self.scaleh), gpu(self.indexh)

    def forward(self, **kw):
        return tw.bl_adapter_forward(self.x, self.a, self.b, self.index, **({"scale": self.scale, "base": self.base} | kw))

    def backward(self, h, **kw):
        return tw.bl_adapter_backward(self.x, self.a, self.b, self.index, h, self.dy, **({"scale": self.scale, "base": self.dbase} | kw))

    def check_forward(self, y, h, baseh=None, scaleh=None):
        baseh = self.baseh if baseh is None else baseh
        ref, href, mag, hmag = oa.forward(self.xh, self.ah, self.bh, self.indexh, self.scaleh if scaleh is None else scaleh, baseh)
        close(h, href, (self.K / 4 + 64) * u * hmag, "fp32", "h")
        close(y, ref, (self.K / 4 + self.R + 72) * u * mag + u * np.abs(ref), self.out, "y")
        bare = (self.indexh < 0) | (self.indexh >= self.L)
        assert np.array_equal(host(y)[bare], baseh[bare]) and not host(h)[bare].any()

    def check_backward(self, got, h, dbaseh=None, add=(0, 0)):
        dx, da, db = got
        dbaseh = self.dbaseh if dbaseh is None else dbaseh
        ref, mag = oa.backward(self.xh, self.ah, self.bh, self.indexh, self.scaleh, host(h), self.dyh, dbaseh)
        if dx is not None:
            close(dx, ref["dx"], (self.N / 4 + self.R + 72) * u * mag["dx"] + u * np.abs(ref["dx"]), self.out, "dx")
            bare = (self.indexh < 0) | (self.indexh >= self.L)
            assert np.array_equal(host(dx)[bare], dbaseh[bare])
        for t, name, n, more in ((da, "da", self.N / 4 + self.M / 4 + 136, add[0]), (db, "db", self.M / 4 + 72, add[1])):
            assert t.dtype == torch.float32
            close(t, ref[name] + more, n * u * mag[name] + u * np.abs(ref[name]), "fp32", name)
        without = np.setdiff1d(np.arange(self.L), self.indexh)
        if not np.any(add[0]):
            assert not host(da)[without].any() and not host(db)[without].any()


@pytest.mark.parametrize("dtype,out", PAIRS)
@pytest.mark.parametrize("M,K,N,L,R", SHAPES + SORTED)
def test_forward_and_backward(M, K, N, L, R, dtype, out):
    say("adapter", M, K, N, L, R, dtype, out)
    c = Case(M, K, N, L, R, dtype, out, M + 3 * K + 5 * N)
    y, h = c.forward()
    assert y.dtype == TYPES[out] and tuple(y.shape) == (M, N) and tuple(h.shape) == (M, R)
    c.check_forward(y, h)
    c.check_backward(c.backward(h), h)


@pytest.mark.parametrize("dtype,out", PAIRS)
def test_without_base_scale_or_dx(dtype, out):
    say("adapter bare", dtype, out)
    c = Case(45, 136, 72, 4, 12, dtype, out, 1)
    y, h = c.forward(scale=None, base=None, out_dtype=TYPES[out])
    c.check_forward(y, h, np.zeros_like(c.baseh), np.ones(4))
    c.check_backward(c.backward(h, base=None, out_dtype=TYPES[out]), h, np.zeros_like(c.dbaseh))
    dx, da, db = c.backward(h, base=None, need_dx=False)
    assert dx is None
    c.check_backward((dx, da, db), h)


@pytest.mark.parametrize("dtype,out", PAIRS)
@pytest.mark.parametrize("M", [3, 90, 66000])
def test_in_place_equals_apart(dtype, out, M):
    say("adapter in place", dtype, out, M)
    c = Case(M, 264, 200, 3, 20, dtype, out, 2)
    y, h = c.forward()
    room = c.base.clone()
    y2, h2 = c.forward(base=room, out=room)
    assert y2 is room and torch.equal(y, room) and torch.equal(h, h2)
    dx, da, db = c.backward(h)
    room = c.dbase.clone()
    dx2, da2, db2 = c.backward(h, base=room, out=room)
    assert torch.equal(dx, room) and torch.equal(da, da2) and torch.equal(db, db2)


@pytest.mark.parametrize("M", [4, 77, 66000])
@pytest.mark.parametrize("shift", [8, 3])
@pytest.mark.parametrize("dtype,out", PAIRS)
def test_strided_and_unaligned_rows(dtype, out, shift, M):
    """Columns of wider tensors, at 16-byte addresses and at others; what lies around stays."""
    say("adapter strided", dtype, out, shift, M)
    c = Case(M, 96, 160, 3, 9, dtype, out, 3)
    y, h = c.forward()
    dx, da, db = c.backward(h)

    def inside(t):
        room = torch.full((t.shape[0], t.shape[1] + 4 * shift), 7.0, dtype=t.dtype, device=DEV)
        room[:, shift:shift + t.shape[1]] = t
        return room, room[:, shift:shift + t.shape[1]]

    (_, c.x), (_, c.base), (_, c.dy), (_, c.dbase) = inside(c.x), inside(c.base), inside(c.dy), inside(c.dbase)
    yroom, yv = inside(torch.zeros_like(y))
    xroom, dxv = inside(torch.zeros_like(dx))
    y2, h2 = c.forward(out=yv)
    got = c.backward(h2, out=dxv)
    c.check_forward(y2, h2)
    c.check_backward(got, h2)
    for room, n in ((yroom, 160), (xroom, 96)):
        assert torch.all(room[:, :shift] == 7) and torch.all(room[:, shift + n:] == 7)


def test_gradients_are_added_onto():
    say("adapter add")
    c = Case(150, 208, 88, 5, 10, "bf16", "bf16", 4)
    c.indexh[:] = np.where(c.indexh == 2, 3, c.indexh)           # adapter 2 has no rows
    c.index = gpu(c.indexh)
    h = c.forward()[1]
    da, dah = values((5, 10, 208), "fp32", 50)
    db, dbh = values((5, 10, 88), "fp32", 51)
    got = c.backward(h, da=da, db=db)
    assert got[1] is da and got[2] is db
    c.check_backward(got, h, add=(dah, dbh))
    assert np.array_equal(host(da)[2], dah[2]) and np.array_equal(host(db)[2], dbh[2])


@pytest.mark.parametrize("M", [1, 40, 200, 70000])
def test_no_row_has_an_adapter(M):
    say("adapter none", M)
    c = Case(M, 64, 72, 2, 8, "bf16", "bf16", 5)
    c.indexh[:] = -1
    c.index = gpu(c.indexh)
    y, h = c.forward()
    c.check_forward(y, h)
    dx, da, db = c.backward(h)
    assert torch.equal(y, c.base) and torch.equal(dx, c.dbase) and not h.any() and not da.any() and not db.any()


@pytest.mark.parametrize("M,L,rows", [(70, 64, 70), (300, 1024, 300), (2048, 1, 40), (2048, 3, 70), (20000, 5, 97), (66000, 2, 200), (513, 700, 33)])
@pytest.mark.parametrize("K,N,R", [(96, 264, 9), (1032, 130, 33)])
@pytest.mark.parametrize("dtype", list(TYPES))
def test_few_tiles_of_many_possible_ones(M, L, rows, K, N, R, dtype):
    """One adapter of many for all rows, or few rows of many with one: far fewer tiles than a call of its
    sizes may have, and less than it has shares for them."""
    say("adapter few tiles", M, L, rows, K, N, R, dtype)
    c = Case(M, K, N, L, R, dtype, dtype, 11)
    c.indexh[:] = -1
    c.indexh[np.sort(np.random.default_rng(12).permutation(M)[:rows])] = L // 2
    c.index = gpu(c.indexh)
    y, h = c.forward()
    c.check_forward(y, h)
    nan = lambda *shape: torch.full(shape, float("nan"), device=DEV)      # what fresh memory may hold
    room = [nan(L, R, K), nan(L, R, N)]
    del room
    c.check_backward(c.backward(h), h)
    da, dah = values((L, R, K), "fp32", 13)
    db, dbh = values((L, R, N), "fp32", 14)
    c.check_backward(c.backward(h, da=da, db=db), h, add=(dah, dbh))


@pytest.mark.parametrize("M", [2, 70, 400, 66000])
@pytest.mark.parametrize("dtype", list(TYPES))
def test_nan_and_infinity_stay_in_their_rows_and_adapters(M, dtype):
    say("adapter nan", M, dtype)
    c = Case(M, 200, 136, 4, 12, dtype, dtype, 6)
    c.indexh[:] = np.arange(M) % 3                                # adapter 3 has no rows
    c.index = gpu(c.indexh)
    clean, h0 = c.forward()
    g0 = c.backward(h0)
    c.x[0, 17] = float("nan")
    c.a[3], c.b[3] = float("nan"), float("inf")                   # reached by nothing
    c.a[1, 11, 199] = float("inf")
    y, h = c.forward()
    bad = (c.indexh == 1) | (np.arange(M) == 0)
    assert torch.isnan(y[0]).all() and not torch.isfinite(h[gpu(c.indexh == 1)][:, 11]).any()
    assert torch.equal(y[gpu(~bad)], clean[gpu(~bad)]) and torch.equal(h[gpu(~bad)], h0[gpu(~bad)])
    dx, da, db = c.backward(h0)
    ok = gpu(c.indexh != 1)
    assert torch.equal(dx[ok], g0[0][ok])                         # a[1] alone reaches dx
    assert torch.isnan(da[0, :, 17]).all() and not da[3].any() and not db[3].any()
    assert torch.equal(da[1:3], g0[1][1:3]) and torch.equal(db, g0[2])
    keep = torch.arange(200, device=DEV) != 17
    assert torch.equal(da[0][:, keep], g0[1][0][:, keep])


@pytest.mark.parametrize("M", [3, 70, 66000])
@pytest.mark.parametrize("dtype", list(TYPES))
def test_infinities_give_nothing_finite(M, dtype):
    """Coefficients that 16 bits hold whole, whose further parts are zeros, times infinities."""
    say("adapter infinity", M, dtype)
    K, N, L, R = 40, 136, 2, 5
    t = lambda v: v.to(DEV).to(TYPES[dtype])
    x, a, b, dy = torch.zeros(M, K), torch.ones(L, R, K), torch.ones(L, R, N), torch.zeros(M, N)
    x[:, 0], dy[:, 0] = 1.0, 1.0
    b[0, 2, 77] = float("inf")
    index = torch.arange(M, dtype=torch.int32, device=DEV) % 2
    y, h = tw.bl_adapter_forward(t(x), t(a), t(b), index)
    mine = index == 0
    assert torch.all(h == 1) and not torch.isfinite(y[mine][:, 77]).any()
    y[mine.nonzero()[:, 0], 77] = 5.0
    assert torch.all(y == 5)
    x[2, 7], dy[1, 9] = float("inf"), float("inf")
    dx, da, db = tw.bl_adapter_backward(t(x), t(a), t(torch.ones(L, R, N)), index, h, t(dy))
    assert not torch.isfinite(da[0, :, 7]).any() and not torch.isfinite(db[1, :, 9]).any() and not torch.isfinite(dx[1]).any()
    assert torch.isfinite(da[0, :, 8:]).all() and torch.isfinite(db[0]).all() and torch.isfinite(db[1, :, 10:]).all()
    assert torch.all(dx[0] == R) and torch.all(dx[2:] == R)


@pytest.mark.parametrize("M,L", [(8192, 3), (8193, 5), (20000, 1024), (16384, 1), (1000, 1024), (9000, 700)])
@pytest.mark.parametrize("kind", ["mixed", "runs"])
def test_many_rows_and_adapters(M, L, kind):
    say("adapter many", M, L, kind)
    c = Case(M, 32, 40, L, 4, "bf16", "bf16", 7, kind)
    y, h = c.forward()
    c.check_forward(y, h)
    c.check_backward(c.backward(h), h)


@pytest.mark.parametrize("M,K,N,L,R", [(3, 1024, 300, 2, 16), (48, 512, 264, 5, 16), (200, 640, 512, 1, 40), (700, 256, 136, 3, 8), (66000, 48, 40, 40, 8)])
@pytest.mark.parametrize("dtype", list(TYPES))
def test_exact_on_small_integers(M, K, N, L, R, dtype):
    """Sums of small whole numbers stay below 2^24 and come back exactly, whatever the order."""
    say("adapter exact", M, K, N, L, R, dtype)
    g = np.random.default_rng(8)
    x, a, b = g.integers(-2, 3, (M, K)), g.integers(-1, 2, (L, R, K)), g.integers(-1, 2, (L, R, N))
    index = g.integers(-1, L, M).astype(np.int32)
    t = lambda v: gpu(v.astype(np.float32)).to(TYPES[dtype])
    base = g.integers(-9, 10, (M, N))
    scale = np.full(L, 2.0, np.float32)
    y, h = tw.bl_adapter_forward(t(x), t(a), t(b), gpu(index), scale=gpu(scale), base=gpu(base.astype(np.float32)))
    ref, href, _, _ = oa.forward(x, a, b, index, scale, base)
    assert np.abs(ref).max() < 2 ** 24 and np.array_equal(host(y), ref) and np.array_equal(host(h), href)
    # the gradients: h in place of a small matrix, so that sums over rows stay small too
    hs, dy = g.integers(-2, 3, (M, R)), g.integers(-1, 2, (M, N))
    dx, da, db = tw.bl_adapter_backward(t(x), t(a), t(b), gpu(index), gpu(hs.astype(np.float32)), t(dy), scale=gpu(scale),
                                        base=gpu(np.zeros((M, K), np.float32)))
    ref, mag = oa.backward(x, a, b, index, scale, hs, dy, np.zeros((M, K)))
    assert max(m.max() for m in mag.values()) < 2 ** 24
    for got, name in ((dx, "dx"), (da, "da"), (db, "db")):
        assert np.array_equal(host(got), ref[name]), name


@pytest.mark.parametrize("dtype,out", PAIRS)
@pytest.mark.parametrize("M", [9, 600, 1300])
def test_results_keep_the_precision_of_their_type(dtype, out, M):
    """Far below the worst case: errors of n roundings add up as their square root, so fp32 sums stay
    within 2^-19 of the root of their summed squares, and 16-bit results within 1.01 of their rounding."""
    say("adapter precision", dtype, out, M)
    c = Case(M, 2064, 1536, 2, 32, dtype, out, 9, "runs")
    y, h = c.forward()
    hsize = np.sqrt(np.stack([np.square(c.xh[m]) @ np.square(c.ah[e]).T for m, e in enumerate(c.indexh)]))
    ref, href, _, _ = oa.forward(c.xh, c.ah, c.bh, c.indexh, c.scaleh, c.baseh)
    assert np.all(np.abs(host(h) - href) <= 2.0 ** -19 * hsize)
    size = np.stack([abs(c.scaleh[e]) * np.sqrt(np.square(hsize[m]) @ np.square(c.bh[e])) for m, e in enumerate(c.indexh)])
    assert np.all(np.abs(host(y) - ref) <= 1.01 * UNIT[out] * np.abs(ref) + 2.0 ** -19 * size)
    dx, da, db = c.backward(h)
    ref, _ = oa.backward(c.xh, c.ah, c.bh, c.indexh, c.scaleh, host(h), c.dyh, c.dbaseh)
    assert np.all(np.abs(host(dx) - ref["dx"]) <= 1.01 * UNIT[out] * np.abs(ref["dx"]) + 2.0 ** -19 * np.sqrt(1536) * 3)
    for got, name in ((da, "da"), (db, "db")):
        rms = np.sqrt(np.mean(np.square(ref[name])))
        assert np.sqrt(np.mean(np.square(host(got) - ref[name]))) <= 2.0 ** -21 * rms, name


@pytest.mark.parametrize("M,L", [(5, 3), (300, 3), (9000, 2)])
def test_same_bits_on_every_run_and_stream(M, L):
    say("adapter repeat", M, L)
    c = Case(M, 520, 264, L, 16, "bf16", "bf16", 10)
    y, h = c.forward()
    first = (y, h, *c.backward(h))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for i in range(4):
        with torch.cuda.stream(streams[i % 2]):
            y, h = c.forward()
            got.append((y, h, *c.backward(h)))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for g in got for a, b in zip(first, g))


@pytest.mark.parametrize("M", [1, 16, 300, 66000])
def test_replayed_from_a_graph(M):
    """Two graphs and eager calls in turn, with new inputs and new adapters' rows between replays."""
    say("adapter graph", M)
    cases = [Case(M, 264, 320, 4, 16, "bf16", "bf16", 11 + i) for i in range(2)]

    def step(c):
        y, h = c.forward()
        return (y, h, *c.backward(h))

    graphs, outs = [], []
    for c in cases:
        step(c)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(step(c))
        graphs.append(graph)
    for turn in range(4):
        for i, c in enumerate(cases):
            c.x.copy_(values((M, 264), "bf16", 100 + 7 * turn + i)[0])
            c.index.copy_(gpu(rows_of(M, 4, 200 + 5 * turn + i)))
            graphs[i].replay()
        torch.cuda.synchronize()
        for i, c in enumerate(cases):
            assert all(torch.equal(a, b) for a, b in zip(outs[i], step(c)))
        torch.cuda.synchronize()


def test_offsets_past_32_bits():
    """Rows 2^16 elements apart: the last ones lie past 2^32 elements from the first."""
    say("adapter large offsets")
    M, K, N, L, R = 70000, 40, 24, 2, 8
    wide = torch.zeros((M, 1 << 16), dtype=torch.bfloat16, device=DEV)
    c = Case(M, K, N, L, R, "bf16", "bf16", 12, "runs")
    y, h = c.forward()
    got = c.backward(h)
    # x, base and y, and then dy and dx, as columns of one tensor; base and y are the same columns
    wide[:, :K], wide[:, 1024:1024 + N] = c.x, c.base
    apart = torch.zeros((M, N), dtype=torch.bfloat16, device=DEV)
    y2, h2 = tw.bl_adapter_forward(wide[:, :K], c.a, c.b, c.index, scale=c.scale, base=wide[:, 1024:1024 + N], out=apart)
    assert torch.equal(y2, y) and torch.equal(h2, h)
    wide[:, 2048:2048 + N] = c.dy
    got2 = tw.bl_adapter_backward(c.x, c.a, c.b, c.index, h, wide[:, 2048:2048 + N], scale=c.scale, base=c.dbase)
    assert all(torch.equal(a, b) for a, b in zip(got, got2))
    got2 = tw.bl_adapter_backward(wide[:, :K], c.a, c.b, c.index, h, c.dy, scale=c.scale, base=c.dbase)
    assert all(torch.equal(a, b) for a, b in zip(got, got2))
    wide[:, 4096:4096 + N] = c.base
    y2, h2 = tw.bl_adapter_forward(c.x, c.a, c.b, c.index, scale=c.scale, base=wide[:, 4096:4096 + N], out=wide[:, 4096:4096 + N])
    assert torch.equal(y2, y)


def test_most_rows():
    """2^20 rows, 128 chunks of the sort, against 64 bits on the GPU."""
    say("adapter most rows")
    M, K, N, L, R = 1 << 20, 16, 12, 7, 2
    gen = torch.Generator(device=DEV).manual_seed(0)
    x = torch.randn(M, K, generator=gen, device=DEV).bfloat16()
    a, b = (torch.randn(L, R, n, generator=gen, device=DEV).bfloat16() for n in (K, N))
    index = torch.randint(-1, L, (M,), generator=gen, device=DEV, dtype=torch.int32)
    dy = torch.randn(M, N, generator=gen, device=DEV).bfloat16()
    y, h = tw.bl_adapter_forward(x, a, b, index)
    dx, da, db = tw.bl_adapter_backward(x, a, b, index, h, dy)
    at, held = index.long().clamp_min(0), (index >= 0).double()[:, None]
    xd, dyd = x.double(), dy.double()
    hd = (a.double()[at] * xd[:, None]).sum(2) * held
    assert torch.all((h - hd).abs() <= 20 * u * (a.double().abs()[at] * xd.abs()[:, None]).sum(2) * held)
    yd = (b.double()[at] * h.double()[:, :, None]).sum(1)
    assert torch.all((y - yd).abs() <= 20 * u * (b.double().abs()[at] * h.double().abs()[:, :, None]).sum(1) + u * yd.abs())
    dh = (b.double()[at] * dyd[:, None]).sum(2) * held
    mag = (b.double().abs()[at] * dyd.abs()[:, None]).sum(2) * held
    dxd = (a.double()[at] * dh[:, :, None]).sum(1)
    assert torch.all((dx - dxd).abs() <= 40 * u * (a.double().abs()[at] * mag[:, :, None]).sum(1) + u * dxd.abs())
    for e in range(L):
        rows = (index == e).nonzero()[:, 0]
        # the roundings of M / L additions add up as their square root: 400, and three times that
        for got, c, cm, s in ((da[e], dh[rows], mag[rows], xd[rows]), (db[e], h[rows].double(), h[rows].double().abs(), dyd[rows])):
            ref, size = c.t() @ s, (cm.t() @ s.abs())
            assert torch.all((got - ref).abs() <= 1200 * u * size)


def test_adapters_past_32_bits():
    """Matrices of 2^32 values: the last adapter's lie far past 2^31 from the first's."""
    say("adapter large matrices")
    M, K, N, L, R = 70, 16384, 40, 1024, 256
    a = torch.zeros((L, R, K), dtype=torch.bfloat16, device=DEV)
    b = torch.zeros((L, R, N), dtype=torch.bfloat16, device=DEV)
    gen = torch.Generator(device=DEV).manual_seed(1)
    for e in (0, 1023):
        a[e] = torch.randn(R, K, generator=gen, device=DEV).bfloat16() * K ** -0.5
        b[e] = torch.randn(R, N, generator=gen, device=DEV).bfloat16()
    x, dy = torch.randn(M, K, generator=gen, device=DEV).bfloat16(), torch.randn(M, N, generator=gen, device=DEV).bfloat16()
    index = torch.where(torch.arange(M, device=DEV) % 3 == 0, 0, 1023).int()
    few = torch.where(index == 0, 0, 1).int()
    pair = [t[[0, 1023]].contiguous() for t in (a, b)]
    for rows in (M, 5):                             # sorted, and each row by itself
        y, h = tw.bl_adapter_forward(x[:rows], a, b, index[:rows])
        y2, h2 = tw.bl_adapter_forward(x[:rows], *pair, few[:rows])
        size = (pair[0].double().abs()[few[:rows].long()] * x[:rows].double().abs()[:, None]).sum(2)
        bound = 2 * (K / 4 + 64) * u * size
        assert torch.all((h - h2).abs() <= bound)
        assert torch.all((y - y2).abs() <= (pair[1].double().abs()[few[:rows].long()] * (bound + 2 * R * u * h.abs())[:, :, None]).sum(1))
    dx, da, db = tw.bl_adapter_backward(x, a, b, index, h := tw.bl_adapter_forward(x, a, b, index)[1], dy)
    dx2, da2, db2 = tw.bl_adapter_backward(x, *pair, few, h, dy)
    assert torch.equal(dx, dx2) and torch.equal(db[[0, 1023]], db2) and not db[1:1023].any()
    assert torch.equal(da[[0, 1023]], da2) and not any(da[e].any() for e in (1, 2, 511, 1022))
