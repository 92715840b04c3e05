"""GPU numerics of the training operators against plain float64 forms.

Tolerances are written down from the arithmetic: u = 2^-24 is half a step of
float32, a store in bf16 adds half a step of bf16, 2^-8 relative, and a sum of
n terms is off by at most n u times the sum of their magnitudes."""
import ctypes

import pytest
import torch

from mixture_experts_layer_56_b200 import _lib as L

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF_STEP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
DT = {torch.float32: L.MOE_DTYPE_F32, torch.bfloat16: L.MOE_DTYPE_BF16}
BOTH = [torch.bfloat16, torch.float32]


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    yield


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *shape, dtype=torch.float32, std=1.0):
    return (torch.randn(*shape, device="cuda", generator=g) * std).to(dtype)


def scratch(nbytes):
    # no call may depend on what its workspace held
    return torch.full((max(256, nbytes),), 0xFF, dtype=torch.uint8, device="cuda")


def clear_status(ws):
    ws[:4] = 0
    return ws


def assert_close(got, ref, tol, what):
    got = got.double()
    bad = ~((got - ref).abs() <= tol)
    assert not bad.any(), (what, int(bad.sum()), float((got - ref).abs().max()),
                           bad.nonzero()[:3].tolist())


# ------------------------------------------------------------ grouped products
def group_tol(a, b, length, dtype, out_dtype):
    """a @ b in 64 bits and how far the kernel may be: |a| @ |b| sums the
    magnitudes; fp32 FMA chains round once a term (u each), the tensor cores
    truncate (2u) at most once per term they add."""
    ref = a @ b
    mag = a.abs() @ b.abs()
    per = 2 * U if dtype == torch.bfloat16 else U
    return ref, (length + 2) * per * mag + HALF_STEP[out_dtype] * ref.abs() + 1e-38


def run_grouped(sizes, n, k, dtype, lead=0, tail=0, seed=0, dw_f32=False, dirs=("fwd", "dx", "dw")):
    """Groups of `sizes` rows between `lead` and `tail` rows that nobody owns;
    those hold NaN and their outputs must stay as they were."""
    g = gen(seed)
    G, rows = len(sizes), lead + sum(sizes) + tail
    off = [lead]
    for s in sizes:
        off.append(off[-1] + s)
    offsets = torch.tensor(off, dtype=torch.int32, device="cuda")
    x, dy = randn(g, rows, k, dtype=dtype), randn(g, rows, n, dtype=dtype)
    w = randn(g, G, n, k, dtype=dtype)
    owned = torch.zeros(rows, dtype=torch.bool, device="cuda")
    owned[lead:off[-1]] = True
    x[~owned] = float("nan")
    dy[~owned] = float("nan")
    flags = L.MOE_GROUPED_DW_F32 if dw_f32 else 0
    shape = L.make_grouped_shape(rows, G, n, k, DT[dtype], flags)
    ws = clear_status(scratch(L.moe_grouped_workspace_size(shape)))
    got = {}
    spans = list(zip(off[:-1], off[1:]))
    mark = 7.0
    if "fwd" in dirs:
        y = torch.full((rows, n), mark, dtype=dtype, device="cuda")
        L.moe_grouped_matmul(shape, x, offsets, w, y, ws)
        assert (y[~owned] == mark).all()
        for e, (a, b) in enumerate(spans):
            ref, tol = group_tol(x[a:b].double(), w[e].double().T, k, dtype, dtype)
            assert_close(y[a:b], ref, tol, ("fwd", e))
        got["y"] = y
    if "dx" in dirs:
        dx = torch.full((rows, k), mark, dtype=dtype, device="cuda")
        L.moe_grouped_matmul_dx(shape, dy, offsets, w, dx, ws)
        assert (dx[~owned] == mark).all()
        for e, (a, b) in enumerate(spans):
            ref, tol = group_tol(dy[a:b].double(), w[e].double(), n, dtype, dtype)
            assert_close(dx[a:b], ref, tol, ("dx", e))
        got["dx"] = dx
    if "dw" in dirs:
        odt = torch.float32 if dw_f32 else dtype
        dw = torch.full((G, n, k), float("nan"), dtype=odt, device="cuda")
        L.moe_grouped_matmul_dw(shape, dy, x, offsets, dw, ws)
        for e, (a, b) in enumerate(spans):
            ref, tol = group_tol(dy[a:b].double().T, x[a:b].double(), b - a, dtype, odt)
            assert_close(dw[e], ref, tol, ("dw", e))
            if a == b:
                assert (dw[e] == 0).all()
        got["dw"] = dw
    assert L.moe_read_status(ws) == 0
    return got


SIZES = {
    "one_row": [1],
    "one_each": [1] * 9,
    "tile_edges": [63, 64, 65, 127, 128, 129],
    "pair_edges": [255, 256, 257, 511],
    "empty_around": [0, 0, 37, 0, 300, 0],
    "all_empty": [0, 0, 0],
    "heavy": [5, 1200, 0, 17, 2],
}


@pytest.mark.parametrize("n,k", [(8, 8), (72, 264), (256, 128), (520, 200)])
@pytest.mark.parametrize("sizes", SIZES.values(), ids=SIZES.keys())
def test_grouped_bf16(sizes, n, k):
    run_grouped(sizes, n, k, torch.bfloat16, lead=3, tail=5)


@pytest.mark.parametrize("n,k", [(1, 1), (7, 33), (64, 64), (130, 65)])
@pytest.mark.parametrize("sizes", SIZES.values(), ids=SIZES.keys())
def test_grouped_f32(sizes, n, k):
    run_grouped(sizes, n, k, torch.float32, lead=2, tail=1)


@pytest.mark.parametrize("sizes,n,k", [([700, 0, 333], 1288, 776), ([1] * 200 + [90] * 56, 136, 1032),
                                       ([40, 0, 1, 3000], 2048, 512)])
def test_grouped_bf16_many_tiles(sizes, n, k):
    run_grouped(sizes, n, k, torch.bfloat16, tail=9)


def test_grouped_dw_in_f32():
    run_grouped(SIZES["pair_edges"] + [0, 3], 264, 136, torch.bfloat16, lead=1, dw_f32=True,
                dirs=("dw",))


@pytest.mark.parametrize("dtype", BOTH)
def test_grouped_dw_accumulates(dtype):
    sizes, n, k = [70, 0, 1, 129], 72, 136
    g = gen(3)
    rows = sum(sizes)
    offsets = torch.tensor([0, 70, 70, 71, 200], dtype=torch.int32, device="cuda")
    x, dy = randn(g, rows, k, dtype=dtype), randn(g, rows, n, dtype=dtype)
    dw = randn(g, len(sizes), n, k)
    before = dw.clone()
    shape = L.make_grouped_shape(rows, len(sizes), n, k, DT[dtype],
                                 L.MOE_GROUPED_DW_F32 | L.MOE_GROUPED_DW_ACCUMULATE)
    ws = clear_status(scratch(256))
    L.moe_grouped_matmul_dw(shape, dy, x, offsets, dw, ws)
    assert torch.equal(dw[1], before[1])
    a = 0
    for e, s in enumerate(sizes):
        ref, tol = group_tol(dy[a:a + s].double().T, x[a:a + s].double(), s, dtype, torch.float32)
        full = ref + before[e].double()
        assert_close(dw[e], full, tol + U * full.abs(), e)
        a += s
    # no rows at all: nothing is added, or everything is zeroed
    none = L.make_grouped_shape(0, len(sizes), n, k, DT[dtype],
                                L.MOE_GROUPED_DW_F32 | L.MOE_GROUPED_DW_ACCUMULATE)
    kept = dw.clone()
    L.moe_grouped_matmul_dw(none, None, None, None, dw, ws)
    assert torch.equal(dw, kept)
    none.flags = L.MOE_GROUPED_DW_F32
    L.moe_grouped_matmul_dw(none, None, None, None, dw, ws)
    assert (dw == 0).all()


@pytest.mark.parametrize("dtype", BOTH)
def test_grouped_offsets_out_of_range_are_clamped(dtype):
    """Offsets past the rows, negative or falling reach no memory outside and
    give no row to two groups."""
    n = k = 64
    rows = 100
    g = gen(5)
    x, w = randn(g, rows, k, dtype=dtype), randn(g, 4, n, k, dtype=dtype)
    off = torch.tensor([-50, 30, 10, 4000, 2**31 - 1], dtype=torch.int32, device="cuda")
    # taken as [0, 30), [30, 30), [30, 100), [100, 100)
    y = torch.zeros(rows, n, dtype=dtype, device="cuda")
    dw = torch.full((4, n, k), float("nan"), device="cuda", dtype=dtype)
    shape = L.make_grouped_shape(rows, 4, n, k, DT[dtype])
    ws = clear_status(scratch(256))
    L.moe_grouped_matmul(shape, x, off, w, y, ws)
    ref, tol = group_tol(x[30:].double(), w[2].double().T, k, dtype, dtype)
    assert_close(y[30:], ref, tol, "rows of group 2")
    ref, tol = group_tol(x[:30].double(), w[0].double().T, k, dtype, dtype)
    assert_close(y[:30], ref, tol, "rows of group 0")
    L.moe_grouped_matmul_dw(shape, y, x, off, dw, ws)
    assert (dw[1] == 0).all() and (dw[3] == 0).all() and torch.isfinite(dw.float()).all()
    assert L.moe_read_status(ws) == 0


@pytest.mark.parametrize("dtype", BOTH)
def test_grouped_nan_stays_in_its_group(dtype):
    """A NaN in one group's rows reaches that group's outputs alone, also
    where a k-block of the weight gradient spans two groups."""
    sizes, n, k = [40, 24, 70], 64, 64
    g = gen(6)
    offsets = torch.tensor([0, 40, 64, 134], dtype=torch.int32, device="cuda")
    x, dy = randn(g, 134, k, dtype=dtype), randn(g, 134, n, dtype=dtype)
    x[45, 3] = float("nan")
    dy[50, 1] = float("inf")
    w = randn(g, 3, n, k, dtype=dtype)
    y, dw = torch.empty_like(dy), torch.empty_like(w)
    shape = L.make_grouped_shape(134, 3, n, k, DT[dtype])
    ws = clear_status(scratch(256))
    L.moe_grouped_matmul(shape, x, offsets, w, y, ws)
    L.moe_grouped_matmul_dw(shape, dy, x, offsets, dw, ws)
    nan_rows = torch.isnan(y.float()).any(1).nonzero().flatten().tolist()
    assert nan_rows == [45]
    assert torch.isfinite(dw[0].float()).all() and torch.isfinite(dw[2].float()).all()
    assert not torch.isfinite(dw[1].float()).all()


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("groups", [1, 31, 32, 33, 256])
def test_grouped_with_every_number_of_groups_and_any_offsets(groups, dtype):
    """Spans of random offsets, as the header defines them, for group counts
    around a warp's width and at the limit."""
    g = gen(groups)
    rows, n, k = 500, 16, 24
    off = torch.randint(-100, 700, (groups + 1,), generator=g, device="cuda", dtype=torch.int32)
    held = torch.cummax(off.clamp(0, rows), 0).values.tolist()
    x, dy = randn(g, rows, k, dtype=dtype), randn(g, rows, n, dtype=dtype)
    w = randn(g, groups, n, k, dtype=dtype)
    y, dx = torch.full_like(dy, 7.0), torch.full_like(x, 7.0)
    dw = torch.full_like(w, float("nan"))
    shape = L.make_grouped_shape(rows, groups, n, k, DT[dtype])
    ws = clear_status(scratch(256))
    L.moe_grouped_matmul(shape, x, off, w, y, ws)
    L.moe_grouped_matmul_dx(shape, dy, off, w, dx, ws)
    L.moe_grouped_matmul_dw(shape, dy, x, off, dw, ws)
    assert (y[:held[0]] == 7).all() and (y[held[-1]:] == 7).all()
    assert (dx[:held[0]] == 7).all() and (dx[held[-1]:] == 7).all()
    for e, (a, b) in enumerate(zip(held[:-1], held[1:])):
        assert_close(y[a:b], *group_tol(x[a:b].double(), w[e].double().T, k, dtype, dtype), e)
        assert_close(dx[a:b], *group_tol(dy[a:b].double(), w[e].double(), n, dtype, dtype), e)
        assert_close(dw[e], *group_tol(dy[a:b].double().T, x[a:b].double(), b - a, dtype, dtype), e)
    assert L.moe_read_status(ws) == 0


# Average rows per group on either side of every choice of tile (32, 48, 112
# and 512 rows; widths below 256), with sizes spread around it.
@pytest.mark.parametrize("per,n,k,groups", [(3, 320, 72, 9), (40, 264, 136, 20), (47, 512, 64, 8),
                                            (49, 264, 200, 8), (100, 776, 64, 6), (113, 520, 136, 5),
                                            (200, 264, 72, 7), (511, 264, 64, 3), (513, 264, 64, 3),
                                            (700, 1040, 80, 2), (130, 600, 512, 6), (200, 520, 776, 7),
                                            (300, 1288, 520, 4)])
def test_grouped_bf16_at_every_tile_choice(per, n, k, groups):
    g = torch.Generator().manual_seed(per)
    sizes = torch.randint(0, 2 * per + 1, (groups,), generator=g).tolist()
    sizes[0] += max(0, groups * per - sum(sizes))
    run_grouped(sizes, n, k, torch.bfloat16, dirs=("fwd", "dx"))


@pytest.mark.parametrize("sizes,n,k", [([300, 0, 129], 70, 300), ([700], 33, 520),
                                       ([40] * 5, 520, 264), ([3], 17, 2000), ([2500, 1], 130, 70),
                                       ([900, 0, 800], 520, 136)])
def test_grouped_f32_few_tiles_and_long_sums(sizes, n, k):
    """Clusters share a tile's reduction, or 128 x 128 tiles."""
    run_grouped(sizes, n, k, torch.float32, lead=1, tail=2)


@pytest.mark.parametrize("n,k", [(1, 1), (33, 130), (70, 1025), (2500, 128), (1030, 260), (513, 2047)])
@pytest.mark.parametrize("sizes", [[1], [2, 0, 3], [8], [9, 1, 0, 4], [1] * 40, [0] * 30 + [50, 5],
                                   [0] * 7 + [17]])
def test_grouped_f32_few_rows(sizes, n, k):
    """Groups of few rows on average, whose matrices are streamed."""
    run_grouped(sizes, n, k, torch.float32, lead=3, tail=2, seed=n + len(sizes))


def test_grouped_f32_few_rows_accumulate():
    """Onto what is there, a group of more rows than are added at once and
    empty ones among them."""
    g = gen(8)
    sizes, n, k = [0, 1, 21, 0, 8, 2], 150, 262
    off = torch.tensor([0] + sizes).cumsum(0).int().cuda()
    x, dy = randn(g, sum(sizes), k), randn(g, sum(sizes), n)
    dw = randn(g, len(sizes), n, k)
    before = dw.clone()
    shape = L.make_grouped_shape(sum(sizes), len(sizes), n, k, L.MOE_DTYPE_F32,
                                 L.MOE_GROUPED_DW_ACCUMULATE)
    ws = clear_status(scratch(L.moe_grouped_workspace_size(shape)))
    L.moe_grouped_matmul_dw(shape, dy, x, off, dw, ws)
    for e in range(len(sizes)):
        a, b = int(off[e]), int(off[e + 1])
        ref, tol = group_tol(dy[a:b].double().T, x[a:b].double(), b - a, torch.float32, torch.float32)
        full = ref + before[e].double()
        # each of the three additions onto the sum rounds once
        assert_close(dw[e], full, tol + 3 * U * (before[e].double().abs() + dy[a:b].double().abs().T
                                                 @ x[a:b].double().abs()), e)
        if a == b:
            assert torch.equal(dw[e], before[e])


# ------------------------------------------------------------------- SwiGLU
def swiglu_ref(gu, da):
    b = gu.double().view(gu.shape[0], -1, 2, 64)
    g, u = b[:, :, 0], b[:, :, 1]
    s = torch.sigmoid(g)
    a = g * s * u
    d = da.double().view(g.shape)
    dg = d * u * s * (1 + g * (1 - s))
    du = d * g * s
    flat = lambda t: t.reshape(gu.shape[0], -1)  # noqa: E731
    # |dg| before its factor 1 + g (1 - s) cancels
    mag = (d * u).abs() * s * (1 + g.abs() * (1 - s))
    return (flat(a), flat(torch.stack([dg, du], 2)),
            flat(torch.stack([mag, du.abs()], 2)), flat(g.abs()),
            flat(torch.stack([g.abs(), g.abs()], 2)))


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("rows,inter", [(1, 64), (3, 64), (1, 1408), (257, 192), (1000, 896)])
def test_swiglu(rows, inter, dtype):
    g = gen(rows)
    gu = randn(g, rows, 2 * inter, dtype=dtype, std=3.0)
    da = randn(g, rows, inter, dtype=dtype)
    gu[0, :8] = torch.tensor([0.0, -0.0, 60.0, -60.0, 100.0, -100.0, 1e-30, -1e4], device="cuda")
    a, dgu = torch.empty_like(da), torch.empty_like(gu)
    shape = L.make_swiglu_shape(rows, inter, DT[dtype])
    L.moe_swiglu(shape, gu, a)
    L.moe_swiglu_backward(shape, gu, da, dgu)
    ra, rd, mag, absg, absg2 = swiglu_ref(gu, da)
    # s: the exponent's rounding is |g| u relative, and a few u for exp and the
    # reciprocal; below e^-87 it may be flushed to 0
    tiny = 2.0 ** -120 * 2e4
    assert_close(a, ra, (HALF_STEP[dtype] + (8 + 2 * absg) * U) * ra.abs() + tiny * 100, "a")
    assert_close(dgu, rd, HALF_STEP[dtype] * rd.abs() + (16 + 4 * absg2) * U * mag + tiny * 100,
                 "dgu")
    # the gradient may overwrite gu
    gu2 = gu.clone()
    L.moe_swiglu_backward(shape, gu2, da, gu2)
    assert torch.equal(gu2, dgu)


# --------------------------------------------------------------- layer norm
def norm_check(T, d, dtype, offset=0.0, eps=1e-5, beta=True, const_row=False, seed=1):
    g = gen(seed)
    x = (randn(g, T, d) + offset).to(dtype)
    if const_row:
        x[T // 2] = 1.5
    dy = randn(g, T, d, dtype=dtype)
    gamma, bt = 1 + 0.3 * randn(g, d), randn(g, d) if beta else None
    shape = L.make_norm_shape(T, d, DT[dtype], eps)
    y, dx = torch.empty_like(x), torch.empty_like(x)
    mean, rstd = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    dgamma, dbeta = torch.empty(d, device="cuda"), torch.empty(d, device="cuda")
    ws = scratch(L.moe_layer_norm_workspace_size(shape))
    L.moe_layer_norm(shape, x, gamma, bt, y, mean, rstd)
    L.moe_layer_norm_backward(shape, dy, x, gamma, mean, rstd, dx, dgamma, dbeta, ws)
    X, G, DY = x.double(), gamma.double(), dy.double()
    eps = ctypes.c_float(eps).value  # as the library receives it
    mu = X.mean(1, keepdim=True)
    var = ((X - mu) ** 2).mean(1, keepdim=True)
    rs = (var + eps) ** -0.5
    h = (X - mu) * rs
    # chains of at most n additions: a thread's own values (a wide row's: d /
    # 512), 5 shuffles, 16 warps, and a few operations on top
    n = max(16, d / 512) + 32
    e_mu = n * U * X.abs().mean(1, keepdim=True)
    # an error of the mean adds its square to the variance
    e_rs = (n * U + e_mu ** 2 * rs ** 2) * rs
    e_h = (e_mu + U * (X - mu).abs()) * rs + (X - mu).abs() * e_rs + 2 * U * h.abs()
    assert_close(mean, mu[:, 0], (e_mu + U * mu.abs())[:, 0], "mean")
    assert_close(rstd, rs[:, 0], (e_rs + 2 * U * rs)[:, 0], "rstd")
    ry = h * G + (bt.double() if beta else 0.0)
    assert_close(y, ry, HALF_STEP[dtype] * ry.abs() + e_h * G.abs() + 2 * U * (h * G).abs()
                 + U * ry.abs(), "y")
    v = DY * G
    s1, s2 = v.mean(1, keepdim=True), (v * h).mean(1, keepdim=True)
    rdx = rs * (v - s1 - h * s2)
    e_s1 = (n + 1) * U * v.abs().mean(1, keepdim=True)
    e_s2 = (n + 2) * U * (v * h).abs().mean(1, keepdim=True) + (v.abs() * e_h).mean(1, keepdim=True)
    e_dx = rs * (3 * U * (v.abs() + s1.abs() + (h * s2).abs()) + e_s1 + h.abs() * e_s2
                 + e_h * s2.abs()) + e_rs * (v - s1 - h * s2).abs()
    assert_close(dx, rdx, HALF_STEP[dtype] * rdx.abs() + e_dx + 2 * U * rdx.abs(), "dx")
    # column sums: a block's rows (T over 148 blocks or 64 slices at least),
    # then the partial rows in 8 slices
    m = T / 64 + 8 + 3000 / 8 + 8
    assert_close(dgamma, (DY * h).sum(0), m * U * (DY * h).abs().sum(0) + (DY.abs() * e_h).sum(0)
                 + 1e-30, "dgamma")
    assert_close(dbeta, DY.sum(0), m * U * DY.abs().sum(0) + 1e-30, "dbeta")
    # in place: the same bits
    y2, dx2 = x.clone(), dy.clone()
    L.moe_layer_norm(shape, y2, gamma, bt, y2, None, None)
    assert torch.equal(y2, y)
    dg2 = torch.empty_like(dgamma)
    L.moe_layer_norm_backward(shape, dx2, x, gamma, mean, rstd, dx2, dg2, None, ws)
    assert torch.equal(dx2, dx) and torch.equal(dg2, dgamma)


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("T,d", [(1, 1), (1, 2), (5, 7), (1, 64), (3, 250), (9, 256), (2, 513),
                                 (301, 1280), (33, 2048), (2, 2049), (700, 1283), (65, 4096),
                                 (7, 4104), (3, 8192), (5, 8200), (2, 20001)])
def test_layer_norm(T, d, dtype):
    norm_check(T, d, dtype)


@pytest.mark.parametrize("dtype", BOTH)
def test_layer_norm_many_rows(dtype):
    norm_check(5003, 320, dtype)
    norm_check(2500, 72, dtype, beta=False)


def test_layer_norm_far_from_zero():
    """A mean of 1000 standard deviations: the variance is taken about it."""
    norm_check(40, 768, torch.float32, offset=1000.0)
    norm_check(4, 10000, torch.float32, offset=1000.0)


def test_layer_norm_constant_row_and_no_eps():
    norm_check(9, 640, torch.float32, const_row=True)
    norm_check(9, 640, torch.bfloat16, eps=0.0)


def test_layer_norm_of_no_rows_zeroes_its_weights_gradient():
    s = L.make_norm_shape(0, 100)
    dg, db = torch.ones(100, device="cuda"), torch.ones(100, device="cuda")
    L.moe_layer_norm_backward(s, None, None, None, None, None, None, dg, db, None, ws_bytes=0)
    assert (dg == 0).all() and (db == 0).all()


def test_layer_norm_gradient_against_differences():
    """d sum(y w) / d x by central differences of the float64 form."""
    g = gen(9)
    T, d = 2, 40
    x, w, gamma = randn(g, T, d), randn(g, T, d), 1 + 0.3 * randn(g, d)
    shape = L.make_norm_shape(T, d, L.MOE_DTYPE_F32)
    y, dx = torch.empty_like(x), torch.empty_like(x)
    mean, rstd = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    dg = torch.empty(d, device="cuda")
    L.moe_layer_norm(shape, x, gamma, None, y, mean, rstd)
    L.moe_layer_norm_backward(shape, w, x, gamma, mean, rstd, dx, dg, None,
                              scratch(L.moe_layer_norm_workspace_size(shape)))

    def loss(t, gm):
        m = t.mean(1, keepdim=True)
        return (((t - m) / ((t - m).square().mean(1, keepdim=True) + 1e-5).sqrt()) * gm
                * w.double()).sum()
    step = 1e-5  # differences are off by step^2 f''' ~ 1e-9 and 1e-15 / step
    for i, j in ((0, 0), (1, 17), (1, 39)):
        e = torch.zeros(T, d, dtype=torch.float64, device="cuda")
        e[i, j] = step
        num = (loss(x.double() + e, gamma.double()) - loss(x.double() - e, gamma.double())) / (2 * step)
        assert abs(float(num) - float(dx[i, j])) < 1e-5 * (1 + abs(float(num)))
    e = torch.zeros(d, dtype=torch.float64, device="cuda")
    e[5] = step
    num = (loss(x.double(), gamma.double() + e) - loss(x.double(), gamma.double() - e)) / (2 * step)
    assert abs(float(num) - float(dg[5])) < 1e-5 * (1 + abs(float(num)))


# ----------------------------------------------------------- Newton-Schulz
COEF = (3.4445, -4.7750, 2.0315)


def ns64(m, steps=5, coef=None):
    x = m.double()
    x = x / (x.square().sum((-2, -1), keepdim=True).sqrt() + 1e-7)
    for i in range(steps):
        a, b, c = coef[3 * i:3 * i + 3] if coef else COEF
        if x.shape[-2] <= x.shape[-1]:
            q = x @ x.mT
            x = a * x + (b * q + c * (q @ q)) @ x
        else:
            q = x.mT @ x
            x = a * x + x @ (b * q + c * (q @ q))
    return x


# Relative to |O|_F, per matrix: bf16's half step, and fp16's half step (2^-11)
# for each rounded operand of a step (hi, A, B) times the step's gain on it,
# at most |b| + 2 |c| < 9 for singular values up to 1.15.  Earlier steps' share
# is passed on with a slope under 1.7 and was measured, in a simulation of the
# same roundings, at 2e-3 in all for random matrices and less for structured
# ones: 24 half steps hold it with room.
ORTHO_TOL = 2.0 ** -8 + 24 * 2.0 ** -11


def ortho(m, steps=5, coef=None):
    n, r, c = m.shape
    shape = L.make_ortho_shape(n, r, c, steps, DT[m.dtype])
    ws = clear_status(scratch(L.moe_orthogonalize_workspace_size(shape)))
    o = torch.full(m.shape, float("nan"), dtype=torch.bfloat16, device="cuda")
    L.moe_orthogonalize(shape, m, o, ws, coef=coef)
    assert L.moe_read_status(ws) == 0
    return o


def ortho_check(m, steps=5, coef=None):
    o, ref = ortho(m, steps, coef).double(), ns64(m, steps, coef)
    off = (o - ref).flatten(1).norm(dim=1)
    assert (off <= ORTHO_TOL * ref.flatten(1).norm(dim=1)).all(), off / ref.flatten(1).norm(dim=1)
    return o


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("n,r,c", [(1, 1, 1), (3, 1, 50), (2, 50, 1), (1, 8, 8), (5, 33, 70),
                                   (4, 70, 33), (2, 128, 128), (2, 256, 264), (3, 300, 257),
                                   (1, 64, 2048), (2, 1000, 520), (70, 40, 24)])
def test_orthogonalize(n, r, c, dtype):
    ortho_check(randn(gen(r + c), n, r, c, dtype=dtype))


@pytest.mark.parametrize("kind", ["rank1", "rank8", "spiked", "decaying", "one_entry", "identity"])
@pytest.mark.parametrize("r,c", [(96, 200), (200, 96), (520, 776)])
def test_orthogonalize_structured(kind, r, c):
    g = gen(11)
    m = randn(g, 2, r, c)
    if kind == "rank1":
        m = randn(g, 2, r, 1) @ randn(g, 2, 1, c)
    elif kind == "rank8":
        m = randn(g, 2, r, 8) @ randn(g, 2, 8, c)
    elif kind == "spiked":
        m = 0.1 * m + randn(g, 2, r, 4) @ randn(g, 2, 4, c)
    elif kind == "decaying":
        m = m / torch.arange(1, r + 1, device="cuda")[:, None]
    elif kind == "one_entry":
        m = torch.zeros_like(m)
        m[0, r - 1, 2] = -3.0
        m[1, 0, c - 1] = 1e-3
    elif kind == "identity":
        m = torch.eye(r, c, device="cuda").expand(2, r, c).contiguous()
    ortho_check(m)


def test_orthogonalize_scales():
    """The result does not depend on the scale of M, up to the 1e-7 in the
    norm; squares of its entries may overflow float32."""
    m = randn(gen(2), 3, 48, 80)
    for scale in (1e30, 1e-3, 2.0 ** 100):
        ortho_check(m * scale)


def test_orthogonalize_steps_and_coefficients():
    m = randn(gen(4), 2, 72, 40, dtype=torch.bfloat16)
    ortho_check(m, steps=1)
    ortho_check(m, steps=2)
    # the cubic iteration (c = 0), and other coefficients at every step
    ortho_check(m, steps=3, coef=[1.5, -0.5, 0.0] * 3)
    ortho_check(m, steps=4, coef=[4.0848, -6.8946, 2.9270, 3.9505, -6.3029, 2.6377,
                                  3.7418, -5.5913, 2.3037, 2.8769, -3.1427, 1.2046])


def test_orthogonalize_zeros_and_nan():
    m = randn(gen(5), 4, 40, 56)
    good = ortho(m)
    m[1] = 0
    m[2, 3, 4] = float("nan")
    m[3, 0, 0] = float("inf")
    o = ortho(m)
    assert torch.equal(o[0], good[0])
    assert (o[1] == 0).all()
    assert torch.isnan(o[2].float()).any() and torch.isnan(o[3].float()).any()


# ---------------------------------------------------- streams, graphs, order
def training_step(g, sizes, d, inter, dtype=torch.bfloat16):
    """Buffers of one expert training step, and a function that runs it."""
    G, rows = len(sizes), sum(sizes)
    off = torch.tensor([0] + list(torch.tensor(sizes).cumsum(0)), dtype=torch.int32, device="cuda")
    t = {"x": randn(g, rows, d, dtype=dtype), "gamma": 1 + 0.1 * randn(g, d),
         "beta": 0.1 * randn(g, d),
         "w13": randn(g, G, 2 * inter, d, dtype=dtype, std=d ** -0.5),
         "w2": randn(g, G, d, inter, dtype=dtype, std=inter ** -0.5),
         "dy": randn(g, rows, d, dtype=dtype)}
    new = lambda *s, dt=dtype: torch.empty(*s, dtype=dt, device="cuda")  # noqa: E731
    t |= {"h": new(rows, d), "mean": new(rows, dt=torch.float32), "rstd": new(rows, dt=torch.float32),
          "gu": new(rows, 2 * inter), "a": new(rows, inter), "y": new(rows, d),
          "da": new(rows, inter), "dgu": new(rows, 2 * inter), "dh": new(rows, d),
          "dw13": new(G, 2 * inter, d), "dw2": new(G, d, inter), "dx": new(rows, d),
          "dgamma": new(d, dt=torch.float32), "dbeta": new(d, dt=torch.float32),
          "up13": new(G, 2 * inter, d, dt=torch.bfloat16)}
    nrm = L.make_norm_shape(rows, d, DT[dtype])
    up = L.make_grouped_shape(rows, G, 2 * inter, d, DT[dtype])
    down = L.make_grouped_shape(rows, G, d, inter, DT[dtype])
    sw = L.make_swiglu_shape(rows, inter, DT[dtype])
    om = L.make_ortho_shape(G, 2 * inter, d, 5, DT[dtype])
    ws = clear_status(scratch(256))
    wn = scratch(L.moe_layer_norm_workspace_size(nrm))
    wo = clear_status(scratch(L.moe_orthogonalize_workspace_size(om)))

    def step(stream=None):
        L.moe_layer_norm(nrm, t["x"], t["gamma"], t["beta"], t["h"], t["mean"], t["rstd"], stream=stream)
        L.moe_grouped_matmul(up, t["h"], off, t["w13"], t["gu"], ws, stream=stream)
        L.moe_swiglu(sw, t["gu"], t["a"], stream=stream)
        L.moe_grouped_matmul(down, t["a"], off, t["w2"], t["y"], ws, stream=stream)
        L.moe_grouped_matmul_dx(down, t["dy"], off, t["w2"], t["da"], ws, stream=stream)
        L.moe_grouped_matmul_dw(down, t["dy"], t["a"], off, t["dw2"], ws, stream=stream)
        L.moe_swiglu_backward(sw, t["gu"], t["da"], t["dgu"], stream=stream)
        L.moe_grouped_matmul_dx(up, t["dgu"], off, t["w13"], t["dh"], ws, stream=stream)
        L.moe_grouped_matmul_dw(up, t["dgu"], t["h"], off, t["dw13"], ws, stream=stream)
        L.moe_layer_norm_backward(nrm, t["dh"], t["x"], t["gamma"], t["mean"], t["rstd"], t["dx"],
                                  t["dgamma"], t["dbeta"], wn, stream=stream)
        L.moe_orthogonalize(om, t["dw13"], t["up13"], wo, stream=stream)
    return t, off, step


OUTS = ("h", "gu", "a", "y", "da", "dw2", "dgu", "dh", "dw13", "dx", "dgamma", "dbeta", "up13")


def test_training_step_end_to_end():
    """Layer norm, experts and their gradients, strung together as a step uses
    them, against autograd in float64."""
    t, off, step = training_step(gen(21), [50, 0, 129, 7], 128, 64)
    step()
    leaf = {k: t[k].double().requires_grad_() for k in ("x", "gamma", "beta", "w13", "w2")}
    h = torch.nn.functional.layer_norm(leaf["x"], (128,), leaf["gamma"], leaf["beta"], 1e-5)
    ys = []
    o = off.tolist()
    for e in range(4):
        gu = (h[o[e]:o[e + 1]] @ leaf["w13"][e].T).view(-1, 1, 2, 64)
        a = torch.nn.functional.silu(gu[:, :, 0]) * gu[:, :, 1]
        ys.append(a.reshape(-1, 64) @ leaf["w2"][e].T)
    y = torch.cat(ys)
    y.backward(t["dy"].double())
    # every intermediate is rounded to bf16, at most 6 of them in a row, each
    # half a step (2^-8) at most and of random sign: 6 half steps in norm
    for name, ref in (("y", y), ("dx", leaf["x"].grad), ("dw13", leaf["w13"].grad),
                      ("dw2", leaf["w2"].grad), ("dgamma", leaf["gamma"].grad),
                      ("dbeta", leaf["beta"].grad)):
        off_ = (t[name].double() - ref).norm() / ref.norm()
        assert off_ <= 6 * 2.0 ** -8, (name, float(off_))
    ref = ns64(t["dw13"])
    live = ref.flatten(1).norm(dim=1) > 0
    assert live.tolist() == [True, False, True, True]
    err = (t["up13"].double() - ref).flatten(1).norm(dim=1)
    assert (err <= ORTHO_TOL * ref.flatten(1).norm(dim=1)).all()


def test_training_step_repeats_bit_for_bit_and_replays():
    t, _, step = training_step(gen(22), [300, 3, 0, 260, 90], 256, 128)
    step()
    torch.cuda.synchronize()
    first = {k: t[k].clone() for k in OUTS}
    for k in OUTS:
        t[k].fill_(float("nan"))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    step(stream=side)
    side.synchronize()
    for k in OUTS:
        assert torch.equal(t[k], first[k]), k
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    # other inputs, then the first ones again
    x0 = t["x"].clone()
    t["x"].normal_()
    graph.replay()
    assert not torch.equal(t["y"], first["y"])
    t["x"].copy_(x0)
    for k in OUTS:
        t[k].fill_(float("nan"))
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    for k in OUTS:
        assert torch.equal(t[k], first[k]), k


def test_two_streams_at_once():
    """Two steps on two streams, each with its own workspaces."""
    a, b = training_step(gen(23), [200, 100], 128, 64), training_step(gen(24), [10, 333], 128, 64)
    want = []
    for t, _, step in (a, b):
        step()
        torch.cuda.synchronize()
        want.append({k: t[k].clone() for k in OUTS})
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    for st in s:
        st.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        for (t, _, step), st in zip((a, b), s):
            step(stream=st)
    torch.cuda.synchronize()
    for (t, _, _), w in zip((a, b), want):
        for k in OUTS:
            assert torch.equal(t[k], w[k]), k


def test_first_calls_in_a_capture():
    """A process whose first calls are captured: nothing that a call sets up
    is left out of, or breaks, the capture."""
    import subprocess
    import sys
    code = """
import torch
from tests import test_train_ops as T
t, off, step = T.training_step(T.gen(1), [40, 0, 200], 256, 64)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    step()
g.replay()
torch.cuda.synchronize()
first = {k: t[k].clone() for k in T.OUTS}
for k in T.OUTS:
    t[k].fill_(float('nan'))
step()
torch.cuda.synchronize()
assert all(torch.equal(t[k], first[k]) for k in T.OUTS)
print('same')
"""
    from tests.conftest import ROOT
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and "same" in r.stdout, r.stderr[-2000:]


def test_stages_are_traced():
    t, _, step = training_step(gen(25), [64, 64], 128, 64)
    L.moe_profile_enable(True)
    try:
        step()
        names = [n for n, _ in L.moe_profile_read()]
    finally:
        L.moe_profile_enable(False)
    assert names == ["layer_norm", "grouped_matmul", "swiglu", "grouped_matmul", "grouped_matmul_dx",
                     "grouped_matmul_dw", "swiglu_backward", "grouped_matmul_dx",
                     "grouped_matmul_dw", "layer_norm_backward", "orthogonalize"]
