"""Calls of the training operators that a program makes beside the plain ones:
several at once, stacks past what the GPU holds, large gradients, infinities."""
import pytest
import torch

from mixture_experts_layer_56_b200 import _lib as L
from tests.test_train_ops import U, assert_close, group_tol, ns64, ortho, ortho_check, run_grouped

pytestmark = pytest.mark.gpu

DT = {torch.float32: L.MOE_DTYPE_F32, torch.bfloat16: L.MOE_DTYPE_BF16}


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    yield


def randn(seed, *shape, dtype=torch.float32):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, device="cuda", generator=g).to(dtype)


def ortho_call(m, o, steps=5):
    n, r, c = m.shape
    shape = L.make_ortho_shape(n, r, c, steps, DT[m.dtype])
    ws = torch.zeros(max(256, L.moe_orthogonalize_workspace_size(shape)), dtype=torch.uint8,
                     device="cuda")
    return lambda stream=None: L.moe_orthogonalize(shape, m, o, ws, stream=stream), ws


@pytest.mark.parametrize("r,c", [(64, 330), (1100, 40), (128, 2048)])
def test_orthogonalize_more_clusters_than_fit(r, c):
    """Clusters that start late, beside one another and behind other work, some
    of whose CTAs own no column (330 of 512): each matrix comes out as alone."""
    m = randn(r, 150, r, c)
    outs = [torch.empty(m.shape, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    calls = [ortho_call(m, o) for o in outs]
    streams = [torch.cuda.Stream() for _ in calls]
    big = randn(1, 4096, 4096)
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        for (call, _), s in zip(calls, streams):
            with torch.cuda.stream(s):
                big @ big
            call(stream=s)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], outs[1])
    for i in (0, 77, 149):
        one = torch.empty(1, r, c, dtype=torch.bfloat16, device="cuda")
        ortho_call(m[i:i + 1].contiguous(), one)[0]()
        assert torch.equal(one[0], outs[0][i])
    assert [L.moe_read_status(ws) for _, ws in calls] == [0, 0]


def test_inputs_let_go_of_while_a_side_stream_reads_them():
    """Nothing but the module holds x, and nothing dy and u, once the calls have
    returned: the current stream gets none of their memory before the side
    stream, which starts late, is done."""
    from mixture_experts_layer_56_b200 import training as TR
    bf = torch.bfloat16
    w13, w2 = randn(1, 4, 512, 192, dtype=bf) * 0.1, randn(2, 4, 192, 256, dtype=bf) * 0.1
    gamma = randn(3, 192)
    off = torch.tensor([0, 100, 100, 450, 600], dtype=torch.int32, device="cuda")

    def run(stream=None):
        ex, nm = TR.TrainableExperts(w13, w2), TR.LayerNorm(gamma)
        x, u, dy, m = (randn(s, 600, 192, dtype=bf) for s in (4, 5, 6, 7))
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(stream):
                torch.cuda._sleep(200_000_000)  # some 100 ms
        y = ex.forward(x, off.clone(), stream=stream)
        h = nm.forward(u, stream=stream)
        o = TR.orthogonalize(m.view(1, 600, 192), stream=stream)
        del x, u, m
        dx = ex.backward(dy, stream=stream)
        du = nm.backward(dy, stream=stream)
        del dy
        return [y, h, o, dx, du, ex.dW13, ex.dW2, nm.dgamma], (ex, nm)

    want, _ = run()
    torch.cuda.synchronize()
    junk = [torch.full((600, 192), 7.0, dtype=bf, device="cuda") for _ in range(16)]
    torch.cuda.synchronize()
    del junk
    side = torch.cuda.Stream()
    got, keep = run(side)
    late = not side.query()
    junk = [torch.full((600, 192), 7.0, dtype=bf, device="cuda") for _ in range(16)]
    junk += [torch.zeros(5, dtype=torch.int32, device="cuda") for _ in range(16)]
    assert late, "the side stream was done before the current one could get in its way"
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    assert keep[0].status() == 0 and junk


def test_the_default_stream_by_its_raw_handle():
    """stream=0 beside a current stream of its own: what the call allocates
    belongs to the default stream."""
    from mixture_experts_layer_56_b200 import training as TR
    default, side = torch.cuda.default_stream(), torch.cuda.Stream()
    for raw in (0, 1):
        assert TR._torch_stream(raw) == default
        with TR._on(raw):
            assert torch.cuda.current_stream() == default
    assert TR._torch_stream(side.cuda_stream).cuda_stream == side.cuda_stream
    nm, x = TR.LayerNorm(torch.ones(64, device="cuda")), randn(1, 8, 64)
    want = nm.forward(x)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        y = nm.forward(x, stream=0)
        default.synchronize()
        assert torch.equal(y, want)


def test_status_of_work_on_a_side_stream():
    """A word that is written late, on the stream of the last call, is seen,
    and cleared once."""
    from mixture_experts_layer_56_b200 import training as TR
    ex = TR.TrainableExperts(randn(1, 1, 128, 64), randn(2, 1, 64, 64))
    off = torch.tensor([0, 8], dtype=torch.int32, device="cuda")
    x, side = randn(3, 8, 64), torch.cuda.Stream()
    torch.cuda.synchronize()
    ex.forward(x, off, stream=side)
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)  # some 100 ms
        ex.ws.view(torch.int32)[:1].fill_(L.MOE_ERR_DEVICE_CHECK)
    assert not side.query()
    assert ex.status() == L.MOE_ERR_DEVICE_CHECK
    assert ex.status() == L.MOE_OK
    ex.backward(x, stream=side)
    assert ex.status(stream=side) == L.MOE_OK
    # the last call on the default stream, the word asked for beside another one
    ex.forward(x, off)
    torch.cuda._sleep(200_000_000)
    ex.ws.view(torch.int32)[:1].fill_(L.MOE_ERR_DEVICE_CHECK)
    with torch.cuda.stream(side):
        assert ex.status() == L.MOE_ERR_DEVICE_CHECK


@pytest.mark.parametrize("shape", [(2, 64, 100), (2, 200, 300)])
def test_orthogonalize_with_a_workspace_of_its_own(shape):
    """One workspace serves call after call, and tells how they went."""
    from mixture_experts_layer_56_b200 import training as TR
    m = randn(1, *shape)
    ws = TR.orthogonalize_workspace(m)
    want = TR.orthogonalize(m)
    for _ in range(2):
        assert torch.equal(TR.orthogonalize(m, ws=ws), want)
    assert L.moe_read_status(ws) == L.MOE_OK
    # what it held does not matter
    ws[4:] = 0xFF
    assert torch.equal(TR.orthogonalize(m, ws=ws), want)
    assert L.moe_read_status(ws) == L.MOE_OK
    with pytest.raises(L.MoeError):
        TR.orthogonalize(m, ws=ws[:128])


@pytest.mark.parametrize("own_stream", [False, True])
def test_norm_gradients_of_two_micro_batches(own_stream):
    """Their sum is that of the two calls, rounded once, and not far from the
    whole batch's."""
    from mixture_experts_layer_56_b200 import training as TR
    T, d = 300, 200
    x, dy, gamma, beta = randn(1, 2 * T, d), randn(2, 2 * T, d), randn(3, d), randn(4, d)
    stream = torch.cuda.Stream() if own_stream else None
    torch.cuda.synchronize()
    nm, parts = TR.LayerNorm(gamma, beta), []
    for half in (slice(0, T), slice(T, 2 * T)):
        alone = TR.LayerNorm(gamma, beta)
        for n in (nm, alone):
            n.forward(x[half], stream=stream)
            n.backward(dy[half], stream=stream, accumulate=True)
        parts.append(alone)
    torch.cuda.synchronize()
    for name in ("dgamma", "dbeta"):
        a, b = (getattr(p, name) for p in parts)
        assert torch.equal(getattr(nm, name), a + b)
    X = x.double()
    h = (X - X.mean(1, keepdim=True)) * (X.var(1, unbiased=False, keepdim=True) + 1e-5).rsqrt()
    for got, ref, mag in ((nm.dgamma, (dy.double() * h).sum(0), (dy.double() * h).abs().sum(0)),
                          (nm.dbeta, dy.double().sum(0), dy.double().abs().sum(0))):
        # sums of 2 T terms, each from a dozen roundings of half a step
        assert ((got.double() - ref).abs() <= (2 * T + 12) * 2.0 ** -24 * mag).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("d", [64, 512, 2048, 4096, 16384])
def test_layer_norm_rstd_of_an_exact_variance(d, dtype):
    """Rows of v and -v in turn, v of at most 11 bits: mean 0 and variance v^2
    are exact, and rstd is off by rsqrtf's 2 steps at most, 4 x 2^-24.  (A
    thread's sum of squares is k v^2 of 22 bits, exact for odd k up to 3, and
    equal sums of all threads double exactly.)  Rows past the registers take 1 /
    sqrtf: 2^-24 where the variance is exact, and so is its root.  With 32 values
    per thread, at d = 16384 in float32, the sum goes through 20 v^2 and 28 v^2,
    of 25 bits: two roundings of 5/8 and 7/8 of 2^-24 of the total, half of that
    in its root, and the root's own: 2.75 x 2^-24."""
    bits = 11 if dtype == torch.float32 else 8
    v = (2 ** (bits - 1) + torch.arange(500, device="cuda") % 2 ** (bits - 1)).float()
    v *= 2.0 ** (torch.arange(500, device="cuda") % 9 - 12)
    x = v[:, None] * (1 - 2 * (torch.arange(d, device="cuda") % 2))
    assert torch.equal(x, x.to(dtype).float())
    x = x.to(dtype)
    shape = L.make_norm_shape(500, d, DT[dtype], 0.0)
    y, mean, rstd = torch.empty_like(x), torch.empty(500, device="cuda"), torch.empty(500, device="cuda")
    L.moe_layer_norm(shape, x, torch.ones(d, device="cuda"), None, y, mean, rstd)
    assert (mean == 0).all()
    off = (rstd.double() * v.double() - 1).abs()
    tol = 2.0 ** -24 * (4 if d < 16384 else 2.75 if dtype == torch.float32 else 1)
    assert (off <= tol).all(), (int((off > tol).sum()), float(off.max()) * 2 ** 24)


# ------------------------------------------------------ infinities and NaN
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_swiglu_of_infinities_and_nan(dtype):
    """Each element is its own formula's: infinite and NaN where that is, the
    bits of a run without them elsewhere."""
    inf, nan = float("inf"), float("nan")
    gu, da = randn(1, 9, 256, dtype=dtype), randn(2, 9, 128, dtype=dtype)
    shape = L.make_swiglu_shape(9, 128, DT[dtype])

    def run():
        a, dgu = torch.empty_like(da), torch.empty_like(gu)
        L.moe_swiglu(shape, gu, a)
        L.moe_swiglu_backward(shape, gu, da, dgu)
        return a.double(), dgu.double()

    clean = run()
    odd = torch.tensor([inf, -inf, nan], device="cuda", dtype=dtype)
    gu[1, 3:6] = odd            # gates
    gu[4, 64 + 9:64 + 12] = odd  # ups
    da[7, 70:73] = odd
    b = gu.double().view(9, -1, 2, 64)
    g, u, d = b[:, :, 0], b[:, :, 1], da.double().view(9, -1, 64)
    s = 1 / (1 + torch.exp(-g))
    refs = ((g * s * u).reshape(9, -1),
            torch.stack([d * u * s * (1 + g * (1 - s)), d * g * s], 2).reshape(9, -1))
    for got, want, ref in zip(run(), clean, refs):
        fine = ref.isfinite()
        assert 3 <= int((~fine).sum()) <= 18
        assert torch.equal(got[~fine].nan_to_num(7), ref[~fine].nan_to_num(7))
        assert got[fine].isfinite().all()
        # what has no odd operand keeps its bits
        touched = torch.zeros(9, 2, 2, 64, dtype=torch.bool, device="cuda")
        touched[1, 0, :, 3:6] = touched[4, 0, :, 9:12] = touched[7, 1, :, 6:9] = True
        touched = (touched[:, :, 0] if got.shape[1] == 128 else touched).reshape(9, -1)
        assert torch.equal(got[~touched], want[~touched])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("d", [7, 72, 600, 1283, 4099, 4104, 8200, 20001])
def test_layer_norm_of_infinities_and_nan(d, dtype):
    """They stay in their row, and reach the columns' sums as any term does."""
    T = 700
    x, dy, gamma, beta = randn(1, T, d, dtype=dtype), randn(2, T, d, dtype=dtype), randn(3, d), randn(4, d)
    shape = L.make_norm_shape(T, d, DT[dtype])
    ws = torch.empty(L.moe_layer_norm_workspace_size(shape), dtype=torch.uint8, device="cuda")

    def run():
        y, dx = torch.empty_like(x), torch.empty_like(x)
        st = [torch.empty(T, device="cuda") for _ in range(2)]
        sums = [torch.empty(d, device="cuda") for _ in range(2)]
        L.moe_layer_norm(shape, x, gamma, beta, y, *st)
        L.moe_layer_norm_backward(shape, dy, x, gamma, *st, dx, *sums, ws)
        return y.float(), dx.float(), *sums

    y0, dx0, _, db0 = run()
    x[3, d // 2], x[T - 1, 0], dy[350, d - 1] = float("nan"), float("inf"), float("nan")
    y, dx, dg, db = run()
    rows = torch.ones(T, dtype=torch.bool, device="cuda")
    rows[[3, T - 1]] = False
    assert torch.equal(y[rows], y0[rows]) and y[~rows].isnan().all()
    rows[350] = False
    assert torch.equal(dx[rows], dx0[rows]) and dx[~rows].isnan().all()
    # every h of the two rows is NaN, and dy of one column
    assert dg.isnan().all() and db[d - 1].isnan()
    assert torch.equal(db[:d - 1], db0[:d - 1])


# ------------------------------------------------- groups, sizes and types
def heavy():
    return [0] * 40 + [1400] + [1] * 22 + [78]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_grouped_where_one_group_has_nearly_all_rows(dtype):
    """The averages that choose kernels and tiles say nothing of this group."""
    run_grouped(heavy(), 136, 264, dtype, lead=1, tail=3, seed=3)
    run_grouped([2] * 255 + [1000], 72, 40, dtype, seed=4)
    run_grouped([0] * 200 + [3000] + [0] * 55, 264, 136, dtype, tail=1, seed=5)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("sizes,n,k", [([600, 0, 300, 5], 520, 776), ([3] * 40, 264, 1032),
                                       ([0, 2000], 1288, 72), (heavy(), 136, 264)])
def test_grouped_dw_in_f32_and_accumulated(sizes, n, k, dtype):
    """Several tiles per group, written and then added to."""
    G, rows = len(sizes), sum(sizes)
    off = torch.tensor([0] + sizes).cumsum(0).int().cuda()
    x, dy = randn(1, rows, k, dtype=dtype), randn(2, rows, n, dtype=dtype)
    dw = torch.full((G, n, k), float("nan"), device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    for flags in (L.MOE_GROUPED_DW_F32, L.MOE_GROUPED_DW_F32 | L.MOE_GROUPED_DW_ACCUMULATE):
        before = dw.clone()
        shape = L.make_grouped_shape(rows, G, n, k, DT[dtype], flags)
        L.moe_grouped_matmul_dw(shape, dy, x, off, dw, ws)
        for e in range(G):
            a, b = int(off[e]), int(off[e + 1])
            ref, tol = group_tol(dy[a:b].double().T, x[a:b].double(), b - a, dtype, torch.float32)
            if flags & L.MOE_GROUPED_DW_ACCUMULATE:
                # once per 8 rows where few rows are streamed, else once
                times = (b - a + 7) // 8
                mag = dy[a:b].double().abs().T @ x[a:b].double().abs() + before[e].double().abs()
                ref, tol = ref + before[e].double(), tol + times * U * mag
                if a == b:
                    assert torch.equal(dw[e], before[e])
            assert_close(dw[e], ref, tol, (flags, e))
    assert L.moe_read_status(ws) == 0


# ------------------------------------------------------------ Newton-Schulz
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n,r,c", [(4, 33, 70), (4, 70, 33), (2, 128, 128), (1, 64, 2048),
                                   (2, 2048, 128), (1, 128, 2049), (2, 129, 200), (1, 200, 129),
                                   (2, 256, 264), (2, 300, 257), (2, 1000, 520), (1, 520, 1288)])
def test_orthogonalize_keeps_its_documented_error(n, r, c, dtype):
    """2e-3 of the norm, bf16's rounding (1.7e-3 of evenly spread values) among
    it, with half as much again for single matrices: on chip, around the limits
    of what stays there, and past them."""
    m = randn(r + c, n, r, c, dtype=dtype)
    ref = ns64(m)
    off = (ortho(m).double() - ref).flatten(1).norm(dim=1) / ref.flatten(1).norm(dim=1)
    assert (off <= 3e-3).all(), off


def test_orthogonalize_sixteen_steps():
    for r, c in ((40, 72), (72, 40), (160, 200)):
        m = randn(r, 2, r, c)
        ortho_check(m, steps=16, coef=[1.5, -0.5, 0.0] * 16)


# ------------------------------------------------------------------- graphs
def test_a_captured_step_of_the_module():
    """training.py's calls in a graph, replayed on other inputs, beside an
    eager step of the same weights."""
    from mixture_experts_layer_56_b200 import training as TR
    bf = torch.bfloat16
    w13, w2, gamma = randn(1, 3, 256, 72, dtype=bf) * 0.1, randn(2, 3, 72, 128, dtype=bf) * 0.1, randn(3, 72)
    off = torch.tensor([0, 50, 50, 90], dtype=torch.int32, device="cuda")
    u, dy = randn(4, 90, 72, dtype=bf), randn(5, 90, 72, dtype=bf)

    def make():
        ex, nm = TR.TrainableExperts(w13, w2), TR.LayerNorm(gamma)

        def step():
            y = ex.forward(nm.forward(u), off)
            du = nm.backward(ex.backward(dy), accumulate=True)
            return y, du, TR.orthogonalize(ex.dW2)
        return ex, nm, step

    ex, nm, step = make()
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for seed in (6, 7):
        u.copy_(randn(seed, 90, 72, dtype=bf))
        # the captured backward adds to what is there: the same start for both
        eager = make()
        eager[2]()
        for mine, theirs in ((ex.dW13, eager[0].dW13), (ex.dW2, eager[0].dW2), (nm.dgamma, eager[1].dgamma)):
            mine.copy_(theirs)
        want = eager[2]()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip([*got, ex.dW13, ex.dW2, nm.dgamma],
                        [*want, eager[0].dW13, eager[0].dW2, eager[1].dgamma]):
            assert torch.equal(a, b)


@pytest.mark.parametrize("one_sign,per_row", [(False, 1.5e-9), (True, 6e-9)])
def test_dw_in_f32_keeps_its_documented_error(one_sign, per_row):
    """The header's figures for long groups, with half a step of float32 on top
    (and, for mixed signs, half as much again for one matrix of 64 x 72)."""
    for rows in (1000, 16384, 60000):
        x, dy = randn(1, rows, 72, dtype=torch.bfloat16), randn(2, rows, 64, dtype=torch.bfloat16)
        if one_sign:
            x, dy = x.abs(), dy.abs()
        off = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
        dw = torch.empty(1, 64, 72, device="cuda")
        ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
        L.moe_grouped_matmul_dw(L.make_grouped_shape(rows, 1, 64, 72, L.MOE_DTYPE_BF16, L.MOE_GROUPED_DW_F32),
                                dy, x, off, dw, ws)
        ref = dy.double().T @ x.double()
        off_ = float((dw[0].double() - ref).norm() / ref.norm())
        assert off_ <= per_row * rows + U, (rows, off_ / rows)
