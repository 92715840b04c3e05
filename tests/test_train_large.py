"""The training operators on tensors of more than 2^31 elements: the rows,
groups and matrices at both ends and around element 2^31 against plain float64
forms (tolerances as for the small ones: half a step of the stored type, and
of fp32 per term of a sum)."""
import pytest
import torch

from mixture_experts_layer_56_b200 import _lib as L

pytestmark = pytest.mark.gpu

U, HALF_BF16 = 2.0 ** -24, 2.0 ** -8


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    if torch.cuda.get_device_properties(0).total_memory < 100 << 30:
        pytest.skip("less than 100 GB")
    import __graft_entry__
    __graft_entry__.build()
    yield
    torch.cuda.empty_cache()


def rnd(*shape, std=1.0):
    # a tile of random rows, repeated: filling all of it at random takes longer than the tests
    g = torch.Generator(device="cuda").manual_seed(shape[-1])
    rows = 1
    for s in shape[:-1]:
        rows *= s
    t = torch.randn(min(rows, 1009), shape[-1], generator=g, device="cuda").mul_(std).bfloat16()
    return t[torch.arange(rows, device="cuda") % t.shape[0]].view(shape)


def close(got, ref, tol):
    assert ((got.double() - ref).abs() <= tol).all(), float((got.double() - ref).abs().max())


def spots(n, per):
    """First, last and those around element 2^31 of n things of `per` elements."""
    mid = 2 ** 31 // per
    assert 0 < mid < n - 1
    return [0, mid - 1, mid, mid + 1, n - 1]


@pytest.mark.parametrize("dx", [False, True])
@pytest.mark.parametrize("groups", [2, 256])
def test_grouped_rows(groups, dx):
    # 256 groups: rows as columns of the tile (few rows); 2: as its rows
    rows, wide, k = (40000, 54000, 520) if groups == 256 else (270000, 8200, 64)
    w = rnd(groups, k, wide, std=0.1) if dx else rnd(groups, wide, k, std=0.1)
    x = rnd(rows, k)
    off = torch.linspace(0, rows, groups + 1, dtype=torch.float64).int().cuda()
    shape = L.make_grouped_shape(rows, groups, k if dx else wide, wide if dx else k)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    y = torch.empty(rows, wide, dtype=torch.bfloat16, device="cuda")
    (L.moe_grouped_matmul_dx if dx else L.moe_grouped_matmul)(shape, x, off, w, y, ws)
    for r in spots(rows, wide):
        g = int((off[1:] <= r).sum())
        wg = w[g].double() if dx else w[g].double().T
        ref, mag = x[r].double() @ wg, x[r].double().abs() @ wg.abs()
        close(y[r], ref, (k + 2) * 2 * U * mag + HALF_BF16 * ref.abs())
    assert L.moe_read_status(ws) == 0


def test_grouped_input_and_matrices():
    """The reduction's operands are the large ones."""
    rows, k, n, groups = 262200, 8200, 64, 2
    x, w = rnd(rows, k), rnd(groups, n, k, std=0.1)
    off = torch.tensor([0, 1000, rows], dtype=torch.int32, device="cuda")
    shape = L.make_grouped_shape(rows, groups, n, k)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    y = torch.empty(rows, n, dtype=torch.bfloat16, device="cuda")
    L.moe_grouped_matmul(shape, x, off, w, y, ws)
    for r in spots(rows, k):
        wg = w[0 if r < 1000 else 1].double().T
        ref, mag = x[r].double() @ wg, x[r].double().abs() @ wg.abs()
        close(y[r], ref, (k + 2) * 2 * U * mag + HALF_BF16 * ref.abs())
    # the weight gradient over its last 100 rows
    off = torch.tensor([rows - 100, rows - 100, rows], dtype=torch.int32, device="cuda")
    dy = rnd(rows, n)
    dw = torch.empty(groups, n, k, dtype=torch.bfloat16, device="cuda")
    L.moe_grouped_matmul_dw(shape, dy, x, off, dw, ws)
    a, b = dy[-100:].double().T, x[-100:].double()
    ref = a @ b
    close(dw[1], ref, 102 * 2 * U * (a.abs() @ b.abs()) + HALF_BF16 * ref.abs())
    assert (dw[0] == 0).all()
    assert L.moe_read_status(ws) == 0


def test_grouped_weight_gradient():
    groups, n, k, per = 66, 8192, 4104, 24
    x, dy = rnd(groups * per, k), rnd(groups * per, n)
    off = (torch.arange(groups + 1, device="cuda") * per).int()
    shape = L.make_grouped_shape(groups * per, groups, n, k, flags=L.MOE_GROUPED_DW_F32)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    dw = torch.empty(groups, n, k, device="cuda")
    L.moe_grouped_matmul_dw(shape, dy, x, off, dw, ws)
    for g in spots(groups, n * k):
        a, b = dy[g * per:(g + 1) * per].double().T, x[g * per:(g + 1) * per].double()
        close(dw[g], a @ b, (per + 2) * 2 * U * (a.abs() @ b.abs()))
    assert L.moe_read_status(ws) == 0


def test_grouped_f32():
    rows, k, n, groups = 270000, 16, 8200, 3
    x, w = rnd(rows, k).float(), rnd(groups, n, k).float()
    off = torch.tensor([0, 5, 100000, rows], dtype=torch.int32, device="cuda")
    shape = L.make_grouped_shape(rows, groups, n, k, L.MOE_DTYPE_F32)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    y = torch.empty(rows, n, device="cuda")
    L.moe_grouped_matmul(shape, x, off, w, y, ws)
    for r in spots(rows, n):
        g = int((off[1:] <= r).sum())
        wg = w[g].double().T
        close(y[r], x[r].double() @ wg, (k + 2) * U * (x[r].double().abs() @ wg.abs()))


def test_grouped_f32_few_rows():
    groups, n, k = 66, 8192, 4104
    w = rnd(groups, n, k).float()
    x, dy = rnd(groups, k).float(), rnd(groups, n).float()
    off = torch.arange(groups + 1, device="cuda").int()
    shape = L.make_grouped_shape(groups, groups, n, k, L.MOE_DTYPE_F32)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    y, dx, dw = torch.empty_like(dy), torch.empty_like(x), torch.empty_like(w)
    L.moe_grouped_matmul(shape, x, off, w, y, ws)
    L.moe_grouped_matmul_dx(shape, dy, off, w, dx, ws)
    L.moe_grouped_matmul_dw(shape, dy, x, off, dw, ws)
    for g in spots(groups, n * k):
        wg, xg, dg = w[g].double(), x[g].double(), dy[g].double()
        close(y[g], wg @ xg, (k + 2) * U * (wg.abs() @ xg.abs()))
        close(dx[g], dg @ wg, (n + 2) * U * (dg.abs() @ wg.abs()))
        close(dw[g], torch.outer(dg, xg), 2 * U * torch.outer(dg, xg).abs())


def test_swiglu():
    rows, inter = 300000, 4096  # gu passes 2^31 elements, and 2^32 bytes
    gu, da = rnd(rows, 2 * inter), rnd(rows, inter)
    sw = L.make_swiglu_shape(rows, inter)
    a, dgu = torch.empty_like(da), torch.empty_like(gu)
    L.moe_swiglu(sw, gu, a)
    L.moe_swiglu_backward(sw, gu, da, dgu)
    for r in spots(rows, 2 * inter):
        t = gu[r].double().view(-1, 2, 64).requires_grad_()
        ref = torch.nn.functional.silu(t[:, 0]) * t[:, 1]
        close(a[r], ref.detach().reshape(-1), 64 * U * t.detach().abs().amax() ** 2
              + HALF_BF16 * ref.detach().abs().reshape(-1))
        ref.backward(da[r].double().view(-1, 64))
        want = t.grad.reshape(-1)
        scale = da[r].double().abs().max() * (t.detach().abs().max() + 1) ** 2
        close(dgu[r], want, 64 * U * scale + HALF_BF16 * want.abs())


def test_layer_norm():
    T, d = 530000, 4100
    x, dy = rnd(T, d), rnd(T, d, std=0.5)
    gamma, beta = rnd(1, d)[0].float(), rnd(1, d)[0].float()
    nm = L.make_norm_shape(T, d)
    y, dx = torch.empty_like(x), torch.empty_like(x)
    mean, rstd = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    dg, db = torch.empty_like(gamma), torch.empty_like(beta)
    wn = torch.empty(L.moe_layer_norm_workspace_size(nm), dtype=torch.uint8, device="cuda")
    L.moe_layer_norm(nm, x, gamma, beta, y, mean, rstd)
    L.moe_layer_norm_backward(nm, dy, x, gamma, mean, rstd, dx, dg, db, wn)
    for r in spots(T, d):
        t = x[r].double().requires_grad_()
        ref = torch.nn.functional.layer_norm(t, (d,), gamma.double(), beta.double(), 1e-5)
        # the sums' d terms and a dozen operations in fp32
        slack = (d + 12) * U
        close(y[r], ref.detach(), slack * (ref.detach().abs() + gamma.abs().max())
              + HALF_BF16 * ref.detach().abs())
        ref.backward(dy[r].double())
        big = (dy[r].double() * gamma.double()).abs().max() * 8
        close(dx[r], t.grad, slack * big + HALF_BF16 * t.grad.abs())


def test_orthogonalize():
    """Small matrices, then ones past the on-chip kernel, each copies of 5."""
    for n, r, c in ((65535, 128, 260), (7000, 256, 1240)):
        base = rnd(5, r, c)
        m = base[torch.arange(n, device="cuda") % 5]
        sh = L.make_ortho_shape(n, r, c, steps=1)
        ws = torch.zeros(L.moe_orthogonalize_workspace_size(sh), dtype=torch.uint8, device="cuda")
        o = torch.empty_like(m)
        L.moe_orthogonalize(sh, m, o, ws)
        x = base.double()
        x = x / (x.flatten(1).norm(dim=1)[:, None, None] + 1e-7)
        a = x @ x.mT
        want = 3.4445 * x + (-4.7750 * a + 2.0315 * a @ a) @ x
        for i in spots(n, r * c):
            # the documented 2e-3 of the norm
            assert (o[i].double() - want[i % 5]).norm() <= 2e-3 * want[i % 5].norm()
        assert L.moe_read_status(ws) == 0
        del m, o, ws
