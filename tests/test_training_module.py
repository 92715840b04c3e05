"""training.py: the experts' and the norm's steps as a training program takes
them, against autograd in float64, and their argument checks."""
import pytest
import torch

from mixture_experts_layer_56_b200 import _lib as L


def test_checks_before_any_call():
    from mixture_experts_layer_56_b200 import training as TR
    w13, w2 = torch.zeros(2, 128, 16), torch.zeros(2, 16, 64)
    with pytest.raises(ValueError):
        TR.TrainableExperts(w13, w2.transpose(1, 2))
    with pytest.raises(ValueError):
        TR.TrainableExperts(w13.double(), w2.double())
    with pytest.raises(ValueError):
        TR.TrainableExperts(torch.zeros(2, 96, 16), torch.zeros(2, 16, 48))
    ex = TR.TrainableExperts(w13, w2)
    off = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError):
        ex.forward(torch.zeros(4, 8), off)
    with pytest.raises(ValueError):
        ex.forward(torch.zeros(4, 16).bfloat16(), off)
    with pytest.raises(ValueError):
        ex.forward(torch.zeros(4, 16), off.long())
    with pytest.raises(ValueError):
        ex.forward(torch.zeros(4, 32)[:, ::2], off)
    with pytest.raises(ValueError):
        ex.forward(torch.zeros(4, 16), off)      # not on a GPU
    with pytest.raises(RuntimeError):
        ex.backward(torch.zeros(4, 16))
    with pytest.raises(ValueError):
        TR.LayerNorm(torch.ones(8).bfloat16())
    with pytest.raises(ValueError):
        TR.LayerNorm(torch.ones(8), torch.ones(7))
    nm = TR.LayerNorm(torch.ones(8))
    with pytest.raises(ValueError):
        nm.forward(torch.zeros(3, 9))
    with pytest.raises(ValueError):
        nm.forward(torch.zeros(3, 8))
    with pytest.raises(ValueError):
        TR.orthogonalize(torch.zeros(1, 3, 8))
    with pytest.raises(RuntimeError):
        nm.backward(torch.zeros(3, 8))
    with pytest.raises(ValueError):
        TR.orthogonalize(torch.zeros(3, 8))


@pytest.fixture(scope="module")
def TR():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    from mixture_experts_layer_56_b200 import training
    return training


def expert_ref(x, off, w13, w2):
    """FFN_g of each group's rows, packed W13."""
    inter = w2.shape[2]
    ys = []
    for g in range(w13.shape[0]):
        gu = (x[off[g]:off[g + 1]] @ w13[g].T).view(-1, inter // 64, 2, 64)
        a = torch.nn.functional.silu(gu[:, :, 0]) * gu[:, :, 1]
        ys.append(a.reshape(-1, inter) @ w2[g].T)
    return torch.cat(ys)


# Relative to the gradient's norm.  fp32: every product sums at most 300 terms
# in a chain, four products deep, each term off by half a step (2^-24): 1200
# half steps at the very most.  bf16: six roundings of half a step (2^-8) each
# between the input and any gradient.
TOL = {torch.float32: 1200 * 2.0 ** -24, torch.bfloat16: 6 * 2.0 ** -8}


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_experts_and_norm_against_autograd(TR, dtype):
    g = torch.Generator(device="cuda").manual_seed(5)

    def rand(*s, std=1.0, dt=dtype):
        return (torch.randn(*s, device="cuda", generator=g) * std).to(dt)

    n, d, inter = 5, 72, 128
    w13, w2 = rand(n, 2 * inter, d, std=d ** -0.5), rand(n, d, inter, std=inter ** -0.5)
    gamma, beta = 1 + 0.1 * rand(d, dt=torch.float32), rand(d, dt=torch.float32)
    ex, nm = TR.TrainableExperts(w13, w2), TR.LayerNorm(gamma, beta)
    leaf = {k: t.double().requires_grad_() for k, t in
            dict(w13=w13, w2=w2, gamma=gamma, beta=beta).items()}
    # two backward passes: the weights' gradients add up
    for sizes in ([40, 0, 133, 1, 90], [0, 64, 3, 200, 0]):
        off = [0]
        for s in sizes:
            off.append(off[-1] + s)
        offsets = torch.tensor(off, dtype=torch.int32, device="cuda")
        u, dy = rand(off[-1], d), rand(off[-1], d)
        y = ex.forward(nm.forward(u), offsets)
        du = nm.backward(ex.backward(dy))
        leaf["gamma"].grad = leaf["beta"].grad = None  # the norm's are overwritten
        ud = u.double().requires_grad_()
        ref = expert_ref(torch.nn.functional.layer_norm(ud, (d,), leaf["gamma"], leaf["beta"], 1e-5),
                         off, leaf["w13"], leaf["w2"])
        ref.backward(dy.double())
        for name, got, want in (("y", y, ref), ("du", du, ud.grad),
                                ("dgamma", nm.dgamma, leaf["gamma"].grad),
                                ("dbeta", nm.dbeta, leaf["beta"].grad),
                                ("dW13", ex.dW13, leaf["w13"].grad), ("dW2", ex.dW2, leaf["w2"].grad)):
            rel = float((got.double() - want).norm() / want.norm())
            assert rel <= TOL[dtype], (name, rel)
    kept = ex.dW2.clone()
    ex.zero_grad()
    ex.forward(rand(10, d), torch.tensor([0, 10, 10, 10, 10, 10], dtype=torch.int32, device="cuda"))
    ex.backward(rand(10, d))
    assert (ex.dW2[1:] == 0).all() and not torch.equal(ex.dW2[0], kept[0])
    with pytest.raises(RuntimeError):
        ex.backward(rand(10, d))
    assert ex.status() == 0


@pytest.mark.gpu
def test_update_of_the_packed_matrix_is_that_of_its_halves(TR):
    """orthogonalize(packed W13) unpacks to orthogonalize([W1; W3])."""
    g = torch.Generator(device="cuda").manual_seed(6)
    inter, d = 128, 200
    w1, w3 = (torch.randn(1, inter, d, device="cuda", generator=g) for _ in range(2))
    packed = torch.stack([w1.view(1, -1, 64, d), w3.view(1, -1, 64, d)], 2).reshape(1, 2 * inter, d)
    a = TR.orthogonalize(packed.contiguous()).view(1, -1, 2, 64, d)
    b = TR.orthogonalize(torch.cat([w1, w3], 1)).view(1, 2, inter, d)
    got = torch.stack([a[:, :, 0].reshape(1, inter, d), a[:, :, 1].reshape(1, inter, d)], 1)
    # the same sums in another order: both are within the operator's own
    # tolerance (2^-8 + 24 x 2^-11, relative) of one exact value
    assert float((got.double() - b.double()).norm() / b.double().norm()) <= 2 * (2.0 ** -8 + 24 * 2.0 ** -11)


@pytest.mark.gpu
def test_a_layer_step_with_the_norm_and_its_gradient(TR):
    """norm, route, dispatch, experts, combine and back: the step of the
    module's docstring, the router's gates held fixed."""
    g = torch.Generator(device="cuda").manual_seed(7)
    T, d, n, inter, k = 96, 128, 8, 64, 2
    bf = torch.bfloat16

    def rand(*s, std=1.0, dt=bf):
        return (torch.randn(*s, device="cuda", generator=g) * std).to(dt)

    u, E = rand(T, d), rand(n, d, std=d ** -0.5)
    w13, w2 = rand(n, 2 * inter, d, std=d ** -0.5), rand(n, d, inter, std=inter ** -0.5)
    ex, nm = TR.TrainableExperts(w13, w2), TR.LayerNorm(torch.ones(d, device="cuda"))
    shape = L.make_shape(T, d, n, 0, inter, k)
    ws = torch.zeros(L.moe_workspace_size(shape), dtype=torch.uint8, device="cuda")
    i32 = lambda *s: torch.empty(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    idx, w = i32(T, k), torch.empty(T, k, device="cuda")
    counts, offsets, perm, inv = i32(n), i32(n + 1), i32(T * k), i32(T * k)
    x = nm.forward(u)
    L.moe_route(shape, x, E, None, idx, w)
    L.moe_dispatch(shape, idx, counts, offsets, perm, inv, ws)
    rows = x[(perm // k).long()].contiguous()
    y = ex.forward(rows, offsets)
    h, none = torch.empty_like(u), torch.zeros(T, d, device="cuda")
    L.moe_combine(shape, u, none, y, w, inv, h)
    dh = rand(T, d)
    dy = (w.view(-1)[perm.long()][:, None] * dh[(perm // k).long()].float()).to(bf)
    dx_rows = ex.backward(dy)
    # a token's rows add up as the combine adds them, with gates of one
    dx = torch.empty_like(u)
    zero = torch.zeros_like(u)
    L.moe_combine(shape, zero, none, dx_rows, torch.ones_like(w), inv, dx)
    du = nm.backward(dx)
    ud = u.double().requires_grad_()
    xd = torch.nn.functional.layer_norm(ud, (d,), eps=1e-5)
    hd = ud.clone()
    yd = expert_ref(xd[(perm // k).long()], offsets.tolist(), w13.double(), w2.double())
    hd = hd.index_add(0, (perm // k).long(), w.double().view(-1)[perm.long()][:, None] * yd)
    hd.backward(dh.double())
    # nine roundings of half a bf16 step at most on the way, the residual's
    # gradient apart
    assert float((h.double() - hd).norm() / hd.norm()) <= 6 * 2.0 ** -8
    want = ud.grad - dh.double()
    assert float((du.double() - want).norm() / want.norm()) <= 9 * 2.0 ** -8


def _steps(TR):
    """A forward and backward of the norm and the experts, and an update, over
    the same inputs: a function of the stream."""
    g = torch.Generator(device="cuda").manual_seed(23)

    def rnd(*s, scale=1.0):
        return (torch.randn(*s, generator=g, device="cuda") * scale).bfloat16()

    w13, w2 = rnd(4, 512, 192, scale=0.1), rnd(4, 192, 256, scale=0.1)
    gamma, beta = rnd(192).float(), rnd(192).float()
    u, dy, m = rnd(600, 192), rnd(600, 192), rnd(2, 200, 300)
    off = torch.tensor([0, 100, 100, 450, 600], dtype=torch.int32, device="cuda")

    def run(stream=None):
        ex, nm = TR.TrainableExperts(w13, w2), TR.LayerNorm(gamma, beta)
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(stream):
                torch.cuda._sleep(200_000_000)  # some 100 ms: what follows runs late
        x = nm.forward(u, stream=stream)
        y = ex.forward(x, off, stream=stream)
        dx = ex.backward(dy, stream=stream)
        du = nm.backward(dx, stream=stream)
        o = TR.orthogonalize(m, stream=stream)
        return [y, dx, du, o, ex.dW13, ex.dW2, nm.dgamma, nm.dbeta], (ex, nm)

    return run


@pytest.mark.gpu
def test_a_stream_of_its_own_keeps_its_temporaries(TR):
    """What the calls allocate for themselves belongs to the stream they run
    on: the current stream neither gets that memory while they run, nor do they
    write into what it got."""
    run = _steps(TR)
    want, _ = run()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()

    def fill():
        # every size that the calls allocate
        return ([torch.full((600, c), 7.0, dtype=torch.bfloat16, device="cuda")
                 for c in (192, 256, 512) for _ in range(8)]
                + [torch.full((n,), 255, dtype=torch.uint8, device="cuda")
                   for n in (2400, 1 << 14, 1 << 17, 1 << 20, 1 << 21) for _ in range(4)])

    fill()  # its kernels are loaded, its memory is in the pool
    torch.cuda.synchronize()
    got, keep = run(side)
    late = not side.query()
    junk = fill()
    assert late, "the side stream was done before the current one could get in its way"
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    for t in junk:
        assert (t == (7.0 if t.is_floating_point() else 255)).all()
    assert keep[0].status() == 0


@pytest.mark.gpu
def test_backward_on_another_stream_than_its_forward(TR):
    u = torch.randn(8, 64, device="cuda")
    nm = TR.LayerNorm(torch.ones(64, device="cuda"))
    nm.forward(u)
    with pytest.raises(ValueError, match="stream"):
        nm.backward(u, stream=torch.cuda.Stream())
    nm.backward(u)  # and the forward is still there
    ex = TR.TrainableExperts(torch.ones(1, 128, 64, device="cuda"),
                             torch.ones(1, 64, 64, device="cuda"))
    off = torch.tensor([0, 8], dtype=torch.int32, device="cuda")
    ex.forward(u, off)
    with pytest.raises(ValueError, match="stream"):
        ex.backward(u, stream=torch.cuda.Stream().cuda_stream)
    ex.backward(u)
    torch.cuda.synchronize()
