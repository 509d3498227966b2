"""Embedding lookup and the gradient of its table against plain definitions.

The lookup is one fp32 product rounded once: equal bit for bit to torch's.  The
gradient of a row is an fp32 sum of its c entries and one product: its error is
at most (c + 1) 2^-24 |scale| sum |dy|.  A bf16 gradient is that fp32 value,
rounded: equal bit for bit to the fp32 gradient's rounding."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"
IO = {"bf16": torch.bfloat16, "f32": torch.float32}


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("n,rows,dim", [(1, 1, 1), (7, 5, 3), (300, 100, 64), (1000, 37, 100),
                                        (65, 1000, 769), (2, 9, 5000), (4097, 50, 8), (33, 4, 7)])
def test_lookup(gpu, n, rows, dim, io):
    g = gen(n)
    w = torch.randn(rows, dim, generator=g, device=DEV).to(IO[io])
    ids = torch.randint(0, rows, (n,), generator=g, device=DEV)
    for scale in (1.0, 27.7):
        want = (w.float() * scale).to(IO[io])[ids]
        assert torch.equal(gpu.embed_fwd(ids, w, scale=scale), want)
        assert torch.equal(gpu.embed_fwd(ids.int(), w, scale=scale), want)
    bad = ids.clone()
    bad[0], bad[n // 2], bad[n - 1] = -1, rows, 1 << 40
    out = gpu.embed_fwd(bad, w, out=torch.full((n, dim), float("nan"), device=DEV, dtype=IO[io]))
    want = w[bad.clamp(0, rows - 1)]
    want[(bad < 0) | (bad >= rows)] = 0
    assert torch.equal(out, want)


def check_grad(gpu, ids, dy, rows, scale=1.0, padding=-1, grad_dtype=None):
    flat, d2 = ids.reshape(-1).cpu().long(), dy.reshape(-1, dy.shape[-1]).cpu().double()
    keep = (flat >= 0) & (flat < rows) & (flat != padding)
    want = torch.zeros(rows, dy.shape[-1], dtype=torch.float64)
    size = torch.zeros_like(want)
    want.index_add_(0, flat[keep], d2[keep])
    size.index_add_(0, flat[keep], d2[keep].abs())
    count = torch.bincount(flat[keep], minlength=rows).double().unsqueeze(1)
    want *= scale
    got = gpu.embed_bwd(ids, dy, rows, scale=scale, padding=padding, grad_dtype=grad_dtype,
                        dweight=torch.full((rows, dy.shape[-1]), float("nan"), device=DEV,
                                           dtype=grad_dtype or dy.dtype))
    lim = (count + 1) * 2.0 ** -24 * abs(scale) * size
    if got.dtype == torch.bfloat16:
        wide = gpu.embed_bwd(ids, dy, rows, scale=scale, padding=padding,
                             grad_dtype=torch.float32)
        assert torch.equal(got, wide.bfloat16())
        got = wide
    err = (got.cpu().double() - want).abs()
    assert (err <= lim).all(), float((err / lim.clamp_min(1e-300)).max())
    assert torch.equal(got[(count == 0).squeeze(1).to(DEV)],
                       torch.zeros_like(got[(count == 0).squeeze(1).to(DEV)]))
    return got


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("n,rows,dim", [(1, 1, 1), (5, 3, 2), (31, 40, 8), (32, 7, 33), (33, 1, 64),
                                        (1000, 17, 100), (2048, 2000, 24), (2049, 9, 16),
                                        (9000, 600, 40), (70000, 300, 12), (600, 300000, 9),
                                        (64, 5, 2500), (16384, 5000, 8), (16385, 5000, 8),
                                        (20000, 300000, 3), (17000, 1, 100)])
def test_gradient(gpu, n, rows, dim, io):
    g = gen(n + rows)
    dy = torch.randn(n, dim, generator=g, device=DEV).to(IO[io])
    # a few tokens hold much of the batch
    ids = (rows * torch.rand(n, generator=g, device=DEV) ** 6).long().clamp(0, rows - 1)
    check_grad(gpu, ids, dy, rows, scale=3.5)
    check_grad(gpu, ids.int(), dy, rows, padding=int(ids[0]), grad_dtype=torch.float32)
    check_grad(gpu, ids, dy, rows, grad_dtype=torch.bfloat16)


@pytest.mark.parametrize("n", [32, 33, 64, 100, 127, 128, 129, 5000, 6144, 6145, 30000])
def test_runs_across_workgroups(gpu, n):
    g = gen(n)
    dy = torch.randn(n, 20, generator=g, device=DEV)
    same = torch.full((n,), 3, device=DEV)
    check_grad(gpu, same, dy, 7)
    check_grad(gpu, torch.arange(n, device=DEV) // 31, dy, n // 31 + 2)
    check_grad(gpu, torch.arange(n, device=DEV).flip(0), dy, n)
    check_grad(gpu, torch.arange(n, device=DEV) % 2 * (n - 1), dy, n)


@pytest.mark.parametrize("n", [1, 2, 63, 64, 65, 128, 130, 200, 256, 257])
@pytest.mark.parametrize("dim", [1, 3, 5, 8, 100, 1030])
def test_few_entries(gpu, n, dim):
    """Rows that start and end inside a 16-byte vector, beside zeros; tokens that
    occur again; first, last and neighbouring rows; ids without a row."""
    g = gen(n * dim)
    dy = torch.randn(n, dim, generator=g, device=DEV)
    rows = 301
    ids = torch.randint(-2, rows + 2, (n,), generator=g, device=DEV)
    ids[0] = rows - 1
    ids[n // 2:n // 2 + 3] = torch.arange(3, device=DEV)[:max(min(3, n - n // 2), 0)]
    ids[n - 1] = ids[0]
    check_grad(gpu, ids, dy, rows, scale=0.3)
    check_grad(gpu, ids, dy.bfloat16(), rows, padding=1)
    check_grad(gpu, ids.int(), dy.bfloat16(), rows, grad_dtype=torch.float32)
    check_grad(gpu, torch.full_like(ids, 1), dy, 3, grad_dtype=torch.bfloat16)


def test_ignored_ids_and_shapes(gpu):
    g = gen(5)
    ids = torch.randint(-3, 14, (4, 50), generator=g, device=DEV)
    ids[0, 0], ids[3, 49] = 1 << 40, -(1 << 40)
    dy = torch.randn(4, 50, 48, generator=g, device=DEV)
    check_grad(gpu, ids, dy, 10, padding=4)
    check_grad(gpu, torch.full_like(ids, 99), dy, 10)  # nothing in the table
    assert gpu.embed_fwd(ids, torch.ones(10, 48, device=DEV)).shape == (4, 50, 48)
    none = torch.empty(0, dtype=torch.int64, device=DEV)
    assert gpu.embed_fwd(none, torch.ones(10, 48, device=DEV)).shape == (0, 48)
    got = gpu.embed_bwd(none, torch.empty(0, 48, device=DEV), 10,
                        dweight=torch.ones(10, 48, device=DEV))
    assert torch.equal(got, torch.zeros_like(got))


def test_sums_in_order_and_repeats(gpu):
    """Entries of a token are added in the order of their positions: 2^24, then
    ones that fp32 cannot add to it one by one."""
    dy = torch.ones(20, 4, device=DEV)
    dy[0] = 2.0 ** 24
    ids = torch.zeros(20, dtype=torch.int64, device=DEV)
    got = gpu.embed_bwd(ids, dy, 2)
    assert torch.equal(got[0], torch.full((4,), 2.0 ** 24, device=DEV))
    g = gen(9)
    ids = (200 * torch.rand(50000, generator=g, device=DEV) ** 5).long()
    dy = torch.randn(50000, 72, generator=g, device=DEV)
    first = gpu.embed_bwd(ids, dy, 200)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (None, side, side.cuda_stream):
        again = gpu.embed_bwd(ids, dy, 200, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(again, first)


def test_in_a_graph(gpu):
    g = gen(10)
    ids = torch.randint(0, 500, (6000,), generator=g, device=DEV)
    dy = torch.randn(6000, 40, generator=g, device=DEV)
    w = torch.randn(500, 40, generator=g, device=DEV)
    ws = torch.empty(gpu.embed_bwd_workspace_bytes(6000, 500, 40, gpu.MS_F32), dtype=torch.uint8,
                     device=DEV)
    out, dw = torch.empty(6000, 40, device=DEV), torch.empty(500, 40, device=DEV)

    def call():
        gpu.embed_fwd(ids, w, scale=2.0, out=out)
        gpu.embed_bwd(ids, dy, 500, scale=2.0, dweight=dw, workspace=ws)

    call()
    torch.cuda.synchronize()
    o, d = out.clone(), dw.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for rep in range(3):
        out.fill_(float("nan"))
        dw.fill_(float("nan"))
        ws.fill_(0xa5 + rep)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, o) and torch.equal(dw, d), rep
        call()
        torch.cuda.synchronize()


def test_autograd(gpu):
    g = gen(12)
    w = torch.randn(30, 16, generator=g, device=DEV, requires_grad=True)
    ids = torch.randint(0, 30, (3, 40), generator=g, device=DEV)
    dy = torch.randn(3, 40, 16, generator=g, device=DEV)
    (gpu.embed(ids, w, padding=2) * dy).sum().backward()
    want = torch.zeros(30, 16, dtype=torch.float64)
    want.index_add_(0, ids.reshape(-1).cpu(), dy.reshape(-1, 16).cpu().double() * 4.0)
    want[2] = 0
    assert (w.grad.cpu().double() - want).abs().max() <= 1e-4


def test_refusals(gpu):
    w = torch.zeros(10, 8, device=DEV)
    ids = torch.zeros(4, dtype=torch.int64, device=DEV)
    with pytest.raises(TypeError, match="int32 or int64"):
        gpu.embed_fwd(ids.float(), w)
    with pytest.raises(TypeError):
        gpu.embed_fwd(ids, w.half())
    with pytest.raises(ValueError, match="device"):
        gpu.embed_fwd(ids, w.cpu())
    with pytest.raises(ValueError, match="device"):
        gpu.embed_fwd(ids.cpu(), w)
    with pytest.raises(ValueError, match="contiguous"):
        gpu.embed_fwd(ids, torch.zeros(8, 10, device=DEV).t())
    with pytest.raises(gpu.MsError, match="scale"):
        gpu.embed_fwd(ids, w, scale=float("inf"))
    with pytest.raises(ValueError, match="shape"):
        gpu.embed_bwd(ids, torch.zeros(5, 8, device=DEV), 10)
    with pytest.raises(TypeError, match="grad_dtype"):
        gpu.embed_bwd(ids, torch.zeros(4, 8, device=DEV), 10, grad_dtype=torch.float16)
    with pytest.raises(gpu.MsError):
        gpu.embed_bwd(ids, torch.zeros(4, 8, device=DEV), 0)
    ids = torch.zeros(4000, dtype=torch.int64, device=DEV)  # a few need no workspace
    with pytest.raises(gpu.MsError, match="workspace"):
        gpu.embed_bwd(ids, torch.zeros(4000, 8, device=DEV), 10,
                      workspace=torch.empty(16, dtype=torch.uint8, device=DEV))


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("n", [50, 7000])
def test_ids_and_gradients_off_16_bytes(gpu, n, io):
    """ids after the first of a text, and gradients as torch.cat hands them on:
    contiguous, aligned to their element."""
    g = gen(n)
    text = torch.randint(0, 90, (n + 1,), generator=g, device=DEV)
    dy = torch.randn(n * 37 + 1, generator=g, device=DEV).to(IO[io])[1:].view(n, 37)
    w = torch.randn(90, 37, generator=g, device=DEV).to(IO[io])
    for ids in (text[1:], text.int()[1:]):
        assert ids.data_ptr() % 16 and dy.data_ptr() % 16
        assert torch.equal(gpu.embed_fwd(ids, w), w[ids.long()])
        assert torch.equal(gpu.embed_bwd(ids, dy, 90), gpu.embed_bwd(ids.clone(), dy.clone(), 90))
    one = w.clone().requires_grad_()
    up = torch.randn(n + 3, 37, generator=g, device=DEV).to(IO[io])
    (torch.cat([gpu.embed(text[:3], one), gpu.embed(text[1:], one)]) * up).sum().backward()
    want = gpu.embed_bwd(text[:3].clone(), up[:3].clone(), 90, scale=37 ** 0.5) + \
        gpu.embed_bwd(text[1:].clone(), up[3:].clone(), 90, scale=37 ** 0.5)
    assert torch.equal(one.grad, want)


def test_autograd_takes_slices_of_a_token_tensor(gpu):
    g = gen(14)
    tokens = torch.randint(0, 30, (4, 41), generator=g, device=DEV)
    dy = torch.randn(4, 40, 16, generator=g, device=DEV)
    grads = []
    for ids in (tokens[:, :-1], tokens[:, :-1].contiguous()):
        w = torch.randn(30, 16, generator=gen(15), device=DEV, requires_grad=True)
        gpu.embed(ids, w).backward(dy)
        grads.append(w.grad)
    assert torch.equal(*grads)
