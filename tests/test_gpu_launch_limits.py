"""Row and chunk counts whose threads no single launch can hold (2^32 per grid
dimension): the calls around the projection answer them like any other."""
import ctypes

import pytest

from tests.gpu_util import announce, torch_cuda

pytestmark = pytest.mark.gpu


def test_norm_of_2_24_rows():
    torch = torch_cuda()
    import w8a8_integer_linear_amd as qlin
    rows, cols = (1 << 24) + 3, 16
    announce("rmsnorm_quant", rows, cols)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((rows, cols), generator=g, device="cuda").to(torch.bfloat16)
    res = torch.randn((rows, cols), generator=g, device="cuda").to(torch.bfloat16)
    gamma = torch.rand(cols, generator=g, device="cuda") + 0.5
    got = qlin.qlin_rmsnorm_quant(x, gamma, 1e-6, residual=res, had_block=16, want_y=True)
    step = 5_000_000        # (pieces that do not end where a launch may)
    for at in range(0, rows, step):
        part = slice(at, min(rows, at + step))
        want = qlin.qlin_rmsnorm_quant(x[part], gamma, 1e-6, residual=res[part], had_block=16,
                                       want_y=True)
        for a, b in zip(got, want):
            assert torch.equal(a[part], b)


def test_norm_backward_of_2_22_long_rows():
    """(69 GB each for h, which serves as dn too, and dh.)"""
    torch = torch_cuda()
    import w8a8_integer_linear_amd as qlin
    rows, cols = (1 << 22) + 3, 8208
    if torch.cuda.mem_get_info()[0] < 180 << 30:
        pytest.skip("needs 180 GB of the card's memory")
    announce("rmsnorm_bwd", rows, cols)
    g = torch.Generator(device="cuda").manual_seed(1)
    piece = torch.randn((1 << 14, cols), generator=g, device="cuda").to(torch.bfloat16)
    h = torch.empty((rows, cols), dtype=torch.bfloat16, device="cuda")
    rstd = torch.empty(rows, device="cuda")
    for at in range(0, rows, 1 << 14):
        n = min(1 << 14, rows - at)
        h[at:at + n] = piece[:n]
        rstd[at:at + n] = torch.rand(n, generator=g, device="cuda") + 0.5
    gamma = torch.rand(cols, generator=g, device="cuda") + 0.5
    dh, dgamma = qlin.qlin_rmsnorm_bwd(h, h, rstd, gamma)
    for at in (0, (1 << 21) - 5, 1 << 21, (1 << 22) - 5, rows - 5):
        part = h[at:at + 5]
        want, _ = qlin.qlin_rmsnorm_bwd(part, part, rstd[at:at + 5].clone(), gamma)
        assert torch.equal(dh[at:at + 5], want)
    # The sum over the rows, whose pieces repeat: terms of one sign, added by 64
    # runs of rows one after another and then the 64.
    scale = torch.zeros(1 << 14, dtype=torch.float64, device="cuda")
    for at in range(0, rows, 1 << 14):
        n = min(1 << 14, rows - at)
        scale[:n] += rstd[at:at + n]
    want = (piece.double().square() * scale[:, None]).sum(0)
    assert ((dgamma - want).abs() <= want * (rows / 64 + 64 + 4) * 2.0 ** -24).all()
    del h, dh
    torch.cuda.empty_cache()


def test_adamw_of_2_24_chunks():
    """A list of 2^24 + 3 chunks.  The image says so by hand: its second tensor has
    the last chunk, its first one all the others, of which only the first lies
    within the memory that the first tensor's size admits."""
    torch = torch_cuda()
    import w8a8_integer_linear_amd as qlin
    from w8a8_integer_linear_amd import _native
    chunks = (1 << 24) + 3
    announce("adamw_tensors", chunks)
    g = torch.Generator(device="cuda").manual_seed(1)
    ts = [dict(p=torch.randn(n, generator=g, device="cuda"), g=torch.randn(n, generator=g, device="cuda"),
               m=torch.zeros(n, device="cuda"), v=torch.zeros(n, device="cuda")) for n in (4096, 1000)]
    want = [{k: t.clone() for k, t in d.items()} for d in ts]
    plan, small = qlin.qlin_adamw_tensors_plan(ts), qlin.qlin_adamw_tensors_plan(want)
    image = torch.zeros(2 * 80 + 4 * chunks, dtype=torch.uint8, device="cuda")
    image[:160] = plan.image[:160]
    entry = image[80:160].cpu()
    ctypes.c_int64.from_address(entry.data_ptr() + 64).value = chunks - 1      # its first chunk
    image[80:160] = entry.cuda()
    image[-4:] = torch.tensor([1, 0, 0, 0], dtype=torch.uint8, device="cuda")
    step = (1e-3, 0.9, 0.999, 1e-8, 1, 1)
    _native._check("qlin_adamw_tensors", _native.lib().qlin_adamw_tensors(
        image.data_ptr(), 2, chunks, *step, _native._stream(None)))
    qlin.qlin_adamw_tensors(small, *step)
    for a, b in zip(ts, want):
        for k in "pmv":
            assert torch.equal(a[k], b[k])


def test_few_tokens_of_2_28_outputs():
    """The projection of a few tokens, alone and with adapters, whose outputs are more
    than one launch of the weight-streaming kernel has, against pieces of it."""
    torch = torch_cuda()
    import w8a8_integer_linear_amd as qlin
    M, N, K, R = 2, (1 << 28) + 64, 16, 8
    announce("few tokens", M, N, K)
    g = torch.Generator(device="cuda").manual_seed(1)
    codes = lambda *s: torch.randint(-127, 128, s, generator=g, device="cuda", dtype=torch.int8)  # noqa: E731
    qx, qw = codes(M, K), codes(N, K)
    sx, sw = torch.rand(M, generator=g, device="cuda"), torch.rand(N, generator=g, device="cuda")
    a = torch.randn((1, R, K), generator=g, device="cuda").to(torch.bfloat16)
    b = torch.randn((1, N, R), generator=g, device="cuda", dtype=torch.bfloat16)
    scale, ids = torch.ones(1, device="cuda"), torch.tensor([0, -1], dtype=torch.int32, device="cuda")
    y = qlin.qlin_fwd(qx, sx, qw, sw)
    z, u = qlin.qlin_adapter_fwd(qx, sx, qw, sw, a, b, scale, ids)
    assert torch.equal(y[1], z[1]) and (u[1] == 0).all()
    step = 5_000_000 // 16 * 16
    for at in range(0, N, step):
        part = slice(at, min(N, at + step))
        assert torch.equal(y[:, part], qlin.qlin_fwd(qx, sx, qw[part], sw[part]))
        low = u[:1].double() @ b[0, part].double().T
        size = u[:1].double().abs() @ b[0, part].double().abs().T
        # R products and sums, then the sum with the projection's part
        bound = (R + 8) * 2.0 ** -24 * size + 2.0 ** -23 * (y[:1, part].double().abs() + size)
        assert ((z[:1, part] - (y[:1, part].double() + low)).abs() <= bound).all()


def test_rotation_of_2_35_values():
    """In place, 137 GB; the rows repeat a few."""
    torch = torch_cuda()
    import w8a8_integer_linear_amd as qlin
    rows, cols, piece = (1 << 24) + 1, 2048, 1 << 12
    if torch.cuda.mem_get_info()[0] < 150 << 30:
        pytest.skip("needs 150 GB of the card's memory")
    announce("hadamard", rows, cols)
    x = torch.empty((rows, cols), device="cuda")
    few = torch.randn((piece, cols), generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
    for at in range(0, rows, piece):
        x[at:at + piece] = few[:min(piece, rows - at)]
    qlin.qlin_hadamard(x, 512, y=x)
    want = qlin.qlin_hadamard(few, 512)
    for at in range(0, rows, piece):
        assert torch.equal(x[at:at + piece], want[:min(piece, rows - at)])
    del x
    torch.cuda.empty_cache()


def test_weight_of_2_35_values():
    torch = torch_cuda()
    import w8a8_integer_linear_amd as qlin
    rows, cols, piece = (1 << 24) + 1, 2048, 1 << 12
    if torch.cuda.mem_get_info()[0] < 190 << 30:
        pytest.skip("needs 190 GB of the card's memory")
    announce("dequantize_weight", rows, cols)
    g = torch.Generator(device="cuda").manual_seed(1)
    few = torch.randint(-127, 128, (piece, cols), generator=g, device="cuda", dtype=torch.int8)
    sw = torch.rand(piece, generator=g, device="cuda")
    q, s = torch.empty((rows, cols), dtype=torch.int8, device="cuda"), torch.empty(rows, device="cuda")
    for at in range(0, rows, piece):
        n = min(piece, rows - at)
        q[at:at + n], s[at:at + n] = few[:n], sw[:n]
    for had in (0, 64):
        w = qlin.qlin_dequantize_weight(q, s, had_block=had)
        want = qlin.qlin_dequantize_weight(few, sw, had_block=had)
        for at in range(0, rows, piece):
            assert torch.equal(w[at:at + piece], want[:min(piece, rows - at)])
        del w
    del q
    torch.cuda.empty_cache()
