"""AdamW over many tensors against the formula in 64 bits.

Bounds: every fp32 operation is within 2^-24 of its result's magnitude (2^-22 for
a quotient or a root of approximate instructions); m' and v' take three of them,
the step about eight, of sizes |m'| c1 / d.  An e4m3 code is within half a step
(2^-4 of the value, or 2^-10 below 2^-6) to nearest, within a whole one
stochastically."""
import math

import numpy as np
import pytest

from tests.gpu_util import announce, torch_cuda

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
LR, B1, B2, EPS = 1e-3, 0.9, 0.999, 1e-8
SEED = 0x123456789ABCDEF


def _tensors(torch, sizes, p, g, bits, seed=0):
    kind = {"f32": torch.float32, "bf16": torch.bfloat16}
    gen = torch.Generator().manual_seed(seed)
    rand = lambda n, s: torch.randn(n, generator=gen) * s          # noqa: E731
    out = []
    for k, n in enumerate(sizes):
        t = dict(p=rand(n, 0.02).to(kind[p]).cuda(), g=rand(n, 1e-2).to(kind[g]).cuda(),
                 weight_decay=0.1 * (k % 2))
        if bits == 32:
            t["m"], t["v"] = rand(n, 1e-2).cuda(), rand(n, 1e-2).square().cuda()
        else:
            for key, low in (("m", None), ("v", 0.0)):
                x = (torch.randn(n, generator=gen) * 100).clamp(low, 448)
                t[key] = x.clamp(-448, 448).to(torch.float8_e4m3fn).cuda()
                t[key + "_scale"] = (torch.rand(-(-n // 256), generator=gen) * 1e-4 + 1e-6).cuda()
        out.append(t)
    return out


def _blocks(np_scale, n):
    return np.repeat(np_scale, 256)[:n]


def _np(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def _step64(t, step, eight):
    """p', m', v' and the size of the step, in 64 bits."""
    p, g, m, v = (_np(t[k]) for k in ("p", "g", "m", "v"))
    n = p.size
    if eight:
        m = m * _blocks(_np(t["m_scale"]), n)
        v = (v * _blocks(_np(t["v_scale"]), n)) ** 2
    m1, v1 = B1 * m + (1 - B1) * g, B2 * v + (1 - B2) * g * g
    msize = B1 * np.abs(m) + (1 - B1) * np.abs(g)
    d = np.sqrt(v1) / math.sqrt(1 - B2 ** step) + EPS
    move = LR / (1 - B1 ** step) * m1 / d
    size = LR / (1 - B1 ** step) * msize / d
    return p * (1 - LR * t["weight_decay"]) - move, m1, msize, v1, np.abs(p) + size, size


SIZES = [[1], [7, 8, 9], [255, 256, 257, 1], [4095, 4096, 4097], [100_003, 0, 33, 5000, 8192]]


@pytest.mark.parametrize("sizes", SIZES)
@pytest.mark.parametrize("p", ["f32", "bf16"])
@pytest.mark.parametrize("g", ["f32", "bf16"])
@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("step", [1, 1000])
def test_step(sizes, p, g, bits, step):
    torch = torch_cuda()
    import w8a8_integer_linear_amd as qlin
    announce("adamw_tensors", sizes, p, g, bits, step)
    ts = _tensors(torch, sizes, p, g, bits)
    before = [{k: (v.clone() if hasattr(v, "clone") else v) for k, v in t.items()} for t in ts]
    plan = qlin.qlin_adamw_tensors_plan(ts)
    qlin.qlin_adamw_tensors(plan, LR, B1, B2, EPS, SEED, step)
    torch.cuda.synchronize()
    for t, old in zip(ts, before):
        n = t["p"].numel()
        assert torch.equal(t["g"], old["g"])
        if n == 0:
            continue
        p1, m1, msize, v1, psize, size = _step64(old, step, bits == 8)
        # the step's size has a sum in m' and a root and a quotient; hyperparameters
        # are rounded once
        bound = psize * 4 * U + size * 32 * U
        if p == "bf16":
            bound = bound + np.maximum(np.abs(p1), 2.0 ** -126) * 2.0 ** -7
        assert (np.abs(_np(t["p"]) - p1) <= bound).all()
        if bits == 32:
            assert (np.abs(_np(t["m"]) - m1) <= 4 * U * msize).all()
            assert (np.abs(_np(t["v"]) - v1) <= 8 * U * v1).all()
            continue
        for key, want, size, near in (("m", m1, msize, 0.5), ("v", np.sqrt(v1), np.sqrt(v1), 1.0)):
            sc = _np(t[key + "_scale"])
            pad = np.zeros(-(-n // 256) * 256)
            pad[:n] = np.abs(want)
            top = pad.reshape(-1, 256).max(1)
            assert (np.abs(sc * 448 - top) <= 16 * U * np.maximum(top, 1e-30) + 8 * U * size.max()).all()
            s = _blocks(sc, n)
            code = _np(t[key])
            x = want / np.where(s > 0, s, 1)
            unit = np.maximum(2.0 ** (np.floor(np.log2(np.maximum(np.abs(x), 2.0 ** -6))) - 3), 2.0 ** -9)
            slack = 32 * U * size / np.where(s > 0, s, 1)
            ok = np.abs(code - x) <= near * unit * (1 + 1e-5) + slack
            if key == "v":      # a value above zero keeps the smallest code
                ok |= (code == 2.0 ** -9) & (x < 2.0 ** -9)
                assert (code[want > 0] > 0).all()
            assert ok.all()


def test_uniforms_are_philox():
    """The stochastic codes are those that Philox4x32-10 with key seed and counter
    (index >> 3, step) gives, but where the fp32 value decides by its last bits."""
    torch = torch_cuda()
    import w8a8_integer_linear_amd as qlin
    n, step, index0 = 20_000, 77, 4096
    ts = _tensors(torch, [n], "bf16", "f32", 8)
    old = {k: (v.clone() if hasattr(v, "clone") else v) for k, v in ts[0].items()}
    ts[0]["index0"] = index0
    qlin.qlin_adamw_tensors(qlin.qlin_adamw_tensors_plan(ts), LR, B1, B2, EPS, SEED, step)
    torch.cuda.synchronize()
    p1, _, _, v1, _, _ = _step64(old, step, True)

    def uniforms(top):
        out = np.empty(n, np.int64)
        for blk in range(n // 8):
            i = index0 // 8 + blk
            ctr = np.array([i, 0, step, top], np.uint32)
            key = np.array([SEED & 0xFFFFFFFF, SEED >> 32], np.uint32)
            w = _philox(ctr, key)
            out[8 * blk:8 * blk + 8] = [(int(w[e >> 1]) >> (16 * (e & 1))) & 0xFFFF for e in range(8)]
        return out

    s = _blocks(_np(ts[0]["v_scale"]), n)
    t = np.minimum(np.sqrt(v1) / s, 448).astype(np.float32)
    low = np.where(t < 2.0 ** -6, np.float32(2.0 ** -6), np.float32(0))
    bits = ((t + low).view(np.uint32).astype(np.int64) + (uniforms(0) << 4)) & ~0xFFFFF
    want = bits.astype(np.uint32).view(np.float32) - low
    want = np.where(t > 0, np.maximum(want, np.float32(2.0 ** -9)), want)
    assert np.mean(want != _np(ts[0]["v"])) < 1e-3
    bits = (p1.astype(np.float32).view(np.uint32).astype(np.int64) + uniforms(1 << 31)) & ~0xFFFF
    assert np.mean(bits.astype(np.uint32).view(np.float32) != _np(ts[0]["p"])) < 1e-3


def _philox(ctr, key):
    c, k = [int(x) for x in ctr], [int(x) for x in key]
    for r in range(10):
        p0, p1 = 0xD2511F53 * c[0], 0xCD9E8D57 * c[2]
        c = [(p1 >> 32) ^ c[1] ^ k[0], p1 & 0xFFFFFFFF, (p0 >> 32) ^ c[3] ^ k[1], p0 & 0xFFFFFFFF]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return c


def test_second_moment_moves_in_the_mean():
    """Ten thousand equal elements whose moment should shrink by a part in a
    thousand per step: to nearest it would stay; stochastically its mean follows."""
    torch = torch_cuda()
    import w8a8_integer_linear_amd as qlin
    n, steps = 256 * 40, 200
    t = dict(p=torch.zeros(n, device="cuda"), g=torch.zeros(n, device="cuda"),
             m=torch.zeros(n, device="cuda").to(torch.float8_e4m3fn),
             v=torch.full((n,), 100.0, device="cuda").to(torch.float8_e4m3fn),
             m_scale=torch.zeros(40, device="cuda"), v_scale=torch.ones(40, device="cuda"))
    start = t["v"].float()[0].item()
    # one element per block stays on top, so that the block's scale does not follow
    plan = qlin.qlin_adamw_tensors_plan([t])
    top = torch.arange(0, n, 256, device="cuda")
    for k in range(steps):
        v = t["v"].float()
        v[top] = 448.0
        t["v"].copy_(v.to(torch.float8_e4m3fn))
        t["v_scale"].fill_(1.0)
        t["g"][top] = 448.0
        qlin.qlin_adamw_tensors(plan, LR, B1, B2, EPS, 5, k + 1)
    mean = (t["v"].float() * t["v_scale"].repeat_interleave(256)).view(-1, 256)[:, 1:].mean().item()
    want = start * B2 ** (steps / 2)
    # standard error: steps of 8 with p (1 - p) <= p, p = 0.0005 * 100 / 8 each step
    sd = 8 * math.sqrt(steps * 0.00625 / (n - 40))
    assert abs(mean - want) < 6 * sd + 0.1


def test_not_finite_gradients_stay_in_their_block():
    torch = torch_cuda()
    import w8a8_integer_linear_amd as qlin
    for bits in (32, 8):
        announce("not finite", bits)
        ts = _tensors(torch, [2000], "f32", "f32", bits)
        ref = [{k: (v.clone() if hasattr(v, "clone") else v) for k, v in t.items()} for t in ts]
        ts[0]["g"][300] = float("nan")
        for t in (ts, ref):
            qlin.qlin_adamw_tensors(qlin.qlin_adamw_tensors_plan(t), LR, B1, B2, EPS, 1, 3)
        torch.cuda.synchronize()
        assert ts[0]["p"][300].isnan()
        keep = torch.ones(2000, dtype=torch.bool, device="cuda")
        keep[300] = False
        assert torch.equal(ts[0]["p"][keep], ref[0]["p"][keep])
        if bits == 8:
            assert ts[0]["m_scale"][1].isnan() and ts[0]["v_scale"][1].isnan()
            keep[256:512] = False
            assert not ts[0]["m_scale"][0].isnan()
        for k in ("m", "v"):
            assert torch.equal(ts[0][k].float()[keep], ref[0][k].float()[keep])


def test_zero_blocks_stay_zero():
    torch = torch_cuda()
    import w8a8_integer_linear_amd as qlin
    n = 700
    z = lambda k: torch.zeros(k, device="cuda")                    # noqa: E731
    t = dict(p=torch.ones(n, device="cuda"), g=z(n), m=z(n).to(torch.float8_e4m3fn),
             v=z(n).to(torch.float8_e4m3fn), m_scale=z(3), v_scale=z(3))
    qlin.qlin_adamw_tensors(qlin.qlin_adamw_tensors_plan([t]), LR, B1, B2, EPS, 1, 1)
    assert (t["p"] == 1).all() and (t["m"].float() == 0).all() and (t["v"].float() == 0).all()
    assert (t["m_scale"] == 0).all() and (t["v_scale"] == 0).all()
    # a gradient of 1e-32 is kept by fp32 moments alone; 8-bit blocks drop it
    t["g"].fill_(1e-32)
    qlin.qlin_adamw_tensors(qlin.qlin_adamw_tensors_plan([t]), LR, B1, B2, EPS, 1, 1)
    assert t["p"].isfinite().all() and (t["m_scale"] == 0).all()


def test_order_of_the_list_and_of_the_launch_does_not_matter():
    """Tensors with their own index0 are updated alike alone and in a list, on
    another stream and in a graph."""
    torch = torch_cuda()
    import w8a8_integer_linear_amd as qlin
    sizes = [3000, 17, 9000, 256]

    def fresh():
        ts = _tensors(torch, sizes, "bf16", "bf16", 8)
        for k, t in enumerate(ts):
            t["index0"] = 65536 * k
        return ts

    a, b, c = fresh(), fresh(), fresh()
    qlin.qlin_adamw_tensors(qlin.qlin_adamw_tensors_plan(a), LR, B1, B2, EPS, SEED, 9)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for t in reversed(b):
        qlin.qlin_adamw_tensors(qlin.qlin_adamw_tensors_plan([t]), LR, B1, B2, EPS, SEED, 9, stream=side)
    side.synchronize()
    plan = qlin.qlin_adamw_tensors_plan(c)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qlin.qlin_adamw_tensors(plan, LR, B1, B2, EPS, SEED, 9)
    graph.replay()
    torch.cuda.synchronize()
    for x in (b, c):
        for s, t in zip(a, x):
            for k in ("p", "m", "v", "m_scale", "v_scale"):
                assert torch.equal(s[k].float(), t[k].float()), k
