"""8-bit rows, their products and the gradients against the oracle (needs a
gfx950 GPU).

Tolerances.  Integers, scales, values read back and products are compared bit
for bit: every rounding of theirs is stated.  A gradient sums C products of a
bf16 value and a value v = scale * q; with A = sum |grad_y| |v|,
  * v enters rounded to bf16 (half a step: 2^-8), or, for fp32 outputs, as it
    is, after one fp32 rounding of scale * q (2^-24);
  * the fp32 sum: every addition rounds at most 2^-23 (half a step, or the
    matrix cores' truncation) of a partial sum that A bounds, C + 8 of them;
  * storing: half a step of the output's type, and 2^-24 more of the sum with
    what was there.
"""
import sys

import numpy as np
import pytest
import torch

from newton_schulz_amd import Context, MuonError, MuonStep, Rows8, linear8_workspace_bytes
from oracle import linear8_oracle as lo

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def ctx():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    c = Context(DEV, 64 << 20)
    yield c
    c.close()


def values(rows, cols, dtype, seed, scale=1.0, pad=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, cols + pad, generator=g) * scale
    x = x * torch.exp(torch.randn(cols + pad, generator=g) * 0.7)
    return x.to(dtype).to(DEV)[:, :cols]


def eight(ctx, rows, cols, seed, least=-127):
    """8-bit rows of any integers, with something behind each row."""
    g = torch.Generator().manual_seed(seed)
    out = ctx.rows8(rows, cols)
    if out.q.numel():
        base = out.q._base
        base.copy_(torch.randint(least, 128, base.shape, generator=g, dtype=torch.int8))
    out.scale.copy_(torch.rand(rows, generator=g) * 0.02 + 1e-3)
    return out


def bits(t):
    return t.cpu().view({2: torch.int16, 4: torch.int32, 1: torch.int8}[t.element_size()])


ROWS = [(1, 1), (1, 16), (2, 15), (3, 17), (5, 64), (4, 255), (7, 257), (1, 1000), (33, 1101), (2, 4096), (3, 9728),
        (2, 20001), (1, 131071), (1500, 40), (300, 2560)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,cols", ROWS)
@pytest.mark.parametrize("pad", [0, 3, 8])
def test_rows_there_and_back(ctx, dtype, rows, cols, pad):
    x = values(rows, cols, dtype, rows * 31 + cols, pad=pad)
    out = eight(ctx, rows, cols, 5)
    behind = out.q._base[:, cols:].clone()
    ctx.quantize_rows(x, out)
    q, s = lo.quantize_ref(x.float().cpu().numpy())
    assert np.array_equal(out.scale.cpu().numpy().view(np.uint32), s.view(np.uint32))
    assert np.array_equal(out.q.cpu().numpy(), q)
    assert torch.equal(out.q._base[:, cols:], behind), "bytes behind a row were written"
    for dt in (BF, F32):
        back = torch.full((rows, cols + pad), 7.0, dtype=dt, device=DEV)
        ctx.dequantize_rows(out, back[:, :cols])
        want = (torch.from_numpy(s)[:, None] * torch.from_numpy(q).float()).to(dt)
        assert torch.equal(bits(back[:, :cols].contiguous()), bits(want))
        assert (back[:, cols:] == 7.0).all()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_rows_out_of_the_ordinary(ctx, dtype):
    """Zeros, denormals, the largest and smallest magnitudes, ties at halves, and what is not finite."""
    top = float(torch.finfo(dtype).max)
    tiny = float(torch.tensor(1.0, dtype=dtype).mul(2.0 ** -133).item()) or 2.0 ** -133
    rows = [torch.zeros(64), torch.full((64,), tiny), torch.full((64,), -0.0), torch.linspace(-top, top, 64),
            torch.arange(64) * 2.0 ** -126, torch.cat([torch.tensor([127.0, -127.0]), torch.arange(62) - 30.5]),
            torch.cat([torch.tensor([254.0]), 2.0 * torch.arange(63) - 63]), torch.randn(64) * 1e-38,
            torch.randn(64), torch.linspace(-1, 1, 64) * top, torch.randn(64), torch.randn(64), torch.randn(64)]
    rows[-1][3], rows[-2][63], rows[-3][0] = float("nan"), float("inf"), -float("inf")
    x = torch.stack([r.float() for r in rows]).to(dtype)
    out = ctx.rows8(len(x), 64)
    ctx.quantize_rows(x.to(DEV), out)
    q, s = lo.quantize_ref(x.float().numpy())
    got = out.scale.cpu().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(s))
    assert np.array_equal(got[~np.isnan(s)].view(np.uint32), s[~np.isnan(s)].view(np.uint32))
    assert np.array_equal(out.q.cpu().numpy(), q)
    back = torch.empty(len(x), 64, dtype=dtype, device=DEV)
    ctx.dequantize_rows(out, back)
    # (a linspace between the largest numbers overflows on the way: its row is not finite either)
    finite = torch.isfinite(x).all(1)
    assert finite.sum() == len(x) - 4 and finite[-4]
    assert torch.isnan(back[~finite.to(DEV)]).all() and torch.isfinite(back[finite.to(DEV)]).all()


@pytest.mark.parametrize("cols", [200, 1048])
def test_quotients_next_to_halves(ctx, cols):
    """fp32 values a few units in the last place around every half step of many scales."""
    g = torch.Generator().manual_seed(3)
    x = torch.empty(400, cols)
    for r in range(400):
        top = torch.rand(1, generator=g).item() * 2.0 ** float(torch.randint(-20, 20, (1,), generator=g)) + 1e-6
        s = np.float32(top) / np.float32(127)
        half = (np.arange(cols) % 253 - 126.5).astype(np.float64) * np.float64(s)
        v = torch.from_numpy(half.astype(np.float32)).view(torch.int32) + torch.randint(-2, 3, (cols,), generator=g, dtype=torch.int32)
        x[r] = v.view(torch.float32).clamp(-top, top)
        x[r, 0] = float(np.float32(top))
    out = ctx.rows8(400, cols)
    ctx.quantize_rows(x.to(DEV), out)
    q, s = lo.quantize_ref(x.numpy())
    assert np.array_equal(out.scale.cpu().numpy(), s) and np.array_equal(out.q.cpu().numpy(), q)


PRODUCTS = [  # m, n, k
    (1, 1, 1), (1, 7, 15), (1, 640, 256), (2, 33, 16), (3, 65, 1000), (5, 1001, 64), (13, 257, 2560), (16, 4096, 128), (17, 300, 333),
    (31, 129, 4097), (32, 2560, 9728), (33, 64, 65), (63, 63, 63), (64, 1000, 512), (65, 130, 129), (127, 255, 1237),
    (128, 128, 64), (129, 1001, 777), (256, 256, 1024), (300, 515, 130), (511, 770, 2049), (1, 151, 131071), (40, 60, 100000),
    (1025, 1100, 256), (2, 20000, 40),
]


def check_product(ctx, a, b, dtype, ldo=0):
    m, n = len(a.scale), len(b.scale)
    out = torch.full((m, n + ldo), 3.0, dtype=dtype, device=DEV)
    ctx.matmul8(a, b, out[:, :n])
    host = [t.cpu().numpy() for t in (a.q, a.scale, b.q, b.scale)]
    want = torch.from_numpy(lo.matmul8_ref(*host)).to(dtype)
    assert torch.equal(bits(out[:, :n].contiguous()), bits(want))
    assert (out[:, n:] == 3.0).all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("m,n,k", PRODUCTS)
def test_product(ctx, dtype, m, n, k):
    check_product(ctx, eight(ctx, m, k, m + k, least=-128), eight(ctx, n, k, n, least=-128), dtype, ldo=(0, 5, 8)[(m + n) % 3])


def test_product_of_extremes(ctx):
    """The largest sum that 32 bits hold, of both signs."""
    a, b = ctx.rows8(20, 131071), ctx.rows8(70, 131071)
    a.q.fill_(-128)
    b.q.fill_(-128)
    b.q[::2] = 127
    a.scale.fill_(1.0)
    b.scale.fill_(0.5)
    check_product(ctx, a, b, F32)


@pytest.mark.parametrize("m,n,k", [(70, 90, 50), (3, 40, 64), (300, 300, 300)])
def test_scales_that_are_not_finite_stay_in_their_rows(ctx, m, n, k):
    a, b = eight(ctx, m, k, 1), eight(ctx, n, k, 2)
    a.scale[1], a.scale[2] = float("nan"), 0.0
    b.scale[n - 1] = float("inf")
    out = torch.empty(m, n, device=DEV)
    ctx.matmul8(a, b, out)
    assert torch.isnan(out[1]).all() and (out[2, :-1] == 0).all() and torch.isfinite(out[3:, :-1]).all()
    assert torch.isfinite(out[0, :-1]).all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("keep", [False, True])
@pytest.mark.parametrize("m,n,k", [(1, 9, 40), (1, 2560, 1101), (4, 1000, 64), (16, 300, 2560), (37, 301, 1237), (300, 500, 96)])
def test_linear_is_quantisation_and_product(ctx, dtype, keep, m, n, k):
    x, w = values(m, k, dtype, m + n, pad=2), eight(ctx, n, k, 9)
    out = torch.empty(m, n, dtype=dtype, device=DEV)
    x8 = ctx.rows8(m, k) if keep else None
    ctx.linear8(x, w, out, x8=x8)
    q, s = lo.quantize_ref(x.float().cpu().numpy())
    want = torch.from_numpy(lo.matmul8_ref(q, s, w.q.cpu().numpy(), w.scale.cpu().numpy())).to(dtype)
    assert torch.equal(bits(out), bits(want))
    if keep:
        assert np.array_equal(x8.q.cpu().numpy(), q) and np.array_equal(x8.scale.cpu().numpy(), s)


GRADS = [  # tokens, n, k
    (1, 1, 1), (1, 7, 5), (2, 33, 16), (5, 64, 130), (16, 1000, 40), (31, 65, 257), (61, 301, 1237), (64, 64, 64),
    (100, 130, 200), (127, 512, 96), (128, 256, 128), (129, 257, 255), (256, 256, 256), (300, 520, 264), (1000, 72, 136),
    (1500, 40, 48), (40, 3000, 64), (64, 48, 4000), (2050, 330, 200), (513, 770, 1030), (33, 9000, 100), (7000, 64, 72),
]


def check_grads(ctx, t, n, k, dtype, accumulate, pad=0, seed=0):
    g = torch.Generator().manual_seed(seed + t)
    y = (torch.randn(t, n + pad, generator=g) * 1e-3).to(BF).to(DEV)[:, :n]
    w, x = eight(ctx, n, k, n + 1), eight(ctx, t, k, t + 2)
    gx = torch.randn(t, k + pad, generator=g).mul_(1e-2).to(dtype).to(DEV)
    gw = torch.randn(n, k + pad, generator=g).mul_(1e-2).to(dtype).to(DEV)
    was = [gx.clone(), gw.clone()]
    ctx.input_grad8(y, w, gx[:, :k], accumulate=accumulate)
    ctx.weight_grad8(y, x, gw[:, :k], accumulate=accumulate)
    yd = y.double().cpu().numpy()
    for got, old, a, rows8 in ((gx, was[0], yd, w), (gw, was[1], yd.T, x)):
        v = lo.values_ref(rows8.q.cpu().numpy(), rows8.scale.cpu().numpy())
        want = a @ v
        size = np.abs(a) @ np.abs(v)
        before = old[:, :k].double().cpu().numpy() if accumulate else 0.0
        want = want + before
        half = torch.finfo(dtype).eps / 2
        tol = size * ((2.0 ** -8 if dtype == BF else 0.0) + 2.0 ** -24 + (a.shape[1] + 8) * 2.0 ** -23)
        tol = tol * (1 + half) + (half + 2.0 ** -24) * np.abs(want) + 2.0 ** -130
        off = np.abs(got[:, :k].double().cpu().numpy() - want)
        assert (off <= tol).all(), f"off by {off.max():.3e}, {(off / tol).max():.2f} of the tolerance"
        assert torch.equal(got[:, k:], old[:, k:]), "columns behind the output were written"


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("t,n,k", GRADS)
def test_gradients(ctx, dtype, accumulate, t, n, k):
    check_grads(ctx, t, n, k, dtype, accumulate, pad=(0, 1, 8)[(t + k) % 3])


def test_gradients_follow_differences(ctx):
    """Of a loss sum(y * g) in the values of x and w: a product's differences are its gradient."""
    t, n, k = 6, 5, 24
    x, w = eight(ctx, t, k, 1), eight(ctx, n, k, 2)
    g = torch.randn(t, n, generator=torch.Generator().manual_seed(0)).to(BF).to(DEV)
    gx, gw = torch.empty(t, k, device=DEV), torch.empty(n, k, device=DEV)
    ctx.input_grad8(g, w, gx)
    ctx.weight_grad8(g, x, gw)
    out, gd = torch.empty(t, n, device=DEV), g.double()

    def loss():
        ctx.matmul8(x, w, out)
        return (out.double() * gd).sum().item()

    for rows8, grad in ((x, gx), (w, gw)):
        for r, c in ((0, 0), (3, 11), (4, 23)):
            q0 = rows8.q[r, c].item()
            rows8.q[r, c] = q0 + 1 if q0 < 100 else q0 - 1
            up = loss()
            rows8.q[r, c] = q0
            d = (up - loss()) / (rows8.scale[r].item() * (1 if q0 < 100 else -1))
            # 2^-24 of each of 30 products of size up to 24 * 127^2 * 0.02^2, against one step of 1e-3
            assert abs(d - grad[r, c].item()) < 30 * 2 * 2.0 ** -22 * 155 * 3 / 1e-3 + 2.0 ** -15 * abs(d)


def test_nothing_to_do(ctx):
    w, none = eight(ctx, 9, 20, 1), ctx.rows8(0, 20)
    out = torch.empty(0, 9, dtype=BF, device=DEV)
    ctx.matmul8(none, w, out)
    ctx.linear8(torch.empty(0, 20, dtype=BF, device=DEV), w, out, x8=none)
    ctx.quantize_rows(torch.empty(0, 20, device=DEV), none)
    ctx.dequantize_rows(none, torch.empty(0, 20, device=DEV))
    ctx.input_grad8(torch.empty(0, 9, dtype=BF, device=DEV), w, torch.empty(0, 20, device=DEV))
    gw = torch.ones(9, 20, device=DEV)
    ctx.weight_grad8(torch.empty(0, 9, dtype=BF, device=DEV), none, gw, accumulate=True)
    assert (gw == 1).all()
    ctx.weight_grad8(torch.empty(0, 9, dtype=BF, device=DEV), none, gw)
    assert (gw == 0).all()


def test_rows_that_repeat_and_leading_dimensions(ctx):
    """Stride 0 inputs, [batch, seq, k] activations, a single row of any stride."""
    w = eight(ctx, 130, 64, 1)
    row = values(1, 64, BF, 3)
    many = row.expand(70, 64)
    a, b = torch.empty(70, 130, device=DEV), torch.empty(1, 130, device=DEV)
    ctx.linear8(many, w, a)
    ctx.linear8(row, w, b)
    assert torch.equal(a, b.expand(70, 130))
    x = values(70, 64, BF, 4)
    ctx.linear8(x.view(7, 10, 64), w, a.view(7, 10, 130))
    c = torch.empty(70, 130, device=DEV)
    ctx.linear8(x, w, c)
    assert torch.equal(a, c)


def test_another_stream_and_a_graph(ctx):
    """Each replay of recorded calls, with eager work in between, equals the eager calls."""
    t, n, k = 70, 260, 300
    w = eight(ctx, n, k, 1)
    x = values(t, k, BF, 2)
    gy = values(t, n, BF, 3, scale=1e-3).contiguous()
    y, x8 = torch.empty(t, n, dtype=BF, device=DEV), ctx.rows8(t, k)
    gx, gw = torch.empty(t, k, dtype=BF, device=DEV), torch.zeros(n, k, device=DEV)

    def calls(stream=None):
        ctx.linear8(x, w, y, x8=x8, stream=stream)
        ctx.input_grad8(gy, w, gx, stream=stream)
        ctx.weight_grad8(gy, x8, gw, stream=stream)

    calls()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    first = [v.clone() for v in (y, gx, gw)]
    torch.cuda.synchronize()
    calls(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, (y, gx, gw)))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        calls(side)
    for i in range(4):
        x.copy_(values(t, k, BF, 10 + i))
        gy.copy_(values(t, n, BF, 20 + i, scale=1e-3))
        calls()
        want = [v.clone() for v in (y, gx, gw)]
        for v in (y, gx, gw):
            v.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, (y, gx, gw))), f"replay {i}"


def test_same_bits_twice(ctx):
    t, n, k = 1000, 520, 640
    y, x8 = values(t, n, BF, 1, scale=1e-3), eight(ctx, t, k, 2)
    a, b = torch.empty(n, k, device=DEV), torch.empty(n, k, device=DEV)
    ctx.weight_grad8(y, x8, a)
    ctx.weight_grad8(y, x8, b)
    assert torch.equal(a, b)


@pytest.mark.parametrize("inflight", [1, 2])
def test_step_keeps_8_bit_weights(inflight):
    """A step's 8-bit weights are the rounding of its master weights, and its
    other results those of a step without them."""
    shapes = [(256, 512, 0), (512, 256, 0), (130, 202, 0), (130, 202, 0), (128, 640, 64), (64, 37, 0)]
    a = MuonStep(shapes, DEV, cap_bytes=1 << 19, inflight=inflight, keep_int8_weights=True)
    b = MuonStep(shapes, DEV, cap_bytes=1 << 19, inflight=inflight)
    g = torch.Generator(device=DEV).manual_seed(1)
    for m in (a, b):
        g.manual_seed(1)
        m.master.normal_(0, 0.02, generator=g)
        m.grad.copy_(torch.randn(m.numel, generator=g, device=DEV) * 1e-3)
    a.quantize_weights()

    def check():
        for i in range(len(shapes)):
            q, s = lo.quantize_ref(a.view(a.master, i).cpu().numpy())
            assert np.array_equal(a.weight8(i).q.cpu().numpy(), q) and np.array_equal(a.weight8(i).scale.cpu().numpy(), s), i

    check()
    for _ in range(2):
        a.step()
        b.step()
    torch.cuda.synchronize()
    assert torch.equal(a.master, b.master)
    check()
    with pytest.raises(ValueError, match="keep_int8_weights"):
        b.weight8(0)


def test_layer_trains_through_the_step(ctx):
    """Forward, both gradients and the step together: the weights' gradient goes
    into the step's buffer, the next forward reads the moved weights."""
    t, n, k = 96, 200, 136
    step = MuonStep([(n, k, 0)], DEV, lr=0.05, grad_dtype=F32, keep_int8_weights=True)
    step.view(step.master, 0).copy_(torch.randn(n, k, generator=torch.Generator().manual_seed(0)) * k ** -0.5)
    step.quantize_weights()
    x = values(t, k, BF, 1)
    x8, y, gx = ctx.rows8(t, k), torch.empty(t, n, device=DEV), torch.empty(t, k, device=DEV)
    for i in range(2):
        ctx.linear8(x, step.weight8(0), y, x8=x8)
        w = lo.values_ref(step.weight8(0).q.cpu().numpy(), step.weight8(0).scale.cpu().numpy())
        xs = lo.values_ref(x8.q.cpu().numpy(), x8.scale.cpu().numpy())
        want = xs @ w.T
        assert np.abs(y.cpu().numpy() - want).max() <= 2.0 ** -21 * np.abs(want).max()
        gy = y.to(BF)
        ctx.input_grad8(gy, step.weight8(0), gx)
        ctx.weight_grad8(gy, x8, step.view(step.grad, 0))
        yd = gy.double().cpu().numpy()
        for got, ref, size in ((gx, yd @ w, np.abs(yd) @ np.abs(w)),
                               (step.view(step.grad, 0), yd.T @ xs, np.abs(yd.T) @ np.abs(xs))):
            tol = size * (2.0 ** -24 + 210 * 2.0 ** -23) + 2.0 ** -24 * np.abs(ref)
            assert (np.abs(got.cpu().numpy() - ref) <= tol).all()
        before = step.view(step.master, 0).clone()
        step.step()
        torch.cuda.synchronize()
        assert not torch.equal(before, step.view(step.master, 0))
        print(f"  pass {i} done", file=sys.stderr, flush=True)


def test_offsets_past_32_bits(ctx):
    """More than 2^31 elements of activations, of their 8-bit rows and of the
    gradient of y: the first and last rows against the oracle, and the weights'
    gradient against sums of 64 bits."""
    t, n, k = (1 << 20) + 300, 2064, 2064
    g = torch.Generator(device=DEV).manual_seed(7)
    x = torch.empty(t, k, dtype=BF, device=DEV).normal_(generator=g)
    x8, w = ctx.rows8(t, k), eight(ctx, n, k, 3)
    ctx.quantize_rows(x, x8)
    ends = [slice(0, 70), slice(t - 70, t)]
    for e in ends:
        q, s = lo.quantize_ref(x[e].float().cpu().numpy())
        assert np.array_equal(x8.q[e].cpu().numpy(), q) and np.array_equal(x8.scale[e].cpu().numpy(), s)
    back = torch.empty_like(x)
    ctx.dequantize_rows(x8, back)
    for e in ends:
        assert torch.equal(back[e], (x8.scale[e, None] * x8.q[e].float()).to(BF))
    print("  rows done", file=sys.stderr, flush=True)
    y = back  # [t, n]
    ctx.matmul8(x8, w, y)
    for e in ends:
        want = torch.from_numpy(lo.matmul8_ref(*(v.cpu().numpy() for v in (x8.q[e], x8.scale[e], w.q, w.scale)))).to(BF)
        assert torch.equal(bits(y[e]), bits(want))
    print("  product done", file=sys.stderr, flush=True)
    gx = x
    ctx.input_grad8(y, w, gx)
    v = lo.values_ref(w.q.cpu().numpy(), w.scale.cpu().numpy())
    for e in ends:
        yd = y[e].double().cpu().numpy()
        tol = np.abs(yd) @ np.abs(v) * (2.0 ** -8 + 2.0 ** -24 + (n + 8) * 2.0 ** -23) * (1 + 2.0 ** -8)
        want = yd @ v
        assert (np.abs(gx[e].double().cpu().numpy() - want) <= tol + 2.0 ** -8 * np.abs(want)).all()
    # a few columns of the weights' gradient
    gw = torch.empty(n, k, device=DEV)
    ctx.weight_grad8(y, x8, gw)
    some = torch.tensor([0, 1, 77, 1031, k - 1], device=DEV)
    want, size = torch.zeros(n, 5, dtype=torch.float64, device=DEV), torch.zeros(n, 5, dtype=torch.float64, device=DEV)
    for i in range(0, t, 1 << 17):
        a = y[i:i + (1 << 17)].double()
        b = x8.q[i:i + (1 << 17)][:, some].double() * x8.scale[i:i + (1 << 17), None].double()
        want += a.t() @ b
        size += a.abs().t() @ b.abs()
    # every addition rounds at most 2^-23 of a partial sum, of random signs: a
    # partial sum is bounded by `size`, and t roundings of that size and random
    # sign exceed 8 sqrt(t) of them nowhere
    tol = size * (2.0 ** -24 + 8 * t ** 0.5 * 2.0 ** -23) + 2.0 ** -24 * want.abs()
    assert ((gw[:, some].double() - want).abs() <= tol).all()


def test_two_contexts_at_once():
    """Calls on two streams, each with a context of its own, keep their results."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    both = []
    for i in range(2):
        c = Context(DEV, 64 << 20)
        t, n, k = 130 + i, 520, 1032
        both.append((c, torch.cuda.Stream(), values(t, k, BF, i), eight(c, n, k, i), values(t, n, BF, 5 + i, scale=1e-3).contiguous(),
                     torch.empty(t, n, device=DEV), c.rows8(t, k), torch.empty(n, k, device=DEV)))

    def calls(c, s, x, w, gy, y, x8, gw):
        c.linear8(x, w, y, x8=x8, stream=s)
        c.weight_grad8(gy, x8, gw, stream=s)

    for args in both:
        calls(args[0], None, *args[2:])
    want = [(a[5].clone(), a[7].clone()) for a in both]
    torch.cuda.synchronize()
    for _ in range(20):
        for args in both:
            calls(*args)
    torch.cuda.synchronize()
    for args, (y, gw) in zip(both, want):
        assert torch.equal(args[5], y) and torch.equal(args[7], gw)
        args[0].close()


def test_recorded_step_and_offloaded_step_keep_8_bit_weights():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from newton_schulz_amd.offload import MuonOffloadStep
    shapes = [(256, 512, 0), (130, 202, 0), (64, 37, 0)]
    steps = [MuonStep(shapes, DEV, cap_bytes=1 << 19, keep_int8_weights=True) for _ in range(2)]
    steps.append(MuonOffloadStep(shapes, DEV, cap_bytes=1 << 19, keep_int8_weights=True, grads_on_host=False))
    for m in steps:
        g = torch.Generator(device=DEV).manual_seed(1)
        m.master.normal_(0, 0.02, generator=g)
        m.grad.copy_(torch.randn(m.numel, generator=g, device=DEV) * 1e-3)
    steps[0].capture()
    for _ in range(3):
        steps[0].replay()
        steps[1].step()
        steps[2].step()
        torch.cuda.synchronize()
        for m in steps[:1] + steps[2:]:
            for i in range(len(shapes)):
                assert torch.equal(m.weight8(i).q, steps[1].weight8(i).q)
                assert torch.equal(m.weight8(i).scale, steps[1].weight8(i).scale)
    q, s = lo.quantize_ref(steps[0].view(steps[0].master, 1).cpu().numpy())
    assert np.array_equal(steps[0].weight8(1).q.cpu().numpy(), q)


def test_refusals_of_the_binding(ctx):
    w, x = eight(ctx, 9, 20, 1), torch.zeros(4, 20, device=DEV)
    with pytest.raises(ValueError, match="no one stride"):
        ctx.linear8(torch.zeros(2, 3, 20, device=DEV).transpose(0, 1), w, torch.empty(6, 9, device=DEV))
    with pytest.raises(ValueError, match="contiguous"):
        ctx.linear8(torch.zeros(20, 4, device=DEV).t(), w, torch.empty(4, 9, device=DEV))
    with pytest.raises(ValueError, match="tensor on"):
        ctx.linear8(x.cpu(), w, torch.empty(4, 9, device=DEV))
    with pytest.raises(TypeError, match="dtype"):
        ctx.linear8(x.half(), w, torch.empty(4, 9, device=DEV))
    with pytest.raises(MuonError, match="do not match"):
        ctx.linear8(x, w, torch.empty(4, 8, device=DEV))
    with pytest.raises(MuonError, match="bf16"):
        ctx.input_grad8(torch.zeros(4, 9, device=DEV), w, torch.empty(4, 20, device=DEV))
    with pytest.raises(MuonError, match="16 bytes"):
        ctx.quantize_rows(x, Rows8(torch.zeros(4, 20, dtype=torch.int8, device=DEV), torch.zeros(4, device=DEV)))
    small = Context(DEV, 16)
    with pytest.raises(MuonError, match="workspace"):
        small.linear8(torch.zeros(64, 2000, device=DEV), eight(ctx, 9, 2000, 1), torch.empty(64, 9, device=DEV))
    small.close()


def test_workspace_is_what_a_call_needs():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    t, n, k = 64, 512, 4096
    need = linear8_workspace_bytes(t, n, k)
    c = Context(DEV, need)
    w, out = eight(c, n, k, 1), torch.empty(t, n, device=DEV)
    c.linear8(values(t, k, F32, 1), w, out)
    gy = values(t, n, BF, 2)
    c.input_grad8(gy, w, torch.empty(t, k, device=DEV))
    c.weight_grad8(gy, eight(c, t, k, 3), torch.empty(n, k, device=DEV))
    torch.cuda.synchronize()
    c.close()


@pytest.mark.parametrize("rows,cols", [(2047, 2560), (2048, 2560), (2049, 2561), (2048, 2568), (1030, 1281), (3, 512), (3, 513)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_rows_of_a_wave_and_of_a_workgroup(ctx, dtype, rows, cols):
    """Either side of the sizes at which a row goes to a wave or to a workgroup."""
    x, out = values(rows, cols, dtype, cols), ctx.rows8(rows, cols)
    ctx.quantize_rows(x, out)
    q, s = lo.quantize_ref(x.float().cpu().numpy())
    assert np.array_equal(out.scale.cpu().numpy(), s) and np.array_equal(out.q.cpu().numpy(), q)


@pytest.mark.parametrize("m,n,k", [
    (13, 17003, 2560), (16, 4096, 2816), (16, 4096, 2817), (16, 4095, 2816), (32, 4100, 1408), (5, 20005, 3000),
    (17, 30001, 100), (16, 4099, 1024), (16, 4099, 1025), (64, 8192, 130), (64, 8193, 130),
])
def test_few_rows_by_many_columns(ctx, m, n, k):
    """Rows held by workgroups that walk the columns, up to what one holds, and beyond."""
    check_product(ctx, eight(ctx, m, k, m + k, least=-128), eight(ctx, n, k, n, least=-128), BF)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("m,n,k", [(1, 40003, 2560), (6, 17000, 2560), (1, 20000, 2047), (3, 30005, 200), (16, 20001, 1024), (20, 9000, 777),
                                   (4, 40, 4096), (4, 17001, 4097)])
def test_rounding_on_the_way_to_many_columns(ctx, dtype, m, n, k):
    """linear8 in one launch, several columns' groups a workgroup; and just beyond its room."""
    x, w, x8 = values(m, k, dtype, m + n), eight(ctx, n, k, 9), ctx.rows8(m, k)
    out = torch.empty(m, n, dtype=BF, device=DEV)
    ctx.linear8(x, w, out, x8=x8)
    q, s = lo.quantize_ref(x.float().cpu().numpy())
    want = torch.from_numpy(lo.matmul8_ref(q, s, w.q.cpu().numpy(), w.scale.cpu().numpy())).to(BF)
    assert torch.equal(bits(out), bits(want))
    assert np.array_equal(x8.q.cpu().numpy(), q) and np.array_equal(x8.scale.cpu().numpy(), s)
