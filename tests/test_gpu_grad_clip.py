"""Global gradient norm, scaling and the clipped momentum pass against the
binary64 oracle (needs a gfx950 GPU).

Tolerances: every square is exact in binary64 and n of them are summed with
at most 2^-53 (n / threads + joins) relative error each, all of one sign, so
the sum is within n 2^-53 of exact, its root and the coefficient within that
too.  A scaled gradient has the coefficient's rounding to binary32, the
product's, and that of storing it (half a step of the type).
"""
import numpy as np
import pytest
import torch

from newton_schulz_amd import Context, MuonError, MuonStep, grad_norm_workspace_bytes
import oracle
from oracle import loss_oracle as lo

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def ctx():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    c = Context(DEV, 8 << 20)
    yield c
    c.close()


def tensors(sizes, dtype, seed=0, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return [(torch.randn(n, generator=g) * scale).to(BF if dtype == "mixed" and i % 2 else F32 if dtype == "mixed" else dtype).to(DEV)
            for i, n in enumerate(sizes)]


LISTS = {
    "one": [1],
    "few": [7, 8, 9, 0, 4096, 4095, 4097],
    "many": [(37 * i) % 301 for i in range(300)],        # three launches, empty tensors among them
    "exactly a table": [5] * 128,
    "one past a table": [5] * 129,
    "large": [1 << 20, 3, (1 << 22) + 5, 70001],
}


@pytest.mark.parametrize("dtype", [BF, F32, "mixed"])
@pytest.mark.parametrize("name", LISTS)
def test_norm_and_scaling(ctx, name, dtype):
    ts = tensors(LISTS[name], dtype)
    total = sum(LISTS[name])
    norm = torch.full((3,), -1.0, dtype=torch.float64, device=DEV)
    ctx.grad_norm(ts, norm, max_norm=0.75)
    s, size, c = lo.grad_norm_ref([t.double().cpu().numpy() for t in ts], 0.75)
    got = norm.cpu().numpy()
    assert np.abs(got - [s, size, c]).max() <= (total + 4) * 2.0 ** -53 * max(s, 1.0), (got, s, size, c)
    again = torch.empty_like(norm)
    ctx.grad_norm(ctx.tensor_list(ts), again, max_norm=0.75)
    assert torch.equal(norm, again)
    # into tensors of the other type that start at odd addresses
    outs = [torch.full((t.numel() + 2,), 9.0, dtype=BF if t.dtype == F32 else F32, device=DEV) for t in ts]
    views = [o[1:1 + t.numel()] for o, t in zip(outs, ts)]
    ctx.scale_grads(ts, norm, out=views)
    coef = np.float32(got[2])
    for t, v, o in zip(ts, views, outs):
        want = t.float() * torch.tensor(coef, device=DEV)     # one binary32 product
        assert torch.equal(v, want.to(v.dtype))
        assert o[0] == 9 and o[-1] == 9
    before = [t.clone() for t in ts]
    ctx.scale_grads(ts, norm)
    for t, b in zip(ts, before):
        assert torch.equal(t, (b.float() * torch.tensor(coef, device=DEV)).to(t.dtype))
        eps = torch.finfo(t.dtype).eps / 2
        want = b.double() * c
        assert ((t.double() - want).abs() <= want.abs() * (eps + 3 * 2.0 ** -24) + 1e-40).all()


def test_no_clipping_changes_nothing(ctx):
    ts = tensors([1000, 5], "mixed", scale=1e-3)
    before, norm = [t.clone() for t in ts], torch.empty(3, dtype=torch.float64, device=DEV)
    ctx.clip_grads(ts, norm, max_norm=1.0)
    assert norm[2] == 1 and all(torch.equal(a, b) for a, b in zip(ts, before))
    ctx.grad_norm(ts, norm)                                   # infinite limit
    assert norm[2] == 1
    ctx.grad_norm([], norm, max_norm=1.0)
    assert norm.tolist() == [0.0, 0.0, 1.0]
    ctx.grad_norm([torch.zeros(9, device=DEV)], norm, max_norm=1.0, eps=0.0)
    assert norm.tolist() == [0.0, 0.0, 1.0]


def test_huge_and_tiny_values_and_nonfinite(ctx):
    norm = torch.empty(3, dtype=torch.float64, device=DEV)
    for dtype in (BF, F32):
        big = torch.full((5000,), 3e38, dtype=dtype, device=DEV)
        ctx.grad_norm([big], norm, max_norm=1.0)
        v = big[0].double().item()
        assert norm[1].item() == pytest.approx(v * 5000 ** 0.5, rel=1e-12)
        small = torch.full((5000,), 1e-38, dtype=dtype, device=DEV)
        ctx.grad_norm([small], norm, max_norm=1.0)
        assert norm[1].item() == pytest.approx(small[0].double().item() * 5000 ** 0.5, rel=1e-12)
        denormal = torch.full((64,), 1e-40, dtype=dtype, device=DEV)
        ctx.grad_norm([denormal], norm, max_norm=1.0)
        assert norm[1].item() == pytest.approx(denormal[0].double().item() * 8, rel=1e-12)
        for bad in (float("inf"), float("nan")):
            t = torch.ones(5000, dtype=dtype, device=DEV)
            t[4097] = bad
            ctx.clip_grads([t], norm, max_norm=1.0)
            if bad == float("inf"):
                assert norm[1] == bad and norm[2] == 0
                assert (t[:4097] == 0).all() and t[4097].isnan()
            else:
                assert norm.isnan().all() and t.isnan().all()


def test_coefficient_after_a_sum_over_ranks(ctx):
    a, b = tensors([5000], BF, 1), tensors([3000], F32, 2)
    n1, n2, both = (torch.empty(3, dtype=torch.float64, device=DEV) for _ in range(3))
    ctx.grad_norm(a, n1, max_norm=0.5)
    ctx.grad_norm(b, n2, max_norm=0.5)
    n1[0] += n2[0]
    ctx.clip_coef(n1, max_norm=0.5)
    s, size, c = lo.grad_norm_ref([t.double().cpu().numpy() for t in a + b], 0.5)
    assert np.allclose(n1.cpu().numpy(), [s, size, c], rtol=8000 * 2.0 ** -53, atol=0)
    ctx.grad_norm(a + b, both, max_norm=0.5)
    assert np.allclose(both.cpu().numpy(), [s, size, c], rtol=8000 * 2.0 ** -53, atol=0)


@pytest.mark.parametrize("gdt,udt", [(BF, BF), (BF, F32), (F32, BF), (F32, F32)])
@pytest.mark.parametrize("numel,offset", [(1, 0), (4096, 0), (12345, 0), (8191, 1)])
@pytest.mark.parametrize("nesterov", [True, False])
def test_clipped_momentum_is_bit_exact(ctx, numel, offset, gdt, udt, nesterov):
    """The momentum pass of c * g, each operation one binary32 rounding."""
    g = torch.Generator().manual_seed(numel)
    grad = torch.randn(numel + offset, generator=g).to(gdt).to(DEV)[offset:]
    mom = torch.randn(numel + offset, generator=g).to(DEV)[offset:]
    upd = torch.empty(numel + offset, dtype=udt, device=DEV)[offset:]
    sq = torch.empty((numel + 4095) // 4096, dtype=torch.float64, device=DEV)
    norm = torch.tensor([0.0, 0.0, 0.3], dtype=torch.float64, device=DEV)
    gc = grad.float().cpu().numpy() * np.float32(0.3)
    want_m, want_u = oracle.momentum_ref(gc, mom.cpu().numpy().copy(), 0.95, nesterov)
    ctx.momentum_update(grad, mom, upd, 0.95, nesterov, sq_partials=sq, grad_scale=norm)
    assert np.array_equal(mom.cpu().numpy(), want_m)
    if udt == BF:
        want_u = oracle.bf16_round(want_u)
    assert np.array_equal(upd.float().cpu().numpy(), want_u)
    assert np.allclose(sq.sum().item(), np.square(want_u.astype(np.float64)).sum(), rtol=1e-12)
    # without partials the same bits
    mom2 = torch.zeros(numel, device=DEV)
    upd2, upd3 = torch.empty(numel, dtype=udt, device=DEV), torch.empty(numel, dtype=udt, device=DEV)
    ctx.momentum_update(grad.clone(), mom2, upd2, 0.95, nesterov, grad_scale=norm)
    ctx.momentum_update(torch.from_numpy(gc).to(DEV), torch.zeros(numel, device=DEV), upd3, 0.95, nesterov)
    assert torch.equal(upd2, upd3)


def test_refusals_of_the_binding(ctx):
    t = [torch.ones(8, device=DEV)]
    norm = torch.empty(3, dtype=torch.float64, device=DEV)
    for bad in (norm.float(), norm[:2], norm.cpu()):
        with pytest.raises((ValueError, TypeError)):
            ctx.grad_norm(t, bad)
    with pytest.raises(TypeError):
        ctx.grad_norm([t[0].half()], norm)
    with pytest.raises(ValueError):
        ctx.grad_norm([torch.ones(8, 8, device=DEV).t()[:3]], norm)
    with pytest.raises(ValueError):
        ctx.scale_grads(t, norm, out=t + t)
    with pytest.raises(MuonError) as e:
        ctx.grad_norm(t, norm, max_norm=0.0)
    assert e.value.status == 1
    with pytest.raises(MuonError):
        ctx.scale_grads(t + t, norm)
    c = Context(DEV, 256)
    many = [torch.ones(4, device=DEV) for _ in range(100)]
    with pytest.raises(MuonError) as e:
        c.grad_norm(many, norm)
    assert e.value.status == 4 and grad_norm_workspace_bytes(many) > 256
    c.close()


def test_clipping_in_a_recorded_graph(ctx):
    ts = tensors(LISTS["many"], "mixed")
    outs = [torch.empty_like(t) for t in ts]
    norm = torch.empty(3, dtype=torch.float64, device=DEV)
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream(DEV)
    side.wait_stream(torch.cuda.current_stream(DEV))
    with torch.cuda.graph(graph, stream=side):
        ctx.clip_grads(ts, norm, max_norm=0.5, out=outs, stream=side)
    torch.cuda.current_stream(DEV).wait_stream(side)
    for k in range(4):
        for t, n in zip(ts, tensors(LISTS["many"], "mixed", seed=k + 9)):
            t.copy_(n)
        graph.replay()
        torch.cuda.synchronize()
        want, eager = torch.empty_like(norm), [torch.empty_like(t) for t in ts]
        ctx.clip_grads(ts, want, max_norm=0.5, out=eager)
        assert torch.equal(norm, want) and all(torch.equal(a, b) for a, b in zip(outs, eager)), k


@pytest.mark.parametrize("dtype", [BF, F32])
def test_lists_of_one_launch_and_of_several(ctx, dtype):
    """Sizes on both sides of the limit of a single launch (1024 chunks of 2048
    to 8192 elements, 128 tensors), in turn, twice, with a loss call between."""
    lists = [[1 << 21], [(1 << 21) - 2048, 1, 1], [2049] * 127, [2049] * 129, [(1 << 23) - 4096], [1 << 23, 5], [3]]
    first = {}
    logits, labels = torch.randn(4, 9, 700, device=DEV), torch.zeros(4, 9, dtype=torch.int64, device=DEV)
    logps = torch.empty(4, 9, device=DEV)
    for turn in range(2):
        for i, sizes in enumerate(lists):
            ts = tensors(sizes, dtype, seed=i)
            norm = torch.full((3,), -1.0, dtype=torch.float64, device=DEV)
            ctx.grad_norm(ts, norm, max_norm=2.0)
            ctx.token_logps(logits, labels, logps)
            got = norm.cpu().numpy()
            if turn:
                assert np.array_equal(got, first[i]), sizes
                continue
            first[i] = got
            want = lo.grad_norm_ref([t.double().cpu().numpy() for t in ts], 2.0)
            assert np.abs(got - want).max() <= (sum(sizes) + 4) * 2.0 ** -53 * max(want[0], 1.0), sizes
