"""Verification of drafted tokens against the oracle (needs a gfx950 GPU).

Tokens and counts are equal: decisions are binary64 on both sides.  A
log-probability lp = (z - max) / T - log S is formed in binary64 from
exponentials good to 2^-22 at least and stored in fp32: 2^-22 + 2^-24 |lp| and
2^-22 of the scores' distance.
"""
import numpy as np
import pytest
import torch

from newton_schulz_amd import Context, verify_workspace_bytes
from oracle import linear8_oracle as lo

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def ctx():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    c = Context(DEV, 16 << 20)
    yield c
    c.close()


def make(batch, draft, vocab, dtype, seed, noise=0.7, with_draft=True, t=1.0, ragged=False, pad=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(batch, draft + 1, vocab + pad, generator=g) * 2
    if vocab > 8:
        x.scatter_add_(-1, torch.randint(vocab, (batch, draft + 1, 4), generator=g), torch.rand(batch, draft + 1, 4, generator=g) * 8)
    d = x[:, :draft] + noise * torch.randn(batch, draft, vocab + pad, generator=g)
    x, d = x.to(dtype), d.to(dtype)
    z = d[..., :vocab].float()
    if with_draft and t:
        z = z / t - torch.log(-torch.log(torch.rand(z.shape, generator=g).clamp(min=1e-30)))
    y = z.argmax(-1) if draft else torch.zeros(batch, 0, dtype=torch.int64)
    if ragged:
        y[torch.rand(batch, draft, generator=g) < 0.25] = -1
    u = torch.rand(batch, draft + 1, generator=g)
    return x.to(DEV)[..., :vocab], y.to(DEV), (d.to(DEV)[..., :vocab] if with_draft else None), u.to(DEV)


def call(ctx, x, y, d, u, t, logps=True, stream=None):
    b, k1, _ = x.shape
    tokens = torch.full((b, k1), -7, dtype=torch.int64, device=DEV)
    accepted = torch.full((b,), -7, dtype=torch.int64, device=DEV)
    lp = torch.full((b, k1), 7.0, device=DEV) if logps else None
    ctx.verify_draft(x, y, tokens, accepted, draft_logits=d, uniforms=u, logps=lp, temperature=t, stream=stream)
    return tokens, accepted, lp


def check(ctx, x, y, d, u, t):
    tokens, accepted, lp = call(ctx, x, y, d, u, t)
    ref = [None if v is None else v.double().cpu().numpy() if v.is_floating_point() else v.cpu().numpy() for v in (x, y, d, u)]
    want = lo.verify_ref(*ref, t)
    assert np.array_equal(accepted.cpu().numpy(), want[1]), (accepted.tolist(), want[1].tolist())
    assert np.array_equal(tokens.cpu().numpy(), want[0])
    got = lp.double().cpu().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(want[2]))
    ok = ~np.isnan(want[2])
    assert (np.abs(got - want[2])[ok] <= (2.0 ** -22 + 2.0 ** -21 * np.abs(want[2]))[ok]).all()
    return want


SHAPES = [  # batch, draft, vocab, pad
    (1, 0, 1, 0), (1, 1, 1, 0), (3, 1, 2, 1), (2, 4, 7, 0), (5, 3, 8, 0), (4, 2, 63, 2), (3, 5, 64, 0), (2, 1, 65, 1), (8, 4, 257, 0),
    (1, 4, 1000, 0), (16, 2, 4099, 0), (3, 8, 16384, 8), (2, 3, 33003, 5), (4, 7, 50257, 0), (2, 5, 151936, 0), (1, 1, 1 << 19, 0),
    (70, 1, 300, 0), (1, 40, 999, 0), (9, 0, 20011, 0), (300, 2, 40, 0),
]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("t", [1.0, 0.6, 0.0])
def test_with_a_draft_model(ctx, dtype, shape, t):
    b, k, v, pad = shape
    check(ctx, *make(b, k, v, dtype, b + k + v, t=t, pad=pad), t)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("shape", SHAPES[3::2])
@pytest.mark.parametrize("t", [1.3, 0.0])
def test_deterministic_drafts_of_different_lengths(ctx, dtype, shape, t):
    b, k, v, pad = shape
    check(ctx, *make(b, k, v, dtype, b + k + v, t=t, pad=pad, with_draft=False, ragged=True), t)


def test_target_and_draft_of_different_types_and_strides(ctx):
    x, y, d, u = make(6, 3, 700, F32, 2, ragged=True)
    wide = torch.empty(3, 6, 701, dtype=BF, device=DEV)
    seq_major = wide.transpose(0, 1)[..., :700]  # rows of one place lie together
    seq_major.copy_(d)
    check(ctx, x, y, seq_major, u, 0.9)
    # one row of scores for every place of every sequence
    check(ctx, x[:1, :1].expand(6, 4, 700), y, seq_major, u, 0.9)


def test_everything_is_kept(ctx):
    x, y, _, u = make(9, 6, 3001, BF, 3)
    want = check(ctx, x, y, x[:, :6], u, 1.0)  # the draft is the target: u q < p whatever u
    assert (want[1] == 6).all()


def test_first_and_last_tokens(ctx):
    """u at and past its ends, and numbers that are none."""
    x, y, d, u = make(7, 2, 500, F32, 4)
    u[:, :2] = 1.0  # refuses nearly everywhere
    for i, v in enumerate((0.0, 1.0 - 2.0 ** -24, 1.0, 2.0, float("nan"), -1.0, float("inf"))):
        u[i, 2] = v
    check(ctx, x, y, d, u, 1.0)
    u[:, 0] = float("nan")
    check(ctx, x, y, d, u, 1.0)


def test_masked_scores(ctx):
    """-infinity in both rows, rows of one token, weights that leave nothing."""
    inf = float("inf")
    x, y, d, u = make(8, 3, 300, F32, 5)
    x[0, 0, 10:] = -inf                      # target: ten tokens
    d[1, 0, 5:] = -inf                       # draft: five
    x[2, 0] = -inf
    x[2, 0, 77] = 3.0                        # one token
    x[3, 1] = d[3, 1]                        # equal rows: refused only by u = 1, nothing left over
    u[3, :2] = torch.tensor([0.0, 1.0])
    x[4] = torch.finfo(F32).min              # the type's lowest value everywhere: uniform
    x[5, 0, :299] = torch.finfo(F32).min
    x[6, 0, y[6, 0]] = -inf                  # the drafted token is impossible
    y[7, 0] = 300                            # names no token
    y[7, 1] = 1 << 40
    check(ctx, x, y, d, u, 1.0)
    check(ctx, x, y, None, u, 1.0)
    check(ctx, x, y, d, u, 0.0)


@pytest.mark.parametrize("vocab", [300, 3001, 40000])
def test_the_lowest_number_passes_over_masked_tokens(ctx, vocab):
    """u = 0 takes the first token with any probability, u = 1 the last."""
    x, y, d, u = make(6, 1, vocab, F32, 8)
    x[..., :9] = x[..., -5:] = -float("inf")
    d[:, :, 20:30] = -float("inf")
    x[1, :, 12] = -2000.0  # as good as masked, in 64 bits too
    u[:, 0] = 1.0
    u[::2, 1], u[1::2, 1] = 0.0, 1.0
    for scores in (d, None):
        for end in (0.0, 1.0):
            u[:, 1] = end
            tokens = check(ctx, x, y, scores, u, 1.0)[0]
            assert ((tokens < 0) | (tokens >= 9) & (tokens < vocab - 5)).all()


@pytest.mark.parametrize("t", [1.0, 0.0])
@pytest.mark.parametrize("vocab", [40, 3001, 40000])
def test_rows_without_a_distribution(ctx, vocab, t):
    inf, nan = float("inf"), float("nan")
    x, y, d, u = make(9, 2, vocab, F32, 6, noise=0.05)
    u[:, :2] = 0.01
    x[0, 0, 7] = nan
    x[1, 1, vocab - 1] = inf
    x[2, 0] = -inf
    x[3, 2, 0] = nan
    d[4, 0, 3] = nan
    d[5, 0] = -inf
    d[6, 1, 9] = inf
    x[7, 1] = nan
    check(ctx, x, y, d, u, t)


def test_ties_go_to_the_lowest_token(ctx):
    x = torch.zeros(4, 3, 1037, dtype=BF, device=DEV)
    x[1, :, 1000:] = 4.0
    x[2, :, 513] = x[2, :, 1036] = 2.0
    y = torch.tensor([[0, 0], [1000, 1001], [1036, 513], [1, 0]], device=DEV)
    tokens, accepted, _ = call(ctx, x, y, None, None, 0.0)
    assert tokens.tolist() == [[0, 0, 0], [1000, 1000, -1], [513, -1, -1], [0, -1, -1]]
    assert accepted.tolist() == [2, 1, 0, 0]


@pytest.mark.parametrize("with_draft", [True, False])
def test_tokens_follow_the_target(ctx, with_draft):
    """First tokens of 60000 verifications are distributed as the target is:
    chi-square over 12 tokens, 11 degrees of freedom, below its 1 - 1e-6
    quantile 51."""
    n, v = 60000, 12
    g = torch.Generator(device=DEV).manual_seed(8)
    z = torch.randn(1, 2, v, generator=g, device=DEV) * 1.5
    zd = torch.randn(1, 1, v, generator=g, device=DEV) * 1.5
    if with_draft:
        y = (zd.expand(n, 1, v) - torch.log(torch.empty(n, 1, v, device=DEV).exponential_(generator=g))).argmax(-1)
    else:
        y = torch.full((n, 1), 3, device=DEV)
    u = torch.rand(n, 2, generator=g, device=DEV)
    tokens, accepted, _ = call(ctx, z.expand(n, 2, v), y, zd.expand(n, 1, v) if with_draft else None, u, 1.0)
    want = torch.softmax(z[0, 0].double(), -1).cpu().numpy() * n
    seen = np.bincount(tokens[:, 0].cpu().numpy(), minlength=v)
    assert ((seen - want) ** 2 / want).sum() < 51


def test_streams_graphs_and_no_log_probabilities(ctx):
    x, y, d, u = make(4, 3, 50257, BF, 11)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a = call(ctx, x, y, d, u, 1.0)
    torch.cuda.synchronize()
    b = call(ctx, x, y, d, u, 1.0, logps=False, stream=side)
    side.synchronize()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    tokens, accepted, lp = torch.empty_like(a[0]), torch.empty_like(a[1]), torch.empty_like(a[2])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        ctx.verify_draft(x, y, tokens, accepted, draft_logits=d, uniforms=u, logps=lp, stream=side)
    for i in range(4):
        nx, ny, nd, nu = make(4, 3, 50257, BF, 20 + i)
        for old, new in ((x, nx), (y, ny), (d, nd), (u, nu)):
            old.copy_(new)
        want = call(ctx, x, y, d, u, 1.0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(tokens, want[0]) and torch.equal(accepted, want[1]) and torch.equal(lp, want[2])


def test_more_sequences_than_a_launch_counts(ctx):
    """Launches are cut where the counters of their sequences would not fit."""
    c = Context(DEV, 256 << 20)
    x, y, d, u = make(5000, 1, 50, F32, 13)
    check(c, x, y, d, u, 1.0)
    x, y, d, u = make(1, 2, 33000, BF, 14)  # three slices a row
    many = 3000
    args = [v.expand(many, *v.shape[1:]) for v in (x, d)]
    u = torch.rand(many, 3, generator=torch.Generator().manual_seed(1)).to(DEV)
    y = y.expand(many, 2).contiguous()
    tokens, accepted, lp = call(c, args[0], y, args[1], u, 1.0)
    for i in (0, 1, 511, 1024, 2047, 2048, many - 1):
        one = call(c, x, y[:1], d, u[i:i + 1].contiguous(), 1.0)
        assert torch.equal(tokens[i], one[0][0]) and accepted[i] == one[1][0] and torch.equal(lp[i], one[2][0]), i
    c.close()


def test_long_drafts(ctx):
    """A thousand places, refused at once, at the end and not at all."""
    c = Context(DEV, 256 << 20)
    for dtype, vocab in ((F32, 60), (BF, 9000)):
        x, y, d, u = make(4, 1024, vocab, dtype, 15, noise=0.01)
        u[0, :] = 0.5
        u[1, :1024] = 0.0
        u[2, :1024] = 0.0
        u[2, 1023] = 1.5
        want = check(c, x, y, d, u, 1.0)
        assert want[1][1] == 1024 and want[1][2] == 1023
    c.close()


def test_empty_batch_and_exact_workspace(ctx):
    call(ctx, torch.empty(0, 3, 50, device=DEV), torch.empty(0, 2, dtype=torch.int64, device=DEV), None,
         torch.empty(0, 3, device=DEV), 1.0)
    c = Context(DEV, verify_workspace_bytes(5, 4, 151936))
    x, y, d, u = make(5, 4, 151936, BF, 12)
    check(c, x, y, d, u, 1.0)
    c.close()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("shape", [(2, 5, 2047, 1), (2, 5, 2048, 0), (2, 5, 2049, 0), (3, 6, 40, 0), (3, 6, 2048, 3), (4, 11, 500, 0),
                                   (4, 12, 500, 0), (2, 1, 8192, 0), (2, 1, 16385, 0)])
@pytest.mark.parametrize("t", [0.9, 0.0])
def test_either_side_of_one_workgroup(ctx, dtype, shape, t):
    """Rows and vocabularies up to what one workgroup takes, and just beyond, with
    a draft model and without."""
    b, k, v, pad = shape
    check(ctx, *make(b, k, v, dtype, b + k + v + 1, t=t, pad=pad), t)
    check(ctx, *make(b, k, v, dtype, b + k + v + 2, t=t, pad=pad, with_draft=False, ragged=True), t)
