"""nld_sample against the float64 oracle: equal tokens; probabilities to 2^-24 (their fp32 rounding)
and 2^18 * 2^-45 / total < 2^-26 (the fixed-point weights of a vocabulary of 2^18), 2^-22 together with
room for exp's own rounding."""
import math

import pytest
import torch

from oracle import operators as oop

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def run(x, u, t=None, k=None, p=None, mp=None, prob=True):
    import self_speculation_b200 as nb
    n = x.shape[0]
    f = lambda v, dt=torch.float32: None if v is None else torch.tensor(v, dtype=dt, device="cuda").expand(n).contiguous()  # noqa: E731
    tok = torch.full((n,), -9, dtype=torch.int32, device="cuda")
    pr = torch.full((n,), -9.0, device="cuda") if prob else None
    nb.nld_sample(x if x.is_cuda else x.cuda(), f(u), tok, pr, temperature=f(t), top_k=f(k, torch.int32), top_p=f(p),
                  min_p=f(mp))
    torch.cuda.synchronize()
    return tok.cpu().tolist(), pr.cpu().tolist() if prob else None


def check(x, u, t=None, k=None, p=None, mp=None):
    n = x.shape[0]
    # the numbers as the call gets them: fp32
    at = lambda v, i, off: off if v is None else torch.tensor(v, dtype=torch.float32).expand(n)[i].item()  # noqa: E731
    tok, pr = run(x, u, t, k, p, mp)
    for i in range(n):
        want, prob = oop.sample_token(x[i], at(u, i, 0.0), at(t, i, 1.0), int(at(k, i, 0)), at(p, i, 1.0), at(mp, i, 0.0))
        assert tok[i] == want, (i, tok[i], want)
        assert abs(pr[i] - prob) <= 2.0 ** -22 * prob, (i, pr[i], prob)


def logits(rows, vocab, dtype="f32", seed=0, spread=2.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(rows, vocab, generator=g) * spread).to(DT[dtype])


def us(n, seed=0):
    return torch.rand(n, generator=torch.Generator().manual_seed(seed + 100)).tolist()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("vocab", [1, 2, 33, 1000, 1024, 5000, 20001])
@pytest.mark.parametrize("t,k,p,mp", [(None, None, None, None), (0.7, None, None, None), (1.3, 20, None, None),
                                      (1.0, None, 0.9, None), (0.8, None, None, 0.05), (1.5, 300, 0.95, 0.02),
                                      (1.0, 1, None, None), (1.0, None, 0.0, None), (1.0, None, None, 1.0),
                                      (0.6, 7, 0.3, None)])
def test_filters(dtype, vocab, t, k, p, mp):
    check(logits(6, vocab, dtype, seed=vocab), us(6), t, k, p, mp)


def test_settings_of_each_row():
    n = 24
    x = logits(n, 3001, "f32", seed=1)
    check(x, us(n), t=[0.0, 0.5, 1.0, 2.0] * 6, k=[0, 5, 3001, 9999, -1, 50] * 4,
          p=[1.0, 0.5, 0.9] * 8, mp=[0.0, 0.1] * 12)


@pytest.mark.parametrize("u", [0.0, 0.99999994, 1.0, -1.0, 2.0, float("nan")])
def test_ends_of_u(u):
    x = logits(2, 500, seed=2)
    check(x, [u, u])
    check(x, [u, u], 1.0, 10, 0.9, 0.01)


def test_equal_logits_keep_the_lowest_indexes():
    x = torch.zeros(5, 4097)
    check(x, us(5), k=[7] * 5)
    check(x, us(5), p=[0.5] * 5)
    check(x, us(5), k=[1000] * 5, p=[0.25] * 5)
    x = torch.zeros(4, 3000)
    x[:, ::3] = 1.0
    x[:, 5] = -0.0
    check(x, us(4), k=[1500] * 4)
    check(x, us(4), p=[0.8] * 4)
    check(x, us(4), 1.0, 1200, 0.9, 0.5)


@pytest.mark.parametrize("p", [None, 0.9])
def test_infinities_and_nan(p):
    inf, nan = float("inf"), float("nan")
    rows = torch.tensor([[0.0, -inf, 1.0, -inf, 2.0], [-inf, -inf, -inf, -inf, 3.0], [nan, 1.0, nan, 1.0, -inf],
                         [-inf] * 5, [nan] * 5, [inf, 0.0, inf, 1.0, -inf], [nan, -inf, nan, inf, 5.0]])
    for u in (0.0, 0.3, 0.9):
        check(rows, [u] * 7, 1.0, None, p)
        check(rows, [u] * 7, 0.5, 2, p)
        check(rows, [u] * 7, 0.0, None, p)


@pytest.mark.parametrize("t", [1e-30, 1e-3, 1e6, float("inf"), float("nan"), -1.0])
def test_extreme_temperatures(t):
    x = logits(4, 700, seed=3)
    check(x, us(4), [t] * 4)
    check(x, us(4), [t] * 4, 100, 0.7)


@pytest.mark.parametrize("scale", [1e-30, 1e4, 1e30])
def test_extreme_logits(scale):
    x = logits(4, 700, seed=4) * scale
    check(x, us(4))
    check(x, us(4), 1.0, 100, 0.7)
    check(x, us(4), scale, 300, 0.9)


def test_one_outlier_far_below_and_above():
    x = logits(4, 2000, seed=5)
    x[0, 7] = -1e30
    x[1, 9] = 1e30
    x[2] = x[2].sign() * torch.exp2(torch.randint(-60, 3, (2000,), generator=torch.Generator().manual_seed(1)).float())
    check(x, us(4), p=[0.9] * 4)
    check(x, us(4), k=[100] * 4, p=[0.99] * 4)


@pytest.mark.parametrize("dtype,vocab", [("f32", 151936), ("bf16", 151936), ("f32", 128000)])
def test_whole_vocabularies(dtype, vocab):
    x = logits(6, vocab, dtype, seed=6)
    check(x, us(6), [0.7, 1.0, 1.3, 1.0, 1.0, 0.9], [0, 50, 0, 1000, 60000, 0], [1.0, 1.0, 0.9, 0.95, 0.99, 0.5],
          [0.0, 0.0, 0.0, 0.0, 0.0, 0.01])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_largest_vocabulary(dtype):
    # fp32: slices over the shared memory
    x = logits(3, 1 << 19, dtype, seed=8)
    check(x, us(3), [1.0, 0.8, 1.2], [0, 3000, 0], [1.0, 0.9, 0.97], [0.001, 0.0, 0.0])


@pytest.mark.parametrize("dtype,vocab", [("f32", 8191), ("f32", 16385), ("bf16", 40000), ("f32", 70001)])
def test_rows_at_every_alignment(dtype, vocab):
    # views into one row of numbers, each an element further on
    flat = logits(1, vocab + 9, dtype, seed=9)[0].cuda()
    for off in range(9):
        x = flat[off:off + vocab][None]
        check(x, us(1, seed=off), 1.1, 40 if off % 2 else None, 0.95)


def test_flat_and_narrow_distributions():
    # a whole vocabulary in one bin of the first search, and logits around zero
    g = torch.Generator().manual_seed(3)
    x = torch.rand(4, 50000, generator=g) * 1e-3
    x[1] = torch.randn(50000, generator=g) * 1e-30
    x[2] = 7.0 + torch.randint(0, 40, (50000,), generator=g) * 2.0 ** -20
    check(x, us(4), 1.0, [30000, 0, 20000, 0], [0.4, 0.7, 1.0, 0.31])
    check(x, us(4), [1e-4, 1e-31, 1e-6, 1e30], [0, 500, 0, 100], [0.8, 1.0, 0.5, 0.5], 0.1)


def test_strided_rows_side_stream_graph_and_no_prob():
    import self_speculation_b200 as nb
    big = logits(5, 4000, seed=7).cuda()
    x = big[:, 1:3001]                     # rows 4000 apart, 4-byte aligned only
    u = us(5)
    check(x.cpu(), u, 0.9, 40, 0.9)
    tok, _ = run(x, u, 0.9, 40, 0.9, prob=False)
    want, _ = run(x.cpu(), u, 0.9, 40, 0.9)
    assert tok == want
    ut = torch.tensor(u, device="cuda")
    k = torch.full((5,), 40, dtype=torch.int32, device="cuda")
    out = torch.zeros(5, dtype=torch.int32, device="cuda")
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        nb.nld_sample(x, ut, out, top_k=k)
    st.synchronize()
    first = out.cpu().tolist()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        nb.nld_sample(x, ut, out, top_k=k)
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert out.cpu().tolist() == first == run(x, u, k=40)[0]


def test_frequencies_follow_the_probabilities():
    """u on an even grid gives each kept token its share of the grid, to one step at either end."""
    x = logits(1, 50, seed=8)
    n = 2000
    u = [(i + 0.5) / n for i in range(n)]
    tok, pr = run(x.expand(n, 50).contiguous(), u, k=5)
    w = torch.softmax(torch.topk(x[0].double(), 5).values, 0)
    for i, t in enumerate(torch.topk(x[0], 5).indices.tolist()):
        assert abs(tok.count(t) - n * w[i].item()) <= 1


def test_refusals():
    import self_speculation_b200 as nb
    x = torch.zeros(2, 10, device="cuda")
    u, tok = torch.zeros(2, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")
    nb.nld_sample(x, u, tok)
    for a in ((x.cpu(), u, tok), (x.half(), u, tok), (x[0], u, tok), (x, u[:1], tok), (x, u, tok.long()),
              (x.t(), u, tok)):
        with pytest.raises(ValueError):
            nb.nld_sample(*a)
    with pytest.raises(ValueError):
        nb.nld_sample(x, u, tok, top_k=u)
    torch.cuda.synchronize()
