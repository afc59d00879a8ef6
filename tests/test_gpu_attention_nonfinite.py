"""NaN, infinities, scores and weights far out of the ordinary in nld_attention_q8 and nld_attention_shared: what the
definition makes of them, alike for small and wide query tiles, with and without splits of the keys.

Rows are worked on apart, so a row without such a number has the bits of the same call without any."""
import math

import pytest
import torch

import test_gpu_attention_q8 as q8
import test_gpu_attention_shared as shared

pytestmark = pytest.mark.gpu

HQ, HKV = 8, 4

# keys of one sequence: a page, several streams, splits; 1 row (small tiles) and 40 rows (wide ones)
SHAPES = [(m, n) for m in (1, 40) for n in (0, 64, 128, 900)]
# (prefix, own keys): one page of either; splits of the prefix; none
SHARED_SHAPES = [(m, p, n) for m in (1, 40) for p, n in ((1, 0), (65, 64), (512, 300), (2200, 5), (0, 130))]
RUNS = (33, 3137, 20, 10)   # rows, prefix, own keys, sequences: a prefix pass in runs of pages (HKV = HQ = 53)


def q8_at(m, n):
    return q8.make([n], m, HQ, HKV, seed=m + n)


def shared_at(m, p, n):
    return shared.make(p, [n], m, HQ, HKV, seed=m + p + n)


def poison_keys(s, pages, first, end, head):
    """NaN in the K rows first..end-1 of a list of pages."""
    j = torch.arange(first, end)
    if s["pool"].dtype == torch.bfloat16:
        s["pool"][pages[j // 64].long(), 0, head, j % 64, 5] = float("nan")
    else:
        s["pool"].view(torch.uint8)[pages[j // 64].long(), 0, head, j % 64, 5] = 0xff


def only_rows_are_nan(out, clean, bad):
    """bad: truth value of each (sequence, row, head)."""
    out, clean = out.float(), clean.float()
    assert out[bad].isnan().all(), out[bad]
    assert torch.equal(out[~bad], clean[~bad])


def poison_query(s, value, at):
    s["q"][at][3] = value
    bad = torch.zeros(s["q"].shape[:3], dtype=torch.bool)
    bad[at] = True
    return bad


@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("m,n", SHAPES)
def test_q8_query(m, n, value):
    s = q8_at(m, n)
    clean = q8.run(s, m)
    bad = poison_query(s, value, (0, m // 2, 5))
    only_rows_are_nan(q8.run(s, m), clean, bad)


@pytest.mark.parametrize("m,p,n", SHARED_SHAPES)
def test_shared_query(m, p, n):
    s = shared_at(m, p, n)
    clean = shared.run(s, m)
    bad = poison_query(s, float("nan"), (0, m // 2, 5))
    only_rows_are_nan(shared.run(s, m), clean, bad)


def test_shared_query_with_infinities():
    """Every key's score is -inf: 0 / 0."""
    for m in (1, 40):
        s = shared_at(m, 512, 300)
        s["pool"][..., 3] = s["pool"][..., 3].abs() + 1     # (NaN slots stay)
        clean = shared.run(s, m)
        bad = poison_query(s, float("-inf"), (0, m // 2, 5))
        only_rows_are_nan(shared.run(s, m), clean, bad)


def head_rows(s, head):
    bad = torch.zeros(s["q"].shape[:3], dtype=torch.bool)
    bad[:, :, head * HQ // HKV:(head + 1) * HQ // HKV] = True
    return bad


@pytest.mark.parametrize("m,n", SHAPES)
def test_q8_first_new_key(m, n):
    """At a page's start it is the only key of a stream, or of a key group, that the first row sees."""
    s = q8_at(m, n)
    clean = q8.run(s, 1)
    poison_keys(s, s["table"][0], n, n + 1, 2)
    only_rows_are_nan(q8.run(s, 1), clean, head_rows(s, 2))


@pytest.mark.parametrize("m,max_len", [(1, 512), (16, 512), (40, 512), (40, 64 * 9)])
def test_q8_keys_of_a_split(m, max_len):
    """Of 3 pages the last, with a split of its own."""
    s = q8_at(m, 128)
    s["table"] = torch.cat((s["table"], s["table"].new_zeros(1, 8)), 1).contiguous()
    clean = q8.run(s, 1, max_len=max_len)
    poison_keys(s, s["table"][0], 128, 128 + m, 1)
    only_rows_are_nan(q8.run(s, 1, max_len=max_len), clean, head_rows(s, 1))


@pytest.mark.parametrize("m,p,n", [a for a in SHARED_SHAPES if a[1]])
@pytest.mark.parametrize("where", ["last key of the prefix", "last half of the prefix", "first new key"])
def test_shared_keys(m, p, n, where):
    s = shared_at(m, p, n)
    clean = shared.run(s, 1)
    if where == "first new key":
        poison_keys(s, s["table"][0], n, n + 1, 2)
    else:
        poison_keys(s, s["sp"], p - 1 if where[5] == "k" else (p + 63) // 128 * 64, p, 2)
    only_rows_are_nan(shared.run(s, 1), clean, head_rows(s, 2))


def test_shared_runs_of_pages():
    m, p, n, batch = RUNS
    s = shared.make(p, [n] * batch, m, 53, 53, seed=1)
    clean = shared.run(s, 1)
    bad = poison_query(s, float("nan"), (batch - 1, 7, 50))
    only_rows_are_nan(shared.run(s, 1), clean, bad)
    s = shared.make(p, [n] * batch, m, 53, 53, seed=1)
    poison_keys(s, s["sp"], 64, p, 20)
    bad = torch.zeros(batch, m, 53, dtype=torch.bool)
    bad[:, :, 20] = True
    only_rows_are_nan(shared.run(s, 1), clean, bad)


VANISHING = [(100, 70), (100, 5), (900, 70), (900, 470), (900, 700)]   # cached keys, the one whose V is not finite


def check_vanishing(out):
    head = slice(2 * HQ // HKV, 3 * HQ // HKV)
    assert not torch.isfinite(out[:, head, 5]).any()
    assert torch.isfinite(out[:, head, 6:]).all() and torch.isfinite(out[:, :head.start]).all()


@pytest.mark.parametrize("m", [1, 40])
@pytest.mark.parametrize("n,at", VANISHING)
def test_q8_visible_value_of_vanishing_weight(m, n, at):
    """Key 3's weight is about 2^200 times the others': that of NaN rounds to 0, in the stream, key group or split of
    key 3 or in another, and 0 times NaN is NaN."""
    s = q8.make([n], m, HQ, HKV, seed=n)
    raw = s["pool"].view(torch.uint8)
    raw[s["table"][0, 0], 0, :, 3, 7] = 0x7e     # 448
    raw[s["table"][0, at // 64], 1, 2, at % 64, 5] = 0xff
    s["ks"] = torch.ones(HKV)
    s["q"].zero_()
    s["q"][..., 7] = 200 * math.log(2) * 128 ** 0.5 / 448
    check_vanishing(q8.run(s, 1)[0].float())


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("m", [1, 40])
@pytest.mark.parametrize("n,at", VANISHING)
def test_shared_visible_value_of_vanishing_weight(m, n, at, value):
    """The same; an infinity gives NaN or an infinity."""
    p = n // 2
    s = shared.make(p, [n - p], m, HQ, HKV, seed=n)
    s["pool"][s["sp"][0], 0, :, 3, 7] = 448
    page = s["sp"][at // 64] if at < p else s["table"][0, (at - p) // 64]
    s["pool"][page, 1, 2, (at if at < p else at - p) % 64, 5] = value
    s["q"].zero_()
    s["q"][..., 7] = 200 * math.log(2) * 128 ** 0.5 / 448
    check_vanishing(shared.run(s, 1)[0].float())


@pytest.mark.parametrize("m", [1, 16, 40])
@pytest.mark.parametrize("nats", [8.0, 17.0, 20.0])
def test_q8_many_keys_of_little_weight(m, nats):
    """The row's likeliest key has a V of zeros, n others e^-nats of its weight and a V of ones: o = n e^-nats /
    (1 + n e^-nats) comes from weights that fp16 alone holds badly (17 nats are 2^-24.5).

    The probabilities go in as fp16 of 2^15 p or less, 2^11 p at least for the likeliest key: off by 2^-11 of each, and
    by 2^-36 of the likeliest's each: 2^-11 o + n 2^-36; the scores by d = 136 2^-24 A (A the largest sum |q k| scale), and
    ex2's 2^-22 beside it, which moves o by 2 (d + 2^-22) o; sums in fp32 n 2^-23 o; the output 2^-8 o."""
    n = 3000
    s = q8.make([n], m, HQ, HKV, seed=m)
    j = torch.arange(n + m)
    rows = torch.zeros(n + m, 2, HKV, 128)
    rows[:, 1] = 1.0
    rows[100, 0, :, 7] = 8.0
    rows[100, 1] = 0.0
    s["pool"].view(torch.uint8)[s["table"][0, j // 64].long(), :, :, j % 64] = rows.to(torch.float8_e4m3fn).view(torch.uint8)
    s["ks"], s["vs"] = torch.ones(HKV), torch.full((HKV,), 3.0)
    s["q"].zero_()
    s["q"][..., 7] = nats * 128 ** 0.5 / 8
    score = float(s["q"][0, 0, 0, 7].double()) * 8 * 128 ** -0.5      # of the likeliest key, the others' being 0
    others = (n + torch.arange(m)).double()                         # that row i sees
    little = others * torch.exp(torch.tensor(-score, dtype=torch.float64))
    want = 3 * (little / (1 + little))[:, None, None]
    tol = want * (2.0 ** -8 + 2.0 ** -11 + 2 * (136 * 2.0 ** -24 * score + 2.0 ** -22) + n * 2.0 ** -23) + 3 * n * 2.0 ** -36
    got = q8.run(s, 1)[0].double()
    assert ((got - want).abs() <= tol).all(), (got[0, 0, 0], want[0], tol[0])


# scores of 2^(size - 4) and more, where fp32's step comes to be far over 1
@pytest.mark.parametrize("size", [20, 24, 27, 33, 40, 80])
@pytest.mark.parametrize("m", [1, 16, 40])
@pytest.mark.parametrize("at", [0, 70, 899])
def test_huge_scores_leave_the_likeliest_key(m, size, at):
    """One key is aligned with the queries, the others' products are lower by a quarter of its own, which is
    64 2^12 / sqrt(128) nats at least: o is that key's V row, off by the output's rounding 2^-8, that of its P, 2^-11 (bf16:
    2^-8), and ex2's 2^-22, the fp32 scales' and quotient's 2^-21."""
    g = torch.Generator().manual_seed(size + at)
    x = torch.randn(128, generator=g).sign()
    keys = torch.randn(900 + m, HKV, 128, generator=g).to(torch.float8_e4m3fn).float()
    keys[at] = 2 * x
    products = (keys @ x).flatten().topk(HKV + 1).values
    assert products[HKV - 1] == 256 and products[HKV] < 192
    up = torch.linspace(1, 1.5, m * HQ).view(1, m, HQ, 1)            # rows of different sizes
    s = q8.make([900], m, HQ, HKV, seed=1)
    j = torch.arange(900 + m)
    page = s["table"][0, j // 64].long()
    s["pool"].view(torch.uint8)[page, 0, :, j % 64] = keys.to(torch.float8_e4m3fn).view(torch.uint8)
    s["ks"] = torch.full((HKV,), 2.0 ** (size - 8))
    s["q"] = (up * x).to(torch.bfloat16)
    want = s["pool"][page[at], 1, :, at % 64].float() * s["vs"][:, None]
    want = want.repeat_interleave(HQ // HKV, 0)
    got = q8.run(s, 1)[0].float()
    assert ((got - want).abs() <= want.abs() * (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -20)).all(), got[:, :, 0]
    s = shared.make(700, [200], m, HQ, HKV, seed=1)
    for pages, first, end in ((s["sp"], 0, 700), (s["table"][0], 700, 900 + m)):
        j = torch.arange(end - first)
        s["pool"][pages[j // 64].long(), 0, :, j % 64] = keys[first:end].to(torch.bfloat16)
    s["q"] = (up * x * 2.0 ** (size - 8)).to(torch.bfloat16)
    pages, j = (s["sp"], at) if at < 700 else (s["table"][0], at - 700)
    want = s["pool"][pages[j // 64].long(), 1, :, j % 64].float().repeat_interleave(HQ // HKV, 0)
    got = shared.run(s, 1)[0].float()
    assert ((got - want).abs() <= want.abs() * (2 * 2.0 ** -8 + 2.0 ** -20)).all(), got[:, :, 0]
