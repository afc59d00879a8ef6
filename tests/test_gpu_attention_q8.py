"""nld_attention_q8 against the float64 oracle on the values that the e4m3 cache stands for.

Tolerance of an output o = sum p v / sum p over n keys, V = max |v|:
  the bf16 output                    2^-8 |o|
  P rounded to fp16                  2^-11 of each p, and 2^-25 where p is below fp16's normal range:
                                     V (2^-11 + n 2^-25), the sum of the p's being at least 1
  the scores                         off by d = A (128 + 8) 2^-24 + A' where A = max sum |q k| scale, and
                                     A' = 128 2^-25 2 max|q| max|k| scale (what fp16 drops of a row's small
                                     elements): each p by a factor e^d, ex2's 2^-22 beside it: 2 V (d + 2^-22)
  sums in fp32                       V n 2^-23
"""
import pytest
import torch

import synth
from oracle import operators as oop

pytestmark = pytest.mark.gpu


def tolerance(q, k, v, o, scale, p_step, q_small):
    """q, k, v float64 rows of one kv head's worth each; o the oracle's output."""
    A = (q.abs().flatten(0, 1) @ k.abs().amax(1).transpose(0, 1)).max().item() * scale
    n, V = k.shape[0], v.abs().max().item()
    d = A * 136 * 2.0 ** -24 + q_small * 128 * 2.0 ** -24 * q.abs().max().item() * k.abs().max().item() * scale
    return 2.0 ** -8 * o.abs() + V * (p_step + n * 2.0 ** -25 + 2 * (d + 2.0 ** -22) + n * 2.0 ** -23)


def make(lens, m, hq, hkv, seed=0, extra=2, kscale=1.0, vscale=1.0):
    g = torch.Generator().manual_seed(seed)
    B = len(lens)
    pps = (max(lens) + m + 63) // 64 + 1
    n_pages = B * pps + extra
    # slots that no row sees hold NaN patterns
    pool = torch.full((n_pages, 2, hkv, 64, 128), 0x7f, dtype=torch.uint8).view(torch.float8_e4m3fn)
    table = torch.randperm(n_pages, generator=g)[:B * pps].view(B, pps).to(torch.int32)
    raw = pool.view(torch.uint8)
    for b, n in enumerate(lens):
        rows = torch.randn(n + m, 2, hkv, 128, generator=g).to(torch.float8_e4m3fn).view(torch.uint8)
        j = torch.arange(n + m)
        raw[table[b, j // 64].long(), :, :, j % 64] = rows
    ks = (0.5 + torch.rand(hkv, generator=g)) * kscale
    vs = (0.5 + torch.rand(hkv, generator=g)) * vscale
    q = torch.randn(B, m, hq, 128, generator=g).to(torch.bfloat16)
    return dict(q=q, pool=pool, ks=ks, vs=vs, table=table, lens=torch.tensor(lens, dtype=torch.int32), m=m)


def run(s, bs, max_len=None, err=None):
    import self_speculation_b200 as nb
    d = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in s.items()}
    out = torch.full(s["q"].shape, float("nan"), dtype=torch.bfloat16, device="cuda")
    if max_len is None:
        max_len = int(s["lens"].max()) + s["m"]
    nb.nld_attention_q8(d["q"], d["pool"], d["ks"], d["vs"], d["table"], d["lens"], bs, max_len, out, err=err)
    torch.cuda.synchronize()
    return out.cpu()


def check(s, out, bs, seqs=None):
    B, m, hq, _ = s["q"].shape
    for b in seqs if seqs is not None else range(B):
        k, v = oop.paged_rows(s["pool"], s["table"][b].tolist(), int(s["lens"][b]) + m)
        k, v = k * s["ks"].double()[:, None], v * s["vs"].double()[:, None]
        want = oop.block_causal_attention(s["q"][b], k, v, bs)
        tol = tolerance(s["q"][b].double(), k, v, want, 128 ** -0.5, 2.0 ** -11, 1.0)
        d = (out[b].double() - want).abs()
        assert (d <= tol).all(), (b, (d - tol).max().item(), d.max().item())


# one token, the smallest batches; several row tiles; heads that do not divide a tile; one kv head for all
@pytest.mark.parametrize("hq,hkv", [(32, 8), (10, 2), (4, 4), (48, 1)])
@pytest.mark.parametrize("lens,m,bs", [([0], 1, 1), ([62, 63, 64, 1], 1, 1), ([0, 127], 2, 1), ([130, 5], 33, 1),
                                       ([700], 32, 32), ([31, 200], 32, 8), ([100], 50, 7)])
def test_shapes(lens, m, bs, hq, hkv):
    s = make(lens, m, hq, hkv, seed=m + len(lens))
    check(s, run(s, bs), bs)


def test_long_and_split():
    s = make([5000, 17], 1, 32, 8, seed=1)
    check(s, run(s, 1), 1)
    # an upper bound far over the lengths, with splits that hold no key
    s2 = make([40], 1, 8, 8, seed=2)
    s2["table"] = torch.cat((s2["table"], s2["table"].new_zeros(1, 200)), 1).contiguous()
    check(s2, run(s2, 1, max_len=200 * 64), 1)


@pytest.mark.parametrize("kscale,vscale", [(1e-3, 1e3), (4.0, 1e-4)])
def test_scales(kscale, vscale):
    s = make([90, 300], 4, 8, 2, seed=3, kscale=kscale, vscale=vscale)
    check(s, run(s, 1), 1)


@pytest.mark.parametrize("size", [2.0 ** -60, 2.0 ** 40])
def test_queries_of_any_size(size):
    """fp16 operands: a row's size is taken out by a power of two."""
    s = make([70], 3, 8, 2, seed=4, kscale=1.0 / size)
    s["q"] = (s["q"].float() * size).to(torch.bfloat16)
    check(s, run(s, 1), 1)


def test_zero_query_row_is_the_mean():
    s = make([9], 1, 4, 4, seed=5)
    s["q"].zero_()
    check(s, run(s, 1), 1)


def test_repeated_calls_identical():
    s = make([3000, 100], 1, 32, 8, seed=6)
    assert torch.equal(run(s, 1), run(s, 1))


def test_clamped_length_and_bad_page_are_flagged():
    s = make([64, 64], 1, 8, 2, seed=7)
    s["lens"][0] = 10000
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = run(s, 1, max_len=65, err=err)
    assert int(err) == 1
    check(s, out, 1, seqs=[1])
    s = make([64, 64], 1, 8, 2, seed=7)
    s["table"][0, 1] = -5
    s["table"][0, 0] = 1 << 30
    err.zero_()
    out = run(s, 1, max_len=65, err=err)
    assert int(err) == 1 and torch.isfinite(out[0].float()).all()
    check(s, out, 1, seqs=[1])


def test_side_stream_and_graph():
    import self_speculation_b200 as nb
    s = make([400, 31], 1, 32, 8, seed=8)
    want = run(s, 1)
    d = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in s.items()}
    out = torch.zeros(s["q"].shape, dtype=torch.bfloat16, device="cuda")
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        nb.nld_attention_q8(d["q"], d["pool"], d["ks"], d["vs"], d["table"], d["lens"], 1, 401, out)
    st.synchronize()
    assert torch.equal(out.cpu(), want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        nb.nld_attention_q8(d["q"], d["pool"], d["ks"], d["vs"], d["table"], d["lens"], 1, 401, out)
    d["lens"][0] = 77
    s["lens"][0] = 77
    graph.replay()
    torch.cuda.synchronize()
    check(s, out.cpu(), 1)


def test_refusals():
    import self_speculation_b200 as nb
    s = make([10], 1, 4, 2)
    d = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in s.items()}
    out = torch.empty_like(d["q"])

    def call(**kw):
        a = {**d, "out": out, **kw}
        nb.nld_attention_q8(a["q"], a["pool"], a["ks"], a["vs"], a["table"], a["lens"], 1, 11, a["out"])
    call()
    for kw in (dict(pool=d["pool"].to(torch.bfloat16)), dict(q=d["q"].float()), dict(out=out.float()), dict(ks=d["ks"][:1]),
               dict(lens=d["lens"].long()), dict(table=d["table"].cpu()), dict(q=d["q"].expand(2, 1, 4, 128))):
        with pytest.raises(ValueError):
            call(**kw)
    torch.cuda.synchronize()
