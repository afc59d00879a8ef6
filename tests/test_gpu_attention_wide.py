"""Wide query tiles of nld_attention_q8 and nld_attention_shared (33 rows of a kv head and more), and what both
their kernels have to do alike: references that move, NaN in the cache, negative scales, pages outside the
pool.  Against the float64 oracle, with the tolerances of test_gpu_attention_q8 and test_gpu_attention_shared."""
import pytest
import torch

import test_gpu_attention_q8 as q8
import test_gpu_attention_shared as shared
from oracle import operators as oop

pytestmark = pytest.mark.gpu

# rows of a kv head: just over the small tiles, a whole tile, one over, two tiles that do not fill, many
ROWS = [(33, 1, 4, 4), (11, 11, 32, 8), (32, 32, 32, 8), (43, 5, 6, 2), (129, 64, 2, 2), (50, 1, 10, 2), (200, 16, 4, 1)]


@pytest.mark.parametrize("m,bs,hq,hkv", ROWS)
@pytest.mark.parametrize("lens", [[0], [1], [63, 64, 65], [127, 20], [900, 3]])
def test_q8_rows(lens, m, bs, hq, hkv):
    s = q8.make(lens, m, hq, hkv, seed=m + len(lens))
    q8.check(s, q8.run(s, bs), bs)


@pytest.mark.parametrize("prefix,lens,m,bs,hq,hkv", [
    (1, [0], 33, 33, 4, 4), (63, [5], 40, 1, 8, 2), (64, [0, 1, 2, 3, 4, 5, 6, 7, 8], 1, 1, 32, 8), (65, [300, 0], 64, 8, 4, 2),
    (2049, [7] * 9, 1, 1, 8, 2), (2111, [0] * 33, 1, 1, 4, 2), (700, [90] * 70, 1, 1, 8, 4), (129, [64], 129, 129, 2, 2)])
def test_shared_rows(prefix, lens, m, bs, hq, hkv):
    s = shared.make(prefix, lens, m, hq, hkv, seed=prefix)
    shared.check(s, shared.run(s, bs), bs)


# a prefix pass of more query tiles than SMs: CTAs take runs of pages across them, and the own pass (wide, then
# small tiles) adds two or three parts of a row
@pytest.mark.parametrize("prefix,lens,m,bs,hq,hkv,seqs", [
    (4133, [20] * 16, 32, 32, 40, 8, [0, 3, 4, 15]), (3190, [20] * 30, 16, 16, 40, 40, [0, 7, 8, 29]),
    (3137, [0, 70, 5, 64, 0, 1, 2, 3, 4, 9], 33, 1, 53, 53, [0, 4, 9])])
def test_shared_runs_of_pages(prefix, lens, m, bs, hq, hkv, seqs):
    s = shared.make(prefix, lens, m, hq, hkv, seed=prefix)
    out = shared.run(s, bs)
    shared.check(s, out, bs, seqs=seqs)
    assert torch.equal(out, shared.run(s, bs))


def climb(pool, pages, n, raw):
    """Keys whose scores climb page by page (by far more than 2^8 altogether), then fall."""
    j = torch.arange(n)
    c = (0.25 * (j // 64).float()).clamp(max=2.5) - 1.0 - (j > n - 70).float()
    k = pool[pages[j // 64].long(), 0, :, j % 64].float() * 0.2 + c[:, None, None]
    if raw:
        pool.view(torch.uint8)[pages[j // 64].long(), 0, :, j % 64] = k.to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        pool[pages[j // 64].long(), 0, :, j % 64] = k.to(pool.dtype)


@pytest.mark.parametrize("m", [1, 8, 32])
def test_moving_maximum(m):
    s = q8.make([1000], m, 8, 2, seed=m)
    climb(s["pool"], s["table"][0], 1000 + m, True)
    s["q"] = (s["q"].float() * 0.3 + 0.8).to(torch.bfloat16)
    q8.check(s, q8.run(s, m), m)
    s = shared.make(1000, [130], m, 8, 2, seed=m)
    climb(s["pool"], s["sp"], 1000, False)
    s["q"] = (s["q"].float() * 0.3 + 0.8).to(torch.bfloat16)
    shared.check(s, shared.run(s, m), m)


@pytest.mark.parametrize("m", [1, 20])
@pytest.mark.parametrize("zero", ["keys", "queries"])
def test_scores_that_underflow_weigh_all_keys_alike(m, zero):
    """A scale of zero (a head whose keys are all zero), a query of zeros with a tiny scale."""
    s = q8.make([75], m, 8, 2, seed=40 + m, kscale=1e-9 if zero == "queries" else 0.0)
    if zero == "queries":
        s["q"].zero_()
    q8.check(s, q8.run(s, 1), 1)


@pytest.mark.parametrize("m", [1, 32])
def test_negative_scales(m):
    s = q8.make([200], m, 8, 2, seed=20 + m)
    s["ks"], s["vs"] = -s["ks"], s["vs"] * torch.tensor([1.0, -1.0])
    q8.check(s, q8.run(s, 1), 1)


@pytest.mark.parametrize("size", [2.0 ** -60, 2.0 ** 40])
def test_wide_queries_of_any_size(size):
    s = q8.make([70], 20, 8, 2, seed=4, kscale=1.0 / size)
    s["q"] = (s["q"].float() * size).to(torch.bfloat16)
    q8.check(s, q8.run(s, 1), 1)


@pytest.mark.parametrize("size", [2.0 ** 7, 2.0 ** 9, 2.0 ** 12])
def test_wide_queries_with_a_large_element(size):
    """A row's elements below 2^-9 of its largest may each be off by 2^-17 of it: the scores by
    max|q| 2^-17 sum |k| scale."""
    s = q8.make([300], 20, 8, 2, seed=5, kscale=1.0 / size)
    s["q"][..., 77] = torch.copysign(torch.full((), size), s["q"][..., 77].float()).to(torch.bfloat16)
    out = q8.run(s, 1)[0].double()
    k, v = oop.paged_rows(s["pool"], s["table"][0].tolist(), 320)
    k, v = k * s["ks"].double()[:, None], v * s["vs"].double()[:, None]
    q, scale = s["q"][0].double(), 128 ** -0.5
    want = oop.block_causal_attention(s["q"][0], k, v, 1)
    off = q.abs().max().item() * 2.0 ** -17 * k.abs().sum(-1).max().item() * scale
    tol = q8.tolerance(q, k, v, want, scale, 2.0 ** -11, 1.0) + 2 * v.abs().max().item() * off
    assert ((out - want).abs() <= tol).all()


@pytest.mark.parametrize("m", [1, 40])
@pytest.mark.parametrize("which", [0, 1])
def test_nan_in_a_visible_row_comes_out(m, which):
    """K: in every row that sees the key; V: in that dim of those rows."""
    s = q8.make([100], m, 4, 4, seed=30)
    s["pool"].view(torch.uint8)[s["table"][0, 1], which, 2, 100 % 64, 5] = 0xff      # the first new key, kv head 2
    out = q8.run(s, 1)[0].float()
    clean = [h for h in range(4) if h != 2]
    assert torch.isfinite(out[:, clean]).all()
    assert out[:, 2].isnan().all() if which == 0 else (out[:, 2, 5].isnan().all() and torch.isfinite(out[:, 2, 6:]).all())


@pytest.mark.parametrize("m", [1, 40])
def test_pages_outside_the_pool_read_as_zeros(m):
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    s = q8.make([64, 100], m, 8, 2, seed=7)
    s["table"][0, 0], s["table"][0, 1] = 1 << 30, -5
    out = q8.run(s, 1, err=err)
    assert int(err) == 1 and (out[0] == 0).all()     # every V row is 0
    q8.check(s, out, 1, seqs=[1])
    s = shared.make(100, [64, 60], m, 8, 2, seed=7, fill=0.0)
    err.zero_()
    s["table"][0] = torch.tensor([s["pool"].shape[0], -1, 1 << 30, -(1 << 30)], dtype=torch.int32)[:s["table"].shape[1]]
    out = shared.run(s, 1, err=err)
    assert int(err) == 1 and torch.isfinite(out[0].float()).all()
    shared.check(s, out, 1, seqs=[1])


@pytest.mark.parametrize("m", [1, 40])
def test_repeated_calls_and_streams_at_once(m):
    """The same bits every time, from two streams at once too (a workspace each)."""
    import self_speculation_b200 as nb
    s, t = q8.make([800, 100], m, 8, 2, seed=9), shared.make(900, [40, 333], m, 8, 2, seed=9)
    want = q8.run(s, 1), shared.run(t, 1)
    d = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in s.items()}
    e = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in t.items()}
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [(torch.empty_like(d["q"]), torch.empty_like(e["q"])) for _ in streams]
    size = nb.nld_attention_shared_workspace_size(2, m, 8)
    ws = [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in streams]
    torch.cuda.synchronize()
    for _ in range(5):
        for st, (a, b), w in zip(streams, outs, ws):
            with torch.cuda.stream(st):
                nb.nld_attention_q8(d["q"], d["pool"], d["ks"], d["vs"], d["table"], d["lens"], 1, 800 + m, a)
                nb.nld_attention_shared(e["q"], e["pool"], e["sp"], 900, e["table"], e["lens"], 1, 333 + m, b, w)
    torch.cuda.synchronize()
    for a, b in outs:
        assert torch.equal(a.cpu(), want[0]) and torch.equal(b.cpu(), want[1])
