"""nld_qk_norm_rope against the float64 oracle: norms, rotation, and the rows of the paged cache.

Tolerances, per output o = y c - y' s with y = x inv gain.  In fp32 (step 2^-24 relative): the sum of
hd squares is a chain of hd/lanes terms and log2(lanes) shuffles, 32 + 4 roundings at most, halved
by the root; with rsqrt (2^-22.9), two products, the table's rounding, the rotation's product and sum
o is off by at most 32 * 2^-24 (|y| + |y'|).  A bf16 output adds 2^-8 |o|, an e4m3 one (of o / scale)
2^-4 of it and 2^-10, half its smallest step."""
import pytest
import torch

import synth
from oracle import operators as oop

pytestmark = pytest.mark.gpu

THETA, EPS = 10000.0, 1e-6
DT = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}


def rope_table(n, hd, theta=THETA):
    i = torch.arange(hd // 2, dtype=torch.float64)
    ang = torch.arange(n, dtype=torch.float64)[:, None] * theta ** (-2.0 * i / hd)
    return torch.stack((ang.cos(), ang.sin()), -1).float()


def make(lens, m, hq, hkv, hd, dtype, cache, seed=0, norm=True, rows=None, offset=0):
    g = torch.Generator().manual_seed(seed)
    B = len(lens)
    pps = (max(lens) + m + 63) // 64
    n_pages = B * pps + 2
    s = dict(m=m, lens=torch.tensor(lens, dtype=torch.int32), offset=offset)
    s["qkv"] = (torch.randn(B, m, hq + 2 * hkv, hd, generator=g) * 2).to(DT[dtype])
    s["gq"] = (1 + 0.3 * torch.randn(hd, generator=g)).to(DT[dtype]) if norm else None
    s["gk"] = (1 + 0.3 * torch.randn(hd, generator=g)).to(DT[dtype]) if norm else None
    s["rope"] = rope_table(offset + max(lens) + m, hd)
    s["table"] = torch.randperm(n_pages, generator=g)[:B * pps].view(B, pps).to(torch.int32)
    s["pool"] = torch.full((n_pages, 2, hkv, 64, hd), 7.0).to(DT[cache])
    s["ks"] = 0.01 + 0.02 * torch.rand(hkv, generator=g) if cache == "e4m3" else None
    s["vs"] = 0.01 + 0.02 * torch.rand(hkv, generator=g) if cache == "e4m3" else None
    s["rows"] = torch.tensor(rows, dtype=torch.int32) if rows is not None else None
    s["heads"] = (hq, hkv, hd)
    return s


def run(s, q_out=None):
    import self_speculation_b200 as nb
    hq, hkv, hd = s["heads"]
    d = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in s.items()}
    q, k, v = d["qkv"][:, :, :hq], d["qkv"][:, :, hq:hq + hkv], d["qkv"][:, :, hq + hkv:]
    out = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda") if q_out is None else q_out
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    nb.nld_qk_norm_rope(q, k, v, d["gq"], d["gk"], EPS, d["rope"], d["lens"], out, d["pool"], d["table"],
                        position_offset=s["offset"], rows=d["rows"], k_scale=d["ks"], v_scale=d["vs"], err=err)
    torch.cuda.synchronize()
    return out.cpu(), d["pool"].cpu(), int(err)


def check(s, out, pool):
    hq, hkv, hd = s["heads"]
    qkv = s["qkv"].double()
    step = {torch.bfloat16: 2.0 ** -8, torch.float32: 0.0, torch.float8_e4m3fn: 2.0 ** -4}
    least = 2.0 ** -10 if pool.dtype == torch.float8_e4m3fn else 0.0
    want_pool = s["pool"].double().clone()
    tol_pool = torch.zeros_like(want_pool)
    for b in range(qkv.shape[0]):
        n = s["m"] if s["rows"] is None else int(s["rows"][b])
        first = int(s["lens"][b])
        pos = torch.arange(first, first + n) + s["offset"]
        x = qkv[b, :n]
        wq = oop.norm_rope(x[:, :hq], s["gq"], EPS, pos, THETA)
        wk = oop.norm_rope(x[:, hq:hq + hkv], s["gk"], EPS, pos, THETA)
        # |y| + |y'| of a pair is at most sqrt(2) of its length, which the rotation keeps
        size = lambda o: (o.square() + o.roll(hd // 2, -1).square()).sqrt() * 2 ** 0.5 * 32 * 2.0 ** -24  # noqa: E731
        assert ((out[b, :n].double() - wq).abs() <= size(wq) + step[out.dtype] * wq.abs()).all()
        assert (out[b, n:] == 7.0).all()
        for which, w, t in ((0, wk, size(wk)), (1, x[:, hq + hkv:], torch.zeros_like(wk))):
            sc = s["ks" if which == 0 else "vs"]
            if sc is not None:
                w, t = w / sc.double()[:, None], t / sc.double()[:, None] + 2.0 ** -23 * (w / sc.double()[:, None]).abs()
                w = w.clamp(-448, 448)
            for i in range(n):
                at = (int(s["table"][b, (first + i) // 64]), which, slice(None), (first + i) % 64)
                want_pool[at] = w[i]
                tol_pool[at] = t[i] + step[pool.dtype] * w[i].abs() + least
    d = (pool.double() - want_pool).abs()
    assert (d <= tol_pool).all(), (d - tol_pool).max()


@pytest.mark.parametrize("cache", ["bf16", "f32", "e4m3"])
@pytest.mark.parametrize("dtype,hq,hkv,hd", [("bf16", 32, 8, 128), ("bf16", 4, 4, 64), ("f32", 5, 1, 128), ("f32", 4, 2, 64)])
@pytest.mark.parametrize("lens,m", [([0], 1), ([63, 64, 130], 1), ([5, 61, 0, 190], 33), ([3], 200)])
def test_rows(lens, m, dtype, hq, hkv, hd, cache):
    s = make(lens, m, hq, hkv, hd, dtype, cache, seed=len(lens) + m)
    out, pool, err = run(s)
    assert err == 0
    check(s, out, pool)


def test_no_norm_offset_and_padded_rows():
    s = make([10, 0, 64, 5], 40, 8, 2, 128, "bf16", "bf16", norm=False, rows=[40, 0, 1, 17], offset=4133)
    out, pool, err = run(s)
    assert err == 0
    check(s, out, pool)


def test_far_positions():
    s = make([32767, 100000], 2, 4, 1, 128, "f32", "f32", seed=3)
    out, pool, err = run(s)
    assert err == 0
    check(s, out, pool)


def test_many_tokens_and_determinism():
    s = make([0, 100, 7], 700, 32, 8, 128, "bf16", "e4m3", seed=4)
    out, pool, err = run(s)
    check(s, out, pool)
    out2, pool2, _ = run(s)
    assert torch.equal(out, out2) and torch.equal(pool.view(torch.uint8), pool2.view(torch.uint8))


def test_saturation_and_nan():
    s = make([0], 2, 1, 1, 128, "f32", "e4m3", norm=False)
    s["ks"][:] = s["vs"][:] = 1.0
    v = s["qkv"][0, 0, 2]
    v[:6] = torch.tensor([1e6, -1e6, float("inf"), float("-inf"), float("nan"), 449.0])
    _, pool, _ = run(s)
    got = pool[int(s["table"][0, 0]), 1, 0, 0, :6].float()
    assert got[:4].tolist() == [448.0, -448.0, 448.0, -448.0] and torch.isnan(got[4]) and got[5] == 448.0


def test_in_place_q():
    import self_speculation_b200 as nb
    s = make([9, 70], 3, 8, 2, 128, "bf16", "bf16", seed=6)
    want, pool, _ = run(s)
    d = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in s.items()}
    q = d["qkv"][:, :, :8].contiguous()
    k, v = d["qkv"][:, :, 8:10].contiguous(), d["qkv"][:, :, 10:].contiguous()
    nb.nld_qk_norm_rope(q, k, v, d["gq"], d["gk"], EPS, d["rope"], d["lens"], q, d["pool"], d["table"])
    assert torch.equal(q.cpu(), want) and torch.equal(d["pool"].cpu(), pool)


@pytest.mark.parametrize("what", ["slot", "negative", "position", "page"])
def test_rows_out_of_bounds_are_left_out_and_flagged(what):
    s = make([10, 20], 4, 4, 2, 128, "bf16", "bf16", seed=7)
    if what == "slot":
        s["lens"][1] = 62          # rows 2 and 3 fall behind the one page
    elif what == "negative":
        s["lens"][1] = -2          # rows 0 and 1 fall before it
    elif what == "position":
        s["rope"] = s["rope"][:22].contiguous()   # positions 22 and 23 of sequence 1
    else:
        s["table"][1, 0] = s["pool"].shape[0]
    if what == "slot":
        s["rope"] = rope_table(80, 128)
    out, pool, err = run(s)
    assert err == 1
    live = {"slot": [0, 1], "negative": [2, 3], "position": [0, 1], "page": []}[what]
    for i in range(4):
        assert (out[1, i] == 7.0).all() == (i not in live)
    # sequence 0 is what it is without the bad one
    ref = make([10, 20], 4, 4, 2, 128, "bf16", "bf16", seed=7)
    want, _, _ = run(ref)
    assert torch.equal(out[0], want[0])
    untouched = torch.ones(pool.shape[0], 64, dtype=torch.bool)
    untouched[int(s["table"][0, 0]), 10:14] = False
    if what != "page":
        for i in live:
            untouched[int(s["table"][1, 0]), int(s["lens"][1]) + i] = False
    assert (pool.transpose(1, 3).flatten(2)[untouched] == 7.0).all()


def test_matches_the_models_own_cache_rows():
    """Without norms the rows equal rope_rotate of the same projections, the model's convention."""
    s = make([17], 5, 4, 2, 128, "f32", "f32", norm=False, seed=8)
    out, pool, _ = run(s)
    check(s, out, pool)


def test_refusals():
    import self_speculation_b200 as nb
    s = make([0], 2, 4, 2, 128, "bf16", "e4m3")
    d = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in s.items()}
    q, k, v = d["qkv"][:, :, :4], d["qkv"][:, :, 4:6], d["qkv"][:, :, 6:]
    out = torch.empty(1, 2, 4, 128, dtype=torch.bfloat16, device="cuda")
    call = lambda **kw: nb.nld_qk_norm_rope(  # noqa: E731
        kw.get("q", q), kw.get("k", k), v, kw.get("gq", d["gq"]), d["gk"], kw.get("eps", EPS), d["rope"], d["lens"],
        kw.get("out", out), kw.get("pool", d["pool"]), d["table"], k_scale=kw.get("ks", d["ks"]), v_scale=d["vs"])
    call()
    for kw, exc in ((dict(ks=None), nb.NldError), (dict(gq=None), nb.NldError), (dict(eps=float("nan")), nb.NldError),
                    (dict(q=q.float()), ValueError), (dict(q=q.cpu()), ValueError), (dict(k=k[..., :64]), ValueError),
                    (dict(out=out.float()), ValueError), (dict(pool=d["pool"].half()), ValueError),
                    (dict(q=q.transpose(2, 3)), ValueError)):
        with pytest.raises(exc):
            call(**kw)
    torch.cuda.synchronize()
