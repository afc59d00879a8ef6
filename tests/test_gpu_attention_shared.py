"""nld_attention_shared against the float64 oracle over the prefix's keys and the sequence's own.

Tolerance of an output o = sum p v / sum p over n keys, V = max |v|: the bf16 output 2^-8 |o|; P
rounded to bf16 2^-8 V; the scores off by d = max sum |q k| scale * 136 * 2^-24, so each p by 2 (d + 2^-22);
sums in fp32 n 2^-23."""
import pytest
import torch

from oracle import operators as oop

pytestmark = pytest.mark.gpu

KERNELS = {"planned": (0, 0), "mma_sync": (2, 0), "tcgen05_2_k64": (3, 64), "tcgen05_2_k128": (3, 128),
           "tcgen05_4_k64": (4, 64), "tcgen05_4_k128": (4, 128)}


@pytest.fixture(params=list(KERNELS))
def attention_kernel(request):
    import self_speculation_b200 as nb
    lib = nb.load_library()
    kernel, tile = KERNELS[request.param]
    assert lib.nld_debug_attention_kernel(kernel) == 0 and lib.nld_debug_attention_tile(tile) == 0
    yield request.param
    assert lib.nld_debug_attention_kernel(0) == 0 and lib.nld_debug_attention_tile(0) == 0


def make(prefix, lens, m, hq, hkv, seed=0, fill=float("nan")):
    g = torch.Generator().manual_seed(seed)
    B = len(lens)
    pps = (max(lens) + m + 63) // 64
    shared = (prefix + 63) // 64
    n_pages = B * pps + shared + 2
    pool = torch.full((n_pages, 2, hkv, 64, 128), fill, dtype=torch.bfloat16)   # slots without a key
    ids = torch.randperm(n_pages, generator=g).to(torch.int32)
    sp, table = ids[:shared].contiguous(), ids[shared:shared + B * pps].view(B, pps).contiguous()
    for pages, n in [(sp, prefix)] + [(table[b], lens[b] + m) for b in range(B)]:
        j = torch.arange(n)
        pool[pages[j // 64].long(), :, :, j % 64] = torch.randn(n, 2, hkv, 128, generator=g).to(torch.bfloat16)
    q = torch.randn(B, m, hq, 128, generator=g).to(torch.bfloat16)
    return dict(q=q, pool=pool, sp=sp, table=table, lens=torch.tensor(lens, dtype=torch.int32), m=m, prefix=prefix)


def run(s, bs, err=None, ws=None, stream=None, out=None, d=None):
    import self_speculation_b200 as nb
    d = d or {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in s.items()}
    B, m, hq, _ = s["q"].shape
    if out is None:
        out = torch.full(s["q"].shape, float("nan"), dtype=torch.bfloat16, device="cuda")
    if ws is None:
        ws = torch.full((nb.nld_attention_shared_workspace_size(B, m, hq),), 0xff, dtype=torch.uint8, device="cuda")
    nb.nld_attention_shared(d["q"], d["pool"], d["sp"], s["prefix"], d["table"], d["lens"], bs,
                            int(s["lens"].max()) + m, out, ws, err=err, stream=stream)
    torch.cuda.synchronize()
    return out.cpu()


def check(s, out, bs, seqs=None):
    B, m, _, _ = s["q"].shape
    k0, v0 = oop.paged_rows(s["pool"], s["sp"].tolist(), s["prefix"])
    for b in seqs if seqs is not None else range(B):
        k, v = oop.paged_rows(s["pool"], s["table"][b].tolist(), int(s["lens"][b]) + m)
        k, v = torch.cat((k0, k)), torch.cat((v0, v))
        want = oop.block_causal_attention(s["q"][b], k, v, bs)
        q = s["q"][b].double()
        A = (q.abs().flatten(0, 1) @ k.abs().amax(1).transpose(0, 1)).max().item() * 128 ** -0.5
        V, n = v.abs().max().item(), k.shape[0]
        tol = 2.0 ** -8 * want.abs() + V * (2.0 ** -8 + 2 * (A * 136 * 2.0 ** -24 + 2.0 ** -22) + n * 2.0 ** -23)
        d = (out[b].double() - want).abs()
        assert (d <= tol).all(), (b, (d - tol).max().item(), d.max().item())


# prefixes that end inside a page, at its end, of one key; own parts without a cached key; blocks
@pytest.mark.parametrize("prefix,lens,m,bs,hq,hkv", [
    (1, [0], 1, 1, 4, 4), (64, [0, 63, 64], 1, 1, 32, 8), (100, [5, 70], 33, 1, 8, 2), (200, [10] * 5, 32, 32, 10, 2),
    (333, [0, 129], 16, 8, 32, 8), (65, [1] * 40, 1, 1, 40, 8)])
def test_shapes(attention_kernel, prefix, lens, m, bs, hq, hkv):
    s = make(prefix, lens, m, hq, hkv, seed=prefix)
    check(s, run(s, bs), bs)


@pytest.mark.parametrize("prefix,lens,m,bs", [(3000, [100, 7, 511], 1, 1), (2111, [300, 64], 32, 32)])
def test_longer(prefix, lens, m, bs):
    s = make(prefix, lens, m, 32, 8, seed=9)
    check(s, run(s, bs), bs)


def test_without_a_prefix():
    import self_speculation_b200 as nb
    s = make(0, [100, 3], 4, 8, 2, seed=1)
    want = run(s, 1)
    check(s, want, 1)
    d = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in s.items()}
    out = torch.empty_like(d["q"])
    nb.nld_attention_shared(d["q"], d["pool"], None, 0, d["table"], d["lens"], 1, 104, out, None)
    assert torch.equal(out.cpu(), want)


def test_equals_attention_over_the_whole_sequence():
    """One sequence whose prefix is a whole number of pages is nld_attention over all of them."""
    import self_speculation_b200 as nb
    s = make(256, [90], 8, 32, 8, seed=2, fill=0.0)
    got = run(s, 1)
    table = torch.cat((s["sp"], s["table"][0])).view(1, -1).cuda()
    out = torch.empty(s["q"].shape, dtype=torch.bfloat16, device="cuda")
    nb.nld_attention(s["q"].cuda(), s["pool"].cuda(), table, torch.tensor([346], dtype=torch.int32).cuda(), 1, 354, out)
    torch.cuda.synchronize()
    # each is within V (2^-8 + ..) + 2^-8 |o| of the exact value; V < 6 over these normal numbers
    assert (got.float() - out.cpu().float()).abs().max() <= 2 * 6 * (2.0 ** -8 + 2.0 ** -9)


def test_repeated_calls_identical_and_reused_workspace():
    import self_speculation_b200 as nb
    s = make(500, [20, 300, 7], 1, 32, 8, seed=3)
    ws = torch.empty(nb.nld_attention_shared_workspace_size(3, 1, 32), dtype=torch.uint8, device="cuda")
    a = run(s, 1, ws=ws)
    b = run(make(700, [5, 5, 5], 1, 32, 8, seed=4), 1, ws=ws)
    assert torch.equal(run(s, 1, ws=ws), a) and not torch.equal(a, b)


def test_side_stream_and_graphs_in_turn():
    """Two captured calls share one workspace and run one after the other."""
    import self_speculation_b200 as nb
    one, two = make(700, [20, 3], 1, 32, 8, seed=5), make(130, [64, 1], 1, 32, 8, seed=6)
    want = run(one, 1), run(two, 1)
    st = torch.cuda.Stream()
    ws = torch.empty(nb.nld_attention_shared_workspace_size(2, 1, 32), dtype=torch.uint8, device="cuda")
    dev, outs, graphs = [], [], []
    for s in (one, two):
        d = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in s.items()}
        out = torch.empty_like(d["q"])
        torch.cuda.synchronize()
        with torch.cuda.stream(st):
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=st):
                nb.nld_attention_shared(d["q"], d["pool"], d["sp"], s["prefix"], d["table"], d["lens"], 1,
                                        int(s["lens"].max()) + 1, out, ws)
        dev.append(d), outs.append(out), graphs.append(graph)
    with torch.cuda.stream(st):
        for _ in range(3):
            for graph in graphs:
                graph.replay()
    st.synchronize()
    assert torch.equal(outs[0].cpu(), want[0]) and torch.equal(outs[1].cpu(), want[1])


def test_clamped_length_is_flagged():
    s = make(100, [64, 60], 1, 8, 2, seed=7, fill=0.0)
    good = s["lens"].clone()
    s["lens"][0] = -3
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = run(s, 1, err=err)
    assert int(err) == 1
    s["lens"] = good
    check(s, out, 1, seqs=[1])


def test_refusals():
    import self_speculation_b200 as nb
    s = make(100, [10], 1, 4, 2)
    d = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in s.items()}
    out = torch.empty_like(d["q"])
    ws = torch.empty(nb.nld_attention_shared_workspace_size(1, 1, 4), dtype=torch.uint8, device="cuda")

    def call(prefix=100, **kw):
        a = {**d, "out": out, "ws": ws, **kw}
        nb.nld_attention_shared(a["q"], a["pool"], a["sp"], prefix, a["table"], a["lens"], 1, 11, a["out"], a["ws"])
    call()
    for kw, exc in ((dict(prefix=129), nb.NldError), (dict(ws=ws[:-1]), nb.NldError), (dict(ws=None), nb.NldError),
                    (dict(sp=None), nb.NldError), (dict(pool=d["pool"].float()), ValueError),
                    (dict(sp=d["sp"].cpu()), ValueError), (dict(out=out[:, :, :2]), ValueError)):
        with pytest.raises(exc):
            call(**kw)
    torch.cuda.synchronize()
