"""The same odd lengths, masks and prefixes through every pair of kernels that nld_attention_q8 and nld_attention_shared are
made of: query rows of a kv head (positions x heads; for the prefix pass, of the whole batch) on either side of the small
tiles' 32, and of their 16 for a prefix over 2048 keys.  (Prefix passes in runs of pages: test_gpu_attention_wide.)"""
import pytest
import torch

import test_gpu_attention_q8 as q8
import test_gpu_attention_shared as shared
import test_gpu_qk_norm_rope as write

pytestmark = pytest.mark.gpu

LENS = [[0, 63], [64, 1], [127, 300]]


# rows of a kv head: 1, 31, 32 | 33, 40
@pytest.mark.parametrize("m,hq,hkv", [(1, 2, 2), (31, 2, 2), (8, 8, 2), (33, 2, 2), (8, 10, 2)])
@pytest.mark.parametrize("block", ["causal", "of 3", "whole"])
@pytest.mark.parametrize("lens", LENS)
def test_q8(lens, m, hq, hkv, block):
    bs = {"causal": 1, "of 3": 3, "whole": m}[block]
    s = q8.make(lens, m, hq, hkv, seed=m)
    q8.check(s, q8.run(s, bs), bs)


# rows of the prefix pass and of a sequence's own: 2 and 1, 32 and 16 (small, small; wide, small over 2048 keys) | 64 and 32 (wide,
# small) | 66 and 33 (wide, wide)
@pytest.mark.parametrize("m,hq,hkv", [(1, 2, 2), (4, 8, 2), (8, 8, 2), (33, 2, 2)])
@pytest.mark.parametrize("prefix", [1, 63, 64, 65, 2048, 2049])
@pytest.mark.parametrize("lens", LENS)
def test_shared(lens, prefix, m, hq, hkv):
    s = shared.make(prefix, lens, m, hq, hkv, seed=prefix)
    for bs in (1, 3, m):
        shared.check(s, shared.run(s, bs), bs)


@pytest.mark.parametrize("lens,m,hq,hkv", [([0], 700, 8, 2), ([100, 0], 333, 5, 1)])
def test_prompts(lens, m, hq, hkv):
    """Many query tiles a sequence, some of which cut a position's heads."""
    s = q8.make(lens, m, hq, hkv, seed=m)
    q8.check(s, q8.run(s, 1), 1)
    s = shared.make(70, lens, m, hq, hkv, seed=m)
    shared.check(s, shared.run(s, 1), 1)


@pytest.mark.parametrize("m", [1, 40])
def test_pages_past_4_gb(m):
    """The same call with its pages at the far end of a pool of 4.3 GB (bf16: 8.6 GB)."""
    import self_speculation_b200 as nb
    s, t = q8.make([200], m, 8, 8, seed=3), shared.make(100, [70], m, 8, 8, seed=3)
    want = q8.run(s, 1), shared.run(t, 1)
    far = 33000      # pages of 128 KB
    d = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in s.items()}
    e = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in t.items()}
    for c in (d, e):
        pool = torch.zeros(far + c["pool"].shape[0], *c["pool"].shape[1:], dtype=torch.uint8 if c is d else torch.bfloat16, device="cuda")
        pool = pool.view(c["pool"].dtype)
        (pool.view(torch.uint8) if c is d else pool)[far:] = c["pool"].view(torch.uint8) if c is d else c["pool"]
        c["pool"], c["table"] = pool, c["table"] + far
    out, other = torch.empty_like(d["q"]), torch.empty_like(e["q"])
    ws = torch.empty(nb.nld_attention_shared_workspace_size(1, m, 8), dtype=torch.uint8, device="cuda")
    nb.nld_attention_q8(d["q"], d["pool"], d["ks"], d["vs"], d["table"], d["lens"], 1, 200 + m, out)
    nb.nld_attention_shared(e["q"], e["pool"], e["sp"] + far, 100, e["table"], e["lens"], 1, 70 + m, other, ws)
    torch.cuda.synchronize()
    assert torch.equal(out.cpu(), want[0]) and torch.equal(other.cpu(), want[1])


def test_cache_write_past_4_gb():
    s = write.make([5], 3, 4, 8, 128, "bf16", "e4m3", seed=1)
    out, pool, err = write.run(s)
    far = 33000
    import self_speculation_b200 as nb
    d = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in s.items()}
    big = torch.zeros(far + pool.shape[0], *pool.shape[1:], dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    big.view(torch.uint8)[far:] = d["pool"].view(torch.uint8)
    x, q = d["qkv"], torch.empty_like(out, device="cuda")
    nb.nld_qk_norm_rope(x[:, :, :4], x[:, :, 4:12], x[:, :, 12:], d["gq"], d["gk"], write.EPS, d["rope"], d["lens"], q, big, d["table"] + far,
                        k_scale=d["ks"], v_scale=d["vs"])
    torch.cuda.synchronize()
    assert err == 0 and torch.equal(q.cpu(), out)
    assert torch.equal(big.view(torch.uint8)[far:].cpu(), pool.view(torch.uint8)) and not big.view(torch.uint8)[:far].any()
