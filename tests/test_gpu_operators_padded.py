"""A padded prefill as a serving program makes it: nld_qk_norm_rope writes the live rows of every sequence, and
nld_attention_q8 or nld_attention_shared reads the cache with m rows a sequence; the live rows have to be right, whatever
the padding queries hold, with one page of zeros behind every padding slot that has no page of its own."""
import pytest
import torch

import test_gpu_attention_q8 as q8
import test_gpu_attention_shared as shared
import test_gpu_qk_norm_rope as write
from oracle import operators as oop

pytestmark = pytest.mark.gpu

HQ, HKV = 8, 2


def make(lens, rows, m, prefix, e4m3, seed):
    """Own pages for the live keys alone; the others of a table row are the zero page."""
    g = torch.Generator().manual_seed(seed)
    B, pps = len(lens), (max(lens) + m + 63) // 64
    n_shared = (prefix + 63) // 64
    pool = torch.zeros(B * pps + n_shared + 1, 2, HKV, 64, 128, dtype=torch.bfloat16)
    ids = torch.randperm(pool.shape[0], generator=g).to(torch.int32)
    zero, sp, own = ids[0], ids[1:1 + n_shared].contiguous(), ids[1 + n_shared:].view(B, pps)
    table = torch.full((B, pps), int(zero), dtype=torch.int32)
    fill = lambda pages, n: pool.__setitem__(  # noqa: E731
        (pages[torch.arange(n) // 64].long(), slice(None), slice(None), torch.arange(n) % 64), torch.randn(n, 2, HKV, 128, generator=g).to(pool.dtype))
    fill(sp, prefix)
    for b in range(B):
        n = (lens[b] + rows[b] + 63) // 64
        table[b, :n] = own[b, :n]
        fill(table[b], lens[b])
    qkv = torch.randn(B, m, HQ + 2 * HKV, 128, generator=g).to(torch.bfloat16)
    for b in range(B):
        qkv[b, rows[b]:] = float("nan")      # not read
    return dict(pool=pool.to(torch.float8_e4m3fn) if e4m3 else pool, sp=sp, table=table, qkv=qkv, lens=torch.tensor(lens, dtype=torch.int32),
                rows=torch.tensor(rows, dtype=torch.int32), ks=0.01 + 0.01 * torch.rand(HKV, generator=g), vs=0.01 + 0.01 * torch.rand(HKV, generator=g),
                rope=write.rope_table(prefix + max(lens) + m, 128), prefix=prefix, zero=int(zero))


@pytest.mark.parametrize("lens,rows,m,bs", [
    ([0, 0, 0], [40, 1, 17], 40, 1), ([3, 130, 64], [8, 0, 5], 8, 1), ([0, 70], [16, 32], 48, 16), ([10, 0, 100, 64], [200, 64, 65, 1], 200, 1),
    ([63, 0], [1, 4], 4, 1)])
@pytest.mark.parametrize("prefix,e4m3", [(0, True), (0, False), (150, False)])
def test_live_rows(lens, rows, m, bs, prefix, e4m3):
    import self_speculation_b200 as nb
    s = make(lens, rows, m, prefix, e4m3, seed=m + len(lens))
    d = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in s.items()}
    x, B = d["qkv"], len(lens)
    q = torch.zeros(B, m, HQ, 128, dtype=torch.bfloat16, device="cuda")
    out, err = torch.zeros_like(q), torch.zeros(1, dtype=torch.int32, device="cuda")
    scales = dict(k_scale=d["ks"], v_scale=d["vs"]) if e4m3 else {}
    nb.nld_qk_norm_rope(x[:, :, :HQ], x[:, :, HQ:HQ + HKV], x[:, :, HQ + HKV:], None, None, 1e-6, d["rope"], d["lens"], q, d["pool"],
                        d["table"], position_offset=prefix, rows=d["rows"], err=err, **scales)
    for b in range(B):
        q[b, rows[b]:] = float("nan") if b % 2 else 1e30
    if e4m3:
        nb.nld_attention_q8(q, d["pool"], d["ks"], d["vs"], d["table"], d["lens"], bs, max(lens) + m, out, err=err)
    else:
        ws = torch.empty(nb.nld_attention_shared_workspace_size(B, m, HQ), dtype=torch.uint8, device="cuda")
        nb.nld_attention_shared(q, d["pool"], d["sp"], prefix, d["table"], d["lens"], bs, max(lens) + m, out, ws, err=err)
    torch.cuda.synchronize()
    assert int(err) == 0
    pool, q, out = d["pool"].cpu(), q.cpu(), out.cpu()
    assert (pool[s["zero"]].float() == 0).all()
    seen = {**s, "pool": pool}
    for b in range(B):
        if rows[b]:      # sequence b's live rows alone, as a batch of their own
            one = {**seen, "q": q[b:b + 1, :rows[b]], "table": s["table"][b:b + 1], "lens": s["lens"][b:b + 1], "m": rows[b]}
            (q8 if e4m3 else shared).check(one, out[b:b + 1, :rows[b]], bs)
