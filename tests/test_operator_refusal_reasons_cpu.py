"""Each refusal of the operators around the paged cache is the one that the bad argument calls for: all other arguments
are good, the workspace's size too, and the message names the reason (no GPU: refused before any CUDA call)."""
import pytest

import self_speculation_b200 as nb
import test_operator_refusals_cpu as r

P = r.P
SIZE = nb.nld_attention_shared_workspace_size(1, 1, 32)
SHARED = {**r.SHARED, "ws_bytes": SIZE}


def refused(fn, defaults, bad, status, reason):
    assert r.status(fn, defaults, **bad) == status
    said = nb.load_library().nld_last_error(None).decode()
    assert reason in said, said


NULL, HEADS, MAX_LEN, ALIGNED = "NULL pointer argument", "bad batch/m/head counts", "max_len outside", "must be 16-byte aligned"
ATTN = [(dict([(name, None)]), 1, NULL) for name in ("q", "pool", "table", "lens", "out")] + [
    (dict(batch=0), 1, HEADS), (dict(m=0), 1, HEADS), (dict(hq=12), 1, HEADS), (dict(hkv=0), 1, HEADS), (dict(hq=0), 1, HEADS),
    (dict(hd=64), 8, "head_dim must be 128"), (dict(block=0), 1, "block_size must be >= 1"), (dict(max_len=65), 1, MAX_LEN),
    (dict(max_len=0), 1, MAX_LEN), (dict(m=2, max_len=1), 1, MAX_LEN), (dict(pps=0), 1, MAX_LEN), (dict(pps=1 << 26), 1, MAX_LEN),
    (dict(n_pages=0), 1, "bad pool size"), (dict(n_pages=1 << 28), 1, "bad pool size"),
    (dict(q=P + 8), 1, ALIGNED), (dict(out=P + 4), 1, ALIGNED), (dict(pool=P + 2), 1, ALIGNED),
    (dict(batch=1 << 20, m=64, hq=64), 1, "batch * m * heads too large")]


@pytest.mark.parametrize("bad,status,reason", ATTN + [(dict(ks=None), 1, "NULL scale pointer"), (dict(vs=None), 1, "NULL scale pointer"),
                                                      (dict(batch=65536), 1, "batch*query tiles too large")])
def test_attention_q8(bad, status, reason):
    refused("nld_attention_q8", r.Q8, bad, status, reason)


PREFIX, WORKSPACE = "shared_len outside", "workspace must be 16-byte aligned and at least"


@pytest.mark.parametrize("bad,status,reason", ATTN + [
    (dict(shared=None), 1, PREFIX), (dict(shared_len=-1), 1, PREFIX), (dict(shared_len=129), 1, PREFIX), (dict(n_shared=0), 1, PREFIX),
    (dict(n_shared=1, shared_len=65), 1, PREFIX), (dict(ws=None), 1, WORKSPACE), (dict(ws=P + 8), 1, WORKSPACE),
    (dict(ws_bytes=SIZE - 1), 1, WORKSPACE), (dict(ws_bytes=0), 1, WORKSPACE),
    (dict(batch=2), 1, WORKSPACE), (dict(m=33, max_len=33), 1, WORKSPACE),      # the size for one row
    (dict(batch=65536, ws_bytes=1 << 40), 1, "batch*query tiles too large")])
def test_attention_shared(bad, status, reason):
    refused("nld_attention_shared", SHARED, bad, status, reason)


def test_attention_shared_workspace_size_is_named():
    refused("nld_attention_shared", SHARED, dict(ws_bytes=SIZE - 1), 1, f"at least {SIZE} bytes")


COUNTS, ROWS16, ALIGNED_W, CACHE = "bad batch/m/head counts", "row distances must hold a row", "pointers must be 16-byte aligned", "bad page table or pool size"


@pytest.mark.parametrize("bad,status,reason", [(dict([(name, None)]), 1, NULL) for name in ("q", "k", "v", "rope", "lens", "out", "pool", "table")] + [
    (dict(dtype=2), 1, "dtype must be"), (dict(kv=3), 1, "kv_dtype must be"), (dict(gq=None), 1, "both or neither"), (dict(gk=None), 1, "both or neither"),
    (dict(ks=None), 1, "needs k and v scales"), (dict(vs=None), 1, "needs k and v scales"), (dict(hd=96), 8, "head_dim must be 64 or 128"),
    (dict(batch=0), 1, COUNTS), (dict(m=0), 1, COUNTS), (dict(hq=0), 1, COUNTS), (dict(hkv=-1), 1, COUNTS), (dict(hq=65537, q_ld=65537 * 128), 1, COUNTS),
    (dict(eps=float("nan")), 1, "rms_eps must be >= 0"), (dict(eps=-1.0), 1, "rms_eps must be >= 0"), (dict(rope_rows=0), 1, "bad rope_rows"),
    (dict(offset=-1), 1, "position_offset"), (dict(pps=0), 1, CACHE), (dict(pps=1 << 26), 1, CACHE), (dict(n_pages=0), 1, CACHE),
    (dict(q_ld=4088), 1, ROWS16), (dict(q_ld=4100), 1, ROWS16), (dict(k_ld=1016), 1, ROWS16), (dict(v_ld=1025), 1, ROWS16),
    (dict(q=P + 2), 1, ALIGNED_W), (dict(pool=P + 8), 1, ALIGNED_W), (dict(rope=P + 4), 1, ALIGNED_W), (dict(gk=P + 2), 1, ALIGNED_W),
    (dict(out=P + 8), 1, ALIGNED_W), (dict(batch=1 << 24, m=1 << 24), 1, "batch * m too large")])
def test_cache_write(bad, status, reason):
    refused("nld_qk_norm_rope", r.WRITE, bad, status, reason)


@pytest.mark.parametrize("bad,reason", [(dict([(name, None)]), NULL) for name in ("x", "u", "tokens")] + [
    (dict(dtype=2), "dtype must be"), (dict(rows=0), "vocab in 1..2^19"), (dict(vocab=0), "vocab in 1..2^19"),
    (dict(vocab=(1 << 19) + 1, ld=1 << 20), "vocab in 1..2^19"), (dict(rows=(1 << 28)), "too many rows"), (dict(ld=99), "ld must be"),
    (dict(x=P + 2), "aligned to their type"), (dict(x=P + 1, dtype=1), "aligned to their type")])
def test_sample(bad, reason):
    refused("nld_sample", r.SAMPLE, bad, 1, reason)
