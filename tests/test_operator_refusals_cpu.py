"""The operators around the paged cache refuse bad arguments on the host, before any CUDA call (no
GPU: the pointers here are never read)."""
import pytest

import self_speculation_b200 as nb

P = 0x1000     # a 16-byte aligned address that nothing reads


def status(fn, defaults, **kw):
    lib = nb.load_library()
    args = dict(defaults)
    assert set(kw) <= set(args), kw
    args.update(kw)
    return getattr(lib, fn)(*args.values())


WRITE = dict(q=P, q_ld=4096, k=P, k_ld=1024, v=P, v_ld=1024, dtype=1, gq=P, gk=P, eps=1e-6, rope=P, rope_rows=64,
             offset=0, lens=P, rows=None, batch=1, m=1, hq=32, hkv=8, hd=128, out=P, pool=P, kv=2, ks=P, vs=P,
             table=P, pps=1, n_pages=1, err=None, stream=None)
Q8 = dict(q=P, pool=P, ks=P, vs=P, table=P, pps=1, n_pages=1, lens=P, batch=1, m=1, hq=32, hkv=8, hd=128, block=1,
          max_len=64, out=P, err=None, stream=None)
SHARED = dict(q=P, pool=P, shared=P, n_shared=2, shared_len=100, table=P, pps=1, n_pages=1, lens=P, batch=1, m=1, hq=32,
              hkv=8, hd=128, block=1, max_len=64, out=P, ws=P, ws_bytes=1 << 20, err=None, stream=None)
SAMPLE = dict(x=P, dtype=0, ld=100, rows=1, vocab=100, u=P, t=None, k=None, p=None, min_p=None, tokens=P, prob=None,
              stream=None)


@pytest.mark.parametrize("bad,want", [
    (dict(q=None), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(rope=None), 1), (dict(lens=None), 1),
    (dict(out=None), 1), (dict(pool=None), 1), (dict(table=None), 1), (dict(dtype=2), 1), (dict(kv=3), 1),
    (dict(gq=None), 1), (dict(ks=None), 1), (dict(vs=None), 1), (dict(hd=96), 8), (dict(batch=0), 1), (dict(m=0), 1),
    (dict(hq=0), 1), (dict(hkv=-1), 1), (dict(eps=float("nan")), 1), (dict(eps=-1.0), 1), (dict(rope_rows=0), 1),
    (dict(offset=-1), 1), (dict(pps=0), 1), (dict(n_pages=0), 1), (dict(q_ld=4095), 1), (dict(q_ld=4100), 1),
    (dict(k_ld=1000), 1), (dict(v_ld=1001), 1), (dict(q=P + 2), 1), (dict(pool=P + 8), 1), (dict(rope=P + 4), 1),
    (dict(gk=P + 2), 1), (dict(batch=1 << 24, m=1 << 24), 1)])
def test_cache_write(bad, want):
    assert status("nld_qk_norm_rope", WRITE, **bad) == want


ATTN = [(dict(q=None), 1), (dict(pool=None), 1), (dict(table=None), 1), (dict(lens=None), 1), (dict(out=None), 1),
        (dict(batch=0), 1), (dict(m=0), 1), (dict(hq=12), 1), (dict(hkv=0), 1), (dict(hd=64), 8), (dict(block=0), 1),
        (dict(max_len=65), 1), (dict(max_len=0), 1), (dict(m=2, max_len=1), 1), (dict(pps=0), 1), (dict(n_pages=0), 1),
        (dict(n_pages=1 << 28), 1), (dict(q=P + 8), 1), (dict(out=P + 4), 1), (dict(pool=P + 2), 1),
        (dict(batch=70000, hkv=32), 1), (dict(batch=1 << 20, m=64, max_len=64, hq=64), 1)]


@pytest.mark.parametrize("bad,want", ATTN + [(dict(ks=None), 1), (dict(vs=None), 1)])
def test_attention_q8(bad, want):
    assert status("nld_attention_q8", Q8, **bad) == want


@pytest.mark.parametrize("bad,want", ATTN[:-2] + [
    (dict(shared=None), 1), (dict(shared_len=-1), 1), (dict(shared_len=129), 1), (dict(n_shared=0), 1), (dict(ws=None), 1),
    (dict(ws=P + 8), 1), (dict(ws_bytes=32 * 130 * 4 - 1), 1)])
def test_attention_shared(bad, want):
    assert status("nld_attention_shared", SHARED, **bad) == want


def test_attention_shared_workspace_size():
    assert nb.nld_attention_shared_workspace_size(4, 33, 32) == (4 * 33 * 32 + 128 * (32 + 160)) * 130 * 4
    assert nb.nld_attention_shared_workspace_size(0, 1, 32) == 0
    assert nb.nld_attention_shared_workspace_size(1, -1, 32) == 0


@pytest.mark.parametrize("bad,want", [
    (dict(x=None), 1), (dict(u=None), 1), (dict(tokens=None), 1), (dict(dtype=2), 1), (dict(rows=0), 1),
    (dict(vocab=0), 1), (dict(vocab=(1 << 19) + 1, ld=1 << 20), 1), (dict(ld=99), 1), (dict(x=P + 2), 1),
    (dict(x=P + 1, dtype=1), 1)])
def test_sample(bad, want):
    assert status("nld_sample", SAMPLE, **bad) == want
    assert nb.load_library().nld_last_error(None)
