"""The same odd lengths, masks and prefixes through every pair of kernels that nld_attention_q8 and nld_attention_shared are
made of: query rows of a kv head (positions x heads; for the prefix pass, of the whole batch) on either side of the small
tiles' 32, and of their 16 for a prefix over 2048 keys.  (Prefix passes in runs of pages: test_gpu_attention_wide.)"""
import pytest

import test_gpu_attention_q8 as q8
import test_gpu_attention_shared as shared

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
