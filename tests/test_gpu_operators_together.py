"""One decode step as a serving loop makes it: nld_qk_norm_rope writes the new rows, nld_attention_q8 or
nld_attention_shared reads the cache, nld_sample draws the tokens; eagerly and from a captured graph, several
steps in a row.  Each stage is compared with the float64 oracle on what the stage before left."""
import pytest
import torch

import test_gpu_attention_q8 as q8
import test_gpu_attention_shared as shared
import test_gpu_qk_norm_rope as write
import test_gpu_sample as sample

pytestmark = pytest.mark.gpu


class Step:
    """Two sequences of 8 / 2 heads; logits are a fixed projection of the attention's output."""

    def __init__(self, m, prefix, e4m3):
        self.m, self.prefix = m, prefix
        lens = [70, 3]
        self.s = shared.make(prefix, lens, m + 8, 8, 2, seed=m, fill=0.0)
        if e4m3:
            self.s["pool"] = self.s["pool"].to(torch.float8_e4m3fn)
        self.s.update(lens=torch.tensor(lens, dtype=torch.int32), m=m, prefix=prefix)
        g = torch.Generator().manual_seed(m + 1)
        self.qkv = torch.randn(2, m, 12, 128, generator=g).to(torch.bfloat16)
        self.gain = (1 + 0.2 * torch.randn(2, 128, generator=g)).to(torch.bfloat16)
        self.rope = write.rope_table(prefix + 100 + m, 128)
        self.ks, self.vs = 0.02 + torch.rand(2, generator=g) * 0.01, 0.02 + torch.rand(2, generator=g) * 0.01
        self.head = torch.randn(8 * 128, 3000, generator=g) * 0.3
        self.u = torch.rand(2 * m, generator=g)
        self.cuda = {k: v.cuda() for k, v in dict(qkv=self.qkv, gain=self.gain, rope=self.rope, ks=self.ks, vs=self.vs,
                                                  head=self.head, u=self.u, pool=self.s["pool"], sp=self.s["sp"],
                                                  table=self.s["table"], lens=self.s["lens"]).items()}
        import self_speculation_b200 as nb
        c = self.cuda
        c["q"] = torch.zeros(2, m, 8, 128, dtype=torch.bfloat16, device="cuda")
        c["out"] = torch.zeros_like(c["q"])
        c["tok"] = torch.zeros(2 * m, dtype=torch.int32, device="cuda")
        c["k"] = torch.full((2 * m,), 50, dtype=torch.int32, device="cuda")
        c["p"] = torch.full((2 * m,), 0.9, device="cuda")
        c["err"] = torch.zeros(1, dtype=torch.int32, device="cuda")
        c["ws"] = torch.empty(nb.nld_attention_shared_workspace_size(2, m, 8), dtype=torch.uint8, device="cuda")
        self.e4m3 = e4m3

    def run(self):
        import self_speculation_b200 as nb
        c, m = self.cuda, self.m
        x = c["qkv"]
        q8_scales = dict(k_scale=c["ks"], v_scale=c["vs"]) if self.e4m3 else {}
        nb.nld_qk_norm_rope(x[:, :, :8], x[:, :, 8:10], x[:, :, 10:], c["gain"][0], c["gain"][1], 1e-6, c["rope"], c["lens"],
                            c["q"], c["pool"], c["table"], position_offset=self.prefix, err=c["err"], **q8_scales)
        if self.e4m3:
            nb.nld_attention_q8(c["q"], c["pool"], c["ks"], c["vs"], c["table"], c["lens"], 1, 90 + m, c["out"], err=c["err"])
        else:
            nb.nld_attention_shared(c["q"], c["pool"], c["sp"], self.prefix, c["table"], c["lens"], 1, 90 + m, c["out"],
                                    c["ws"], err=c["err"])
        c["logits"] = c["out"].float().view(2 * m, -1) @ c["head"]
        nb.nld_sample(c["logits"], c["u"], c["tok"], top_k=c["k"], top_p=c["p"])

    def check(self):
        import oracle.operators as oop
        torch.cuda.synchronize()
        c, s, m = self.cuda, self.s, self.m
        assert int(c["err"]) == 0
        q, pool, out = c["q"].cpu(), c["pool"].cpu(), c["out"].cpu()
        for b in range(2):
            first = int(s["lens"][b])
            pos = torch.arange(first, first + m) + self.prefix
            want = oop.norm_rope(self.qkv[b, :, :8], self.gain[0], 1e-6, pos, write.THETA)
            # the tolerance of test_gpu_qk_norm_rope
            size = (want.square() + want.roll(64, -1).square()).sqrt() * 2 ** 0.5 * 32 * 2.0 ** -24
            assert ((q[b].double() - want).abs() <= size + 2.0 ** -8 * want.abs()).all()
        seen = {**s, "q": q, "pool": pool, "ks": self.ks, "vs": self.vs}
        (q8 if self.e4m3 else shared).check(seen, out, 1)
        logits = c["logits"].cpu()
        for i in range(2 * m):
            want, _ = oop.sample_token(logits[i], float(self.u[i]), 1.0, 50, float(torch.tensor(0.9)))
            assert int(c["tok"][i]) == want

    def advance(self):
        self.s["lens"] += self.m
        self.cuda["lens"] += self.m


@pytest.mark.parametrize("m,prefix,e4m3", [(1, 0, True), (1, 150, False), (4, 0, True), (4, 150, False)])
def test_steps(m, prefix, e4m3):
    step = Step(m, prefix, e4m3)
    step.run()
    step.check()
    step.advance()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step.run()
    for _ in range(2):
        graph.replay()
        step.check()
        step.advance()


@pytest.mark.parametrize("dtype,vocab", [("f32", 700), ("f32", 4001), ("bf16", 20001), ("bf16", 40007)])
def test_many_rows_by_temperature(dtype, vocab):
    """Batches that fill the machine, without filters: the token is the first whose cumulated weight exceeds u of
    the total, taken in 64 bits; a sum within 2^-36 of the border would be open (none of these is)."""
    import self_speculation_b200 as nb
    rows = 600
    x = sample.logits(rows, vocab, dtype, seed=vocab)
    g = torch.Generator().manual_seed(1)
    u, t = torch.rand(rows, generator=g), 0.5 + torch.rand(rows, generator=g)
    tok = torch.zeros(rows, dtype=torch.int32, device="cuda")
    nb.nld_sample(x.cuda(), u.cuda(), tok, temperature=t.cuda())
    v = x.double()
    c = torch.exp((v - v.amax(1, keepdim=True)) / t.double()[:, None]).cumsum(1)
    at = u.double() * c[:, -1]
    assert ((c - at[:, None]).abs().amin(1) > 2.0 ** -36 * c[:, -1]).all()
    assert torch.equal(tok.cpu().long(), (c <= at[:, None]).sum(1))
