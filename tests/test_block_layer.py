"""A transformer layer on block-scaled codes, as a server runs it: each call takes
what the one before wrote, among the library's own (QKV split, paged cache and
attention), and each is checked against the oracle on those inputs; then the whole
as one CUDA graph, replayed on other tokens."""
import numpy as np
import pytest
import torch

from oracle import block, ops
from oracle.formats import bf16_decode, bf16_encode
from parity import from_bits, to_bits
from test_parity_block_linear import check as check_linear
from test_parity_block_quant import check_codes, check_norm, gated_ref

pytestmark = pytest.mark.gpu

HQ, HKV, D, FFN, BLOCK = 6, 2, 64, 400, 16
H = HQ * D


class Layer:
    def __init__(self, gbf, tokens, seed):
        self.gbf, self.t = gbf, tokens
        rng = np.random.default_rng(seed)
        dev = lambda dtype, *s: torch.zeros(*s, dtype=dtype, device="cuda")                  # noqa: E731
        bf, u8, f32, i32 = torch.bfloat16, torch.uint8, torch.float32, torch.int32
        self.w = {}
        for name, (n, k) in dict(qkv=((HQ + 2 * HKV) * D, H), out=(H, H), up=(2 * FFN, H), down=(H, FFN)).items():
            w = from_bits(bf16_encode(rng.standard_normal((n, k)) * k ** -0.5))
            q, s = dev(u8, n, k), dev(f32, block.block_count(n), block.block_count(k))
            gbf.quantize_fp8_block(w, q, s, block_rows=128)
            self.w[name] = q, s
        vec = lambda *s: from_bits(bf16_encode(1 + 0.1 * rng.standard_normal(s)))            # noqa: E731
        self.norm1, self.norm2, self.qn, self.kn = vec(H), vec(H), vec(D), vec(D)
        t = tokens
        self.x, self.res = dev(bf, t, H), dev(bf, t, H)
        self.res1, self.res2 = dev(bf, t, H), dev(bf, t, H)
        codes = lambda k: (dev(u8, t, k), dev(f32, t, block.block_count(k)))                 # noqa: E731
        self.c1, self.c2, self.c3, self.c4 = codes(H), codes(H), codes(H), codes(FFN)
        self.qkv, self.o, self.up, self.y = dev(bf, t, (HQ + 2 * HKV) * D), dev(bf, t, H), dev(bf, t, 2 * FFN), dev(bf, t, H)
        self.q, self.attn = dev(bf, t, HQ, D), dev(bf, t, HQ, D)
        rows = 4 * t * BLOCK
        self.k, self.v = dev(bf, rows, HKV, D), dev(bf, rows, HKV, D)
        self.lens, self.new = dev(i32, t), torch.ones(t, dtype=i32, device="cuda")
        self.table, self.free = dev(i32, t, 4), torch.arange(4 * t, dtype=i32, device="cuda")
        self.ring = torch.tensor([0, 4 * t], dtype=i32, device="cuda")
        self.slots, self.pos = dev(i32, t), dev(i32, t)
        self.ws = dev(u8, gbf.paged_attention_workspace(HQ, HKV, D))

    def set(self, seed):
        rng = np.random.default_rng(seed)
        self.x.copy_(from_bits(bf16_encode(rng.standard_normal((self.t, H)))))
        self.res.copy_(from_bits(bf16_encode(rng.standard_normal((self.t, H)) * 2)))

    def step(self):
        g = self.gbf
        g.add_rmsnorm_fp8_block(self.x, self.res, self.res1, *self.c1, g.NORM_WEIGHT, weight=self.norm1)
        g.linear_fp8_block(*self.c1, *self.w["qkv"], None, self.qkv, act=g.ACT_NONE)
        g.paged_slots(self.lens, self.new, self.table, self.free, self.ring, BLOCK, self.lens, self.ring, self.slots, self.pos)
        g.qkv_split_norm_rope(self.qkv, HQ, HKV, D, g.QKNORM_PER_HEAD, self.qn, self.kn, 1e-6, g.ROPE_1D, self.pos, 1e4,
                              self.q, self.k, self.v, slots=self.slots)
        g.paged_attention(self.q, self.k, self.v, self.table, self.lens, BLOCK, self.attn, self.ws)
        g.quantize_fp8_block(self.attn.view(self.t, H), *self.c2)
        g.linear_fp8_block(*self.c2, *self.w["out"], None, self.o, act=g.ACT_NONE)
        g.add_rmsnorm_fp8_block(self.o, self.res1, self.res2, *self.c3, g.NORM_WEIGHT, weight=self.norm2)
        g.linear_fp8_block(*self.c3, *self.w["up"], None, self.up, act=g.ACT_NONE)
        g.gated_act_fp8_block(self.up, *self.c4, act=g.ACT_SILU)
        g.linear_fp8_block(*self.c4, *self.w["down"], None, self.y, act=g.ACT_NONE)

    def outputs(self):
        return [t.clone() for t in (self.res1, *self.c1, self.qkv, self.attn, *self.c2, self.o, self.res2, *self.c3, self.up,
                                    *self.c4, self.y)]

    def check(self):
        n = lambda t: t.cpu().numpy()                                                         # noqa: E731
        lin = lambda c, w, y: check_linear(bf16_decode(to_bits(y)), dict(                     # noqa: E731
            xq=n(c[0]), x_scales=n(c[1]), wq=n(self.w[w][0]), w_scales=n(self.w[w][1]), bias=None))
        norm = lambda x, r, o, c, w: check_norm((to_bits(o), n(c[0]), n(c[1])), dict(         # noqa: E731
            x=to_bits(x), res=to_bits(r), weight=to_bits(w)))
        norm(self.x, self.res, self.res1, self.c1, self.norm1)
        lin(self.c1, "qkv", self.qkv)
        attn = bf16_decode(to_bits(self.attn)).reshape(self.t, H)
        q, s = block.quantize(attn)
        assert np.array_equal(n(self.c2[0]), q) and np.array_equal(n(self.c2[1]), s)
        lin(self.c2, "out", self.o)
        norm(self.o, self.res1, self.res2, self.c3, self.norm2)
        lin(self.c3, "up", self.up)
        check_codes(n(self.c4[0]), n(self.c4[1]), *gated_ref(to_bits(self.up), FFN, "silu"))
        lin(self.c4, "down", self.y)
        assert self.gbf.device_status()[0] == 0


@pytest.mark.parametrize("tokens", [1, 5, 40, 150, 300])
def test_layer(tokens):
    import fusion_add_rmsnorm_gb300 as gbf
    layer = Layer(gbf, tokens, tokens)
    layer.set(1)
    layer.step()
    torch.cuda.synchronize()
    layer.check()


@pytest.mark.parametrize("tokens", [3, 200])
def test_layer_in_a_graph(tokens):
    """Captured once; replayed on other tokens it gives what eager calls give, on a cache that grows the same way."""
    import fusion_add_rmsnorm_gb300 as gbf
    eager, graph = Layer(gbf, tokens, 7), Layer(gbf, tokens, 7)
    for l in (eager, graph):
        l.set(0)
        l.step()                                     # the first token
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        graph.step()
    for seed in (1, 2, 3):
        for l in (eager, graph):
            l.set(seed)
        eager.step()
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(eager.outputs(), graph.outputs()):
            assert torch.equal(a, b)
    graph.check()


def test_the_layer_is_close_to_one_without_codes():
    """What the codes cost: the down projection's output against float64 on the same bf16 weights.  Each E4M3
    rounding is off by at most 2^-4 of its value, about 0.026 in the mean square; a product of two such
    operands by sqrt(2) times that, independent from term to term, so the output's relative error is about 0.04."""
    import fusion_add_rmsnorm_gb300 as gbf
    rng = np.random.default_rng(3)
    t, k, n = 64, 512, 256
    x, w = bf16_encode(rng.standard_normal((t, 2 * k))), bf16_encode(rng.standard_normal((n, k)) * k ** -0.5)
    q, s = torch.empty(t, k, dtype=torch.uint8, device="cuda"), torch.empty(t, k // 128, device="cuda")
    wq, ws = torch.empty(n, k, dtype=torch.uint8, device="cuda"), torch.empty(n // 128, k // 128, device="cuda")
    y = torch.empty(t, n, dtype=torch.bfloat16, device="cuda")
    gbf.gated_act_fp8_block(from_bits(x), q, s, act=gbf.ACT_SILU)
    gbf.quantize_fp8_block(from_bits(w), wq, ws, block_rows=128)
    gbf.linear_fp8_block(q, s, wq, ws, None, y, act=gbf.ACT_NONE)
    torch.cuda.synchronize()
    v = bf16_decode(x)
    ref = ops.gated_activation(v[:, :k], v[:, k:], 3) @ bf16_decode(w).T
    err = np.linalg.norm(bf16_decode(to_bits(y)) - ref) / np.linalg.norm(ref)
    assert err < 0.06, err
