"""The decode-step operators together with the library's own, as a server runs
them: prompts enter the paged cache, a captured step then decodes token after
token for the whole batch (block tables and slots from the lengths, packed QKV
into the cache, attention over it with E4M3 codes out, the E4M3 Linear, logits,
the next token, which feeds the next step), a request ends and another takes its
place and its blocks.  Every operator is compared with the oracle on the inputs
it was given, so that one operator's rounding is not another's error."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from oracle import chains, decode, formats
from parity import assert_bf16_close, from_bits, to_bits

pytestmark = pytest.mark.gpu

HQ, HKV, D, HIDDEN, VOCAB, BLOCK, BLOCKS, WIDTH = 8, 2, 64, 256, 1008, 16, 40, 6
PACK, SCALE, CODES = (HQ + 2 * HKV) * D, D ** -0.5, 0.02


@pytest.fixture(scope="module")
def gbf():
    import fusion_add_rmsnorm_gb300 as g
    assert g.device_status()[0] == g.OK
    return g


def bf(rng, *shape, std=1.0):
    return torch.from_numpy((rng.standard_normal(shape) * std).astype(np.float32)).to(torch.bfloat16).cuda()


def i32(*a):
    return torch.tensor(a, dtype=torch.int32, device="cuda")


class Server:
    def __init__(self, gbf, batch, seed):
        rng = np.random.default_rng(seed)
        self.gbf, self.batch = gbf, batch
        self.embed = bf(rng, VOCAB, HIDDEN)
        self.w_qkv, self.w_logits = bf(rng, PACK, HIDDEN, std=0.06), bf(rng, VOCAB, HIDDEN, std=0.15)
        self.q_w, self.k_w = bf(rng, D, std=0.1) + 1, bf(rng, D, std=0.1) + 1
        w = rng.standard_normal((HIDDEN, HQ * D)).astype(np.float32) * 0.05
        self.w_scale = torch.full((HIDDEN,), 0.001, device="cuda")
        self.w_out = torch.from_numpy((w / 0.001).clip(-448, 448)).to(torch.float8_e4m3fn).view(torch.uint8).cuda()
        # the cache starts as NaN: nothing that was never written may be read
        self.k = torch.full((BLOCKS * BLOCK, HKV, D), float("nan"), dtype=torch.bfloat16, device="cuda")
        self.v = self.k.clone()
        self.table = torch.full((batch, WIDTH), -1, dtype=torch.int32, device="cuda")
        self.free = torch.from_numpy(rng.permutation(BLOCKS).astype(np.int32)).cuda()
        self.ring, self.lens = i32(0, BLOCKS), torch.zeros(batch, dtype=torch.int32, device="cuda")
        self.ws = torch.empty(gbf.paged_attention_workspace(HQ, HKV, D), dtype=torch.uint8, device="cuda")
        self.tokens = torch.zeros(batch, dtype=torch.int32, device="cuda")
        e = lambda *s, t=torch.bfloat16: torch.empty(*s, dtype=t, device="cuda")        # noqa: E731
        self.x, self.qkv, self.q = e(batch, HIDDEN), e(batch, PACK), e(batch, HQ, D)
        self.codes, self.y, self.logits = e(batch, HQ * D, t=torch.uint8), e(batch, HIDDEN), e(batch, VOCAB)
        self.slots, self.pos = e(batch, t=torch.int32), e(batch, t=torch.int32)
        self.one = torch.ones(batch, dtype=torch.int32, device="cuda")
        self.u = e(batch, t=torch.float32)
        self.temperature = torch.full((batch,), 0.8, device="cuda")
        self.top_p = torch.full((batch,), 0.9, device="cuda")
        self.top_k = torch.full((batch,), 50, dtype=torch.int32, device="cuda")

    def enter(self, new, prompts):
        """Prompts (or ended requests) through the block tables and into the cache."""
        n = sum(max(x, 0) for x in new)
        slots, pos = (torch.full((n,), -1, dtype=torch.int32, device="cuda") for _ in range(2))
        self.gbf.paged_slots(self.lens, i32(*new), self.table, self.free, self.ring, BLOCK, self.lens, self.ring, slots, pos)
        if n:
            qkv, q = torch.empty(n, PACK, dtype=torch.bfloat16, device="cuda"), torch.empty(n, HQ, D, dtype=torch.bfloat16,
                                                                                         device="cuda")
            self.gbf.linear_bias_gelu(self.embed[prompts], self.w_qkv, None, qkv, act=self.gbf.ACT_NONE)
            self.gbf.qkv_split_norm_rope(qkv, HQ, HKV, D, 0, self.q_w, self.k_w, 1e-6, 0, pos, 1e4, q, self.k, self.v,
                                         slots=slots)

    def step(self):
        g = self.gbf
        self.x.copy_(self.embed[self.tokens.long()])
        g.paged_slots(self.lens, self.one, self.table, self.free, self.ring, BLOCK, self.lens, self.ring, self.slots,
                      self.pos)
        g.linear_bias_gelu(self.x, self.w_qkv, None, self.qkv, act=g.ACT_NONE)
        g.qkv_split_norm_rope(self.qkv, HQ, HKV, D, 0, self.q_w, self.k_w, 1e-6, 0, self.pos, 1e4, self.q, self.k,
                              self.v, slots=self.slots)
        g.paged_attention(self.q, self.k, self.v, self.table, self.lens, BLOCK, self.codes, self.ws, out_scale=CODES)
        g.linear_fp8_act(self.codes, CODES, self.w_out, self.w_scale, None, self.y, act=g.ACT_NONE)
        g.linear_bias_gelu(self.y, self.w_logits, None, self.logits, act=g.ACT_NONE)
        g.sample_tokens(self.logits, self.u, self.tokens, temperature=self.temperature, top_k=self.top_k,
                        top_p=self.top_p)


def np_(t):
    return t.cpu().numpy()


def check_slots(s, before, new):
    p, seq, slots, pos, _, refused = decode.paged_slots(before["lens"], new, before["table"], before["free"],
                                                        before["ring"], BLOCK)
    assert not refused.any()
    assert np.array_equal(np_(s.table), p.table) and np.array_equal(np_(s.free), p.free_ring)
    assert np.array_equal(np_(s.lens), seq) and np_(s.ring).tolist() == [p.head, p.count]
    return slots, pos


def state(s):
    return {k: np_(getattr(s, k)).copy() for k in ("lens", "table", "free", "ring", "tokens")}


def check_step(s, before):
    """The step that led from `before` to the server's state, operator by operator."""
    slots, pos = check_slots(s, before, np.ones(s.batch, int))
    assert np.array_equal(np_(s.slots), slots) and np.array_equal(np_(s.pos), pos)
    assert np.array_equal(to_bits(s.x), to_bits(s.embed)[before["tokens"]])
    rq, rk, rv = chains.qkv_split_norm_rope(to_bits(s.qkv), HQ, HKV, D, 0, to_bits(s.q_w), to_bits(s.k_w), 1e-6, 0, pos,
                                            1e4, slots=slots, cache_rows=BLOCKS * BLOCK)
    assert_bf16_close(to_bits(s.q), rq, "q")
    assert_bf16_close(to_bits(s.k)[slots], rk[slots], "k")
    assert np.array_equal(to_bits(s.v)[slots], rv[slots])
    k, v = (np.nan_to_num(formats.bf16_decode(to_bits(t))) for t in (s.k, s.v))
    out, _, size, _ = decode.paged_attention(formats.bf16_decode(to_bits(s.q)), k, v, np_(s.table), np_(s.lens), BLOCK,
                                             SCALE)
    want, got = np.clip(out / np.float32(CODES), -448, 448), formats.e4m3_decode(np_(s.codes)).reshape(out.shape)
    # half a step of E4M3, or of its smallest subnormal, and 2^-12 of what the weighted sum is made of
    assert (np.abs(got - want) <= 2.0 ** -4 * np.abs(want) + 2.0 ** -10 + 2.0 ** -12 * size / CODES).all()
    y = chains.linear_fp8_act(np_(s.codes), np.float32(CODES), np_(s.w_out), np_(s.w_scale))
    assert_bf16_close(to_bits(s.y), y, "output projection")
    assert_bf16_close(to_bits(s.logits), chains.linear_bias_gelu(to_bits(s.y), to_bits(s.w_logits), act_gelu=False),
                      "logits")
    l, u, sampled = s.logits.float().cpu().numpy(), np_(s.u), np_(s.tokens)
    for b in range(s.batch):
        token, _, margin, total = decode.sample_row(l[b], u[b], float(np.float32(0.8)), 50, float(np.float32(0.9)))
        assert sampled[b] == token or margin < 4 * (2.0 ** -37 + VOCAB * 2.0 ** -44 / total)


def test_a_server_decodes(gbf):
    s = Server(gbf, 5, seed=3)
    rng = np.random.default_rng(4)
    before = state(s)
    new = [17, 1, 40, 16, 5]
    s.enter(new, torch.from_numpy(rng.integers(0, VOCAB, sum(new))).cuda())
    torch.cuda.synchronize()
    check_slots(s, before, new)
    s.tokens.copy_(i32(*rng.integers(0, VOCAB, 5)))
    # one step by itself (also the warm-up that a capture needs), then the captured one over and over
    before = state(s)
    s.u.copy_(torch.rand(5))
    s.step()
    torch.cuda.synchronize()
    check_step(s, before)
    graph = torch.cuda.CUDAGraph()
    before = state(s)
    with torch.cuda.graph(graph):
        s.step()
    for t in range(20):                                     # every request crosses a block border
        s.u.copy_(torch.from_numpy(rng.random(5).astype(np.float32)))
        graph.replay()
        torch.cuda.synchronize()
        check_step(s, before)
        before = state(s)
    # request 2 ends: its blocks go to the ring's end, and a new prompt takes its place
    s.enter([0, 0, -1, 0, 0], None)
    torch.cuda.synchronize()
    check_slots(s, before, [0, 0, -1, 0, 0])
    assert int(s.lens[2]) == 0 and int(s.ring[1]) == int(before["ring"][1]) + 4
    before = state(s)
    s.enter([0, 0, 33, 0, 0], torch.from_numpy(rng.integers(0, VOCAB, 33)).cuda())
    torch.cuda.synchronize()
    check_slots(s, before, [0, 0, 33, 0, 0])
    before = state(s)
    graph.replay()
    torch.cuda.synchronize()
    check_step(s, before)
    assert gbf.device_status()[0] == gbf.OK


FIRST = """
import torch, fusion_add_rmsnorm_gb300 as gbf
z = lambda *s, t=torch.int32: torch.zeros(*s, dtype=t, device="cuda")
bf = torch.bfloat16
lens, new, table, free = z(2), torch.ones(2, dtype=torch.int32, device="cuda"), z(2, 4), torch.arange(8, device="cuda").int()
ring, seq, ring_out, slots, pos = torch.tensor([0, 8], device="cuda").int(), z(2), z(2), z(2), z(2)
q, k, out, ws = z(2, 4, 64, t=bf) + 1, z(128, 2, 64, t=bf) + 1, z(2, 4, 64, t=bf), z(1 << 22, t=torch.uint8)
logits, u, tokens = z(2, 1000, t=bf), z(2, t=torch.float32) + 0.5, z(2)
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    gbf.paged_slots(lens, new, table, free, ring, 16, seq, ring_out, slots, pos)
    gbf.paged_attention(q, k, k, table, seq, 16, out, ws)
    gbf.sample_tokens(logits, u, tokens)
g.replay()
torch.cuda.synchronize()
assert slots.tolist() == [0, 16] and tokens.tolist() == [500, 500] and (out == 1).all() and gbf.device_status()[0] == gbf.OK
"""


def test_first_calls_of_a_process_in_a_capture():
    """What a call sets up once per device is set up while a stream is being captured too."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
