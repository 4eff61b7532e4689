"""The block around the layer in one call: against the chain of its steps, against a plain form, in a captured graph,
on other streams, in place."""

import numpy as np
import pytest
import torch

import workloads as W
from expert_serving_amd import abi

import plain_block as P
from gpu_util import dev, f32, i32, rms, say

pytestmark = pytest.mark.gpu

EPS = 1e-5


def np64(t):
    return t.detach().cpu().double().numpy()


class Block:
    """Inputs of one block of a workload's shape, its int8 weights beside the bf16 ones."""

    def __init__(self, cfg, stream="bf16", seed=0, offline=(), norms=True, gate="channel", scale=1.0):
        self.cfg, self.T, self.H = cfg, cfg.tokens, cfg.hidden
        self.inp = W.make_layer_inputs(cfg, dev(), salt=seed)
        self.shape = abi.make_shape(cfg)
        T, H = self.T, self.H
        st = torch.bfloat16 if stream == "bf16" else torch.float32
        self.x = W.normal((T, H), 2.0, W.DT_F32, dev(), 11 + seed).to(st)
        bias = W.normal((cfg.experts,), 0.05, W.DT_F32, dev(), 12 + seed)
        for e in offline:
            bias[e] = float("-inf")
        self.pre = 1 + W.normal((H,), 0.1, W.DT_F32, dev(), 13 + seed) if norms else None
        self.post = 1 + W.normal((H,), 0.1, W.DT_F32, dev(), 14 + seed) if norms else None
        g = {"channel": (1, H), "token": (T, 1), None: None}[gate]
        self.gate = None if g is None else W.normal(g, 1.0, W.DT_F32, dev(), 15 + seed).to(torch.bfloat16)
        self.bias = bias
        self.scale = scale
        self.block = abi.make_block(bias, self.pre, self.post, EPS, self.gate, scale,
                                    abi.MOE_BF16 if stream == "bf16" else abi.MOE_F32)
        if cfg.dtype == W.DT_BF16 and cfg.hidden % 128 == 0 and cfg.inter % 128 == 0:
            q = {k: abi.quantize_int8(self.inp[k]) for k in ("w_gate", "w_up", "w_down")}
            self.experts = abi.int8_ffn(q["w_gate"], q["w_up"], q["w_down"])
            self.shared = None
            if cfg.shared_inter:
                q = {k: abi.quantize_int8(self.inp[k]) for k in ("ws_gate", "ws_up", "ws_down")}
                self.shared = abi.int8_ffn(q["ws_gate"], q["ws_up"], q["ws_down"])

    def debug(self):
        T, k, E = self.T, self.cfg.top_k, self.cfg.experts
        return dict(logits=f32((T, E)), topk_ids=i32((T, k)), topk_gates=f32((T, k)), expert_counts=i32(E),
                    expert_offsets=i32(E + 1), row_of_slot=i32((T, k)), num_dropped=i32(1), row_token=i32(T * k, 0))

    def workspace(self, int8):
        n = abi.moe_workspace_size_int8(self.shape) if int8 else abi.moe_workspace_size_block(self.shape)
        return torch.empty(n, dtype=torch.uint8, device=dev())

    def run(self, int8, out, ws, dbg=None, x=None, stream=None):
        x = self.x if x is None else x
        i = self.inp
        if int8:
            abi.moe_block_forward_int8(self.shape, self.block, x, i["w_router"], i["bias"], i["k_per_token"],
                                       self.experts, self.shared, out, dbg, ws, stream=stream)
        else:
            abi.moe_block_forward(self.shape, self.block, x, i["w_router"], i["bias"], i["k_per_token"], i["w_gate"],
                                  i["w_up"], i["w_down"], i["ws_gate"], i["ws_up"], i["ws_down"], out, dbg, ws,
                                  stream=stream)

    def plain(self, int8, d, tokens):
        """The block of some tokens in fp64, on the GPU's own logits (h through int8 codes where int8)."""
        c, i = self.cfg, self.inp
        lg = np64(d["logits"])[tokens].astype(np.float32)
        kpt = None if i["k_per_token"] is None else i["k_per_token"].cpu().numpy()[tokens]
        ids, gates = P.route_biased(lg, self.bias.cpu().numpy(), c.top_k, kpt,
                                    "sigmoid" if c.score else "softmax", bool(c.renormalize), c.routed_scale,
                                    c.num_groups, c.topk_groups, c.group_topn)
        assert np.array_equal(d["topk_ids"].cpu().numpy()[tokens], ids)
        ros = d["row_of_slot"].cpu().numpy()[tokens]
        x = np64(self.x)[tokens]
        n = x if self.pre is None else P.rms_norm(x, np64(self.pre), EPS)
        if not int8:
            n = np64(torch.from_numpy(n).to(torch.bfloat16)) if c.dtype == W.DT_BF16 else n
        else:
            n = P.codes(n)[0] * P.codes(n)[1][:, None]

        def ffn(v, g, u, dn):
            a, b = v @ np64(g).T, v @ np64(u).T
            h = a / (1 + np.exp(-a)) * b
            if int8:
                h = h.astype(np.float16).astype(np.float64)
                q, s = P.codes(h)
                h = q * s[:, None]
            return h @ np64(dn).T

        if int8:
            def deq(p, e=None):
                co, s = (p[0], p[1]) if e is None else (p[0][e], p[1][e])
                return co.double() * s.double().unsqueeze(-1)
            w = lambda e: (deq(self.experts["gate"], e), deq(self.experts["up"], e), deq(self.experts["down"], e))
        else:
            w = lambda e: (i["w_gate"][e], i["w_up"][e], i["w_down"][e])
        y = np.zeros((len(tokens), self.H))
        for e in np.unique(ids[ids >= 0]):
            m = (ids == e) & (ros >= 0)
            at = np.nonzero(m.any(1))[0]
            if len(at):
                y[at] += (gates * m).sum(1)[at, None] * ffn(n[at], *w(e))
        if c.shared_inter:
            sw = [deq(self.shared[k]) for k in ("gate", "up", "down")] if int8 else \
                [i["ws_gate"], i["ws_up"], i["ws_down"]]
            y += ffn(n, *sw)
        if self.post is not None:
            y = P.rms_norm(y, np64(self.post), EPS)
        if self.gate is not None:
            g = np64(self.gate)
            y = y * (g if g.shape[0] == 1 else g[tokens])
        return self.scale * x + y


def tiny(**kw):
    return W.CONFIGS["qwen3_skewed"].replace(name="block_small", hidden=512, inter=256, experts=16, zipf_s=0.3, **kw)


CONFIGS = {
    "small": tiny(tokens=77, top_k=4, k_choices=None, capacity_factor=0.0),
    "small_dropping": tiny(tokens=300, top_k=4, k_choices=(1, 3, 4), capacity_factor=1.0),
    "groups_shared": tiny(tokens=150, top_k=4, score=W.SCORE_SIGMOID, num_groups=4, topk_groups=2, group_topn=2,
                          shared_inter=384, routed_scale=2.5, k_choices=None, capacity_factor=0.0),
    "one_token": tiny(tokens=1, top_k=2, k_choices=None, capacity_factor=0.0, shared_inter=256),
    "big_tiles": tiny(tokens=2100, top_k=3, k_choices=None, capacity_factor=0.0, shared_inter=256),
    "decode": W.CONFIGS["mixtral_decode"].replace(name="block_decode", inter=4096, tokens=9),
}


@pytest.mark.parametrize("int8", [False, True], ids=["bf16", "int8"])
@pytest.mark.parametrize("name", CONFIGS)
def test_block_against_the_plain_form(name, int8):
    """Largest error within 2e-2 of the rms, the layer's own tolerance: its h is rounded to 11 bits (or to codes,
    whose flips move an output by one part in some hundred of its rms at most), its outputs to bf16 here."""
    cfg = CONFIGS[name]
    say(f"block {name} int8={int8}")
    b = Block(cfg, stream="f32", seed=1, offline=(3,))
    out, d, ws = f32((b.T, b.H)), b.debug(), b.workspace(int8)
    b.run(int8, out, ws, d)
    torch.cuda.synchronize()
    tokens = np.arange(b.T) if b.T <= 300 else np.random.default_rng(1).choice(b.T, 200, replace=False)
    want = b.plain(int8, d, tokens)
    err = np.abs(np64(out)[tokens] - want)
    say(f"  max err / rms {err.max() / rms(want):.2e}")
    assert err.max() <= 2e-2 * rms(want)
    assert abi.moe_read_device_flags(ws) == 0
    assert int(d["expert_counts"][3]) == 0             # out of service


@pytest.mark.parametrize("name", ["small", "small_dropping", "big_tiles"])
def test_int8_block_is_the_chain_of_its_steps(name):
    """Where the down projection is not split, the block's bits are those of its steps called one by one."""
    cfg = CONFIGS[name].replace(shared_inter=0)
    b = Block(cfg, seed=2)
    T, H, k, E = b.T, b.H, cfg.top_k, cfg.experts
    s = b.shape
    out, ws = torch.empty(T, H, dtype=torch.bfloat16, device=dev()), b.workspace(True)
    b.run(True, out, ws)
    xn, xq, xs = torch.empty(T, H, dtype=torch.bfloat16, device=dev()), \
        torch.empty(T, H, dtype=torch.int8, device=dev()), f32(T)
    abi.moe_norm(T, H, abi.MOE_BF16, b.x, b.pre, EPS, abi.MOE_BF16, xn, xq, xs)
    ids, gates, cnt, off, ros, rt, nd = i32((T, k)), f32((T, k)), i32(E), i32(E + 1), i32((T, k)), i32(T * k, 0), i32(1)
    ws0 = torch.empty(abi.moe_workspace_size(s), dtype=torch.uint8, device=dev())
    abi.moe_route_biased(s, xn, b.inp["w_router"], b.inp["bias"], b.bias, None, None, b.inp["k_per_token"], ids, gates,
                         ws0)
    abi.moe_dispatch(s, None, ids, cnt, off, ros, rt, nd, None, ws0)
    y = torch.empty(T * k, H, dtype=torch.float16, device=dev())
    abi.moe_grouped_ffn_int8(s, xq[rt.long()], xs[rt.long()], off, b.experts, abi.MOE_F16, y, ws)
    chain = torch.empty_like(out)
    abi.moe_combine_norm(s, b.block, abi.MOE_F16, y, ros, gates, None, b.x, chain)
    assert torch.equal(out, chain)


def test_block_without_anything_is_the_layer():
    """No norm, gate, residual or balance bias: the layer call's own result."""
    for name in ("small", "groups_shared", "one_token"):
        cfg = CONFIGS[name].replace(k_choices=None)
        b = Block(cfg, seed=3, norms=False, gate=None, scale=0.0)
        b.block.select_bias = None
        out = torch.empty(b.T, b.H, dtype=torch.bfloat16, device=dev())
        b.run(False, out, b.workspace(False))
        i = b.inp
        s = abi.make_shape(cfg, out_dtype=abi.MOE_BF16)
        ws = torch.empty(abi.moe_workspace_size(s), dtype=torch.uint8, device=dev())
        want = torch.empty_like(out)
        abi.moe_layer_forward(s, b.x, i["w_router"], i["bias"], None, i["w_gate"], i["w_up"], i["w_down"],
                              i["ws_gate"], i["ws_up"], i["ws_down"], want, None, ws)
        assert torch.equal(out, want), name


def test_fp32_block():
    cfg = W.CONFIGS["tiny_fp32"].replace(name="block_f32", tokens=50)
    b = Block(cfg, stream="f32", seed=4, gate="token")
    out, d = f32((b.T, b.H)), b.debug()
    b.run(False, out, b.workspace(False), d)
    want = b.plain(False, d, np.arange(b.T))
    assert np.abs(np64(out) - want).max() <= 1e-4 * rms(want)


@pytest.mark.parametrize("int8", [False, True], ids=["bf16", "int8"])
@pytest.mark.parametrize("name", ["small_dropping", "one_token", "big_tiles", "decode"])
def test_block_in_a_graph(name, int8):
    """Captured once and replayed, with eager calls between, bit for bit; two graphs with a workspace each, replayed
    in turn and on different streams."""
    b = Block(CONFIGS[name], seed=5)
    x0 = b.x.clone()
    ref = torch.empty_like(x0)
    b.run(int8, ref, b.workspace(int8))
    b2 = Block(CONFIGS[name], seed=6)
    ref2 = torch.empty_like(x0)
    b2.run(int8, ref2, b2.workspace(int8))
    torch.cuda.synchronize()
    graphs = []
    for blk in (b, b2):
        ws, out = blk.workspace(int8), torch.empty_like(x0)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            blk.run(int8, out, ws)
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            blk.run(int8, out, ws)
        graphs.append((g, ws, out))
    for i in range(4):
        for (g, ws, out), want in zip(graphs, (ref, ref2)):
            out.fill_(float("nan"))
            ws.fill_(0xA5)
            torch.cuda.synchronize()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want), i
        eager = torch.empty_like(x0)
        b.run(int8, eager, b.workspace(int8))
        torch.cuda.synchronize()
        assert torch.equal(eager, ref)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for (g, ws, out), st in zip(graphs, streams):
        out.fill_(float("nan"))
    torch.cuda.synchronize()
    for _ in range(3):
        for (g, ws, out), st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    assert torch.equal(graphs[0][2], ref) and torch.equal(graphs[1][2], ref2)


@pytest.mark.parametrize("int8", [False, True], ids=["bf16", "int8"])
def test_block_on_two_streams_and_in_place(int8):
    b, b2 = Block(CONFIGS["groups_shared"], seed=7), Block(CONFIGS["groups_shared"], seed=8)
    refs = []
    for blk in (b, b2):
        out = torch.empty_like(blk.x)
        blk.run(int8, out, blk.workspace(int8))
        refs.append(out)
    torch.cuda.synchronize()
    work = [(blk, torch.empty_like(blk.x), blk.workspace(int8), torch.cuda.Stream()) for blk in (b, b2)]
    torch.cuda.synchronize()
    for _ in range(5):                                 # two calls at once, a workspace each
        for blk, out, ws, st in work:
            blk.run(int8, out, ws, stream=st.cuda_stream)
    torch.cuda.synchronize()
    for (blk, out, ws, st), want in zip(work, refs):
        assert torch.equal(out, want)
    x = b.x.clone()
    b.run(int8, x, b.workspace(int8), x=x)             # the residual stream updated in place
    assert torch.equal(x, refs[0])


def test_zero_tokens_enqueue_nothing():
    b = Block(CONFIGS["small"].replace(tokens=4), seed=9)
    b.shape.num_tokens = 0
    out = torch.full((4, b.H), 3.0, device=dev(), dtype=torch.bfloat16)
    ws = torch.empty(1 << 20, dtype=torch.uint8, device=dev())
    for int8 in (False, True):
        b.run(int8, out, ws)
    torch.cuda.synchronize()
    assert (out == 3.0).all()
