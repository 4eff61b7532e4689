"""Routing with a balance bias against the plain 64-bit form: the choice exact, gates within one rounding to fp32
(2^-24 relative, and 1e-13 for the 64-bit steps before it)."""

import numpy as np
import pytest
import torch

import workloads as W
from expert_serving_amd import abi

import plain_block as P
from gpu_util import dev, f32, i32, say, workspace

pytestmark = pytest.mark.gpu
NEG = -np.inf


def shape_of(T, E, k, o):
    return abi.make_shape(num_tokens=T, hidden=64, num_experts=E, intermediate=64, top_k=k,
                          score=int(o.get("score", "sigmoid") == "sigmoid"), renormalize=int(o.get("renorm", True)),
                          routed_scale=o.get("scale", 1.0), num_groups=o.get("G", 1), topk_groups=o.get("keep", 1),
                          group_topn=o.get("topn", 0))


def route(logits, bias, k, kpt=None, **o):
    T, E = logits.shape
    s = shape_of(T, E, k, o)
    ids, gates, ws = i32(T * k, -7).view(T, k), f32((T, k)).fill_(-7.0), workspace(s)
    kd = None if kpt is None else torch.from_numpy(np.asarray(kpt, np.int32)).to(dev())
    abi.moe_route_biased(s, None, None, None, torch.from_numpy(bias).to(dev()), torch.from_numpy(logits).to(dev()),
                         None, kd, ids, gates, ws)
    torch.cuda.synchronize()
    return ids.cpu().numpy(), gates.cpu().numpy(), abi.moe_read_device_flags(ws)


def check(logits, bias, k, kpt=None, **o):
    logits, bias = np.ascontiguousarray(logits, np.float32), np.ascontiguousarray(bias, np.float32)
    ids, gates, flags = route(logits, bias, k, kpt, **o)
    want, w = P.route_biased(logits, bias, k, kpt, **o)
    assert np.array_equal(ids, want), np.nonzero((ids != want).any(1))[0][:5]
    assert np.all(np.abs(gates - w) <= (P.U32 + 1e-13) * np.abs(w) + 1e-45)
    # many tokens share wavefronts, few have one each: the same tokens in a large and odd batch (the fp64 sums of
    # gates may be formed in another order)
    T = len(logits)
    if T <= 1024:
        n = 1027 // T + 1
        many, g2, f2 = route(np.tile(logits, (n, 1)), bias, k, None if kpt is None else np.tile(kpt, n), **o)
        assert np.array_equal(many, np.tile(ids, (n, 1))) and f2 == flags
        assert np.all(np.abs(g2 - np.tile(w, (n, 1))) <= (P.U32 + 1e-13) * np.abs(np.tile(w, (n, 1))) + 1e-45)
    return ids, gates, flags


CASES = {
    "one_token_groups": (1, 256, 8, dict(G=8, keep=4, topn=2, scale=2.5)),
    "groups_256": (1003, 256, 8, dict(G=8, keep=4, topn=2, scale=2.5)),
    "groups_512_topn8": (67, 512, 16, dict(G=4, keep=2, topn=8)),
    "groups_lds": (130, 72, 6, dict(G=6, keep=3, topn=3)),
    "groups_lds_64": (31, 448, 5, dict(G=64, keep=20, topn=2, score="softmax")),
    "groups_of_one": (33, 60, 4, dict(G=60, keep=7)),
    "groups_all_kept": (40, 96, 8, dict(G=3, keep=3, topn=1, score="softmax")),
    "softmax": (515, 128, 8, dict(score="softmax")),
    "softmax_plain_gates": (100, 511, 3, dict(score="softmax", renorm=False, scale=2.0)),
    "sigmoid_plain_gates": (100, 65, 1, dict(renorm=False)),
    "all_experts": (9, 8, 8, dict()),
    "one_expert": (5, 1, 1, dict(score="softmax")),
}


@pytest.mark.parametrize("name", CASES)
def test_choice_and_gates(name):
    T, E, k, o = CASES[name]
    say(f"route_biased {name}")
    r = np.random.default_rng(len(name) * 1000 + E)
    logits = r.normal(size=(T, E)) * 2
    bias = r.normal(size=E) * (0.2 if o.get("score", "sigmoid") == "sigmoid" else 0.5 / E)
    check(logits, bias, k, **o)


@pytest.mark.parametrize("score,G", [("sigmoid", 1), ("softmax", 1), ("sigmoid", 4)])
def test_equal_keys_go_to_the_lower_expert(score, G):
    r = np.random.default_rng(5)
    logits, bias = r.normal(size=(200, 64)).astype(np.float32), (r.normal(size=64) * 0.1).astype(np.float32)
    logits[:, 32:] = logits[:, :32]           # experts e and e + 32 tie in every token
    bias[32:] = bias[:32]
    logits[::7] = 0.25                        # and here whole rows do
    ids, _, _ = check(logits, bias, 8, score=score, G=G, keep=max(1, G // 2), topn=2)
    bias[:] = 0
    ids, _, _ = check(logits, bias, 8, score=score, G=G, keep=max(1, G // 2), topn=2)
    if G == 1:
        assert np.array_equal(ids[0], np.arange(8))


def test_saturated_scores_keep_their_order():
    """Logits 16 to 23: one fp32 sigmoid, eight different scores; the choice follows the logit."""
    logits = np.tile(np.arange(16, 24, dtype=np.float32), (3, 1))
    ids, _, _ = check(logits, np.zeros(8), 4)
    assert np.array_equal(ids[0], [7, 6, 5, 4])


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_experts_out_of_service_nan_and_infinite_logits(score):
    r = np.random.default_rng(9)
    logits, bias = r.normal(size=(120, 40)).astype(np.float32), np.zeros(40, np.float32)
    bias[[3, 17, 39]] = NEG
    bias[8] = np.nan
    logits[:, 17] = np.nan                    # a masked place may hold anything
    logits[:, 39] = np.inf
    logits[5, :] = np.nan                     # nothing left
    logits[6, 1:] = np.nan                    # one expert left
    logits[7, 4], logits[8, 4], logits[9, 4] = np.inf, -np.inf, np.nan
    logits[10, :] = -np.inf
    logits[11, 0:20] = np.inf
    logits[12, :] = -3.0e38
    ids, gates, _ = check(logits, bias, 6, score=score)
    assert (ids[5] == -1).all() and (gates[5] == 0).all() and (ids[6][1:] == -1).all()
    assert not np.isin(ids, [3, 8, 17, 39]).any() and np.isfinite(gates).all()
    check(logits, bias, 6, score=score, G=4, keep=2, topn=2)
    bias[:] = NEG
    ids, gates, _ = check(logits, bias, 6, score=score)
    assert (ids == -1).all() and (gates == 0).all()
    bias[:] = 0
    bias[[2, 30]] = np.inf                    # forced into every token
    ids, _, _ = check(logits[:5], bias, 6, score=score)
    assert (ids[:, 0] == 2).all() and (ids[:, 1] == 30).all()


def test_groups_with_few_available_experts():
    r = np.random.default_rng(11)
    logits, bias = r.normal(size=(64, 32)).astype(np.float32), np.zeros(32, np.float32)
    bias[0:8] = NEG                           # group 0 has none
    bias[9:16] = NEG                          # group 1 has one
    ids, _, _ = check(logits, bias, 5, G=4, keep=3, topn=3)
    assert not (ids == 0).any()
    bias[16:32] = NEG                         # one expert in all
    ids, _, _ = check(logits, bias, 5, G=4, keep=3, topn=3)
    assert (ids[:, 0] == 8).all() and (ids[:, 1:] == -1).all()


def test_gates_of_scores_that_vanish():
    logits = np.full((2, 4), -3.0e38, np.float32)
    _, gates, _ = check(logits, np.zeros(4), 2)            # sigmoid 0 everywhere: gates of 0
    assert (gates == 0).all()


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E,G,keep,topn", [(256, 1, 1, 1), (256, 8, 4, 2), (72, 6, 2, 3), (16, 1, 1, 1), (512, 4, 3, 1)])
def test_keys_closer_than_fp32_can_tell(score, E, G, keep, topn):
    """Logits one fp32 step apart around a few values, and biases that put different logits at nearly one key: the
    order is that of the fp64 keys."""
    r = np.random.default_rng(E + G)
    T = 130
    base = r.choice(np.array([-2.0, 0.25, 1.0, 1.5], np.float32), size=(T, E))
    logits = base.copy()
    for _ in range(3):
        logits = np.where(r.random((T, E)) < 0.5, np.nextafter(logits, np.float32(9)), logits)
    check(logits, np.zeros(E), 8, score=score, G=G, keep=keep, topn=topn)
    if score == "sigmoid":   # sigmoid(1) - sigmoid(0.25) between the two halves, to fp32
        gap = np.float32(1 / (1 + np.exp(-1.0)) - 1 / (1 + np.exp(-0.25)))
        logits[:, :E // 2] = np.where(r.random((T, E // 2)) < 0.5, 1.0, np.nextafter(np.float32(1), np.float32(2)))
        logits[:, E // 2:] = np.where(r.random((T, E // 2)) < 0.5, 0.25, np.nextafter(np.float32(0.25), np.float32(1)))
        bias = np.zeros(E, np.float32)
        bias[E // 2:] = gap
        bias[::3] = np.nextafter(bias[::3], np.float32(1))
        check(logits, bias, 8, score=score, G=G, keep=keep, topn=topn)
        check(logits, bias * np.float32(-1e4), 8, score=score, G=G, keep=keep, topn=topn)
    # one token in which only one pair is close, at every place of the order
    for j in range(8):
        one = np.arange(E, 0, -1).astype(np.float32)[None] * np.float32(0.01)
        one[0, j + 1] = np.nextafter(one[0, j], np.float32(9 if j % 2 else -9))
        check(one, np.zeros(E), 8, score=score, G=G, keep=keep, topn=topn)


@pytest.mark.parametrize("k", [15, 16])
def test_close_keys_with_every_slot_used(k):
    r = np.random.default_rng(k)
    logits = (np.float32(1) + r.integers(0, 40, (50, 128)) * np.float32(2 ** -23)).astype(np.float32)
    check(logits, np.zeros(128), k)
    kpt = r.integers(1, k + 1, 50)
    check(logits, np.zeros(128), k, kpt)


def test_many_tokens_with_k_per_token():
    """More tokens than one launch looks through for bad budgets."""
    T = 40000
    lg = W.make_logits(T, 16, "cpu", seed=4).numpy()
    kpt = np.full(T, 2, np.int32)
    for bad in (None, T - 1):
        if bad is not None:
            kpt[bad] = 5
        ids, gates, flags = route(lg, np.zeros(16, np.float32), 4, kpt)
        assert flags == (0 if bad is None else abi.MOE_FLAG_BAD_K)
        want, _ = P.route_biased(lg[-50:], np.zeros(16), 4, kpt[-50:])
        assert np.array_equal(ids[-50:], want)


def test_k_per_token_and_bad_k():
    r = np.random.default_rng(3)
    logits, bias = r.normal(size=(300, 128)), r.normal(size=128) * 0.1
    kpt = r.integers(1, 9, 300)
    _, _, flags = check(logits, bias, 8, kpt)
    assert flags == 0
    kpt[[0, 4, 299]] = [0, 9, -3]
    _, _, flags = check(logits, bias, 8, kpt)
    assert flags == abi.MOE_FLAG_BAD_K


@pytest.mark.parametrize("T,E,H", [(5, 16, 512), (40, 64, 1024), (2048, 128, 1024), (2049, 256, 2048)])
def test_from_activations(T, E, H):
    """With x and a router: the choice on the logits it reports (the last two sizes split the router's K)."""
    k = 4
    x = W.normal((T, H), 1.0, W.DT_BF16, dev(), 1)
    wr = W.normal((E, H), H ** -0.5, W.DT_BF16, dev(), 2)
    rb = W.normal((E,), 0.3, W.DT_F32, dev(), 3)
    bias = W.normal((E,), 0.1, W.DT_F32, dev(), 4)
    s = abi.make_shape(num_tokens=T, hidden=H, num_experts=E, intermediate=64, top_k=k, score=1)
    ids, gates, lo, ws = i32((T, k)), f32((T, k)), f32((T, E)), workspace(s)
    abi.moe_route_biased(s, x, wr, rb, bias, None, lo, None, ids, gates, ws)
    torch.cuda.synchronize()
    own = x.double().cpu() @ wr.double().cpu().t() + rb.double().cpu()
    assert (lo.double().cpu() - own).abs().max() <= 1e-5 * own.square().mean().sqrt()
    n = min(T, 300)
    want, w = P.route_biased(lo[:n].cpu().numpy(), bias.cpu().numpy(), k)
    assert np.array_equal(ids[:n].cpu().numpy(), want)
    assert np.all(np.abs(gates[:n].cpu().numpy() - w) <= (P.U32 + 1e-13) * w)


def test_a_zero_bias_is_the_plain_router():
    """Bias 0, one group: the ids of moe_route_topk (gates too, to two roundings of its fp32 steps)."""
    lg = W.make_logits(700, 128, dev(), seed=8, tie_fraction=0.1)
    s = abi.make_shape(num_tokens=700, hidden=64, num_experts=128, intermediate=64, top_k=6)
    a, b, ga, gb, ws = i32((700, 6)), i32((700, 6)), f32((700, 6)), f32((700, 6)), workspace(s)
    abi.moe_route_topk(s, None, None, None, lg, None, None, a, ga, ws)
    abi.moe_route_biased(s, None, None, None, torch.zeros(128, device=dev()), lg, None, None, b, gb, ws)
    assert torch.equal(a, b) and torch.allclose(ga, gb, rtol=1e-6, atol=0)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E,topn", [(2, 1), (16, 1), (16, 2), (72, 1), (72, 2), (72, 3), (256, 1), (256, 2), (256, 3),
                                    (256, 8), (510, 2), (512, 3)])
def test_two_groups(E, topn, score):
    """Half the experts a group: the widest merges of the groups' lists, with keys far apart and closer than fp32."""
    say(f"route_biased two groups of {E // 2}, topn {topn}, {score}")
    r = np.random.default_rng(E * 10 + topn)
    k = min(8, E // 2)
    o = dict(score=score, G=2, topn=topn)
    for T in (1, 203):
        logits, bias = r.normal(size=(T, E)) * 2, r.normal(size=E) * (0.2 if score == "sigmoid" else 0.5 / E)
        check(logits, bias, k, keep=1, **o)
        check(logits, bias, k, keep=2, **o)
        base = r.choice(np.array([-2.0, 0.25, 1.0], np.float32), size=(T, E))
        near = np.where(r.random((T, E)) < 0.5, np.nextafter(base, np.float32(9)), base)
        near[:, E // 2:] = near[:, :E // 2]               # equal groups: the lower one
        near[1::3, E - 1] = np.nextafter(np.float32(1), np.float32(9))
        check(near, np.zeros(E), k, keep=1, **o)
        out = np.zeros(E)
        out[:E // 2 - 1] = NEG                            # one expert left in the first group
        check(logits, out, k, keep=1, **o)
        check(logits, out, k, keep=2, **o)


def test_keys_that_are_equal_in_fp64_go_to_the_lower_expert():
    """Sigmoids of logits from 37 on are 1; scores far below a bias's resolution leave its keys equal."""
    logits = np.tile(np.arange(30, 46, dtype=np.float32), (3, 1))
    ids, gates, _ = check(logits, np.zeros(16), 12)
    assert np.array_equal(ids[0], [7, 8, 9, 10, 11, 12, 13, 14, 15, 6, 5, 4]) and (gates[0, :9] == gates[0, 0]).all()
    ids, _, _ = check(logits[:, ::-1], np.zeros(16), 4)
    assert np.array_equal(ids[0], [0, 1, 2, 3])
    ids, _, _ = check(logits, np.zeros(16), 4, G=4, keep=2, topn=2)      # groups 2 and 3 tie, then their experts
    assert np.array_equal(ids[0], [8, 9, 10, 11])
    small = np.array([[-43, -42, -41, -40, 0]] * 2, np.float32)
    ids, _, _ = check(small, np.zeros(5), 4, score="softmax")
    assert np.array_equal(ids[0], [4, 3, 2, 1])
    ids, _, _ = check(small, np.full(5, 100.0), 4, score="softmax")
    assert np.array_equal(ids[0], [4, 0, 1, 2])
