"""The mixture-of-experts layer for a few tokens on the GPU against its definition in 64 bits, at the sizes,
layouts and values where it can go wrong.  Tolerances come from the arithmetic (more_ref.py)."""
import pytest
import torch

import dense_bf16_gemm_persistent_gb300 as gb
from tests import more_ref
from tests.block_ref import assert_within

pytestmark = pytest.mark.gpu

DEV, BF16 = "cuda", torch.bfloat16


def normal(*shape, seed, std=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return (torch.randn(shape, generator=g, device=DEV) * std).to(BF16)


def wide(*shape, seed, std):
    """Rows that start 16-byte aligned whatever their length."""
    pitch = -(-shape[-1] // 8) * 8
    t = torch.full((*shape[:-1], pitch), float("nan"), dtype=BF16, device=DEV)[..., :shape[-1]]
    t.copy_(normal(*shape, seed=seed, std=std))
    return t


def layer(t, d, inner, experts, seed=0, residual=True):
    return dict(X=wide(t, d, seed=seed, std=1.0), router=wide(experts, d, seed=seed + 1, std=2 * d ** -0.5),
                W1=wide(experts, inner, d, seed=seed + 2, std=d ** -0.5),
                W3=wide(experts, inner, d, seed=seed + 3, std=d ** -0.5),
                W2=wide(experts, d, inner, seed=seed + 4, std=inner ** -0.5),
                R=normal(t, d, seed=seed + 5) if residual else None)


def check(a, top_k, renormalize=True, **kw):
    out, ids, weights = gb.moe_ffn_gated(**a, top_k=top_k, renormalize=renormalize, **kw)
    want_ids, want_w = more_ref.routing(a["X"], a["router"], top_k, renormalize)
    assert ids.dtype == torch.int32 and torch.equal(ids.long(), want_ids)
    # exp to 2 ulp of its value and 2^-24 of its argument (below 64 here), a tree of sums, a quotient
    assert_within(weights, want_w, want_w * 2.0 ** -17 + 1e-38, "weights")
    want, tol = more_ref.moe(a["X"], a["W1"], a["W3"], a["W2"], a["R"], want_ids, want_w)
    assert_within(out, want, tol + 2.0 ** -17 * (want - (a["R"].double() if a["R"] is not None else 0)).abs() * 4, "D")
    return out, ids, weights


@pytest.mark.parametrize("t", [1, 2, 5, 8, 9, 16, 17, 31, 33, 63, 64])
@pytest.mark.parametrize("experts,top_k", [(1, 1), (4, 2), (8, 8), (40, 3)])
def test_tokens_and_experts(t, experts, top_k):
    check(layer(t, 256, 96, experts, seed=t), top_k, renormalize=t % 2 == 0)


@pytest.mark.parametrize("d,inner", [(1, 1), (8, 1), (7, 9), (31, 33), (32, 32), (40, 17), (100, 250), (264, 1000), (1000, 264),
                                     (4096, 48), (48, 4096), (2056, 1416), (4099, 515)])
@pytest.mark.parametrize("t", [1, 11])
def test_sizes(d, inner, t):
    check(layer(t, d, inner, 6, seed=d + inner, residual=t == 11), 2)


@pytest.mark.parametrize("experts,top_k", [(2, 1), (33, 16), (64, 8), (100, 6), (256, 8), (1024, 16)])
def test_many_experts(experts, top_k):
    check(layer(23, 64, 40, experts, seed=experts), top_k)
    check(layer(64, 64, 24, experts, seed=experts + 1), top_k, renormalize=False)


@pytest.mark.parametrize("t", [65, 128, 150])
def test_more_tokens_than_a_pass(t):
    check(layer(t, 136, 72, 12, seed=t), 4)


def test_every_token_chooses_the_same_expert():
    a = layer(64, 128, 80, 8, seed=3)
    a["X"] = normal(64, 128, seed=1).abs() + 0.5
    a["router"][5] = 1.0
    _, ids, _ = check(a, 1)
    assert (ids == 5).all()


def test_equal_logits_go_to_the_lower_expert():
    a = layer(7, 64, 32, 40, seed=1)
    a["router"][:] = a["router"][0]
    _, ids, w = check(a, 5)
    assert torch.equal(ids, torch.arange(5, dtype=torch.int32, device=DEV).expand(7, 5))
    a["router"][:] = 0  # (and all of them zero)
    check(a, 3, renormalize=False)


def test_logits_that_32_bits_cannot_tell_apart():
    """The logits differ by 2^-20 and pass through sums of 2^11, beside which fp32 keeps 2^-13."""
    a = layer(4, 512, 32, 4, seed=2)
    a["X"][:] = 1.0
    a["router"][:] = 0
    a["router"][:, 0:128], a["router"][:, 384:512] = 256.0, -256.0
    a["router"][2, 256], a["router"][1, 256] = 2.0 ** -20, 2.0 ** -19
    _, ids, _ = check(a, 2)
    assert torch.equal(ids, torch.tensor([[1, 2]] * 4, dtype=torch.int32, device=DEV))


def test_nan_and_infinities_stay_with_their_tokens():
    a = layer(9, 96, 64, 8, seed=4)
    a["X"][2, 3], a["X"][5, 95] = float("nan"), float("inf")
    out, ids, w = gb.moe_ffn_gated(**a, top_k=2)
    good = [0, 1, 3, 4, 6, 7, 8]
    b = dict(a, X=a["X"][good].contiguous(), R=a["R"][good].contiguous())
    want_ids, want_w = more_ref.routing(b["X"], b["router"], 2, True)
    assert torch.equal(ids[good].long(), want_ids)
    want, tol = more_ref.moe(b["X"], b["W1"], b["W3"], b["W2"], b["R"], want_ids, want_w)
    assert_within(out[good], want, tol + 2.0 ** -14 * (want - b["R"].double()).abs())
    assert torch.isnan(out[2]).all() and torch.isnan(w[2]).all()
    for row in ids.tolist():  # every choice is one of distinct experts
        assert len(set(row)) == 2 and all(0 <= e < 8 for e in row)


def test_a_logit_that_is_nan_is_chosen_last():
    a = layer(3, 64, 32, 5, seed=5)
    a["router"][1, 0] = float("nan")
    _, ids, w = gb.moe_ffn_gated(**a, top_k=5)
    assert (ids[:, 4] == 1).all() and torch.isnan(w).all()


def test_large_logits_and_weights_of_one_expert():
    a = layer(5, 128, 64, 6, seed=6)
    a["router"] *= 200  # softmax: one expert has all of it, and others underflow
    out, ids, w = check(a, 3, renormalize=False)
    assert w[:, 0].min() > 0.2


def test_layouts_of_weights():
    a = layer(6, 72, 56, 4, seed=7)
    joined = torch.empty((4, 2, 56, 80), dtype=BF16, device=DEV)  # W1 and W3 of an expert beside each other
    joined[:, 0, :, :72], joined[:, 1, :, :72] = a["W1"], a["W3"]
    a["W1"], a["W3"] = joined[:, 0, :, :72], joined[:, 1, :, :72]
    big = torch.empty((4, 72, 64), dtype=BF16, device=DEV)
    big[:, :, :56] = a["W2"]
    a["W2"] = big[:, :, :56]
    a["X"] = torch.cat([a["X"], a["X"]], dim=1)[:, :72]
    check(a, 2)
    a["W1"] = a["W1"].flip(0)  # (a copy: distances of experts are positive)
    check(a, 2)


def test_out_and_residual_of_any_stride_and_in_place():
    a = layer(10, 88, 48, 4, seed=8)
    buf = torch.full((10, 95), 9.0, dtype=BF16, device=DEV)
    buf2 = torch.full((10 * 91 + 1,), 9.0, dtype=BF16, device=DEV)
    r = buf2[1:].view(10, 91)[:, 3:]
    r.copy_(a["R"])
    a["R"] = r
    want = check(a, 2)[0]
    out = buf[:, 5:93]
    got = check(a, 2, out=out)[0]
    assert got is out and torch.equal(out, want) and (buf[:, :5] == 9).all() and (buf[:, 93:] == 9).all()
    gb.moe_ffn_gated(**a, top_k=2, out=r)
    assert torch.equal(r, want)


def test_no_tokens():
    a = layer(3, 64, 32, 4)
    a["X"], a["R"] = a["X"][:0], a["R"][:0]
    out, ids, w = gb.moe_ffn_gated(**a, top_k=2)
    assert out.shape == (0, 64) and ids.shape == w.shape == (0, 2)


def test_a_long_stack_of_experts():
    """Offsets of experts pass 2^31 elements."""
    experts, inner, d = 72, 3840, 8192
    a = dict(X=normal(4, d, seed=1), router=torch.zeros((experts, d), dtype=BF16, device=DEV), R=None)
    for name, shape in (("W1", (experts, inner, d)), ("W3", (experts, inner, d)), ("W2", (experts, d, inner))):
        a[name] = torch.randn(shape, dtype=BF16, device=DEV) * shape[2] ** -0.5
    assert a["W1"].numel() > 2 ** 31
    a["router"][70], a["router"][71] = normal(d, seed=2, std=0.001).abs(), normal(d, seed=3, std=0.001).abs()
    a["X"].abs_()
    _, ids, _ = check(a, 2)
    assert (ids >= 70).all()


def test_results_repeat_also_in_a_graph_on_another_stream():
    a = layer(19, 520, 200, 16, seed=9)
    first = [t.clone() for t in gb.moe_ffn_gated(**a, top_k=4)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    again = gb.moe_ffn_gated(**a, top_k=4, stream=side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = gb.moe_ffn_gated(**a, top_k=4)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    for x, y, z in zip(first, again, captured):
        assert torch.equal(x, y) and torch.equal(x, z)
    a["X"].copy_(normal(19, 520, seed=77))  # a replayed graph chooses again
    graph.replay()
    torch.cuda.synchronize()
    for x, y in zip(gb.moe_ffn_gated(**a, top_k=4), captured):
        assert torch.equal(x, y)


def test_the_workspace_is_checked_and_any_contents_do():
    a = layer(5, 64, 33, 6, seed=10)
    need = gb.moe_ffn_gated_workspace_bytes(5, 33, 6, 2)
    check(a, 2, workspace=torch.full((need,), 255, dtype=torch.uint8, device=DEV))
    with pytest.raises(ValueError, match="workspace"):
        gb.moe_ffn_gated(**a, top_k=2, workspace=torch.empty(need - 1, dtype=torch.uint8, device=DEV))


def test_wrong_tensors_are_refused():
    a = layer(3, 64, 32, 4)
    for change, error, what in (
            (dict(X=a["X"].float()), TypeError, "X"), (dict(router=a["router"][:, :32]), ValueError, "router"),
            (dict(W1=a["W1"][:3]), ValueError, "W1"), (dict(W3=a["W1"][0]), ValueError, "W3"),
            (dict(W2=a["W1"]), ValueError, "W2"), (dict(W2=a["W1"].transpose(1, 2)), ValueError, "W2"),
            (dict(R=a["R"][:2]), ValueError, "R"), (dict(top_k=0), gb.GBError, "top_k"),
            (dict(top_k=5), gb.GBError, "top_k"), (dict(X=torch.zeros((3, 68), dtype=BF16, device=DEV)[:, 4:]), gb.GBError, "X"),
            (dict(W1=a["W1"].reshape(-1)[:4 * 30 * 64].view(4, 30, 64)), ValueError, "W3"),
            (dict(W1=torch.zeros((4, 32 * 64 + 4), dtype=BF16, device=DEV)[:, :2048].view(4, 32, 64)), gb.GBError, "W1")):
        with pytest.raises(error, match=what):
            gb.moe_ffn_gated(**{**a, "top_k": 2, **change})
