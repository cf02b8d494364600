"""Low-rank adapters of many requests on the GPU against their definition in 64 bits, at the sizes, layouts, orders
and values where they can go wrong.  Tolerances come from the arithmetic (more_ref.py)."""
import pytest
import torch

import dense_bf16_gemm_persistent_gb300 as gb
from tests import more_ref
from tests.block_ref import HALF_BF16, assert_within

pytestmark = pytest.mark.gpu

DEV, BF16 = "cuda", torch.bfloat16


def normal(*shape, seed, std=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return (torch.randn(shape, generator=g, device=DEV) * std).to(BF16)


def wide(*shape, seed, std):
    """Rows that start 16-byte aligned whatever their length, NaN between them."""
    pitch = -(-shape[-1] // 8) * 8
    t = torch.full((*shape[:-1], pitch), float("nan"), dtype=BF16, device=DEV)[..., :shape[-1]]
    t.copy_(normal(*shape, seed=seed, std=std))
    return t


def pick(m, low, high, seed):
    return torch.randint(low, high, (m,), generator=torch.Generator(device=DEV).manual_seed(seed), device=DEV).to(torch.int32)


def problem(m, n, k, r, adapters, seed=0, residual=True):
    return dict(X=wide(m, k, seed=seed, std=1.0), A=wide(adapters, r, k, seed=seed + 1, std=max(k, 1) ** -0.5),
                B=wide(adapters, n, r, seed=seed + 2, std=max(r, 1) ** -0.5), ids=pick(m, -1, adapters, seed + 3),
                scale=torch.rand(adapters, generator=torch.Generator(device=DEV).manual_seed(seed + 4), device=DEV) + 0.5,
                R=normal(m, n, seed=seed + 5) if residual else None)


def check(q, act="none", **kw):
    d = gb.lora(**q, act=act, **kw)
    assert_within(d, *more_ref.lora(q["X"], q["A"], q["B"], q["ids"], q["scale"], q["R"], act))
    return d


@pytest.mark.parametrize("m", [1, 2, 3, 7, 16, 31, 48, 64, 65, 200, 1000])
@pytest.mark.parametrize("adapters,r", [(1, 16), (5, 8), (40, 64)])
def test_rows_and_adapters(m, adapters, r):
    check(problem(m, 328, 512, r, adapters, seed=m + r))


@pytest.mark.parametrize("r", [1, 4, 8, 15, 16, 17, 24, 32, 33, 48, 64, 100, 128, 129, 250, 256])
@pytest.mark.parametrize("m", [3, 70])
def test_ranks(r, m):
    check(problem(m, 136, 264, r, 3, seed=r))


@pytest.mark.parametrize("n,k", [(1, 1), (1, 8), (7, 31), (8, 32), (33, 33), (127, 40), (129, 255), (1000, 96), (96, 1000),
                                 (4099, 72), (72, 4099), (2048, 14336), (14336, 256)])
@pytest.mark.parametrize("m", [1, 20, 130])
def test_sizes(n, k, m):
    check(problem(m, n, k, 16, 4, seed=n + k, residual=m != 20))


@pytest.mark.parametrize("m", [4096, 8191])
def test_many_rows(m):
    q = problem(m, 520, 1032, 32, 6, seed=m)
    check(q)
    q["ids"] = q["ids"].sort().values  # rows of a request together
    check(q)


@pytest.mark.parametrize("m", [31, 32, 64, 500, 8193, 20000])
@pytest.mark.parametrize("adapters", [1, 2, 300, 8191, 8192])
@pytest.mark.parametrize("r", [8, 24])
def test_pools_of_many_adapters(m, adapters, r):
    """Rows are sorted by up to 8191 adapters, and tile by tile beyond that; most tiles have one row of many, or all."""
    q = problem(m, 72, 64, r, adapters, seed=m + adapters)
    check(q)
    q["ids"] = pick(m, adapters - 1, adapters + 1, 3)  # the last one, or none
    d = check(q)
    assert torch.equal(d, gb.lora(**q))


@pytest.mark.parametrize("m", [32, 33, 63, 96, 127, 128, 129])
@pytest.mark.parametrize("adapters,r", [(1, 16), (2, 40), (3, 16), (90, 20), (9000, 16)])
def test_rows_that_each_block_sorts(m, adapters, r):
    """Tiles of 64 or 32 rows of one adapter, whole and cut off, and rows without one."""
    q = problem(m, 264, 200, r, adapters, seed=m + adapters)
    for ids in (pick(m, -2, adapters + 1, 1), pick(m, 0, 1, 2), pick(m, -1, 1, 3), pick(m, -5, 0, 4),
                torch.arange(m, dtype=torch.int32, device=DEV).flip(0) // 3):
        q["ids"] = ids
        d = check(q)
        assert torch.equal(d, gb.lora(**q))


@pytest.mark.parametrize("m,n", [(200, 4099), (300, 33), (65, 1001)])
@pytest.mark.parametrize("r", [16, 32, 64, 130])
def test_rows_that_start_anywhere_in_any_order(m, n, r):
    q = problem(m, n, 96, r, 7, seed=r)
    want = check(q)
    out = torch.full((m * n + 3,), 9.0, dtype=BF16, device=DEV)
    gb.lora(**q, out=out[1:1 + m * n].view(m, n))
    assert torch.equal(out[1:1 + m * n].view(m, n), want) and (out[[0, -2, -1]] == 9).all()


@pytest.mark.parametrize("act", ["none", "gelu_tanh", "silu", "relu"])
@pytest.mark.parametrize("residual", [True, False])
def test_epilogue(act, residual):
    check(problem(37, 200, 304, 16, 4, seed=3, residual=residual), act)


def test_a_scale_of_one_and_ids_that_name_no_adapter():
    q = problem(50, 96, 128, 16, 4, seed=6)
    q["scale"] = None
    q["ids"] = pick(50, -3, 9, 1)
    q["ids"][0], q["ids"][1] = 2 ** 31 - 1, -2 ** 31
    d = check(q)
    none = (q["ids"] < 0) | (q["ids"] >= 4)
    assert torch.equal(d[none], q["R"][none])


@pytest.mark.parametrize("m", [1, 33, 300])
def test_no_row_has_an_adapter(m):
    q = problem(m, 100, 64, 8, 3, seed=7)
    q["ids"][:] = -1
    assert torch.equal(gb.lora(**q), q["R"])
    q["R"] = None
    assert not gb.lora(**q).any()


def test_what_a_row_without_an_adapter_does_not_meet():
    """Neither NaN in X nor in the adapters reaches a row that has none, nor one that has another."""
    q = problem(40, 72, 96, 16, 3, seed=8)
    q["ids"][:] = torch.arange(40, device=DEV) % 3 - 1  # -1, 0, 1
    want, tol = more_ref.lora(q["X"], q["A"], q["B"], q["ids"], q["scale"], q["R"])
    q["A"][2], q["B"][2], q["scale"][2] = float("nan"), float("nan"), float("nan")
    q["X"][0], q["X"][3] = float("nan"), float("inf")
    q["X"][1, 5] = float("nan")
    d = gb.lora(**q)
    good = [i for i in range(40) if i != 1]
    assert_within(d[good], want[good], tol[good])
    assert torch.isnan(d[1]).all()


def test_infinities_of_x_come_out_as_they_are():
    q = problem(4, 24, 32, 8, 2, seed=9, residual=False)
    q["ids"][:] = 0
    q["A"][0] = 1.0
    q["B"][0] = torch.where(torch.arange(24, device=DEV)[:, None] % 2 == 0, 1.0, -1.0).to(BF16)
    q["X"][1, 3], q["X"][2, 4] = float("inf"), 3e38
    q["X"][2, 5] = 3e38
    d = gb.lora(**q)
    sign = torch.where(torch.arange(24, device=DEV) % 2 == 0, float("inf"), -float("inf"))
    assert torch.equal(d[1].float(), sign) and torch.equal(d[2].float(), sign)
    assert torch.isfinite(d[[0, 3]].float()).all()


def test_a_row_does_not_depend_on_the_others():
    q = problem(64, 264, 520, 24, 7, seed=10)
    d = gb.lora(**q)
    ids = q["ids"].clone()
    for change in (torch.full_like(ids, -1), (ids + 1) % 7, ids.flip(0)):
        keep = torch.arange(64, device=DEV) % 5 == 2
        q["ids"] = torch.where(keep, ids, change.to(torch.int32))
        assert torch.equal(gb.lora(**q)[keep], d[keep])


@pytest.mark.parametrize("extra,offset", [(8, 0), (3, 0), (0, 1), (5, 3)])
@pytest.mark.parametrize("m,n", [(5, 96), (19, 1000), (70, 333)])
def test_strides_and_offsets_of_r_and_d(m, n, extra, offset):
    q = problem(m, n, 64, 16, 3, seed=11)
    want = check(q)

    def buffer():
        return torch.full((m * (n + extra) + offset,), 9.0, dtype=BF16, device=DEV)[offset:].view(m, n + extra)
    r, out = buffer(), buffer()
    r[:, :n] = q["R"]
    q["R"] = r[:, :n]
    assert torch.equal(gb.lora(**q, out=out[:, :n]), want) and (out[:, n:] == 9).all()
    gb.lora(**q, out=r[:, :n])  # in place
    assert torch.equal(r[:, :n], want) and (r[:, n:] == 9).all()


def test_layouts_of_adapters():
    q = problem(30, 96, 128, 16, 4, seed=12)
    pool = torch.full((4, 16 * 128 + 96 * 24 + 8), float("nan"), dtype=BF16, device=DEV)  # an adapter's both together
    a = pool[:, :16 * 128].view(4, 16, 128)
    b = pool[:, 16 * 128:16 * 128 + 96 * 24].view(4, 96, 24)[:, :, :16]
    a.copy_(q["A"])
    b.copy_(q["B"])
    want = check(q)
    q["A"], q["B"] = a, b
    assert torch.equal(gb.lora(**q), want)


def test_single_rows_of_any_stride():
    """The stride of a dimension of one says nothing."""
    q = problem(1, 40, 64, 1, 1, seed=21)
    q["ids"][:] = 0
    want = check(q)
    far = 1 << 40
    q["X"], q["R"] = q["X"].as_strided((1, 64), (far, 1)), q["R"].as_strided((1, 40), (far, 1))
    q["A"] = q["A"].as_strided((1, 1, 64), (far, far, 1))
    assert torch.equal(gb.lora(**q), want)
    q = problem(70, 1, 64, 8, 2, seed=22)
    want = check(q)
    q["B"] = q["B"].as_strided((2, 1, 8), (q["B"].stride(0), far, 1))
    assert torch.equal(gb.lora(**q), want)


def test_a_long_pool_of_adapters():
    """Offsets of adapters pass 2^31 elements."""
    count, r, k, n = 1100, 128, 16384, 40
    q = dict(X=normal(6, k, seed=1), B=normal(count, n, r, seed=2, std=0.1), scale=None, R=None,
             A=torch.randn((count, r, k), dtype=BF16, device=DEV) * k ** -0.5,
             ids=torch.tensor([count - 1, 0, 1050, 1050, -1, 1099], dtype=torch.int32, device=DEV))
    assert q["A"].numel() > 2 ** 31
    check(q)


@pytest.mark.parametrize("m", [5, 40, 200])
def test_millions_of_adapters(m):
    """More than are sorted by: tiles of consecutive rows."""
    count = (1 << 22) + 3
    q = dict(X=normal(m, 8, seed=1), A=normal(count, 1, 8, seed=2), B=normal(count, 8, 8, seed=3)[:, :, :1], scale=None,
             R=normal(m, 8, seed=4), ids=pick(m, count - 5, count + 2, 5))
    assert torch.equal(check(q), gb.lora(**q))


@pytest.mark.parametrize("m", [5, 40, 130])
def test_rows_that_lie_far_apart(m):
    """A matrix of 2^31 elements and more, whose rows' distances are not counted in 32 bits: X, then R and D."""
    ld = (2 ** 31 // m // 8 + 1) * 8
    q = problem(m, 72, 64, 16, 3, seed=m)
    want = check(q)
    far = torch.empty(m * ld, dtype=BF16, device=DEV)
    wide = far.as_strided((m, 72), (ld, 1))
    assert m * ld > 2 ** 31
    x = q["X"]
    q["X"] = wide[:, :64].copy_(x)
    check(q)
    q["X"], r = x, q["R"]
    q["R"] = wide.copy_(r)
    d = gb.lora(**q, out=wide)
    assert_within(d, *more_ref.lora(x, q["A"], q["B"], q["ids"], q["scale"], r))
    assert d.shape == want.shape


def test_nothing_to_do():
    q = problem(5, 48, 64, 8, 3, seed=13)
    for change in (dict(A=q["A"][:0], B=q["B"][:0], scale=q["scale"][:0]), dict(X=q["X"][:, :0], A=q["A"][:, :, :0]),
                   dict(A=q["A"][:, :0], B=q["B"][:, :, :0])):
        assert torch.equal(gb.lora(**{**q, **change}), q["R"])
    assert gb.lora(**{**q, "X": q["X"][:0], "ids": q["ids"][:0], "R": q["R"][:0]}).shape == (0, 48)
    assert gb.lora(**{**q, "B": q["B"][:, :0], "R": None}).shape == (5, 0)


def test_results_repeat_also_in_a_graph_on_another_stream():
    q = problem(100, 520, 1000, 32, 9, seed=14)
    first = gb.lora(**q).clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    again = gb.lora(**q, stream=side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = gb.lora(**q)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(first, again) and torch.equal(first, captured)
    q["ids"].copy_(pick(100, -1, 9, 99))  # a replayed graph reads the ids again
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(captured, gb.lora(**q))


@pytest.mark.parametrize("m", [20, 48, 300])
def test_a_graph_of_one_request_serves_many(m):
    """How many tiles there are changes from replay to replay: from one adapter's to one for each row."""
    q = problem(m, 264, 520, 40, 300, seed=m)
    q["ids"].zero_()
    gb.lora(**q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = gb.lora(**q)
    for ids in (torch.arange(m), torch.arange(m) // 7 * 3 - 1, torch.full((m,), -1), torch.zeros(m)):
        q["ids"].copy_(ids)
        graph.replay()
        torch.cuda.synchronize()
        assert_within(captured, *more_ref.lora(q["X"], q["A"], q["B"], q["ids"], q["scale"], q["R"]))


def test_the_workspace_is_checked_and_any_contents_do():
    q = problem(20, 96, 512, 16, 4, seed=15)
    need = gb.lora_workspace_bytes(20, 96, 512, 16)
    check(q, workspace=torch.full((need,), 255, dtype=torch.uint8, device=DEV))
    with pytest.raises(ValueError, match="workspace"):
        gb.lora(**q, workspace=torch.empty(need - 1, dtype=torch.uint8, device=DEV))


@pytest.mark.parametrize("m", [4, 600])
def test_beside_a_shared_projection(m):
    """Adapters first and the projection on top, and the projection first with its activation after the adapters."""
    q = problem(m, 256, 512, 16, 5, seed=16, residual=False)
    w, bias, r = normal(256, 512, seed=17, std=512 ** -0.5), normal(256, seed=18), normal(m, 256, seed=19)
    x = q["X"]
    delta, tol = more_ref.lora(x, q["A"], q["B"], q["ids"], q["scale"], r)
    base = x.double() @ w.double().T + bias.double()
    size = (512 + 8) * 2.0 ** -23 * (x.double().abs() @ w.double().abs().T) + 2.0 ** -23 * base.abs()
    want = base + delta
    d = gb.linear(x, w, bias, R=gb.lora(**{**q, "R": r}))
    assert_within(d, want, tol + size + HALF_BF16 * (want.abs() + tol + size) + 1e-37)
    z = gb.linear(x, w, bias)
    got = gb.lora(**{**q, "R": z}, act="gelu_tanh")
    assert_within(got, *more_ref.lora(x, q["A"], q["B"], q["ids"], q["scale"], z, "gelu_tanh"))


def test_wrong_tensors_are_refused():
    q = problem(4, 48, 64, 16, 3, seed=20)
    for change, error, what in (
            (dict(X=q["X"].float()), TypeError, "X"), (dict(A=q["A"][0]), ValueError, "A"), (dict(B=q["B"][:2]), ValueError, "B"),
            (dict(A=q["A"][:, :8]), ValueError, "B"), (dict(ids=q["ids"].long()), TypeError, "ids"),
            (dict(ids=q["ids"][:2]), ValueError, "ids"), (dict(ids=None), TypeError, "ids"),
            (dict(scale=q["scale"].double()), TypeError, "scale"), (dict(scale=q["scale"][:1]), ValueError, "scale"),
            (dict(R=q["R"][:, :40]), ValueError, "R"), (dict(act="tanh"), ValueError, "act"),
            (dict(A=q["A"].transpose(1, 2)), ValueError, "A"),
            (dict(X=torch.zeros((4, 68), dtype=BF16, device=DEV)[:, :64]), gb.GBError, "X"),
            (dict(A=torch.zeros((3, 260, 64), dtype=BF16, device=DEV), B=torch.zeros((3, 48, 260), dtype=BF16, device=DEV)),
             gb.GBError, "rank")):
        with pytest.raises(error, match=what):
            gb.lora(**{**q, **change})
