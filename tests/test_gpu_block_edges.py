"""Calls around the products that were once answered wrongly, refused or unsafe, each against its definition in
64 bits (block_ref.py)."""
import pytest
import torch

import dense_bf16_gemm_persistent_gb300 as gb
from tests import block_ref as ref
from tests.block_ref import HALF_BF16, TINY, assert_within
from tests.test_gpu_block import BF16, DEV, check_linear_result, normal, w4_input, w4_weights

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------------------------- scales of 8-bit rows

def test_w4_row_scales_in_one_dimension():
    """[M] scales, contiguous and with a stride, are the [M,1] ones."""
    m, n, k, group = 9, 70, 288, 64
    q, s, z = w4_weights(n, k, group, True, 1)
    x, xs = w4_input(m, k, "row", 2)
    xs = xs * torch.arange(1, m + 1, device=DEV)[:, None]  # (each row's own)
    want = gb.linear_w4(x, q, s, zeros=z, group=group, x_scale=xs)
    check_linear_result(want, x, xs, q, s, z, None, None, "none", group)
    apart = torch.full((m, 3), float("nan"), device=DEV)
    apart[:, 1] = xs[:, 0]
    for scale in (xs[:, 0], xs.reshape(m).clone(), apart[:, 1]):
        assert scale.dim() == 1
        assert torch.equal(gb.linear_w4(x, q, s, zeros=z, group=group, x_scale=scale), want)
    one = gb.linear_w4(x[:1], q, s, zeros=z, group=group, x_scale=xs[0].expand(1))
    assert torch.equal(one, gb.linear_w4(x[:1], q, s, zeros=z, group=group, x_scale=xs[:1]))


def test_w4_refuses_a_scale_expanded_over_the_rows():
    """One element of storage for all rows: no row but the first has a scale in memory."""
    m, k = 4, 64
    q, s, z = w4_weights(8, k, 64, False, 1)
    x, xs = w4_input(m, k, "row", 2)
    for scale in (xs[0].expand(m), xs[:1].expand(m, 1)):
        with pytest.raises((ValueError, gb.GBError), match="x_scale|ldxs"):
            gb.linear_w4(x, q, s, group=64, x_scale=scale)
        with pytest.raises((ValueError, gb.GBError), match="x_scale|ldxs"):
            gb.ffn_gated_w4(x, q, s, q, s, group=64, x_scale=scale)


# ---------------------------------------------------------------------------------- memory on a stream that is given

def every_call():
    """Name and call of every operator, each of a stream and with everything made by the call."""
    x, w, r = normal(32, 512, seed=1), normal(96, 512, seed=2), normal(32, 96, seed=3)
    weight, rstd = normal(512, seed=4), torch.rand(32, device=DEV) + 0.5
    q, s, z = w4_weights(96, 512, 64, True, 5)
    return {
        "linear": lambda st: gb.linear(x, w, stream=st),
        "linear split": lambda st: gb.linear(x, w, split_k=4, stream=st),
        "linear_preact": lambda st: gb.linear_preact(x, w, act="silu", stream=st),
        "matmul": lambda st: gb.matmul(r, w, stream=st),
        "linear_dact": lambda st: gb.linear_dact(r, w, x, act="silu", stream=st),
        "ffn_gated": lambda st: gb.ffn_gated(x, w, w, stream=st),
        "ffn_gated split": lambda st: gb.ffn_gated(x, w, w, split_k=4, stream=st),
        "linear_w4": lambda st: gb.linear_w4(x, q, s, zeros=z, group=64, stream=st),
        "ffn_gated_w4": lambda st: gb.ffn_gated_w4(x, q, s, q, s, group=64, stream=st),
        "dropout": lambda st: gb.dropout(x, 0.1, 5, stream=st),
        "add_rms_norm": lambda st: gb.add_rms_norm(x, weight, x, p=0.1, seed=1, stream=st),
        "add_rms_norm_q8": lambda st: gb.add_rms_norm_q8(x, weight, x, stream=st),
        "add_rms_norm_backward": lambda st: gb.add_rms_norm_backward(x, x, weight, rstd, p=0.1, seed=1, stream=st),
    }


def tensors(result):
    return result if isinstance(result, tuple) else (result,)


@pytest.mark.parametrize("form", ["stream", "number"])
def test_what_a_call_makes_is_memory_of_its_stream(form):
    """The allocator's own record: nothing that a call on a side stream makes comes from another stream's memory."""
    calls, side = every_call(), torch.cuda.Stream()
    given = side if form == "stream" else side.cuda_stream
    torch.cuda.synchronize()
    for name, call in calls.items():
        want = [t.clone() for t in tensors(call(None))]
        torch.cuda.synchronize()
        torch.cuda.memory._record_memory_history(max_entries=1000)
        try:
            got = tensors(call(given))
            trace = torch.cuda.memory._snapshot()["device_traces"][torch.cuda.current_device()]
        finally:
            torch.cuda.memory._record_memory_history(enabled=None)
        made = [e["stream"] for e in trace if e["action"] == "alloc"]
        assert len(made) >= len({t.data_ptr() for t in got}) and set(made) == {side.cuda_stream}, (name, made)
        side.synchronize()
        if "split" in name:
            continue  # (split-K's order of additions is not fixed: two calls may differ by rounding)
        for a, b in zip(got, want):
            if a.dtype == torch.float8_e4m3fn:
                a, b = a.view(torch.uint8), b.view(torch.uint8)
            assert torch.equal(a, b), name


@pytest.mark.parametrize("number", [0, 1])
def test_default_stream_by_its_number(number):
    x = normal(8, 64, seed=1)
    want = gb.dropout(x, 0.3, 1)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = gb.dropout(x, 0.3, 1, stream=number)
    torch.cuda.synchronize()
    assert torch.equal(got, want)


def test_workspace_of_a_busy_side_stream_is_not_given_away():
    """The call returns long before its kernels run; what the current stream allocates and writes then is not theirs."""
    m, d = 900, 2100
    dy, h, w = normal(m, d, seed=1), normal(m, d, seed=2), normal(d, seed=3)
    rstd = (h.float().square().mean(dim=1) + 1e-6).rsqrt()
    want = [t.clone() for t in gb.add_rms_norm_backward(dy, h, w, rstd, p=0.1, seed=5)]
    need, side = gb.add_rms_norm_backward_workspace_bytes(m, d), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)
    got = gb.add_rms_norm_backward(dy, h, w, rstd, p=0.1, seed=5, stream=side)
    gb.add_rms_norm_backward(dy, h, w, rstd, p=0.1, seed=6, stream=side)  # (its outputs are dropped at once)
    others = [torch.full((need,), 255, dtype=torch.uint8, device=DEV) for _ in range(8)]
    others += [torch.full((m, d), float("nan"), dtype=BF16, device=DEV) for _ in range(8)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert all((t == 255).all() for t in others[:8]) and all(t.isnan().all() for t in others[8:])


# ---------------------------------------------------------------------------------- sizes of x and of the scales

@pytest.mark.parametrize("x8", ["no", "row", "group"])
@pytest.mark.parametrize("m,group", [(1, 128), (5, 64), (16, 32), (12, 128)])
@pytest.mark.parametrize("x_exp,s_exp", [(126, -20), (121, -2), (60, 58), (20, 98), (-30, 90), (-100, 90), (-115, 98)])
def test_w4_finite_results_of_large_factors(x_exp, s_exp, m, group, x8):
    """x near bf16's largest value, scales near 2^100: what the product of the two is, and nothing else.  Weights one
    step from the zero point at most, so that results are finite; rows and a group of weights at it, which add nothing."""
    n, k = 48, 800
    g = torch.Generator(device=DEV).manual_seed(7)
    q = torch.randint(7, 10, (n, k), generator=g, device=DEV, dtype=torch.int64)
    q[:4] = 8
    q[:, 128:256] = 8
    packed = (q[:, 0::2] | q[:, 1::2] << 4).to(torch.uint8)
    groups = -(-k // group)
    s = ((torch.rand((n, groups), generator=g, device=DEV) + 0.5) * 2.0 ** s_exp).to(BF16)
    v = torch.randn((m, k), generator=g, device=DEV).clamp(-1.9, 1.9)
    if x8 == "no":
        x, xs = (v.double() * 2.0 ** x_exp).to(BF16), None
    else:
        x = (v * 200).to(torch.float8_e4m3fn)
        xs = torch.full((m, 1 if x8 == "row" else -(-k // 128)), 2.0 ** x_exp / 200, dtype=torch.float64, device=DEV).float()
    d = gb.linear_w4(x, packed, s, group=group, x_scale=xs)
    assert d.isfinite().all() and not d[:, :4].any()
    check_linear_result(d, x, xs, packed, s, None, None, None, "none", group)
    zeros = torch.full((n, groups), 8, dtype=torch.uint8, device=DEV)
    assert torch.equal(gb.linear_w4(x, packed, s, zeros=zeros, group=group, x_scale=xs), d)


# ---------------------------------------------------------------------------------- the longest row

@pytest.mark.parametrize("offset,p,residual", [(0, 0.5, False), (1, 0.5, False), (1, 0.0, True), (7, 0.5, False)])
def test_dropout_of_the_longest_row(offset, p, residual):
    """As many columns as a row may have: those of its last chunk still are signed 32-bit numbers."""
    n, step = (1 << 31) - 16, 1 << 26
    pattern = (torch.arange(step, device=DEV) % 251 + 1).to(BF16)
    buf = pattern.repeat(n // step + 1)
    assert buf.numel() >= n + 1
    buf = torch.cat([buf[:8], buf])  # (room for the offset)
    x = buf[offset:offset + n].view(1, n)
    guard = torch.full((n + 24,), -3.0, dtype=BF16, device=DEV)
    out = guard[offset:offset + n].view(1, n)
    gb.dropout(x, p, 11, 5, R=x if residual else None, out=out)
    assert (guard[:offset] == -3).all() and (guard[offset + n:] == -3).all()
    for at in range(0, n, step):
        a, b = x[0, at:at + step], out[0, at:at + step]
        assert ((b == 2 * a) | ((b == 0) if p else (b == 2 * a))).all(), at
    if p:
        for first in (0, (n - 61) // 4 * 4):  # the mask itself at both ends, by its counters
            groups = torch.arange(first // 4, first // 4 + 16).numpy().astype("uint64")
            words = ref.philox([groups, groups * 0, groups * 0 + 5, groups * 0], (11, 0))
            keep = torch.stack([torch.from_numpy((w >= round(p * 2 ** 32))) for w in words], dim=1).reshape(-1)
            keep = keep[:min(64, n - first)].to(DEV)
            assert torch.equal(out[0, first:first + keep.numel()] != 0, keep)


# ---------------------------------------------------------------------------------- many tokens

@pytest.mark.parametrize("x8", ["no", "row", "group"])
@pytest.mark.parametrize("m", [(1 << 20) - 1, (1 << 20) + 35])
def test_w4_more_tokens_than_one_launch_has_passes_for(m, x8):
    n, k, group = 9, 160, 32
    q, s, z = w4_weights(n, k, group, True, 1)
    x, xs = w4_input(m, k, x8, 2)
    r = normal(m, n, seed=3)
    d = gb.linear_w4(x, q, s, R=r, zeros=z, group=group, x_scale=xs)
    check_linear_result(d, x, xs, q, s, z, None, r, "none", group)
    d = gb.ffn_gated_w4(x, q, s, q, s, zeros1=z, group=group, x_scale=xs)
    few = gb.ffn_gated_w4(x[-40:], q, s, q, s, zeros1=z, group=group, x_scale=None if xs is None else xs[-40:])
    a, off_a = ref.w4_products(x, xs, ref.unpack_w4(q, s, z, group, k))
    b, off_b = ref.w4_products(x, xs, ref.unpack_w4(q, s, None, group, k))
    gate = ref.act(a, "silu")
    tol = (1.13 * off_a + 2.0 ** -20 * a.abs()) * (b.abs() + off_b) + gate.abs() * off_b
    tol = tol * (1 + HALF_BF16) + HALF_BF16 * (gate * b).abs() + TINY
    assert_within(d, gate * b, tol)
    assert_within(few, (gate * b)[-40:], tol[-40:])


# ---------------------------------------------------------------------------------- zero points

@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("m", [1, 8, 12])
def test_w4_zero_points_are_the_low_four_bits(m, group):
    """In every variant (z off the sums, z off each weight, infinities added one by one): the same as without the rest."""
    n, k = 70, 416
    q, s, z = w4_weights(n, k, group, True, 1)
    high = torch.randint(0, 16, z.shape, generator=torch.Generator(device=DEV).manual_seed(2), device=DEV).to(torch.uint8) << 4
    x, r = normal(m, k, seed=3), normal(m, n, seed=4)
    for odd in (False, True):
        if odd:
            x[0, 7] = float("inf")
        want = gb.linear_w4(x, q, s, R=r, zeros=z, group=group)
        assert torch.equal(gb.linear_w4(x, q, s, R=r, zeros=z | high, group=group).nan_to_num(), want.nan_to_num())
        pair = gb.ffn_gated_w4(x, q, s, q, s, zeros1=z, zeros3=z, group=group)
        got = gb.ffn_gated_w4(x, q, s, q, s, zeros1=z | high, zeros3=z | high, group=group)
        assert torch.equal(got.nan_to_num(), pair.nan_to_num())
    check_linear_result(gb.linear_w4(x[1:], q, s, zeros=z | high, group=group) if m > 1 else want[1:], x[1:], None, q, s, z,
                        None, None, "none", group)


# ---------------------------------------------------------------------------------- the plan that is reported

def test_plan_of_a_call_without_work():
    """Not the plan of the call before it."""
    w = normal(64, seed=1)
    empty = torch.empty(0, 64, dtype=BF16, device=DEV)
    q, s, _ = w4_weights(8, 64, 64, False, 1)
    for call in (lambda: gb.dropout(empty, 0.1, 1), lambda: gb.add_rms_norm(empty, w), lambda: gb.add_rms_norm_q8(empty, w),
                 lambda: gb.linear_w4(empty, q, s, group=64), lambda: gb.ffn_gated_w4(empty, q, s, q, s, group=64)):
        gb.dropout(normal(3, 64, seed=2), 0.1, 1)
        assert "kernel=dropout" in gb.last_plan()
        call()
        assert gb.last_plan() == "empty (no launch)"
    gb.add_rms_norm_backward(empty, empty, w, torch.empty(0, device=DEV))  # (dweight is written)
    assert "kernel=add_rms_norm_backward blocks=0" in gb.last_plan()


# ---------------------------------------------------------------------------------- arguments

def test_norm_q8_refuses_a_scale_group_that_is_no_int():
    """Cut to 32 bits, these would be 0 and 128."""
    x, w = normal(4, 96, seed=1), normal(96, seed=2)
    for group in (1 << 32, (1 << 32) + 128, -(1 << 32), (1 << 63) - 1):
        with pytest.raises(gb.GBError, match="scale_group"):
            gb.add_rms_norm_q8(x, w, scale_group=group)


@pytest.mark.parametrize("m", [1, 5, 16])
def test_w4_one_row_of_weights_with_any_stride(m):
    """A row cut out of a wider buffer: its stride leads to no row, and may be no multiple of 16 bytes."""
    k, group = 96, 32
    q, s, z = w4_weights(2, k, group, True, 1)
    buf = torch.zeros(2, k // 2 + 5, dtype=torch.uint8, device=DEV)
    assert buf.data_ptr() % 16 == 0
    buf[:1, :k // 2] = q[:1]
    row = buf[:1, :k // 2]
    assert row.stride(0) % 16
    x = normal(m, k, seed=2)
    d = gb.linear_w4(x, row, s[:1], zeros=z[:1], group=group)
    check_linear_result(d, x, None, q[:1], s[:1], z[:1], None, None, "none", group)
    assert torch.equal(d, gb.linear_w4(x, q[:1], s[:1], zeros=z[:1], group=group))
    pair = gb.ffn_gated_w4(x, row, s[:1], row, s[:1], zeros1=z[:1], group=group)
    assert torch.equal(pair, gb.ffn_gated_w4(x, q[:1], s[:1], q[:1], s[:1], zeros1=z[:1], group=group))
    with pytest.raises(gb.GBError, match="16 bytes"):
        gb.linear_w4(x, buf[:, :k // 2], s, group=group)


@pytest.fixture
def another_device_is_current():
    """The binding, told that the current device is one that no tensor is on."""
    m = gb.block.binding()
    gb.block._bind(m, gb.lib(), lambda: 1)
    yield
    gb.block._bind(m, gb.lib())


def test_tensors_of_another_device_are_refused(another_device_is_current):
    """A kernel would run on the current device's stream, with addresses of another device's memory."""
    calls = every_call()
    for name in ("linear_w4", "ffn_gated_w4", "dropout", "add_rms_norm", "add_rms_norm_q8", "add_rms_norm_backward"):
        with pytest.raises(ValueError, match="on cuda:0, the current device is cuda:1"):
            calls[name](None)


# ---------------------------------------------------------------------------------- threads

def test_a_launch_that_waits_lets_other_threads_run():
    """More launches than the GPU's queue holds, behind a second of work: the thread that makes them waits without
    Python's lock."""
    import threading
    import time
    x = normal(4, 64, seed=1)
    out = torch.empty_like(x)
    gb.dropout(x, 0.1, 1, out=out)
    torch.cuda.synchronize()
    stream = torch.cuda.current_stream()
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    begin.record()
    torch.cuda._sleep(2_000_000_000)
    end.record()

    def launch():
        with torch.cuda.stream(stream):
            for _ in range(4000):
                gb.dropout(x, 0.1, 1, out=out)
    thread = threading.Thread(target=launch)
    longest, last, start = 0.0, time.perf_counter(), time.perf_counter()
    thread.start()
    while thread.is_alive():
        time.sleep(0.001)
        now = time.perf_counter()
        longest, last = max(longest, now - last), now
    took = last - start
    torch.cuda.synchronize()
    busy = begin.elapsed_time(end) / 1000
    assert busy > 0.5 and took > 0.5 * busy, (busy, took)  # (the thread did wait)
    assert longest < 0.25 * busy, (busy, took, longest)


# ---------------------------------------------------------------------------------- a seed in device memory

@pytest.mark.parametrize("m,d", [(5, 512), (40, 1027), (700, 1500), (60, 16384)])
def test_norm_backward_with_the_seed_in_device_memory(m, d):
    """The same bits as with the numbers, and what a replayed graph finds in the memory when it runs."""
    dy, h, w, dh = normal(m, d, seed=1), normal(m, d, seed=2), normal(d, seed=3), normal(m, d, seed=4)
    rstd = (h.float().square().mean(dim=1) + 1e-6).rsqrt()
    seed, p = (1 << 40) + 12345, 0.3
    want = [gb.add_rms_norm_backward(dy, h, w, rstd, dh, p=p, seed=seed, offset=o) for o in (0, 3, 1 << 33)]
    state = torch.tensor([seed, 0], dtype=torch.int64, device=DEV)
    ws = torch.empty(gb.add_rms_norm_backward_workspace_bytes(m, d), dtype=torch.uint8, device=DEV)
    got = gb.add_rms_norm_backward(dy, h, w, rstd, dh, p=p, seed=state, workspace=ws)
    assert all(torch.equal(a, b) for a, b in zip(got, want[0]))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = gb.add_rms_norm_backward(dy, h, w, rstd, dh, p=p, seed=state, workspace=ws)
    for offset, expected in zip((3, 1 << 33), want[1:]):
        state[1] = offset
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, expected))
    keep = ref.keep_mask(m, d, p, seed, 3).to(DEV)
    assert torch.equal(want[1][0] != 0, keep & (want[1][1] != 0))


# ---------------------------------------------------------------------------------- a step at the norm's limits, in a graph

@pytest.mark.parametrize("m,d", [(3, 1), (9, 64), (4, 16383), (300, 16384)])
def test_norm_forward_and_backward_in_one_graph(m, d):
    """The narrowest and the widest rows; every tensor made outside, as a captured step has them."""
    x, r, w, dy, dh = (normal(*shape, seed=i) for i, shape in enumerate(((m, d), (m, d), (d,), (m, d), (m, d))))

    def step():
        y, h, rstd = gb.add_rms_norm(x, w, r, p=0.1, seed=7, offset=1)
        return y, h, rstd, *gb.add_rms_norm_backward(dy, h, w, rstd, dh, p=0.1, seed=7, offset=1)
    want = [t.clone() for t in step()]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for _ in range(2):
        for t in got:
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    hw = ref.dropped(x, 0.1, 7, 1) + r.double()
    rw = (hw.square().mean(dim=1) + 1e-6).rsqrt()
    assert_within(want[2], rw, rw * 2.0 ** -17, "rstd")
    dr, dw = ref.norm_gradient(dy, want[1], w, dh, 1e-6, want[2])
    xhat, g = want[1].double() * want[2].double()[:, None], dy.double() * w.double()
    size = want[2].double()[:, None] * (g.abs() + xhat.abs() * (g * xhat).abs().mean(dim=1, keepdim=True))
    slack = 2.0 ** -17 * size + 2.0 ** -22 * dh.double().abs()
    assert_within(want[4], dr, HALF_BF16 * dr.abs() + slack * (1 + HALF_BF16) + TINY, "dR")
    assert_within(want[5], dw, (m / 8 + 72) * 2.0 ** -24 * (dy.double() * xhat).abs().sum(dim=0) + TINY, "dweight")
