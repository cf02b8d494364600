"""A feed-forward block with the library's operators: one training step, and serving one token at a time.

    x -> H = dropout(x) + R -> N = rms_norm(H) -> A = silu(N W1^T) * (N W3^T) -> H + dropout(A W2^T)

Training runs in bf16 (the products with tensor cores, the norm with its gradient, dropout whose mask is
drawn again instead of stored); serving runs the same block on 4-bit weights, the norm's output in 8 bits.

    python examples/ffn_block.py            # on a GB300
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import dense_bf16_gemm_persistent_gb300 as gb  # noqa: E402

EPS, P, GROUP = 1e-6, 0.1, 128


def quantize_w4(w: torch.Tensor, group: int = GROUP):
    """(packed, scales, zeros) of a bf16 weight [N,K], as linear_w4() takes them: each group of a row between
    its least and greatest value, in steps of a bf16 scale."""
    n, k = w.shape
    parts = torch.nn.functional.pad(w.float(), (0, -k % group)).view(n, -1, group)
    low, high = parts.amin(dim=2).clamp_max(0), parts.amax(dim=2).clamp_min(0)
    scales = ((high - low) / 15).clamp_min(1e-8).to(torch.bfloat16)
    zeros = (-low / scales.float()).round().clamp(0, 15)
    q = (parts / scales.float()[:, :, None] + zeros[:, :, None]).round().clamp(0, 15).to(torch.uint8)
    q = q.view(n, -1)[:, :k]
    return (q[:, 0::2] | q[:, 1::2] << 4).contiguous(), scales, zeros.to(torch.uint8)


def forward(x, r, weight, w1, w3, w2, seed):
    """The block's output and what its backward pass needs.  Each dropout has an offset of its own."""
    n, h, rstd = gb.add_rms_norm(x, weight, r, eps=EPS, p=P, seed=seed, offset=0)
    a1, z1 = gb.linear_preact(n, w1, act="silu")
    z3 = gb.linear(n, w3)
    a = (a1.float() * z3.float()).to(torch.bfloat16)
    out = gb.dropout(gb.linear(a, w2), P, seed, offset=1, R=h)
    return out, (n, h, rstd, a1, z1, z3, a)


def backward(dout, saved, weight, w1, w3, w2, seed):
    """Gradients of x, r, the norm's weight and the three matrices."""
    n, h, rstd, a1, z1, z3, a = saved
    dy = gb.dropout(dout, P, seed, offset=1)                         # the same mask, drawn again
    dw2 = gb.matmul(dy.t().contiguous(), a)
    da = gb.matmul(dy, w2)
    dz3 = (da.float() * a1.float()).to(torch.bfloat16)
    s = torch.sigmoid(z1.float())
    dz1 = (da.float() * z3.float() * s * (1 + z1.float() * (1 - s))).to(torch.bfloat16)
    dw1, dw3 = gb.matmul(dz1.t().contiguous(), n), gb.matmul(dz3.t().contiguous(), n)
    dn = gb.matmul(dz3, w3, R=gb.matmul(dz1, w1))
    dx, dr, dweight = gb.add_rms_norm_backward(dn, h, weight, rstd, dH=dout, p=P, seed=seed, offset=0)
    return dx, dr, dweight, dw1, dw3, dw2


def serve(x, r, weight, w1, w3, w2):
    """The block for a few tokens on 4-bit weights (each matrix a (packed, scales, zeros) of quantize_w4)."""
    q, scale, h = gb.add_rms_norm_q8(x, weight, r, eps=EPS)
    a = gb.ffn_gated_w4(q, w1[0], w1[1], w3[0], w3[1], zeros1=w1[2], zeros3=w3[2], group=GROUP, x_scale=scale)
    return gb.linear_w4(a, w2[0], w2[1], R=h, zeros=w2[2], group=GROUP)


def make(tokens: int, width: int, inner: int, seed: int = 0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, std=1.0):
        return (torch.randn(shape, generator=g, device="cuda") * std).to(torch.bfloat16)
    return {"x": normal(tokens, width), "r": normal(tokens, width), "weight": normal(width, std=0.1) + 1,
            "w1": normal(inner, width, std=width ** -0.5), "w3": normal(inner, width, std=width ** -0.5),
            "w2": normal(width, inner, std=inner ** -0.5)}


def main() -> None:
    t = make(tokens=4096, width=4096, inner=14336)
    matrices = t["w1"], t["w3"], t["w2"]
    out, saved = forward(t["x"], t["r"], t["weight"], *matrices, seed=7)
    grads = backward(torch.ones_like(out), saved, t["weight"], *matrices, seed=7)
    gb.device_status()
    print("training: output", tuple(out.shape), "gradients", [tuple(g.shape) for g in grads])

    packed = [quantize_w4(w) for w in matrices]
    x, r = t["x"][:1].contiguous(), t["r"][:1].contiguous()
    serve(x, r, t["weight"], *packed)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        token = serve(x, r, t["weight"], *packed)
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    for _ in range(3):
        graph.replay()
    begin.record()
    for _ in range(100):
        graph.replay()
    end.record()
    end.synchronize()
    print(f"serving: one token {tuple(token.shape)} in {begin.elapsed_time(end) * 10:.1f} us")


if __name__ == "__main__":
    main()
