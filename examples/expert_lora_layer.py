"""A LoRA-served expert layer, and a training step of its experts.

    python examples/expert_lora_layer.py

Serving: the layer's experts are held in 4 or in 8 bits (one backbone copy), every token goes to its
router's two best experts, and every row gets its own adapter's low-rank update on top.
Training: forward and both gradients of the 16-bit experts, and a whole layer whose products are in
8 bits, with the gradients of the router's logits and of the rows.  Each result is compared with the same
arithmetic in float64 torch operations, and each step is timed.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import adapter_gemv_amd as sgmv  # noqa: E402


def route(x, router, top_k):
    """The router's top_k experts for each token and their weights."""
    return sgmv.route((x @ router).float(), top_k)


def serve(x, router, experts, adapters, A, B, scale, top_k=2):
    """y[t] = sum over t's experts e of gate * (x[t] W[e]^T + scale (x[t] A[a_t]) B[a_t]); the experts
    an MxTensor or an Fp8Weight."""
    tokens, _ = x.shape
    _, h_out, _ = experts.shape
    routes = route(x, router, top_k)
    groups = sgmv.group_rows(routes.ids.view(-1), experts.shape[0])
    rows = x.new_empty(tokens * top_k, h_out)
    product = sgmv.fp8_matmul if isinstance(experts, sgmv.Fp8Weight) else sgmv.mx_matmul
    product(rows, x, experts, groups)                            # top_k rows share one x
    sgmv.lora_add_pool(rows, x.repeat_interleave(top_k, 0), adapters.repeat_interleave(top_k), A, B, scale)
    return sgmv.combine_rows(x.new_empty(tokens, h_out), rows, routes.weights), routes


def train_step(x, ids, W, dy):
    """The experts' products and their gradients: (y, gradient of x, gradient of W)."""
    groups = sgmv.group_rows(ids, W.shape[0])
    y = sgmv.group_matmul(torch.empty_like(dy), x, W, groups)
    dxs = sgmv.group_matmul_dx(x.new_empty(ids.shape[0], x.shape[1]), dy, W, groups)
    dW = sgmv.group_matmul_dw(torch.empty_like(W), x, dy, groups)
    return y, sgmv.combine_rows(torch.empty_like(x), dxs), dW


def train_layer(x, logits, W, dout, top_k=2):
    """A layer's forward and backward pass with 8-bit products: (out, gradients of x, of the logits and
    of W)."""
    tokens, E = logits.shape
    routes = sgmv.route(logits, top_k)
    groups = sgmv.group_rows(routes.ids.view(-1), E)
    held = sgmv.fp8_quantize_weight(W)
    rows = sgmv.fp8_matmul(x.new_empty(tokens * top_k, W.shape[1]), x, held, groups)
    out = sgmv.combine_rows(torch.empty_like(dout), rows, routes.weights)
    dweights = torch.empty_like(routes.weights)
    drows, _ = sgmv.combine_rows_backward(torch.empty_like(rows), dweights, dout, rows, routes.weights)
    dxs = sgmv.fp8_matmul_dx(x.new_empty(tokens * top_k, x.shape[1]), drows, held, groups)
    dW = sgmv.group_matmul_dw(torch.empty_like(W), x, drows, groups)
    dlogits = sgmv.route_backward(torch.empty_like(logits), dweights, logits, routes)
    return out, sgmv.combine_rows(torch.empty_like(x), dxs), dlogits, dW


def _timed(f, n=20):
    f()
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record()
    for _ in range(n):
        f()
    b.record()
    torch.cuda.synchronize()
    return a.elapsed_time(b) / n * 1e3


def main(tokens=32, experts=8, pool=16, h_in=4096, h_out=4096, rank=16, train_tokens=2048, say=print):
    """Each use once, checked; returns the relative errors (serving in 4 and 8 bits, dx, dW, and of the 8-bit
    layer the output and the gradient of the logits)."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(0)

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, generator=gen, device="cuda") * std).to(torch.bfloat16)

    def error(got, ref):
        return float((got.double() - ref).norm() / ref.norm())

    W = normal(experts, h_out, h_in, std=h_in ** -0.5)
    router = normal(h_in, experts, std=h_in ** -0.5)
    A, B = normal(pool, rank, h_in, std=h_in ** -0.5), normal(pool, h_out, rank, std=rank ** -0.5)
    x = normal(tokens, h_in)
    adapters = torch.randint(0, pool, (tokens,), generator=gen, device="cuda", dtype=torch.int32)
    off = []
    for bits, held in ((4, sgmv.mx_quantize(W)), (8, sgmv.fp8_quantize_weight(W))):
        y, routes = serve(x, router, held, adapters, A, B, 2.0)
        values, rows = torch.empty_like(W), x
        if bits == 4:
            sgmv.mx_dequantize(values, held)
        else:
            sgmv.fp8_dequantize(values, held)
            rows = sgmv.fp8_dequantize(torch.empty_like(x), sgmv.fp8_quantize(x))
        ref = torch.zeros(tokens, h_out, dtype=torch.float64, device="cuda")
        for t in range(tokens):
            a = adapters[t]
            low = 2.0 * (B[a].double() @ (A[a].double() @ x[t].double()))
            for e, gate in zip(routes.ids[t], routes.weights[t]):
                ref[t] += gate.double() * (values[e].double() @ rows[t].double() + low)
        off.append(error(y, ref))
        us = _timed(lambda: serve(x, router, held, adapters, A, B, 2.0))
        say(f"serving {tokens} tokens, 2 of {experts} experts in {bits} bits, LoRA rank {rank}: "
            f"{us:.0f} us, relative error {off[-1]:.2e}")

    x, dy = normal(train_tokens, h_in), normal(2 * train_tokens, h_out, std=h_out ** -0.5)
    ids = route(x, router, 2).ids.view(-1)
    y, dx, dW = train_step(x, ids, W, dy)
    rx = torch.zeros(2 * train_tokens, h_in, dtype=torch.float64, device="cuda")
    for e in range(experts):
        mine = torch.nonzero(ids == e).flatten()
        rx[mine] = dy[mine].double() @ W[e].double()
    rx = rx.view(train_tokens, 2, -1).sum(1)
    mine = torch.nonzero(ids == 0).flatten()
    rw = dy[mine].double().t() @ x[mine // 2].double()
    off += [error(dx, rx), error(dW[0], rw)]
    us = _timed(lambda: train_step(x, ids, W, dy))
    say(f"training step of {train_tokens} tokens: {us:.0f} us, relative error of dx {off[-2]:.2e}, "
        f"of dW {off[-1]:.2e}")

    logits, dout = (x @ router).float(), dy[::2]
    out, dx, dlogits, _ = train_layer(x, logits, W, dout)
    values = sgmv.fp8_dequantize(torch.empty_like(W), sgmv.fp8_quantize_weight(W))
    rows = sgmv.fp8_dequantize(torch.empty_like(x), sgmv.fp8_quantize(x)).double().requires_grad_()
    l = logits.double().requires_grad_()
    top, at = l.topk(2, 1)
    ref = torch.zeros(train_tokens, h_out, dtype=torch.float64, device="cuda")
    for j, gate in enumerate(top.softmax(1).t()):
        for e in range(experts):
            mine = torch.nonzero(at[:, j] == e).flatten()
            ref = ref.index_add(0, mine, gate[mine, None] * (rows[mine] @ values[e].double().t()))
    ref.backward(dout.double())
    off += [error(out, ref.detach()), error(dlogits, l.grad)]
    us = _timed(lambda: train_layer(x, logits, W, dout))
    # dy is taken to 8 bits on its way to dx: half a step of 2^-3 is 2^-4 of a value at most
    say(f"8-bit layer's training step of {train_tokens} tokens: {us:.0f} us, relative error of the output "
        f"{off[-2]:.2e}, of the logits' gradient {off[-1]:.2e}, of dx {error(dx, rows.grad):.2e} (dy in 8 bits)")
    return off


if __name__ == "__main__":
    main()
