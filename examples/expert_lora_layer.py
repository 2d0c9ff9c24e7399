"""A LoRA-served expert layer, and a training step of its experts.

    python examples/expert_lora_layer.py

Serving: the layer's experts are held in 4 bits (one backbone copy), every token goes to its
router's two best experts, and every row gets its own adapter's low-rank update on top.
Training: forward and both gradients of the 16-bit experts.  Each result is compared with the
same arithmetic in float64 torch operations, and each step is timed.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import adapter_gemv_amd as sgmv  # noqa: E402


def route(x, router, top_k):
    """The router's top_k experts for each token and their weights: (ids [tokens * top_k], gates)."""
    top = torch.topk((x @ router).float(), top_k, dim=1)
    return top.indices.to(torch.int32).reshape(-1), torch.softmax(top.values, 1)


def serve(x, router, experts, adapters, A, B, scale, top_k=2):
    """y[t] = sum over t's experts e of gate * (x[t] W[e]^T + scale (x[t] A[a_t]) B[a_t])."""
    tokens, _ = x.shape
    _, h_out, _ = experts.shape
    ids, gates = route(x, router, top_k)
    groups = sgmv.group_rows(ids, experts.shape[0])
    rows = x.new_empty(tokens * top_k, h_out)
    sgmv.mx_matmul(rows, x, experts, groups)                     # top_k rows share one x
    sgmv.lora_add_pool(rows, x.repeat_interleave(top_k, 0), adapters.repeat_interleave(top_k), A, B, scale)
    return (rows.view(tokens, top_k, h_out) * gates[..., None]).sum(1).to(x.dtype), ids, gates


def train_step(x, ids, W, dy):
    """The experts' products and their gradients: (y, gradient of x, gradient of W)."""
    share = ids.shape[0] // x.shape[0]
    groups = sgmv.group_rows(ids, W.shape[0])
    y = sgmv.group_matmul(torch.empty_like(dy), x, W, groups)
    dx = sgmv.group_matmul_dx(x.new_empty(ids.shape[0], x.shape[1]), dy, W, groups)
    dW = sgmv.group_matmul_dw(torch.empty_like(W), x, dy, groups)
    return y, dx.view(x.shape[0], share, -1).float().sum(1).to(x.dtype), dW


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
    """Both uses once, checked; returns the relative errors (serving, dx, dW)."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(0)

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, generator=gen, device="cuda") * std).to(torch.bfloat16)

    W = normal(experts, h_out, h_in, std=h_in ** -0.5)
    router = normal(h_in, experts, std=h_in ** -0.5)
    A, B = normal(pool, rank, h_in, std=h_in ** -0.5), normal(pool, h_out, rank, std=rank ** -0.5)
    x = normal(tokens, h_in)
    adapters = torch.randint(0, pool, (tokens,), generator=gen, device="cuda", dtype=torch.int32)
    held = sgmv.mx_quantize(W)
    y, ids, gates = serve(x, router, held, adapters, A, B, 2.0)

    Wd = sgmv.mx_dequantize(torch.empty_like(W), held).double()
    ref = torch.zeros(tokens, h_out, dtype=torch.float64, device="cuda")
    for t in range(tokens):
        a = adapters[t]
        low = 2.0 * (B[a].double() @ (A[a].double() @ x[t].double()))
        for k in range(gates.shape[1]):
            ref[t] += gates[t, k].double() * (Wd[ids[t * gates.shape[1] + k]] @ x[t].double() + low)
    off = [float((y.double() - ref).norm() / ref.norm())]
    us = _timed(lambda: serve(x, router, held, adapters, A, B, 2.0))
    say(f"serving {tokens} tokens, 2 of {experts} experts in 4 bits, LoRA rank {rank}: "
        f"{us:.0f} us, relative error {off[0]:.2e}")

    x, dy = normal(train_tokens, h_in), normal(2 * train_tokens, h_out, std=h_out ** -0.5)
    ids, _ = route(x, router, 2)
    y, dx, dW = train_step(x, ids, W, dy)
    rx = torch.zeros(2 * train_tokens, h_in, dtype=torch.float64, device="cuda")
    for e in range(experts):
        mine = torch.nonzero(ids == e).flatten()
        rx[mine] = dy[mine].double() @ W[e].double()
    rx = rx.view(train_tokens, 2, -1).sum(1)
    mine = torch.nonzero(ids == 0).flatten()
    rw = dy[mine].double().t() @ x[mine // 2].double()
    off += [float((dx.double() - rx).norm() / rx.norm()), float((dW[0].double() - rw).norm() / rw.norm())]
    us = _timed(lambda: train_step(x, ids, W, dy))
    say(f"training step of {train_tokens} tokens: {us:.0f} us, relative error of dx {off[1]:.2e}, "
        f"of dW {off[2]:.2e}")
    return off


if __name__ == "__main__":
    main()
