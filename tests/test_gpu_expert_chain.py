"""An expert layer of routing, 8-bit products and the weighted sum, forwards and back, as a training
step and a serving loop run them: against the oracles of each, differences, and in HIP graphs."""
import numpy as np
import pytest

from oracle import block_oracle as B
from oracle import grouped_oracle as G
from oracle import routing_oracle as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch


def f64(t):
    return t.double().cpu().numpy()


CUT = 7 * 2.0 ** -13   # of the 8-bit products, as in their own tests


def close(got, ref, mag, depth, what, cut=0.0):
    tol = 2.0 ** -8 * np.abs(ref) + 2.0 ** -134 + (1 + 2.0 ** -8) * ((depth + 32) * 2.0 ** -23 + cut) * mag
    err = np.abs(got - ref)
    print(f"{what}: worst err/tol {(err / tol).max() if err.size else 0:.3f}", flush=True)
    assert np.all(err <= tol), f"{what}: {int((err > tol).sum())} of {err.size} outside"


class Layer:
    """x [T, h] -> route -> one 8-bit product by expert -> weighted sum."""

    def __init__(self, torch, T, k, E, h_in, h_out, seed=0):
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)
        self.torch, self.T, self.k, self.E = torch, T, k, E
        bf = torch.bfloat16
        self.logits = torch.randn(T, E, generator=gen, device="cuda")
        self.logits[T // 3] = float("-inf")                      # a padded token
        self.bias = torch.randn(E, generator=gen, device="cuda") * 0.05
        self.x = torch.randn(T, h_in, generator=gen, device="cuda").to(bf)
        self.W = (torch.randn(E, h_out, h_in, generator=gen, device="cuda") * h_in ** -0.5).to(bf)
        self.dout = torch.randn(T, h_out, generator=gen, device="cuda").to(bf)
        e = lambda *s: torch.empty(*s, dtype=bf, device="cuda")  # noqa: E731
        self.y, self.out = e(T * k, h_out), e(T, h_out)
        self.dy, self.dxs, self.dx = e(T * k, h_out), e(T * k, h_in), e(T, h_in)
        self.dW = torch.empty_like(self.W)
        self.dw, self.dlogits = torch.empty(T, k, device="cuda"), torch.empty_like(self.logits)

    def forward(self):
        import adapter_gemv_amd as sgmv
        self.routes = sgmv.route(self.logits, self.k, bias=self.bias, scores="sigmoid", expert_groups=2, keep_groups=1, scale=2.0)
        self.groups = sgmv.group_rows(self.routes.ids.view(-1), self.E)
        self.Wq = sgmv.fp8_quantize_weight(self.W)
        sgmv.fp8_matmul(self.y, self.x, self.Wq, self.groups)
        return sgmv.combine_rows(self.out, self.y, self.routes.weights)

    def backward(self):
        import adapter_gemv_amd as sgmv
        sgmv.combine_rows_backward(self.dy, self.dw, self.dout, self.y, self.routes.weights)
        sgmv.fp8_matmul_dx(self.dxs, self.dy, self.Wq, self.groups)
        sgmv.group_matmul_dw(self.dW, self.x, self.dy, self.groups)
        sgmv.combine_rows(self.dx, self.dxs)
        sgmv.route_backward(self.dlogits, self.dw, self.logits, self.routes)

    def results(self):
        return [self.out, self.dx, self.dW, self.dw, self.dlogits, self.routes.ids, self.routes.weights]


@pytest.mark.parametrize("size", [(1, 2, 8, 256, 400), (9, 2, 6, 272, 144), (150, 4, 8, 400, 272), (1100, 2, 4, 272, 528)],
                         ids=lambda s: "x".join(map(str, s)))
def test_each_step_of_a_training_step(torch, size):
    T, k, E, K, N = size
    L = Layer(torch, *size, seed=T)
    if T == 1:
        L.logits.copy_(torch.linspace(-1, 1, E, device="cuda"))
    L.forward()
    L.backward()
    ids, w = R.route(f64(L.logits), k, f64(L.bias), "sigmoid", 2, 1, 2, True, 2.0)
    assert np.array_equal(L.routes.ids.cpu().numpy(), ids)
    assert np.abs(f64(L.routes.weights) - w).max() < 2.0 * 100 * 2.0 ** -24
    if T > 1:
        assert (ids[T // 3] == -1).all() and not L.out[T // 3].any() and not L.dx[T // 3].any()
    flat = ids.reshape(-1)
    parts = [B.encode(v, 128) for v in f64(L.W)]
    Wd = np.stack([B.decode(*p, 128) for p in parts])
    close(f64(L.y), *G.group_matmul(B.decode(*B.encode(f64(L.x), 1), 1), Wd, flat, k), K, "y", CUT)
    close(f64(L.out), *R.combine(f64(L.y), f64(L.routes.weights), k), k, "out")
    dy, dw, mag = R.combine_backward(f64(L.dout), f64(L.y), f64(L.routes.weights), k)
    close(f64(L.dy), dy, np.abs(dy), 1, "dy")
    assert np.all(np.abs(f64(L.dw) - dw) <= 2.0 ** -24 * (N + 8) * mag + 2.0 ** -140)
    close(f64(L.dxs), *G.group_matmul_dx(B.decode(*B.encode(f64(L.dy), 1), 1), Wd, flat), N, "dx of each row", CUT)
    close(f64(L.dx), *R.combine(f64(L.dxs), None, k), k, "dx")
    close(f64(L.dW), *G.group_matmul_dw(f64(L.x), f64(L.dy), flat, E, k), T * k, "dW")
    dl, mag = R.route_backward(f64(L.logits), ids, f64(L.dw), "sigmoid", True, 2.0)
    assert np.all(np.abs(f64(L.dlogits) - dl) <= 2.0 ** -24 * np.abs(dl) + 300 * 2.0 ** -24 * mag + 2.0 ** -140)


@pytest.mark.parametrize("size", [(4, 2, 8, 256, 400), (500, 2, 4, 272, 528)], ids=lambda s: "x".join(map(str, s)))
def test_two_graphs_and_eager_calls(torch, size):
    """A forward and backward pass captured, replayed with new inputs, another graph and eager passes
    between: every replay is the eager pass bit for bit."""
    a, b, eager = (Layer(torch, *size, seed=s) for s in (1, 2, 3))
    graphs = []
    for L in (a, b):
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            L.forward()
            L.backward()
        torch.cuda.current_stream().wait_stream(side)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            L.forward()
            L.backward()
        graphs.append(g)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(7)
    for r in range(4):
        for L, g in zip((a, b), graphs):
            L.logits.copy_(torch.randn(L.logits.shape, generator=gen, device="cuda"))
            L.x.copy_(torch.randn(L.x.shape, generator=gen, device="cuda"))
            L.dout.copy_(torch.randn(L.dout.shape, generator=gen, device="cuda"))
            for name in ("logits", "bias", "x", "W", "dout"):
                getattr(eager, name).copy_(getattr(L, name))
            for t in L.results():
                t.fill_(3)
            eager.forward()
            eager.backward()
            want = [t.clone() for t in eager.results()]
            g.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(u, v) for u, v in zip(want, L.results())), f"replay {r}"


def test_steps_on_two_streams(torch):
    """Two layers at once, each on a stream of its own with workspaces of its own."""
    layers = [Layer(torch, 300, 2, 4, 400, 272, seed=s) for s in (1, 2)]
    want = []
    for L in layers:
        L.forward()
        L.backward()
        want.append([t.clone() for t in L.results()])
        for t in L.results():
            t.zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in layers]
    for _ in range(3):
        for L, s in zip(layers, streams):
            with torch.cuda.stream(s):
                L.forward()
        for L, s in zip(layers, streams):
            with torch.cuda.stream(s):
                L.backward()
    torch.cuda.synchronize()
    for L, w in zip(layers, want):
        assert all(torch.equal(u, v) for u, v in zip(w, L.results()))


def test_gradients_in_autograd(torch):
    """The calls wrapped as torch.autograd functions give the layer's gradients: the router's against differences of
    the layer's output (weights enter it linearly, so of the exact weights), the input's by its own linearity."""
    import adapter_gemv_amd as sgmv

    class Experts(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, logits, W, k):
            routes = sgmv.route(logits, k)
            groups = sgmv.group_rows(routes.ids.view(-1), W.shape[0])
            y = sgmv.fp8_matmul(x.new_empty(x.shape[0] * k, W.shape[1]), x, W, groups)
            ctx.parts = (x, logits, W, routes, groups, y)
            return sgmv.combine_rows(x.new_empty(x.shape[0], W.shape[1]), y, routes.weights)

        @staticmethod
        def backward(ctx, dout):
            x, logits, W, routes, groups, y = ctx.parts
            dw = torch.empty_like(routes.weights)
            dy, _ = sgmv.combine_rows_backward(torch.empty_like(y), dw, dout.contiguous(), y, routes.weights)
            dxs = sgmv.fp8_matmul_dx(x.new_empty(y.shape[0], x.shape[1]), dy, W, groups)
            dx = sgmv.combine_rows(torch.empty_like(x), dxs)
            return dx, sgmv.route_backward(torch.empty_like(logits), dw, logits, routes), None, None

    gen = torch.Generator(device="cuda")
    gen.manual_seed(3)
    T, E, K, N, k = 6, 4, 144, 272, 2
    x = torch.randn(T, K, generator=gen, device="cuda").bfloat16().requires_grad_()
    logits = torch.randn(T, E, generator=gen, device="cuda").requires_grad_()
    Wq = sgmv.fp8_quantize_weight((torch.randn(E, N, K, generator=gen, device="cuda") * K ** -0.5).bfloat16())
    g = torch.randn(T, N, generator=gen, device="cuda").bfloat16()
    out = Experts.apply(x, logits, Wq, k)
    out.backward(g)
    Wd = np.stack([B.decode(c, s, 128) for c, s in zip(Wq.codes.view(torch.uint8).cpu().numpy(), f64(Wq.scales))])
    X8, l, D = B.decode(*B.encode(f64(x.detach()), 1), 1), f64(logits.detach()), f64(g)
    ids, _ = R.route(l, k)

    def layer(logits64):
        total = 0.0
        for t in range(T):
            for j, w in enumerate(R.shares(list(logits64[t]), list(ids[t]), "softmax", True)):
                total += w * float(D[t] @ (Wd[ids[t][j]] @ X8[t]))
        return total

    large = np.array([max(np.abs(D[t]) @ (np.abs(W) @ np.abs(X8[t])) for W in Wd) for t in range(T)])
    size = np.abs(D) @ np.abs(np.concatenate([Wd.reshape(-1, K) @ X8.T]).reshape(E, N, T).max(0))
    step = 1e-5
    for t in range(T):
        for e in range(E):
            a, b = l.copy(), l.copy()
            a[t, e] += step
            b[t, e] -= step
            want = (layer(a) - layer(b)) / (2 * step)
            # y is rounded to bfloat16 (2^-8) and cut (CUT, of magnitudes) before its gradient is taken
            assert abs(float(logits.grad[t, e]) - want) <= 2 * (2.0 ** -8 * size[t, t] + CUT * large[t]) + 1e-6
    assert x.grad.shape == x.shape and bool(x.grad.isfinite().all())
