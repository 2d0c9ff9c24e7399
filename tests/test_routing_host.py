"""Refusals of routing, of the sums of expert rows and of the 8-bit products: every bad argument is
an error code (or an exception of the binding) before any HIP call."""
import pytest

from adapter_gemv_amd import _lib

# fake, aligned "device" addresses: never dereferenced, every call below is refused
A, B, C, D, E, F, G = (i << 40 for i in range(1, 8))
ROUTE = dict(stream=None, dtype=2, ids=A, weights=B, logits=C, ld=64, bias=D, n=100, E=64, k=4, groups=8, keep=2,
             best=2, scores=1, normalize=1, scale=1.0)
BACK = dict(stream=None, dtype=1, dlogits=A, ld_d=64, dweights=B, logits=C, ld=64, ids=D, n=100, E=64, k=4, scores=0,
            normalize=0, scale=1.0)
SUM = dict(stream=None, dtype=1, out=A, ld_out=256, y=B, ld_y=256, weights=C, n=100, k=4, h=256, add=0)
SUM_BACK = dict(stream=None, dtype=0, dy=A, ld_dy=256, dweights=B, dout=C, ld_dout=256, y=D, ld_y=256, weights=E,
                n=100, k=4, h=256)
QUANT = dict(stream=None, dtype=1, codes=A, scales=B, x=C, ld=256, rows=100, h=256)
DEQUANT = dict(stream=None, dtype=1, x=C, ld=256, codes=A, scales=B, rows=100, h=256)
WEIGHT = dict(stream=None, dtype=1, codes=A, scales=B, W=C, stride=256 * 512, G=4, h_in=256, h_out=512)
DEWEIGHT = dict(stream=None, dtype=1, W=C, stride=256 * 512, codes=A, scales=B, G=4, h_in=256, h_out=512)
TAIL = dict(w=D, ws=E, starts=F, perm=F + 4096, n=64, G=4, h_in=256, h_out=512)
SPACE = dict(workspace=G, bytes=1 << 20)
MUL = dict(stream=None, dtype=1, y=A, ld_y=512, x=B, ld_x=256, share=1, **TAIL, **SPACE)
MUL_Q = dict(stream=None, dtype=1, y=A, ld_y=512, x=B, xs=C, share=1, **TAIL)
DX = dict(stream=None, dtype=1, y=A, ld_y=256, x=B, ld_x=512, **TAIL, **SPACE)
DX_Q = dict(stream=None, dtype=1, y=A, ld_y=256, x=B, xs=C, **TAIL)
CALLS = {"sgmv_route": ROUTE, "sgmv_route_backward": BACK, "sgmv_combine_rows": SUM,
         "sgmv_combine_rows_backward": SUM_BACK, "sgmv_block_quantize": QUANT, "sgmv_block_dequantize": DEQUANT,
         "sgmv_block_quantize_weight": WEIGHT, "sgmv_block_dequantize_weight": DEWEIGHT, "sgmv_block_matmul": MUL,
         "sgmv_block_matmul_quantized": MUL_Q, "sgmv_block_matmul_dx": DX, "sgmv_block_matmul_dx_quantized": DX_Q}
U, S, N, L, O, V = (_lib.ERR_UNSUPPORTED, _lib.ERR_SHAPE, _lib.ERR_NULL, _lib.ERR_ALIGNMENT, _lib.ERR_ALIAS,
                    _lib.ERR_WORKSPACE)
ROUTES, SUMS = ("sgmv_route", "sgmv_route_backward"), ("sgmv_combine_rows", "sgmv_combine_rows_backward")
MULS = ("sgmv_block_matmul", "sgmv_block_matmul_quantized", "sgmv_block_matmul_dx", "sgmv_block_matmul_dx_quantized")
SIXTEEN = MULS[0::2]
WEIGHTS = ("sgmv_block_quantize_weight", "sgmv_block_dequantize_weight")
ROWS = ("sgmv_block_quantize", "sgmv_block_dequantize")
BAD = [
    (ROUTES, dict(dtype=3), U), (ROUTES, dict(dtype=-1), U), (ROUTES, dict(scores=2), U), (ROUTES, dict(n=-1), S),
    (ROUTES, dict(n=(1 << 25) + 1), S), (ROUTES, dict(E=0), S), (ROUTES, dict(k=0), S), (ROUTES, dict(k=65), S),
    (ROUTES, dict(E=1032, ld=2048, ld_d=2048), U), (ROUTES, dict(E=128, k=65, ld=128, ld_d=128), U),
    (ROUTES, dict(ld=63), S), (ROUTES, dict(ids=None), N), (ROUTES, dict(logits=None), N),
    (ROUTES, dict(logits=C + 1), L), (ROUTES, dict(ids=A + 2), L),
    (ROUTES[:1], dict(weights=None), N), (ROUTES[:1], dict(groups=7), S), (ROUTES[:1], dict(groups=0), S),
    (ROUTES[:1], dict(keep=0), S), (ROUTES[:1], dict(keep=9), S), (ROUTES[:1], dict(best=0), S),
    (ROUTES[:1], dict(best=3), U), (ROUTES[:1], dict(E=1024, ld=1024, groups=128), U),
    (ROUTES[:1], dict(logits=C + 2), L), (ROUTES[:1], dict(bias=D + 2), L), (ROUTES[:1], dict(weights=B + 1), L),
    (ROUTES[:1], dict(ids=B + 4 * 399), O), (ROUTES[:1], dict(weights=C + 4), O), (ROUTES[:1], dict(ids=C + 25596), O),
    (ROUTES[:1], dict(bias=A + 16), O), (ROUTES[:1], dict(bias=B - 4 * 63), O),
    (ROUTES[1:], dict(ld_d=63), S), (ROUTES[1:], dict(dlogits=None), N), (ROUTES[1:], dict(dweights=None), N),
    (ROUTES[1:], dict(dlogits=A + 1), L), (ROUTES[1:], dict(dweights=B + 2), L), (ROUTES[1:], dict(dlogits=C), O),
    (ROUTES[1:], dict(dweights=A + 12796), O), (ROUTES[1:], dict(ids=A - 1596), O),
    (SUMS, dict(dtype=2), U), (SUMS, dict(n=-1), S), (SUMS, dict(k=0), S), (SUMS, dict(n=1 << 28, k=8), S),
    (SUMS, dict(n=1 << 24, k=2), S), (SUMS, dict(h=0), S), (SUMS, dict(h=252), L), (SUMS, dict(ld_y=248), S),
    (SUMS, dict(ld_y=260), L), (SUMS, dict(weights=C + 2), L), (SUMS, dict(y=None), N), (SUMS, dict(y=B + 8), L),
    (SUMS[:1], dict(ld_out=248), S), (SUMS[:1], dict(out=None), N), (SUMS[:1], dict(out=A + 8), L),
    (SUMS[:1], dict(out=B), O), (SUMS[:1], dict(out=B + 512 * 400 - 16), O), (SUMS[:1], dict(weights=A), O),
    (SUMS[1:], dict(ld_dy=248), S), (SUMS[1:], dict(ld_dout=248), S), (SUMS[1:], dict(dy=None), N),
    (SUMS[1:], dict(dout=None), N), (SUMS[1:], dict(dweights=None), N), (SUMS[1:], dict(dy=A + 8), L),
    (SUMS[1:], dict(dout=C + 8), L), (SUMS[1:], dict(dweights=B + 2), L), (SUMS[1:], dict(dy=C), O),
    (SUMS[1:], dict(dy=D), O), (SUMS[1:], dict(weights=A), O), (SUMS[1:], dict(dweights=A), O),
    (SUMS[1:], dict(dweights=C), O), (SUMS[1:], dict(dweights=D), O), (SUMS[1:], dict(dweights=E), O),
    (ROWS, dict(dtype=2), U), (ROWS, dict(rows=-1), S), (ROWS, dict(rows=1 << 40), S), (ROWS, dict(h=0), S),
    (ROWS, dict(h=248), L), (ROWS, dict(h=1 << 23, ld=1 << 23), S), (ROWS, dict(ld=240), S), (ROWS, dict(ld=260), L),
    (ROWS, dict(codes=None), N), (ROWS, dict(scales=None), N), (ROWS, dict(x=None), N), (ROWS, dict(codes=A + 8), L),
    (ROWS, dict(scales=B + 2), L), (ROWS, dict(x=C + 8), L), (ROWS, dict(x=A), O), (ROWS, dict(x=B), O),
    (ROWS[:1], dict(scales=A + 25596), O),
    (WEIGHTS, dict(dtype=2), U), (WEIGHTS, dict(G=0), S), (WEIGHTS, dict(G=1025), U), (WEIGHTS, dict(h_in=248), L),
    (WEIGHTS, dict(h_out=0), S), (WEIGHTS, dict(stride=256 * 512 - 8), S), (WEIGHTS, dict(stride=256 * 512 + 4), L),
    (WEIGHTS, dict(h_in=1 << 22, h_out=1 << 22, stride=1 << 44), S), (WEIGHTS, dict(W=None), N),
    (WEIGHTS, dict(codes=None), N), (WEIGHTS, dict(scales=None), N), (WEIGHTS, dict(W=C + 8), L),
    (WEIGHTS, dict(codes=A + 8), L), (WEIGHTS, dict(scales=B + 1), L), (WEIGHTS, dict(W=A), O),
    (WEIGHTS, dict(scales=C), O), (WEIGHTS, dict(scales=A), O),
    (MULS, dict(dtype=2), U), (MULS, dict(n=-1), S), (MULS, dict(n=(1 << 30) + 1), S), (MULS, dict(G=0), S),
    (MULS, dict(G=1025), U), (MULS, dict(starts=None), N), (MULS, dict(perm=None), N), (MULS, dict(h_in=0), S),
    (MULS, dict(h_in=248), L), (MULS, dict(h_out=516, ld_x=516, ld_y=516), L),
    (MULS[3:], dict(h_out=520, ld_x=520), L), (WEIGHTS, dict(h_out=508), L), (MULS, dict(ld_y=248), S),
    (MULS, dict(ld_y=1028), L), (MULS, dict(y=None), N), (MULS, dict(x=None), N), (MULS, dict(w=None), N),
    (MULS, dict(ws=None), N), (MULS, dict(y=A + 8), L), (MULS, dict(x=B + 8), L), (MULS, dict(w=D + 8), L),
    (MULS, dict(ws=E + 2), L), (MULS, dict(y=B), O), (MULS, dict(y=D), O), (MULS, dict(y=D + 4 * 256 * 512 - 16), O),
    (MULS, dict(ws=A), O), (MULS, dict(starts=A), O), (MULS, dict(perm=A), O),
    (MULS, dict(n=1 << 30, h_in=1 << 22, h_out=1 << 22, ld_x=1 << 22, ld_y=1 << 22, bytes=1 << 60), S),
    (MULS[:2], dict(share=0), S), (MULS[:2], dict(share=1 << 26), S), (MULS[1::2], dict(xs=None), N),
    (MULS[1::2], dict(xs=C + 2), L), (MULS[1::2], dict(xs=A), O),
    (SIXTEEN, dict(ld_x=248), S), (SIXTEEN, dict(ld_x=516), L),
]
# the forms that take room: rows enough
ROOM = dict(n=4096, starts=None, perm=None, G=1, h_in=2048, h_out=2048, ld_x=2048, ld_y=2048, bytes=1 << 30)
BAD_ROOM = [(dict(workspace=None), V), (dict(workspace=G + 8), V), (dict(bytes=4096 * 2048 + 4096 * 64 - 1), V),
            (dict(workspace=A), O), (dict(workspace=B), O), (dict(workspace=D), O), (dict(workspace=E), O)]


@pytest.mark.parametrize("names,kw,code", BAD, ids=lambda v: str(v) if not isinstance(v, tuple) else v[0])
def test_refusals(names, kw, code):
    met = 0
    for name in names:
        args = {**CALLS[name], **{key: v for key, v in kw.items() if key in CALLS[name]}}
        if args != CALLS[name]:
            assert getattr(_lib.lib(), name)(*args.values()) == code, name
            met += 1
    assert met


@pytest.mark.parametrize("name", SIXTEEN)
@pytest.mark.parametrize("kw,code", BAD_ROOM, ids=lambda v: str(v))
def test_refusals_of_the_workspace(name, kw, code):
    assert getattr(_lib.lib(), name)(*{**CALLS[name], **ROOM, **kw}.values()) == code
    assert getattr(_lib.lib(), name)(*{**CALLS[name], **ROOM, **kw, "starts": F, "perm": G - 4, "G": 4,
                                       "workspace": kw.get("workspace", G)}.values()) in (V, O)


def test_nothing_to_do_is_fine():
    for name in (*ROUTES, *SUMS, *MULS):
        assert getattr(_lib.lib(), name)(*{**CALLS[name], "n": 0}.values()) == 0
    for name in ROWS:
        assert getattr(_lib.lib(), name)(*{**CALLS[name], "rows": 0}.values()) == 0


def test_without_weights():
    call = _lib.lib().sgmv_combine_rows_backward
    assert call(*{**SUM_BACK, "weights": None, "dweights": None, "y": None, "ld_y": 0, "dy": C}.values()) == O


def test_workspace_bytes():
    L = _lib.lib()
    assert L.sgmv_block_workspace_bytes(0, 1, 1, 0, 256, 256) == 0
    assert L.sgmv_block_dx_workspace_bytes(0, 256) == 0
    # codes, rounded up to 256, and a scale for each block that was begun
    assert L.sgmv_block_dx_workspace_bytes(100, 272) == (100 * 272 + 255) // 256 * 256 + 100 * 3 * 4
    assert L.sgmv_block_dx_workspace_bytes(100, 264) == (100 * 272 + 255) // 256 * 256 + 100 * 3 * 4
    assert L.sgmv_block_workspace_bytes(8192, 4, 1, 0, 2048, 2048) == 2048 * 2048 + 2048 * 16 * 4
    assert L.sgmv_block_dx_workspace_bytes(1 << 30, 1 << 22) == (1 << 52) + (1 << 30) * (1 << 15) * 4


def test_binding_refusals():
    import torch
    from adapter_gemv_amd import fp8, grouped, routing
    bf, f32, i32, f8 = torch.bfloat16, torch.float32, torch.int32, torch.float8_e4m3fn
    logits, bias = torch.zeros(6, 16), torch.zeros(16)
    R = routing.Routes(torch.zeros(6, 2, dtype=i32), torch.zeros(6, 2))
    y, out, w = torch.zeros(12, 64, dtype=bf), torch.zeros(6, 64, dtype=bf), torch.zeros(6, 2)
    q = fp8.Fp8Weight(torch.zeros(3, 32, 64, dtype=f8), torch.zeros(3, 1, 1))
    groups = grouped.RowGroups(12, 3, torch.zeros(16, dtype=i32))
    y32 = torch.zeros(12, 32, dtype=bf)
    value = [
        lambda: routing.route(logits[0], 2), lambda: routing.route(logits.t(), 2),
        lambda: routing.route(torch.zeros(6, 0), 2), lambda: routing.route(logits, 2, scores="relu"),
        lambda: routing.route(logits, 2, bias=bias[:15]), lambda: routing.route(logits, 2, bias=bias.double()),
        lambda: routing.route(logits, 2),                                              # not on a GPU
        lambda: routing.route_backward(logits[:5], w, logits, R), lambda: routing.route_backward(logits, w[:, :1], logits, R),
        lambda: routing.route_backward(logits, w.double(), logits, R),
        lambda: routing.route_backward(logits, w, logits, routing.Routes(R.ids.long(), w)),
        lambda: routing.route_backward(logits, w, logits, routing.Routes(R.ids[0], w)),
        lambda: routing.route_backward(logits, w, logits, routing.Routes(R.ids, w, scores="x")),
        lambda: routing.combine_rows(out, y[:11], w), lambda: routing.combine_rows(out, y, w[:5]),
        lambda: routing.combine_rows(out, y, w.half()), lambda: routing.combine_rows(out, y, w[:, 0]),
        lambda: routing.combine_rows(out, y[:, :32], w), lambda: routing.combine_rows(out[:, ::2], y, w),
        lambda: routing.combine_rows(out, y[:5]), lambda: routing.combine_rows(out, y, w),
        lambda: routing.combine_rows_backward(y, w, out), lambda: routing.combine_rows_backward(y, None, out, y, w.double()),
        lambda: routing.combine_rows_backward(y, w, out, y[:11], w), lambda: routing.combine_rows_backward(y, w[:5], out, y, w),
        lambda: routing.combine_rows_backward(y, w, out, y[:, :32], w),
        lambda: fp8.Fp8Rows(torch.zeros(3, 144, dtype=f8), torch.zeros(3, 1)),
        lambda: fp8.Fp8Rows(torch.zeros(144, 3, dtype=f8).t(), torch.zeros(3, 2)),
        lambda: fp8.Fp8Weight(torch.zeros(144, dtype=f8), torch.zeros(2)),
        lambda: fp8.Fp8Weight(torch.zeros(144, 64, dtype=f8), torch.zeros(1, 1)),
        lambda: fp8.Fp8Weight(torch.zeros(144, 64, dtype=f8), torch.zeros(2, 2)[:, :1]),
        lambda: fp8.fp8_quantize(torch.zeros(4, 0, dtype=bf)), lambda: fp8.fp8_quantize(y[:, ::2]),
        lambda: fp8.fp8_quantize(y), lambda: fp8.fp8_quantize_weight(y[0]), lambda: fp8.fp8_quantize_weight(y.t()),
        lambda: fp8.fp8_dequantize(y, q), lambda: fp8.fp8_matmul(y32, y, q), lambda: fp8.fp8_matmul(y, y, q, groups),
        lambda: fp8.fp8_matmul(y32, y32, q, groups), lambda: fp8.fp8_matmul(y32, y[:5], q, groups),
        lambda: fp8.fp8_matmul(y32, y, q, grouped.RowGroups(12, 3, torch.zeros(15, dtype=i32))),
        lambda: fp8.fp8_matmul_dx(y, y32[:6], q, groups), lambda: fp8.fp8_matmul_dx(y32, y, q, groups),
        lambda: fp8.fp8_matmul(y32, y, q, groups),
    ]
    for i, call in enumerate(value):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i} went through")
    kind = [
        lambda: routing.route(logits.double(), 2), lambda: routing.route(logits.int(), 2),
        lambda: routing.route_backward(logits.half(), w, logits, R), lambda: routing.combine_rows(out.half(), y, w),
        lambda: routing.combine_rows(out.float(), y.float(), w),
        lambda: routing.combine_rows_backward(y, w, out, y.half(), w),
        lambda: fp8.Fp8Rows(torch.zeros(3, 144, dtype=torch.uint8), torch.zeros(3, 2)),
        lambda: fp8.Fp8Rows(torch.zeros(3, 144, dtype=f8), torch.zeros(3, 2, dtype=torch.float16)),
        lambda: fp8.fp8_quantize(logits), lambda: fp8.fp8_quantize_weight(logits), lambda: fp8.fp8_matmul(y32.half(), y, q, groups),
    ]
    for i, call in enumerate(kind):
        with pytest.raises(TypeError):
            call()
            pytest.fail(f"call {i} went through")
    with pytest.raises(_lib.SgmvError):
        routing.route(logits, 17)
    with pytest.raises(_lib.SgmvError):
        routing.route(logits, 1 << 40)
