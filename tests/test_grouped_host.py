"""Refusals of the grouped products and of the 4-bit calls: every bad argument is an error
code (or an exception of the binding) before any HIP call."""
import pytest

from adapter_gemv_amd import _lib, grouped, mx

# fake, aligned "device" addresses: never dereferenced, every call below is refused
X, Y, W, T, S = 1 << 40, 2 << 40, 3 << 40, 4 << 40, 5 << 40


def _call(name, base, kw):
    a = dict(base)
    a.update(kw)
    return getattr(_lib.lib(), name)(*a.values())


FWD = dict(stream=None, dtype=1, y=Y, ld_y=512, x=X, ld_x=256, share=1, W=W, W_stride=512 * 256,
           starts=T, perm=T + 4096, n=64, n_groups=4, h_in=256, h_out=512)
DX = dict(stream=None, dtype=1, y=Y, ld_y=256, dy=X, ld_x=512, W=W, W_stride=512 * 256, starts=T,
          perm=T + 4096, n=64, n_groups=4, h_in=256, h_out=512)
DW = dict(stream=None, dtype=1, dW=W, W_stride=512 * 256, x=X, ld_x=256, share=1, y=Y, ld_y=512,
          starts=T, perm=T + 4096, n=64, n_groups=4, h_in=256, h_out=512)
MX = dict(stream=None, dtype=1, y=Y, ld_y=512, x=X, ld_x=256, share=1, W=W, W_scales=S, starts=T,
          perm=T + 4096, n=64, n_groups=4, h_in=256, h_out=512)
MXQ = dict(stream=None, dtype=1, y=Y, ld_y=512, x=X, x_scales=S + (1 << 30), share=1, W=W,
           W_scales=S, starts=T, perm=T + 4096, n=64, n_groups=4, h_in=256, h_out=512)

COMMON = [
    ("dtype", dict(dtype=2), _lib.ERR_UNSUPPORTED),
    ("n<0", dict(n=-1), _lib.ERR_SHAPE),
    ("n", dict(n=(1 << 30) + 1), _lib.ERR_SHAPE),
    ("tiles", dict(n=1 << 30, h_in=1 << 22, h_out=1 << 22), _lib.ERR_SHAPE),
    ("no group", dict(n_groups=0), _lib.ERR_SHAPE),
    ("groups", dict(n_groups=1025), _lib.ERR_UNSUPPORTED),
    ("starts null", dict(starts=None), _lib.ERR_NULL),
    ("starts alone", dict(perm=None), _lib.ERR_NULL),
    ("perm alone", dict(starts=None, n_groups=1), _lib.ERR_NULL),
    ("x null", dict(x=None, dy=None), _lib.ERR_NULL),
    ("x misaligned", dict(x=X + 8, dy=X + 8), _lib.ERR_ALIGNMENT),
    ("y null", dict(y=None), _lib.ERR_NULL),
    ("y misaligned", dict(y=Y + 4), _lib.ERR_ALIGNMENT),
    ("h_in", dict(h_in=0), _lib.ERR_SHAPE),
    ("h_in % 8", dict(h_in=252), _lib.ERR_ALIGNMENT),
    ("h_out % 8", dict(h_out=508), _lib.ERR_ALIGNMENT),
    ("ld_y", dict(ld_y=248), _lib.ERR_SHAPE),
    ("ld_y % 8", dict(ld_y=1028), _lib.ERR_ALIGNMENT),
    ("alias", dict(y=X + 32, dW=X + 32), _lib.ERR_ALIAS),
    ("share", dict(share=0), _lib.ERR_SHAPE),
    ("share too large", dict(share=1 << 26), _lib.ERR_SHAPE),
]
CALLS = [("sgmv_group_matmul", FWD), ("sgmv_group_matmul_dx", DX), ("sgmv_group_matmul_dw", DW),
         ("sgmv_mx_matmul", MX), ("sgmv_mx_matmul_quantized", MXQ)]


@pytest.mark.parametrize("name,base", CALLS, ids=[c[0] for c in CALLS])
@pytest.mark.parametrize("what,kw,code", COMMON, ids=[c[0] for c in COMMON])
def test_common_refusals(name, base, what, kw, code):
    kw = {k: v for k, v in kw.items() if k in base}
    if not kw or (what == "alias" and name == "sgmv_group_matmul_dw" and "dW" not in kw):
        pytest.skip("no such argument")
    assert _call(name, base, kw) == code


@pytest.mark.parametrize("name,base,out", [("sgmv_group_matmul", FWD, "y"),
                                           ("sgmv_group_matmul_dx", DX, "y"),
                                           ("sgmv_group_matmul_dw", DW, "dW")])
def test_weight_refusals(name, base, out):
    assert _call(name, base, dict(W_stride=512 * 256 - 8)) == _lib.ERR_SHAPE
    assert _call(name, base, dict(W_stride=512 * 256 + 4)) == _lib.ERR_ALIGNMENT
    key = "W" if out == "y" else "dW"
    assert _call(name, base, {key: None}) == _lib.ERR_NULL
    assert _call(name, base, {key: W + 2}) == _lib.ERR_ALIGNMENT
    # an output inside the last group's weight (or rows inside the last group's gradient)
    assert _call(name, base, dict(y=W + 2 * (3 * 512 * 256 + 64))) == _lib.ERR_ALIAS


def test_mx_refusals():
    for name, base in (("sgmv_mx_matmul", MX), ("sgmv_mx_matmul_quantized", MXQ)):
        assert _call(name, base, dict(W=None)) == _lib.ERR_NULL
        assert _call(name, base, dict(W_scales=None)) == _lib.ERR_NULL
        assert _call(name, base, dict(W=W + 8)) == _lib.ERR_ALIGNMENT
        assert _call(name, base, dict(W_scales=S + 4)) == _lib.ERR_ALIGNMENT
        assert _call(name, base, dict(h_in=248)) == _lib.ERR_ALIGNMENT       # not whole blocks
        assert _call(name, base, dict(y=W)) == _lib.ERR_ALIAS
        assert _call(name, base, dict(y=S + 16)) == _lib.ERR_ALIAS
    assert _call("sgmv_mx_matmul_quantized", MXQ, dict(x_scales=None)) == _lib.ERR_NULL
    assert _call("sgmv_mx_matmul_quantized", MXQ, dict(x_scales=S + 4)) == _lib.ERR_ALIGNMENT
    Q = dict(stream=None, dtype=0, codes=Y, scales=S, x=X, ld=256, rows=16, h=256)
    D = dict(stream=None, dtype=0, x=X, ld=256, codes=Y, scales=S, rows=16, h=256)
    for name, base in (("sgmv_mx_quantize", Q), ("sgmv_mx_dequantize", D)):
        assert _call(name, base, dict(dtype=3)) == _lib.ERR_UNSUPPORTED
        assert _call(name, base, dict(h=0)) == _lib.ERR_SHAPE
        assert _call(name, base, dict(h=240)) == _lib.ERR_ALIGNMENT
        assert _call(name, base, dict(ld=248)) == _lib.ERR_SHAPE
        assert _call(name, base, dict(ld=260)) == _lib.ERR_ALIGNMENT
        assert _call(name, base, dict(rows=-1)) == _lib.ERR_SHAPE
        assert _call(name, base, dict(codes=None)) == _lib.ERR_NULL
        assert _call(name, base, dict(codes=Y + 8)) == _lib.ERR_ALIGNMENT
        assert _call(name, base, dict(scales=S + 1)) == _lib.ERR_ALIGNMENT
        assert _call(name, base, dict(codes=X + 512)) == _lib.ERR_ALIAS
        assert _call(name, base, dict(rows=0, codes=None, x=None)) == _lib.OK
    assert _call("sgmv_mx_quantize", Q, dict(scales=Y + 64)) == _lib.ERR_ALIAS


def test_group_rows_refusals():
    L = _lib.lib()
    assert L.sgmv_group_rows(None, T, -1, 4, Y, S) == _lib.ERR_SHAPE
    assert L.sgmv_group_rows(None, T, (1 << 30) + 1, 4, Y, S) == _lib.ERR_SHAPE
    assert L.sgmv_group_rows(None, T, 5, 0, Y, S) == _lib.ERR_SHAPE
    assert L.sgmv_group_rows(None, T, 5, 1025, Y, S) == _lib.ERR_UNSUPPORTED
    assert L.sgmv_group_rows(None, None, 5, 4, Y, S) == _lib.ERR_NULL
    assert L.sgmv_group_rows(None, T, 5, 4, None, S) == _lib.ERR_NULL
    assert L.sgmv_group_rows(None, T, 5, 4, Y, None) == _lib.ERR_NULL


def test_no_rows_is_ok_without_launch():
    for name, base in CALLS:
        if name != "sgmv_group_matmul_dw":
            assert _call(name, base, dict(n=0)) == _lib.OK


def test_binding_refusals():
    import torch
    bf, u8 = torch.bfloat16, torch.uint8
    x, y = torch.zeros(6, 64, dtype=bf), torch.zeros(12, 32, dtype=bf)
    Wt = torch.zeros(3, 32, 64, dtype=bf)
    i32 = torch.int32
    g = grouped.RowGroups(12, 3, torch.zeros(16, dtype=i32))
    for bad in (lambda: grouped.group_matmul(y[:11], x, Wt, g),                  # 11 rows share 6
                lambda: grouped.group_matmul(y, x, Wt[:2], g),                   # two groups' weights
                lambda: grouped.group_matmul(y, x[:, :56], Wt, g),               # h_in
                lambda: grouped.group_matmul(y[:, :24], x, Wt, g),               # h_out
                lambda: grouped.group_matmul(y, x, Wt.transpose(1, 2), g),       # not row-major
                lambda: grouped.group_matmul(y.t(), x, Wt, g),
                lambda: grouped.group_matmul_dx(x, y, Wt, g),                    # rows differ
                lambda: grouped.group_matmul_dw(Wt, x[:5], y, g),
                lambda: grouped.group_rows(torch.zeros(4, dtype=torch.int64), 3),
                lambda: mx.mx_quantize(torch.zeros(4, 48, dtype=bf)),
                lambda: mx.MxTensor(torch.zeros(4, 32, dtype=u8), torch.zeros(4, 4, dtype=u8)),
                lambda: mx.mx_dequantize(x, mx.MxTensor(torch.zeros(6, 64, dtype=u8),
                                                        torch.zeros(6, 8, dtype=u8))),
                lambda: grouped.group_matmul(y, x, Wt, g)):                      # not on a GPU
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: grouped.group_matmul(y, x.half(), Wt, g),
                lambda: grouped.group_matmul(y.float(), x.float(), Wt.float(), g),
                lambda: mx.mx_quantize(torch.zeros(4, 64)),
                lambda: mx.MxTensor(torch.zeros(4, 32), torch.zeros(4, 2, dtype=u8))):
        with pytest.raises(TypeError):
            bad()
