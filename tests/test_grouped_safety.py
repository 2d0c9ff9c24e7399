"""Calls of the grouped and 4-bit products that would read or write out of range, or compute
something else than was asked, are refused before any HIP call."""
import pytest

from adapter_gemv_amd import _lib

# fake device addresses: never dereferenced, every call below is refused
IDS, PERM, STARTS = 1 << 40, 2 << 40, 3 << 40


@pytest.mark.parametrize("n", [1, 64, 8192, 1 << 30])
def test_group_rows_outputs_stand_alone(n):
    """Workgroups read ids while others write the tables."""
    rows = _lib.lib().sgmv_group_rows
    for perm, starts in ((IDS, STARTS), (IDS + 4 * n - 4, STARTS), (IDS - 4 * n + 4, STARTS),
                         (PERM, IDS), (PERM, IDS + 4 * n - 4), (PERM, IDS - 4 * 7), (PERM, PERM),
                         (PERM, PERM + 4 * n - 4), (PERM, PERM - 4 * 7)):
        assert rows(None, IDS, n, 7, perm, starts) == _lib.ERR_ALIAS


X, Y, W, SX, SW = 4 << 40, 5 << 40, 6 << 40, 7 << 40, 8 << 40
N, G, H_IN, H_OUT = 64, 4, 256, 512
TAIL = dict(starts=STARTS, perm=PERM, n=N, n_groups=G, h_in=H_IN, h_out=H_OUT)
# name, arguments, the output's name and bytes
PRODUCTS = [
    ("sgmv_group_matmul", dict(stream=None, dtype=1, y=Y, ld_y=H_OUT, x=X, ld_x=H_IN, share=1, W=W,
                               W_stride=H_IN * H_OUT, **TAIL), "y", 2 * N * H_OUT),
    ("sgmv_group_matmul_dx", dict(stream=None, dtype=1, dx=Y, ld_dx=H_IN, dy=X, ld_dy=H_OUT, W=W,
                                  W_stride=H_IN * H_OUT, **TAIL), "dx", 2 * N * H_IN),
    ("sgmv_group_matmul_dw", dict(stream=None, dtype=1, dW=W, dW_stride=H_IN * H_OUT, x=X, ld_x=H_IN,
                                  share=1, dy=Y, ld_dy=H_OUT, **TAIL), "dW", 2 * G * H_IN * H_OUT),
    ("sgmv_mx_matmul", dict(stream=None, dtype=1, y=Y, ld_y=H_OUT, x=X, ld_x=H_IN, share=1, W=W,
                            W_scales=SW, **TAIL), "y", 2 * N * H_OUT),
    ("sgmv_mx_matmul_quantized", dict(stream=None, dtype=1, y=Y, ld_y=H_OUT, x=X, x_scales=SX, share=1,
                                      W=W, W_scales=SW, **TAIL), "y", 2 * N * H_OUT),
]


@pytest.mark.parametrize("name,args,out,size", PRODUCTS, ids=[p[0] for p in PRODUCTS])
def test_products_do_not_write_over_their_tables(name, args, out, size):
    """Rows are looked up in the tables until the last of them is written."""
    call = getattr(_lib.lib(), name)
    at = args[out]
    for kw in (dict(perm=at), dict(perm=at + size - 4), dict(perm=at - 4 * N + 4),
               dict(starts=at + 64), dict(starts=at + size - 4), dict(starts=at - 4 * G)):
        assert call(*{**args, **kw}.values()) == _lib.ERR_ALIAS, kw


def test_products_do_not_read_past_a_table():
    """RowGroups is public: a table that is too short, of other integers or with gaps."""
    import torch
    from adapter_gemv_amd import grouped, mx
    i32, bf, u8 = torch.int32, torch.bfloat16, torch.uint8
    x, y, w = torch.zeros(12, 64, dtype=bf), torch.zeros(12, 32, dtype=bf), torch.zeros(3, 32, 64, dtype=bf)
    q = mx.MxTensor(torch.zeros(3, 32, 32, dtype=u8), torch.zeros(3, 32, 2, dtype=u8))
    for table in (torch.zeros(15, dtype=i32), torch.zeros(17, dtype=i32), torch.zeros(16, dtype=torch.int64),
                  torch.zeros(16), torch.zeros(32, dtype=i32)[::2], torch.zeros(16, 1, dtype=i32),
                  torch.zeros(0, dtype=i32)):
        g = grouped.RowGroups(12, 3, table)
        for call in (lambda: grouped.group_matmul(y, x, w, g), lambda: grouped.group_matmul_dx(x, y, w, g),
                     lambda: grouped.group_matmul_dw(w, x, y, g), lambda: mx.mx_matmul(y, x, q, g)):
            with pytest.raises(ValueError, match="groups"):
                call()


def recorded(monkeypatch):
    """The bindings with their C calls written down instead of made (tensors may be of any device)."""
    from adapter_gemv_amd import grouped, mx
    calls = []

    class Recorder:
        def __getattr__(self, name):
            return lambda *args: calls.append((name, args)) or 0

    recorder = Recorder()
    monkeypatch.setattr(_lib, "lib", lambda: recorder)
    monkeypatch.setattr(_lib, "status_string", lambda status: str(status))
    for module in (grouped, mx):
        monkeypatch.setattr(module, "_stream_of", lambda stream, *tensors: 0)
    return grouped, mx, calls


def test_sizes_past_32_bits_are_refused(monkeypatch):
    """Sizes travel as 32-bit integers: 2^32 + 16 rows are not 16."""
    import torch
    grouped, mx, calls = recorded(monkeypatch)
    bf, u8, far = torch.bfloat16, torch.uint8, (1 << 32) + 32

    def empty(*shape, dtype=bf):
        return torch.empty(*shape, dtype=dtype, device="meta")

    x, w, q = empty(far, 32), empty(32, 32), mx.MxTensor(empty(32, 16, dtype=u8), empty(32, 1, dtype=u8))
    wide, tall = empty(32, far), empty(far, 32)
    ids = torch.empty(4, dtype=torch.int32)
    for call in (lambda: grouped.group_matmul(x, x, w), lambda: grouped.group_matmul_dx(x, x, w),
                 lambda: grouped.group_matmul_dw(w, x, x),
                 lambda: grouped.group_matmul(empty(4, 32), empty(4, far), wide),
                 lambda: grouped.group_matmul(empty(4, far), empty(4, 32), tall),
                 lambda: grouped.group_matmul_dx(empty(4, far), empty(4, 32), wide),
                 lambda: grouped.group_matmul_dw(tall, empty(4, 32), empty(4, far)),
                 lambda: grouped.group_rows(empty(far, dtype=torch.int32), 3),
                 lambda: grouped.group_rows(ids, (1 << 32) + 3), lambda: grouped.group_rows(ids, 1 << 32),
                 lambda: mx.mx_matmul(x, x, q), lambda: mx.mx_matmul(x, mx.MxTensor(
                     empty(far, 16, dtype=u8), empty(far, 1, dtype=u8)), q),
                 lambda: mx.mx_matmul(empty(4, 32), empty(4, far), mx.MxTensor(
                     empty(32, far // 2, dtype=u8), empty(32, far // 32, dtype=u8))),
                 lambda: mx.mx_matmul(empty(4, far), empty(4, 32), mx.MxTensor(
                     empty(far, 16, dtype=u8), empty(far, 1, dtype=u8))),
                 lambda: mx.mx_quantize(empty(far)), lambda: mx.mx_quantize(wide),
                 lambda: mx.mx_dequantize(empty(far), mx.MxTensor(empty(far // 2, dtype=u8),
                                                                  empty(far // 32, dtype=u8)))):
        with pytest.raises(_lib.SgmvError):
            call()
    assert not calls
    # as many rows of a matrix as there are: 64-bit
    mx.mx_quantize(tall)
    assert calls[0][1][-2:] == (far, 32)


@pytest.mark.parametrize("n_groups,status", [(-7, _lib.ERR_SHAPE), (0, _lib.ERR_SHAPE),
                                             (1025, _lib.ERR_UNSUPPORTED), (1 << 40, _lib.ERR_UNSUPPORTED)])
def test_group_rows_refuses_before_it_allocates(monkeypatch, n_groups, status):
    import torch
    grouped, _, calls = recorded(monkeypatch)
    with pytest.raises(_lib.SgmvError) as refused:
        grouped.group_rows(torch.empty(4, dtype=torch.int32), n_groups)
    assert refused.value.status == status and not calls


def test_one_row_of_any_stride(monkeypatch):
    """The distance to a next row means nothing where there is one row: tensors whose stride there
    is 1, or no multiple of 8, are taken as mx_quantize takes them."""
    import torch
    grouped, mx, calls = recorded(monkeypatch)
    bf = torch.bfloat16
    w = torch.zeros(64, 32, dtype=bf)
    q = mx.MxTensor(torch.zeros(64, 16, dtype=torch.uint8), torch.zeros(64, 1, dtype=torch.uint8))

    def rows(h):
        return torch.zeros(h, 1, dtype=bf).t(), torch.zeros(5, h + 3, dtype=bf)[:1, :h], torch.zeros(0, h, dtype=bf)

    for x, y in zip(rows(32), rows(64)):
        grouped.group_matmul(y, x, w)
        grouped.group_matmul_dx(x, y, w)
        grouped.group_matmul_dw(w, x, y)
        mx.mx_matmul(y, x, q)
        mx.mx_matmul(y, mx.mx_quantize(x), q)
    strides = dict(sgmv_group_matmul=((3, 64), (5, 32)), sgmv_group_matmul_dx=((3, 32), (5, 64)),
                   sgmv_group_matmul_dw=((5, 32), (8, 64)), sgmv_mx_matmul=((3, 64), (5, 32)),
                   sgmv_mx_matmul_quantized=((3, 64),), sgmv_mx_quantize=((5, 32),))
    assert len(calls) == 3 * 6
    for name, args in calls:
        assert all(args[at] == ld for at, ld in strides[name]), (name, args)


def test_launches_past_the_threads_of_a_grid_are_refused():
    """A grid has fewer than 2^32 threads; products of more, which only many groups of very wide
    weights reach, are refused with the code that the header names, not by the launch."""
    wide = dict(n=1024, n_groups=1024)
    for name, args, _, _ in PRODUCTS:
        call = getattr(_lib.lib(), name)
        if name == "sgmv_group_matmul":
            kw = dict(ld_y=1 << 22, ld_x=8, W_stride=1 << 25, h_in=8, h_out=1 << 22)
        elif name == "sgmv_group_matmul_dx":
            kw = dict(ld_dx=1 << 22, ld_dy=8, W_stride=1 << 25, h_in=1 << 22, h_out=8)
        elif name == "sgmv_group_matmul_dw":
            kw = dict(dW_stride=1 << 40, ld_x=1 << 19, ld_dy=1 << 21, h_in=1 << 19, h_out=1 << 21,
                      x=X << 12, dy=Y << 12, starts=STARTS << 12, perm=PERM << 12)
        else:
            kw = dict(ld_y=1 << 22, h_in=32, h_out=1 << 22)
            if "ld_x" in args:
                kw["ld_x"] = 32
        assert call(*{**args, **wide, **kw}.values()) == _lib.ERR_SHAPE, name
    for call in (_lib.lib().sgmv_mx_quantize, _lib.lib().sgmv_mx_dequantize):
        assert call(None, 1, X, X << 4, X << 8, 256, 1 << 29, 256) == _lib.ERR_SHAPE
