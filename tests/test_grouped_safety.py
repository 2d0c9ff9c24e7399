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
