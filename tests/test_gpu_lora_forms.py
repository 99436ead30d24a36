"""The adapters' kernels where many rows make blocks go through several columns
each, and ranks between the powers of two."""
import pytest
import torch

from test_gpu_lora import _by_row, _gen, _ids, _want, _want_grads, _whole, test_add, test_add_exact, test_gradients, test_gradients_exact

pytestmark = pytest.mark.gpu

for _name in ("test_add", "test_add_exact", "test_gradients", "test_gradients_exact"):      # run here by others' cases alone
    globals()["check" + _name[4:]] = globals().pop(_name)


def _loops(rows, r, N, dtype, cus):
    """Whether the second product of a call with so many sorted rows goes through its columns in a loop"""
    blocks = rows // 32
    alone = r > 64 or blocks > cus + cus // 16              # the products are not in one launch
    groups = blocks if dtype is torch.float32 else -(-blocks // 2)
    return alone and groups * -(-N // 256) >= 2 * (1 if r > 64 else 2) * cus


# T, E, r, K, N: bf16 results take 64 rows a block, which then have two adapters, or rows of padding
LOOPS = [(9200, 9, 16, 64, 2056), (9200, 60, 32, 72, 2048), (9200, 60, 40, 64, 2048), (9216, 1, 64, 64, 2048), (4200, 7, 72, 64, 2048),
         (4200, 40, 120, 64, 2056), (4200, 5, 128, 2048, 2048), (4224, 2, 96, 64, 2176)]


@pytest.mark.parametrize("T,E,r,K,N", LOOPS)
def test_columns_in_loops(mx, T, E, r, K, N):
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    rows = mx.route_tables(_ids(T, E, T).view(-1, 1), E).row_token.numel()
    for dtype in (torch.bfloat16, torch.float32):
        assert _loops(rows, r, N, dtype, cus)
        check_add_exact(mx, T, E, r, K, N, dtype)
    check_gradients_exact(mx, T, E, r, N, K)                # d_x has K columns
    check_gradients_exact(mx, T, E, r, K, N)


@pytest.mark.parametrize("T,E,r,K,N", [LOOPS[1], LOOPS[5]])
def test_columns_in_loops_real_values(mx, T, E, r, K, N):
    check_add(mx, T, E, r, K, N)
    check_gradients(mx, T, E, r, N, K)


def test_whole_blocks_in_loops(mx):
    """Every row has a token, two adapters with whole blocks each: nothing is masked.  Strided y."""
    T, E, r, K, N = 9280, 2, 48, 64, 2048
    g = _gen(1)
    ids = (torch.arange(T, device="cuda") >= 4640).to(torch.int32)          # 145 blocks of 32: the 73rd pair has both
    tables = mx.route_tables(ids.view(-1, 1), E)
    tables = mx.RouteTables(tables.offsets, tables.counts, tables.row_token[:T], tables.pair_row, tables.pad)
    assert bool((tables.row_token >= 0).all()) and int(tables.offsets[-1]) == T
    x, a, b = _whole((T, K), g, 1), _whole((E, r, K), g, 1), _whole((E, N, r), g, 1)
    for dtype in (torch.bfloat16, torch.float32):
        wide = _whole((T, N + 24), g, 4, dtype)
        before = wide.clone()
        want, h, _, _ = _want(wide[:, 8:8 + N].contiguous(), x, a, b, ids, None)
        hidden = mx.lora_add_(wide[:, 8:8 + N], x, a, b, tables, keep_hidden=True)
        assert torch.equal(hidden.double(), _by_row(h, tables.row_token))
        before[:, 8:8 + N] = want.to(dtype)
        assert torch.equal(wide, before)


@pytest.mark.parametrize("r", [72, 80, 104, 120])
def test_ranks_between(mx, r):
    for T, E, K, N in ((33, 2, 96, 136), (500, 4, 264, 320)):
        for dtype in (torch.bfloat16, torch.float32):
            check_add_exact(mx, T, E, r, K, N, dtype)
        check_add(mx, T, E, r, K, N)
        check_gradients_exact(mx, T, E, r, K, N)
        check_gradients(mx, T, E, r, K, N)
